// ffn_bwd.cu -- backward pass of the grouped SwiGLU expert FFN with its dispatch and combine,
// on the 5th-generation tensor cores, from kept token rows (bf16, or an 8-bit checkpoint).
//
// For the pair r = (token t, slot j) of expert e, x = X[t], d = dY[t], w = topk_w[t, j]:
//   g = x W1, u = x W3, p = d W2^T, s = sigmoid(g), h = g s u
//   d topk_w[t, j] = <p, h>
//   dg = w p u s (1 + g (1 - s)),  du = w p g s,  hw = w h
//   dX[t] = sum_j (dg W1^T + du W3^T)_(t,j)
//   dW1 = X^T dg, dW3 = X^T du, dW2 = hw^T dY        (sums over the expert's rows)
// Nothing of the forward pass is kept but X: g and u are computed again.  The slot weight is
// applied after the product with W2, so <p, h> needs no expert output.
//
// Launches, in stream order:
//   plan     padded row offsets of the groups (multiples of 64 rows), offsets checked (few tokens:
//            within gather)
//   gather   the rows of X (taken back from 8 bits) and dY in padded group order, bf16; the
//            rows up to the next multiple of 64 are zeros, so no product needs a mask
//   products one persistent launch over a list of units:
//     gates   a tile of 256 columns of I x up to 256 token rows: p, u and g one after the other
//             in tensor memory, the formulas above in the epilogue; dg, du, hw (bf16, in blocks
//             of 64 token rows: [rows / 64][I][64]) and partial sums of <p, h>
//     rows    dg W1^T + du W3^T: tiles of 256 columns of H x up to 256 token rows, fp32
//     dW1, dW3, dW2   tiles of 256 x 256, the expert's padded rows as the depth
//   finish   dX and d topk_w: sums over the slots, over the partials, in a fixed order
// No atomics on results: they repeat bit for bit.
//
// Rounding.  dg, du and hw are operands of bf16 products and are rounded to bf16 once each; the
// rows of dX stay fp32 until their sum over the slots is rounded.  (Stored in bf16, they would
// add a third rounding to dX's two.)
//
// d topk_w is fp32, and the tensor core's sums are not quite: at every MMA (16 products) it cuts
// the sum towards zero, so that a sum of n MMAs comes out 1 to 4 n 2^-26 short (7e-6 at a depth of
// 7168, 3e-5 where all terms have one sign), and <p, h> inherits that three times.  The sums of p, u and g therefore leave
// tensor memory every few stages and are continued in fp32 registers (two buffers in turn):
// d topk_w is then off by 0.3 to 1.0e-6 (2-norm), and a batch of 4096 tokens takes 6.0 ms; without,
// 1.3e-5 and 5.7 ms.
//
// Tiles.  Clusters of two CTAs issue 2-SM MMAs of M = 256: the weights' columns (or rows) are the
// MMA's rows, the token rows its columns, N = 64 .. 256, so a group's last tile costs what it
// holds.  (Token rows as M, in tiles of 256, multiplied 11% more zeros at 1024 rows a group.)
// The epilogue of the gates has a row of I per lane and token rows in its registers: dg, du and
// hw are stored as they lie there, and read as MN- or K-major operands.
// Roles per CTA: warp 0 TMA producer (5 stages of 32 KB), warp 1 MMA issuer (even CTA), warp 2
// claims units (even CTA), warps 4..11 epilogue (two per lane quarter, each half of the
// columns).  A weight gradient's tiles are stored by TMA from 4 KB slabs: whole 128-byte lines.
// (Plain 16-byte stores of rows: 1.55 ms for rows and weight gradients of 32 tokens, slabs 0.94.)
//
// What bounds it.  Many rows an expert: the tensor cores (19 experts of 1024 rows, 7168 x 2048:
// 1615 TFLOP/s in this launch; measured peak 1936 in a burst, 1713 sustained).  Few rows: memory
// -- the gates stream the weights at 6.9 TB/s, the weight gradients are written at 4.5 TB/s (a
// plain fill reaches 4.0), W1 and W3 are read twice.
//
// Every wait is bounded as in ffn_tc.cu (MOE_ERR_DEVICE_TIMEOUT in the status word).
#include <cuda.h>

#include <cstring>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int PADR = 64;                  // groups start at multiples of this many rows
constexpr int TM = 256, TN = 256;         // tile of a cluster (TN: at most)
constexpr int BK = 64;                    // depth of a stage
constexpr int N_EPI = 8;                  // epilogue warps
constexpr int CLAIM_WARP = 2;
constexpr int EPI0 = 4;                   // first epilogue warp (its warpgroup's start)
constexpr int NT = 32 * (EPI0 + N_EPI);
// Registers: 384 threads launch with 168 each; the first warpgroup hands its share on
// (128 x 88 + 256 x 208 = 384 x 168) for the sums that an epilogue thread holds.
constexpr int REGS_FEW = 88, REGS_MANY = 208;
constexpr int MAXG = 1024;
constexpr int HALF = 8192;                // one 64 x 64 bf16 box
constexpr int STAGE = 4 * HALF;           // A: 128 of the tile's rows; B: 128 of its columns
constexpr int STAGES = 5;
constexpr int SLAB = 8192;                // an epilogue warp's store buffer
constexpr int TQ = 4;                     // slots that hand claimed units to the roles
constexpr int AHEAD = 24;                 // stages left to load of a unit when the next one is claimed
// Stages of one sum in tensor memory in the products that d topk_w comes from (see above): a
// token row from an 8-bit checkpoint makes shorter products, which lose less.
constexpr int CHUNK_E4M3 = 8, CHUNK_BF16 = 6;
constexpr int STASH = 32 * N_EPI * 2 * 128;   // floats of a CTA's stash: p and u of a unit

// What the plan kernel leaves in the workspace.
struct Plan {
    int *ok;        // 1: offsets valid
    int *cnt;       // [E] rows
    int *src;       // [E] first row in the caller's order
    int *pos;       // [E + 1] first padded row
    int *tiles;     // [E + 1] 256-row tiles before the group
    int *ready;     // [E] epilogue warps that are done with a unit of the group (zeroed)
    int *next;      // the next unit to be claimed (zeroed)
};

struct GemmArgs {
    // loads: rows of X and dY in boxes of 128 and of 32; those, the weights and blocks of dg, du
    // and hw ([rows / 64][I][64]) in boxes of 64 x 64
    CUtensorMap x128, d128, x32, d32, xb, db, gb, ub, hb, w1, w3, w2;
    // stores: dg, du, hw (32 token rows x 32 of I), rows of dX (32 fp32 x 32), weight gradients
    CUtensorMap gs, us, hs, xs, s1, s3, s2;
    Plan plan;
    int E, H, I, chunk;
    const float *wrow;               // [padded rows] slot weights
    float *dwp;                      // [I / 32][padded rows] partial sums of <p, h>
    long long ld_dwp;
    float *stash;                    // [CTAs][STASH]
    int *status;
    unsigned long long timeout_ns;
    int inject;
};

__device__ __forceinline__ int pad_rows(int m) { return (m + PADR - 1) & ~(PADR - 1); }

__device__ __forceinline__ float fast_sigmoid(float g)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + __expf(-g)));
    return r;
}

// ----------------------------------------------------------------------------- plan
// By a whole CTA: rows, first row and first padded row of each group to cnt, src and pos, and with
// `out` the rest of the plan; whether the offsets are valid (cnt is 0 throughout if not).
__device__ __forceinline__ bool plan_groups(const int32_t *__restrict__ offsets, int E, int rows, const Plan &p,
                                            bool out, int *cnt, int *src, int *pos, int *status)
{
    __shared__ int a[32], b[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (E + blockDim.x - 1) / blockDim.x, g0 = threadIdx.x * per, g1 = min(E, g0 + per);
    int bad = 0;
    for (int g = g0; g < g1; ++g) {
        const int lo = offsets[g], hi = offsets[g + 1];
        bad |= lo < 0 || hi < lo || hi > rows;
        src[g] = lo;
        cnt[g] = hi - lo;
    }
    const bool ok = !__syncthreads_or(bad);
    int np = 0, nt = 0;
    for (int g = g0; g < g1; ++g) {
        if (!ok) cnt[g] = 0;
        np += pad_rows(cnt[g]);
        nt += (cnt[g] + TM - 1) / TM;
    }
    int ip = np, it = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int vp = __shfl_up_sync(kFullMask, ip, o), vt = __shfl_up_sync(kFullMask, it, o);
        if (lane >= o) { ip += vp; it += vt; }
    }
    if (lane == 31) { a[warp] = ip; b[warp] = it; }
    __syncthreads();
    for (int w = 0; w < warp; ++w) { ip += a[w]; it += b[w]; }
    if (out && g0 < g1 && g1 == E) {
        p.pos[E] = ip;
        p.tiles[E] = it;
    }
    ip -= np;
    it -= nt;
    for (int g = g0; g < g1; ++g) {
        pos[g] = ip;
        if (out) {
            p.cnt[g] = cnt[g];
            p.src[g] = src[g];
            p.pos[g] = ip;
            p.tiles[g] = it;
            p.ready[g] = 0;
        }
        ip += pad_rows(cnt[g]);
        it += (cnt[g] + TM - 1) / TM;
    }
    if (out && threadIdx.x == 0) {
        *p.ok = ok ? 1 : 0;
        *p.next = 0;
        if (!ok) report(status, MOE_ERR_INVALID_ARG);
    }
    return ok;
}

__global__ void __launch_bounds__(1024) plan_kernel(const int32_t *__restrict__ offsets, int E, int rows,
                                                    Plan p, int *status)
{
    pdl_wait();
    plan_groups(offsets, E, rows, p, true, p.cnt, p.src, p.pos, status);
}

// --------------------------------------------------------------------------- gather
// CTA (t, y) of the first T: token t's row, columns of part y, to the padded rows of its
// slots.  CTA (T + g, y): the zero rows at the end of group g.
constexpr int GT = 128;
constexpr int GCOLS = GT * 8;
// With at most this many CTAs each makes the plan for itself (PLAN), which saves a launch; the
// first of them leaves it to the products.
// (16 x 256, 16 experts: 27.5 us with the launch, 25.9 without; 1000 tokens 36.3 and 34.5; 2000
// tokens, 2016 CTAs, 39.8 and 40.0; 1024 experts 148.8 and 150.5.)
constexpr unsigned PLAN_CTAS = 1024;
constexpr int PLAN_E = 256;

template <bool PLAN>
__global__ void __launch_bounds__(GT) gather_kernel(const void *__restrict__ x, const int8_t *__restrict__ xs,
                                                    const uint16_t *__restrict__ dY,
                                                    const int32_t *__restrict__ offsets,
                                                    const int32_t *__restrict__ slot_pos,
                                                    const float *__restrict__ topk_w, int T, int H, int E,
                                                    int K, Plan p, uint16_t *__restrict__ X,
                                                    uint16_t *__restrict__ D, float *__restrict__ wrow,
                                                    int *__restrict__ prow, int *__restrict__ status)
{
    __shared__ int dst[32];
    __shared__ int own[PLAN ? 3 * PLAN_E : 1];
    pdl_wait();
    const int *cnt = p.cnt, *src = p.src, *pos = p.pos;
    if (PLAN) {
        int *c = own, *f = own + PLAN_E, *q = own + 2 * PLAN_E;
        if (!plan_groups(offsets, E, T * K, p, (blockIdx.x | blockIdx.y) == 0, c, f, q, status)) return;
        __syncthreads();
        cnt = c; src = f; pos = q;
    } else if (!*p.ok) {
        return;
    }
    const int c = blockIdx.y * GCOLS + threadIdx.x * 8;
    if (blockIdx.x >= static_cast<unsigned>(T)) {
        const int g = blockIdx.x - T;
        const int m = cnt[g], n = pad_rows(m);
        for (int r = m; r < n; ++r) {
            const size_t row = static_cast<size_t>(pos[g] + r);
            if (c < H) {
                *reinterpret_cast<uint4 *>(X + row * H + c) = make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4 *>(D + row * H + c) = make_uint4(0, 0, 0, 0);
            }
            if (blockIdx.y == 0 && threadIdx.x == 0) wrow[row] = 0.f;
        }
        return;
    }
    const int t = blockIdx.x;
    if (threadIdx.x < K) {
        const size_t pair = static_cast<size_t>(t) * K + threadIdx.x;
        const int r = slot_pos[pair];
        int q = -1;
        if (r >= 0 && r < src[E - 1] + cnt[E - 1]) {
            int lo = 0, hi = E - 1;        // last group whose first row is <= r
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (src[mid] <= r) lo = mid; else hi = mid - 1;
            }
            const int k = r - src[lo];
            if (k >= 0 && k < cnt[lo]) q = pos[lo] + k;
        }
        dst[threadIdx.x] = q;
        if (blockIdx.y == 0) {
            prow[pair] = q;
            if (q >= 0) wrow[q] = topk_w ? topk_w[pair] : 1.f;
        }
    }
    __syncthreads();
    if (c >= H) return;
    const size_t off = static_cast<size_t>(t) * H + c;
    uint4 v;
    if (xs) {
        const int nb = (H + 127) / 128;
        v = e4m3x8_to_bf16x8(*reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(x) + off),
                             pow2f(xs[static_cast<size_t>(t) * nb + c / 128]));
    } else {
        v = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(x) + off);
    }
    const uint4 d = *reinterpret_cast<const uint4 *>(dY + off);
    for (int j = 0; j < K; ++j) {
        if (dst[j] < 0) continue;
        const size_t row = static_cast<size_t>(dst[j]) * H + c;
        *reinterpret_cast<uint4 *>(X + row) = v;
        *reinterpret_cast<uint4 *>(D + row) = d;
    }
}

// ------------------------------------------------------------------------- products
enum { P, U, G, ROWS, DW1, DW3, DW2 };     // p, u, g; rows of dX; weight gradients

// What a cluster claims at a time: a tile's three products (P, U, G), or a run of tiles of one
// kind side by side (ROWS along H, weight gradients along their columns).
struct Unit {
    int kind, g;
    int row0;       // P, ROWS: first padded row of the tile's token rows (its columns); weight
                    // gradients: first padded row of the group (the depth)
    int m0;         // first row of the first tile: of I (P, U, G), H (ROWS), the gradient
    int n0, n;      // columns in the group, columns of a tile; weight gradients: first column, -
    int kb;         // stages of a tile
    int parts;      // tiles
};
constexpr int RUN_DW = 4;     // weight-gradient tiles of a unit at most

struct Tile { int kind, m0, n0, n; };

__device__ __forceinline__ void tma_store_2d(const void *tmap, const void *src, int c0, int c1)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];"
                 ::"l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(smem_u32(src)) : "memory");
}

__device__ __forceinline__ void tma_store_3d(const void *tmap, const void *src, int c0, int c1, int c2)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];"
                 ::"l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(src)) : "memory");
}

// The warp's slab may be written again: the stores before it have read it.
__device__ __forceinline__ void slab_free(int lane)
{
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
}

// The slab is written: order it before the store that lane 0 issues next.
__device__ __forceinline__ void slab_ready()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
}

__device__ __forceinline__ void slab_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }

// 32 fp32 -> 32 bf16 of the lane's row of 64, from chunk c0 (of 8), in the 128-byte swizzle
__device__ __forceinline__ void slab_bf16(unsigned char *slab, int lane, const float (&v)[32], int c0)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4 *>(slab + lane * 128 + (((c0 + i) ^ (lane & 7)) << 4)) =
            make_uint4(f32x2_to_bf16x2(v[8 * i + 1], v[8 * i]), f32x2_to_bf16x2(v[8 * i + 3], v[8 * i + 2]),
                       f32x2_to_bf16x2(v[8 * i + 5], v[8 * i + 4]), f32x2_to_bf16x2(v[8 * i + 7], v[8 * i + 6]));
}

// 16 bytes to chunk c (of 4) of the lane's row of 64 bytes, in the 64-byte swizzle
__device__ __forceinline__ void slab_row64(unsigned char *slab, int lane, int c, uint4 v)
{
    *reinterpret_cast<uint4 *>(slab + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) = v;
}

__device__ __forceinline__ int ld_acquire(const int *p)
{
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ void fence_proxy_async_global()
{
    asm volatile("fence.proxy.async.global;" ::: "memory");
}

__global__ void __launch_bounds__(NT, 1) bwd_gemm_kernel(const __grid_constant__ GemmArgs p)
{
    constexpr int TCOLS = 512;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *ring = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char *slabs = ring + STAGES * STAGE;
    __shared__ uint64_t full[STAGES], empty[STAGES], tfull[2], tempty[2], tqf[TQ], tqe[TQ], want, drain;
    __shared__ int tq[TQ][8];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_s;
    volatile int *abort_flag = &abort_s;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const uint64_t tmo = p.timeout_ns;
    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 2 * N_EPI);
        }
        for (int q = 0; q < TQ; ++q) {
            mbar_init(&tqf[q], 1);
            mbar_init(&tqe[q], 2 * N_EPI + 3);   // both epilogues and producers, the MMA issuer
        }
        mbar_init(&want, 1);
        mbar_init(&drain, 1);
        abort_s = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(&tmem_slot, TCOLS);
        tmem_relinquish_pair();
    }
    pdl_wait();
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    const int E = p.E, H = p.H, I = p.I;
    const int ok = *p.plan.ok;
    const int row_tiles = ok ? p.plan.tiles[E] : 0;
    const int nI = (I + TM - 1) / TM, nH = (H + TM - 1) / TM;
    // units of a group beside its gates: ROWS per tile of token rows, DW1 or DW3, DW2
    const int rr = max(1, min(8, 32 / (I / BK)));    // H tiles of a ROWS unit
    const int u_rows = (nH + rr - 1) / rr;
    const int r13 = (nI + RUN_DW - 1) / RUN_DW, r2 = (nH + RUN_DW - 1) / RUN_DW;
    const int u_dw13 = nH * r13, u_dw = 2 * u_dw13 + nI * r2;
    const int n_gates = row_tiles * nI;
    const int n_units = ok ? n_gates + row_tiles * u_rows + E * u_dw : 0;

    // Unit `t` of the list; from: a group at or before its own (the search starts there).
    auto decode = [&](int t, int &from) -> Unit {
        Unit T{};
        const bool gates = t < n_gates;
        const int v = gates ? t : t - n_gates;
        const int nr = gates ? nI : u_rows, nw = gates ? 0 : u_dw;
        auto first = [&](int g) -> int { return p.plan.tiles[g] * nr + g * nw; };   // units before group g
        int lo = from;
        if (first(lo) > v) lo = 0;
        int near = 0;
        while (near < 8 && first(lo + 1) <= v) { ++lo; ++near; }
        if (near == 8) {
            int hi = E - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (first(mid) <= v) lo = mid; else hi = mid - 1;
            }
        }
        from = lo;
        T.g = lo;
        T.row0 = p.plan.pos[lo];
        const int rows = pad_rows(p.plan.cnt[lo]);
        int l = v - first(lo);
        const int mt = (rows + TN - 1) / TN;         // tiles of token rows, innermost: they share the weights
        if (l < mt * nr) {
            const int c = l / mt, m = l - c * mt;
            T.row0 += m * TN;
            T.n0 = min(TN, rows - m * TN);
            T.n = T.n0 == 192 ? 256 : T.n0;          // (its halves: whole blocks of 64, or half of one)
            if (gates) {
                T.kind = P;
                T.m0 = c * TM;
                T.kb = H / BK;
                T.parts = 3;
            } else {
                T.kind = ROWS;
                T.m0 = c * rr * TM;
                T.kb = 2 * (I / BK);
                T.parts = min(rr, nH - c * rr);
            }
        } else {
            l -= mt * nr;
            int w = 0;
            while (w < 2 && l >= u_dw13) { l -= u_dw13; ++w; }
            const int nc = w < 2 ? nI : nH, runs = w < 2 ? r13 : r2;
            const int m = l / runs, c = (l - m * runs) * RUN_DW;
            T.kind = DW1 + w;
            T.m0 = m * TM;
            T.n0 = c * TN;
            T.kb = rows / BK;
            T.parts = min(RUN_DW, nc - c);
        }
        return T;
    };
    auto tile_of = [&](const Unit &u, int part) -> Tile {
        Tile T{u.kind, u.m0, u.n0, u.n};
        if (u.kind == P) T.kind = P + part;
        else if (u.kind == ROWS) T.m0 += part * TM;
        else {
            T.n0 += part * TN;
            T.n = min(TN, (u.kind == DW2 ? H : I) - T.n0);
        }
        return T;
    };
    auto slot_read = [&](int q) -> Unit {
        const int *e = tq[q];
        return Unit{e[0], e[1], e[2], e[3], e[4], e[5], e[6], e[7]};
    };
    // Units are claimed from a counter by a warp of the even CTA, in order, and handed to every
    // role of both CTAs through TQ slots (kind -1 ends): the counter's round trip and the search
    // for the group stay off the producer's thread, whose pause empties the ring.  A unit is
    // claimed when the one before it has AHEAD stages left to load: claimed as early as the slots
    // allow, a few units would go to the first clusters alone (one expert of 7168 x 2048, one
    // token: 176 us, now 161).  All of a group's gates come
    // before the tiles that need them, so a cluster that waits holds nothing they need.
    auto slot_done = [&](int q) {
        if (leader) mbar_arrive(&tqe[q]);
        else mbar_arrive_cluster(mapa_shared(smem_u32(&tqe[q]), 0));
    };

    if (warp < EPI0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_FEW));
    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0 && !p.inject) {
            uint32_t s = 0, ph = 0, it = 0, qs = 0, qph = 0;
            const uint32_t full0 = mapa_shared(smem_u32(full), 0);
            const int r = static_cast<int>(rank);
            bool good = true;
            while (good) {
                if (!mbar_wait_cluster(&tqf[qs], qph, abort_flag, p.status, tmo)) break;
                const Unit u = slot_read(qs);
                slot_done(qs);
                if (++qs == TQ) { qs = 0; qph ^= 1u; }
                if (u.kind < 0) break;
                if (u.kind >= ROWS && u.kb > 0) {
                    // dg, du and hw of the group: every epilogue warp of its units is done
                    const int need = (p.plan.tiles[u.g + 1] - p.plan.tiles[u.g]) * nI * 2 * N_EPI;
                    const int *flag = p.plan.ready + u.g;
                    if (ld_acquire(flag) < need) {
                        const uint64_t t0 = globaltimer_ns();
                        while (ld_acquire(flag) < need) {
                            if (*abort_flag) { good = false; break; }
                            if (globaltimer_ns() - t0 > tmo) {
                                *abort_flag = 1;
                                report(p.status, MOE_ERR_DEVICE_TIMEOUT);
                                good = false;
                                break;
                            }
                            __nanosleep(64);
                        }
                        if (!good) break;
                    }
                    fence_proxy_async_global();
                }
                int left = u.parts * u.kb;           // stages
                bool asked = !leader;
                if (!asked && left <= AHEAD) { mbar_arrive(&want); asked = true; }
                for (int part = 0; part < u.parts && good; ++part) {
                    const Tile T = tile_of(u, part);
                    const int nb = T.n / 2;          // this CTA's columns
                    const bool boxes = T.kind >= ROWS;   // B in boxes of 64 x 64
                    const uint32_t bytes = 2 * HALF + (boxes ? (nb > 64 ? 2 : 1) * HALF : nb * 128);
                    const int m = T.m0 + 128 * r;
                    const int n = (T.kind >= DW1 ? T.n0 : u.row0) + nb * r;
                    for (int kb = 0; kb < u.kb; ++kb, ++it) {
                        if (!mbar_wait(&empty[s], ph ^ 1u, abort_flag, p.status, tmo)) { good = false; break; }
                        unsigned char *a = ring + s * STAGE, *b = a + 2 * HALF;
                        const uint32_t fb = full0 + 8u * s;
                        if (leader) mbar_arrive_expect_tx(&full[s], 2u * bytes);
                        int k = kb * BK;
                        if (T.kind < ROWS) {
                            if (T.kind == P) {           // rows of W2
                                tma_load_3d_pair(a, &p.w2, fb, k, m, u.g);
                                tma_load_3d_pair(a + HALF, &p.w2, fb, k, m + 64, u.g);
                            } else {                     // columns of W3, W1
                                const CUtensorMap *wm = T.kind == U ? &p.w3 : &p.w1;
                                tma_load_3d_pair(a, wm, fb, m, k, u.g);
                                tma_load_3d_pair(a + HALF, wm, fb, m + 64, k, u.g);
                            }
                            if (nb == 128) {
                                tma_load_2d_pair(b, T.kind == P ? &p.d128 : &p.x128, fb, k, n);
                            } else {
                                const CUtensorMap *bm = T.kind == P ? &p.d32 : &p.x32;
                                for (int j = 0; j < nb; j += 32) tma_load_2d_pair(b + j * 128, bm, fb, k, n + j);
                            }
                        } else if (T.kind == ROWS) {     // rows of W1, then of W3; dg, then du
                            const bool second = k >= I;
                            if (second) k -= I;
                            const CUtensorMap *wm = second ? &p.w3 : &p.w1, *bm = second ? &p.ub : &p.gb;
                            tma_load_3d_pair(a, wm, fb, k, m, u.g);
                            tma_load_3d_pair(a + HALF, wm, fb, k, m + 64, u.g);
                            tma_load_3d_pair(b, bm, fb, n & 63, k, n >> 6);
                            if (nb > 64) tma_load_3d_pair(b + HALF, bm, fb, 0, k, (n >> 6) + 1);
                        } else {
                            k += u.row0;
                            if (T.kind == DW2) {         // hw as it lies; columns of dY
                                tma_load_3d_pair(a, &p.hb, fb, 0, m, k >> 6);
                                tma_load_3d_pair(a + HALF, &p.hb, fb, 0, m + 64, k >> 6);
                                tma_load_2d_pair(b, &p.db, fb, n, k);
                                if (nb > 64) tma_load_2d_pair(b + HALF, &p.db, fb, n + 64, k);
                            } else {                     // columns of X; dg or du as it lies
                                const CUtensorMap *bm = T.kind == DW3 ? &p.ub : &p.gb;
                                tma_load_2d_pair(a, &p.xb, fb, m, k);
                                tma_load_2d_pair(a + HALF, &p.xb, fb, m + 64, k);
                                tma_load_3d_pair(b, bm, fb, 0, n, k >> 6);
                                if (nb > 64) tma_load_3d_pair(b + HALF, bm, fb, 0, n + 64, k >> 6);
                            }
                        }
                        if (++s == STAGES) { s = 0; ph ^= 1u; }
                        if (--left <= AHEAD && !asked) { mbar_arrive(&want); asked = true; }
                    }
                }
            }
            // Every copy issued lands before the CTAs can exit: the even CTA's barriers count both
            // CTAs' copies.  After a wait that ran out the odd CTA may have issued stages that the
            // even one has not, whose barriers then say nothing: it stays as long as the even one
            // waits for a stage at most.
            if (!leader && *abort_flag) {
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 20000000ull) __nanosleep(1000);
            }
            if (leader) {
                const uint32_t n = it < STAGES ? it : STAGES;
                for (uint32_t j = it - n; j < it; ++j) {
                    int dummy = 0;
                    mbar_wait(&full[j % STAGES], (j / STAGES) & 1u, &dummy, nullptr, 20000000ull);
                }
            }
        }
    } else if (warp == 1) {
        // -------------------------------------------------------------- MMA issuer
        if (lane == 0 && leader) {
            const uint32_t ring0 = smem_u32(ring);
            uint32_t s = 0, ph = 0, b = 0, tph = 0, qs = 0, qph = 0;
            bool good = true;
            while (good) {
                if (!mbar_wait(&tqf[qs], qph, abort_flag, p.status, tmo)) break;
                const Unit un = slot_read(qs);
                slot_done(qs);
                if (++qs == TQ) { qs = 0; qph ^= 1u; }
                if (un.kind < 0) break;
                const int chunk = un.kind == P ? p.chunk : un.kb;
                for (int part = 0; part < un.parts && good; ++part) {
                    const Tile T = tile_of(un, part);
                    // MN-major where the operand lies with the tile's rows (columns) contiguous
                    const bool amn = T.kind == U || T.kind == G || T.kind == DW1 || T.kind == DW3;
                    const bool bmn = T.kind == ROWS || T.kind == DW2;
                    const uint64_t ad0 = smem_desc_sw128(ring0, amn ? HALF : 16, 1024);
                    const uint64_t bd0 = smem_desc_sw128(ring0 + 2 * HALF, bmn ? HALF : 16, 1024);
                    const uint32_t as = amn ? 128u : 2u, bs = bmn ? 128u : 2u;
                    const uint32_t id = idesc_bf16_f32(TM, static_cast<uint32_t>(T.n), amn, bmn);
                    int kb = 0;
                    do {
                        // (what this orders is tensor memory, by the tcgen05 fences on both
                        // sides: an acquire of wider scope, 3.24 instead of 3.13 ms for 19 x
                        // 1024 rows, would add nothing)
                        if (!mbar_wait(&tempty[b], tph ^ 1u, abort_flag, p.status, tmo)) { good = false; break; }
                        tc_fence_after();
                        const uint32_t d = tmem + b * TN;
                        const int end = min(kb + chunk, un.kb);
                        for (int k0 = kb; kb < end; ++kb) {
                            if (!mbar_wait(&full[s], ph, abort_flag, p.status, tmo)) { good = false; break; }
                            tc_fence_after();
                            const uint64_t o = static_cast<uint64_t>(s * (STAGE >> 4));
                            const uint64_t ad = ad0 + o, bd = bd0 + o;
                            tc_mma_bf16_pair(d, ad, bd, id, kb > k0 ? 1u : 0u);
                            tc_mma_bf16_pair(d, ad + as, bd + bs, id, 1u);
                            tc_mma_bf16_pair(d, ad + 2 * as, bd + 2 * bs, id, 1u);
                            tc_mma_bf16_pair(d, ad + 3 * as, bd + 3 * bs, id, 1u);
                            tc_commit_pair_mc(&empty[s], 3);
                            if (++s == STAGES) { s = 0; ph ^= 1u; }
                        }
                        if (!good) break;
                        tc_commit_pair_mc(&tfull[b], 3);
                        b ^= 1u;
                        if (b == 0) tph ^= 1u;
                    } while (kb < un.kb);
                }
            }
            tc_commit_pair_mc(&drain, 1);
            int dummy = 0;
            mbar_wait(&drain, 0, &dummy, nullptr, 20000000ull);
        }
    } else if (warp == CLAIM_WARP) {
        // ------------------------------------------------------------------ claims
        if (lane == 0 && leader) {
            uint32_t qs = 0, qph = 0;
            uint32_t wph = 1;                        // (the first claim waits for nothing)
            int from = 0;
            int t = 0;
            do {
                if (!mbar_wait(&want, wph, abort_flag, p.status, tmo)) break;
                wph ^= 1u;
                if (!mbar_wait_cluster(&tqe[qs], qph ^ 1u, abort_flag, p.status, tmo)) break;
                t = atomicAdd(p.plan.next, 1);
                Unit u{};
                if (t < n_units) u = decode(t, from);
                else u.kind = -1;
                const int vals[8] = {u.kind, u.g, u.row0, u.m0, u.n0, u.n, u.kb, u.parts};
                const uint32_t other = mapa_shared(smem_u32(tq[qs]), 1);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    tq[qs][j] = vals[j];
                    st_shared_cluster(other + 4u * j, vals[j]);
                }
                mbar_arrive(&tqf[qs]);
                mbar_arrive_cluster(mapa_shared(smem_u32(&tqf[qs]), 1));
                if (++qs == TQ) { qs = 0; qph ^= 1u; }
            } while (t < n_units);
        }
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_MANY));
        // ---------------------------------------------------------------- epilogue
        const int q = warp & 3, half = (warp - EPI0) >> 2;   // lane quarter, half of the columns
        const uint32_t tm0 = tmem + (static_cast<uint32_t>(32 * q) << 16);
        const uint32_t tempty0 = mapa_shared(smem_u32(tempty), 0);
        const int r0 = 128 * static_cast<int>(rank) + 32 * q;   // the warp's first row of a tile
        unsigned char *slab = slabs + (warp - EPI0) * SLAB;
        uint32_t b = 0, tph = 0, qs = 0, qph = 0;
        // a wait by one lane (every lane then observes the phase itself)
        auto wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {
            bool good = true;
            if (lane == 0) good = mbar_wait_cluster(bar, parity, abort_flag, p.status, tmo);
            good = __shfl_sync(kFullMask, good, 0);
            if (good) mbar_try_wait_cluster(bar, parity);
            return good;
        };
        auto sums_ready = [&]() -> bool {
            bool good = true;
            if (lane == 0) good = mbar_wait(&tfull[b], tph, abort_flag, p.status, tmo);
            good = __shfl_sync(kFullMask, good, 0);
            if (good) mbar_try_wait(&tfull[b], tph);
            tc_fence_after();
            return good;
        };
        auto sums_read = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(tempty0 + 8u * b);
            b ^= 1u;
            if (b == 0) tph ^= 1u;
        };
        // the slab's halves in turn: the store before the last has read its own
        uint32_t turn = 0;
        auto slab_turn = [&](int ln) -> unsigned char * {
            if (ln == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
            __syncwarp();
            turn ^= 1u;
            return slab + (turn ? SLAB / 2 : 0);
        };
        // this thread's stash: p, then u, of its row, float4 i at i * SROW (256 threads side by side)
        float4 *stash = reinterpret_cast<float4 *>(p.stash + static_cast<size_t>(blockIdx.x) * STASH) + (tid - 32 * EPI0);
        constexpr int SROW = 32 * N_EPI;
        bool good = true;
        while (good) {
            if (!wait_all(&tqf[qs], qph)) break;
            const Unit u = slot_read(qs);
            __syncwarp();
            if (lane == 0) slot_done(qs);
            if (++qs == TQ) { qs = 0; qph ^= 1u; }
            if (u.kind < 0) break;
            if (u.kind == P) {
                // 32-column pieces of this warp's half that are in the group
                const int nc = max(0, min(u.n / 2, u.n0 - half * (u.n / 2))) / 32;
                const uint32_t at = tm0 + static_cast<uint32_t>(half * (u.n / 2));
                float acc[128];                      // row i of the tile, its half of the token rows
#pragma unroll 1
                for (int part = P; part <= G; ++part) {
                    // sums over the chunks, in registers
#pragma unroll
                    for (int i = 0; i < 128; ++i) acc[i] = 0.f;
#pragma unroll 1
                    for (int kb = 0; kb < u.kb; kb += p.chunk) {
                        if (!sums_ready()) { good = false; break; }
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            if (c >= nc) continue;
                            float v[32];
                            __syncwarp();
                            tmem_ld32(at + b * TN + 32 * c, v);
#pragma unroll
                            for (int i = 0; i < 32; ++i) acc[32 * c + i] += v[i];
                        }
                        sums_read();
                    }
                    if (!good) break;
                    if (part != G) {
                        float4 *st = stash + part * 32 * SROW;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (i < 8 * nc) st[i * SROW] = make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
                    }
                }
                if (!good) break;
                // g in acc; p and u in the stash.  32 token rows at a time: dg, du, hw and the
                // terms of <p, h>
                const int col = u.m0 + r0;           // the warp's columns of I
                const int tok = u.row0 + half * (u.n / 2);
                float *dwp = p.dwp + static_cast<size_t>(col / 32) * p.ld_dwp + tok + lane;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (c >= nc) continue;
                    const float4 *wv = reinterpret_cast<const float4 *>(p.wrow + tok + 32 * c);
                    slab_free(lane);
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        uint32_t og[4], ou[4], hw[4];
#pragma unroll
                        for (int y = 0; y < 8; y += 4) {
                            const int j = i + y;
                            const float4 p4 = stash[(8 * c + j / 4) * SROW], u4 = stash[(32 + 8 * c + j / 4) * SROW], w4 = wv[j / 4];
                            const float pp[4] = {p4.x, p4.y, p4.z, p4.w}, uu[4] = {u4.x, u4.y, u4.z, u4.w};
                            const float ww[4] = {w4.x, w4.y, w4.z, w4.w};
                            float a[4], e[4], hv[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float g = acc[32 * c + j + k];
                                const float s = fast_sigmoid(g), gs = g * s, h = gs * uu[k], pw = pp[k] * ww[k];
                                a[k] = pw * uu[k] * s * fmaf(g, 1.f - s, 1.f);
                                e[k] = pw * gs;
                                hv[k] = ww[k] * h;
                                acc[32 * c + j + k] = pp[k] * h;
                            }
                            og[y / 2] = f32x2_to_bf16x2(a[1], a[0]);
                            og[y / 2 + 1] = f32x2_to_bf16x2(a[3], a[2]);
                            ou[y / 2] = f32x2_to_bf16x2(e[1], e[0]);
                            ou[y / 2 + 1] = f32x2_to_bf16x2(e[3], e[2]);
                            hw[y / 2] = f32x2_to_bf16x2(hv[1], hv[0]);
                            hw[y / 2 + 1] = f32x2_to_bf16x2(hv[3], hv[2]);
                        }
                        slab_row64(slab, lane, i / 8, make_uint4(og[0], og[1], og[2], og[3]));
                        slab_row64(slab + 2048, lane, i / 8, make_uint4(ou[0], ou[1], ou[2], ou[3]));
                        slab_row64(slab + 4096, lane, i / 8, make_uint4(hw[0], hw[1], hw[2], hw[3]));
                    }
                    slab_ready();
                    if (lane == 0 && col < I) {
                        const int t0 = tok + 32 * c;
                        tma_store_3d(&p.gs, slab, t0 & 63, col, t0 >> 6);
                        tma_store_3d(&p.us, slab + 2048, t0 & 63, col, t0 >> 6);
                        tma_store_3d(&p.hs, slab + 4096, t0 & 63, col, t0 >> 6);
                        slab_commit();
                    }
                    // sum over the warp's 32 columns of I: lane j ends up with token row j
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                        for (int k = 0; k < o; ++k) {
                            const bool up = lane & o;
                            const float send = up ? acc[32 * c + k] : acc[32 * c + k + o];
                            const float keep = up ? acc[32 * c + k + o] : acc[32 * c + k];
                            acc[32 * c + k] = keep + __shfl_xor_sync(kFullMask, send, o);
                        }
                    if (col < I) dwp[32 * c] = acc[32 * c];
                }
                // the unit's dg, du and hw are in global memory: tell the group
                if (lane == 0) {
                    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
                    fence_proxy_async_global();
                    __threadfence();
                    atomicAdd(p.plan.ready + u.g, 1);
                }
                __syncwarp();
                continue;
            }
#pragma unroll 1
            for (int part = 0; part < u.parts; ++part) {
                const Tile T = tile_of(u, part);
                if (!sums_ready()) { good = false; break; }
                if (T.kind == ROWS) {
                    const int col = T.m0 + r0, tok = u.row0 + half * (T.n / 2);
                    const uint32_t at = tm0 + b * TN + static_cast<uint32_t>(half * (T.n / 2));
#pragma unroll 1
                    for (int c = 0; c < max(0, min(T.n / 2, u.n0 - half * (T.n / 2))) / 32; ++c) {
                        float v[32];
                        __syncwarp();
                        tmem_ld32(at + 32 * c, v);
                        unsigned char *buf = slab_turn(lane);
                        float *sl = reinterpret_cast<float *>(buf);
#pragma unroll
                        for (int i = 0; i < 32; ++i) sl[i * 32 + lane] = v[i];
                        slab_ready();
                        if (lane == 0) {
                            if (col < H) tma_store_2d(&p.xs, buf, col, tok + 32 * c);
                            slab_commit();
                        }
                    }
                } else {
                    const int M = T.kind == DW2 ? I : H;
                    const CUtensorMap *sm = T.kind == DW1 ? &p.s1 : (T.kind == DW3 ? &p.s3 : &p.s2);
#pragma unroll 1
                    for (int c = 0; c < 2; ++c) {
                        const int lc = 128 * half + 64 * c;
                        if (lc >= T.n) break;
                        float v[32], y[32];
                        __syncwarp();
                        tmem_ld32(tm0 + b * TN + lc, v);
                        tmem_ld32(tm0 + b * TN + lc + 32, y);
                        if (u.kb == 0) {             // an expert without rows
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = y[i] = 0.f;
                        }
                        unsigned char *buf = slab_turn(lane);
                        slab_bf16(buf, lane, v, 0);
                        slab_bf16(buf, lane, y, 4);
                        slab_ready();
                        if (lane == 0) {
                            if (T.m0 + r0 < M) tma_store_3d(sm, buf, T.n0 + lc, T.m0 + r0, u.g);
                            slab_commit();
                        }
                    }
                }
                sums_read();
            }
        }
        // the last stores have left shared memory and reached global memory
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem, TCOLS);
    }
}

// --------------------------------------------------------------------------- finish
// CTA (t, y): dX[t] of 1024 columns (slots in order); part 0 also d topk_w, a warp a slot.
__global__ void __launch_bounds__(GT) finish_kernel(const float *__restrict__ dxp,
                                                    const int *__restrict__ prow,
                                                    const float *__restrict__ dwp, long long ld, int parts,
                                                    const int *__restrict__ ok, int H, int K,
                                                    uint16_t *__restrict__ dX, float *__restrict__ d_topk_w)
{
    __shared__ int src[32];
    pdl_wait();
    if (!*ok) return;
    const int t = blockIdx.x, lane = threadIdx.x & 31;
    if (threadIdx.x < K) src[threadIdx.x] = prow[static_cast<size_t>(t) * K + threadIdx.x];
    __syncthreads();
    if (blockIdx.y == 0 && d_topk_w) {
        for (int j = threadIdx.x >> 5; j < K; j += GT / 32) {
            float v = 0.f;
            if (src[j] >= 0)
                for (int k = lane; k < parts; k += 32) v += dwp[static_cast<size_t>(k) * ld + src[j]];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
            if (lane == 0) d_topk_w[static_cast<size_t>(t) * K + j] = v;
        }
    }
    const int c = blockIdx.y * GCOLS + threadIdx.x * 8;
    if (c >= H) return;
    float a[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = 0.f;
    for (int j = 0; j < K; ++j) {
        if (src[j] < 0) continue;
        const float4 *v = reinterpret_cast<const float4 *>(dxp + static_cast<size_t>(src[j]) * H + c);
        const float4 lo = v[0], hi = v[1];
        a[0] += lo.x; a[1] += lo.y; a[2] += lo.z; a[3] += lo.w;
        a[4] += hi.x; a[5] += hi.y; a[6] += hi.z; a[7] += hi.w;
    }
    *reinterpret_cast<uint4 *>(dX + static_cast<size_t>(t) * H + c) =
        make_uint4(f32x2_to_bf16x2(a[1], a[0]), f32x2_to_bf16x2(a[3], a[2]), f32x2_to_bf16x2(a[5], a[4]),
                   f32x2_to_bf16x2(a[7], a[6]));
}

// ------------------------------------------------------------------------ host side
using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion,
                                   CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
{
    static const EncodeTiledFn fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeTiledFn>(ptr);
        return static_cast<EncodeTiledFn>(nullptr);
    }();
    return fn;
}

// [groups][rows][cols] (groups == 0: [rows][cols]) of bf16, or fp32, in boxes of box_cols columns
// x box_rows rows: 64 bf16 in the 128-byte swizzle, 32 bf16 in the 64-byte one, 32 fp32 as they
// stand.  (A box narrower than its swizzle's span is stored from rows of the whole span: it
// would read past a slab.)
bool encode(CUtensorMap *m, const void *base, int groups, long long rows, int cols, int box_rows,
            int box_cols = 64, bool fp32 = false)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t es = fp32 ? 4 : 2;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(groups)};
    const cuuint64_t strides[2] = {cols * es, cols * es * static_cast<cuuint64_t>(rows)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, groups ? 3 : 2,
              const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              fp32 ? CU_TENSOR_MAP_SWIZZLE_NONE : (box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B),
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t al256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }

int gemm_ctas() { return num_sms() / 2 * 2; }
int dw_parts(int I) { return I / 32; }    // partial sums of <p, h>

struct Layout {
    long long rows;        // padded rows at most
    size_t plan, wrow, prow, X, D, dg, du, hw, dwp, dxp, stash, bytes;
};
Layout layout(int T, int H, int E, int K, int I)
{
    Layout L{};
    const long long TK = static_cast<long long>(T) * K;
    const long long used = TK < E ? TK : E;
    L.rows = (TK + (PADR - 1) * used + PADR - 1) / PADR * PADR;
    const size_t R = static_cast<size_t>(L.rows);
    size_t o = 0;
    auto take = [&](size_t b) { const size_t at = o; o += al256(b); return at; };
    L.plan = take((5 * (MAXG + 1) + 2) * sizeof(int));
    L.wrow = take(R * 4);
    L.prow = take(static_cast<size_t>(TK) * 4);
    L.X = take(R * H * 2);
    L.D = take(R * H * 2);
    L.dg = take(R * I * 2);
    L.du = take(R * I * 2);
    L.hw = take(R * I * 2);
    L.dwp = take(R * dw_parts(I) * 4);
    L.dxp = take(R * H * 4);
    L.stash = take(static_cast<size_t>(gemm_ctas()) * STASH * 4);
    L.bytes = o;
    return L;
}

}  // namespace

long long ffn_bwd_rows(int T, int E, int K) { return layout(T, 64, E, K, 64).rows; }

size_t ffn_bwd_bytes(int T, int H, int E, int K, int I) { return layout(T, H, E, K, I).bytes; }

cudaError_t launch_ffn_bwd(const FfnBwd &f, void *scratch, int *status, unsigned long long timeout_ns,
                           int inject, cudaStream_t s)
{
    const int T = f.T, H = f.H, E = f.E, K = f.K, I = f.I;
    const Layout L = layout(T, H, E, K, I);
    unsigned char *w = static_cast<unsigned char *>(scratch);
    int *pl = reinterpret_cast<int *>(w + L.plan);
    Plan plan{pl, pl + 2, pl + 2 + MAXG, pl + 2 + 2 * MAXG, pl + 3 + 3 * MAXG, pl + 4 + 4 * MAXG, pl + 1};
    uint16_t *X = reinterpret_cast<uint16_t *>(w + L.X), *D = reinterpret_cast<uint16_t *>(w + L.D);
    float *wrow = reinterpret_cast<float *>(w + L.wrow), *dwp = reinterpret_cast<float *>(w + L.dwp);
    float *dxp = reinterpret_cast<float *>(w + L.dxp);
    int *prow = reinterpret_cast<int *>(w + L.prow);

    // dg, du and hw lie in blocks of 64 token rows: [rows / 64][I][64]
    void *dg = w + L.dg, *du = w + L.du, *hw = w + L.hw;
    const int blocks = static_cast<int>(L.rows / 64);
    GemmArgs a;
    memset(&a, 0, sizeof a);
    if (!encode(&a.x128, X, 0, L.rows, H, 128) || !encode(&a.d128, D, 0, L.rows, H, 128) ||
        !encode(&a.x32, X, 0, L.rows, H, 32) || !encode(&a.d32, D, 0, L.rows, H, 32) ||
        !encode(&a.xb, X, 0, L.rows, H, 64) || !encode(&a.db, D, 0, L.rows, H, 64) ||
        !encode(&a.gb, dg, blocks, I, 64, 64) || !encode(&a.ub, du, blocks, I, 64, 64) ||
        !encode(&a.hb, hw, blocks, I, 64, 64) || !encode(&a.w1, f.W1, E, H, I, 64) ||
        !encode(&a.w3, f.W3, E, H, I, 64) || !encode(&a.w2, f.W2, E, I, H, 64) ||
        !encode(&a.gs, dg, blocks, I, 64, 32, 32) || !encode(&a.us, du, blocks, I, 64, 32, 32) ||
        !encode(&a.hs, hw, blocks, I, 64, 32, 32) || !encode(&a.xs, dxp, 0, L.rows, H, 32, 32, true) ||
        !encode(&a.s1, f.dW1, E, H, I, 32) || !encode(&a.s3, f.dW3, E, H, I, 32) ||
        !encode(&a.s2, f.dW2, E, I, H, 32))
        return cudaErrorInvalidValue;
    a.plan = plan;
    a.E = E; a.H = H; a.I = I;
    a.chunk = f.x_scale ? CHUNK_E4M3 : CHUNK_BF16;
    a.wrow = wrow;
    a.dwp = dwp;
    a.ld_dwp = L.rows;
    a.stash = reinterpret_cast<float *>(w + L.stash);
    a.status = status;
    a.timeout_ns = timeout_ns;
    a.inject = inject;

    const unsigned parts = (H + GCOLS - 1) / GCOLS;
    const bool fused = E <= PLAN_E && static_cast<size_t>(T + E) * parts <= PLAN_CTAS;
    cudaError_t e = cudaSuccess;
    if (!fused) e = launch_pdl(plan_kernel, dim3(1), dim3(1024), 0, s, 1, f.offsets, E, T * K, plan, status);
    if (e != cudaSuccess) return e;
    e = launch_pdl(fused ? gather_kernel<true> : gather_kernel<false>, dim3(T + E, parts), dim3(GT), 0, s, 1, f.x,
                   f.x_scale, static_cast<const uint16_t *>(f.dY), f.offsets, f.slot_pos, f.topk_w, T, H, E, K,
                   plan, X, D, wrow, prow, status);
    if (e != cudaSuccess) return e;
    const unsigned ctas = gemm_ctas();
    const size_t smem = 1024 + STAGES * STAGE + N_EPI * SLAB;
    if ((e = ensure_smem(reinterpret_cast<const void *>(bwd_gemm_kernel), smem)) != cudaSuccess) return e;
    if ((e = launch_pdl(bwd_gemm_kernel, dim3(ctas), dim3(NT), smem, s, 2, a)) != cudaSuccess) return e;
    return launch_pdl(finish_kernel, dim3(T, parts), dim3(GT), 0, s, 1, static_cast<const float *>(dxp),
                      static_cast<const int *>(prow), static_cast<const float *>(dwp), L.rows, dw_parts(I),
                      static_cast<const int *>(plan.ok), H, K, static_cast<uint16_t *>(f.dX), f.d_topk_w);
}

}  // namespace moe
