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
//   plan     padded row offsets of the groups (multiples of 64 rows), offsets checked
//   gather   the rows of X (taken back from 8 bits) and dY in padded group order, bf16; the
//            rows up to the next multiple of 64 are zeros, so no product needs a mask
//   gates    three products per tile in tensor memory (g, u, p), the formulas above in the
//            epilogue; writes dg, du, hw (bf16) and partial sums of <p, h>
//   grads    dg W1^T + du W3^T (fp32 rows) and the three weight gradients, one tile list
//   finish   dX and d topk_w: sums over the slots, over the partials, in a fixed order
// No atomics on results: they repeat bit for bit.
//
// Rounding.  dg, du and hw are operands of bf16 products and are rounded to bf16 once each;
// products are summed in fp32 (tensor memory), the rows of dX stay fp32 until their sum over
// the slots is rounded.  d topk_w is fp32 throughout.
//
// Tiles.  Clusters of two CTAs issue 2-SM MMAs of M = 256.  "gates": 256 token rows x 128
// columns of I, 3 x 128 columns of tensor memory.  "grads": 256 x 256, two buffers of 256
// columns.  Roles per CTA: warp 0 TMA producer, warp 1 MMA issuer (even CTA), warps 2..9
// epilogue (two per lane quarter, each half of the columns).  Tiles are dealt to the clusters
// in turn; every role walks the same list.
//
// Every wait is bounded as in ffn_tc.cu (MOE_ERR_DEVICE_TIMEOUT in the status word).
#include <cuda.h>

#include <cstring>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int PADR = 64;                  // groups start at multiples of this many rows
constexpr int TM = 256, TN = 256;         // tile of a cluster
constexpr int BK = 64;                    // depth of a stage
constexpr int N_EPI = 8;                  // epilogue warps
constexpr int NT = 64 + 32 * N_EPI;        // at most 168 registers a thread
constexpr int MAXG = 1024;
constexpr int HALF = 8192;                // one 64 x 64 bf16 box
constexpr int STAGE = 4 * HALF;           // A: 128 rows of this CTA; B: 128 of the tile's columns
constexpr int STAGES = 6;
constexpr int SLAB = 4096;                // an epilogue warp's store buffer: 32 rows of 128 bytes
// Stages of one sum in tensor memory in the products that d topk_w comes from (see above).
constexpr int CHUNK = 8;
constexpr int STASH = 32 * N_EPI * 128;   // floats of a CTA's stash: p of a unit

// What the plan kernel leaves in the workspace.
struct Plan {
    int *ok;        // 1: offsets valid
    int *cnt;       // [E] rows
    int *src;       // [E] first row in the caller's order
    int *pos;       // [E + 1] first padded row
    int *tiles;     // [E + 1] 256-row tiles before the group
};

struct GemmArgs {
    // loads: token rows (boxes of 128 rows; of 64 x 64), weights (64 x 64)
    CUtensorMap xa, da, ga, ua, xb, db, gb, ub, hb, w1, w3, w2;
    // stores: dg, du, hw (64 columns x 32 rows), rows of dX (32 fp32 x 32), weight gradients
    CUtensorMap gs, us, hs, xs, s1, s3, s2;
    Plan plan;
    int E, H, I;
    const float *wrow;               // [padded rows] slot weights
    float *dwp;                      // [2 ceil(I / 128)][padded rows] partial sums of <p, h>
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
__global__ void __launch_bounds__(1024) plan_kernel(const int32_t *__restrict__ offsets, int E, int rows,
                                                    Plan p, int *status)
{
    __shared__ int a[32], b[32];
    pdl_wait();
    const int g = threadIdx.x, lane = g & 31, warp = g >> 5;
    const int lo = g < E ? offsets[g] : 0, hi = g < E ? offsets[g + 1] : 0;
    const int bad = lo < 0 || hi < lo || hi > rows;
    const bool ok = !__syncthreads_or(bad);
    const int m = ok ? hi - lo : 0;
    const int np = pad_rows(m), nt = (m + TM - 1) / TM;
    int ip = np, it = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int vp = __shfl_up_sync(kFullMask, ip, o), vt = __shfl_up_sync(kFullMask, it, o);
        if (lane >= o) { ip += vp; it += vt; }
    }
    if (lane == 31) { a[warp] = ip; b[warp] = it; }
    __syncthreads();
    for (int w = 0; w < warp; ++w) { ip += a[w]; it += b[w]; }
    if (g < E) {
        p.cnt[g] = m;
        p.src[g] = lo;
        p.pos[g] = ip - np;
        p.tiles[g] = it - nt;
    }
    if (g == E - 1) {
        p.pos[E] = ip;
        p.tiles[E] = it;
    }
    if (g == 0) {
        *p.ok = ok ? 1 : 0;
        if (!ok) report(status, MOE_ERR_INVALID_ARG);
    }
}

// --------------------------------------------------------------------------- gather
// CTA (t, y) of the first T: token t's row, columns of part y, to the padded rows of its
// slots.  CTA (T + g, y): the zero rows at the end of group g.
constexpr int GT = 128;
constexpr int GCOLS = GT * 8;

__global__ void __launch_bounds__(GT) gather_kernel(const void *__restrict__ x, const int8_t *__restrict__ xs,
                                                    const uint16_t *__restrict__ dY,
                                                    const int32_t *__restrict__ slot_pos,
                                                    const float *__restrict__ topk_w, int T, int H, int E,
                                                    int K, Plan p, uint16_t *__restrict__ X,
                                                    uint16_t *__restrict__ D, float *__restrict__ wrow,
                                                    int *__restrict__ prow)
{
    __shared__ int dst[32];
    pdl_wait();
    if (!*p.ok) return;
    const int c = blockIdx.y * GCOLS + threadIdx.x * 8;
    if (blockIdx.x >= static_cast<unsigned>(T)) {
        const int g = blockIdx.x - T;
        const int m = p.cnt[g], n = pad_rows(m);
        for (int r = m; r < n; ++r) {
            const size_t row = static_cast<size_t>(p.pos[g] + r);
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
        if (r >= 0 && r < p.src[E - 1] + p.cnt[E - 1]) {
            int lo = 0, hi = E - 1;        // last group whose first row is <= r
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (p.src[mid] <= r) lo = mid; else hi = mid - 1;
            }
            const int k = r - p.src[lo];
            if (k >= 0 && k < p.cnt[lo]) q = p.pos[lo] + k;
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
enum { GU, PR, ROWS, DW1, DW3, DW2, END };     // g and u; p; rows of dX; weight gradients

struct Tile {
    int kind, g;
    int row0;       // first padded row of the tile (weight gradients: of the group)
    int live;       // padded rows of the group from row0 on
    int m0;         // weight gradients: first output row
    int col0;       // first output column
    int kb, chunk;  // stages, and stages of one sum in tensor memory
};

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

// The warp's slab may be written again: the store before it has read it.
__device__ __forceinline__ void slab_free(int lane)
{
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
}

// 16 bytes to chunk c (of 8) of the lane's row, in the 128-byte swizzle
__device__ __forceinline__ void slab_put(unsigned char *slab, int lane, int c, uint4 v)
{
    *reinterpret_cast<uint4 *>(slab + lane * 128 + ((c ^ (lane & 7)) << 4)) = v;
}

// The slab is written: order it before the store that lane 0 issues next.
__device__ __forceinline__ void slab_ready()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
}

__device__ __forceinline__ void slab_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }

// 64 fp32 -> the lane's row of 64 bf16
__device__ __forceinline__ void slab_bf16(unsigned char *slab, int lane, const float *v, int c0)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        slab_put(slab, lane, c0 + i,
                 make_uint4(f32x2_to_bf16x2(v[8 * i + 1], v[8 * i]), f32x2_to_bf16x2(v[8 * i + 3], v[8 * i + 2]),
                            f32x2_to_bf16x2(v[8 * i + 5], v[8 * i + 4]), f32x2_to_bf16x2(v[8 * i + 7], v[8 * i + 6])));
}

// GATES: units of (p of 256 columns; g and u of 128 of them, twice); else: tiles of dX's
// rows, then of the weight gradients.
template <bool GATES>
__global__ void __launch_bounds__(NT, 1) bwd_gemm_kernel(const __grid_constant__ GemmArgs p)
{
    constexpr int TCOLS = 512;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *ring = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char *slabs = ring + STAGES * STAGE;
    __shared__ uint64_t full[STAGES], empty[STAGES], tfull[2], tempty[2], drain;
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
    const int nI = (I + TN - 1) / TN, nH = (H + TN - 1) / TN;
    const int n_rows = row_tiles * (GATES ? nI : nH);
    const int per_w = nH * nI;                       // tiles of one weight gradient
    const int n_units = GATES ? n_rows : (ok ? n_rows + 3 * E * per_w : 0);
    const int step = gridDim.x >> 1;

    // The tiles of this cluster, in order: `next` takes (unit, part of the unit) on.
    struct Walk { int unit, part, g; };
    auto start = [&]() -> Walk { return Walk{static_cast<int>(blockIdx.x >> 1), 0, 0}; };
    auto tile_of = [&](Walk &w) -> Tile {
        Tile T{};
        T.kind = END;
        bool last = true;                            // of its unit
        if (w.unit >= n_units) return T;
        if (w.unit < n_rows) {
            // column by column, a group's row tiles innermost (they share the weights)
            const int nc = GATES ? nI : nH;
            // the group with tiles[g] * nc <= unit < tiles[g + 1] * nc: mostly the last tile's or
            // one of the next
            int lo = w.g, near = 0;
            while (near < 8 && p.plan.tiles[lo + 1] * nc <= w.unit) { ++lo; ++near; }
            if (near == 8) {
                int hi = E - 1;
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (p.plan.tiles[mid] * nc <= w.unit) lo = mid; else hi = mid - 1;
                }
            }
            w.g = lo;
            const int mt = p.plan.tiles[lo + 1] - p.plan.tiles[lo];
            const int l = w.unit - p.plan.tiles[lo] * nc;
            const int c = l / mt, m = l - c * mt;
            T.g = lo;
            T.row0 = p.plan.pos[lo] + m * TM;
            T.live = pad_rows(p.plan.cnt[lo]) - m * TM;
            T.col0 = c * TN;
            if (GATES) {
                // p of 256 columns, then g and u of the first 128 and (where there are any) of
                // the other 128
                T.kind = w.part == 0 ? PR : GU;
                if (w.part == 2) T.col0 += 128;
                last = w.part == 2 || (w.part == 1 && T.col0 + 128 >= I);
                T.kb = H / BK;
                T.chunk = CHUNK;
            } else {
                T.kind = ROWS;
                T.kb = T.chunk = 2 * (I / BK);
            }
        } else {
            int v = w.unit - n_rows;
            T.g = v / (3 * per_w);
            v -= T.g * 3 * per_w;
            const int m = v / per_w;
            v -= m * per_w;
            const int nc = m < 2 ? nI : nH;
            T.kind = DW1 + m;
            T.m0 = v / nc * TM;
            T.col0 = (v - v / nc * nc) * TN;
            T.row0 = p.plan.pos[T.g];
            T.kb = T.chunk = pad_rows(p.plan.cnt[T.g]) / BK;
        }
        if (!last) ++w.part;
        else { w.unit += step; w.part = 0; }
        return T;
    };

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0 && !p.inject) {
            uint32_t s = 0, ph = 0, it = 0;
            const uint32_t full0 = mapa_shared(smem_u32(full), 0);
            const int r = static_cast<int>(rank);
            bool good = true;
            Walk w = start();
            while (good) {
                const Tile T = tile_of(w);
                if (T.kind == END) break;
                for (int kb = 0; kb < T.kb; ++kb, ++it) {
                    if (!mbar_wait(&empty[s], ph ^ 1u, abort_flag, p.status, tmo)) { good = false; break; }
                    unsigned char *a = ring + s * STAGE, *b = a + 2 * HALF;
                    const uint32_t fb = full0 + 8u * s;
                    if (leader) mbar_arrive_expect_tx(&full[s], 2u * STAGE);
                    const int k = kb * BK;
                    if (GATES) {
                        const int row = T.row0 + 128 * r, col = T.col0 + 64 * r;
                        if (T.kind == GU) {
                            // this CTA's 128 of the tile's columns: 64 of W1, the same 64 of W3
                            tma_load_2d_pair(a, &p.xa, fb, k, row);
                            tma_load_3d_pair(b, &p.w1, fb, col, k, T.g);
                            tma_load_3d_pair(b + HALF, &p.w3, fb, col, k, T.g);
                        } else {
                            // ... the columns whose g and u this CTA's half came from
                            tma_load_2d_pair(a, &p.da, fb, k, row);
                            tma_load_3d_pair(b, &p.w2, fb, k, col, T.g);
                            tma_load_3d_pair(b + HALF, &p.w2, fb, k, col + 128, T.g);
                        }
                    } else if (T.kind == ROWS) {
                        const bool second = kb >= I / BK;
                        const int c = second ? k - I : k, col = T.col0 + 128 * r;
                        const CUtensorMap *wm = second ? &p.w3 : &p.w1;
                        tma_load_2d_pair(a, second ? &p.ua : &p.ga, fb, c, T.row0 + 128 * r);
                        tma_load_3d_pair(b, wm, fb, c, col, T.g);
                        tma_load_3d_pair(b + HALF, wm, fb, c, col + 64, T.g);
                    } else {
                        const CUtensorMap *ma = T.kind == DW2 ? &p.hb : &p.xb;
                        const CUtensorMap *mb = T.kind == DW2 ? &p.db : (T.kind == DW3 ? &p.ub : &p.gb);
                        const int row = T.row0 + k, m = T.m0 + 128 * r, n = T.col0 + 128 * r;
                        tma_load_2d_pair(a, ma, fb, m, row);
                        tma_load_2d_pair(a + HALF, ma, fb, m + 64, row);
                        tma_load_2d_pair(b, mb, fb, n, row);
                        tma_load_2d_pair(b + HALF, mb, fb, n + 64, row);
                    }
                    if (++s == STAGES) { s = 0; ph ^= 1u; }
                }
            }
            // every copy issued lands before the CTAs can exit (the even CTA's barriers
            // count both CTAs' copies)
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
            uint32_t s = 0, ph = 0, b = 0, tph = 0;
            bool good = true;
            Walk w = start();
            while (good) {
                const Tile T = tile_of(w);
                if (T.kind == END) break;
                // A: rows K-major, or (weight gradients) rows as the depth, MN-major; B: columns
                // of W1 and W3 as they lie (g, u) and rows as the depth are MN-major
                const bool amn = T.kind >= DW1, bmn = T.kind >= DW1 || T.kind == GU;
                const uint64_t ad0 = smem_desc_sw128(ring0, amn ? HALF : 16, 1024);
                const uint64_t bd0 = smem_desc_sw128(ring0 + 2 * HALF, bmn ? HALF : 16, 1024);
                const uint32_t as = amn ? 128u : 2u, bs = bmn ? 128u : 2u;
                const uint32_t id = idesc_bf16_f32(TM, TN, amn, bmn);
                int kb = 0;
                do {
                    if (!mbar_wait_cluster(&tempty[b], tph ^ 1u, abort_flag, p.status, tmo)) { good = false; break; }
                    tc_fence_after();
                    const uint32_t d = tmem + b * TN;
                    const int end = min(kb + T.chunk, T.kb);
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
                } while (kb < T.kb);
            }
            tc_commit_pair_mc(&drain, 1);
            int dummy = 0;
            mbar_wait(&drain, 0, &dummy, nullptr, 20000000ull);
        }
    } else {
        // ---------------------------------------------------------------- epilogue
        const int q = warp & 3, half = (warp - 2) >> 2;   // lane quarter, column half
        const uint32_t tm0 = tmem + (static_cast<uint32_t>(32 * q) << 16) + 128u * half;
        const uint32_t tempty0 = mapa_shared(smem_u32(tempty), 0);
        unsigned char *slab = slabs + (warp - 2) * SLAB;
        uint32_t b = 0, tph = 0;
        // the sums of buffer b are complete (every lane observes the phase itself)
        auto sums_ready = [&]() -> bool {
            bool good = true;
            if (lane == 0) good = mbar_wait(&tfull[b], tph, abort_flag, p.status, tmo);
            good = __shfl_sync(kFullMask, good, 0);
            if (good) {
                mbar_try_wait(&tfull[b], tph);
                tc_fence_after();
            }
            return good;
        };
        auto sums_read = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(tempty0 + 8u * b);
            b ^= 1u;
            if (b == 0) tph ^= 1u;
        };
        // float4 i of this thread's stash (256 threads side by side)
        float4 *stash = reinterpret_cast<float4 *>(p.stash + static_cast<size_t>(blockIdx.x) * STASH) + (tid - 64);
        constexpr int SROW = 32 * N_EPI;
        int part = 0;                                // of the unit: its tiles of g and u so far
        float dw = 0.f;
        Walk w = start();
        bool good = true;
        while (good) {
            const Tile T = tile_of(w);
            if (T.kind == END) break;
            const int r0 = 128 * static_cast<int>(rank) + 32 * q;   // the warp's first row of the tile
            if (GATES) {
                const bool rows = r0 < T.live;
                const size_t row = static_cast<size_t>(T.row0 + r0 + lane);
                // sums over the chunks, in registers
                float acc[128];
#pragma unroll
                for (int i = 0; i < 128; ++i) acc[i] = 0.f;
#pragma unroll 1
                for (int kb = 0; kb < T.kb; kb += CHUNK) {
                    if (!sums_ready()) { good = false; break; }
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        float v[16];
                        __syncwarp();
                        tmem_ld16(tm0 + b * TN + 16 * c, v);
#pragma unroll
                        for (int i = 0; i < 16; ++i) acc[16 * c + i] += v[i];
                    }
                    sums_read();
                }
                if (!good) break;
                if (T.kind == PR) {
                    // kept for the unit's next tiles: acc[0..63] are columns of the first 128,
                    // acc[64..127] of the second
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        stash[i * SROW] = make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
                    part = 0;
                    dw = 0.f;
                } else {
                    // g of 64 columns in acc[0..63], u of the same in acc[64..127], p in the stash.
                    // In their place: dg and du (bf16 pair), hw.
                    const float wr = rows ? p.wrow[row] : 0.f;
                    const float4 *st = stash + part * 16 * SROW;
                    const int col = T.col0 + 64 * half;
#pragma unroll
                    for (int i = 0; i < 64; i += 4) {
                        const float4 p4 = st[i / 4 * SROW];
                        const float pp[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float g = acc[i + k], u = acc[64 + i + k];
                            const float s = fast_sigmoid(g), gs = g * s, h = gs * u, pw = pp[k] * wr;
                            dw = fmaf(pp[k], h, dw);
                            acc[i + k] = __uint_as_float(f32x2_to_bf16x2(pw * gs, pw * u * s * fmaf(g, 1.f - s, 1.f)));
                            acc[64 + i + k] = wr * h;
                        }
                    }
#pragma unroll
                    for (int x = 0; x < 3; ++x) {    // dg, du, hw
                        slab_free(lane);
#pragma unroll
                        for (int i = 0; i < 64; i += 8) {
                            uint32_t o[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                o[k] = x < 2 ? __byte_perm(__float_as_uint(acc[i + 2 * k]), __float_as_uint(acc[i + 2 * k + 1]),
                                                           x == 0 ? 0x5410 : 0x7632)
                                             : f32x2_to_bf16x2(acc[64 + i + 2 * k + 1], acc[64 + i + 2 * k]);
                            slab_put(slab, lane, i / 8, make_uint4(o[0], o[1], o[2], o[3]));
                        }
                        slab_ready();
                        if (lane == 0 && rows && col < I) {
                            tma_store_2d(x == 0 ? &p.gs : (x == 1 ? &p.us : &p.hs), slab, col, T.row0 + r0);
                            slab_commit();
                        }
                    }
                    // (each of the unit's tiles leaves its own partial sum)
                    if (rows) p.dwp[static_cast<size_t>(2 * (T.col0 / 128) + half) * p.ld_dwp + row] = dw;
                    dw = 0.f;
                    ++part;
                }
            } else {
                if (!sums_ready()) { good = false; break; }
                const uint32_t at = tm0 + b * TN;
                if (T.kind == ROWS) {
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        const int col = T.col0 + 128 * half + 32 * c;
                        float v[32];
                        __syncwarp();
                        tmem_ld32(at + 32 * c, v);
                        slab_free(lane);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            slab_put(slab, lane, i, make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                                               __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3])));
                        slab_ready();
                        if (lane == 0 && r0 < T.live && col < H) {
                            tma_store_2d(&p.xs, slab, col, T.row0 + r0);
                            slab_commit();
                        }
                    }
                } else {
                    const int M = T.kind == DW2 ? I : H, N = T.kind == DW2 ? H : I;
                    const CUtensorMap *sm = T.kind == DW1 ? &p.s1 : (T.kind == DW3 ? &p.s3 : &p.s2);
#pragma unroll 1
                    for (int c = 0; c < 2; ++c) {
                        const int col = T.col0 + 128 * half + 64 * c;
                        float v[32], u[32];
                        __syncwarp();
                        tmem_ld32(at + 64 * c, v);
                        tmem_ld32(at + 64 * c + 32, u);
                        if (T.kb == 0) {             // an expert without rows
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = u[i] = 0.f;
                        }
                        slab_free(lane);
                        slab_bf16(slab, lane, v, 0);
                        slab_bf16(slab, lane, u, 4);
                        slab_ready();
                        if (lane == 0 && T.m0 + r0 < M && col < N) {
                            tma_store_3d(sm, slab, col, T.m0 + r0, T.g);
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

// [groups][rows][cols] (groups == 0: [rows][cols]) of bf16, or fp32, in boxes of 128 bytes x
// box_rows rows in the 128-byte swizzle.
bool encode(CUtensorMap *m, const void *base, int groups, long long rows, int cols, int box_rows,
            bool fp32 = false)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t es = fp32 ? 4 : 2;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(groups)};
    const cuuint64_t strides[2] = {cols * es, cols * es * static_cast<cuuint64_t>(rows)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / es), static_cast<cuuint32_t>(box_rows), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, groups ? 3 : 2,
              const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t al256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }

int gemm_ctas() { return num_sms() / 2 * 2; }
int dw_parts(int I) { return 2 * ((I + 127) / 128); }    // partial sums of <p, h>

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
    L.plan = take((4 * (MAXG + 1) + 1) * sizeof(int));
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
    Plan plan{pl, pl + 1, pl + 1 + MAXG, pl + 1 + 2 * MAXG, pl + 2 + 3 * MAXG};
    uint16_t *X = reinterpret_cast<uint16_t *>(w + L.X), *D = reinterpret_cast<uint16_t *>(w + L.D);
    float *wrow = reinterpret_cast<float *>(w + L.wrow), *dwp = reinterpret_cast<float *>(w + L.dwp);
    float *dxp = reinterpret_cast<float *>(w + L.dxp);
    int *prow = reinterpret_cast<int *>(w + L.prow);

    void *dg = w + L.dg, *du = w + L.du, *hw = w + L.hw;
    GemmArgs a;
    memset(&a, 0, sizeof a);
    if (!encode(&a.xa, X, 0, L.rows, H, 128) || !encode(&a.da, D, 0, L.rows, H, 128) ||
        !encode(&a.ga, dg, 0, L.rows, I, 128) || !encode(&a.ua, du, 0, L.rows, I, 128) ||
        !encode(&a.xb, X, 0, L.rows, H, 64) || !encode(&a.db, D, 0, L.rows, H, 64) ||
        !encode(&a.gb, dg, 0, L.rows, I, 64) || !encode(&a.ub, du, 0, L.rows, I, 64) ||
        !encode(&a.hb, hw, 0, L.rows, I, 64) || !encode(&a.w1, f.W1, E, H, I, 64) ||
        !encode(&a.w3, f.W3, E, H, I, 64) || !encode(&a.w2, f.W2, E, I, H, 64) ||
        !encode(&a.gs, dg, 0, L.rows, I, 32) || !encode(&a.us, du, 0, L.rows, I, 32) ||
        !encode(&a.hs, hw, 0, L.rows, I, 32) || !encode(&a.xs, dxp, 0, L.rows, H, 32, true) ||
        !encode(&a.s1, f.dW1, E, H, I, 32) || !encode(&a.s3, f.dW3, E, H, I, 32) ||
        !encode(&a.s2, f.dW2, E, I, H, 32))
        return cudaErrorInvalidValue;
    a.plan = plan;
    a.E = E; a.H = H; a.I = I;
    a.wrow = wrow;
    a.dwp = dwp;
    a.ld_dwp = L.rows;
    a.stash = reinterpret_cast<float *>(w + L.stash);
    a.status = status;
    a.timeout_ns = timeout_ns;
    a.inject = inject;

    cudaError_t e = launch_pdl(plan_kernel, dim3(1), dim3(1024), 0, s, 1, f.offsets, E, T * K, plan, status);
    if (e != cudaSuccess) return e;
    const unsigned parts = (H + GCOLS - 1) / GCOLS;
    e = launch_pdl(gather_kernel, dim3(T + E, parts), dim3(GT), 0, s, 1, f.x, f.x_scale,
                   static_cast<const uint16_t *>(f.dY), f.slot_pos, f.topk_w, T, H, E, K, plan, X, D, wrow, prow);
    if (e != cudaSuccess) return e;
    const unsigned ctas = gemm_ctas();
    const size_t smem = 1024 + STAGES * STAGE + N_EPI * SLAB;
    if ((e = ensure_smem(reinterpret_cast<const void *>(bwd_gemm_kernel<true>), smem)) != cudaSuccess) return e;
    if ((e = ensure_smem(reinterpret_cast<const void *>(bwd_gemm_kernel<false>), smem)) != cudaSuccess) return e;
    if ((e = launch_pdl(bwd_gemm_kernel<true>, dim3(ctas), dim3(NT), smem, s, 2, a)) != cudaSuccess) return e;
    if ((e = launch_pdl(bwd_gemm_kernel<false>, dim3(ctas), dim3(NT), smem, s, 2, a)) != cudaSuccess) return e;
    return launch_pdl(finish_kernel, dim3(T, parts), dim3(GT), 0, s, 1, static_cast<const float *>(dxp),
                      static_cast<const int *>(prow), static_cast<const float *>(dwp), L.rows, dw_parts(I),
                      static_cast<const int *>(plan.ok), H, K, static_cast<uint16_t *>(f.dX), f.d_topk_w);
}

}  // namespace moe
