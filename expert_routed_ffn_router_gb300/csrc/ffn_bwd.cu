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
constexpr int TM = 256;                   // rows of a tile (a cluster)
constexpr int BK = 64;                    // depth of a stage
constexpr int N_EPI = 8;                  // epilogue warps
constexpr int NT = 64 + 32 * N_EPI;
constexpr int MAXG = 1024;
constexpr int HALF = 8192;                // one 64 x 64 bf16 box
constexpr int STAGE_GATES = 2 * 16384 + 3 * HALF;   // X, dY rows; W1, W3, W2 boxes
constexpr int STAGE_GRADS = 2 * 16384;
constexpr int S_GATES = 4, S_GRADS = 6;
constexpr int GN = 128;                   // "gates": columns of a tile
constexpr int DN = 256;                   // "grads": columns of a tile

// What the plan kernel leaves in the workspace.
struct Plan {
    int *ok;        // 1: offsets valid
    int *cnt;       // [E] rows
    int *src;       // [E] first row in the caller's order
    int *pos;       // [E + 1] first padded row
    int *tiles;     // [E + 1] 256-row tiles before the group
};

struct GemmArgs {
    CUtensorMap xa, da;              // gates: X, dY rows, boxes of 128 rows
    CUtensorMap w1, w3, w2;          // weights, 64 x 64 boxes
    CUtensorMap ga, ua;              // grads: dg, du rows, boxes of 128 rows
    CUtensorMap xb, db, gb, ub, hb;  // grads: X, dY, dg, du, hw, 64 x 64 boxes
    Plan plan;
    int E, H, I;
    const float *wrow;               // [padded rows] slot weights
    uint16_t *dg, *du, *hw;          // [padded rows][I]
    float *dwp;                      // [I / 64][padded rows] partial sums of <p, h>
    long long ld_dwp;
    float *dxp;                      // [padded rows][H]
    uint16_t *dW1, *dW3, *dW2;
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
struct Tile {
    int kind;       // 0 gates; 1 rows of dX; 2, 3, 4 dW1, dW3, dW2
    int g, row0, live, col0, kb, m0;
    // gates, dX rows: row0 the tile's first padded row, live its rows from there to the end
    // of the group (padded), col0 the first column; weight gradients: m0, col0 the tile's
    // first output row and column, row0 the group's first padded row
};

template <bool GATES>
__global__ void __launch_bounds__(NT, 1) bwd_gemm_kernel(const __grid_constant__ GemmArgs p)
{
    constexpr int S = GATES ? S_GATES : S_GRADS;
    constexpr int STAGE = GATES ? STAGE_GATES : STAGE_GRADS;
    constexpr int TCOLS = 512;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *ring = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ uint64_t full[S], empty[S], tfull[2], tempty[2], drain;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_s;
    volatile int *abort_flag = &abort_s;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const uint64_t tmo = p.timeout_ns;
    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
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
    const int nI = GATES ? (I + GN - 1) / GN : (I + DN - 1) / DN;      // tiles along I
    const int nH = (H + DN - 1) / DN;
    const int n_rows = row_tiles * (GATES ? nI : nH);
    const int per_w = nH * nI;                                         // tiles of one weight matrix
    const int n_tiles = GATES ? n_rows : (ok ? n_rows + 3 * E * per_w : 0);
    const int unit = blockIdx.x >> 1, units = gridDim.x >> 1;

    auto decode = [&](int t) -> Tile {
        Tile T{};
        if (GATES || t < n_rows) {
            // a group's tiles: column by column, its row tiles innermost (they share the
            // weights)
            const int nc = GATES ? nI : nH;
            int lo = 0, hi = E - 1;      // last group with tiles[g] * nc <= t
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (p.plan.tiles[mid] * nc <= t) lo = mid; else hi = mid - 1;
            }
            const int mt = p.plan.tiles[lo + 1] - p.plan.tiles[lo];
            const int l = t - p.plan.tiles[lo] * nc;
            const int c = l / mt, m = l - c * mt;
            T.kind = GATES ? 0 : 1;
            T.g = lo;
            T.row0 = p.plan.pos[lo] + m * TM;
            T.live = (GATES ? pad_rows(p.plan.cnt[lo]) : p.plan.cnt[lo]) - m * TM;
            T.col0 = c * (GATES ? GN : DN);
            T.kb = GATES ? H / BK : 2 * (I / BK);
        } else {
            int v = t - n_rows;
            const int g = v / (3 * per_w);
            v -= g * 3 * per_w;
            const int w = v / per_w;
            v -= w * per_w;
            const int nc = w < 2 ? nI : nH;
            T.kind = 2 + w;
            T.g = g;
            T.m0 = v / nc * TM;
            T.col0 = (v - v / nc * nc) * DN;
            T.row0 = p.plan.pos[g];
            T.kb = pad_rows(p.plan.cnt[g]) / BK;
        }
        return T;
    };

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0 && !p.inject) {
            uint32_t s = 0, ph = 0, it = 0;
            const uint32_t full0 = mapa_shared(smem_u32(full), 0);
            bool good = true;
            for (int t = unit; t < n_tiles && good; t += units) {
                const Tile T = decode(t);
                const int r = static_cast<int>(rank);
                for (int kb = 0; kb < T.kb; ++kb, ++it) {
                    if (!mbar_wait(&empty[s], ph ^ 1u, abort_flag, p.status, tmo)) { good = false; break; }
                    unsigned char *a = ring + s * STAGE;
                    const uint32_t fb = full0 + 8u * s;
                    if (leader) mbar_arrive_expect_tx(&full[s], 2u * STAGE);
                    if (GATES) {
                        const int row = T.row0 + 128 * r, col = T.col0 + 64 * r, k = kb * BK;
                        tma_load_2d_pair(a, &p.xa, fb, k, row);
                        tma_load_2d_pair(a + 16384, &p.da, fb, k, row);
                        tma_load_3d_pair(a + 32768, &p.w1, fb, col, k, T.g);
                        tma_load_3d_pair(a + 32768 + HALF, &p.w3, fb, col, k, T.g);
                        tma_load_3d_pair(a + 32768 + 2 * HALF, &p.w2, fb, k, col, T.g);
                    } else if (T.kind == 1) {
                        const bool second = kb >= I / BK;
                        const int k = (second ? kb - I / BK : kb) * BK, col = T.col0 + 128 * r;
                        tma_load_2d_pair(a, second ? &p.ua : &p.ga, fb, k, T.row0 + 128 * r);
                        const CUtensorMap *w = second ? &p.w3 : &p.w1;
                        tma_load_3d_pair(a + 16384, w, fb, k, col, T.g);
                        tma_load_3d_pair(a + 16384 + HALF, w, fb, k, col + 64, T.g);
                    } else {
                        const CUtensorMap *ma = T.kind == 4 ? &p.hb : &p.xb;
                        const CUtensorMap *mb = T.kind == 4 ? &p.db : (T.kind == 3 ? &p.ub : &p.gb);
                        const int k = T.row0 + kb * BK, m = T.m0 + 128 * r, n = T.col0 + 128 * r;
                        tma_load_2d_pair(a, ma, fb, m, k);
                        tma_load_2d_pair(a + HALF, ma, fb, m + 64, k);
                        tma_load_2d_pair(a + 16384, mb, fb, n, k);
                        tma_load_2d_pair(a + 16384 + HALF, mb, fb, n + 64, k);
                    }
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
            }
            // every copy issued lands before the CTAs can exit (the even CTA's barriers
            // count both CTAs' copies)
            if (leader) {
                const uint32_t n = it < S ? it : S;
                for (uint32_t j = it - n; j < it; ++j) {
                    int dummy = 0;
                    mbar_wait(&full[j % S], (j / S) & 1u, &dummy, nullptr, 20000000ull);
                }
            }
        }
    } else if (warp == 1) {
        // -------------------------------------------------------------- MMA issuer
        if (lane == 0 && leader) {
            const uint32_t ring0 = smem_u32(ring);
            uint32_t s = 0, ph = 0, tc = 0;
            bool good = true;
            for (int t = unit; t < n_tiles && good; t += units, ++tc) {
                const Tile T = decode(t);
                const uint32_t b = GATES ? 0u : tc & 1u, tph = GATES ? tc & 1u : (tc >> 1) & 1u;
                if (!mbar_wait_cluster(&tempty[b], tph ^ 1u, abort_flag, p.status, tmo)) { good = false; break; }
                tc_fence_after();
                for (int kb = 0; kb < T.kb; ++kb) {
                    if (!mbar_wait(&full[s], ph, abort_flag, p.status, tmo)) { good = false; break; }
                    tc_fence_after();
                    const uint32_t a = ring0 + s * STAGE;
                    if (GATES) {
                        // rows K-major; W1 and W3 boxes are columns of I (MN-major), W2's K-major
                        const uint64_t xd = smem_desc_sw128(a, 16, 1024), dd = smem_desc_sw128(a + 16384, 16, 1024);
                        const uint64_t b1 = smem_desc_sw128(a + 32768, HALF, 1024);
                        const uint64_t b3 = smem_desc_sw128(a + 32768 + HALF, HALF, 1024);
                        const uint64_t b2 = smem_desc_sw128(a + 32768 + 2 * HALF, 16, 1024);
                        constexpr uint32_t iw = idesc_bf16_f32(TM, GN, false, true);
                        constexpr uint32_t ik = idesc_bf16_f32(TM, GN, false, false);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t acc = kb | k ? 1u : 0u;
                            tc_mma_bf16_pair(tmem, xd + 2 * k, b1 + 128 * k, iw, acc);
                            tc_mma_bf16_pair(tmem + GN, xd + 2 * k, b3 + 128 * k, iw, acc);
                            tc_mma_bf16_pair(tmem + 2 * GN, dd + 2 * k, b2 + 2 * k, ik, acc);
                        }
                    } else {
                        const uint32_t d = tmem + b * DN;
                        const bool rows = T.kind == 1;
                        const uint64_t ad = rows ? smem_desc_sw128(a, 16, 1024) : smem_desc_sw128(a, HALF, 1024);
                        const uint64_t bd = rows ? smem_desc_sw128(a + 16384, 16, 1024)
                                                 : smem_desc_sw128(a + 16384, HALF, 1024);
                        const uint32_t step = rows ? 2u : 128u;
                        const uint32_t id = rows ? idesc_bf16_f32(TM, DN, false, false)
                                                 : idesc_bf16_f32(TM, DN, true, true);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            tc_mma_bf16_pair(d, ad + step * k, bd + step * k, id, kb | k ? 1u : 0u);
                    }
                    tc_commit_pair_mc(&empty[s], 3);
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
                if (!good) break;
                tc_commit_pair_mc(&tfull[b], 3);
            }
            tc_commit_pair_mc(&drain, 1);
            int dummy = 0;
            mbar_wait(&drain, 0, &dummy, nullptr, 20000000ull);
        }
    } else {
        // ---------------------------------------------------------------- epilogue
        const int q = warp & 3, half = (warp - 2) >> 2;   // lane quarter, column half
        const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
        const uint32_t tempty0 = mapa_shared(smem_u32(tempty), 0);
        uint32_t tc = 0;
        for (int t = unit; t < n_tiles; t += units, ++tc) {
            const Tile T = decode(t);
            const uint32_t b = GATES ? 0u : tc & 1u, tph = GATES ? tc & 1u : (tc >> 1) & 1u;
            bool good = true;
            if (lane == 0) good = mbar_wait(&tfull[b], tph, abort_flag, p.status, tmo);
            good = __shfl_sync(kFullMask, good, 0);
            if (!good) break;
            // (every lane observes the completed phase itself before it reads tensor memory)
            mbar_try_wait(&tfull[b], tph);
            tc_fence_after();
            const int lrow = 128 * static_cast<int>(rank) + 32 * q + lane;   // row of the tile
            if (GATES) {
                const bool on = lrow < T.live;
                const size_t row = static_cast<size_t>(T.row0 + lrow);
                const float w = on ? p.wrow[row] : 0.f;
                const int c0 = T.col0 + 64 * half;
                const bool cols = c0 < I;
                float dw = 0.f;
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    const uint32_t at = tmem + lanes + 64 * half + 32 * c;
                    float g[32], u[32], pv[32];
                    __syncwarp();
                    tmem_ld32(at, g);
                    tmem_ld32(at + GN, u);
                    tmem_ld32(at + 2 * GN, pv);
                    uint32_t og[16], ou[16], oh[16];
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        float a[2], bb[2], cc[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float gi = g[i + k], ui = u[i + k], pi = pv[i + k];
                            const float s = fast_sigmoid(gi), gs = gi * s, h = gs * ui;
                            dw = fmaf(pi, h, dw);
                            const float pw = pi * w;
                            a[k] = pw * ui * s * fmaf(gi, 1.f - s, 1.f);
                            bb[k] = pw * gs;
                            cc[k] = w * h;
                        }
                        og[i / 2] = f32x2_to_bf16x2(a[1], a[0]);
                        ou[i / 2] = f32x2_to_bf16x2(bb[1], bb[0]);
                        oh[i / 2] = f32x2_to_bf16x2(cc[1], cc[0]);
                    }
                    if (on && cols) {
                        const size_t o = row * I + c0 + 32 * c;
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {
                            *reinterpret_cast<uint4 *>(p.dg + o + 2 * i) = make_uint4(og[i], og[i + 1], og[i + 2], og[i + 3]);
                            *reinterpret_cast<uint4 *>(p.du + o + 2 * i) = make_uint4(ou[i], ou[i + 1], ou[i + 2], ou[i + 3]);
                            *reinterpret_cast<uint4 *>(p.hw + o + 2 * i) = make_uint4(oh[i], oh[i + 1], oh[i + 2], oh[i + 3]);
                        }
                    }
                }
                if (on && cols) p.dwp[static_cast<size_t>(c0 / 64) * p.ld_dwp + row] = dw;
            } else {
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    const int lc = 128 * half + 32 * c;
                    float v[32];
                    __syncwarp();
                    tmem_ld32(tmem + b * DN + lanes + lc, v);
                    const int col = T.col0 + lc;
                    if (T.kind == 1) {
                        if (lrow < T.live && col < H) {
                            float4 *o = reinterpret_cast<float4 *>(p.dxp + static_cast<size_t>(T.row0 + lrow) * H + col);
#pragma unroll
                            for (int i = 0; i < 8; ++i) o[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                        }
                    } else {
                        const int M = T.kind == 4 ? I : H, N = T.kind == 4 ? H : I, m = T.m0 + lrow;
                        if (m < M && col < N) {
                            uint16_t *base = T.kind == 2 ? p.dW1 : (T.kind == 3 ? p.dW3 : p.dW2);
                            uint4 *o = reinterpret_cast<uint4 *>(base + (static_cast<size_t>(T.g) * M + m) * N + col);
                            if (T.kb == 0) {       // an expert without rows
#pragma unroll
                                for (int i = 0; i < 4; ++i) o[i] = make_uint4(0, 0, 0, 0);
                            } else {
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    o[i] = make_uint4(f32x2_to_bf16x2(v[8 * i + 1], v[8 * i]), f32x2_to_bf16x2(v[8 * i + 3], v[8 * i + 2]),
                                                      f32x2_to_bf16x2(v[8 * i + 5], v[8 * i + 4]), f32x2_to_bf16x2(v[8 * i + 7], v[8 * i + 6]));
                            }
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(tempty0 + 8u * b);
        }
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

// bf16 [groups][rows][cols] (groups == 0: [rows][cols]), boxes of 64 columns x box_rows rows
// in the 128-byte swizzle.
bool encode(CUtensorMap *m, const void *base, int groups, long long rows, int cols, int box_rows)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(groups)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols) * 2, static_cast<cuuint64_t>(cols) * rows * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1}, estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, groups ? 3 : 2, const_cast<void *>(base), dims, strides,
              box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t al256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }

struct Layout {
    long long rows;        // padded rows at most
    size_t plan, wrow, prow, X, D, dg, du, hw, dwp, dxp, bytes;
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
    L.dwp = take(R * (I / 64) * 4);
    L.dxp = take(R * H * 4);
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

    GemmArgs a;
    memset(&a, 0, sizeof a);
    a.dg = reinterpret_cast<uint16_t *>(w + L.dg);
    a.du = reinterpret_cast<uint16_t *>(w + L.du);
    a.hw = reinterpret_cast<uint16_t *>(w + L.hw);
    if (!encode(&a.xa, X, 0, L.rows, H, 128) || !encode(&a.da, D, 0, L.rows, H, 128) ||
        !encode(&a.xb, X, 0, L.rows, H, 64) || !encode(&a.db, D, 0, L.rows, H, 64) ||
        !encode(&a.ga, a.dg, 0, L.rows, I, 128) || !encode(&a.ua, a.du, 0, L.rows, I, 128) ||
        !encode(&a.gb, a.dg, 0, L.rows, I, 64) || !encode(&a.ub, a.du, 0, L.rows, I, 64) ||
        !encode(&a.hb, a.hw, 0, L.rows, I, 64) || !encode(&a.w1, f.W1, E, H, I, 64) ||
        !encode(&a.w3, f.W3, E, H, I, 64) || !encode(&a.w2, f.W2, E, I, H, 64))
        return cudaErrorInvalidValue;
    a.plan = plan;
    a.E = E; a.H = H; a.I = I;
    a.wrow = wrow;
    a.dwp = dwp;
    a.ld_dwp = L.rows;
    a.dxp = dxp;
    a.dW1 = static_cast<uint16_t *>(f.dW1);
    a.dW3 = static_cast<uint16_t *>(f.dW3);
    a.dW2 = static_cast<uint16_t *>(f.dW2);
    a.status = status;
    a.timeout_ns = timeout_ns;
    a.inject = inject;

    cudaError_t e = launch_pdl(plan_kernel, dim3(1), dim3(1024), 0, s, 1, f.offsets, E, T * K, plan, status);
    if (e != cudaSuccess) return e;
    const unsigned parts = (H + GCOLS - 1) / GCOLS;
    e = launch_pdl(gather_kernel, dim3(T + E, parts), dim3(GT), 0, s, 1, f.x, f.x_scale,
                   static_cast<const uint16_t *>(f.dY), f.slot_pos, f.topk_w, T, H, E, K, plan, X, D, wrow, prow);
    if (e != cudaSuccess) return e;
    const unsigned ctas = num_sms() / 2 * 2;
    const size_t sm1 = 1024 + static_cast<size_t>(S_GATES) * STAGE_GATES, sm2 = 1024 + static_cast<size_t>(S_GRADS) * STAGE_GRADS;
    if ((e = ensure_smem(reinterpret_cast<const void *>(bwd_gemm_kernel<true>), sm1)) != cudaSuccess) return e;
    if ((e = ensure_smem(reinterpret_cast<const void *>(bwd_gemm_kernel<false>), sm2)) != cudaSuccess) return e;
    if ((e = launch_pdl(bwd_gemm_kernel<true>, dim3(ctas), dim3(NT), sm1, s, 2, a)) != cudaSuccess) return e;
    if ((e = launch_pdl(bwd_gemm_kernel<false>, dim3(ctas), dim3(NT), sm2, s, 2, a)) != cudaSuccess) return e;
    return launch_pdl(finish_kernel, dim3(T, parts), dim3(GT), 0, s, 1, static_cast<const float *>(dxp),
                      static_cast<const int *>(prow), static_cast<const float *>(dwp), L.rows, I / 64,
                      static_cast<const int *>(plan.ok), H, K, static_cast<uint16_t *>(f.dX), f.d_topk_w);
}

}  // namespace moe
