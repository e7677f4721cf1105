// norm.cu -- layer norm of the token rows in front of the layer, and its backward pass.
//
//   forward   mu = mean(x), r = (mean((x - mu)^2) + eps)^-1/2, y = gamma (x - mu) r + beta
//   backward  a = gamma dy, xh = (x - mu) r,
//             dx = r (a - mean(a) - xh mean(a xh)) (+ dres),
//             dgamma = sum_t dy xh, dbeta = sum_t dy
//
// Both are bound by memory: every row is read from it once, the variance is taken from the
// centred values (no sum of squares, which cancels for rows far from zero), and all sums are
// fp32.  Short rows take one warp each (up to 1024 columns forward, 512 backward), longer ones
// a CTA.  A batch of 128 rows of 7168 takes 5 us on the GPU, less than its launch costs.
//
// Weight gradients.  Each CTA walks rows blockIdx.x, + gridDim.x, ... and keeps the sums of
// its columns in registers; the CTAs' sums go to the workspace ([CTA][2][H]) and a second
// launch adds them in CTA order.  No atomics: the result depends on the sizes alone.
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int WARP_COLS = 1024;       // longest row that one warp takes (forward)
constexpr int WARP_COLS_BWD = 512;    // ... backward (1024 columns take 198 registers: 86 us for
                                      // 16384 fp32 rows with dres, the ring 45)
constexpr int ROWS_PER_CTA = 8;       // ... with this many warps a CTA

__device__ __forceinline__ void unpack8(uint4 u, float (&v)[8])
{
    v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x);
    v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
    v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z);
    v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8])
{
    return make_uint4(f32x2_to_bf16x2(v[1], v[0]), f32x2_to_bf16x2(v[3], v[2]),
                      f32x2_to_bf16x2(v[5], v[4]), f32x2_to_bf16x2(v[7], v[6]));
}

// 8 consecutive elements from `off` of a bf16 or fp32 array
template <bool F32>
__device__ __forceinline__ void load8(const void *p, size_t off, float (&v)[8])
{
    if (F32) {
        const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + off);
        const float4 a = q[0], b = q[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        unpack8(*reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + off), v);
    }
}

template <bool F32>
__device__ __forceinline__ void store8(void *p, size_t off, const float (&v)[8])
{
    if (F32) {
        float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + off);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + off) = pack8(v);
    }
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}

// Sum over the threads of a row: a warp (ONE) or the CTA.  `red` is used by one call at a
// time: the callers alternate two buffers, so one barrier a sum suffices.
template <bool ONE>
__device__ __forceinline__ float row_sum(float v, float *red)
{
    v = warp_sum(v);
    if (ONE) return v;
    const int nw = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < nw ? red[threadIdx.x & 31] : 0.f;
    return warp_sum(v);
}

// ONE: blockDim (32, ROWS_PER_CTA), a row per warp; else a row per CTA.
template <bool XF32, int VPT, bool ONE>
__global__ void __launch_bounds__(ONE ? 32 * ROWS_PER_CTA : 1024)
    norm_fwd_kernel(const void *__restrict__ x, const float *__restrict__ gamma,
                    const float *__restrict__ beta, int T, int H, float eps, uint16_t *__restrict__ y,
                    float *__restrict__ mean, float *__restrict__ rstd)
{
    __shared__ float red[2][32];
    pdl_wait();
    const int row = ONE ? blockIdx.x * ROWS_PER_CTA + threadIdx.y : blockIdx.x;
    if (row >= T) return;
    const size_t base = static_cast<size_t>(row) * H;
    float v[VPT][8];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = 8 * (threadIdx.x + i * blockDim.x);
        if (c < H) {
            load8<XF32>(x, base + c, v[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) s += v[i][j];
        }
    }
    const float inv = 1.f / static_cast<float>(H);
    const float mu = row_sum<ONE>(s, red[0]) * inv;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = 8 * (threadIdx.x + i * blockDim.x);
        if (c < H) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] -= mu;
                q = fmaf(v[i][j], v[i][j], q);
            }
        }
    }
    const float r = 1.f / sqrtf(row_sum<ONE>(q, red[1]) * inv + eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = 8 * (threadIdx.x + i * blockDim.x);
        if (c < H) {
            float g[8], b[8], o[8];
            load8<true>(gamma, c, g);
            if (beta) load8<true>(beta, c, b);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                o[j] = v[i][j] * r * g[j];
                if (beta) o[j] += b[j];
            }
            store8<false>(y, base + c, o);
        }
    }
    if (threadIdx.x == 0) {
        if (mean) mean[row] = mu;
        if (rstd) rstd[row] = r;
    }
}

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// After a wait that ran out, by the thread that issued the copies, fill f to stage f % S: those
// in flight land (the last S at most, each its stage's last) before the CTA leaves.
__device__ __forceinline__ void drain(uint64_t *full, int S, int fills)
{
    int dummy = 0;
    for (int f = max(0, fills - S); f < fills; ++f) mbar_wait(&full[f % S], (f / S) & 1u, &dummy, nullptr, 20000000ull);
}

template <bool F32>
__device__ __forceinline__ float4 load4(const void *p, int c)
{
    if (F32) return *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + c);
    const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + c);
    return make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
}

// Longer rows of a batch that gives every CTA several: the rows of x arrive by bulk copies in a
// ring of shared-memory stages, 4 x VPT columns a thread in registers from there.  A row's
// stage is filled again behind the barrier of its mean.  (A CTA per row, 448 threads of plain
// loads, took 154 us for 16384 rows of 7168 in fp32 and 163 us in bf16; this: 129 and 113 us, 5.5
// and 4.1 TB/s.  Two barriers a row bound it, not the loads: more CTAs an SM would need fewer
// registers.)  The entry point has no status word: a CTA whose wait runs out takes its rows from
// there on by plain loads, so the results hold.
struct NormFwd {
    const void *x;
    const float *gamma, *beta;     // beta nullable
    int T, H;
    float eps;
    uint16_t *y;
    float *mean, *rstd;            // nullable
    int stages, stage_bytes;
    unsigned long long timeout_ns;
    int inject;                    // no copies: every wait runs out (testing)
};

// Rows `row`, + step, ... of the forward ring without it, by the whole CTA (out of line: rare).
template <bool XF32>
__device__ __noinline__ void norm_rows(const NormFwd &p, int row, int step, float (*red)[32])
{
    constexpr int XB = XF32 ? 4 : 2;
    const float inv = 1.f / static_cast<float>(p.H);
    for (; row < p.T; row += step) {
        const size_t base = static_cast<size_t>(row) * p.H;
        const unsigned char *x = static_cast<const unsigned char *>(p.x) + base * XB;
        float a = 0.f;
        for (int c = 4 * threadIdx.x; c < p.H; c += 4 * blockDim.x) {
            const float4 v = load4<XF32>(x, c);
            a += (v.x + v.y) + (v.z + v.w);
        }
        const float mu = row_sum<false>(a, red[0]) * inv;
        a = 0.f;
        for (int c = 4 * threadIdx.x; c < p.H; c += 4 * blockDim.x) {
            float4 v = load4<XF32>(x, c);
            v = make_float4(v.x - mu, v.y - mu, v.z - mu, v.w - mu);
            a += fmaf(v.x, v.x, v.y * v.y) + fmaf(v.z, v.z, v.w * v.w);
        }
        const float r = 1.f / sqrtf(row_sum<false>(a, red[1]) * inv + p.eps);
        for (int c = 4 * threadIdx.x; c < p.H; c += 4 * blockDim.x) {
            const float4 v = load4<XF32>(x, c), g = load4<true>(p.gamma, c);
            const float4 b = p.beta ? load4<true>(p.beta, c) : make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<uint2 *>(p.y + base + c) =
                make_uint2(f32x2_to_bf16x2((v.y - mu) * r * g.y + b.y, (v.x - mu) * r * g.x + b.x),
                           f32x2_to_bf16x2((v.w - mu) * r * g.w + b.w, (v.z - mu) * r * g.z + b.z));
        }
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[row] = mu;
            if (p.rstd) p.rstd[row] = r;
        }
    }
}

template <bool XF32, int VPT, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 512 ? 3 : 1) norm_fwd_ring_kernel(const __grid_constant__ NormFwd p)
{
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ float red[2][32];
    __shared__ uint64_t full[4];
    __shared__ int abort_s;
    volatile int *abort_flag = &abort_s;
    const int tid = threadIdx.x, S = p.stages, H = p.H;
    const int nw = blockDim.x >> 5;
    if (tid == 0) {
        for (int s = 0; s < S; ++s) mbar_init(&full[s], 1);
        abort_s = 0;
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait();
    constexpr int XB = XF32 ? 4 : 2;
    auto fill = [&](int row, int s) {
        mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(H) * XB);
        bulk_load(ring + static_cast<size_t>(s) * p.stage_bytes,
                  static_cast<const unsigned char *>(p.x) + static_cast<size_t>(row) * H * XB, H * XB, &full[s]);
    };
    const int step = gridDim.x;
    int ahead = blockIdx.x;                  // next row to fill (thread 0)
    if (tid == 0 && !p.inject)
        for (int s = 0; s < S && ahead < p.T; ++s, ahead += step) fill(ahead, s);
    const float inv = 1.f / static_cast<float>(H);
    int s = 0;
    uint32_t ph = 0;
    auto sum = [&](float v, float *r) {      // over the CTA; one barrier
        v = warp_sum(v);
        if ((tid & 31) == 0) r[tid >> 5] = v;
        __syncthreads();
        return warp_sum((tid & 31) < nw ? r[tid & 31] : 0.f);
    };
    int row = blockIdx.x;
    for (; row < p.T; row += step) {
        mbar_wait(&full[s], ph, abort_flag, nullptr, p.timeout_ns);
        const unsigned char *st = ring + static_cast<size_t>(s) * p.stage_bytes;
        float4 v[VPT];
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 4 * (tid + i * blockDim.x);
            v[i] = c < H ? load4<XF32>(st, c) : make_float4(0.f, 0.f, 0.f, 0.f);
            a += (v[i].x + v[i].y) + (v[i].z + v[i].w);
        }
        const float mu = sum(a, red[0]) * inv;
        // a wait of this row ran out for some thread (the flag of a later one's comes behind the
        // second barrier, so all threads leave together)
        if (*abort_flag) break;
        // (every thread has read the row: its stage takes a row further on)
        if (tid == 0 && ahead < p.T) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            fill(ahead, s);
            ahead += step;
        }
        a = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (4 * (tid + i * blockDim.x) >= H) continue;
            v[i] = make_float4(v[i].x - mu, v[i].y - mu, v[i].z - mu, v[i].w - mu);
            a += fmaf(v[i].x, v[i].x, v[i].y * v[i].y) + fmaf(v[i].z, v[i].z, v[i].w * v[i].w);
        }
        const float r = 1.f / sqrtf(sum(a, red[1]) * inv + p.eps);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 4 * (tid + i * blockDim.x);
            if (c >= H) continue;
            const float4 g = load4<true>(p.gamma, c);
            const float4 b = p.beta ? load4<true>(p.beta, c) : make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<uint2 *>(p.y + static_cast<size_t>(row) * H + c) =
                make_uint2(f32x2_to_bf16x2(v[i].y * r * g.y + b.y, v[i].x * r * g.x + b.x),
                           f32x2_to_bf16x2(v[i].w * r * g.w + b.w, v[i].z * r * g.z + b.z));
        }
        if (tid == 0) {
            if (p.mean) p.mean[row] = mu;
            if (p.rstd) p.rstd[row] = r;
        }
        if (++s == S) { s = 0; ph ^= 1u; }
    }
    if (row < p.T) {
        if (tid == 0) drain(full, S, (ahead - static_cast<int>(blockIdx.x)) / step);
        norm_rows<XF32>(p, row, step, red);
    }
}

struct NormBwd {
    const uint16_t *dy;
    const void *x;
    const float *gamma, *mean, *rstd;
    const void *dres;      // nullable, the type of x
    void *dx;
    float *part;           // [gridDim.x][2][H]
    int T, H;
    // rows longer than WARP_COLS_BWD: stages of the ring, whether they hold dres, the offsets of
    // dy and dres in a stage, its bytes
    int stages, res_staged, off_dy, off_res, stage_bytes;
    int *status;
    unsigned long long timeout_ns;
    int inject;            // no copies: every wait runs out (testing)
};

// Rows of up to WARP_COLS_BWD columns: a warp per row, its weight sums in registers; the CTA's
// warps' sums are added in warp order.
template <bool XF32, int VPT>
__global__ void __launch_bounds__(32 * ROWS_PER_CTA) norm_bwd_warp_kernel(const NormBwd p)
{
    __shared__ float comb[ROWS_PER_CTA][32 * 8];
    pdl_wait();
    const int lane = threadIdx.x;
    float g[VPT][8], dg[VPT][8], db[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = 8 * (lane + 32 * i);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[i][j] = dg[i][j] = db[i][j] = 0.f;
        if (c < p.H) load8<true>(p.gamma, c, g[i]);
    }
    const float inv = 1.f / static_cast<float>(p.H);
    for (int row = blockIdx.x * ROWS_PER_CTA + threadIdx.y; row < p.T; row += gridDim.x * ROWS_PER_CTA) {
        const size_t base = static_cast<size_t>(row) * p.H;
        const float mu = p.mean[row], r = p.rstd[row];
        float xh[VPT][8], a[VPT][8];
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 8 * (lane + 32 * i);
            if (c < p.H) {
                load8<XF32>(p.x, base + c, xh[i]);
                load8<false>(p.dy, base + c, a[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    xh[i][j] = (xh[i][j] - mu) * r;
                    dg[i][j] = fmaf(a[i][j], xh[i][j], dg[i][j]);
                    db[i][j] += a[i][j];
                    a[i][j] *= g[i][j];
                    s0 += a[i][j];
                    s1 = fmaf(a[i][j], xh[i][j], s1);
                }
            }
        }
        s0 = warp_sum(s0) * inv;
        s1 = warp_sum(s1) * inv;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 8 * (lane + 32 * i);
            if (c < p.H) {
                float e[8];
                if (p.dres) load8<XF32>(p.dres, base + c, e);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    a[i][j] = r * (a[i][j] - s0 - xh[i][j] * s1);
                    if (p.dres) a[i][j] += e[j];
                }
                store8<XF32>(p.dx, base + c, a[i]);
            }
        }
    }
    float *part = p.part + static_cast<size_t>(blockIdx.x) * 2 * p.H;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 8 * (lane + 32 * i);
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j) comb[threadIdx.y][j * 32 + lane] = w ? db[i][j] : dg[i][j];
            __syncthreads();
            // thread (lane, warp y) adds element y of every warp's vector
            float t = 0.f;
#pragma unroll
            for (int y = 0; y < ROWS_PER_CTA; ++y) t += comb[y][threadIdx.y * 32 + lane];
            if (c < p.H) part[w * p.H + c + threadIdx.y] = t;
        }
    }
}

// Longer rows: a CTA per row, 4 x VPT columns a thread.  The rows x, dy (and dres) of the CTA
// arrive by bulk copies in a ring of shared-memory stages, so that loads never wait for a
// row's two sums (plain loads before and after the barriers of two CTAs an SM: 402 us for
// 16384 rows of 7168 in fp32 with dres, 4.1 TB/s; this: 247 us, 6.7 TB/s, 98% of the copy bandwidth).
// One barrier a row: its sums; a row's stage is filled again behind the next row's.  GREG: gamma
// stays in registers.
template <bool XF32, int VPT, bool GREG, int MAXT, int CTAS>
__global__ void __launch_bounds__(MAXT, CTAS) norm_bwd_ring_kernel(const NormBwd p)
{
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ float2 red[2][32];
    __shared__ uint64_t full[4];
    __shared__ int abort_s;
    volatile int *abort_flag = &abort_s;
    const int tid = threadIdx.x, S = p.stages, H = p.H;
    const int nw = blockDim.x >> 5;
    if (tid == 0) {
        for (int s = 0; s < S; ++s) mbar_init(&full[s], 1);
        abort_s = 0;
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait();
    constexpr int XB = XF32 ? 4 : 2;
    auto fill = [&](int row, int s) {
        unsigned char *st = ring + static_cast<size_t>(s) * p.stage_bytes;
        const size_t base = static_cast<size_t>(row) * H;
        mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(H) * (2 + XB + (p.res_staged ? XB : 0)));
        bulk_load(st, static_cast<const unsigned char *>(p.x) + base * XB, H * XB, &full[s]);
        bulk_load(st + p.off_dy, p.dy + base, H * 2, &full[s]);
        if (p.res_staged) bulk_load(st + p.off_res, static_cast<const unsigned char *>(p.dres) + base * XB, H * XB, &full[s]);
    };
    const int first = blockIdx.x, step = gridDim.x;
    int ahead = first;                       // next row to fill (thread 0)
    if (tid == 0 && !p.inject)
        for (int s = 0; s < S && ahead < p.T; ++s, ahead += step) fill(ahead, s);
    float4 g[GREG ? VPT : 1], dg[VPT], db[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = 4 * (tid + i * blockDim.x);
        if (GREG) g[i % (GREG ? VPT : 1)] = c < H ? load4<true>(p.gamma, c) : make_float4(0.f, 0.f, 0.f, 0.f);
        dg[i] = db[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const float inv = 1.f / static_cast<float>(H);
    int s = 0, prev = -1, k = 0;
    uint32_t ph = 0;
    for (int row = first; row < p.T; row += step, k ^= 1) {
        const float mu = p.mean[row], r = p.rstd[row];
        // (a wait that runs out is recorded; the row's results are then void)
        mbar_wait(&full[s], ph, abort_flag, p.status, p.timeout_ns);
        const unsigned char *st = ring + static_cast<size_t>(s) * p.stage_bytes;
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 4 * (tid + i * blockDim.x);
            if (c >= H) continue;
            const float4 x = load4<XF32>(st, c), d = load4<false>(st + p.off_dy, c);
            const float4 gm = GREG ? g[i % (GREG ? VPT : 1)] : load4<true>(p.gamma, c);
            const float4 h = make_float4((x.x - mu) * r, (x.y - mu) * r, (x.z - mu) * r, (x.w - mu) * r);
            dg[i].x = fmaf(d.x, h.x, dg[i].x); dg[i].y = fmaf(d.y, h.y, dg[i].y);
            dg[i].z = fmaf(d.z, h.z, dg[i].z); dg[i].w = fmaf(d.w, h.w, dg[i].w);
            db[i].x += d.x; db[i].y += d.y; db[i].z += d.z; db[i].w += d.w;
            const float4 a = make_float4(gm.x * d.x, gm.y * d.y, gm.z * d.z, gm.w * d.w);
            s0 += (a.x + a.y) + (a.z + a.w);
            s1 += fmaf(a.x, h.x, a.y * h.y) + fmaf(a.z, h.z, a.w * h.w);
        }
        s0 = warp_sum(s0);
        s1 = warp_sum(s1);
        if ((tid & 31) == 0) red[k][tid >> 5] = make_float2(s0, s1);
        __syncthreads();
        // every thread is done with the row before: its stage takes a row further on
        if (tid == 0 && prev >= 0 && ahead < p.T && !*abort_flag) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            fill(ahead, prev);
            ahead += step;
        }
        const float2 q = (tid & 31) < nw ? red[k][tid & 31] : make_float2(0.f, 0.f);
        s0 = warp_sum(q.x) * inv;
        s1 = warp_sum(q.y) * inv;
        const size_t base = static_cast<size_t>(row) * H;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 4 * (tid + i * blockDim.x);
            if (c >= H) continue;
            const float4 x = load4<XF32>(st, c), d = load4<false>(st + p.off_dy, c);
            const float4 gm = GREG ? g[i % (GREG ? VPT : 1)] : load4<true>(p.gamma, c);
            float4 o;
            o.x = r * (gm.x * d.x - s0 - (x.x - mu) * r * s1);
            o.y = r * (gm.y * d.y - s0 - (x.y - mu) * r * s1);
            o.z = r * (gm.z * d.z - s0 - (x.z - mu) * r * s1);
            o.w = r * (gm.w * d.w - s0 - (x.w - mu) * r * s1);
            if (p.dres) {
                const float4 e = p.res_staged ? load4<XF32>(st + p.off_res, c)
                                              : load4<XF32>(static_cast<const unsigned char *>(p.dres) + base * XB, c);
                o.x += e.x; o.y += e.y; o.z += e.z; o.w += e.w;
            }
            if (XF32)
                *reinterpret_cast<float4 *>(static_cast<float *>(p.dx) + base + c) = o;
            else
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.dx) + base + c) =
                    make_uint2(f32x2_to_bf16x2(o.y, o.x), f32x2_to_bf16x2(o.w, o.z));
        }
        prev = s;
        if (++s == S) { s = 0; ph ^= 1u; }
    }
    __syncthreads();
    if (*abort_flag && tid == 0) drain(full, S, (ahead - first) / step);
    float *part = p.part + static_cast<size_t>(blockIdx.x) * 2 * H;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = 4 * (tid + i * blockDim.x);
        if (c >= H) continue;
        *reinterpret_cast<float4 *>(part + c) = dg[i];
        *reinterpret_cast<float4 *>(part + H + c) = db[i];
    }
}

// dgamma | dbeta = sums of the CTAs' partial rows [n][2 H], in order: 32 columns x 8 row
// strands a CTA.
__global__ void __launch_bounds__(256) norm_wgrad_kernel(const float *__restrict__ part, int n, int H,
                                                         float *__restrict__ dgamma,
                                                         float *__restrict__ dbeta)
{
    __shared__ float s[8][32];
    pdl_wait();
    const int c = blockIdx.x * 32 + threadIdx.x;      // (2 H is a multiple of 32)
    float v = 0.f;
    for (int r = threadIdx.y; r < n; r += 8) v += part[static_cast<size_t>(r) * 2 * H + c];
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y == 0) {
        for (int k = 1; k < 8; ++k) v += s[k][threadIdx.x];
        if (c < H) dgamma[c] = v;
        else dbeta[c - H] = v;
    }
}

int cta_threads(int H, int vpt) { return (H / 8 + vpt * 32 - 1) / (vpt * 32) * 32; }

constexpr size_t RING_BYTES = 220 * 1024;     // shared memory of an SM for the rings

int ring_threads(int H, int vpt) { return (H / 4 + vpt * 32 - 1) / (vpt * 32) * 32; }

// Persistent CTAs of the forward ring: as many an SM as threads and two stages a CTA allow
int fwd_ctas(int H, int xb)
{
    const int by_room = static_cast<int>(RING_BYTES / (2 * static_cast<size_t>(H) * xb)), by_threads = 1536 / ring_threads(H, 4);
    const int n = by_room < by_threads ? by_room : by_threads;
    return num_sms() * (n < 1 ? 1 : n);
}

template <bool XF32, int VPT, int MAXT>
cudaError_t fwd_ring(const NormFwd &p, int ctas, cudaStream_t s)
{
    const size_t smem = static_cast<size_t>(p.stages) * p.stage_bytes;
    const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(norm_fwd_ring_kernel<XF32, VPT, MAXT>), smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(norm_fwd_ring_kernel<XF32, VPT, MAXT>, dim3(ctas), dim3(ring_threads(p.H, VPT)),
                      smem, s, 1, p);
}

template <bool XF32>
cudaError_t fwd(const void *x, const float *gamma, const float *beta, int T, int H, float eps, uint16_t *y,
                float *mean, float *rstd, unsigned long long timeout_ns, int inject, cudaStream_t s)
{
    const dim3 warps(32, ROWS_PER_CTA), gw((T + ROWS_PER_CTA - 1) / ROWS_PER_CTA);
    if (H <= 256) return launch_pdl(norm_fwd_kernel<XF32, 1, true>, gw, warps, 0, s, 1, x, gamma, beta, T, H, eps, y, mean, rstd);
    if (H <= 512) return launch_pdl(norm_fwd_kernel<XF32, 2, true>, gw, warps, 0, s, 1, x, gamma, beta, T, H, eps, y, mean, rstd);
    if (H <= WARP_COLS) return launch_pdl(norm_fwd_kernel<XF32, 4, true>, gw, warps, 0, s, 1, x, gamma, beta, T, H, eps, y, mean, rstd);
    // (up to eight rows a CTA of the ring, the plain launch's parallel rows are as fast)
    const int ctas = fwd_ctas(H, XF32 ? 4 : 2);
    if (T >= 8 * ctas) {
        NormFwd p{x, gamma, beta, T, H, eps, y, mean, rstd, 0, H * (XF32 ? 4 : 2), timeout_ns, inject};
        const size_t room = RING_BYTES / (ctas / num_sms());
        p.stages = static_cast<int>(room / p.stage_bytes < 4 ? room / p.stage_bytes : 4);
        return H <= 8192 ? fwd_ring<XF32, 4, 512>(p, ctas, s) : fwd_ring<XF32, 4, 1024>(p, ctas, s);
    }
    return launch_pdl(norm_fwd_kernel<XF32, 2, false>, dim3(T), dim3(cta_threads(H, 2)), 0, s, 1, x, gamma, beta, T, H, eps, y, mean, rstd);
}

// Rows longer than WARP_COLS_BWD: the ring's stages (two at least; three and four where they fit
// with dres, which is otherwise loaded directly) and its shared memory.
size_t plan_ring(NormBwd &p, int xb, bool res, int per_sm)
{
    const size_t room = RING_BYTES / per_sm;
    auto stage = [&](bool with) { return static_cast<size_t>(p.H) * (xb + 2 + (with ? xb : 0)); };
    const bool staged = res && 2 * stage(true) <= room;
    const size_t b = stage(staged);
    p.res_staged = staged ? 1 : 0;
    p.stages = static_cast<int>(room / b < 4 ? room / b : 4);
    p.off_dy = p.H * xb;
    p.off_res = p.H * (xb + 2);
    p.stage_bytes = static_cast<int>(b);
    return b * p.stages;
}

// CTAs of the ring that share an SM: 1024 threads, where two stages of their rows fit.  One CTA a
// row of 7168 leaves the SM idle between a row's barriers (bf16 without dres, 16384 rows: 190 us
// with one, 165 us with two).
int ring_ctas(int H, int row_bytes)
{
    const int most = 1024 / ring_threads(H, H <= 2048 ? 2 : 4);
    const int n = static_cast<int>(RING_BYTES / (2 * static_cast<size_t>(row_bytes)));
    return n < 1 ? 1 : (n < most ? n : most);
}

template <bool XF32, int VPT, bool GREG, int MAXT, int CTAS>
cudaError_t ring(NormBwd &p, int per_sm, int n, cudaStream_t s)
{
    const size_t smem = plan_ring(p, XF32 ? 4 : 2, p.dres != nullptr, per_sm);
    const void *fn = reinterpret_cast<const void *>(norm_bwd_ring_kernel<XF32, VPT, GREG, MAXT, CTAS>);
    const cudaError_t e = ensure_smem(fn, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(norm_bwd_ring_kernel<XF32, VPT, GREG, MAXT, CTAS>, dim3(n), dim3(ring_threads(p.H, VPT)),
                      smem, s, 1, p);
}

// n: CTAs launched
template <bool XF32>
cudaError_t bwd(NormBwd &p, int &n, cudaStream_t s)
{
    const dim3 warps(32, ROWS_PER_CTA);
    if (p.H <= WARP_COLS_BWD) {
        n = norm_bwd_ctas(p.T, p.H);
        if (p.H <= 256) return launch_pdl(norm_bwd_warp_kernel<XF32, 1>, dim3(n), warps, 0, s, 1, p);
        return launch_pdl(norm_bwd_warp_kernel<XF32, 2>, dim3(n), warps, 0, s, 1, p);
    }
    constexpr int XB = XF32 ? 4 : 2;
    const int per_sm = ring_ctas(p.H, p.H * (2 + XB + (p.dres ? XB : 0)));
    n = per_sm * num_sms();
    if (n > p.T) n = p.T;
    if (p.H <= 2048) return ring<XF32, 2, true, 256, 4>(p, per_sm, n, s);
    if (p.H > 8192) return ring<XF32, 4, false, 1024, 1>(p, per_sm, n, s);
    return per_sm > 1 ? ring<XF32, 4, false, 512, 2>(p, per_sm, n, s) : ring<XF32, 4, true, 512, 1>(p, per_sm, n, s);
}

}  // namespace

// CTAs of the backward launch at most, for any type (their partial sums take 8 H bytes each).
int norm_bwd_ctas(int T, int H)
{
    const int units = H <= WARP_COLS_BWD ? (T + ROWS_PER_CTA - 1) / ROWS_PER_CTA : T;
    const int most = (H <= WARP_COLS_BWD ? 2 : ring_ctas(H, 4 * H)) * num_sms();
    return units < most ? (units > 0 ? units : 1) : most;
}

cudaError_t launch_norm(const void *x, int x_fp32, const float *gamma, const float *beta, int T, int H,
                        float eps, void *y, float *mean, float *rstd, unsigned long long timeout_ns, int inject,
                        cudaStream_t s)
{
    uint16_t *o = static_cast<uint16_t *>(y);
    return x_fp32 ? fwd<true>(x, gamma, beta, T, H, eps, o, mean, rstd, timeout_ns, inject, s)
                  : fwd<false>(x, gamma, beta, T, H, eps, o, mean, rstd, timeout_ns, inject, s);
}

cudaError_t launch_norm_bwd(const void *dy, const void *x, int x_fp32, const float *gamma, const float *mean,
                            const float *rstd, const void *dres, int T, int H, void *dx, float *dgamma,
                            float *dbeta, float *part, int *status, unsigned long long timeout_ns,
                            int inject, cudaStream_t s)
{
    NormBwd p{static_cast<const uint16_t *>(dy), x, gamma, mean, rstd, dres, dx, part, T, H, 0, 0, 0, 0, 0,
              status, timeout_ns, inject};
    int n = 0;
    const cudaError_t e = x_fp32 ? bwd<true>(p, n, s) : bwd<false>(p, n, s);
    if (e != cudaSuccess) return e;
    return launch_pdl(norm_wgrad_kernel, dim3(2 * H / 32), dim3(32, 8), 0, s, 1, static_cast<const float *>(part),
                      n, H, dgamma, dbeta);
}

}  // namespace moe
