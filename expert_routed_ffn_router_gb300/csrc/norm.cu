// norm.cu -- layer norm of the token rows in front of the layer, and its backward pass.
//
//   forward   mu = mean(x), r = (mean((x - mu)^2) + eps)^-1/2, y = gamma (x - mu) r + beta
//   backward  a = gamma dy, xh = (x - mu) r,
//             dx = r (a - mean(a) - xh mean(a xh)) (+ dres),
//             dgamma = sum_t dy xh, dbeta = sum_t dy
//
// Both are bound by memory: every row is read once and kept in registers, the variance is
// taken from the centred values (no sum of squares, which cancels for rows far from zero),
// and all sums are fp32.  Rows of up to 1024 columns take one warp each, longer ones a CTA.
//
// Weight gradients.  Each CTA walks rows blockIdx.x, + gridDim.x, ... and keeps the sums of
// its columns in registers; the CTAs' sums go to the workspace ([CTA][2][H]) and a second
// launch adds them in CTA order.  No atomics: the result depends on the sizes alone.
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int WARP_COLS = 1024;       // longest row that one warp takes
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

struct NormBwd {
    const uint16_t *dy;
    const void *x;
    const float *gamma, *mean, *rstd;
    const void *dres;      // nullable, the type of x
    void *dx;
    float *part;           // [gridDim.x][2][H]
    int T, H;
};

// One row of the backward pass from this thread's columns; adds to its weight sums.
template <bool XF32, int VPT, bool ONE>
__device__ __forceinline__ void norm_bwd_row(const NormBwd &p, int row, const float (&g)[VPT][8],
                                             float (&dg)[VPT][8], float (&db)[VPT][8], float (*red)[32])
{
    const size_t base = static_cast<size_t>(row) * p.H;
    const float mu = p.mean[row], r = p.rstd[row];
    float xh[VPT][8], a[VPT][8];
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = 8 * (threadIdx.x + i * blockDim.x);
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
    const float inv = 1.f / static_cast<float>(p.H);
    s0 = row_sum<ONE>(s0, red[0]) * inv;
    s1 = row_sum<ONE>(s1, red[1]) * inv;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = 8 * (threadIdx.x + i * blockDim.x);
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

template <bool XF32, int VPT, bool ONE, int MAXT = 32 * ROWS_PER_CTA>
__global__ void __launch_bounds__(MAXT) norm_bwd_kernel(const NormBwd p)
{
    __shared__ float red[4][32];
    __shared__ float comb[ONE ? ROWS_PER_CTA : 1][ONE ? 32 * 8 : 1];
    pdl_wait();
    float g[VPT][8], dg[VPT][8], db[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = 8 * (threadIdx.x + i * blockDim.x);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[i][j] = dg[i][j] = db[i][j] = 0.f;
        if (c < p.H) load8<true>(p.gamma, c, g[i]);
    }
    if (ONE) {
        for (int row = blockIdx.x * ROWS_PER_CTA + threadIdx.y; row < p.T; row += gridDim.x * ROWS_PER_CTA)
            norm_bwd_row<XF32, VPT, ONE>(p, row, g, dg, db, red);
    } else {
        int k = 0;
        for (int row = blockIdx.x; row < p.T; row += gridDim.x, k ^= 2)
            norm_bwd_row<XF32, VPT, ONE>(p, row, g, dg, db, red + k);
    }
    // the CTA's sums (ONE: its warps' sums added in warp order)
    float *part = p.part + static_cast<size_t>(blockIdx.x) * 2 * p.H;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 8 * (threadIdx.x + i * blockDim.x);
            float(&v)[8] = w ? db[i] : dg[i];
            if (ONE) {
                __syncthreads();
#pragma unroll
                for (int j = 0; j < 8; ++j) comb[threadIdx.y][j * 32 + threadIdx.x] = v[j];
                __syncthreads();
                // thread (lane, warp y) adds element y of every warp's vector
                float t = 0.f;
#pragma unroll
                for (int y = 0; y < ROWS_PER_CTA; ++y) t += comb[y][threadIdx.y * 32 + threadIdx.x];
                if (c < p.H) part[w * p.H + c + threadIdx.y] = t;
            } else if (c < p.H) {
                store8<true>(part, static_cast<size_t>(w) * p.H + c, v);
            }
        }
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

template <bool XF32>
cudaError_t fwd(const void *x, const float *gamma, const float *beta, int T, int H, float eps, uint16_t *y,
                float *mean, float *rstd, cudaStream_t s)
{
    const dim3 warps(32, ROWS_PER_CTA), gw((T + ROWS_PER_CTA - 1) / ROWS_PER_CTA);
    if (H <= 256) return launch_pdl(norm_fwd_kernel<XF32, 1, true>, gw, warps, 0, s, 1, x, gamma, beta, T, H, eps, y, mean, rstd);
    if (H <= 512) return launch_pdl(norm_fwd_kernel<XF32, 2, true>, gw, warps, 0, s, 1, x, gamma, beta, T, H, eps, y, mean, rstd);
    if (H <= WARP_COLS) return launch_pdl(norm_fwd_kernel<XF32, 4, true>, gw, warps, 0, s, 1, x, gamma, beta, T, H, eps, y, mean, rstd);
    return launch_pdl(norm_fwd_kernel<XF32, 2, false>, dim3(T), dim3(cta_threads(H, 2)), 0, s, 1, x, gamma, beta, T, H, eps, y, mean, rstd);
}

template <bool XF32>
cudaError_t bwd(const NormBwd &p, int n, cudaStream_t s)
{
    const dim3 warps(32, ROWS_PER_CTA), g(n);
    if (p.H <= 256) return launch_pdl(norm_bwd_kernel<XF32, 1, true>, g, warps, 0, s, 1, p);
    if (p.H <= 512) return launch_pdl(norm_bwd_kernel<XF32, 2, true>, g, warps, 0, s, 1, p);
    if (p.H <= WARP_COLS) return launch_pdl(norm_bwd_kernel<XF32, 4, true>, g, warps, 0, s, 1, p);
    // (up to 8192 columns 512 threads of at most 128 registers; the longest rows spill)
    if (p.H <= 8192) return launch_pdl(norm_bwd_kernel<XF32, 2, false, 512>, g, dim3(cta_threads(p.H, 2)), 0, s, 1, p);
    return launch_pdl(norm_bwd_kernel<XF32, 2, false, 1024>, g, dim3(cta_threads(p.H, 2)), 0, s, 1, p);
}

}  // namespace

// CTAs of the backward launch: as many rows in flight as fit, so that the partial sums (8 H
// bytes a CTA) stay small beside the rows.
int norm_bwd_ctas(int T, int H)
{
    const int units = H <= WARP_COLS ? (T + ROWS_PER_CTA - 1) / ROWS_PER_CTA : T;
    const int most = 2 * num_sms();
    return units < most ? (units > 0 ? units : 1) : most;
}

cudaError_t launch_norm(const void *x, int x_fp32, const float *gamma, const float *beta, int T, int H,
                        float eps, void *y, float *mean, float *rstd, cudaStream_t s)
{
    uint16_t *o = static_cast<uint16_t *>(y);
    return x_fp32 ? fwd<true>(x, gamma, beta, T, H, eps, o, mean, rstd, s)
                  : fwd<false>(x, gamma, beta, T, H, eps, o, mean, rstd, s);
}

cudaError_t launch_norm_bwd(const void *dy, const void *x, int x_fp32, const float *gamma, const float *mean,
                            const float *rstd, const void *dres, int T, int H, void *dx, float *dgamma,
                            float *dbeta, float *part, cudaStream_t s)
{
    NormBwd p{static_cast<const uint16_t *>(dy), x, gamma, mean, rstd, dres, dx, part, T, H};
    const int n = norm_bwd_ctas(T, H);
    const cudaError_t e = x_fp32 ? bwd<true>(p, n, s) : bwd<false>(p, n, s);
    if (e != cudaSuccess) return e;
    return launch_pdl(norm_wgrad_kernel, dim3(2 * H / 32), dim3(32, 8), 0, s, 1, static_cast<const float *>(part),
                      n, H, dgamma, dbeta);
}

}  // namespace moe
