// residual.cuh -- what the forward (residual_fwd.cu) and the backward pass (residual_bwd.cu) of the joined
// residual share: the rows' threads, their columns and their copies.
//
//   forward   b = post(y),  r = alpha x + g_t g_h b,  n = pre(r)
//             post, pre: none, layer norm or RMS norm (gamma, beta); g_h a gate for each channel,
//             g_t one for each token
//   backward  d  = dr + pre'(dn)                  the stream's gradient
//             dx = alpha d
//             dy = post'(g_t g_h d)
//             dgamma_pre = sum_t dn rh, dbeta_pre = sum_t dn                  (rh, yh: normalised rows)
//             S1 = sum_t g_t d yh, S0 = sum_t g_t d:  dgamma_post = g_h S1, dbeta_post = g_h S0,
//             dgate_h = gamma_post S1 + beta_post S0;  dgate_t = sum_h g_h d b
//   with norm'(a) = rstd (a - [layer] mean(a) - xh mean(a xh)),  a = gamma times the gradient
//
// Both are bound by memory: every row is read and written once.  A row is taken by a warp (up to 512
// columns) or by a CTA of N threads, each of which has the columns 4 tid .. 4 tid + 3 of every 4 N, VPT
// times at most; N is known to the kernel, so that a thread's columns lie at fixed distances.  The
// rows arrive ahead of time by asynchronous copies; every thread copies the columns that it will read
// itself, so nothing but the sums of a row crosses threads.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace residual {

constexpr int VPT = 4;               // vectors of 4 columns a thread
constexpr int WARP_COLS = 32 * 4 * VPT;   // longest row of one warp
constexpr int WARPS = 8;             // rows of a CTA then
constexpr size_t ROOM = 220 * 1024;  // shared memory of an SM for the staged rows of several CTAs
constexpr size_t MOST = 225 * 1024;  // of one CTA, beside its static arrays

struct Args {
    ResidualOpts o;
    int T, H, x_fp32, y_fp32;
    const void *x, *y, *dr;          // dr nullable
    const uint16_t *dn;
    void *r;                         // forward: out; backward: in
    uint16_t *n;
    float4 *stats;                   // [T]: mean and rstd of y, of r
    void *dx;
    uint16_t *dy;
    float *d_token, *part;           // part [CTAs][4][H]: dgamma_pre, dbeta_pre, S1, S0
    ResidualGrads g;                 // backward: the CTAs are one cluster, which adds its own sums (joined)
    int joined;
    int stages, stage_bytes;         // of a row's threads
    int row_bytes, dr_once;          // backward: shared memory of a row's threads; dr is staged once
    int off[4];                      // the staged arrays in a stage, -1: read directly
    int sum[2];                      // backward: two of the sums in shared memory
};

// The type of an array: known to the kernel, or (RUNTIME) told by a flag.
enum { BF16, FP32, RUNTIME };

template <int TY>
__device__ __forceinline__ bool wide(bool fp32) { return TY == RUNTIME ? fp32 : TY == FP32; }

// Vector k N of 4 elements from `p` on (this thread's first vector)
template <int TY, int N>
__device__ __forceinline__ float4 ld4(const void *p, int k, bool fp32)
{
    if (wide<TY>(fp32)) return static_cast<const float4 *>(p)[k * N];
    const uint2 u = static_cast<const uint2 *>(p)[k * N];
    return make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
}

template <int TY, int N>
__device__ __forceinline__ void st4(void *p, int k, bool fp32, float4 v)
{
    if (wide<TY>(fp32)) static_cast<float4 *>(p)[k * N] = v;
    else static_cast<uint2 *>(p)[k * N] = make_uint2(f32x2_to_bf16x2(v.y, v.x), f32x2_to_bf16x2(v.w, v.z));
}

// This thread's first vector of row `row` of an array
template <int TY>
__device__ __forceinline__ unsigned char *row_at(const void *p, int row, int H, int tid, bool fp32)
{
    return const_cast<unsigned char *>(static_cast<const unsigned char *>(p)) +
           (static_cast<size_t>(row) * H + 4 * tid) * (wide<TY>(fp32) ? 4 : 2);
}

__device__ __forceinline__ float sum4(float4 v) { return (v.x + v.y) + (v.z + v.w); }
__device__ __forceinline__ float dot4(float4 a, float4 b) { return fmaf(a.x, b.x, a.y * b.y) + fmaf(a.z, b.z, a.w * b.w); }
__device__ __forceinline__ float4 add4(float4 a, float4 b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); }
// (rounded products, never part of an fma: which one the compiler forms would depend on the branch
// around it, and dx and dy on which gradients are wanted)
__device__ __forceinline__ float4 mul4(float4 a, float4 b)
{
    return make_float4(__fmul_rn(a.x, b.x), __fmul_rn(a.y, b.y), __fmul_rn(a.z, b.z), __fmul_rn(a.w, b.w));
}
__device__ __forceinline__ float4 scale4(float4 a, float s) { return mul4(a, make_float4(s, s, s, s)); }
__device__ __forceinline__ float4 norm4(float4 v, float m, float s)
{
    return make_float4((v.x - m) * s, (v.y - m) * s, (v.z - m) * s, (v.w - m) * s);
}
__device__ __forceinline__ float4 fma4(float4 a, float4 b, float4 c)
{
    return make_float4(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y), fmaf(a.z, b.z, c.z), fmaf(a.w, b.w, c.w));
}
__device__ __forceinline__ float4 all4(float v) { return make_float4(v, v, v, v); }

// Vector k of a parameter of the columns, `absent` where there is none
template <int N>
__device__ __forceinline__ float4 col4(const float *p, int tid, int k, float absent)
{
    return p ? reinterpret_cast<const float4 *>(p)[tid + k * N] : all4(absent);
}

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// The copies of all groups but the last `left` (at most 5) have arrived.
__device__ __forceinline__ void copies_wait(int left)
{
    if (left == 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (left == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else if (left == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (left == 3) asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (left == 4) asm volatile("cp.async.wait_group 4;" ::: "memory");
    else asm volatile("cp.async.wait_group 5;" ::: "memory");
}

template <int BYTES, int OFF>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src)
{
    if (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %2], 16;" ::"r"(dst), "l"(src), "n"(OFF) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0 + %2], [%1 + %2], 8;" ::"r"(dst), "l"(src), "n"(OFF) : "memory");
}

// The columns' vectors that a thread has: the first SURE ones always (row_threads)
template <int N>
struct Columns {
    static constexpr int SURE = N == 32 ? 0 : (N == 448 ? 3 : 2);
    int vec, tid;                    // vectors of a row, thread in the row
    __device__ __forceinline__ bool operator()(int k) const { return k < SURE || tid + k * N < vec; }
};

template <int BYTES, int N, int K = 0>
__device__ __forceinline__ void copy_row(uint32_t dst, const void *src, const Columns<N> &in)
{
    if constexpr (K < VPT) {
        if (in(K)) copy_async<BYTES, K * N * BYTES>(dst, src);
        copy_row<BYTES, N, K + 1>(dst, src, in);
    }
}

// The columns of this thread of row `row` of an array, to its place in a stage
template <int TY, int N>
__device__ __forceinline__ void stage_in(uint32_t st, const void *p, int row, int H, bool fp32, const Columns<N> &in)
{
    const unsigned char *src = row_at<TY>(p, row, H, in.tid, fp32);
    if (wide<TY>(fp32)) copy_row<16, N>(st + in.tid * 16, src, in);
    else copy_row<8, N>(st + in.tid * 8, src, in);
}

// This thread's first vector of an array in a stage
template <int TY>
__device__ __forceinline__ const unsigned char *staged(const unsigned char *st, int tid, bool fp32)
{
    return st + tid * (wide<TY>(fp32) ? 16 : 8);
}

// Sums of a and of b over the warp: that of a ends up in lanes 0 .. 15, that of b in lanes 16 .. 31 (half
// the shuffles of two sums).
__device__ __forceinline__ float warp_pair(float a, float b)
{
    const bool up = threadIdx.x & 16;
    float t = (up ? b : a) + __shfl_xor_sync(kFullMask, up ? a : b, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(kFullMask, t, o);
    return t;
}
// Both sums on every lane
__device__ __forceinline__ float2 warp_pair_all(float a, float b)
{
    const float t = warp_pair(a, b), u = __shfl_xor_sync(kFullMask, t, 16);
    return threadIdx.x & 16 ? make_float2(u, t) : make_float2(t, u);
}

// The warps of a row exchange four numbers each, through two buffers in turn: one barrier.
template <int N>
struct Exchange {
    float4 (*red)[N / 32];
    int tid;
    int turn = 0;

    // x, y: of lane 0 and of lane 16; z, w: likewise -> on lane k those of warp k, 0 beyond the last warp
    __device__ __forceinline__ float4 operator()(float xy, float zw)
    {
        float *r = reinterpret_cast<float *>(&red[turn][tid >> 5]);
        const int lane = tid & 31;
        if ((lane & 15) == 0) {
            r[lane >> 4] = xy;
            r[2 + (lane >> 4)] = zw;
        }
        __syncthreads();
        const float4 got = lane < N / 32 ? red[turn][lane] : make_float4(0.f, 0.f, 0.f, 0.f);
        turn ^= 1;
        return got;
    }
};

// Columns of warp `w` of a row
template <int N>
__device__ __forceinline__ float warp_columns(int H, int w)
{
    int k = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) k += max(0, min(128, H - 128 * w - 4 * i * N));
    return static_cast<float>(k);
}

// Threads of a row
inline int row_threads(int H) { return H <= WARP_COLS ? 32 : H <= 1024 ? 64 : H <= 2048 ? 128 : H <= 4096 ? 256 : H <= 8192 ? 512 : 1024; }

}  // namespace residual
}  // namespace moe
