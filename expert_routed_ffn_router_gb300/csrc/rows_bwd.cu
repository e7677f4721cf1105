// rows_bwd.cu -- gradients of the layer's two row movements, for experts whose own backward pass
// the caller has: of the combine (combine.cu) and of the dispatch's row gather (dispatch.cu).
//
//   combine    Y[t] = sum_j w[t, j] Yp[slot(t, j)]:
//              dYp[slot(t, j)] = w[t, j] dY[t],  dw[t, j] = <dY[t], Yp[slot(t, j)]>
//   dispatch   Xp[slot(t, j)] = X[t]:  dX[t] = sum_j dXp[slot(t, j)] (+ dres[t])
//
// Both go by the token: a slot's row belongs to one pair, so every row of Yp is read and every
// row of dYp written once, and no sum crosses tokens (no atomics, a fixed order).  Both are bound
// by memory: 16384 tokens x 7168, 8 slots, an fp32 gradient of the combine 617 us (6.85 TB/s, the copy
// bandwidth), the dispatch's with a second gradient added 345 us (6.8 TB/s).
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}

__device__ __forceinline__ void unpack8(uint4 u, float (&v)[8])
{
    v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x);
    v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
    v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z);
    v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
}

// 8 consecutive elements from element `off` (a multiple of 8) of a bf16 or fp32 array
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

// ---------------------------------------------------------------------------- combine
// A CTA a token: each thread holds CV vectors of 8 columns of dY (as many as the row needs, 4 at most,
// in turns beyond: 1777 x 2112, 3 slots: 15.4 us with 4, 11.7 us with the 2 that it needs) and goes through
// the token's slots with them; the row of the next slot is loaded before the one at hand is stored.  (dYp may
// be Yp's own memory: a thread has read what it overwrites, and no other one touches it.)
constexpr int CT = 256;

template <bool F32, bool DOT, int CV>
__global__ void __launch_bounds__(CT) combine_bwd_kernel(const void *__restrict__ dY, const uint4 *Yp,
                                                         const int32_t *__restrict__ slot_pos,
                                                         const float *__restrict__ topk_w, int H, int K,
                                                         uint4 *dYp, float *__restrict__ d_topk_w)
{
    __shared__ int row_s[32];
    __shared__ float w_s[32];
    __shared__ float part[32][CT / 32];
    pdl_wait();
    const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned n_rows = gridDim.x * static_cast<unsigned>(K);
    if (tid < K) {
        const size_t pair = static_cast<size_t>(t) * K + tid;
        const int r = slot_pos[pair];
        row_s[tid] = static_cast<unsigned>(r) < n_rows ? r : -1;
        w_s[tid] = topk_w ? topk_w[pair] : 1.f;
    }
    __syncthreads();
    const int vec = H / 8, span = blockDim.x * CV;
    for (int v0 = 0; v0 < vec; v0 += span) {
        float d[CV][8];
#pragma unroll
        for (int i = 0; i < CV; ++i) {
            const int c = v0 + tid + i * blockDim.x;
            if (c < vec) load8<F32>(dY, (static_cast<size_t>(t) * vec + c) * 8, d[i]);
        }
        uint4 next[DOT ? CV : 1];
        auto fetch = [&](int j) {
            if constexpr (DOT) {
                if (j >= K || row_s[j] < 0) return;
#pragma unroll
                for (int i = 0; i < CV; ++i) {
                    const int c = v0 + tid + i * blockDim.x;
                    if (c < vec) next[i] = Yp[static_cast<size_t>(row_s[j]) * vec + c];
                }
            }
        };
        fetch(0);
        for (int j = 0; j < K; ++j) {
            const int r = row_s[j];
            const float w = w_s[j];
            uint4 y[DOT ? CV : 1];
#pragma unroll
            for (int i = 0; i < (DOT ? CV : 1); ++i) y[i] = next[i];
            fetch(j + 1);
            float s = 0.f;
            if (r >= 0) {
#pragma unroll
                for (int i = 0; i < CV; ++i) {
                    const int c = v0 + tid + i * blockDim.x;
                    if (c >= vec) continue;
                    if (DOT) {
                        float v[8];
                        unpack8(y[i % (DOT ? CV : 1)], v);
#pragma unroll
                        for (int k = 0; k < 8; ++k) s = fmaf(d[i][k], v[k], s);
                    }
                    dYp[static_cast<size_t>(r) * vec + c] =
                        make_uint4(f32x2_to_bf16x2(w * d[i][1], w * d[i][0]), f32x2_to_bf16x2(w * d[i][3], w * d[i][2]),
                                   f32x2_to_bf16x2(w * d[i][5], w * d[i][4]), f32x2_to_bf16x2(w * d[i][7], w * d[i][6]));
                }
            }
            if (DOT) {
                s = warp_sum(s);
                if (lane == 0) part[j][warp] = v0 ? part[j][warp] + s : s;
            }
        }
    }
    if (!DOT) return;
    __syncthreads();
    const int nw = blockDim.x >> 5;
    for (int j = warp; j < K; j += nw) {
        const float s = warp_sum(lane < nw ? part[j][lane] : 0.f);
        if (lane == 0) d_topk_w[static_cast<size_t>(t) * K + j] = s;
    }
}

// --------------------------------------------------------------------------- dispatch
// A CTA 1024 columns of a token, as the combine; the rows of up to eight slots are in flight.
constexpr int DT = 128;

template <bool F32>
__global__ void __launch_bounds__(DT) dispatch_bwd_kernel(const uint4 *__restrict__ dXp,
                                                          const int32_t *__restrict__ slot_pos, const void *dres,
                                                          int H, int K, void *dX)
{
    __shared__ int row_s[32];
    pdl_wait();
    const int t = blockIdx.x;
    const unsigned n_rows = gridDim.x * static_cast<unsigned>(K);
    if (threadIdx.x < K) {
        const int r = slot_pos[static_cast<size_t>(t) * K + threadIdx.x];
        row_s[threadIdx.x] = static_cast<unsigned>(r) < n_rows ? r : -1;
    }
    __syncthreads();
    const int vec = H / 8, c = blockIdx.y * DT + threadIdx.x;
    if (c >= vec) return;
    const size_t at = (static_cast<size_t>(t) * vec + c) * 8;
    float a[8], e[8];
    if (dres) load8<F32>(dres, at, e);
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = 0.f;
    for (int j0 = 0; j0 < K; j0 += 8) {
        uint4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            v[u] = j0 + u < K && row_s[j0 + u] >= 0 ? __ldg(dXp + static_cast<size_t>(row_s[j0 + u]) * vec + c)
                                                    : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            float x[8];
            unpack8(v[u], x);
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] += x[i];
        }
    }
    if (dres)
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] += e[i];
    if (F32) {
        float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(dX) + at);
        o[0] = make_float4(a[0], a[1], a[2], a[3]);
        o[1] = make_float4(a[4], a[5], a[6], a[7]);
    } else {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(dX) + at) =
            make_uint4(f32x2_to_bf16x2(a[1], a[0]), f32x2_to_bf16x2(a[3], a[2]), f32x2_to_bf16x2(a[5], a[4]),
                       f32x2_to_bf16x2(a[7], a[6]));
    }
}

template <bool F32, bool DOT>
cudaError_t combine(const void *dY, const void *Yp, const int32_t *slot_pos, const float *topk_w, int T, int H,
                    int K, void *dYp, float *d_topk_w, cudaStream_t s)
{
    // threads such that every one has the same number of vectors, where the row allows it
    const int vec = H / 8, rounds = (vec + CT - 1) / CT;
    const int threads = ((vec + rounds - 1) / rounds + 31) / 32 * 32;
    // (fewer vectors, fewer registers, more rows on their way: 1777 x 2112, 3 slots: 15.4 us with 4, 11.7 us with 2)
    const auto kernel = rounds == 1 ? combine_bwd_kernel<F32, DOT, 1>
                                    : (rounds == 2 ? combine_bwd_kernel<F32, DOT, 2> : combine_bwd_kernel<F32, DOT, 4>);
    return launch_pdl(kernel, dim3(T), dim3(threads), 0, s, 1, dY, static_cast<const uint4 *>(Yp), slot_pos, topk_w, H, K,
                      static_cast<uint4 *>(dYp), d_topk_w);
}

}  // namespace

cudaError_t launch_combine_bwd(const void *dY, int dY_fp32, const void *Yp, const int32_t *slot_pos,
                               const float *topk_w, int T, int H, int K, void *dYp, float *d_topk_w, cudaStream_t s)
{
    if (dY_fp32)
        return d_topk_w ? combine<true, true>(dY, Yp, slot_pos, topk_w, T, H, K, dYp, d_topk_w, s)
                        : combine<true, false>(dY, Yp, slot_pos, topk_w, T, H, K, dYp, d_topk_w, s);
    return d_topk_w ? combine<false, true>(dY, Yp, slot_pos, topk_w, T, H, K, dYp, d_topk_w, s)
                    : combine<false, false>(dY, Yp, slot_pos, topk_w, T, H, K, dYp, d_topk_w, s);
}

cudaError_t launch_dispatch_bwd(const void *dXp, const int32_t *slot_pos, const void *dres, int T, int H, int K,
                                void *dX, int dX_fp32, cudaStream_t s)
{
    const dim3 grid(T, (H / 8 + DT - 1) / DT);
    return launch_pdl(dX_fp32 ? dispatch_bwd_kernel<true> : dispatch_bwd_kernel<false>, grid, dim3(DT), 0, s, 1,
                      static_cast<const uint4 *>(dXp), slot_pos, dres, H, K, dX);
}

}  // namespace moe
