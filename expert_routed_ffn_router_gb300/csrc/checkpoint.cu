// checkpoint.cu -- token rows kept for the backward pass in 8 bits: E4M3 bytes with one
// power-of-two scale per 128 columns of a row, and the way back to bf16.
//
// The format is the FP8 layer's activation format (fp8.cu): scale 2^k with k the smallest
// integer such that amax <= 448 2^k, k in [-124, 127], round to nearest even; a value taken
// back, q 2^k, is exact in bf16.  The exponents are kept as int8 [rows][ceil(n / 128)].  A
// block with an infinity has k = 127: it comes back infinite.  A NaN stays a NaN.
//
// Bound by memory: 3 + 1/128 bytes an element each way.  16 lanes hold a block (16 bytes a
// lane), so its maximum takes four shuffles.
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int CB = 128;    // columns that share a scale

__global__ void __launch_bounds__(256) ckpt_pack_kernel(const uint16_t *__restrict__ in, unsigned n_vec,
                                                        unsigned nb, int n, uint8_t *__restrict__ q,
                                                        int8_t *__restrict__ sc)
{
    pdl_wait();
    const unsigned vec = blockIdx.x * 16u + (threadIdx.x >> 4);
    const int l = threadIdx.x & 15;
    const unsigned row = vec / nb;
    const int c = static_cast<int>(vec - row * nb) * CB + 8 * l;
    const bool on = vec < n_vec && c < n;     // (the last block of a row may hold 64 columns)
    const size_t off = static_cast<size_t>(row) * n + c;
    uint4 u = make_uint4(0, 0, 0, 0);
    if (on) u = *reinterpret_cast<const uint4 *>(in + off);
    const float v[8] = {bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y),
                        bf16_lo(u.z), bf16_hi(u.z), bf16_lo(u.w), bf16_hi(u.w)};
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, o));
    const int k = ckpt_scale_exp(amax);
    const float inv = pow2f(-k);
    if (!on) return;
    uint2 o;
    o.x = f32x2_to_e4m3x2(v[1] * inv, v[0] * inv) |
          static_cast<uint32_t>(f32x2_to_e4m3x2(v[3] * inv, v[2] * inv)) << 16;
    o.y = f32x2_to_e4m3x2(v[5] * inv, v[4] * inv) |
          static_cast<uint32_t>(f32x2_to_e4m3x2(v[7] * inv, v[6] * inv)) << 16;
    *reinterpret_cast<uint2 *>(q + off) = o;
    if (l == 0) sc[vec] = static_cast<int8_t>(k);
}

__global__ void __launch_bounds__(256) ckpt_unpack_kernel(const uint8_t *__restrict__ q,
                                                          const int8_t *__restrict__ sc, unsigned n_vec,
                                                          unsigned nb, int n, uint16_t *__restrict__ out)
{
    pdl_wait();
    const unsigned vec = blockIdx.x * 16u + (threadIdx.x >> 4);
    const unsigned row = vec / nb;
    const int c = static_cast<int>(vec - row * nb) * CB + 8 * (threadIdx.x & 15);
    if (vec >= n_vec || c >= n) return;
    const size_t off = static_cast<size_t>(row) * n + c;
    const uint2 u = *reinterpret_cast<const uint2 *>(q + off);
    const float s = pow2f(sc[vec]);
    *reinterpret_cast<uint4 *>(out + off) = e4m3x8_to_bf16x8(u, s);
}

}  // namespace

cudaError_t launch_ckpt_pack(const void *in, long long rows, int n, void *q, int8_t *sc, cudaStream_t s)
{
    const unsigned nb = (n + CB - 1) / CB;
    const unsigned n_vec = static_cast<unsigned>(rows) * nb;
    return launch_pdl(ckpt_pack_kernel, dim3((n_vec + 15) / 16), dim3(256), 0, s, 1,
                      static_cast<const uint16_t *>(in), n_vec, nb, n, static_cast<uint8_t *>(q), sc);
}

cudaError_t launch_ckpt_unpack(const void *q, const int8_t *sc, long long rows, int n, void *out,
                               cudaStream_t s)
{
    const unsigned nb = (n + CB - 1) / CB;
    const unsigned n_vec = static_cast<unsigned>(rows) * nb;
    return launch_pdl(ckpt_unpack_kernel, dim3((n_vec + 15) / 16), dim3(256), 0, s, 1,
                      static_cast<const uint8_t *>(q), sc, n_vec, nb, n, static_cast<uint16_t *>(out));
}

}  // namespace moe
