// checkpoint.cu -- token rows kept for the backward pass in 8 bits: E4M3 bytes with one
// power-of-two scale per 128 columns of a row, and the way back to bf16.
//
// The format is the FP8 layer's activation format (fp8.cu): scale 2^k with k the smallest
// integer such that amax <= 448 2^k, k in [-124, 127], round to nearest even; a value taken
// back, q 2^k, is exact in bf16.  The exponents are kept as int8 [rows][ceil(n / 128)].  A
// block with an infinity has k = 127: it comes back infinite.  A NaN stays a NaN.
//
// Bound by memory: 3 + 1/128 bytes an element each way.  8 lanes hold a block, 16 columns (32
// bytes of bf16, 16 of E4M3) a lane, so its maximum takes three shuffles and every access is
// 16 bytes wide (8 columns a lane, with 8-byte accesses to the bytes, measured 129 us for 16384
// rows of 7168 packed and taken back; this: 107.5 us, 6.57 TB/s).
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int CB = 128;    // columns that share a scale
constexpr int VEC_CTA = 32;   // blocks a CTA of 256 threads takes

__global__ void __launch_bounds__(256) ckpt_pack_kernel(const uint16_t *__restrict__ in, unsigned n_vec,
                                                        unsigned nb, int n, uint8_t *__restrict__ q,
                                                        int8_t *__restrict__ sc)
{
    const unsigned vec = blockIdx.x * VEC_CTA + (threadIdx.x >> 3);
    const int l = threadIdx.x & 7;
    const unsigned row = vec / nb;
    const int c = static_cast<int>(vec - row * nb) * CB + 16 * l;
    const bool on = vec < n_vec && c < n;     // (the last block of a row may hold 64 columns)
    const size_t off = static_cast<size_t>(row) * n + c;
    pdl_wait();
    uint32_t w[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    if (on) {
        const uint4 a = *reinterpret_cast<const uint4 *>(in + off), b = *reinterpret_cast<const uint4 *>(in + off + 8);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, o));
    const int k = ckpt_scale_exp(amax);
    const float inv = pow2f(-k);
    if (!on) return;
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[i] = f32x2_to_e4m3x2(bf16_hi(w[2 * i]) * inv, bf16_lo(w[2 * i]) * inv) |
               static_cast<uint32_t>(f32x2_to_e4m3x2(bf16_hi(w[2 * i + 1]) * inv, bf16_lo(w[2 * i + 1]) * inv)) << 16;
    *reinterpret_cast<uint4 *>(q + off) = make_uint4(o[0], o[1], o[2], o[3]);
    if (l == 0) sc[vec] = static_cast<int8_t>(k);
}

__global__ void __launch_bounds__(256) ckpt_unpack_kernel(const uint8_t *__restrict__ q,
                                                          const int8_t *__restrict__ sc, unsigned n_vec,
                                                          unsigned nb, int n, uint16_t *__restrict__ out)
{
    const unsigned vec = blockIdx.x * VEC_CTA + (threadIdx.x >> 3);
    const unsigned row = vec / nb;
    const int c = static_cast<int>(vec - row * nb) * CB + 16 * (threadIdx.x & 7);
    pdl_wait();
    if (vec >= n_vec || c >= n) return;
    const size_t off = static_cast<size_t>(row) * n + c;
    const uint4 u = *reinterpret_cast<const uint4 *>(q + off);
    const float s = pow2f(sc[vec]);
    *reinterpret_cast<uint4 *>(out + off) = e4m3x8_to_bf16x8(make_uint2(u.x, u.y), s);
    *reinterpret_cast<uint4 *>(out + off + 8) = e4m3x8_to_bf16x8(make_uint2(u.z, u.w), s);
}

}  // namespace

cudaError_t launch_ckpt_pack(const void *in, long long rows, int n, void *q, int8_t *sc, cudaStream_t s)
{
    const unsigned nb = (n + CB - 1) / CB;
    const unsigned n_vec = static_cast<unsigned>(rows) * nb;
    return launch_pdl(ckpt_pack_kernel, dim3((n_vec + VEC_CTA - 1) / VEC_CTA), dim3(256), 0, s, 1,
                      static_cast<const uint16_t *>(in), n_vec, nb, n, static_cast<uint8_t *>(q), sc);
}

cudaError_t launch_ckpt_unpack(const void *q, const int8_t *sc, long long rows, int n, void *out,
                               cudaStream_t s)
{
    const unsigned nb = (n + CB - 1) / CB;
    const unsigned n_vec = static_cast<unsigned>(rows) * nb;
    return launch_pdl(ckpt_unpack_kernel, dim3((n_vec + VEC_CTA - 1) / VEC_CTA), dim3(256), 0, s, 1,
                      static_cast<const uint8_t *>(q), sc, n_vec, nb, n, static_cast<uint16_t *>(out));
}

}  // namespace moe
