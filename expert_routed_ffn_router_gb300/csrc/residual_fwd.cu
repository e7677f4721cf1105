// residual_fwd.cu -- a block's branch joined to the residual stream, with the norm behind the branch, its
// gates, the stream's scale and the next block's norm (formulas: residual.cuh).
//
// Statistics.  A row's mean and variance take one exchange between the warps: each warp forms the
// mean and the centred square sum of its own columns, and these are merged with the warps' means
// (sum of n_w (m_w - mean)^2): the variance is that of centred values, as in norm.cu.  A turn of the loop
// takes the statistics of y of one row and of r of the row before it through the same exchange: a
// row costs one barrier, and the two chains of shuffles around it run side by side (16384 x 7168 in
// fp32 with two norms: 326 us with an exchange for each, 277 us so).
//
// What bounds it: memory in fp32 (16384 x 7168, RMS norm of y, layer norm of r: 240 us, 6.8 TB/s, the copy
// bandwidth); in bf16 (180-190 us, 5.2 TB/s) memory is at three quarters and the schedulers at 59%.
//
// The next norm's statistics are those of r as it is stored: with a bf16 stream, what the backward
// pass reads.
#include "residual.cuh"

namespace moe {
namespace residual {
namespace {

// N: threads of a row (32: a warp, with WARPS rows a CTA); the columns' parameters stay in registers, from
// 64 to 512 (read once a CTA instead of once a row).  CY, CR: the norm of y, of r is centred (a layer
// norm).
template <int N, int XT, int YT, int CY, int CR>
__global__ void __launch_bounds__(N == 32 ? 32 * WARPS : N) join_kernel(const __grid_constant__ Args p)
{
    constexpr bool ONE = N == 32, PREG = N >= 64 && N <= 512;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float4 red[2][N / 32];
    const int H = p.H, S = p.stages, lane = threadIdx.x & 31;
    const bool xf = p.x_fp32, yf = p.y_fp32;
    const ResidualOpts &o = p.o;
    const int tid = threadIdx.x;
    const Columns<N> in{H / 4, tid};
    Exchange<N> exchange{red, tid};
    const float n_w = warp_columns<N>(H, tid >> 5), n_l = warp_columns<N>(H, lane);   // of this warp, of warp `lane`
    unsigned char *ring = smem + (ONE ? threadIdx.y * S * p.stage_bytes : 0);
    const uint32_t ring_at = smem_u32(ring);
    const int first = ONE ? blockIdx.x * WARPS + threadIdx.y : blockIdx.x, step = ONE ? gridDim.x * WARPS : gridDim.x;
    pdl_wait();
    // (a thread's copies of x and y are groups of their own, in turn: 2 S - 1 are behind the one it needs)
    auto fetch_x = [&](int row, int s) {
        if (row < p.T) stage_in<XT, N>(ring_at + s * p.stage_bytes + p.off[0], p.x, row, H, xf, in);
        copies_commit();
    };
    auto fetch_y = [&](int row, int s) {
        if (row < p.T) stage_in<YT, N>(ring_at + s * p.stage_bytes + p.off[1], p.y, row, H, yf, in);
        copies_commit();
    };
    for (int s = 0; s < S; ++s) {
        fetch_y(first + s * step, s);
        fetch_x(first + s * step, s);
    }
    // gate and norm of the branch as one scale and shift, the next norm's
    auto scale = [&](int k) { return mul4(col4<N>(o.gate, tid, k, 1.f), col4<N>(o.gamma_post, tid, k, 1.f)); };
    auto shift = [&](int k) {
        return o.beta_post ? mul4(col4<N>(o.gate, tid, k, 1.f), col4<N>(o.beta_post, tid, k, 0.f)) : all4(0.f);
    };
    auto param = [&](int j, int k) {
        return j == 0 ? scale(k) : j == 1 ? shift(k) : j == 2 ? col4<N>(o.gamma_pre, tid, k, 1.f) : col4<N>(o.beta_pre, tid, k, 0.f);
    };
    constexpr int PJ = PREG ? 4 : 1, PK = PREG ? VPT : 1;
    float4 reg[PJ][PK];
    if (PREG) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < VPT; ++k)
                if (in(k)) reg[j % PJ][k % PK] = param(j, k);
    }
    auto take = [&](int j, int k) -> float4 { return PREG ? reg[j % PJ][k % PK] : param(j, k); };
    const float inv = 1.f / static_cast<float>(H), n_inv = n_w > 0.f ? 1.f / n_w : 0.f;
    const bool stat = o.post || o.pre;
    float4 u[VPT];                           // r of the row before
#pragma unroll
    for (int k = 0; k < VPT; ++k) u[k] = all4(0.f);
    float2 sy_before = make_float2(0.f, 1.f);
    int s = 0, before = -1;
    for (int row = first; row < p.T || before >= 0; row += step) {
        const bool now = row < p.T;
        const unsigned char *st = ring + s * p.stage_bytes;
        float gt = 1.f;
        float4 v[VPT];
        if (now) {
            copies_wait(2 * S - 1);
            if (o.gate_token) gt = o.gate_token[row];
        }
        const unsigned char *ys = staged<YT>(st + p.off[1], tid, yf);
#pragma unroll
        for (int k = 0; k < VPT; ++k) v[k] = now && in(k) ? ld4<YT, N>(ys, k, yf) : all4(0.f);
        if (now) fetch_y(row + S * step, s);
        float2 sy = make_float2(0.f, 1.f), sr = sy;
        if (stat) {
            // of this warp's columns: the means (of y, of r before), then the square sums around them
            float2 m = make_float2(0.f, 0.f), q = m;
            if (CY || CR) {
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    if (CY) m.x += sum4(v[k]);
                    if (CR) m.y += sum4(u[k]);
                }
                m = warp_pair_all(m.x, m.y);
                m.x *= n_inv;
                m.y *= n_inv;
            }
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                if (!in(k)) continue;
                const float4 a = CY ? make_float4(v[k].x - m.x, v[k].y - m.x, v[k].z - m.x, v[k].w - m.x) : v[k];
                const float4 b = CR ? make_float4(u[k].x - m.y, u[k].y - m.y, u[k].z - m.y, u[k].w - m.y) : u[k];
                q.x += dot4(a, a);
                q.y += dot4(b, b);
            }
            if (ONE) {
                q = warp_pair_all(q.x, q.y);
            } else {
                // the warps' means and square sums
                const float4 w = exchange(threadIdx.x & 16 ? m.y : m.x, warp_pair(q.x, q.y));
                q = make_float2(w.z, w.w);
                if (CY || CR) {
                    m = warp_pair_all(w.x * n_l, w.y * n_l);
                    m.x *= inv;
                    m.y *= inv;
                    if (lane < N / 32) {
                        if (CY) q.x = fmaf(n_l * (w.x - m.x), w.x - m.x, q.x);
                        if (CR) q.y = fmaf(n_l * (w.y - m.y), w.y - m.y, q.y);
                    }
                }
                q = warp_pair_all(q.x, q.y);
            }
            if (o.post) sy = make_float2(CY ? m.x : 0.f, 1.f / sqrtf(q.x * inv + o.eps_post));
            if (o.pre) sr = make_float2(CR ? m.y : 0.f, 1.f / sqrtf(q.y * inv + o.eps_pre));
        }
        if (before >= 0) {                   // the row before: its norm
            if (o.pre) {
                unsigned char *to = row_at<BF16>(p.n, before, H, tid, false);
#pragma unroll
                for (int k = 0; k < VPT; ++k)
                    if (in(k))
                        st4<BF16, N>(to, k, false, fma4(norm4(u[k], sr.x, sr.y), take(2, k), take(3, k)));
            }
            if (p.stats && tid == 0) p.stats[before] = make_float4(sy_before.x, sy_before.y, sr.x, sr.y);
        }
        before = -1;
        if (!now) continue;
        copies_wait(2 * S - 1);
        const unsigned char *xs = staged<XT>(st + p.off[0], tid, xf);
        unsigned char *to = row_at<XT>(p.r, row, H, tid, xf);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            if (!in(k)) continue;
            float4 b = fma4(norm4(v[k], sy.x, sy.y), take(0, k), take(1, k));
            const float4 x = ld4<XT, N>(xs, k, xf);
            b = make_float4(fmaf(o.alpha, x.x, gt * b.x), fmaf(o.alpha, x.y, gt * b.y), fmaf(o.alpha, x.z, gt * b.z),
                            fmaf(o.alpha, x.w, gt * b.w));
            if (!wide<XT>(xf)) {     // what is stored
                const uint2 h = make_uint2(f32x2_to_bf16x2(b.y, b.x), f32x2_to_bf16x2(b.w, b.z));
                b = make_float4(bf16_lo(h.x), bf16_hi(h.x), bf16_lo(h.y), bf16_hi(h.y));
            }
            st4<XT, N>(to, k, xf, b);
            u[k] = b;
        }
        fetch_x(row + S * step, s);
        if (++s == S) s = 0;
        before = row;
        sy_before = sy;
    }
}

using Kernel = void (*)(const Args);

template <int N, int CY, int CR>
Kernel of_types(int x_fp32, int y_fp32)
{
    return x_fp32 ? (y_fp32 ? join_kernel<N, FP32, FP32, CY, CR> : join_kernel<N, FP32, BF16, CY, CR>)
                  : (y_fp32 ? join_kernel<N, BF16, FP32, CY, CR> : join_kernel<N, BF16, BF16, CY, CR>);
}

template <int N>
Kernel of_kinds(const ResidualOpts &o, int x_fp32, int y_fp32)
{
    if constexpr (N == 1024)
        return o.post == 1 ? (o.pre == 1 ? join_kernel<N, RUNTIME, RUNTIME, 1, 1> : join_kernel<N, RUNTIME, RUNTIME, 1, 0>)
                           : (o.pre == 1 ? join_kernel<N, RUNTIME, RUNTIME, 0, 1> : join_kernel<N, RUNTIME, RUNTIME, 0, 0>);
    else
        return o.post == 1 ? (o.pre == 1 ? of_types<N, 1, 1>(x_fp32, y_fp32) : of_types<N, 1, 0>(x_fp32, y_fp32))
                           : (o.pre == 1 ? of_types<N, 0, 1>(x_fp32, y_fp32) : of_types<N, 0, 0>(x_fp32, y_fp32));
}

}  // namespace
}  // namespace residual

cudaError_t launch_join(const ResidualOpts &o, const void *x, int x_fp32, const void *y, int y_fp32, int T, int H,
                        void *r, void *n, float *stats, cudaStream_t s)
{
    using namespace residual;
    Args p{};
    p.o = o;
    p.T = T; p.H = H; p.x_fp32 = x_fp32; p.y_fp32 = y_fp32;
    p.x = x; p.y = y; p.r = r; p.n = static_cast<uint16_t *>(n);
    p.stats = reinterpret_cast<float4 *>(stats);
    p.off[0] = 0;
    p.off[1] = H * (x_fp32 ? 4 : 2);
    p.stage_bytes = p.off[1] + H * (y_fp32 ? 4 : 2);
    // (448 where every thread has four vectors then)
    const int threads = H > 6144 && H <= 7168 ? 448 : row_threads(H);
    const bool one = threads == 32;
    // Rows on their way: about AHEAD bytes an SM.  More of them cost bandwidth (16384 x 7168 in fp32, without and
    // with a norm of y, n by RMS norm and layer norm: 281 and 271 us with three stages of 57 KB, 254 and
    // 241 us with one; in bf16 153 and 190 us with two stages of 29 KB, 165 and 191 us with one).
    constexpr size_t AHEAD = 72 * 1024;
    const size_t unit = static_cast<size_t>(p.stage_bytes) * (one ? WARPS : 1);     // a stage of a CTA
    const int units = one ? (T + WARPS - 1) / WARPS : T, room = one ? 4 : 512 / threads;
    int ctas = static_cast<int>(AHEAD / unit);
    ctas = ctas < 1 ? 1 : (ctas > room ? (room < 1 ? 1 : room) : ctas);
    const int fit = static_cast<int>(AHEAD / (unit * ctas));
    p.stages = fit < 1 ? 1 : (fit > 3 ? 3 : fit);
    const dim3 block = one ? dim3(32, WARPS) : dim3(threads), grid(units < ctas * num_sms() ? units : ctas * num_sms());
    const size_t smem = static_cast<size_t>(p.stages) * p.stage_bytes * (one ? WARPS : 1);
    const Kernel kernel = threads == 32    ? of_kinds<32>(o, x_fp32, y_fp32)
                          : threads == 64  ? of_kinds<64>(o, x_fp32, y_fp32)
                          : threads == 128 ? of_kinds<128>(o, x_fp32, y_fp32)
                          : threads == 256 ? of_kinds<256>(o, x_fp32, y_fp32)
                          : threads == 448 ? of_kinds<448>(o, x_fp32, y_fp32)
                          : threads == 512 ? of_kinds<512>(o, x_fp32, y_fp32) : of_kinds<1024>(o, x_fp32, y_fp32);
    const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(kernel), smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, grid, block, smem, s, 1, p);
}

}  // namespace moe
