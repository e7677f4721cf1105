// residual_fwd.cu -- a block's branch joined to the residual stream, with the norm behind the branch, its
// gates, the stream's scale and the next block's norm (formulas: residual.cuh).
//
// Statistics.  A row's mean and variance take one exchange between the warps: each warp forms the
// mean and the centred square sum of its own columns, and these are merged with the warps' means
// (sum of n_w (m_w - mean)^2): the variance is that of centred values, as in norm.cu.  A turn of the loop
// takes the statistics of y of one row and of r of the row before it through the same exchange: a
// row costs one barrier, and the two chains of shuffles around it run side by side (16384 x 7168 in
// fp32 with two norms: 326 us with an exchange for each, @FWD@ so).
//
// The next norm's statistics are those of r as it is stored: with a bf16 stream, what the backward
// pass reads.
#include "residual.cuh"

namespace moe {
namespace residual {
namespace {

// N: threads of a row (32: a warp, with WARPS rows a CTA).  PREG: the columns' parameters stay in
// registers (read once a CTA instead of once a row).
template <int N, bool PREG, int XT, int YT>
__global__ void __launch_bounds__(N == 32 ? 32 * WARPS : N) join_kernel(const __grid_constant__ Args p)
{
    constexpr bool ONE = N == 32;
    extern __shared__ __align__(16) unsigned char stages[];
    __shared__ float red[2][5][N / 32];
    const int H = p.H, S = p.stages, lane = threadIdx.x & 31;
    const bool xf = p.x_fp32, yf = p.y_fp32;
    const ResidualOpts &o = p.o;
    const Columns<N> in{H / 4, static_cast<int>(threadIdx.x)};
    const int tid = in.tid;
    Exchange<N> exchange{red};
    const float n_w = warp_columns<N>(H, tid >> 5), n_l = warp_columns<N>(H, lane);   // of this warp, of warp `lane`
    unsigned char *ring = stages + (ONE ? threadIdx.y * S * p.stage_bytes : 0);
    const uint32_t ring_at = smem_u32(ring);
    const int first = ONE ? blockIdx.x * WARPS + threadIdx.y : blockIdx.x, step = ONE ? gridDim.x * WARPS : gridDim.x;
    pdl_wait();
    auto fetch = [&](int row, int s) {
        if (row < p.T) {
            const uint32_t st = ring_at + s * p.stage_bytes;
            stage_in<XT, N>(st + p.off[0], p.x, row, H, xf, in);
            stage_in<YT, N>(st + p.off[1], p.y, row, H, yf, in);
        }
        copies_commit();
    };
    for (int s = 0; s < S; ++s) fetch(first + s * step, s);
    // gate and norm of the branch as one scale and shift, the next norm's
    auto scale = [&](int k) { return mul4(col4<N>(o.gate, tid, k, 1.f), col4<N>(o.gamma_post, tid, k, 1.f)); };
    auto shift = [&](int k) {
        return o.beta_post ? mul4(col4<N>(o.gate, tid, k, 1.f), col4<N>(o.beta_post, tid, k, 0.f)) : all4(0.f);
    };
    constexpr int PV = PREG ? VPT : 1;
    float4 ps[PV], pt[PV], ns[PV], nt[PV];
    if (PREG)
#pragma unroll
        for (int k = 0; k < PV; ++k) {
            if (!in(k)) continue;
            ps[k] = scale(k);
            pt[k] = shift(k);
            ns[k] = col4<N>(o.gamma_pre, tid, k, 1.f);
            nt[k] = col4<N>(o.beta_pre, tid, k, 0.f);
        }
    const float inv = 1.f / static_cast<float>(H), n_inv = n_w > 0.f ? 1.f / n_w : 0.f;
    const bool stat = o.post || o.pre, centred = o.post == 1 || o.pre == 1;
    const float ly = o.post == 1 ? 1.f : 0.f, lr = o.pre == 1 ? 1.f : 0.f;
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
            copies_wait(S - 1);
            if (o.gate_token) gt = o.gate_token[row];
        }
        const unsigned char *ys = staged<YT>(st + p.off[1], tid, yf);
#pragma unroll
        for (int k = 0; k < VPT; ++k) v[k] = now && in(k) ? ld4<YT, N>(ys, k, yf) : all4(0.f);
        float2 sy = make_float2(0.f, 1.f), sr = sy;
        if (stat) {
            // of this warp's columns: the means (of y, of r before), then the square sums around them
            float m[2] = {0.f, 0.f}, q[2] = {0.f, 0.f};
            if (centred) {
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    m[0] += sum4(v[k]);
                    m[1] += sum4(u[k]);
                }
                warp_sums(m);
                m[0] *= n_inv * ly;
                m[1] *= n_inv * lr;
            }
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                if (!in(k)) continue;
                const float4 a = make_float4(v[k].x - m[0], v[k].y - m[0], v[k].z - m[0], v[k].w - m[0]);
                const float4 b = make_float4(u[k].x - m[1], u[k].y - m[1], u[k].z - m[1], u[k].w - m[1]);
                q[0] += dot4(a, a);
                q[1] += dot4(b, b);
            }
            warp_sums(q);
            if (!ONE) {
                float e[4] = {m[0], m[1], q[0], q[1]};
                exchange(e);
                q[0] = e[2];
                q[1] = e[3];
                if (centred) {
                    m[0] = e[0] * n_l;
                    m[1] = e[1] * n_l;
                    warp_sums(m);
                    m[0] *= inv;
                    m[1] *= inv;
                    if (lane < N / 32) {
                        q[0] = fmaf(n_l * ly * (e[0] - m[0]), e[0] - m[0], q[0]);
                        q[1] = fmaf(n_l * lr * (e[1] - m[1]), e[1] - m[1], q[1]);
                    }
                }
                warp_sums(q);
            }
            if (o.post) sy = make_float2(m[0], 1.f / sqrtf(q[0] * inv + o.eps_post));
            if (o.pre) sr = make_float2(m[1], 1.f / sqrtf(q[1] * inv + o.eps_pre));
        }
        if (before >= 0) {                   // the row before: its norm
            if (o.pre) {
                unsigned char *to = row_at<BF16>(p.n, before, H, tid, false);
#pragma unroll
                for (int k = 0; k < VPT; ++k)
                    if (in(k))
                        st4<BF16, N>(to, k, false, fma4(norm4(u[k], sr.x, sr.y), PREG ? ns[k % PV] : col4<N>(o.gamma_pre, tid, k, 1.f),
                                                        PREG ? nt[k % PV] : col4<N>(o.beta_pre, tid, k, 0.f)));
            }
            if (p.stats && tid == 0) p.stats[before] = make_float4(sy_before.x, sy_before.y, sr.x, sr.y);
        }
        before = -1;
        if (!now) continue;
        const unsigned char *xs = staged<XT>(st + p.off[0], tid, xf);
        unsigned char *to = row_at<XT>(p.r, row, H, tid, xf);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            if (!in(k)) continue;
            float4 b = fma4(norm4(v[k], sy.x, sy.y), PREG ? ps[k % PV] : scale(k), PREG ? pt[k % PV] : shift(k));
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
        fetch(row + S * step, s);
        if (++s == S) s = 0;
        before = row;
        sy_before = sy;
    }
}

using Kernel = void (*)(const Args);

template <int N, bool PREG>
Kernel of_types(int x_fp32, int y_fp32)
{
    return x_fp32 ? (y_fp32 ? join_kernel<N, PREG, FP32, FP32> : join_kernel<N, PREG, FP32, BF16>)
                  : (y_fp32 ? join_kernel<N, PREG, BF16, FP32> : join_kernel<N, PREG, BF16, BF16>);
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
    const int threads = row_threads(H);
    const bool one = threads == 32;
    dim3 block, grid;
    if (one) {
        p.stages = 2;
        block = dim3(32, WARPS);
        const int units = (T + WARPS - 1) / WARPS, most = 4 * num_sms();
        grid = dim3(units < most ? units : most);
    } else {
        const int fit = static_cast<int>(ROOM / p.stage_bytes);
        int ctas = 512 / threads;
        if (ctas > fit / 2) ctas = fit / 2;
        if (ctas < 1) ctas = 1;
        p.stages = fit / ctas > 3 ? 3 : fit / ctas;
        block = dim3(threads);
        grid = dim3(T < ctas * num_sms() ? T : ctas * num_sms());
    }
    const Kernel kernel = threads == 32    ? of_types<32, false>(x_fp32, y_fp32)
                          : threads == 128 ? of_types<128, true>(x_fp32, y_fp32)
                          : threads == 256 ? of_types<256, true>(x_fp32, y_fp32)
                          : threads == 512 ? of_types<512, true>(x_fp32, y_fp32)
                                           : join_kernel<1024, false, RUNTIME, RUNTIME>;
    const size_t smem = static_cast<size_t>(p.stages) * p.stage_bytes * (one ? WARPS : 1);
    const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(kernel), smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, grid, block, smem, s, 1, p);
}

}  // namespace moe
