// residual.cu -- a block's branch joined to the residual stream, with the norm behind the branch,
// its gates, the stream's scale and the next block's norm; forward and backward.
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
// Both are bound by memory: every row is read and written once.  The rows of a CTA (of a warp, up
// to WARP_COLS columns) arrive ahead of time by asynchronous copies; every thread copies the
// columns that it will read itself, so nothing but the sums of a row crosses threads.
//
// Statistics.  A row's mean and variance take one exchange between the warps: each warp forms the
// mean and the centred square sum of its own columns, and these are merged with the warps' means
// (sum of n_w (m_w - mean)^2): the variance is that of centred values, as in norm.cu.
//
// The next norm's statistics are those of r as it is stored: with a bf16 stream, what the backward
// pass reads.
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int VPT = 4;               // vectors of 4 columns a thread
constexpr int WARP_COLS = 32 * 4 * VPT;   // longest row of one warp
constexpr int WARPS = 8;             // rows of a CTA then
constexpr size_t ROOM = 220 * 1024;  // shared memory of an SM for the staged rows

struct Residual {
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
    int stages, stage_bytes;         // of a CTA (of a warp: short rows)
    int off[4];                      // the staged arrays in a stage, -1: read directly
};

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}

__device__ __forceinline__ float4 ld4(const void *p, size_t i, bool fp32)
{
    if (fp32) return *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
    const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i);
    return make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
}

__device__ __forceinline__ void st4(void *p, size_t i, bool fp32, float4 v)
{
    if (fp32)
        *reinterpret_cast<float4 *>(static_cast<float *>(p) + i) = v;
    else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p) + i) =
            make_uint2(f32x2_to_bf16x2(v.y, v.x), f32x2_to_bf16x2(v.w, v.z));
}

__device__ __forceinline__ float4 col4(const float *p, int c, float absent)
{
    return p ? *reinterpret_cast<const float4 *>(p + c) : make_float4(absent, absent, absent, absent);
}

__device__ __forceinline__ float sum4(float4 v) { return (v.x + v.y) + (v.z + v.w); }
__device__ __forceinline__ float dot4(float4 a, float4 b) { return fmaf(a.x, b.x, a.y * b.y) + fmaf(a.z, b.z, a.w * b.w); }
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

__device__ __forceinline__ void copy_async(void *dst, const void *src, bool wide)
{
    if (wide)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// The copies of all groups but the last `left` (at most 2) have arrived.
__device__ __forceinline__ void copies_wait(int left)
{
    if (left == 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (left == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 2;" ::: "memory");
}

// A row's threads: a warp (ONE) or the CTA.
template <bool ONE>
struct Row {
    int tid, n, nw;              // thread in the row, threads and warps of the row
    float n_w;                   // columns of this warp
    float (*red)[4][32];         // [2] buffers in turn
    const float *cols;           // [32] columns of each warp
    int turn;

    // sums of three values over the row's threads: one exchange
    __device__ __forceinline__ void sum3(float &a, float &b, float &c)
    {
        a = warp_sum(a); b = warp_sum(b); c = warp_sum(c);
        if (ONE) return;
        float (*r)[32] = red[turn];
        turn ^= 1;
        const int lane = tid & 31;
        if (lane == 0) { r[0][tid >> 5] = a; r[1][tid >> 5] = b; r[2][tid >> 5] = c; }
        __syncthreads();
        const bool in = lane < nw;
        a = warp_sum(in ? r[0][lane] : 0.f);
        b = warp_sum(in ? r[1][lane] : 0.f);
        c = warp_sum(in ? r[2][lane] : 0.f);
    }
    __device__ __forceinline__ void sum2(float &a, float &b)
    {
        a = warp_sum(a); b = warp_sum(b);
        if (ONE) return;
        float (*r)[32] = red[turn];
        turn ^= 1;
        const int lane = tid & 31;
        if (lane == 0) { r[0][tid >> 5] = a; r[1][tid >> 5] = b; }
        __syncthreads();
        const bool in = lane < nw;
        a = warp_sum(in ? r[0][lane] : 0.f);
        b = warp_sum(in ? r[1][lane] : 0.f);
    }
    // mean (0 for an RMS norm) and 1 / sqrt(variance + eps) of the row's columns v
    __device__ __forceinline__ float2 statistics(const float4 (&v)[VPT], int H, bool layer, float eps)
    {
        const float inv = 1.f / static_cast<float>(H);
        float m = 0.f;
        if (layer) {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (4 * (tid + i * n) < H) m += sum4(v[i]);
            m = warp_sum(m);
            m = n_w > 0.f ? m / n_w : 0.f;
        }
        float q = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (4 * (tid + i * n) < H) {
                const float4 c = make_float4(v[i].x - m, v[i].y - m, v[i].z - m, v[i].w - m);
                q += dot4(c, c);
            }
        q = warp_sum(q);
        if (!ONE) {
            float (*r)[32] = red[turn];
            turn ^= 1;
            const int lane = tid & 31;
            if (lane == 0) { r[0][tid >> 5] = m; r[1][tid >> 5] = q; }
            __syncthreads();
            const bool in = lane < nw;
            if (layer) {
                const float mw = in ? r[0][lane] : 0.f, k = in ? cols[lane] : 0.f;
                m = warp_sum(mw * k) * inv;
                q = in ? fmaf(k * (mw - m), mw - m, r[1][lane]) : 0.f;
            } else {
                q = in ? r[1][lane] : 0.f;
            }
            q = warp_sum(q);
        }
        return make_float2(m, 1.f / sqrtf(q * inv + eps));
    }
};

template <bool ONE>
__device__ __forceinline__ Row<ONE> row_threads(int H, float (*red)[4][32], float *cols)
{
    Row<ONE> w;
    w.tid = threadIdx.x;
    w.n = blockDim.x;
    w.nw = ONE ? 1 : blockDim.x >> 5;
    w.red = red;
    w.cols = cols;
    w.turn = 0;
    int k = 0;
    const int first = 4 * (threadIdx.x & ~31);
#pragma unroll
    for (int i = 0; i < VPT; ++i) k += max(0, min(128, H - first - 4 * i * w.n));
    w.n_w = static_cast<float>(k);
    if (!ONE && (threadIdx.x & 31) == 0) cols[threadIdx.x >> 5] = w.n_w;
    return w;
}

// The columns of this thread of row `row` of an array, to its place in a stage
__device__ __forceinline__ void stage_in(unsigned char *st, const void *p, int row, int H, bool fp32, int tid, int n)
{
    const size_t at = static_cast<size_t>(row) * H;
    const int b = fp32 ? 4 : 2;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = 4 * (tid + i * n);
        if (c < H) copy_async(st + c * b, static_cast<const unsigned char *>(p) + (at + c) * b, fp32);
    }
}

// ---------------------------------------------------------------------------- forward
// PREG: the columns' parameters stay in registers (read once a CTA instead of once a row).
template <bool ONE, int MAXT, bool PREG>
__global__ void __launch_bounds__(MAXT) join_kernel(const __grid_constant__ Residual p)
{
    extern __shared__ __align__(16) unsigned char stages[];
    __shared__ float red[2][4][32], cols[32];
    Row<ONE> w = row_threads<ONE>(p.H, red, cols);
    const int H = p.H, S = p.stages;
    const bool xf = p.x_fp32, yf = p.y_fp32;
    const ResidualOpts &o = p.o;
    unsigned char *ring = stages + (ONE ? threadIdx.y * S * p.stage_bytes : 0);
    const int first = ONE ? blockIdx.x * WARPS + threadIdx.y : blockIdx.x, step = ONE ? gridDim.x * WARPS : gridDim.x;
    if (!ONE) __syncthreads();
    pdl_wait();
    auto fetch = [&](int row, int s) {
        if (row < p.T) {
            unsigned char *st = ring + s * p.stage_bytes;
            stage_in(st + p.off[0], p.x, row, H, xf, w.tid, w.n);
            stage_in(st + p.off[1], p.y, row, H, yf, w.tid, w.n);
        }
        copies_commit();
    };
    for (int s = 0; s < S; ++s) fetch(first + s * step, s);
    // gate and norm of the branch as one scale and shift, the next norm's
    auto scale = [&](int c) { return mul4(col4(o.gate, c, 1.f), col4(o.gamma_post, c, 1.f)); };
    auto shift = [&](int c) {
        return o.beta_post ? mul4(col4(o.gate, c, 1.f), col4(o.beta_post, c, 0.f)) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    constexpr int PV = PREG ? VPT : 1;
    float4 ps[PV], pt[PV], ns[PV], nt[PV];
    if (PREG)
#pragma unroll
        for (int i = 0; i < PV; ++i) {
            const int c = 4 * (w.tid + i * w.n);
            if (c >= H) continue;
            ps[i] = scale(c);
            pt[i] = shift(c);
            ns[i] = col4(o.gamma_pre, c, 1.f);
            nt[i] = col4(o.beta_pre, c, 0.f);
        }
    int s = 0;
    for (int row = first; row < p.T; row += step) {
        copies_wait(S - 1);
        const unsigned char *st = ring + s * p.stage_bytes;
        const size_t base = static_cast<size_t>(row) * H;
        float4 v[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 4 * (w.tid + i * w.n);
            v[i] = c < H ? ld4(st + p.off[1], c, yf) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float2 sy = make_float2(0.f, 1.f), sr = sy;
        if (o.post) sy = w.statistics(v, H, o.post == 1, o.eps_post);
        const float gt = o.gate_token ? o.gate_token[row] : 1.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 4 * (w.tid + i * w.n);
            if (c >= H) continue;
            float4 b = fma4(norm4(v[i], sy.x, sy.y), PREG ? ps[i % PV] : scale(c), PREG ? pt[i % PV] : shift(c));
            const float4 x = ld4(st + p.off[0], c, xf);
            b = make_float4(fmaf(o.alpha, x.x, gt * b.x), fmaf(o.alpha, x.y, gt * b.y), fmaf(o.alpha, x.z, gt * b.z),
                            fmaf(o.alpha, x.w, gt * b.w));
            if (!xf) {               // what is stored
                const uint2 u = make_uint2(f32x2_to_bf16x2(b.y, b.x), f32x2_to_bf16x2(b.w, b.z));
                b = make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
            }
            st4(p.r, base + c, xf, b);
            v[i] = b;
        }
        fetch(row + S * step, s);
        if (o.pre) {
            sr = w.statistics(v, H, o.pre == 1, o.eps_pre);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = 4 * (w.tid + i * w.n);
                if (c >= H) continue;
                st4(p.n, base + c, false, fma4(norm4(v[i], sr.x, sr.y), PREG ? ns[i % PV] : col4(o.gamma_pre, c, 1.f),
                                               PREG ? nt[i % PV] : col4(o.beta_pre, c, 0.f)));
            }
        }
        if (p.stats && w.tid == 0) p.stats[row] = make_float4(sy.x, sy.y, sr.x, sr.y);
        if (++s == S) s = 0;
    }
}

// --------------------------------------------------------------------------- backward
// Staged arrays: 0 dn, 1 r, 2 y, 3 dr.  S0: with beta_post, whose gradient and the gate's need those sums.  PREG as above.
template <bool ONE, int MAXT, bool S0, bool PREG>
__global__ void __launch_bounds__(MAXT, MAXT <= 256 ? 2 : 1) join_bwd_kernel(const __grid_constant__ Residual p)
{
    extern __shared__ __align__(16) unsigned char stages[];
    __shared__ float red[2][4][32], cols[32];
    Row<ONE> w = row_threads<ONE>(p.H, red, cols);
    const int H = p.H, S = p.stages;
    const bool xf = p.x_fp32, yf = p.y_fp32;
    const ResidualOpts &o = p.o;
    unsigned char *ring = stages + (ONE ? threadIdx.y * S * p.stage_bytes : 0);
    const int first = ONE ? blockIdx.x * WARPS + threadIdx.y : blockIdx.x, step = ONE ? gridDim.x * WARPS : gridDim.x;
    if (!ONE) __syncthreads();
    pdl_wait();
    auto fetch = [&](int row, int s) {
        if (row < p.T) {
            unsigned char *st = ring + s * p.stage_bytes;
            if (p.off[0] >= 0) stage_in(st + p.off[0], p.dn, row, H, false, w.tid, w.n);
            if (p.off[1] >= 0) stage_in(st + p.off[1], p.r, row, H, xf, w.tid, w.n);
            if (p.off[2] >= 0) stage_in(st + p.off[2], p.y, row, H, yf, w.tid, w.n);
            if (p.off[3] >= 0) stage_in(st + p.off[3], p.dr, row, H, xf, w.tid, w.n);
        }
        copies_commit();
    };
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int PV = PREG ? VPT : 1, SV = S0 ? VPT : 1;
    float4 p1[VPT], p0[VPT], s1[VPT], s0[SV], ga[PV], gb[PV];
    auto scale = [&](int c) { return mul4(col4(o.gate, c, 1.f), col4(o.gamma_post, c, 1.f)); };
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        p1[i] = p0[i] = s1[i] = s0[i % SV] = zero;
        const int c = 4 * (w.tid + i * w.n);
        if (PREG && c < H) {
            ga[i % PV] = col4(o.gamma_pre, c, 1.f);
            gb[i % PV] = scale(c);
        }
    }
    auto gamma = [&](int i, int c) { return PREG ? ga[i % PV] : col4(o.gamma_pre, c, 1.f); };
    auto branch = [&](int i, int c) { return PREG ? gb[i % PV] : scale(c); };
    const float inv = 1.f / static_cast<float>(H);
    const bool token = p.d_token != nullptr;
    for (int s = 0; s < S; ++s) fetch(first + s * step, s);
    int s = 0;
    for (int row = first; row < p.T; row += step) {
        float4 st = p.stats[row];
        if (!o.post) { st.x = 0.f; st.y = 1.f; }
        const float gt = o.gate_token ? o.gate_token[row] : 1.f;
        copies_wait(S - 1);
        const unsigned char *sm = ring + s * p.stage_bytes;
        const size_t base = static_cast<size_t>(row) * H;
        float4 d[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 4 * (w.tid + i * w.n);
            d[i] = zero;
            if (c < H && p.dr) d[i] = p.off[3] >= 0 ? ld4(sm + p.off[3], c, xf) : ld4(p.dr, base + c, xf);
        }
        if (o.pre) {
            float a0 = 0.f, a1 = 0.f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = 4 * (w.tid + i * w.n);
                if (c >= H) continue;
                const float4 e = ld4(sm + p.off[0], c, false), h = norm4(ld4(sm + p.off[1], c, xf), st.z, st.w);
                p1[i] = fma4(e, h, p1[i]);
                p0[i] = make_float4(p0[i].x + e.x, p0[i].y + e.y, p0[i].z + e.z, p0[i].w + e.w);
                const float4 a = mul4(e, gamma(i, c));
                a0 += sum4(a);
                a1 += dot4(a, h);
            }
            w.sum2(a0, a1);
            a0 = o.pre == 1 ? a0 * inv : 0.f;
            a1 *= inv;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = 4 * (w.tid + i * w.n);
                if (c >= H) continue;
                const float4 e = ld4(sm + p.off[0], c, false), h = norm4(ld4(sm + p.off[1], c, xf), st.z, st.w);
                const float4 a = mul4(e, gamma(i, c));
                d[i].x = fmaf(st.w, a.x - a0 - h.x * a1, d[i].x);
                d[i].y = fmaf(st.w, a.y - a0 - h.y * a1, d[i].y);
                d[i].z = fmaf(st.w, a.z - a0 - h.z * a1, d[i].z);
                d[i].w = fmaf(st.w, a.w - a0 - h.w * a1, d[i].w);
            }
        }
        // the branch: f = g_h gamma_post d
        float a0 = 0.f, a1 = 0.f, a2 = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 4 * (w.tid + i * w.n);
            if (c >= H) continue;
            st4(p.dx, base + c, xf, scale4(d[i], o.alpha));
            if (!p.y) continue;
            const float4 h = norm4(ld4(sm + p.off[2], c, yf), st.x, st.y), g = scale4(d[i], gt);
            s1[i] = fma4(g, h, s1[i]);
            if (S0) s0[i % SV] = make_float4(s0[i % SV].x + g.x, s0[i % SV].y + g.y, s0[i % SV].z + g.z, s0[i % SV].w + g.w);
            const float4 f = mul4(d[i], branch(i, c));
            a0 += sum4(f);
            a1 += dot4(f, h);
            if (token && o.beta_post) a2 += dot4(mul4(d[i], col4(o.gate, c, 1.f)), col4(o.beta_post, c, 0.f));
        }
        if (o.post || token) {
            w.sum3(a0, a1, a2);
            if (token && w.tid == 0) p.d_token[row] = a1 + a2;
            a0 = o.post == 1 ? a0 * inv : 0.f;
            a1 = o.post ? a1 * inv : 0.f;
        } else {
            a0 = a1 = 0.f;
        }
        const float rs = gt * st.y;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 4 * (w.tid + i * w.n);
            if (c >= H) continue;
            float4 f = mul4(d[i], branch(i, c));
            if (o.post) {
                const float4 h = norm4(ld4(sm + p.off[2], c, yf), st.x, st.y);
                f = make_float4(f.x - a0 - h.x * a1, f.y - a0 - h.y * a1, f.z - a0 - h.z * a1, f.w - a0 - h.w * a1);
            }
            st4(p.dy, base + c, false, scale4(f, o.post ? rs : gt));
        }
        fetch(row + S * step, s);
        if (++s == S) s = 0;
    }
    float *part = p.part + static_cast<size_t>(blockIdx.x) * 4 * H;
    if (!ONE) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 4 * (w.tid + i * w.n);
            if (c >= H) continue;
            *reinterpret_cast<float4 *>(part + c) = p1[i];
            *reinterpret_cast<float4 *>(part + H + c) = p0[i];
            *reinterpret_cast<float4 *>(part + 2 * H + c) = s1[i];
            *reinterpret_cast<float4 *>(part + 3 * H + c) = s0[i % SV];
        }
        return;
    }
    // the warps' sums, added in their order
    __shared__ float4 comb[WARPS][33];
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 4 * (w.tid + 32 * i);
            __syncthreads();
            comb[threadIdx.y][w.tid] = k == 0 ? p1[i] : k == 1 ? p0[i] : k == 2 ? s1[i] : s0[i % SV];
            __syncthreads();
            if (threadIdx.y == 0 && c < H) {
                float4 t = comb[0][w.tid];
                for (int q = 1; q < WARPS; ++q) {
                    const float4 u = comb[q][w.tid];
                    t = make_float4(t.x + u.x, t.y + u.y, t.z + u.z, t.w + u.w);
                }
                *reinterpret_cast<float4 *>(part + k * H + c) = t;
            }
        }
}

// The gradients of the columns' parameters from the CTAs' partial sums [n][4][H], added in order:
// 32 columns x 8 strands a CTA.
__global__ void __launch_bounds__(256) join_wgrad_kernel(const float *__restrict__ part, int n, int H, ResidualOpts o,
                                                         ResidualGrads g)
{
    __shared__ float s[4][8][32];
    pdl_wait();
    const int c = blockIdx.x * 32 + threadIdx.x;     // (H is a multiple of 32)
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int r = threadIdx.y; r < n; r += 8)
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] += part[(static_cast<size_t>(r) * 4 + k) * H + c];
#pragma unroll
    for (int k = 0; k < 4; ++k) s[k][threadIdx.y][threadIdx.x] = v[k];
    __syncthreads();
    if (threadIdx.y != 0) return;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        for (int q = 1; q < 8; ++q) v[k] += s[k][q][threadIdx.x];
    if (g.gamma_pre) g.gamma_pre[c] = v[0];
    if (g.beta_pre) g.beta_pre[c] = v[1];
    const float gate = o.gate ? o.gate[c] : 1.f;
    if (g.gamma_post) g.gamma_post[c] = gate * v[2];
    if (g.beta_post) g.beta_post[c] = gate * v[3];
    if (g.gate) g.gate[c] = fmaf(o.gamma_post ? o.gamma_post[c] : 1.f, v[2], o.beta_post ? o.beta_post[c] * v[3] : 0.f);
}

int row_threads_of(int H) { return (H / 4 + VPT * 32 - 1) / (VPT * 32) * 32; }

}  // namespace

// CTAs of the backward launch (each leaves 16 H bytes of partial sums).
int join_bwd_ctas(int T, int H)
{
    if (T <= 0) return 1;
    const int units = H <= WARP_COLS ? (T + WARPS - 1) / WARPS : T;
    const int most = num_sms() * (H <= WARP_COLS ? 2 : (row_threads_of(H) <= 256 ? 2 : 1));
    return units < most ? units : most;
}

cudaError_t launch_join(const ResidualOpts &o, const void *x, int x_fp32, const void *y, int y_fp32, int T, int H,
                        void *r, void *n, float *stats, cudaStream_t s)
{
    Residual p{};
    p.o = o;
    p.T = T; p.H = H; p.x_fp32 = x_fp32; p.y_fp32 = y_fp32;
    p.x = x; p.y = y; p.r = r; p.n = static_cast<uint16_t *>(n);
    p.stats = reinterpret_cast<float4 *>(stats);
    p.off[0] = 0;
    p.off[1] = H * (x_fp32 ? 4 : 2);
    p.stage_bytes = p.off[1] + H * (y_fp32 ? 4 : 2);
    const bool one = H <= WARP_COLS;
    const int threads = row_threads_of(H);
    dim3 block, grid;
    void (*kernel)(const Residual);
    if (one) {
        p.stages = 2;
        block = dim3(32, WARPS);
        const int units = (T + WARPS - 1) / WARPS, most = 4 * num_sms();
        grid = dim3(units < most ? units : most);
        kernel = join_kernel<true, 32 * WARPS, false>;
    } else {
        const int fit = static_cast<int>(ROOM / p.stage_bytes);
        int ctas = 512 / threads;
        if (ctas > fit / 2) ctas = fit / 2;
        if (ctas < 1) ctas = 1;
        p.stages = fit / ctas > 3 ? 3 : fit / ctas;
        block = dim3(threads);
        grid = dim3(T < ctas * num_sms() ? T : ctas * num_sms());
        kernel = threads <= 512 ? join_kernel<false, 512, true> : join_kernel<false, 1024, false>;
    }
    const size_t smem = static_cast<size_t>(p.stages) * p.stage_bytes * (one ? WARPS : 1);
    const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(kernel), smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, grid, block, smem, s, 1, p);
}

cudaError_t launch_join_bwd(const ResidualOpts &o, const void *dn, const void *dr, const void *y, int y_fp32,
                            const void *r, int x_fp32, const float *stats, int T, int H, void *dx, void *dy,
                            const ResidualGrads &g, float *part, cudaStream_t s)
{
    Residual p{};
    p.o = o;
    p.T = T; p.H = H; p.x_fp32 = x_fp32; p.y_fp32 = y_fp32;
    p.dn = static_cast<const uint16_t *>(dn);
    p.dr = dr;
    p.y = o.post || g.gate || g.gate_token ? y : nullptr;    // what nothing depends on is not read
    p.r = const_cast<void *>(r);
    p.stats = reinterpret_cast<float4 *>(const_cast<float *>(stats));
    p.dx = dx; p.dy = static_cast<uint16_t *>(dy);
    p.d_token = g.gate_token;
    p.part = part;
    const int xb = H * (x_fp32 ? 4 : 2), yb = H * (y_fp32 ? 4 : 2);
    int at = 0;
    auto take = [&](bool have, int bytes) {
        const int q = have ? at : -1;
        if (have) at += bytes;
        return q;
    };
    p.off[0] = take(o.pre != 0, H * 2);
    p.off[1] = take(o.pre != 0, xb);
    p.off[2] = take(p.y != nullptr, yb);
    const bool one = H <= WARP_COLS;
    const int ctas = join_bwd_ctas(T, H), per_sm = one ? 2 * WARPS : (row_threads_of(H) <= 256 ? 2 : 1);
    const size_t room = ROOM / per_sm;
    // dr is staged with the others where two stages fit so
    p.off[3] = take(dr && 2 * static_cast<size_t>(at + xb) <= room, xb);
    p.stage_bytes = at > 0 ? at : 16;
    const size_t fit = room / p.stage_bytes;
    p.stages = fit < 1 ? 1 : (fit > 3 ? 3 : static_cast<int>(fit));
    const size_t smem = static_cast<size_t>(p.stages) * p.stage_bytes * (one ? WARPS : 1);
    const int threads = row_threads_of(H);
    const bool s0 = o.beta_post != nullptr;
    void (*kernel)(const Residual) =
        one ? join_bwd_kernel<true, 32 * WARPS, true, false>
        : threads <= 256 ? (s0 ? join_bwd_kernel<false, 256, true, true> : join_bwd_kernel<false, 256, false, true>)
        : threads <= 448 ? (s0 ? join_bwd_kernel<false, 448, true, true> : join_bwd_kernel<false, 448, false, true>)
        : threads <= 512 ? (s0 ? join_bwd_kernel<false, 512, true, false> : join_bwd_kernel<false, 512, false, true>)
                         : join_bwd_kernel<false, 1024, true, false>;
    cudaError_t e = ensure_smem(reinterpret_cast<const void *>(kernel), smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kernel, dim3(ctas), one ? dim3(32, WARPS) : dim3(threads), smem, s, 1, p);
    if (e != cudaSuccess) return e;
    if (!g.gamma_post && !g.beta_post && !g.gate && !g.gamma_pre && !g.beta_pre) return cudaSuccess;
    return launch_pdl(join_wgrad_kernel, dim3(H / 32), dim3(32, 8), 0, s, 1, static_cast<const float *>(part), ctas, H, o, g);
}

}  // namespace moe
