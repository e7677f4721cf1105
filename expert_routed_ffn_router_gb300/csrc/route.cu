// route.cu -- top-K routing from given gate logits, and the gradient of its weights.
//
// "Lower latency and higher throughput with multi-node DeepSeek deployment", section "MoE
// Router": one router for every MoE model; here its scoring and selection alone, for a gate
// that the caller computes (fp32, with a mask or noise on its logits) and trains.
//
//   s = sigmoid(l) or softmax(l), sel = s + bias; the topk_group groups with the largest
//   group score (sum of the 1 or 2 largest sel), the K largest sel among their experts,
//   equal values by index; w = s / sum of the selected s, or s.
//
// One warp per token.  The selection is exact: without a bias sel is ordered as the logits
// are, and those are compared as they stand; otherwise sel is held in fp32 with a bound on
// its error, and a token with two neighbours in the order closer than their bounds (and not
// equal in logit and bias) is selected again in fp64.
//
// Gradient (D = sum_k w_k dw_k over the selected):
//   sigmoid, renormalised  dl_j = w_j (1 - s_j) (dw_j - D)
//   sigmoid                dl_j = s_j (1 - s_j) dw_j
//   softmax, renormalised  dl_j = w_j (dw_j - D)            (a softmax of the selected logits)
//   softmax                dl_e = s_e ([e selected] dw_e - sum_k s_k dw_k)    for every e
#include <cfloat>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int WPC = 4;                    // warps (tokens) a CTA
constexpr float kMaskedLogit = -3.38953139e38f;   // bf16's lowest value: at or below it, masked
constexpr double kMaskedSel = -1e300;     // fp64 order: a masked expert of a kept group

// Keys that order as the floats do; 0: not selectable, 1: masked or NaN.
__device__ __forceinline__ uint32_t order_key(float v)
{
    const uint32_t u = __float_as_uint(v);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFullMask, v, o));
    return v;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}

__device__ __forceinline__ float logit_at(const void *p, int fp32, size_t i)
{
    return fp32 ? static_cast<const float *>(p)[i]
                : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(p)[i]) << 16);
}

__device__ __forceinline__ float sigmoid(float l) { return 1.f / (1.f + expf(-l)); }

template <typename F>
__device__ __forceinline__ void push2(F v, F &a, F &b)
{
    if (v > a) { b = a; a = v; }
    else if (v > b) b = v;
}

struct RouteArgs {
    const void *logits;
    const float *bias;      // nullable
    int fp32, T, E, K;
    int softmax, n_group, topk_group, group_top, renorm;
    int32_t *idx;
    float *w;
};

// Groups kept (bit g) by their scores, from the warp's sel values in shared memory; *gap: the
// smallest kept score less the largest one not kept.
template <typename F>
__device__ __forceinline__ uint32_t keep_groups(const RouteArgs &a, const F *sel, int lane, F lowest, F *gap)
{
    const int G = a.E / a.n_group;
    F s1 = lowest, s2 = lowest;
    if (lane < a.n_group)
        for (int i = 0; i < G; ++i) push2(sel[lane * G + i], s1, s2);
    F score = a.group_top == 2 ? s1 + s2 : s1;
    if (!(score >= lowest)) score = lowest;     // (-inf, NaN)
    bool open = lane < a.n_group;
    uint32_t kept = 0;
    F last = 0, next = lowest;
    for (int r = 0; r <= a.topk_group && r < a.n_group; ++r) {
        F best = open ? score : lowest;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const F v = __shfl_xor_sync(kFullMask, best, o);
            best = v > best ? v : best;
        }
        const uint32_t at = __ballot_sync(kFullMask, open && score == best);
        const int g = __ffs(at) - 1;
        if (r == a.topk_group) { next = best; break; }
        last = best;
        kept |= 1u << g;
        if (lane == g) open = false;
    }
    *gap = last - next;
    return kept;
}

// The selection in fp64 (lane j ends up with the j-th expert).  sel: E doubles of this warp.
template <int NV>
__device__ __noinline__ int select_fp64(const RouteArgs &a, size_t base, int lane, double *sel)
{
    double m = 0.0, z = 1.0;
    if (a.softmax) {
        m = -DBL_MAX;
        for (int e = lane; e < a.E; e += 32) {
            const float l = logit_at(a.logits, a.fp32, base + e);
            if (l > kMaskedLogit) m = fmax(m, static_cast<double>(l));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(kFullMask, m, o));
        z = 0.0;
        for (int e = lane; e < a.E; e += 32) {
            const float l = logit_at(a.logits, a.fp32, base + e);
            if (l > kMaskedLogit) z += exp(static_cast<double>(l) - m);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kFullMask, z, o);
    }
    for (int e = lane; e < a.E; e += 32) {
        const double l = static_cast<double>(logit_at(a.logits, a.fp32, base + e));
        double v = a.softmax ? exp(l - m) / z : 1.0 / (1.0 + exp(-l));
        if (a.bias) v += static_cast<double>(a.bias[e]);
        // (a bias of -inf ranks above a mask, and every entry stays above what is taken out)
        sel[e] = l > kMaskedLogit && v == v ? fmax(v, 0.1 * kMaskedSel) : kMaskedSel;
    }
    __syncwarp();
    uint32_t kept = kFullMask;
    const int G = a.E / a.n_group;
    if (a.n_group > 1) {
        double gap;
        kept = keep_groups<double>(a, sel, lane, 2 * kMaskedSel, &gap);
    }
    for (int e = lane; e < a.E; e += 32)
        if (a.n_group > 1 && !((kept >> (e / G)) & 1u)) sel[e] = -DBL_MAX;
    __syncwarp();
    int mine = 0;
    for (int k = 0; k < a.K; ++k) {
        double best = -DBL_MAX;
        int at = a.E;
        for (int e = lane; e < a.E; e += 32)
            if (sel[e] > best) { best = sel[e]; at = e; }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double v = __shfl_xor_sync(kFullMask, best, o);
            const int i = __shfl_xor_sync(kFullMask, at, o);
            if (v > best || (v == best && i < at)) { best = v; at = i; }
        }
        if (lane == k) mine = at;
        if (lane == (at & 31)) sel[at] = -DBL_MAX;
        __syncwarp();
    }
    return mine;
}

template <int NV>
__global__ void __launch_bounds__(32 * WPC) route_fwd_kernel(const RouteArgs a)
{
    extern __shared__ double sm_sel[];      // [WPC][E] (fp32 for the group scores, fp64 again)
    pdl_wait();
    const int lane = threadIdx.x, t = blockIdx.x * WPC + threadIdx.y;
    if (t >= a.T) return;
    const size_t base = static_cast<size_t>(t) * a.E;
    double *sel64 = sm_sel + static_cast<size_t>(threadIdx.y) * a.E;
    float *sel32 = reinterpret_cast<float *>(sel64);

    float l[NV], v[NV];        // logit; then score
    uint32_t key[NV];
    float m = -FLT_MAX;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane + 32 * i;
        l[i] = e < a.E ? logit_at(a.logits, a.fp32, base + e) : -INFINITY;
        if (l[i] > kMaskedLogit) m = fmaxf(m, l[i]);
        else if (l[i] <= kMaskedLogit) l[i] = -INFINITY;     // (NaN stays)
    }
    float z = 1.f;
    if (a.softmax) {
        m = warp_max(m);
        z = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            v[i] = expf(l[i] - m);
            z += v[i];
        }
        z = warp_sum(z);
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = z > 0.f || z != z ? v[i] / z : 0.f;
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = sigmoid(l[i]);
    }
    // Order keys.  No bias and no sum of two scores: the logits themselves, exactly.
    const bool scored = a.bias || (a.n_group > 1 && a.group_top == 2);
    float most = 0.f;          // largest |sel| (scales the error bound)
    float bv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane + 32 * i;
        bv[i] = a.bias && e < a.E ? a.bias[e] : 0.f;
        const float s = a.bias ? v[i] + bv[i] : l[i] + 0.f;     // (-0 ranks as +0)
        const bool ok = l[i] > -INFINITY && s == s;
        key[i] = e >= a.E ? 0u : (ok ? order_key(s) : 1u);
        if (scored && ok && fabsf(s) < INFINITY) most = fmaxf(most, fabsf(v[i] + bv[i]));
    }
    // Error of sel: fp32 exp, sum and division of s <= 1, and the rounding of s + bias.  For
    // the softmax an error of the argument l - m and of the sum of up to 1024 terms comes in.
    float bound = 0.f;
    if (scored) bound = 6e-7f + 1.5e-7f * warp_max(most) + (a.softmax ? 2.5e-6f : 0.f);
    bool sure = true;
    if (a.n_group > 1) {
        const int G = a.E / a.n_group;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E) {
                // (masked: below every sel, their sum above `lowest`; below every logit)
                sel32[e] = key[i] <= 1u ? (scored ? -1e38f : -3.395e38f) : (scored ? v[i] + bv[i] : l[i]);
            }
        }
        __syncwarp();
        float gap;
        const uint32_t kept = keep_groups<float>(a, sel32, lane, -FLT_MAX, &gap);
        if (scored && a.topk_group < a.n_group) sure = gap > 4.f * bound;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E && !((kept >> (e / G)) & 1u)) key[i] = 0u;
        }
    }
    int mine = 0;
    float prev = 0.f, prev_l = 0.f, prev_b = 0.f;
    uint32_t prev_key = 0u;
    for (int k = 0; k <= a.K && sure; ++k) {
        uint32_t best = 0u;
#pragma unroll
        for (int i = 0; i < NV; ++i) best = key[i] > best ? key[i] : best;
        const uint32_t top = __reduce_max_sync(kFullMask, best);
        if (top == 0u || (k == a.K && !a.bias)) break;
        int at = 1 << 30;
        float wl = 0.f, wb = 0.f;
#pragma unroll
        for (int i = NV - 1; i >= 0; --i)
            if (key[i] == top) { at = lane + 32 * i; wl = l[i]; wb = bv[i]; }
        const int win = __reduce_min_sync(kFullMask, at);
        if (a.bias) {
            // certified against the one before it
            wl = __shfl_sync(kFullMask, wl, win & 31);
            wb = __shfl_sync(kFullMask, wb, win & 31);
            const float cur = top > 1u ? __uint_as_float((top >> 31) ? top & 0x7fffffffu : ~top) : -INFINITY;
            if (k > 0 && top > 1u && prev_key > 1u && !(prev - cur > 2.f * bound) && !(prev_l == wl && prev_b == wb))
                sure = false;
            prev = cur; prev_l = wl; prev_b = wb; prev_key = top;
        }
        if (k == a.K) break;
        if (lane == k) mine = win;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (lane + 32 * i == win) key[i] = 0u;
    }
    if (!sure) {
        __syncwarp();
        mine = select_fp64<NV>(a, base, lane, sel64);
    }
    // weights: the selected scores (a masked expert's is 0), over their sum
    float s = 0.f;
    if (lane < a.K) {
        float lj = logit_at(a.logits, a.fp32, base + mine);
        if (lj <= kMaskedLogit) lj = -INFINITY;
        s = !a.softmax ? sigmoid(lj) : (z > 0.f || z != z ? expf(lj - m) / z : 0.f);
    }
    if (a.renorm) {
        const float sum = warp_sum(s);
        s = sum == 0.f ? 0.f : s / sum;
    }
    if (lane < a.K) {
        a.idx[static_cast<size_t>(t) * a.K + lane] = mine;
        a.w[static_cast<size_t>(t) * a.K + lane] = s;
    }
}

struct RouteBwdArgs {
    const void *logits;
    int fp32, T, E, K, softmax, renorm;
    const int32_t *idx;
    const float *dw;
    void *dl;
};

__global__ void __launch_bounds__(32 * WPC) route_bwd_kernel(const RouteBwdArgs a)
{
    extern __shared__ float sm_row[];       // [WPC][E]
    pdl_wait();
    const int lane = threadIdx.x, t = blockIdx.x * WPC + threadIdx.y;
    if (t >= a.T) return;
    const size_t base = static_cast<size_t>(t) * a.E;
    float *row = sm_row + static_cast<size_t>(threadIdx.y) * a.E;
    int e = -1;
    float dw = 0.f, l = -INFINITY;
    if (lane < a.K) {
        e = a.idx[static_cast<size_t>(t) * a.K + lane];
        if (e < 0 || e >= a.E) e = -1;      // (a rejected pair has no gradient)
        else {
            dw = a.dw[static_cast<size_t>(t) * a.K + lane];
            l = logit_at(a.logits, a.fp32, base + e);
            if (l <= kMaskedLogit) l = -INFINITY;
        }
    }
    float d;
    const bool dense = a.softmax && !a.renorm;
    float m = -FLT_MAX, z = 0.f, dot = 0.f;
    if (dense) {
        for (int i = lane; i < a.E; i += 32) {
            const float v = logit_at(a.logits, a.fp32, base + i);
            row[i] = v <= kMaskedLogit ? -INFINITY : v;
            if (!(v <= kMaskedLogit)) m = fmaxf(m, v);
        }
        m = warp_max(m);
        for (int i = lane; i < a.E; i += 32) {
            row[i] = expf(row[i] - m);
            z += row[i];
        }
        z = warp_sum(z);
        const float r = z == 0.f ? 0.f : 1.f / z;
        const float s = e >= 0 ? expf(l - m) * r : 0.f;
        dot = warp_sum(s * dw);
        for (int i = lane; i < a.E; i += 32) row[i] *= -dot * r;
        __syncwarp();
        d = s * dw;      // added to its entry of the row
    } else {
        for (int i = lane; i < a.E; i += 32) row[i] = 0.f;
        __syncwarp();
        float s, w;
        if (a.softmax) {     // renormalised: a softmax of the selected logits
            m = warp_max(l > -INFINITY || l != l ? l : -FLT_MAX);
            s = e >= 0 ? expf(l - m) : 0.f;
        } else {
            s = e >= 0 ? sigmoid(l) : 0.f;
        }
        if (a.renorm) {
            const float sum = warp_sum(s);
            w = sum == 0.f ? 0.f : s / sum;
            d = w * (dw - warp_sum(w * dw));
            if (!a.softmax) d *= 1.f - s;
        } else {
            d = s * (1.f - s) * dw;
        }
    }
    if (e >= 0) row[e] += d;
    __syncwarp();
    for (int i = lane; i < a.E; i += 32) {
        if (a.fp32) static_cast<float *>(a.dl)[base + i] = row[i];
        else static_cast<uint16_t *>(a.dl)[base + i] = static_cast<uint16_t>(f32x2_to_bf16x2(0.f, row[i]));
    }
}

template <int NV>
cudaError_t fwd(const RouteArgs &a, cudaStream_t s)
{
    const size_t smem = static_cast<size_t>(WPC) * a.E * sizeof(double);
    const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(route_fwd_kernel<NV>), smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(route_fwd_kernel<NV>, dim3((a.T + WPC - 1) / WPC), dim3(32, WPC), smem, s, 1, a);
}

}  // namespace

cudaError_t launch_route(const void *logits, int fp32, const float *bias, int T, int E, int K,
                         const RoutingOpts &ro, int32_t *idx, float *w, cudaStream_t s)
{
    const RouteArgs a{logits, bias, fp32, T, E, K, ro.scoring, ro.n_group, ro.topk_group, ro.group_top,
                      ro.renorm, idx, w};
    if (E <= 32) return fwd<1>(a, s);
    if (E <= 64) return fwd<2>(a, s);
    if (E <= 128) return fwd<4>(a, s);
    if (E <= 256) return fwd<8>(a, s);
    if (E <= 512) return fwd<16>(a, s);
    return fwd<32>(a, s);
}

cudaError_t launch_route_bwd(const void *logits, int fp32, int T, int E, int K, const RoutingOpts &ro,
                             const int32_t *idx, const float *dw, void *dl, cudaStream_t s)
{
    const RouteBwdArgs a{logits, fp32, T, E, K, ro.scoring, ro.renorm, idx, dw, dl};
    return launch_pdl(route_bwd_kernel, dim3((T + WPC - 1) / WPC), dim3(32, WPC),
                      static_cast<size_t>(WPC) * E * sizeof(float), s, 1, a);
}

}  // namespace moe
