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
// One warp per token, NV consecutive experts a lane.  Selection without a loop over K: a value
// that K of the 32 lanes' maxima reach (six halvings from their range come close to the K-th
// largest) is reached by K experts, so only the values at or above it, a dozen for K = 8, are
// candidates; they go to one lane each, in expert order, and every lane counts the candidates
// ahead of its own.  (Taking the maximum K times measured 26.6 us for 16384 tokens of 256
// experts, K = 8, without groups or bias; this 10.8 us.)  More than 32 candidates (many equal
// values) take that loop.
//
// The selection is exact: without a bias sel is ordered as the logits are, and those are
// compared as they stand.  Otherwise sel is held in fp32 with a bound on its error; the
// candidates reach down by twice that bound, and where two of them are closer than it, they
// are evaluated again in fp64, one a lane (a softmax, or group scores too close: the whole
// row, rare).
//
// The batch above with 8 groups (4 kept, two values each) and a bias takes 19 us: about 800
// instructions a token, where its bytes would take 2.6 us.  Two tokens take the launch's time.
//
// Gradient (D = sum_k w_k dw_k over the selected):
//   sigmoid, renormalised  dl_j = w_j (1 - s_j) (dw_j - D)
//   sigmoid                dl_j = s_j (1 - s_j) dw_j
//   softmax, renormalised  dl_j = w_j (dw_j - D)            (a softmax of the selected logits)
//   softmax                dl_e = s_e ([e selected] dw_e - sum_k s_k dw_k)    for every e
// (1 - s is taken as sigmoid(-l): the difference would lose what a saturated gate has left, 1e-3
// of it at a logit of 10 and all of it from 17 on.)
#include <cfloat>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int WPC = 8;                    // warps (tokens) a CTA
constexpr int MANY = 28;                  // candidates that are more than wanted (32 have a lane)
constexpr float kMaskedLogit = -3.38953139e38f;   // bf16's lowest value: at or below it, masked

// Values that rank below every sel or logit: masked ones (sums of two of them stay above
// the lowest float), and ones out of the running.
constexpr float kMaskedRank = -1e38f, kLeastRank = -9e37f;    // sel is kept at or above the latter
constexpr float kMaskedRankLogit = -3.395e38f;
// The same in fp64: values and sums of two of them in the same order as in fp32.
constexpr double kMaskedSel = -1e300, kLeastSel = 0.9 * kMaskedSel;
constexpr float kOut = -INFINITY;

// Integers that order as the floats do (for the warp-wide integer maximum).
__device__ __forceinline__ uint32_t order_key(float v)
{
    const uint32_t u = __float_as_uint(v);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k)
{
    return __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k);
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

__device__ __forceinline__ float fast_rcp(float v)      // within one step (0 for +inf, +inf for 0)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float sigmoid(float l) { return fast_rcp(1.f + expf(-l)); }

__device__ __forceinline__ void push2(float v, float &a, float &b)
{
    b = fmaxf(b, fminf(a, v));
    a = fmaxf(a, v);
}
__device__ __forceinline__ void push2(double v, double &a, double &b)
{
    if (v > a) { b = a; a = v; }
    else if (v > b) b = v;
}

// The lanes' scores up to a common factor, the largest near 1, where their sum is all that they
// are divided by: a softmax of the selected logits alone.  (The row's maximum need not be among
// them: 95 below it, where a bias chose them, their scores are denormal, and 0 from 104 on.)
// Masked logits are -inf here and give 0.
__device__ __forceinline__ float selected_exp(float l, bool on)
{
    const float top = key_value(__reduce_max_sync(kFullMask, order_key(on && l > -INFINITY ? l : -FLT_MAX)));
    return on ? expf(l - top) : 0.f;
}

// Sigmoids whose sum is below kSmallSum are e^l to 1e-12 of themselves, and below 2^-126 fp32 does
// not hold them: the same.  (0 where they are 0 in 64 bits too.)
constexpr float kSmallSum = 1e-12f, kNoScore = -708.f;

__device__ __forceinline__ float small_scores(float l, bool on)
{
    const float s = selected_exp(l, on);
    return __any_sync(kFullMask, on && l > kNoScore) ? s : 0.f;
}

// sigmoid from the hardware exp2 and reciprocal, for the selection (its error is in the bound)
__device__ __forceinline__ float rough_sigmoid(float l) { return fast_rcp(1.f + __expf(-l)); }

struct RouteArgs {
    const void *logits;
    const float *bias;      // nullable
    int fp32, T, E, K;
    int softmax, n_group, topk_group, group_top, renorm;
    int G;           // experts of a group
    // Experts of a lane: with lane_shift >= 0 a group has 2^lane_shift lanes, `per` consecutive
    // experts each (the last fewer); else the lanes take NV consecutive experts each.
    int lane_shift, per;
    int vec;         // lanes' experts start at multiples of 16 bytes of logits (and of 4 experts)
    int32_t *idx;
    float *w;
};

// The lane's experts: the first, and how many.
template <int NV>
__device__ __forceinline__ int lane_experts(const RouteArgs &a, int lane, int &live)
{
    if (a.lane_shift < 0) {
        live = a.E - lane * NV;
        return lane * NV;
    }
    const int g = lane >> a.lane_shift, r = (lane & ((1 << a.lane_shift) - 1)) * a.per;
    live = g < a.n_group ? min(a.per, a.G - r) : 0;
    return g * a.G + r;
}

// Rank of each lane's score among those of the first n lanes: descending, equal scores by lane.
template <typename F>
__device__ __forceinline__ int lane_rank(F score, int lane, int n)
{
    int rank = 0;
    for (int h = 0; h < n; ++h) {
        const F v = __shfl_sync(kFullMask, score, h);
        rank += v > score || (v == score && h < lane);
    }
    return rank;
}

// The same of the first n of a warp's values in shared memory (36 of them, kOut past n), which
// every lane reads four at a time.
__device__ __forceinline__ int rank_of(const float *f, float mine, int lane, int n)
{
    int rank = 0;
    for (int j = 0; j < n; j += 4) {
        const float4 o = *reinterpret_cast<const float4 *>(f + j);
        rank += j < lane ? o.x >= mine : o.x > mine;
        rank += j + 1 < lane ? o.y >= mine : o.y > mine;
        rank += j + 2 < lane ? o.z >= mine : o.z > mine;
        rank += j + 3 < lane ? o.w >= mine : o.w > mine;
    }
    return rank;
}

template <typename F>
__device__ __forceinline__ void merge2(F &a, F &b, int off)
{
    const F oa = __shfl_xor_sync(kFullMask, a, off), ob = __shfl_xor_sync(kFullMask, b, off);
    push2(oa, a, b);
    push2(ob, a, b);
}

// Lane g: the two largest of the values of group g (v: the lane's experts, `lowest` past them).
template <typename F, int NV>
__device__ __forceinline__ void group_top2(const RouteArgs &a, const F (&v)[NV], int lane, F lowest, F &s1, F &s2)
{
    const int G = a.G;
    F x = lowest, y = lowest;
    s1 = s2 = lowest;
    if (a.lane_shift >= 0) {
        // whole lanes hold a group
#pragma unroll
        for (int i = 0; i < NV; ++i) push2(v[i], x, y);
        for (int o = 1; o < 1 << a.lane_shift; o <<= 1) merge2(x, y, o);
        s1 = __shfl_sync(kFullMask, x, (lane << a.lane_shift) & 31);
        s2 = __shfl_sync(kFullMask, y, (lane << a.lane_shift) & 31);
        return;
    }
    for (int g = 0; g < a.n_group; ++g) {       // (lanes of NV experts)
        x = y = lowest;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = lane * NV + i;
            if (e >= g * G && e < (g + 1) * G) push2(v[i], x, y);
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) merge2(x, y, o);
        if (lane == g) { s1 = x; s2 = y; }
    }
}

// The selection in fp64, row by row as written down: lane j ends up with the j-th expert.
template <int NV>
__device__ __noinline__ int select_fp64(const RouteArgs &a, size_t base, int lane)
{
    double v[NV], m = -DBL_MAX, z = 0.0;
    int live;
    const int e0 = lane_experts<NV>(a, lane, live);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = e0 + i;
        const float l = i < live ? logit_at(a.logits, a.fp32, base + e) : -INFINITY;
        v[i] = l > kMaskedLogit ? static_cast<double>(l) : (l <= kMaskedLogit ? -INFINITY : NAN);
        if (l > kMaskedLogit) m = fmax(m, v[i]);
    }
    if (a.softmax) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(kFullMask, m, o));
        for (int i = 0; i < NV; ++i) z += exp(v[i] - m);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kFullMask, z, o);
    }
    const double inv = a.softmax ? 1.0 / z : 0.0;
    for (int i = 0; i < NV; ++i) {
        const int e = e0 + i;
        const bool on = v[i] > -INFINITY;
        double s = a.softmax ? exp(v[i] - m) * inv : 1.0 / (1.0 + exp(-v[i]));
        if (a.bias && i < live) s += static_cast<double>(a.bias[e]);
        // (a bias of -inf ranks above a mask, and every entry stays above what is taken out)
        v[i] = i >= live ? -DBL_MAX : (on && s == s ? fmax(s, kLeastSel) : kMaskedSel);
    }
    if (a.n_group > 1) {
        const int G = a.E / a.n_group;
        double s1, s2;
        group_top2<double, NV>(a, v, lane, 2 * kMaskedSel, s1, s2);
        const double score = a.group_top == 2 ? s1 + s2 : s1;
        const int rank = lane_rank(score, lane, a.n_group);
        const uint32_t kept = __ballot_sync(kFullMask, lane < a.n_group && rank < a.topk_group);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i < live && !((kept >> ((e0 + i) / G)) & 1u)) v[i] = -DBL_MAX;
    }
    int mine = 0;
    for (int k = 0; k < a.K; ++k) {
        double best = -DBL_MAX;
        int at = a.E - 1;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (v[i] > best) { best = v[i]; at = e0 + i; }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double w = __shfl_xor_sync(kFullMask, best, o);
            const int j = __shfl_xor_sync(kFullMask, at, o);
            if (w > best || (w == best && j < at)) { best = w; at = j; }
        }
        if (lane == k) mine = at;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i < live && e0 + i == at) v[i] = -DBL_MAX;
    }
    return mine;
}

// The groups kept (a bit each), by scores in fp64.  With a bias, of every lane's two largest
// values (sel within `bound`), where lanes hold whole groups, the score is a sigmoid and no
// lane's third value comes close to its second; 0 where that does not hold.  (Out of line, on
// values of its own: it is rare, and arrays handed to it would keep the caller's in local memory.)
template <int NV>
__device__ __noinline__ uint32_t groups_fp64(const RouteArgs &a, size_t base, int lane, float bound)
{
    int live;
    const int e0 = lane_experts<NV>(a, lane, live);
    if (!a.bias) {
        // the logits order a group's values exactly: its two largest logits, then their scores
        // (a softmax's up to a factor)
        float l[NV], m = -FLT_MAX, s1, s2;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            l[i] = i < live ? logit_at(a.logits, a.fp32, base + e0 + i) : kOut;
            if (i < live) l[i] = fmaxf(l[i] <= kMaskedLogit ? kMaskedRankLogit : l[i], kMaskedRankLogit);
            m = fmaxf(m, l[i]);
        }
        m = warp_max(m);
        group_top2<float, NV>(a, l, lane, -FLT_MAX, s1, s2);
        auto score = [&](float x) -> double {
            if (!(x > kMaskedLogit)) return kMaskedSel;
            const double d = static_cast<double>(x);
            return a.softmax ? exp(d - static_cast<double>(m)) : 1.0 / (1.0 + exp(-d));
        };
        const double two = score(s1) + (a.group_top == 2 ? score(s2) : 0.0);
        const int rank = lane_rank(two, lane, a.n_group);
        return __ballot_sync(kFullMask, lane < a.n_group && rank < a.topk_group);
    }
    if (a.softmax || a.lane_shift < 0) return 0u;
    const int per = 1 << a.lane_shift;
    float v1 = -FLT_MAX, v2 = -FLT_MAX, v3 = -FLT_MAX, l1 = 0.f, l2 = 0.f;
    int e1 = 0, e2 = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = e0 + i;
        if (i >= live) break;
        const float l = logit_at(a.logits, a.fp32, base + e);
        const float v = l <= kMaskedLogit ? kMaskedRank
                                          : fmaxf(rough_sigmoid(l) + (a.bias ? a.bias[e] : 0.f), kLeastRank);
        if (v > v1) {
            v3 = v2; v2 = v1; l2 = l1; e2 = e1;
            v1 = v; l1 = l; e1 = e;
        } else if (v > v2) {
            v3 = v2; v2 = v; l2 = l; e2 = e;
        } else {
            v3 = fmaxf(v3, v);
        }
    }
    if (__any_sync(kFullMask, v3 > kMaskedRank && !(v2 - v3 > 2.f * bound))) return 0u;
    auto exact = [&](float s, float x, int e) -> double {
        if (!(s > kMaskedRank)) return kMaskedSel;
        const double d = 1.0 / (1.0 + exp(-static_cast<double>(x)));
        return fmax(a.bias ? d + static_cast<double>(a.bias[e]) : d, kLeastSel);
    };
    const double d1 = exact(v1, l1, e1), d2 = exact(v2, l2, e2);
    double x = fmax(d1, d2), y = fmin(d1, d2);
    for (int o = 1; o < per; o <<= 1) merge2(x, y, o);
    x = __shfl_sync(kFullMask, x, lane * per & 31);
    y = __shfl_sync(kFullMask, y, lane * per & 31);
    const int rank = lane_rank(a.group_top == 2 ? x + y : x, lane, a.n_group);
    return __ballot_sync(kFullMask, lane < a.n_group && rank < a.topk_group);
}

// FULL: every lane holds NV experts.
template <int NV, bool F32, bool FULL>
__global__ void __launch_bounds__(32 * WPC, NV <= 8 ? 4 : 1) route_fwd_kernel(const __grid_constant__ RouteArgs a)
{
    __shared__ __align__(16) float cand_f[WPC][36];      // candidates in expert order
    __shared__ int cand_e[WPC][32];
    const int lane = threadIdx.x, wy = threadIdx.y, t = blockIdx.x * WPC + wy;
    pdl_wait();
    if (t >= a.T) return;
    const size_t base = static_cast<size_t>(t) * a.E;
    int live;                                // experts i < live of this lane exist
    const int e0 = lane_experts<NV>(a, lane, live);
    auto has = [&](int i) -> bool { return FULL || i < live; };

    float l[NV];
    if (F32 && NV % 4 == 0 && a.vec) {
        const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(a.logits) + base + e0);
#pragma unroll
        for (int i = 0; i < NV; i += 4) {
            const float4 v = has(i) ? src[i / 4] : make_float4(0.f, 0.f, 0.f, 0.f);
            l[i] = v.x; l[(i + 1) % NV] = v.y; l[(i + 2) % NV] = v.z; l[(i + 3) % NV] = v.w;
        }
    } else if (!F32 && NV % 8 == 0 && a.vec) {
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.logits) + base + e0);
#pragma unroll
        for (int i = 0; i < NV; i += 8) {
            const uint4 v = has(i) ? src[i / 8] : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) l[(i + k) % NV] = k & 1 ? bf16_hi(w[k / 2]) : bf16_lo(w[k / 2]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) l[i] = has(i) ? logit_at(a.logits, F32, base + e0 + i) : 0.f;
    }
    float m = -FLT_MAX, z = 1.f;
    if (a.softmax) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (has(i) && l[i] > kMaskedLogit) m = fmaxf(m, l[i]);
        m = warp_max(m);
        z = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) z += has(i) && !(l[i] <= kMaskedLogit) ? expf(l[i] - m) : 0.f;
        z = warp_sum(z);
    }
    // What the experts are ranked by: sel where there is a bias, else the logits, exactly.  The
    // groups are by sums of two scores even then.
    const bool scored = a.bias || (a.n_group > 1 && a.group_top == 2);
    const float inv = a.softmax && z != 0.f ? fast_rcp(z) : 0.f;
    auto by_logit = [&](float lg) -> float {     // (-0 ranks as +0, NaN as the lowest)
        return fmaxf(lg <= kMaskedLogit ? kMaskedRankLogit : lg + 0.f, kMaskedRankLogit);
    };
    auto by_score = [&](float lg, float bv) -> float {
        const float s = (a.softmax ? __expf(lg - m) * inv : rough_sigmoid(lg)) + bv;
        return lg <= kMaskedLogit ? kMaskedRank : fmaxf(s, kLeastRank);
    };
    // Error of a score: the sigmoid's is below 4e-7 (exp2, its argument's rounding, the
    // reciprocal).  The softmax's largest score is 1 / z; a score e^-x / z is off by 4 steps and
    // 2 x steps of 2^-24 of itself, and all by what z is: NV + 6 roundings of its sum and 3 of
    // its terms.  The rounding of s + bias comes to it: 1.5e-7 |sel|.
    const float error = scored ? (a.softmax ? (9e-7f + 6e-8f * NV) * inv : 4e-7f) : 0.f;
    float f[NV];
    if (a.bias && NV % 4 == 0 && a.vec) {
#pragma unroll
        for (int i = 0; i < NV; i += 4) {
            const float4 x = has(i) ? *reinterpret_cast<const float4 *>(a.bias + e0 + i) : make_float4(0.f, 0.f, 0.f, 0.f);
            f[i] = by_score(l[i], x.x);
            f[(i + 1) % NV] = by_score(l[(i + 1) % NV], x.y);
            f[(i + 2) % NV] = by_score(l[(i + 2) % NV], x.z);
            f[(i + 3) % NV] = by_score(l[(i + 3) % NV], x.w);
        }
    } else if (scored) {
#pragma unroll
        for (int i = 0; i < NV; ++i) f[i] = by_score(l[i], a.bias && has(i) ? a.bias[e0 + i] : 0.f);
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) f[i] = by_logit(l[i]);
    }
    if (!FULL) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (!has(i)) f[i] = kOut;
    }
    bool sure = true;
    if (a.n_group > 1) {
        float s1, s2;
        group_top2<float, NV>(a, f, lane, -FLT_MAX, s1, s2);
        const float score = a.group_top == 2 ? s1 + s2 : s1;
        const bool mine = lane < a.n_group;
        cand_f[wy][lane] = mine ? score : kOut;
        __syncwarp();
        const int rank = rank_of(cand_f[wy], score, lane, a.n_group);
        __syncwarp();
        uint32_t kept = __ballot_sync(kFullMask, mine && rank < a.topk_group);
        if (scored && a.topk_group < a.n_group) {
            const float lo = __shfl_sync(kFullMask, score, __ffs(__ballot_sync(kFullMask, mine && rank == a.topk_group - 1)) - 1);
            const float hi = __shfl_sync(kFullMask, score, __ffs(__ballot_sync(kFullMask, mine && rank == a.topk_group)) - 1);
            // (a score is the sum of two values, each within the bound at its own size, which the
            // sum need not have: values of opposite sign cancel; any group may be out of place)
            auto size = [](float v) -> float { return v > kLeastRank ? fabsf(v) : 0.f; };
            const float most = mine ? size(s1) + (a.group_top == 2 ? size(s2) : 0.f) : 0.f;
            const float bound = error + 1.5e-7f * __uint_as_float(__reduce_max_sync(kFullMask, __float_as_uint(most)));
            sure = lo - hi > 4.f * bound;
            if (!sure) {
                kept = groups_fp64<NV>(a, base, lane, bound);
                sure = kept != 0u;
            }
        }
        if (scored && !a.bias) {
#pragma unroll
            for (int i = 0; i < NV; ++i) f[i] = has(i) ? by_logit(l[i]) : kOut;
        }
        if (a.lane_shift >= 0) {
            // (by selection: a branch on the lane would split the warp for all that follows)
            const bool in = live > 0 && ((kept >> (lane >> a.lane_shift)) & 1u);
#pragma unroll
            for (int i = 0; i < NV; ++i) f[i] = in ? f[i] : kOut;
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (has(i) && !((kept >> ((e0 + i) / a.G)) & 1u)) f[i] = kOut;
        }
    }
    int expert = 0, place = 32;              // this lane's expert and its place in the order
    float lg = 0.f;                          // ... and its logit
    if (sure) {
        float x = kOut;                      // the lane's maximum
#pragma unroll
        for (int i = 0; i < NV; ++i) x = fmaxf(x, f[i]);
        // A value that K lanes' maxima reach (so K experts do), close to the K-th largest of them:
        // six halvings between the smallest and the largest maximum.
        float least = -FLT_MAX;
        const uint32_t some = __ballot_sync(kFullMask, x > kOut);
        const float top = key_value(__reduce_max_sync(kFullMask, order_key(x)));
        if (__popc(some) >= a.K) {
            float lo = key_value(__reduce_min_sync(kFullMask, x > kOut ? order_key(x) : 0xffffffffu)), hi = top;
#pragma unroll
            for (int r = 0; r < 6; ++r) {
                const float mid = 0.5f * lo + 0.5f * hi;
                const bool enough = __popc(__ballot_sync(kFullMask, x >= mid)) >= a.K;
                lo = enough ? mid : lo;
                hi = enough ? hi : mid;
            }
            least = lo;
        }
        // Where that leaves many candidates (few lanes hold what is in the running), halvings
        // over the experts themselves, from the lowest unmasked one.
        auto reach = [&](float v) -> int {       // experts at or above v
            int n = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) n += f[i] >= v;
            return static_cast<int>(__reduce_add_sync(kFullMask, n));
        };
        if (reach(least) > MANY) {
            const float floor_rank = a.bias ? kLeastRank : kMaskedRankLogit;
            uint32_t low = 0xffffffffu;
#pragma unroll
            for (int i = 0; i < NV; ++i) low = min(low, f[i] > floor_rank ? order_key(f[i]) : 0xffffffffu);
            low = __reduce_min_sync(kFullMask, low);
            float lo = fmaxf(least, low == 0xffffffffu ? -FLT_MAX : key_value(low)), hi = top;
            int n = reach(lo);
            if (n >= a.K) {
                for (int r = 0; r < 12 && n > MANY; ++r) {
                    const float mid = 0.5f * lo + 0.5f * hi;
                    const int c = reach(mid);
                    if (c >= a.K) { lo = mid; n = c; }
                    else hi = mid;
                }
                least = lo;
            }
        }
        float bound = 0.f;
        if (a.bias) {
            bound = error + 1.5e-7f * fmaxf(fabsf(top), fabsf(fmaxf(least, kLeastRank)));
            least -= 2.f * bound;
        }
        least = fmaxf(least, -FLT_MAX);
        uint32_t chosen = 0u;
#pragma unroll
        for (int i = 0; i < NV; ++i) chosen |= f[i] >= least ? 1u << i : 0u;
        const int n = __popc(chosen);
        int at = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int w = __shfl_up_sync(kFullMask, at, o);
            if (lane >= o) at += w;
        }
        const int C = __shfl_sync(kFullMask, at, 31);
        if (C <= 32) {
            at -= n;
            while (chosen) {
                cand_e[wy][at++] = e0 + __ffs(chosen) - 1;
                chosen &= chosen - 1u;
            }
            __syncwarp();
            float mine = kOut;
            if (lane < C) {
                expert = cand_e[wy][lane];
                lg = logit_at(a.logits, F32, base + expert);
                mine = a.bias ? by_score(lg, a.bias[expert]) : by_logit(lg);     // (as above)
            }
            cand_f[wy][lane] = mine;
            if (lane < 4) cand_f[wy][32 + lane] = kOut;
            __syncwarp();
            const int rank = rank_of(cand_f[wy], mine, lane, C);
            place = lane < C ? rank : 32;
            if (a.bias) {
                // neighbours in the order that the bound does not tell apart (masked experts
                // and biases of -inf are equal among themselves)
                __syncwarp();
                if (lane < C) cand_f[wy][rank] = mine;
                __syncwarp();
                const float next = lane < C ? cand_f[wy][rank + 1] : kOut;
                const bool close = mine > kLeastRank && next > kLeastRank && !(mine - next > 2.f * bound);
                if (__any_sync(kFullMask, close)) {
                    if (a.softmax) {
                        // z is known to (NV + 9) 2^-24 of it, so differences of the scores are
                        // to as much of themselves; closer than that, the whole row
                        double q = 0.0, d = -DBL_MAX;
                        if (lane < C) {
                            q = mine <= kMaskedRank ? 0.0 : exp(static_cast<double>(lg) - static_cast<double>(m)) / static_cast<double>(z);
                            d = mine <= kMaskedRank ? kMaskedSel : fmax(q + static_cast<double>(a.bias[expert]), kLeastSel);
                        }
                        int r64 = 0;
                        bool tie = false;
                        for (int h = 0; h < C; ++h) {
                            const double od = __shfl_sync(kFullMask, d, h), oq = __shfl_sync(kFullMask, q, h);
                            r64 += od > d || (od == d && h < lane);
                            tie = tie || (h != lane && fabs(od - d) <= (5e-7 + 1e-7 * NV) * fabs(oq - q) && oq != q);
                        }
                        if (lane < C) place = r64;
                        sure = !__any_sync(kFullMask, lane < C && (tie || !(q == q)));
                    } else {
                        double d = -DBL_MAX;
                        if (lane < C) {
                            d = 1.0 / (1.0 + exp(-static_cast<double>(lg))) + static_cast<double>(a.bias[expert]);
                            d = mine <= kMaskedRank ? kMaskedSel : fmax(d, kLeastSel);
                        }
                        const int r64 = lane_rank(d, lane, C);
                        if (lane < C) place = r64;
                    }
                }
            }
        } else if (a.bias) {
            sure = false;
        } else {
            for (int r = 0; r < a.K; ++r) {
                float best = kOut;
                int e = 1 << 30;
#pragma unroll
                for (int i = NV - 1; i >= 0; --i)
                    if (f[i] >= best && f[i] > kOut) { best = f[i]; e = e0 + i; }
                const uint32_t key = order_key(best), most = __reduce_max_sync(kFullMask, key);
                const int win = __reduce_min_sync(kFullMask, key == most ? e : 1 << 30);
                if (lane == r) { expert = win; place = r; }
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (e0 + i == win) f[i] = kOut;
            }
            if (place < a.K) lg = logit_at(a.logits, F32, base + expert);
        }
    }
    if (!sure) {
        expert = select_fp64<NV>(a, base, lane);
        place = lane;
        if (place < a.K) lg = logit_at(a.logits, F32, base + expert);
    }
    // weights: the selected scores (a masked expert's is 0), over their sum
    const bool on = place < a.K;
    if (on && lg <= kMaskedLogit) lg = -INFINITY;
    float s = 0.f;
    if (a.renorm) {
        s = a.softmax ? selected_exp(lg, on) : (on ? sigmoid(lg) : 0.f);
        float sum = warp_sum(s);
        if (!a.softmax && sum < kSmallSum) {
            s = small_scores(lg, on);
            sum = warp_sum(s);
        }
        s = sum == 0.f ? 0.f : s * fast_rcp(sum);
    } else if (on) {
        s = a.softmax ? expf(lg - m) * inv : sigmoid(lg);
    }
    if (on) {
        a.idx[static_cast<size_t>(t) * a.K + place] = expert;
        a.w[static_cast<size_t>(t) * a.K + place] = s;
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
        // (a softmax is renormalised here)
        float s = a.softmax ? selected_exp(l, e >= 0) : (e >= 0 ? sigmoid(l) : 0.f);
        if (a.renorm) {
            float sum = warp_sum(s);
            if (!a.softmax && sum < kSmallSum) {
                s = small_scores(l, e >= 0);
                sum = warp_sum(s);
            }
            const float w = sum == 0.f ? 0.f : s / sum;
            d = w * (dw - warp_sum(w * dw)) * (a.softmax ? 1.f : sigmoid(-l));
        } else {
            d = s * sigmoid(-l) * dw;
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
    const dim3 grid((a.T + WPC - 1) / WPC), block(32, WPC);
    const bool full = a.lane_shift >= 0 && a.per == NV && a.n_group << a.lane_shift == 32 && a.G == NV << a.lane_shift;
    if (full)
        return a.fp32 ? launch_pdl(route_fwd_kernel<NV, true, true>, grid, block, 0, s, 1, a)
                      : launch_pdl(route_fwd_kernel<NV, false, true>, grid, block, 0, s, 1, a);
    return a.fp32 ? launch_pdl(route_fwd_kernel<NV, true, false>, grid, block, 0, s, 1, a)
                  : launch_pdl(route_fwd_kernel<NV, false, false>, grid, block, 0, s, 1, a);
}

}  // namespace

cudaError_t launch_route(const void *logits, int fp32, const float *bias, int T, int E, int K,
                         const RoutingOpts &ro, int32_t *idx, float *w, cudaStream_t s)
{
    RouteArgs a{logits, bias, fp32, T, E, K, ro.scoring, ro.n_group, ro.topk_group, ro.group_top,
                ro.renorm, E / ro.n_group, 0, 0, 0, idx, w};
    // 2^lane_shift lanes a group, whole vectors of experts a lane where that fits
    while (ro.n_group << (a.lane_shift + 1) <= 32) ++a.lane_shift;
    const int lanes = 1 << a.lane_shift, v = fp32 ? 4 : 8;
    a.per = (a.G + lanes - 1) / lanes;
    if ((a.per + v - 1) / v * v <= 32) a.per = a.per > v / 2 ? (a.per + v - 1) / v * v : a.per;
    a.vec = a.G % v == 0 && a.per % v == 0;
    int nv = a.per;
    if (nv > 32) {                  // many groups of many experts: lanes and groups do not align
        a.lane_shift = -1;
        nv = (E + 31) / 32;
        a.vec = 0;
    }
    if (nv <= 1) return fwd<1>(a, s);
    if (nv <= 2) return fwd<2>(a, s);
    if (nv <= 4) return fwd<4>(a, s);
    if (nv <= 8) return fwd<8>(a, s);
    if (nv <= 16) return fwd<16>(a, s);
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
