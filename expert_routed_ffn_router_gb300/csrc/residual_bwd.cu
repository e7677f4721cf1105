// residual_bwd.cu -- backward pass of the joined residual (formulas: residual.cuh).
//
// A turn of the loop takes the branch's sums of one row (whose d is in registers) and the next norm's
// sums of the following one through the same exchange: a row costs one barrier.  d stays in registers
// from one to the other; dn, r, dr and y are staged in shared memory.
//
// The parameters' gradients.  Each CTA walks rows blockIdx.x, + gridDim.x, ... and keeps the sums
// of its columns in registers; the CTAs' sums go to the workspace ([CTA][4][H]) and a second
// launch (or, where up to eight CTAs do, their cluster) adds them in CTA order.  No atomics: for the same
// sizes, types and set of arrays (they decide how many CTAs there are) the result repeats bit for bit.
//
// What bounds it: memory in fp32 (16384 x 7168, RMS norm of y, layer norm of r: 350 us, 6.7 TB/s, 99% of
// the copy bandwidth).  In bf16 (302 us, 4.7 TB/s) neither memory nor the schedulers (58% of the issue slots) are
// at their end.  Two stages at most: with three of bf16 rows that call takes 386 us.  Rows of more than 8192
// columns (1024 threads of 64 registers, types told by flags) spill 540 bytes a thread: 4096 x 8192 in fp32
// 116 us, 4096 x 8256 406 us; in bf16 100 and 382 us.
#include "residual.cuh"

namespace moe {
namespace residual {
namespace {

// The columns' gradients from their sums v: of dn rh, of dn, S1, S0.
__device__ __forceinline__ void store_columns(const ResidualOpts &o, const ResidualGrads &g, int c, const float (&v)[4])
{
    if (g.gamma_pre) g.gamma_pre[c] = v[0];
    if (g.beta_pre) g.beta_pre[c] = v[1];
    const float gate = o.gate ? o.gate[c] : 1.f;
    if (g.gamma_post) g.gamma_post[c] = gate * v[2];
    if (g.beta_post) g.beta_post[c] = gate * v[3];
    if (g.gate) g.gate[c] = fmaf(o.gamma_post ? o.gamma_post[c] : 1.f, v[2], o.beta_post ? o.beta_post[c] * v[3] : 0.f);
}

// Staged arrays: 0 dn, 1 r, 2 dr (of a row's first part), 3 y (of its second one).  Where dr does not fit
// `stages` times with the others it is staged once (dr_once): a row's is read at the end of a turn, and
// the next one has a turn to arrive.  N: threads of a row (32: a warp, with WARPS rows a CTA).
// The columns' parameters stay in registers, and with them the sums p1 and s1; those of plain rows, p0 and
// (BOTH: with beta_post) s0, in shared memory, every thread its own columns.  Where that is full
// (IN_MEMORY) all sums are in registers and the parameters in memory.  (Everything in registers spills, and
// with most of an SM's L1 taken as shared memory spills go to L2: 16384 x 7168 in fp32, RMS norm and layer
// norm, two spilled registers: 592 us, 350 us so; with beta_post and gates of both kinds 693 us with
// IN_MEMORY, 1000 us with spills, 490 us with BOTH.)
enum { ONE_SHARED, BOTH, IN_MEMORY };

template <int N, int SUMS, int XT, int YT>
__global__ void __launch_bounds__(N == 32 ? 32 * WARPS : N, N <= 512 ? 512 / (N == 32 ? 256 : N) : 1)
    join_bwd_kernel(const __grid_constant__ Args p)
{
    constexpr bool ONE = N == 32, S0 = SUMS != ONE_SHARED, PREG = SUMS != IN_MEMORY;
    extern __shared__ __align__(16) unsigned char stages[];
    __shared__ float4 red[2][N / 32];
    __shared__ float red_token[2][N / 32];
    const int H = p.H, S = p.stages;
    const bool xf = p.x_fp32, yf = p.y_fp32;
    const ResidualOpts &o = p.o;
    const Columns<N> in{H / 4, static_cast<int>(threadIdx.x)};
    const int tid = in.tid;
    Exchange<N> exchange{red, tid};
    unsigned char *ring = stages + (ONE ? threadIdx.y * p.row_bytes : 0);
    const uint32_t ring_at = smem_u32(ring);
    const int first = ONE ? blockIdx.x * WARPS + threadIdx.y : blockIdx.x, step = ONE ? gridDim.x * WARPS : gridDim.x;
    pdl_wait();
    auto fetch_first = [&](int row, int s) {         // what the first part of a row reads
        if (row >= p.T) return;
        const uint32_t st = ring_at + s * p.stage_bytes;
        if (p.off[0] >= 0) stage_in<BF16, N>(st + p.off[0], p.dn, row, H, false, in);
        if (p.off[1] >= 0) stage_in<XT, N>(st + p.off[1], p.r, row, H, xf, in);
        if (p.off[2] >= 0 && !p.dr_once) stage_in<XT, N>(st + p.off[2], p.dr, row, H, xf, in);
    };
    auto fetch_dr = [&](int row) {
        if (row < p.T && p.dr_once) stage_in<XT, N>(ring_at + p.off[2], p.dr, row, H, xf, in);
        copies_commit();
    };
    auto fetch_second = [&](int row, int s) {
        if (row < p.T && p.off[3] >= 0) stage_in<YT, N>(ring_at + s * p.stage_bytes + p.off[3], p.y, row, H, yf, in);
    };
    constexpr int PV = PREG ? VPT : 1, SV = SUMS == IN_MEMORY ? VPT : 1;
    float4 p1[VPT], p0[SV], s1[VPT], s0[SV], ga[PV], gb[PV];
    float4 *p0s = reinterpret_cast<float4 *>(ring + p.sum[0]) + tid, *s0s = reinterpret_cast<float4 *>(ring + p.sum[1]) + tid;
    auto scale = [&](int k) { return mul4(col4<N>(o.gate, tid, k, 1.f), col4<N>(o.gamma_post, tid, k, 1.f)); };
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        p1[k] = p0[k % SV] = s1[k] = s0[k % SV] = all4(0.f);
        if (PREG && in(k)) {
            p0s[k * N] = all4(0.f);
            if (S0) s0s[k * N] = all4(0.f);
        }
        if (PREG && in(k)) {
            ga[k % PV] = col4<N>(o.gamma_pre, tid, k, 1.f);
            gb[k % PV] = scale(k);
        }
    }
    auto gamma = [&](int k) { return PREG ? ga[k % PV] : col4<N>(o.gamma_pre, tid, k, 1.f); };
    auto branch = [&](int k) { return PREG ? gb[k % PV] : scale(k); };
    const float inv = 1.f / static_cast<float>(H);
    const bool token = p.d_token != nullptr, sums = o.pre || o.post || token, y = p.y != nullptr;
    const float ly = o.post == 1 ? inv : 0.f, py = o.post ? inv : 0.f, lr = o.pre == 1 ? inv : 0.f;

    // A turn's copies, to the places that it has just read: dr of the row after the next one; the first part
    // of the row S further on with the second part of the one before that.
    for (int s = 0; s < S; ++s) {
        if (s == S - 1) fetch_dr(first);
        else copies_commit();
        fetch_first(first + s * step, s);
        if (s > 0) fetch_second(first + (s - 1) * step, s - 1);
        copies_commit();
    }
    auto row_stats = [&](int row) {
        float4 v = row < p.T ? p.stats[row] : all4(0.f);
        if (!o.post) { v.x = 0.f; v.y = 1.f; }
        return v;
    };
    auto row_gate = [&](int row) { return o.gate_token && row < p.T ? o.gate_token[row] : 1.f; };
    float4 st = all4(0.f), st_next = row_stats(first);   // statistics of the row at hand, of the next one
    float gt = 1.f, gt_next = row_gate(first);
    float4 d[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) d[k] = all4(0.f);
    int s = 0, sp = S - 1;                           // places of the next row, of the one at hand
    for (int next = first, row = -1; next < p.T || row >= 0; next += step) {
        const bool has = row >= 0, more = next < p.T;
        const unsigned char *sm = ring + s * p.stage_bytes;
        const unsigned char *gs = staged<BF16>(sm + p.off[0], tid, false), *rs = staged<XT>(sm + p.off[1], tid, xf);
        const unsigned char *ys = staged<YT>(ring + sp * p.stage_bytes + p.off[3], tid, yf);
        copies_wait(2 * (S - 1));
        float e[5] = {0.f, 0.f, 0.f, 0.f, 0.f};
        if (more && o.pre) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                if (!in(k)) continue;
                const float4 g = ld4<BF16, N>(gs, k, false), h = norm4(ld4<XT, N>(rs, k, xf), st_next.z, st_next.w);
                p1[k] = fma4(g, h, p1[k]);
                if (PREG) p0s[k * N] = add4(p0s[k * N], g);
                else p0[k % SV] = add4(p0[k % SV], g);
                const float4 a = mul4(g, gamma(k));
                e[0] += sum4(a);
                e[1] += dot4(a, h);
            }
        }
        if (has) {
            unsigned char *to = row_at<XT>(p.dx, row, H, tid, xf);
#pragma unroll
            for (int k = 0; k < VPT; ++k)
                if (in(k)) st4<XT, N>(to, k, xf, scale4(d[k], o.alpha));
            if (y) {                                 // the branch: f = g_h gamma_post d
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    if (!in(k)) continue;
                    const float4 h = norm4(ld4<YT, N>(ys, k, yf), st.x, st.y), g = scale4(d[k], gt);
                    s1[k] = fma4(g, h, s1[k]);
                    if (SUMS == BOTH) s0s[k * N] = add4(s0s[k * N], g);
                    else if (S0) s0[k % SV] = add4(s0[k % SV], g);
                    const float4 f = mul4(d[k], branch(k));
                    e[2] += sum4(f);
                    e[3] += dot4(f, h);
                }
            }
            if (S0 && token) {
#pragma unroll
                for (int k = 0; k < VPT; ++k)
                    if (in(k)) e[4] += dot4(mul4(d[k], col4<N>(o.gate, tid, k, 1.f)), col4<N>(o.beta_post, tid, k, 0.f));
            }
        }
        if (sums) {
            if (ONE) {
                const float2 a = warp_pair_all(e[0], e[1]), f = warp_pair_all(e[2], e[3]);
                e[0] = a.x; e[1] = a.y; e[2] = f.x; e[3] = f.y;
                if (S0 && token) e[4] = warp_pair_all(e[4], 0.f).x;
            } else {
                if (S0 && token) {
                    e[4] = warp_pair(e[4], 0.f);
                    if ((tid & 31) == 0) red_token[exchange.turn][tid >> 5] = e[4];
                }
                const int turn = exchange.turn;
                const float4 w = exchange(warp_pair(e[0], e[1]), warp_pair(e[2], e[3]));
                const float2 a = warp_pair_all(w.x, w.y), f = warp_pair_all(w.z, w.w);
                e[0] = a.x; e[1] = a.y; e[2] = f.x; e[3] = f.y;
                if (S0 && token) e[4] = warp_pair_all((tid & 31) < N / 32 ? red_token[turn][tid & 31] : 0.f, 0.f).x;
            }
        }
        if (has) {
            if (token && tid == 0) p.d_token[row] = e[3] + e[4];
            const float a0 = e[2] * ly, a1 = e[3] * py, z = o.post ? gt * st.y : gt;
            unsigned char *to = row_at<BF16>(p.dy, row, H, tid, false);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                if (!in(k)) continue;
                float4 f = mul4(d[k], branch(k));
                if (o.post) {
                    const float4 h = norm4(ld4<YT, N>(ys, k, yf), st.x, st.y);
                    f = make_float4(f.x - a0 - h.x * a1, f.y - a0 - h.y * a1, f.z - a0 - h.z * a1, f.w - a0 - h.w * a1);
                }
                st4<BF16, N>(to, k, false, scale4(f, z));
            }
        }
        if (more) {
            // (a row of dr that is not staged comes from memory)
            const unsigned char *ds = p.off[2] < 0 ? row_at<XT>(p.dr, next, H, tid, xf)
                                                   : staged<XT>((p.dr_once ? ring : sm) + p.off[2], tid, xf);
            if (p.dr_once) copies_wait(1);
#pragma unroll
            for (int k = 0; k < VPT; ++k) d[k] = p.dr && in(k) ? ld4<XT, N>(ds, k, xf) : all4(0.f);
            if (o.pre) {
                const float a0 = e[0] * lr, a1 = e[1] * inv, z = st_next.w;
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    if (!in(k)) continue;
                    const float4 h = norm4(ld4<XT, N>(rs, k, xf), st_next.z, z), a = mul4(ld4<BF16, N>(gs, k, false), gamma(k));
                    d[k].x = fmaf(z, a.x - a0 - h.x * a1, d[k].x);
                    d[k].y = fmaf(z, a.y - a0 - h.y * a1, d[k].y);
                    d[k].z = fmaf(z, a.z - a0 - h.z * a1, d[k].z);
                    d[k].w = fmaf(z, a.w - a0 - h.w * a1, d[k].w);
                }
            }
        }
        st = st_next;
        gt = gt_next;
        st_next = row_stats(next + step);
        gt_next = row_gate(next + step);
        fetch_dr(next + step);
        fetch_first(next + S * step, s);
        fetch_second(next + (S - 1) * step, sp);
        copies_commit();
        row = more ? next : -1;
        sp = s;
        if (++s == S) s = 0;
    }
    float4 *part = reinterpret_cast<float4 *>(p.part + static_cast<size_t>(blockIdx.x) * 4 * H) + tid;
    const int vec = H / 4;
    if constexpr (!ONE) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            if (!in(k)) continue;
            part[k * N] = p1[k];
            part[vec + k * N] = PREG ? p0s[k * N] : p0[k % SV];
            part[2 * vec + k * N] = s1[k];
            part[3 * vec + k * N] = SUMS == BOTH ? s0s[k * N] : s0[k % SV];
        }
    } else {
        // the warps' sums, added in their order
        __shared__ float4 comb[WARPS][33];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                __syncthreads();
                comb[threadIdx.y][tid] = j == 0 ? p1[k] : j == 1 ? p0[k % SV] : j == 2 ? s1[k] : s0[k % SV];
                __syncthreads();
                if (threadIdx.y == 0 && in(k)) {
                    float4 t = comb[0][tid];
                    for (int q = 1; q < WARPS; ++q) t = add4(t, comb[q][tid]);
                    part[j * vec + k * N] = t;
                }
            }
    }
    // Few CTAs are one cluster: its columns' sums are added here, in the order of join_wgrad_kernel (45 x 256: a
    // launch less, 17.9 -> 14.7 us a call).
    if (p.joined) {
        cluster_sync();
        const int threads = ONE ? 32 * WARPS : N, me = ONE ? threadIdx.y * 32 + threadIdx.x : threadIdx.x;
        for (int c = blockIdx.x * threads + me; c < H; c += gridDim.x * threads) {
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            for (int q = 0; q < static_cast<int>(gridDim.x); ++q)
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] += __ldcg(p.part + (static_cast<size_t>(q) * 4 + k) * H + c);
            store_columns(o, p.g, c, v);
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
#pragma unroll 4
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
    store_columns(o, g, c, v);
}

using Kernel = void (*)(const Args);

template <int N, int SUMS>
Kernel of_types(int x_fp32, int y_fp32)
{
    return x_fp32 ? (y_fp32 ? join_bwd_kernel<N, SUMS, FP32, FP32> : join_bwd_kernel<N, SUMS, FP32, BF16>)
                  : (y_fp32 ? join_bwd_kernel<N, SUMS, BF16, FP32> : join_bwd_kernel<N, SUMS, BF16, BF16>);
}

template <int N>
Kernel of_rows(int sums, int x_fp32, int y_fp32)
{
    return sums == ONE_SHARED ? of_types<N, ONE_SHARED>(x_fp32, y_fp32)
           : sums == BOTH     ? of_types<N, BOTH>(x_fp32, y_fp32) : of_types<N, IN_MEMORY>(x_fp32, y_fp32);
}

constexpr int CLUSTER = 8;
// CTAs that share an SM, at most
int per_sm(int H) { const int n = row_threads(H); return n == 32 ? 2 : (n < 512 ? 512 / n : 1); }

}  // namespace
}  // namespace residual

// CTAs of the backward launch at most (each leaves 16 H bytes of partial sums).  Up to CLUSTER they may be a
// cluster, whose size is a power of two: CTAs without a row leave zeros.
int join_bwd_ctas(int T, int H)
{
    using namespace residual;
    if (T <= 0) return 1;
    const int units = H <= WARP_COLS ? (T + WARPS - 1) / WARPS : T;
    const int most = num_sms() * per_sm(H);
    if (units <= residual::CLUSTER) return units <= 1 ? 1 : units <= 2 ? 2 : units <= 4 ? 4 : 8;
    return units < most ? units : most;
}

cudaError_t launch_join_bwd(const ResidualOpts &o, const void *dn, const void *dr, const void *y, int y_fp32,
                            const void *r, int x_fp32, const float *stats, int T, int H, void *dx, void *dy,
                            const ResidualGrads &g, float *part, cudaStream_t s)
{
    using namespace residual;
    Args p{};
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
    const int threads = row_threads(H);
    const bool one = threads == 32;
    p.off[0] = take(o.pre != 0, H * 2);
    p.off[1] = take(o.pre != 0, xb);
    p.off[3] = take(p.y != nullptr, yb);
    // As many CTAs an SM as have room for two stages, dr and the sums of plain rows.  Then dr in every stage
    // where two fit so, else once, else not at all.
    const size_t own = (o.beta_post ? 8 : 4) * static_cast<size_t>(H);
    auto room_of = [&](int k) { return (k == 1 ? MOST : ROOM) / (k * (one ? WARPS : 1)); };
    int ctas_sm = per_sm(H), sums = IN_MEMORY;
    for (int k = ctas_sm; !one && threads <= 512 && k >= 1 && sums == IN_MEMORY; --k)
        if (2 * static_cast<size_t>(at) + (dr ? xb : 0) + own <= room_of(k)) {
            sums = o.beta_post ? BOTH : ONE_SHARED;
            ctas_sm = k;
        }
    const size_t room = room_of(ctas_sm), rows = room - (sums != IN_MEMORY ? own : 0);
    p.off[2] = -1;
    if (dr && 2 * static_cast<size_t>(at + xb) <= rows) {
        p.off[2] = take(true, xb);
    } else if (dr && static_cast<size_t>(at + xb) <= rows) {
        p.dr_once = 1;
    }
    p.stage_bytes = at > 0 ? at : 16;
    const size_t fit = (rows - (p.dr_once ? xb : 0)) / p.stage_bytes;
    p.stages = fit > 2 ? 2 : static_cast<int>(fit);
    int end = p.stages * p.stage_bytes;
    if (p.dr_once) { p.off[2] = end; end += xb; }
    if (sums != IN_MEMORY) {
        p.sum[0] = end;
        p.sum[1] = end + 4 * H;
        end += static_cast<int>(own);
    }
    p.row_bytes = end;
    const size_t smem = static_cast<size_t>(end) * (one ? WARPS : 1);
    const Kernel kernel = threads == 32    ? of_types<32, IN_MEMORY>(x_fp32, y_fp32)
                          : threads == 64  ? of_rows<64>(sums, x_fp32, y_fp32)
                          : threads == 128 ? of_rows<128>(sums, x_fp32, y_fp32)
                          : threads == 256 ? of_rows<256>(sums, x_fp32, y_fp32)
                          : threads == 512 ? of_rows<512>(sums, x_fp32, y_fp32)
                                           : join_bwd_kernel<1024, IN_MEMORY, RUNTIME, RUNTIME>;
    cudaError_t e = ensure_smem(reinterpret_cast<const void *>(kernel), smem);
    if (e != cudaSuccess) return e;
    const int units = one ? (T + WARPS - 1) / WARPS : T;
    const bool wanted = g.gamma_post || g.beta_post || g.gate || g.gamma_pre || g.beta_pre;
    const bool joined = wanted && units <= CLUSTER;
    const int ctas = joined ? join_bwd_ctas(T, H) : (units < ctas_sm * num_sms() ? units : ctas_sm * num_sms());
    p.g = g;
    p.joined = joined;
    e = launch_pdl(kernel, dim3(ctas), one ? dim3(32, WARPS) : dim3(threads), smem, s, joined ? ctas : 1, p);
    if (e != cudaSuccess || joined || !wanted) return e;
    return launch_pdl(join_wgrad_kernel, dim3(H / 32), dim3(32, 8), 0, s, 1, static_cast<const float *>(part), ctas, H, o, g);
}

}  // namespace moe
