// ortho.cu -- orthogonalised updates of a batch of matrices by Newton-Schulz products (the update
// of the Muon optimiser), on the 5th-generation tensor cores.
//
//   m <- mu m + g,  u = m or g + mu m (with momentum), else g
//   X = u / |u|_F;  every step:  A = X X^T,  P = b A + c A A,  X <- (a I + P) X;   out = scale X
//
// with A on the smaller side (for matrices with more rows than columns A = X^T X and X <- X
// (a I + P): A and P are symmetric, so the matrices stay as they lie).  A step's polynomial a s + b s^3 +
// c s^5 acts on every singular value s of X.
//
// Launches: the size of u from a sample; the momentum, u as two fp16 numbers at the power of two that the
// sample gives, and its norm (what is left of it, a factor near 1, goes into the first step); one
// persistent launch over all steps' products, a list of tiles claimed in order:
//   gram     A: the tiles on and below the diagonal, each stored twice (the mirror image too)
//   square   a I + P: likewise, with a I + b A added as the tile leaves tensor memory
//   apply    X: the product of a I + P and X, the last step's into `out`
// A matrix's tiles of one product start when those of the one before are stored (a counter a matrix);
// they come earlier in the list, so whoever waits holds nothing that they need.  Other matrices' tiles
// fill the gaps.  (With a launch for each product: 6.9 ms for 16 matrices of 7168 x 2048, 1.42 ms for 24 of
// 2112 x 1088; with this 6.7 and 1.34 ms, before the steps noted below.)
//
// Numbers.  The products take fp16 operands (11 bits; entries of X are at most 1.2 and typically
// (rows columns)^-1/2, so a fixed power of two keeps them normal) with fp32 sums.  What is carried
// from step to step is X in two fp16 numbers, 22 bits: a direction with a small singular value
// is multiplied by a = 3.4 in every step, 485 over five, and a rounding of X with it.  The products take
// the first number; of the second one, a times itself is added (what P would make of it is small).
// The last step does without: its factor of 3.4 on a rounding does not show.  (Rounded to fp16 in every
// step, gradients of rank 16 come out 3e-2 off, in bf16 0.2; so they are 1.5e-3 off.)  A and a I + P are
// rounded to fp16 once each: their error acts through products with X alone, and what X has not is not
// amplified.  In all 0.5e-3 to 2.0e-3 off over random matrices with five default steps, the most for flat
// spectra, and 2.1e-3 to 2.8e-3 with a rank of one; the rounding of the bf16 result is 1.7e-3.  Over few directions
// A's and P's roundings do not average out: up to FEW on the smaller side these are two fp16 numbers each, and where
// one launch does all steps X is too (TWO, SIDE 64 below).
//
// Tiles, roles and waits as in ffn_bwd.cu: clusters of two CTAs, 2-SM MMAs of 256 x 256, 64 deep
// stages of 32 KB a CTA, two accumulators in tensor memory, eight epilogue warps, all waits
// bounded (MOE_ERR_DEVICE_TIMEOUT in the status word).
//
// What bounds it: large matrices the tensor cores (16 of 7168 x 2048: 5.1 ms in the products of one call,
// 1630 TFLOP/s with the diagonal tiles computed whole; 5.8 ms in calls one after the other, under the power
// cap at 1500 MHz, where the library's products are 5% faster) and 0.5 ms of memory before them; 24 of 2112 x
// 1088: 1.0 ms in the products, operands that come late from L2 and tiles of 17 stages; few matrices: 7 us a
// product, in turn.
#include <cuda.h>

#include <cmath>
#include <cstring>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

// Powers of two that X, A and P are stored with: |X|_2 <= 1.2 (default coefficients), room for 16;
// |A| <= 1.5, |P| <= 7, room for 128.  An entry of 2^-26 (X), 2^-23 (A, P) is still normal.
constexpr float SX = 4096.f, SA = 512.f;
constexpr float SLO = 2048.f;             // the second number of X: its own power of two on top

constexpr int TM = 256, TN = 256, BK = 64;   // tiles of a cluster (at most)
constexpr int N_EPI = 8, EPI0 = 4;
constexpr int NT = 32 * (EPI0 + N_EPI);
constexpr int HALF = 8192;                // 64 x 64 fp16
constexpr int STAGE = 4 * HALF;
constexpr int PC = 32;                    // columns of an epilogue's piece
constexpr int PIECES = 4;                 // of a warp's part of a tile, at most
constexpr int PIECE = 32 * PC * 2;
// The ring's stages, and an epilogue warp's buffers: ARRIVE that pieces arrive in, two that leave.  With 5 stages
// two pieces arrive ahead of time, with 4 all of them: long sums gain by the stages (24 of 2112 x 1088: 1.09 and
// 1.05 ms, 8 of 1536 x 4096: 1.02 and 0.98), short ones lose by the pieces (30 of 300 x 700: 315 and 329 us, 20
// of 600 x 1300: 579 and 586).
template <int STAGES>
struct Ring {
    static constexpr int ARRIVE = STAGES == 5 ? 2 : 4;
    static constexpr int SLAB = (ARRIVE + 2) * PIECE;
    static constexpr int BYTES = 1024 + STAGES * STAGE + N_EPI * SLAB;
};
constexpr int LONG_SUMS = 1024;           // the smaller side from which on there are 5 stages

enum { GRAM, SQUARE, APPLY, LAST };

constexpr int TQ = 8;                     // slots that hand claimed tiles to the roles
constexpr int AHEAD = 24;                 // stages left to load of a tile when the next one is claimed
constexpr int CLAIM_WARP = 2, TELL_WARP = 3;
constexpr int DONE = 4;                   // tiles that the epilogue's warps may be apart
constexpr int MAX_STEPS = 32;

struct Args {
    // loads: X of either buffer as the operand of gram and of apply, A, P; K-major operands in boxes
    // of 128 x 64, MN-major ones (gram's X of tall matrices, apply's X of others) of 64 x 64
    CUtensorMap xg[2], xa[2], a, p;
    // the epilogue's pieces of 32 x 32, both ways: A, P, X's first and second numbers, out
    CUtensorMap pa, pp, px[2], pl, po;
    CUtensorMap a2, p2, pa2, pp2;     // second numbers of A and P (TWO), likewise
    int tall, steps, B, m, R, C;  // m: the smaller side
    int side, n_side;             // tiles of A and P: rows and columns that are kept, tiles of a side
    int tn, nM, nN;               // tiles of X: columns that are kept, tiles in each direction
    int sym, app, units;          // tiles of A (or P), of X of a matrix; in all
    int group;                    // matrices that go through the steps together
    int split;                    // parts of gram's sums
    int tma_out;                  // rows of `out` are multiples of 16 bytes
    float c[3 * MAX_STEPS];
    float scale;
    uint16_t *out;                // bf16 [B][R][C]
    const float *rest;            // [B] what the first X still has to be multiplied by
    unsigned *count;              // [B] epilogue warps that are done with a tile (zeroed)
    int *next;                    // the next tile to be claimed (zeroed)
    float *sums;                  // [B][tiles of A][split][2][N_EPI] parts of the sums, PIECES 32 x 32 each
    unsigned *ticket;             // [B][tiles of A][2][N_EPI] how many of them are there (zeroed)
    int *status;
    unsigned long long timeout_ns;
    int inject;
};

__device__ __forceinline__ uint32_t f32x2_to_f16x2(float hi, float lo)
{
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ float f16_lo(uint32_t v)
{
    float f;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(v));
    return f;
}
__device__ __forceinline__ float f16_hi(uint32_t v)
{
    float f;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, h;\n\t}" : "=f"(f) : "r"(v));
    return f;
}

// fp16 operands (formats 0 in bits 7-9 and 10-12), else as idesc_bf16_f32
__device__ __forceinline__ uint32_t idesc_f16_f32(uint32_t M, uint32_t N, bool a_mn, bool b_mn)
{
    return idesc_bf16_f32(M, N, a_mn, b_mn) & ~((7u << 7) | (7u << 10));
}

__device__ __forceinline__ void tma_store_3d(const void *tmap, const void *src, int c0, int c1, int c2)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];"
                 ::"l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(src)) : "memory");
}

__device__ __forceinline__ unsigned ld_acquire(const unsigned *p)
{
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// Whether a phase is complete, without waiting (try_wait may suspend the thread for a while).
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return ok != 0;
}

__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

// The tile's product and step, matrix and place, part of the sums, and the arrivals at the matrix's counter that
// it needs.
struct Tile { int mode, k, b, m0, n0, part; unsigned need; };

__device__ __forceinline__ Tile tile_at(const Args &p, int t)
{
    Tile T;
    const int per = (p.split + 1) * p.sym + p.app, all = p.steps * p.group * per;
    const int g0 = t / all * p.group, n = min(p.group, p.B - g0), step = n * per;
    t -= g0 * p.steps * per;
    T.k = t / step;
    int l = t - T.k * step;
    T.need = 2 * N_EPI * static_cast<unsigned>(T.k * (2 * p.sym + p.app));
    T.part = 0;
    const int gram = n * p.sym * p.split;
    if (l < gram + n * p.sym) {
        if (l < gram) {
            T.mode = GRAM;
            T.part = l % p.split;
            l /= p.split;
        } else {
            T.mode = SQUARE;
            T.need += 2 * N_EPI * p.sym;
            l -= gram;
        }
        T.b = l / p.sym;
        l -= T.b * p.sym;
        T.b += g0;
        int i = static_cast<int>((sqrtf(8.f * l + 1.f) - 1.f) * 0.5f);
        while (i * (i + 1) / 2 > l) --i;
        while ((i + 1) * (i + 2) / 2 <= l) ++i;
        T.m0 = i * p.side;
        T.n0 = (l - i * (i + 1) / 2) * p.side;
        return T;
    }
    l -= gram + n * p.sym;
    T.mode = T.k + 1 < p.steps ? APPLY : LAST;
    T.need += 2 * N_EPI * 2 * p.sym;
    T.b = l / p.app;
    l -= T.b * p.app;
    T.b += g0;
    // the smaller side's tiles innermost: they share a part of X (rows innermost for tall matrices:
    // 695 instead of 672 us for 16 of 7168 x 2048)
    int i, j;
    if (p.nM > p.nN) { i = l / p.nN; j = l - i * p.nN; }
    else { j = l / p.nM; i = l - j * p.nM; }
    T.m0 = i * TM;
    T.n0 = j * p.tn;
    return T;
}

// Products that follow one another in a tile's sums: where A and P are two numbers each (TWO), A A is A A + A A2 + A2 A
// and P X is P X + P2 X.
template <bool TWO>
__device__ __forceinline__ int terms_of(int mode) { return !TWO || mode == GRAM ? 1 : mode == SQUARE ? 3 : 2; }

// TWO: A and P in two fp16 numbers at the same power of two (up to FEW on the smaller side, whose single tile they
// are).  Their roundings do not average out over few directions: with one number, the worst of 64 random matrices of
// 4 x 4096 is 8.2e-3 off, of 16 of 4096 x 33 3.6e-3; so 1.4e-3 at most, what X's rounding leaves (1 of 7168 x 24:
// 117 us with one number, 129 so; 30 of 7168 x 64 304 and 317).  X in two numbers as well: 1e-4, and 165 and 499 us.
template <int STAGES, bool TWO>
__global__ void __launch_bounds__(NT, 1) ortho_gemm_kernel(const __grid_constant__ Args p)
{
    constexpr int ARRIVE = Ring<STAGES>::ARRIVE, SLAB = Ring<STAGES>::SLAB;
    constexpr int TCOLS = 512;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *ring = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char *slabs = ring + STAGES * STAGE;
    __shared__ uint64_t full[STAGES], empty[STAGES], tfull[2], tempty[2], tqf[TQ], tqe[TQ], piece[N_EPI][ARRIVE], want, drain;
    __shared__ uint64_t drained[2], done[DONE];
    __shared__ unsigned told[DONE];
    __shared__ int tq[TQ][6];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_s;
    volatile int *abort_flag = &abort_s;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const uint64_t tmo = p.timeout_ns;
    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 2);
            mbar_init(&drained[b], N_EPI);
        }
        for (int i = 0; i < DONE; ++i) {
            mbar_init(&done[i], N_EPI);
            told[i] = 0;
        }
        for (int q = 0; q < TQ; ++q) {
            mbar_init(&tqf[q], 1);
            mbar_init(&tqe[q], 5);       // both producers, the MMA issuer, both warps that tell
        }
        for (int w = 0; w < N_EPI; ++w)
            for (int b = 0; b < ARRIVE; ++b) mbar_init(&piece[w][b], 1);
        mbar_init(&want, 1);
        mbar_init(&drain, 1);
        abort_s = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(&tmem_slot, TCOLS);
        tmem_relinquish_pair();
    }
    pdl_wait();
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const int gram_kbs = ((p.tall ? p.R : p.C) + BK - 1) / BK, m_kbs = (p.m + BK - 1) / BK;

    // Tiles are claimed from a counter by a warp of the even CTA, the next one when that at hand has AHEAD
    // stages left to load.  It decodes them, waits for what they build on, and hands them to every role of
    // both CTAs through TQ slots (mode -1 ends).
    auto slot_done = [&](int q) {
        if (leader) mbar_arrive(&tqe[q]);
        else mbar_arrive_cluster(mapa_shared(smem_u32(&tqe[q]), 0));
    };
    auto slot_read = [&](int q) { return Tile{tq[q][0], tq[q][1], tq[q][2], tq[q][3], tq[q][4], tq[q][5], 0u}; };
    // the stages of a part of gram's sums
    auto first_stage = [&](int part) { return gram_kbs * part / p.split; };

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0 && !p.inject) {
            uint32_t s = 0, ph = 0, it = 0, qs = 0, qph = 0;
            const uint32_t full0 = mapa_shared(smem_u32(full), 0);
            const int r = static_cast<int>(rank);
            bool good = true;
            while (good) {
                if (!mbar_wait_cluster(&tqf[qs], qph, abort_flag, p.status, tmo)) break;
                const Tile T = slot_read(qs);
                slot_done(qs);
                if (++qs == TQ) { qs = 0; qph ^= 1u; }
                if (T.mode < 0) break;
                fence_proxy_async_global();
                const bool sym = T.mode <= SQUARE;
                const int m = T.m0 + 128 * r, n = T.n0 + (sym ? p.side : p.tn) / 2 * r, kb0 = T.mode == GRAM ? first_stage(T.part) : 0;
                const int each = T.mode == GRAM ? first_stage(T.part + 1) - kb0 : m_kbs, kbs = terms_of<TWO>(T.mode) * each;
                const CUtensorMap *am, *bm;
                bool amn = false, bmn = false;
                if (T.mode == GRAM) { am = bm = &p.xg[T.k & 1]; amn = bmn = p.tall; }
                else if (T.mode == SQUARE) { am = bm = &p.a; }
                else if (p.tall) { am = &p.xa[T.k & 1]; bm = &p.p; }
                else { am = &p.p; bm = &p.xa[T.k & 1]; bmn = true; }
                bool asked = !leader;
                for (int kb = 0; kb < kbs; ++kb, ++it) {
                    if (!asked && kbs - kb <= AHEAD) { mbar_arrive(&want); asked = true; }
                    if (!mbar_wait(&empty[s], ph ^ 1u, abort_flag, p.status, tmo)) { good = false; break; }
                    unsigned char *a = ring + s * STAGE, *b = a + 2 * HALF;
                    const uint32_t fb = full0 + 8u * s;
                    if (leader) mbar_arrive_expect_tx(&full[s], 2u * STAGE);
                    int k = (kb0 + kb) * BK;
                    if (TWO && T.mode != GRAM) {
                        const int term = kb / each;
                        k -= term * each * BK;
                        if (T.mode == SQUARE) {
                            am = term == 2 ? &p.a2 : &p.a;
                            bm = term == 1 ? &p.a2 : &p.a;
                        } else {
                            (p.tall ? bm : am) = term == 1 ? &p.p2 : &p.p;
                        }
                    }
                    if (amn) {
                        tma_load_3d_pair(a, am, fb, m, k, T.b);
                        tma_load_3d_pair(a + HALF, am, fb, m + 64, k, T.b);
                    } else {
                        tma_load_3d_pair(a, am, fb, k, m, T.b);
                    }
                    if (bmn) {
                        tma_load_3d_pair(b, bm, fb, n, k, T.b);
                        tma_load_3d_pair(b + HALF, bm, fb, n + 64, k, T.b);
                    } else {
                        tma_load_3d_pair(b, bm, fb, k, n, T.b);
                    }
                    if (++s == STAGES) { s = 0; ph ^= 1u; }
                }
            }
            // Every copy issued lands before the CTAs can exit: the even CTA's barriers count both
            // CTAs' copies.  After a wait that ran out the odd CTA may have issued stages that the
            // even one has not: it stays as long as the even one waits for a stage at most.
            if (!leader && *abort_flag) {
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 20000000ull) __nanosleep(1000);
            }
            if (leader) {
                const uint32_t n = it < STAGES ? it : STAGES;
                for (uint32_t j = it - n; j < it; ++j) {
                    int dummy = 0;
                    mbar_wait(&full[j % STAGES], (j / STAGES) & 1u, &dummy, nullptr, 20000000ull);
                }
            }
        }
    } else if (warp == 1) {
        // -------------------------------------------------------------- MMA issuer
        if (lane == 0 && leader) {
            const uint32_t ring0 = smem_u32(ring);
            uint32_t s = 0, ph = 0, b = 0, tph = 0, qs = 0, qph = 0;
            bool good = true;
            while (good) {
                if (!mbar_wait(&tqf[qs], qph, abort_flag, p.status, tmo)) break;
                const Tile T = slot_read(qs);
                slot_done(qs);
                if (++qs == TQ) { qs = 0; qph ^= 1u; }
                if (T.mode < 0) break;
                const bool amn = T.mode == GRAM && p.tall, bmn = amn || (T.mode >= APPLY && !p.tall);
                const uint64_t ad0 = smem_desc_sw128(ring0, amn ? HALF : 16, 1024);
                const uint64_t bd0 = smem_desc_sw128(ring0 + 2 * HALF, bmn ? HALF : 16, 1024);
                const uint32_t as = amn ? 128u : 2u, bs = bmn ? 128u : 2u;
                const uint32_t id = idesc_f16_f32(TM, static_cast<uint32_t>(T.mode <= SQUARE ? p.side : p.tn), amn, bmn);
                const int kbs = terms_of<TWO>(T.mode) * (T.mode == GRAM ? first_stage(T.part + 1) - first_stage(T.part) : m_kbs);
                if (!mbar_wait(&tempty[b], tph ^ 1u, abort_flag, p.status, tmo)) break;
                tc_fence_after();
                const uint32_t d = tmem + b * TN;
                for (int kb = 0; kb < kbs; ++kb) {
                    if (!mbar_wait(&full[s], ph, abort_flag, p.status, tmo)) { good = false; break; }
                    tc_fence_after();
                    const uint64_t o = static_cast<uint64_t>(s * (STAGE >> 4));
                    const uint64_t ad = ad0 + o, bd = bd0 + o;
                    tc_mma_bf16_pair(d, ad, bd, id, kb > 0 ? 1u : 0u);
                    tc_mma_bf16_pair(d, ad + as, bd + bs, id, 1u);
                    tc_mma_bf16_pair(d, ad + 2 * as, bd + 2 * bs, id, 1u);
                    tc_mma_bf16_pair(d, ad + 3 * as, bd + 3 * bs, id, 1u);
                    tc_commit_pair_mc(&empty[s], 3);
                    if (++s == STAGES) { s = 0; ph ^= 1u; }
                }
                if (!good) break;
                tc_commit_pair_mc(&tfull[b], 3);
                b ^= 1u;
                if (b == 0) tph ^= 1u;
            }
            tc_commit_pair_mc(&drain, 1);
            int dummy = 0;
            mbar_wait(&drain, 0, &dummy, nullptr, 20000000ull);
        }
    } else if (warp == CLAIM_WARP) {
        // ------------------------------------------------------------------ claims
        if (lane == 0 && leader) {
            uint32_t qs = 0, qph = 0, wph = 1;       // (the first claim waits for nothing)
            bool more = true;
            while (more) {
                if (!mbar_wait(&want, wph, abort_flag, p.status, tmo)) break;
                wph ^= 1u;
                const int t = atomicAdd(p.next, 1);
                more = t < p.units;
                Tile T{-1, 0, 0, 0, 0, 0, 0u};
                if (more) T = tile_at(p, t);
                if (!mbar_wait_cluster(&tqe[qs], qph ^ 1u, abort_flag, p.status, tmo)) break;
                const int vals[6] = {T.mode, T.k, T.b, T.m0, T.n0, T.part};
                const uint32_t other = mapa_shared(smem_u32(tq[qs]), 1);
#pragma unroll
                for (int j = 0; j < 6; ++j) {
                    tq[qs][j] = vals[j];
                    st_shared_cluster(other + 4u * j, vals[j]);
                }
                // The tiles that it builds on are stored.  (Waited for after the slot is written: the arrival in the
                // other CTA then has no store to wait for.)
                const unsigned *n = p.count + T.b;
                if (T.need && ld_acquire(n) < T.need) {
                    const uint64_t t0 = globaltimer_ns();
                    bool good = true;
                    for (int i = 1; good && ld_acquire(n) < T.need; ++i) {
                        if (*abort_flag) good = false;
                        else if (i % 16 == 0 && globaltimer_ns() - t0 > tmo) {
                            *abort_flag = 1;
                            report(p.status, MOE_ERR_DEVICE_TIMEOUT);
                            good = false;
                        }
                    }
                    if (!good) break;
                }
                mbar_arrive(&tqf[qs]);
                mbar_arrive_cluster(mapa_shared(smem_u32(&tqf[qs]), 1));
                if (++qs == TQ) { qs = 0; qph ^= 1u; }
            }
        }
    } else if (warp == TELL_WARP) {
        // -------------------------------------------------------------------- news
        // What the epilogue has to tell other CTAs: that a tile's accumulator and slot are free, and that its
        // results are in memory.  (Arrivals and counts at those scopes hold up a thread for 1 to 3 thousand cycles;
        // with the epilogue's own threads telling, 24 of 2112 x 1088 took 1.12 ms, 1.09 so.)
        if (lane == 0) {
            uint32_t qs = 0, qph = 0, b = 0, bph = 0, i = 0, iph = 0;
            const uint32_t tempty0 = mapa_shared(smem_u32(tempty), 0);
            while (true) {
                if (!mbar_wait_cluster(&tqf[qs], qph, abort_flag, p.status, tmo)) break;
                const Tile T = slot_read(qs);
                if (T.mode < 0) break;
                if (!mbar_wait(&drained[b], bph, abort_flag, p.status, tmo)) break;
                tc_fence_after();
                tc_fence_before();
                mbar_arrive_cluster(tempty0 + 8u * b);
                slot_done(qs);
                if (++qs == TQ) { qs = 0; qph ^= 1u; }
                b ^= 1u;
                if (b == 0) bph ^= 1u;
                if (!mbar_wait(&done[i], iph, abort_flag, p.status, tmo)) break;
                const unsigned n = told[i];
                told[i] = 0;
                if (n) {
                    fence_proxy_async_global();
                    __threadfence();
                    atomicAdd(p.count + T.b, n);
                }
                if (++i == DONE) { i = 0; iph ^= 1u; }
            }
        }
    } else if (warp >= EPI0) {
        // ---------------------------------------------------------------- epilogue
        // What is added to a piece's sums (SQUARE: A; APPLY: X's second number) arrives by TMA, NEXT pieces ahead;
        // the result and what goes beside it (the mirror image; a second number) leave from a buffer each.
        constexpr int EACH = TWO ? 2 : 1, NEXT = ARRIVE / EACH;      // buffers of a piece, pieces
        const int q = warp & 3, half = (warp - EPI0) >> 2;   // lane quarter, half of the columns
        const uint32_t tm0 = tmem + (static_cast<uint32_t>(32 * q) << 16);
        const int r0 = 128 * static_cast<int>(rank) + 32 * q;
        unsigned char *slab = slabs + (warp - EPI0) * SLAB;
        uint64_t *arrived = piece[warp - EPI0];
        uint32_t b = 0, tph = 0, qs = 0, qph = 0, pph = 0;   // pph: phases of the buffers' barriers
        uint32_t flight = 0;                         // buffers that a copy is on its way to (lane 0)
        uint32_t tile = 0;
        int owed = -1;                               // the last tile's place in done, if it is not arrived at (lane 0)
        bool counts = false;                         // whether that tile counts
        // a wait by one lane (every lane then observes the phase itself)
        auto wait_all = [&](uint64_t *bar, uint32_t parity, bool cluster) -> bool {
            bool good = true;
            if (lane == 0)
                good = cluster ? mbar_wait_cluster(bar, parity, abort_flag, p.status, tmo)
                               : mbar_wait(bar, parity, abort_flag, p.status, tmo);
            good = __shfl_sync(kFullMask, good, 0);
            if (good) {
                if (cluster) mbar_try_wait_cluster(bar, parity);
                else mbar_try_wait(bar, parity);
            }
            return good;
        };
        // The warp's part of its last tile is in memory (lane 0, which has committed `newer` groups since).
        auto settle = [&](int newer) {
            if (owed < 0) return;
            if (newer == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
            else if (newer == 1) asm volatile("cp.async.bulk.wait_group 1;" ::: "memory");
            else asm volatile("cp.async.bulk.wait_group 2;" ::: "memory");
            if (counts) atomicAdd(&told[owed], 1u);
            mbar_arrive(&done[owed]);
            owed = -1;
        };
        bool good = true;
        while (good) {
            // (the next tile may wait for the last one; else that is seen to while this one's sums are formed, or
            // after its second piece)
            if (lane == 0 && owed >= 0 && !mbar_test(&tqf[qs], qph)) settle(0);
            if (!wait_all(&tqf[qs], qph, true)) break;
            const Tile T = slot_read(qs);
            __syncwarp();
            if (++qs == TQ) { qs = 0; qph ^= 1u; }
            if (T.mode < 0) {
                if (lane == 0) settle(0);
                break;
            }
            const bool sym = T.mode <= SQUARE, loads = T.mode == SQUARE || T.mode == APPLY;
            const int M = sym ? p.m : p.R, N = sym ? p.m : p.C, width = sym ? p.side : p.tn;
            const int m0 = T.m0 + r0, row = m0 + lane;
            const bool mirror = !TWO && sym && T.m0 != T.n0;
            // X of the step before the last one goes on in its first number alone
            const bool second = (T.mode == APPLY && T.k + 2 < p.steps) || (TWO && sym);
            // this warp's pieces: c0 .. end
            const int pieces = width / PC, c0 = half ? (pieces + 1) / 2 : 0;
            int end = half ? pieces : (pieces + 1) / 2;
            if ((sym && r0 >= p.side) || m0 >= M) end = c0;
            end = max(c0, min(end, (N - T.n0 + PC - 1) / PC));
            // (lane 0; the warp has read what the buffer held)
            auto load = [&](int c) {
                const int i = (c - c0) % NEXT * EACH;
                mbar_arrive_expect_tx(&arrived[i], PIECE);
                tma_load_3d(slab + i * PIECE, T.mode == SQUARE ? &p.pa : &p.pl, &arrived[i], T.n0 + PC * c, m0, T.b);
                flight |= 1u << i;
                if (TWO && sym) {
                    mbar_arrive_expect_tx(&arrived[i + 1], PIECE);
                    tma_load_3d(slab + (i + 1) * PIECE, &p.pa2, &arrived[i + 1], T.n0 + PC * c, m0, T.b);
                    flight |= 2u << i;
                }
            };
            if (lane == 0) {
                if (loads && c0 < end && !p.inject) {
                    fence_proxy_async_global();
                    for (int c = c0; c < min(end, c0 + NEXT); ++c) load(c);
                }
                if (owed >= 0 && !mbar_test(&tfull[b], tph)) settle(0);
            }
            __syncwarp();
            if (!wait_all(&tfull[b], tph, false)) break;
            tc_fence_after();
            const bool direct = T.mode == LAST && !p.tma_out;
            const float rest = T.k == 0 ? p.rest[T.b] : 1.f;
            const float ca = p.c[3 * T.k], cb = p.c[3 * T.k + 1], cc = p.c[3 * T.k + 2] / SA;
            const float gram = SA / (SX * SX) * rest * rest, apply = rest / SA, again = ca / SLO * rest;
            // A part of gram's sums goes to memory; the warp whose part is the last one there adds all of them, in
            // their order.
            const bool parts = T.mode == GRAM && p.split > 1;
            float4 *sums = nullptr;
            bool last = T.mode != LAST;              // whether the tile is done with this one
            constexpr int REGION = PIECES * 32 * 32 / 4;
            if (parts) {
                const int i = T.m0 / p.side, tile = T.b * p.sym + i * (i + 1) / 2 + T.n0 / p.side;
                const int who = static_cast<int>(rank) * N_EPI + warp - EPI0;
                sums = reinterpret_cast<float4 *>(p.sums) + (static_cast<size_t>(tile) * p.split * 2 * N_EPI + who) * REGION + lane;
                float4 *mine = sums + static_cast<size_t>(T.part) * 2 * N_EPI * REGION;
#pragma unroll 1
                for (int c = c0; c < end; ++c) {
                    float v[32];
                    tmem_ld32(tm0 + b * TN + PC * c, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        __stcg(mine + (c - c0) * 256 + i * 32, make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
                }
                __threadfence();
                __syncwarp();
                unsigned *ticket = p.ticket + tile * 2 * N_EPI + who;
                unsigned there = lane == 0 ? atomicAdd(ticket, 1u) + 1 : 0u;
                there = __shfl_sync(kFullMask, there, 0);
                __threadfence();
                if (there == static_cast<unsigned>(p.split)) {
                    if (lane == 0) *ticket = 0;      // (for the next step, which comes after this tile is stored)
                } else {
                    last = false;
                    end = c0;
                }
            }
            const CUtensorMap *sm = T.mode == GRAM ? &p.pa : T.mode == SQUARE ? &p.pp : T.mode == APPLY ? &p.px[(T.k + 1) & 1] : &p.po;
#pragma unroll 1
            for (int c = c0; c < end; ++c) {
                const int col = T.n0 + PC * c;
                // (an address in the 64-byte swizzle goes by the lane's row: 16 bytes i of 64)
                unsigned char *in = slab + (c - c0) % NEXT * EACH * PIECE, *first = slab + ARRIVE * PIECE, *side = first + PIECE;
                auto at = [&](unsigned char *s, int i) -> uint4 * {
                    return reinterpret_cast<uint4 *>(s + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4));
                };
                __syncwarp();
                if (loads) {
                    const int i = (c - c0) % NEXT * EACH;
                    if (!wait_all(&arrived[i], (pph >> i) & 1u, false)) { good = false; break; }
                    pph ^= 1u << i;
                    flight &= ~(1u << i);
                    if (TWO && sym) {
                        if (!wait_all(&arrived[i + 1], (pph >> (i + 1)) & 1u, false)) { good = false; break; }
                        pph ^= 2u << i;
                        flight &= ~(2u << i);
                    }
                }
                float v[32];
                if (!parts) {
                    tmem_ld32(tm0 + b * TN + PC * c, v);
                } else {
                    const float4 *q = sums + (c - c0) * 256;
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0.f;
#pragma unroll 2
                    for (int s = 0; s < p.split; ++s, q += 2 * N_EPI * REGION) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 w = __ldcg(q + i * 32);
                            v[4 * i] += w.x; v[4 * i + 1] += w.y; v[4 * i + 2] += w.z; v[4 * i + 3] += w.w;
                        }
                    }
                }
                if (T.mode == GRAM) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] *= gram;
                } else if (T.mode == SQUARE) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 h = *at(in, i), l = TWO ? *at(in + PIECE, i) : make_uint4(0, 0, 0, 0);
                        const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int j = 8 * i + 2 * k;
                            v[j] = fmaf(cb, TWO ? f16_lo(hw[k]) + f16_lo(lw[k]) : f16_lo(hw[k]), v[j] * cc);
                            v[j + 1] = fmaf(cb, TWO ? f16_hi(hw[k]) + f16_hi(lw[k]) : f16_hi(hw[k]), v[j + 1] * cc);
                        }
                    }
                    if (!mirror) {                   // on the diagonal
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (col + i == row) v[i] = fmaf(ca, SA, v[i]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] *= apply;
                    if (T.mode == APPLY) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint4 l = *at(in, i);
                            const uint32_t lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                v[8 * i + 2 * k] = fmaf(again, f16_lo(lw[k]), v[8 * i + 2 * k]);
                                v[8 * i + 2 * k + 1] = fmaf(again, f16_hi(lw[k]), v[8 * i + 2 * k + 1]);
                            }
                        }
                    }
                }
                // (what the piece before left in its buffers has left them)
                __syncwarp();
                if (lane == 0) {
                    if (loads && c + NEXT < end && !p.inject) load(c + NEXT);
                    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                }
                __syncwarp();
                const float f = p.scale / SX;
                if (direct) {
                    if (row < M) {
                        uint16_t *o = p.out + (static_cast<size_t>(T.b) * M + row) * N + col;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (col + i < N) o[i] = static_cast<uint16_t>(f32x2_to_bf16x2(0.f, v[i] * f));
                    }
                    continue;
                }
                uint32_t w[16];
                if (T.mode == LAST) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) w[i] = f32x2_to_bf16x2(v[2 * i + 1] * f, v[2 * i] * f);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) w[i] = f32x2_to_f16x2(v[2 * i + 1], v[2 * i]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) *at(first, i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                if (second) {
                    const float up = TWO && sym ? 1.f : SLO;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t y[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            y[k] = f32x2_to_f16x2((v[8 * i + 2 * k + 1] - f16_hi(w[4 * i + k])) * up,
                                                  (v[8 * i + 2 * k] - f16_lo(w[4 * i + k])) * up);
                        *at(side, i) = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                }
                if (mirror) {
                    // row j of the mirror image: this lane's number of column j
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        *reinterpret_cast<uint16_t *>(side + j * 64 + (((lane >> 3) ^ ((j >> 1) & 3)) << 4) + (lane & 7) * 2) =
                            static_cast<uint16_t>(j & 1 ? w[j / 2] >> 16 : w[j / 2]);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    tma_store_3d(sm, first, col, m0, T.b);
                    if (second) tma_store_3d(T.mode == APPLY ? &p.pl : T.mode == GRAM ? &p.pa2 : &p.pp2, side, col, m0, T.b);
                    if (mirror) tma_store_3d(sm, side, m0, col, T.b);
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    if (c == c0 + 1) settle(2);
                }
            }
            if (!good) break;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&drained[b]);
                settle(direct || end == c0 ? 0 : 1);
                owed = static_cast<int>(tile % DONE);
                counts = last;
            }
            __syncwarp();
            ++tile;
            b ^= 1u;
            if (b == 0) tph ^= 1u;
        }
        if (lane == 0) {
            // pieces still on their way (after a wait that ran out), and the last stores
            for (int i = 0; i < ARRIVE; ++i) {
                int dummy = 0;
                if (flight >> i & 1u) mbar_wait(&arrived[i], (pph >> i) & 1u, &dummy, nullptr, 20000000ull);
            }
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem, TCOLS);
    }
}

// ------------------------------------------------------------------ momentum, norm, X
constexpr int PT = 256;               // threads
constexpr int MAX_PARTS = 256;        // chunks of a matrix

struct Prepare {
    const void *g;
    int g_fp32;
    float *m;                         // nullable
    float mu;
    int nesterov;
    int R, C, ld;
    long long chunk;                  // elements, a multiple of 8
    int parts;
    float4 *part;                     // [B][parts]: square sums at three scales
    uint16_t *hi, *lo;                // [B][R][ld]
    unsigned *count;                  // [B] and the next tile to be claimed: zeroed here
    unsigned *ticket;                 // `tickets` for each matrix: zeroed here
    int tickets;
    float2 *size;                     // [B] the sample's factor, in two
    float *rest;                      // [B] what X's numbers still have to be multiplied by
};

template <bool VEC>
struct Elements { static constexpr int N = VEC ? 8 : 1; };

template <bool VEC>
__device__ __forceinline__ void load_g(const Prepare &p, size_t i, float (&v)[Elements<VEC>::N])
{
    if constexpr (VEC) {
        if (p.g_fp32) {
            const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p.g) + i);
            const float4 a = q[0], b = q[1];
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
            const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.g) + i);
            v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
            v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z); v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
        }
    } else {
        v[0] = p.g_fp32 ? static_cast<const float *>(p.g)[i] : bf16_lo(static_cast<const uint16_t *>(p.g)[i]);
    }
}

template <bool VEC>
__device__ __forceinline__ void load_m(const float *m, size_t i, float (&v)[Elements<VEC>::N])
{
    if constexpr (VEC) {
        const float4 *q = reinterpret_cast<const float4 *>(m + i);
        const float4 a = q[0], b = q[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        v[0] = m[i];
    }
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}

// Square sums of u, of 2^90 u and of 2^-80 u: one of them holds |u| to fp32's precision whatever the
// size of the entries, subnormal ones too (2^-149 and up: the square of 2^90 u is 2^-118 then).
constexpr float TWO_30 = 1073741824.f, TWO_40 = 1024.f * TWO_30, TWO_60 = TWO_30 * TWO_30;
constexpr float UP = TWO_60 * TWO_30, DOWN = 1.f / (TWO_40 * TWO_40);

// SX x = (u f) times the result, f a power of two, from the square sums.  (One of u below 2^-60 may have
// lost terms to underflow, one above 2^100 to overflow; those at the other scales are then within
// range: that of 2^90 u below 2^120.)  A matrix of zeros stays one; an infinity or a NaN makes it NaN.
__device__ __forceinline__ float x_factor(float s0, float s1, float s2, float &f)
{
    float s = s0;
    f = 1.f;
    if (!(s0 >= 1.f / TWO_60)) { f = UP; s = s1; }
    else if (!(s0 <= TWO_60 * TWO_40)) { f = DOWN; s = s2; }
    return s > 0.f ? (s <= 3.402823466e38f ? SX / sqrtf(s) : s - s) : s;
}

// Sums over the CTA's PT threads (and the largest d) to all of them
__device__ __forceinline__ float4 cta_sums(float a, float b, float c, float d)
{
    __shared__ float4 red[PT / 32];
    a = warp_sum(a); b = warp_sum(b); c = warp_sum(c);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d = fmaxf(d, __shfl_xor_sync(kFullMask, d, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float4(a, b, c, d);
    __syncthreads();
    float4 t = red[0];
    for (int k = 1; k < PT / 32; ++k) t = make_float4(t.x + red[k].x, t.y + red[k].y, t.z + red[k].z, fmaxf(t.w, red[k].w));
    return t;
}

__device__ __forceinline__ void add_squares(float u, float &s0, float &s1, float &s2)
{
    s0 = fmaf(u, u, s0);
    const float a = u * UP, b = u * DOWN;
    s1 = fmaf(a, a, s1);
    s2 = fmaf(b, b, s2);
}

// CTA a matrix: a power of two that brings u to the size of SX X, by SAMPLE of its entries.
constexpr int SAMPLE = 8 * PT;
__global__ void __launch_bounds__(PT) ortho_sample_kernel(const Prepare p)
{
    pdl_wait();
    for (int i = threadIdx.x; i < p.tickets; i += PT) p.ticket[static_cast<size_t>(blockIdx.x) * p.tickets + i] = 0;
    const unsigned long long n = static_cast<unsigned long long>(p.R) * p.C;
    const size_t base = static_cast<size_t>(blockIdx.x) * n;
    float s0 = 0.f, s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < SAMPLE / PT; ++k) {
        // (multiples of the golden ratio, modulo 1: even over the matrix, no row or column preferred)
        const size_t i = base + __umul64hi((k * PT + threadIdx.x + 1) * 0x9E3779B97F4A7C15ull, n);
        float u[1];
        load_g<false>(p, i, u);
        if (p.m) {
            const float m = fmaf(p.mu, p.m[i], u[0]);
            u[0] = p.nesterov ? fmaf(p.mu, m, u[0]) : m;
        }
        add_squares(u[0], s0, s1, s2);
    }
    const float4 t = cta_sums(s0, s1, s2, 0.f);
    if (threadIdx.x != 0) return;
    float f;
    const float inv = x_factor(t.x, t.y, t.z, f) * sqrtf(static_cast<float>(SAMPLE) / static_cast<float>(n));   // SX / |u f|
    int e = 0, g = 0;
    if (inv > 0.f && inv <= 3.402823466e38f) {
        frexpf(inv, &e);
        frexpf(f, &g);
        e += g - 2;
    }
    e = max(-200, min(200, e));
    p.size[blockIdx.x] = make_float2(pow2f(e / 2), pow2f(e - e / 2));
    p.count[blockIdx.x] = 0;
    if (blockIdx.x == 0) p.count[gridDim.x] = 0;
}

// Where element i of matrix `b` lies in X's arrays (their rows are as long as the matrix's where it is VEC).
template <bool VEC>
__device__ __forceinline__ size_t x_at(const Prepare &p, int b, size_t base, long long i)
{
    if constexpr (VEC) return base + i;
    const long long r = i / p.C;
    return (static_cast<size_t>(b) * p.R + r) * p.ld + (i - r * p.C);
}

// N numbers from `at` on as two fp16 numbers each
template <int N>
__device__ __forceinline__ void store_numbers(const Prepare &p, size_t at, const float (&v)[N])
{
    if constexpr (N == 8) {
        uint32_t h[4], l[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            h[k] = f32x2_to_f16x2(v[2 * k + 1], v[2 * k]);
            l[k] = f32x2_to_f16x2((v[2 * k + 1] - f16_hi(h[k])) * SLO, (v[2 * k] - f16_lo(h[k])) * SLO);
        }
        *reinterpret_cast<uint4 *>(p.hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4 *>(p.lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
    } else {
        const uint32_t h = f32x2_to_f16x2(0.f, v[0]);
        p.hi[at] = static_cast<uint16_t>(h);
        p.lo[at] = static_cast<uint16_t>(f32x2_to_f16x2(0.f, (v[0] - f16_lo(h)) * SLO));
    }
}

// VEC: R C and C are multiples of 8.  CTA (part, matrix): the momentum, u times the sample's factor, and the
// chunk's square sums.
template <bool VEC>
__global__ void __launch_bounds__(PT) ortho_momentum_kernel(const Prepare p)
{
    constexpr int N = Elements<VEC>::N;
    pdl_wait();
    const long long n = static_cast<long long>(p.R) * p.C;
    const size_t base = static_cast<size_t>(blockIdx.y) * n;
    const long long lo = blockIdx.x * p.chunk, hi = min(n, lo + p.chunk);
    const float2 size = p.size[blockIdx.y];
    float s0 = 0.f, s1 = 0.f, s2 = 0.f, most = 0.f;
    for (long long i = lo + threadIdx.x * N; i < hi; i += PT * N) {
        float u[N];
        load_g<VEC>(p, base + i, u);
        if (p.m) {
            float m[N];
            load_m<VEC>(p.m, base + i, m);
#pragma unroll
            for (int k = 0; k < N; ++k) {
                m[k] = fmaf(p.mu, m[k], u[k]);
                u[k] = p.nesterov ? fmaf(p.mu, m[k], u[k]) : m[k];
            }
            if constexpr (VEC) {
                float4 *q = reinterpret_cast<float4 *>(p.m + base + i);
                q[0] = make_float4(m[0], m[1], m[2], m[3]);
                q[1] = make_float4(m[4], m[5], m[6], m[7]);
            } else {
                p.m[base + i] = m[0];
            }
        }
        float v[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            add_squares(u[k], s0, s1, s2);
            v[k] = u[k] * size.x * size.y;
            most = fmaxf(most, fabsf(v[k]));
        }
        store_numbers(p, x_at<VEC>(p, blockIdx.y, base, i), v);
    }
    const float4 t = cta_sums(s0, s1, s2, most);
    if (threadIdx.x == 0) p.part[static_cast<size_t>(blockIdx.y) * p.parts + blockIdx.x] = t;
}

// CTAs of a matrix: the factor that is left.  Where the sample was so far off that X's numbers have left
// fp16's range or come near its end, they are made again.
template <bool VEC>
__global__ void __launch_bounds__(PT) ortho_scale_kernel(const Prepare p)
{
    constexpr int N = Elements<VEC>::N;
    pdl_wait();
    float s0 = 0.f, s1 = 0.f, s2 = 0.f, most = 0.f;
    for (int k = threadIdx.x; k < p.parts; k += PT) {
        const float4 v = p.part[static_cast<size_t>(blockIdx.y) * p.parts + k];
        s0 += v.x; s1 += v.y; s2 += v.z;
        most = fmaxf(most, v.w);
    }
    const float4 t = cta_sums(s0, s1, s2, most);
    const float2 size = p.size[blockIdx.y];
    float f;
    const float inv = x_factor(t.x, t.y, t.z, f), rest = inv * (f / size.x) / size.y;
    // (a matrix of zeros: 0; one that holds a NaN or an infinity: NaN)
    const bool far = inv > 0.f && !(rest >= 1.f / 16 && rest <= 16.f && t.w <= 60000.f);
    if (blockIdx.x == 0 && threadIdx.x == 0) p.rest[blockIdx.y] = far ? 1.f : (inv > 0.f ? rest : inv);
    if (!far) return;
    const long long n = static_cast<long long>(p.R) * p.C;
    const size_t base = static_cast<size_t>(blockIdx.y) * n;
    const long long step = static_cast<long long>(gridDim.x) * PT * N;
    for (long long i = (static_cast<long long>(blockIdx.x) * PT + threadIdx.x) * N; i < n; i += step) {
        float u[N];
        if (!p.m || p.nesterov) load_g<VEC>(p, base + i, u);
        if (p.m) {
            float m[N];
            load_m<VEC>(p.m, base + i, m);
#pragma unroll
            for (int k = 0; k < N; ++k) u[k] = p.nesterov ? fmaf(p.mu, m[k], u[k]) : m[k];
        }
#pragma unroll
        for (int k = 0; k < N; ++k) u[k] = u[k] * f * inv;
        store_numbers(p, x_at<VEC>(p, blockIdx.y, base, i), u);
    }
}

// ---------------------------------------------------------------------- small matrices
// Matrices of up to 128 on the smaller side and eight times 384 on the larger: a cluster of CL CTAs a matrix, each
// with up to 384 columns of X, all steps in one launch.  X as the products' operand (fp16), A and P lie
// in shared memory, X itself (fp32) in tensor memory, times a SA: the product with P is added to it there.
// With several CTAs, each takes the sums of a part of A's rows from all of them and gives it to all: two
// barriers of the cluster a step.  (16 matrices of 256 x 128: 100 us with the launches for large ones, 27 us
// with this; one of 128 x 1000: 116 and 43 us; 76 of 128 x 1536: 303 and 174 us.)
//
// SIDE 64: up to FEW on the smaller side, every operand is two fp16 numbers, hi + lo (22 bits; lo at hi's power
// of two, where its last bit is 2^-24 / SX or less), and a product is hi hi + hi lo + lo hi.  With one number
// the roundings of X, A and P do not average out over few directions: of 64 random matrices of 2 x 2 the worst
// comes out 9.8e-3 off, of 4 x 3000 7.3e-3, of 32 x 3000 3.5e-3; so 1e-5, and up to 3e-4 with ranks far below the sides
// (700 of 24 x 17: 74 us with one number, 89 so; 16 of 64 x 256 24 and 34 us; 8 of 64 x 3000, a cluster of
// eight each, 55 and 53).  A chunk of an operand is 64 rows then: as the first operand of a product of 128 rows
// it reads on into what lies behind it, for rows of the sums that nothing reads.
constexpr int SM_SIDE = 128, SM_LONG = 384, SM_CTAS = 8, FEW = 64;
constexpr int ST = 512;               // threads: four warps for each 32 rows, which share the columns
constexpr int PITCH = 132;            // of 128 rows of a tall matrix on their way, in fp32

// Shared memory from its first multiple of 1024 on: X (SIDE 64: its second numbers), A and P (likewise), this CTA's
// sums of A where there are several CTAs, fp32 [SIDE][SIDE], and what a chunk of 64 rows is read on into.
template <int SIDE>
struct Places {
    static constexpr int NUMBERS = SIDE == 64 ? 2 : 1;
    static constexpr int CHUNK = SIDE * 128;             // SIDE rows x 64 fp16
    static constexpr int SQUARE_OF = SIDE / 64 * CHUNK;  // one number of A or P
    static constexpr int x(int np) { return np / 64 * CHUNK; }
    static constexpr size_t bytes(int np, int cl)
    {
        const size_t all = NUMBERS * (x(np) + 2 * SQUARE_OF) + (cl > 1 ? SIDE * SIDE * 4 : 0) + (SIDE == 64 ? CHUNK : 0);
        const size_t turn = SIDE == 64 ? 128 * PITCH * 4 : 0;    // (within the rest for 128)
        return 1024 + (all > turn ? all : turn);
    }
};

struct Small {
    Prepare q;                        // of it: the matrices and the momentum
    int tall, m, n, np;               // sides of X (m <= n), columns of a CTA (a multiple of 64)
    int steps;
    float c[3 * MAX_STEPS];
    float scale;
    uint16_t *out;
    int *status;
    unsigned long long timeout_ns;
    int inject;
};

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&v)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};"
        ::"f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
          "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]),
          "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]),
          "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// u at element i (8 of them from i on with VEC), after the momentum's update
template <bool VEC>
__device__ __forceinline__ void small_load(const Prepare &q, size_t i, float (&u)[Elements<VEC>::N])
{
    constexpr int N = Elements<VEC>::N;
    load_g<VEC>(q, i, u);
    if (!q.m) return;
    float m[N];
    load_m<VEC>(q.m, i, m);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        m[k] = fmaf(q.mu, m[k], u[k]);
        u[k] = q.nesterov ? fmaf(q.mu, m[k], u[k]) : m[k];
    }
    if constexpr (VEC) {
        float4 *o = reinterpret_cast<float4 *>(q.m + i);
        o[0] = make_float4(m[0], m[1], m[2], m[3]);
        o[1] = make_float4(m[4], m[5], m[6], m[7]);
    } else {
        q.m[i] = m[0];
    }
}

__device__ __forceinline__ float4 ld_cluster(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// Two numbers of fp16, of each of a pair
__device__ __forceinline__ void two_numbers(float v1, float v0, uint32_t &hi, uint32_t &lo)
{
    hi = f32x2_to_f16x2(v1, v0);
    lo = f32x2_to_f16x2(v1 - f16_hi(hi), v0 - f16_lo(hi));
}

template <bool VEC, int CL, int SIDE>
__global__ void __launch_bounds__(ST, 1) ortho_small_kernel(const __grid_constant__ Small p)
{
    constexpr uint32_t TCOLS = 512, TD = SM_LONG;    // X, then the sums of A and A A
    constexpr bool TWO = SIDE == 64;
    constexpr int CHUNK = Places<SIDE>::CHUNK, ALO = Places<SIDE>::SQUARE_OF, TERMS = TWO ? 3 : 1;
    const int XLO = Places<SIDE>::x(p.np);
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sx = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char *sa = sx + Places<SIDE>::NUMBERS * XLO, *sp = sa + Places<SIDE>::NUMBERS * ALO;
    unsigned char *part = sp + Places<SIDE>::NUMBERS * ALO;      // CL > 1: this CTA's sums of A
    __shared__ uint64_t done;
    __shared__ uint32_t tmem_slot;
    __shared__ float red[3][ST / 32];
    __shared__ __align__(16) float total[4];
    __shared__ int abort_s;
    volatile int *abort_flag = &abort_s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        mbar_init(&done, 1);
        abort_s = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&tmem_slot, TCOLS);
        tmem_relinquish();
    }
    pdl_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    // this thread's row, and its columns: 32 from `col` on of every 128
    const int q = warp & 3, col = 32 * (warp >> 2), row = 32 * q + lane;
    const bool rows = 32 * q < SIDE, square = rows && col < SIDE;    // whether it has numbers of X, of A and P
    const uint32_t tm0 = tmem + (static_cast<uint32_t>(32 * q) << 16);
    const int rank = CL > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int x0 = rank * p.np, own = max(0, min(p.np, p.n - x0));   // this CTA's columns of X
    const size_t base = static_cast<size_t>(blockIdx.x / CL) * p.m * p.n;
    // 32 numbers of the thread's row, from column c of an operand of 64-column chunks
    auto put = [&](unsigned char *s, int c, const uint32_t (&w)[16]) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4 *>(s + (c >> 6) * CHUNK + row * 128 + ((((c & 63) / 8 + i) ^ (row & 7)) << 4)) =
                make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    };

    // u to tensor memory, and its square sums (see UP).  A tall matrix passes through
    // shared memory, 128 of its rows (columns of X) at a time: [column][128 + 4 rows] of fp32.
    float s0 = 0.f, s1 = 0.f, s2 = 0.f;
    float *turn = reinterpret_cast<float *>(sx);
    constexpr int N = Elements<VEC>::N;
    for (int c0 = 0; c0 < p.np; c0 += 128) {
        if (p.tall) {
            __syncthreads();
            const int per = p.m / N;
            for (int i = tid; i < 128 * per; i += ST) {
                const int r = i / per, k = (i - r * per) * N;
                if (c0 + r >= own) break;
                float u[N];
                small_load<VEC>(p.q, base + static_cast<size_t>(x0 + c0 + r) * p.m + k, u);
#pragma unroll
                for (int j = 0; j < N; ++j) turn[r * PITCH + k + j] = u[j];
            }
            __syncthreads();
        }
        const int c = c0 + col;
        if (c >= p.np) continue;
        float v[32];
        if (p.tall) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = row < p.m && c + i < own ? turn[(col + i) * PITCH + row] : 0.f;
        } else {
#pragma unroll
            for (int i = 0; i < 32 / N; ++i) {
                float u[N];
#pragma unroll
                for (int k = 0; k < N; ++k) u[k] = 0.f;
                if (row < p.m && c + N * i < own) small_load<VEC>(p.q, base + static_cast<size_t>(row) * p.n + x0 + c + N * i, u);
#pragma unroll
                for (int k = 0; k < N; ++k) v[N * i + k] = u[k];
            }
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) add_squares(v[i], s0, s1, s2);
        __syncwarp();
        tmem_st32(tm0 + c, v);
    }
    tmem_st_wait();
    s0 = warp_sum(s0); s1 = warp_sum(s1); s2 = warp_sum(s2);
    if (lane == 0) { red[0][warp] = s0; red[1][warp] = s1; red[2][warp] = s2; }
    __syncthreads();
    s0 = s1 = s2 = 0.f;
    for (int k = 0; k < ST / 32; ++k) { s0 += red[0][k]; s1 += red[1][k]; s2 += red[2][k]; }
    if (CL > 1) {
        if (tid == 0) { total[0] = s0; total[1] = s1; total[2] = s2; total[3] = 0.f; }
        __syncwarp();
        cluster_sync();
        s0 = s1 = s2 = 0.f;
        for (int r = 0; r < CL; ++r) {
            const float4 t = ld_cluster(mapa_shared(smem_u32(total), r));
            s0 += t.x; s1 += t.y; s2 += t.z;
        }
    }
    float f;
    const float inv = x_factor(s0, s1, s2, f);

    // (Several CTAs: every one goes through all steps, whatever it waited for in vain, so that they meet at
    // the barriers.)
    uint32_t ph = 0;
    bool good = true;
    // every MMA since the last call is done: its sums may be read, its operands overwritten
    auto finished = [&]() {
        good = mbar_wait(&done, ph, abort_flag, p.status, p.timeout_ns) && good;
        ph ^= 1u;
        __syncwarp();
        tc_fence_after();
    };
    // operands and sums of all threads are in place for the next MMAs
    auto in_place = [&]() {
        tmem_st_wait();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_before();
        good = __syncthreads_and(good) != 0;
        tc_fence_after();
    };
    const bool issuer = tid == 0 && !p.inject;
    const uint32_t ux = smem_u32(sx), ua = smem_u32(sa), up = smem_u32(sp);
    for (int k = 0; k <= p.steps; ++k) {
        // X of this step: the operand, and a SA X in tensor memory; after the last one, the result
        const bool last = k == p.steps;
        const float take = k == 0 ? f : 1.f / SA, mul = k == 0 ? inv : 1.f, keep = last ? 0.f : p.c[3 * k] * SA;
        for (int c = rows ? col : p.np; c < p.np; c += 128) {
            float v[32];
            __syncwarp();
            tmem_ld32(tm0 + c, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = v[i] * take * mul;
            if (!last) {
                uint32_t w[16], l[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) two_numbers(v[2 * i + 1], v[2 * i], w[i], l[i]);
                put(sx, c, w);
                if (TWO) put(sx + XLO, c, l);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] *= keep;
                tmem_st32(tm0 + c, v);
                continue;
            }
            const float o = p.scale / SX;
            if (p.tall) {            // [column][128 + 8 rows] of bf16 in shared memory
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    reinterpret_cast<uint16_t *>(sx)[(c + i) * 136 + row] = static_cast<uint16_t>(f32x2_to_bf16x2(0.f, v[i] * o));
                continue;
            }
            if (row >= p.m) continue;
            uint16_t *to = p.out + base + static_cast<size_t>(row) * p.n + x0 + c;
            if constexpr (VEC) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c + 8 * i < own)
                        reinterpret_cast<uint4 *>(to)[i] =
                            make_uint4(f32x2_to_bf16x2(v[8 * i + 1] * o, v[8 * i] * o), f32x2_to_bf16x2(v[8 * i + 3] * o, v[8 * i + 2] * o),
                                       f32x2_to_bf16x2(v[8 * i + 5] * o, v[8 * i + 4] * o), f32x2_to_bf16x2(v[8 * i + 7] * o, v[8 * i + 6] * o));
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (c + i < own) to[i] = static_cast<uint16_t>(f32x2_to_bf16x2(0.f, v[i] * o));
            }
        }
        if (last && p.tall) {
            __syncthreads();
            const int per = p.m / N;
            const uint16_t *from = reinterpret_cast<const uint16_t *>(sx);
            for (int i = tid; i < own * per; i += ST) {
                const int r = i / per, k = (i - r * per) * N;
                uint16_t *to = p.out + base + static_cast<size_t>(x0 + r) * p.m + k;
                if constexpr (VEC) *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(from + r * 136 + k);
                else *to = from[r * 136 + k];
            }
        }
        if (last) break;
        in_place();
        if (CL == 1 && !good) break;
        if (issuer && good) {                        // A = X X^T
            const uint32_t id = idesc_f16_f32(128, SIDE, false, false);
            for (int i = 0; i < p.np / 16; ++i) {
                const uint32_t at = ux + (i >> 2) * CHUNK + (i & 3) * 32;
                const uint64_t d = smem_desc_sw128(at, 16, 1024);
                tc_mma_bf16(tmem + TD, d, d, id, i > 0 ? 1u : 0u);
                if (TWO) {
                    const uint64_t l = smem_desc_sw128(at + XLO, 16, 1024);
                    tc_mma_bf16(tmem + TD, d, l, id, 1u);
                    tc_mma_bf16(tmem + TD, l, d, id, 1u);
                }
            }
            tc_commit(&done);
        }
        finished();
        constexpr float S = SA / (SX * SX);
        uint32_t a[16], al[16];                      // A, of the thread's row and columns
        float v[32];
        if (square) tmem_ld32(tm0 + TD + col, v);
        if (CL == 1) {
            if (square) {
#pragma unroll
                for (int i = 0; i < 16; ++i) two_numbers(v[2 * i + 1] * S, v[2 * i] * S, a[i], al[i]);
                put(sa, col, a);
                if (TWO) put(sa + ALO, col, al);
            }
        } else {
            // vector j of 4 columns of a row lies at j ^ row (modulo the vectors)
            constexpr int V = SIDE / 4;
            if (square)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<float4 *>(part + row * (SIDE * 4) + (((col / 4 + i) ^ (row & (V - 1))) << 4)) =
                        make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            __syncwarp();
            cluster_sync();
            constexpr int MINE = SIDE / CL * V;      // vectors of this CTA's rows
#pragma unroll
            for (int j = 0; j < (MINE + ST - 1) / ST; ++j) {
                const int e = j * ST + tid, r = rank * (SIDE / CL) + e / V, n = e % V;
                if (MINE % ST && e >= MINE) break;
                const uint32_t at = smem_u32(part) + r * (SIDE * 4) + ((n ^ (r & (V - 1))) << 4);
                float4 t[CL];
#pragma unroll
                for (int k2 = 0; k2 < CL; ++k2) t[k2] = ld_cluster(mapa_shared(at, k2));
#pragma unroll
                for (int k2 = 1; k2 < CL; ++k2) t[0] = make_float4(t[0].x + t[k2].x, t[0].y + t[k2].y, t[0].z + t[k2].z, t[0].w + t[k2].w);
                uint32_t h0, h1, l0, l1;
                two_numbers(t[0].y * S, t[0].x * S, h0, l0);
                two_numbers(t[0].w * S, t[0].z * S, h1, l1);
                const uint32_t to = ua + (n >> 4) * CHUNK + r * 128 + ((((n & 15) >> 1) ^ (r & 7)) << 4) + (n & 1) * 8;
#pragma unroll
                for (int k2 = 0; k2 < CL; ++k2) {
                    const uint32_t there = mapa_shared(to, k2);
                    asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(there), "r"(h0), "r"(h1) : "memory");
                    if (TWO) asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(there + ALO), "r"(l0), "r"(l1) : "memory");
                }
            }
            asm volatile("fence.proxy.async;" ::: "memory");
            __syncwarp();
            cluster_sync();
            auto get = [&](const unsigned char *s, uint32_t (&w)[16]) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(s + (col >> 6) * CHUNK + row * 128 + ((((col & 63) / 8 + i) ^ (row & 7)) << 4));
                    w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
                }
            };
            if (square) {
                get(sa, a);
                if (TWO) get(sa + ALO, al);
            }
        }
        in_place();
        if (CL == 1 && !good) break;
        if (issuer && good) {                        // A A
            const uint32_t id = idesc_f16_f32(128, SIDE, false, false);
#pragma unroll
            for (int i = 0; i < SIDE / 16; ++i) {
                const uint32_t at = ua + (i >> 2) * CHUNK + (i & 3) * 32;
                const uint64_t d = smem_desc_sw128(at, 16, 1024);
                tc_mma_bf16(tmem + TD, d, d, id, i > 0 ? 1u : 0u);
                if (TWO) {
                    const uint64_t l = smem_desc_sw128(at + ALO, 16, 1024);
                    tc_mma_bf16(tmem + TD, d, l, id, 1u);
                    tc_mma_bf16(tmem + TD, l, d, id, 1u);
                }
            }
            tc_commit(&done);
        }
        finished();
        const float cb = p.c[3 * k + 1], cc = p.c[3 * k + 2] / SA;
        if (square) {
            tmem_ld32(tm0 + TD + col, v);
            uint32_t w[16], l[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float a1 = f16_hi(a[i]), a0 = f16_lo(a[i]);
                if (TWO) { a1 += f16_hi(al[i]); a0 += f16_lo(al[i]); }
                two_numbers(fmaf(cb, a1, v[2 * i + 1] * cc), fmaf(cb, a0, v[2 * i] * cc), w[i], l[i]);
            }
            put(sp, col, w);
            if (TWO) put(sp + ALO, col, l);
        }
        in_place();
        if (CL == 1 && !good) break;
        if (issuer && good) {                        // a X + P X
            for (int n0 = 0; n0 < p.np; n0 += 256) {
                const int n = min(256, p.np - n0);
                const uint32_t id = idesc_f16_f32(128, static_cast<uint32_t>(n), false, true);
#pragma unroll
                for (int t = 0; t < TERMS; ++t)      // P X, P lo X, P X lo
#pragma unroll
                    for (int i = 0; i < SIDE / 16; ++i)
                        tc_mma_bf16(tmem + n0, smem_desc_sw128(up + (t == 1 ? ALO : 0) + (i >> 2) * CHUNK + (i & 3) * 32, 16, 1024),
                                    smem_desc_sw128(ux + (t == 2 ? XLO : 0) + (n0 >> 6) * CHUNK + i * 2048, CHUNK, 1024), id, 1u);
            }
            tc_commit(&done);
        }
        finished();
    }
    // (after a wait that ran out, MMAs still on their way)
    if (!good && issuer) {
        int dummy = 0;
        mbar_wait(&done, ph ^ 1u, &dummy, nullptr, 20000000ull);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, TCOLS);
    }
}

// ------------------------------------------------------------------------ host side
using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion,
                                   CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
{
    static const EncodeTiledFn fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeTiledFn>(ptr);
        return static_cast<EncodeTiledFn>(nullptr);
    }();
    return fn;
}

// fp16 [B][rows][cols] in rows of ld elements (a multiple of 8), boxes of box_rows x box_cols: 64
// columns in the 128-byte swizzle, 32 in the 64-byte one.  What is outside reads as 0.
bool encode(CUtensorMap *m, const void *base, int B, int rows, int cols, int ld, int box_rows, int box_cols)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(B)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(ld) * 2 * rows};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t al256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }
int up8(int n) { return (n + 7) & ~7; }

template <bool VEC, int SIDE>
auto small_kernel(int cl) -> void (*)(const Small)
{
    return cl == 1   ? ortho_small_kernel<VEC, 1, SIDE>
           : cl == 2 ? ortho_small_kernel<VEC, 2, SIDE>
           : cl == 4 ? ortho_small_kernel<VEC, 4, SIDE> : ortho_small_kernel<VEC, 8, SIDE>;
}

bool is_small(int m, int n) { return m <= SM_SIDE && n <= SM_CTAS * SM_LONG; }
int tiles_of(int n, int t) { return (n + t - 1) / t; }

// Tiles of a call's products (Args); B > 0.
struct Plan { int side, n_side, sym, tn, nM, nN, app, group, split, two; };
Plan plan_of(int B, int R, int C)
{
    Plan a{};
    const int most = num_sms() / 2;      // clusters
    const int m = R < C ? R : C, n = R < C ? C : R;
    a.two = m <= FEW && !is_small(m, n);
    // Sides of the symmetric results' tiles and widths of X's: multiples of 32 up to 256, those whose tiles
    // take least.  What a tile takes beside its columns is worth about 200 of them (24 of 2112 x 1088, widths
    // of X's tiles 224, 192, 128: 1.13, 1.18, 1.40 ms), and 224 columns take as long as 256 (24 of 1088 x 2112:
    // 1.17 ms with ten tiles of 224, 1.12 with nine of 256).  The tiles of few matrices follow each other in
    // rounds of the clusters.
    const auto pick = [&](int n, auto count) {
        int best = 0;
        double least = 0;
        for (int k = tiles_of(n, 256); k <= 4 * tiles_of(n, 256); ++k) {
            const int t = (tiles_of(n, k) + 31) / 32 * 32;
            const long long all = static_cast<long long>(B) * count(tiles_of(n, t));
            const double rounds = B < 4 || all < most ? static_cast<double>((all + most - 1) / most) : static_cast<double>(all) / most;
            const double cost = rounds * ((t > 192 ? 256 : t) + 200);
            if (!best || cost < least) { least = cost; best = t; }
        }
        return best;
    };
    const auto triangle = [](long long k) { return k * (k + 1) / 2; };
    a.split = 1;
    if (B * triangle(tiles_of(m, 256)) >= most || is_small(m, n)) {
        a.side = a.two ? tiles_of(m, 32) * 32 : pick(m, triangle);
    } else {
        // A round holds all of A's tiles, and gram's sums may go in parts.  Microseconds: a stage about 0.3 whatever
        // the width (latency: four are on their way), a piece of 32 columns 0.7, a part 2 in all and 0.4 for a
        // piece.  (1 of 7168 x 100: 391 us in whole sums, 180 in parts; 6 of 7168 x 200: 422 and 264; 1 of 7168 x
        // 512: 313 and 211; 1 of 7168 x 2048: 562 and 527.)
        const int gram = tiles_of(n, BK), square = (a.two ? 3 : 1) * tiles_of(m, BK);
        double least = 0;
        for (int k = tiles_of(m, 256); k <= (a.two ? 1 : 4 * tiles_of(m, 256)); ++k) {
            const int t = (tiles_of(m, k) + 31) / 32 * 32, pieces = (t / PC + 1) / 2;
            const long long all = B * triangle(tiles_of(m, t));
            if (all > most) break;
            int split = static_cast<int>(sqrt(0.75 * gram / pieces));
            if (split > most / all) split = static_cast<int>(most / all);
            if (split > gram / 4) split = gram / 4;
            for (int i = 0; i < 2; ++i, split = 1) {
                const int parts = split < 2 ? 1 : split;
                const double us = (tiles_of(gram, parts) + square) * (0.26 + 0.0003 * t) + 1.4 * pieces +
                                  (parts > 1 ? 2 + 0.4 * parts * pieces : 0);
                if (!least || us < least) { least = us; a.side = t; a.split = parts; }
            }
        }
    }
    a.n_side = tiles_of(m, a.side);
    a.sym = a.n_side * (a.n_side + 1) / 2;
    a.nM = tiles_of(R, TM);
    a.tn = pick(C, [&](long long k) { return k * a.nM; });
    a.nN = tiles_of(C, a.tn);
    a.app = a.nM * a.nN;
    // Matrices go through all steps in groups: what a group's products hand on is more often still in L2 (16 of
    // 7168 x 2048, without momentum: 5.88 ms in one group, 5.67 in two or in four; 1% in calls one after the
    // other, under the power cap).  A group's tiles of A go around the clusters 2.5 times, or the next product
    // waits (24 of 2112 x 1088: 1.13 ms in one or two groups, 1.22 in three, 1.32 in four; 48: 2.33 ms in
    // one, 2.25 in three); a rest of few matrices would, too.
    const int least = static_cast<int>((5ll * most / 2 + a.sym - 1) / a.sym);
    a.group = B < 2 * least ? B : (B + B / least - 1) / (B / least);
    while (B % a.group && B % a.group < least) ++a.group;
    return a;
}

struct Layout {
    int m, ld, ldm, parts;
    long long chunk;
    size_t count, size, rest, part, hi[2], lo, A, P, A2, P2, ticket, sums, bytes;
};
Layout layout(int B, int R, int C, const Plan &t)
{
    Layout L{};
    L.m = R < C ? R : C;
    L.ld = up8(C);
    L.ldm = up8(L.m);
    const long long n = static_cast<long long>(R) * C;
    // chunks of 16384 elements or more, MAX_PARTS at most
    long long chunk = (n + MAX_PARTS - 1) / MAX_PARTS;
    if (chunk < 16384) chunk = 16384;
    L.chunk = (chunk + 7) / 8 * 8;
    L.parts = static_cast<int>((n + L.chunk - 1) / L.chunk);
    size_t o = 0;
    auto take = [&](size_t b) { const size_t at = o; o += al256(b); return at; };
    const size_t x = static_cast<size_t>(B) * R * L.ld * 2, a = static_cast<size_t>(B) * L.m * L.ldm * 2;
    L.count = take((static_cast<size_t>(B) + 1) * sizeof(unsigned));
    L.size = take(static_cast<size_t>(B) * sizeof(float2));
    L.rest = take(static_cast<size_t>(B) * sizeof(float));
    L.part = take(static_cast<size_t>(B) * L.parts * sizeof(float4));
    L.hi[0] = take(x);
    L.hi[1] = take(x);
    L.lo = take(x);
    L.A = take(a);
    L.P = take(a);
    L.A2 = take(t.two ? a : 0);
    L.P2 = take(t.two ? a : 0);
    const size_t each = t.split > 1 ? static_cast<size_t>(B) * t.sym * 2 * N_EPI : 0;
    L.ticket = take(each * sizeof(unsigned));
    L.sums = take(each * t.split * PIECES * 32 * 32 * sizeof(float));
    L.bytes = o;
    return L;
}

}  // namespace

// (small matrices need none: ortho_small_kernel)
size_t ortho_bytes(int B, int R, int C)
{
    return B > 0 && !is_small(R < C ? R : C, R < C ? C : R) ? layout(B, R, C, plan_of(B, R, C)).bytes : 0;
}

cudaError_t launch_ortho(const Ortho &f, void *scratch, int *status, unsigned long long timeout_ns, int inject,
                         cudaStream_t s)
{
    const int B = f.B, R = f.R, C = f.C;
    const Plan t = plan_of(B, R, C);
    const Layout L = layout(B, R, C, t);
    unsigned char *w = static_cast<unsigned char *>(scratch);
    Prepare q{f.g, f.g_fp32, f.momentum, f.mu, f.nesterov, R, C, L.ld, L.chunk, L.parts,
              reinterpret_cast<float4 *>(w + L.part), reinterpret_cast<uint16_t *>(w + L.hi[0]),
              reinterpret_cast<uint16_t *>(w + L.lo), reinterpret_cast<unsigned *>(w + L.count),
              reinterpret_cast<unsigned *>(w + L.ticket), t.split > 1 ? t.sym * 2 * N_EPI : 0,
              reinterpret_cast<float2 *>(w + L.size), reinterpret_cast<float *>(w + L.rest)};
    const bool vec = C % 8 == 0;
    const bool tall = R > C;             // the smaller side is the columns
    const int m = L.m, n = tall ? R : C;
    cudaError_t e;
    if (is_small(m, n)) {
        const int cl = n <= SM_LONG ? 1 : n <= 2 * SM_LONG ? 2 : n <= 4 * SM_LONG ? 4 : SM_CTAS;
        Small p{};
        p.q = q;
        p.tall = tall;
        p.m = m; p.n = n; p.np = ((n + cl - 1) / cl + 63) / 64 * 64;
        p.steps = f.steps;
        memcpy(p.c, f.coeffs, 3 * f.steps * sizeof(float));
        p.scale = f.scale;
        p.out = static_cast<uint16_t *>(f.out);
        p.status = status;
        p.timeout_ns = timeout_ns;
        p.inject = inject;
        const size_t smem = m <= FEW ? Places<64>::bytes(p.np, cl) : Places<128>::bytes(p.np, cl);
        void (*kernel)(const Small) = m <= FEW ? (vec ? small_kernel<true, 64>(cl) : small_kernel<false, 64>(cl))
                                               : (vec ? small_kernel<true, 128>(cl) : small_kernel<false, 128>(cl));
        if ((e = ensure_smem(reinterpret_cast<const void *>(kernel), smem)) != cudaSuccess) return e;
        return launch_pdl(kernel, dim3(B * cl), dim3(ST), smem, s, cl, p);
    }
    const dim3 grid(L.parts, B);
    if ((e = launch_pdl(ortho_sample_kernel, dim3(B), dim3(PT), 0, s, 1, q)) != cudaSuccess) return e;
    e = launch_pdl(vec ? ortho_momentum_kernel<true> : ortho_momentum_kernel<false>, grid, dim3(PT), 0, s, 1, q);
    if (e != cudaSuccess) return e;
    const int rest = (2 * num_sms() + B - 1) / B;
    e = launch_pdl(vec ? ortho_scale_kernel<true> : ortho_scale_kernel<false>, dim3(L.parts < rest ? L.parts : rest, B),
                   dim3(PT), 0, s, 1, q);
    if (e != cudaSuccess) return e;

    void *A = w + L.A, *P = w + L.P;
    Args a;
    memset(&a, 0, sizeof a);
    const int most = num_sms() / 2;      // clusters
    a.tall = tall;
    a.steps = f.steps;
    a.B = B; a.m = m; a.R = R; a.C = C;
    a.side = t.side; a.n_side = t.n_side; a.sym = t.sym;
    a.tn = t.tn; a.nM = t.nM; a.nN = t.nN; a.app = t.app;
    a.group = t.group; a.split = t.split;
    const long long units = static_cast<long long>(f.steps) * B * ((a.split + 1) * a.sym + a.app);
    if (units >= (1ll << 31) - 65536) return cudaErrorInvalidValue;
    a.units = static_cast<int>(units);
    a.tma_out = C % 8 == 0 ? 1 : 0;
    memcpy(a.c, f.coeffs, 3 * f.steps * sizeof(float));
    a.scale = f.scale;
    a.out = static_cast<uint16_t *>(f.out);
    a.rest = q.rest;
    a.count = q.count;
    a.next = reinterpret_cast<int *>(q.count + B);
    a.sums = reinterpret_cast<float *>(w + L.sums);
    a.ticket = q.ticket;
    a.status = status;
    a.timeout_ns = timeout_ns;
    a.inject = inject;
    bool ok = encode(&a.a, A, B, m, m, L.ldm, 128, 64) && encode(&a.p, P, B, m, m, L.ldm, 128, 64) &&
              encode(&a.pa, A, B, m, m, L.ldm, 32, 32) && encode(&a.pp, P, B, m, m, L.ldm, 32, 32) &&
              encode(&a.pl, w + L.lo, B, R, C, L.ld, 32, 32);
    for (int i = 0; i < 2; ++i) {
        void *x = w + L.hi[i];
        ok = ok && encode(&a.xg[i], x, B, R, C, L.ld, tall ? 64 : 128, 64) &&
             encode(&a.xa[i], x, B, R, C, L.ld, tall ? 128 : 64, 64) && encode(&a.px[i], x, B, R, C, L.ld, 32, 32);
    }
    if (t.two)
        ok = ok && encode(&a.a2, w + L.A2, B, m, m, L.ldm, 128, 64) && encode(&a.p2, w + L.P2, B, m, m, L.ldm, 128, 64) &&
             encode(&a.pa2, w + L.A2, B, m, m, L.ldm, 32, 32) && encode(&a.pp2, w + L.P2, B, m, m, L.ldm, 32, 32);
    if (a.tma_out) ok = ok && encode(&a.po, f.out, B, R, C, C, 32, 32);
    if (!ok) return cudaErrorInvalidValue;
    const bool longer = m >= LONG_SUMS;
    void (*kernel)(const Args) = longer ? ortho_gemm_kernel<5, false> : t.two ? ortho_gemm_kernel<4, true> : ortho_gemm_kernel<4, false>;
    const size_t smem = longer ? Ring<5>::BYTES : Ring<4>::BYTES;
    if ((e = ensure_smem(reinterpret_cast<const void *>(kernel), smem)) != cudaSuccess) return e;
    const int gram = a.split * a.sym, widest = B * (gram > a.app ? gram : a.app);
    return launch_pdl(kernel, dim3(2 * (widest < most ? widest : most)), dim3(NT), smem, s, 2, a);
}

}  // namespace moe
