// ccc_scan_tc.cu -- the selective scan on the tensor cores (tcgen05), for
// states of up to 128 values and heads of up to 64 channels or a multiple of
// 64 (cut into tiles of 64): a walk over chunks of Q = 128 tokens that keeps
// the state on the chip.
//
// For a chunk that the state S enters (h: one head, all exponents in powers
// of two, a_t the running sum of dt A log2 e):
//     CB = C B^T                                    [t][s], shared by the pair of heads
//     M_ts = CB_ts dt_s 2^(a_t - a_s), s <= t       rounded to BF16 once
//     y_t = (M x)_t + 2^a_t (C S^T)_t + D x_t
//     S' = 2^a_end S + (w x)^T B,  w_s = dt_s 2^(a_end - a_s)
// S stays in FP32 in TMEM; its BF16 copy feeds C S^T.  w x is rounded to a
// BF16 high and low part, both multiplied: the state keeps 16 bits of each
// term.  x, B and C are BF16 and exact.
//
// A CTA has a pair of heads (128 rows of S) and four kinds of warps, so that a
// chunk's decays and M, its state, its loads and its products overlap with one
// another and with the next chunk's:
//   16 warps     M, the scaling of C S^T, y: a warpgroup takes a block of 32
//                columns of M for both heads, and half of a head's y
//   four warps   the state: its BF16 copy and its decay
//   four warps   w x
//   two warps    steps and decays, a head each
//   one warp     finds the chunks and loads them by TMA: B and x two chunks
//                deep, C one
//   one warp     issues the products
// Each kind runs its own code once a chunk, so the loops inside are kept
// rolled: with everything unrolled the warps waited for instructions half of
// the time.  (Eight warps for M and y: 956 us for the prompts below, products
// issued by a fixed lane in place of an elected one 916.)
// Measured: 64 prompts of 65536 tokens in all, 96 heads of 64, N = 128, 855 us or
// 2.55 TB/s of the bytes it cannot do without; one prompt of 65536 with 32 heads
// 363 us, 38 of them for the tails.  A chunk of a pair takes some 8900 cycles:
// neither memory (3300) nor the products (2300) bound it, but the chain CB -> M ->
// M x -> the next CB over one copy of C and one of M, the most that shared memory
// and TMEM hold, and on it M of the last block of rows, which one SM quarter does.
// TMEM (512 columns): CB, replaced by M of both heads as it is read | y: C S^T,
// scaled in place, then M x added | w x, high and low | S in FP32, decayed in
// place, then (w x)^T B added.
//
// Decays.  Within a block of 32 rows (a warp's) 2^(p_t - p_s) from the block's
// own running sums p; from block j to a later block q
//     2^(a_t - a_s) = [2^(P_j - p_s)] [2^(p_t + P_j+1 + .. + P_q-1)],
// P the blocks' totals: one exponential per s, three per t, in place of one per
// pair, neither factor above one for a decaying state.  P_j - p_s, like the decay
// to the chunk's end, is a sum over the tokens behind s, not that difference; within
// a block of 32, p_t - p_s is one of sums of 32 (M leaves in 8 bits).
#include <algorithm>

#include "ccc_checks.h"
#include "ccc_scan_tc.cuh"

namespace ccc {

namespace {

constexpr int Q = kTcChunk;
constexpr int kThreads = 896;
constexpr int kStateWarp = 16, kWxWarp = 20, kTmaWarp = 24, kMmaWarp = 25, kStepWarp = 26;  // from 0: M and y
constexpr uint32_t kOffC = 0, kOffK = 2 * kTile, kOffV = 6 * kTile, kOffS = 10 * kTile, kOffArr = 12 * kTile;
// A chunk's arrays, [head][token]: running sums within a block of 32, steps,
// decayed steps to the block's end, weights of w x; the blocks' totals.
struct Arrays {
    float p[2][Q], dt[2][Q], c[2][Q], w[2][Q], total[2][4];
};
using Desc = ChunkDesc;
constexpr int kDescs = 8, kAhead = 3;  // published ahead of the loads; a slot is written again when every warp is past it
constexpr uint32_t kOffDesc = kOffArr + 2 * sizeof(Arrays);
constexpr uint32_t kOffBar = kOffDesc + kDescs * sizeof(Desc);
constexpr uint32_t kSmem = kOffBar + 512;

constexpr uint32_t kColM = 0, kColY = 128, kColX = 256, kColS = 384;

enum Bar {
    // A waiter looks at a phase's parity alone: it must never be two phases late.  Where a barrier's next-but-one phase
    // does not need the waiter, there is one barrier per stage, whose phases do.
    kDesc0,
    kFullK0 = kDesc0 + kDescs, kFullK1, kFullV0, kFullV1, kFullC,       // TMA -> all
    kEmptyK0, kEmptyK1, kEmptyV0, kEmptyV1, kEmptyC,  // -> TMA
    kCbFull, kY1Full, kYFull, kDsFull,                // products done
    kSteps0, kSteps1, kArrays0, kArrays1,             // arrays ready / free
    kMReady, kYFree, kSReady, kXReady, kClean,
    kYWritten0, kYWritten1,                           // a head's y lies in shared memory
    kBars
};
static_assert(kSmem <= 232448 && 8 * kBars + sizeof(WaitState) <= 512, "shared memory of a CTA");

// NB: tiles of 64 state values.
template <int NB>
__global__ void __launch_bounds__(kThreads, 1) walk_kernel(const __grid_constant__ ScanTcArgs a) {
    extern __shared__ __align__(1024) unsigned char smem[];
    constexpr int NW = 64 * NB;  // state columns
    constexpr int kParts = 2;  // BF16 parts of w x
    const uint32_t base = smem_addr(smem);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const auto bar = [&](int b) { return base + kOffBar + 8 * b; };
    WaitState *const wait = reinterpret_cast<WaitState *>(smem + kOffBar + 8 * kBars);
    volatile int *failed = &wait->failed;
    Arrays *arrays = reinterpret_cast<Arrays *>(smem + kOffArr);
    if (tid == 0) {
        for (int b = 0; b < kSteps0; ++b) bar_init(bar(b), 1);
        for (int b : {kEmptyV0, kEmptyV1}) bar_init(bar(b), 2);  // the heads' y stores
        for (int b : {kSteps0, kSteps1}) bar_init(bar(b), 2);
        for (int b : {kArrays0, kArrays1}) bar_init(bar(b), 24);
        for (int b : {kMReady, kYFree}) bar_init(bar(b), 16);
        for (int b : {kSReady, kXReady, kClean}) bar_init(bar(b), 4);
        for (int b : {kYWritten0, kYWritten1}) bar_init(bar(b), 8);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        wait->failed = 0, wait->limit = a.waits.limit;
    }
    if (warp == kMmaWarp) tmem_alloc(smem_addr(&wait->tmem), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = wait->tmem;
    grid_dependents_launch();
    if (warp != kTmaWarp) grid_dependency_wait();  // (that warp looks for its chunks first)
    const auto desc = [&](int k) -> const Desc & {
        bar_wait(bar(kDesc0 + k % kDescs), (k / kDescs) & 1, failed);
        return reinterpret_cast<const Desc *>(smem + kOffDesc)[k % kDescs];
    };

    if (warp == kTmaWarp) {  // ------------------------------- chunks and loads
        Walk<false> wk;
        wk.init(a.s, a.pairs, blockIdx.x, gridDim.x);
        grid_dependency_wait();
        int dead = 0;
        int published = 0;
        bool open = true;
        const auto publish = [&] {  // the next chunk's description, or that there is none
            if (!open) return;
            if (wk.more && wk.fresh) dead = scan_padded(a.s, wk.n) ? kDead : 0;
            if (lane == 0) {
                describe(wk, dead, reinterpret_cast<Desc *>(smem + kOffDesc)[published % kDescs]);
                bar_arrive(bar(kDesc0 + published % kDescs));
            }
            __syncwarp();
            ++published;
            open = wk.more;
            if (!open) return;
            wk.next(a.s);
        };
        for (int i = 0; i < kAhead; ++i) publish();
        int k = 0, loaded_k = 0, loaded_c = 0, loaded_v = 0;
        for (;;) {
            const int st = k & 1;
            const Desc &d = reinterpret_cast<const Desc *>(smem + kOffDesc)[k % kDescs];
            const int row = d.row, pair = d.pair;
            if (__any_sync(kFull, *failed || !(d.flags & kMore))) break;
            const uint32_t free = ((k >> 1) & 1) ^ 1;
            publish();  // well ahead of the loads: the steps start from it
            if (lane == 0) {
                const int g = pair / a.pairs_per_group;
                bar_wait(bar(kEmptyK0 + st), free, failed);
                if (!*failed) {
                    ++loaded_k;
                    bar_expect(bar(kFullK0 + st), NB * kTile);
#pragma unroll
                    for (int b = 0; b < NB; ++b) tma_load(base + kOffK + (2 * st + b) * kTile, &a.mk, bar(kFullK0 + st), b * 64, g, row);
                }
                bar_wait(bar(kEmptyC), (k & 1) ^ 1, failed);
                if (!*failed) {
                    ++loaded_c;
                    bar_expect(bar(kFullC), NB * kTile);
#pragma unroll
                    for (int b = 0; b < NB; ++b) tma_load(base + kOffC + b * kTile, &a.mc, bar(kFullC), b * 64, g, row);
                }
                bar_wait(bar(kEmptyV0 + st), free, failed);
                if (!*failed) {
                    ++loaded_v;
                    bar_expect(bar(kFullV0 + st), 2 * kTile);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const Head h = head_of(a, pair, i);
                        tma_load(base + kOffV + (2 * st + i) * kTile, &a.mv, bar(kFullV0 + st), h.tile * 64, h.h, row);
                    }
                }
            }
            __syncwarp();
            ++k;
        }
        if (lane == 0) wait->started[0] = loaded_k, wait->started[1] = loaded_c, wait->started[2] = loaded_v;
    } else if (warp == kMmaWarp) {  // -------------------------------- products
        int k = 0;
        for (;; ++k) {
            const Desc &d = desc(k);
            if (__any_sync(kFull, *failed || !(d.flags & kMore))) break;
            const int st = k & 1;
            const uint32_t par = k & 1, was = par ^ 1, ring = (k >> 1) & 1;
            const uint32_t sc = base + kOffC, sk = base + kOffK + 2 * st * kTile, sv = base + kOffV + 2 * st * kTile, ss = base + kOffS;
            bar_wait(bar(kFullK0 + st), ring, failed);
            bar_wait(bar(kFullC), par, failed);
            if (k > 0) bar_wait(bar(kYFull), was, failed);  // M of the chunk before has been multiplied
            tc_fence_after();
            if (tc_elect()) {
#pragma unroll
                for (int i = 0; i < 4 * NB; ++i)
                        tc_mma_ss(tmem + kColM, tc_desc(sc + (i / 4) * kTile + (i % 4) * 32, 16, 1024),
                                  tc_desc(sk + (i / 4) * kTile + (i % 4) * 32, 16, 1024), tc_idesc(128, false, false), i > 0);
                tc_commit(bar(kCbFull));
            }
            __syncwarp();
            bar_wait(bar(kSReady), par, failed);
            if (k > 0) bar_wait(bar(kYFree), was, failed);
            tc_fence_after();
            if (tc_elect()) {
#pragma unroll
                for (int i = 0; i < 4 * NB; ++i)
                        tc_mma_ss(tmem + kColY, tc_desc(sc + (i / 4) * kTile + (i % 4) * 32, 16, 1024),
                                  tc_desc(ss + (i / 4) * kTile + (i % 4) * 32, 16, 1024), tc_idesc(128, false, false), i > 0);
                tc_commit(bar(kY1Full));
                tc_commit(bar(kEmptyC));
            }
            __syncwarp();
            bar_wait(bar(kXReady), par, failed);
            tc_fence_after();
            if (tc_elect()) {
#pragma unroll
                for (int i = 0; i < 8 * kParts; ++i)
                        tc_mma_ts(tmem + kColS, tmem + kColX + i * 8, tc_desc(sk + (i % 8) * 2048, kTile, 1024), tc_idesc(NW, false, true), true);
                tc_commit(bar(kDsFull));
                tc_commit(bar(kEmptyK0 + st));
            }
            __syncwarp();
            bar_wait(bar(kFullV0 + st), ring, failed);
            bar_wait(bar(kMReady), par, failed);
            tc_fence_after();
            if (tc_elect()) {
#pragma unroll
                for (int i = 0; i < 8; ++i)  // tokens 16 i ..: eight columns of each head
#pragma unroll
                        for (int h = 0; h < 2; ++h)  // (in turn: one head's products each wait for the one before)
                            tc_mma_ts(tmem + kColY + h * 64, tmem + kColM + i * 16 + h * 8,
                                      tc_desc(sv + h * kTile + i * 2048, kTile, 1024), tc_idesc(64, false, true), true);
                tc_commit(bar(kYFull));
            }
            __syncwarp();
        }
        if (lane == 0) wait->started[3] = k;
    } else if (warp >= kStepWarp) {  // ---------------------- steps and decays
        const int hd = warp - kStepWarp;
        int pair = -1, ahead_pair = -1;
        Head mine{}, ahead{};
        float A2 = 0.0f, bias = 0.0f;
        uint32_t raw[4], next[4];
        const auto fetch = [&](int k, uint32_t (&to)[4]) {  // false past the last chunk
            const Desc &d = desc(k);
            if (__any_sync(kFull, *failed || !(d.flags & kMore))) return false;
            if (d.pair != ahead_pair) {
                ahead_pair = d.pair;
                ahead = head_of(a, ahead_pair, hd);
            }
            fetch_steps(a, d, ahead, to);
            return true;
        };
        bool more = fetch(0, raw);
        for (int k = 0; more; ++k) {
            const Desc &d = desc(k);
            const int len = d.len;
            if (d.pair != pair) {
                pair = d.pair;
                mine = ahead;
                A2 = mine.ok ? par(a.s.A, a.s.p_bf16, mine.h) * kLog2e : 0.0f;
                bias = mine.ok && a.s.dt_bias ? par(a.s.dt_bias, a.s.p_bf16, mine.h) : 0.0f;
            }
            more = fetch(k + 1, next);
            float dt[4], v[4], p[4], P[4], to_end[4], after = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                dt[i] = mine.ok && 32 * i + lane < len ? step_of(dt_value(a.s, raw[i]) + bias, a.s.softplus) : 0.0f;
                v[i] = p[i] = dt[i] * A2;
            }
            block_sums(p, P);
            block_after(v, p, P, to_end);
            bar_wait(bar(kArrays0 + (k & 1)), ((k >> 1) & 1) ^ 1, failed);
            Arrays &r = arrays[k & 1];
#pragma unroll
            for (int i = 3; i >= 0; --i) {
                const int t = 32 * i + lane;
                const float c = dt[i] * ex2_approx(to_end[i]);
                r.p[hd][t] = p[i];
                r.dt[hd][t] = dt[i];
                r.c[hd][t] = c;
                r.w[hd][t] = c * ex2_approx(after);
                after += P[i];
            }
            if (lane < 4) r.total[hd][lane] = lane == 0 ? P[0] : lane == 1 ? P[1] : lane == 2 ? P[2] : P[3];
            warp_arrive(bar(kSteps0 + (k & 1)));
#pragma unroll
            for (int i = 0; i < 4; ++i) raw[i] = next[i];  // (waits for the loads)
        }
    } else if (warp < kStateWarp) {  // ---------------------------------- M and y
        const int wg = warp / 4, q = warp % 4, t = tid % 128;  // the warpgroup's block of M; the thread's row
        const int hd = wg / 2, half = wg % 2;                  // .. its head and its 32 channels of y
        const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
        const bool stores = half == 0 && t == 0;
        int pair = -1;
        Head mine{};
        float D = 0.0f;
        for (int k = 0;; ++k) {
            const Desc &d = desc(k);
            if (__any_sync(kFull, *failed || !(d.flags & kMore))) break;
            const int st = k & 1, len = d.len, row = d.row;
            const uint32_t parity = k & 1;
            const bool zero = d.flags & kDead;
            if (d.pair != pair) {
                pair = d.pair;
                mine = head_of(a, pair, hd);
                D = mine.ok && a.s.D ? par(a.s.D, a.s.p_bf16, mine.h) : 0.0f;
            }
            const Arrays &r = arrays[k & 1];
            bar_wait(bar(kSteps0 + st), (k >> 1) & 1, failed);
            // ---- M of both heads, the columns of block wg, over CB as it is read
            bar_wait(bar(kCbFull), parity, failed);
            tc_fence_after();
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {  // 16 columns of CB become 8 of either head's M
                const int s0 = wg * 32 + b * 16;
                uint32_t cb[16], m[8];
                if (wg <= q) {
                    tmem_ld16(tmem + lanes + kColM + s0, cb);
                    tmem_wait_ld();
                }
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    const float pt = r.p[h][t];
                    if (wg > q) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) m[i] = 0u;
                    } else if (wg == q) {
                        const int last = lane - b * 16;  // of these columns, the last one at or before the row
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {
                            const float4 ps = *reinterpret_cast<const float4 *>(&r.p[h][s0 + i]);
                            const float4 ds = *reinterpret_cast<const float4 *>(&r.dt[h][s0 + i]);
                            const float2 minus = make_float2(-1.0f, -1.0f), pp = make_float2(pt, pt);
                            const float2 a0 = __ffma2_rn(make_float2(ps.x, ps.y), minus, pp), a1 = __ffma2_rn(make_float2(ps.z, ps.w), minus, pp);
                            const float2 c0 = __fmul2_rn(make_float2(__uint_as_float(cb[i]), __uint_as_float(cb[i + 1])), make_float2(ds.x, ds.y));
                            const float2 c1 = __fmul2_rn(make_float2(__uint_as_float(cb[i + 2]), __uint_as_float(cb[i + 3])), make_float2(ds.z, ds.w));
                            const float2 v0 = __fmul2_rn(c0, make_float2(ex2_approx(a0.x), ex2_approx(a0.y)));
                            const float2 v1 = __fmul2_rn(c1, make_float2(ex2_approx(a1.x), ex2_approx(a1.y)));
                            m[i / 2] = pack2(i <= last ? v0.x : 0.0f, i + 1 <= last ? v0.y : 0.0f);
                            m[i / 2 + 1] = pack2(i + 2 <= last ? v1.x : 0.0f, i + 3 <= last ? v1.y : 0.0f);
                        }
                    } else {
                        float between = pt;
                        if (wg < 1 && q > 1) between += r.total[h][1];
                        if (wg < 2 && q > 2) between += r.total[h][2];
                        const float e = ex2_approx(between);
                        const float2 ee = make_float2(e, e);
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {
                            const float4 cs = *reinterpret_cast<const float4 *>(&r.c[h][s0 + i]);
                            const float2 u = __fmul2_rn(make_float2(cs.x, cs.y), ee), v = __fmul2_rn(make_float2(cs.z, cs.w), ee);
                            m[i / 2] = f2_to_bf2(__fmul2_rn(make_float2(__uint_as_float(cb[i]), __uint_as_float(cb[i + 1])), u));
                            m[i / 2 + 1] = f2_to_bf2(__fmul2_rn(make_float2(__uint_as_float(cb[i + 2]), __uint_as_float(cb[i + 3])), v));
                        }
                    }
                    tmem_st8(tmem + lanes + kColM + s0 + h * 8, m);
                }
            }
            // ---- C S^T scaled by the decay since the chunk's start
            float a_t = r.p[hd][t];
#pragma unroll
            for (int j = 0; j < 3; ++j) a_t += j < q ? r.total[hd][j] : 0.0f;
            const float e = ex2_approx(a_t);
            warp_arrive(bar(kArrays0 + st));
            bar_wait(bar(kY1Full), parity, failed);
            tc_fence_after();
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
                uint32_t y[16];
                tmem_ld16(tmem + lanes + kColY + wg * 32 + b * 16, y);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * e);
                tmem_st16(tmem + lanes + kColY + wg * 32 + b * 16, y);
            }
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(bar(kMReady));
            // ---- y, over x in its place
            unsigned char *tile = smem + kOffV + (2 * st + hd) * kTile + t * 128;
            const bool whole = len == Q;
            bar_wait(bar(kFullV0 + st), (k >> 1) & 1, failed);
            bar_wait(bar(kYFull), parity, failed);  // (w x)^T B was issued before M x: w x has been made, x is free too
            tc_fence_after();
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
                uint32_t y[16];
                tmem_ld16(tmem + lanes + kColY + wg * 32 + b * 16, y);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint4 *at = reinterpret_cast<uint4 *>(tile + (((half * 4 + b * 2 + i) ^ (t & 7)) << 4));
                    const uint4 xr = *at;
                    const uint32_t xs[4] = {xr.x, xr.y, xr.z, xr.w};
                    uint32_t o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int c = i * 8 + j * 2;
                        o[j] = f2_to_bf2(__ffma2_rn(make_float2(D, D), bf2_to_f2(xs[j]), make_float2(__uint_as_float(y[c]), __uint_as_float(y[c + 1]))));
                        if (zero) o[j] = 0u;
                    }
                    *at = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            tc_fence_before();
            warp_arrive(bar(kYFree));
            if (!whole && mine.ok && t < len) {  // a chunk that ends early: its rows alone
                uint16_t *to = a.s.out + (static_cast<int64_t>(row) + t) * a.s.out_rs + mine.h * a.s.P + mine.tile * 64;
#pragma unroll 1
                for (int i = half * 4; i < min(half * 4 + 4, (a.s.P - mine.tile * 64) / 8); ++i)
                    *reinterpret_cast<uint4 *>(to + i * 8) = *reinterpret_cast<const uint4 *>(tile + ((i ^ (t & 7)) << 4));
            }
            fence_async();
            warp_arrive(bar(kYWritten0 + hd));
            if (stores) {
                bar_wait(bar(kYWritten0 + hd), parity, failed);
                if (whole && mine.ok) {
                    tma_store(&a.mo, base + kOffV + (2 * st + hd) * kTile, mine.tile * 64, mine.h, row);
                    bulk_wait_read();
                }
                bar_arrive(bar(kEmptyV0 + st));
            }
            __syncwarp();
        }
        if (stores) bulk_wait_all();
    } else if (warp < kWxWarp) {  // -------------------------------- the state
        const int q = warp % 4, t = tid % 128, lh = t / 64, lp = t % 64;  // the thread's row
        const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
        const int64_t open = (static_cast<int64_t>(blockIdx.x) * Q + t) * NW;
        int pair = -1, k = 0, flags = 0, n = -1;
        Head state{};
        while (true) {
            const Desc &d = desc(k);
            const bool more = !__any_sync(kFull, *failed || !(d.flags & kMore));
            if (k > 0) {
                bar_wait(bar(kDsFull), (k - 1) & 1, failed);
                tc_fence_after();
                if ((flags & kLeaves) && !(flags & kDead)) {  // a sequence ends: its state goes out
                    float *to = scan_final(a.s, n);
                    if (to)
#pragma unroll 1
                        for (int b = 0; b < 4 * NB; ++b) {
                            float S[16];
                            tmem_ld16(tmem + lanes + kColS + b * 16, reinterpret_cast<uint32_t(&)[16]>(S));
                            tmem_wait_ld();
                            store_state(a, to, state, lp, b * 16, S);
                        }
                }
            }
            if (!more) break;
            const int st = k & 1;
            const uint32_t parity = k & 1, ring = (k >> 1) & 1;
            const Arrays &r = arrays[k & 1];
            flags = d.flags, n = d.n;
            if (d.pair != pair) {
                pair = d.pair;
                state = head_of(a, pair, lh);
            }
            // where a sequence's first state comes from
            const bool fresh = flags & kFresh, enters = flags & kEnters;
            const float *from = nullptr;
            int carry = -1;
            if (fresh && enters && !(flags & kDead)) from = scan_initial(a.s, n);
            if (fresh && !enters) carry = carry_from<false>(a);
            bar_wait(bar(kSteps0 + st), ring, failed);
            const float keep = ex2_approx(r.total[lh][0] + r.total[lh][1] + (r.total[lh][2] + r.total[lh][3]));
            if (k > 0) bar_wait(bar(kY1Full), parity ^ 1, failed);  // the chunk before's C S^T has read the BF16 copy
#pragma unroll 1
            for (int b = 0; b < 4 * NB; ++b) {
                float S[16];
                if (!fresh) {
                    tmem_ld16(tmem + lanes + kColS + b * 16, reinterpret_cast<uint32_t(&)[16]>(S));
                    tmem_wait_ld();
                } else if (carry >= 0) {
                    carry_in<false>(a, carry, t, lh, NW, b * 16, S);
                } else if (from && a.s.pool && (flags & kOpenEnd)) {
                    // the slot's last state may be there already (another CTA writes it): the copy that the first pass took
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 v = *reinterpret_cast<const float4 *>(a.staged + open + b * 16 + i);
                        S[i] = v.x, S[i + 1] = v.y, S[i + 2] = v.z, S[i + 3] = v.w;
                    }
                } else {
                    load_state(a, from, state, lp, b * 16, S);
                }
                // the BF16 copy
                unsigned char *rowp = smem + kOffS + (b / 4) * kTile + t * 128;
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    *reinterpret_cast<uint4 *>(rowp + (((b % 4 * 2 + i) ^ (t & 7)) << 4)) =
                        make_uint4(pack2(S[8 * i], S[8 * i + 1]), pack2(S[8 * i + 2], S[8 * i + 3]), pack2(S[8 * i + 4], S[8 * i + 5]),
                                   pack2(S[8 * i + 6], S[8 * i + 7]));
#pragma unroll
                for (int i = 0; i < 16; ++i) S[i] *= keep;
                tmem_st16(tmem + lanes + kColS + b * 16, reinterpret_cast<const uint32_t(&)[16]>(S));
            }
            tmem_wait_st();
            tc_fence_before();
            fence_async();
            warp_arrive(bar(kSReady));
            warp_arrive(bar(kArrays0 + st));
            ++k;
        }
    } else {  // ----------------------------------------------- w x, transposed
        const int q = warp % 4;  // 32 channels of the pair
        const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
        int clean = 0;
        for (int k = 0;; ++k) {
            const Desc &d = desc(k);
            if (__any_sync(kFull, *failed || !(d.flags & kMore))) break;
            const int st = k & 1, len = d.len;
            const uint32_t ring = (k >> 1) & 1;
            bar_wait(bar(kFullV0 + st), ring, failed);
            if (len < Q) {  // rows of the next sequence or of none: zeros, so that nothing of theirs is multiplied
                bar_wait(bar(kFullK0 + st), ring, failed);
                const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
                for (int i = len * 8 + tid % 128; i < Q * 8; i += 128) {
#pragma unroll
                    for (int b = 0; b < NB; ++b) *reinterpret_cast<uint4 *>(smem + kOffK + (2 * st + b) * kTile + i * 16) = zero;
#pragma unroll
                    for (int b = 0; b < 2; ++b) *reinterpret_cast<uint4 *>(smem + kOffV + (2 * st + b) * kTile + i * 16) = zero;
                }
                fence_async();
                warp_arrive(bar(kClean));
                bar_wait(bar(kClean), clean++ & 1, failed);  // this warp reads rows that others clear
            }
            bar_wait(bar(kSteps0 + st), ring, failed);
            if (k > 0) bar_wait(bar(kDsFull), (k - 1) & 1, failed);  // the chunk before's w x has been multiplied
            tc_fence_after();
            // ldmatrix hands a lane the channel lane / 4 and two tokens of each 8 x 8 block, as a 16x128b store to TMEM
            // takes them.  This lane's row of the four blocks: token lane % 8, channel block lane / 8 % 2, token block lane / 16.
            const float *w = arrays[st].w[q / 2];
            const uint32_t rows = base + kOffV + (2 * st + q / 2) * kTile + (lane / 16 * 8 + lane % 8) * 128;
#pragma unroll 1
            for (int hf = 0; hf < 8; ++hf) {  // 16 channels, 32 tokens
                const uint32_t chunk = ((q % 2 * 4 + hf / 4 * 2 + lane / 8 % 2) ^ (lane & 7)) << 4;
                uint32_t part[kParts][8];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t m[4];
                    const int s = hf % 4 * 32 + i * 16;
                    ldmatrix_trans(rows + s * 128 + chunk, m);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float2 v = __fmul2_rn(bf2_to_f2(m[j]), *reinterpret_cast<const float2 *>(w + s + j / 2 * 8 + lane % 4 * 2));
#pragma unroll
                        for (int e = 0; e < kParts; ++e) {
                            part[e][4 * i + j] = f2_to_bf2(v);
                            v = __ffma2_rn(bf2_to_f2(part[e][4 * i + j]), make_float2(-1.0f, -1.0f), v);
                        }
                    }
                }
                const uint32_t at = tmem + lanes + (static_cast<uint32_t>(hf / 4 * 16) << 16) + kColX + hf % 4 * 16;
#pragma unroll
                for (int e = 0; e < kParts; ++e) tmem_st_16x128b_x4(at + e * 64, part[e]);
            }
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(bar(kXReady));
            warp_arrive(bar(kArrays0 + st));
        }
    }
    tc_fence_before();
    __syncthreads();
    if (*failed) {
        if (tid == 0) {
            bar_drain(bar(kFullK0), 2, wait->started[0]);
            bar_drain(bar(kFullC), 1, wait->started[1]);
            bar_drain(bar(kFullV0), 2, wait->started[2]);
            bar_drain(bar(kYFull), 1, wait->started[3]);
        }
        __syncthreads();
    }
    tc_fence_after();
    if (warp == kMmaWarp) tmem_free(tmem, 512);
    if (tid == 0 && *failed) *a.status = 1, report_given_up(a.waits);
}

}  // namespace

bool make_scan_map(CUtensorMap *map, const uint16_t *p, int size, int count, int64_t rows, int64_t rs, int box_rows) {
    using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<Encode>(f);
    }();
    if (!encode) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(size), static_cast<cuuint64_t>(count), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(size) * 2, static_cast<cuuint64_t>(rs) * 2};
    const cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(box_rows)}, one[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(p), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

template <int NB>
cudaError_t launch_walk(const ScanTcArgs &a, int parts, bool first, cudaStream_t st) {
    const auto kernel = walk_kernel<NB>;
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem)) return e;
    return launch_behind(kernel, dim3(parts), kThreads, kSmem, first, st, a);
}

}  // namespace

ScanTcPlan scan_tc_plan(int64_t rows, int n_seqs, int H, int P, int G, int N) {
    ScanTcPlan p = {};
    p.ok = N <= 128 && (P <= 64 || P % 64 == 0);
    if (!p.ok || rows <= 0 || n_seqs <= 0) return p;
    p.nb = N <= 64 ? 1 : 2;
    p.tiles = P <= 64 ? 1 : P / 64;
    p.pairs_per_group = (H / G * p.tiles + 1) / 2;
    p.pairs = p.pairs_per_group * G;
    // One CTA per SM (152, fixed: the cuts decide the order of sums), but at
    // least two chunks a CTA where that many pairs exist, and no cuts where a pair
    // has about eight chunks or fewer: a second launch takes as long (one
    // 1000-token prompt: 42 us without, 45-50 with cuts every four, three, two).
    const int64_t chunks = (rows + Q - 1) / Q + n_seqs / 2, most = static_cast<int64_t>(p.pairs) * ((chunks + 1) / 2);
    p.parts = static_cast<int>(chunks <= 8 ? p.pairs : std::min<int64_t>(152, std::max<int64_t>(most, p.pairs)));
    p.cuts = p.pairs % p.parts != 0;
    const size_t state = static_cast<size_t>(p.parts) * Q * 64 * p.nb * 4;
    p.status = 0;
    p.keep = kAlignWs;
    p.flag = p.keep + round_up(static_cast<size_t>(p.parts) * 8, kAlignWs);
    p.local = p.flag + round_up(static_cast<size_t>(p.parts) * 4, kAlignWs);
    p.staged = p.local + state;
    p.bytes = p.cuts ? p.staged + state : kAlignWs;
    return p;
}

cudaError_t launch_scan_tc_fwd(const ScanArgs &s, const ScanTcPlan &plan, unsigned char *ws, int *launches, cudaStream_t st) {
    ScanTcArgs a = {};
    a.s = s;
    a.pairs = plan.pairs, a.pairs_per_group = plan.pairs_per_group, a.tiles = plan.tiles;
    a.status = reinterpret_cast<int *>(ws + plan.status);
    a.waits = current_waits();
    a.local = reinterpret_cast<float *>(ws + plan.local);
    a.keep = reinterpret_cast<float *>(ws + plan.keep);
    a.flag = reinterpret_cast<int *>(ws + plan.flag);
    a.staged = s.pool ? reinterpret_cast<float *>(ws + plan.staged) : nullptr;
    if (!make_scan_map(&a.mv, s.x, s.P, s.H, s.rows, s.x_rs, Q) || !make_scan_map(&a.mk, s.B, s.N, s.G, s.rows, s.b_rs, Q) ||
        !make_scan_map(&a.mc, s.C, s.N, s.G, s.rows, s.c_rs, Q) || !make_scan_map(&a.mo, s.out, s.P, s.H, s.rows, s.out_rs, Q))
        return cudaErrorInvalidValue;
    *launches = 1;
    if (s.final_state) {
        if (cudaError_t e = launch_edge_states(s, s.final_state, false, st)) return e;
        ++*launches;
    }
    if (plan.cuts) {
        if (cudaError_t e = launch_scan_tc_tails(a, plan, false, false, *launches == 1, st)) return e;
        ++*launches;
    }
    return plan.nb == 1 ? launch_walk<1>(a, plan.parts, *launches == 1, st) : launch_walk<2>(a, plan.parts, *launches == 1, st);
}

}  // namespace ccc
