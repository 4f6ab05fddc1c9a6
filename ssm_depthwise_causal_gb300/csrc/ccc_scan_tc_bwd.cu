// ccc_scan_tc_bwd.cu -- the backward of the selective scan on the tensor
// cores, from the state S before each chunk and the state gradient G after it
// (both from the walks of ccc_scan_tc_states.cu, as three BF16 parts: all 24 bits).
//
// Per chunk of Q = 128 tokens and head, exponents in powers of two, L_ts =
// 2^(a_t - a_s) for s <= t:
//     dC_t = sum_h [ sum_s L_ts dt_s (dy_t.x_s) B_s + 2^a_t dy_t S ]
//     dB_s = sum_h [ sum_t L_ts dt_s (dy_t.x_s) C_t + dt_s 2^(a_end - a_s) x_s G ]
//     dx_s = dt_s sum_t L_ts (C_t.B_s) dy_t + dt_s 2^(a_end - a_s) G B_s + D dy_s
// The first two are one computation with the roles exchanged: rows i with Q, U
// and columns j with K, V, and a state E:
//     T1 = Q K^T, T2 = U V^T, W = T2 L dt, out_i = (W K)_i + s_i (U E)_i
//     forward  rows t: Q = C, U = dy, K = B, V = x,  E = S, s_t = 2^a_t
//     reverse  rows s: Q = B, U = x,  K = C, V = dy, E = G, s_s = dt_s 2^(a_end - a_s)
// and the reverse one has M = T1 L for dx besides.  Each row's share of the
// decays' gradient is the row sum of T1 T2 L, which stays in FP32, and Q_i.(U E)_i
// with all parts of E; that way both orientations of the sums are a thread's own.
// Rounded to BF16, once each: W and M, as operands of products whose results leave
// in 16 bits (dC, dB, dx), where they cost a unit roundoff of each term.  U E has all
// 24 bits of the state; dx's G B has two parts of G, 16 bits: the second one makes
// dx's state term as good as its own rounding (one part: off by a unit more) and
// takes no measurable time, a third one 4 of 601 us.
// dt, A, D and dt_bias follow from them (finish_kernel):
// d(dt A)_t is the sum over all pairs (s, u) with s < t <= u of what s gives to
// u, for s before the chunk and u behind it too.  For pairs of one block of 32
// tokens that is a difference of running sums of rows and columns; pairs of two
// blocks, and those with S or G, are added up as they are, so that nothing longer
// than a block cancels.
//
// A CTA takes a chunk and a group and goes through the group's heads, so that
// dB and dC are summed over the heads in TMEM and registers.  Sixteen warps of
// arithmetic (row = lane; a warpgroup takes a block of 32 columns, a quarter of
// the others), one for the steps, one for the loads (two heads deep), one that
// issues the products, one through which dx leaves.  TMEM: T1 | T2, replaced by W
// (and M) | W K summed over the heads | U E, then the two parts of dx.
// 16384 tokens, 32 heads of 64 in 8 groups, N = 128: 94 us forward, 172 reverse
// (x, dy and a state, 80 KB a head and chunk, reverse dx and the other state too:
// 3.5 TB/s in both).  A head takes 4000 cycles forward, the chain T2 -> W -> W K in
// which the last (first, reverse) block of rows has four blocks of W to make, and
// reverse dx behind it; a group's first head some 4000 more, since there is no room
// for the next Q and K.  Eight warps with two blocks each: 105 and 162 us without
// the product below.  <G, S>, each chunk's share of all decays that pass through it,
// is taken while dx is being multiplied, G from shared memory, S from L2: 40 us;
// 55 in a kernel that reads both again, 110 a row a thread in the walk that makes G.
#include <algorithm>

#include "ccc_checks.h"
#include "ccc_scan_tc.h"
#include "ccc_scan_walk.cuh"
#include "ccc_tc.cuh"

namespace ccc {

namespace {

constexpr int Q = kTcChunk;
constexpr int kThreads = 640;
constexpr int kTmaWarp = 16, kMmaWarp = 17, kStepWarp = 18;  // 0-15: arithmetic, 19: stores
constexpr uint32_t kTile = 16384;  // 128 rows of 64 BF16
constexpr uint32_t kOffQ = 0, kOffK = 2 * kTile, kOffU = 4 * kTile;  // a head's stage: U, V, E (three parts; two halves of 64 columns each)
constexpr uint32_t kHead = 5 * kTile;
constexpr uint32_t kOffArr = kOffU + 2 * kHead;
struct Arrays {
    float p[Q], dt[Q], c[Q], total[4];
};
struct Desc {
    int slot, row, len, g, flags, pad[3];
};
enum : int { kMore = 1, kDead = 2 };
constexpr int kDescs = 4;
constexpr uint32_t kOffDesc = kOffArr + sizeof(Arrays);
constexpr uint32_t kOffBar = kOffDesc + kDescs * sizeof(Desc);
constexpr uint32_t kSmem = kOffBar + 512;

constexpr uint32_t kColT1 = 0, kColW = 128, kColAcc = 256, kColE = 384;

// As in ccc_scan_tc.cu: a waiter looks at parities alone, so it must never be two phases late, nor one early.
enum Bar {
    kDesc0,
    kFullQK = kDesc0 + kDescs, kFullU0, kFullU1,
    kEmptyQK, kEmptyU0, kEmptyU1,
    kT1Full, kT2Full, kEFull, kWUsed, kDxFull,
    kSteps, kArrays,
    kWReady, kERead, kDxRead, kAccRead,
    kDxWritten0, kDxWritten1,
    kBars
};
static_assert(kSmem <= 232448 && 8 * kBars + sizeof(WaitState) <= 512, "shared memory of a CTA");

struct BwdTcArgs {
    CUtensorMap mq, mk, mu, mv, me, mdx;  // rows' and columns' sides, states (boxes of 64 rows), dx
    ScanArgs s;
    int pairs, pairs_per_group, tiles, heads;  // heads: head tiles of all groups
    int64_t slots;
    const uint16_t *states;  // reverse: the states before the chunks
    float *sums;             // [chunk][head tile][kPlanes][128]
    int *status;
    Waits waits;
};

// Planes of `sums`, the sums of T1 T2 L over a row: within the diagonal block
// (without the diagonal), over each other block, Q_i.(U E)_i (four quarters),
// forward and reverse; dy_t.x_t, and that times C_t.B_t; <G, S>, a part from each
// of the 16 warps.
enum { kRowDiag, kRowOff, kRowIn = 4, kColDiag = 8, kColOff, kColIn = 12, kDiag = 16, kDiagZ, kDot, kPlanes };

__device__ __forceinline__ uint32_t pack2(float lo, float hi) { return f2_to_bf2(make_float2(lo, hi)); }

__device__ __forceinline__ void warp_arrive(uint32_t bar) {
    __syncwarp();
    if (threadIdx.x % 32 == 0) bar_arrive(bar);
}

template <int NB, bool R>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const __grid_constant__ BwdTcArgs a) {
    extern __shared__ __align__(1024) unsigned char smem[];
    constexpr int NW = 64 * NB;
    const uint32_t base = smem_addr(smem);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const auto bar = [&](int b) { return base + kOffBar + 8 * b; };
    WaitState *const wait = reinterpret_cast<WaitState *>(smem + kOffBar + 8 * kBars);
    volatile int *failed = &wait->failed;
    Arrays &r = *reinterpret_cast<Arrays *>(smem + kOffArr);
    const int rep = a.s.H / a.s.G * a.tiles;  // head tiles of a group
    if (tid == 0) {
        for (int b = 0; b < kWReady; ++b)
            bar_init(bar(b), b == kArrays ? 16 : b == kEmptyQK ? 17 : 1);
        for (int b = kWReady; b < kBars; ++b) bar_init(bar(b), 16);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        wait->failed = 0, wait->limit = a.waits.limit;
    }
    if (warp == kMmaWarp) tmem_alloc(smem_addr(&wait->tmem), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = wait->tmem;
    grid_dependents_launch();
    grid_dependency_wait();
    const auto desc = [&](int k) -> const Desc & {
        bar_wait(bar(kDesc0 + k % kDescs), (k / kDescs) & 1, failed);
        return reinterpret_cast<const Desc *>(smem + kOffDesc)[k % kDescs];
    };

    if (warp == kTmaWarp) {  // ------------------------------- tasks and loads
        if (lane == 0) {
            int task = 0, k = 0;  // tasks published, heads gone through
            int loaded_qk = 0, loaded_u = 0;
            const auto publish = [&](int64_t &at) {  // the next chunk and group that exist; false after the last
                Desc &d = reinterpret_cast<Desc *>(smem + kOffDesc)[task % kDescs];
                d.flags = 0;
                for (; at < a.slots * a.s.G; at += gridDim.x) {
                    const Chunk c = scan_chunk(a.s, at / a.s.G, Q);
                    if (c.len == 0) continue;
                    d.slot = static_cast<int>(at / a.s.G), d.row = static_cast<int>(c.row), d.len = c.len, d.g = static_cast<int>(at % a.s.G);
                    d.flags = kMore | (scan_padded(a.s, c.n) ? kDead : 0);
                    at += gridDim.x;
                    break;
                }
                const bool more = d.flags & kMore;
                bar_arrive(bar(kDesc0 + task % kDescs));
                ++task;
                return more;
            };
            int64_t at = blockIdx.x;
            bool more = publish(at);
            for (int t = 0; more; ++t) {
                const Desc d = reinterpret_cast<const Desc *>(smem + kOffDesc)[t % kDescs];
                const Desc &next = reinterpret_cast<const Desc *>(smem + kOffDesc)[(t + 1) % kDescs];
                for (int v = 0; v < rep; ++v, ++k) {
                    const int st = k & 1;
                    bar_wait(bar(kEmptyU0 + st), ((k >> 1) & 1) ^ 1, failed);
                    if (*failed) continue;
                    const uint32_t to = base + kOffU + st * kHead, full = bar(kFullU0 + st);
                    const int h = d.g * (a.s.H / a.s.G) + v / a.tiles, tile = v % a.tiles;
                    ++loaded_u;
                    bar_expect(full, 2 * kTile + 3 * NB * (kTile / 2));
                    tma_load(to, &a.mu, full, tile * 64, h, d.row);
                    tma_load(to + kTile, &a.mv, full, tile * 64, h, d.row);
                    const int pair = d.g * a.pairs_per_group + v / 2;
#pragma unroll
                    for (int part = 0; part < 3; ++part)
#pragma unroll
                        for (int b = 0; b < NB; ++b)
                            tma_load(to + 2 * kTile + part * kTile + b * (kTile / 2), &a.me, full, b * 64, 0,
                                     ((d.slot * a.pairs + pair) * 3 + part) * Q + v % 2 * 64);
                    if (R) {
                        const uint16_t *S = a.states + ((static_cast<int64_t>(d.slot) * a.pairs + pair) * 3 * Q + v % 2 * 64) * NW;
#pragma unroll
                        for (int part = 0; part < 3; ++part) l2_prefetch(S + part * Q * NW, 64 * NW * 2);
                    }
                    if (v == 0) {
                        bar_wait(bar(kEmptyQK), (t & 1) ^ 1, failed);
                        if (!*failed) {
                            ++loaded_qk;
                            bar_expect(bar(kFullQK), 2 * NB * kTile);
#pragma unroll
                            for (int b = 0; b < NB; ++b) {
                                tma_load(base + kOffQ + b * kTile, &a.mq, bar(kFullQK), b * 64, d.g, d.row);
                                tma_load(base + kOffK + b * kTile, &a.mk, bar(kFullQK), b * 64, d.g, d.row);
                            }
                        }
                        more = publish(at);  // (the steps look two heads ahead)
#pragma unroll
                        for (int b = 0; b < NB && more; ++b) {  // there is no room for the next one's Q and K: into L2 at least
                            tma_prefetch(&a.mq, b * 64, next.g, next.row);
                            tma_prefetch(&a.mk, b * 64, next.g, next.row);
                        }
                    }
                }
                if (*failed) break;
            }
            wait->started[0] = loaded_u, wait->started[1] = loaded_qk;
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {  // -------------------------------- products
        int k = 0;
        for (int t = 0;; ++t) {
            const int flags = desc(t).flags;
            if (__any_sync(kFull, *failed || !(flags & kMore))) break;
            const uint32_t sq = base + kOffQ, sk = base + kOffK;
            bar_wait(bar(kFullQK), t & 1, failed);
            tc_fence_after();
            if (tc_elect()) {
#pragma unroll
                    for (int i = 0; i < 4 * NB; ++i)
                        tc_mma_ss(tmem + kColT1, tc_desc(sq + (i / 4) * kTile + (i % 4) * 32, 16, 1024),
                                  tc_desc(sk + (i / 4) * kTile + (i % 4) * 32, 16, 1024), tc_idesc(128, false, false), i > 0);
                tc_commit(bar(kT1Full));
            }
            __syncwarp();
            for (int v = 0; v < rep; ++v, ++k) {
                const int st = k & 1;
                const uint32_t ph = k & 1, was = ph ^ 1;
                const uint32_t su = base + kOffU + st * kHead, sv = su + kTile, se = sv + kTile;
                bar_wait(bar(kFullU0 + st), (k >> 1) & 1, failed);
                if (k > 0) bar_wait(bar(kWUsed), was, failed);  // W of the head before has been multiplied
                tc_fence_after();
                if (tc_elect()) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            tc_mma_ss(tmem + kColW, tc_desc(su + i * 32, 16, 1024), tc_desc(sv + i * 32, 16, 1024), tc_idesc(128, false, false), i > 0);
                    tc_commit(bar(kT2Full));
                }
                __syncwarp();
                if (k > 0) bar_wait(bar(R ? kDxRead : kERead), was, failed);
                tc_fence_after();
                if (tc_elect()) {
#pragma unroll
                        for (int i = 0; i < 12; ++i)  // the three parts: 64 channels each
                            tc_mma_ss(tmem + kColE, tc_desc(su + (i % 4) * 32, 16, 1024), tc_desc(se + (i / 4) * kTile + (i % 4) * 2048, kTile / 2, 1024),
                                      tc_idesc(NW, false, true), i > 0);
                    tc_commit(bar(kEFull));
                }
                __syncwarp();
                bar_wait(bar(kWReady), ph, failed);
                if (v == 0 && t > 0) bar_wait(bar(kAccRead), (t - 1) & 1, failed);
                tc_fence_after();
                if (tc_elect()) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)  // columns 16 i ..
                            tc_mma_ts(tmem + kColAcc, tmem + kColW + i * 16, tc_desc(sk + i * 2048, kTile, 1024),
                                      tc_idesc(NW, false, true), v > 0 || i > 0);
                }
                __syncwarp();
                if (R) {
                    bar_wait(bar(kERead), ph, failed);
                    tc_fence_after();
                    if (tc_elect()) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {  // dx: M dy, and B G^T with two parts of G, in turn
                            tc_mma_ts(tmem + kColE, tmem + kColW + i * 16 + 8, tc_desc(sv + i * 2048, kTile, 1024),
                                      tc_idesc(64, false, true), i > 0);
#pragma unroll
                            for (int part = 0; part < 2 && i < 4 * NB; ++part)
                                tc_mma_ss(tmem + kColE + 64, tc_desc(sq + (i / 4) * kTile + (i % 4) * 32, 16, 1024),
                                          tc_desc(se + part * kTile + (i / 4) * (kTile / 2) + (i % 4) * 32, 16, 1024), tc_idesc(64, false, false),
                                          i > 0 || part > 0);
                        }
                        tc_commit(bar(kDxFull));
                    }
                    __syncwarp();
                }
                if (tc_elect()) {
                    tc_commit(bar(kWUsed));
                    if (!R) tc_commit(bar(kEmptyU0 + st));
                    if (v == rep - 1) tc_commit(bar(kEmptyQK));
                }
                __syncwarp();
            }
        }
        if (lane == 0) wait->started[2] = k;
    } else if (warp == kStepWarp) {  // ------------------- steps and decays
        struct Raw {
            uint32_t A, bias, dt[4];  // as loaded
            int len;
        };
        int ft = 0, fv = 0;  // the head to fetch
        const auto fetch = [&](Raw &to) {
            const Desc &d = desc(ft);
            to.len = -1;
            if (__any_sync(kFull, *failed || !(d.flags & kMore))) return;
            const int h = d.g * (a.s.H / a.s.G) + fv / a.tiles;
            to.len = d.len;
            to.A = par_bits(a.s.A, a.s.p_bf16, h);
            to.bias = a.s.dt_bias ? par_bits(a.s.dt_bias, a.s.p_bf16, h) : 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                to.dt[i] = 0u;
                if (32 * i + lane < d.len) to.dt[i] = dt_bits(a.s, static_cast<int64_t>(d.row) + 32 * i + lane, h);
            }
            if (++fv == rep) fv = 0, ++ft;
        };
        Raw now, next;
        fetch(now);
        next.len = -1;
        if (now.len >= 0) fetch(next);  // (two heads are loaded before the first is done)
        for (int k = 0; now.len >= 0; ++k) {
            const float A2 = par_value(a.s.p_bf16, now.A) * kLog2e, bias = par_value(a.s.p_bf16, now.bias);
            float dt[4], p[4], P[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                dt[i] = 32 * i + lane < now.len ? step_of(dt_value(a.s, now.dt[i]) + bias, a.s.softplus) : 0.0f;
                p[i] = dt[i] * A2;
            }
#pragma unroll
            for (int j = 1; j < 32; j *= 2)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float o = __shfl_up_sync(kFull, p[i], j);
                    if (lane >= j) p[i] += o;
                }
#pragma unroll
            for (int i = 0; i < 4; ++i) P[i] = __shfl_sync(kFull, p[i], 31);
            if (k > 0) bar_wait(bar(kArrays), (k - 1) & 1, failed);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                r.p[32 * i + lane] = p[i];
                r.dt[32 * i + lane] = dt[i];
                r.c[32 * i + lane] = R ? ex2_approx(p[i]) : dt[i] * ex2_approx(P[i] - p[i]);
            }
            if (lane < 4) r.total[lane] = lane == 0 ? P[0] : lane == 1 ? P[1] : lane == 2 ? P[2] : P[3];
            warp_arrive(bar(kSteps));
            if (__any_sync(kFull, *failed)) break;
            now = next;  // (waits for its loads)
            if (now.len >= 0) fetch(next);
        }
    } else if (warp > kStepWarp) {  // ------------------------- dx leaves
        if (R && lane == 0) {
            int k = 0;
            for (int t = 0;; ++t) {
                const Desc d = desc(t);
                if (*failed || !(d.flags & kMore)) break;
                const bool whole = d.len == Q;  // (a chunk that ends early is written row by row)
                for (int v = 0; v < rep; ++v, ++k) {
                    bar_wait(bar(kDxWritten0 + (k & 1)), (k >> 1) & 1, failed);
                    if (whole) {
                        tma_store(&a.mdx, base + kOffU + (k & 1) * kHead + kTile, v % a.tiles * 64, d.g * (a.s.H / a.s.G) + v / a.tiles, d.row);
                        bulk_wait_read();
                    }
                    bar_arrive(bar(kEmptyU0 + (k & 1)));
                }
            }
            bulk_wait_all();
        }
        __syncwarp();
    } else {  // --------------------------------------------------- arithmetic
        const int j = warp / 4, q = warp % 4, i0 = tid % 128;  // the block of columns (a quarter of the others), the thread's row
        const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
        constexpr int kC8 = 2 * NB;  // 16-byte chunks of a quarter of NW columns
        int k = 0;
        for (int t = 0;; ++t) {
            const Desc &d = desc(t);
            if (__any_sync(kFull, *failed || !(d.flags & kMore))) break;
            const int len = d.len;
            const bool whole = len == Q, dead = d.flags & kDead;
            float2 out[NB * 8];  // sum over the heads of s_i (U E)_i
#pragma unroll
            for (int i = 0; i < NB * 8; ++i) out[i] = f2_zero();
            bar_wait(bar(kFullQK), t & 1, failed);
            if (!whole)  // rows of the next sequence or of none
                for (int i = len * 8 + tid; i < Q * 8; i += 512)
#pragma unroll
                    for (int b = 0; b < NB; ++b) *reinterpret_cast<uint4 *>(smem + kOffK + b * kTile + i * 16) = make_uint4(0u, 0u, 0u, 0u);
            bar_wait(bar(kT1Full), t & 1, failed);
            for (int v = 0; v < rep; ++v, ++k) {
                const int st = k & 1;
                const uint32_t ph = k & 1, ring = (k >> 1) & 1;
                unsigned char *sv = smem + kOffU + st * kHead + kTile;
                if (!whole) {
                    bar_wait(bar(kFullU0 + st), ring, failed);
                    for (int i = len * 8 + tid; i < Q * 8; i += 512) *reinterpret_cast<uint4 *>(sv + i * 16) = make_uint4(0u, 0u, 0u, 0u);
                    fence_async();
                }
                bar_wait(bar(kSteps), ph, failed);
                const float pi = r.p[i0], dti = r.dt[i0];
                // ---- W (and M), over T2 as it is read: 16 columns of each at a time
                bar_wait(bar(kT2Full), ph, failed);
                tc_fence_after();
                float *sums = a.sums + (static_cast<int64_t>(d.slot) * a.heads + d.g * rep + v) * kPlanes * Q + i0;
                const uint32_t at = tmem + lanes + kColW + j * 32;
                if (R ? j < q : j > q) {
                    uint32_t zero[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) zero[i] = 0u;
                    tmem_st16(at, zero);
                    tmem_st16(at + 16, zero);
                } else if (j == q) {
                    float own = 0.0f, diag = 0.0f, diagz = 0.0f;
#pragma unroll 1
                    for (int hf = 0; hf < 32; hf += 16) {
                        uint32_t t1[16], t2[16], w[8], m[8];
                        tmem_ld16(tmem + lanes + kColT1 + j * 32 + hf, t1);
                        tmem_ld16(at + hf, t2);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const float2 pj = *reinterpret_cast<const float2 *>(&r.p[j * 32 + hf + i]);
                            const float2 dj = R ? make_float2(dti, dti) : *reinterpret_cast<const float2 *>(&r.dt[j * 32 + hf + i]);
                            const float pjs[2] = {pj.x, pj.y}, djs[2] = {dj.x, dj.y};
                            float wv[2], mv[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int col = hf + i + e;
                                const bool on = R ? col >= lane && j * 32 + col < len : col <= lane;
                                const float l = on ? ex2_approx(R ? pjs[e] - pi : pi - pjs[e]) : 0.0f;  // (off the triangle it may be infinite)
                                const float u = on ? __uint_as_float(t2[i + e]) * l : 0.0f;
                                const float c = on ? __uint_as_float(t1[i + e]) : 0.0f;
                                wv[e] = u * djs[e];
                                mv[e] = c * l;
                                if (col == lane) diag = u, diagz = u * c;
                                else own = fmaf(c, R ? u : wv[e], own);
                            }
                            w[i / 2] = pack2(wv[0], wv[1]);
                            m[i / 2] = pack2(mv[0], mv[1]);
                        }
                        tmem_st8(at + hf, w);
                        if (R) tmem_st8(at + hf + 8, m);
                    }
                    sums[(R ? kColDiag : kRowDiag) * Q] = own;
                    if (!R) sums[kDiag * Q] = diag, sums[kDiagZ * Q] = diagz;
                } else {
                    float e = R ? r.total[q] - pi : pi;  // to the end of the row's block; and the blocks between
#pragma unroll
                    for (int b = 1; b < 3; ++b) e += (R ? b > q && b < j : b > j && b < q) ? r.total[b] : 0.0f;
                    e = ex2_approx(e);
                    const float2 ee = make_float2(e, e), dd = make_float2(dti, dti);
                    float2 s2 = f2_zero();
#pragma unroll 1
                    for (int hf = 0; hf < 32; hf += 16) {
                        uint32_t t1[16], t2[16], w[8], m[8];
                        tmem_ld16(tmem + lanes + kColT1 + j * 32 + hf, t1);
                        tmem_ld16(at + hf, t2);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const int col = j * 32 + hf + i;
                            const float2 l = __fmul2_rn(*reinterpret_cast<const float2 *>(&r.c[col]), ee);
                            float2 u = __fmul2_rn(make_float2(__uint_as_float(t2[i]), __uint_as_float(t2[i + 1])), l);
                            float2 c = make_float2(__uint_as_float(t1[i]), __uint_as_float(t1[i + 1]));
                            if (R) {  // columns past the chunk's end
                                if (col >= len) u.x = c.x = 0.0f;
                                if (col + 1 >= len) u.y = c.y = 0.0f;
                            }
                            s2 = __ffma2_rn(c, u, s2);
                            w[i / 2] = f2_to_bf2(R ? __fmul2_rn(u, dd) : u);
                            if (R) m[i / 2] = f2_to_bf2(__fmul2_rn(c, l));
                        }
                        tmem_st8(at + hf, w);
                        if (R) tmem_st8(at + hf + 8, m);
                    }
                    sums[(R ? kColOff + j - 1 : kRowOff + j) * Q] = s2.x + s2.y;
                }
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(bar(kWReady));
                // ---- U E
                float e = R ? r.total[q] - pi : pi;
#pragma unroll
                for (int b = 0; b < 4; ++b) e += (R ? b > q : b < q) ? r.total[b] : 0.0f;
                e = ex2_approx(e);
                warp_arrive(bar(kArrays));
                const float scale = R ? e * dti : e;
                bar_wait(bar(kEFull), ph, failed);
                tc_fence_after();
                float2 in2 = f2_zero();
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    uint32_t u[16];
                    const int c0 = j * kC8 + b * 2;  // first 16-byte chunk of the row's NW values
                    tmem_ld16(tmem + lanes + kColE + c0 * 8, u);
                    uint4 qr[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) qr[i] = *reinterpret_cast<const uint4 *>(smem + kOffQ + (c0 / 8) * kTile + i0 * 128 + (((c0 + i) % 8 ^ (i0 & 7)) << 4));
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t qs = i % 4 == 0 ? qr[i / 4].x : i % 4 == 1 ? qr[i / 4].y : i % 4 == 2 ? qr[i / 4].z : qr[i / 4].w;
                        const float2 uv = make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
                        out[b * 8 + i] = __ffma2_rn(make_float2(scale, scale), uv, out[b * 8 + i]);
                        in2 = __ffma2_rn(bf2_to_f2(qs), uv, in2);
                    }
                }
                tc_fence_before();
                warp_arrive(bar(kERead));
                if (v == rep - 1) warp_arrive(bar(kEmptyQK));
                sums[((R ? kColIn : kRowIn) + j) * Q] = (in2.x + in2.y) * e;
                if (R) {  // ---- dx, over dy in its place
                    const int h = d.g * (a.s.H / a.s.G) + v / a.tiles, tile = v % a.tiles;
                    const float D = a.s.D ? par(a.s.D, a.s.p_bf16, h) : 0.0f;
                    bar_wait(bar(kFullU0 + st), ring, failed);
                    {  // <G, S>, while dx is being multiplied
                        const uint16_t *S = a.states + ((static_cast<int64_t>(d.slot) * a.pairs + d.g * a.pairs_per_group + v / 2) * 3 * Q + v % 2 * 64) * NW + tid * 8;
                        const unsigned char *G = sv + kTile;
                        uint4 s[NB][3];
#pragma unroll
                        for (int b = 0; b < NB; ++b)
#pragma unroll
                            for (int part = 0; part < 3; ++part) s[b][part] = __ldcs(reinterpret_cast<const uint4 *>(S + part * Q * NW + b * 4096));
                        float dot = 0.0f;
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            const int i = b * 512 + tid, row = i / (8 * NB), c8 = i % (8 * NB);
                            const unsigned char *at = G + c8 / 8 * (kTile / 2) + row * 128 + (((c8 ^ row) & 7) << 4);
                            const uint4 g0 = *reinterpret_cast<const uint4 *>(at), g1 = *reinterpret_cast<const uint4 *>(at + kTile),
                                        g2 = *reinterpret_cast<const uint4 *>(at + 2 * kTile);
                            const auto add = [&](uint32_t s0, uint32_t s1, uint32_t s2, uint32_t h0, uint32_t h1, uint32_t h2) {
                                const float2 u = __fadd2_rn(bf2_to_f2(s0), __fadd2_rn(bf2_to_f2(s1), bf2_to_f2(s2)));
                                const float2 w = __fadd2_rn(bf2_to_f2(h0), __fadd2_rn(bf2_to_f2(h1), bf2_to_f2(h2)));
                                dot = fmaf(u.x, w.x, fmaf(u.y, w.y, dot));
                            };
                            add(s[b][0].x, s[b][1].x, s[b][2].x, g0.x, g1.x, g2.x);
                            add(s[b][0].y, s[b][1].y, s[b][2].y, g0.y, g1.y, g2.y);
                            add(s[b][0].z, s[b][1].z, s[b][2].z, g0.z, g1.z, g2.z);
                            add(s[b][0].w, s[b][1].w, s[b][2].w, g0.w, g1.w, g2.w);
                        }
#pragma unroll
                        for (int j2 = 16; j2; j2 /= 2) dot += __shfl_xor_sync(kFull, dot, j2);
                        if (lane == 0) sums[kDot * Q - i0 + warp] = dot;
                    }
                    bar_wait(bar(kDxFull), ph, failed);
                    tc_fence_after();
                    uint32_t x1[16], x2[16];
                    tmem_ld16(tmem + lanes + kColE + j * 16, x1);
                    tmem_ld16(tmem + lanes + kColE + 64 + j * 16, x2);
                    tmem_wait_ld();
                    tc_fence_before();
                    warp_arrive(bar(kDxRead));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint4 *place = reinterpret_cast<uint4 *>(sv + i0 * 128 + (((j * 2 + i) ^ (i0 & 7)) << 4));
                        const uint4 g = *place;
                        const uint32_t gs[4] = {g.x, g.y, g.z, g.w};
                        uint32_t o[4];
#pragma unroll
                        for (int c2 = 0; c2 < 4; ++c2) {
                            const int c = i * 8 + c2 * 2;
                            float2 x = __fmul2_rn(make_float2(dti, dti), make_float2(__uint_as_float(x1[c]), __uint_as_float(x1[c + 1])));
                            x = __ffma2_rn(make_float2(scale, scale), make_float2(__uint_as_float(x2[c]), __uint_as_float(x2[c + 1])), x);
                            x = __ffma2_rn(make_float2(D, D), bf2_to_f2(gs[c2]), x);
                            o[c2] = dead ? 0u : f2_to_bf2(x);
                        }
                        *place = make_uint4(o[0], o[1], o[2], o[3]);
                        if (!whole && i0 < len && (j * 2 + i) * 8 < a.s.P - tile * 64)  // a chunk that ends early: its rows alone
                            *reinterpret_cast<uint4 *>(a.s.dx + (static_cast<int64_t>(d.row) + i0) * a.s.dx_rs + h * a.s.P + tile * 64 + (j * 2 + i) * 8) = *place;
                    }
                    fence_async();
                    warp_arrive(bar(kDxWritten0 + st));
                }
            }
            // ---- dC (dB), from the registers: Q's place is the next chunk's already
            bar_wait(bar(kWUsed), (k - 1) & 1, failed);
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                uint32_t u[16];
                const int c0 = j * kC8 + b * 2;
                tmem_ld16(tmem + lanes + kColAcc + c0 * 8, u);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t o[4];
#pragma unroll
                    for (int c2 = 0; c2 < 4; ++c2) {
                        const int c = i * 4 + c2;
                        o[c2] = dead ? 0u : f2_to_bf2(__fadd2_rn(out[b * 8 + c], make_float2(__uint_as_float(u[2 * c]), __uint_as_float(u[2 * c + 1]))));
                    }
                    const uint4 val = make_uint4(o[0], o[1], o[2], o[3]);
                    if (i0 < len && (c0 + i) * 8 < a.s.N)
                        *reinterpret_cast<uint4 *>((R ? a.s.dB + (static_cast<int64_t>(d.row) + i0) * a.s.db_rs : a.s.dC + (static_cast<int64_t>(d.row) + i0) * a.s.dc_rs) +
                                                   d.g * a.s.N + (c0 + i) * 8) = val;
                }
            }
            tc_fence_before();
            warp_arrive(bar(kAccRead));
        }
    }
    tc_fence_before();
    __syncthreads();
    if (*failed) {
        if (tid == 0) {
            bar_drain(bar(kFullU0), 2, wait->started[0]);
            bar_drain(bar(kFullQK), 1, wait->started[1]);
            bar_drain(bar(kWUsed), 1, wait->started[2]);
        }
        __syncthreads();
    }
    tc_fence_after();
    if (warp == kMmaWarp) tmem_free(tmem, 512);
    if (tid == 0 && *failed) *a.status = 1, report_given_up(a.waits);
}

// ddt of a chunk and head, and its share of dA, dD, ddt_bias, from the sums: a thread per token.
__global__ void __launch_bounds__(Q) finish_kernel(const BwdTcArgs a, float *part) {
    __shared__ float s_w[6][4];
    grid_dependents_launch();
    const int h = blockIdx.y, t = threadIdx.x, warp = t / 32, lane = t % 32;
    const int64_t slot = blockIdx.x;
    const Chunk c = scan_chunk(a.s, slot, Q);
    grid_dependency_wait();
    if (c.len == 0 || scan_padded(a.s, c.n)) {
        if (t < 3) part[(slot * a.s.H + h) * 3 + t] = 0.0f;
        if (t < c.len) {
            const int64_t at = (c.row + t) * a.s.ddt_rs + h;
            if (a.s.dt_bf16) static_cast<uint16_t *>(a.s.ddt)[at] = 0; else static_cast<float *>(a.s.ddt)[at] = 0.0f;
        }
        return;
    }
    const int rep = a.s.H / a.s.G, g = h / rep;
    const float A = par(a.s.A, a.s.p_bf16, h);
    float slope = 0.0f, dt = 0.0f, dD = 0.0f, diag = 0.0f, gs = 0.0f;
    float row_own = 0.0f, row_off = 0.0f, row_in = 0.0f, col_own = 0.0f, col_off = 0.0f, col_in = 0.0f;
    if (t < c.len) dt = scan_dt(a.s, c.row + t, h, a.s.dt_bias ? par(a.s.dt_bias, a.s.p_bf16, h) : 0.0f, &slope);
    for (int tile = 0; tile < a.tiles; ++tile) {
        const int v = h % rep * a.tiles + tile;
        const float *s = a.sums + (slot * a.heads + g * rep * a.tiles + v) * kPlanes * Q + t;
        if (t < c.len) {
            row_own += s[kRowDiag * Q];
            col_own += s[kColDiag * Q];
            for (int j = 0; j < 3; ++j) {  // the other blocks: before the row's forward, after it reverse
                if (j < warp) row_off += s[(kRowOff + j) * Q];
                if (j >= warp) col_off += s[(kColOff + j) * Q];
            }
            row_in += (s[kRowIn * Q] + s[(kRowIn + 1) * Q]) + (s[(kRowIn + 2) * Q] + s[(kRowIn + 3) * Q]);
            col_in += (s[kColIn * Q] + s[(kColIn + 1) * Q]) + (s[(kColIn + 2) * Q] + s[(kColIn + 3) * Q]);
            dD += s[kDiag * Q];
            diag += s[kDiagZ * Q];
        }
        if (t < 16) gs += s[kDot * Q];
    }
    // Sums within the block of 32: over the tokens from t on (own, off, in), over those before t.
    float own = row_own - dt * col_own, off = row_off, in = row_in, off_c = dt * col_off, in_c = dt * col_in, all = dt * A * kLog2e;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const float l0 = __shfl_down_sync(kFull, own, d), l1 = __shfl_down_sync(kFull, off, d), l2 = __shfl_down_sync(kFull, in, d);
        const float e0 = __shfl_up_sync(kFull, off_c, d), e1 = __shfl_up_sync(kFull, in_c, d);
        if (lane + d < 32) own += l0, off += l1, in += l2;
        if (lane >= d) off_c += e0, in_c += e1;
        all += __shfl_xor_sync(kFull, all, d);
        gs += __shfl_xor_sync(kFull, gs, d);
    }
    if (lane == 0) s_w[0][warp] = off, s_w[1][warp] = in, s_w[4][warp] = all, s_w[5][warp] = gs;
    if (lane == 31) s_w[2][warp] = off_c, s_w[3][warp] = in_c;
    __syncthreads();
    off_c = __shfl_up_sync(kFull, off_c, 1);
    in_c = __shfl_up_sync(kFull, in_c, 1);
    if (lane == 0) off_c = in_c = 0.0f;
    float end = 0.0f;
    for (int w = 0; w < 4; ++w) {
        if (w > warp) in += s_w[1][w];
        if (w < warp) in_c += s_w[3][w];
        end += s_w[4][w];
    }
    // pairs of an earlier and a later block: what the first gives to all but this one, and the last gets from all but this one
    const float across = warp == 1 ? s_w[2][0] - s_w[0][1] : warp == 2 ? s_w[0][3] - s_w[2][2] : 0.0f;
    gs = (s_w[5][0] + s_w[5][1]) + (s_w[5][2] + s_w[5][3]);
    const float through = own + (off + off_c) + across + (in + in_c) + ex2_approx(end) * gs;
    const float raw = (diag + col_own + col_off + col_in + A * through) * slope;
    float dA = dt * through, db = 0.0f;
    if (t < c.len) {
        const int64_t at = (c.row + t) * a.s.ddt_rs + h;
        if (a.s.dt_bf16) static_cast<uint16_t *>(a.s.ddt)[at] = f_to_bf(raw); else static_cast<float *>(a.s.ddt)[at] = raw;
        db = raw;
    } else {
        dA = 0.0f;
    }
#pragma unroll
    for (int d = 16; d; d /= 2) {
        dA += __shfl_xor_sync(kFull, dA, d);
        dD += __shfl_xor_sync(kFull, dD, d);
        db += __shfl_xor_sync(kFull, db, d);
    }
    __syncthreads();
    if (lane == 0) s_w[0][warp] = dA, s_w[1][warp] = dD, s_w[2][warp] = db;
    __syncthreads();
    if (t < 3) part[(slot * a.s.H + h) * 3 + t] = (s_w[t][0] + s_w[t][1]) + (s_w[t][2] + s_w[t][3]);
}

template <int NB, bool R>
cudaError_t launch_chunks(const BwdTcArgs &a, cudaStream_t st) {
    const auto kernel = chunk_kernel<NB, R>;
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem)) return e;
    return launch_behind(kernel, dim3(static_cast<unsigned>(std::min<int64_t>(a.slots * a.s.G, 152))), kThreads, kSmem, false, st, a);
}

}  // namespace

ScanTcBwdPlan scan_tc_bwd_plan(int64_t rows, int n_seqs, int H, int P, int G, int N) {
    ScanTcBwdPlan p = {};
    p.walk = scan_tc_plan(rows, n_seqs, H, P, G, N);
    if (!p.walk.ok || rows <= 0 || n_seqs <= 0) return p;
    p.slots = scan_chunk_slots(rows, n_seqs, Q);
    p.heads = H * p.walk.tiles;
    p.ok = p.slots * p.walk.pairs * 3 * Q <= INT32_MAX && p.slots * G <= INT32_MAX;  // rows of the stores, tasks
    const size_t store = static_cast<size_t>(p.slots) * p.walk.pairs * 3 * Q * 64 * p.walk.nb * 2;
    p.s_store = round_up(p.walk.bytes, kAlignWs);
    p.g_store = p.s_store + store;
    p.sums = p.g_store + store;
    p.part = p.sums + static_cast<size_t>(p.slots) * p.heads * kPlanes * Q * 4;
    p.bytes = p.part + round_up(static_cast<size_t>(p.slots) * H * 3 * 4, kAlignWs);
    return p;
}

cudaError_t launch_scan_tc_bwd(const ScanArgs &s, const ScanTcBwdPlan &plan, unsigned char *ws, float *dA, float *dD, float *dbias,
                               int *launches, cudaStream_t st) {
    uint16_t *s_store = reinterpret_cast<uint16_t *>(ws + plan.s_store), *g_store = reinterpret_cast<uint16_t *>(ws + plan.g_store);
    float *part = reinterpret_cast<float *>(ws + plan.part);
    *launches = 0;
    // Either walk's store is read right behind it, while part of it is still in L2.
    if (cudaError_t e = launch_scan_tc_states(s, plan.walk, ws, false, s_store, launches, st)) return e;
    BwdTcArgs a = {};
    a.s = s;
    a.pairs = plan.walk.pairs, a.pairs_per_group = plan.walk.pairs_per_group, a.tiles = plan.walk.tiles, a.heads = plan.heads;
    a.slots = plan.slots;
    a.sums = reinterpret_cast<float *>(ws + plan.sums);
    a.status = reinterpret_cast<int *>(ws + plan.walk.status);
    a.waits = current_waits();
    const int nw = 64 * plan.walk.nb;
    const int64_t store_rows = plan.slots * plan.walk.pairs * 3 * Q;
    CUtensorMap x, dy, b, c, es, eg;
    if (!make_scan_map(&x, s.x, s.P, s.H, s.rows, s.x_rs, Q) || !make_scan_map(&dy, s.dy, s.P, s.H, s.rows, s.dy_rs, Q) ||
        !make_scan_map(&b, s.B, s.N, s.G, s.rows, s.b_rs, Q) || !make_scan_map(&c, s.C, s.N, s.G, s.rows, s.c_rs, Q) ||
        !make_scan_map(&es, s_store, nw, 1, store_rows, nw, 64) || !make_scan_map(&eg, g_store, nw, 1, store_rows, nw, 64) ||
        !make_scan_map(&a.mdx, s.dx, s.P, s.H, s.rows, s.dx_rs, Q))
        return cudaErrorInvalidValue;
    a.mq = c, a.mk = b, a.mu = dy, a.mv = x, a.me = es;
    if (cudaError_t e = plan.walk.nb == 1 ? launch_chunks<1, false>(a, st) : launch_chunks<2, false>(a, st)) return e;
    if (cudaError_t e = launch_scan_tc_states(s, plan.walk, ws, true, g_store, launches, st)) return e;
    a.mq = b, a.mk = c, a.mu = x, a.mv = dy, a.me = eg, a.states = s_store;
    if (cudaError_t e = plan.walk.nb == 1 ? launch_chunks<1, true>(a, st) : launch_chunks<2, true>(a, st)) return e;
    if (cudaError_t e = launch_behind(finish_kernel, dim3(static_cast<unsigned>(plan.slots), s.H), Q, 0, false, st, a, part)) return e;
    *launches += 4;
    return launch_scan_sums(part, plan.slots, s.H, dA, dD, dbias, false, st);
}

}  // namespace ccc
