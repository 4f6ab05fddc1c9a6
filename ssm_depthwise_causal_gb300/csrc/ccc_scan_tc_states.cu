// ccc_scan_tc_states.cu -- the states of the selective scan alone, on the
// tensor cores: for the forward, what a cut leaves open (the walk of
// ccc_scan_tc.cu then starts from it); for the backward, the state before each
// chunk and, in reverse with x, B replaced by dy, C, the state gradient after
// each chunk.
//
//     S' = 2^a_end S + (w v)^T K,  w_s = dt_s 2^(a_end - a_s); reverse w_t = 2^a_t
// (exponents in powers of two, a the running sum of dt A log2 e in the chunk.)
// w v is rounded to PARTS BF16 parts and multiplied by K, which is exact; the sum and
// S are FP32.  Three parts are all 24 bits: what leaves here for the backward is as good
// as 32-bit arithmetic.  The forward's tails have two, 16 bits, as its walk has.
//
// A CTA has a pair of heads (128 rows of S): four warps make w v, transposed by
// ldmatrix into TMEM, two chunks deep; eight hold S in registers and add the
// products to it; two compute the steps, one finds and loads the chunks, one
// issues the products.  The products of a chunk (24 steps of 128 x 128 x 16, 1536
// cycles) and the addition follow each other; all else overlaps.  A stored state
// goes out by TMA as three BF16 parts, 96 KB a chunk and pair.
// 16384 tokens, 32 heads of 64, N = 128: 38 us without the store (3200 cycles a
// chunk and pair, the time of w v: its four warps split 128 x 128 values three
// ways), 62 with it (0.2 GB written: 3.2 TB/s).  Both steps' warps twice, 576
// threads with 96 registers: 40 and 70.
#include <algorithm>

#include "ccc_checks.h"
#include "ccc_scan_tc.cuh"

namespace ccc {

namespace {

constexpr int Q = kTcChunk;
constexpr int kThreads = 512;
constexpr int kTmaWarp = 12, kMmaWarp = 13, kStepWarp = 14;  // 0-3: w v, 4-11: the state
constexpr uint32_t kOffK = 0, kOffV = 4 * kTile, kOffOut = 8 * kTile, kOffArr = 14 * kTile;
struct Arrays {
    float w[2][Q], total[2][4];
};
using Desc = ChunkDesc;
constexpr int kDescs = 8, kAhead = 3;  // published ahead of the loads; a slot is written again when every warp is past it
constexpr uint32_t kOffDesc = kOffArr + 2 * sizeof(Arrays);
constexpr uint32_t kOffBar = kOffDesc + kDescs * sizeof(Desc);
constexpr uint32_t kSmem = kOffBar + 512;
constexpr uint32_t kColX = 0, kColsX = 192, kColD = 384;  // w v twice; the products

// A waiter looks at a phase's parity alone: never two phases late, nor one early (ccc_scan_tc.cu).
enum Bar {
    kDesc0,
    kFullK0 = kDesc0 + kDescs, kFullK1, kFullV0, kFullV1, kEmptyK0, kEmptyK1, kXFree0, kXFree1, kDFull, kOutFree,
    kEmptyV0, kEmptyV1, kXReady0, kXReady1, kDRead, kClean, kOutWritten,
    kSteps0, kSteps1, kArrays0, kArrays1,
    kBars
};
static_assert(kSmem <= 232448 && 8 * kBars + sizeof(WaitState) <= 512, "shared memory of a CTA");

template <int NB, bool REV, int PARTS>
__global__ void __launch_bounds__(kThreads, 1) states_kernel(const __grid_constant__ ScanTcArgs a) {
    extern __shared__ __align__(1024) unsigned char smem[];
    constexpr int NW = 64 * NB;
    const uint32_t base = smem_addr(smem);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const auto bar = [&](int b) { return base + kOffBar + 8 * b; };
    WaitState *const wait = reinterpret_cast<WaitState *>(smem + kOffBar + 8 * kBars);
    volatile int *failed = &wait->failed;
    Arrays *arrays = reinterpret_cast<Arrays *>(smem + kOffArr);
    if (tid == 0) {
        for (int b = 0; b < kEmptyV0; ++b) bar_init(bar(b), 1);
        for (int b = kEmptyV0; b < kDRead; ++b) bar_init(bar(b), 4);  // the warps of w v
        bar_init(bar(kClean), 4);
        for (int b : {kDRead, kOutWritten}) bar_init(bar(b), 8);        // the state's
        for (int b : {kSteps0, kSteps1}) bar_init(bar(b), 2);
        for (int b : {kArrays0, kArrays1}) bar_init(bar(b), 12);
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

    if (warp >= kTmaWarp) {
        if (warp == kTmaWarp) {  // --------------------------- chunks and loads
            if (lane == 0) {
                tma_prefetch_map(&a.mv);
                tma_prefetch_map(&a.mk);
            }
            Walk<REV> wk;
            if (a.tail) wk.init_tail(a.s, a.pairs, blockIdx.x, gridDim.x);
            else wk.init(a.s, a.pairs, blockIdx.x, gridDim.x);
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
                prefetch_steps(a, wk.row, wk.valid, wk.pair);
                wk.next(a.s);
            };
            for (int i = 0; i < kAhead; ++i) publish();
            int k = 0, loaded_k = 0, loaded_v = 0;
            for (;;) {
                const int st = k & 1;
                const Desc &d = reinterpret_cast<const Desc *>(smem + kOffDesc)[k % kDescs];
                const int row = d.row, pair = d.pair;
                if (__any_sync(kFull, *failed || !(d.flags & kMore))) break;
                const uint32_t free = ((k >> 1) & 1) ^ 1;
                publish();  // well ahead of the loads: the steps start from it
                if (lane == 0) {
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
                    bar_wait(bar(kEmptyK0 + st), free, failed);
                    if (!*failed) {
                        ++loaded_k;
                        bar_expect(bar(kFullK0 + st), NB * kTile);
#pragma unroll
                        for (int b = 0; b < NB; ++b)
                            tma_load(base + kOffK + (2 * st + b) * kTile, &a.mk, bar(kFullK0 + st), b * 64, pair / a.pairs_per_group, row);
                    }
                }
                __syncwarp();
                ++k;
            }
            if (lane == 0) wait->started[0] = loaded_k, wait->started[1] = loaded_v;
        } else if (warp == kMmaWarp) {  // ---------------------------- products
            int k = 0;
            for (;; ++k) {
                const Desc &d = desc(k);
                if (__any_sync(kFull, *failed || !(d.flags & kMore))) break;
                const int st = k & 1;
                const uint32_t ring = (k >> 1) & 1, sk = base + kOffK + 2 * st * kTile;
                bar_wait(bar(kFullK0 + st), ring, failed);
                bar_wait(bar(kXReady0 + st), ring, failed);
                if (k > 0) bar_wait(bar(kDRead), (k - 1) & 1, failed);
                tc_fence_after();
                if (tc_elect()) {
#pragma unroll
                    for (int i = 0; i < 8 * PARTS; ++i)
                            tc_mma_ts(tmem + kColD, tmem + kColX + st * kColsX + i * 8, tc_desc(sk + (i % 8) * 2048, kTile, 1024),
                                      tc_idesc(NW, false, true), i > 0);
                    tc_commit(bar(kDFull));
                    tc_commit(bar(kXFree0 + st));
                    tc_commit(bar(kEmptyK0 + st));
                }
                __syncwarp();
            }
            if (lane == 0) wait->started[2] = k;
        } else {  // ------------------------------------------ steps and decays
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
                float dt[4], v[4], p[4], P[4], to_end[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    dt[i] = mine.ok && 32 * i + lane < len ? step_of(dt_value(a.s, raw[i]) + bias, a.s.softplus) : 0.0f;
                    v[i] = p[i] = dt[i] * A2;
                }
                block_sums(p, P);
                if (!REV) block_after(v, p, P, to_end);
                bar_wait(bar(kArrays0 + (k & 1)), ((k >> 1) & 1) ^ 1, failed);
                Arrays &r = arrays[k & 1];
                // the blocks before (reverse) or after a block, with the distance inside it
                r.w[hd][lane] = REV ? ex2_approx(p[0]) : dt[0] * ex2_approx(to_end[0] + (P[1] + (P[2] + P[3])));
                r.w[hd][32 + lane] = REV ? ex2_approx(P[0] + p[1]) : dt[1] * ex2_approx(to_end[1] + (P[2] + P[3]));
                r.w[hd][64 + lane] = REV ? ex2_approx((P[0] + P[1]) + p[2]) : dt[2] * ex2_approx(to_end[2] + P[3]);
                r.w[hd][96 + lane] = REV ? ex2_approx((P[0] + P[1] + P[2]) + p[3]) : dt[3] * ex2_approx(to_end[3]);
                if (lane < 4) r.total[hd][lane] = lane == 0 ? P[0] : lane == 1 ? P[1] : lane == 2 ? P[2] : P[3];
                warp_arrive(bar(kSteps0 + (k & 1)));
#pragma unroll
                for (int i = 0; i < 4; ++i) raw[i] = next[i];  // (waits for the loads)
            }
        }
    } else if (warp < 4) {  // ----------------------------------------- w v
        const int q = warp;  // 32 channels of the pair
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
                for (int i = len * 8 + tid; i < Q * 8; i += 128) {
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
            bar_wait(bar(kXFree0 + st), ring ^ 1, failed);
            tc_fence_after();
            const float *w = arrays[st].w[q / 2];
            // this lane's row of the four blocks: token lane % 8, channel block lane / 8 % 2, token block lane / 16
            const uint32_t rows = base + kOffV + (2 * st + q / 2) * kTile + (lane / 16 * 8 + lane % 8) * 128;
#pragma unroll 1
            for (int hf = 0; hf < 8; ++hf) {  // 16 channels, 32 tokens
                const uint32_t chunk = ((q % 2 * 4 + hf / 4 * 2 + lane / 8 % 2) ^ (lane & 7)) << 4;
                uint32_t part[PARTS][8];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t m[4];
                    const int s = hf % 4 * 32 + i * 16;
                    ldmatrix_trans(rows + s * 128 + chunk, m);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float2 v = __fmul2_rn(bf2_to_f2(m[j]), *reinterpret_cast<const float2 *>(w + s + j / 2 * 8 + lane % 4 * 2));
#pragma unroll
                        for (int e = 0; e < PARTS; ++e) {
                            part[e][4 * i + j] = f2_to_bf2(v);
                            v = __ffma2_rn(bf2_to_f2(part[e][4 * i + j]), make_float2(-1.0f, -1.0f), v);
                        }
                    }
                }
                const uint32_t at = tmem + lanes + (static_cast<uint32_t>(hf / 4 * 16) << 16) + kColX + st * kColsX + hf % 4 * 16;
#pragma unroll
                for (int e = 0; e < PARTS; ++e) tmem_st_16x128b_x4(at + e * 64, part[e]);
            }
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(bar(kXReady0 + st));
            warp_arrive(bar(kEmptyV0 + st));
            warp_arrive(bar(kArrays0 + st));
        }
    } else {  // ------------------------------------------------------- the state
        const int wg = warp / 4 - 1, q = warp % 4, t = tid % 128;
        const int lh = t / 64, lp = t % 64, c0 = wg * 32 * NB;  // the thread's row, and its columns' start
        const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
        const int64_t open = (static_cast<int64_t>(blockIdx.x) * Q + t) * NW + c0;
        float S[NB][32], total_keep = 1.0f;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 32; ++i) S[b][i] = 0.0f;
        bool entered = false;
        int pair = -1;
        Head state{};
        for (int k = 0;; ++k) {
            const Desc &d = desc(k);
            if (__any_sync(kFull, *failed || !(d.flags & kMore))) break;
            const int st = k & 1, flags = d.flags, n = d.n;
            const uint32_t ring = (k >> 1) & 1;
            const int64_t place = (static_cast<int64_t>(d.row) / Q + n) * a.pairs + d.pair;
            if (d.pair != pair) {
                pair = d.pair;
                state = head_of(a, pair, lh);
            }
            if (flags & kFresh) {
                if (flags & kEnters) {
                    const float *from = nullptr;
                    if (!(flags & kDead)) {
                        if (REV) from = a.s.d_final ? a.s.d_final + static_cast<int64_t>(n) * a.s.H * a.s.P * a.s.N : nullptr;
                        else from = scan_initial(a.s, n);
                    }
                    entered = true;
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        load_state(a, from, state, lp, c0 + b * 32, S[b]);
                        if (a.tail && a.staged) copy_out(a.staged + open + b * 32, S[b]);
                    }
                } else if (!a.tail) {
                    const int carry = carry_from<REV>(a);
#pragma unroll
                    for (int b = 0; b < NB; ++b) carry_in<REV>(a, carry, t, lh, NW, c0 + b * 32, S[b]);
                }
            }
            if (a.store) {  // three BF16 parts, over the chunk before's, which the stores have read
                if (k > 0) bar_wait(bar(kOutFree), (k - 1) & 1, failed);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const int at = c0 / 8 + b * 4;  // first 16-byte chunk of the row's NW values
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float2 v[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[j] = make_float2(S[b][8 * i + 2 * j], S[b][8 * i + 2 * j + 1]);
#pragma unroll
                        for (int e = 0; e < 3; ++e) {
                            uint32_t p[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                p[j] = f2_to_bf2(v[j]);
                                v[j] = __ffma2_rn(bf2_to_f2(p[j]), make_float2(-1.0f, -1.0f), v[j]);
                            }
                            *reinterpret_cast<uint4 *>(smem + kOffOut + (e * NB + at / 8) * kTile + t * 128 + (((at + i) % 8 ^ (t & 7)) << 4)) =
                                make_uint4(p[0], p[1], p[2], p[3]);
                        }
                    }
                }
                fence_async();
                warp_arrive(bar(kOutWritten));
                if (tid == 128) {
                    bar_wait(bar(kOutWritten), k & 1, failed);
#pragma unroll
                    for (int e = 0; e < 3; ++e)
#pragma unroll
                        for (int b = 0; b < NB; ++b)
                            tma_store(&a.ms, base + kOffOut + (e * NB + b) * kTile, b * 64, 0, static_cast<int>((place * 3 + e) * Q));
                }
                __syncwarp();
            }
            bar_wait(bar(kSteps0 + st), ring, failed);
            const float *total = arrays[st].total[lh];
            const float keep = ex2_approx(total[0] + total[1] + (total[2] + total[3]));
            warp_arrive(bar(kArrays0 + st));
            total_keep *= keep;
            bar_wait(bar(kDFull), k & 1, failed);
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                uint32_t ds[32];
                tmem_ld32(tmem + lanes + kColD + c0 + b * 32, ds);
                tmem_wait_ld();
                if (b + 1 == NB) {
                    tc_fence_before();
                    warp_arrive(bar(kDRead));
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) S[b][i] = fmaf(keep, S[b][i], __uint_as_float(ds[i]));
            }
            if (REV && !a.tail && (flags & kLeaves) && !(flags & kDead) && a.s.d_initial)
#pragma unroll
                for (int b = 0; b < NB; ++b)
                    store_state(a, a.s.d_initial + static_cast<int64_t>(n) * a.s.H * a.s.P * a.s.N, state, lp, c0 + b * 32, S[b]);
            if (a.store) {
                if (tid == 128) {
                    bulk_wait_read();
                    bar_arrive(bar(kOutFree));
                }
                __syncwarp();
            }
        }
        if (a.tail) {
#pragma unroll
            for (int b = 0; b < NB; ++b) copy_out(a.local + open + b * 32, S[b]);
            if (wg == 0 && lp == 0) a.keep[blockIdx.x * 2 + lh] = total_keep;
            if (tid == 128) a.flag[blockIdx.x] = entered;
        } else if (tid == 128) {
            bulk_wait_all();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (*failed) {
        if (tid == 0) {
            bar_drain(bar(kFullK0), 2, wait->started[0]);
            bar_drain(bar(kFullV0), 2, wait->started[1]);
            bar_drain(bar(kEmptyK0), 2, wait->started[2]);
        }
        __syncthreads();
    }
    tc_fence_after();
    if (warp == kMmaWarp) tmem_free(tmem, 512);
    if (tid == 0 && *failed) *a.status = 1, report_given_up(a.waits);
}

__global__ void edge_states_kernel(const ScanArgs a, float *to, bool gradient) {
    grid_dependents_launch();
    grid_dependency_wait();
    const int n = blockIdx.x;
    const Seq s = scan_seq(a, n);
    const bool dead = scan_padded(a, n);
    if (s.end > s.begin && !dead) return;
    const int64_t hpn = static_cast<int64_t>(a.H) * a.P * a.N;
    const float *from = gradient ? scan_edge_gradient(a, n, dead) : dead ? nullptr : scan_initial(a, n);
    for (int64_t i = threadIdx.x; i < hpn; i += blockDim.x) to[n * hpn + i] = from ? from[i] : 0.0f;
}

cudaError_t launch_states(const ScanTcArgs &a, const ScanTcPlan &plan, bool reverse, bool fine, bool first, cudaStream_t st) {
    const auto kernel = plan.nb == 1 ? (reverse ? states_kernel<1, true, 3> : fine ? states_kernel<1, false, 3> : states_kernel<1, false, 2>)
                                     : (reverse ? states_kernel<2, true, 3> : fine ? states_kernel<2, false, 3> : states_kernel<2, false, 2>);
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem)) return e;
    return launch_behind(kernel, dim3(plan.parts), kThreads, kSmem, first, st, a);
}

}  // namespace

cudaError_t launch_edge_states(const ScanArgs &a, float *to, bool gradient, cudaStream_t st) {
    edge_states_kernel<<<a.n_seqs, 256, 0, st>>>(a, to, gradient);
    return cudaGetLastError();
}

cudaError_t launch_scan_tc_tails(ScanTcArgs a, const ScanTcPlan &plan, bool reverse, bool fine, bool first, cudaStream_t st) {
    a.tail = 1;
    a.store = nullptr;
    return launch_states(a, plan, reverse, fine, first, st);
}

cudaError_t launch_scan_tc_states(const ScanArgs &s, const ScanTcPlan &plan, unsigned char *ws, bool reverse, uint16_t *store,
                                  int *launches, cudaStream_t st) {
    ScanTcArgs a = {};
    a.s = s;
    a.pairs = plan.pairs, a.pairs_per_group = plan.pairs_per_group, a.tiles = plan.tiles;
    a.status = reinterpret_cast<int *>(ws + plan.status);
    a.waits = current_waits();
    a.local = reinterpret_cast<float *>(ws + plan.local);
    a.keep = reinterpret_cast<float *>(ws + plan.keep);
    a.flag = reinterpret_cast<int *>(ws + plan.flag);
    const int nw = 64 * plan.nb;
    if (!make_scan_map(&a.mv, reverse ? s.dy : s.x, s.P, s.H, s.rows, reverse ? s.dy_rs : s.x_rs, Q) ||
        !make_scan_map(&a.mk, reverse ? s.C : s.B, s.N, s.G, s.rows, reverse ? s.c_rs : s.b_rs, Q) ||
        !make_scan_map(&a.ms, store, nw, 1, scan_chunk_slots(s.rows, s.n_seqs, Q) * plan.pairs * 3 * Q, nw, Q))
        return cudaErrorInvalidValue;
    if (reverse && s.d_initial) {
        if (cudaError_t e = launch_edge_states(s, s.d_initial, true, st)) return e;
        ++*launches;
    }
    if (plan.cuts) {
        if (cudaError_t e = launch_scan_tc_tails(a, plan, reverse, true, *launches == 0, st)) return e;
        ++*launches;
    }
    a.store = store;
    ++*launches;
    return launch_states(a, plan, reverse, true, *launches == 1, st);
}

}  // namespace ccc
