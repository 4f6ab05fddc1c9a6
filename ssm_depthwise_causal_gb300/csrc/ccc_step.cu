// ccc_step.cu -- the decode step of an SSM mixer in one launch: the short
// causal convolution (+ SiLU) of a few new tokens per request from the
// conv_state pool, the selective-scan update of the ssm_state pool with its
// results, and both pools' update for the next step.
//
// Per new token and head, in FP32 (the convolution's results stay in 32
// bits between the two):
//     u = act(bias + sum_k w_k line[j + k]),  u = [x | B | C]
//     h = exp(dt A) h + dt x B^T,   y = h C + D x.
// What it cannot do without is the state, read and written once (P N floats
// a head): memory bound for a batch, latency bound for one request.
//
// A cluster of CTAs takes one (request, group); each CTA some of the group's
// heads, whose P rows of N state values follow each other in memory: they come
// into shared memory by bulk copies of 32 KB, two in flight a CTA and three CTAs
// an SM, while the convolution is computed.  A row lies in LR lanes of a warp, NV
// float4 each.  A CTA computes its heads' x channels and an equal share of the
// group's B and C channels, whose results the others fetch from its shared
// memory, so that every channel's history is read and written by one thread.
// (Every CTA computing all of B and C, the history written behind a second
// barrier: 370 us for the 256-request step; the state loaded into registers in
// place of the copies: 392; CTAs that stay and take one request after another:
// 420.)
#include <cooperative_groups.h>

#include <algorithm>
#include <climits>

#include "ccc.h"
#include "ccc_checks.h"
#include "ccc_scan_device.cuh"
#include "ccc_tc.cuh"

namespace ccc {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kStages = 2;  // pieces of the state in shared memory
constexpr int kTokens = 4;  // tokens whose convolution results are staged at a time

struct StepArgs {
    ScanArgs s;  // dt, parameters, sizes, cu, cache, pool (position 0), out
    const uint16_t *xbc;
    int64_t xs;
    const void *w, *b;
    int w_bf16, b_kind, width, act;
    uint16_t *conv;
    int state_len;
    int64_t st_slot, st_c, st_l;
    int held;         // positions of the ssm_state pool
    int64_t st_pos;
    const int32_t *accepted;
    int heads_per_cta, ctas;  // of a group
    int state_at;             // where the state begins in shared memory, in floats
    Waits waits;
};

__device__ __forceinline__ float silu1(float z) {
    return z * rcp_approx(1.0f + ex2_approx(-kLog2e * z));
}

template <int LR, int NV>
__global__ void __launch_bounds__(kThreads, 3) step_kernel(const StepArgs a) {
    namespace cg = cooperative_groups;
    extern __shared__ __align__(128) float smem[];
    __shared__ uint64_t s_full[kStages];
    __shared__ WaitState s_wait;
    constexpr int kRows = 8 / NV;                       // rows of a lane in a piece
    constexpr int kPiece = kWarps * (32 / LR) * kRows;  // rows of a piece: up to 32 KB
    const ScanArgs &s = a.s;
    const int rep = s.H / s.G;
    const int n = blockIdx.x / (s.G * a.ctas), part = blockIdx.x % a.ctas, g = blockIdx.x / a.ctas % s.G;
    const int h0 = g * rep + part * a.heads_per_cta, hc = min(a.heads_per_cta, rep - part * a.heads_per_cta);
    const int xw = hc * s.P, bc = 2 * s.N;
    // B and C come first: their place is the same in every CTA
    float *bcs = smem, *xs = bcs + kTokens * bc, *ys = xs + kTokens * xw, *s_dt = ys + kTokens * xw, *s_decay = s_dt + kTokens * hc;
    float *state = smem + a.state_at;
    volatile int *const failed = &s_wait.failed;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const Seq seq = scan_seq(s, n);
    const int len = static_cast<int>(seq.end - seq.begin);
    const int slot = s.cache[n];
    if (len == 0) return;  // the same for every CTA of the cluster
    if (slot < 0 || slot >= s.n_slots) {
        for (int64_t i = tid; i < static_cast<int64_t>(len) * xw; i += kThreads)
            s.out[(seq.begin + i / xw) * s.out_rs + h0 * s.P + i % xw] = 0;
        return;
    }
    // the accepted count, clamped to the positions that both pools have: history and state are those behind the same token
    const int acc = min(max(a.accepted ? a.accepted[n] : 1, 1), min(a.state_len - a.width + 2, a.held));
    float *pool = s.pool + slot * s.st_slot + static_cast<int64_t>(h0) * s.P * s.N;
    const int pieces = (xw + kPiece - 1) / kPiece;
    // With more tokens than are staged at a time, the convolution is computed again for every piece, by every CTA of the
    // cluster as often.
    const int rounds = len > kTokens ? (a.heads_per_cta * s.P + kPiece - 1) / kPiece : pieces;
    const auto load = [&](int i) {  // piece i, by one thread
        const uint32_t bar = smem_addr(&s_full[i % kStages]);
        const uint32_t bytes = static_cast<uint32_t>(min(kPiece, xw - i * kPiece)) * s.N * 4;
        bar_expect(bar, bytes);
        bulk_load(smem_addr(state + i % kStages * kPiece * s.N), pool + (acc - 1) * a.st_pos + static_cast<int64_t>(i) * kPiece * s.N, bytes, bar);
    };
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) bar_init(smem_addr(&s_full[i]), 1);
        s_wait.failed = 0, s_wait.limit = a.waits.limit;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        for (int i = 0; i < min(kStages, pieces); ++i) load(i);
    }
    const int b0 = bc * part / a.ctas, own = xw + bc * (part + 1) / a.ctas - b0;  // this CTA's share of B and C; its channels
    const int keep = min(len + a.width - 2, a.state_len);

    const int col = lane % LR * 4, sub = lane / LR;
    int started = min(kStages, pieces);  // copies (thread 0's count)
    // A warp whose wait ran out has no state: it stores none any more, and waits no more (a phase too far ahead would pass for
    // done).  Its rows of y are undefined.  (Leaving them unwritten as well, by a look at the CTA's flag behind each piece, cost
    // the 256-request step 2 of 293 us.)
    bool here = true;
    for (int i = 0; i < rounds; ++i) {
        const int base = i * kPiece;
        float *piece = state + i % kStages * kPiece * s.N;
        for (int t0 = 0; t0 < len; t0 += kTokens) {
            const int nt = min(kTokens, len - t0);
            if (i == 0 || len > kTokens) {
                if (i > 0 || t0 > 0) {
                    if (a.ctas > 1) cg::this_cluster().sync();  // the tokens before have been used
                    else __syncthreads();
                }
                for (int e = tid; e < own; e += kThreads) {
                    const int b = b0 + e - xw;  // B or C: value b of the two
                    const int c = e < xw ? h0 * s.P + e : s.H * s.P + (b < s.N ? g * s.N + b : s.G * s.N + g * s.N + b - s.N);
                    const float bias = a.b_kind == 0 ? 0.0f : par(a.b, a.b_kind == 2, c);
                    const uint16_t *x = a.xbc + (seq.begin + t0) * a.xs + c;
                    uint16_t *past = a.conv + slot * a.st_slot + c * a.st_c;
                    uint16_t old[3];
                    float tap[4], win[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) tap[k] = k < a.width ? par(a.w, a.w_bf16, c * a.width + k) : 0.0f;
#pragma unroll
                    for (int k = 0; k < 3; ++k) {  // (past the first tokens the window is all tokens)
                        old[k] = k < a.width - 1 ? (t0 == 0 ? past[(acc - 1 + k) * a.st_l] : x[(k + 1 - a.width) * a.xs]) : uint16_t{0};
                        win[k] = bf_to_f(old[k]);
                    }
                    for (int j = 0; j < nt; ++j) {
                        const float now = bf_to_f(x[j * a.xs]);
                        win[1] = a.width == 2 ? now : win[1];
                        win[2] = a.width == 3 ? now : win[2];
                        win[3] = now;
                        float z = bias;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (k < a.width) z = fmaf(tap[k], win[k], z);
                        if (a.act) z = silu1(z);
                        if (e < xw) xs[j * xw + e] = z; else bcs[j * bc + b] = z;
#pragma unroll
                        for (int k = 0; k < 3; ++k) win[k] = win[k + 1];
                    }
                    if (t0 == 0 && (len <= kTokens || i + 1 == rounds))  // the history for the next step, behind the last read
                        for (int p = 0; p < keep; ++p)
                            past[p * a.st_l] = p < a.width - 2 ? (p == 0 ? old[1] : old[2]) : x[(p + 2 - a.width) * a.xs];
                }
                for (int e = tid; e < nt * hc; e += kThreads) {
                    const int j = e / hc, h = h0 + e % hc;
                    const float dt = scan_dt(s, seq.begin + t0 + j, h, s.dt_bias ? par(s.dt_bias, s.p_bf16, h) : 0.0f);
                    s_dt[e] = dt;
                    s_decay[e] = ex2_approx(dt * par(s.A, s.p_bf16, h) * kLog2e);
                }
                if (a.ctas > 1) {  // the other CTAs' shares
                    cg::this_cluster().sync();
                    for (int e = tid; e < nt * bc; e += kThreads) {
                        const int b = e % bc;
                        int of = min(b * a.ctas / bc, a.ctas - 1);  // the part whose share holds b
                        if (b >= bc * (of + 1) / a.ctas) ++of;
                        if (of != part) bcs[e] = cg::this_cluster().map_shared_rank(bcs, of)[e];
                    }
                }
                __syncthreads();
            }
            if (i >= pieces) continue;
            if (t0 == 0) {
                const uint32_t bar = smem_addr(&s_full[i % kStages]), parity = (i / kStages) & 1;
                here = here && __all_sync(kFull, a.waits.limit > 0 ? bar_wait(bar, parity, failed) : bar_look(bar, parity, failed));
            }
            for (int j = 0; here && j < nt; ++j) {
                const float *bj = bcs + j * bc, *xj = xs + j * xw;
                const bool kept = t0 + j < a.held, last = t0 + j + 1 == len;
                float4 bv[NV], cv[NV];
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const int k = col + v * LR * 4;
                    bv[v] = cv[v] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (k < s.N) {
                        bv[v] = *reinterpret_cast<const float4 *>(bj + k);
                        cv[v] = *reinterpret_cast<const float4 *>(bj + s.N + k);
                    }
                }
                float y[kRows];
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    const int in = (r * kWarps + warp) * (32 / LR) + sub, row = base + in;
                    y[r] = 0.0f;
                    if (row >= xw) continue;
                    const int hd = row / s.P;
                    const float decay = s_decay[j * hc + hd], xd = s_dt[j * hc + hd] * xj[row];
                    float *to = pool + (t0 + j) * a.st_pos + static_cast<int64_t>(row) * s.N + col;
#pragma unroll
                    for (int v = 0; v < NV; ++v) {
                        if (col + v * LR * 4 >= s.N) continue;
                        float4 *at = reinterpret_cast<float4 *>(piece + in * s.N + col + v * LR * 4);
                        float4 q = *at;
                        q.x = fmaf(decay, q.x, xd * bv[v].x);
                        q.y = fmaf(decay, q.y, xd * bv[v].y);
                        q.z = fmaf(decay, q.z, xd * bv[v].z);
                        q.w = fmaf(decay, q.w, xd * bv[v].w);
                        y[r] += q.x * cv[v].x + q.y * cv[v].y + q.z * cv[v].z + q.w * cv[v].w;
                        if (kept) __stcs(reinterpret_cast<float4 *>(to + v * LR * 4), q);
                        if (!last) *at = q;  // for the next token (this thread's own values)
                    }
                }
                // The rows' sums over their LR lanes: at each halving a lane passes half of its sums on and keeps the
                // rest, so that it ends with one row's.
                int mine = 0;
#pragma unroll
                for (int half = kRows / 2, mask = LR / 2; half; half /= 2, mask /= 2) {
                    const bool up = lane & mask;
#pragma unroll
                    for (int e = 0; e < half; ++e) {
                        const float send = up ? y[e] : y[e + half], stay = up ? y[e + half] : y[e];
                        y[e] = stay + __shfl_xor_sync(kFull, send, mask);
                    }
                    mine += up ? half : 0;
                }
#pragma unroll
                for (int mask = LR / 2 / kRows; mask; mask /= 2) y[0] += __shfl_xor_sync(kFull, y[0], mask);
                const int row = base + (mine * kWarps + warp) * (32 / LR) + sub;
                if (row < xw && lane % (LR / kRows) == 0) {
                    const float D = s.D ? par(s.D, s.p_bf16, h0 + row / s.P) : 0.0f;
                    ys[j * xw + row] = fmaf(D, xj[row], y[0]);
                }
            }
            __syncthreads();
            if (t0 + kTokens >= len && tid == 0 && i + kStages < pieces && here) {
                fence_async();  // the piece has been read (and written): a copy may follow
                load(i + kStages);
                ++started;
            }
            const int wide = min(base + kPiece, xw) - base;
            for (int e = tid; e < nt * wide; e += kThreads) {
                const int j = e / wide, row = base + e % wide;
                s.out[(seq.begin + t0 + j) * s.out_rs + h0 * s.P + row] = f_to_bf(ys[j * xw + row]);
            }
        }
    }
    if (a.ctas > 1) cg::this_cluster().sync();  // the others have fetched this CTA's share
    if (tid == 0 && *failed) {
        bar_drain(smem_addr(&s_full[0]), kStages, started);  // no copy may be in flight when the CTA ends
        report_given_up(a.waits);
    }
}

template <int LR, int NV>
cudaError_t launch_step(const StepArgs &a, cudaStream_t st) {
    StepArgs b = a;
    b.state_at = (kTokens * 2 * (a.s.N + a.heads_per_cta * (a.s.P + 1)) + 31) / 32 * 32;
    const size_t bytes = (static_cast<size_t>(b.state_at) + kStages * kWarps * (32 / LR) * (8 / NV) * a.s.N) * 4;
    if (cudaError_t e = cudaFuncSetAttribute(step_kernel<LR, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes))) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(a.ctas);
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = a.ctas > 1 ? 1 : 0;
    cfg.gridDim = dim3(static_cast<unsigned>(a.s.n_seqs) * a.s.G * a.ctas);
    return cudaLaunchKernelEx(&cfg, step_kernel<LR, NV>, b);
}

// Shared memory beside the state's.
int64_t staged_bytes(int64_t heads, int P, int N) { return 4 * kTokens * (2 * heads * P + 2 * N + 2 * heads); }

// Heads of a CTA: those that make a cluster of one, two, four or eight CTAs,
// the fewest that give the device two rounds of CTAs (three an SM; eight rounds:
// 310 us in place of 292 for 256 requests, 93 in place of 88 for 64 with four tokens), but 8192
// state values (32 KB) a CTA at least.  A CTA with more heads computes B and C
// once for all of them and waits less in proportion; one of few is done sooner.
int step_heads(int64_t tasks, int rep, int P, int N) {
    int heads = rep;
    for (int ctas = 2; ctas <= 8 && tasks * ((rep + heads - 1) / heads) < 152 * 3 * 2; ctas *= 2) {
        const int fewer = (rep + ctas - 1) / ctas;
        if (fewer * P * N < 8192) break;
        heads = fewer;
    }
    return std::max(heads, (rep + 7) / 8);
}

}  // namespace

}  // namespace ccc

using namespace ccc;

extern "C" int ccc_ssm_update(const void *xBC, int64_t rows, int32_t H, int32_t P, int32_t G, int32_t N_state, int64_t x_row_stride,
                              const void *weight, int32_t w_dtype, int32_t width, const void *bias, int32_t b_dtype,
                              int32_t activation, void *conv_state, int32_t n_slots, int32_t state_len,
                              int64_t st_slot, int64_t st_c, int64_t st_l,
                              const void *dt, int32_t dt_dtype, int64_t dt_row_stride, int32_t dt_softplus,
                              const void *A, const void *D, const void *dt_bias, int32_t p_dtype,
                              float *ssm_state, int32_t ssm_len, int64_t ssm_st_slot, int64_t ssm_st_pos,
                              const int32_t *cu_seqlens, int32_t N, const int32_t *cache_indices,
                              const int32_t *num_accepted, void *out, int64_t out_row_stride, void *cuda_stream) {
    if (rows < 0 || rows > INT32_MAX || N < 0 || H <= 0 || G <= 0 || H % G || P <= 0 || P % 8 || P > CCC_SCAN_MAX_HEAD ||
        N_state <= 0 || N_state % 8 || N_state > CCC_SCAN_MAX_STATE)
        return CCC_ERR_SHAPE;
    const int64_t hp = static_cast<int64_t>(H) * P, gn = static_cast<int64_t>(G) * N_state, channels = hp + 2 * gn, hpn = hp * N_state;
    if (channels > INT32_MAX / 4 || x_row_stride < channels || x_row_stride % 8 || out_row_stride < hp || out_row_stride % 8 || dt_row_stride < H)
        return CCC_ERR_SHAPE;
    if (width < 2 || width > 4 || (activation != CCC_ACT_NONE && activation != CCC_ACT_SILU)) return CCC_ERR_SHAPE;
    if (n_slots < 1 || state_len < width - 1 || ssm_len < 1) return CCC_ERR_SHAPE;
    if ((w_dtype != CCC_F32 && w_dtype != CCC_BF16) || (dt_dtype != CCC_F32 && dt_dtype != CCC_BF16) ||
        (p_dtype != CCC_F32 && p_dtype != CCC_BF16))
        return CCC_ERR_DTYPE;
    if (bias ? (b_dtype != CCC_F32 && b_dtype != CCC_BF16) : (b_dtype != CCC_NONE)) return CCC_ERR_DTYPE;
    if (!weight || !conv_state || !ssm_state || !A || !cu_seqlens || !cache_indices || (rows > 0 && (!xBC || !dt || !out))) return CCC_ERR_NULL;
    if (!state_layout_ok(n_slots, static_cast<int>(channels), state_len, st_slot, st_c, st_l)) return CCC_ERR_SHAPE;
    // [slots][positions][H][P][N] with the last three contiguous
    if (ssm_st_slot % 4 || ssm_st_pos % 4 || ssm_st_slot < 0 || ssm_st_pos < 0) return CCC_ERR_SHAPE;
    if (ssm_len > 1 && ssm_st_pos < hpn) return CCC_ERR_SHAPE;
    if (n_slots > 1 && ssm_st_slot < (ssm_len - 1) * ssm_st_pos + hpn) return CCC_ERR_SHAPE;
    const int ps = dtype_size(p_dtype);
    if (!aligned(xBC, 16) || !aligned(out, 16) || !aligned(ssm_state, 16) || !aligned(conv_state, 2) || !aligned(weight, dtype_size(w_dtype)) ||
        (bias && !aligned(bias, dtype_size(b_dtype))) || !aligned(dt, dtype_size(dt_dtype)) || !aligned(A, ps) || !aligned(D, ps) ||
        !aligned(dt_bias, ps) || !aligned(cu_seqlens, 4) || !aligned(cache_indices, 4) || !aligned(num_accepted, 4))
        return CCC_ERR_ALIGN;
    const Span made[] = {span(out, mat_bytes(rows, out_row_stride, static_cast<int>(hp))),
                         span(conv_state, static_cast<size_t>((n_slots - 1) * st_slot + (channels - 1) * st_c + (state_len - 1) * st_l + 1) * 2),
                         span(ssm_state, static_cast<size_t>((n_slots - 1) * ssm_st_slot + (ssm_len - 1) * ssm_st_pos + hpn) * 4)};
    const Span in[] = {span(xBC, mat_bytes(rows, x_row_stride, static_cast<int>(channels))),
                       span(weight, static_cast<size_t>(channels) * width * dtype_size(w_dtype)),
                       span(bias, bias ? static_cast<size_t>(channels) * dtype_size(b_dtype) : 0),
                       span(dt, rows > 0 ? static_cast<size_t>((rows - 1) * dt_row_stride + H) * dtype_size(dt_dtype) : 0),
                       span(A, static_cast<size_t>(H) * ps), span(D, static_cast<size_t>(H) * ps), span(dt_bias, static_cast<size_t>(H) * ps),
                       span(cu_seqlens, (static_cast<size_t>(N) + 1) * 4), span(cache_indices, static_cast<size_t>(N) * 4),
                       span(num_accepted, static_cast<size_t>(N) * 4)};
    for (int i = 0; i < 3; ++i) {
        for (const Span &o : in)
            if (overlap(made[i], o)) return CCC_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(made[i], made[j])) return CCC_ERR_ALIAS;
    }
    StepArgs a = {};
    a.s.rows = rows, a.s.H = H, a.s.P = P, a.s.G = G, a.s.N = N_state;
    a.s.dt = dt, a.s.dt_rs = dt_row_stride, a.s.dt_bf16 = dt_dtype == CCC_BF16, a.s.softplus = dt_softplus != 0;
    a.s.A = A, a.s.D = D, a.s.dt_bias = dt_bias, a.s.p_bf16 = p_dtype == CCC_BF16;
    a.s.cu = cu_seqlens, a.s.n_seqs = N, a.s.cache = cache_indices;
    a.s.pool = ssm_state, a.s.n_slots = n_slots, a.s.st_slot = ssm_st_slot;
    a.s.out = static_cast<uint16_t *>(out), a.s.out_rs = out_row_stride;
    a.xbc = static_cast<const uint16_t *>(xBC), a.xs = x_row_stride;
    a.w = weight, a.w_bf16 = w_dtype == CCC_BF16, a.width = width, a.act = activation;
    a.b = bias, a.b_kind = bias ? (b_dtype == CCC_F32 ? 1 : 2) : 0;
    a.conv = static_cast<uint16_t *>(conv_state), a.state_len = state_len, a.st_slot = st_slot, a.st_c = st_c, a.st_l = st_l;
    a.held = ssm_len, a.st_pos = ssm_st_pos, a.accepted = num_accepted;
    const int rep = H / G;
    a.waits = current_waits();
    a.heads_per_cta = step_heads(static_cast<int64_t>(N) * G, rep, P, N_state);
    while (a.heads_per_cta > 1 && staged_bytes(a.heads_per_cta, P, N_state) > 48 * 1024) a.heads_per_cta = (a.heads_per_cta + 1) / 2;
    a.heads_per_cta = std::max(a.heads_per_cta, (rep + 7) / 8);
    a.ctas = (rep + a.heads_per_cta - 1) / a.heads_per_cta;
    if (static_cast<int64_t>(N) * G * a.ctas > INT32_MAX) return CCC_ERR_SHAPE;
    if (staged_bytes(a.heads_per_cta, P, N_state) > 150 * 1024) return CCC_ERR_SHAPE;  // more heads in a group than eight CTAs can stage
    set_last_launches(0);
    if (rows == 0 || N == 0) return CCC_OK;
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    const cudaError_t e = N_state <= 32 ? launch_step<8, 1>(a, st) : N_state <= 64 ? launch_step<16, 1>(a, st)
                        : N_state <= 128 ? launch_step<32, 1>(a, st) : launch_step<32, 2>(a, st);
    if (e != cudaSuccess) return CCC_ERR_CUDA;
    set_last_launches(1);
    return CCC_OK;
}

extern "C" int ccc_ssm_update_v(const int64_t *args) { return call_packed(ccc_ssm_update, args); }
