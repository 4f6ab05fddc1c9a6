// ccc_scan.cu -- the selective scan of an SSM mixer over packed sequences,
// for every head size and state size: forward and backward in chunks of
// Q = 64 tokens, all products in FP32 from shared memory.
//
// With a_t the running sum of dt A in a chunk, the recurrence
//     h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t^T,   y_t = h_t C_t + D x_t
// is, inside a chunk that the state S enters and the gradient G leaves,
//     y_t  = sum_{s<=t} exp(a_t - a_s) dt_s (C_t.B_s) x_s + exp(a_t) S C_t + D x_t
//     S'   = exp(a_end) S + sum_s exp(a_end - a_s) dt_s x_s B_s^T
//     dx_s = sum_{t>=s} exp(a_t - a_s) dt_s (C_t.B_s) dy_t + exp(a_end - a_s) dt_s G B_s + D dy_s
//     G'   = exp(a_end) G + sum_t exp(a_t) dy_t C_t^T
// so one kernel walks the states (forward, and G the other way with x, B
// replaced by dy, C) and one handles all chunks side by side.
#include "ccc_scan_device.cuh"

namespace ccc {

namespace {

constexpr int Q = kScanChunk;
constexpr int kThreads = 256;

// out[i][j] = sum_k fa(i, k) fb(j, k) for i < m, j < n (multiples of 4), a
// 4 x 4 block at a time per thread; epi(i, j, value).
template <class FA, class FB, class EPI>
__device__ __forceinline__ void product(int m, int n, int k_end, FA fa, FB fb, EPI epi) {
    const int nb = n / 4;
    for (int blk = threadIdx.x; blk < (m / 4) * nb; blk += kThreads) {
        const int i0 = blk / nb * 4, j0 = blk % nb * 4;
        float acc[4][4] = {};
        for (int k = 0; k < k_end; ++k) {
            float u[4], v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = fa(i0 + i, k);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = fb(j0 + j, k);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(u[i], v[j], acc[i][j]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) epi(i0 + i, j0 + j, acc[i][j]);
    }
}

// Rows [row, row + len) of a BF16 matrix into shared memory; the rows up to Q as zeros.
__device__ __forceinline__ void load_rows(uint16_t *dst, int pitch, const uint16_t *src, int64_t rs, int64_t row, int len,
                                          int width) {
    const int per = width / 8;
    for (int i = threadIdx.x; i < Q * per; i += kThreads) {
        const int r = i / per, c = i % per * 8;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (r < len) v = *reinterpret_cast<const uint4 *>(src + (row + r) * rs + c);
        *reinterpret_cast<uint4 *>(dst + r * pitch + c) = v;
    }
}

// dt, its slope, the running sum of dt A log2(e) of a chunk's tokens and the sum behind each (the decay from a token to the
// chunk's end: a sum of its own, as the difference of two long running sums would lose its bits); past the end dt = 0.
struct Steps {
    float dt[Q], slope[Q], a[Q], after[Q];
};

__device__ __forceinline__ void load_steps(const ScanArgs &a, int h, int64_t row, int len, Steps &s) {
    if (threadIdx.x < Q) {
        const int t = threadIdx.x;
        float dt = 0.0f, slope = 0.0f;
        if (t < len) dt = scan_dt(a, row + t, h, a.dt_bias ? par(a.dt_bias, a.p_bf16, h) : 0.0f, &slope);
        float v = dt * par(a.A, a.p_bf16, h) * kLog2e, w = v;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const float o = __shfl_up_sync(kFull, v, d), u = __shfl_down_sync(kFull, w, d);
            if ((t & 31) >= d) v += o;
            if ((t & 31) + d < 32) w += u;
        }
        s.dt[t] = dt;
        s.slope[t] = slope;
        s.a[t] = v;
        s.after[t ? t - 1 : Q - 1] = t ? w : 0.0f;
    }
    __syncthreads();
    static_assert(Q == 64, "two warps");
    if (threadIdx.x >= 32 && threadIdx.x < Q) s.a[threadIdx.x] += s.a[31];
    if (threadIdx.x < 31) s.after[threadIdx.x] += s.after[31];
    __syncthreads();
}

// The state before each chunk (forward) or the state gradient after each
// chunk (reverse), and what leaves the sequence.  A CTA per sequence and
// head; a thread's elements of the state are its own all along.
__global__ void __launch_bounds__(kThreads) states_kernel(const ScanArgs a, bool reverse) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ Steps st;
    const int n = blockIdx.x, h = blockIdx.y, P = a.P, N = a.N;
    const Seq s = scan_seq(a, n);
    const int64_t hpn = static_cast<int64_t>(a.H) * P * N;
    const int64_t head = static_cast<int64_t>(h) * P * N;
    const bool dead = scan_padded(a, n);
    if (s.end == s.begin || dead) {
        if (reverse && a.d_initial) {
            const float *from = scan_edge_gradient(a, n, dead);
            for (int i = threadIdx.x; i < P * N; i += kThreads) a.d_initial[n * hpn + head + i] = from ? from[head + i] : 0.0f;
        }
        if (!reverse && !a.pool && a.final_state) {
            // an empty sequence hands its initial state on, a padded request none
            const float *from = dead ? nullptr : scan_initial(a, n);
            for (int i = threadIdx.x; i < P * N; i += kThreads) a.final_state[n * hpn + head + i] = from ? from[head + i] : 0.0f;
        }
        return;
    }
    const int pk = N + 8, pv = P + 8;
    uint16_t *ks = reinterpret_cast<uint16_t *>(smem), *vs = ks + Q * pk;
    const int chunks = static_cast<int>((s.end - s.begin + Q - 1) / Q);
    const int64_t slot0 = s.begin / Q + n;
    float *ws = reverse ? a.g_ws : a.s_ws;
    const float *init = reverse ? (a.d_final ? a.d_final + n * hpn : nullptr) : scan_initial(a, n);
    float *leave = reverse ? (a.d_initial ? a.d_initial + n * hpn : nullptr) : scan_final(a, n);
    {
        float *to = ws + (slot0 + (reverse ? chunks - 1 : 0)) * hpn + head;
        product(P, N, 0, [](int, int) { return 0.0f; }, [](int, int) { return 0.0f; },
                [&](int p, int c, float) { to[p * N + c] = init ? init[head + p * N + c] : 0.0f; });
    }
    const int g = h / (a.H / a.G);
    for (int i = 0; i < chunks; ++i) {
        const int c = reverse ? chunks - 1 - i : i;
        const int64_t row = s.begin + static_cast<int64_t>(c) * Q;
        const int len = static_cast<int>(min(static_cast<int64_t>(Q), s.end - row));
        __syncthreads();
        load_rows(ks, pk, (reverse ? a.C : a.B) + g * N, reverse ? a.c_rs : a.b_rs, row, len, N);
        load_rows(vs, pv, (reverse ? a.dy : a.x) + h * P, reverse ? a.dy_rs : a.x_rs, row, len, P);
        load_steps(a, h, row, len, st);
        const float end = st.a[Q - 1], keep = ex2_approx(end);
        if (threadIdx.x < Q) st.slope[threadIdx.x] = reverse ? ex2_approx(st.a[threadIdx.x]) : ex2_approx(st.after[threadIdx.x]) * st.dt[threadIdx.x];
        __syncthreads();
        const float *from = ws + (slot0 + c) * hpn + head;
        float *to = i + 1 == chunks ? (leave ? leave + head : nullptr) : ws + (slot0 + c + (reverse ? -1 : 1)) * hpn + head;
        if (to)
            product(P, N, len, [&](int p, int t) { return bf_to_f(vs[t * pv + p]) * st.slope[t]; },
                    [&](int c2, int t) { return bf_to_f(ks[t * pk + c2]); },
                    [&](int p, int c2, float v) { to[p * N + c2] = fmaf(keep, from[p * N + c2], v); });
    }
}

__global__ void __launch_bounds__(kThreads) chunks_fwd_kernel(const ScanArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ Steps st;
    const int h = blockIdx.y, P = a.P, N = a.N, g = h / (a.H / a.G);
    const int64_t slot = blockIdx.x;
    const Chunk c = scan_chunk(a, slot, Q);
    if (c.len == 0) return;
    uint16_t *out = a.out + c.row * a.out_rs + h * P;
    if (scan_padded(a, c.n)) {
        for (int i = threadIdx.x; i < c.len * P; i += kThreads) out[i / P * a.out_rs + i % P] = 0;
        return;
    }
    const int pk = N + 8, pv = P + 8, pm = Q + 4;
    float *m = reinterpret_cast<float *>(smem);
    uint16_t *bs = reinterpret_cast<uint16_t *>(m + Q * pm), *cs = bs + Q * pk, *xs = cs + Q * pk;
    load_rows(bs, pk, a.B + g * N, a.b_rs, c.row, c.len, N);
    load_rows(cs, pk, a.C + g * N, a.c_rs, c.row, c.len, N);
    load_rows(xs, pv, a.x + h * P, a.x_rs, c.row, c.len, P);
    load_steps(a, h, c.row, c.len, st);
    product(Q, Q, N, [&](int t, int k) { return bf_to_f(cs[t * pk + k]); }, [&](int s, int k) { return bf_to_f(bs[s * pk + k]); },
            [&](int t, int s, float v) { m[t * pm + s] = s <= t ? v * ex2_approx(st.a[t] - st.a[s]) * st.dt[s] : 0.0f; });
    __syncthreads();
    const float D = a.D ? par(a.D, a.p_bf16, h) : 0.0f;
    const float *S = a.s_ws + (slot * a.H + h) * P * N;
    // The two sums of an output, over the chunk's tokens and over the state, as one of length Q + N.
    product(Q, P, Q + N,
            [&](int t, int k) { return k < Q ? m[t * pm + k] : ex2_approx(st.a[t]) * bf_to_f(cs[t * pk + k - Q]); },
            [&](int p, int k) { return k < Q ? bf_to_f(xs[k * pv + p]) : S[p * N + k - Q]; },
            [&](int t, int p, float v) { if (t < c.len) out[t * a.out_rs + p] = f_to_bf(fmaf(D, bf_to_f(xs[t * pv + p]), v)); });
}

__global__ void __launch_bounds__(kThreads) chunks_bwd_kernel(const ScanArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ Steps st;
    __shared__ float s_row[Q], s_col[Q], s_in[Q], s_out[Q], s_tmp[Q], s_sum[kThreads / 32];
    const int g = blockIdx.y, P = a.P, N = a.N, rep = a.H / a.G;
    const int64_t slot = blockIdx.x;
    const Chunk c = scan_chunk(a, slot, Q);
    const bool dead = c.len > 0 && scan_padded(a, c.n);
    const int tid = threadIdx.x;
    if (c.len == 0 || dead) {
        for (int i = tid; i < 3 * rep; i += kThreads) a.part[(slot * a.H + g * rep) * 3 + i] = 0.0f;
        for (int i = tid; i < c.len * N; i += kThreads) {
            a.dB[(c.row + i / N) * a.db_rs + g * N + i % N] = 0;
            a.dC[(c.row + i / N) * a.dc_rs + g * N + i % N] = 0;
        }
        for (int i = tid; i < c.len * rep * P; i += kThreads) a.dx[(c.row + i / (rep * P)) * a.dx_rs + g * rep * P + i % (rep * P)] = 0;
        for (int i = tid; i < c.len * rep; i += kThreads) {
            const int64_t at = (c.row + i / rep) * a.ddt_rs + g * rep + i % rep;
            if (a.dt_bf16) static_cast<uint16_t *>(a.ddt)[at] = 0; else static_cast<float *>(a.ddt)[at] = 0.0f;
        }
        return;
    }
    const int pk = N + 8, pv = P + 8, pm = Q + 4;
    float *cb = reinterpret_cast<float *>(smem), *m = cb + Q * pm, *w = m + Q * pm;
    uint16_t *bs = reinterpret_cast<uint16_t *>(w + Q * pm), *cs = bs + Q * pk, *xs = cs + Q * pk, *ys = xs + Q * pv;
    load_rows(bs, pk, a.B + g * N, a.b_rs, c.row, c.len, N);
    load_rows(cs, pk, a.C + g * N, a.c_rs, c.row, c.len, N);
    __syncthreads();
    product(Q, Q, N, [&](int t, int k) { return bf_to_f(cs[t * pk + k]); }, [&](int s, int k) { return bf_to_f(bs[s * pk + k]); },
            [&](int t, int s, float v) { cb[t * pm + s] = v; });
    for (int r = 0; r < rep; ++r) {
        const int h = g * rep + r;
        const float A = par(a.A, a.p_bf16, h), D = a.D ? par(a.D, a.p_bf16, h) : 0.0f;
        __syncthreads();
        load_rows(xs, pv, a.x + h * P, a.x_rs, c.row, c.len, P);
        load_rows(ys, pv, a.dy + h * P, a.dy_rs, c.row, c.len, P);
        load_steps(a, h, c.row, c.len, st);
        const float end = st.a[Q - 1];
        const float *S = a.s_ws + (slot * a.H + h) * P * N, *G = a.g_ws + (slot * a.H + h) * P * N;
        if (tid < Q) s_row[tid] = s_col[tid] = s_in[tid] = s_out[tid] = 0.0f;
        // W = exp(a_t - a_s) dt_s (dy_t.x_s), M = exp(a_t - a_s) dt_s (C_t.B_s) for s <= t
        product(Q, Q, P, [&](int t, int k) { return bf_to_f(ys[t * pv + k]); }, [&](int s, int k) { return bf_to_f(xs[s * pv + k]); },
                [&](int t, int s, float v) {
                    const float l = s <= t ? ex2_approx(st.a[t] - st.a[s]) : 0.0f;
                    w[t * pm + s] = v * l;
                    m[t * pm + s] = cb[t * pm + s] * l;
                    if (s == t) s_tmp[t] = v;  // dy_t.x_t
                });
        __syncthreads();
        // Row and column sums of exp(a_t - a_s) (C_t.B_s) (dy_t.x_s) without the diagonal, which no decay is part of
        float dD = 0.0f, diag = 0.0f;
        if (tid < Q) {
            dD = s_tmp[tid];
            diag = dD * cb[tid * pm + tid];
            float row = 0.0f, col = 0.0f;
            for (int k = 0; k < tid; ++k) row = fmaf(w[tid * pm + k] * cb[tid * pm + k], st.dt[k], row);
            for (int k = tid + 1; k < Q; ++k) col = fmaf(w[k * pm + tid], cb[k * pm + tid], col);
            s_row[tid] = row;
            s_col[tid] = col;  // without dt_s
        }
        // exp(a_t) C_t . S^T dy_t and exp(a_end - a_s) x_s . G B_s, a warp per token, lanes over the channels
        for (int t = tid / 32; t < c.len; t += kThreads / 32) {
            float in = 0.0f, out = 0.0f;
            for (int p = 0; p < P; ++p) {
                float u = 0.0f, v = 0.0f;
                for (int k = tid % 32; k < N; k += 32) {
                    u = fmaf(S[p * N + k], bf_to_f(cs[t * pk + k]), u);
                    v = fmaf(G[p * N + k], bf_to_f(bs[t * pk + k]), v);
                }
                in = fmaf(u, bf_to_f(ys[t * pv + p]), in);
                out = fmaf(v, bf_to_f(xs[t * pv + p]), out);
            }
            for (int d = 16; d; d /= 2) {
                in += __shfl_xor_sync(kFull, in, d);
                out += __shfl_xor_sync(kFull, out, d);
            }
            if (tid % 32 == 0) {
                s_in[t] = in * ex2_approx(st.a[t]);
                s_out[t] = out * ex2_approx(st.after[t]);  // without dt_s
            }
        }
        // <G, S>, in a fixed order
        float gs = 0.0f;
        for (int i = tid; i < P * N; i += kThreads) gs = fmaf(G[i], S[i], gs);
        for (int d = 16; d; d /= 2) gs += __shfl_xor_sync(kFull, gs, d);
        if (tid % 32 == 0) s_sum[tid / 32] = gs;
        __syncthreads();
        gs = 0.0f;
        for (int i = 0; i < kThreads / 32; ++i) gs += s_sum[i];
        // d(dt A)_t: pairs with s < t <= u, the entering state's with u >= t, the leaving gradient's with s < t, and both
        float through = 0.0f, dstep = 0.0f;
        if (tid < Q) {
            for (int u = Q - 1; u >= tid; --u) through += s_row[u] - s_col[u] * st.dt[u];
            float late = 0.0f, early = 0.0f;
            for (int u = Q - 1; u >= tid; --u) late += s_in[u];
            for (int s = 0; s < tid; ++s) early = fmaf(s_out[s], st.dt[s], early);
            through += late + early + ex2_approx(end) * gs;
            if (tid < c.len) {
                dstep = diag + s_col[tid] + s_out[tid] + A * through;
                const float raw = dstep * st.slope[tid];
                const int64_t at = (c.row + tid) * a.ddt_rs + h;
                if (a.dt_bf16) static_cast<uint16_t *>(a.ddt)[at] = f_to_bf(raw); else static_cast<float *>(a.ddt)[at] = raw;
                dstep = raw;
            }
        }
        // the chunk's share of dA, dD, ddt_bias
        float dA = tid < c.len ? st.dt[tid] * through : 0.0f, db = tid < c.len ? dstep : 0.0f;
        for (int d = 16; d; d /= 2) {
            dA += __shfl_xor_sync(kFull, dA, d);
            dD += __shfl_xor_sync(kFull, dD, d);
            db += __shfl_xor_sync(kFull, db, d);
        }
        __syncthreads();
        if (tid == 0 || tid == 32) { s_tmp[tid] = dA; s_tmp[tid + 1] = dD; s_tmp[tid + 2] = db; }
        __syncthreads();
        if (tid < 3) a.part[(slot * a.H + h) * 3 + tid] = s_tmp[tid] + s_tmp[32 + tid];
        uint16_t *dx = a.dx + c.row * a.dx_rs + h * P;
        product(Q, P, Q + N, [&](int s, int k) { return k < Q ? m[k * pm + s] : ex2_approx(st.after[s]) * bf_to_f(bs[s * pk + k - Q]); },
                [&](int p, int k) { return k < Q ? bf_to_f(ys[k * pv + p]) : G[p * N + k - Q]; },
                [&](int s, int p, float v) { if (s < c.len) dx[s * a.dx_rs + p] = f_to_bf(fmaf(D, bf_to_f(ys[s * pv + p]), v * st.dt[s])); });
        // dB_s and dC_t: sums over the group's heads in FP32, the same thread's elements each time
        product(Q, N, Q + P, [&](int s, int k) { return k < Q ? w[k * pm + s] : ex2_approx(st.after[s]) * bf_to_f(xs[s * pv + k - Q]); },
                [&](int j, int k) { return k < Q ? bf_to_f(cs[k * pk + j]) : G[(k - Q) * N + j]; },
                [&](int s, int j, float v) {
                    if (s >= c.len) return;
                    float *sum = a.db_ws + ((c.row + s) * a.G + g) * N + j;
                    v = fmaf(v, st.dt[s], r ? *sum : 0.0f);
                    if (r + 1 < rep) *sum = v; else a.dB[(c.row + s) * a.db_rs + g * N + j] = f_to_bf(v);
                });
        product(Q, N, Q + P, [&](int t, int k) { return k < Q ? w[t * pm + k] * st.dt[k] : ex2_approx(st.a[t]) * bf_to_f(ys[t * pv + k - Q]); },
                [&](int j, int k) { return k < Q ? bf_to_f(bs[k * pk + j]) : S[(k - Q) * N + j]; },
                [&](int t, int j, float v) {
                    if (t >= c.len) return;
                    float *sum = a.dc_ws + ((c.row + t) * a.G + g) * N + j;
                    v += r ? *sum : 0.0f;
                    if (r + 1 < rep) *sum = v; else a.dC[(c.row + t) * a.dc_rs + g * N + j] = f_to_bf(v);
                });
    }
}

// dA, dD and ddt_bias of a head: its chunks' shares, each lane every 32nd in order, then the lanes' sums.
__global__ void scan_sums_kernel(const float *part, int64_t slots, int H, float *dA, float *dD, float *dbias) {
    grid_dependency_wait();  // (launched behind the kernel before it by the tensor-core path)
    const int h = blockIdx.x * 8 + threadIdx.x / 32, lane = threadIdx.x % 32;
    if (h >= H) return;
    float v[3] = {0.0f, 0.0f, 0.0f};
    for (int64_t s = lane; s < slots; s += 32)
#pragma unroll
        for (int k = 0; k < 3; ++k) v[k] += part[(s * H + h) * 3 + k];
#pragma unroll
    for (int k = 0; k < 3; ++k)
        for (int d = 16; d; d /= 2) v[k] += __shfl_xor_sync(kFull, v[k], d);
    if (lane == 0) {
        dA[h] = v[0];
        if (dD) dD[h] = v[1];
        if (dbias) dbias[h] = v[2];
    }
}

template <class K>
cudaError_t shared_for(K kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
}

}  // namespace

cudaError_t launch_scan_states(const ScanArgs &a, bool reverse, cudaStream_t st) {
    const size_t bytes = static_cast<size_t>(Q) * (a.N + 8 + a.P + 8) * 2;
    if (cudaError_t e = shared_for(states_kernel, bytes)) return e;
    states_kernel<<<dim3(a.n_seqs, a.H), kThreads, bytes, st>>>(a, reverse);
    return cudaGetLastError();
}

cudaError_t launch_scan_chunks_fwd(const ScanArgs &a, cudaStream_t st) {
    const size_t bytes = static_cast<size_t>(Q) * ((Q + 4) * 4 + (2 * (a.N + 8) + a.P + 8) * 2);
    if (cudaError_t e = shared_for(chunks_fwd_kernel, bytes)) return e;
    chunks_fwd_kernel<<<dim3(static_cast<unsigned>(scan_chunk_slots(a.rows, a.n_seqs, Q)), a.H), kThreads, bytes, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_scan_chunks_bwd(const ScanArgs &a, cudaStream_t st) {
    const size_t bytes = static_cast<size_t>(Q) * (3 * (Q + 4) * 4 + 2 * (a.N + 8 + a.P + 8) * 2);
    if (cudaError_t e = shared_for(chunks_bwd_kernel, bytes)) return e;
    chunks_bwd_kernel<<<dim3(static_cast<unsigned>(scan_chunk_slots(a.rows, a.n_seqs, Q)), a.G), kThreads, bytes, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_scan_sums(const float *part, int64_t slots, int H, float *dA, float *dD, float *dbias,
                             bool first, cudaStream_t st) {
    return launch_behind(scan_sums_kernel, dim3((H + 7) / 8), 256, 0, first, st, part, slots, H, dA, dD, dbias);
}

}  // namespace ccc
