// ccc_scan_api.cu -- the C ABI of the selective scan (include/ccc.h):
// host-side checks, workspace carve-up and launches.
#include <algorithm>
#include <climits>
#include <iterator>

#include "ccc.h"
#include "ccc_checks.h"
#include "ccc_scan.h"
#include "ccc_scan_tc.h"

namespace {

using namespace ccc;

// A [rows][stride] matrix with `width` used elements of `size` bytes a row.
struct Mat {
    const void *p = nullptr;
    int64_t rows = 0, stride = 0, width = 0;
    int size = 2;
    Span whole() const {
        return span(p, rows > 0 ? static_cast<size_t>(((rows - 1) * stride + width) * size) : 0);
    }
};

// Whether two matrices share an element.  Column slices of one buffer (the
// same row stride, other columns) do not, although their spans overlap.
bool overlap(const Mat &a, const Mat &b) {
    if (!ccc::overlap(a.whole(), b.whole())) return false;
    if (a.stride * a.size != b.stride * b.size) return true;
    const int64_t pitch = a.stride * a.size;
    int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p)) % pitch;
    if (d < 0) d += pitch;
    return d < a.width * a.size || d + b.width * b.size > pitch;
}

Mat flat(const void *p, int64_t n, int size) { return Mat{p, 1, n, n, size}; }

struct Sizes {
    size_t s = 0, g = 0, db = 0, dc = 0, part = 0;
    size_t total() const { return s + g + db + dc + part; }
};

bool sizes_ok(int64_t rows, int32_t n_seqs, int32_t H, int32_t P, int32_t G, int32_t N) {
    return rows >= 0 && rows <= INT32_MAX && n_seqs >= 0 && H > 0 && H <= 65535 && G > 0 && H % G == 0 && P > 0 &&
           P % 8 == 0 && P <= CCC_SCAN_MAX_HEAD && N > 0 && N % 8 == 0 && N <= CCC_SCAN_MAX_STATE;
}

Sizes sizes_of(int64_t rows, int32_t n_seqs, int32_t H, int32_t P, int32_t G, int32_t N, bool bwd) {
    Sizes z;
    if (!sizes_ok(rows, n_seqs, H, P, G, N) || rows == 0 || n_seqs == 0) return z;
    const ScanTcPlan plan = scan_tc_plan(rows, n_seqs, H, P, G, N);
    const ScanTcBwdPlan back = scan_tc_bwd_plan(rows, n_seqs, H, P, G, N);
    if (bwd ? back.ok : plan.ok) {
        z.s = bwd ? back.bytes : plan.bytes;
        return z;
    }
    const int64_t slots = scan_chunk_slots(rows, n_seqs, kScanChunk);
    z.s = round_up(static_cast<size_t>(slots) * H * P * N * 4, kAlignWs);
    if (!bwd) return z;
    z.g = z.s;
    z.db = z.dc = H == G ? 0 : round_up(static_cast<size_t>(rows) * G * N * 4, kAlignWs);
    z.part = round_up(static_cast<size_t>(slots) * H * 3 * 4, kAlignWs);
    return z;
}

int check_inputs(const ScanArgs &a, int dt_dtype, int p_dtype) {
    if (!sizes_ok(a.rows, a.n_seqs, a.H, a.P, a.G, a.N)) return CCC_ERR_SHAPE;
    if (a.x_rs < static_cast<int64_t>(a.H) * a.P || a.dt_rs < a.H || a.b_rs < static_cast<int64_t>(a.G) * a.N ||
        a.c_rs < static_cast<int64_t>(a.G) * a.N || a.x_rs % 8 || a.b_rs % 8 || a.c_rs % 8)
        return CCC_ERR_SHAPE;
    if (std::max({a.x_rs, a.dt_rs, a.b_rs, a.c_rs}) > INT32_MAX) return CCC_ERR_SHAPE;
    if ((dt_dtype != CCC_F32 && dt_dtype != CCC_BF16) || (p_dtype != CCC_F32 && p_dtype != CCC_BF16)) return CCC_ERR_DTYPE;
    if (!a.A || !a.cu || (a.rows > 0 && (!a.x || !a.dt || !a.B || !a.C))) return CCC_ERR_NULL;
    const int ps = dtype_size(p_dtype);
    if (!aligned(a.x, 16) || !aligned(a.B, 16) || !aligned(a.C, 16) || !aligned(a.dt, dtype_size(dt_dtype)) ||
        !aligned(a.A, ps) || !aligned(a.D, ps) || !aligned(a.dt_bias, ps) || !aligned(a.cu, 4) || !aligned(a.cache, 4) ||
        !aligned(a.initial, 16))
        return CCC_ERR_ALIGN;
    return CCC_OK;
}

}  // namespace

extern "C" {

size_t ccc_scan_workspace_size(int64_t rows, int32_t n_seqs, int32_t H, int32_t P, int32_t G, int32_t N_state,
                               int32_t for_bwd) {
    return sizes_of(rows, n_seqs, H, P, G, N_state, for_bwd != 0).total();
}

int ccc_scan_fwd(const void *x, int64_t rows, int32_t H, int32_t P, int64_t x_row_stride,
                 const void *dt, int32_t dt_dtype, int64_t dt_row_stride, int32_t dt_softplus,
                 const void *A, const void *D, const void *dt_bias, int32_t p_dtype,
                 const void *B, int64_t b_row_stride, const void *C, int64_t c_row_stride, int32_t G, int32_t N_state,
                 float *ssm_state, int32_t n_slots, int64_t st_slot,
                 const float *initial_state, float *final_state,
                 const int32_t *cu_seqlens, int32_t N, const int32_t *cache_indices, const uint8_t *has_initial_state,
                 void *out, int64_t out_row_stride,
                 void *workspace, size_t workspace_bytes, void *cuda_stream) {
    ScanArgs a = {};
    a.x = static_cast<const uint16_t *>(x);
    a.dt = dt;
    a.B = static_cast<const uint16_t *>(B);
    a.C = static_cast<const uint16_t *>(C);
    a.rows = rows;
    a.x_rs = x_row_stride;
    a.dt_rs = dt_row_stride;
    a.b_rs = b_row_stride;
    a.c_rs = c_row_stride;
    a.H = H, a.P = P, a.G = G, a.N = N_state;
    a.dt_bf16 = dt_dtype == CCC_BF16;
    a.softplus = dt_softplus != 0;
    a.A = A, a.D = D, a.dt_bias = dt_bias;
    a.p_bf16 = p_dtype == CCC_BF16;
    a.cu = cu_seqlens;
    a.n_seqs = N;
    a.cache = cache_indices;
    a.has_init = has_initial_state;
    a.pool = ssm_state;
    a.n_slots = n_slots;
    a.st_slot = st_slot;
    a.initial = initial_state;
    a.final_state = final_state;
    a.out = static_cast<uint16_t *>(out);
    a.out_rs = out_row_stride;
    if (int rc = check_inputs(a, dt_dtype, p_dtype)) return rc;
    const int64_t hpn = static_cast<int64_t>(H) * P * N_state, hp = static_cast<int64_t>(H) * P;
    const int64_t gn = static_cast<int64_t>(G) * N_state;
    if (out_row_stride < hp || out_row_stride % 8 || out_row_stride > INT32_MAX) return CCC_ERR_SHAPE;
    if (ssm_state && (initial_state || final_state || n_slots < 1 || st_slot < hpn || st_slot % 4)) return CCC_ERR_SHAPE;
    if ((ssm_state && !cache_indices) || (rows > 0 && !out)) return CCC_ERR_NULL;
    if (!aligned(out, 16) || !aligned(ssm_state, 16) || !aligned(final_state, 16)) return CCC_ERR_ALIGN;
    const Sizes z = sizes_of(rows, N, H, P, G, N_state, false);
    if (z.total() && (!workspace || workspace_bytes < z.total())) return CCC_ERR_WORKSPACE;
    if (z.total() && !aligned(workspace, kAlignWs)) return CCC_ERR_ALIGN;
    const int ps = dtype_size(p_dtype);
    const Mat in[] = {{x, rows, x_row_stride, hp, 2}, {B, rows, b_row_stride, gn, 2}, {C, rows, c_row_stride, gn, 2},
                      {dt, rows, dt_row_stride, H, dtype_size(dt_dtype)}, flat(A, H, ps), flat(D, H, ps), flat(dt_bias, H, ps),
                      flat(initial_state, N * hpn, 4), flat(cu_seqlens, N + int64_t{1}, 4), flat(cache_indices, N, 4),
                      flat(has_initial_state, N, 1)};
    const Mat made[] = {{out, rows, out_row_stride, hp, 2}, flat(ssm_state, ssm_state ? (n_slots - 1) * st_slot + hpn : 0, 4),
                        flat(final_state, N * hpn, 4), flat(workspace, z.total(), 1)};
    for (size_t i = 0; i < std::size(made); ++i) {
        for (const Mat &o : in)
            if (overlap(made[i], o)) return CCC_ERR_ALIAS;
        for (size_t j = 0; j < i; ++j)
            if (overlap(made[i], made[j])) return CCC_ERR_ALIAS;
    }
    set_last_launches(0);
    if (N == 0) return CCC_OK;
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    if (rows == 0 && !final_state) return CCC_OK;
    const ScanTcPlan plan = scan_tc_plan(rows, N, H, P, G, N_state);
    if (plan.ok && rows > 0) {
        int launches = 0;
        if (launch_scan_tc_fwd(a, plan, static_cast<unsigned char *>(workspace), &launches, st) != cudaSuccess) return CCC_ERR_CUDA;
        set_last_launches(launches);
        return CCC_OK;
    }
    a.s_ws = static_cast<float *>(workspace);
    if (launch_scan_states(a, false, st) != cudaSuccess) return CCC_ERR_CUDA;
    if (rows > 0 && launch_scan_chunks_fwd(a, st) != cudaSuccess) return CCC_ERR_CUDA;
    set_last_launches(rows > 0 ? 2 : 1);
    return CCC_OK;
}

int ccc_scan_bwd_ex(const void *x, int64_t rows, int32_t H, int32_t P, int64_t x_row_stride,
                 const void *dt, int32_t dt_dtype, int64_t dt_row_stride, int32_t dt_softplus,
                 const void *A, const void *D, const void *dt_bias, int32_t p_dtype,
                 const void *B, int64_t b_row_stride, const void *C, int64_t c_row_stride, int32_t G, int32_t N_state,
                 const float *initial_state,
                 const int32_t *cu_seqlens, int32_t N, const int32_t *cache_indices,
                 const void *dy, int64_t dy_row_stride, const float *d_final_state,
                 void *dx, int64_t dx_row_stride, void *ddt, int64_t ddt_row_stride,
                 void *dB, int64_t db_row_stride, void *dC, int64_t dc_row_stride,
                 float *dA, float *dD, float *d_dt_bias, float *d_initial_state,
                 void *workspace, size_t workspace_bytes, uint32_t options, void *cuda_stream) {
    if (options & ~static_cast<uint32_t>(CCC_OPT_CARRY_EMPTY)) return CCC_ERR_SHAPE;
    ScanArgs a = {};
    a.x = static_cast<const uint16_t *>(x);
    a.dt = dt;
    a.B = static_cast<const uint16_t *>(B);
    a.C = static_cast<const uint16_t *>(C);
    a.dy = static_cast<const uint16_t *>(dy);
    a.rows = rows;
    a.x_rs = x_row_stride;
    a.dt_rs = dt_row_stride;
    a.b_rs = b_row_stride;
    a.c_rs = c_row_stride;
    a.dy_rs = dy_row_stride;
    a.H = H, a.P = P, a.G = G, a.N = N_state;
    a.dt_bf16 = dt_dtype == CCC_BF16;
    a.softplus = dt_softplus != 0;
    a.A = A, a.D = D, a.dt_bias = dt_bias;
    a.p_bf16 = p_dtype == CCC_BF16;
    a.cu = cu_seqlens;
    a.n_seqs = N;
    a.cache = cache_indices;
    a.initial = initial_state;
    a.d_final = d_final_state;
    a.carry_empty = (options & CCC_OPT_CARRY_EMPTY) != 0;
    a.dx = static_cast<uint16_t *>(dx);
    a.dB = static_cast<uint16_t *>(dB);
    a.dC = static_cast<uint16_t *>(dC);
    a.ddt = ddt;
    a.dx_rs = dx_row_stride;
    a.db_rs = db_row_stride;
    a.dc_rs = dc_row_stride;
    a.ddt_rs = ddt_row_stride;
    a.d_initial = d_initial_state;
    if (int rc = check_inputs(a, dt_dtype, p_dtype)) return rc;
    const int64_t hpn = static_cast<int64_t>(H) * P * N_state, hp = static_cast<int64_t>(H) * P;
    const int64_t gn = static_cast<int64_t>(G) * N_state;
    if (dy_row_stride < hp || dx_row_stride < hp || ddt_row_stride < H || db_row_stride < gn || dc_row_stride < gn ||
        dy_row_stride % 8 || dx_row_stride % 8 || db_row_stride % 8 || dc_row_stride % 8 ||
        std::max({dy_row_stride, dx_row_stride, ddt_row_stride, db_row_stride, dc_row_stride}) > INT32_MAX)
        return CCC_ERR_SHAPE;
    if (!dA || (D && !dD) || (dt_bias && !d_dt_bias) || (rows > 0 && (!dy || !dx || !ddt || !dB || !dC))) return CCC_ERR_NULL;
    if (!aligned(dy, 16) || !aligned(dx, 16) || !aligned(dB, 16) || !aligned(dC, 16) || !aligned(ddt, dtype_size(dt_dtype)) ||
        !aligned(dA, 4) || !aligned(dD, 4) || !aligned(d_dt_bias, 4) || !aligned(d_final_state, 16) ||
        !aligned(d_initial_state, 16))
        return CCC_ERR_ALIGN;
    const Sizes z = sizes_of(rows, N, H, P, G, N_state, true);
    if (z.total() && (!workspace || workspace_bytes < z.total())) return CCC_ERR_WORKSPACE;
    if (z.total() && !aligned(workspace, kAlignWs)) return CCC_ERR_ALIGN;
    const int ps = dtype_size(p_dtype), ds = dtype_size(dt_dtype);
    const Mat in[] = {{x, rows, x_row_stride, hp, 2}, {B, rows, b_row_stride, gn, 2}, {C, rows, c_row_stride, gn, 2},
                      {dt, rows, dt_row_stride, H, ds}, {dy, rows, dy_row_stride, hp, 2}, flat(A, H, ps), flat(D, H, ps),
                      flat(dt_bias, H, ps), flat(initial_state, N * hpn, 4), flat(d_final_state, N * hpn, 4),
                      flat(cu_seqlens, N + int64_t{1}, 4), flat(cache_indices, N, 4)};
    const Mat made[] = {{dx, rows, dx_row_stride, hp, 2}, {dB, rows, db_row_stride, gn, 2}, {dC, rows, dc_row_stride, gn, 2},
                        {ddt, rows, ddt_row_stride, H, ds}, flat(dA, H, 4), flat(dD, H, 4), flat(d_dt_bias, H, 4),
                        flat(d_initial_state, N * hpn, 4), flat(workspace, z.total(), 1)};
    for (size_t i = 0; i < std::size(made); ++i) {
        for (const Mat &o : in)
            if (overlap(made[i], o)) return CCC_ERR_ALIAS;
        for (size_t j = 0; j < i; ++j)
            if (overlap(made[i], made[j])) return CCC_ERR_ALIAS;
    }
    set_last_launches(0);
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    if (rows == 0 || N == 0) {  // no token: the gradients are zero, but for what an empty sequence hands on
        const size_t bytes = static_cast<size_t>(H) * 4;
        if (cudaMemsetAsync(dA, 0, bytes, st) != cudaSuccess || (dD && cudaMemsetAsync(dD, 0, bytes, st) != cudaSuccess) ||
            (d_dt_bias && cudaMemsetAsync(d_dt_bias, 0, bytes, st) != cudaSuccess))
            return CCC_ERR_CUDA;
        if (!d_initial_state || N == 0) return CCC_OK;
        if (!a.carry_empty)
            return cudaMemsetAsync(d_initial_state, 0, static_cast<size_t>(N) * hpn * 4, st) == cudaSuccess ? CCC_OK : CCC_ERR_CUDA;
        if (launch_edge_states(a, d_initial_state, true, st) != cudaSuccess) return CCC_ERR_CUDA;
        set_last_launches(1);
        return CCC_OK;
    }
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    const ScanTcBwdPlan plan = scan_tc_bwd_plan(rows, N, H, P, G, N_state);
    if (plan.ok) {
        int launches = 0;
        if (launch_scan_tc_bwd(a, plan, ws, dA, dD, d_dt_bias, &launches, st) != cudaSuccess) return CCC_ERR_CUDA;
        set_last_launches(launches);
        return CCC_OK;
    }
    a.s_ws = reinterpret_cast<float *>(ws);
    a.g_ws = reinterpret_cast<float *>(ws += z.s);
    a.db_ws = reinterpret_cast<float *>(ws += z.g);
    a.dc_ws = reinterpret_cast<float *>(ws += z.db);
    a.part = reinterpret_cast<float *>(ws += z.dc);
    if (launch_scan_states(a, false, st) != cudaSuccess || launch_scan_states(a, true, st) != cudaSuccess ||
        launch_scan_chunks_bwd(a, st) != cudaSuccess ||
        launch_scan_sums(a.part, scan_chunk_slots(rows, N, kScanChunk), H, dA, dD, d_dt_bias, true, st) != cudaSuccess)
        return CCC_ERR_CUDA;
    set_last_launches(4);
    return CCC_OK;
}

int ccc_scan_bwd(const void *x, int64_t rows, int32_t H, int32_t P, int64_t x_row_stride,
                 const void *dt, int32_t dt_dtype, int64_t dt_row_stride, int32_t dt_softplus,
                 const void *A, const void *D, const void *dt_bias, int32_t p_dtype,
                 const void *B, int64_t b_row_stride, const void *C, int64_t c_row_stride, int32_t G, int32_t N_state,
                 const float *initial_state,
                 const int32_t *cu_seqlens, int32_t N, const int32_t *cache_indices,
                 const void *dy, int64_t dy_row_stride, const float *d_final_state,
                 void *dx, int64_t dx_row_stride, void *ddt, int64_t ddt_row_stride,
                 void *dB, int64_t db_row_stride, void *dC, int64_t dc_row_stride,
                 float *dA, float *dD, float *d_dt_bias, float *d_initial_state,
                 void *workspace, size_t workspace_bytes, void *cuda_stream) {
    return ccc_scan_bwd_ex(x, rows, H, P, x_row_stride, dt, dt_dtype, dt_row_stride, dt_softplus, A, D, dt_bias, p_dtype, B, b_row_stride, C,
                           c_row_stride, G, N_state, initial_state, cu_seqlens, N, cache_indices, dy, dy_row_stride, d_final_state, dx,
                           dx_row_stride, ddt, ddt_row_stride, dB, db_row_stride, dC, dc_row_stride, dA, dD, d_dt_bias, d_initial_state, workspace,
                           workspace_bytes, 0, cuda_stream);
}

int ccc_scan_fwd_v(const int64_t *args) { return call_packed(ccc_scan_fwd, args); }

int ccc_scan_bwd_v(const int64_t *args) { return call_packed(ccc_scan_bwd, args); }

int ccc_scan_bwd_ex_v(const int64_t *args) { return call_packed(ccc_scan_bwd_ex, args); }

}  // extern "C"
