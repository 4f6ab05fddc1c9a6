// ccc_scan.h -- what the selective-scan kernels share: the argument block,
// the chunk numbering and the launch interface behind ccc_scan_api.cu.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace ccc {

struct ScanArgs {
    const uint16_t *x;   // BF16 [rows][x_rs], head h at h * P
    const void *dt;      // [rows][dt_rs]
    const uint16_t *B, *C;  // BF16 [rows][.._rs], group g at g * N
    const uint16_t *dy;  // BF16 [rows][dy_rs] (backward)
    int64_t rows, x_rs, dt_rs, b_rs, c_rs, dy_rs;
    int H, P, G, N;      // heads, head size, groups, state size
    int dt_bf16, softplus;
    const void *A, *D, *dt_bias;  // [H]; D and dt_bias may be null
    int p_bf16;
    const int32_t *cu;
    int n_seqs;
    const int32_t *cache;
    const uint8_t *has_init;
    float *pool;         // [slots][st_slot], [H][P][N] contiguous inside
    int n_slots;
    int64_t st_slot;
    const float *initial;  // [n_seqs][H][P][N] instead of a pool
    float *final_state;    // [n_seqs][H][P][N] instead of a pool
    uint16_t *out;
    int64_t out_rs;
    // backward
    const float *d_final;
    int carry_empty;       // CCC_OPT_CARRY_EMPTY: an empty sequence's d_initial is its d_final, not zeros
    uint16_t *dx, *dB, *dC;
    int64_t dx_rs, db_rs, dc_rs, ddt_rs;
    void *ddt;
    float *d_initial;
    // workspace
    float *s_ws, *g_ws;    // [slots of chunks][H][P][N]: state before, gradient after each chunk
    float *db_ws, *dc_ws;  // [rows][G][N]
    float *part;           // [slots of chunks][H][3]: dA, dD, ddt_bias
};

// A kernel of a call behind another one of the same call: it may begin (barriers,
// TMEM, its search for chunks) while that one ends, and waits for it before it
// reads anything that kernels write.
template <class... P, class... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, int threads, size_t smem, bool first, cudaStream_t st, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = first ? 0 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Chunks of a packed batch are numbered without a table: chunk k of sequence
// n, which starts at row cu[n] + k Q, has the number floor(row / Q) + n.  It
// grows by one along a sequence and by at least one from a sequence to the
// next, so numbers are unique, at most rows / Q + n_seqs of them.
inline int64_t scan_chunk_slots(int64_t rows, int n_seqs, int q) { return rows / q + n_seqs; }

constexpr int kScanChunk = 64;  // tokens of a chunk of the kernels for every size

cudaError_t launch_scan_states(const ScanArgs &a, bool reverse, cudaStream_t st);
cudaError_t launch_scan_chunks_fwd(const ScanArgs &a, cudaStream_t st);
cudaError_t launch_scan_chunks_bwd(const ScanArgs &a, cudaStream_t st);
cudaError_t launch_scan_sums(const float *part, int64_t slots, int H, float *dA, float *dD, float *dbias,
                             bool first, cudaStream_t st);

}  // namespace ccc
