// ccc_scan_device.cuh -- device helpers of the selective-scan kernels.
#pragma once

#include <cuda_bf16.h>

#include "ccc_device.cuh"
#include "ccc_scan.h"

namespace ccc {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float bf_to_f(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

__device__ __forceinline__ uint16_t f_to_bf(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

__device__ __forceinline__ float par(const void *p, int bf16, int i) {
    return bf16 ? bf_to_f(static_cast<const uint16_t *>(p)[i]) : static_cast<const float *>(p)[i];
}

// The same as loaded, and its value: a conversion would wait for the load.
__device__ __forceinline__ uint32_t par_bits(const void *p, int bf16, int i) {
    return bf16 ? static_cast<const uint16_t *>(p)[i] : static_cast<const uint32_t *>(p)[i];
}

__device__ __forceinline__ float par_value(int bf16, uint32_t bits) { return __uint_as_float(bf16 ? bits << 16 : bits); }

// A sequence's rows, clamped to [0, rows] whatever cu_seqlens holds.
struct Seq {
    int64_t begin, end;
};

__device__ __forceinline__ Seq scan_seq(const ScanArgs &a, int n) {
    const int64_t lo = min(max(static_cast<int64_t>(a.cu[n]), int64_t{0}), a.rows);
    const int64_t hi = min(max(static_cast<int64_t>(a.cu[n + 1]), lo), a.rows);
    return {lo, hi};
}

// A request with a -1 slot: zero output and gradients, no state access.
__device__ __forceinline__ bool scan_padded(const ScanArgs &a, int n) { return a.cache && a.cache[n] == -1; }

// Where sequence n's initial state lies (null: zeros), and where its final one goes (null: nowhere).
__device__ __forceinline__ const float *scan_initial(const ScanArgs &a, int n) {
    if (a.pool) {
        const int q = a.cache[n];
        return (a.has_init && a.has_init[n] && q >= 0 && q < a.n_slots) ? a.pool + q * a.st_slot : nullptr;
    }
    return a.initial && !scan_padded(a, n) ? a.initial + static_cast<int64_t>(n) * a.H * a.P * a.N : nullptr;
}

__device__ __forceinline__ float *scan_final(const ScanArgs &a, int n) {
    if (a.pool) {
        const int q = a.cache[n];
        return q >= 0 && q < a.n_slots ? a.pool + q * a.st_slot : nullptr;
    }
    return a.final_state && !scan_padded(a, n) ? a.final_state + static_cast<int64_t>(n) * a.H * a.P * a.N : nullptr;
}

// The gradient of the initial state of a sequence without rows (null: zeros).  An empty sequence's final state is its
// initial one; a padded request's is zeros whatever it started from.
__device__ __forceinline__ const float *scan_edge_gradient(const ScanArgs &a, int n, bool dead) {
    return a.carry_empty && a.d_final && !dead ? a.d_final + static_cast<int64_t>(n) * a.H * a.P * a.N : nullptr;
}

// The step of dt_raw + dt_bias.  log1p(exp(v)) is v to the last bit of 32 for v > 20.
__device__ __forceinline__ float step_of(float v, int softplus) {
    return !softplus || v > 20.0f ? v : log1pf(expf(v));
}

// The step dt of one token and head, and d dt / d dt_raw.
__device__ __forceinline__ float scan_dt(const ScanArgs &a, int64_t row, int h, float bias, float *slope = nullptr) {
    const int64_t i = row * a.dt_rs + h;
    const float v = (a.dt_bf16 ? bf_to_f(static_cast<const uint16_t *>(a.dt)[i]) : static_cast<const float *>(a.dt)[i]) + bias;
    if (slope) *slope = a.softplus ? 1.0f / (1.0f + expf(-v)) : 1.0f;
    return step_of(v, a.softplus);
}

__device__ __forceinline__ uint32_t dt_bits(const ScanArgs &a, int64_t row, int h) {
    const int64_t i = row * a.dt_rs + h;
    return a.dt_bf16 ? static_cast<const uint16_t *>(a.dt)[i] : static_cast<const uint32_t *>(a.dt)[i];
}

__device__ __forceinline__ float dt_value(const ScanArgs &a, uint32_t bits) { return par_value(a.dt_bf16, bits); }

// The chunk with number `slot` (scan_chunk_slots): its sequence and rows; len = 0 if there is none.
struct Chunk {
    int n, len;
    int64_t row;
};

__device__ __forceinline__ Chunk scan_chunk(const ScanArgs &a, int64_t slot, int q) {
    int lo = 0, hi = a.n_seqs - 1;  // the last n whose first number is at most `slot`
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (scan_seq(a, mid).begin / q + mid <= slot) lo = mid; else hi = mid - 1;
    }
    const Seq s = scan_seq(a, lo);
    const int64_t row = s.begin + (slot - s.begin / q - lo) * q;
    Chunk c{lo, 0, row};
    if (row >= s.begin && row < s.end) c.len = static_cast<int>(min(static_cast<int64_t>(q), s.end - row));
    return c;
}

}  // namespace ccc
