// ccc_scan_tc.cuh -- device helpers that the two walks of the tensor-core scan
// share: chunk descriptions, head tiles, states in global memory.
#pragma once

#include "ccc_scan_tc.h"
#include "ccc_scan_walk.cuh"
#include "ccc_tc.cuh"

namespace ccc {

constexpr uint32_t kTile = 16384;  // 128 rows of 64 BF16, 128-byte swizzle

// A chunk as the warp that finds them tells the others.
enum : int { kMore = 1, kFresh = 2, kEnters = 4, kLeaves = 8, kDead = 16, kOpenEnd = 32 };
struct ChunkDesc {
    int row, len, n, pair, flags, pad[3];
};

template <bool REV>
__device__ __forceinline__ void describe(const Walk<REV> &wk, int dead, ChunkDesc &d) {
    d.flags = 0;
    if (!wk.more) return;
    d.row = static_cast<int>(wk.row), d.len = wk.len(), d.n = wk.n, d.pair = wk.pair;
    d.flags = kMore | dead | (wk.fresh ? kFresh : 0) | (wk.enters() ? kEnters : 0) | (wk.leaves() ? kLeaves : 0) | (wk.s.end > wk.hi ? kOpenEnd : 0);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) { return f2_to_bf2(make_float2(lo, hi)); }

// What a pair of heads is: head, tile of 64 channels, and whether it is there.
struct Head {
    int h, tile;
    bool ok;
};

__device__ __forceinline__ Head head_of(const ScanTcArgs &a, int pair, int i) {
    const int v = pair % a.pairs_per_group * 2 + i, g = pair / a.pairs_per_group, rep = a.s.H / a.s.G;
    Head r{g * rep + v / a.tiles, v % a.tiles, v < rep * a.tiles};
    if (!r.ok) r.h = a.s.H;  // past the end: TMA reads zeros
    return r;
}

// W columns from c0 of a row (head, channel lp of its tile) of a state
// buffer [H][P][N]; zeros where there are none.
template <int W>
__device__ __forceinline__ void load_state(const ScanTcArgs &a, const float *from, const Head &h, int lp, int c0, float (&S)[W]) {
    const int p = h.tile * 64 + lp;
    const bool ok = from && h.ok && p < a.s.P;
    const float *row = from + (static_cast<int64_t>(h.h) * a.s.P + p) * a.s.N + c0;
#pragma unroll
    for (int i = 0; i < W; i += 4) {
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (ok && c0 + i < a.s.N) v = *reinterpret_cast<const float4 *>(row + i);
        S[i] = v.x, S[i + 1] = v.y, S[i + 2] = v.z, S[i + 3] = v.w;
    }
}

template <int W>
__device__ __forceinline__ void store_state(const ScanTcArgs &a, float *to, const Head &h, int lp, int c0, const float (&S)[W]) {
    const int p = h.tile * 64 + lp;
    if (!to || !h.ok || p >= a.s.P) return;
    float *row = to + (static_cast<int64_t>(h.h) * a.s.P + p) * a.s.N + c0;
#pragma unroll
    for (int i = 0; i < W; i += 4)
        if (c0 + i < a.s.N) *reinterpret_cast<float4 *>(row + i) = make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
}

template <int W>
__device__ __forceinline__ void copy_out(float *to, const float (&S)[W]) {
#pragma unroll
    for (int i = 0; i < W; i += 4) *reinterpret_cast<float4 *>(to + i) = make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
}

// A state that enters a CTA's part inside a sequence comes from the parts
// before it (after it, reverse) back to the one that holds the sequence's
// start: that part's number.
template <bool REV>
__device__ __forceinline__ int carry_from(const ScanTcArgs &a) {
    constexpr int dir = REV ? 1 : -1;
    const int me = blockIdx.x, lane = threadIdx.x % 32, parts = gridDim.x;
    for (int at = me + dir; at >= 0 && at < parts; at += 32 * dir) {
        const int j = at + lane * dir;
        const unsigned found = __ballot_sync(kFull, j >= 0 && j < parts && a.flag[j]);
        if (found) return at + (__ffs(found) - 1) * dir;
    }
    return me;
}

// W columns from c0 of that state: each part's own state decayed by the parts since.
template <bool REV, int W>
__device__ __forceinline__ void carry_in(const ScanTcArgs &a, int from, int t, int lh, int width, int c0, float (&S)[W]) {
    constexpr int dir = REV ? 1 : -1, Q = kTcChunk;
#pragma unroll
    for (int i = 0; i < W; ++i) S[i] = 0.0f;
    for (int j = from; j != static_cast<int>(blockIdx.x); j -= dir) {
        const float keep = a.keep[j * 2 + lh];
        const float *r = a.local + (static_cast<int64_t>(j) * Q + t) * width + c0;
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(r + i);
            S[i] = fmaf(keep, S[i], v.x);
            S[i + 1] = fmaf(keep, S[i + 1], v.y);
            S[i + 2] = fmaf(keep, S[i + 2], v.z);
            S[i + 3] = fmaf(keep, S[i + 3], v.w);
        }
    }
}

__device__ __forceinline__ void warp_arrive(uint32_t bar) {
    __syncwarp();
    if (threadIdx.x % 32 == 0) bar_arrive(bar);
}

// dt_raw of row 32 i + lane of a chunk, i = 0 .. 3, for one head, as loaded.
__device__ __forceinline__ void fetch_steps(const ScanTcArgs &a, const ChunkDesc &d, const Head &h, uint32_t (&to)[4]) {
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        to[i] = 0u;
        if (h.ok && 32 * i + lane < d.len) to[i] = dt_bits(a.s, static_cast<int64_t>(d.row) + 32 * i + lane, h.h);
    }
}

// The same rows into L2, well ahead: the loads' latency is the steps' time.
__device__ __forceinline__ void prefetch_steps(const ScanTcArgs &a, int64_t row, int64_t valid, int pair) {
    const int lane = threadIdx.x % 32, h = head_of(a, pair, 0).h;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t at = row + 32 * i + lane;
        if (at < valid) l2_line(static_cast<const unsigned char *>(a.s.dt) + (at * a.s.dt_rs + h) * (a.s.dt_bf16 ? 2 : 4));
    }
}

// Running sums over each block of 32, one block per register.
__device__ __forceinline__ void block_sums(float (&p)[4], float (&total)[4]) {
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int j = 1; j < 32; j *= 2)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float o = __shfl_up_sync(kFull, p[i], j);
            if (lane >= j) p[i] += o;
        }
#pragma unroll
    for (int i = 0; i < 4; ++i) total[i] = __shfl_sync(kFull, p[i], 31);
}

// The sums behind each token in its block of 32 from the values, their running sums and totals.  The difference of the last
// two is off by up to 2^-23 of the total: by 2^-16 for totals up to 128, some 5 a token.  Above they are added up on their
// own, from the end.  The gradient kernels take the difference: what leaves them through it has 16 bits, or is a sum over
// tokens, and the sums cost them 20 of 1562 us of the packed training step.
__device__ __forceinline__ void block_after(const float (&v)[4], const float (&p)[4], const float (&total)[4], float (&after)[4]) {
    const int lane = threadIdx.x % 32;
    if (fmaxf(fmaxf(fabsf(total[0]), fabsf(total[1])), fmaxf(fabsf(total[2]), fabsf(total[3]))) <= 128.0f) {  // (the same for the warp)
#pragma unroll
        for (int i = 0; i < 4; ++i) after[i] = total[i] - p[i];
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) after[i] = v[i];
#pragma unroll 1
    for (int j = 1; j < 32; j *= 2)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float o = __shfl_down_sync(kFull, after[i], j);
            if (lane + j < 32) after[i] += o;
        }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        after[i] = __shfl_down_sync(kFull, after[i], 1);
        if (lane == 31) after[i] = 0.0f;
    }
}

}  // namespace ccc
