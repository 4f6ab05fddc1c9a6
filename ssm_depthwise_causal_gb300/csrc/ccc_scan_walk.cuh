// ccc_scan_walk.cuh -- how the walking scan kernels divide their work.
//
// Work is a line of `pairs` x T positions: for each pair of heads, the T
// valid rows.  CTA i takes the part [i W / n, (i + 1) W / n) of the line
// (W = pairs T), so that every CTA gets the same number of rows whatever the
// lengths, and walks it pair by pair and sequence by sequence in chunks of
// 128 rows counted from the sequence's start.  Cuts are moved up to the next
// chunk or sequence end.  A cut inside a sequence leaves a CTA's first
// sequence open at its start, and the CTA before it open at its end: the
// state crosses there (ccc_scan_tc.cu).
#pragma once

#include "ccc_scan_device.cuh"

namespace ccc {

constexpr int kTcChunk = 128;

// The last sequence that starts at or before row q, by a whole warp, 32 offsets a step.
__device__ __forceinline__ int warp_find_seq(const ScanArgs &a, int64_t q) {
    int lo = 0, hi = a.n_seqs;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, i = lo + static_cast<int>(threadIdx.x % 32) * step;
        const int below = __popc(__ballot_sync(kFull, i < hi && a.cu[i] <= q));
        lo += max(below - 1, 0) * step;
        hi = min(lo + step, hi);
    }
    return lo;
}

// The valid rows, clamped.
__device__ __forceinline__ int64_t scan_valid(const ScanArgs &a) {
    return min(max(static_cast<int64_t>(a.cu[a.n_seqs]), int64_t{0}), a.rows);
}

// Row q moved up to the start of a chunk or the end of its sequence.
__device__ __forceinline__ int64_t align_cut(const ScanArgs &a, int64_t q, int64_t valid) {
    if (q <= 0) return 0;
    if (q >= valid) return valid;
    const Seq s = scan_seq(a, warp_find_seq(a, q));
    return min(s.begin + (q - s.begin + kTcChunk - 1) / kTcChunk * kTcChunk, s.end);
}

// In how many of `parts` parts the line is cut, by a whole warp.  Where all
// sequences have the same length, the largest number whose cuts are all between
// sequences: the first pass over what cuts leave open (half of a walk's time) is
// then empty, unless over a third of the CTAs would be idle.  Eight sequences of
// 2048, 32 heads of 64, N = 128: forward 83 us so, 104 us with one of them eight
// tokens shorter; backward 438 and 503 us.
__device__ __forceinline__ int walk_parts(const ScanArgs &a, int64_t valid, int pairs, int parts) {
    const int lane = threadIdx.x % 32;
    const int64_t length = valid / a.n_seqs, lines = static_cast<int64_t>(pairs) * a.n_seqs;
    bool even = a.n_seqs <= 1024;
    for (int i = lane; even && i <= a.n_seqs; i += 32) even = a.cu[i] == i * length;
    if (!__all_sync(kFull, even)) return parts;
    for (int top = parts; 3 * top > 2 * parts; top -= 32) {
        const int d = top - lane;
        const unsigned fits = __ballot_sync(kFull, 3 * d > 2 * parts && lines % d == 0);
        if (fits) return top - (__ffs(fits) - 1);
    }
    return parts;
}

// The chunks of a CTA's part in walking order, forward or reverse; every
// method is called by whole warps.
template <bool REV>
struct Walk {
    int64_t valid, from, to;  // the CTA's part of the line
    int pair, pair_end;       // the current pair and one past the last one (first one less one, reverse)
    int64_t lo, hi;           // the CTA's rows of the current pair
    int n;                    // the current sequence
    Seq s;
    int64_t row;              // the current chunk
    bool fresh;               // the chunk is the first one of its sequence in this segment
    bool more;

    __device__ __forceinline__ void segment(const ScanArgs &a) {
        const int64_t base = static_cast<int64_t>(pair) * valid;
        lo = align_cut(a, max(from - base, int64_t{0}), valid);
        hi = align_cut(a, min(to - base, valid), valid);
        n = warp_find_seq(a, REV ? hi - 1 : lo);
        s = scan_seq(a, n);
        place();
    }
    // the first chunk of sequence n inside [lo, hi)
    __device__ __forceinline__ void place() {
        if (REV) {
            const int64_t end = min(s.end, hi);
            row = s.begin + (end - 1 - s.begin) / kTcChunk * kTcChunk;
            if (end <= s.begin) row = s.begin - 1;
        } else {
            row = max(s.begin, lo);
        }
        fresh = true;
    }
    __device__ __forceinline__ bool here() const {
        return lo < hi && (REV ? row >= max(s.begin, lo) && row < min(s.end, hi) : row < min(s.end, hi));
    }
    __device__ __forceinline__ void settle(const ScanArgs &a) {
        while (!here()) {
            const bool in_pair = lo < hi && (REV ? n > 0 && s.begin > lo : n + 1 < a.n_seqs && s.end < hi);
            if (in_pair) {
                const bool run = s.end == s.begin;
                n += REV ? -1 : 1;
                s = scan_seq(a, n);
                // A second empty sequence in turn: over the whole run at once, since others wait for this with a limit.  (The
                // search is a round trip to L2: for each single empty one it cost the 1025-row training batch 2 of 113 us.)
                if (run && s.end == s.begin) {
                    const int to = warp_find_seq(a, REV ? s.begin - 1 : s.begin);
                    n = REV ? min(n, to) : max(n, to);
                    s = scan_seq(a, n);
                }
                place();
                continue;
            }
            pair += REV ? -1 : 1;
            if (pair == pair_end) {
                more = false;
                return;
            }
            segment(a);
        }
    }
    __device__ __forceinline__ void init(const ScanArgs &a, int pairs, int part, int parts) {
        valid = scan_valid(a);
        const int64_t w = valid * pairs;
        parts = walk_parts(a, valid, pairs, parts);
        from = min(w, w * part / parts);
        to = min(w, w * (part + 1) / parts);
        more = from < to;
        if (!more) return;
        const int first = static_cast<int>(from / valid), last = static_cast<int>((to - 1) / valid);
        pair = REV ? last : first;
        pair_end = REV ? first - 1 : last + 1;
        segment(a);
        settle(a);
    }
    // Only the sequence that the CTA's part leaves open at its end (its start, reverse), if there is one.
    __device__ __forceinline__ void init_tail(const ScanArgs &a, int pairs, int part, int parts) {
        valid = scan_valid(a);
        const int64_t w = valid * pairs;
        parts = walk_parts(a, valid, pairs, parts);
        from = min(w, w * part / parts);
        to = min(w, w * (part + 1) / parts);
        more = from < to;
        if (!more) return;
        pair = static_cast<int>((REV ? from : to - 1) / valid);
        pair_end = REV ? pair - 1 : pair + 1;
        const int64_t base = static_cast<int64_t>(pair) * valid;
        lo = align_cut(a, max(from - base, int64_t{0}), valid);
        hi = align_cut(a, min(to - base, valid), valid);
        const int64_t cut = REV ? lo : hi;
        more = lo < hi && cut > 0 && cut < valid;
        if (!more) return;
        n = warp_find_seq(a, cut);
        s = scan_seq(a, n);
        more = s.begin < cut;
        if (!more) return;
        if (REV) hi = min(hi, s.end); else lo = max(lo, s.begin);
        place();
        more = here();
    }
    __device__ __forceinline__ void next(const ScanArgs &a) {
        row += REV ? -kTcChunk : kTcChunk;
        fresh = false;
        settle(a);
    }
    __device__ __forceinline__ int len() const { return static_cast<int>(min(s.end - row, static_cast<int64_t>(kTcChunk))); }
    // whether the walk meets its sequence at that sequence's own edge, and leaves it at the other
    __device__ __forceinline__ bool enters() const { return REV ? s.end <= hi : s.begin >= lo; }
    __device__ __forceinline__ bool leaves() const { return REV ? row == s.begin : row + kTcChunk >= s.end; }
};

}  // namespace ccc
