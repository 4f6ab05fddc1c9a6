// ccc_checks.h -- host-side helpers of the entry points' argument checks.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cstring>
#include <type_traits>
#include <utility>

#include "ccc.h"

namespace ccc {

constexpr size_t kAlignWs = 256;

inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Byte span [lo, hi) of a buffer, or empty.
struct Span {
    uintptr_t lo = 0, hi = 0;
    bool empty() const { return hi <= lo; }
};

inline Span span(const void *p, size_t bytes) {
    Span s;
    if (p && bytes) {
        s.lo = reinterpret_cast<uintptr_t>(p);
        s.hi = s.lo + bytes;
    }
    return s;
}

inline bool overlap(const Span &a, const Span &b) {
    return !a.empty() && !b.empty() && a.lo < b.hi && b.lo < a.hi;
}

// Rows of a [rows][stride] BF16 matrix with C used columns, in bytes.
inline size_t mat_bytes(int64_t rows, int64_t stride, int C) {
    return rows > 0 ? static_cast<size_t>(((rows - 1) * stride + C) * 2) : 0;
}

inline int dtype_size(int code) { return code == CCC_F32 ? 4 : (code == CCC_BF16 ? 2 : 0); }

// Whether a conv_state pool's strides are usable (ccc_api.cu).
bool state_layout_ok(int n_slots, int C, int L, int64_t s_slot, int64_t s_c, int64_t s_l);

// What ccc_last_launch_count reports for this host thread.
void set_last_launches(int n);

// f with its arguments from an array of 64-bit integers (the _v entry points).
template <class T>
T unpacked(int64_t v) {
    if constexpr (std::is_pointer_v<T>) {
        return reinterpret_cast<T>(static_cast<uintptr_t>(v));
    } else if constexpr (std::is_floating_point_v<T>) {
        const uint32_t bits = static_cast<uint32_t>(v);
        T f;
        static_assert(sizeof(f) == sizeof(bits));
        std::memcpy(&f, &bits, sizeof(f));
        return f;
    } else {
        return static_cast<T>(v);
    }
}

template <class... A, size_t... I>
int call_packed(int (*f)(A...), const int64_t *args, std::index_sequence<I...>) {
    return args ? f(unpacked<A>(args[I])...) : CCC_ERR_NULL;
}

template <class... A>
int call_packed(int (*f)(A...), const int64_t *args) {
    return call_packed(f, args, std::index_sequence_for<A...>());
}

}  // namespace ccc
