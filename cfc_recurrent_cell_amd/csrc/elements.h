// elements.h -- element types and argument checks that delta_rule.hip and rms_norm.hip
// share.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "delta_rule.h" /* CFC_TYPE_*, status codes */

namespace {

// What a type's tensors hold, and as 32-bit floats.
struct F32 {
    using S = float;
    static constexpr int NP = 3;  // bf16 parts that hold a value exactly
    static __device__ __forceinline__ float load(S x) { return x; }
    static __device__ __forceinline__ S store(float x) { return x; }
};
struct BF16 {
    using S = uint16_t;
    static constexpr int NP = 1;
    static __device__ __forceinline__ float load(S x) { return __uint_as_float((uint32_t)x << 16); }
    static __device__ __forceinline__ S store(float x) { return __builtin_bit_cast(S, (__bf16)x); }
};
struct F16 {
    using S = _Float16;
    static constexpr int NP = 2;
    static __device__ __forceinline__ float load(S x) { return (float)x; }
    static __device__ __forceinline__ S store(float x) { return (_Float16)x; }
};

inline int size_of(int type) { return type == CFC_TYPE_F32 ? 4 : 2; }

// An argument's bytes; none of a null pointer.
struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};
inline Range bytes_of(const void* p, long long n) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{lo, lo + (uintptr_t)(p ? n : 0)};
}
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi; }
inline bool same(Range a, Range b) { return a.lo == b.lo && a.hi == b.hi; }
inline bool outputs_disjoint(const Range* outs, int n_out, const Range* ins, int n_in) {
    for (int o = 0; o < n_out; ++o) {
        for (int i = 0; i < n_in; ++i)
            if (overlap(outs[o], ins[i])) return false;
        for (int p = o + 1; p < n_out; ++p)
            if (overlap(outs[o], outs[p])) return false;
    }
    return true;
}

inline int launch_status() { return hipGetLastError() == hipSuccess ? CFC_OK : CFC_ERR_HIP; }

}  // namespace
