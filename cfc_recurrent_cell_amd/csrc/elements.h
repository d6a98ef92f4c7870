// elements.h -- element types, their loads and argument checks that the kernels share
// (all but cfc.hip's).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>

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

// 16 and 8 bytes at an address that the element's size divides; the memory takes them at any.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));

// V consecutive elements as they lie in memory, 8 bytes of them or a multiple of 16.
template <class TY, int V>
struct Packed {
    uint32_t w[V * sizeof(typename TY::S) / 4];
};

// Columns c ... c + V - 1 of a row, zero from `width` on, in two steps: `fetch` loads them,
// `unpack` turns them to 32-bit floats.  TAIL: the width need be no multiple of V; where a row
// ends among the columns its last V are loaded, so that no lane's load waits for another's,
// and moved to where they belong when they are unpacked.
template <class TY, int V, bool TAIL>
__device__ __forceinline__ Packed<TY, V> fetch(const typename TY::S* row, int c, int width) {
    constexpr int N = V * sizeof(typename TY::S) / 4;
    Packed<TY, V> e;
#pragma unroll
    for (int i = 0; i < N; ++i) e.w[i] = 0;
    if (TAIL ? width >= V : c < width) {
        const char* from = reinterpret_cast<const char*>(row + (TAIL ? min(c, width - V) : c));
        if constexpr (N == 2) {
            const u32x2_any a = *reinterpret_cast<const u32x2_any*>(from);
            e.w[0] = a[0], e.w[1] = a[1];
        } else {
#pragma unroll
            for (int i = 0; i < N / 4; ++i) {
                const u32x4_any a = *reinterpret_cast<const u32x4_any*>(from + 16 * i);
#pragma unroll
                for (int j = 0; j < 4; ++j) e.w[4 * i + j] = a[j];
            }
        }
    } else if constexpr (TAIL) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (c + j < width) {
                if constexpr (sizeof(typename TY::S) == 4)
                    e.w[j] = __builtin_bit_cast(uint32_t, row[c + j]);
                else
                    e.w[j >> 1] |= (uint32_t)__builtin_bit_cast(uint16_t, row[c + j]) << (16 * (j & 1));
            }
    }
    return e;
}
template <class TY, int V, bool TAIL>
__device__ __forceinline__ void unpack(Packed<TY, V> e, int c, int width, float (&x)[V]) {
    constexpr int N = V * sizeof(typename TY::S) / 4, per = V / N;  // elements of a word
    const int over = TAIL && width >= V ? c + V - width : 0;        // columns that the row has not
    if (over > 0) {
#pragma unroll
        for (int by = N / 2; by > 0; by >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) e.w[i] = over & (by * per) ? (i + by < N ? e.w[i + by] : 0) : e.w[i];
        if constexpr (per == 2) {
#pragma unroll
            for (int i = 0; i < N; ++i) e.w[i] = over & 1 ? e.w[i] >> 16 | (i + 1 < N ? e.w[i + 1] << 16 : 0) : e.w[i];
        }
#pragma unroll
        for (int i = 0; i < N; ++i) e.w[i] = over >= V ? 0 : e.w[i];
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if constexpr (sizeof(typename TY::S) == 4)
            x[j] = __builtin_bit_cast(float, e.w[j]);
        else
            x[j] = TY::load(__builtin_bit_cast(typename TY::S,
                                               (uint16_t)(j & 1 ? e.w[j >> 1] >> 16 : e.w[j >> 1] & 0xffff)));
    }
}
template <class TY, int V, bool TAIL>
__device__ __forceinline__ void load(const typename TY::S* row, int c, int width, float (&x)[V]) {
    unpack<TY, V, TAIL>(fetch<TY, V, TAIL>(row, c, width), c, width, x);
}
template <class TY, int V, bool TAIL>
__device__ __forceinline__ void store(typename TY::S* row, int c, int width, const float (&x)[V]) {
    if (TAIL ? c + V <= width : c < width) {
        Packed<TY, V> e;
        if constexpr (sizeof(typename TY::S) == 4) {
#pragma unroll
            for (int j = 0; j < V; ++j) e.w[j] = __builtin_bit_cast(uint32_t, x[j]);
        } else {
#pragma unroll
            for (int j = 0; j < V / 2; ++j)
                e.w[j] = (uint32_t)__builtin_bit_cast(uint16_t, TY::store(x[2 * j])) |
                         (uint32_t)__builtin_bit_cast(uint16_t, TY::store(x[2 * j + 1])) << 16;
        }
        if constexpr (sizeof(e) == 8) {
            *reinterpret_cast<u32x2_any*>(row + c) = u32x2_any{e.w[0], e.w[1]};
        } else {
#pragma unroll
            for (int i = 0; i < (int)sizeof(e) / 16; ++i)
                *reinterpret_cast<u32x4_any*>(reinterpret_cast<char*>(row + c) + 16 * i) =
                    u32x4_any{e.w[4 * i], e.w[4 * i + 1], e.w[4 * i + 2], e.w[4 * i + 3]};
        }
    } else if constexpr (TAIL) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (c + j < width) row[c + j] = TY::store(x[j]);
    }
}

// Memory through buffer descriptors: a uniform base, a lane's 32-bit offset and a
// uniform one cost no address arithmetic on the vector units, and what lies behind
// the descriptor's end reads as zero and is not written, so that accesses need no
// branches.  kNowhere is behind every end.
constexpr uint32_t kNowhere = 0x80000000u;
typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ __forceinline__ Buffer buffer_of(const void* p, long long bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
}
// Workgroups are dealt to the 8 dies in turn; `count` logical ones in order, so
// that neighbours (tiles of one head, heads of one key head, channels of one row) share a die's L2.
__device__ __forceinline__ long long on_die(long long block, long long count) {
    const long long each = (count + 7) / 8;
    return (block % 8) * each + block / 8;
}
inline unsigned dealt(long long count) { return (unsigned)((count + 7) / 8 * 8); }

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

// Whether addresses are multiples of `size` (null ones are).
inline bool fits(std::initializer_list<const void*> ps, int size) {
    for (const void* p : ps)
        if (reinterpret_cast<uintptr_t>(p) % size) return false;
    return true;
}

inline int launch_status() { return hipGetLastError() == hipSuccess ? CFC_OK : CFC_ERR_HIP; }

}  // namespace
