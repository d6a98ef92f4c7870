// rows.h -- what the norms' kernels share (rms_norm.hip, layer_norm.hip): a row's
// threads, the sums over them, the sizes and types that they take.
#pragma once

#include <hip/hip_runtime.h>

#include <climits>
#include <type_traits>

#include "elements.h"

namespace {

// A row's threads' values together, the same bits in all of them.  `red` holds a
// value a wave; calls that follow each other take it in turn (`turn`), so one
// barrier each is enough: a wave is at most one call ahead.
template <int TPR, class F>
__device__ __forceinline__ float over_row(float x, F join, float (*red)[16], int turn) {
#pragma unroll
    for (int off = 1; off < (TPR < 64 ? TPR : 64); off <<= 1) x = join(x, __shfl_xor(x, off));
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) red[turn][threadIdx.x >> 6] = x;
        __syncthreads();
        const int first = threadIdx.x / TPR * (TPR / 64);
        x = red[turn][first];
#pragma unroll
        for (int i = 1; i < TPR / 64; ++i) x = join(x, red[turn][first + i]);
    }
    return x;
}
constexpr int threads_of(int tpr) { return tpr < 256 ? 256 : tpr; }

// ---------------------------------------------------------- host helpers
inline bool is_type(int t) { return t == CFC_TYPE_F32 || t == CFC_TYPE_BF16 || t == CFC_TYPE_F16; }

constexpr long long kMaxRowWidth = 16384;

inline int check_sizes(int type, int stream_type, long long rows, long long width) {
    if (!is_type(type) || (stream_type != type && stream_type != CFC_TYPE_F32)) return CFC_ERR_UNSUPPORTED;
    if (rows < 0 || width < 1) return CFC_ERR_DIM;
    if (width > kMaxRowWidth) return CFC_ERR_UNSUPPORTED;
    if (rows > LLONG_MAX / 8 / width) return CFC_ERR_DIM;
    return CFC_OK;
}

// Threads and 8-column vectors of a row: the rule on the width alone, as few threads as
// hold the row with one vector each.  More leave lanes idle (forward | backward in us,
// bf16): 300000 x 128 with 16 lanes a row 25 | 43, with 64 61 | 106; 100000 x 512 with 64
// 34 | 63, with 256 74 | 180; 65536 x 1024 with 128 45 | 85, with 256 56 | 139.  Fewer, with
// two vectors, leave less in flight: 16384 x 4096 with 512 threads 43 | 86, with 256
// 47 | 126.  Beyond 8192 columns a workgroup has no more threads.
template <class F>
int with_tiling(long long width, F f) {
    const std::integral_constant<int, 1> one;
    if (width <= 128) return f(std::integral_constant<int, 16>{}, one);
    if (width <= 512) return f(std::integral_constant<int, 64>{}, one);
    if (width <= 1024) return f(std::integral_constant<int, 128>{}, one);
    if (width <= 2048) return f(std::integral_constant<int, 256>{}, one);
    if (width <= 4096) return f(std::integral_constant<int, 512>{}, one);
    if (width <= 8192) return f(std::integral_constant<int, 1024>{}, one);
    return f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
}
inline long long rows_at_once(long long width) { return width <= 128 ? 16 : width <= 512 ? 4 : width <= 1024 ? 2 : 1; }

template <class F>
int with_types(int type, int stream_type, F f) {
    if (type == CFC_TYPE_F32) return f(F32{}, F32{});
    if (type == CFC_TYPE_BF16) return stream_type == CFC_TYPE_F32 ? f(BF16{}, F32{}) : f(BF16{}, BF16{});
    return stream_type == CFC_TYPE_F32 ? f(F16{}, F32{}) : f(F16{}, F16{});
}

}  // namespace
