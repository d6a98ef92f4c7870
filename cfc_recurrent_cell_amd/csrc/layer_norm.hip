// layer_norm.hip -- gfx950 kernels and C ABI of the layer norm (see
// include/layer_norm.h).
//
// Memory is the bound, so a row is read once into registers, 8 consecutive columns
// a lane, and mean and variance are two sums over its lanes: the variance from the
// differences to the mean, which loses nothing where the mean is far from zero.
// Rows of any width and address are read in 16-byte loads (the memory takes them at
// any alignment); a lane whose columns end inside its 8 loads the row's last 8 instead.
// 16384 x 4096 in bf16 with a 32-bit residual stream (805 MB) 151 us, 5.3 TB/s; the gradients
// of 9999 x 1500 in bf16 34 us and 5 for the sums of weight's and bias's.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "columns.h"
#include "elements.h"
#include "layer_norm.h"
#include "rows.h"

namespace {

static_assert(LAYER_NORM_MAX_WIDTH == kMaxRowWidth, "the width that check_sizes holds rows to");

__device__ __forceinline__ float plus(float p, float q) { return p + q; }

// over_row of two sums at once, with one barrier.
template <int TPR>
__device__ __forceinline__ void over_row_two(float2& s, float (*red)[2][16], int turn) {
#pragma unroll
    for (int off = 1; off < (TPR < 64 ? TPR : 64); off <<= 1) s.x += __shfl_xor(s.x, off), s.y += __shfl_xor(s.y, off);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) red[turn][0][threadIdx.x >> 6] = s.x, red[turn][1][threadIdx.x >> 6] = s.y;
        __syncthreads();
        const int first = threadIdx.x / TPR * (TPR / 64);
        s = {red[turn][0][first], red[turn][1][first]};
#pragma unroll
        for (int i = 1; i < TPR / 64; ++i) s.x += red[turn][0][first + i], s.y += red[turn][1][first + i];
    }
}

template <class TX, class TH, int TPR, int NV, bool TAIL>
__global__ __launch_bounds__(threads_of(TPR)) void layer_norm_kernel(
    long long rows, int width, const typename TX::S* x, const typename TH::S* residual,
    const typename TX::S* __restrict__ weight, const typename TX::S* __restrict__ bias, float eps,
    typename TX::S* __restrict__ y, typename TH::S* h, float* __restrict__ mean, float* __restrict__ rstd) {
    constexpr int RPW = threads_of(TPR) / TPR;
    __shared__ float red[2][16];
    const int sub = threadIdx.x % TPR;
    float w[NV][8], b[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        load<TX, 8, TAIL>(weight, 8 * (v * TPR + sub), width, w[v]);
#pragma unroll
        for (int j = 0; j < 8; ++j) b[v][j] = 0.0f;
        if (bias) load<TX, 8, TAIL>(bias, 8 * (v * TPR + sub), width, b[v]);
    }
    for (long long r0 = (long long)blockIdx.x * RPW; r0 < rows; r0 += (long long)gridDim.x * RPW) {
        const long long row = r0 + threadIdx.x / TPR;
        const bool in = row < rows;  // lanes of a row behind the last compute and write nothing
        const long long at = (in ? row : rows - 1) * width;
        float a[NV][8];
        Packed<TX, 8> xr[NV];
        Packed<TH, 8> rr[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            xr[v] = fetch<TX, 8, TAIL>(x + at, 8 * (v * TPR + sub), width);
            if (residual) rr[v] = fetch<TH, 8, TAIL>(residual + at, 8 * (v * TPR + sub), width);
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) unpack<TX, 8, TAIL>(xr[v], 8 * (v * TPR + sub), width, a[v]);
        if (residual) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float e[8];
                const int c = 8 * (v * TPR + sub);
                unpack<TH, 8, TAIL>(rr[v], c, width, e);
#pragma unroll
                for (int j = 0; j < 8; ++j) a[v][j] = TH::load(TH::store(a[v][j] + e[j]));
                if (h && in) store<TH, 8, TAIL>(h + at, c, width, a[v]);
            }
        }
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j) s += a[v][j];
        const float m = over_row<TPR>(s, plus, red, 0) / (float)width;
        s = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                a[v][j] -= m;
                if (8 * (v * TPR + sub) + j < width) s += a[v][j] * a[v][j];
            }
        const float rs = 1.0f / sqrtf(over_row<TPR>(s, plus, red, 1) / (float)width + eps);
        if (sub == 0 && in) {
            if (mean) mean[row] = m;
            if (rstd) rstd[row] = rs;
        }
        if (in) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
#pragma unroll
                for (int j = 0; j < 8; ++j) a[v][j] = a[v][j] * rs * w[v][j] + b[v][j];
                store<TX, 8, TAIL>(y + at, 8 * (v * TPR + sub), width, a[v]);
            }
        }
    }
}

// A row's loads are in flight while the row before is worked on.
// The weight's and the bias's terms are summed over the workgroup's rows in registers,
// in 64 bits (beyond 8192 columns in 32, over 16 rows at most), then over its row slots
// through LDS, and rounded to 32 bits into part[2 * blockIdx.x] and the row behind it;
// column_sums_kernel sums those in 64.
template <class TX, class TH, int TPR, int NV, bool TAIL>
__global__ __launch_bounds__(threads_of(TPR)) void layer_norm_backward_kernel(
    long long rows, int width, const typename TX::S* __restrict__ gy, const typename TH::S* __restrict__ h,
    const typename TX::S* __restrict__ weight, const float* __restrict__ mean, const float* __restrict__ rstd,
    const typename TH::S* gh, typename TH::S* gx, float* __restrict__ part) {
    constexpr int RPW = threads_of(TPR) / TPR;
    __shared__ float red[2][2][16];
    const int sub = threadIdx.x % TPR, slot = threadIdx.x / TPR;
    float w[NV][8];
    // (two vectors a lane would not fit the registers in 64 bits: few rows a workgroup instead)
    using Sum = std::conditional_t<NV == 1, double, float>;
    Sum gw[NV][8], gb[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        load<TX, 8, TAIL>(weight, 8 * (v * TPR + sub), width, w[v]);
#pragma unroll
        for (int j = 0; j < 8; ++j) gw[v][j] = gb[v][j] = 0.0;
    }
    Packed<TH, 8> hr[NV], gr[NV];
    Packed<TX, 8> yr[NV];
    float rs = 0.0f, m = 0.0f;
    auto fetch_row = [&](long long r0) {
        const long long row = min(r0 + slot, rows - 1);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = 8 * (v * TPR + sub);
            hr[v] = fetch<TH, 8, TAIL>(h + row * width, c, width);
            yr[v] = fetch<TX, 8, TAIL>(gy + row * width, c, width);
            if (gh) gr[v] = fetch<TH, 8, TAIL>(gh + row * width, c, width);
        }
        rs = rstd[row], m = mean[row];
    };
    int turn = 0;
    const long long stride = (long long)gridDim.x * RPW;
    if constexpr (NV == 1) fetch_row((long long)blockIdx.x * RPW);
    for (long long r0 = (long long)blockIdx.x * RPW; r0 < rows; r0 += stride) {
        const long long row = r0 + slot;
        const bool in = row < rows;  // lanes of a row behind the last compute and write nothing
        float n[NV][8], d[NV][8], o[NV][8];
        if constexpr (NV > 1) fetch_row(r0);
        const float rsn = rs;
        float2 s = {0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = 8 * (v * TPR + sub);
            unpack<TH, 8, TAIL>(hr[v], c, width, n[v]);
            unpack<TX, 8, TAIL>(yr[v], c, width, d[v]);
            if (gh) unpack<TH, 8, TAIL>(gr[v], c, width, o[v]);
            const float rsv = TAIL || c < width ? rsn : 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // columns behind the last have d = 0, and n = 0: -m * rstd may be infinite
                n[v][j] = !TAIL || c + j < width ? (n[v][j] - m) * rsv : 0.0f;
                if (in) {
                    gw[v][j] += d[v][j] * n[v][j];
                    gb[v][j] += d[v][j];
                }
                d[v][j] *= w[v][j];
                s.x += d[v][j];
                s.y += d[v][j] * n[v][j];
                if (!gh) o[v][j] = 0.0f;
            }
        }
        if constexpr (NV == 1)  // while the sums are exchanged
            if (r0 + stride < rows) fetch_row(r0 + stride);
        over_row_two<TPR>(s, red, turn);
        const float s1 = s.x / (float)width, sn = s.y / (float)width;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
#pragma unroll
            for (int j = 0; j < 8; ++j) o[v][j] += rsn * (d[v][j] - s1 - n[v][j] * sn);
            if (in) store<TH, 8, TAIL>(gx + row * width, 8 * (v * TPR + sub), width, o[v]);
        }
        turn ^= 1;
    }
    float* to = part + 2LL * blockIdx.x * width;
    if constexpr (RPW > 1) {
        __shared__ double sum[RPW][8 * TPR * NV + 2];
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[slot][8 * (v * TPR + sub) + j] = which ? gb[v][j] : gw[v][j];
            __syncthreads();
            for (int c = threadIdx.x; c < width; c += threads_of(TPR)) {
                double x = sum[0][c];
#pragma unroll
                for (int i = 1; i < RPW; ++i) x += sum[i][c];
                to[(long long)which * width + c] = (float)x;
            }
        }
    } else {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = (float)gw[v][j];
            store<F32, 8, TAIL>(to, 8 * (v * TPR + sub), width, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = (float)gb[v][j];
            store<F32, 8, TAIL>(to + width, 8 * (v * TPR + sub), width, x);
        }
    }
}

// Where the sums of the columns go: the first half into gw, the other into gb (or nowhere).
struct Weights {
    float *gw, *gb;
    int width;
    __device__ __forceinline__ void operator()(long long c, float x) const {
        if (c < width)
            gw[c] = x;
        else if (gb)
            gb[c - width] = x;
    }
};

// Workgroups of the backward, each with two rows of partial sums: enough to fill the chip, few
// enough that the sums over them stay small.  bf16, in us, 512 | 1024 | 2048 of them: 16384 x 1001
// 49 | 36 | 44, 16384 x 768 27.5 | 26.1 | 31.9, 9999 x 1536 31.5 | 30.7 | 37.6, 99991 x 128 20.3 |
// 21.2 | 26.6; 16384 x 4096 110 | 114 | 127.
inline long long parts_of(long long rows, long long width) {
    const long long need = (rows + rows_at_once(width) - 1) / rows_at_once(width);
    // 32-bit sums, beyond 8192 columns, are over 16 rows at most
    return std::max(std::min(need, width <= 2048 ? 1024LL : 512LL), width <= 8192 ? 0 : (rows + 15) / 16);
}

template <class F>
int with_rows(long long width, F f) {
    return with_tiling(width, [&](auto tpr, auto nv) {
        return width % 8 ? f(tpr, nv, std::true_type{}) : f(tpr, nv, std::false_type{});
    });
}

}  // namespace

// ================================================================ C ABI
extern "C" int layer_norm_forward(int type, int stream_type, long long rows, long long width, const void* x,
                                  const void* residual, const void* weight, const void* bias, float eps, void* y,
                                  void* h, float* mean, float* rstd, hipStream_t stream) {
    if (const int e = check_sizes(type, stream_type, rows, width)) return e;
    if (!std::isfinite(eps) || eps < 0.0f) return CFC_ERR_DT;
    if (!residual && (h || stream_type != type)) return CFC_ERR_DIM;
    if (rows == 0) return CFC_OK;
    if (!x || !weight || !y) return CFC_ERR_NULL;
    if (!fits({x, weight, bias, y}, size_of(type)) || !fits({residual, h}, size_of(stream_type)) ||
        !fits({mean, rstd}, 4))
        return CFC_ERR_DIM;
    const long long n = rows * width;
    const Range rx = bytes_of(x, n * size_of(type)), rr = bytes_of(residual, n * size_of(stream_type)),
                rh = bytes_of(h, n * size_of(stream_type));
    const bool over_x = same(rh, rx) && stream_type == type, over_r = same(rh, rr);
    const Range outs[] = {bytes_of(y, n * size_of(type)), rh, bytes_of(mean, rows * 4), bytes_of(rstd, rows * 4)};
    const Range ins[] = {bytes_of(weight, width * size_of(type)), bytes_of(bias, width * size_of(type)),
                         over_x ? Range{0, 0} : rx, over_r ? Range{0, 0} : rr};
    if (!outputs_disjoint(outs, 4, ins, 4)) return CFC_ERR_OVERLAP;
    return with_types(type, stream_type, [&](auto tx, auto th) {
        return with_rows(width, [&](auto tpr, auto nv, auto tail) {
            using TX = decltype(tx);
            using TH = decltype(th);
            constexpr int T = decltype(tpr)::value, V = decltype(nv)::value;
            constexpr bool TAIL = decltype(tail)::value;
            const long long need = (rows + rows_at_once(width) - 1) / rows_at_once(width);
            const unsigned grid = (unsigned)std::min(need, (long long)256 * 8 * 256 / threads_of(T));
            hipLaunchKernelGGL((layer_norm_kernel<TX, TH, T, V, TAIL>), dim3(grid), dim3(threads_of(T)), 0, stream, rows,
                               (int)width, (const typename TX::S*)x, (const typename TH::S*)residual,
                               (const typename TX::S*)weight, (const typename TX::S*)bias, eps, (typename TX::S*)y,
                               (typename TH::S*)h, mean, rstd);
            return launch_status();
        });
    });
}

extern "C" long long layer_norm_backward_workspace(long long rows, long long width) {
    if (check_sizes(CFC_TYPE_F32, CFC_TYPE_F32, rows, width) != CFC_OK) return -1;
    return (parts_of(rows, width) * width * 8 + 15) / 16 * 16;
}

extern "C" int layer_norm_backward(int type, int stream_type, long long rows, long long width, const void* grad_y,
                                   const void* h, const void* weight, const float* mean, const float* rstd,
                                   const void* grad_h, void* grad_x, float* grad_weight, float* grad_bias,
                                   void* workspace, long long workspace_bytes, hipStream_t stream) {
    if (const int e = check_sizes(type, stream_type, rows, width)) return e;
    if (!grad_weight) return CFC_ERR_NULL;
    const long long need = layer_norm_backward_workspace(rows, width), parts = parts_of(rows, width);
    if (rows) {
        if (!grad_y || !h || !weight || !mean || !rstd || !grad_x || !workspace) return CFC_ERR_NULL;
        if (workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 16) return CFC_ERR_DIM;
    }
    if (!fits({grad_y, weight}, size_of(type)) || !fits({h, grad_h, grad_x}, size_of(stream_type)) ||
        !fits({mean, rstd, grad_weight, grad_bias}, 4))
        return CFC_ERR_DIM;
    const long long n = rows * width;
    const Range rgh = bytes_of(grad_h, n * size_of(stream_type)), rgx = bytes_of(grad_x, n * size_of(stream_type));
    const Range outs[] = {rgx, bytes_of(grad_weight, width * 4), bytes_of(grad_bias, width * 4),
                          bytes_of(rows ? workspace : nullptr, need)};
    const Range ins[] = {bytes_of(grad_y, n * size_of(type)),
                         bytes_of(h, n * size_of(stream_type)),
                         bytes_of(rows ? weight : nullptr, width * size_of(type)),
                         bytes_of(mean, rows * 4),
                         bytes_of(rstd, rows * 4),
                         same(rgh, rgx) ? Range{0, 0} : rgh};
    if (!outputs_disjoint(outs, 4, ins, 6)) return CFC_ERR_OVERLAP;
    float* part = static_cast<float*>(workspace);
    if (rows) {
        const int e = with_types(type, stream_type, [&](auto tx, auto th) {
            return with_rows(width, [&](auto tpr, auto nv, auto tail) {
                using TX = decltype(tx);
                using TH = decltype(th);
                constexpr int T = decltype(tpr)::value, V = decltype(nv)::value;
                constexpr bool TAIL = decltype(tail)::value;
                hipLaunchKernelGGL((layer_norm_backward_kernel<TX, TH, T, V, TAIL>), dim3((unsigned)parts),
                                   dim3(threads_of(T)), 0, stream, rows, (int)width, (const typename TX::S*)grad_y,
                                   (const typename TH::S*)h, (const typename TX::S*)weight, mean, rstd,
                                   (const typename TH::S*)grad_h, (typename TH::S*)grad_x, part);
                return launch_status();
            });
        });
        if (e != CFC_OK) return e;
    }
    sum_columns(part, parts, 2 * width, Weights{grad_weight, grad_bias, (int)width}, stream);
    return launch_status();
}
