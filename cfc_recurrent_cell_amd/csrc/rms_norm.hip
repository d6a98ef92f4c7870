// rms_norm.hip -- gfx950 kernels and C ABI of the root-mean-square norm (see
// include/rms_norm.h).
//
// Memory is the bound: a row is read once into registers (8 consecutive columns
// a lane, 16 bytes of a 16-bit type), squared and summed over its lanes, and
// written from the registers.  TPR threads have a row: 16 lanes up to 128
// columns (four rows a wave), a wave up to 512, several waves beyond, which join
// their sums through LDS.  Workgroups stride over the rows with the weight in
// registers.  In bf16, where a large copy reaches 4.7 TB/s: 16384 x 4096 with a residual,
// 537 MB, in 99 us, 5.4 TB/s; its backward (with grad_h, 537 MB) in 110 us, 4.9 TB/s;
// the backward of 99991 x 128 (77 MB) in 19.8 us, 3.9 TB/s, 5 of them the column sum's
// own launch; 32 rows of 4096 to e4m3 in 4.4 us on the GPU, a launch's time.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "elements.h"
#include "rms_norm.h"

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Columns c ... c + 7 of a row; zero from `width` on.
template <class TY>
__device__ __forceinline__ void load8(const typename TY::S* row, int c, int width, bool vec, float (&x)[8]) {
    if (vec) {
        const bool in = c < width;
        if constexpr (sizeof(typename TY::S) == 4) {
            f32x4 a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
            if (in) {
                a = *reinterpret_cast<const f32x4*>(row + c);
                b = *reinterpret_cast<const f32x4*>(row + c + 4);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = a[j], x[j + 4] = b[j];
        } else {
            u32x4 a = {0, 0, 0, 0};
            if (in) a = *reinterpret_cast<const u32x4*>(row + c);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = TY::load(__builtin_bit_cast(typename TY::S,
                                                   (uint16_t)(j & 1 ? a[j >> 1] >> 16 : a[j >> 1] & 0xffff)));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = c + j < width ? TY::load(row[c + j]) : 0.0f;
    }
}
template <class TY>
__device__ __forceinline__ void store8(typename TY::S* row, int c, int width, bool vec, const float (&x)[8]) {
    if (vec) {
        if (c >= width) return;
        if constexpr (sizeof(typename TY::S) == 4) {
            *reinterpret_cast<f32x4*>(row + c) = f32x4{x[0], x[1], x[2], x[3]};
            *reinterpret_cast<f32x4*>(row + c + 4) = f32x4{x[4], x[5], x[6], x[7]};
        } else {
            u32x4 a;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                a[j] = (uint32_t)__builtin_bit_cast(uint16_t, TY::store(x[2 * j])) |
                       (uint32_t)__builtin_bit_cast(uint16_t, TY::store(x[2 * j + 1])) << 16;
            *reinterpret_cast<u32x4*>(row + c) = a;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < width) row[c + j] = TY::store(x[j]);
    }
}

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

// E4: y in e4m3 with the scale of each `group` columns (0: the row).
template <class TX, class TH, int TPR, int NV, bool E4>
__global__ __launch_bounds__(threads_of(TPR)) void rms_norm_kernel(
    long long rows, int width, const typename TX::S* x, const typename TH::S* residual,
    const typename TX::S* __restrict__ weight, float eps, void* __restrict__ y, float* __restrict__ scales,
    typename TH::S* h, float* __restrict__ rstd, int group, bool vec) {
    constexpr int RPW = threads_of(TPR) / TPR;
    __shared__ float red[4][16];
    const int sub = threadIdx.x % TPR;
    float w[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) load8<TX>(weight, 8 * (v * TPR + sub), width, vec, w[v]);
    int turn = 0;
    for (long long r0 = (long long)blockIdx.x * RPW; r0 < rows; r0 += (long long)gridDim.x * RPW) {
        const long long row = r0 + threadIdx.x / TPR;
        const bool in = row < rows;  // lanes of a row behind the last compute and write nothing
        const long long at = (in ? row : rows - 1) * width;
        float a[NV][8];
        float ss = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) load8<TX>(x + at, 8 * (v * TPR + sub), width, vec, a[v]);
        if (residual) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float b[8];
                const int c = 8 * (v * TPR + sub);
                load8<TH>(residual + at, c, width, vec, b);
#pragma unroll
                for (int j = 0; j < 8; ++j) a[v][j] = TH::load(TH::store(a[v][j] + b[j]));
                if (h && in) store8<TH>(h + at, c, width, vec, a[v]);
            }
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j) ss += a[v][j] * a[v][j];
        ss = over_row<TPR>(ss, [](float p, float q) { return p + q; }, red, turn);
        const float rs = 1.0f / sqrtf(ss / (float)width + eps);
        if (rstd && sub == 0 && in) rstd[row] = rs;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j) a[v][j] = a[v][j] * rs * w[v][j];
        if constexpr (!E4) {
            if (in) {
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    store8<TX>(static_cast<typename TX::S*>(y) + at, 8 * (v * TPR + sub), width, vec, a[v]);
            }
        } else {
            const int groups = group ? (width + group - 1) / group : 1;
            float top[NV];
            float all = 0.0f;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                top[v] = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) top[v] = fmaxf(top[v], fabsf(a[v][j]));
                all = fmaxf(all, top[v]);
            }
            if (group == 0) {
                all = over_row<TPR>(all, [](float p, float q) { return fmaxf(p, q); }, red, turn + 2);
#pragma unroll
                for (int v = 0; v < NV; ++v) top[v] = all;
            } else {
                // group / 8 neighbouring lanes have a group's columns
                const int lanes = min(group / 8, min(TPR, 64));
                for (int off = 1; off < lanes; off <<= 1)
#pragma unroll
                    for (int v = 0; v < NV; ++v) top[v] = fmaxf(top[v], __shfl_xor(top[v], off));
            }
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = 8 * (v * TPR + sub);
                const float t = top[v] == 0.0f ? 1.0f : top[v];
                const bool head = group ? c % group == 0 : c == 0;
                if (in && head && c < width) scales[row * groups + (group ? c / group : 0)] = t / 448.0f;
                // a power of two keeps 448 / t finite where t is next to nothing
                const float up = t < 1e-30f ? 0x1p64f : 1.0f;
                const float inv = 448.0f / (t * up);
                uint32_t two[2] = {0, 0};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    two[i] = __builtin_amdgcn_cvt_pk_fp8_f32(a[v][4 * i] * up * inv, a[v][4 * i + 1] * up * inv, two[i],
                                                             false);
                    two[i] = __builtin_amdgcn_cvt_pk_fp8_f32(a[v][4 * i + 2] * up * inv, a[v][4 * i + 3] * up * inv,
                                                             two[i], true);
                }
                uint8_t* to = static_cast<uint8_t*>(y) + at;
                if (in) {
                    if (vec) {
                        if (c < width) *reinterpret_cast<u32x2*>(to + c) = u32x2{two[0], two[1]};
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (c + j < width) to[c + j] = (uint8_t)(two[j >> 2] >> (8 * (j & 3)));
                    }
                }
            }
        }
        turn ^= 1;
    }
}

// The weight gradient's terms are summed over the workgroup's rows in registers,
// then over its row slots through LDS, into row blockIdx.x of `part`; reduce_axis0
// sums those.  In 64 bits, since a slot's rows are up to a 512th of all: of 2^19 rows
// alike, a 32-bit sum is off by 7.6e-6 of its size, this one by less than 2.4e-7.
// 16384 x 4096 takes 109.6 us for it and 107.8 in 32 bits, 99991 x 128 21.2 and 20.8.
template <class TX, class TH, int TPR, int NV>
__global__ __launch_bounds__(threads_of(TPR)) void rms_norm_backward_kernel(
    long long rows, int width, const typename TX::S* __restrict__ gy, const typename TH::S* __restrict__ h,
    const typename TX::S* __restrict__ weight, const float* __restrict__ rstd, const typename TH::S* gh,
    typename TH::S* gx, float* __restrict__ part, bool vec) {
    constexpr int RPW = threads_of(TPR) / TPR;
    __shared__ float red[2][16];
    const int sub = threadIdx.x % TPR, slot = threadIdx.x / TPR;
    float w[NV][8];
    double gw[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        load8<TX>(weight, 8 * (v * TPR + sub), width, vec, w[v]);
#pragma unroll
        for (int j = 0; j < 8; ++j) gw[v][j] = 0.0;
    }
    int turn = 0;
    for (long long r0 = (long long)blockIdx.x * RPW; r0 < rows; r0 += (long long)gridDim.x * RPW) {
        const long long row = r0 + slot;
        const bool in = row < rows;
        const long long at = (in ? row : rows - 1) * width;
        const float rs = in ? rstd[row] : 0.0f;
        float n[NV][8], d[NV][8];
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            load8<TH>(h + at, 8 * (v * TPR + sub), width, vec, n[v]);
            load8<TX>(gy + at, 8 * (v * TPR + sub), width, vec, d[v]);
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                n[v][j] *= rs;
                if (in) gw[v][j] += d[v][j] * n[v][j];
                d[v][j] *= w[v][j];
                s += d[v][j] * n[v][j];
            }
        s = over_row<TPR>(s, [](float p, float q) { return p + q; }, red, turn) / (float)width;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = 8 * (v * TPR + sub);
            float o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = rs * (d[v][j] - n[v][j] * s);
            if (gh) {
                float e[8];
                load8<TH>(gh + at, c, width, vec, e);
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] += e[j];
            }
            if (in) store8<TH>(gx + at, c, width, vec, o);
        }
        turn ^= 1;
    }
    if constexpr (RPW > 1) {
        __shared__ float sum[RPW][8 * TPR * NV + 4];
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[slot][8 * (v * TPR + sub) + j] = (float)gw[v][j];
        __syncthreads();
        for (int c = threadIdx.x; c < width; c += threads_of(TPR)) {
            double x = sum[0][c];
#pragma unroll
            for (int i = 1; i < RPW; ++i) x += sum[i][c];
            part[(long long)blockIdx.x * width + c] = (float)x;
        }
    } else {
        // rows of `part` are aligned where the arguments' rows are
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = (float)gw[v][j];
            store8<F32>(part + (long long)blockIdx.x * width, 8 * (v * TPR + sub), width, vec, x);
        }
    }
}

// ---------------------------------------------------------- host helpers
inline bool is_type(int t) { return t == CFC_TYPE_F32 || t == CFC_TYPE_BF16 || t == CFC_TYPE_F16; }

int check_sizes(int type, int stream_type, long long rows, long long width) {
    if (!is_type(type) || (stream_type != type && stream_type != CFC_TYPE_F32)) return CFC_ERR_UNSUPPORTED;
    if (rows < 0 || width < 1) return CFC_ERR_DIM;
    if (width > RMS_NORM_MAX_WIDTH) return CFC_ERR_UNSUPPORTED;
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
inline bool aligned(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (reinterpret_cast<uintptr_t>(p) % 16) return false;
    return true;
}

template <bool E4>
int run_forward(int type, int stream_type, long long rows, long long width, const void* x, const void* residual,
                const void* weight, float eps, int group, void* y, float* scales, void* h, float* rstd,
                hipStream_t stream) {
    if (const int e = check_sizes(type, stream_type, rows, width)) return e;
    if (!std::isfinite(eps) || eps < 0.0f) return CFC_ERR_DT;
    if (E4 && group != 0 && (group < 16 || group > 512 || (group & (group - 1)))) return CFC_ERR_DIM;
    if (!residual && (h || stream_type != type)) return CFC_ERR_DIM;
    if (rows == 0) return CFC_OK;
    if (!x || !weight || !y || (E4 && !scales)) return CFC_ERR_NULL;
    const long long n = rows * width, groups = group ? (width + group - 1) / group : 1;
    const Range rx = bytes_of(x, n * size_of(type)), rr = bytes_of(residual, n * size_of(stream_type)),
                rh = bytes_of(h, n * size_of(stream_type));
    const bool over_x = same(rh, rx) && stream_type == type, over_r = same(rh, rr);
    const Range outs[] = {bytes_of(y, n * (E4 ? 1 : size_of(type))), rh, bytes_of(rstd, rows * 4),
                          bytes_of(E4 ? scales : nullptr, rows * groups * 4)};
    const Range ins[] = {bytes_of(weight, width * size_of(type)), over_x ? Range{0, 0} : rx,
                         over_r ? Range{0, 0} : rr};
    if (!outputs_disjoint(outs, 4, ins, 3)) return CFC_ERR_OVERLAP;
    const bool vec = width % 8 == 0 && aligned({x, residual, weight, y, h});
    return with_types(type, stream_type, [&](auto tx, auto th) {
        return with_tiling(width, [&](auto tpr, auto nv) {
            using TX = decltype(tx);
            using TH = decltype(th);
            constexpr int T = decltype(tpr)::value, V = decltype(nv)::value;
            const long long need = (rows + rows_at_once(width) - 1) / rows_at_once(width);
            const unsigned grid = (unsigned)std::min(need, (long long)256 * 8 * 256 / threads_of(T));
            hipLaunchKernelGGL((rms_norm_kernel<TX, TH, T, V, E4>), dim3(grid), dim3(threads_of(T)), 0, stream, rows,
                               (int)width, (const typename TX::S*)x, (const typename TH::S*)residual,
                               (const typename TX::S*)weight, eps, y, scales, (typename TH::S*)h, rstd, group, vec);
            return launch_status();
        });
    });
}

// Workgroups of the backward, each with a row of partial weight gradients.
inline long long parts_of(long long rows, long long width) {
    const long long need = (rows + rows_at_once(width) - 1) / rows_at_once(width);
    // narrow rows' partial sums are small, and more workgroups hide more of the loads:
    // 99991 x 128 with 512 23.7 us, with 1024 21.5, with 2048 25.3; 32768 x 2048 135, 86
    // and 91; 16384 x 4096 86, 89 and 100
    return std::min(need, width <= 2048 ? 1024LL : 512LL);
}

}  // namespace

// ================================================================ C ABI
extern "C" int rms_norm_forward(int type, int stream_type, long long rows, long long width, const void* x,
                                const void* residual, const void* weight, float eps, void* y, void* h, float* rstd,
                                hipStream_t stream) {
    return run_forward<false>(type, stream_type, rows, width, x, residual, weight, eps, 0, y, nullptr, h, rstd, stream);
}

extern "C" int rms_norm_forward_e4m3(int type, int stream_type, long long rows, long long width, const void* x,
                                     const void* residual, const void* weight, float eps, int group, void* y,
                                     float* scales, void* h, float* rstd, hipStream_t stream) {
    return run_forward<true>(type, stream_type, rows, width, x, residual, weight, eps, group, y, scales, h, rstd,
                             stream);
}

extern "C" long long rms_norm_backward_workspace(long long rows, long long width) {
    if (check_sizes(CFC_TYPE_F32, CFC_TYPE_F32, rows, width) != CFC_OK) return -1;
    return (parts_of(rows, width) * width * 4 + 15) / 16 * 16;
}

extern "C" int rms_norm_backward(int type, int stream_type, long long rows, long long width, const void* grad_y,
                                 const void* h, const void* weight, const float* rstd, const void* grad_h,
                                 void* grad_x, float* grad_weight, void* workspace, long long workspace_bytes,
                                 hipStream_t stream) {
    if (const int e = check_sizes(type, stream_type, rows, width)) return e;
    if (!grad_weight) return CFC_ERR_NULL;
    if (rows == 0) return reduce_axis0(nullptr, 0, width, grad_weight, stream);
    if (!grad_y || !h || !weight || !rstd || !grad_x || !workspace) return CFC_ERR_NULL;
    const long long need = rms_norm_backward_workspace(rows, width), parts = parts_of(rows, width);
    if (workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 16) return CFC_ERR_DIM;
    const long long n = rows * width;
    const Range rgh = bytes_of(grad_h, n * size_of(stream_type)), rgx = bytes_of(grad_x, n * size_of(stream_type));
    const Range outs[] = {rgx, bytes_of(grad_weight, width * 4), bytes_of(workspace, need)};
    const Range ins[] = {bytes_of(grad_y, n * size_of(type)), bytes_of(h, n * size_of(stream_type)),
                         bytes_of(weight, width * size_of(type)), bytes_of(rstd, rows * 4),
                         same(rgh, rgx) ? Range{0, 0} : rgh};
    if (!outputs_disjoint(outs, 3, ins, 5)) return CFC_ERR_OVERLAP;
    const bool vec = width % 8 == 0 && aligned({grad_y, h, weight, grad_h, grad_x});
    float* part = static_cast<float*>(workspace);
    const int e = with_types(type, stream_type, [&](auto tx, auto th) {
        return with_tiling(width, [&](auto tpr, auto nv) {
            using TX = decltype(tx);
            using TH = decltype(th);
            constexpr int T = decltype(tpr)::value, V = decltype(nv)::value;
            hipLaunchKernelGGL((rms_norm_backward_kernel<TX, TH, T, V>), dim3((unsigned)parts), dim3(threads_of(T)), 0,
                               stream, rows, (int)width, (const typename TX::S*)grad_y, (const typename TH::S*)h,
                               (const typename TX::S*)weight, rstd, (const typename TH::S*)grad_h,
                               (typename TH::S*)grad_x, part, vec);
            return launch_status();
        });
    });
    if (e != CFC_OK) return e;
    return reduce_axis0(part, parts, width, grad_weight, stream);
}
