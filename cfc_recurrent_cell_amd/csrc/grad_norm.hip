// grad_norm.hip -- gfx950 kernels and C ABI of the norm over many gradients and of
// clipping to it (see include/grad_norm.h).
//
// Memory is the bound: every gradient is read for the norm, and read again and written
// for the clipping.  Tensors go by the batch: a launch takes up to kBatch of them in its
// arguments, so nothing is copied to the GPU, and its workgroups stride over the chunks of
// all of them.  Each workgroup of the first pass leaves one partial sum of squares; those
// of the second sum the partial ones again, each for itself, which costs less than a
// launch.  62 tensors of 513 MB: 123 us for the squares and 175 for the clipping, 1540 MB at
// 5.2 TB/s; two tensors of the smallest model 3.8 and 4.1 us, of 17 for the call on the host.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>
#include <vector>

#include "elements.h"
#include "grad_norm.h"

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 112;          // tensors of a launch, whose arguments have 4 KB
constexpr int kParts = 2048;         // workgroups of a launch, at most
constexpr int kStep = 8 * kThreads;  // elements that a workgroup takes at once

struct Batch {
    const void* grad[kBatch];
    void* out[kBatch];
    long long numel[kBatch];
    unsigned chunk0[kBatch];  // the tensor's first chunk among the batch's
    uint8_t type[kBatch];
    int count;
    unsigned chunks;
    int steps;  // kStep elements of a chunk
};
static_assert(sizeof(Batch) + 64 <= 4096, "a launch's arguments");

// The tensor that a chunk belongs to: the last one that begins there or before (those
// without elements begin where the next one does).
__device__ __forceinline__ int tensor_of(const Batch& b, unsigned chunk) {
    int lo = 0, n = b.count;
    while (n > 1) {
        const int half = n / 2;
        if (b.chunk0[lo + half] <= chunk) {
            lo += half;
            n -= half;
        } else {
            n = half;
        }
    }
    return lo;
}

// Calls f(first element, eight as they lie in memory, whether some are missing, how many there are) for
// a thread's eights of [at, end); kUnroll of them are loaded at once.
constexpr int kUnroll = 4;
template <class TY, class F>
__device__ __forceinline__ void each_eight(const void* grad, long long at, long long end, F f) {
    const auto* p = static_cast<const typename TY::S*>(grad);
    long long i = at + 8 * threadIdx.x;
    for (; i + (kUnroll - 1) * kStep + 8 <= end; i += kUnroll * kStep) {
        Packed<TY, 8> e[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) e[k] = fetch<TY, 8, false>(p + i + k * kStep, 0, 8);
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) f(i + k * kStep, e[k], std::false_type{}, 8);
    }
    for (; i < end; i += kStep) {
        const int n = (int)min(end - i, 8LL);
        f(i, fetch<TY, 8, true>(p + i, 0, n), std::true_type{}, n);
    }
}
template <class TY>
__device__ __forceinline__ void squares(const void* grad, long long at, long long end, double& s0, double& s1) {
    each_eight<TY>(grad, at, end, [&](long long, const Packed<TY, 8>& e, auto tail, int n) {
        float x[8];
        unpack<TY, 8, decltype(tail)::value>(e, 0, n, x);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const double a = x[j], b = x[j + 1];
            s0 += a * a;
            s1 += b * b;
        }
    });
}

__device__ __forceinline__ double over_block(double x, double* red) {
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) x += __shfl_xor(x, off);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
    __syncthreads();
    x = red[0];
#pragma unroll
    for (int i = 1; i < kThreads / 64; ++i) x += red[i];
    return x;
}

__global__ __launch_bounds__(kThreads) void squares_kernel(Batch b, double* __restrict__ part) {
    __shared__ double red[kThreads / 64];
    double s0 = 0.0, s1 = 0.0;
    for (unsigned chunk = blockIdx.x; chunk < b.chunks; chunk += gridDim.x) {
        const int t = tensor_of(b, chunk);
        const long long at = (long long)(chunk - b.chunk0[t]) * b.steps * kStep;
        const long long end = min(at + (long long)b.steps * kStep, b.numel[t]);
        if (b.type[t] == CFC_TYPE_F32)
            squares<F32>(b.grad[t], at, end, s0, s1);
        else if (b.type[t] == CFC_TYPE_BF16)
            squares<BF16>(b.grad[t], at, end, s0, s1);
        else
            squares<F16>(b.grad[t], at, end, s0, s1);
    }
    const double s = over_block(s0 + s1, red);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// The sum of n partial sums, the same bits in every thread.
__device__ __forceinline__ double total_of(const double* __restrict__ part, int n, double* red) {
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads) s += part[i];
    return over_block(s, red);
}

// The norm, and the partial sums as one.
__global__ __launch_bounds__(kThreads) void total_kernel(const double* __restrict__ part, int n, float* __restrict__ norm,
                                                         double* __restrict__ total) {
    __shared__ double red[kThreads / 64];
    const double s = total_of(part, n, red);
    if (threadIdx.x == 0) {
        *norm = (float)sqrt(s);
        if (total) *total = s;
    }
}

template <class TY>
__device__ __forceinline__ void scale(const void* grad, void* out, long long at, long long end, float factor) {
    auto* o = static_cast<typename TY::S*>(out);
    each_eight<TY>(grad, at, end, [&](long long i, const Packed<TY, 8>& e, auto tail, int n) {
        float x[8];
        unpack<TY, 8, decltype(tail)::value>(e, 0, n, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= factor;
        store<TY, 8, decltype(tail)::value>(o + i, 0, n, x);
    });
}

__global__ __launch_bounds__(kThreads) void clip_kernel(Batch b, const double* __restrict__ part, int parts,
                                                        float max_norm, float* __restrict__ norm) {
    __shared__ double red[kThreads / 64];
    const double whole = sqrt(total_of(part, parts, red));
    const float given = (float)whole;  // the norm that the caller gets: infinite where it passes 32 bits
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = given;
    double ratio = isinf(max_norm) ? 1.0 : isinf(given) ? 0.0 : (double)max_norm / (whole + 1e-6);
    if (ratio > 1.0) ratio = 1.0;  // not where it is NaN
    if (isinf(max_norm) && whole != whole) ratio = whole;
    const float factor = (float)ratio;
    // from the last chunk on, which the norm has read last and the last-level cache still holds:
    // 513 MB 299 us instead of 306
    for (unsigned k = blockIdx.x; k < b.chunks; k += gridDim.x) {
        const unsigned chunk = b.chunks - 1 - k;
        const int t = tensor_of(b, chunk);
        const long long at = (long long)(chunk - b.chunk0[t]) * b.steps * kStep;
        const long long end = min(at + (long long)b.steps * kStep, b.numel[t]);
        if (b.type[t] == CFC_TYPE_F32)
            scale<F32>(b.grad[t], b.out[t], at, end, factor);
        else if (b.type[t] == CFC_TYPE_BF16)
            scale<BF16>(b.grad[t], b.out[t], at, end, factor);
        else
            scale<F16>(b.grad[t], b.out[t], at, end, factor);
    }
}

// ---------------------------------------------------------- host helpers
inline int batches_of(int count) { return count / kBatch + (count % kBatch != 0); }

int check_tensors(const grad_tensor_t* tensors, int count, const float* norm, const void* workspace,
                  long long workspace_bytes, bool clip) {
    if (count < 0) return CFC_ERR_DIM;
    if (!norm || (count && !tensors) || !workspace) return CFC_ERR_NULL;
    const long long need = grad_norm_workspace(count);
    if (workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 16 || !fits({norm}, 4)) return CFC_ERR_DIM;
    struct Span {
        Range r;
        int tensor;
        bool out;
    };
    std::vector<Span> spans;
    spans.reserve((size_t)count * (clip ? 2 : 1) + 2);
    auto add = [&](const void* p, long long bytes, int tensor, bool out) {
        if (p && bytes) spans.push_back(Span{bytes_of(p, bytes), tensor, out});
    };
    add(norm, 4, -1, true);
    add(workspace, need, -2, true);
    for (int i = 0; i < count; ++i) {
        const grad_tensor_t& t = tensors[i];
        if (t.type != CFC_TYPE_F32 && t.type != CFC_TYPE_BF16 && t.type != CFC_TYPE_F16) return CFC_ERR_UNSUPPORTED;
        if (t.numel < 0 || t.numel > (1LL << 42)) return CFC_ERR_DIM;
        if (t.numel && (!t.grad || (clip && !t.out))) return CFC_ERR_NULL;
        const int size = size_of(t.type);
        if (!fits({t.grad}, size) || (clip && !fits({t.out}, size))) return CFC_ERR_DIM;
        add(t.grad, t.numel * size, i, false);
        if (clip) add(t.out, t.numel * size, i, true);
    }
    // Outputs share no memory with anything but, as a whole, their own tensor's gradient.  In
    // the order of their beginnings, a span overlaps those before that it begins within.
    std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.r.lo < b.r.lo; });
    std::vector<const Span*> open;
    open.reserve(spans.size());
    for (const Span& s : spans) {
        open.erase(std::remove_if(open.begin(), open.end(), [&](const Span* o) { return o->r.hi <= s.r.lo; }), open.end());
        for (const Span* o : open)
            if ((o->out || s.out) && !(o->tensor == s.tensor && o->out != s.out && same(o->r, s.r))) return CFC_ERR_OVERLAP;
        open.push_back(&s);
    }
    return CFC_OK;
}

// The batch of tensors from `at` on.  Chunks as short as one step where there is little to
// do, so that all CUs have some of it, and longer ones where a workgroup has many (513 MB of
// bf16 in chunks of 16 | 4 | 1 steps: 298 | 299 | 420 us).
Batch batch_of(const grad_tensor_t* tensors, int count, int at) {
    Batch b;
    b.count = std::min(kBatch, count - at);
    long long all = 0;
    for (int i = 0; i < b.count; ++i) all += tensors[at + i].numel;
    b.steps = (int)std::min(16LL, std::max(1LL, all / kStep / (2 * kParts)));
    while (all / kStep / b.steps > (1LL << 31)) b.steps *= 2;
    long long chunks = 0;
    for (int i = 0; i < b.count; ++i) {
        const grad_tensor_t& t = tensors[at + i];
        b.grad[i] = t.grad;
        b.out[i] = t.out;
        b.numel[i] = t.numel;
        b.type[i] = (uint8_t)t.type;
        b.chunk0[i] = (unsigned)chunks;
        chunks += (t.numel + (long long)b.steps * kStep - 1) / ((long long)b.steps * kStep);
    }
    b.chunks = (unsigned)chunks;
    return b;
}
inline int blocks_of(const Batch& b) { return (int)std::max(1u, std::min(b.chunks, (unsigned)kParts)); }

int run(const grad_tensor_t* tensors, int count, bool clip, float max_norm, float* norm, void* workspace,
        hipStream_t stream) {
    double* part = static_cast<double*>(workspace);
    int parts = 0;
    const int batches = batches_of(count);
    for (int i = 0; i < batches; ++i) {
        const Batch b = batch_of(tensors, count, i * kBatch);
        if (b.chunks == 0) continue;
        const int blocks = blocks_of(b);
        hipLaunchKernelGGL(squares_kernel, dim3(blocks), dim3(kThreads), 0, stream, b, part + parts);
        parts += blocks;
    }
    // several batches' partial sums are one before every workgroup reads them
    const bool joined = !clip || parts == 0 || batches > 1;
    double* total = part + (long long)batches * kParts;
    if (joined)
        hipLaunchKernelGGL(total_kernel, dim3(1), dim3(kThreads), 0, stream, part, parts, norm, clip ? total : nullptr);
    if (clip && parts) {
        for (int i = batches - 1; i >= 0; --i) {
            const Batch b = batch_of(tensors, count, i * kBatch);
            if (b.chunks == 0) continue;
            hipLaunchKernelGGL(clip_kernel, dim3(blocks_of(b)), dim3(kThreads), 0, stream, b, joined ? total : part,
                               joined ? 1 : parts, max_norm, joined ? nullptr : norm);
        }
    }
    return launch_status();
}

}  // namespace

// ================================================================ C ABI
extern "C" long long grad_norm_workspace(int count) {
    return count < 0 ? -1 : ((long long)batches_of(count) * kParts + 2) * 8;
}

extern "C" int grad_norm(const grad_tensor_t* tensors, int count, float* norm, void* workspace,
                         long long workspace_bytes, hipStream_t stream) try {
    if (const int e = check_tensors(tensors, count, norm, workspace, workspace_bytes, false)) return e;
    return run(tensors, count, false, 0.0f, norm, workspace, stream);
} catch (const std::bad_alloc&) {
    return CFC_ERR_DIM;
}

extern "C" int clip_grad_norm(const grad_tensor_t* tensors, int count, float max_norm, float* norm, void* workspace,
                              long long workspace_bytes, hipStream_t stream) try {
    if (!(max_norm >= 0.0f)) return CFC_ERR_DT;
    if (const int e = check_tensors(tensors, count, norm, workspace, workspace_bytes, true)) return e;
    return run(tensors, count, true, max_norm, norm, workspace, stream);
} catch (const std::bad_alloc&) {
    return CFC_ERR_DIM;
}
