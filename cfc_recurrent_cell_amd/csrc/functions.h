// functions.h -- the gates' functions in 32 bits (short_conv.hip, selective_scan.hip).
#pragma once

#include <hip/hip_runtime.h>

namespace {

constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// exp(x) for x <= 0: the rounding of x log2(e) is put right, so that a step of a
// thousandth, exp(-7), is as exact as one of one.
__device__ __forceinline__ float exp_of(float x) {
    constexpr float low = 1.92596299e-8f;  // log2(e) - kLog2e
    x = x < -1000.0f ? -1000.0f : x;  // (a NaN stays one)
    const float t = x * kLog2e, e = fmaf(x, low, fmaf(x, kLog2e, -t));
    const float p = exp2_of(t);
    return fmaf(p, e * kLn2, p);
}
__device__ __forceinline__ float reciprocal(float x) { return __builtin_amdgcn_rcpf(x); }
// 1 / (1 + exp(-x)), with e = exp(-|x|)
__device__ __forceinline__ float sigmoid_of(float x, float e) {
    const float r = reciprocal(1.0f + e);
    return x >= 0.0f ? r : e * r;
}
__device__ __forceinline__ float sigmoid_of(float x) { return sigmoid_of(x, exp_of(-fabsf(x))); }
// The same for what is rounded to a type of 16 bits: off by |x| 2^-24, where exp_of's and the
// choice of sides cost as much again.
template <class TY>
__device__ __forceinline__ float gate_of(float x) {
    if constexpr (sizeof(typename TY::S) == 4)
        return sigmoid_of(x);
    else
        return reciprocal(1.0f + exp2_of(-kLog2e * x));
}
// max(x, 0) + log(1 + e) with e = exp(-|x|); the logarithm as 2 artanh(e / (2 + e)) by its
// series, whose argument is at most a third, so that small results lose nothing.
__device__ __forceinline__ float softplus_of(float x, float e) {
    const float s = e * reciprocal(2.0f + e), z = s * s;
    float p = 1.0f / 15;
    p = fmaf(p, z, 1.0f / 13);
    p = fmaf(p, z, 1.0f / 11);
    p = fmaf(p, z, 1.0f / 9);
    p = fmaf(p, z, 1.0f / 7);
    p = fmaf(p, z, 1.0f / 5);
    p = fmaf(p, z, 1.0f / 3);
    p = fmaf(p, z, 1.0f);
    return fmaf(2.0f * s, p, fmaxf(x, 0.0f));
}
__device__ __forceinline__ float softplus_of(float x) { return softplus_of(x, exp_of(-fabsf(x))); }

}  // namespace
