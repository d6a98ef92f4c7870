// sequences.h -- where a call's sequences lie among its token rows (short_conv.hip,
// selective_scan.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>

#include "elements.h"

namespace {

struct Sequences {
    const int* offsets;  // or null: n_seq of seq_len rows each
    int n_seq, seq_len, n_tokens;
};

// Rows [first, end) of sequence s, within the tokens whatever the offsets say.
__device__ __forceinline__ void span_of(const Sequences& q, int s, int& first, int& end) {
    if (!q.offsets) {
        first = s * q.seq_len;
        end = first + q.seq_len;
        return;
    }
    first = min(max(__builtin_amdgcn_readfirstlane(q.offsets[s]), 0), q.n_tokens);
    end = min(max(__builtin_amdgcn_readfirstlane(q.offsets[s + 1]), first), q.n_tokens);
}

// The last sequence that begins at row t or before (0 if none does), by a whole wave: 64
// beginnings are looked at at once, so two rounds do for 4096 sequences.
__device__ __forceinline__ int sequence_of(const Sequences& q, int t) {
    if (!q.offsets) return min(t / q.seq_len, q.n_seq - 1);
    const int lane = threadIdx.x & 63;
    int lo = 0, n = q.n_seq;
    while (n > 1) {
        const int step = (n + 63) / 64, i = lane * step;
        const unsigned long long m = __ballot(i < n && q.offsets[lo + min(i, n - 1)] <= t);
        const int k = max(__popcll(m), 1) - 1;
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}

// The first row from `from` on, of `rows` in all, that names `slot`, or `rows`; by a whole wave.  Rows
// of a step that name one slot are taken one after the other by the waves of the first of them, so
// each wave looks through all the slots: for 4096 channels x 16 states in bf16 256 rows of the scan
// take 34 us with slots and 31 without, 1024 146 and 104, 4096 979 and 422; 4096 rows of the
// convolution of 8192 channels 357 and 94.
__device__ __forceinline__ int row_of_slot(const int* slots, int slot, int from, int rows) {
    const int lane = threadIdx.x & 63;
    for (int j = from; j < rows; j += 64) {
        const unsigned long long m = __ballot(j + lane < rows && slots[min(j + lane, rows - 1)] == slot);
        if (m) return j + __builtin_ctzll(m);
    }
    return rows;
}

// ---------------------------------------------------------- host helpers
inline bool mul_ok(long long a, long long b, long long* r) {
    if (a < 0 || b < 0) return false;
    if (a != 0 && b > (LLONG_MAX / 16) / a) return false;
    *r = a * b;
    return true;
}

// Bytes from the first to the last element of a strided [rows, groups, dim] array.
inline bool extent(long long rows, long long groups, long long dim, long long st, long long sg, int size, long long* r) {
    long long x, y;
    *r = 0;
    if (rows == 0) return true;
    return mul_ok(rows - 1, st, &x) && mul_ok(groups - 1, sg, &y) && mul_ok(x + y + dim, size, r);
}

inline int check_sequences(const int* offsets, int n_seq, int seq_len, long long n_tokens, Sequences* q) {
    if (n_seq < 0 || n_tokens < 0) return CFC_ERR_DIM;
    if (n_tokens > INT_MAX) return CFC_ERR_UNSUPPORTED;
    if (!offsets) {
        if (seq_len < 0 || (long long)n_seq * seq_len != n_tokens) return CFC_ERR_DIM;
    } else if (n_seq == INT_MAX) {
        return CFC_ERR_UNSUPPORTED;
    }
    *q = Sequences{offsets, n_seq, offsets ? 0 : seq_len, n_seq ? (int)n_tokens : 0};
    return CFC_OK;
}
inline Range offsets_range(const Sequences& q) {
    return bytes_of(q.offsets, q.offsets ? ((long long)q.n_seq + 1) * 4 : 0);
}

}  // namespace
