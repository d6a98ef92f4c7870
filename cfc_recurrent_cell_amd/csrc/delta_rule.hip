// delta_rule.hip -- gfx950 kernels and C ABI of the gated delta rule (see
// include/delta_rule.h).
//
// The chunked form.  Over a chunk of C = 64 tokens that starts from state S0,
// with G_i the sum of the chunk's decays up to token i, gamma_i = exp(G_i),
// e_i = exp(G_63 - G_i), Gamma_ij = exp(G_i - G_j) for i >= j, the recurrence is
//
//   L_ij = beta_i Gamma_ij k_i.k_j  (i > j),   T = (I + L)^-1 diag(beta)
//   U    = T (V - diag(gamma) K S0)
//   O    = scale diag(gamma) Q S0 + M U,       M_ij = scale Gamma_ij q_i.k_j (i >= j)
//   S1   = gamma_63 S0 + K^T diag(e) U
//
// so a chunk is a handful of matrix products, and only S0 -> S1 runs along the
// sequence.  All decays are exponentials of sums of non-positive numbers (for
// g <= 0), never of their negatives, so none overflows; the sums are held in 64
// bits, since differences of large ones count.
//
// Arithmetic.  Products run on the bf16 matrix cores with 32-bit sums, at 32-bit
// accuracy: a float is the sum of three bf16 numbers of 8 bits each, exactly, and a
// product takes the six pairs of parts that reach above 2^-24.  Each part is what is
// left, rounded: the pairs left out are then below 2^-25 and of both signs, where parts that
// are cut off leave out 2^-24 on average and always of one sign (as many
// instructions; gradients of 256 x 64 in fp32 off by 3.1e-7 of their size where cut
// off, by 2.8e-7 rounded).  bf16 inputs are one part, fp16 two, float32 three.  The
// matrix cores' own 32-bit form has 1/16 of the rate of bf16, so even six
// products of parts are 2.7 times faster.  That holds for o of 16-bit types too: Q S0
// and M U can be far larger than their sum (a key's old value is taken back), so two
// parts of each are not enough for it.
//
// Kernels
//   delta_prep_kernel      for all chunks at once: T, M (transposed for the
//       gradients) and the parts of K, Q, K^T, Q^T, all stored in the order in
//       which the matrix cores' operands lie in a wave's registers, so that the
//       chain below loads them 16 bytes a lane, without masks
//   delta_chain_kernel     along each sequence, for a tile of dim_v: O and the states
//   delta_chains_kernel    for the gradients: the states' chain again, keeping U and
//       every chunk's S0, and the gradients' chain from the last chunk to the first
//   delta_grads_kernel     for all chunks at once: grad_q, grad_k, grad_g, grad_beta
//   delta_token_kernel     the recurrence token by token (a decode step, and
//       sequences too short for chunks)
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "elements.h"
#include "delta_rule.h"

namespace {

constexpr int kC = 64;        // tokens of a chunk
constexpr int kThreads = 256; // 4 wave64

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// ------------------------------------------------------------------ bf16 parts
// Two floats rounded to bf16.
__device__ __forceinline__ uint32_t pair_of(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}
__device__ __forceinline__ float low_of(uint32_t pair) { return __uint_as_float(pair << 16); }
__device__ __forceinline__ float high_of(uint32_t pair) { return __uint_as_float(pair & 0xffff0000u); }
// x = p[0] + p[1] + ... with 8 bits in each part, and its sign
template <int NP>
__device__ __forceinline__ void split8(float (&x)[8], u32x4 (&p)[NP]) {
#pragma unroll
    for (int n = 0; n < NP; ++n) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            p[n][j] = pair_of(x[2 * j], x[2 * j + 1]);
            if (n + 1 < NP) x[2 * j] -= low_of(p[n][j]), x[2 * j + 1] -= high_of(p[n][j]);
        }
    }
}
template <int NP>
__device__ __forceinline__ void split4(f32x4 x, u32x2 (&p)[NP]) {
#pragma unroll
    for (int n = 0; n < NP; ++n) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            p[n][j] = pair_of(x[2 * j], x[2 * j + 1]);
            if (n + 1 < NP) x[2 * j] -= low_of(p[n][j]), x[2 * j + 1] -= high_of(p[n][j]);
        }
    }
}
// c += a b over the pairs of parts that together reach ORD places of 8 bits
template <int ORD, int NA, int NB>
__device__ __forceinline__ void mma(const u32x4 (&a)[NA], const u32x4 (&b)[NB], f32x4& c) {
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            if (i + j < ORD)
                c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a[i]),
                                                            __builtin_bit_cast(bf16x8, b[j]), c, 0, 0, 0);
}

// Operand order.  A 16x16x32 product's operands hold, in lane l, row (column)
// l & 15 and 8 of the 32 summed places; which 8 is free as long as both operands
// agree.  Here group g = l >> 4 has places 4g .. 4g+3 of the first 16 and of the
// second 16: that is how two 16x16 results lie in the registers (row 4g + r,
// column l & 15), so a result becomes the next product's operand as it is.
__device__ __forceinline__ int place_of(int ks, int g, int j) { return 32 * ks + (j < 4 ? 4 * g + j : 12 + 4 * g + j); }

// Memory through buffer descriptors: a uniform base, a lane's 32-bit offset and a
// uniform one cost no address arithmetic on the vector units, and what lies behind
// the descriptor's end reads as zero and is not written, so that accesses need no
// branches.  kNowhere is behind every end.
constexpr uint32_t kNowhere = 0x80000000u;
typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ __forceinline__ Buffer buffer_of(const void* p, long long bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
}
// The n'th operand part (64 lanes of 16 bytes) of an array of `parts`, and this lane's own of it.
struct Parts {
    Buffer b;
    uint32_t at;
    __device__ __forceinline__ Parts(const u32x4* p, long long parts_before, int parts, int lane)
        : b(buffer_of(p + parts_before * 64, (long long)parts * 1024)), at(16 * lane) {}
    __device__ __forceinline__ u32x4 operator[](int n) const {
        return __builtin_amdgcn_raw_buffer_load_b128(b, at, 1024 * n, 0);
    }
};

// Column c of the row at byte `row`, zero from D on and where !ok.
template <class TY>
__device__ __forceinline__ float load1(Buffer b, uint32_t row, int c, int D, bool ok) {
    using S = typename TY::S;
    const uint32_t at = ok && c < D ? row + c * (uint32_t)sizeof(S) : kNowhere;
    if constexpr (sizeof(S) == 4)
        return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(b, at, 0, 0));
    else
        return TY::load(__builtin_bit_cast(S, __builtin_amdgcn_raw_buffer_load_b16(b, at, 0, 0)));
}
// Columns c ... c + 7 of the row at byte `row`, zero from D on and where !ok.
template <class TY>
__device__ __forceinline__ void load8(Buffer b, uint32_t row, int c, int D, bool ok, bool vec, float (&x)[8]) {
    constexpr int Z = sizeof(typename TY::S);
    if (vec) {  // 4 elements are one aligned load
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t at = ok && c + 4 * h < D ? row + (c + 4 * h) * Z : kNowhere;
            if constexpr (Z == 4) {
                const u32x4 y = __builtin_amdgcn_raw_buffer_load_b128(b, at, 0, 0);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[4 * h + j] = __uint_as_float(y[j]);
            } else {
                const u32x2 y = __builtin_amdgcn_raw_buffer_load_b64(b, at, 0, 0);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    x[4 * h + j] = TY::load(__builtin_bit_cast(
                        typename TY::S, (uint16_t)(j & 1 ? y[j >> 1] >> 16 : y[j >> 1] & 0xffff)));
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = load1<TY>(b, row, c + j, D, ok);
    }
}

// ------------------------------------------------------------ decays
constexpr float kMinDecay = -1e5f;  // exp of it is 0; keeps sums of -inf finite
// 2^d of a 64-bit argument, to 32 bits: what the float argument leaves out counts
// where it is large.  (The hardware's exponential flushes results below 2^-126.)
__device__ __forceinline__ float exp2_of(double d) {
    const float x = (float)d;
    return __builtin_amdgcn_exp2f(x) * fmaf((float)(d - (double)x), 0.69314718f, 1.0f);
}

// 2^((h1 + l1) - (h2 + l2)) of sums held in two floats: the difference is off by half
// a step, so what it gives by |difference| 2^-25, of a result that is 2^difference.
__device__ __forceinline__ float exp2_of(float h1, float l1, float h2, float l2) {
    return __builtin_amdgcn_exp2f((h1 - h2) + (l1 - l2));
}

// --------------------------------------------------------------- arguments
struct Shape {
    int n_seq, seq_len, n_tokens;
    const int* offsets;
    int hk, hv, dk, dv;
    float scale;
    long long qt, qh, kt, kh, vt, vh, gt, gh;
    long long slots;
    int chunks;  // of a sequence, where all have the same length
    bool qvec, kvec, vvec, gvec;
};

// Where a value head's and a key head's parts of a chunk lie in the workspace.
struct Space {
    u32x4 *kf, *qf, *kt, *qt;    // a key head's: operands of K, Q, K^T, Q^T
    u32x4 *t, *m, *tt, *mt;      // a value head's: T, M, T^T, M^T
    struct Gates* gates;
    float *s0, *ds, *u, *dr;     // rows [dk padded][dv padded] and [64][dv padded]
    int dvp;                     // dim_v rounded up to 32
};
struct Gates {
    double G[kC];  // sums of g log2(e)
    float gamma[kC], e[kC], beta[kC];
};

// Slot -> sequence, chunk.  Chunk c of sequence s has slot base(s) + c; with
// packed tokens base(s) = offsets[s] / 64 + s, which leaves each sequence at
// least its ceil(length / 64) slots and needs no sums over the lengths.
struct Chunk {
    int s, c, tok0, n;  // n <= 0: the slot is empty
};
__device__ __forceinline__ int offset_of(const Shape& a, int s) { return min(max(a.offsets[s], 0), a.n_tokens); }
__device__ __forceinline__ long long base_of(const Shape& a, int s) {
    return a.offsets ? (long long)(offset_of(a, s) / kC) + s : (long long)s * a.chunks;
}
__device__ __forceinline__ void span_of(const Shape& a, int s, int& tok0, int& len) {
    if (a.offsets) {
        tok0 = offset_of(a, s);
        len = max(0, offset_of(a, s + 1) - tok0);
    } else {
        tok0 = s * a.seq_len;
        len = a.seq_len;
    }
}
__device__ __forceinline__ Chunk chunk_of(const Shape& a, long long slot) {
    Chunk k;
    if (a.offsets) {  // the last sequence whose base is not behind the slot, 64 at a time
        int lo = 0, n = a.n_seq;
        while (n > 1) {
            const int step = (n + 63) / 64, at = lo + (int)(threadIdx.x & 63) * step;
            const bool before = at < lo + n && base_of(a, min(at, a.n_seq - 1)) <= slot;
            const int more = max(__popcll(__ballot(before)) - 1, 0) * step;
            lo += more;
            n = min(step, n - more);
        }
        k.s = __builtin_amdgcn_readfirstlane(lo);
    } else {
        k.s = (int)((uint32_t)slot / (uint32_t)a.chunks);
    }
    k.c = (int)(slot - base_of(a, k.s));
    int tok0, len;
    span_of(a, k.s, tok0, len);
    k.n = k.c < 0 ? 0 : (int)min((long long)kC, (long long)len - (long long)k.c * kC);
    k.n = __builtin_amdgcn_readfirstlane(k.n);
    k.tok0 = __builtin_amdgcn_readfirstlane(tok0 + k.c * kC);
    return k;
}

// Workgroups are dealt to the 8 dies in turn; `count` logical ones in order, so
// that neighbours (tiles of one head, heads of one key head) share a die's L2.
__device__ __forceinline__ long long on_die(long long block, long long count) {
    const long long each = (count + 7) / 8;
    return (block % 8) * each + block / 8;
}
inline unsigned dealt(long long count) { return (unsigned)((count + 7) / 8 * 8); }

// Sums over lanes that stay on the vector units.
template <int N>
__device__ __forceinline__ float from_lane_behind(float x) {  // N lanes on, within the 16 of a group
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x120 + N, 0xf, 0xf, true));
}
__device__ __forceinline__ float over_eights(float x) {  // over lanes l, l + 8, ... l + 56 (mod 64)
    x += from_lane_behind<8>(x);
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

__device__ __forceinline__ int wave_of() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// =========================================================== all chunks: prep
// grid: (slots, hv + hk).  The first hv make T and M of a value head, the others
// the operands of a key head.  M's triangle and the inverse's 16 x 16 blocks are worked
// on by one wave each, the inverse on the 32-bit matrix cores: its products are 1/50 of
// the chunk's and wait for each other, so parts would only make them longer.  Bound by
// the chunk's chain of latencies (products, decays, inverse, each behind a barrier)
// with 4 workgroups a CU: 128 chunks of 32 + 16 heads (bf16, dim_k 128) in 88 us; for the
// gradients 128 of 16 + 8 in 52.
//
// A chunk's rows of a key head's tensor as operands, VEC: 4 elements at a time.
template <class TY, bool VEC>
struct KeyRows {
    using S = typename TY::S;
    Buffer b;
    uint32_t step;
    int n, D;
    __device__ __forceinline__ KeyRows(const S* p, long long stride, int n_, int D_)
        : step((uint32_t)(stride * sizeof(S))), n(n_), D(D_) {
        b = buffer_of(p, ((long long)(n - 1) * stride + D) * (long long)sizeof(S));
    }
    // lane's row 16 rt + col, 8 places of ks
    __device__ __forceinline__ void load(int rt, int ks, int lane, u32x4 (&p)[TY::NP]) const {
        constexpr uint32_t Z = sizeof(S);
        const int row = 16 * rt + (lane & 15), grp = lane >> 4;
        const uint32_t at = row < n ? row * step : kNowhere;
        float x[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = place_of(ks, grp, 4 * h);
            if constexpr (VEC && Z == 2) {
                const u32x2 y = __builtin_amdgcn_raw_buffer_load_b64(b, c < D ? at + Z * c : kNowhere, 0, 0);
                if constexpr (TY::NP == 1) {
                    p[0][2 * h] = y[0], p[0][2 * h + 1] = y[1];
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        x[4 * h + j] = TY::load(
                            __builtin_bit_cast(S, (uint16_t)(j & 1 ? y[j >> 1] >> 16 : y[j >> 1] & 0xffff)));
                }
            } else if constexpr (VEC) {
                const u32x4 y = __builtin_amdgcn_raw_buffer_load_b128(b, c < D ? at + Z * c : kNowhere, 0, 0);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[4 * h + j] = __uint_as_float(y[j]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t to = c + j < D ? at + Z * (c + j) : kNowhere;
                    if constexpr (Z == 4)
                        x[4 * h + j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(b, to, 0, 0));
                    else
                        x[4 * h + j] =
                            TY::load(__builtin_bit_cast(S, __builtin_amdgcn_raw_buffer_load_b16(b, to, 0, 0)));
                }
            }
        }
        if constexpr (!(VEC && TY::NP == 1)) split8<TY::NP>(x, p);
    }
};

// The chunk's 64 tokens of 32 places of dim_k, as rows and, transposed, as columns.
// The matrix cores turn them: times the identity, rows come out as a result lies
// (token 4 grp + r, place l & 15), which is half of the operand with tokens summed;
// ones and zeros leave every part as it is.
template <class TY, int KS, bool TURN, bool VEC>
__device__ __forceinline__ void key_operands(const KeyRows<TY, VEC>& from, int ks, int lane, u32x4* rows,
                                             u32x4* columns) {
    constexpr int NP = TY::NP;
    const int col = lane & 15, grp = lane >> 4;
    u32x4 x[4][NP];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) from.load(rt, ks, lane, x[rt]);
#pragma unroll
    for (int rt = 0; rt < 4; ++rt)
#pragma unroll
        for (int i = 0; i < NP; ++i) rows[((rt * KS + ks) * NP + i) * 64 + lane] = x[rt][i];
    if constexpr (TURN) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            u32x4 one[1] = {{0, 0, 0, 0}};  // column `col` of the identity's half: place 16 half + col
            if (grp == (col >> 2)) one[0][2 * half + ((col >> 1) & 1)] = col & 1 ? 0x3f800000u : 0x3f80u;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                u32x4 out[2];
#pragma unroll
                for (int rt = 0; rt < 4; ++rt) {
                    f32x4 y = {0, 0, 0, 0};
                    const u32x4 part[1] = {x[rt][i]};
                    mma<1>(part, one, y);
                    out[rt >> 1][2 * (rt & 1)] = pair_of(y[0], y[1]);
                    out[rt >> 1][2 * (rt & 1) + 1] = pair_of(y[2], y[3]);
                }
#pragma unroll
                for (int ts = 0; ts < 2; ++ts)
                    columns[(((2 * ks + half) * 2 + ts) * NP + i) * 64 + lane] = out[ts];
            }
        }
    }
}

template <class TY, int KS, bool GRAD, bool VEC>
__global__ __launch_bounds__(kThreads) void delta_prep_kernel(Shape a, Space w, const typename TY::S* __restrict__ q,
                                                              const typename TY::S* __restrict__ k,
                                                              const float* __restrict__ g,
                                                              const float* __restrict__ beta) {
    using S = typename TY::S;
    constexpr int NP = TY::NP;
    const long long slot = blockIdx.x;
    const Chunk ch = chunk_of(a, slot);
    if (ch.n <= 0) return;
    const int t = threadIdx.x, lane = t & 63, wv = wave_of(), col = lane & 15, grp = lane >> 4;

    if ((int)blockIdx.y >= a.hv) {  // operands of a key head
        const int h = blockIdx.y - a.hv;
        const long long at = (slot * a.hk + h) * 4 * KS * NP * 64;
        const S* kp = k + (long long)ch.tok0 * a.kt + h * a.kh;
        const S* qp = q + (long long)ch.tok0 * a.qt + h * a.qh;
        for (int f = wv; f < 2 * KS; f += 4) {
            if (f < KS)
                key_operands<TY, KS, true, VEC>(KeyRows<TY, VEC>(kp, a.kt, ch.n, a.dk), f, lane, w.kf + at, w.kt + at);
            else
                key_operands<TY, KS, GRAD, VEC>(KeyRows<TY, VEC>(qp, a.qt, ch.n, a.dk), f - KS, lane, w.qf + at,
                                                w.qt + at);
        }
        return;
    }

    __shared__ float Gh[kC], Gl[kC];  // sums of g log2(e), each in two floats
    __shared__ float Bt[kC];
    __shared__ __align__(16) float L[kC][kC + 4];  // k's rows, then L, then M
    __shared__ __align__(16) float X[kC][kC + 4];  // q's rows, then (I + L)^-1
    const int h = blockIdx.y;
    const int hk = h / (a.hv / a.hk);
    const long long vs = slot * a.hv + h;
    const S* const kp = k + (long long)ch.tok0 * a.kt + hk * a.kh;
    const S* const qp = q + (long long)ch.tok0 * a.qt + hk * a.qh;
    // One part and aligned rows: through LDS, loaded once and 16 bytes a lane.  (As
    // operands straight from memory they cost 4 times the cache lookups: 7000 cycles
    // of a workgroup's 21000.)
    constexpr bool STAGED = VEC && NP == 1;
    if constexpr (STAGED) {
        constexpr int CH = 4 * KS, AT = kThreads / CH;  // 16-byte pieces of a row, rows at once
        const int row = t / CH, c = t % CH;
        const KeyRows<TY, VEC> kr(kp, a.kt, ch.n, a.dk), qr(qp, a.qt, ch.n, a.dk);
        u32x4 x[kC / AT], y[kC / AT];
#pragma unroll
        for (int i = 0; i < kC / AT; ++i) {
            const int r = row + i * AT;
            const bool in = r < ch.n && 8 * c < a.dk;
            x[i] = __builtin_amdgcn_raw_buffer_load_b128(kr.b, in ? r * kr.step + 16 * c : kNowhere, 0, 0);
            y[i] = __builtin_amdgcn_raw_buffer_load_b128(qr.b, in ? r * qr.step + 16 * c : kNowhere, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kC / AT; ++i) {
            *reinterpret_cast<u32x4*>(&L[row + i * AT][4 * c]) = x[i];
            *reinterpret_cast<u32x4*>(&X[row + i * AT][4 * c]) = y[i];
        }
    }
    double G_own = 0.0;
    if (wv == 0) {
        const long long at = (long long)(ch.tok0 + lane) * a.hv + h;
        const float gv = lane < ch.n ? g[at] : 0.0f;
        double G0 = (double)(gv < kMinDecay ? kMinDecay : gv) * 1.4426950408889634;
        for (int off = 1; off < 64; off <<= 1) {
            const double o = __shfl_up(G0, off);
            if (lane >= off) G0 += o;
        }
        G_own = G0;
        Gh[lane] = (float)G0;
        Gl[lane] = (float)(G0 - (double)(float)G0);
        Bt[lane] = lane < ch.n ? beta[at] : 0.0f;
    }
    // k.k and q.k: wave wv has row tile wv of k.k and row tile 3 - wv of q.k, five
    // tiles of the lower triangle for each wave
    const int qrow = 3 - wv;
    f32x4 kk[4], qk[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) kk[i] = f32x4{0, 0, 0, 0}, qk[i] = f32x4{0, 0, 0, 0};
    if constexpr (STAGED) {
        __syncthreads();
        auto part = [&](const float (*rows)[kC + 4], int rt, int ks, u32x4 (&p)[NP]) {
            p[0] = *reinterpret_cast<const u32x4*>(&rows[16 * rt + col][16 * ks + 4 * grp]);
        };
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            u32x4 ka[NP], qa[NP], kb[NP];
            part(L, wv, ks, ka);
            part(X, qrow, ks, qa);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i > wv && i > qrow) continue;
                part(L, i, ks, kb);
                if (i <= wv) mma<3>(ka, kb, kk[i]);
                if (i <= qrow) mma<3>(qa, kb, qk[i]);
            }
        }
    } else {
        const KeyRows<TY, VEC> kr(kp, a.kt, ch.n, a.dk), qr(qp, a.qt, ch.n, a.dk);
        constexpr int AT_ONCE = NP == 1 ? KS : 1;
#pragma unroll
        for (int k0 = 0; k0 < KS; k0 += AT_ONCE) {
            u32x4 ka[AT_ONCE][NP], qa[AT_ONCE][NP], kb[AT_ONCE][4][NP];
#pragma unroll
            for (int ks = 0; ks < AT_ONCE; ++ks) {
                kr.load(wv, k0 + ks, lane, ka[ks]);
                qr.load(qrow, k0 + ks, lane, qa[ks]);
#pragma unroll
                for (int i = 0; i < 4; ++i) kr.load(i, k0 + ks, lane, kb[ks][i]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i <= wv) {
#pragma unroll
                    for (int ks = 0; ks < AT_ONCE; ++ks) mma<3>(ka[ks], kb[ks][i], kk[i]);
                }
                if (i <= qrow) {
#pragma unroll
                    for (int ks = 0; ks < AT_ONCE; ++ks) mma<3>(qa[ks], kb[ks][i], qk[i]);
                }
            }
        }
    }
    __syncthreads();
    {
        float kh[4], kl[4], qh[4], ql[4], bk[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            kh[r] = Gh[16 * wv + 4 * grp + r], kl[r] = Gl[16 * wv + 4 * grp + r];
            qh[r] = Gh[16 * qrow + 4 * grp + r], ql[r] = Gl[16 * qrow + 4 * grp + r];
            bk[r] = Bt[16 * wv + 4 * grp + r];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = 16 * i + col;
            const float ch_ = Gh[c], cl = Gl[c];
            if (i <= wv) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 16 * wv + 4 * grp + r;
                    L[row][c] = c < row ? bk[r] * exp2_of(kh[r], kl[r], ch_, cl) * kk[i][r] : 0.0f;
                }
            }
            if (i <= qrow) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 16 * qrow + 4 * grp + r;
                    qk[i][r] = c <= row ? a.scale * exp2_of(qh[r], ql[r], ch_, cl) * qk[i][r] : 0.0f;
                }
            }
        }
    }
    if (wv == 0) {
        const double last = __shfl(G_own, 63);
        Gates& ga = w.gates[vs];
        ga.G[lane] = G_own;
        ga.gamma[lane] = exp2_of(G_own);
        ga.e[lane] = exp2_of(last - G_own);
        ga.beta[lane] = Bt[lane];
    }
    __syncthreads();
    // The 16 x 16 blocks on the diagonal, one for each wave: column `col` of
    // (I + L)^-1 by substitution.
    {
        const int r0 = 16 * wv;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float even = i == col ? 1.0f : 0.0f, odd = 0.0f;
#pragma unroll
            for (int m4 = 0; m4 < i; m4 += 4) {
                const f32x4 l = *reinterpret_cast<const f32x4*>(&L[r0 + i][r0 + m4]);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (m4 + j < i) (j & 1 ? odd : even) -= l[j] * x[m4 + j];
            }
            x[i] = even + odd;
        }
        if (grp == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) X[r0 + i][r0 + col] = x[i];
        }
    }
    __syncthreads();
    // Below it, block column wv: X_rc = -X_rr sum_m L_rm X_mc, on the 32-bit matrix
    // cores; summed place 4 s + ... of a product is row 4 grp + s, so a result is
    // the next product's right operand as it lies.
    {
        f32x4 xc[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) xc[0][r] = X[16 * wv + 4 * grp + r][16 * wv + col];
#pragma unroll
        for (int d = 1; d < 4; ++d) {
            const int rt = wv + d;
            if (rt < 4) {
                f32x4 y = {0, 0, 0, 0}, z = {0, 0, 0, 0};
#pragma unroll
                for (int m = 0; m < d; ++m) {
                    const f32x4 l = *reinterpret_cast<const f32x4*>(&L[16 * rt + col][16 * (wv + m) + 4 * grp]);
#pragma unroll
                    for (int s = 0; s < 4; ++s) y = __builtin_amdgcn_mfma_f32_16x16x4f32(l[s], xc[m][s], y, 0, 0, 0);
                }
                const f32x4 l = *reinterpret_cast<const f32x4*>(&X[16 * rt + col][16 * rt + 4 * grp]);
#pragma unroll
                for (int s = 0; s < 4; ++s) z = __builtin_amdgcn_mfma_f32_16x16x4f32(-l[s], y[s], z, 0, 0, 0);
                xc[d] = z;
#pragma unroll
                for (int r = 0; r < 4; ++r) X[16 * rt + 4 * grp + r][16 * wv + col] = z[r];
            }
            if (d <= wv) {  // the blocks above the diagonal
#pragma unroll
                for (int r = 0; r < 4; ++r) X[16 * (wv - d) + 4 * grp + r][16 * wv + col] = 0.0f;
            }
        }
    }
    __syncthreads();
    // M in L's place
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) L[16 * qrow + 4 * grp + r][16 * i + col] = i <= qrow ? qk[i][r] : 0.0f;
    __syncthreads();
    // Operands, row tile rt and half ts of the summed tokens; those that are zero
    // (above the diagonal, below it in the transposed ones) are not stored.
    for (int f = wv; f < 8; f += 4) {
        const int rt = f >> 1, ts = f & 1, row = 16 * rt + col;
        float x[8];
        if (ts <= (rt >> 1)) {
            u32x4 p[3];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = X[row][place_of(ts, grp, j)] * Bt[place_of(ts, grp, j)];
            split8<3>(x, p);
#pragma unroll
            for (int n = 0; n < 3; ++n) w.t[((vs * 8 + f) * 3 + n) * 64 + lane] = p[n];
            if (!GRAD) {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = L[row][place_of(ts, grp, j)];
                split8<3>(x, p);
#pragma unroll
                for (int n = 0; n < 3; ++n) w.m[((vs * 8 + f) * 3 + n) * 64 + lane] = p[n];
            }
        }
        if (GRAD && ts >= (rt >> 1)) {
            u32x4 p[3];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = X[place_of(ts, grp, j)][row];
            split8<3>(x, p);
#pragma unroll
            for (int n = 0; n < 3; ++n) w.tt[((vs * 8 + f) * 3 + n) * 64 + lane] = p[n];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = L[place_of(ts, grp, j)][row];
            split8<3>(x, p);
#pragma unroll
            for (int n = 0; n < 3; ++n) w.mt[((vs * 8 + f) * 3 + n) * 64 + lane] = p[n];
        }
    }
}

// ================================================ along a sequence: the states
// A workgroup has a head's tile of 16 NCT columns of dim_v; wave wv has token tile
// wv of the chunk and KS / 2 row tiles of the state, which stays in its registers
// in 32 bits.  What all waves need of each other (parts of S, of the bracket
// before T, of U) goes through LDS in operand order, three exchanges a chunk.
//
// With one wave a SIMD nothing hides a latency but the wave itself.  So each of a
// chunk's operands is loaded again, for the next chunk, as soon as its last product has
// read it.  (Two register sets, loaded two chunks ahead, gave nothing with 16-bit types,
// o then in two parts: 16 prompts of fp16 with dim_k 64 81.5 us with two, 76.6 with one,
// 8192 tokens of bf16 317 with either; in fp32 with 128 keys they do not fit: 413 instead of 333 us for 4096 tokens
// of 32 heads.)  All loads and stores are unconditional (bounds are the buffer
// descriptors'), so that the compiler's counts of what is in flight stay exact and no
// load waits for a store.  LDS reads are issued together behind each barrier, and the
// products that the chain does not wait for (Q S, and M U with the stores of o, one
// chunk later) run in their latency.
//
// Bound by the way from one state to the next: a chunk is 4700 cycles of three
// exchanges, each a split, an LDS write, a barrier, an LDS read and a product; o's products
// add 20 us of 250 with three parts instead of two (four more waves that made o beside the
// chain gave nothing: 321 us for 319, with two).  1 x 8192 tokens, 32 heads, bf16, dims of
// 128: 256 workgroups, 128 chunks, 250 us, 1.95 us a chunk.  16
// packed fp16 prompts (of 8 heads, dim_k 64) 62 us; the states' chain for the
// gradients of 4 x 2048 (64 heads in all, wide tiles) 100 us.  Left alone: no LDS and a
// wave for each tile (365 us instead of then 237, each wave splits S by itself), scalar
// cursors instead of multiplied slots (253 instead of 230).
template <int N, int NCT, int KSN>
struct Exchange {  // [part][ks][column tile][lane]
    u32x4 v[N][KSN][NCT][64];
    // a result of row tile rt becomes half of the operand of its pair of row tiles
    __device__ __forceinline__ void put(int rt, int ct, int lane, const u32x2 (&p)[N]) {
#pragma unroll
        for (int n = 0; n < N; ++n) reinterpret_cast<u32x2*>(&v[n][rt >> 1][ct][lane])[rt & 1] = p[n];
    }
    __device__ __forceinline__ void get(int lane, u32x4 (&p)[KSN][NCT][N]) const {
#pragma unroll
        for (int ks = 0; ks < KSN; ++ks)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                for (int n = 0; n < N; ++n) p[ks][ct][n] = v[n][ks][ct][lane];
    }
};
__device__ __forceinline__ void reads_first() { __builtin_amdgcn_sched_barrier(0); }

// A tile of token rows in global memory, as a result lies in registers (row 16 wv +
// 4 grp + r, column n0 + 16 ct + col): byte offsets from the chunk's first row.
template <class TY, int NCT>
struct Tile {
    using S = typename TY::S;
    uint32_t at[NCT], step;  // of row r: at + r step
    __device__ __forceinline__ Tile(long long stride, int n0, int D, int wv, int lane) {
        // (only where a chunk has no second row is the stride larger: any then puts it behind the end)
        step = (uint32_t)min(stride * (long long)sizeof(S), 1LL << 25);
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) {
            const int c = n0 + 16 * ct + (lane & 15);
            at[ct] = c < D ? (uint32_t)(16 * wv + 4 * (lane >> 4)) * step + c * (uint32_t)sizeof(S) : kNowhere;
        }
    }
    // the descriptor of n rows (none: every access is dropped)
    static __device__ __forceinline__ Buffer rows(const S* p, long long stride, int n, int D) {
        const long long bytes = n > 0 ? ((long long)(min(n, kC) - 1) * stride + D) * (long long)sizeof(S) : 0;
        return buffer_of(p, bytes);
    }
    __device__ __forceinline__ void load(Buffer b, S (&x)[NCT][4]) const {
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if constexpr (sizeof(S) == 4)
                    x[ct][r] = __builtin_bit_cast(S, __builtin_amdgcn_raw_buffer_load_b32(b, at[ct] + r * step, 0, 0));
                else
                    x[ct][r] = __builtin_bit_cast(S, __builtin_amdgcn_raw_buffer_load_b16(b, at[ct] + r * step, 0, 0));
            }
    }
    __device__ __forceinline__ void store(Buffer b, int ct, f32x4 x) const {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const S y = TY::store(x[r]);
            if constexpr (sizeof(S) == 4)
                __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, y), b, at[ct] + r * step, 0, 0);
            else
                __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, y), b, at[ct] + r * step, 0, 0);
        }
    }
};

// One wave's operands of a key or value head's chunk, from the workspace.
template <int KS, int NP>
__device__ __forceinline__ void load_rows(const u32x4* f, long long ks0, int wv, int lane, u32x4 (&x)[KS][NP]) {
    const Parts p(f, (ks0 * 4 + wv) * KS * NP, KS * NP, lane);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int n = 0; n < NP; ++n) x[ks][n] = p[ks * NP + n];
}
template <int KS, int NP>
__device__ __forceinline__ void load_columns(const u32x4* f, long long ks0, int wv, int lane,
                                             u32x4 (&x)[KS / 2][2][NP]) {
    const Parts p(f, (ks0 * 4 + wv) * KS * NP, KS * NP, lane);
#pragma unroll
    for (int i = 0; i < KS / 2; ++i)
#pragma unroll
        for (int ts = 0; ts < 2; ++ts)
#pragma unroll
            for (int n = 0; n < NP; ++n) x[i][ts][n] = p[(i * 2 + ts) * NP + n];
}
// Of a triangle: half 0 of the tokens, and half 1 where the wave's row tile has it
// (UPPER: the other way round); the half that is zero is loaded as the other one's
// copy and not used.
template <int N, bool UPPER>
__device__ __forceinline__ void load_triangle(const u32x4* f, long long vs, int wv, int lane, u32x4 (&x)[2][N]) {
    const Parts p(f, (vs * 4 + wv) * 2 * N, 2 * N, lane);
#pragma unroll
    for (int ts = 0; ts < 2; ++ts) {
        const int from = UPPER ? max(ts, wv >> 1) : min(ts, wv >> 1);
#pragma unroll
        for (int n = 0; n < N; ++n) x[ts][n] = p[from * N + n];
    }
}
__device__ __forceinline__ f32x4 as_floats(u32x4 x) { return __builtin_bit_cast(f32x4, x); }
template <bool BETA>
struct RowGates {
    f32x4 gamma, e, beta;
    float last;
    __device__ __forceinline__ void load(const Gates* g, long long vs, int wv, int lane) {
        const Buffer b = buffer_of(g + vs, sizeof(Gates));
        const uint32_t r = 64 * wv + 16 * (lane >> 4);
        gamma = as_floats(__builtin_amdgcn_raw_buffer_load_b128(b, r, offsetof(Gates, gamma), 0));
        e = as_floats(__builtin_amdgcn_raw_buffer_load_b128(b, r, offsetof(Gates, e), 0));
        if constexpr (BETA) beta = as_floats(__builtin_amdgcn_raw_buffer_load_b128(b, r, offsetof(Gates, beta), 0));
        last = g[vs].gamma[kC - 1];
    }
};
// A state's rows and columns of this lane.
template <int NR, int NCT, class F>
__device__ __forceinline__ void each_of_state(int wv, int lane, int n0, F f) {
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                f(i, ct, r, 16 * (wv * NR + i) + 4 * (lane >> 4) + r, n0 + 16 * ct + (lane & 15));
}

// Results into the workspace's rows of dvp floats.
template <int KS, int NCT>
__device__ __forceinline__ void keep_state(float* to, long long vs, int dvp, int n0, int wv, int lane,
                                           const f32x4 (&st)[KS / 2][NCT]) {
    const Buffer b = buffer_of(to + vs * 32 * KS * dvp, (long long)128 * KS * dvp);
    const uint32_t at = 4 * ((16 * wv * (KS / 2) + 4 * (lane >> 4)) * dvp + (lane & 15));
#pragma unroll
    for (int i = 0; i < KS / 2; ++i)
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(st[i][ct][r]), b, at,
                                                      4 * ((16 * i + r) * dvp + n0 + 16 * ct), 0);
}
__device__ __forceinline__ void keep_rows(float* to, long long vs, int dvp, int n0, int wv, int lane, f32x4 x) {
    const Buffer b = buffer_of(to + vs * kC * dvp, (long long)4 * kC * dvp);
    const uint32_t at = 4 * ((16 * wv + 4 * (lane >> 4)) * dvp + (lane & 15));
#pragma unroll
    for (int r = 0; r < 4; ++r)
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x[r]), b, at, 4 * (r * dvp + n0), 0);
}

template <int NCT, int KS, bool GRAD>
struct ChainLds {
    Exchange<3, NCT, KS> s;     // S
    Exchange<3, NCT, 2> p, e;   // the bracket before T; e U
    Exchange<GRAD ? 1 : 3, GRAD ? 1 : NCT, 2> u;  // U; unused for the gradients
};

template <class TY, int KS, int NCT, bool GRAD>
__device__ __forceinline__ void chain_task(unsigned block, void* lds, const Shape& a, const Space& w,
                                           const typename TY::S* __restrict__ v, const float* initial,
                                           typename TY::S* __restrict__ o, float* final_state) {
    using S = typename TY::S;
    constexpr int NP = TY::NP, NR = KS / 2;
    auto& sm = *static_cast<ChainLds<NCT, KS, GRAD>*>(lds);
    auto& xs = sm.s;
    auto &xp = sm.p, &xe = sm.e;
    auto& xu = sm.u;
    // for the gradients all of the padded columns: the workspace's rows are read whole
    const int tiles = ((GRAD ? w.dvp : a.dv) + 16 * NCT - 1) / (16 * NCT);
    const long long count = (long long)a.n_seq * a.hv * tiles;
    const long long at = on_die(block, count);
    if (at >= count) return;
    const int n0 = (int)(at % tiles) * 16 * NCT;
    const long long sh = at / tiles;
    const int h = (int)(sh % a.hv), s = (int)(sh / a.hv), hk = h / (a.hv / a.hk);
    const int lane = threadIdx.x & 63, wv = wave_of();
    int tok0, len;
    span_of(a, s, tok0, len);
    tok0 = __builtin_amdgcn_readfirstlane(tok0);
    len = __builtin_amdgcn_readfirstlane(len);
    const int chunks = (int)(((long long)len + kC - 1) / kC);
    const long long base = base_of(a, s);

    f32x4 st[NR][NCT];
    const long long sbase = sh * a.dk * a.dv;
    each_of_state<NR, NCT>(wv, lane, n0, [&](int i, int ct, int r, int row, int c) {
        st[i][ct][r] = initial && row < a.dk && c < a.dv ? initial[sbase + (long long)row * a.dv + c] : 0.0f;
    });

    struct Set {
        u32x4 kf[KS][NP], qf[GRAD ? 1 : KS][NP], kt[NR][2][NP], t[2][3], m[2][GRAD ? 1 : 3];
        S v[NCT][4];
        RowGates<false> g;
    };
    const Tile<TY, NCT> vt(a.vt, n0, a.dv, wv, lane);
    const Tile<TY, NCT> ot((long long)a.hv * a.dv, n0, a.dv, wv, lane);
    const S* const v0 = v + (long long)tok0 * a.vt + h * a.vh;
    S* const o0 = o + ((long long)tok0 * a.hv + h) * a.dv;
    auto kslot = [&](int c) { return (base + min(c, chunks - 1)) * a.hk + hk; };
    auto vslot = [&](int c) { return (base + min(c, chunks - 1)) * a.hv + h; };
    auto load_v = [&](Set& x, int c) {
        c = min(c, chunks - 1);
        vt.load(vt.rows(v0 + (long long)c * kC * a.vt, a.vt, len - c * kC, a.dv), x.v);
    };
    auto put_state = [&]() {
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) {
                u32x2 p[3];
                split4<3>(st[i][ct], p);
                xs.put(wv * NR + i, ct, lane, p);
            }
    };
    f32x4 qs[NCT];
#pragma unroll
    for (int ct = 0; ct < NCT; ++ct) qs[ct] = f32x4{0, 0, 0, 0};
    // o of chunk c: what Q S gave, and M U
    auto finish_o = [&](const Set& x, const u32x4 (&b)[2][NCT][GRAD ? 1 : 3], int c) {
        if constexpr (!GRAD) {
            const auto to = ot.rows(o0 + (long long)c * kC * a.hv * a.dv, (long long)a.hv * a.dv,
                                    c >= 0 ? len - c * kC : 0, a.dv);
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) mma<3>(x.m[0], b[0][ct], qs[ct]);
            if (wv >= 2) {
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct) mma<3>(x.m[1], b[1][ct], qs[ct]);
            }
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) ot.store(to, ct, qs[ct]);
        }
    };
    auto step = [&](Set& x, int c) {
        const long long vs = vslot(c);
        __syncthreads();
        u32x4 b[KS][NCT][3], bu[2][NCT][GRAD ? 1 : 3];
        xs.get(lane, b);
        if constexpr (!GRAD) xu.get(lane, bu);
        reads_first();
        if constexpr (GRAD) {
            keep_state<KS, NCT>(w.s0, vs, w.dvp, n0, wv, lane, st);
        }
        f32x4 kx[NCT];
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) kx[ct] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) mma<3>(x.kf[ks], b[ks][ct], kx[ct]);
        load_rows<KS, NP>(w.kf, kslot(c + 1), wv, lane, x.kf);
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) {
            f32x4 y;
#pragma unroll
            for (int r = 0; r < 4; ++r) y[r] = TY::load(x.v[ct][r]) - x.g.gamma[r] * kx[ct][r];
            u32x2 p[3];
            split4<3>(y, p);
            xp.put(wv, ct, lane, p);
        }
        load_v(x, c + 1);
        if constexpr (!GRAD) {
            finish_o(x, bu, c - 1);
            load_triangle<3, false>(w.m, vs, wv, lane, x.m);
        }
        __syncthreads();
        u32x4 bp[2][NCT][3];
        xp.get(lane, bp);
        reads_first();
        if constexpr (!GRAD) {
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) {
                qs[ct] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) mma<3>(x.qf[ks], b[ks][ct], qs[ct]);
            }
            load_rows<KS, NP>(w.qf, kslot(c + 1), wv, lane, x.qf);
        }
        f32x4 u[NCT];
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) {
            u[ct] = f32x4{0, 0, 0, 0};
            mma<3>(x.t[0], bp[0][ct], u[ct]);
        }
        if (wv >= 2) {
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) mma<3>(x.t[1], bp[1][ct], u[ct]);
        }
        load_triangle<3, false>(w.t, vslot(c + 1), wv, lane, x.t);
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) {
            u32x2 p[3];
            split4<3>(u[ct] * x.g.e, p);
            xe.put(wv, ct, lane, p);
            if constexpr (GRAD) {
                keep_rows(w.u, vs, w.dvp, n0 + 16 * ct, wv, lane, u[ct]);
            } else {
                u32x2 pu[3];
                split4<3>(u[ct], pu);
                xu.put(wv, ct, lane, pu);
                qs[ct] = qs[ct] * x.g.gamma * a.scale;
            }
        }
        __syncthreads();
        u32x4 be[2][NCT][3];
        xe.get(lane, be);
        reads_first();
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) st[i][ct] *= x.g.last;
        x.g.load(w.gates, vslot(c + 1), wv, lane);
#pragma unroll
        for (int ts = 0; ts < 2; ++ts)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                for (int i = 0; i < NR; ++i) mma<3>(x.kt[i][ts], be[ts][ct], st[i][ct]);
        load_columns<KS, NP>(w.kt, kslot(c + 1), wv, lane, x.kt);
        put_state();
    };
    if (chunks > 0) {
        Set x;
        load_rows<KS, NP>(w.kf, kslot(0), wv, lane, x.kf);
        load_v(x, 0);
        if constexpr (!GRAD) load_rows<KS, NP>(w.qf, kslot(0), wv, lane, x.qf);
        load_triangle<3, false>(w.t, vslot(0), wv, lane, x.t);
        x.g.load(w.gates, vslot(0), wv, lane);
        load_columns<KS, NP>(w.kt, kslot(0), wv, lane, x.kt);
        if constexpr (!GRAD) load_triangle<3, false>(w.m, vslot(0), wv, lane, x.m);
        put_state();
        for (int c = 0; c < chunks; ++c) step(x, c);
        if constexpr (!GRAD) {
            __syncthreads();
            u32x4 bu[2][NCT][3];
            xu.get(lane, bu);
            finish_o(x, bu, chunks - 1);
        }
    }
    if (final_state)
        each_of_state<NR, NCT>(wv, lane, n0, [&](int i, int ct, int r, int row, int c) {
            if (row < a.dk && c < a.dv) final_state[sbase + (long long)row * a.dv + c] = st[i][ct][r];
        });
}

// With fp16 and dim_k <= 64 two workgroups share a CU where the compiler would take 6
// registers too many for that: 16 packed prompts 85.5 us, with one 88.3.
template <class TY, int KS, int NCT, bool GRAD>
__global__ __launch_bounds__(kThreads, TY::NP == 2 && KS == 2 ? 2 : 1) void delta_chain_kernel(Shape a, Space w, const typename TY::S* __restrict__ v,
                                                               const float* initial, typename TY::S* __restrict__ o,
                                                               float* final_state) {
    __shared__ __align__(16) ChainLds<NCT, KS, GRAD> sm;
    chain_task<TY, KS, NCT, GRAD>(blockIdx.x, &sm, a, w, v, initial, o, final_state);
}

// ========================================= along a sequence: the gradients' chain
// With dS the gradient of the chunk's last state, dO that of O and R = (I + L)^-1,
//   dU  = M^T dO + diag(e) K dS           dR = R^T dU   (of beta times the bracket)
//   dV  = diag(beta) dR
//   dS0 = gamma_63 dS + scale Q^T diag(gamma) dO - K^T diag(gamma beta) dR
// The same tiles and exchanges as the states' chain, from the last
// chunk on, and bound alike: 4 x 2048 tokens of 16 heads each in 135 us, 4.2 us a chunk
// of a wide tile with one more state-sized product than the states' chain.
template <int NP, int NCT, int KS>
struct ReverseLds {
    Exchange<3, NCT, KS> s;
    Exchange<NP, NCT, 2> o;       // dO
    Exchange<3, NCT, 2> g, u, r;  // scale gamma dO; dU; -gamma beta dR
};

template <class TY, int KS, int NCT>
__device__ __forceinline__ void reverse_task(unsigned block, void* lds, const Shape& a, const Space& w,
                                             const typename TY::S* __restrict__ go, const float* grad_final,
                                             typename TY::S* __restrict__ gv, float* grad_initial) {
    using S = typename TY::S;
    constexpr int NP = TY::NP, NR = KS / 2;
    auto& sh_ = *static_cast<ReverseLds<NP, NCT, KS>*>(lds);
    auto& xs = sh_.s;
    auto& xo = sh_.o;
    auto &xg = sh_.g, &xu = sh_.u, &xr = sh_.r;
    const int tiles = w.dvp / (16 * NCT);
    const long long count = (long long)a.n_seq * a.hv * tiles;
    const long long at = on_die(block, count);
    if (at >= count) return;
    const int n0 = (int)(at % tiles) * 16 * NCT;
    const long long sh = at / tiles;
    const int h = (int)(sh % a.hv), s = (int)(sh / a.hv), hk = h / (a.hv / a.hk);
    const int lane = threadIdx.x & 63, wv = wave_of();
    int tok0, len;
    span_of(a, s, tok0, len);
    tok0 = __builtin_amdgcn_readfirstlane(tok0);
    len = __builtin_amdgcn_readfirstlane(len);
    const int chunks = (int)(((long long)len + kC - 1) / kC);
    const long long base = base_of(a, s);

    f32x4 st[NR][NCT];
    const long long sbase = sh * a.dk * a.dv;
    each_of_state<NR, NCT>(wv, lane, n0, [&](int i, int ct, int r, int row, int c) {
        st[i][ct][r] = grad_final && row < a.dk && c < a.dv ? grad_final[sbase + (long long)row * a.dv + c] : 0.0f;
    });
    struct Set {
        u32x4 kf[KS][NP], kt[NR][2][NP], qt[NR][2][NP], tt[2][3], mt[2][3];
        S o[NCT][4];
        RowGates<true> g;
    };
    const Tile<TY, NCT> got(a.gt, n0, a.dv, wv, lane);
    const Tile<TY, NCT> gvt((long long)a.hv * a.dv, n0, a.dv, wv, lane);
    const S* const go0 = go + (long long)tok0 * a.gt + h * a.gh;
    S* const gv0 = gv + ((long long)tok0 * a.hv + h) * a.dv;
    auto kslot = [&](int c) { return (base + max(c, 0)) * a.hk + hk; };
    auto vslot = [&](int c) { return (base + max(c, 0)) * a.hv + h; };
    auto load_o = [&](Set& x, int c) {
        c = max(c, 0);
        got.load(got.rows(go0 + (long long)c * kC * a.gt, a.gt, len - c * kC, a.dv), x.o);
    };
    // what a chunk's first stage reads: dS, and its dO
    auto put_first = [&](const Set& x) {
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) {
                u32x2 p[3];
                split4<3>(st[i][ct], p);
                xs.put(wv * NR + i, ct, lane, p);
            }
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) {
            f32x4 y;
#pragma unroll
            for (int r = 0; r < 4; ++r) y[r] = TY::load(x.o[ct][r]);
            u32x2 p[NP], p3[3];
            split4<NP>(y, p);
            xo.put(wv, ct, lane, p);
            split4<3>(y * x.g.gamma * a.scale, p3);
            xg.put(wv, ct, lane, p3);
        }
    };
    auto step = [&](Set& x, int c) {
        const long long vs = vslot(c);
        __syncthreads();
        u32x4 b[KS][NCT][3], bo[2][NCT][NP];
        xs.get(lane, b);
        xo.get(lane, bo);
        reads_first();
        keep_state<KS, NCT>(w.ds, vs, w.dvp, n0, wv, lane, st);
        f32x4 y[NCT];
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) y[ct] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) mma<3>(x.kf[ks], b[ks][ct], y[ct]);
        load_rows<KS, NP>(w.kf, kslot(c - 1), wv, lane, x.kf);
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) {
            y[ct] *= x.g.e;
            mma<3>(x.mt[1], bo[1][ct], y[ct]);
        }
        if (wv < 2) {
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) mma<3>(x.mt[0], bo[0][ct], y[ct]);
        }
        load_triangle<3, true>(w.mt, vslot(c - 1), wv, lane, x.mt);
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) {
            u32x2 p[3];
            split4<3>(y[ct], p);
            xu.put(wv, ct, lane, p);
        }
        load_o(x, c - 1);
        __syncthreads();
        u32x4 bu[2][NCT][3], bg[2][NCT][3];
        xu.get(lane, bu);
        xg.get(lane, bg);
        reads_first();
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) {
            y[ct] = f32x4{0, 0, 0, 0};
            mma<3>(x.tt[1], bu[1][ct], y[ct]);
        }
        if (wv < 2) {
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) mma<3>(x.tt[0], bu[0][ct], y[ct]);
        }
        load_triangle<3, true>(w.tt, vslot(c - 1), wv, lane, x.tt);
        const auto to = gvt.rows(gv0 + (long long)c * kC * a.hv * a.dv, (long long)a.hv * a.dv, len - c * kC, a.dv);
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) {
            const f32x4 dv = y[ct] * x.g.beta;
            u32x2 p[3];
            split4<3>(-(dv * x.g.gamma), p);
            xr.put(wv, ct, lane, p);
            keep_rows(w.dr, vs, w.dvp, n0 + 16 * ct, wv, lane, y[ct]);
            gvt.store(to, ct, dv);
        }
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) st[i][ct] *= x.g.last;
        x.g.load(w.gates, vslot(c - 1), wv, lane);
#pragma unroll
        for (int ts = 0; ts < 2; ++ts)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                for (int i = 0; i < NR; ++i) mma<3>(x.qt[i][ts], bg[ts][ct], st[i][ct]);
        load_columns<KS, NP>(w.qt, kslot(c - 1), wv, lane, x.qt);
        __syncthreads();
        u32x4 br[2][NCT][3];
        xr.get(lane, br);
        reads_first();
#pragma unroll
        for (int ts = 0; ts < 2; ++ts)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                for (int i = 0; i < NR; ++i) mma<3>(x.kt[i][ts], br[ts][ct], st[i][ct]);
        load_columns<KS, NP>(w.kt, kslot(c - 1), wv, lane, x.kt);
        put_first(x);
    };
    if (chunks > 0) {
        Set x;
        const int last = chunks - 1;
        load_o(x, last);
        x.g.load(w.gates, vslot(last), wv, lane);
        load_rows<KS, NP>(w.kf, kslot(last), wv, lane, x.kf);
        load_triangle<3, true>(w.mt, vslot(last), wv, lane, x.mt);
        load_triangle<3, true>(w.tt, vslot(last), wv, lane, x.tt);
        load_columns<KS, NP>(w.qt, kslot(last), wv, lane, x.qt);
        load_columns<KS, NP>(w.kt, kslot(last), wv, lane, x.kt);
        put_first(x);
        for (int c = last; c >= 0; --c) step(x, c);
    }
    if (grad_initial)
        each_of_state<NR, NCT>(wv, lane, n0, [&](int i, int ct, int r, int row, int c) {
            if (row < a.dk && c < a.dv) grad_initial[sbase + (long long)row * a.dv + c] = st[i][ct][r];
        });
}

template <class TY, int KS, int NCT>
__global__ __launch_bounds__(kThreads) void delta_reverse_kernel(Shape a, Space w,
                                                                 const typename TY::S* __restrict__ go,
                                                                 const float* grad_final,
                                                                 typename TY::S* __restrict__ gv,
                                                                 float* grad_initial) {
    extern __shared__ __align__(16) unsigned char lds[];
    reverse_task<TY, KS, NCT>(blockIdx.x, lds, a, w, go, grad_final, gv, grad_initial);
}

// Both chains of the gradients in one launch: neither reads what the other writes, and
// with one of each on a CU two waves share a SIMD, each running where the other waits.
// The longer one's workgroups come first, so that a CU gets one of each.  Half of the
// registers have to do for that.  Narrow tiles of 16-bit types fit: 324 narrow
// tiles of 9 sequences of up to 1000 tokens take 50 us instead of 28 + 51.  Wide ones and
// those of fp32 with dim_k over 64 do not: 282 us instead of 102 + 134 (256 wide tiles of
// 2048 tokens, bf16), 117 instead of 78 (1024 narrow tiles of 256 tokens, fp32).
template <class TY, int KS>
constexpr bool kJoined = TY::NP < 3 || KS == 2;

template <class TY, int KS>
__global__ __launch_bounds__(kThreads, 2) void delta_chains_kernel(
    Shape a, Space w, unsigned each, const typename TY::S* __restrict__ v, const float* initial,
    const typename TY::S* __restrict__ go, const float* grad_final, typename TY::S* __restrict__ gv,
    float* grad_initial) {
    extern __shared__ __align__(16) unsigned char lds[];
    if (blockIdx.x < each)
        reverse_task<TY, KS, 1>(blockIdx.x, lds, a, w, go, grad_final, gv, grad_initial);
    else
        chain_task<TY, KS, 1, true>(blockIdx.x - each, lds, a, w, v, initial, nullptr, nullptr);
}

// ====================================================== all chunks: the gradients
// With dM = dO U^T and dL = -dR U^T (their lower triangles), F = scale Gamma dM,
// E = beta Gamma dL and X = dR S0^T:
//   dQ = scale gamma dO S0^T + F K
//   dK = -beta gamma X + e U dS^T + F^T Q + (E + E^T) K
//   dbeta_i = dR_i.v_i - gamma_i k_i.X_i + sum_j dL_ij Gamma_ij k_i.k_j
//   dG_i = sum_j D_ij - sum_j D_ji + q_i.(scale gamma dO S0^T)_i - k_i.(beta gamma X)_i - d_i
// with D = dM M + dL L below the diagonal (on it both sums take the same) and
// d_i = e_i k_i.(U dS^T)_i; the chunk's last token also gets sum_i d_i +
// gamma_63 <dS, S0>; dg_i is the sum of dG over i and all later tokens.
//
// A workgroup has a key head of a chunk and takes its value heads in turn, adding
// up dQ and dK in registers.  Its 8 waves are 4 token tiles by 2 halves of dim_k;
// the halves also share the triangles, the first has dM (and q.k), the second dL
// (and k.k).  Wave w shares its SIMD with wave w + 4: that one has token tile 3 - w,
// so that the triangles are even.  dim_v is summed in slices of 32: S0 (with dO and dR as
// left operands) and dS (with U) are split into parts once for the workgroup and shared
// through LDS, the next slice's loads in flight under the products.  q and k in result
// order are products with the identity.
//
// Bound by latency: 99 KB of LDS leave one workgroup (two waves a SIMD) a CU, and a
// slice's loads, split, barrier and products follow each other.  4 x 2048 tokens, 8 key
// and 16 value heads, bf16, dims of 128: 240 us, 75000 cycles for a chunk's value head,
// of which 5000 to 10000 are each of the 4 slices; 0.54 GB of states and rows, 2.3 TB/s.
// Slices in two LDS buffers, or v and dO loaded ahead too, need more registers than there
// are (510 us).
__device__ __forceinline__ float over_columns(float x) {  // over the 16 lanes of a group
    x += from_lane_behind<8>(x);
    x += from_lane_behind<4>(x);
    x += from_lane_behind<2>(x);
    return x + from_lane_behind<1>(x);
}
__device__ __forceinline__ float over_groups(float x) {
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

constexpr int kGradThreads = 512;
template <int KS>
struct GradsLds {
    double G[kC];
    float gamma[kC], e_[kC], beta[kC], drv[kC];
    float row[2][4][kC];     // of each half: sums over a row of D, b, q and k products, d
    float col_d[2][4][kC];   // of each half and row tile: D's column sums
    float dotted[8];
    float f[kC][kC + 4], e[kC][kC + 4];
    u32x4 s[2 * KS][3][64], d[2 * KS][3][64];  // S0's and dS's slices
    u32x4 u[4][3][64];                         // U's
};

// Row `row` of 32 floats of the slice, 8 of them for each of 4 threads, to LDS as parts.
__device__ __forceinline__ void put_parts(u32x4 (*to)[3][64], int row, int g8, const f32x4 (&x)[2]) {
    u32x4 p[3];
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = x[j >> 2][j & 3];
    split8<3>(y, p);
#pragma unroll
    for (int n = 0; n < 3; ++n) to[row >> 4][n][16 * g8 + ((row & 15) ^ (2 * g8))] = p[n];
}
// ... from which lane l reads its operand: rows are turned by 2 places a group, so
// that of 8 lanes neither the writes (of 2 rows) nor the reads meet in a bank.
__device__ __forceinline__ void get_parts(const u32x4 (&from)[3][64], int lane, u32x4 (&b)[3]) {
#pragma unroll
    for (int n = 0; n < 3; ++n) b[n] = from[n][lane ^ (2 * (lane >> 4))];
}
// A row operand's 16 places `half` as a result lies: token 4 grp + r, place l & 15.
template <int NP>
__device__ __forceinline__ f32x4 as_result(const u32x4 (&x)[NP], int half, int lane) {
    const int col = lane & 15, grp = lane >> 4;
    u32x4 one[1] = {{0, 0, 0, 0}};
    if (grp == (col >> 2)) one[0][2 * half + ((col >> 1) & 1)] = col & 1 ? 0x3f800000u : 0x3f80u;
    f32x4 y = {0, 0, 0, 0};
    mma<NP>(x, one, y);
    return y;
}

template <class TY, int KS>
__global__ __launch_bounds__(kGradThreads, 2) void delta_grads_kernel(
    Shape a, Space w, const typename TY::S* __restrict__ v, const typename TY::S* __restrict__ go,
    typename TY::S* __restrict__ gq, typename TY::S* __restrict__ gk, float* __restrict__ gg,
    float* __restrict__ gbeta) {
    using S = typename TY::S;
    constexpr int NP = TY::NP, CT = KS;  // a wave's column tiles of dim_k
    extern __shared__ __align__(16) unsigned char lds[];
    GradsLds<KS>& sm = *reinterpret_cast<GradsLds<KS>*>(lds);
    const long long slot = blockIdx.x;
    const Chunk ch = chunk_of(a, slot);
    if (ch.n <= 0) return;
    const int t = threadIdx.x, lane = t & 63, wave = wave_of(), col = lane & 15, grp = lane >> 4;
    const int half = wave >> 2, wv = half ? 7 - wave : wave;
    const int hk = blockIdx.y, rep = a.hv / a.hk;
    const long long ks0 = slot * a.hk + hk;
    const int arow = 16 * wv + col;  // this lane's row as a left operand
    const bool aok = arow < ch.n;
    const int trow = t >> 2, tg = t & 3;  // this thread's row and 8 columns of a slice
    const bool task_s = trow < 32 * KS, task_u = trow < kC;
    const uint32_t tat = 4 * (trow * w.dvp + 8 * tg), aat = 4 * (arow * w.dvp + 8 * grp);
    const uint32_t vrow = arow * (uint32_t)(a.vt * sizeof(S)), orow = arow * (uint32_t)(a.gt * sizeof(S));
    const Parts kf(w.kf, ks0 * 4 * KS * NP, 4 * KS * NP, lane), qf(w.qf, ks0 * 4 * KS * NP, 4 * KS * NP, lane),
        kt(w.kt, ks0 * 4 * KS * NP, 4 * KS * NP, lane), qt(w.qt, ks0 * 4 * KS * NP, 4 * KS * NP, lane);
    auto two = [](Buffer b, uint32_t at, int more, f32x4 (&x)[2]) {
        x[0] = as_floats(__builtin_amdgcn_raw_buffer_load_b128(b, at, more, 0));
        x[1] = as_floats(__builtin_amdgcn_raw_buffer_load_b128(b, at + 16, more, 0));
    };

    f32x4 dq[CT], dk[CT];
#pragma unroll
    for (int i = 0; i < CT; ++i) dq[i] = f32x4{0, 0, 0, 0}, dk[i] = f32x4{0, 0, 0, 0};
#pragma unroll 1
    for (int hr = 0; hr < rep; ++hr) {
        const int h = hk * rep + hr;
        const long long vs = slot * a.hv + h;
        const Buffer s0 = buffer_of(w.s0 + vs * 32 * KS * w.dvp, (long long)128 * KS * w.dvp);
        const Buffer ds = buffer_of(w.ds + vs * 32 * KS * w.dvp, (long long)128 * KS * w.dvp);
        const Buffer ub = buffer_of(w.u + vs * kC * w.dvp, (long long)4 * kC * w.dvp);
        const Buffer rb = buffer_of(w.dr + vs * kC * w.dvp, (long long)4 * kC * w.dvp);
        const Buffer ob = Tile<TY, 1>::rows(go + (long long)ch.tok0 * a.gt + h * a.gh, a.gt, ch.n, a.dv);
        const Buffer vb = Tile<TY, 1>::rows(v + (long long)ch.tok0 * a.vt + h * a.vh, a.vt, ch.n, a.dv);
        f32x4 xs[2], xd[2], xu[2], xr[2];
        two(s0, tat, 0, xs);
        two(ds, tat, 0, xd);
        two(ub, tat, 0, xu);
        two(rb, aat, 0, xr);
        __syncthreads();  // the last head is done with the shared arrays
        if (t < kC) {
            const Gates& gs = w.gates[vs];
            sm.G[t] = gs.G[t];
            sm.gamma[t] = gs.gamma[t];
            sm.e_[t] = gs.e[t];
            sm.beta[t] = gs.beta[t];
        }
        // ---- dO S0^T, dR S0^T, U dS^T; dO U^T or dR U^T
        f32x4 so[CT], sr[CT], ud[CT], tri[4];
#pragma unroll
        for (int i = 0; i < CT; ++i)
            so[i] = f32x4{0, 0, 0, 0}, sr[i] = f32x4{0, 0, 0, 0}, ud[i] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) tri[i] = f32x4{0, 0, 0, 0};
        float drv = 0.0f, dss = 0.0f;
#pragma unroll 1
        for (int n0 = 0; n0 < w.dvp; n0 += 32) {
            const int next = n0 + 32 < w.dvp ? n0 + 32 : 0;
            u32x4 oa[NP], rp[3];
            {
                float x[8];
                const int c0 = n0 + 8 * grp;
                if (half == 0) {
                    load8<TY>(vb, vrow, c0, a.dv, aok, a.vvec, x);
#pragma unroll
                    for (int j = 0; j < 8; ++j) drv += x[j] * xr[j >> 2][j & 3];
                }
                load8<TY>(ob, orow, c0, a.dv, aok, a.gvec, x);
                split8<NP>(x, oa);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = xr[j >> 2][j & 3];
                split8<3>(x, rp);
            }
            if (n0) __syncthreads();
            if (task_s) {
#pragma unroll
                for (int j = 0; j < 8; ++j) dss += xs[j >> 2][j & 3] * xd[j >> 2][j & 3];
                put_parts(sm.s, trow, tg, xs);
                put_parts(sm.d, trow, tg, xd);
            }
            if (task_u) put_parts(sm.u, trow, tg, xu);
            two(s0, tat, 4 * next, xs);
            two(ds, tat, 4 * next, xd);
            two(ub, tat, 4 * next, xu);
            two(rb, aat, 4 * next, xr);
            __syncthreads();
            u32x4 ua[3];
            get_parts(sm.u[wv], lane, ua);
#pragma unroll
            for (int i = 0; i < CT; ++i) {
                u32x4 b[3];
                get_parts(sm.s[half * CT + i], lane, b);
                mma<3>(oa, b, so[i]);
                mma<3>(rp, b, sr[i]);
                get_parts(sm.d[half * CT + i], lane, b);
                mma<3>(ua, b, ud[i]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i <= wv) {
                    u32x4 b[3];
                    get_parts(sm.u[i], lane, b);
                    if (half == 0)
                        mma<3>(oa, b, tri[i]);
                    else
                        mma<3>(rp, b, tri[i]);
                }
        }
        const f32x4 gam = *reinterpret_cast<const f32x4*>(&sm.gamma[16 * wv + 4 * grp]);
        const f32x4 end = *reinterpret_cast<const f32x4*>(&sm.e_[16 * wv + 4 * grp]);
        const f32x4 bet = *reinterpret_cast<const f32x4*>(&sm.beta[16 * wv + 4 * grp]);
        // ---- q.k or k.k again: the triangle of F or E, and what the gates get of it
        float dsum[4] = {0, 0, 0, 0}, bsum[4] = {0, 0, 0, 0};  // rows 16 wv + 4 grp + r
        const Parts own = half == 0 ? qf : kf;
        float(*const square)[kC + 4] = half == 0 ? sm.f : sm.e;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = 16 * i + col;
            float down = 0.0f;
            f32x4 z = {0, 0, 0, 0};
            if (i <= wv) {
                f32x4 dot = {0, 0, 0, 0};
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    u32x4 x[NP], b[NP];
#pragma unroll
                    for (int n = 0; n < NP; ++n) {
                        x[n] = own[(wv * KS + ks) * NP + n];
                        b[n] = kf[(i * KS + ks) * NP + n];
                    }
                    mma<3>(x, b, dot);
                }
                const double Gc = sm.G[c];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 16 * wv + 4 * grp + r;
                    const float decay = c <= row ? exp2_of(sm.G[row] - Gc) : 0.0f;
                    const float low = c < row ? 1.0f : 0.0f;  // below the diagonal
                    float d;
                    if (half == 0) {
                        z[r] = a.scale * decay * tri[i][r];
                        d = low * z[r] * dot[r];
                    } else {
                        const float x = -low * decay * tri[i][r];  // dL Gamma
                        const float b = x * dot[r];
                        bsum[r] += b;
                        z[r] = bet[r] * x;
                        d = bet[r] * b;
                    }
                    dsum[r] += d;
                    down += d;
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) square[16 * wv + 4 * grp + r][c] = z[r];
            down = over_groups(down);
            if (grp == 0) sm.col_d[half][wv][c] = down;
        }
        // ---- the states' parts of dQ and dK, and their products with q and k
        float qdot[4] = {0, 0, 0, 0}, kdot[4] = {0, 0, 0, 0}, gone[4] = {0, 0, 0, 0};
#pragma unroll
        for (int ks = 0; ks < KS / 2; ++ks) {
            u32x4 ka[NP], qa[NP];
#pragma unroll
            for (int n = 0; n < NP; ++n) {
                ka[n] = kf[(wv * KS + half * (KS / 2) + ks) * NP + n];
                qa[n] = qf[(wv * KS + half * (KS / 2) + ks) * NP + n];
            }
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int i = 2 * ks + p;
                const f32x4 qv = as_result<NP>(qa, p, lane), kv = as_result<NP>(ka, p, lane);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float x = a.scale * gam[r] * so[i][r], y = gam[r] * sr[i][r], z = end[r] * ud[i][r];
                    qdot[r] += qv[r] * x;
                    kdot[r] += kv[r] * y;
                    gone[r] += kv[r] * z;
                    dq[i][r] += x;
                    dk[i][r] += z - bet[r] * y;
                }
            }
        }
        // ---- the gates' sums, of each half
        drv = over_groups(drv);
        if (half == 0 && grp == 0) sm.drv[arow] = drv;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) dss += __shfl_xor(dss, off);
        if (lane == 0) sm.dotted[wave] = dss;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 16 * wv + 4 * grp + r;
            const float d = over_columns(dsum[r]), b = over_columns(bsum[r]);
            const float x = over_columns(qdot[r]), y = over_columns(kdot[r]), z = over_columns(gone[r]);
            if (col == 0) {
                sm.row[half][0][row] = d + (x - bet[r] * y);
                sm.row[half][1][row] = b;
                sm.row[half][2][row] = y;
                sm.row[half][3][row] = z;
            }
        }
        __syncthreads();
        if (wave == 0) {
            const float z = sm.row[0][3][lane] + sm.row[1][3][lane];
            float all = z;
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) all += __shfl_xor(all, off);
            float d = (sm.row[0][0][lane] + sm.row[1][0][lane]) - z;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i >= (lane >> 4)) d -= sm.col_d[0][i][lane] + sm.col_d[1][i][lane];
            double x = d;
            if (lane == kC - 1) {
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) sum += sm.dotted[i];
                x += (double)all + (double)exp2_of(sm.G[kC - 1]) * sum;
            }
            for (int off = 1; off < 64; off <<= 1) {
                const double o = __shfl_down(x, off);
                if (lane + off < 64) x += o;
            }
            if (lane < ch.n) {
                const long long to = (long long)(ch.tok0 + lane) * a.hv + h;
                gg[to] = (float)x;
                gbeta[to] = sm.drv[lane] - (sm.row[0][2][lane] + sm.row[1][2][lane]) + sm.row[1][1][lane];
            }
        }
        // ---- F K, F^T Q and (E + E^T) K
#pragma unroll
        for (int ts = 0; ts < 2; ++ts) {
            float x[8];
            u32x4 fa[3];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = place_of(ts, grp, j);
                x[j] = sm.e[arow][c] + sm.e[c][arow];
            }
            split8<3>(x, fa);
#pragma unroll
            for (int i = 0; i < CT; ++i) {
                u32x4 kb[NP];
#pragma unroll
                for (int n = 0; n < NP; ++n) kb[n] = kt[((half * CT + i) * 2 + ts) * NP + n];
                mma<3>(fa, kb, dk[i]);
            }
            if (ts <= (wv >> 1)) {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = sm.f[arow][place_of(ts, grp, j)];
                split8<3>(x, fa);
#pragma unroll
                for (int i = 0; i < CT; ++i) {
                    u32x4 kb[NP];
#pragma unroll
                    for (int n = 0; n < NP; ++n) kb[n] = kt[((half * CT + i) * 2 + ts) * NP + n];
                    mma<3>(fa, kb, dq[i]);
                }
            }
            if (ts >= (wv >> 1)) {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = sm.f[place_of(ts, grp, j)][arow];
                split8<3>(x, fa);
#pragma unroll
                for (int i = 0; i < CT; ++i) {
                    u32x4 qb[NP];
#pragma unroll
                    for (int n = 0; n < NP; ++n) qb[n] = qt[((half * CT + i) * 2 + ts) * NP + n];
                    mma<3>(fa, qb, dk[i]);
                }
            }
        }
    }
    const Tile<TY, CT> to((long long)a.hk * a.dk, 16 * CT * half, a.dk, wv, lane);
    const long long first = ((long long)ch.tok0 * a.hk + hk) * a.dk;
    const Buffer qb = Tile<TY, CT>::rows(gq + first, (long long)a.hk * a.dk, ch.n, a.dk);
    const Buffer kb = Tile<TY, CT>::rows(gk + first, (long long)a.hk * a.dk, ch.n, a.dk);
#pragma unroll
    for (int i = 0; i < CT; ++i) {
        to.store(qb, i, dq[i]);
        to.store(kb, i, dk[i]);
    }
}

// ======================================================== token by token
// A wave has a tile of 32 columns of a head's state (a cache line of each row) in
// registers: lane l has columns 4 (l & 7) ... + 3 of the NR rows from NR (l >> 3)
// on, so all of the tile's loads are in flight at once and the sums over dim_k are
// in-lane and then over 8 lanes.  S'^T k and S'^T q are summed together, and
// o = S'^T q + u (k.q), so a token is one pass over the state.
//
// STEP: a decode step (`slots`, or all rows in order); otherwise the sequence form of
// short sequences, the next token's rows in flight while one is worked on.  A step is
// bound by reading and writing the states: 256 rows x 16 heads of 128 x 128, 13 rows idle
// (513 MB), in 113 us, 4.5 TB/s where a large copy reaches 4.7; 32 heads of one row in 7 us,
// latency.  It keeps
// 3 waves a SIMD at 128 keys: with 2, where the compiler would leave it, 129 us.
//
// PAST: states that the 256 MB of the last-level cache will not hold until their next step
// pass it by (non-temporal loads and stores).  Between two steps of a layer all the others'
// run, so what counts is all layers' states: from 32 MB of one call's on, eight layers
// fill the cache.  Steps of bf16, 16 heads of 128 x 128, with | without, us: 2 GB (at most 24
// layers) of other states between, 64 MB 34 | 41, 128 MB 64 | 76, 190 MB 80 | 90, 256 MB 119 |
// 145 (and 50 MB of weights between: 35 | 42, 65 | 78, 81 | 89, 120 | 141); the same states
// again and again, which no model of more layers does, 31 | 28, 62 | 50, 80 | 68, 118 | 105.
// At 16 MB, where fewer than 16 layers stay cached, 15 | 17 and 17 | 17.
constexpr long long kPastCache = 32LL << 20;
template <class TY, int NR, bool STEP, bool PAST>
__global__ __launch_bounds__(kThreads, STEP && NR == 16 ? 3 : 1) void delta_token_kernel(
    Shape a, const typename TY::S* __restrict__ q, const typename TY::S* __restrict__ k,
    const typename TY::S* __restrict__ v, const float* __restrict__ g, const float* __restrict__ beta,
    const float* in, float* out, typename TY::S* __restrict__ o, const int* __restrict__ slots, int pool,
    bool vec) {
    using S = typename TY::S;
    const int tiles = (a.dv + 31) / 32;
    const long long count = (long long)a.n_seq * a.hv * tiles, blocks = (count + 3) / 4;
    const long long block = on_die(blockIdx.x, blocks);
    const long long at = block * 4 + wave_of();
    if (at >= count) return;
    const int lane = threadIdx.x & 63, rg = lane >> 3;
    const int c0 = (int)(at % tiles) * 32 + 4 * (lane & 7);
    const long long sh = at / tiles;
    const int h = (int)(sh % a.hv), hk = h / (a.hv / a.hk), r0 = NR * rg;
    int b = (int)(sh / a.hv), tok, end;
    long long state = b;
    if constexpr (STEP) {
        tok = b;
        end = b + 1;
        if (slots) {
            const int sl = slots[b];
            if (sl < 0 || sl >= pool) {
                if (rg == 0)
                    for (int j = 0; j < 4; ++j)
                        if (c0 + j < a.dv) o[((long long)b * a.hv + h) * a.dv + c0 + j] = TY::store(0.0f);
                return;
            }
            state = sl;
        }
    } else {
        int len;
        span_of(a, b, tok, len);
        tok = __builtin_amdgcn_readfirstlane(tok);
        end = tok + __builtin_amdgcn_readfirstlane(len);
    }
    const long long sbase = (state * a.hv + h) * a.dk * a.dv + c0;
    f32x4 s[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int row = r0 + i;
        s[i] = f32x4{0, 0, 0, 0};
        if (in && row < a.dk) {
            const float* p = in + sbase + (long long)row * a.dv;
            if (vec) {
                if (c0 < a.dv)
                    s[i] = PAST ? __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p))
                                : *reinterpret_cast<const f32x4*>(p);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c0 + j < a.dv) s[i][j] = p[j];
            }
        }
    }
    if (STEP && slots)  // rows of one slot: the first of them takes all
        for (int j0 = 0; j0 < b; j0 += 64)
            if (__ballot(j0 + lane < b && slots[j0 + lane] == (int)state)) return;
    struct Row {
        float k[NR], q[NR], g, beta;
        f32x4 v;
    };
    // Without branches between the loads, so that all are in flight at once.
    auto fetch_as = [&](int t, Row& x, bool four) {
        constexpr int Z = sizeof(S);
        const Buffer kb = buffer_of(k + (long long)t * a.kt + hk * a.kh, a.dk * Z);
        const Buffer qb = buffer_of(q + (long long)t * a.qt + hk * a.qh, a.dk * Z);
        const Buffer vb = buffer_of(v + (long long)t * a.vt + h * a.vh, a.dv * Z);
        x.g = g[(long long)t * a.hv + h], x.beta = beta[(long long)t * a.hv + h];
        if constexpr (NR >= 8) {
#pragma unroll
            for (int i = 0; i < NR; i += 8) {
                float e[8], f[8];
                load8<TY>(kb, 0, r0 + i, a.dk, true, four, e);
                load8<TY>(qb, 0, r0 + i, a.dk, true, four, f);
#pragma unroll
                for (int j = 0; j < 8; ++j) x.k[i + j] = e[j], x.q[i + j] = f[j];
            }
        } else {
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                x.k[i] = load1<TY>(kb, 0, r0 + i, a.dk, true);
                x.q[i] = load1<TY>(qb, 0, r0 + i, a.dk, true);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) x.v[j] = load1<TY>(vb, 0, c0 + j, a.dv, true);
    };
    auto fetch = [&](int t, Row& x) {
        if (a.kvec && a.qvec)
            fetch_as(t, x, true);
        else
            fetch_as(t, x, false);
    };
    Row x;
    if (tok < end) fetch(tok, x);
    while (tok < end) {
        int next = tok + 1;
        if constexpr (STEP) {
            if (slots) {  // the next row of the same slot
                end = next;
                for (int j0 = next; j0 < a.n_seq; j0 += 64) {
                    const unsigned long long m = __ballot(j0 + lane < a.n_seq && slots[j0 + lane] == (int)state);
                    if (m) {
                        next = j0 + __builtin_ctzll(m);
                        end = next + 1;
                        break;
                    }
                }
            }
        }
        Row then = x;
        if (!STEP && next < end) fetch(next, then);  // in flight while this token is worked on
        const float al = expf(x.g);
        f32x4 pk = {0, 0, 0, 0}, pq = {0, 0, 0, 0};
        float kq = 0.0f;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            s[i] *= al;
            pk += s[i] * x.k[i];
            pq += s[i] * x.q[i];
            kq += x.k[i] * x.q[i];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) pk[j] = over_eights(pk[j]), pq[j] = over_eights(pq[j]);
        kq = over_eights(kq);
        const f32x4 u = (x.v - pk) * x.beta;
        const f32x4 y = (pq + u * kq) * a.scale;
#pragma unroll
        for (int i = 0; i < NR; ++i) s[i] += u * x.k[i];
        if (rg == 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c0 + j < a.dv) o[((long long)tok * a.hv + h) * a.dv + c0 + j] = TY::store(y[j]);
        }
        tok = next;
        if constexpr (STEP) {
            if (tok < end) fetch(tok, x);
        } else {
            x = then;
        }
    }
    if (!out) return;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int row = r0 + i;
        if (row < a.dk) {
            float* p = out + sbase + (long long)row * a.dv;
            if (vec) {
                if (c0 < a.dv) {
                    if constexpr (PAST)
                        __builtin_nontemporal_store(s[i], reinterpret_cast<f32x4*>(p));
                    else
                        *reinterpret_cast<f32x4*>(p) = s[i];
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c0 + j < a.dv) p[j] = s[i][j];
            }
        }
    }
}

// ---------------------------------------------------------- host helpers
inline bool mul_ok(long long a, long long b, long long* r) {
    if (a < 0 || b < 0) return false;
    if (a != 0 && b > (LLONG_MAX / 16) / a) return false;
    *r = a * b;
    return true;
}

// Bytes from the first to the last element of a strided [tokens, heads, dim] array.
inline bool extent(long long tokens, int heads, int dim, long long st, long long sh, int size, long long* r) {
    long long x, y;
    if (tokens == 0) {
        *r = 0;
        return true;
    }
    if (!mul_ok(tokens - 1, st, &x) || !mul_ok(heads - 1, sh, &y)) return false;
    return mul_ok(x + y + dim, size, r);
}

constexpr long long kMaxBlocks = (1LL << 32) / kGradThreads - 8;  // a grid has fewer than 2^32 work-items

int check_shape(const delta_rule_shape_t* p, bool step, Shape* a) {
    if (!p) return CFC_ERR_NULL;
    const int n_seq = step ? (int)std::min(p->n_tokens, (long long)INT_MAX) : p->n_seq;
    if (p->type != CFC_TYPE_F32 && p->type != CFC_TYPE_BF16 && p->type != CFC_TYPE_F16) return CFC_ERR_UNSUPPORTED;
    if (n_seq < 0 || p->n_tokens < 0 || p->n_tokens > INT_MAX - 2 * kC) return CFC_ERR_DIM;
    if (p->heads_k < 1 || p->heads_v < 1 || p->heads_v % p->heads_k || p->dim_k < 1 || p->dim_v < 1) return CFC_ERR_DIM;
    if (!std::isfinite(p->scale)) return CFC_ERR_DT;
    for (long long st : {p->q_stride_t, p->q_stride_h, p->k_stride_t, p->k_stride_h, p->v_stride_t, p->v_stride_h,
                         p->go_stride_t, p->go_stride_h})
        if (st < 0) return CFC_ERR_DIM;
    const bool dense = !step && !p->offsets;
    if (dense && (p->seq_len < 0 || (long long)p->seq_len * n_seq != p->n_tokens)) return CFC_ERR_DIM;
    if (p->dim_k > DELTA_MAX_DIM_K || p->dim_v > DELTA_MAX_DIM_V) return CFC_ERR_UNSUPPORTED;
    if ((long long)p->heads_v + p->heads_k > 65535) return CFC_ERR_UNSUPPORTED;
    long long n;
    if (!mul_ok((long long)p->dim_k * p->dim_v * 4, p->heads_v, &n) || !mul_ok(n, n_seq, &n)) return CFC_ERR_DIM;
    *a = Shape{};
    a->n_seq = n_seq;
    a->seq_len = dense ? p->seq_len : 0;
    a->n_tokens = (int)p->n_tokens;
    a->offsets = step ? nullptr : p->offsets;
    a->hk = p->heads_k;
    a->hv = p->heads_v;
    a->dk = p->dim_k;
    a->dv = p->dim_v;
    a->scale = p->scale;
    a->qt = p->q_stride_t, a->qh = p->q_stride_h;
    a->kt = p->k_stride_t, a->kh = p->k_stride_h;
    a->vt = p->v_stride_t, a->vh = p->v_stride_h;
    a->gt = p->go_stride_t, a->gh = p->go_stride_h;
    a->chunks = dense ? (int)(((long long)p->seq_len + kC - 1) / kC) : 0;
    a->slots = dense ? (long long)a->chunks * n_seq : p->n_tokens / kC + n_seq;
    const long long tiles = (p->dim_v + 31) / 32 * 2;
    if (a->slots > kMaxBlocks || (long long)n_seq * p->heads_v > kMaxBlocks / 2 / tiles) return CFC_ERR_UNSUPPORTED;
    return CFC_OK;
}
// The chunks' kernels address a chunk's rows with 31 bits.  (Where a chunk has one row its
// stride is not used, and the token kernel's rows have 64.)
bool rows_fit(const delta_rule_shape_t* p) {
    if ((p->offsets ? p->n_tokens : p->seq_len) <= 1) return true;
    for (long long st : {p->q_stride_t, p->k_stride_t, p->v_stride_t, p->go_stride_t, (long long)p->heads_k * p->dim_k,
                         (long long)p->heads_v * p->dim_v})
        if (st > INT_MAX || (kC * st + DELTA_MAX_DIM_V) * size_of(p->type) > INT_MAX) return false;
    return true;
}
// Four elements of a row are one aligned load.
inline bool fours(const void* p, long long st, long long sh, int dim, int size) {
    const uintptr_t step = 4 * size;
    return (reinterpret_cast<uintptr_t>(p) % step) == 0 && st % 4 == 0 && sh % 4 == 0 && dim % 4 == 0;
}
inline void set_vec(const delta_rule_shape_t* p, Shape* a, const void* q, const void* k, const void* v,
                    const void* go) {
    const int z = size_of(p->type);
    a->qvec = fours(q, a->qt, a->qh, a->dk, z);
    a->kvec = fours(k, a->kt, a->kh, a->dk, z);
    a->vvec = fours(v, a->vt, a->vh, a->dv, z);
    a->gvec = go && fours(go, a->gt, a->gh, a->dv, z);
}

// Sequences so short that they are run token by token: 7 to 8 us and 1.2 a token for up to
// 256 heads' states (8 tokens 17 to 19 us, 32 45 to 48), while the chunks' two kernels take
// 17.4 for 32 heads, 30 for 128, 44 for 256, 81 for 512, whatever the length up to 64 (32
// heads x 1, 4, 8 and 16 sequences, dims of 128, bf16): they are even at 8, 18, 28 and 40
// tokens, and at 36 to 40 for more sequences.  Packed sequences' lengths are not known on
// the host; as many tokens in all are as short as that whatever their lengths.
inline bool is_short(const Shape& a) {
    const long long most = 8 + std::min((long long)a.n_seq * a.hv / 16, 24LL);
    return (a.offsets ? a.n_tokens : a.seq_len) <= most;
}

// The workspace's arrays, one behind the other; returns its bytes.
long long lay_out(const Shape& a, int type, bool grad, void* base, Space* w) {
    const int np = type == CFC_TYPE_BF16 ? 1 : type == CFC_TYPE_F16 ? 2 : 3;
    const int ks = a.dk <= 64 ? 2 : 4;
    const long long kslots = a.slots * a.hk, vslots = a.slots * a.hv;
    char* at = static_cast<char*>(base);
    long long total = 0;
    auto take = [&](long long bytes) {
        char* p = at ? at + total : nullptr;
        total += bytes;
        return p;
    };
    w->dvp = (a.dv + 31) / 32 * 32;
    const long long kb = kslots * 4 * ks * np * 1024, state = vslots * ks * 32 * w->dvp * 4,
                    rows = vslots * kC * w->dvp * 4;
    w->kf = (u32x4*)take(kb);
    w->qf = (u32x4*)take(kb);
    w->kt = (u32x4*)take(kb);
    w->qt = (u32x4*)take(grad ? kb : 0);
    w->t = (u32x4*)take(vslots * 8 * 3 * 1024);
    w->m = (u32x4*)take(grad ? 0 : vslots * 8 * 3 * 1024);
    w->tt = (u32x4*)take(grad ? vslots * 8 * 3 * 1024 : 0);
    w->mt = (u32x4*)take(grad ? vslots * 8 * 3 * 1024 : 0);
    w->gates = (Gates*)take(vslots * (long long)sizeof(Gates));
    w->s0 = (float*)take(grad ? state : 0);
    w->ds = (float*)take(grad ? state : 0);
    w->u = (float*)take(grad ? rows : 0);
    w->dr = (float*)take(grad ? rows : 0);
    return total;
}

// Sixteens of columns of a chain's workgroup.  Its products are the same whatever the
// tile, so a wide one only saves loads; narrow ones make more workgroups, as long as
// there is a CU for each, or half of one where the registers allow it: in bf16, and in the
// joined chains.  1024 tokens, dims of 128, in us, narrow tiles | half as many wide ones.
// Forward, of 288 and 496 tiles: fp16 94 | 81 and 104 | 90, fp32 107 | 86 and 124 | 102; bf16 62 | 66
// and 69 | 71, of 528 90 | 114, of 768 99 | 121, of 1024 129 | 135, of 2048 316 | 289, and with
// dim_k 64 of 768 76 | 77, of 896 89 | 79.  Gradients of 288 and 496 tiles: fp32 313 | 281 and
// 433 | 372; joined, in bf16 of 288, 384 and 496 173 | 197, 197 | 210 and 262 | 254.
inline int chain_tiles(const Shape& a, long long most) {
    const long long narrow = (long long)a.n_seq * a.hv * ((a.dv + 15) / 16);
    return narrow > most && a.dv > 16 ? 2 : 1;
}
template <class TY>
constexpr long long kForwardNarrow = TY::NP == 1 ? 768 : 256;
template <class TY, int KS>
constexpr long long kBackwardNarrow = kJoined<TY, KS> ? 384 : 256;

// Eight elements of a 16-bit row are one aligned load.
inline bool eights(const void* p, long long st, long long sh, int dim) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && st % 8 == 0 && sh % 8 == 0 && dim % 8 == 0;
}

template <class TY, int KS, bool GRAD>
void launch_prep(const Shape& a, const Space& w, const void* q, const void* k, const float* g, const float* beta,
                 hipStream_t stream) {
    using S = typename TY::S;
    if (a.slots == 0) return;
    const bool vec = sizeof(S) == 4 ? a.qvec && a.kvec : eights(q, a.qt, a.qh, a.dk) && eights(k, a.kt, a.kh, a.dk);
    const auto kernel = vec ? delta_prep_kernel<TY, KS, GRAD, true> : delta_prep_kernel<TY, KS, GRAD, false>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)a.slots, a.hv + a.hk), dim3(kThreads), 0, stream, a, w, (const S*)q,
                       (const S*)k, g, beta);
}
template <class TY, int KS, int NCT, bool GRAD>
void launch_chain(const Shape& a, const Space& w, const void* v, const float* initial, void* o, float* final_state,
                  hipStream_t stream) {
    using S = typename TY::S;
    const int dv = GRAD ? w.dvp : a.dv;
    const long long count = (long long)a.n_seq * a.hv * ((dv + 16 * NCT - 1) / (16 * NCT));
    hipLaunchKernelGGL((delta_chain_kernel<TY, KS, NCT, GRAD>), dim3(dealt(count)), dim3(kThreads), 0, stream, a, w,
                       (const S*)v, initial, (S*)o, final_state);
}

template <class TY, int KS>
int run_forward(const Shape& a, const Space& w, const void* q, const void* k, const void* v, const float* g,
                const float* beta, const float* initial, void* o, float* final_state, hipStream_t stream) {
    launch_prep<TY, KS, false>(a, w, q, k, g, beta, stream);
    if (chain_tiles(a, kForwardNarrow<TY>) == 2)
        launch_chain<TY, KS, 2, false>(a, w, v, initial, o, final_state, stream);
    else
        launch_chain<TY, KS, 1, false>(a, w, v, initial, o, final_state, stream);
    return launch_status();
}

template <class TY, int KS, int NCT>
int run_backward(const Shape& a, const Space& w, const void* q, const void* k, const void* v, const float* g,
                 const float* beta, const float* initial, const void* go, const float* grad_final, void* gq, void* gk,
                 void* gv, float* gg, float* gbeta, float* grad_initial, hipStream_t stream) {
    using S = typename TY::S;
    constexpr bool joined = NCT == 1 && kJoined<TY, KS>;
    constexpr size_t lds_back = sizeof(ReverseLds<TY::NP, NCT, KS>);
    constexpr size_t lds = joined ? std::max(lds_back, sizeof(ChainLds<NCT, KS, true>)) : lds_back;
    // idempotent, and 160 KB is what a gfx950 workgroup can have
    auto allow = [](const void* kernel, size_t bytes) {
        return bytes <= 64 * 1024 || hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                                                         (int)bytes) == hipSuccess;
    };
    const void* chains;
    if constexpr (joined)
        chains = reinterpret_cast<const void*>(&delta_chains_kernel<TY, KS>);
    else
        chains = reinterpret_cast<const void*>(&delta_reverse_kernel<TY, KS, NCT>);
    if (!allow(chains, lds) ||
        !allow(reinterpret_cast<const void*>(&delta_grads_kernel<TY, KS>), sizeof(GradsLds<KS>)))
        return CFC_ERR_HIP;
    launch_prep<TY, KS, true>(a, w, q, k, g, beta, stream);
    const unsigned each = dealt((long long)a.n_seq * a.hv * (w.dvp / (16 * NCT)));
    if constexpr (joined) {
        hipLaunchKernelGGL((delta_chains_kernel<TY, KS>), dim3(2 * each), dim3(kThreads), lds, stream, a, w, each,
                           (const S*)v, initial, (const S*)go, grad_final, (S*)gv, grad_initial);
    } else {
        launch_chain<TY, KS, NCT, true>(a, w, v, initial, nullptr, nullptr, stream);
        hipLaunchKernelGGL((delta_reverse_kernel<TY, KS, NCT>), dim3(each), dim3(kThreads), lds, stream, a, w,
                           (const S*)go, grad_final, (S*)gv, grad_initial);
    }
    if (a.slots)
        hipLaunchKernelGGL((delta_grads_kernel<TY, KS>), dim3((unsigned)a.slots, a.hk), dim3(kGradThreads),
                           sizeof(GradsLds<KS>), stream, a,
                           w, (const S*)v, (const S*)go, (S*)gq, (S*)gk, gg, gbeta);
    return launch_status();
}

template <class TY, bool STEP>
int run_tokens(const Shape& a, const void* q, const void* k, const void* v, const float* g, const float* beta,
               const float* in, float* out, void* o, const int* slots, int pool, hipStream_t stream) {
    using S = typename TY::S;
    const long long count = (long long)a.n_seq * a.hv * ((a.dv + 31) / 32);
    const bool vec = a.dv % 4 == 0 && reinterpret_cast<uintptr_t>(in) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(out) % 16 == 0;
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(dealt((count + 3) / 4)), dim3(kThreads), 0, stream, a, (const S*)q,
                           (const S*)k, (const S*)v, g, beta, in, out, (S*)o, slots, pool, vec);
    };
    const bool past = (long long)a.n_seq * a.hv * a.dk * a.dv * 4 >= kPastCache;
    auto rows = [&](auto n) {
        constexpr int NR = decltype(n)::value;
        if constexpr (STEP) {
            if (past) return go(delta_token_kernel<TY, NR, true, true>);
        }
        go(delta_token_kernel<TY, NR, STEP, false>);
    };
    if (a.dk <= 16)
        rows(std::integral_constant<int, 2>{});
    else if (a.dk <= 32)
        rows(std::integral_constant<int, 4>{});
    else if (a.dk <= 64)
        rows(std::integral_constant<int, 8>{});
    else
        rows(std::integral_constant<int, 16>{});
    return launch_status();
}

struct Sizes {  // bytes of the arguments
    long long q, k, v, go, dq, dv, gates, states;
};
bool sizes_of(const delta_rule_shape_t* p, const Shape& a, Sizes* z) {
    const int size = size_of(p->type);
    const long long t = p->n_tokens;
    return extent(t, a.hk, a.dk, a.qt, a.qh, size, &z->q) && extent(t, a.hk, a.dk, a.kt, a.kh, size, &z->k) &&
           extent(t, a.hv, a.dv, a.vt, a.vh, size, &z->v) && extent(t, a.hv, a.dv, a.gt, a.gh, size, &z->go) &&
           mul_ok(t, (long long)a.hk * a.dk * size, &z->dq) && mul_ok(t, (long long)a.hv * a.dv * size, &z->dv) &&
           mul_ok(t, (long long)a.hv * 4, &z->gates) &&
           mul_ok((long long)a.n_seq * a.hv, (long long)a.dk * a.dv * 4, &z->states);
}
inline Range offsets_range(const Shape& a) {
    return bytes_of(a.offsets, a.offsets ? ((long long)a.n_seq + 1) * 4 : 0);
}

}  // namespace

// ================================================================ C ABI
extern "C" long long delta_rule_forward_workspace(const delta_rule_shape_t* shape) {
    Shape a;
    Space w;
    if (check_shape(shape, false, &a) != CFC_OK) return -1;
    if (is_short(a)) return 0;
    return rows_fit(shape) ? lay_out(a, shape->type, false, nullptr, &w) : -1;
}

extern "C" long long delta_rule_backward_workspace(const delta_rule_shape_t* shape) {
    Shape a;
    Space w;
    if (check_shape(shape, false, &a) != CFC_OK || !rows_fit(shape)) return -1;
    return lay_out(a, shape->type, true, nullptr, &w);
}

extern "C" int delta_rule_forward(const delta_rule_shape_t* shape, const void* q, const void* k, const void* v,
                                  const float* g, const float* beta, const float* initial_state, void* o,
                                  float* final_state, void* workspace, long long workspace_bytes,
                                  hipStream_t stream) {
    Shape a;
    if (const int e = check_shape(shape, false, &a)) return e;
    const bool brief = is_short(a);
    if (!brief && !rows_fit(shape)) return CFC_ERR_UNSUPPORTED;
    Sizes z;
    if (!sizes_of(shape, a, &z)) return CFC_ERR_DIM;
    if (a.n_seq == 0) return CFC_OK;
    if (a.n_tokens && (!q || !k || !v || !g || !beta || !o)) return CFC_ERR_NULL;
    Space w{};
    const long long need = brief ? 0 : lay_out(a, shape->type, false, workspace, &w);
    if (need) {
        if (!workspace) return CFC_ERR_NULL;
        if (workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 16) return CFC_ERR_DIM;
    }
    const Range fin = bytes_of(final_state, z.states), ini = bytes_of(initial_state, z.states);
    const Range outs[] = {bytes_of(o, z.dv), fin, bytes_of(need ? workspace : nullptr, need)};
    const Range ins[] = {bytes_of(q, z.q),        bytes_of(k, z.k), bytes_of(v, z.v), bytes_of(g, z.gates),
                         bytes_of(beta, z.gates), offsets_range(a), same(fin, ini) ? Range{0, 0} : ini};
    if (!outputs_disjoint(outs, 3, ins, 7)) return CFC_ERR_OVERLAP;
    set_vec(shape, &a, q, k, v, nullptr);
    if (brief) {
        auto tokens = [&](auto type) {
            return run_tokens<decltype(type), false>(a, q, k, v, g, beta, initial_state, final_state, o, nullptr, 0,
                                                     stream);
        };
        switch (shape->type) {
            case CFC_TYPE_F32: return tokens(F32{});
            case CFC_TYPE_BF16: return tokens(BF16{});
            default: return tokens(F16{});
        }
    }
    auto go = [&](auto type) {
        using TY = decltype(type);
        return a.dk <= 64 ? run_forward<TY, 2>(a, w, q, k, v, g, beta, initial_state, o, final_state, stream)
                          : run_forward<TY, 4>(a, w, q, k, v, g, beta, initial_state, o, final_state, stream);
    };
    switch (shape->type) {
        case CFC_TYPE_F32: return go(F32{});
        case CFC_TYPE_BF16: return go(BF16{});
        default: return go(F16{});
    }
}

extern "C" int delta_rule_backward(const delta_rule_shape_t* shape, const void* q, const void* k, const void* v,
                                   const float* g, const float* beta, const float* initial_state,
                                   const void* grad_o, const float* grad_final_state, void* grad_q, void* grad_k,
                                   void* grad_v, float* grad_g, float* grad_beta, float* grad_initial_state,
                                   void* workspace, long long workspace_bytes, hipStream_t stream) {
    Shape a;
    if (const int e = check_shape(shape, false, &a)) return e;
    if (!rows_fit(shape)) return CFC_ERR_UNSUPPORTED;
    Sizes z;
    if (!sizes_of(shape, a, &z)) return CFC_ERR_DIM;
    if (a.n_seq == 0) return CFC_OK;
    if (a.n_tokens &&
        (!q || !k || !v || !g || !beta || !grad_o || !grad_q || !grad_k || !grad_v || !grad_g || !grad_beta))
        return CFC_ERR_NULL;
    Space w{};
    const long long need = lay_out(a, shape->type, true, workspace, &w);
    if (need) {
        if (!workspace) return CFC_ERR_NULL;
        if (workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 16) return CFC_ERR_DIM;
    }
    const Range gin = bytes_of(grad_initial_state, z.states), gfin = bytes_of(grad_final_state, z.states);
    const Range outs[] = {bytes_of(grad_q, z.dq), bytes_of(grad_k, z.dq), bytes_of(grad_v, z.dv),
                          bytes_of(grad_g, z.gates), bytes_of(grad_beta, z.gates), bytes_of(workspace, need), gin};
    const Range ins[] = {bytes_of(q, z.q), bytes_of(k, z.k), bytes_of(v, z.v), bytes_of(g, z.gates),
                         bytes_of(beta, z.gates), bytes_of(grad_o, z.go), bytes_of(initial_state, z.states),
                         offsets_range(a), same(gin, gfin) ? Range{0, 0} : gfin};
    if (!outputs_disjoint(outs, 7, ins, 9)) return CFC_ERR_OVERLAP;
    set_vec(shape, &a, q, k, v, grad_o);
    auto go = [&](auto type) {
        using TY = decltype(type);
        auto run = [&](auto f) {
            return f(a, w, q, k, v, g, beta, initial_state, grad_o, grad_final_state, grad_q, grad_k, grad_v, grad_g,
                     grad_beta, grad_initial_state, stream);
        };
        if (a.dk <= 64)
            return chain_tiles(a, kBackwardNarrow<TY, 2>) == 2 ? run(run_backward<TY, 2, 2>) : run(run_backward<TY, 2, 1>);
        return chain_tiles(a, kBackwardNarrow<TY, 4>) == 2 ? run(run_backward<TY, 4, 2>) : run(run_backward<TY, 4, 1>);
    };
    switch (shape->type) {
        case CFC_TYPE_F32: return go(F32{});
        case CFC_TYPE_BF16: return go(BF16{});
        default: return go(F16{});
    }
}

extern "C" int delta_rule_step(const delta_rule_shape_t* shape, const void* q, const void* k, const void* v,
                               const float* g, const float* beta, float* states, int pool, const int* slots, void* o,
                               hipStream_t stream) {
    Shape a;
    if (const int e = check_shape(shape, true, &a)) return e;
    Sizes z;
    long long held;
    if (pool < 0 || (!slots && pool < a.n_seq) || !sizes_of(shape, a, &z) ||
        !mul_ok((long long)pool * a.hv, (long long)a.dk * a.dv * 4, &held))
        return CFC_ERR_DIM;
    if (a.n_seq == 0) return CFC_OK;
    if (!q || !k || !v || !g || !beta || !o || (pool && !states)) return CFC_ERR_NULL;
    const Range outs[] = {bytes_of(o, z.dv), bytes_of(states, held)};
    const Range ins[] = {bytes_of(q, z.q), bytes_of(k, z.k), bytes_of(v, z.v), bytes_of(g, z.gates),
                         bytes_of(beta, z.gates), bytes_of(slots, (long long)a.n_seq * 4)};
    if (!outputs_disjoint(outs, 2, ins, 6)) return CFC_ERR_OVERLAP;
    set_vec(shape, &a, q, k, v, nullptr);
    switch (shape->type) {
        case CFC_TYPE_F32: return run_tokens<F32, true>(a, q, k, v, g, beta, states, states, o, slots, pool, stream);
        case CFC_TYPE_BF16: return run_tokens<BF16, true>(a, q, k, v, g, beta, states, states, o, slots, pool, stream);
        default: return run_tokens<F16, true>(a, q, k, v, g, beta, states, states, o, slots, pool, stream);
    }
}
