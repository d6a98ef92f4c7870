// selective_scan.hip -- gfx950 kernels and C ABI of the selective scan (see
// include/selective_scan.h).
//
// h_t = a_t h_{t-1} + b_t is linear in h, so a stretch of tokens from any state h is
// P h + h', with P the product of its a_t (one exponential of the sum of the steps) and h'
// what it makes of zeros.  A workgroup has 16 channels of a sequence and goes along it by
// blocks of tokens, each of its waves with T of a block's: a wave computes its P and h' with
// its a_t and b_t kept in registers, the waves exchange P and h' through LDS, and each goes
// over its tokens again from the state that it now knows, one multiply-add each and no
// exponential.
//
// Four lanes have a channel, with S states each.  What is done once for each token and
// channel (softplus, the gate) lane j of the four does for the tokens 4 i + j, and the
// others take it through a lane permutation; b and c are turned to 32 bits once for all of
// a wave's channels and read from LDS.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>

#include "elements.h"
#include "functions.h"
#include "selective_scan.h"
#include "sequences.h"

namespace {

constexpr int kGroupCh = 16;  // channels of a workgroup

// Tokens of a wave and waves of a workgroup, by the states of a lane: what is kept of a
// token are 2 S registers.
constexpr int tokens_of(int s) { return s <= 4 ? 8 : 4; }
constexpr int waves_of(int s) { return s <= 8 ? 8 : 4; }
constexpr int forward_tokens(int s) { return s <= 2 ? 8 : 4; }
// Workgroups (16 channels of a sequence each) up to which each has 16 waves instead of 8, since
// there is at most one for a CU.  bf16, in us, 16 waves | 8: 4096 tokens in 256 workgroups with 4
// states 73 | 94, 8 states 79 | 100, 16 states 104 | 129, 32 states 180 | 218 (the kernel of 16
// waves spills 11 registers there, and is faster all the same); in 16 workgroups 54 | 78, 61 | 90,
// 96 | 128, 175 | 213; 2048 tokens in 512 workgroups 75 | 75, 82 | 83, 110 | 107, 186 | 172.  The
// gradients' states of 4096 tokens in 256 workgroups, with all of the gradients: 4 states 273 | 282,
// 16 states 495 | 510; 2048 in 512 the same.  Overlapping rows of b and c are left to 8: the branch
// for them (Shared::load) costs the kernel of 16 waves 20 of its 200 us.
constexpr long long kFewWorkgroups = 256;
constexpr int block_of(int s) { return tokens_of(s) * waves_of(s); }
constexpr int forward_block(int s, int waves) { return forward_tokens(s) * waves; }
// Rows of a block are reached from its first one by 32 bits, with kNowhere behind all of them:
// what every call's strides leave room for.  Blocks of more rows ask for themselves (reaches).
constexpr int kBlockRows = 64;

struct Scan {
    Sequences q;
    int channels, groups, share, state;  // share: channels of a group
    int softplus, clear;
    long long xt, dtt, zt, gt, bt, bg, ct, cg;
    bool single;   // sequences of one row, whose strides may be anything
    bool overlap;  // rows of b or c behind a sequence's end read as some of its own
};

// ------------------------------------------------------------------- lanes
template <int CTRL>
__device__ __forceinline__ float quad_perm(float x) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}
// Lane J of each four lanes' value.
template <int J>
__device__ __forceinline__ float from_lane(float x) {
    return quad_perm<J * 0x55>(x);
}
// Lane j of each four gets the sum over them of v[j].
__device__ __forceinline__ float over_four(const float (&v)[4]) {
    const bool odd = threadIdx.x & 1, high = threadIdx.x & 2;
    const float a = (odd ? v[1] : v[0]) + quad_perm<0xB1>(odd ? v[0] : v[1]);
    const float b = (odd ? v[3] : v[2]) + quad_perm<0xB1>(odd ? v[2] : v[3]);
    return (high ? b : a) + quad_perm<0x4E>(high ? a : b);
}

// The lanes' channels of a sixteen of a group of those that share b and c.
struct Place {
    int ch, quad, j;
    bool in;
};
__device__ __forceinline__ Place place_of(int share, int group, int sixteen) {
    const int lane = threadIdx.x & 63;
    Place p;
    p.quad = lane >> 2;
    p.j = lane & 3;
    const int at = sixteen * kGroupCh + p.quad;
    p.in = at < share;
    p.ch = group * share + min(at, share - 1);
    return p;
}

// S values from `n` on of a row of `state` floats; `none` beyond.
template <int S>
__device__ __forceinline__ void load_states(const float* row, int n, int state, float none, float (&h)[S]) {
#pragma unroll
    for (int s = 0; s < S; ++s) h[s] = n + s < state ? row[n + s] : none;
}

// What a wave's lanes write to LDS for each other: its own LDS instructions go in order.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}
// The barrier of a workgroup's exchanges through LDS; global loads stay in flight.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// An element as it lies in memory, through a descriptor.
template <class TY>
__device__ __forceinline__ uint32_t load_raw(Buffer b, uint32_t at) {
    if constexpr (sizeof(typename TY::S) == 4)
        return __builtin_amdgcn_raw_buffer_load_b32(b, at, 0, 0);
    else
        return __builtin_amdgcn_raw_buffer_load_b16(b, at, 0, 0);
}
template <class TY>
__device__ __forceinline__ float value_of(uint32_t raw) {
    if constexpr (sizeof(typename TY::S) == 4)
        return __uint_as_float(raw);
    else
        return TY::load(__builtin_bit_cast(typename TY::S, (uint16_t)raw));
}
template <class TY>
__device__ __forceinline__ void store_to(Buffer b, uint32_t at, float x) {
    if constexpr (sizeof(typename TY::S) == 4)
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x), b, at, 0, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, TY::store(x)), b, at, 0, 0);
}

// The rows of a tensor from one on, for a block of tokens at a time: those behind the
// sequence's end read as zeros and are not written, so that nothing needs a branch.  (Where
// rows overlap, at a stride below their width, they read as something, so what is made of
// them is set to zero: an infinite one times a step of zero would be no number.)
struct Rows {
    const char* at;
    int bytes, width;  // from a row to the next, and of a row
    template <class E>
    __device__ __forceinline__ Rows(const E* p, long long row, long long stride, bool single, int elements)
        : at(p ? reinterpret_cast<const char*>(p + row * stride) : nullptr),
          bytes(p && !single ? (int)stride * (int)sizeof(E) : 0), width(p ? elements * (int)sizeof(E) : 0) {}
    // The next n of them, of which there are some (or there may be none).
    __device__ __forceinline__ Buffer some(int n) const { return buffer_of(at, (n - 1) * bytes + width); }
    __device__ __forceinline__ Buffer next(int n) const { return buffer_of(at, n > 0 ? (n - 1) * bytes + width : 0); }
    __device__ __forceinline__ void move(int n) { at += (long long)n * bytes; }
};
// A lane's places in a block: its element of the rows row, row + 4, ...
template <class TY, int Q>
struct Places {
    uint32_t at[Q];
    __device__ __forceinline__ Places(const Rows& r, int row, int column) {
#pragma unroll
        for (int i = 0; i < Q; ++i) at[i] = (row + 4 * i) * (uint32_t)r.bytes + column * (uint32_t)sizeof(typename TY::S);
    }
};
// b or c of a wave's T tokens: loaded as they are, and put to LDS as 32-bit floats [T][4 S].
template <class TY, int S, int T>
struct Shared {
    static constexpr int N = (T * 4 * S + 63) / 64;
    static constexpr bool all = T * 4 * S % 64 == 0;
    uint32_t at[N], raw[N];
    __device__ __forceinline__ Shared(const Rows& r, int row, int state) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = i * 64 + (threadIdx.x & 63), n = e % (4 * S);
            at[i] = n < state && (all || e < T * 4 * S)
                        ? (row + e / (4 * S)) * (uint32_t)r.bytes + n * (uint32_t)sizeof(typename TY::S)
                        : kNowhere;
        }
    }
    // `left`: of the wave's tokens, those that there are.  Rows behind them read as zeros by
    // themselves, except where rows overlap.
    __device__ __forceinline__ void load(Buffer b, bool overlap, int left) {
        if (overlap && left < T) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int e = i * 64 + (threadIdx.x & 63);
                raw[i] = load_raw<TY>(b, e / (4 * S) < left ? at[i] : kNowhere);
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) raw[i] = load_raw<TY>(b, at[i]);
        }
    }
    __device__ __forceinline__ void put(float* to) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = i * 64 + (threadIdx.x & 63);
            if (all || e < T * 4 * S) to[e] = value_of<TY>(raw[i]);
        }
    }
};

// S floats of each lane in LDS: [S / V][64 lanes][V], V of them one access.  As a whole
// they are 64 S floats, of channel quad_of(f) and state state_of(f).
template <int S>
struct Lanes {
    static constexpr int V = S < 4 ? S : 4;
    typedef float vec __attribute__((ext_vector_type(V)));
    alignas(16) float x[64 * S];
    __device__ __forceinline__ void put(int lane, const float (&h)[S]) {
#pragma unroll
        for (int i = 0; i < S / V; ++i) {
            vec v;
#pragma unroll
            for (int k = 0; k < V; ++k) v[k] = h[i * V + k];
            *reinterpret_cast<vec*>(x + (i * 64 + lane) * V) = v;
        }
    }
    __device__ __forceinline__ void get(int lane, float (&h)[S]) const {
#pragma unroll
        for (int i = 0; i < S / V; ++i) {
            const vec v = *reinterpret_cast<const vec*>(x + (i * 64 + lane) * V);
#pragma unroll
            for (int k = 0; k < V; ++k) h[i * V + k] = v[k];
        }
    }
    static __device__ __forceinline__ int quad_of(int f) { return f % (64 * V) / V >> 2; }
    static __device__ __forceinline__ int state_of(int f) { return (f % (64 * V) / V & 3) * S + f / (64 * V) * V + f % V; }
};
// S neighbouring floats, V of them one access.
template <int S>
__device__ __forceinline__ void get_states(const float* p, float (&h)[S]) {
    constexpr int V = S < 4 ? S : 4;
    typedef float vec __attribute__((ext_vector_type(V)));
#pragma unroll
    for (int i = 0; i < S / V; ++i) {
        const vec v = *reinterpret_cast<const vec*>(p + i * V);
#pragma unroll
        for (int k = 0; k < V; ++k) h[i * V + k] = v[k];
    }
}

// The sum of a stretch's steps from four lanes' own, finite where the steps are: a rate of zero (that
// of a lane's states behind `state` among them) keeps its state.  Only rates under 2^-120 tell the
// largest float from what a sum beyond it should be.
__device__ __forceinline__ float steps_of(float all) {
    all += quad_perm<0xB1>(all);
    all += quad_perm<0x4E>(all);
    return __builtin_amdgcn_fmed3f(all, -FLT_MAX, FLT_MAX);
}
// A state behind a stretch, where going along all of them has ended in no number: P may be infinite
// and the state zero.  (Taken at every stretch, the choice would cost 8192 tokens 242 us, not 195.)
__device__ __forceinline__ float behind(float p, float h, float made) { return h == 0.0f ? made : fmaf(p, h, made); }

// The waves' exchange, between two barriers: a thread has one or several of the 64 S states
// of the workgroup's channels (of a state's gradients, with `back`), and goes along the
// waves' stretches, leaving each the state that it begins with in the place of what it made
// of zeros.  F states a thread, f = f0 + i * threads.
template <int S, int NW, bool back>
__device__ __forceinline__ float along(const Lanes<S> (&product)[NW], Lanes<S> (&made)[NW], int f, float h) {
    float p[NW], m[NW];
#pragma unroll
    for (int i = 0; i < NW; ++i) p[i] = product[i].x[f], m[i] = made[i].x[f];
    const float begin = h;
#pragma unroll
    for (int k = 0; k < NW; ++k) {
        const int i = back ? NW - 1 - k : k;
        made[i].x[f] = h;
        h = fmaf(p[i], h, m[i]);
    }
    if (__builtin_expect(__any(h != h), 0)) {
        h = begin;
#pragma unroll
        for (int k = 0; k < NW; ++k) {
            const int i = back ? NW - 1 - k : k;
            made[i].x[f] = h;
            h = behind(p[i], h, m[i]);
        }
    }
    return h;
}

// -------------------------------------------------------------------- forward
// Bound by the vector units: an element (token, channel, state) takes an exponential, its
// argument's product, D x b, the two passes' multiply-adds and c's, and a token and channel's
// softplus and gate about 60 instructions over its 16 states: 10.3 instructions by the counters,
// 11.8 issue slots, for which 8192 tokens x 4096 channels x 16 states keep the vector units
// busy 161 us of 202.  Measured 181 in four sequences, 195 in one (1.38 TB/s).
template <class TY, int S, int NW>
__global__ __launch_bounds__(64 * NW, S == 16 ? 2 : S == 8 || S == 2 || NW == 16 ? 4 : 6) void scan_kernel(
    Scan a, int sixteens, const typename TY::S* __restrict__ x, const typename TY::S* __restrict__ dt,
    const float* __restrict__ decay, const typename TY::S* __restrict__ b, const typename TY::S* __restrict__ c,
    const float* __restrict__ d, const typename TY::S* __restrict__ z, const float* __restrict__ dt_bias,
    const float* initial, typename TY::S* __restrict__ y, float* final) {
    constexpr int T = forward_tokens(S), Q = T / 4, BT = forward_block(S, NW), F = (S + NW - 1) / NW;
    static_assert(NW == 16 || BT <= kBlockRows, "rows of a block");
    __shared__ Lanes<S> product[NW], made[NW];  // P and h' of each wave
    __shared__ alignas(16) float bc[NW][2][T * 4 * S];
    const long long count = (long long)a.groups * sixteens * a.q.n_seq, index = on_die(blockIdx.x, count);
    if (index >= count) return;
    const int sixteen = (int)(index % sixteens), group = (int)(index / sixteens % a.groups);
    const int seq = (int)(index / sixteens / a.groups), lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Place p = place_of(a.share, group, sixteen);
    const int n0 = p.j * S, row = w * T + p.j;
    int first, end;
    span_of(a.q, seq, first, end);
    const int len = end - first;
    float a2[S];
    load_states<S>(decay + (long long)p.ch * a.state, n0, a.state, 0.0f, a2);
#pragma unroll
    for (int s = 0; s < S; ++s) a2[s] *= kLog2e;
    const float skip = d ? d[p.ch] : 0.0f, bias = dt_bias ? dt_bias[p.ch] : 0.0f;
    // the states that this thread takes along, as the exchange has them
    const long long kept = ((long long)seq * a.channels + group * a.share) * a.state;
    auto state_at = [&](int i, long long* at) {
        const int f = threadIdx.x + i * 64 * NW, ch = sixteen * kGroupCh + Lanes<S>::quad_of(f), n = Lanes<S>::state_of(f);
        *at = kept + (long long)ch * a.state + n;
        return f < 64 * S && ch < a.share && n < a.state;
    };
    float h[F];
#pragma unroll
    for (int i = 0; i < F; ++i) {
        long long at;
        h[i] = state_at(i, &at) && initial ? initial[at] : 0.0f;
    }
    Rows xs(x, first, a.xt, a.single, a.channels), dts(dt, first, a.dtt, a.single, a.channels),
        zs(z, first, a.zt, a.single, a.channels), bs(b + group * a.bg, first, a.bt, a.single, a.state),
        cs(c + group * a.cg, first, a.ct, a.single, a.state), ys(y, first, a.channels, false, a.channels);
    const Places<TY, Q> xa(xs, row, p.ch), dta(dts, row, p.ch), za(zs, row, p.ch), ya(ys, row, p.ch);
    Shared<TY, S, T> bl(bs, w * T, a.state), cl(cs, w * T, a.state);
    uint32_t xr[Q], dtr[Q], zr[Q];
    auto fetch = [&](int left) {
        const int n = min(left, BT);
        const Buffer xb = xs.next(n), db = dts.next(n), zb = zs.next(n);
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            xr[i] = load_raw<TY>(xb, xa.at[i]);
            dtr[i] = load_raw<TY>(db, dta.at[i]);
            zr[i] = load_raw<TY>(zb, za.at[i]);
        }
        bl.load(bs.next(n), NW < 16 && a.overlap, n - w * T);
        cl.load(cs.next(n), NW < 16 && a.overlap, n - w * T);
        xs.move(BT), dts.move(BT), zs.move(BT), bs.move(BT), cs.move(BT);
    };
    fetch(len);
    for (int left = len; left > 0; left -= BT) {
        wave_fence();
        bl.put(bc[w][0]);
        cl.put(bc[w][1]);
        wave_fence();
        float xv[Q], step[Q], u[Q], gate[Q], all = 0.0f;
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            const bool in = row + 4 * i < left;
            xv[i] = in ? value_of<TY>(xr[i]) : 0.0f;
            const float pre = value_of<TY>(dtr[i]) + bias;
            step[i] = in ? (a.softplus ? softplus_of(pre) : pre) : 0.0f;
            u[i] = step[i] * xv[i];
            all += step[i];
            const float zv = value_of<TY>(zr[i]);
            gate[i] = z ? zv * gate_of<TY>(zv) : 1.0f;
        }
        fetch(left - BT);  // while this block is worked on
        all = steps_of(all);
        float at[T][S], add[T][S], hl[S], pw[S];
#pragma unroll
        for (int s = 0; s < S; ++s) hl[s] = 0.0f, pw[s] = exp2_of(all * a2[s]);
        auto one = [&](auto k, int i) {
            constexpr int J = decltype(k)::value;
            const int t = 4 * i + J;
            const float dl = from_lane<J>(step[i]), ul = from_lane<J>(u[i]);
            float bv[S];
            get_states<S>(&bc[w][0][t * 4 * S + n0], bv);
#pragma unroll
            for (int s = 0; s < S; ++s) {
                at[t][s] = exp2_of(dl * a2[s]);
                add[t][s] = ul * bv[s];
                hl[s] = fmaf(at[t][s], hl[s], add[t][s]);
            }
        };
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            one(std::integral_constant<int, 0>{}, i);
            one(std::integral_constant<int, 1>{}, i);
            one(std::integral_constant<int, 2>{}, i);
            one(std::integral_constant<int, 3>{}, i);
        }
        product[w].put(lane, pw);
        made[w].put(lane, hl);
        lds_barrier();
#pragma unroll
        for (int i = 0; i < F; ++i)
            if (w * 64 + i * 64 * NW < 64 * S) h[i] = along<S, NW, false>(product, made, threadIdx.x + i * 64 * NW, h[i]);
        lds_barrier();
        made[w].get(lane, hl);
        const Buffer yb = ys.next(min(left, BT));
        ys.move(BT);
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = 4 * i + k;
                float cv[S];
                get_states<S>(&bc[w][1][t * 4 * S + n0], cv);
                v[k] = 0.0f;
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    hl[s] = fmaf(at[t][s], hl[s], add[t][s]);
                    v[k] = fmaf(cv[s], hl[s], v[k]);
                }
            }
            store_to<TY>(yb, p.in ? ya.at[i] : kNowhere, fmaf(skip, xv[i], over_four(v)) * gate[i]);
        }
    }
    if (final)
#pragma unroll
        for (int i = 0; i < F; ++i) {
            long long at;
            if (state_at(i, &at)) final[at] = h[i];
        }
    if ((a.clear & SELECTIVE_SCAN_CLEAR_Y) && seq == a.q.n_seq - 1 && p.in)
        for (int t = end + 4 * w + p.j; t < a.q.n_tokens; t += 4 * NW)
            y[(long long)t * a.channels + p.ch] = TY::store(0.0f);
}

// ------------------------------------------------------------------- backward
// With G_t the gradient of h_t, and e what comes to it from behind,
//   G_t = c_t gy_t + e,  e' = a_t G_t,
// which is linear in e as the forward is in h, and is cut into the same stretches.

// The states before each block of block_of(S) tokens, to kept[slot][group][sixteen][64 S] as
// the exchange has them: the forward without its second pass, 69 us of the 391 of the
// gradients of 4 x 2048 tokens x 2048 channels x 16 states, 73 % of them the vector units'.
template <class TY, int S, int NW>
__global__ __launch_bounds__(64 * NW) void scan_states_kernel(
    Scan a, int sixteens, const typename TY::S* __restrict__ x, const typename TY::S* __restrict__ dt,
    const float* __restrict__ decay, const typename TY::S* __restrict__ b, const float* __restrict__ dt_bias,
    const float* __restrict__ initial, float* __restrict__ kept) {
    constexpr int BT = block_of(S), T = BT / NW, Q = T / 4, F = (S + NW - 1) / NW;
    static_assert(BT <= kBlockRows, "rows of a block");
    __shared__ Lanes<S> product[2][NW], made[2][NW];
    __shared__ alignas(16) float bc[NW][T * 4 * S];
    const long long count = (long long)a.groups * sixteens * a.q.n_seq, index = on_die(blockIdx.x, count);
    if (index >= count) return;
    const int sixteen = (int)(index % sixteens), group = (int)(index / sixteens % a.groups);
    const int seq = (int)(index / sixteens / a.groups), lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Place p = place_of(a.share, group, sixteen);
    const int n0 = p.j * S, row = w * T + p.j;
    int first, end;
    span_of(a.q, seq, first, end);
    const int len = end - first;
    float a2[S];
    load_states<S>(decay + (long long)p.ch * a.state, n0, a.state, 0.0f, a2);
#pragma unroll
    for (int s = 0; s < S; ++s) a2[s] *= kLog2e;
    const float bias = dt_bias ? dt_bias[p.ch] : 0.0f;
    float h[F];
#pragma unroll
    for (int i = 0; i < F; ++i) {
        const int f = threadIdx.x + i * 64 * NW, ch = sixteen * kGroupCh + Lanes<S>::quad_of(f), n = Lanes<S>::state_of(f);
        h[i] = initial && f < 64 * S && ch < a.share && n < a.state
                   ? initial[((long long)seq * a.channels + group * a.share + ch) * a.state + n]
                   : 0.0f;
    }
    Rows xs(x, first, a.xt, a.single, a.channels), dts(dt, first, a.dtt, a.single, a.channels),
        bs(b + group * a.bg, first, a.bt, a.single, a.state);
    const Places<TY, Q> xa(xs, row, p.ch), dta(dts, row, p.ch);
    Shared<TY, S, T> bl(bs, w * T, a.state);
    uint32_t xr[Q], dtr[Q];
    auto fetch = [&](int left) {
        const int n = min(left, BT);
        const Buffer xb = xs.next(n), db = dts.next(n);
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            xr[i] = load_raw<TY>(xb, xa.at[i]);
            dtr[i] = load_raw<TY>(db, dta.at[i]);
        }
        bl.load(bs.next(n), NW < 16 && a.overlap, n - w * T);
        xs.move(BT), dts.move(BT), bs.move(BT);
    };
    fetch(len);
    const long long pitch = (long long)a.groups * sixteens * (64 * S);
    float* to = kept + ((long long)first / BT + seq) * pitch + ((long long)group * sixteens + sixteen) * (64 * S);
    int turn = 0;  // one barrier a block: the exchange is done with one while the next is made
    for (int left = len; left > 0; left -= BT, to += pitch, turn ^= 1) {
        wave_fence();
        bl.put(bc[w]);
        wave_fence();
        float step[Q], u[Q], all = 0.0f;
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            const bool in = row + 4 * i < left && p.in;
            const float pre = value_of<TY>(dtr[i]) + bias;
            step[i] = in ? (a.softplus ? softplus_of(pre) : pre) : 0.0f;
            u[i] = step[i] * (in ? value_of<TY>(xr[i]) : 0.0f);
            all += step[i];
        }
        fetch(left - BT);  // while this block is worked on
        all = steps_of(all);
        float hl[S], pw[S];
#pragma unroll
        for (int s = 0; s < S; ++s) hl[s] = 0.0f, pw[s] = exp2_of(all * a2[s]);
        auto one = [&](auto k, int i) {
            constexpr int J = decltype(k)::value;
            const float dl = from_lane<J>(step[i]), ul = from_lane<J>(u[i]);
            float bv[S];
            get_states<S>(&bc[w][(4 * i + J) * 4 * S + n0], bv);
#pragma unroll
            for (int s = 0; s < S; ++s) hl[s] = fmaf(exp2_of(dl * a2[s]), hl[s], ul * bv[s]);
        };
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            one(std::integral_constant<int, 0>{}, i);
            one(std::integral_constant<int, 1>{}, i);
            one(std::integral_constant<int, 2>{}, i);
            one(std::integral_constant<int, 3>{}, i);
        }
        product[turn][w].put(lane, pw);
        made[turn][w].put(lane, hl);
        lds_barrier();
#pragma unroll
        for (int i = 0; i < F; ++i)
            if (w * 64 + i * 64 * NW < 64 * S) {
                const int f = threadIdx.x + i * 64 * NW;
                to[f] = h[i];
                const float begin = h[i];
#pragma unroll
                for (int k = 0; k < NW; ++k) h[i] = fmaf(product[turn][k].x[f], h[i], made[turn][k].x[f]);
                if (__builtin_expect(__any(h[i] != h[i]), 0)) {
                    h[i] = begin;
                    for (int k = 0; k < NW; ++k) h[i] = behind(product[turn][k].x[f], h[i], made[turn][k].x[f]);
                }
            }
    }
}

struct Grads {  // the backward's outputs and workspace
    void *x, *dt, *z;
    float *initial, *kept, *part_b, *part_c, *part_a, *part_d, *part_bias;
    long long rows;  // of part_b and part_c: n_tokens * groups * state
};

// Sums over the 16 lanes of the same place in their four: of 16 values, lane l gets that of
// value sixteenth_of(l).  Two lanes' halves change places and are added, four times over.
__device__ __forceinline__ int sixteenth_of(int lane) {
    return (lane >> 5 & 1) + 2 * (lane >> 4 & 1) + 4 * (lane >> 3 & 1) + 8 * (lane >> 2 & 1);
}
__device__ __forceinline__ float over_quads(const float (&v)[16]) {
    float a[8], b[4], c[2];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[2 * i]), __float_as_uint(v[2 * i + 1]), false, false);
        a[i] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(a[2 * i]), __float_as_uint(a[2 * i + 1]), false, false);
        b[i] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    }
    const bool eight = threadIdx.x & 8, four = threadIdx.x & 4;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        // 8 lanes on
        const float lo = b[2 * i] + quad_perm<0x128>(b[2 * i]), hi = b[2 * i + 1] + quad_perm<0x128>(b[2 * i + 1]);
        c[i] = eight ? hi : lo;
    }
    const float lo = c[0] + quad_perm<0x104>(c[0]), hi = c[1] + quad_perm<0x114>(c[1]);  // 4 lanes on, 4 back
    return four ? hi : lo;
}

// A workgroup has K times 16 channels of a group, one after the other for each block of
// tokens, so that b's and c's gradients are summed over them before they leave it; and every
// parts-th sequence.  Bound by the vector units: 32 instructions an element by the counters, 34.7
// issue slots, of which the sums over channels and states are 6 and the passes of h and e 12;
// 302 us of the 391 above, 76 % of them those slots', with two waves a SIMD between its two
// barriers a step.
//
// What only a sequence's or the kernel's beginning and end need of the arguments is read from
// their segment again there (`fresh`): kept in scalar registers all along, it had those of the
// inner loop spilled to vector lanes, 150 of its 1400 instructions.
struct BackwardArgs {
    Scan a;
    int sixteens, wg_groups, parts;
    const void *x, *dt, *b, *c, *z, *gy;
    const float *decay, *d, *dt_bias, *gfinal;
    Grads g;
};
template <class A>
__device__ __forceinline__ const __attribute__((address_space(4))) A* fresh() {
    auto p = (const __attribute__((address_space(4))) A*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return p;
}

template <class TY, int S, int K>
__global__ __launch_bounds__(64 * waves_of(S)) void scan_backward_kernel(BackwardArgs) {
    constexpr int T = tokens_of(S), NW = waves_of(S), Q = T / 4, BT = T * NW, F = (2 * S + NW - 1) / NW;
    constexpr int N16 = (T * S + 15) / 16;
    static_assert(BT <= kBlockRows, "rows of a block");
    using E = typename TY::S;
    __shared__ Lanes<S> product[NW], made[NW], given[NW];  // P, h' and e' of each wave
    __shared__ Lanes<S> carry[K], rate[K];                 // e before a block, and log2(e) a
    __shared__ float2 skip_bias[K][kGroupCh];
    __shared__ alignas(16) float bc[NW][2][T * 4 * S];
    __shared__ double total[K][NW][S + 1][64];  // a's gradients, and d's and dt_bias's in lanes 0 and 1 of four
    const auto* const args = fresh<BackwardArgs>();
    const int wg_groups = args->wg_groups, parts = args->parts, sixteens = args->sixteens, groups = args->a.groups;
    const int share = args->a.share, state_size = args->a.state, channels = args->a.channels, n_seq = args->a.q.n_seq;
    const bool softplus = args->a.softplus, gated = args->z != nullptr, overlap = args->a.overlap;
    const long long count = (long long)wg_groups * parts, index = on_die(blockIdx.x, count);
    if (index >= count) return;
    const int wg = (int)(index % wg_groups), part = (int)(index / wg_groups);
    const int per_group = wg_groups / groups, group = wg / per_group, in_group = wg % per_group;
    const int k0 = in_group * K, nk = min(K, sixteens - k0);
    const int lane = threadIdx.x & 63, quad = lane >> 2, j = lane & 3;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n0 = j * S, row = w * T + j;
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int s = 0; s <= S; ++s) total[k][w][s][lane] = 0.0;
        if (w == k % NW && k < nk) {
            const Place p = place_of(share, group, k0 + k);
            float r[S];
            load_states<S>(args->decay + (long long)p.ch * state_size, n0, state_size, 0.0f, r);
#pragma unroll
            for (int s = 0; s < S; ++s) r[s] *= kLog2e;
            rate[k].put(lane, r);
            if (j == 0) skip_bias[k][quad] = float2{args->d ? args->d[p.ch] : 0.0f, args->dt_bias ? args->dt_bias[p.ch] : 0.0f};
        }
    }
    const long long pitch = (long long)groups * sixteens * (64 * S);
    __syncthreads();
    for (int seq = part; seq < n_seq; seq += parts) {
        const auto* const in = fresh<BackwardArgs>();
        int first, end;
        span_of(Sequences{in->a.q.offsets, n_seq, in->a.q.seq_len, in->a.q.n_tokens}, seq, first, end);
        const int len = end - first, blocks = (len + BT - 1) / BT;
        // states in the exchange's order: where they lie in a state array
        const long long state0 = ((long long)seq * channels + group * share) * state_size;
        auto state_at = [&](int f, int k, long long* at) {
            const int ch = (k0 + k) * kGroupCh + Lanes<S>::quad_of(f), n = Lanes<S>::state_of(f);
            *at = state0 + (long long)ch * state_size + n;
            return ch < share && n < state_size;
        };
        const float* const gfinal = in->gfinal;
        float* const initial = in->g.initial;
        // (a thread reads and writes its own of `carry` alone)
        for (int k = 0; k < nk; ++k)
#pragma unroll
            for (int i = 0; i < F; ++i) {
                const int f = threadIdx.x + i * 64 * NW - 64 * S;
                long long at;
                if (f >= 0 && f < 64 * S) carry[k].x[f] = state_at(f, k, &at) && gfinal ? gfinal[at] : 0.0f;
            }
        if (blocks) {
            const long long from = first + (blocks - 1) * (long long)BT;
            const bool single = in->a.single;
            Rows xs((const E*)in->x, from, in->a.xt, single, channels), dts((const E*)in->dt, from, in->a.dtt, single, channels),
                zs((const E*)in->z, from, in->a.zt, single, channels), gs((const E*)in->gy, from, in->a.gt, single, channels),
                bs((const E*)in->b + group * in->a.bg, from, in->a.bt, single, state_size),
                cs((const E*)in->c + group * in->a.cg, from, in->a.ct, single, state_size);
            const int pitch_out = channels * (int)sizeof(E);  // bytes of an output's row
            long long out_at = from * pitch_out;              // of the block's first
            const Places<TY, Q> xa(xs, row, group * share), dta(dts, row, group * share), za(zs, row, group * share),
                ga(gs, row, group * share);
            Shared<TY, S, T> bl(bs, w * T, state_size), cl(cs, w * T, state_size);
            const float* kept = in->g.kept + ((long long)first / BT + seq + blocks - 1) * pitch +
                                ((long long)group * sixteens + k0) * (64 * S);
            // where b's and c's gradients of the block go
            const long long row_bc = (long long)groups * state_size, leave0 = in_group * in->g.rows + group * state_size;
            uint32_t xr[Q], dtr[Q], zr[Q], gr[Q];
            float hr[F];
            auto fetch = [&](int n, int k) {
                const uint32_t off = min((k0 + k) * kGroupCh + quad, share - 1) * (uint32_t)sizeof(E);
                const Buffer xb = xs.some(n), db = dts.some(n), zb = zs.some(n), gb = gs.some(n);
#pragma unroll
                for (int i = 0; i < Q; ++i) {
                    xr[i] = load_raw<TY>(xb, xa.at[i] + off);
                    dtr[i] = load_raw<TY>(db, dta.at[i] + off);
                    zr[i] = load_raw<TY>(zb, za.at[i] + off);
                    gr[i] = load_raw<TY>(gb, ga.at[i] + off);
                }
                if (k == 0) {
                    bl.load(bs.some(n), overlap, n - w * T);
                    cl.load(cs.some(n), overlap, n - w * T);
                }
#pragma unroll
                for (int i = 0; i < F; ++i)
                    if (w * 64 + i * 64 * NW < 64 * S) hr[i] = kept[k * (64 * S) + threadIdx.x + i * 64 * NW];
            };
            int n = len - (blocks - 1) * BT;  // tokens of the block
            fetch(n, 0);
            for (int block = blocks - 1; block >= 0; --block, n = BT) {
                wave_fence();
                bl.put(bc[w][0]);
                cl.put(bc[w][1]);
                wave_fence();
                // over the K times 16 channels; the lane's of T * S values are those at 16 i + mine
                float sum_b[N16], sum_c[N16];
#pragma unroll
                for (int i = 0; i < N16; ++i) sum_b[i] = sum_c[i] = 0.0f;
                for (int k = 0; k < nk; ++k) {
                    const int ch = (k0 + k) * kGroupCh + quad;
                    const bool here = ch < share;
                    const float2 sb = skip_bias[k][quad];
                    float xv[Q], slope[Q], step[Q], u[Q], gv[Q], zv[Q], sig[Q], gp[Q], a2[S], all = 0.0f;
                    rate[k].get(lane, a2);
#pragma unroll
                    for (int i = 0; i < Q; ++i) {
                        const bool in = row + 4 * i < n && here;
                        xv[i] = in ? value_of<TY>(xr[i]) : 0.0f;
                        const float pre = value_of<TY>(dtr[i]) + sb.y, ex = exp_of(-fabsf(pre));
                        step[i] = in ? (softplus ? softplus_of(pre, ex) : pre) : 0.0f;
                        slope[i] = softplus ? sigmoid_of(pre, ex) : 1.0f;
                        u[i] = step[i] * xv[i];
                        all += step[i];
                        gv[i] = in ? value_of<TY>(gr[i]) : 0.0f;
                        zv[i] = in ? value_of<TY>(zr[i]) : 0.0f;
                        sig[i] = gated ? gate_of<TY>(zv[i]) : 1.0f;
                        gp[i] = gated ? gv[i] * (zv[i] * sig[i]) : gv[i];
                    }
                    float h0[F];
#pragma unroll
                    for (int i = 0; i < F; ++i) h0[i] = hr[i];
                    if (k + 1 < nk) {  // while this step is worked on
                        fetch(n, k + 1);
                    } else if (block) {
                        xs.move(-BT), dts.move(-BT), zs.move(-BT), gs.move(-BT), bs.move(-BT), cs.move(-BT);
                        kept -= pitch;
                        fetch(BT, 0);
                    }
                    all = steps_of(all);
                    float at[T][S], add[T][S], h[S], e[S], pw[S];
#pragma unroll
                    for (int s = 0; s < S; ++s) h[s] = e[s] = 0.0f, pw[s] = exp2_of(all * a2[s]);
                    auto one = [&](auto kk, int i) {
                        constexpr int J = decltype(kk)::value;
                        const int t = 4 * i + J;
                        const float dl = from_lane<J>(step[i]), ul = from_lane<J>(u[i]);
                        float bv[S];
                        get_states<S>(&bc[w][0][t * 4 * S + n0], bv);
#pragma unroll
                        for (int s = 0; s < S; ++s) {
                            at[t][s] = exp2_of(dl * a2[s]);
                            add[t][s] = ul * bv[s];
                            h[s] = fmaf(at[t][s], h[s], add[t][s]);
                        }
                    };
                    auto one_back = [&](auto kk, int i) {
                        constexpr int J = decltype(kk)::value;
                        const int t = 4 * i + J;
                        const float gl = from_lane<J>(gp[i]);
                        float cv[S];
                        get_states<S>(&bc[w][1][t * 4 * S + n0], cv);
#pragma unroll
                        for (int s = 0; s < S; ++s) e[s] = at[t][s] * fmaf(cv[s], gl, e[s]);
                    };
#pragma unroll
                    for (int i = 0; i < Q; ++i) {
                        one(std::integral_constant<int, 0>{}, i);
                        one(std::integral_constant<int, 1>{}, i);
                        one(std::integral_constant<int, 2>{}, i);
                        one(std::integral_constant<int, 3>{}, i);
                    }
#pragma unroll
                    for (int i = Q - 1; i >= 0; --i) {
                        one_back(std::integral_constant<int, 3>{}, i);
                        one_back(std::integral_constant<int, 2>{}, i);
                        one_back(std::integral_constant<int, 1>{}, i);
                        one_back(std::integral_constant<int, 0>{}, i);
                    }
                    product[w].put(lane, pw);
                    made[w].put(lane, h);
                    given[w].put(lane, e);
                    lds_barrier();
#pragma unroll
                    for (int i = 0; i < F; ++i) {
                        const int f = threadIdx.x + i * 64 * NW, wave0 = w * 64 + i * 64 * NW;
                        if (wave0 < 64 * S) {
                            along<S, NW, false>(product, made, f, h0[i]);
                        } else if (wave0 < 2 * 64 * S) {
                            const int r = f - 64 * S;
                            const float before = along<S, NW, true>(product, given, r, carry[k].x[r]);
                            carry[k].x[r] = before;
                            long long to;
                            if (block == 0 && initial && state_at(r, k, &to)) initial[to] = before;
                        }
                    }
                    lds_barrier();
                    made[w].get(lane, h);
                    given[w].get(lane, e);
                    float ypre[Q], gu[Q], gd[Q], das[S], vb[T * S], vc[T * S];
                    auto sum16 = [&](const float* from, float& to) {
                        float v[16];
#pragma unroll
                        for (int q = 0; q < 16; ++q) v[q] = from[q];
                        to += over_quads(v);
                    };
#pragma unroll
                    for (int s = 0; s < S; ++s) das[s] = 0.0f;
                    // forward: `add` becomes h_{t-1}
                    auto ahead = [&](auto kk, int i, float (&v)[4]) {
                        constexpr int J = decltype(kk)::value;
                        const int t = 4 * i + J;
                        const float gl = from_lane<J>(gp[i]);
                        float cv[S];
                        get_states<S>(&bc[w][1][t * 4 * S + n0], cv);
                        v[J] = 0.0f;
#pragma unroll
                        for (int s = 0; s < S; ++s) {
                            const float before = h[s];
                            h[s] = fmaf(at[t][s], before, add[t][s]);
                            add[t][s] = before;
                            v[J] = fmaf(cv[s], h[s], v[J]);
                            vc[t * S + s] = gl * h[s];
                        }
                    };
#pragma unroll
                    for (int i = 0; i < Q; ++i) {
                        float v[4];
                        ahead(std::integral_constant<int, 0>{}, i, v);
                        ahead(std::integral_constant<int, 1>{}, i, v);
                        ahead(std::integral_constant<int, 2>{}, i, v);
                        ahead(std::integral_constant<int, 3>{}, i, v);
                        ypre[i] = over_four(v);
#pragma unroll
                        for (int q = 0; q < S / 4; ++q) sum16(vc + (i * (S / 4) + q) * 16, sum_c[i * (S / 4) + q]);
                    }
                    auto back = [&](auto kk, int i, float (&v)[4], float (&r)[4]) {
                        constexpr int J = decltype(kk)::value;
                        const int t = 4 * i + J;
                        const float dl = from_lane<J>(step[i]), ul = from_lane<J>(u[i]), gl = from_lane<J>(gp[i]);
                        float bv[S], cv[S];
                        get_states<S>(&bc[w][0][t * 4 * S + n0], bv);
                        get_states<S>(&bc[w][1][t * 4 * S + n0], cv);
                        v[J] = r[J] = 0.0f;
#pragma unroll
                        for (int s = 0; s < S; ++s) {
                            const float G = fmaf(cv[s], gl, e[s]);
                            vb[t * S + s] = G * ul;
                            v[J] = fmaf(G, bv[s], v[J]);
                            e[s] = at[t][s] * G;
                            const float q = e[s] * add[t][s];
                            r[J] = fmaf(q, a2[s], r[J]);
                            das[s] = fmaf(q, dl, das[s]);
                        }
                    };
#pragma unroll
                    for (int i = Q - 1; i >= 0; --i) {
                        float v[4], r[4];
                        back(std::integral_constant<int, 3>{}, i, v, r);
                        back(std::integral_constant<int, 2>{}, i, v, r);
                        back(std::integral_constant<int, 1>{}, i, v, r);
                        back(std::integral_constant<int, 0>{}, i, v, r);
                        gu[i] = over_four(v);
                        gd[i] = over_four(r);
#pragma unroll
                        for (int q = 0; q < S / 4; ++q) sum16(vb + (i * (S / 4) + q) * 16, sum_b[i * (S / 4) + q]);
                    }
                    if constexpr (S == 2) {
                        sum16(vb, sum_b[0]);
                        sum16(vc, sum_c[0]);
                    } else if constexpr (S == 1) {  // eight of each are sixteen
                        float v[16];
#pragma unroll
                        for (int q = 0; q < 8; ++q) v[q] = vb[q], v[q + 8] = vc[q];
                        sum16(v, sum_b[0]);
                    }
                    const auto* const out = fresh<BackwardArgs>();
                    const Buffer gxb = buffer_of((char*)out->g.x + out_at, n * pitch_out),
                                 gdb = buffer_of((char*)out->g.dt + out_at, n * pitch_out),
                                 gzb = buffer_of((char*)out->g.z + out_at, n * pitch_out);
                    const uint32_t own = row * (uint32_t)pitch_out + (group * share + ch) * (uint32_t)sizeof(E);
                    float dd = 0.0f, db = 0.0f;
#pragma unroll
                    for (int i = 0; i < Q; ++i) {
                        const uint32_t to = here ? own + 4 * i * (uint32_t)pitch_out : kNowhere;
                        const float gdt = fmaf(gu[i], xv[i], gd[i] * kLn2) * slope[i];
                        store_to<TY>(gxb, to, fmaf(gu[i], step[i], sb.x * gp[i]));
                        store_to<TY>(gdb, to, gdt);
                        if (gated)
                            store_to<TY>(gzb, to, gv[i] * fmaf(sb.x, xv[i], ypre[i]) * (sig[i] * (1.0f + zv[i] * (1.0f - sig[i]))));
                        dd = fmaf(gp[i], xv[i], dd);
                        db += row + 4 * i < n && here ? gdt : 0.0f;
                    }
                    dd += quad_perm<0xB1>(dd);
                    dd += quad_perm<0x4E>(dd);
                    db += quad_perm<0xB1>(db);
                    db += quad_perm<0x4E>(db);
#pragma unroll
                    for (int s = 0; s < S; ++s) total[k][w][s][lane] += das[s];
                    total[k][w][S][lane] += j == 0 ? dd : db;
                }
                out_at -= BT * (long long)pitch_out;
                const int mine = sixteenth_of(lane);
                auto leave = [&](float v, int at, float* to) {  // of value `at` of the wave's T * S
                    const int t = w * T + at / S, state = n0 + at % S;
                    if (t < n && state < state_size) to[(first + block * (long long)BT + t) * row_bc + leave0 + state] = v;
                };
                const auto* const out = fresh<BackwardArgs>();
                float *const to_b = out->g.part_b, *const to_c = out->g.part_c;
                if constexpr (S == 1) {
                    leave(sum_b[0], mine % 8, mine < 8 ? to_b : to_c);
                } else {
#pragma unroll
                    for (int i = 0; i < N16; ++i) {
                        leave(sum_b[i], 16 * i + mine, to_b);
                        leave(sum_c[i], 16 * i + mine, to_c);
                    }
                }
            }
        } else if (initial) {  // its final state is its initial one
            for (int k = 0; k < nk; ++k)
#pragma unroll
                for (int i = 0; i < F; ++i) {
                    const int f = threadIdx.x + i * 64 * NW - 64 * S;
                    long long at;
                    if (f >= 0 && f < 64 * S && state_at(f, k, &at)) initial[at] = carry[k].x[f];
                }
        }
        const auto* const out = fresh<BackwardArgs>();
        const int clear = out->a.clear;
        if (clear && seq == n_seq - 1)
            for (int k = 0; k < nk; ++k) {
                const Place p = place_of(share, group, k0 + k);
                if (!p.in) continue;
                for (int t = end + 4 * w + j; t < out->a.q.n_tokens; t += 4 * NW) {
                    const long long to = (long long)t * channels + p.ch;
                    if (clear & SELECTIVE_SCAN_CLEAR_GRAD_X) ((E*)out->g.x)[to] = TY::store(0.0f);
                    if (clear & SELECTIVE_SCAN_CLEAR_GRAD_DT) ((E*)out->g.dt)[to] = TY::store(0.0f);
                    if (gated && (clear & SELECTIVE_SCAN_CLEAR_GRAD_Z)) ((E*)out->g.z)[to] = TY::store(0.0f);
                }
            }
    }
    // the waves' sums together, a wave for each sixteen channels
    __syncthreads();
    const auto* const out = fresh<BackwardArgs>();
    for (int k = w; k < nk; k += NW) {
        const Place p = place_of(share, group, k0 + k);
        if (!p.in) continue;
#pragma unroll
        for (int s = 0; s <= S; ++s) {
            double v = total[k][0][s][lane];
#pragma unroll
            for (int i = 1; i < NW; ++i) v += total[k][i][s][lane];
            if (s < S) {
                if (n0 + s < state_size) out->g.part_a[((long long)part * channels + p.ch) * state_size + n0 + s] = (float)v;
            } else if (j < 2) {
                (j == 0 ? out->g.part_d : out->g.part_bias)[(long long)part * channels + p.ch] = (float)v;
            }
        }
    }
}

// What the workgroups left, summed (21 us of the 391, 68 MB): b's and c's gradients over the
// channels' workgroups, a's, d's and dt_bias's over the sequences' parts.  A thread has an
// element.
constexpr int kSumThreads = 256;
template <class TY>
__global__ __launch_bounds__(kSumThreads) void scan_sums_kernel(Scan a, Grads g, int in_group, int parts,
                                                                typename TY::S* __restrict__ gb,
                                                                typename TY::S* __restrict__ gc, float* __restrict__ ga,
                                                                float* __restrict__ gd, float* __restrict__ gbias) {
    long long i = (long long)blockIdx.x * kSumThreads + threadIdx.x;
    const long long row = (long long)a.groups * a.state;
    if (i < 2 * g.rows) {
        const bool is_c = i >= g.rows;
        if (is_c) i -= g.rows;
        const float* from = is_c ? g.part_c : g.part_b;
        typename TY::S* to = is_c ? gc : gb;
        const int last = a.q.offsets ? min(max(a.q.offsets[a.q.n_seq], 0), a.q.n_tokens) : a.q.n_tokens;
        if (i / row >= last) {
            if (a.clear & (is_c ? SELECTIVE_SCAN_CLEAR_GRAD_C : SELECTIVE_SCAN_CLEAR_GRAD_B)) to[i] = TY::store(0.0f);
            return;
        }
        double v = 0.0;
        for (int k = 0; k < in_group; ++k) v += from[k * g.rows + i];
        to[i] = TY::store((float)v);
        return;
    }
    i -= 2 * g.rows;
    const long long na = (long long)a.channels * a.state;
    const float* from;
    float* to;
    long long n;
    if (i < na) {
        from = g.part_a, to = ga, n = na;
    } else if (i < na + 2LL * a.channels) {
        i -= na;
        const bool second = i >= a.channels;
        if (second) i -= a.channels;
        from = second ? g.part_bias : g.part_d, to = second ? gbias : gd, n = a.channels;
    } else {
        return;
    }
    if (!to) return;
    double v = 0.0;
    for (int k = 0; k < parts; ++k) v += from[k * n + i];
    to[i] = (float)v;
}

// ----------------------------------------------------------------------- step
// A lane's S states of a row, j of its channel's four: V neighbours at 4 V i + V j, so that
// the four read and write whole pieces of a cache line.  At any address; zero behind `state`.
template <class TY, int S, bool PAST>
__device__ __forceinline__ void load_row(const typename TY::S* row, int j, int state, float (&h)[S]) {
    using E = typename TY::S;
    constexpr int V = S < 4 ? S : 4;
    typedef E vec __attribute__((ext_vector_type(V), aligned(sizeof(E))));
#pragma unroll
    for (int i = 0; i < S / V; ++i) {
        const int n = (4 * i + j) * V;
        if (n + V <= state) {
            const vec* p = reinterpret_cast<const vec*>(row + n);
            const vec v = PAST ? __builtin_nontemporal_load(p) : *p;
#pragma unroll
            for (int k = 0; k < V; ++k) h[i * V + k] = TY::load(v[k]);
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) h[i * V + k] = n + k < state ? TY::load(row[n + k]) : 0.0f;
        }
    }
}
template <int S, bool PAST>
__device__ __forceinline__ void store_row(float* row, int j, int state, const float (&h)[S]) {
    constexpr int V = S < 4 ? S : 4;
    typedef float vec __attribute__((ext_vector_type(V), aligned(4)));
#pragma unroll
    for (int i = 0; i < S / V; ++i) {
        const int n = (4 * i + j) * V;
        if (n + V <= state) {
            vec v;
#pragma unroll
            for (int k = 0; k < V; ++k) v[k] = h[i * V + k];
            vec* p = reinterpret_cast<vec*>(row + n);
            if constexpr (PAST)
                __builtin_nontemporal_store(v, p);
            else
                *p = v;
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (n + k < state) row[n + k] = h[i * V + k];
        }
    }
}

// A wave has C times 16 channels of a row, their states in registers, all loads in flight at
// once.  The steps and the gates are computed by a lane for each channel and taken from there
// by the channel's four.  Bound by reading and writing the states: 243 rows of 4096 channels x
// 16 states (136 MB) in 33.5 us, 4.1 TB/s; one row in 4.3, latency.
constexpr int kStepThreads = 256;
// States of 32 MB a call and more pass the last-level cache by, since between two steps of a
// layer all the others' states pass through it (16 states of 4096 channels in bf16, us, with |
// without: 16 layers of 34 MB 19 | 23, 8 of 67 MB 35 | 41, 16 of 67 MB in 64 states 39 | 43; two
// of 67 MB, which it would hold, 35 | 33).
constexpr long long kPastCache = 32LL << 20;
// Times 16 channels from which on a wave has C of them instead of one (4096 channels, on the
// GPU alone, us, one | C = 4): one row 4.3 | 4.8, 16 rows 6.0 | 6.0, 32 rows 8.8 | 7.1, 64 rows
// 13.7 | 9.4, 256 rows 44 | 33.5.
constexpr long long kStepFew = 4096;
template <class TY, int S, int C, bool PAST>
__global__ __launch_bounds__(kStepThreads) void scan_step_kernel(
    Scan a, long long waves, int parts, const typename TY::S* __restrict__ x, const typename TY::S* __restrict__ dt,
    const float* __restrict__ decay, const typename TY::S* __restrict__ b, const typename TY::S* __restrict__ c,
    const float* __restrict__ d, const typename TY::S* __restrict__ z, const float* __restrict__ dt_bias, float* states,
    int pool, const int* __restrict__ slots, typename TY::S* __restrict__ y) {
    const long long index = on_die(blockIdx.x, (waves + kStepThreads / 64 - 1) / (kStepThreads / 64));
    const long long wave = index * (kStepThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (wave >= waves) return;
    const int part = (int)(wave % parts), group = (int)(wave / parts % a.groups), rows = a.q.n_tokens;
    const int lane = threadIdx.x & 63, quad = lane >> 2, four = lane & 3;
    int row = (int)(wave / parts / a.groups), slot = row;
    // the lane's channel, of those of the group
    const int ch = part * (C * kGroupCh) + lane;
    const bool own = lane < C * kGroupCh && ch < a.share;
    const int at = group * a.share + min(ch, a.share - 1);
    if (slots) {
        slot = __builtin_amdgcn_readfirstlane(slots[row]);
        if (slot < 0 || slot >= pool) {
            if (own) y[(long long)row * a.channels + at] = TY::store(0.0f);
            return;
        }
    }
    float h[C][S], a2[C][S];
    auto state_of = [&](int i, bool* in) {
        const int k = part * (C * kGroupCh) + i * kGroupCh + quad;
        *in = k < a.share;
        return group * a.share + min(k, a.share - 1);
    };
#pragma unroll
    for (int i = 0; i < C; ++i) {
        bool in;
        const int k = state_of(i, &in);
        load_row<F32, S, PAST>(states + ((long long)slot * a.channels + k) * a.state, four, a.state, h[i]);
        load_row<F32, S, false>(decay + (long long)k * a.state, four, a.state, a2[i]);
    }
    const float skip = d ? d[at] : 0.0f, bias = dt_bias ? dt_bias[at] : 0.0f;
    b += group * a.bg;
    c += group * a.cg;
    struct Row {
        float x, dt, z, b[S], c[S];
    };
    auto fetch = [&](Row& r) {
        r.x = TY::load(x[row * a.xt + at]);
        r.dt = TY::load(dt[row * a.dtt + at]);
        r.z = z ? TY::load(z[row * a.zt + at]) : 0.0f;
        load_row<TY, S, false>(b + row * a.bt, four, a.state, r.b);
        load_row<TY, S, false>(c + row * a.ct, four, a.state, r.c);
    };
    Row r;
    fetch(r);
    if (slots && row_of_slot(slots, slot, 0, row) < row) return;  // the first row of a slot takes all
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
        for (int s = 0; s < S; ++s) a2[i][s] *= kLog2e;
    while (true) {
        const float pre = r.dt + bias, step = a.softplus ? softplus_of(pre) : pre, u = step * r.x;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const float dl = __shfl(step, i * kGroupCh + quad), ul = __shfl(u, i * kGroupCh + quad);
            float v = 0.0f;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                h[i][s] = fmaf(exp2_of(dl * a2[i][s]), h[i][s], ul * r.b[s]);
                v = fmaf(r.c[s], h[i][s], v);
            }
            v += quad_perm<0xB1>(v);
            v += quad_perm<0x4E>(v);
            const float mine = __shfl(v, 4 * (lane & 15));
            if (lane >> 4 == i) sum = mine;
        }
        float out = fmaf(skip, r.x, sum);
        if (z) out *= r.z * gate_of<TY>(r.z);
        if (own) y[(long long)row * a.channels + at] = TY::store(out);
        if (!slots) break;
        row = row_of_slot(slots, slot, row + 1, rows);
        if (row >= rows) break;
        fetch(r);
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
        bool in;
        const int k = state_of(i, &in);
        if (in) store_row<S, PAST>(states + ((long long)slot * a.channels + k) * a.state, four, a.state, h[i]);
    }
}

// ---------------------------------------------------------- host helpers
constexpr long long kMaxTokens = (1LL << 31) - (1LL << 16);
constexpr long long kMaxBlocks = (1LL << 32) / 512 - 8;  // a grid has fewer than 2^32 work-items

// Whether blocks of so many rows of every argument and output are less than 2^31 bytes.
bool reaches(const selective_scan_shape_t* p, const Scan& a, int rows) {
    long long far = p->channels;
    if (!a.single)
        for (const long long stride : {p->x_stride, p->dt_stride, p->z_stride, p->grad_y_stride, p->b_stride_t, p->c_stride_t})
            far = std::max(far, stride);
    return far <= INT_MAX / (rows * size_of(p->type)) - (long long)p->channels - p->state;
}

int check_shape(const selective_scan_shape_t* p, bool step, Scan* a) {
    if (!p) return CFC_ERR_NULL;
    if (p->type != CFC_TYPE_F32 && p->type != CFC_TYPE_BF16 && p->type != CFC_TYPE_F16) return CFC_ERR_UNSUPPORTED;
    if (p->channels < 1 || p->groups < 1 || p->channels % p->groups || p->state < 1) return CFC_ERR_DIM;
    for (const long long stride : {p->x_stride, p->dt_stride, p->z_stride, p->grad_y_stride, p->b_stride_t,
                                   p->b_stride_g, p->c_stride_t, p->c_stride_g})
        if (stride < 0) return CFC_ERR_DIM;
    if (p->state > SELECTIVE_SCAN_MAX_STATE || p->n_tokens > kMaxTokens) return CFC_ERR_UNSUPPORTED;
    if (step) {
        if (p->n_tokens < 0) return CFC_ERR_DIM;
        a->q = Sequences{nullptr, (int)p->n_tokens, 1, (int)p->n_tokens};
    } else if (const int e = check_sequences(p->offsets, p->n_seq, p->seq_len, p->n_tokens, &a->q)) {
        return e;
    }
    a->channels = p->channels;
    a->groups = p->groups;
    a->share = p->channels / p->groups;
    a->state = p->state;
    a->softplus = p->softplus;
    a->clear = p->offsets ? p->clear_rest : 0;
    a->xt = p->x_stride, a->dtt = p->dt_stride, a->zt = p->z_stride, a->gt = p->grad_y_stride;
    a->bt = p->b_stride_t, a->bg = p->b_stride_g, a->ct = p->c_stride_t, a->cg = p->c_stride_g;
    a->single = (p->offsets ? p->n_tokens : step ? 1 : p->seq_len) <= 1;
    a->overlap = a->single || p->b_stride_t < p->state || p->c_stride_t < p->state;
    if (!reaches(p, *a, kBlockRows)) return CFC_ERR_UNSUPPORTED;
    const long long groups = (long long)a->groups * ((a->share + kGroupCh - 1) / kGroupCh);
    return groups * std::max(1, a->q.n_seq) > kMaxBlocks ? CFC_ERR_UNSUPPORTED : CFC_OK;
}
inline int sixteens_of(const Scan& a) { return (a.share + kGroupCh - 1) / kGroupCh; }

struct Sizes {  // bytes of the arguments
    long long x, dt, z, gy, b, c, rows, shared, a, d, states;
};
bool sizes_of(const selective_scan_shape_t* p, const Scan& a, Sizes* z) {
    const int size = size_of(p->type);
    const long long t = p->n_tokens;
    long long each;
    z->a = (long long)a.channels * a.state * 4;
    z->d = (long long)a.channels * 4;
    return extent(t, 1, a.channels, a.xt, 0, size, &z->x) && extent(t, 1, a.channels, a.dtt, 0, size, &z->dt) &&
           extent(t, 1, a.channels, a.zt, 0, size, &z->z) && extent(t, 1, a.channels, a.gt, 0, size, &z->gy) &&
           extent(t, a.groups, a.state, a.bt, a.bg, size, &z->b) && extent(t, a.groups, a.state, a.ct, a.cg, size, &z->c) &&
           mul_ok(t, (long long)a.channels * size, &z->rows) && mul_ok((long long)a.groups * a.state, size, &each) &&
           mul_ok(t, each, &z->shared) && mul_ok(a.q.n_seq, z->a, &z->states);
}

// Calls f with the type and the states of a lane, a power of two that four lanes hold `state` in.
template <class F>
int with_state(int type, int state, F f) {
    auto go = [&](auto ty) {
        if (state <= 4) return f(ty, std::integral_constant<int, 1>{});
        if (state <= 8) return f(ty, std::integral_constant<int, 2>{});
        if (state <= 16) return f(ty, std::integral_constant<int, 4>{});
        if (state <= 32) return f(ty, std::integral_constant<int, 8>{});
        return f(ty, std::integral_constant<int, 16>{});
    };
    if (type == CFC_TYPE_F32) return go(F32{});
    return type == CFC_TYPE_BF16 ? go(BF16{}) : go(F16{});
}
inline int lane_states(int state) { return state <= 4 ? 1 : state <= 8 ? 2 : state <= 16 ? 4 : state <= 32 ? 8 : 16; }

// How many times 16 channels a workgroup of the backward has: more of them leave fewer partial
// sums of b's and c's gradients, as long as all CUs have one (4 x 2048 tokens, bf16, us, with one,
// 2 and 4: 2048 channels 440, 391; 4096 channels 880, 779, 746).  Beyond 16 states LDS holds one.
inline int sixteens_at_once(const Scan& a) {
    if (a.state > 16) return 1;
    const long long all = (long long)a.groups * sixteens_of(a) * a.q.n_seq;
    return all >= 4 * 256 ? 4 : all >= 2 * 256 ? 2 : 1;
}
inline int wg_groups_of(const Scan& a) {
    const int k = sixteens_at_once(a);
    return a.groups * ((sixteens_of(a) + k - 1) / k);
}
// The sequences go to as many workgroups of the same channels as fill the chip, since each
// leaves a row of partial sums.
inline int parts_of(const Scan& a) {
    return std::min(a.q.n_seq, std::max(1, 1024 / wg_groups_of(a)));
}

// Bytes of the backward's workspace, laid out from `base` on.
long long lay_out(const Scan& a, void* base, Grads* g) {
    const int s = lane_states(a.state);
    const long long slots = a.q.n_tokens / block_of(s) + a.q.n_seq;
    const long long in_group = wg_groups_of(a) / a.groups, parts = parts_of(a);
    long long kept, bc, pa, all = 0;
    g->rows = (long long)a.q.n_tokens * a.groups * a.state;
    if (!mul_ok(slots * a.groups, (long long)sixteens_of(a) * (64 * s * 4), &kept) || !mul_ok(g->rows, in_group * 4, &bc) ||
        !mul_ok(parts, (long long)a.channels * a.state * 4, &pa) ||
        2 * g->rows + (long long)a.channels * (a.state + 2) > kMaxBlocks * 256)
        return -1;
    auto take = [&](long long bytes) {
        float* at = reinterpret_cast<float*>(reinterpret_cast<uintptr_t>(base) + all);
        all += (bytes + 15) / 16 * 16;
        return at;
    };
    g->kept = take(kept);
    g->part_b = take(bc);
    g->part_c = take(bc);
    g->part_a = take(pa);
    g->part_d = take(parts * a.channels * 4);
    g->part_bias = take(parts * a.channels * 4);
    return all;
}

}  // namespace

// ================================================================ C ABI
extern "C" int selective_scan_forward(const selective_scan_shape_t* shape, const void* x, const void* dt, const float* a_,
                                      const void* b, const void* c, const float* d, const void* z, const float* dt_bias,
                                      const float* initial_state, void* y, float* final_state, hipStream_t stream) {
    Scan a;
    Sizes n;
    if (const int e = check_shape(shape, false, &a)) return e;
    if (!sizes_of(shape, a, &n)) return CFC_ERR_DIM;
    if (a.q.n_seq == 0) return CFC_OK;
    if (!a_ || (a.q.n_tokens && (!x || !dt || !b || !c || !y))) return CFC_ERR_NULL;
    if (!fits({x, dt, b, c, z, y}, size_of(shape->type)) || !fits({a_, d, dt_bias, initial_state, final_state}, 4))
        return CFC_ERR_DIM;
    const Range ini = bytes_of(initial_state, n.states), fin = bytes_of(final_state, n.states);
    const Range outs[] = {bytes_of(y, n.rows), fin};
    const Range ins[] = {bytes_of(x, n.x), bytes_of(dt, n.dt), bytes_of(a_, n.a), bytes_of(b, n.b), bytes_of(c, n.c),
                         bytes_of(d, n.d), bytes_of(z, n.z), bytes_of(dt_bias, n.d), offsets_range(a.q),
                         same(ini, fin) ? Range{0, 0} : ini};
    if (!outputs_disjoint(outs, 2, ins, 10) || overlap(outs[0], ini)) return CFC_ERR_OVERLAP;
    return with_state(shape->type, a.state, [&](auto ty, auto states) {
        using TY = decltype(ty);
        using E = typename TY::S;
        constexpr int S = decltype(states)::value;
        const int sixteens = sixteens_of(a);
        const long long count = (long long)a.groups * sixteens * a.q.n_seq;
        auto go = [&](auto kernel, int waves) {
            hipLaunchKernelGGL(kernel, dim3(dealt(count)), dim3(64 * waves), 0, stream, a, sixteens, (const E*)x,
                               (const E*)dt, a_, (const E*)b, (const E*)c, d, (const E*)z, dt_bias, initial_state, (E*)y,
                               final_state);
        };
        if constexpr (S <= 8) {
            if (count <= kFewWorkgroups && !a.overlap && reaches(shape, a, forward_block(S, 16))) {
                go(scan_kernel<TY, S, 16>, 16);
                return launch_status();
            }
        }
        go(scan_kernel<TY, S, 8>, 8);
        return launch_status();
    });
}

extern "C" long long selective_scan_backward_workspace(const selective_scan_shape_t* shape) {
    Scan a;
    Grads g;
    return check_shape(shape, false, &a) == CFC_OK ? lay_out(a, nullptr, &g) : -1;
}

extern "C" int selective_scan_backward(const selective_scan_shape_t* shape, const void* x, const void* dt,
                                       const float* a_, const void* b, const void* c, const float* d, const void* z,
                                       const float* dt_bias, const float* initial_state, const void* grad_y,
                                       const float* grad_final_state, void* grad_x, void* grad_dt, float* grad_a,
                                       void* grad_b, void* grad_c, float* grad_d, void* grad_z, float* grad_dt_bias,
                                       float* grad_initial_state, void* workspace, long long workspace_bytes,
                                       hipStream_t stream) {
    Scan a;
    Sizes n;
    Grads g;
    if (const int e = check_shape(shape, false, &a)) return e;
    const long long need = lay_out(a, workspace, &g);
    if (!sizes_of(shape, a, &n) || need < 0) return CFC_ERR_DIM;
    if (!a_ || !grad_a || (need && !workspace) ||
        (a.q.n_tokens && (!x || !dt || !b || !c || !grad_y || !grad_x || !grad_dt || !grad_b || !grad_c || (z && !grad_z))))
        return CFC_ERR_NULL;
    if (need && (workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 16)) return CFC_ERR_DIM;
    if (!z && grad_z) return CFC_ERR_DIM;
    if (!fits({x, dt, b, c, z, grad_y, grad_x, grad_dt, grad_b, grad_c, grad_z}, size_of(shape->type)) ||
        !fits({a_, d, dt_bias, initial_state, grad_final_state, grad_a, grad_d, grad_dt_bias, grad_initial_state}, 4))
        return CFC_ERR_DIM;
    const Range gin = bytes_of(grad_initial_state, n.states), gfin = bytes_of(grad_final_state, n.states);
    const Range outs[] = {bytes_of(grad_x, n.rows), bytes_of(grad_dt, n.rows), bytes_of(grad_a, n.a),
                          bytes_of(grad_b, n.shared), bytes_of(grad_c, n.shared), bytes_of(grad_d, n.d),
                          bytes_of(grad_z, n.rows), bytes_of(grad_dt_bias, n.d), gin, bytes_of(need ? workspace : nullptr, need)};
    const Range ins[] = {bytes_of(x, n.x), bytes_of(dt, n.dt), bytes_of(a_, n.a), bytes_of(b, n.b), bytes_of(c, n.c),
                         bytes_of(d, n.d), bytes_of(z, n.z), bytes_of(dt_bias, n.d), bytes_of(initial_state, n.states),
                         bytes_of(grad_y, n.gy), offsets_range(a.q), same(gin, gfin) ? Range{0, 0} : gfin};
    if (!outputs_disjoint(outs, 10, ins, 12)) return CFC_ERR_OVERLAP;
    for (int i = 0; same(gin, gfin) && i < 10; ++i)
        if (i != 8 && overlap(outs[i], gfin)) return CFC_ERR_OVERLAP;
    g.x = grad_x, g.dt = grad_dt, g.z = grad_z, g.initial = grad_initial_state;
    return with_state(shape->type, a.state, [&](auto ty, auto states) {
        using TY = decltype(ty);
        using E = typename TY::S;
        constexpr int S = decltype(states)::value;
        const int sixteens = sixteens_of(a), wg_groups = wg_groups_of(a), parts = parts_of(a);
        if (a.q.n_seq) {
            const long long count = (long long)a.groups * sixteens * a.q.n_seq;
            auto states_of = [&](auto kernel, int waves) {
                hipLaunchKernelGGL(kernel, dim3(dealt(count)), dim3(64 * waves), 0, stream, a, sixteens, (const E*)x,
                                   (const E*)dt, a_, (const E*)b, dt_bias, initial_state, g.kept);
            };
            if constexpr (S <= 4) {
                if (count <= kFewWorkgroups && !a.overlap)
                    states_of(scan_states_kernel<TY, S, 16>, 16);
                else
                    states_of(scan_states_kernel<TY, S, 8>, 8);
            } else {
                states_of(scan_states_kernel<TY, S, waves_of(S)>, waves_of(S));
            }
            const BackwardArgs args{a, sixteens, wg_groups, parts, x, dt, b, c, z, grad_y, a_, d, dt_bias, grad_final_state, g};
            auto go = [&](auto kernel) {
                hipLaunchKernelGGL(kernel, dim3(dealt((long long)wg_groups * parts)), dim3(64 * waves_of(S)), 0, stream, args);
            };
            const int at_once = sixteens_at_once(a);
            if constexpr (S <= 4) {
                if (at_once == 4)
                    go(scan_backward_kernel<TY, S, 4>);
                else if (at_once == 2)
                    go(scan_backward_kernel<TY, S, 2>);
                else
                    go(scan_backward_kernel<TY, S, 1>);
            } else {
                go(scan_backward_kernel<TY, S, 1>);
            }
        }
        const long long elements = 2 * g.rows + (long long)a.channels * (a.state + 2);
        hipLaunchKernelGGL((scan_sums_kernel<TY>), dim3((unsigned)((elements + kSumThreads - 1) / kSumThreads)),
                           dim3(kSumThreads), 0, stream, a, g, wg_groups / a.groups, parts, (E*)grad_b, (E*)grad_c, grad_a,
                           grad_d, grad_dt_bias);
        return launch_status();
    });
}

extern "C" int selective_scan_step(const selective_scan_shape_t* shape, const void* x, const void* dt, const float* a_,
                                   const void* b, const void* c, const float* d, const void* z, const float* dt_bias,
                                   float* states, int pool, const int* slots, void* y, hipStream_t stream) {
    Scan a;
    Sizes n;
    long long held;
    if (const int e = check_shape(shape, true, &a)) return e;
    if (pool < 0 || (!slots && pool < a.q.n_tokens) || !sizes_of(shape, a, &n) || !mul_ok(pool, n.a, &held))
        return CFC_ERR_DIM;
    if (a.q.n_tokens == 0) return CFC_OK;
    if (!x || !dt || !a_ || !b || !c || !y || (pool && !states)) return CFC_ERR_NULL;
    if (!fits({x, dt, b, c, z, y}, size_of(shape->type)) || !fits({a_, d, dt_bias, states, slots}, 4)) return CFC_ERR_DIM;
    const Range outs[] = {bytes_of(y, n.rows), bytes_of(states, held)};
    const Range ins[] = {bytes_of(x, n.x), bytes_of(dt, n.dt), bytes_of(a_, n.a), bytes_of(b, n.b), bytes_of(c, n.c),
                         bytes_of(d, n.d), bytes_of(z, n.z), bytes_of(dt_bias, n.d),
                         bytes_of(slots, (long long)a.q.n_tokens * 4)};
    if (!outputs_disjoint(outs, 2, ins, 9)) return CFC_ERR_OVERLAP;
    return with_state(shape->type, a.state, [&](auto ty, auto s) {
        using TY = decltype(ty);
        using E = typename TY::S;
        constexpr int S = decltype(s)::value;
        constexpr int per = kStepThreads / 64, C = S <= 4 ? 4 : S == 8 ? 2 : 1;
        auto go = [&](auto kernel, int at_once) {
            const int parts = (sixteens_of(a) + at_once - 1) / at_once;
            const long long waves = (long long)a.groups * parts * a.q.n_tokens;
            hipLaunchKernelGGL(kernel, dim3(dealt((waves + per - 1) / per)), dim3(kStepThreads), 0, stream, a, waves, parts,
                               (const E*)x, (const E*)dt, a_, (const E*)b, (const E*)c, d, (const E*)z, dt_bias, states,
                               pool, slots, (E*)y);
        };
        const bool past = (long long)a.q.n_tokens * n.a >= kPastCache;
        if ((long long)a.groups * sixteens_of(a) * a.q.n_tokens < kStepFew)
            go(scan_step_kernel<TY, S, 1, false>, 1);
        else if (past)
            go(scan_step_kernel<TY, S, C, true>, C);
        else
            go(scan_step_kernel<TY, S, C, false>, C);
        return launch_status();
    });
}
