// short_conv.hip -- gfx950 kernels and C ABI of the short causal convolution (see
// include/short_conv.h).
//
// Memory is the bound: each input is read once and each output written once, so a wave
// has a tile of tokens and 4 channels a lane, four to eight rows' loads in flight at once,
// and the last width - 1 inputs in registers as it goes from token to token.  Rows that a
// tile shares with the one before are read twice, mostly from the cache.  16 packed prompts,
// 5969 tokens of 8192 channels in bf16 (197 MB): 46 us, 4.3 TB/s (a call whose inputs all come
// from memory 51, one whose inputs the last-level cache holds 44); the gradients of 4 x 2048
// tokens x 4096 channels (201 MB) 64 us and 6 for the sums of the weight's (74 and 56); a step of
// one row 2.8, latency.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "columns.h"
#include "elements.h"
#include "functions.h"
#include "sequences.h"
#include "short_conv.h"

namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kTile = 16;  // tokens of a wave, forward
constexpr int kAhead = 4;  // rows that are loaded at once, while as many are worked on
// Channels of a lane, 8 bytes of a 16-bit type.  Eight of them take twice the registers, so
// half the waves: the forward of 16 packed prompts of 8192 channels 55 us instead of 45, the
// gradients of 4 x 2048 x 4096 75 instead of 70.
constexpr int kLane = 4;

struct Conv {
    Sequences q;
    int channels, silu, clear;
    int grad_tile;  // tokens of a wave, backward: a row of partial sums each
    long long xt, gt;
};
inline __host__ __device__ int parts_of(const Conv& a) { return (a.channels + 64 * kLane - 1) / (64 * kLane); }

// The channels' weights as w[tap][channel], zero behind the last channel.
template <class TY, int W, int V, bool TAIL>
__device__ __forceinline__ void load_weights(const typename TY::S* weight, int c, int channels, float (&w)[W][V]) {
    float f[W][V];
#pragma unroll
    for (int i = 0; i < W; ++i) load<TY, V, TAIL>(weight, c * W + V * i, channels * W, f[i]);
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) w[j][e] = f[(e * W + j) / V][(e * W + j) % V];
}
template <class TY, int V, bool TAIL>
__device__ __forceinline__ void load_or_zero(const typename TY::S* row, int c, int channels, float (&x)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = 0.0f;
    if (row) load<TY, V, TAIL>(row, c, channels, x);
}

// The width - 1 inputs before row t of the sequence s that begins at `first`: its own rows,
// or its initial state's.
template <class TY, int W, int V, bool TAIL>
__device__ __forceinline__ void load_window(const Conv& a, const typename TY::S* x, const typename TY::S* initial, int s,
                                            int first, int t, int c, float (&win)[W - 1][V]) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int row = t - (W - 1) + j;
        const typename TY::S* from = nullptr;
        if (row >= first)
            from = x + row * a.xt;
        else if (initial)
            from = initial + ((long long)s * (W - 1) + min(max(row - first + W - 1, 0), W - 2)) * a.channels;
        load_or_zero<TY, V, TAIL>(from, c, a.channels, win[j]);
    }
}

// p of the next token, whose input is `now`.
template <int W, int V>
__device__ __forceinline__ void apply(const float (&w)[W][V], const float (&b)[V], const float (&win)[W - 1][V],
                                      const float (&now)[V], float (&p)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
        p[e] = b[e];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) p[e] += w[j][e] * win[j][e];
        p[e] += w[W - 1][e] * now[e];
    }
}
template <int W, int V>
__device__ __forceinline__ void shift(float (&win)[W - 1][V], const float (&now)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j) win[j][e] = win[j + 1][e];
        win[W - 2][e] = now[e];
    }
}

// Waves `begin` ... of the tiles' waves and, behind them, of the final states', a sequence
// and 256 channels each.
template <class TY, int W, bool TAIL>
__global__ __launch_bounds__(kThreads) void conv_kernel(Conv a, long long begin, long long end_wave, long long tiles,
                                                        const typename TY::S* __restrict__ x,
                                                        const typename TY::S* __restrict__ weight,
                                                        const typename TY::S* __restrict__ bias,
                                                        const typename TY::S* initial, typename TY::S* __restrict__ y,
                                                        typename TY::S* final) {
    constexpr int V = kLane;
    const long long block = on_die(blockIdx.x, (end_wave - begin + kWaves - 1) / kWaves);
    const long long wave = begin + block * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (wave >= end_wave) return;
    const int parts = parts_of(a);
    const int c = (int)(wave % parts) * 64 * V + (threadIdx.x & 63) * V;
    const long long at = wave / parts;
    int first, end;
    if (at >= tiles) {
        const int s = (int)(at - tiles);
        span_of(a.q, s, first, end);
        float win[W - 1][V];
        load_window<TY, W, V, TAIL>(a, x, initial, s, first, end, c, win);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            store<TY, V, TAIL>(final + ((long long)s * (W - 1) + j) * a.channels, c, a.channels, win[j]);
        return;
    }
    const int t0 = (int)at * kTile, n = min(kTile, a.q.n_tokens - t0);
    int s = sequence_of(a.q, t0);
    span_of(a.q, s, first, end);
    Packed<TY, V> rows[2][kAhead];
    auto ahead = [&](Packed<TY, V>(&to)[kAhead], int i0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (i0 + i < n) to[i] = fetch<TY, V, TAIL>(x + (t0 + i0 + i) * a.xt, c, a.channels);
    };
    ahead(rows[0], 0);
    ahead(rows[1], kAhead);
    float w[W][V], b[V], win[W - 1][V];
    load_weights<TY, W, V, TAIL>(weight, c, a.channels, w);
    load_or_zero<TY, V, TAIL>(bias, c, a.channels, b);
    bool live = t0 >= first && t0 < end;  // or behind the last sequence
    if (live) load_window<TY, W, V, TAIL>(a, x, initial, s, first, t0, c, win);
    auto some = [&](Packed<TY, V>(&from)[kAhead], int i0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int t = t0 + i0 + i;
            if (live && t >= end) {
                s = sequence_of(a.q, t);
                span_of(a.q, s, first, end);
                live = t >= first && t < end;
                if (live) load_window<TY, W, V, TAIL>(a, x, initial, s, first, t, c, win);
            }
            if (i0 + i < n && live) {
                float now[V], p[V];
                unpack<TY, V, TAIL>(from[i], c, a.channels, now);
                apply<W, V>(w, b, win, now, p);
                shift<W, V>(win, now);
                if (a.silu) {
#pragma unroll
                    for (int e = 0; e < V; ++e) p[e] *= gate_of<TY>(p[e]);
                }
                store<TY, V, TAIL>(y + (long long)t * a.channels, c, a.channels, p);
            } else if (i0 + i < n && a.clear) {
                const float none[V] = {};
                store<TY, V, TAIL>(y + (long long)t * a.channels, c, a.channels, none);
            }
        }
    };
    for (int i = 0; i < kTile; i += 2 * kAhead) {
        some(rows[0], i);
        ahead(rows[0], i + 2 * kAhead);
        some(rows[1], i + kAhead);
        ahead(rows[1], i + 3 * kAhead);
    }
}

// grad_p = grad_y * y'(p)
template <class TY, int V>
__device__ __forceinline__ void through(int silu, const float (&p)[V], float (&g)[V]) {
    if (!silu) return;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const float sig = gate_of<TY>(p[e]);
        g[e] *= sig * (1.0f + p[e] * (1.0f - sig));
    }
}

// A wave has a.grad_tile tokens and 256 channels.  It computes p again for its own tokens
// and, since grad_x_t takes grad_p of the width - 1 tokens behind t, for as many behind
// them; `next` holds what the tokens up to now give to the gradients of the last width - 1
// inputs.  Behind the tiles' waves the initial states', a sequence each.
template <class TY, int W, bool TAIL>
__global__ __launch_bounds__(kThreads) void conv_backward_kernel(
    Conv a, long long waves, long long tiles, const typename TY::S* __restrict__ x,
    const typename TY::S* __restrict__ weight, const typename TY::S* __restrict__ bias,
    const typename TY::S* __restrict__ initial, const typename TY::S* __restrict__ gy,
    const typename TY::S* __restrict__ gfinal, typename TY::S* __restrict__ gx, typename TY::S* __restrict__ ginit,
    float* __restrict__ part) {
    constexpr int V = kLane;
    const long long block = on_die(blockIdx.x, (waves + kWaves - 1) / kWaves);
    const long long wave = block * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (wave >= waves) return;
    const int parts = parts_of(a);
    const int c = (int)(wave % parts) * 64 * V + (threadIdx.x & 63) * V;
    const long long at = wave / parts;
    float w[W][V], b[V], win[W - 1][V];
    auto final_row = [&](int s, int row) {
        return gfinal ? gfinal + ((long long)s * (W - 1) + row) * a.channels : nullptr;
    };
    int first, end;
    if (at >= tiles) {
        load_weights<TY, W, V, TAIL>(weight, c, a.channels, w);
        load_or_zero<TY, V, TAIL>(bias, c, a.channels, b);
        const int s = (int)(at - tiles);
        span_of(a.q, s, first, end);
        load_window<TY, W, V, TAIL>(a, x, initial, s, first, first, c, win);
        float g0[W - 1][V] = {};
#pragma unroll
        for (int p = 0; p < W - 1; ++p) {
            if (first + p >= end) break;
            float now[V], pre[V], g[V];
            load<TY, V, TAIL>(x + (first + p) * a.xt, c, a.channels, now);
            load<TY, V, TAIL>(gy + (first + p) * a.gt, c, a.channels, g);
            apply<W, V>(w, b, win, now, pre);
            shift<W, V>(win, now);
            through<TY, V>(a.silu, pre, g);
            // kept input i is the tap i - p of place p
#pragma unroll
            for (int i = p; i < W - 1; ++i)
#pragma unroll
                for (int e = 0; e < V; ++e) g0[i][e] += w[i - p][e] * g[e];
        }
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            const int kept = i - (end - first);  // where it is in the final state
            if (kept >= 0) {
                float f[V];
                load_or_zero<TY, V, TAIL>(final_row(s, kept), c, a.channels, f);
#pragma unroll
                for (int e = 0; e < V; ++e) g0[i][e] += f[e];
            }
            store<TY, V, TAIL>(ginit + ((long long)s * (W - 1) + i) * a.channels, c, a.channels, g0[i]);
        }
        return;
    }
    const int t0 = (int)at * a.grad_tile, own = min(t0 + a.grad_tile, a.q.n_tokens);
    const int all = min(own + W - 1, a.q.n_tokens) - t0;  // rows that it reads
    int s = sequence_of(a.q, t0);
    span_of(a.q, s, first, end);
    Packed<TY, V> xr[2][kAhead], gr[2][kAhead];
    auto ahead = [&](int k, int i0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (i0 + i < all) {
                xr[k][i] = fetch<TY, V, TAIL>(x + (t0 + i0 + i) * a.xt, c, a.channels);
                gr[k][i] = fetch<TY, V, TAIL>(gy + (t0 + i0 + i) * a.gt, c, a.channels);
            }
    };
    ahead(0, 0);
    ahead(1, kAhead);
    load_weights<TY, W, V, TAIL>(weight, c, a.channels, w);
    load_or_zero<TY, V, TAIL>(bias, c, a.channels, b);
    bool live = t0 >= first && t0 < end;  // or behind the last sequence, or done
    if (live) load_window<TY, W, V, TAIL>(a, x, initial, s, first, t0, c, win);
    float next[W - 1][V] = {};  // next[k] of the input k tokens back
    float sum[W + 1][V] = {};
    // the gradients of a sequence's last inputs, which its final state holds too
    auto finish = [&] {
#pragma unroll
        for (int k = W - 2; k >= 0; --k) {
            const int done = end - 1 - k;
            if (done >= t0 && done >= first && done < own) {
                float f[V];
                load_or_zero<TY, V, TAIL>(final_row(s, W - 2 - k), c, a.channels, f);
#pragma unroll
                for (int e = 0; e < V; ++e) f[e] += next[k][e];
                store<TY, V, TAIL>(gx + (long long)done * a.channels, c, a.channels, f);
            }
        }
    };
    auto some = [&](int k, int i0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int t = t0 + i0 + i;
            if (live && t >= end) {
                finish();
                live = t < own;
                if (live) {
                    s = sequence_of(a.q, t);
                    span_of(a.q, s, first, end);
                    live = t >= first && t < end;
                }
                if (live) {
                    load_window<TY, W, V, TAIL>(a, x, initial, s, first, t, c, win);
#pragma unroll
                    for (int q = 0; q < W - 1; ++q)
#pragma unroll
                        for (int e = 0; e < V; ++e) next[q][e] = 0.0f;
                }
            }
            if (live && i0 + i < all) {
                float now[V], p[V], g[V];
                unpack<TY, V, TAIL>(xr[k][i], c, a.channels, now);
                unpack<TY, V, TAIL>(gr[k][i], c, a.channels, g);
                apply<W, V>(w, b, win, now, p);
                through<TY, V>(a.silu, p, g);
                if (t < own) {
#pragma unroll
                    for (int e = 0; e < V; ++e) {
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) sum[j][e] += g[e] * win[j][e];
                        sum[W - 1][e] += g[e] * now[e];
                        sum[W][e] += g[e];
                    }
                }
                shift<W, V>(win, now);
                // input t - k is the tap W - 1 - k of token t
                float done[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    done[e] = next[W - 2][e] + w[0][e] * g[e];
#pragma unroll
                    for (int q = W - 2; q > 0; --q) next[q][e] = next[q - 1][e] + w[W - 1 - q][e] * g[e];
                    next[0][e] = w[W - 1][e] * g[e];
                }
                const int which = t - (W - 1);
                if (which >= t0 && which >= first) store<TY, V, TAIL>(gx + (long long)which * a.channels, c, a.channels, done);
            } else if (a.clear && t < own && !live) {
                const float none[V] = {};
                store<TY, V, TAIL>(gx + (long long)t * a.channels, c, a.channels, none);
            }
        }
    };
    for (int i = 0; i < a.grad_tile + W - 1; i += 2 * kAhead) {
        some(0, i);
        ahead(0, i + 2 * kAhead);
        some(1, i + kAhead);
        ahead(1, i + 3 * kAhead);
    }
    if (live && end <= t0 + all) finish();
#pragma unroll
    for (int j = 0; j <= W; ++j) store<F32, V, TAIL>(part + (at * (W + 1) + j) * a.channels, c, a.channels, sum[j]);
}

// Where the sums over the tiles of [width + 1, channels] go: the last of the width + 1 into gb (or
// nowhere), the others into gw [channels, width].
struct Weights {
    float *gw, *gb;
    int channels, width;
    __device__ __forceinline__ void operator()(long long c, float x) const {
        const int j = (int)(c / channels);
        const long long ch = c % channels;
        if (j < width)
            gw[ch * width + j] = x;
        else if (gb)
            gb[ch] = x;
    }
};

template <class TY, int W, bool TAIL>
__global__ __launch_bounds__(kThreads) void conv_step_kernel(Conv a, long long waves, const typename TY::S* __restrict__ x,
                                                             const typename TY::S* __restrict__ weight,
                                                             const typename TY::S* __restrict__ bias,
                                                             typename TY::S* states, int pool,
                                                             const int* __restrict__ slots, typename TY::S* __restrict__ y) {
    const long long wave = (long long)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (wave >= waves) return;
    constexpr int V = kLane;
    const int parts = parts_of(a), lane = threadIdx.x & 63;
    const int c = (int)(wave % parts) * 64 * V + lane * V;
    const int rows = a.q.n_tokens;
    int row = (int)(wave / parts), slot = row;
    if (slots) {
        slot = __builtin_amdgcn_readfirstlane(slots[row]);
        if (slot < 0 || slot >= pool) {
            const float none[V] = {};
            store<TY, V, TAIL>(y + (long long)row * a.channels, c, a.channels, none);
            return;
        }
        if (row_of_slot(slots, slot, 0, row) < row) return;  // the first row of a slot takes all
    }
    float w[W][V], b[V], win[W - 1][V];
    load_weights<TY, W, V, TAIL>(weight, c, a.channels, w);
    load_or_zero<TY, V, TAIL>(bias, c, a.channels, b);
    typename TY::S* state = states + (long long)slot * (W - 1) * a.channels;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load<TY, V, TAIL>(state + (long long)j * a.channels, c, a.channels, win[j]);
    while (row < rows) {
        float now[V], p[V];
        load<TY, V, TAIL>(x + row * a.xt, c, a.channels, now);
        apply<W, V>(w, b, win, now, p);
        shift<W, V>(win, now);
        if (a.silu) {
#pragma unroll
            for (int e = 0; e < V; ++e) p[e] *= gate_of<TY>(p[e]);
        }
        store<TY, V, TAIL>(y + (long long)row * a.channels, c, a.channels, p);
        if (!slots) break;
        row = row_of_slot(slots, slot, row + 1, rows);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store<TY, V, TAIL>(state + (long long)j * a.channels, c, a.channels, win[j]);
}

// ---------------------------------------------------------- host helpers
constexpr long long kMaxTokens = (1LL << 31) - (1LL << 16);
constexpr long long kMaxGrid = (1LL << 32) / kThreads - 8;  // a grid has fewer than 2^32 work-items

inline long long blocks_of(long long waves) { return (waves + kWaves - 1) / kWaves; }

int check_shape(const short_conv_shape_t* p, bool step, Conv* a) {
    if (!p) return CFC_ERR_NULL;
    if (p->type != CFC_TYPE_F32 && p->type != CFC_TYPE_BF16 && p->type != CFC_TYPE_F16) return CFC_ERR_UNSUPPORTED;
    if (p->channels < 1 || p->width < 1 || p->x_stride < 0 || p->grad_y_stride < 0) return CFC_ERR_DIM;
    if (p->width < 2 || p->width > SHORT_CONV_MAX_WIDTH) return CFC_ERR_UNSUPPORTED;
    // a lane's first weight is at 4 times its channel
    if (p->channels > INT_MAX / SHORT_CONV_MAX_WIDTH - 64 * kLane || p->n_tokens > kMaxTokens) return CFC_ERR_UNSUPPORTED;
    if (step) {
        if (p->n_tokens < 0) return CFC_ERR_DIM;
        a->q = Sequences{nullptr, (int)p->n_tokens, 1, (int)p->n_tokens};
    } else if (const int e = check_sequences(p->offsets, p->n_seq, p->seq_len, p->n_tokens, &a->q)) {
        return e;
    }
    a->channels = p->channels;
    a->silu = p->silu;
    a->clear = p->clear_rest && p->offsets;
    a->xt = p->x_stride;
    a->gt = p->grad_y_stride;
    // 32 tokens a wave share their halo and their row of partial sums; with 16 twice as many
    // waves hide the loads' latency where there are few: 3056 tokens of 1111 channels in 27
    // instead of 42 us, but 8192 of 4096 in 78 instead of 70.
    a->grad_tile = ((long long)a->q.n_tokens / 32 + 1) * parts_of(*a) < 2048 ? 16 : 32;
    // (the forward's tiles are the most)
    const long long most = ((long long)a->q.n_tokens / (step ? 1 : kTile) + 1 + a->q.n_seq) * parts_of(*a);
    return blocks_of(most) > kMaxGrid ? CFC_ERR_UNSUPPORTED : CFC_OK;
}

struct Sizes {  // bytes of the arguments
    long long x, gy, y, weight, bias, states;
};
bool sizes_of(const short_conv_shape_t* p, const Conv& a, Sizes* z) {
    const int size = size_of(p->type);
    long long kept;
    z->weight = (long long)a.channels * p->width * size;
    z->bias = (long long)a.channels * size;
    return extent(p->n_tokens, 1, a.channels, a.xt, 0, size, &z->x) &&
           extent(p->n_tokens, 1, a.channels, a.gt, 0, size, &z->gy) && mul_ok(p->n_tokens, (long long)a.channels * size, &z->y) &&
           mul_ok(a.q.n_seq, p->width - 1, &kept) && mul_ok(kept, (long long)a.channels * size, &z->states);
}
inline long long workspace_of(const Conv& a, int width) {
    const long long tiles = ((long long)a.q.n_tokens + a.grad_tile - 1) / a.grad_tile;
    long long n;
    return mul_ok(tiles * (width + 1), (long long)a.channels * 4, &n) ? (n + 15) / 16 * 16 : -1;
}

template <class F>
int with_width(const short_conv_shape_t* p, F f) {
    auto typed = [&](auto ty, auto tail) {
        if (p->width == 2) return f(ty, std::integral_constant<int, 2>{}, tail);
        if (p->width == 3) return f(ty, std::integral_constant<int, 3>{}, tail);
        return f(ty, std::integral_constant<int, 4>{}, tail);
    };
    auto go = [&](auto ty) { return p->channels % kLane ? typed(ty, std::true_type{}) : typed(ty, std::false_type{}); };
    if (p->type == CFC_TYPE_F32) return go(F32{});
    return p->type == CFC_TYPE_BF16 ? go(BF16{}) : go(F16{});
}

}  // namespace

// ================================================================ C ABI
extern "C" int short_conv_forward(const short_conv_shape_t* shape, const void* x, const void* weight, const void* bias,
                                  const void* initial_state, void* y, void* final_state, hipStream_t stream) {
    Conv a;
    Sizes z;
    if (const int e = check_shape(shape, false, &a)) return e;
    if (!sizes_of(shape, a, &z)) return CFC_ERR_DIM;
    if (a.q.n_seq == 0) return CFC_OK;
    if (!weight || (a.q.n_tokens && (!x || !y))) return CFC_ERR_NULL;
    if (!fits({x, weight, bias, initial_state, y, final_state}, size_of(shape->type))) return CFC_ERR_DIM;
    const Range ini = bytes_of(initial_state, z.states), fin = bytes_of(final_state, z.states);
    const bool over = same(ini, fin);
    const Range outs[] = {bytes_of(y, z.y), fin};
    const Range ins[] = {bytes_of(x, z.x), bytes_of(weight, z.weight), bytes_of(bias, z.bias), offsets_range(a.q),
                         over ? Range{0, 0} : ini};
    if (!outputs_disjoint(outs, 2, ins, 5) || (over && overlap(outs[0], ini))) return CFC_ERR_OVERLAP;
    return with_width(shape, [&](auto ty, auto width, auto tail) {
        using TY = decltype(ty);
        using S = typename TY::S;
        constexpr int W = decltype(width)::value;
        constexpr bool TAIL = decltype(tail)::value;
        const long long tiles = (a.q.n_tokens + kTile - 1) / kTile, parts = parts_of(a);
        const long long split = tiles * parts, all = (tiles + (final_state ? a.q.n_seq : 0)) * parts;
        auto go = [&](long long from, long long to) {
            if (from < to)
                hipLaunchKernelGGL((conv_kernel<TY, W, TAIL>), dim3(dealt(blocks_of(to - from))), dim3(kThreads), 0, stream,
                                   a, from, to, tiles, (const S*)x, (const S*)weight, (const S*)bias,
                                   (const S*)initial_state, (S*)y, (S*)final_state);
        };
        if (over && final_state) {  // the tiles read what the final states overwrite
            go(0, split);
            go(split, all);
        } else {
            go(0, all);
        }
        return launch_status();
    });
}

extern "C" long long short_conv_backward_workspace(const short_conv_shape_t* shape) {
    Conv a;
    return check_shape(shape, false, &a) == CFC_OK ? workspace_of(a, shape->width) : -1;
}

extern "C" int short_conv_backward(const short_conv_shape_t* shape, const void* x, const void* weight, const void* bias,
                                   const void* initial_state, const void* grad_y, const void* grad_final_state,
                                   void* grad_x, float* grad_weight, float* grad_bias, void* grad_initial_state,
                                   void* workspace, long long workspace_bytes, hipStream_t stream) {
    Conv a;
    Sizes z;
    if (const int e = check_shape(shape, false, &a)) return e;
    const long long need = workspace_of(a, shape->width);
    if (!sizes_of(shape, a, &z) || need < 0) return CFC_ERR_DIM;
    if (!weight || !grad_weight || (a.q.n_tokens && (!x || !grad_y || !grad_x)) || (need && !workspace))
        return CFC_ERR_NULL;
    if (need && (workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 16)) return CFC_ERR_DIM;
    if (!fits({x, weight, bias, initial_state, grad_y, grad_final_state, grad_x, grad_initial_state},
              size_of(shape->type)) ||
        !fits({grad_weight, grad_bias}, 4))
        return CFC_ERR_DIM;
    const Range outs[] = {bytes_of(grad_x, z.y),
                          bytes_of(grad_weight, (long long)a.channels * shape->width * 4),
                          bytes_of(grad_bias, (long long)a.channels * 4),
                          bytes_of(grad_initial_state, z.states),
                          bytes_of(need ? workspace : nullptr, need)};
    const Range ins[] = {bytes_of(x, z.x),
                         bytes_of(weight, z.weight),
                         bytes_of(bias, z.bias),
                         bytes_of(initial_state, z.states),
                         bytes_of(grad_y, z.gy),
                         bytes_of(grad_final_state, z.states),
                         offsets_range(a.q)};
    if (!outputs_disjoint(outs, 5, ins, 7)) return CFC_ERR_OVERLAP;
    return with_width(shape, [&](auto ty, auto width, auto tail) {
        using TY = decltype(ty);
        using S = typename TY::S;
        constexpr int W = decltype(width)::value;
        constexpr bool TAIL = decltype(tail)::value;
        const long long tiles = ((long long)a.q.n_tokens + a.grad_tile - 1) / a.grad_tile, parts = parts_of(a);
        const long long waves = (tiles + (grad_initial_state ? a.q.n_seq : 0)) * parts;
        float* part = static_cast<float*>(workspace);
        if (waves)
            hipLaunchKernelGGL((conv_backward_kernel<TY, W, TAIL>), dim3(dealt(blocks_of(waves))), dim3(kThreads), 0, stream,
                               a, waves, tiles, (const S*)x, (const S*)weight, (const S*)bias, (const S*)initial_state,
                               (const S*)grad_y, (const S*)grad_final_state, (S*)grad_x, (S*)grad_initial_state, part);
        sum_columns(part, tiles, (long long)(W + 1) * a.channels, Weights{grad_weight, grad_bias, a.channels, W}, stream);
        return launch_status();
    });
}

extern "C" int short_conv_step(const short_conv_shape_t* shape, const void* x, const void* weight, const void* bias,
                               void* states, int pool, const int* slots, void* y, hipStream_t stream) {
    Conv a;
    Sizes z;
    long long held;
    if (const int e = check_shape(shape, true, &a)) return e;
    if (pool < 0 || (!slots && pool < a.q.n_tokens) || !sizes_of(shape, a, &z) ||
        !mul_ok((long long)pool * (shape->width - 1), (long long)a.channels * size_of(shape->type), &held))
        return CFC_ERR_DIM;
    if (a.q.n_tokens == 0) return CFC_OK;
    if (!x || !weight || !y || (pool && !states)) return CFC_ERR_NULL;
    if (!fits({x, weight, bias, states, y}, size_of(shape->type)) || !fits({slots}, 4)) return CFC_ERR_DIM;
    const Range outs[] = {bytes_of(y, z.y), bytes_of(states, held)};
    const Range ins[] = {bytes_of(x, z.x), bytes_of(weight, z.weight), bytes_of(bias, z.bias),
                         bytes_of(slots, (long long)a.q.n_tokens * 4)};
    if (!outputs_disjoint(outs, 2, ins, 4)) return CFC_ERR_OVERLAP;
    return with_width(shape, [&](auto ty, auto width, auto tail) {
        using TY = decltype(ty);
        using S = typename TY::S;
        constexpr int W = decltype(width)::value;
        constexpr bool TAIL = decltype(tail)::value;
        const long long waves = (long long)a.q.n_tokens * parts_of(a);
        hipLaunchKernelGGL((conv_step_kernel<TY, W, TAIL>), dim3((unsigned)blocks_of(waves)), dim3(kThreads), 0, stream, a,
                           waves, (const S*)x, (const S*)weight, (const S*)bias, (S*)states, pool, slots, (S*)y);
        return launch_status();
    });
}
