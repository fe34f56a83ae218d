// Short causal convolution of each channel,
//     pre_t = bias + sum_{k < W} w_k x_{t-W+1+k},   y = act(pre),
// its gradients, with d = dy act'(pre) (0 past the last token),
//     dx_t = sum_k w_k d_{t+W-1-k},   dw_k = sum_t d_t x_{t-W+1+k},   dbias = sum_t d_t,
// and its single-token form.
//
// Bound: bytes.  A thread takes V adjacent channels (8 bytes in the forward, two
// channels in the gradients, where sizes, strides and alignment allow, one
// channel otherwise) and walks `run` tokens with the last W - 1 in registers, so
// that a token is read once and, at the ends of runs, W - 1 times more.  Wider
// vectors leave too few waves: 16 bytes take 62 us where 8 take 50 (8 x 4096
// tokens of 2048 channels, 4 taps, bfloat16), the gradients of four channels 123
// where two take 104.  The number of taps is known to the compiler: with a
// branch a tap the gradients of 3 and 8 taps take 209 and 419 us, not 94 and 168.
//
// Measured at that size: 50 us, 5.4 TB/s (part of it from the cache); gradients
// 104, 3.9 TB/s, and 7 for the sums; in float32 105 and 186, 5.1 and 4.3 TB/s.
// Single tokens of 256 x 4096 channels 6.6 us.

#include <algorithm>
#include <type_traits>

#include "pn_ssm.hpp"
#include "pn_ssm_device.hpp"

namespace pn {
namespace {

constexpr int kBlock = 256;

struct ConvCut {
    int64_t run;             // tokens of a thread
    int64_t runs;            // of a sequence
    int vecs;                // threads across the channels
};

template <typename T, int V>
__device__ __forceinline__ void load(const T* p, float* v) {
    const Pack<T, V> q = *reinterpret_cast<const Pack<T, V>*>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = to_f32(q.v[i]);
}
// Binary16 is rounded from the float32 value everywhere: a product and sum that
// round to 16 bits at once, where the compiler finds them, would make a token's
// last bit depend on its place in a run.
template <typename T, int V>
__device__ __forceinline__ void store(T* p, const float* v) {
    Pack<T, V> q;
#pragma unroll
    for (int i = 0; i < V; ++i) q.v[i] = from_f32<T>(std::is_same<T, f16>::value ? pinned(v[i]) : v[i]);
    *reinterpret_cast<Pack<T, V>*>(p) = q;
}

// Token t >= -(W - 1) of a sequence of n tokens (0 before the initial state and from n on).
template <typename T, int V>
__device__ __forceinline__ void token(const pn_conv_args& a, int64_t b, int64_t t, int64_t n, int d, float* v) {
    const int64_t past = a.W - 1;
    if (t >= 0 && t < n) {
        load<T, V>(static_cast<const T*>(a.x.p) + b * a.x.sb + t * a.x.st + d, v);
    } else if (t < 0 && t >= -past && a.initial_state) {
        load<T, V>(static_cast<const T*>(a.initial_state) + (b * past + past + t) * a.D + d, v);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 0.0f;
    }
}

// The taps of V channels.
template <int V, int W>
__device__ __forceinline__ void weights(const float* weight, int d, float (*w)[V]) {
#pragma unroll
    for (int k = 0; k < W; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) w[k][i] = weight[static_cast<int64_t>(d + i) * W + k];
}

struct Place {
    int64_t b, run;
    int d;
    bool on;
};
template <int V>
__device__ __forceinline__ Place place(const pn_conv_args& a, const ConvCut& c) {
    const int64_t id = static_cast<int64_t>(block_id()) * kBlock + threadIdx.x;
    Place p;
    const int64_t r = id / c.vecs;
    p.d = static_cast<int>(id - r * c.vecs) * V;
    p.b = r / c.runs;
    p.run = r - p.b * c.runs;
    p.on = p.b < a.B;
    return p;
}
__device__ __forceinline__ int64_t length(const pn_conv_args& a, int64_t b) {
    return a.lengths ? max(static_cast<int64_t>(0), min(static_cast<int64_t>(a.lengths[b]), a.T)) : a.T;
}

// Four tokens at a time; the next four are loaded before the products of these.
template <typename T, int V, int W>
__global__ __launch_bounds__(kBlock) void conv(pn_conv_args a, ConvCut c) {
    const Place p = place<V>(a, c);
    if (!p.on) return;
    const int64_t n = length(a, p.b), t0 = p.run * c.run, t1 = min(t0 + c.run, a.T), end = min(t1, n);
    T* y = static_cast<T*>(a.y) + p.b * a.T * a.D + p.d;
    if (p.run == 0 && a.final_state)
        for (int64_t r = 0; r < W - 1; ++r) {
            float v[V];
            token<T, V>(a, p.b, n - (W - 1) + r, n, p.d, v);
            store<T, V>(static_cast<T*>(a.final_state) + (p.b * (W - 1) + r) * a.D + p.d, v);
        }
    if (t0 < end) {
        float w[W][V], bias[V], x[W - 1 + 4][V];
        weights<V, W>(a.weight, p.d, w);
#pragma unroll
        for (int i = 0; i < V; ++i) bias[i] = a.bias ? a.bias[p.d + i] : 0.0f;
#pragma unroll
        for (int k = 0; k < W - 1; ++k) token<T, V>(a, p.b, t0 - (W - 1) + k, n, p.d, x[k]);
        const T* row = static_cast<const T*>(a.x.p) + p.b * a.x.sb + p.d;
        Pack<T, V> next[4];
        auto fetch = [&](int64_t t) {                    // rows behind the last are the last again: not stored
#pragma unroll
            for (int j = 0; j < 4; ++j) next[j] = *reinterpret_cast<const Pack<T, V>*>(row + min(t + j, end - 1) * a.x.st);
        };
        fetch(t0);
        for (int64_t t = t0; t < end; t += 4) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) x[W - 1 + j][i] = to_f32(next[j].v[i]);
            if (t + 4 < end) fetch(t + 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float v[V];
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = bias[i];
#pragma unroll
                for (int k = 0; k < W; ++k)
#pragma unroll
                    for (int i = 0; i < V; ++i) v[i] = fmaf(w[k][i], x[j + k][i], v[i]);
                if (a.activation)
#pragma unroll
                    for (int i = 0; i < V; ++i) v[i] *= logistic(v[i]);
                if (t + j < end) store<T, V>(y + (t + j) * a.D, v);
            }
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) x[k][i] = x[k + 4][i];
        }
    }
    const float zero[V] = {};
    for (int64_t t = max(end, t0); t < t1; ++t) store<T, V>(y + t * a.D, zero);
}

// Gradients.  The walk goes over tokens t0 .. t1 + W - 2: each gives d_t from
// its W tokens, and with it dx of the token W - 1 before.
template <typename T, int V, int W>
__global__ __launch_bounds__(kBlock) void conv_backward(pn_conv_args a, ConvCut c, float* part) {
    constexpr int past = W - 1;
    const Place p = place<V>(a, c);
    if (!p.on) return;
    const int64_t n = length(a, p.b), t0 = p.run * c.run, t1 = min(t0 + c.run, a.T);
    float w[W][V], bias[V], x[W][V], d[W][V], dw[W][V], db[V];
    weights<V, W>(a.weight, p.d, w);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        bias[i] = a.bias ? a.bias[p.d + i] : 0.0f;
        db[i] = 0.0f;
#pragma unroll
        for (int k = 0; k < W; ++k) dw[k][i] = d[k][i] = x[k][i] = 0.0f;
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k) token<T, V>(a, p.b, t0 - (W - 1) + k, n, p.d, x[k + 1]);
    const T* xrow = static_cast<const T*>(a.x.p) + p.b * a.x.sb + p.d;
    const T* grow = static_cast<const T*>(a.dy.p) + p.b * a.dy.sb + p.d;
    constexpr int AHEAD = 4;                             // tokens loaded at a time, while those before are worked on
    Pack<T, V> nx[AHEAD], ng[AHEAD], cx[AHEAD], cg[AHEAD];
    auto fetch = [&](int64_t s) {                        // rows behind the last are the last again: not used
        if (n <= 0) return;
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const int64_t t = min(s + j, n - 1);
            nx[j] = *reinterpret_cast<const Pack<T, V>*>(xrow + t * a.x.st);
            ng[j] = *reinterpret_cast<const Pack<T, V>*>(grow + t * a.dy.st);
        }
    };
    // x[k] and d[k]: of token t - (W - 1) + k.  Whole: all tokens up to the tile's
    // end are the run's and the sequence's and dx is the run's, so that nothing
    // is looked up.
    auto tile = [&](int64_t s, auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const int64_t t = s + j;
            if (!WHOLE && t >= t1 + past) break;
            const bool on = WHOLE || t < n;
#pragma unroll
            for (int i = 0; i < V; ++i) {
#pragma unroll
                for (int k = 0; k < W - 1; ++k) {
                    d[k][i] = d[k + 1][i];
                    x[k][i] = x[k + 1][i];
                }
                x[W - 1][i] = on ? to_f32(cx[j].v[i]) : 0.0f;
                float pre = bias[i];
#pragma unroll
                for (int k = 0; k < W; ++k)
                    pre = fmaf(w[k][i], x[k][i], pre);
                const float g = to_f32(cg[j].v[i]), q = logistic(pre), by = a.activation ? q * fmaf(pre, 1.0f - q, 1.0f) : 1.0f;
                d[W - 1][i] = on ? g * by : 0.0f;
            }
            if (WHOLE || t < t1)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    db[i] += d[W - 1][i];
#pragma unroll
                    for (int k = 0; k < W; ++k)
                        dw[k][i] = fmaf(d[W - 1][i], x[k][i], dw[k][i]);
                }
            const int64_t at = t - past;                 // W - 1 tokens back: d[W - W + q] is that of token at + q
            if (!WHOLE && at < t0 && !(p.run == 0 && a.d_initial_state)) continue;
            float v[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[i] = 0.0f;
#pragma unroll
                for (int k = 0; k < W; ++k)
                    v[i] = fmaf(w[k][i], d[W - 1 - k][i], v[i]);
                if (!WHOLE && at >= n) v[i] = 0.0f;
            }
            if (!WHOLE && a.d_final_state && at < n && at >= n - past) {
                float f[V];
                load<T, V>(static_cast<const T*>(a.d_final_state) + (p.b * past + at - (n - past)) * a.D + p.d, f);
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] += f[i];
            }
            if (WHOLE || at >= 0) store<T, V>(static_cast<T*>(a.dx) + (p.b * a.T + at) * a.D + p.d, v);
            else store<T, V>(static_cast<T*>(a.d_initial_state) + (p.b * past + past + at) * a.D + p.d, v);
        }
    };
    fetch(t0);
    for (int64_t s = t0; s < t1 + past; s += AHEAD) {
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            cx[j] = nx[j];
            cg[j] = ng[j];
        }
        if (s + AHEAD < t1 + past) fetch(s + AHEAD);
        if (s - past >= t0 && s + AHEAD <= min(t1, n)) tile(s, std::true_type());
        else tile(s, std::false_type());
    }
    float* q = part + (p.b * c.runs + p.run) * (W + 1) * a.D;
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int k = 0; k < W; ++k)
            q[(p.d + i) * a.W + k] = dw[k][i];
        q[a.W * a.D + p.d + i] = db[i];
    }
}

// No token: the initial state is the final one.
template <typename T>
__global__ __launch_bounds__(kBlock) void conv_state_gradient(const T* d_final, T* d_initial, int64_t n) {
    const int64_t i = static_cast<int64_t>(block_id()) * kBlock + threadIdx.x;
    if (i < n) d_initial[i] = d_final ? d_final[i] : from_f32<T>(0.0f);
}

// A channel's taps are read together: one by one, a line of memory a lane, they
// take longer than the states (14.6 us where the call above takes 6.6).
template <typename T, int V, int W>
__global__ __launch_bounds__(kBlock) void conv_step(pn_conv_step_args a, int vecs) {
    const int64_t id = static_cast<int64_t>(block_id()) * kBlock + threadIdx.x, b = id / vecs;
    if (b >= a.B) return;
    const int d = static_cast<int>(id - b * vecs) * V;
    const int64_t slot = a.slots ? a.slots[b] : b;
    T* y = static_cast<T*>(a.y) + b * a.D + d;
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 0.0f;
    if (slot < 0 || slot >= a.n_slots) {
        store<T, V>(y, v);
        return;
    }
    T* s = static_cast<T*>(a.state) + slot * (W - 1) * a.D + d;
    Pack<T, V> row[W];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) row[k] = *reinterpret_cast<const Pack<T, V>*>(s + k * a.D);
    row[W - 1] = *reinterpret_cast<const Pack<T, V>*>(static_cast<const T*>(a.x.p) + b * a.x.sb + d);
    float w[W][V];
    weights<V, W>(a.weight, d, w);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = a.bias ? a.bias[d + i] : 0.0f;
#pragma unroll
    for (int k = 0; k < W; ++k) {
        if (k > 0) *reinterpret_cast<Pack<T, V>*>(s + (k - 1) * a.D) = row[k];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = fmaf(w[k][i], to_f32(row[k].v[i]), v[i]);
    }
    if (a.activation)
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= logistic(v[i]);
    store<T, V>(y, v);
}

// Whether V channels of every row can be moved together.
template <typename... P>
bool aligned(int64_t D, int64_t elem, int V, int64_t strides, P... p) {
    return D % V == 0 && ((strides * elem) | (reinterpret_cast<intptr_t>(p) | ...)) % (V * elem) == 0;
}
int64_t strides(const pn_tokens& x, int64_t B, int64_t T) { return (B > 1 ? x.sb : 0) | (T > 1 ? x.st : 0); }

// Tokens of a thread: 64, or down to `least` while 2^18 threads (four waves for
// every SIMD) are not reached.
ConvCut cut(const pn_conv_args& a, int V, int least) {
    ConvCut c;
    c.vecs = static_cast<int>(a.D / V);
    c.run = 64;
    while (c.run > least && a.B * c.vecs * ((a.T + c.run - 1) / c.run) < (1 << 18)) c.run /= 2;
    c.runs = std::max<int64_t>(1, (a.T + c.run - 1) / c.run);
    return c;
}

// f(the number of taps, known to the compiler: no branch a tap).
template <typename F>
hipError_t with_taps(int64_t W, F f) {
    switch (W) {
        case 1: return f(std::integral_constant<int, 1>());
        case 2: return f(std::integral_constant<int, 2>());
        case 3: return f(std::integral_constant<int, 3>());
        case 4: return f(std::integral_constant<int, 4>());
        case 5: return f(std::integral_constant<int, 5>());
        case 6: return f(std::integral_constant<int, 6>());
        case 7: return f(std::integral_constant<int, 7>());
        default: return f(std::integral_constant<int, 8>());
    }
}

template <typename T>
hipError_t conv_typed(const pn_conv_args& a, hipStream_t st) {
    constexpr int V = 8 / sizeof(T);
    const bool wide = aligned(a.D, sizeof(T), V, strides(a.x, a.B, a.T), a.x.p, a.initial_state, a.y, a.final_state);
    const ConvCut c = cut(a, wide ? V : 1, 8);
    const dim3 grid = grid_of((a.B * c.runs * c.vecs + kBlock - 1) / kBlock, kBlock);
    return with_taps(a.W, [&](auto taps) {
        constexpr int W = decltype(taps)::value;
        if (wide) conv<T, V, W><<<grid, kBlock, 0, st>>>(a, c);
        else conv<T, 1, W><<<grid, kBlock, 0, st>>>(a, c);
        return hipGetLastError();
    });
}

// The gradients' runs are those of single channels, so that the workspace
// does not depend on alignment.
template <typename T>
hipError_t backward_typed(const pn_conv_args& a, hipStream_t st) {
    constexpr int V = 2;
    const bool wide = aligned(a.D, sizeof(T), V, strides(a.x, a.B, a.T) | strides(a.dy, a.B, a.T), a.x.p, a.dy.p,
                              a.initial_state, a.d_final_state, a.dx, a.d_initial_state);
    ConvCut c = cut(a, 1, 16);
    if (wide) c.vecs = static_cast<int>(a.D / V);
    const dim3 grid = grid_of((a.B * c.runs * c.vecs + kBlock - 1) / kBlock, kBlock);
    float* part = static_cast<float*>(a.workspace);
    const hipError_t e = with_taps(a.W, [&](auto taps) {
        constexpr int W = decltype(taps)::value;
        if (wide) conv_backward<T, V, W><<<grid, kBlock, 0, st>>>(a, c, part);
        else conv_backward<T, 1, W><<<grid, kBlock, 0, st>>>(a, c, part);
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    return launch_column_sum(ColumnSum{part, a.B * c.runs, (a.W + 1) * a.D, 2, {0, a.W * a.D}, {a.dweight, a.bias ? a.dbias : nullptr}}, st);
}

template <typename T>
hipError_t step_typed(const pn_conv_step_args& a, hipStream_t st) {
    constexpr int V = 8 / sizeof(T);                     // a few channels: there are few threads in all
    const bool wide = aligned(a.D, sizeof(T), V, a.B > 1 ? a.x.sb : 0, a.x.p, a.state, a.y);
    const int vecs = static_cast<int>(wide ? a.D / V : a.D);
    const dim3 grid = grid_of((a.B * vecs + kBlock - 1) / kBlock, kBlock);
    return with_taps(a.W, [&](auto taps) {
        constexpr int W = decltype(taps)::value;
        if (wide) conv_step<T, V, W><<<grid, kBlock, 0, st>>>(a, vecs);
        else conv_step<T, 1, W><<<grid, kBlock, 0, st>>>(a, vecs);
        return hipGetLastError();
    });
}

}  // namespace

hipError_t launch_conv(const pn_conv_args& a, hipStream_t st) {
    switch (a.dtype) {
        case PN_F32: return conv_typed<float>(a, st);
        case PN_BF16: return conv_typed<bf16>(a, st);
        default: return conv_typed<f16>(a, st);
    }
}

size_t conv_workspace(const pn_conv_args& a) {
    return sizeof(float) * static_cast<size_t>(a.B * cut(a, 1, 16).runs) * static_cast<size_t>((a.W + 1) * a.D);
}

hipError_t launch_conv_backward(const pn_conv_args& a, hipStream_t st) {
    switch (a.dtype) {
        case PN_F32: return backward_typed<float>(a, st);
        case PN_BF16: return backward_typed<bf16>(a, st);
        default: return backward_typed<f16>(a, st);
    }
}

hipError_t launch_conv_state(const pn_conv_args& a, hipStream_t st) {
    const int64_t n = a.B * (a.W - 1) * a.D;
    const dim3 grid = grid_of((n + kBlock - 1) / kBlock, kBlock);
    auto run = [&](auto zero) {
        using T = decltype(zero);
        conv_state_gradient<T><<<grid, kBlock, 0, st>>>(static_cast<const T*>(a.d_final_state), static_cast<T*>(a.d_initial_state), n);
        return hipGetLastError();
    };
    switch (a.dtype) {
        case PN_F32: return run(float{});
        case PN_BF16: return run(bf16{});
        default: return run(f16{});
    }
}

hipError_t launch_conv_step(const pn_conv_step_args& a, hipStream_t st) {
    switch (a.dtype) {
        case PN_F32: return step_typed<float>(a, st);
        case PN_BF16: return step_typed<bf16>(a, st);
        default: return step_typed<f16>(a, st);
    }
}

}  // namespace pn
