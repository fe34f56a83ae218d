// Short causal convolution of each channel,
//     pre_t = bias + sum_{k < W} w_k x_{t-W+1+k},   y = act(pre),
// its gradients, with d = dy act'(pre) (0 past the last token),
//     dx_t = sum_k w_k d_{t+W-1-k},   dw_k = sum_t d_t x_{t-W+1+k},   dbias = sum_t d_t,
// and its single-token form.
//
// Bound: bytes.  A thread takes V adjacent channels (16 bytes where sizes,
// strides and alignment allow, one channel otherwise) and walks `run` tokens
// with the last W - 1 in registers, so that a token is read once and, at the
// ends of runs, W - 1 times more.

#include <algorithm>

#include "pn_seq_device.hpp"
#include "pn_ssm.hpp"

namespace pn {
namespace {

constexpr int kBlock = 256;
constexpr float kLog2e = 1.4426950408889634f;

struct ConvCut {
    int64_t run;             // tokens of a thread
    int64_t runs;            // of a sequence
    int vecs;                // threads across the channels
};

// e^-v past float32 is infinite and its reciprocal 0: -0 for v far below 0.
__device__ __forceinline__ float logistic(float v) { return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-v * kLog2e)); }

template <typename T, int V>
__device__ __forceinline__ void load(const T* p, float* v) {
    const Pack<T, V> q = *reinterpret_cast<const Pack<T, V>*>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = to_f32(q.v[i]);
}
template <typename T, int V>
__device__ __forceinline__ void store(T* p, const float* v) {
    Pack<T, V> q;
#pragma unroll
    for (int i = 0; i < V; ++i) q.v[i] = from_f32<T>(v[i]);
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

// The taps of V channels, in the last W of K places.
template <int V, int K>
__device__ __forceinline__ void taps(const pn_conv_args& a, int d, float (*w)[V]) {
    const int W = static_cast<int>(a.W);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) w[k][i] = k >= K - W ? a.weight[static_cast<int64_t>(d + i) * W + k - (K - W)] : 0.0f;
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

// K: 4 or 8 places for taps.  Four tokens at a time, their loads together.
template <typename T, int V, int K>
__global__ __launch_bounds__(kBlock) void conv(pn_conv_args a, ConvCut c) {
    const Place p = place<V>(a, c);
    if (!p.on) return;
    const int W = static_cast<int>(a.W);
    const int64_t n = length(a, p.b), t0 = p.run * c.run, t1 = min(t0 + c.run, a.T), end = min(t1, n);
    T* y = static_cast<T*>(a.y) + p.b * a.T * a.D + p.d;
    if (p.run == 0 && a.final_state)
        for (int64_t r = 0; r < W - 1; ++r) {
            float v[V];
            token<T, V>(a, p.b, n - (W - 1) + r, n, p.d, v);
            store<T, V>(static_cast<T*>(a.final_state) + (p.b * (W - 1) + r) * a.D + p.d, v);
        }
    float w[K][V], bias[V], x[K - 1 + 4][V];
    taps<V, K>(a, p.d, w);
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = a.bias ? a.bias[p.d + i] : 0.0f;
#pragma unroll
    for (int k = 0; k < K - 1; ++k)
        if (k >= K - W) token<T, V>(a, p.b, t0 - (K - 1) + k, n, p.d, x[k]);
    for (int64_t t = t0; t < end; t += 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) token<T, V>(a, p.b, t + j, end, p.d, x[K - 1 + j]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float v[V];
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = bias[i];
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (k >= K - W)                          // taps that are not there touch no token
#pragma unroll
                    for (int i = 0; i < V; ++i) v[i] = fmaf(w[k][i], x[j + k][i], v[i]);
            if (a.activation)
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] *= logistic(v[i]);
            if (t + j < end) store<T, V>(y + (t + j) * a.D, v);
        }
#pragma unroll
        for (int k = 0; k < K - 1; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) x[k][i] = x[k + 4][i];
    }
    const float zero[V] = {};
    for (int64_t t = max(end, t0); t < t1; ++t) store<T, V>(y + t * a.D, zero);
}

// Gradients.  The walk goes over tokens t0 .. t1 + W - 2: each gives d_t from
// its W tokens, and with it dx of the token W - 1 before.
template <typename T, int V, int K>
__global__ __launch_bounds__(kBlock) void conv_backward(pn_conv_args a, ConvCut c, float* part) {
    const Place p = place<V>(a, c);
    if (!p.on) return;
    const int W = static_cast<int>(a.W), past = W - 1;
    const int64_t n = length(a, p.b), t0 = p.run * c.run, t1 = min(t0 + c.run, a.T);
    float w[K][V], bias[V], x[K][V], d[K][V], dw[K][V], db[V];
    taps<V, K>(a, p.d, w);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        bias[i] = a.bias ? a.bias[p.d + i] : 0.0f;
        db[i] = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) dw[k][i] = d[k][i] = x[k][i] = 0.0f;
    }
#pragma unroll
    for (int k = 0; k < K - 1; ++k)
        if (k >= K - W) token<T, V>(a, p.b, t0 - (K - 1) + k, n, p.d, x[k + 1]);
    // x[k] and d[k]: of token t - (K - 1) + k
    for (int64_t t = t0; t < t1 + past; ++t) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int k = 0; k < K - 1; ++k) {
                d[k][i] = d[k + 1][i];
            }
            d[K - 1][i] = 0.0f;
        }
        token<T, V>(a, p.b, t, n, p.d, x[0]);
        {
            float fresh[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                fresh[i] = x[0][i];
#pragma unroll
                for (int k = 0; k < K - 1; ++k) x[k][i] = x[k + 1][i];
                x[K - 1][i] = fresh[i];
            }
        }
        if (t < n) {
            float dy[V];
            load<T, V>(static_cast<const T*>(a.dy.p) + p.b * a.dy.sb + t * a.dy.st + p.d, dy);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float pre = bias[i];
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (k >= K - W) pre = fmaf(w[k][i], x[k][i], pre);
                float g = dy[i];
                if (a.activation) {
                    const float s = logistic(pre);
                    g *= s * fmaf(pre, 1.0f - s, 1.0f);
                }
                d[K - 1][i] = g;
                if (t < t1) {
                    db[i] += g;
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        if (k >= K - W) dw[k][i] = fmaf(g, x[k][i], dw[k][i]);
                }
            }
        }
        const int64_t at = t - past;                     // W - 1 tokens back: d[K - W + j] is that of token at + j
        if (at < t0 && !(p.run == 0 && a.d_initial_state)) continue;
        float v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 0.0f;
        if (at < n) {
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (j >= K - W)
#pragma unroll
                    for (int i = 0; i < V; ++i) v[i] = fmaf(w[K - 1 - (j - (K - W))][i], d[j][i], v[i]);
            if (a.d_final_state && at >= n - past) {
                float f[V];
                load<T, V>(static_cast<const T*>(a.d_final_state) + (p.b * past + at - (n - past)) * a.D + p.d, f);
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] += f[i];
            }
        }
        if (at >= 0) store<T, V>(static_cast<T*>(a.dx) + (p.b * a.T + at) * a.D + p.d, v);
        else store<T, V>(static_cast<T*>(a.d_initial_state) + (p.b * past + past + at) * a.D + p.d, v);
    }
    float* q = part + (p.b * c.runs + p.run) * (W + 1) * a.D + p.d;
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (k >= K - W) q[static_cast<int64_t>(p.d + i) * (W - 1) + i + k - (K - W)] = dw[k][i];
        q[static_cast<int64_t>(W) * a.D + i] = db[i];
    }
}

// No token: the initial state is the final one.
template <typename T>
__global__ __launch_bounds__(kBlock) void conv_state_gradient(const T* d_final, T* d_initial, int64_t n) {
    const int64_t i = static_cast<int64_t>(block_id()) * kBlock + threadIdx.x;
    if (i < n) d_initial[i] = d_final ? d_final[i] : from_f32<T>(0.0f);
}

template <typename T, int V>
__global__ __launch_bounds__(kBlock) void conv_step(pn_conv_step_args a, int vecs) {
    const int64_t id = static_cast<int64_t>(block_id()) * kBlock + threadIdx.x, b = id / vecs;
    if (b >= a.B) return;
    const int d = static_cast<int>(id - b * vecs) * V, W = static_cast<int>(a.W);
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
    Pack<T, V> row[8];
#pragma unroll
    for (int k = 0; k < 7; ++k)
        if (k < W - 1) row[k] = *reinterpret_cast<const Pack<T, V>*>(s + k * a.D);
    const Pack<T, V> x = *reinterpret_cast<const Pack<T, V>*>(static_cast<const T*>(a.x.p) + b * a.x.sb + d);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = a.bias ? a.bias[d + i] : 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if (k > W - 1) continue;
        const Pack<T, V> t = k == W - 1 ? x : row[k];
        if (k > 0) *reinterpret_cast<Pack<T, V>*>(s + (k - 1) * a.D) = t;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = fmaf(a.weight[static_cast<int64_t>(d + i) * W + k], to_f32(t.v[i]), v[i]);
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

// Tokens of a thread: 64, or fewer while 2^18 threads (four waves for every
// SIMD) are not reached.
ConvCut cut(const pn_conv_args& a, int V) {
    ConvCut c;
    c.vecs = static_cast<int>(a.D / V);
    c.run = 64;
    while (c.run > 8 && a.B * c.vecs * ((a.T + c.run - 1) / c.run) < (1 << 18)) c.run /= 2;
    c.runs = std::max<int64_t>(1, (a.T + c.run - 1) / c.run);
    return c;
}

template <typename T>
hipError_t conv_typed(const pn_conv_args& a, hipStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const bool wide = aligned(a.D, sizeof(T), V, strides(a.x, a.B, a.T), a.x.p, a.initial_state, a.y, a.final_state);
    const ConvCut c = cut(a, wide ? V : 1);
    const dim3 grid = grid_of((a.B * c.runs * c.vecs + kBlock - 1) / kBlock, kBlock);
    if (wide && a.W <= 4) conv<T, V, 4><<<grid, kBlock, 0, st>>>(a, c);
    else if (wide) conv<T, V, 8><<<grid, kBlock, 0, st>>>(a, c);
    else if (a.W <= 4) conv<T, 1, 4><<<grid, kBlock, 0, st>>>(a, c);
    else conv<T, 1, 8><<<grid, kBlock, 0, st>>>(a, c);
    return hipGetLastError();
}

// The gradients' runs are those of single channels, so that the workspace
// does not depend on alignment.
template <typename T>
hipError_t backward_typed(const pn_conv_args& a, hipStream_t st) {
    constexpr int V = 8 / sizeof(T);
    const bool wide = aligned(a.D, sizeof(T), V, strides(a.x, a.B, a.T) | strides(a.dy, a.B, a.T), a.x.p, a.dy.p,
                              a.initial_state, a.d_final_state, a.dx, a.d_initial_state);
    ConvCut c = cut(a, 1);
    if (wide) c.vecs = static_cast<int>(a.D / V);
    const dim3 grid = grid_of((a.B * c.runs * c.vecs + kBlock - 1) / kBlock, kBlock);
    float* part = static_cast<float*>(a.workspace);
    if (wide && a.W <= 4) conv_backward<T, V, 4><<<grid, kBlock, 0, st>>>(a, c, part);
    else if (wide) conv_backward<T, V, 8><<<grid, kBlock, 0, st>>>(a, c, part);
    else if (a.W <= 4) conv_backward<T, 1, 4><<<grid, kBlock, 0, st>>>(a, c, part);
    else conv_backward<T, 1, 8><<<grid, kBlock, 0, st>>>(a, c, part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return launch_column_sum(ColumnSum{part, a.B * c.runs, (a.W + 1) * a.D, 2, {0, a.W * a.D}, {a.dweight, a.bias ? a.dbias : nullptr}}, st);
}

template <typename T>
hipError_t step_typed(const pn_conv_step_args& a, hipStream_t st) {
    constexpr int V = 8 / sizeof(T);                     // a few channels: there are few threads in all
    const bool wide = aligned(a.D, sizeof(T), V, a.B > 1 ? a.x.sb : 0, a.x.p, a.state, a.y);
    const int vecs = static_cast<int>(wide ? a.D / V : a.D);
    const dim3 grid = grid_of((a.B * vecs + kBlock - 1) / kBlock, kBlock);
    if (wide) conv_step<T, V><<<grid, kBlock, 0, st>>>(a, vecs);
    else conv_step<T, 1><<<grid, kBlock, 0, st>>>(a, vecs);
    return hipGetLastError();
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
    return sizeof(float) * static_cast<size_t>(a.B * cut(a, 1).runs) * static_cast<size_t>((a.W + 1) * a.D);
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
