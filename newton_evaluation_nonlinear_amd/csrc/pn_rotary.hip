// Rotation by position, alone or after the norm of each head, and the
// gradients of the two together.
//
// A pair (a, b) of channels turns by the angle of its table row,
//     (a, b) -> (a c - b s, b c + a s);
// the norm before it is y = w x r, r = (mean x^2 + eps)^{-1/2}.  With g the
// gradient turned back, e = w g and n = x r:
//     dw = sum over tokens of g n,   dx = r (e - n mean(e n)).
//
// Bound: bytes.  Each row (one head of one token) is read once and written
// once, the row's sum taken across the lanes that hold it.  A group of L
// lanes holds a row, each lane "units" of V channel pairs: for the half
// layout V channels at i and V at i + R/2, so that a pair never leaves its
// lane; V is the widest access that sizes, strides and alignment allow (16
// bytes when all are multiples of it, single channels otherwise).
//
// Measured (a large copy moves 4.7 TB/s): norm and rotation of 8 x 4096 tokens,
// 16 + 4 heads of 128, bfloat16, 77 us, 4.4 TB/s; rotation of 32768 tokens, 16
// heads of 64, float32, 63 us, 4.3 TB/s (55 to 57 over the same 268 MB again and
// again, partly from cache); gradients of 4 x 4095 tokens, 16 + 16 heads of 128,
// bfloat16, 117 us, 4.6 TB/s, and 9 us for the weights' sums.

#include "pn_seq.hpp"
#include "pn_seq_device.hpp"

namespace pn {
namespace {

constexpr int kBlock = 256;

struct TableFreq {
    double f[128];
};
__global__ __launch_bounds__(kBlock) void fill_table(TableFreq freq, int n_freq, int64_t n, double magnitude,
                                                     float* table) {
    const int64_t e = static_cast<int64_t>(block_id()) * kBlock + threadIdx.x;
    if (e >= n) return;
    const int64_t p = e / n_freq;
    double s, c;
    sincos(static_cast<double>(p) * freq.f[e - p * n_freq], &s, &c);
    table[2 * e] = static_cast<float>(magnitude * c);
    table[2 * e + 1] = static_cast<float>(magnitude * s);
}

// How a row is cut into units (see the head of the file).
struct Cut {
    int L;         // lanes per row (power of two, <= 64)
    int n_rot;     // units that rotate; the others pass
    int n_units;
};

// N floats at p, which is aligned to min(N, 4) floats.
template <int N>
__device__ __forceinline__ void load_floats(const float* p, float* v) {
    constexpr int W = N < 4 ? N : 4;
#pragma unroll
    for (int i = 0; i < N; i += W) {
        const Pack<float, W> w = *reinterpret_cast<const Pack<float, W>*>(p + i);
#pragma unroll
        for (int j = 0; j < W; ++j) v[i + j] = w.v[j];
    }
}

// The channels of one lane: NU units of 2 V channels, as V pairs (a, b).
template <typename T, int V, int NU, bool INTER>
struct Lane {
    int at[NU], bt[NU];      // first channel of the two vectors
    bool on[NU], both[NU], rot[NU];
    int unit[NU];

    __device__ __forceinline__ Lane(const Cut& c, int lane, int D, int R) {
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            const int u = lane + n * c.L;
            unit[n] = u;
            on[n] = u < c.n_units;
            rot[n] = u < c.n_rot;
            if (!rot[n]) {
                at[n] = R + (u - c.n_rot) * 2 * V;
                bt[n] = at[n] + V;
            } else if (INTER) {
                at[n] = 2 * u * V;
                bt[n] = at[n] + V;
            } else {
                at[n] = u * V;
                bt[n] = R / 2 + u * V;
            }
            both[n] = on[n] && bt[n] < D;
        }
    }
    // A rotating unit of the interleaved layout holds its pairs side by side.
    __device__ __forceinline__ static void order(const float* e, float* f, bool pairs_adjacent) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            f[i] = pairs_adjacent ? e[2 * i] : e[i];
            f[V + i] = pairs_adjacent ? e[2 * i + 1] : e[V + i];
        }
    }
    __device__ __forceinline__ static void unorder(const float* f, float* e, bool pairs_adjacent) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            e[pairs_adjacent ? 2 * i : i] = f[i];
            e[pairs_adjacent ? 2 * i + 1 : V + i] = f[V + i];
        }
    }
    __device__ __forceinline__ void load(const T* row, float (*x)[2 * V]) const {
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            Pack<T, V> a{}, b{};
            if (on[n]) a = *reinterpret_cast<const Pack<T, V>*>(row + at[n]);
            if (both[n]) b = *reinterpret_cast<const Pack<T, V>*>(row + bt[n]);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                x[n][i] = to_f32(a.v[i]);
                x[n][V + i] = to_f32(b.v[i]);
            }
        }
    }
    __device__ __forceinline__ void store(T* row, const float (*x)[2 * V]) const {
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            Pack<T, V> a, b;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                a.v[i] = from_f32<T>(x[n][i]);
                b.v[i] = from_f32<T>(x[n][V + i]);
            }
            if (on[n]) *reinterpret_cast<Pack<T, V>*>(row + at[n]) = a;
            if (both[n]) *reinterpret_cast<Pack<T, V>*>(row + bt[n]) = b;
        }
    }
    // Weights in the order of load(); 1 without a weight.
    __device__ __forceinline__ void weights(const float* w, float (*x)[2 * V]) const {
#pragma unroll
        for (int n = 0; n < NU; ++n) {
#pragma unroll
            for (int i = 0; i < 2 * V; ++i) x[n][i] = 1.0f;
            if (w && on[n]) load_floats<V>(w + at[n], x[n]);
            if (w && both[n]) load_floats<V>(w + bt[n], x[n] + V);
        }
    }
    // (cos, sin) of the lane's pairs from table row p; NaN outside the table.
    __device__ __forceinline__ void angles(const float* table, int64_t p, int64_t n_pos, int R, float sign,
                                           float (*cs)[2 * V]) const {
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            if (rot[n] && p >= 0 && p < n_pos) {
                load_floats<2 * V>(table + p * R + 2 * unit[n] * V, cs[n]);
            } else {
#pragma unroll
                for (int i = 0; i < 2 * V; ++i) cs[n][i] = __builtin_nanf("");
            }
#pragma unroll
            for (int i = 0; i < V; ++i) cs[n][2 * i + 1] *= sign;
        }
    }
    __device__ __forceinline__ void turn(float (*x)[2 * V], const float (*cs)[2 * V]) const {
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            if (!rot[n]) continue;
            float f[2 * V];
            order(x[n], f, INTER);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float a = f[i], b = f[V + i], c = cs[n][2 * i], s = cs[n][2 * i + 1];
                f[i] = a * c - b * s;
                f[V + i] = b * c + a * s;
            }
            unorder(f, x[n], INTER);
        }
    }
};

__device__ __forceinline__ float row_sum(float v, int L) {
    for (int m = 1; m < L; m <<= 1) v += __shfl_xor(v, m);
    return v;
}

__device__ __forceinline__ int64_t position(const pn_rotary_args& a, int64_t b, int64_t t) {
    if (!a.positions) return a.offset + t;
    const int64_t at = b * a.pos_sb + t * a.pos_st;
    return a.pos64 ? static_cast<const int64_t*>(a.positions)[at] : static_cast<const int32_t*>(a.positions)[at];
}

// Heads of one token: a group takes `per` of the hq + hk heads, so that the
// angles are read once for them: 8 where there are rows enough to fill the
// device all the same, one for a few single tokens (latency: 3.8 us for 64
// tokens of 16 heads of 128).
template <typename T, int V, int NU, bool INTER, bool NORM>
__global__ __launch_bounds__(kBlock) void rotate(pn_rotary_args a, Cut cut, int per, int splits) {
    const int64_t g = static_cast<int64_t>(block_id()) * (kBlock / cut.L) + threadIdx.x / cut.L;
    const int lane = threadIdx.x & (cut.L - 1);
    const int64_t token = g / splits;
    if (token >= a.B * a.T) return;
    const int D = static_cast<int>(a.D), R = static_cast<int>(a.R), hq = static_cast<int>(a.hq);
    const int h0 = static_cast<int>(g - token * splits) * per;
    const int h1 = min(h0 + per, static_cast<int>(a.hq + a.hk));
    const int64_t b = token / a.T, t = token - b * a.T;
    const Lane<T, V, NU, INTER> ln(cut, lane, D, R);
    float cs[NU][2 * V], w[NU][2 * V];
    ln.angles(a.table, position(a, b, t), a.n_pos, R, a.inverse ? -1.0f : 1.0f, cs);
    const T* qrow = static_cast<const T*>(a.q.p) + b * a.q.sb + t * a.q.st;
    const T* krow = static_cast<const T*>(a.k.p) + b * a.k.sb + t * a.k.st;
    for (int h = h0; h < h1; ++h) {
        const bool isq = h < hq;
        const int hh = isq ? h : h - hq;
        float x[NU][2 * V];
        ln.load(isq ? qrow + hh * a.q.sh : krow + hh * a.k.sh, x);
        if (NORM) {
            const int64_t wsh = isq ? a.qw_sh : a.kw_sh;
            const float* wp = isq ? a.qw : a.kw;
            if (h == h0 || wsh != 0 || h == hq) ln.weights(wp ? wp + hh * wsh : nullptr, w);
            float ss = 0.0f;
#pragma unroll
            for (int n = 0; n < NU; ++n)
#pragma unroll
                for (int i = 0; i < 2 * V; ++i) ss += x[n][i] * x[n][i];
            const float r = 1.0f / sqrtf(row_sum(ss, cut.L) / static_cast<float>(D) + static_cast<float>(a.eps));
#pragma unroll
            for (int n = 0; n < NU; ++n)
#pragma unroll
                for (int i = 0; i < 2 * V; ++i) x[n][i] = x[n][i] * r * w[n][i];
        }
        ln.turn(x, cs);
        T* out = isq ? static_cast<T*>(a.q_out) + (token * a.hq + hh) * D
                     : static_cast<T*>(a.k_out) + (token * a.hk + hh) * D;
        ln.store(out, x);
    }
}

// Gradients.  A workgroup takes one head and `tokens` tokens, a group of lanes
// every (kBlock / L)-th of them, so that each lane keeps the sums of g n of
// its channels in registers; the groups' sums are added through LDS in a
// fixed order and go to part[head][workgroup][D] for weight_sum.
template <typename T, int V, int NU, bool INTER>
__global__ __launch_bounds__(kBlock) void norm_rotate_backward(pn_rotary_args a, Cut cut, int64_t tokens, int n_wg,
                                                               float* part) {
    extern __shared__ float red[];
    const int D = static_cast<int>(a.D), R = static_cast<int>(a.R), hq = static_cast<int>(a.hq);
    const int groups = kBlock / cut.L, group = threadIdx.x / cut.L, lane = threadIdx.x & (cut.L - 1);
    const uint32_t id = block_id(), heads = static_cast<uint32_t>(a.hq + a.hk);
    const int h = static_cast<int>(id % heads), wg = static_cast<int>(id / heads);
    if (wg >= n_wg) return;
    const bool isq = h < hq;
    const int hh = isq ? h : h - hq;
    const Lane<T, V, NU, INTER> ln(cut, lane, D, R);
    const pn_tokens xin = isq ? a.q : a.k, gin = isq ? a.dq : a.dk;
    const int64_t nh = isq ? a.hq : a.hk;
    const float* wp = isq ? a.qw : a.kw;
    float w[NU][2 * V], acc[NU][2 * V];
    ln.weights(wp ? wp + hh * (isq ? a.qw_sh : a.kw_sh) : nullptr, w);
#pragma unroll
    for (int n = 0; n < NU; ++n)
#pragma unroll
        for (int i = 0; i < 2 * V; ++i) acc[n][i] = 0.0f;
    const int64_t end = min(static_cast<int64_t>(wg + 1) * tokens, a.B * a.T);
    for (int64_t token = wg * tokens + group; token < end; token += groups) {
        const int64_t b = token / a.T, t = token - b * a.T;
        float cs[NU][2 * V], x[NU][2 * V], e[NU][2 * V];
        ln.load(static_cast<const T*>(xin.p) + b * xin.sb + t * xin.st + hh * xin.sh, x);
        ln.load(static_cast<const T*>(gin.p) + b * gin.sb + t * gin.st + hh * gin.sh, e);
        ln.angles(a.table, position(a, b, t), a.n_pos, R, -1.0f, cs);
        ln.turn(e, cs);
        float ss = 0.0f, en = 0.0f;
#pragma unroll
        for (int n = 0; n < NU; ++n)
#pragma unroll
            for (int i = 0; i < 2 * V; ++i) {
                ss += x[n][i] * x[n][i];
                en += e[n][i] * w[n][i] * x[n][i];
            }
        const float d = static_cast<float>(D);
        const float r = 1.0f / sqrtf(row_sum(ss, cut.L) / d + static_cast<float>(a.eps));
        const float mean = row_sum(en, cut.L) * r / d;
#pragma unroll
        for (int n = 0; n < NU; ++n)
#pragma unroll
            for (int i = 0; i < 2 * V; ++i) {
                const float hat = x[n][i] * r;
                acc[n][i] += e[n][i] * hat;
                x[n][i] = r * (e[n][i] * w[n][i] - hat * mean);
            }
        ln.store(static_cast<T*>(isq ? a.q_out : a.k_out) + (token * nh + hh) * D, x);
    }
    if (!wp) return;
#pragma unroll
    for (int n = 0; n < NU; ++n)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (ln.on[n]) red[group * D + ln.at[n] + i] = acc[n][i];
            if (ln.both[n]) red[group * D + ln.bt[n] + i] = acc[n][V + i];
        }
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += kBlock) {
        float s = 0.0f;
        for (int g = 0; g < groups; ++g) s += red[g * D + c];
        part[(static_cast<int64_t>(h) * n_wg + wg) * D + c] = s;
    }
}

// dw[x] = the sum of `rows` partial rows, x over channels (and heads, where
// each has its weight): 16 lanes of rows per channel, added in order in
// float64.  Latency: with one load at a time 1024 rows took 20 us, with 16 in
// flight 9.
__global__ __launch_bounds__(1024) void weight_sum(const float* part, int D, int n_wg, int hq, int hk, int q_own,
                                                   int k_own, float* dqw, float* dkw) {
    __shared__ double red[16][65];
    const int col = threadIdx.x % 64, lane = threadIdx.x / 64;
    const int nq = dqw ? (q_own ? hq : 1) : 0;
    const int nk = dkw ? (k_own ? hk : 1) : 0;
    const uint32_t col_blocks = (D + 63) / 64, id = block_id();
    const int sum = static_cast<int>(id / col_blocks);
    if (sum >= nq + nk) return;
    const bool isq = sum < nq;
    const int own = isq ? sum : sum - nq;
    const bool each = isq ? q_own : k_own;
    const int head = (isq ? 0 : hq) + (each ? own : 0);
    const int64_t rows = static_cast<int64_t>(each ? 1 : (isq ? hq : hk)) * n_wg;
    const int c = static_cast<int>(id % col_blocks) * 64 + col;
    const float* p = part + static_cast<int64_t>(head) * n_wg * D + c;
    double s = 0.0;
    if (c < D)
        for (int64_t r0 = lane; r0 < rows; r0 += 16 * 16) {
            float x[16];                                 // 16 loads in flight, added in order
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = p[min(r0 + 16 * i, rows - 1) * D];
#pragma unroll
            for (int i = 0; i < 16; ++i) s += r0 + 16 * i < rows ? x[i] : 0.0f;
        }
    red[lane][col] = s;
    __syncthreads();
    if (lane == 0 && c < D) {
        double v = 0.0;
        for (int i = 0; i < 16; ++i) v += red[i][col];
        (isq ? dqw : dkw)[static_cast<int64_t>(each ? own : 0) * D + c] = static_cast<float>(v);
    }
}

// ---------------------------------------------------------------- choice of the access

int64_t bits(const pn_tokens& x, const pn_rotary_args& a, int64_t heads, int64_t elem) {
    // what has to be a multiple of the access, in bytes; the stride of a
    // dimension of one is never used
    return reinterpret_cast<intptr_t>(x.p) | (a.B > 1 ? x.sb * elem : 0) | (a.T > 1 ? x.st * elem : 0) |
           (heads > 1 ? x.sh * elem : 0);
}

int widest(const pn_rotary_args& a, bool norm, bool backward) {
    const int64_t elem = a.dtype == PN_F32 ? 4 : 2;
    int64_t m = bits(a.q, a, a.hq, elem) | reinterpret_cast<intptr_t>(a.q_out);
    if (a.hk) m |= bits(a.k, a, a.hk, elem) | reinterpret_cast<intptr_t>(a.k_out);
    if (backward) m |= bits(a.dq, a, a.hq, elem) | (a.hk ? bits(a.dk, a, a.hk, elem) : 0);
    intptr_t f = reinterpret_cast<intptr_t>(a.table);
    if (norm) f |= reinterpret_cast<intptr_t>(a.qw) | reinterpret_cast<intptr_t>(a.kw);
    for (int V = static_cast<int>(16 / elem); V > 1; V /= 2) {
        const int64_t fa = 4 * (V < 4 ? V : 4);      // weights: V floats per access, at most 4
        if ((a.R / 2) % V == 0 && (a.D - a.R) % (2 * V) == 0 && m % (V * elem) == 0 && f % fa == 0 &&
            (a.R == 0 || reinterpret_cast<intptr_t>(a.table) % 16 == 0))
            return V;
    }
    return 1;
}

Cut cut_row(const pn_rotary_args& a, int V) {
    Cut c;
    c.n_rot = static_cast<int>((a.R / 2 + V - 1) / V);
    c.n_units = c.n_rot + static_cast<int>((a.D - a.R + 2 * V - 1) / (2 * V));
    c.L = 1;
    while (c.L < c.n_units && c.L < 64) c.L *= 2;
    return c;
}

// f(integral constants V, NU) for the access V and units per lane of `c`.
template <int V_, int NU_>
struct Form {
    static constexpr int V = V_, NU = NU_;
};
template <typename T, typename F>
hipError_t with_form(int V, const Cut& c, F f) {
    if (V == 8) {
        if constexpr (sizeof(T) == 2) return f(Form<8, 1>{});
        return hipErrorInvalidValue;
    }
    if (V == 4) return f(Form<4, 1>{});
    if (V == 2) return f(Form<2, 1>{});
    if (c.n_units > 64) return f(Form<1, 2>{});
    return f(Form<1, 1>{});
}

// Rows in flight per compute unit below which a group takes fewer heads: 16
// waves each.
constexpr int64_t kFillWaves = 256 * 16;

template <typename T, bool NORM>
hipError_t rotate_typed(const pn_rotary_args& a, hipStream_t st) {
    const int V = widest(a, NORM, false);
    const Cut c = cut_row(a, V);
    const int heads = static_cast<int>(a.hq + a.hk);
    const int64_t rows = a.B * a.T * heads, rows_per_wave = 64 / c.L;
    int per = 1;
    while (per < 8 && per < heads && rows / rows_per_wave / (2 * per) >= kFillWaves) per *= 2;
    const int splits = (heads + per - 1) / per;
    const int64_t groups = a.B * a.T * splits, per_block = kBlock / c.L;
    const dim3 grid = grid_of((groups + per_block - 1) / per_block, kBlock);
    return with_form<T>(V, c, [&](auto form) {
        constexpr int W = decltype(form)::V, NU = decltype(form)::NU;
        if (a.interleaved) rotate<T, W, NU, true, NORM><<<grid, kBlock, 0, st>>>(a, c, per, splits);
        else rotate<T, W, NU, false, NORM><<<grid, kBlock, 0, st>>>(a, c, per, splits);
        return hipGetLastError();
    });
}

// Workgroups per head of the backward, and the tokens of each.
void backward_split(const pn_rotary_args& a, int* n_wg, int64_t* tokens) {
    const int64_t n = a.B * a.T, heads = a.hq + a.hk;
    int64_t want = (2048 + heads - 1) / heads;
    const int64_t most = (n + 31) / 32;
    if (want > most) want = most;
    *tokens = (n + want - 1) / want;
    *n_wg = static_cast<int>((n + *tokens - 1) / *tokens);
}

template <typename T>
hipError_t backward_typed(const pn_rotary_args& a, hipStream_t st) {
    const int V = widest(a, true, true);
    const Cut c = cut_row(a, V);
    int n_wg;
    int64_t tokens;
    backward_split(a, &n_wg, &tokens);
    float* part = static_cast<float*>(a.workspace);
    const dim3 grid = grid_of(n_wg * (a.hq + a.hk), kBlock);
    const size_t lds = sizeof(float) * (kBlock / c.L) * a.D;
    hipError_t e = with_form<T>(V, c, [&](auto form) {
        constexpr int W = decltype(form)::V, NU = decltype(form)::NU;
        if (a.interleaved)
            norm_rotate_backward<T, W, NU, true><<<grid, kBlock, lds, st>>>(a, c, tokens, n_wg, part);
        else
            norm_rotate_backward<T, W, NU, false><<<grid, kBlock, lds, st>>>(a, c, tokens, n_wg, part);
        return hipGetLastError();
    });
    float* dqw = a.qw ? a.dqw : nullptr;
    float* dkw = a.kw && a.hk ? a.dkw : nullptr;
    if (e != hipSuccess || (!dqw && !dkw)) return e;
    const int q_own = a.qw_sh != 0, k_own = a.kw_sh != 0;
    const int64_t sums = (dqw ? (q_own ? a.hq : 1) : 0) + (dkw ? (k_own ? a.hk : 1) : 0);
    weight_sum<<<grid_of((a.D + 63) / 64 * sums, 1024), 1024, 0, st>>>(
        part, static_cast<int>(a.D), n_wg, static_cast<int>(a.hq), static_cast<int>(a.hk), q_own, k_own, dqw, dkw);
    return hipGetLastError();
}

template <typename T>
hipError_t rotate_pass(const pn_rotary_args& a, RotaryPass pass, hipStream_t st) {
    return pass == kNormRotate ? rotate_typed<T, true>(a, st) : rotate_typed<T, false>(a, st);
}

}  // namespace

hipError_t launch_rotary_table(const double* freq, int n_freq, int64_t n_pos, double magnitude, float* table,
                               hipStream_t st) {
    TableFreq f{};
    for (int i = 0; i < n_freq; ++i) f.f[i] = freq[i];
    const int64_t n = n_pos * n_freq;
    fill_table<<<grid_of((n + kBlock - 1) / kBlock, kBlock), kBlock, 0, st>>>(f, n_freq, n, magnitude, table);
    return hipGetLastError();
}

__global__ __launch_bounds__(kBlock) void fill_zero(float* p, int64_t n) {
    const int64_t e = static_cast<int64_t>(block_id()) * kBlock + threadIdx.x;
    if (e < n) p[e] = 0.0f;
}

hipError_t launch_fill(float* p, int64_t n, hipStream_t st) {
    if (n <= 0) return hipSuccess;
    fill_zero<<<grid_of((n + kBlock - 1) / kBlock, kBlock), kBlock, 0, st>>>(p, n);
    return hipGetLastError();
}

hipError_t launch_rotary(const pn_rotary_args& a, RotaryPass pass, hipStream_t st) {
    switch (a.dtype) {
        case PN_F32: return rotate_pass<float>(a, pass, st);
        case PN_BF16: return rotate_pass<bf16>(a, pass, st);
        default: return rotate_pass<f16>(a, pass, st);
    }
}

size_t rotary_backward_workspace(const pn_rotary_args& a) {
    int n_wg;
    int64_t tokens;
    backward_split(a, &n_wg, &tokens);
    return sizeof(float) * static_cast<size_t>(n_wg) * static_cast<size_t>(a.hq + a.hk) * static_cast<size_t>(a.D);
}

hipError_t launch_rotary_backward(const pn_rotary_args& a, hipStream_t st) {
    switch (a.dtype) {
        case PN_F32: return backward_typed<float>(a, st);
        case PN_BF16: return backward_typed<bf16>(a, st);
        default: return backward_typed<f16>(a, st);
    }
}

}  // namespace pn
