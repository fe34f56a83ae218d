// The norms around a block, with its gate and the scaled residual,
//     u = x silu(gate),  p = pw u ru,  s = residual + scale p,  y = w s rs,
// ru = (mean u^2 + eps)^{-1/2} and rs likewise of s; and the gradients, with
// n = u ru, m = s rs and t the gradient of s as a whole,
//     e = w dy,  t = ds + rs (e - m mean(e m)),  dresidual = t,  dw = sum dy m,
//     q = pw scale t,  du = ru (q - n mean(q n)),  dpw = scale sum t n,
//     dscale = pw sum t n,  dx = du silu(gate),  dgate = du x silu'(gate).
//
// A row whose squares pass float32 has ru or rs of 0: nothing goes through that
// norm, and neither does a gradient, also where the sums of its products are
// past float32.
//
// The gradients form s again from what the forward took, in float32: from s
// as it was stored in 16 bits, dw would keep its rounding.
//
// Bound: bytes.  A row stays in the registers of the lanes that hold it, NU
// units of V channels each, so everything is read once and written once; sums
// over a row go through the lanes and, in workgroups of several waves, LDS.
// V: 16 bytes of the storage type where sizes, strides and alignment allow,
// two channels or one otherwise.
//
// Measured: 8 x 4096 rows of 2048 channels, bfloat16, gate, norms, scale and
// residual: 130 to 140 us, 4.8 to 5.1 TB/s; half as many with gradients 76 and
// 120, 4.4 and 4.5 TB/s, and 8 for the weights' sums; 8192 channels, 4 x 4096
// rows: 272 and 674, 4.9 and 3.1 TB/s (the gradients hold 16 channels a lane
// and run 8 waves a unit).  4 x 2047 rows of 2050 channels on a float32 residual,
// two channels at a time: 66 and 89, 6 for the sums.  Odd widths go channel by
// channel: 2049 channels, 4 x 4096 rows, 164 to 173 and 172 to 177.

#include <algorithm>

#include "pn_ssm.hpp"
#include "pn_ssm_device.hpp"

namespace pn {
namespace {

// Sums of two values over the workgroup, in every lane.
template <int THREADS>
__device__ __forceinline__ void row_sums(float& x, float& y, float* lds) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        x += __shfl_xor(x, m);
        y += __shfl_xor(y, m);
    }
    if (THREADS == 64) return;
    constexpr int WAVES = THREADS / 64;
    __syncthreads();                                     // the last sums have been read
    if (threadIdx.x % 64 == 0) {
        lds[threadIdx.x / 64] = x;
        lds[WAVES + threadIdx.x / 64] = y;
    }
    __syncthreads();
    x = y = 0.0f;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
        x += lds[i];
        y += lds[WAVES + i];
    }
}

// The channels of one lane: unit u is V channels from at(u).
template <int V, int NU, int THREADS>
struct Row {
    int D;
    __device__ __forceinline__ int at(int u) const { return (static_cast<int>(threadIdx.x) + u * THREADS) * V; }
    __device__ __forceinline__ bool on(int u) const { return at(u) < D; }     // V divides D
    // A row as it is stored, so that it can be on its way while another is worked on.
    template <typename T>
    __device__ __forceinline__ void fetch(const T* row, Pack<T, V>* q) const {
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            q[u] = Pack<T, V>{};
            if (on(u)) q[u] = *reinterpret_cast<const Pack<T, V>*>(row + at(u));
        }
    }
    template <typename T>
    __device__ __forceinline__ static void widen(const Pack<T, V>* q, float (*v)[V]) {
        each([&](int u, int i) { v[u][i] = to_f32(q[u].v[i]); });
    }
    template <typename T>
    __device__ __forceinline__ void load(const T* row, float (*v)[V]) const {
        Pack<T, V> q[NU];
        fetch(row, q);
        widen(q, v);
    }
    template <typename T>
    __device__ __forceinline__ void store(T* row, const float (*v)[V]) const {
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            Pack<T, V> q;
#pragma unroll
            for (int i = 0; i < V; ++i) q.v[i] = from_f32<T>(v[u][i]);
            if (on(u)) *reinterpret_cast<Pack<T, V>*>(row + at(u)) = q;
        }
    }
    // f(u, i) for all values of the lane.
    template <typename F>
    __device__ __forceinline__ static void each(F f) {
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
            for (int i = 0; i < V; ++i) f(u, i);
    }
};

__device__ __forceinline__ const char* row_of(const pn_tokens& x, int64_t b, int64_t t, int elem) {
    return static_cast<const char*>(x.p) + (b * x.sb + t * x.st) * elem;
}
template <typename T>
__device__ __forceinline__ const T* row_of(const pn_tokens& x, int64_t b, int64_t t) {
    return reinterpret_cast<const T*>(row_of(x, b, t, sizeof(T)));
}

template <typename T, typename R, int V, int NU, int THREADS>
__global__ __launch_bounds__(THREADS) void block_norm(pn_block_norm_args a) {
    __shared__ float lds[2 * (THREADS / 64)];
    const int64_t row = block_id();
    if (row >= a.B * a.T) return;
    const int64_t b = row / a.T, t = row - b * a.T;
    const Row<V, NU, THREADS> r{static_cast<int>(a.D)};
    const float eps = static_cast<float>(a.eps), inv = 1.0f / static_cast<float>(a.D);
    float x[NU][V], s[NU][V];
    r.load(row_of<T>(a.x, b, t), x);
    if (a.residual.p) {
        r.load(row_of<R>(a.residual, b, t), s);
    } else {
        r.each([&](int u, int i) { s[u][i] = 0.0f; });
    }
    if (a.gate.p) {
        float g[NU][V];
        r.load(row_of<T>(a.gate, b, t), g);
        r.each([&](int u, int i) { x[u][i] *= g[u][i] * logistic(g[u][i]); });
    }
    float unused = 0.0f;
    if (a.post_weight) {
        float w[NU][V], ss = 0.0f;
        r.load(a.post_weight, w);
        r.each([&](int u, int i) { ss = fmaf(x[u][i], x[u][i], ss); });
        row_sums<THREADS>(ss, unused, lds);
        const float ru = 1.0f / sqrtf(fmaf(ss, inv, eps));
        r.each([&](int u, int i) { x[u][i] = x[u][i] * ru * w[u][i]; });
    }
    if (a.scale) {
        float w[NU][V];
        r.load(a.scale, w);
        r.each([&](int u, int i) { s[u][i] = fmaf(w[u][i], x[u][i], s[u][i]); });
    } else {
        r.each([&](int u, int i) { s[u][i] += x[u][i]; });
    }
    r.store(static_cast<R*>(a.s) + row * a.D, s);
    if (!a.weight) return;
    float w[NU][V], ss = 0.0f;
    r.load(a.weight, w);
    r.each([&](int u, int i) { ss = fmaf(s[u][i], s[u][i], ss); });
    row_sums<THREADS>(ss, unused, lds);
    const float rs = 1.0f / sqrtf(fmaf(ss, inv, eps));
    r.each([&](int u, int i) { s[u][i] = s[u][i] * rs * w[u][i]; });
    r.store(static_cast<T*>(a.y) + row * a.D, s);
}

// A workgroup takes `rows` rows one after the other; each lane keeps the sums
// of its channels' weight gradients, which go to part[workgroup][3][D].  The
// weights wait in LDS, so that the next row can be on its way in registers
// (not beside 16 values a lane).
template <typename T, typename R, int V, int NU, int THREADS>
__global__ __launch_bounds__(THREADS) __attribute__((amdgpu_waves_per_eu(THREADS > 256 || V * NU > 8 ? 2 : 3)))
void block_norm_backward(pn_block_norm_args a, int64_t rows, int64_t n_wg, float* part) {
    __shared__ float lds[2 * (THREADS / 64)];
    extern __shared__ __align__(32) float weights[];     // [3][D]: weight, post_weight, scale
    const int64_t wg = block_id();
    if (wg >= n_wg) return;
    const Row<V, NU, THREADS> r{static_cast<int>(a.D)};
    const float eps = static_cast<float>(a.eps), inv = 1.0f / static_cast<float>(a.D);
    float dw[NU][V], tn[NU][V];                          // sums of dy m and of t n (t u without post_weight)
    {
        float v[NU][V];                                  // a lane reads what it wrote itself
        r.each([&](int u, int i) {
            dw[u][i] = tn[u][i] = 0.0f;
            v[u][i] = 1.0f;
        });
        if (a.weight) r.load(a.weight, v);
        r.store(weights, v);
        r.each([&](int u, int i) { v[u][i] = 1.0f; });
        if (a.scale) r.load(a.scale, v);
        r.store(weights + 2 * a.D, v);
        r.each([&](int u, int i) { v[u][i] = 1.0f; });
        if (a.post_weight) r.load(a.post_weight, v);
        r.store(weights + a.D, v);
    }
    Pack<T, V> px[NU] = {}, pg[NU] = {}, pe[NU] = {};
    Pack<R, V> ps[NU] = {}, pt[NU] = {};
    auto fetch_first = [&](int64_t row) {
        const int64_t b = row / a.T, tok = row - b * a.T;
        r.fetch(row_of<T>(a.x, b, tok), px);
        if (a.gate.p) r.fetch(row_of<T>(a.gate, b, tok), pg);
        if (a.residual.p) r.fetch(row_of<R>(a.residual, b, tok), ps);
    };
    auto fetch_last = [&](int64_t row) {
        const int64_t b = row / a.T, tok = row - b * a.T;
        if (a.weight) r.fetch(row_of<T>(a.dy, b, tok), pe);
        if (a.ds.p) r.fetch(row_of<R>(a.ds, b, tok), pt);
    };
    const int64_t end = min((wg + 1) * rows, a.B * a.T);
    constexpr bool AHEAD = V * NU < 16;
    if (AHEAD) {
        fetch_first(wg * rows);
        fetch_last(wg * rows);
    }
    for (int64_t row = wg * rows; row < end; ++row) {
        float t[NU][V], x[NU][V], g[NU][V], s[NU][V], e[NU][V], act[NU][V], w[NU][V], sc[NU][V];
        if (!AHEAD) fetch_first(row);
        r.widen(px, x);
        r.widen(pg, g);
        r.widen(ps, s);
        if (AHEAD) {
            r.widen(pt, t);
            r.widen(pe, e);
            if (row + 1 < end) {
                fetch_first(row + 1);
                fetch_last(row + 1);
            }
        } else {
            fetch_last(row);
        }
        // the forward: act is the gate's sigmoid, which is multiplied with before the gate: 0 for a gate of the
        // type's lowest value, whose product with x or a gradient may be past float32
        r.each([&](int u, int i) { act[u][i] = a.gate.p ? logistic(g[u][i]) : 1.0f; });
        auto block = [&](int u, int i) { return a.gate.p ? x[u][i] * act[u][i] * g[u][i] : x[u][i]; };
        float ru = 1.0f, uu = 0.0f, unused = 0.0f;
        if (a.post_weight) {
            r.each([&](int u, int i) { uu = fmaf(block(u, i), block(u, i), uu); });
            row_sums<THREADS>(uu, unused, lds);
            ru = 1.0f / sqrtf(fmaf(uu, inv, eps));
        }
        if (!AHEAD) {
            r.widen(pt, t);
            r.widen(pe, e);
        }
        if (a.weight) {
            float ss = 0.0f, es = 0.0f;
            r.load(weights + a.D, w);
            r.load(weights + 2 * a.D, sc);
            r.each([&](int u, int i) { s[u][i] = fmaf(sc[u][i], block(u, i) * ru * w[u][i], s[u][i]); });
            r.load(weights, w);
            r.each([&](int u, int i) {
                w[u][i] *= e[u][i];
                ss = fmaf(s[u][i], s[u][i], ss);
                es = fmaf(w[u][i], s[u][i], es);
            });
            row_sums<THREADS>(ss, es, lds);
            const float rs = 1.0f / sqrtf(fmaf(ss, inv, eps)), mean = rs > 0.0f ? es * rs * inv : 0.0f;
            r.each([&](int u, int i) {
                const float m = s[u][i] * rs;
                dw[u][i] = fmaf(e[u][i], m, dw[u][i]);
                t[u][i] = fmaf(rs, fmaf(-m, mean, w[u][i]), t[u][i]);
            });
        }
        if (a.dresidual) r.store(static_cast<R*>(a.dresidual) + row * a.D, t);
        if (a.post_weight) {
            float qu = 0.0f;
            r.load(weights + a.D, w);
            r.load(weights + 2 * a.D, sc);
            r.each([&](int u, int i) {
                w[u][i] *= sc[u][i] * t[u][i];
                qu = fmaf(w[u][i], block(u, i), qu);
            });
            row_sums<THREADS>(qu, unused, lds);
            const float mean = ru > 0.0f ? qu * ru * inv : 0.0f;
            r.each([&](int u, int i) {
                const float n = block(u, i) * ru;
                tn[u][i] = fmaf(t[u][i], n, tn[u][i]);
                t[u][i] = ru * fmaf(-n, mean, w[u][i]);
            });
        } else if (a.scale) {
            r.load(weights + 2 * a.D, sc);
            r.each([&](int u, int i) {
                tn[u][i] = fmaf(t[u][i], block(u, i), tn[u][i]);
                t[u][i] *= sc[u][i];
            });
        }
        if (a.gate.p) {
            r.each([&](int u, int i) {                   // x: dgate, t: dx
                const float p = act[u][i], du = t[u][i] * p;
                x[u][i] = du * x[u][i] * fmaf(g[u][i], 1.0f - p, 1.0f);
                t[u][i] = du * g[u][i];
            });
            r.store(static_cast<T*>(a.dgate) + row * a.D, x);
        }
        r.store(static_cast<T*>(a.dx) + row * a.D, t);
    }
    float* q = part + wg * 3 * a.D;
    if (a.weight) r.store(q, dw);
    float v[NU][V];
    if (a.post_weight) {                                 // dpw = scale sum t n
        r.load(weights + 2 * a.D, v);
        r.each([&](int u, int i) { v[u][i] *= tn[u][i]; });
        r.store(q + a.D, v);
    }
    if (a.scale) {                                       // dscale = pw sum t n
        r.each([&](int u, int i) { v[u][i] = 1.0f; });
        if (a.post_weight) r.load(weights + a.D, v);
        r.each([&](int u, int i) { v[u][i] *= tn[u][i]; });
        r.store(q + 2 * a.D, v);
    }
}

// ---------------------------------------------------------------- choice of the form

template <int V_, int NU_, int THREADS_>
struct Form {
    static constexpr int V = V_, NU = NU_, THREADS = THREADS_;
};

// The widest access that every row of the call allows.
template <typename T, typename R>
int widest(const pn_block_norm_args& a, bool backward) {
    auto bits = [&](const pn_tokens& x, int64_t elem) {
        return x.p ? reinterpret_cast<intptr_t>(x.p) | (a.B > 1 ? x.sb * elem : 0) | (a.T > 1 ? x.st * elem : 0) : 0;
    };
    auto ptr = [](const void* p) { return reinterpret_cast<intptr_t>(p); };
    int64_t t = bits(a.x, sizeof(T)) | bits(a.gate, sizeof(T)), r = 0;
    if (backward) {
        t |= (a.weight ? bits(a.dy, sizeof(T)) : 0) | ptr(a.dx) | (a.gate.p ? ptr(a.dgate) : 0);
        r |= bits(a.ds, sizeof(R)) | bits(a.residual, sizeof(R)) | ptr(a.dresidual);
    } else {
        t |= a.weight ? ptr(a.y) : 0;
        r |= bits(a.residual, sizeof(R)) | ptr(a.s);
    }
    const int64_t f = ptr(a.weight) | ptr(a.post_weight) | ptr(a.scale);
    for (int V : {static_cast<int>(16 / sizeof(T)), 2}) {
        // (a pack of more than 16 bytes is aligned to its size here, and moved in pieces)
        if (a.D % V == 0 && t % (V * static_cast<int64_t>(sizeof(T))) == 0 && r % (V * static_cast<int64_t>(sizeof(R))) == 0 &&
            f % (V * 4) == 0)
            return V;
    }
    return 1;
}

// f(form) for rows of D channels, V at a time: the fewest waves that hold a
// row in 8 values a lane (16 past 4096 channels), or ten in units of one or two
// channels, where rows of 2049 to 2560 would leave half of twice the waves idle
// (32768 rows in bfloat16 in 256 and in 512 threads, forward and gradients:
// 2050 channels in pairs 233 and 281, 283 and 499 us; 2304 in pairs 245 and 300,
// 289 and 498; 2559 one by one 383 and 421, 360 and 591; 2560 in pairs 255 and
// 310, 298 and 500).  In units of 16 bytes, 512 threads: 2304 channels 186 and
// 462, 2560 191 and 463; ten values are no whole number of such units.  With 16
// values the gradients have no registers for the next row (2050 channels in
// pairs, float32 residual, 8188 rows: 217 us).
template <int V, typename F>
hipError_t with_threads(int64_t D, F f) {
    constexpr int NU = 8 / V;
    if (D <= 512) return f(Form<V, NU, 64>{});
    if (D <= 1024) return f(Form<V, NU, 128>{});
    if (D <= 2048) return f(Form<V, NU, 256>{});
    if constexpr (V <= 2)
        if (D <= 2560) return f(Form<V, 10 / V, 256>{});
    if (D <= 4096) return f(Form<V, NU, 512>{});
    return f(Form<V, 2 * NU, 512>{});
}

template <typename T, typename R, typename F>
hipError_t with_form(const pn_block_norm_args& a, int V, F f) {
    constexpr int W = 16 / sizeof(T);
    if (V == W) return with_threads<W>(a.D, f);
    if (V == 2) return with_threads<2>(a.D, f);
    return with_threads<1>(a.D, f);
}

template <typename T, typename R>
hipError_t forward_typed(const pn_block_norm_args& a, hipStream_t st) {
    const int64_t rows = a.B * a.T;
    return with_form<T, R>(a, widest<T, R>(a, false), [&](auto form) {
        using Fm = decltype(form);
        block_norm<T, R, Fm::V, Fm::NU, Fm::THREADS><<<grid_of(rows, Fm::THREADS), Fm::THREADS, 0, st>>>(a);
        return hipGetLastError();
    });
}

// Rows of a workgroup of the gradients: as many workgroups as run at once (12
// waves a unit up to 2048 channels, 8 in the larger forms), or a multiple of
// them (of 2049 to 2560 channels in units of 16 bytes, whose workgroup has 8
// waves and not 4, always: the split is one of sizes alone; that form takes 462
// us where half as many workgroups take 458, 32768 rows of 2304).  A lane adds the weights' gradients of at most 128 rows in float32, the
// rest of the sum is column_sum's in float64.
void backward_split(const pn_block_norm_args& a, int64_t* rows, int64_t* n_wg) {
    const int64_t n = a.B * a.T;
    const int64_t at_once = 256 * (a.D <= 512 ? 12 : a.D <= 1024 ? 6 : a.D <= 2048 ? 3 : a.D <= 2560 ? 2 : 1);
    const int64_t wgs = at_once * std::max<int64_t>(1, (n + 128 * at_once - 1) / (128 * at_once));
    *rows = std::max<int64_t>(1, (n + wgs - 1) / wgs);
    *n_wg = (n + *rows - 1) / *rows;
}

template <typename T, typename R>
hipError_t backward_typed(const pn_block_norm_args& a, hipStream_t st) {
    int64_t rows, n_wg;
    backward_split(a, &rows, &n_wg);
    float* part = static_cast<float*>(a.workspace);
    const hipError_t e = with_form<T, R>(a, widest<T, R>(a, true), [&](auto form) {
        using Fm = decltype(form);
        const auto kernel = block_norm_backward<T, R, Fm::V, Fm::NU, Fm::THREADS>;
        const int lds = static_cast<int>(12 * a.D);
        if (lds > 48 * 1024) {
            const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
            if (e != hipSuccess) return e;
        }
        kernel<<<grid_of(n_wg, Fm::THREADS), Fm::THREADS, lds, st>>>(a, rows, n_wg, part);
        return hipGetLastError();
    });
    float *dw = a.weight ? a.dweight : nullptr, *dpw = a.post_weight ? a.dpost_weight : nullptr, *dsc = a.scale ? a.dscale : nullptr;
    if (e != hipSuccess || (!dw && !dpw && !dsc)) return e;
    return launch_column_sum(ColumnSum{part, n_wg, 3 * a.D, 3, {0, a.D, 2 * a.D}, {dw, dpw, dsc}}, st);
}

}  // namespace

hipError_t launch_block_norm(const pn_block_norm_args& a, hipStream_t st) {
    if (a.dtype == PN_F32) return forward_typed<float, float>(a, st);
    if (a.dtype == PN_BF16)
        return a.residual_dtype == PN_F32 ? forward_typed<bf16, float>(a, st) : forward_typed<bf16, bf16>(a, st);
    return a.residual_dtype == PN_F32 ? forward_typed<f16, float>(a, st) : forward_typed<f16, f16>(a, st);
}

size_t block_norm_workspace(const pn_block_norm_args& a) {
    if (!a.weight && !a.post_weight && !a.scale) return 0;
    int64_t rows, n_wg;
    backward_split(a, &rows, &n_wg);
    return sizeof(float) * static_cast<size_t>(n_wg) * 3 * static_cast<size_t>(a.D);
}

hipError_t launch_block_norm_backward(const pn_block_norm_args& a, hipStream_t st) {
    if (a.dtype == PN_F32) return backward_typed<float, float>(a, st);
    if (a.dtype == PN_BF16)
        return a.residual_dtype == PN_F32 ? backward_typed<bf16, float>(a, st) : backward_typed<bf16, bf16>(a, st);
    return a.residual_dtype == PN_F32 ? backward_typed<f16, float>(a, st) : backward_typed<f16, f16>(a, st);
}

}  // namespace pn
