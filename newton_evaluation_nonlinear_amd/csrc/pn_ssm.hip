// The selective scan's plan, launches and sums, and its single-token form.
//
// Single tokens: bound by the states' bytes, 8 N per channel.  A group of lanes
// holds a channel, V adjacent states a lane.  256 sequences of 4096 channels of
// 16 states (143 MB) in 32 us, 4.5 TB/s, nearly the rate of a large copy.

#include <algorithm>
#include <cmath>

#include "pn_ssm.hpp"
#include "pn_ssm_device.hpp"

namespace pn {
namespace {

// 16 rows of lanes per 64 columns, added in order in float64.
__global__ __launch_bounds__(1024) void column_sum(ColumnSum a) {
    __shared__ double red[16][65];
    const int col = threadIdx.x % 64, lane = threadIdx.x / 64;
    const int64_t c = static_cast<int64_t>(block_id()) * 64 + col;
    double s = 0.0;
    if (c < a.cols)
        for (int64_t r0 = lane; r0 < a.rows; r0 += 16 * 16) {
            float x[16];                                 // 16 loads in flight, added in order
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = a.in[min(r0 + 16 * i, a.rows - 1) * a.cols + c];
#pragma unroll
            for (int i = 0; i < 16; ++i) s += r0 + 16 * i < a.rows ? x[i] : 0.0f;
        }
    red[lane][col] = s;
    __syncthreads();
    if (lane != 0 || c >= a.cols) return;
    double v = 0.0;
    for (int i = 0; i < 16; ++i) v += red[i][col];
    int part = 0;
#pragma unroll
    for (int i = 1; i < 4; ++i)
        if (i < a.n_parts && c >= a.from[i]) part = i;
    float* out = a.out[part];
    if (out) out[c - a.from[part]] = static_cast<float>(v);
}

// db and dc: the sums of the workgroups' shares [workgroup][b, t][2][NP].
template <typename T>
__global__ __launch_bounds__(256) void bc_sum(pn_ssm_args a, SsmPlan p, const float* part) {
    const int64_t N = a.N, GN = a.G * N, rows = a.B * a.T, NP = static_cast<int64_t>(p.blocks) * p.states;
    const int64_t i = static_cast<int64_t>(block_id()) * 256 + threadIdx.x;
    if (i >= rows * 2 * GN) return;
    const int64_t row = i / (2 * GN), o = i - row * 2 * GN, which = o / GN, gn = o - which * GN, g = gn / N;
    const int64_t b = row / a.T;
    float v = 0.0f;
    if (!a.lengths || row - b * a.T < a.lengths[b]) {
        const int per = p.per_group / p.wide;
        const float* q = part + ((g * per * rows + row) * 2 + which) * NP + (gn - g * N);
        for (int k = 0; k < per; ++k) v += q[k * rows * 2 * NP];
    }
    static_cast<T*>(which ? a.dc : a.db)[row * GN + gn] = from_f32<T>(v);
}

// L lanes per channel, NU units of V states each; b and c are read W at a time.
template <typename T, int V, int NU, int W>
__global__ __launch_bounds__(256) void ssm_step(pn_ssm_step_args a, int L) {
    const int64_t g = static_cast<int64_t>(block_id()) * (256 / L) + threadIdx.x / L;
    const int lane = threadIdx.x & (L - 1);
    if (g >= a.B * a.D) return;
    const int64_t b = g / a.D;
    const int d = static_cast<int>(g - b * a.D), N = static_cast<int>(a.N);
    const int64_t slot = a.slots ? a.slots[b] : b;
    T* y = static_cast<T*>(a.y) + g;
    if (slot < 0 || slot >= a.n_slots) {
        if (lane == 0) *y = from_f32<T>(0.0f);
        return;
    }
    float* hp = a.state + (slot * a.D + d) * N;
    const float* Ap = a.A + static_cast<int64_t>(d) * N;
    Pack<float, V> h[NU], A[NU];
    Pack<T, V> bv[NU], cv[NU];
    const int group = d / static_cast<int>(a.D / a.G);
    const T* bp = static_cast<const T*>(a.b.p) + b * a.b.sb + group * a.b.sh;
    const T* cp = static_cast<const T*>(a.c.p) + b * a.c.sb + group * a.c.sh;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
        const int n = (lane + u * L) * V;                // V divides N
        h[u] = A[u] = Pack<float, V>{};
        bv[u] = cv[u] = Pack<T, V>{};
        if (n < N) {
            h[u] = *reinterpret_cast<const Pack<float, V>*>(hp + n);
            A[u] = *reinterpret_cast<const Pack<float, V>*>(Ap + n);
#pragma unroll
            for (int i = 0; i < V / W; ++i) {
                *reinterpret_cast<Pack<T, W>*>(bv[u].v + i * W) = *reinterpret_cast<const Pack<T, W>*>(bp + n + i * W);
                *reinterpret_cast<Pack<T, W>*>(cv[u].v + i * W) = *reinterpret_cast<const Pack<T, W>*>(cp + n + i * W);
            }
        }
    }
    const float x = to_f32(static_cast<const T*>(a.x.p)[b * a.x.sb + d]);
    const float raw = to_f32(static_cast<const T*>(a.dt.p)[b * a.dt.sb + d]) + (a.dt_bias ? a.dt_bias[d] : 0.0f);
    float slope;
    const float delta = a.softplus ? softplus(raw, &slope) : raw;
    const float ux = delta * x;
    float acc = 0.0f;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
        const int n = (lane + u * L) * V;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            h[u].v[i] = fmaf(__builtin_amdgcn_exp2f(delta * kLog2e * A[u].v[i]), h[u].v[i], ux * to_f32(bv[u].v[i]));
            acc = fmaf(to_f32(cv[u].v[i]), h[u].v[i], acc);
        }
        if (n < N) *reinterpret_cast<Pack<float, V>*>(hp + n) = h[u];
    }
    for (int m = 1; m < L; m <<= 1) acc += __shfl_xor(acc, m);
    if (lane != 0) return;
    if (a.skip) acc = fmaf(a.skip[d], x, acc);
    if (a.gate.p) {
        const float z = to_f32(static_cast<const T*>(a.gate.p)[b * a.gate.sb + d]);
        acc *= z * logistic(z);
    }
    *y = from_f32<T>(acc);
}

template <typename T>
hipError_t step_typed(const pn_ssm_step_args& a, hipStream_t st) {
    const bool wide = a.N % 4 == 0 && (reinterpret_cast<uintptr_t>(a.state) | reinterpret_cast<uintptr_t>(a.A)) % 16 == 0;
    const int units = static_cast<int>(wide ? a.N / 4 : a.N);
    int L = 1;
    while (L < units && L < 64) L *= 2;
    const int64_t per = 256 / L;
    const dim3 grid = grid_of((a.B * a.D + per - 1) / per, 256);
    const int64_t bc = reinterpret_cast<intptr_t>(a.b.p) | reinterpret_cast<intptr_t>(a.c.p) |
                       ((a.B > 1 ? a.b.sb | a.c.sb : 0) | (a.G > 1 ? a.b.sh | a.c.sh : 0)) * static_cast<int64_t>(sizeof(T));
    if (wide && bc % (4 * sizeof(T)) == 0) ssm_step<T, 4, 1, 4><<<grid, 256, 0, st>>>(a, L);
    else if (wide) ssm_step<T, 4, 1, 1><<<grid, 256, 0, st>>>(a, L);
    else if (units <= 64) ssm_step<T, 1, 1, 1><<<grid, 256, 0, st>>>(a, L);
    else ssm_step<T, 1, 2, 1><<<grid, 256, 0, st>>>(a, L);
    return hipGetLastError();
}

hipError_t pass(const pn_ssm_args& a, const SsmPlan& p, SsmPass which, hipStream_t st) {
    switch (a.dtype) {
        case PN_F32: return launch_ssm_pass<float>(a, p, which, st);
        case PN_BF16: return launch_ssm_pass<bf16>(a, p, which, st);
        default: return launch_ssm_pass<f16>(a, p, which, st);
    }
}

}  // namespace

// Segments of 32 tokens or more: 6144 waves, six for every SIMD, of which the
// oldest run first and the others fill their waits (65536 tokens of 2048
// channels in 2048, 4096, 6144 and 12288 waves: 1461, 1416, 1267 and 1334 us).
// Two sweeps then take the place of one, so two segments gain nothing, and from
// 2048 waves on one is enough (2048 tokens of 16 states, microseconds in one and
// in several: 1536 waves 673 and 655, with gradients 3212 and 2735; 2048 waves
// 688 and 861, 3479 and 3624).  Up to a wave for every SIMD a call takes as long
// as one wave's tokens, and segments may be shorter, 16 tokens and in the
// gradients 8 (2048 channels of 16 states, 32 and less: 64 tokens 16.4 and
// 15.1 us, with gradients 84.5 and 46.1; 256 tokens 19.1 and 15.3, 76.6 and
// 65.1).  With 2048 such waves in place of 1024 nothing is gained (512 tokens:
// 21.5 and 24.1, 84.1 and 86.1), and below 64 tokens one sweep is as fast.  A
// segment goes over the ends of those before it, so there are at most 64 or
// the root of the tokens (256 channels, 65536 tokens in 768 and 256: 351 and
// 182 us, with gradients 1174 and 638; 1024 channels, 4096 tokens in 128 and 64:
// 74 and 55, 237 and 178; half and three halves as many are slower).
SsmPlan plan_ssm(const pn_ssm_args& a, bool backward) {
    SsmPlan p{};
    p.states = a.N <= 4 ? 4 : a.N <= 8 ? 8 : 16;
    p.blocks = static_cast<int32_t>((a.N + 15) / 16);
    // channel blocks of a workgroup of the gradients: 4, or fewer where that
    // many leave more than an eighth of them empty
    const int64_t per_group = (a.D / a.G + 31) / 32;
    p.wide = backward && p.blocks == 1 ? 4 : 1;
    while (p.wide > 1 && ((per_group + p.wide - 1) / p.wide * p.wide - per_group) * 8 > per_group) p.wide /= 2;
    p.per_group = static_cast<int32_t>((per_group + p.wide - 1) / p.wide * p.wide);
    p.chans = static_cast<int32_t>(a.G) * p.per_group;
    const int64_t rows = a.B * p.chans, waves = rows * p.blocks;
    p.tiles = (a.T + kSsmTile - 1) / kSsmTile;
    int64_t n = std::min<int64_t>((6144 + waves - 1) / waves, a.T / 32);
    if (a.T >= (backward ? 24 : 64)) n = std::max(n, std::min<int64_t>(1024 / waves, a.T / (backward ? 8 : 16)));
    n = std::min(n, std::max<int64_t>(64, static_cast<int64_t>(std::sqrt(static_cast<double>(a.T)))));
    if (waves >= 2048 || n < 3) n = 1;
    const int64_t per = std::max<int64_t>(1, (p.tiles + n - 1) / n);
    p.seg = per * kSsmTile;
    p.n_seg = static_cast<int32_t>(std::max<int64_t>(1, (p.tiles + per - 1) / per));
    const int64_t state = rows * p.blocks * p.states * 32;
    int64_t at = 0;
    auto take = [&](int64_t floats) {
        const int64_t from = at;
        at += (floats + 63) / 64 * 64;
        return from;
    };
    if (p.n_seg > 1) {
        p.ends = take(p.n_seg * state);
        p.decay = take(p.n_seg * rows * 32);
        if (backward) p.rends = take(p.n_seg * state);
    }
    if (backward) {
        p.marks = take(p.tiles * state);
        p.since = take(p.tiles * rows * 32);
        p.part_bc = take(p.chans / p.wide * a.B * a.T * 2 * p.blocks * p.states);
        p.part_A = take(a.B * p.n_seg * a.D * a.N);
        p.part_vec = take(a.B * p.n_seg * p.blocks * 2 * a.D);
    }
    p.total = at;
    return p;
}

bool ssm_fits(const pn_ssm_args& a, const SsmPlan& p) {
    const int64_t limit = (int64_t(1) << 31) - 1, rows = a.B * p.chans * p.n_seg;
    return rows <= limit && a.B * a.T <= limit * 64 / (a.G * a.N);
}

hipError_t launch_column_sum(const ColumnSum& s, hipStream_t st) {
    if (s.cols <= 0) return hipSuccess;
    column_sum<<<grid_of((s.cols + 63) / 64, 1024), 1024, 0, st>>>(s);
    return hipGetLastError();
}

hipError_t launch_ssm(const pn_ssm_args& a, const SsmPlan& p, hipStream_t st) {
    if (p.n_seg > 1) {
        const hipError_t e = pass(a, p, kSsmEnds, st);
        if (e != hipSuccess) return e;
    }
    return pass(a, p, kSsmOutputs, st);
}

hipError_t launch_ssm_backward(const pn_ssm_args& a, const SsmPlan& p, hipStream_t st) {
    hipError_t e = a.T > 0 ? pass(a, p, p.n_seg > 1 ? kSsmMarksBoth : kSsmMarks, st) : hipSuccess;
    if (e == hipSuccess) e = pass(a, p, kSsmGradients, st);
    if (e != hipSuccess) return e;
    float* ws = static_cast<float*>(a.workspace);
    if (a.T > 0) {
        const dim3 grid = grid_of((a.B * a.T * 2 * a.G * a.N + 255) / 256, 256);
        switch (a.dtype) {
            case PN_F32: bc_sum<float><<<grid, 256, 0, st>>>(a, p, ws + p.part_bc); break;
            case PN_BF16: bc_sum<bf16><<<grid, 256, 0, st>>>(a, p, ws + p.part_bc); break;
            default: bc_sum<f16><<<grid, 256, 0, st>>>(a, p, ws + p.part_bc); break;
        }
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    e = launch_column_sum(ColumnSum{ws + p.part_A, a.B * p.n_seg, a.D * a.N, 1, {0}, {a.dA}}, st);
    if (e != hipSuccess) return e;
    float *dskip = a.skip ? a.dskip : nullptr, *dbias = a.dt_bias ? a.ddt_bias : nullptr;
    if (!dskip && !dbias) return hipSuccess;
    return launch_column_sum(ColumnSum{ws + p.part_vec, a.B * p.n_seg * p.blocks, 2 * a.D, 2, {0, a.D}, {dskip, dbias}}, st);
}

hipError_t launch_ssm_step(const pn_ssm_step_args& a, hipStream_t st) {
    switch (a.dtype) {
        case PN_F32: return step_typed<float>(a, st);
        case PN_BF16: return step_typed<bf16>(a, st);
        default: return step_typed<f16>(a, st);
    }
}

}  // namespace pn
