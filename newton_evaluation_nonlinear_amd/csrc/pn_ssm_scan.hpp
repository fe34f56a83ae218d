// The passes of the selective scan over the tokens,
//     h_t = exp(delta_t A) h_{t-1} + u_t b_t,   u = delta x,   y_t = c_t . h_t,
// and of its gradients: with r_t the gradient of h_t (r_T that of the final
// state) and g the gradient of c . h,
//     r_t = exp(delta_{t+1} A) r_{t+1} + g_t c_t,   e_t = exp(delta_t A) h_{t-1},
//     du = r . b,   ddelta = x du + sum_n r e A,   dA = sum r e delta,
//     db = sum over channels of r u,   dc = sum over channels of g h.
//
// Layout.  A wave (a workgroup of its own up to 16 states) holds 64 channels.
// In a quad of lanes each lane holds S of the 4 S states of the quad's four
// channels, in registers over all tokens: b and c are read from LDS once for
// four channels, and the sums over channels in db and dc are a fourth the
// work of lanes that hold whole channels.  What belongs to a channel and not
// to a state (step, gate, products with x) is computed by the one lane whose
// number is the channel's, so tokens move 64 adjacent elements at a time; the
// quad passes these values on by DPP, and sums of its four lanes go back to
// the channel's own lane.  More than 16 states are blocks of 16 in as many
// waves, which add their shares of such sums through LDS.
//
// Time.  Where channels do not fill the device the tokens are cut into
// segments: a first pass takes the state that a segment leaves alone
// (kSsmEnds), and a segment of the next starts from those before it, faded by
// the sum of their steps.  The gradients' first pass marks the state at every
// tile of 8 tokens (kSsmMarks) and, for segments, in the same sweep what each
// gives to the gradient before it (kSsmMarksBoth: the sum of g c times the
// decay since the segment's start); the second walks the tiles backwards,
// each once forward from its mark with e kept in registers, once back.
#pragma once

#include "pn_seq_device.hpp"
#include "pn_ssm.hpp"

namespace pn {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// A value of the quad's lane K in all four lanes.
template <int K>
__device__ __forceinline__ float quad_lane(float v) {
    int r = __builtin_amdgcn_mov_dpp(__float_as_int(v), K * 0x55, 0xf, 0xf, true);
    asm("" : "+v"(r));           // kept apart: one move and plain products take less than DPP in every product
    return __int_as_float(r);
}
__device__ __forceinline__ void quad_lanes(float v, float* k) {
    k[0] = quad_lane<0>(v);
    k[1] = quad_lane<1>(v);
    k[2] = quad_lane<2>(v);
    k[3] = quad_lane<3>(v);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
// Lane j of a quad gets the sum of the quad's p[j].
__device__ __forceinline__ float quad_sum(const float* p, int j) {
    const bool hi = j & 2, odd = j & 1;
    float a = hi ? p[2] : p[0], b = hi ? p[3] : p[1];
    a += dpp<0x4E>(hi ? p[0] : p[2]);                    // of lane j ^ 2
    b += dpp<0x4E>(hi ? p[1] : p[3]);
    return (odd ? b : a) + dpp<0xB1>(odd ? a : b);       // of lane j ^ 1
}

// Orders LDS accesses of the lanes of one wave, which runs them in order.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// log(1 + e^v) = max(v, 0) + log(1 + t), t = e^-|v|; log(1 + t) as
// log(w) t / (w - 1) with w = 1 + t rounded: the error of w cancels.
__device__ __forceinline__ float softplus(float v, float* slope) {
    const float t = __builtin_amdgcn_exp2f(-fabsf(v) * kLog2e), w = 1.0f + t;
    const float l = w == 1.0f ? t : __builtin_amdgcn_logf(w) * kLn2 * t * __builtin_amdgcn_rcpf(w - 1.0f);
    *slope = (v >= 0.0f ? 1.0f : t) * __builtin_amdgcn_rcpf(w);
    return fmaxf(v, 0.0f) + l;
}
__device__ __forceinline__ float logistic(float v) { return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-v * kLog2e)); }

// Where a wave works.
template <typename T, int S, bool MULTI>
struct SsmWave {
    static constexpr int E = 4 * S;                      // states of a quad's channel, and values of a lane
    static constexpr int M = kSsmTile * E / 64 > 0 ? kSsmTile * E / 64 : 1;
    const pn_ssm_args& a;
    const SsmPlan& p;
    int lane, j, blk, seg, cb, ch, first, n0, behind;    // n0: the lane's first state; behind: the channel after the group
    int64_t b, row, begin, stop, end;                    // row: (b, channel block); stop: of the segment, end: of its tokens
    bool own;                                            // whether the lane's channel exists
    const T *xp, *dp, *zp, *bp, *cp;

    __device__ __forceinline__ SsmWave(const pn_ssm_args& a_, const SsmPlan& p_) : a(a_), p(p_) {
        lane = threadIdx.x & 63;
        j = lane & 3;
        blk = MULTI ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
        const uint32_t id = block_id(), B = static_cast<uint32_t>(a.B), chans = static_cast<uint32_t>(p.chans);
        cb = static_cast<int>(id % chans);
        b = id / chans % B;
        seg = static_cast<int>(id / chans / B);
        row = b * chans + cb;
        const int group = cb / p.per_group, DG = static_cast<int>(a.D / a.G), in = cb % p.per_group * 64;
        first = group * DG + in;
        behind = (group + 1) * DG;
        own = in + lane < DG;
        ch = group * DG + min(in + lane, DG - 1);
        n0 = blk * E + j * S;
        begin = seg * p.seg;
        stop = min(begin + p.seg, a.T);
        int64_t len = a.T;
        if (a.lengths) len = max(static_cast<int64_t>(0), min(static_cast<int64_t>(a.lengths[b]), a.T));
        end = min(stop, len);
        xp = static_cast<const T*>(a.x.p) + b * a.x.sb;
        dp = static_cast<const T*>(a.dt.p) + b * a.dt.sb;
        zp = a.gate.p ? static_cast<const T*>(a.gate.p) + b * a.gate.sb : nullptr;
        bp = static_cast<const T*>(a.b.p) + b * a.b.sb + group * a.b.sh;
        cp = static_cast<const T*>(a.c.p) + b * a.c.sb + group * a.c.sh;
    }
    // Channel k of the lane's quad, and whether it exists.
    __device__ __forceinline__ int chan(int k) const { return first + (lane & ~3) + k; }
    __device__ __forceinline__ bool has(int k) const { return chan(k) < behind; }

    // f(k, s, index in [D, N]) for the states that exist.
    template <typename F>
    __device__ __forceinline__ void states(F f) const {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (has(k) && n0 + s < a.N) f(k, s, static_cast<int64_t>(chan(k)) * a.N + n0 + s);
    }
    __device__ __forceinline__ void decays(float (*A2)[S]) const {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int s = 0; s < S; ++s) A2[k][s] = 0.0f;
        states([&](int k, int s, int64_t i) { A2[k][s] = a.A[i] * kLog2e; });
    }
    // A state array of the workspace: [.., row, block, k, lane, s].
    __device__ __forceinline__ float* at(float* base, int64_t n) const {
        return base + (((n * a.B * p.chans + row) * p.blocks + blk) * 256 + lane) * S;
    }
    __device__ __forceinline__ void put(float* q, const float (*h)[S]) const {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            Pack<float, S> v;
#pragma unroll
            for (int s = 0; s < S; ++s) v.v[s] = h[k][s];
            *reinterpret_cast<Pack<float, S>*>(q + k * 64 * S) = v;
        }
    }
    __device__ __forceinline__ void get(const float* q, float (*h)[S]) const {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const Pack<float, S> v = *reinterpret_cast<const Pack<float, S>*>(q + k * 64 * S);
#pragma unroll
            for (int s = 0; s < S; ++s) h[k][s] = v.v[s];
        }
    }
    // h = exp(sum of steps * A) h + more
    __device__ __forceinline__ void fade(float (*h)[S], float steps, const float (*A2)[S], const float (*more)[S]) const {
        float d[4];
        quad_lanes(steps, d);
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int s = 0; s < S; ++s) h[k][s] = fmaf(__builtin_amdgcn_exp2f(d[k] * A2[k][s]), h[k][s], more[k][s]);
    }
    __device__ __forceinline__ int64_t own_at(int64_t n) const { return (n * a.B * p.chans + row) * 64 + lane; }
    // The state before segment seg > 0 from the ends of those before it.
    __device__ __forceinline__ void carried(float* ws, const float (*A2)[S], float (*h)[S]) const {
        get(at(ws + p.ends, 0), h);
        for (int i = 1; i < seg; ++i) {
            float more[4][S];
            get(at(ws + p.ends, i), more);
            fade(h, ws[p.decay + own_at(i)], A2, more);
        }
    }

    // The b and c of a tile, to LDS as [token][b | c][E].
    __device__ __forceinline__ void load_bc(const T* src, int64_t st, int64_t t0, float* v) const {
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int i = lane + 64 * m, tok = i / E, n = blk * E + i % E;
            const bool on = i < kSsmTile * E && t0 + tok < end && n < a.N;
            v[m] = on ? to_f32(src[(t0 + tok) * st + n]) : 0.0f;
        }
    }
    __device__ __forceinline__ void store_bc(float* lds, int which, const float* v) const {
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int i = lane + 64 * m;
            if (i < kSsmTile * E) lds[(i / E * 2 + which) * E + i % E] = v[m];
        }
    }
    __device__ __forceinline__ void read_bc(const float* lds, int i, int which, float* v) const {
        const Pack<float, S> q = *reinterpret_cast<const Pack<float, S>*>(lds + (i * 2 + which) * E + j * S);
#pragma unroll
        for (int s = 0; s < S; ++s) v[s] = q.v[s];
    }
    // The lane's channel of a token row; rows at and after `end` are not read.
    __device__ __forceinline__ void load_rows(const T* src, int64_t st, int64_t t0, T* v) const {
#pragma unroll
        for (int i = 0; i < kSsmTile; ++i) {
            const int64_t t = min(t0 + i, end - 1);
            v[i] = (src + t * st)[ch];
        }
    }
};

// Sums over the waves of a workgroup: wave w gets its tokens w, w + blocks, ..
template <int S, bool MULTI>
__device__ __forceinline__ float joined(const float* ex, int blocks, int i, int lane) {
    float v = 0.0f;
    for (int w = 0; w < blocks; ++w) v += ex[(w * kSsmTile + i) * 64 + lane];
    return v;
}

template <typename T, int S, bool MULTI, int PASS>
__global__ __launch_bounds__(MULTI ? 512 : 64) void ssm_pass(pn_ssm_args a, SsmPlan p) {
    constexpr int E = 4 * S, WAVES = MULTI ? 8 : 1;
    constexpr bool OUT = PASS == kSsmOutputs, MARKS = PASS == kSsmMarks || PASS == kSsmMarksBoth, BACK = PASS == kSsmMarksBoth;
    __shared__ __align__(16) float bc_lds[WAVES][kSsmTile * 2 * E];
    __shared__ float ex[MULTI && OUT ? WAVES * kSsmTile * 64 : 1];
    const SsmWave<T, S, MULTI> w(a, p);
    if (w.seg >= (PASS == kSsmEnds ? p.n_seg - 1 : p.n_seg)) return;
    float* ws = static_cast<float*>(a.workspace);
    float* lds = bc_lds[MULTI ? w.blk : 0];
    const float bias = a.dt_bias ? a.dt_bias[w.ch] : 0.0f, skip = a.skip ? a.skip[w.ch] : 0.0f;
    const T* gp = BACK ? static_cast<const T*>(a.dy.p) + w.b * a.dy.sb : nullptr;
    T* yp = static_cast<T*>(a.y);
    float A2[4][S], h[4][S], R[BACK ? 4 : 1][S], P[BACK ? 4 : 1][S];
    w.decays(A2);
    if (OUT && w.seg > 0) {
        w.carried(ws, A2, h);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int s = 0; s < S; ++s) h[k][s] = 0.0f;
        if (w.seg == 0 && a.initial_state)
            w.states([&](int k, int s, int64_t i) { h[k][s] = a.initial_state[w.b * a.D * a.N + i]; });
    }
    if (BACK) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int s = 0; s < S; ++s) {
                R[k][s] = 0.0f;
                P[k][s] = 1.0f;
            }
    }
    float since = 0.0f;                                  // sum of the lane's steps
    constexpr bool C = OUT || BACK, Z = OUT || BACK;
    T x[kSsmTile], dt[kSsmTile], z[kSsmTile], gy[kSsmTile];
    float bv[w.M], cv[w.M];
    auto load = [&](int64_t t0) {
        w.load_rows(w.xp, a.x.st, t0, x);
        w.load_rows(w.dp, a.dt.st, t0, dt);
        if (Z && w.zp) w.load_rows(w.zp, a.gate.st, t0, z);
        if (BACK) w.load_rows(gp, a.dy.st, t0, gy);
        w.load_bc(w.bp, a.b.st, t0, bv);
        if (C) w.load_bc(w.cp, a.c.st, t0, cv);
    };
    if (w.begin < w.end) load(w.begin);
    for (int64_t t0 = w.begin; t0 < w.end; t0 += kSsmTile) {
        float dl[kSsmTile], xs[kSsmTile], g[kSsmTile];
#pragma unroll
        for (int i = 0; i < kSsmTile; ++i) {
            const bool on = t0 + i < w.end;
            const float raw = to_f32(dt[i]) + bias;
            float slope;
            dl[i] = on ? (a.softplus ? softplus(raw, &slope) : raw) : 0.0f;
            xs[i] = on ? to_f32(x[i]) : 0.0f;
            if (Z) {
                const float zf = w.zp ? to_f32(z[i]) : 0.0f;
                g[i] = w.zp ? zf * logistic(zf) : 1.0f;
                if (BACK) g[i] = on ? g[i] * to_f32(gy[i]) : 0.0f;
            }
        }
        wave_sync();
        w.store_bc(lds, 0, bv);
        if (C) w.store_bc(lds, 1, cv);
        wave_sync();
        if (t0 + kSsmTile < w.end) load(t0 + kSsmTile);
        if (MARKS) {
            w.put(w.at(ws + p.marks, t0 / kSsmTile), h);
            if (!MULTI || w.blk == 0) ws[p.since + w.own_at(t0 / kSsmTile)] = since;
        }
#pragma unroll
        for (int i = 0; i < kSsmTile; ++i) {
            float bi[S], ci[S], d[4], u[4], gk[4], part[4];
            w.read_bc(lds, i, 0, bi);
            if (C) w.read_bc(lds, i, 1, ci);
            quad_lanes(dl[i], d);
            quad_lanes(dl[i] * xs[i], u);
            if (BACK) quad_lanes(g[i], gk);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                part[k] = 0.0f;
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    const float f = __builtin_amdgcn_exp2f(d[k] * A2[k][s]);
                    h[k][s] = fmaf(u[k], bi[s], f * h[k][s]);
                    if (OUT) part[k] = fmaf(ci[s], h[k][s], part[k]);
                    if (BACK) {
                        P[k][s] *= f;
                        R[k][s] = fmaf(P[k][s], ci[s] * gk[k], R[k][s]);
                    }
                }
            }
            since += dl[i];
            if (OUT) {
                float y = quad_sum(part, w.j);
                if (MULTI) {
                    ex[(w.blk * kSsmTile + i) * 64 + w.lane] = y;
                } else if (t0 + i < w.end && w.own) {
                    y = (y + skip * xs[i]) * g[i];
                    yp[(w.b * a.T + t0 + i) * a.D + w.ch] = from_f32<T>(y);
                }
            }
        }
        if (OUT && MULTI) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kSsmTile; ++i)
                if (i % p.blocks == w.blk && t0 + i < w.end && w.own) {
                    const float y = joined<S, MULTI>(ex, p.blocks, i, w.lane);
                    yp[(w.b * a.T + t0 + i) * a.D + w.ch] = from_f32<T>((y + skip * xs[i]) * g[i]);
                }
            __syncthreads();
        }
    }
    if (OUT) {
        for (int64_t t = max(w.end, w.begin) + w.blk; t < w.stop; t += p.blocks)
            if (w.own) yp[(w.b * a.T + t) * a.D + w.ch] = from_f32<T>(0.0f);
        if (w.seg == p.n_seg - 1 && a.final_state)
            w.states([&](int k, int s, int64_t i) { a.final_state[w.b * a.D * a.N + i] = h[k][s]; });
        return;
    }
    if (p.n_seg > 1) {
        w.put(w.at(ws + p.ends, w.seg), h);
        if (!MULTI || w.blk == 0) ws[p.decay + w.own_at(w.seg)] = since;
        if (BACK) w.put(w.at(ws + p.rends, w.seg), R);
    }
}

// Sum over the 16 quads of a wave of V values a lane (2 S: those of b, then
// those of c), V a power of two; afterwards the value number of() is in the
// lanes with writes().
template <int S>
struct ChannelSum {
    // lanes that end with a value: bit 5 tells b from c, the next ones the state
    __device__ __forceinline__ static int of(int lane) {
        return (lane >> 5) * S + (S == 4 ? (lane >> 3) & 3 : S == 2 ? (lane >> 4) & 1 : 0);
    }
    __device__ __forceinline__ static bool writes(int lane) {
        return S == 4 ? !(lane & 4) : S == 2 ? !(lane & 12) : !(lane & 28);
    }
    __device__ __forceinline__ static void swap32(float& x, float y) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(y), false, false);
        x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    __device__ __forceinline__ static void swap16(float& x, float y) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(y), false, false);
        x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    __device__ __forceinline__ static float sum(const float* b, const float* c, int lane) {
        float v[S];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            v[s] = b[s];
            swap32(v[s], c[s]);
        }
        if (S == 4) {
            swap16(v[0], v[2]);                          // lanes with bit 4: states 2 and 3
            swap16(v[1], v[3]);
            const bool up = lane & 8;
            v[0] = (up ? v[1] : v[0]) + dpp<0x128>(up ? v[0] : v[1]);    // of lane ^ 8
        } else if (S == 2) {
            swap16(v[0], v[1]);
            v[0] += dpp<0x128>(v[0]);
        } else {
            swap16(v[0], v[0]);
            v[0] += dpp<0x128>(v[0]);
        }
        return v[0] + dpp<0x104>(v[0]);                  // of lane + 4, where bit 2 is 0
    }
};

template <typename T, int S, bool MULTI>
__global__ __launch_bounds__(MULTI ? 512 : 64) __attribute__((amdgpu_waves_per_eu(2)))
void ssm_gradients(pn_ssm_args a, SsmPlan p) {
    constexpr int E = 4 * S, WAVES = MULTI ? 8 : 1;
    __shared__ __align__(16) float bc_lds[WAVES][kSsmTile * 2 * E];
    __shared__ float ex[3][MULTI ? WAVES * kSsmTile * 64 : 1];
    const SsmWave<T, S, MULTI> w(a, p);
    if (w.seg >= p.n_seg) return;
    float* ws = static_cast<float*>(a.workspace);
    float* lds = bc_lds[MULTI ? w.blk : 0];
    const float bias = a.dt_bias ? a.dt_bias[w.ch] : 0.0f, skip = a.skip ? a.skip[w.ch] : 0.0f;
    const T* gp = static_cast<const T*>(a.dy.p) + w.b * a.dy.sb;
    T *dxp = static_cast<T*>(a.dx), *ddp = static_cast<T*>(a.ddt), *dzp = static_cast<T*>(a.dgate);
    float A2[4][S], in[4][S], r[4][S], dA[4][S];
    w.decays(A2);
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int s = 0; s < S; ++s) in[k][s] = r[k][s] = dA[k][s] = 0.0f;
    if (w.seg > 0) w.carried(ws, A2, in);
    if (a.d_final_state)
        w.states([&](int k, int s, int64_t i) { r[k][s] = a.d_final_state[w.b * a.D * a.N + i]; });
    for (int i = p.n_seg - 1; i > w.seg; --i) {          // what the segments behind give
        float more[4][S];
        w.get(w.at(ws + p.rends, i), more);
        w.fade(r, ws[p.decay + w.own_at(i)], A2, more);
    }
    float dskip = 0.0f, dbias = 0.0f;
    const int64_t rows = w.b * a.T;
    const int NP = p.blocks * E;
    float* bc_out = ws + p.part_bc + (static_cast<int64_t>(w.cb) * a.B * a.T + rows) * 2 * NP;
    const int value = ChannelSum<S>::of(w.lane);
    const int bc_at = (value / S) * NP + w.n0 + value % S;
    const bool bc_on = ChannelSum<S>::writes(w.lane);
    for (int64_t t = max(w.end, w.begin) + w.blk; t < w.stop; t += p.blocks)
        if (w.own) {
            const int64_t o = (rows + t) * a.D + w.ch;
            dxp[o] = from_f32<T>(0.0f);
            ddp[o] = from_f32<T>(0.0f);
            if (w.zp) dzp[o] = from_f32<T>(0.0f);
        }
    for (int64_t t0 = w.begin + (w.end - 1 - w.begin) / kSsmTile * kSsmTile; w.begin < w.end && t0 >= w.begin; t0 -= kSsmTile) {
        float dl[kSsmTile], xs[kSsmTile], g[kSsmTile], slope[kSsmTile], dz[kSsmTile], e[kSsmTile][4][S], h[4][S];
        {
            T x[kSsmTile], dt[kSsmTile], z[kSsmTile], gy[kSsmTile];
            float bv[w.M], cv[w.M];
            w.load_rows(w.xp, a.x.st, t0, x);
            w.load_rows(w.dp, a.dt.st, t0, dt);
            if (w.zp) w.load_rows(w.zp, a.gate.st, t0, z);
            w.load_rows(gp, a.dy.st, t0, gy);
            w.load_bc(w.bp, a.b.st, t0, bv);
            w.load_bc(w.cp, a.c.st, t0, cv);
            w.get(w.at(ws + p.marks, t0 / kSsmTile), h);
            if (w.seg > 0) {
                float mark[4][S];
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int s = 0; s < S; ++s) {
                        mark[k][s] = h[k][s];
                        h[k][s] = in[k][s];
                    }
                w.fade(h, ws[p.since + w.own_at(t0 / kSsmTile)], A2, mark);
            }
#pragma unroll
            for (int i = 0; i < kSsmTile; ++i) {
                const bool on = t0 + i < w.end;
                const float raw = to_f32(dt[i]) + bias, dy = to_f32(gy[i]);
                float sl = 1.0f;
                const float v = a.softplus ? softplus(raw, &sl) : raw;
                dl[i] = on ? v : 0.0f;
                slope[i] = sl;
                xs[i] = on && w.own ? to_f32(x[i]) : 0.0f;
                const float zf = w.zp ? to_f32(z[i]) : 0.0f, sg = logistic(zf);
                g[i] = on && w.own ? (w.zp ? dy * zf * sg : dy) : 0.0f;
                dz[i] = dy * sg * fmaf(zf, 1.0f - sg, 1.0f);
            }
            wave_sync();
            w.store_bc(lds, 0, bv);
            w.store_bc(lds, 1, cv);
            wave_sync();
        }
#pragma unroll
        for (int i = 0; i < kSsmTile; ++i) {
            float bi[S], ci[S], d[4], u[4], part[4];
            w.read_bc(lds, i, 0, bi);
            w.read_bc(lds, i, 1, ci);
            quad_lanes(dl[i], d);
            quad_lanes(dl[i] * xs[i], u);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                part[k] = 0.0f;
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    e[i][k][s] = __builtin_amdgcn_exp2f(d[k] * A2[k][s]) * h[k][s];
                    h[k][s] = fmaf(u[k], bi[s], e[i][k][s]);
                    part[k] = fmaf(ci[s], h[k][s], part[k]);
                }
            }
            if (w.zp) {
                const float y = quad_sum(part, w.j);
                if (MULTI) ex[0][(w.blk * kSsmTile + i) * 64 + w.lane] = y;
                else if (t0 + i < w.end && w.own) dzp[(rows + t0 + i) * a.D + w.ch] = from_f32<T>(dz[i] * fmaf(skip, xs[i], y));
            }
        }
#pragma unroll
        for (int i = kSsmTile - 1; i >= 0; --i) {
            float bi[S], ci[S], d[4], u[4], gk[4], s1[4], s2[4], db[S], dc[S], gu = 0.0f;
            w.read_bc(lds, i, 0, bi);
            w.read_bc(lds, i, 1, ci);
            quad_lanes(dl[i], d);
            quad_lanes(dl[i] * xs[i], u);
            quad_lanes(g[i], gk);
#pragma unroll
            for (int s = 0; s < S; ++s) db[s] = dc[s] = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                s1[k] = s2[k] = 0.0f;
                gu = fmaf(gk[k], u[k], gu);
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    r[k][s] = fmaf(gk[k], ci[s], r[k][s]);
                    db[s] = fmaf(r[k][s], u[k], db[s]);
                    dc[s] = fmaf(gk[k], e[i][k][s], dc[s]);
                    s1[k] = fmaf(r[k][s], bi[s], s1[k]);
                    const float x = r[k][s] * e[i][k][s];
                    s2[k] = fmaf(x, A2[k][s], s2[k]);
                    dA[k][s] = fmaf(x, d[k], dA[k][s]);
                    r[k][s] *= __builtin_amdgcn_exp2f(d[k] * A2[k][s]);
                }
            }
#pragma unroll
            for (int s = 0; s < S; ++s) dc[s] = fmaf(gu, bi[s], dc[s]);      // h = e + u b
            const float sum = ChannelSum<S>::sum(db, dc, w.lane);
            if (bc_on && t0 + i < w.end) bc_out[(t0 + i) * 2 * NP + bc_at] = sum;
            const float du = quad_sum(s1, w.j), dd = quad_sum(s2, w.j) * kLn2;
            if (MULTI) {
                ex[1][(w.blk * kSsmTile + i) * 64 + w.lane] = du;
                ex[2][(w.blk * kSsmTile + i) * 64 + w.lane] = dd;
            } else if (t0 + i < w.end && w.own) {
                const int64_t o = (rows + t0 + i) * a.D + w.ch;
                const float ddt = fmaf(xs[i], du, dd) * slope[i];
                dxp[o] = from_f32<T>(fmaf(dl[i], du, skip * g[i]));
                ddp[o] = from_f32<T>(ddt);
                dskip = fmaf(g[i], xs[i], dskip);
                dbias += ddt;
            }
        }
        if (MULTI) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kSsmTile; ++i)
                if (i % p.blocks == w.blk && t0 + i < w.end && w.own) {
                    const int64_t o = (rows + t0 + i) * a.D + w.ch;
                    const float du = joined<S, MULTI>(ex[1], p.blocks, i, w.lane);
                    const float dd = joined<S, MULTI>(ex[2], p.blocks, i, w.lane);
                    const float ddt = fmaf(xs[i], du, dd) * slope[i];
                    dxp[o] = from_f32<T>(fmaf(dl[i], du, skip * g[i]));
                    ddp[o] = from_f32<T>(ddt);
                    if (w.zp) dzp[o] = from_f32<T>(dz[i] * fmaf(skip, xs[i], joined<S, MULTI>(ex[0], p.blocks, i, w.lane)));
                    dskip = fmaf(g[i], xs[i], dskip);
                    dbias += ddt;
                }
            __syncthreads();
        }
    }
    const int64_t part = w.b * p.n_seg + w.seg;
    w.states([&](int k, int s, int64_t i) { ws[p.part_A + part * a.D * a.N + i] = dA[k][s]; });
    if (w.own) {
        float* v = ws + p.part_vec + (part * p.blocks + w.blk) * 2 * a.D + w.ch;
        v[0] = dskip;
        v[a.D] = dbias;
    }
    if (w.seg == 0 && a.d_initial_state)
        w.states([&](int k, int s, int64_t i) { a.d_initial_state[w.b * a.D * a.N + i] = r[k][s]; });
}

template <typename T, int S, bool MULTI>
hipError_t ssm_launch(const pn_ssm_args& a, const SsmPlan& p, SsmPass pass, hipStream_t st) {
    const int threads = MULTI ? 64 * p.blocks : 64;
    const int64_t segs = pass == kSsmEnds ? p.n_seg - 1 : p.n_seg;
    const dim3 grid = grid_of(segs * a.B * p.chans, threads);
    switch (pass) {
        case kSsmEnds: ssm_pass<T, S, MULTI, kSsmEnds><<<grid, threads, 0, st>>>(a, p); break;
        case kSsmOutputs: ssm_pass<T, S, MULTI, kSsmOutputs><<<grid, threads, 0, st>>>(a, p); break;
        case kSsmMarks: ssm_pass<T, S, MULTI, kSsmMarks><<<grid, threads, 0, st>>>(a, p); break;
        case kSsmMarksBoth: ssm_pass<T, S, MULTI, kSsmMarksBoth><<<grid, threads, 0, st>>>(a, p); break;
        default: ssm_gradients<T, S, MULTI><<<grid, threads, 0, st>>>(a, p); break;
    }
    return hipGetLastError();
}

}  // namespace

template <typename T>
hipError_t launch_ssm_pass(const pn_ssm_args& a, const SsmPlan& p, SsmPass pass, hipStream_t st) {
    if (p.blocks > 1) return ssm_launch<T, 4, true>(a, p, pass, st);
    if (p.states == 4) return ssm_launch<T, 1, false>(a, p, pass, st);
    if (p.states == 8) return ssm_launch<T, 2, false>(a, p, pass, st);
    return ssm_launch<T, 4, false>(a, p, pass, st);
}

}  // namespace pn
