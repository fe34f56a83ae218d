// The passes of the selective scan over the tokens,
//     h_t = exp(delta_t A) h_{t-1} + u_t b_t,   u = delta x,   y_t = c_t . h_t,
// and of its gradients: with r_t the gradient of h_t (r_T that of the final
// state) and g the gradient of c . h,
//     r_t = exp(delta_{t+1} A) r_{t+1} + g_t c_t,   e_t = exp(delta_t A) h_{t-1},
//     du = r . b,   ddelta = x du + sum_n r e A,   dA = sum r e delta,
//     db = sum over channels of r u,   dc = sum over channels of g h.
//
// Layout.  A wave holds 32 channels.  In a quad of lanes each lane holds S of
// the 4 S states of the quad's two channels, in registers over all tokens.
// What belongs to a channel and not to a state (step, gate, products with x)
// is computed once, by the lane of the channel (bit 0 of its number in the
// quad) and of the token's parity (bit 1); such values pass to the quad
// through LDS, and sums over its four lanes go back by DPP to the lane they
// belong to.  More than 16 states are blocks of 16 in as many waves, which add
// their shares of such sums through LDS.
//
// Bound: instructions, of which a state and token take an exponential, three
// products and sums to move it, one for y, and nine and a second exponential
// for its gradients.  On one SIMD an exponential takes 3.5 ns, a product or sum
// of vector registers 1.1 where two waves issue them together and 2.1 alone, a
// DPP move or a product with a scalar register 1.8; eight states moved by a
// token (8 exponentials, 24 others) 64 ns, in whatever order and from one wave
// on to eight.  So a tile is kept free of branches (rows past the end and
// channels that do not exist are left to range-checked buffer accesses, values
// that are not wanted to selects), and waves are kept small: with four channels
// a quad the gradients spilled and took 2490 us where they now take 995.  The
// vector units are busy more than 90 % of the time in kSsmEnds, kSsmOutputs
// (where channels fill the device) and kSsmMarksBoth, and 80 % in the
// gradients, which hold 240 registers and run two waves on a SIMD.
//
// Measured, bfloat16, 16 states (us, medians of traced calls): 65536 tokens of
// 2048 channels: ends 424, outputs 641 (1.0 TB/s in all); 8 x 4096 tokens of
// 2048 channels: ends 195, outputs 297, marks 355, gradients 995, the sums of db
// and dc 23.  4 x 4096 tokens of 512 channels with 128 states, as many states in
// all as the second: ends 183, outputs 296, gradients 1025, sums 81.
//
// Time.  Where channels do not fill the device the tokens are cut into
// segments: a first pass takes the state that a segment leaves alone
// (kSsmEnds), and a segment of the next starts from those before it, faded by
// the sum of their steps.  The gradients' first pass marks the state at every
// tile of 8 tokens (kSsmMarks) and, for segments, in the same sweep what each
// gives to the gradient before it (kSsmMarksBoth: the sum of g c times the
// decay since the segment's start); the second walks the tiles backwards,
// each once forward from its mark with e kept in registers, once back.  Its sums
// over tokens (dA, dskip, ddt_bias) are float32 over 8 tiles and float64, in LDS,
// over the rest of the segment.  One float32 sum over the segment took 1359 us a
// call where this takes 1355 (8 x 4096 tokens of 2048 channels of 16 states), 1450
// where this takes 1480 (4 x 4096, 512, 128 states), and 16384 equal terms left it
// by up to 9e-5.
#pragma once

#include <cfloat>

#include "pn_ssm.hpp"
#include "pn_ssm_device.hpp"

namespace pn {
namespace {

// A value of the quad's lane K in all four lanes.
template <int K>
__device__ __forceinline__ float quad_lane(float v) {
    int r = __builtin_amdgcn_mov_dpp(__float_as_int(v), K * 0x55, 0xf, 0xf, true);
    asm("" : "+v"(r));           // kept apart: one move and plain products take less than DPP in every product
    return __int_as_float(r);
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

constexpr int kChans = 32;               // channels of a wave
constexpr int kOwn = kSsmTile / 2;       // tokens of a tile that belong to a lane: 2 m + its parity

// Where a wave works.  WIDE: the waves of a workgroup are adjacent channel
// blocks, otherwise the blocks of states of one.
template <typename T, int S, bool WIDE>
struct SsmWave {
    static constexpr int E = 4 * S;                      // states of a wave
    static constexpr int M = (kSsmTile * E + 63) / 64;   // values of b that a lane loads for a tile
    const pn_ssm_args& a;
    const SsmPlan& p;
    int lane, j, odd, blk, seg, cb, ch, first, n0, behind;    // n0: the lane's first state; behind: the channel after the group
    int64_t b, row, begin, stop, end, behind_tiles;      // row: (b, channel block); stop: of the segment, end: of its tokens
    bool own;                                            // whether the lane's channel exists
    const T *bp, *cp;

    __device__ __forceinline__ SsmWave(const pn_ssm_args& a_, const SsmPlan& p_) : a(a_), p(p_) {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        lane = threadIdx.x & 63;
        j = lane & 3;
        odd = j >> 1;
        blk = WIDE ? 0 : wave;
        const uint32_t id = block_id(), B = static_cast<uint32_t>(a.B);
        const uint32_t chans = static_cast<uint32_t>(WIDE ? p.chans / p.wide : p.chans);
        cb = static_cast<int>(id % chans);
        if (WIDE) cb = cb * p.wide + wave;
        b = id / chans % B;
        seg = static_cast<int>(id / chans / B);
        row = b * p.chans + cb;
        const int group = cb / p.per_group, DG = static_cast<int>(a.D / a.G), in = cb % p.per_group * kChans;
        const int mine = in + (lane >> 2) * 2 + (j & 1);
        first = group * DG + in;
        behind = (group + 1) * DG;
        own = mine < DG;
        ch = group * DG + min(mine, DG - 1);
        n0 = blk * E + j * S;
        begin = seg * p.seg;
        stop = min(begin + p.seg, a.T);
        int64_t len = a.T;
        if (a.lengths) len = max(static_cast<int64_t>(0), min(static_cast<int64_t>(__builtin_amdgcn_readfirstlane(a.lengths[b])), a.T));
        end = min(stop, len);
        behind_tiles = end > begin ? min(stop, begin + (end - begin + kSsmTile - 1) / kSsmTile * kSsmTile) : begin;
        bp = static_cast<const T*>(a.b.p) + b * a.b.sb + group * a.b.sh;
        cp = static_cast<const T*>(a.c.p) + b * a.c.sb + group * a.c.sh;
    }
    // Channel k of the lane's quad, and whether it exists.
    __device__ __forceinline__ int chan(int k) const { return first + (lane >> 2) * 2 + k; }
    __device__ __forceinline__ bool has(int k) const { return chan(k) < behind; }

    // f(k, s, index in [D, N]) for the states that exist.
    template <typename F>
    __device__ __forceinline__ void states(F f) const {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (has(k) && n0 + s < a.N) f(k, s, static_cast<int64_t>(chan(k)) * a.N + n0 + s);
    }
    // A log2(e), finite for every finite A: tokens without a step (those behind the last) multiply it with 0.
    __device__ __forceinline__ void decays(float (*A2)[S]) const {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int s = 0; s < S; ++s) A2[k][s] = 0.0f;
        states([&](int k, int s, int64_t i) {
            const float v = a.A[i] * kLog2e;
            A2[k][s] = fabsf(v) > FLT_MAX ? copysignf(FLT_MAX, v) : v;
        });
    }
    // A state array of the workspace: [.., row, block, k, lane, s].
    __device__ __forceinline__ float* at(float* base, int64_t n) const {
        return base + (((n * a.B * p.chans + row) * p.blocks + blk) * 128 + lane) * S;
    }
    __device__ __forceinline__ void put(float* q, const float (*h)[S]) const {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            Pack<float, S> v;
#pragma unroll
            for (int s = 0; s < S; ++s) v.v[s] = h[k][s];
            *reinterpret_cast<Pack<float, S>*>(q + k * 64 * S) = v;
        }
    }
    __device__ __forceinline__ void get(const float* q, float (*h)[S]) const {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const Pack<float, S> v = *reinterpret_cast<const Pack<float, S>*>(q + k * 64 * S);
#pragma unroll
            for (int s = 0; s < S; ++s) h[k][s] = v.v[s];
        }
    }
    // h = exp(sum of steps * A) h + more; steps: of the lane's channel, in its lanes of both parities
    __device__ __forceinline__ void fade(float (*h)[S], float steps, const float (*A2)[S], const float (*more)[S]) const {
        const float d[2] = {quad_lane<0>(steps), quad_lane<1>(steps)};
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int s = 0; s < S; ++s) h[k][s] = fmaf(__builtin_amdgcn_exp2f(d[k] * A2[k][s]), h[k][s], more[k][s]);
    }
    // A number of each channel of the workspace.
    __device__ __forceinline__ int64_t own_at(int64_t n) const {
        return (n * a.B * p.chans + row) * kChans + (lane >> 2) * 2 + (j & 1);
    }
    // h faded over `count` segments from first_seg on, each of which adds its
    // own end.  The loads of eight go out together: one by one, 95 segments take
    // 25 us more.
    __device__ __forceinline__ void over_segments(float* ws, int64_t ends, int first_seg, int step, int count, const float (*A2)[S],
                                                  float (*h)[S]) const {
        constexpr int TOGETHER = 8;
        for (int i = 0; i < count; i += TOGETHER) {
            float more[TOGETHER][2][S], steps[TOGETHER];
#pragma unroll
            for (int u = 0; u < TOGETHER; ++u) {         // behind the last one: the last one again, not used
                const int at_seg = first_seg + min(i + u, count - 1) * step;
                get(at(ws + ends, at_seg), more[u]);
                steps[u] = ws[p.decay + own_at(at_seg)];
            }
#pragma unroll
            for (int u = 0; u < TOGETHER; ++u)
                if (i + u < count) fade(h, steps[u], A2, more[u]);
        }
    }
    // The state before segment seg > 0 from the ends of those before it.
    __device__ __forceinline__ void carried(float* ws, const float (*A2)[S], float (*h)[S]) const {
        get(at(ws + p.ends, 0), h);
        over_segments(ws, p.ends, 1, 1, seg - 1, A2, h);
    }

    // Step and u of the lane's tokens, to LDS as [token][channel][2], and those of the quad's two channels from there.
    __device__ __forceinline__ void store_du(float* lds, int m, float d, float u) const {
        *reinterpret_cast<Pack<float, 2>*>(lds + ((2 * m + odd) * kChans + (lane >> 2) * 2 + (j & 1)) * 2) = {d, u};
    }
    __device__ __forceinline__ void read_du(const float* lds, int i, float* d, float* u) const {
        const Pack<float, 4> q = *reinterpret_cast<const Pack<float, 4>*>(lds + (i * kChans + (lane >> 2) * 2) * 2);
        d[0] = q.v[0];
        u[0] = q.v[1];
        d[1] = q.v[2];
        u[1] = q.v[3];
    }
    // Likewise g, as [token][channel].
    __device__ __forceinline__ void store_g(float* lds, int m, float g) const {
        lds[(2 * m + odd) * kChans + (lane >> 2) * 2 + (j & 1)] = g;
    }
    __device__ __forceinline__ void read_g(const float* lds, int i, float* g) const {
        const Pack<float, 2> q = *reinterpret_cast<const Pack<float, 2>*>(lds + i * kChans + (lane >> 2) * 2);
        g[0] = q.v[0];
        g[1] = q.v[1];
    }
    // Tokens of the tile at t0 that exist.
    __device__ __forceinline__ int left(int64_t t0) const { return static_cast<int>(min(end - t0, static_cast<int64_t>(kSsmTile))); }
    // `rows` rows from p, `width` elements of each: accesses behind the last
    // read 0 and write nothing (offsets within a tile are 32 bits: sizes and
    // strides are checked).
    __device__ __forceinline__ static __amdgpu_buffer_rsrc_t rows_at(const T* p, int64_t st, int rows, int width) {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(p), static_cast<short>(0),
                                                 static_cast<int>(((rows - 1) * static_cast<uint32_t>(st) + width) * sizeof(T)), 0x00020000);
    }
    // An element as it is stored, in a register of its own (kept as 16-bit
    // values the compiler packs them in pairs, which costs more than it saves).
    __device__ __forceinline__ static uint32_t read(__amdgpu_buffer_rsrc_t r, uint32_t at) {
        if constexpr (sizeof(T) == 4) return __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0);
        else return __builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0);
    }
    __device__ __forceinline__ static float widen(uint32_t v) {
        if constexpr (sizeof(T) == 4) return __uint_as_float(v);
        else if constexpr (__is_same(T, bf16)) return __uint_as_float(v << 16);
        else return to_f32(__builtin_bit_cast(T, static_cast<uint16_t>(v)));
    }
    __device__ __forceinline__ static void write(__amdgpu_buffer_rsrc_t r, uint32_t at, float v) {
        if constexpr (sizeof(T) == 4) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), r, at, 0, 0);
        else __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, from_f32<T>(v)), r, at, 0, 0);
    }
    static constexpr uint32_t kNowhere = 0x80000000u;    // behind every tile
    // The lane's tokens and channel of x.
    __device__ __forceinline__ void load_rows(const pn_tokens& x, int64_t t0, uint32_t* v) const {
        const __amdgpu_buffer_rsrc_t r = rows_at(static_cast<const T*>(x.p) + b * x.sb + t0 * x.st, x.st, left(t0), static_cast<int>(a.D));
        const uint32_t st = static_cast<uint32_t>(x.st) * sizeof(T), at = odd * st + ch * sizeof(T);
#pragma unroll
        for (int m = 0; m < kOwn; ++m) v[m] = read(r, at + 2 * m * st);
    }
    // Rows of an output [B, T, D] from t0 on, and where the lane writes.
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(void* out, int64_t t0) const {
        return rows_at(static_cast<const T*>(out) + (b * a.T + t0) * a.D, a.D,
                       static_cast<int>(min(a.T - t0, static_cast<int64_t>(kSsmTile))), static_cast<int>(a.D));
    }
    // An output that is not wanted: nothing is written.
    __device__ __forceinline__ static __amdgpu_buffer_rsrc_t no_rows() {
        return __builtin_amdgcn_make_buffer_rsrc(nullptr, static_cast<short>(0), 0, 0x00020000);
    }
    __device__ __forceinline__ uint32_t row_at(int m) const {
        const uint32_t st = static_cast<uint32_t>(a.D) * sizeof(T);
        return (own ? odd * st + ch * sizeof(T) : kNowhere) + 2 * m * st;
    }
    // The b and c of a tile, to LDS as [token][b | c][E]; 0 for states and tokens that do not exist.
    __device__ __forceinline__ void load_bc(const T* src, int64_t st, int64_t t0, uint32_t* v) const {
        const __amdgpu_buffer_rsrc_t r = rows_at(src + t0 * st, st, left(t0), static_cast<int>(a.N));
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int i = lane + 64 * m, n = blk * E + i % E;
            v[m] = read(r, n < a.N && i < kSsmTile * E ? (i / E * static_cast<uint32_t>(st) + n) * sizeof(T) : kNowhere);
        }
    }
    __device__ __forceinline__ void store_bc(float* lds, int which, const uint32_t* v) const {
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int i = lane + 64 * m;
            if (i < kSsmTile * E) lds[(i / E * 2 + which) * E + i % E] = widen(v[m]);
        }
    }
    __device__ __forceinline__ void read_bc(const float* lds, int i, int which, float* v) const {
        const Pack<float, S> q = *reinterpret_cast<const Pack<float, S>*>(lds + (i * 2 + which) * E + j * S);
#pragma unroll
        for (int s = 0; s < S; ++s) v[s] = q.v[s];
    }
};

// The sum over the waves of a workgroup of their values for a lane's token m.
__device__ __forceinline__ float joined(const float* ex, int blocks, int m, int lane) {
    float v = 0.0f;
    for (int w = 0; w < blocks; ++w) v += ex[(w * kOwn + m) * 64 + lane];
    return v;
}

// BLOCKS: the most waves that share the states of a channel.
template <typename T, int S, int BLOCKS, int PASS>
__global__ __launch_bounds__(64 * BLOCKS) __attribute__((amdgpu_waves_per_eu(4, 4)))
void ssm_pass(pn_ssm_args a, SsmPlan p) {
    constexpr int E = 4 * S, WAVES = BLOCKS;
    constexpr bool MULTI = BLOCKS > 1;
    constexpr bool OUT = PASS == kSsmOutputs, MARKS = PASS == kSsmMarks || PASS == kSsmMarksBoth, BACK = PASS == kSsmMarksBoth;
    __shared__ __align__(16) float bc_lds[WAVES][kSsmTile * 2 * E];
    __shared__ __align__(16) float du_lds[WAVES][kSsmTile * kChans * 2], g_lds[BACK ? WAVES : 1][BACK ? kSsmTile * kChans : 2];
    __shared__ float ex[MULTI && OUT ? WAVES * kOwn * 64 : 1];
    const SsmWave<T, S, false> w(a, p);
    if (w.seg >= (PASS == kSsmEnds ? p.n_seg - 1 : p.n_seg)) return;
    float* ws = static_cast<float*>(a.workspace);
    float *lds = bc_lds[MULTI ? w.blk : 0], *du_of = du_lds[MULTI ? w.blk : 0], *g_of = g_lds[MULTI && BACK ? w.blk : 0];
    const float bias = a.dt_bias ? a.dt_bias[w.ch] : 0.0f, skip = a.skip ? a.skip[w.ch] : 0.0f;
    const bool gated = a.gate.p != nullptr;
    T* yp = static_cast<T*>(a.y);
    float A2[2][S], h[2][S], R[BACK ? 2 : 1][S], P[BACK ? 2 : 1][S];
    w.decays(A2);
    if (OUT && w.seg > 0) {
        w.carried(ws, A2, h);
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int s = 0; s < S; ++s) h[k][s] = 0.0f;
        if (w.seg == 0 && a.initial_state)
            w.states([&](int k, int s, int64_t i) { h[k][s] = a.initial_state[w.b * a.D * a.N + i]; });
    }
    if (BACK) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int s = 0; s < S; ++s) {
                R[k][s] = 0.0f;
                P[k][s] = 1.0f;
            }
    }
    float since = 0.0f;                                  // sum of the channel's steps
    constexpr bool C = OUT || BACK;
    uint32_t x[kOwn], dt[kOwn], z[kOwn], gy[kOwn], bv[w.M], cv[w.M];
    auto load = [&](int64_t t0) {
        w.load_rows(a.x, t0, x);
        w.load_rows(a.dt, t0, dt);
        if (C && gated) w.load_rows(a.gate, t0, z);
        if (BACK) w.load_rows(a.dy, t0, gy);
        w.load_bc(w.bp, a.b.st, t0, bv);
        if (C) w.load_bc(w.cp, a.c.st, t0, cv);
    };
    if (w.begin < w.end) load(w.begin);
    for (int64_t t0 = w.begin; t0 < w.end; t0 += kSsmTile) {
        const int left = w.left(t0) - w.odd;             // the lane's token m exists if 2 m < left
        float dl[kOwn], xs[kOwn], g[kOwn], steps = 0.0f;
#pragma unroll
        for (int m = 0; m < kOwn; ++m) {
            const bool on = 2 * m < left;
            const float raw = w.widen(dt[m]) + bias;
            float slope;
            const float soft = pinned(softplus(raw, &slope));
            dl[m] = on ? (a.softplus ? soft : raw) : 0.0f;
            xs[m] = on ? w.widen(x[m]) : 0.0f;
            steps += dl[m];
            if (C) {
                const float zf = gated ? w.widen(z[m]) : 0.0f, act = pinned(zf * logistic(zf));
                g[m] = gated ? act : 1.0f;
                if (BACK) g[m] = on ? g[m] * w.widen(gy[m]) : 0.0f;
            }
        }
        wave_sync();
#pragma unroll
        for (int m = 0; m < kOwn; ++m) {
            w.store_du(du_of, m, dl[m], dl[m] * xs[m]);
            if (BACK) w.store_g(g_of, m, g[m]);
        }
        w.store_bc(lds, 0, bv);
        if (C) w.store_bc(lds, 1, cv);
        wave_sync();
        if (t0 + kSsmTile < w.end) load(t0 + kSsmTile);
        if (MARKS) {
            w.put(w.at(ws + p.marks, t0 / kSsmTile), h);
            if (!MULTI || w.blk == 0) ws[p.since + w.own_at(t0 / kSsmTile)] = since;
        }
        since += steps + dpp<0x4E>(steps);               // and of the other parity
        [[maybe_unused]] const __amdgpu_buffer_rsrc_t y_rows = w.rows_of(a.y, t0);
#pragma unroll
        for (int m = 0; m < kOwn; ++m) {
            float part[4];
#pragma unroll
            for (int par = 0; par < 2; ++par) {
                float bi[S], ci[S], d[2], u[2], gk[2];
                w.read_bc(lds, 2 * m + par, 0, bi);
                if (C) w.read_bc(lds, 2 * m + par, 1, ci);
                w.read_du(du_of, 2 * m + par, d, u);
                if (BACK) w.read_g(g_of, 2 * m + par, gk);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float y = 0.0f;
#pragma unroll
                    for (int s = 0; s < S; ++s) {
                        const float f = __builtin_amdgcn_exp2f(d[k] * A2[k][s]);
                        h[k][s] = fmaf(u[k], bi[s], f * h[k][s]);
                        if (OUT) y = fmaf(ci[s], h[k][s], y);
                        if (BACK) {
                            P[k][s] *= f;
                            R[k][s] = fmaf(P[k][s], ci[s] * gk[k], R[k][s]);
                        }
                    }
                    part[2 * par + k] = y;
                }
            }
            if (OUT) {
                const float y = quad_sum(part, w.j);
                if (MULTI) ex[(w.blk * kOwn + m) * 64 + w.lane] = y;
                else w.write(y_rows, w.row_at(m), kept(2 * m < left, fmaf(skip, xs[m], y) * g[m]));
            }
        }
        if (OUT && MULTI) {
            __syncthreads();
#pragma unroll
            for (int m = 0; m < kOwn; ++m)
                if (m % p.blocks == w.blk)
                    w.write(y_rows, w.row_at(m), 2 * m < left ? fmaf(skip, xs[m], joined(ex, p.blocks, m, w.lane)) * g[m] : 0.0f);
            __syncthreads();
        }
    }
    if (OUT) {
        for (int64_t t = w.behind_tiles + 2 * w.blk + w.odd; t < w.stop; t += 2 * p.blocks)
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

// Tiles whose shares of dA, dskip and ddt_bias are added in float32; such sums
// are joined in float64, here in LDS and at last in column_sum.
constexpr int kJoin = 8;
// Bytes of LDS that a wave of the gradients keeps for itself: those sums and
// the segment's first state.
template <int S>
constexpr int kept_lds_bytes() { return 64 * ((2 * S + 2) * 8 + 2 * S * 4); }

// The waves of a workgroup: blocks of states (MULTI), or adjacent channel
// blocks, whose shares of db and dc are added in LDS before they are written.
template <typename T, int S, int BLOCKS>
__global__ __launch_bounds__(BLOCKS > 1 ? 64 * BLOCKS : 256) __attribute__((amdgpu_waves_per_eu(2)))
void ssm_gradients(pn_ssm_args a, SsmPlan p) {
    constexpr int E = 4 * S, WAVES = BLOCKS > 1 ? BLOCKS : 4;
    constexpr bool MULTI = BLOCKS > 1;
    __shared__ __align__(16) float bc_lds[WAVES][kSsmTile * 2 * E];
    __shared__ __align__(16) float du_lds[WAVES][kSsmTile * kChans * 2], g_lds[WAVES][kSsmTile * kChans];
    __shared__ float ex[3][MULTI ? WAVES * kOwn * 64 : 1];
    __shared__ float shares[2][MULTI ? 1 : WAVES][MULTI ? 1 : kSsmTile * 2 * E];
    extern __shared__ __align__(16) char kept_lds[];
    const SsmWave<T, S, !MULTI> w(a, p);
    if (w.seg >= p.n_seg) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    float* ws = static_cast<float*>(a.workspace);
    float *lds = bc_lds[wave], *du_of = du_lds[wave], *g_of = g_lds[wave];
    const float bias = a.dt_bias ? a.dt_bias[w.ch] : 0.0f, skip = a.skip ? a.skip[w.ch] : 0.0f;
    const bool gated = a.gate.p != nullptr;
    T *dxp = static_cast<T*>(a.dx), *ddp = static_cast<T*>(a.ddt), *dzp = static_cast<T*>(a.dgate);
    float A2[2][S], r[2][S], dA[2][S];
    w.decays(A2);
    // the lane's own: sums (those of dA, dskip, ddt_bias) and the segment's first state in put()'s order
    double* sums = reinterpret_cast<double*>(kept_lds + wave * kept_lds_bytes<S>()) + w.lane;
    float* in = reinterpret_cast<float*>(kept_lds + wave * kept_lds_bytes<S>() + 64 * (2 * S + 2) * 8) + w.lane * S;
#pragma unroll
    for (int i = 0; i < 2 * S + 2; ++i) sums[64 * i] = 0.0;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int s = 0; s < S; ++s) r[k][s] = dA[k][s] = 0.0f;
    if (w.seg > 0) {
        float h[2][S];
        w.carried(ws, A2, h);
        w.put(in, h);
    }
    if (a.d_final_state)
        w.states([&](int k, int s, int64_t i) { r[k][s] = a.d_final_state[w.b * a.D * a.N + i]; });
    w.over_segments(ws, p.rends, p.n_seg - 1, -1, p.n_seg - 1 - w.seg, A2, r);   // what the segments behind give
    float dskip = 0.0f, dbias = 0.0f;
    const int NP = p.blocks * E;
    float* bc_out = ws + p.part_bc + (static_cast<int64_t>(MULTI ? w.cb : w.cb / p.wide) * a.B + w.b) * a.T * 2 * NP;
    const int value = ChannelSum<S>::of(w.lane);
    const int bc_at = (value / S) * NP + w.n0 + value % S;
    const bool bc_on = ChannelSum<S>::writes(w.lane);
    for (int64_t t = w.behind_tiles + 2 * w.blk + w.odd; t < w.stop; t += 2 * p.blocks)
        if (w.own) {
            const int64_t o = (w.b * a.T + t) * a.D + w.ch;
            dxp[o] = from_f32<T>(0.0f);
            ddp[o] = from_f32<T>(0.0f);
            if (gated) dzp[o] = from_f32<T>(0.0f);
        }
    auto join = [&]() {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int s = 0; s < S; ++s) {
                sums[64 * (k * S + s)] += dA[k][s];
                dA[k][s] = 0.0f;
            }
        sums[64 * 2 * S] += dskip;
        sums[64 * (2 * S + 1)] += dbias;
        dskip = dbias = 0.0f;
    };
    int turn = 0, since_join = 0;
    uint32_t x[kOwn], dt[kOwn], z[kOwn], gy[kOwn], bv[w.M], cv[w.M];
    float mark[2][S], since = 0.0f;
    auto load = [&](int64_t t0) {
        w.get(w.at(ws + p.marks, t0 / kSsmTile), mark);
        since = w.seg > 0 ? ws[p.since + w.own_at(t0 / kSsmTile)] : 0.0f;
        w.load_rows(a.x, t0, x);
        w.load_rows(a.dt, t0, dt);
        if (gated) w.load_rows(a.gate, t0, z);
        w.load_rows(a.dy, t0, gy);
        w.load_bc(w.bp, a.b.st, t0, bv);
        w.load_bc(w.cp, a.c.st, t0, cv);
    };
    const int64_t last = w.begin + (w.end - 1 - w.begin) / kSsmTile * kSsmTile;
    if (w.begin < w.end) load(last);
    for (int64_t t0 = last; w.begin < w.end && t0 >= w.begin; t0 -= kSsmTile) {
        const int left = w.left(t0) - w.odd;             // the lane's token m exists if 2 m < left
        float dl[kOwn], xs[kOwn], g[kOwn], slope[kOwn], dz[kOwn], e[kSsmTile][2][S], h[2][S];
        wave_sync();                                     // the last tile's have been read
#pragma unroll
        for (int m = 0; m < kOwn; ++m) {
            const bool on = 2 * m < left, mine = on && w.own;
            const float raw = w.widen(dt[m]) + bias, dy = w.widen(gy[m]);
            float sl = 1.0f;
            const float soft = pinned(softplus(raw, &sl));
            dl[m] = on ? (a.softplus ? soft : raw) : 0.0f;
            const float rise = pinned(sl);
            slope[m] = a.softplus ? rise : 1.0f;
            xs[m] = mine ? w.widen(x[m]) : 0.0f;
            const float zf = gated ? w.widen(z[m]) : 0.0f, sg = logistic(zf), act = pinned(zf * sg);
            g[m] = kept(mine, dy * (gated ? act : 1.0f));
            dz[m] = pinned(dy * sg * fmaf(zf, 1.0f - sg, 1.0f));
            w.store_du(du_of, m, dl[m], dl[m] * xs[m]);
            w.store_g(g_of, m, g[m]);
        }
        if (w.seg > 0) {
            w.get(in, h);
            w.fade(h, since, A2, mark);
        } else {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int s = 0; s < S; ++s) h[k][s] = mark[k][s];
        }
        w.store_bc(lds, 0, bv);
        w.store_bc(lds, 1, cv);
        wave_sync();
        if (t0 > w.begin) load(t0 - kSsmTile);
        const __amdgpu_buffer_rsrc_t dx_rows = w.rows_of(a.dx, t0), dd_rows = w.rows_of(a.ddt, t0);
        const __amdgpu_buffer_rsrc_t dz_rows = gated ? w.rows_of(a.dgate, t0) : w.no_rows();
#pragma unroll
        for (int m = 0; m < kOwn; ++m) {
            float part[4];
#pragma unroll
            for (int par = 0; par < 2; ++par) {
                const int i = 2 * m + par;
                float bi[S], ci[S], d[2], u[2];
                w.read_bc(lds, i, 0, bi);
                w.read_bc(lds, i, 1, ci);
                w.read_du(du_of, i, d, u);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float y = 0.0f;
#pragma unroll
                    for (int s = 0; s < S; ++s) {
                        e[i][k][s] = __builtin_amdgcn_exp2f(d[k] * A2[k][s]) * h[k][s];
                        h[k][s] = fmaf(u[k], bi[s], e[i][k][s]);
                        y = fmaf(ci[s], h[k][s], y);
                    }
                    part[2 * par + k] = y;
                }
            }
            {
                const float y = quad_sum(part, w.j);
                if (MULTI) ex[0][(w.blk * kOwn + m) * 64 + w.lane] = y;
                else w.write(dz_rows, w.row_at(m), kept(2 * m < left, dz[m] * fmaf(skip, xs[m], y)));
            }
        }
#pragma unroll
        for (int m = kOwn - 1; m >= 0; --m) {
            float s1[4], s2[4];
#pragma unroll
            for (int par = 1; par >= 0; --par) {
                const int i = 2 * m + par;
                float bi[S], ci[S], d[2], u[2], gk[2], db[S], dc[S], gu = 0.0f;
                w.read_bc(lds, i, 0, bi);
                w.read_bc(lds, i, 1, ci);
                w.read_du(du_of, i, d, u);
                w.read_g(g_of, i, gk);
#pragma unroll
                for (int s = 0; s < S; ++s) db[s] = dc[s] = 0.0f;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float du = 0.0f, dd = 0.0f;
                    gu = fmaf(gk[k], u[k], gu);
#pragma unroll
                    for (int s = 0; s < S; ++s) {
                        r[k][s] = fmaf(gk[k], ci[s], r[k][s]);
                        db[s] = fmaf(r[k][s], u[k], db[s]);
                        dc[s] = fmaf(gk[k], e[i][k][s], dc[s]);
                        du = fmaf(r[k][s], bi[s], du);
                        const float x = r[k][s] * e[i][k][s];
                        dd = fmaf(x, A2[k][s], dd);
                        dA[k][s] = fmaf(x, d[k], dA[k][s]);
                        r[k][s] *= __builtin_amdgcn_exp2f(d[k] * A2[k][s]);
                    }
                    s1[2 * par + k] = du;
                    s2[2 * par + k] = dd;
                }
#pragma unroll
                for (int s = 0; s < S; ++s) dc[s] = fmaf(gu, bi[s], dc[s]);  // h = e + u b
                const float sum = ChannelSum<S>::sum(db, dc, w.lane);
                if (MULTI) {
                    if (bc_on && t0 + i < w.end) bc_out[(t0 + i) * 2 * NP + bc_at] = sum;
                } else if (bc_on) {
                    shares[turn][wave][i * 2 * E + bc_at] = sum;
                }
            }
            const float du = quad_sum(s1, w.j), dd = quad_sum(s2, w.j) * kLn2;
            if (MULTI) {
                ex[1][(w.blk * kOwn + m) * 64 + w.lane] = du;
                ex[2][(w.blk * kOwn + m) * 64 + w.lane] = dd;
            } else {
                const float ddt = kept(2 * m < left, fmaf(xs[m], du, dd) * slope[m]);
                w.write(dx_rows, w.row_at(m), kept(2 * m < left, fmaf(dl[m], du, skip * g[m])));
                w.write(dd_rows, w.row_at(m), ddt);
                dskip = fmaf(g[m], xs[m], dskip);
                dbias += ddt;
            }
        }
        if (MULTI) {
            __syncthreads();
#pragma unroll
            for (int m = 0; m < kOwn; ++m)
                if (m % p.blocks == w.blk) {
                    const float du = joined(ex[1], p.blocks, m, w.lane), dd = joined(ex[2], p.blocks, m, w.lane);
                    const float ddt = kept(2 * m < left, fmaf(xs[m], du, dd) * slope[m]);
                    w.write(dx_rows, w.row_at(m), kept(2 * m < left, fmaf(dl[m], du, skip * g[m])));
                    w.write(dd_rows, w.row_at(m), ddt);
                    if (gated)
                        w.write(dz_rows, w.row_at(m), 2 * m < left ? dz[m] * fmaf(skip, xs[m], joined(ex[0], p.blocks, m, w.lane)) : 0.0f);
                    dskip = fmaf(g[m], xs[m], dskip);
                    dbias += ddt;
                }
            __syncthreads();
        } else {
            __syncthreads();                             // the other half of shares is free since the last
            for (int i = threadIdx.x; i < kSsmTile * 2 * E; i += 64 * p.wide) {
                float v = 0.0f;
                for (int q = 0; q < p.wide; ++q) v += shares[turn][q][i];
                if (i < (w.end - t0) * 2 * E) bc_out[t0 * 2 * E + i] = v;
            }
            turn ^= 1;
        }
        if (++since_join == kJoin) {
            join();
            since_join = 0;
        }
    }
    join();
    // the two parities of a channel
    dskip = static_cast<float>(sums[64 * 2 * S]);
    dbias = static_cast<float>(sums[64 * (2 * S + 1)]);
    dskip += dpp<0x4E>(dskip);
    dbias += dpp<0x4E>(dbias);
    const int64_t part = w.b * p.n_seg + w.seg;
    w.states([&](int k, int s, int64_t i) {
        ws[p.part_A + part * a.D * a.N + i] = static_cast<float>(sums[64 * (k * S + s)]);
    });
    if (w.own && w.odd == 0) {
        float* v = ws + p.part_vec + (part * p.blocks + w.blk) * 2 * a.D + w.ch;
        v[0] = dskip;
        v[a.D] = dbias;
    }
    if (w.seg == 0 && a.d_initial_state)
        w.states([&](int k, int s, int64_t i) { a.d_initial_state[w.b * a.D * a.N + i] = r[k][s]; });
}

template <typename T, int S, int BLOCKS>
hipError_t ssm_launch(const pn_ssm_args& a, const SsmPlan& p, SsmPass pass, hipStream_t st) {
    const bool wide = BLOCKS == 1 && pass == kSsmGradients;
    const int threads = 64 * (wide ? p.wide : p.blocks);
    const int64_t segs = pass == kSsmEnds ? p.n_seg - 1 : p.n_seg;
    const dim3 grid = grid_of(segs * a.B * (wide ? p.chans / p.wide : p.chans), threads);
    switch (pass) {
        case kSsmEnds: ssm_pass<T, S, BLOCKS, kSsmEnds><<<grid, threads, 0, st>>>(a, p); break;
        case kSsmOutputs: ssm_pass<T, S, BLOCKS, kSsmOutputs><<<grid, threads, 0, st>>>(a, p); break;
        case kSsmMarks: ssm_pass<T, S, BLOCKS, kSsmMarks><<<grid, threads, 0, st>>>(a, p); break;
        case kSsmMarksBoth: ssm_pass<T, S, BLOCKS, kSsmMarksBoth><<<grid, threads, 0, st>>>(a, p); break;
        default: {
            const auto kernel = ssm_gradients<T, S, BLOCKS>;
            const int lds = threads / 64 * kept_lds_bytes<S>();
            if (lds > 48 * 1024) {
                const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
                if (e != hipSuccess) return e;
            }
            kernel<<<grid, threads, lds, st>>>(a, p);
        }
    }
    return hipGetLastError();
}

}  // namespace

template <typename T>
hipError_t launch_ssm_pass(const pn_ssm_args& a, const SsmPlan& p, SsmPass pass, hipStream_t st) {
    if (p.blocks > 4) return ssm_launch<T, 4, 8>(a, p, pass, st);
    if (p.blocks > 2) return ssm_launch<T, 4, 4>(a, p, pass, st);
    if (p.blocks > 1) return ssm_launch<T, 4, 2>(a, p, pass, st);
    if (p.states == 4) return ssm_launch<T, 1, 1>(a, p, pass, st);
    if (p.states == 8) return ssm_launch<T, 2, 1>(a, p, pass, st);
    return ssm_launch<T, 4, 1>(a, p, pass, st);
}

}  // namespace pn
