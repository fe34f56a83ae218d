// Linear attention with a decay per head: segments of the time axis, the scan
// over them, and the form for single tokens (the chunk kernels are in
// pn_linattn_chunk.hpp).
//
// The operator, for one sequence and head, over tokens i (LaOp):
//     S_i = lam S_{i-1} + ws K_i^T V_i,   O_i = inter * Q_i S_i.
// With R the gradient of the state (R_i = lam R_{i+1} + scale q_i^T do_i),
//     dq_i = scale do_i S_i^T,   dk_i = v_i R_i^T,   dv_i = k_i R_i,
// so the gradients are the same operator: dq with (Q, K, V) = (do, v, k), and,
// over reversed time, dv with (k, q, do) and dk with (v, do, q).

#include <algorithm>

#include "pn_linattn_chunk.hpp"

namespace pn {
namespace {

// The state before each segment from the states the segments leave alone:
//     S_{n+1} = lam^{tokens of n} S_n + U_n,
// in place, element by element; slot n holds U_n, then S_{n+1}.  Bandwidth: a
// workgroup takes 1024 elements of one state, so that few form its decays (a
// thread for each element took 23 us for 3 x 128 states of 128 x 128, so 12).
// Decays and running state are float64: a float32 decay would be off to the same
// side at each of up to 127 steps.
constexpr int kCarryElems = 1024;
__global__ __launch_bounds__(256) void la_carry(LaChunkArgs g, int blocks) {
    __shared__ double decay[2];                          // over a whole segment, over the last one
    const LaOp& op = g.a.op[blockIdx.y];
    const int n = op.DK * op.DV, bh = blockIdx.x / blocks, first = (blockIdx.x - bh * blocks) * kCarryElems;
    if (first >= n) return;
    const int64_t total = static_cast<int64_t>(g.a.B) * g.a.H * n;
    const int h = bh % g.a.H, b = bh / g.a.H;
    const int64_t len = seq_len(g.a.lengths, b, static_cast<int>(g.a.T));
    if (threadIdx.x < 2)
        decay[threadIdx.x] = exp(static_cast<double>(g.a.log_decay[h]) * static_cast<double>(threadIdx.x == 0 ? g.seg : len % g.seg));
    __syncthreads();
    double s[4];
    float* u[4];
    bool on[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int at = first + k * 256 + threadIdx.x, row = at / op.DV, col = at - row * op.DV;
        on[k] = at < n;
        u[k] = g.carry[blockIdx.y] + static_cast<int64_t>(bh) * n + (on[k] ? at : 0);
        s[k] = on[k] && op.s_in ? op.s_in[static_cast<int64_t>(bh) * n + row * op.s_k + col * op.s_v] : 0.0;
    }
    const int slots = g.n_seg - 1;
    for (int i0 = 0; i0 < slots; i0 += 4) {
        float x[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) x[j][k] = u[k][min(i0 + j, slots - 1) * total];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (i0 + j >= slots) break;
            const int64_t left = len - (i0 + j) * g.seg;
            const double d = left >= g.seg ? decay[0] : (left <= 0 ? 1.0 : decay[1]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                s[k] = d * s[k] + x[j][k];
                if (on[k]) u[k][(i0 + j) * total] = static_cast<float>(s[k]);
            }
        }
    }
}

// Operators whose states between segments are formed: the first ones that
// read their own (dk reads dv's, transposed).
int carried(const LaArgs& a) { return a.n_ops == 3 ? 2 : a.n_ops; }

// Segments of the time axis: the number n with the least estimated time.  In
// units of a chunk's outputs, the device full: a workgroup takes its chunks and
// kStart before them, and runs alone in kAlone of the time; the pass for the
// segments' states takes kStates of it, with half as many workgroups more at a
// time.  Measured on one training pass (8 x 4096 tokens, 16 heads of 128,
// bfloat16): outputs 5.1 us a chunk and pair of workgroups, 3.6 alone; states 2.5
// (2.1 since the state is faded late).
constexpr int64_t kFillWaves = 2048;     // two on each of the 4 SIMDs of 256 compute units
constexpr double kStart = 2.0, kAlone = 0.7, kStates = 0.5;
constexpr double kClear = 0.85;          // more segments, with their traffic, only for a clear gain

void segments(const LaArgs& a, int64_t* seg, int* n_seg) {
    int dv = 0;
    for (int w = 0; w < a.n_ops; ++w) dv = a.op[w].DV > dv ? a.op[w].DV : dv;
    const int64_t chunks = (a.T + kChunk - 1) / kChunk, nw = la_waves(a), cols = 32 * nw;
    const int64_t heads = static_cast<int64_t>(a.B) * a.H * ((dv + cols - 1) / cols), slots = kFillWaves / nw;
    auto rounds = [](int64_t groups, int64_t at_once) {
        return groups <= at_once / 2 ? kAlone : static_cast<double>((groups + at_once - 1) / at_once);
    };
    double least = 0.0;
    int64_t best = 1;
    for (int64_t n = 1; n <= chunks / 4 && n <= 128; ++n) {
        const double per = static_cast<double>((chunks + n - 1) / n) + kStart;
        double t = per * rounds(heads * a.n_ops * n, slots);
        if (n > 1) t += kStates * per * rounds(heads * carried(a) * (n - 1), slots * 3 / 2) + kStart;
        if (n == 1 || t < kClear * least) {
            least = t;
            best = n;
        }
    }
    const int64_t per = chunks > 0 ? (chunks + best - 1) / best : 1;
    *seg = per * kChunk;
    *n_seg = chunks > 0 ? static_cast<int>((chunks + per - 1) / per) : 1;
}

// An operand that can be read (or the output written) 16 bytes at a time, the
// tokens of a chunk within 2^31 bytes.
bool wide(const void* p, int64_t sb, int64_t st, int64_t sh, int D, int elem) {
    return D % 8 == 0 && st < (int64_t(1) << 24) && ((reinterpret_cast<intptr_t>(p) | sb * elem | st * elem | sh * elem) & 15) == 0;
}
bool wide(const LaOperand& x, int D, const LaArgs& a) {
    const int elem = a.dtype == PN_F32 ? 4 : 2;
    return wide(x.p, a.B > 1 ? x.sb : 0, x.st, a.H / x.div > 1 ? x.sh : 0, D, elem);
}

template <typename T>
__global__ __launch_bounds__(256) void la_group_sum(const float* in, T* out, int64_t n, int G, int D) {
    const int64_t e = static_cast<int64_t>(block_id()) * 256 + threadIdx.x;
    if (e >= n) return;
    const int64_t row = e / D;
    const int d = static_cast<int>(e - row * D);
    float s = 0.0f;
    for (int g = 0; g < G; ++g) s += in[(row * G + g) * D + d];
    out[e] = from_f32<T>(s);
}

// One token.  The state is read and written once, 8 DK DV bytes for 5 DK DV
// operations: bandwidth, or latency where there are few heads.  A workgroup
// takes LC * V columns of a head: LC lanes of V columns by 256 / LC groups of
// rows, every group 8 rows at a time, all loads of which are issued before
// the first store.  For a slow decay lam S + k v is taken as
// S + (S (lam - 1) + k v): lam - 1 keeps it exact over many steps, where lam
// itself, rounded, would be off by up to 2^-25 at each.  (S times
// lam - 1 takes an infinite S as the largest finite one, or the sum were a NaN.)
// Measured: 256 sequences of 16 heads, 128 x 128 (537 MB), 112 us, 4.8 TB/s, the
// rate of a large copy; 4 sequences 5.4 us.
template <typename T, int V, int LC>
__global__ __launch_bounds__(256) void la_step(pn_linattn_step_args a) {
    constexpr int RG = 256 / LC, ROWS = 8;
    __shared__ float sq[256 + RG * ROWS], sk[256 + RG * ROWS], part[4][LC * V];
    const int tid = threadIdx.x, lane = tid % LC, group = tid / LC;
    const int H = static_cast<int>(a.H), DK = static_cast<int>(a.dk), DV = static_cast<int>(a.dv);
    const int h = blockIdx.x % H, b = blockIdx.x / H;
    const int c = (blockIdx.y * LC + lane) * V;
    const bool live = c < DV;                            // V divides DV
    const int64_t slot = a.slots ? a.slots[b] : b;
    const bool idle = slot < 0 || slot >= a.n_slots;
    T* o = static_cast<T*>(a.o) + (static_cast<int64_t>(b) * H + h) * DV;
    if (idle) {
        if (group == 0 && live)
            for (int i = 0; i < V; ++i) o[c + i] = from_f32<T>(0.0f);
        return;
    }
    const int hk = h / static_cast<int>(a.H / a.HK);
    const T* qp = static_cast<const T*>(a.q.p) + b * a.q.sb + h * a.q.sh;
    const T* kp = static_cast<const T*>(a.k.p) + b * a.k.sb + hk * a.k.sh;
    const T* vp = static_cast<const T*>(a.v.p) + b * a.v.sb + hk * a.v.sh;
    float* S = a.state + (slot * H + h) * DK * DV + c;
    const float g = a.log_decay[h];
    const bool slow = g > -0.5f;
    const float f = slow ? expm1f(g) : expf(g);
    float x[ROWS][V], acc[V], v[V];
    auto load = [&](int r0) {
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            const int r = r0 + j * RG + group;
            Pack<float, V> p{};
            if (live && r < DK) p = *reinterpret_cast<const Pack<float, V>*>(S + r * DV);
#pragma unroll
            for (int i = 0; i < V; ++i) x[j][i] = p.v[i];
        }
    };
    load(0);
    for (int r = tid; r < 256 + RG * ROWS; r += 256) {
        sq[r] = r < DK ? to_f32(qp[r]) : 0.0f;
        sk[r] = r < DK ? to_f32(kp[r]) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        v[i] = live ? to_f32(vp[c + i]) : 0.0f;
        acc[i] = 0.0f;
    }
    __syncthreads();
    for (int r0 = 0;;) {
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            const int r = r0 + j * RG + group;
            const float k = sk[r], q = sq[r];
            Pack<float, V> n;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float finite = __builtin_amdgcn_fmed3f(x[j][i], -3.402823466e38f, 3.402823466e38f);
                const float t = fmaf(slow ? finite : x[j][i], f, k * v[i]);
                n.v[i] = slow ? x[j][i] + t : t;
                acc[i] = fmaf(q, n.v[i], acc[i]);
            }
            if (live && r < DK) *reinterpret_cast<Pack<float, V>*>(S + r * DV) = n;
        }
        r0 += RG * ROWS;
        if (r0 >= DK) break;
        load(r0);
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int m = LC; m < 64; m *= 2) acc[i] += __shfl_xor(acc[i], m);
    if (tid % 64 < LC)
#pragma unroll
        for (int i = 0; i < V; ++i) part[tid / 64][lane * V + i] = acc[i];
    __syncthreads();
    if (group == 0 && live)
#pragma unroll
        for (int i = 0; i < V; ++i)
            o[c + i] = from_f32<T>(static_cast<float>(a.scale) * (part[0][lane * V + i] + part[1][lane * V + i] +
                                                                  part[2][lane * V + i] + part[3][lane * V + i]));
}

template <typename T>
hipError_t step_typed(const pn_linattn_step_args& a, hipStream_t st) {
    const uint32_t heads = static_cast<uint32_t>(a.B * a.H);
    const uint32_t dv = static_cast<uint32_t>(a.dv);
    if (a.dv % 4 == 0 && reinterpret_cast<uintptr_t>(a.state) % 16 == 0) {
        // 32 columns per workgroup while that is what fills the device
        if (heads * ((dv + 127) / 128) >= 2048) la_step<T, 4, 32><<<dim3(heads, (dv + 127) / 128), 256, 0, st>>>(a);
        else la_step<T, 4, 8><<<dim3(heads, (dv + 31) / 32), 256, 0, st>>>(a);
    } else {
        la_step<T, 1, 32><<<dim3(heads, (dv + 31) / 32), 256, 0, st>>>(a);
    }
    return hipGetLastError();
}

}  // namespace

size_t linattn_workspace(const LaArgs& a) {
    int64_t seg;
    int n_seg;
    segments(a, &seg, &n_seg);
    size_t n = 0;
    for (int w = 0; w < carried(a); ++w)
        n += sizeof(float) * static_cast<size_t>(n_seg - 1) * a.B * a.H * a.op[w].DK * a.op[w].DV;
    return n;
}

bool linattn_fits(const LaArgs& a) {
    int64_t seg, state = 0;
    int n_seg, dv = 0;
    segments(a, &seg, &n_seg);
    for (int w = 0; w < a.n_ops; ++w) {
        dv = a.op[w].DV > dv ? a.op[w].DV : dv;
        state = std::max<int64_t>(state, a.op[w].DK * a.op[w].DV);
    }
    const int64_t heads = static_cast<int64_t>(a.B) * a.H, limit = int64_t(1) << 32;
    const int64_t cols = 32 * la_waves(a), chunks = heads * n_seg * a.n_ops * ((dv + cols - 1) / cols);
    return chunks * 2 * cols < limit && (n_seg == 1 || heads * ((state + kCarryElems - 1) / kCarryElems) * 256 < limit);
}

hipError_t launch_linattn(const LaArgs& a, void* workspace, hipStream_t st) {
    LaChunkArgs g{};
    g.a = a;
    segments(a, &g.seg, &g.n_seg);
    float* ws = static_cast<float*>(workspace);
    int most = 0;
    for (int w = 0; w < a.n_ops; ++w) {
        const LaOp& op = a.op[w];
        g.wide[w] = wide(op.q, op.DK, a) && wide(op.k, op.DK, a) && wide(op.v, op.DV, a) &&
                    wide(op.o, 0, static_cast<int64_t>(a.H) * op.DV, 0, op.DV, 4);
        const int64_t n = static_cast<int64_t>(a.B) * a.H * op.DK * op.DV;
        const int blocks = (op.DK * op.DV + kCarryElems - 1) / kCarryElems;
        most = blocks > most ? blocks : most;
        if (op.carry_from == w) {
            g.carry[w] = ws;
            g.c_k[w] = op.DV;
            g.c_v[w] = 1;
            ws += (g.n_seg - 1) * n;
        } else {
            g.carry[w] = g.carry[op.carry_from];
            g.c_k[w] = 1;
            g.c_v[w] = op.DK;
        }
    }
    auto run = [&](const LaChunkArgs& c, bool out) {
        switch (a.dtype) {
            case PN_F32: return launch_chunks<float>(c, out, st);
            case PN_BF16: return launch_chunks<bf16>(c, out, st);
            default: return launch_chunks<f16>(c, out, st);
        }
    };
    if (g.n_seg > 1) {
        LaChunkArgs c = g;
        c.a.n_ops = carried(a);
        hipError_t e = run(c, false);
        if (e != hipSuccess) return e;
        la_carry<<<dim3(static_cast<uint32_t>(a.B * a.H * most), c.a.n_ops), 256, 0, st>>>(c, most);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.n_ops == 3 && a.op[1].o_f32) {                 // a launch has one type of output
        LaChunkArgs c = g;
        c.a.n_ops = 1;
        const hipError_t e = run(c, true);
        if (e != hipSuccess) return e;
        for (int w = 0; w < 2; ++w) {
            c.a.op[w] = g.a.op[w + 1];
            c.carry[w] = g.carry[w + 1];
            c.c_k[w] = g.c_k[w + 1];
            c.c_v[w] = g.c_v[w + 1];
            c.wide[w] = g.wide[w + 1];
        }
        c.a.n_ops = 2;
        return run(c, true);
    }
    return run(g, true);
}

hipError_t launch_group_sum(const float* in, void* out, int dtype, int64_t rows, int G, int D, hipStream_t st) {
    const int64_t n = rows * D;
    const dim3 grid = grid_of((n + 255) / 256, 256);
    switch (dtype) {
        case PN_F32: la_group_sum<float><<<grid, 256, 0, st>>>(in, static_cast<float*>(out), n, G, D); break;
        case PN_BF16: la_group_sum<bf16><<<grid, 256, 0, st>>>(in, static_cast<bf16*>(out), n, G, D); break;
        default: la_group_sum<f16><<<grid, 256, 0, st>>>(in, static_cast<f16*>(out), n, G, D); break;
    }
    return hipGetLastError();
}

hipError_t launch_linattn_step(const pn_linattn_step_args& a, hipStream_t st) {
    switch (a.dtype) {
        case PN_F32: return step_typed<float>(a, st);
        case PN_BF16: return step_typed<bf16>(a, st);
        default: return step_typed<f16>(a, st);
    }
}

}  // namespace pn
