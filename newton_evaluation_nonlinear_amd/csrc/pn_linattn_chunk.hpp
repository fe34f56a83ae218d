// The chunked form of the operator in pn_seq.hpp (LaOp), on the matrix cores.
//
// A chunk of C tokens with state S before it, for i, j inside the chunk:
//     O_i = f lam^{i+1} Q_i S + p sum_{j <= i} lam^{i-j} (Q_i . K_j) V_j
//     S  <- lam^C S + ws sum_j lam^{C-1-j} K_j^T V_j
// (time reversed: lam^{i} and lam^{C-j}, since lam then follows a token).
//
// A wave owns 32 columns (value channels) of a state and walks the chunks of
// its part of the sequence with that state, DK x 32 float32, in its
// accumulators.  Nothing of it goes through LDS: an accumulator tile's lanes
// are columns and its registers rows, which is how the next product wants
// its operand, once the rows are dealt to the registers as perm() does and
// the float32 values are cut into bfloat16 parts.  The same holds for the
// scores, which are formed transposed (K Q^T) and feed the product with V.
// So a chunk's products are, per wave,
//     scores^T = K Q^T,   O^T = S^T Q^T (scaled) + V^T scores^T,   S += K^T (w V).
// The waves of a workgroup (32 NW columns) share Q, K and K^T in LDS; V^T is
// read by the wave that owns its columns.
//
// Precision.  A float32 operand is a sum of bfloat16 parts of 8 bits each, a
// product of two the sum of the parts' products of order below `LIM`; a
// storage type has NP parts (bfloat16 1, binary16 2, float32 3, all exact).
// Outputs in 16 bits take LIM 2 (2^-16 per operand); the state, and float32
// outputs, LIM 3 (2^-24).
#pragma once

#include <type_traits>

#include "pn_seq.hpp"
#include "pn_seq_device.hpp"

namespace pn {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <typename T>
struct Parts;
template <>
struct Parts<bf16> { static constexpr int NP = 1, LIM = 2, C = 64; };
template <>
struct Parts<f16> { static constexpr int NP = 2, LIM = 2, C = 32; };
template <>
struct Parts<float> { static constexpr int NP = 3, LIM = 3, C = 32; };

// One launch of chunk workgroups (pn_linattn.hip).
struct LaChunkArgs {
    LaArgs a;
    int64_t seg;           // tokens of a segment (a multiple of C)
    int32_t n_seg;
    int32_t vec[3];        // operands of op[w] readable 16 bytes at a time (bits q 1, k 2, v 4), output writable (8)
    // [n_seg - 1][B * H] states, of each segment alone, then before the next
    // segment; element (x, y) of one at x * c_k + y * c_v
    float* carry[3];
    int32_t c_k[3], c_v[3];
};

// The workgroup's place in the launch, so that neighbours (columns of a head,
// operators and segments of it, heads that share keys and values) are on one
// of the 8 dies, and in its L2: ids go to the dies in turn.
__device__ __forceinline__ int neighbour_id(int id, int total) {
    const int die = id & 7, q = total >> 3, r = total & 7;
    return (die < r ? die * (q + 1) : r * (q + 1) + (die - r) * q) + (id >> 3);
}

__device__ __forceinline__ int seq_len(const int32_t* lengths, int b, int T) {
    if (!lengths) return T;
    const int n = lengths[b];
    return n < 0 ? 0 : (n > T ? T : n);
}

// Row (or column) of a 32-wide tile that lane index m stands for: register r
// of half h of an accumulator tile then holds row 16 (r / 8) + 8 h + r % 8.
__device__ __forceinline__ int perm(int m) { return 16 * (m >> 4) + 8 * ((m >> 2) & 1) + 4 * ((m >> 3) & 1) + (m & 3); }

// Elements from one LDS row of W to the next: 16 bytes of padding put the
// 16-byte reads of neighbouring rows into different banks, and keep every
// read of a lane at a constant distance from its first.  (The float32 parts
// of 256 rows leave no room for it.)
template <typename T, int DKP>
constexpr int pitch(int W) { return W + (sizeof(T) == 4 && DKP == 256 ? 0 : 8); }

// 8 float32 values as N bfloat16 parts.
template <int N>
__device__ __forceinline__ void split(const float* x, bf16x8* part) {
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bf16x2 p = __builtin_convertvector((f32x2){r[2 * i], r[2 * i + 1]}, bf16x2);
            w[i] = __builtin_bit_cast(uint32_t, p);
            if (n + 1 < N) {
                r[2 * i] -= __uint_as_float(w[i] << 16);
                r[2 * i + 1] -= __uint_as_float(w[i] & 0xffff0000u);
            }
        }
        part[n] = __builtin_bit_cast(bf16x8, w);
    }
}

// 8 values of a storage type as its NP parts.
template <typename T>
__device__ __forceinline__ void parts_of(const Pack<T, 8>& x, bf16x8* part) {
    if constexpr (sizeof(T) == 2 && Parts<T>::NP == 1) {
        part[0] = __builtin_bit_cast(bf16x8, x);
    } else {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = to_f32(x.v[i]);
        split<Parts<T>::NP>(f, part);
    }
}

template <int NP>
__device__ __forceinline__ void sum_parts(const bf16x8* part, float* x) {
#pragma unroll
    for (int n = NP - 1; n >= 0; --n) {
        const u32x4 w = __builtin_bit_cast(u32x4, part[n]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = __uint_as_float(w[i] << 16), b = __uint_as_float(w[i] & 0xffff0000u);
            x[2 * i] = n == NP - 1 ? a : x[2 * i] + a;
            x[2 * i + 1] = n == NP - 1 ? b : x[2 * i + 1] + b;
        }
    }
}

// c += the products of the parts of a (NA) and b (NB) of order below LIM.
template <int NA, int NB, int LIM>
__device__ __forceinline__ f32x16 product(const bf16x8* a, const bf16x8* b, f32x16 c) {
#pragma unroll
    for (int o = (NA + NB - 2 < LIM - 1 ? NA + NB - 2 : LIM - 1); o >= 0; --o)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (o - i >= 0 && o - i < NB) c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[o - i], c, 0, 0, 0);
    return c;
}

// Rows of one operand on their way from memory to LDS: units of 4 tokens x 8
// channels, UNITS per thread.  An operand that is stored transposed has
// neighbouring lanes on neighbouring tokens, so that their stores join in an
// LDS row; one that is not has them on neighbouring channels.  A chunk's tokens past the last one repeat it:
// what they add is dropped (rows not stored) or weighted 0.
template <typename T, int C, int W, int NT, bool COLS>
struct Stage {
    static constexpr int NU = (C / 4) * (W / 8);                 // units of a chunk
    static constexpr int UNITS = (NU + NT - 1) / NT;
    Pack<T, 8> x[UNITS][4];
    const T* p[UNITS];       // the unit's first token in the next chunk to load
    int64_t step;            // elements from one token to the next
    int valid;               // channels from the operand's first on
    bool vec;

    __device__ __forceinline__ static int token(int u) {
        const int i = threadIdx.x + u * NT;
        return (COLS ? i % (C / 4) : i / (W / 8)) * 4;
    }
    __device__ __forceinline__ static int channel(int u) {
        const int i = threadIdx.x + u * NT;
        return (COLS ? i / (C / 4) : i % (W / 8)) * 8;
    }

    // `base`: channel 0 of the first token of the first chunk.
    __device__ __forceinline__ void open(const T* base, int64_t step_, bool vec_, int c0, int D) {
        step = step_;
        vec = vec_;
        valid = D - c0;
#pragma unroll
        for (int u = 0; u < UNITS; ++u) p[u] = base + token(u) * step + c0 + channel(u);
    }
    // The next chunk, of which L tokens exist.
    __device__ __forceinline__ void load(int L) {
        const bool full = L >= C;
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const int left = valid - channel(u), last = L - 1 - token(u);
            const bool on = (NU % NT == 0 || static_cast<int>(threadIdx.x) + u * NT < NU) && left > 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[u][j] = Pack<T, 8>{};
            if (on) {
                if (vec && full) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[u][j] = *reinterpret_cast<const Pack<T, 8>*>(p[u] + j * step);
                } else if (vec) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        x[u][j] = *reinterpret_cast<const Pack<T, 8>*>(p[u] + (j < last ? j : last) * step);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const T* row = p[u] + (j < last ? j : last) * step;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (e < left) x[u][j].v[e] = row[e];
                    }
                }
            }
            p[u] += C * step;
        }
    }
    // To LDS as rows[part][token][channel] and / or cols[part][channel][token].
    template <bool ROWS, int RP, int CP>
    __device__ __forceinline__ void store(bf16* rows, bf16* cols) const {
        constexpr int NP = Parts<T>::NP;
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            if (NU % NT != 0 && static_cast<int>(threadIdx.x) + u * NT >= NU) continue;
            const int ch = channel(u), tk = token(u);
            bf16x8 p[4][NP];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                parts_of<T>(x[u][j], p[j]);
                if (ROWS)
#pragma unroll
                    for (int n = 0; n < NP; ++n) *reinterpret_cast<bf16x8*>(rows + (n * C + tk + j) * RP + ch) = p[j][n];
            }
            if (COLS)
#pragma unroll
                for (int n = 0; n < NP; ++n) {
                    u32x4 w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = __builtin_bit_cast(u32x4, p[j][n]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        // channel e of the 4 tokens: the low or high halves of word e / 2
                        const uint32_t sel = e % 2 ? 0x07060302u : 0x05040100u;
                        const u32x2 v = {__builtin_amdgcn_perm(w[1][e / 2], w[0][e / 2], sel),
                                         __builtin_amdgcn_perm(w[3][e / 2], w[2][e / 2], sel)};
                        *reinterpret_cast<u32x2*>(cols + (n * W + ch + e) * CP + tk) = v;
                    }
                }
        }
    }
};

// 8 values of an output tile (registers 8 t ..) to channels ch .. of a row.
template <typename T>
__device__ __forceinline__ void put(T* row, int ch, int D, bool vec, const f32x16& o, int t) {
    Pack<T, 8> v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v.v[e] = from_f32<T>(o[8 * t + e]);
    if (vec) {
        if (ch < D) *reinterpret_cast<Pack<T, 8>*>(row + ch) = v;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (ch + e < D) row[ch + e] = v.v[e];
    }
}

template <typename T, int DKP, int NW, bool OUT>
struct alignas(16) LaShared {
    static constexpr int NP = Parts<T>::NP, C = Parts<T>::C;
    static constexpr int RP = pitch<T, DKP>(DKP), CP = pitch<T, DKP>(C);
    alignas(16) bf16 q[OUT ? NP * C * RP : 8];      // [part][token][channel]
    alignas(16) bf16 k[OUT ? NP * C * RP : 8];
    alignas(16) bf16 kt[NP * DKP * CP];             // [part][channel][token]
    alignas(16) bf16 vt[NP * NW * 32 * CP];
    alignas(16) float w[C];         // weights of V in the state
    alignas(16) float back[32];     // lam^{32 - j}
    float m[64];                    // at 31 - i + j: scale lam^{i - j}, 0 for i < j
    float pw[C + 4];                // lam^0 .. lam^C
};

// Waves per SIMD (4 to a compute unit): two where two workgroups of four waves,
// or four of two, fit into 160 KB of LDS.
template <typename T, int DKP, int NW, bool OUT>
constexpr int la_occupancy() { return sizeof(LaShared<T, DKP, NW, OUT>) * (8 / NW) <= 160 * 1024 ? 2 : 1; }

__device__ __forceinline__ bf16x8 fragment(const bf16* p) { return *reinterpret_cast<const bf16x8*>(p); }

// S += K^T (w V), w V in N parts.
template <typename T, int DKP, int CP, int N>
__device__ __forceinline__ void add_tokens(f32x16* S, const bf16* kt, const float* w, const bf16x8 (*vf)[Parts<T>::NP]) {
    constexpr int NP = Parts<T>::NP, C = Parts<T>::C;
#pragma unroll
    for (int t = 0; t < C / 16; ++t) {
        float v8[8];
        bf16x8 wv[N];
        sum_parts<NP>(vf[t], v8);
        const Pack<float, 4> w0 = *reinterpret_cast<const Pack<float, 4>*>(w + 16 * t);
        const Pack<float, 4> w1 = *reinterpret_cast<const Pack<float, 4>*>(w + 16 * t + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v8[e] *= w0.v[e];
            v8[4 + e] *= w1.v[e];
        }
        split<N>(v8, wv);
#pragma unroll
        for (int kt_i = 0; kt_i < DKP / 32; ++kt_i) {
            bf16x8 kf[NP];
#pragma unroll
            for (int n = 0; n < NP; ++n) kf[n] = fragment(kt + (n * DKP + 32 * kt_i) * CP + 16 * t);
            S[kt_i] = product<NP, N, N>(kf, wv, S[kt_i]);
        }
    }
}

// OUT: outputs of a segment, from the state before it.  Otherwise the state
// that a segment leaves alone (from zero), for the scan over segments.
// EXACT: the state is a result, not only a term of 16-bit outputs.
template <typename T, int DKP, int NW, bool OUT, bool EXACT>
__global__ __launch_bounds__(64 * NW, (la_occupancy<T, DKP, NW, OUT>())) void la_chunk(LaChunkArgs g, int col_blocks) {
    constexpr int NP = Parts<T>::NP, LIM = Parts<T>::LIM, C = Parts<T>::C, NT = 64 * NW;
    constexpr int KT = DKP / 32, IT = C / 32;
    __shared__ LaShared<T, DKP, NW, OUT> sh;
    const LaArgs& a = g.a;
    const int segs = OUT ? g.n_seg : g.n_seg - 1;
    int id = neighbour_id(blockIdx.x, gridDim.x);
    const int c0 = id % col_blocks * 32 * NW;
    id /= col_blocks;
    const int op_i = id % a.n_ops;
    id /= a.n_ops;
    const int sg = id % segs, bh = id / segs;
    const LaOp& op = a.op[op_i];
    const int DK = op.DK, DV = op.DV;
    if (c0 >= DV) return;
    const int h = bh % a.H, b = bh / a.H;
    const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64, half = lane / 32, l32 = lane % 32, pl = perm(l32);
    const int N = static_cast<int>(a.T), len = seq_len(a.lengths, b, N), vec = g.vec[op_i];
    const bool reverse = op.reverse;
    const int i_begin = static_cast<int>(sg * g.seg);
    const int i_end = static_cast<int>(min(static_cast<int64_t>(N), (sg + 1) * g.seg));
    const int n_end = min(i_end, len);                   // tokens that count
    const double gl = a.log_decay[h];

    constexpr int RP = decltype(sh)::RP, CP = decltype(sh)::CP;
    Stage<T, C, DKP, NT, true> kst;
    Stage<T, C, DKP, NT, false> qst;
    Stage<T, C, 32 * NW, NT, true> vst;
    {
        const int64_t t0 = reverse ? len - 1 - i_begin : i_begin;
        const int sign = reverse ? -1 : 1;
        kst.open(static_cast<const T*>(op.k.p) + b * op.k.sb + (h / op.k.div) * op.k.sh + t0 * op.k.st, sign * op.k.st, vec & 2, 0, DK);
        vst.open(static_cast<const T*>(op.v.p) + b * op.v.sb + (h / op.v.div) * op.v.sh + t0 * op.v.st, sign * op.v.st, vec & 4, c0, DV);
        if (OUT)
            qst.open(static_cast<const T*>(op.q.p) + b * op.q.sb + (h / op.q.div) * op.q.sh + t0 * op.q.st, sign * op.q.st, vec & 1, 0, DK);
    }
    if (i_begin < n_end) {
        kst.load(n_end - i_begin);
        vst.load(n_end - i_begin);
        if (OUT) qst.load(n_end - i_begin);
    }

    if (tid <= C) sh.pw[tid] = tid == 0 ? 1.0f : static_cast<float>(exp(gl * tid));
    __syncthreads();
    if (tid < C) sh.w[tid] = op.ws * sh.pw[C - 1 - tid + (reverse ? 1 : 0)];
    if (tid < 32) sh.back[tid] = sh.pw[32 - tid];

    const float pscale = op.inter * op.ws;
    const float down = pscale * sh.pw[l32];
    if (OUT && tid < 64) sh.m[tid] = tid < 32 ? pscale * sh.pw[31 - tid] : 0.0f;

    const int64_t state_at = static_cast<int64_t>(bh) * DK * DV;
    const int col = c0 + 32 * wave + pl;                 // this lane's column of the state
    f32x16 S[KT];
    const float* from = OUT ? (sg > 0 ? g.carry[op_i] + static_cast<int64_t>(sg - 1) * a.B * a.H * DK * DV : op.s_in) : nullptr;
#pragma unroll
    for (int t = 0; t < KT; ++t) S[t] = (f32x16)(0.0f);
    if (from) {
        const int sk = sg > 0 ? g.c_k[op_i] : op.s_k, sv = sg > 0 ? g.c_v[op_i] : op.s_v;
        const float* at = from + state_at + min(col, DV - 1) * sv;
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int row = 32 * t + 16 * (r / 8) + 8 * half + r % 8;
                const float v = at[min(row, DK - 1) * sk];
                S[t][r] = row < DK && col < DV ? v : 0.0f;
            }
    }
    const bf16* q_at = sh.q + l32 * RP + 8 * half;       // this lane's first fragments
    const bf16* k_at = sh.k + pl * RP + 8 * half;
    const bf16* kt_at = sh.kt + pl * CP + 8 * half;
    const bf16* vt_at = sh.vt + (32 * wave + pl) * CP + 8 * half;

    for (int i0 = i_begin; i0 < n_end; i0 += C) {
        const int L = min(C, n_end - i0);
        __syncthreads();                                  // the chunk before is read
        kst.template store<OUT, RP, CP>(sh.k, sh.kt);
        vst.template store<false, RP, CP>(nullptr, sh.vt);
        if (OUT) qst.template store<true, RP, CP>(sh.q, nullptr);
        if (L < C && tid < C) sh.w[tid] = tid < L ? op.ws * sh.pw[L - 1 - tid + (reverse ? 1 : 0)] : 0.0f;
        __syncthreads();
        // the next chunk's loads: in flight over this chunk's products, and ahead
        // of its stores, which complete in order with them
        if (i0 + C < n_end) {
            const int left = n_end - i0 - C;
            kst.load(left);
            vst.load(left);
            if (OUT) qst.load(left);
        }
        bf16x8 vf[C / 16][NP];
        auto load_v = [&]() {
#pragma unroll
            for (int t = 0; t < C / 16; ++t)
#pragma unroll
                for (int n = 0; n < NP; ++n) vf[t][n] = fragment(vt_at + n * 32 * NW * CP + 16 * t);
        };
        if (!OUT) load_v();
        if (OUT) {
            f32x16 P[IT][IT], O[IT];                       // P[i][j], j <= i
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                O[i] = (f32x16)(0.0f);
#pragma unroll
                for (int j = 0; j <= i; ++j) P[i][j] = (f32x16)(0.0f);
            }
#pragma unroll
            for (int t = 0; t < DKP / 16; ++t) {
                bf16x8 qf[IT][NP], kf[IT][NP], sf[LIM];
#pragma unroll
                for (int i = 0; i < IT; ++i)
#pragma unroll
                    for (int n = 0; n < NP; ++n) {
                        qf[i][n] = fragment(q_at + (n * C + 32 * i) * RP + 16 * t);
                        kf[i][n] = fragment(k_at + (n * C + 32 * i) * RP + 16 * t);
                    }
                float s8[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) s8[e] = S[t / 2][8 * (t % 2) + e];
                split<LIM>(s8, sf);
#pragma unroll
                for (int i = 0; i < IT; ++i) {
#pragma unroll
                    for (int j = 0; j <= i; ++j) P[i][j] = product<NP, NP, 3>(kf[j], qf[i], P[i][j]);
                    O[i] = product<LIM, NP, LIM>(sf, qf[i], O[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < IT; ++i) O[i] *= op.inter * sh.pw[32 * i + l32 + (reverse ? 0 : 1)];
            load_v();
#pragma unroll
            for (int i = 0; i < IT; ++i)
#pragma unroll
                for (int j = 0; j <= i; ++j)
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        float p8[8];
                        bf16x8 pf[LIM];
                        const float* m = i == j ? sh.m + 31 - l32 + 8 * half : sh.back + 8 * half;
#pragma unroll
                        for (int e = 0; e < 8; ++e) p8[e] = P[i][j][8 * t + e] * (i == j ? m[16 * t + e] : down * m[16 * t + e]);
                        split<LIM>(p8, pf);
                        O[i] = product<NP, LIM, LIM>(vf[2 * j + t], pf, O[i]);
                    }
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int row = 32 * i + l32;
                if (row < L) {
                    const int64_t tok = reverse ? len - 1 - (i0 + row) : i0 + row;
                    const int64_t at = ((b * a.T + tok) * a.H + h) * DV;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int ch = c0 + 32 * wave + 16 * t + 8 * half;
                        if (op.o_f32) put(static_cast<float*>(op.o) + at, ch, DV, vec & 8, O[i], t);
                        else put(static_cast<T*>(op.o) + at, ch, DV, vec & 8, O[i], t);
                    }
                }
            }
        }
        const float decay = sh.pw[L];
#pragma unroll
        for (int t = 0; t < KT; ++t) S[t] *= decay;
        add_tokens<T, DKP, CP, EXACT ? 3 : LIM>(S, kt_at, sh.w + 8 * half, vf);
    }
    if (OUT) {
        // padding rows
        for (int64_t e = static_cast<int64_t>(max(i_begin, n_end)) * 32 * NW + tid; e < static_cast<int64_t>(i_end) * 32 * NW; e += NT) {
            const int64_t t = e / (32 * NW);
            const int c = c0 + static_cast<int>(e % (32 * NW));
            const int64_t at = ((b * a.T + t) * a.H + h) * DV + c;
            if (c < DV) {
                if (op.o_f32) static_cast<float*>(op.o)[at] = 0.0f;
                else static_cast<T*>(op.o)[at] = from_f32<T>(0.0f);
            }
        }
    }
    float* to = OUT ? (sg == segs - 1 ? op.s_out : nullptr) : g.carry[op_i] + static_cast<int64_t>(sg) * a.B * a.H * DK * DV;
    if (to && col < DV) {
        to += state_at + col;
        if (DK == DKP) {
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) to[(32 * t + 16 * (r / 8) + 8 * half + r % 8) * DV] = S[t][r];
        } else {
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int row = 32 * t + 16 * (r / 8) + 8 * half + r % 8;
                    if (row < DK) to[row * DV] = S[t][r];
                }
        }
    }
}

// Columns per workgroup of a launch, and its padded rows.
inline int la_waves(const LaArgs& a) {
    int dk = 0, dv = 0;
    for (int w = 0; w < a.n_ops; ++w) {
        if (a.op[w].DK > dk) dk = a.op[w].DK;
        if (a.op[w].DV > dv) dv = a.op[w].DV;
    }
    // float32 parts of 256 rows and 128 columns pass the 160 KB of LDS
    return dv <= 64 || (dk > 128 && a.dtype == PN_F32) ? 2 : 4;
}

template <typename T>
hipError_t launch_chunks(const LaChunkArgs& g, bool out, hipStream_t st) {
    int dk = 0, dv = 0;
    for (int w = 0; w < g.a.n_ops; ++w) {
        if (g.a.op[w].DK > dk) dk = g.a.op[w].DK;
        if (g.a.op[w].DV > dv) dv = g.a.op[w].DV;
    }
    const int nw = la_waves(g.a);
    const int segs = out ? g.n_seg : g.n_seg - 1;
    const int col_blocks = (dv + 32 * nw - 1) / (32 * nw);
    const dim3 grid(static_cast<uint32_t>(g.a.B * g.a.H * segs * g.a.n_ops * col_blocks));
    auto go = [&](auto rows, auto waves) {
        constexpr int DKP = decltype(rows)::value, NW = decltype(waves)::value;
        bool exact = Parts<T>::LIM == 3;
        for (int w = 0; w < g.a.n_ops; ++w) exact = exact || g.a.op[w].exact;
        if (exact) {
            if (out) la_chunk<T, DKP, NW, true, true><<<grid, 64 * NW, 0, st>>>(g, col_blocks);
            else la_chunk<T, DKP, NW, false, true><<<grid, 64 * NW, 0, st>>>(g, col_blocks);
        } else if constexpr (Parts<T>::LIM < 3) {
            if (out) la_chunk<T, DKP, NW, true, false><<<grid, 64 * NW, 0, st>>>(g, col_blocks);
            else la_chunk<T, DKP, NW, false, false><<<grid, 64 * NW, 0, st>>>(g, col_blocks);
        }
        return hipGetLastError();
    };
    using std::integral_constant;
    using W2 = integral_constant<int, 2>;
    using W4 = integral_constant<int, 4>;
    auto rows = [&](auto r) {
        using R = decltype(r);
        if constexpr (R::value == 256 && sizeof(T) == 4) return go(r, W2{});
        else return nw == 2 ? go(r, W2{}) : go(r, W4{});
    };
    if (dk <= 32) return rows(integral_constant<int, 32>{});
    if (dk <= 64) return rows(integral_constant<int, 64>{});
    if (dk <= 128) return rows(integral_constant<int, 128>{});
    return rows(integral_constant<int, 256>{});
}
extern template hipError_t launch_chunks<float>(const LaChunkArgs&, bool, hipStream_t);
extern template hipError_t launch_chunks<bf16>(const LaChunkArgs&, bool, hipStream_t);
extern template hipError_t launch_chunks<f16>(const LaChunkArgs&, bool, hipStream_t);

}  // namespace pn
