// The chunked form of the operator in pn_seq.hpp (LaOp), on the matrix cores.
//
// A chunk of C = 32 tokens with state S before it, for i, j inside the chunk:
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
// The waves of a workgroup (32 NW columns) share Q and K in LDS; V is read by
// the wave that owns its columns.  K and V are kept as they come, a row per
// token: K^T and V^T are read across the rows (fragment_across).
//
// Precision.  A float32 operand is a sum of bfloat16 parts of 8 bits each, a
// product of two the sum of the parts' products of order below `LIM`; a
// storage type has NP parts (bfloat16 1, binary16 2, float32 3, all exact).
// Outputs in 16 bits take LIM 2 (2^-16 per operand, far below their rounding);
// the state, and float32 outputs, LIM 3 (2^-24).  With LIM 3 for all, the error
// against 64 bits was the same to four digits in every output (1.66e-3 bfloat16,
// 2.07e-4 binary16, of the norm) and the time more: 417 -> 466 us for 65536
// tokens, 620 -> 760 for a training pass (16 heads of 128, bfloat16), 1013 -> 1236
// for one in binary16.
//
// Decay.  Between chunks the state is faded late: it is held as S / lam^n, n
// tokens after it was last faded, and faded when lam^n leaves [1/2, 2].  So a slow
// memory is not rounded once a chunk.
//
// Bound and measurements (8 x 4096 tokens, 16 heads of 128 x 128, bfloat16).
// Per wave and chunk of 32 tokens: 52 matrix instructions (8 scores, 16 with S,
// 4 with V, 24 for the state in three parts) of 32 cycles, and 434 vector ones of
// 4, most of them the 64 values of S cut into parts.  Two waves per
// SIMD keep the matrix units busy for 45 % and the vector units for 48 % of the
// time; sustained, the card lowers its clock from 2.0 to about 1.5 GHz.  Outputs
// of 4 segments: 166 us (537 MB, 3.2 TB/s; 140 us with every load from cache),
// the states of 3 of them 64 to 67 us.  With chunks of 64 tokens and K and V transposed
// through registers on their way into LDS the same outputs took 257 us, and 206
// with the loads ahead of the stores.
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
struct Parts<bf16> { static constexpr int NP = 1, LIM = 2; };
template <>
struct Parts<f16> { static constexpr int NP = 2, LIM = 2; };
template <>
struct Parts<float> { static constexpr int NP = 3, LIM = 3; };

constexpr int kChunk = 32;     // tokens of a chunk: one tile of the matrix instruction

// One launch of chunk workgroups (pn_linattn.hip).
struct LaChunkArgs {
    LaArgs a;
    int64_t seg;           // tokens of a segment (a multiple of C)
    int32_t n_seg;
    int32_t wide[3];       // 1: operands of op[w] can be read, its output written, 16 bytes at a time
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

// e^{g n}, 1 for n = 0, to a few 2^-24: the rounding of g n, which the
// exponential would magnify, is put back as its first-order factor.
__device__ __forceinline__ float decay_power(float g, float n) {
    const float x = g * n;
    if (n == 0.0f) return 1.0f;
    const float e = expf(x);
    return e == 0.0f || __builtin_isinf(x) ? e : fmaf(e, fmaf(g, n, -x), e);
}

// Row (or column) of a 32-wide tile that lane index m stands for: register r
// of half h of an accumulator tile then holds row 16 (r / 8) + 8 h + r % 8.
__device__ __forceinline__ int perm(int m) { return 16 * (m >> 4) + 8 * ((m >> 2) & 1) + 4 * ((m >> 3) & 1) + (m & 3); }

// Which of a row's 16-byte blocks (W / 8 of them) LDS holds at block b, so
// that no two lanes that read at once meet in a bank: rows of Q are read by 8
// neighbouring lanes; rows of K by the 8 lanes of perm(), 4 neighbouring ones
// also across (the transposing read), like those of V.
template <int W>
__device__ __forceinline__ int q_block(int row, int b) { return b ^ (row & 7 & (W / 8 - 1)); }
template <int W>
__device__ __forceinline__ int kv_block(int row, int b) { return b ^ ((2 * (row & 3) | ((row >> 3) & 1)) & (W / 8 - 1)); }

// (-1, 0) and (0, -1) as bfloat16 pairs, for split().  They are kept from the
// compiler's sight: as an immediate of the dot product it encodes the first
// like the second.
struct Minus {
    uint32_t lo, hi;
    __device__ __forceinline__ Minus() : lo(0x0000bf80u), hi(0xbf800000u) { asm volatile("" : "+s"(lo), "+s"(hi)); }
};

// 8 float32 values as N bfloat16 parts: each part is what the ones before it
// leave, rounded.  The remainder x - part, exact in float32, is a subtraction
// of the unpacked part, or, where x is not needed again (LAST), one dot product
// of the packed parts with (-1, 0) or (0, -1) added to x in place.
template <int N, bool LAST = true>
__device__ __forceinline__ void split(const float* x, bf16x8* part, const Minus& minus) {
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
            if (n + 1 == N) continue;
            if (LAST || n > 0) {
                r[2 * i] = __builtin_amdgcn_fdot2_f32_bf16(p, __builtin_bit_cast(bf16x2, minus.lo), r[2 * i], false);
                r[2 * i + 1] = __builtin_amdgcn_fdot2_f32_bf16(p, __builtin_bit_cast(bf16x2, minus.hi), r[2 * i + 1], false);
            } else {
                r[2 * i] -= __uint_as_float(w[i] << 16);
                r[2 * i + 1] -= __uint_as_float(w[i] & 0xffff0000u);
            }
        }
        part[n] = __builtin_bit_cast(bf16x8, w);
    }
}

// 8 values of a storage type as its NP parts.
template <typename T>
__device__ __forceinline__ void parts_of(const Pack<T, 8>& x, bf16x8* part, const Minus& minus) {
    if constexpr (sizeof(T) == 2 && Parts<T>::NP == 1) {
        part[0] = __builtin_bit_cast(bf16x8, x);
    } else {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = to_f32(x.v[i]);
        split<Parts<T>::NP>(f, part, minus);
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

// Products of parts that product() forms.
template <int NA, int NB, int LIM>
constexpr int products() {
    int n = 0;
    for (int i = 0; i < NA; ++i)
        for (int j = 0; j < NB; ++j) n += i + j < LIM;
    return n;
}

// Asks the scheduler for M matrix instructions with V vector instructions
// after each: the two run side by side in one wave.
template <int M, int V>
__device__ __forceinline__ void interleave() {
#pragma unroll
    for (int i = 0; i < M; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x2, V, 0);
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

// Rows of one operand on their way from memory to LDS: units of 8 channels of
// a token, UNITS per thread.  A chunk's tokens past the last one repeat it:
// what they add is dropped (rows not stored) or weighted 0.  Units past the
// last token or channel are read from the first and kept out of the rows (they
// go to `spare`), so that no access stands behind a branch: the wait for the
// loads then counts past the stores issued after them.
// VEC: 16-byte accesses; otherwise channel by channel.
template <typename T, int W, int NT, bool KV, bool VEC>
struct Stage {
    static constexpr int NU = kChunk * (W / 8);                  // units of a chunk
    static constexpr int UNITS = (NU + NT - 1) / NT;
    Pack<T, 8> x[UNITS];
    uint32_t off[UNITS];     // bytes from `base` to the unit
    int to[UNITS], part_step[UNITS];   // the unit's place in LDS, and from part to part
    const T* base;           // the lowest address of the next chunk, its channel 0
    int64_t st;              // elements from one token to the next
    int valid;               // channels from the operand's first on
    bool reverse;

    __device__ __forceinline__ static int token(int u) { return (threadIdx.x + u * NT) / (W / 8); }
    __device__ __forceinline__ static int block(int u) { return (threadIdx.x + u * NT) % (W / 8); }
    __device__ __forceinline__ bool here(int u) const {
        return (NU % NT == 0 || static_cast<int>(threadIdx.x) + u * NT < NU) && 8 * block(u) < valid;
    }
    __device__ __forceinline__ int row(int token) const { return reverse ? kChunk - 1 - token : token; }
    __device__ __forceinline__ uint32_t offset(int u, int last) const {
        return (row(min(min(token(u), kChunk - 1), last)) * static_cast<uint32_t>(st) + (here(u) ? 8 * block(u) : 0)) * sizeof(T);
    }

    // `first`: the operand's first channel of the first token of the first
    // chunk; `spare`: LDS for 8 elements, counted from the rows.
    __device__ __forceinline__ void open(const T* first, int64_t st_, bool reverse_, int channels, int spare) {
        st = st_;
        reverse = reverse_;
        valid = channels;
        base = first - (reverse ? (kChunk - 1) * st : 0);
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const int r = token(u), b = KV ? kv_block<W>(r, block(u)) : q_block<W>(r, block(u));
            off[u] = offset(u, kChunk - 1);
            to[u] = here(u) ? r * W + 8 * b : spare;
            part_step[u] = here(u) ? kChunk * W : 0;
        }
    }
    // The next chunk, of which L tokens exist.
    __device__ __forceinline__ void load(int L) {
        if (VEC) {
            const char* from = reinterpret_cast<const char*>(base);
            uint32_t at[UNITS];
#pragma unroll
            for (int u = 0; u < UNITS; ++u) at[u] = off[u];
            if (L < kChunk)
#pragma unroll
                for (int u = 0; u < UNITS; ++u) at[u] = offset(u, L - 1);
#pragma unroll
            for (int u = 0; u < UNITS; ++u) x[u] = *reinterpret_cast<const Pack<T, 8>*>(from + at[u]);
        } else {
            // Every element is read, those past the last channel from it: no
            // branch and no wait between the loads (4 x 4096 tokens, 8 heads of
            // 100 channels in bf16: 174 us, 226 us with a branch each; 82 us at
            // 104 channels, 16 bytes at a time).
#pragma unroll
            for (int u = 0; u < UNITS; ++u) {
                const T* at = base + row(min(min(token(u), kChunk - 1), L - 1)) * st;
#pragma unroll
                for (int e = 0; e < 8; ++e) x[u].v[e] = at[min(8 * block(u) + e, valid - 1)];
            }
#pragma unroll
            for (int u = 0; u < UNITS; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (8 * block(u) + e >= valid) x[u].v[e] = static_cast<T>(0.0f);
        }
        base += reverse ? -kChunk * st : kChunk * st;
    }
    // To LDS as rows[part][token][channel], blocks in their places.
    __device__ __forceinline__ void store(bf16* rows, const Minus& minus) const {
        constexpr int NP = Parts<T>::NP;
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            bf16x8 part[NP];
            parts_of<T>(x[u], part, minus);
#pragma unroll
            for (int n = 0; n < NP; ++n) *reinterpret_cast<bf16x8*>(rows + to[u] + n * part_step[u]) = part[n];
        }
    }
};

// The 16 values of an output tile that a lane holds, to channels ch .. ch + 7
// and ch + 16 .. ch + 23 of its row.
template <typename T>
__device__ __forceinline__ void put(T* row, int ch, int D, const f32x16& o) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const int c = ch + 16 * (e / 8) + e % 8;
        if (c < D) row[c] = from_f32<T>(o[e]);
    }
}
// The same 16 bytes at a time, at bytes `at` and `at` + 16 sizeof(T) of `out`;
// an offset of 2^31 or more is past the buffer and writes nothing.
template <typename T>
__device__ __forceinline__ void put_wide(__amdgpu_buffer_rsrc_t out, uint32_t at0, uint32_t at1, const f32x16& o) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        Pack<T, 8> v;
#pragma unroll
        for (int e = 0; e < 8; ++e) v.v[e] = from_f32<T>(o[8 * t + e]);
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) {
            u32x4 w;
            __builtin_memcpy(&w, reinterpret_cast<const char*>(&v) + 16 * i, 16);
            __builtin_amdgcn_raw_buffer_store_b128(w, out, (t ? at1 : at0) + 16 * i, 0, 0);
        }
    }
}
constexpr uint32_t kNoWrite = 0x80000000u;

// A pointer that is the same in every lane, in scalar registers.
__device__ __forceinline__ char* uniform(char* p) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
    return reinterpret_cast<char*>(static_cast<uint64_t>(hi) << 32 | lo);
}

__device__ __forceinline__ float uniform(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(uint32_t, x)));
}

// Channels of an LDS row that DKP of are used: a power of two, for q_block()
// and kv_block().
constexpr int row_width(int DKP) { return DKP == 96 ? 128 : DKP; }

template <typename T, int DKP, int NW, bool OUT>
struct alignas(16) LaShared {
    static constexpr int NP = Parts<T>::NP;
    alignas(16) bf16 q[OUT ? NP * kChunk * row_width(DKP) : 8];       // [part][token][channel]
    alignas(16) bf16 k[NP * kChunk * row_width(DKP)];
    alignas(16) bf16 v[NP * kChunk * NW * 32];
    alignas(16) bf16 spare[8];
    alignas(16) float w[kChunk];    // weights of V in the state
    float m[64];                    // at 31 - i + j: scale lam^{i - j}, 0 for i < j
    float pw[kChunk + 4];           // lam^0 .. lam^32
};

// Waves per SIMD that the registers are held to.  Three for the outputs of 128
// rows (168 registers) spill the loads in flight.
template <typename T, int DKP, bool OUT>
constexpr int la_occupancy() {
    return DKP == 256 ? (OUT ? 1 : 2) : (Parts<T>::NP == 1 && !OUT ? 3 : 2);
}

__device__ __forceinline__ bf16x8 fragment(const bf16* p) { return *reinterpret_cast<const bf16x8*>(p); }

// 8 tokens (rows, W elements apart) of a lane's channel: the transposing read
// gives lane 4 c + e of 16 element e of the 4 channels that lanes c, c + 4,
// c + 8 and c + 12 point at, one row each.
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
template <int W>
__device__ __forceinline__ bf16x8 fragment_across(const bf16* p) {
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * W));
    const u32x2 a = __builtin_bit_cast(u32x2, lo), b = __builtin_bit_cast(u32x2, hi);
    return __builtin_bit_cast(bf16x8, (u32x4){a[0], a[1], b[0], b[1]});
}
// Where this lane points for channels 32 x .. of the tokens 8 half ..
template <int W>
__device__ __forceinline__ int across_at(int lane, int x) {
    const int i = lane % 16, row = 8 * (lane / 32) + i / 4, c = i % 4;
    return row * W + 8 * kv_block<W>(row, 4 * x + 2 * ((lane / 16) & 1) + (c & 1)) + 4 * (c >> 1);
}

// OUT: outputs of a segment, from the state before it.  Otherwise the state
// that a segment leaves alone (from zero), for the scan over segments.
// EXACT: the state is a result, not only a term of 16-bit outputs.
// VEC: operands are read, and the output written, 16 bytes at a time.  TO: the
// output's type.
template <typename T, typename TO, int DKP, int NW, bool OUT, bool EXACT, bool VEC>
__global__ __launch_bounds__(64 * NW, (la_occupancy<T, DKP, OUT>())) void la_chunk(LaChunkArgs g, int col_blocks) {
    constexpr int NP = Parts<T>::NP, LIM = Parts<T>::LIM, NT = 64 * NW, KT = DKP / 32, VW = 32 * NW, RW = row_width(DKP);
    constexpr int SP = EXACT ? 3 : LIM;                  // parts of w V
    __shared__ LaShared<T, DKP, NW, OUT> sh;
    const LaArgs& a = g.a;
    const int segs = OUT ? g.n_seg : g.n_seg - 1;
    int id = neighbour_id(blockIdx.x, gridDim.x);
    const int c0 = id % col_blocks * VW;
    id /= col_blocks;
    const int op_i = id % a.n_ops;
    id /= a.n_ops;
    const int sg = id % segs, bh = id / segs;
    const LaOp& op = a.op[op_i];
    const int DK = op.DK, DV = op.DV;
    if (c0 >= DV) return;
    const int h = bh % a.H, b = bh / a.H;
    const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64, half = lane / 32, l32 = lane % 32, pl = perm(l32);
    const int N = static_cast<int>(a.T), len = seq_len(a.lengths, b, N);
    const bool reverse = op.reverse;
    const int i_begin = static_cast<int>(sg * g.seg);
    const int i_end = static_cast<int>(min(static_cast<int64_t>(N), (sg + 1) * g.seg));
    const int n_end = min(i_end, len);                   // tokens that count
    const float gl = a.log_decay[h];
    const Minus minus;

    Stage<T, RW, NT, true, VEC> kst;
    Stage<T, RW, NT, false, VEC> qst;
    Stage<T, VW, NT, true, VEC> vst;
    const int64_t t0 = reverse ? len - 1 - i_begin : i_begin;            // the first token
    kst.open(static_cast<const T*>(op.k.p) + b * op.k.sb + (h / op.k.div) * op.k.sh + t0 * op.k.st, op.k.st, reverse, DK,
             static_cast<int>(sh.spare - sh.k));
    vst.open(static_cast<const T*>(op.v.p) + b * op.v.sb + (h / op.v.div) * op.v.sh + t0 * op.v.st + c0, op.v.st, reverse, DV - c0,
             static_cast<int>(sh.spare - sh.v));
    if (OUT)
        qst.open(static_cast<const T*>(op.q.p) + b * op.q.sb + (h / op.q.div) * op.q.sh + t0 * op.q.st, op.q.st, reverse, DK,
                 static_cast<int>(sh.spare - sh.q));
    if (i_begin < n_end) {
        kst.load(n_end - i_begin);
        vst.load(n_end - i_begin);
        if (OUT) qst.load(n_end - i_begin);
    }

    if (DK < DKP)                                        // channels that no store reaches
        for (int e = tid; e < NP * kChunk * RW / 8; e += NT) {
            reinterpret_cast<u32x4*>(sh.k)[e] = (u32x4)(0u);
            if (OUT) reinterpret_cast<u32x4*>(sh.q)[e] = (u32x4)(0u);
        }
    // The tables are written by every thread, the same values to the same places,
    // not by as many threads as they have entries: after a branch on the thread
    // the compiler has saved registers to scratch before it restored the mask of
    // lanes, and lost those of the others (256 rows, float32 and binary16).
    const int n32 = min(tid, kChunk), m32 = tid % kChunk, m64 = tid % 64;
    sh.pw[n32] = decay_power(gl, static_cast<float>(n32));
    __syncthreads();
    sh.w[m32] = op.ws * sh.pw[kChunk - 1 - m32 + (reverse ? 1 : 0)];
    if (OUT) sh.m[m64] = m64 < 32 ? op.inter * op.ws * sh.pw[31 - m32] : 0.0f;
    const float inter = op.inter * sh.pw[l32 + (reverse ? 0 : 1)];      // of this lane's token

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
                S[t][r] = at[min(row, DK - 1) * sk];
            }
        if (DK < DKP || c0 + VW > DV)                    // after the loads: none waits for another
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int row = 32 * t + 16 * (r / 8) + 8 * half + r % 8;
                    S[t][r] = row < DK && col < DV ? S[t][r] : 0.0f;
                }
    }
    // this lane's first fragments; the others are at a distance or, where the
    // block changes, at an exclusive or
    const int q_at = l32 * RW + 8 * q_block<RW>(l32, half), k_at = pl * RW + 8 * kv_block<RW>(pl, half);
    const int kt_at = across_at<RW>(lane, 0), vt_at = across_at<VW>(lane, wave);

    // the output's rows of the chunk: the lowest address, and this lane's bytes
    // from it (up to 2^31)
    const int o_size = sizeof(TO), ch = c0 + 32 * wave + 8 * half;
    const int64_t o_row = static_cast<int64_t>(a.H) * DV * o_size;
    char* out = static_cast<char*>(op.o) + (b * a.T + t0 - (reverse ? kChunk - 1 : 0)) * o_row + static_cast<int64_t>(h) * DV * o_size;
    const int64_t out_step = (reverse ? -kChunk : kChunk) * o_row;
    const int64_t o_lane = (reverse ? kChunk - 1 - l32 : l32) * o_row;
    const uint32_t o_at0 = ch < DV ? static_cast<uint32_t>(o_lane) + ch * o_size : kNoWrite;
    const uint32_t o_at1 = ch + 16 < DV ? static_cast<uint32_t>(o_lane) + (ch + 16) * o_size : kNoWrite;

    // the loaded chunk, of which L tokens exist, to LDS
    auto stage = [&](int L) {
        kst.store(sh.k, minus);
        vst.store(sh.v, minus);
        if (OUT) qst.store(sh.q, minus);
        if (L < kChunk) sh.w[m32] = m32 < L ? op.ws * sh.pw[max(L - 1 - m32, 0) + (reverse ? 1 : 0)] : 0.0f;
    };
    if (i_begin < n_end) {
        __syncthreads();
        stage(n_end - i_begin);
    }
    float fade = 1.0f;                                   // the state is fade S, fade = lam^since
    int since = 0;
    for (int i0 = i_begin; i0 < n_end; i0 += kChunk) {
        const int left = n_end - i0, L = min(kChunk, left);
        __syncthreads();
        // the next chunk's loads: in flight over this chunk's products, and ahead
        // of its stores, which complete in order with them
        if (left > kChunk) {
            kst.load(left - kChunk);
            vst.load(left - kChunk);
            if (OUT) qst.load(left - kChunk);
        }
        // fragments of K^T: of one part all held, of more read as they are used
        constexpr bool HOLD = NP == 1;
        bf16x8 vf[2][NP], kx[HOLD ? 2 : 1][HOLD ? KT : 1][NP], wv[2][SP];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int n = 0; n < NP; ++n) vf[t][n] = fragment_across<VW>(sh.v + (n * kChunk + 16 * t) * VW + vt_at);
        auto across_k = [&](int t, int x, bf16x8* f) {
#pragma unroll
            for (int n = 0; n < NP; ++n) f[n] = fragment_across<RW>(sh.k + (n * kChunk + 16 * t) * RW + (kt_at ^ (32 * x)));
        };
        auto load_kx = [&](int t) {
            if constexpr (HOLD)
#pragma unroll
                for (int x = 0; x < KT; ++x) across_k(t, x, kx[t][x]);
        };
        // S is faded once lam^since leaves [1/2, 2]; until then what comes in is
        // scaled up instead.  A factor lam^32 for every chunk, rounded, would
        // take a state kept for 1024 chunks 7e-5 from its value.
        const float after = uniform(decay_power(gl, static_cast<float>(since + L)));
        const bool keep = after >= 0.5f && after <= 2.0f;
        const float up = keep ? uniform(__builtin_amdgcn_rcpf(after)) : 1.0f;
        // Of three parts without a branch (152 us, 156 with, for a ragged float32
        // batch), of one and two with it (618 us, 636 without, for a bfloat16
        // training pass).  Early, before the fragments, where registers are short
        // (256 rows or single channels: 12 to 290 bytes of scratch otherwise),
        // else under their loads (67 us, 78 early, for the states of 128 rows).
        constexpr bool EARLY = !OUT && (DKP == 256 || !VEC);
        auto fade_s = [&] {
            if (NP == 3 || !keep)
#pragma unroll
                for (int t = 0; t < KT; ++t) S[t] *= keep ? 1.0f : after;
        };
        auto weigh_v = [&](int t) {
            float v8[8];
            sum_parts<NP>(vf[t], v8);
            const float* w = sh.w + 16 * t + 8 * half;
            const Pack<float, 4> w0 = *reinterpret_cast<const Pack<float, 4>*>(w), w1 = *reinterpret_cast<const Pack<float, 4>*>(w + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v8[e] *= up * w0.v[e];
                v8[4 + e] *= up * w1.v[e];
            }
            split<SP>(v8, wv[t], minus);
        };
        if (OUT) {
            // P and O step by step over 16 channels, the next step's fragments and
            // parts of S prepared under this step's products
            constexpr int TT = DKP / 16;
            f32x16 P = (f32x16)(0.0f), O = (f32x16)(0.0f);
            bf16x8 qf[2][NP], kf[2][NP], sf[2][LIM];
            auto load_step = [&](int t) {
#pragma unroll
                for (int n = 0; n < NP; ++n) {
                    qf[t % 2][n] = fragment(sh.q + n * kChunk * RW + (q_at ^ (16 * t)));
                    kf[t % 2][n] = fragment(sh.k + n * kChunk * RW + (k_at ^ (16 * t)));
                }
            };
            auto split_step = [&](int t) {
                float s8[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) s8[e] = S[t / 2][8 * (t % 2) + e];
                split<LIM, false>(s8, sf[t % 2], minus);
            };
            // (of three parts there are too many to hold ahead: the compiler's order)
            constexpr bool AHEAD = NP < 3;
            if (AHEAD) {
                load_step(0);
                split_step(0);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                constexpr int M = products<NP, NP, 3>() + products<LIM, NP, LIM>();
                if (!AHEAD || t + 1 < TT) load_step(AHEAD ? t + 1 : t);
                if (!AHEAD) split_step(t);
                P = product<NP, NP, 3>(kf[t % 2], qf[t % 2], P);
                O = product<LIM, NP, LIM>(sf[t % 2], qf[t % 2], O);
                if (AHEAD) {
                    if (t + 1 < TT) split_step(t + 1);
                    __builtin_amdgcn_sched_group_barrier(0x100, 2 * NP, 0);
                    interleave<M, 24 / M + 1>();
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            float m[2][8];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 8; ++e) m[t][e] = sh.m[31 - l32 + 16 * t + 8 * half + e];
            load_kx(0);
            O *= inter * fade;
            bf16x8 pf[2][LIM];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                float p8[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) p8[e] = P[8 * t + e] * m[t][e];
                split<LIM>(p8, pf[t], minus);
            }
            weigh_v(0);
#pragma unroll
            for (int t = 0; t < 2; ++t) O = product<NP, LIM, LIM>(vf[t], pf[t], O);
            if (VEC) {
                const __amdgpu_buffer_rsrc_t to = __builtin_amdgcn_make_buffer_rsrc(uniform(out), static_cast<short>(0), 0x7fffffff, 0x00020000);
                const uint32_t at0 = l32 < L ? o_at0 : kNoWrite, at1 = l32 < L ? o_at1 : kNoWrite;
                put_wide<TO>(to, at0, at1, O);
            } else if (l32 < L) {
                put(reinterpret_cast<TO*>(out + o_lane), ch, DV, O);
            }
            out += out_step;
        } else {
            if (EARLY) fade_s();
            load_kx(0);
            weigh_v(0);
        }
        // fade S = lam^L fade S + K^T (w V)
        load_kx(1);
        if (!EARLY) fade_s();
        fade = keep ? after : 1.0f;
        since = keep ? since + L : 0;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int x = 0; x < KT; ++x) {
                bf16x8* f = HOLD ? kx[HOLD ? t : 0][HOLD ? x : 0] : kx[0][0];
                if (!HOLD) across_k(t, x, f);
                S[x] = product<NP, SP, SP>(f, wv[t], S[x]);
            }
            if (t == 0) weigh_v(1);
        }
        if (left > kChunk) {
            __syncthreads();                              // this chunk is read
            stage(left - kChunk);
        }
    }
    if (OUT) {
        // padding rows
        for (int64_t e = static_cast<int64_t>(max(i_begin, n_end)) * 32 * NW + tid; e < static_cast<int64_t>(i_end) * 32 * NW; e += NT) {
            const int64_t t = e / (32 * NW);
            const int c = c0 + static_cast<int>(e % (32 * NW));
            const int64_t at = ((b * a.T + t) * a.H + h) * DV + c;
            if (c < DV) static_cast<TO*>(op.o)[at] = from_f32<TO>(0.0f);
        }
    }
    float* to = OUT ? (sg == segs - 1 ? op.s_out : nullptr) : g.carry[op_i] + static_cast<int64_t>(sg) * a.B * a.H * DK * DV;
    if (to && col < DV) {
        to += state_at + col;
        if (DK == DKP) {
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) to[(32 * t + 16 * (r / 8) + 8 * half + r % 8) * DV] = fade * S[t][r];
        } else {
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int row = 32 * t + 16 * (r / 8) + 8 * half + r % 8;
                    if (row < DK) to[row * DV] = fade * S[t][r];
                }
        }
    }
}

// Waves, of 32 columns each, of a launch's workgroups.
inline int la_waves(const LaArgs& a) {
    int dv = 0;
    for (int w = 0; w < a.n_ops; ++w) dv = a.op[w].DV > dv ? a.op[w].DV : dv;
    return dv <= 64 ? 2 : 4;
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
        bool exact = Parts<T>::LIM == 3, vec = true;
        for (int w = 0; w < g.a.n_ops; ++w) {
            exact = exact || g.a.op[w].exact;
            vec = vec && g.wide[w];
        }
        auto form = [&](auto ex, auto wide) {
            constexpr bool E = decltype(ex)::value, V = decltype(wide)::value;
            if (!out) la_chunk<T, T, DKP, NW, false, E, V><<<grid, 64 * NW, 0, st>>>(g, col_blocks);
            else if (g.a.op[0].o_f32) la_chunk<T, float, DKP, NW, true, E, V><<<grid, 64 * NW, 0, st>>>(g, col_blocks);
            else la_chunk<T, T, DKP, NW, true, E, V><<<grid, 64 * NW, 0, st>>>(g, col_blocks);
            return hipGetLastError();
        };
        // channel by channel, the parts are not what takes the time: one form
        if (!vec) return form(std::true_type{}, std::false_type{});
        if constexpr (Parts<T>::LIM < 3)
            if (!exact) return form(std::false_type{}, std::true_type{});
        return form(std::true_type{}, std::true_type{});
    };
    using std::integral_constant;
    using W2 = integral_constant<int, 2>;
    using W4 = integral_constant<int, 4>;
    auto rows = [&](auto r) {
        return nw == 2 ? go(r, W2{}) : go(r, W4{});
    };
    if (dk <= 32) return rows(integral_constant<int, 32>{});
    if (dk <= 64) return rows(integral_constant<int, 64>{});
    if (dk <= 96) return rows(integral_constant<int, 96>{});
    if (dk <= 128) return rows(integral_constant<int, 128>{});
    return rows(integral_constant<int, 256>{});
}
extern template hipError_t launch_chunks<float>(const LaChunkArgs&, bool, hipStream_t);
extern template hipError_t launch_chunks<bf16>(const LaChunkArgs&, bool, hipStream_t);
extern template hipError_t launch_chunks<f16>(const LaChunkArgs&, bool, hipStream_t);

}  // namespace pn
