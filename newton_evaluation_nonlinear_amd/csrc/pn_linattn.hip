// Linear attention with a decay per head.
//
// The operator, for one sequence and head, over tokens i (LaOp):
//     S_i = lam S_{i-1} + ws K_i^T V_i,   O_i = inter * Q_i S_i.
// With R the gradient of the state (R_i = lam R_{i+1} + scale q_i^T do_i),
//     dq_i = scale do_i S_i^T,   dk_i = v_i R_i^T,   dv_i = k_i R_i,
// so the gradients are the same operator: dq with (Q, K, V) = (do, v, k), and,
// over reversed time, dv with (k, q, do) and dk with (v, do, q).

#include "pn_seq.hpp"
#include "pn_seq_device.hpp"

namespace pn {
namespace {

constexpr int kCols = 64;

__device__ __forceinline__ int seq_len(const int32_t* lengths, int b, int T) {
    if (!lengths) return T;
    const int n = lengths[b];
    return n < 0 ? 0 : (n > T ? T : n);
}

// The recurrence as written: a workgroup owns one head's state for 64 columns,
// each of its 4 waves a quarter of the rows in registers, and walks the tokens.
template <typename T, int ROWS>
__global__ __launch_bounds__(256) void la_recurrent(LaArgs a, int which) {
    const LaOp op = a.op[which];
    __shared__ float sq[256], sk[256], part[4][kCols];
    const int tid = threadIdx.x, col = tid % kCols, wv = tid / kCols;
    const int h = blockIdx.x % a.H, b = blockIdx.x / a.H;
    const int vv = blockIdx.y * kCols + col;
    const int N = static_cast<int>(a.T), len = seq_len(a.lengths, b, N);
    const bool live = vv < op.DV;
    const float lam = expf(a.log_decay[h]);
    float S[ROWS];
    const int64_t sbase = (static_cast<int64_t>(b) * a.H + h) * op.DK * op.DV;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int r = wv * ROWS + i;
        S[i] = op.s_in && live && r < op.DK ? op.s_in[sbase + r * op.s_k + vv * op.s_v] : 0.0f;
    }
    const T* qp = static_cast<const T*>(op.q.p) + b * op.q.sb + (h / op.q.div) * op.q.sh;
    const T* kp = static_cast<const T*>(op.k.p) + b * op.k.sb + (h / op.k.div) * op.k.sh;
    const T* vp = static_cast<const T*>(op.v.p) + b * op.v.sb + (h / op.v.div) * op.v.sh;
    for (int i = 0; i < N; ++i) {
        const int64_t t = op.reverse && i < len ? len - 1 - i : i;
        float o = 0.0f;
        if (i < len) {
            __syncthreads();
            sq[tid] = tid < op.DK ? to_f32(qp[t * op.q.st + tid]) : 0.0f;
            sk[tid] = tid < op.DK ? to_f32(kp[t * op.k.st + tid]) : 0.0f;
            const float v = live ? op.ws * to_f32(vp[t * op.v.st + vv]) : 0.0f;
            __syncthreads();
            const float before = op.reverse ? 1.0f : lam, after = op.reverse ? lam : 1.0f;
            float s = 0.0f;
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                const float n = before * S[j] + sk[wv * ROWS + j] * v;
                s += sq[wv * ROWS + j] * n;
                S[j] = after * n;
            }
            part[wv][col] = s;
            __syncthreads();
            o = op.inter * (part[0][col] + part[1][col] + part[2][col] + part[3][col]);
        }
        if (wv == 0 && live) {
            const int64_t at = ((b * a.T + t) * a.H + h) * op.DV + vv;
            if (op.o_f32) static_cast<float*>(op.o)[at] = o;
            else static_cast<T*>(op.o)[at] = from_f32<T>(o);
        }
    }
    if (op.s_out && live)
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int r = wv * ROWS + i;
            if (r < op.DK) op.s_out[sbase + static_cast<int64_t>(r) * op.DV + vv] = S[i];
        }
}

template <typename T>
hipError_t launch_recurrent(const LaArgs& a, hipStream_t st) {
    for (int w = 0; w < a.n_ops; ++w) {
        const dim3 grid(a.B * a.H, (a.op[w].DV + kCols - 1) / kCols);
        if (a.op[w].DK <= 128) la_recurrent<T, 32><<<grid, 256, 0, st>>>(a, w);
        else la_recurrent<T, 64><<<grid, 256, 0, st>>>(a, w);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <typename T>
__global__ __launch_bounds__(256) void la_group_sum(const float* in, T* out, int64_t n, int G, int D) {
    const int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (e >= n) return;
    const int64_t row = e / D;
    const int d = static_cast<int>(e - row * D);
    float s = 0.0f;
    for (int g = 0; g < G; ++g) s += in[(row * G + g) * D + d];
    out[e] = from_f32<T>(s);
}

template <typename T>
__global__ __launch_bounds__(256) void la_step(pn_linattn_step_args a) {
    __shared__ float sq[256], sk[256], part[4][kCols];
    const int tid = threadIdx.x, col = tid % kCols, wv = tid / kCols;
    const int H = static_cast<int>(a.H), DK = static_cast<int>(a.dk), DV = static_cast<int>(a.dv);
    const int h = blockIdx.x % H, b = blockIdx.x / H;
    const int vv = blockIdx.y * kCols + col;
    const bool live = vv < DV;
    const int64_t slot = a.slots ? a.slots[b] : b;
    T* o = static_cast<T*>(a.o) + (static_cast<int64_t>(b) * H + h) * DV;
    if (slot < 0 || slot >= a.n_slots) {
        if (wv == 0 && live) o[vv] = from_f32<T>(0.0f);
        return;
    }
    const int hk = h / static_cast<int>(a.H / a.HK);
    const T* qp = static_cast<const T*>(a.q.p) + b * a.q.sb + h * a.q.sh;
    const T* kp = static_cast<const T*>(a.k.p) + b * a.k.sb + hk * a.k.sh;
    const T* vp = static_cast<const T*>(a.v.p) + b * a.v.sb + hk * a.v.sh;
    sq[tid] = tid < DK ? to_f32(qp[tid]) : 0.0f;
    sk[tid] = tid < DK ? to_f32(kp[tid]) : 0.0f;
    const float v = live ? to_f32(vp[vv]) : 0.0f;
    __syncthreads();
    const float lam = expf(a.log_decay[h]);
    float* S = a.state + (slot * H + h) * DK * DV;
    float s = 0.0f;
    for (int r = wv; r < DK; r += 4)
        if (live) {
            const float n = lam * S[r * DV + vv] + sk[r] * v;
            S[r * DV + vv] = n;
            s += sq[r] * n;
        }
    part[wv][col] = s;
    __syncthreads();
    if (wv == 0 && live)
        o[vv] = from_f32<T>(static_cast<float>(a.scale) * (part[0][col] + part[1][col] + part[2][col] + part[3][col]));
}

}  // namespace

hipError_t launch_linattn(const LaArgs& a, hipStream_t st) {
    switch (a.dtype) {
        case PN_F32: return launch_recurrent<float>(a, st);
        case PN_BF16: return launch_recurrent<bf16>(a, st);
        default: return launch_recurrent<f16>(a, st);
    }
}

hipError_t launch_group_sum(const float* in, void* out, int dtype, int64_t rows, int G, int D, hipStream_t st) {
    const int64_t n = rows * D;
    const dim3 grid(static_cast<uint32_t>((n + 255) / 256));
    switch (dtype) {
        case PN_F32: la_group_sum<float><<<grid, 256, 0, st>>>(in, static_cast<float*>(out), n, G, D); break;
        case PN_BF16: la_group_sum<bf16><<<grid, 256, 0, st>>>(in, static_cast<bf16*>(out), n, G, D); break;
        default: la_group_sum<f16><<<grid, 256, 0, st>>>(in, static_cast<f16*>(out), n, G, D); break;
    }
    return hipGetLastError();
}

hipError_t launch_linattn_step(const pn_linattn_step_args& a, hipStream_t st) {
    const dim3 grid(static_cast<uint32_t>(a.B * a.H), static_cast<uint32_t>((a.dv + kCols - 1) / kCols));
    switch (a.dtype) {
        case PN_F32: la_step<float><<<grid, 256, 0, st>>>(a); break;
        case PN_BF16: la_step<bf16><<<grid, 256, 0, st>>>(a); break;
        default: la_step<f16><<<grid, 256, 0, st>>>(a); break;
    }
    return hipGetLastError();
}

}  // namespace pn
