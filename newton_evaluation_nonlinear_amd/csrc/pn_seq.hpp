// Internal declarations of the sequence-layer operators (pn_rotary.hip,
// pn_linattn.hip) and their C entries (pn_seq_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/pn.h"

namespace pn {

// pn_api.cpp: the calling thread's error message.
int set_error(int code, const char* msg);
void clear_error();

// A launch of `blocks` workgroups, along x and y: HIP takes less than 2^32
// threads along one of them.  The last of them have no work (block_id()).
inline dim3 grid_of(int64_t blocks, int threads) {
    const int64_t most = (int64_t(1) << 31) / threads, x = blocks < most ? blocks : most;
    return dim3(static_cast<uint32_t>(x), static_cast<uint32_t>((blocks + x - 1) / x));
}

hipError_t launch_rotary_table(const double* freq, int n_freq, int64_t n_pos, double magnitude, float* table,
                               hipStream_t st);

enum RotaryPass { kRotate = 0, kNormRotate = 1 };
hipError_t launch_rotary(const pn_rotary_args& a, RotaryPass pass, hipStream_t st);
size_t rotary_backward_workspace(const pn_rotary_args& a);
hipError_t launch_fill(float* p, int64_t n, hipStream_t st);   // zeros (pn_rotary.hip)
hipError_t launch_rotary_backward(const pn_rotary_args& a, hipStream_t st);

// One causal operator with a decay and a matrix state (pn_linattn.hip):
//     S_i = lam S_{i-1} + ws K_i^T V_i,   O_i = inter * Q_i S_i.
// Forward attention is one; each of the gradients of q, k and v is another,
// with the operands in other places and, for k and v, time reversed.
struct LaOperand {
    const void* p;
    int64_t sb, st, sh;      // st is 0 for a single token
    int32_t div;             // head h of the operator reads head h / div
};
struct LaOp {
    LaOperand q, k, v;
    void* o;                 // [B, T, H, DV], float32 if o_f32, else the storage type
    int32_t o_f32;
    int32_t reverse;         // 1: i runs from the last token to the first, and lam applies
                             //    after a token instead of before it
    int32_t DK, DV;
    float inter;             // scale of the output
    float ws;                // scale of K^T V in the state
    const float* s_in;       // [B, H, ., .] or null; element (x, y) at x * s_k + y * s_v
    int32_t s_k, s_v;
    float* s_out;            // [B, H, DK, DV] or null
    int32_t exact;           // 1: the state is a result, not only a term of 16-bit outputs
    int32_t carry_from;      // the operator whose states between segments this one reads
};
struct LaArgs {
    LaOp op[3];
    int32_t n_ops;
    int32_t dtype;
    int32_t B, H;
    int64_t T;
    const float* log_decay;
    const int32_t* lengths;
};
size_t linattn_workspace(const LaArgs& a);      // bytes; sizes of `a` only
bool linattn_fits(const LaArgs& a);             // whether its launches can be made
hipError_t launch_linattn(const LaArgs& a, void* workspace, hipStream_t st);
// out[b, t, x, d] = sum over g of in[b, t, x * G + g, d]
hipError_t launch_group_sum(const float* in, void* out, int dtype, int64_t rows, int G, int D, hipStream_t st);
hipError_t launch_linattn_step(const pn_linattn_step_args& a, hipStream_t st);

}  // namespace pn
