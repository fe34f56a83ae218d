// Internal declarations of the state-space operators (pn_ssm*.hip,
// pn_conv.hip, pn_block_norm.hip) and their C entries (pn_ssm_api.cpp).
#pragma once

#include "pn_seq.hpp"

namespace pn {

// out[c] = sum over r of in[r * cols + c], in float64 and a fixed order
// (pn_ssm.hip).  Up to four parts of the columns, each with an output of its
// own (null: not wanted).
struct ColumnSum {
    const float* in;
    int64_t rows, cols;
    int n_parts;
    int64_t from[4];         // first column of each part
    float* out[4];
};
hipError_t launch_column_sum(const ColumnSum& s, hipStream_t st);

// Short convolution (pn_conv.hip).
hipError_t launch_conv(const pn_conv_args& a, hipStream_t st);
size_t conv_workspace(const pn_conv_args& a);
hipError_t launch_conv_backward(const pn_conv_args& a, hipStream_t st);
hipError_t launch_conv_state(const pn_conv_args& a, hipStream_t st);   // the backward of no token: d_initial_state
hipError_t launch_conv_step(const pn_conv_step_args& a, hipStream_t st);

// Norms around a block (pn_block_norm.hip).
hipError_t launch_block_norm(const pn_block_norm_args& a, hipStream_t st);
size_t block_norm_workspace(const pn_block_norm_args& a);
hipError_t launch_block_norm_backward(const pn_block_norm_args& a, hipStream_t st);

// Selective scan (pn_ssm.hip; its passes in pn_ssm_scan.hpp, built per
// storage type).
constexpr int kSsmTile = 8;      // tokens that a wave holds at a time
struct SsmPlan {
    int32_t states;              // padded states of a wave: 4, 8 or 16
    int32_t blocks;              // waves that share the states of a channel
    int32_t wide;                // channel blocks of a workgroup of the gradients
    int32_t per_group;           // blocks of 32 channels in a group of b and c (whole workgroups)
    int32_t chans;               // channel blocks in all
    int32_t n_seg;               // segments of the time axis
    int64_t seg, tiles;          // tokens per segment, tiles of a sequence
    // parts of the workspace, in floats
    int64_t ends, decay, rends, marks, since, part_bc, part_A, part_vec, total;
};
SsmPlan plan_ssm(const pn_ssm_args& a, bool backward);
bool ssm_fits(const pn_ssm_args& a, const SsmPlan& p);
hipError_t launch_ssm(const pn_ssm_args& a, const SsmPlan& p, hipStream_t st);
hipError_t launch_ssm_backward(const pn_ssm_args& a, const SsmPlan& p, hipStream_t st);
hipError_t launch_ssm_step(const pn_ssm_step_args& a, hipStream_t st);

// The passes of one storage type (T: float, bf16, f16).
enum SsmPass { kSsmEnds = 0, kSsmOutputs = 1, kSsmMarks = 2, kSsmMarksBoth = 3, kSsmGradients = 4 };
template <typename T>
hipError_t launch_ssm_pass(const pn_ssm_args& a, const SsmPlan& p, SsmPass pass, hipStream_t st);

}  // namespace pn
