// kda_serve.cuh -- launchers of the operators of a decode step over few tokens (arguments validated
// by the caller): 4-bit weights, the mixture of experts, the verification of drafts.
#pragma once

#include "kda_internal.cuh"

namespace kda {

cudaError_t launch_pack4(const kda_pack4_args& a, cudaStream_t s);
cudaError_t launch_unpack4(const kda_pack4_args& a, cudaStream_t s);
size_t gemm4_workspace(const kda_gemm4_args& a);
cudaError_t launch_gemm4(const kda_gemm4_args& a, cudaStream_t s);

// Parts of kda_moe's workspace, as byte offsets.
struct MoePlan {
    size_t logits;    // [M][E] pairs of fp32
    size_t key;      // [M][E] uint64: what the choice is made by, ordered as integers
    size_t done;     // int: tokens whose choice is made
    size_t ids;      // [M * top] int: experts by token and rank
    size_t weights;  // [M * top] fp32
    size_t lists;    // int: [1] experts in use, [E] which, [E + 1] where their slots begin, [M * top] slots
    size_t x_columns; // the tokens' columns: digits and scales (e2m1 experts), bf16 rows, or fp16 and factors (integer codes)
    size_t hidden;    // the same of the hidden values: eight digits, four bf16 or two fp16 columns each
    size_t parts;    // [M * top][D] fp32
    size_t workspace;
};
MoePlan moe_plan(const kda_moe_args& a);
cudaError_t launch_moe(const kda_moe_args& a, const MoePlan& p, cudaStream_t s);

cudaError_t launch_verify(const kda_verify_args& a, cudaStream_t s);

// log2(group / 32) of a supported group (32, 64, 128).
inline int group_shift(int group) { return group == 128 ? 2 : group == 64 ? 1 : 0; }

}  // namespace kda
