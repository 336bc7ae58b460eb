// mt_seq.h -- interface between the C-ABI layer of the sequence-model calls
// (mt_seq_abi.cu) and their kernels. Not installed; not part of the public ABI.
#pragma once

#include "mt_internal.h"
#include "mt_scan.h"

namespace mt {

// ---- embedding lookup and its table's gradient (mt_embed.cu) ------------------
struct EmbedGradPlan {
    int64_t rows_per_cta;  // table rows whose tokens one CTA of the sort places
    int64_t ctas;          // CTAs of the sort
    int64_t piece;         // sorted tokens per piece of the sum
    int64_t pieces;
    int64_t start_slots, order_slots, last_slots, partial_slots;  // 8-byte slots of the scratch's parts
};
EmbedGradPlan embed_grad_plan(int64_t tokens, int64_t vocab, int64_t dim);
cudaError_t embed_launch(const void *tokens, bool wide_tokens, int64_t ntokens, const void *table, int64_t vocab,
                         int64_t dim, int dtype, float scale, void *out, const Launch &L);
cudaError_t embed_grad_launch(const void *tokens, bool wide_tokens, int64_t ntokens, const void *dout, int dtype,
                              int64_t vocab, int64_t dim, float scale, void *dtable, int grad_dtype, bool accumulate,
                              uint64_t *scratch, const Launch &L);

// ---- short causal convolution (mt_conv.cu) -------------------------------------
int64_t conv_grad_scratch_slots(int64_t batch, int64_t len, int64_t dim, int64_t width);
cudaError_t conv_launch(const mt_conv_args &a, const Launch &L);
cudaError_t conv_step_launch(const mt_conv_args &a, const Launch &L);
cudaError_t conv_grad_launch(const mt_conv_args &a, const Launch &L);

// ---- selective state space scan (mt_ssm*.cu) -----------------------------------
constexpr int kSsmTile = 8;  // tokens per checkpoint
struct SsmPlan {
    int lanes;         // lanes that share a channel's states, four states each
    int64_t segments;  // pieces of the token axis that run side by side
    int64_t seg_len;   // tokens per segment, a multiple of 8
    int64_t ctiles;    // channel tiles per group (forward: of a warp; gradient: of a CTA)
    int64_t carry_slots, decay_slots, shared_slots, param_slots;  // 8-byte slots of the scratch's parts
};
SsmPlan ssm_plan(int64_t batch, int64_t len, int64_t dim, int64_t nstate, int64_t groups, bool grad, bool lens);
cudaError_t ssm_launch(const mt_ssm_args &a, const Launch &L);
cudaError_t ssm_grad_launch(const mt_ssm_args &a, const Launch &L);
cudaError_t ssm_step_launch(const mt_ssm_args &a, const Launch &L);

// ---- gated scan (mt_gated*.cu) ---------------------------------------------------
constexpr int kGatedTile = 16;  // tokens per checkpoint
constexpr int64_t kGatedMost = INT32_MAX - 65536;  // tokens of a sequence: they are counted in 32 bits
int64_t gated_scratch_slots(int64_t batch, int64_t len, int64_t dim);
cudaError_t gated_launch(const mt_gated_args &a, const Launch &L);
cudaError_t gated_step_launch(const mt_gated_args &a, const Launch &L);
cudaError_t gated_grad_launch(const mt_gated_args &a, const Launch &L);
cudaError_t gated_f32_take_error(int *code);  // of each translation unit's error word
cudaError_t gated_bf16_take_error(int *code);
cudaError_t gated_f16_take_error(int *code);
cudaError_t gated_grad_f32_take_error(int *code);
cudaError_t gated_grad_bf16_take_error(int *code);
cudaError_t gated_grad_f16_take_error(int *code);

// ---- beam search's selection (mt_beam.cu) and copies between slots (mt_copy.cu) ----
constexpr int kBeamsMost = 32;
int64_t beam_scratch_slots(int64_t batch, int64_t beams, int64_t beams_out, int64_t vocab);
cudaError_t beam_launch(const mt_beam_args &a, const Launch &L);
cudaError_t copy_launch(const int32_t *src, const int32_t *dst, int64_t pairs, const mt_pool *pools, int64_t npools,
                        const Launch &L);

}  // namespace mt
