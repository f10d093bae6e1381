// ssu_hybrid.h -- parameters shared by the host layer and the kernels of the
// operators around the state update: linear attention on the slot pool, the
// residual-adding RMS norm, token log probabilities.  Not part of the public
// ABI (that is include/ssu.h).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "ssu_internal.h"

namespace ssu {

// Linear attention with a decay for each head (ssu_linattn_step.cu,
// ssu_linattn_prefill.cu).  Strides are in elements: [token, head]; the
// innermost stride is one.
struct LinattnParams {
    int64_t slots, rows, nseq;
    int32_t H, G, share;  // heads, key/value heads, heads / key/value heads
    int32_t P, N;         // dim (values), dstate (keys)
    int32_t io_dtype, state_dtype;
    float scale;
    int64_t pad;
    void *state;
    const void *q, *k, *v;
    const float *log_decay;
    void *out;
    int64_t qs[2], ks[2], vs[2], os[2];
    SlotTab rd, wr;
    const void *cu;  // prefill: [nseq + 1]
    int32_t meta_is_i64;
    int32_t *status;
};
constexpr int kLinattnMaxDim = 128;  // largest dim and dstate

cudaError_t launch_linattn_step(const LinattnParams &p, cudaStream_t stream);
// How a prefill is split over the GPU, and the workspace it needs for that:
// byte offsets of its parts (bytes == 0: none, one unit per CTA).
struct LinattnSplit {
    int64_t cut_len;   // sequences longer than this are cut
    int64_t max_cuts, max_states;  // most sequences that can be, and pieces that makes
    uint64_t cuts, pieces, states, bytes;
};
LinattnSplit linattn_split(int64_t rows, int64_t nseq, int64_t heads, int64_t dim, int64_t dstate, int64_t max_seqlen);
cudaError_t launch_linattn_prefill(const LinattnParams &p, const LinattnSplit &split, void *workspace, cudaStream_t stream);

// RMS norm (ssu_norm.cu).
enum : int32_t { kQuantNone = 0, kQuantRow = 1, kQuantBlock = 2 };
constexpr int kNormBlock = 128;       // columns of one scale (kQuantBlock)
constexpr int kNormMaxHidden = 32768;  // a row is held by one CTA's registers
struct NormParams {
    int64_t rows;
    int32_t hidden, dtype, weight_dtype, quant;
    float eps;
    const void *x, *residual, *weight;
    void *residual_out, *y;
    float *scales;
    int64_t xs, rs, ros, ys;  // row strides (elements)
};
cudaError_t launch_norm(const NormParams &p, cudaStream_t stream);

// Token log probabilities (ssu_logprobs.cu).
constexpr int kMaxTopK = 32;
struct LogprobParams {
    int64_t rows, row_stride;
    int32_t vocab, dtype, top_k, tok_is_i64;
    const void *logits, *tokens;
    float *logprob, *entropy, *top_logprob;
    void *top_ids;  // the tokens' integer type
    int32_t *status;
};
cudaError_t launch_logprobs(const LogprobParams &p, cudaStream_t stream);

}  // namespace ssu
