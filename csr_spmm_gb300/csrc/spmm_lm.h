// Internal interfaces of the language-model operators (embedding, layer norm,
// token log probabilities and their gradients) between their host driver
// (spmm_lm_api.cu) and their kernel translation units.  Not part of the
// public ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "csr_spmm.h"

namespace spmm {

inline int lm_elem_size(spmm_type_t t) { return t == SPMM_F32 ? 4 : 2; }

// ---- the handle, for spmm_lm_api.cu (spmm_api.cu) ----
// The current device must be the handle's; *num_sms is its SM count.
spmm_status_t lm_device(spmm_handle_t h, int* num_sms);
// The handle's scratch for these operators, grown to at least `bytes` for a call on `st`.
spmm_status_t lm_scratch(spmm_handle_t h, size_t bytes, cudaStream_t st, char** base);

// ---- embedding and its gradient (spmm_embed.cu) ----
struct EmbedParams {
    const int* ids;
    int64_t tokens;
    const void* table;
    int64_t ld_table;
    int64_t vocab;
    int64_t dim;
    void* out;
    int64_t ld_out;
    float scale;
};
cudaError_t launch_embedding(spmm_type_t type, const EmbedParams& p, int num_sms,
                             cudaStream_t st);

struct EmbedGradParams {
    const int* ids;
    int64_t tokens;
    const void* dout;
    int64_t ld_dout;
    void* dtable;
    int64_t ld_dtable;
    int64_t vocab;
    int64_t dim;
    float scale;
    float beta;
};
size_t embed_grad_scratch(int64_t tokens, int64_t dim);
size_t embed_grad_scratch_upto(int64_t tokens, int64_t dim);   // of every call up to that
cudaError_t launch_embedding_grad(spmm_type_t type, spmm_type_t grad_type,
                                  const EmbedGradParams& p, char* scratch, int num_sms,
                                  cudaStream_t st);

// ---- layer norm and its gradient (spmm_norm.cu) ----
struct NormParams {
    const void* x;
    int64_t ldx;
    int64_t rows;
    int64_t dim;
    const void* weight;      // or NULL
    const void* bias;        // or NULL
    float eps;
    void* y;
    int64_t ldy;
    float* mean;             // or NULL
    float* rstd;             // or NULL
};
cudaError_t launch_layer_norm(spmm_type_t type, spmm_type_t param_type, const NormParams& p,
                              int num_sms, cudaStream_t st);

struct NormGradParams {
    const void* dy;
    int64_t ld_dy;
    const void* x;
    int64_t ldx;
    const float* mean;
    const float* rstd;
    const void* weight;      // or NULL
    int64_t rows;
    int64_t dim;
    void* dx;
    int64_t ld_dx;
    void* dweight;           // or NULL
    void* dbias;             // or NULL
    float* part;             // scratch: partial sums of dweight and dbias
    float* means;            // scratch: two means per row (set by the launch)
};
size_t norm_grad_scratch(int64_t rows, int64_t dim, int num_sms);
cudaError_t launch_layer_norm_grad(spmm_type_t type, spmm_type_t param_type,
                                   const NormGradParams& p, int num_sms, cudaStream_t st);

// ---- token log probabilities and their gradient (spmm_logprob.cu) ----
struct LogprobParams {
    const void* logits;
    int64_t ld;
    int64_t rows;
    int64_t vocab;
    float alpha;
    const int* targets;      // or NULL
    int top_k;
    float* logprob;          // or NULL (with targets)
    float* entropy;          // or NULL
    float* lse;              // or NULL
    float* top_logprob;      // [rows, top_k]
    int* top_index;          // [rows, top_k]
};
cudaError_t launch_token_logprob(spmm_type_t type, const LogprobParams& p, int num_sms,
                                 cudaStream_t st);

struct LogprobGradParams {
    const void* logits;
    int64_t ld;
    int64_t rows;
    int64_t vocab;
    float alpha;
    const int* targets;      // or NULL (with dlogprob)
    const float* lse;
    const float* entropy;    // or NULL (with dentropy)
    const float* dlogprob;   // or NULL
    const float* dentropy;   // or NULL
    void* dlogits;
    int64_t ld_out;
};
cudaError_t launch_token_logprob_grad(spmm_type_t type, const LogprobGradParams& p, int num_sms,
                                      cudaStream_t st);

}  // namespace spmm
