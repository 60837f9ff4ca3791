// Host driver of the language-model operators behind the C ABI in
// include/csr_spmm.h: argument validation and scratch; the kernels are in
// spmm_embed.cu, spmm_norm.cu and spmm_logprob.cu.  No step synchronises the
// stream; no device value is read back.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "spmm_lm.h"

using namespace spmm;

namespace {

constexpr int64_t MAX_COUNT = INT_MAX - 1;      // rows, tokens, ids: 32-bit indices
constexpr int64_t MAX_TOKENS = 1LL << 30;       // sorted tokens: room for padding in 32 bits
constexpr int64_t MAX_WIDTH = 1LL << 28;        // columns, likewise, and as grid rows of 8192

inline bool bad_type(spmm_type_t t) { return t != SPMM_F32 && t != SPMM_F16 && t != SPMM_BF16; }
// Parameters and gradients have the operands' type or binary32.
inline bool bad_pair(spmm_type_t t, spmm_type_t other) {
    return bad_type(t) || (other != t && other != SPMM_F32);
}
inline bool bad_count(int64_t n, int64_t most) { return n < 0 || n > most; }
inline bool short_ld(int64_t ld, int64_t cols) { return ld < std::max<int64_t>(1, cols); }

inline spmm_status_t launched(cudaError_t e) { return e == cudaSuccess ? SPMM_OK : SPMM_ERR_CUDA; }

}  // namespace

extern "C" {

spmm_status_t spmm_reserve_lm(spmm_handle_t h, int64_t rows, int64_t dim) {
    if (!h || bad_count(rows, MAX_TOKENS) || bad_count(dim, MAX_WIDTH))
        return SPMM_ERR_INVALID_ARGUMENT;
    int sms = 0;
    spmm_status_t s = lm_device(h, &sms);
    if (s != SPMM_OK) return s;
    char* base = nullptr;
    return lm_scratch(h, std::max(embed_grad_scratch_upto(rows, dim),
                                  norm_grad_scratch(rows, dim, sms)), nullptr, &base);
}

spmm_status_t spmm_embedding(spmm_handle_t h, spmm_type_t type, float scale, const int32_t* ids,
                             int64_t tokens, const void* table, int64_t ld_table, int64_t vocab,
                             int64_t dim, void* out, int64_t ld_out, void* stream) {
    if (!h || bad_type(type) || bad_count(tokens, MAX_COUNT) || bad_count(vocab, MAX_COUNT) ||
        bad_count(dim, MAX_WIDTH))
        return SPMM_ERR_INVALID_ARGUMENT;
    if (short_ld(ld_table, dim) || short_ld(ld_out, dim)) return SPMM_ERR_DIMENSION_MISMATCH;
    if (tokens == 0 || dim == 0) return SPMM_OK;
    if (scale == 0.0f) vocab = 0;                // zeros, the table not read
    if (!ids || !out || (vocab > 0 && !table)) return SPMM_ERR_NULL_POINTER;
    int sms = 0;
    spmm_status_t s = lm_device(h, &sms);
    if (s != SPMM_OK) return s;
    const EmbedParams p{ids, tokens, table, ld_table, vocab, dim, out, ld_out, scale};
    return launched(launch_embedding(type, p, sms, reinterpret_cast<cudaStream_t>(stream)));
}

spmm_status_t spmm_embedding_grad(spmm_handle_t h, spmm_type_t type, spmm_type_t grad_type,
                                  float scale, const int32_t* ids, int64_t tokens,
                                  const void* dout, int64_t ld_dout, float beta, void* dtable,
                                  int64_t ld_dtable, int64_t vocab, int64_t dim, void* stream) {
    if (!h || bad_pair(type, grad_type) || bad_count(tokens, MAX_TOKENS) ||
        bad_count(vocab, MAX_COUNT) || bad_count(dim, MAX_WIDTH))
        return SPMM_ERR_INVALID_ARGUMENT;
    if (short_ld(ld_dout, dim) || short_ld(ld_dtable, dim)) return SPMM_ERR_DIMENSION_MISMATCH;
    if (vocab == 0 || dim == 0) return SPMM_OK;
    if (scale == 0.0f) tokens = 0;               // dtable = beta * dtable, dout not read
    if (!dtable || (tokens > 0 && (!ids || !dout))) return SPMM_ERR_NULL_POINTER;
    int sms = 0;
    spmm_status_t s = lm_device(h, &sms);
    if (s != SPMM_OK) return s;
    char* scratch = nullptr;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    s = lm_scratch(h, embed_grad_scratch(tokens, dim), st, &scratch);
    if (s != SPMM_OK) return s;
    const EmbedGradParams p{ids,       tokens, dout, ld_dout, dtable,
                            ld_dtable, vocab,  dim,  scale,   beta};
    return launched(launch_embedding_grad(type, grad_type, p, scratch, sms, st));
}

spmm_status_t spmm_layer_norm(spmm_handle_t h, spmm_type_t type, spmm_type_t param_type,
                              const void* x, int64_t ldx, int64_t rows, int64_t dim,
                              const void* weight, const void* bias, float eps, void* y,
                              int64_t ldy, float* mean, float* rstd, void* stream) {
    if (!h || bad_pair(type, param_type) || bad_count(rows, MAX_COUNT) ||
        bad_count(dim, MAX_WIDTH) || !(eps >= 0.0f))
        return SPMM_ERR_INVALID_ARGUMENT;
    if (short_ld(ldx, dim) || short_ld(ldy, dim)) return SPMM_ERR_DIMENSION_MISMATCH;
    if (rows == 0 || dim == 0) return SPMM_OK;
    if (!x || !y) return SPMM_ERR_NULL_POINTER;
    int sms = 0;
    spmm_status_t s = lm_device(h, &sms);
    if (s != SPMM_OK) return s;
    const NormParams p{x, ldx, rows, dim, weight, bias, eps, y, ldy, mean, rstd};
    return launched(launch_layer_norm(type, param_type, p, sms,
                                      reinterpret_cast<cudaStream_t>(stream)));
}

spmm_status_t spmm_layer_norm_grad(spmm_handle_t h, spmm_type_t type, spmm_type_t param_type,
                                   const void* dy, int64_t ld_dy, const void* x, int64_t ldx,
                                   const float* mean, const float* rstd, const void* weight,
                                   int64_t rows, int64_t dim, void* dx, int64_t ld_dx,
                                   void* dweight, void* dbias, void* stream) {
    if (!h || bad_pair(type, param_type) || bad_count(rows, MAX_COUNT) ||
        bad_count(dim, MAX_WIDTH))
        return SPMM_ERR_INVALID_ARGUMENT;
    if (short_ld(ld_dy, dim) || short_ld(ldx, dim) || short_ld(ld_dx, dim))
        return SPMM_ERR_DIMENSION_MISMATCH;
    if (dim == 0 || (rows == 0 && !dweight && !dbias)) return SPMM_OK;
    if (rows > 0 && (!dy || !x || !mean || !rstd || !dx)) return SPMM_ERR_NULL_POINTER;
    int sms = 0;
    spmm_status_t s = lm_device(h, &sms);
    if (s != SPMM_OK) return s;
    char* scratch = nullptr;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    s = lm_scratch(h, norm_grad_scratch(rows, dim, sms), st, &scratch);
    if (s != SPMM_OK) return s;
    const NormGradParams p{dy, ld_dy, x,     ldx,     mean,  rstd, weight, rows,
                           dim, dx,   ld_dx, dweight, dbias, reinterpret_cast<float*>(scratch),
                           nullptr};
    return launched(launch_layer_norm_grad(type, param_type, p, sms, st));
}

spmm_status_t spmm_token_logprob(spmm_handle_t h, spmm_type_t type, float alpha,
                                 const void* logits, int64_t ld, int64_t rows, int64_t vocab,
                                 const int32_t* targets, int32_t top_k, float* logprob,
                                 float* entropy, float* lse, float* top_logprob,
                                 int32_t* top_index, void* stream) {
    if (!h || bad_type(type) || bad_count(rows, MAX_COUNT) || bad_count(vocab, MAX_COUNT) ||
        !(alpha > 0.0f) || std::isinf(alpha) || top_k < 0 || top_k > SPMM_TOP_MAX)
        return SPMM_ERR_INVALID_ARGUMENT;
    if (short_ld(ld, vocab)) return SPMM_ERR_DIMENSION_MISMATCH;
    if (rows == 0) return SPMM_OK;
    if ((vocab > 0 && !logits) || !targets != !logprob ||
        (top_k > 0 && (!top_logprob || !top_index)))
        return SPMM_ERR_NULL_POINTER;
    int sms = 0;
    spmm_status_t s = lm_device(h, &sms);
    if (s != SPMM_OK) return s;
    const LogprobParams p{logits,  ld,      rows, vocab,       alpha,    targets, top_k,
                          logprob, entropy, lse,  top_logprob, top_index};
    return launched(launch_token_logprob(type, p, sms, reinterpret_cast<cudaStream_t>(stream)));
}

spmm_status_t spmm_token_logprob_grad(spmm_handle_t h, spmm_type_t type, float alpha,
                                      const void* logits, int64_t ld, int64_t rows,
                                      int64_t vocab, const int32_t* targets, const float* lse,
                                      const float* entropy, const float* dlogprob,
                                      const float* dentropy, void* dlogits, int64_t ld_dlogits,
                                      void* stream) {
    if (!h || bad_type(type) || bad_count(rows, MAX_COUNT) || bad_count(vocab, MAX_COUNT) ||
        !(alpha > 0.0f) || std::isinf(alpha))
        return SPMM_ERR_INVALID_ARGUMENT;
    if (short_ld(ld, vocab) || short_ld(ld_dlogits, vocab)) return SPMM_ERR_DIMENSION_MISMATCH;
    if (rows == 0 || vocab == 0) return SPMM_OK;
    if (!logits || !lse || !dlogits || !targets != !dlogprob || (dentropy && !entropy))
        return SPMM_ERR_NULL_POINTER;
    int sms = 0;
    spmm_status_t s = lm_device(h, &sms);
    if (s != SPMM_OK) return s;
    const LogprobGradParams p{logits, ld,      rows,     vocab,    alpha,   targets,
                              lse,    entropy, dlogprob, dentropy, dlogits, ld_dlogits};
    return launched(launch_token_logprob_grad(type, p, sms,
                                              reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
