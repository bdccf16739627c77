// tv_sample_filtered: see tv_filtered.cuh, whose kernel this unit compiles for
// sampling (the masks are compiled apart, beside it).
#define TV_FILT_SPACE sampling
#define TV_FILT_THREADS 256
#include "tv_filtered.cuh"

extern "C" int tv_sample_filtered(int32_t dtype, const void* logits, int64_t logits_ld, const float* gumbel,
                                  int64_t gumbel_ld, const int32_t* cu_nodes, const float* temperature,
                                  const int32_t* top_k, const float* top_p, const float* min_p, int32_t batch,
                                  int32_t max_nodes, int32_t vocab, int32_t* tokens, float* logp, int32_t* status,
                                  void* stream) {
  int rc = tv::sampling::check_filter(dtype, logits, logits_ld, batch, max_nodes, vocab);
  if (rc != TV_OK) return rc;
  if (gumbel && gumbel_ld < vocab) return TV_ERR_BAD_SIZE;
  if (batch == 0) return TV_OK;
  if (!logits || !cu_nodes || !temperature || !tokens || !status) return TV_ERR_NULL_POINTER;
  const int per = dtype == TV_DTYPE_F32 ? 4 : 8;
  if (!tv::aligned(logits, 16) || logits_ld % per || (gumbel && (!tv::aligned(gumbel, 16) || gumbel_ld % 4)))
    return TV_ERR_MISALIGNED;
  tv::sampling::FiltParams p = {};
  p.logits = logits; p.logits_ld = logits_ld; p.gumbel = gumbel; p.gumbel_ld = gumbel_ld;
  p.cu_nodes = cu_nodes; p.temperature = temperature; p.top_k = top_k; p.top_p = top_p; p.min_p = min_p;
  p.max_nodes = max_nodes; p.vocab = vocab; p.tokens = tokens; p.logp = logp; p.status = status;
  return tv::sampling::launch_filtered<true>(dtype, p, batch, stream);
}
