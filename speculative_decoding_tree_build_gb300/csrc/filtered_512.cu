// tv_filter_logits: see tv_filtered.cuh.
#define TV_FILT_SPACE masking
#define TV_FILT_THREADS 512
#include "tv_filtered.cuh"

extern "C" int tv_filter_logits(int32_t dtype, const void* logits, int64_t logits_ld, const int32_t* cu_nodes,
                                const float* temperature, const int32_t* top_k, const float* top_p,
                                const float* min_p, int32_t batch, int32_t max_nodes, int32_t vocab, void* out,
                                int64_t out_ld, int32_t* kept, int32_t* status, void* stream) {
  int rc = tv::masking::check_filter(dtype, logits, logits_ld, batch, max_nodes, vocab);
  if (rc != TV_OK) return rc;
  if (out_ld < vocab) return TV_ERR_BAD_SIZE;
  if (batch == 0) return TV_OK;
  if (!logits || !cu_nodes || !temperature || !out || !status) return TV_ERR_NULL_POINTER;
  const int per = dtype == TV_DTYPE_F32 ? 4 : 8;
  if (!tv::aligned(logits, 16) || logits_ld % per || !tv::aligned(out, 16) || out_ld % per) return TV_ERR_MISALIGNED;
  tv::masking::FiltParams p = {};
  p.logits = logits; p.logits_ld = logits_ld;
  p.cu_nodes = cu_nodes; p.temperature = temperature; p.top_k = top_k; p.top_p = top_p; p.min_p = min_p;
  p.max_nodes = max_nodes; p.vocab = vocab; p.out = out; p.out_ld = out_ld; p.kept = kept; p.status = status;
  return tv::masking::launch_filtered<false>(dtype, p, batch, stream);
}
