// tv_sample_filtered and tv_filter_logits: checks, and which of the kernel's two forms
// (tv_filtered.cuh) makes the call.
#include "tv_common.cuh"
#include "tv_filter_params.h"

namespace tv {

// Rows that are looked at more than once (masks; top-p without top-k) go to CTAs of 512
// threads where they are long, since half as many rows are then in flight and stay in L2, or
// where they are few, since a row then takes less time. Short rows in large calls go to
// 256 threads, as do rows that one look settles (us, 512 and 256 threads):
//   masks, 2064 rows of 32000 in bf16           232  160    (65536: 282  236)
//   masks, 2064 rows of 128256 in bf16          445  560
//   masks, 512 rows of 50000 in bf16            152  183
//   top-p 0.95, 2064 rows of 32000 in float32   281  230    (65536: 390  354)
//   top-p 0.95, 2064 rows of 151936 in float32  677  789
//   top-p 0.9, 512 rows of 65536 in bf16        226  305
//   top-k 64, 4112 rows of 151936 in float32    758  592
constexpr int kLongRow = 1 << 16;
constexpr int kResident = 4;               // CTAs of 256 threads an SM

static int launch_form(bool sampling, bool looks, int dtype, FiltParams& p, void* stream) {
  const int dev = current_device();
  const int sms = dev < 0 ? -1 : device_sm_count(dev);
  if (sms <= 0) return TV_ERR_CUDA;
  const bool wide = looks && (p.vocab > kLongRow || static_cast<long long>(p.batch) * p.max_nodes <= sms * kResident);
  return (wide ? launch_filtered_512 : launch_filtered_256)(sampling, dtype, p, stream);
}

static int check_filter(int dtype, const void* logits, long long ld, int batch, int max_nodes, int vocab) {
  if (dtype != TV_DTYPE_BF16 && dtype != TV_DTYPE_F32) return TV_ERR_BAD_GEOMETRY;
  if (batch < 0 || batch > 65535 || max_nodes < 1 || max_nodes > TV_MAX_NODES || vocab < 1 || vocab > (1 << 30) || ld < vocab)
    return TV_ERR_BAD_SIZE;
  return TV_OK;
}

}  // namespace tv

extern "C" int tv_sample_filtered(int32_t dtype, const void* logits, int64_t logits_ld, const float* gumbel,
                                  int64_t gumbel_ld, const int32_t* cu_nodes, const float* temperature,
                                  const int32_t* top_k, const float* top_p, const float* min_p, int32_t batch,
                                  int32_t max_nodes, int32_t vocab, int32_t* tokens, float* logp, int32_t* status,
                                  void* stream) {
  int rc = tv::check_filter(dtype, logits, logits_ld, batch, max_nodes, vocab);
  if (rc != TV_OK) return rc;
  if (gumbel && gumbel_ld < vocab) return TV_ERR_BAD_SIZE;
  if (batch == 0) return TV_OK;
  if (!logits || !cu_nodes || !temperature || !tokens || !status) return TV_ERR_NULL_POINTER;
  const int per = dtype == TV_DTYPE_F32 ? 4 : 8;
  if (!tv::aligned(logits, 16) || logits_ld % per || (gumbel && (!tv::aligned(gumbel, 16) || gumbel_ld % 4)))
    return TV_ERR_MISALIGNED;
  tv::FiltParams p = {};
  p.logits = logits; p.logits_ld = logits_ld; p.gumbel = gumbel; p.gumbel_ld = gumbel_ld;
  p.cu_nodes = cu_nodes; p.temperature = temperature; p.top_k = top_k; p.top_p = top_p; p.min_p = min_p;
  p.batch = batch; p.max_nodes = max_nodes; p.vocab = vocab; p.tokens = tokens; p.logp = logp; p.status = status;
  return tv::launch_form(true, top_p && !top_k, dtype, p, stream);
}

extern "C" int tv_filter_logits(int32_t dtype, const void* logits, int64_t logits_ld, const int32_t* cu_nodes,
                                const float* temperature, const int32_t* top_k, const float* top_p,
                                const float* min_p, int32_t batch, int32_t max_nodes, int32_t vocab, void* out,
                                int64_t out_ld, int32_t* kept, int32_t* status, void* stream) {
  int rc = tv::check_filter(dtype, logits, logits_ld, batch, max_nodes, vocab);
  if (rc != TV_OK) return rc;
  if (out_ld < vocab) return TV_ERR_BAD_SIZE;
  if (batch == 0) return TV_OK;
  if (!logits || !cu_nodes || !temperature || !out || !status) return TV_ERR_NULL_POINTER;
  const int per = dtype == TV_DTYPE_F32 ? 4 : 8;
  if (!tv::aligned(logits, 16) || logits_ld % per || !tv::aligned(out, 16) || out_ld % per) return TV_ERR_MISALIGNED;
  tv::FiltParams p = {};
  p.logits = logits; p.logits_ld = logits_ld;
  p.cu_nodes = cu_nodes; p.temperature = temperature; p.top_k = top_k; p.top_p = top_p; p.min_p = min_p;
  p.batch = batch; p.max_nodes = max_nodes; p.vocab = vocab; p.out = out; p.out_ld = out_ld; p.kept = kept; p.status = status;
  return tv::launch_form(false, true, dtype, p, stream);
}
