// What the entry points of filtered sampling hand to the kernel's two forms.
#pragma once

#include <cstdint>

namespace tv {

struct FiltParams {
  const void* logits;
  long long logits_ld;
  const float* gumbel;
  long long gumbel_ld;
  const int32_t* cu_nodes;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int max_nodes, vocab, bits;
  int csize;                   // CTAs of a cluster
  int rows, batch;             // rows = batch * max_nodes
  bool reorder;
  int32_t* tokens;
  float* logp;
  void* out;
  long long out_ld;
  int32_t* kept;
  int32_t* status;
};

// The kernel with CTAs of 256 threads, four an SM, and of 512 threads, two an SM.
int launch_filtered_256(bool sampling, int dtype, FiltParams& p, void* stream);
int launch_filtered_512(bool sampling, int dtype, FiltParams& p, void* stream);

}  // namespace tv
