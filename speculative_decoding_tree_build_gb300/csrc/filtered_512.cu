// See tv_filtered.cuh.
#define TV_FILT_THREADS 512
#define TV_FILT_SPACE threads_512
#include "tv_filtered.cuh"

namespace tv {

int launch_filtered_512(bool sampling, int dtype, FiltParams& p, void* stream) {
  return sampling ? threads_512::launch_filtered<true>(dtype, p, stream) : threads_512::launch_filtered<false>(dtype, p, stream);
}

}  // namespace tv
