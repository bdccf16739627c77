// See tv_filtered.cuh.
#define TV_FILT_THREADS 256
#define TV_FILT_SPACE threads_256
#include "tv_filtered.cuh"

namespace tv {

int launch_filtered_256(bool sampling, int dtype, FiltParams& p, void* stream) {
  return sampling ? threads_256::launch_filtered<true>(dtype, p, stream) : threads_256::launch_filtered<false>(dtype, p, stream);
}

}  // namespace tv
