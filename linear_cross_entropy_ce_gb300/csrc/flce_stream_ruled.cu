// The streaming form of the constrained log probabilities: launches.
#include "flce_stream.cuh"

namespace flce {

cudaError_t stream_ruled_prepare() { return prepare_all<LISTS_RULED>(); }

cudaError_t launch_stream_ruled(const StreamArgs& a, const StreamMaps& m, const StreamLists& l, bool beside,
                                cudaStream_t s) {
  const cudaError_t e = launch_all<LISTS_RULED>(a, m, l, beside, s);
  if (e != cudaSuccess) return e;
  return launch_dependent(logprob_stream_merge_kernel<true>, a.N, MERGE_THREADS, s, a, l.lists);
}

}  // namespace flce
