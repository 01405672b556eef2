// The streaming form of the distillation loss: launch.
#include "flce_stream.cuh"

namespace flce {

cudaError_t stream_taken_prepare() { return prepare_all<LISTS_TAKEN>(); }

cudaError_t launch_stream_taken(const StreamArgs& a, const StreamMaps& m, const StreamLists& l, cudaStream_t s) {
  return launch_all<LISTS_TAKEN>(a, m, l, true, s);
}

}  // namespace flce
