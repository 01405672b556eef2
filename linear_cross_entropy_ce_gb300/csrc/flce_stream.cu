// The streaming form of the token log probabilities without lists: launches.
#include "flce_stream.cuh"

namespace flce {
namespace {

__global__ void clear_groups_kernel(uint32_t* group_max, int n) {
  ptx::grid_launch_dependents();
  for (int i = threadIdx.x; i < n; i += blockDim.x) group_max[i] = 0u;
}

}  // namespace

int stream_max_tiles(long long V, int ctas) {
  return static_cast<int>(cdiv(cdiv(cdiv(V, UNIT_ROWS), ctas), TILE_ROWS / UNIT_ROWS));
}

int stream_ctas(long long V, int sms) {
  const long long units = cdiv(V, UNIT_ROWS);
  return static_cast<int>(units < sms ? units : sms);
}

cudaError_t stream_prepare() {
  cudaError_t e = prepare_all<LISTS_NONE>();
  if (e == cudaSuccess) e = stream_ruled_prepare();
  if (e == cudaSuccess) e = stream_taken_prepare();
  return e;
}

int stream_tokens(int N) { return N <= 16 ? 16 : (N <= 32 ? 32 : (N <= 64 ? 64 : 128)); }

cudaError_t launch_stream(const StreamArgs& a, const StreamMaps& m, cudaStream_t s) {
  if (a.group_max) {
    clear_groups_kernel<<<1, 512, 0, s>>>(a.group_max, a.N * TopK::MAX);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const cudaError_t e = launch_all<LISTS_NONE>(a, m, StreamLists{}, a.group_max != nullptr, s);
  if (e != cudaSuccess) return e;
  return launch_dependent(logprob_stream_merge_kernel<false>, a.N, MERGE_THREADS, s, a, ListView{});
}

}  // namespace flce
