// decay_tc_64.cu -- the tensor-core passes of decay_tc.cuh for heads of 64 columns.
#include "decay_tc.cuh"

namespace slim {
namespace decay {

cudaError_t tc_passes_64(const TcArgs &a, bool total, bool rev, bool grouped, cudaStream_t st) {
  return launch_passes<64>(a, total, rev, grouped, st);
}

}  // namespace decay
}  // namespace slim
