// decay_tc_128.cu -- the tensor-core passes of decay_tc.cuh for heads of 128 columns.
#include "decay_tc.cuh"

namespace slim {
namespace decay {

cudaError_t tc_passes_128(const TcArgs &a, bool total, bool rev, bool grouped, cudaStream_t st) {
  return launch_passes<128>(a, total, rev, grouped, st);
}

}  // namespace decay
}  // namespace slim
