// decay_tc_args.h -- what the host and the tensor-core kernels of the decay attention share.
#pragma once

#include <cuda.h>

#include "decay.h"

namespace slim {
namespace decay {

// Passes of one direction in one launch.
struct TcArgs {
  CUtensorMap maps[4], outs[3];
  Work work;
  const float *log_decay;
  int *status;
  int mixes;
  Mix mix[3];
  signed char a[3], b[3], c[3];  // the operands' maps
};

// decay_tc_64.cu, decay_tc_128.cu
cudaError_t tc_passes_64(const TcArgs &a, bool total, bool rev, bool grouped, cudaStream_t st);
cudaError_t tc_passes_128(const TcArgs &a, bool total, bool rev, bool grouped, cudaStream_t st);

}  // namespace decay
}  // namespace slim
