// va_weights.cuh -- parameters shared by the weight kernels and their host code.
#pragma once

#include "va_chunk.cuh"

namespace va {

// Clusters of the tensor-core kernel that a GB300's 152 SMs hold at most; the
// workspace is sized for them, so that sizing it takes no device call.
constexpr int kWeightClusters = 152;

struct WeightTcParams {
  ChunkParams c;
  const float* win;
  float* wout;
  int clusters, tile_keys;
  uint32_t* cta_flags;   // [152] status bits of each CTA
  int32_t* cont_entry;   // [clusters] first entry of the key tile a run begins inside of, or -1
  float* cont;           // [clusters][256] that tile's share
  float* sums;           // [num_entries] every other share
};

cudaError_t init_weights_tc();
cudaError_t launch_weights_tc(const WeightTcParams& p, bool pair, cudaStream_t st);

}  // namespace va
