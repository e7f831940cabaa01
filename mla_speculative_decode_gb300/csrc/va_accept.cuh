// va_accept.cuh -- the walk of a draft tree along the target's tokens, shared by greedy
// acceptance (va_accept.cu) and acceptance by sampling (va_sample.cu).
#pragma once

#include "va_common.cuh"

namespace va {

struct AcceptParams {
  const float* root_logits;   // [B, V]
  const float* logits;        // [B, T, V]
  int64_t V;
  const int32_t* tokens;      // [B, T]
  const int32_t* parent;      // [B, T]
  const int32_t* slots;       // [B, T] or NULL
  int B, T, chunks;
  int64_t chunk_len;
  float* part_val;            // [B*(T+1)][chunks]
  int32_t* part_idx;          // [B*(T+1)][chunks]
  bool flag_empty;            // a row at -inf sets VA_STATUS_EMPTY_ROW
  uint32_t* status;
  int32_t* accept_len;        // [B]
  int32_t* accept_nodes;      // [B, T]
  int32_t* accept_slots;      // [B, T] or NULL
  int32_t* bonus;             // [B]
};

// One kernel, a programmatic dependent of the one that wrote part_val and part_idx (and
// cleared the status word).
cudaError_t launch_accept_walk(const AcceptParams& a, cudaStream_t st);

}  // namespace va
