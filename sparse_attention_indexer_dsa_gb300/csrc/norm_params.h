// Parameter blocks and launchers of the query/key norms with rotation
// (norm_rope.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace dsa {

// Angles as fixed-point turns: a position times 64 bits of frequency, modulo
// one turn, is exact wherever the position is.
struct RopeTable {
  uint64_t freq[64];   // turns per position, in units of 2^-64
  int dim;             // rotated dimensions (first ones of the head), a multiple of 8
  int interleaved;     // pairs (2i, 2i + 1) instead of (i, i + dim / 2)
};

struct NormRopeParams {
  RopeTable rope;
  const void* x[2];          // queries, keys
  int64_t x_stride[2];       // elements from one token to the next
  void* y[2];
  int64_t y_stride[2];
  const void* w[2];          // null: ones
  const void* b[2];          // null: zeros
  const int32_t* pos;
  int heads[2];
  int tokens;
  int share, parts;          // rows of a token that a warp takes, such shares of a token
  float eps;
  int layer, in_bf16, out_bf16, w_bf16;
};

struct NormRopeBackParams {
  NormRopeParams f;          // y: gradients of the inputs (in_bf16); b unused
  const void* dy[2];
  int64_t dy_stride[2];
  int dy_bf16;
  float* dw[2];              // null: not wanted
  float* db[2];
  float* part;               // [blocks][4][D]: dw of queries and keys, db of both
  int* hdr;
};

constexpr int kNormThreads = 256;
constexpr int kNormBackBlocks = 1024;   // blocks of the backward kernel, at most

cudaError_t launch_norm_rope(const NormRopeParams& p, int D, int sm_count, cudaStream_t stream);
cudaError_t launch_norm_rope_back(const NormRopeBackParams& p, int D, int sm_count, cudaStream_t stream);

}  // namespace dsa
