// Parameter blocks and launchers of the operators that bound a paged cache:
// the attention weight of its rows (weigh.cuh), the choice of the rows that
// stay and their moving together (evict.cu).
#pragma once

#include "paged_params.h"

namespace dsa {

struct WeighParams {
  CUtensorMap tm_q;   // queries as [tokens][heads][D]: a box per tile (weigh_tiles.cu)
  PagedCacheView c;
  float* weights;     // [num_pages][n_kv][page_size]
  const void* q;
  int64_t q_stride;   // elements from one token to the next
  const float* lse;   // [total_q][n_heads]
  const int32_t* cu_q;
  const int32_t* cu_k;
  int num_seqs, total_q, max_seqlen_q, max_seqlen_k, n_heads, group;
  uint32_t group_mul; // 2^32 / group, rounded up (group 1: not used)
  float scale_log2;   // sm_scale * log2(e)
  int step_rows;      // query rows of a sequence up to which its keys stream past them
  int step_blocks, tile_blocks;
  int* hdr;
  float* part;        // [tile_blocks][2][kWeighKeys] sums of divided units: that a block ends, that it begins
  int fault_inject;
  unsigned long long timeout_ns;
};

// Query rows of a sequence up to which its keys stream past them, 8-bit ones and BF16 ones (the tile kernel has to
// widen 8-bit keys to BF16 first, and its query tiles are empty but for these rows).  Streaming / tiles, us, 32 sequences of
// 2048 - 8192 keys, 8 key heads:
//   128 elements   16 rows       32 rows       64 rows       128 rows
//     BF16         75 / 97      127 / 93      218 / 96      403 / 115
//     MXFP8        78 / 163     104 / 160     158 / 158     266 / 180
//     FP8          78 / 164     105 / 163     160 / 163     267 / 176
//   64 elements
//     BF16         44 / 84       65 / 82      113 / 89      207 / 111
//     MXFP8        52 / 102      72 / 97      114 / 106     200 / 127
//     FP8          53 / 102      73 / 97      115 / 106     202 / 127
// One bound for both sizes of a head: of 64 elements 32 rows of BF16 take 82 in place of 65, 64 8-bit ones 114 in
// place of 106.
constexpr int kWeighStepRows8 = 64, kWeighStepRows16 = 16;
constexpr int kWeighCols = 256;    // query rows of a tile
constexpr int kWeighKeys = 256;    // keys of a unit
struct SelectParams {
  const float* weights;
  const int32_t* table;
  int num_pages, page_shift, n_kv, max_pages;
  const int32_t* cu_k;
  int num_seqs, max_seqlen_k;
  int budget, sinks, recent, shared;
  int32_t* kept;       // [num_seqs][shared ? 1 : n_kv][budget]
  int32_t* kept_len;   // [num_seqs]
  int cached;          // rows of a block whose bits its shared memory holds
  int* hdr;
};

struct CompactParams {
  PagedCacheView c;
  float* weights;          // null: none
  const int32_t* kept;     // [num_seqs][heads][width], ascending
  const int32_t* kept_len; // [num_seqs]
  int num_seqs, heads, width;
  int row_bytes;           // of a row of keys or values
  int* hdr;
};

int weigh_step_blocks(const WeighParams& p, int sm_count);
cudaError_t launch_weigh_steps(const WeighParams& p, int D, int blocks, cudaStream_t stream);
cudaError_t launch_weigh_tiles(const WeighParams& p, int D, cudaStream_t stream);
cudaError_t launch_evict_select(const SelectParams& p, int sm_count, cudaStream_t stream);
cudaError_t launch_cache_compact(const CompactParams& p, int sm_count, cudaStream_t stream);

}  // namespace dsa
