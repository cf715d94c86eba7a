// Parameter blocks and launchers of the paged-cache operators (paged_cache.cu,
// paged_attn.cuh) and the device view of a paged cache.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "dsa_status_codes.h"

namespace dsa {

// Pages [num_pages][n_kv][page_size][D]; the rows of one (page, head) are
// contiguous.  Scales follow the same order, `sw` bytes per row.
struct PagedCacheView {
  void* k;
  uint8_t* k_scale;
  void* v;            // null: a cache of keys alone
  uint8_t* v_scale;
  const int32_t* table;   // [num_seqs][max_pages]
  int num_pages, page_shift, n_kv, max_pages;
  int fmt;            // dsa_precision_t
  int sw;             // scale bytes per row (0 for BF16)
};

struct CacheWriteParams {
  PagedCacheView c;
  const void* k;
  const void* v;
  const uint8_t* k_scale;   // source in operand form: its scale bytes
  const uint8_t* v_scale;
  int64_t k_stride, v_stride;   // elements from one token to the next
  const int32_t* cu_q;
  const int32_t* cu_k;
  int num_seqs, total_q;
  int src;            // 0 FP32, 1 BF16, 2 operand form (codes and scales)
  int rule;
  int* hdr;
};

struct CacheReadParams {
  PagedCacheView c;
  const int32_t* cu_k;
  int num_seqs, total_k;
  int dequant;        // 0: rows and scales as stored, 1: BF16 values
  void* k;
  uint8_t* k_scale;
  void* v;
  uint8_t* v_scale;
  int* hdr;
};

constexpr int kAttnKeys = 128;      // keys per tile
constexpr int kAttnRows = 128;      // query rows (token, head of the group) per tile
// Key tiles of a divided range, at least.  1 / 2 / 4: 16 tokens over 2048 keys of one head 24.1 / 20.8 / 21.2 us,
// 2048 listed rows of one token 24.9 / 23.3 / 25.4, of 32 tokens over MXFP8 32.7 / 32.7 / 35.8.
constexpr int kAttnMinChunk = 2;
constexpr int kAttnNarrow = 16;              // query rows of a narrow tile (columns of its products)
constexpr int kAttnNarrowP = kAttnNarrow * kAttnKeys * 2;   // bytes of its weights
constexpr int kAttnBars = 2 * 32 + 2 * 10;   // barriers of a block
constexpr uint32_t kAttnSmemMax = 232448;   // 227 KB
constexpr int kAttnSms = 152;       // the grid's upper bound, for workspace sizes

// How one call is laid out (attn_plan): tiles, shared memory and splits.
struct AttnPlan {
  int pair;        // two query tiles share one key stream (long chunks); else two independent streams
  int gather;      // rows resolved and copied one by one (listed keys, short page scales)
  int tq;          // tokens per query tile
  int rows_cap;    // rows of a tile that can be live
  int nst;         // key/value stages per ring
  int nraw;        // tiles of stored 8-bit rows per ring
  int narrow;      // at most kAttnNarrow rows to a tile: the products have the keys as rows, the queries as columns
  int max_units;   // units with room for a partial result; 0: key ranges are never divided
  uint32_t q_bytes;                                        // query tile in shared memory
  uint32_t off_p, off_ring, off_raw, off_rows, off_red, off_mask, off_bars, off_tab, smem;
};

struct AttnParams {
  CUtensorMap tm_k, tm_v;   // pages as [pages * heads][page_size][D]: a box per page and tile
  PagedCacheView c;
  AttnPlan plan;
  const void* q;
  int64_t q_stride;   // elements from one token to the next
  const int32_t* cu_q;
  const int32_t* cu_k;
  const int32_t* topk_idx;   // null: every visible key
  const int32_t* topk_len;
  int topk_width;
  int num_seqs, total_q, max_seqlen_q, max_seqlen_k, n_heads, group;
  float scale_log2;   // sm_scale * log2(e)
  void* out;
  float* lse;
  int* hdr;
  int* doc_base;      // [num_seqs] first unit of each sequence
  float* part_o;      // [units (x 2)][rows_cap][D] sums not yet divided
  float2* part_ml;    // [units (x 2)][rows_cap] running maximum (log2) and sum
  int fault_inject;
  unsigned long long timeout_ns;
};

// Header words of an attention workspace beside the status words.
constexpr int kAttnHdrChunk = 8;    // key tiles per split

void attn_plan(AttnPlan* pl, int num_seqs, int total_q, int max_seqlen_q, int max_seqlen_k, int n_heads, int n_kv, int D,
               int sw, int page_size, int topk_width);
size_t attn_workspace_bytes(const AttnPlan& pl, int num_seqs, int D);

cudaError_t launch_cache_write(const CacheWriteParams& p, int D, int sm_count, cudaStream_t stream);
cudaError_t launch_cache_read(const CacheReadParams& p, int D, int sm_count, cudaStream_t stream);
// One launcher per head size and width of the cached elements (a file each).
cudaError_t launch_paged_attention_128(const AttnParams& p, int grid, int sm_count, cudaStream_t stream);
cudaError_t launch_paged_attention_64(const AttnParams& p, int grid, int sm_count, cudaStream_t stream);
cudaError_t launch_paged_attention_128_q8(const AttnParams& p, int grid, int sm_count, cudaStream_t stream);
cudaError_t launch_paged_attention_64_q8(const AttnParams& p, int grid, int sm_count, cudaStream_t stream);

#ifdef __CUDACC__
// Sequence of packed row `r`: the last d with cu[d] <= r (cu[0] = 0).
__device__ __forceinline__ int find_seq(const int32_t* __restrict__ cu, int num_seqs, int r) {
  int lo = 0, hi = num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(cu + mid) <= r) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Row of the cache (in rows of D elements) that holds position `pos` of
// sequence `d`, head `h`; -1 where the table or the page list does not cover it.
__device__ __forceinline__ int64_t cache_row(const PagedCacheView& c, int d, int pos, int h) {
  const int pi = pos >> c.page_shift;
  if (pos < 0 || pi >= c.max_pages) return -1;
  const int page = __ldg(c.table + (int64_t)d * c.max_pages + pi);
  if ((unsigned)page >= (unsigned)c.num_pages) return -1;
  return (((int64_t)page * c.n_kv + h) << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
}

// Every block of a launch records its status (0 or an error code).
__device__ __forceinline__ void put_block_status(int* hdr, int code) {
  hdr[DSA_DEV_STATUS_FIRST + blockIdx.x] = code;
  if (blockIdx.x == 0) {
    hdr[0] = DSA_DEV_STATUS_PER_BLOCK;
    hdr[1] = gridDim.x;
  }
}
#endif

}  // namespace dsa
