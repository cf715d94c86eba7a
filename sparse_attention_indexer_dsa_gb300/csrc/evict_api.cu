// C ABI of the operators that bound a paged cache (include/dsa_idx.h):
// host-side validation and launches.  Never allocates, frees or synchronises.
#include <cuda_runtime.h>

#include <cmath>

#include "dsa_idx.h"
#include "dsa_status_codes.h"
#include "evict_params.h"
#include "host_util.h"

using namespace dsa;

extern "C" {

size_t dsa_idx_weigh_workspace_size(int total_q, int num_seqs, int max_seqlen_q, int n_heads, int n_kv_heads,
                                    int head_dim) {
  if (total_q < 0 || num_seqs < 1 || max_seqlen_q < 0 || n_kv_heads < 1 || n_heads < 1 || n_heads % n_kv_heads != 0 ||
      n_heads / n_kv_heads > 128 || (head_dim != 64 && head_dim != 128))
    return 0;
  // the sums of divided units where a sequence may have more query rows than the step kernel takes
  const bool tiles = (int64_t)max_seqlen_q * (n_heads / n_kv_heads) > kWeighStepRows16;
  return DSA_DEV_STATUS_HEADER_BYTES + (tiles ? (size_t)kAttnSms * 2 * kWeighKeys * sizeof(float) : 0);
}

dsa_status_t dsa_idx_cache_weigh(const void* q, int64_t q_stride, const float* lse, const void* k_pages,
                                 const uint8_t* k_page_scale, float* weights, int num_pages, int page_size, int n_heads,
                                 int n_kv_heads, int head_dim, dsa_precision_t prec, const int32_t* page_table,
                                 int max_pages, const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int num_seqs,
                                 int total_q, int max_seqlen_q, int max_seqlen_k, float sm_scale, void* ws,
                                 size_t ws_bytes, dsa_stream_t stream) {
  WeighParams p{};
  dsa_status_t s = check_cache(&p.c, k_pages, k_page_scale, nullptr, nullptr, num_pages, page_size, n_kv_heads, head_dim,
                               prec, page_table, max_pages, num_seqs, cu_seqlens_k);
  if (s != DSA_OK) return s;
  if (!weights || !cu_seqlens_q || (total_q > 0 && (!q || !lse))) return fail(DSA_ERR_INVALID_ARG, "null pointer");
  if (total_q < 0 || max_seqlen_q < 0 || max_seqlen_k < 0) return fail(DSA_ERR_INVALID_ARG, "sizes");
  if (n_heads < 1 || n_heads % n_kv_heads != 0 || n_heads / n_kv_heads > 128)
    return fail(DSA_ERR_UNSUPPORTED, "n_heads must be a multiple of n_kv_heads, at most 128 heads to one");
  if ((int64_t)total_q * n_heads >= (int64_t)1 << 30) return fail(DSA_ERR_UNSUPPORTED, "total_q * n_heads above 2^30");
  if (max_seqlen_k > (1 << 30)) return fail(DSA_ERR_UNSUPPORTED, "max_seqlen_k is at most 2^30");
  // The attention's own scale, so that weights and lse fit together.  The tensor cores' FP32 sums truncate: a logit of
  // 128 products of BF16 values comes out short by 0.9 - 1.5e-7 of itself on average, one of 64 by 0.4 - 0.8e-7
  // (mma.sync and tcgen05 alike; rows normal, with outliers, uniform, of one sign).  The attention's lse is short alike:
  // with it the weights of a chunk's tokens add up to their heads within 2.5e-7 on average at mean logits up to 30;
  // with the lse of exact logits they are short by the logit's part (2.7e-6 at 25).
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  if (!(sm_scale >= 0.f) || std::isinf(p.scale_log2))
    return fail(DSA_ERR_INVALID_ARG, "sm_scale and sm_scale * log2(e) must be finite and >= 0");
  if (!aligned16(q) || !aligned16(weights)) return fail(DSA_ERR_INVALID_ARG, "q and weights must be 16-byte aligned");
  if ((s = check_stride(&q_stride, n_heads, head_dim, 2, "q")) != DSA_OK) return s;
  if ((s = check_ws(ws, ws_bytes, dsa_idx_weigh_workspace_size(total_q, num_seqs, max_seqlen_q, n_heads, n_kv_heads, head_dim))) !=
      DSA_OK)
    return s;
  DevInfo di;
  if ((s = device_info(&di)) != DSA_OK) return s;
  p.weights = weights;
  p.q = q;
  p.q_stride = q_stride;
  p.lse = lse;
  p.cu_q = cu_seqlens_q;
  p.cu_k = cu_seqlens_k;
  p.num_seqs = num_seqs;
  p.total_q = total_q;
  p.max_seqlen_q = max_seqlen_q;
  p.max_seqlen_k = max_seqlen_k;
  p.n_heads = n_heads;
  p.group = n_heads / n_kv_heads;
  p.group_mul = p.group > 1 ? (uint32_t)(((uint64_t)1 << 32) / p.group + 1) : 0;
  p.hdr = reinterpret_cast<int*>(ws);
  p.part = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(ws) + DSA_DEV_STATUS_HEADER_BYTES);
  p.timeout_ns = wait_timeout_ns();
  p.fault_inject = fault_inject_mode();
  // Long chunks have a kernel of their own; each of the two takes the sequences that are its own, by
  // their lengths on the device.
  p.step_rows = prec == DSA_PREC_BF16 ? kWeighStepRows16 : kWeighStepRows8;
  const bool tiles = total_q > 0 && (int64_t)max_seqlen_q * p.group > p.step_rows;
  p.step_blocks = weigh_step_blocks(p, di.sm_count);
  p.tile_blocks = tiles ? (di.sm_count < kAttnSms ? di.sm_count : kAttnSms) : 0;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (tiles && (s = make_queries_map(&p.tm_q, q, total_q, q_stride, n_heads, head_dim, p.group, kWeighCols / p.group)) != DSA_OK)
    return s;
  cudaError_t e = launch_weigh_steps(p, head_dim, p.step_blocks, st);
  if (e == cudaSuccess && tiles) e = launch_weigh_tiles(p, head_dim, st);
  if (e != cudaSuccess) return cuda_fail(e, "cache weigh launch");
  return DSA_OK;
}

dsa_status_t dsa_idx_evict_select(const float* weights, int num_pages, int page_size, int n_kv_heads,
                                  const int32_t* page_table, int max_pages, const int32_t* cu_seqlens_k, int num_seqs,
                                  int max_seqlen_k, int budget, int sinks, int recent, int shared, int32_t* kept,
                                  int32_t* kept_len, void* ws, size_t ws_bytes, dsa_stream_t stream) {
  SelectParams p{};
  PagedCacheView c{};   // (the geometry's checks; the pages themselves are not read)
  dsa_status_t s = check_cache(&c, weights, nullptr, nullptr, nullptr, num_pages, page_size, n_kv_heads, 64, DSA_PREC_BF16,
                               page_table, max_pages, num_seqs, cu_seqlens_k);
  if (s != DSA_OK) return s;
  if (!kept || !kept_len) return fail(DSA_ERR_INVALID_ARG, "null pointer");
  if ((int64_t)num_seqs * n_kv_heads >= (int64_t)1 << 30) return fail(DSA_ERR_UNSUPPORTED, "num_seqs * n_kv_heads above 2^30");
  if (max_seqlen_k < 0 || max_seqlen_k > (1 << 30)) return fail(DSA_ERR_INVALID_ARG, "max_seqlen_k must be in [0, 2^30]");
  if (budget < 1 || budget > (1 << 30)) return fail(DSA_ERR_INVALID_ARG, "budget must be in [1, 2^30]");
  if (sinks < 0 || recent < 0 || (int64_t)sinks + recent > budget)
    return fail(DSA_ERR_INVALID_ARG, "sinks and recent must be >= 0 and fit into the budget");
  if ((s = check_ws(ws, ws_bytes, DSA_DEV_STATUS_HEADER_BYTES)) != DSA_OK) return s;
  DevInfo di;
  if ((s = device_info(&di)) != DSA_OK) return s;
  p.weights = weights;
  p.table = page_table;
  p.num_pages = num_pages;
  p.page_shift = c.page_shift;
  p.n_kv = n_kv_heads;
  p.max_pages = max_pages;
  p.cu_k = cu_seqlens_k;
  p.num_seqs = num_seqs;
  p.max_seqlen_k = max_seqlen_k;
  p.budget = budget;
  p.sinks = sinks;
  p.recent = recent;
  p.shared = shared ? 1 : 0;
  p.kept = kept;
  p.kept_len = kept_len;
  p.hdr = reinterpret_cast<int*>(ws);
  cudaError_t e = launch_evict_select(p, di.sm_count, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "evict select launch");
  return DSA_OK;
}

dsa_status_t dsa_idx_cache_compact(void* k_pages, uint8_t* k_page_scale, void* v_pages, uint8_t* v_page_scale,
                                   float* weights, int num_pages, int page_size, int n_kv_heads, int head_dim,
                                   dsa_precision_t prec, const int32_t* page_table, int max_pages, const int32_t* kept,
                                   const int32_t* kept_len, int num_seqs, int kept_heads, int kept_width, void* ws,
                                   size_t ws_bytes, dsa_stream_t stream) {
  CompactParams p{};
  dsa_status_t s = check_cache(&p.c, k_pages, k_page_scale, v_pages, v_page_scale, num_pages, page_size, n_kv_heads,
                               head_dim, prec, page_table, max_pages, num_seqs, kept_len);
  if (s != DSA_OK) return s;
  if (!kept) return fail(DSA_ERR_INVALID_ARG, "null pointer");
  if ((int64_t)num_seqs * n_kv_heads >= (int64_t)1 << 30) return fail(DSA_ERR_UNSUPPORTED, "num_seqs * n_kv_heads above 2^30");
  if (kept_heads != 1 && kept_heads != n_kv_heads) return fail(DSA_ERR_INVALID_ARG, "kept has one head, or the cache's");
  if (kept_width < 1 || kept_width > (1 << 30)) return fail(DSA_ERR_INVALID_ARG, "kept_width must be in [1, 2^30]");
  if (!aligned16(weights)) return fail(DSA_ERR_INVALID_ARG, "weights must be 16-byte aligned");
  if ((s = check_ws(ws, ws_bytes, DSA_DEV_STATUS_HEADER_BYTES)) != DSA_OK) return s;
  DevInfo di;
  if ((s = device_info(&di)) != DSA_OK) return s;
  p.weights = weights;
  p.kept = kept;
  p.kept_len = kept_len;
  p.num_seqs = num_seqs;
  p.heads = kept_heads;
  p.width = kept_width;
  p.row_bytes = head_dim * (prec == DSA_PREC_BF16 ? 2 : 1);
  p.hdr = reinterpret_cast<int*>(ws);
  cudaError_t e = launch_cache_compact(p, di.sm_count, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "cache compact launch");
  return DSA_OK;
}

}  // extern "C"
