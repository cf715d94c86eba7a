// C ABI of the paged-cache operators (include/dsa_idx.h): host-side validation
// and launches.  Never allocates, frees or synchronises.
#include <cuda_runtime.h>

#include <cmath>
#include <limits>

#include "dsa_idx.h"
#include "dsa_status_codes.h"
#include "host_util.h"
#include "paged_params.h"

using namespace dsa;

namespace {

// Scale bytes of a row.
int scale_width(dsa_precision_t prec, int head_dim) {
  return prec == DSA_PREC_MXFP8 ? head_dim / 32 : (prec == DSA_PREC_FP8 ? 1 : 0);
}

}  // namespace

namespace dsa {

dsa_status_t check_cache(PagedCacheView* c, const void* k_pages, const uint8_t* k_page_scale, const void* v_pages,
                         const uint8_t* v_page_scale, int num_pages, int page_size, int n_kv_heads, int head_dim,
                         dsa_precision_t prec, const int32_t* page_table, int max_pages, int num_seqs,
                         const int32_t* cu_seqlens_k) {
  if (!k_pages || !page_table || !cu_seqlens_k) return fail(DSA_ERR_INVALID_ARG, "null pointer");
  if (prec != DSA_PREC_BF16 && prec != DSA_PREC_MXFP8 && prec != DSA_PREC_FP8) return fail(DSA_ERR_INVALID_ARG, "prec");
  if (head_dim != 64 && head_dim != 128) return fail(DSA_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (num_pages < 1 || n_kv_heads < 1 || max_pages < 1 || num_seqs < 1) return fail(DSA_ERR_INVALID_ARG, "sizes");
  if (page_size < 8 || page_size > 1024 || (page_size & (page_size - 1)) != 0)
    return fail(DSA_ERR_UNSUPPORTED, "page_size must be a power of two in [8, 1024]");
  if ((int64_t)num_pages * n_kv_heads >= ((int64_t)1 << 31) / page_size)
    return fail(DSA_ERR_UNSUPPORTED, "a cache holds fewer than 2^31 rows");
  if (!aligned16(k_pages) || !aligned16(v_pages)) return fail(DSA_ERR_INVALID_ARG, "pages must be 16-byte aligned");
  if (prec != DSA_PREC_BF16) {
    if (!k_page_scale || (v_pages && !v_page_scale)) return fail(DSA_ERR_INVALID_ARG, "8-bit caches need their scales");
    if (!aligned16(k_page_scale) || !aligned16(v_page_scale))
      return fail(DSA_ERR_INVALID_ARG, "page scales must be 16-byte aligned");
  }
  c->k = const_cast<void*>(k_pages);
  c->k_scale = const_cast<uint8_t*>(k_page_scale);
  c->v = const_cast<void*>(v_pages);
  c->v_scale = const_cast<uint8_t*>(v_page_scale);
  c->table = page_table;
  c->num_pages = num_pages;
  c->page_shift = 0;
  while ((1 << c->page_shift) < page_size) ++c->page_shift;
  c->n_kv = n_kv_heads;
  c->max_pages = max_pages;
  c->fmt = (int)prec;
  c->sw = scale_width(prec, head_dim);
  return DSA_OK;
}

dsa_status_t check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (!ws) return fail(DSA_ERR_WORKSPACE, "workspace is NULL");
  if (ws_bytes < need) return fail(DSA_ERR_WORKSPACE, "workspace %zu bytes, need %zu", ws_bytes, need);
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return fail(DSA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  return DSA_OK;
}

dsa_status_t check_stride(int64_t* stride, int heads, int head_dim, int elem_bytes, const char* name) {
  const int64_t packed = (int64_t)heads * head_dim;
  if (*stride == 0) *stride = packed;
  if (*stride < packed || (*stride * elem_bytes) % 16 != 0)
    return fail(DSA_ERR_INVALID_ARG, "%s: a token stride covers its heads and is a multiple of 16 bytes", name);
  return DSA_OK;
}

}  // namespace dsa

namespace {

constexpr uint32_t round16(uint32_t x) { return (x + 15) / 16 * 16; }
size_t round256(size_t x) { return (x + 255) / 256 * 256; }

// Streams of a launch, and units of one query tile (or pair) up to which key ranges are divided: four to a
// stream, two pairs to a block.  Half as many / as many / twice as many: a token of each of 64 sequences over MXFP8 439 / 416 / 417 us, 200
// short sequences 136 / 136 / 144, ragged chunks over FP8 490 / 490 / 508; but 2048 tokens over 4096 BF16
// keys 141 / 150 / 150.
int64_t all_streams(bool pair) { return pair ? kAttnSms : 2 * kAttnSms; }
int64_t most_undivided(bool pair) { return (pair ? 2 : 4) * all_streams(pair); }

// Workspace bytes with `slots` rows of partial results.
size_t with_partials(int num_seqs, size_t slots, int D) {
  return DSA_DEV_STATUS_HEADER_BYTES + round256((size_t)num_seqs * 4) + round256(slots * 8) + round256(slots * D * 4);
}

}  // namespace

namespace dsa {

// Two query tiles to a block when the average sequence fills more than one
// 128-row tile: its keys are then read once for both.  Otherwise the two
// streams of a block work on their own; tiles of at most 16 rows with
// gathered keys are narrow (the figures are with the kernel).  Key ranges are divided only while
// there are at most four units to a stream, or two pairs to a block (more
// balance themselves), and a call's workspace has room for as many more.
// The plan is the call's, not a sequence's: a long chunk makes the tiles of
// single tokens beside it pairs, one of the two empty, and their ranges whole.
// 2048 tokens of one sequence and one of each of 63 others (64 heads, 8 key
// heads, 2048 - 16384 keys): 791 us over BF16 and 1123 over MXFP8, in two calls
// 348 + 389 and 455 + 419.
void attn_plan(AttnPlan* pl, int num_seqs, int total_q, int max_seqlen_q, int max_seqlen_k, int n_heads, int n_kv, int D,
               int sw, int page_size, int topk_width) {
  *pl = AttnPlan{};
  const bool eight_bit = sw > 0;
  const int group = n_heads / n_kv;
  // a page's part of a tile must have scales in whole 16 bytes for the bulk copy
  pl->gather = topk_width > 0 || (eight_bit && ((page_size < kAttnKeys ? page_size : kAttnKeys) * sw) % 16 != 0);
  pl->tq = topk_width > 0 ? 1 : kAttnRows / group;
  pl->pair = !pl->gather && max_seqlen_q > pl->tq && (int64_t)total_q * group > (int64_t)kAttnRows * num_seqs;
  const int tok = pl->tq < max_seqlen_q ? pl->tq : (max_seqlen_q > 0 ? max_seqlen_q : 1);
  pl->rows_cap = tok * group;
  const int per = pl->pair ? 2 * pl->tq : pl->tq;
  // every tile but a sequence's last is full, and a tile holds a token at least
  int64_t tiles = (int64_t)total_q / per + num_seqs;
  if (tiles > total_q) tiles = total_q;
  const int64_t base = tiles * n_kv;
  const int64_t most = most_undivided(pl->pair);
  // (a range of kAttnMinChunk tiles is not divided: no partial results, no joining launch)
  const bool divide = base <= most && (topk_width > 0 ? topk_width : max_seqlen_k) > kAttnMinChunk * kAttnKeys;
  pl->max_units = divide ? (int)(base + most) : 0;
  pl->narrow = pl->gather && D == 128 && pl->rows_cap <= kAttnNarrow;
  const int qrows = pl->narrow ? kAttnNarrow : pl->pair || pl->rows_cap > 64 ? 128 : (pl->rows_cap > 32 ? 64 : 32);
  pl->q_bytes = (uint32_t)qrows * D * 2;
  constexpr uint32_t kRows = 64;   // (visible rows of a stored tile)
  constexpr uint32_t kMask = 2 * 8 * 4 * 4, kBars = 8 * kAttnBars + 32, kTab = round16((64 + 1) * 4);
  // The largest plans fit: 128 rows of 128 elements to a query tile, with a stored tile (a pair: one for
  // each team of workers) and two stages to a ring (a pair of an 8-bit cache: three).
  constexpr uint32_t kStageMax = kAttnKeys * 128 * 2, kRawMax = kAttnKeys * 128 + 512;
  constexpr uint32_t kFixedMax = 2 * kAttnRows * 128 * 2 + kRows + kMask + kBars + kTab;
  static_assert(kFixedMax + 2 * (2 * kStageMax + kRawMax) <= kAttnSmemMax, "two streams");
  static_assert(kFixedMax + 3 * kStageMax + 2 * kRawMax <= kAttnSmemMax, "a pair");
  const uint32_t stage = kAttnKeys * D * 2, raw = kAttnKeys * D + 512, rings = pl->pair ? 1 : 2;
  const uint32_t mask = pl->gather ? kMask : 0, red = pl->narrow ? 2 * 9 * kAttnNarrow * 4 : 0;
  const uint32_t q = 2 * pl->q_bytes + (pl->narrow ? 4 * kAttnNarrowP : 0);
  const uint32_t avail = kAttnSmemMax - q - (kRows + red + mask + kBars + kTab);
  if (eight_bit) {
    pl->nst = pl->pair ? 3 : 2;
    pl->nraw = (int)((avail - rings * pl->nst * stage) / (rings * raw));
    if (pl->nraw > 6) pl->nraw = 6;
  } else {
    pl->nst = (int)(avail / (rings * stage));
    if (pl->nst > 8) pl->nst = 8;
    pl->nraw = 0;
  }
  pl->off_p = 2 * pl->q_bytes;
  pl->off_ring = q;
  pl->off_raw = pl->off_ring + rings * pl->nst * stage;
  pl->off_rows = pl->off_raw + rings * pl->nraw * raw;
  pl->off_red = pl->off_rows + kRows;
  pl->off_mask = pl->off_red + red;
  pl->off_bars = pl->off_mask + mask;
  pl->off_tab = pl->off_bars + kBars;
  pl->smem = pl->off_tab + kTab;
}

size_t attn_workspace_bytes(const AttnPlan& pl, int num_seqs, int D) {
  if (pl.max_units == 0) return DSA_DEV_STATUS_HEADER_BYTES;
  return with_partials(num_seqs, (size_t)pl.max_units * (pl.pair ? 2 : 1) * pl.rows_cap, D);
}

}  // namespace dsa

namespace {

bool sizes_ok(int total_q, int num_seqs, int max_seqlen_q, int n_heads, int n_kv, int D, int topk_width) {
  return total_q >= 0 && num_seqs >= 1 && max_seqlen_q >= 0 && n_heads >= 1 && n_kv >= 1 && n_heads % n_kv == 0 &&
         n_heads / n_kv <= kAttnRows && (D == 64 || D == 128) && topk_width >= 0;
}

}  // namespace

extern "C" {

size_t dsa_idx_cache_workspace_size(void) { return DSA_DEV_STATUS_HEADER_BYTES; }

dsa_status_t dsa_idx_cache_write(const void* k, int64_t k_stride, const uint8_t* k_scale, const void* v, int64_t v_stride,
                                 const uint8_t* v_scale, dsa_dtype_t in_dtype, dsa_mx_scale_rule_t scale_rule,
                                 const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int num_seqs, int total_q,
                                 const int32_t* page_table, int max_pages, void* k_pages, uint8_t* k_page_scale,
                                 void* v_pages, uint8_t* v_page_scale, int num_pages, int page_size, int n_kv_heads,
                                 int head_dim, dsa_precision_t prec, void* ws, size_t ws_bytes, dsa_stream_t stream) {
  CacheWriteParams p{};
  dsa_status_t s = check_cache(&p.c, k_pages, k_page_scale, v_pages, v_page_scale, num_pages, page_size, n_kv_heads,
                               head_dim, prec, page_table, max_pages, num_seqs, cu_seqlens_k);
  if (s != DSA_OK) return s;
  if ((!k && total_q > 0) || !cu_seqlens_q) return fail(DSA_ERR_INVALID_ARG, "null pointer");
  if (total_q > 0 && (v != nullptr) != (v_pages != nullptr))
    return fail(DSA_ERR_INVALID_ARG, "v and v_pages must both be given or both be NULL");
  if (total_q < 0) return fail(DSA_ERR_INVALID_ARG, "sizes");
  if ((int64_t)total_q * n_kv_heads >= (int64_t)1 << 30) return fail(DSA_ERR_UNSUPPORTED, "total_q * n_kv_heads above 2^30");
  if (scale_rule != DSA_MX_SCALE_NOSAT && scale_rule != DSA_MX_SCALE_FLOOR) return fail(DSA_ERR_INVALID_ARG, "scale_rule");
  int elem;
  if (in_dtype == DSA_DTYPE_OPERAND && prec != DSA_PREC_BF16) {
    if (total_q > 0 && (!k_scale || (v && !v_scale))) return fail(DSA_ERR_INVALID_ARG, "codes come with their scales");
    p.src = 2;
    elem = 1;
  } else if (in_dtype == DSA_DTYPE_F32) {
    p.src = 0;
    elem = 4;
  } else if (in_dtype == DSA_DTYPE_BF16 || in_dtype == DSA_DTYPE_OPERAND) {   // a BF16 cache stores the operand itself
    p.src = 1;
    elem = 2;
  } else {
    return fail(DSA_ERR_INVALID_ARG, "in_dtype");
  }
  if (!aligned16(k) || !aligned16(v)) return fail(DSA_ERR_INVALID_ARG, "k and v must be 16-byte aligned");
  if ((s = check_stride(&k_stride, n_kv_heads, head_dim, elem, "k")) != DSA_OK) return s;
  if (v && (s = check_stride(&v_stride, n_kv_heads, head_dim, elem, "v")) != DSA_OK) return s;
  if ((s = check_ws(ws, ws_bytes, DSA_DEV_STATUS_HEADER_BYTES)) != DSA_OK) return s;
  DevInfo di;
  if ((s = device_info(&di)) != DSA_OK) return s;
  p.k = k;
  p.v = v;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.cu_q = cu_seqlens_q;
  p.cu_k = cu_seqlens_k;
  p.num_seqs = num_seqs;
  p.total_q = total_q;
  p.rule = (int)scale_rule;
  p.hdr = reinterpret_cast<int*>(ws);
  cudaError_t e = launch_cache_write(p, head_dim, di.sm_count, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "cache write launch");
  return DSA_OK;
}

dsa_status_t dsa_idx_cache_read(const void* k_pages, const uint8_t* k_page_scale, const void* v_pages,
                                const uint8_t* v_page_scale, int num_pages, int page_size, int n_kv_heads, int head_dim,
                                dsa_precision_t prec, const int32_t* page_table, int max_pages,
                                const int32_t* cu_seqlens_k, int num_seqs, int total_k, int dequantize, void* k_out,
                                uint8_t* k_scale_out, void* v_out, uint8_t* v_scale_out, void* ws, size_t ws_bytes,
                                dsa_stream_t stream) {
  CacheReadParams p{};
  dsa_status_t s = check_cache(&p.c, k_pages, k_page_scale, v_pages, v_page_scale, num_pages, page_size, n_kv_heads,
                               head_dim, prec, page_table, max_pages, num_seqs, cu_seqlens_k);
  if (s != DSA_OK) return s;
  if (!k_out && total_k > 0) return fail(DSA_ERR_INVALID_ARG, "null pointer");
  if (v_out && !v_pages) return fail(DSA_ERR_INVALID_ARG, "the cache has no values");
  if (total_k < 0) return fail(DSA_ERR_INVALID_ARG, "sizes");
  if ((int64_t)total_k * n_kv_heads >= (int64_t)1 << 30) return fail(DSA_ERR_UNSUPPORTED, "total_k * n_kv_heads above 2^30");
  if (total_k > 0 && prec != DSA_PREC_BF16 && !dequantize && (!k_scale_out || (v_out && !v_scale_out)))
    return fail(DSA_ERR_INVALID_ARG, "codes come with their scales");
  if (!aligned16(k_out) || !aligned16(v_out)) return fail(DSA_ERR_INVALID_ARG, "outputs must be 16-byte aligned");
  if ((s = check_ws(ws, ws_bytes, DSA_DEV_STATUS_HEADER_BYTES)) != DSA_OK) return s;
  DevInfo di;
  if ((s = device_info(&di)) != DSA_OK) return s;
  p.cu_k = cu_seqlens_k;
  p.num_seqs = num_seqs;
  p.total_k = total_k;
  p.dequant = dequantize && prec != DSA_PREC_BF16;
  p.k = k_out;
  p.k_scale = k_scale_out;
  p.v = v_out;
  p.v_scale = v_scale_out;
  p.hdr = reinterpret_cast<int*>(ws);
  cudaError_t e = launch_cache_read(p, head_dim, di.sm_count, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "cache read launch");
  return DSA_OK;
}

size_t dsa_idx_attention_workspace_size(int total_q, int num_seqs, int max_seqlen_q, int n_heads, int n_kv_heads,
                                        int head_dim, int topk_width) {
  if (!sizes_ok(total_q, num_seqs, max_seqlen_q, n_heads, n_kv_heads, head_dim, topk_width)) return 0;
  // The most that attn_plan asks for at any format and at any sizes up to these: fewer tokens may need
  // more, as the key ranges of many tiles are not divided.
  const int group = n_heads / n_kv_heads, tq = topk_width > 0 ? 1 : kAttnRows / group;
  const int tok = max_seqlen_q < 1 ? 1 : (max_seqlen_q < tq ? max_seqlen_q : tq);
  size_t slots = 0;
  for (bool pair : {false, true}) {
    if (pair && (topk_width > 0 || max_seqlen_q <= tq)) continue;
    int64_t tiles = (int64_t)total_q / (pair ? 2 * tq : tq) + num_seqs;
    if (tiles > total_q) tiles = total_q;
    int64_t base = tiles * n_kv_heads;
    if (base > most_undivided(pair)) base = most_undivided(pair);
    const size_t n = (size_t)(base + most_undivided(pair)) * (pair ? 2 : 1) * (size_t)(tok * group);
    slots = n > slots ? n : slots;
  }
  return with_partials(num_seqs, slots, head_dim);
}

size_t dsa_idx_attention_call_workspace_size(int total_q, int num_seqs, int max_seqlen_q, int max_seqlen_k, int n_heads,
                                             int n_kv_heads, int head_dim, int page_size, dsa_precision_t prec,
                                             int topk_width) {
  if (!sizes_ok(total_q, num_seqs, max_seqlen_q, n_heads, n_kv_heads, head_dim, topk_width) || max_seqlen_k < 0 ||
      page_size < 1)
    return 0;
  AttnPlan pl;
  attn_plan(&pl, num_seqs, total_q, max_seqlen_q, max_seqlen_k, n_heads, n_kv_heads, head_dim, scale_width(prec, head_dim),
            page_size, topk_width);
  return attn_workspace_bytes(pl, num_seqs, head_dim);
}

dsa_status_t dsa_idx_paged_attention(const void* q, int64_t q_stride, const void* k_pages, const uint8_t* k_page_scale,
                                     const void* v_pages, const uint8_t* v_page_scale, int num_pages, int page_size,
                                     int n_heads, int n_kv_heads, int head_dim, dsa_precision_t prec,
                                     const int32_t* page_table, int max_pages, const int32_t* cu_seqlens_q,
                                     const int32_t* cu_seqlens_k, int num_seqs, int total_q, int max_seqlen_q,
                                     int max_seqlen_k, float sm_scale, const int32_t* topk_idx, const int32_t* topk_len,
                                     int topk_width, void* out, float* lse, void* ws, size_t ws_bytes,
                                     dsa_stream_t stream) {
  AttnParams p{};
  dsa_status_t s = check_cache(&p.c, k_pages, k_page_scale, v_pages, v_page_scale, num_pages, page_size, n_kv_heads,
                               head_dim, prec, page_table, max_pages, num_seqs, cu_seqlens_k);
  if (s != DSA_OK) return s;
  if (!v_pages || !cu_seqlens_q || (total_q > 0 && (!q || !out))) return fail(DSA_ERR_INVALID_ARG, "null pointer");
  if (total_q < 0 || max_seqlen_q < 0 || max_seqlen_k < 0) return fail(DSA_ERR_INVALID_ARG, "sizes");
  if (n_heads < 1 || n_heads % n_kv_heads != 0 || n_heads / n_kv_heads > 128)
    return fail(DSA_ERR_UNSUPPORTED, "n_heads must be a multiple of n_kv_heads, at most 128 heads to one");
  if ((int64_t)total_q * n_heads >= (int64_t)1 << 30) return fail(DSA_ERR_UNSUPPORTED, "total_q * n_heads above 2^30");
  // (key tiles are counted in 32 bits)
  if (max_seqlen_k > (1 << 30) || topk_width > (1 << 30))
    return fail(DSA_ERR_UNSUPPORTED, "max_seqlen_k and topk_width are at most 2^30");
  const float scale_log2 = sm_scale * 1.4426950408889634f;
  if (!(sm_scale >= 0.f) || std::isinf(scale_log2))
    return fail(DSA_ERR_INVALID_ARG, "sm_scale and sm_scale * log2(e) must be finite and >= 0");
  // (an empty list tensor has no address)
  if (topk_width < 0 || (topk_idx && topk_width < 1) || (!topk_idx && total_q > 0 && (topk_width > 0 || topk_len)))
    return fail(DSA_ERR_INVALID_ARG, "topk_width and topk_len belong to topk_idx");
  if (!aligned16(q) || !aligned16(out)) return fail(DSA_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  if ((s = check_stride(&q_stride, n_heads, head_dim, 2, "q")) != DSA_OK) return s;
  attn_plan(&p.plan, num_seqs, total_q, max_seqlen_q, max_seqlen_k, n_heads, n_kv_heads, head_dim, p.c.sw, page_size,
            topk_width);
  const size_t need = attn_workspace_bytes(p.plan, num_seqs, head_dim);
  if ((s = check_ws(ws, ws_bytes, need)) != DSA_OK) return s;
  DevInfo di;
  if ((s = device_info(&di)) != DSA_OK) return s;
  p.q = q;
  p.q_stride = q_stride;
  p.cu_q = cu_seqlens_q;
  p.cu_k = cu_seqlens_k;
  p.topk_idx = topk_idx;
  p.topk_len = topk_len;
  p.topk_width = topk_width;
  p.num_seqs = num_seqs;
  p.total_q = total_q;
  p.max_seqlen_q = max_seqlen_q;
  p.max_seqlen_k = max_seqlen_k;
  p.n_heads = n_heads;
  p.group = n_heads / n_kv_heads;
  // a masked logit is -inf times the scale: 0 is stood in for by the least number, times which the
  // largest logit is 2^-21
  p.scale_log2 = fmaxf(scale_log2, std::numeric_limits<float>::denorm_min());
  p.out = out;
  p.lse = lse;
  p.hdr = reinterpret_cast<int*>(ws);
  p.timeout_ns = wait_timeout_ns();
  p.fault_inject = fault_inject_mode();
  if (p.plan.max_units > 0) {
    const size_t slots = (size_t)p.plan.max_units * (p.plan.pair ? 2 : 1) * p.plan.rows_cap;
    uint8_t* w = reinterpret_cast<uint8_t*>(ws) + DSA_DEV_STATUS_HEADER_BYTES;
    p.doc_base = reinterpret_cast<int*>(w);
    w += round256((size_t)num_seqs * 4);
    p.part_ml = reinterpret_cast<float2*>(w);
    w += round256(slots * 8);
    p.part_o = reinterpret_cast<float*>(w);
  }
  if (!p.plan.gather) {
    const int64_t groups = (int64_t)num_pages * n_kv_heads;
    const int box = page_size < kAttnKeys ? page_size : kAttnKeys;
    const bool b8 = prec != DSA_PREC_BF16;
    if ((s = make_pages_map(&p.tm_k, k_pages, groups, page_size, head_dim, box, b8)) != DSA_OK) return s;
    if ((s = make_pages_map(&p.tm_v, v_pages, groups, page_size, head_dim, box, b8)) != DSA_OK) return s;
  }
  // no more blocks than there can be units
  const int per = p.plan.pair ? 2 * p.plan.tq : p.plan.tq;
  const int64_t keys = topk_idx ? topk_width : max_seqlen_k;
  int64_t bound = ((int64_t)total_q / per + num_seqs) * n_kv_heads * (p.plan.max_units > 0 ? keys / (kAttnMinChunk * kAttnKeys) + 1 : 1);
  if (bound > di.sm_count) bound = di.sm_count;
  if (bound > DSA_DEV_STATUS_MAX_BLOCKS) bound = DSA_DEV_STATUS_MAX_BLOCKS;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool q8 = prec != DSA_PREC_BF16;
  cudaError_t e = head_dim == 128 ? (q8 ? launch_paged_attention_128_q8(p, (int)bound, di.sm_count, st)
                                        : launch_paged_attention_128(p, (int)bound, di.sm_count, st))
                                  : (q8 ? launch_paged_attention_64_q8(p, (int)bound, di.sm_count, st)
                                        : launch_paged_attention_64(p, (int)bound, di.sm_count, st));
  if (e != cudaSuccess) return cuda_fail(e, "paged attention launch");
  return DSA_OK;
}

}  // extern "C"
