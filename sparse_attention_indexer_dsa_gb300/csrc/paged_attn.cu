// Attention of new tokens over a paged cache:
//   o[t, h] = sum_s softmax_s(sm_scale q[t, h] . k[s, h / G]) v[s, h / G]
// over the visible keys s of token t (all positions up to its own, or the
// listed ones among them).  One warp per (token, head), one pass over the keys
// with the running maximum and sum in FP32.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "dsa_device.cuh"
#include "paged_params.h"

namespace dsa {

namespace {

constexpr int kThreads = 128;

template <int D, int FMT>
__device__ __forceinline__ void load_cached(const PagedCacheView& c, const void* base, const uint8_t* scale, int64_t row,
                                            int lane, float (&x)[D / 32]) {
  constexpr int VEC = D / 32;
  if constexpr (FMT == 0) {
    const uint16_t* s = reinterpret_cast<const uint16_t*>(base) + row * D + lane * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = __uint_as_float((uint32_t)s[i] << 16);
  } else {
    const uint8_t* s = reinterpret_cast<const uint8_t*>(base) + row * D + lane * VEC;
    const uint32_t e = scale[row * c.sw + (c.sw > 1 ? lane * VEC / 32 : 0)];
    const float f = e == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(e << 23);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const __half_raw h = __nv_cvt_fp8_to_halfraw(s[i], __NV_E4M3);
      x[i] = __half2float(*reinterpret_cast<const __half*>(&h)) * f;
    }
  }
}

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads) paged_attention_kernel(const AttnParams p) {
  constexpr int VEC = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t rows = (int64_t)p.total_q * p.n_heads;
  bool bad = blockIdx.x == 0 && threadIdx.x == 0 && __ldg(p.cu_q + p.num_seqs) > p.total_q;
  for (int64_t r = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); r < rows;
       r += (int64_t)gridDim.x * (kThreads / 32)) {
    const int t = (int)(r / p.n_heads), h = (int)(r % p.n_heads);
    const int d = find_seq(p.cu_q, p.num_seqs, t);
    const int q0 = __ldg(p.cu_q + d), q1 = __ldg(p.cu_q + d + 1);
    const int S = __ldg(p.cu_k + d + 1) - __ldg(p.cu_k + d);
    if (t < q0 || t >= q1) continue;
    if (q1 - q0 > S || q1 - q0 > p.max_seqlen_q || S > p.max_seqlen_k) { bad = true; continue; }
    const int pos = S - (q1 - t);
    float q[VEC], o[VEC];
    const uint16_t* qs = reinterpret_cast<const uint16_t*>(p.q) + (int64_t)t * p.q_stride + h * D + lane * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) { q[i] = __uint_as_float((uint32_t)qs[i] << 16); o[i] = 0.f; }
    float m = -INFINITY, l = 0.f;
    int n = pos + 1;
    if (p.topk_idx) {
      n = p.topk_width;
      if (p.topk_len) n = max(0, min(n, p.topk_len[t]));
    }
    for (int j = 0; j < n; ++j) {
      const int key = p.topk_idx ? p.topk_idx[(int64_t)t * p.topk_width + j] : j;
      if (key < 0 || key > pos) continue;
      const int64_t row = cache_row(p.c, d, key, h / p.group);
      if (row < 0) { bad = true; continue; }
      float k[VEC], v[VEC];
      load_cached<D, FMT>(p.c, p.c.k, p.c.k_scale, row, lane, k);
      load_cached<D, FMT>(p.c, p.c.v, p.c.v_scale, row, lane, v);
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < VEC; ++i) s = fmaf(q[i], k[i], s);
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      s *= p.scale_log2;
      const float mn = fmaxf(m, s);
      const float a = m == -INFINITY ? 0.f : exp2f(m - mn), w = mn == -INFINITY ? 0.f : exp2f(s - mn);
      l = l * a + w;
#pragma unroll
      for (int i = 0; i < VEC; ++i) o[i] = fmaf(w, v[i], o[i] * a);
      m = mn;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.out) + r * D + lane * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) out[i] = __float2bfloat16_rn(o[i] * inv);
    if (p.lse && lane == 0) p.lse[r] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
  }
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) put_block_status(p.hdr, any ? DSA_DEV_ERR_INVALID_ARG : 0);
}

template <int D>
void launch_d(const AttnParams& p, unsigned blocks, cudaStream_t st) {
  if (p.c.fmt == 0) paged_attention_kernel<D, 0><<<blocks, kThreads, 0, st>>>(p);
  else if (p.c.fmt == 1) paged_attention_kernel<D, 1><<<blocks, kThreads, 0, st>>>(p);
  else paged_attention_kernel<D, 2><<<blocks, kThreads, 0, st>>>(p);
}

}  // namespace

cudaError_t launch_paged_attention(const AttnParams& p, int D, int sm_count, cudaStream_t stream) {
  int64_t blocks = ((int64_t)p.total_q * p.n_heads + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > sm_count * 12) blocks = sm_count * 12;
  if (blocks > DSA_DEV_STATUS_MAX_BLOCKS) blocks = DSA_DEV_STATUS_MAX_BLOCKS;
  if (blocks < 1) blocks = 1;
  if (D == 128) launch_d<128>(p, (unsigned)blocks, stream);
  else launch_d<64>(p, (unsigned)blocks, stream);
  return cudaGetLastError();
}

}  // namespace dsa
