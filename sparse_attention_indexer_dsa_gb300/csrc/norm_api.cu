// C ABI of the query/key norms with rotation (include/dsa_idx.h): host-side
// validation and launches.  Never allocates, frees or synchronises.
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "dsa_idx.h"
#include "dsa_status_codes.h"
#include "host_util.h"
#include "norm_params.h"

using namespace dsa;

namespace {

int elem_bytes(dsa_dtype_t t) { return t == DSA_DTYPE_BF16 ? 2 : 4; }

// What the parts of 1 / (2 pi) below leave out grows with the frequency: at the farthest position 2^-28 of a turn here.
constexpr double kMostFreq = 0x1p48;

// A frequency as turns per position, modulo one, in units of 2^-64.  A position multiplies what is lost
// here by up to 2^31, so 1 / (2 pi) comes in two parts and the product's rounding is kept.
uint64_t turns_of(double freq) {
  constexpr double kHigh = 0x1.45f306dc9c883p-3, kLow = -0x1.6b01ec5417056p-57;
  auto units = [](double turns) {
    turns -= std::nearbyint(turns);   // (exact, in [-1/2, 1/2])
    const double u = std::ldexp(turns, 64);
    return u < 0x1p63 ? (uint64_t)(int64_t)u : (uint64_t)1 << 63;
  };
  const double turns = freq * kHigh;
  return units(turns) + units(std::fma(freq, kHigh, -turns) + freq * kLow);
}

// What forward and backward share; y: outputs, or gradients of the inputs.
dsa_status_t fill(NormRopeParams* p, const void* q, int64_t q_stride, const void* k, int64_t k_stride, dsa_dtype_t in_dtype,
                  const void* q_weight, const void* k_weight, const void* q_bias, const void* k_bias,
                  dsa_dtype_t weight_dtype, dsa_norm_t norm, float eps, const int32_t* positions, int total_tokens,
                  int n_heads, int n_kv_heads, int head_dim, int rope_dim, double rope_base, const double* inv_freq,
                  int rope_interleaved, void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                  dsa_dtype_t out_dtype) {
  if (total_tokens < 0 || n_heads < 1 || n_kv_heads < 0) return fail(DSA_ERR_INVALID_ARG, "sizes");
  if (n_heads > 1024 || n_kv_heads > 1024) return fail(DSA_ERR_UNSUPPORTED, "at most 1024 heads");
  if (head_dim != 64 && head_dim != 128) return fail(DSA_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (total_tokens > 0 && (!q || !q_out || (n_kv_heads > 0 && (!k || !k_out)) || (rope_dim > 0 && !positions)))
    return fail(DSA_ERR_INVALID_ARG, "null pointer");
  for (dsa_dtype_t t : {in_dtype, out_dtype, weight_dtype})
    if (t != DSA_DTYPE_F32 && t != DSA_DTYPE_BF16) return fail(DSA_ERR_INVALID_ARG, "dtype");
  if (norm != DSA_NORM_RMS && norm != DSA_NORM_LAYER) return fail(DSA_ERR_INVALID_ARG, "norm");
  if (norm == DSA_NORM_RMS && (q_bias || k_bias)) return fail(DSA_ERR_INVALID_ARG, "an RMS norm takes no biases");
  if (!(eps >= 0.f) || std::isinf(eps)) return fail(DSA_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (rope_dim < 0 || rope_dim > head_dim || rope_dim % 8 != 0)
    return fail(DSA_ERR_INVALID_ARG, "rope_dim must be a multiple of 8 in [0, head_dim]");
  if (rope_dim > 0 && !inv_freq && !(rope_base > 0.0 && std::isfinite(rope_base)))
    return fail(DSA_ERR_INVALID_ARG, "rope_base must be finite and > 0");
  for (const void* a : {q, k, (const void*)q_out, (const void*)k_out, q_weight, k_weight, q_bias, k_bias})
    if (!aligned16(a)) return fail(DSA_ERR_INVALID_ARG, "tensors must be 16-byte aligned");
  dsa_status_t s;
  if ((s = check_stride(&q_stride, n_heads, head_dim, elem_bytes(in_dtype), "q")) != DSA_OK) return s;
  if ((s = check_stride(&q_out_stride, n_heads, head_dim, elem_bytes(out_dtype), "q_out")) != DSA_OK) return s;
  if (n_kv_heads > 0) {
    if ((s = check_stride(&k_stride, n_kv_heads, head_dim, elem_bytes(in_dtype), "k")) != DSA_OK) return s;
    if ((s = check_stride(&k_out_stride, n_kv_heads, head_dim, elem_bytes(out_dtype), "k_out")) != DSA_OK) return s;
  }
  if (inv_freq) {
    for (int i = 0; i < rope_dim / 2; ++i) {
      if (!(std::fabs(inv_freq[i]) <= kMostFreq)) return fail(DSA_ERR_INVALID_ARG, "inv_freq must be finite, and 2^48 at most");
      p->rope.freq[i] = turns_of(inv_freq[i]);
    }
  } else if (rope_dim > 0) {
    // (a power of a few hundred nanoseconds for each pair: the last table of the thread is kept)
    static thread_local double base = 0.0;
    static thread_local int dim = 0;
    static thread_local uint64_t table[64];
    if (base != rope_base || dim != rope_dim) {
      // (a base below one: its frequencies rise)
      if (!(std::pow(rope_base, -2.0 * (rope_dim / 2 - 1) / (double)rope_dim) <= kMostFreq))
        return fail(DSA_ERR_INVALID_ARG, "rope_base gives frequencies above 2^48");
      for (int i = 0; i < rope_dim / 2; ++i) table[i] = turns_of(std::pow(rope_base, -2.0 * i / (double)rope_dim));
      base = rope_base;
      dim = rope_dim;
    }
    std::memcpy(p->rope.freq, table, sizeof(uint64_t) * (rope_dim / 2));
  }
  p->rope.dim = rope_dim;
  p->rope.interleaved = rope_interleaved ? 1 : 0;
  p->x[0] = q;
  p->x[1] = k;
  p->x_stride[0] = q_stride;
  p->x_stride[1] = k_stride;
  p->y[0] = q_out;
  p->y[1] = k_out;
  p->y_stride[0] = q_out_stride;
  p->y_stride[1] = k_out_stride;
  p->w[0] = q_weight;
  p->w[1] = k_weight;
  p->b[0] = q_bias;
  p->b[1] = k_bias;
  p->pos = positions;
  p->heads[0] = n_heads;
  p->heads[1] = n_kv_heads;
  p->tokens = total_tokens;
  p->eps = eps;
  p->layer = norm == DSA_NORM_LAYER;
  p->in_bf16 = in_dtype == DSA_DTYPE_BF16;
  p->out_bf16 = out_dtype == DSA_DTYPE_BF16;
  p->w_bf16 = weight_dtype == DSA_DTYPE_BF16;
  return DSA_OK;
}

}  // namespace

extern "C" {

dsa_status_t dsa_idx_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, dsa_dtype_t in_dtype,
                               const void* q_weight, const void* k_weight, const void* q_bias, const void* k_bias,
                               dsa_dtype_t weight_dtype, dsa_norm_t norm, float eps, const int32_t* positions,
                               int total_tokens, int n_heads, int n_kv_heads, int head_dim, int rope_dim,
                               double rope_base, const double* inv_freq, int rope_interleaved, void* q_out,
                               int64_t q_out_stride, void* k_out, int64_t k_out_stride, dsa_dtype_t out_dtype,
                               dsa_stream_t stream) {
  NormRopeParams p{};
  dsa_status_t s = fill(&p, q, q_stride, k, k_stride, in_dtype, q_weight, k_weight, q_bias, k_bias, weight_dtype, norm, eps,
                        positions, total_tokens, n_heads, n_kv_heads, head_dim, rope_dim, rope_base, inv_freq,
                        rope_interleaved, q_out, q_out_stride, k_out, k_out_stride, out_dtype);
  if (s != DSA_OK) return s;
  DevInfo di;
  if ((s = device_info(&di)) != DSA_OK) return s;
  cudaError_t e = launch_norm_rope(p, head_dim, di.sm_count, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "norm and rotation launch");
  return DSA_OK;
}

size_t dsa_idx_norm_rope_workspace_size(int head_dim) {
  if (head_dim != 64 && head_dim != 128) return 0;
  return DSA_DEV_STATUS_HEADER_BYTES + (size_t)kNormBackBlocks * 4 * head_dim * sizeof(float);
}

dsa_status_t dsa_idx_norm_rope_backward(const void* dq_out, int64_t dq_out_stride, const void* dk_out,
                                        int64_t dk_out_stride, dsa_dtype_t grad_dtype, const void* q, int64_t q_stride,
                                        const void* k, int64_t k_stride, dsa_dtype_t in_dtype, const void* q_weight,
                                        const void* k_weight, dsa_dtype_t weight_dtype, dsa_norm_t norm, float eps,
                                        const int32_t* positions, int total_tokens, int n_heads, int n_kv_heads,
                                        int head_dim, int rope_dim, double rope_base, const double* inv_freq,
                                        int rope_interleaved, void* dq, int64_t dq_stride, void* dk, int64_t dk_stride,
                                        float* dq_weight, float* dk_weight, float* dq_bias, float* dk_bias, void* ws,
                                        size_t ws_bytes, dsa_stream_t stream) {
  NormRopeBackParams p{};
  dsa_status_t s = fill(&p.f, q, q_stride, k, k_stride, in_dtype, q_weight, k_weight, nullptr, nullptr, weight_dtype, norm,
                        eps, positions, total_tokens, n_heads, n_kv_heads, head_dim, rope_dim, rope_base, inv_freq,
                        rope_interleaved, dq, dq_stride, dk, dk_stride, in_dtype);
  if (s != DSA_OK) return s;
  if (total_tokens > 0 && (!dq_out || (n_kv_heads > 0 && !dk_out))) return fail(DSA_ERR_INVALID_ARG, "null pointer");
  if (grad_dtype != DSA_DTYPE_F32 && grad_dtype != DSA_DTYPE_BF16) return fail(DSA_ERR_INVALID_ARG, "dtype");
  if (!aligned16(dq_out) || !aligned16(dk_out)) return fail(DSA_ERR_INVALID_ARG, "tensors must be 16-byte aligned");
  if ((s = check_stride(&dq_out_stride, n_heads, head_dim, elem_bytes(grad_dtype), "dq_out")) != DSA_OK) return s;
  if (n_kv_heads > 0 && (s = check_stride(&dk_out_stride, n_kv_heads, head_dim, elem_bytes(grad_dtype), "dk_out")) != DSA_OK)
    return s;
  if (norm == DSA_NORM_RMS && (dq_bias || dk_bias)) return fail(DSA_ERR_INVALID_ARG, "biases of an RMS norm have no gradient here");
  if ((s = check_ws(ws, ws_bytes, dsa_idx_norm_rope_workspace_size(head_dim))) != DSA_OK) return s;
  DevInfo di;
  if ((s = device_info(&di)) != DSA_OK) return s;
  p.dy[0] = dq_out;
  p.dy[1] = dk_out;
  p.dy_stride[0] = dq_out_stride;
  p.dy_stride[1] = dk_out_stride;
  p.dy_bf16 = grad_dtype == DSA_DTYPE_BF16;
  p.dw[0] = dq_weight;
  p.dw[1] = dk_weight;
  p.db[0] = dq_bias;
  p.db[1] = dk_bias;
  p.hdr = reinterpret_cast<int*>(ws);
  p.part = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(ws) + DSA_DEV_STATUS_HEADER_BYTES);
  cudaError_t e = launch_norm_rope_back(p, head_dim, di.sm_count, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "norm and rotation gradient launch");
  return DSA_OK;
}

}  // extern "C"
