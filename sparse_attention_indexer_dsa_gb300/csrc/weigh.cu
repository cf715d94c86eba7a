// The attention weight that cached rows gather:
//   W[s, h] += sum_t sum_j exp(sm_scale q[t, j] . k[s, h] - lse[t, j])
// over the new tokens t that see row s and the heads j of key head h; rows of
// the new tokens themselves begin at 0.  With the lse of the attention the
// summands are its softmax weights, so a token adds its number of heads in all.
//
// A warp takes 32 keys of one head at a time and forms their products with 8
// query rows (token, head of the group) by mma.sync m16n8k16.  The operands go
// from memory to registers as they lie: the sum over the head's elements has no
// order, so a lane's 16 contiguous bytes of a row stand for the fragment's
// elements, of queries and keys alike, and nothing passes through shared
// memory.  8-bit rows are widened on the way; E4M3 x 2^e is exact in BF16.
#include <cuda_bf16.h>

#include "dsa_device.cuh"
#include "e4m3_widen.cuh"
#include "weigh.cuh"

namespace dsa {

namespace weigh {

using attn::ex2;
using attn::widen16;

constexpr int kThreads = 256;
constexpr int kKeys = 32;     // keys of a warp's step

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A row is read once: not kept in L1.
__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// First of the groups of kKeys keys of sequence d, in a numbering with room for all of each sequence.
__device__ __forceinline__ int group_base(const WeighParams& p, int d) { return __ldg(p.cu_k + d) / kKeys + d; }

template <int D, bool Q8>
__global__ void __launch_bounds__(kThreads, 2) weigh_kernel(const __grid_constant__ WeighParams p) {
  constexpr int kPieces = Q8 ? D / 64 : D / 32;   // 16-byte pieces of a row to a lane
  constexpr int kQ = D / 32;                      // of a query row
  const int tid = threadIdx.x, lane = tid & 31, t = lane & 3, g = lane >> 2;
  int code = 0;
  // Prefixes that fall make rows count for several sequences, or for none: nothing is computed.
  bool falls = false;
  for (int d = tid; d < p.num_seqs; d += kThreads) {
    Doc o;
    if (!doc_info(p, d, &o)) {
      code = DSA_DEV_ERR_INVALID_ARG;
      falls |= __ldg(p.cu_k + d) < 0 || __ldg(p.cu_k + d + 1) < __ldg(p.cu_k + d) || __ldg(p.cu_q + d) < 0 ||
               __ldg(p.cu_q + d + 1) < __ldg(p.cu_q + d);
    }
  }
  if (tid == 0 && __ldg(p.cu_q + p.num_seqs) > p.total_q) code = DSA_DEV_ERR_INVALID_ARG;
  const bool none = __syncthreads_or(falls);
  const int n_groups = none ? 0 : group_base(p, p.num_seqs);
  const int64_t units = (int64_t)n_groups * p.c.n_kv, warps = (int64_t)gridDim.x * (kThreads / 32);
  const int64_t per = (units + warps - 1) / warps;
  int64_t u = ((int64_t)blockIdx.x * (kThreads / 32) + (tid >> 5)) * per;
  const int64_t u_end = u + per < units ? u + per : units;

  int d = -1, h = -1, base = 0, next_base = 0, n_rows = 0, P0 = 0;
  Doc doc{};
  uint4 qf[kQ];        // rows of the first eight (with n_rows <= 8: of every step)
  float2 bias;
  auto load_q = [&](int r0) {   // query rows r0 .. r0 + 7 (row r0 + g to this lane), and the biases of rows r0 + 2 t, + 1
    auto row = [&](int r, int* tok) {
      *tok = p.group == 1 ? r : (n_rows < 65536 ? (int)__umulhi((uint32_t)r, p.group_mul) : r / p.group);
      return h * p.group + r - *tok * p.group;
    };
    int tok;
    const bool there = r0 + g < n_rows;
    const int hh = row(there ? r0 + g : 0, &tok);
    const uint16_t* src = reinterpret_cast<const uint16_t*>(p.q) + (int64_t)(doc.q0 + tok) * p.q_stride + (int64_t)hh * D;
#pragma unroll
    for (int c = 0; c < kQ; ++c) {
      // the elements that this lane's piece of a key row holds
      const int at = Q8 ? (c >> 1) * 64 + 16 * t + (c & 1) * 8 : c * 32 + 8 * t;
      qf[c] = there ? __ldg(reinterpret_cast<const uint4*>(src + at)) : make_uint4(0, 0, 0, 0);
    }
    float v[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = r0 + 2 * t + e;
      int tk;
      const int hr = row(r < n_rows ? r : 0, &tk);
      const float l = __ldg(p.lse + (int64_t)(doc.q0 + tk) * p.n_heads + hr);
      v[e] = r < n_rows && l != -INFINITY ? -l * kLog2e : -INFINITY;   // (a row that sees no key weighs none)
    }
    bias = make_float2(v[0], v[1]);
  };
  for (; u < u_end; ++u) {
    const int hu = (int)(u / n_groups), gu = (int)(u - (int64_t)hu * n_groups);
    if (d < 0 || hu != h || gu >= next_base) {   // another sequence or head
      int lo = 0, hi = p.num_seqs - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (group_base(p, mid) <= gu) lo = mid; else hi = mid - 1;
      }
      d = lo;
      h = hu;
      base = group_base(p, d);
      next_base = group_base(p, d + 1);
      if (!doc_info(p, d, &doc)) code = DSA_DEV_ERR_INVALID_ARG;
      n_rows = by_steps(p, doc.T) ? doc.T * p.group : 0;
      P0 = doc.S - doc.T;
      if (n_rows > 0 && n_rows <= 8) load_q(0);
    }
    const int key0 = (gu - base) * kKeys;
    if (n_rows == 0 || key0 >= doc.S) {   // to the next sequence
      u += next_base - 1 - gu;
      continue;
    }
    const int64_t mine = key0 + lane < doc.S ? cache_row(p.c, d, key0 + lane, h) : -1;   // this lane's key
    if (key0 + lane < doc.S && mine < 0) code = DSA_DEV_ERR_INVALID_ARG;
    const uint32_t row32 = mine < 0 ? ~0u : (uint32_t)mine;
    uint32_t a[4][kPieces][Q8 ? 8 : 4];   // keys g, g + 8, g + 16, g + 24 as pairs of BF16
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t r = __shfl_sync(0xffffffffu, row32, i * 8 + g);
      if constexpr (Q8) {
        const uint8_t* src = reinterpret_cast<const uint8_t*>(p.c.k) + (size_t)(r == ~0u ? 0 : r) * D + 16 * t;
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {
          const uint4 v = r == ~0u ? make_uint4(0, 0, 0, 0) : load_once(src + c * 64);
          a[i][c][0] = v.x; a[i][c][1] = v.y; a[i][c][2] = v.z; a[i][c][3] = v.w;
          a[i][c][4] = r == ~0u ? 0 : __ldg(p.c.k_scale + (size_t)r * p.c.sw + (p.c.sw == 1 ? 0 : 2 * c + (t >> 1)));
        }
      } else {
        const uint16_t* src = reinterpret_cast<const uint16_t*>(p.c.k) + (size_t)(r == ~0u ? 0 : r) * D + 8 * t;
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {
          const uint4 v = r == ~0u ? make_uint4(0, 0, 0, 0) : load_once(src + c * 32);
          a[i][c][0] = v.x; a[i][c][1] = v.y; a[i][c][2] = v.z; a[i][c][3] = v.w;
        }
      }
    }
    if constexpr (Q8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {
          const uint32_t w4[4] = {a[i][c][0], a[i][c][1], a[i][c][2], a[i][c][3]}, e8 = a[i][c][4];
          if (e8 <= 134u) widen16<false>(w4, e8, a[i][c]);
          else widen16<true>(w4, e8, a[i][c]);
        }
      }
    }
    float sum[4] = {0.f, 0.f, 0.f, 0.f};   // of keys g, g + 8, g + 16, g + 24
    const bool edge = key0 + kKeys > P0 + 1;   // some token does not see some key
    const int r_first = edge && key0 > P0 ? (key0 - P0) * p.group : 0;   // rows before it see none of these keys
    for (int r0 = r_first & ~7; r0 < n_rows; r0 += 8) {
      if (n_rows > 8) load_q(r0);
      float acc[2][4] = {};
#pragma unroll
      for (int c = 0; c < kQ; ++c) {
        const uint32_t* const qw = reinterpret_cast<const uint32_t*>(&qf[c]);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int pc = Q8 ? c >> 1 : c, o = Q8 ? (c & 1) * 4 + 2 * s : 2 * s;
#pragma unroll
          for (int m = 0; m < 2; ++m)
            mma_16816(acc[m], a[2 * m][pc][o], a[2 * m + 1][pc][o], a[2 * m][pc][o + 1], a[2 * m + 1][pc][o + 1], qw[2 * s],
                      qw[2 * s + 1]);
        }
      }
      float w[2][4];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
#pragma unroll
        for (int e = 0; e < 4; ++e) w[m][e] = ex2(fmaf(acc[m][e], p.scale_log2, e & 1 ? bias.y : bias.x));
      }
      if (edge) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = r0 + 2 * t + e;
          const int vis = P0 + (p.group == 1 ? r : (n_rows < 65536 ? (int)__umulhi((uint32_t)r, p.group_mul) : r / p.group));
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            if (key0 + m * 16 + g > vis) w[m][e] = 0.f;
            if (key0 + m * 16 + 8 + g > vis) w[m][2 + e] = 0.f;
          }
        }
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        sum[2 * m] += w[m][0] + w[m][1];
        sum[2 * m + 1] += w[m][2] + w[m][3];
      }
    }
    // sums over the four lanes of a row; lane t ends with key group t
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float give = t & 2 ? sum[e] : sum[e + 2], keep = t & 2 ? sum[e + 2] : sum[e];
      sum[e] = keep + __shfl_xor_sync(0xffffffffu, give, 2);
    }
    const float give = t & 1 ? sum[0] : sum[1], keep = t & 1 ? sum[1] : sum[0];
    const float got = keep + __shfl_xor_sync(0xffffffffu, give, 1);
    const int mykey = t * 8 + g;
    const uint32_t r = __shfl_sync(0xffffffffu, row32, mykey);
    if (r != ~0u) p.weights[r] = key0 + mykey >= P0 ? got : p.weights[r] + got;
  }
  code = __syncthreads_or(code != 0) ? DSA_DEV_ERR_INVALID_ARG : 0;
  if (tid == 0) put_status(p, blockIdx.x, code);
}

}  // namespace weigh

int weigh_step_blocks(const WeighParams& p, int sm_count) {
  // no more blocks than there can be groups of keys
  const int64_t groups = ((int64_t)p.max_seqlen_k / weigh::kKeys + 1) * p.num_seqs * p.c.n_kv;
  const int64_t blocks = (groups + weigh::kThreads / 32 - 1) / (weigh::kThreads / 32);
  return (int)(blocks < 2 * sm_count ? blocks : 2 * sm_count);
}

cudaError_t launch_weigh_steps(const WeighParams& p, int D, int blocks, cudaStream_t stream) {
  using namespace weigh;
  const bool q8 = p.c.fmt != 0;
  if (D == 128) {
    if (q8) weigh_kernel<128, true><<<blocks, kThreads, 0, stream>>>(p);
    else weigh_kernel<128, false><<<blocks, kThreads, 0, stream>>>(p);
  } else {
    if (q8) weigh_kernel<64, true><<<blocks, kThreads, 0, stream>>>(p);
    else weigh_kernel<64, false><<<blocks, kThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace dsa
