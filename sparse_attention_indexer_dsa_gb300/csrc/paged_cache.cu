// Writing new tokens into a paged cache (quantised on the way) and reading a
// cache back as packed rows.  Both are HBM-bound copies of rows of D elements:
//   write  x -> BF16, or codes E4M3(x * 2^-e) with e the smallest exponent that
//          saturates nothing (per 32 elements: MXFP8, per row: FP8), at the
//          position's page and slot;
//   read   the rows of positions 0 .. S_d - 1, as stored or as code * 2^e.
//
// A row is handled by D / 8 consecutive lanes, eight elements each, so a lane
// moves 16 bytes of BF16 and an E4M3 row of 128 is one full line.  A warp takes
// kUnroll steps of consecutive (token, head) rows at a time and requests all of
// them before it looks up where they go, so the loads and the page lookups
// overlap.  Keys and values are two halves of one row range: one launch.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "dsa_device.cuh"
#include "mx_scale.cuh"
#include "paged_params.h"

namespace dsa {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

// Position of a packed row's token: the sequence it was in last time, or a
// search when it has left it.
struct SeqCursor {
  int d = -1, lo = 0, hi = 0;   // rows [lo, hi) of sequence d
  __device__ __forceinline__ void seek(const int32_t* cu, int num_seqs, int t) {
    if (d >= 0 && t >= lo && t < hi) return;
    d = find_seq(cu, num_seqs, t);
    lo = __ldg(cu + d);
    hi = __ldg(cu + d + 1);
  }
};

// Eight elements of a source row, as FP32 bits or as two words of codes.
template <int SRC>
struct Piece {
  float x[8];
};
template <>
struct Piece<2> {
  uint2 codes;
};

template <int SRC>
__device__ __forceinline__ void load_piece(Piece<SRC>& p, const void* base, int64_t elem) {
  if constexpr (SRC == 0) {
    const float4* s = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + elem);
    const float4 a = __ldg(s), b = __ldg(s + 1);
    p.x[0] = a.x; p.x[1] = a.y; p.x[2] = a.z; p.x[3] = a.w;
    p.x[4] = b.x; p.x[5] = b.y; p.x[6] = b.z; p.x[7] = b.w;
  } else if constexpr (SRC == 1) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(base) + elem));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p.x[2 * i] = __uint_as_float(w[i] << 16);
      p.x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    p.codes = __ldg(reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(base) + elem));
  }
}

// Eight elements to E4M3 codes; lanes of one scale block (GL of them) agree on
// the exponent.
template <int GL>
__device__ __forceinline__ uint2 quant8(const float (&x)[8], uint32_t carry, int* scale_byte) {
  uint32_t am = 0;   // magnitudes compare as unsigned integers
#pragma unroll
  for (int i = 0; i < 8; ++i) am = max(am, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = 1; o < GL; o <<= 1) am = max(am, __shfl_xor_sync(0xffffffffu, am, o));
  const int e = mx_exponent_bits(am, carry);
  const float mul = exp2_neg(e);
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] * mul, x[2 * i + 1] * mul), __NV_SATFINITE, __NV_E4M3);
  *scale_byte = e + 127;
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// FMT: 0 BF16, 1 MXFP8, 2 FP8 (dsa_precision_t).  SRC: 0 FP32, 1 BF16, 2 codes.
template <int D, int FMT, int SRC>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const CacheWriteParams p) {
  constexpr int LPR = D / 8;          // lanes per row
  constexpr int RPS = 32 / LPR;       // rows per warp step
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPR, li = lane % LPR;
  const uint32_t n_kv = p.c.n_kv;               // rows stay below 2^31 (checked by the caller)
  const uint32_t half = p.total_q * n_kv;
  const uint32_t rows = p.v ? 2 * half : half;
  const uint32_t carry = mx_carry(p.rule);
  const uint32_t step = gridDim.x * (kThreads / 32) * (RPS * kUnroll);
  bool bad = blockIdx.x == 0 && threadIdx.x == 0 && __ldg(p.cu_q + p.num_seqs) > p.total_q;
  SeqCursor cur;
  for (uint32_t r0 = (blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * (RPS * kUnroll); r0 < rows;
       r0 += step) {
    Piece<SRC> x[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t r = r0 + u * RPS + sub;
      x[u] = Piece<SRC>{};
      if (r < rows) {
        const bool isv = r >= half;
        const uint32_t rr = isv ? r - half : r;
        const uint32_t t = rr / n_kv, h = rr - t * n_kv;
        load_piece<SRC>(x[u], isv ? p.v : p.k, (int64_t)t * (isv ? p.v_stride : p.k_stride) + (int)(h * D + li * 8));
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t r = r0 + u * RPS + sub;
      const bool isv = r >= half;
      const uint32_t rr = isv ? r - half : r;
      const int t = (int)(rr / n_kv), h = (int)(rr - (uint32_t)t * n_kv);
      int64_t row = -1;
      if (r < rows) {
        cur.seek(p.cu_q, p.num_seqs, t);
        if (t >= cur.lo && t < cur.hi) {   // rows behind the last sequence are left alone
          const int s = __ldg(p.cu_k + cur.d + 1) - __ldg(p.cu_k + cur.d);
          row = cache_row(p.c, cur.d, s - (cur.hi - t), h);
          if (s < cur.hi - cur.lo) row = -1;   // more new tokens than cached ones
          bad |= row < 0;
        }
      }
      uint8_t* dst = reinterpret_cast<uint8_t*>(isv ? p.c.v : p.c.k);
      uint8_t* dsc = isv ? p.c.v_scale : p.c.k_scale;
      if constexpr (FMT == 0) {
        uint4 o;
        __nv_bfloat162 b;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          b = __floats2bfloat162_rn(x[u].x[2 * i], x[u].x[2 * i + 1]);
          reinterpret_cast<uint32_t*>(&o)[i] = *reinterpret_cast<uint32_t*>(&b);
        }
        if (row >= 0) *reinterpret_cast<uint4*>(dst + (row * D + li * 8) * 2) = o;
      } else if constexpr (SRC == 2) {
        if (row >= 0) {
          *reinterpret_cast<uint2*>(dst + row * D + li * 8) = x[u].codes;
          constexpr int SW = FMT == 1 ? D / 32 : 1;
          if (li < SW) dsc[row * SW + li] = __ldg((isv ? p.v_scale : p.k_scale) + (size_t)rr * SW + li);
        }
      } else {
        constexpr int GL = FMT == 1 ? 4 : LPR;
        int sb;
        const uint2 c = quant8<GL>(x[u].x, carry, &sb);
        if (row >= 0) {
          *reinterpret_cast<uint2*>(dst + row * D + li * 8) = c;
          if (li % GL == 0) dsc[row * (FMT == 1 ? D / 32 : 1) + li / GL] = (uint8_t)sb;
        }
      }
    }
  }
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) put_block_status(p.hdr, any ? DSA_DEV_ERR_INVALID_ARG : 0);
}

// Rows of ROWB bytes (stored) copied 16 bytes a lane.
template <int D, int FMT, bool DEQ>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const CacheReadParams p) {
  constexpr int ESZ = FMT == 0 ? 2 : 1;
  constexpr int BPL = DEQ ? 8 : 16;           // stored bytes per lane: eight codes widen to 16 bytes
  constexpr int LPR = D * ESZ / BPL;
  constexpr int RPS = 32 / LPR;
  constexpr int SW = FMT == 1 ? D / 32 : (FMT == 2 ? 1 : 0);
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPR, li = lane % LPR;
  const uint32_t n_kv = p.c.n_kv;               // rows stay below 2^31 (checked by the caller)
  const uint32_t half = p.total_k * n_kv;
  const uint32_t rows = p.v ? 2 * half : half;
  const uint32_t step = gridDim.x * (kThreads / 32) * (RPS * kUnroll);
  bool bad = blockIdx.x == 0 && threadIdx.x == 0 && __ldg(p.cu_k + p.num_seqs) > p.total_k;
  SeqCursor cur;
  for (uint32_t r0 = (blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * (RPS * kUnroll); r0 < rows;
       r0 += step) {
    uint4 x[kUnroll];
    uint32_t sc[kUnroll];
    bool ok[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t r = r0 + u * RPS + sub;
      const bool isv = r >= half;
      const uint32_t rr = isv ? r - half : r;
      const int t = (int)(rr / n_kv), h = (int)(rr - (uint32_t)t * n_kv);
      ok[u] = false;
      x[u] = make_uint4(0, 0, 0, 0);
      sc[u] = 0;
      if (r < rows) {
        cur.seek(p.cu_k, p.num_seqs, t);
        if (t >= cur.lo && t < cur.hi) {
          const int64_t row = cache_row(p.c, cur.d, t - cur.lo, h);
          if (row < 0) {
            bad = true;
          } else {
            ok[u] = true;
            const uint8_t* src = reinterpret_cast<const uint8_t*>(isv ? p.c.v : p.c.k) + row * (D * ESZ) + li * BPL;
            const uint8_t* ssc = isv ? p.c.v_scale : p.c.k_scale;
            if constexpr (BPL == 16) {
              x[u] = __ldg(reinterpret_cast<const uint4*>(src));
              if constexpr (SW > 0) {
                if (li < SW) sc[u] = __ldg(ssc + row * SW + li);
              }
            } else {
              const uint2 c = __ldg(reinterpret_cast<const uint2*>(src));
              x[u].x = c.x;
              x[u].y = c.y;
              sc[u] = __ldg(ssc + row * SW + (SW > 1 ? li / 4 : 0));
            }
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (!ok[u]) continue;
      const uint32_t r = r0 + u * RPS + sub;
      const bool isv = r >= half;
      const uint32_t rr = isv ? r - half : r;
      uint8_t* dst = reinterpret_cast<uint8_t*>(isv ? p.v : p.k);
      if constexpr (!DEQ) {
        *reinterpret_cast<uint4*>(dst + (size_t)rr * (D * ESZ) + li * 16) = x[u];
        if constexpr (SW > 0) {
          if (li < SW) (isv ? p.v_scale : p.k_scale)[(size_t)rr * SW + li] = (uint8_t)sc[u];
        }
      } else {
        // code * 2^e is exact in FP32, and in BF16 unless it is below BF16's range
        const float f = sc[u] == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(sc[u] << 23);
        const uint32_t w[2] = {x[u].x, x[u].y};
        uint4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
          const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&hr));
          const __nv_bfloat162 b = __floats2bfloat162_rn(v.x * f, v.y * f);
          reinterpret_cast<uint32_t*>(&o)[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(dst + ((size_t)rr * D + li * 8) * 2) = o;
      }
    }
  }
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) put_block_status(p.hdr, any ? DSA_DEV_ERR_INVALID_ARG : 0);
}

// Blocks for `rows` rows at `rps` rows a block, at most eight per SM (the
// header has a status word for each).
unsigned blocks_for(int64_t rows, int rows_per_block, int sm_count) {
  int64_t b = (rows + rows_per_block - 1) / rows_per_block;
  int64_t cap = (int64_t)sm_count * 8;
  if (cap > DSA_DEV_STATUS_MAX_BLOCKS) cap = DSA_DEV_STATUS_MAX_BLOCKS;
  if (b > cap) b = cap;
  return (unsigned)(b < 1 ? 1 : b);
}

template <int D, int FMT>
void write_src(const CacheWriteParams& p, unsigned blocks, cudaStream_t st) {
  if (p.src == 0) cache_write_kernel<D, FMT, 0><<<blocks, kThreads, 0, st>>>(p);
  else if (p.src == 1) cache_write_kernel<D, FMT, 1><<<blocks, kThreads, 0, st>>>(p);
  else if constexpr (FMT != 0) cache_write_kernel<D, FMT, 2><<<blocks, kThreads, 0, st>>>(p);
}

template <int D>
void write_fmt(const CacheWriteParams& p, unsigned blocks, cudaStream_t st) {
  if (p.c.fmt == 0) write_src<D, 0>(p, blocks, st);
  else if (p.c.fmt == 1) write_src<D, 1>(p, blocks, st);
  else write_src<D, 2>(p, blocks, st);
}

template <int D>
void read_fmt(const CacheReadParams& p, unsigned blocks, cudaStream_t st) {
  if (p.c.fmt == 0) cache_read_kernel<D, 0, false><<<blocks, kThreads, 0, st>>>(p);
  else if (p.c.fmt == 1 && p.dequant) cache_read_kernel<D, 1, true><<<blocks, kThreads, 0, st>>>(p);
  else if (p.c.fmt == 1) cache_read_kernel<D, 1, false><<<blocks, kThreads, 0, st>>>(p);
  else if (p.dequant) cache_read_kernel<D, 2, true><<<blocks, kThreads, 0, st>>>(p);
  else cache_read_kernel<D, 2, false><<<blocks, kThreads, 0, st>>>(p);
}

}  // namespace

cudaError_t launch_cache_write(const CacheWriteParams& p, int D, int sm_count, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.total_q * p.c.n_kv * (p.v ? 2 : 1);
  const unsigned blocks = blocks_for(rows, kThreads / (D / 8) * kUnroll, sm_count);
  if (D == 128) write_fmt<128>(p, blocks, stream);
  else write_fmt<64>(p, blocks, stream);
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const CacheReadParams& p, int D, int sm_count, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.total_k * p.c.n_kv * (p.v ? 2 : 1);
  const int lanes = p.c.fmt == 0 || p.dequant ? D / 8 : D / 16;
  const unsigned blocks = blocks_for(rows, kThreads / lanes * kUnroll, sm_count);
  if (D == 128) read_fmt<128>(p, blocks, stream);
  else read_fmt<64>(p, blocks, stream);
  return cudaGetLastError();
}

}  // namespace dsa
