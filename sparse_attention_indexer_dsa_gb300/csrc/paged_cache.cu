// Writing new tokens into a paged cache (quantised on the way) and reading a
// cache back as packed rows.  Both are HBM-bound copies of rows of D elements:
//   write  x -> BF16, or codes E4M3(x * 2^-e) with e the smallest exponent that
//          saturates nothing (per 32 elements: MXFP8, per row: FP8), at the
//          position's page and slot;
//   read   the rows of positions 0 .. S_d - 1, as stored or as code * 2^e.
//
// A row is handled by D / 8 consecutive lanes, eight elements each, so a lane
// moves 16 bytes of BF16 and an E4M3 row of 128 is one full line.  A warp takes
// consecutive tokens of one head: their rows, and their scales, are neighbours in
// a page.  (Token by token, eight heads a warp, the rows of a line's neighbours
// came from other blocks: 62 against 43 us for 32768 tokens x 8 heads x 128 of K
// and V into MXFP8.)  U steps of rows are requested before it is looked up where
// they go; where is looked up once per page.  Keys and values are one launch.
// Rows are read once, so 16-byte reads are marked as streaming (index keys as
// stored, 52 MB of them, 15.7 against 17.0 us).  That write is at 70 % of the copy
// rate, bounded by its instructions (issue slots 69 % used, ALU pipe 66 %: the
// quantising, and 8-byte pieces of codes with their places); 8-bit rows back as
// BF16 (212 MB read and written) take 41 us, 76 % of it.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "dsa_device.cuh"
#include "mx_scale.cuh"
#include "paged_params.h"

namespace dsa {

namespace {

constexpr int kThreads = 256;

// Where packed tokens' rows are in the cache, looked up once per page.
struct Place {
  int lo = 0, hi = -1;   // packed tokens [lo, hi): of one sequence and in one page
  int64_t base = -1;     // cache row of token lo, head 0; -1: not there
  bool fits = true;      // false: the sequence or the page does not fit (reported)
  // cu packs the tokens; TAIL: they are the last of the sequence's positions in cu_k.
  template <bool TAIL>
  __device__ __forceinline__ void seek(const PagedCacheView& c, const int32_t* cu, const int32_t* cu_k, int num_seqs, int t) {
    if (t >= lo && t < hi) return;
    const int d = find_seq(cu, num_seqs, t);
    const int s0 = __ldg(cu + d), s1 = __ldg(cu + d + 1);
    lo = t;
    hi = t + 1;
    base = -1;
    fits = true;
    if (t < s0 || t >= s1) return;   // behind the last sequence: left alone
    const int first = TAIL ? __ldg(cu_k + d + 1) - __ldg(cu_k + d) - (s1 - s0) : 0;
    if (first >= 0) base = cache_row(c, d, first + (t - s0), 0);   // else more new tokens than cached ones
    fits = base >= 0;
    if (fits) hi = min(s1, t + (1 << c.page_shift) - ((first + (t - s0)) & ((1 << c.page_shift) - 1)));
  }
};

// Whether a prefix falls, or (packed rows) starts below 0: tokens would count for several sequences or
// for none.  The grid's threads look at a sequence each; what one finds goes to its block's status.
template <bool PACKED>
__device__ __forceinline__ bool falls(const int32_t* cu, int num_seqs) {
  bool bad = false;
  for (uint32_t d = blockIdx.x * kThreads + threadIdx.x; d < (uint32_t)num_seqs; d += gridDim.x * kThreads) {
    const int a = __ldg(cu + d);
    bad |= __ldg(cu + d + 1) < a || (PACKED && a < 0);
  }
  return bad;
}

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
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(base) + elem));
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
template <int D, int FMT, int SRC, int U>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const CacheWriteParams p) {
  constexpr int LPR = D / 8;          // lanes per row
  constexpr int RPS = 32 / LPR;       // rows per step
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPR, li = lane % LPR;
  const uint32_t n_kv = p.c.n_kv, heads = p.v ? 2 * n_kv : n_kv;   // key heads, then value heads
  const uint32_t items = ((p.total_q + RPS * U - 1) / (RPS * U)) * heads;   // below 2^31 (checked by the caller)
  const uint32_t carry = mx_carry(p.rule);
  bool bad = blockIdx.x == 0 && threadIdx.x == 0 && __ldg(p.cu_q + p.num_seqs) > p.total_q;
  bad |= falls<true>(p.cu_q, p.num_seqs) | falls<false>(p.cu_k, p.num_seqs);
  Place at;
  for (uint32_t it = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); it < items; it += gridDim.x * (kThreads / 32)) {
    const uint32_t block = it / heads, hh = it - block * heads;
    const bool isv = hh >= n_kv;
    const uint32_t h = isv ? hh - n_kv : hh;
    const void* src = isv ? p.v : p.k;
    const int64_t stride = isv ? p.v_stride : p.k_stride;
    const int t0 = (int)(block * (RPS * U)) + sub;
    Piece<SRC> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      x[u] = Piece<SRC>{};
      if (t0 + u * RPS < p.total_q) load_piece<SRC>(x[u], src, (t0 + u * RPS) * stride + (int)(h * D + li * 8));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + u * RPS;
      int64_t row = -1;
      if (t < p.total_q) {
        at.seek<true>(p.c, p.cu_q, p.cu_k, p.num_seqs, t);
        bad |= !at.fits;
        if (at.base >= 0) row = at.base + (t - at.lo) + ((int64_t)h << p.c.page_shift);
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
          if (li < SW) dsc[row * SW + li] = __ldg((isv ? p.v_scale : p.k_scale) + ((size_t)t * n_kv + h) * SW + li);
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

template <int D, int FMT, bool DEQ, int U>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const CacheReadParams p) {
  constexpr int ESZ = FMT == 0 ? 2 : 1;
  constexpr int BPL = DEQ ? 8 : 16;           // stored bytes per lane: eight codes widen to 16 bytes
  constexpr int LPR = D * ESZ / BPL;
  constexpr int RPS = 32 / LPR;
  constexpr int SW = FMT == 1 ? D / 32 : (FMT == 2 ? 1 : 0);
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPR, li = lane % LPR;
  const uint32_t n_kv = p.c.n_kv, heads = p.v ? 2 * n_kv : n_kv;   // key heads, then value heads
  const uint32_t items = ((p.total_k + RPS * U - 1) / (RPS * U)) * heads;   // below 2^31 (checked by the caller)
  bool bad = blockIdx.x == 0 && threadIdx.x == 0 && __ldg(p.cu_k + p.num_seqs) > p.total_k;
  bad |= falls<true>(p.cu_k, p.num_seqs);
  Place at;
  for (uint32_t it = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); it < items; it += gridDim.x * (kThreads / 32)) {
    const uint32_t block = it / heads, hh = it - block * heads;
    const bool isv = hh >= n_kv;
    const uint32_t h = isv ? hh - n_kv : hh;
    const uint8_t* pages = reinterpret_cast<const uint8_t*>(isv ? p.c.v : p.c.k) + li * BPL;
    const uint8_t* page_scales = isv ? p.c.v_scale : p.c.k_scale;
    const int t0 = (int)(block * (RPS * U)) + sub;
    uint4 x[U];
    uint32_t sc[U];
    bool ok[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + u * RPS;
      ok[u] = false;
      x[u] = make_uint4(0, 0, 0, 0);
      sc[u] = 0;
      if (t < p.total_k) {
        at.seek<false>(p.c, p.cu_k, p.cu_k, p.num_seqs, t);
        bad |= !at.fits;
        if (at.base >= 0) {
          const int64_t row = at.base + (t - at.lo) + ((int64_t)h << p.c.page_shift);
          ok[u] = true;
          if constexpr (BPL == 16) {
            x[u] = __ldcs(reinterpret_cast<const uint4*>(pages + row * (D * ESZ)));
            if constexpr (SW > 0) {
              if (li < SW) sc[u] = __ldg(page_scales + row * SW + li);
            }
          } else {
            const uint2 c = __ldg(reinterpret_cast<const uint2*>(pages + row * (D * ESZ)));
            x[u].x = c.x;
            x[u].y = c.y;
            sc[u] = __ldg(page_scales + row * SW + (SW > 1 ? li / 4 : 0));
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!ok[u]) continue;
      const size_t rr = (size_t)(t0 + u * RPS) * n_kv + h;
      uint8_t* dst = reinterpret_cast<uint8_t*>(isv ? p.v : p.k);
      if constexpr (!DEQ) {
        *reinterpret_cast<uint4*>(dst + rr * (D * ESZ) + li * 16) = x[u];
        if constexpr (SW > 0) {
          if (li < SW) (isv ? p.v_scale : p.k_scale)[rr * SW + li] = (uint8_t)sc[u];
        }
      } else {
        // code * 2^e is exact in FP32, and in BF16 unless it is below BF16's range
        const float f = __uint_as_float(max(sc[u] << 23, 0x00400000u) | (sc[u] + 1) >> 8 << 22);   // (255: NaN)
        const uint32_t w[2] = {x[u].x, x[u].y};
        uint4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
          const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&hr));
          const __nv_bfloat162 b = __floats2bfloat162_rn(v.x * f, v.y * f);
          reinterpret_cast<uint32_t*>(&o)[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(dst + (rr * D + li * 8) * 2) = o;
      }
    }
  }
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) put_block_status(p.hdr, any ? DSA_DEV_ERR_INVALID_ARG : 0);
}

// Blocks for `items` warp items, at most twelve per SM (the header has a status
// word for each).
unsigned blocks_for(int64_t items, int sm_count) {
  int64_t b = (items + kThreads / 32 - 1) / (kThreads / 32);
  int64_t cap = (int64_t)sm_count * 12;
  if (cap > DSA_DEV_STATUS_MAX_BLOCKS) cap = DSA_DEV_STATUS_MAX_BLOCKS;
  if (b > cap) b = cap;
  return (unsigned)(b < 1 ? 1 : b);
}

// Steps of rows a warp requests at once: four, and one where four would leave SMs
// without work (the lookups of a few tokens then run side by side).  Always four,
// this rule, always one: 16 tokens x 8 heads into MXFP8 5.1 / 2.8 / 2.8 us, the
// 32768-token write 42.7 / 42.7 / 68.5, 1024 tokens 3.6 / 3.6 / 4.4.
constexpr int kUnroll = 4;
bool few(int64_t steps, int sm_count) { return steps < (int64_t)sm_count * (kThreads / 32) * kUnroll; }

template <int D, int FMT, int SRC>
void write_u(const CacheWriteParams& p, int sm_count, cudaStream_t st) {
  constexpr int RPS = 32 / (D / 8);
  const int64_t heads = (int64_t)p.c.n_kv * (p.v ? 2 : 1), steps = ((int64_t)p.total_q + RPS - 1) / RPS;
  if (few(steps * heads, sm_count))
    cache_write_kernel<D, FMT, SRC, 1><<<blocks_for(steps * heads, sm_count), kThreads, 0, st>>>(p);
  else
    cache_write_kernel<D, FMT, SRC, kUnroll>
        <<<blocks_for((steps + kUnroll - 1) / kUnroll * heads, sm_count), kThreads, 0, st>>>(p);
}

template <int D, int FMT>
void write_src(const CacheWriteParams& p, int sm_count, cudaStream_t st) {
  if (p.src == 0) write_u<D, FMT, 0>(p, sm_count, st);
  else if (p.src == 1) write_u<D, FMT, 1>(p, sm_count, st);
  else if constexpr (FMT != 0) write_u<D, FMT, 2>(p, sm_count, st);
}

template <int D>
void write_fmt(const CacheWriteParams& p, int sm_count, cudaStream_t st) {
  if (p.c.fmt == 0) write_src<D, 0>(p, sm_count, st);
  else if (p.c.fmt == 1) write_src<D, 1>(p, sm_count, st);
  else write_src<D, 2>(p, sm_count, st);
}

template <int D, int FMT, bool DEQ>
void read_u(const CacheReadParams& p, int sm_count, cudaStream_t st) {
  constexpr int RPS = 32 / (D * (FMT == 0 ? 2 : 1) / (DEQ ? 8 : 16));
  const int64_t heads = (int64_t)p.c.n_kv * (p.v ? 2 : 1), steps = ((int64_t)p.total_k + RPS - 1) / RPS;
  if (few(steps * heads, sm_count))
    cache_read_kernel<D, FMT, DEQ, 1><<<blocks_for(steps * heads, sm_count), kThreads, 0, st>>>(p);
  else
    cache_read_kernel<D, FMT, DEQ, kUnroll>
        <<<blocks_for((steps + kUnroll - 1) / kUnroll * heads, sm_count), kThreads, 0, st>>>(p);
}

template <int D>
void read_fmt(const CacheReadParams& p, int sm_count, cudaStream_t st) {
  if (p.c.fmt == 0) read_u<D, 0, false>(p, sm_count, st);
  else if (p.c.fmt == 1 && p.dequant) read_u<D, 1, true>(p, sm_count, st);
  else if (p.c.fmt == 1) read_u<D, 1, false>(p, sm_count, st);
  else if (p.dequant) read_u<D, 2, true>(p, sm_count, st);
  else read_u<D, 2, false>(p, sm_count, st);
}

}  // namespace

cudaError_t launch_cache_write(const CacheWriteParams& p, int D, int sm_count, cudaStream_t stream) {
  if (D == 128) write_fmt<128>(p, sm_count, stream);
  else write_fmt<64>(p, sm_count, stream);
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const CacheReadParams& p, int D, int sm_count, cudaStream_t stream) {
  if (D == 128) read_fmt<128>(p, sm_count, stream);
  else read_fmt<64>(p, sm_count, stream);
  return cudaGetLastError();
}

}  // namespace dsa
