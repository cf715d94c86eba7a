// Norms of queries and keys for each head with the position rotation in the
// same pass, and their gradients.
//   n = x / sqrt(mean x^2 + eps)                    (rms)
//   n = (x - mean x) / sqrt(var x + eps)            (layer, biased variance)
//   y = R(pos) (n w + b)
// R turns the pair i of the first `dim` elements by pos * freq_i.  Backwards,
// with g = R(-pos) dy and gw = g w:
//   dw = sum g n,  db = sum g,  dx = (gw - n mean(gw n) [- mean gw, layer]) / std.
//
// A row of D elements is handled by D / 8 lanes.  Each holds two groups of four
// elements, chosen so that both elements of a pair are its own: the rotation
// needs no exchange between lanes and half as many factors.  The rows of a
// tile of tokens (one token of many heads, several of few) are spread over the
// block; a token's cos and sin are formed once, in shared memory, while the
// rows are on their way.
//
// An angle is pos * freq in turns, modulo one: 64-bit fixed point, so far
// positions lose nothing (in FP32 a position of 2^20 would be off by 0.06 rad).
#include <cuda_bf16.h>

#include "norm_params.h"

namespace dsa {

namespace {

// Where a lane's two groups of four are, and the index of the angle of each of its four pairs
// ((e, e + 4), or (2e, 2e + 1) interleaved); -1: not rotated.
template <int D>
struct Lane {
  int a, b;
  int angle[4];
  __device__ __forceinline__ Lane(const RopeTable& r, int l) {
    const int half = r.dim / 2;
    if (r.interleaved) {
      a = 8 * l;
      b = a + 4;
#pragma unroll
      for (int e = 0; e < 4; ++e) angle[e] = a + 2 * e < r.dim ? a / 2 + e : -1;
    } else {
      const bool rot = 4 * l < half;
      a = rot ? 4 * l : half + 4 * l;                 // (r.dim + (4 l - half))
      b = rot ? a + half : a + (D - r.dim) / 2;
#pragma unroll
      for (int e = 0; e < 4; ++e) angle[e] = rot ? 4 * l + e : -1;
    }
  }
};

// Four consecutive elements as loaded.
template <bool BF16>
struct Raw {
  float4 v;
};
template <>
struct Raw<true> {
  uint2 v;
};

template <bool BF16>
__device__ __forceinline__ void load4(Raw<BF16>& r, const void* base, int64_t elem) {
  if constexpr (BF16)
    r.v = __ldcs(reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(base) + elem));
  else
    r.v = __ldcs(reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + elem));
}

template <bool BF16>
__device__ __forceinline__ void widen4(const Raw<BF16>& r, float* x) {
  if constexpr (BF16) {
    x[0] = __uint_as_float(r.v.x << 16);
    x[1] = __uint_as_float(r.v.x & 0xFFFF0000u);
    x[2] = __uint_as_float(r.v.y << 16);
    x[3] = __uint_as_float(r.v.y & 0xFFFF0000u);
  } else {
    x[0] = r.v.x; x[1] = r.v.y; x[2] = r.v.z; x[3] = r.v.w;
  }
}

template <bool BF16>
__device__ __forceinline__ void store4(void* base, int64_t elem, const float* x) {
  if constexpr (BF16) {
    __nv_bfloat162 lo = __floats2bfloat162_rn(x[0], x[1]), hi = __floats2bfloat162_rn(x[2], x[3]);
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(base) + elem) =
        make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
  } else {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + elem) = make_float4(x[0], x[1], x[2], x[3]);
  }
}

// A lane's eight weights (or shifts); `none` where the call has none.
template <int D>
__device__ __forceinline__ void load_w(const void* w, int w_bf16, const Lane<D>& at, float none, float (&o)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int d = (e < 4 ? at.a : at.b) + (e & 3);
    if (!w) o[e] = none;
    else if (w_bf16) o[e] = __uint_as_float((uint32_t)__ldg(reinterpret_cast<const uint16_t*>(w) + d) << 16);
    else o[e] = __ldg(reinterpret_cast<const float*>(w) + d);
  }
}

// Sum over the lanes of a row.
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// x -> n; returns 1 / std.
template <int D>
__device__ __forceinline__ float normalise(float (&x)[8], bool layer, float eps) {
  constexpr int LPR = D / 8;
  if (layer) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s += x[e];
    const float mean = row_sum<LPR>(s) * (1.f / D);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] -= mean;
  }
  float s2 = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) s2 = fmaf(x[e], x[e], s2);
  const float inv = 1.f / sqrtf(row_sum<LPR>(s2) * (1.f / D) + eps);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] *= inv;
  return inv;
}

// The pairs turned by their angles (with sn negated: back).
__device__ __forceinline__ void turn(float (&y)[8], const float (&cs)[4], const float (&sn)[4], bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = y[2 * e], b = y[2 * e + 1];
      y[2 * e] = fmaf(a, cs[e], -b * sn[e]);
      y[2 * e + 1] = fmaf(b, cs[e], a * sn[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = y[e], b = y[e + 4];
      y[e] = fmaf(a, cs[e], -b * sn[e]);
      y[e + 4] = fmaf(b, cs[e], a * sn[e]);
    }
  }
}

// cos and sin of the tile's tokens [tile][dim / 2], by the block's threads.
__device__ __forceinline__ void fill_angles(const NormRopeParams& p, int t0, int n, float2* tab) {
  const int half = p.rope.dim / 2;
  for (int i = threadIdx.x; i < n * half; i += kNormThreads) {
    const int t = i / half, f = i - t * half;
    const uint64_t turns = (uint64_t)(int64_t)__ldg(p.pos + t0 + t) * p.rope.freq[f];
    // the upper 32 bits as a signed part of a turn; sincospif takes half turns
    const float x = (float)(int32_t)(uint32_t)(turns >> 32) * 0x1p-31f;
    float sv, cv;
    sincospif(x, &sv, &cv);
    tab[i] = make_float2(cv, sv);
  }
}

// A lane's factors of token t of the tile.
template <int D>
__device__ __forceinline__ void load_angles(const float2* tab, int half, int t, const Lane<D>& at, float (&cs)[4],
                                            float (&sn)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 v = at.angle[e] >= 0 ? tab[t * half + at.angle[e]] : make_float2(1.f, 0.f);
    cs[e] = v.x;
    sn[e] = v.y;
  }
}

// Row r of a tile: token, head, and whether it is a key's.
__device__ __forceinline__ void row_at(const NormRopeParams& p, int r, int* tok, int* head, int* kind) {
  const int rows = p.heads[0] + p.heads[1];
  *tok = rows == 1 ? r : (int)__umulhi((uint32_t)r, p.row_mul);   // r / rows
  const int h = r - *tok * rows;
  *kind = h >= p.heads[0];
  *head = *kind ? h - p.heads[0] : h;
}

constexpr int kBatch = 4;   // rows of a lane that are requested together

template <int D, bool IN, bool OUT>
__global__ void __launch_bounds__(kNormThreads) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int LPR = D / 8, RPS = kNormThreads / LPR;
  extern __shared__ float2 tab[];
  const int half = p.rope.dim / 2;
  const int t0 = blockIdx.x * p.tile, n = min(p.tile, p.tokens - t0);
  const int rows = n * (p.heads[0] + p.heads[1]);
  const Lane<D> at(p.rope, threadIdx.x % LPR);
  const int sub = threadIdx.x / LPR;
  float cs[4], sn[4], w[8], b[8];
  int cur_tok = -1, cur_kind = -1;
  bool first = true;
  for (int r0 = 0; r0 < rows; r0 += RPS * kBatch) {
    Raw<IN> raw[kBatch][2];
    int tok[kBatch], head[kBatch], kind[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r0 + i * RPS + sub;
      row_at(p, min(r, rows - 1), &tok[i], &head[i], &kind[i]);   // (all lanes take part in the sums)
      const int64_t e = (int64_t)(t0 + tok[i]) * p.x_stride[kind[i]] + head[i] * D;
      load4<IN>(raw[i][0], p.x[kind[i]], e + at.a);
      load4<IN>(raw[i][1], p.x[kind[i]], e + at.b);
    }
    if (first) {
      if (half > 0) fill_angles(p, t0, n, tab);
      __syncthreads();
      first = false;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r0 + i * RPS + sub;
      if (r0 + i * RPS >= rows) break;
      if (tok[i] != cur_tok) {
        cur_tok = tok[i];
        load_angles<D>(tab, half, cur_tok, at, cs, sn);
      }
      if (kind[i] != cur_kind) {
        cur_kind = kind[i];
        load_w<D>(p.w[cur_kind], p.w_bf16, at, 1.f, w);
        load_w<D>(p.b[cur_kind], p.w_bf16, at, 0.f, b);
      }
      float x[8];
      widen4<IN>(raw[i][0], x);
      widen4<IN>(raw[i][1], x + 4);
      normalise<D>(x, p.layer, p.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = fmaf(x[e], w[e], b[e]);
      turn(x, cs, sn, p.rope.interleaved);
      if (r < rows) {
        const int64_t o = (int64_t)(t0 + tok[i]) * p.y_stride[kind[i]] + head[i] * D;
        store4<OUT>(p.y[kind[i]], o + at.a, x);
        store4<OUT>(p.y[kind[i]], o + at.b, x + 4);
      }
    }
  }
}

// Blocks take tiles in turn and keep the gradients of the weights in registers, each lane those of its
// own eight columns; what a block has gathered goes to the workspace, and a second kernel adds the
// blocks' sums in their order, so that the same inputs give the same bits.
constexpr int kBackBatch = 2;

template <int D, bool IN, bool GRAD>
__global__ void __launch_bounds__(kNormThreads, 2) norm_rope_back_kernel(const __grid_constant__ NormRopeBackParams q) {
  constexpr int LPR = D / 8, RPS = kNormThreads / LPR;
  extern __shared__ float2 tab[];
  const NormRopeParams& p = q.f;
  const int half = p.rope.dim / 2;
  const Lane<D> at(p.rope, threadIdx.x % LPR);
  const int sub = threadIdx.x / LPR;
  float dw[2][8], db[2][8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[0][e] = dw[1][e] = db[0][e] = db[1][e] = 0.f;
  const int tiles = (p.tokens + p.tile - 1) / p.tile;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int t0 = tile * p.tile, n = min(p.tile, p.tokens - t0);
    __syncthreads();   // (the last tile's angles have been read)
    if (half > 0) fill_angles(p, t0, n, tab);
    __syncthreads();
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      const int heads = p.heads[kind], rows = n * heads;
      if (rows == 0) continue;
      float w[8];
      load_w<D>(p.w[kind], p.w_bf16, at, 1.f, w);
      for (int r0 = 0; r0 < rows; r0 += RPS * kBackBatch) {
        Raw<IN> raw[kBackBatch][2];
        Raw<GRAD> grad[kBackBatch][2];
        int tok[kBackBatch], head[kBackBatch];
#pragma unroll
        for (int i = 0; i < kBackBatch; ++i) {
          const int r = min(r0 + i * RPS + sub, rows - 1);
          tok[i] = p.tile == 1 ? 0 : r / heads;
          head[i] = r - tok[i] * heads;
          const int64_t e = (int64_t)(t0 + tok[i]) * p.x_stride[kind] + head[i] * D;
          const int64_t g = (int64_t)(t0 + tok[i]) * q.dy_stride[kind] + head[i] * D;
          load4<IN>(raw[i][0], p.x[kind], e + at.a);
          load4<IN>(raw[i][1], p.x[kind], e + at.b);
          load4<GRAD>(grad[i][0], q.dy[kind], g + at.a);
          load4<GRAD>(grad[i][1], q.dy[kind], g + at.b);
        }
#pragma unroll
        for (int i = 0; i < kBackBatch; ++i) {
          if (r0 + i * RPS >= rows) break;
          const bool live = r0 + i * RPS + sub < rows;
          float cs[4], sn[4], x[8], g[8];
          load_angles<D>(tab, half, tok[i], at, cs, sn);
#pragma unroll
          for (int e = 0; e < 4; ++e) sn[e] = -sn[e];
          widen4<IN>(raw[i][0], x);
          widen4<IN>(raw[i][1], x + 4);
          widen4<GRAD>(grad[i][0], g);
          widen4<GRAD>(grad[i][1], g + 4);
          const float inv = normalise<D>(x, p.layer, p.eps);
          turn(g, cs, sn, p.rope.interleaved);
          float dot = 0.f, sum = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (live) {
              dw[kind][e] = fmaf(g[e], x[e], dw[kind][e]);
              db[kind][e] += g[e];
            }
            g[e] *= w[e];
            dot = fmaf(g[e], x[e], dot);
            sum += g[e];
          }
          dot = row_sum<LPR>(dot) * (1.f / D);
          sum = p.layer ? row_sum<LPR>(sum) * (1.f / D) : 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] = (g[e] - fmaf(x[e], dot, sum)) * inv;
          if (live) {
            const int64_t o = (int64_t)(t0 + tok[i]) * p.y_stride[kind] + head[i] * D;
            store4<IN>(p.y[kind], o + at.a, g);
            store4<IN>(p.y[kind], o + at.b, g + 4);
          }
        }
      }
    }
  }
  // rows of lanes -> one row of columns, in their order
  float* const red = reinterpret_cast<float*>(tab);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float(&v)[8] = j < 2 ? dw[j & 1] : db[j & 1];
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) red[sub * D + (e < 4 ? at.a : at.b) + (e & 3)] = v[e];
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += kNormThreads) {
      float s = 0.f;
      for (int r = 0; r < RPS; ++r) s += red[r * D + c];
      q.part[((int64_t)blockIdx.x * 4 + j) * D + c] = s;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) q.hdr[0] = 0;
}

// Sums of the blocks' parts: a block to one of the four rows, 8 warps x 32 columns at a time.
__global__ void __launch_bounds__(256) norm_rope_join_kernel(const __grid_constant__ NormRopeBackParams q, int D, int blocks) {
  __shared__ float red[8][32];
  const int j = blockIdx.x, c = blockIdx.y * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
  float* const out = j < 2 ? q.dw[j & 1] : q.db[j & 1];
  if (!out) return;
  float s = 0.f;
  for (int i = w; i < blocks; i += 8) s += q.part[((int64_t)i * 4 + j) * D + c];
  red[w][threadIdx.x & 31] = s;
  __syncthreads();
  if (w == 0) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += red[i][threadIdx.x];
    out[c] = t;
  }
}

template <int D>
cudaError_t run(const NormRopeParams& p, cudaStream_t stream) {
  const int blocks = (p.tokens + p.tile - 1) / p.tile;
  const size_t smem = (size_t)p.tile * (p.rope.dim / 2) * sizeof(float2);
  if (p.in_bf16) {
    if (p.out_bf16) norm_rope_kernel<D, true, true><<<blocks, kNormThreads, smem, stream>>>(p);
    else norm_rope_kernel<D, true, false><<<blocks, kNormThreads, smem, stream>>>(p);
  } else {
    if (p.out_bf16) norm_rope_kernel<D, false, true><<<blocks, kNormThreads, smem, stream>>>(p);
    else norm_rope_kernel<D, false, false><<<blocks, kNormThreads, smem, stream>>>(p);
  }
  return cudaGetLastError();
}

template <int D>
cudaError_t run_back(const NormRopeBackParams& q, int sm_count, cudaStream_t stream) {
  const NormRopeParams& p = q.f;
  int blocks = (p.tokens + p.tile - 1) / p.tile;
  const int cap = 2 * sm_count < kNormBackBlocks ? 2 * sm_count : kNormBackBlocks;
  if (blocks > cap) blocks = cap;
  if (blocks > 0) {
    size_t smem = (size_t)p.tile * (p.rope.dim / 2) * sizeof(float2);
    const size_t red = (size_t)(kNormThreads / (D / 8)) * D * sizeof(float);
    if (red > smem) smem = red;
    if (p.in_bf16) {
      if (q.dy_bf16) norm_rope_back_kernel<D, true, true><<<blocks, kNormThreads, smem, stream>>>(q);
      else norm_rope_back_kernel<D, true, false><<<blocks, kNormThreads, smem, stream>>>(q);
    } else {
      if (q.dy_bf16) norm_rope_back_kernel<D, false, true><<<blocks, kNormThreads, smem, stream>>>(q);
      else norm_rope_back_kernel<D, false, false><<<blocks, kNormThreads, smem, stream>>>(q);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  norm_rope_join_kernel<<<dim3(4, D / 32), 256, 0, stream>>>(q, D, blocks);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, int D, cudaStream_t stream) {
  if (p.tokens == 0) return cudaSuccess;
  return D == 128 ? run<128>(p, stream) : run<64>(p, stream);
}

cudaError_t launch_norm_rope_back(const NormRopeBackParams& p, int D, int sm_count, cudaStream_t stream) {
  return D == 128 ? run_back<128>(p, sm_count, stream) : run_back<64>(p, sm_count, stream);
}

}  // namespace dsa
