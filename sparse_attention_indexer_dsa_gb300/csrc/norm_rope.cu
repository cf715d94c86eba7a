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
// needs no exchange between lanes and half as many factors.  A warp takes some of
// a token's rows (all of them where there are tokens enough) and forms the
// token's cos and sin itself, each lane those of its pairs, while the first rows
// are on their way; warps share nothing.
//
// An angle is pos * freq in turns, modulo one: 64-bit fixed point, of which the
// last step alone keeps 24 bits, so far positions lose no more than near ones (in
// FP32 a position of 2^20 would be off by 0.06 rad).
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

// A lane's eight elements: its two groups of four, as pairs for packed arithmetic.
struct Elems {
  float2 v[4];
};

template <bool BF16>
__device__ __forceinline__ void widen4(const Raw<BF16>& r, float2* x) {
  if constexpr (BF16) {
    x[0] = make_float2(__uint_as_float(r.v.x << 16), __uint_as_float(r.v.x & 0xFFFF0000u));
    x[1] = make_float2(__uint_as_float(r.v.y << 16), __uint_as_float(r.v.y & 0xFFFF0000u));
  } else {
    x[0] = make_float2(r.v.x, r.v.y);
    x[1] = make_float2(r.v.z, r.v.w);
  }
}

template <bool BF16>
__device__ __forceinline__ Elems widen(const Raw<BF16> (&r)[2]) {
  Elems x;
  widen4<BF16>(r[0], x.v);
  widen4<BF16>(r[1], x.v + 2);
  return x;
}

template <bool BF16>
__device__ __forceinline__ void store4(void* base, int64_t elem, const float2* x) {
  if constexpr (BF16) {
    __nv_bfloat162 lo = __floats2bfloat162_rn(x[0].x, x[0].y), hi = __floats2bfloat162_rn(x[1].x, x[1].y);
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(base) + elem) =
        make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
  } else {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + elem) = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
  }
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// A lane's eight weights (or shifts); `none` where the call has none.
template <int D>
__device__ __forceinline__ Elems load_w(const void* w, int w_bf16, const Lane<D>& at, float none) {
  Elems o;
  if (!w) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o.v[i] = both(none);
  } else if (w_bf16) {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(w);
    Raw<true> r[2];
    r[0].v = __ldg(reinterpret_cast<const uint2*>(p + at.a));
    r[1].v = __ldg(reinterpret_cast<const uint2*>(p + at.b));
    o = widen<true>(r);
  } else {
    const float* p = reinterpret_cast<const float*>(w);
    Raw<false> r[2];
    r[0].v = __ldg(reinterpret_cast<const float4*>(p + at.a));
    r[1].v = __ldg(reinterpret_cast<const float4*>(p + at.b));
    o = widen<false>(r);
  }
  return o;
}

// Sum of a lane's elements, over the lanes of a row.
template <int LPR>
__device__ __forceinline__ float row_sum(float2 a) {
  float v = a.x + a.y;
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// x -> n; returns 1 / std.
template <int D, bool LAYER>
__device__ __forceinline__ float normalise(Elems& x, float eps) {
  constexpr int LPR = D / 8;
  if (LAYER) {
    const float2 mean = both(row_sum<LPR>(__fadd2_rn(__fadd2_rn(x.v[0], x.v[1]), __fadd2_rn(x.v[2], x.v[3]))) * (-1.f / D));
#pragma unroll
    for (int i = 0; i < 4; ++i) x.v[i] = __fadd2_rn(x.v[i], mean);
  }
  float2 s2 = __fmul2_rn(x.v[0], x.v[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s2 = __ffma2_rn(x.v[i], x.v[i], s2);
  const float inv = rsqrtf(fmaf(row_sum<LPR>(s2), 1.f / D, eps));
#pragma unroll
  for (int i = 0; i < 4; ++i) x.v[i] = __fmul2_rn(x.v[i], both(inv));
  return inv;
}

// The factors of a lane's pairs: of pairs (e, e + 4) side by side, of pairs (2e, 2e + 1) one by one.
struct Turn {
  float cs[4], sn[4];
};

// The pairs turned by their angles (BACK: against them).
template <bool BACK>
__device__ __forceinline__ void turn(Elems& y, const Turn& t, bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = y.v[e].x, b = y.v[e].y, s = BACK ? -t.sn[e] : t.sn[e];
      y.v[e] = make_float2(fmaf(a, t.cs[e], -b * s), fmaf(b, t.cs[e], a * s));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 a = y.v[i], b = y.v[i + 2], c = make_float2(t.cs[2 * i], t.cs[2 * i + 1]);
      const float2 s = make_float2(t.sn[2 * i], t.sn[2 * i + 1]), m = make_float2(-s.x, -s.y);
      y.v[i] = __ffma2_rn(a, c, __fmul2_rn(b, BACK ? s : m));
      y.v[i + 2] = __ffma2_rn(b, c, __fmul2_rn(a, BACK ? m : s));
    }
  }
}

// cos and sin of a lane's pairs at a position.
template <int D>
__device__ __forceinline__ Turn angles(const RopeTable& r, int pos, const Lane<D>& at) {
  Turn t;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    t.cs[e] = 1.f;
    t.sn[e] = 0.f;
    if (at.angle[e] >= 0) {
      const uint64_t turns = (uint64_t)(int64_t)pos * r.freq[at.angle[e]];
      // the upper 32 bits as a signed part of a turn; sincospif takes half turns
      sincospif((float)(int32_t)(uint32_t)(turns >> 32) * 0x1p-31f, &t.sn[e], &t.cs[e]);
    }
  }
  return t;
}

// A warp's share of a token: rows [lo, hi) of queries (kind 0) or keys (kind 1).
struct Share {
  int lo, hi;
  __device__ __forceinline__ Share(const NormRopeParams& p, int part, int kind) {
    const int rows = p.heads[0] + p.heads[1], a = part * p.share, b = min(a + p.share, rows);
    lo = kind ? max(a - p.heads[0], 0) : a;
    hi = kind ? b - p.heads[0] : min(b, p.heads[0]);
  }
};

// Rows of a lane that are requested together, and blocks of an SM: as many bytes under way either way.  Four and
// three / two and four: 32768 tokens of 72 heads, BF16, 201 / 208 us; 9001 of 25 narrow ones, FP32, 20.8 / 18.0.
template <bool BF16>
struct Batch {
  static constexpr int kRows = BF16 ? 4 : 2, kBlocks = BF16 ? 3 : 4;
};

template <int D, bool IN, bool OUT, bool LAYER>
__global__ void __launch_bounds__(kNormThreads, Batch<IN>::kBlocks) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int LPR = D / 8, RPS = 32 / LPR, kBatch = Batch<IN>::kRows;
  const int64_t task = (int64_t)blockIdx.x * (kNormThreads / 32) + (threadIdx.x >> 5);
  if (task >= (int64_t)p.tokens * p.parts) return;
  const int tok = (int)(task / p.parts), part = (int)(task - (int64_t)tok * p.parts);
  const int lane = threadIdx.x & 31, sub = lane / LPR;
  const Lane<D> at(p.rope, lane % LPR);
  const int pos = p.rope.dim > 0 ? __ldg(p.pos + tok) : 0;
  Turn tn;
  bool turned = false;
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    const Share sh(p, part, kind);
    if (sh.lo >= sh.hi) continue;
    const Elems w = load_w<D>(p.w[kind], p.w_bf16, at, 1.f);
    const bool shift = p.b[kind] != nullptr;
    Elems b;
    if (shift) b = load_w<D>(p.b[kind], p.w_bf16, at, 0.f);
    const int64_t x0 = (int64_t)tok * p.x_stride[kind], y0 = (int64_t)tok * p.y_stride[kind];
    for (int h0 = sh.lo + sub; h0 - sub < sh.hi; h0 += kBatch * RPS) {
      Raw<IN> raw[kBatch][2];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int64_t e = x0 + min(h0 + i * RPS, sh.hi - 1) * D;   // (all lanes take part in the sums)
        load4<IN>(raw[i][0], p.x[kind], e + at.a);
        load4<IN>(raw[i][1], p.x[kind], e + at.b);
      }
      if (!turned) {
        tn = angles<D>(p.rope, pos, at);
        turned = true;
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (h0 - sub + i * RPS >= sh.hi) break;
        Elems x = widen<IN>(raw[i]);
        normalise<D, LAYER>(x, p.eps);
#pragma unroll
        for (int e = 0; e < 4; ++e) x.v[e] = shift ? __ffma2_rn(x.v[e], w.v[e], b.v[e]) : __fmul2_rn(x.v[e], w.v[e]);
        turn<false>(x, tn, p.rope.interleaved);
        const int h = h0 + i * RPS;
        if (h < sh.hi) {
          store4<OUT>(p.y[kind], y0 + h * D + at.a, x.v);
          store4<OUT>(p.y[kind], y0 + h * D + at.b, x.v + 2);
        }
      }
    }
  }
}

// Warps take shares in turn and keep the gradients of the weights in registers, each lane those of its
// own eight columns; what a block has gathered goes to the workspace, and a second kernel adds the
// blocks' sums in their order, so that the same inputs give the same bits.
constexpr int kBackBatch = 2;

template <int D, bool IN, bool GRAD, bool LAYER>
__global__ void __launch_bounds__(kNormThreads, 2) norm_rope_back_kernel(const __grid_constant__ NormRopeBackParams q) {
  constexpr int LPR = D / 8, RPS = 32 / LPR, kRows = kNormThreads / LPR;
  __shared__ __align__(16) float red[kRows * D];
  const NormRopeParams& p = q.f;
  const int lane = threadIdx.x & 31, sub = lane / LPR;
  const Lane<D> at(p.rope, lane % LPR);
  Elems dw[2], db[2];
#pragma unroll
  for (int e = 0; e < 4; ++e) dw[0].v[e] = dw[1].v[e] = db[0].v[e] = db[1].v[e] = both(0.f);
  const int64_t tasks = (int64_t)p.tokens * p.parts, warps = (int64_t)gridDim.x * (kNormThreads / 32);
  for (int64_t task = (int64_t)blockIdx.x * (kNormThreads / 32) + (threadIdx.x >> 5); task < tasks; task += warps) {
    const int tok = (int)(task / p.parts), part = (int)(task - (int64_t)tok * p.parts);
    const int pos = p.rope.dim > 0 ? __ldg(p.pos + tok) : 0;
    Turn tn;
    bool turned = false;
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      const Share sh(p, part, kind);
      if (sh.lo >= sh.hi) continue;
      const Elems w = load_w<D>(p.w[kind], p.w_bf16, at, 1.f);
      const int64_t x0 = (int64_t)tok * p.x_stride[kind], g0 = (int64_t)tok * q.dy_stride[kind];
      const int64_t y0 = (int64_t)tok * p.y_stride[kind];
      Raw<IN> raw[kBackBatch][2];
      Raw<GRAD> grad[kBackBatch][2];
      auto load = [&](int h0) {
#pragma unroll
        for (int i = 0; i < kBackBatch; ++i) {
          const int h = min(h0 + i * RPS, sh.hi - 1) * D;   // (all lanes take part in the sums)
          load4<IN>(raw[i][0], p.x[kind], x0 + h + at.a);
          load4<IN>(raw[i][1], p.x[kind], x0 + h + at.b);
          load4<GRAD>(grad[i][0], q.dy[kind], g0 + h + at.a);
          load4<GRAD>(grad[i][1], q.dy[kind], g0 + h + at.b);
        }
      };
      load(sh.lo + sub);
      if (!turned) {
        tn = angles<D>(p.rope, pos, at);
        turned = true;
      }
      for (int h0 = sh.lo + sub; h0 - sub < sh.hi; h0 += kBackBatch * RPS) {
        Elems x[kBackBatch], g[kBackBatch];
#pragma unroll
        for (int i = 0; i < kBackBatch; ++i) {
          x[i] = widen<IN>(raw[i]);
          g[i] = widen<GRAD>(grad[i]);
        }
        load(h0 + kBackBatch * RPS);   // (the next ones are on their way meanwhile; behind the last: the last once more)
#pragma unroll
        for (int i = 0; i < kBackBatch; ++i) {
          if (h0 - sub + i * RPS >= sh.hi) break;
          const int h = h0 + i * RPS;
          const bool live = h < sh.hi;
          const float inv = normalise<D, LAYER>(x[i], p.eps);
          turn<true>(g[i], tn, p.rope.interleaved);
          float2 dot, sum;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (live) {
              dw[kind].v[e] = __ffma2_rn(g[i].v[e], x[i].v[e], dw[kind].v[e]);
              if (LAYER) db[kind].v[e] = __fadd2_rn(db[kind].v[e], g[i].v[e]);
            }
            g[i].v[e] = __fmul2_rn(g[i].v[e], w.v[e]);
            dot = e == 0 ? __fmul2_rn(g[i].v[e], x[i].v[e]) : __ffma2_rn(g[i].v[e], x[i].v[e], dot);
            if (LAYER) sum = e == 0 ? g[i].v[e] : __fadd2_rn(sum, g[i].v[e]);
          }
          const float2 md = both(row_sum<LPR>(dot) * (-1.f / D));
          if (LAYER) sum = both(row_sum<LPR>(sum) * (-1.f / D));
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 t = __ffma2_rn(x[i].v[e], md, g[i].v[e]);
            g[i].v[e] = __fmul2_rn(LAYER ? __fadd2_rn(t, sum) : t, both(inv));
          }
          if (live) {
            store4<IN>(p.y[kind], y0 + h * D + at.a, g[i].v);
            store4<IN>(p.y[kind], y0 + h * D + at.b, g[i].v + 2);
          }
        }
      }
    }
  }
  // rows of lanes -> one row of columns, in their order
  const int row = threadIdx.x / LPR;
#pragma unroll
  for (int j = 0; j < (LAYER ? 4 : 2); ++j) {
    const Elems& v = j < 2 ? dw[j & 1] : db[j & 1];
    __syncthreads();
    store4<false>(red, row * D + at.a, v.v);
    store4<false>(red, row * D + at.b, v.v + 2);
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += kNormThreads) {
      float s = 0.f;
#pragma unroll
      for (int r = 0; r < kRows; ++r) s += red[r * D + c];
      q.part[((int64_t)blockIdx.x * 4 + j) * D + c] = s;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) q.hdr[0] = 0;
}

// Sums of the blocks' parts: a block to 32 columns of one of the four rows.  Sums that the backward
// kernel does not form (db of an rms norm) are not asked for.
constexpr int kJoinWarps = 32;

__global__ void __launch_bounds__(32 * kJoinWarps) norm_rope_join_kernel(const __grid_constant__ NormRopeBackParams q, int D, int blocks) {
  __shared__ float red[kJoinWarps][32];
  const int j = blockIdx.x, lane = threadIdx.x & 31, c = blockIdx.y * 32 + lane, w = threadIdx.x >> 5;
  float* const out = j < 2 ? q.dw[j & 1] : q.db[j & 1];
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && blocks == 0) q.hdr[0] = 0;
  if (!out) return;
  float s = 0.f;
  for (int i = w; i < blocks; i += kJoinWarps) s += q.part[((int64_t)i * 4 + j) * D + c];
  red[w][lane] = s;
  __syncthreads();
  if (w == 0) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < kJoinWarps; ++i) t += red[i][lane];
    out[c] = t;
  }
}

// Rows of a warp's share: a whole token where the tokens alone fill the GPU's warps, else fewer, down to
// one batch of the loop.
void divide(NormRopeParams* p, int D, int batch, int warps) {
  const int rows = p->heads[0] + p->heads[1], least = 32 / (D / 8) * batch;
  int parts = p->tokens > 0 ? (warps + p->tokens - 1) / p->tokens : 1;
  if (parts > (rows + least - 1) / least) parts = (rows + least - 1) / least;
  if (parts < 1) parts = 1;
  p->share = ((rows + parts - 1) / parts + least - 1) / least * least;
  p->parts = (rows + p->share - 1) / p->share;
}

template <int D, bool LAYER>
void run(const NormRopeParams& p, cudaStream_t stream) {
  const int64_t tasks = (int64_t)p.tokens * p.parts;
  const unsigned blocks = (unsigned)((tasks + kNormThreads / 32 - 1) / (kNormThreads / 32));
  if (p.in_bf16) {
    if (p.out_bf16) norm_rope_kernel<D, true, true, LAYER><<<blocks, kNormThreads, 0, stream>>>(p);
    else norm_rope_kernel<D, true, false, LAYER><<<blocks, kNormThreads, 0, stream>>>(p);
  } else {
    if (p.out_bf16) norm_rope_kernel<D, false, true, LAYER><<<blocks, kNormThreads, 0, stream>>>(p);
    else norm_rope_kernel<D, false, false, LAYER><<<blocks, kNormThreads, 0, stream>>>(p);
  }
}

template <int D, bool LAYER>
void run_back(const NormRopeBackParams& q, int blocks, cudaStream_t stream) {
  if (q.f.in_bf16) {
    if (q.dy_bf16) norm_rope_back_kernel<D, true, true, LAYER><<<blocks, kNormThreads, 0, stream>>>(q);
    else norm_rope_back_kernel<D, true, false, LAYER><<<blocks, kNormThreads, 0, stream>>>(q);
  } else {
    if (q.dy_bf16) norm_rope_back_kernel<D, false, true, LAYER><<<blocks, kNormThreads, 0, stream>>>(q);
    else norm_rope_back_kernel<D, false, false, LAYER><<<blocks, kNormThreads, 0, stream>>>(q);
  }
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& call, int D, int sm_count, cudaStream_t stream) {
  if (call.tokens == 0) return cudaSuccess;
  NormRopeParams p = call;
  divide(&p, D, p.in_bf16 ? Batch<true>::kRows : Batch<false>::kRows, 24 * sm_count);
  if (D == 128) {
    if (p.layer) run<128, true>(p, stream);
    else run<128, false>(p, stream);
  } else {
    if (p.layer) run<64, true>(p, stream);
    else run<64, false>(p, stream);
  }
  return cudaGetLastError();
}

cudaError_t launch_norm_rope_back(const NormRopeBackParams& call, int D, int sm_count, cudaStream_t stream) {
  NormRopeBackParams q = call;
  int cap = 2 * sm_count < kNormBackBlocks ? 2 * sm_count : kNormBackBlocks;
  divide(&q.f, D, kBackBatch, 2 * cap * (kNormThreads / 32));   // (two shares to a warp: they differ in length)
  const int64_t tasks = (int64_t)q.f.tokens * q.f.parts;
  int blocks = cap;
  if ((tasks + kNormThreads / 32 - 1) / (kNormThreads / 32) < cap) blocks = (int)((tasks + kNormThreads / 32 - 1) / (kNormThreads / 32));
  if (blocks > 0) {
    if (D == 128) {
      if (q.f.layer) run_back<128, true>(q, blocks, stream);
      else run_back<128, false>(q, blocks, stream);
    } else {
      if (q.f.layer) run_back<64, true>(q, blocks, stream);
      else run_back<64, false>(q, blocks, stream);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  norm_rope_join_kernel<<<dim3(4, D / 32), 32 * kJoinWarps, 0, stream>>>(q, D, blocks);
  return cudaGetLastError();
}

}  // namespace dsa
