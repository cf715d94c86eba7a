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
//
// Memory bounds both directions where tokens are many: 32768 tokens of 72 heads of 128,
// BF16, forward 203 us = 88 % of the copy rate, 16384 of 40 backward 88 us = 84 %; 9001 of
// 25 heads of 64, FP32, 17.7 us = 72 %, less than two rounds of the GPU's warps.  A few tokens
// cost a launch, 3.7 us (7.2 backward, with the launch that adds up the blocks' sums).
#include <cuda_bf16.h>

#include <atomic>

#include "norm_params.h"

namespace dsa {

namespace {

// Where a lane's two groups of four are, whether they are rotated (dim is a multiple of 8: all or none) and the index
// of the angle of the first of its four pairs, (e, e + 4), or (2e, 2e + 1) interleaved.
template <int D>
struct Lane {
  int a, b;
  bool rot;
  int angle;
  __device__ __forceinline__ Lane(const RopeTable& r, int l) {
    const int half = r.dim / 2;
    if (r.interleaved) {
      a = 8 * l;
      b = a + 4;
      rot = a < r.dim;
    } else {
      rot = 4 * l < half;
      a = rot ? 4 * l : half + 4 * l;                 // (r.dim + (4 l - half))
      b = rot ? a + half : a + (D - r.dim) / 2;
    }
    angle = 4 * l;
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

__device__ __forceinline__ float keep(float v, uint32_t mask) { return __uint_as_float(__float_as_uint(v) & mask); }

// The pairs turned by their angles (BACK: against them).  mask: all bits, or none where the lane's elements are not
// rotated (0 times a non-finite element would reach its partner; without masks 201 and 87 us in place of the 203 and
// 88 above, a branch around the turn 210 and 90).
template <bool BACK>
__device__ __forceinline__ void turn(Elems& y, const Turn& t, bool interleaved, uint32_t mask) {
  if (interleaved) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = y.v[e].x, b = y.v[e].y, s = BACK ? -t.sn[e] : t.sn[e];
      y.v[e] = make_float2(fmaf(a, t.cs[e], -keep(b, mask) * s), fmaf(b, t.cs[e], keep(a, mask) * s));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 a = y.v[i], b = y.v[i + 2], c = make_float2(t.cs[2 * i], t.cs[2 * i + 1]);
      const float2 s = make_float2(t.sn[2 * i], t.sn[2 * i + 1]), m = make_float2(-s.x, -s.y);
      const float2 ka = make_float2(keep(a.x, mask), keep(a.y, mask)), kb = make_float2(keep(b.x, mask), keep(b.y, mask));
      y.v[i] = __ffma2_rn(a, c, __fmul2_rn(kb, BACK ? s : m));
      y.v[i + 2] = __ffma2_rn(b, c, __fmul2_rn(ka, BACK ? m : s));
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
    if (at.rot) {
      const uint64_t turns = (uint64_t)(int64_t)pos * r.freq[at.angle + e];
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
// three / two and four: 32768 tokens of 72 heads, BF16, 203 / 211 us; 9001 of 25 narrow ones, FP32, 20.7 / 17.6.
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
  const uint32_t mask = at.rot ? ~0u : 0u;
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
        turn<false>(x, tn, p.rope.interleaved, mask);
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
// blocks' sums in their order, so that the same inputs give the same bits.  The rows of the steps to come
// are copied into shared memory of the warp's own, beyond a token's end too.  16384 tokens of 40 heads, BF16:
// 88 us = 84 % of the copy rate; with the next rows in registers 96, steps of 2 rows to a lane 93, four
// stages (one block to an SM) 129.
constexpr int kBackWide = 4;     // rows of a lane in a step, of 16-bit rows
constexpr int kBackRows = 2;     // of others, and of a share at least
constexpr int kBackStages = 3;   // steps of a warp in shared memory
constexpr int kBackBlocks = 2;   // of an SM

// A warp's way through its shares, a step's rows at a time.
template <int ROWS>
struct Walk {
  unsigned tok, dtok;
  int part, dpart, kind, h, hi;
  bool live;
  __device__ __forceinline__ Walk(const NormRopeParams& p, unsigned first, unsigned warps) {
    tok = first / p.parts;
    part = (int)(first - tok * p.parts);
    dtok = warps / p.parts;
    dpart = (int)(warps - dtok * p.parts);
    enter(p);
  }
  __device__ __forceinline__ void enter(const NormRopeParams& p) {
    live = tok < (unsigned)p.tokens;
    const Share s(p, part, 0);
    kind = 0;
    h = s.lo;
    hi = s.hi;
    if (h >= hi) keys(p);
  }
  __device__ __forceinline__ bool keys(const NormRopeParams& p) {
    const Share s(p, part, 1);
    kind = 1;
    h = s.lo;
    hi = s.hi;
    return h < hi;
  }
  __device__ __forceinline__ void next(const NormRopeParams& p) {
    h += ROWS;
    if (h < hi || (kind == 0 && keys(p))) return;
    tok += dtok;
    part += dpart;
    if (part >= p.parts) {
      part -= p.parts;
      ++tok;
    }
    enter(p);
  }
};

__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Sizes of a step in shared memory.
template <int D, bool IN, bool GRAD>
struct BackStep {
  static constexpr int kEach = IN && GRAD ? kBackWide : kBackRows;
  static constexpr int kRows = kEach * 32 / (D / 8);
  static constexpr int kX = kRows * D * (IN ? 2 : 4), kG = kRows * D * (GRAD ? 2 : 4);
  static constexpr int kBytes = kX + kG + 16;   // rows, their gradients, the token's position
  static constexpr int kSmem = kNormThreads / 32 * kBackStages * kBytes;
  static_assert(kSmem >= kNormThreads * 8 * 4, "the lanes' sums meet in the same place");
};

template <bool BF16>
__device__ __forceinline__ void read4(Raw<BF16>& r, const uint8_t* base, int elem) {
  if constexpr (BF16) r.v = *reinterpret_cast<const uint2*>(base + elem * 2);
  else r.v = *reinterpret_cast<const float4*>(base + elem * 4);
}

template <int D, bool IN, bool GRAD, bool LAYER>
__global__ void __launch_bounds__(kNormThreads, kBackBlocks) norm_rope_back_kernel(const __grid_constant__ NormRopeBackParams q) {
  using St = BackStep<D, IN, GRAD>;
  constexpr int LPR = D / 8, RPS = 32 / LPR, kRows = kNormThreads / LPR;
  extern __shared__ __align__(128) uint8_t ring[];
  const NormRopeParams& p = q.f;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / LPR;
  const Lane<D> at(p.rope, lane % LPR);
  const uint32_t mask = at.rot ? ~0u : 0u;
  uint8_t* const own = ring + warp * kBackStages * St::kBytes;
  const uint32_t sown = (uint32_t)__cvta_generic_to_shared(own);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // (the sums' kernel waits for this one's end)
  // sums of the kind of rows at hand, and of the other
  Elems dw, db, dw2, db2;
#pragma unroll
  for (int e = 0; e < 4; ++e) dw.v[e] = db.v[e] = dw2.v[e] = db2.v[e] = both(0.f);
  const unsigned first = blockIdx.x * (kNormThreads / 32) + warp, warps = gridDim.x * (kNormThreads / 32);
  Walk<St::kRows> ahead(p, first, warps), now = ahead;
  int put = 0, get = 0;   // slots
  auto fetch = [&] {
    if (ahead.live) {
      const int n = min(St::kRows, ahead.hi - ahead.h) * D;
      const uint8_t* const x = reinterpret_cast<const uint8_t*>(p.x[ahead.kind]) +
                               ((int64_t)ahead.tok * p.x_stride[ahead.kind] + ahead.h * D) * (IN ? 2 : 4);
      const uint8_t* const g = reinterpret_cast<const uint8_t*>(q.dy[ahead.kind]) +
                               ((int64_t)ahead.tok * q.dy_stride[ahead.kind] + ahead.h * D) * (GRAD ? 2 : 4);
      const uint32_t dst = sown + put * St::kBytes;
#pragma unroll
      for (int o = 0; o < St::kX; o += 512)
        if (o + lane * 16 < n * (IN ? 2 : 4)) copy_async(dst + o + lane * 16, x + o + lane * 16);
#pragma unroll
      for (int o = 0; o < St::kG; o += 512)
        if (o + lane * 16 < n * (GRAD ? 2 : 4)) copy_async(dst + St::kX + o + lane * 16, g + o + lane * 16);
      if (p.rope.dim > 0 && lane == 0)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst + St::kX + St::kG), "l"(p.pos + ahead.tok) : "memory");
      ahead.next(p);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    put = put + 1 < kBackStages ? put + 1 : 0;
  };
#pragma unroll
  for (int i = 0; i < kBackStages - 1; ++i) fetch();
  Turn tn;
  Elems w;
  int kind = -1;   // whose sums dw and db are
  unsigned tok = ~0u;
  while (now.live) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kBackStages - 2) : "memory");
    __syncwarp();
    fetch();   // (into the slot that all lanes have read a step ago)
    const uint8_t* const slot = own + get * St::kBytes;
    get = get + 1 < kBackStages ? get + 1 : 0;
    if (now.tok != tok) {
      tok = now.tok;
      tn = angles<D>(p.rope, p.rope.dim > 0 ? *reinterpret_cast<const int*>(slot + St::kX + St::kG) : 0, at);
    }
    if (now.kind != kind) {   // (at first both are zeros)
      kind = now.kind;
      w = load_w<D>(p.w[kind], p.w_bf16, at, 1.f);
      Elems t = dw;
      dw = dw2;
      dw2 = t;
      t = db;
      db = db2;
      db2 = t;
    }
    const int64_t y0 = (int64_t)now.tok * p.y_stride[kind];
#pragma unroll
    for (int i = 0; i < St::kEach; ++i) {
      if (now.h + i * RPS >= now.hi) break;
      const int r = i * RPS + sub, h = now.h + r;
      const bool there = h < now.hi;   // (else what the slot held before: all lanes take part in the sums)
      Raw<IN> raw[2];
      Raw<GRAD> grad[2];
      read4<IN>(raw[0], slot, r * D + at.a);
      read4<IN>(raw[1], slot, r * D + at.b);
      read4<GRAD>(grad[0], slot + St::kX, r * D + at.a);
      read4<GRAD>(grad[1], slot + St::kX, r * D + at.b);
      Elems x = widen<IN>(raw), g = widen<GRAD>(grad);
      const float inv = normalise<D, LAYER>(x, p.eps);
      turn<true>(g, tn, p.rope.interleaved, mask);
      float2 dot, sum;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (there) {
          dw.v[e] = __ffma2_rn(g.v[e], x.v[e], dw.v[e]);
          if (LAYER) db.v[e] = __fadd2_rn(db.v[e], g.v[e]);
        }
        g.v[e] = __fmul2_rn(g.v[e], w.v[e]);
        dot = e == 0 ? __fmul2_rn(g.v[e], x.v[e]) : __ffma2_rn(g.v[e], x.v[e], dot);
        if (LAYER) sum = e == 0 ? g.v[e] : __fadd2_rn(sum, g.v[e]);
      }
      const float2 md = both(row_sum<LPR>(dot) * (-1.f / D));
      if (LAYER) sum = both(row_sum<LPR>(sum) * (-1.f / D));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 t = __ffma2_rn(x.v[e], md, g.v[e]);
        g.v[e] = __fmul2_rn(LAYER ? __fadd2_rn(t, sum) : t, both(inv));
      }
      if (there) {
        store4<IN>(p.y[kind], y0 + h * D + at.a, g.v);
        store4<IN>(p.y[kind], y0 + h * D + at.b, g.v + 2);
      }
    }
    now.next(p);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  // rows of lanes -> one row of columns, in their order
  float* const red = reinterpret_cast<float*>(ring);
  const int row = threadIdx.x / LPR;
#pragma unroll
  for (int j = 0; j < (LAYER ? 4 : 2); ++j) {
    const bool mine = (j & 1) == kind;   // (by kinds: queries' and keys' in turn)
    Elems v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v.v[e] = j < 2 ? (mine ? dw.v[e] : dw2.v[e]) : (mine ? db.v[e] : db2.v[e]);
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
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the blocks' sums are there
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

template <int D, bool IN, bool GRAD, bool LAYER>
cudaError_t run_back(const NormRopeBackParams& q, int blocks, cudaStream_t stream) {
  constexpr int kSmem = BackStep<D, IN, GRAD>::kSmem;
  auto kernel = norm_rope_back_kernel<D, IN, GRAD, LAYER>;
  static std::atomic<uint64_t> ready{0};   // devices on which this kernel is set up
  int dev = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if (!(ready.load(std::memory_order_acquire) >> (dev & 63) & 1)) {
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem)) != cudaSuccess) return e;
    ready.fetch_or(1ull << (dev & 63), std::memory_order_release);
  }
  kernel<<<blocks, kNormThreads, kSmem, stream>>>(q);
  return cudaGetLastError();
}

template <int D, bool LAYER>
cudaError_t run_back(const NormRopeBackParams& q, int blocks, cudaStream_t stream) {
  if (q.f.in_bf16)
    return q.dy_bf16 ? run_back<D, true, true, LAYER>(q, blocks, stream) : run_back<D, true, false, LAYER>(q, blocks, stream);
  return q.dy_bf16 ? run_back<D, false, true, LAYER>(q, blocks, stream) : run_back<D, false, false, LAYER>(q, blocks, stream);
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
  const int cap = kBackBlocks * sm_count < kNormBackBlocks ? kBackBlocks * sm_count : kNormBackBlocks;
  divide(&q.f, D, kBackRows, 2 * cap * (kNormThreads / 32));   // (two shares to a warp: they differ in length)
  const int64_t tasks = (int64_t)q.f.tokens * q.f.parts;
  int blocks = cap;
  if ((tasks + kNormThreads / 32 - 1) / (kNormThreads / 32) < cap) blocks = (int)((tasks + kNormThreads / 32 - 1) / (kNormThreads / 32));
  if (blocks > 0) {
    const cudaError_t e = D == 128 ? (q.f.layer ? run_back<128, true>(q, blocks, stream) : run_back<128, false>(q, blocks, stream))
                                   : (q.f.layer ? run_back<64, true>(q, blocks, stream) : run_back<64, false>(q, blocks, stream));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = blocks > 0;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(4, D / 32);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_rope_join_kernel, q, D, blocks);
}

}  // namespace dsa
