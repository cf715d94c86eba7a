// Gathered attention weight of long chunks, on the tensor cores: the keys are the
// products' rows, the queries their columns, S^T = K Q^T, so that a thread has
// a key and adds up its weights exp(scale s - lse) over the queries in registers.
//
// A unit is 256 keys of one head of one sequence and a range of the tokens that
// see them; its keys stay in shared memory as two tiles of 128 (two streams,
// 256 TMEM columns each) while tiles of 256 query rows (tokens x heads of the
// group) pass.  While one stream's warpgroup turns its columns into weights the
// tensor core forms the other's: per 128 x 256 tile the products take 1024
// cycles of an SM and the exponentials as long.  (Keys of one tile alone would
// have each query row read from the L2 twice as often.)
//
// Queries come by TMA (a box of tokens x heads is the tile as the MMA reads it),
// keys row by row through the page table, 8-bit ones widened on the way; they
// change once a unit.  Where a call has few units the tokens are divided too,
// and a second kernel adds the parts in their order.
#include <cuda_bf16.h>

#include <atomic>

#include "e4m3_widen.cuh"
#include "tile_pipeline.cuh"
#include "weigh.cuh"

namespace dsa {

namespace weigh {

using namespace attn;

constexpr int kTileThreads = 512;
constexpr int kGroups = 64;            // sequences are counted in this many groups
constexpr int kHalf = kWeighCols / 2;   // columns of a product and of a hand-over
constexpr int kBiasRing = 4;
constexpr int kMinTiles = 8;           // query tiles of a part, at least
// barriers
enum { K_FULL = 0, K_EMPTY = 2, S_FULL = 4, S_EMPTY = 8, B_FULL = 12, B_EMPTY = B_FULL + kBiasRing, DRAIN = B_EMPTY + kBiasRing,
       Q_FULL, kMaxStages = 4, Q_EMPTY = Q_FULL + kMaxStages, kBars = Q_EMPTY + kMaxStages };

template <int D>
struct Layout {
  static constexpr uint32_t kKeyTile = 128 * D * 2;              // one stream's keys
  static constexpr uint32_t kQueryTile = kWeighCols * D * 2;
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr uint32_t kOffQ = 2 * kKeyTile;
  static constexpr uint32_t kOffBias = kOffQ + kStages * kQueryTile;   // [kBiasRing][256] bias, then [kBiasRing][256] last key seen
  static constexpr uint32_t kOffBars = kOffBias + 2 * kBiasRing * kWeighCols * 4;
  static constexpr uint32_t kOffCtl = kOffBars + kBars * 8;      // status, abort, tmem, tiles of a part
  static constexpr uint32_t kOffTab = kOffCtl + 16;
  static constexpr uint32_t kSmem = kOffTab + (kGroups + 1) * 4;
  static_assert(kSmem <= kAttnSmemMax, "shared memory");
};

// The units of a call, the same in every block: `tab` the first unit of each group of sequences.
struct Units {
  const int* tab;
  int gsz;     // sequences of a group
  int chunk;   // query tiles of a part, at most
};

__device__ __forceinline__ int tiles_of(int tokens, int tq) { return (tokens + tq - 1) / tq; }
__device__ __forceinline__ int parts_of(int tiles, int chunk) { return tiles <= chunk ? 1 : (tiles + chunk - 1) / chunk; }

// A sequence's key pairs of tiles and query tiles; 0 where it is not this kernel's.
__device__ __forceinline__ void doc_tiles(const WeighParams& p, int d, Doc* o, int* kt, int* mt) {
  doc_info(p, d, o);
  const bool ours = !by_steps(p, o->T);
  *kt = ours ? (o->S + kWeighKeys - 1) / kWeighKeys : 0;
  *mt = ours ? tiles_of(o->T, kWeighCols / p.group) : 0;
}

// Counts the units.  `scratch` 2 * kGroups floats, `tab` kGroups + 1, in shared memory; the whole block calls.
// Returns the query tiles of a part; tab[kGroups] the number of units.
__device__ __forceinline__ int count_units(const WeighParams& p, int gsz, int* tab, float* scratch) {
  const int tid = threadIdx.x;
  __shared__ int chunk_of;
  bool falls = false;   // prefixes that fall: nothing is computed
  float work = 0.f, units = 0.f;
  if (tid < kGroups) {
    for (int i = 0; i < gsz && tid * gsz + i < p.num_seqs; ++i) {
      const int d = tid * gsz + i;
      Doc o;
      int kt, mt;
      doc_tiles(p, d, &o, &kt, &mt);
      work += (float)kt * mt * p.c.n_kv;
      units += (float)kt * p.c.n_kv;
      falls |= __ldg(p.cu_k + d) < 0 || __ldg(p.cu_k + d + 1) < __ldg(p.cu_k + d) || __ldg(p.cu_q + d) < 0 ||
               __ldg(p.cu_q + d + 1) < __ldg(p.cu_q + d);
    }
    scratch[tid] = work;
    scratch[kGroups + tid] = units;
  }
  const bool none = __syncthreads_or(falls);
  if (tid < 32) {
    float w = scratch[tid] + scratch[tid + 32], u = scratch[kGroups + tid] + scratch[kGroups + tid + 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      w += __shfl_xor_sync(0xffffffffu, w, o);
      u += __shfl_xor_sync(0xffffffffu, u, o);
    }
    // enough units, or nothing to share out, or (sequences that share pages) more than can be counted
    if (tid == 0)
      chunk_of = none || u > 1e9f ? 0 : (u >= kWeighBalance ? 0x7FFFFFFF : max(kMinTiles, (int)ceilf(w / kWeighBalance)));
  }
  __syncthreads();
  const int chunk = chunk_of;
  int mine = 0;
  if (tid < kGroups && chunk > 0) {
    for (int i = 0; i < gsz && tid * gsz + i < p.num_seqs; ++i) {
      Doc o;
      int kt, mt;
      doc_tiles(p, tid * gsz + i, &o, &kt, &mt);
      mine += kt * p.c.n_kv * parts_of(mt, chunk);
    }
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if ((tid & 31) >= o) incl += y;
  }
  if (tid == 31) tab[kGroups] = incl;
  __syncthreads();
  const int before = incl - mine + (tid >= 32 ? tab[kGroups] : 0);
  __syncthreads();
  if (tid < kGroups) tab[tid] = before;
  if (tid == kGroups - 1) tab[kGroups] = before + mine;
  __syncthreads();
  return chunk;
}

struct Unit {
  int d, h, key0, parts, part;
  int q0, T, S, P0;
  int i0, n;     // first token, query tiles
};

__device__ __forceinline__ Unit decode_unit(const WeighParams& p, const Units& us, int u) {
  int lo = 0, hi = kGroups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (us.tab[mid] <= u) lo = mid; else hi = mid - 1;
  }
  int rem = u - us.tab[lo], d = lo * us.gsz;
  Unit x;
  Doc o;
  int kt, mt;
  for (;; ++d) {
    doc_tiles(p, d, &o, &kt, &mt);
    x.parts = parts_of(mt, us.chunk);
    const int units = kt * p.c.n_kv * x.parts;
    if (rem < units || d + 1 >= p.num_seqs) break;
    rem -= units;
  }
  x.d = d;
  x.part = rem % x.parts;
  rem /= x.parts;
  x.h = rem % p.c.n_kv;
  x.key0 = rem / p.c.n_kv * kWeighKeys;     // (the keys that most tokens see first)
  x.q0 = o.q0;
  x.T = o.T;
  x.S = o.S;
  x.P0 = o.S - o.T;
  const int tq = kWeighCols / p.group, first = max(0, x.key0 - x.P0), n = tiles_of(x.T - first, tq);
  const int a = (int)((int64_t)n * x.part / x.parts), b = (int)((int64_t)n * (x.part + 1) / x.parts);
  x.i0 = first + a * tq;
  x.n = b - a;
  return x;
}

template <int D, bool Q8>
__global__ void __launch_bounds__(kTileThreads, 1) weigh_tiles_kernel(const __grid_constant__ WeighParams p) {
  using L = Layout<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sbase = smem_u32(smem);
  const uint64_t tmo = p.timeout_ns;
  int* const ctl = reinterpret_cast<int*>(smem + L::kOffCtl);
  int* const status = ctl;
  volatile int* const abort_flag = ctl + 1;
  auto bar = [&](int i) { return sbase + L::kOffBars + 8u * i; };
  constexpr int kMmaWarp = 14;
  if (tid == 0) {
    ctl[0] = (sbase & 1023u) ? DSA_DEV_ERR_BOUNDS : 0;   // the swizzle needs a 1024-byte base
    ctl[1] = (sbase & 1023u) ? 1 : 0;
    for (int w = 0; w < 2; ++w) {
      mbar_init(bar(K_FULL + w), 4);
      mbar_init(bar(K_EMPTY + w), 1);
    }
    for (int i = 0; i < 4; ++i) {   // half tiles: 2 w + half
      mbar_init(bar(S_FULL + i), 1);
      mbar_init(bar(S_EMPTY + i), 4);
    }
    for (int s = 0; s < kBiasRing; ++s) {
      mbar_init(bar(B_FULL + s), 1);
      mbar_init(bar(B_EMPTY + s), 8);
    }
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(bar(Q_FULL + s), 1);
      mbar_init(bar(Q_EMPTY + s), 1);
    }
    mbar_init(bar(DRAIN), 1);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc(smem_u32(ctl + 2), 512);
  // rows that no box covers (heads that do not divide 256) read as zeros
  for (uint32_t i = tid * 16; i < L::kStages * L::kQueryTile; i += kTileThreads * 16)
    *reinterpret_cast<uint4*>(smem + L::kOffQ + i) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  Units us;
  int* const tab = reinterpret_cast<int*>(smem + L::kOffTab);
  us.tab = tab;
  us.gsz = (p.num_seqs + kGroups - 1) / kGroups;
  us.chunk = count_units(p, us.gsz, tab, reinterpret_cast<float*>(smem + L::kOffBias));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)ctl[2];
  const int n_units = tab[kGroups], tq = kWeighCols / p.group;

  if (warp < 8) {
    // ======================= weights: a key to a thread =======================
    const int w = warp >> 2, quarter = warp & 3;
    const uint32_t t_s = tmem + (uint32_t)w * kWeighCols + ((uint32_t)quarter << 21);
    const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
    uint32_t nt = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < n_units && ok; u += gridDim.x) {
      const Unit x = decode_unit(p, us, u);
      const int wkey = x.key0 + w * 128 + quarter * 32, key = wkey + lane;   // the warp's first key, this thread's
      float2 sum[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] = make_float2(0.f, 0.f);
      for (int j = 0; j < x.n; ++j, ++nt) {
        const int slot = nt % kBiasRing;
        const int i0 = x.i0 + j * tq, tokens = min(tq, x.T - i0), cols = tokens * p.group;
        const float* const bias = reinterpret_cast<const float*>(smem + L::kOffBias) + slot * kWeighCols;
        const int* const seen = reinterpret_cast<const int*>(smem + L::kOffBias) + (kBiasRing + slot) * kWeighCols;
        const bool any = wkey <= x.P0 + i0 + tokens - 1 && wkey < x.S;   // (else no token of the tile sees a key of the warp)
        // some key that some token does not see, or columns of other sequences' tokens
        const bool edge = wkey + 31 > x.P0 + i0 || tokens < tq;
        ok = __all_sync(0xffffffffu, wait_bar(bar(B_FULL + slot), (nt / kBiasRing) & 1u, abort_flag, status, tmo));
#pragma unroll 1
        for (int half = 0; half < 2 && ok; ++half) {
          const int c0 = half * kHalf;
          ok = __all_sync(0xffffffffu, wait_bar(bar(S_FULL + 2 * w + half), nt & 1u, abort_flag, status, tmo));
          if (!ok) break;
          tc_fence_after();
          auto release = [&] {   // the half's columns have been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(S_EMPTY + 2 * w + half));
          };
          if (!any || c0 >= cols) {
            release();
          } else if (!edge) {
            // the next 32 columns are on their way while these become weights
            uint32_t s[2][32];
            tmem_ld_x32(t_s + c0, s[0]);
#pragma unroll
            for (int c = 0; c < kHalf / 32; ++c) {
              tmem_ld_wait_tied<32>(s[c & 1]);
              if (c + 1 < kHalf / 32) tmem_ld_x32(t_s + c0 + 32 * (c + 1), s[(c + 1) & 1]);
              else release();
              const float* const b32 = bias + c0 + 32 * c;
              const uint32_t* const v = s[c & 1];
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
                const float4 b = *reinterpret_cast<const float4*>(b32 + 2 * i);
                float2 e0 = ffma2(as_f2(v[2 * i], v[2 * i + 1]), sc2, make_float2(b.x, b.y));
                float2 e1 = ffma2(as_f2(v[2 * i + 2], v[2 * i + 3]), sc2, make_float2(b.z, b.w));
                e0.x = ex2(e0.x);
                e0.y = ex2(e0.y);
                e1.x = ex2(e1.x);
                e1.y = ex2(e1.y);
                sum[i & 2] = __fadd2_rn(sum[i & 2], e0);
                sum[(i & 2) + 1] = __fadd2_rn(sum[(i & 2) + 1], e1);
              }
            }
          } else {
            const int end = min(cols, c0 + kHalf);
#pragma unroll 1
            for (int c = c0; c < end; c += 32) {
              uint32_t s[32];
              tmem_ld_x32(t_s + c, s);
              tmem_ld_wait_tied<32>(s);
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float e = ex2(fmaf(__uint_as_float(s[i]), p.scale_log2, bias[c + i]));
                sum[(i >> 1) & 3].x += key <= seen[c + i] ? e : 0.f;
              }
            }
            release();
          }
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_EMPTY + slot));
      }
      if (!ok) break;
      const float total = ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y)) + ((sum[2].x + sum[2].y) + (sum[3].x + sum[3].y));
      if (x.parts > 1) {
        p.part[(int64_t)u * kWeighKeys + w * 128 + quarter * 32 + lane] = total;
      } else if (key < x.S) {
        const int64_t r = cache_row(p.c, x.d, key, x.h);   // (-1 is reported by the loaders)
        if (r >= 0) p.weights[r] = key >= x.P0 ? total : p.weights[r] + total;
      }
    }
  } else if (warp < 12) {
    // ======================= keys =======================
    const int kw = warp - 8;   // a quarter of a tile
    uint32_t nk = 0;
    bool ok = true, bad_page = false;
    for (int u = blockIdx.x; u < n_units && ok; u += gridDim.x) {
      const Unit x = decode_unit(p, us, u);
      if (x.n == 0) continue;
#pragma unroll 1
      for (int w = 0; w < 2 && ok; ++w) {
        const int key = x.key0 + w * 128 + kw * 32 + lane;
        const int64_t mine = key < x.S ? cache_row(p.c, x.d, key, x.h) : -1;
        if (key < x.S && mine < 0) bad_page = true;
        const uint32_t row32 = mine < 0 ? ~0u : (uint32_t)mine;
        if (nk > 0) ok = __all_sync(0xffffffffu, wait_bar(bar(K_EMPTY + w), (nk - 1) & 1u, abort_flag, status, tmo));
        if (!ok) break;
        const uint32_t dst = sbase + w * L::kKeyTile + kw * 32 * 128;
        if constexpr (Q8) {
          constexpr int PPR = D / 16, RPP = 32 / PPR, kPasses = 32 / RPP, kBatch = 4;
          const int c = lane % PPR, rsub = lane / PPR;
          const uint8_t* const src = reinterpret_cast<const uint8_t*>(p.c.k) + c * 16;
          const int sc = p.c.sw == 1 ? 0 : c >> 1;
#pragma unroll 1
          for (int i0 = 0; i0 < kPasses; i0 += kBatch) {
            uint4 v[kBatch];
            uint32_t e8[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              const uint32_t r = __shfl_sync(0xffffffffu, row32, (i0 + i) * RPP + rsub);
              v[i] = r == ~0u ? make_uint4(0, 0, 0, 0) : __ldg(reinterpret_cast<const uint4*>(src + (size_t)r * D));
              e8[i] = r == ~0u ? 0u : __ldg(p.c.k_scale + (size_t)r * p.c.sw + sc);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              const int r = (i0 + i) * RPP + rsub;
              const uint32_t w4[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
              uint32_t o[8];
              if (e8[i] <= 134u) widen<false>(w4, e8[i], o);
              else widen<true>(w4, e8[i], o);
              const uint32_t at = dst + (uint32_t)(c >> 2) * (128 * 128) + r * 128;
              st_shared_v4(at + ((((c & 3) * 2) ^ (r & 7)) << 4), o[0], o[1], o[2], o[3]);
              st_shared_v4(at + ((((c & 3) * 2 + 1) ^ (r & 7)) << 4), o[4], o[5], o[6], o[7]);
            }
          }
        } else {
          constexpr int PPR = D / 8, RPP = 32 / PPR;
          const int c = lane % PPR, rsub = lane / PPR;
          const uint16_t* const src = reinterpret_cast<const uint16_t*>(p.c.k) + c * 8;
#pragma unroll
          for (int i = 0; i < 32; i += RPP) {
            const uint32_t e = __shfl_sync(0xffffffffu, row32, i + rsub);
            const int r = i + rsub;
            cp_async16(dst + (uint32_t)(c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                       src + (size_t)(e == ~0u ? 0 : e) * D, e != ~0u);
          }
          cp_wait_all();
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(K_FULL + w));
      }
      ++nk;
    }
    if (bad_page) set_status(status, DSA_DEV_ERR_INVALID_ARG);
  } else if (warp == 12) {
    // ======================= queries =======================
    const uint32_t bytes = (uint32_t)tq * p.group * D * 2;
    uint32_t nt = 0;
    bool ok = true, withheld = false;
    for (int u = blockIdx.x; u < n_units && ok; u += gridDim.x) {
      const Unit x = decode_unit(p, us, u);
      for (int j = 0; j < x.n; ++j, ++nt) {
        const uint32_t st = nt % L::kStages, round = nt / L::kStages;
        if (round > 0) ok = __all_sync(0xffffffffu, wait_bar(bar(Q_EMPTY + st), (round - 1) & 1u, abort_flag, status, tmo));
        if (!ok) break;
        withheld = p.fault_inject == 1 && nt == 0;   // (tests)
        if (!withheld && elect_one()) {
          mbar_arrive_expect_tx(bar(Q_FULL + st), bytes);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(sbase + L::kOffQ + st * L::kQueryTile + c * (kWeighCols * 128), &p.tm_q, bar(Q_FULL + st), c * 64,
                        x.h * p.group, x.q0 + x.i0 + j * tq);
        }
        __syncwarp();
      }
    }
    // After an abort: the copies in flight land before the block ends (the last use of every stage).
    if (*abort_flag && elect_one()) {
      const uint32_t last = nt < L::kStages ? 0 : nt - L::kStages;
      for (uint32_t i = last; i < nt; ++i)
        if (!(p.fault_inject == 1 && i == 0)) drain_wait(bar(Q_FULL + i % L::kStages), (i / L::kStages) & 1u, tmo);
    }
    __syncwarp();
  } else if (warp == 13) {
    // ======================= biases, and the last key that a row sees =======================
    uint32_t nt = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < n_units && ok; u += gridDim.x) {
      const Unit x = decode_unit(p, us, u);
      for (int j = 0; j < x.n; ++j, ++nt) {
        const uint32_t slot = nt % kBiasRing, round = nt / kBiasRing;
        const int i0 = x.i0 + j * tq, tokens = min(tq, x.T - i0);
        float b[kWeighCols / 32];
        int s[kWeighCols / 32];
#pragma unroll
        for (int i = 0; i < kWeighCols / 32; ++i) {
          int g;
          const int t = token_of(p, i * 32 + lane, &g);
          const bool there = t < tokens;
          b[i] = there ? __ldg(p.lse + (int64_t)(x.q0 + i0 + t) * p.n_heads + x.h * p.group + g) : -INFINITY;
          s[i] = there ? x.P0 + i0 + t : -1;
        }
        if (round > 0) ok = __all_sync(0xffffffffu, wait_bar(bar(B_EMPTY + slot), (round - 1) & 1u, abort_flag, status, tmo));
        if (!ok) break;
        float* const bias = reinterpret_cast<float*>(smem + L::kOffBias) + slot * kWeighCols;
        int* const seen = reinterpret_cast<int*>(smem + L::kOffBias) + (kBiasRing + slot) * kWeighCols;
#pragma unroll
        for (int i = 0; i < kWeighCols / 32; ++i) {
          bias[i * 32 + lane] = bias_of(b[i]);
          seen[i * 32 + lane] = s[i];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_FULL + slot));
      }
    }
  } else if (warp == kMmaWarp) {
    // ======================= products =======================
    if (elect_one()) {
      constexpr uint32_t idesc = idesc_bf16(128, kHalf);
      uint32_t nt = 0, nk = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < n_units && ok; u += gridDim.x) {
        const Unit x = decode_unit(p, us, u);
        for (int j = 0; j < x.n && ok; ++j, ++nt) {
          const uint32_t st = nt % L::kStages;
          ok = wait_bar(bar(Q_FULL + st), (nt / L::kStages) & 1u, abort_flag, status, tmo);
          const uint64_t q0 = sw128_kmajor_desc(sbase + L::kOffQ + st * L::kQueryTile, 0);
#pragma unroll 1
          for (int i = 0; i < 4 && ok; ++i) {   // the streams in turn: half i / 2 of stream i % 2
            const int w = i & 1, half = i >> 1;
            if (j == 0 && half == 0) ok = wait_bar(bar(K_FULL + w), nk & 1u, abort_flag, status, tmo);
            if (ok && nt > 0) ok = wait_bar(bar(S_EMPTY + 2 * w + half), (nt - 1) & 1u, abort_flag, status, tmo);
            if (!ok) break;
            tc_fence_after();
            uint64_t kd = sw128_kmajor_desc(sbase + w * L::kKeyTile, 0), qd = q0 + half * ((kHalf * 128) >> 4);
#pragma unroll
            for (int c = 0; c < D / 64; ++c, kd += (128 * 128) >> 4, qd += (kWeighCols * 128) >> 4) {
#pragma unroll
              for (int k = 0; k < 4; ++k)   // 32 bytes a step
                mma_bf16(tmem + w * kWeighCols + half * kHalf, kd + 2 * k, qd + 2 * k, idesc, c + k > 0);
            }
            tc_commit(bar(S_FULL + 2 * w + half));
            if (j + 1 == x.n && half == 1) tc_commit(bar(K_EMPTY + w));
          }
          if (ok) tc_commit(bar(Q_EMPTY + st));
        }
        if (x.n > 0) ++nk;
      }
      if (!ok) {   // what was issued completes before the tensor memory is given back
        tc_commit(bar(DRAIN));
        drain_wait(bar(DRAIN), 0, tmo);
      }
    }
    __syncwarp();
  }
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
  if (tid == 0) put_status(p, p.step_blocks + blockIdx.x, *status);
}

// Adds the parts of divided units, in their order: a block to a unit's keys.
__global__ void __launch_bounds__(kWeighKeys) weigh_join_kernel(const __grid_constant__ WeighParams p) {
  __shared__ int tab[kGroups + 1];
  __shared__ float scratch[2 * kGroups];
  Units us;
  us.tab = tab;
  us.gsz = (p.num_seqs + kGroups - 1) / kGroups;
  us.chunk = count_units(p, us.gsz, tab, scratch);
  if (us.chunk == 0x7FFFFFFF) return;   // none is divided
  const int n_units = tab[kGroups];
  for (int u = blockIdx.x; u < n_units; u += gridDim.x) {
    const Unit x = decode_unit(p, us, u);
    const int key = x.key0 + threadIdx.x;
    if (x.parts == 1 || x.part > 0 || key >= x.S) continue;
    const int64_t r = cache_row(p.c, x.d, key, x.h);
    if (r < 0) continue;
    float total = 0.f;
    for (int i = 0; i < x.parts; ++i) total += p.part[(int64_t)(u + i) * kWeighKeys + threadIdx.x];
    p.weights[r] = key >= x.P0 ? total : p.weights[r] + total;
  }
}

template <int D, bool Q8>
cudaError_t launch_tiles(const WeighParams& p, int sm_count, cudaStream_t stream) {
  auto kernel = weigh_tiles_kernel<D, Q8>;
  int dev = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  static std::atomic<uint64_t> ready{0};   // devices on which this kernel is set up
  if (!(ready.load(std::memory_order_acquire) >> (dev & 63) & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<D>::kSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(1ull << (dev & 63), std::memory_order_release);
  }
  kernel<<<p.tile_blocks, kTileThreads, Layout<D>::kSmem, stream>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  weigh_join_kernel<<<2 * sm_count, kWeighKeys, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace weigh

cudaError_t launch_weigh_tiles(const WeighParams& p, int D, int sm_count, cudaStream_t stream) {
  const bool q8 = p.c.fmt != 0;
  if (D == 128) return q8 ? weigh::launch_tiles<128, true>(p, sm_count, stream) : weigh::launch_tiles<128, false>(p, sm_count, stream);
  return q8 ? weigh::launch_tiles<64, true>(p, sm_count, stream) : weigh::launch_tiles<64, false>(p, sm_count, stream);
}

}  // namespace dsa
