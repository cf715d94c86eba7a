// Gathered attention weight of long chunks, on the tensor cores: the keys are the
// products' rows, the queries their columns, S^T = K Q^T, so that a thread has
// a key and adds up its weights exp(scale s - lse) over the queries in registers.
//
// A unit is 256 keys of one head of one sequence and the tokens that see them; its
// keys stay in shared memory as two tiles of 128 while tiles of 256 query rows
// (tokens x heads of the group) pass.  A product is 128 keys x 128 query rows:
// four have room in tensor memory, one to each of four warpgroups that turn them
// into weights, and a warp to either tile of keys issues them.  A product takes
// 512 cycles of an SM, its exponentials as long, and its way through a warpgroup
// several times that, so it is the number under way that counts.  4096 tokens over
// 32768 BF16 keys, 64 heads, 8 key heads: 1.45 ms, with products of 256 rows (two
// under way) 1.56, with the keys in tensor memory and products of 96 rows 1.52, with
// one warp for all products 1.76; the products alone take 1.15 ms at this pace, 1.3
// with all but the exponentials.  (Keys of one tile alone would have each query row
// read from the L2 twice as often.)
//
// Queries come by TMA (a box of tokens x heads is the tile as the MMA reads it),
// keys row by row through the page table, 8-bit ones widened on the way: that takes a
// warp some 1500 cycles for 32 rows, so eight warps do it, and the warps that weigh keep
// their 80 registers (ragged chunks over FP8 rows 143 -> 141 us; 8 tokens of each of 32
// sequences of 2048 - 8192 MXFP8 rows, which change keys all the time, 221 -> 157; four
// warps of BF16 rows have but copies to issue, 96 us for the latter).  At the 72
// registers of its launch the form for 8-bit keys spills 96 - 132 bytes.  The
// query tiles of all units in a row are shared out evenly: a block takes a
// consecutive part, so that it changes keys seldom and all end together.  Where a
// part's end divides a unit, a second kernel adds the pieces in their order.
#include <cuda_bf16.h>

#include <atomic>

#include "e4m3_widen.cuh"
#include "tile_pipeline.cuh"
#include "weigh.cuh"

namespace dsa {

namespace weigh {

using namespace attn;

constexpr int kGroups = 64;            // sequences are counted in this many groups
constexpr int kHalf = kWeighCols / 2;  // columns of a product and of a hand-over
constexpr int kBiasRing = 4;
// What a unit's change of keys counts beside its query tiles.  1 / 3 / 6 / 12: ragged chunks of 1 - 1500 tokens of six
// sequences over BF16 131 / 131 / 138 / 145 us, FP8 156 / 140 / 145 / 152, MXFP8 156 / 139 / 145 / 152; heads of 64
// elements 123 / 129 / 136 / 143, 8-bit 127 / 131 / 140 / 146; 16 tokens of each of 32 sequences the same within 1 %.
constexpr int kUnitCost = 3;
constexpr int kMinPart = 2 * kUnitCost;   // length of a block's part, at least
// barriers (halves: 2 * stream + half)
enum { K_FULL = 0, K_EMPTY = 2, S_FULL = 4, S_EMPTY = 8, B_FULL = 12, B_EMPTY = B_FULL + kBiasRing, DRAIN = B_EMPTY + kBiasRing,
       Q_FULL = DRAIN + 2, kMaxStages = 4, Q_EMPTY = Q_FULL + kMaxStages, kBars = Q_EMPTY + kMaxStages };

// The units in a row: sequence by sequence, head by head, keys ascending; each as long as its query
// tiles and kUnitCost before them.  The same in every block.
struct Row {
  long long tab[kGroups + 1];   // where each group of sequences begins
  long long each;               // a part's length: the first `more` are longer by one
  int parts, more;
  // a block's part begins in this unit, `off` behind its begin
  int d, h, kt, off;
};

template <int D>
struct Layout {
  static constexpr uint32_t kKeyTile = 128 * D * 2;              // one stream's keys
  static constexpr uint32_t kQueryTile = kWeighCols * D * 2;
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr uint32_t kOffQ = 2 * kKeyTile;
  static constexpr uint32_t kOffBias = kOffQ + kStages * kQueryTile;   // [kBiasRing][256] bias, then [kBiasRing][256] last key seen
  static constexpr uint32_t kOffSums = kOffBias + 2 * kBiasRing * kWeighCols * 4;   // [2][2][128] of the second halves
  static constexpr uint32_t kOffBars = kOffSums + 2 * 2 * 128 * 4;
  static constexpr uint32_t kOffCtl = kOffBars + kBars * 8;      // status, abort, tmem
  static constexpr uint32_t kOffRow = kOffCtl + 16;
  static constexpr uint32_t kSmem = kOffRow + sizeof(Row);
  static_assert(kOffRow % 8 == 0 && kSmem <= kAttnSmemMax, "shared memory");
};

__device__ __forceinline__ int tiles_of(int tokens, int tq) { return (tokens + tq - 1) / tq; }

// One sequence's units.
struct DocUnits {
  Doc o;
  int kt;   // units of a head; 0 where the sequence is not this kernel's
  int tq, P0;
  __device__ __forceinline__ DocUnits(const WeighParams& p, int d) {
    doc_info(p, d, &o);
    kt = by_steps(p, o.T) ? 0 : (o.S + kWeighKeys - 1) / kWeighKeys;
    tq = kWeighCols / p.group;
    P0 = o.S - o.T;
  }
  __device__ __forceinline__ int first(int k) const { return max(0, k * kWeighKeys - P0); }   // token that sees unit k
  __device__ __forceinline__ int length(int k) const { return tiles_of(o.T - first(k), tq) + kUnitCost; }
  __device__ __forceinline__ int whole() const { return min(kt, P0 / kWeighKeys + 1); }       // units that every token sees
  __device__ __forceinline__ long long of_head() const {
    if (kt == 0) return 0;
    long long n = (long long)whole() * length(0);
    for (int k = whole(); k < kt; ++k) n += length(k);
    return n;
  }
};

// Where part i begins.
__device__ __forceinline__ long long part_begin(const Row& r, int i) { return i * r.each + min(i, r.more); }

// Lays the units out in a row and divides it among the call's blocks; the whole block calls.
__device__ __forceinline__ void lay_out(const WeighParams& p, Row* row) {
  const int tid = threadIdx.x, gsz = (p.num_seqs + kGroups - 1) / kGroups;
  bool falls = false;   // prefixes that fall: nothing is computed
  long long mine = 0;
  if (tid < kGroups) {
    for (int i = 0; i < gsz && tid * gsz + i < p.num_seqs; ++i) {
      const int d = tid * gsz + i;
      mine += DocUnits(p, d).of_head() * p.c.n_kv;
      falls |= __ldg(p.cu_k + d) < 0 || __ldg(p.cu_k + d + 1) < __ldg(p.cu_k + d) || __ldg(p.cu_q + d) < 0 ||
               __ldg(p.cu_q + d + 1) < __ldg(p.cu_q + d);
    }
  }
  const bool none = __syncthreads_or(falls);
  if (none) mine = 0;
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if ((tid & 31) >= o) incl += y;
  }
  if (tid == 31) row->tab[kGroups] = incl;
  __syncthreads();
  const long long before = incl - mine + (tid >= 32 ? row->tab[kGroups] : 0);
  __syncthreads();
  if (tid < kGroups) row->tab[tid] = before;
  if (tid == kGroups - 1) {
    const long long end = before + mine, most = (end + kMinPart - 1) / kMinPart;
    row->tab[kGroups] = end;
    row->parts = most < p.tile_blocks ? max((int)most, 1) : p.tile_blocks;
    row->each = end / row->parts;
    row->more = (int)(end - row->each * row->parts);
  }
  __syncthreads();
}

// The unit that position `at` of the row is in.
__device__ __forceinline__ void locate(const WeighParams& p, Row* row, long long at) {
  const int gsz = (p.num_seqs + kGroups - 1) / kGroups;
  int lo = 0, hi = kGroups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (row->tab[mid] <= at) lo = mid; else hi = mid - 1;
  }
  long long rem = at - row->tab[lo];
  for (int d = lo * gsz; d < p.num_seqs; ++d) {
    const DocUnits x(p, d);
    const long long head = x.of_head();
    if (rem >= head * p.c.n_kv) {
      rem -= head * p.c.n_kv;
      continue;
    }
    row->d = d;
    row->h = (int)(rem / head);
    rem -= row->h * head;
    const long long full = (long long)x.whole() * x.length(0);
    int k = rem < full ? (int)(rem / x.length(0)) : x.whole();
    rem -= rem < full ? (long long)k * x.length(0) : full;
    while (rem >= x.length(k)) rem -= x.length(k++);
    row->kt = k;
    row->off = (int)rem;
    return;
  }
}

// A piece of a unit in a block's part.
struct Piece {
  int d, h, key0;
  int q0, T, S, P0;
  int i0, n;        // first token, query tiles
  bool begins, ends;   // with its unit
};

struct Cursor {
  const WeighParams& p;
  DocUnits x;
  int d, h, kt, off;
  long long left;   // of the part
  __device__ __forceinline__ Cursor(const WeighParams& p, const Row& r, long long left)
      : p(p), x(p, r.d), d(r.d), h(r.h), kt(r.kt), off(r.off), left(left) {}
  __device__ __forceinline__ bool next(Piece* s) {
    if (left <= 0) return false;
    while (kt >= x.kt) {
      kt = 0;
      if (x.kt == 0 || ++h == p.c.n_kv) {
        h = 0;
        if (++d >= p.num_seqs) return false;
        x = DocUnits(p, d);
      }
    }
    const int length = x.length(kt), to = left < length - off ? off + (int)left : length;
    const int a = max(off - kUnitCost, 0), b = max(to - kUnitCost, 0);
    s->d = d;
    s->h = h;
    s->key0 = kt * kWeighKeys;
    s->q0 = x.o.q0;
    s->T = x.o.T;
    s->S = x.o.S;
    s->P0 = x.P0;
    s->i0 = x.first(kt) + a * x.tq;
    s->n = b - a;
    s->begins = off == 0;
    s->ends = to == length;
    left -= to - off;
    off = to;
    if (to == length) {
      off = 0;
      ++kt;
    }
    return true;
  }
};

// Warps of a block: sixteen turn products into weights, four (BF16) or eight (8-bit keys, which they widen) bring keys,
// the last four queries, biases and products.
template <bool Q8>
struct Roles {
  static constexpr int kKeyWarps = Q8 ? 8 : 4;
  static constexpr int kThreads = 32 * (16 + kKeyWarps + 4);
  // registers of a thread with 8-bit keys, whose warpgroups share them unevenly: 72 each at launch
  static constexpr int kWeighRegs = 80, kKeyRegs = 64, kRestRegs = 56;
  static_assert(512 * kWeighRegs + 256 * kKeyRegs + 128 * kRestRegs <= 896 * 72, "no more than the block was launched with");
};

template <int D, bool Q8>
__global__ void __launch_bounds__(Roles<Q8>::kThreads, 1) weigh_tiles_kernel(const __grid_constant__ WeighParams p) {
  using L = Layout<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sbase = smem_u32(smem);
  const uint64_t tmo = p.timeout_ns;
  int* const ctl = reinterpret_cast<int*>(smem + L::kOffCtl);
  int* const status = ctl;
  volatile int* const abort_flag = ctl + 1;
  auto bar = [&](int i) { return sbase + L::kOffBars + 8u * i; };
  using R = Roles<Q8>;
  constexpr int kThreads = R::kThreads, kKeyWarp = 16, kQueryWarp = kKeyWarp + R::kKeyWarps, kBiasWarp = kQueryWarp + 1;
  constexpr int kMmaWarp = kQueryWarp + 2;
  if (tid == 0) {
    ctl[0] = (sbase & 1023u) ? DSA_DEV_ERR_BOUNDS : 0;   // the swizzle needs a 1024-byte base
    ctl[1] = (sbase & 1023u) ? 1 : 0;
    for (int w = 0; w < 2; ++w) {
      mbar_init(bar(K_FULL + w), 4);
      mbar_init(bar(K_EMPTY + w), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(S_FULL + i), 1);
      mbar_init(bar(S_EMPTY + i), 4);
    }
    for (int s = 0; s < kBiasRing; ++s) {
      mbar_init(bar(B_FULL + s), 1);
      mbar_init(bar(B_EMPTY + s), 16);
    }
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(bar(Q_FULL + s), 1);
      mbar_init(bar(Q_EMPTY + s), 2);
    }
    for (int w = 0; w < 2; ++w) mbar_init(bar(DRAIN + w), 1);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc(smem_u32(ctl + 2), 512);
  if (kWeighCols % p.group != 0) {   // rows that no box covers read as zeros
    for (uint32_t i = tid * 16; i < L::kStages * L::kQueryTile; i += kThreads * 16)
      *reinterpret_cast<uint4*>(smem + L::kOffQ + i) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  Row* const row = reinterpret_cast<Row*>(smem + L::kOffRow);
  lay_out(p, row);
  const long long begin = (int)blockIdx.x < row->parts ? part_begin(*row, blockIdx.x) : 0;
  const long long end = (int)blockIdx.x < row->parts ? part_begin(*row, blockIdx.x + 1) : 0;
  if (tid == 0) {
    row->d = row->h = row->kt = row->off = 0;
    if (begin < end) locate(p, row, begin);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)ctl[2];
  const int tq = kWeighCols / p.group;
  Cursor cur(p, *row, end - begin);
  Piece x;

  if (warp < 16) {
    // ======================= weights: a key to a thread =======================
    if constexpr (Q8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R::kWeighRegs));
    const int w = (warp >> 2) & 1, half = warp >> 3, quarter = warp & 3, c0 = half * kHalf;
    const uint32_t t_s = tmem + (uint32_t)(w * kWeighCols + c0) + ((uint32_t)quarter << 21);
    const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
    float* const sums = reinterpret_cast<float*>(smem + L::kOffSums) + w * 128 + quarter * 32 + lane;
    uint32_t nt = 0, nx = 0;
    bool ok = true;
    for (; ok && cur.next(&x); ++nx) {
      const int wkey = x.key0 + w * 128 + quarter * 32, key = wkey + lane;   // the warp's first key, this thread's
      float total = 0.f;   // sums of products are added to it: a sum over all columns one by one would lose bits
      for (int j = 0; j < x.n; ++j, ++nt) {
        const int slot = nt % kBiasRing;
        const int i0 = x.i0 + j * tq, tokens = min(tq, x.T - i0), cols = tokens * p.group - c0;   // this half's live columns
        const float* const bias = reinterpret_cast<const float*>(smem + L::kOffBias) + slot * kWeighCols + c0;
        const int* const seen = reinterpret_cast<const int*>(smem + L::kOffBias) + (kBiasRing + slot) * kWeighCols + c0;
        // (else no token of the tile sees a key of the warp)
        const bool any = wkey <= x.P0 + i0 + tokens - 1 && wkey < x.S && cols > 0;
        // some key that some token does not see, or columns of other sequences' tokens
        const bool edge = wkey + 31 > x.P0 + i0 || tokens < tq;
        ok = __all_sync(0xffffffffu, wait_bar(bar(B_FULL + slot), (nt / kBiasRing) & 1u, abort_flag, status, tmo) &&
                                         wait_bar(bar(S_FULL + 2 * w + half), nt & 1u, abort_flag, status, tmo));
        if (!ok) break;
        tc_fence_after();
        float2 sum[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = make_float2(0.f, 0.f);
        auto release = [&] {   // the half's columns have been read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(S_EMPTY + 2 * w + half));
        };
        // 32 columns, all of whose tokens see all the warp's keys
        auto weigh32 = [&](const uint32_t (&v)[32], int c) {
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float4 b = *reinterpret_cast<const float4*>(bias + c + 2 * i);
            float2 e0 = ffma2(as_f2(v[2 * i], v[2 * i + 1]), sc2, make_float2(b.x, b.y));
            float2 e1 = ffma2(as_f2(v[2 * i + 2], v[2 * i + 3]), sc2, make_float2(b.z, b.w));
            e0.x = ex2(e0.x);
            e0.y = ex2(e0.y);
            e1.x = ex2(e1.x);
            e1.y = ex2(e1.y);
            sum[i & 2] = __fadd2_rn(sum[i & 2], e0);
            sum[(i & 2) + 1] = __fadd2_rn(sum[(i & 2) + 1], e1);
          }
        };
        if (any && !edge) {
#pragma unroll
          for (int c = 0; c < kHalf; c += 32) {
            uint32_t s[32];
            tmem_ld_x32(t_s + c, s);
            tmem_ld_wait_tied<32>(s);
            if (c + 32 == kHalf) release();
            weigh32(s, c);
          }
        } else if (any) {
#pragma unroll 1
          for (int c = 0; c < min(cols, kHalf); c += 32) {
            int g;
            if (wkey > x.P0 + i0 + token_of(p, c0 + c + 31, &g)) continue;   // none of these tokens sees a key of the warp
            uint32_t s[32];
            tmem_ld_x32(t_s + c, s);
            tmem_ld_wait_tied<32>(s);
            if (c + 32 <= cols && wkey + 31 <= x.P0 + i0 + token_of(p, c0 + c, &g)) {
              weigh32(s, c);
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float e = ex2(fmaf(__uint_as_float(s[i]), p.scale_log2, bias[c + i]));
                sum[(i >> 1) & 3].x += key <= seen[c + i] ? e : 0.f;
              }
            }
          }
          release();
        } else {
          release();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_EMPTY + slot));
        total += ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y)) + ((sum[2].x + sum[2].y) + (sum[3].x + sum[3].y));
      }
      // The halves' sums meet (in two places in turn).  Whatever a warp has waited for in vain, it comes
      // here: both warpgroups leave together.
      if (half == 1) sums[(nx & 1) * 256] = total;
      ok = !named_bar_or(1 + w, 256, !ok);
      if (!ok) break;
      if (half == 1) continue;
      total += sums[(nx & 1) * 256];
      if (!x.begins || !x.ends) {
        p.part[((int64_t)blockIdx.x * 2 + (x.begins ? 1 : 0)) * kWeighKeys + w * 128 + quarter * 32 + lane] = total;
      } else if (key < x.S) {
        const int64_t r = cache_row(p.c, x.d, key, x.h);   // (-1 is reported by the loaders)
        if (r >= 0) p.weights[r] = key >= x.P0 ? total : p.weights[r] + total;
      }
    }
  } else if (warp < kQueryWarp) {
    // ======================= keys =======================
    if constexpr (Q8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::kKeyRegs));
    // a quarter of a tile: of both in turn, or (8-bit keys) of one
    constexpr int kTiles = Q8 ? 1 : 2;
    const int kw = (warp - kKeyWarp) & 3, w0 = (warp - kKeyWarp) >> 2;
    uint32_t nk = 0;
    bool ok = true, bad_page = false;
    while (ok && cur.next(&x)) {
      if (x.n == 0) continue;
      uint32_t rows[kTiles];   // this lane's
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        const int key = x.key0 + (w0 + i) * 128 + kw * 32 + lane;
        const int64_t mine = key < x.S ? cache_row(p.c, x.d, key, x.h) : -1;
        if (key < x.S && mine < 0) bad_page = true;
        rows[i] = mine < 0 ? ~0u : (uint32_t)mine;
        if (!Q8 && rows[i] != ~0u) {   // on its way to the L2 while the last unit's keys are still in use
#pragma unroll
          for (int o = 0; o < D * 2; o += 128)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const uint8_t*>(p.c.k) + (size_t)rows[i] * (D * 2) + o));
        }
      }
#pragma unroll 1
      for (int i = 0; i < kTiles && ok; ++i) {
        const int w = w0 + i;
        const uint32_t row32 = kTiles == 2 && i ? rows[kTiles - 1] : rows[0], dst = sbase + w * L::kKeyTile + kw * 32 * 128;
        auto wait_empty = [&] {
          if (nk > 0) ok = __all_sync(0xffffffffu, wait_bar(bar(K_EMPTY + w), (nk - 1) & 1u, abort_flag, status, tmo));
        };
        if constexpr (Q8) {
          // the rows are on their way while the last unit's keys are still in use
          constexpr int PPR = D / 16, RPP = 32 / PPR, kPasses = 32 / RPP;
          const int c = lane % PPR, rsub = lane / PPR;
          const uint8_t* const src = reinterpret_cast<const uint8_t*>(p.c.k) + c * 16;
          uint32_t scales = 0;   // of this lane's row, a byte to each block
          if (row32 != ~0u) {
            if (p.c.sw == 1) scales = __ldg(p.c.k_scale + row32) * 0x01010101u;
            else if constexpr (D == 128) scales = __ldg(reinterpret_cast<const uint32_t*>(p.c.k_scale) + row32);
            else scales = __ldg(reinterpret_cast<const uint16_t*>(p.c.k_scale) + row32);
          }
          uint4 v[kPasses];
#pragma unroll
          for (int j = 0; j < kPasses; ++j) {
            const uint32_t r = __shfl_sync(0xffffffffu, row32, j * RPP + rsub);
            v[j] = r == ~0u ? make_uint4(0, 0, 0, 0) : __ldg(reinterpret_cast<const uint4*>(src + (size_t)r * D));
          }
          wait_empty();
          if (!ok) break;
#pragma unroll
          for (int j = 0; j < kPasses; ++j) {
            const int r = j * RPP + rsub;
            const uint32_t w4[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
            uint32_t o[8];
            const uint32_t e8 = (__shfl_sync(0xffffffffu, scales, r) >> (8 * (c >> 1))) & 255u;
            if (e8 <= 134u) widen<false>(w4, e8, o);
            else widen<true>(w4, e8, o);
            const uint32_t at = dst + (uint32_t)(c >> 2) * (128 * 128) + r * 128;
            st_shared_v4(at + ((((c & 3) * 2) ^ (r & 7)) << 4), o[0], o[1], o[2], o[3]);
            st_shared_v4(at + ((((c & 3) * 2 + 1) ^ (r & 7)) << 4), o[4], o[5], o[6], o[7]);
          }
        } else {
          constexpr int PPR = D / 8, RPP = 32 / PPR;
          const int c = lane % PPR, rsub = lane / PPR;
          const uint16_t* const src = reinterpret_cast<const uint16_t*>(p.c.k) + c * 8;
          wait_empty();
          if (!ok) break;
#pragma unroll
          for (int j = 0; j < 32; j += RPP) {
            const uint32_t e = __shfl_sync(0xffffffffu, row32, j + rsub);
            const int r = j + rsub;
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
  } else {
    if constexpr (Q8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::kRestRegs));
    if (warp == kQueryWarp) {
      // ======================= queries =======================
      const uint32_t bytes = (uint32_t)tq * p.group * D * 2;
      uint32_t nt = 0;
      bool ok = true;
      while (ok && cur.next(&x)) {
        for (int j = 0; j < x.n; ++j, ++nt) {
          const uint32_t st = nt % L::kStages, round = nt / L::kStages;
          if (round > 0) ok = __all_sync(0xffffffffu, wait_bar(bar(Q_EMPTY + st), (round - 1) & 1u, abort_flag, status, tmo));
          if (!ok) break;
          const bool withheld = p.fault_inject == 1 && nt == 0;   // (tests)
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
    } else if (warp == kBiasWarp) {
      // ======================= biases, and the last key that a row sees =======================
      uint32_t nt = 0;
      bool ok = true;
      while (ok && cur.next(&x)) {
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
    } else {
      // ======================= products: a warp to a tile of keys =======================
      const int w = warp - kMmaWarp;
      if (elect_one()) {
        constexpr uint32_t idesc = idesc_bf16(128, kHalf);
        const uint64_t k0 = sw128_kmajor_desc(sbase + w * L::kKeyTile, 0);
        uint32_t nt = 0, nk = 0;
        bool ok = true;
        while (ok && cur.next(&x)) {
          for (int j = 0; j < x.n && ok; ++j, ++nt) {
            const uint32_t st = nt % L::kStages;
            ok = wait_bar(bar(Q_FULL + st), (nt / L::kStages) & 1u, abort_flag, status, tmo);
            if (ok && j == 0) ok = wait_bar(bar(K_FULL + w), nk & 1u, abort_flag, status, tmo);
            const uint64_t q0 = sw128_kmajor_desc(sbase + L::kOffQ + st * L::kQueryTile, 0);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              if (ok && nt > 0) ok = wait_bar(bar(S_EMPTY + 2 * w + half), (nt - 1) & 1u, abort_flag, status, tmo);
              if (!ok) break;
              tc_fence_after();
              uint64_t kd = k0, qd = q0 + half * ((kHalf * 128) >> 4);
#pragma unroll
              for (int c = 0; c < D / 64; ++c, kd += (128 * 128) >> 4, qd += (kWeighCols * 128) >> 4) {
#pragma unroll
                for (int k = 0; k < 4; ++k)   // 32 bytes a step
                  mma_bf16(tmem + w * kWeighCols + half * kHalf, kd + 2 * k, qd + 2 * k, idesc, c + k > 0);
              }
              tc_commit(bar(S_FULL + 2 * w + half));
            }
            if (ok) tc_commit(bar(Q_EMPTY + st));
            if (ok && j + 1 == x.n) tc_commit(bar(K_EMPTY + w));
          }
          if (x.n > 0) ++nk;
        }
        if (!ok) {   // what was issued completes before the tensor memory is given back
          tc_commit(bar(DRAIN + w));
          drain_wait(bar(DRAIN + w), 0, tmo);
        }
      }
      __syncwarp();
    }
  }
  // The steps' kernel, whose rows are those of other sequences, is over when this one is; the next may begin.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
  if (tid == 0) put_status(p, p.step_blocks + blockIdx.x, *status);
}

// Adds the pieces of units that parts' ends divide, in their order: a block to each end but the last.
__global__ void __launch_bounds__(kWeighKeys) weigh_join_kernel(const __grid_constant__ WeighParams p) {
  __shared__ Row row;
  lay_out(p, &row);
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the tiles' kernel is over
  const int b = blockIdx.x + 1;
  if (b >= row.parts) return;
  const long long at = part_begin(row, b), before = part_begin(row, b - 1);
  if (threadIdx.x == 0) locate(p, &row, at);
  __syncthreads();
  const long long begin = at - row.off;
  if (row.off == 0 || before > begin) return;   // not divided, or by an end before it too
  const DocUnits x(p, row.d);
  const long long end = begin + x.length(row.kt);
  const int key = row.kt * kWeighKeys + threadIdx.x;
  if (key >= x.o.S) return;
  const int64_t r = cache_row(p.c, row.d, key, row.h);
  if (r < 0) return;
  float total = p.part[((int64_t)(b - 1) * 2 + 1) * kWeighKeys + threadIdx.x];
  for (int i = b; i < row.parts && part_begin(row, i) < end; ++i) total += p.part[((int64_t)i * 2) * kWeighKeys + threadIdx.x];
  p.weights[r] = key >= x.P0 ? total : p.weights[r] + total;
}

template <int D, bool Q8>
cudaError_t launch_tiles(const WeighParams& p, cudaStream_t stream) {
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
  // each may begin while the kernel before it is ending
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(p.tile_blocks);
  cfg.blockDim = dim3(Roles<Q8>::kThreads);
  cfg.dynamicSmemBytes = Layout<D>::kSmem;
  if ((e = cudaLaunchKernelEx(&cfg, kernel, p)) != cudaSuccess || p.tile_blocks == 1) return e;
  cfg.gridDim = dim3(p.tile_blocks - 1);
  cfg.blockDim = dim3(kWeighKeys);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, weigh_join_kernel, p);
}

}  // namespace weigh

cudaError_t launch_weigh_tiles(const WeighParams& p, int D, cudaStream_t stream) {
  const bool q8 = p.c.fmt != 0;
  if (D == 128) return q8 ? weigh::launch_tiles<128, true>(p, stream) : weigh::launch_tiles<128, false>(p, stream);
  return q8 ? weigh::launch_tiles<64, true>(p, stream) : weigh::launch_tiles<64, false>(p, stream);
}

}  // namespace dsa
