// Bounding a paged cache: the choice of the rows that stay, and their moving
// together in place.
//
// evict_select: of the S rows of a sequence the `budget` that come first by
// (sinks and recent rows, weight descending, position ascending), written in
// ascending order.  A cluster of 1 to 8 blocks takes one head of one sequence
// (or the sum of its heads), each block a range of the rows, and finds the
// weight of the last row that stays by digits of its order-preserving bits: 12,
// 12 and 8 of them, counted in shared memory and added up over the cluster.
// With the last value known, the number of rows above it and how many of the
// equal ones stay, each block writes its rows behind those of the blocks before.
//
// cache_compact: row j takes the place of row kept[j], kept ascending, so that
// kept[j] >= j: a block moves a part of each row of one head in ascending
// chunks.  A chunk's rows are read whole before any of them is written, and
// the rows that later chunks read lie behind everything written before them, so
// reads run several chunks ahead.
#include <cooperative_groups.h>

#include <atomic>

#include "dsa_device.cuh"
#include "evict_params.h"

namespace dsa {

namespace {

namespace cg = cooperative_groups;

// ---------------------------------------------------------------- choice

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 4096;
constexpr int kLastBins = 256;
constexpr uint32_t kMust = 0xFFFFFFFFu;   // above every weight's bits
constexpr int kSelCluster = 8;            // blocks of a cluster, at most
constexpr int kSelRows = 40 * 1024;       // rows of a block whose bits fit into its shared memory
constexpr int kSelFixed = 2 * kBins + kLastBins;   // words of the counts
constexpr int kSelFew = kSelThreads;

// Order-preserving bits of a weight; NaN below everything, -0 as +0.
__device__ __forceinline__ uint32_t weight_bits(float w) { return w != w ? 0u : orderable_key(w); }

struct Select {
  const SelectParams& p;
  int d, h, S;
  bool bad = false;
  __device__ __forceinline__ uint32_t at(int i) {   // of row i
    if (i < p.sinks || i >= S - p.recent) return kMust;
    const int page = __ldg(p.table + (int64_t)d * p.max_pages + (i >> p.page_shift));
    if ((unsigned)page >= (unsigned)p.num_pages) {
      bad = true;
      return 0u;
    }
    const int slot = i & ((1 << p.page_shift) - 1);
    const float* w = p.weights + (((int64_t)page * p.n_kv + h) << p.page_shift) + slot;
    float v = __ldg(w);
    if (p.shared) {   // the heads' sum, one after the other
#pragma unroll 8
      for (int k = 1; k < p.n_kv; ++k) v += __ldg(w + ((int64_t)k << p.page_shift));
    }
    return weight_bits(v);
  }
};

// Finds the bin of the `want`-th largest entry of the cluster's counts hist[n] and takes off `want` what
// lies above it; *count: entries of the bin.  The whole cluster calls, after its counts are complete;
// every thread gets the result.
__device__ __forceinline__ int find_bin(cg::cluster_group& cluster, uint32_t* hist, int n, int* want, int* count,
                                        int (*scratch)[kSelWarps + 3]) {
  const int tid = threadIdx.x, lane = tid & 31;
  int c[4] = {0, 0, 0, 0};   // of four bins, from the top down over the threads
  const int top = n - 4 * tid;
  const unsigned blocks = cluster.num_blocks();
  if (top > 0) {
    for (unsigned r = 0; r < blocks; ++r) {
      const uint4 v = *reinterpret_cast<const uint4*>((blocks > 1 ? cluster.map_shared_rank(hist, r) : hist) + top - 4);
      c[0] += v.w;
      c[1] += v.z;
      c[2] += v.y;
      c[3] += v.x;
    }
  }
  const int mine = (c[0] + c[1]) + (c[2] + c[3]);
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) (*scratch)[tid >> 5] = incl;
  __syncthreads();
  int before = (*scratch)[lane];
  before = __reduce_add_sync(0xffffffffu, lane < (tid >> 5) ? before : 0);
  int above = before + incl - mine;
  const int w = *want;
  if (above < w && above + mine >= w) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (above < w && above + c[j] >= w) {
        (*scratch)[kSelWarps] = top - 1 - j;
        (*scratch)[kSelWarps + 1] = w - above;
        (*scratch)[kSelWarps + 2] = c[j];
      }
      above += c[j];
    }
  }
  __syncthreads();
  *want = (*scratch)[kSelWarps + 1];
  *count = (*scratch)[kSelWarps + 2];
  return (*scratch)[kSelWarps];
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const __grid_constant__ SelectParams p) {
  extern __shared__ __align__(16) uint32_t sm[];
  uint32_t* const hist[3] = {sm, sm + kBins, sm + 2 * kBins};
  uint32_t* const bits = sm + kSelFixed;     // [p.cached]
  __shared__ int scratch[3][kSelWarps + 3];
  __shared__ int counts[2][kSelWarps];
  __shared__ int total[2];
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int heads = p.shared ? 1 : p.n_kv, blocks = cluster.num_blocks(), rank = cluster.block_rank();
  int code = 0;
  auto sync = [&] {
    if (blocks > 1) cluster.sync(); else __syncthreads();
  };
  for (int u = blockIdx.x / blocks; u < p.num_seqs * heads; u += gridDim.x / blocks) {
    const int d = u / heads, h = u - d * heads;
    int32_t* const out = p.kept + (int64_t)u * p.budget;
    const int k0 = __ldg(p.cu_k + d), k1 = __ldg(p.cu_k + d + 1);
    int S = k1 - k0;
    if (k0 < 0 || k1 < k0 || S > p.max_seqlen_k || (int64_t)S > ((int64_t)p.max_pages << p.page_shift)) {
      code = DSA_DEV_ERR_INVALID_ARG;
      S = 0;
    }
    if (h == 0 && tid == 0 && rank == 0) p.kept_len[d] = min(S, p.budget);
    if (S <= p.budget) {
      for (int i = rank * kSelThreads + tid; i < p.budget; i += blocks * kSelThreads) out[i] = i < S ? i : -1;
      continue;
    }
    const int per = ((S + blocks - 1) / blocks + 31) & ~31;   // this block's rows: a whole number of warps' steps
    const int lo = min(S, rank * per), n = min(S, lo + per) - lo;
    const bool cached = per <= p.cached;
    Select sel{p, d, h, S};
    auto value = [&](int i) { return cached ? bits[i] : sel.at(lo + i); };
    for (int i = tid; i < kSelFixed; i += kSelThreads) sm[i] = 0;
    if (tid == 0) total[0] = 0;
    __syncthreads();
    int want = p.budget;
    uint32_t prefix = 0;
    // 12 bits, then 12 and 8 among the rows that share those before them
#pragma unroll 1
    for (int step = 0; step < 3; ++step) {
      const int shift = step == 0 ? 20 : (step == 1 ? 8 : 0), bins = step == 2 ? kLastBins : kBins;
      uint32_t* const count = hist[step];
      constexpr int U = 8;   // rows of a thread whose loads go together
      for (int i0 = 0; i0 < n; i0 += U * kSelThreads) {
        uint32_t b[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const int i = i0 + k * kSelThreads + tid;
          b[k] = 0;
          if (i < n) {
            b[k] = step == 0 ? sel.at(lo + i) : value(i);
            if (cached && step == 0) bits[i] = b[k];
          }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const int i = i0 + k * kSelThreads + tid;
          const bool in = i < n && (step == 0 || (b[k] >> (shift + (step == 2 ? 8 : 12))) == prefix);
          const uint32_t digit = (b[k] >> shift) & (bins - 1);
          // many equal rows (none ever looked at): one count for the warp
          const uint32_t live = __ballot_sync(0xffffffffu, in);
          if (live) {
            const uint32_t first = __shfl_sync(0xffffffffu, digit, __ffs(live) - 1);
            const uint32_t same = __ballot_sync(0xffffffffu, in && digit == first);
            if (in && digit == first) {
              if (lane == __ffs(same) - 1) atomicAdd(&count[first], __popc(same));
            } else if (in) {
              atomicAdd(&count[digit], 1u);
            }
          }
        }
      }
      sync();
      int in_bin;
      prefix = (prefix << (step == 2 ? 8 : 12)) | (uint32_t)find_bin(cluster, count, bins, &want, &in_bin, &scratch[step]);
      if (step == 0 && blocks == 1 && in_bin <= kSelFew) {
        // few rows share the last one's first digit: each is ranked among them at once
        unsigned long long* const few = reinterpret_cast<unsigned long long*>(hist[1]);
        for (int i = tid; i < n; i += kSelThreads) {
          const uint32_t b = value(i);
          if ((b >> 20) == prefix) few[atomicAdd(&total[0], 1)] = (unsigned long long)(~b) << 32 | (unsigned)i;
        }
        __syncthreads();
        if (tid < in_bin) {
          const unsigned long long mine = few[tid];
          int rank = 0, above = 0;
          for (int i = 0; i < in_bin; ++i) {
            const unsigned long long other = few[i];
            rank += other < mine;
            above += (uint32_t)(other >> 32) < (uint32_t)(mine >> 32);
          }
          if (rank == want - 1) {   // the last that stays
            counts[0][0] = (int)~(uint32_t)(mine >> 32);
            counts[0][1] = want - above;
          }
        }
        __syncthreads();
        prefix = (uint32_t)counts[0][0];
        want = counts[0][1];
        __syncthreads();
        break;
      }
    }
    // `prefix` is the last value that stays, `want` the number of rows of that value that do
    const int wper = ((n + kSelWarps - 1) / kSelWarps + 31) & ~31;
    const int wlo = min(n, warp * wper), whi = min(n, wlo + wper);
    int n_above = 0, n_equal = 0;
    for (int i0 = wlo; i0 < whi; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t b = i < whi ? value(i) : 0u;
      n_above += __popc(__ballot_sync(0xffffffffu, i < whi && b > prefix));
      n_equal += __popc(__ballot_sync(0xffffffffu, i < whi && b == prefix));
    }
    if (lane == 0) {
      counts[0][warp] = n_above;
      counts[1][warp] = n_equal;
    }
    __syncthreads();
    int above = __reduce_add_sync(0xffffffffu, lane < warp ? counts[0][lane] : 0);   // before this warp's rows
    int equal = __reduce_add_sync(0xffffffffu, lane < warp ? counts[1][lane] : 0);
    if (tid == kSelThreads - 1) {
      total[0] = above + n_above;
      total[1] = equal + n_equal;
    }
    sync();
    for (int r = 0; r < rank; ++r) {
      const int* const t = cluster.map_shared_rank(total, r);
      above += t[0];
      equal += t[1];
    }
    for (int i0 = wlo; i0 < whi; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t b = i < whi ? value(i) : 0u;
      const uint32_t ab = __ballot_sync(0xffffffffu, i < whi && b > prefix), eq = __ballot_sync(0xffffffffu, i < whi && b == prefix);
      const uint32_t before = (1u << lane) - 1u;
      const int e = equal + __popc(eq & before);
      const bool stays = ((ab >> lane) & 1u) || (((eq >> lane) & 1u) && e < want);
      if (stays) out[above + __popc(ab & before) + min(e, want)] = lo + i;
      above += __popc(ab);
      equal += __popc(eq);
    }
    if (sel.bad) code = DSA_DEV_ERR_INVALID_ARG;
    sync();   // (what other blocks read of this one's shared memory has been read)
  }
  code = __syncthreads_or(code != 0) ? DSA_DEV_ERR_INVALID_ARG : 0;
  if (tid == 0) put_block_status(p.hdr, code);
}

// ---------------------------------------------------------------- moving

constexpr int kMoveThreads = 256;
constexpr int kMovePer = 2;              // 16-byte pieces of a thread in a chunk
constexpr int kMoveChunkBytes = kMoveThreads * kMovePer * 16;
constexpr int kMoveStages = 6;

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// One head of one sequence.
struct Move {
  const CompactParams& p;
  int d, h, n;
  const int32_t* kept;
  bool bad = false;
  __device__ __forceinline__ int entry(int j) { return j < n ? __ldg(kept + j) : -1; }
  // Page of position i; -1: not one of the table's.
  __device__ __forceinline__ int page(int i) {
    const int pi = i >> p.c.page_shift;
    return i >= 0 && pi < p.c.max_pages ? __ldg(p.c.table + (int64_t)d * p.c.max_pages + pi) : -1;
  }
  // Cache row of position i on its page, ~0: there is none (reported).
  __device__ __forceinline__ uint32_t row(int i, int page) {
    if ((unsigned)page >= (unsigned)p.c.num_pages) {
      bad = true;
      return ~0u;
    }
    return (uint32_t)((((int64_t)page * p.c.n_kv + h) << p.c.page_shift) + (i & ((1 << p.c.page_shift) - 1)));
  }
  // Row that row j (< n) comes from, its entry being i; ~0: none, or already there.
  __device__ __forceinline__ uint32_t source(int j, int i, int page) {
    if (i < j) {   // not ascending
      bad = true;
      return ~0u;
    }
    const uint32_t r = row(i, page);
    return i == j ? ~0u : r;
  }
};

// A part of each row of keys or values.  Looking up where a row is takes two dependent loads: a chunk's
// entries are requested three steps before its copies, its pages one.
__device__ __forceinline__ void move_rows(Move& m, uint8_t* base, int row_bytes, int bytes, int off, uint8_t* ring, uint32_t sring) {
  const int tid = threadIdx.x, pieces = bytes / 16, rows = kMoveThreads / pieces, sub = tid / pieces;
  off += (tid % pieces) * 16;
  const int chunks = (m.n + rows * kMovePer - 1) / (rows * kMovePer);
  auto j_of = [&](int c, int i) { return (c * kMovePer + i) * rows + sub; };
  int ea[kMovePer], eb[kMovePer], pb[kMovePer], pt[kMovePer];   // entries of chunk f + 1, entries and pages of f; pages written to
#pragma unroll
  for (int i = 0; i < kMovePer; ++i) {
    eb[i] = m.entry(j_of(0, i));
    ea[i] = m.entry(j_of(1, i));
    pt[i] = m.page(j_of(0, i));
  }
#pragma unroll
  for (int i = 0; i < kMovePer; ++i) pb[i] = m.page(eb[i]);
  uint32_t moves = 0;   // a bit for each piece in the ring
  for (int c = 1 - kMoveStages; c < chunks; ++c) {
    const int f = c + kMoveStages - 1, stage = f % kMoveStages;
    if (f < chunks) {
#pragma unroll
      for (int i = 0; i < kMovePer; ++i) {
        const int j = j_of(f, i);
        const uint32_t src = j < m.n ? m.source(j, eb[i], pb[i]) : ~0u;
        if (src != ~0u) {
          cp_async_16(sring + stage * kMoveChunkBytes + (i * kMoveThreads + tid) * 16, base + (size_t)src * row_bytes + off);
          moves |= 1u << (stage * kMovePer + i);
        }
        eb[i] = ea[i];
        pb[i] = m.page(eb[i]);
        ea[i] = m.entry(j_of(f + 2, i));
      }
    }
    cp_commit();
    if (c < 0) continue;
    cp_wait<kMoveStages - 1>();
    __syncthreads();              // the whole chunk has been read
    const int at = c % kMoveStages;
#pragma unroll
    for (int i = 0; i < kMovePer; ++i) {
      const uint32_t bit = 1u << (at * kMovePer + i);
      const int page = pt[i];
      pt[i] = m.page(j_of(c + 1, i));
      if (!(moves & bit)) continue;
      moves ^= bit;
      const uint32_t dst = m.row(j_of(c, i), page);
      if (dst != ~0u)
        *reinterpret_cast<uint4*>(base + (size_t)dst * row_bytes + off) =
            *reinterpret_cast<const uint4*>(ring + at * kMoveChunkBytes + (i * kMoveThreads + tid) * 16);
    }
  }
  cp_wait<0>();
}

// Scales and weights: a chunk of four rows a thread at a time.  Its elements have been read when every
// thread has reached the barrier, and the next chunk reads behind what this one writes.
template <class T>
__device__ __forceinline__ void move_small(Move& m, T* ks, T* vs, float* w) {
  constexpr int U = 4;
  for (int j0 = 0; j0 < m.n; j0 += U * kMoveThreads) {
    int e[U], before[U], page[U];
    uint32_t src[U];
    T k[U], v[U];
    float x[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int j = j0 + i * kMoveThreads + threadIdx.x;
      e[i] = m.entry(j);
      before[i] = j > 0 ? m.entry(j - 1) : -1;
    }
#pragma unroll
    for (int i = 0; i < U; ++i) page[i] = m.page(e[i]);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int j = j0 + i * kMoveThreads + threadIdx.x;
      src[i] = j < m.n ? m.source(j, e[i], page[i]) : ~0u;
      if (j < m.n && e[i] <= before[i]) m.bad = true;
      page[i] = m.page(j < m.n ? j : -1);
      if (src[i] != ~0u) {
        if (ks) k[i] = *reinterpret_cast<volatile T*>(ks + src[i]);
        if (vs) v[i] = *reinterpret_cast<volatile T*>(vs + src[i]);
        if (w) x[i] = *reinterpret_cast<volatile float*>(w + src[i]);
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (src[i] == ~0u) continue;
      const uint32_t dst = m.row(j0 + i * kMoveThreads + threadIdx.x, page[i]);
      if (dst == ~0u) continue;
      if (ks) ks[dst] = k[i];
      if (vs) vs[dst] = v[i];
      if (w) w[dst] = x[i];
    }
  }
}

__global__ void __launch_bounds__(kMoveThreads, 4) cache_compact_kernel(const __grid_constant__ CompactParams p) {
  extern __shared__ __align__(16) uint8_t ring[];
  const int tensors = p.c.v ? 2 : 1, parts = tensors * p.slices + 1;   // of one head of one sequence
  const int64_t units = (int64_t)p.num_seqs * p.c.n_kv * parts;
  const uint32_t sring = smem_u32(ring);
  int code = 0;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int part = (int)(u % parts), dh = (int)(u / parts), d = dh / p.c.n_kv, h = dh - d * p.c.n_kv;
    const int n = __ldg(p.kept_len + d);
    if (n < 0 || n > p.width) {
      code = DSA_DEV_ERR_INVALID_ARG;
      continue;
    }
    Move m{p, d, h, n, p.kept + ((int64_t)d * p.heads + (p.heads > 1 ? h : 0)) * p.width};
    if (part > 0) {
      const int slice = (part - 1) % p.slices, bytes = p.row_bytes / p.slices;
      move_rows(m, reinterpret_cast<uint8_t*>(part <= p.slices ? p.c.k : p.c.v), p.row_bytes, bytes, slice * bytes, ring, sring);
    } else if (p.c.sw == 4) {
      move_small(m, reinterpret_cast<uint32_t*>(p.c.k_scale), reinterpret_cast<uint32_t*>(p.c.v_scale), p.weights);
    } else if (p.c.sw == 2) {
      move_small(m, reinterpret_cast<uint16_t*>(p.c.k_scale), reinterpret_cast<uint16_t*>(p.c.v_scale), p.weights);
    } else {   // (BF16: no scales; the list is looked over here all the same)
      move_small(m, p.c.sw ? p.c.k_scale : nullptr, p.c.sw ? p.c.v_scale : nullptr, p.weights);
    }
    if (m.bad) code = DSA_DEV_ERR_INVALID_ARG;
    __syncthreads();
  }
  code = __syncthreads_or(code != 0) ? DSA_DEV_ERR_INVALID_ARG : 0;
  if (threadIdx.x == 0) put_block_status(p.hdr, code);
}

// Once per device: the kernel's shared memory beyond the default.
template <class K>
cudaError_t allow_smem(std::atomic<uint64_t>& ready, K kernel, int bytes) {
  int dev = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if (ready.load(std::memory_order_acquire) >> (dev & 63) & 1) return cudaSuccess;
  if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) != cudaSuccess) return e;
  ready.fetch_or(1ull << (dev & 63), std::memory_order_release);
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_evict_select(const SelectParams& call, int sm_count, cudaStream_t stream) {
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(ready, evict_select_kernel, (kSelFixed + kSelRows) * 4);
  if (e != cudaSuccess) return e;
  SelectParams p = call;
  const int64_t units = (int64_t)p.num_seqs * (p.shared ? 1 : p.n_kv);
  // more blocks to a head while there are SMs for them and eight rows to a thread, or to hold its rows' bits
  int blocks = 1;
  while (blocks < kSelCluster && ((units * blocks < sm_count && p.max_seqlen_k / blocks > 8 * kSelThreads) ||
                                  p.max_seqlen_k / blocks > kSelRows))
    blocks *= 2;
  const int64_t rows = ((int64_t)(p.max_seqlen_k + blocks - 1) / blocks + 31) & ~31;
  p.cached = (int)(rows < kSelRows ? rows : kSelRows);
  int64_t clusters = DSA_DEV_STATUS_MAX_BLOCKS / blocks;
  if (clusters > units) clusters = units;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = blocks;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(clusters * blocks));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = (size_t)(kSelFixed + p.cached) * 4;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel, p);
}

cudaError_t launch_cache_compact(const CompactParams& call, int sm_count, cudaStream_t stream) {
  constexpr int kSmem = kMoveChunkBytes * kMoveStages;
  // A row in parts of its own blocks while there are fewer than four blocks to an SM, down to 64 bytes.
  CompactParams p = call;
  const int64_t whole = (int64_t)p.num_seqs * p.c.n_kv * (p.c.v ? 2 : 1);
  for (p.slices = 1; p.row_bytes / p.slices > 64 && whole * p.slices < 4 * sm_count;) p.slices *= 2;
  const int64_t units = (int64_t)p.num_seqs * p.c.n_kv * ((p.c.v ? 2 : 1) * p.slices + 1);
  const int64_t grid = units < DSA_DEV_STATUS_MAX_BLOCKS ? units : DSA_DEV_STATUS_MAX_BLOCKS;
  cache_compact_kernel<<<(unsigned)grid, kMoveThreads, kSmem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace dsa
