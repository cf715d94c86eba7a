// Bounding a paged cache: the choice of the rows that stay, and their moving
// together in place.
//
// evict_select: of the S rows of a sequence the `budget` that come first by
// (sinks and recent rows, weight descending, position ascending), written in
// ascending order.  A cluster of 1 to 16 blocks takes one head of one sequence
// (or the sum of its heads), each block a range of the rows, and finds the
// weight of the last row that stays by the first 12 of its order-preserving
// bits, counted in shared memory and added up over the cluster; the rows that
// share them are few as a rule and ranked among one another, else (equal weights)
// the next 12 and the last 8 bits are counted.  With the last value known, the
// number of rows above it and how many of the equal ones stay, each block writes its
// rows behind those of the blocks before.  It is latency that this costs: the rows'
// loads take 2 to 5 us, every barrier of a cluster 1.  2048 rows of some 2200, 16
// sequences of 8 heads, a block each and no such barrier: 10.3 to 11.7 us (a launch is
// 3.7), for one chain of loads and then counts to clear, to count into and to pass over,
// and four passes over two or three rows a thread.  4096 of up to 65536 by the sums of 8
// heads, 3 sequences, 16 blocks each: 20 to 22.5 us; where they took 20, 8 blocks took
// 22, all digits counted and all counts read from every block 30.
//
// cache_compact: row j takes the place of row kept[j], kept ascending, so that
// kept[j] >= j: a cluster of 1 to 8 blocks moves the rows of one head in ascending
// chunks.  A chunk is read whole by all its blocks before any of them writes, and
// the rows that later chunks read lie behind everything written before them, so
// reads run a chunk ahead.  One thread looks a row up for all that copy its
// pieces: at 16 bytes a look-up the instructions, not the memory, took the time.  The
// rows of 16 sequences, 2048 of some 2200, 8 heads, MXFP8: 26 us = 80 % of the copy
// rate; 16384 of up to 65536 BF16 rows of 5 sequences, clusters of seven: 109.5 us =
// 91 %.  (Chunks of 16 KB, three blocks to an SM, reads a chunk or two ahead 27.4 and
// 108 or 110, clusters of powers of two alone 116; chunks of 8 KB two ahead 28 and 118; 5
// stages and two blocks 28 and 164; blocks with a part of each row, no barrier between them
// and a look-up to every piece 39 and 172.)
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
constexpr int kSelCluster = 16;           // blocks of a cluster, at most
constexpr int kCoarse = 64;               // counts of as many neighbouring bins each
constexpr int kSelRows = 40 * 1024;       // rows of a block whose bits fit into its shared memory
constexpr int kSelFixed = 2 * kBins + kLastBins;   // words of the counts
constexpr int kSelFew = 512;              // rows that are ranked among one another, at most

// Order-preserving bits of a weight; NaN below everything, -0 as +0.
__device__ __forceinline__ uint32_t weight_bits(float w) { return w != w ? 0u : orderable_key(w); }

struct Select {
  const SelectParams& p;
  int d, h, S;
  bool bad = false;
  // Bits of U rows, kSelThreads apart from row i on; rows from `end` on are not looked at.  The rows' loads
  // go together: their pages, then head by head their weights.
  template <int U>
  __device__ __forceinline__ void load(int i, int end, uint32_t (&b)[U]) {
    const float* w[U];
    int page[U];
    float v[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int r = i + k * kSelThreads;
      page[k] = r < end ? __ldg(p.table + (int64_t)d * p.max_pages + (r >> p.page_shift)) : -1;
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int r = i + k * kSelThreads;
      const bool there = (unsigned)page[k] < (unsigned)p.num_pages;
      const bool must = r < p.sinks || r >= S - p.recent;
      if (r < end && !there) bad = true;
      b[k] = must ? kMust : 0u;   // (a row on no page: as NaN)
      w[k] = there && !must ? p.weights + (((int64_t)page[k] * p.n_kv + h) << p.page_shift) + (r & ((1 << p.page_shift) - 1)) : nullptr;
      v[k] = w[k] ? __ldg(w[k]) : 0.f;
    }
    if (p.shared) {   // the heads' sum, one after the other
#pragma unroll 4
      for (int x = 1; x < p.n_kv; ++x) {
#pragma unroll
        for (int k = 0; k < U; ++k) v[k] += w[k] ? __ldg(w[k] + ((int64_t)x << p.page_shift)) : 0.f;
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (w[k]) b[k] = weight_bits(v[k]);
    }
  }
  __device__ __forceinline__ uint32_t at(int i) {   // of row i
    uint32_t b[1];
    load<1>(i, S, b);
    return b[0];
  }
};

// What finding a bin leaves for all threads, and what it counts with.
struct Find {
  int bin, want, count, here;       // here: it was this block that found it
  int coarse[3][kCoarse];           // of this block's counts, of each step (others read them until the next but one barrier)
  int sum[2][kCoarse];              // of the cluster's: coarse, then of one coarse count's bins
};

// Of 64 counts, from the top down, the one that holds the `want`-th entry; one warp calls.  Lane 0 stores
// its index, its size and what is left of `want`.
__device__ __forceinline__ void find_of_64(const int* counts, int want, Find* f) {
  const int lane = threadIdx.x & 31, a = counts[63 - 2 * lane], b = counts[62 - 2 * lane];
  int incl = a + b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  const int above = incl - a - b;
  if (above < want && incl >= want) {
    const bool first = above + a >= want;
    f->bin = first ? 63 - 2 * lane : 62 - 2 * lane;
    f->count = first ? a : b;
    f->want = first ? want - above : want - above - a;
  }
}

// Finds the bin of the `want`-th largest entry of the cluster's counts hist[n] and takes off `want` what
// lies above it; *count: entries of the bin.  The whole cluster calls, each block's counts being complete;
// every thread gets the result.  Counts of n / 64 neighbouring bins first, so that little is read from
// other blocks.  f->sum is zero before the unit's first call and after every call.
__device__ __forceinline__ int find_bin(cg::cluster_group& cluster, uint32_t* hist, int n, int step, int* want, int* count, Find* f) {
  const int tid = threadIdx.x, blocks = cluster.num_blocks(), fine = n / kCoarse;
  {
    const int per = n / kSelThreads > 0 ? n / kSelThreads : 1;   // bins of a thread; threads to a coarse count
    int c = 0;
    if (tid * per < n)
      for (int i = 0; i < per; ++i) c += hist[tid * per + i];
    for (int o = fine / per / 2; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    if (tid * per < n && tid % (fine / per) == 0) f->coarse[step][tid * per / fine] = c;
  }
  if (blocks > 1) cluster.sync(); else __syncthreads();
  auto gather = [&](int* from, int* to, int size) {   // `size` (at most 64) counts of all blocks
    if (blocks > 1) {
      if (tid < size * blocks) {
        const int v = *(cluster.map_shared_rank(from, tid / size) + tid % size);
        if (v) atomicAdd(to + tid % size, v);
      }
    } else if (tid < size) {
      to[tid] = from[tid];
    }
    __syncthreads();
  };
  gather(f->coarse[step], f->sum[0], kCoarse);
  if (tid < 32) find_of_64(f->sum[0], *want, f);
  __syncthreads();
  const int top = f->bin, left = f->want;
  gather(reinterpret_cast<int*>(hist) + top * fine, f->sum[1], fine);
  if (tid < 32) find_of_64(f->sum[1], left, f);
  __syncthreads();
  if (tid < kCoarse) f->sum[0][tid] = f->sum[1][tid] = 0;
  *want = f->want;
  *count = f->count;
  return top * fine + f->bin;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const __grid_constant__ SelectParams p) {
  extern __shared__ __align__(16) uint32_t sm[];
  uint32_t* const hist[3] = {sm, sm + kBins, sm + 2 * kBins};
  uint32_t* const bits = sm + kSelFixed;     // [p.cached]
  __shared__ Find found;
  __shared__ int counts[2][kSelWarps];
  __shared__ int total[3];   // few rows collected; rows above and at the last value
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
      if (h == 0) {   // (no weight is read, but a page that does not exist is reported)
        const int pages = (S + (1 << p.page_shift) - 1) >> p.page_shift;
        for (int i = rank * kSelThreads + tid; i < pages; i += blocks * kSelThreads)
          if ((unsigned)__ldg(p.table + (int64_t)d * p.max_pages + i) >= (unsigned)p.num_pages) code = DSA_DEV_ERR_INVALID_ARG;
      }
      for (int i = rank * kSelThreads + tid; i < p.budget; i += blocks * kSelThreads) out[i] = i < S ? i : -1;
      continue;
    }
    const int per = ((S + blocks - 1) / blocks + 31) & ~31;   // this block's rows: a whole number of warps' steps
    const int lo = min(S, rank * per), n = min(S, lo + per) - lo;
    const bool cached = per <= p.cached;
    Select sel{p, d, h, S};
    auto value = [&](int i) { return cached ? bits[i] : sel.at(lo + i); };
    for (int i = tid; i < kSelFixed; i += kSelThreads) sm[i] = 0;
    if (tid == 0) total[0] = found.here = 0;
    if (tid < kCoarse) found.sum[0][tid] = found.sum[1][tid] = 0;
    __syncthreads();
    int want = p.budget;
    uint32_t prefix = 0;
    // 12 bits, then 12 and 8 among the rows that share those before them
#pragma unroll 1
    for (int step = 0; step < 3; ++step) {
      const int shift = step == 0 ? 20 : (step == 1 ? 8 : 0), bins = step == 2 ? kLastBins : kBins;
      uint32_t* const count = hist[step];
      constexpr int U = 4;   // rows of a thread whose loads go together
      for (int i0 = 0; i0 < n; i0 += U * kSelThreads) {
        uint32_t b[U];
        if (step == 0 || !cached) sel.load<U>(lo + i0 + tid, lo + n, b);
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const int i = i0 + k * kSelThreads + tid;
          if (cached && i < n) {
            if (step == 0) bits[i] = b[k];
            else b[k] = bits[i];
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
      __syncthreads();
      int in_bin;
      prefix = (prefix << (step == 2 ? 8 : 12)) | (uint32_t)find_bin(cluster, count, bins, step, &want, &in_bin, &found);
      if (step == 0 && in_bin <= kSelFew) {
        // few rows share the last one's first digit: every block collects its own, then all of them
        unsigned long long* const own = reinterpret_cast<unsigned long long*>(hist[1]);
        unsigned long long* const few = blocks > 1 ? own + kSelFew : own;
        for (int i = tid; i < n; i += kSelThreads) {
          const uint32_t b = value(i);
          if ((b >> 20) == prefix) own[atomicAdd(&total[0], 1)] = (unsigned long long)(~b) << 32 | (unsigned)(lo + i);
        }
        sync();
        if (blocks > 1) {
          // of entry `tid`: its block and its place there
          int end = lane < blocks ? *cluster.map_shared_rank(total, lane) : 0;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, end, o);
            if (lane >= o) end += y;
          }
          int block = 0, at = tid;
          for (int r = 0; r < blocks; ++r) {
            const int e = __shfl_sync(0xffffffffu, end, r);
            if (tid >= e) {
              block = r + 1;
              at = tid - e;
            }
          }
          if (tid < in_bin) few[tid] = cluster.map_shared_rank(own, block)[at];
        }
        __syncthreads();
        // a warp ranks one of the block's own among all
        for (int c = warp; c < total[0]; c += kSelWarps) {
          const unsigned long long mine = own[c];
          int before = 0, above = 0;
          for (int i = lane; i < in_bin; i += 32) {
            const unsigned long long other = few[i];
            before += other < mine;
            above += (uint32_t)(other >> 32) < (uint32_t)(mine >> 32);
          }
          if (__reduce_add_sync(0xffffffffu, before) == want - 1) {   // the last that stays
            above = __reduce_add_sync(0xffffffffu, above);
            if (lane == 0) {
              found.bin = (int)~(uint32_t)(mine >> 32);
              found.want = want - above;
              found.here = 1;
            }
          }
        }
        sync();
        const Find* f = &found;
        if (blocks > 1) {
          const uint32_t there = __ballot_sync(0xffffffffu, lane < blocks && cluster.map_shared_rank(&found, lane % blocks)->here);
          f = cluster.map_shared_rank(&found, __ffs(there) - 1);
        }
        prefix = (uint32_t)f->bin;
        want = f->want;
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
      total[1] = above + n_above;
      total[2] = equal + n_equal;
    }
    sync();
    if (blocks > 1) {   // rows of the blocks before
      const int* const t = cluster.map_shared_rank(total, lane < rank ? lane : rank);
      above += __reduce_add_sync(0xffffffffu, lane < rank ? t[1] : 0);
      equal += __reduce_add_sync(0xffffffffu, lane < rank ? t[2] : 0);
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
constexpr int kMovePer = 3;                                          // 16-byte pieces of a thread in a chunk
constexpr int kMoveChunkBytes = kMoveThreads * kMovePer * 16;
constexpr int kMoveStages = 2;
constexpr int kMoveRows = kMoveChunkBytes / 64;                      // of a chunk, at most: one to a thread
constexpr int kMoveCluster = 8;                                      // blocks of a cluster, at most
static_assert(kMoveRows <= kMoveThreads, "a thread to a row");

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Shared memory of a block: the chunks' rows, the cache rows that they come from and go to, their weights
// and the words that hold their scales.
// A chunk is looked up kMoveStages steps before it is written, and a thread may be a step ahead of another's
// writing: two slots more than lie between.
constexpr int kMoveSlots = kMoveStages + 2;
struct MoveRing {
  uint4 rows[kMoveStages][kMoveChunkBytes / 16];
  uint32_t from[kMoveSlots][kMoveRows], to[kMoveSlots][kMoveRows];
  uint32_t weight[kMoveSlots][kMoveRows], scale[kMoveSlots][kMoveRows];
};

// What the cluster's threads have read before it is read before any writes behind it, and the block's shared
// memory is visible to it.  What has been read is in shared memory or registers by then, so nothing has to
// be made visible to other blocks: a release would wait for the last chunk's writes (some 1 us a chunk).
__device__ __forceinline__ void move_barrier(int blocks) {
  if (blocks > 1) {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
  }
  __syncthreads();
}

// Keys or values of one head of one sequence, with their scales (T, null: none) and, with the keys, the
// rows' weights.  Thread t looks up row t of a chunk: the rows' entries are requested two steps before they
// are looked up, their pages one; then a chunk's rows are requested, a chunk before they are written.
template <class T>
__device__ __forceinline__ bool move_head(const CompactParams& p, int d, int h, int n, uint8_t* base, T* scales, float* weights,
                                          int blocks, int rank, MoveRing* ring) {
  const int tid = threadIdx.x, pieces = p.row_bytes / 16, rows = kMoveChunkBytes / p.row_bytes;
  const int32_t* const kept = p.kept + ((int64_t)d * p.heads + (p.heads > 1 ? h : 0)) * p.width;
  const int32_t* const table = p.c.table + (int64_t)d * p.c.max_pages;
  const int chunk = blocks * rows, chunks = (n + chunk - 1) / chunk, mask = (1 << p.c.page_shift) - 1;
  bool bad = false;
  const int j0 = rank * rows + tid;   // this thread's row of the first chunk
  auto entry = [&](int j) { return tid < rows && j < n ? __ldg(kept + j) : -1; };
  auto page = [&](int i) { return i >= 0 && (i >> p.c.page_shift) < p.c.max_pages ? __ldg(table + (i >> p.c.page_shift)) : -1; };
  auto row = [&](int i, int page) {   // cache row of position i on its page, ~0: there is none (reported)
    if ((unsigned)page < (unsigned)p.c.num_pages) return (uint32_t)((((int64_t)page * p.c.n_kv + h) << p.c.page_shift) + (i & mask));
    bad = true;
    return ~0u;
  };
  int e0 = entry(j0), e1 = entry(j0 + chunk), before = j0 > 0 ? entry(j0 - 1) : -1, before1 = entry(j0 + chunk - 1);
  int pf = page(e0), pt = page(tid < rows && j0 < n ? j0 : -1);
  // Looks up this thread's row of chunk f, and requests what the next ones need.
  auto look_up = [&](int f) {
    const int j = j0 + f * chunk, slot = f % kMoveSlots;
    uint32_t from = ~0u, to = ~0u;
    if (tid < rows && j < n) {
      if (e0 < j || e0 <= before) {   // not ascending
        bad = true;
      } else {
        from = row(e0, pf);
        to = row(j, pt);
        if (from == ~0u || to == ~0u || e0 == j) from = to = ~0u;   // nothing to move
      }
    }
    if (from != ~0u) {
      // (a scale of one or two bytes comes with the word that it is in)
      if (scales) cp_async_4(smem_u32(&ring->scale[slot][tid]), reinterpret_cast<const uint32_t*>(scales) + from * sizeof(T) / 4);
      if (weights) cp_async_4(smem_u32(&ring->weight[slot][tid]), weights + from);
    }
    if (tid < rows) {
      ring->from[slot][tid] = from;
      ring->to[slot][tid] = to;
    }
    e0 = e1;
    before = before1;
    pf = page(e0);
    pt = page(tid < rows && j + chunk < n ? j + chunk : -1);
    e1 = entry(j + 2 * chunk);
    before1 = entry(j + 2 * chunk - 1);
  };
  look_up(0);
  __syncthreads();
  for (int c = 1 - kMoveStages; c < chunks; ++c) {
    const int f = c + kMoveStages - 1;
    if (f < chunks) {
      const uint32_t dst = smem_u32(&ring->rows[f % kMoveStages][tid]);
#pragma unroll
      for (int s = 0; s < kMovePer; ++s) {
        const int x = s * kMoveThreads + tid;
        const uint32_t from = ring->from[f % kMoveSlots][x / pieces];
        if (from != ~0u) cp_async_16(dst + s * kMoveThreads * 16, base + (size_t)from * p.row_bytes + (x & (pieces - 1)) * 16);
      }
    }
    cp_commit();        // (with the scales and weights that the last look-up requested)
    look_up(f + 1);
    cp_wait<kMoveStages - 1>();
    move_barrier(blocks);   // the whole chunk c has been read
    if (c < 0) continue;
#pragma unroll
    for (int s = 0; s < kMovePer; ++s) {
      const int x = s * kMoveThreads + tid;
      const uint32_t dst = ring->to[c % kMoveSlots][x / pieces];
      if (dst != ~0u) *reinterpret_cast<uint4*>(base + (size_t)dst * p.row_bytes + (x & (pieces - 1)) * 16) = ring->rows[c % kMoveStages][x];
    }
    const int slot = c % kMoveSlots;
    const uint32_t to = tid < rows ? ring->to[slot][tid] : ~0u;
    if (to != ~0u) {
      if (scales) {
        const uint32_t from = ring->from[slot][tid], word = ring->scale[slot][tid];
        scales[to] = (T)(word >> (from * sizeof(T) % 4 * 8));
      }
      if (weights) weights[to] = __uint_as_float(ring->weight[slot][tid]);
    }
  }
  cp_wait<0>();
  __syncthreads();
  return bad;
}

__global__ void __launch_bounds__(kMoveThreads, 4) cache_compact_kernel(const __grid_constant__ CompactParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  MoveRing* const ring = reinterpret_cast<MoveRing*>(smem);
  cg::cluster_group cluster = cg::this_cluster();
  const int blocks = cluster.num_blocks(), rank = cluster.block_rank(), tensors = p.c.v ? 2 : 1;
  const int64_t units = (int64_t)p.num_seqs * p.c.n_kv * tensors;
  int code = 0;
  for (int64_t u = blockIdx.x / blocks; u < units; u += gridDim.x / blocks) {
    const bool values = u % tensors != 0;
    const int dh = (int)(u / tensors), d = dh / p.c.n_kv, h = dh - d * p.c.n_kv, n = __ldg(p.kept_len + d);
    if (n < 0 || n > p.width) {
      code = DSA_DEV_ERR_INVALID_ARG;
      continue;
    }
    uint8_t* const base = reinterpret_cast<uint8_t*>(values ? p.c.v : p.c.k);
    uint8_t* const scales = values ? p.c.v_scale : p.c.k_scale;
    float* const weights = values ? nullptr : p.weights;
    bool bad;
    if (p.c.sw == 4) bad = move_head(p, d, h, n, base, reinterpret_cast<uint32_t*>(scales), weights, blocks, rank, ring);
    else if (p.c.sw == 2) bad = move_head(p, d, h, n, base, reinterpret_cast<uint16_t*>(scales), weights, blocks, rank, ring);
    else bad = move_head(p, d, h, n, base, p.c.sw ? scales : nullptr, weights, blocks, rank, ring);
    if (bad) code = DSA_DEV_ERR_INVALID_ARG;
  }
  code = __syncthreads_or(code != 0) ? DSA_DEV_ERR_INVALID_ARG : 0;
  if (threadIdx.x == 0) put_block_status(p.hdr, code);
}

// Once per device: the kernel's shared memory beyond the default, and clusters of sixteen blocks.
template <class K>
cudaError_t allow_smem(std::atomic<uint64_t>& ready, K kernel, int bytes, bool sixteen = false) {
  int dev = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if (ready.load(std::memory_order_acquire) >> (dev & 63) & 1) return cudaSuccess;
  if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) != cudaSuccess) return e;
  if (sixteen && (e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return e;
  ready.fetch_or(1ull << (dev & 63), std::memory_order_release);
  return cudaSuccess;
}

cudaLaunchConfig_t cluster_config(cudaLaunchAttribute* attr, int clusters, int blocks, int threads, int smem, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = blocks;
  attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(clusters * blocks));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <class K, class P>
cudaError_t launch_clusters(K kernel, const P& p, int clusters, int blocks, int threads, int smem, cudaStream_t stream) {
  cudaLaunchAttribute attr{};
  const cudaLaunchConfig_t cfg = cluster_config(&attr, clusters, blocks, threads, smem, stream);
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_evict_select(const SelectParams& call, int sm_count, cudaStream_t stream) {
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(ready, evict_select_kernel, (kSelFixed + kSelRows) * 4, true);
  if (e != cudaSuccess) return e;
  SelectParams p = call;
  const int64_t units = (int64_t)p.num_seqs * (p.shared ? 1 : p.n_kv);
  // more blocks to a head while there are SMs for them and eight rows to a thread, or to hold its rows' bits
  // (sixteen of them, which not every cluster of SMs has room for at any time, for few heads alone)
  int blocks = 1;
  while (blocks < kSelCluster / 2 && ((units * blocks * 2 <= sm_count && p.max_seqlen_k / blocks > 8 * kSelThreads) ||
                                      p.max_seqlen_k / blocks > kSelRows))
    blocks *= 2;
  static std::atomic<uint64_t> sixteen{0}, asked{0};
  if (blocks == kSelCluster / 2 && units * kSelCluster <= sm_count / 2 && p.max_seqlen_k / blocks > 4 * kSelThreads) {
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(asked.load(std::memory_order_acquire) & bit)) {   // once per device: whether it has room for one
      cudaLaunchAttribute attr{};
      const cudaLaunchConfig_t cfg = cluster_config(&attr, 1, kSelCluster, kSelThreads, (kSelFixed + kSelRows) * 4, stream);
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, evict_select_kernel, &cfg) != cudaSuccess) cudaGetLastError();
      if (n > 0) sixteen.fetch_or(bit, std::memory_order_release);
      asked.fetch_or(bit, std::memory_order_release);
    }
    if (sixteen.load(std::memory_order_acquire) & bit) blocks = kSelCluster;
  }
  const int64_t rows = ((int64_t)(p.max_seqlen_k + blocks - 1) / blocks + 31) & ~31;
  p.cached = (int)(rows < kSelRows ? rows : kSelRows);
  int64_t clusters = DSA_DEV_STATUS_MAX_BLOCKS / blocks;
  if (clusters > units) clusters = units;
  return launch_clusters(evict_select_kernel, p, (int)clusters, blocks, kSelThreads, (kSelFixed + p.cached) * 4, stream);
}

cudaError_t launch_cache_compact(const CompactParams& p, int sm_count, cudaStream_t stream) {
  constexpr int kResident = 4;   // blocks of an SM
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(ready, cache_compact_kernel, sizeof(MoveRing));
  if (e != cudaSuccess) return e;
  // more blocks to a head while all of them are on the SMs at once
  const int64_t units = (int64_t)p.num_seqs * p.c.n_kv * (p.c.v ? 2 : 1);
  int blocks = 1;
  while (blocks < kMoveCluster && units * (blocks + 1) <= kResident * sm_count) ++blocks;
  int64_t clusters = DSA_DEV_STATUS_MAX_BLOCKS / blocks;
  if (clusters > units) clusters = units;
  return launch_clusters(cache_compact_kernel, p, (int)clusters, blocks, kMoveThreads, sizeof(MoveRing), stream);
}

}  // namespace dsa
