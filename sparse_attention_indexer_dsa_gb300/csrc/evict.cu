// Bounding a paged cache: the choice of the rows that stay, and their moving
// together in place.
//
// evict_select: of the S rows of a sequence the `budget` that come first by
// (sinks and recent rows, weight descending, position ascending), written in
// ascending order.  A block takes one head of one sequence (or the sum of its
// heads) and finds the weight of the last row that stays by digits of its
// order-preserving bits: 12, 12 and 8 of them, a count of 4096 (256) values
// each.  With the last value known, the number of rows above it and how many
// of the equal ones stay, the rows are written by a count over the block.
//
// cache_compact: row j takes the place of row kept[j], kept ascending, so that
// kept[j] >= j: a block moves a part of each row of one head in ascending
// chunks.  A chunk's rows are read whole before any of them is written, and
// the rows that later chunks read lie behind everything written before them, so
// reads run several chunks ahead.
#include "dsa_device.cuh"
#include "evict_params.h"

namespace dsa {

namespace {

// ---------------------------------------------------------------- choice

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 4096;
constexpr uint32_t kMust = 0xFFFFFFFFu;   // above every weight's bits

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
      for (int k = 1; k < p.n_kv; ++k) v += __ldg(w + ((int64_t)k << p.page_shift));
    }
    return weight_bits(v);
  }
};

// Finds the bin of the `want`-th largest entry and takes off `want` what lies above it.
// hist[n] in shared memory, n a multiple of the block's threads or less; all threads get the result.
__device__ __forceinline__ int find_bin(const uint32_t* hist, int n, int* want, int* scratch) {
  // thread i holds bins from the top down: n - 1 - i * per ..
  const int tid = threadIdx.x, per = (n + kSelThreads - 1) / kSelThreads;
  int mine = 0;
  for (int j = 0; j < per; ++j) {
    const int b = n - 1 - (tid * per + j);
    if (b >= 0) mine += hist[b];
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if ((tid & 31) >= o) incl += y;
  }
  if ((tid & 31) == 31) scratch[tid >> 5] = incl;
  __syncthreads();
  if (tid < 32) {
    int v = scratch[tid];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, o);
      if (tid >= o) v += y;
    }
    scratch[tid] = v;
  }
  __syncthreads();
  int above = incl - mine + (tid >= 32 ? scratch[(tid >> 5) - 1] : 0);
  const int w = *want;
  __syncthreads();
  if (above < w && above + mine >= w) {
    for (int j = 0; j < per; ++j) {
      const int b = n - 1 - (tid * per + j);
      if (b < 0) break;
      const int c = hist[b];
      if (above + c >= w) {
        scratch[0] = b;
        scratch[1] = w - above;
        break;
      }
      above += c;
    }
  }
  __syncthreads();
  const int bin = scratch[0];
  *want = scratch[1];
  __syncthreads();
  return bin;
}

// CACHED: the rows' bits are kept in shared memory (else they are formed again for each count).
template <bool CACHED>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const __grid_constant__ SelectParams p) {
  extern __shared__ uint32_t sm[];
  uint32_t* const hist = sm;                 // [kBins]
  uint32_t* const bits = sm + kBins;         // [S] when CACHED
  __shared__ int scratch[kSelWarps];
  __shared__ int counts[2][kSelWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int heads = p.shared ? 1 : p.n_kv;
  int code = 0;
  for (int u = blockIdx.x; u < p.num_seqs * heads; u += gridDim.x) {
    const int d = u / heads, h = u - d * heads;
    int32_t* const out = p.kept + (int64_t)u * p.budget;
    const int k0 = __ldg(p.cu_k + d), k1 = __ldg(p.cu_k + d + 1);
    int S = k1 - k0;
    if (k0 < 0 || k1 < k0 || S > p.max_seqlen_k || (int64_t)S > ((int64_t)p.max_pages << p.page_shift)) {
      code = DSA_DEV_ERR_INVALID_ARG;
      S = 0;
    }
    if (h == 0 && tid == 0) p.kept_len[d] = min(S, p.budget);
    if (S <= p.budget) {
      for (int i = tid; i < p.budget; i += kSelThreads) out[i] = i < S ? i : -1;
      continue;
    }
    Select sel{p, d, h, S};
    auto value = [&](int i) { return CACHED ? bits[i] : sel.at(i); };
    int want = p.budget;
    uint32_t prefix = 0;
    // 12 bits, then 12 and 8 among the rows that share those before them
#pragma unroll
    for (int step = 0; step < 3; ++step) {
      const int shift = step == 0 ? 20 : (step == 1 ? 8 : 0), n = step == 2 ? 256 : kBins;
      __syncthreads();
      for (int i = tid; i < n; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int i0 = 0; i0 < S; i0 += kSelThreads) {
        const int i = i0 + tid;
        uint32_t b = 0;
        if (i < S) {
          b = step == 0 ? sel.at(i) : value(i);
          if (CACHED && step == 0) bits[i] = b;
        }
        const bool in = i < S && (step == 0 || (b >> (shift + (step == 2 ? 8 : 12))) == prefix);
        const uint32_t digit = (b >> shift) & (n - 1);
        // many equal rows (none ever looked at): one count for the warp
        const uint32_t live = __ballot_sync(0xffffffffu, in);
        if (live) {
          const uint32_t first = __shfl_sync(0xffffffffu, digit, __ffs(live) - 1);
          const uint32_t same = __ballot_sync(0xffffffffu, in && digit == first);
          if (same == live) {
            if (lane == 0) atomicAdd(&hist[first], __popc(live));
          } else if (in) {
            atomicAdd(&hist[digit], 1u);
          }
        }
      }
      __syncthreads();
      prefix = (prefix << (step == 2 ? 8 : 12)) | (uint32_t)find_bin(hist, n, &want, scratch);
    }
    // `prefix` is the last value that stays, `want` the number of rows of that value that do
    const int per = ((S + kSelWarps - 1) / kSelWarps + 31) & ~31;
    const int lo = min(S, warp * per), hi = min(S, lo + per);
    int n_above = 0, n_equal = 0;
    for (int i0 = lo; i0 < hi; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t b = i < hi ? value(i) : 0u;
      n_above += __popc(__ballot_sync(0xffffffffu, i < hi && b > prefix));
      n_equal += __popc(__ballot_sync(0xffffffffu, i < hi && b == prefix));
    }
    if (lane == 0) {
      counts[0][warp] = n_above;
      counts[1][warp] = n_equal;
    }
    __syncthreads();
    int above = 0, equal = 0;   // before this warp's rows
    for (int w = 0; w < warp; ++w) {
      above += counts[0][w];
      equal += counts[1][w];
    }
    for (int i0 = lo; i0 < hi; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t b = i < hi ? value(i) : 0u;
      const uint32_t ab = __ballot_sync(0xffffffffu, i < hi && b > prefix), eq = __ballot_sync(0xffffffffu, i < hi && b == prefix);
      const uint32_t before = (1u << lane) - 1u;
      const int e = equal + __popc(eq & before);
      const bool stays = ((ab >> lane) & 1u) || (((eq >> lane) & 1u) && e < want);
      if (stays) out[above + __popc(ab & before) + min(e, want)] = i;
      above += __popc(ab);
      equal += __popc(eq);
    }
    if (sel.bad) code = DSA_DEV_ERR_INVALID_ARG;
    __syncthreads();   // (the next unit's counts)
  }
  code = __syncthreads_or(code != 0) ? DSA_DEV_ERR_INVALID_ARG : 0;
  if (tid == 0) put_block_status(p.hdr, code);
}

// ---------------------------------------------------------------- moving

constexpr int kMoveThreads = 256;
constexpr int kMoveChunkBytes = 16384;   // of a ring's stage
constexpr int kMoveStages = 4;

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
  // Cache row that row j comes from, -1: none (not a row, or already there).
  __device__ __forceinline__ int64_t source(int j) {
    if (j >= n) return -1;
    const int i = __ldg(kept + j);
    const int64_t r = i >= j ? cache_row(p.c, d, i, h) : -1;
    if (r < 0 || (j > 0 && __ldg(kept + j - 1) >= i)) bad = true;   // ascending, of the sequence's pages
    return i == j ? -1 : r;
  }
  __device__ __forceinline__ int64_t target(int j) {
    const int64_t r = cache_row(p.c, d, j, h);
    if (r < 0) bad = true;
    return r;
  }
};

// Small elements (scales, weights): read by the thread that writes them, a chunk of four rows a thread at a time.
template <class T>
__device__ __forceinline__ void move_small(Move& m, T* base) {
  constexpr int U = 4;
  for (int j0 = 0; j0 < m.n; j0 += U * kMoveThreads) {
    int64_t src[U];
    T v[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      src[k] = m.source(j0 + k * kMoveThreads + threadIdx.x);
      if (src[k] >= 0) v[k] = *reinterpret_cast<volatile T*>(base + src[k]);
    }
    __syncthreads();   // the chunk has been read
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (src[k] < 0) continue;
      const int64_t dst = m.target(j0 + k * kMoveThreads + threadIdx.x);
      if (dst >= 0) base[dst] = v[k];
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kMoveThreads) cache_compact_kernel(const __grid_constant__ CompactParams p) {
  extern __shared__ __align__(16) uint8_t ring[];
  const int tid = threadIdx.x;
  const int tensors = p.c.v ? 2 : 1;
  const bool small = p.weights || p.c.sw > 0;
  const int parts = tensors * p.slices + (small ? 1 : 0);   // of one head of one sequence
  const int64_t units = (int64_t)p.num_seqs * p.c.n_kv * parts;
  const uint32_t sbase = smem_u32(ring);
  int code = 0;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int part = (int)(u % parts), dh = (int)(u / parts), d = dh / p.c.n_kv, h = dh - d * p.c.n_kv;
    int n = __ldg(p.kept_len + d);
    if (n < 0 || n > p.width) {
      code = DSA_DEV_ERR_INVALID_ARG;
      continue;
    }
    Move m{p, d, h, n, p.kept + ((int64_t)d * p.heads + (p.heads > 1 ? h : 0)) * p.width};
    if (part < tensors * p.slices) {
      uint8_t* const base = reinterpret_cast<uint8_t*>(part < p.slices ? p.c.k : p.c.v);
      const int bytes = p.row_bytes / p.slices, pieces = bytes / 16, rows = kMoveThreads / pieces;   // a step: a row to `pieces` threads
      const int per = kMoveChunkBytes / 16 / kMoveThreads;   // steps of a chunk
      const int off = (part % p.slices) * bytes + (tid % pieces) * 16, sub = tid / pieces;
      const int chunks = (n + rows * per - 1) / (rows * per);
      auto fetch = [&](int c) {
        if (c < chunks) {
#pragma unroll
          for (int i = 0; i < per; ++i) {
            const int64_t src = m.source((c * per + i) * rows + sub);
            if (src >= 0)
              cp_async_16(sbase + (c % kMoveStages) * kMoveChunkBytes + (i * kMoveThreads + tid) * 16, base + src * p.row_bytes + off);
          }
        }
        cp_commit();
      };
      for (int c = 0; c < kMoveStages - 1; ++c) fetch(c);
      for (int c = 0; c < chunks; ++c) {
        fetch(c + kMoveStages - 1);   // (into the stage that this thread has emptied)
        cp_wait<kMoveStages - 1>();
        __syncthreads();              // the whole chunk has been read
#pragma unroll
        for (int i = 0; i < per; ++i) {
          const int j = (c * per + i) * rows + sub;
          if (m.source(j) < 0) continue;
          const int64_t dst = m.target(j);
          if (dst >= 0)
            *reinterpret_cast<uint4*>(base + dst * p.row_bytes + off) =
                *reinterpret_cast<const uint4*>(ring + (c % kMoveStages) * kMoveChunkBytes + (i * kMoveThreads + tid) * 16);
        }
      }
      cp_wait<0>();
    } else {
      if (p.weights) move_small(m, p.weights);
      for (int t = 0; t < (p.c.sw > 0 ? tensors : 0); ++t) {
        uint8_t* s = t ? p.c.v_scale : p.c.k_scale;
        if (p.c.sw == 4) move_small(m, reinterpret_cast<uint32_t*>(s));
        else if (p.c.sw == 2) move_small(m, reinterpret_cast<uint16_t*>(s));
        else move_small(m, s);
      }
    }
    if (m.bad) code = DSA_DEV_ERR_INVALID_ARG;
    __syncthreads();
  }
  code = __syncthreads_or(code != 0) ? DSA_DEV_ERR_INVALID_ARG : 0;
  if (tid == 0) put_block_status(p.hdr, code);
}

}  // namespace

cudaError_t launch_evict_select(const SelectParams& p, int sm_count, cudaStream_t stream) {
  constexpr int kSmem = 200 * 1024;
  const int64_t units = (int64_t)p.num_seqs * (p.shared ? 1 : p.n_kv);
  const int grid = (int)(units < DSA_DEV_STATUS_MAX_BLOCKS ? units : DSA_DEV_STATUS_MAX_BLOCKS);
  const size_t cached = ((size_t)kBins + (size_t)p.max_seqlen_k) * 4;
  if (cached <= kSmem) {
    const cudaError_t e = cudaFuncSetAttribute(evict_select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    evict_select_kernel<true><<<grid, kSelThreads, cached, stream>>>(p);
  } else {
    evict_select_kernel<false><<<grid, kSelThreads, kBins * 4, stream>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_cache_compact(const CompactParams& call, int sm_count, cudaStream_t stream) {
  // A row in parts of its own blocks while there are fewer than three blocks to an SM, down to 32 bytes (a sector).
  CompactParams p = call;
  const int64_t whole = (int64_t)p.num_seqs * p.c.n_kv * (p.c.v ? 2 : 1);
  for (p.slices = 1; p.row_bytes / p.slices > 32 && whole * p.slices < 3 * sm_count;) p.slices *= 2;
  constexpr int kSmem = kMoveChunkBytes * kMoveStages;
  const cudaError_t e = cudaFuncSetAttribute(cache_compact_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const int64_t units = (int64_t)p.num_seqs * p.c.n_kv * ((p.c.v ? 2 : 1) * p.slices + 1);
  int64_t grid = 3 * (int64_t)sm_count;
  if (grid > units) grid = units;
  if (grid > DSA_DEV_STATUS_MAX_BLOCKS) grid = DSA_DEV_STATUS_MAX_BLOCKS;
  cache_compact_kernel<<<(unsigned)grid, kMoveThreads, kSmem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace dsa
