// The attention weight that cached rows gather:
//   W[s, h] += sum_t sum_j exp(sm_scale q[t, j] . k[s, h] - lse[t, j])
// over the new tokens t that see row s and the heads j of key head h; rows of
// the new tokens themselves begin at 0.  With the lse of the attention the
// summands are its softmax weights, so a token adds its number of heads in all.
//
// A warp walks along the keys of one head, a step of 4 KB at a time: it copies the
// steps ahead of it into shared memory of its own, and forms the products of a
// step's keys with 8 query rows (token, head of the group) at a time by mma.sync
// m16n8k16.  (The tensor memory of tcgen05 would have 128 rows of keys wait for
// one another; here the keys are read once and the products are small.)  The sum
// over the head's elements has no order, so a lane's consecutive bytes of a row
// stand for the fragment's elements, of queries and keys alike.  64 sequences of 2048 -
// 16384 rows, a token each, 64 heads on 8: 185 us over BF16 rows = 95 % of the copy rate;
// 110 over MXFP8 ones = 85 %, where the instructions that turn codes into FP16 and apply
// the scales count too (114 with two halves of a word taken apart by shifts and rows
// looked up one by one; refilling the ring before the products gains nothing; of the four
// forms that of 128 8-bit elements alone spills, 88 bytes at its 128 registers).
//
// 8-bit rows: E4M3 is exact in FP16, and with at most eight query rows so are the
// queries once each row is scaled by a power of two, unless its elements span
// more than 2^31 or are so far from one that the scaled products could leave FP32.
// The codes then take one conversion to a pair, and the blocks' scales are applied
// to the products of a block.  Else the rows are widened to BF16, in which E4M3 x
// 2^e is exact (32 query rows, 32 such sequences: 165 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "e4m3_widen.cuh"
#include "tile_pipeline.cuh"
#include "weigh.cuh"

namespace dsa {

namespace weigh {

using attn::ex2;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kStepBytes = 4096;   // of keys
constexpr int kSteps = 3;          // in a warp's ring

// Keys of a step.
template <int D, bool Q8>
struct Step {
  static constexpr int kRow = D * (Q8 ? 1 : 2);                           // bytes
  static constexpr int kKeys = kRow == 256 ? 16 : 32;
  static constexpr int kUnit = Q8 ? 32 : 64;                              // bytes of a row that four lanes read together
  // Units of neighbouring rows change places, so that what a quarter (half) of a warp reads at a time is
  // spread over all banks.
  static __device__ __forceinline__ uint32_t at(int row, int unit) {
    const int x = Q8 ? (kRow == 128 ? row & 3 : (row >> 1) & 1) : row & 1;
    return row * kRow + (unit ^ x) * kUnit;
  }
};

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_16816_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four E4M3 codes as FP16.
__device__ __forceinline__ void codes_f16(uint32_t four, uint32_t (&o)[2]) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(o[0]), "=r"(o[1])
      : "r"(four));
}

// First of the steps of sequence d, in a numbering from 0 with room for all of each sequence; k0: the key
// prefix's first entry (not 0 where it is a part of a longer batch's).
template <int kKeys>
__device__ __forceinline__ int step_base(const WeighParams& p, int k0, int d) {
  return (__ldg(p.cu_k + d) - k0) / kKeys + d;
}

template <int D, bool Q8>
__global__ void __launch_bounds__(kThreads, 2) weigh_kernel(const __grid_constant__ WeighParams p) {
  using St = Step<D, Q8>;
  constexpr int kKeys = St::kKeys;
  constexpr int kBlocks = D / 32;                 // blocks of 32 elements: of a query row 16 bytes to a lane each
  extern __shared__ __align__(128) uint8_t ring[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, t = lane & 3, g = lane >> 2;
  const uint32_t sring = smem_u32(ring) + warp * kSteps * kStepBytes;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // (the tiles' kernel, where the call has one)
  const bool together = (1 << p.c.page_shift) >= kKeys;   // the rows of a step are one piece of a page
  int code = 0;
  // Prefixes that fall make rows count for several sequences, or for none: nothing is computed.
  bool falls = false, any = false;   // any: sequences of this kernel
  for (int d = tid; d < p.num_seqs; d += kThreads) {
    Doc o;
    if (!doc_info(p, d, &o)) {
      code = DSA_DEV_ERR_INVALID_ARG;
      falls |= __ldg(p.cu_k + d) < 0 || __ldg(p.cu_k + d + 1) < __ldg(p.cu_k + d) || __ldg(p.cu_q + d) < 0 ||
               __ldg(p.cu_q + d + 1) < __ldg(p.cu_q + d);
    }
    any |= o.T > 0 && by_steps(p, o.T);
  }
  if (tid == 0 && __ldg(p.cu_q + p.num_seqs) > p.total_q) code = DSA_DEV_ERR_INVALID_ARG;
  const bool none = __syncthreads_or(falls) || !__syncthreads_or(any);
  const int k0 = __ldg(p.cu_k), n_steps = none ? 0 : step_base<kKeys>(p, k0, p.num_seqs);
  const int64_t units = (int64_t)n_steps * p.c.n_kv, warps = (int64_t)gridDim.x * kWarps;
  const int64_t per = (units + warps - 1) / warps;
  int64_t u = ((int64_t)blockIdx.x * kWarps + warp) * per;
  const int64_t u_end = u + per < units ? u + per : units;

  while (u < u_end) {
    // ---- a run: consecutive steps of one sequence and head ----
    const int h = (int)(u / n_steps), su = (int)(u - (int64_t)h * n_steps);
    int lo = 0, hi = p.num_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (step_base<kKeys>(p, k0, mid) <= su) lo = mid; else hi = mid - 1;
    }
    const int d = lo, base = step_base<kKeys>(p, k0, d), next_base = step_base<kKeys>(p, k0, d + 1);
    Doc doc;
    doc_info(p, d, &doc);
    const int64_t run_end = u + (next_base - su) < u_end ? u + (next_base - su) : u_end;
    const int n_rows = by_steps(p, doc.T) ? doc.T * p.group : 0, P0 = doc.S - doc.T, first = (su - base) * kKeys;
    int n = (int)(run_end - u);
    if (n > (doc.S - first + kKeys - 1) / kKeys) n = (doc.S - first + kKeys - 1) / kKeys;
    u = run_end;
    if (n_rows == 0 || n <= 0) continue;

    uint4 qf[kBlocks];   // query row r0 + g: elements c * 32 + 8 t ..
    float2 bias;         // of rows r0 + 2 t and the next one
    auto load_q = [&](int r0) {
      int hg;
      const bool there = r0 + g < n_rows;
      const int tok = token_of(p, there ? r0 + g : 0, &hg);
      const uint16_t* src =
          reinterpret_cast<const uint16_t*>(p.q) + (int64_t)(doc.q0 + tok) * p.q_stride + (int64_t)(h * p.group + hg) * D + 8 * t;
#pragma unroll
      for (int c = 0; c < kBlocks; ++c)
        qf[c] = there ? __ldg(reinterpret_cast<const uint4*>(src + c * 32)) : make_uint4(0, 0, 0, 0);
      float v[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = r0 + 2 * t + e;
        const int tk = token_of(p, r < n_rows ? r : 0, &hg);
        const float l = __ldg(p.lse + (int64_t)(doc.q0 + tk) * p.n_heads + h * p.group + hg);
        v[e] = r < n_rows ? bias_of(l) : -INFINITY;
      }
      bias = make_float2(v[0], v[1]);
    };
    if (n_rows <= 8) load_q(0);
    // FP16 queries, where that loses nothing
    bool half = false;
    float2 colscale = make_float2(p.scale_log2, p.scale_log2);
    if (Q8 && n_rows <= 8) {
      uint32_t top = 0, low = 0x7FFFu;   // magnitudes of this lane's elements as BF16 bits: largest, smallest but 0
#pragma unroll
      for (int c = 0; c < kBlocks; ++c) {
        const uint32_t w[4] = {qf[c].x, qf[c].y, qf[c].z, qf[c].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t m = (i & 1 ? w[i >> 1] >> 16 : w[i >> 1]) & 0x7FFFu;
          top = max(top, m);
          low = min(low, m == 0 ? 0x7FFFu : m);
        }
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        low = min(low, __shfl_xor_sync(0xffffffffu, low, o));
      }
      // the largest element goes to exponent 14, the least bit of the smallest stays at 2^-24 or above; and FP32 holds
      // the scaled products wherever it holds the logit: one that leaves it stands for a logit of 2^24 and more, of
      // whose weight nothing is left in FP32, and what it loses at its lower end is below 2^-40 of a logit
      const int e_top = top >> 7, e_low = low >> 7;
      const float back = top == 0 ? 1.f : __uint_as_float((uint32_t)max(e_top - 14, 0) << 23), scale = back * p.scale_log2;
      const bool fits = (top == 0 || (e_top >= 15 && e_top < 255 && e_low >= 1 && e_top - e_low <= 31)) && scale >= 0x1p-104f &&
                        scale <= 0x1p104f;
      half = __all_sync(0xffffffffu, fits);
      if (half) {
        const float f = top == 0 ? 1.f : __uint_as_float((uint32_t)(14 + 254 - e_top) << 23);   // 2^(14 - (e_top - 127))
#pragma unroll
        for (int c = 0; c < kBlocks; ++c) {
          uint32_t w[4] = {qf[c].x, qf[c].y, qf[c].z, qf[c].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const __half2 v = __floats2half2_rn(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xFFFF0000u) * f);
            w[i] = *reinterpret_cast<const uint32_t*>(&v);
          }
          qf[c] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        // of columns 2 t and 2 t + 1 (rows that lanes 8 t and 8 t + 4 hold)
        colscale = make_float2(__shfl_sync(0xffffffffu, scale, 8 * t), __shfl_sync(0xffffffffu, scale, 8 * t + 4));
      }
    }

    // ---- a lane looks up one key of a step: its row, its scales, its weight so far ----
    struct Ahead {
      uint32_t row, scale;
      float old;
    };
    bool bad = false;
    const int64_t table = (int64_t)d * p.c.max_pages;
    auto key_of = [&](int i) { return i < n && lane < kKeys ? first + i * kKeys + lane : doc.S; };   // (doc.S: none)
    auto page_of = [&](int i) {
      const int key = key_of(i);
      return key < doc.S ? __ldg(p.c.table + table + (key >> p.c.page_shift)) : 0;
    };
    auto fetch = [&](int i, int page) {
      Ahead a{~0u, 0u, 0.f};
      const int key = key_of(i);
      if (key < doc.S) {
        if ((unsigned)page < (unsigned)p.c.num_pages) {
          a.row = (uint32_t)((((int64_t)page * p.c.n_kv + h) << p.c.page_shift) + (key & ((1 << p.c.page_shift) - 1)));
          if (key < P0) a.old = __ldcg(p.weights + a.row);
          if constexpr (Q8) {   // a byte to each block
            if (p.c.sw == 1) a.scale = __ldg(p.c.k_scale + a.row) * 0x01010101u;
            else if constexpr (D == 128) a.scale = __ldg(reinterpret_cast<const uint32_t*>(p.c.k_scale) + a.row);
            else a.scale = __ldg(reinterpret_cast<const uint16_t*>(p.c.k_scale) + a.row);
          }
        } else {
          bad = true;
        }
      }
      if (i < n) {
        constexpr int PPR = St::kRow / 16, RPI = 32 / PPR;   // 16-byte pieces of a row, rows of an instruction
        const int piece = lane % PPR, rsub = lane / PPR;
        const uint8_t* const src = reinterpret_cast<const uint8_t*>(p.c.k) + piece * 16;
        const uint32_t dst = sring + (i % kSteps) * kStepBytes + piece * 16 % St::kUnit;
        if (together) {   // (behind a sequence's last row what the page holds: of no consequence to other keys)
          const uint32_t row = __shfl_sync(0xffffffffu, a.row, 0);
          const uint8_t* const at = src + (size_t)(row == ~0u ? 0 : row + rsub) * St::kRow;
#pragma unroll
          for (int r = 0; r < kKeys; r += RPI)
            attn::cp_async16(dst + St::at(r + rsub, piece * 16 / St::kUnit), at + r * St::kRow, row != ~0u);
        } else {
#pragma unroll
          for (int r = 0; r < kKeys; r += RPI) {
            const uint32_t row = __shfl_sync(0xffffffffu, a.row, r + rsub);
            attn::cp_async16(dst + St::at(r + rsub, piece * 16 / St::kUnit), src + (size_t)(row == ~0u ? 0 : row) * St::kRow, row != ~0u);
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      return a;
    };
    Ahead a0 = fetch(0, page_of(0)), a1 = fetch(1, page_of(1)), a2 = fetch(2, page_of(2));
    int page = page_of(3);
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kSteps - 1) : "memory");
      __syncwarp();
      const uint32_t step = sring + (i % kSteps) * kStepBytes;
      const int key0 = first + i * kKeys;
      const bool edge = key0 + kKeys > P0 + 1;   // some token does not see some key
      const int r_first = edge && key0 > P0 ? (key0 - P0) * p.group : 0;   // rows before it see none of these keys
      constexpr int kTiles = kKeys / 16;
      float sum[2 * kTiles];   // of keys g, g + 8, ..
#pragma unroll
      for (int m = 0; m < 2 * kTiles; ++m) sum[m] = 0.f;
      // the weights of keys 16 m + g (and + 8) under query rows r0 + 2 t and the next one
      auto add = [&](const float (&acc)[4], int m, int r0) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = ex2(fmaf(acc[e], e & 1 ? colscale.y : colscale.x, e & 1 ? bias.y : bias.x));
        if (edge) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            int hg;
            const int vis = P0 + token_of(p, r0 + 2 * t + e, &hg);
            if (key0 + 16 * m + g > vis) w[e] = 0.f;
            if (key0 + 16 * m + 8 + g > vis) w[2 + e] = 0.f;
          }
        }
        sum[2 * m] += w[0] + w[1];
        sum[2 * m + 1] += w[2] + w[3];
      };
      if (Q8 && half) {
#pragma unroll
        for (int m = 0; m < kTiles; ++m) {
          const int ra = m * 16 + g, rb = ra + 8;   // this lane's keys
          const uint32_t ca = __shfl_sync(0xffffffffu, a0.scale, ra), cb = __shfl_sync(0xffffffffu, a0.scale, rb);
          float total[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < kBlocks; ++c) {
            uint32_t xa[2], xb[2];
            asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(xa[0]), "=r"(xa[1]) : "r"(step + St::at(ra, c) + 8 * t));
            asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(xb[0]), "=r"(xb[1]) : "r"(step + St::at(rb, c) + 8 * t));
            const uint32_t qw[4] = {qf[c].x, qf[c].y, qf[c].z, qf[c].w};
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              uint32_t fa[2], fb[2];
              codes_f16(xa[s], fa);
              codes_f16(xb[s], fb);
              mma_16816_f16(acc, fa[0], fb[0], fa[1], fb[1], qw[2 * s], qw[2 * s + 1]);
            }
            // 2^(byte - 127) from its bits (byte 0: a subnormal)
            const float fa = __uint_as_float(max(((ca >> (8 * c)) & 255u) << 23, 0x00400000u));
            const float fb = __uint_as_float(max(((cb >> (8 * c)) & 255u) << 23, 0x00400000u));
#pragma unroll
            for (int e = 0; e < 4; ++e) total[e] = fmaf(acc[e], e < 2 ? fa : fb, total[e]);
          }
          add(total, m, 0);
        }
      } else {
        uint32_t a[kTiles][2][kBlocks][4];   // the keys as pairs of BF16
#pragma unroll
        for (int i = 0; i < 2 * kTiles; ++i) {
          const int row = i * 8 + g;
          if constexpr (Q8) {
            const uint32_t sc = __shfl_sync(0xffffffffu, a0.scale, row);
#pragma unroll
            for (int c = 0; c < kBlocks; ++c) {
              uint32_t w2[2];
              asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w2[0]), "=r"(w2[1]) : "r"(step + St::at(row, c) + 8 * t));
              const uint32_t e8 = (sc >> (8 * c)) & 255u;
              if (e8 <= 134u) attn::widen<false>(w2, e8, a[i >> 1][i & 1][c]);
              else attn::widen<true>(w2, e8, a[i >> 1][i & 1][c]);
            }
          } else {
#pragma unroll
            for (int c = 0; c < kBlocks; ++c) attn::ld_shared_v4(step + St::at(row, c) + 16 * t, a[i >> 1][i & 1][c]);
          }
        }
        for (int r0 = r_first & ~7; r0 < n_rows; r0 += 8) {
          if (n_rows > 8) load_q(r0);
          float acc[kTiles][4] = {};
#pragma unroll
          for (int c = 0; c < kBlocks; ++c) {
            const uint32_t qw[4] = {qf[c].x, qf[c].y, qf[c].z, qf[c].w};
#pragma unroll
            for (int s = 0; s < 2; ++s) {
#pragma unroll
              for (int m = 0; m < kTiles; ++m)
                mma_16816(acc[m], a[m][0][c][2 * s], a[m][1][c][2 * s], a[m][0][c][2 * s + 1], a[m][1][c][2 * s + 1], qw[2 * s],
                          qw[2 * s + 1]);
            }
          }
#pragma unroll
          for (int m = 0; m < kTiles; ++m) add(acc[m], m, r0);
        }
      }
      // sums over the four lanes of a row; lane (g, t) ends with key 8 t + g (16 keys: t of 0 and 1)
      float got;
      if constexpr (kKeys == 32) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float give = t & 2 ? sum[e] : sum[e + 2], keep = t & 2 ? sum[e + 2] : sum[e];
          sum[e] = keep + __shfl_xor_sync(0xffffffffu, give, 2);
        }
        const float give = t & 1 ? sum[0] : sum[1], keep = t & 1 ? sum[1] : sum[0];
        got = keep + __shfl_xor_sync(0xffffffffu, give, 1);
      } else {
        const float give = t & 1 ? sum[0] : sum[1], keep = t & 1 ? sum[1] : sum[0];
        got = keep + __shfl_xor_sync(0xffffffffu, give, 1);
        got += __shfl_xor_sync(0xffffffffu, got, 2);
      }
      got = __shfl_sync(0xffffffffu, got, (lane & 7) * 4 + (lane >> 3) % (kKeys / 8));   // key `lane`
      if (a0.row != ~0u) p.weights[a0.row] = a0.old + got;
      // the next steps (the syncs keep the copies behind every lane's reads)
      __syncwarp();
      a0 = a1;
      a1 = a2;
      a2 = fetch(i + kSteps, page);
      page = page_of(i + kSteps + 1);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
    if (bad) code = DSA_DEV_ERR_INVALID_ARG;
  }
  code = __syncthreads_or(code != 0) ? DSA_DEV_ERR_INVALID_ARG : 0;
  if (tid == 0) put_status(p, blockIdx.x, code);
}

template <int D, bool Q8>
cudaError_t launch_steps(const WeighParams& p, int blocks, cudaStream_t stream) {
  constexpr int kSmem = kWarps * kSteps * kStepBytes;
  auto kernel = weigh_kernel<D, Q8>;
  int dev = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  static std::atomic<uint64_t> ready{0};   // devices on which this kernel is set up
  if (!(ready.load(std::memory_order_acquire) >> (dev & 63) & 1)) {
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem)) != cudaSuccess) return e;
    ready.fetch_or(1ull << (dev & 63), std::memory_order_release);
  }
  kernel<<<blocks, kThreads, kSmem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace weigh

int weigh_step_blocks(const WeighParams& p, int sm_count) {
  // no more blocks than there can be steps (of 16 keys or more)
  const int64_t steps = ((int64_t)p.max_seqlen_k / 16 + 1) * p.num_seqs * p.c.n_kv;
  const int64_t blocks = (steps + weigh::kWarps - 1) / weigh::kWarps;
  return (int)(blocks < 2 * sm_count ? blocks : 2 * sm_count);
}

cudaError_t launch_weigh_steps(const WeighParams& p, int D, int blocks, cudaStream_t stream) {
  const bool q8 = p.c.fmt != 0;
  if (D == 128) return q8 ? weigh::launch_steps<128, true>(p, blocks, stream) : weigh::launch_steps<128, false>(p, blocks, stream);
  return q8 ? weigh::launch_steps<64, true>(p, blocks, stream) : weigh::launch_steps<64, false>(p, blocks, stream);
}

}  // namespace dsa
