// Attention of new tokens over a paged cache on the tensor cores:
//   o[t, h] = sum_s softmax_s(sm_scale q[t, h] . k[s, h / G]) v[s, h / G]
// over the keys s that token t sees (all positions up to its own, or the
// listed ones among them).
//
// Tiles.  A query tile is 128 rows: tq tokens x the G heads that share a key
// head (one token when every token has its own list).  Keys come in tiles of
// 128.  Per tile S = Q K^T (K = head_dim) goes to TMEM, the softmax warps turn
// it into P = 2^(c S - m) in BF16 in the same TMEM columns, and O += P V reads
// P from TMEM.  m is the running row maximum (log2 domain), raised only when a
// row exceeds it by more than 20, so the accumulator in TMEM is hardly ever
// rescaled: weights up to 2^20 keep their relative precision in BF16, and the
// sums and O in FP32 are far from its range.  (A warp rescales when one of its
// 32 rows must: at a margin of 8 that was every fourth tile of N(0, 1) inputs
// with outliers.)  P is rounded to BF16 because the PV product has
// BF16 operands; the sum l adds the unrounded weights.
//
// Streams.  One block per SM with two streams, each a TMEM half (S/P 128
// columns, O head_dim columns), a softmax warpgroup (a row to a thread) and an
// MMA warp: while one stream's softmax runs, the tensor core works for the
// other.  (Two warpgroups to a stream, 64 key columns each, measured 15 % slower:
// the step from S to P got no shorter, and the halves wait for each other.)
//   PAIR: the streams hold two neighbouring query tiles and share one ring of
//         key/value stages (long chunks: the keys are read half as often);
//   else: the streams are independent, each with its own units and ring
//         (single tokens, short chunks, selected rows).
// Narrow tiles.  At most 16 query rows (single tokens of few heads; head_dim
// 128) would leave seven eighths of the 128 TMEM lanes, and three of four
// softmax warps, to rows that are not there.  There the keys are the products'
// rows: S^T = K Q^T (128 keys x 16), a key to a softmax thread, P^T through
// shared memory, O^T += V^T P^T (head_dim x 16).  S and P have two buffers, so
// the next tile's logits are formed meanwhile.  4 tokens of each of 64
// sequences, 64 heads, 8 key heads, 2048 listed keys, against tiles of 128 rows:
// 482 us against 550 over MXFP8, 263 against 308 over BF16; one token and every
// key, FP8 in pages of 8: 507 against 583.  Rows that TMA brings stay with tiles
// of 128 rows, which were as fast when narrow ones were tried for them: a token
// of each of the 64 over 2048 - 16384 keys 379 us over BF16 (2.4 GB, 93 % of the
// copy rate) either way, 427 against 429 over MXFP8 (1.2 GB; 415 now).
// Over 8-bit caches the latency of a stored tile (its load, its widening, the
// hand-overs) bounds them: shared memory holds two stored tiles to a ring beside
// the widened ones, of more than 32 rows one.
// Loaders.  TMA brings all visible keys as a box per page; listed rows are copied
// one by one with cp.async (TMA row gathers of four came to 27 bytes a cycle and
// SM, cp.async from eight warps to 60); BF16 in the 128-byte swizzled layout the
// MMA reads.
// Listed position -> page -> row is resolved a step per tile, ahead of the
// copies, so its dependent loads are off the path.  Rows that are not there are
// zero-filled, so nothing outside a sequence's own rows enters a product.  Tiles
// of 8-bit caches are fetched as stored and widened to BF16 by worker warps on
// the way into a stage; E4M3 x 2^e is exact in BF16.
// Issue.  TMA and MMA instructions take their operands from uniform registers:
// issued under `lane == 0` each was a loop over lanes (some 400 cycles to a TMA
// copy beside busy workers), from an elected lane it is not: 4096 tokens over
// 32768 BF16 keys 3.13 -> 2.88 ms, ragged chunks over FP8 0.57 -> 0.50 ms.
//
// Units.  (sequence, key head, query tile, range of key tiles).  Every block
// derives the same list from the prefixes: the number of key tiles per range is
// the one of eight candidates with the shortest estimated schedule.  Divided
// ranges leave (O, m, l) in the workspace and a second kernel joins them.
#pragma once

#include <cuda_bf16.h>

#include <atomic>
#include <type_traits>

#include "dsa_device.cuh"
#include "paged_params.h"

namespace dsa {

namespace attn {

constexpr int kGroups = 64;         // sequences are counted in this many groups
// Start and end of a unit, in key tiles, and the same when its result is joined later: what the estimate of
// a schedule counts beside the tiles.  With 0 for the first 100 tokens over 700 listed rows take 30.7 against
// 29.8 us, 12 changes nothing; with 4 for the second nothing changes, 12 takes 416 to 391 us for a token of each
// of 64 sequences over MXFP8 and 29.8 to 30.4 for the listed rows.  (Other calls tried: within 1 %.)
constexpr int kOverhead = 4;
constexpr int kSplitOverhead = 6;
constexpr int kMaskRing = 8;
constexpr float kRaise = 20.f;      // log2 of the largest weight before the maximum is raised

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// True for one lane of the warp (lane 0), in a form that tells the compiler that it is one: the
// operands of TMA and MMA instructions then go to uniform registers without a loop over lanes.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Arrives (without raising the count) once this thread's earlier cp.async have landed.
__device__ __forceinline__ void cp_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The loads' destination registers named, so that no use moves above the wait.
template <int N>
__device__ __forceinline__ void tmem_ld_wait_tied(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// D[tmem] (+)= A[tmem] * B[smem], kind::f16 (BF16 operands, FP32 accumulate)
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Up to `polls` tests of a phase in a loop of four instructions.
__device__ __forceinline__ bool poll_bar(uint32_t bar, uint32_t parity, uint32_t polls) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
      "mov.u32 n, %3;\n"
      "POLL_%=:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE_%=;\n\t"
      "sub.u32 n, n, 1;\n\t"
      "setp.ne.u32 q, n, 0;\n\t"
      "@q bra POLL_%=;\n"
      "DONE_%=:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(polls)
      : "memory");
  return ok != 0;
}

// Whether a phase is over, at once (try_wait may suspend the thread while it is not).
__device__ __forceinline__ bool test_bar(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Bounded wait on phase `parity`, as mbar_wait but without the suspend hint: the
// hint's sleep and the clock read of every poll cost the waiting warps' wake-up
// and took a third of a block's issue slots.  The clock and the abort flag are
// looked at every 1024 polls.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status,
                                         uint64_t timeout_ns) {
  if (poll_bar(bar, parity, 1024)) return true;
  const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
  for (;;) {
    if (poll_bar(bar, parity, 1024)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > timeout_ns) {
      set_status(status, DSA_DEV_ERR_TIMEOUT);
      *abort_flag = 1;
      return false;
    }
  }
}

// Wait while draining after an abort: ignores the abort flag, still bounded.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, uint64_t timeout_ns) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait_sleep(bar, parity, kWaitHintNs) && globaltimer_ns() - t0 < timeout_ns) {
  }
}

struct Doc {
  int q0, T, S;
};

// A sequence's sizes; T = 0 (and false) when they are inconsistent.
__device__ __forceinline__ bool doc_info(const AttnParams& p, int d, Doc* o) {
  const int q0 = __ldg(p.cu_q + d), q1 = __ldg(p.cu_q + d + 1);
  const int k0 = __ldg(p.cu_k + d), k1 = __ldg(p.cu_k + d + 1);
  o->q0 = q0;
  o->T = q1 - q0;
  o->S = k1 - k0;
  const bool ok = q0 >= 0 && q1 >= q0 && q1 <= p.total_q && k1 >= k0 && o->S >= o->T && o->T <= p.max_seqlen_q &&
                  o->S <= p.max_seqlen_k && (int64_t)o->S <= ((int64_t)p.c.max_pages << p.c.page_shift);
  if (!ok) o->T = 0;
  return ok;
}

// Query tiles (pairs of them with PAIR) and key tiles of a sequence.
template <bool kPair>
__device__ __forceinline__ void doc_tiles(const AttnParams& p, const Doc& o, int* mt, int* kt) {
  const int per = kPair ? 2 * p.plan.tq : p.plan.tq;
  *mt = (o.T + per - 1) / per;
  *kt = ((p.topk_idx ? p.topk_width : o.S) + kAttnKeys - 1) / kAttnKeys;
}

__device__ __forceinline__ int splits_of(int kt, int chunk) { return kt <= chunk ? 1 : (kt + chunk - 1) / chunk; }

// One unit as one stream sees it.
struct Unit {
  int d, h, split, ns;
  int q0, P0;        // first packed query row of the sequence, keys before its first query
  int i0, i1;        // tokens of this stream's tile
  int last;          // end of the unit's tokens (PAIR: of both tiles)
  int lo, n;         // first key tile, number of key tiles of this stream
  int n_list;        // listed positions to look at
  int n_shared;      // key tiles the loader brings (PAIR: the longer of the two)
};

// tab: first unit of each of the kGroups groups of sequences (+ the total).
template <bool kPair>
__device__ __forceinline__ Unit decode_unit(const AttnParams& p, const int* tab, int gsz, int chunk, int u, int w) {
  int lo = 0, hi = kGroups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab[mid] <= u) lo = mid; else hi = mid - 1;
  }
  int rem = u - tab[lo];
  int d = lo * gsz;
  Doc o;
  int mt, kt, ns;
  for (;;) {
    doc_info(p, d, &o);
    doc_tiles<kPair>(p, o, &mt, &kt);
    ns = splits_of(kt, chunk);
    const int units = mt * ns * p.c.n_kv;
    if (rem < units || d + 1 >= p.num_seqs) break;
    rem -= units;
    ++d;
  }
  Unit x;
  x.d = d;
  x.ns = ns;
  x.q0 = o.q0;
  x.P0 = o.S - o.T;
  x.split = rem % ns;
  rem /= ns;
  const int tile = mt - 1 - rem % mt;   // the longest first
  x.h = rem / mt;
  const int t = kPair ? 2 * tile + w : tile;
  x.i0 = min(t * p.plan.tq, o.T);
  x.i1 = min(x.i0 + p.plan.tq, o.T);
  x.last = kPair ? min((2 * tile + 2) * p.plan.tq, o.T) : x.i1;
  int kt_own, kt_all;
  if (p.topk_idx) {
    int n = p.topk_width;
    if (p.topk_len) n = max(0, min(n, __ldg(p.topk_len + o.q0 + x.i0)));
    x.n_list = n;
    kt_own = (n + kAttnKeys - 1) / kAttnKeys;
    kt_all = kt;
  } else {
    x.n_list = 0;
    kt_own = x.i0 < x.i1 ? (x.P0 + x.i1 + kAttnKeys - 1) / kAttnKeys : 0;
    kt_all = (x.P0 + x.last + kAttnKeys - 1) / kAttnKeys;
  }
  const int per = (kt_all + ns - 1) / ns;
  x.lo = x.split * per;
  x.n = max(0, min(x.lo + per, kt_own) - x.lo);
  x.n_shared = kPair ? max(0, min(x.lo + per, kt_all) - x.lo) : x.n;
  return x;
}

__device__ __forceinline__ float2 as_f2(uint32_t a, uint32_t b) {
  return make_float2(__uint_as_float(a), __uint_as_float(b));
}

// Sixteen E4M3 codes to BF16, times 2^(e8 - 127).  Code bits s.eeee.mmm placed at a BF16's sign, low
// exponent and high mantissa bits read as value * 2^-120 (subnormals included); one exact product with
// 2^(120 + e) restores it.  That is a BF16 up to e8 = 134; FAR: beyond it (values over 2^16) there is a
// second factor.  The NaN code reads as 480 that way.  The quantisers' scale of a block with a NaN is at
// least 247 (the bits of its magnitude are the largest), so every NaN that they stored is FAR, and is put
// back there; so is scale 255, which is NaN.
template <bool FAR>
__device__ __forceinline__ void widen16(const uint32_t (&w4)[4], uint32_t e8, uint32_t (&o)[8]) {
  const uint32_t first = FAR ? 254u : e8 + 120u;               // 2^(first - 127): BF16 ends at 2^127
  __nv_bfloat162 f;
  *reinterpret_cast<uint32_t*>(&f) = (first << 7) * 0x00010001u;
#pragma unroll
  for (int q4 = 0; q4 < 4; ++q4) {
#pragma unroll
    for (int hlf = 0; hlf < 2; ++hlf) {
      const uint32_t t = __byte_perm(w4[q4], 0, hlf ? 0x3424 : 0x1404);
      uint32_t b = (t & 0x80008000u) | ((t >> 4) & 0x07F007F0u);
      __nv_bfloat162 v = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&b), f);
      o[2 * q4 + hlf] = *reinterpret_cast<uint32_t*>(&v);
    }
  }
  if constexpr (FAR) {
    __nv_bfloat162 f2;
    *reinterpret_cast<uint32_t*>(&f2) = ((e8 - 134u + 127u) << 7) * 0x00010001u;
    const __nv_bfloat162 most = __float2bfloat162_rn(e8 == 255u ? -1.f : 57344.f);   // 448 * 2^7: of the numbers
#pragma unroll
    for (int q8 = 0; q8 < 8; ++q8) {
      const __nv_bfloat162 w = *reinterpret_cast<__nv_bfloat162*>(&o[q8]);
      __nv_bfloat162 v = __hmul2(w, f2);
      o[q8] = *reinterpret_cast<uint32_t*>(&v) | __hgt2_mask(__habs2(w), most);
    }
  }
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint16_t x) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(x) : "memory");
}
__device__ __forceinline__ uint16_t bf16_bits(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
__device__ __forceinline__ void ld_shared_v4(uint32_t addr, uint32_t (&w)[4]) {
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr) : "memory");
}

// Kernel kinds: two query tiles on one stream of keys; independent streams that see every key up to
// their own; independent streams with rows gathered one by one (listed keys, and caches whose page
// scales are too short for a bulk copy).
enum { PAIR = 0, SOLO = 1, GATHER = 2 };

// Warps: 8 softmax; workers (16, or 12 of gathered rows, widen 8-bit tiles; 8 bring gathered BF16
// rows); 4 that bring gathered 8-bit rows; the rest: key loaders (TMA), query loaders, MMA 0 and 1
// last.  (The four warps of an SM's sub-partition are those of equal number modulo 4; loaders and MMA
// warps are kept on different ones.)  The shares of registers leave spills, most in the kernel of
// gathered 8-bit rows (some 580 bytes of stores and 680 of loads in the code; the other kernels of
// 128-row tiles 124 - 168 and 148 - 240).  What they cost has not been measured.
template <bool Q8, int MODE, bool NARROW>
struct Roles {
  static constexpr int kWorkWarps = MODE == GATHER ? (Q8 ? 12 : 8) : (Q8 ? 16 : 0);
  static constexpr int kBringWarps = MODE == GATHER && Q8 ? 4 : 0;
  static constexpr int kWarps = kWorkWarps > 0 ? 12 + kWorkWarps + kBringWarps : 16;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kQueryWarp = kWorkWarps > 0 ? kWarps - 4 : 10;         // and the next one
  static constexpr int kKeyWarp = kWorkWarps > 0 ? kWarps - 4 : 8;            // TMA: and the next one
  // registers: shares of what the launch holds (threads x the launch's count, a multiple of 8)
  static constexpr int kLaunchRegs = Q8 ? 72 : (MODE == GATHER ? 96 : 128);
  static constexpr int kSoftmaxRegs = Q8 ? 104 : (MODE == GATHER ? 128 : 192);
  static constexpr int kWorkRegs = Q8 ? 56 : 72;
  static constexpr int kBringRegs = 64;
  static constexpr int kAuxRegs = Q8 ? (MODE == GATHER ? 64 : 72) : (MODE == GATHER ? 80 : 64);
  static_assert(2 * kSoftmaxRegs + kWorkWarps / 4 * kWorkRegs + kBringWarps / 4 * kBringRegs +
                        (kWarps - 8 - kWorkWarps - kBringWarps) / 4 * kAuxRegs <=
                    kWarps / 4 * kLaunchRegs, "shares");
};

// Sums (or maxima) over a warp's lanes of N values a lane: half of the values change hands in every step, so it takes
// N - 1 + log2(32 / N) exchanges; lanes 32 / N * r end with value r's result.
template <int N, class F>
__device__ __forceinline__ float warp_join(float (&v)[N], int lane, F f) {
  int bit = 16;
#pragma unroll
  for (int n = N / 2; n >= 1; n >>= 1, bit >>= 1) {
    const bool up = lane & bit;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
      v[i] = f(keep, __shfl_xor_sync(0xffffffffu, give, bit));
    }
  }
  for (; bit >= 1; bit >>= 1) v[0] = f(v[0], __shfl_xor_sync(0xffffffffu, v[0], bit));
  return v[0];
}

// True for all 128 threads of a named barrier when it is for one of them (orders their shared memory).
__device__ __forceinline__ bool any_of_128(int id, bool x) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id)
      : "memory");
  return r != 0;
}

template <int D, bool Q8, int MODE, bool NARROW>
__global__ void __launch_bounds__(Roles<Q8, MODE, NARROW>::kThreads, 1)
    paged_attention_kernel(const __grid_constant__ AttnParams p) {
  using R = Roles<Q8, MODE, NARROW>;
  static_assert(!NARROW || (D == 128 && MODE == GATHER), "a narrow tile's values are the 128 rows of its second product");
  constexpr bool kPair = MODE == PAIR;
  constexpr bool kWorkerCopies = MODE == GATHER && !Q8;   // stages written by cp.async: fenced by the MMA warp
  constexpr uint32_t kStage = kAttnKeys * D * 2;     // one tile of keys or values
  constexpr uint32_t kChunk = kAttnKeys * 128;       // 64 of its columns
  constexpr int kRings = kPair ? 1 : 2;
  // One ring's workers are two teams, one widening the keys' tiles and one the values': most of a
  // tile's time is latency (waits, fences), which then overlaps.
  constexpr int kTeams = Q8 && kRings == 1 ? 2 : 1;
  constexpr int kLoaders = R::kWorkWarps > 0 ? 32 * R::kWorkWarps / (kRings * kTeams) : 32;   // threads of a team
  constexpr uint32_t kRawItem = kAttnKeys * D + 512;   // a tile as stored, with its scales
  extern __shared__ __align__(1024) uint8_t smem[];
  const AttnPlan& pl = p.plan;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sbase = smem_u32(smem);
  const uint64_t tmo = p.timeout_ns;
  const bool listed = MODE == GATHER && p.topk_idx != nullptr;

  // barriers: per ring full/empty (BF16 tiles) and raw full/empty (stored 8-bit tiles); per stream
  // q_full, q_empty, o_full, drain, and s_full, p_full, p_empty (two of each with NARROW)
  const uint32_t bars = sbase + pl.off_bars;
  int* const ctl = reinterpret_cast<int*>(smem + pl.off_bars + 8 * kAttnBars);   // status, abort, tmem base, chunk, turn
  int* const status = ctl;
  volatile int* const abort_flag = ctl + 1;
  int* const tab = reinterpret_cast<int*>(smem + pl.off_tab);
  auto bar_full = [&](int ring, int s) { return bars + 8u * (ring * 32 + s); };
  auto bar_empty = [&](int ring, int s) { return bars + 8u * (ring * 32 + 8 + s); };
  auto bar_raw_full = [&](int ring, int s) { return bars + 8u * (ring * 32 + 16 + s); };
  auto bar_raw_empty = [&](int ring, int s) { return bars + 8u * (ring * 32 + 24 + s); };
  auto bar_st = [&](int w, int i) { return bars + 8u * (64 + w * 10 + i); };
  enum { Q_FULL, Q_EMPTY, O_FULL, DRAIN, S_FULL, P_FULL = S_FULL + 2, P_EMPTY = P_FULL + 2 };
  constexpr int kMmaWarp = R::kWarps - 2;

  if (tid == 0) {
    ctl[0] = (sbase & 1023u) ? DSA_DEV_ERR_BOUNDS : 0;   // the swizzle needs a 1024-byte base
    ctl[1] = (sbase & 1023u) ? 1 : 0;
    ctl[4] = 0;
    for (int r = 0; r < kRings; ++r) {
      for (int s = 0; s < pl.nst; ++s) {
        mbar_init(bar_full(r, s), kWorkerCopies ? kLoaders + kLoaders / 32 : (R::kWorkWarps > 0 ? kLoaders / 32 : 1));
        mbar_init(bar_empty(r, s), kPair ? 2 : 1);
      }
      for (int s = 0; s < pl.nraw; ++s) {
        mbar_init(bar_raw_full(r, s), MODE == GATHER ? 64 + 2 : 1);   // (two warps: their threads' copies, their scales)
        mbar_init(bar_raw_empty(r, s), kLoaders / 32);
      }
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(bar_st(w, Q_FULL), 32);
      mbar_init(bar_st(w, Q_EMPTY), 1);
      for (int b = 0; b < 2; ++b) {
        mbar_init(bar_st(w, S_FULL + b), 1);
        mbar_init(bar_st(w, P_FULL + b), 4);
        mbar_init(bar_st(w, P_EMPTY + b), 1);
      }
      mbar_init(bar_st(w, O_FULL), 1);
      mbar_init(bar_st(w, DRAIN), 1);
    }
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc(smem_u32(ctl + 2), 512);

  // ---- the unit list (every block the same) ----
  const int gsz = (p.num_seqs + kGroups - 1) / kGroups;
  const int n_streams = (kPair ? 1 : 2) * (int)gridDim.x;
  {
    float* const red = reinterpret_cast<float*>(smem);   // scratch before any tile is loaded
    long long work = 0;
    int kmax = 0;
    bool bad = tid == 0 && (__ldg(p.cu_q + p.num_seqs) > p.total_q);
    bool broken = false;   // cu_q falls: tokens could count for several sequences, so nothing is computed
    if (tid < kGroups) {
      for (int i = 0; i < gsz; ++i) {
        const int d = tid * gsz + i;
        if (d >= p.num_seqs) break;
        Doc o;
        int mt, kt;
        bad |= !doc_info(p, d, &o);
        broken |= __ldg(p.cu_q + d) < 0 || __ldg(p.cu_q + d + 1) < __ldg(p.cu_q + d);
        doc_tiles<kPair>(p, o, &mt, &kt);
        work += (long long)mt * kt * p.c.n_kv;
        if (mt > 0) kmax = max(kmax, kt);
      }
    }
    float wsum = (float)work;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      wsum += __shfl_xor_sync(0xffffffffu, wsum, o);
      kmax = max(kmax, __shfl_xor_sync(0xffffffffu, kmax, o));
    }
    if (lane == 0 && warp < kGroups / 32) {
      red[warp] = wsum;
      red[4 + warp] = (float)kmax;
    }
    const int any_bad = __syncthreads_or(bad);
    if (any_bad && tid == 0) set_status(status, DSA_DEV_ERR_INVALID_ARG);
    const bool none = any_bad && __syncthreads_or(broken);
    wsum = red[0] + red[1];
    kmax = (int)fmaxf(red[4], red[5]);
    int chunk = none ? 0x7FFFFFFF : max(kmax, 1);
    if (pl.max_units > 0 && !none && kmax > kAttnMinChunk) {
      int cand[8];
      int units[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        units[i] = 0;
        cand[i] = i == 0 ? kmax : min(kmax, max(kAttnMinChunk, (int)ceilf(wsum / (float)(n_streams * i))));
      }
      if (tid < kGroups) {
        for (int i = 0; i < gsz; ++i) {
          const int d = tid * gsz + i;
          if (d >= p.num_seqs) break;
          Doc o;
          int mt, kt;
          doc_info(p, d, &o);
          doc_tiles<kPair>(p, o, &mt, &kt);
#pragma unroll
          for (int c = 0; c < 8; ++c) units[c] += mt * p.c.n_kv * splits_of(kt, cand[c]);
        }
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) units[c] = __reduce_add_sync(0xffffffffu, units[c]);
      if (lane == 0 && warp < kGroups / 32) {
#pragma unroll
        for (int c = 0; c < 8; ++c) reinterpret_cast<int*>(red)[16 + warp * 8 + c] = units[c];
      }
      __syncthreads();
      float best = 3e38f;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const int* r = reinterpret_cast<const int*>(red) + 16 + c;
        const int n = r[0] + r[8];
        if (c > 0 && (cand[c] >= kmax || n > pl.max_units)) continue;
        const float rounds = (float)((n + n_streams - 1) / n_streams);
        const float est = rounds * (float)(cand[c] + (c == 0 ? kOverhead : kSplitOverhead));
        if (est < best) {
          best = est;
          chunk = cand[c];
        }
      }
    }
    int mine = 0;
    if (tid < kGroups && !none) {
      for (int i = 0; i < gsz; ++i) {
        const int d = tid * gsz + i;
        if (d >= p.num_seqs) break;
        Doc o;
        int mt, kt;
        doc_info(p, d, &o);
        doc_tiles<kPair>(p, o, &mt, &kt);
        mine += mt * p.c.n_kv * splits_of(kt, chunk);
      }
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31 && warp < kGroups / 32) reinterpret_cast<int*>(red)[8 + warp] = incl;
    __syncthreads();
    if (tid < kGroups) {
      int before = incl - mine;
      for (int i = 0; i < warp; ++i) before += reinterpret_cast<int*>(red)[8 + i];
      tab[tid] = before;
      if (tid == kGroups - 1) tab[kGroups] = before + mine;
      if (blockIdx.x == 0 && pl.max_units > 0 && !none) {   // for the joining kernel
        for (int i = 0; i < gsz; ++i) {
          const int d = tid * gsz + i;
          if (d >= p.num_seqs) break;
          Doc o;
          int mt, kt;
          doc_info(p, d, &o);
          doc_tiles<kPair>(p, o, &mt, &kt);
          p.doc_base[d] = before;
          before += mt * p.c.n_kv * splits_of(kt, chunk);
        }
      }
    }
    if (tid == 0) {
      ctl[3] = chunk;
      if (blockIdx.x == 0) p.hdr[kAttnHdrChunk] = chunk;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  const uint32_t tmem = (uint32_t)ctl[2];
  const int chunk = ctl[3];
  const int n_units = tab[kGroups];
  const int wg = warp >> 2;
  // Independent streams: all first streams of the grid before the second ones, so few units spread over all SMs.
  auto first_unit = [&](int w) {
    return kPair ? (int)blockIdx.x : w * (int)gridDim.x + (int)blockIdx.x;
  };
  // Independent streams with at most 64 live rows: the second stream's rows are TMEM lanes (and so
  // warps and sub-partitions of the SM) that the first one's do not use.
  const int q_rows = (int)(pl.q_bytes / (D * 2));
  auto first_row = [&](int w) { return !kPair && w == 1 && q_rows <= kAttnRows / 2 ? q_rows : 0; };
  // The query tile of a unit, by one warp (zeros behind its last row).
  auto load_q = [&](const Unit& x, int w) {
    constexpr int PPR = D / 8;
    constexpr int RPP = 32 / PPR;
    const int rows = q_rows;
    const int c = lane % PPR, rsub = lane / PPR;
    const uint32_t qb = sbase + (uint32_t)w * pl.q_bytes + (uint32_t)(c >> 3) * (uint32_t)(rows * 128);
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p.q) + c * 8;
    const int tokens = x.i1 - x.i0;
    const uint16_t* src = q + (int64_t)(x.q0 + x.i0) * p.q_stride + (int64_t)(x.h * p.group) * D;
    int tok = 0, g = rsub;
    for (int r = rsub; r < rows; r += RPP, g += RPP) {
      while (g >= p.group) {
        g -= p.group;
        ++tok;
      }
      const bool there = tok < tokens;
      cp_async16(qb + r * 128 + (((c & 7) ^ (r & 7)) << 4), there ? src + tok * p.q_stride + g * D : q, there);
    }
    cp_arrive(bar_st(w, Q_FULL));
  };

  // Listed keys (or, without a list, all of them) as cache rows, tile by tile, for one warp: position ->
  // page -> row, a step per tile, so that the dependent loads of a tile are spread over the tiles before
  // it.  kRowsPer rows a lane from row row0 of the tile on; use(rows) returns false to give up.
  auto gather = [&](int ring, int row0, auto rows_per, auto use) {
    constexpr int kRowsPer = decltype(rows_per)::value;
    int fu = first_unit(ring), fj = -1;
    Unit fx{};
    struct Step {
      bool live = false;          // holds a tile
      int d = 0, h = 0, lim = 0;  // its sequence, key head, keys visible to the unit
      int u = -1;                 // its unit, where it is the first tile (else -1)
      int v[kRowsPer];            // listed position, then page
      int pos[kRowsPer];
    } s1, s2;
    struct Last {
      bool live = false;
      int u = -1;
      uint32_t row[kRowsPer], sck[kRowsPer], scv[kRowsPer];
    } s3;
    bool bad_page = false;
    auto row_of = [&](int i) { return row0 + i * 32 + lane; };
    auto row_from = [&](const Step& s, int i, uint32_t* row) {
      *row = ~0u;
      if (s.pos[i] >= 0) {
        if ((unsigned)s.v[i] < (unsigned)p.c.num_pages)
          *row = (uint32_t)((((int64_t)s.v[i] * p.c.n_kv + s.h) << p.c.page_shift) +
                            (s.pos[i] & ((1 << p.c.page_shift) - 1)));
        else
          bad_page = true;
      }
    };
    Last out;       // rows (and scales) of the tile furthest on, next to become readable
    auto prepare = [&] {
      if constexpr (Q8) {
        out = s3;
        s3.live = s2.live;
        s3.u = s2.u;
      } else {
        out.live = s2.live;
        out.u = s2.u;
      }
      if (s2.live) {
        Last& l = Q8 ? s3 : out;
#pragma unroll
        for (int i = 0; i < kRowsPer; ++i) {
          row_from(s2, i, &l.row[i]);
          if constexpr (Q8) {
            l.sck[i] = l.scv[i] = 0;
            const uint32_t cr = l.row[i];
            if (cr != ~0u) {
              if (p.c.sw == 1) {
                l.sck[i] = __ldg(p.c.k_scale + cr);
                l.scv[i] = __ldg(p.c.v_scale + cr);
              } else if constexpr (D == 128) {
                l.sck[i] = __ldg(reinterpret_cast<const uint32_t*>(p.c.k_scale) + cr);
                l.scv[i] = __ldg(reinterpret_cast<const uint32_t*>(p.c.v_scale) + cr);
              } else {
                l.sck[i] = __ldg(reinterpret_cast<const uint16_t*>(p.c.k_scale) + cr);
                l.scv[i] = __ldg(reinterpret_cast<const uint16_t*>(p.c.v_scale) + cr);
              }
            }
          }
        }
      }
      // listed positions have arrived: request the pages
      s2 = s1;
      if (s2.live) {
#pragma unroll
        for (int i = 0; i < kRowsPer; ++i) {
          const int pos = s1.v[i];
          s2.pos[i] = pos >= 0 && pos < s2.lim ? pos : -1;
          const int pi = pos >> p.c.page_shift;
          s2.v[i] = s2.pos[i] >= 0 && pi < p.c.max_pages ? __ldg(p.c.table + (int64_t)s2.d * p.c.max_pages + pi) : -1;
        }
      }
      // the next tile enters: request its listed positions
      if (fu < n_units && ++fj >= fx.n_shared) {
        fj = 0;
        if (fx.n_shared > 0) fu += n_streams;   // (0: nothing decoded yet)
        for (; fu < n_units; fu += n_streams) {
          fx = decode_unit<false>(p, tab, gsz, chunk, fu, ring);
          if (fx.n_shared > 0) break;
        }
      }
      s1.live = fu < n_units;
      if (s1.live) {
        s1.d = fx.d;
        s1.u = fj == 0 ? fu : -1;
        s1.h = fx.h;
        s1.lim = fx.P0 + (p.topk_idx ? fx.i0 + 1 : fx.last);   // keys behind the last visible one are never read
#pragma unroll
        for (int i = 0; i < kRowsPer; ++i) {
          const int j = (fx.lo + fj) * kAttnKeys + row_of(i);
          s1.v[i] = j;
          if (p.topk_idx)
            s1.v[i] = j < fx.n_list ? __ldg(p.topk_idx + (int64_t)(fx.q0 + fx.i0) * p.topk_width + j) : -1;
        }
      }
    };
    prepare();
    prepare();
    prepare();
    if constexpr (Q8) prepare();
    while (out.live && use(out)) prepare();
    if (bad_page) set_status(status, DSA_DEV_ERR_INVALID_ARG);
  };

  if (R::kWorkWarps > 0 && wg >= 2 && wg < 2 + R::kWorkWarps / 4) {
    // ======================= workers =======================
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::kWorkRegs));
    const int ring = kRings == 1 ? 0 : (tid - 256) / kLoaders, team = kTeams == 1 ? 0 : (tid - 256) / kLoaders;
    const int lt = (tid - 256) % kLoaders;           // thread of this team
    const uint32_t ring_base = sbase + pl.off_ring + (uint32_t)ring * pl.nst * kStage;
    bool ok = true;
    int st = team;          // (at least two stages and stored tiles to a ring of two teams)
    uint32_t ph = 0;
    bool wrapped = false;   // every stage has been used once
    auto advance = [&] {
      st += kTeams;
      if (st >= pl.nst) {
        st -= pl.nst;
        ph ^= 1u;
        wrapped = true;
      }
    };
    if constexpr (Q8) {
      // Stored tiles (keys, values, keys, ...) to BF16 stages.
      constexpr int PPR = D / 16;                  // 16-code pieces per row
      constexpr int RPP = kLoaders / PPR;
      constexpr int kPasses = (kAttnKeys + RPP - 1) / RPP;   // (12 workers: the last pass is not whole)
      // (of two neighbouring rows, one's first half beside the other's second in eight lanes: a 64-column
      // chunk's pieces of one row alone would be 2-way bank conflicts of the stores)
      const int c = lt % PPR, rsub = D == 128 ? ((lt / PPR) & ~1) | (((lt / PPR) ^ (c >> 2)) & 1) : lt / PPR;
      const uint32_t raw_base = sbase + pl.off_raw + (uint32_t)ring * pl.nraw * kRawItem + rsub * D + c * 16;
      const int* const meta = reinterpret_cast<const int*>(smem + pl.off_rows) + ring * 8;
      const uint32_t dcol = (uint32_t)(c >> 2) * kChunk + rsub * 128;
      // the two 16-byte pieces in their 128-byte span (a pass is a multiple of 8 rows)
      static_assert(!Q8 || RPP % 8 == 0, "swizzle");
      const uint32_t at0 = dcol + ((uint32_t)(((c & 3) * 2) ^ (rsub & 7)) << 4), at1 = at0 ^ 16u;
      const int sw = p.c.sw, s0 = rsub * sw + (sw == 1 ? 0 : c >> 1);
      int slot = team;
      uint32_t rph = 0;
      for (int u = first_unit(ring); u < n_units && ok; u += n_streams) {
        const int n = decode_unit<kPair>(p, tab, gsz, chunk, u, kPair ? 0 : ring).n_shared;
        for (int it = team; it < 2 * n; it += kTeams) {
          ok = __all_sync(0xffffffffu, wait_bar(bar_raw_full(ring, slot), rph, abort_flag, status, tmo) &&
                                           (!wrapped || wait_bar(bar_empty(ring, st), ph ^ 1u, abort_flag, status, tmo)));
          if (!ok) break;
          const uint32_t raw = raw_base + (uint32_t)slot * kRawItem;
          const uint8_t* scales = smem + pl.off_raw + (size_t)(ring * pl.nraw + slot) * kRawItem + kAttnKeys * D + s0;
          const int valid = meta[slot] - rsub;
          const uint32_t dst = ring_base + (uint32_t)st * kStage;
          uint32_t top = 0;   // of the tile's scales
          constexpr int kBatch = kPasses % 4 == 0 ? 4 : (kPasses % 2 == 0 ? 2 : 1);   // passes whose loads go first
#pragma unroll
          for (int i0 = 0; i0 < kPasses; i0 += kBatch) {
            uint32_t w4[kBatch][4], e8[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              if (kAttnKeys % RPP == 0 || (i0 + i) * RPP + rsub < kAttnKeys) {
                ld_shared_v4(raw + (i0 + i) * RPP * D, w4[i]);
                e8[i] = scales[(i0 + i) * RPP * sw];
              }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              if (kAttnKeys % RPP != 0 && (i0 + i) * RPP + rsub >= kAttnKeys) break;
              uint32_t o[8];
              if ((i0 + i) * RPP >= valid) {   // nothing of the page's other slots
                e8[i] = 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) w4[i][q] = 0;
              }
              top = max(top, e8[i]);
              widen16<false>(w4[i], e8[i], o);
              st_shared_v4(dst + at0 + (i0 + i) * RPP * 128, o[0], o[1], o[2], o[3]);
              st_shared_v4(dst + at1 + (i0 + i) * RPP * 128, o[4], o[5], o[6], o[7]);
            }
          }
          // Far scales once more, in a loop of its own: as code of every unrolled pass it cost all tiles
          // (a token of each of 64 sequences over MXFP8 441 against 416 us).
          if (top > 134u) {
#pragma unroll 1
            for (int r = 0; r < kAttnKeys - rsub; r += RPP) {
              const uint32_t e = scales[r * sw];
              if (e <= 134u || r >= valid) continue;
              uint32_t w4[4], o[8];
              ld_shared_v4(raw + r * D, w4);
              widen16<true>(w4, e, o);
              st_shared_v4(dst + at0 + r * 128, o[0], o[1], o[2], o[3]);
              st_shared_v4(dst + at1 + r * 128, o[4], o[5], o[6], o[7]);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_raw_empty(ring, slot));
          slot += kTeams;
          if (slot >= pl.nraw) {
            slot -= pl.nraw;
            rph ^= 1u;
          }
          // (one arrival a warp: 32 lanes' arrivals at one barrier are worked off one after the other)
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_full(ring, st));
          advance();
        }
      }
    } else {
      // BF16 rows copied one by one; a warp brings a quarter of a tile.
      constexpr int PPR = D / 8;                   // 16-byte pieces per row
      constexpr int RPP = 32 / PPR;                // rows per pass
      const int wq = lt >> 5, c = lane % PPR, rsub = lane / PPR;
      const uint32_t dcol = (uint32_t)(c >> 3) * kChunk + (wq * 32 + rsub) * 128;
      int t = 0;
      gather(ring, wq * 32, std::integral_constant<int, 1>{}, [&](const auto& out) {
        const uint32_t seen = __ballot_sync(0xffffffffu, out.row[0] != ~0u);
        if (lane == 0) reinterpret_cast<uint32_t*>(smem + pl.off_mask)[(ring * kMaskRing + t % kMaskRing) * 4 + wq] = seen;
        for (int kv = 0; kv < 2; ++kv) {
          if (wrapped) ok = __all_sync(0xffffffffu, wait_bar(bar_empty(ring, st), ph ^ 1u, abort_flag, status, tmo));
          if (!ok) return false;
          const uint32_t dst = ring_base + (uint32_t)st * kStage + dcol;
          const uint16_t* src = reinterpret_cast<const uint16_t*>(kv ? p.c.v : p.c.k) + c * 8;
#pragma unroll
          for (int i = 0; i < 32; i += RPP) {
            const uint32_t e = __shfl_sync(0xffffffffu, out.row[0], i + rsub);
            const bool there = e != ~0u;
            cp_async16(dst + i * 128 + (((c & 7) ^ ((i + rsub) & 7)) << 4), src + (size_t)(there ? e : 0) * D, there);
          }
          if (p.fault_inject != 1 || t > 0 || kv > 0) {   // (the tests' withheld first stage)
            if (lane == 0) mbar_arrive(bar_full(ring, st));   // the mask
            cp_arrive(bar_full(ring, st));                    // the rows, when they have landed
          }
          advance();
        }
        ++t;
        return true;
      });
      cp_wait_all();
    }
  } else if (R::kBringWarps > 0 && wg >= 2 && wg < 2 + (R::kWorkWarps + R::kBringWarps) / 4) {
    // ======================= gathered rows of an 8-bit cache, as stored =======================
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::kBringRegs));
    const int ring = (warp >> 1) & 1, part = warp & 1;   // two warps to a ring, half a tile each
    constexpr int PPR = D / 16;                          // 16-byte pieces per row
    constexpr int RPP = 32 / PPR;                        // rows per pass
    const int c = lane % PPR, rsub = lane / PPR;
    const uint32_t raw_base = sbase + pl.off_raw + (uint32_t)ring * pl.nraw * kRawItem;
    int* const meta = reinterpret_cast<int*>(smem + pl.off_rows) + ring * 8;
    uint32_t* const masks = reinterpret_cast<uint32_t*>(smem + pl.off_mask) + ring * kMaskRing * 4 + part * 2;
    int slot = 0, t = 0;
    uint32_t rph = 0;
    bool wrapped = false;
    gather(ring, part * 64, std::integral_constant<int, 2>{}, [&](const auto& out) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t seen = __ballot_sync(0xffffffffu, out.row[i] != ~0u);
        if (lane == 0) masks[(t % kMaskRing) * 4 + i] = seen;
      }
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        if (wrapped && !__all_sync(0xffffffffu, wait_bar(bar_raw_empty(ring, slot), rph ^ 1u, abort_flag, status, tmo)))
          return false;
        const uint32_t bar = bar_raw_full(ring, slot), dst = raw_base + (uint32_t)slot * kRawItem;
        uint8_t* sc = smem + (dst - sbase) + kAttnKeys * D;
        const uint8_t* src = reinterpret_cast<const uint8_t*>(kv ? p.c.v : p.c.k) + c * 16;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = part * 64 + i * 32 + lane;
          const uint32_t e = kv ? out.scv[i] : out.sck[i];
          if (p.c.sw == 1) sc[r] = (uint8_t)e;
          else if constexpr (D == 128) reinterpret_cast<uint32_t*>(sc)[r] = e;
          else reinterpret_cast<uint16_t*>(sc)[r] = (uint16_t)e;
#pragma unroll 4
          for (int g = 0; g < 32; g += RPP) {
            const uint32_t cr = __shfl_sync(0xffffffffu, out.row[i], g + rsub);
            const bool there = cr != ~0u;
            cp_async16(dst + (part * 64 + i * 32 + g + rsub) * D + c * 16, src + (size_t)(there ? cr : 0) * D, there);
          }
        }
        if (part == 0 && lane == 0) meta[slot] = kAttnKeys;
        if (p.fault_inject != 1 || t > 0 || kv > 0) {   // (the tests' withheld first tile)
          __syncwarp();
          if (lane == 0) mbar_arrive(bar);   // the scales
          cp_arrive(bar);                    // the codes, when they have landed
        }
        if (++slot == pl.nraw) {
          slot = 0;
          rph ^= 1u;
          wrapped = true;
        }
      }
      ++t;
      return true;
    });
    cp_wait_all();
  } else if (wg >= 2) {
    // ======================= loaders and MMA =======================
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::kAuxRegs));
    // Every visible key of a BF16 cache: TMA, a box per page, issued by one warp.  The unit's last
    // tile may end inside a page whose other slots hold anything: the warp copies that one row by
    // row, with zeros behind the last visible key.
    // After an abort a loader waits (again with a limit) for the copies it has in flight: the last use
    // of every stage, those from st on being of the round before.
    auto drain_ring = [&](auto bar, int ring, int count, int st, uint32_t ph, bool wrapped) {
      if (lane == 0) {
        for (int s = 0; s < (wrapped ? count : st); ++s) drain_wait(bar(ring, s), s < st ? ph : ph ^ 1u, tmo);
      }
      __syncwarp();
    };
    auto load_tma = [&](int ring) {
      const uint32_t ring_base = sbase + pl.off_ring + (uint32_t)ring * pl.nst * kStage;
      const int shift = p.c.page_shift;
      const int box = min(kAttnKeys, 1 << shift);               // keys per box
      const int boxes = kAttnKeys / box;
      int st = 0;
      uint32_t ph = 0;
      bool wrapped = false, bad_page = false;
      for (int u = first_unit(ring); u < n_units; u += n_streams) {
        const Unit x = decode_unit<kPair>(p, tab, gsz, chunk, u, kPair ? 0 : ring);
        const int32_t* table = p.c.table + (int64_t)x.d * p.c.max_pages;
        const int last = x.P0 + x.last;                         // keys visible to the unit
        auto page_of = [&](int key) {
          return key < last ? __ldg(table + (key >> shift)) : 0;   // (doc_info: within max_pages)
        };
        int page = x.n_shared > 0 && lane < boxes ? page_of(x.lo * kAttnKeys + lane * box) : 0;
        for (int j = 0; j < x.n_shared; ++j) {
          const int key0 = (x.lo + j) * kAttnKeys;
          const int now = page;
          if (j + 1 < x.n_shared && lane < boxes) page = page_of(key0 + kAttnKeys + lane * box);
          const bool whole = key0 + kAttnKeys <= last;
          const bool good = (unsigned)now < (unsigned)p.c.num_pages;
          const bool mine = whole && lane < boxes && good;
          const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, mine)) * (uint32_t)box * D * 2;
          if (whole && lane < boxes && !good) bad_page = true;
          for (int kv = 0; kv < 2; ++kv) {
            if (wrapped && !__all_sync(0xffffffffu, wait_bar(bar_empty(ring, st), ph ^ 1u, abort_flag, status, tmo))) {
              drain_ring(bar_full, ring, pl.nst, st, ph, wrapped);
              return;
            }
            const uint32_t dst = ring_base + (uint32_t)st * kStage;
            const bool withheld = p.fault_inject == 1 && u == first_unit(ring) && j == 0 && kv == 0;   // (tests)
            if (whole) {
              if (!withheld) {
                if (lane == 0) mbar_arrive_expect_tx(bar_full(ring, st), bytes);
#pragma unroll 1
                for (int i = 0; i < boxes; ++i) {   // (one lane and uniform coordinates: a lane to a box issues slower)
                  const int pg = __shfl_sync(0xffffffffu, now, i);
                  if ((unsigned)pg < (unsigned)p.c.num_pages && elect_one()) {
                    const int slot = (key0 + i * box) & ((1 << shift) - 1), z = pg * p.c.n_kv + x.h;
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
                      tma_load_3d(dst + c * kChunk + i * box * 128, kv ? &p.tm_v : &p.tm_k, bar_full(ring, st), c * 64, slot, z);
                  }
                }
              }
            } else {
              constexpr int PPR = D / 8;
              const int c = lane % PPR;
              const uint16_t* src = reinterpret_cast<const uint16_t*>(kv ? p.c.v : p.c.k) + c * 8;
#pragma unroll 4
              for (int r = lane / PPR; r < kAttnKeys; r += 32 / PPR) {
                const int64_t cr = key0 + r < last ? cache_row(p.c, x.d, key0 + r, x.h) : -1;
                if (key0 + r < last && cr < 0) bad_page = true;
                cp_async16(dst + (uint32_t)(c >> 3) * kChunk + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                           src + (cr < 0 ? 0 : cr * D), cr >= 0);
              }
              cp_wait_all();
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0 && !withheld) mbar_arrive(bar_full(ring, st));
            }
            if (++st == pl.nst) {
              st = 0;
              ph ^= 1u;
              wrapped = true;
            }
          }
        }
      }
      if (*abort_flag) drain_ring(bar_full, ring, pl.nst, st, ph, wrapped);
      if (bad_page) set_status(status, DSA_DEV_ERR_INVALID_ARG);
    };
    // Every visible key of an 8-bit cache, as stored: tiles of codes (a TMA box per page) and their
    // scales (a bulk copy per page); the workers learn how many rows of a tile are visible.  The
    // stream's query tile is loaded on the way.
    auto load_raw = [&](int ring) {
      const uint32_t raw_base = sbase + pl.off_raw + (uint32_t)ring * pl.nraw * kRawItem;
      int* const meta = reinterpret_cast<int*>(smem + pl.off_rows) + ring * 8;
      const int shift = p.c.page_shift, sw = p.c.sw;
      const int box = min(kAttnKeys, 1 << shift), boxes = kAttnKeys / box;
      int slot = 0;
      uint32_t rph = 0, nq = 0;
      bool wrapped = false, bad_page = false;
      for (int u = first_unit(ring); u < n_units; u += n_streams) {
        const Unit x = decode_unit<kPair>(p, tab, gsz, chunk, u, kPair ? 0 : ring);
        const int32_t* table = p.c.table + (int64_t)x.d * p.c.max_pages;
        const int last = x.P0 + x.last;                         // keys visible to the unit
        auto page_of = [&](int key) {
          return key < last ? __ldg(table + (key >> shift)) : -1;   // (doc_info: within max_pages)
        };
        int page = x.n_shared > 0 && lane < boxes ? page_of(x.lo * kAttnKeys + lane * box) : 0;
        for (int j = 0; j < x.n_shared; ++j) {
          const int key0 = (x.lo + j) * kAttnKeys;
          const int now = page;
          if (j + 1 < x.n_shared && lane < boxes) page = page_of(key0 + kAttnKeys + lane * box);
          const bool good = (unsigned)now < (unsigned)p.c.num_pages;
          if (lane < boxes && key0 + lane * box < last && !good) bad_page = true;
          const uint32_t have = __ballot_sync(0xffffffffu, lane < boxes && good);
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv) {
            if (wrapped &&
                !__all_sync(0xffffffffu, wait_bar(bar_raw_empty(ring, slot), rph ^ 1u, abort_flag, status, tmo))) {
              cp_wait_all();
              drain_ring(bar_raw_full, ring, pl.nraw, slot, rph, wrapped);
              return;
            }
            const uint32_t bar = bar_raw_full(ring, slot), dst = raw_base + (uint32_t)slot * kRawItem;
            const bool withheld = p.fault_inject == 1 && u == first_unit(ring) && j == 0 && kv == 0;   // (tests)
            if (lane == 0 && !withheld) {
              meta[slot] = min(kAttnKeys, last - key0);
              mbar_arrive_expect_tx(bar, __popc(have) * (uint32_t)(box * (D + sw)));
            }
            const uint8_t* sc = kv ? p.c.v_scale : p.c.k_scale;
#pragma unroll 1
            for (int i = 0; i < boxes; ++i) {   // (one lane and uniform coordinates: a lane to a box issues slower)
              const int pg = __shfl_sync(0xffffffffu, now, i);
              if (!withheld && ((have >> i) & 1u) && elect_one()) {
                const int in_page = (key0 + i * box) & ((1 << shift) - 1), z = pg * p.c.n_kv + x.h;
                tma_load_3d(dst + i * box * D, kv ? &p.tm_v : &p.tm_k, bar, 0, in_page, z);
                bulk_load(dst + kAttnKeys * D + i * box * sw, sc + ((((int64_t)z << shift) + in_page) * sw), box * sw, bar);
              }
            }
            if (++slot == pl.nraw) {
              slot = 0;
              rph ^= 1u;
              wrapped = true;
            }
          }
          if (!kPair && j == 0) {
            if (nq > 0 &&
                !__all_sync(0xffffffffu, wait_bar(bar_st(ring, Q_EMPTY), (nq - 1) & 1u, abort_flag, status, tmo))) {
              cp_wait_all();
              drain_ring(bar_raw_full, ring, pl.nraw, slot, rph, wrapped);
              return;
            }
            ++nq;
            load_q(x, ring);
          }
        }
      }
      cp_wait_all();
      if (*abort_flag) drain_ring(bar_raw_full, ring, pl.nraw, slot, rph, wrapped);
      if (bad_page) set_status(status, DSA_DEV_ERR_INVALID_ARG);
    };
    // Query tiles of streams w0 .. w1 - 1, each as soon as its stream's last product with the one before is done.
    auto load_queries = [&](int w0, int w1) {
      uint32_t nq[2] = {0, 0};
      for (int u = first_unit(w0); u < n_units; u += n_streams) {
        for (int w = w0; w < w1; ++w) {
          const Unit x = decode_unit<kPair>(p, tab, gsz, chunk, u, w);
          if (x.n == 0) continue;
          if (nq[w - w0] > 0 && !__all_sync(0xffffffffu, mbar_wait(bar_st(w, Q_EMPTY), (nq[w - w0] - 1) & 1u, abort_flag,
                                                                    status, tmo))) {
            cp_wait_all();
            return;
          }
          ++nq[w - w0];
          load_q(x, w);
        }
      }
      cp_wait_all();
    };
    if (warp < kMmaWarp) {
      if constexpr (MODE != GATHER && Q8) {
        if (warp == R::kKeyWarp) load_raw(0);
        else if (warp == R::kKeyWarp + 1 && kPair) load_queries(0, 2);
        else if (warp == R::kKeyWarp + 1) load_raw(1);
      } else {
        if (MODE != GATHER && warp >= R::kKeyWarp && warp < R::kKeyWarp + kRings) load_tma(warp - R::kKeyWarp);
        else if (warp == R::kQueryWarp) load_queries(0, 1);
        else if (warp == R::kQueryWarp + 1) load_queries(1, 2);
      }
      __syncwarp();
    } else {
      const int w = warp - kMmaWarp;
      const int ring = kPair ? 0 : w;
      const uint32_t ring_base = sbase + pl.off_ring + (uint32_t)ring * pl.nst * kStage;
      if constexpr (NARROW) {
        // S^T = K Q^T into one of two buffers, O^T += V^T P^T with P from shared memory: the next tile's
        // S^T is formed while the softmax warps are at this one.
        constexpr int N = kAttnNarrow;
        const uint32_t t_s = tmem + (uint32_t)w * 2 * N, t_o = tmem + 4 * N + (uint32_t)w * N;
        constexpr uint32_t idesc_qk = idesc_bf16(kAttnKeys, N);
        constexpr uint32_t idesc_pv = idesc_bf16(D, N) | (1u << 15);   // V: rows of keys, M contiguous
        if (elect_one()) {
          const uint64_t qd0 = sw128_kmajor_desc(sbase + (uint32_t)w * pl.q_bytes, 0);
          const uint64_t pd0 = sw128_kmajor_desc(sbase + pl.off_p + (uint32_t)w * 2 * kAttnNarrowP, 0);
          int st[2] = {0, 1};   // stage and phase of the next keys and of the next values
          uint32_t ph[2] = {0, 0}, nq = 0, nt = 0;
          bool ok = true;
          auto advance = [&](int i) {
            st[i] += 2;
            if (st[i] >= pl.nst) {
              st[i] -= pl.nst;
              ph[i] ^= 1u;
            }
          };
          for (int u = first_unit(w); u < n_units && ok; u += n_streams) {
            const Unit x = decode_unit<false>(p, tab, gsz, chunk, u, w);
            if (x.n == 0) continue;
            ok = wait_bar(bar_st(w, Q_FULL), nq & 1u, abort_flag, status, tmo);
            if (!ok) break;
            ++nq;
            // Whichever product's operands are there: S^T of tile jk (P of tile jk - 2 has been waited for,
            // so that buffer's S^T is read), PV of tile jv.
            int jk = 0, jv = 0;
            uint32_t polls = 0;
            uint64_t t0 = 0;
            while (jv < x.n) {
              const uint32_t t = nt + jv, bv = t & 1u, bk = (nt + jk) & 1u;
              if (jk < x.n && jk <= jv + 1 && test_bar(bar_full(ring, st[0]), ph[0])) {
                fence_proxy_async_smem();   // cp.async's writes (query tile, copied rows), seen through the barriers
                tc_fence_after();
                uint64_t qd = qd0, kd = sw128_kmajor_desc(ring_base + (uint32_t)st[0] * kStage, 0);
#pragma unroll
                for (int c = 0; c < D / 64; ++c, qd += (N * 128) >> 4, kd += kChunk >> 4) {
#pragma unroll
                  for (int k = 0; k < 4; ++k) mma_bf16(t_s + bk * N, kd + 2 * k, qd + 2 * k, idesc_qk, c + k > 0);
                }
                tc_commit(bar_st(w, S_FULL + bk));
                tc_commit(bar_empty(ring, st[0]));
                if (++jk == x.n) tc_commit(bar_st(w, Q_EMPTY));
                advance(0);
                polls = 0;
              } else if (jv < jk && test_bar(bar_st(w, P_FULL + bv), (t >> 1) & 1u) &&
                         test_bar(bar_full(ring, st[1]), ph[1])) {
                if (kWorkerCopies) fence_proxy_async_smem();
                tc_fence_after();
                uint64_t vd = smem_desc(ring_base + (uint32_t)st[1] * kStage, kChunk, 1024, 2), pd = pd0 + bv * (kAttnNarrowP >> 4);
#pragma unroll
                for (int k = 0; k < kAttnKeys / 16; ++k, vd += 2048 >> 4)
                  mma_bf16(t_o, vd, pd + (k >> 2) * ((N * 128) >> 4) + (k & 3) * 2, idesc_pv, (jv > 0 || k > 0) ? 1u : 0u);
                tc_commit(bar_empty(ring, st[1]));
                tc_commit(bar_st(w, P_EMPTY + bv));
                if (++jv == x.n) tc_commit(bar_st(w, O_FULL));
                advance(1);
                polls = 0;
              } else if ((++polls & 1023u) == 0) {   // bounded, as wait_bar
                if (polls == 1024u) t0 = globaltimer_ns();
                if (*abort_flag) {
                  ok = false;
                } else if (globaltimer_ns() - t0 > tmo) {
                  set_status(status, DSA_DEV_ERR_TIMEOUT);
                  *abort_flag = 1;
                  ok = false;
                }
                if (!ok) break;
              }
            }
            nt += x.n;
          }
          if (!ok) {   // what was issued completes before the tensor memory is given back
            tc_commit(bar_st(w, DRAIN));
            drain_wait(bar_st(w, DRAIN), 0, tmo);
          }
        }
      } else {
        // ---- tiles of 128 query rows ----
        const uint32_t t_s = tmem + (uint32_t)w * 128, t_o = tmem + 256 + (uint32_t)w * 128;
        constexpr uint32_t idesc_qk = idesc_bf16(kAttnRows, kAttnKeys);
        constexpr uint32_t idesc_pv = idesc_bf16(kAttnRows, D) | (1u << 16);   // V: rows of keys, N contiguous
        if (elect_one()) {
          const uint32_t q_rows_bytes = pl.q_bytes / (D / 64);   // one 64-column chunk of the query tile
          // The streams issue PV and the next QK as one block, in turns, so that one's softmax runs beside
          // the other's products: a token of each of 64 sequences over MXFP8 415 against 434 us, ragged
          // chunks over FP8 492 against 495, 4096 tokens over 32768 BF16 keys 2.87 against 2.88 ms.  (Gathered
          // rows take the same time either way.)
          // Nothing is waited for inside a turn, so a turn always comes; only the times depend on it.
          constexpr bool kTurns = MODE != GATHER;
          int* const turn = ctl + 4;
          auto take_turn = [&] {
            for (int i = 0; kTurns && i < (1 << 20) && atomicCAS_block(turn, 0, 1) != 0; ++i) {
            }
          };
          auto end_turn = [&] {
            if (kTurns) atomicExch_block(turn, 0);
          };
          // (the 128 rows that the products read begin before the tile when its rows are not the first:
          // with 32 or 64 rows a tile, still inside the first stream's)
          const uint64_t qd0 = sw128_kmajor_desc(sbase + (uint32_t)w * pl.q_bytes - first_row(w) * 128, 0);
          int st = 0;
          uint32_t ph = 0, nq = 0, nt = 0;
          bool ok = true;
          auto advance = [&] {
            if (++st == pl.nst) {
              st = 0;
              ph ^= 1u;
            }
          };
          for (int u = first_unit(w); u < n_units && ok; u += n_streams) {
            const Unit x = decode_unit<kPair>(p, tab, gsz, chunk, u, w);
            if (x.n > 0) {
              ok = wait_bar(bar_st(w, Q_FULL), nq & 1u, abort_flag, status, tmo);
              fence_proxy_async_smem();   // the query tile's cp.async writes
            }
            // iteration j: O += P V of tile j - 1, S = Q K^T of tile j
#pragma unroll 1
            for (int j = 0; x.n > 0 && j <= x.n; ++j) {
              const bool next = j < x.n;
              bool have_k = false;
              if (j > 0) {
                // everything but P is waited for first
                ok = wait_bar(bar_full(ring, st), ph, abort_flag, status, tmo);
                if (!ok) break;
                // N-major operand: 64-column chunks kChunk apart, groups of 8 keys 1024 bytes apart
                uint64_t vd = smem_desc(ring_base + (uint32_t)st * kStage, kChunk, 1024, 2);
                const uint32_t v_empty = bar_empty(ring, st);
                advance();
                have_k = next && test_bar(bar_full(ring, st), ph);
                if (kWorkerCopies) fence_proxy_async_smem();   // the workers' cp.async writes, seen through the barriers
                // (P of a unit's first tile also says that the softmax warps have read the last unit's O)
                ok = wait_bar(bar_st(w, P_FULL), nt & 1u, abort_flag, status, tmo);
                if (!ok) break;
                ++nt;
                if (next && !have_k) {   // once more: the next QK in this turn
                  have_k = test_bar(bar_full(ring, st), ph);
                  if (kWorkerCopies && have_k) fence_proxy_async_smem();
                }
                tc_fence_after();
                take_turn();
#pragma unroll
                for (int k = 0; k < kAttnKeys / 16; ++k, vd += 2048 >> 4)
                  mma_bf16_ts(t_o, t_s + k * 8, vd, idesc_pv, (j > 1 || k > 0) ? 1u : 0u);
                tc_commit(v_empty);
                if (!next) tc_commit(bar_st(w, O_FULL));
              }
              if (next) {
                if (!have_k) {
                  if (j > 0) end_turn();
                  ok = wait_bar(bar_full(ring, st), ph, abort_flag, status, tmo);
                  if (!ok) break;
                  if (kWorkerCopies) fence_proxy_async_smem();
                  tc_fence_after();
                  take_turn();
                }
                uint64_t qd = qd0, kd = sw128_kmajor_desc(ring_base + (uint32_t)st * kStage, 0);
#pragma unroll
                for (int c = 0; c < D / 64; ++c, qd += q_rows_bytes >> 4, kd += kChunk >> 4) {
#pragma unroll
                  for (int k = 0; k < 4; ++k) mma_bf16(t_s, qd + 2 * k, kd + 2 * k, idesc_qk, c + k > 0);   // 32 bytes a step
                }
                tc_commit(bar_st(w, S_FULL));
                tc_commit(bar_empty(ring, st));
                if (j + 1 == x.n) tc_commit(bar_st(w, Q_EMPTY));
                advance();
              }
              end_turn();
            }
            if (x.n > 0) ++nq;
            if constexpr (kPair) {   // stages only the other stream needs
              for (int j = 2 * x.n; j < 2 * x.n_shared && ok; ++j) {
                ok = wait_bar(bar_full(ring, st), ph, abort_flag, status, tmo);
                if (ok) mbar_arrive(bar_empty(ring, st));
                advance();
              }
            }
          }
          if (!ok) {   // what was issued completes before the tensor memory is given back
            tc_commit(bar_st(w, DRAIN));
            drain_wait(bar_st(w, DRAIN), 0, tmo);
          }
        }
      }
      __syncwarp();
    }
  } else if constexpr (NARROW) {
    // ======================= softmax warpgroups, a key to a thread =======================
    // The rows' maxima are the block's: the warpgroup votes whether a logit exceeds its row's, and raises
    // them together.  Whatever a warp has waited for in vain, it takes part in every vote: all leave at one.
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R::kSoftmaxRegs));
    constexpr int N = kAttnNarrow;
    const int w = wg, quarter = warp & 3, key = quarter * 32 + lane, bar_id = 1 + w;
    const uint32_t lane_off = (uint32_t)quarter << 21;    // TMEM lane 32 * quarter
    const uint32_t t_s = tmem + (uint32_t)w * 2 * N + lane_off, t_o = tmem + 4 * N + (uint32_t)w * N + lane_off;
    float* const m_tab = reinterpret_cast<float*>(smem + pl.off_red) + w * 9 * N;   // running maximum of each row
    float* const m_of = m_tab + N;                                                  // [4][N] a warp's maxima
    float* const l_of = m_tab + 5 * N;                                              // [4][N] a warp's sums
    const uint32_t* const masks = reinterpret_cast<const uint32_t*>(smem + pl.off_mask) + w * kMaskRing * 4;
    // this key's 2 bytes of each row of P (K-major, 64 keys to a 128-byte row, swizzled)
    const uint32_t p_at = sbase + pl.off_p + (uint32_t)w * 2 * kAttnNarrowP + (uint32_t)(key >> 6) * (N * 128) + (key & 7) * 2;
    const uint32_t piece = (key & 63) >> 3;
    const float scale = p.scale_log2;
    constexpr int kLanesPerRow = 32 / N;
    uint32_t nt = 0, nq = 0;
    bool ok = true;
    Unit x{}, nx{};
    if (first_unit(w) < n_units) x = decode_unit<false>(p, tab, gsz, chunk, first_unit(w), w);
    for (int u = first_unit(w); u < n_units && ok; u += n_streams, x = nx) {
      const int live = (x.i1 - x.i0) * p.group;
      const int vis0 = x.P0 + x.i0 + 1;   // keys that the first token sees
      float l[N];
#pragma unroll
      for (int r = 0; r < N; ++r) l[r] = 0.f;
      if (x.n > 0) {
        any_of_128(bar_id, false);        // (the last unit's maxima and sums have been read)
        if (key < N) m_tab[key] = key < live ? -INFINITY : INFINITY;
        any_of_128(bar_id, false);
      }
      for (int j = 0; j < x.n; ++j, ++nt) {
        const uint32_t b = nt & 1u;
        if (ok) ok = __all_sync(0xffffffffu, wait_bar(bar_st(w, S_FULL + b), (nt >> 1) & 1u, abort_flag, status, tmo));
        float s[N];
        bool over = false;
        if (ok) {
          tc_fence_after();
          uint32_t raw[N];
          tmem_ld_x16(t_s + b * N, raw);
          tmem_ld_wait_tied<N>(raw);
          const int at = (x.lo + j) * kAttnKeys + key;
          const bool hidden = listed ? ((masks[(nt % kMaskRing) * 4 + quarter] >> lane) & 1u) == 0 : false;
          if (__any_sync(0xffffffffu, hidden || (!listed && at >= vis0))) {
            int tok = 0, g = 0;
#pragma unroll
            for (int r = 0; r < N; ++r) {
              if (hidden || (!listed && at >= vis0 + tok)) raw[r] = 0xFF800000u;
              if (++g == p.group) {
                g = 0;
                ++tok;
              }
            }
          }
#pragma unroll
          for (int r = 0; r < N; ++r) s[r] = __uint_as_float(raw[r]);
#pragma unroll
          for (int r = 0; r < N; ++r) {
            if (r % 8 == 0 && r >= live) break;
            over |= s[r] * scale > m_tab[r] + kRaise;   // (rows that are not live: never)
          }
        }
        if (any_of_128(bar_id, over || !ok)) {
          if (ok) {
            float v[N];
#pragma unroll
            for (int r = 0; r < N; ++r) v[r] = s[r];
            const float mx = warp_join<N>(v, lane, [](float a, float c) { return fmaxf(a, c); });
            if (lane % kLanesPerRow == 0) m_of[quarter * N + lane / kLanesPerRow] = mx;
            if (j > 0)   // O so far
              ok = __all_sync(0xffffffffu, wait_bar(bar_st(w, P_EMPTY + (b ^ 1u)), ((nt - 1) >> 1) & 1u, abort_flag, status, tmo));
          }
          ok = !any_of_128(bar_id, !ok);
          if (!ok) break;
          float alpha[N], mine = 0.f;
#pragma unroll
          for (int r = 0; r < N; ++r) {
            const float top = fmaxf(fmaxf(m_of[r], m_of[N + r]), fmaxf(m_of[2 * N + r], m_of[3 * N + r]));
            const float mt = top == -INFINITY ? -INFINITY : top * scale, m = m_tab[r];
            const bool raise = mt > m + kRaise;
            alpha[r] = raise ? ex2(m - mt) : 1.f;      // 0 when m = -inf
            l[r] *= alpha[r];
            if (r == key) mine = raise ? mt : m;
          }
          if (j > 0) {
            tc_fence_after();
            uint32_t o[N];
            tmem_ld_x16(t_o, o);
            tmem_ld_wait_tied<N>(o);
#pragma unroll
            for (int r = 0; r < N; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * alpha[r]);
            tmem_st_x16(t_o, o);
            tmem_st_wait();
          }
          any_of_128(bar_id, false);
          if (key < N) m_tab[key] = mine;
          any_of_128(bar_id, false);
        }
        if (nt >= 2)
          ok = __all_sync(0xffffffffu, wait_bar(bar_st(w, P_EMPTY + b), ((nt >> 1) - 1u) & 1u, abort_flag, status, tmo));
        if (ok) {
#pragma unroll
          for (int r = 0; r < N; ++r) {
            if (r % 8 == 0 && r >= live) break;   // (columns of the product that nobody reads)
            const float m = m_tab[r];
            s[r] = ex2(fmaf(s[r], scale, m == -INFINITY ? 0.f : -m));   // (m = inf where no row is live: 0)
            l[r] += s[r];
          }
#pragma unroll
          for (int r = 0; r < N; ++r) {
            if (r % 8 == 0 && r >= live) break;
            st_shared_u16(p_at + b * kAttnNarrowP + (r >> 3) * 1024 + (r & 7) * 128 + ((piece ^ (r & 7)) << 4), bf16_bits(s[r]));
          }
          fence_proxy_async_smem();
          tc_fence_before();
        }
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(bar_st(w, P_FULL + b));
      }
      if (u + n_streams < n_units) nx = decode_unit<false>(p, tab, gsz, chunk, u + n_streams, w);   // (while O is formed)
      uint32_t o[N];
      if (x.n > 0) {
        if (ok) ok = __all_sync(0xffffffffu, wait_bar(bar_st(w, O_FULL), nq & 1u, abort_flag, status, tmo));
        ++nq;
        const float sum = warp_join<N>(l, lane, [](float a, float c) { return a + c; });
        if (lane % kLanesPerRow == 0) l_of[quarter * N + lane / kLanesPerRow] = sum;
        ok = !any_of_128(bar_id, !ok);
        if (!ok) break;
        tc_fence_after();
        tmem_ld_x16(t_o, o);   // (the next unit's first PV waits for its P, which follows these reads)
        tmem_ld_wait_tied<N>(o);
      }
      // thread `key` has element `key` of every row's result
      int64_t orow = (int64_t)(x.q0 + x.i0) * p.n_heads + x.h * p.group;
      const int64_t prow = (int64_t)u * pl.rows_cap;
      int g = 0;
#pragma unroll
      for (int r = 0; r < N; ++r) {
        if (r < live) {
          float lr = 0.f, m = -INFINITY, v = 0.f;
          if (x.n > 0) {
            lr = (l_of[r] + l_of[N + r]) + (l_of[2 * N + r] + l_of[3 * N + r]);
            m = m_tab[r];
            v = __uint_as_float(o[r]);
          }
          if (x.ns == 1) {
            reinterpret_cast<uint16_t*>(p.out)[orow * D + key] = bf16_bits(lr == 0.f ? 0.f : v * (1.f / lr));
            if (p.lse && key == r) p.lse[orow] = lr == 0.f ? -INFINITY : (m + log2f(lr)) * 0.6931471805599453f;
          } else {
            if (x.n > 0) p.part_o[(prow + r) * D + key] = v;   // (else (m, l) = (-inf, 0) tells as much)
            if (key == r) p.part_ml[prow + r] = make_float2(m, lr);
          }
        }
        ++orow;
        if (++g == p.group) {
          g = 0;
          orow += p.n_heads - p.group;
        }
      }
    }
  } else {
    // ======================= softmax warpgroups =======================
    // (shares of the launch's registers: Roles)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R::kSoftmaxRegs));
    const int w = wg;
    const int quarter = warp & 3;
    const int r0 = quarter * 32 - first_row(w);   // this warp's first row of the tile (below 0: none)
    const int r = r0 + lane;
    const uint32_t lane_off = (uint32_t)quarter << 21;    // TMEM lane 32 * quarter
    const uint32_t t_s = tmem + (uint32_t)w * 128 + lane_off, t_o = tmem + 256 + (uint32_t)w * 128 + lane_off;
    const uint32_t* const masks = reinterpret_cast<const uint32_t*>(smem + pl.off_mask) + w * kMaskRing * 4;
    const float scale = p.scale_log2;
    uint32_t nt = 0, nq = 0;
    bool ok = true;
    Unit x{}, nx{};
    if (first_unit(w) < n_units) x = decode_unit<kPair>(p, tab, gsz, chunk, first_unit(w), w);
    for (int u = first_unit(w); u < n_units && ok; u += n_streams, x = nx) {
      const int live = (x.i1 - x.i0) * p.group;
      const bool warp_live = r0 >= 0 && r0 < live;
      const int tok = r / p.group, g = r - tok * p.group;
      const int vis = r0 >= 0 && r < live ? x.P0 + x.i0 + tok + 1 : 0x7FFFFFFF;   // visible keys of this row
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < x.n; ++j, ++nt) {
        ok = __all_sync(0xffffffffu, wait_bar(bar_st(w, S_FULL), nt & 1u, abort_flag, status, tmo));
        if (!ok) break;
        if (warp_live) {
          tc_fence_after();
          // Pages by TMA in BF16: the row's 128 logits stay in registers.  With copying workers beside
          // them: 64, the others being read from TMEM twice, for the maximum and for the weights; with
          // widening ones, 32 in a rolled loop (slower on its own, but it leaves them the registers).
          constexpr int kHeld = R::kWorkWarps == 16 ? 32 : (R::kWorkWarps > 0 ? 64 : kAttnKeys);
          constexpr int kUnroll = kHeld == 32 ? 1 : kAttnKeys / kHeld;
          uint32_t s[kHeld];
          const int lim = vis - (x.lo + j) * kAttnKeys;
          const uint32_t* const mask = masks + (nt % kMaskRing) * 4;
          auto load_s = [&](int c0) {   // logits c0 .., those of keys not seen replaced by -inf
#pragma unroll
            for (int c = 0; c < kHeld; c += 32) tmem_ld_x32(t_s + c0 + c, s + c);
            tmem_ld_wait_tied<kHeld>(s);
            if (!listed) {
              if (__any_sync(0xffffffffu, lim < c0 + kHeld)) {
#pragma unroll
                for (int c = 0; c < kHeld; ++c) s[c] = c0 + c < lim ? s[c] : 0xFF800000u;
              }
            } else {
#pragma unroll
              for (int c = 0; c < kHeld; c += 32) {
                const uint32_t mk = mask[(c0 + c) >> 5];
                if (mk != 0xFFFFFFFFu) {
#pragma unroll
                  for (int i = 0; i < 32; ++i) s[c + i] = (mk >> i) & 1u ? s[c + i] : 0xFF800000u;
                }
              }
            }
          };
          float mx[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) mx[c] = -INFINITY;
#pragma unroll kUnroll
          for (int c0 = kAttnKeys - kHeld; c0 >= 0; c0 -= kHeld) {   // (the first ones stay)
            load_s(c0);
#pragma unroll
            for (int c = 0; c < kHeld; c += 2)
              mx[(c >> 1) & 7] = fmaxf(mx[(c >> 1) & 7], fmaxf(__uint_as_float(s[c]), __uint_as_float(s[c + 1])));
          }
          const float top = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                  fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
          const float mt = top == -INFINITY ? -INFINITY : top * scale;
          const bool raise = r < live && mt > m + kRaise;      // m = -inf: any finite maximum
          if (__any_sync(0xffffffffu, raise)) {
            const float alpha = raise ? ex2(m - mt) : 1.f;     // 0 when m = -inf
            if (raise) m = mt;
            l *= alpha;
            if (j > 0) {   // the previous tile's PV completed before this S
#pragma unroll 1
              for (int d = 0; d < D; d += 16) {
                uint32_t o[16];
                tmem_ld_x16(t_o + d, o);
                tmem_ld_wait_tied<16>(o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                tmem_st_x16(t_o + d, o);
              }
            }
          }
          const float mref = m == -INFINITY ? 0.f : m;
          const float2 sc2 = make_float2(scale, scale), mm2 = make_float2(-mref, -mref);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll kUnroll
          for (int c0 = 0; c0 < kAttnKeys; c0 += kHeld) {
            if (c0 > 0) load_s(c0);
#pragma unroll
            for (int c = 0; c < kHeld; c += 32) {
              uint32_t pk[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float2 e = ffma2(as_f2(s[c + 2 * i], s[c + 2 * i + 1]), sc2, mm2);
                e.x = ex2(e.x);
                e.y = ex2(e.y);
                sum[i & 1] = __fadd2_rn(sum[i & 1], e);
                pk[i] = pack_bf16(e.x, e.y);
              }
              tmem_st_x16(t_s + (c0 + c) / 2, pk);   // over logits already read
            }
          }
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          tmem_st_wait();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_st(w, P_FULL));
      }
      if (!ok) break;
      if (u + n_streams < n_units) nx = decode_unit<kPair>(p, tab, gsz, chunk, u + n_streams, w);   // (while O is formed)
      const bool mine = r0 >= 0 && r < live;
      const int64_t orow = (int64_t)(x.q0 + x.i0 + tok) * p.n_heads + x.h * p.group + g;
      const int64_t prow = (int64_t)(kPair ? 2 * u + w : u) * pl.rows_cap + r;
      if (x.n > 0) {
        ok = __all_sync(0xffffffffu, wait_bar(bar_st(w, O_FULL), nq & 1u, abort_flag, status, tmo));
        if (!ok) break;
        ++nq;
        tc_fence_after();   // (the next unit's first PV waits for its P, which follows these reads)
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          if (warp_live) {
            tmem_ld_x32(t_o + c, o);
            tmem_ld_wait_tied<32>(o);
          }
          if (mine) {
            if (x.ns == 1) {
              uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out) + orow * D + c);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  v[e] = pack_bf16(__uint_as_float(o[8 * i + 2 * e]) * inv, __uint_as_float(o[8 * i + 2 * e + 1]) * inv);
                dst[i] = make_uint4(v[0], v[1], v[2], v[3]);
              }
            } else {
              uint4* dst = reinterpret_cast<uint4*>(p.part_o + prow * D + c);
#pragma unroll
              for (int i = 0; i < 8; ++i) dst[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
          }
        }
      } else if (mine && x.ns == 1) {   // no key tile at all (a joined unit's (m, l) = (-inf, 0) tells as much)
        uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out) + orow * D);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) dst[i] = make_uint4(0, 0, 0, 0);
      }
      if (mine) {
        if (x.ns > 1) p.part_ml[prow] = make_float2(m, l);
        else if (p.lse) p.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      }
    }
  }
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
  if (tid == 0) put_block_status(p.hdr, *status);
}

// Joins the partial results of divided key ranges: one warp per (token, head).
template <int D, bool kPair>
__global__ void __launch_bounds__(256) paged_attention_join_kernel(const AttnParams p) {
  constexpr int VEC = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t rows = (int64_t)p.total_q * p.n_heads;
  const int chunk = p.hdr[kAttnHdrChunk];
  for (int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); row < rows; row += (int64_t)gridDim.x * 8) {
    const int t = (int)(row / p.n_heads), hh = (int)(row % p.n_heads);
    const int d = find_seq(p.cu_q, p.num_seqs, t);
    Doc o;
    if (!doc_info(p, d, &o) || t < o.q0 || t >= o.q0 + o.T) continue;
    int mt, kt;
    doc_tiles<kPair>(p, o, &mt, &kt);
    const int ns = splits_of(kt, chunk);
    if (ns == 1) continue;
    const int i = t - o.q0, tile = i / p.plan.tq;
    const int ut = kPair ? tile >> 1 : tile;
    const int u0 = p.doc_base[d] + ((hh / p.group) * mt + (mt - 1 - ut)) * ns;
    const int r = (i - tile * p.plan.tq) * p.group + hh % p.group;
    auto slot = [&](int s) { return (int64_t)(kPair ? 2 * (u0 + s) + (tile & 1) : u0 + s) * p.plan.rows_cap + r; };
    float m = -INFINITY;
    for (int s = lane; s < ns; s += 32) {
      const float2 ml = p.part_ml[slot(s)];
      if (ml.y != 0.f) m = fmaxf(m, ml.x);
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
    float l = 0.f, acc[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int s = 0; s < ns; ++s) {
      const float2 ml = p.part_ml[slot(s)];
      const float f = ml.y == 0.f ? 0.f : exp2f(ml.x - m);
      const float* src = p.part_o + slot(s) * D + lane * VEC;
      l = fmaf(ml.y, f, l);
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] = f == 0.f ? acc[e] : fmaf(src[e], f, acc[e]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint16_t* dst = reinterpret_cast<uint16_t*>(p.out) + row * D + lane * VEC;
#pragma unroll
    for (int e = 0; e < VEC; e += 2) *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
    if (p.lse && lane == 0) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
  }
}

template <int D, bool Q8, int MODE, bool NARROW = false>
cudaError_t launch(const AttnParams& p, int grid, int sm_count, cudaStream_t stream) {
  auto kernel = paged_attention_kernel<D, Q8, MODE, NARROW>;
  cudaError_t e;
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  static std::atomic<uint64_t> ready{0};   // devices on which this kernel is set up
  if (!(ready.load(std::memory_order_acquire) >> (dev & 63) & 1)) {
    // The warpgroups' register shares add up to kLaunchRegs a thread: fewer at launch would leave them waiting.
    cudaFuncAttributes a;
    if ((e = cudaFuncGetAttributes(&a, kernel)) != cudaSuccess) return e;
    if (a.numRegs < Roles<Q8, MODE, NARROW>::kLaunchRegs) return cudaErrorInvalidDeviceFunction;
    // always the same value: calls of several threads do not disturb one another
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kAttnSmemMax);
    if (e != cudaSuccess) return e;
    ready.fetch_or(1ull << (dev & 63), std::memory_order_release);
  }
  kernel<<<grid, Roles<Q8, MODE, NARROW>::kThreads, p.plan.smem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.plan.max_units == 0 || p.total_q == 0) return e;
  const int64_t blocks = ((int64_t)p.total_q * p.n_heads + 7) / 8;
  paged_attention_join_kernel<D, MODE == PAIR><<<(unsigned)(blocks < 8 * sm_count ? blocks : 8 * sm_count), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace attn

}  // namespace dsa
