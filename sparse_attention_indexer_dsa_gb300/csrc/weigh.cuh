// What the two kernels of cache_weigh share (weigh.cu, weigh_tiles.cu).
#pragma once

#include "dsa_device.cuh"
#include "evict_params.h"

namespace dsa {

namespace weigh {

constexpr float kLog2e = 1.4426950408889634f;

struct Doc {
  int q0, T, S;
};

// A sequence's sizes; T = 0 (and false) when they are inconsistent.
__device__ __forceinline__ bool doc_info(const WeighParams& p, int d, Doc* o) {
  const int q0 = __ldg(p.cu_q + d), q1 = __ldg(p.cu_q + d + 1);
  const int k0 = __ldg(p.cu_k + d), k1 = __ldg(p.cu_k + d + 1);
  o->q0 = q0;
  o->T = q1 - q0;
  o->S = k1 - k0;
  const bool ok = q0 >= 0 && q1 >= q0 && q1 <= p.total_q && k0 >= 0 && k1 >= k0 && o->S >= o->T &&
                  o->T <= p.max_seqlen_q && o->S <= p.max_seqlen_k &&
                  (int64_t)o->S <= ((int64_t)p.c.max_pages << p.c.page_shift);
  if (!ok) o->T = 0;
  return ok;
}

// Whether a sequence's query rows (tokens x heads of the group) are few: its keys then stream past them
// (weigh.cu), else the queries past tiles of keys (weigh_tiles.cu).
__device__ __forceinline__ bool by_steps(const WeighParams& p, int T) { return (int64_t)T * p.group <= p.step_rows; }

// Row r of a sequence's query rows: its token, its head of the group.
__device__ __forceinline__ int token_of(const WeighParams& p, int r, int* g) {
  const int t = p.group == 1 ? r : (r < 65536 ? (int)__umulhi((uint32_t)r, p.group_mul) : r / p.group);
  *g = r - t * p.group;
  return t;
}

// The bias that turns a scaled logit into the exponent of its weight; a row that saw no key weighs none.
__device__ __forceinline__ float bias_of(float lse) { return lse != -INFINITY ? -lse * kLog2e : -INFINITY; }

// Every block of the call's launches records its status.
__device__ __forceinline__ void put_status(const WeighParams& p, int block, int code) {
  p.hdr[DSA_DEV_STATUS_FIRST + block] = code;
  if (block == 0) {
    p.hdr[0] = DSA_DEV_STATUS_PER_BLOCK;
    p.hdr[1] = p.step_blocks + p.tile_blocks;
  }
}

}  // namespace weigh

}  // namespace dsa
