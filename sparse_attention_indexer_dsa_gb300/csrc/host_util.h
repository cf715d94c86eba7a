// Host helpers shared by the C ABI's entry points: the error message of
// dsa_idx_last_error() and the device facts.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "dsa_idx.h"

namespace dsa {

struct DevInfo {
  int sm_count = 0, major = 0, minor = 0;
};

// Records the message and returns the code.
dsa_status_t fail(dsa_status_t s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
dsa_status_t cuda_fail(cudaError_t e, const char* what);
// Facts of the current device; refuses anything but sm_103.
dsa_status_t device_info(DevInfo* out);

dsa_status_t make_pages_map(CUtensorMap* m, const void* base, int64_t groups, int rows, int D, int box_rows, bool b8);

// Queries [tokens][heads][D] BF16 as boxes of `tokens_per` tokens x `heads_per` heads x 64 elements.
dsa_status_t make_queries_map(CUtensorMap* m, const void* q, int tokens, int64_t stride, int heads, int D, int heads_per,
                              int tokens_per);

// Checks that the paged-cache operators share.  The first fills the device view.
struct PagedCacheView;
dsa_status_t check_cache(PagedCacheView* c, const void* k_pages, const uint8_t* k_page_scale, const void* v_pages,
                         const uint8_t* v_page_scale, int num_pages, int page_size, int n_kv_heads, int head_dim,
                         dsa_precision_t prec, const int32_t* page_table, int max_pages, int num_seqs,
                         const int32_t* cu_seqlens_k);
dsa_status_t check_ws(const void* ws, size_t ws_bytes, size_t need);
// Token stride of a [tokens, heads, head_dim] tensor: 0 = packed.
dsa_status_t check_stride(int64_t* stride, int heads, int head_dim, int elem_bytes, const char* name);

// Limit of the kernels' bounded waits, and the fault injection of the tests.
unsigned long long wait_timeout_ns();
int fault_inject_mode();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace dsa
