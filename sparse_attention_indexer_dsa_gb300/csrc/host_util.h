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

// Limit of the kernels' bounded waits, and the fault injection of the tests.
unsigned long long wait_timeout_ns();
int fault_inject_mode();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace dsa
