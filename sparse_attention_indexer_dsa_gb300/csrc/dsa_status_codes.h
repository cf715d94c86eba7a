// Codes the device writes into the workspace status word.  They equal the
// public dsa_status_t values of include/dsa_idx.h.
#pragma once
#define DSA_DEV_OK 0
#define DSA_DEV_ERR_INVALID_ARG 1
#define DSA_DEV_ERR_TIMEOUT 5
#define DSA_DEV_ERR_BOUNDS 6   // checked build only: a device-side bounds check failed
// A kernel without a launch before it that could clear the status word gives
// each of its blocks a word of its own, always written: the header's word 0
// then holds DSA_DEV_STATUS_PER_BLOCK, word 1 the number of blocks, and block
// b's code is word DSA_DEV_STATUS_FIRST + b (dsa_idx_read_status reduces them).
#define DSA_DEV_STATUS_PER_BLOCK 0x100
#define DSA_DEV_STATUS_FIRST 64
#define DSA_DEV_STATUS_HEADER_BYTES 8192
#define DSA_DEV_STATUS_MAX_BLOCKS ((DSA_DEV_STATUS_HEADER_BYTES / 4) - DSA_DEV_STATUS_FIRST)
