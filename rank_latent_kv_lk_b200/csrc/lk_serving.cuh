// Device-side helpers of the serving operators, beside lk_common.cuh.
#pragma once

#include "lk_common.cuh"
#include "lk_serving_internal.h"

// Codes of the device status word beside those of an expired wait.
enum : unsigned int {
  LK_DEV_BAD_PAGE = 4u,    // a page table entry lies outside the pool
  LK_DEV_BAD_LENGTH = 8u,  // an append does not fit in the page table
};

// lk_mma_bf16_16816 with fp16 operands.
LK_DEVICE void lk_mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two values as packed fp16 (first in the low half), round to nearest even.
LK_DEVICE uint32_t lk_pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Row index (of the [n_pages, n_kv_heads, page_size] rows) of a slot, given
// its page; -1 (and the device status word set) if the page lies outside the
// pool.  Rows stay below 2^31 (checked on the host); byte offsets are 64-bit.
LK_DEVICE int lk_paged_row(int page, int slot, int h, int n_pages, int n_kv_heads, int page_shift) {
  if ((unsigned)page >= (unsigned)n_pages) {
    lk_dev_fail(LK_DEV_BAD_PAGE);
    return -1;
  }
  return ((page * n_kv_heads + h) << page_shift) | (slot & ((1 << page_shift) - 1));
}
