// ne_paged.cuh -- addressing of the paged key/value cache, and its 8-bit type.
#pragma once

#include "ne_common.cuh"

namespace ne {
namespace kv {

// The (row, head) of a thread and where it lies in the cache.
struct Place {
  long long src;   // element offset of the row in the packed tensors
  long long slot;  // (page * Hkv + h) * page_size + slot: row index in the pools
  int pos;
};

// Row index in the pools of (page, head, position), or -1 for a page outside
// the pool.
__host__ __device__ __forceinline__ long long pool_row(const PagedCache& pc, int page, int h,
                                                       int pos) {
  if (page < 0 || page >= pc.n_pages) return -1;
  return ((static_cast<long long>(page) * pc.Hkv + h) << pc.page_shift) +
         (pos & ((1 << pc.page_shift) - 1));
}

// Where (row, head) pair `rh` lies.  0: placed; -1: a row of no sequence (left
// alone); NE_DEV_BAD_SEQLEN: a position outside [0, max_seqlen);
// NE_DEV_BAD_PAGE: a page outside the pool.
__host__ __device__ __forceinline__ int place(const PagedCache& pc, const int* cu,
                                              const int* start_pos, int nseq, int rh, Place& pl) {
  const int r = rh / pc.Hkv, h = rh - r * pc.Hkv;
  const int s = find_sequence(cu, nseq, r);
  if (s < 0) return -1;
  const long long pos = static_cast<long long>(load_int(start_pos + s)) + (r - load_int(cu + s));
  if (pos < 0 || pos >= pc.max_seqlen) return NE_DEV_BAD_SEQLEN;
  const int page = load_int(pc.block_table + static_cast<long long>(s) * pc.max_pages +
                            (pos >> pc.page_shift));
  const long long slot = pool_row(pc, page, h, static_cast<int>(pos));
  if (slot < 0) return NE_DEV_BAD_PAGE;
  pl.pos = static_cast<int>(pos);
  pl.src = static_cast<long long>(rh) * kHD;
  pl.slot = slot;
  return 0;
}

// The value of a scale byte: 2^(byte - 127), NaN for 255.
__device__ __forceinline__ float scale_value(int byte) {
  return __uint_as_float(byte == 255 ? 0x7fc00000u
                                     : byte == 0 ? 0x00400000u
                                                 : static_cast<uint32_t>(byte) << 23);
}

// Two e4m3 bytes (low half of `two`) -> two halves (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return h;
}
// Two e4m3 bytes -> two fp32 (exact).
__device__ __forceinline__ void unpack_e4m3x2(uint32_t two, float& a, float& b) {
  asm("{\n\t.reg .f16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
      : "=f"(a), "=f"(b)
      : "r"(e4m3x2_to_f16x2(two)));
}

}  // namespace kv
}  // namespace ne
