// ne_paged.cuh -- addressing of the paged key/value cache, and its 8-bit and 4-bit types.
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

// The value of a scale byte: 2^(byte - 127), NaN for 255.  (Both ends differ from the
// exponent alone by the mantissa's first bit: 2^-127 and a NaN.  Without branches: a
// choice here became a second copy of what follows it, 128 instructions a tile of the
// 4-bit decode.)
__device__ __forceinline__ float scale_value(uint32_t byte) {
  const uint32_t ends = static_cast<uint32_t>(static_cast<int>((byte + 1u) & 0xfeu) - 1) >> 31;
  return __uint_as_float((byte << 23) | (ends << 22));
}

// Two e4m3 bytes (low half of `two`) -> two halves (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return h;
}
// Two halves -> two fp32 (exact).
__device__ __forceinline__ void f16x2_to_f32(uint32_t h, float& a, float& b) {
  asm("{\n\t.reg .f16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
      : "=f"(a), "=f"(b)
      : "r"(h));
}
// Two e4m3 bytes -> two fp32 (exact).
__device__ __forceinline__ void unpack_e4m3x2(uint32_t two, float& a, float& b) {
  f16x2_to_f32(e4m3x2_to_f16x2(two), a, b);
}

// The four bytes of a word, two e2m1 values each -> halves (exact), the low one
// first.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// Eight fp32 of magnitude at most 6 -> e2m1 (round to nearest, ties to even), two to
// a byte, the first in the low half.
__device__ __forceinline__ uint32_t pack_e2m1x8(const float (&x)[8]) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return w;
}

}  // namespace kv
}  // namespace ne
