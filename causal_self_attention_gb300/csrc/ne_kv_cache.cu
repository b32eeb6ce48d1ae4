// ne_kv_cache.cu -- writing rows into a paged key/value cache and reading them
// back, sm_103a.
//
// Append: row i of sequence s of the packed k, v [n_tot, Hkv, 64] goes to
// position start_pos[s] + i.  The key is rotated there (k' = R(n) k, the fp32
// rule of the attention kernels; not when the caller passes k' already), and
// both rows are stored as bf16 or, each with a scale of its own, as e4m3:
//   e = the smallest integer >= -100 with max |x| <= 448 * 2^e,
//   byte = e + 127,  x8 = round to nearest even (x * 2^-e) in e4m3.
// A power of two as the scale makes x * 2^-e exact, so a value is rounded
// once (at most half an e4m3 step, 2^-4 of it; below 2^-6 * 2^e half of
// 2^-9 * 2^e), the scale is a single byte, and dequantised values are exact
// in bf16.  The key is quantised from its fp32 rotation, not from the bf16
// rounding of it.  e2m1: the same for each half of a row, the 32 dims that the
// other 32 are rotated with, with max |x| <= 6 * 2^e and e <= 125 (so that 6 * 2^e
// is finite in bf16; larger values become that).  Read: the mirror image, bf16 out.
//
// Both move bytes and nothing else: per (row, head) 256 in and 256 (bf16), 130
// (e4m3) or 68 (e2m1) out, or the reverse.  Four lanes take the 64 dims of a (row,
// head), lane c the 16-byte chunks c and c + 4 of K and of V, so that each
// rotation pair (i, i + 32) sits in one lane, a warp moves eight neighbouring
// 128-byte rows of each tensor, and every thread has four loads in flight.
// A row's way is a chain of loads -- its sequence (two rounds of probes for 64
// sequences), the position, the page, the row -- so that small calls are its
// latency and large ones hide it under the other CTAs' rows.  Measured: a token
// each for 64 sequences, 4 heads, 2.4 us; 32 prompts, 19,540 rows of 4 heads, to
// e4m3 6.9 us (4.3 TB/s; the rows of the output stay in L2); 77,305 rows of 8
// heads read from e4m3 38.1 us (6.3 TB/s, 92% of the copy rate); 69,524 rows of 12 heads
// to e2m1 55.3 us (4.9 TB/s), back 44.0 us (6.1 TB/s).
#include "ne_attn_debug.h"
#include "ne_paged.cuh"
#include "ne_sm100.cuh"

namespace ne {

namespace kv {
// Small CTAs, whose loads and stores overlap others': 69,524 rows of 12 heads to e2m1 55.2 us of
// 64 threads, 55.3 of 128, 60.6 of 256, back 43.8, 44.0, 44.3; 32 prompts to e4m3 6.8, 6.9, 7.6.
constexpr int kThreads = 128;
constexpr int kParts = 4;  // lanes per (row, head)

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16lo_to_f32(u[i]);
    x[2 * i + 1] = bf16hi_to_f32(u[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// Four fp32 -> four e4m3 bytes (round to nearest even; nothing exceeds 448).
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return lo | (static_cast<uint32_t>(hi) << 16);
}
// The scale of a row whose 64 values' |bits| have the maximum `top` (bits
// compare like magnitudes, with NaN above infinity above every number).
__device__ __forceinline__ int scale_byte(uint32_t top) {
  if (top >= 0x7f800000u) return 255;
  const int e = static_cast<int>(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, -100) + 127;  // e <= 120
}

// One row's 16 values of a lane into the e4m3 pool, and its scale (lane 0 of
// the four).  Every lane of the warp calls this (shuffles).
__device__ __forceinline__ void store_e4m3(const float (&lo)[8], const float (&hi)[8], int c,
                                           bool valid, long long slot, uint8_t* pool,
                                           uint8_t* scale) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    top = max(top, __float_as_uint(lo[i]) & 0x7fffffffu);
    top = max(top, __float_as_uint(hi[i]) & 0x7fffffffu);
  }
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const int byte = scale_byte(top);
  // 2^-e, e = byte - 127; a row marked 255 stores e4m3 NaNs.
  const float inv = byte == 255 ? __uint_as_float(0x7fc00000u)
                                : __uint_as_float(static_cast<uint32_t>(254 - byte) << 23);
  if (!valid) return;
  uint8_t* row = pool + slot * kHD;
  reinterpret_cast<uint2*>(row)[c] =
      make_uint2(pack_e4m3x4(lo[0] * inv, lo[1] * inv, lo[2] * inv, lo[3] * inv),
                 pack_e4m3x4(lo[4] * inv, lo[5] * inv, lo[6] * inv, lo[7] * inv));
  reinterpret_cast<uint2*>(row)[c + 4] =
      make_uint2(pack_e4m3x4(hi[0] * inv, hi[1] * inv, hi[2] * inv, hi[3] * inv),
                 pack_e4m3x4(hi[4] * inv, hi[5] * inv, hi[6] * inv, hi[7] * inv));
  if (c == 0) scale[slot] = static_cast<uint8_t>(byte);
}
// The scale of 32 values in e2m1.
__device__ __forceinline__ int scale_byte_e2m1(uint32_t top) {
  if (top >= 0x7f800000u) return 255;
  const int e = static_cast<int>(top >> 23) - 127 - 2 + ((top & 0x7fffffu) > 0x400000u ? 1 : 0);
  return min(max(e, -100), 125) + 127;
}

// One row's 16 values of a lane, 8 of each half, into the e2m1 pool, and the
// row's two scales (lane 0 of the four).  Every lane of the warp calls this.
__device__ __forceinline__ void store_e2m1(float (&lo)[8], float (&hi)[8], int c, bool valid,
                                           long long slot, uint8_t* pool, uint8_t* scale) {
  uint32_t top0 = 0, top1 = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    top0 = max(top0, __float_as_uint(lo[i]) & 0x7fffffffu);
    top1 = max(top1, __float_as_uint(hi[i]) & 0x7fffffffu);
  }
#pragma unroll
  for (int sh = 1; sh < kParts; sh <<= 1) {
    top0 = max(top0, __shfl_xor_sync(0xffffffffu, top0, sh));
    top1 = max(top1, __shfl_xor_sync(0xffffffffu, top1, sh));
  }
  const int b0 = scale_byte_e2m1(top0), b1 = scale_byte_e2m1(top1);
  // 2^-e, e = byte - 127; a half marked 255 stores zeros.
  const float inv0 = b0 == 255 ? 0.f : __uint_as_float(static_cast<uint32_t>(254 - b0) << 23);
  const float inv1 = b1 == 255 ? 0.f : __uint_as_float(static_cast<uint32_t>(254 - b1) << 23);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo[i] = b0 == 255 ? 0.f : lo[i] * inv0;
    hi[i] = b1 == 255 ? 0.f : hi[i] * inv1;
  }
  if (!valid) return;
  // Words 2c and 2c + 1: four values of each half.
  const uint32_t l = pack_e2m1x8(lo), h = pack_e2m1x8(hi);
  reinterpret_cast<uint2*>(pool + slot * (kHD / 2))[c] =
      make_uint2(__byte_perm(l, h, 0x5410), __byte_perm(l, h, 0x7632));
  if (c == 0)
    reinterpret_cast<uint16_t*>(scale)[slot] = static_cast<uint16_t>(b0 | (b1 << 8));
}
}  // namespace kv

// kType: the pools' type.  kHeads: neighbouring heads of a row that a quad takes, whose
// place is found once (Hkv is a multiple of it).  rope.cs == nullptr: the keys come rotated.
template <Kv kType, int kHeads>
__global__ void __launch_bounds__(kv::kThreads)
    ne_kv_append_kernel(const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v,
                        const int* __restrict__ cu, const int* __restrict__ start_pos, int nseq,
                        int n_tot, const PagedCache pc, RopeTable rope, int* status) {
  using namespace kv;
  pdl_wait();  // the kernel that wrote k, v (and anything before it) has completed
  const long long w = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const int c = static_cast<int>(w % kParts);
  const long long rh = w / kParts * kHeads;
  Place pl = {0, 0, 0};
  int code = -1;
  if (rh < static_cast<long long>(n_tot) * pc.Hkv)
    code = place(pc, cu, start_pos, nseq, static_cast<int>(rh), pl);
  if (code > 0) atomicCAS(status, 0, code);
  const bool valid = code == 0;
  // A lane with nothing to do reads row 0 of each tensor and discards it.
  const uint4* kr = reinterpret_cast<const uint4*>(k + pl.src) + c;
  const uint4* vr = reinterpret_cast<const uint4*>(v + pl.src) + c;
  uint4 k0[kHeads], k1[kHeads], v0[kHeads], v1[kHeads];
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    k0[h] = __ldg(kr + 8 * h);
    k1[h] = __ldg(kr + 8 * h + 4);
    v0[h] = __ldg(vr + 8 * h);
    v1[h] = __ldg(vr + 8 * h + 4);
  }
  float4 cs[4];  // (cos, sin) of dims 8c + 2u and 8c + 2u + 1
  if (rope.cs) {
    const float4* t =
        reinterpret_cast<const float4*>(rope.cs + static_cast<long long>(pl.pos) * 32 + 8 * c);
#pragma unroll
    for (int u = 0; u < 4; ++u) cs[u] = __ldg(t + u);
  }
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    const long long slot = pl.slot + (static_cast<long long>(h) << pc.page_shift);
    float a[8], b[8];
    unpack8(k0[h], a);
    unpack8(k1[h], b);
    if (rope.cs) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float4 t = cs[u];
        const float lo0 = __fmaf_rn(a[2 * u], t.x, -__fmul_rn(b[2 * u], t.y));
        const float hi0 = __fmaf_rn(b[2 * u], t.x, __fmul_rn(a[2 * u], t.y));
        const float lo1 = __fmaf_rn(a[2 * u + 1], t.z, -__fmul_rn(b[2 * u + 1], t.w));
        const float hi1 = __fmaf_rn(b[2 * u + 1], t.z, __fmul_rn(a[2 * u + 1], t.w));
        a[2 * u] = lo0;
        b[2 * u] = hi0;
        a[2 * u + 1] = lo1;
        b[2 * u + 1] = hi1;
      }
    }
    if constexpr (kType == Kv::kE4m3) {
      store_e4m3(a, b, c, valid, slot, static_cast<uint8_t*>(pc.k), pc.k_scale);
      unpack8(v0[h], a);
      unpack8(v1[h], b);
      store_e4m3(a, b, c, valid, slot, static_cast<uint8_t*>(pc.v), pc.v_scale);
    } else if constexpr (kType == Kv::kE2m1) {
      store_e2m1(a, b, c, valid, slot, static_cast<uint8_t*>(pc.k), pc.k_scale);
      unpack8(v0[h], a);
      unpack8(v1[h], b);
      store_e2m1(a, b, c, valid, slot, static_cast<uint8_t*>(pc.v), pc.v_scale);
    } else if (valid) {
      uint4* ko = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(pc.k) + slot * kHD);
      uint4* vo = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(pc.v) + slot * kHD);
      ko[c] = pack8(a);
      ko[c + 4] = pack8(b);
      vo[c] = v0[h];
      vo[c + 4] = v1[h];
    }
  }
}

template <Kv kType, int kHeads>
__global__ void __launch_bounds__(kv::kThreads)
    ne_kv_read_kernel(__nv_bfloat16* __restrict__ k, __nv_bfloat16* __restrict__ v,
                      const int* __restrict__ cu, const int* __restrict__ start_pos, int nseq,
                      int n_tot, const PagedCache pc, int* status) {
  using namespace kv;
  pdl_wait();  // the kernel that filled the cache has completed
  const long long w = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const int c = static_cast<int>(w % kParts);
  const long long rh = w / kParts * kHeads;
  if (rh >= static_cast<long long>(n_tot) * pc.Hkv) return;
  Place pl = {0, 0, 0};
  const int code = place(pc, cu, start_pos, nseq, static_cast<int>(rh), pl);
  if (code > 0) atomicCAS(status, 0, code);
  if (code != 0) return;
  // Loads of all heads first.
  constexpr int kWords = kType == Kv::kBf16 ? 4 : kType == Kv::kE4m3 ? 2 : 1;  // uint2 of a lane
  uint2 kw[kHeads][kWords], vw[kHeads][kWords];
  int ks[kHeads], vs[kHeads];
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    const long long slot = pl.slot + (static_cast<long long>(h) << pc.page_shift);
    auto load = [&](const void* pool, const uint8_t* scale, uint2 (&to)[kWords], int& byte) {
      if constexpr (kType == Kv::kBf16) {
        const uint4* src =
            reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(pool) + slot * kHD);
        const uint4 x = src[c], y = src[c + 4];
        to[0] = make_uint2(x.x, x.y);
        to[1] = make_uint2(x.z, x.w);
        to[2] = make_uint2(y.x, y.y);
        to[3] = make_uint2(y.z, y.w);
        byte = 0;
      } else if constexpr (kType == Kv::kE4m3) {
        const uint2* src =
            reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(pool) + slot * kHD);
        to[0] = src[c];
        to[1] = src[c + 4];
        byte = scale[slot];
      } else {
        to[0] = reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(pool) + slot * (kHD / 2))[c];
        byte = reinterpret_cast<const uint16_t*>(scale)[slot];
      }
    };
    load(pc.k, pc.k_scale, kw[h], ks[h]);
    load(pc.v, pc.v_scale, vw[h], vs[h]);
  }
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    auto store = [&](const uint2 (&w)[kWords], int byte, uint4* out) {
      if constexpr (kType == Kv::kBf16) {
        out[0] = make_uint4(w[0].x, w[0].y, w[1].x, w[1].y);
        out[4] = make_uint4(w[2].x, w[2].y, w[3].x, w[3].y);
      } else if constexpr (kType == Kv::kE4m3) {
        const float f = scale_value(byte);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float x[8];
          unpack_e4m3x2(w[u].x, x[0], x[1]);
          unpack_e4m3x2(w[u].x >> 16, x[2], x[3]);
          unpack_e4m3x2(w[u].y, x[4], x[5]);
          unpack_e4m3x2(w[u].y >> 16, x[6], x[7]);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] *= f;
          out[4 * u] = pack8(x);
        }
      } else {
        // (low halves of the two words: dims 8c .. 8c + 7; high halves: 32 + 8c ..)
        const uint32_t half[2] = {__byte_perm(w[0].x, w[0].y, 0x5410),
                                  __byte_perm(w[0].x, w[0].y, 0x7632)};
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float f = scale_value(u ? byte >> 8 : byte & 255);
          uint32_t two[4];
          e2m1x8_to_f16x2(half[u], two);
          float x[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f16x2_to_f32(two[i], x[2 * i], x[2 * i + 1]);
            x[2 * i] *= f;
            x[2 * i + 1] *= f;
          }
          out[4 * u] = pack8(x);
        }
      }
    };
    store(kw[h], ks[h], reinterpret_cast<uint4*>(k + pl.src + h * kHD) + c);
    store(vw[h], vs[h], reinterpret_cast<uint4*>(v + pl.src + h * kHD) + c);
  }
}

namespace {
template <Kv kType, int kHeads>
cudaError_t append(const __nv_bfloat16* k, const __nv_bfloat16* v, const int* cu,
                   const int* start_pos, int nseq, int n_tot, const PagedCache& pc,
                   const RopeTable& rope, int* status, cudaStream_t stream) {
  const long long items = static_cast<long long>(n_tot) * (pc.Hkv / kHeads) * kv::kParts;
  return launch_pdl(ne_kv_append_kernel<kType, kHeads>,
                    dim3(static_cast<unsigned>((items + kv::kThreads - 1) / kv::kThreads)),
                    dim3(kv::kThreads), 0, stream, k, v, cu, start_pos, nseq, n_tot, pc, rope, status);
}
template <Kv kType, int kHeads>
cudaError_t read(__nv_bfloat16* k, __nv_bfloat16* v, const int* cu, const int* start_pos, int nseq,
                 int n_tot, const PagedCache& pc, int* status, cudaStream_t stream) {
  const long long items = static_cast<long long>(n_tot) * (pc.Hkv / kHeads) * kv::kParts;
  return launch_pdl(ne_kv_read_kernel<kType, kHeads>,
                    dim3(static_cast<unsigned>((items + kv::kThreads - 1) / kv::kThreads)),
                    dim3(kv::kThreads), 0, stream, k, v, cu, start_pos, nseq, n_tot, pc, status);
}

// Two heads a quad for rows with scales, once they fill the GPU: what finds a row's place is
// half of the instructions of a (row, head) otherwise.  (69,524 rows of 12 heads, a head and
// two: e2m1 written 70.2 and 60.6 us, read 51.8 and 44.3; e4m3 63.7 and 59.2, 53.6 and 51.4;
// bf16, which only moves bytes, 67.3 and 65.5, 65.5 and 66.5.  Four: as two, or slower.  CTAs
// of 256 threads.)
bool two_heads(int n_tot, int Hkv) {
  return Hkv % 2 == 0 && static_cast<long long>(n_tot) * Hkv >= 1 << 16;
}
}  // namespace

cudaError_t launch_kv_append(const __nv_bfloat16* k, const __nv_bfloat16* v, const int* cu,
                             const int* start_pos, int nseq, int n_tot, const PagedCache& pc,
                             Kv type, const RopeTable& rope, int* status, cudaStream_t stream) {
  const bool two = two_heads(n_tot, pc.Hkv);
  auto* go = type == Kv::kE2m1   ? (two ? append<Kv::kE2m1, 2> : append<Kv::kE2m1, 1>)
             : type == Kv::kE4m3 ? (two ? append<Kv::kE4m3, 2> : append<Kv::kE4m3, 1>)
                                 : append<Kv::kBf16, 1>;
  return go(k, v, cu, start_pos, nseq, n_tot, pc, rope, status, stream);
}

cudaError_t launch_kv_read(__nv_bfloat16* k, __nv_bfloat16* v, const int* cu,
                           const int* start_pos, int nseq, int n_tot, const PagedCache& pc,
                           Kv type, int* status, cudaStream_t stream) {
  const bool two = two_heads(n_tot, pc.Hkv);
  auto* go = type == Kv::kE2m1   ? (two ? read<Kv::kE2m1, 2> : read<Kv::kE2m1, 1>)
             : type == Kv::kE4m3 ? (two ? read<Kv::kE4m3, 2> : read<Kv::kE4m3, 1>)
                                 : read<Kv::kBf16, 1>;
  return go(k, v, cu, start_pos, nseq, n_tot, pc, status, stream);
}

}  // namespace ne

// Host only: the kernels' own placement of one (row, head) pair.
extern "C" int ne_debug_kv_place(const int* cu_seqlens, const int* start_pos,
                                 const int* block_table, int nseq, int Hkv, int max_pages,
                                 int n_pages, int page_shift, int max_seqlen, int pair,
                                 long long* src, long long* slot, int* pos) {
  ne::PagedCache pc = {};
  pc.block_table = block_table;
  pc.max_pages = max_pages;
  pc.n_pages = n_pages;
  pc.page_shift = page_shift;
  pc.Hkv = Hkv;
  pc.max_seqlen = max_seqlen;
  ne::kv::Place pl = {-1, -1, -1};
  const int code = ne::kv::place(pc, cu_seqlens, start_pos, nseq, pair, pl);
  *src = pl.src;
  *slot = pl.slot;
  *pos = pl.pos;
  return code;
}
