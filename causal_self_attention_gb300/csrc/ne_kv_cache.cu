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
// rounding of it.  Read: the mirror image, bf16 out.
//
// Both move bytes and nothing else: per (row, head) 256 in and 256 (bf16) or
// 130 (e4m3) out, or the reverse.  Four lanes take the 64 dims of a (row,
// head), lane c the 16-byte chunks c and c + 4 of K and of V, so that each
// rotation pair (i, i + 32) sits in one lane, a warp moves eight neighbouring
// 128-byte rows of each tensor, and every thread has four loads in flight.
// A row's way is a chain of loads -- its sequence (two rounds of probes for 64
// sequences), the position, the page, the row -- so that small calls are its
// latency and large ones hide it under the other CTAs' rows.  Measured: a token
// each for 64 sequences, 4 heads, 2.6 us; 32 prompts, 19,540 rows of 4 heads, to
// e4m3 8.9 us (3.4 TB/s; the rows of the output stay in L2); 77,305 rows of 8
// heads read from e4m3 40.9 us (5.8 TB/s, 87% of the copy rate).
#include "ne_attn_debug.h"
#include "ne_paged.cuh"
#include "ne_sm100.cuh"

namespace ne {

namespace kv {
constexpr int kThreads = 256;
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
}  // namespace kv

// kE4m3: the pools' type.  rope.cs == nullptr: the keys come rotated.
template <bool kE4m3>
__global__ void __launch_bounds__(kv::kThreads)
    ne_kv_append_kernel(const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v,
                        const int* __restrict__ cu, const int* __restrict__ start_pos, int nseq,
                        int n_tot, const PagedCache pc, RopeTable rope, int* status) {
  using namespace kv;
  pdl_wait();  // the kernel that wrote k, v (and anything before it) has completed
  const long long w = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const int c = static_cast<int>(w % kParts);
  const long long rh = w / kParts;
  Place pl = {0, 0, 0};
  int code = -1;
  if (rh < static_cast<long long>(n_tot) * pc.Hkv)
    code = place(pc, cu, start_pos, nseq, static_cast<int>(rh), pl);
  if (code > 0) atomicCAS(status, 0, code);
  const bool valid = code == 0;
  // A lane with nothing to do reads row 0 of each tensor and discards it.
  const uint4* kr = reinterpret_cast<const uint4*>(k + pl.src);
  const uint4* vr = reinterpret_cast<const uint4*>(v + pl.src);
  const uint4 k0 = __ldg(kr + c), k1 = __ldg(kr + c + 4);
  const uint4 v0 = __ldg(vr + c), v1 = __ldg(vr + c + 4);
  float a[8], b[8];
  unpack8(k0, a);
  unpack8(k1, b);
  if (rope.cs) {
    const float4* cs =
        reinterpret_cast<const float4*>(rope.cs + static_cast<long long>(pl.pos) * 32 + 8 * c);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float4 t = __ldg(cs + u);  // (cos, sin) of dims 8c + 2u and 8c + 2u + 1
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
  if constexpr (kE4m3) {
    store_e4m3(a, b, c, valid, pl.slot, static_cast<uint8_t*>(pc.k), pc.k_scale);
    unpack8(v0, a);
    unpack8(v1, b);
    store_e4m3(a, b, c, valid, pl.slot, static_cast<uint8_t*>(pc.v), pc.v_scale);
  } else if (valid) {
    uint4* ko = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(pc.k) + pl.slot * kHD);
    uint4* vo = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(pc.v) + pl.slot * kHD);
    ko[c] = pack8(a);
    ko[c + 4] = pack8(b);
    vo[c] = v0;
    vo[c + 4] = v1;
  }
}

template <bool kE4m3>
__global__ void __launch_bounds__(kv::kThreads)
    ne_kv_read_kernel(__nv_bfloat16* __restrict__ k, __nv_bfloat16* __restrict__ v,
                      const int* __restrict__ cu, const int* __restrict__ start_pos, int nseq,
                      int n_tot, const PagedCache pc, int* status) {
  using namespace kv;
  pdl_wait();  // the kernel that filled the cache has completed
  const long long w = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const int c = static_cast<int>(w % kParts);
  const long long rh = w / kParts;
  if (rh >= static_cast<long long>(n_tot) * pc.Hkv) return;
  Place pl = {0, 0, 0};
  const int code = place(pc, cu, start_pos, nseq, static_cast<int>(rh), pl);
  if (code > 0) atomicCAS(status, 0, code);
  if (code != 0) return;
  uint4* ko = reinterpret_cast<uint4*>(k + pl.src);
  uint4* vo = reinterpret_cast<uint4*>(v + pl.src);
  if constexpr (kE4m3) {
    auto row = [&](const void* pool, const uint8_t* scale, uint4* out) {
      const uint2* src =
          reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(pool) + pl.slot * kHD);
      const uint2 w[2] = {src[c], src[c + 4]};
      const float f = scale_value(scale[pl.slot]);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float x[8];
        unpack_e4m3x2(w[u].x, x[0], x[1]);
        unpack_e4m3x2(w[u].x >> 16, x[2], x[3]);
        unpack_e4m3x2(w[u].y, x[4], x[5]);
        unpack_e4m3x2(w[u].y >> 16, x[6], x[7]);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= f;
        out[c + 4 * u] = pack8(x);
      }
    };
    row(pc.k, pc.k_scale, ko);
    row(pc.v, pc.v_scale, vo);
  } else {
    const uint4* kr =
        reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(pc.k) + pl.slot * kHD);
    const uint4* vr =
        reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(pc.v) + pl.slot * kHD);
    const uint4 k0 = kr[c], k1 = kr[c + 4], v0 = vr[c], v1 = vr[c + 4];
    ko[c] = k0;
    ko[c + 4] = k1;
    vo[c] = v0;
    vo[c + 4] = v1;
  }
}

namespace {
dim3 kv_grid(int n_tot, int Hkv) {
  const long long items = static_cast<long long>(n_tot) * Hkv * kv::kParts;
  return dim3(static_cast<unsigned>((items + kv::kThreads - 1) / kv::kThreads));
}
}  // namespace

cudaError_t launch_kv_append(const __nv_bfloat16* k, const __nv_bfloat16* v, const int* cu,
                             const int* start_pos, int nseq, int n_tot, const PagedCache& pc,
                             bool e4m3, const RopeTable& rope, int* status, cudaStream_t stream) {
  return launch_pdl(e4m3 ? ne_kv_append_kernel<true> : ne_kv_append_kernel<false>,
                    kv_grid(n_tot, pc.Hkv), dim3(kv::kThreads), 0, stream, k, v, cu, start_pos,
                    nseq, n_tot, pc, rope, status);
}

cudaError_t launch_kv_read(__nv_bfloat16* k, __nv_bfloat16* v, const int* cu,
                           const int* start_pos, int nseq, int n_tot, const PagedCache& pc,
                           bool e4m3, int* status, cudaStream_t stream) {
  return launch_pdl(e4m3 ? ne_kv_read_kernel<true> : ne_kv_read_kernel<false>,
                    kv_grid(n_tot, pc.Hkv), dim3(kv::kThreads), 0, stream, k, v, cu, start_pos,
                    nseq, n_tot, pc, status);
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
