// ne_attn_paged.cu -- attention of one new token per sequence over a paged
// key/value cache, sm_103a.
//
//   q' = bf16(R(n - 1) q),  s_j = scale * q'.k_j,  j < n = seq_lens[b],
//   lse = log sum_j exp(s_j),  o = sum_j exp(s_j - lse) v_j
// for every query head; query head h reads the cached head h / (H / Hkv).
//
// Two kernels: a CTA per (query head, chunk of kChunk positions, sequence)
// forms the chunk's running maximum, sum and output with eight lanes per key
// (8 dims each), and a merge kernel joins the chunks of a (sequence, head).
// A sequence whose length is outside [0, max_seqlen], or that has a page
// outside the pool in one of its chunks, is reported and gets o = 0,
// lse = -inf.
#include "ne_paged.cuh"
#include "ne_sm100.cuh"

namespace ne {

namespace paged {
constexpr int kChunk = 256;
constexpr int kWarps = 4;
constexpr int kPartFloats = 68;  // m, l, 2 pad, o[64]; l < 0 marks a bad page
}  // namespace paged

template <bool kE4m3>
__global__ void __launch_bounds__(paged::kWarps * 32)
    ne_attn_paged_split_kernel(const __nv_bfloat16* __restrict__ q, const PagedCache pc,
                               const int* __restrict__ seq_lens, int H, RopeTable rope,
                               float scale_log2, float* __restrict__ part, int n_chunks,
                               int* status) {
  using namespace paged;
  __shared__ float red[kWarps * 4][66];
  pdl_wait();
  pdl_launch_dependents();
  const int h = blockIdx.x, c = blockIdx.y, b = blockIdx.z;
  const int group = threadIdx.x >> 3, cl = threadIdx.x & 7;  // 16 groups of 8 lanes
  int n = __ldg(seq_lens + b);
  if (n < 0 || n > pc.max_seqlen) {
    if (threadIdx.x == 0) atomicCAS(status, 0, NE_DEV_BAD_SEQLEN);
    n = 0;
  }
  const int hk = h / (H / pc.Hkv);
  float qv[8];
  {
    const __nv_bfloat16* row = q + (static_cast<long long>(b) * H + h) * kHD;
    const float2* cs = rope.cs ? rope.cs + static_cast<long long>(max(n - 1, 0)) * 32 : nullptr;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int d = 8 * cl + i;
      const float x = __bfloat162float(row[d]), y = __bfloat162float(row[d ^ 32]);
      float r = x;
      if (cs) {
        const float2 t = __ldg(cs + (d & 31));
        r = d < 32 ? __fmaf_rn(x, t.x, -__fmul_rn(y, t.y)) : __fmaf_rn(x, t.x, __fmul_rn(y, t.y));
      }
      qv[i] = __bfloat162float(__float2bfloat16(r));
    }
  }
  float m = -INFINITY, l = 0.f, o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  bool bad = false;
  const int end = min((c + 1) * kChunk, n);
  for (int j0 = c * kChunk; j0 < end; j0 += 16) {
    const int j = j0 + group;
    const int jj = min(j, end - 1);
    const int page = __ldg(pc.block_table + static_cast<long long>(b) * pc.max_pages +
                           (jj >> pc.page_shift));
    const bool page_ok = page >= 0 && page < pc.n_pages;
    bad |= !page_ok;
    const long long slot = kv::pool_row(pc, page_ok ? page : 0, hk, jj);
    float kk[8], vv[8];
    if constexpr (kE4m3) {
      for (int u = 0; u < 2; ++u) {
        const uint8_t* pool = static_cast<const uint8_t*>(u ? pc.v : pc.k);
        const float f = kv::scale_value((u ? pc.v_scale : pc.k_scale)[slot]);
        const uint2 w = reinterpret_cast<const uint2*>(pool + slot * kHD)[cl];
        float* x = u ? vv : kk;
        kv::unpack_e4m3x2(w.x, x[0], x[1]);
        kv::unpack_e4m3x2(w.x >> 16, x[2], x[3]);
        kv::unpack_e4m3x2(w.y, x[4], x[5]);
        kv::unpack_e4m3x2(w.y >> 16, x[6], x[7]);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= f;
      }
    } else {
      const uint4 kw = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(pc.k) + slot * kHD)[cl];
      const uint4 vw = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(pc.v) + slot * kHD)[cl];
      const uint32_t ku[4] = {kw.x, kw.y, kw.z, kw.w}, vu[4] = {vw.x, vw.y, vw.z, vw.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        kk[2 * i] = bf16lo_to_f32(ku[i]);
        kk[2 * i + 1] = bf16hi_to_f32(ku[i]);
        vv[2 * i] = bf16lo_to_f32(vu[i]);
        vv[2 * i + 1] = bf16hi_to_f32(vu[i]);
      }
    }
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) dot = __fmaf_rn(qv[i], kk[i], dot);
    dot += __shfl_xor_sync(0xffffffffu, dot, 1);
    dot += __shfl_xor_sync(0xffffffffu, dot, 2);
    dot += __shfl_xor_sync(0xffffffffu, dot, 4);
    if (j < end && page_ok) {
      const float s = dot * scale_log2;
      const float mn = fmaxf(m, s);
      const float a = m == mn ? 1.f : ex2_approx(m - mn), p = ex2_approx(s - mn);
      l = l * a + p;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = o[i] * a + p * vv[i];
      m = mn;
    }
  }
  red[group][0] = m;
  red[group][1] = l;
#pragma unroll
  for (int i = 0; i < 8; ++i) red[group][2 + 8 * cl + i] = o[i];
  bad = __syncthreads_or(bad);
  if (bad && threadIdx.x == 0) atomicCAS(status, 0, NE_DEV_BAD_PAGE);
  if (threadIdx.x < 64) {
    float M = -INFINITY, L = 0.f, O = 0.f;
    for (int g = 0; g < kWarps * 4; ++g) M = fmaxf(M, red[g][0]);
    for (int g = 0; g < kWarps * 4; ++g) {
      const float a = red[g][1] == 0.f ? 0.f : ex2_approx(red[g][0] - M);
      L += red[g][1] * a;
      O += red[g][2 + threadIdx.x] * a;
    }
    float* dst = part + ((static_cast<long long>(b) * H + h) * n_chunks + c) * kPartFloats;
    dst[4 + threadIdx.x] = O;
    if (threadIdx.x == 0) {
      dst[0] = M;
      dst[1] = bad ? -1.f : L;
    }
  }
}

__global__ void __launch_bounds__(32)
    ne_attn_paged_merge_kernel(const float* __restrict__ part, int n_chunks,
                               __nv_bfloat16* __restrict__ out, float* __restrict__ lse) {
  using namespace paged;
  pdl_wait();
  pdl_launch_dependents();
  const long long bh = blockIdx.x;
  const int lane = threadIdx.x;
  const float* src = part + bh * n_chunks * kPartFloats;
  float M = -INFINITY;
  bool bad = false;
  for (int c = 0; c < n_chunks; ++c) {
    M = fmaxf(M, src[c * kPartFloats]);
    bad |= src[c * kPartFloats + 1] < 0.f;
  }
  float L = 0.f, o0 = 0.f, o1 = 0.f;
  for (int c = 0; c < n_chunks && !bad; ++c) {
    const float* p = src + c * kPartFloats;
    const float a = p[1] == 0.f ? 0.f : ex2_approx(p[0] - M);
    L += p[1] * a;
    o0 += p[4 + 2 * lane] * a;
    o1 += p[5 + 2 * lane] * a;
  }
  const bool none = L == 0.f;
  const float inv = none ? 0.f : 1.f / L;
  reinterpret_cast<uint32_t*>(out + bh * kHD)[lane] = pack_bf16x2(o0 * inv, o1 * inv);
  if (lane == 0) lse[bh] = none ? -INFINITY : (M + __log2f(L)) * 0.69314718055994531f;
}

size_t paged_part_bytes(int B, int H, int max_seqlen) {
  return static_cast<size_t>(B) * H * ((max_seqlen + paged::kChunk - 1) / paged::kChunk) *
         paged::kPartFloats * sizeof(float);
}

cudaError_t launch_decode_paged(const __nv_bfloat16* q, const PagedCache& pc, bool e4m3,
                                const int* seq_lens, int B, int H, const RopeTable& rope,
                                float scale_log2, float* part, __nv_bfloat16* out, float* lse,
                                int* status, cudaStream_t stream) {
  const int n_chunks = (pc.max_seqlen + paged::kChunk - 1) / paged::kChunk;
  cudaError_t e = launch_pdl(
      e4m3 ? ne_attn_paged_split_kernel<true> : ne_attn_paged_split_kernel<false>,
      dim3(H, n_chunks, B), dim3(paged::kWarps * 32), 0, stream, q, pc, seq_lens, H, rope,
      scale_log2, part, n_chunks, status);
  if (e != cudaSuccess) return e;
  return launch_pdl(ne_attn_paged_merge_kernel, dim3(B * H), dim3(32), 0, stream, part, n_chunks,
                    out, lse);
}

}  // namespace ne
