// ne_qk_norm.cu -- RMS norm of every head of the queries and keys, with the
// position rotation in the same pass, and its gradients, sm_103a.
//
//   r = 1 / sqrt(mean(x^2) + eps),  y = w * x * r,  out = R(p) y
// over the 64 dims of a head, w one weight [64] for all query heads and one for
// all key heads, p the row's position.  Backward, from the gradient g' of out:
//   g = R(p)^T g',  dw = sum over rows and heads of g * x * r,
//   dx = r * (g * w - x * r * mean(g * w * x * r)).
// The forward saves nothing: a row of 64 is in registers here anyway, and its r
// costs less to form again than to write and read.
//
// What bounds both is the rows' bytes, 256 a (row, head) forward and 384
// backward.  Four lanes take a (row, head), lane c the 16-byte chunks c and c +
// 4, so that each rotation pair (i, i + 32) sits in one lane and the sums over
// the head are two shuffles.  All arithmetic is fp32; each output is rounded
// once (bf16; dw is fp32).
// Measured, forward: 92,604 rows of 40 heads 145 us (6.5 TB/s, 96% of the copy rate),
// 18,641 of 16 heads 13.4 us where passes write the same memory (5.7 TB/s: part of it stays in
// L2), 15.3 where each writes its own (5.0 TB/s), 64 of 16 heads 1.5 us (a launch); backward:
// 65,536 rows of 40 heads 180 us (5.6 TB/s, 83%), 8192 of 16 heads 15.4 us (3.3 TB/s: two
// rounds of loads that wait, the sums of dw, the CTA that adds them up).
#include "ne_sm100.cuh"

namespace ne {

namespace qkn {
constexpr int kParts = 4;  // lanes per (row, head)
constexpr int kQkNormSms = 160;  // an upper bound on the part's SMs (152), and on the backward's CTAs

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
// The sum over a head: this lane's value and the other three lanes'.
__device__ __forceinline__ float head_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}
__device__ __forceinline__ float rstd_of(const float (&a)[8], const float (&b)[8], float eps) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss += a[i] * a[i] + b[i] * b[i];
  return rsqrtf(head_sum(ss) * (1.f / kHD) + eps);
}
// The lane's 8 rotation pairs (a, b) turned by their position's angles, or back.  cs[u]:
// (cos, sin) of dims 8c + 2u and 8c + 2u + 1.
template <bool kBack>
__device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], const float4 (&cs)[4]) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const float4 t = cs[u];
    const float s0 = kBack ? -t.y : t.y, s1 = kBack ? -t.w : t.w;
    const float lo0 = __fmaf_rn(a[2 * u], t.x, -__fmul_rn(b[2 * u], s0));
    const float hi0 = __fmaf_rn(b[2 * u], t.x, __fmul_rn(a[2 * u], s0));
    const float lo1 = __fmaf_rn(a[2 * u + 1], t.z, -__fmul_rn(b[2 * u + 1], s1));
    const float hi1 = __fmaf_rn(b[2 * u + 1], t.z, __fmul_rn(a[2 * u + 1], s1));
    a[2 * u] = lo0;
    b[2 * u] = hi0;
    a[2 * u + 1] = lo1;
    b[2 * u + 1] = hi1;
  }
}
// The position of a row: -1 for one to leave alone (a row of no sequence, or a
// position outside [0, max_seqlen), which is reported).
__device__ __forceinline__ int position(const QkNormParams& p, int row) {
  if (!p.positions) return 0;
  const int pos = __ldg(p.positions + row);
  if (pos >= 0 && pos < p.max_seqlen) return pos;
  if (pos != -1) atomicCAS(p.status, 0, NE_DEV_BAD_SEQLEN);
  return -1;
}
}  // namespace qkn

namespace qkn {
constexpr int kFwdThreads = 64;
constexpr int kFwdQuads = kFwdThreads / kParts;

// The lane's chunks of w, 8 dims each, times r.
__device__ __forceinline__ void scale8(float (&x)[8], const uint4& w, float r) {
  float v[8];
  unpack8(w, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = x[i] * r * v[i];
}
}  // namespace qkn

// A quad takes kHeads heads of a row, `groups` apart (so that neighbouring quads read
// neighbouring heads), all their loads in flight at once: the row's position and its row of
// the table are fetched once for them.
template <int kHeads, int kCtas>
__global__ void __launch_bounds__(qkn::kFwdThreads, kCtas) ne_qk_norm_rope_kernel(const QkNormParams p,
                                                                           uint32_t groups) {
  using namespace qkn;
  pdl_wait();
  const int c = threadIdx.x % kParts;
  const uint32_t unit = blockIdx.x * kFwdQuads + threadIdx.x / kParts;
  const uint32_t at = unit / groups;
  const bool live = at < static_cast<uint32_t>(p.n_tot);
  const long long row = live ? at : p.n_tot - 1;  // (past the end: read, not written)
  const int heads = p.H + p.Hkv, h0 = static_cast<int>(unit - at * groups);
  const int pos = live ? position(p, static_cast<int>(row)) : -1;
  const uint4* q = reinterpret_cast<const uint4*>(p.q + row * p.q_stride) + c;
  const uint4* k = reinterpret_cast<const uint4*>(p.k + row * p.k_stride) + c;
  uint4 lo[kHeads], hi[kHeads];
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    const int h = min(h0 + j * static_cast<int>(groups), heads - 1);
    const uint4* src = h < p.H ? q + h * (kHD / 8) : k + (h - p.H) * (kHD / 8);
    lo[j] = __ldg(src);
    hi[j] = __ldg(src + 4);
  }
  const uint4* qw = reinterpret_cast<const uint4*>(p.qw) + c;
  const uint4* kw = reinterpret_cast<const uint4*>(p.kw) + c;
  const uint4 qw0 = __ldg(qw), qw1 = __ldg(qw + 4), kw0 = __ldg(kw), kw1 = __ldg(kw + 4);
  float4 cs[4];  // (cos, sin) of dims 8c + 2u and 8c + 2u + 1
  if (p.rope.cs) {
    const float4* t = reinterpret_cast<const float4*>(p.rope.cs + static_cast<long long>(max(pos, 0)) * 32) + 4 * c;
#pragma unroll
    for (int u = 0; u < 4; ++u) cs[u] = __ldg(t + u);
  }
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    const int h = h0 + j * static_cast<int>(groups);
    const bool is_k = h >= p.H;
    float a[8], b[8];
    unpack8(lo[j], a);
    unpack8(hi[j], b);
    const float r = rstd_of(a, b, p.eps);
    scale8(a, is_k ? kw0 : qw0, r);
    scale8(b, is_k ? kw1 : qw1, r);
    if (p.rope.cs) turn<false>(a, b, cs);
    if (pos < 0 || h >= heads) continue;
    uint4* dst = reinterpret_cast<uint4*>(is_k ? p.kr + (row * p.Hkv + (h - p.H)) * kHD
                                               : p.qr + (row * p.H + h) * kHD) + c;
    dst[0] = pack8(a);
    dst[4] = pack8(b);
  }
}

namespace qkn {

// One tensor's rows (the queries' or the keys'): gradients dx, and this lane's
// part of dw in acc[16] (dims 8c .. 8c + 7, then 32 + 8c ..).  A quad takes kHeads heads of a
// row at a time, as in the forward.
template <int kThreads, int kHeads>
__device__ __forceinline__ void grad_rows(const QkNormParams& p, const __nv_bfloat16* __restrict__ dr,
                                          const __nv_bfloat16* __restrict__ x, long long x_stride,
                                          const __nv_bfloat16* __restrict__ w, int H,
                                          __nv_bfloat16* __restrict__ dx, long long dx_stride,
                                          int c, int quad, float (&acc)[16]) {
  constexpr uint32_t kQuads = kThreads / kParts;
  const uint4* wr = reinterpret_cast<const uint4*>(w) + c;
  const uint4 wl = __ldg(wr), wh = __ldg(wr + 4);
  const uint32_t groups = (H + kHeads - 1) / kHeads, units = groups * p.n_tot;
  const uint32_t step = gridDim.x * kQuads;
  // (Whole warps take part in the sums over the heads: a quad past the end reads
  // the last row and adds nothing.)
  for (uint32_t u0 = blockIdx.x * kQuads; u0 < units; u0 += step) {
    const uint32_t unit = u0 + quad, at = unit / groups;
    const bool live = at < static_cast<uint32_t>(p.n_tot);
    const long long row = live ? at : p.n_tot - 1;
    const int h0 = static_cast<int>(unit - at * groups);
    const int pos = live ? position(p, static_cast<int>(row)) : -1;
    uint4 xl[kHeads], xh[kHeads], gl[kHeads], gh[kHeads];
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      const int h = min(h0 + j * static_cast<int>(groups), H - 1);
      const uint4* xs = reinterpret_cast<const uint4*>(x + row * x_stride + h * kHD) + c;
      const uint4* gs = reinterpret_cast<const uint4*>(dr + (row * H + h) * kHD) + c;
      xl[j] = __ldg(xs);
      xh[j] = __ldg(xs + 4);
      gl[j] = __ldg(gs);
      gh[j] = __ldg(gs + 4);
    }
    float4 cs[4];
    if (p.rope.cs) {
      const float4* t = reinterpret_cast<const float4*>(p.rope.cs + static_cast<long long>(max(pos, 0)) * 32) + 4 * c;
#pragma unroll
      for (int u = 0; u < 4; ++u) cs[u] = __ldg(t + u);
    }
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      const int h = h0 + j * static_cast<int>(groups);
      const bool there = pos >= 0 && h < H;
      float a[8], b[8], ga[8], gb[8], v[8];
      unpack8(xl[j], a);
      unpack8(xh[j], b);
      unpack8(gl[j], ga);
      unpack8(gh[j], gb);
      const float r = rstd_of(a, b, p.eps);
      if (p.rope.cs) turn<true>(ga, gb, cs);
      float along = 0.f;
      unpack8(wl, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] *= r;
        const float d = ga[i] * a[i];
        acc[i] += there ? d : 0.f;
        ga[i] *= v[i];
        along += d * v[i];
      }
      unpack8(wh, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        b[i] *= r;
        const float d = gb[i] * b[i];
        acc[8 + i] += there ? d : 0.f;
        gb[i] *= v[i];
        along += d * v[i];
      }
      along = head_sum(along) * (1.f / kHD);
      if (!there) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] = r * (ga[i] - a[i] * along);
        b[i] = r * (gb[i] - b[i] * along);
      }
      uint4* dst = reinterpret_cast<uint4*>(dx + row * dx_stride + h * kHD) + c;
      dst[0] = pack8(a);
      dst[4] = pack8(b);
    }
  }
}

// The warp's sum of acc into row[64] (in shared memory), in a fixed order.  (By halves,
// 14 exchanges for these 48: 0.3 us less for 8192 rows of 16 heads, and 3% more for 65,536 of
// 40, whose loop the compiler then arranges otherwise.)
__device__ __forceinline__ void warp_sum(float (&acc)[16], int c, float* row) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
#pragma unroll
    for (int sh = 4; sh < 32; sh <<= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], sh);
    if (lane < kParts) row[(j & 8) * 4 + 8 * c + (j & 7)] = acc[j];
    acc[j] = 0.f;
  }
}
}  // namespace qkn

// Each CTA takes its share of the queries' (row, head) pairs, then of the keys',
// and leaves a partial of each dw; the CTA that arrives last adds them up, in
// their order: one launch, and the same bits whichever CTA is last.
template <int kThreads, int kHeads, int kCtas>
__global__ void __launch_bounds__(kThreads, kCtas) ne_qk_norm_rope_bwd_kernel(const QkNormParams p) {
  using namespace qkn;
  constexpr int kWarps = kThreads / 32;
  __shared__ float sum[kWarps][2][kHD];
  __shared__ int last;
  pdl_wait();
  const int c = threadIdx.x % kParts, quad = threadIdx.x / kParts;
  float acc[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) acc[j] = 0.f;
  float* part = p.part + static_cast<long long>(blockIdx.x) * 2 * kHD;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grad_rows<kThreads, kHeads>(p, p.dqr, p.q, p.q_stride, p.qw, p.H, p.dq, p.dq_stride, c, quad, acc);
  warp_sum(acc, c, sum[warp][0]);
  grad_rows<kThreads, kHeads>(p, p.dkr, p.k, p.k_stride, p.kw, p.Hkv, p.dk, p.dk_stride, c, quad, acc);
  warp_sum(acc, c, sum[warp][1]);
  __syncthreads();
  if (threadIdx.x < 2 * kHD) {  // in the order of the warps
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += sum[w][threadIdx.x / kHD][threadIdx.x % kHD];
    part[threadIdx.x] = s;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();  // the CTA's partials (ordered before this by the barrier), then the arrival
    last = atomicAdd(p.arrived, 1) == static_cast<int>(gridDim.x) - 1;
    if (last) *p.arrived = 0;  // as the next launch wants it
    __threadfence();           // and the other partials after it
  }
  __syncthreads();
  if (!last) return;
  // Thread t: columns 4 (t % 32) .. + 3 of every 16th partial.
  const float4* src = reinterpret_cast<const float4*>(p.part);
  const int n = gridDim.x;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kEach = (kQkNormSms + kWarps - 1) / kWarps;  // all of them on their way at once
  float4 v[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    v[i] = warp + i * kWarps < n ? __ldcg(src + (warp + i * kWarps) * 32 + lane)
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    s.x += v[i].x;
    s.y += v[i].y;
    s.z += v[i].z;
    s.w += v[i].w;
  }
  __shared__ float4 all[kWarps][32];
  all[warp][lane] = s;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float4 v = all[w][lane];
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    float* dw = lane < 16 ? p.dqw : p.dkw;
    reinterpret_cast<float4*>(dw)[lane & 15] = s;
  }
}

size_t qk_norm_part_bytes() { return qkn::kQkNormSms * 2 * kHD * sizeof(float); }

namespace {
template <int kHeads, int kCtas>
cudaError_t launch_forward(const QkNormParams& p, cudaStream_t stream) {
  const uint32_t groups = (p.H + p.Hkv + kHeads - 1) / kHeads;
  const long long units = static_cast<long long>(p.n_tot) * groups;
  return launch_pdl(ne_qk_norm_rope_kernel<kHeads, kCtas>,
                    dim3(static_cast<unsigned>((units + qkn::kFwdQuads - 1) / qkn::kFwdQuads)),
                    dim3(qkn::kFwdThreads), 0, stream, p, groups);
}
}  // namespace

// What a quad takes decides how many bytes are on their way: 80,000 rows of 40 heads take
// 135 us by eight heads, 161 by four, 188 by two, 187 by one (each with the registers and
// CTAs that suit it best, 256 threads).  Few rows are spread wide instead, and eight
// where they leave four slots or more empty are four: 8192 rows of 16 heads 7.5 us by
// eight, 7.8 by four, 8.8 by one.  Small CTAs end and begin one by one, so that loads and
// stores of different rows overlap: of 64 threads 129 us (6.4 TB/s), of 128 130, of 256
// 135; 18,600 rows of 16 heads, outputs of its own each pass, 15.3, 15.5, 16.2.
cudaError_t launch_qk_norm(const QkNormParams& p, int sms, cudaStream_t stream) {
  const int heads = p.H + p.Hkv;
  const long long pairs = static_cast<long long>(p.n_tot) * heads;
  if (pairs < 512LL * sms || heads < 4) return launch_forward<1, 16>(p, stream);
  return (heads + 7) / 8 * 8 - heads < 4 ? launch_forward<8, 8>(p, stream)
                                         : launch_forward<4, 8>(p, stream);
}

namespace {
template <int kThreads, int kHeads, int kCtas>
cudaError_t launch_backward(const QkNormParams& p, int sms, cudaStream_t stream) {
  static_assert(kCtas == 1, "the workspace and the sums of dw have a place for one an SM");
  constexpr int kQuads = kThreads / qkn::kParts;
  const int H = p.H > p.Hkv ? p.H : p.Hkv;
  const long long units = static_cast<long long>(p.n_tot) * ((H + kHeads - 1) / kHeads);
  long long ctas = (units + kQuads - 1) / kQuads;
  if (sms > qkn::kQkNormSms) sms = qkn::kQkNormSms;
  if (ctas > kCtas * sms) ctas = kCtas * sms;
  return launch_pdl(ne_qk_norm_rope_bwd_kernel<kThreads, kHeads, kCtas>, dim3(static_cast<unsigned>(ctas)),
                    dim3(kThreads), 0, stream, p);
}
}  // namespace

// A CTA of 512 threads an SM, two heads a quad: what is in flight is bounded by the
// registers, 128 of each thread.  (65,536 rows of 40 heads, 18,600 and 8192 of 16: 184, 28.5
// and 16.7 us, before the two sums of dw shared a barrier; 384 threads and four heads, the
// table and weights read again for each, 181, 33.7 and 19.5; 384 threads with the next unit's
// rows on their way 199 for the first, through shared memory by asynchronous copies 203;
// the next unit's rows fetched into L2, 194; two CTAs' work an SM, one after the other, 187.)
cudaError_t launch_qk_norm_bwd(const QkNormParams& p, int sms, cudaStream_t stream) {
  return launch_backward<512, 2, 1>(p, sms, stream);
}

}  // namespace ne
