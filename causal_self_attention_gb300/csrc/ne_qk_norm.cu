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
#include "ne_sm100.cuh"

namespace ne {

namespace qkn {
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
// The lane's 8 rotation pairs (a, b) turned by their position's angles, or back.
template <bool kBack>
__device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], const float2* table_row,
                                     int c) {
  const float4* cs = reinterpret_cast<const float4*>(table_row + 8 * c);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const float4 t = __ldg(cs + u);  // (cos, sin) of dims 8c + 2u and 8c + 2u + 1
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
constexpr int kFwdThreads = 256;
constexpr int kFwdQuads = kFwdThreads / kParts;
}  // namespace qkn

// kItems (row, head) pairs per quad, all their loads in flight at once.
template <int kItems>
__global__ void __launch_bounds__(qkn::kFwdThreads) ne_qk_norm_rope_kernel(const QkNormParams p) {
  using namespace qkn;
  pdl_wait();
  const int c = threadIdx.x % kParts, quad = threadIdx.x / kParts;
  const int heads = p.H + p.Hkv;
  const long long items = static_cast<long long>(p.n_tot) * heads;
  const long long first = static_cast<long long>(blockIdx.x) * (kItems * kFwdQuads) + quad;
  uint4 lo[kItems], hi[kItems];
  int row[kItems], head[kItems], pos[kItems];
#pragma unroll
  for (int u = 0; u < kItems; ++u) {
    const long long i = min(first + u * kFwdQuads, items - 1);  // (past the end: not written)
    row[u] = static_cast<int>(i / heads);
    head[u] = static_cast<int>(i - static_cast<long long>(row[u]) * heads);
    const bool is_k = head[u] >= p.H;
    const __nv_bfloat16* x =
        is_k ? p.k + row[u] * p.k_stride + (head[u] - p.H) * kHD : p.q + row[u] * p.q_stride + head[u] * kHD;
    const uint4* src = reinterpret_cast<const uint4*>(x);
    lo[u] = __ldg(src + c);
    hi[u] = __ldg(src + c + 4);
    pos[u] = first + u * kFwdQuads < items ? position(p, row[u]) : -1;
  }
#pragma unroll
  for (int u = 0; u < kItems; ++u) {
    const bool is_k = head[u] >= p.H;
    const uint4* wr = reinterpret_cast<const uint4*>(is_k ? p.kw : p.qw);
    float a[8], b[8], w[8];
    unpack8(lo[u], a);
    unpack8(hi[u], b);
    const float r = rstd_of(a, b, p.eps);
    unpack8(__ldg(wr + c), w);
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = a[i] * r * w[i];
    unpack8(__ldg(wr + c + 4), w);
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = b[i] * r * w[i];
    if (pos[u] < 0) continue;
    if (p.rope.cs) turn<false>(a, b, p.rope.cs + static_cast<long long>(pos[u]) * 32, c);
    __nv_bfloat16* y = is_k ? p.kr + (static_cast<long long>(row[u]) * p.Hkv + (head[u] - p.H)) * kHD
                            : p.qr + (static_cast<long long>(row[u]) * p.H + head[u]) * kHD;
    uint4* dst = reinterpret_cast<uint4*>(y);
    dst[c] = pack8(a);
    dst[c + 4] = pack8(b);
  }
}

namespace qkn {
constexpr int kBwdThreads = 512;
constexpr int kBwdQuads = kBwdThreads / kParts;
constexpr int kBwdWarps = kBwdThreads / 32;

// One tensor's rows (the queries' or the keys'): gradients dx, and this lane's
// part of dw in acc[16] (dims 8c .. 8c + 7, then 32 + 8c ..).
__device__ __forceinline__ void grad_rows(const QkNormParams& p, const __nv_bfloat16* __restrict__ dr,
                                          const __nv_bfloat16* __restrict__ x, long long x_stride,
                                          const __nv_bfloat16* __restrict__ w, int H,
                                          __nv_bfloat16* __restrict__ dx, long long dx_stride,
                                          int c, int quad, float (&acc)[16]) {
  const uint4* wr = reinterpret_cast<const uint4*>(w);
  const uint4 wl = __ldg(wr + c), wh = __ldg(wr + c + 4);
  const long long items = static_cast<long long>(p.n_tot) * H;
  const long long step = static_cast<long long>(gridDim.x) * kBwdQuads;
  // (Whole warps take part in the sums over the heads: a quad past the end reads
  // the last row and adds nothing.)
  for (long long i0 = static_cast<long long>(blockIdx.x) * kBwdQuads; i0 < items; i0 += step) {
    const long long i = min(i0 + quad, items - 1);
    const int row = static_cast<int>(i / H), head = static_cast<int>(i - static_cast<long long>(row) * H);
    const uint4* xs = reinterpret_cast<const uint4*>(x + row * x_stride + head * kHD);
    const uint4* gs = reinterpret_cast<const uint4*>(dr + i * kHD);
    const uint4 x0 = __ldg(xs + c), x1 = __ldg(xs + c + 4);
    const uint4 g0 = __ldg(gs + c), g1 = __ldg(gs + c + 4);
    const int pos = i0 + quad < items ? position(p, row) : -1;
    float a[8], b[8], ga[8], gb[8], v[8];
    unpack8(x0, a);
    unpack8(x1, b);
    unpack8(g0, ga);
    unpack8(g1, gb);
    const float r = rstd_of(a, b, p.eps);
    if (p.rope.cs) turn<true>(ga, gb, p.rope.cs + static_cast<long long>(max(pos, 0)) * 32, c);
    float along = 0.f;
    unpack8(wl, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      a[j] *= r;
      if (pos >= 0) acc[j] += ga[j] * a[j];
      ga[j] *= v[j];
      along += ga[j] * a[j];
    }
    unpack8(wh, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      b[j] *= r;
      if (pos >= 0) acc[8 + j] += gb[j] * b[j];
      gb[j] *= v[j];
      along += gb[j] * b[j];
    }
    along = head_sum(along) * (1.f / kHD);
    if (pos < 0) continue;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      a[j] = r * (ga[j] - a[j] * along);
      b[j] = r * (gb[j] - b[j] * along);
    }
    uint4* dst = reinterpret_cast<uint4*>(dx + row * dx_stride + head * kHD);
    dst[c] = pack8(a);
    dst[c + 4] = pack8(b);
  }
}

// The CTA's sum of acc into row[64] (a partial of dw), in a fixed order.
__device__ __forceinline__ void cta_sum(float (&acc)[16], int c, float (*sum)[kHD], float* row) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
#pragma unroll
    for (int sh = 4; sh < 32; sh <<= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], sh);
    if (lane < kParts) sum[warp][(j & 8) * 4 + 8 * c + (j & 7)] = acc[j];
    acc[j] = 0.f;
  }
  __syncthreads();
  if (threadIdx.x < kHD) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kBwdWarps; ++w) s += sum[w][threadIdx.x];
    row[threadIdx.x] = s;
  }
  __syncthreads();
}
}  // namespace qkn

// Each CTA takes its share of the queries' (row, head) pairs, then of the keys',
// and leaves a partial of each dw; the CTA that arrives last adds them up, in
// their order: one launch, and the same bits whichever CTA is last.
__global__ void __launch_bounds__(qkn::kBwdThreads) ne_qk_norm_rope_bwd_kernel(const QkNormParams p) {
  using namespace qkn;
  __shared__ float sum[kBwdWarps][kHD];
  __shared__ int last;
  pdl_wait();
  const int c = threadIdx.x % kParts, quad = threadIdx.x / kParts;
  float acc[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) acc[j] = 0.f;
  float* part = p.part + static_cast<long long>(blockIdx.x) * 2 * kHD;
  grad_rows(p, p.dqr, p.q, p.q_stride, p.qw, p.H, p.dq, p.dq_stride, c, quad, acc);
  cta_sum(acc, c, sum, part);
  grad_rows(p, p.dkr, p.k, p.k_stride, p.kw, p.Hkv, p.dk, p.dk_stride, c, quad, acc);
  cta_sum(acc, c, sum, part + kHD);
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
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = gridDim.x;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int i = warp; i < n; i += kBwdWarps) {
    const float4 v = __ldcg(src + i * 32 + lane);
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
  }
  __shared__ float4 all[kBwdWarps][32];
  all[warp][lane] = s;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int w = 1; w < kBwdWarps; ++w) {
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

namespace {
constexpr int kQkNormSms = 160;  // an upper bound on the part's SMs (152), for the workspace's size
}

size_t qk_norm_part_bytes() { return kQkNormSms * 2 * kHD * sizeof(float); }

cudaError_t launch_qk_norm(const QkNormParams& p, int sms, cudaStream_t stream) {
  const long long items = static_cast<long long>(p.n_tot) * (p.H + p.Hkv);
  if (items >= 4LL * sms * qkn::kFwdQuads) {
    const long long per = 4 * qkn::kFwdQuads;
    return launch_pdl(ne_qk_norm_rope_kernel<4>, dim3(static_cast<unsigned>((items + per - 1) / per)),
                      dim3(qkn::kFwdThreads), 0, stream, p);
  }
  return launch_pdl(ne_qk_norm_rope_kernel<1>,
                    dim3(static_cast<unsigned>((items + qkn::kFwdQuads - 1) / qkn::kFwdQuads)),
                    dim3(qkn::kFwdThreads), 0, stream, p);
}

cudaError_t launch_qk_norm_bwd(const QkNormParams& p, int sms, cudaStream_t stream) {
  const long long items = static_cast<long long>(p.n_tot) * (p.H > p.Hkv ? p.H : p.Hkv);
  long long ctas = (items + qkn::kBwdQuads - 1) / qkn::kBwdQuads;
  if (sms > kQkNormSms) sms = kQkNormSms;
  if (ctas > sms) ctas = sms;
  return launch_pdl(ne_qk_norm_rope_bwd_kernel, dim3(static_cast<unsigned>(ctas)),
                    dim3(qkn::kBwdThreads), 0, stream, p);
}

}  // namespace ne
