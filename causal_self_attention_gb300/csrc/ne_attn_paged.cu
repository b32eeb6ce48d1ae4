// ne_attn_paged.cu -- attention of one new token per sequence over a paged
// key/value cache, with key/value heads shared by groups of query heads, sm_103a.
//
//   q' = bf16(R(n - 1) q),  s_j = scale * q'.k_j,  j < n = seq_lens[b],
//   lse = log sum_j exp(s_j),  o = sum_j exp(s_j - lse) v_j
// for every query head; query head h reads the cached head h / (H / Hkv).
//
// What bounds it: every cached row is read once and serves the G = H / Hkv
// query heads of its group, 4 G flop a byte in bf16 (8 G in e4m3): the cache's
// bytes, as long as the arithmetic keeps up.  At 6.7 TB/s an SM gets 23 bytes
// a cycle, a bf16 key of a head every 11 cycles; on the CUDA cores G = 8 query
// heads would need 16 FMA cycles for it, so the products run on the tensor
// cores (mma.sync m16n8k16, the group's heads as the 16 rows of A: a tile of
// tcgen05 has 64 rows at the least, and one query row per head fills neither).
//
// Work: the batch's tiles of kTile keys, in the order (sequence, cached head,
// position), are dealt to the CTAs in equal contiguous ranges, whatever the
// sequences' lengths (each CTA forms the prefix sums of the lengths itself).
// A range is a run of segments, each the part of one (sequence, head) that
// falls into it.  A segment that is a whole (sequence, head) is written out
// directly; the parts of one that crosses ranges go to the workspace, and the
// CTA that arrives last joins them by their log-sum-exp, in the order of the
// ranges: one launch, and the same bits whichever CTA is last.
//
// A CTA: warp 4 looks the pages up (32 table entries per load) and keeps a ring
// of kStages tiles in flight -- bf16 through TMA boxes with the 128-byte
// swizzle, e4m3 rows (64 bytes) and their scale bytes as plain bulk copies of
// the contiguous (page, head) block -- and warps 0-3 take kKeys keys of each
// tile.  A warp keeps its own online softmax (running maximum, sum, output in
// registers; the maximum moves only when a score exceeds it by 2^8, so that the
// output is rarely rescaled); the four meet at the end of a segment.
//
// bf16: scores in fp32, weights rounded to bf16 for the product with v.
// e4m3: the bytes become halves (exact, one instruction for two), q' is scaled
//   by a power of two into the halves' range (exact but for elements 2^-14 of
//   the largest, off by 2^-25 of it), and a key's scale multiplies its score.
//   A value row's scale is 2^ev: the weight that the product takes is
//   2^(s + ev - m2) with a maximum m2 of its own, so that it is at most 2^8 and
//   loses nothing however far the rows' scales are apart; the sum of weights
//   runs against the scores' own maximum m.  Rounding to half: 2^-11.
//
// Keys of a tile past the sequence's end (what the page holds there, or an
// older tile's bytes) get the score -inf, and their value rows are cleared in
// shared memory, as 0 * NaN would show.
#include "ne_paged.cuh"
#include "ne_sm100.cuh"

namespace ne {

namespace paged {
constexpr int kWarps = 4;                      // consumers
constexpr int kThreads = (kWarps + 1) * 32;    // and the loading warp
constexpr int kStages = 5;
constexpr int kMaxBatch = 1024;                // sequences per launch (prefix sums in shared memory)
constexpr int kCtasPerSm = 2;
constexpr int kMaxParts = 64;                  // parts of one (sequence, head)
constexpr int kPartRow = 68;                   // floats: lse (log2 units), 3 pad, o[64]
constexpr float kBad = INFINITY;               // lse of a part that met a page outside the pool

template <bool kE4m3>
struct Tile {
  static constexpr int kKeys = kE4m3 ? 32 : 16;         // of a warp
  static constexpr int kTile = kWarps * kKeys;          // 128 / 64 keys
  static constexpr int kRowBytes = kE4m3 ? kHD : 2 * kHD;
  static constexpr int kPool = kTile * kRowBytes;       // 8 KiB of K, and of V
  static constexpr int kStageBytes = 2 * kPool + (kE4m3 ? 2 * kTile : 0);
};

template <bool kE4m3, int kRows>
struct Smem {
  static constexpr int OFF_RED = kStages * Tile<kE4m3>::kStageBytes;
  static constexpr int kRedRow = kHD + 4;                // m, l, m2, pad, o[64]
  static constexpr int OFF_PREFIX = OFF_RED + kWarps * kRows * kRedRow * 4;
  static constexpr int OFF_BAR = OFF_PREFIX + (kMaxBatch + 2) * 4;
  static constexpr int BYTES = OFF_BAR + 2 * kStages * 8 + kStages * 4 + 32 + 1024;
};

struct Params {
  PagedCache pc;
  const __nv_bfloat16* q;
  const int* seq_lens;
  int B, H;
  int group;     // query heads per cached head
  int row_tiles; // groups of at most kRows query heads per cached head
  RopeTable rope;
  float scale_log2;
  float* part;   // [workers][2][kRows][kPartRow]
  int* arrived;  // [workers], zero before and after the launch
  __nv_bfloat16* out;
  float* lse;
  int* status;
};

// The part of one unit -- (sequence, cached head, row tile) -- in a range.
struct Segment {
  int b, j;       // sequence; unit of the sequence (cached head * row_tiles + row tile)
  int t0, t1;     // its tiles
  int n_tiles;    // of the whole unit
  long long at;   // flat index of the unit's first tile
};

// The flat tile order: sequence b's tiles start at prefix[b] * J, unit j's at
// + j * tiles(b).
__device__ __forceinline__ Segment segment_at(const int* prefix, int B, int J, long long x,
                                              long long end) {
  const int y = static_cast<int>(x / J);
  int lo = 0, hi = B;  // prefix[lo] <= y < prefix[hi]: the last such lo has tiles
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= y) lo = mid; else hi = mid;
  }
  Segment s;
  s.b = lo;
  s.n_tiles = prefix[lo + 1] - prefix[lo];
  const long long first = static_cast<long long>(prefix[lo]) * J;
  const long long rem = x - first;
  s.j = static_cast<int>(rem / s.n_tiles);
  s.t0 = static_cast<int>(rem - static_cast<long long>(s.j) * s.n_tiles);
  s.at = first + static_cast<long long>(s.j) * s.n_tiles;
  const long long left = end - x;
  s.t1 = static_cast<int>(left < s.n_tiles - s.t0 ? s.t0 + left : s.n_tiles);
  return s;
}

// D += A * B, m16n8k16, fp32 accumulators; A row-major, B column-major.
template <bool kHalf>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (kHalf)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Key of a warp's e4m3 slice that stands at column n of score tile u (8 columns
// each).  A lane's columns 2c, 2c + 1 of a pair of tiles are rows c, 4 + (c ^ 1),
// 8 + c, 12 + (c ^ 1) of the pair's 16: the two rows that a quarter warp reads of
// K then differ in parity (64-byte rows: all banks once), and the four lanes c
// read neighbouring rows of V.
__device__ __forceinline__ int e4m3_key(int u, int n) {
  const int c = n >> 1;
  return 8 * u + ((n & 1) ? 4 + (c ^ 1) : c);
}
}  // namespace paged

template <bool kE4m3, int kRows>
__global__ void __launch_bounds__(paged::kThreads, paged::kCtasPerSm)
    ne_attn_paged_kernel(const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const paged::Params p) {
  using namespace paged;
  using T = Tile<kE4m3>;
  using L = Smem<kE4m3, kRows>;
  constexpr int kHalves = kRows / 8;     // accumulator row halves in use
  constexpr int kScoreTiles = T::kKeys / 8;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  int* prefix = reinterpret_cast<int*>(smem + L::OFF_PREFIX);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* empty = full + kStages;
  volatile int* stage_bad = reinterpret_cast<volatile int*>(empty + kStages);
  volatile int* abort_flag = stage_bad + kStages;
  volatile int* last_flag = abort_flag + 1;
  float* red = reinterpret_cast<float*>(smem + L::OFF_RED);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kWarps);
    }
    *abort_flag = 0;
    mbar_fence_init();
  }
  pdl_wait();  // whatever wrote q, the lengths and the cache has completed
  pdl_launch_dependents();

  // Tiles of every sequence, then their prefix sums.
  const int B = p.B, J = p.pc.Hkv * p.row_tiles;
  for (int b = tid; b < B; b += kThreads) {
    const int n = __ldg(p.seq_lens + b);
    const bool ok = n >= 0 && n <= p.pc.max_seqlen;
    if (!ok && blockIdx.x == 0) atomicCAS(p.status, 0, NE_DEV_BAD_SEQLEN);
    prefix[b + 1] = ok ? (n + T::kTile - 1) / T::kTile : 0;
  }
  __syncthreads();
  int units = 0;  // with something to attend to
  if (warp == 0) {
    int carry = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
      int v = b0 + lane < B ? prefix[b0 + lane + 1] : 0;
      units += __popc(__ballot_sync(0xffffffffu, v > 0));
#pragma unroll
      for (int sh = 1; sh < 32; sh <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, sh);
        if (lane >= sh) v += u;
      }
      if (b0 + lane < B) prefix[b0 + lane + 1] = carry + v;
      carry += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) {
      prefix[0] = 0;
      prefix[kMaxBatch + 1] = units;
    }
  }
  __syncthreads();
  units = prefix[kMaxBatch + 1];
  // Sequences with nothing to attend to (and bad ones): zero, -inf.
  for (int b = blockIdx.x; b < B; b += gridDim.x)
    if (prefix[b + 1] == prefix[b]) {
      uint32_t* o = reinterpret_cast<uint32_t*>(p.out + static_cast<long long>(b) * p.H * kHD);
      for (int i = tid; i < p.H * (kHD / 2); i += kThreads) o[i] = 0u;
      for (int i = tid; i < p.H; i += kThreads) p.lse[static_cast<long long>(b) * p.H + i] = -INFINITY;
    }
  const long long total = static_cast<long long>(prefix[B]) * J;
  const long long most = static_cast<long long>(units) * J * kMaxParts;
  long long W = gridDim.x;
  W = W < total ? W : total;
  W = W < most ? W : most;
  const long long w = blockIdx.x;
  if (w >= W) return;
  const long long x0 = total * w / W, x1 = total * (w + 1) / W;

  if (warp == kWarps) {
    // ------------------------------------------------------------ the loads
    if constexpr (!kE4m3) {
      if (lane == 0) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
      }
    }
    const int page_size = 1 << p.pc.page_shift;
    const int box = page_size < T::kTile ? page_size : T::kTile;  // keys per copy
    bool ok = true;
    int g = 0;  // tiles loaded
    for (long long x = x0; ok && x < x1;) {
      const Segment s = segment_at(prefix, B, J, x, x1);
      x += s.t1 - s.t0;
      const int hk = s.j / p.row_tiles;
      const int n = __ldg(p.seq_lens + s.b);
      const int pages = (n + page_size - 1) >> p.pc.page_shift;
      const int* table = p.pc.block_table + static_cast<long long>(s.b) * p.pc.max_pages;
      int have = -1, id = 0;  // lane i holds the entry of page have + i
      for (int t = s.t0; t < s.t1; ++t, ++g) {
        const int key0 = t * T::kTile;
        const int pg0 = key0 >> p.pc.page_shift;
        const int pg1 = min((key0 + T::kTile - 1) >> p.pc.page_shift, pages - 1);
        if (have < 0 || pg1 >= have + 32) {
          have = pg0;
          id = __ldg(table + min(pg0 + lane, pages - 1));
        }
        const int st = g % kStages;
        if (g >= kStages && !mbar_wait_warp(&empty[st], ((g - kStages) / kStages) & 1, abort_flag,
                                            p.status, 60)) {
          ok = false;
          break;
        }
        const bool mine = have + lane >= pg0 && have + lane <= pg1;
        const bool bad = __any_sync(0xffffffffu, mine && (id < 0 || id >= p.pc.n_pages));
        uint8_t* sk = smem + st * T::kStageBytes;
        uint8_t* sv = sk + T::kPool;
        if (lane == 0) {
          stage_bad[st] = bad;
          if (bad) atomicCAS(p.status, 0, NE_DEV_BAD_PAGE);
          const uint32_t copies = pg1 - pg0 + 1;
          mbar_arrive_expect_tx(&full[st], copies * box * (2 * T::kRowBytes + (kE4m3 ? 2 : 0)));
        }
        __syncwarp();
        for (int pg = pg0; pg <= pg1; ++pg) {
          int page = __shfl_sync(0xffffffffu, id, pg - have);
          if (page < 0 || page >= p.pc.n_pages) page = 0;  // reported; its rows are not used
          if (lane == 0) {
            const int off = (pg - pg0) * box;  // first key of the copy in the tile
            const long long row =
                kv::pool_row(p.pc, page, hk, page_size < T::kTile ? 0 : key0);
            if constexpr (kE4m3) {
              bulk_load(sk + off * kHD, static_cast<const uint8_t*>(p.pc.k) + row * kHD, box * kHD,
                        &full[st]);
              bulk_load(sv + off * kHD, static_cast<const uint8_t*>(p.pc.v) + row * kHD, box * kHD,
                        &full[st]);
              bulk_load(sv + T::kPool + off, p.pc.k_scale + row, box, &full[st]);
              bulk_load(sv + T::kPool + T::kTile + off, p.pc.v_scale + row, box, &full[st]);
            } else {
              tma_load_2d(sk + off * 128, &tmK, &full[st], 0, static_cast<int>(row));
              tma_load_2d(sv + off * 128, &tmV, &full[st], 0, static_cast<int>(row));
            }
          }
        }
      }
    }
    // After an abort, the copies in flight land before the CTA exits (on the
    // normal path the consumers have waited for them).
    if (!ok || *abort_flag)
      for (int i = (g > kStages ? g - kStages : 0); i < g; ++i) {
        const long long c0 = clock64();
        while (!mbar_try_wait(&full[i % kStages], (i / kStages) & 1) &&
               clock64() - c0 < NE_WAIT_LIMIT_CYCLES) {
        }
      }
    return;
  }

  // -------------------------------------------------------------- consumers
  const int r = lane >> 2, c = lane & 3;  // accumulator row (and r + 8), column pair
  bool ok = true;
  int g = 0;
  for (long long x = x0; x < x1;) {
    const Segment s = segment_at(prefix, B, J, x, x1);
    x += s.t1 - s.t0;
    const int n = __ldg(p.seq_lens + s.b);
    const int hk = s.j / p.row_tiles, h0 = hk * p.group + (s.j - hk * p.row_tiles) * kRows;
    const int rows = min(kRows, (hk + 1) * p.group - h0);  // query heads of this unit

    // q' as A fragments, k-step by k-step; a row past the group reads its last
    // head and is not written.  f[hf]: the factor that turns a product into a
    // score in log2 units.
    uint32_t qa[4][4];
    float f[kHalves];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      if (hf >= kHalves) {
#pragma unroll
        for (int k = 0; k < 4; ++k) qa[k][1] = qa[k][3] = 0u;
        break;
      }
      const int h = h0 + min(r + 8 * hf, rows - 1);
      const uint32_t* row = reinterpret_cast<const uint32_t*>(
          p.q + (static_cast<long long>(s.b) * p.H + h) * kHD);
      // The words of this lane: bf16: k-step k holds dims 16 k + 2 c (+ 1) and
      // + 8 (+ 9).  e4m3: dims 16 c + 4 k .. + 3 (any order of the contraction
      // will do, if K's has it too).  Both with the rotation's partners: bf16
      // in k-step k + 2, e4m3 at the words of dims ^ 32.
      float a[4][4];
      float top = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int d = kE4m3 ? 16 * c + 4 * k + 2 * u : 16 * k + 2 * c + 8 * u;
          const uint32_t me = __ldg(row + d / 2);
          float v0 = bf16lo_to_f32(me), v1 = bf16hi_to_f32(me);
          if (p.rope.cs) {
            const uint32_t other = __ldg(row + (d ^ 32) / 2);
            const float4 t = __ldg(reinterpret_cast<const float4*>(
                p.rope.cs + static_cast<long long>(n - 1) * 32 + (d & 31)));
            const float y0 = bf16lo_to_f32(other), y1 = bf16hi_to_f32(other);
            const float sg = d < 32 ? -1.f : 1.f;
            v0 = __fmaf_rn(v0, t.x, sg * __fmul_rn(y0, t.y));
            v1 = __fmaf_rn(v1, t.z, sg * __fmul_rn(y1, t.w));
          }
          const uint32_t w2 = pack_bf16x2(v0, v1);  // the operator's q'
          if constexpr (kE4m3) {
            a[k][2 * u] = bf16lo_to_f32(w2);
            a[k][2 * u + 1] = bf16hi_to_f32(w2);
            top = fmaxf(top, fmaxf(fabsf(a[k][2 * u]), fabsf(a[k][2 * u + 1])));
          } else {
            qa[k][2 * u + hf] = w2;
          }
        }
      f[hf] = p.scale_log2;
      if constexpr (kE4m3) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^-e with 2^e <= top < 2^(e+1): |q' 2^-e| < 2.  (0 and what is not
        // finite or normal keep 1.)
        const uint32_t eb = (__float_as_uint(top) >> 23) & 255u;
        const bool plain = eb >= 1u && eb <= 253u;
        const float down = plain ? __uint_as_float((254u - eb) << 23) : 1.f;
        f[hf] *= plain ? __uint_as_float(eb << 23) : 1.f;
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int u = 0; u < 2; ++u)
            qa[k][2 * u + hf] = pack_f16x2(a[k][2 * u] * down, a[k][2 * u + 1] * down);
      }
    }

    float m[kHalves], m2[kHalves], l[kHalves];
    float o[8][4];
#pragma unroll
    for (int hf = 0; hf < kHalves; ++hf) {
      m[hf] = m2[hf] = -INFINITY;
      l[hf] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    bool bad = false;

    for (int t = s.t0; t < s.t1; ++t, ++g) {
      const int st = g % kStages;
      // (A wait that gave up is carried to the segment's vote.)
      if (!ok || !(ok = mbar_wait_warp(&full[st], (g / kStages) & 1, abort_flag, p.status, 61)))
        continue;
      bad |= stage_bad[st] != 0;
      uint8_t* sk = smem + st * T::kStageBytes + warp * T::kKeys * T::kRowBytes;
      uint8_t* sv = sk + T::kPool;
      const int live = n - t * T::kTile - warp * T::kKeys;  // of this warp's keys, from the first
      if (live < T::kKeys) {
        // Past the end: clear the value rows (16 bytes a lane and step).
        const int first = max(live, 0) * T::kRowBytes;
        for (int i = first + 16 * lane; i < T::kKeys * T::kRowBytes; i += 512)
          *reinterpret_cast<uint4*>(sv + i) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();  // before the stage's next copy
        __syncwarp();
      }
      float sc[kScoreTiles][4];
#pragma unroll
      for (int u = 0; u < kScoreTiles; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[u][e] = 0.f;
      float ev[kScoreTiles][2];  // e4m3: exponents of the value rows' scales
      if constexpr (kE4m3) {
        const uint8_t* scales = smem + st * T::kStageBytes + 2 * T::kPool + warp * T::kKeys;
        const int kb = scales[lane], vb = scales[T::kTile + lane];
        const float kf = kv::scale_value(kb);
        const float vf = vb == 255 ? __uint_as_float(0x7fc00000u) : static_cast<float>(vb - 127);
#pragma unroll
        for (int u = 0; u < kScoreTiles; ++u) {
          const uint4 w4 = *reinterpret_cast<const uint4*>(sk + e4m3_key(u, r) * kHD + 16 * c);
          const uint32_t ws[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma16816<true>(sc[u], qa[k], kv::e4m3x2_to_f16x2(ws[k]),
                           kv::e4m3x2_to_f16x2(ws[k] >> 16));
        }
#pragma unroll
        for (int u = 0; u < kScoreTiles; ++u)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = e4m3_key(u, 2 * c + e);
            const float ks = __shfl_sync(0xffffffffu, kf, key);
            ev[u][e] = __shfl_sync(0xffffffffu, vf, key);
#pragma unroll
            for (int hf = 0; hf < kHalves; ++hf) sc[u][e + 2 * hf] *= ks * f[hf];
          }
      } else {
        const uint32_t kbase = smem_u32(sk);
#pragma unroll
        for (int u = 0; u < kScoreTiles; ++u)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t kb[4];  // k-steps 2 half, 2 half + 1
            ldsm_x4(kbase + sw128_offset(8 * u + (lane & 7), 4 * half + (lane >> 3)), kb);
            mma16816<false>(sc[u], qa[2 * half], kb[0], kb[1]);
            mma16816<false>(sc[u], qa[2 * half + 1], kb[2], kb[3]);
          }
#pragma unroll
        for (int u = 0; u < kScoreTiles; ++u)
#pragma unroll
          for (int e = 0; e < 2 * kHalves; ++e) sc[u][e] *= f[e >> 1];
      }
      if (live < T::kKeys) {
#pragma unroll
        for (int u = 0; u < kScoreTiles; ++u)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = kE4m3 ? e4m3_key(u, 2 * c + e) : 8 * u + 2 * c + e;
            if (key >= live) {
#pragma unroll
              for (int hf = 0; hf < kHalves; ++hf) sc[u][e + 2 * hf] = -INFINITY;
              if (kE4m3) ev[u][e] = 0.f;
            }
          }
      }
      // Row maxima (of the scores; e4m3 also of score + value exponent) over
      // the row's four lanes; the references move when exceeded by 2^8.
      bool moved = false;
      float alpha[kHalves];
#pragma unroll
      for (int hf = 0; hf < kHalves; ++hf) {
        float mx = -INFINITY, mx2 = -INFINITY;
#pragma unroll
        for (int u = 0; u < kScoreTiles; ++u)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx = fmaxf(mx, sc[u][e + 2 * hf]);
            if (kE4m3) mx2 = fmaxf(mx2, sc[u][e + 2 * hf] + ev[u][e]);
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        if (kE4m3) {
          mx2 = fmaxf(mx2, __shfl_xor_sync(0xffffffffu, mx2, 1));
          mx2 = fmaxf(mx2, __shfl_xor_sync(0xffffffffu, mx2, 2));
        }
        alpha[hf] = 1.f;
        if (mx > m[hf] + 8.f) {  // also the first key (m = -inf)
          const float a = ex2_approx(m[hf] - mx);
          l[hf] *= a;
          if (!kE4m3) alpha[hf] = a;
          m[hf] = mx;
          moved |= !kE4m3;
        }
        if (kE4m3 && mx2 > m2[hf] + 8.f) {
          alpha[hf] = ex2_approx(m2[hf] - mx2);
          m2[hf] = mx2;
          moved = true;
        }
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < 2 * kHalves; ++e) o[i][e] *= alpha[e >> 1];
      }
      // Weights; a row none of whose keys is live yet (m = -inf) takes none.
      uint32_t pw[kScoreTiles][2];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        if (hf >= kHalves) {
#pragma unroll
          for (int u = 0; u < kScoreTiles; ++u) pw[u][1] = 0u;
          break;
        }
        const float ref = m[hf] == -INFINITY ? 0.f : m[hf];
        const float ref2 = m2[hf] == -INFINITY ? 0.f : m2[hf];
#pragma unroll
        for (int u = 0; u < kScoreTiles; ++u) {
          const float s0 = sc[u][2 * hf], s1 = sc[u][2 * hf + 1];
          const float p0 = ex2_approx(s0 - ref), p1 = ex2_approx(s1 - ref);
          l[hf] += p0 + p1;
          if constexpr (kE4m3)
            pw[u][hf] = pack_f16x2(ex2_approx(s0 + ev[u][0] - ref2), ex2_approx(s1 + ev[u][1] - ref2));
          else
            pw[u][hf] = pack_bf16x2(p0, p1);
        }
      }
      // o += P V, 16 keys a step.
#pragma unroll
      for (int k = 0; k < T::kKeys / 16; ++k) {
        const uint32_t pa[4] = {pw[2 * k][0], pw[2 * k][1], pw[2 * k + 1][0], pw[2 * k + 1][1]};
        if constexpr (kE4m3) {
          // Dims 8 r .. 8 r + 7 of the lane's four keys: dim 8 r + i is column
          // r of output tile i.
          uint2 vw[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            vw[i] = *reinterpret_cast<const uint2*>(
                sv + e4m3_key(2 * k + (i >> 1), 2 * c + (i & 1)) * kHD + 8 * r);
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // bytes i of both words: output tiles i and i + 4
            const uint32_t sel = 0x0040u + 0x0011u * i;  // bytes i of the two keys
            const uint32_t b0 = __byte_perm(vw[0].x, vw[1].x, sel);
            const uint32_t b1 = __byte_perm(vw[2].x, vw[3].x, sel);
            const uint32_t d0 = __byte_perm(vw[0].y, vw[1].y, sel);
            const uint32_t d1 = __byte_perm(vw[2].y, vw[3].y, sel);
            mma16816<true>(o[i], pa, kv::e4m3x2_to_f16x2(b0), kv::e4m3x2_to_f16x2(b1));
            mma16816<true>(o[i + 4], pa, kv::e4m3x2_to_f16x2(d0), kv::e4m3x2_to_f16x2(d1));
          }
        } else {
          const uint32_t vbase = smem_u32(sv);
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            uint32_t vb[4];
            ldsm_x4_trans(vbase + sw128_offset(16 * k + (lane & 15), i + (lane >> 4)), vb);
            mma16816<false>(o[i], pa, vb[0], vb[1]);
            mma16816<false>(o[i + 1], pa, vb[2], vb[3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }

    // ---- the segment's end: the four warps' states, then out or a part ----
#pragma unroll
    for (int hf = 0; hf < kHalves; ++hf) {
      l[hf] += __shfl_xor_sync(0xffffffffu, l[hf], 1);
      l[hf] += __shfl_xor_sync(0xffffffffu, l[hf], 2);
      float* dst = red + (warp * kRows + r + 8 * hf) * L::kRedRow;
      if (c == 0) {
        dst[0] = m[hf];
        dst[1] = l[hf];
        dst[2] = kE4m3 ? m2[hf] : m[hf];
        dst[3] = bad ? 1.f : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          dst[4 + (kE4m3 ? 8 * (2 * c + e) + i : 8 * i + 2 * c + e)] = o[i][2 * hf + e];
    }
    if (!named_bar_and(1, kWarps * 32, ok)) break;
    const bool whole = s.t0 == 0 && s.t1 == s.n_tiles;
    // Workers of this unit: the first takes its slot 1, the others slot 0.
    const int w_first = static_cast<int>(((s.at + 1) * W - 1) / total);
    const int w_last = static_cast<int>(((s.at + s.n_tiles) * W - 1) / total);
    float* part = p.part + (static_cast<long long>(w) * 2 + (s.t0 == 0 ? 1 : 0)) * kRows * kPartRow;
    // Eight threads a row, 8 dims each.
    for (int row = tid >> 3; row < rows; row += kWarps * 4) {
      const int d0 = (tid & 7) * 8;
      float M = -INFINITY;
      bool any_bad = false;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) {
        const float* src = red + (v * kRows + row) * L::kRedRow;
        M = fmaxf(M, src[0]);
        any_bad |= src[3] != 0.f;
      }
      const float ref = M == -INFINITY ? 0.f : M;
      float sum = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int v = 0; v < kWarps; ++v) {
        const float* src = red + (v * kRows + row) * L::kRedRow;
        if (src[2] == -INFINITY && src[0] == -INFINITY && src[1] == 0.f) continue;  // no keys
        sum += src[1] * ex2_approx(src[0] - ref);
        const float wt = ex2_approx(src[2] - ref);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += src[4 + d0 + e] * wt;
      }
      const float inv = 1.f / sum;
      const float lse2 = any_bad ? kBad : ref + __log2f(sum);
      if (whole) {
        const long long oh = static_cast<long long>(s.b) * p.H + h0 + row;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (!any_bad)
          v = make_uint4(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv),
                         pack_bf16x2(acc[4] * inv, acc[5] * inv), pack_bf16x2(acc[6] * inv, acc[7] * inv));
        *reinterpret_cast<uint4*>(p.out + oh * kHD + d0) = v;
        if (d0 == 0) p.lse[oh] = any_bad ? -INFINITY : lse2 * 0.69314718055994531f;
      } else {
        float* dst = part + row * kPartRow;
        *reinterpret_cast<float4*>(dst + 4 + d0) =
            make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
        *reinterpret_cast<float4*>(dst + 8 + d0) =
            make_float4(acc[4] * inv, acc[5] * inv, acc[6] * inv, acc[7] * inv);
        if (d0 == 0) dst[0] = lse2;
      }
    }
    if (whole) {
      named_bar_sync(1, kWarps * 32);  // red is free again
      continue;
    }
    __threadfence();
    named_bar_sync(1, kWarps * 32);
    if (tid == 0) {
      const int n_parts = w_last - w_first + 1;
      const bool last = atomicAdd(p.arrived + w_first, 1) == n_parts - 1;
      if (last) p.arrived[w_first] = 0;  // as the next launch wants it
      *last_flag = last;
      __threadfence();
    }
    named_bar_sync(1, kWarps * 32);
    if (!*last_flag) continue;
    // ---- the last to arrive joins the parts, in the workers' order ----
    const int n_parts = w_last - w_first + 1;
    auto part_row = [&](int i, int row) {
      return p.part + (static_cast<long long>(w_first + i) * 2 + (i == 0 ? 1 : 0)) * kRows * kPartRow +
             row * kPartRow;
    };
    for (int row = tid >> 3; row < rows; row += kWarps * 4) {
      const int d0 = (tid & 7) * 8;
      const unsigned lanes = 0xffu << (lane & 24);  // the row's eight threads
      float M = -INFINITY;
      for (int i = tid & 7; i < n_parts; i += 8) M = fmaxf(M, __ldcg(part_row(i, row)));
#pragma unroll
      for (int sh = 1; sh < 8; sh <<= 1) M = fmaxf(M, __shfl_xor_sync(lanes, M, sh));
      const bool any_bad = M == kBad;
      const float ref = M == -INFINITY ? 0.f : M;
      float sum = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int i = 0; i < n_parts; ++i) {
        const float* src = part_row(i, row);
        const float wt = ex2_approx(__ldcg(src) - ref);
        const float4 a = __ldcg(reinterpret_cast<const float4*>(src + 4 + d0));
        const float4 b = __ldcg(reinterpret_cast<const float4*>(src + 8 + d0));
        sum += wt;
        acc[0] += a.x * wt; acc[1] += a.y * wt; acc[2] += a.z * wt; acc[3] += a.w * wt;
        acc[4] += b.x * wt; acc[5] += b.y * wt; acc[6] += b.z * wt; acc[7] += b.w * wt;
      }
      const float inv = 1.f / sum;
      const long long oh = static_cast<long long>(s.b) * p.H + h0 + row;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (!any_bad)
        v = make_uint4(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv),
                       pack_bf16x2(acc[4] * inv, acc[5] * inv), pack_bf16x2(acc[6] * inv, acc[7] * inv));
      *reinterpret_cast<uint4*>(p.out + oh * kHD + d0) = v;
      if (d0 == 0) p.lse[oh] = any_bad ? -INFINITY : (ref + __log2f(sum)) * 0.69314718055994531f;
    }
  }
}

namespace {
using namespace paged;

int paged_rows(int H, int Hkv) { return H / Hkv <= 8 ? 8 : 16; }

// Launched CTAs: no more than the batch can have tiles.
int paged_ctas(long long B, int H, int Hkv, int max_seqlen, bool e4m3, int sms) {
  const int rows = paged_rows(H, Hkv), tile = e4m3 ? Tile<true>::kTile : Tile<false>::kTile;
  const long long units = B * Hkv * ((H / Hkv + rows - 1) / rows);
  const long long tiles = units * ((max_seqlen + tile - 1) / tile);
  const long long full = static_cast<long long>(kCtasPerSm) * sms;
  return static_cast<int>(tiles < full ? tiles : full);
}

template <bool kE4m3, int kRows>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const Params& p, int ctas,
                   cudaStream_t stream) {
  static bool attr_set = false;
  constexpr int bytes = Smem<kE4m3, kRows>::BYTES;
  static_assert(kCtasPerSm * (bytes + 1024) <= 233472, "CTAs of an SM share its 228 KiB");
  if (!attr_set) {
    const cudaError_t e = cudaFuncSetAttribute(
        ne_attn_paged_kernel<kE4m3, kRows>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    attr_set = true;
  }
  return launch_pdl(ne_attn_paged_kernel<kE4m3, kRows>, dim3(ctas), dim3(kThreads), bytes, stream,
                    tk, tv, p);
}
}  // namespace

constexpr int kPagedSms = 160;  // an upper bound on the part's SMs (152), for the workspace's size

size_t paged_part_bytes(int B, int H, int Hkv, int max_seqlen) {
  const long long b = B < kMaxBatch ? B : kMaxBatch;
  const long long n = paged_ctas(b, H, Hkv, max_seqlen, false, kPagedSms);  // the smaller tile
  return static_cast<size_t>(n) * 2 * paged_rows(H, Hkv) * kPartRow * sizeof(float);
}

unsigned paged_box_rows(int page_size) {
  return page_size < Tile<false>::kTile ? page_size : Tile<false>::kTile;
}

size_t paged_counter_bytes() { return kPagedSms * kCtasPerSm * sizeof(int); }

// tmK, tmV: the bf16 pools as [rows, 64] in boxes of paged_box_rows rows
// (unused for e4m3).  arrived: paged_counter_bytes of zeros.
cudaError_t launch_decode_paged(const CUtensorMap& tmK, const CUtensorMap& tmV,
                                const __nv_bfloat16* q, const PagedCache& pc, bool e4m3,
                                const int* seq_lens, int B, int H, const RopeTable& rope,
                                float scale_log2, float* part, int* arrived, __nv_bfloat16* out,
                                float* lse, int sms, int* status, cudaStream_t stream) {
  if (sms > kPagedSms) sms = kPagedSms;
  Params p;
  p.pc = pc;
  p.H = H;
  p.group = H / pc.Hkv;
  const int rows = paged_rows(H, pc.Hkv);
  p.row_tiles = (p.group + rows - 1) / rows;
  p.rope = rope;
  p.scale_log2 = scale_log2;
  p.part = part;
  p.arrived = arrived;
  p.status = status;
  for (int b0 = 0; b0 < B; b0 += kMaxBatch) {
    p.B = B - b0 < kMaxBatch ? B - b0 : kMaxBatch;
    p.q = q + static_cast<long long>(b0) * H * kHD;
    p.seq_lens = seq_lens + b0;
    p.pc.block_table = pc.block_table + static_cast<long long>(b0) * pc.max_pages;
    p.out = out + static_cast<long long>(b0) * H * kHD;
    p.lse = lse + static_cast<long long>(b0) * H;
    const int ctas = paged_ctas(p.B, H, pc.Hkv, pc.max_seqlen, e4m3, sms);
    const cudaError_t e =
        e4m3 ? (rows == 8 ? launch<true, 8>(tmK, tmV, p, ctas, stream)
                          : launch<true, 16>(tmK, tmV, p, ctas, stream))
             : (rows == 8 ? launch<false, 8>(tmK, tmV, p, ctas, stream)
                          : launch<false, 16>(tmK, tmV, p, ctas, stream));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace ne
