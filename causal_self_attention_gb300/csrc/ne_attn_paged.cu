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
// cores: mma.sync m16n8k16 with 16 keys (or 16 dims of v) as its rows and 8
// query heads as its columns (a tile of tcgen05 has 64 rows and wants its
// second operand in shared memory: the weights of a few heads would have to go
// there and back for every tile).
//
// Work: the batch's tiles of kTile keys, in the order (sequence, cached head,
// position), are dealt to the CTAs in equal contiguous ranges, whatever the
// sequences' lengths (each CTA forms the prefix sums of the lengths itself);
// a (sequence, head) counts as kOverhead tiles more than it has, which its
// start and end cost.  A range is a run of segments, each the part of one
// (sequence, head) that falls into it.  A segment that is a whole (sequence,
// head) is written out directly; the parts of one that crosses ranges go to
// the workspace, and the CTA that arrives last joins them by their
// log-sum-exp, in the order of the ranges: one launch, and the same bits
// whichever CTA is last.
//
// A CTA: warp 4 looks the pages up (32 table entries per load) and keeps a ring
// of tiles in flight -- bf16 through TMA boxes with the 128-byte swizzle, e4m3
// rows (64 bytes) and their scale bytes as plain bulk copies of the contiguous
// (page, head) block -- and the next segment's q rows and RoPE table row in a
// ring of their own.  Warps 0-3 take kKeys keys of each tile.  A warp keeps its
// own online softmax (reference maximum, sum, output in registers); a
// reference moves only when some score exceeds it by 2^8, which one vote finds
// out, so that most tiles need neither the maximum over the lanes nor a rescale
// of the output.  The four warps meet at the end of a segment.
//
// bf16: scores in fp32, weights rounded to bf16 for the product with v.
// e4m3: the bytes become halves (exact, one instruction for two), q' is scaled
//   by a power of two into the halves' range (exact but for elements 2^-14 of
//   the largest, off by 2^-25 of it), and a key's scale multiplies its score.
//   A value row's scale is 2^ev: the weight that the product takes is
//   2^(s + ev - m2) with a reference m2 of its own, so that it is at most 2^8 and
//   loses nothing however far the rows' scales are apart; the sum of weights
//   runs against the scores' own reference m.  Rounding to half: 2^-11.
//
// Measured: 16 sequences of 16k, 32 heads on 8, bf16 80.5 us (6.3 TB/s, 94% of the
// copy rate); 64 ragged sequences of 1 to 16k, e4m3, 28.0 us (3.7 TB/s: the
// products, weights and conversions of a key take 43% of the issue slots, and
// the segments' ends, joins and the slowest CTA the rest); one sequence of 777,
// 7.4 us (launch, prefix sums, a short ring, the join).  Tried: four CTAs an SM
// with two stages, three q slots, other overheads (2, 3, 6) and part limits
// (16-256): none faster on all of these.
//
// Keys of a tile past the sequence's end (what the page holds there, or an
// older tile's bytes) get the score -inf, and their value rows are cleared in
// shared memory, as 0 * NaN would show.
#include <algorithm>

#include "ne_paged.cuh"
#include "ne_sm100.cuh"

namespace ne {

namespace paged {
constexpr int kWarps = 4;                      // consumers
constexpr int kThreads = (kWarps + 1) * 32;    // and the loading warp
constexpr int kMaxBatch = 512;                 // sequences per launch (prefix sums in shared memory)
constexpr int kMaxParts = 96;                  // parts of one (sequence, head), about
constexpr int kOverhead = 4;                   // tiles that a segment's start and end cost
constexpr int kPartRow = 68;                   // floats: lse (log2 units), 3 pad, o[64]
constexpr float kBad = INFINITY;               // lse of a part that met a page outside the pool
constexpr int kQRow = 144;                     // bytes of a q row in shared memory (banks)
constexpr int kQSlots = 2;

template <bool kE4m3>
struct Tile {
  static constexpr int kKeys = kE4m3 ? 32 : 16;         // of a warp
  static constexpr int kTile = kWarps * kKeys;          // 128 / 64 keys
  static constexpr int kRowBytes = kE4m3 ? kHD : 2 * kHD;
  static constexpr int kPool = kTile * kRowBytes;       // 8 KiB of K, and of V
  static constexpr int kStageBytes = 2 * kPool + (kE4m3 ? 2 * kTile : 0);
};

template <bool kE4m3, int kRows>
struct Cfg {
  static constexpr int kCtas = kRows == 8 ? 3 : 2;      // per SM
  static constexpr int kStages = kRows == 8 ? 3 : 4;
  static constexpr int OFF_RED = kStages * Tile<kE4m3>::kStageBytes;
  static constexpr int kRedRow = kHD + 4;                // m, l, m2, bad, o[64]
  static constexpr int OFF_Q = OFF_RED + kWarps * kRows * kRedRow * 4;
  static constexpr int kQBytes = kRows * kQRow + 256;    // q rows, one row of the RoPE table
  static constexpr int OFF_PREFIX = OFF_Q + kQSlots * kQBytes;
  static constexpr int OFF_LEN = OFF_PREFIX + (kMaxBatch + 2) * 4;
  static constexpr int OFF_BAR = OFF_LEN + kMaxBatch * 4;
  static constexpr int BYTES = OFF_BAR + 2 * (kStages + kQSlots) * 8 + kStages * 4 + 16 + 1024;
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
  int drop_cta;  // kDrop: whose first tile is never loaded
};

// The part of one unit -- (sequence, cached head, row tile) -- in a range.
struct Segment {
  int b, j;     // sequence; unit of the sequence (cached head * row_tiles + row tile)
  int t0, t1;   // its tiles (t0 >= t1: none, only overhead falls into the range)
  int n_tiles;  // of the whole unit
  int at;       // the flat position of the unit's first tile
  int next;     // the flat position behind the segment
};

// The flat order: sequence b's units start at prefix[b] * J, unit j's at + j *
// cost(b), cost(b) = kOverhead + its tiles, the overhead first.  (Positions are
// below 2^31: the launch sees to it.)
__device__ __forceinline__ void clip_segment(Segment& s, int unit, int x, int end) {
  s.at = unit + kOverhead;
  s.next = min(s.at + s.n_tiles, end);
  s.t0 = max(x - s.at, 0);
  s.t1 = max(s.next - s.at, 0);
}
__device__ __forceinline__ Segment first_segment(const int* prefix, int B, int J, int x, int end) {
  const int y = x / J;
  int lo = 0, hi = B;  // prefix[lo] <= y < prefix[hi]: the last such lo has tiles
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= y) lo = mid; else hi = mid;
  }
  Segment s;
  s.b = lo;
  const int cost = prefix[lo + 1] - prefix[lo], first = prefix[lo] * J;
  s.j = (x - first) / cost;
  s.n_tiles = cost - kOverhead;
  clip_segment(s, first + s.j * cost, x, end);
  return s;
}
// The segment that starts where s ends (s.next < end).
__device__ __forceinline__ void next_segment(Segment& s, const int* prefix, int J, int end) {
  if (++s.j == J) {
    s.j = 0;
    do ++s.b; while (prefix[s.b + 1] == prefix[s.b]);
    s.n_tiles = prefix[s.b + 1] - prefix[s.b] - kOverhead;
  }
  clip_segment(s, s.next, s.next, end);
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
// The transpose of an 8 x 8 matrix of 16-bit values, in the fragment layout
// (lane 4 r + c: row r, columns 2 c and 2 c + 1).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Key of a warp's e4m3 slice that stands in row x of score tile mt (16 rows
// each).  The rows of a lane are then c, 4 + (c ^ 1), 8 + c, 12 + (c ^ 1) as the
// contraction with v wants them in pairs 2 c, 2 c + 1: the two rows that a
// quarter warp reads of K differ in parity (64-byte rows: all banks once), and
// the four lanes c read neighbouring rows of V.
__device__ __forceinline__ int e4m3_key(int mt, int x) {
  const int c = (x & 7) >> 1;
  return 16 * mt + (x & 8) + ((x & 1) ? 4 + (c ^ 1) : c);
}
}  // namespace paged

// kDrop: a tile of one CTA never arrives, for the tests of a wait that runs out.
template <bool kE4m3, int kRows, bool kDrop>
__global__ void __launch_bounds__(paged::kThreads, paged::Cfg<kE4m3, kRows>::kCtas)
    ne_attn_paged_kernel(const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const paged::Params p) {
  using namespace paged;
  using T = Tile<kE4m3>;
  using L = Cfg<kE4m3, kRows>;
  constexpr int kStages = L::kStages;
  constexpr int kNT = kRows / 8;           // column tiles: 8 query heads each
  constexpr int kMT = T::kKeys / 16;       // row tiles of a warp's keys
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  int* prefix = reinterpret_cast<int*>(smem + L::OFF_PREFIX);
  int* lens = reinterpret_cast<int*>(smem + L::OFF_LEN);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* empty = full + kStages;
  uint64_t* qfull = empty + kStages;
  uint64_t* qempty = qfull + kQSlots;
  volatile int* stage_bad = reinterpret_cast<volatile int*>(qempty + kQSlots);
  volatile int* abort_flag = stage_bad + kStages;
  volatile int* last_flag = abort_flag + 1;
  float* red = reinterpret_cast<float*>(smem + L::OFF_RED);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kWarps);
    }
    for (int s = 0; s < kQSlots; ++s) {
      mbar_init(&qfull[s], 1);
      mbar_init(&qempty[s], kWarps);
    }
    *abort_flag = 0;
    mbar_fence_init();
  }
  pdl_wait();  // whatever wrote q, the lengths and the cache has completed

  // The cost of every sequence's units, then their prefix sums.
  const int B = p.B, J = p.pc.Hkv * p.row_tiles;
  for (int b = tid; b < B; b += kThreads) {
    const int n = __ldg(p.seq_lens + b);
    const bool ok = n >= 0 && n <= p.pc.max_seqlen;
    if (!ok && blockIdx.x == 0) atomicCAS(p.status, 0, NE_DEV_BAD_SEQLEN);
    lens[b] = n;
    prefix[b + 1] = ok && n > 0 ? (n + T::kTile - 1) / T::kTile + kOverhead : 0;
  }
  __syncthreads();
  if (warp == 0) {
    int carry = 0, used = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
      int v = b0 + lane < B ? prefix[b0 + lane + 1] : 0;
      used += __popc(__ballot_sync(0xffffffffu, v > 0));
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
      prefix[kMaxBatch + 1] = used;  // sequences with something to attend to
    }
  }
  __syncthreads();
  // Sequences with nothing to attend to (and bad ones): zero, -inf.
  for (int b = blockIdx.x; b < B; b += gridDim.x)
    if (prefix[b + 1] == prefix[b]) {
      uint32_t* o = reinterpret_cast<uint32_t*>(p.out + static_cast<long long>(b) * p.H * kHD);
      for (int i = tid; i < p.H * (kHD / 2); i += kThreads) o[i] = 0u;
      for (int i = tid; i < p.H; i += kThreads) p.lse[static_cast<long long>(b) * p.H + i] = -INFINITY;
    }
  // Equal ranges, of two tiles of work at the least, and at most about kMaxParts
  // to a unit.
  const int total = prefix[B] * J;
  int W = static_cast<int>(gridDim.x);
  if (total / kMaxParts < W) W = min(W, max(1, prefix[kMaxBatch + 1] * J) * kMaxParts);
  const int range = max((total + W - 1) / W, 2);
  const int w = blockIdx.x;
  const int x0 = w * range, x1 = min(x0 + range, total);
  if (x0 >= total) return;

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
    int g = 0, nq = 0;  // tiles, segments loaded
    for (Segment s = first_segment(prefix, B, J, x0, x1);; next_segment(s, prefix, J, x1)) {
      if (s.t0 >= s.t1) {
        if (s.next >= x1) break;
        continue;
      }
      const int hk = s.j / p.row_tiles, h0 = hk * p.group + (s.j - hk * p.row_tiles) * kRows;
      const int rows = min(kRows, (hk + 1) * p.group - h0);
      const int n = lens[s.b];
      const int pages = (n + page_size - 1) >> p.pc.page_shift;
      const int* table = p.pc.block_table + static_cast<long long>(s.b) * p.pc.max_pages;
      int have = (s.t0 * T::kTile) >> p.pc.page_shift;  // lane i holds the entry of page have + i
      int id = __ldg(table + min(have + lane, pages - 1));
      // q rows and the table row of the query's position.
      const int slot = nq % kQSlots;
      if (nq >= kQSlots && !mbar_wait_warp(&qempty[slot], ((nq - kQSlots) / kQSlots) & 1,
                                           abort_flag, p.status, 62)) {
        ok = false;
        break;
      }
      ++nq;
      uint8_t* sq = smem + L::OFF_Q + slot * L::kQBytes;
      if (lane == 0) mbar_arrive_expect_tx(&qfull[slot], rows * 2 * kHD + (p.rope.cs ? 256 : 0));
      __syncwarp();
      if (lane < rows)
        bulk_load(sq + lane * kQRow, p.q + (static_cast<long long>(s.b) * p.H + h0 + lane) * kHD,
                  2 * kHD, &qfull[slot]);
      if (lane == 31 && p.rope.cs)
        bulk_load(sq + kRows * kQRow, p.rope.cs + static_cast<long long>(n - 1) * 32, 256,
                  &qfull[slot]);
      for (int t = s.t0; t < s.t1; ++t, ++g) {
        const int key0 = t * T::kTile;
        const int pg0 = key0 >> p.pc.page_shift;
        const int pg1 = min((key0 + T::kTile - 1) >> p.pc.page_shift, pages - 1);
        if (pg1 >= have + 32) {
          have = pg0;
          id = __ldg(table + min(pg0 + lane, pages - 1));
        }
        const int st = g % kStages;
        if (g >= kStages && !mbar_wait_warp(&empty[st], ((g - kStages) / kStages) & 1, abort_flag,
                                            p.status, 60)) {
          ok = false;
          break;
        }
        // Lane i copies page pg0 + i.
        int page = __shfl_sync(0xffffffffu, id, (pg0 - have + lane) & 31);
        const bool mine = pg0 + lane <= pg1;
        const bool page_ok = page >= 0 && page < p.pc.n_pages;
        if (!page_ok) page = 0;  // reported; its rows are not used
        const bool bad = __any_sync(0xffffffffu, mine && !page_ok);
        if (kDrop && g == 0 && w == p.drop_cta) continue;
        uint8_t* sk = smem + st * T::kStageBytes;
        uint8_t* sv = sk + T::kPool;
        if (lane == 0) {
          stage_bad[st] = bad;
          if (bad) atomicCAS(p.status, 0, NE_DEV_BAD_PAGE);
          const uint32_t copies = pg1 - pg0 + 1;
          mbar_arrive_expect_tx(&full[st], copies * box * (2 * T::kRowBytes + (kE4m3 ? 2 : 0)));
        }
        __syncwarp();
        if (mine) {
          const int off = lane * box;  // first key of the copy in the tile
          const long long row = kv::pool_row(p.pc, page, hk, page_size < T::kTile ? 0 : key0);
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
        __syncwarp();
      }
      if (!ok || s.next >= x1) break;
    }
    // After an abort, the copies in flight land before the CTA exits (on the
    // normal path the consumers have waited for them).
    if (!ok || *abort_flag) {
      const long long c0 = clock64();
      for (int i = (g > kStages ? g - kStages : 0); i < g; ++i)
        while (!mbar_try_wait(&full[i % kStages], (i / kStages) & 1) &&
               clock64() - c0 < NE_WAIT_LIMIT_CYCLES) {
        }
      for (int i = (nq > kQSlots ? nq - kQSlots : 0); i < nq; ++i)
        while (!mbar_try_wait(&qfull[i % kQSlots], (i / kQSlots) & 1) &&
               clock64() - c0 < NE_WAIT_LIMIT_CYCLES) {
        }
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  // Fragments: a lane 4 r + c holds, of the scores, keys r and r + 8 of each row
  // tile and heads 2 c and 2 c + 1 of each column tile; of the output, two dims
  // of each of four row tiles and the same heads.
  const int r = lane >> 2, c = lane & 3;
  bool ok = true;
  int g = 0, nq = 0;
  Segment s = first_segment(prefix, B, J, x0, x1);
  for (bool begun = false;; begun = true) {
    if (begun) {
      if (s.next >= x1) break;
      next_segment(s, prefix, J, x1);
    }
    if (s.t0 >= s.t1) continue;
    const int n = lens[s.b];
    const int hk = s.j / p.row_tiles, h0 = hk * p.group + (s.j - hk * p.row_tiles) * kRows;
    const int rows = min(kRows, (hk + 1) * p.group - h0);  // query heads of this unit

    // q' as B fragments, k-step by k-step; a column past the group takes its
    // last head and is not written.  f: the factor that turns a product into a
    // score in log2 units.
    const int slot = nq % kQSlots;
    ok = ok && mbar_wait_warp(&qfull[slot], (nq / kQSlots) & 1, abort_flag, p.status, 63);
    ++nq;
    uint32_t qb[kNT][4][2];
    float f[kNT][2];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      const uint8_t* sq = smem + L::OFF_Q + slot * L::kQBytes;
      const uint8_t* row = sq + min(8 * nt + r, rows - 1) * kQRow;
      const float* tab = reinterpret_cast<const float*>(sq + kRows * kQRow);
      float a[4][4];
      float top = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          // bf16: k-step k holds dims 16 k + 2 c (+ 1) and + 8 (+ 9).  e4m3:
          // dims 16 c + 4 k .. + 3 (any order of the contraction will do, if
          // K's has it too).
          const int d = kE4m3 ? 16 * c + 4 * k + 2 * u : 16 * k + 2 * c + 8 * u;
          const uint32_t me = *reinterpret_cast<const uint32_t*>(row + 2 * d);
          float v0 = bf16lo_to_f32(me), v1 = bf16hi_to_f32(me);
          if (p.rope.cs) {
            const uint32_t other = *reinterpret_cast<const uint32_t*>(row + 2 * (d ^ 32));
            const float4 t = *reinterpret_cast<const float4*>(tab + 2 * (d & 31));
            const float sg = d < 32 ? -1.f : 1.f;
            v0 = __fmaf_rn(v0, t.x, sg * __fmul_rn(bf16lo_to_f32(other), t.y));
            v1 = __fmaf_rn(v1, t.z, sg * __fmul_rn(bf16hi_to_f32(other), t.w));
          }
          const uint32_t w2 = pack_bf16x2(v0, v1);  // the operator's q'
          if constexpr (kE4m3) {
            a[k][2 * u] = bf16lo_to_f32(w2);
            a[k][2 * u + 1] = bf16hi_to_f32(w2);
            top = fmaxf(top, fmaxf(fabsf(a[k][2 * u]), fabsf(a[k][2 * u + 1])));
          } else {
            qb[nt][k][u] = w2;
          }
        }
      f[nt][0] = f[nt][1] = p.scale_log2;
      if constexpr (kE4m3) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^-e with 2^e <= top < 2^(e+1): |q' 2^-e| < 2.  (0 and what is not
        // finite or normal keep 1.)
        const uint32_t eb = (__float_as_uint(top) >> 23) & 255u;
        const bool plain = eb >= 1u && eb <= 253u;
        const float down = plain ? __uint_as_float((254u - eb) << 23) : 1.f;
        const float up = p.scale_log2 * (plain ? __uint_as_float(eb << 23) : 1.f);  // of head r
        f[nt][0] = __shfl_sync(0xffffffffu, up, 8 * c);
        f[nt][1] = __shfl_sync(0xffffffffu, up, 8 * c + 4);
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int u = 0; u < 2; ++u)
            qb[nt][k][u] = pack_f16x2(a[k][2 * u] * down, a[k][2 * u + 1] * down);
      }
    }
    __syncwarp();
    if (ok && lane == 0) mbar_arrive(&qempty[slot]);

    // References (the same in every lane of a column), sums (this lane's keys).
    float m[kNT][2], m2[kNT][2], l[kNT][2];
    float o[kNT][4][4];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nt][e] = m2[nt][e] = -INFINITY;
        l[nt][e] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
    }
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
      // Scores: [row tile][column tile][key r: heads 2c, 2c+1; key r + 8: the same].
      float sc[kMT][kNT][4];
      float ev[kMT][2];  // e4m3: exponents of the value rows' scales
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[mt][nt][e] = 0.f;
      if constexpr (kE4m3) {
        const uint8_t* scales = smem + st * T::kStageBytes + 2 * T::kPool + warp * T::kKeys;
        const int kb = scales[lane], vb = scales[T::kTile + lane];
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
          const uint4 w0 = *reinterpret_cast<const uint4*>(sk + e4m3_key(mt, r) * kHD + 16 * c);
          const uint4 w1 = *reinterpret_cast<const uint4*>(sk + e4m3_key(mt, r + 8) * kHD + 16 * c);
          const uint32_t ws[2][4] = {{w0.x, w0.y, w0.z, w0.w}, {w1.x, w1.y, w1.z, w1.w}};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t ka[4] = {kv::e4m3x2_to_f16x2(ws[0][k]), kv::e4m3x2_to_f16x2(ws[1][k]),
                                    kv::e4m3x2_to_f16x2(ws[0][k] >> 16),
                                    kv::e4m3x2_to_f16x2(ws[1][k] >> 16)};
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
              mma16816<true>(sc[mt][nt], ka, qb[nt][k][0], qb[nt][k][1]);
          }
        }
        const float kf = kv::scale_value(kb);
        const float vf = vb == 255 ? __uint_as_float(0x7fc00000u) : static_cast<float>(vb - 127);
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int key = e4m3_key(mt, r + 8 * hf);
            const float ks = __shfl_sync(0xffffffffu, kf, key);
            ev[mt][hf] = __shfl_sync(0xffffffffu, vf, key);
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) sc[mt][nt][2 * hf + e] *= ks * f[nt][e];
          }
      } else {
        const uint32_t kbase = smem_u32(sk);
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t ka[4];
            ldsm_x4(kbase + sw128_offset(16 * mt + (lane & 15), 2 * k + (lane >> 4)), ka);
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
              mma16816<false>(sc[mt][nt], ka, qb[nt][k][0], qb[nt][k][1]);
          }
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[mt][nt][e] *= p.scale_log2;
      }
      if (live < T::kKeys) {
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int key = kE4m3 ? e4m3_key(mt, r + 8 * hf) : 16 * mt + r + 8 * hf;
            if (key >= live) {
#pragma unroll
              for (int nt = 0; nt < kNT; ++nt)
                sc[mt][nt][2 * hf] = sc[mt][nt][2 * hf + 1] = -INFINITY;
              if (kE4m3) ev[mt][hf] = 0.f;
            }
          }
      }
      // A score above its reference by more than 2^8 anywhere in the warp (the
      // first keys: m = -inf): move the references to the maxima.
      float mx[kNT][2], mx2[kNT][2];
      bool over = false;
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[nt][e] = mx2[nt][e] = -INFINITY;
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              mx[nt][e] = fmaxf(mx[nt][e], sc[mt][nt][2 * hf + e]);
              if (kE4m3) mx2[nt][e] = fmaxf(mx2[nt][e], sc[mt][nt][2 * hf + e] + ev[mt][hf]);
            }
          over |= mx[nt][e] > m[nt][e] + 8.f;
          if (kE4m3) over |= mx2[nt][e] > m2[nt][e] + 8.f;
        }
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float a = mx[nt][e], b = mx2[nt][e];
#pragma unroll
            for (int sh = 4; sh < 32; sh <<= 1) {
              a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, sh));
              if (kE4m3) b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, sh));
            }
            // (-inf stays until a finite score comes; a factor of 0 / 0 = NaN
            // cannot come up: the new reference is finite or +inf.)
            float up = 1.f;
            if (a > m[nt][e]) {
              up = ex2_approx(m[nt][e] - a);
              l[nt][e] *= up;
              m[nt][e] = a;
            }
            if (kE4m3) {
              up = 1.f;
              if (b > m2[nt][e]) {
                up = ex2_approx(m2[nt][e] - b);
                m2[nt][e] = b;
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              o[nt][i][e] *= up;
              o[nt][i][2 + e] *= up;
            }
          }
      }
      // Weights, transposed into B fragments (keys x heads); a column none of
      // whose keys is live yet (m = -inf) takes none.
      uint32_t pb[kMT][kNT][2];
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        float ref[2], ref2[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          ref[e] = m[nt][e] == -INFINITY ? 0.f : m[nt][e];
          ref2[e] = m2[nt][e] == -INFINITY ? 0.f : m2[nt][e];
        }
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const float s0 = sc[mt][nt][2 * hf], s1 = sc[mt][nt][2 * hf + 1];
            const float p0 = ex2_approx(s0 - ref[0]), p1 = ex2_approx(s1 - ref[1]);
            l[nt][0] += p0;
            l[nt][1] += p1;
            uint32_t w2;
            if constexpr (kE4m3)
              w2 = pack_f16x2(ex2_approx(s0 + ev[mt][hf] - ref2[0]),
                              ex2_approx(s1 + ev[mt][hf] - ref2[1]));
            else
              w2 = pack_bf16x2(p0, p1);
            pb[mt][nt][hf] = transpose8x8(w2);
          }
      }
      // o^T += V^T P^T, 16 keys a step.
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
        if constexpr (kE4m3) {
          // Dims 8 r .. 8 r + 7 of the lane's four keys: row tile i holds dims
          // 8 r + 2 i (row r) and 8 r + 2 i + 1 (row r + 8).
          uint2 vw[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            vw[i] = *reinterpret_cast<const uint2*>(
                sv + e4m3_key(mt, 8 * (i >> 1) + 2 * c + (i & 1)) * kHD + 8 * r);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // Of two keys' words: bytes (2 i, 2 i) then (2 i + 1, 2 i + 1).
            const uint32_t a = i < 2 ? vw[0].x : vw[0].y, b = i < 2 ? vw[1].x : vw[1].y;
            const uint32_t d = i < 2 ? vw[2].x : vw[2].y, e = i < 2 ? vw[3].x : vw[3].y;
            const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
            const uint32_t lo = __byte_perm(a, b, sel), hi = __byte_perm(d, e, sel);
            const uint32_t va[4] = {kv::e4m3x2_to_f16x2(lo), kv::e4m3x2_to_f16x2(lo >> 16),
                                    kv::e4m3x2_to_f16x2(hi), kv::e4m3x2_to_f16x2(hi >> 16)};
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
              mma16816<true>(o[nt][i], va, pb[mt][nt][0], pb[mt][nt][1]);
          }
        } else {
          const uint32_t vbase = smem_u32(sv);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t va[4];
            ldsm_x4_trans(vbase + sw128_offset(16 * mt + ((lane >> 4) << 3) + (lane & 7),
                                               2 * i + ((lane >> 3) & 1)),
                          va);
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
              mma16816<false>(o[nt][i], va, pb[mt][nt][0], pb[mt][nt][1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }

    // ---- the segment's end: the four warps' states, then out or a part ----
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[nt][e];
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, sh);
        float* dst = red + (warp * kRows + 8 * nt + 2 * c + e) * L::kRedRow;
        if (r == 0) {
          dst[0] = m[nt][e];
          dst[1] = sum;
          dst[2] = kE4m3 ? m2[nt][e] : m[nt][e];
          dst[3] = bad ? 1.f : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
            dst[4 + (kE4m3 ? 8 * r + 2 * i + hf : 16 * i + r + 8 * hf)] = o[nt][i][2 * hf + e];
      }
    // A wait that gave up (reported): this segment and the CTA's later ones have no
    // result.  They still count as arrived, as bad parts, so that the counters are
    // zero again after the launch; no further wait is made.
    ok = named_bar_and(1, kWarps * 32, ok);
    const bool whole = s.t0 == 0 && s.t1 == s.n_tiles;
    // Of the workers of a unit the first takes its slot 1, the others slot 0.
    float* part = p.part + (static_cast<long long>(w) * 2 + (s.t0 == 0 ? 1 : 0)) * kRows * kPartRow;
    // Eight threads a row, 8 dims each.
    for (int row = tid >> 3; row < rows; row += kWarps * 4) {
      const int d0 = (tid & 7) * 8;
      float M = -INFINITY;
      bool any_bad = !ok;
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
      float inv = 1.f / sum;
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
        if (sum == 0.f) inv = 0.f;  // scores of -inf alone: a part of weight zero, not NaN
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
    const int w_first = s.at / range, w_last = (s.at + s.n_tiles - 1) / range;
    const int n_parts = w_last - w_first + 1;
    named_bar_sync(1, kWarps * 32);
    if (tid == 0) {
      __threadfence();  // the CTA's part (ordered before this by the barrier), then the arrival
      const bool last = atomicAdd(p.arrived + w_first, 1) == n_parts - 1;
      if (last) p.arrived[w_first] = 0;  // as the next launch wants it
      *last_flag = last;
      __threadfence();  // and the other parts after it
    }
    named_bar_sync(1, kWarps * 32);
    if (!*last_flag) continue;
    // ---- the last to arrive joins the parts ----
    // Eight threads a row, 8 dims each; what threads are left form further
    // groups, and group i takes the parts 8 i .. 8 i + 7, then those 8 groups on
    // (one row's parts in flight at once: a part's latency, not its bytes, is
    // what joining costs).  The order of every sum is fixed by the split.
    const int row_slots = rows <= 1 ? 1 : rows <= 2 ? 2 : rows <= 4 ? 4 : rows <= 8 ? 8 : 16;
    const int groups = kWarps * 4 / row_slots;
    const int group = (tid >> 3) / row_slots, row = (tid >> 3) % row_slots;
    const int d0 = (tid & 7) * 8;
    const unsigned lanes = 0xffu << (lane & 24);  // the row's eight threads
    auto part_row = [&](int i) {
      return p.part + (static_cast<long long>(w_first + i) * 2 + (i == 0 ? 1 : 0)) * kRows * kPartRow +
             min(row, rows - 1) * kPartRow;
    };
    float ref = -INFINITY, sum = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    bool any_bad = false;
    for (int i0 = 8 * group; i0 < n_parts; i0 += 8 * groups) {
      const int i = i0 + (tid & 7);
      float4 va[8], vb[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float* src = part_row(min(i0 + u, n_parts - 1)) + 4 + d0;
        va[u] = __ldcg(reinterpret_cast<const float4*>(src));
        vb[u] = __ldcg(reinterpret_cast<const float4*>(src + 4));
      }
      const float le = __ldcg(part_row(min(i, n_parts - 1)));  // this thread weighs one part
      any_bad |= le == kBad;
      float mx = le;
#pragma unroll
      for (int sh = 1; sh < 8; sh <<= 1) mx = fmaxf(mx, __shfl_xor_sync(lanes, mx, sh));
      if (mx > ref) {
        const float a = ex2_approx(ref - mx);
        sum *= a;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] *= a;
        ref = mx;
      }
      const float mine = ex2_approx(le - (ref == -INFINITY ? 0.f : ref));
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float wt = __shfl_sync(lanes, mine, (lane & 24) + u);
        if (i0 + u >= n_parts) continue;
        sum += wt;
        acc[0] += va[u].x * wt; acc[1] += va[u].y * wt; acc[2] += va[u].z * wt; acc[3] += va[u].w * wt;
        acc[4] += vb[u].x * wt; acc[5] += vb[u].y * wt; acc[6] += vb[u].z * wt; acc[7] += vb[u].w * wt;
      }
    }
#pragma unroll
    for (int sh = 1; sh < 8; sh <<= 1) any_bad |= __shfl_xor_sync(lanes, any_bad, sh);
    float* mine = red + (group * row_slots + row) * L::kRedRow;
    if (d0 == 0) {
      mine[0] = any_bad ? kBad : ref;
      mine[1] = sum;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) mine[4 + d0 + e] = acc[e];
    named_bar_sync(1, kWarps * 32);
    if (group == 0 && row < rows) {
      float M = -INFINITY;
      for (int i = 0; i < groups; ++i) M = fmaxf(M, red[(i * row_slots + row) * L::kRedRow]);
      any_bad = M == kBad;
      const float top = M == -INFINITY ? 0.f : M;
      sum = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = 0.f;
      for (int i = 0; i < groups; ++i) {
        const float* src = red + (i * row_slots + row) * L::kRedRow;
        if (8 * i >= n_parts) break;  // a group without parts
        // (-inf: scores of -inf alone, sums of zero, or NaN; any finite factor will do.)
        const float wt = src[0] == -INFINITY ? 1.f : ex2_approx(src[0] - top);
        sum += src[1] * wt;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += src[4 + d0 + e] * wt;
      }
      const float inv = 1.f / sum;
      const long long oh = static_cast<long long>(s.b) * p.H + h0 + row;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (!any_bad)
        v = make_uint4(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv),
                       pack_bf16x2(acc[4] * inv, acc[5] * inv), pack_bf16x2(acc[6] * inv, acc[7] * inv));
      *reinterpret_cast<uint4*>(p.out + oh * kHD + d0) = v;
      if (d0 == 0) p.lse[oh] = any_bad ? -INFINITY : (top + __log2f(sum)) * 0.69314718055994531f;
    }
    named_bar_sync(1, kWarps * 32);  // red is free again
  }
}

namespace {
using namespace paged;

// Query heads (columns of the products) that a unit takes.  16 where a group has
// more than 8, so that its keys and values are read and converted once: 16 x
// 16k, 16 heads a group, e4m3 24.6 us against 27.9 by two units of 8 (bf16 31.7
// and 31.9: L2 serves the second).  Smaller groups would only pad: a ragged
// e4m3 batch with 4 heads a group 28.1 by 8, 36.9 by 16.
int paged_rows(int H, int Hkv) { return H / Hkv <= 8 ? 8 : 16; }

// Launched CTAs: no more than the batch can have tiles.
int paged_ctas(long long B, int H, int Hkv, int max_seqlen, bool e4m3, int sms) {
  const int rows = paged_rows(H, Hkv), tile = e4m3 ? Tile<true>::kTile : Tile<false>::kTile;
  const long long units = B * Hkv * ((H / Hkv + rows - 1) / rows);
  const long long tiles = units * ((max_seqlen + tile - 1) / tile);
  const long long full =
      static_cast<long long>(rows == 8 ? Cfg<false, 8>::kCtas : Cfg<false, 16>::kCtas) * sms;
  return static_cast<int>(tiles < full ? tiles : full);
}

template <bool kE4m3, int kRows, bool kDrop = false>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const Params& p, int ctas,
                   cudaStream_t stream) {
  constexpr int bytes = Cfg<kE4m3, kRows>::BYTES;
  static_assert(Cfg<kE4m3, kRows>::kCtas * (bytes + 1024) <= 233472,
                "CTAs of an SM share its 228 KiB");
  static bool done[64] = {};
  const cudaError_t e = allow_smem(ne_attn_paged_kernel<kE4m3, kRows, kDrop>, bytes, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(ne_attn_paged_kernel<kE4m3, kRows, kDrop>, dim3(ctas), dim3(kThreads), bytes, stream,
                    tk, tv, p);
}
}  // namespace

// Sequences that a launch takes: what its shared memory holds, and so many that
// their tiles and overheads are numbered in 31 bits (0: not one).
int paged_batch(int H, int Hkv, int max_seqlen) {
  const int rows = paged_rows(H, Hkv), tile = Tile<false>::kTile;  // the smaller tile
  const long long J = static_cast<long long>(Hkv) * ((H / Hkv + rows - 1) / rows);
  const long long one = J * ((max_seqlen + tile - 1) / tile + kOverhead);
  return static_cast<int>(std::min<long long>(kMaxBatch, ((1LL << 31) - (1 << 25)) / one));
}

constexpr int kPagedSms = 160;  // an upper bound on the part's SMs (152), for the workspace's size

size_t paged_part_bytes(int B, int H, int Hkv, int max_seqlen) {
  const long long b = B < kMaxBatch ? B : kMaxBatch;
  const long long n = paged_ctas(b, H, Hkv, max_seqlen, false, kPagedSms);  // the smaller tile
  return static_cast<size_t>(n) * 2 * paged_rows(H, Hkv) * kPartRow * sizeof(float);
}

unsigned paged_box_rows(int page_size) {
  return page_size < Tile<false>::kTile ? page_size : Tile<false>::kTile;
}

size_t paged_counter_bytes() { return kPagedSms * Cfg<false, 8>::kCtas * sizeof(int); }

// tmK, tmV: the bf16 pools as [rows, 64] in boxes of paged_box_rows rows
// (unused for e4m3).  arrived: paged_counter_bytes of zeros.  drop_cta: -1, or (bf16,
// groups of at most 8) the CTA whose first tile is never loaded.
cudaError_t launch_decode_paged(const CUtensorMap& tmK, const CUtensorMap& tmV,
                                const __nv_bfloat16* q, const PagedCache& pc, bool e4m3,
                                const int* seq_lens, int B, int H, const RopeTable& rope,
                                float scale_log2, float* part, int* arrived, __nv_bfloat16* out,
                                float* lse, int sms, int* status, cudaStream_t stream,
                                int drop_cta) {
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
  p.drop_cta = drop_cta;
  if (drop_cta >= 0 && (e4m3 || rows != 8)) return cudaErrorInvalidValue;
  const int batch = paged_batch(H, pc.Hkv, pc.max_seqlen);
  for (int b0 = 0; b0 < B; b0 += batch) {
    p.B = B - b0 < batch ? B - b0 : batch;
    p.q = q + static_cast<long long>(b0) * H * kHD;
    p.seq_lens = seq_lens + b0;
    p.pc.block_table = pc.block_table + static_cast<long long>(b0) * pc.max_pages;
    p.out = out + static_cast<long long>(b0) * H * kHD;
    p.lse = lse + static_cast<long long>(b0) * H;
    const int ctas = paged_ctas(p.B, H, pc.Hkv, pc.max_seqlen, e4m3, sms);
    const cudaError_t e =
        drop_cta >= 0 ? launch<false, 8, true>(tmK, tmV, p, ctas, stream)
        : e4m3 ? (rows == 8 ? launch<true, 8>(tmK, tmV, p, ctas, stream)
                          : launch<true, 16>(tmK, tmV, p, ctas, stream))
             : (rows == 8 ? launch<false, 8>(tmK, tmV, p, ctas, stream)
                          : launch<false, 16>(tmK, tmV, p, ctas, stream));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace ne
