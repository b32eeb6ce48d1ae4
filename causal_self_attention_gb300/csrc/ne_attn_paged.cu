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
// e2m1: as e4m3, in tiles of 64 keys a warp, with other weights: FourBit says which.
//
// Measured: 16 sequences of 16k, 32 heads on 8, bf16 80.5 us (6.3 TB/s, 94% of the
// copy rate); 64 ragged sequences of 1 to 16k, e4m3, 26.8 us (3.9 TB/s: the
// products, weights and conversions of a key take 43% of the issue slots, and
// the segments' ends, joins and the slowest CTA the rest); one sequence of 777,
// 7.4 us (launch, prefix sums, a short ring, the join).  Tried: four CTAs an SM
// with two stages, three q slots, other overheads (2, 3, 6) and part limits
// (16-256): none faster on all of these.
// e2m1: 64 sequences of 16k, 32 heads on 8, 110 us (5.0 TB/s, 73% of the copy rate; a
// byte has four times the keys of bf16, and what bounds a tile is its arithmetic: the
// integer pipe busy half of the time, issue slots 54%, three dependent warps a scheduler);
// 64 ragged ones 31.0 us (2.8 TB/s), 777 keys 8.5 us, 64 of 2000 28.8 us, 96 of 512 19.2,
// 16 of 16k with 16 heads a group 26.8 (a tile of 64 keys by 16 heads spills).  Tried: four
// CTAs an SM with two stages (136, 40, 11 and 37 us: 96 registers spill), tiles of 32
// keys a warp, warps that take tiles of their own without meeting (113, 33 us).
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
constexpr int kMaxJoin = 512;                  // more than CTAs can have a part of one
constexpr int kPartRow = 68;                   // floats: lse (log2 units), 3 pad, o[64]
constexpr float kBad = INFINITY;               // lse of a part that met a page outside the pool
constexpr int kQRow = 144;                     // bytes of a q row in shared memory (banks)
constexpr int kQSlots = 2;
// e2m1: pages from 2^7 keys on come as bulk copies, smaller ones by copies of 16 bytes a
// lane.  (A bulk copy costs 60 cycles and more: 64 sequences of 2000 with pages of 16, 37.4 us
// by bulk copies, 27.9 by lanes; 64 of 16k with pages of 128, 109 and 114 us.)
constexpr int kBulkShift = 7;

template <Kv kType>
struct Tile {
  static constexpr int kKeys = kType == Kv::kBf16 ? 16 : kType == Kv::kE4m3 ? 32 : 64;  // of a warp
  static constexpr int kTile = kWarps * kKeys;                // 64, 128, 256 keys
  static constexpr int kRowBytes = kType == Kv::kE2m1 ? kHD / 2 : kType == Kv::kE4m3 ? kHD : 2 * kHD;
  static constexpr int kScales = kType == Kv::kE2m1 ? 2 : kType == Kv::kE4m3 ? 1 : 0;  // of a row
  static constexpr int kPool = kTile * kRowBytes;             // 8 KiB of K, and of V
  static constexpr int kStageBytes = 2 * kPool + 2 * kScales * kTile;
  static constexpr int kOverhead = kType == Kv::kE2m1 ? 2 : 4;  // tiles that a segment's start and end cost
};

template <Kv kType, int kRows>
struct Cfg {
  static constexpr int kCtas = kRows == 8 ? 3 : 2;      // per SM
  static constexpr int kStages = kRows == 8 ? 3 : 4;
  static constexpr int OFF_RED = kStages * Tile<kType>::kStageBytes;
  // m, l, m2, bad, o[64]; e2m1: m2 above m, behind o the other half's
  static constexpr int kRedRow = kHD + (kType == Kv::kE2m1 ? 8 : 4);
  static constexpr int kScratch = kType == Kv::kE2m1 ? 768 : 0;  // of a warp: FourBit's
  static constexpr int OFF_SCRATCH = OFF_RED + kWarps * kRows * kRedRow * 4;
  static constexpr int OFF_Q = OFF_SCRATCH + kWarps * kScratch;
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
  int least;     // tiles of a range, its units' overheads among them
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
template <int kOverhead>
__device__ __forceinline__ void clip_segment(Segment& s, int unit, int x, int end) {
  s.at = unit + kOverhead;
  s.next = min(s.at + s.n_tiles, end);
  s.t0 = max(x - s.at, 0);
  s.t1 = max(s.next - s.at, 0);
}
template <int kOverhead>
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
  clip_segment<kOverhead>(s, first + s.j * cost, x, end);
  return s;
}
// The segment that starts where s ends (s.next < end).
template <int kOverhead>
__device__ __forceinline__ void next_segment(Segment& s, const int* prefix, int J, int end) {
  if (++s.j == J) {
    s.j = 0;
    do ++s.b; while (prefix[s.b + 1] == prefix[s.b]);
    s.n_tiles = prefix[s.b + 1] - prefix[s.b] - kOverhead;
  }
  clip_segment<kOverhead>(s, s.next, s.next, end);
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

// 16 bytes into shared memory, asynchronously; the lane's arrival once its copies are there.
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
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
// The same for e2m1, whose rows are 32 bytes: the four rows that a half warp reads
// of K (8 bytes a lane) and the four lanes c of V (4 bytes) differ mod 4.
__device__ __forceinline__ int e2m1_key(int mt, int x) {
  const int c = (x & 7) >> 1;
  return 16 * mt + (x & 8) + ((x & 1) ? 4 + (c ^ 2) : c);
}

// The state of a warp's softmax over 4-bit rows, and a tile of 64 keys, two a lane.
//
// Scores: the products with the two halves of a key's row, each with its scale: x = f (s0
// a0 + s1 a1), in log2 units.  The scales are taken 2^-10 down and f 2^10 up: |a| <= 2^9, so
// that no sum overflows before f, however large the keys and small the query.  (f from 2^117
// on: the query's halves are 2^10 up instead.)  Weights p = 2^(x - m), in halves, with a
// reference m that was kHeadroom below the largest score when it was set; for a value row's half h
// they take its scale, p 2^(e_h - E_h), E_h an exponent that the warp keeps, so that a
// weight is formed once and scaled by a product of two halves.  E_h - e_h is 0 .. 7 for
// every row that the warp has seen, zeros aside.  What halves cost is their smallest step, two
// roundings of at most 2^-25 + 2^-26 of 2^(m + E_h) for a key; the key of the largest score
// alone has a term of 2^(m + 8 + E_h - 7), so that it is less than 2^-25 of the largest term.
// Where a score exceeds the reference's by more than 2^7, or an exponent its range, or the
// sequence ends in the tile -- one vote tells --, the tile takes a longer way, on which the
// references move.  Rows whose scales differ by more, and a row of zeros with the largest score
// (which has no term), put the warp into another mode for the rest of the segment: a reference
// of its own for every (query head, half), 2^(x - m + e_h - m2), which loses nothing however far
// the scales are apart.  (Taken from m on: beside a score of 2^24 an exponent would be lost.)
//
// What bounds a tile is the integer pipe: 128 of its conversions take two cycles each,
// so that choices are made by masks and pairs of bytes are looked at together.
template <int kNT>
struct FourBit {
  static constexpr float kNone = -3.402823466e38f;  // no score yet: the lowest number
  static constexpr float kScoreUp = 1024.f;         // what f has more, and the scales less
  static constexpr float kLargeF = 1.6615349947311448e35f;  // 2^117
  static constexpr int kMT = 4;           // row tiles of 16 keys
  static constexpr int kRange = 7;
  static constexpr float kHeadroom = 8.f;  // weights of 2^15 at most: within a half
  // The scale byte of zeros, 2^-100; rows of it or less count as zeros beside rows 2^kFar above.
  static constexpr int kZero = 27, kFar = 32;
  static constexpr int kUnset = -1000;
  static constexpr int kScratch = 16 * kMT * 12;  // a warp's: key scales (float2), value factors
  float m[kNT][2], l[kNT][2];             // l: of this lane's keys
  float o[kNT][4][4];                     // row tiles 0, 1: the first half's dims; 2, 3: the second's
  uint32_t base;                          // E_h + 127 - kRange, as one word's halves
  uint32_t lowest;                        // smallest scale bytes of this lane's rows, 16 bits each
  bool slow;
  float m2[kNT][2][2];                    // slow: o's references, above m

  __device__ __forceinline__ void begin() {
    slow = false;
    set_base(kUnset, kUnset);
    lowest = 0xffffffffu;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nt][e] = kNone;
        m2[nt][e][0] = m2[nt][e][1] = l[nt][e] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
    }
  }
  __device__ __forceinline__ void set_base(int b0, int b1) {
    base = static_cast<uint32_t>(b0 - kRange) + (static_cast<uint32_t>(b1 - kRange) << 16);
  }
  __device__ __forceinline__ int eb(int h) const {  // E_h + 127
    const int low = static_cast<int16_t>(base & 0xffffu);
    return (h ? static_cast<int>(base - static_cast<uint32_t>(low)) >> 16 : low) + kRange;
  }
  // The references as the segment's end wants them.
  __device__ __forceinline__ float ref(int nt, int e) const {
    return m[nt][e] > kNone ? m[nt][e] : -INFINITY;
  }
  __device__ __forceinline__ float above(int nt, int e, int h) const {  // o's, above m
    return slow ? m2[nt][e][h] : static_cast<float>(eb(h) - 127);
  }

  // Where the keys of a lane, j and j + 32, stand: rows r of tiles t = 2 mt + hf and t + 4
  // (row r + 8 hf of score tile mt).
  struct Slots {
    int k, v;  // in a warp's scratch: of its key scales (float2), of its value factors (uint16)
    __device__ __forceinline__ explicit Slots(int lane) {
      const int t = lane >> 3, y = lane & 7;
      const int r = y < 4 ? 2 * y : 2 * ((y - 4) ^ 2) + 1;  // e2m1_key's inverse
      k = 2 * kMT * r + t;
      v = 2 * (2 * kMT * (r >> 1) + t) + (r & 1);
    }
  };
  static constexpr int kOther = 16 * kMT;  // from a half's factors to the other's (uint16)

  // 2^(byte - 127 - E_h) as a half: NaN for a row marked so, zero for zeros far below.
  __device__ __forceinline__ uint32_t factor(int byte, int h) const {
    const int u = byte - eb(h) + kRange;
    return byte == 255 ? 0x7e00u
                       : u >= 0 && u <= kRange ? static_cast<uint32_t>(u + 15 - kRange) << 10 : 0u;
  }
  static __device__ __forceinline__ float column_max(float v) {
#pragma unroll
    for (int sh = 4; sh < 32; sh <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, sh));
    return v;
  }

  __device__ __forceinline__ void add_sums(const float2 (&sum)[kNT]) {
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      l[nt][0] += sum[nt].x;
      l[nt][1] += sum[nt].y;
    }
  }

  __device__ __forceinline__ void turn() {  // o stays as it is, under the reference that it has
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int h = 0; h < 2; ++h) m2[nt][e][h] = above(nt, e, h);
    slow = true;
  }

  // Whether a row of zeros (of a scale far below) has one of the weights w, which are 2^8 for a
  // column's largest score yet; from 2^7 on, or, where scores have coarse steps, from 2^-1.
  __device__ __forceinline__ bool zeros_on_top(const uint32_t (&w)[kMT][kNT][2], const uint16_t* vs,
                                               int live, int r) const {
    uint32_t found = 0u;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      const bool coarse = fmaxf(fabsf(m[nt][0]), fabsf(m[nt][1])) >= 16777216.f;
      const uint32_t up = coarse ? 0x48004800u : 0x28002800u;  // 2^-1 or 2^7 becomes the sign
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int key = e2m1_key(mt, r + 8 * hf);
          const int b0 = vs[key] & 255, b1 = vs[key] >> 8;
          if (key < live && (b0 < eb(0) - kRange || b1 < eb(1) - kRange))
            found |= w[mt][nt][hf] + up;
        }
    }
    return __any_sync(0xffffffffu, (found & 0x80008000u) != 0u);
  }

  // Moves the references to what this tile holds (vb: the scale bytes of this lane's value
  // rows, -1 for none).  Returns whether the mode changed; zeros: this lane has a row of them.
  __device__ __forceinline__ bool move(const float (&x)[kMT][kNT][4], const int (&vb)[2][2],
                                       bool& zeros) {
    bool turned = false;
    zeros = false;
    if (!slow) {
      int hi[2];
      uint32_t low[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        int most = eb(h), least = static_cast<int>(h ? lowest >> 16 : lowest & 0xffffu);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (vb[i][h] != 255) most = max(most, vb[i][h]);
        hi[h] = __reduce_max_sync(0xffffffffu, most);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (vb[i][h] < 0 || vb[i][h] == 255) continue;
          if (vb[i][h] > kZero || hi[h] < kZero + kFar) least = min(least, vb[i][h]);
          zeros |= vb[i][h] < hi[h] - kRange;
        }
        turned |= __reduce_min_sync(0xffffffffu, least) < hi[h] - kRange;
        low[h] = static_cast<uint32_t>(least);
      }
      lowest = low[0] | low[1] << 16;
      if (turned) {
        turn();
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float down = ex2_approx(static_cast<float>(eb(h) - hi[h]));
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int i = 2 * h; i < 2 * h + 2; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[nt][i][e] *= down;
        }
        set_base(hi[0], hi[1]);
      }
    }
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float a = -INFINITY;
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) a = fmaxf(a, fmaxf(x[mt][nt][e], x[mt][nt][2 + e]));
        const float top = column_max(a);
        a = top - kHeadroom;
        if (top - a > 15.f) a = top;  // (steps of 16 there: weights stay within a half)
        if (a > m[nt][e]) {
          const float by = m[nt][e] - a, up = ex2_approx(by);
          m[nt][e] = a;
          l[nt][e] *= up;
          if (slow) {
#pragma unroll
            for (int h = 0; h < 2; ++h) m2[nt][e][h] = fmaxf(m2[nt][e][h] + by, kNone);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              o[nt][i][e] *= up;
              o[nt][i][2 + e] *= up;
            }
          }
        }
      }
    return turned;
  }

  // The other mode: o's references for this tile, ev its value rows' exponents in half h.
  // first: the mode's first tile, where a reference may be far above o's size (exponents of
  // rows without weight made it): there it comes down to that size.
  __device__ __forceinline__ void far_references(const float (&x)[kMT][kNT][4],
                                                 const float (&ev)[kMT][2], int h, bool first) {
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float t = -INFINITY, size = 0.f;
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
            t = fmaxf(t, x[mt][nt][2 * hf + e] - m[nt][e] + ev[mt][hf]);
#pragma unroll
        for (int i = 2 * h; i < 2 * h + 2; ++i)
          size = fmaxf(size, fmaxf(fabsf(o[nt][i][e]), fabsf(o[nt][i][2 + e])));
        t = column_max(t) - kHeadroom;
        const float old = m2[nt][e][h];
        float now = fmaxf(t, old);
        bool empty = false;
        if (first) {
          size = column_max(size);
          empty = size == 0.f;
          now = fmaxf(t, empty ? kNone : old + __log2f(size));
        }
        m2[nt][e][h] = now;
        // (2^(old - now) may leave fp32's range; zero is zero under any reference, also under
        // one so far below that the factor is infinite.)
        const float part = empty ? 1.f : ex2_approx(0.5f * (old - now));
#pragma unroll
        for (int i = 2 * h; i < 2 * h + 2; ++i) {
          o[nt][i][e] = o[nt][i][e] * part * part;
          o[nt][i][2 + e] = o[nt][i][2 + e] * part * part;
        }
      }
  }

  // o^T += V^T P^T, 16 keys.  A word is dims 4 r .. 4 r + 3 of each half of a key's row: row
  // tile i holds the word's byte i, its low value (row r) and its high one (row r + 8).
  // Two keys' low values make a byte, and two keys' high ones.  b: the weights as B
  // fragments (keys x heads) for each half.
  __device__ __forceinline__ void add_values(const uint8_t* sv, int mt, int r, int c,
                                             const uint32_t (&b)[2][kNT][2]) {
    uint32_t vw[4], va[4][4];  // [operand register][row tile]
#pragma unroll
    for (int i = 0; i < 4; ++i)
      vw[i] = *reinterpret_cast<const uint32_t*>(
          sv + e2m1_key(mt, 8 * (i >> 1) + 2 * c + (i & 1)) * (kHD / 2) + 4 * r);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t x = vw[2 * j], y = vw[2 * j + 1];
      kv::e2m1x8_to_f16x2((x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u), va[2 * j]);
      kv::e2m1x8_to_f16x2(((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u), va[2 * j + 1]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v4[4] = {va[0][i], va[1][i], va[2][i], va[3][i]};
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
        mma16816<true>(o[nt][i], v4, b[i >> 1][nt][0], b[i >> 1][nt][1]);
    }
  }

  // 64 keys: rows sk, sv of 32 bytes, scale bytes ks, vs, the first `live` of them the
  // sequence's (what the others hold is finite but for their scales, which are not
  // used).  scratch: kScratch bytes of the warp's own.
  __device__ __forceinline__ void tile(const uint8_t* sk, const uint8_t* sv, const uint16_t* ks,
                                       const uint16_t* vs, uint8_t* scratch, const Slots& at,
                                       int live, const uint32_t (&qb)[kNT][4][2],
                                       const float (&f)[kNT][2], int lane) {
    const int r = lane >> 2, c = lane & 3;
    uint16_t* factors = reinterpret_cast<uint16_t*>(scratch + 128 * kMT);
    uint32_t bytes[2];
    bool longer = live < 16 * kMT;
    longer |= slow;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t kb = ks[lane + 32 * i];
      bytes[i] = vs[lane + 32 * i];
      reinterpret_cast<float2*>(scratch)[at.k + 4 * i] =
          make_float2(kv::scale_value(kb & 255u) * (1.f / kScoreUp),
                      kv::scale_value(kb >> 8) * (1.f / kScoreUp));
      const uint32_t u = __byte_perm(bytes[i], 0u, 0x4140) - base;
      static_assert(kRange == 7, "three bits, and 2^-7 as a half: 8 << 10");
      longer |= (u & 0xfff8fff8u) != 0u;
      const uint32_t two = (u << 10) + 0x20002000u;
      factors[at.v + 8 * i] = static_cast<uint16_t>(two);
      factors[at.v + 8 * i + kOther] = static_cast<uint16_t>(two >> 16);
    }
    __syncwarp();
    float x[kMT][kNT][4];
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
      const uint2 w0 = *reinterpret_cast<const uint2*>(sk + e2m1_key(mt, r) * (kHD / 2) + 8 * c);
      const uint2 w1 = *reinterpret_cast<const uint2*>(sk + e2m1_key(mt, r + 8) * (kHD / 2) + 8 * c);
      uint32_t x0[2][4], x1[2][4];  // [word][byte]: halves of rows r, r + 8
      kv::e2m1x8_to_f16x2(w0.x, x0[0]);
      kv::e2m1x8_to_f16x2(w0.y, x0[1]);
      kv::e2m1x8_to_f16x2(w1.x, x1[0]);
      kv::e2m1x8_to_f16x2(w1.y, x1[1]);
      // (s0, s1) of row r, of row r + 8
      const float4 s = reinterpret_cast<const float4*>(scratch)[kMT * r + mt];
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        float a[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t lo[4] = {x0[k][0], x1[k][0], x0[k][1], x1[k][1]};
          const uint32_t hi[4] = {x0[k][2], x1[k][2], x0[k][3], x1[k][3]};
          mma16816<true>(a[0], lo, qb[nt][k][0], qb[nt][k][1]);
          mma16816<true>(a[1], hi, qb[nt][2 + k][0], qb[nt][2 + k][1]);
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float s0 = hf ? s.z : s.x, s1 = hf ? s.w : s.y;
          const float2 sum = make_float2(__fmaf_rn(a[1][2 * hf], s1, a[0][2 * hf] * s0),
                                         __fmaf_rn(a[1][2 * hf + 1], s1, a[0][2 * hf + 1] * s0));
          const float2 score = mul2(sum, make_float2(f[nt][0], f[nt][1]));
          x[mt][nt][2 * hf] = score.x;
          x[mt][nt][2 * hf + 1] = score.y;
        }
      }
    }
    uint32_t w[kMT][kNT][2];
    float2 sum[kNT];
    uint32_t top;  // halves that are not negative compare as their bits do
    auto weigh = [&]() {
      top = 0u;
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        sum[nt] = make_float2(0.f, 0.f);
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const float2 y = add2(make_float2(x[mt][nt][2 * hf], x[mt][nt][2 * hf + 1]),
                                  make_float2(-m[nt][0], -m[nt][1]));
            const float2 p = make_float2(ex2_approx(y.x), ex2_approx(y.y));
            sum[nt] = add2(sum[nt], p);
            w[mt][nt][hf] = pack_f16x2(p.x, p.y);
            top = __vmaxu2(top, w[mt][nt][hf]);
          }
      }
    };
    weigh();
    longer |= ((top + 0x07ff07ffu) & 0x80008000u) != 0u;  // above 2^15 = 0x7800
    if (__any_sync(0xffffffffu, longer)) {
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
          if (e2m1_key(mt, r + 8 * hf) >= live) {
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) x[mt][nt][2 * hf] = x[mt][nt][2 * hf + 1] = -INFINITY;
          }
      int vb[2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool mine = lane + 32 * i < live;
        vb[i][0] = mine ? static_cast<int>(bytes[i] & 255u) : -1;
        vb[i][1] = mine ? static_cast<int>(bytes[i] >> 8) : -1;
      }
      bool zeros, first = move(x, vb, zeros);
      weigh();
      if (!slow && __any_sync(0xffffffffu, zeros) && zeros_on_top(w, vs, live, r)) {
        turn();
        first = true;
      }
      if (slow) {
        far_values(x, sv, vs, live, first, r, c);
        add_sums(sum);
        return;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          factors[at.v + 8 * i + kOther * h] =
              static_cast<uint16_t>(vb[i][h] < 0 ? 0u : factor(vb[i][h], h));
      __syncwarp();
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        lowest = __vminu2(lowest, __byte_perm(bytes[i], 0u, 0x4140));
    }
    add_sums(sum);
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
      uint32_t b[2][kNT][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint2 fw = reinterpret_cast<const uint2*>(factors + kOther * h)[kMT * c + mt];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          if (h == 0) {
            w[mt][nt][0] = transpose8x8(w[mt][nt][0]);
            w[mt][nt][1] = transpose8x8(w[mt][nt][1]);
          }
          b[h][nt][0] = mul_f16x2(w[mt][nt][0], fw.x);
          b[h][nt][1] = mul_f16x2(w[mt][nt][1], fw.y);
        }
      }
      add_values(sv, mt, r, c, b);
    }
  }

  __device__ __forceinline__ void far_values(const float (&x)[kMT][kNT][4], const uint8_t* sv,
                                             const uint16_t* vs, int live, bool first, int r, int c) {
    float ev[2][kMT][2];
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int key = e2m1_key(mt, r + 8 * hf);
          const int byte = h ? vs[key] >> 8 : vs[key] & 255;
          ev[h][mt][hf] = key >= live ? 0.f : byte == 255 ? NAN : static_cast<float>(byte - 127);
        }
#pragma unroll
    for (int h = 0; h < 2; ++h) far_references(x, ev[h], h, first);
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
      uint32_t b[2][kNT][2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
            b[h][nt][hf] = transpose8x8(pack_f16x2(
                ex2_approx(x[mt][nt][2 * hf] - m[nt][0] + ev[h][mt][hf] - m2[nt][0][h]),
                ex2_approx(x[mt][nt][2 * hf + 1] - m[nt][1] + ev[h][mt][hf] - m2[nt][1][h])));
      add_values(sv, mt, r, c, b);
    }
  }
};
}  // namespace paged

// kDrop: a tile of one CTA never arrives, for the tests of a wait that runs out.
template <Kv kType, int kRows, bool kDrop>
__global__ void __launch_bounds__(paged::kThreads, paged::Cfg<kType, kRows>::kCtas)
    ne_attn_paged_kernel(const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const paged::Params p) {
  using namespace paged;
  using T = Tile<kType>;
  using L = Cfg<kType, kRows>;
  constexpr int kStages = L::kStages;
  constexpr int kNT = kRows / 8;           // column tiles: 8 query heads each
  constexpr bool kE4m3 = kType == Kv::kE4m3, kE2m1 = kType == Kv::kE2m1;
  constexpr bool kF16 = kE4m3 || kE2m1;  // products of halves
  static_assert(!kE2m1 || (L::kScratch == FourBit<kNT>::kScratch && T::kKeys == 16 * FourBit<kNT>::kMT),
                "FourBit's tile");
  constexpr int kMT = T::kKeys / 16;       // row tiles of a warp's keys
  extern __shared__ uint8_t smem_raw[];
  // (An offset, not a rounded address: the loads below stay loads of shared memory.)
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
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
  // Pages far below a tile of e2m1 come by copies of 16 bytes a lane.
  const bool by_lanes = kE2m1 && p.pc.page_shift < kBulkShift;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], by_lanes ? 33 : 1);  // (32 lanes' copies, and what lane 0 says)
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
    prefix[b + 1] = ok && n > 0 ? (n + T::kTile - 1) / T::kTile + T::kOverhead : 0;
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
  // Equal ranges, of p.least tiles of work at the least, and at most about kMaxParts
  // to a unit.
  const int total = prefix[B] * J;
  int W = static_cast<int>(gridDim.x);
  if (total / kMaxParts < W) W = min(W, max(1, prefix[kMaxBatch + 1] * J) * kMaxParts);
  const int range = max((total + W - 1) / W, p.least);
  const int w = blockIdx.x;
  const int x0 = w * range, x1 = min(x0 + range, total);
  if (x0 >= total) return;

  if (warp == kWarps) {
    // ------------------------------------------------------------ the loads
    if constexpr (!kF16) {
      if (lane == 0) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
      }
    }
    const int page_size = 1 << p.pc.page_shift;
    const int box = page_size < T::kTile ? page_size : T::kTile;  // keys per copy
    bool ok = true;
    int g = 0, nq = 0;  // tiles, segments loaded
    for (Segment s = first_segment<T::kOverhead>(prefix, B, J, x0, x1);; next_segment<T::kOverhead>(s, prefix, J, x1)) {
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
      bool seg_bad = false;  // (lane 0's; the consumers ask for it at the segment's last tile)
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
        if constexpr (kE2m1) {
          if (by_lanes) {
            // Lane i: the pool's row of key key0 + 16 i (16 keys are 512 bytes, 16 a lane).
            const int key = key0 + 16 * (lane & 15), pg = min(key >> p.pc.page_shift, pg1);
            int page = __shfl_sync(0xffffffffu, id, (pg - have) & 31);
            const bool page_ok = page >= 0 && page < p.pc.n_pages;
            if (!page_ok) page = 0;  // reported; its rows are not used
            const bool bad = __any_sync(0xffffffffu, !page_ok);
            if (lane == 0) {
              stage_bad[st] = seg_bad |= bad;
              if (bad) atomicCAS(p.status, 0, NE_DEV_BAD_PAGE);
            }
            // (Rows of a pool are numbered in 31 bits.)
            const int row = ((page * p.pc.Hkv + hk) << p.pc.page_shift) + (key & (page_size - 1));
            const uint32_t to = smem_u32(smem + st * T::kStageBytes) + 16 * lane;
            const uint8_t* k_from = static_cast<const uint8_t*>(p.pc.k) + 16 * lane;
            const uint8_t* v_from = static_cast<const uint8_t*>(p.pc.v) + 16 * lane;
            const int some = min(T::kTile, (pages << p.pc.page_shift) - key0) >> 4;
#pragma unroll 4
            for (int i = 0; i < some; ++i) {
              const long long from = static_cast<long long>(__shfl_sync(0xffffffffu, row, i)) * T::kRowBytes;
              copy16(to + 512 * i, k_from + from);
              copy16(to + T::kPool + 512 * i, v_from + from);
            }
            // Scales: 8 keys a lane.
            const long long scale = 2LL * (__shfl_sync(0xffffffffu, row, lane >> 1) + 8 * (lane & 1));
            copy16(to + 2 * T::kPool, p.pc.k_scale + scale);
            copy16(to + 2 * T::kPool + 2 * T::kTile, p.pc.v_scale + scale);
            copies_arrive(&full[st]);
            if (lane == 0) mbar_arrive(&full[st]);
            __syncwarp();
            continue;
          }
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
          stage_bad[st] = seg_bad |= bad;
          if (bad) atomicCAS(p.status, 0, NE_DEV_BAD_PAGE);
          const uint32_t copies = pg1 - pg0 + 1;
          mbar_arrive_expect_tx(&full[st], copies * box * 2 * (T::kRowBytes + T::kScales));
        }
        __syncwarp();
        if (mine) {
          const int off = lane * box;  // first key of the copy in the tile
          const long long row = kv::pool_row(p.pc, page, hk, page_size < T::kTile ? 0 : key0);
          if constexpr (kF16) {
            constexpr int kB = T::kRowBytes, kS = T::kScales;
            bulk_load(sk + off * kB, static_cast<const uint8_t*>(p.pc.k) + row * kB, box * kB,
                      &full[st]);
            bulk_load(sv + off * kB, static_cast<const uint8_t*>(p.pc.v) + row * kB, box * kB,
                      &full[st]);
            bulk_load(sv + T::kPool + off * kS, p.pc.k_scale + row * kS, box * kS, &full[st]);
            bulk_load(sv + T::kPool + (T::kTile + off) * kS, p.pc.v_scale + row * kS, box * kS,
                      &full[st]);
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
  const typename FourBit<kNT>::Slots slots(lane);
  bool ok = true;
  int st = 0, nq = 0;
  uint32_t phase = 0u;  // of the ring's slot st
  Segment s = first_segment<T::kOverhead>(prefix, B, J, x0, x1);
  for (bool begun = false;; begun = true) {
    if (begun) {
      if (s.next >= x1) break;
      next_segment<T::kOverhead>(s, prefix, J, x1);
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
          // K's has it too).  e2m1: k-steps 0, 1 the first half, dims 8 c + 4 k ..,
          // 2, 3 the second.
          const int d = kE2m1   ? 32 * (k >> 1) + 8 * c + 4 * (k & 1) + 2 * u
                        : kE4m3 ? 16 * c + 4 * k + 2 * u
                                : 16 * k + 2 * c + 8 * u;
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
          if constexpr (kF16) {
            a[k][2 * u] = bf16lo_to_f32(w2);
            a[k][2 * u + 1] = bf16hi_to_f32(w2);
            top = fmaxf(top, fmaxf(fabsf(a[k][2 * u]), fabsf(a[k][2 * u + 1])));
          } else {
            qb[nt][k][u] = w2;
          }
        }
      f[nt][0] = f[nt][1] = p.scale_log2;
      if constexpr (kF16) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^-e with 2^e <= top < 2^(e+1): |q' 2^-e| < 2.  (0 and what is not
        // finite or normal keep 1.)
        uint32_t eb = (__float_as_uint(top) >> 23) & 255u;
        if (kE2m1 && eb != 255u) eb = min(max(eb, 1u), 253u);  // (all finite ones: |q' 2^-e| < 4)
        const bool plain = eb >= 1u && eb <= 253u;
        float down = plain ? __uint_as_float((254u - eb) << 23) : 1.f;
        float up = p.scale_log2 * (plain ? __uint_as_float(eb << 23) : 1.f);  // of head r
        if (kE2m1) {  // as FourBit wants it
          if (up >= FourBit<kNT>::kLargeF) down *= FourBit<kNT>::kScoreUp;
          else up *= FourBit<kNT>::kScoreUp;
        }
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
    FourBit<kNT> four;
    if constexpr (kE2m1) four.begin();

    auto advance = [&]() {
      const bool wrap = ++st == kStages;
      st = wrap ? 0 : st;
      phase ^= wrap ? 1u : 0u;
    };
    for (int t = s.t0; t < s.t1; ++t, advance()) {
      // (A wait that gave up is carried to the segment's vote.)
      if (!ok || !(ok = mbar_wait_warp(&full[st], phase, abort_flag, p.status, 61)))
        continue;
      if (t + 1 == s.t1) bad = stage_bad[st] != 0;
      uint8_t* sk = smem + st * T::kStageBytes + warp * T::kKeys * T::kRowBytes;
      uint8_t* sv = sk + T::kPool;
      const int live = n - t * T::kTile - warp * T::kKeys;  // of this warp's keys, from the first
      if constexpr (kE2m1) {
        const uint16_t* scales =
            reinterpret_cast<const uint16_t*>(smem + st * T::kStageBytes + 2 * T::kPool) +
            warp * T::kKeys;
        four.tile(sk, sv, scales, scales + T::kTile,
                  smem + L::OFF_SCRATCH + warp * L::kScratch, slots, live, qb, f, lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
        continue;
      }
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
        float sum = kE2m1 ? four.l[nt][e] : l[nt][e];
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, sh);
        float* dst = red + (warp * kRows + 8 * nt + 2 * c + e) * L::kRedRow;
        if (r == 0) {
          dst[0] = kE2m1 ? four.ref(nt, e) : m[nt][e];
          dst[1] = sum;
          dst[2] = kE2m1 ? four.above(nt, e, 0) : kE4m3 ? m2[nt][e] : m[nt][e];
          dst[3] = bad ? 1.f : 0.f;
          if (kE2m1) dst[4 + kHD] = four.above(nt, e, 1);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
            dst[4 + (kE2m1   ? 32 * (i >> 1) + 4 * r + 2 * (i & 1) + hf
                     : kE4m3 ? 8 * r + 2 * i + hf
                             : 16 * i + r + 8 * hf)] =
                kE2m1 ? four.o[nt][i][2 * hf + e] : o[nt][i][2 * hf + e];
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
      auto no_keys = [](const float* src) {
        return (kE2m1 || src[2] == -INFINITY) && src[0] == -INFINITY && src[1] == 0.f;
      };
#pragma unroll
      for (int v = 0; v < kWarps; ++v) {
        const float* src = red + (v * kRows + row) * L::kRedRow;
        if (!no_keys(src)) sum += src[1] * ex2_approx(src[0] - ref);
      }
      const float lse2 = any_bad ? kBad : ref + __log2f(sum);
      // e2m1: the weights' size, 2^8 and more of a half's headroom, leaves before the values'
      // scales come in, which may be 2^125: the sum's power of two, exact.
      float down = 0.f, inv = 1.f / sum;
      if constexpr (kE2m1) {
        const uint32_t bits = __float_as_uint(sum), eb = bits >> 23;  // (sum >= 0, or NaN)
        if (eb - 1u < 254u) {
          down = static_cast<float>(static_cast<int>(eb) - 126);
          inv = 1.f / __uint_as_float((bits & 0x7fffffu) | 126u << 23);
        }
      }
#pragma unroll
      for (int v = 0; v < kWarps; ++v) {
        const float* src = red + (v * kRows + row) * L::kRedRow;
        if (no_keys(src)) continue;
        const float wt = kE2m1 ? ex2_approx(src[0] - ref + (src[d0 < kHD / 2 ? 2 : 4 + kHD] - down))
                               : ex2_approx(src[2] - ref);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += src[4 + d0 + e] * wt;
      }
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
      if (last) __threadfence();  // and the other parts after it
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
    // e2m1: a sum of up to kMaxJoin rows of values that may fill fp32's range, scaled for it.
    constexpr float kJoin = kE2m1 ? 1.f / kMaxJoin : 1.f;
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
        const float wv = wt * kJoin;
        acc[0] += va[u].x * wv; acc[1] += va[u].y * wv; acc[2] += va[u].z * wv; acc[3] += va[u].w * wv;
        acc[4] += vb[u].x * wv; acc[5] += vb[u].y * wv; acc[6] += vb[u].z * wv; acc[7] += vb[u].w * wv;
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
      const float inv = 1.f / kJoin / sum;
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
int paged_ctas(long long B, int H, int Hkv, int max_seqlen, Kv type, int sms) {
  const int rows = paged_rows(H, Hkv);
  const long long units = B * Hkv * ((H / Hkv + rows - 1) / rows);
  auto of_tile = [&](int tile) { return (max_seqlen + tile - 1) / tile; };
  // (e2m1: a range may be one tile of the flat order, overheads among them; never more than
  // bf16's, which the workspace is sized for.)
  const int each = type == Kv::kE2m1 ? std::min(of_tile(Tile<Kv::kE2m1>::kTile) + Tile<Kv::kE2m1>::kOverhead,
                                                of_tile(Tile<Kv::kBf16>::kTile))
                                     : of_tile(type == Kv::kE4m3 ? Tile<Kv::kE4m3>::kTile : Tile<Kv::kBf16>::kTile);
  const long long tiles = units * each;
  const long long full =
      static_cast<long long>(rows == 8 ? Cfg<Kv::kBf16, 8>::kCtas : Cfg<Kv::kBf16, 16>::kCtas) * sms;
  return static_cast<int>(tiles < full ? tiles : full);
}

// The tiles of a range at the least.  e2m1, whose tiles take 1 us: units of three tiles or
// fewer whole (a join costs 2 us: 4 sequences of 500, 7.4 us whole, 9.1 by single tiles),
// others of up to 18 by single tiles (one sequence of 1000 8.8 us, by two 9.7; 4000 9.4 and
// 10.2), longer ones not (8000 10.5 by two, 10.9 by single tiles; 12000 10.9 and 13.0).  The
// rule goes by the caller's bound on the lengths, which the host knows, not by the lengths:
// with a bound of 16384 one sequence of 777 takes 9.4 us (8.5 to 8.8), of 4000 10.1 (9.0).
int paged_least(int max_seqlen, Kv type) {
  if (type != Kv::kE2m1) return 2;
  const int each = (max_seqlen + Tile<Kv::kE2m1>::kTile - 1) / Tile<Kv::kE2m1>::kTile;
  return each <= 3 ? each + Tile<Kv::kE2m1>::kOverhead : each <= 18 ? 1 : 2;
}

template <Kv kType, int kRows, bool kDrop = false>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const Params& p, int ctas,
                   cudaStream_t stream) {
  constexpr int bytes = Cfg<kType, kRows>::BYTES;
  static_assert(Cfg<kType, kRows>::kCtas * (bytes + 1024) <= 233472,
                "CTAs of an SM share its 228 KiB");
  static bool done[64] = {};
  const cudaError_t e = allow_smem(ne_attn_paged_kernel<kType, kRows, kDrop>, bytes, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(ne_attn_paged_kernel<kType, kRows, kDrop>, dim3(ctas), dim3(kThreads), bytes, stream,
                    tk, tv, p);
}
}  // namespace

// Sequences that a launch takes: what its shared memory holds, and so many that
// their tiles and overheads are numbered in 31 bits (0: not one).
int paged_batch(int H, int Hkv, int max_seqlen) {
  const int rows = paged_rows(H, Hkv), tile = Tile<Kv::kBf16>::kTile;  // the smaller tile
  const long long J = static_cast<long long>(Hkv) * ((H / Hkv + rows - 1) / rows);
  const long long one = J * ((max_seqlen + tile - 1) / tile + Tile<Kv::kBf16>::kOverhead);
  return static_cast<int>(std::min<long long>(kMaxBatch, ((1LL << 31) - (1 << 25)) / one));
}

constexpr int kPagedSms = 160;  // an upper bound on the part's SMs (152), for the workspace's size

size_t paged_part_bytes(int B, int H, int Hkv, int max_seqlen) {
  const long long b = B < kMaxBatch ? B : kMaxBatch;
  const long long n = paged_ctas(b, H, Hkv, max_seqlen, Kv::kBf16, kPagedSms);  // the smaller tile
  return static_cast<size_t>(n) * 2 * paged_rows(H, Hkv) * kPartRow * sizeof(float);
}

unsigned paged_box_rows(int page_size) {
  return page_size < Tile<Kv::kBf16>::kTile ? page_size : Tile<Kv::kBf16>::kTile;
}

static_assert(kPagedSms * Cfg<Kv::kBf16, 8>::kCtas <= kMaxJoin, "parts of a unit");
size_t paged_counter_bytes() { return kPagedSms * Cfg<Kv::kBf16, 8>::kCtas * sizeof(int); }

// tmK, tmV: the bf16 pools as [rows, 64] in boxes of paged_box_rows rows
// (unused for the others).  arrived: paged_counter_bytes of zeros.  drop_cta: -1, or (bf16,
// groups of at most 8) the CTA whose first tile is never loaded.
cudaError_t launch_decode_paged(const CUtensorMap& tmK, const CUtensorMap& tmV,
                                const __nv_bfloat16* q, const PagedCache& pc, Kv type,
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
  p.least = paged_least(pc.max_seqlen, type);
  p.drop_cta = drop_cta;
  if (drop_cta >= 0 && (type != Kv::kBf16 || rows != 8)) return cudaErrorInvalidValue;
  const int batch = paged_batch(H, pc.Hkv, pc.max_seqlen);
  for (int b0 = 0; b0 < B; b0 += batch) {
    p.B = B - b0 < batch ? B - b0 : batch;
    p.q = q + static_cast<long long>(b0) * H * kHD;
    p.seq_lens = seq_lens + b0;
    p.pc.block_table = pc.block_table + static_cast<long long>(b0) * pc.max_pages;
    p.out = out + static_cast<long long>(b0) * H * kHD;
    p.lse = lse + static_cast<long long>(b0) * H;
    const int ctas = paged_ctas(p.B, H, pc.Hkv, pc.max_seqlen, type, sms);
    const cudaError_t e =
        drop_cta >= 0 ? launch<Kv::kBf16, 8, true>(tmK, tmV, p, ctas, stream)
        : type == Kv::kE2m1 ? (rows == 8 ? launch<Kv::kE2m1, 8>(tmK, tmV, p, ctas, stream)
                                         : launch<Kv::kE2m1, 16>(tmK, tmV, p, ctas, stream))
        : type == Kv::kE4m3 ? (rows == 8 ? launch<Kv::kE4m3, 8>(tmK, tmV, p, ctas, stream)
                                         : launch<Kv::kE4m3, 16>(tmK, tmV, p, ctas, stream))
                            : (rows == 8 ? launch<Kv::kBf16, 8>(tmK, tmV, p, ctas, stream)
                                         : launch<Kv::kBf16, 16>(tmK, tmV, p, ctas, stream));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace ne
