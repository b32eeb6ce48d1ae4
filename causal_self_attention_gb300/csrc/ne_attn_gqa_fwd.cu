// ne_attn_gqa_fwd.cu -- forward causal attention over packed prompts with
// key/value heads shared by groups of query heads, sm_103a.
//
//   O_m = sum_{n<=m} softmax_n(scale * q'_m . k'_n) v_n,  LSE_m = log sum exp(...)
// for every query head, query head h with key/value head h / group; q', k'
// rotated beforehand by the pass at the end of this file.  The pipeline is that
// of ne_attn_fwd.cu -- a persistent CTA per SM; per work item two 128-row query
// tiles A and B against shared K', V tiles; S = Q' K'^T and O += P V on tcgen05
// with S, P and O in TMEM; a softmax whose reference maximum moves only when
// exceeded by 2^8 -- with two differences.
//
// * Items.  Where a group has two query heads left, A and B are the same 128
//   rows of those two heads: they share every K'/V tile and end on the same
//   diagonal tile, and a sequence of up to 128 rows still fills both.  The odd
//   head of a group takes two consecutive row tiles.  (An item's tiles that end
//   apart hold each other up: the issuing warps take A and B in turn.)
//
// * Warps 8-11, which have nothing to rotate here, are the epilogue: they wait
//   for an item's last P V, divide by the softmax sums (through shared memory)
//   and store O, while the softmax warps take the next item's scores.
//
// * The items are taken from a counter, longest first, by the thread that loads
//   K', once the loads of the item before are issued (a ring of tiles ahead of
//   the softmax), and handed to the other roles through shared memory.  When
//   every role looked its items up itself -- the list, the sequence's bounds,
//   four divisions -- a softmax warp spent 2,600 cycles an item on it, and items
//   dealt in fixed rounds left the slowest CTA 18% behind the mean (now 8%).
//   (Packed prompts of 64 to 2048 tokens 67.4 -> 63 us; which CTA computes an
//   item does not change its results.)
//
// What bounds it (clock stamps, 16384 tokens): the two softmax warps of an SM
// sub-partition, 1,970 cycles for a step of both, of which the exponential unit
// is busy 1,024 and, with the maxima, the packed products, sums and roundings
// issued beside them, a loop of that arithmetic alone takes 1,500 (a
// probe with two warps a sub-partition).  Each branch in the loop costs more than
// its instructions (the unrolled body is some 10 KB of code): a wait that polls
// once for the whole warp with a 32-bit clock as its limit, phase parity instead
// of a test for the first step, selects for the moving reference, and registers
// enough (192) to spill nothing took a step from 2,300 to 1,970 cycles.  Slower
// were: one arrival a warp (a branch and a reconvergence: 421 against 361 us),
// the maximum of a half row while the other half loads (380), the two tiles'
// exponentials in turns (457 against 413), sixteen softmax warps of half a row
// (507 against 410), the softmax first in the code (424 against 413).
// 357-363 us for 16384 tokens, 12 heads on 2 (1,145 TFLOP/s with the pass); 57 us
// for the packed prompts, 12 heads on 4, of which the pass is 16, the way to the
// first scores 3, and a CTA's six items of four steps each the rest.  (Clearing V
// behind a sequence's end took 55.7 to 57.0, by the test's presence alone: the
// same where it is never true, 57.1 with the epilogue warps clearing, 57.7 before
// the scores.)
//
// Warp roles (512 threads, registers re-split per warpgroup with setmaxnreg):
//   warps 0-3   softmax A: thread t owns row t of tile A (TMEM lane t), 192 regs
//   warps 4-7   softmax B: same for tile B
//   warps 8-11  epilogue, 80 regs
//   warp 12     MMA: allocates TMEM; one elected lane issues S_X = Q_X K^T
//   warp 13     TMA: lane 0 takes the items, loads Q_A, Q_B and the K' ring
//   warp 14     TMA: lane 0 loads the V ring; lane 1 stores whole O tiles
//   warp 15     MMA: clears V behind a sequence's end; one elected lane issues
//               O_X += P_X V; warps 12-15 at 48 regs
// TMEM columns: S_A 0-127, S_B 128-255, O_A 256-319, O_B 320-383,
// P_A 384-447, P_B 448-511 (bf16 pairs: P is the TMEM A operand of P V).
//
// Barrier phases: the K and V rings count key tiles over all items of the CTA;
// S_* / P_FULL / PV_DONE of tile X count the steps of tile X over all items;
// Q_* (per Q buffer), IT_* (per slot), SUM_FULL, O_* count items.
#include <algorithm>

#include "ne_items.cuh"
#include "ne_sm100.cuh"

namespace ne {

namespace gqa {

constexpr int kThreads = 512;
// Registers per thread of each warpgroup after setmaxnreg (launch: 128).
constexpr uint32_t kRegsSoftmax = 192, kRegsEpilogue = 80, kRegsOther = 48;
static_assert(valid_reg_split(kRegsSoftmax, kRegsEpilogue, kRegsOther), "register split");
constexpr int kStages = 5;                            // K ring and V ring
constexpr int kSlots = 4;     // items between the thread that takes them and the roles
constexpr int kReaders = 16;  // of an item: 12 + 2 warps, two lanes of warp 14
constexpr int OFF_Q = 0;                              // 2 buffers x (Q_A, Q_B)
constexpr int OFF_K = OFF_Q + 4 * kTileBytes;         // kStages
constexpr int OFF_V = OFF_K + kStages * kTileBytes;   // kStages
constexpr int OFF_BAR = OFF_V + kStages * kTileBytes;
constexpr int kBarBytes = 512;                // mbarriers, TMEM address, abort flag
constexpr int OFF_SUM = OFF_BAR + kBarBytes;  // the rows' softmax sums, 2 x 128 fp32
constexpr int OFF_ITEM = OFF_SUM + 2 * 128 * 4;  // kSlots items of 8 ints
constexpr int SMEM_BYTES = OFF_ITEM + kSlots * 32 + 1024;  // + slack for 1024-byte alignment
static_assert(SMEM_BYTES <= 232448, "more shared memory than an sm_103 CTA may have");

enum Bar {
  B_Q_FULL = 0,                    // per Q buffer
  B_Q_EMPTY = B_Q_FULL + 2,        // the item's last S MMA and its O tile stores
  B_K_FULL = B_Q_EMPTY + 2,        // kStages
  B_K_EMPTY = B_K_FULL + kStages,  // kStages
  B_V_FULL = B_K_EMPTY + kStages,  // kStages
  B_V_EMPTY = B_V_FULL + kStages,  // kStages
  B_S_FULL = B_V_EMPTY + kStages,  // per tile X
  B_S_FREE = B_S_FULL + 2,
  B_P_FULL = B_S_FREE + 2,
  B_PV_DONE = B_P_FULL + 2,
  B_O_FINAL = B_PV_DONE + 2,       // per tile: the item's last P V completed
  B_O_FREE = B_O_FINAL + 2,        // per tile: the epilogue has read O_X and the sums
  B_SUM_FULL = B_O_FREE + 2,       // per tile: the rows' sums are in shared memory
  B_OST_FULL = B_SUM_FULL + 2,     // per tile: O_X (bf16) staged in its Q slot
  B_MMA_DONE = B_OST_FULL + 2,     // per issuing warp (S, P V)
  B_IT_FULL = B_MMA_DONE + 2,      // kSlots: an item is in its slot
  B_IT_EMPTY = B_IT_FULL + kSlots, // kSlots: every role has read it
  B_COUNT = B_IT_EMPTY + kSlots
};
static_assert(8 * B_COUNT + 8 <= kBarBytes, "barrier region overflow");

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0;    // S_X at 128 * X
constexpr uint32_t kColO = 256;  // O_X at 256 + 64 * X
constexpr uint32_t kColP = 384;  // P_X at 384 + 64 * X

constexpr uint32_t kIdescS = make_idesc_bf16(128, 128, false, false);  // Q K^T
constexpr uint32_t kIdescO = make_idesc_bf16(128, 64, false, true);    // P V (V MN-major)

struct Params {
  Problem pb;
  __nv_bfloat16* out;
  float* lse;
  float scale_log2;  // softmax scale * log2(e)
  int* status;
  const int* list;   // the non-empty items, longest first (build_items), or nullptr
  ItemList items;    // the numbering of the items (list or not)
};

// One work item: tile X is head h + X * head_step, rows from rowA + X * row_step
// of its sequence.
struct Item {
  int h, hk;       // tile A's query head; the key/value head
  int start, len;  // the sequence's first row in the packed tensors, its length
  int rowA;
  int row_step, head_step;
  bool hasB;            // tile B has rows inside the sequence
  int nkvA, nkvB, nkv;  // key tiles of A, of B, and of the item (causal)
};

// Item r.  False for an empty one (the sequence has no such block, or a bad
// cu_seqlens entry, which is reported).
__device__ __forceinline__ bool get_item(const Params& p, int r, Item& it, bool report) {
  const bool pairs = r < p.items.second;  // two heads, one row tile; or one head, two tiles
  const int q = pairs ? r : r - p.items.second;
  const int n_h = pairs ? p.items.n_heads : p.items.n_heads2;
  const int n_blk = pairs ? p.items.n_blocks : p.items.n_blocks2;
  const int n_sh = p.pb.nseq * n_h;
  const int up = q / n_sh, sh = q - up * n_sh;
  const int seq = sh / n_h, i = sh - seq * n_h;
  const int blk = n_blk - 1 - up;
  if (!seq_bounds(p.pb, seq, it.start, it.len, (report && blk == 0) ? p.status : nullptr))
    return false;
  const int G = p.pb.group;
  if (pairs) {
    const int per = G / 2;
    it.hk = i / per;
    it.h = it.hk * G + 2 * (i - it.hk * per);
    it.rowA = blk * kBM;
    it.row_step = 0;
    it.head_step = 1;
    it.hasB = true;
    it.nkvA = it.nkvB = blk + 1;
  } else {
    it.hk = i;
    it.h = i * G + G - 1;
    it.rowA = 2 * blk * kBM;
    it.row_step = kBM;
    it.head_step = 0;
    it.hasB = it.rowA + kBM < it.len;
    it.nkvA = 2 * blk + 1;
    it.nkvB = it.hasB ? 2 * blk + 2 : 0;
  }
  it.nkv = it.hasB ? it.nkvB : it.nkvA;
  return it.rowA < it.len;
}

}  // namespace gqa

// kList: the items come from a list, which has no empty ones but those of
// sequences with bad bounds; without one (more items than it holds, for a bound
// far above the lengths) nearly all may be empty.
template <bool kList>
__global__ void __launch_bounds__(gqa::kThreads, 1)
    ne_attn_gqa_fwd_kernel(const __grid_constant__ CUtensorMap tmQ,
                           const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV,
                           const __grid_constant__ CUtensorMap tmO, const gqa::Params p,
                           int n_items) {
  using namespace gqa;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_BAR + 8 * B_COUNT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_BAR + 8 * B_COUNT + 4);

  const int G = gridDim.x;
  const int cta = blockIdx.x;
  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars[B_Q_FULL + b], 1);
      mbar_init(&bars[B_Q_EMPTY + b], 2);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars[B_K_FULL + s], 1);
      mbar_init(&bars[B_K_EMPTY + s], 1);
      mbar_init(&bars[B_V_FULL + s], 1);
      mbar_init(&bars[B_V_EMPTY + s], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars[B_S_FULL + x], 1);
      mbar_init(&bars[B_S_FREE + x], 128);
      mbar_init(&bars[B_P_FULL + x], 128);
      mbar_init(&bars[B_PV_DONE + x], 1);
      mbar_init(&bars[B_O_FINAL + x], 1);
      mbar_init(&bars[B_O_FREE + x], 128);
      mbar_init(&bars[B_SUM_FULL + x], 128);
      mbar_init(&bars[B_OST_FULL + x], 128);
      mbar_init(&bars[B_MMA_DONE + x], 1);
    }
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&bars[B_IT_FULL + s], 1);
      mbar_init(&bars[B_IT_EMPTY + s], kReaders);
    }
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 12) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // The rotation pass (and what ran before it) has completed.  No early trigger:
  // the next pass's CTAs would take the place of this grid's last ones.
  pdl_wait();

  uint8_t* sQ = smem + OFF_Q;  // buffer b: Q_A at 2b tiles, Q_B at 2b + 1
  uint8_t* sK = smem + OFF_K;
  uint8_t* sV = smem + OFF_V;
  // The items of this CTA: warp 13, lane 0 finds them and puts them into the
  // slots, the other roles read them there (nkvA = 0: empty; -1: no more).
  int4* slots = reinterpret_cast<int4*>(smem + OFF_ITEM);
  auto read_slot = [&](int k, Item& it) {
    const int4 a = slots[2 * (k % kSlots)], b = slots[2 * (k % kSlots) + 1];
    it.start = a.x;
    it.len = a.y;
    it.rowA = a.z;
    it.h = a.w;
    it.hk = b.x;
    it.row_step = b.y;
    it.head_step = b.y ? 0 : 1;
    it.nkvA = b.z;
    it.nkvB = b.w;
    it.hasB = b.w > 0;
    it.nkv = max(b.z, b.w);
    return b.z;
  };
  auto next_warp = [&](int& k, Item& it) {  // for a whole warp
    while (mbar_poll_warp(&bars[B_IT_FULL + k % kSlots], (k / kSlots) & 1, abort_flag, p.status,
                          19)) {
      const int steps = read_slot(k, it);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[B_IT_EMPTY + k % kSlots]);
      if (kList || steps) return steps > 0;
      ++k;
    }
    return false;
  };
  auto next_lane = [&](int& k, Item& it) {  // for a single lane
    while (mbar_wait(&bars[B_IT_FULL + k % kSlots], (k / kSlots) & 1, abort_flag, p.status, 19)) {
      const int steps = read_slot(k, it);
      mbar_arrive(&bars[B_IT_EMPTY + k % kSlots]);
      if (kList || steps) return steps > 0;
      ++k;
    }
    return false;
  };
#define NE_FOR_EACH_ITEM(it, next) \
  Item it;                         \
  for (int k_ = 0; next(k_, it); ++k_)

  if (warp == 13 || warp == 14) {
    // ------------------------------------ TMA producers: warp 13 K, warp 14 V
    regs_decrease<kRegsOther>();
    if (lane == 0) {
      const bool isK = (warp == 13);
      const CUtensorMap* tm = isK ? &tmK : &tmV;
      uint8_t* ring = isK ? sK : sV;
      uint64_t* full = &bars[isK ? B_K_FULL : B_V_FULL];
      uint64_t* empty = &bars[isK ? B_K_EMPTY : B_V_EMPTY];
      tma_prefetch_desc(tm);
      if (isK) tma_prefetch_desc(&tmQ);
      bool ok = true;
      int g = 0;   // K (or V) tiles loaded so far by this CTA
      int nq = 0;  // items whose Q has been loaded
      // The CTA's first item is that of its number; the next is taken once the
      // loads of the last are issued, a ring of tiles ahead of the softmax.
      const int n = kList ? __ldg(p.list) : n_items;
      const int head = kList ? __ldg(p.list + 1 + cta) : cta;
      bool first = true;
      // False: none left.  Without a list an empty one (nkv = 0) goes through the
      // slots as well, so that no role waits for long while a CTA passes many.
      auto take = [&](Item& it) {
        while (true) {
          const unsigned m = first ? cta : G + atomicAdd(p.items.counter, 1);
          if (m >= static_cast<unsigned>(n)) return false;
          const int r = first ? head : kList ? __ldg(p.list + 1 + m) : static_cast<int>(m);
          first = false;
          if (get_item(p, r, it, true)) return true;
          if (!kList) {
            it.nkvA = it.nkvB = it.nkv = 0;
            return true;
          }
        }
      };
      for (int k = 0;; ++k) {
        Item it{};
        if (isK) {
          const bool more = take(it);
          const int s = k % kSlots;
          if (k >= kSlots && !mbar_wait(&bars[B_IT_EMPTY + s], ((k - kSlots) / kSlots) & 1,
                                        abort_flag, p.status, 20)) {
            ok = false;
            break;
          }
          slots[2 * s] = make_int4(it.start, it.len, it.rowA, it.h);
          slots[2 * s + 1] = make_int4(it.hk, it.row_step, more ? it.nkvA : -1, it.nkvB);
          mbar_arrive(&bars[B_IT_FULL + s]);
          if (!more) break;
          if (!kList && it.nkv == 0) continue;
          const int b = nq & 1;
          if (nq >= 2 && !mbar_wait(&bars[B_Q_EMPTY + b], ((nq - 2) >> 1) & 1, abort_flag,
                                    p.status, 14)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&bars[B_Q_FULL + b], 2 * kTileBytes);
          // (Tile B outside the sequence: rows that are not used, read all the same.)
          tma_load_3d(sQ + 2 * b * kTileBytes, &tmQ, &bars[B_Q_FULL + b], 0, it.h,
                      it.start + it.rowA);
          tma_load_3d(sQ + (2 * b + 1) * kTileBytes, &tmQ, &bars[B_Q_FULL + b], 0,
                      it.h + it.head_step, it.start + it.rowA + it.row_step);
          ++nq;
        } else if (!next_lane(k, it)) {
          break;
        }
        for (int j = 0; ok && j < it.nkv; ++j, ++g) {
          const int s = g % kStages;
          if (g >= kStages &&
              !mbar_wait(&empty[s], ((g - kStages) / kStages) & 1, abort_flag, p.status,
                         isK ? 1 : 12)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[s], kTileBytes);
          tma_load_3d(ring + s * kTileBytes, tm, &full[s], 0, it.hk, it.start + j * kBN);
        }
        if (!ok) break;
      }
      if (!ok || *abort_flag) {
        // Let the copies still in flight land before the CTA exits: every
        // issued load completes its FULL barrier phase.
        for (int s = 0; s < kStages; ++s) {
          if (g > s) {
            const int last = s + ((g - 1 - s) / kStages) * kStages;  // last tile loaded into s
            const long long t0 = clock64();
            while (!mbar_try_wait(&full[s], (last / kStages) & 1) &&
                   clock64() - t0 < NE_WAIT_LIMIT_CYCLES) {
            }
          }
        }
        if (isK)
          for (int q = (nq >= 2 ? nq - 2 : 0); q < nq; ++q) {
            const long long t0 = clock64();
            while (!mbar_try_wait(&bars[B_Q_FULL + (q & 1)], (q >> 1) & 1) &&
                   clock64() - t0 < NE_WAIT_LIMIT_CYCLES) {
            }
          }
      }
    } else if (warp == 14 && lane == 1) {
      // O tile stores, once the epilogue has staged a tile in its Q slot; when
      // both tiles of the item are stored (their smem read), the Q buffer goes
      // back to the loader.
      tma_prefetch_desc(&tmO);
      int nq = 0, nst[2] = {0, 0};
      NE_FOR_EACH_ITEM(it, next_lane) {
        const int b = nq & 1;
        bool ok = true;
        for (int x = 0; x < 2 && ok; ++x) {
          if (x == 1 && !it.hasB) continue;
          if (!(ok = mbar_wait(&bars[B_OST_FULL + x], nst[x] & 1, abort_flag, p.status, 16))) break;
          ++nst[x];
          const int row0 = it.rowA + x * it.row_step;
          if (row0 + kBM <= it.len)
            tma_store_3d(&tmO, sQ + (2 * b + x) * kTileBytes, 0, it.h + x * it.head_step,
                         it.start + row0);
        }
        if (!ok) break;
        bulk_commit_group();
        bulk_wait_group_read0();
        mbar_arrive(&bars[B_Q_EMPTY + b]);
        ++nq;
      }
      bulk_wait_group0();  // the stores have completed before the kernel ends
    }
  } else if (warp == 12 || warp == 15) {
    // ------------------------------------------------------------ MMA issuers
    // Warp 12 issues S_X = Q_X K^T and warp 15 issues O_X += P_X V, both walking
    // the same items; each commit sits on the warp whose MMAs it tracks.  The
    // whole warp runs the loop and waits; the elected lane issues each group of
    // MMAs together with its commits.  Shared-memory descriptors are built once:
    // a K step, a tile or a ring stage only adds a constant to the start-address
    // field (16-byte units).
    regs_decrease<kRegsOther>();
    const bool isS = (warp == 12);
    constexpr uint64_t kTileD = kTileBytes >> 4;
    const uint64_t dQ0 = make_sdesc_sw128(smem_u32(sQ), 16, 1024);          // Q K-major
    const uint64_t dK0 = make_sdesc_sw128(smem_u32(sK), 16, 1024);          // K K-major
    const uint64_t dV0 = make_sdesc_sw128(smem_u32(sV), kTileBytes, 1024);  // V MN-major
    bool ok = true;
    int g = 0;            // K / V tiles consumed
    int nq = 0;           // items started (Q buffer and phase)
    int cnt[2] = {0, 0};  // steps of tile X over all items
    int nit[2] = {0, 0};  // items in which tile X took part
    NE_FOR_EACH_ITEM(it, next_warp) {
      if (!ok) break;
      const int b = nq & 1;
      if (isS) {
        ok = mbar_poll_warp(&bars[B_Q_FULL + b], (nq >> 1) & 1, abort_flag, p.status, 2);
        for (int j = 0; ok && j < it.nkv; ++j) {
          const int gj = g + j, s = gj % kStages;
          if (!mbar_poll_warp(&bars[B_K_FULL + s], (gj / kStages) & 1, abort_flag, p.status, 3)) {
            ok = false;
            break;
          }
          const uint64_t dK = dK0 + kTileD * s;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (!ok || j >= (x ? it.nkvB : it.nkvA)) continue;
            const int c = cnt[x] + j;
            if (c >= 1 && !mbar_poll_warp(&bars[B_S_FREE + x], (c - 1) & 1, abort_flag, p.status, 4)) {
              ok = false;
              continue;
            }
            tc_fence_after();
            if (elect_one()) {
              // Descriptors formed at issue, not hoisted out of the loop.
              const uint64_t dQ = opaque_u64(dQ0) + kTileD * (2 * b + x);
              const uint64_t dKs = opaque_u64(dK);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)  // K = 64 head dims: 32 bytes per step
                umma_bf16_ss(tmem + kColS + 128 * x, dQ + 2 * kk, dKs + 2 * kk, kIdescS,
                             kk > 0 ? 1u : 0u);
              umma_commit(&bars[B_S_FULL + x]);
              if (x == 1 || j >= it.nkvB) umma_commit(&bars[B_K_EMPTY + s]);
              if (j == it.nkv - 1 && (x == 1 || !it.hasB)) umma_commit(&bars[B_Q_EMPTY + b]);
            }
            __syncwarp();
          }
        }
      } else {
        for (int jj = 0; ok && jj < it.nkv; ++jj) {
          const int gj = g + jj, s = gj % kStages;
          if (!mbar_poll_warp(&bars[B_V_FULL + s], (gj / kStages) & 1, abort_flag, p.status, 13)) {
            ok = false;
            break;
          }
          // The item's last tile: rows of V behind the sequence (a neighbour's, or
          // padding that may hold anything) are cleared, as their weight is zero and
          // 0 * NaN would show.  By this warp, which waits for the softmax next.
          if (it.len - jj * kBN < kBN) clear_rows(sV + s * kTileBytes, it.len - jj * kBN);
          const uint64_t dV = dV0 + kTileD * s;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (!ok || jj >= (x ? it.nkvB : it.nkvA)) continue;
            const int c = cnt[x] + jj;
            if (!mbar_poll_warp(&bars[B_P_FULL + x], c & 1, abort_flag, p.status, 5)) {
              ok = false;
              continue;
            }
            // The first P V of an item overwrites O_X: the previous item's
            // epilogue must have read it.
            if (jj == 0 && nit[x] >= 1 &&
                !mbar_poll_warp(&bars[B_O_FREE + x], (nit[x] - 1) & 1, abort_flag, p.status, 15)) {
              ok = false;
              continue;
            }
            tc_fence_after();
            if (elect_one()) {
              const uint32_t acc0 = jj > 0 ? 1u : 0u;
              const uint64_t dVs = opaque_u64(dV);
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)  // K = 128 keys: 8 packed P columns, 16 V rows
                umma_bf16_ts(tmem + kColO + 64 * x, tmem + kColP + 64 * x + 8 * kk, dVs + 128 * kk,
                             kIdescO, kk > 0 ? 1u : acc0);
              umma_commit(&bars[B_PV_DONE + x]);
              if (jj == (x ? it.nkvB : it.nkvA) - 1) umma_commit(&bars[B_O_FINAL + x]);
              if (x == 1 || jj >= it.nkvB) umma_commit(&bars[B_V_EMPTY + s]);
            }
            __syncwarp();
          }
        }
      }
      g += it.nkv;
      cnt[0] += it.nkvA;
      cnt[1] += it.nkvB;
      nit[0] += 1;
      nit[1] += it.hasB ? 1 : 0;
      ++nq;
    }
    // Drain: every MMA this warp issued completes before TMEM is released.
    uint64_t* done = &bars[B_MMA_DONE + (isS ? 0 : 1)];
    if (elect_one()) umma_commit(done);
    __syncwarp();
    const long long t0 = clock64();
    while (!mbar_try_wait(done, 0) && clock64() - t0 < NE_WAIT_LIMIT_CYCLES) {
    }
    __syncwarp();
  } else if (warp >= 8) {
    // -------------------------------------------------------- epilogue warps
    regs_decrease<kRegsEpilogue>();
    const int wq = warp & 3;
    const int r = wq * 32 + lane;  // row in tile
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const float* sums = reinterpret_cast<const float*>(smem + OFF_SUM);
    bool ok = true;
    int nq = 0, nit[2] = {0, 0};
    NE_FOR_EACH_ITEM(it, next_warp) {
      if (!ok) break;
#pragma unroll 1
      for (int x = 0; x < 2; ++x) {
        if (x == 1 && !it.hasB) continue;
        const int ph = nit[x] & 1;
        ok = mbar_poll_warp(&bars[B_SUM_FULL + x], ph, abort_flag, p.status, 17) &&
             mbar_poll_warp(&bars[B_O_FINAL + x], ph, abort_flag, p.status, 11);
        if (!ok) break;
        ++nit[x];
        tc_fence_after();
        const float inv_l = 1.f / sums[x * 128 + r];
        const uint32_t tO = tmem + lane_base + kColO + 64 * x;
        const int row0 = it.rowA + x * it.row_step, row = row0 + r;
        // A whole tile goes into the swizzled Q slot of this tile (no S MMA reads
        // it any more), and warp 14, lane 1 stores it with TMA; the sequence's
        // last, partial tile is written one row per thread.
        const bool whole = row0 + kBM <= it.len;
        uint8_t* slot = sQ + (2 * (nq & 1) + x) * kTileBytes;
        uint4* dst = reinterpret_cast<uint4*>(
            p.out + (static_cast<long long>(it.start + row) * p.pb.H + it.h + x * it.head_step) * kHD);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {  // (half a row at a time: registers)
          uint32_t o[32];
          tmem_ld_x32(tO + 32 * half, o);
          tmem_ld_wait(o);
          if (half) {
            tc_fence_before();
            mbar_arrive(&bars[B_O_FREE + x]);  // O_X and the sums may be overwritten
          }
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            uint4 w;
            w.x = pack_bf16x2(__uint_as_float(o[8 * cc + 0]) * inv_l, __uint_as_float(o[8 * cc + 1]) * inv_l);
            w.y = pack_bf16x2(__uint_as_float(o[8 * cc + 2]) * inv_l, __uint_as_float(o[8 * cc + 3]) * inv_l);
            w.z = pack_bf16x2(__uint_as_float(o[8 * cc + 4]) * inv_l, __uint_as_float(o[8 * cc + 5]) * inv_l);
            w.w = pack_bf16x2(__uint_as_float(o[8 * cc + 6]) * inv_l, __uint_as_float(o[8 * cc + 7]) * inv_l);
            if (whole)
              *reinterpret_cast<uint4*>(slot + sw128_offset(r, 4 * half + cc)) = w;
            else if (row < it.len)
              dst[4 * half + cc] = w;
          }
        }
        if (whole) fence_proxy_async_smem();
        mbar_arrive(&bars[B_OST_FULL + x]);
      }
      ++nq;
    }
  } else {
    // --------------------------------------------------------- softmax warps
    regs_increase<kRegsSoftmax>();
    const int x = warp >> 2;            // tile A (0) or B (1)
    const int wq = warp & 3;            // TMEM lane quarter
    const int r = wq * 32 + lane;       // row in tile
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + lane_base + kColS + 128 * x;
    const uint32_t tO = tmem + lane_base + kColO + 64 * x;
    const uint32_t tP = tmem + lane_base + kColP + 64 * x;
    const float sl2 = p.scale_log2;
    bool ok = true;
    int cnt = 0;  // steps of this tile over all items
    int nit = 0;  // items in which this tile took part
    NE_FOR_EACH_ITEM(it, next_warp) {
      if (!ok) break;
      const int nkv_x = x ? it.nkvB : it.nkvA;
      if (nkv_x == 0) continue;  // tile B outside the sequence
      const int row0 = it.rowA + x * it.row_step;
      // Index of this row's LSE, or -1 past the sequence's end.
      const int lse_at = row0 + r < it.len ? (it.h + x * it.head_step) * p.pb.n_tot + it.start +
                                                 row0 + r
                                           : -1;
      float m_ref = -INFINITY;  // reference max (log2 units) the P values are taken against
      float l_sum = 0.f;        // 0: no key with a weight yet (the first adds 1, or NaN)
#pragma unroll 1
      for (int left = nkv_x; left > 0; --left, ++cnt) {
        if (!(ok = mbar_poll_warp(&bars[B_S_FULL + x], cnt & 1, abort_flag, p.status, 8))) break;
        tc_fence_after();
        // The whole S row in one TMEM round trip; S_X is then free for Q_X K_{j+1}^T.
        uint32_t sr[128];
        tmem_ld_x32(tS + 0, sr + 0);
        tmem_ld_x32(tS + 32, sr + 32);
        tmem_ld_x32(tS + 64, sr + 64);
        tmem_ld_x32(tS + 96, sr + 96);
        tmem_ld_wait(sr + 0);
        tmem_ld_wait(sr + 32);
        tmem_ld_wait(sr + 64);
        tmem_ld_wait(sr + 96);
        tc_fence_before();
        mbar_arrive(&bars[B_S_FREE + x]);
        if (left == 1) {  // diagonal tile: keys after the query get no weight
#pragma unroll
          for (int cc = 0; cc < 128; ++cc)
            if (cc > r) sr[cc] = 0xff800000u;  // -inf
        }
        // Row max of the raw scores (the scale is positive), four chains.
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int cc = 0; cc < 128; cc += 8)
#pragma unroll
          for (int u = 0; u < 4; ++u)
            m4[u] = fmax3(m4[u], __uint_as_float(sr[cc + 2 * u]),
                          __uint_as_float(sr[cc + 2 * u + 1]));
        const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * sl2;
        // Move the reference max only when the row max outgrows it by more
        // than 2^8 (exact: O and l keep a common reference).
        const bool first = l_sum == 0.f;
        const bool grow = first || (mx > m_ref + 8.0f);
        const float m_new = grow ? mx : m_ref;
        const float alpha = first ? 0.f : ex2_approx(m_ref - m_new);
        m_ref = m_new;
        // P = 2^(x - m_ref) in bf16 pairs, half a row at a time: the second half's
        // exponentials overlap the store of the first.
        const uint64_t sl2x2 = f2_pack(sl2, sl2);
        // (-inf: no finite score yet, nor a weight; not -inf + inf.)
        const float neg = m_ref == -INFINITY ? 0.f : -m_ref;
        const uint64_t negm2 = f2_pack(neg, neg);
        uint64_t acc[2] = {0, 0};  // packed partial row sums (0 = +0.f, +0.f)
        uint32_t pw[64];
        auto exponentials = [&](int half) {
#pragma unroll
          for (int cc = 64 * half; cc < 64 * half + 64; cc += 2) {
            const uint64_t t = f2_fma(f2_pack(__uint_as_float(sr[cc]), __uint_as_float(sr[cc + 1])),
                                      sl2x2, negm2);
            float t0, t1;
            f2_unpack(t, t0, t1);
            const float p0 = ex2_approx(t0), p1 = ex2_approx(t1);
            acc[(cc >> 1) & 1] = f2_add(acc[(cc >> 1) & 1], f2_pack(p0, p1));
            pw[cc >> 1] = pack_bf16x2(p0, p1);
          }
        };
        exponentials(0);
        // P_X and O_X are in use by the P V of the tile's previous step until it
        // completes (waited every step, so PV_DONE is never two phases behind;
        // before the first step of all the parity is that of the phase before).
        if (!(ok = mbar_poll_warp(&bars[B_PV_DONE + x], (cnt - 1) & 1, abort_flag, p.status, 9))) break;
        tc_fence_after();
        if (__any_sync(0xffffffffu, grow && !first)) {
          uint32_t o[32];
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            tmem_ld_x32(tO + half * 32, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int cc = 0; cc < 32; ++cc) o[cc] = __float_as_uint(__uint_as_float(o[cc]) * alpha);
            tmem_st_x32(tO + half * 32, o);
            tmem_st_wait();  // the store has consumed `o` before it is reloaded
          }
        }
        tmem_st_x32(tP, pw);
        exponentials(1);
        tmem_st_x32(tP + 32, pw + 32);
        float rs0, rs1;
        f2_unpack(f2_add(acc[0], acc[1]), rs0, rs1);
        const float rs = rs0 + rs1;
        tmem_st_wait();
        l_sum = l_sum * alpha + rs;
        tc_fence_before();
        mbar_arrive(&bars[B_P_FULL + x]);
      }
      if (!ok) break;
      // LSE in natural-log units: (m_ref + log2 l) * ln 2.
      if (lse_at >= 0) p.lse[lse_at] = (m_ref + __log2f(l_sum)) * 0.69314718055994531f;
      // The sums' place is free once the previous item's epilogue is done with
      // O_X (waited every item, so O_FREE is never two phases behind).
      if (nit >= 1 && !(ok = mbar_poll_warp(&bars[B_O_FREE + x], (nit - 1) & 1, abort_flag,
                                            p.status, 18)))
        break;
      reinterpret_cast<float*>(smem + OFF_SUM)[x * 128 + r] = l_sum;
      mbar_arrive(&bars[B_SUM_FULL + x]);
      ++nit;
    }
  }
#undef NE_FOR_EACH_ITEM

  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// The items of a batch whose longest sequence has n_qtiles tiles of 128 rows:
// their numbering, and how many numbers there are.
ItemList gqa_fwd_items(const Problem& pb, int n_qtiles, long long* n_items) {
  ItemList l;
  const int Hkv = pb.H / pb.group;
  l.kind = Items::kHeadPairs;
  l.n_blocks = n_qtiles;
  l.n_heads = Hkv * (pb.group / 2);
  l.n_blocks2 = (n_qtiles + 1) / 2;
  l.n_heads2 = pb.group % 2 ? Hkv : 0;
  l.n_buckets = 2 * l.n_blocks2 + 1;
  const long long first = static_cast<long long>(l.n_blocks) * pb.nseq * l.n_heads;
  *n_items = first + static_cast<long long>(l.n_blocks2) * pb.nseq * l.n_heads2;
  l.second = static_cast<int>(first);
  return l;
}

cudaError_t launch_gqa_fwd(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                           const CUtensorMap& tmO, const Problem& pb, __nv_bfloat16* out,
                           float* lse, float scale_log2, const ItemList& items, int n_items,
                           int sms, int* status, cudaStream_t stream) {
  static bool done[2][64] = {};
  cudaError_t e = allow_smem(ne_attn_gqa_fwd_kernel<false>, gqa::SMEM_BYTES, done[0]);
  if (e == cudaSuccess) e = allow_smem(ne_attn_gqa_fwd_kernel<true>, gqa::SMEM_BYTES, done[1]);
  if (e != cudaSuccess) return e;
  gqa::Params p;
  p.pb = pb;
  p.out = out;
  p.lse = lse;
  p.scale_log2 = scale_log2;
  p.status = status;
  p.list = items.out;
  p.items = items;
  // One persistent CTA per SM (at most one per item).
  return launch_pdl(items.out ? ne_attn_gqa_fwd_kernel<true> : ne_attn_gqa_fwd_kernel<false>,
                    dim3(n_items < sms ? n_items : sms), dim3(gqa::kThreads), gqa::SMEM_BYTES,
                    stream, tmQ, tmK, tmV, tmO, p, n_items);
}

// ---------------------------------------------------------------------------
// Rotation pass: q' = R(m) q over H heads and k' = R(n) k over H / group, with the
// fp32 rule of ne_attn_rope_rows_kernel (bitwise its values), and, by the first
// CTA, the attention kernel's work list.
//
// It moves bytes: 256 in and out per (row, head), ~13 us for 2 x 33.6 MB (5.2
// TB/s read and written).  The CTAs take the packed rows in equal blocks (not
// sequence by sequence: a grid of the longest sequence times nseq had half its
// CTAs empty on a batch of 64 to 2048 rows), so the sequence of a row is
// searched, once per row and CTA, while the first loads are in flight; a
// persistent form with the next block's loads and search ahead was no faster.
// Rows of no sequence, or of one with bad bounds (the attention kernel reports
// it), are left alone.  (The queries rotated by the attention kernel's epilogue
// warps instead, an item ahead: the first scores wait for it, 59.5 us against 55.1
// for the packed prompts, 13.6 against 10.9 for short ones.)
//
// Four lanes take a (row, head), lane c the 16-byte chunks c and c + 4; a CTA's
// (row, head) pairs -- the keys' heads behind the queries' -- go round its 64
// quads, each quad moving on by 64 pairs with an addition (a division per pair
// was a third of the instructions).
// ---------------------------------------------------------------------------
constexpr int kRopeThreads = 256, kRopeParts = 4;
constexpr int kGqaItems = 2;   // pairs of a quad in flight
constexpr int kGqaRounds = 1;  // rounds of a CTA, about

__global__ void __launch_bounds__(kRopeThreads)
    ne_attn_gqa_rotate_kernel(const __nv_bfloat16* __restrict__ q, __nv_bfloat16* __restrict__ qr,
                              const __nv_bfloat16* __restrict__ k, __nv_bfloat16* __restrict__ kr,
                              const Problem pb, RopeTable rope, int rows_per_cta,
                              const ItemList list) {
  extern __shared__ int dyn[];  // the list's buckets, or the rows' positions
  pdl_wait();                   // the kernel that wrote q, k (and anything before it) has completed
  if (blockIdx.x == 0 && threadIdx.x == 0) *list.counter = 0;
  if (blockIdx.x == 0 && list.out) {
    build_items(pb, list, dyn);
    return;
  }
  constexpr int kQuads = kRopeThreads / kRopeParts;
  const int row0 = (static_cast<int>(blockIdx.x) - (list.out ? 1 : 0)) * rows_per_cta;
  const int rows = min(rows_per_cta, pb.n_tot - row0);
  const int H = pb.H, Hkv = pb.H / pb.group, heads = H + Hkv;
  q += static_cast<long long>(row0) * H * kHD;
  qr += static_cast<long long>(row0) * H * kHD;
  k += static_cast<long long>(row0) * Hkv * kHD;
  kr += static_cast<long long>(row0) * Hkv * kHD;
  const int c = threadIdx.x % kRopeParts;
  const int row_step = kQuads / heads, head_step = kQuads - row_step * heads;
  int row = (threadIdx.x / kRopeParts) / heads;
  int head = threadIdx.x / kRopeParts - row * heads;
  bool first = true;
  while (true) {
    uint4 lo[kGqaItems], hi[kGqaItems];
    int rr[kGqaItems], off[kGqaItems];  // the pairs' rows, and offsets in 16-byte units
    bool is_k[kGqaItems];
#pragma unroll
    for (int u = 0; u < kGqaItems; ++u) {
      rr[u] = row;
      is_k[u] = head >= H;
      const int r = min(row, rows - 1);  // a quad past the last row reads that one, discarded
      off[u] = (is_k[u] ? r * Hkv + (head - H) : r * H + head) * (kHD / 8) + c;
      const uint4* src = reinterpret_cast<const uint4*>(is_k[u] ? k : q) + off[u];
      lo[u] = __ldg(src);
      hi[u] = __ldg(src + 4);
      row += row_step;
      head += head_step;
      if (head >= heads) {
        head -= heads;
        ++row;
      }
    }
    if (first) {
      first = false;
      for (int r = threadIdx.x; r < rows; r += kRopeThreads) {
        const int s = find_sequence(pb.cu_seqlens, pb.nseq, row0 + r);
        int start = 0, len = 0;
        dyn[r] = s >= 0 && seq_bounds(pb, s, start, len, nullptr) ? row0 + r - start : -1;
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kGqaItems; ++u) {
      if (rr[u] >= rows) return;
      const int pos = dyn[rr[u]];
      if (pos < 0) continue;
      const float4* cs =
          reinterpret_cast<const float4*>(rope.cs + static_cast<long long>(pos) * 32 + 8 * c);
      uint32_t wl[4] = {lo[u].x, lo[u].y, lo[u].z, lo[u].w};
      uint32_t wh[4] = {hi[u].x, hi[u].y, hi[u].z, hi[u].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 t = __ldg(cs + j);  // (cos, sin) of dims 8c + 2j and 8c + 2j + 1
        const float a0 = bf16lo_to_f32(wl[j]), a1 = bf16hi_to_f32(wl[j]);
        const float b0 = bf16lo_to_f32(wh[j]), b1 = bf16hi_to_f32(wh[j]);
        const float lo0 = __fmaf_rn(a0, t.x, -__fmul_rn(b0, t.y));
        const float hi0 = __fmaf_rn(b0, t.x, __fmul_rn(a0, t.y));
        const float lo1 = __fmaf_rn(a1, t.z, -__fmul_rn(b1, t.w));
        const float hi1 = __fmaf_rn(b1, t.z, __fmul_rn(a1, t.w));
        wl[j] = pack_bf16x2(lo0, lo1);
        wh[j] = pack_bf16x2(hi0, hi1);
      }
      uint4* dst = reinterpret_cast<uint4*>(is_k[u] ? kr : qr) + off[u];
      dst[0] = make_uint4(wl[0], wl[1], wl[2], wl[3]);
      dst[4] = make_uint4(wh[0], wh[1], wh[2], wh[3]);
    }
  }
}

cudaError_t launch_gqa_rotate(const __nv_bfloat16* q, __nv_bfloat16* qr, const __nv_bfloat16* k,
                              __nv_bfloat16* kr, const Problem& pb, const RopeTable& rope,
                              const ItemList& list, cudaStream_t stream) {
  const int heads = pb.H + pb.H / pb.group;
  const int rows = std::max(1, kGqaRounds * kGqaItems * kRopeThreads / kRopeParts / heads);
  const int ctas = (pb.n_tot + rows - 1) / rows + (list.out ? 1 : 0);
  const size_t smem = sizeof(int) * std::max(rows, list.out ? list.n_buckets : 0);
  return launch_pdl(ne_attn_gqa_rotate_kernel, dim3(ctas), dim3(kRopeThreads), smem, stream, q, qr,
                    k, kr, pb, rope, rows, list);
}

}  // namespace ne
