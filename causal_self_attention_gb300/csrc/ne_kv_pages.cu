// ne_kv_pages.cu -- the pages of a paged key/value cache handed out and taken
// back on the GPU, and the positions and slots of a step's new rows, sm_103a.
//
// The free pages are a stack.  Reserve: sequence s, holding n_s positions, gets
// m_s new rows; with had(s) = ceil(n_s / P) and take(s) = ceil((n_s + m_s) / P) -
// had(s) pages of P positions, the t-th page taken (in the order of the sequences,
// within one of its positions) is the t-th from the top of the stack:
//   first(s) = sum_{s' < s} take(s'),   cu(s) = sum_{s' < s} m_s',
//   block_table[s, had(s) + j] = free[n_free - 1 - (first(s) + j)],
//   row cu(s) + i: position n_s + i, slot page * P + position % P.
// Release: the pages of finished sequences go onto the stack in the same order.
//
// Both are a prefix sum over the sequences and a few words for every row.  Every
// CTA forms the sums itself, in shared memory (16384 sequences take 192 KB: the
// limit); then each takes its share of the rows and of the pages, finding a row's
// sequence by bisection.  What is kept for the next step (lengths, the stack's height)
// may be updated in place, and no CTA may read a new value for an old one.  Reserve:
// nothing waits for another CTA, the one that has read last does that (one CTA: itself).
// A page taken is entered into the block table by its first row's thread.  Release: all or
// nothing wants every entry looked at before one is pushed, so that its CTAs, eight at the
// most, are a cluster: each looks at its share, and the cluster's barrier says that all have.
//
// What bounds it is latency and, with thousands of sequences, every CTA's instructions for
// their sums.  Measured: 64 sequences, a row each, 3.8 us (launch, the lengths, two barriers,
// a bisection, a table entry); 4096 sequences with a million rows in all 10.1 us (the rows'
// 8 MB alone 1.2 us), with a row each 9.4: the sums, every warp's of all warps' in each round;
// 16384 with a row each 21.8 us.  (Sequences in runs of a thread's own 4.7,
// 12.8 and 46.6 us; two CTAs an SM 12 to 14% slower for the second; lengths updated behind the
// rows' stores, whose fence waits for them, or all threads waiting for the arrival, 1 to 2 us
// more.)
// Release, pages of 16 each: a tenth of 64 sequences 5.5 us, of 4096 9.3; 16384 at once, 262,144
// pages, 71.  (Without a look at the entries first 4.8, 9.2 and 32, but an entry that is no page
// would be handed out to the next sequence.)
#include <algorithm>

#include "ne_paged.cuh"
#include "ne_sm100.cuh"

namespace ne {

namespace pages {
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kRowsPerThread = 4;

constexpr int kMaxRounds = (kMaxPagedSequences + kThreads - 1) / kThreads;
constexpr uint32_t kMany = 0x7fffffffu;  // sums stop here: more than any bound allows

struct Shared {
  uint2 sums[kMaxRounds][kWarps];  // a warp's rows and pages
  int last, n_free;
  int wrong;  // release: an entry of the CTA's share is no page of the pool
};

__device__ __forceinline__ uint2 add(uint2 a, uint2 b) {
  return make_uint2(min(a.x + b.x, kMany), min(a.y + b.y, kMany));
}
// Inclusive sums over the lanes.
__device__ __forceinline__ uint2 scan_warp(uint2 v, int lane) {
#pragma unroll
  for (int sh = 1; sh < 32; sh <<= 1) {
    const uint2 u = make_uint2(__shfl_up_sync(0xffffffffu, v.x, sh), __shfl_up_sync(0xffffffffu, v.y, sh));
    if (lane >= sh) v = add(v, u);
  }
  return v;
}
__device__ __forceinline__ uint2 from_lane(uint2 v, int lane) {
  return make_uint2(__shfl_sync(0xffffffffu, v.x, lane), __shfl_sync(0xffffffffu, v.y, lane));
}

// The last s with first[s] <= x (first[0] = 0, nondecreasing, first[n] > x).
__device__ __forceinline__ int find(const int* first, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// Exclusive prefix sums of rows(s) and pages(s) over the sequences into shared
// memory, [nseq + 1] each, and their totals (at most kMany).  load(s): what is known of sequence
// s, one(s, what, rows, pages): what it adds (at most 65535 * 128 rows).  Every thread calls
// it.  A round is a sequence a thread, neighbours side by side (loads and shared memory
// without conflicts: 16384 sequences in runs of 16 a thread took 46 us); the warps' sums of
// all rounds are exchanged once.
template <typename Load, typename One>
__device__ __forceinline__ void prefix_sums(int nseq, int* row_at, int* page_at, Shared& sh,
                                            int& rows, int& pages, Load load, One one) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rounds = (nseq + kThreads - 1) / kThreads;
  constexpr int kAhead = 4;  // rounds whose loads are on their way together
  for (int r0 = 0; r0 < rounds; r0 += kAhead) {
    int2 what[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int s = (r0 + i) * kThreads + threadIdx.x;
      what[i] = s < nseq ? load(s) : make_int2(0, 0);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (r0 + i >= rounds) break;
      const int s = (r0 + i) * kThreads + threadIdx.x;
      int m = 0, t = 0;
      if (s < nseq) one(s, what[i], m, t);
      const uint2 sum = scan_warp(make_uint2(m, t), lane);
      if (s < nseq) {
        row_at[s] = static_cast<int>(sum.x) - m;
        page_at[s] = static_cast<int>(sum.y) - t;
      }
      if (lane == 31) sh.sums[r0 + i][warp] = sum;
    }
  }
  __syncthreads();
  uint2 before = make_uint2(0u, 0u);  // the rounds before
  for (int r = 0; r < rounds; ++r) {
    const uint2 sum = scan_warp(sh.sums[r][lane], lane);
    const uint2 left = from_lane(sum, max(warp - 1, 0));
    const uint2 mine = add(before, warp ? left : make_uint2(0u, 0u));
    const int s = r * kThreads + threadIdx.x;
    if (s < nseq) {
      row_at[s] = static_cast<int>(min(mine.x + row_at[s], kMany));
      page_at[s] = static_cast<int>(min(mine.y + page_at[s], kMany));
    }
    before = add(before, from_lane(sum, 31));
  }
  rows = static_cast<int>(before.x);
  pages = static_cast<int>(before.y);
  if (threadIdx.x == 0) {
    row_at[nseq] = rows;
    page_at[nseq] = pages;
  }
  __syncthreads();
}

// A CTA's reads of what is updated in place are behind it (and it has stored nothing yet,
// which the fence would wait for): thread 0 says so, and the others need not wait for it.
__device__ __forceinline__ void has_read(int* arrived, Shared& sh) {
  if (threadIdx.x != 0) return;
  sh.last = 1;
  if (gridDim.x == 1) return;
  __threadfence();
  sh.last = atomicAdd(arrived, 1) == static_cast<int>(gridDim.x) - 1;
  if (sh.last) {
    *arrived = 0;  // as the next launch wants it
    __threadfence();
  }
}
// Whether this CTA was the launch's last to say so.  Every thread calls it.
__device__ __forceinline__ bool last_to_read(const Shared& sh) {
  __syncthreads();
  return sh.last != 0;
}
}  // namespace pages

__global__ void __launch_bounds__(pages::kThreads) ne_kv_reserve_kernel(const PagesParams p) {
  using namespace pages;
  extern __shared__ int dyn[];
  __shared__ Shared sh;
  int* row_at = dyn;                  // [nseq + 1] first row of each sequence
  int* page_at = row_at + p.nseq + 1; // [nseq + 1] first page taken for it
  int* lens = page_at + p.nseq + 1;   // [nseq] positions that it holds
  pdl_wait();
  const int P1 = (1 << p.page_shift) - 1;
  if (threadIdx.x == 0) sh.n_free = __ldcg(p.n_free);  // (read for good before the sums' barrier)
  bool bad = false;
  int rows, taken;
  auto load = [&](int s) { return make_int2(__ldcg(p.seq_lens + s), __ldg(p.new_lens + s)); };
  prefix_sums(p.nseq, row_at, page_at, sh, rows, taken, load, [&](int s, int2 what, int& m, int& t) {
    const int n = what.x;
    m = what.y;
    lens[s] = n;
    if (n < 0 || m < 0 || n > p.max_seqlen || m > p.max_seqlen - n) {
      bad = true;
      m = 0;
      return;
    }
    t = ((n + m + P1) >> p.page_shift) - ((n + P1) >> p.page_shift);
  });
  bad = __syncthreads_or(bad) || rows > p.max_rows;
  has_read(p.arrived, sh);
  const int n_free = sh.n_free;
  const bool short_of = taken > n_free || n_free > p.n_pages || n_free < 0;
  const bool ok = !bad && !short_of;
  if (!ok && blockIdx.x == 0 && threadIdx.x == 0)
    atomicCAS(p.status, 0, bad ? NE_DEV_BAD_SEQLEN : NE_DEV_NO_PAGES);

  const int id = blockIdx.x * kThreads + threadIdx.x, all = gridDim.x * kThreads;
  // The pages taken, into the block table, where no row's thread does it.
  if (ok && p.n_tot == 0)
    for (int t = id; t < taken; t += all) {
      const int s = find(page_at, p.nseq, t);
      const int at = ((lens[s] + P1) >> p.page_shift) + t - page_at[s];
      p.block_table[static_cast<long long>(s) * p.max_pages + at] = __ldg(p.free_pages + n_free - 1 - t);
    }
  // Positions and slots, neighbouring rows in a thread's hands; the first row of a new page
  // enters it into the block table.
  const int n_rows = ok ? rows : 0;
  const bool aligned = ((reinterpret_cast<uintptr_t>(p.positions) | reinterpret_cast<uintptr_t>(p.slots)) & 15) == 0;
  for (int r0 = id * kRowsPerThread; r0 < p.n_tot; r0 += all * kRowsPerThread) {
    int s = r0 < n_rows ? find(row_at, p.nseq, r0) : 0;
    int pos[kRowsPerThread], slot[kRowsPerThread], page[kRowsPerThread];
    int* enter[kRowsPerThread];
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {  // (all entries on their way before one is used)
      const int r = r0 + i;
      pos[i] = page[i] = -1;
      enter[i] = nullptr;
      if (r >= n_rows) continue;
      while (row_at[s + 1] <= r) ++s;
      const int n = lens[s], had = (n + P1) >> p.page_shift;
      pos[i] = n + r - row_at[s];
      const int at = pos[i] >> p.page_shift;
      int* entry = p.block_table + static_cast<long long>(s) * p.max_pages + at;
      page[i] = __ldcg(at < had ? entry : p.free_pages + n_free - 1 - (page_at[s] + at - had));
      if (at >= had && (pos[i] & P1) == 0) enter[i] = entry;
    }
    bool outside = false;
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {
      if (enter[i]) *enter[i] = page[i];
      const bool there = page[i] >= 0 && page[i] < p.n_pages;
      slot[i] = there ? (page[i] << p.page_shift) + (pos[i] & P1) : -1;
      outside |= !there && pos[i] >= 0;
    }
    if (outside) atomicCAS(p.status, 0, NE_DEV_BAD_PAGE);
    if (aligned && r0 + kRowsPerThread <= p.n_tot) {
      if (p.positions) *reinterpret_cast<int4*>(p.positions + r0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      if (p.slots) *reinterpret_cast<int4*>(p.slots + r0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    } else {
#pragma unroll
      for (int i = 0; i < kRowsPerThread; ++i) {
        if (p.positions && r0 + i < p.n_tot) p.positions[r0 + i] = pos[i];
        if (p.slots && r0 + i < p.n_tot) p.slots[r0 + i] = slot[i];
      }
    }
  }
  for (int s = id; s <= p.nseq; s += all) {
    if (p.cu_seqlens) p.cu_seqlens[s] = ok ? row_at[s] : 0;
    if (p.start_pos && s < p.nseq) p.start_pos[s] = lens[s];
  }
  if (!last_to_read(sh)) return;
  for (int s = threadIdx.x; s < p.nseq; s += kThreads)
    p.seq_lens_out[s] = ok ? lens[s] + row_at[s + 1] - row_at[s] : lens[s];
  if (threadIdx.x == 0) *p.n_free_out = ok ? n_free - taken : n_free;
}

__global__ void __launch_bounds__(pages::kThreads) ne_kv_release_kernel(const PagesParams p) {
  using namespace pages;
  extern __shared__ int dyn[];
  __shared__ Shared sh;
  int* row_at = dyn;                   // (finished sequences before each)
  int* page_at = row_at + p.nseq + 1;  // [nseq + 1] first page given back by it
  pdl_wait();
  const int P1 = (1 << p.page_shift) - 1;
  if (threadIdx.x == 0) sh.n_free = __ldcg(p.n_free);  // (read for good before the sums' barrier)
  bool bad = false;
  int done, given;
  auto load = [&](int s) { return make_int2(__ldcg(p.seq_lens + s), __ldg(p.finished + s)); };
  prefix_sums(p.nseq, row_at, page_at, sh, done, given, load, [&](int s, int2 what, int& m, int& t) {
    const int n = what.x;
    m = what.y != 0;
    if (!m) return;
    if (n < 0 || n > p.max_seqlen) {
      bad = true;
      return;
    }
    t = (n + P1) >> p.page_shift;
  });
  bad = __syncthreads_or(bad);
  const int n_free = sh.n_free;
  const bool over = n_free < 0 || n_free > p.n_pages || given > p.n_pages - n_free;
  const int id = blockIdx.x * kThreads + threadIdx.x, all = gridDim.x * kThreads;
  // (The same in every CTA: nobody writes before the cluster's barrier.)
  const int n_given = bad || over ? 0 : given;
  // Some entries of the thread's share at a time, the pages t, t + all, ...
  constexpr int kEach = 4;
  int* entry[kEach];
  int page[kEach];
  bool wrong = false;
  auto look = [&](int t) {
#pragma unroll
    for (int i = 0; i < kEach; ++i, t += all) {
      entry[i] = nullptr;
      if (t >= n_given) continue;
      const int s = find(page_at, p.nseq, t);
      entry[i] = p.block_table + static_cast<long long>(s) * p.max_pages + t - page_at[s];
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      page[i] = entry[i] ? __ldcg(entry[i]) : 0;
      wrong |= page[i] < 0 || page[i] >= p.n_pages;
    }
  };
  for (int t = id + kEach * all; t < n_given; t += kEach * all) look(t);
  look(id);  // (the first ones last: they are at hand below)
  wrong = __syncthreads_or(wrong);
  if (threadIdx.x == 0) sh.wrong = wrong;
  cluster_arrive();
  cluster_wait();
  wrong = threadIdx.x < gridDim.x && cluster_load(&sh.wrong, threadIdx.x) != 0;
  cluster_arrive();  // (a CTA's shared memory stays until all have read it: the wait at the end)
  wrong = __syncthreads_or(wrong);
  if ((bad || over || wrong) && id == 0)
    atomicCAS(p.status, 0, bad ? NE_DEV_BAD_SEQLEN : over ? NE_DEV_NO_PAGES : NE_DEV_BAD_PAGE);
  if (!bad && !over && !wrong) {
    for (int t = id;;) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        if (!entry[i]) continue;
        p.free_pages_out[n_free + t + i * all] = page[i];
        *entry[i] = -1;
      }
      t += kEach * all;
      if (t >= n_given) break;
      look(t);
    }
    for (int s = id; s < p.nseq; s += all)
      if (row_at[s + 1] != row_at[s]) p.seq_lens_out[s] = 0;
    if (id == 0) *p.n_free_out = n_free + given;
  }
  cluster_wait();
}

namespace {
// The dynamic shared memory of `arrays` words a sequence (and one), allowed for the kernel.
cudaError_t allow(void (*kernel)(const PagesParams), int arrays, int nseq, bool (&done)[64],
                  int* bytes) {
  *bytes = arrays * (nseq + 1) * static_cast<int>(sizeof(int));
  if (*bytes <= 48 * 1024 - static_cast<int>(sizeof(pages::Shared))) return cudaSuccess;
  return allow_smem(kernel, arrays * (kMaxPagedSequences + 1) * static_cast<int>(sizeof(int)), done);
}
}  // namespace

cudaError_t launch_kv_reserve(const PagesParams& p, int sms, cudaStream_t stream) {
  static bool done[64] = {};
  int bytes;
  const cudaError_t e = allow(ne_kv_reserve_kernel, 3, p.nseq, done, &bytes);
  if (e != cudaSuccess) return e;
  constexpr int kRows = pages::kThreads * pages::kRowsPerThread;
  const int ctas = std::min(std::max((p.n_tot + kRows - 1) / kRows, 1), sms);
  return launch_pdl(ne_kv_reserve_kernel, dim3(ctas), dim3(pages::kThreads), bytes, stream, p);
}

// (The pages given back are not known on the host: a CTA for every 1024 sequences, eight at
// the most, a cluster that any part can hold.)
cudaError_t launch_kv_release(const PagesParams& p, cudaStream_t stream) {
  static bool done[64] = {};
  int bytes;
  const cudaError_t e = allow(ne_kv_release_kernel, 2, p.nseq, done, &bytes);
  if (e != cudaSuccess) return e;
  const unsigned ctas = std::min((p.nseq + pages::kThreads - 1) / pages::kThreads, 8);
  return launch_pdl_clusters(ctas, ne_kv_release_kernel, dim3(ctas), dim3(pages::kThreads), bytes,
                             stream, p);
}

}  // namespace ne
