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
// limit), so that nothing has to wait for another CTA; then each takes its share
// of the rows and of the pages, finding a row's sequence by bisection.  What is
// kept for the next step (lengths, the stack's height) may be updated in place:
// the CTA that has read it last does that (one CTA: itself), so that no CTA reads
// a new value for an old one.
//
// What bounds it is latency: launch, the lengths' loads, two exchanges of the sums, a
// row's bisection in shared memory and its table entry.  Measured: 64 sequences, a row
// each, 4.6 us; 4096 sequences with a million rows in all 12.4 us (the rows' 8 MB alone
// 1.2 us): every CTA sums the 4096 lengths, and a thread's four rows take a bisection of 12
// steps.  (Two CTAs an SM where they fit; the sums updated behind the rows' stores,
// whose fence waits for them, 14.6 us.)
#include "ne_paged.cuh"
#include "ne_sm100.cuh"

namespace ne {

namespace pages {
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kRowsPerThread = 4;

struct Shared {
  uint32_t warp_rows[kWarps], warp_pages[kWarps];
  int last;
};

// Inclusive sums over the lanes.
template <typename T>
__device__ __forceinline__ T scan_warp(T v, int lane) {
#pragma unroll
  for (int sh = 1; sh < 32; sh <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, v, sh);
    if (lane >= sh) v += u;
  }
  return v;
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
// memory, [nseq + 1] each, and their totals (64 bits: the entries hold where the
// totals fit).  one(s, rows, pages): what sequence s adds, at most 65535 * 128 rows, so that
// a warp's 512 sequences fit 32 bits.  Every thread calls it, with neighbouring sequences of
// its own: one exchange between the warps, however many there are.
template <typename One>
__device__ __forceinline__ void prefix_sums(int nseq, int* row_at, int* page_at, Shared& sh,
                                            long long& rows, long long& pages, One one) {
  static_assert(kMaxPagedSequences <= 16 * kThreads, "32 bits for a warp's sums");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (nseq + kThreads - 1) / kThreads;
  const int s0 = min(static_cast<int>(threadIdx.x) * per, nseq), s1 = min(s0 + per, nseq);
  uint32_t m_sum = 0, t_sum = 0;
#pragma unroll 4
  for (int s = s0; s < s1; ++s) {
    int m = 0, t = 0;
    one(s, m, t);
    row_at[s] = m;
    page_at[s] = t;
    m_sum += m;
    t_sum += t;
  }
  const uint32_t a = scan_warp(m_sum, lane), b = scan_warp(t_sum, lane);
  if (lane == 31) {
    sh.warp_rows[warp] = a;
    sh.warp_pages[warp] = b;
  }
  __syncthreads();
  const long long wr = scan_warp(static_cast<long long>(sh.warp_rows[lane]), lane);
  const long long wp = scan_warp(static_cast<long long>(sh.warp_pages[lane]), lane);
  rows = __shfl_sync(0xffffffffu, wr, 31);
  pages = __shfl_sync(0xffffffffu, wp, 31);
  long long r = __shfl_sync(0xffffffffu, wr, max(warp - 1, 0)), p = __shfl_sync(0xffffffffu, wp, max(warp - 1, 0));
  r = (warp ? r : 0) + a - m_sum;
  p = (warp ? p : 0) + b - t_sum;
  for (int s = s0; s < s1; ++s) {
    const int m = row_at[s], t = page_at[s];
    row_at[s] = static_cast<int>(r);
    page_at[s] = static_cast<int>(p);
    r += m;
    p += t;
  }
  if (threadIdx.x == 0) {
    row_at[nseq] = static_cast<int>(rows);
    page_at[nseq] = static_cast<int>(pages);
  }
  __syncthreads();
}

// Whether this CTA is the last of the launch to come here, with its reads of what is
// updated in place behind it (and no store, which the fence would wait for).  Every
// thread calls it.
__device__ __forceinline__ bool last_to_read(int* arrived, Shared& sh) {
  if (gridDim.x == 1) return true;
  if (threadIdx.x == 0) {
    __threadfence();
    sh.last = atomicAdd(arrived, 1) == static_cast<int>(gridDim.x) - 1;
    if (sh.last) {
      *arrived = 0;  // as the next launch wants it
      __threadfence();
    }
  }
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
  const int n_free = __ldcg(p.n_free);
  bool bad = false;
  long long rows, taken;
  prefix_sums(p.nseq, row_at, page_at, sh, rows, taken, [&](int s, int& m, int& t) {
    const int n = __ldcg(p.seq_lens + s);
    m = __ldg(p.new_lens + s);
    lens[s] = n;
    if (n < 0 || m < 0 || n > p.max_seqlen || m > p.max_seqlen - n) {
      bad = true;
      m = 0;
      return;
    }
    t = ((n + m + P1) >> p.page_shift) - ((n + P1) >> p.page_shift);
  });
  const bool updates = last_to_read(p.arrived, sh);
  bad = __syncthreads_or(bad) || rows > p.max_rows;
  const bool short_of = taken > n_free || n_free > p.n_pages || n_free < 0;
  const bool ok = !bad && !short_of;
  if (!ok && blockIdx.x == 0 && threadIdx.x == 0)
    atomicCAS(p.status, 0, bad ? NE_DEV_BAD_SEQLEN : NE_DEV_NO_PAGES);

  const int id = blockIdx.x * kThreads + threadIdx.x, all = gridDim.x * kThreads;
  // The pages taken, into the block table.
  if (ok)
    for (int t = id; t < static_cast<int>(taken); t += all) {
      const int s = find(page_at, p.nseq, t);
      const int at = ((lens[s] + P1) >> p.page_shift) + t - page_at[s];
      p.block_table[static_cast<long long>(s) * p.max_pages + at] = __ldg(p.free_pages + n_free - 1 - t);
    }
  // Positions and slots, neighbouring rows in a thread's hands (a page looked up once).
  const int n_rows = ok ? static_cast<int>(rows) : 0;
  const bool aligned = ((reinterpret_cast<uintptr_t>(p.positions) | reinterpret_cast<uintptr_t>(p.slots)) & 15) == 0;
  for (int r0 = id * kRowsPerThread; r0 < p.n_tot; r0 += all * kRowsPerThread) {
    int s = r0 < n_rows ? find(row_at, p.nseq, r0) : 0;
    int pos[kRowsPerThread], slot[kRowsPerThread], seen = -1, page = -1;
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {
      const int r = r0 + i;
      pos[i] = slot[i] = -1;
      if (r >= n_rows) continue;
      while (row_at[s + 1] <= r) {
        ++s;
        seen = -1;
      }
      pos[i] = lens[s] + r - row_at[s];
      const int at = pos[i] >> p.page_shift;
      if (at != seen) {
        const int had = (lens[s] + P1) >> p.page_shift;
        page = at < had ? __ldcg(p.block_table + static_cast<long long>(s) * p.max_pages + at)
                        : __ldg(p.free_pages + n_free - 1 - (page_at[s] + at - had));
        seen = at;
      }
      if (page >= 0 && page < p.n_pages)
        slot[i] = (page << p.page_shift) + (pos[i] & P1);
      else
        atomicCAS(p.status, 0, NE_DEV_BAD_PAGE);
    }
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
  if (!updates) return;
  for (int s = threadIdx.x; s < p.nseq; s += kThreads)
    p.seq_lens_out[s] = ok ? lens[s] + row_at[s + 1] - row_at[s] : lens[s];
  if (threadIdx.x == 0) *p.n_free_out = ok ? n_free - static_cast<int>(taken) : n_free;
}

__global__ void __launch_bounds__(pages::kThreads) ne_kv_release_kernel(const PagesParams p) {
  using namespace pages;
  extern __shared__ int dyn[];
  __shared__ Shared sh;
  int* row_at = dyn;                   // (finished sequences before each)
  int* page_at = row_at + p.nseq + 1;  // [nseq + 1] first page given back by it
  pdl_wait();
  const int P1 = (1 << p.page_shift) - 1;
  const int n_free = __ldcg(p.n_free);
  bool bad = false;
  long long done, given;
  prefix_sums(p.nseq, row_at, page_at, sh, done, given, [&](int s, int& m, int& t) {
    m = __ldg(p.finished + s) != 0;
    if (!m) return;
    const int n = __ldcg(p.seq_lens + s);
    if (n < 0 || n > p.max_seqlen) {
      bad = true;
      return;
    }
    t = (n + P1) >> p.page_shift;
  });
  const bool updates = last_to_read(p.arrived, sh);
  bad = __syncthreads_or(bad);
  const bool over = n_free < 0 || n_free > p.n_pages || given > p.n_pages - n_free;
  const bool ok = !bad && !over;
  if (!ok && blockIdx.x == 0 && threadIdx.x == 0)
    atomicCAS(p.status, 0, bad ? NE_DEV_BAD_SEQLEN : NE_DEV_NO_PAGES);
  const int id = blockIdx.x * kThreads + threadIdx.x, all = gridDim.x * kThreads;
  if (ok)
    for (int t = id; t < static_cast<int>(given); t += all) {
      const int s = find(page_at, p.nseq, t);
      int* entry = p.block_table + static_cast<long long>(s) * p.max_pages + t - page_at[s];
      p.free_pages_out[n_free + t] = *entry;
      *entry = -1;
    }
  if (!updates || !ok) return;
  for (int s = threadIdx.x; s < p.nseq; s += kThreads)
    if (row_at[s + 1] != row_at[s]) p.seq_lens_out[s] = 0;
  if (threadIdx.x == 0) *p.n_free_out = n_free + static_cast<int>(given);
}

namespace {
cudaError_t launch(void (*kernel)(const PagesParams), int arrays, long long work,
                   const PagesParams& p, int sms, bool (&done)[64], cudaStream_t stream) {
  const int bytes = arrays * (p.nseq + 1) * static_cast<int>(sizeof(int));
  if (bytes > 48 * 1024 - static_cast<int>(sizeof(pages::Shared))) {
    const cudaError_t e =
        allow_smem(kernel, arrays * (kMaxPagedSequences + 1) * static_cast<int>(sizeof(int)), done);
    if (e != cudaSuccess) return e;
  }
  long long ctas = (work + pages::kThreads * pages::kRowsPerThread - 1) /
                   (pages::kThreads * pages::kRowsPerThread);
  const long long most = bytes <= 96 * 1024 ? 2LL * sms : sms;  // (resident at once)
  ctas = ctas < 1 ? 1 : ctas > most ? most : ctas;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(ctas)), dim3(pages::kThreads), bytes, stream,
                    p);
}
}  // namespace

cudaError_t launch_kv_reserve(const PagesParams& p, int sms, cudaStream_t stream) {
  static bool done[64] = {};
  return launch(ne_kv_reserve_kernel, 3, p.n_tot, p, sms, done, stream);
}

// (The pages given back are not known on the host: a CTA for every 1024 sequences.)
cudaError_t launch_kv_release(const PagesParams& p, int sms, cudaStream_t stream) {
  static bool done[64] = {};
  return launch(ne_kv_release_kernel, 2, static_cast<long long>(p.nseq) * pages::kRowsPerThread, p,
                sms, done, stream);
}

}  // namespace ne
