// ne_items.cuh -- the work list of a packed batch with shared key/value heads,
// built by one CTA of the pass that runs before the attention kernel anyway.
//
// As ne_compact_items_kernel (ne_sched.cu): the items that are not empty,
// longest first by a counting sort over their steps, those of a sequence with
// bad bounds last.  The heads of a sequence have the same items, so the sort
// runs over (block, sequence) pairs and each pair is written n_heads times: a
// twelfth of the passes for 12 heads, and hidden behind the other CTAs (a
// launch of its own took 4-7 us before the attention could start).
#pragma once

#include "ne_sm100.cuh"

namespace ne {

enum class Items {
  kHeadPairs,  // forward: 128-row block n_blocks - 1 - i of two heads, steps = its key tiles
  kKeyTiles    // backward: key tile i, steps = query tiles from it to its sequence's end
};

// Items are numbered block * nseq * n_heads + sequence * n_heads + head; a
// forward's second kind (odd heads: 256-row block n_blocks2 - 1 - i of one head,
// steps = key tiles of its last row tile) follows from `second` on.
struct ItemList {
  Items kind = Items::kKeyTiles;
  int n_blocks = 0;   // blocks (key tiles) of the longest sequence
  int n_heads = 0;    // head pairs, or units per sequence and key tile
  int n_blocks2 = 0;
  int n_heads2 = 0;   // odd heads (0: none)
  int second = 0;
  int n_buckets = 0;  // the most steps an item can have, plus one
  int* out = nullptr; // [1 + number of items]: count, items; nullptr: none wanted
  int* counter = nullptr;  // forward: how many items past the first of each CTA are taken
};

// Bucket (steps) of pair i = block * nseq + sequence, the second kind's behind
// the first's n1; 0: bad bounds, -1: empty.
__device__ __forceinline__ int pair_bucket(const Problem& pb, const ItemList& l, int i, int n1) {
  const bool two = i >= n1;
  if (two) i -= n1;
  const int blk = i / pb.nseq, seq = i - blk * pb.nseq;
  int start, len;
  if (!seq_bounds(pb, seq, start, len, nullptr)) return 0;
  if (two) {
    const int b = l.n_blocks2 - 1 - blk;
    if (2 * b * kBM >= len) return -1;
    return (2 * b + 1) * kBM < len ? 2 * b + 2 : 2 * b + 1;
  }
  const int b = l.kind == Items::kKeyTiles ? blk : l.n_blocks - 1 - blk;
  if (b * kBM >= len) return -1;
  return l.kind == Items::kHeadPairs ? b + 1 : (len + kBM - 1) / kBM - b;
}

// Every thread of the CTA calls this; bucket: n_buckets ints of shared memory.
__device__ __forceinline__ void build_items(const Problem& pb, const ItemList& l, int* bucket) {
  const int n1 = l.n_heads ? l.n_blocks * pb.nseq : 0;
  const int n = n1 + (l.n_heads2 ? l.n_blocks2 * pb.nseq : 0);
  for (int b = threadIdx.x; b < l.n_buckets; b += blockDim.x) bucket[b] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int b = pair_bucket(pb, l, i, n1);
    if (b >= 0) atomicAdd(bucket + b, i < n1 ? l.n_heads : l.n_heads2);
  }
  __syncthreads();
  if (threadIdx.x < 32) {  // first slots: the most steps first, bucket 0 last
    const int lane = threadIdx.x;
    int at = 0;
    for (int b0 = l.n_buckets - 1; b0 >= 0; b0 -= 32) {
      const int b = b0 - lane;
      const int c = b >= 0 ? bucket[b] : 0;
      int v = c;
#pragma unroll
      for (int sh = 1; sh < 32; sh <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, sh);
        if (lane >= sh) v += u;
      }
      if (b >= 0) bucket[b] = at + v - c;
      at += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) l.out[0] = at;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int b = pair_bucket(pb, l, i, n1);
    if (b < 0) continue;
    const int heads = i < n1 ? l.n_heads : l.n_heads2;
    const int first = i < n1 ? i * heads : l.second + (i - n1) * heads;
    // (items of equal length in no fixed order: each is computed the same way
    // by whichever CTA gets it)
    int* dst = l.out + 1 + atomicAdd(bucket + b, heads);
    for (int h = 0; h < heads; ++h) dst[h] = first + h;
  }
}

}  // namespace ne
