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
  kRowPairs,   // forward: block n_blocks - 1 - i of 256 rows, steps = key tiles of its last tile
  kHeadPairs,  // forward: block n_blocks - 1 - i of 128 rows, steps = its key tiles
  kKeyTiles    // backward: key tile i, steps = query tiles from it to its sequence's end
};

struct ItemList {
  Items kind = Items::kRowPairs;
  int n_blocks = 0;   // blocks (key tiles) of the longest sequence
  int n_heads = 0;    // heads, head pairs, or units per sequence and key tile
  int n_buckets = 0;  // the most steps an item can have, plus one
  int* out = nullptr; // [1 + n_blocks * nseq * n_heads]: count, items; nullptr: none wanted
};

// Bucket (steps) of pair i = block * nseq + sequence; 0: bad bounds, -1: empty.
__device__ __forceinline__ int pair_bucket(const Problem& pb, const ItemList& l, int i) {
  const int blk = i / pb.nseq, seq = i - blk * pb.nseq;
  int start, len;
  if (!seq_bounds(pb, seq, start, len, nullptr)) return 0;
  const int b = l.kind == Items::kKeyTiles ? blk : l.n_blocks - 1 - blk;
  if (l.kind == Items::kRowPairs) {
    if (2 * b * kBM >= len) return -1;
    return (2 * b + 1) * kBM < len ? 2 * b + 2 : 2 * b + 1;
  }
  if (b * kBM >= len) return -1;
  return l.kind == Items::kHeadPairs ? b + 1 : (len + kBM - 1) / kBM - b;
}

// Every thread of the CTA calls this; bucket: n_buckets ints of shared memory.
__device__ __forceinline__ void build_items(const Problem& pb, const ItemList& l, int* bucket) {
  const int n = l.n_blocks * pb.nseq;
  for (int b = threadIdx.x; b < l.n_buckets; b += blockDim.x) bucket[b] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int b = pair_bucket(pb, l, i);
    if (b >= 0) atomicAdd(bucket + b, 1);
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
    if (lane == 0) l.out[0] = at * l.n_heads;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int b = pair_bucket(pb, l, i);
    if (b < 0) continue;
    const int slot = atomicAdd(bucket + b, 1);
    int* dst = l.out + 1 + static_cast<long long>(slot) * l.n_heads;
    // (items of equal length in no fixed order: each is computed the same way
    // by whichever CTA gets it)
    for (int h = 0; h < l.n_heads; ++h) dst[h] = i * l.n_heads + h;
  }
}

}  // namespace ne
