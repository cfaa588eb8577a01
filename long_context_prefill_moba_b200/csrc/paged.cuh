// Work division shared by the kernels of the attention over a paged cache.
//
// An item is one kv head of one sequence and `BR` of its rows (row i: new token
// i / G, query head i % G of the group), with the key tiles (BK keys each) that
// its last row may see.  The items of a call, in the order sequence, head, row
// tile, form one line of W key tiles; worker w of E takes tiles [w W / E,
// (w+1) W / E) of it, so that every worker has the same number of tiles (+- 1)
// whatever the lengths are, and no host knowledge of them is needed.  An item
// cut by a worker's border leaves fp32 partial results (at most two cut items
// a worker: slot 2w the one it continues, slot 2w + 1 the one it begins), which
// the combine kernel joins; the others are written by their worker.
#pragma once

#include <cuda.h>

#include "launch.h"

namespace moba {

struct PagedSeq {
  int first;   // row of its first new token
  int n;       // new tokens
  int len;     // keys, new tokens included
};

MOBA_DEV PagedSeq paged_seq(const int32_t* __restrict__ cu, const int32_t* __restrict__ kv_len, const PagedDims& dm,
                            int b) {
  PagedSeq s;
  s.first = min(max(cu[b], 0), dm.tokens);
  s.n = max(min(cu[b + 1], dm.tokens) - s.first, 0);
  // a length that the table's row cannot hold is cut to it (the status word says so)
  const int64_t cap = (int64_t)dm.max_pages << dm.page_shift;
  s.len = (int)min((int64_t)max(kv_len[b], 0), cap);
  return s;
}

// keys that the row tile [rt BR, ..) may see, in tiles; one tile at least, so
// that rows that see nothing are written too.  (Rows of a call are below 2^31.)
// X is an item's fixed cost in tiles: the line counts it as tiles at the item's
// start that hold no keys.
template <int BR, int BK, int X>
MOBA_DEV int paged_tiles(const PagedSeq& s, int G, int rt) {
  const uint32_t end = min((uint32_t)s.n * G, (uint32_t)(rt + 1) * BR);
  const int last = (int)((end - 1) / (uint32_t)G);
  const int keys = max(s.len - s.n + last + 1, 0);
  return max((keys + BK - 1) / BK, 1) + X;
}
template <int BR>
MOBA_DEV int paged_row_tiles(const PagedSeq& s, int G) { return (int)(((uint32_t)s.n * G + BR - 1) / BR); }

// tiles of one kv head of a sequence; the whole warp, each lane its own
// sequence (n = 0: none).  Long sequences are summed by all lanes in turn.
template <int BR, int BK, int X>
MOBA_DEV int64_t paged_head_tiles(const PagedSeq& s, int G) {
  const int nrt = paged_row_tiles<BR>(s, G), lane = threadIdx.x & 31;
  int64_t w = 0;
  for (int rt = 0; rt < min(nrt, 4); ++rt) w += paged_tiles<BR, BK, X>(s, G, rt);
  for (uint32_t todo = __ballot_sync(0xffffffffu, nrt > 4); todo != 0; todo &= todo - 1) {
    const int src = __ffs(todo) - 1;
    PagedSeq x;
    x.first = 0;
    x.n = __shfl_sync(0xffffffffu, s.n, src);
    x.len = __shfl_sync(0xffffffffu, s.len, src);
    const int m = __shfl_sync(0xffffffffu, nrt, src);
    int64_t v = 0;
    for (int rt = 4 + lane; rt < m; rt += 32) v += paged_tiles<BR, BK, X>(x, G, rt);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == src) w += v;
  }
  return w;
}

template <int NT>
struct PagedPlan {
  int64_t before[NT + 1];   // tiles before the sequences of thread t
  int64_t warp_sum[NT / 32];
};

// Whole block: exclusive prefix of v over its threads, and the sum.
template <int NT>
MOBA_DEV int64_t block_prefix(int64_t v, int64_t (&warp_sum)[NT / 32], int64_t& sum) {
  const int t = threadIdx.x, lane = t & 31;
  int64_t inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) warp_sum[t >> 5] = inc;
  __syncthreads();
  int64_t base = 0;
  for (int i = 0; i < (t >> 5); ++i) base += warp_sum[i];
  sum = base;
  for (int i = t >> 5; i < NT / 32; ++i) sum += warp_sum[i];
  __syncthreads();
  return base + inc - v;
}

// Whole block of NT threads: fills the plan, returns W.  `items` (where wanted): the
// items before the sequences of each thread, and the largest item's tiles.
template <int BR, int BK, int X, int NT>
MOBA_DEV int64_t paged_plan(PagedPlan<NT>& p, const int32_t* __restrict__ cu, const int32_t* __restrict__ kv_len,
                            const PagedDims& dm, int64_t* items = nullptr, int* largest = nullptr) {
  const int per = (dm.batch + NT - 1) / NT, t = threadIdx.x;
  int64_t w = 0, n = 0, sum;
  int most = 1;
  for (int i = 0; i < per; ++i) {
    const int b = t * per + i;
    PagedSeq x = {0, 0, 0};
    if (b < dm.batch) x = paged_seq(cu, kv_len, dm, b);
    w += paged_head_tiles<BR, BK, X>(x, dm.G) * dm.hkv;
    if (items != nullptr && x.n > 0) {
      const int nrt = paged_row_tiles<BR>(x, dm.G);
      n += (int64_t)nrt * dm.hkv;
      most = max(most, paged_tiles<BR, BK, X>(x, dm.G, nrt - 1));
    }
  }
  if (items != nullptr) {
    if (t == 0) *largest = 1;
    most = __reduce_max_sync(0xffffffffu, most);
    int64_t all;
    items[t] = block_prefix<NT>(n, p.warp_sum, all);   // its barriers order the line above before the maxima
    if ((t & 31) == 0) atomicMax(largest, most);
  }
  p.before[t] = block_prefix<NT>(w, p.warp_sum, sum);
  if (t == 0) p.before[NT] = sum;
  __syncthreads();
  return sum;
}

struct PagedItem {
  int b, h, rt;
  int tile, tiles;   // the position in it, and its key tiles
  PagedSeq s;
};

// the item that holds tile `at` of the line (at < W); the whole warp, same `at`
template <int BR, int BK, int X, int NT>
MOBA_DEV PagedItem paged_locate(const PagedPlan<NT>& p, int64_t at, const int32_t* __restrict__ cu,
                                const int32_t* __restrict__ kv_len, const PagedDims& dm) {
  const int per = (dm.batch + NT - 1) / NT, lane = threadIdx.x & 31;
  int lo = 0, hi = NT - 1;   // the last thread whose sequences begin at or before `at`
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.before[mid] <= at) lo = mid; else hi = mid - 1;
  }
  PagedItem it;
  int64_t off = at - p.before[lo], head = 0;
  it.b = lo * per;
  for (;; ++it.b) {
    it.s = paged_seq(cu, kv_len, dm, it.b);
    const PagedSeq none = {0, 0, 0};
    head = __shfl_sync(0xffffffffu, paged_head_tiles<BR, BK, X>(lane == 0 ? it.s : none, dm.G), 0);
    if (off < head * dm.hkv || it.b + 1 >= dm.batch) break;
    off -= head * dm.hkv;
  }
  it.h = (int)(off / head);
  off -= it.h * head;
  // the row tile: 32 at a time, the first whose tiles reach beyond `off`
  const int nrt = paged_row_tiles<BR>(it.s, dm.G);
  for (it.rt = 0;; it.rt += 32) {
    const int rt = it.rt + lane, mine = rt < nrt ? paged_tiles<BR, BK, X>(it.s, dm.G, rt) : 0;
    int64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, off < inc);
    if (hit != 0 || it.rt + 32 >= nrt) {
      const int src = hit != 0 ? __ffs(hit) - 1 : 0;
      it.rt += src;
      it.tiles = __shfl_sync(0xffffffffu, mine, src);
      it.tile = (int)(off - __shfl_sync(0xffffffffu, inc - mine, src));
      return it;
    }
    off -= __shfl_sync(0xffffffffu, inc, 31);
  }
}

// the item after a finished one; call only while tiles of the line are left
template <int BR, int BK, int X>
MOBA_DEV void paged_next(PagedItem& it, const int32_t* __restrict__ cu, const int32_t* __restrict__ kv_len,
                         const PagedDims& dm) {
  it.tile = 0;
  if (++it.rt >= paged_row_tiles<BR>(it.s, dm.G)) {
    it.rt = 0;
    if (++it.h >= dm.hkv) {
      it.h = 0;
      do {
        ++it.b;
        it.s = paged_seq(cu, kv_len, dm, it.b);
      } while (it.s.n == 0 && it.b + 1 < dm.batch);
    }
  }
  it.tiles = paged_tiles<BR, BK, X>(it.s, dm.G, it.rt);
}

// Rounds of whole items.  Workers that go through items of one head at the same
// pace share its keys in L2; workers at different places of them read the keys
// again and again from memory.  So each worker first takes k whole items, item
// r E + w in round r, and only the rest of the line is cut: worker w then takes
// of it what is missing to its W / E tiles.  k is W / E over the largest item's
// tiles (less one tile: every worker keeps a part of the rest, which the joining
// of cut items counts on).
template <int NT, int MAXE>
struct PagedRounds {
  int64_t items[NT + 1];      // items before the sequences of thread t
  int64_t start[MAXE + 1];    // where the workers' parts of the rest begin, as positions in the line
  unsigned long long whole[MAXE];
  int rounds, largest;
};

template <int BR, int BK, int X, int NT, int MAXE>
MOBA_DEV PagedItem paged_locate_item(const PagedRounds<NT, MAXE>& r, int64_t at, const int32_t* __restrict__ cu,
                                     const int32_t* __restrict__ kv_len, const PagedDims& dm) {
  const int per = (dm.batch + NT - 1) / NT;
  int lo = 0, hi = NT - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (r.items[mid] <= at) lo = mid; else hi = mid - 1;
  }
  PagedItem it;
  int64_t off = at - r.items[lo];
  int nrt = 0;
  it.b = lo * per;
  for (;; ++it.b) {
    it.s = paged_seq(cu, kv_len, dm, it.b);
    nrt = paged_row_tiles<BR>(it.s, dm.G);
    if (off < (int64_t)nrt * dm.hkv || it.b + 1 >= dm.batch) break;
    off -= (int64_t)nrt * dm.hkv;
  }
  it.h = (int)(off / nrt);
  it.rt = (int)(off % nrt);
  it.tile = 0;
  it.tiles = paged_tiles<BR, BK, X>(it.s, dm.G, it.rt);
  return it;
}

// Whole block, after paged_plan has filled r.items and r.largest.  Ends with a block barrier.
template <int BR, int BK, int X, int NT, int MAXE>
MOBA_DEV void paged_rounds(PagedRounds<NT, MAXE>& r, PagedPlan<NT>& p, int64_t W, int E, const int32_t* __restrict__ cu,
                           const int32_t* __restrict__ kv_len, const PagedDims& dm) {
  const int t = threadIdx.x, rounds = (int)((W / E - 1) / r.largest);
  int64_t before = 0, sum = 0;   // tiles in whole items: of the workers before this thread's, and of all
  if (rounds > 0) {
    for (int i = t; i < MAXE; i += NT) r.whole[i] = 0;
    __syncthreads();
    for (int64_t i = t; i < (int64_t)rounds * E; i += NT)
      atomicAdd(&r.whole[i % E], (unsigned long long)paged_locate_item<BR, BK, X>(r, i, cu, kv_len, dm).tiles);
    __syncthreads();
    before = block_prefix<NT>(t < E ? (int64_t)r.whole[t] : 0, p.warp_sum, sum);
  }
  if (t < E) r.start[t] = sum + t * W / E - before;
  if (t == 0) {
    r.start[E] = W;
    r.rounds = rounds;
  }
  __syncthreads();
}

// Workspace of a call: E headers, then the partial results.
struct PagedHeader {
  int parts;       // workers the item is spread over if this worker begins it, else 0
  int first, h, row0, rows;
  int pad[3];
};

struct PagedWs {
  PagedHeader* hdr;
  float *part_o, *part_ml;   // [2 E, BR, D] sums and [2 E, BR] (base, denominator)
};
inline PagedWs paged_ws_layout(void* ws, int64_t E, int BR) {
  PagedWs l;
  char* p = (char*)ws;
  l.hdr = (PagedHeader*)p;
  p += E * sizeof(PagedHeader);
  l.part_ml = (float*)p;
  p += 2 * E * BR * 2 * sizeof(float);
  l.part_o = (float*)p;
  return l;
}
inline size_t paged_ws_bytes(int64_t E, int BR, int D) {
  return E * sizeof(PagedHeader) + 2 * E * BR * (size_t)(D + 2) * sizeof(float);
}
cudaError_t launch_paged_combine(int dtype, int d, const PagedWs& l, int E, int BR, const PagedArgs& a, const PagedDims& dm,
                                 cudaStream_t stream, int* launches);

// 4-D tensor map of a bf16 pool, [pages][heads][slots][D], boxes of `box` slots x 64 channels, 128-byte swizzle
bool make_pool_map(CUtensorMap* map, const void* pool, const PagedDims& dm, int D, int64_t page_stride, int box);

// parts of the item that worker w begins at tile `at` of the line and that ends
// at tile `end`: the workers whose ranges reach into [at, end)
MOBA_DEV int paged_parts(int64_t end, int64_t W, int64_t E, int64_t w) {
  // the last worker v with v W / E < end
  int64_t v = (end * E + W - 1) / W;
  if (v > E) v = E;
  while (v > 0 && (v - 1) * W / E >= end) --v;
  while (v < E && v * W / E < end) ++v;
  return (int)(v - w);
}

}  // namespace moba
