// Shared definitions of the tree attention kernels: launch parameters, the
// geometry of a lane, and the walk that turns an item index into work.
//
// A lane's q_len rows are the nodes of a tree of drafted tokens (parents
// precede children); with past = ctx - q_len, node j's K/V row is key
// past + j and node j attends
//   keys 0 .. past - 1                      (the lane's cache) and
//   key past + i for i = j and every ancestor i of j.
// Scores t = scale q.k, p = softmax over those keys, out = sum p v.
//
// The keys of a lane are cut into splits of tree_split_len(past, row tiles)
// keys; the last split also takes the tree's own keys. The cut depends on the
// lane's own lengths alone, a split is reduced in ascending key order, and
// the splits are folded left to right in fp32, so a row's bits depend on its
// own lane only.
#pragma once

#include <cfloat>

#include "pa_common.cuh"

namespace pa {

constexpr int kTreeMaxNodes = PA_TREE_MAX_NODES;
// (row, head) pairs of one kv head that a row tile holds: M of the products
constexpr int kTreeRows = 128;

struct TreeParams {
  const void* q;
  void* out;
  const void* k_cache;
  const void* v_cache;
  const int* block_tables;
  const int* cu_seqlens;
  const int* ctx_lens;
  const int* parents;
  int* status;
  int max_blocks;
  int B, T, H, Hkv, D, bs, NB;
  int max_q_len, max_ctx_len;
  int tile_rows;     // nodes per row tile: floor(pairs per tile / g)
  int split0;        // shortest split
  int grow;          // 1: splits grow with the lane's pairs (tree_split_len), 0: not
  float scale_log2;  // scale * log2(e) (* k_scale): base-2 score domain
  float v_scale;     // factor of every output (1 but for e4m3 caches)
  float2* ml;        // partials: (m, l) per (row, split) pair and head
  float* acc;        // and D sums
  long long capacity;  // pairs the workspace holds
  uint8_t* q_pieces;   // e4m3 caches: q as two e4m3 pieces [2][T][H][D]
  uint8_t* q_exp;      // and the biased exponent of each row's largest |q| [T][H]
  unsigned long long* counter;  // next item (0 at launch), or NULL: items by CTA index
  int4* lane_info;     // per lane: first pair (two words), nodes, splits (0 nodes: nothing to fold)
  long long wait_cycles;
  long long skip_item;  // test hook: no copy of this item's first K tile (-1: none)
};

// Split length in keys, from the lane's own keys and (node, head) pairs per
// kv head. Short splits keep few lanes' long contexts on many SMs; a split
// writes its pairs' partials (D + 2 floats each) beside the 4 D bytes a key
// of K/V, so its length grows with the pairs: 16 keys per pair up to 2048,
// which keeps the partials under a sixteenth of the K/V bytes one way for
// lanes of one row tile (16 nodes x 64 heads over 19 lanes of 8176 keys: 120
// us; with 8 keys per pair 133, with 4 163). At most PA_TREE_MAX_SPLITS
// splits bound the workspace.
__host__ __device__ __forceinline__ int tree_split_len(long long past, int pairs, int split0) {
  long long s = split0;
  while (s < 2048 && s < 16LL * pairs) s <<= 1;
  while ((past + s - 1) / s > PA_TREE_MAX_SPLITS) s <<= 1;
  return (int)(s < 0x40000000LL ? s : 0x40000000LL);
}

// What a split leaves of a row: its maximum and sum. A split whose scores are
// all -inf has l = 0 and sums of 0; its maximum is kept finite, since two such
// splits must not meet in the fold as -inf - -inf.
__device__ __forceinline__ float2 tree_ml(float m, float l) { return make_float2(fmaxf(m, -FLT_MAX), l); }

struct TreeLane {
  int q, c, cu0;  // nodes, keys (nodes included), first row
  int ns, len;    // splits and their length
  int tiles;      // row tiles
};

// Geometry of lane b; false (with a status flag when `report`) for a lane
// that is malformed or has no rows.
__device__ __forceinline__ bool tree_lane(const TreeParams& p, int b, bool report,
                                          TreeLane& ln) {
  const int cu1 = p.cu_seqlens[b + 1];
  ln.cu0 = p.cu_seqlens[b];
  ln.c = p.ctx_lens[b];
  ln.q = cu1 - ln.cu0;
  ln.ns = ln.len = ln.tiles = 0;
  int bad = 0;
  if (ln.cu0 < 0 || cu1 < ln.cu0 || cu1 > p.T || (b == 0 && ln.cu0 != 0) ||
      (b == p.B - 1 && cu1 != p.T))
    bad = PA_FLAG_CU_SEQLENS;
  else if (ln.c < 0 || (long long)ln.c > (long long)p.max_blocks * p.bs)
    bad = PA_FLAG_CTX_RANGE;
  else if (ln.q > ln.c)
    bad = PA_FLAG_QLEN_RANGE;
  else if (ln.q > p.max_q_len || ln.c > p.max_ctx_len)
    bad = PA_FLAG_HOST_BOUND;
  if (bad) {
    if (report) raise_flag(p.status, bad);
    ln.q = 0;
    return false;
  }
  if (ln.q == 0) return false;
  ln.tiles = (ln.q + p.tile_rows - 1) / p.tile_rows;
  const int past = ln.c - ln.q;
  ln.len = tree_split_len(past, p.grow * ln.q * (p.H / p.Hkv), p.split0);
  ln.ns = past > ln.len ? (past + ln.len - 1) / ln.len : 1;
  return true;
}

// Items in order: by length class, longest first, where CTAs take several in
// turn (the last to start are then short: 24 ragged lanes of 3000 keys in the
// median take 96 us, 109 in lane order); within a class by lane, split, kv
// head, row tile -- the tiles that read the same keys next to each other. A
// warp walks the lanes 32 at a time, once per class (each thread holds one
// lane of the window), with running sums of the items and of the partial
// pairs before the window: ascending item indexes need no plan in memory.
constexpr int kTreeClasses = 4;
// Class of a split of n 64-key units: 24 and more, 16, 8, fewer.
__device__ __forceinline__ int tree_class(int n) { return n >= 24 ? 0 : n >= 16 ? 1 : n >= 8 ? 2 : 3; }

struct TreeWalk {
  int cls;                     // class of the walk
  int fulls, lasts;            // this thread's lane: its full splits and last split in the class
  int b0;                      // first lane of the window
  long long items0, pairs0;    // before the window
  long long items_in, items_ex, pair_base;  // this thread's lane
  long long win_items, win_pairs;
  TreeLane ln;
  bool ok;

  __device__ __forceinline__ static long long warp_scan(long long v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    return v;
  }
  // the window's lanes
  __device__ __forceinline__ void window(const TreeParams& p, int lane, bool report) {
    const int b = b0 + lane;
    ok = b < p.B && tree_lane(p, b, report, ln);
    const long long pairs = ok && ln.ns > 1 ? (long long)ln.q * ln.ns : 0;
    const long long pin = warp_scan(pairs, lane);
    pair_base = pairs0 + pin - pairs;
    if (ok && pairs0 + pin > p.capacity && pairs > 0) {
      if (report) raise_flag(p.status, PA_FLAG_WORKSPACE);
      ok = false;
    }
    // one reporting warp sees every lane: it leaves the fold what it needs
    if (report && p.lane_info && b < p.B)
      p.lane_info[b] = make_int4((int)(uint32_t)pair_base, (int)(pair_base >> 32), ok ? ln.q : 0, ln.ns);
    win_pairs = __shfl_sync(0xffffffffu, pin, 31);
  }
  // and their items of the class
  __device__ __forceinline__ void count(const TreeParams& p, int lane) {
    const bool all = !p.counter;  // one class
    fulls = ok && (all || tree_class(ln.len / 64) == cls) ? ln.ns - 1 : 0;
    lasts = ok && (all || tree_class((ln.c - (ln.ns - 1) * ln.len + 63) / 64) == cls) ? 1 : 0;
    const long long items = ok ? (long long)(fulls + lasts) * ln.tiles * p.Hkv : 0;
    items_in = warp_scan(items, lane);
    items_ex = items_in - items;
    win_items = __shfl_sync(0xffffffffu, items_in, 31);
  }
  __device__ __forceinline__ void start(const TreeParams& p, int lane, bool report) {
    b0 = cls = 0;
    items0 = pairs0 = 0;
    window(p, lane, report);
    count(p, lane);
  }
  // The window holding `item` (ascending from call to call); false past the
  // last item. On true, src is the thread whose lane has it; item_of says
  // which of the lane's items it is.
  __device__ __forceinline__ bool find(const TreeParams& p, int lane, bool report,
                                       long long item, int& src) {
    while (item >= items0 + win_items) {
      const bool over = b0 + 32 >= p.B;
      if (over && (!p.counter || cls + 1 == kTreeClasses)) return false;
      items0 += win_items;
      pairs0 = over ? 0 : pairs0 + win_pairs;
      b0 = over ? 0 : b0 + 32;
      cls += over;
      if (p.B > 32) window(p, lane, report && cls == 0);  // else the same lanes again
      count(p, lane);
    }
    src = __ffs(__ballot_sync(0xffffffffu, items_in > item - items0)) - 1;
    return true;
  }

  // The reporting warp, at its end: the windows that it has not come to (it may
  // leave early, when a wait runs out), so that the fold finds every lane's entry.
  __device__ __forceinline__ void finish(const TreeParams& p, int lane) {
    while (cls == 0 && b0 + 32 < p.B) {
      pairs0 += win_pairs;
      b0 += 32;
      window(p, lane, true);
    }
  }

  // Split of the thread's lane that `item` belongs to, and the item's index
  // among the split's (kv head, row tile) pairs.
  __device__ __forceinline__ void item_of(const TreeParams& p, long long item, int& split, int& rest) const {
    const int per = ln.tiles * p.Hkv;
    const int rel = (int)(item - items0 - items_ex);
    const int i = rel / per;
    split = i < fulls ? i : ln.ns - 1;
    rest = rel - i * per;
  }
};

// Visible keys of node `node` among the 32 NW keys from tile0 on, as bits:
// cache keys (below past), then the node's own chain of ancestors. A parent
// outside [-1, child) ends the chain (the caller raises the flag).
template <int NW>
__device__ __forceinline__ void tree_mask(const int* parents, int node, int past, int tile0,
                                          uint32_t (&w)[NW]) {
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    const int left = past - (tile0 + 32 * i);
    w[i] = left >= 32 ? 0xffffffffu : left > 0 ? (1u << left) - 1u : 0u;
  }
  for (int a = node; a >= 0;) {
    const int c = past + a - tile0;
    if (c < 0) break;  // ancestors only have smaller indexes
    if (c < 32 * NW) {
      const uint32_t bit = 1u << (c & 31);
#pragma unroll
      for (int i = 0; i < NW; ++i)
        if ((c >> 5) == i) w[i] |= bit;
    }
    const int up = parents[a];
    if (up >= a) break;
    a = up;
  }
}

}  // namespace pa
