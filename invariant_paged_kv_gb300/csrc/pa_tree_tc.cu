// Tree attention over bf16 and e4m3 caches on the 5th-generation tensor
// cores (tcgen05).
//
// A row tile is up to 128 (node, head) pairs of one lane and one kv head: R =
// floor(128 / g) nodes times the g query heads, so that a key staged once
// serves every head of the group, and a tree of a handful of nodes still
// fills rows of the product. Work item = (lane, split, kv head, row tile);
// keys go by in tiles of 64, and two CTAs share an SM: one streams while the
// other starts or ends an item (a split's first scores and last stores leave
// a CTA's loads idle for a quarter of the time that 1024 keys take).
//   S = Q K^T         M = 128, N = 64, fp32 in TMEM, two buffers: S of tile t + 1
//                     is made while tile t is in the softmax
//   p, m, l           thread r = row r: one read of its 64 scores, p written
//                     back over S as 16-bit values (bf16) or 8-bit pieces (e4m3)
//   O = O alpha + P V A = P from TMEM, B = V (MN-major)
// The running max moves only when a tile's exceeds it by more than kLazy
// (log2), so O is seldom rescaled. bf16: p is rounded to bf16 (within 2^-8 of
// itself: the products take 16-bit operands), l adds the p before rounding.
//
// Lanes of one row tile are bound by reading K and V once (24 ragged lanes of
// 3000 keys in the median: 416 MB in 76 us, 5.5 TB/s; e4m3, 32 lanes: 258 MB in
// 74 us, there the softmax and its 8-bit pieces take longer); those of several
// read them from L2 (their items are neighbours in the order) and are bound
// by the chain softmax - P V - next S of a CTA, whose products take their
// turns with the other CTA's (64 nodes x 64 heads over 19 lanes of 8128 keys:
// 308 us, 1.05 PFLOP/s; of a tile's 1800 cycles a CTA's products are being
// issued for 770, its softmax works for 870). A variant with one CTA per SM
// and two row tiles over each staged tile of 128 keys was no faster than this
// one's first form there (343 us both) and slower wherever lanes had one.
//
// A mask is needed only in the tiles that hold the lane's own nodes ("tree
// tiles", in its last split): there each thread walks up its node's parents
// and keeps 64 bits. A hidden key's score is replaced by -inf, so infinities
// and NaN in it do not reach the row. P V multiplies every V row of the tile,
// and 0 * Inf is NaN: a warp of its own looks over a tree tile's V rows before
// the product, zeroes those past the lane's end and the values that are not
// finite, and the epilogue adds the latter to the rows that attend them.
//
// e4m3 caches are multiplied as they are (kind::f8f6f4), nothing is converted
// on the way: q and p are split into 8-bit pieces whose products with the
// codes are exact in the accumulator.
//   q  = q_hi + q_lo, both e4m3, q scaled by a power of two per row so that its
//        largest element is in [128, 256): a bf16 value has 8 significant
//        bits, a piece 4, so the sum is exact down to 2^-9 of the row's
//        largest element and within 2^-17 of it below; S = q_hi K^T + q_lo K^T
//   p  = p_1 + p_2 + p_3, e5m2 (3 significant bits each): the upper bytes of
//        an f16 value and of what is left of it. p 2^11 (at most 2^15: kLazy is
//        4 here) is rounded to f16, then to 9 significant bits: within
//        2^-9 + 2^-11 of itself, and 2^-27 of the row's largest p for tiny
//        ones; O sums three products
// That costs 2 and 3 products of the double-rate kind where a conversion of
// K and V to f16 would cost 2 cvt instructions per 4 codes and as much shared
// memory traffic again.
//
// Warps: 0-3 softmax, 4 products, 5 finds the items and loads K, 7 loads Q and
// V (TMA, a box per block of the table), 6 looks over tree tiles. K and V
// tiles share one ring; every wait is bounded (PA_FLAG_TIMEOUT).
#include "pa_tc_wait.cuh"
#include "pa_tree.cuh"

namespace pa {

namespace {

constexpr int kKeys = 64;
constexpr int kRows = kTreeRows;
constexpr int kThreads = 8 * 32;
constexpr uint32_t kTmemCols = 256;  // S: 2 x 64, O: 128
constexpr int kSlots = 4;            // item queue
constexpr int kBadSlots = 8;
constexpr int kNodes = kTreeMaxNodes;

__device__ __forceinline__ void st_global_v8(void* ptr, const uint32_t (&r)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(ptr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void st_shared_v4(uint32_t a, uint32_t x, uint32_t y, uint32_t z,
                                             uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

// 8 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// 5-D tiled TMA load global -> shared with an L2 policy, completion counted on `bar`.
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int c3, int c4,
                                            uint32_t bar, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %2, %2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(c3), "r"(c4), "r"(bar), "l"(pol)
      : "memory");
}

// Element d of a V row in global memory.
template <int D, bool FP8>
__device__ __forceinline__ float v_elem(const TreeParams& p, long long slot, int kvh, int d) {
  const size_t at = ((size_t)slot * p.Hkv + kvh) * D + d;
  if (FP8) {
    const uint32_t c = static_cast<const uint8_t*>(p.v_cache)[at];
    return f16_lo(e4m3x2_to_f16x2(c));
  }
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p.v_cache)[at]);
}

// (rare) Add the values that P V left out because they are not finite -- of
// the nodes in badw that the row attends -- to what the row has stored. Any
// weight leaves an infinity or NaN what it is, but one of 0 (with m the row's
// maximum) makes NaN of an infinity, as the product makes of a cache key's. A
// call of its own, so that its code stays out of the way.
template <int D, bool FP8>
__device__ __noinline__ void tree_add_bad(const TreeParams& p, int lane_b, int kvh, int past, int node,
                                          const int* par, const uint32_t* badw, bool single,
                                          size_t out_at, long long entry, float m) {
  const int* table = p.block_tables + (size_t)lane_b * p.max_blocks;
  for (int a = node; a >= 0;) {
    if ((badw[a >> 5] >> (a & 31)) & 1u) {
      const int key = past + a;
      int blk = table[key / p.bs];
      blk = blk < 0 || blk >= p.NB ? 0 : blk;
      const long long slot = (long long)blk * p.bs + key % p.bs;
      bool nothing = false;
      if (!FP8) {  // (e4m3 codes have no infinity)
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + out_at;
        const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(p.k_cache) + ((size_t)slot * p.Hkv + kvh) * D;
        float s = 0.f;
        for (int d = 0; d < D; ++d) s = fmaf(__bfloat162float(q[d]), __bfloat162float(k[d]), s);
        nothing = ex2_approx(s * p.scale_log2 - m) == 0.f;
      }
      for (int d = 0; d < D; ++d) {
        float v = v_elem<D, FP8>(p, slot, kvh, d);
        if (isfinite(v)) continue;
        if (nothing) v = NAN;
        if (single) {
          __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + out_at + d;
          *o = __float2bfloat16_rn(__bfloat162float(*o) + v);
        } else {
          p.acc[(size_t)entry * D + d] += v;
        }
      }
    }
    const int up = par[a];
    a = up < a ? up : -1;
  }
}

// Store 32 sums of one row (elements 32 c on): as the output (scaled by inv)
// or as a split's partial sums.
template <int D>
__device__ __forceinline__ void tree_emit(const TreeParams& p, const uint32_t (&ov)[32], int c,
                                          bool single, float inv, size_t out_at, long long entry) {
  if (single) {
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + out_at + c * 32;
#pragma unroll
    for (int j = 0; j < 32; j += 8) {
      uint32_t v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        v[k] = pack_bf16x2(__uint_as_float(ov[j + 2 * k]) * inv, __uint_as_float(ov[j + 2 * k + 1]) * inv);
      *reinterpret_cast<uint4*>(out + j) = make_uint4(v[0], v[1], v[2], v[3]);
    }
  } else {
    float* acc = p.acc + (size_t)entry * D + c * 32;
#pragma unroll
    for (int j = 0; j < 32; j += 8) {
      const uint32_t v[8] = {ov[j], ov[j + 1], ov[j + 2], ov[j + 3],
                             ov[j + 4], ov[j + 5], ov[j + 6], ov[j + 7]};
      st_global_v8(acc + j, v);
    }
  }
}

template <int D, bool FP8>
struct Cfg {
  // a half: 64 elements (bf16) or D codes (e4m3) of each row; rows of kRowB bytes
  static constexpr int kRowB = FP8 ? D : 128;
  static constexpr int kHalves = FP8 ? 1 : D / 64;
  // a K or V tile: 8-key groups, in each the halves' 8 rows one after another
  // (one box brings a block's groups with both halves)
  static constexpr int kHalf = 8 * kRowB;
  static constexpr int kGroup = kHalves * kHalf;
  static constexpr int kTileBytes = kKeys / 8 * kGroup;
  static constexpr int kQPart = kRows * kRowB;  // a half (bf16) or a piece (e4m3) of Q
  static constexpr int kQParts = FP8 ? 2 : kHalves;
  static constexpr int kQBytes = kQParts * kQPart;
  // 113 KB a CTA: 80 KB of ring at D = 128, 64 KB at D = 64
  static constexpr int kRing = D == 128 ? (FP8 ? 10 : 5) : (FP8 ? 16 : 8);
  static constexpr int kRing0 = kQBytes;
  static constexpr int kCtl = kRing0 + kRing * kTileBytes;
  static constexpr float kLazy = FP8 ? 4.f : 8.f;
  static constexpr float kBias = FP8 ? 11.f : 0.f;  // log2 of the factor on p
};

struct Item {
  int lane, kvh, node0, q, c, cu0, ns, split;
  int kt0, nkt;  // first key tile and their number (0: no more items)
  int tree0;     // first tree tile, relative to kt0 (>= nkt: none)
  long long pair_base;
};

template <int kRing>
struct Ctl {
  // ring slots: the tile has landed, the products that read it are done (of K:
  // S is there, of V: O is); one commit each, for every warp that waits for it
  uint64_t full[kRing], done[kRing];
  // tree tiles of V: a load into the slot is under way (the look-over warp
  // waits for full[] only from then on: a parity wait must not meet a barrier
  // more than one phase away), and the tile has been looked over
  uint64_t go[kRing], fixed[kRing];
  uint32_t uses[kRing];  // loads into each slot so far
  uint64_t qfull;
  uint64_t p[2];  // by tile parity
  uint64_t fin;
  uint64_t item_full[kSlots], item_free[kSlots];
  Item items[kSlots];
  // nodes whose V holds a value that is not finite, by item number mod 8 (the
  // look-over warp is at most kSlots items ahead of the epilogue that reads it)
  uint32_t bad[kBadSlots][kNodes / 32];
  uint32_t tmem;
  int abort;
};

template <int D, bool FP8>
using CtlOf = Ctl<Cfg<D, FP8>::kRing>;

template <int D, bool FP8>
constexpr int smem_bytes() {
  return Cfg<D, FP8>::kCtl + (int)sizeof(CtlOf<D, FP8>);
}
static_assert(smem_bytes<128, false>() <= 115712 && smem_bytes<128, true>() <= 115712,
              "two CTAs an SM");

// Address of 16-byte chunk ch of row r < 8 of a swizzled half whose rows have
// kRowB bytes (the 128-byte or the 64-byte pattern).
template <int kRowB>
__device__ __forceinline__ uint32_t chunk_at(uint32_t half, int r, int ch) {
  return kRowB == 128 ? half + r * 128 + ((ch ^ r) << 4) : half + r * 64 + ((ch ^ (r >> 1)) << 4);
}

// Shared-memory matrix descriptor: 8-row groups `sbo` apart, `lbo` between
// 64-element halves where the operand is MN-major.
template <int kRowB>
__device__ __forceinline__ uint64_t half_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = umma_desc_sw128(saddr, lbo, sbo);
  if (kRowB == 64) d = (d & ~(7ull << 61)) | (4ull << 61);  // 64-byte swizzle
  return d;
}

// kind::f8f6f4 instruction descriptor: A e4m3 (0) or e5m2 (1), B e4m3, fp32.
constexpr uint32_t idesc_f8(int a_fmt, int M, int N, int b_mn) {
  return (1u << 4) | ((uint32_t)a_fmt << 7) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void umma_f8_w(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_f8_tmem_a_w(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc,
                                                 uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 16-bit packed difference of f16 pairs (exact where it is used).
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Places of tile kt's K and V among an item's 2 nkt ring tiles: K 0, K 1, V 0,
// K 2, V 1, .., the order in which the products take them, so that every slot
// comes free as early before its next use (with V kt next to K kt, a K tile has
// one tile's time to land: 24 ragged lanes 93.8 us, so 90.4).
__device__ __forceinline__ uint32_t k_at(int kt) { return kt ? 2 * kt - 1 : 0; }
__device__ __forceinline__ uint32_t v_at(int kt, int nkt) { return kt + 1 < nkt ? 2 * kt + 2 : 2 * nkt - 1; }

// wait_or_abort with the loop for a barrier that is not ready as a call of its
// own, shared by every wait. A warp's role is a different part of the code, two
// CTAs run them all at once on an SM, and they contend for its instruction
// cache: with the loop in each place up to 17 % of the fetches missed it (32
// ragged e4m3 lanes: 91 us, 81 with the call; 32 bf16 lanes of 64 nodes, 4000
// keys in the median, 372 and 362).
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                       int* status, long long limit) {
  return wait_or_abort_1(bar, parity, abort_flag, status, limit);
}
// Whether the phase of that parity is over, as this thread sees it.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_w(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                       int* status, long long limit) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity) ||
                                     wait_slow(bar, parity, abort_flag, status, limit));
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads, 2)
    tree_tc_kernel(const TreeParams p, const __grid_constant__ CUtensorMap tmQ,
                   const __grid_constant__ CUtensorMap tmQh,
                   const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV) {
  using C = Cfg<D, FP8>;
  extern __shared__ __align__(1024) uint8_t dsmem[];
  auto& ctl = *reinterpret_cast<CtlOf<D, FP8>*>(dsmem + C::kCtl);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(dsmem);
  const uint32_t sQ = base, sR = base + C::kRing0;
  if (base & 1023u) {  // the swizzled tiles need it; dynamic shared memory alone starts so
    if (threadIdx.x == 0) raise_flag(p.status, PA_FLAG_TIMEOUT);
    return;
  }
  const uint32_t bfull = smem_u32(&ctl.full[0]), bdone = smem_u32(&ctl.done[0]);
  const uint32_t bgo = smem_u32(&ctl.go[0]), bfixed = smem_u32(&ctl.fixed[0]);
  const uint32_t bqf = smem_u32(&ctl.qfull);
  auto bP = [&](uint32_t t) -> uint32_t { return smem_u32(&ctl.p[0]) + 8 * (t & 1); };
  const uint32_t bitem = smem_u32(&ctl.item_full[0]), bfree = smem_u32(&ctl.item_free[0]);

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kRing; ++i) {
      ctl.uses[i] = 0;
      mbar_init(bfull + 8 * i, 1);
      mbar_init(bdone + 8 * i, 1);
      mbar_init(bgo + 8 * i, 1);
      mbar_init(bfixed + 8 * i, 1);
    }
    mbar_init(bqf, 1);
    for (int i = 0; i < 2; ++i) mbar_init(bP(i), kRows);
    mbar_init(smem_u32(&ctl.fin), 1);
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(bitem + 8 * i, 1);
      mbar_init(bfree + 8 * i, 7);  // every warp but the one that finds items reads them
    }
    ctl.abort = 0;
    fence_mbar_init();
  }
  if (warp == 5 && lane == 0) {
    prefetch_tensormap(&tmQ);
    prefetch_tensormap(&tmQh);
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  if (warp == 4) tmem_alloc(smem_u32(&ctl.tmem), kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem, tO = tmem + 128;
  auto tS = [&](uint32_t t) -> uint32_t { return tmem + 64 * (t & 1); };
  volatile int* ab = &ctl.abort;
  const long long lim = p.wait_cycles;
  const int g = p.H / p.Hkv;
  // A lane of at most 64 pairs needs half of the rows: in one of the SM's two
  // CTAs (told apart by their TMEM) it takes the upper half, whose softmax
  // warps sit on the other two schedulers. No row's bits depend on its place.
  const int half_rows = 64 / g;
  const int upper = (tmem & 0xffffu) >= kTmemCols ? 64 : 0;

  // the products that read the tile at place f are done
  auto wait_done = [&](uint32_t f) -> bool {
    return wait_w(bdone + 8 * (f % C::kRing), (f / C::kRing) & 1, ab, p.status, lim);
  };
  auto read_item = [&](uint32_t n, Item& it) -> bool {
    if (!wait_w(bitem + 8 * (n % kSlots), (n / kSlots) & 1, ab, p.status, lim)) return false;
    it = ctl.items[n % kSlots];
    __syncwarp();
    if (lane == 0) mbar_arrive(bfree + 8 * (n % kSlots));
    return it.nkt > 0;
  };
  // running counters, the same in every role: items, ring tiles, key tiles
  uint32_t n_item = 0, n_ring = 0, n_t = 0;
  uint32_t issued_q = 0;  // warp 7: Q loads under way or landed

  // e4m3: q's pieces come from a kernel before, which this one may overlap
  if (FP8) asm volatile("griddepcontrol.wait;" ::: "memory");

  if (warp == 5 || warp == 7) {
    // -------- loads: warp 5 finds the items and loads K, warp 7 Q and V -------
    // (one warp for both was slower: 330 us, two 312, for 19 lanes of 64 nodes x
    // 64 heads over 8128 keys)
    const bool vs = warp == 7;
    const CUtensorMap* tm = vs ? &tmV : &tmK;
    // keys that one item reads go first from L2, those of several row tiles last
    const uint64_t once = l2_evict_first(), keep = l2_evict_last();
    const int blocks = kKeys / p.bs;
    uint32_t q_last = 0;  // place of the last K tile of the item before
    TreeWalk walk;
    if (!vs) walk.start(p, lane, blockIdx.x == 0);
    for (;; ++n_item) {
      const uint32_t n = n_item;
      Item it;
      long long idx = -1;
      if (vs) {
        if (!read_item(n, it)) break;
      } else {
        if (n >= kSlots &&
            !wait_w(bfree + 8 * (n % kSlots), ((n / kSlots) - 1) & 1, ab, p.status, lim))
          break;
        // the first item by CTA index, the others as CTAs become free (a counter
        // decides only who computes an item)
        idx = blockIdx.x + (long long)n * gridDim.x;
        if (p.counter && n > 0) {
          if (lane == 0) idx = (long long)gridDim.x + (long long)atomicAdd(p.counter, 1ull);
          idx = __shfl_sync(0xffffffffu, idx, 0);
        }
        int src = 0;
        const bool have = walk.find(p, lane, blockIdx.x == 0, idx, src);
        if (have) {
          if (lane == src) {
            const TreeLane& ln = walk.ln;
            int rest;
            walk.item_of(p, idx, it.split, rest);
            it.kvh = rest / ln.tiles;
            it.node0 = (rest - it.kvh * ln.tiles) * p.tile_rows;
            it.lane = walk.b0 + lane;
            it.q = ln.q;
            it.c = ln.c;
            it.cu0 = ln.cu0;
            it.ns = ln.ns;
            it.kt0 = it.split * (ln.len / kKeys);
            const bool last = it.split + 1 == ln.ns;
            const int end = last ? (ln.c + kKeys - 1) / kKeys : (it.split + 1) * (ln.len / kKeys);
            it.nkt = end - it.kt0;
            it.tree0 = last ? (ln.c - ln.q) / kKeys - it.kt0 : it.nkt;
            it.pair_base = walk.pair_base;
            ctl.items[n % kSlots] = it;
          }
        } else if (lane == 0) {
          ctl.items[n % kSlots].nkt = 0;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bitem + 8 * (n % kSlots));
        if (!have) break;
        it = ctl.items[n % kSlots];
      }
      const int* table = p.block_tables + (size_t)it.lane * p.max_blocks;
      const uint64_t pol = it.q > p.tile_rows ? keep : once;
      // thread l copies the tile's l-th block (both halves of its rows at
      // once); block ids one tile ahead
      auto load_blk = [&](int kt) -> int {
        const int key = (it.kt0 + kt) * kKeys + lane * p.bs;
        return lane < blocks && key < it.c ? table[key / p.bs] : -1;
      };
      int blk_next = load_blk(0);
      bool ok = true;
      if (vs) {
        // Q's buffer serves the item before until that item's last S is done
        ok = n < 1 || wait_done(q_last);
        if (!ok) break;
        q_last = n_ring + k_at(it.nkt - 1);
        issued_q = n + 1;
        if (lane == 0) {
          const bool half = it.q <= half_rows;
          mbar_expect_tx(bqf, (uint32_t)(g * (half ? half_rows : p.tile_rows)) * C::kRowB * C::kQParts);
#pragma unroll
          for (int h = 0; h < C::kQParts; ++h)  // halves; or the pieces, T rows apart
            tma_load_3d(sQ + h * C::kQPart + (half ? upper * C::kRowB : 0), half ? &tmQh : &tmQ,
                        FP8 ? 0 : h * 64, it.kvh * g, it.cu0 + it.node0 + (FP8 ? h * p.T : 0), bqf);
        }
      }
#pragma unroll 1
      for (int kt = 0; kt < it.nkt; ++kt) {
        const int nblk = min(blocks, (it.c - (it.kt0 + kt) * kKeys + p.bs - 1) / p.bs);
        const bool mine = lane < nblk;
        int blk = blk_next;
        if (kt + 1 < it.nkt) blk_next = load_blk(kt + 1);
        if (mine && (blk < 0 || blk >= p.NB)) {
          raise_flag(p.status, PA_FLAG_BLOCK_RANGE);
          blk = 0;
        }
        const uint32_t f = n_ring + (vs ? v_at(kt, it.nkt) : k_at(kt));
        const uint32_t st = f % C::kRing, use = f / C::kRing;
        ok = use < 1 || wait_done(f - C::kRing);
        if (!ok) break;
        if (kt == 0 && idx >= 0 && idx == p.skip_item) continue;  // (test hook)
        if (lane == 0) {
          ctl.uses[st] = use + 1;
          mbar_expect_tx(bfull + 8 * st, (uint32_t)(nblk * p.bs / 8) * C::kGroup);
        }
        __syncwarp();
        if (vs && kt >= it.tree0 && lane == 0) mbar_arrive(bgo + 8 * st);
        if (mine)
          tma_load_5d(sR + st * C::kTileBytes + lane * (p.bs / 8) * C::kGroup, tm, blk * (p.bs / 8),
                      it.kvh, bfull + 8 * st, pol);
      }
      if (!ok) break;
      n_ring += 2 * it.nkt;
    }
    if (!vs && blockIdx.x == 0) walk.finish(p, lane);
    if (!vs) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  } else if (warp == 6) {
    // ------------------------- look over the tree tiles ----------------------
    uint32_t go_par = 0;  // bit st: parity of the next use of go[st]
    for (;; ++n_item) {
      Item it;
      if (!read_item(n_item, it)) break;
      if (it.split + 1 != it.ns) {
        n_ring += 2 * it.nkt;
        continue;
      }
      const int past = it.c - it.q;
      const int* par = p.parents + it.cu0;
      if (it.kvh == 0 && it.node0 == 0) {  // each lane's parents once
        bool bad = false;
        for (int j = lane; j < it.q; j += 32) bad |= par[j] < -1 || par[j] >= j;
        if (__any_sync(0xffffffffu, bad) && lane == 0) raise_flag(p.status, PA_FLAG_TREE);
      }
      uint32_t* badw = ctl.bad[n_item % kBadSlots];
      if (lane < kNodes / 32) badw[lane] = 0;
      __syncwarp();
      bool ok = true;
      for (int kt = it.tree0; ok && kt < it.nkt; ++kt) {
        const uint32_t f = n_ring + v_at(kt, it.nkt), st = f % C::kRing;
        ok = wait_w(bgo + 8 * st, (go_par >> st) & 1, ab, p.status, lim) &&
             wait_w(bfull + 8 * st, (f / C::kRing) & 1, ab, p.status, lim);
        go_par ^= 1u << st;
        if (!ok) break;
        const int key0 = (it.kt0 + kt) * kKeys;
        const int r1 = min(kKeys, it.c - key0);  // rows of the lane
        const int r0 = max(0, past - key0);      // first node's row
        const uint32_t tile = sR + st * C::kTileBytes;
        constexpr int kCh = C::kRowB / 16;        // chunks of a half's row
        constexpr int kRowCh = kCh * C::kHalves;  // and of a row
        // a thread takes a 16-byte chunk; values that are not finite: all
        // exponent bits of a bf16 set, all bits but the sign of an e4m3 code
        auto odd_bits = [](uint32_t x) -> uint32_t {
          if (FP8) {
            const uint32_t m = (((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
            return m * 0xffu;
          }
          return ((x & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) |
                 ((x & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
        };
        auto at = [&](int r, int ch) -> uint32_t {
          return chunk_at<C::kRowB>(tile + (r >> 3) * C::kGroup + (ch / kCh) * C::kHalf, r & 7, ch % kCh);
        };
        // (bf16: rolled, 32 lanes of 64 nodes 348 us, with four chunks at a time
        // 343; e4m3 tiles are half as large, 32 lanes 80 us rolled, 82.5 so)
#pragma unroll(FP8 ? 1 : 4)
        for (int i = r0 * kRowCh + lane; i < kKeys * kRowCh; i += 32) {
          const int r = i / kRowCh, ch = i % kRowCh;
          const uint32_t a = at(r, ch);
          if (r >= r1) {
            st_shared_v4(a, 0, 0, 0, 0);
          } else {
            const uint4 v = lds128(a);
            if (odd_bits(v.x) | odd_bits(v.y) | odd_bits(v.z) | odd_bits(v.w)) {
              const int node = key0 + r - past;
              atomicOr(&badw[node >> 5], 1u << (node & 31));
            }
          }
        }
        __syncwarp();
        // (rare) zero those values; the epilogue adds them to the rows that attend them
        const uint32_t any = lane < kNodes / 32 ? reinterpret_cast<volatile uint32_t*>(badw)[lane] : 0;
        const int r_end = __any_sync(0xffffffffu, any != 0) ? r1 : r0;
        for (int r = r0; r < r_end; ++r) {
          const int node = key0 + r - past;
          if (!((reinterpret_cast<volatile uint32_t*>(badw)[node >> 5] >> (node & 31)) & 1u)) continue;
          if (lane < kRowCh) {
            const uint32_t a = at(r, lane);
            const uint4 v = lds128(a);
            st_shared_v4(a, v.x & ~odd_bits(v.x), v.y & ~odd_bits(v.y), v.z & ~odd_bits(v.z),
                         v.w & ~odd_bits(v.w));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bfixed + 8 * st);
      }
      if (!ok) break;
      n_ring += 2 * it.nkt;
    }
  } else if (warp == 4) {
    // -------------------------------- products ------------------------------
    const uint64_t dQ = half_desc<C::kRowB>(sQ, 16, 8 * C::kRowB);
    const uint64_t dK0 = half_desc<C::kRowB>(sR, 16, C::kGroup);
    const uint64_t dV0 = half_desc<C::kRowB>(sR, C::kHalf, C::kGroup);
    uint32_t fix_par = 0;        // bit st: parity of the next use of fixed[st]
    uint32_t v1 = 0, v2 = 0;     // places of the last V tile and of the one before
    for (;; ++n_item) {
      Item it;
      if (!read_item(n_item, it)) break;
      bool ok = wait_w(bqf, n_item & 1, ab, p.status, lim);
      // S of tile kt, once its K has landed and P V of tile kt - 2, which
      // read the P that this S overwrites, has finished
      auto issue_s = [&](int kt) {
        const uint32_t f = n_ring + k_at(kt), st = f % C::kRing, t = n_t + kt;
        // (the waits' latencies side by side)
        const bool landed = mbar_test(bfull + 8 * st, (f / C::kRing) & 1);
        if (t >= 2) ok = ok && wait_done(kt ? v1 : v2);
        if (!__all_sync(0xffffffffu, landed)) ok = ok && wait_w(bfull + 8 * st, (f / C::kRing) & 1, ab, p.status, lim);
        if (!ok) return;
        tc_fence_after();
        const uint64_t dk = dK0 + (uint64_t)((st * C::kTileBytes) >> 4);
        if constexpr (FP8) {
          constexpr uint32_t id = idesc_f8(0, kRows, kKeys, 0);
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
              umma_f8_w(tS(t), dQ + ((q * C::kQPart + kk * 32) >> 4), dk + ((kk * 32) >> 4), id,
                        q || kk ? 1u : 0u);
        } else {
          constexpr uint32_t id = umma_idesc_bf16(kRows, kKeys, 0, 0);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_bf16_w(tS(t), dQ + (((kk >> 2) * C::kQPart + (kk & 3) * 32) >> 4),
                        dk + (((kk >> 2) * C::kHalf + (kk & 3) * 32) >> 4), id, kk ? 1u : 0u);
        }
        umma_commit_w(bdone + 8 * st);
      };
      // (few copies of it in the code: the warps of the two CTAs, each in a
      // different part of the code, contend for the instruction cache)
#pragma unroll 1
      for (int kt = 0; kt < 2 && kt < it.nkt; ++kt) issue_s(kt);
#pragma unroll 1
      for (int kt = 0; ok && kt < it.nkt; ++kt) {
        const uint32_t f = n_ring + v_at(kt, it.nkt), st = f % C::kRing, t = n_t + kt;
        const bool tree = kt >= it.tree0;
        const uint32_t bar = (tree ? bfixed : bfull) + 8 * st, par = (tree ? fix_par >> st : f / C::kRing) & 1;
        if (tree) fix_par ^= 1u << st;
        const bool landed = mbar_test(bar, par);
        ok = wait_w(bP(t), (t >> 1) & 1, ab, p.status, lim);
        if (!__all_sync(0xffffffffu, landed)) ok = ok && wait_w(bar, par, ab, p.status, lim);
        v2 = v1;
        v1 = f;
        if (!ok) break;
        tc_fence_after();
        const uint64_t dv = dV0 + (uint64_t)((st * C::kTileBytes) >> 4);
        if constexpr (FP8) {
          constexpr uint32_t id = idesc_f8(1, kRows, D, 1);
#pragma unroll
          for (int q = 0; q < 3; ++q)
#pragma unroll
            for (int k = 0; k < kKeys / 32; ++k)
              umma_f8_tmem_a_w(tO, tS(t) + q * 16 + k * 8, dv + ((k * 4 * C::kGroup) >> 4), id,
                               kt || q || k ? 1u : 0u);
        } else {
          constexpr uint32_t id = umma_idesc_bf16(kRows, D, 0, 1);
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            umma_bf16_tmem_a_w(tO, tS(t) + k * 8, dv + ((k * 2 * C::kGroup) >> 4), id, kt || k ? 1u : 0u);
        }
        umma_commit_w(bdone + 8 * st);
        if (kt + 2 < it.nkt) issue_s(kt + 2);
      }
      if (!ok) break;
      n_ring += 2 * it.nkt;
      n_t += it.nkt;
    }
  } else {
    // -------------------------------- softmax rows --------------------------
    const int r = threadIdx.x;  // row == TMEM lane
    const int rj0 = r / g, rh0 = r % g;
    const int rj1 = r < upper ? 128 : (r - upper) / g, rh1 = r < upper ? 0 : (r - upper) % g;
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    for (;; ++n_item) {
      Item it;
      if (!read_item(n_item, it)) break;
      const bool half = it.q <= half_rows;
      const int rj = half ? rj1 : rj0, rh = half ? rh1 : rh0;
      const int node = it.node0 + rj;
      const bool valid = rj < p.tile_rows && node < it.q;
      const bool warp_valid = __any_sync(0xffffffffu, valid);
      const int past = it.c - it.q;
      const int* par = p.parents + it.cu0;
      const size_t row = (size_t)it.cu0 + (valid ? node : 0);
      const int head = it.kvh * g + rh;
      float c2 = p.scale_log2;
      if constexpr (FP8) {
        const int e = valid ? p.q_exp[row * p.H + head] : 127;
        // 2^(exponent - 7); neither 0 nor infinite, as the scale itself (a row of
        // zeros, whose exponent is the smallest, under a small scale)
        c2 = fminf(fmaxf(c2 * __uint_as_float((uint32_t)(e - 7) << 23), FLT_TRUE_MIN), FLT_MAX);
      }
      float m = -INFINITY, l = 0.f;
      bool ok = true;
#pragma unroll 1
      for (int kt = 0; kt < it.nkt; ++kt) {
        const uint32_t t = n_t + kt;
        const uint32_t tSr = tS(t) + lane_off;
        const bool tree = kt >= it.tree0;
        uint32_t w[2] = {0, 0};
        if (tree && valid) tree_mask<2>(par, node, past, (it.kt0 + kt) * kKeys, w);
        if (!wait_done(n_ring + k_at(kt))) { ok = false; break; }
        tc_fence_after();
        if (!warp_valid) {  // no row of this warp exists: P keeps what it holds
          tc_fence_before();
          mbar_arrive(bP(t));
          continue;
        }
        uint32_t sc[2][32];
        tmem_ld32(tSr, sc[0]);
        tmem_ld32(tSr + 32, sc[1]);
        tmem_wait_ld();
        if (tree) {
          // hidden keys' scores are replaced: whatever they held is gone
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 32; ++j) sc[h][j] = (w[h] >> j) & 1 ? sc[h][j] : 0xff800000u;
        }
        float m8[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) m8[j] = -INFINITY;
#pragma unroll
        for (int j = 0; j < 64; j += 2)
          m8[(j >> 1) & 7] = fmax3(m8[(j >> 1) & 7], __uint_as_float(sc[j >> 5][j & 31]),
                                   __uint_as_float(sc[j >> 5][(j & 31) + 1]));
#pragma unroll
        for (int h = 4; h >= 1; h >>= 1)
#pragma unroll
          for (int j = 0; j < h; ++j) m8[j] = fmaxf(m8[j], m8[j + h]);
        const float mx = m8[0] * c2;
        // a row may see no key of a tree tile: it keeps m = -inf, l = 0, O = 0
        const bool grow = valid && (m == -INFINITY || mx > m + C::kLazy);
        const float mn = grow ? fmaxf(m, mx) : m;
        const float alpha = grow && m != -INFINITY ? ex2_approx(m - mn) : 1.f;
        m = mn;
        const float neg = mn == -INFINITY ? 0.f : C::kBias - mn;
        const uint64_t c2x2 = f32x2(c2, c2), negx2 = f32x2(neg, neg);
        uint64_t r4[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) r4[j] = f32x2(0.f, 0.f);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float t0, t1;
            f32x2_split(fma_f32x2(f32x2(__uint_as_float(sc[h][2 * j]), __uint_as_float(sc[h][2 * j + 1])),
                                  c2x2, negx2),
                        t0, t1);
            const float e0 = ex2_approx(t0);
            const float e1 = ex2_approx(t1);
            pk[j] = FP8 ? pack_f16x2(e0, e1) : pack_bf16x2(e0, e1);
            r4[j & 3] = add_f32x2(r4[j & 3], f32x2(e0, e1));
          }
          if constexpr (FP8) {
            // 9 significant bits, then the upper byte three times over
            uint32_t p1[8], p2[8], p3[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint32_t x0 = (pk[2 * j] + 0x00020002u) & 0xfffcfffcu;
              const uint32_t x1 = (pk[2 * j + 1] + 0x00020002u) & 0xfffcfffcu;
              const uint32_t y0 = hsub2(x0, x0 & 0xff00ff00u), y1 = hsub2(x1, x1 & 0xff00ff00u);
              const uint32_t z0 = hsub2(y0, y0 & 0xff00ff00u), z1 = hsub2(y1, y1 & 0xff00ff00u);
              p1[j] = prmt(x0, x1, 0x7531);
              p2[j] = prmt(y0, y1, 0x7531);
              p3[j] = prmt(z0, z1, 0x7531);
            }
            tmem_st8(tSr + 8 * h, p1);
            tmem_st8(tSr + 16 + 8 * h, p2);
            tmem_st8(tSr + 32 + 8 * h, p3);
          } else {
            tmem_st16(tSr + 16 * h, pk);
          }
        }
        r4[0] = add_f32x2(r4[0], r4[2]);
        r4[1] = add_f32x2(r4[1], r4[3]);
        r4[0] = add_f32x2(r4[0], r4[1]);
        float rlo, rhi;
        f32x2_split(r4[0], rlo, rhi);
        l = fmaf(l, alpha, rlo + rhi);
        if (kt > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          if (!wait_done(n_ring + v_at(kt - 1, it.nkt))) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t ov[32];
            tmem_ld32(tO + lane_off + c * 32, ov);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * alpha);
            tmem_st32(tO + lane_off + c * 32, ov);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bP(t));
      }
      if (!ok) break;
      // the row's sums once its last P V has finished; the next item's first
      // P V waits for this group's first P of that item
      if (!wait_done(n_ring + v_at(it.nkt - 1, it.nkt))) break;
      tc_fence_after();
      if (warp_valid) {
        const bool single = it.ns == 1;
        const float inv = single ? p.v_scale / l : 1.f;  // one division per row
        const long long e =
            single ? 0 : (it.pair_base + (long long)node * it.ns + it.split) * p.H + head;
        bool any_bad = false;
        const uint32_t* badw = ctl.bad[n_item % kBadSlots];
        if (it.tree0 < it.nkt) {
#pragma unroll
          for (int k = 0; k < kNodes / 32; ++k) any_bad |= badw[k] != 0;
        }
        if (!single && valid) p.ml[e] = tree_ml(m, l);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ov[32];
          tmem_ld32(tO + lane_off + c * 32, ov);
          tmem_wait_ld();
          if (valid) tree_emit<D>(p, ov, c, single, inv, (row * p.H + head) * D, e);
        }
        if (any_bad && valid)
          tree_add_bad<D, FP8>(p, it.lane, it.kvh, past, node, par, badw, single, (row * p.H + head) * D, e, m);
      }
      tc_fence_before();
      n_ring += 2 * it.nkt;
      n_t += it.nkt;
    }
  }
  // every product issued has completed and every copy has landed before the
  // tensor memory is released and the CTA leaves
  if (warp == 4) {
    umma_commit_w(smem_u32(&ctl.fin));
    mbar_wait_bounded(smem_u32(&ctl.fin), 0, kWaitCycles);
  }
  if (warp == 7 && lane == 0 && issued_q) mbar_wait_bounded(bqf, (issued_q - 1) & 1, kWaitCycles);
  __syncthreads();
  if (warp == 7 && lane < C::kRing && ctl.uses[lane])
    mbar_wait_bounded(bfull + 8 * lane, (ctl.uses[lane] - 1) & 1, kWaitCycles);
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, bool FP8>
cudaError_t launch_tc(const TreeParams& p, const CUtensorMap& q, const CUtensorMap& qh,
                      const CUtensorMap& k, const CUtensorMap& v, int grid, cudaStream_t s) {
  auto kern = tree_tc_kernel<D, FP8>;
  // no more than two CTAs an SM: their TMEM fills it
  constexpr int smem = smem_bytes<D, FP8>() > 79872 ? smem_bytes<D, FP8>() : 79872;
  static unsigned long long done = 0;
  cudaError_t e = smem_opt_in(kern, smem, &done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = FP8 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p, q, qh, k, v);
}

// q's rows in e4m3 pieces (see above): pieces [2][T][H][D], exponents [T][H];
// and the item counter at 0. One warp per row; latency only (its reads are
// small beside K and V), and the kernel that follows starts while it runs.
template <int D>
__global__ void __launch_bounds__(256) tree_q_pieces_kernel(const TreeParams p) {
  constexpr int V = D / 32;  // elements of a thread
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.counter) *p.counter = 0;
  if (row >= (long long)p.T * p.H) return;
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) + row * D + lane * V;
  float x[V];
  if constexpr (V == 4) {
    const uint2 v = *reinterpret_cast<const uint2*>(src);
    x[0] = bf16_lo(v.x);
    x[1] = bf16_hi(v.x);
    x[2] = bf16_lo(v.y);
    x[3] = bf16_hi(v.y);
  } else {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(src);
    x[0] = bf16_lo(v);
    x[1] = bf16_hi(v);
  }
  float mx = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) mx = fmaxf(mx, fabsf(x[k]));
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  // times 2^(7 - exponent of the largest element); the score scale takes it
  // back (both factors are normal from 8 to 254: rows under 2^-119 take 8, rows
  // with an infinity 254)
  int e = (int)(__float_as_uint(mx) >> 23);
  e = min(max(e, 8), 254);
  const float up = __uint_as_float((uint32_t)(127 + 7 - (e - 127)) << 23);
  uint32_t hi = 0, lo = 0;
#pragma unroll
  for (int k = 0; k < V; k += 2) {
    // an infinity has no place in the pieces: NaN, which its row ends in anyway
    const float f0 = isfinite(x[k]) ? x[k] * up : NAN, f1 = isfinite(x[k + 1]) ? x[k + 1] * up : NAN;
    const uint32_t h = f32x2_to_e4m3x2(f0, f1), back = e4m3x2_to_f16x2(h);
    hi |= h << (8 * k);
    lo |= f32x2_to_e4m3x2(f0 - f16_lo(back), f1 - f16_hi(back)) << (8 * k);
  }
  uint8_t* dst = p.q_pieces + row * D + lane * V;
  const size_t apart = (size_t)p.T * p.H * D;
  if constexpr (V == 4) {
    *reinterpret_cast<uint32_t*>(dst) = hi;
    *reinterpret_cast<uint32_t*>(dst + apart) = lo;
  } else {
    *reinterpret_cast<uint16_t*>(dst) = (uint16_t)hi;
    *reinterpret_cast<uint16_t*>(dst + apart) = (uint16_t)lo;
  }
  if (lane == 0) p.q_exp[row] = (uint8_t)e;
}

}  // namespace

cudaError_t launch_tree_q_pieces(const TreeParams& p, cudaStream_t s) {
  const unsigned grid = (unsigned)(((long long)p.T * p.H + 7) / 8);
  if (p.D == 128)
    tree_q_pieces_kernel<128><<<grid, 256, 0, s>>>(p);
  else
    tree_q_pieces_kernel<64><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_tree_tc(const TreeParams& p, bool fp8, const CUtensorMap& q,
                           const CUtensorMap& qh, const CUtensorMap& k, const CUtensorMap& v,
                           int grid, cudaStream_t s) {
  if (p.D == 128)
    return fp8 ? launch_tc<128, true>(p, q, qh, k, v, grid, s)
               : launch_tc<128, false>(p, q, qh, k, v, grid, s);
  return fp8 ? launch_tc<64, true>(p, q, qh, k, v, grid, s)
             : launch_tc<64, false>(p, q, qh, k, v, grid, s);
}

}  // namespace pa
