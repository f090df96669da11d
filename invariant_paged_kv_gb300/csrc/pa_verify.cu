// Verification of trees of drafted tokens against the target's probabilities,
// from given random numbers.
//
// A lane's nodes are its flat rows; node 0 is the lane's last token, row i of
// target_probs is the target's distribution p_i after node i, row i of
// draft_probs the distribution q_i its children were drawn from. The walk
// starts at node 0; at node i the children c = c_1, c_2, .. (by index) are
// tried in turn against the residual r, at first p_i with mass Z = 1:
//   accept c      if u_c Z q_i(x_c) < r(x_c); the walk goes on at c
//   else          r = max(r - Z q_i, 0), Z = sum r; that is r = max(p_i - A q_i, 0)
//                 with A the sum of the Z so far
// and where no child is accepted the token that follows is drawn from r / Z:
// the first x whose running sum of r passes u_sample sum(r). Every step keeps
// the target's distribution: the output token of a node is distributed as p_i.
// Without draft_probs a child is taken as certain (q = 1 at its own token):
// accept if u Z < r(x), else r(x) = 0, Z = Z - r(x).
//
// Whole numbers come out, so the sums must tell apart neighbours in a
// vocabulary of 10^5 entries, whose running sum a float resolves to 6e-8
// only, and must not depend on the batch. FP64 would do but runs at 2
// operations per clock and SM here. A thread adds its entries in three floats
// (Sums below): the rounding error of every addition is known exactly and
// added to the next float, which leaves less than V 2^-58 of a row behind.
// Threads' sums then become 64-bit integers in units of 2^-62, exact and
// associative, and so do the entries of the one run of the vocabulary that
// the draw ends in. Which thread adds what depends on the vocabulary alone.
//
// A lane is a cluster of up to 8 CTAs. All of them walk the tree alike, from
// the two numbers of each node gathered up front; only a rejection that has a
// further child to try and the final draw read rows, each CTA a slice of the
// vocabulary, with the slices' sums exchanged through distributed shared
// memory. A row is read once per pass (the draw's second look at one 128-entry
// run comes out of L2), and a lane's passes follow one another: the lanes with
// the most rejections bound a batch. 64 trees of 16 nodes, vocabulary 248320:
// 81 us, 142 MB over all passes (1.8 TB/s, about 5 us a pass); 24 trees of 25
// chosen drafts, vocabulary 100003, one pass each: 13.7 us; one chain,
// vocabulary 32000: 7.7 us. 16 CTAs a lane or 512 threads were no faster.
#include <cooperative_groups.h>

#include "pa_tcgen05.cuh"
#include "pa_verify.cuh"

namespace pa {

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kRuns = 64;  // parts of a warp's slice that the draw looks through
constexpr int kNodes = PA_TREE_MAX_NODES;
constexpr unsigned long long kNothing = 1ull << 22;  // 2^-40 of a row

typedef unsigned long long u64;

// x in [0, 2) (-0 included) to units of 2^-62, truncated.
__device__ __forceinline__ u64 to_fix(float x) {
  const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
  const int sh = (int)(b >> 23) - 88;
  const u64 m = (b & 0x7fffffu) | 0x800000u;
  return sh >= 0 ? m << sh : sh > -24 ? m >> -sh : 0ull;
}
__device__ __forceinline__ double fix_to_double(u64 v) { return (double)v * 0x1p-62; }

__device__ __forceinline__ bool prob_ok(float x) { return x >= 0.f && x < 2.f; }

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_sum_f(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ u64 warp_incl(u64 v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

template <int N>
struct Count {
  static constexpr int value = N;
};

struct Shared {
  int par[kNodes], tok[kNodes];
  float u[kNodes], pc[kNodes], qc[kNodes];
  int path[kNodes];
  // the residual of the current node: max(p - A q, 0) (with draft_probs), A
  // also as two floats and in units of 2^-54, or the tokens taken out (without)
  double a;
  float ah, al;
  u64 afix;
  int gone[kNodes];
  int n_rej;
  int cur, count, last, action;
  double mass;
  int bad;
  u64 runs[kRuns];
  u64 wsum[kWarps];  // sums of the CTA's warps
  float fsum[kWarps], qsum[kWarps];  // of the target's entries, of the draft's
  int wbad;          // whether it met a value that is no probability
  // by pass parity: what every CTA of the cluster left here
  u64 csum[2][kMaxCluster];
  float cfsum[2][kMaxCluster], cqsum[2][kMaxCluster];
  int cbad[2][kMaxCluster];
};

// Residual of entry v of the row, in fixed point.
__device__ __forceinline__ u64 residual(const Shared& sm, bool with_q, int n_rej, float pv, float qv,
                                        int v) {
  u64 r = to_fix(pv);
  if (with_q) {
    if (n_rej) {
      const u64 q = to_fix(qv);
      const u64 hi = __umul64hi(sm.afix, q);
      const u64 aq = hi >> 54 ? ~0ull : (hi << 10) | ((sm.afix * q) >> 54);  // 4 and more: past any p
      r = r > aq ? r - aq : 0;
    }
  } else {
    for (int k = 0; k < n_rej; ++k)
      if (sm.gone[k] == v) r = 0;
  }
  return r;
}

// A signed float of magnitude under 2 in units of 2^-62.
__device__ __forceinline__ long long to_fix_signed(float x) {
  const long long m = (long long)to_fix(fabsf(x));
  return x < 0.f ? -m : m;
}

// Sums of non-negative values of total under 2, two at a time. s1 holds 4 + the
// sum, so its last place is 2^-21 and every value and partial sum is smaller than
// it: t = s1 + h rounds, and h - (t - s1) is what it lost, exactly. That goes to
// s2, and what s2 loses to s3. Those two hold a bias of their own and stay in its
// binade over the few values between two calls of take(), so what they gathered
// is the difference of their bits, in whole last places (2^-40 and 2^-58). The
// only error is s3's, 2^-59 for each value added: V 2^-58 of a row at the worst,
// 2^-40 for 248320 entries. (With no integer behind them, s3 without a bias, it
// was 2^-46 there and 2^-32 for 2^24 entries, on ordinary rows.)
struct Sums {
  static constexpr float kBias2 = 0x1.8p-17f, kBias3 = 0x1.8p-35f;
  uint64_t s1, s2, s3;
  long long low;  // taken out of s2 and s3, in units of 2^-58
  __device__ __forceinline__ void start() {
    s1 = f32x2(4.f, 4.f);
    s2 = f32x2(kBias2, kBias2);
    s3 = f32x2(kBias3, kBias3);
    low = 0;
  }
  __device__ __forceinline__ void add(uint64_t h) {
    const uint64_t neg = f32x2(-1.f, -1.f);
    const uint64_t t = add_f32x2(s1, h);
    add_low(fma_f32x2(fma_f32x2(s1, neg, t), neg, h));
    s1 = t;
  }
  // (values up to 2^-22)
  __device__ __forceinline__ void add_low(uint64_t e) {
    const uint64_t neg = f32x2(-1.f, -1.f);
    const uint64_t t = add_f32x2(s2, e);
    s3 = add_f32x2(s3, fma_f32x2(fma_f32x2(s2, neg, t), neg, e));
    s2 = t;
  }
  // after every 8 calls of add and 8 of add_low: s2 is within 2^-18 of its bias
  // (8 2^-22, the low parts 2^-23 in all), s3 within 2^-36 (16 2^-41)
  __device__ __forceinline__ void take() {
    low += (long long)places(s2, kBias2) * (1 << 18) + places(s3, kBias3);
    s2 = f32x2(kBias2, kBias2);
    s3 = f32x2(kBias3, kBias3);
  }
  __device__ __forceinline__ static int places(uint64_t s, float bias) {
    float a, b;
    f32x2_split(s, a, b);
    return (int)(__float_as_uint(a) + __float_as_uint(b) - 2 * __float_as_uint(bias));
  }
  __device__ __forceinline__ long long total() const {
    float a, b;
    f32x2_split(s1, a, b);
    return low * 16 + (to_fix_signed(a - 4.f) + to_fix_signed(b - 4.f));
  }
};

// max(h - A q, 0) as h + l, A = ah + al. Where it is positive, h >= A q makes
// the loss of the difference exact; A, its product and the loss less the
// product's low part each round by 2^-49 of h: 2^-47 of it in all.
__device__ __forceinline__ void less_pair(float& h, float& l, float ah, float al, float q) {
  const float ph = ah * q;
  const float pl = fmaf(al, q, fmaf(ah, q, -ph));
  const float d = h - ph;
  const float rest = ((h - d) - ph) - pl;
  const float v = d + rest;
  h = v > 0.f ? v : 0.f;
  l = v > 0.f ? rest - (v - d) : 0.f;
}

enum { kSum = 1, kDraw = 2, kBadLane = 3 };

__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyParams p) {
  __shared__ Shared sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int b = blockIdx.x / ranks;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cu0 = p.cu[b], cu1 = p.cu[b + 1], n = cu1 - cu0;
  const bool cu_bad = cu0 < 0 || cu1 < cu0 || cu1 > p.T || (b == 0 && cu0 != 0) ||
                      (b == p.B - 1 && cu1 != p.T);
  if (cu_bad || n > p.max_q_len || n == 0) {  // no row of this lane is known
    if (rank == 0 && tid == 0) {
      if (cu_bad || n > 0) raise_flag(p.status, cu_bad ? PA_FLAG_CU_SEQLENS : PA_FLAG_HOST_BOUND);
      p.n_accepted[b] = -1;
    }
    return;  // the same in every CTA of the cluster
  }
  // no CTA writes to another's shared memory before all of the cluster have
  // started: waited for before the first sums are handed round (behind the
  // gather one chain took 8.05 us, here 7.7)
  cluster.barrier_arrive();
  const bool with_q = p.q != nullptr;
  // ---- the nodes: parents, tokens, numbers, and p, q of each at its parent's row
  if (tid == 0) sm.bad = sm.wbad = 0;
  __syncthreads();
  for (int j = tid; j < n; j += kThreads) {
    const int par = p.parents[cu0 + j], tok = p.tokens[cu0 + j];
    sm.par[j] = par;
    sm.tok[j] = tok;
    int bad = 0;
    if (j == 0) {
      if (par != -1) bad = PA_FLAG_TREE;
    } else if (par < 0 || par >= j || tok < 0 || tok >= p.V) {
      bad = PA_FLAG_TREE;
    } else {
      const size_t at = (size_t)(cu0 + par) * p.V + tok;
      sm.u[j] = p.u_accept[cu0 + j];
      sm.pc[j] = p.p[at];
      sm.qc[j] = with_q ? p.q[at] : 1.f;
    }
    if (bad) atomicOr(&sm.bad, bad);
  }
  const float us = p.u_sample[b];
  if (tid == 0) {
    if (!(us >= 0.f && us < 1.f)) atomicOr(&sm.bad, PA_FLAG_PROB);
    sm.cur = sm.count = sm.last = sm.n_rej = 0;
    sm.path[0] = 0;
    sm.mass = 1.0;
    sm.a = 0.0;
  }
  __syncthreads();

  int owner = 0;
  for (int pass = 0;; ++pass) {
    if (warp == 0) {
      // walk on from child index last + 1 of node cur until a row is needed
      int cur = sm.cur, count = sm.count, last = sm.last, n_rej = sm.n_rej, bad = sm.bad;
      double mass = sm.mass, a = sm.a;
      int action = bad ? kBadLane : 0;
      // child of cur after index j, or n
      auto next_child = [&](int j) -> int {
        for (int j0 = j + 1; j0 < n; j0 += 32) {
          const unsigned m = __ballot_sync(0xffffffffu, j0 + lane < n && sm.par[j0 + lane] == cur);
          if (m) return j0 + __ffs(m) - 1;
        }
        return n;
      };
      int c = action ? n : next_child(last);
      while (!action) {
        if (c >= n) {
          action = kDraw;
          break;
        }
        last = c;
        const float pc = sm.pc[c], qc = sm.qc[c], uc = sm.u[c];
        if (!prob_ok(pc) || !prob_ok(qc) || !(uc >= 0.f && uc < 1.f)) {
          bad |= PA_FLAG_PROB;
          action = kBadLane;
          break;
        }
        // r(x_c) after the rejections so far
        double rx = with_q ? fmax((double)pc - a * (double)qc, 0.0) : (double)pc;
        if (!with_q)
          for (int k = 0; k < n_rej; ++k)
            if (sm.gone[k] == sm.tok[c]) rx = 0.0;
        if ((double)uc * mass * (double)qc < rx) {
          cur = c;
          ++count;
          if (lane == 0) sm.path[count] = c;
          n_rej = 0;
          mass = 1.0;
          a = 0.0;
          c = next_child(c);
          continue;
        }
        if (with_q) {
          // r - Z q = max(p - A q, 0) - Z q: the same with A + Z (where p - A q
          // was negative it stays so). Z is 1 for the first rejection, else
          // what the last sum found
          a += mass;
          ++n_rej;
          c = next_child(c);
          if (c < n) {
            action = kSum;
            break;
          }
        } else {
          if (lane == 0) sm.gone[n_rej] = sm.tok[c];
          __syncwarp();
          ++n_rej;
          mass = mass - rx;
          c = next_child(c);
        }
      }
      if (lane == 0) {
        sm.cur = cur;
        sm.count = count;
        sm.last = last;
        sm.n_rej = n_rej;
        sm.mass = mass;
        sm.a = a;
        sm.ah = (float)a;
        sm.al = (float)(a - (double)(float)a);
        sm.afix = (u64)(a * 0x1p54);
        sm.bad = bad;
        sm.action = action;
      }
    }
    __syncthreads();
    if (sm.action == kBadLane) {  // alike in every CTA: from the same numbers
      if (pass == 0) cluster.barrier_wait();
      break;
    }

    // ---- sum of the residual row, by slices of runs of 128 entries
    const int n_rej = sm.n_rej, par = pass & 1;
    const size_t row_at = (size_t)(cu0 + sm.cur) * p.V;
    const bool use_q = with_q && n_rej > 0;
    // entries in groups of 4 at 16-byte boundaries: `skew` entries before
    // entry 0 share its group
    const int skew = (int)(row_at & 3);
    const float* pr = p.p + row_at - skew;
    const float* qr = use_q ? p.q + row_at - skew : nullptr;
    const int groups = (p.V + skew + 3) / 4;
    const int warps = ranks * kWarps, gw = rank * kWarps + warp;
    const int iters = (groups + 32 * warps - 1) / (32 * warps);  // of 32 groups, per warp
    const int per_run = (iters + kRuns - 1) / kRuns;
    // the four entries of group grp; 0 outside the row. The first and last
    // group may reach into a neighbouring row (or past the tensor).
    auto load = [&](int grp, float4& pv, float4& qv) {
      pv = qv = make_float4(0, 0, 0, 0);
      if (grp >= groups) return;
      const int v0 = grp * 4 - skew;
      if (v0 >= 0 && v0 + 4 <= p.V) {
        pv = __ldg(reinterpret_cast<const float4*>(pr) + grp);
        if (use_q) qv = __ldg(reinterpret_cast<const float4*>(qr) + grp);
      } else {
        float x[4] = {0, 0, 0, 0}, y[4] = {0, 0, 0, 0};
        for (int k = 0; k < 4; ++k)
          if (v0 + k >= 0 && v0 + k < p.V) {
            x[k] = pr[grp * 4 + k];
            if (use_q) y[k] = qr[grp * 4 + k];
          }
        pv = make_float4(x[0], x[1], x[2], x[3]);
        qv = make_float4(y[0], y[1], y[2], y[3]);
      }
    };
    // residuals of a group in fixed point
    auto fix = [&](int grp, const float4& pv, const float4& qv, u64 (&r)[4]) {
      const float x[4] = {pv.x, pv.y, pv.z, pv.w}, y[4] = {qv.x, qv.y, qv.z, qv.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) r[k] = residual(sm, with_q, n_rej, x[k], y[k], grp * 4 - skew + k);
    };
    Sums sums;
    sums.start();
    uint32_t top = 0;          // largest bit pattern met: a negative value or NaN is large
    uint64_t psum = f32x2(0.f, 0.f), qsum = psum;
    const int g0 = gw * iters * 32 + lane;
    const float ah = sm.ah, al = sm.al;
    // kRej: rejections, 2 standing for more
    auto slice = [&](auto rej) {
      constexpr int kRej = decltype(rej)::value;
      constexpr int kAhead = 4;  // iterations whose loads are in flight
      for (int i0 = 0; i0 < iters; i0 += kAhead) {
        float4 pv[kAhead], qv[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) load(i0 + k < iters ? g0 + 32 * (i0 + k) : groups, pv[k], qv[k]);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          float h[4] = {pv[k].x, pv[k].y, pv[k].z, pv[k].w}, l[4] = {0, 0, 0, 0};
          const float q[4] = {qv[k].x, qv[k].y, qv[k].z, qv[k].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) top = max(top, max(__float_as_uint(h[j]), __float_as_uint(q[j])));
          psum = add_f32x2(psum, add_f32x2(f32x2(h[0], h[1]), f32x2(h[2], h[3])));
          if constexpr (kRej >= 1) qsum = add_f32x2(qsum, add_f32x2(f32x2(q[0], q[1]), f32x2(q[2], q[3])));
          if constexpr (kRej == 1) {  // A = 1
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float d = h[j] - q[j];
              l[j] = d > 0.f ? (h[j] - d) - q[j] : 0.f;
              h[j] = d > 0.f ? d : 0.f;
            }
          } else if constexpr (kRej == 2) {
#pragma unroll
            for (int j = 0; j < 4; ++j) less_pair(h[j], l[j], ah, al, q[j]);
          }
          sums.add(f32x2(h[0], h[1]));
          sums.add(f32x2(h[2], h[3]));
          if constexpr (kRej >= 1) {
            sums.add_low(f32x2(l[0], l[1]));
            sums.add_low(f32x2(l[2], l[3]));
          }
        }
        sums.take();
      }
    };
    if (!use_q)
      slice(Count<0>());
    else if (n_rej == 1)
      slice(Count<1>());
    else
      slice(Count<2>());
    long long mine_fix = sums.total();
    bool took = false;
    if (!with_q) {
      // tokens taken out of the row: each once, by the thread that added it
      for (int k = 0; k < n_rej; ++k) {
        const int x = sm.gone[k], grp = (x + skew) >> 2;
        bool again = false;
        for (int j = 0; j < k; ++j) again |= sm.gone[j] == x;
        if (!again && grp / 32 / iters == gw && (grp & 31) == lane) {
          mine_fix -= (long long)to_fix(p.p[row_at + x]);
          took = true;
        }
      }
    }
    float fs, fs1, qs, qs1;
    f32x2_split(psum, fs, fs1);
    f32x2_split(qsum, qs, qs1);
    fs += fs1;
    // (rare) next to nothing is left, and it may be no more than what the sums
    // rounded: 2^-58 beside each token taken out, 2^-47 of p where p is A q. The
    // draw must not land on what is not there, so such a thread sums its entries
    // anew, as the draw reads them. (After one rejection with draft rows every
    // difference is exact, and what is left of it is there.)
    if (mine_fix > 0 && (with_q ? n_rej >= 2 && (float)mine_fix < fs * 0x1p17f : took && mine_fix < (1 << 17))) {
      mine_fix = 0;
      for (int i = 0; i < iters; ++i) {
        float4 pv, qv;
        load(g0 + 32 * i, pv, qv);
        u64 r[4];
        fix(g0 + 32 * i, pv, qv, r);
        mine_fix += (long long)((r[0] + r[1]) + (r[2] + r[3]));
      }
    }
    const u64 total_w = warp_sum((u64)(mine_fix > 0 ? mine_fix : 0));
    bool bad = top >= 0x40000000u;  // 2.0f
    if (bad) {  // (rare) look again: it may have been -0
      bad = false;
      for (int i = 0; i < iters; ++i) {
        float4 pv, qv;
        load(g0 + 32 * i, pv, qv);
        bad |= !(prob_ok(pv.x) && prob_ok(pv.y) && prob_ok(pv.z) && prob_ok(pv.w) && prob_ok(qv.x) &&
                 prob_ok(qv.y) && prob_ok(qv.z) && prob_ok(qv.w));
      }
    }
    fs = warp_sum_f(fs);
    qs = warp_sum_f(qs + qs1);
    if (lane == 0) {
      sm.wsum[warp] = total_w;
      sm.fsum[warp] = fs;
      sm.qsum[warp] = qs;
    }
    if (__syncthreads_or(bad)) sm.wbad = 1;  // the same value from every thread
    if (pass == 0) cluster.barrier_wait();
    if (warp == 0) {
      // its sums to every CTA of the cluster (the barrier makes them seen)
      const u64 all = warp_sum(lane < kWarps ? sm.wsum[lane] : 0);
      const float f = warp_sum_f(lane < kWarps ? sm.fsum[lane] : 0.f);
      const float q = warp_sum_f(lane < kWarps ? sm.qsum[lane] : 0.f);
      __syncwarp();
      if (lane < ranks) {
        Shared* o = cluster.map_shared_rank(&sm, lane);
        o->csum[par][rank] = all;
        o->cfsum[par][rank] = f;
        o->cqsum[par][rank] = q;
        o->cbad[par][rank] = sm.wbad;
      }
    }
    cluster.sync();
    const u64 mine = lane < ranks ? sm.csum[par][lane] : 0;
    const float fall = warp_sum_f(lane < ranks ? sm.cfsum[par][lane] : 0.f);
    const float qall = warp_sum_f(lane < ranks ? sm.cqsum[par][lane] : 0.f);
    int badall = lane < ranks ? sm.cbad[par][lane] : 0;
    const u64 incl = warp_incl(mine, lane);
    const u64 total = __shfl_sync(0xffffffffu, incl, 31);
    // rows that hold a value outside [0, 2), sum to 2 or more (and would not fit
    // the fixed point; the floats' sum, within 2^-13, is held against 1.99) or to
    // next to nothing are no probabilities
    auto no_row = [](float sum) -> bool { return !(sum < 1.99f && sum >= 0x1p-40f); };
    badall = __any_sync(0xffffffffu, badall) || no_row(fall) || (use_q && no_row(qall));
    const bool empty = total < kNothing;
    if (badall || (empty && n_rej == 0)) {
      __syncthreads();
      if (tid == 0) {
        sm.bad |= PA_FLAG_PROB;
        sm.action = kBadLane;
      }
      __syncthreads();
      break;
    }
    if (sm.action == kSum) {
      __syncthreads();
      if (tid == 0) {
        sm.mass = fix_to_double(total);
      }
      __syncthreads();
      continue;
    }
    if (empty) {
      // nothing is left of the residual (p <= q everywhere, up to the rows'
      // own rounding): the draw is from p itself
      __syncthreads();
      if (tid == 0) {
        sm.n_rej = 0;
        sm.a = 0.0;
        sm.last = n;  // no further child
      }
      __syncthreads();
      continue;
    }
    // ---- the draw: first entry whose running sum exceeds u_sample * total
    const uint32_t ub = __float_as_uint(us);
    const int sh = (int)(ub >> 23) - 86;
    const u64 um = (ub & 0x7fffffu) | 0x800000u;
    const u64 u64f = sh >= 0 ? um << sh : sh > -24 ? um >> -sh : 0ull;  // us 2^64
    const u64 t = __umul64hi(total, u64f);
    const unsigned hit = __ballot_sync(0xffffffffu, incl > t);
    const int src = __ffs(hit) - 1;  // t < total, so there is one
    u64 base = __shfl_sync(0xffffffffu, incl - mine, src);
    owner = src;
    if (rank == owner) {
      // the warp whose slice it falls in; the CTA looks through that slice:
      // sums of its runs, then the entries of one run
      const u64 ws = lane < kWarps ? sm.wsum[lane] : 0;
      const u64 win = warp_incl(ws, lane);
      const unsigned which = __ballot_sync(0xffffffffu, base + win > t);
      const int wl = __ffs(which) - 1;  // one of the CTA's: its own sum is beyond t
      base += __shfl_sync(0xffffffffu, win - ws, wl);
      const int w0 = (rank * kWarps + wl) * iters;
      constexpr int kAt = 2;  // runs of a warp at a time: their loads go out together
      for (int run0 = warp; run0 * per_run < iters; run0 += kAt * kWarps) {
        u64 acc[kAt] = {};
        for (int i = 0; i < per_run; ++i) {
          float4 pv[kAt], qv[kAt];
          auto group_of = [&](int k) {
            const int at = (run0 + k * kWarps) * per_run + i;
            return at < iters ? (w0 + at) * 32 + lane : groups;
          };
#pragma unroll
          for (int k = 0; k < kAt; ++k) load(group_of(k), pv[k], qv[k]);
#pragma unroll
          for (int k = 0; k < kAt; ++k) {
            u64 r[4];
            fix(group_of(k), pv[k], qv[k], r);
            acc[k] += (r[0] + r[1]) + (r[2] + r[3]);
          }
        }
#pragma unroll
        for (int k = 0; k < kAt; ++k) {
          const u64 sum = warp_sum(acc[k]);
          if (lane == 0 && run0 + k * kWarps < kRuns) sm.runs[run0 + k * kWarps] = sum;
        }
      }
      __syncthreads();
      if (warp == 0) {
        const u64 ra = 2 * lane * per_run < iters ? sm.runs[2 * lane] : 0;
        const u64 rb = (2 * lane + 1) * per_run < iters ? sm.runs[2 * lane + 1] : 0;
        const u64 in = warp_incl(ra + rb, lane);
        unsigned hits = __ballot_sync(0xffffffffu, base + in > t);
        // the slice's own sum, of entries cut to 2^-62, may end short of the
        // threads': then the last run that holds anything
        const unsigned held = __ballot_sync(0xffffffffu, ra + rb > 0);
        if (!hits) hits = held ? 0x80000000u >> __clz(held) : 1u;
        const int s2 = __ffs(hits) - 1;
        u64 at = base + __shfl_sync(0xffffffffu, in - ra - rb, s2);
        const u64 fr = __shfl_sync(0xffffffffu, ra, s2), sr = __shfl_sync(0xffffffffu, rb, s2);
        int run = 2 * s2;
        if (at + fr <= t && sr > 0) {
          ++run;
          at += fr;
        }
        // first entry past t, else the run's last that is not 0
        int found = -1, last = -1;
        for (int i = run * per_run; found < 0 && i < min(iters, (run + 1) * per_run); ++i) {
          u64 r[4];
          const int grp = (w0 + i) * 32 + lane;
          float4 pv, qv;
          load(grp, pv, qv);
          fix(grp, pv, qv, r);
          const u64 s4 = (r[0] + r[1]) + (r[2] + r[3]);
          const u64 in4 = warp_incl(s4, lane);
          u64 x = at + in4 - s4;
          int mine_at = -1, mine_last = -1;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x += r[k];
            if (r[k] && x > t && mine_at < 0) mine_at = grp * 4 - skew + k;
            if (r[k]) mine_last = grp * 4 - skew + k;
          }
          const unsigned m4 = __ballot_sync(0xffffffffu, mine_at >= 0);
          const unsigned l4 = __ballot_sync(0xffffffffu, mine_last >= 0);
          if (l4) last = __shfl_sync(0xffffffffu, mine_last, 31 - __clz(l4));
          if (m4) found = __shfl_sync(0xffffffffu, mine_at, __ffs(m4) - 1);
          at += __shfl_sync(0xffffffffu, in4, 31);
        }
        if (lane == 0) p.out_tokens[cu0 + sm.count] = found >= 0 ? found : max(last, 0);
      }
    }
    break;
  }
  __syncthreads();
  const bool bad_lane = sm.action == kBadLane;
  if (rank == 0) {
    const int count = bad_lane ? -1 : sm.count;
    if (tid == 0) {
      p.n_accepted[b] = count;
      if (bad_lane) raise_flag(p.status, sm.bad);
    }
    for (int i = tid; i < n; i += kThreads) {
      p.path[cu0 + i] = i <= count ? sm.path[i] : -1;
      if (i != count) p.out_tokens[cu0 + i] = i < count ? sm.tok[sm.path[i + 1]] : -1;
    }
  }
  // (no CTA writes to another's shared memory after the last barrier, so each may leave)
}

}  // namespace

cudaError_t launch_verify(const VerifyParams& p, cudaStream_t s) {
  // 2048 entries per CTA or more: below, the exchange costs more than the
  // slice saves
  int ranks = 1;
  while (ranks < kMaxCluster && (long long)ranks * 2048 < p.V) ranks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.B * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ranks;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_kernel, p);
}

}  // namespace pa
