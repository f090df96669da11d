// Tree attention: the fold of split partials, and the fp32 kernel.
#include "pa_tree.cuh"

namespace pa {

int num_sms();

namespace {

// ---------------------------------------------------------------------------
// The fold: out = (sum_i acc_i 2^(m_i - M)) / (sum_i l_i 2^(m_i - M)), splits
// left to right. A warp takes one (node, head) row at a time, a thread D / 32
// of its sums, four splits' loads in flight. Bound by reading the partials
// (mostly still in L2) where there are many rows, by its chain of dependent
// loads where there are few: a warp takes several rows, one after another,
// only once there are CTAs enough to fill the SMs. 23 MB of partials of 24
// ragged lanes, cold: 15.5 us; with the next row's loads ahead of the current
// row's sums it was slower (fewer warps fit).
// ---------------------------------------------------------------------------
constexpr int kFoldWarps = 4;

template <int D, bool F32>
__global__ void __launch_bounds__(kFoldWarps * 32) tree_fold_kernel(const TreeParams p, int rows_per_warp) {
  constexpr int V = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_cta = kFoldWarps * rows_per_warp;
  const int per_lane = (p.max_q_len * p.H + per_cta - 1) / per_cta;
  const int b = blockIdx.x / per_lane;
  const int r0 = (blockIdx.x - b * per_lane) * per_cta + warp;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 info = p.lane_info[b];
  const int cu0 = p.cu_seqlens[b];
  const long long base = ((long long)info.y << 32) | (uint32_t)info.x;
  const int ns = info.w, rows = info.z * p.H;
  // (an entry outside the call's bounds is none, and nothing is touched for it)
  if (ns < 2 || ns > PA_TREE_MAX_SPLITS || info.z < 0 || info.z > p.max_q_len || cu0 < 0 ||
      (long long)cu0 + info.z > p.T || base < 0 || base > p.capacity - (long long)info.z * ns)
    return;
#pragma unroll 1
  for (int k = 0; k < rows_per_warp; ++k) {
    const int rh = r0 + k * kFoldWarps;
    if (rh >= rows) return;
    const int node = rh / p.H, head = rh - node * p.H;
    const long long e0 = (base + (long long)node * ns) * p.H + head;
    const float2* ml = p.ml + e0;
    const float* acc = p.acc + e0 * D + lane * V;
    Fold f;
    float a[V];
    constexpr int kAhead = 4;
    float2 mlv[kAhead];
    float av[kAhead][V];
    auto load = [&](int i, int slot) {
      mlv[slot] = ml[(long long)i * p.H];
      const float* src = acc + (long long)i * p.H * D;
      if constexpr (V == 4) {
        const float4 x = *reinterpret_cast<const float4*>(src);
        av[slot][0] = x.x;
        av[slot][1] = x.y;
        av[slot][2] = x.z;
        av[slot][3] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(src);
        av[slot][0] = x.x;
        av[slot][1] = x.y;
      }
    };
    for (int i0 = 0; i0 < ns; i0 += kAhead) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (i0 + j < ns) load(i0 + j, j);
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (i0 + j >= ns) break;
        if (i0 + j == 0) {
          f.first(mlv[0].x, mlv[0].y);
#pragma unroll
          for (int d = 0; d < V; ++d) a[d] = av[0][d];
        } else {
          float ea, eb;
          f.next(mlv[j].x, mlv[j].y, ea, eb);
#pragma unroll
          for (int d = 0; d < V; ++d) a[d] = fmaf(a[d], ea, av[j][d] * eb);
        }
      }
    }
    const float inv = p.v_scale / f.L;
    const size_t o = ((size_t)(cu0 + node) * p.H + head) * D + lane * V;
#pragma unroll
    for (int d = 0; d < V; ++d) a[d] *= inv;
    if constexpr (F32) {
      float* out = static_cast<float*>(p.out) + o;
      if constexpr (V == 4)
        *reinterpret_cast<float4*>(out) = make_float4(a[0], a[1], a[2], a[3]);
      else
        *reinterpret_cast<float2*>(out) = make_float2(a[0], a[1]);
    } else {
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + o;
      if constexpr (V == 4)
        *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]));
      else
        *reinterpret_cast<uint32_t*>(out) = pack_bf16x2(a[0], a[1]);
    }
  }
}

// ---------------------------------------------------------------------------
// fp32 caches: plain FMA on the CUDA cores (TF32 would lose 13 bits). One CTA
// per (lane, split, kv head, row tile of MR (node, head) pairs), 64 keys at a
// time: scores from Q and K in shared memory, 16 x 16 threads of MR / 16 rows
// x 4 keys each; p through shared memory; sums of MR / 16 rows x D / 16 dims
// in registers. Bound by FMA issue where a lane has many pairs (MR = 64 reuses
// each key 64 times), so steps of few pairs take MR = 32 or 16, which do less
// padded work (the rows' bits are the same); and by latency where it has few
// keys, so splits start at 128 keys and the next tile is on its way (K and V
// twice, block ids two tiles ahead) while one is worked on. 8 lanes of 2-13
// nodes over 1000 keys, 4 heads of 64: 21.5 us, issue slots 43% used.
// ---------------------------------------------------------------------------
constexpr int kF32Keys = 64;

template <int D, int MR>
struct F32Smem {
  static constexpr int kPitch = D + 4;  // rows 16 bytes apart modulo 128: no bank conflicts
  static constexpr int kPPitch = MR + 4;
  float q[MR * kPitch];
  float k[2][kF32Keys * kPitch];
  float v[2][kF32Keys * kPitch];
  float p[kF32Keys * kPPitch];  // [key][row]; -1 = hidden
  uint32_t mask[MR][2];
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool take) {
  const int n = take ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n)
               : "memory");
}

template <int D, int MR>
__global__ void __launch_bounds__(256) tree_f32_kernel(const TreeParams p) {
  using S = F32Smem<D, MR>;
  extern __shared__ __align__(16) uint8_t dsmem[];
  S& sm = *reinterpret_cast<S*>(dsmem);
  __shared__ int s_it[8];
  __shared__ long long s_base;
  constexpr int RPT = MR / 16;  // rows of a thread
  constexpr int DPT = D / 16;   // dims of a thread
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int g = p.H / p.Hkv, R = p.tile_rows;
  const float* qg = static_cast<const float*>(p.q);
  const float* kc = static_cast<const float*>(p.k_cache);
  const float* vc = static_cast<const float*>(p.v_cache);
  TreeWalk walk;
  if (warp == 0) walk.start(p, lane, blockIdx.x == 0);
  for (long long idx = blockIdx.x;; idx += gridDim.x) {
    __syncthreads();
    if (warp == 0) {
      int src = 0;
      const bool have = walk.find(p, lane, blockIdx.x == 0, idx, src);
      if (!have) {
        if (lane == 0) s_it[0] = -1;
      } else if (lane == src) {
        const TreeLane& ln = walk.ln;
        int split, rest;
        walk.item_of(p, idx, split, rest);
        s_it[0] = walk.b0 + lane;
        s_it[1] = rest / ln.tiles;
        s_it[2] = split;
        s_it[3] = rest % ln.tiles * R;
        s_it[4] = ln.q;
        s_it[5] = ln.c;
        s_it[6] = ln.cu0;
        s_it[7] = ln.ns;
        s_base = walk.pair_base;
      }
    }
    __syncthreads();
    const int b = s_it[0];
    if (b < 0) break;
    const int kvh = s_it[1], split = s_it[2], node0 = s_it[3], q_len = s_it[4], c = s_it[5],
              cu0 = s_it[6], ns = s_it[7];
    const long long pair_base = s_base;
    const int past = c - q_len;
    const int len = tree_split_len(past, p.grow * q_len * g, p.split0);
    const int t0 = split * len, t1 = split + 1 == ns ? c : t0 + len;
    const int* table = p.block_tables + (size_t)b * p.max_blocks;
    const int* par = p.parents + cu0;
    if (kvh == 0 && node0 == 0 && split + 1 == ns) {  // each lane's parents once
      for (int j = threadIdx.x; j < q_len; j += 256)
        if (par[j] < -1 || par[j] >= j) raise_flag(p.status, PA_FLAG_TREE);
    }
    // Q tile: pair r = (node r / g, head r % g); rows past the lane's stay zero
    for (int i = threadIdx.x; i < MR * (D / 4); i += 256) {
      const int r = i / (D / 4), d = (i % (D / 4)) * 4;
      const int node = node0 + r / g;
      float4 x = make_float4(0, 0, 0, 0);
      if (r / g < R && node < q_len)
        x = *reinterpret_cast<const float4*>(qg + ((size_t)(cu0 + node) * p.H + kvh * g + r % g) * D + d);
      *reinterpret_cast<float4*>(&sm.q[r * S::kPitch + d]) = x;
    }
    float m[RPT], l[RPT], o[RPT][DPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int j = 0; j < DPT; ++j) o[i][j] = 0.f;
    }
    // a thread copies the same 16-byte column of kLoads rows, kStep apart: as
    // many as share a block, so one block id each
    constexpr int kStep = 256 / (D / 4), kLoads = kF32Keys / kStep;
    const int lr = threadIdx.x / (D / 4), ld = threadIdx.x % (D / 4) * 4;
    int ids[kLoads];
    auto fetch_ids = [&](int key0) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int key = key0 + i * kStep;
        ids[i] = key < t1 ? table[key / p.bs] : 0;
      }
    };
    auto load_tile = [&](int key0, int buf) {  // zeros past the end
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = i * kStep + lr, key = key0 + r;
        int blk = ids[i];
        if (blk < 0 || blk >= p.NB) {
          raise_flag(p.status, PA_FLAG_BLOCK_RANGE);
          blk = 0;
        }
        const bool in = key < t1;
        const size_t at = (((size_t)blk * p.bs + (in ? key % p.bs : 0)) * p.Hkv + kvh) * D + ld;
        cp_async16(&sm.k[buf][r * S::kPitch + ld], kc + at, in);
        cp_async16(&sm.v[buf][r * S::kPitch + ld], vc + at, in);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch_ids(t0);
    load_tile(t0, 0);
    fetch_ids(t0 + kF32Keys);
    int buf = 0;
    for (int key0 = t0; key0 < t1; key0 += kF32Keys, buf ^= 1) {
      if (key0 + kF32Keys < t1) {
        load_tile(key0 + kF32Keys, buf ^ 1);
        fetch_ids(key0 + 2 * kF32Keys);
      }
      const bool tree = key0 + kF32Keys > past;
      if (tree && threadIdx.x < MR) {
        uint32_t w[2] = {0, 0};
        const int node = node0 + threadIdx.x / g;
        if ((int)threadIdx.x / g < R && node < q_len) tree_mask<2>(par, node, past, key0, w);
        sm.mask[threadIdx.x][0] = w[0];
        sm.mask[threadIdx.x][1] = w[1];
      }
      if (key0 + kF32Keys < t1)
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      else
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncthreads();
      // scores of rows ty RPT .. and keys tx + 16 j
      float sc[RPT][4];
#pragma unroll
      for (int i = 0; i < RPT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[i][j] = 0.f;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float4 qv[RPT], kv[4];
#pragma unroll
        for (int i = 0; i < RPT; ++i)
          qv[i] = *reinterpret_cast<const float4*>(&sm.q[(ty * RPT + i) * S::kPitch + d]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          kv[j] = *reinterpret_cast<const float4*>(&sm.k[buf][(tx + 16 * j) * S::kPitch + d]);
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            sc[i][j] = fmaf(qv[i].x, kv[j].x, sc[i][j]);
            sc[i][j] = fmaf(qv[i].y, kv[j].y, sc[i][j]);
            sc[i][j] = fmaf(qv[i].z, kv[j].z, sc[i][j]);
            sc[i][j] = fmaf(qv[i].w, kv[j].w, sc[i][j]);
          }
      }
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const int r = ty * RPT + i;
        bool vis[4];
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = tx + 16 * j;
          vis[j] = !tree || ((sm.mask[r][k >> 5] >> (k & 31)) & 1u);
          sc[i][j] *= p.scale_log2;
          if (vis[j]) mx = fmaxf(mx, sc[i][j]);
        }
#pragma unroll
        for (int w = 8; w >= 1; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
        const float mn = fmaxf(m[i], mx);
        const float ref = mn == -INFINITY ? 0.f : mn;  // no key so far: p = 0, l = 0
        const float al = m[i] == -INFINITY ? 1.f : exp2f(m[i] - mn);
        m[i] = mn;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = vis[j] ? exp2f(sc[i][j] - ref) : 0.f;
          sum += e;
          sm.p[(tx + 16 * j) * S::kPPitch + r] = vis[j] ? e : -1.f;
        }
#pragma unroll
        for (int w = 8; w >= 1; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
        l[i] = fmaf(l[i], al, sum);
#pragma unroll
        for (int j = 0; j < DPT; ++j) o[i][j] *= al;
      }
      __syncthreads();
      const int n = min(kF32Keys, t1 - key0);
#pragma unroll 4
      for (int k = 0; k < n; ++k) {
        float pv[RPT];
        if constexpr (RPT == 2) {
          const float2 x = *reinterpret_cast<const float2*>(&sm.p[k * S::kPPitch + ty * 2]);
          pv[0] = x.x;
          pv[1] = x.y;
        } else if constexpr (RPT == 4) {
          const float4 x = *reinterpret_cast<const float4*>(&sm.p[k * S::kPPitch + ty * 4]);
          pv[0] = x.x;
          pv[1] = x.y;
          pv[2] = x.z;
          pv[3] = x.w;
        } else {
          pv[0] = sm.p[k * S::kPPitch + ty];
        }
        float vv[DPT];
#pragma unroll
        for (int j = 0; j < DPT; j += 4) {
          const float4 x = *reinterpret_cast<const float4*>(&sm.v[buf][k * S::kPitch + tx * 4 + 16 * j]);
          vv[j] = x.x;
          vv[j + 1] = x.y;
          vv[j + 2] = x.z;
          vv[j + 3] = x.w;
        }
        // a hidden key's V may be infinite or NaN: it is left out, not multiplied by 0
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
          for (int j = 0; j < DPT; ++j)
            o[i][j] = !tree || pv[i] >= 0.f || pv[i] != pv[i] ? fmaf(pv[i], vv[j], o[i][j]) : o[i][j];
      }
      __syncthreads();  // the next load goes over this tile
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int r = ty * RPT + i, node = node0 + r / g, head = kvh * g + r % g;
      if (r / g >= R || node >= q_len) continue;
      float* dst;
      float f = 1.f;
      if (ns == 1) {
        f = 1.f / l[i];
        dst = static_cast<float*>(p.out) + ((size_t)(cu0 + node) * p.H + head) * D;
      } else {
        const long long e = (pair_base + (long long)node * ns + split) * p.H + head;
        if (tx == 0) p.ml[e] = tree_ml(m[i], l[i]);
        dst = p.acc + (size_t)e * D;
      }
#pragma unroll
      for (int j = 0; j < DPT; j += 4)
        *reinterpret_cast<float4*>(dst + tx * 4 + 16 * j) =
            make_float4(o[i][j] * f, o[i][j + 1] * f, o[i][j + 2] * f, o[i][j + 3] * f);
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <int D, int MR>
cudaError_t launch_f32(const TreeParams& p, int grid, cudaStream_t s) {
  auto kern = tree_f32_kernel<D, MR>;
  static unsigned long long done = 0;
  cudaError_t e = smem_opt_in(kern, (int)sizeof(F32Smem<D, MR>), &done);
  if (e != cudaSuccess) return e;
  kern<<<grid, 256, sizeof(F32Smem<D, MR>), s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_f32(const TreeParams& p, int tile_pairs, int grid, cudaStream_t s) {
  if (p.D == 128)
    return tile_pairs == 64   ? launch_f32<128, 64>(p, grid, s)
           : tile_pairs == 32 ? launch_f32<128, 32>(p, grid, s)
                              : launch_f32<128, 16>(p, grid, s);
  return tile_pairs == 64   ? launch_f32<64, 64>(p, grid, s)
         : tile_pairs == 32 ? launch_f32<64, 32>(p, grid, s)
                            : launch_f32<64, 16>(p, grid, s);
}

// Launched so that its CTAs may start while the kernel before it ends; they
// wait for its results.
cudaError_t launch_tree_fold(const TreeParams& p, bool f32, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  const long long rows = (long long)p.max_q_len * p.H;
  // four rows of each warp that an SM holds: from there a warp takes several
  const long long waves = rows * p.B / ((long long)num_sms() * 64 * 4);
  const int rows_per_warp = waves < 1 ? 1 : waves > 4 ? 4 : (int)waves;
  const int per_cta = kFoldWarps * rows_per_warp;
  cfg.gridDim = dim3((unsigned)((rows + per_cta - 1) / per_cta * p.B));
  cfg.blockDim = dim3(kFoldWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto kern = p.D == 128 ? (f32 ? tree_fold_kernel<128, true> : tree_fold_kernel<128, false>)
                         : (f32 ? tree_fold_kernel<64, true> : tree_fold_kernel<64, false>);
  return cudaLaunchKernelEx(&cfg, kern, p, rows_per_warp);
}

}  // namespace pa
