// C ABI of the speculative decoding operators: host-side validation and
// launch sequencing. Declarations and contracts are in include/pa.h.
#include <cfloat>
#include <cstring>
#include <initializer_list>

#include "pa_host.cuh"
#include "pa_pages.cuh"
#include "pa_tree.cuh"
#include "pa_verify.cuh"

namespace pa {

cudaError_t launch_tree_tc(const TreeParams& p, bool fp8, const CUtensorMap& q,
                           const CUtensorMap& qh, const CUtensorMap& k, const CUtensorMap& v,
                           int grid, cudaStream_t s);
cudaError_t launch_tree_q_pieces(const TreeParams& p, cudaStream_t s);
cudaError_t launch_tree_f32(const TreeParams& p, int tile_pairs, int grid, cudaStream_t s);
cudaError_t launch_tree_fold(const TreeParams& p, bool f32, cudaStream_t s);
cudaError_t launch_verify(const VerifyParams& p, cudaStream_t s);
cudaError_t launch_compact(PageParams& p, cudaStream_t s);
cudaError_t launch_copy_blocks(PageParams& p, cudaStream_t s);

namespace {

// Shortest split of a lane's keys (tree_split_len).
int tree_split0(pa_dtype dtype) { return dtype == PA_F32 ? 128 : 256; }

// A factor of scores as a float that is neither 0 nor infinite: a hidden key's
// score of -inf times 0, or a score of 0 times infinity, would be NaN.
float tree_score_scale(double x) {
  const float f = (float)x;
  return f < FLT_TRUE_MIN ? FLT_TRUE_MIN : f > FLT_MAX ? FLT_MAX : f;
}

// (node, head) pairs of a row tile.
int tile_pairs_of(pa_dtype dtype, int32_t max_q_len, int32_t g) {
  if (dtype != PA_F32) return kTreeRows;
  const long long pairs = (long long)max_q_len * g;
  return pairs <= 16 ? 16 : pairs <= 32 ? 32 : 64;
}

// Splits a lane of at most max_ctx_len keys can have (longer splits of lanes
// with more pairs only lower it).
long long max_tree_splits(int32_t max_ctx_len, pa_dtype dtype) {
  const long long s0 = tree_split0(dtype), n = ((long long)max_ctx_len + s0 - 1) / s0;
  return n < PA_TREE_MAX_SPLITS ? n : PA_TREE_MAX_SPLITS;
}

// The workspace: q's pieces (e4m3 caches), then what the fold reads (lanes
// that may be split).
struct TreeLayout {
  size_t counter, pieces, exps, info, ml, acc, bytes;
  long long pairs;
};

TreeLayout tree_layout(int32_t B, int32_t T, int32_t max_ctx_len, int32_t H, int32_t D, pa_dtype dtype) {
  TreeLayout L;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t was = at;
    at += align_up(n);
    return was;
  };
  const size_t rows = (size_t)T * H;
  L.counter = take(T > 0 && dtype != PA_F32 ? sizeof(unsigned long long) : 0);
  L.pieces = take(dtype == PA_FP8_E4M3 ? 2 * rows * D : 0);
  L.exps = take(dtype == PA_FP8_E4M3 ? rows : 0);
  const long long ns = max_tree_splits(max_ctx_len, dtype);
  L.pairs = ns > 1 ? (long long)T * ns : 0;
  L.info = take(L.pairs ? (size_t)B * sizeof(int4) : 0);
  L.ml = take((size_t)L.pairs * H * sizeof(float2));
  L.acc = take((size_t)L.pairs * H * D * sizeof(float));
  L.bytes = at;
  return L;
}

// q [T, H, D] bf16; box = 64 elements x the g heads of a kv head x R nodes:
// the 128-byte rows of one row tile, 128-byte swizzle.
bool encode_tree_q_map(CUtensorMap* map, const void* q, int T, int H, int D, int g, int R) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)H * D * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)g, (cuuint32_t)R};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// A cache as [Hkv][NB bs / 8 groups][halves][8 tokens][64 elements] (e4m3: one
// "half" of D codes); box = a block's groups of one head, which land as the
// 8-row, 128-byte (64-byte) swizzled groups of an operand tile.
bool encode_tree_cache_map(CUtensorMap* map, const void* cache, int NB, int bs, int Hkv, int D, bool fp8) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t e = fp8 ? 1 : 2, tok = (cuuint64_t)Hkv * D * e;
  const cuuint32_t inner = fp8 ? (cuuint32_t)D : 64, halves = (cuuint32_t)D / inner;
  cuuint64_t dims[5] = {inner, 8, halves, (cuuint64_t)NB * (cuuint64_t)bs / 8, (cuuint64_t)Hkv};
  cuuint64_t strides[4] = {tok, inner * e, 8 * tok, (cuuint64_t)D * e};
  cuuint32_t box[5] = {inner, 8, halves, (cuuint32_t)bs / 8, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  CUresult r = fn(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
                  const_cast<void*>(cache), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  inner * e == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// q's e4m3 pieces [2 T, H, D]; box = D codes x the g heads x R nodes.
bool encode_tree_pieces_map(CUtensorMap* map, const void* q, int T, int H, int D, int g, int R) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T * 2};
  cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)H * D};
  cuuint32_t box[3] = {(cuuint32_t)D, (cuuint32_t)g, (cuuint32_t)R};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(q), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE,
                  D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// 32-bit arrays (NULL is)
bool aligned4(std::initializer_list<const void*> ptrs) {
  for (const void* a : ptrs)
    if (reinterpret_cast<uintptr_t>(a) & 3u) return false;
  return true;
}

// Whether two arrays share a byte.
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

pa_status check_caches(void* const* k, void* const* v, int32_t layers) {
  for (int32_t i = 0; i < layers; ++i)
    if (!k[i] || !v[i] || !aligned16(k[i]) || !aligned16(v[i])) return PA_ERR_INVALID_ARG;
  return PA_OK;
}

// Bytes of a cache element.
int cache_bytes_of(pa_dtype d) { return d == PA_F32 ? 4 : d == PA_BF16 ? 2 : 1; }

// Launch in runs of at most kPageLayers layers.
template <typename Launch>
pa_status for_layers(PageParams& p, void* const* k, void* const* v, int32_t layers, Launch launch) {
  for (int32_t at = 0; at < layers; at += kPageLayers) {
    p.layers = layers - at < kPageLayers ? layers - at : kPageLayers;
    std::memcpy(p.k, k + at, p.layers * sizeof(void*));
    std::memcpy(p.v, v + at, p.layers * sizeof(void*));
    if (launch(p) != cudaSuccess) return PA_ERR_CUDA;
    count_launches(1);
  }
  return PA_OK;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

size_t pa_tree_workspace_bytes(int32_t B, int32_t T, int32_t max_q_len, int32_t max_ctx_len,
                               int32_t H, int32_t Hkv, int32_t D, int32_t block_size,
                               pa_dtype dtype) {
  if (B < 0 || T < 0 || max_q_len < 0 || max_ctx_len < 0 || max_q_len > PA_TREE_MAX_NODES ||
      max_ctx_len > (1 << 30))
    return 0;
  if (check_geometry(H, Hkv, D, block_size, dtype) != PA_OK) return 0;
  const size_t n = tree_layout(B, T, max_ctx_len, H, D, dtype).bytes;
  return n ? n : 256;  // 0 stands for unsupported arguments
}

pa_status pa_attention_tree(const void* q, const void* k_cache, const void* v_cache,
                            const int32_t* block_tables, int32_t max_blocks_per_seq,
                            const int32_t* cu_seqlens_q, const int32_t* ctx_lens,
                            const int32_t* tree_parents, const int64_t* slot_mapping,
                            const void* k_new, const void* v_new, void* out, int32_t B,
                            int32_t T, int32_t H, int32_t Hkv, int32_t D, int32_t block_size,
                            int32_t num_blocks, int32_t max_q_len, int32_t max_ctx_len,
                            float scale, pa_dtype dtype, float k_scale, float v_scale,
                            void* workspace, size_t workspace_bytes, int32_t* status,
                            void* stream) {
  // ---- host validation: nothing below touches CUDA until it all passes ----
  if (B < 0 || T < 0 || num_blocks <= 0 || max_q_len < 0 || max_ctx_len < 0)
    return PA_ERR_INVALID_ARG;
  pa_status st = check_geometry(H, Hkv, D, block_size, dtype);
  if (st != PA_OK) return st;
  if (max_q_len > PA_TREE_MAX_NODES || max_ctx_len > (1 << 30)) return PA_ERR_UNSUPPORTED;
  if (!std::isfinite(scale) || !(scale > 0.f)) return PA_ERR_INVALID_ARG;
  const bool fp8 = dtype == PA_FP8_E4M3, f32 = dtype == PA_F32;
  if (fp8 && !scales_ok(k_scale, v_scale)) return PA_ERR_INVALID_ARG;
  const bool with_write = slot_mapping || k_new || v_new;
  if (with_write && !(slot_mapping && k_new && v_new)) return PA_ERR_INVALID_ARG;
  if ((long long)num_blocks * block_size > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
  if (T > 0 && B == 0) return PA_ERR_INVALID_ARG;
  if (T == 0 || B == 0) return PA_OK;
  if (max_q_len > T) max_q_len = T;  // no lane has more rows; grids go by it
  if (!q || !k_cache || !v_cache || !block_tables || !cu_seqlens_q || !ctx_lens || !tree_parents ||
      !out || max_blocks_per_seq <= 0)
    return PA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out))
    return PA_ERR_INVALID_ARG;
  if (!aligned4({block_tables, cu_seqlens_q, ctx_lens, tree_parents, status})) return PA_ERR_INVALID_ARG;
  if (with_write && (!aligned16(k_new) || !aligned16(v_new) || (reinterpret_cast<uintptr_t>(slot_mapping) & 7u)))
    return PA_ERR_INVALID_ARG;
  const int g = H / Hkv;
  const long long ns = max_tree_splits(max_ctx_len, dtype);
  if (((long long)max_q_len * H + 7) / 8 * B > 0x7fffffffLL || ((long long)T * H + 7) / 8 > 0x7fffffffLL ||
      (long long)max_q_len * H * D > 0x7fffffffLL)
    return PA_ERR_UNSUPPORTED;
  const TreeLayout L = tree_layout(B, T, max_ctx_len, H, D, dtype);
  if (L.bytes && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)) ||
                  workspace_bytes < L.bytes))
    return PA_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (with_write) {
    st = pa_write_kv_scaled(k_new, v_new, const_cast<void*>(k_cache), const_cast<void*>(v_cache),
                            slot_mapping, T, num_blocks, block_size, Hkv, D, dtype, k_scale,
                            v_scale, status, stream);
    if (st != PA_OK) return st;
  }

  TreeParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = q;
  p.out = out;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.block_tables = block_tables;
  p.cu_seqlens = cu_seqlens_q;
  p.ctx_lens = ctx_lens;
  p.parents = tree_parents;
  p.status = status;
  p.max_blocks = max_blocks_per_seq;
  p.B = B;
  p.T = T;
  p.H = H;
  p.Hkv = Hkv;
  p.D = D;
  p.bs = block_size;
  p.NB = num_blocks;
  p.max_q_len = max_q_len;
  p.max_ctx_len = max_ctx_len;
  const int pairs = tile_pairs_of(dtype, max_q_len, g);
  p.tile_rows = pairs / g;
  p.split0 = tree_split0(dtype);
  p.grow = f32 ? 0 : 1;  // fp32 is bound by FMA: short splits spread it over the SMs
  p.scale_log2 = tree_score_scale((double)scale * 1.4426950408889634 * (fp8 ? (double)k_scale : 1.0));
  p.v_scale = fp8 ? v_scale : 1.f;
  p.wait_cycles = wait_cycles();
  p.skip_item = test_skip_item();
  char* ws = static_cast<char*>(workspace);
  if (fp8) {
    p.q_pieces = reinterpret_cast<uint8_t*>(ws + L.pieces);
    p.q_exp = reinterpret_cast<uint8_t*>(ws + L.exps);
  }
  if (L.pairs) {
    p.capacity = L.pairs;
    p.lane_info = reinterpret_cast<int4*>(ws + L.info);
    p.ml = reinterpret_cast<float2*>(ws + L.ml);
    p.acc = reinterpret_cast<float*>(ws + L.acc);
  }
  const long long tiles = (max_q_len + p.tile_rows - 1) / p.tile_rows;
  // at most; with max_q_len 0 one CTA says that the lanes' rows exceed it
  const long long items = max_q_len ? (long long)B * Hkv * (ns > 0 ? ns : 1) * tiles : 1;
  cudaError_t e;
  if (f32) {
    const long long most = 4LL * num_sms();
    e = launch_tree_f32(p, pairs, (int)(items < most ? items : most), s);
  } else {
    CUtensorMap tmQ, tmQh, tmK, tmV;
    if (!encode_tree_cache_map(&tmK, k_cache, num_blocks, block_size, Hkv, D, fp8) ||
        !encode_tree_cache_map(&tmV, v_cache, num_blocks, block_size, Hkv, D, fp8))
      return PA_ERR_CUDA;
    // q by whole row tiles and by half ones (lanes of at most 64 pairs)
    for (int half = 0; half < 2; ++half) {
      CUtensorMap* map = half ? &tmQh : &tmQ;
      const int rows = half ? kTreeRows / 2 / g : p.tile_rows;
      if (fp8 ? !encode_tree_pieces_map(map, p.q_pieces, T, H, D, g, rows)
              : !encode_tree_q_map(map, q, T, H, D, g, rows))
        return PA_ERR_CUDA;
    }
    const long long most = 2LL * num_sms();
    if (items > most) {
      p.counter = reinterpret_cast<unsigned long long*>(ws + L.counter);
      if (!fp8 && cudaMemsetAsync(p.counter, 0, sizeof(*p.counter), s) != cudaSuccess) return PA_ERR_CUDA;
    }
    e = fp8 ? launch_tree_q_pieces(p, s) : cudaSuccess;
    if (fp8) count_launches(1);
    if (e == cudaSuccess)
      e = launch_tree_tc(p, fp8, tmQ, tmQh, tmK, tmV, (int)(items < most ? items : most), s);
  }
  if (e != cudaSuccess) return PA_ERR_CUDA;
  count_launches(1);
  if (L.pairs && max_q_len) {
    if (launch_tree_fold(p, f32, s) != cudaSuccess) return PA_ERR_CUDA;
    count_launches(1);
  }
  return PA_OK;
}

pa_status pa_verify_tree(const float* target_probs, const float* draft_probs,
                         const int32_t* draft_tokens, const int32_t* tree_parents,
                         const int32_t* cu_seqlens_q, const float* u_accept,
                         const float* u_sample, int32_t* n_accepted, int32_t* path,
                         int32_t* tokens, int32_t B, int32_t T, int32_t vocab,
                         int32_t max_q_len, int32_t* status, void* stream) {
  if (B < 0 || T < 0 || vocab <= 0 || max_q_len <= 0) return PA_ERR_INVALID_ARG;
  if (max_q_len > PA_TREE_MAX_NODES || vocab > (1 << 24) || B > (1 << 27)) return PA_ERR_UNSUPPORTED;
  if (T > 0 && B == 0) return PA_ERR_INVALID_ARG;
  if (B == 0) return PA_OK;
  if (!cu_seqlens_q || !n_accepted) return PA_ERR_INVALID_ARG;
  if (T > 0 && (!target_probs || !draft_tokens || !tree_parents || !u_accept || !u_sample || !path ||
                !tokens))
    return PA_ERR_INVALID_ARG;
  if (!aligned16(target_probs) || !aligned16(draft_probs)) return PA_ERR_INVALID_ARG;
  if (!aligned4({draft_tokens, tree_parents, cu_seqlens_q, u_accept, u_sample, n_accepted, path, tokens, status}))
    return PA_ERR_INVALID_ARG;
  VerifyParams p;
  p.p = target_probs;
  p.q = draft_probs;
  p.tokens = draft_tokens;
  p.parents = tree_parents;
  p.cu = cu_seqlens_q;
  p.u_accept = u_accept;
  p.u_sample = u_sample;
  p.n_accepted = n_accepted;
  p.path = path;
  p.out_tokens = tokens;
  p.status = status;
  p.B = B;
  p.T = T;
  p.V = vocab;
  p.max_q_len = max_q_len;
  if (launch_verify(p, static_cast<cudaStream_t>(stream)) != cudaSuccess) return PA_ERR_CUDA;
  count_launches(1);
  return PA_OK;
}

pa_status pa_compact_kv(void* const* k_caches, void* const* v_caches, int32_t layers,
                        const int32_t* block_tables, int32_t max_blocks_per_seq,
                        const int32_t* cu_seqlens_q, const int32_t* ctx_lens,
                        const int32_t* path, const int32_t* n_accepted, int32_t* new_ctx_lens,
                        int32_t B, int32_t T, int32_t num_blocks, int32_t block_size,
                        int32_t Hkv, int32_t D, pa_dtype dtype, int32_t* status, void* stream) {
  if (layers < 0 || B < 0 || T < 0 || num_blocks <= 0) return PA_ERR_INVALID_ARG;
  pa_status st = check_geometry(Hkv, Hkv, D, block_size, dtype);
  if (st != PA_OK) return st;
  if ((long long)num_blocks * block_size > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
  if (T > 0 && B == 0) return PA_ERR_INVALID_ARG;
  if (B == 0 || layers == 0) return layers == 0 && B > 0 ? PA_ERR_INVALID_ARG : PA_OK;
  if (!k_caches || !v_caches || !block_tables || !cu_seqlens_q || !ctx_lens || (T > 0 && !path) ||
      !n_accepted || !new_ctx_lens || max_blocks_per_seq <= 0)
    return PA_ERR_INVALID_ARG;
  if (!aligned4({block_tables, cu_seqlens_q, ctx_lens, path, n_accepted, new_ctx_lens, status}))
    return PA_ERR_INVALID_ARG;
  // several CTAs, and the launches of further layers, read a lane's lengths and
  // path after one of them has written its new length
  const size_t i32 = sizeof(int32_t), new_bytes = (size_t)B * i32;
  if (overlap(new_ctx_lens, new_bytes, ctx_lens, (size_t)B * i32) ||
      overlap(new_ctx_lens, new_bytes, cu_seqlens_q, ((size_t)B + 1) * i32) ||
      overlap(new_ctx_lens, new_bytes, path, (size_t)T * i32) ||
      overlap(new_ctx_lens, new_bytes, n_accepted, (size_t)B * i32) ||
      overlap(new_ctx_lens, new_bytes, block_tables, (size_t)B * max_blocks_per_seq * i32))
    return PA_ERR_INVALID_ARG;
  st = check_caches(k_caches, v_caches, layers);
  if (st != PA_OK) return st;
  PageParams p;
  std::memset(&p, 0, sizeof(p));
  p.row_vecs = Hkv * D * cache_bytes_of(dtype) / 16;
  p.block_vecs = p.row_vecs * block_size;
  p.NB = num_blocks;
  p.bs = block_size;
  p.status = status;
  p.block_tables = block_tables;
  p.max_blocks = max_blocks_per_seq;
  p.cu = cu_seqlens_q;
  p.ctx = ctx_lens;
  p.path = path;
  p.n_accepted = n_accepted;
  p.new_ctx = new_ctx_lens;
  p.B = B;
  p.T = T;
  if ((long long)p.row_vecs * 2 * kPageLayers > 0x7fffffffLL || B > (1 << 20)) return PA_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return for_layers(p, k_caches, v_caches, layers, [s](PageParams& x) { return launch_compact(x, s); });
}

pa_status pa_copy_blocks(void* const* k_caches, void* const* v_caches, int32_t layers,
                         const int32_t* pairs, int32_t n, int32_t num_blocks,
                         int32_t block_size, int32_t Hkv, int32_t D, pa_dtype dtype,
                         int32_t* status, void* stream) {
  if (layers < 0 || n < 0 || num_blocks <= 0) return PA_ERR_INVALID_ARG;
  pa_status st = check_geometry(Hkv, Hkv, D, block_size, dtype);
  if (st != PA_OK) return st;
  if ((long long)num_blocks * block_size > 0x7fffffffLL || n > (1 << 16)) return PA_ERR_UNSUPPORTED;
  if (n == 0 || layers == 0) return PA_OK;
  if (!k_caches || !v_caches || !pairs || (reinterpret_cast<uintptr_t>(pairs) & 7u) || !aligned4({status}))
    return PA_ERR_INVALID_ARG;
  st = check_caches(k_caches, v_caches, layers);
  if (st != PA_OK) return st;
  PageParams p;
  std::memset(&p, 0, sizeof(p));
  p.row_vecs = Hkv * D * cache_bytes_of(dtype) / 16;
  p.block_vecs = p.row_vecs * block_size;
  p.NB = num_blocks;
  p.status = status;
  p.pairs = pairs;
  p.n = n;
  if ((long long)p.block_vecs * 2 > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return for_layers(p, k_caches, v_caches, layers, [s](PageParams& x) { return launch_copy_blocks(x, s); });
}

}  // extern "C"
