// Host side of the verify step's other operators: the 8-bit paged cache with
// its attention and eviction, and token log-probabilities (include/
// spec_verify.h). Argument validation, grids and launches; every kernel is
// launched with programmatic stream serialization and waits before it reads.

#include <algorithm>
#include <climits>
#include <cmath>

#include "spec_verify.h"
#include "host_util.cuh"
#include "attn_q8.cuh"
#include "attn_q8_rows.cuh"
#include "attn_weights_q8.cuh"
#include "kv_append_q8.cuh"
#include "kv_evict_q8.cuh"
#include "token_logprobs.cuh"

namespace {

using namespace sv;

constexpr size_t kAlign = 256;

sv_status done(cudaError_t e) { return e == cudaSuccess ? SV_OK : SV_ERR_CUDA; }

bool valid_cache(const sv_q8_cache* c) {
  return c && c->k && c->v && c->k_scale && c->v_scale && c->page_table && aligned(c->k, 16) && aligned(c->v, 16) &&
         aligned(c->k_scale, 4) && aligned(c->v_scale, 4) && aligned(c->page_table, 4) && c->num_pages >= 1 &&
         c->Hkv >= 1 && (c->D == 64 || c->D == 128) &&
         (c->page_size == 16 || c->page_size == 32 || c->page_size == 64 || c->page_size == 128) && c->max_pages >= 1 &&
         static_cast<int64_t>(c->max_pages) * c->page_size <= INT32_MAX - 255;   // positions and the ends of their tiles fit
}

Q8View view(const sv_q8_cache& c) {
  Q8View v;
  v.k = static_cast<uint8_t*>(c.k);
  v.v = static_cast<uint8_t*>(c.v);
  v.ks = c.k_scale;
  v.vs = c.v_scale;
  v.table = c.page_table;
  v.num_pages = c.num_pages;
  v.Hkv = c.Hkv;
  v.page_shift = c.page_size == 16 ? 4 : c.page_size == 32 ? 5 : c.page_size == 64 ? 6 : 7;
  v.max_pages = c.max_pages;
  return v;
}

bool valid_rows(const sv_rows* r, int es) {
  return r && r->data && aligned(r->data, 16) && r->stride_b * es % 16 == 0 && r->stride_n * es % 16 == 0 &&
         r->stride_h * es % 16 == 0;
}

int esize(int32_t dtype) { return dtype == SV_F32 ? 4 : dtype == SV_BF16 || dtype == SV_F16 ? 2 : 0; }

// ------------------------------------------------------------------ append

// Passes of a CTA's threads over rows: as many as the new rows can touch, up to
// four of 16-bit rows or two of 32-bit ones (64 or 128 bytes a thread held in
// registers), and a page at least. Measured with 3 prompts of 4099 tokens, 8
// heads of 128: bf16, pages of 16, four passes 17.4 us, two 18.4, one 20.5;
// fp32, pages of 64, two passes 21.6 us, four 24.5.
int append_passes(int64_t N, int P, int D, int es) {
  const int per = kAppendThreads / (D / kAppendEls);
  const int64_t rows = std::max<int64_t>(std::min<int64_t>(P - 1 + N, 8 / es * per), P);
  const int passes = static_cast<int>((rows + per - 1) / per);
  return passes == 3 ? 4 : passes;
}

template <typename T, int D>
cudaError_t launch_append(const AppendArgs& a, int passes, cudaStream_t st) {
  const int grid = 2 * a.B * a.c.Hkv * a.W;
  return passes == 1   ? launch(kv_append_q8_kernel<T, D, 1>, grid, kAppendThreads, 0, st, true, a)
         : passes == 2 ? launch(kv_append_q8_kernel<T, D, 2>, grid, kAppendThreads, 0, st, true, a)
                       : launch(kv_append_q8_kernel<T, D, 4>, grid, kAppendThreads, 0, st, true, a);
}

template <typename T>
cudaError_t launch_append(const AppendArgs& a, int passes, int D, cudaStream_t st) {
  return D == 128 ? launch_append<T, 128>(a, passes, st) : launch_append<T, 64>(a, passes, st);
}

// --------------------------------------------------------------- attention

// Rows of a kv head that a call takes. A row's node is the high word of a product
// with inv_g, which is over 2^32 / G by `over` / G: exact for rows below 2^32 / over.
bool valid_row_count(int64_t rows, int64_t G, uint64_t inv_g) {
  const int64_t over = static_cast<int64_t>(inv_g * G - (uint64_t{1} << 32));
  return rows <= SV_MAX_TREE_NODES * 1024 && rows * over <= int64_t{1} << 32;
}

// Rows of a block: all of a kv head's as columns where they are at most 32 (in
// one or two groups of 16), else blocks of 128 lanes. 32 requests of up to 8192
// tokens, 8 heads of 128, when the rule was set: 16 rows took 82 us in one group,
// 93 in two, 136 as lanes; 24 rows 96 and 138 us, 32 rows 98 and 140; 64 rows 145
// as lanes. (Now 16 rows 78, 24 rows 92.)
int attn_block(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 128; }

constexpr int kAttnGridMost = 320;   // CTAs a workspace is sized for: two an SM of 152, whatever the device

// cuTensorMapEncodeTiled of the loaded driver.
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled() {
  static std::atomic<void*> found{nullptr};
  void* f = found.load(std::memory_order_acquire);
  if (!f) {
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      return nullptr;
    found.store(f, std::memory_order_release);
  }
  return reinterpret_cast<EncodeTiled>(f);
}

// The codes as [pages * heads][page rows][D bytes], read in boxes of a page's
// head, swizzled for the tensor cores.
bool code_map(const sv_q8_cache& c, void* codes, CUtensorMap* m) {
  const EncodeTiled f = encode_tiled();
  if (!f) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c.D), static_cast<cuuint64_t>(c.page_size),
                              static_cast<cuuint64_t>(c.num_pages) * c.Hkv};
  const cuuint64_t strides[2] = {dims[0], dims[0] * dims[1]};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(c.D), static_cast<cuuint32_t>(c.page_size), 1}, one[3] = {1, 1, 1};
  return f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, codes, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
           c.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D, int MT>
cudaError_t launch_join(const AttnArgs& a, int64_t items, cudaStream_t st) {
  const int64_t grid = items * 4 * MT + (a.status ? a.B : 0);
  return launch(attn_q8_combine_kernel<T, D, MT>, static_cast<int>(grid), kAttnThreads, 0, st, true, a);
}

template <typename T, int D, int NT>
cudaError_t launch_rows(const sv_q8_cache& c, AttnArgs& a, int64_t items, cudaStream_t st) {
  CUtensorMap k;
  if (!code_map(c, c.k, &k)) return cudaErrorInvalidValue;
  using L = RowLayout<D, NT>;
  const int smem = L::bytes(L::nodes(a.N, a.G), (a.N + 31) / 32);
  if (2 * (smem + 1024) > 228 * 1024) a.grid = std::min(a.grid, sm_count());   // one CTA an SM
  const cudaError_t e = launch_smem<attn_q8_rows_kernel<T, D, NT>>(a.grid, kRowThreads, smem, L::most(), st, k, a);
  return e != cudaSuccess ? e : launch_join<T, D, 8>(a, items, st);
}

template <typename T, int D, int MT, int NT>
cudaError_t launch_cols(const sv_q8_cache& c, const AttnArgs& a, int64_t items, cudaStream_t st) {
  CUtensorMap k, v;
  if (!code_map(c, c.k, &k) || !code_map(c, c.v, &v)) return cudaErrorInvalidValue;
  constexpr int kSmem = ColLayout<D, MT, NT>::bytes(1);   // at most 32 rows, so 32 nodes: one mask word
  const cudaError_t e = launch_smem<attn_q8_cols_kernel<T, D, MT, NT>>(a.grid, ColLayout<D, MT, NT>::kThreads, kSmem, kSmem, st, k, v, a);
  return e != cudaSuccess ? e : launch_join<T, D, MT>(a, items, st);
}

template <typename T, int D, int MT, int NT>
cudaError_t launch_weights(const sv_q8_cache& c, const WeightArgs& a, cudaStream_t st) {
  CUtensorMap k;
  if (!code_map(c, c.k, &k)) return cudaErrorInvalidValue;
  constexpr int kSmem = WtLayout<D, MT, NT>::kBytes;
  return launch_smem<attn_weights_q8_kernel<T, D, MT, NT>>(a.grid, kWtThreads, kSmem, kSmem, st, k, a);
}

// Columns for the rows there are: 8 requests of up to 65536 tokens, 64 query
// heads on 8 of 64, 16 rows 46.7 us (49.4 with columns for 64), 32 rows 53.1
// (54.9).
template <typename T, int D, int NT>
cudaError_t launch_weights(const sv_q8_cache& c, const WeightArgs& a, int64_t rows, cudaStream_t st) {
  return rows <= 16   ? launch_weights<T, D, 1, NT>(c, a, st)
         : rows <= 32 ? launch_weights<T, D, 2, NT>(c, a, st)
                      : launch_weights<T, D, 4, NT>(c, a, st);
}

size_t attn_ws_part_bytes(int block, int D) {
  return align_up(static_cast<size_t>(2) * kAttnGridMost * block * (D + 4) * sizeof(float), kAlign);
}

// ---------------------------------------------------------------- logprobs

int64_t lp_vecs(int64_t V, int es) { return (V * es + 30) / 16; }   // a row's hull, wherever it starts

bool valid_t(float t) { return std::isfinite(t) && t >= 1e-4f; }

struct LpPlan {
  int threads = 0, segs = 0, per = 0;   // CTAs' threads, equal segments, in vectors
  size_t off_cand = 0, total = 0;
};

bool lp_plan(int64_t rows, int64_t V, int es, int n_top, LpPlan* p) {
  if (rows < 0 || V < 1 || es == 0 || n_top < 0 || n_top > SV_MAX_TOP_ALTERNATIVES) return false;
  const int64_t vecs = lp_vecs(V, es);
  p->threads = n_top ? kLpTopThreads : kLpThreads;
  const int most = p->threads * kLpVecs;
  p->segs = static_cast<int>((vecs + most - 1) / most);
  p->per = static_cast<int>(align_up((vecs + p->segs - 1) / p->segs, p->threads));
  if (rows * p->segs > INT32_MAX) return false;
  p->off_cand = align_up(static_cast<size_t>(rows) * p->segs * (p->threads / 32) * sizeof(LpPartial), kAlign);
  p->total = p->off_cand + align_up(static_cast<size_t>(rows) * p->segs * n_top * sizeof(uint64_t), kAlign);
  if (p->total < kAlign) p->total = kAlign;
  return true;
}

}  // namespace

extern "C" {

sv_status spec_kv_append_q8(const sv_q8_cache* cache, const sv_rows* k_new, const sv_rows* v_new, int32_t dtype,
                            int32_t B, int32_t N, const int32_t* seq_base, const int32_t* path_nodes,
                            int32_t path_cols, const int32_t* num_accepted, int32_t* out_len, int32_t* out_status,
                            void* stream) {
  const int es = esize(dtype);
  if (es == 0) return SV_ERR_UNSUPPORTED_DTYPE;
  if (B < 0 || N < 1 || (path_nodes && (path_cols < 1 || !num_accepted))) return SV_ERR_INVALID_ARG;
  if (B == 0) return SV_OK;
  if (!valid_cache(cache) || !valid_rows(k_new, es) || !valid_rows(v_new, es) || !seq_base || !out_len ||
      !aligned(seq_base, 4) || !aligned(path_nodes, 4) || !aligned(num_accepted, 4) || !aligned(out_len, 4) ||
      !aligned(out_status, 4))
    return SV_ERR_INVALID_ARG;
  AppendArgs a;
  const sv_rows* r[2] = {k_new, v_new};
  for (int i = 0; i < 2; ++i) {
    a.x[i] = static_cast<const uint8_t*>(r[i]->data);
    a.sb[i] = r[i]->stride_b * es;
    a.sn[i] = r[i]->stride_n * es;
    a.sh[i] = r[i]->stride_h * es;
  }
  a.c = view(*cache);
  a.base = seq_base;
  a.path = path_nodes;
  a.num_acc = num_accepted;
  a.path_cols = path_cols;
  a.N = N;
  const int P = cache->page_size, D = cache->D, passes = append_passes(N, P, D, es);
  const int64_t rows = std::min<int64_t>(P - 1 + static_cast<int64_t>(N), static_cast<int64_t>(cache->max_pages) * P);
  const int tile = passes * (kAppendThreads / (D / kAppendEls));
  a.W = static_cast<int32_t>((rows + tile - 1) / tile);
  a.B = B;
  a.out_len = out_len;
  a.status = out_status;
  if (2ll * B * cache->Hkv * a.W > INT32_MAX) return SV_ERR_INVALID_ARG;
  if (out_len == seq_base || out_len == num_accepted) return SV_ERR_INVALID_ARG;   // read by CTAs that start later
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return done(dtype == SV_F32    ? launch_append<TypeF32>(a, passes, D, st)
              : dtype == SV_BF16 ? launch_append<TypeBf16>(a, passes, D, st)
                                 : launch_append<TypeF16>(a, passes, D, st));
}

size_t spec_attention_q8_workspace_size(int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D) {
  if (B < 0 || N < 1 || N > SV_MAX_TREE_NODES || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || (D != 64 && D != 128)) return 0;
  return attn_ws_part_bytes(attn_block(static_cast<int64_t>(N) * (Hq / Hkv)), D) + align_up(kAttnGridMost * sizeof(uint32_t), kAlign) +
         align_up((static_cast<size_t>(B) + 1) * sizeof(int32_t), kAlign);
}

sv_status spec_attention_q8(const sv_rows* q, int32_t dtype, const sv_q8_cache* cache, int32_t B, int32_t N, int32_t Hq,
                            const int32_t* seq_base, const int32_t* parents, const int32_t* n_nodes, float sm_scale,
                            void* out, float* out_lse, int32_t* out_status, void* workspace, size_t workspace_bytes,
                            void* stream) {
  if (dtype != SV_BF16 && dtype != SV_F16) return SV_ERR_UNSUPPORTED_DTYPE;
  if (B < 0 || N < 1 || N > SV_MAX_TREE_NODES || !std::isfinite(sm_scale)) return SV_ERR_INVALID_ARG;
  if (B == 0) return SV_OK;
  if (!valid_cache(cache) || Hq < cache->Hkv || Hq % cache->Hkv != 0 || !valid_rows(q, 2) || !seq_base || !out ||
      !workspace || !aligned(seq_base, 4) || !aligned(parents, 4) || !aligned(n_nodes, 4) || !aligned(out, 16) ||
      !aligned(out_lse, 4) || !aligned(out_status, 4) || !aligned(workspace, 16))
    return SV_ERR_INVALID_ARG;
  const size_t need = spec_attention_q8_workspace_size(B, N, Hq, cache->Hkv, cache->D);
  if (need == 0) return SV_ERR_INVALID_ARG;
  if (workspace_bytes < need) return SV_ERR_WORKSPACE_TOO_SMALL;
  AttnArgs a;
  a.q = static_cast<const uint8_t*>(q->data);
  a.sqb = q->stride_b * 2;
  a.sqn = q->stride_n * 2;
  a.sqh = q->stride_h * 2;
  a.c = view(*cache);
  a.base = seq_base;
  a.n_nodes = n_nodes;
  a.parents = parents;
  a.out = out;
  a.lse = out_lse;
  a.status = out_status;
  a.B = B;
  a.N = N;
  a.Hq = Hq;
  a.G = Hq / cache->Hkv;
  a.inv_g = ((1ull << 32) + a.G - 1) / a.G;
  const int64_t rows = static_cast<int64_t>(N) * a.G;
  if (!valid_row_count(rows, a.G, a.inv_g)) return SV_ERR_INVALID_ARG;
  const int block = attn_block(rows);
  a.RB = static_cast<int32_t>((rows + block - 1) / block);
  a.coef = static_cast<float>(static_cast<double>(sm_scale) * 1.4426950408889634);
  a.part = static_cast<float*>(workspace);
  uint8_t* after = static_cast<uint8_t*>(workspace) + attn_ws_part_bytes(block, cache->D);
  a.failed = reinterpret_cast<uint32_t*>(after);
  a.plan = reinterpret_cast<int32_t*>(after + align_up(kAttnGridMost * sizeof(uint32_t), kAlign));
  const int64_t items = static_cast<int64_t>(B) * cache->Hkv * a.RB;
  const int64_t tiles = (static_cast<int64_t>(cache->max_pages) * cache->page_size + kColTile - 1) / kColTile;
  if (items * 32 + B > INT32_MAX || items * tiles > INT32_MAX) return SV_ERR_INVALID_ARG;
  a.grid = static_cast<int32_t>(std::min<int64_t>({2 * sm_count(), kAttnGridMost, items * tiles}));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const sv_q8_cache& c = *cache;
  const bool wide = c.D == 128;
  cudaError_t e;
  if (dtype == SV_BF16)
    e = block == 128  ? (wide ? launch_rows<TypeBf16, 128, 2>(c, a, items, st) : launch_rows<TypeBf16, 64, 2>(c, a, items, st))
        : block == 32 ? (wide ? launch_cols<TypeBf16, 128, 2, 2>(c, a, items, st) : launch_cols<TypeBf16, 64, 2, 2>(c, a, items, st))
                      : (wide ? launch_cols<TypeBf16, 128, 1, 2>(c, a, items, st) : launch_cols<TypeBf16, 64, 1, 2>(c, a, items, st));
  else
    e = block == 128  ? (wide ? launch_rows<TypeF16, 128, 3>(c, a, items, st) : launch_rows<TypeF16, 64, 3>(c, a, items, st))
        : block == 32 ? (wide ? launch_cols<TypeF16, 128, 2, 3>(c, a, items, st) : launch_cols<TypeF16, 64, 2, 3>(c, a, items, st))
                      : (wide ? launch_cols<TypeF16, 128, 1, 3>(c, a, items, st) : launch_cols<TypeF16, 64, 1, 3>(c, a, items, st));
  return done(e);
}

sv_status spec_attention_weights_q8(const sv_rows* q, int32_t dtype, const float* lse, const sv_q8_cache* cache,
                                    int32_t B, int32_t N, int32_t Hq, const int32_t* seq_base,
                                    const int32_t* path_nodes, int32_t path_cols, const int32_t* num_accepted,
                                    float sm_scale, float decay, const float* scores, float* out_scores, int32_t S,
                                    int32_t* out_status, void* stream) {
  if (dtype != SV_BF16 && dtype != SV_F16) return SV_ERR_UNSUPPORTED_DTYPE;
  if (B < 0 || N < 1 || S < 1 || !std::isfinite(sm_scale) || !std::isfinite(decay) ||
      (path_nodes && (path_cols < 1 || !num_accepted)))
    return SV_ERR_INVALID_ARG;
  if (B == 0) return SV_OK;
  if (!valid_cache(cache) || Hq < cache->Hkv || Hq % cache->Hkv != 0 || !valid_rows(q, 2) || !lse || !seq_base || !scores ||
      !out_scores || !aligned(lse, 4) || !aligned(seq_base, 4) || !aligned(path_nodes, 4) || !aligned(num_accepted, 4) ||
      !aligned(scores, 4) || !aligned(out_scores, 4) || !aligned(out_status, 4))
    return SV_ERR_INVALID_ARG;
  WeightArgs a;
  a.q = static_cast<const uint8_t*>(q->data);
  a.sqb = q->stride_b * 2;
  a.sqn = q->stride_n * 2;
  a.sqh = q->stride_h * 2;
  a.lse = lse;
  a.c = view(*cache);
  a.base = seq_base;
  a.path = path_nodes;
  a.num_acc = num_accepted;
  a.scores = scores;
  a.out = out_scores;
  a.status = out_status;
  a.path_cols = path_cols;
  a.B = B;
  a.N = N;
  a.G = Hq / cache->Hkv;
  a.Hq = Hq;
  a.S = S;
  a.coef = static_cast<float>(static_cast<double>(sm_scale) * 1.4426950408889634);
  a.decay = decay;
  const int64_t rows = static_cast<int64_t>(path_nodes ? std::min(path_cols, N) : N) * a.G;
  a.inv_g = ((1ull << 32) + a.G - 1) / a.G;
  if (!valid_row_count(rows, a.G, a.inv_g)) return SV_ERR_INVALID_ARG;
  const int64_t items = static_cast<int64_t>(B) * cache->Hkv;
  const int64_t tiles = (static_cast<int64_t>(cache->max_pages) * cache->page_size + kColTile - 1) / kColTile;
  if (items > INT32_MAX || items * tiles > INT32_MAX) return SV_ERR_INVALID_ARG;
  a.grid = static_cast<int32_t>(std::min<int64_t>(2 * sm_count(), items * tiles));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const sv_q8_cache& c = *cache;
  if (dtype == SV_BF16)
    return done(c.D == 128 ? launch_weights<TypeBf16, 128, 2>(c, a, rows, st) : launch_weights<TypeBf16, 64, 2>(c, a, rows, st));
  return done(c.D == 128 ? launch_weights<TypeF16, 128, 3>(c, a, rows, st) : launch_weights<TypeF16, 64, 3>(c, a, rows, st));
}

size_t spec_kv_evict_q8_workspace_size(int32_t B, int32_t Hkv, int32_t keep) {
  if (B < 0 || Hkv < 1 || keep < 1) return 0;
  const size_t bh = static_cast<size_t>(B) * Hkv;
  return align_up((2 * bh * keep + bh) * sizeof(int32_t), kAlign) + kAlign;
}

sv_status spec_kv_evict_q8(const sv_q8_cache* cache, int32_t B, const int32_t* seq_len, const float* scores,
                           const int32_t* positions, int32_t S, int32_t keep, int32_t sinks,
                           const int32_t* protect_from, float* out_scores, int32_t* out_positions, int32_t* out_len,
                           int32_t* out_status, void* workspace, size_t workspace_bytes, void* stream) {
  if (B < 0 || S < 1 || keep < 1) return SV_ERR_INVALID_ARG;
  if (B == 0) return SV_OK;
  if (!valid_cache(cache) || keep % cache->page_size != 0 || keep > S || S > 1 << 30 ||
      static_cast<int64_t>(cache->num_pages) * cache->Hkv > (int64_t{1} << 32) / cache->page_size ||
      keep > static_cast<int64_t>(cache->max_pages) * cache->page_size || !seq_len || !scores || !positions ||
      !out_scores || !out_positions || !out_len || !workspace || !aligned(seq_len, 4) || !aligned(scores, 4) ||
      !aligned(positions, 4) || !aligned(protect_from, 4) || !aligned(out_scores, 4) || !aligned(out_positions, 4) ||
      !aligned(out_len, 4) || !aligned(out_status, 4) || !aligned(workspace, 16))
    return SV_ERR_INVALID_ARG;
  if (workspace_bytes < spec_kv_evict_q8_workspace_size(B, cache->Hkv, keep)) return SV_ERR_WORKSPACE_TOO_SMALL;
  if (out_len == seq_len || out_len == protect_from) return SV_ERR_INVALID_ARG;   // read by CTAs that start later
  const int64_t bh = static_cast<int64_t>(B) * cache->Hkv;
  const int64_t per_cta = static_cast<int64_t>(kMvWarps) * std::max(cache->page_size, 32);
  const int64_t groups = (keep + per_cta - 1) / per_cta;
  if (bh * groups > INT32_MAX) return SV_ERR_INVALID_ARG;
  EvictArgs a;
  a.c = view(*cache);
  a.seq_len = seq_len;
  a.scores = scores;
  a.positions = positions;
  a.protect_from = protect_from;
  a.out_scores = out_scores;
  a.out_positions = out_positions;
  a.out_len = out_len;
  a.status = out_status;
  a.src = static_cast<uint32_t*>(workspace);
  a.movers = a.src + bh * keep;
  a.n_moves = reinterpret_cast<int32_t*>(a.movers + bh * keep);
  a.B = B;
  a.S = S;
  a.keep = keep;
  a.sinks = sinks;
  a.n_keys = std::min(S, kEvMaxKeys);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t smem = (kEvBins + static_cast<size_t>(a.n_keys)) * sizeof(uint32_t);
  const size_t most = (kEvBins + static_cast<size_t>(kEvMaxKeys)) * sizeof(uint32_t);
  cudaError_t e = launch_smem<kv_evict_select_kernel>(static_cast<int>(bh), kEvThreads, smem, most, st, a);
  if (e != cudaSuccess) return SV_ERR_CUDA;
  const int grid = static_cast<int>(bh * groups);
  return done(cache->D == 128 ? launch(kv_evict_move_kernel<128>, grid, kMvWarps * 32, 0, st, true, a)
                              : launch(kv_evict_move_kernel<64>, grid, kMvWarps * 32, 0, st, true, a));
}

size_t spec_token_logprobs_workspace_size(int32_t rows, int32_t V, int32_t dtype, int32_t n_top) {
  LpPlan p;
  return lp_plan(rows, V, dtype == SV_F16 ? 0 : esize(dtype), n_top, &p) ? p.total : 0;
}

sv_status spec_token_logprobs(const void* logits, int32_t dtype, int64_t row_stride, const int32_t* tokens,
                              int32_t rows, int32_t V, float temperature, int32_t n_top, float* out_logprob,
                              float* out_entropy, float* out_lse, float* out_saved, int32_t* out_top_tokens,
                              float* out_top_logprobs, int32_t* out_status, void* workspace, size_t workspace_bytes,
                              void* stream) {
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_UNSUPPORTED_DTYPE;
  const int es = esize(dtype);
  LpPlan p;
  if (!lp_plan(rows, V, es, n_top, &p) || row_stride < V || !valid_t(temperature)) return SV_ERR_INVALID_ARG;
  if (rows == 0) return SV_OK;
  if (!logits || !tokens || !out_logprob || !workspace || (n_top > 0 && (!out_top_tokens || !out_top_logprobs)) ||
      !aligned(logits, es) || !aligned(tokens, 4) || !aligned(out_logprob, 4) || !aligned(out_entropy, 4) ||
      !aligned(out_lse, 4) || !aligned(out_saved, 16) || !aligned(out_top_tokens, 4) || !aligned(out_top_logprobs, 4) ||
      !aligned(out_status, 4) || !aligned(workspace, 16))
    return SV_ERR_INVALID_ARG;
  if (workspace_bytes < p.total) return SV_ERR_WORKSPACE_TOO_SMALL;
  LogprobArgs a;
  a.x = static_cast<const uint8_t*>(logits);
  a.stride = row_stride * es;
  a.tokens = tokens;
  a.rows = rows;
  a.V = V;
  a.segs = p.segs;
  a.per = p.per;
  a.n_top = n_top;
  a.c = static_cast<float>(1.4426950408889634 / temperature);
  a.inv_t = static_cast<float>(1.0 / temperature);
  a.part = static_cast<LpPartial*>(workspace);
  a.cand = reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(workspace) + p.off_cand);
  a.logprob = out_logprob;
  a.entropy = out_entropy;
  a.lse = out_lse;
  a.saved = reinterpret_cast<float4*>(out_saved);
  a.top_tokens = out_top_tokens;
  a.top_logprobs = out_top_logprobs;
  a.status = out_status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int grid = rows * p.segs, join = (rows + kLpJoinWarps - 1) / kLpJoinWarps;
  cudaError_t e;
  if (es == 2)
    e = n_top ? launch(token_logprobs_kernel<2, true>, grid, p.threads, 0, st, true, a)
              : launch(token_logprobs_kernel<2, false>, grid, p.threads, 0, st, true, a);
  else
    e = n_top ? launch(token_logprobs_kernel<4, true>, grid, p.threads, 0, st, true, a)
              : launch(token_logprobs_kernel<4, false>, grid, p.threads, 0, st, true, a);
  if (e != cudaSuccess) return SV_ERR_CUDA;
  return done(es == 2 ? launch(token_logprobs_join_kernel<2>, join, kLpJoinWarps * 32, 0, st, true, a)
                      : launch(token_logprobs_join_kernel<4>, join, kLpJoinWarps * 32, 0, st, true, a));
}

sv_status spec_token_logprobs_backward(const void* logits, int32_t dtype, int64_t row_stride, const int32_t* tokens,
                                       const float* saved, const float* grad_logprob, const float* grad_entropy,
                                       int32_t rows, int32_t V, float temperature, void* out_grad,
                                       int64_t grad_row_stride, void* stream) {
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_UNSUPPORTED_DTYPE;
  const int es = esize(dtype);
  LpPlan p;
  if (!lp_plan(rows, V, es, 0, &p) || row_stride < V || grad_row_stride < V || !valid_t(temperature) ||
      (out_grad == logits && row_stride != grad_row_stride))
    return SV_ERR_INVALID_ARG;
  if (rows == 0) return SV_OK;
  if (!logits || !tokens || !saved || !grad_logprob || !out_grad || !aligned(logits, es) || !aligned(tokens, 4) ||
      !aligned(saved, 16) || !aligned(grad_logprob, 4) || !aligned(grad_entropy, 4) || !aligned(out_grad, es))
    return SV_ERR_INVALID_ARG;
  LogprobGradArgs a;
  a.x = static_cast<const uint8_t*>(logits);
  a.stride = row_stride * es;
  a.dx = static_cast<uint8_t*>(out_grad);
  a.dstride = grad_row_stride * es;
  a.tokens = tokens;
  a.saved = reinterpret_cast<const float4*>(saved);
  a.g = grad_logprob;
  a.h = grad_entropy;
  a.rows = rows;
  a.V = V;
  a.segs = p.segs;
  a.per = p.per;
  a.c = static_cast<float>(1.4426950408889634 / temperature);
  a.inv_t = static_cast<float>(1.0 / temperature);
  const bool vec = (reinterpret_cast<uintptr_t>(logits) - reinterpret_cast<uintptr_t>(out_grad)) % 16 == 0 &&
                   (a.stride - a.dstride) % 16 == 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int grid = rows * p.segs;
  if (es == 2)
    return done(vec ? launch(token_logprobs_grad_kernel<2, true>, grid, p.threads, 0, st, true, a)
                    : launch(token_logprobs_grad_kernel<2, false>, grid, p.threads, 0, st, true, a));
  return done(vec ? launch(token_logprobs_grad_kernel<4, true>, grid, p.threads, 0, st, true, a)
                  : launch(token_logprobs_grad_kernel<4, false>, grid, p.threads, 0, st, true, a));
}

}  // extern "C"
