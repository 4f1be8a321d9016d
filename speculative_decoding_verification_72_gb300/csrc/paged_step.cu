// Host side of the 16-bit paged cache's operators: appending with rotation, and
// attention (include/spec_verify.h). Argument validation, grids and launches;
// every kernel is launched with programmatic stream serialization and waits
// before it reads.

#include <algorithm>
#include <climits>
#include <cmath>

#include "spec_verify.h"
#include "host_util.cuh"
#include "attn_paged_rows.cuh"
#include "kv_append_rope.cuh"

namespace {

using namespace sv;

constexpr size_t kAlign = 256;

int64_t stride_or(int64_t stride, int64_t size, int64_t other) { return size == 1 ? other : stride; }

// A tensor's byte strides of page, token and head; a dimension of one has none of its own.
bool strides_of(const sv_paged_cache& c, const int64_t* given, int64_t* page, int64_t* token, int64_t* head) {
  const int64_t row = 2ll * c.D;
  *token = given[1] * 2;
  *head = stride_or(given[2] * 2, c.Hkv, row);
  *page = stride_or(given[0] * 2, c.num_pages, row);
  for (int64_t s : {*page, *token, *head})
    if (s < row || s % 16 != 0 || s >= int64_t{1} << 40) return false;
  return true;
}

bool view(const sv_paged_cache* c, PagedView* v) {
  if (!c || !c->k || !c->v || !c->page_table || !aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->page_table, 4) ||
      c->num_pages < 1 || c->Hkv < 1 || (c->D != 64 && c->D != 128) || c->max_pages < 1 ||
      (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) ||
      static_cast<int64_t>(c->max_pages) * c->page_size > INT32_MAX - 255)   // positions and the ends of their tiles fit
    return false;
  v->x[0] = static_cast<uint8_t*>(c->k);
  v->x[1] = static_cast<uint8_t*>(c->v);
  if (!strides_of(*c, c->k_strides, &v->sp[0], &v->st[0], &v->sh[0]) || !strides_of(*c, c->v_strides, &v->sp[1], &v->st[1], &v->sh[1]))
    return false;
  v->table = c->page_table;
  v->num_pages = c->num_pages;
  v->Hkv = c->Hkv;
  v->page_shift = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
  v->max_pages = c->max_pages;
  return true;
}

// K or V as [page][head][token][element], read in boxes of 64 elements of a
// page's tokens, swizzled for the tensor cores.
bool page_map(const sv_paged_cache& c, const PagedView& v, int kv, CUtensorMap* m) {
  const EncodeTiled f = encode_tiled();
  if (!f) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.D), static_cast<cuuint64_t>(c.page_size), static_cast<cuuint64_t>(c.Hkv),
                              static_cast<cuuint64_t>(c.num_pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(v.st[kv]), static_cast<cuuint64_t>(v.sh[kv]),
                                 static_cast<cuuint64_t>(v.sp[kv])};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(c.page_size), 1, 1}, one[4] = {1, 1, 1, 1};
  return f(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, v.x[kv], dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// --------------------------------------------------------------- attention

// Rows of a block: all of a kv head's as columns where they are at most 32 (in
// one or two groups of 16), as 128 lanes that share the tiles between their two
// copies where they are at most 128, else blocks of 256 lanes. Each is there for
// its time: 16 requests of 48 rows over a window of 4096 took 49 us as 128 lanes
// that share tiles and 58 us as lanes of one half; with 32 rows as lanes
// half of what the tensor cores do would be rows that are not there.
int paged_block(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 128 ? 128 : kPgRowBlock; }

// What an item's beginning and end (q, first products, the last rows out) cost, in
// tiles. Of few rows: 32 chains of 24 rows 144 us at 0, 140 at 1, 138 at 2. Of many:
// prompts of 4099 329 us at 2, 279 at 3, 257 at 4, 262 at 6; capped trees 127 at 3, 130 at 4.
constexpr int kPagedColExtra = 2, kPagedRowExtra = 4;

constexpr int kPagedGridMost = 160;   // CTAs a workspace is sized for: one an SM, whatever the device
constexpr int64_t kPagedMostRows = int64_t{1} << 26;   // rows of a kv head; their node is exact up to 2^32 / G

struct PagedPlan {
  int block = 0;
  int64_t RB = 0;
  size_t off_first = 0, off_failed = 0, off_plan = 0, total = 0;
};

bool paged_plan(int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D, PagedPlan* p) {
  if (B < 0 || N < 1 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || (D != 64 && D != 128)) return false;
  const int64_t G = Hq / Hkv, rows = N * G;
  if (rows > kPagedMostRows || rows > (int64_t{1} << 32) / G - kPgRowBlock) return false;
  p->block = paged_block(rows);
  p->RB = (rows + p->block - 1) / p->block;
  if (B * p->RB > INT32_MAX - 1) return false;
  p->off_first = align_up(size_t{2} * kPagedGridMost * p->block * (D + 2) * sizeof(float), kAlign);
  p->off_failed = p->off_first + align_up(kPagedGridMost * sizeof(int4), kAlign);
  p->off_plan = p->off_failed + align_up(kPagedGridMost * sizeof(uint32_t), kAlign);
  p->total = p->off_plan + align_up((static_cast<size_t>(B) * p->RB + 1) * sizeof(int32_t), kAlign);
  return true;
}

template <typename T, int D, bool kLanes>
cudaError_t launch_join(const PagedAttnArgs& a, cudaStream_t st) {
  const int grid = (a.grid - 1) * (a.R / kPgJoinRows) + (a.status ? a.B : 0);
  return grid ? launch(attn_paged_join_kernel<T, D, kLanes>, grid, kPgJoinThreads, 0, st, true, a) : cudaSuccess;
}

template <typename T, int D, int MT>
cudaError_t launch_cols(const CUtensorMap& k, const CUtensorMap& v, const PagedAttnArgs& a, cudaStream_t st) {
  using L = PgColLayout<D, MT>;
  const cudaError_t e = launch_smem<attn_paged_cols_kernel<T, D, MT>>(a.grid, L::kThreads, L::kBytes, L::kBytes, st, k, v, a);
  return e != cudaSuccess ? e : launch_join<T, D, false>(a, st);
}

template <typename T, int D, bool kVar>
cudaError_t launch_rows(const CUtensorMap& k, const CUtensorMap& v, const PagedAttnArgs& a, cudaStream_t st) {
  using L = PgRowLayout<D>;
  const cudaError_t e = launch_smem<attn_paged_rows_kernel<T, D, kVar>>(a.grid, kPgRowThreads, L::kBytes, L::kBytes, st, k, v, a);
  return e != cudaSuccess ? e : launch_join<T, D, true>(a, st);
}

template <typename T, int D>
cudaError_t launch_attention(const CUtensorMap& k, const CUtensorMap& v, const PagedAttnArgs& a, cudaStream_t st) {
  if (a.R == 16) return launch_cols<T, D, 1>(k, v, a, st);
  if (a.R == 32) return launch_cols<T, D, 2>(k, v, a, st);
  return a.cap != 0.f || a.slopes || !(a.coef > 0.f) ? launch_rows<T, D, true>(k, v, a, st) : launch_rows<T, D, false>(k, v, a, st);
}

}  // namespace

extern "C" {

sv_status spec_kv_append_rope(const sv_paged_cache* cache, int32_t dtype, const sv_rows* k_new, const sv_rows* v_new,
                              const sv_rows* q, int32_t B, int32_t N, int32_t Hq, const int32_t* seq_base,
                              const int32_t* parents, const int32_t* n_nodes, const float* inv_freq, int32_t rotary_dims,
                              int32_t interleaved, void* out_q, int32_t* out_len, int32_t* out_status, void* stream) {
  if (dtype != SV_BF16 && dtype != SV_F16) return SV_ERR_UNSUPPORTED_DTYPE;
  RopeArgs a;
  if (B < 0 || N < 1 || (parents && N > SV_MAX_TREE_NODES) || Hq < 0) return SV_ERR_INVALID_ARG;
  if (B == 0) return SV_OK;
  if (!view(cache, &a.c) || !valid_rows(k_new, 2) || !valid_rows(v_new, 2) || (q ? !valid_rows(q, 2) || Hq < 1 || !out_q : Hq != 0) ||
      !seq_base || !inv_freq || !out_len || rotary_dims < 16 || rotary_dims > cache->D || rotary_dims % 16 != 0 ||
      !aligned(seq_base, 4) || !aligned(parents, 4) || !aligned(n_nodes, 4) || !aligned(inv_freq, 4) || !aligned(out_q, 16) ||
      !aligned(out_len, 4) || !aligned(out_status, 4))
    return SV_ERR_INVALID_ARG;
  if (out_len == seq_base || out_len == n_nodes) return SV_ERR_INVALID_ARG;   // read by CTAs that start later
  const sv_rows* r[3] = {k_new, v_new, q};
  for (int i = 0; i < 3; ++i) {
    a.x[i] = r[i] ? static_cast<const uint8_t*>(r[i]->data) : nullptr;
    a.sb[i] = r[i] ? r[i]->stride_b * 2 : 0;
    a.sn[i] = r[i] ? r[i]->stride_n * 2 : 0;
    a.sh[i] = r[i] ? r[i]->stride_h * 2 : 0;
  }
  const int64_t heads = 2ll * cache->Hkv + Hq;
  if (heads > 16384) return SV_ERR_INVALID_ARG;   // a unit's row is exact
  a.q_out = static_cast<uint8_t*>(out_q);
  a.base = seq_base;
  a.n_nodes = n_nodes;
  a.parents = parents;
  a.inv_freq = inv_freq;
  a.out_len = out_len;
  a.status = out_status;
  a.B = B;
  a.N = N;
  a.Hq = Hq;
  a.rot = rotary_dims;
  a.interleaved = interleaved != 0;
  a.inv_heads = static_cast<uint32_t>(((1ll << 32) + heads - 1) / heads);
  // Rows a CTA: enough units for each thread to have kRopeBatch in flight (12297 rows of prompts take 52 us so, 57 with
  // twice and 67 with half as many), fewer where that would leave SMs without a CTA.
  const int64_t units = heads * (cache->D / 16);
  int64_t R = std::max<int64_t>(1, kRopeBatch * kRopeThreads / units);
  R = std::min<int64_t>({R, kRopeRows, N, std::max<int64_t>(1, static_cast<int64_t>(B) * N / (2 * sm_count()))});
  a.R = static_cast<int32_t>(R);
  a.blocks = static_cast<int32_t>((N + R - 1) / R);
  if (static_cast<int64_t>(B) * a.blocks > INT32_MAX) return SV_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int grid = B * a.blocks;
  const bool wide = cache->D == 128;
  return done(dtype == SV_BF16 ? (wide ? launch(kv_append_rope_kernel<TypeBf16, 128>, grid, kRopeThreads, 0, st, true, a)
                                       : launch(kv_append_rope_kernel<TypeBf16, 64>, grid, kRopeThreads, 0, st, true, a))
                               : (wide ? launch(kv_append_rope_kernel<TypeF16, 128>, grid, kRopeThreads, 0, st, true, a)
                                       : launch(kv_append_rope_kernel<TypeF16, 64>, grid, kRopeThreads, 0, st, true, a)));
}

size_t spec_attention_workspace_size(int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D) {
  PagedPlan p;
  return paged_plan(B, N, Hq, Hkv, D, &p) ? p.total : 0;
}

sv_status spec_attention(const sv_rows* q, int32_t dtype, const sv_paged_cache* cache, int32_t B, int32_t N, int32_t Hq,
                         const int32_t* seq_base, const int32_t* parents, const int32_t* n_nodes, float sm_scale, float softcap,
                         int32_t window, const float* slopes, void* out, float* out_lse, int32_t* out_status, void* workspace,
                         size_t workspace_bytes, void* stream) {
  if (dtype != SV_BF16 && dtype != SV_F16) return SV_ERR_UNSUPPORTED_DTYPE;
  if (B < 0 || N < 1 || (parents && N > SV_MAX_TREE_NODES) || !std::isfinite(sm_scale) || !std::isfinite(softcap) || softcap < 0.f ||
      window < 0)
    return SV_ERR_INVALID_ARG;
  if (B == 0) return SV_OK;
  PagedAttnArgs a;
  if (!view(cache, &a.c) || !valid_rows(q, 2) || !seq_base || !out || !workspace || !aligned(seq_base, 4) || !aligned(parents, 4) ||
      !aligned(n_nodes, 4) || !aligned(slopes, 4) || !aligned(out, 16) || !aligned(out_lse, 4) || !aligned(out_status, 4) ||
      !aligned(workspace, 16))
    return SV_ERR_INVALID_ARG;
  PagedPlan p;
  if (!paged_plan(B, N, Hq, cache->Hkv, cache->D, &p)) return SV_ERR_INVALID_ARG;
  if (workspace_bytes < p.total) return SV_ERR_WORKSPACE_TOO_SMALL;
  const double scale = static_cast<double>(sm_scale) * 1.4426950408889634;
  a.coef = static_cast<float>(softcap > 0.f ? 2.0 * scale / softcap : scale);
  a.cap = static_cast<float>(softcap * 1.4426950408889634);
  a.lin = static_cast<float>(scale);
  if (!std::isfinite(a.coef) || !std::isfinite(a.cap) || !std::isfinite(a.lin)) return SV_ERR_INVALID_ARG;
  a.q = static_cast<const uint8_t*>(q->data);
  a.sqb = q->stride_b * 2;
  a.sqn = q->stride_n * 2;
  a.sqh = q->stride_h * 2;
  a.base = seq_base;
  a.n_nodes = n_nodes;
  a.parents = parents;
  a.slopes = slopes;
  a.out = out;
  a.lse = out_lse;
  a.status = out_status;
  a.B = B;
  a.N = N;
  a.Hq = Hq;
  a.G = Hq / cache->Hkv;
  a.inv_g = ((1ull << 32) + a.G - 1) / a.G;
  a.R = p.block;
  a.RB = static_cast<int32_t>(p.RB);
  a.window = window ? window : INT32_MAX;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.part = reinterpret_cast<float*>(ws);
  a.first = reinterpret_cast<int4*>(ws + p.off_first);
  a.failed = reinterpret_cast<uint32_t*>(ws + p.off_failed);
  a.plan = reinterpret_cast<int32_t*>(ws + p.off_plan);
  const int64_t items = B * p.RB * cache->Hkv;
  const int64_t tiles = (static_cast<int64_t>(cache->max_pages) * cache->page_size + kPgTile - 1) / kPgTile;
  a.extra = p.block >= 128 ? kPagedRowExtra : kPagedColExtra;
  if (items > INT32_MAX / (tiles + a.extra) || static_cast<int64_t>(cache->max_pages) * cache->page_size + N > INT32_MAX - 255) return SV_ERR_INVALID_ARG;
  a.grid = static_cast<int32_t>(std::min<int64_t>({sm_count(), kPagedGridMost, items * (tiles + a.extra)}));
  CUtensorMap k, v;
  if (!page_map(*cache, a.c, 0, &k) || !page_map(*cache, a.c, 1, &v)) return SV_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool wide = cache->D == 128;
  return done(dtype == SV_BF16 ? (wide ? launch_attention<TypeBf16, 128>(k, v, a, st) : launch_attention<TypeBf16, 64>(k, v, a, st))
                               : (wide ? launch_attention<TypeF16, 128>(k, v, a, st) : launch_attention<TypeF16, 64>(k, v, a, st)));
}

}  // extern "C"
