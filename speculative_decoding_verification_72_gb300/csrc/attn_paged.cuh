// Attention of new rows over the 16-bit paged cache: what its kernels share.
//
// For row n of request b (slot base_b + n, position pos_n) and head h of group h / G:
//   z_j = sm q.k_j, under a cap z_j = cap tanh(z_j / cap), with a bias z_j - slope_h (pos_n - pos_j),
//   o = sum_j softmax(z)_j v_j, lse = ln sum_j exp z_j
// over the visible slots: every j < base, and j = base + m where m is n itself
// or an ancestor of n (parents given) or m <= n (a chain or a prompt); with a
// window, those of them with pos_n - pos_j < window. A row that sees nothing
// gets o = 0 and lse = -inf.
//
// The N G rows of one kv head share its keys and are packed as r = n G + g.
// Up to 32 are columns of a product with the tokens as its rows
// (attn_paged_cols.cuh, bound by memory); more are lanes, in blocks of 128 or 256
// (attn_paged_rows.cuh, bound by the tensor cores and the exponentials).
//
// Split. A block of rows has the 128-slot tiles from its window's start to its
// last visible slot. The tiles of all (request, block, kv head) items, each with
// `extra` places before its first for what its beginning and end cost, are one
// line, cut into equal ranges, one per CTA, so mixed lengths load every CTA
// alike. A range that holds only part of an item's tiles writes a partial (max,
// sum, unnormalised o) that attn_paged_join_kernel joins, in a fixed order.
//
// Non-finite values. A slot's values multiply weights of 0 in rows that do not
// see it, so a tile that not every row sees whole has infinities and NaN taken
// out of its V, noted, and put into the output of the rows that do see them.
#pragma once

#include <cuda.h>

#include "attn_q8.cuh"
#include "paged_common.cuh"
#include "tc_common.cuh"

namespace sv {

constexpr int kPgTile = 128;

struct PagedAttnArgs {
  const uint8_t* q;
  int64_t sqb, sqn, sqh;       // bytes: request, row, head
  PagedView c;
  const int32_t* base;         // [B]
  const int32_t* n_nodes;      // [B] or nullptr
  const int32_t* parents;      // [B, N] or nullptr (chain)
  const float* slopes;         // [Hq] or nullptr
  void* out;                   // [B, N, Hq, D]
  float* lse;                  // [B, N, Hq] or nullptr
  int32_t* status;             // [B] or nullptr
  int32_t B, N, G, Hq, R, RB;  // R: rows of a block, RB: blocks per kv head
  uint64_t inv_g;              // ceil(2^32 / G): r / G = r inv_g >> 32 for r G < 2^32
  float coef;                  // of q.k: sm log2(e), or 2 sm log2(e) / cap
  float cap;                   // cap log2(e), or 0
  float lin;                   // sm log2(e)
  int32_t window;              // 2^31 - 1 for none
  float* part;                 // [2 grid][R (D + 2)]
  int32_t* plan;               // [B RB + 1] places before the blocks, and in all, for one kv head
  int4* first;                 // [grid]: the first item a CTA has tiles of: place of its first tile, tiles, block (of B RB), head
  uint32_t* failed;            // [grid]: whether a wait of the CTA gave up
  int32_t grid, extra;
};

// A request's rows and length, clamped to the page table's capacity (out_status
// reports what was clamped).
struct PagedReq {
  int base, n, len;
};

__device__ __forceinline__ PagedReq paged_req(const PagedAttnArgs& a, int b) {
  PagedReq r;
  const int cap = a.c.max_pages << a.c.page_shift;
  r.base = a.base[b];
  r.n = a.n_nodes ? min(max(a.n_nodes[b], 0), a.N) : a.N;
  if (r.base < 0) r.base = r.n = 0;
  r.base = min(r.base, cap);
  r.len = r.n > cap - r.base ? cap : r.base + r.n;
  return r;
}

__device__ __forceinline__ int paged_node(const PagedAttnArgs& a, int r) {
  return static_cast<int>(static_cast<uint64_t>(r) * a.inv_g >> 32);
}

// What the rows of one block need: slots [first, end), from tile t on.
struct PagedSpan {
  int node0, first, end, clear, t, tiles;   // clear: every row of the block sees the slots below it (but for windows)
  __device__ __forceinline__ PagedSpan(const PagedAttnArgs& a, const PagedReq& r, int block) {
    node0 = paged_node(a, block * a.R);
    const int last = min(paged_node(a, block * a.R + a.R - 1), r.n - 1);
    end = last < node0 ? 0 : a.parents ? r.len : min(r.len, r.base + last + 1);
    clear = a.parents ? r.base : r.base + min(node0 + 1, r.n);
    first = min(max(r.base + (a.parents ? 0 : node0) - a.window + 1, 0), max(end - 1, 0));
    t = first / kPgTile;
    tiles = max(1, (end + kPgTile - 1) / kPgTile - t);
  }
  // Past every row's window start, as slots: tiles from here on need no mask of it.
  __device__ __forceinline__ int inside(const PagedAttnArgs& a, const PagedReq& r, int block) const {
    return r.base + (a.parents ? r.n - 1 : min(paged_node(a, block * a.R + a.R - 1), r.n - 1)) - a.window + 1;
  }
};

// A CTA's walk over its range of the line.
struct PagedCursor {
  int32_t pos, off;
  PagedReq rq;
  int b, block, tiles, h, t0, n, node0, end, clear, inside;   // the piece: tiles t0 .. t0 + n - 1 of item (b, block, h)
  bool whole, fresh;                                          // whole: the piece is all of its item

  __device__ __forceinline__ void start(const PagedAttnArgs& a, const AttnLine& line, int32_t lo) {
    pos = lo;
    off = line.off;
    b = line.b / a.RB;
    block = line.b - b * a.RB;
    n = 0;
    fresh = true;
  }
  // The next piece that has tiles, from place pos on; pos is then the place of its first tile, or at least hi if there is none.
  __device__ __forceinline__ void piece(const PagedAttnArgs& a, int32_t hi) {
    if (fresh) rq = paged_req(a, b);
    fresh = false;
    PagedSpan s(a, rq, block);
#pragma unroll 1
    while (pos >= (off + s.tiles + a.extra) * a.c.Hkv) {
      off += s.tiles + a.extra;
      if (++block == a.RB) {
        block = 0;
        rq = paged_req(a, ++b);
      }
      s = PagedSpan(a, rq, block);
    }
    tiles = s.tiles;
    const int rel = pos - off * a.c.Hkv, places = tiles + a.extra;
    h = rel / places;
    const int t = max(rel - h * places - a.extra, 0);
    pos = off * a.c.Hkv + h * places + a.extra + t;
    n = min(tiles - t, hi - pos);
    whole = n == tiles;
    t0 = s.t + t;
    node0 = s.node0;
    end = s.end;
    clear = s.clear;
    inside = s.inside(a, rq, block);
  }
  // Whether some row of the block does not see all of the tile from tok0 on, of whose pages `there` are there.
  __device__ __forceinline__ bool special(const PagedAttnArgs& a, int tok0, uint32_t there) const {
    return tok0 + kPgTile > clear || tok0 < inside || there != (1u << (kPgTile >> a.c.page_shift)) - 1u;
  }
  // Of the CTA's first piece.
  __device__ __forceinline__ int4 item(const PagedAttnArgs& a) const {
    return make_int4(off * a.c.Hkv + h * (tiles + a.extra) + a.extra, tiles, b * a.RB + block, h);
  }
};

// A warp's cursor, in shared memory, moved on to its next piece (`to` may be
// `from`). One copy of the code for all roles, which run at once and share the
// instruction cache.
__device__ __noinline__ void next_piece(const PagedAttnArgs& a, const PagedCursor* from, PagedCursor* to, int32_t hi) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    PagedCursor c = *from;
    c.pos += c.n;
    if (c.pos < hi) c.piece(a, hi);
    *to = c;
  }
  __syncwarp();
}

// The line for one CTA: every kernel's prologue. [lo, hi) of it is the CTA's.
template <int kThreads>
__device__ __forceinline__ void paged_line(const PagedAttnArgs& a, AttnLine* s_line, int32_t* s_warp, int32_t& lo, int32_t& hi) {
  const int cta = blockIdx.x;
  const AttnRanges ranges = attn_scan<kThreads>(
      a.B * a.RB,
      [&](int e) {
        const int b = e / a.RB;
        return PagedSpan(a, paged_req(a, b), e - b * a.RB).tiles + a.extra;
      },
      a.grid, cta, s_line, s_warp, a.c.Hkv, cta == 0 ? a.plan : nullptr);
  if (cta == 0 && threadIdx.x == 0) a.plan[a.B * a.RB] = s_line->total;
  lo = cta < ranges.n ? ranges.begin(cta) : 0;
  hi = cta < ranges.n ? ranges.begin(cta + 1) : 0;
  if (threadIdx.x == 0) a.first[cta] = make_int4(INT_MAX, 0, 0, 0);   // unless it has a piece
}

// Pages of a walk through one request, 32 a load: lane l has page 32 g + l of
// group g, and the next group is on its way.
struct PagedLook {
  int group, now, next;
  __device__ __forceinline__ static int at(const PagedAttnArgs& a, int b, int lp, int end) {
    return lp << a.c.page_shift < end ? paged_page(a.c, b, lp) : -1;
  }
  __device__ __forceinline__ void start(const PagedAttnArgs& a, int b, int lp, int end, int lane) {
    group = lp >> 5;
    now = at(a, b, group * 32 + lane, end);
    next = at(a, b, group * 32 + 32 + lane, end);
  }
  // Page lp (the lanes ask for pages of one tile, so of one group).
  __device__ __forceinline__ int page(const PagedAttnArgs& a, int b, int lp, int end, int lane) {
    const int g = __shfl_sync(0xffffffffu, lp, 0) >> 5;
    if (g != group) {
      group = g;
      now = next;
      next = at(a, b, g * 32 + 32 + lane, end);
    }
    return __shfl_sync(0xffffffffu, now, lp & 31);
  }
};

// From this cap on (in units of log2) its 2^-20, by which capped scores are off,
// would show in a weight: at 128 a score is off by 2^-13, a weight by half of what
// f16 rounds off of it.
constexpr float kPgFarCap = 128.f * kLog2e;

// Scores to cap tanh(z / cap) under a large cap: below a quarter of the cap by
// tanh u = u - u^3 / 3 + 2 u^5 / 15 - 17 u^7 / 315, to 2^-21 of itself. Rarely taken,
// so out of line, on a copy, and short.
template <int kN>
__device__ __noinline__ void far_caps(float* s, float coef, float cap, float lin) {
#pragma unroll 1
  for (int e = 0; e < kN; ++e) {
    const float t = s[e] * coef, u = t * (0.5f * kLn2), u2 = u * u;
    s[e] = fabsf(u) < 0.25f ? s[e] * lin * fmaf(u2, fmaf(u2, fmaf(u2, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.f)
                            : cap * fmaf(-2.f, 1.f / (1.f + ex2(t)), 1.f);
  }
}
template <int kN>
__device__ __forceinline__ void cap_far(uint32_t (&x)[kN], const PagedAttnArgs& a) {
  float y[kN];
#pragma unroll
  for (int e = 0; e < kN; ++e) y[e] = __uint_as_float(x[e]);
  far_caps<kN>(y, a.coef, a.cap, a.lin);
#pragma unroll
  for (int e = 0; e < kN; ++e) x[e] = __float_as_uint(y[e]);
}

// A score in units of log2, before mask and maximum, under no cap or one up to kPgFarCap.
__device__ __forceinline__ float paged_score(const PagedAttnArgs& a, float s) {
  s *= a.coef;
  if (a.cap == 0.f) return s;
  // cap tanh(z / cap) = cap (1 - 2 / (1 + e^(2 z / cap)))
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2(s)));
  return fmaf(-2.f * a.cap, r, a.cap);
}

// Whether any 16-bit element of a 16-byte piece of V is not finite: in the sign's
// places of the result, where an all-ones exponent carries to.
template <typename T>
__device__ __forceinline__ uint32_t nonfinite8(const uint4& w) {
  constexpr uint32_t e = T::kExpBits == 8 ? 0x7f807f80u : 0x7c007c00u, one = T::kExpBits == 8 ? 0x00800080u : 0x04000400u;
  return (((w.x & e) + one) | ((w.y & e) + one) | ((w.z & e) + one) | ((w.w & e) + one)) & 0x80008000u;
}

// Takes the values that are not finite out of a piece of V; what they were, as
// bits: NaN and +inf in the low byte, NaN and -inf in the next.
template <typename T>
__device__ __forceinline__ uint32_t take_out8(uint4* p) {
  constexpr uint32_t e = T::kExpBits == 8 ? 0x7f80u : 0x7c00u;
  uint16_t* v = reinterpret_cast<uint16_t*>(p);
  uint32_t r = 0;
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    const uint32_t x = v[i];
    if ((x & e) != e) continue;
    const bool nan = (x & 0x7fffu) != e;
    r |= (nan || !(x & 0x8000u) ? 1u : 0u) << i | (nan || (x & 0x8000u) ? 1u : 0u) << (8 + i);
    v[i] = 0;
  }
  return r;
}

// An element of the output and what was taken out of V in its column.
__device__ __forceinline__ float put_back(float o, bool pos, bool neg) {
  if (pos) o += INFINITY;
  if (neg) o -= INFINITY;
  return o;
}

// ------------------------------------------------------------------- join

constexpr int kPgJoinThreads = 128;
constexpr int kPgJoinRows = 16;        // rows a CTA
constexpr int kPgJoinBatch = 8;

// Joins the pieces of items that several CTAs shared (4 to 8 us, most of them the
// launch and two dependent reads); B more CTAs, before these, check the requests'
// pages, lengths and trees (128 pages at a time: one token after a million slots
// takes 614 us on pages of 128, 874 on pages of 16). A partial is o [R][D] with (max, sum)
// behind ([R][2]), or, where the lanes that wrote it were rows, o [D][R]: kLanes.
template <typename T, int D, bool kLanes>
__global__ void __launch_bounds__(kPgJoinThreads) attn_paged_join_kernel(const PagedAttnArgs a) {
  const int tid = threadIdx.x;
  grid_dep_wait();
  grid_dep_launch();
  const int groups = a.R / kPgJoinRows;
  const int total = a.plan[a.B * a.RB] * a.c.Hkv;
  const AttnRanges ranges(a.grid, total);
  const int join = static_cast<int>(blockIdx.x) - (a.status ? a.B : 0);
  if (join < 0) {
    const int b = blockIdx.x;
    const PagedReq rq = paged_req(a, b);
    bool bad_page = a.base[b] < 0 || (a.n_nodes && (a.n_nodes[b] < 0 || a.n_nodes[b] > a.N)) || rq.len - rq.n != a.base[b];
#pragma unroll 1
    for (int j = (rq.n > 0 ? max(rq.base - a.window + 1, 0) >> a.c.page_shift : INT_MAX / 2) + tid;
         j < (rq.len + (1 << a.c.page_shift) - 1) >> a.c.page_shift; j += kPgJoinThreads)
      bad_page = bad_page || paged_page(a.c, b, j) < 0;
    bool tree = false;
    if (a.parents)
#pragma unroll 1
      for (int n = tid; n < rq.n; n += kPgJoinThreads) tree = tree || bad_parent(a.parents[static_cast<int64_t>(b) * a.N + n], n);
    const int last = ranges.cta_of(a.plan[(b + 1) * a.RB] * a.c.Hkv - 1);
    bool late = false;
#pragma unroll 1
    for (int i = ranges.cta_of(a.plan[b * a.RB] * a.c.Hkv) + tid; i <= last; i += kPgJoinThreads) late = late || a.failed[i] != 0;
    bad_page = __syncthreads_or(bad_page);
    tree = __syncthreads_or(tree);
    late = __syncthreads_or(late);
    if (tid == 0)
      a.status[b] = (bad_page ? SV_STATUS_BAD_PAGE : 0) | (tree ? SV_STATUS_BAD_PARENT : 0) | (late ? SV_STATUS_TIMEOUT : 0);
    return;
  }
  // One group of CTAs a boundary between ranges; the first boundary within an item joins it.
  const int at = join / groups + 1;
  if (at >= ranges.n) return;
  const int4 item = a.first[at];
  if (ranges.begin(at) <= item.x) return;   // the CTA begins with its item, or has none
  const int t0 = item.x, e = item.z, h = item.w, c0 = ranges.cta_of(t0), c1 = ranges.cta_of(t0 + item.y - 1);
  if (at != c0 + 1) return;
  const int in_block = (join - (at - 1) * groups) * kPgJoinRows;
  const int b = e / a.RB, row0 = (e - b * a.RB) * a.R + in_block;   // of the kv head
  if (row0 >= a.N * a.G) return;
  const int slot0 = ranges.begin(c0) >= t0 - a.extra ? 0 : 1;   // of what came before the item it has the last tile
  auto partial = [&](int i) { return a.part + static_cast<int64_t>(2 * i + (i == c0 ? slot0 : 0)) * a.R * (D + 2); };

  // A thread has one row and D / 8 of its elements: 8 threads a row.
  constexpr int kPer = D / 8;
  __shared__ __align__(16) uint16_t s_o[kPgJoinRows][D + 8];
  const int r = kLanes ? tid % kPgJoinRows : tid >> 3, d0 = kLanes ? tid / kPgJoinRows * kPer : (tid & 7) * 4;
  const int row = in_block + r;
  float m = -INFINITY, l = 0.f, v[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) v[k] = 0.f;
  // Blocks of many rows are mostly in two pieces (taken two at a time trees need 99 us, four at a time 102), of few rows in many.
  constexpr int kBatch = kLanes ? 2 : D == 128 ? kPgJoinBatch / 2 : kPgJoinBatch;
#pragma unroll 1
  for (int i0 = c0; i0 <= c1; i0 += kBatch) {
    float2 ml[kBatch];
    float t[kBatch][kPer];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float* p = partial(min(i0 + k, c1));
      ml[k] = *reinterpret_cast<const float2*>(p + a.R * D + row * 2);
      if (kLanes) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) t[k][j] = p[(d0 + j) * a.R + row];
      } else {
#pragma unroll
        for (int j = 0; j < kPer; j += 4) {
          const float4 x = *reinterpret_cast<const float4*>(p + row * D + d0 + j * 8);
          t[k][j] = x.x;
          t[k][j + 1] = x.y;
          t[k][j + 2] = x.z;
          t[k][j + 3] = x.w;
        }
      }
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) top = i0 + k <= c1 ? fmaxf(top, ml[k].x) : top;
    const float top0 = top == -INFINITY ? 0.f : top, f0 = ex2(m - top0);
    l *= f0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) v[j] *= f0;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (i0 + k > c1) break;
      const float f = ex2(ml[k].x - top0);
      // Where a piece saw nothing of the row, o is 0 and so is the factor's product.
      l = fmaf(ml[k].y, f, l);
#pragma unroll
      for (int j = 0; j < kPer; ++j) v[j] = fmaf(t[k][j], f, v[j]);
    }
    m = top;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int j = 0; j < kPer; j += 2) {
    const int d = kLanes ? d0 + j : d0 + (j >> 2) * 32 + (j & 3);
    *reinterpret_cast<uint32_t*>(&s_o[r][d]) = T::pack2(v[j] * inv, v[j + 1] * inv);
  }
  const int R = row0 + r;
  if (a.lse && d0 == 0 && R < a.N * a.G) {
    const int n = paged_node(a, R);
    a.lse[(static_cast<int64_t>(b) * a.N + n) * a.Hq + h * a.G + (R - n * a.G)] =
        l == 0.f ? -INFINITY : ((m == -INFINITY ? 0.f : m) + log2f(l)) * kLn2;
  }
  __syncthreads();
#pragma unroll 1
  for (int i = tid; i < kPgJoinRows * (D / 8); i += kPgJoinThreads) {
    const int rr = i / (D / 8), ch = i % (D / 8), RR = row0 + rr;
    if (RR >= a.N * a.G) break;
    const int n = paged_node(a, RR);
    const int64_t at = (static_cast<int64_t>(b) * a.N + n) * a.Hq + h * a.G + (RR - n * a.G);
    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + at * D * 2 + ch * 16) = *reinterpret_cast<const uint4*>(&s_o[rr][ch * 8]);
  }
}

}  // namespace sv
