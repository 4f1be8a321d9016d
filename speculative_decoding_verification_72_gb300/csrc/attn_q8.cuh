// The verify pass's attention over the 8-bit paged cache: what its kernels share.
//
// For node n of request b (position base_b + n) and head h of group h / G:
//   s_j = sm_scale * q . (ck_j * ks), o = sum_j softmax(s)_j * (cv_j * vs), lse = ln sum_j exp s_j
// over the visible positions: every j < base, and j = base + m where m is n
// itself or an ancestor of n (parents given) or m <= n (a chain). A row that
// sees nothing gets o = 0 and lse = -inf.
//
// Rows. The N * G rows of one kv head share its keys, so they are packed as
// r = n * G + g: up to 32 of them are columns of one product
// (attn_q8_cols.cuh, bound by memory), more are blocks of 128 lanes
// (attn_q8_rows.cuh, bound by the tensor cores).
//
// Split. The work of all (request, kv head, row block) items is one line of
// 128-token tiles, cut into equal ranges, one per CTA, so mixed lengths load
// every CTA alike. A range that holds only part of an item writes a partial
// (max, sum, unnormalised o) that attn_q8_combine_kernel joins.
#pragma once

#include "q8_common.cuh"

namespace sv {

constexpr int kAttnThreads = 128;
constexpr int kAttnWarps = 4;

struct AttnArgs {
  const uint8_t* q;
  int64_t sqb, sqn, sqh;       // bytes: request, node, head
  Q8View c;
  const int32_t* base;         // [B]
  const int32_t* n_nodes;      // [B] or nullptr
  const int32_t* parents;      // [B, N] or nullptr (chain)
  void* out;                   // [B, N, Hq, D]
  float* lse;                  // [B, N, Hq] or nullptr
  int32_t* status;             // [B] or nullptr
  int32_t B, N, G, Hq, RB;     // RB: row blocks per kv head
  uint64_t inv_g;              // ceil(2^32 / G): r / G = r * inv_g >> 32 for r * G < 2^32
  float coef;                  // sm_scale * log2(e)
  float* part;                 // [2 grid][rows of a block][D + 4]: o, then (max, sum) in the pad
  int32_t* plan;               // [B + 1] tile offsets of the requests, and their total
  uint32_t* failed;            // [grid]: whether a wait of the CTA gave up, or nullptr
  int32_t grid;
};

struct AttnReq {
  int base, n, len;
};

__device__ __forceinline__ int attn_node(const AttnArgs& a, int r) {
  return static_cast<int>(static_cast<uint64_t>(r) * a.inv_g >> 32);
}

// Base, node count and length of a request, clamped to the page table's
// capacity (out_status reports what was clamped).
__device__ __forceinline__ AttnReq attn_req(const AttnArgs& a, int b) {
  AttnReq r;
  const int cap = a.c.max_pages << a.c.page_shift;
  r.base = a.base[b];
  r.n = a.n_nodes ? min(max(a.n_nodes[b], 0), a.N) : a.N;
  if (r.base < 0) r.base = r.n = 0;
  r.base = min(r.base, cap);
  r.len = min(r.base + r.n, cap);
  return r;
}

template <int kTile>
__device__ __forceinline__ int attn_tiles(const AttnReq& r) {
  return max(1, (r.len + kTile - 1) / kTile);
}

// The line of tiles: tiles_of(b) for each of ipr items of every request b. The
// entry point sees to it that it has fewer than 2^31.
struct AttnLine {
  int32_t total;   // tiles of all requests (one item each)
  int32_t off;     // tiles before request b
  int32_t b;
};

// Equal ranges of TT tiles for n CTAs, the first TT % n of them one longer.
struct AttnRanges {
  int32_t n, per, more;
  __device__ __forceinline__ AttnRanges(int32_t grid, int32_t TT) {
    n = TT < grid ? TT : grid;
    per = n > 0 ? TT / n : 0;
    more = TT - per * n;
  }
  __device__ __forceinline__ int32_t begin(int32_t cta) const { return cta * per + min(cta, more); }
  __device__ __forceinline__ int32_t cta_of(int32_t tile) const {   // tile < TT
    const int32_t first = more * (per + 1);
    return tile < first ? tile / (per + 1) : more + (tile - first) / per;
  }
};

// CTA-wide: sums the requests' tiles, and finds the request that holds the
// first tile of the CTA's range; offsets go to `store` if given. The result is
// in shared memory.
template <int kThreads, typename F>
__device__ __forceinline__ AttnRanges attn_scan(int B, F&& tiles_of, int32_t grid, int32_t cta, AttnLine* s_line, int32_t* s_warp,
                                                int32_t ipr, int32_t* store) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t run = 0, off = 0, t = 0, total = 0;
  AttnRanges ranges(grid, 0);
  // One chunk of kThreads requests serves both passes; more take each again.
  const int chunks = (B + kThreads - 1) / kThreads;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
      if (pass == 0 || chunks > 1) {
        const int b = c * kThreads + tid;
        t = b < B ? tiles_of(b) : 0;
        int32_t inc = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int32_t up = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += up;
        }
        __syncthreads();
        if (lane == 31) s_warp[warp] = inc;
        __syncthreads();
        off = run + inc - t;
#pragma unroll 1
        for (int w = 0; w < kThreads / 32; ++w) {
          const int32_t s = s_warp[w];
          if (w < warp) off += s;
          run += s;
        }
        if (store && pass == 0 && b < B) store[b] = off;
      }
      if (pass == 1) {
        const int32_t find = ranges.begin(cta);
        if (c * kThreads + tid < B && off * ipr <= find && find < (off + t) * ipr) {
          s_line->off = off;
          s_line->b = c * kThreads + tid;
        }
      }
    }
    if (pass == 0) {
      total = run;
      run = 0;
      ranges = AttnRanges(grid, total * ipr);
    }
  }
  if (tid == 0) s_line->total = total;
  __syncthreads();
  return ranges;
}

// A CTA's walk over its range of the line: the pieces of items it has.
struct AttnCursor {
  int32_t pos, off;
  AttnReq rq;
  int b, tiles, h, rb, t0, n;   // request, its tiles, kv head, row block, first tile and tiles of the piece

  __device__ __forceinline__ void start(const AttnArgs& a, const AttnLine& line, int32_t lo) {
    pos = lo;
    off = line.off;
    b = line.b;
    n = 0;
  }
  // The next piece (called while pos + n < hi); pos is then its first tile.
  template <int kTile>
  __device__ __forceinline__ void piece(const AttnArgs& a, int32_t hi, int ipr) {
    rq = attn_req(a, b);
    tiles = attn_tiles<kTile>(rq);
    while (pos >= (off + tiles) * ipr) {
      off += tiles;
      rq = attn_req(a, ++b);
      tiles = attn_tiles<kTile>(rq);
    }
    const int rel = pos - off * ipr;
    const int item = rel / tiles;
    t0 = rel - item * tiles;
    n = min(tiles - t0, hi - pos);
    h = item / a.RB;
    rb = item - h * a.RB;
  }
};

template <int D>
struct AttnLayout {
  static constexpr int kPitch = D + 4;   // floats per row of a partial: o, then (max, sum)
};

// Byte offset of 16-byte chunk ch of token row `row` within a unit.
template <int D>
__device__ __forceinline__ uint32_t unit_off(int row, int ch) {
  if (D == 128) return row * 128 + ((ch ^ (row & 7)) << 4);
  return row * 64 + ((ch ^ ((row >> 1) & 3)) << 4);
}

// V's scale as an exponent counts it, for a warp whose lanes hold pages' scales
// (there: whether the lane has a page). A page of zeros has scale 2^-100, or 0 if
// it was never written: as an exponent that far below the others the weights of
// its positions would fall out of fp32's range. It counts as 2^60 below the
// largest scale so far (`most`, a lane's own, kept by the caller), or as 2^-100;
// codes that are not zero under such a scale add less than 2^-51 of that scale.
__device__ __forceinline__ float attn_v_scale(float vs, bool there, float& most) {
  most = fmaxf(most, vs);
  const bool zeros = there && vs >= 0.f && vs <= 0x1p-100f;
  if (__any_sync(0xffffffffu, zeros)) {
    const float m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
    if (zeros) vs = fmaxf(0x1p-100f, fminf(m, 0x1p126f) * 0x1p-60f);
  }
  return vs;
}

// A partial's (max, sum) for the join, its sum brought into [1, 2): the exponent
// goes into the maximum and out of `f`, the factor of o. A piece's own maximum
// counts V's scales relative to its first page, so the maxima of two pieces may
// lie further apart than fp32's exponents reach where their weights do not (a
// page of zeros has scale 2^-100).
__device__ __forceinline__ float2 attn_partial(float m, float l, float& f) {
  if (l == 0.f) return make_float2(-INFINITY, 0.f);
  const int e = min(max(static_cast<int>(__float_as_uint(l) >> 23) - 127, -126), 126);
  const float down = exp2_int(-e);
  f *= down;
  return make_float2(m + static_cast<float>(e), l * down);
}

// Joins the pieces of items that several CTAs shared, one warp a row; B more
// CTAs check the requests' pages, lengths and trees. All loads of a row's first
// eight pieces go out together, after one for the plan.
constexpr int kJoinBatch = 8;

template <typename T, int D, int MT>
__global__ void __launch_bounds__(kAttnThreads) attn_q8_combine_kernel(const AttnArgs a) {
  constexpr int kRows = 16 * MT, kPitch = AttnLayout<D>::kPitch;
  constexpr int kV = D / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ipr = a.c.Hkv * a.RB;
  grid_dep_wait();
  grid_dep_launch();
  const int join = static_cast<int>(blockIdx.x) - (a.status ? a.B : 0);
  const bool check = join < 0;
  const int b = check ? blockIdx.x : join / (kRows / 4) / ipr;
  const int off = a.plan[b], total = a.plan[a.B], next = a.plan[b + 1], tiles = next - off;
  const AttnRanges ranges(a.grid, total * ipr);
  if (check) {
    const AttnReq rq = attn_req(a, b);
    bool bad_page = a.base[b] < 0 || (a.n_nodes && (a.n_nodes[b] < 0 || a.n_nodes[b] > a.N)) || rq.len != a.base[b] + rq.n;
    for (int j = tid; j < (rq.len + (1 << a.c.page_shift) - 1) >> a.c.page_shift; j += kAttnThreads)
      bad_page = bad_page || q8_page(a.c, b, j) < 0;
    bool bad_parent = false;
    if (a.parents)
      for (int n = tid; n < rq.n; n += kAttnThreads) {
        const int p = a.parents[static_cast<int64_t>(b) * a.N + n];
        bad_parent = bad_parent || (n == 0 ? p != -1 : p < 0 || p >= n);
      }
    bool late = false;
    if (a.failed) {
      const int last = ranges.cta_of(next * ipr - 1);
      for (int i = ranges.cta_of(off * ipr) + tid; i <= last; i += kAttnThreads) late = late || a.failed[i] != 0;
    }
    bad_page = __syncthreads_or(bad_page);
    bad_parent = __syncthreads_or(bad_parent);
    late = __syncthreads_or(late);
    if (tid == 0)
      a.status[b] = (bad_page ? SV_STATUS_BAD_PAGE : 0) | (bad_parent ? SV_STATUS_BAD_PARENT : 0) | (late ? SV_STATUS_TIMEOUT : 0);
    return;
  }
  const int item = join / (kRows / 4) - b * ipr;
  const int t0 = off * ipr + item * tiles;
  const int c0 = ranges.cta_of(t0), c1 = ranges.cta_of(t0 + tiles - 1);
  if (c0 == c1) return;   // one CTA had all of it
  const int h = item / a.RB, rb = item - h * a.RB;
  const int slot0 = ranges.begin(c0) == t0 ? 0 : 1;
  const int r = join % (kRows / 4) * 4 + warp, R = rb * kRows + r;
  if (R >= a.N * a.G) return;
  float m = -INFINITY, l = 0.f, v[kV];
#pragma unroll
  for (int k = 0; k < kV; ++k) v[k] = 0.f;
  for (int i0 = c0; i0 <= c1; i0 += kJoinBatch) {
    float2 ml[kJoinBatch];
    float t[kJoinBatch][kV];
#pragma unroll
    for (int k = 0; k < kJoinBatch; ++k) {
      const int i = min(i0 + k, c1);
      const float* p = a.part + static_cast<int64_t>((2 * i + (i == c0 ? slot0 : 0)) * kRows + r) * kPitch;
      ml[k] = *reinterpret_cast<const float2*>(p + D);
      if (kV == 4) {
        const float4 x = *reinterpret_cast<const float4*>(p + lane * 4);
        t[k][0] = x.x;
        t[k][1] = x.y;
        t[k][2 % kV] = x.z;
        t[k][3 % kV] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(p + lane * 2);
        t[k][0] = x.x;
        t[k][1] = x.y;
      }
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < kJoinBatch; ++k) top = i0 + k <= c1 ? fmaxf(top, ml[k].x) : top;
    const float top0 = top == -INFINITY ? 0.f : top;
    const float f0 = ex2(m - top0);
    l *= f0;
#pragma unroll
    for (int e = 0; e < kV; ++e) v[e] *= f0;
#pragma unroll
    for (int k = 0; k < kJoinBatch; ++k) {
      const float f = ex2(ml[k].x - top0);
      if (i0 + k <= c1) {
        l = fmaf(ml[k].y, f, l);
#pragma unroll
        for (int e = 0; e < kV; ++e) v[e] = fmaf(t[k][e], f, v[e]);
      }
    }
    m = top;
  }
  const float m0 = m == -INFINITY ? 0.f : m;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int n = attn_node(a, R);
  const int64_t row = (static_cast<int64_t>(b) * a.N + n) * a.Hq + h * a.G + (R - n * a.G);
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.out) + row * D * 2) + lane * (kV / 2);
  dst[0] = T::pack2(v[0] * inv, v[1] * inv);
  if (kV == 4) dst[1] = T::pack2(v[2 % kV] * inv, v[3 % kV] * inv);
  if (a.lse && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (m0 + log2f(l)) * kLn2;
}

}  // namespace sv
