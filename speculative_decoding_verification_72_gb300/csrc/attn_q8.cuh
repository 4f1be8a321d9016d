// The verify pass's attention over the 8-bit paged cache.
//
// For node n of request b (position base_b + n) and head h of group h / G:
//   s_j = sm_scale * q . (ck_j * ks), o = sum_j softmax(s)_j * (cv_j * vs), lse = ln sum_j exp s_j
// over the visible positions: every j < base, and j = base + m where m is n
// itself or an ancestor of n (parents given) or m <= n (a chain). A row that
// sees nothing gets o = 0 and lse = -inf.
//
// Rows. The N * G rows of one kv head share its keys, so they are packed as
// r = n * G + g and taken in blocks of 16 * MT.
//
// Split. The work of all (request, kv head, row block) items is one line of
// 64-token tiles, cut into equal ranges, one per CTA, so mixed lengths load
// every CTA alike. A range that holds only part of an item writes a partial
// (max, sum, unnormalised o) that attn_q8_combine_kernel joins.
//
// One pass per range: running maximum and sum per row (fp32), o in registers
// (fp32), keys and values read once. Each warp takes 16 tokens of a tile on
// its own: its 4 KB of codes arrive by cp.async in a ring private to the warp,
// and are turned into f16 fragments in registers. e4m3 to f16 is exact; q is
// scaled per row by a power of two so that bf16 fits f16 exactly; so the
// scores are exact products summed in fp32. P is rounded to f16 (relative
// 2^-11, like the f16 output it feeds and finer than bf16), values are exact.
//
// Layout of the fragments. m16n8k16 leaves the order of k free as long as A
// and B agree. For S = Q K^T lane quad c takes d in [c D/4, (c+1) D/4), so a
// token's codes are 32 contiguous bytes per lane (D = 128). For O = P V the
// rows of a k step are native, and lane group g takes the n columns
// d = (D/8) g + j of n-tile j: 16 contiguous bytes of a token, two byte
// permutes pairing two tokens' codes. Shared rows are swizzled (16-byte chunk
// index xor row) so both patterns are free of bank conflicts at D = 128.
//
// Scales. A 16-token unit lies in one page, so ks and vs are uniform in the
// warp: ks joins the softmax coefficient, vs multiplies p relative to the
// largest |vs| so far (P stays within f16's range), o is rescaled when that
// grows. The row maximum is raised only when a score exceeds it by 2^8 (P and
// its sum stay far inside f16's and fp32's range), so most units need neither
// a maximum across lanes nor a rescale.
#pragma once

#include "q8_common.cuh"

namespace sv {

constexpr int kAttnThreads = 128;
constexpr int kAttnWarps = 4;
constexpr int kAttnTile = 64;        // tokens per CTA step: 16 per warp
constexpr int kAttnStages = 4;
constexpr float kAttnSlack = 8.f;    // log2 by which a score may exceed the running maximum

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
  float* part;                 // [2 grid][16 MT][D + 4]: o, then (max, sum) in the pad
  int64_t* plan;               // [B + 1] tile offsets of the requests, then the CTAs in use
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

// The line of tiles: tiles_of(b) for each of ipr items of every request b.
struct AttnLine {
  int64_t total;   // tiles of all requests (one item each)
  int64_t off;     // tiles before request b
  int32_t b;
};

// CTA-wide: sums the requests' tiles, and finds the request that holds the
// first tile of the CTA's range, first_of(total); offsets go to `store` if given.
// The result is in shared memory.
template <int kThreads, typename F, typename G>
__device__ __forceinline__ void attn_scan(int B, F&& tiles_of, G&& first_of, AttnLine* s_line, int64_t* s_warp, int64_t ipr,
                                          int64_t* store) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t run = 0, off = 0;
  int32_t t = 0;
  auto chunk = [&](int c0) {   // off, t: of request c0 + tid
    const int b = c0 + tid;
    t = b < B ? tiles_of(b) : 0;
    int64_t inc = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    off = run + inc - t;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) off += s_warp[w];
      run += s_warp[w];
    }
    if (store && b < B) store[b] = off;
  };
  for (int c0 = 0; c0 < B; c0 += kThreads) chunk(c0);
  const int64_t total = run, find = first_of(total);
  for (int c0 = 0; c0 < B; c0 += kThreads) {
    if (B > kThreads) {   // more requests than threads: the chunks again
      if (c0 == 0) run = 0;
      chunk(c0);
    }
    if (c0 + tid < B && off * ipr <= find && find < (off + t) * ipr) {
      s_line->off = off;
      s_line->b = c0 + tid;
    }
  }
  if (tid == 0) s_line->total = total;
  __syncthreads();
}

// CTAs that share TT tiles: all of the grid, or one per tile.
__device__ __forceinline__ int64_t attn_ctas(int64_t grid, int64_t TT) { return TT < grid ? TT : grid; }

// A CTA's walk over its range of the line: the pieces of items it has.
struct AttnCursor {
  int64_t pos, off;
  AttnReq rq;
  int b, tiles, h, rb, t0, n;   // request, its tiles, kv head, row block, first tile and tiles of the piece

  __device__ void start(const AttnArgs& a, const AttnLine& line, int64_t lo) {
    pos = lo;
    off = line.off;
    b = line.b;
    n = 0;
  }
  // The next piece (called while pos + n < hi); pos is then its first tile.
  template <int kTile>
  __device__ void piece(const AttnArgs& a, int64_t hi, int ipr) {
    rq = attn_req(a, b);
    tiles = attn_tiles<kTile>(rq);
    while (pos >= (off + tiles) * ipr) {
      off += tiles;
      rq = attn_req(a, ++b);
      tiles = attn_tiles<kTile>(rq);
    }
    const int rel = static_cast<int>(pos - off * ipr);
    const int item = rel / tiles;
    t0 = rel - item * tiles;
    n = static_cast<int>(min(static_cast<int64_t>(tiles - t0), hi - pos));
    h = item / a.RB;
    rb = item - h * a.RB;
  }
};

template <int D>
struct AttnLayout {
  static constexpr int kUnitBytes = 16 * D;             // 16 tokens of K or V
  static constexpr int kStageBytes = 2 * kUnitBytes;
  static constexpr int kRingBytes = kAttnWarps * kAttnStages * kStageBytes;
  static constexpr int kPitch = D + 4;                  // floats per row of the merge buffer
};

// The ring, and over it the buffer that joins the warps' rows.
template <int D, int MT>
__host__ __device__ constexpr int attn_buf_bytes() {
  constexpr int merge = kAttnWarps * 16 * MT * AttnLayout<D>::kPitch * 4;
  return merge > AttnLayout<D>::kRingBytes ? merge : AttnLayout<D>::kRingBytes;
}
template <int D, int MT>
constexpr int attn_smem_bytes(int N) {
  return attn_buf_bytes<D, MT>() + MT * (D / 16) * 512 + 16 * MT * 4 + kAttnWarps * 16 * MT * 8 + 16 * MT * ((N + 31) / 32) * 4;
}

// Byte offset of 16-byte chunk ch of token row `row` within a unit.
template <int D>
__device__ __forceinline__ uint32_t unit_off(int row, int ch) {
  if (D == 128) return row * 128 + ((ch ^ (row & 7)) << 4);
  return row * 64 + ((ch ^ ((row >> 1) & 3)) << 4);
}

// Q rows of a row block as A fragments of the permuted S product: per m-tile
// and k step, 16 bytes a lane. Row r's factor (a power of two) goes to s_qs.
template <typename T, int D, int MT, int TH>
__device__ __forceinline__ void load_q_frags(const uint8_t* q, int64_t sqn, int64_t sqh, int rows_total, int row0, int G,
                                             const int32_t* node_of, int n_lim, uint32_t* s_q, float* s_qs) {
  constexpr int kKs = D / 16, kDpc = D / 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int rr = 0; rr < 16 * MT; rr += TH / 32) {
    const int r = rr + warp;
    const int R = row0 + r;
    float f[4] = {0.f, 0.f, 0.f, 0.f};
    const int d0 = lane * 4;
    if (R < rows_total && d0 < D) {
      int n = R / G;
      const int g = R - n * G;
      if (node_of) n = node_of[n];
      if (n >= 0 && n < n_lim) T::load4(q + n * sqn + g * sqh + d0 * 2, f);
    }
    float m = fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3])));
    m = warp_max(m);
    // 2^x that brings the row's maximum into [2^14, 2^15)
    const int e = m > 0.f ? static_cast<int>(__float_as_uint(m) >> 23) - 127 : 14;
    const int x = min(max(14 - e, -126), 126);
    const float up = exp2_int(x);
    if (d0 < D) {
      const int c = d0 / kDpc, ks = (d0 % kDpc) / 4, mt = r >> 4, hi = (r >> 3) & 1;
      uint32_t* dst = s_q + (((mt * kKs + ks) * 32 + (r & 7) * 4 + c) << 2) + hi;
      dst[0] = pack_half2(f[0] * up, f[1] * up);
      dst[2] = pack_half2(f[2] * up, f[3] * up);
    }
    if (lane == 0) s_qs[r] = exp2_int(-x);
  }
}

// S of 16 tokens (two n-tiles) for MT m-tiles from a unit of K codes in shared memory.
template <int D, int MT>
__device__ __forceinline__ void unit_scores(uint32_t k_unit, const uint4* s_q, int lane, float (&s)[MT][2][4]) {
  constexpr int kKs = D / 16;
  const int g = lane >> 2, c = lane & 3;
  uint32_t kw[2][kKs];
#pragma unroll
  for (int nt = 0; nt < 2; ++nt) {
    const int row = nt * 8 + g;
    if (D == 128) {
      const uint4 x = lds128(k_unit + unit_off<D>(row, 2 * c)), y = lds128(k_unit + unit_off<D>(row, 2 * c + 1));
      kw[nt][0] = x.x; kw[nt][1] = x.y; kw[nt][2] = x.z; kw[nt][3] = x.w;
      kw[nt][4 % kKs] = y.x; kw[nt][5 % kKs] = y.y; kw[nt][6 % kKs] = y.z; kw[nt][7 % kKs] = y.w;
    } else {
      const uint4 x = lds128(k_unit + unit_off<D>(row, c));
      kw[nt][0] = x.x; kw[nt][1] = x.y; kw[nt][2] = x.z; kw[nt][3] = x.w;
    }
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[mt][nt][i] = 0.f;
#pragma unroll
  for (int ks = 0; ks < kKs; ++ks) {
    uint32_t b[2][2];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      b[nt][0] = e4m3x2_lo(kw[nt][ks]);
      b[nt][1] = e4m3x2_hi(kw[nt][ks]);
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const uint4 qa = s_q[(mt * kKs + ks) * 32 + lane];
      mma_f16(s[mt][0], qa, b[0][0], b[0][1]);
      mma_f16(s[mt][1], qa, b[1][0], b[1][1]);
    }
  }
}

__device__ __forceinline__ uint32_t nan_ones(uint32_t h2) {   // f16x2: 1 where NaN, else 0
  return ((h2 & 0x7fffu) > 0x7c00u ? 0x3c00u : 0u) | ((h2 >> 16 & 0x7fffu) > 0x7c00u ? 0x3c000000u : 0u);
}
__device__ __forceinline__ uint32_t nan_zero(uint32_t h2) {   // f16x2: 0 where NaN
  return ((h2 & 0x7fffu) > 0x7c00u ? 0u : h2 & 0xffffu) | ((h2 >> 16 & 0x7fffu) > 0x7c00u ? 0u : h2 & 0xffff0000u);
}

template <typename T, int D, int MT>
__global__ void __launch_bounds__(kAttnThreads, MT == 1 ? 3 : 2) attn_q8_kernel(const AttnArgs a) {
  using L = AttnLayout<D>;
  constexpr int kKs = D / 16;
  constexpr int kRows = 16 * MT;
  constexpr int kNt = D / 8;                 // n-tiles of O
  constexpr int kChunks = 16 * (D / 16);     // 16-byte chunks per unit of K or V
  extern __shared__ __align__(128) uint8_t smem[];
  uint4* s_q = reinterpret_cast<uint4*>(smem + attn_buf_bytes<D, MT>());         // MT * kKs * 32
  float* s_qs = reinterpret_cast<float*>(s_q + MT * kKs * 32);                 // kRows
  float2* s_ml = reinterpret_cast<float2*>(s_qs + kRows);                      // [warps][kRows]
  uint32_t* s_anc = reinterpret_cast<uint32_t*>(s_ml + kAttnWarps * kRows);    // [nodes of the block][words]
  __shared__ AttnLine s_line;
  __shared__ int64_t s_warp[kAttnWarps];
  float* s_o = reinterpret_cast<float*>(smem);                                 // merge buffer over the ring

  grid_dep_wait();
  grid_dep_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int ipr = a.c.Hkv * a.RB;            // items per request
  const int cta = blockIdx.x;
  attn_scan<kAttnThreads>(
      a.B, [&](int r) { return attn_tiles<kAttnTile>(attn_req(a, r)); },
      [&](int64_t total) { return total * ipr * cta / attn_ctas(a.grid, total * ipr); }, &s_line, s_warp, ipr,
      cta == 0 ? a.plan : nullptr);
  const int64_t TT = s_line.total * ipr;
  const int64_t Ge = attn_ctas(a.grid, TT);
  if (cta == 0 && tid == 0) {
    a.plan[a.B] = s_line.total;
    a.plan[a.B + 1] = Ge;
  }
  if (cta >= Ge) return;
  const int64_t lo = TT * cta / Ge, hi = TT * (cta + 1) / Ge;
  const uint32_t ring = smem_u32(smem) + warp * (kAttnStages * L::kStageBytes);

  AttnCursor cur;
  for (cur.start(a, s_line, lo); cur.pos < hi; cur.pos += cur.n) {
    cur.piece<kAttnTile>(a, hi, ipr);
    const AttnReq rq = cur.rq;
    const int b = cur.b, h = cur.h, t0 = cur.t0, nt_ = cur.n, tiles = cur.tiles;
    const int64_t pos = cur.pos;
    const int row0 = cur.rb * kRows;
    const int rows_total = a.N * a.G, words = (a.N + 31) / 32;

    // ---- page ids and scales of 32 units at a time, one per lane
    int pid = -1, pid_n = -1;
    float ksv = 0.f, vsv = 0.f, ks_n = 0.f, vs_n = 0.f;
    auto fetch = [&](int i0, int& p, float& k_, float& v_) {
      const int tok = (t0 + i0 + lane) * kAttnTile + warp * 16;
      p = i0 + lane < nt_ && tok < rq.len ? q8_page(a.c, b, tok >> a.c.page_shift) : -1;
      k_ = v_ = 0.f;
      if (p >= 0) {
        const int64_t o = static_cast<int64_t>(p) * a.c.Hkv + h;
        k_ = a.c.ks[o];
        v_ = a.c.vs[o];
      }
    };
    auto issue = [&](int i, int page) {
      if (i < nt_) {
        const int tok = (t0 + i) * kAttnTile + warp * 16;
        const int valid = page < 0 ? 0 : rq.len - tok;
        const int64_t o =
            (((static_cast<int64_t>(max(page, 0)) * a.c.Hkv + h) << a.c.page_shift) + (tok & ((1 << a.c.page_shift) - 1))) * D;
        const uint32_t dst = ring + (i % kAttnStages) * L::kStageBytes;
#pragma unroll
        for (int it = 0; it < kChunks / 32; ++it) {
          const int ch = it * 32 + lane;
          const int row = ch / (D / 16), col = ch % (D / 16);
          const uint32_t to = dst + unit_off<D>(row, col);
          cp_async16(to, a.c.k + o + ch * 16, row < valid);
          cp_async16(to + L::kUnitBytes, a.c.v + o + ch * 16, row < valid);
        }
      }
      cp_async_commit();
    };
    fetch(0, pid, ksv, vsv);
    if (nt_ > 32) fetch(32, pid_n, ks_n, vs_n);
#pragma unroll
    for (int i = 0; i < kAttnStages - 1; ++i) issue(i, __shfl_sync(0xffffffffu, pid, i));

    // ---- the row block's queries and its nodes' ancestor sets
    load_q_frags<T, D, MT, kAttnThreads>(a.q + b * a.sqb + static_cast<int64_t>(h) * a.G * a.sqh, a.sqn, a.sqh, rows_total,
                                         row0, a.G, nullptr, rq.n, reinterpret_cast<uint32_t*>(s_q), s_qs);
    const int node0 = row0 / a.G;
    const bool tail = (t0 + nt_) * kAttnTile > rq.base;
    if (tail && a.parents) {
      const int nodes = min((row0 + kRows - 1) / a.G, a.N - 1) - node0 + 1;
      for (int i = tid; i < nodes * words; i += kAttnThreads) s_anc[i] = 0;
      __syncthreads();
      const int32_t* par = a.parents + static_cast<int64_t>(b) * a.N;
      for (int i = tid; i < nodes; i += kAttnThreads) {
        int n = node0 + i;
        while (n >= 0) {
          s_anc[i * words + (n >> 5)] |= 1u << (n & 31);
          const int up = par[n];
          n = up < n ? up : -1;   // a parent precedes its child; anything else ends the path
        }
      }
    }
    __syncthreads();

    float o[MT][kNt][4];
    float m_run[MT][2], l_run[MT][2], cq[MT][2];
    int node[MT][2];
    float ref = 1e-30f;   // largest |vs| so far
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int j = 0; j < kNt; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[mt][j][i] = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = mt * 16 + i * 8 + g;
        m_run[mt][i] = -INFINITY;
        l_run[mt][i] = 0.f;
        cq[mt][i] = s_qs[r] * a.coef;
        const int R = row0 + r;
        node[mt][i] = R < rows_total && R / a.G < rq.n ? R / a.G : -1;
      }
    }

    for (int i = 0; i < nt_; ++i) {
      const int page = __shfl_sync(0xffffffffu, pid, i & 31);
      const float ks = __shfl_sync(0xffffffffu, ksv, i & 31), vs = __shfl_sync(0xffffffffu, vsv, i & 31);
      cp_async_wait<kAttnStages - 2>();
      __syncwarp();
      // The slot of unit i - 1 is free now; fill it.
      {
        const int j = i + kAttnStages - 1;
        const int pj = __shfl_sync(0xffffffffu, (j ^ i) & ~31 ? pid_n : pid, j & 31);
        issue(j, pj);
      }
      if ((i & 31) == 31) {
        pid = pid_n;
        ksv = ks_n;
        vsv = vs_n;
        fetch(i + 33, pid_n, ks_n, vs_n);
      }
      if (page < 0) continue;   // past the end, or a page that is not there
      const uint32_t k_unit = ring + (i % kAttnStages) * L::kStageBytes, v_unit = k_unit + L::kUnitBytes;
      float s[MT][2][4];
      unit_scores<D, MT>(k_unit, s_q, lane, s);
      const int tok = (t0 + i) * kAttnTile + warp * 16;
      const bool edge = tok + 16 > rq.base;   // holds new nodes or the end
      bool raise = false;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x = s[mt][nt][e] * (cq[mt][e >> 1] * ks);
            if (edge) {
              const int m = tok + nt * 8 + 2 * c + (e & 1) - rq.base;
              const int n = node[mt][e >> 1];
              bool see = n >= 0 && m < rq.n;
              if (see && m >= 0) {
                see = m <= n;
                if (see && a.parents) see = s_anc[(n - node0) * words + (m >> 5)] >> (m & 31) & 1;
              }
              if (!see) x = -INFINITY;
            } else if (node[mt][e >> 1] < 0) {
              x = -INFINITY;
            }
            s[mt][nt][e] = x;
            raise = raise || x > m_run[mt][e >> 1] + kAttnSlack;
          }
      const float av = fabsf(vs);
      if (__any_sync(0xffffffffu, raise || av > ref)) {
        const float ref_new = fmaxf(ref, av);
        const float fr = ref / ref_new;
        ref = ref_new;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i2 = 0; i2 < 2; ++i2) {
            float mx = fmaxf(fmaxf(s[mt][0][2 * i2], s[mt][0][2 * i2 + 1]), fmaxf(s[mt][1][2 * i2], s[mt][1][2 * i2 + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            mx = fmaxf(mx, m_run[mt][i2]);
            const float f = m_run[mt][i2] == -INFINITY ? 0.f : ex2(m_run[mt][i2] - mx);
            m_run[mt][i2] = mx;
            l_run[mt][i2] *= f;
#pragma unroll
            for (int j = 0; j < kNt; ++j) {
              o[mt][j][2 * i2] *= f * fr;
              o[mt][j][2 * i2 + 1] *= f * fr;
            }
          }
      }
      const float vr = vs / ref;
      uint4 pa[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float p[2][4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float m = m_run[mt][e >> 1];
            p[nt][e] = ex2(s[mt][nt][e] - (m == -INFINITY ? 0.f : m));
            l_run[mt][e >> 1] += p[nt][e];
          }
        pa[mt].x = pack_half2(p[0][0] * vr, p[0][1] * vr);
        pa[mt].y = pack_half2(p[0][2] * vr, p[0][3] * vr);
        pa[mt].z = pack_half2(p[1][0] * vr, p[1][1] * vr);
        pa[mt].w = pack_half2(p[1][2] * vr, p[1][3] * vr);
      }
      // V rows 2c, 2c+1, 2c+8, 2c+9, D/8 codes from column (D/8) g
      uint32_t vw[4][D / 32];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int row = 2 * c + (t & 1) + (t >> 1) * 8;
        if (D == 128) {
          const uint4 w = lds128(v_unit + unit_off<D>(row, g));
          vw[t][0] = w.x; vw[t][1] = w.y; vw[t][2 % (D / 32)] = w.z; vw[t][3 % (D / 32)] = w.w;
        } else {
          const uint2 w = lds64(v_unit + unit_off<D>(row, g >> 1) + (g & 1) * 8);
          vw[t][0] = w.x; vw[t][1] = w.y;
        }
      }
      bool bad = false;   // NaN codes among positions that some rows do not see
      if (edge) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int w = 0; w < D / 32; ++w) {
            const uint32_t x = vw[t][w] & 0x7f7f7f7fu;
            bad = bad || ((x + 0x01010101u) & 0x80808080u) != 0;
          }
        bad = __any_sync(0xffffffffu, bad);
      }
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        const uint32_t x0 = __byte_perm(vw[0][w], vw[1][w], 0x5140), x1 = __byte_perm(vw[0][w], vw[1][w], 0x7362);
        const uint32_t y0 = __byte_perm(vw[2][w], vw[3][w], 0x5140), y1 = __byte_perm(vw[2][w], vw[3][w], 0x7362);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t xs = e < 2 ? x0 : x1, ys = e < 2 ? y0 : y1;
          uint32_t b0 = e & 1 ? e4m3x2_hi(xs) : e4m3x2_lo(xs), b1 = e & 1 ? e4m3x2_hi(ys) : e4m3x2_lo(ys);
          if (bad) {
            // A NaN value reaches the rows that see its position and no other:
            // a product of visibility and NaN-ness finds them.
            const uint32_t n0 = nan_ones(b0), n1 = nan_ones(b1);
            b0 = nan_zero(b0);
            b1 = nan_zero(b1);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              uint4 see;
              uint32_t* sw = reinterpret_cast<uint32_t*>(&see);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                sw[k] = (s[mt][k >> 1][2 * (k & 1)] != -INFINITY ? 0x3c00u : 0u) |
                        (s[mt][k >> 1][2 * (k & 1) + 1] != -INFINITY ? 0x3c000000u : 0u);
              float hit[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16(hit, see, n0, n1);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (hit[k] > 0.f) o[mt][w * 4 + e][k] = __int_as_float(0x7fc00000);
            }
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) mma_f16(o[mt][w * 4 + e], pa[mt], b0, b1);
        }
      }
    }
    cp_async_wait<0>();
    __syncthreads();

    // ---- join the four warps
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i2 = 0; i2 < 2; ++i2) {
        float l = l_run[mt][i2];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        const int r = mt * 16 + i2 * 8 + g;
        if (c == 0) s_ml[warp * kRows + r] = make_float2(m_run[mt][i2], l);
        // columns 2c and 2c + 1 of the n-tiles: d = kNt * 2c + j and kNt * (2c + 1) + j
        float* dst = s_o + (warp * kRows + r) * L::kPitch + 2 * c * kNt;
#pragma unroll
        for (int j = 0; j < kNt; j += 4) {
          *reinterpret_cast<float4*>(dst + j) = make_float4(o[mt][j][2 * i2] * ref, o[mt][j + 1][2 * i2] * ref,
                                                            o[mt][j + 2][2 * i2] * ref, o[mt][j + 3][2 * i2] * ref);
          *reinterpret_cast<float4*>(dst + kNt + j) =
              make_float4(o[mt][j][2 * i2 + 1] * ref, o[mt][j + 1][2 * i2 + 1] * ref, o[mt][j + 2][2 * i2 + 1] * ref,
                          o[mt][j + 3][2 * i2 + 1] * ref);
        }
      }
    __syncthreads();
    const bool whole = nt_ == tiles;
    float* part = a.part + static_cast<int64_t>(2 * cta + (pos == lo ? 0 : 1)) * kRows * L::kPitch;
    for (int x = tid; x < kRows * (D / 4); x += kAttnThreads) {
      const int r = x / (D / 4), d = (x % (D / 4)) * 4;
      const int R = row0 + r;
      if (R >= rows_total) break;
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int w = 0; w < kAttnWarps; ++w) m = fmaxf(m, s_ml[w * kRows + r].x);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      const float m0 = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int w = 0; w < kAttnWarps; ++w) {
        const float2 ml = s_ml[w * kRows + r];
        const float f = ex2(ml.x - m0);
        const float4 t = *reinterpret_cast<const float4*>(s_o + (w * kRows + r) * L::kPitch + d);
        l += ml.y * f;
        v.x += t.x * f;
        v.y += t.y * f;
        v.z += t.z * f;
        v.w += t.w * f;
      }
      if (whole) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int n = R / a.G;
        const int64_t row = (static_cast<int64_t>(b) * a.N + n) * a.Hq + h * a.G + (R - n * a.G);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + (row * D + d) * 2) =
            make_uint2(T::pack2(v.x * inv, v.y * inv), T::pack2(v.z * inv, v.w * inv));
        if (a.lse && d == 0) a.lse[row] = l == 0.f ? -INFINITY : (m0 + log2f(l)) * kLn2;
      } else {
        *reinterpret_cast<float4*>(part + r * L::kPitch + d) = v;
        if (d == 0) *reinterpret_cast<float2*>(part + r * L::kPitch + D) = make_float2(m, l);
      }
    }
    __syncthreads();
  }
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
  const int64_t join = blockIdx.x - static_cast<int64_t>(a.status ? a.B : 0);
  const bool check = join < 0;
  const int b = check ? blockIdx.x : static_cast<int>(join / (kRows / 4) / ipr);
  const int64_t off = a.plan[b], total = a.plan[a.B], Ge = a.plan[a.B + 1];
  const int64_t next = b + 1 < a.B ? a.plan[b + 1] : total;
  const int64_t tiles = next - off, TT = total * ipr;
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
      const int64_t first = ((off * ipr + 1) * Ge - 1) / TT, last = (next * ipr * Ge - 1) / TT;
      for (int64_t i = first + tid; i <= last; i += kAttnThreads) late = late || a.failed[i] != 0;
    }
    bad_page = __syncthreads_or(bad_page);
    bad_parent = __syncthreads_or(bad_parent);
    late = __syncthreads_or(late);
    if (tid == 0)
      a.status[b] = (bad_page ? SV_STATUS_BAD_PAGE : 0) | (bad_parent ? SV_STATUS_BAD_PARENT : 0) | (late ? SV_STATUS_TIMEOUT : 0);
    return;
  }
  const int item = static_cast<int>(join / (kRows / 4) - static_cast<int64_t>(b) * ipr);
  const int64_t t0 = off * ipr + item * tiles, t1 = t0 + tiles;
  const int64_t c0 = ((t0 + 1) * Ge - 1) / TT, c1 = (t1 * Ge - 1) / TT;
  if (c0 == c1) return;   // one CTA had all of it
  const int h = item / a.RB, rb = item - h * a.RB;
  const int slot0 = TT * c0 / Ge == t0 ? 0 : 1;
  const int r = static_cast<int>(join % (kRows / 4)) * 4 + warp, R = rb * kRows + r;
  if (R >= a.N * a.G) return;
  float m = -INFINITY, l = 0.f, v[kV];
#pragma unroll
  for (int k = 0; k < kV; ++k) v[k] = 0.f;
  for (int64_t i0 = c0; i0 <= c1; i0 += kJoinBatch) {
    float2 ml[kJoinBatch];
    float t[kJoinBatch][kV];
#pragma unroll
    for (int k = 0; k < kJoinBatch; ++k) {
      const int64_t i = min(i0 + k, c1);
      const float* p = a.part + ((2 * i + (i == c0 ? slot0 : 0)) * kRows + r) * kPitch;
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
