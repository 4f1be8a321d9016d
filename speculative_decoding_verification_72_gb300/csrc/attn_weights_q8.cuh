// Accumulated attention weight of the accepted rows, the score that eviction
// ranks by.
//
// Row i of request b (i = 0 .. num_accepted[b]; node path_nodes[b, i] of the
// verify pass, or node i) is the token at position base_b + i. With the
// attention's own lse, per kv head:
//   w_j = sum over rows i and the G heads of the group of exp(s_ij - lse_i), j <= base + i
//   out_j = decay * scores_j + w_j (j < base), w_j (base <= j < length), 0 (j >= length)
//
// The verify pass cannot do this itself: which rows count is known only after
// verification. Keys alone are read again (half of a position's bytes), and
// since lse is known there is no maximum, no sum and nothing to join: each
// tile gives its own weights.
//
// The product is attn_q8_cols.cuh's S^T = K q^T, straight from the codes, with
// q as e4m3 terms in columns. Lane = token makes a weight one thread's sum over
// its rows of S^T: no thread talks to another. q's first term and the rest
// (scaled by 32; for f16 in two terms of that one scale) take two columns a
// row, which leave 2^-22 of the row's largest element; weights are formed and
// summed in fp32. 64 rows a pass over the keys; more take more passes.
//
// Measured: 8 requests of up to 65536 tokens, 64 query heads on 8 of 64: f16 48
// rows 64 us, 32 rows 53, 16 rows 47, bf16 48 rows 63; the bytes alone would take
// 28. Exponentials are not the bound (their pipe is at 16 %, an instruction
// issues in half of the clocks): the warps, two CTAs of eight an SM, wait for
// TMEM reads, which they await a group of 16 rows at a time, and for scales.
//
// Warps 0-3 take even tiles, 4-7 odd ones; 8: TMA; 9: MMA. Two CTAs an SM.
#pragma once

#include "attn_q8_cols.cuh"

namespace sv {

constexpr int kWtThreads = 320;
constexpr int kWtSoft = 256;

struct WeightArgs {
  const uint8_t* q;
  int64_t sqb, sqn, sqh;       // bytes: request, node, head
  const float* lse;            // [B, N, Hq]
  Q8View c;
  const int32_t* base;         // [B]
  const int32_t* path;         // [B, path_cols] or nullptr
  const int32_t* num_acc;      // [B] or nullptr (all N rows)
  const float* scores;         // [B, Hkv, S]
  float* out;                  // [B, Hkv, S]
  int32_t* status;             // [B] or nullptr
  int32_t path_cols, B, N, G, Hq, S, grid;
  uint64_t inv_g;              // as in AttnArgs
  float coef, decay;
};

// n = rows that count; len = positions that hold a token.
__device__ __forceinline__ AttnReq weight_req(const WeightArgs& a, int b) {
  AttnReq r;
  const int cap = min(a.c.max_pages << a.c.page_shift, a.S);
  r.base = a.base[b];
  r.n = a.num_acc ? min(max(a.num_acc[b] + 1, 0), a.path ? min(a.path_cols, a.N) : a.N) : a.N;
  if (r.base < 0) r.base = r.n = 0;
  r.base = min(r.base, cap);
  r.len = min(r.base + r.n, cap);
  return r;
}

// A CTA's walk over its range: pieces of (request, head) items, each as many
// times as its rows take passes.
struct WeightCursor {
  int32_t pos, off;
  AttnReq rq;
  int b, h, t0, n, passes;
  __device__ __forceinline__ void start(const AttnLine& line, int32_t lo) {
    pos = lo;
    off = line.off;
    b = line.b;
    n = 0;
  }
  __device__ __forceinline__ void piece(const WeightArgs& a, int32_t hi, int rows) {
    rq = weight_req(a, b);
    int tiles = (rq.len + kColTile - 1) / kColTile;
    while (pos >= (off + tiles) * a.c.Hkv) {
      off += tiles;
      rq = weight_req(a, ++b);
      tiles = (rq.len + kColTile - 1) / kColTile;
    }
    const int rel = pos - off * a.c.Hkv;
    h = rel / tiles;
    t0 = rel - h * tiles;
    n = min(tiles - t0, hi - pos);
    passes = max(1, (rq.n * a.G + rows - 1) / rows);
  }
};

template <int D, int MT, int NT>
struct WtLayout {
  static constexpr int R = 16 * MT;
  static constexpr int kTileBytes = kColTile * D;
  static constexpr int kKs = D == 128 ? 4 : 6;
  static constexpr int kNs = 2 * R;                                // columns of S^T: first terms, then the rest
  static constexpr int kTmem = 2 * kNs <= 64 ? 64 : 2 * kNs <= 128 ? 128 : 256;
  static constexpr int kQBytes = NT * R * D;
  static constexpr int kOffQ = kKs * kTileBytes;
  static constexpr int kOffMisc = kOffQ + (kQBytes + 1023) / 1024 * 1024;
  static constexpr int kBytes = 1024 + kOffMisc + 3 * R * 4 + 16 * 8 * 8;
};

template <typename T, int D, int MT, int NT>
__global__ void __launch_bounds__(kWtThreads, 2)
    attn_weights_q8_kernel(const __grid_constant__ CUtensorMap k_map, const WeightArgs a) {
  using L = WtLayout<D, MT, NT>;
  constexpr int R = L::R;
  extern __shared__ uint8_t raw[];
  __shared__ AttnLine s_line;
  __shared__ int32_t s_warp[kWtThreads / 32];
  __shared__ __align__(8) uint64_t s_bar[2 * L::kKs + 5];
  __shared__ uint32_t s_tmem, s_fail;
  const uint32_t smem0 = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t* smem = raw + (smem0 - smem_u32(raw));
  float* s_cq = reinterpret_cast<float*>(smem + L::kOffMisc);    // [R] q's factor * coef
  float* s_l2 = s_cq + R;                                        // [R] lse (log2)
  int32_t* s_at = reinterpret_cast<int32_t*>(s_l2 + R);          // [R] the row's position past base, -1: no row
  float2* s_sc = reinterpret_cast<float2*>(s_at + R);            // [16 tiles][8 pages]: ks, page there

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t full_k = smem_u32(s_bar), empty_k = full_k + 8 * L::kKs;
  const uint32_t s_ready = empty_k + 8 * L::kKs, s_free = s_ready + 16, q_ready = s_free + 16;
  if (tid == 0) {
    s_fail = 0;
    for (int i = 0; i < L::kKs; ++i) {
      mbar_init(full_k + 8 * i, 1);
      mbar_init(empty_k + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_ready + 8 * i, 1);
      mbar_init(s_free + 8 * i, 4);
    }
    mbar_init(q_ready, kWtSoft);
    fence_barrier_init();
  }
  if (warp == 9) tmem_alloc(smem_u32(&s_tmem), L::kTmem);
  if (warp == 8 && lane == 0) tma_prefetch_map(&k_map);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  grid_dep_wait();
  grid_dep_launch();
  const int H = a.c.Hkv, cta = blockIdx.x;
  const AttnRanges ranges = attn_scan<kWtThreads>(
      a.B, [&](int r) { return (weight_req(a, r).len + kColTile - 1) / kColTile; }, a.grid, cta, &s_line, s_warp, H, nullptr);
  const int lo = cta < ranges.n ? ranges.begin(cta) : 0, hi = cta < ranges.n ? ranges.begin(cta + 1) : 0;
  WeightCursor cur;   // every role walks the same pieces and passes; n counts tiles across them
  cur.start(s_line, lo);
  uint32_t n = 0;
  volatile uint32_t* fail = &s_fail;

  if (warp == 8) {
    // ------------------------------------------------------------- K, scales
    bool ok = true;
    const int shift = 7 - a.c.page_shift, boxes = 1 << shift, batch = 32 >> shift;   // boxes of a tile, tiles of a batch
    const int box_bytes = D << a.c.page_shift;
    for (; ok && cur.pos < hi; cur.pos += cur.n) {
      cur.piece(a, hi, R);
#pragma unroll 1
      for (int pass = 0; ok && pass < cur.passes; ++pass) {
        // A page a lane, so 32 / boxes tiles at a time, two and one such batches ahead: a
        // tile at a time, each waited for a scale's latency (8 requests of up to 65536
        // tokens, 64 query heads on 8 of 64, 16 rows: 56 us, 47 in batches).
        auto page_of = [&](int first) {
          const int i = first + (lane >> shift), tok = (cur.t0 + i) * kColTile + ((lane & (boxes - 1)) << a.c.page_shift);
          return i < cur.n && tok < cur.rq.len ? q8_page(a.c, cur.b, tok >> a.c.page_shift) : -1;
        };
        auto scale_of = [&](int p) { return p >= 0 ? a.c.ks[static_cast<int64_t>(p) * H + cur.h] : 0.f; };
        int page = page_of(0), page1 = page_of(batch);
        float ks = scale_of(page);
#pragma unroll 1
        for (int i0 = 0; ok && i0 < cur.n; i0 += batch) {
          const int page2 = page_of(i0 + 2 * batch);
          const float ks1 = scale_of(page1);
          const uint32_t there = __ballot_sync(0xffffffffu, page >= 0);
#pragma unroll 1
          for (int j = 0; j < batch && i0 + j < cur.n; ++j, ++n) {
            const uint32_t bytes = __popc(there >> (j << shift) & ((1u << boxes) - 1)) * box_bytes;
            const uint32_t st = n % L::kKs, ph = n / L::kKs;
            if (lane == 0 && ph > 0) ok = wait_or_fail(empty_k + 8 * st, (ph - 1) & 1, fail);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            const bool mine = lane >> shift == j;
            const int box = lane & (boxes - 1);
            if (mine) s_sc[(n & 15) * 8 + box] = make_float2(ks, page >= 0 ? 1.f : 0.f);
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(full_k + 8 * st, bytes);
            __syncwarp();
            if (mine && page >= 0)
              tma_load_3d(smem0 + st * L::kTileBytes + box * box_bytes, &k_map, 0, page * H + cur.h, full_k + 8 * st);
          }
          page = page1;
          page1 = page2;
          ks = ks1;
        }
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------------ MMA
    if (lane == 0) {
      constexpr uint32_t kSw = D == 128 ? 2 : 4, kSbo = 8 * D;
      constexpr uint32_t kId2 = tc_idesc(0, false, false, 128, 2 * R), kId1 = tc_idesc(0, false, false, 128, R);
      bool ok = true;
      uint32_t loads = 0;
      for (; ok && cur.pos < hi; cur.pos += cur.n) {
        cur.piece(a, hi, R);
#pragma unroll 1
        for (int pass = 0; ok && pass < cur.passes; ++pass) {
          ok = wait_or_fail(q_ready, loads++ & 1, fail);
          for (int i = 0; i < cur.n && ok; ++i, ++n) {
            const uint32_t st = n % L::kKs, sb = n & 1;
            ok = wait_or_fail(full_k + 8 * st, (n / L::kKs) & 1, fail) &&
                 (n < 2 || wait_or_fail(s_free + 8 * sb, (n / 2 - 1) & 1, fail));
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
              tc_mma_f8(tmem + sb * L::kNs, tc_desc(smem0 + st * L::kTileBytes + 32 * k, 16, kSbo, kSw),
                        tc_desc(smem0 + L::kOffQ + 32 * k, 16, kSbo, kSw), kId2, k > 0);
            if (NT == 3) {
#pragma unroll
              for (int k = 0; k < D / 32; ++k)
                tc_mma_f8(tmem + sb * L::kNs + R, tc_desc(smem0 + st * L::kTileBytes + 32 * k, 16, kSbo, kSw),
                          tc_desc(smem0 + L::kOffQ + 2 * R * D + 32 * k, 16, kSbo, kSw), kId1, true);
            }
            tc_commit(empty_k + 8 * st);
            tc_commit(s_ready + 8 * sb);
          }
        }
      }
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- weights
    // A wait that gives up ends no loop here: these warps meet at barriers, so all
    // run on to the end (every later wait then returns at once), without meaning.
    const int set = warp >> 2, row = tid & 127;   // even or odd tiles; the token within a tile
    const uint32_t t_s = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + set * L::kNs;
    for (; cur.pos < hi; cur.pos += cur.n) {
      cur.piece(a, hi, R);
      const AttnReq rq = cur.rq;
      const int32_t* path = a.path ? a.path + static_cast<int64_t>(cur.b) * a.path_cols : nullptr;
      const float* sc = a.scores + (static_cast<int64_t>(cur.b) * H + cur.h) * a.S;
      float* out = a.out + (static_cast<int64_t>(cur.b) * H + cur.h) * a.S;
      const uint8_t* q = a.q + cur.b * a.sqb + static_cast<int64_t>(cur.h) * a.G * a.sqh;
      const int rows_total = rq.n * a.G;
#pragma unroll 1
      for (int pass = 0; pass < cur.passes; ++pass) {
        const int row0 = pass * R;
        // ---- q as e4m3 terms: D / 8 lanes a row, eight elements each
        constexpr int kLpr = D / 8, kRpi = kWtSoft / kLpr;
        named_barrier_sync(1, kWtSoft);   // the last pass's rows have been used, its weights are written
#pragma unroll
        for (int r0 = 0; r0 < R; r0 += kRpi) {
          const int r = r0 + tid / kLpr, ql = tid % kLpr;
          if (R < kRpi && r >= R) continue;
          const int Rg = row0 + r, at = static_cast<int>(static_cast<uint64_t>(Rg) * a.inv_g >> 32), g = Rg - at * a.G;
          int node = -1;
          if (Rg < rows_total) node = path ? path[at] : at;
          if (node >= a.N) node = -1;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (node >= 0) v = *reinterpret_cast<const uint4*>(q + node * a.sqn + g * a.sqh + ql * 16);
          float f[8];
          T::load8(&v, f);
          float m = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
          const uint32_t lanes = kLpr == 16 ? 0xffffu << (lane & 16) : 0xffu << (lane & 24);
#pragma unroll
          for (int o = kLpr / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(lanes, m, o));
          const int e = m > 0.f ? static_cast<int>(__float_as_uint(m) >> 23) - 127 : 7;   // the maximum into [2^7, 2^8)
          const int x = min(max(7 - e, -126), 126);
          const float up = exp2_int(x);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] *= up;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            uint32_t w[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              w[k] = e4m3_pack4(f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]);
              const float2 x0 = half2_bits(e4m3x2_lo(w[k])), x1 = half2_bits(e4m3x2_hi(w[k]));
              const float s = t == 0 ? 32.f : 1.f;
              f[4 * k] = (f[4 * k] - x0.x) * s;
              f[4 * k + 1] = (f[4 * k + 1] - x0.y) * s;
              f[4 * k + 2] = (f[4 * k + 2] - x1.x) * s;
              f[4 * k + 3] = (f[4 * k + 3] - x1.y) * s;
            }
            *reinterpret_cast<uint2*>(smem + L::kOffQ + unit_off<D>(t * R + r, ql >> 1) + (ql & 1) * 8) = make_uint2(w[0], w[1]);
          }
          if (ql == 0) {
            // Infinities saturate in e4m3, so the factor makes their row NaN (NaN codes stay NaN).
            s_cq[r] = m == INFINITY ? __int_as_float(0x7fc00000) : exp2_int(-x) * a.coef;
            s_at[r] = node >= 0 ? at : -1;
            // A row that saw nothing (lse -inf) gives no weight, like one that does not count.
            const float l2 = node >= 0 ? a.lse[(static_cast<int64_t>(cur.b) * a.N + node) * a.Hq + cur.h * a.G + g] * kLog2e : INFINITY;
            s_l2[r] = l2 == -INFINITY ? INFINITY : l2;
          }
        }
        fence_async_smem();
        mbar_arrive(q_ready);
        named_barrier_sync(1, kWtSoft);
        // what a tile's weights are added to, loaded before its product is awaited
        auto old_of = [&](int i) {
          const int tok = (cur.t0 + i) * kColTile + row;
          if (i >= cur.n || tok >= rq.len) return 0.f;
          return pass > 0 ? out[tok] : tok < rq.base ? a.decay * sc[tok] : 0.f;
        };
        const int groups = min(MT, (rows_total - row0 + 15) / 16);   // of 16 rows, with a row in them
        const int first = (n ^ set) & 1;   // this group's first tile of the pass
        float old = old_of(first);
#pragma unroll 1
        for (int i = first; i < cur.n; i += 2) {
          const uint32_t m = n + i;
          const int tok = (cur.t0 + i) * kColTile + row;
          const float next = old_of(i + 2);
          const bool there = wait_or_fail(s_ready + 8 * set, (m / 2) & 1, fail);
          tc_fence_after();
          const float2 s = s_sc[(m & 15) * 8 + (row >> a.c.page_shift)];
          const bool edge = (cur.t0 + i + 1) * kColTile > rq.base;
          const int at = tok - rq.base;
          float2 w = make_float2(0.f, 0.f);
#pragma unroll 1
          for (int g = 0; g < groups; ++g) {
            uint32_t x0[16], x1[16];
            tmem_ld16(t_s + g * 16, x0);
            tmem_ld16(t_s + R + g * 16, x1);
            tmem_ld_wait();
            tmem_use(x0);
            tmem_use(x1);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float4 cc = reinterpret_cast<const float4*>(s_cq + g * 16)[j], ll = reinterpret_cast<const float4*>(s_l2 + g * 16)[j];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int r = 4 * j + 2 * k;
                const float2 v = __ffma2_rn(make_float2(__uint_as_float(x1[r]), __uint_as_float(x1[r + 1])),
                                            make_float2(1.f / 32.f, 1.f / 32.f),
                                            make_float2(__uint_as_float(x0[r]), __uint_as_float(x0[r + 1])));
                const float2 c = __fmul2_rn(k ? make_float2(cc.z, cc.w) : make_float2(cc.x, cc.y), make_float2(s.x, s.x));
                const float2 y = __ffma2_rn(v, c, k ? make_float2(-ll.z, -ll.w) : make_float2(-ll.x, -ll.y));
                float2 p = make_float2(ex2(y.x), ex2(y.y));
                if (edge) {
                  if (at > s_at[g * 16 + r]) p.x = 0.f;
                  if (at > s_at[g * 16 + r + 1]) p.y = 0.f;
                }
                w = __fadd2_rn(w, p);
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_free + 8 * set);
          float add = s.y != 0.f && rows_total > 0 ? w.x + w.y : 0.f;
          if (!there) add = __int_as_float(0x7fc00000);   // no product came: NaN, whatever becomes of the status bit
          if (tok < rq.len) out[tok] = old + add;
          old = next;
        }
        n += cur.n;
      }
    }
  }
  // Positions past the end, and what is wrong with a request, spread over the CTAs.
  for (int x = cta; x < a.B * H; x += gridDim.x) {
    const int len = weight_req(a, x / H).len;
    for (int j = len + tid; j < a.S; j += kWtThreads) a.out[static_cast<int64_t>(x) * a.S + j] = 0.f;
  }
  __syncthreads();
  const bool late = s_fail != 0;
  if (late) {   // a wait gave up: leave time for copies and products in flight before TMEM goes
    const uint64_t t = global_timer_ns();
    for (int i = 0; i < (1 << 20) && global_timer_ns() - t < 2000000; ++i) {
    }
  }
  if (a.status)
    for (int b = cta; b < a.B; b += gridDim.x) {
      const AttnReq rq = weight_req(a, b);
      const int rows = a.num_acc ? a.num_acc[b] + 1 : a.N;
      bool bad = a.base[b] < 0 || rows < 0 || rows != rq.n || rq.len != a.base[b] + rows;
      for (int j = tid; j < (rq.len + (1 << a.c.page_shift) - 1) >> a.c.page_shift; j += kWtThreads)
        bad = bad || q8_page(a.c, b, j) < 0;
      if (a.path)
        for (int i = tid; i < rq.n; i += kWtThreads) {
          const int p = a.path[static_cast<int64_t>(b) * a.path_cols + i];
          bad = bad || p < 0 || p >= a.N;
        }
      bad = __syncthreads_or(bad);
      if (tid == 0) a.status[b] = bad ? SV_STATUS_BAD_PAGE : 0;
    }
  __syncthreads();
  // A wait that gave up: its scores are NaN, and the flag goes to all requests.
  // A CTA that reports a request later than this may write over the bit; the
  // NaN stays.
  if (late && a.status)
    for (int b = tid; b < a.B; b += kWtThreads) atomicOr(&a.status[b], SV_STATUS_TIMEOUT);
  if (warp == 9) tmem_free(tmem, L::kTmem);
}

}  // namespace sv
