// Attention over the 8-bit cache for many rows a kv head (draft trees, long
// chains), bound by the tensor cores.
//
// A block is 128 rows of one kv head, and rows are the lanes:
//   S [128 rows, 128 tokens] = q K^T     K as it lies in shared memory (e4m3),
//                                        q as a sum of e4m3 terms of one scale
//   O [128 rows, D] += P V               P f16 in TMEM, V converted to f16
// q's terms (two for bf16, three for f16) add up in one accumulator; they leave
// 2^-17 of the row's largest element. P in e4m3 terms would need its columns
// per term twice over in TMEM, and there are 128 x 128 of them a tile, so P is
// f16 (rounded by 2^-11 of its value at most, or by 2^-25 below f16's normal
// numbers, where the row's largest is 1 to 2^8) and V, of which there are 128 x
// D, is converted (exactly) by four warps on its way from global to shared
// memory. Sums of P take it before it is rounded. MMA time per tile: 512 clocks
// for S (two terms at twice f16's rate) and 512 for P V.
//
// Lane = row keeps the softmax within a thread, or two: two groups of four
// warps take 64 tokens of a tile each, so that a row's exponentials are shared
// by two threads (at one thread a row they were 2250 of 6000 clocks a tile).
// A thread reads its half row of S twice: for the maximum, on which the CTA
// votes (only if a score is more than 2^8 above its row's running maximum do
// maxima rise and is O rescaled in TMEM), and for the exponentials, which it
// writes over the part of S that it has read. Holding P in registers between
// one pass and the vote instead took 88 registers and more a thread, and two
// CTAs leave 72.
//
// S and P share TMEM columns, so within a CTA S, softmax and P V of a tile
// follow each other; two CTAs an SM fill each other's gaps.
//
// Measured: 16 requests of 64-node trees over about 5100 tokens, 32 heads on 8
// of 128: bf16 158 us, 0.54 PFLOP/s of the products that the mask leaves; f16 229
// (its third term of q leaves room for one CTA an SM with heads of 128). What
// bounds it is the softmax warps' own pace, about 5.6 clocks an instruction at
// seven warps a scheduler; the tensor pipe is a third busy. Halves of a tile
// with barriers of their own, one's products under the other's softmax, took
// 173 us.
//
// Warps 0-7: softmax. 8-11: V. 12: TMA (K) and the pages' scales. 13: MMA.
// Masks, NaN codes, scales, work split and join as in attn_q8_cols.cuh; here
// the rows that see a NaN code note its column in registers.
#pragma once

#include <algorithm>

#include <cuda.h>

#include "attn_q8_cols.cuh"

namespace sv {

constexpr int kRowThreads = 448;
constexpr int kRowSoft = 256;          // softmax threads
constexpr int kRowTmem = 256;
constexpr float kRowSlack = 8.f;

template <int D, int NT>
struct RowLayout {
  static constexpr int kTileBytes = kColTile * D;                 // K codes
  static constexpr int kQBytes = NT * kTileBytes;
  static constexpr int kVBytes = kColTile * D * 2;                // V in f16
  static constexpr int kKs = 2, kVb = D == 128 ? 1 : 2;           // ring depths
  static constexpr int kOffK = kQBytes;
  static constexpr int kOffV = kOffK + kKs * kTileBytes;
  static constexpr int kOffMisc = kOffV + kVb * kVBytes;
  static constexpr int kMiscBytes = kVb * 128 * (D / 32) * 4 + 1024 + 128 * 4 + 256 * 12 + 256 * 4;
  // Nodes that a block's 128 rows can belong to, G rows a node.
  static int nodes(int N, int G) { return std::min(N, (126 + G) / G + 1); }
  static int bytes(int nodes, int words) { return 1024 + kOffMisc + kMiscBytes + nodes * words * 4; }
  static int most() { return bytes(nodes(SV_MAX_TREE_NODES, 1), SV_MAX_TREE_NODES / 32); }
};

// O (TMEM) = P (TMEM, f16) V (shared memory, f16) (+ O if acc).
__device__ __forceinline__ void tc_mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))
      : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(addr)
               : "memory");
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kRowThreads, 2)
    attn_q8_rows_kernel(const __grid_constant__ CUtensorMap k_map, const AttnArgs a) {
  using L = RowLayout<D, NT>;
  constexpr int kPitch = AttnLayout<D>::kPitch;
  extern __shared__ uint8_t raw[];
  __shared__ AttnLine s_line;
  __shared__ int32_t s_warp[kRowThreads / 32];
  __shared__ __align__(8) uint64_t s_bar[2 * L::kKs + 2 * L::kVb + 4];
  __shared__ uint32_t s_tmem, s_fail, s_bad[2], s_whole[8];   // s_whole: by tile, every page is there; s_bad: by V buffer, the last tile (+ 1) with NaN codes taken out
  const uint32_t smem0 = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t* smem = raw + (smem0 - smem_u32(raw));
  float4* s_sc = reinterpret_cast<float4*>(smem + L::kOffMisc);          // [8 tiles][8 pages]: ks, log2(vs / v0), v0 / vs, v0
  float* s_cq = reinterpret_cast<float*>(s_sc + 64);                     // [128]
  uint32_t* s_nan = reinterpret_cast<uint32_t*>(s_cq + 128);             // [kVb][128 tokens][D / 32]
  uint32_t* s_vis = s_nan + L::kVb * 128 * (D / 32);                     // [256][3]: tokens of an edge tile that a half row sees
  float* s_half = reinterpret_cast<float*>(s_vis + 256 * 3);             // [256]
  uint32_t* s_anc = reinterpret_cast<uint32_t*>(s_half + 256);           // [nodes of the block][words]

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t full_k = smem_u32(s_bar), empty_k = full_k + 8 * L::kKs, v_ready = empty_k + 8 * L::kKs;
  const uint32_t v_free = v_ready + 8 * L::kVb, s_ready = v_free + 8 * L::kVb, p_ready = s_ready + 8, o_done = p_ready + 8;
  const uint32_t q_ready = o_done + 8;
  if (tid == 0) {
    s_fail = s_bad[0] = s_bad[1] = 0;
    for (int i = 0; i < L::kKs; ++i) {
      mbar_init(full_k + 8 * i, 1);
      mbar_init(empty_k + 8 * i, 1);
    }
    for (int i = 0; i < L::kVb; ++i) {
      mbar_init(v_ready + 8 * i, 128);
      mbar_init(v_free + 8 * i, 1);
    }
    mbar_init(s_ready, 1);
    mbar_init(p_ready, kRowSoft);
    mbar_init(o_done, 1);
    mbar_init(q_ready, kRowSoft);
    fence_barrier_init();
  }
  if (warp == 13) tmem_alloc(smem_u32(&s_tmem), kRowTmem);
  if (warp == 12 && lane == 0) tma_prefetch_map(&k_map);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  grid_dep_wait();
  grid_dep_launch();
  const int ipr = a.c.Hkv * a.RB;
  const int cta = blockIdx.x;
  const AttnRanges ranges = attn_scan<kRowThreads>(
      a.B, [&](int r) { return attn_tiles<kColTile>(attn_req(a, r)); }, a.grid, cta, &s_line, s_warp, ipr, cta == 0 ? a.plan : nullptr);
  if (cta == 0 && tid == 0) a.plan[a.B] = s_line.total;
  const int lo = cta < ranges.n ? ranges.begin(cta) : 0, hi = cta < ranges.n ? ranges.begin(cta + 1) : 0;
  AttnCursor cur;   // every role walks the same pieces; n counts tiles across them
  cur.start(a, s_line, lo);
  uint32_t n = 0;
  volatile uint32_t* fail = &s_fail;

  if (warp == 12) {
    // ------------------------------------------------------------- K, scales
    bool ok = true;
    const int boxes = kColTile >> a.c.page_shift;
    const int box_bytes = D << a.c.page_shift;
    for (; ok && cur.pos < hi; cur.pos += cur.n) {
      cur.piece<kColTile>(a, hi, ipr);
      auto page_of = [&](int i) {
        const int tok = (cur.t0 + i) * kColTile + (lane << a.c.page_shift);
        return i < cur.n && lane < boxes && tok < cur.rq.len ? q8_page(a.c, cur.b, tok >> a.c.page_shift) : -1;
      };
      auto scales_of = [&](int p) {
        const int64_t o = static_cast<int64_t>(max(p, 0)) * a.c.Hkv + cur.h;
        return p >= 0 ? make_float2(a.c.ks[o], a.c.vs[o]) : make_float2(0.f, 0.f);
      };
      int page = page_of(0), page1 = page_of(1);
      float2 sc = scales_of(page);
      float v0 = 1.f, most = 0.f;
      for (int i = 0; i < cur.n; ++i, ++n) {
        const int page2 = page_of(i + 2);
        const float2 sc1 = scales_of(page1);
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, page >= 0)) * box_bytes;
        const uint32_t st = n % L::kKs, ph = n / L::kKs;
        if (lane == 0 && ph > 0) ok = wait_or_fail(empty_k + 8 * st, (ph - 1) & 1, fail);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        const bool whole = __popc(__ballot_sync(0xffffffffu, page >= 0)) == boxes;
        sc.y = attn_v_scale(sc.y, page >= 0, most);
        if (i == 0) {
          v0 = __shfl_sync(0xffffffffu, sc.y, 0);
          v0 = v0 > 0.f && v0 < INFINITY ? v0 : 1.f;
        }
        if (lane == 0) s_whole[n & 7] = whole;
        if (lane < 8) {
          const float rel = sc.y / v0;
          const float lv = rel == rel ? fmaxf(lg2(rel), -100.f) : rel;
          s_sc[(n & 7) * 8 + lane] = make_float4(sc.x, lv, page >= 0 ? ex2(-lv) : -1.f, v0);   // -1: no page
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(full_k + 8 * st, bytes);
        __syncwarp();
        if (page >= 0)
          tma_load_3d(smem0 + L::kOffK + st * L::kTileBytes + lane * box_bytes, &k_map, 0, page * a.c.Hkv + cur.h, full_k + 8 * st);
        page = page1;
        page1 = page2;
        sc = sc1;
      }
    }
  } else if (warp == 13) {
    // ------------------------------------------------------------------ MMA
    if (lane == 0) {
      constexpr uint32_t kSw = D == 128 ? 2 : 4, kSbo = 8 * D;
      constexpr uint32_t kIdS = tc_idesc(0, false, false, 128, 128), kIdO = tc_idesc(0, false, true, 128, D);
      bool ok = true;
      uint32_t pieces = 0;
      auto scores = [&](uint32_t m) {
        const uint32_t st = m % L::kKs;
        ok = ok && wait_or_fail(full_k + 8 * st, (m / L::kKs) & 1, fail);
        if (!ok) return;
        tc_fence_after();
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k = 0; k < D / 32; ++k)
            tc_mma_f8(tmem, tc_desc(smem0 + t * L::kTileBytes + 32 * k, 16, kSbo, kSw),
                      tc_desc(smem0 + L::kOffK + st * L::kTileBytes + 32 * k, 16, kSbo, kSw), kIdS, t > 0 || k > 0);
        tc_commit(empty_k + 8 * st);
        tc_commit(s_ready);
      };
      for (; ok && cur.pos < hi; cur.pos += cur.n) {
        cur.piece<kColTile>(a, hi, ipr);
        ok = wait_or_fail(q_ready, pieces++ & 1, fail);
        if (!ok) break;
        scores(n);
        for (int i = 0; i < cur.n && ok; ++i, ++n) {
          const uint32_t vb = n % L::kVb;
          ok = ok && wait_or_fail(v_ready + 8 * vb, (n / L::kVb) & 1, fail) && wait_or_fail(p_ready, n & 1, fail);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < kColTile / 16; ++k)
            tc_mma_f16_ts(tmem + 128, tmem + (k & 3) * 8 + (k >> 2) * 64, tc_desc(smem0 + L::kOffV + vb * L::kVBytes + 2048 * k, 16384, 1024, 2), kIdO,
                          i > 0 || k > 0);
          tc_commit(v_free + 8 * vb);
          tc_commit(o_done);
          // The next S overwrites this P: products of one CTA run in the order they are issued.
          if (i + 1 < cur.n) scores(n + 1);
        }
      }
    }
    __syncwarp();
  } else if (warp >= 8 && warp < 12) {
    // -------------------------------------------------------------------- V
    constexpr int kIts = kColTile * D / 16 / 128;   // 16-byte chunks a thread
    constexpr int kCpr = D / 16;                    // chunks a token
    const int vt = tid - kRowSoft, r0 = vt / kCpr, ch = vt % kCpr;
    constexpr int kStep = 128 / kCpr;               // tokens an iteration: 16 or 32
    uint4 v[kIts];
    for (; cur.pos < hi; cur.pos += cur.n) {
      cur.piece<kColTile>(a, hi, ipr);
      // pages of a tile's eight 16-token units, one a lane
      auto pages_of = [&](int i) {
        const int tok = (cur.t0 + i) * kColTile + (lane & 7) * 16;
        return i < cur.n && tok < cur.rq.len ? q8_page(a.c, cur.b, tok >> a.c.page_shift) : -1;
      };
      auto load = [&](int i, int pages) {
#pragma unroll
        for (int it = 0; it < kIts; ++it) {
          const int row = it * kStep + r0, tok = (cur.t0 + i) * kColTile + row;
          const int page = __shfl_sync(0xffffffffu, pages, row >> 4);
          v[it] = make_uint4(0, 0, 0, 0);
          if (page >= 0 && tok < cur.rq.len) {
            const int64_t o = (((static_cast<int64_t>(page) * a.c.Hkv + cur.h) << a.c.page_shift) +
                               (tok & ((1 << a.c.page_shift) - 1))) * D + ch * 16;
            v[it] = *reinterpret_cast<const uint4*>(a.c.v + o);
          }
        }
      };
      int pages1 = pages_of(1);
      load(0, pages_of(0));
      for (int i = 0; i < cur.n; ++i, ++n) {
        const int pages2 = pages_of(i + 2);
        const uint32_t vb = n % L::kVb;
        if (n >= L::kVb) wait_or_fail(v_free + 8 * vb, (n / L::kVb - 1) & 1, fail);
        const bool edge = (cur.t0 + i + 1) * kColTile > cur.rq.base;
        if (edge) {
          // NaN codes of nodes, which not every row may see: taken out, noted by column
#pragma unroll
          for (int it = 0; it < kIts; ++it) {
            const int row = it * kStep + r0;
            if ((cur.t0 + i) * kColTile + row < cur.rq.base) continue;
            uint32_t* w = reinterpret_cast<uint32_t*>(&v[it]);
            uint32_t cols = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t bad = ((w[j] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
              cols |= ((bad >> 7 & 1) | (bad >> 14 & 2) | (bad >> 21 & 4) | (bad >> 28 & 8)) << (4 * j);
              w[j] &= ~((bad >> 7) * 0xffu);
            }
            reinterpret_cast<uint16_t*>(s_nan)[(vb * 128 + row) * (D / 16) + ch] = static_cast<uint16_t>(cols);
            if (cols) *const_cast<volatile uint32_t*>(&s_bad[vb]) = n + 1;
          }
        }
        // d = 16 ch ..: two 16-byte chunks of block ch / 4 (64 columns a block), odd blocks' stores in the other order;
        // row & 7 is the same for all of a thread's rows
        uint8_t* dst = smem + L::kOffV + vb * L::kVBytes + (ch >> 2) * 16384 + r0 * 128;
        const bool odd = ch >> 2 & 1;
        const int c0 = (ch & 3) * 2;
        const int o1 = ((c0 + odd) ^ (r0 & 7)) << 4, o2 = ((c0 + !odd) ^ (r0 & 7)) << 4;
#pragma unroll
        for (int it = 0; it < kIts; ++it) {
          const uint4 w = v[it];
          const uint4 x = make_uint4(e4m3x2_lo(w.x), e4m3x2_hi(w.x), e4m3x2_lo(w.y), e4m3x2_hi(w.y));
          const uint4 y = make_uint4(e4m3x2_lo(w.z), e4m3x2_hi(w.z), e4m3x2_lo(w.w), e4m3x2_hi(w.w));
          *reinterpret_cast<uint4*>(dst + it * kStep * 128 + o1) = odd ? y : x;
          *reinterpret_cast<uint4*>(dst + it * kStep * 128 + o2) = odd ? x : y;
        }
        fence_async_smem();
        mbar_arrive(v_ready + 8 * vb);
        if (i + 1 < cur.n) load(i + 1, pages1);
        pages1 = pages2;
      }
    }
  } else if (warp < 8) {
    // -------------------------------------------------------------- softmax
    // A wait that gives up ends no loop here: these warps meet at barriers, so all
    // run on to the end (every later wait then returns at once), without meaning:
    // the rows of every piece that ends after it are NaN.
    const int half = warp >> 2, row = tid & 127;   // the thread's 64 tokens of a tile, its row
    const uint32_t t_lane = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t t_s = t_lane + half * 64, t_o = t_lane + 128 + half * (D / 2);
    const int rows_total = a.N * a.G, words = (a.N + 31) / 32;
    for (; cur.pos < hi; cur.pos += cur.n) {
      cur.piece<kColTile>(a, hi, ipr);
      const AttnReq rq = cur.rq;
      const int row0 = cur.rb * 128, node0 = attn_node(a, row0);
      const int Rg = row0 + row, my_at = attn_node(a, Rg);
      const int node = Rg < rows_total && my_at < rq.n ? my_at : -1;

      // ---- q as e4m3 terms: D / 8 lanes a row, eight elements each, four loads of a warp in flight
      const uint8_t* q = a.q + cur.b * a.sqb + static_cast<int64_t>(cur.h) * a.G * a.sqh;
      constexpr int kLpr = D / 8, kRpw = 32 / kLpr;
      const int ql = lane % kLpr;
#pragma unroll 1
      for (int r0 = warp * 16; r0 < warp * 16 + 16; r0 += 4 * kRpw) {
        uint4 raw4[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int R = row0 + r0 + u * kRpw + lane / kLpr, at = attn_node(a, R);
          raw4[u] = make_uint4(0, 0, 0, 0);
          if (R < rows_total && at < rq.n)
            raw4[u] = *reinterpret_cast<const uint4*>(q + at * a.sqn + (R - at * a.G) * a.sqh + ql * 16);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int r = r0 + u * kRpw + lane / kLpr;
          float f[8];
          T::load8(&raw4[u], f);
          float m = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
#pragma unroll
          for (int o = kLpr / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          const int e = m > 0.f ? static_cast<int>(__float_as_uint(m) >> 23) - 127 : 7;
          const int x = min(max(7 - e, -126), 126);
          const float up = a.coef < 0.f ? -exp2_int(x) : exp2_int(x);   // scores grow with S
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] *= up;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            uint32_t w[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              w[k] = e4m3_pack4(f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]);
              const float2 x0 = half2_bits(e4m3x2_lo(w[k])), x1 = half2_bits(e4m3x2_hi(w[k]));
              f[4 * k] -= x0.x;
              f[4 * k + 1] -= x0.y;
              f[4 * k + 2] -= x1.x;
              f[4 * k + 3] -= x1.y;
            }
            *reinterpret_cast<uint2*>(smem + t * L::kTileBytes + unit_off<D>(r, ql >> 1) + (ql & 1) * 8) = make_uint2(w[0], w[1]);
          }
          if (ql == 0) s_cq[r] = m == INFINITY ? __int_as_float(0x7fc00000) : exp2_int(-x) * fabsf(a.coef);
        }
      }
      const bool tail = (cur.t0 + cur.n) * kColTile > rq.base;
      if (tail && a.parents) {
        const int nodes = min(attn_node(a, row0 + 127), a.N - 1) - node0 + 1;
        static_assert(256 * 3 + 256 >= SV_MAX_TREE_NODES, "parents fit in s_vis and s_half");
        int32_t* par = reinterpret_cast<int32_t*>(s_vis);   // free until the first tile
        const int32_t* parents = a.parents + static_cast<int64_t>(cur.b) * a.N;
        for (int i = tid; i < a.N; i += kRowSoft) par[i] = parents[i];
        for (int i = tid; i < nodes * words; i += kRowSoft) s_anc[i] = 0;
        named_barrier_sync(1, kRowSoft);
        for (int i = tid; i < nodes; i += kRowSoft) {
          int m = node0 + i;
          while (m >= 0) {
            s_anc[i * words + (m >> 5)] |= 1u << (m & 31);
            const int up = par[m];
            m = up < m ? up : -1;
          }
        }
      }
      fence_async_smem();
      mbar_arrive(q_ready);
      named_barrier_sync(1, kRowSoft);
      const float cq = s_cq[row];
      // 32 bits of what the row sees of the nodes, from node 32 k
      auto sees = [&](int k) -> uint32_t {
        if (node < 0 || k < 0 || k >= words) return 0u;
        if (a.parents) return s_anc[(node - node0) * words + k];
        const int x = node - 32 * k;
        return x < 0 ? 0u : x >= 31 ? 0xffffffffu : (2u << x) - 1u;
      };

      // A score's factor; 0 would make NaN of -inf.
      auto factor = [&](float k) {
        const float c = cq * k;
        return c == 0.f ? 1e-30f : c;
      };
      float m_run = 0.f, l = 0.f, v0 = 1.f;   // m_run means something once the row has seen a token
      bool seen = false;
      uint32_t nan_cols[D / 32];
#pragma unroll
      for (int j = 0; j < D / 32; ++j) nan_cols[j] = 0;
#pragma unroll 1
      for (int i = 0; i < cur.n; ++i, ++n) {
        const int tok0 = (cur.t0 + i) * kColTile;
        const bool edge = tok0 + kColTile > rq.base;
        wait_or_fail(s_ready, n & 1, fail);   // and every product before this S is done
        tc_fence_after();
        const float4* sc = s_sc + (n & 7) * 8;
        if (edge || !s_whole[n & 7]) {   // the same for every row: what it does not see becomes -inf in S
#pragma unroll 1
          for (int j = 0; j < 2; ++j) {
            const int c0 = half * 64 + 32 * j, m0 = tok0 + c0 - rq.base;   // the word's first token, as a node
            uint32_t bits = node < 0 ? 0u : 0xffffffffu;
            if (edge && m0 > -32) {
              bits = m0 < 0 ? sees(0) << -m0 | (node < 0 ? 0u : (1u << -m0) - 1u)
                            : __funnelshift_r(sees(m0 >> 5), sees((m0 >> 5) + 1), m0 & 31);
              const int left = rq.n - m0;   // nodes from the word's first on
              if (left < 32) bits &= left <= 0 ? 0u : (1u << left) - 1u;
            }
            if (sc[c0 >> a.c.page_shift].z < 0.f) bits &= 0xffff0000u;
            if (sc[(c0 + 16) >> a.c.page_shift].z < 0.f) bits &= 0x0000ffffu;
            s_vis[tid * 3 + j] = bits;
#pragma unroll 1
            for (int g = 2 * j; g < 2 * j + 2; ++g, bits >>= 16) {
              uint32_t s[16];
              tmem_ld16(t_s + g * 16, s);
              tmem_ld_wait();
              tmem_use(s);
#pragma unroll
              for (int k = 0; k < 16; ++k) s[k] = bits >> k & 1 ? s[k] : 0xff800000u;
              tmem_st16(t_s + g * 16, s);
            }
          }
          tmem_st_wait();
        }
        // ---- maximum
        float top = -INFINITY;
        uint32_t w[2][16];
        tmem_ld16(t_s, w[0]);
#pragma unroll 1
        for (int g = 0; g < 4; g += 2) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            tmem_ld_wait();
            tmem_use(w[u]);
            if (u == 0 || g < 2) tmem_ld16(t_s + (g + u + 1) * 16, w[u ^ 1]);
            float mx[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mx[j] = fmaxf(fmaxf(__uint_as_float(w[u][4 * j]), __uint_as_float(w[u][4 * j + 1])),
                            fmaxf(__uint_as_float(w[u][4 * j + 2]), __uint_as_float(w[u][4 * j + 3])));
            const float4 k = sc[(half * 64 + (g + u) * 16) >> a.c.page_shift];
            top = fmaxf(top, fmaf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), factor(k.x), k.y - m_run));
          }
        }
        if (named_barrier_or(1, kRowSoft, top > kRowSlack || (!seen && top > -INFINITY))) {
          s_half[tid] = top;
          named_barrier_sync(1, kRowSoft);
          top = fmaxf(top, s_half[tid ^ 128]);
          const bool raise = seen ? top > kRowSlack : top > -INFINITY;
          const float f = raise && seen ? ex2(-top) : 1.f;
          if (raise) m_run += top;
          seen = seen || raise;
          l *= f;
          if (i > 0 && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
            for (int g = 0; g < D / 32; ++g) {
              uint32_t o[16];
              tmem_ld16(t_o + g * 16, o);
              tmem_ld_wait();
              tmem_use(o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st16(t_o + g * 16, o);
            }
          }
        }
        // ---- exponentials: P over the columns of S that have been read
        tmem_ld16(t_s, w[0]);
#pragma unroll 1
        for (int g = 0; g < 4; g += 2) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            tmem_ld_wait();
            tmem_use(w[u]);
            if (u == 0 || g < 2) tmem_ld16(t_s + (g + u + 1) * 16, w[u ^ 1]);
            const uint32_t* s = w[u];
            const float4 k = sc[(half * 64 + (g + u) * 16) >> a.c.page_shift];
            const float c = factor(k.x), b = k.y - m_run;
            const float2 c2 = make_float2(c, c), b2 = make_float2(b, b);
            uint32_t h[8];
            float2 part = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), c2, b2);
              const float2 p = make_float2(ex2(x.x), ex2(x.y));
              part = __fadd2_rn(part, p);
              h[j] = pack_half2(p.x, p.y);
            }
            const float total = part.x + part.y;
            l += total == 0.f ? 0.f : total * k.z;   // 0 where a missing page has no factor
            tmem_st8(t_s + (g + u) * 8, h);
          }
        }
        if (i == 0) v0 = sc[0].w;
        if (edge) {   // NaN values among the nodes that this row sees
          const uint32_t vb = n % L::kVb;
          wait_or_fail(v_ready + 8 * vb, (n / L::kVb) & 1, fail);
          if (*const_cast<volatile uint32_t*>(&s_bad[vb]) == n + 1) {
#pragma unroll 1
            for (int t = max(half * 64, rq.base - tok0); t < min(half * 64 + 64, rq.len - tok0); ++t)
              if (s_vis[tid * 3 + (t >> 5 & 1)] >> (t & 31) & 1)
#pragma unroll
                for (int j = 0; j < D / 32; ++j) nan_cols[j] |= s_nan[(vb * 128 + t) * (D / 32) + j];
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(p_ready);
      }
      // ---- the piece's rows: the two halves' sums, D / 2 columns of O each
      s_half[tid] = l;
      wait_or_fail(o_done, (n - 1) & 1, fail);
      named_barrier_sync(1, kRowSoft);
      l += s_half[tid ^ 128];
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {   // a NaN that either half of the row saw
        s_vis[tid] = nan_cols[j];
        named_barrier_sync(1, kRowSoft);
        nan_cols[j] |= s_vis[tid ^ 128];
        named_barrier_sync(1, kRowSoft);
      }
      tc_fence_after();
      const bool whole = cur.n == cur.tiles;
      if (*fail) l = __int_as_float(0x7fc00000);
      if (node < 0) l = 0.f;
      float f = l == 0.f ? 0.f : whole ? v0 / l : v0;
      float2 ml = make_float2(m_run, l);
      if (!whole) ml = attn_partial(m_run, l, f);
      const int64_t at = (static_cast<int64_t>(cur.b) * a.N + my_at) * a.Hq + cur.h * a.G + (Rg - my_at * a.G);
      float* part = a.part + (static_cast<int64_t>(2 * cta + (cur.pos == lo ? 0 : 1)) * 128 + row) * kPitch;
      const bool mine = Rg < rows_total;
#pragma unroll
      for (int g = 0; g < D / 32; ++g) {
        const int d0 = half * (D / 2) + g * 16;
        uint32_t o[16];
        tmem_ld16(t_o + g * 16, o);
        tmem_ld_wait();
        tmem_use(o);
        float y[16];
        uint32_t bits = 0;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) bits = (d0 >> 5) == k ? nan_cols[k] : bits;
        bits >>= d0 & 31;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          y[j] = f == 0.f ? 0.f : __uint_as_float(o[j]) * f;
          if (bits >> j & 1) y[j] = __int_as_float(0x7fc00000);
        }
        if (mine && whole) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + (at * D + d0) * 2);
          dst[0] = make_uint4(T::pack2(y[0], y[1]), T::pack2(y[2], y[3]), T::pack2(y[4], y[5]), T::pack2(y[6], y[7]));
          dst[1] = make_uint4(T::pack2(y[8], y[9]), T::pack2(y[10], y[11]), T::pack2(y[12], y[13]), T::pack2(y[14], y[15]));
        } else if (mine) {
#pragma unroll
          for (int j = 0; j < 16; j += 4)
            *reinterpret_cast<float4*>(part + d0 + j) = make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
        }
      }
      if (mine && half == 0) {
        if (whole) {
          if (a.lse) a.lse[at] = l == 0.f ? -INFINITY : (m_run + log2f(l)) * kLn2;
        } else {
          *reinterpret_cast<float2*>(part + D) = ml;
        }
      }
      tc_fence_before();
      named_barrier_sync(1, kRowSoft);   // the shared rows are free for the next piece
    }
  }
  __syncthreads();
  if (s_fail) {   // a wait gave up: leave time for copies and products in flight before TMEM goes
    const uint64_t t = global_timer_ns();
    for (int i = 0; i < (1 << 20) && global_timer_ns() - t < 2000000; ++i) {
    }
  }
  __syncthreads();
  if (tid == 0) a.failed[cta] = s_fail;
  if (warp == 13) tmem_free(tmem, kRowTmem);
}

}  // namespace sv
