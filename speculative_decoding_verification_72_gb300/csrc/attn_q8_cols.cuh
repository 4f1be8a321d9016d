// Attention over the 8-bit cache for up to 32 rows a kv head (single tokens and
// short chains), on the tensor cores straight from the 8-bit codes.
//
// Codes need no conversion if both operands are e4m3, and q and P, which are
// not, are few here: they are split into sums of e4m3 terms instead,
//   q = qs (q1 + q2 / 32 [+ q3 / 1024]),  P = (p1 + p2 / 32 + p3 / 1024) / 4,
// each term the rounding of 32 times what the one before left. Two terms hold a
// bf16 q and three an f16 q exactly (down to 2^-14 of the row's maximum). P is
// rounded to f16 first, 2^-11 of its value at most, since packed f16 halves the
// instructions of the split; its three terms hold that exactly, or leave 2^-22 of
// the row's largest P. Sums of P (the softmax's) take it before it is rounded.
// The terms are columns of one product, with tokens as its 128 rows:
//   S^T [128 tokens, terms x rows] = K [tokens, D] q^T,
//   O^T [D, 3 x rows] += V^T [D, tokens] P.
// A tile of 128 tokens is the A operand of both, K as it lies (K-major), V
// transposed by the descriptor (MN-major), so each code goes from HBM by TMA
// into shared memory and from there into the tensor core, touched by no thread.
//
// Lane = token in S^T, so a thread has one token's scores for all rows: its
// page's scales are scalars, sums over tokens stay in its registers until the
// end, and P is one 16-byte store per 16 rows and term. The running maximum is
// raised only when a score exceeds it by 2^6 (a vote per tile), which takes the
// slow path: maxima across the CTA and a rescale of O^T in TMEM. So does every
// tile until each row has seen a position, as a row's first maximum may lie
// anywhere (the first positions of a piece may all be on no page).
//
// A token's vs is part of its exponent, P = 2^(s + log2 vs - m), with m the
// maximum of s + log2 vs: whatever the pages' scales, a row's P fills e4m3's
// range. The softmax's sum takes P / vs.
//
// 16 rows take one group of four softmax warps (a thread has one token and 16
// rows), 32 rows two groups, each with its own maxima, sums and columns; one
// warp issues TMA, one MMA. Two CTAs an SM, so one's softmax runs under the
// other's copies.
//
// A tile with new nodes, the end, or a missing page also takes the slow path:
// its V rows that are not positions are zeroed in shared memory (0 * NaN would
// reach every row), and NaN codes of nodes, which only some rows may see, are
// taken out and their rows and columns noted for the end.
//
// Work split, partials and their join are attn_q8.cuh's.
//
// Measured: 32 requests of 6 rows over up to 8192 tokens, 32 heads on 8 of 128,
// 339 MB: bf16 92 us, 3.7 TB/s, f16 89; one request of 1000 tokens, one row: 11
// us. The softmax is not the bound (without any, 89 us of what then were 95), nor
// are the pipes (tensor 15 %, exponentials 7 %, an instruction issued in half of
// the clocks): most warps wait for memory. A CTA has two stages each of K and V,
// which one warp fills in order, so that a V still in use holds back the next K,
// and it looks up pages and scales a tile at a time.
#pragma once

#include <cuda.h>

#include "attn_q8.cuh"
#include "tc_common.cuh"

namespace sv {

constexpr int kColTile = 128;
constexpr int kColTmem = 256;
constexpr float kColSlack = 6.f;     // log2 by which a term may exceed the running maximum: P <= 4 * 2^6 fits e4m3

template <int D, int MT, int NT>
struct ColLayout {
  static constexpr int R = 16 * MT;
  static constexpr int kThreads = 128 * MT + 64;
  static constexpr int kTileBytes = kColTile * D;
  static constexpr int kKs = D == 128 ? 2 : 4, kVs = kKs;          // ring depth
  static constexpr int kNs = NT * R, kNo = 3 * R;                  // columns of S^T and O^T
  static constexpr int kNb = 2 * kNs + kNo <= kColTmem ? 2 : 1;    // S^T buffers
  static constexpr int kQBytes = (kNs * D + 1023) / 1024 * 1024;
  static constexpr int kPBytes = kColTile * 128;
  // Two P tiles where two CTAs still fit an SM.
  static constexpr int kPb = 2 * kKs * kTileBytes + 2 * kPBytes + kQBytes <= 106 * 1024 ? 2 : 1;
  static constexpr int kOffV = kKs * kTileBytes;
  static constexpr int kOffP = kOffV + kVs * kTileBytes;
  static constexpr int kOffQ = kOffP + kPb * kPBytes;
  static constexpr int kOffMisc = kOffQ + kQBytes;
  static constexpr int kMiscBytes = MT * (16 * (7 + 5 + 4 + D / 32) * 4 + 64 * 4) + 1024 + 64;
  static constexpr int bytes(int words) { return 1024 + kOffMisc + kMiscBytes + R * words * 4; }
};

// f16x2 helpers of the P split.
__device__ __forceinline__ uint32_t e4m3x2_of_half2(uint32_t h2) {   // two codes in the low 16 bits
  uint32_t r;
  asm("{\n\t.reg .b16 c;\n\tcvt.rn.satfinite.e4m3x2.f16x2 c, %1;\n\tmov.b32 %0, {c, c};\n\t}" : "=r"(r) : "r"(h2));
  return r;
}
__device__ __forceinline__ uint32_t half2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t half2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <typename T, int D, int MT, int NT>
__global__ void __launch_bounds__(ColLayout<D, MT, NT>::kThreads, 2)
    attn_q8_cols_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map, const AttnArgs a) {
  using L = ColLayout<D, MT, NT>;
  constexpr int R = L::R;
  constexpr int kSoft = 128 * MT;   // softmax threads
  extern __shared__ uint8_t raw[];
  __shared__ AttnLine s_line;
  __shared__ int32_t s_warp[L::kThreads / 32];
  __shared__ __align__(8) uint64_t s_bar[2 * L::kKs + 2 * L::kVs + 2 * L::kNb + 2 * L::kPb + 1];
  __shared__ uint32_t s_tmem, s_fail;
  const uint32_t smem0 = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t* smem = raw + (smem0 - smem_u32(raw));
  // per group of 16 rows
  float* s_m0 = reinterpret_cast<float*>(smem + L::kOffMisc);          // [R] running maximum (log2)
  float* s_cq = s_m0 + R;                                               // [R] q's factor * coef
  float* s_up = s_cq + R;                                               // [R] what a slow path subtracts
  float* s_f = s_up + R;                                                // [R] and multiplies by
  int32_t* s_node = reinterpret_cast<int32_t*>(s_f + R);                // [R]
  int32_t* s_seen = s_node + R;                                         // [R] whether the row has seen a position
  float* s_max = reinterpret_cast<float*>(s_seen + R);                  // [4 MT][20]
  int4* s_out = reinterpret_cast<int4*>(s_max + 80 * MT);               // [R] where a row's output goes
  uint32_t* s_nan = reinterpret_cast<uint32_t*>(s_out + R);             // [R][D / 32]
  float4* s_sc = reinterpret_cast<float4*>(s_nan + R * (D / 32));       // [8 tiles][8 pages]: ks, vs, page there
  uint32_t* s_anc = reinterpret_cast<uint32_t*>(s_sc + 64);             // [R][words]

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t bar0 = smem_u32(s_bar);
  const uint32_t full_k = bar0, empty_k = full_k + 8 * L::kKs, full_v = empty_k + 8 * L::kKs, empty_v = full_v + 8 * L::kVs;
  const uint32_t s_ready = empty_v + 8 * L::kVs, s_free = s_ready + 8 * L::kNb;
  const uint32_t p_ready = s_free + 8 * L::kNb, p_free = p_ready + 8 * L::kPb, q_ready = p_free + 8 * L::kPb;
  if (tid == 0) {
    s_fail = 0;
    for (int i = 0; i < L::kKs; ++i) {
      mbar_init(full_k + 8 * i, 1);
      mbar_init(empty_k + 8 * i, 1);
      mbar_init(full_v + 8 * i, 1);
      mbar_init(empty_v + 8 * i, 1);
    }
    for (int i = 0; i < L::kNb; ++i) {
      mbar_init(s_ready + 8 * i, 1);
      mbar_init(s_free + 8 * i, 4 * MT);
    }
    for (int i = 0; i < L::kPb; ++i) {
      mbar_init(p_ready + 8 * i, kSoft);
      mbar_init(p_free + 8 * i, 1);
    }
    mbar_init(q_ready, kSoft);
    fence_barrier_init();
  }
  if (warp == 4 * MT + 1) tmem_alloc(smem_u32(&s_tmem), kColTmem);
  if (warp == 4 * MT && lane == 0) {
    tma_prefetch_map(&k_map);
    tma_prefetch_map(&v_map);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  grid_dep_wait();
  grid_dep_launch();
  const int ipr = a.c.Hkv * a.RB;
  const int cta = blockIdx.x;
  const AttnRanges ranges = attn_scan<L::kThreads>(
      a.B, [&](int r) { return attn_tiles<kColTile>(attn_req(a, r)); }, a.grid, cta, &s_line, s_warp, ipr, cta == 0 ? a.plan : nullptr);
  if (cta == 0 && tid == 0) a.plan[a.B] = s_line.total;
  const int lo = cta < ranges.n ? ranges.begin(cta) : 0, hi = cta < ranges.n ? ranges.begin(cta + 1) : 0;

  // Every role walks the same pieces; n counts tiles across them.
  AttnCursor cur;
  cur.start(a, s_line, lo);
  uint32_t n = 0;
  volatile uint32_t* fail = &s_fail;

  if (warp == 4 * MT) {
    // ------------------------------------------------------------------ TMA
    bool ok = true;
    const int boxes = kColTile >> a.c.page_shift;   // pages a tile
    const int box_bytes = D << a.c.page_shift;
    for (; ok && cur.pos < hi; cur.pos += cur.n) {
      cur.piece<kColTile>(a, hi, ipr);
      // Pages of a tile, one a lane, two tiles ahead; their scales, one tile
      // ahead, go to the softmax warps through shared memory with the codes.
      auto page_of = [&](int i) {
        const int tok = (cur.t0 + i) * kColTile + (lane << a.c.page_shift);
        return i < cur.n && lane < boxes && tok < cur.rq.len ? q8_page(a.c, cur.b, tok >> a.c.page_shift) : -1;
      };
      auto scales_of = [&](int p) {
        const int64_t o = static_cast<int64_t>(max(p, 0)) * a.c.Hkv + cur.h;
        return p >= 0 ? make_float4(a.c.ks[o], a.c.vs[o], 1.f, 0.f) : make_float4(0.f, 0.f, 0.f, 0.f);
      };
      int page = page_of(0), page1 = page_of(1);
      float4 sc = scales_of(page);
      float most = 0.f;
      for (int i = 0; i < cur.n; ++i, ++n) {
        const int page2 = page_of(i + 2);
        const float4 sc1 = scales_of(page1);
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, page >= 0)) * box_bytes;
        const int z = page * a.c.Hkv + cur.h;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          constexpr int kDepth = L::kKs;
          const uint32_t st = n % kDepth, ph = n / kDepth;
          if (lane == 0 && ph > 0) ok = wait_or_fail((kv ? empty_v : empty_k) + 8 * st, (ph - 1) & 1, fail);
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          if (kv == 0) {
            sc.y = attn_v_scale(sc.y, page >= 0, most);
            if (lane < 8) s_sc[(n & 7) * 8 + lane] = sc;
            __syncwarp();
          }
          if (lane == 0) mbar_arrive_expect_tx((kv ? full_v : full_k) + 8 * st, bytes);
          __syncwarp();
          if (page >= 0)
            tma_load_3d(smem0 + (kv ? L::kOffV : 0) + st * L::kTileBytes + lane * box_bytes, kv ? &v_map : &k_map, 0, z,
                        (kv ? full_v : full_k) + 8 * st);
        }
        if (!ok) break;
        page = page1;
        page1 = page2;
        sc = sc1;
      }
    }
  } else if (warp == 4 * MT + 1) {
    // ------------------------------------------------------------------ MMA
    if (lane == 0) {
      constexpr uint32_t kSw = D == 128 ? 2 : 4, kSbo = 8 * D;
      constexpr uint32_t kIdS = tc_idesc(0, false, false, 128, L::kNs), kIdO = tc_idesc(0, true, true, 128, L::kNo);
      bool ok = true;
      uint32_t pieces = 0;
      auto scores = [&](uint32_t m) {
        const uint32_t st = m % L::kKs, sb = m % L::kNb;
        ok = ok && wait_or_fail(full_k + 8 * st, (m / L::kKs) & 1, fail);
        if (m >= L::kNb) ok = ok && wait_or_fail(s_free + 8 * sb, (m / L::kNb - 1) & 1, fail);
        if (!ok) return;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
          tc_mma_f8(tmem + sb * L::kNs, tc_desc(smem0 + st * L::kTileBytes + 32 * k, 16, kSbo, kSw),
                    tc_desc(smem0 + L::kOffQ + 32 * k, 16, kSbo, kSw), kIdS, k > 0);
        tc_commit(empty_k + 8 * st);
        tc_commit(s_ready + 8 * sb);
      };
      for (; ok && cur.pos < hi; cur.pos += cur.n) {
        cur.piece<kColTile>(a, hi, ipr);
        ok = wait_or_fail(q_ready, pieces++ & 1, fail);
        if (!ok) break;
        scores(n);
        for (int i = 0; i < cur.n && ok; ++i, ++n) {
          if (i + 1 < cur.n) scores(n + 1);
          const uint32_t st = n % L::kVs;
          ok = ok && wait_or_fail(full_v + 8 * st, (n / L::kVs) & 1, fail) && wait_or_fail(p_ready + 8 * (n % L::kPb), (n / L::kPb) & 1, fail);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < kColTile / 32; ++k)
            tc_mma_f8(tmem + L::kNb * L::kNs, tc_desc(smem0 + L::kOffV + st * L::kTileBytes + 32 * D * k, 0, kSbo, kSw),
                      tc_desc(smem0 + L::kOffP + (n % L::kPb) * L::kPBytes + 4096 * k, 0, 1024, 2), kIdO, i > 0 || k > 0);
          tc_commit(empty_v + 8 * st);
          tc_commit(p_free + 8 * (n % L::kPb));
        }
      }
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- softmax
    const int grp = warp >> 2, row = tid & 127, r00 = grp * 16;   // the thread's rows r00 .. r00 + 15, token `row` of a tile
    const uint32_t t_lane = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t t_o = t_lane + L::kNb * L::kNs + r00;
    const int bar = 1 + grp;
    const int rows_total = a.N * a.G, words = (a.N + 31) / 32;
    float* max_w = s_max + warp * 20;
    const float* max_g = s_max + grp * 80;
    uint32_t* unseen = reinterpret_cast<uint32_t*>(s_max + grp * 80 + 16);   // whether a row with a node has seen no position yet
    // A wait that gives up ends no loop here: these warps meet at barriers, so all
    // run on to the end (every later wait then returns at once), without meaning:
    // the rows of every piece that ends after it are NaN.
    for (; cur.pos < hi; cur.pos += cur.n) {
      cur.piece<kColTile>(a, hi, ipr);
      const AttnReq rq = cur.rq;
      const int row0 = cur.rb * R;
      const int node0 = attn_node(a, row0);
      // ---- q as e4m3 terms, one warp a row
      const uint8_t* q = a.q + cur.b * a.sqb + static_cast<int64_t>(cur.h) * a.G * a.sqh;
#pragma unroll 4
      for (int r = warp; r < R; r += 4 * MT) {
        const int Rg = row0 + r, at = attn_node(a, Rg);
        const int node = Rg < rows_total && at < rq.n ? at : -1;
        float f[4] = {0.f, 0.f, 0.f, 0.f};
        if (node >= 0 && lane * 4 < D) T::load4(q + node * a.sqn + (Rg - node * a.G) * a.sqh + lane * 8, f);
        const float m = warp_max(fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3]))));
        // the row's maximum into [2^7, 2^8)
        const int e = m > 0.f ? static_cast<int>(__float_as_uint(m) >> 23) - 127 : 7;
        const int x = min(max(7 - e, -126), 126);
        const float up = exp2_int(x);
        if (lane * 4 < D) {
#pragma unroll
          for (int i = 0; i < 4; ++i) f[i] *= up;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint32_t w = e4m3_pack4(f[0], f[1], f[2], f[3]);
            const float2 x0 = half2_bits(e4m3x2_lo(w)), x1 = half2_bits(e4m3x2_hi(w));
            f[0] = (f[0] - x0.x) * 32.f;
            f[1] = (f[1] - x0.y) * 32.f;
            f[2] = (f[2] - x1.x) * 32.f;
            f[3] = (f[3] - x1.y) * 32.f;
            *reinterpret_cast<uint32_t*>(smem + L::kOffQ + unit_off<D>(t * R + r, lane >> 2) + (lane & 3) * 4) = w;
          }
        }
        if (lane == 0) {
          // Infinities saturate in e4m3, so the factor makes their row NaN (NaN codes stay NaN).
          s_cq[r] = m == INFINITY ? __int_as_float(0x7fc00000) : exp2_int(-x) * a.coef;
          s_node[r] = node;
          s_m0[r] = 0.f;
          s_seen[r] = 0;
        }
      }
      for (int i = tid; i < R * (D / 32); i += kSoft) s_nan[i] = 0;
      if (row == 0) *unseen = 1;
      const bool tail = (cur.t0 + cur.n) * kColTile > rq.base;
      if (tail && a.parents) {
        const int nodes = min(attn_node(a, row0 + R - 1), a.N - 1) - node0 + 1;
        for (int i = tid; i < nodes * words; i += kSoft) s_anc[i] = 0;
        named_barrier_sync(3, kSoft);
        const int32_t* par = a.parents + static_cast<int64_t>(cur.b) * a.N;
        for (int i = tid; i < nodes; i += kSoft) {
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
      named_barrier_sync(3, kSoft);
      const uint32_t live = __ballot_sync(0xffffffffu, lane < 16 && s_node[r00 + (lane & 15)] >= 0);   // rows with a node

      float2 l[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) l[r] = make_float2(0.f, 0.f);
      float v0 = 1.f, iv0 = 1.f;
      bool any_nan = false;
      // The products of tile m have read its P.
      auto p_done = [&](uint32_t m) { wait_or_fail(p_free + 8 * (m % L::kPb), (m / L::kPb) & 1, fail); };
#pragma unroll 1
      for (int i = 0; i < cur.n; ++i, ++n) {
        const int tok = (cur.t0 + i) * kColTile + row;
        const bool edge = (cur.t0 + i + 1) * kColTile > rq.base;
        const uint32_t sb = n % L::kNb;
        wait_or_fail(s_ready + 8 * sb, (n / L::kNb) & 1, fail);
        tc_fence_after();
        uint32_t w[NT][16];
#pragma unroll
        for (int t = 0; t < NT; ++t) tmem_ld16(t_lane + sb * L::kNs + t * R + r00, w[t]);
        const float4 sc = s_sc[(n & 7) * 8 + (row >> a.c.page_shift)];
        const float ks = sc.x, vs = sc.y;
        const bool valid = sc.z != 0.f && tok < rq.len;
        if (i == 0) {   // scales relative to the piece's first, so that sums of P / vs stay in fp32's range
          v0 = s_sc[(n & 7) * 8].y;
          v0 = v0 > 0.f && v0 < INFINITY ? v0 : 1.f;
          iv0 = 1.f / v0;
        }
        // P / 4 relative to v0 = 2^x with x = score + log2(vs / v0) + 2 - maximum
        const float rel = vs * iv0;
        const float lv = rel == rel ? fmaxf(lg2(rel), -100.f) : rel, iv = ex2(-lv) * 0.25f;
        const float2 lv2 = make_float2(lv + 2.f, lv + 2.f), ks2 = make_float2(ks, ks);
        tmem_ld_wait();
#pragma unroll
        for (int t = 0; t < NT; ++t) tmem_use(w[t]);
        tc_fence_before();
        if (lane == 0) mbar_arrive(s_free + 8 * sb);
        float2 x[8];
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 mm = reinterpret_cast<const float4*>(s_m0 + r00)[j], cc = reinterpret_cast<const float4*>(s_cq + r00)[j];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int r = j * 4 + k * 2;
            float2 v = make_float2(__uint_as_float(w[NT - 1][r]), __uint_as_float(w[NT - 1][r + 1]));
#pragma unroll
            for (int t = NT - 2; t >= 0; --t)
              v = __ffma2_rn(v, make_float2(1.f / 32.f, 1.f / 32.f),
                             make_float2(__uint_as_float(w[t][r]), __uint_as_float(w[t][r + 1])));
            const float2 c = __fmul2_rn(k ? make_float2(cc.z, cc.w) : make_float2(cc.x, cc.y), ks2);
            const float2 s = __fadd2_rn(lv2, k ? make_float2(-mm.z, -mm.w) : make_float2(-mm.x, -mm.y));
            x[r / 2] = __ffma2_rn(v, c, s);
            top = fmaxf(fmaxf(top, x[r / 2].x), x[r / 2].y);
          }
        }
        if (named_barrier_or(bar, 128, top > kColSlack + 2.f || !valid || edge || *unseen)) {
          // ---- slow path: masks, maxima, V rows that must not be read
          uint32_t see = valid ? 0xffffu : 0u;
          const bool special = named_barrier_or(bar, 128, edge || !valid);   // the same for every group
          if (special && edge) {
            const int m = tok - rq.base;   // the token's node, negative in the prefix
            see = m < rq.n ? see & live : 0u;
            if (m >= 0 && see) {
              uint32_t bits = 0;
#pragma unroll 1
              for (int r = 0; r < 16; ++r) {
                const int node = s_node[r00 + r];
                bool on = m <= node;
                if (on && a.parents) on = s_anc[(node - node0) * words + (m >> 5)] >> (m & 31) & 1;
                bits |= static_cast<uint32_t>(on) << r;
              }
              see &= bits;
            }
          }
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            float& v = r & 1 ? x[r / 2].y : x[r / 2].x;
            if (!(see >> r & 1)) v = -INFINITY;
            const float mx = warp_max(v);
            if (lane == 0) max_w[r] = mx;
          }
          if (special) {
            wait_or_fail(full_v + 8 * (n % L::kVs), (n / L::kVs) & 1, fail);
            uint8_t* vrow = smem + L::kOffV + (n % L::kVs) * L::kTileBytes;
            uint32_t nans = 0;   // 16-byte chunks of the token's V row with NaN codes
            if (valid && tok >= rq.base) {
#pragma unroll
              for (int ch = 0; ch < D / 16; ++ch) {
                const uint4 w = *reinterpret_cast<const uint4*>(vrow + unit_off<D>(row, ch));
                const uint32_t bad = ((w.x & 0x7f7f7f7fu) + 0x01010101u) | ((w.y & 0x7f7f7f7fu) + 0x01010101u) |
                                     ((w.z & 0x7f7f7f7fu) + 0x01010101u) | ((w.w & 0x7f7f7f7fu) + 0x01010101u);
                nans |= static_cast<uint32_t>((bad & 0x80808080u) != 0) << ch;
              }
              any_nan = any_nan || nans != 0;
#pragma unroll 1
              for (int ch = 0; ch < D / 16; ++ch) {
                if (!(nans >> ch & 1)) continue;
                const uint32_t* p = reinterpret_cast<const uint32_t*>(vrow + unit_off<D>(row, ch));
                for (int j = 0; j < 4; ++j) {
                  const uint32_t bad = ((p[j] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                  const int d = ch * 16 + j * 4;
                  const uint32_t bits = (bad >> 7 & 1) | (bad >> 14 & 2) | (bad >> 21 & 4) | (bad >> 28 & 8);
                  for (int r = 0; r < 16; ++r)
                    if (bits && (see >> r & 1)) atomicOr(&s_nan[(r00 + r) * (D / 32) + (d >> 5)], bits << (d & 31));
                }
              }
            }
            named_barrier_sync(3, kSoft);   // every group has read the row, and its maxima are there
            if (grp == 0) {
              if (!valid) {
#pragma unroll
                for (int ch = 0; ch < D / 16; ++ch) *reinterpret_cast<uint4*>(vrow + unit_off<D>(row, ch)) = make_uint4(0, 0, 0, 0);
              }
#pragma unroll 1
              for (int ch = 0; nans; ++ch, nans >>= 1) {
                if (!(nans & 1)) continue;
                uint32_t* p = reinterpret_cast<uint32_t*>(vrow + unit_off<D>(row, ch));
                for (int j = 0; j < 4; ++j) {
                  const uint32_t bad = ((p[j] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                  p[j] &= ~((bad >> 7) * 0xffu);
                }
              }
            }
            fence_async_smem();
          } else {
            named_barrier_sync(bar, 128);
          }
          // one thread per row: by how much its maximum rises; a row's first maximum may lie anywhere
          if (row < 16) {
            const float mx = fmaxf(fmaxf(max_g[row], max_g[20 + row]), fmaxf(max_g[40 + row], max_g[60 + row])) - 2.f;
            const bool seen = s_seen[r00 + row];
            const float up = seen ? fmaxf(mx, 0.f) : mx == -INFINITY ? 0.f : mx;
            s_up[r00 + row] = up;
            s_f[r00 + row] = seen ? ex2(-up) : 1.f;
            s_m0[r00 + row] += up;
            s_seen[r00 + row] = seen || mx != -INFINITY;
            const uint32_t none = __ballot_sync(0xffffu, s_node[r00 + row] >= 0 && !seen && mx == -INFINITY);
            if (row == 0) *unseen = none;
          }
          const bool changed = named_barrier_or(bar, 128, row < 16 && s_f[r00 + (row & 15)] != 1.f);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 up = reinterpret_cast<const float2*>(s_up + r00)[j];
            x[j].x -= up.x;
            x[j].y -= up.y;
          }
          if (changed) {   // no row has seen anything before the first tile
#pragma unroll
            for (int j = 0; j < 8; ++j) l[j] = __fmul2_rn(l[j], reinterpret_cast<const float2*>(s_f + r00)[j]);
            p_done(n - 1);
            tc_fence_after();
#pragma unroll 1
            for (int t = 0; t < 3; ++t) {
              uint32_t v[16];
              tmem_ld16(t_o + t * R, v);
              tmem_ld_wait();
              tmem_use(v);
#pragma unroll
              for (int r = 0; r < 16; ++r) v[r] = __float_as_uint(__uint_as_float(v[r]) * s_f[r00 + r]);
              tmem_st16(t_o + t * R, v);
            }
            tmem_st_wait();
          }
        }
        // ---- P, its sum and its terms
        uint32_t h[8];
        const float2 iv2 = make_float2(iv, iv);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 p = make_float2(ex2(x[j].x), ex2(x[j].y));
          l[j] = __ffma2_rn(p, iv2, l[j]);
          h[j] = pack_half2(p.x, p.y);
        }
        if (n >= L::kPb) p_done(n - L::kPb);
#pragma unroll
        for (int t = 0; t < 3; ++t) {
          uint32_t c[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t c0 = e4m3x2_of_half2(h[2 * j]), c1 = e4m3x2_of_half2(h[2 * j + 1]);
            c[j] = __byte_perm(c0, c1, 0x5410);
            if (t < 2) {   // h = 32 (h - code), exact in f16
              h[2 * j] = half2_fma(e4m3x2_lo(c0), 0xd000d000u, half2_mul(h[2 * j], 0x50005000u));
              h[2 * j + 1] = half2_fma(e4m3x2_lo(c1), 0xd000d000u, half2_mul(h[2 * j + 1], 0x50005000u));
            }
          }
          const int ch = (t * R + r00) / 16;
          *reinterpret_cast<uint4*>(smem + L::kOffP + (n % L::kPb) * L::kPBytes + row * 128 + ((ch ^ (row & 7)) << 4)) = make_uint4(c[0], c[1], c[2], c[3]);
        }
        tc_fence_before();
        fence_async_smem();
        mbar_arrive(p_ready + 8 * (n % L::kPb));
      }
      // ---- the piece's sums and O^T
      p_done(n - 1);
      any_nan = named_barrier_or(bar, 128, any_nan);
      {
        // 16 sums over 32 lanes: halve the rows a lane holds, then the lanes; lane 2 r ends with row r
        float v[16];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          v[2 * r] = l[r].x;
          v[2 * r + 1] = l[r].y;
        }
#pragma unroll
        for (int o = 16, k = 8; o > 1; o >>= 1, k >>= 1) {
#pragma unroll
          for (int r = 0; r < k; ++r) {
            const bool up = lane & o;
            const float give = up ? v[r] : v[r + k], keep = up ? v[r + k] : v[r];
            v[r] = keep + __shfl_xor_sync(0xffffffffu, give, o);
          }
        }
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
        if (!(lane & 1)) max_w[lane >> 1] = v[0];
      }
      named_barrier_sync(bar, 128);
      const bool whole = cur.n == cur.tiles;
      float* part = a.part + static_cast<int64_t>(2 * cta + (cur.pos == lo ? 0 : 1)) * R * AttnLayout<D>::kPitch;
      if (row < 16) {
        const int r = r00 + row, Rg = row0 + r, node = attn_node(a, Rg);
        const float sum = s_node[r] < 0 ? 0.f
                          : *fail       ? __int_as_float(0x7fc00000)
                                        : (max_g[row] + max_g[20 + row]) + (max_g[40 + row] + max_g[60 + row]);
        const int64_t at = (static_cast<int64_t>(cur.b) * a.N + node) * a.Hq + cur.h * a.G + (Rg - node * a.G);
        float f = sum == 0.f ? 0.f : 0.25f * v0;   // a row that saw nothing is zero
        if (Rg < rows_total) {
          if (whole) {
            if (a.lse) a.lse[at] = sum == 0.f ? -INFINITY : (s_m0[r] + log2f(sum)) * kLn2;
          } else {
            *reinterpret_cast<float2*>(part + r * AttnLayout<D>::kPitch + D) = attn_partial(s_m0[r], sum, f);
          }
        }
        s_out[r] = make_int4(static_cast<int>(at & 0xffffffff), static_cast<int>(at >> 32),
                             __float_as_int(whole && sum != 0.f ? f / sum : f), Rg < rows_total);
      }
      named_barrier_sync(bar, 128);
      tc_fence_after();
      if (row < D) {
        uint32_t w[3][16];
#pragma unroll
        for (int t = 0; t < 3; ++t) tmem_ld16(t_o + t * R, w[t]);
        tmem_ld_wait();
#pragma unroll
        for (int t = 0; t < 3; ++t) tmem_use(w[t]);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int r = r00 + j;
          const int4 to = s_out[r];
          if (!to.w) break;
          float o = fmaf(fmaf(__uint_as_float(w[2][j]), 1.f / 32.f, __uint_as_float(w[1][j])), 1.f / 32.f, __uint_as_float(w[0][j]));
          const float f = __int_as_float(to.z);
          o = f == 0.f ? 0.f : o * f;
          if (any_nan && (s_nan[r * (D / 32) + (row >> 5)] >> (row & 31) & 1)) o = __int_as_float(0x7fc00000);
          if (whole) {
            const int64_t at = static_cast<uint32_t>(to.x) | static_cast<int64_t>(to.y) << 32;
            static_cast<uint16_t*>(a.out)[at * D + row] = static_cast<uint16_t>(T::pack2(o, 0.f));
          } else {
            part[r * AttnLayout<D>::kPitch + row] = o;
          }
        }
      }
      tc_fence_before();
      named_barrier_sync(3, kSoft);   // the shared rows are free for the next piece
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
  if (warp == 4 * MT + 1) tmem_free(tmem, kColTmem);
}

}  // namespace sv
