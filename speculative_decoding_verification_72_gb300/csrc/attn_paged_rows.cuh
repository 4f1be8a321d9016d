// Attention over the 16-bit cache for many rows a kv head (draft trees,
// prompts), bound by the tensor cores and the exponentials.
//
// A block is 256 rows of one kv head as two halves of 128 lanes that share K
// and V; for each half g
//   S_g [128 rows, 128 tokens] = q_g K^T,   O_g [128 rows, D] += P_g V,
// K and V as TMA brings them (V transposed by the descriptor), P_g in the type
// of V over the columns of S_g in TMEM. Per tile and half the products take
// 8 D clocks and the 128 x 128 exponentials 1024 (16 a clock), so one half's
// softmax runs under the other's products: the MMA warp issues PV_0, S_0 of the
// next tile, PV_1, S_1 in turn. S and O of both halves fill all 512 columns of
// TMEM; one CTA an SM.
//
// A thread has one row, so maximum, exponentials and sum are its own. It reads
// its 128 scores 64 at a time: the first for the maximum alone, the second for
// maximum and exponentials, then the first again; all 128 at once do not fit its
// registers. The running maximum is raised only
// when a score exceeds it by 2^8; the warp then rescales its rows of O, which no
// product touches between S's arrival and P's. P is rounded to 16 bits (half a
// step of the type: 2^-8 of a bf16 weight, 2^-11 of f16's), its sum is not.
//
// A tile that some row does not see whole is masked in registers by 128 bits that
// the thread works out from its row's position and path.
//
// Warps 0-3 and 4-7: softmax. 8: TMA. 9: MMA.
#pragma once

#include "attn_paged_cols.cuh"
#include "attn_q8_rows.cuh"

namespace sv {

constexpr int kPgRowThreads = 320;
constexpr int kPgRowBlock = 256;

template <int D>
struct PgRowLayout {
  static constexpr int kTileBytes = kPgTile * D * 2;
  static constexpr int kStages = 128 * 1024 / kTileBytes;
  static constexpr int kOffQ = kStages * kTileBytes;                     // [2 halves][128 rows]
  static constexpr int kOffMisc = kOffQ + 2 * kTileBytes;
  // V's non-finite columns by token (two tiles), by row; parents and depths of the nodes
  static constexpr int kMiscBytes = 2 * 128 * (D / 16) * 4 + kPgRowBlock * (D / 16) * 4 + SV_MAX_TREE_NODES * 4 + kPgTile * 4;
  static constexpr int kBytes = 1024 + kOffMisc + kMiscBytes;
};

__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
        "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}

// The bits below bit x of a word.
__device__ __forceinline__ uint32_t below(int x) { return x <= 0 ? 0u : x >= 32 ? 0xffffffffu : (1u << x) - 1u; }

// What was taken out of the tokens of a tile that a row sees, into the row's flags.
template <int D>
__device__ __noinline__ void note_seen(const uint32_t* flags, uint32_t s0, uint32_t s1, uint32_t s2, uint32_t s3, uint32_t* to) {
  const uint32_t see[4] = {s0, s1, s2, s3};
  for (int t = 0; t < kPgTile; ++t)
    if (see[t >> 5] >> (t & 31) & 1)
      for (int w = 0; w < D / 16; ++w) to[w] |= flags[t * (D / 16) + w];
}

// kVar: scores are capped or biased.
template <typename T, int D, bool kVar>
__global__ void __launch_bounds__(kPgRowThreads, 1)
    attn_paged_rows_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map, const PagedAttnArgs a) {
  using L = PgRowLayout<D>;
  constexpr int kSt = L::kStages;
  extern __shared__ uint8_t raw[];
  __shared__ AttnLine s_line;
  __shared__ int32_t s_warp[kPgRowThreads / 32];
  __shared__ __align__(8) uint64_t s_bar[2 * kSt + 7];
  __shared__ uint32_t s_tmem, s_fail, s_there[16];
  const uint32_t smem0 = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t* smem = raw + (smem0 - smem_u32(raw));
  uint32_t* s_tok = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);     // [2][128][2][D / 32] columns with +inf, -inf (NaN: both)
  uint32_t* s_row = s_tok + 2 * 128 * (D / 16);                          // [256][2][D / 32]
  int16_t* s_par = reinterpret_cast<int16_t*>(s_row + kPgRowBlock * (D / 16));   // [nodes]
  int16_t* s_depth = s_par + SV_MAX_TREE_NODES;                          // [nodes]
  float* s_at = reinterpret_cast<float*>(s_depth + SV_MAX_TREE_NODES);   // [128] positions of a tile's tokens

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t full = smem_u32(s_bar), empty = full + 8 * kSt, s_ready = empty + 8 * kSt, p_ready = s_ready + 16;
  const uint32_t o_done = p_ready + 16, q_ready = o_done + 16;
  if (tid == 0) {
    s_fail = 0;
    for (int i = 0; i < kSt; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_ready + 8 * i, 1);
      mbar_init(p_ready + 8 * i, 128);
      mbar_init(o_done + 8 * i, 1);
    }
    mbar_init(q_ready, 256);
    fence_barrier_init();
  }
  if (warp == 9) tmem_alloc(smem_u32(&s_tmem), 512);
  if (warp == 8 && lane == 0) {
    tma_prefetch_map(&k_map);
    tma_prefetch_map(&v_map);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  grid_dep_wait();
  grid_dep_launch();
  int32_t lo, hi;
  paged_line<kPgRowThreads>(a, &s_line, s_warp, lo, hi);
  PagedCursor cur;   // every role walks the same pieces; n counts tiles across them
  cur.start(a, s_line, lo);
  uint32_t n = 0;
  volatile uint32_t* fail = &s_fail;
  const int rows_total = a.N * a.G;
  // Halves of a block that have rows.
  auto halves = [&](int block) { return rows_total - block * kPgRowBlock > 128 ? 2 : 1; };

  if (warp == 8) {
    paged_load<D, kSt>(a, &k_map, &v_map, cur, hi, smem0, full, empty, s_there, fail);
  } else if (warp == 9) {
    // ------------------------------------------------------------------ MMA
    if (lane == 0) {
      constexpr uint32_t kIdS = tc_idesc(T::kMma, false, false, 128, 128), kIdO = tc_idesc(T::kMma, false, true, 128, D);
      bool ok = true;
      uint32_t pieces = 0, done[2] = {0, 0};   // done: tiles of each half whose P has been awaited
      auto scores = [&](uint32_t m, int g, bool last) {
        const uint32_t s = 2 * m, st = s % kSt;
        if (g == 0) ok = ok && wait_or_fail(full + 8 * st, (s / kSt) & 1, fail);
        if (!ok) return;
        tc_fence_after();
        const uint32_t qt = smem0 + L::kOffQ + g * L::kTileBytes, kt = smem0 + st * L::kTileBytes;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc_mma_f16(tmem + g * 128, tc_desc(qt + (k >> 2) * (kPgTile * 128) + (k & 3) * 32, 16, 1024, 2),
                     tc_desc(kt + (k >> 2) * (kPgTile * 128) + (k & 3) * 32, 16, 1024, 2), kIdS, k > 0);
        tc_commit(s_ready + 8 * g);
        if (last) tc_commit(empty + 8 * st);
      };
      for (; ok && cur.pos < hi; cur.pos += cur.n) {
        cur.piece(a, hi);
        const int gs = halves(cur.block);
        ok = wait_or_fail(q_ready, pieces++ & 1, fail);
        for (int g = 0; g < gs && ok; ++g) scores(n, g, g + 1 == gs);
        for (int i = 0; i < cur.n && ok; ++i, ++n) {
          const uint32_t s = 2 * n + 1, st = s % kSt, vt = smem0 + st * L::kTileBytes;
          for (int g = 0; g < gs && ok; ++g) {
            if (g == 0) ok = wait_or_fail(full + 8 * st, (s / kSt) & 1, fail);
            ok = ok && wait_or_fail(p_ready + 8 * g, done[g]++ & 1, fail);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < kPgTile / 16; ++k)   // P's halves lie where those of S did
              tc_mma_f16_ts(tmem + 256 + g * 128, tmem + g * 128 + (k & 3) * 8 + (k >> 2) * 64,
                            tc_desc(vt + 2048 * k, kPgTile * 128, 1024, 2), kIdO, i > 0 || k > 0);
            if (g + 1 == gs) tc_commit(empty + 8 * st);
            // The next S overwrites this P: products of one CTA run in the order they are issued.
            if (i + 1 < cur.n)
              scores(n + 1, g, g + 1 == gs);
            else
              tc_commit(o_done + 8 * g);
          }
        }
      }
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- softmax
    const int g = warp >> 2, row = tid & 127;   // the thread's half, its row of it
    const uint32_t t_lane = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t t_s = t_lane + g * 128, t_o = t_lane + 256 + g * 128;
    uint8_t* qt = smem + L::kOffQ + g * L::kTileBytes;
    uint32_t tiles_done = 0, pieces = 0;   // of this half
    // A wait that gives up ends no loop here: these warps meet at barriers, so all
    // run on to the end (every later wait then returns at once), without meaning:
    // the rows of every piece that ends after it are NaN.
    for (; cur.pos < hi; cur.pos += cur.n) {
      cur.piece(a, hi);
      if (cur.pos == lo && tid == 0) a.first[blockIdx.x] = cur.item(a);
      const PagedReq rq = cur.rq;
      const int gs = halves(cur.block), soft = 128 * gs;
      const int row0 = cur.block * kPgRowBlock + g * 128;
      if (g >= gs) {
        n += cur.n;
        named_barrier_sync(4, kRowSoft);
        continue;
      }
      // ---- q, D / 8 lanes a row
      const uint8_t* q = a.q + cur.b * a.sqb + static_cast<int64_t>(cur.h) * a.G * a.sqh;
#pragma unroll 4
      for (int i = row; i < 128 * (D / 8); i += 128) {
        const int r = i / (D / 8), ch = i % (D / 8), Rg = row0 + r, node = paged_node(a, Rg);
        uint4 w = make_uint4(0, 0, 0, 0);
        if (Rg < rows_total && node < rq.n) w = *reinterpret_cast<const uint4*>(q + node * a.sqn + (Rg - node * a.G) * a.sqh + ch * 16);
        if (a.coef < 0.f) {   // scores grow with S
          w.x ^= 0x80008000u;
          w.y ^= 0x80008000u;
          w.z ^= 0x80008000u;
          w.w ^= 0x80008000u;
        }
        *reinterpret_cast<uint4*>(qt + block_off(128, r, ch)) = w;
      }
      fence_async_smem();
      mbar_arrive(q_ready);
      if (gs == 1) mbar_arrive(q_ready);   // for the other half's thread
      // ---- the thread's row, the request's tree
      const int Rg = row0 + row, at = paged_node(a, Rg);
      const int node = Rg < rows_total && at < rq.n ? at : -1;
      int depth = max(node, 0);
#pragma unroll
      for (int j = 0; j < D / 16; ++j) s_row[(g * 128 + row) * (D / 16) + j] = 0;
      if (a.parents) {
        const int32_t* par = a.parents + static_cast<int64_t>(cur.b) * a.N;
        for (int i = tid; i < rq.n; i += soft) s_par[i] = static_cast<int16_t>(tree_up(par, i));
        named_barrier_sync(1, soft);
        for (int i = tid; i < rq.n; i += soft) {
          int d = 0;
          for (int m = s_par[i]; m >= 0; m = s_par[m]) ++d;
          s_depth[i] = static_cast<int16_t>(d);
        }
        named_barrier_sync(1, soft);
        depth = s_depth[max(node, 0)];
      }
      const int pos = rq.base + depth;
      const float slope = kVar && a.slopes && node >= 0 ? a.slopes[cur.h * a.G + Rg - at * a.G] * kLog2e : 0.f;
      const float coef = fabsf(a.coef);
      const int open = max(pos - a.window + 1, 0);   // the window's first position
      const int pos0 = rq.base;   // positions relative to it are small enough for fp32

      float m_run = 0.f, l = 0.f;   // m_run means something once the row has seen a slot
      bool seen = false;
#pragma unroll 1
      for (int i = 0; i < cur.n; ++i, ++n, ++tiles_done) {
        const int tok0 = (cur.t0 + i) * kPgTile;
        wait_or_fail(s_ready + 8 * g, tiles_done & 1, fail);   // and every product before this S is done
        tc_fence_after();
        const uint32_t there = s_there[n & 15];
        const bool special = cur.special(a, tok0, there);
        uint32_t see[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};   // what the row sees of the tile
        if (special) {
          if (a.parents) {
#pragma unroll
            for (int j = 0; j < 4; ++j) see[j] = below(rq.base - tok0 - 32 * j);
            int far = 0;
            for (int m = node; m >= 0 && far < a.window; m = s_par[m], ++far) {
              const int c = rq.base + m - tok0;
              if (c < 0) break;   // parents come before
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (c >> 5 == j) see[j] |= 1u << (c & 31);
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int c = tok0 + 32 * j;
            if (!a.parents) see[j] = below(rq.base + node + 1 - c);
            const uint32_t prefix = a.parents ? below(rq.base - c) : 0xffffffffu;   // slots whose positions are their places
            see[j] &= below(rq.len - c) & ~(prefix & below(open - c));
            if (!(there >> (32 * j >> a.c.page_shift) & 1)) see[j] &= 0xffff0000u;
            if (!(there >> ((32 * j + 16) >> a.c.page_shift) & 1)) see[j] &= 0x0000ffffu;
            if (node < 0) see[j] = 0;
          }
          // ---- V's rows that must not be read, the same for every row
          const uint32_t s = 2 * n + 1, st = s % kSt;
          wait_or_fail(full + 8 * st, (s / kSt) & 1, fail);
          uint8_t* vt = smem + st * L::kTileBytes;
          const bool valid = there >> (row >> a.c.page_shift) & 1 && tok0 + row < rq.len;
          uint32_t odd = 0;
#pragma unroll
          for (int ch = 0; ch < D / 8; ++ch) {
            if (gs == 2 && ch / (D / 16) != g) continue;   // the thread's pieces of token `row`
            uint4* p = reinterpret_cast<uint4*>(vt + block_off(kPgTile, row, ch));
            if (valid)
              odd |= nonfinite8<T>(*p);
            else
              *p = make_uint4(0, 0, 0, 0);
          }
          if (named_barrier_or(1, soft, odd != 0)) {   // rare
            uint32_t* flags = s_tok + (n & 1) * 128 * (D / 16);
            for (int ch = gs == 2 ? g * (D / 16) : 0; ch < (gs == 2 ? (g + 1) * (D / 16) : D / 8); ++ch) {
              const uint32_t f = valid ? take_out8<T>(reinterpret_cast<uint4*>(vt + block_off(kPgTile, row, ch))) : 0u;
              uint8_t* to = reinterpret_cast<uint8_t*>(flags + row * (D / 16)) + ch;
              to[0] = static_cast<uint8_t>(f);
              to[D / 8] = static_cast<uint8_t>(f >> 8);
            }
            named_barrier_sync(1, soft);
            note_seen<D>(flags, see[0], see[1], see[2], see[3], s_row + (g * 128 + row) * (D / 16));
          }
          fence_async_smem();
          if (kVar && a.slopes && a.parents) {
            named_barrier_sync(1, soft);   // every row has read the last such tile's positions
            const int m = tok0 + row - rq.base;
            if (g == 0) s_at[row] = static_cast<float>(m >= 0 && m < rq.n ? rq.base + s_depth[m] - pos0 : tok0 + row - pos0);
            named_barrier_sync(1, soft);
          }
          __syncwarp();
        }
        // ---- 64 scores, in units of log2
        const float c = kVar ? 1.f : coef;
        auto scores = [&](uint32_t (&w)[64], int half) {
          tmem_ld32(t_s + half * 64, w);
          tmem_ld32(t_s + half * 64 + 32, w + 32);
          tmem_ld_wait();
          tmem_use(w);
          if (kVar) {
            if (a.cap != 0.f) {
#pragma unroll
              for (int j = 0; j < 64; ++j) {
                float r;
                asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2(__uint_as_float(w[j]) * coef)));
                w[j] = __float_as_uint(fmaf(-2.f * a.cap, r, a.cap));
              }
            } else {
#pragma unroll
              for (int j = 0; j < 64; ++j) w[j] = __float_as_uint(__uint_as_float(w[j]) * coef);
            }
            if (a.slopes) {
              if (special && a.parents) {
                const float off = static_cast<float>(pos0 - pos);
#pragma unroll
                for (int j = 0; j < 64; j += 4) {
                  const float4 at4 = *reinterpret_cast<const float4*>(s_at + half * 64 + j);
                  w[j] = __float_as_uint(fmaf(slope, at4.x + off, __uint_as_float(w[j])));
                  w[j + 1] = __float_as_uint(fmaf(slope, at4.y + off, __uint_as_float(w[j + 1])));
                  w[j + 2] = __float_as_uint(fmaf(slope, at4.z + off, __uint_as_float(w[j + 2])));
                  w[j + 3] = __float_as_uint(fmaf(slope, at4.w + off, __uint_as_float(w[j + 3])));
                }
              } else {
                const float off = static_cast<float>(tok0 + half * 64 - pos);
#pragma unroll
                for (int j = 0; j < 64; ++j) w[j] = __float_as_uint(fmaf(slope, off + static_cast<float>(j), __uint_as_float(w[j])));
              }
            }
          }
          if (special) {
#pragma unroll
            for (int j = 0; j < 64; ++j) w[j] = see[half * 2 + (j >> 5)] >> (j & 31) & 1 ? w[j] : 0xff800000u;
          }
        };
        auto largest = [](const uint32_t (&w)[64]) {
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < 64; j += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mx[k] = fmaxf(fmaxf(mx[k], __uint_as_float(w[j + 2 * k])), __uint_as_float(w[j + 2 * k + 1]));
          return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        };
        // ---- exponentials, their sum, P over the scores
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        auto weights = [&](const uint32_t (&w)[64], int half) {
          const float2 c2 = make_float2(c, c), m2 = make_float2(-m_run, -m_run);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t h[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float2 x = __ffma2_rn(make_float2(__uint_as_float(w[32 * j + 2 * k]), __uint_as_float(w[32 * j + 2 * k + 1])), c2, m2);
              const float2 p = make_float2(ex2(x.x), ex2(x.y));
              sum[k & 1] = __fadd2_rn(sum[k & 1], p);
              h[k] = T::pack2(p.x, p.y);
            }
            tmem_st16(t_s + half * 64 + j * 16, h);
          }
        };
        uint32_t w[64];
        scores(w, 0);
        float most = largest(w);
        scores(w, 1);
        most = fmaxf(most, largest(w));
        const float top = most == -INFINITY ? -INFINITY : fmaf(most, c, -m_run);
        const bool raise = seen ? top > kPgSlack + kPgLift<T> : top > -INFINITY;
        if (__any_sync(0xffffffffu, raise)) {
          const float f = raise && seen ? ex2(kPgLift<T> - top) : 1.f;
          if (raise) m_run += top - kPgLift<T>;
          seen = seen || raise;
          l *= f;
          if (i > 0 && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
            for (int j = 0; j < D / 16; ++j) {
              uint32_t o[16];
              tmem_ld16(t_o + j * 16, o);
              tmem_ld_wait();
              tmem_use(o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st16(t_o + j * 16, o);
            }
          }
        }
        weights(w, 1);
        scores(w, 0);
        weights(w, 0);
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(p_ready + 8 * g);
      }
      // ---- the piece's rows
      wait_or_fail(o_done + 8 * g, pieces++ & 1, fail);
      tc_fence_after();
      if (*fail) l = __int_as_float(0x7fc00000);
      if (node < 0) l = 0.f;
      const float f = l == 0.f ? 0.f : cur.whole ? 1.f / l : 1.f;
      float* part = a.part + static_cast<int64_t>(2 * blockIdx.x + (cur.pos == lo ? 0 : 1)) * kPgRowBlock * (D + 2);
#pragma unroll 1
      for (int j = 0; j < D / 32; ++j) {
        uint32_t o[32];
        tmem_ld32(t_o + j * 32, o);
        tmem_ld_wait();
        tmem_use(o);
        const uint32_t up = s_row[(g * 128 + row) * (D / 16) + j], down = s_row[(g * 128 + row) * (D / 16) + D / 32 + j];
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          float y = f == 0.f ? 0.f : __uint_as_float(o[k]) * f;
          if (up | down) y = f == 0.f ? 0.f : put_back(y, up >> k & 1, down >> k & 1);
          o[k] = __float_as_uint(y);
        }
        if (cur.whole) {   // the rows of q are done with: their place takes the output's
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = T::pack2(__uint_as_float(o[8 * k + 2 * e]), __uint_as_float(o[8 * k + 2 * e + 1]));
            *reinterpret_cast<uint4*>(qt + block_off(128, row, j * 4 + k)) = make_uint4(y[0], y[1], y[2], y[3]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) part[(j * 32 + k) * kPgRowBlock + g * 128 + row] = __uint_as_float(o[k]);
        }
      }
      if (!cur.whole)
        *reinterpret_cast<float2*>(part + kPgRowBlock * D + (g * 128 + row) * 2) = make_float2(l == 0.f ? -INFINITY : m_run, l);
      else if (a.lse && Rg < rows_total)
        a.lse[(static_cast<int64_t>(cur.b) * a.N + at) * a.Hq + cur.h * a.G + (Rg - at * a.G)] = l == 0.f ? -INFINITY : (m_run + log2f(l)) * kLn2;
      tc_fence_before();
      named_barrier_sync(2 + g, 128);
      if (cur.whole) {
#pragma unroll 4
        for (int i = row; i < 128 * (D / 8); i += 128) {
          const int r = i / (D / 8), ch = i % (D / 8), RR = row0 + r;
          if (RR >= rows_total) break;
          const int nn = paged_node(a, RR);
          const int64_t to = (static_cast<int64_t>(cur.b) * a.N + nn) * a.Hq + cur.h * a.G + (RR - nn * a.G);
          *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + to * D * 2 + ch * 16) = *reinterpret_cast<const uint4*>(qt + block_off(128, r, ch));
        }
      }
      named_barrier_sync(4, kRowSoft);   // the tree and the rows' places are free for the next piece
    }
  }
  __syncthreads();
  if (s_fail) settle_after_failure();   // before TMEM goes
  __syncthreads();
  if (tid == 0) a.failed[blockIdx.x] = s_fail;
  if (warp == 9) tmem_free(tmem, 512);
}

}  // namespace sv
