// Attention over the 16-bit cache for many rows a kv head (draft trees,
// prompts), bound by the tensor cores and the exponentials.
//
// A block is 256 rows of one kv head as two halves of 128 lanes that share K
// and V; for each half g
//   S_g [128 rows, 128 tokens] = q_g K^T,   O_g [128 rows, D] += P_g V,
// K and V as TMA brings them (V transposed by the descriptor), P_g in the type
// of V over the columns of S_g in TMEM. Per tile the products of a half take
// 8 D clocks and its 128 x 128 exponentials 512 (32 a clock). With 128-wide heads S
// and O of both halves fill all 512 columns of TMEM, so within a half S, softmax
// and P V follow each other and one half's softmax runs under the other's
// products; one CTA an SM. With 64-wide heads there is room for a third S: products
// are taken by turns, S three ahead of P V by a warp of its own, and the softmax
// of neither half waits for them (a piece of 1001 rows 570 us, so 645 without).
//
// Where a kv head has no more than 128 rows, both halves take them, and the tiles
// by turns; at a piece's end one half's O, maxima and sums go to the other.
//
// A thread has one row, so maximum, exponentials and sum are its own. It reads its
// scores twice, for the maximum and for the exponentials, which it writes over
// what it has read; with 128-wide heads P of the first 64 tokens is multiplied
// while those of the others are worked out. The running maximum is raised only when a score exceeds
// it by 2^8; the warp then rescales its rows of O. P is rounded to 16 bits (half a
// step of the type: 2^-8 of a bf16 weight, 2^-11 of f16's), its sum is not.
//
// Capped or biased scores, and those of a tile that some row does not see whole,
// are made final in TMEM on the first reading: -inf where the row's 128 bits say
// so, which the thread works out from its position and path. What must not be read
// of such a tile's V is taken out by warps of their own as soon as it is there.
// The rows of the next piece's q come in under the last products of this one.
//
// The roles run different code at once, and all of it has to stay in the
// instruction cache: loops are rolled, and what is rare is out of line. With the
// 128 columns unrolled and read once (held in registers, no maximum where the
// weights' sum showed that none was too large) a tile took fewer instructions
// and more time: prompts 425 us against 419 before, capped trees 337 against 218.
//
// Measured: two prompts of 4099 rows (32 heads on 8 of 128) 257 us, 1.08 PFLOP/s,
// a tile of two halves 3400 clocks against 2048 of its products: the MMA warp's
// waits for what is there already (150 clocks each, five a half) and its issue.
// 64-wide heads: 1200 clocks a half, all of it softmax, which alone takes 900.
// Trees of 64 nodes on 16 requests of up to 8192 tokens 99 us, 3.6 TB/s. Sixteen
// softmax warps instead of eight took as long (piece 580 us, prompts 267).
//
// Warps 0-3 and 4-7: softmax of the halves. 8: TMA. 9: MMA, which takes the
// halves by turns, so that they fall out of step. 10 and 11: V; with 64-wide
// heads 9 has P V, 10 has S and 11 V.
#pragma once

#include "attn_paged_cols.cuh"
#include "attn_q8_rows.cuh"

namespace sv {

constexpr int kPgRowThreads = 384;
constexpr int kPgRowSoft = 256;       // softmax threads
constexpr int kPgRowBlock = 256;

template <int D>
struct PgRowLayout {
  static constexpr int kTileBytes = kPgTile * D * 2;
  static constexpr int kStages = 128 * 1024 / kTileBytes;
  static constexpr int kDepth = kStages / 2;                             // V tiles in the ring
  static constexpr bool kAhead = D == 64;                                // TMEM has room for a third S
  static constexpr int kBufs = kAhead ? 3 : 2;
  static constexpr int kVThreads = kAhead ? 32 : 64;
  static constexpr int kOffQ = kStages * kTileBytes;                     // [2 halves][128 rows]
  static constexpr int kOffMisc = kOffQ + 2 * kTileBytes;
  // V's non-finite columns by token and by row; parents and depths of the nodes; positions of a tile's tokens by half
  static constexpr int kMiscBytes = (kDepth * 128 + kPgRowBlock) * (D / 16) * 4 + SV_MAX_TREE_NODES * 4 + 2 * kPgTile * 4;
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

// cap tanh(z / cap) = cap (1 - 2 / (1 + e^(2 z / cap))), where coef brings x to the
// exponent. A reciprocal takes the unit that the exponentials need twice as long
// as one of those, so three of four are Newton's, from the bits subtracted from a
// constant: as a number of steps of 2^-23 the bits of d = 2^e (1 + x) are e + 127 + x,
// so those of 253 + c - (e + 127 + x) are of 2^(-1 - e) (1 + c - x), and for x > c of
// 2^(-2 - e) (2 + c - x). Times d that is (1 + x) (1 + c - x) / 2, at most (1 + c / 2)^2 / 2
// and at least (1 + c) / 2; c = sqrt(24) - 4 makes them as far from 1 on both sides,
// 5.1 %, of which three steps leave 1.2e-7, fp32's rounding. (All on the unit:
// capped trees took 145 us, so 134.)
__device__ __forceinline__ void cap_scores(uint32_t (&x)[32], float coef, float cap) {
  const float2 coef2 = make_float2(coef, coef), one = make_float2(1.f, 1.f), two = make_float2(2.f, 2.f);
  const float2 cap2 = make_float2(cap, cap), down = make_float2(-2.f * cap, -2.f * cap);
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    float2 t = __fmul2_rn(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), coef2), r;
    if (e & 6) {
      asm("min.NaN.f32 %0, %0, 0f42800000;" : "+f"(t.x));   // at 64: 1 / (1 + 2^64) is 0 to the sum
      asm("min.NaN.f32 %0, %0, 0f42800000;" : "+f"(t.y));
      const float2 d = __fadd2_rn(make_float2(ex2(t.x), ex2(t.y)), one), n = make_float2(-d.x, -d.y);
      r = make_float2(__uint_as_float(0x7ef311c3u - __float_as_uint(d.x)), __uint_as_float(0x7ef311c3u - __float_as_uint(d.y)));
#pragma unroll
      for (int k = 0; k < 3; ++k) r = __fmul2_rn(r, __ffma2_rn(n, r, two));
    } else {
      const float2 d = __fadd2_rn(make_float2(ex2(t.x), ex2(t.y)), one);
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
    }
    t = __ffma2_rn(r, down, cap2);
    x[e] = __float_as_uint(t.x);
    x[e + 1] = __float_as_uint(t.y);
  }
}

// The bits below bit x of a word.
__device__ __forceinline__ uint32_t below(int x) { return x <= 0 ? 0u : x >= 32 ? 0xffffffffu : (1u << x) - 1u; }

// What was taken out of the tokens of a tile that a row sees, into the row's flags.
template <int D>
__device__ __noinline__ void note_seen(const uint32_t* from, uint32_t s0, uint32_t s1, uint32_t s2, uint32_t s3, uint32_t* to) {
  const uint32_t see[4] = {s0, s1, s2, s3};
#pragma unroll 1
  for (int t = 0; t < kPgTile; ++t)
    if (see[t >> 5] >> (t & 31) & 1)
#pragma unroll 1
      for (int w = 0; w < D / 16; ++w) to[w] |= from[t * (D / 16) + w];
}

// A warp's rows of O (TMEM) with what was taken out of V put back.
template <int D>
__device__ __noinline__ void put_back_rows(uint32_t t_o, const uint32_t* flags) {
#pragma unroll 1
  for (int j = 0; j < D; j += 16) {
    uint32_t o[16];
    __syncwarp();
    tmem_ld16(t_o + j, o);
    const uint32_t up = flags[j / 32] >> (j & 31), down = flags[D / 32 + j / 32] >> (j & 31);
    tmem_ld_wait();
    tmem_use(o);
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(put_back(__uint_as_float(o[e]), up >> e & 1, down >> e & 1));
    tmem_st16(t_o + j, o);
  }
  tmem_st_wait();
}

// 16 bytes from global to shared memory, or zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// kVar: scores are capped or biased, or their factor is negative (the maximum of products is then not that of scores) or
// zero (which a masked product, -inf, must not meet).
template <typename T, int D, bool kVar>
__global__ void __launch_bounds__(kPgRowThreads, 1)
    attn_paged_rows_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                           const __grid_constant__ PagedAttnArgs a) {
  using L = PgRowLayout<D>;
  constexpr int kSt = L::kStages, kDepth = L::kDepth, kBufs = L::kBufs, kVT = L::kVThreads;
  constexpr bool kAhead = L::kAhead;
  extern __shared__ uint8_t raw[];
  __shared__ AttnLine s_line;
  __shared__ int32_t s_warp[kPgRowThreads / 32];
  __shared__ PagedCursor s_cur[kPgRowThreads / 32][2];
  __shared__ float2 s_ml[128];   // split: maxima and sums of half 1 (its other places are in use until half 0 is done)
  __shared__ __align__(8) uint64_t s_bar[2 * kSt + kDepth + 12];
  __shared__ uint32_t s_tmem, s_fail, s_there[16], s_odd[kDepth];   // s_odd: whether values were taken out of a tile's V
  const uint32_t smem0 = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t* smem = raw + (smem0 - smem_u32(raw));
  uint32_t* s_tok = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);     // [kDepth][128][2][D / 32] columns with +inf, -inf (NaN: both)
  uint32_t* s_row = s_tok + kDepth * 128 * (D / 16);                     // [256][2][D / 32]
  float* s_at = reinterpret_cast<float*>(s_row + kPgRowBlock * (D / 16));   // [2][128] positions of a tile's tokens
  int16_t* s_par = reinterpret_cast<int16_t*>(s_at + 2 * kPgTile);       // [nodes]
  int16_t* s_depth = s_par + SV_MAX_TREE_NODES;                          // [nodes]

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t full = smem_u32(s_bar), empty = full + 8 * kSt, v_fit = empty + 8 * kSt, s_ready = v_fit + 8 * kDepth;
  const uint32_t p_ready = s_ready + 8 * kBufs, o_done = p_ready + 32, q_ready = o_done + 8 * kBufs;
  if (tid == 0) {
    s_fail = 0;
#pragma unroll 1
    for (int i = 0; i < kSt; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
#pragma unroll 1
    for (int i = 0; i < kDepth; ++i) mbar_init(v_fit + 8 * i, kVT);
#pragma unroll 1
    for (int i = 0; i < kBufs; ++i) {   // by S's place, which is the half where there are two
      mbar_init(s_ready + 8 * i, 1);
      mbar_init(o_done + 8 * i, 1);
    }
#pragma unroll 1
    for (int i = 0; i < 4; ++i) mbar_init(p_ready + 8 * i, 128);   // by half: tokens 0 .. 63 of a tile, 64 .. 127; or by place
#pragma unroll 1
    for (int i = 0; i < 2; ++i) mbar_init(q_ready + 8 * i, 128);
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
  PagedCursor* place = s_cur[warp];   // every role walks the same pieces; n counts tiles across them
  PagedCursor& cur = place[0];
  if (lane == 0) cur.start(a, s_line, lo);
  next_piece(a, place, place, hi);
  uint32_t n = 0;
  volatile uint32_t* fail = &s_fail;
  const int rows_total = a.N * a.G;
  // Halves of a block that have rows; split: each has all of them, and every second tile.
  const bool split = a.R == 128;
  auto halves = [&](int block) { return split || rows_total - block * kPgRowBlock > 128 ? 2 : 1; };

  if (warp == 8) {
    paged_load<D, kSt>(a, &k_map, &v_map, &cur, hi, smem0, full, empty, s_there, fail);
  } else if (warp >= 12 - kVT / 32) {
    // -------------------------------------------- V's rows that must not be read
    // A wait that gives up ends no loop here either: two warps meet at a barrier.
#pragma unroll 1
    for (; cur.pos < hi; next_piece(a, &cur, &cur, hi)) {
#pragma unroll 1
      for (int i = 0; i < cur.n; ++i, ++n) {
        const int tok0 = (cur.t0 + i) * kPgTile;
        const uint32_t s = 2 * n + 1, st = s % kSt;
        wait_or_fail(full + 8 * st, (s / kSt) & 1, fail);
        const uint32_t there = s_there[n & 15];
        const bool special = cur.special(a, tok0, there);
        uint8_t* vt = smem + st * L::kTileBytes;
        uint32_t odd = 0;
#pragma unroll 1
        for (int row = tid - (kPgRowThreads - kVT); special && row < kPgTile; row += kVT) {
          const bool valid = there >> (row >> a.c.page_shift) & 1 && tok0 + row < cur.rq.len;
#pragma unroll
          for (int ch = 0; ch < D / 8; ++ch) {
            uint4* p = reinterpret_cast<uint4*>(vt + block_off(kPgTile, row, ch));
            if (valid)
              odd |= nonfinite8<T>(*p);
            else
              *p = make_uint4(0, 0, 0, 0);
          }
        }
        odd = named_barrier_or(5, kVT, odd != 0);
        uint32_t* flags = s_tok + (n % kDepth) * 128 * (D / 16);
#pragma unroll 1
        for (int row = tid - (kPgRowThreads - kVT); odd && row < kPgTile; row += kVT) {
          const bool valid = there >> (row >> a.c.page_shift) & 1 && tok0 + row < cur.rq.len;
#pragma unroll 1
          for (int ch = 0; ch < D / 8; ++ch) {
            const uint32_t f = valid ? take_out8<T>(reinterpret_cast<uint4*>(vt + block_off(kPgTile, row, ch))) : 0u;
            uint8_t* to = reinterpret_cast<uint8_t*>(flags + row * (D / 16)) + ch;
            to[0] = static_cast<uint8_t>(f);
            to[D / 8] = static_cast<uint8_t>(f >> 8);
          }
        }
        if (tid == kPgRowThreads - kVT) s_odd[n % kDepth] = odd;
        fence_async_smem();
        mbar_arrive(v_fit + 8 * (n % kDepth));
      }
    }
  } else if (warp >= 9) {
    // ------------------------------------------------------------------ MMA
    constexpr uint32_t kIdS = tc_idesc(T::kMma, false, false, 128, 128), kIdO = tc_idesc(T::kMma, false, true, 128, D);
    // Operands' descriptors: a step of 16 along K is 32 bytes of a row, or 16 rows of V.
    const uint64_t d_q = tc_desc(smem0 + L::kOffQ, 16, 1024, 2), d_k = tc_desc(smem0, 16, 1024, 2);
    const uint64_t d_v = tc_desc(smem0, kPgTile * 128, 1024, 2);
    auto at = [](uint64_t d, uint32_t bytes) { return d + (bytes >> 4); };
    bool ok = true;
    if constexpr (kAhead) {
      // Products of both halves by turns, in order: k counts them.
      const uint32_t tmem = uniform(s_tmem);
      uint32_t k = 0;
      if (warp == 9) {   // P V
#pragma unroll 1
        for (; ok && cur.pos < hi; next_piece(a, &cur, &cur, hi)) {
          const int gs = uniform(halves(cur.block)), tiles = uniform(cur.n);
          const bool both = !split && gs == 2;   // a tile is for both halves
          const int total = both ? 2 * tiles : tiles;
#pragma unroll 1
          for (int j = 0; j < total && ok; ++j, ++k) {
            const uint32_t m = n + (both ? j >> 1 : j), st = (2 * m + 1) % kSt, buf = k % kBufs;
            const int g = gs == 2 ? j & 1 : 0;
            if (!both || !g) ok = warp_wait_or_fail(v_fit + 8 * (m % kDepth), (m / kDepth) & 1, fail);
            ok = ok && warp_wait_or_fail(p_ready + 8 * buf, k / kBufs & 1, fail);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              const uint64_t v = at(d_v, st * L::kTileBytes);
              const uint32_t t_p = tmem + buf * 128, t_o = tmem + kBufs * 128 + g * D;
#pragma unroll
              for (int x = 0; x < 8; ++x)   // P's halves lie where those of S did
                tc_mma_f16_ts(t_o, t_p + (x & 3) * 8 + (x >> 2) * 64, at(v, 2048 * x), kIdO, j >= gs || x > 0);
              tc_commit(o_done + 8 * buf);
              if (!both || g) tc_commit(empty + 8 * st);
            }
            __syncwarp();
          }
          n += tiles;
        }
      } else {   // q K^T
        uint32_t pieces0 = 0, pieces1 = 0;
#pragma unroll 1
        for (; ok && cur.pos < hi; next_piece(a, &cur, &cur, hi)) {
          const int gs = uniform(halves(cur.block)), tiles = uniform(cur.n);
          const bool both = !split && gs == 2;
          const int total = both ? 2 * tiles : tiles;
#pragma unroll 1
          for (int j = 0; j < max(total, gs) && ok; ++j) {
            if (j < gs) ok = warp_wait_or_fail(q_ready + 8 * j, (j ? pieces1++ : pieces0++) & 1, fail);
            if (j >= total) break;
            const uint32_t m = n + (both ? j >> 1 : j), st = 2 * m % kSt, buf = k % kBufs;
            const int g = gs == 2 ? j & 1 : 0;
            if (!both || !g) ok = ok && warp_wait_or_fail(full + 8 * st, (2 * m / kSt) & 1, fail);
            if (k >= kBufs) ok = ok && warp_wait_or_fail(o_done + 8 * buf, (k / kBufs - 1) & 1, fail);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              const uint64_t q = at(d_q, g * L::kTileBytes), kt = at(d_k, st * L::kTileBytes);
#pragma unroll
              for (int x = 0; x < D / 16; ++x) tc_mma_f16(tmem + buf * 128, at(q, x * 32), at(kt, x * 32), kIdS, x > 0);
              tc_commit(s_ready + 8 * buf);
              if (!both || g) tc_commit(empty + 8 * st);
            }
            __syncwarp();
            ++k;
          }
          n += tiles;
        }
      }
    } else {
      uint32_t pieces[2] = {0, 0}, mine[2] = {0, 0};   // by half; mine: tiles
      // In the elected thread: S of tile m.
      auto scores = [&](uint32_t m, int g, bool last) {
        const uint32_t st = 2 * m % kSt;
        const uint64_t q = at(d_q, g * L::kTileBytes), k = at(d_k, st * L::kTileBytes);
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          const uint32_t off = (j >> 2) * (kPgTile * 128) + (j & 3) * 32;
          tc_mma_f16(tmem + g * 128, at(q, off), at(k, off), kIdS, j > 0);
        }
        tc_commit(s_ready + 8 * g);
        if (last) tc_commit(empty + 8 * st);
      };
      auto k_there = [&](uint32_t m) { ok = ok && warp_wait_or_fail(full + 8 * (2 * m % kSt), (2 * m / kSt) & 1, fail); };
#pragma unroll 1
      for (; ok && cur.pos < hi; next_piece(a, &cur, &cur, hi)) {
        const int gs = halves(cur.block), tiles = cur.n;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          if (g == gs || !ok) break;
          const int first = split ? g : 0;   // the half's first tile
          if (g == 0 || (split && tiles > 1)) k_there(n + first);
          ok = ok && warp_wait_or_fail(q_ready + 8 * g, pieces[g]++ & 1, fail);
          if (!ok) break;
          tc_fence_after();
          if (first < tiles && elect_one()) scores(n + first, g, split || g + 1 == gs);
          __syncwarp();
        }
        const int step = split ? 2 : 1;
#pragma unroll 1
        for (int i = 0; i < tiles && ok; ++i, ++n) {
          const uint32_t st = (2 * n + 1) % kSt;
          const uint64_t v = at(d_v, st * L::kTileBytes);
          const bool more = i + step < tiles;
          ok = warp_wait_or_fail(v_fit + 8 * (n % kDepth), (n / kDepth) & 1, fail);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if (g == gs || !ok) break;
            if (split && g != (i & 1)) continue;
            const bool last = split || g + 1 == gs;
            ok = warp_wait_or_fail(p_ready + 16 * g, mine[g] & 1, fail);
            if (!ok) break;
            tc_fence_after();
            // P's halves lie where those of S did.
            if (elect_one())
#pragma unroll
              for (int j = 0; j < 4; ++j)
                tc_mma_f16_ts(tmem + 256 + g * 128, tmem + g * 128 + j * 8, at(v, 2048 * j), kIdO, i >= step || j > 0);
            __syncwarp();
            if (more && (g == 0 || split)) k_there(n + step);   // under these products
            ok = ok && warp_wait_or_fail(p_ready + 16 * g + 8, mine[g] & 1, fail);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int j = 4; j < 8; ++j)
                tc_mma_f16_ts(tmem + 256 + g * 128, tmem + g * 128 + 64 + (j - 4) * 8, at(v, 2048 * j), kIdO, true);
              if (last) tc_commit(empty + 8 * st);
              // The next S overwrites this P: products that one thread issues run in order.
              if (more)
                scores(n + step, g, last);
              else
                tc_commit(o_done + 8 * g);
            }
            __syncwarp();
            ++mine[g];
          }
        }
      }
    }
  } else if (warp < 8) {
    // -------------------------------------------------------------- softmax
    const int g = warp >> 2, row = tid & 127;   // the thread's half, its row of it
    const int bar = 2 + g;                       // of the half's threads
    const uint32_t t_lane = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t t_o = t_lane + kBufs * 128 + g * D;
    uint32_t* flags = s_row + (g * 128 + row) * (D / 16);
    uint32_t mine = 0, pieces = 0;   // tiles and pieces of this half; kAhead: products of both halves before this piece
    // q's rows of a piece, D / 8 threads a row: on their way to their place, and there.
    auto q_start = [&](const PagedCursor& c) {
      constexpr int kLpr = D / 8;
      const int ch = row % kLpr;
      const uint8_t* q = a.q + c.b * a.sqb + static_cast<int64_t>(c.h) * a.G * a.sqh + ch * 16;
      const uint32_t qt = smem0 + L::kOffQ + g * L::kTileBytes;
      const int first = split ? 0 : c.block * kPgRowBlock + g * 128;
#pragma unroll 2
      for (int r = row / kLpr; r < 128; r += 128 / kLpr) {
        const int Rg = first + r, node = paged_node(a, Rg);
        const bool there = Rg < rows_total && node < c.rq.n;
        copy16(qt + block_off(128, r, ch), there ? q + node * a.sqn + (Rg - node * a.G) * a.sqh : a.q, there);
      }
    };
    auto q_end = [&] {
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_async_smem();
      mbar_arrive(q_ready + 8 * g);
    };
    if (place->pos < hi) {
      if (tid == 0) a.first[blockIdx.x] = place->item(a);
      if (g < halves(place->block)) {
        q_start(*place);
        q_end();
      }
    }
    uint32_t count = 0;   // pieces
    // A wait that gives up ends no loop here: these warps meet at barriers, so all
    // run on to the end (every later wait then returns at once), without meaning:
    // the rows of every piece that ends after it are NaN.
#pragma unroll 1
    for (; place[count & 1].pos < hi; ++count) {
      const PagedCursor& cur = place[count & 1];
      const PagedReq& rq = cur.rq;
      const int gs = halves(cur.block), soft = 128 * gs;
      const bool active = g < gs;
      const int row0 = split ? 0 : cur.block * kPgRowBlock + g * 128;
      // ---- the thread's row, the request's tree
      const int Rg = row0 + row, at = paged_node(a, Rg);
      const int node = Rg < rows_total && at < rq.n ? at : -1;
      int depth = max(node, 0);
#pragma unroll
      for (int j = 0; j < D / 16; ++j) flags[j] = 0;
      if (a.parents && active) {
        const int32_t* par = a.parents + static_cast<int64_t>(cur.b) * a.N;
#pragma unroll 1
        for (int i = tid; i < rq.n; i += soft) s_par[i] = static_cast<int16_t>(tree_up(par, i));
        named_barrier_sync(1, soft);
#pragma unroll 1
        for (int i = tid; i < rq.n; i += soft) {
          int d = 0;
#pragma unroll 1
          for (int m = s_par[i]; m >= 0; m = s_par[m]) ++d;
          s_depth[i] = static_cast<int16_t>(d);
        }
        named_barrier_sync(1, soft);
        depth = s_depth[max(node, 0)];
      }
      const int pos = rq.base + depth;
      const int open = max(pos - a.window + 1, 0);   // the window's first position
      const float slope = kVar && a.slopes && node >= 0 ? a.slopes[cur.h * a.G + Rg - at * a.G] * kLog2e : 0.f;

      const int tiles = active ? cur.n : 0, t0 = cur.t0, clear = cur.clear, inside = cur.inside;
      const uint32_t all_pages = (1u << (kPgTile >> a.c.page_shift)) - 1u;
      const float c = kVar ? 1.f : a.coef;   // of what the second reading finds
      float m_run = 0.f, l = 0.f;            // m_run means something once the row has seen a slot
      bool seen = false, any_odd = false;
#pragma unroll 1
      for (int i = split ? g : 0; i < tiles; i += split ? 2 : 1) {
        const uint32_t tile = n + i, k = kAhead ? mine + (split ? i : gs * i + g) : mine++;
        const uint32_t buf = kAhead ? k % kBufs : g, phase = (kAhead ? k / kBufs : k) & 1, t_s = t_lane + buf * 128;
        const int tok0 = (t0 + i) * kPgTile;
        wait_or_fail(s_ready + 8 * buf, phase, fail);   // every product before this S is done, but for kAhead the half's last
        tc_fence_after();
        const uint32_t there = s_there[tile & 15];
        const bool special = tok0 + kPgTile > clear || tok0 < inside || there != all_pages;
        uint32_t see[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};   // what the row sees of the tile
        if (special) {
          if (a.parents) {
            int far = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) see[j] = 0;
#pragma unroll 1
            for (int m = node; m >= 0 && far < a.window; m = s_par[m], ++far) {   // tokens on the row's way up
              const int t = rq.base + m - tok0;
              if (t < 0) break;   // parents come before
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (t >> 5 == j) see[j] |= 1u << (t & 31);
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int t = tok0 + 32 * j;
            const uint32_t before = below((a.parents ? rq.base : rq.base + node + 1) - t) & ~below(open - t);
            see[j] = (a.parents ? see[j] | before : before) & below(rq.len - t);
            if (!(there >> (32 * j >> a.c.page_shift) & 1)) see[j] &= 0xffff0000u;
            if (!(there >> ((32 * j + 16) >> a.c.page_shift) & 1)) see[j] &= 0x0000ffffu;
            if (node < 0) see[j] = 0;
          }
          __syncwarp();
        }
        if (kVar && a.slopes && a.parents) {   // positions of the tile's tokens, relative to base: small enough for fp32
          const int m = tok0 + row - rq.base;
          named_barrier_sync(bar, 128);   // every row has read the last tile's
          s_at[g * 128 + row] = static_cast<float>(m >= 0 && m < rq.n ? s_depth[m] : m);
          named_barrier_sync(bar, 128);
        }
        // ---- maximum
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (kVar || special) {
#pragma unroll 1
          for (int j = 0; j < kPgTile; j += 32) {
            uint32_t x[32];
            tmem_ld32(t_s + j, x);
            const uint32_t on = j == 0 ? see[0] : j == 32 ? see[1] : j == 64 ? see[2] : see[3];
            tmem_ld_wait();
            tmem_use(x);
            if (kVar) {
              if (a.cap > kPgFarCap) {
                cap_far(x, a);
              } else if (a.cap != 0.f) {
                cap_scores(x, a.coef, a.cap);
              } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * a.coef);
              }
              if (a.slopes) {
                const float off = static_cast<float>(a.parents ? -depth : tok0 + j - pos);
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                  const float far = a.parents ? s_at[g * 128 + j + e] : static_cast<float>(e);
                  x[e] = __float_as_uint(fmaf(slope, far + off, __uint_as_float(x[e])));
                }
              }
            }
            if (special) {
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = on >> e & 1 ? x[e] : 0xff800000u;
            }
#pragma unroll
            for (int e = 0; e < 32; e += 2) mx[e >> 1 & 3] = fmaxf(fmaxf(mx[e >> 1 & 3], __uint_as_float(x[e])), __uint_as_float(x[e + 1]));
            tmem_st16(t_s + j, x);
            tmem_st16(t_s + j + 16, x + 16);
          }
          tmem_st_wait();
        } else {
#pragma unroll 1
          for (int j = 0; j < kPgTile; j += 64) {
            uint32_t x[64];
            tmem_ld32(t_s + j, x);
            tmem_ld32(t_s + j + 32, x + 32);
            tmem_ld_wait();
            tmem_use(x);
#pragma unroll
            for (int e = 0; e < 64; e += 2) mx[e >> 1 & 3] = fmaxf(fmaxf(mx[e >> 1 & 3], __uint_as_float(x[e])), __uint_as_float(x[e + 1]));
          }
        }
        const float most = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        const float top = most == -INFINITY ? -INFINITY : fmaf(most, c, -m_run);
        const bool raise = seen ? top > kPgSlack + kPgLift<T> : top > -INFINITY;
        if (__any_sync(0xffffffffu, raise)) {
          const float f = raise && seen ? ex2(kPgLift<T> - top) : 1.f;
          if (raise) m_run += top - kPgLift<T>;
          seen = seen || raise;
          l *= f;
          if (i >= (split ? 2 : 1) && __any_sync(0xffffffffu, f != 1.f)) {   // O holds something
            if (kAhead) {
              wait_or_fail(o_done + 8 * ((k - gs) % kBufs), (k - gs) / kBufs & 1, fail);
              tc_fence_after();
            }
#pragma unroll 1
            for (int j = 0; j < D; j += 16) {
              uint32_t o[16];
              tmem_ld16(t_o + j, o);
              tmem_ld_wait();
              tmem_use(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st16(t_o + j, o);
            }
          }
        }
        // ---- weights over the scores, their sum
        const float2 c2 = make_float2(c, c), m2 = make_float2(-m_run, -m_run);
        float2 sum[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int u = 0; u < 2; ++u) {
          uint32_t x[64];
          tmem_ld32(t_s + u * 64, x);
          tmem_ld32(t_s + u * 64 + 32, x + 32);
          tmem_ld_wait();
          tmem_use(x);
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float2 y = __ffma2_rn(make_float2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), c2, m2);
            const float2 p = make_float2(ex2(y.x), ex2(y.y));
            sum[j & 3] = __fadd2_rn(sum[j & 3], p);
            x[j] = T::pack2(p.x, p.y);
          }
          tmem_st16(t_s + u * 64, x);
          tmem_st16(t_s + u * 64 + 16, x + 16);
          if (special && u == 1) {   // what was taken out of V, before the tile is given up
            wait_or_fail(v_fit + 8 * (tile % kDepth), (tile / kDepth) & 1, fail);
            if (const_cast<volatile uint32_t*>(s_odd)[tile % kDepth]) {
              any_odd = true;
              note_seen<D>(s_tok + (tile % kDepth) * 128 * (D / 16), see[0], see[1], see[2], see[3], flags);
            }
          }
          tmem_st_wait();
          tc_fence_before();
          if (!kAhead || u == 1) mbar_arrive(p_ready + (kAhead ? 8 * buf : 16 * g + 8 * u));
        }
        sum[0] = __fadd2_rn(__fadd2_rn(sum[0], sum[1]), __fadd2_rn(sum[2], sum[3]));
        l += sum[0].x + sum[0].y;
      }
      n += cur.n;
      // ---- the piece's rows, under whose last products the cursor moves on
      const PagedCursor& next = place[~count & 1];
      next_piece(a, &cur, place + (~count & 1), hi);
      const bool bring = next.pos < hi && g < halves(next.block);
      if (bring && !split) q_start(next);   // the half's scores of this piece are done
      if (active) {
        if (!kAhead && (!split || g < tiles)) wait_or_fail(o_done + 8 * g, pieces++ & 1, fail);
        if (kAhead && (!split || g < tiles)) {   // the half's last, and before `other` is written the last S of both
          const uint32_t all = mine + (split ? tiles : gs * tiles) - 1, k = split ? all - ((tiles - 1 - g) & 1) : all - (gs - 1 - g);
          if (split) wait_or_fail(s_ready + 8 * (all % kBufs), all / kBufs & 1, fail);
          wait_or_fail(o_done + 8 * (k % kBufs), k / kBufs & 1, fail);
        }
        tc_fence_after();
        if (any_odd) put_back_rows<D>(t_o, flags);
        float f0 = 1.f, f1 = 0.f;   // of this half's O, and of the other's
        float* other = reinterpret_cast<float*>(smem + L::kOffQ) + row;   // [D][128], where q has been
        if (split) {
          if (g == 1) {
            s_ml[row] = make_float2(m_run, l);
#pragma unroll 1
            for (int j = 0; j < (g < tiles ? D : 0); j += 16) {   // without tiles it has no O, and q is in use
              uint32_t o[16];
              tmem_ld16(t_o + j, o);
              tmem_ld_wait();
              tmem_use(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) other[(j + e) * 128] = __uint_as_float(o[e]);
            }
            tc_fence_before();
          }
          named_barrier_sync(4, kPgRowSoft);
          if (g == 0) {
            const float2 ml = s_ml[row];
            const float m0 = l == 0.f ? -INFINITY : m_run, m1 = ml.y == 0.f ? -INFINITY : ml.x, m = fmaxf(m0, m1);
            f0 = m0 == -INFINITY ? 0.f : ex2(m0 - m);
            f1 = m1 == -INFINITY ? 0.f : ex2(m1 - m);
            if (m != -INFINITY) m_run = m;
            l = fmaf(l, f0, ml.y * f1);   // a factor of 0 is no reason to leave a sum or an O out: 0 times NaN shows
          }
        }
        if (*fail) l = __int_as_float(0x7fc00000);
        if (node < 0) l = 0.f;
        const float f = l == 0.f ? 0.f : cur.whole ? 1.f / l : 1.f;
        f0 *= f;
        f1 *= f;
        const int lane_of = split ? row : g * 128 + row;
        float* part = a.part + static_cast<int64_t>(2 * blockIdx.x + (count == 0 ? 0 : 1)) * a.R * (D + 2) + lane_of;
        const int64_t to = (static_cast<int64_t>(cur.b) * a.N + at) * a.Hq + cur.h * a.G + (Rg - at * a.G);
        uint8_t* out = static_cast<uint8_t*>(a.out) + to * D * 2;
        const bool writes = !split || g == 0;
#pragma unroll 1
        for (int j = 0; j < (writes ? D : 0); j += 32) {
          uint32_t o[32];
          tmem_ld32(t_o + j, o);
          tmem_ld_wait();
          tmem_use(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(f == 0.f ? 0.f : __uint_as_float(o[e]) * f0);
          if (split && tiles > 1 && f != 0.f)   // the other half has an O
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(fmaf(other[(j + e) * 128], f1, __uint_as_float(o[e])));
          if (cur.whole) {
            if (Rg < rows_total) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t y[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) y[x] = T::pack2(__uint_as_float(o[8 * e + 2 * x]), __uint_as_float(o[8 * e + 2 * x + 1]));
                *reinterpret_cast<uint4*>(out + (j + 8 * e) * 2) = make_uint4(y[0], y[1], y[2], y[3]);
              }
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) part[(j + e) * a.R] = __uint_as_float(o[e]);
          }
          __syncwarp();
        }
        if (writes && !cur.whole)
          *reinterpret_cast<float2*>(part + a.R * D + lane_of) = make_float2(l == 0.f ? -INFINITY : m_run, l);
        else if (writes && a.lse && Rg < rows_total)
          a.lse[to] = l == 0.f ? -INFINITY : (m_run + log2f(l)) * kLn2;
        tc_fence_before();
      }
      if (kAhead) mine += split || gs == 1 ? cur.n : 2 * cur.n;
      // The tree's place and the other half's are free for the next piece; a half without rows keeps step (a wait must not
      // be for a phase after the one that is next on its barrier, nor last as long as the other half's piece: of a few
      // million tokens that is longer than the limit). Where both halves' products share places, the other half does not go
      // on alone before this one has seen its last product done.
      const bool alone = kAhead && next.pos < hi && halves(next.block) == 1;
      if (a.parents || split || gs == 1 || alone) named_barrier_sync(4, kPgRowSoft);
      if (bring && split) q_start(next);
      if (bring) q_end();
    }
  }
  __syncthreads();
  if (s_fail) settle_after_failure();   // before TMEM goes
  __syncthreads();
  if (tid == 0) a.failed[blockIdx.x] = s_fail;
  if (warp == 9) tmem_free(tmem, 512);
}

}  // namespace sv
