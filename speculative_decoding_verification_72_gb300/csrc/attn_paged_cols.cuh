// Attention over the 16-bit cache for up to 32 rows a kv head (single tokens,
// short chains), bound by memory.
//
// Rows are columns and tokens the 128 rows of both products:
//   S^T [128 tokens, rows] = K [tokens, D] q^T,
//   O^T [D, terms x rows] += V^T [D, tokens] P.
// A tile of 128 slots is the A operand of both, K as it lies (K-major), V
// transposed by the descriptor (MN-major), so each element goes from HBM by TMA
// into shared memory and from there into the tensor core, touched by no thread.
// P rounded to 16 bits would be off by half a step of the type; it is two terms
// instead, the rounding of P and of what that left (2^-16 of a bf16 weight), as
// columns of one product, which cost nothing here.
//
// Lane = token in S^T, so a thread has one token's scores for 16 rows, sums over
// tokens stay in its registers until the end, and P is two 16-byte stores a
// term. The running maximum is raised only when a score exceeds it by 2^8 (a
// vote per tile), which takes the slow path: maxima across its warps and a
// rescale of O^T in TMEM. So does every tile until each row has seen a slot,
// and every tile that some row does not see whole: masks, and V's rows that are
// no slots of the request (0 * NaN would reach every row) and non-finite values.
//
// One CTA an SM with a ring of 192 KB: three tiles of K and V of 128-wide heads
// (six of 64-wide ones), one of which is multiplied while the others are on their
// way. One warp issues TMA, one MMA, four (for 32 rows, eight) are the softmax.
//
// Measured: one token each of 64 requests of up to 8192 tokens (32 heads on 8 of
// 128) 235 us, 5.7 TB/s; its floor at 6.8 TB/s is 198. Further requests come at
// 6.1 TB/s, and 13 us are the ends of a call, the join among them. 32 chains of six
// rows with capped scores 138 us for 675 MB (a cap is an exponential and a reciprocal
// more a score). One token of one request 14 us, which are launches and latencies
// in a row.
#pragma once

#include "attn_paged.cuh"

namespace sv {

constexpr float kPgSlack = 8.f;   // log2 by which a term may exceed the running maximum
// f16 P is lifted by 2^7, so that its largest are 2^7 to 2^15 and what falls below f16's normal numbers is 2^-21 of them;
// the sum takes it lifted too.
template <typename T>
constexpr float kPgLift = T::kExpBits == 8 ? 0.f : 7.f;

template <int D, int MT>
struct PgColLayout {
  static constexpr int R = 16 * MT;
  static constexpr int kThreads = 128 * MT + 64;
  static constexpr int kTileBytes = kPgTile * D * 2;
  static constexpr int kHalves = D / 64;                       // 128-byte blocks of a row
  static constexpr int kStages = 192 * 1024 / kTileBytes;      // K and V by turns
  static constexpr int kNo = 2 * R;                            // columns of O^T
  static constexpr int kTmem = 2 * R + kNo <= 64 ? 64 : 128;
  static constexpr int kQBytes = R * D * 2;
  static constexpr int kPBytes = kPgTile * 128;
  static constexpr int kOffP = kStages * kTileBytes;
  static constexpr int kOffQ = kOffP + kPBytes;
  static constexpr int kOffMisc = kOffQ + (kQBytes + 1023) / 1024 * 1024;
  static constexpr int kMiscBytes = R * (16 + 4 * 9 + D / 4) + MT * 80 * 4;
  static constexpr int kBytes = 1024 + kOffMisc + kMiscBytes;
};

// D (TMEM) = A B (+ D if acc), 16-bit operands in shared memory.
__device__ __forceinline__ void tc_mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))
      : "memory");
}

__device__ __forceinline__ void tmem_ld4(uint32_t addr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}

// Box of the cache's 4-D map: 64 elements of the tokens of a page, for one head.
__device__ __forceinline__ void tma_load_page(uint32_t dst, const void* map, int x, int head, int page, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(0), "r"(head), "r"(page), "r"(bar)
      : "memory");
}

// Byte offset of 16-byte piece ch of row `row` in a tile of `rows` rows: 128-byte blocks, swizzled.
__device__ __forceinline__ uint32_t block_off(int rows, int row, int ch) {
  return (ch >> 3) * rows * 128 + row * 128 + (((ch & 7) ^ (row & 7)) << 4);
}

// What of a token's V row is not finite goes to the rows that see it.
template <typename T, int D>
__device__ __noinline__ void note_nonfinite(const uint8_t* vt, int row, uint32_t see, uint32_t* s_inf) {
#pragma unroll 1
  for (int ch = 0; see && ch < D / 8; ++ch) {
    uint4 w = *reinterpret_cast<const uint4*>(vt + block_off(kPgTile, row, ch));
    const uint32_t f = take_out8<T>(&w);
#pragma unroll 1
    for (int r = 0; f && r < 16; ++r) {
      if (!(see >> r & 1)) continue;
      uint32_t* to = s_inf + r * (D / 16) + (ch >> 2);
      atomicOr(to, (f & 0xffu) << (ch & 3) * 8);
      atomicOr(to + D / 32, (f >> 8) << (ch & 3) * 8);
    }
  }
}

// The TMA warp of both kernels: K and V of the CTA's tiles, in turns, into a
// ring of kStages tiles. s_there has, by tile, which of its pages there are.
template <int D, int kStages>
__device__ __forceinline__ void paged_load(const PagedAttnArgs& a, const CUtensorMap* k_map, const CUtensorMap* v_map, PagedCursor* place,
                                           int32_t hi, uint32_t ring, uint32_t full, uint32_t empty, uint32_t* s_there,
                                           volatile uint32_t* fail) {
  constexpr int kTileBytes = kPgTile * D * 2;
  const int lane = threadIdx.x & 31;
  const int ppt = kPgTile >> a.c.page_shift, shift = 7 - a.c.page_shift;   // pages a tile
  const int box = 128 << a.c.page_shift;                                    // bytes
  const int mine = lane & (ppt - 1), half = lane >> shift;                   // the lane's page of a tile, and block of its rows
  const uint32_t dst0 = ring + half * kPgTile * 128 + mine * box;
  uint32_t n = 0;
  PagedLook look;
  const PagedCursor& cur = *place;
#pragma unroll 1
  for (; cur.pos < hi; next_piece(a, place, place, hi)) {
    look.start(a, cur.b, cur.t0 << shift, cur.end, lane);
#pragma unroll 1
    for (int i = 0; i < cur.n; ++i, ++n) {
      const int page = look.page(a, cur.b, ((cur.t0 + i) << shift) + mine, cur.end, lane);
      const uint32_t there = __ballot_sync(0xffffffffu, page >= 0) & ((1u << ppt) - 1u);
      const bool load = page >= 0 && half < D / 64;
      const uint32_t bytes = __popc(there) * box * (D / 64);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t s = 2 * n + kv, st = s % kStages, turn = s / kStages;
        bool ok = true;
        if (lane == 0 && turn > 0) ok = wait_or_fail(empty + 8 * st, (turn - 1) & 1, fail);
        if (!__shfl_sync(0xffffffffu, ok, 0)) return;
        if (lane == 0) {
          if (kv == 0) s_there[n & 15] = there;
          mbar_arrive_expect_tx(full + 8 * st, bytes);
        }
        __syncwarp();
        if (load) tma_load_page(dst0 + st * kTileBytes, kv ? v_map : k_map, half * 64, cur.h, page, full + 8 * st);
      }
    }
  }
}

// Leaves time for copies and products in flight after a wait gave up.
__device__ __forceinline__ void settle_after_failure() {
  const uint64_t t = global_timer_ns();
#pragma unroll 1
  for (int i = 0; i < (1 << 20) && global_timer_ns() - t < 2000000; ++i) {
  }
}

template <typename T, int D, int MT>
__global__ void __launch_bounds__(PgColLayout<D, MT>::kThreads, 1)
    attn_paged_cols_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                           const __grid_constant__ PagedAttnArgs a) {
  using L = PgColLayout<D, MT>;
  constexpr int R = L::R, kSt = L::kStages, kSoft = 128 * MT;
  extern __shared__ uint8_t raw[];
  __shared__ AttnLine s_line;
  __shared__ int32_t s_warp[L::kThreads / 32];
  __shared__ PagedCursor s_cur[L::kThreads / 32];
  __shared__ __align__(8) uint64_t s_bar[2 * kSt + 7];
  __shared__ uint32_t s_tmem, s_fail, s_there[16];
  const uint32_t smem0 = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t* smem = raw + (smem0 - smem_u32(raw));
  int4* s_out = reinterpret_cast<int4*>(smem + L::kOffMisc);             // [R] where a row's output goes, its factor
  float* s_m = reinterpret_cast<float*>(s_out + R);                       // [R] running maximum (log2)
  float* s_up = s_m + R;                                                  // [R] what a slow path adds to it
  float* s_f = s_up + R;                                                  // [R] and multiplies by
  float* s_slope = s_f + R;                                               // [R] log2(e) slope
  int32_t* s_node = reinterpret_cast<int32_t*>(s_slope + R);              // [R], -1 for none
  int32_t* s_pos = s_node + R;                                            // [R] position
  int32_t* s_seen = s_pos + R;                                            // [R] whether the row has seen a slot
  uint32_t* s_anc = reinterpret_cast<uint32_t*>(s_seen + R);              // [R] the nodes that the row sees
  int32_t* s_depth = reinterpret_cast<int32_t*>(s_anc + R);               // [R] of the nodes: all of a request's are here
  uint32_t* s_inf = reinterpret_cast<uint32_t*>(s_depth + R);             // [R][2][D / 32] columns with +inf, with -inf (NaN: both)
  float* s_max = reinterpret_cast<float*>(s_inf + R * (D / 16));          // [4 MT][20]

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t full = smem_u32(s_bar), empty = full + 8 * kSt, s_ready = empty + 8 * kSt, s_free = s_ready + 16;
  const uint32_t p_ready = s_free + 16, p_free = p_ready + 8, q_ready = p_free + 8;
  if (tid == 0) {
    s_fail = 0;
#pragma unroll 1
    for (int i = 0; i < kSt; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_ready + 8 * i, 1);
      mbar_init(s_free + 8 * i, 4 * MT);
    }
    mbar_init(p_ready, kSoft);
    mbar_init(p_free, 1);
    mbar_init(q_ready, kSoft);
    fence_barrier_init();
  }
  if (warp == 4 * MT + 1) tmem_alloc(smem_u32(&s_tmem), L::kTmem);
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
  int32_t lo, hi;
  paged_line<L::kThreads>(a, &s_line, s_warp, lo, hi);
  PagedCursor* place = s_cur + warp;   // every role walks the same pieces; n counts tiles across them
  const PagedCursor& cur = *place;
  if (lane == 0) place->start(a, s_line, lo);
  next_piece(a, place, place, hi);
  uint32_t n = 0;
  volatile uint32_t* fail = &s_fail;

  if (warp == 4 * MT) {
    paged_load<D, kSt>(a, &k_map, &v_map, place, hi, smem0, full, empty, s_there, fail);
  } else if (warp == 4 * MT + 1) {
    // ------------------------------------------------------------------ MMA
    constexpr uint32_t kIdS = tc_idesc(T::kMma, false, false, 128, R), kIdO = tc_idesc(T::kMma, true, true, 128, L::kNo);
    // Operands' descriptors: a step of 16 along K is 32 bytes of a row, or 16 rows of V and P. 64-wide heads are half of the
    // product's 128 rows; a block stride of 0 gives the other half the same rows.
    const uint32_t tmem = uniform(s_tmem), smem0 = uniform(smem_u32(smem));
    const uint64_t d_q = tc_desc(smem0 + L::kOffQ, 16, 1024, 2), d_k = tc_desc(smem0, 16, 1024, 2);
    const uint64_t d_v = tc_desc(smem0, D == 128 ? kPgTile * 128 : 0, 1024, 2), d_p = tc_desc(smem0 + L::kOffP, 0, 1024, 2);
    auto at = [](uint64_t d, uint32_t bytes) { return d + (bytes >> 4); };
    bool ok = true;
    uint32_t pieces = 0;
    auto scores = [&](uint32_t m) {
      const uint32_t s = 2 * m, st = s % kSt, sb = m & 1;
      ok = ok && warp_wait_or_fail(full + 8 * st, (s / kSt) & 1, fail);
      if (m >= 2) ok = ok && warp_wait_or_fail(s_free + 8 * sb, ((m >> 1) - 1) & 1, fail);
      if (!ok) return;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t kt = at(d_k, st * L::kTileBytes);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc_mma_f16(tmem + sb * R, at(kt, (k >> 2) * (kPgTile * 128) + (k & 3) * 32), at(d_q, (k >> 2) * (R * 128) + (k & 3) * 32), kIdS, k > 0);
        tc_commit(empty + 8 * st);
        tc_commit(s_ready + 8 * sb);
      }
      __syncwarp();
    };
#pragma unroll 1
    for (; ok && cur.pos < hi; next_piece(a, place, place, hi)) {
      ok = warp_wait_or_fail(q_ready, pieces++ & 1, fail);
      if (!ok) break;
      const int tiles = uniform(cur.n);
      scores(n);
#pragma unroll 1
      for (int i = 0; i < tiles && ok; ++i, ++n) {
        if (i + 1 < tiles) scores(n + 1);
        const uint32_t s = 2 * n + 1, st = s % kSt;
        ok = ok && warp_wait_or_fail(full + 8 * st, (s / kSt) & 1, fail) && warp_wait_or_fail(p_ready, n & 1, fail);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t vt = at(d_v, st * L::kTileBytes);
#pragma unroll
          for (int k = 0; k < kPgTile / 16; ++k) tc_mma_f16(tmem + 2 * R, at(vt, 2048 * k), at(d_p, 2048 * k), kIdO, i > 0 || k > 0);
          tc_commit(empty + 8 * st);
          tc_commit(p_free);
        }
        __syncwarp();
      }
    }
  } else {
    // -------------------------------------------------------------- softmax
    const int grp = warp >> 2, row = tid & 127, r00 = grp * 16;   // the thread's rows r00 .. r00 + 15, token `row` of a tile
    const uint32_t t_lane = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t t_o = t_lane + 2 * R + r00;
    const int bar = 1 + grp;
    const int rows_total = a.N * a.G;
    float* max_w = s_max + warp * 20;
    const float* max_g = s_max + grp * 80;
    uint32_t* unseen = reinterpret_cast<uint32_t*>(s_max + grp * 80 + 16);   // whether a row with a node has seen no slot yet
    const bool plain = a.cap == 0.f && !a.slopes;
    const float2 coef2 = make_float2(a.coef, a.coef);
    // A wait that gives up ends no loop here: these warps meet at barriers, so all
    // run on to the end (every later wait then returns at once), without meaning:
    // the rows of every piece that ends after it are NaN.
#pragma unroll 1
    for (bool first = true; cur.pos < hi; next_piece(a, place, place, hi), first = false) {
      if (first && tid == 0) a.first[blockIdx.x] = cur.item(a);
      const PagedReq rq = cur.rq;
      const int row0 = cur.block * R;
      // ---- the rows: q, positions, what they see of the nodes
      const uint8_t* q = a.q + cur.b * a.sqb + static_cast<int64_t>(cur.h) * a.G * a.sqh;
#pragma unroll 1
      for (int i = tid; i < R * (D / 8); i += kSoft) {
        const int r = i / (D / 8), ch = i % (D / 8), Rg = row0 + r, node = paged_node(a, Rg);
        uint4 w = make_uint4(0, 0, 0, 0);
        if (Rg < rows_total && node < rq.n) w = *reinterpret_cast<const uint4*>(q + node * a.sqn + (Rg - node * a.G) * a.sqh + ch * 16);
        *reinterpret_cast<uint4*>(smem + L::kOffQ + block_off(R, r, ch)) = w;
      }
      if (tid < R) {
        const int Rg = row0 + tid, at = paged_node(a, Rg);
        const int node = Rg < rows_total && at < rq.n ? at : -1;
        s_node[tid] = node;
        uint32_t anc = 0;
        int depth = max(node, 0);
        if (a.parents && node >= 0) {
          const int32_t* par = a.parents + static_cast<int64_t>(cur.b) * a.N;
          depth = -1;
#pragma unroll 1
          for (int m = node; m >= 0; m = tree_up(par, m)) {
            anc |= 1u << m;   // up to 32 rows have up to 32 nodes
            ++depth;
          }
          s_depth[node] = depth;
        } else if (node >= 0) {
          anc = node >= 31 ? 0xffffffffu : (2u << node) - 1u;
          s_depth[node] = node;
        }
        s_anc[tid] = anc;
        s_pos[tid] = rq.base + depth;
        s_slope[tid] = a.slopes && node >= 0 ? a.slopes[cur.h * a.G + Rg - node * a.G] * kLog2e : 0.f;
        s_m[tid] = 0.f;
        s_seen[tid] = 0;
      }
#pragma unroll 1
      for (int i = tid; i < R * (D / 16); i += kSoft) s_inf[i] = 0;
      if (row == 0) *unseen = 1;
      fence_async_smem();
      mbar_arrive(q_ready);
      named_barrier_sync(3, kSoft);
      const uint32_t live = __ballot_sync(0xffffffffu, lane < 16 && s_node[r00 + (lane & 15)] >= 0);   // rows with a node

      float2 l[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) l[r] = make_float2(0.f, 0.f);
      bool any_inf = false;
#pragma unroll 1
      for (int i = 0; i < cur.n; ++i, ++n) {
        const int tok0 = (cur.t0 + i) * kPgTile, tok = tok0 + row;
        const uint32_t sb = n & 1;
        wait_or_fail(s_ready + 8 * sb, (n >> 1) & 1, fail);
        tc_fence_after();
        uint32_t w[16];
        tmem_ld16(t_lane + sb * R + r00, w);
        const uint32_t there = s_there[n & 15];
        const bool special = cur.special(a, tok0, there);   // the same for the whole CTA
        tmem_ld_wait();
        tmem_use(w);
        tc_fence_before();
        if (lane == 0) mbar_arrive(s_free + 8 * sb);
        float2 x[8];
        float top = -INFINITY;
        const int m = tok - rq.base;   // the token's node, negative in the prefix
        if (plain) {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = __fmul2_rn(make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1])), coef2);
        } else {
          if (a.cap > kPgFarCap) {
            cap_far(w, a);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = make_float2(paged_score(a, __uint_as_float(w[2 * j])), paged_score(a, __uint_as_float(w[2 * j + 1])));
          }
          if (a.slopes) {
            const int at = m < 0 || m >= rq.n ? tok : rq.base + s_depth[m];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float2 sl = reinterpret_cast<const float2*>(s_slope + r00)[j];
              const int2 p = reinterpret_cast<const int2*>(s_pos + r00)[j];
              x[j].x = fmaf(sl.x, static_cast<float>(at - p.x), x[j].x);
              x[j].y = fmaf(sl.y, static_cast<float>(at - p.y), x[j].y);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 mm = reinterpret_cast<const float4*>(s_m + r00)[j];
          x[2 * j] = __fadd2_rn(x[2 * j], make_float2(-mm.x, -mm.y));
          x[2 * j + 1] = __fadd2_rn(x[2 * j + 1], make_float2(-mm.z, -mm.w));
          top = fmaxf(fmaxf(fmaxf(top, x[2 * j].x), x[2 * j].y), fmaxf(x[2 * j + 1].x, x[2 * j + 1].y));
        }
        if (named_barrier_or(3, kSoft, top > kPgSlack + kPgLift<T> || special || *unseen)) {   // of one mind, whatever `special` read
          // ---- slow path: masks, maxima, V rows that must not be read
          const bool valid = there >> (row >> a.c.page_shift) & 1 && tok < rq.len;
          uint32_t see = valid ? live : 0u;
          if (see && (tok >= rq.base || tok < cur.inside)) {
            const int at = m < 0 ? tok : rq.base + s_depth[m];
            const uint32_t bit = m < 0 ? 0u : m;
            uint32_t bits = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint4 anc = reinterpret_cast<const uint4*>(s_anc + r00)[j];
              const int4 p = reinterpret_cast<const int4*>(s_pos + r00)[j];
              bits |= ((m < 0 || anc.x >> bit & 1) && p.x - at < a.window ? 1u : 0u) << 4 * j;
              bits |= ((m < 0 || anc.y >> bit & 1) && p.y - at < a.window ? 2u : 0u) << 4 * j;
              bits |= ((m < 0 || anc.z >> bit & 1) && p.z - at < a.window ? 4u : 0u) << 4 * j;
              bits |= ((m < 0 || anc.w >> bit & 1) && p.w - at < a.window ? 8u : 0u) << 4 * j;
            }
            see &= bits;
          }
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            float& v = r & 1 ? x[r / 2].y : x[r / 2].x;
            if (!(see >> r & 1)) v = -INFINITY;
            const float mx = warp_max(v);
            if (lane == 0) max_w[r] = mx;
          }
          if (named_barrier_or(3, kSoft, special)) {
            const uint32_t s = 2 * n + 1, st = s % kSt;
            wait_or_fail(full + 8 * st, (s / kSt) & 1, fail);
            uint8_t* vt = smem + st * L::kTileBytes;
            uint32_t odd = 0;
            if (valid) {
#pragma unroll
              for (int ch = 0; ch < D / 8; ++ch) odd |= nonfinite8<T>(*reinterpret_cast<const uint4*>(vt + block_off(kPgTile, row, ch)));
            } else if (grp == 0) {
#pragma unroll
              for (int ch = 0; ch < D / 8; ++ch) *reinterpret_cast<uint4*>(vt + block_off(kPgTile, row, ch)) = make_uint4(0, 0, 0, 0);
            }
            if (named_barrier_or(3, kSoft, odd != 0)) {   // rare
              any_inf = true;
              note_nonfinite<T, D>(vt, row, odd ? see : 0u, s_inf + r00 * (D / 16));
              named_barrier_sync(3, kSoft);   // every group has read the row
              if (grp == 0 && odd)
#pragma unroll 1
                for (int ch = 0; ch < D / 8; ++ch) take_out8<T>(reinterpret_cast<uint4*>(vt + block_off(kPgTile, row, ch)));
            }
            fence_async_smem();
          }
          // one thread per row: by how much its maximum rises; a row's first maximum may lie anywhere
          if (row < 16) {
            const float mx = fmaxf(fmaxf(max_g[row], max_g[20 + row]), fmaxf(max_g[40 + row], max_g[60 + row])) - kPgLift<T>;
            const bool seen = s_seen[r00 + row];
            const float up = seen ? fmaxf(mx, 0.f) : mx == -INFINITY ? 0.f : mx;
            s_up[r00 + row] = up;
            s_f[r00 + row] = seen ? ex2(-up) : 1.f;
            s_m[r00 + row] += up;
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
            wait_or_fail(p_free, (n - 1) & 1, fail);
            tc_fence_after();
#pragma unroll 1
            for (int t = 0; t < 2; ++t) {
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
        // ---- P, its sum and its two terms
        uint32_t h[2][8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 p = make_float2(ex2(x[j].x), ex2(x[j].y));
          l[j] = __fadd2_rn(l[j], p);
          h[0][j] = T::pack2(p.x, p.y);
          const float2 back = T::unpack2(h[0][j]);
          h[1][j] = T::pack2(p.x - back.x, p.y - back.y);
        }
        if (n > 0) wait_or_fail(p_free, (n - 1) & 1, fail);   // the products of the last tile have read its P
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            *reinterpret_cast<uint4*>(smem + L::kOffP + block_off(kPgTile, row, (t * R + r00) / 8 + k)) =
                make_uint4(h[t][4 * k], h[t][4 * k + 1], h[t][4 * k + 2], h[t][4 * k + 3]);
        tc_fence_before();
        fence_async_smem();
        mbar_arrive(p_ready);
      }
      // ---- the piece's sums and O^T
      wait_or_fail(p_free, (n - 1) & 1, fail);
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
      float* part = a.part + static_cast<int64_t>(2 * blockIdx.x + (first ? 0 : 1)) * R * (D + 2);
      if (row < 16) {
        const int r = r00 + row, Rg = row0 + r, node = paged_node(a, Rg);
        const float sum = s_node[r] < 0 ? 0.f
                          : *fail       ? __int_as_float(0x7fc00000)
                                        : (max_g[row] + max_g[20 + row]) + (max_g[40 + row] + max_g[60 + row]);
        const int64_t at = (static_cast<int64_t>(cur.b) * a.N + node) * a.Hq + cur.h * a.G + (Rg - node * a.G);
        if (cur.whole) {
          if (a.lse && Rg < rows_total) a.lse[at] = sum == 0.f ? -INFINITY : (s_m[r] + log2f(sum)) * kLn2;
        } else {
          *reinterpret_cast<float2*>(part + R * D + r * 2) = make_float2(sum == 0.f ? -INFINITY : s_m[r], sum);
        }
        const float f = sum == 0.f ? 0.f : cur.whole ? 1.f / sum : 1.f;   // a row that saw nothing is zero
        s_out[r] = make_int4(static_cast<int>(at & 0xffffffff), static_cast<int>(at >> 32), __float_as_int(f), Rg < rows_total);
      }
      named_barrier_sync(bar, 128);
      tc_fence_after();
      if (row < D) {
#pragma unroll 1
        for (int j = 0; j < 16 && s_out[r00 + j].w; j += 4) {
          uint32_t w[2][4];
          tmem_ld4(t_o + j, w[0]);
          tmem_ld4(t_o + R + j, w[1]);
          tmem_ld_wait();
          tmem_use(w[0]);
          tmem_use(w[1]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = r00 + j + k;
            const int4 to = s_out[r];
            if (!to.w) break;
            const float f = __int_as_float(to.z);
            float o = f == 0.f ? 0.f : (__uint_as_float(w[0][k]) + __uint_as_float(w[1][k])) * f;
            if (any_inf && f != 0.f)
              o = put_back(o, s_inf[r * (D / 16) + (row >> 5)] >> (row & 31) & 1, s_inf[r * (D / 16) + D / 32 + (row >> 5)] >> (row & 31) & 1);
            if (cur.whole) {
              const int64_t at = static_cast<uint32_t>(to.x) | static_cast<int64_t>(to.y) << 32;
              static_cast<uint16_t*>(a.out)[at * D + row] = static_cast<uint16_t>(T::pack2(o, 0.f));
            } else {
              part[r * D + row] = o;
            }
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      named_barrier_sync(3, kSoft);   // the shared rows are free for the next piece
    }
  }
  __syncthreads();
  if (s_fail) settle_after_failure();   // before TMEM goes
  __syncthreads();
  if (tid == 0) a.failed[blockIdx.x] = s_fail;
  if (warp == 4 * MT + 1) tmem_free(tmem, L::kTmem);
}

}  // namespace sv
