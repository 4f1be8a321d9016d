// Eviction from the 8-bit paged cache by accumulated attention weight.
//
// A (request, kv head) holds n tokens in slots [0, n). Down to a budget of
// `keep` slots (whole pages, so the pages past it fall free), the tokens kept
// are the first `keep` by: protected ones (position below sinks, or at least
// protect_from), then the higher score, then the lower slot. Attention does
// not depend on the order of slots, so nothing is compacted in order: kept
// tokens of slots >= keep move into the slots < keep that lost theirs, the
// i-th mover to the i-th hole (both ascending). Sources and destinations lie
// in different pages, which makes the move race-free in place, and its bytes
// are those of the moved rows alone.
//
// A page's scale becomes the largest of its slots' source pages' scales; rows
// whose scale changes are rescaled (one rounding, exact products for the
// powers of two that the cache is written with).
//
// kv_evict_select_kernel, one CTA per (request, head): keys (the order of the
// scores as unsigned integers) go to shared memory once, three radix passes
// of 11, 11 and 10 bits find the keep-th key, one ordered pass with block
// scans ranks ties, holes and movers. kv_evict_move_kernel, one warp per
// destination page, moves the rows.
#pragma once

#include "q8_common.cuh"

namespace sv {

constexpr int kEvThreads = 1024;
constexpr int kEvPer = 4;                          // consecutive slots per thread in the ordered pass
constexpr int kEvChunk = kEvThreads * kEvPer;
constexpr int kEvBins = 2048;
constexpr int kEvMaxKeys = 40960;                  // keys held in shared memory; later ones are formed again
constexpr int kMvWarps = 4;

struct EvictArgs {
  Q8View c;
  const int32_t* seq_len;      // [B]
  const float* scores;         // [B, H, S]
  const int32_t* positions;    // [B, H, S]
  const int32_t* protect_from; // [B] or nullptr
  float* out_scores;           // [B, H, S]
  int32_t* out_positions;      // [B, H, S]
  int32_t* out_len;            // [B]
  int32_t* status;             // [B] or nullptr
  int32_t* src;                // [B, H, keep]: the slot each kept slot is filled from
  int32_t* movers;             // [B, H, keep]
  int32_t* holes;              // [B, H, keep]
  int32_t* n_moves;            // [B, H]
  int32_t B, S, keep, sinks, n_keys;
};

// Scores as unsigned integers in the same order; -0 as +0, NaN below all.
__device__ __forceinline__ uint32_t evict_key(float s, int pos, int sinks, int from) {
  if (pos < sinks || pos >= from) return 0xffffffffu;
  if (s != s) return 0u;
  const uint32_t u = __float_as_uint(s + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive sum over the CTA of v; *total the CTA's sum.
__device__ __forceinline__ uint32_t evict_scan(uint32_t v, uint32_t* s_warp, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  uint32_t w = s_warp[lane], winc = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t up = __shfl_up_sync(0xffffffffu, winc, o);
    if (lane >= o) winc += up;
  }
  *total = __shfl_sync(0xffffffffu, winc, 31);
  return inc - v + __shfl_sync(0xffffffffu, winc - w, warp);
}

__global__ void __launch_bounds__(kEvThreads, 1) kv_evict_select_kernel(const EvictArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  uint32_t* s_hist = reinterpret_cast<uint32_t*>(smem);   // kEvBins
  uint32_t* s_key = s_hist + kEvBins;                     // n_keys
  __shared__ uint32_t s_warp[32], s_bin, s_above, s_in_bin;
  const int tid = threadIdx.x;
  const int H = a.c.Hkv;
  const int b = blockIdx.x / H;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * a.S;
  grid_dep_wait();
  grid_dep_launch();
  const int n = a.seq_len[b];
  const int from = a.protect_from ? a.protect_from[b] : INT_MAX;
  const float* sc = a.scores + row;
  const int32_t* ps = a.positions + row;
  float* osc = a.out_scores + row;
  int32_t* ops = a.out_positions + row;
  bool ok = n >= 0 && n <= a.S && n <= static_cast<int64_t>(a.c.max_pages) << a.c.page_shift;
  if (ok)
    for (int j = tid; j < (n + (1 << a.c.page_shift) - 1) >> a.c.page_shift; j += kEvThreads)
      ok = ok && q8_page(a.c, b, j) >= 0;
  ok = __syncthreads_and(ok);
  const int keep = a.keep;
  const bool work = ok && n > keep;
  const int left = work ? keep : min(max(n, 0), a.S);   // slots that hold a token afterwards
  if (tid == 0) {
    if (blockIdx.x % H == 0) {
      a.out_len[b] = work ? keep : n;
      if (a.status) a.status[b] = ok ? 0 : SV_STATUS_BAD_PAGE;
    }
    if (!work) a.n_moves[blockIdx.x] = 0;
  }
  if (!work) {
    for (int j = tid; j < a.S; j += kEvThreads) {
      osc[j] = j < left ? sc[j] : 0.f;
      ops[j] = j < left ? ps[j] : -1;
    }
    return;
  }
  // ---- the keep-th largest key
  auto key_of = [&](int j) { return j < a.n_keys ? s_key[j] : evict_key(sc[j], ps[j], a.sinks, from); };
  for (int j = tid; j < n && j < a.n_keys; j += kEvThreads) s_key[j] = evict_key(sc[j], ps[j], a.sinks, from);
  uint32_t prefix = 0, mask = 0, want = keep, in_bin = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digit = pass == 2 ? 1023u : 2047u;
    for (int j = tid; j < kEvBins; j += kEvThreads) s_hist[j] = 0;
    __syncthreads();
    for (int j = tid; j < n; j += kEvThreads) {
      const uint32_t k = key_of(j);
      if ((k & mask) == prefix) atomicAdd(&s_hist[k >> shift & digit], 1u);
    }
    __syncthreads();
    // from the largest digit down: the bin that holds the want-th
    const int b0 = kEvBins - 1 - 2 * tid;
    const uint32_t h0 = s_hist[b0], h1 = s_hist[b0 - 1];
    uint32_t total;
    const uint32_t before = evict_scan(h0 + h1, s_warp, &total);
    if (before < want && want <= before + h0 + h1) {
      const bool first = want <= before + h0;
      s_bin = first ? b0 : b0 - 1;
      s_above = first ? before : before + h0;
      s_in_bin = first ? h0 : h1;
    }
    __syncthreads();
    prefix |= s_bin << shift;
    mask |= digit << shift;
    want -= s_above;
    in_bin = s_in_bin;
    __syncthreads();
  }
  // kept: keys above prefix, and the first `want` of the in_bin slots that equal it
  const bool ties = want != in_bin;
  int32_t* src = a.src + static_cast<int64_t>(blockIdx.x) * keep;
  int32_t* movers = a.movers + static_cast<int64_t>(blockIdx.x) * keep;
  int32_t* holes = a.holes + static_cast<int64_t>(blockIdx.x) * keep;
  uint32_t eq_run = 0, hole_run = 0, move_run = 0;
  for (int j0 = 0; j0 < n; j0 += kEvChunk) {
    const int j = j0 + tid * kEvPer;
    uint32_t k[kEvPer], eq = 0;
#pragma unroll
    for (int i = 0; i < kEvPer; ++i) {
      k[i] = j + i < n ? key_of(j + i) : 0u;
      eq += j + i < n && k[i] == prefix;
    }
    uint32_t rank = 0, total;
    if (ties) {
      rank = eq_run + evict_scan(eq, s_warp, &total);
      eq_run += total;
    }
    uint32_t kept = 0, packed = 0;   // holes in the low half, movers in the high half
#pragma unroll
    for (int i = 0; i < kEvPer; ++i) {
      if (j + i >= n) continue;
      bool yes = k[i] > prefix;
      if (k[i] == prefix) yes = !ties || rank++ < want;
      kept |= static_cast<uint32_t>(yes) << i;
      if (j + i < keep)
        packed += !yes;
      else
        packed += static_cast<uint32_t>(yes) << 16;
    }
    const uint32_t at = evict_scan(packed, s_warp, &total);
    uint32_t hole = hole_run + (at & 0xffffu), move = move_run + (at >> 16);
    hole_run += total & 0xffffu;
    move_run += total >> 16;
#pragma unroll
    for (int i = 0; i < kEvPer; ++i) {
      if (j + i >= n) continue;
      const bool yes = kept >> i & 1;
      if (j + i < keep) {
        if (yes) {
          src[j + i] = j + i;
          osc[j + i] = sc[j + i];
          ops[j + i] = ps[j + i];
        } else {
          holes[hole++] = j + i;
        }
      } else if (yes) {
        movers[move++] = j + i;
      }
    }
  }
  __syncthreads();
  for (uint32_t i = tid; i < move_run; i += kEvThreads) {
    const int to = holes[i], fr = movers[i];
    src[to] = fr;
    osc[to] = sc[fr];
    ops[to] = ps[fr];
  }
  if (tid == 0) a.n_moves[blockIdx.x] = move_run;
  __syncthreads();   // scores may be updated in place: the sources are read before they are cleared
  for (int j = keep + tid; j < a.S; j += kEvThreads) {
    osc[j] = 0.f;
    ops[j] = -1;
  }
}

// One warp per destination page of a (request, head).
template <int D>
__global__ void __launch_bounds__(kMvWarps * 32) kv_evict_move_kernel(const EvictArgs a) {
  constexpr int kLpr = D / 16;          // lanes per row
  constexpr int kRpi = 32 / kLpr;       // rows per iteration
  __shared__ int32_t s_page[kMvWarps][128];   // source page, then row within it, of each slot
  __shared__ int32_t s_row[kMvWarps][128];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int H = a.c.Hkv, P = 1 << a.c.page_shift;
  const int pages = a.keep >> a.c.page_shift;
  const int groups = (pages + kMvWarps - 1) / kMvWarps;
  const int bh = blockIdx.x / groups, pg = (blockIdx.x - bh * groups) * kMvWarps + warp;
  const int b = bh / H, h = bh - b * H;
  grid_dep_wait();
  grid_dep_launch();
  if (pg >= pages || a.n_moves[bh] == 0) return;
  const int32_t* src = a.src + static_cast<int64_t>(bh) * a.keep + (pg << a.c.page_shift);
  const int page = q8_page(a.c, b, pg);
  bool any = false;
  float km = 0.f, vm = 0.f;
  for (int j = lane; j < P; j += 32) {
    const int s = src[j];
    const int sp = q8_page(a.c, b, s >> a.c.page_shift);
    any = any || s != (pg << a.c.page_shift) + j;
    km = fmaxf(km, a.c.ks[static_cast<int64_t>(sp) * H + h]);
    vm = fmaxf(vm, a.c.vs[static_cast<int64_t>(sp) * H + h]);
    s_page[warp][j] = sp;
    s_row[warp][j] = s & (P - 1);
  }
  if (!__any_sync(0xffffffffu, any)) return;
  km = warp_max(km);
  vm = warp_max(vm);
  const int64_t own = static_cast<int64_t>(page) * H + h;
  const float k0 = a.c.ks[own], v0 = a.c.vs[own];
  __syncwarp();
  for (int r0 = 0; r0 < P; r0 += kRpi) {
    const int r = r0 + lane / kLpr;
    const int sp = s_page[warp][r];
    const int64_t from = static_cast<int64_t>(sp) * H + h;
    const bool moved = sp != page;
    const float fk = (moved ? a.c.ks[from] : k0) / km, fv = (moved ? a.c.vs[from] : v0) / vm;
    const int64_t so = ((from << a.c.page_shift) + s_row[warp][r]) * D + lane % kLpr * 16;
    const int64_t to = ((own << a.c.page_shift) + r) * D + lane % kLpr * 16;
    auto put = [&](uint8_t* codes, float f) {
      if (!moved && f == 1.f) return;
      uint4 w = *reinterpret_cast<const uint4*>(codes + so);
      if (f != 1.f) {
        w.x = e4m3_rescale4(w.x, f);
        w.y = e4m3_rescale4(w.y, f);
        w.z = e4m3_rescale4(w.z, f);
        w.w = e4m3_rescale4(w.w, f);
      }
      *reinterpret_cast<uint4*>(codes + to) = w;
    };
    put(a.c.k, fk);
    put(a.c.v, fv);
  }
  if (lane == 0) {
    if (km != k0) a.c.ks[own] = km;
    if (vm != v0) a.c.vs[own] = vm;
  }
}

}  // namespace sv
