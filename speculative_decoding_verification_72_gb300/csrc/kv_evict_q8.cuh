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
// scores as unsigned integers) go to shared memory once; radix passes of 11, 11
// and 10 bits find the keep-th key, and end early once a digit settles it. A
// warp then owns a run of slots: it counts kept ones, holes and movers, takes
// its places from all warps' counts and marks them in order, two sweeps over
// the keys with one barrier between; the last loop fetches what each kept slot
// is filled from. Loads are issued in batches, and code that runs once is kept
// short (its instruction fetches are what a small call waits for). 512 threads, so that two CTAs share an SM
// (24 requests of 8 heads are 192 CTAs: one wave, not two).
// kv_evict_move_kernel, one warp per destination page (two pages of 16), moves
// the rows.
//
// Measured: 24 prompts of up to 8192 tokens down to 4096, 8 heads of 128, pages
// whose scales differ by up to 4: 36 us where an earlier call has already raised
// the scales of the pages that stay (17 select, 16 move; the bytes would take
// 14), and 23 us more, all in the move, on a cache as appends leave it: there
// the rows that stay on a page whose scale rises are rounded again, 139 MB of
// codes read and written instead of 80 (with those the bytes would take 23). 2
// requests of 1090 down to 1024: 12 us and 16. Bound by latencies in a row: the
// selection is one CTA a (request, head), phases with a barrier between; the
// move waits for source, scale and codes (11 of its warps wait an issue).
#pragma once

#include "q8_common.cuh"

namespace sv {

constexpr int kEvThreads = 512;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvStep = 8;                         // slots of a thread whose loads are under way at once
constexpr uint32_t kEvHole = 0x80000000u;
constexpr int kEvBins = 2048;
static_assert(kEvBins == 4 * kEvThreads, "four bins a thread");
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
  uint32_t* src;               // [B, H, keep]: the row (of [pages * H * P]) each kept slot is filled from
  uint32_t* movers;            // [B, H, keep]
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

// Out of line: past the keys held in shared memory.
__device__ __noinline__ uint32_t evict_key_again(const float* s, const int32_t* p, int sinks, int from) {
  return evict_key(*s, *p, sinks, from);
}

__global__ void __launch_bounds__(kEvThreads, 2) kv_evict_select_kernel(const EvictArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  uint32_t* s_hist = reinterpret_cast<uint32_t*>(smem);   // kEvBins
  uint32_t* s_key = s_hist + kEvBins;                     // n_keys
  __shared__ uint32_t s_warp[kEvWarps], s_bin, s_above, s_in_bin;
  __shared__ int4 s_count[kEvWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int H = a.c.Hkv;
  const int b = blockIdx.x / H, h = blockIdx.x - b * H;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * a.S;
  const float* sc = a.scores + row;
  const int32_t* ps = a.positions + row;
  float* osc = a.out_scores + row;
  int32_t* ops = a.out_positions + row;
  reinterpret_cast<uint4*>(s_hist)[tid] = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();
  // The first slots' scores and pages are read with the length, not after it.
  const int32_t* table = a.c.table + static_cast<int64_t>(b) * a.c.max_pages;
  const int32_t page0 = table[min(tid, a.c.max_pages - 1)];
  const int from = a.protect_from ? a.protect_from[b] : INT_MAX;
  const int n = a.seq_len[b];
  const int keep = a.keep;
  const bool fits = n >= 0 && n <= a.S && n <= static_cast<int64_t>(a.c.max_pages) << a.c.page_shift;
  bool ok = fits;
  int last = a.S - 1;
  // ---- keys and the first digit's histogram
#pragma unroll 1
  for (int jj = tid; jj <= last; jj += kEvThreads * kEvStep) {
    float s[kEvStep];
    int32_t p[kEvStep];
#pragma unroll
    for (int i = 0; i < kEvStep; ++i) {
      const int j = min(jj + i * kEvThreads, last);
      s[i] = sc[j];
      p[i] = ps[j];
    }
    last = fits && n > keep ? n - 1 : -1;
#pragma unroll
    for (int i = 0; i < kEvStep; ++i) {
      const int j = jj + i * kEvThreads;
      if (j > last) break;
      const uint32_t k = evict_key(s[i], p[i], a.sinks, from);
      if (j < a.n_keys) s_key[j] = k;
      atomicAdd(&s_hist[k >> 21], 1u);
    }
  }
  if (fits) {
    const int pages = (n + (1 << a.c.page_shift) - 1) >> a.c.page_shift;
    if (tid < pages) ok = page0 >= 0 && page0 < a.c.num_pages;
    for (int j = tid + kEvThreads; j < pages; j += kEvThreads) ok = ok && q8_page(a.c, b, j) >= 0;
  }
  ok = __syncthreads_and(ok);
  const bool work = ok && n > keep;
  const int left = work ? keep : min(max(n, 0), a.S);   // slots that hold a token afterwards
  if (tid == 0) {
    if (h == 0) {
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
  auto key_of = [&](int j) { return j < a.n_keys ? s_key[j] : evict_key_again(sc + j, ps + j, a.sinks, from); };
  uint32_t prefix = 0, mask = 0, want = keep, in_bin = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digit = pass == 2 ? 1023u : 2047u;
    if (pass > 0) {
#pragma unroll 4
      for (int j = tid; j < n; j += kEvThreads) {
        const uint32_t k = key_of(j);
        if ((k & mask) == prefix) atomicAdd(&s_hist[k >> shift & digit], 1u);
      }
      __syncthreads();
    }
    // from the largest digit down, four bins a thread: the one that holds the want-th
    const int b0 = kEvBins / 4 - 1 - tid;
    const uint4 c = reinterpret_cast<const uint4*>(s_hist)[b0];
    reinterpret_cast<uint4*>(s_hist)[b0] = make_uint4(0u, 0u, 0u, 0u);
    const uint32_t sum = c.x + c.y + c.z + c.w;
    uint32_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    uint32_t before = inc - sum + __reduce_add_sync(0xffffffffu, lane < warp ? s_warp[lane] : 0u);
    if (before < want && want <= before + sum) {
      int bin = b0 * 4 + 3;
      uint32_t in = c.w;
      if (want > before + in) before += in, in = c.z, --bin;
      if (want > before + in) before += in, in = c.y, --bin;
      if (want > before + in) before += in, in = c.x, --bin;
      s_bin = bin;
      s_above = before;
      s_in_bin = in;
    }
    __syncthreads();
    prefix |= s_bin << shift;
    mask |= digit << shift;
    want -= s_above;
    in_bin = s_in_bin;
    if (want == in_bin) break;
  }
  // ---- kept: keys above prefix (as far as its digits are settled), and the first `want` slots that equal it.
  // A warp's run of slots: counts above and equal, below slot `keep` and from there on.
  const int run = (n + kEvThreads - 1) / kEvThreads * 32;
  const int j0 = min(warp * run, n), j1 = min(j0 + run, n);
  const int jk = min(max(keep, j0), j1);   // the run's first slot past the budget
  const bool ties = want != in_bin;
  int count[4];
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    int gt = 0, eq = 0;
#pragma unroll 4
    for (int j = (part ? jk : j0) + lane; j < (part ? j1 : jk); j += 32) {
      const uint32_t k = key_of(j) & mask;
      gt += k > prefix;
      eq += k == prefix;
    }
    count[part] = __reduce_add_sync(0xffffffffu, gt);
    count[2 + part] = __reduce_add_sync(0xffffffffu, eq);
  }
  if (lane == 0) s_count[warp] = make_int4(count[0], count[1], count[2], count[3]);
  __syncthreads();
  int eq_at, hole_at, move_at, moves;   // this warp's: equal slots before it, its first places in the lists
  {
    const int4 c = lane < kEvWarps ? s_count[lane] : make_int4(0, 0, 0, 0);
    int eq = c.z + c.w;
#pragma unroll
    for (int o = 1; o < kEvWarps; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, eq, o);
      if (lane >= o) eq += up;
    }
    eq -= c.z + c.w;
    const int room = static_cast<int>(want) - eq;
    const int keep_lo = min(max(room, 0), c.z), keep_hi = min(max(room - c.z, 0), c.w);
    const int r0 = min(min(lane, kEvWarps) * run, n), r1 = min(r0 + run, n);
    const int lo = min(r1, keep) - min(r0, keep);
    const int holes = lane < kEvWarps ? lo - c.x - keep_lo : 0, moved = c.y + keep_hi;
    eq_at = __shfl_sync(0xffffffffu, eq, warp);
    hole_at = __reduce_add_sync(0xffffffffu, lane < warp ? holes : 0);
    move_at = __reduce_add_sync(0xffffffffu, lane < warp ? moved : 0);
    moves = __reduce_add_sync(0xffffffffu, moved);
  }
  // Kept slots below `keep` are marked with themselves, holes with their place
  // in the list of movers; the marks take the place of the keys, each of which
  // is read for the last time by the lane that writes its mark.
  uint32_t* src = a.src + static_cast<int64_t>(blockIdx.x) * keep;
  uint32_t* movers = moves <= kEvBins ? s_hist : a.movers + static_cast<int64_t>(blockIdx.x) * keep;
  const uint32_t below = (1u << lane) - 1;
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {   // the holes, then the movers
    int at = part ? move_at : hole_at;
    const int end = part ? j1 : jk;
#pragma unroll 1
    for (int j = (part ? jk : j0) + lane; j - lane < end; j += 32) {
      const uint32_t k = j < end ? key_of(j) & mask : 0u;
      bool yes = k >= prefix;
      if (ties) {
        const uint32_t eq = __ballot_sync(0xffffffffu, j < end && k == prefix);
        yes = k > prefix || (k == prefix && eq_at + __popc(eq & below) < static_cast<int>(want));
        eq_at += __popc(eq);
      }
      const bool listed = j < end && yes == (part == 1);
      const uint32_t who = __ballot_sync(0xffffffffu, listed);
      const uint32_t place = at + __popc(who & below);
      at += __popc(who);
      if (part == 0) {
        const uint32_t mark = listed ? kEvHole | place : j;
        if (j < end) {
          if (j < a.n_keys)
            s_key[j] = mark;
          else
            src[j] = mark;
        }
      } else if (listed) {
        movers[place] = j;
      }
    }
  }
  if (tid == 0) a.n_moves[blockIdx.x] = moves;
  __syncthreads();
  const int pmask = (1 << a.c.page_shift) - 1;
#pragma unroll 1
  for (int jj = tid; jj < keep; jj += kEvThreads * kEvStep) {
    float s[kEvStep];
    int32_t p[kEvStep];
    uint32_t at[kEvStep];
#pragma unroll
    for (int i = 0; i < kEvStep; ++i) {
      // Past the budget: the thread's own first slot again. Another thread's mark may
      // be gone by now, with a row of the pool in its place (src past n_keys).
      const int j = jj + i * kEvThreads < keep ? jj + i * kEvThreads : jj;
      uint32_t fr = j < a.n_keys ? s_key[j] : src[j];
      if (fr & kEvHole) fr = movers[fr & ~kEvHole];
      at[i] = fr;
    }
#pragma unroll
    for (int i = 0; i < kEvStep; ++i) {
      s[i] = sc[at[i]];
      p[i] = ps[at[i]];
      at[i] = ((static_cast<uint32_t>(table[at[i] >> a.c.page_shift]) * H + h) << a.c.page_shift) + (at[i] & pmask);
    }
#pragma unroll
    for (int i = 0; i < kEvStep; ++i) {
      const int j = jj + i * kEvThreads;
      if (j >= keep) break;
      src[j] = at[i];
      osc[j] = s[i];
      ops[j] = p[i];
    }
  }
  __syncthreads();   // scores may be updated in place: the sources are read before they are cleared
  for (int j = keep + tid; j < a.S; j += kEvThreads) {
    osc[j] = 0.f;
    ops[j] = -1;
  }
}

// One warp per destination page of a (request, head), or per two pages of 16
// slots: lane l looks after slot l of each 32. The rows that change are listed
// in shared memory, and two instructions' worth of them are under way at once
// (24 prompts of 8192 tokens down to 4096, scales settled: 34.8 us the call; with
// four 37.6, with one 37.2, at 8, 12 and 16 CTAs an SM).
template <int D>
__global__ void __launch_bounds__(kMvWarps * 32, 12) kv_evict_move_kernel(const EvictArgs a) {
  constexpr int kLpr = D / 16;          // lanes per row
  constexpr int kRpi = 32 / kLpr;       // rows per instruction
  struct __align__(16) Item {
    uint32_t from, to;                  // rows
    float fk, fv;                       // factors
  };
  __shared__ Item s_item[kMvWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int H = a.c.Hkv, P = 1 << a.c.page_shift;
  const int unit = max(P, 32);          // slots of a warp
  const int groups = (a.keep + kMvWarps * unit - 1) / (kMvWarps * unit);
  const int bh = blockIdx.x / groups, first = ((blockIdx.x - bh * groups) * kMvWarps + warp) * unit;
  const int b = bh / H, h = bh - b * H;
  grid_dep_wait();
  grid_dep_launch();
  if (first >= a.keep) return;
  const bool in = first + lane < a.keep;   // past it: the second of two pages of 16
  const uint32_t* src = a.src + static_cast<int64_t>(bh) * a.keep + first;
  const int32_t own_page = in ? q8_page(a.c, b, (first + lane) >> a.c.page_shift) : -1;   // of the lane's page
  uint32_t from = in ? src[lane] : 0u;   // not to be used as an address before n_moves is known
  if (a.n_moves[bh] == 0 || first >= a.keep) return;
  const uint32_t own = static_cast<uint32_t>(own_page) * H + h;
  const float k0 = in ? a.c.ks[own] : 0.f, v0 = in ? a.c.vs[own] : 0.f;
  // the page's new scale: the largest of its sources'
  float k1 = in ? a.c.ks[from >> a.c.page_shift] : 0.f, v1 = in ? a.c.vs[from >> a.c.page_shift] : 0.f;
  float km = k1, vm = v1;
  bool any = in && from >> a.c.page_shift != own;
#pragma unroll 1
  for (int g = 32; g < P; g += 32) {
    const uint32_t p = src[g + lane] >> a.c.page_shift;
    any = any || p != own;
    km = fmaxf(km, a.c.ks[p]);
    vm = fmaxf(vm, a.c.vs[p]);
  }
  if (!__any_sync(0xffffffffu, any)) return;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
    if (o < P) {
      km = fmaxf(km, __shfl_xor_sync(0xffffffffu, km, o));
      vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, o));
    }
#pragma unroll 1
  for (int g = 0; g < unit; g += 32) {
    if (g > 0) {
      from = src[g + lane];
      k1 = a.c.ks[from >> a.c.page_shift];
      v1 = a.c.vs[from >> a.c.page_shift];
    }
    const uint32_t to = (own << a.c.page_shift) + ((first + g + lane) & (P - 1));
    // a scale of 0 stands for zeros, whatever the codes
    const float fk = k1 == km ? 1.f : k1 / km, fv = v1 == vm ? 1.f : v1 / vm;
    const bool change = in && (from != to || fk != 1.f || fv != 1.f);
    const uint32_t who = __ballot_sync(0xffffffffu, change);
    __syncwarp();
    if (change) s_item[warp][__popc(who & ((1u << lane) - 1))] = {from, to, fk, fv};
    __syncwarp();
    const int count = __popc(who);
#pragma unroll 1
    for (int r0 = lane / kLpr; r0 < count; r0 += kRpi * 2) {
      uint4 k[2], v[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (r0 + i * kRpi < count) {
          const int64_t o = static_cast<int64_t>(s_item[warp][r0 + i * kRpi].from) * D + lane % kLpr * 16;
          k[i] = *reinterpret_cast<const uint4*>(a.c.k + o);
          v[i] = *reinterpret_cast<const uint4*>(a.c.v + o);
        }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (r0 + i * kRpi < count) {
          const Item t = s_item[warp][r0 + i * kRpi];
          const int64_t o = static_cast<int64_t>(t.to) * D + lane % kLpr * 16;
          auto put = [&](uint8_t* codes, uint4 w, float f) {
            if (f != 1.f) {
              w.x = e4m3_rescale4(w.x, f);
              w.y = e4m3_rescale4(w.y, f);
              w.z = e4m3_rescale4(w.z, f);
              w.w = e4m3_rescale4(w.w, f);
            }
            *reinterpret_cast<uint4*>(codes + o) = w;
          };
          put(a.c.k, k[i], t.fk);
          put(a.c.v, v[i], t.fv);
        }
    }
  }
  if (in && (first + lane & (P - 1)) == 0) {
    if (km != k0) a.c.ks[own] = km;
    if (vm != v0) a.c.vs[own] = vm;
  }
}

}  // namespace sv
