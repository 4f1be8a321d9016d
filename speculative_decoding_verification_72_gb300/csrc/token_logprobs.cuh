// Log-probabilities of given tokens, entropy and top alternatives of logit
// rows, and their gradient.
//
// With c = log2(e) / T and m the row's maximum:
//   t_j = (x_j - m) c, s = sum 2^t_j, w = sum t_j 2^t_j
//   lse = m / T + ln s, log p_j = (x_j - m) / T - ln s, H = (log2 s - w / s) ln 2
// The difference is taken first, so logits near the maximum lose nothing
// however large it is, and masks of the type's lowest value overflow nowhere.
// (m, log2 s) is kept for the gradient, which would lose digits to their
// rounded sum lse. Sums are fp32, per thread relative to the thread's own
// maximum, then joined relative to the larger maximum.
//
// Gradient for upstream g (log-prob) and h (entropy):
//   dx_j = (1 / T) [g (1{j = token} - p_j) - h p_j (ln p_j + H)] = p_j (a0 + a1 t'_j) + (g / T) 1{j = token}
// with t' = (x - m) c - log2 s: one more pass over the row, no sums.
//
// Bound by memory: the forward pass reads each row once, the gradient reads and
// writes it once. A row is cut into equal segments of at most 16 KB (32 with
// alternatives); a thread
// has up to eight 16-byte vectors of one in registers, so maximum, sums and
// selection are passes over registers.
//
// Measured: 2048 rows of 50257 bf16, forward 42 us (issue-bound: an exponential
// and five instructions an element) and gradient 62 us (6.6 TB/s); 2048 rows of
// 151936 fp32, both 552 us (6.8 TB/s over its three passes); 192 rows of 128256
// bf16 with 20 alternatives 24 us, 14 without.
//
// Top alternatives by (logit, lower index): a bound that at least n_top
// elements of the segment reach is the n_top-th of the 64 maxima of groups of
// four threads; the few elements that reach it are gathered and ranked. If
// they overflow the buffer (many equal logits, or all but some hundred masked)
// the segment takes n_top rounds of CTA-wide maxima instead. Masked (-inf) tokens are no alternatives.
#pragma once

#include <cuda_bf16.h>

#include "sv_common.cuh"

namespace sv {

// Threads of a CTA: the selection's cost is one per CTA, so it has larger ones
// (192 rows of 128256 bf16, 20 alternatives: 29.8 us with 256, 33.3 with 128);
// without it smaller ones start and end more evenly (2048 rows of 50257 bf16,
// forward and gradient: 115 us with 128, 121 with 256).
constexpr int kLpThreads = 128;
constexpr int kLpTopThreads = 256;
constexpr int kLpVecs = 8;                                   // 16-byte vectors per thread
constexpr int kLpGroup = 4;                                  // threads of a group
constexpr int kLpGroups = kLpTopThreads / kLpGroup;
constexpr int kLpMaxTop = SV_MAX_TOP_ALTERNATIVES;
constexpr int kLpHits = 320;                                 // vectors that reach the bound
constexpr int kLpCand = 512;                                 // elements that do
constexpr float kLpFloor = -300.f;                           // 2^-300 is 0 in fp32

struct __align__(16) LpPartial {
  float m, s, w, pad;
};

struct LogprobArgs {
  const uint8_t* x;
  int64_t stride;              // bytes between rows
  const int32_t* tokens;       // [rows]
  int32_t rows, V, segs, per, n_top;   // per: vectors of a segment, a multiple of the CTA's threads
  float c, inv_t;              // log2(e) / T, 1 / T
  LpPartial* part;             // [rows, segs, warps of the CTA]
  uint64_t* cand;              // [rows, segs, n_top] keys in descending order, 0 past the last
  float* logprob;              // [rows]
  float* entropy;              // [rows] or nullptr
  float* lse;                  // [rows] or nullptr
  float4* saved;               // [rows] or nullptr: m, log2 s, H, 0
  int32_t* top_tokens;         // [rows, n_top]
  float* top_logprobs;         // [rows, n_top]
  int32_t* status;             // [rows] or nullptr
};

// Order of logits, then of lower indices; 0 for -inf and NaN.
__device__ __forceinline__ uint64_t lp_key(float x, int j) {
  if (!(x > -INFINITY)) return 0;
  const uint32_t u = __float_as_uint(x + 0.f);
  return static_cast<uint64_t>(u & 0x80000000u ? ~u : u | 0x80000000u) << 32 | (0xffffffffu - static_cast<uint32_t>(j));
}
__device__ __forceinline__ float lp_key_value(uint64_t k) {
  const uint32_t u = static_cast<uint32_t>(k >> 32);
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

__device__ __forceinline__ void lp_merge(float& m, float& s, float& w, float m2, float s2, float w2, float c) {
  const float M = fmaxf(m, m2);
  if (M == -INFINITY) {   // nothing but masked tokens on either side; NaN sums stay
    s += s2;
    w += w2;
    return;
  }
  const float d1 = (m - M) * c, d2 = (m2 - M) * c;
  const float f1 = ex2(d1), f2 = ex2(d2);
  // a side at -inf (or far below) has f = 0 and must not form 0 * inf
  w = f1 * (w + (f1 > 0.f ? d1 : 0.f) * s) + f2 * (w2 + (f2 > 0.f ? d2 : 0.f) * s2);
  s = s * f1 + s2 * f2;
  m = M;
}

// The 16-byte vectors of a row's hull that a thread holds: elements outside
// the row read as -inf, and only vectors wholly inside it are read as vectors.
template <int ES>
__device__ __noinline__ uint4 lp_load_edge(const uint8_t* p, const uint8_t* row, const uint8_t* end) {
  constexpr uint32_t kNeg = ES == 2 ? 0xff80ff80u : 0xff800000u;
  uint32_t w[4] = {kNeg, kNeg, kNeg, kNeg};
#pragma unroll
  for (int e = 0; e < 16 / ES; ++e) {
    const uint8_t* q = p + e * ES;
    if (q < row || q >= end) continue;
    if (ES == 4) {
      w[e & 3] = *reinterpret_cast<const uint32_t*>(q);
    } else {
      const uint32_t h = *reinterpret_cast<const uint16_t*>(q);
      w[e >> 1] = e & 1 ? (w[e >> 1] & 0xffffu) | h << 16 : (w[e >> 1] & 0xffff0000u) | h;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A thread's vectors of a segment (per of them for the CTA): without tests
// where the segment lies inside the row. Else what is not in the row reads as
// masked; only whole vectors of it are read as vectors, and the one at each of
// its edges, which one thread has, element by element.
template <int ES, int T>
__device__ __forceinline__ void lp_load_all(uint4 (&v)[kLpVecs], const uint8_t* hull, int64_t v0, int per, const uint8_t* row,
                                            const uint8_t* end) {
  constexpr uint32_t kNeg = ES == 2 ? 0xff80ff80u : 0xff800000u;
  const uint8_t* p = hull + v0 * 16;
  const int first = hull < row;                                     // whole vectors: [first, first + whole)
  const int whole = static_cast<int>((end - hull) / 16) - first;
  const int s0 = static_cast<int>(v0) - static_cast<int>(threadIdx.x);
  if (s0 >= first && s0 + per <= first + whole) {
#pragma unroll
    for (int i = 0; i < kLpVecs; ++i) {
      v[i] = make_uint4(kNeg, kNeg, kNeg, kNeg);
      if (i * T < per) v[i] = *reinterpret_cast<const uint4*>(p + i * T * 16);
    }
    return;
  }
  const int at = static_cast<int>(v0) - first;
#pragma unroll
  for (int i = 0; i < kLpVecs; ++i) {
    v[i] = make_uint4(kNeg, kNeg, kNeg, kNeg);
    if (i * T < per && static_cast<unsigned>(at + i * T) < static_cast<unsigned>(max(whole, 0)))
      v[i] = *reinterpret_cast<const uint4*>(p + i * T * 16);
  }
  // the vector before the whole ones, and the one after them (the same, where there are none)
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    const int vec = k == 0 ? first - 1 : first + max(whole, 0);
    const int d = vec - static_cast<int>(v0);
    if (vec < 0 || d < 0 || d % T != 0 || d >= per || hull + vec * 16ll >= end) continue;
    const uint4 e = lp_load_edge<ES>(hull + vec * 16ll, row, end);
#pragma unroll
    for (int i = 0; i < kLpVecs; ++i)
      if (d == i * T) v[i] = e;
  }
}

// max that hands on NaN.
__device__ __forceinline__ float lp_max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ uint32_t lp_max_nan2(uint32_t a, uint32_t b) {   // bf16x2
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A value of the type at which 2^((x - m) c) is 0, below m.
template <int ES>
__device__ __forceinline__ float lp_floor(float m, float c) {
  // the value of the type next below m
  const uint32_t one = ES == 2 ? 0x10000u : 1u;
  const uint32_t b = __float_as_uint(m);
  const float below = __uint_as_float(m > 0.f ? b - one : m < 0.f ? b + one : 0x80000000u + one);
  const float far = m + kLpFloor / c;
  // bf16: cut off to the type's bits, which for a negative number moves it up by less than it lies below
  return fminf(below, ES == 2 ? __uint_as_float(__float_as_uint(far) & 0xffff0000u) : far);
}

// Sum of t 2^t over a vector, with t no less than -300.
template <int ES>
__device__ __noinline__ float lp_weighted(uint4 v, float m, float c) {
  float f[16 / ES], w = 0.f;
  Elem<ES>::unpack(v, f);
#pragma unroll
  for (int e = 0; e < 16 / ES; ++e) {
    const float t = lp_max_nan((f[e] - m) * c, kLpFloor);
    w = fmaf(ex2(t), t, w);
  }
  return w;
}

// The largest element of a vector (NaN ignored).
template <int ES>
__device__ __forceinline__ float lp_vec_max(const uint4& v) {
  if (ES == 4)
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  auto max2 = [](uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  };
  const uint32_t m = max2(max2(v.x, v.y), max2(v.z, v.w));
  return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
}

// The largest key of a vector below `last`, or `best` if that is larger.
template <int ES>
__device__ __noinline__ uint64_t lp_best_below(uint4 v, int j, uint64_t last, uint64_t best) {
  float f[16 / ES];
  Elem<ES>::unpack(v, f);
#pragma unroll
  for (int e = 0; e < 16 / ES; ++e) {
    const uint64_t k = lp_key(f[e], j + e);
    if (k < last && k > best) best = k;
  }
  return best;
}

template <int ES, bool TOP>
__global__ void __launch_bounds__(TOP ? kLpTopThreads : kLpThreads, TOP ? 4 : 8) token_logprobs_kernel(const LogprobArgs a) {
  constexpr int kE = 16 / ES;
  constexpr int T = TOP ? kLpTopThreads : kLpThreads;
  __shared__ __align__(16) float s_group[kLpGroups];
  __shared__ float s_bound;
  __shared__ uint32_t s_hits, s_count;
  __shared__ uint4 s_hit[TOP ? kLpHits : 1];
  __shared__ int32_t s_hit_at[TOP ? kLpHits : 1];
  __shared__ uint64_t s_cand[TOP ? kLpCand : 1];
  __shared__ uint64_t s_best[2][T / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  struct {
    int row, seg, j0;   // j0: row index of the thread's first element
  } x;
  x.row = blockIdx.x / a.segs;
  x.seg = blockIdx.x - x.row * a.segs;
  grid_dep_wait();
  grid_dep_launch();
  uint4 v[kLpVecs];
  {
    const uint8_t* rp = a.x + x.row * a.stride;
    const uint8_t* hull = reinterpret_cast<const uint8_t*>(reinterpret_cast<uintptr_t>(rp) & ~static_cast<uintptr_t>(15));
    const int64_t v0 = static_cast<int64_t>(x.seg) * a.per + tid;
    x.j0 = static_cast<int>((hull - rp) / ES + v0 * kE);
    lp_load_all<ES, T>(v, hull, v0, a.per, rp, rp + static_cast<int64_t>(a.V) * ES);
  }
  const int its = a.per / T;
  {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kLpVecs; ++i) m = fmaxf(m, lp_vec_max<ES>(v[i]));
    if (TOP) {
      float gm = m;
#pragma unroll
      for (int o = 1; o < kLpGroup; o <<= 1) gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, o));
      if (lane % kLpGroup == 0) s_group[tid / kLpGroup] = gm;
      if (tid == 0) s_hits = s_count = 0;
    }
    const float m0 = m == -INFINITY ? 0.f : m;
    // Masked tokens are lifted to where 2^t is 0 but t is finite (0 * -inf is no 0):
    // 300 below the maximum, or the value just below it where that rounds to it.
    float2 s2 = make_float2(0.f, 0.f), w2 = make_float2(0.f, 0.f);
    const float2 m2 = make_float2(-m0, -m0), c2 = make_float2(a.c, a.c);
    const float floor1 = lp_floor<ES>(m0, a.c);
    const uint32_t floor2 = __byte_perm(__float_as_uint(floor1), 0, 0x3232);
#pragma unroll
    for (int i = 0; i < kLpVecs; ++i) {
      if (i >= its) break;
      uint4 q = v[i];
      if (ES == 2) {
        q.x = lp_max_nan2(q.x, floor2);
        q.y = lp_max_nan2(q.y, floor2);
        q.z = lp_max_nan2(q.z, floor2);
        q.w = lp_max_nan2(q.w, floor2);
      }
      float f[kE];
      Elem<ES>::unpack(q, f);
#pragma unroll
      for (int e = 0; e < kE; e += 2) {
        if (ES == 4) {
          f[e] = lp_max_nan(f[e], floor1);
          f[e + 1] = lp_max_nan(f[e + 1], floor1);
        }
        const float2 t = __fmul2_rn(__fadd2_rn(make_float2(f[e], f[e + 1]), m2), c2);
        const float2 p = make_float2(ex2(t.x), ex2(t.y));
        s2 = __fadd2_rn(s2, p);
        w2 = __ffma2_rn(p, t, w2);
      }
    }
    // the warp's sums, relative to its maximum
    const float mr = warp_max(m);
    float s = s2.x + s2.y, w = w2.x + w2.y;
    if (w != w && s == s) {   // the maximum is the type's lowest value: nothing lies below it to lift -inf to
      w = 0.f;
#pragma unroll
      for (int i = 0; i < kLpVecs; ++i)
        if (i < its) w += lp_weighted<ES>(v[i], m0, a.c);
    }
    const float d = m == -INFINITY ? -INFINITY : (m - mr) * a.c, f = ex2(d);
    w = f > 0.f ? f * (w + d * s) : s == s ? 0.f : s;
    s *= f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      w += __shfl_xor_sync(0xffffffffu, w, o);
    }
    // A partial a warp: without the top alternatives no warp of a CTA waits for another.
    if (lane == 0) a.part[(static_cast<int64_t>(x.row) * a.segs + x.seg) * (T / 32) + warp] = {mr, s, w, 0.f};
    if (TOP) {
      __syncthreads();
      // ---- the n_top-th of the group maxima: a group's threads rank its own
      {
        const int i = tid / kLpGroup;
        const float gm = s_group[i];
        int r = 0;
#pragma unroll
        for (int q = 0; q < kLpGroups / kLpGroup / 4; ++q) {
          const int j = (tid % kLpGroup + q * kLpGroup) * 4;
          const float4 o = *reinterpret_cast<const float4*>(s_group + j);
          // equal maxima rank by their index
          r += (j < i ? o.x >= gm : o.x > gm) + (j + 1 < i ? o.y >= gm : o.y > gm) + (j + 2 < i ? o.z >= gm : o.z > gm) +
               (j + 3 < i ? o.w >= gm : o.w > gm);
        }
#pragma unroll
        for (int o = 1; o < kLpGroup; o <<= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
        if (r == a.n_top - 1) s_bound = gm;
      }
      __syncthreads();
      // ---- vectors that hold one that reaches it, then their elements, a thread each
      const float bound = s_bound;
      if (m >= bound && m > -INFINITY) {
#pragma unroll
        for (int i = 0; i < kLpVecs; ++i)
          if (lp_vec_max<ES>(v[i]) >= bound) {
            const uint32_t at = atomicAdd(&s_hits, 1u);
            if (at < kLpHits) {
              s_hit[at] = v[i];
              s_hit_at[at] = x.j0 + i * T * kE;
            }
          }
      }
      __syncthreads();
      const uint32_t hits = s_hits;
#pragma unroll 1
      for (uint32_t i = tid; i < min(hits, kLpHits) * kE; i += T) {
        const uint32_t e = i % kE;
        const float f = ES == 2 ? __uint_as_float(reinterpret_cast<const uint16_t*>(s_hit)[i] << 16)
                                : reinterpret_cast<const float*>(s_hit)[i];
        if (f >= bound && f > -INFINITY) {
          const uint32_t at = atomicAdd(&s_count, 1u);
          if (at < kLpCand) s_cand[at] = lp_key(f, s_hit_at[i / kE] + e);
        }
      }
      __syncthreads();
      const uint32_t n = s_count;
      uint64_t* out = a.cand + (static_cast<int64_t>(x.row) * a.segs + x.seg) * a.n_top;
      if (hits <= kLpHits && n <= kLpCand) {
        // ranks by counting, eight lanes a candidate
#pragma unroll 1
        for (uint32_t i0 = 0; i0 < n; i0 += T / 8) {
          const uint32_t i = i0 + (tid >> 3);
          const uint64_t k = i < n ? s_cand[i] : 0;
          int r = 0;
          for (uint32_t j = tid & 7; j < n; j += 8) r += s_cand[j] > k;
          r += __shfl_xor_sync(0xffffffffu, r, 1);
          r += __shfl_xor_sync(0xffffffffu, r, 2);
          r += __shfl_xor_sync(0xffffffffu, r, 4);
          if (i < n && r < a.n_top && (tid & 7) == 0) out[r] = k;
        }
        if (static_cast<uint32_t>(tid) >= n && tid < a.n_top) out[tid] = 0;
      } else {
        // n_top times the CTA's largest; the thread that had it looks for its next
        uint64_t mine = 0;
#pragma unroll
        for (int i = 0; i < kLpVecs; ++i) mine = lp_best_below<ES>(v[i], x.j0 + i * T * kE, ~0ull, mine);
#pragma unroll 1
        for (int r = 0; r < a.n_top; ++r) {
          const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(mine >> 32));
          const uint32_t lo = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(mine >> 32) == hi ? static_cast<uint32_t>(mine) : 0u);
          if (lane == 0) s_best[r & 1][warp] = static_cast<uint64_t>(hi) << 32 | lo;
          __syncthreads();
          uint64_t best = 0;
#pragma unroll
          for (int i = 0; i < T / 32; ++i) best = s_best[r & 1][i] > best ? s_best[r & 1][i] : best;
          if (tid == 0) out[r] = best;
          if (best != 0 && mine == best) {
            mine = 0;
#pragma unroll
            for (int i = 0; i < kLpVecs; ++i) mine = lp_best_below<ES>(v[i], x.j0 + i * T * kE, best, mine);
          }
        }
      }
    }
  }
}

// One warp per row: joins the segments' sums and sorted lists, which it holds
// in shared memory where they fit (each of the n_top steps needs the head of
// one list, and that is a load on the way of the next step).
constexpr int kLpJoinWarps = 4;
constexpr int kLpJoinKeys = 1024;

template <int ES>
__global__ void __launch_bounds__(kLpJoinWarps * 32) token_logprobs_join_kernel(const LogprobArgs a) {
  __shared__ uint64_t s_keys[kLpJoinWarps][kLpJoinKeys];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x * kLpJoinWarps + warp;
  if (row >= a.rows) {
    grid_dep_wait();
    grid_dep_launch();
    return;
  }
  // The call's own inputs were complete before the first kernel began.
  const int tok = a.tokens[row];
  const bool given = tok >= 0 && tok < a.V;
  const float xt = given ? Elem<ES>::load(a.x + row * a.stride, tok) : 0.f;
  grid_dep_wait();
  grid_dep_launch();
  const int parts = a.segs * ((a.n_top ? kLpTopThreads : kLpThreads) / 32);
  const LpPartial* part = a.part + static_cast<int64_t>(row) * parts;
  const uint64_t* lists = a.cand + static_cast<int64_t>(row) * a.segs * a.n_top;
  const int keys = a.segs * a.n_top;
  const bool held = keys <= kLpJoinKeys;
  if (held) {
#pragma unroll 4
    for (int i = lane; i < keys; i += 32) s_keys[warp][i] = lists[i];
    lists = s_keys[warp];
  }
  float m = -INFINITY, s = 0.f, w = 0.f;
#pragma unroll 1
  for (int i = lane; i < parts; i += 32) {
    const LpPartial p = part[i];
    lp_merge(m, s, w, p.m, p.s, p.w, a.c);
  }
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1)
    lp_merge(m, s, w, __shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, s, o),
             __shfl_xor_sync(0xffffffffu, w, o), a.c);
  const bool empty = m == -INFINITY && s == s;   // every token masked
  const float l2 = empty ? -INFINITY : log2f(s);
  const float ref = empty ? 0.f : m;
  const float ent = empty ? 0.f : fmaxf((l2 - w / s) * kLn2, 0.f);
  const float nan = __int_as_float(0x7fc00000);
  const bool bad = !(s < INFINITY) || !(fabsf(ref) < INFINITY);   // NaN or +inf somewhere
  auto logp = [&](float x) {
    return bad ? nan : x == -INFINITY || empty ? -INFINITY : (x - ref) * a.inv_t - l2 * kLn2;
  };
  if (lane == 0) {
    a.logprob[row] = given ? logp(xt) : 0.f;
    if (a.entropy) a.entropy[row] = bad ? nan : ent;
    if (a.lse) a.lse[row] = bad ? nan : ref * a.inv_t + l2 * kLn2;
    if (a.saved) a.saved[row] = make_float4(bad ? nan : ref, l2, ent, 0.f);
    if (a.status)
      a.status[row] = (tok >= a.V || tok < -1 ? SV_STATUS_BAD_TOKEN : 0) | (bad || empty ? SV_STATUS_NONFINITE_ROW : 0);
  }
  if (a.n_top == 0) return;
  __syncwarp();
  // heads of the sorted lists, list i with lane i % 32; `at` counts what is taken of the lane's own list
  uint64_t last = ~0ull;
  uint64_t head = lane < a.segs ? lists[lane * a.n_top] : 0;
  uint64_t mine = 0;   // the lane's answer: the lane-th largest
  int at = 0;
#pragma unroll 1
  for (int r = 0; r < a.n_top; ++r) {
    uint64_t best = head;
    if (a.segs > 32)   // more lists than lanes: the largest below the last one taken
      for (int i = lane + 32; i < a.segs; i += 32)
        for (int k = 0; k < a.n_top; ++k) {
          const uint64_t e = lists[static_cast<int64_t>(i) * a.n_top + k];
          if (e < last) {
            best = e > best ? e : best;
            break;
          }
        }
    const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(best >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(best >> 32) == hi ? static_cast<uint32_t>(best) : 0u);
    const uint64_t top = static_cast<uint64_t>(hi) << 32 | lo;
    if (top != 0 && head == top) {
      ++at;
      head = at < a.n_top ? lists[lane * a.n_top + at] : 0;
    }
    last = top;
    if (lane == r) mine = top;
  }
  if (lane < a.n_top) {
    a.top_tokens[static_cast<int64_t>(row) * a.n_top + lane] = mine ? static_cast<int32_t>(~static_cast<uint32_t>(mine)) : -1;
    a.top_logprobs[static_cast<int64_t>(row) * a.n_top + lane] = bad ? nan : mine ? logp(lp_key_value(mine)) : -INFINITY;
  }
}

struct LogprobGradArgs {
  const uint8_t* x;
  int64_t stride;              // bytes between rows of x
  uint8_t* dx;
  int64_t dstride;             // bytes between rows of dx
  const int32_t* tokens;       // [rows]
  const float4* saved;         // [rows]
  const float* g;              // [rows]
  const float* h;              // [rows] or nullptr
  int32_t rows, V, segs, per;
  float c, inv_t;
};

// The elements of a vector that lie in the row.
template <int ES>
__device__ __noinline__ void lp_store_edge(uint8_t* dp, int64_t j, int V, uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 16 / ES; ++e) {
    if (j + e < 0 || j + e >= V) continue;
    if (ES == 4)
      reinterpret_cast<uint32_t*>(dp)[j + e] = w[e & 3];
    else
      reinterpret_cast<uint16_t*>(dp)[j + e] = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
  }
}

// Eight 16-byte vectors a thread, as in the forward pass, if x and dx rows
// start at the same place within 16 bytes; else one element at a time.
template <int ES, bool VEC>
__global__ void __launch_bounds__(kLpThreads, 8) token_logprobs_grad_kernel(const LogprobGradArgs a) {
  constexpr int kE = 16 / ES;
  const int tid = threadIdx.x;
  const int row = blockIdx.x / a.segs, seg = blockIdx.x - row * a.segs;
  grid_dep_wait();
  grid_dep_launch();
  const uint8_t* rp = a.x + row * a.stride;
  uint8_t* dp = a.dx + row * a.dstride;
  const uint8_t* end = rp + static_cast<int64_t>(a.V) * ES;
  const uint8_t* hull = reinterpret_cast<const uint8_t*>(reinterpret_cast<uintptr_t>(rp) & ~static_cast<uintptr_t>(15));
  const int64_t v0 = static_cast<int64_t>(seg) * a.per + tid;
  uint4 v[kLpVecs];
  if (VEC) lp_load_all<ES, kLpThreads>(v, hull, v0, a.per, rp, end);
  const int tok = a.tokens[row];
  const float4 st = a.saved[row];
  const bool empty = st.y == -INFINITY;   // no token left: no gradient
  const float g = tok >= 0 && tok < a.V && !empty ? a.g[row] * a.inv_t : 0.f;
  const float h = a.h && !empty ? a.h[row] * a.inv_t : 0.f;
  const float ref = st.x, l2 = empty ? 0.f : st.y;
  const float a0 = -(g + h * st.z), a1 = -h * kLn2;
  auto grad = [&](float x, int64_t j) {
    const float t = lp_max_nan(fmaf(x - ref, a.c, -l2), kLpFloor);
    const float d = ex2(t) * fmaf(a1, t, a0);
    return j == tok ? d + g : d;
  };
  if (!VEC) {
    for (int64_t j = static_cast<int64_t>(seg) * a.per * kE + tid; j < a.V && j < (seg + 1) * static_cast<int64_t>(a.per) * kE;
         j += kLpThreads) {
      const float d = grad(Elem<ES>::load(rp, static_cast<int>(j)), j);
      if (ES == 4)
        reinterpret_cast<float*>(dp)[j] = d;
      else
        reinterpret_cast<__nv_bfloat16*>(dp)[j] = __float2bfloat16_rn(d);
    }
    return;
  }
  const int64_t j0 = (hull - rp) / ES + v0 * kE;
#pragma unroll
  for (int i = 0; i < kLpVecs; ++i) {
    const uint8_t* p = hull + (v0 + i * kLpThreads) * 16;
    if (i * kLpThreads >= a.per || p >= end) continue;
    float f[kE];
    Elem<ES>::unpack(v[i], f);
    const int64_t j = j0 + i * kLpThreads * kE;
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const float t = lp_max_nan(fmaf(f[e] - ref, a.c, -l2), kLpFloor);
      f[e] = ex2(t) * fmaf(a1, t, a0);
    }
    if (tok >= j && tok < j + kE) {
#pragma unroll
      for (int e = 0; e < kE; ++e) f[e] += tok == j + e ? g : 0.f;
    }
    uint4 o;
    if (ES == 4) {
      o = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    } else {
      uint32_t q[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(q[e]) : "f"(f[(2 * e) % kE]), "f"(f[(2 * e + 1) % kE]));
      o = make_uint4(q[0], q[1], q[2], q[3]);
    }
    if (p >= rp && p + 16 <= end)
      *reinterpret_cast<uint4*>(dp + j * ES) = o;
    else
      lp_store_edge<ES>(dp, j, a.V, o);
  }
}

}  // namespace sv
