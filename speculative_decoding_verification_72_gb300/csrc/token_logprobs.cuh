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
// Bound by memory: the forward pass reads each row once (the row is cut into
// 32 KB segments, one CTA each; a thread keeps its eight 16-byte vectors in
// registers, so maximum, sums and selection are passes over registers), the
// gradient reads and writes it once.
//
// Top alternatives by (logit, lower index): a bound that at least n_top
// elements of the segment reach is the n_top-th of the 32 maxima of groups of
// eight threads; the few elements that reach it are gathered and ranked. If
// they overflow the buffer (many equal logits) the segment takes n_top rounds
// of block-wide maxima instead. Masked (-inf) tokens are no alternatives.
#pragma once

#include <cuda_bf16.h>

#include "sv_common.cuh"

namespace sv {

constexpr int kLpThreads = 256;
constexpr int kLpVecs = 8;                                   // 16-byte vectors per thread
constexpr int kLpSegVecs = kLpThreads * kLpVecs;             // 32 KB
constexpr int kLpMaxTop = SV_MAX_TOP_ALTERNATIVES;
constexpr int kLpCand = 512;
constexpr float kLpFloor = -300.f;                           // 2^-300 is 0 in fp32

struct __align__(16) LpPartial {
  float m, s, w, pad;
};

struct LogprobArgs {
  const uint8_t* x;
  int64_t stride;              // bytes between rows
  const int32_t* tokens;       // [rows]
  int32_t rows, V, segs, n_top;
  float c, inv_t;              // log2(e) / T, 1 / T
  LpPartial* part;             // [rows, segs]
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
__device__ __forceinline__ uint4 lp_load(const uint8_t* hull, int64_t vec, const uint8_t* row, const uint8_t* end) {
  const uint8_t* p = hull + vec * 16;
  constexpr uint32_t kNeg = ES == 2 ? 0xff80ff80u : 0xff800000u;
  if (p >= row && p + 16 <= end) return *reinterpret_cast<const uint4*>(p);
  uint4 v = make_uint4(kNeg, kNeg, kNeg, kNeg);
  if (p >= end) return v;
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

template <int ES, bool TOP>
__global__ void __launch_bounds__(kLpThreads, 4) token_logprobs_kernel(const LogprobArgs a) {
  constexpr int kE = 16 / ES;
  __shared__ LpPartial s_part[kLpThreads / 32];
  __shared__ float s_group[32];
  __shared__ uint32_t s_count;
  __shared__ uint64_t s_cand[TOP ? kLpCand : 1];
  __shared__ uint64_t s_best[kLpThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / a.segs, seg = blockIdx.x - row * a.segs;
  if (tid == 0) s_count = 0;
  grid_dep_wait();
  grid_dep_launch();
  const uint8_t* rp = a.x + row * a.stride;
  const uint8_t* end = rp + static_cast<int64_t>(a.V) * ES;
  const uint8_t* hull = reinterpret_cast<const uint8_t*>(reinterpret_cast<uintptr_t>(rp) & ~static_cast<uintptr_t>(15));
  const int64_t v0 = static_cast<int64_t>(seg) * kLpSegVecs + tid;
  uint4 v[kLpVecs];
#pragma unroll
  for (int i = 0; i < kLpVecs; ++i) v[i] = lp_load<ES>(hull, v0 + i * kLpThreads, rp, end);

  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < kLpVecs; ++i) {
    float f[kE];
    Elem<ES>::unpack(v[i], f);
#pragma unroll
    for (int e = 0; e < kE; ++e) m = fmaxf(m, f[e]);
  }
  const float m0 = m == -INFINITY ? 0.f : m;
  float s = 0.f, w = 0.f;
#pragma unroll
  for (int i = 0; i < kLpVecs; ++i) {
    float f[kE];
    Elem<ES>::unpack(v[i], f);
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const float t0 = (f[e] - m0) * a.c;
      const float t = t0 < kLpFloor ? kLpFloor : t0;   // NaN stays
      const float p = ex2(t);
      s += p;
      w = fmaf(p, t, w);
    }
  }
  float mr = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    lp_merge(mr, s, w, __shfl_xor_sync(0xffffffffu, mr, o), __shfl_xor_sync(0xffffffffu, s, o),
             __shfl_xor_sync(0xffffffffu, w, o), a.c);
  if (lane == 0) s_part[warp] = {mr, s, w, 0.f};
  if (TOP) {
    float gm = m;
    gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, 1));
    gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, 2));
    gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, 4));
    if ((lane & 7) == 0) s_group[tid >> 3] = gm;
  }
  __syncthreads();
  if (warp == 0) {
    LpPartial q = s_part[lane & 7];
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
      lp_merge(q.m, q.s, q.w, __shfl_xor_sync(0xffffffffu, q.m, o), __shfl_xor_sync(0xffffffffu, q.s, o),
               __shfl_xor_sync(0xffffffffu, q.w, o), a.c);
    if (lane == 0) a.part[static_cast<int64_t>(row) * a.segs + seg] = q;
  }
  if (!TOP) return;
  // ---- the n_top-th of the 32 group maxima (every warp works it out)
  const float gm = s_group[lane];
  int rank = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const float o = __shfl_sync(0xffffffffu, gm, i);
    rank += o > gm || (o == gm && i < lane);
  }
  const unsigned who = __ballot_sync(0xffffffffu, rank == a.n_top - 1);
  const float bound = __shfl_sync(0xffffffffu, gm, __ffs(who) - 1);
  const int64_t j0 = (hull - rp) / ES;   // row index of the hull's first element (<= 0)
  if (m >= bound && m > -INFINITY) {
#pragma unroll
    for (int i = 0; i < kLpVecs; ++i) {
      float f[kE];
      Elem<ES>::unpack(v[i], f);
#pragma unroll
      for (int e = 0; e < kE; ++e)
        if (f[e] >= bound && f[e] > -INFINITY) {
          const uint32_t at = atomicAdd(&s_count, 1u);
          if (at < kLpCand) s_cand[at] = lp_key(f[e], static_cast<int>(j0 + (v0 + i * kLpThreads) * kE + e));
        }
    }
  }
  __syncthreads();
  const uint32_t n = s_count;
  uint64_t* out = a.cand + (static_cast<int64_t>(row) * a.segs + seg) * a.n_top;
  if (n <= kLpCand) {
    for (uint32_t i = tid; i < n; i += kLpThreads) {
      const uint64_t k = s_cand[i];
      int r = 0;
      for (uint32_t j = 0; j < n; ++j) r += s_cand[j] > k;
      if (r < a.n_top) out[r] = k;
    }
    if (static_cast<uint32_t>(tid) >= n && tid < a.n_top) out[tid] = 0;
    return;
  }
  uint64_t last = ~0ull;
#pragma unroll 1
  for (int r = 0; r < a.n_top; ++r) {
    uint64_t best = 0;
#pragma unroll
    for (int i = 0; i < kLpVecs; ++i) {
      float f[kE];
      Elem<ES>::unpack(v[i], f);
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const uint64_t k = lp_key(f[e], static_cast<int>(j0 + (v0 + i * kLpThreads) * kE + e));
        if (k < last && k > best) best = k;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const uint64_t k = __shfl_xor_sync(0xffffffffu, best, o);
      best = k > best ? k : best;
    }
    __syncthreads();
    if (lane == 0) s_best[warp] = best;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kLpThreads / 32; ++i) best = s_best[i] > best ? s_best[i] : best;
    if (tid == 0) out[r] = best;
    last = best;
  }
}

// One warp per row: joins the segments' sums and sorted lists.
constexpr int kLpJoinWarps = 4;

template <int ES>
__global__ void __launch_bounds__(kLpJoinWarps * 32) token_logprobs_join_kernel(const LogprobArgs a) {
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
  const LpPartial* part = a.part + static_cast<int64_t>(row) * a.segs;
  float m = -INFINITY, s = 0.f, w = 0.f;
  for (int i = lane; i < a.segs; i += 32) {
    const LpPartial p = part[i];
    lp_merge(m, s, w, p.m, p.s, p.w, a.c);
  }
#pragma unroll
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
  }
  if (a.status) {
    const int bits = (tok >= a.V || tok < -1 ? SV_STATUS_BAD_TOKEN : 0) | (bad || empty ? SV_STATUS_NONFINITE_ROW : 0);
    if (lane == 0) a.status[row] = bits;
  }
  if (a.n_top == 0) return;
  // heads of the sorted lists, list i with lane i % 32; `at` counts what is taken of the lane's own list
  const uint64_t* lists = a.cand + static_cast<int64_t>(row) * a.segs * a.n_top;
  uint64_t last = ~0ull;
  uint64_t head = lane < a.segs ? lists[static_cast<int64_t>(lane) * a.n_top] : 0;
  int at = 0;
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
      head = at < a.n_top ? lists[static_cast<int64_t>(lane) * a.n_top + at] : 0;
    }
    last = top;
    if (lane == 0) {
      a.top_tokens[static_cast<int64_t>(row) * a.n_top + r] = top ? static_cast<int32_t>(0xffffffffu - lo) : -1;
      a.top_logprobs[static_cast<int64_t>(row) * a.n_top + r] = bad ? nan : top ? logp(lp_key_value(top)) : -INFINITY;
    }
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
  int32_t rows, V, segs;
  float c, inv_t;
};

// Eight 16-byte vectors a thread, as in the forward pass, if x and dx rows
// start at the same place within 16 bytes; else one element at a time.
template <int ES, bool VEC>
__global__ void __launch_bounds__(kLpThreads, 4) token_logprobs_grad_kernel(const LogprobGradArgs a) {
  constexpr int kE = 16 / ES;
  const int tid = threadIdx.x;
  const int row = blockIdx.x / a.segs, seg = blockIdx.x - row * a.segs;
  grid_dep_wait();
  grid_dep_launch();
  const uint8_t* rp = a.x + row * a.stride;
  uint8_t* dp = a.dx + row * a.dstride;
  const uint8_t* end = rp + static_cast<int64_t>(a.V) * ES;
  const uint8_t* hull = reinterpret_cast<const uint8_t*>(reinterpret_cast<uintptr_t>(rp) & ~static_cast<uintptr_t>(15));
  const int64_t v0 = static_cast<int64_t>(seg) * kLpSegVecs + tid;
  uint4 v[kLpVecs];
  if (VEC) {
#pragma unroll
    for (int i = 0; i < kLpVecs; ++i) v[i] = lp_load<ES>(hull, v0 + i * kLpThreads, rp, end);
  }
  const int tok = a.tokens[row];
  const float4 st = a.saved[row];
  const bool empty = st.y == -INFINITY;   // no token left: no gradient
  const float g = tok >= 0 && tok < a.V && !empty ? a.g[row] * a.inv_t : 0.f;
  const float h = a.h && !empty ? a.h[row] * a.inv_t : 0.f;
  const float ref = st.x, l2 = empty ? 0.f : st.y;
  const float a0 = -(g + h * st.z), a1 = -h * kLn2;
  auto grad = [&](float x, int64_t j) {
    const float t0 = fmaf(x - ref, a.c, -l2);
    const float t = t0 < kLpFloor ? kLpFloor : t0;
    const float d = ex2(t) * fmaf(a1, t, a0);
    return j == tok ? d + g : d;
  };
  if (!VEC) {
    for (int64_t j = static_cast<int64_t>(seg) * kLpSegVecs * kE + tid;
         j < a.V && j < (seg + 1) * static_cast<int64_t>(kLpSegVecs) * kE; j += kLpThreads) {
      const float d = grad(Elem<ES>::load(rp, static_cast<int>(j)), j);
      if (ES == 4)
        reinterpret_cast<float*>(dp)[j] = d;
      else
        reinterpret_cast<__nv_bfloat16*>(dp)[j] = __float2bfloat16_rn(d);
    }
    return;
  }
  const int64_t j0 = (hull - rp) / ES;
#pragma unroll
  for (int i = 0; i < kLpVecs; ++i) {
    const int64_t vec = v0 + i * kLpThreads;
    const uint8_t* p = hull + vec * 16;
    if (p >= end) continue;
    float f[kE];
    Elem<ES>::unpack(v[i], f);
    const int64_t j = j0 + vec * kE;
#pragma unroll
    for (int e = 0; e < kE; ++e) f[e] = grad(f[e], j + e);
    if (p >= rp && p + 16 <= end) {
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
      *reinterpret_cast<uint4*>(dp + j * ES) = o;
    } else {
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        if (j + e < 0 || j + e >= a.V) continue;
        if (ES == 4)
          reinterpret_cast<float*>(dp)[j + e] = f[e];
        else
          reinterpret_cast<__nv_bfloat16*>(dp)[j + e] = __float2bfloat16_rn(f[e]);
      }
    }
  }
}

}  // namespace sv
