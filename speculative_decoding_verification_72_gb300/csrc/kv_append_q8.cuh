// Writing new key / value rows into the 8-bit paged cache.
//
// Row i of request b (its new row i, or row path_nodes[b, i] of the verify
// pass) becomes position base_b + i. Per page and head touched, K and V apart:
//   need  = smallest power of two s with max |x| <= 448 s over the new rows
//   scale = max(need, old scale) if the page keeps positions below base, else need
//   kept codes are rescaled by old / scale (only if it grew), new codes are x / scale.
// A page that starts at or after base holds nothing yet, so its old scale and
// codes do not count. Infinities saturate and NaN stays NaN; neither counts in
// the maximum.
//
// Bound by memory: each row is read once and its codes written once. A CTA
// holds the rows of up to four passes of its threads (128 rows of 128) in
// registers, as read, between the maximum and the rounding:
// several small pages, each with a maximum of its own. All loads that need only
// base go out before the barrier that carries the maxima; what few rows need
// (rescaling, a scale that is no power of two, infinities) is out of line.
// Sixteen elements a thread, for fewer instructions around them (3 prompts of 4099
// bf16 tokens, 8 heads of 128: 16.9 us, 4.5 TB/s; eight elements a thread 19.9).
// What is left is mostly waiting for the rows (an instruction issues in 0.64 of
// the clocks): a CTA has one tile, and no loads under way behind it.
#pragma once

#include "q8_common.cuh"

namespace sv {

constexpr int kAppendThreads = 256;

struct AppendArgs {
  const uint8_t* x[2];       // new K, new V
  int64_t sb[2], sn[2], sh[2];   // strides in bytes: request, row, head
  Q8View c;
  const int32_t* base;       // [B]
  const int32_t* path;       // [B, path_cols] or nullptr (row i is new row i)
  const int32_t* num_acc;    // [B] or nullptr (all N rows)
  int32_t path_cols, B, N, W;   // W: tiles of a CTA that N rows can touch
  int32_t* out_len;          // [B]
  int32_t* status;           // [B] or nullptr
};

// Sixteen elements as read: their absolute values order like the integers of
// their bits, so the maximum is taken on those, two of 16 bits at a time.
constexpr int kAppendEls = 16;
template <typename T>
struct AppendRaw {
  static constexpr int kVecs = T::kBytes;
  uint4 v[kVecs];
  __device__ __forceinline__ void load(const uint8_t* p) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void unpack(float* f) const {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      if constexpr (kVecs == 4)
        Elem<4>::unpack(v[i], f + 4 * i);
      else
        T::unpack8(v[i], f + 8 * i);
    }
  }
  // The bits of the largest magnitude as fp32, at least infinity's if an element is not finite.
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (kVecs == 4)
          m = max(m, w[j] & 0x7fffffffu);
        else
          m = T::max2(m, w[j] & 0x7fff7fffu);
      }
    }
    if constexpr (kVecs == 4)
      return m;
    else
      return __float_as_uint(T::value(static_cast<uint16_t>(max(m & 0xffffu, m >> 16))));
  }
};

__device__ __forceinline__ uint4 append_codes(const float* f) {
  return make_uint4(e4m3_pack4(f[0], f[1], f[2], f[3]), e4m3_pack4(f[4], f[5], f[6], f[7]),
                    e4m3_pack4(f[8], f[9], f[10], f[11]), e4m3_pack4(f[12], f[13], f[14], f[15]));
}

// Largest magnitude of the finite elements. Out of line: few rows hold others.
template <typename T>
__device__ __noinline__ float append_finite_max(AppendRaw<T> x, float m) {
  float f[kAppendEls];
  x.unpack(f);
#pragma unroll
  for (int e = 0; e < kAppendEls; ++e) m = fmaxf(m, fabsf(f[e]) < INFINITY ? fabsf(f[e]) : 0.f);
  return m;
}

// Codes by division. Out of line, like the next: the caches this framework
// writes have scales of powers of two, whose inverse is exact.
template <typename T>
__device__ __noinline__ uint4 append_divide(AppendRaw<T> x, float scale) {
  float f[kAppendEls];
  x.unpack(f);
#pragma unroll
  for (int e = 0; e < kAppendEls; ++e) f[e] /= scale;
  return append_codes(f);
}

__device__ __noinline__ uint4 append_rescale(uint4 w, float old, float scale) {
  const float g = old / scale;
  return make_uint4(e4m3_rescale4(w.x, g), e4m3_rescale4(w.y, g), e4m3_rescale4(w.z, g), e4m3_rescale4(w.w, g));
}

// CTAs of an SM: as many as the rows held in registers leave room for.
template <typename T, int NP>
constexpr int kAppendCtas = NP * T::kBytes <= 4 ? 5 : NP * T::kBytes == 8 ? 4 : 2;

template <typename T, int D, int NP>
__global__ void __launch_bounds__(kAppendThreads, kAppendCtas<T, NP>) kv_append_q8_kernel(const AppendArgs a) {
  constexpr int kTpr = D / kAppendEls;                    // threads per row
  constexpr int kRpp = kAppendThreads / kTpr;    // rows per pass
  constexpr int kWarps = kAppendThreads / 32;
  __shared__ uint32_t s_max[NP * kWarps];
  grid_dep_wait();
  grid_dep_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t x = blockIdx.x;
  const int tile = x % static_cast<uint32_t>(a.W);
  x /= static_cast<uint32_t>(a.W);
  const int h = x % static_cast<uint32_t>(a.c.Hkv);
  x /= static_cast<uint32_t>(a.c.Hkv);
  const int kv = x & 1, b = x >> 1;
  const int shift = a.c.page_shift, P = 1 << shift;
  const int32_t base = a.base[b];
  const int64_t count = a.num_acc ? static_cast<int64_t>(a.num_acc[b]) + 1 : a.N;
  bool ok = base >= 0 && count >= 0 && count <= (a.path ? min(a.path_cols, a.N) : a.N) &&
            base + count <= static_cast<int64_t>(a.c.max_pages) << shift;
  const int n = ok ? static_cast<int>(count) : 0;
  const int first = ok ? base >> shift : 0;
  const int pages = n > 0 ? ((base + (n - 1)) >> shift) - first + 1 : 0;
  const int32_t* table = a.c.table + static_cast<int64_t>(b) * a.c.max_pages + first;
  const int32_t* path = a.path ? a.path + static_cast<int64_t>(b) * a.path_cols : nullptr;
  const int pg0 = tile * (NP * kRpp) >> shift;   // the tile's first page among the request's
  const int r0 = tid / kTpr, d0 = (tid % kTpr) * kAppendEls;
  const uint8_t* xb = a.x[kv] + b * a.sb[kv] + h * a.sh[kv] + d0 * T::kBytes;
  AppendRaw<T> raw[NP];
  bool is_new[NP];
  int32_t page[NP];
  const int i0 = ((first + pg0) << shift) + r0 - base;   // the new row of pass 0
  const uint8_t* xp = xb + i0 * a.sn[kv];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int i = i0 + p * kRpp;
    const int pg = pg0 + ((r0 + p * kRpp) >> shift);
    is_new[p] = static_cast<unsigned>(i) < static_cast<unsigned>(n);
    if (path && is_new[p]) {
      const int row = path[i];
      is_new[p] = row >= 0 && row < a.N;
      xp = xb + row * a.sn[kv];
    }
    if (is_new[p]) raw[p].load(xp);
    xp += kRpp * a.sn[kv];
    page[p] = pg < pages ? table[pg] : -1;
  }
  // Every CTA of a request validates all of it, so a bad request is left
  // untouched by all of them.
  for (int j = tid; j < pages; j += kAppendThreads) ok = ok && table[j] >= 0 && table[j] < a.c.num_pages;
  if (path)
    for (int j = tid; j < n; j += kAppendThreads) ok = ok && path[j] >= 0 && path[j] < a.N;
  float* scales = kv ? a.c.vs : a.c.ks;
  // only the first page keeps rows below base
  const int kept = pg0 == 0 ? base & (P - 1) : 0;
  const int32_t page0 = pg0 < pages ? table[pg0] : -1;
  const float old0 = kept > 0 && page0 >= 0 && page0 < a.c.num_pages ? scales[page0 * static_cast<uint32_t>(a.c.Hkv) + h] : 0.f;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    uint32_t m = is_new[p] ? raw[p].amax() : 0u;
    m = __reduce_max_sync(0xffffffffu, m);
    if (m >= 0x7f800000u)
      m = __reduce_max_sync(0xffffffffu, is_new[p] ? __float_as_uint(append_finite_max<T>(raw[p], 0.f)) : 0u);
    if (lane == 0) s_max[p * kWarps + warp] = m;
  }
  ok = __syncthreads_and(ok);
  if (tile == 0 && h == 0 && kv == 0 && tid == 0) {
    a.out_len[b] = ok ? base + n : base;
    if (a.status) a.status[b] = ok ? 0 : SV_STATUS_BAD_PAGE;
  }
  if (!ok || pg0 >= pages) return;
  // The maxima of pages, a lane an entry: 32 / kTpr rows of a page.
  static_assert(NP * kWarps <= 32, "a lane an entry");
  const int entries = P * kTpr / 32;   // of a page
  uint32_t m = lane < NP * kWarps ? s_max[lane] : 0u;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
    if (o < entries) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  const int need = q8_need_exp(__uint_as_float(m));
  float page_scale = exp2_int(need), page_inv = exp2_int(-need);
  if (lane < entries && old0 > page_scale) {   // of page pg0; old0 is 0 unless that keeps rows
    page_scale = old0;
    // A scale from elsewhere may be no power of two: its quotients are divisions.
    page_inv = (__float_as_uint(old0) & 0x7fffffu) == 0 ? 1.f / old0 : 0.f;
  }
  uint8_t* codes = kv ? a.c.v : a.c.k;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int r = (r0 + p * kRpp) & (P - 1);
    const int pg = pg0 + ((r0 + p * kRpp) >> shift);
    const int entry = p * kWarps + warp;
    const float scale = __shfl_sync(0xffffffffu, page_scale, entry), inv = __shfl_sync(0xffffffffu, page_inv, entry);
    if (pg >= pages) continue;
    const float old = pg == 0 ? old0 : 0.f;
    const uint32_t own = static_cast<uint32_t>(page[p]) * a.c.Hkv + h;
    uint4* dst = reinterpret_cast<uint4*>(codes + (static_cast<int64_t>(own) * (P * D) + (r * D + d0)));
    if (is_new[p]) {
      if (inv != 0.f) {
        float f[kAppendEls];
        raw[p].unpack(f);
#pragma unroll
        for (int e = 0; e < kAppendEls; ++e) f[e] *= inv;
        *dst = append_codes(f);
      } else {
        *dst = append_divide<T>(raw[p], scale);
      }
    } else if (pg == 0 && r < kept && scale != old) {
      *dst = append_rescale(*dst, old, scale);
    }
    if (r == 0 && d0 == 0 && scale != old) scales[own] = scale;
  }
}

}  // namespace sv
