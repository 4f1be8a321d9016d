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
// Bound by memory: each row is read once and its codes written once. One CTA
// per (request, K or V, head, page) holds the page's rows in registers between
// the maximum and the rounding, so nothing is read twice. All loads that need
// only base go out before the barrier that carries the maximum.
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
  int32_t path_cols, N, W;   // W: pages N rows can touch
  int32_t* out_len;          // [B]
  int32_t* status;           // [B] or nullptr
};

template <typename T, int D, int NP>
__global__ void __launch_bounds__(kAppendThreads) kv_append_q8_kernel(const AppendArgs a) {
  constexpr int kTpr = D / 8;                    // threads per row
  constexpr int kRpp = kAppendThreads / kTpr;    // rows per pass
  __shared__ float s_max[kAppendThreads / 32];
  grid_dep_wait();
  grid_dep_launch();
  const int tid = threadIdx.x;
  int x = blockIdx.x;
  const int pg = x % a.W;
  x /= a.W;
  const int h = x % a.c.Hkv;
  x /= a.c.Hkv;
  const int kv = x & 1, b = x >> 1;
  const int P = 1 << a.c.page_shift;
  const int64_t base = a.base[b];
  const int64_t count = a.num_acc ? static_cast<int64_t>(a.num_acc[b]) + 1 : a.N;
  bool ok = base >= 0 && count >= 0 && count <= (a.path ? min(a.path_cols, a.N) : a.N) &&
            base + count <= static_cast<int64_t>(a.c.max_pages) << a.c.page_shift;
  const int first = ok ? static_cast<int>(base >> a.c.page_shift) : 0;
  const int pages = ok && count > 0 ? static_cast<int>((base + count - 1) >> a.c.page_shift) - first + 1 : 0;
  // Every CTA of a request validates all of it, so a bad request is left
  // untouched by all of them.
  for (int j = tid; j < pages; j += kAppendThreads) ok = ok && q8_page(a.c, b, first + j) >= 0;
  const int32_t* path = a.path ? a.path + static_cast<int64_t>(b) * a.path_cols : nullptr;
  if (path && ok)
    for (int64_t j = tid; j < count; j += kAppendThreads) ok = ok && path[j] >= 0 && path[j] < a.N;

  const int page = pg < pages ? q8_page(a.c, b, first + pg) : -1;
  const int64_t start = static_cast<int64_t>(first + pg) << a.c.page_shift;
  const int kept = page < 0 || base <= start ? 0 : static_cast<int>(base - start);
  uint8_t* codes = (kv ? a.c.v : a.c.k) + ((static_cast<int64_t>(max(page, 0)) * a.c.Hkv + h) << a.c.page_shift) * D;
  float* scale_p = (kv ? a.c.vs : a.c.ks) + static_cast<int64_t>(max(page, 0)) * a.c.Hkv + h;
  const uint8_t* xb = a.x[kv] + b * a.sb[kv] + h * a.sh[kv];
  const int r0 = tid / kTpr, d0 = (tid % kTpr) * 8;
  float f[NP][8];
  bool is_new[NP];
  float m = 0.f;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int r = r0 + p * kRpp;
    const int64_t i = start + r - base;
    is_new[p] = page >= 0 && r < P && i >= 0 && i < count;
    int64_t row = i;
    if (is_new[p] && path) {
      row = path[i];
      is_new[p] = row >= 0 && row < a.N;
    }
    if (is_new[p]) T::load8(xb + row * a.sn[kv] + d0 * T::kBytes, f[p]);
  }
  const float old = kept > 0 ? *scale_p : 0.f;
#pragma unroll
  for (int p = 0; p < NP; ++p)
    if (is_new[p]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = fabsf(f[p][e]);
        m = fmaxf(m, v < INFINITY ? v : 0.f);
      }
    }
  m = warp_max(m);
  if (tid % 32 == 0) s_max[tid / 32] = m;
  ok = __syncthreads_and(ok);
  if (pg == 0 && h == 0 && kv == 0 && tid == 0) {
    a.out_len[b] = static_cast<int32_t>(ok ? base + count : base);
    if (a.status) a.status[b] = ok ? 0 : SV_STATUS_BAD_PAGE;
  }
  if (!ok || page < 0) return;
#pragma unroll
  for (int w = 0; w < kAppendThreads / 32; ++w) m = fmaxf(m, s_max[w]);
  const int e = q8_need_exp(m);
  float scale = exp2_int(e), inv = exp2_int(-e);
  if (old > scale) {
    scale = old;
    // A scale from elsewhere may be no power of two: its quotients are divisions.
    inv = (__float_as_uint(old) & 0x7fffffu) == 0 ? 1.f / old : 0.f;
  }
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int r = r0 + p * kRpp;
    uint2* dst = reinterpret_cast<uint2*>(codes + r * D + d0);
    if (is_new[p]) {
      float* v = f[p];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = inv != 0.f ? v[j] * inv : v[j] / scale;
      *dst = make_uint2(e4m3_pack4(v[0], v[1], v[2], v[3]), e4m3_pack4(v[4], v[5], v[6], v[7]));
    } else if (r < kept && scale != old) {
      const uint2 w = *dst;
      const float g = old / scale;
      *dst = make_uint2(e4m3_rescale4(w.x, g), e4m3_rescale4(w.y, g));
    }
  }
  if (tid == 0 && scale != old) *scale_p = scale;
}

}  // namespace sv
