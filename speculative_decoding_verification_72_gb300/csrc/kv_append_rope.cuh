// New keys and values into the 16-bit paged cache, keys and queries rotated by
// position on the way.
//
// Row n of request b has position p = base_b + depth(n) (base_b + n in a chain)
// and slot base_b + n. With a_i = p inv_freq_i, i < R / 2, the pair (x, y) of
// dims (i, i + R / 2), or (2 i, 2 i + 1) where interleaved, becomes
//   (x cos a_i - y sin a_i, y cos a_i + x sin a_i);
// dims from R on, and values, are moved as they are.
//
// Angles are right to 2^-23 of a turn for positions below 2^24 (2^-17 up to
// 2^31) and inv_freq up to 1, without 64 bits: rope_angle.cuh. Rotations are
// fp32, rounded once to the row's type.
//
// A CTA takes a few rows of a request: first the loads of the rows themselves
// (they need neither page nor angle), then pages, depths and angles (one angle
// a thread, shared through shared memory by all heads of the row), then
// rotation and stores. A thread's unit is two 16-byte pieces of a head that use
// the same eight angles. Every CTA looks at all pages that the request's rows
// touch, since a request with a bad one is left untouched.
//
// Bound by memory: 302 MB of three 4099-row prompts (32 heads on 8 of 128) take
// 52 us, 5.8 TB/s of reads and writes mixed. The look at all pages grows with the
// square of a prompt: 131072 rows take 531 us on pages of 128, 959 on pages of 16.
// Sines by thread for a whole row, not by unit, since 48 heads share them. A step's
// 192 or 1024 rows take 8 and 9 us, the launch and three dependent loads.
#pragma once

#include "paged_common.cuh"
#include "rope_angle.cuh"

namespace sv {

constexpr int kRopeThreads = 256;
constexpr int kRopeBatch = 4;          // units a thread has in flight
constexpr int kRopeRows = 16;          // most rows a CTA

struct RopeArgs {
  const uint8_t* x[3];                 // k, v, q (or nullptr)
  int64_t sb[3], sn[3], sh[3];         // bytes: request, row, head
  PagedView c;
  uint8_t* q_out;                      // [B, N, Hq, D]
  const int32_t* base;                 // [B]
  const int32_t* n_nodes;               // [B] or nullptr
  const int32_t* parents;              // [B, N] or nullptr (chain)
  const float* inv_freq;               // [rot / 2]
  int32_t* out_len;
  int32_t* status;
  int32_t B, N, Hq, rot, interleaved;
  int32_t R, blocks;                   // rows a CTA, CTAs a request
  uint32_t inv_heads;                  // ceil(2^32 / (2 Hkv + Hq)): exact for the units of a CTA
};

// cos and sin of p f.
__device__ __forceinline__ float2 rope_angle(int p, float f) {
  float s, c;
  sincospif(2.f * rope_turn(p, f), &s, &c);
  return make_float2(c, s);
}

template <typename T, int D>
__global__ void __launch_bounds__(kRopeThreads) kv_append_rope_kernel(const RopeArgs a) {
  constexpr int kUnits = D / 16;                        // a head
  constexpr int kStep = kRopeThreads / kUnits;          // heads a pass
  __shared__ float s_cos[kRopeRows * (D / 2)], s_sin[kRopeRows * (D / 2)];
  __shared__ int64_t s_off[2][kRopeRows];               // of the row's slot in k and v, -1 if it has none
  __shared__ int32_t s_pos[kRopeRows];
  __shared__ int32_t s_par[SV_MAX_TREE_NODES];
  const int tid = threadIdx.x;
  const int b = blockIdx.x / a.blocks, row0 = (blockIdx.x - b * a.blocks) * a.R;
  const int rows = min(a.R, a.N - row0), heads = 2 * a.c.Hkv + a.Hq;
  const int total = rows * heads, unit = tid % kUnits, half = a.rot >> 1;
  grid_dep_wait();
  grid_dep_launch();

  // Unit `unit` of head slot u (heads of k, of v, of q; row by row) lies in two pieces of 16 bytes.
  struct Unit {
    int row, head, which;
    int d0, d1;   // elements
    bool turn;
  };
  auto unit_of = [&](int u) {
    Unit x;
    x.row = static_cast<int>(__umulhi(static_cast<uint32_t>(u), a.inv_heads));
    x.head = u - x.row * heads;
    x.which = x.head < a.c.Hkv ? 0 : x.head < 2 * a.c.Hkv ? 1 : 2;
    x.head -= x.which * a.c.Hkv;
    x.turn = x.which != 1 && unit * 16 < a.rot;
    const bool apart = x.turn && !a.interleaved;
    x.d0 = apart ? unit * 8 : unit * 16;
    x.d1 = apart ? half + unit * 8 : unit * 16 + 8;
    return x;
  };
  uint4 v[kRopeBatch][2];
  auto load = [&](int it) {
#pragma unroll
    for (int k = 0; k < kRopeBatch; ++k) {
      const int u = (it + k) * kStep + tid / kUnits;
      if (u < total) {
        const Unit x = unit_of(u);
        const uint8_t* p = a.x[x.which] + b * a.sb[x.which] + (row0 + x.row) * a.sn[x.which] + x.head * a.sh[x.which];
        v[k][0] = *reinterpret_cast<const uint4*>(p + x.d0 * 2);
        v[k][1] = *reinterpret_cast<const uint4*>(p + x.d1 * 2);
      }
    }
  };
  load(0);

  // ---- pages, positions, angles
  const int base = a.base[b];
  const int n = a.n_nodes ? min(max(a.n_nodes[b], 0), a.N) : a.N;
  bool bad = base < 0 || (a.n_nodes && (a.n_nodes[b] < 0 || a.n_nodes[b] > a.N));
  const int64_t end = static_cast<int64_t>(max(base, 0)) + n;
  bad = bad || end > static_cast<int64_t>(a.c.max_pages) << a.c.page_shift;
  if (!bad && n > 0)
#pragma unroll 1
    for (int64_t lp = (base >> a.c.page_shift) + tid; lp <= (end - 1) >> a.c.page_shift; lp += kRopeThreads)
      bad = bad || paged_page(a.c, b, static_cast<int>(lp)) < 0;
  bool bad_tree = false;
  if (a.parents) {
    const int upto = row0 == 0 ? n : min(row0 + rows, n);   // the first CTA looks at the whole tree
#pragma unroll 1
    for (int i = tid; i < upto; i += kRopeThreads) {
      s_par[i] = a.parents[static_cast<int64_t>(b) * a.N + i];
      bad_tree = bad_tree || bad_parent(s_par[i], i);
    }
  }
  bad = __syncthreads_or(bad);
  if (row0 == 0) {
    bad_tree = __syncthreads_or(bad_tree);
    if (tid == 0) {
      a.out_len[b] = bad ? base : static_cast<int32_t>(end);
      if (a.status) a.status[b] = (bad ? SV_STATUS_BAD_PAGE : 0) | (bad_tree ? SV_STATUS_BAD_PARENT : 0);
    }
  }
  if (tid < rows) {
    const int r = row0 + tid;
    const bool there = r < n && base >= 0;
    s_pos[tid] = there ? static_cast<int>(static_cast<uint32_t>(base) + (a.parents ? tree_depth(s_par, r) : r)) : -1;   // below 0 past int32 too
    const int slot = static_cast<int>(static_cast<uint32_t>(base) + r);
    const int page = there && !bad ? paged_page(a.c, b, slot >> a.c.page_shift) : -1;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      s_off[i][tid] = page < 0 ? -1 : page * a.c.sp[i] + (slot & ((1 << a.c.page_shift) - 1)) * a.c.st[i];
  }
  __syncthreads();
#pragma unroll 1
  for (int i = tid; i < rows * half; i += kRopeThreads) {
    const int r = i / half, j = i - r * half;
    const float2 cs = rope_angle(max(s_pos[r], 0), a.inv_freq[j]);
    s_cos[r * (D / 2) + j] = cs.x;
    s_sin[r * (D / 2) + j] = cs.y;
  }
  __syncthreads();

  // ---- rotation
#pragma unroll 1
  for (int it = 0; it * kStep < total; it += kRopeBatch) {
    if (it > 0) load(it);
#pragma unroll
    for (int k = 0; k < kRopeBatch; ++k) {
      const int u = (it + k) * kStep + tid / kUnits;
      if (u >= total) break;
      const Unit x = unit_of(u);
      if (x.turn) {
        float e[16], o[16], c[8], s[8];
        T::unpack8(v[k][0], e);
        T::unpack8(v[k][1], e + 8);
        const int at = x.row * (D / 2) + unit * 8;
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
          *reinterpret_cast<float4*>(c + j) = *reinterpret_cast<const float4*>(s_cos + at + j);
          *reinterpret_cast<float4*>(s + j) = *reinterpret_cast<const float4*>(s_sin + at + j);
        }
        if (a.interleaved) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            o[2 * j] = e[2 * j] * c[j] - e[2 * j + 1] * s[j];
            o[2 * j + 1] = e[2 * j + 1] * c[j] + e[2 * j] * s[j];
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            o[j] = e[j] * c[j] - e[8 + j] * s[j];
            o[8 + j] = e[8 + j] * c[j] + e[j] * s[j];
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
          v[k][h] = make_uint4(T::pack2(o[8 * h], o[8 * h + 1]), T::pack2(o[8 * h + 2], o[8 * h + 3]),
                               T::pack2(o[8 * h + 4], o[8 * h + 5]), T::pack2(o[8 * h + 6], o[8 * h + 7]));
      }
      uint8_t* to;
      if (x.which == 2) {
        if (s_pos[x.row] < 0) v[k][0] = v[k][1] = make_uint4(0, 0, 0, 0);   // rows past the request's, positions past int32
        to = a.q_out + ((static_cast<int64_t>(b) * a.N + row0 + x.row) * a.Hq + x.head) * (D * 2);
      } else {
        const int64_t off = s_off[x.which][x.row];
        if (off < 0) continue;
        to = a.c.x[x.which] + off + x.head * a.c.sh[x.which];
      }
      *reinterpret_cast<uint4*>(to + x.d0 * 2) = v[k][0];
      *reinterpret_cast<uint4*>(to + x.d1 * 2) = v[k][1];
    }
  }
}

}  // namespace sv
