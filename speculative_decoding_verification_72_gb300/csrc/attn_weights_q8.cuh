// Accumulated attention weight of the accepted rows, the score that eviction
// ranks by.
//
// Row i of request b (i = 0 .. num_accepted[b]; node path_nodes[b, i] of the
// verify pass, or node i) is the token at position base_b + i. With the
// attention's own lse, per kv head:
//   w_j = sum over rows i and the G heads of the group of exp(s_ij - lse_i), j <= base + i
//   out_j = decay * scores_j + w_j (j < base), w_j (base <= j < length), 0 (j >= length)
//
// The verify pass cannot do this itself: which rows count is known only after
// verification. Keys alone are read again (half of a position's bytes), and
// since lse is known there is no maximum, no sum and nothing to join: each
// 16-token unit gives its own weights. Same line of tiles, private cp.async
// rings and fragments as attn_q8.cuh; weights are formed and summed in fp32.
// Bound by memory up to 64 rows a kv head; more rows take more passes.
#pragma once

#include "attn_q8.cuh"

namespace sv {

constexpr int kWtStages = 6;

struct WeightArgs {
  const uint8_t* q;
  int64_t sqb, sqn, sqh;       // bytes: request, node, head
  const float* lse;            // [B, N, Hq]
  Q8View c;
  const int32_t* base;         // [B]
  const int32_t* path;         // [B, path_cols] or nullptr
  const int32_t* num_acc;      // [B] or nullptr (all N rows)
  const float* scores;         // [B, Hkv, S]
  float* out;                  // [B, Hkv, S]
  int32_t* status;             // [B] or nullptr
  int32_t path_cols, B, N, G, Hq, S, grid;
  float coef, decay;
};

// count = rows that count; len = positions that hold a token.
__device__ __forceinline__ AttnReq weight_req(const WeightArgs& a, int b) {
  AttnReq r;
  const int cap = min(a.c.max_pages << a.c.page_shift, a.S);
  r.base = a.base[b];
  r.n = a.num_acc ? min(max(a.num_acc[b] + 1, 0), a.path ? min(a.path_cols, a.N) : a.N) : a.N;
  if (r.base < 0) r.base = r.n = 0;
  r.base = min(r.base, cap);
  r.len = min(r.base + r.n, cap);
  return r;
}

template <int D, int MT>
constexpr int weight_smem_bytes() {
  return kAttnWarps * kWtStages * 16 * D + MT * (D / 16) * 512 + 16 * MT * 4;
}

template <typename T, int D, int MT>
__global__ void __launch_bounds__(kAttnThreads, MT == 4 ? 3 : 4) attn_weights_q8_kernel(const WeightArgs a) {
  constexpr int kKs = D / 16, kRows = 16 * MT;
  constexpr int kUnit = 16 * D;
  constexpr int kChunks = 16 * (D / 16);
  extern __shared__ __align__(128) uint8_t smem[];
  uint4* s_q = reinterpret_cast<uint4*>(smem + kAttnWarps * kWtStages * kUnit);
  float* s_qs = reinterpret_cast<float*>(s_q + MT * kKs * 32);
  __shared__ AttnLine s_line;
  __shared__ int32_t s_warp[kAttnWarps];

  grid_dep_wait();
  grid_dep_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int H = a.c.Hkv, cta = blockIdx.x;

  const AttnRanges ranges = attn_scan<kAttnThreads>(
      a.B, [&](int r) { return (weight_req(a, r).len + kAttnTile - 1) / kAttnTile; }, a.grid, cta, &s_line, s_warp, H, nullptr);
  const uint32_t ring = smem_u32(smem) + warp * (kWtStages * kUnit);

  if (cta < ranges.n) {
    const int lo = ranges.begin(cta), hi = ranges.begin(cta + 1);
    int b = s_line.b;
    int off = s_line.off;
    AttnReq rq = weight_req(a, b);
    for (int pos = lo; pos < hi;) {
      int tiles = (rq.len + kAttnTile - 1) / kAttnTile;
      while (pos >= (off + tiles) * H) {
        off += tiles;
        rq = weight_req(a, ++b);
        tiles = (rq.len + kAttnTile - 1) / kAttnTile;
      }
      const int rel = pos - off * H;
      const int h = rel / tiles, t0 = rel - h * tiles;
      const int nt_ = min(tiles - t0, hi - pos);
      const int32_t* path = a.path ? a.path + static_cast<int64_t>(b) * a.path_cols : nullptr;
      const float* sc = a.scores + (static_cast<int64_t>(b) * H + h) * a.S;
      float* out = a.out + (static_cast<int64_t>(b) * H + h) * a.S;
      // lane (g, c), g < 4, writes token 8 (g / 2) + 2 c + g % 2 of a unit
      const int my_tok = (g >> 1 & 1) * 8 + 2 * c + (g & 1);
      const int rows_total = rq.n * a.G;

      for (int row0 = 0; row0 == 0 || row0 < rows_total; row0 += kRows) {
        int pid = -1, pid_n = -1;
        float ksv = 0.f, ks_n = 0.f;
        auto fetch = [&](int i0, int& p, float& k_) {
          const int tok = (t0 + i0 + lane) * kAttnTile + warp * 16;
          p = i0 + lane < nt_ && tok < rq.len ? q8_page(a.c, b, tok >> a.c.page_shift) : -1;
          k_ = p >= 0 ? a.c.ks[static_cast<int64_t>(p) * H + h] : 0.f;
        };
        auto issue = [&](int i, int page) {
          if (i < nt_) {
            const int tok = (t0 + i) * kAttnTile + warp * 16;
            const int valid = page < 0 ? 0 : rq.len - tok;
            const int64_t o =
                (((static_cast<int64_t>(max(page, 0)) * H + h) << a.c.page_shift) + (tok & ((1 << a.c.page_shift) - 1))) * D;
            const uint32_t dst = ring + (i % kWtStages) * kUnit;
#pragma unroll
            for (int it = 0; it < kChunks / 32; ++it) {
              const int ch = it * 32 + lane;
              const int row = ch / (D / 16), col = ch % (D / 16);
              cp_async16(dst + unit_off<D>(row, col), a.c.k + o + ch * 16, row < valid);
            }
          }
          cp_async_commit();
        };
        // what a unit's weights are added to, loaded one unit ahead
        auto old_score = [&](int i) {
          const int tok = (t0 + i) * kAttnTile + warp * 16 + my_tok;
          if (g >= 4 || i >= nt_ || tok >= rq.len) return 0.f;
          return row0 > 0 ? out[tok] : tok < rq.base ? a.decay * sc[tok] : 0.f;
        };
        fetch(0, pid, ksv);
        if (nt_ > 32) fetch(32, pid_n, ks_n);
#pragma unroll
        for (int i = 0; i < kWtStages - 1; ++i) issue(i, __shfl_sync(0xffffffffu, pid, i));
        float old = old_score(0);
        load_q_frags<T, D, MT, kAttnThreads>(a.q + b * a.sqb + static_cast<int64_t>(h) * a.G * a.sqh, a.sqn, a.sqh,
                                             rows_total, row0, a.G, path, a.N, reinterpret_cast<uint32_t*>(s_q), s_qs);
        __syncthreads();
        float cq[MT][2], l2[MT][2];
        int at[MT][2];   // the row's own position, relative to base; -1: no row
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = mt * 16 + i * 8 + g, R = row0 + r;
            cq[mt][i] = s_qs[r] * a.coef;
            at[mt][i] = R < rows_total ? R / a.G : -1;
            l2[mt][i] = 0.f;
            if (at[mt][i] >= 0) {
              const int n = path ? path[at[mt][i]] : at[mt][i];
              if (n >= 0 && n < a.N)
                l2[mt][i] = a.lse[(static_cast<int64_t>(b) * a.N + n) * a.Hq + h * a.G + (R - at[mt][i] * a.G)] * kLog2e;
              else
                at[mt][i] = -1;
            }
          }
        for (int i = 0; i < nt_; ++i) {
          const int page = __shfl_sync(0xffffffffu, pid, i & 31);
          const float ks = __shfl_sync(0xffffffffu, ksv, i & 31);
          cp_async_wait<kWtStages - 2>();
          __syncwarp();
          {
            const int j = i + kWtStages - 1;
            const int pj = __shfl_sync(0xffffffffu, (j ^ i) & ~31 ? pid_n : pid, j & 31);
            issue(j, pj);
          }
          const float next = old_score(i + 1);
          if ((i & 31) == 31) {
            pid = pid_n;
            ksv = ks_n;
            fetch(i + 33, pid_n, ks_n);
          }
          const int tok = (t0 + i) * kAttnTile + warp * 16;
          float w[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
          if (page >= 0) {
            float s[MT][2][4];
            unit_scores<D, MT>(ring + (i % kWtStages) * kUnit, s_q, lane, s);
            const bool edge = tok + 16 > rq.base;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int n = at[mt][e >> 1];
                  const float p = ex2(s[mt][nt][e] * (cq[mt][e >> 1] * ks) - l2[mt][e >> 1]);
                  bool see = n >= 0;
                  if (edge) see = see && tok + nt * 8 + 2 * c + (e & 1) - rq.base <= n;
                  w[nt][e & 1] += see ? p : 0.f;
                }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1)
#pragma unroll
              for (int nt = 0; nt < 2; ++nt) {
                w[nt][0] += __shfl_xor_sync(0xffffffffu, w[nt][0], o);
                w[nt][1] += __shfl_xor_sync(0xffffffffu, w[nt][1], o);
              }
          }
          if (g < 4 && tok + my_tok < rq.len)
            out[tok + my_tok] = old + (g >> 1 & 1 ? (g & 1 ? w[1][1] : w[1][0]) : (g & 1 ? w[0][1] : w[0][0]));
          old = next;
        }
        cp_async_wait<0>();
        __syncthreads();
      }
      pos += nt_;
    }
  }
  // Positions past the end, and what is wrong with a request, spread over the CTAs.
  for (int x = cta; x < a.B * H; x += gridDim.x) {
    const int b = x / H;
    const int len = weight_req(a, b).len;
    for (int j = len + tid; j < a.S; j += kAttnThreads) a.out[static_cast<int64_t>(x) * a.S + j] = 0.f;
  }
  if (a.status)
    for (int b = cta; b < a.B; b += gridDim.x) {
      const AttnReq rq = weight_req(a, b);
      const int n = a.num_acc ? a.num_acc[b] + 1 : a.N;
      bool bad = a.base[b] < 0 || n < 0 || n != rq.n || rq.len != a.base[b] + n;
      for (int j = tid; j < (rq.len + (1 << a.c.page_shift) - 1) >> a.c.page_shift; j += kAttnThreads)
        bad = bad || q8_page(a.c, b, j) < 0;
      if (a.path)
        for (int i = tid; i < rq.n; i += kAttnThreads) {
          const int p = a.path[static_cast<int64_t>(b) * a.path_cols + i];
          bad = bad || p < 0 || p >= a.N;
        }
      bad = __syncthreads_or(bad);
      if (tid == 0) a.status[b] = bad ? SV_STATUS_BAD_PAGE : 0;
    }
}

}  // namespace sv
