// The angle of the position rotation, in turns; also compiled by a host
// compiler, for its test.
//
// p f has more bits than fp32 holds, and only its fraction of a turn counts.
// f / 2 pi is taken as a sum of two floats, r + r_lo, and p as p1 + p0 with p0 <
// 2^12, so p1 and p0 are exact and each product's rounding error is had exactly by
// fma. Whole turns are taken off the products and off their sum.
//
// Error, for f up to 1 and p < 2^24 (2^31): the sum of the products' fractions
// is rounded to 2^-25 (2^-25), the end result to 2^-25 (2^-19); the rest, which is
// below 0.4 (48), is summed with roundings of 2^-27, 2^-27 and 2^-26 (2^-20, 2^-20,
// 2^-19), and r + r_lo is off by 2^-50.4 of a turn a position: in all
// below 1.8 2^-24 (2^-17). It grows with f above 1. Every operation is rounded by
// itself: joined into an fma, a product less its whole turns would have its
// rounding error taken off twice.
#pragma once

#include <cmath>

#ifdef __CUDACC__
#define SV_BOTH __host__ __device__ __forceinline__
#else
#define SV_BOTH inline
#endif

namespace sv {

SV_BOTH float lone_mul(float x, float y) {
#ifdef __CUDA_ARCH__
  return __fmul_rn(x, y);
#else
  return x * y;   // to be compiled with -ffp-contract=off
#endif
}
SV_BOTH float lone_add(float x, float y) {
#ifdef __CUDA_ARCH__
  return __fadd_rn(x, y);
#else
  return x + y;
#endif
}

// p f / 2 pi less whole turns: within 1 of 0 for p < 2^24.
SV_BOTH float rope_turn(int p, float f) {
  constexpr float kTurn = 0.15915493667125701904f, kTurnLo = 6.4206383e-9f;   // 1 / 2 pi as a sum of floats
  const float r = lone_mul(f, kTurn), r_lo = fmaf(f, kTurnLo, fmaf(f, kTurn, -r));
  const float p1 = static_cast<float>(p & ~0xfff), p0 = static_cast<float>(p & 0xfff);
  const float x1 = lone_mul(p1, r), x0 = lone_mul(p0, r);
  const float rest = lone_add(lone_add(fmaf(p1, r, -x1), fmaf(p0, r, -x0)), fmaf(p1, r_lo, lone_mul(p0, r_lo)));
  float x = lone_add(lone_add(x1, -rintf(x1)), lone_add(x0, -rintf(x0)));
  x = lone_add(x, -rintf(x));
  return lone_add(x, rest);
}

}  // namespace sv
