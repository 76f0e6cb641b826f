// sample_weight.cuh -- a token's weight exp((x - max) / T) as a whole number of 2^-44, for sums that do not
// depend on their order (sm_103a).
//
// Which token a random number falls on is decided at borders between running sums: of 10^5 tokens, sums that are off
// by 2^-22 of themselves would put one number in a hundred on the wrong side. GB300 has few fp64 units, so the
// exponential is worked out in pairs of fp32 (hi + lo): the exponent's product with its remainder, a table
// of 2^(j/64) with its remainder, and 2^r for |r| <= 1/128 by the series of the exponential. The result is off by
// 2^-36 of itself at most, found over 4 M random x, max and T, beside the rounding to 2^-44; weights below 2^-18
// are off by 2^-40 of the largest.
#pragma once

#include <math_constants.h>

#include "serve.cuh"

namespace mlora {

constexpr int kWeightBits = 44;  // the largest weight is 2^44: MLORA_SAMPLE_MAX_VOCAB of them stay below 2^63
static_assert(MLORA_SAMPLE_MAX_VOCAB < 1 << (63 - kWeightBits), "sums of weights are held in 63 bits");
constexpr uint64_t kWeightOne = 1ull << kWeightBits;
constexpr int kExp2Steps = 65;

// 2^(j / 64) = x + y, j = -32 .. 32 (from the definition, in 50 digits)
__constant__ float2 exp2_steps[kExp2Steps] = {
    {0x1.6a09e6p-1f, 0x1.9fcef4p-27f}, {0x1.6dfb24p-1f, -0x1.cd72e8p-28f}, {0x1.71f75ep-1f, 0x1.1d8beep-26f}, {0x1.75feb6p-1f, -0x1.37b306p-26f},
    {0x1.7a1148p-1f, -0x1.829fdp-26f}, {0x1.7e2f34p-1f, -0x1.261634p-26f}, {0x1.82589ap-1f, -0x1.accc7cp-27f}, {0x1.868d9ap-1f, -0x1.2edb44p-27f},
    {0x1.8ace54p-1f, 0x1.15506ep-28f}, {0x1.8f1aeap-1f, -0x1.baa232p-27f}, {0x1.93737cp-1f, -0x1.e64744p-26f}, {0x1.97d82ap-1f, -0x1.0d8d84p-32f},
    {0x1.9c4918p-1f, 0x1.51f848p-28f}, {0x1.a0c668p-1f, -0x1.2886a6p-27f}, {0x1.a5503cp-1f, -0x1.b83b54p-26f}, {0x1.a9e6b6p-1f, -0x1.50c048p-26f},
    {0x1.ae89fap-1f, -0x1.a94b14p-27f}, {0x1.b33a2cp-1f, -0x1.ec3a82p-27f}, {0x1.b7f77p-1f, -0x1.a09438p-26f}, {0x1.bcc1eap-1f, -0x1.f687c6p-26f},
    {0x1.c199bep-1f, -0x1.3d56b2p-28f}, {0x1.c67f12p-1f, 0x1.cafa2ap-26f}, {0x1.cb720ep-1f, -0x1.8837ccp-28f}, {0x1.d072d4p-1f, 0x1.40f13p-26f},
    {0x1.d5818ep-1f, -0x1.822dbcp-28f}, {0x1.da9e6p-1f, 0x1.ed9942p-28f}, {0x1.dfc974p-1f, -0x1.908c94p-26f}, {0x1.e502eep-1f, 0x1.e2cffep-27f},
    {0x1.ea4afap-1f, 0x1.52486cp-28f}, {0x1.efa1bep-1f, 0x1.cc2b44p-26f}, {0x1.f50766p-1f, -0x1.246ebp-27f}, {0x1.fa7c18p-1f, 0x1.9e90d8p-29f},
    {0x1p0f, 0.f}, {0x1.02c9a4p0f, -0x1.887fap-28f}, {0x1.059b0ep0f, -0x1.9d4f52p-25f}, {0x1.087452p0f, -0x1.e2990ep-26f},
    {0x1.0b5586p0f, 0x1.9f3122p-25f}, {0x1.0e3ec4p0f, -0x1.a585ccp-25f}, {0x1.11301ep0f, -0x1.fdb496p-25f}, {0x1.1429aap0f, 0x1.d525bcp-25f},
    {0x1.172b84p0f, -0x1.c15742p-27f}, {0x1.1a35bep0f, 0x1.6df96ep-25f}, {0x1.1d4874p0f, -0x1.d2e8cap-25f}, {0x1.2063b8p0f, 0x1.0c519ap-25f},
    {0x1.2387a6p0f, 0x1.ceac48p-25f}, {0x1.26b456p0f, 0x1.789f38p-26f}, {0x1.29e9ep0f, -0x1.5c0424p-25f}, {0x1.2d285ap0f, 0x1.b900c2p-26f},
    {0x1.306fep0f, 0x1.4636e2p-25f}, {0x1.33c08cp0f, -0x1.b37d2p-25f}, {0x1.371a74p0f, -0x1.18aac6p-25f}, {0x1.3a7db4p0f, -0x1.634c02p-25f},
    {0x1.3dea64p0f, 0x1.824684p-25f}, {0x1.4160a2p0f, 0x1.f72e2ap-28f}, {0x1.44e086p0f, 0x1.8624b4p-30f}, {0x1.486a2cp0f, -0x1.47d866p-25f},
    {0x1.4bfdaep0f, -0x1.593abcp-25f}, {0x1.4f9b28p0f, -0x1.2c5a6cp-25f}, {0x1.5342b6p0f, -0x1.2c561p-25f}, {0x1.56f474p0f, -0x1.295b04p-25f},
    {0x1.5ab07ep0f, -0x1.5bd5ecp-27f}, {0x1.5e76f2p0f, -0x1.4a5bd6p-25f}, {0x1.6247ecp0f, -0x1.f8b55p-25f}, {0x1.662388p0f, 0x1.2a9112p-27f},
    {0x1.6a09e6p0f, 0x1.9fcef4p-26f},
};

// log2(e) / T = hi + lo, T from 2^-126 on: 0 <= hi < 2^127
struct WeightScale {
  float hi, lo;
};
__device__ __forceinline__ WeightScale weight_scale(float temperature) {
  constexpr float kHi = 1.44269502f, kLo = 1.92596303e-8f;  // log2(e)
  WeightScale s;
  s.hi = kHi / temperature;
  s.lo = (fmaf(-s.hi, temperature, kHi) + kLo) / temperature;
  if (!(fabsf(s.lo) < 3e38f)) s.lo = 0.f;  // (an infinite temperature: every weight is 1)
  return s;
}

// log2 of the weight = hi + lo, for x < top: the difference with its rounding error (Knuth's two-sum), the product with
// its own (an fma). lo may be NaN where hi is far below -kWeightBits.
__device__ __forceinline__ void weight_log2(float x, float top, const WeightScale &c, float &hi, float &lo) {
  const float s = x - top, b = s - x, e = (x - (s - b)) + (-top - b);
  hi = s * c.hi;
  lo = fmaf(s, c.hi, -hi) + fmaf(s, c.lo, e * c.hi);
}

// The weights, 0 .. 2^44, of N logits that are no NaN; `steps`: exp2_steps in shared memory. Whole warps: what no lane needs is
// left out (far below the largest logit, the weights that fp32 holds exactly enough), the rest is without branches.
template <int N>
__device__ __forceinline__ void weights_of(const float (&x)[N], float top, const WeightScale &c, const float2 *steps, uint64_t (&w)[N]) {
  float y[N], yl[N], most = -CUDART_INF_F;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    weight_log2(x[i], top, c, y[i], yl[i]);
    if (x[i] == top) y[i] = yl[i] = 0.f;
    if (!(y[i] > -(float)(kWeightBits + 2))) y[i] = -(float)(kWeightBits + 2), yl[i] = 0.f;  // (also -inf, and its product with 0)
    most = fmaxf(most, y[i]);
    w[i] = 0;
  }
  if (!__any_sync(~0u, most > -(float)(kWeightBits + 2))) return;
  if (!__any_sync(~0u, most >= -18.f)) {
    // Below 2^-18 fp32's exponential is as exact: off by 2^-22 of itself, 2^-40 of the largest weight.
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float k = rintf(y[i]);
      float f;
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(f) : "f"(y[i] - k + yl[i]));
      w[i] = __float2uint_rn(f * __int_as_float(((int)k + kWeightBits + 127) << 23));
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float k = rintf(y[i]), f = y[i] - k;  // 2^k 2^f, |f| <= 1/2
    const float j = rintf(f * 64.f), r = fmaf(j, -1.f / 64.f, f);
    // (r + yl) ln 2 = z + zl
    constexpr float kLn2Hi = 0x1.62e43p-1f, kLn2Lo = -0x1.05c61p-29f;
    const float z = r * kLn2Hi, zl = fmaf(r, kLn2Hi, -z) + fmaf(r, kLn2Lo, yl[i] * kLn2Hi);
    const float q = z * z * fmaf(z, fmaf(z, 1.f / 24.f, 1.f / 6.f), 0.5f);  // z^2/2 + z^3/6 + z^4/24; the next is 2^-44
    const float2 t = steps[(int)j + 32];
    // (t.x + t.y) (1 + z + zl + q + z zl) = h + l; zl^2 / 2 is below 2^-38
    const float a = t.x * z, al = fmaf(t.x, z, -a);
    const float h = t.x + a;
    const float l = ((t.x - h) + a) + (al + fmaf(t.x, fmaf(z, zl, zl + q), fmaf(t.y, z, t.y)));
    const int shift = -(int)k;
    const uint64_t whole = (uint64_t)(((int64_t)__float2int_rn(h * 0x1p24f) << (kWeightBits - 24)) + (int64_t)__float2int_rn(l * 0x1p44f));
    // (below 2^-18 a weight is the one above, whatever its neighbours are)
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(f + yl[i]));
    w[i] = y[i] < -18.f ? (uint64_t)__float2uint_rn(e * __int_as_float(((int)k + kWeightBits + 127) << 23)) : (whole + ((1ull << shift) >> 1)) >> shift;
  }
}

// floor(f s) and ceil(f s) for 0 <= f < 1, exactly: f = m 2^-e with m below 2^24.
__device__ __forceinline__ uint64_t times_floor(float f, uint64_t s, bool *rest = nullptr) {
  const uint32_t bits = __float_as_uint(f);
  const int ex = (int)(bits >> 23);
  const uint64_t m = ex ? (bits & 0x7FFFFFu) | 0x800000u : bits & 0x7FFFFFu;
  const int e = 150 - (ex ? ex : 1);  // 24 or more
  const uint64_t hi = __umul64hi(m, s), lo = m * s;
  uint64_t v, cut;
  if (e >= 128) v = 0, cut = hi | lo;
  else if (e >= 64) v = hi >> (e - 64), cut = lo | (hi & ((1ull << (e - 64)) - 1));
  else v = hi << (64 - e) | lo >> e, cut = lo & ((1ull << e) - 1);
  if (rest) *rest = cut != 0;
  return v;
}
__device__ __forceinline__ uint64_t times_ceil(float f, uint64_t s) {
  bool rest;
  const uint64_t v = times_floor(f, s, &rest);
  return v + rest;
}

}  // namespace mlora
