// Quantising sixteen elements of a head at a time into the cache's format.
#pragma once

#include "kv.cuh"

namespace moe {
namespace {

__device__ __forceinline__ __nv_bfloat162 pair(uint32_t v) { return *reinterpret_cast<const __nv_bfloat162*>(&v); }
__device__ __forceinline__ uint32_t bits(__nv_bfloat162 v) { return *reinterpret_cast<const uint32_t*>(&v); }

// (min x, -max x) of the group that four neighbouring lanes hold, sixteen
// elements each; a NaN among them gives NaN.
__device__ __forceinline__ uint32_t group_range(const uint32_t (&x)[8], unsigned lanes) {
  __nv_bfloat162 lo = pair(x[0]), hi = lo;
#pragma unroll
  for (int j = 1; j < 8; ++j) lo = __hmin2_nan(lo, pair(x[j])), hi = __hmax2_nan(hi, pair(x[j]));
  const uint32_t neg = bits(hi) ^ 0x80008000u;
  __nv_bfloat162 m = __hmin2_nan(pair(__byte_perm(bits(lo), neg, 0x5410)), pair(__byte_perm(bits(lo), neg, 0x7632)));
#pragma unroll
  for (int off = 2; off >= 1; off >>= 1) m = __hmin2_nan(m, pair(__shfl_xor_sync(lanes, bits(m), off)));
  return bits(m);
}

// Eight elements as numbers of the cache's range: the nearest, NaN 0.
__device__ __noinline__ uint4 saturate8(uint4 x4) {
  uint32_t x[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int at = 16 * (j & 1);
    uint32_t e = (x[j / 2] >> at) & 0xFFFFu;
    if ((e & 0x7FFFu) > 0x7F80u)
      e = 0;
    else if ((e & 0x7FFFu) > 0x4780u)  // 2^16
      e = (e & 0x8000u) | 0x4780u;
    x[j / 2] = (x[j / 2] & ~(0xFFFFu << at)) | e << at;
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}

struct Eight {  // elements minus the bias
  float2 a[4];
};

// Code word of eight elements, given as a = x - bias: rne(a / s), at most 15.
// inv: 1 / s, too large by 2^-21 to 2^-19 of it.
//
// q = rne(a * inv), found by adding 1.5 * 2^23, is one too large where a / s is
// a half or within 2^-15 below one, and right elsewhere. The remainder r = a -
// q s is exact in fp32 (q s has 12 bits), and r + s / 2 negative finds the
// latter, 0 the halves, of which odd q step down. As integers: bits(r + s / 2)
// < (q & 1). (Halves are common: bf16 elements lie on a grid. A branch for
// them is taken by most warps.) a / s is below 15.5, the scale being rounded by
// 2^-9 at most, so no code passes 15 but where the scale is subnormal, which
// is left to a division. Two elements per instruction where there is one.
__device__ __forceinline__ uint32_t codes8(const Eight& x, float s, float inv) {
  constexpr float kMagic = 12582912.f;
  const float2 magic = make_float2(kMagic, kMagic), minus = make_float2(-1.f, -1.f);
  const float half = 0.5f * s;
  uint32_t word = 0;
#pragma unroll
  for (int j = 3; j >= 0; --j) {
    const float2 g = __ffma2_rn(x.a[j], make_float2(inv, inv), magic);
    const float2 r = __ffma2_rn(__ffma2_rn(g, minus, magic), make_float2(s, s), x.a[j]);
    const float2 e = __fadd2_rn(r, make_float2(half, half));
#pragma unroll
    for (int i = 1; i >= 0; --i) {
      const uint32_t q = __float_as_uint(i ? g.y : g.x);
      // sum of q 16^j; the constant's bits in every q add up to a known multiple
      word = word * 16u + q;
      if (__float_as_int(i ? e.y : e.x) < int(q & 1u)) --word;
    }
  }
  return word - 0x4B400000u * 0x11111111u;
}
__device__ __noinline__ uint32_t codes8_by_division(Eight x, float s) {
  uint32_t word = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    word |= uint32_t(fminf(rintf(__fdiv_rn(j & 1 ? x.a[j / 2].y : x.a[j / 2].x, s)), 15.f)) << (4 * j);
  return word;
}

// Sixteen elements of a group (four neighbouring lanes hold a group): their
// code words, and the group's scale and bias. `bad` is set if an element of
// the group is not a number of the cache's range.
__device__ __forceinline__ uint2 quantise16(const uint4 (&x4)[2], uint16_t* scale, uint16_t* bias, bool* bad) {
  const unsigned lanes = 0xfu << (threadIdx.x & 28);
  uint32_t x[8] = {x4[0].x, x4[0].y, x4[0].z, x4[0].w, x4[1].x, x4[1].y, x4[1].z, x4[1].w};
  uint32_t m = group_range(x, lanes);
  if (!(fmaxf(fabsf(bf16lo(m)), fabsf(bf16hi(m))) <= kKvLimit) || bf16lo(m) != bf16lo(m) || bf16hi(m) != bf16hi(m)) {
    *bad = true;  // (the four lanes agree)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 y = saturate8(x4[i]);
      x[4 * i] = y.x, x[4 * i + 1] = y.y, x[4 * i + 2] = y.z, x[4 * i + 3] = y.w;
    }
    m = group_range(x, lanes);
  }
  const float lo = bf16lo(m) + 0.f;  // (one zero: a minimum of -0 and +0 may be either)
  const uint16_t sb = f32_to_bf16(__fdiv_rn(-bf16hi(m) - lo, 15.f));
  *scale = sb;
  *bias = f32_to_bf16(lo);
  const float s = bf16_to_f32(sb);
  const float inv = __fdividef(1.f, s) * (1.f + 0x1p-20f);
  uint32_t words[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    Eight a;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      a.a[j] = __fadd2_rn(make_float2(bf16lo(x[4 * i + j]), bf16hi(x[4 * i + j])), make_float2(-lo, -lo));
    words[i] = s >= 1e-30f ? codes8(a, s, inv) : s > 0.f ? codes8_by_division(a, s) : 0;  // (1 / s would overflow)
  }
  return make_uint2(words[0], words[1]);
}

}  // namespace
}  // namespace moe
