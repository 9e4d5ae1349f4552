// The quantiser of the operators beside the step (4-bit cache rows, 4-bit
// matrices): 16 elements to E2M1 codes and an E4M3 scale, as the step's
// activation quantiser gives them.
#pragma once

#include <type_traits>

#include "msk_ops.cuh"

namespace msk {

// 16 consecutive elements of type DT as floats.
template <int DT>
__device__ __forceinline__ void load16(const void* base, long long off, float (&x)[16]) {
  if (DT == MSK_FP32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + off);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = __ldg(p + i);
      x[4 * i] = f.x, x[4 * i + 1] = f.y, x[4 * i + 2] = f.z, x[4 * i + 3] = f.w;
    }
  } else {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + off);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 u = __ldg(p + i);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = unpack16(w[j], DT == MSK_FP16);
        x[8 * i + 2 * j] = f.x, x[8 * i + 2 * j + 1] = f.y;
      }
    }
  }
}

// Two -x / d rounded to nearest (my: two rounded reciprocals of d, negative;
// quotients and remainders within the normal range): Markstein's correction of
// x my by its remainder (IBM J. Res. Dev. 34, 1990).  The codes depend on the
// quotient's last bit where it lies half way between two of them.  The negative
// quotient, because a remainder of 0 is +0: times my it is -0, which leaves the
// sign of a zero alone, and +0, times y, would not.
__device__ __forceinline__ void minus_quotients(float& x0, float& x1, unsigned long long d, unsigned long long my) {
  const unsigned long long x = pair(x0, x1), q = mul2(x, my);
  unpair(fma2(fma2(q, d, x), my, q), x0, x1);
}

// A block of 16 elements over the tensor's scale ts (positive): codes, and the
// scale's code in `sc`.
__device__ __forceinline__ uint2 quantise16(float (&x)[16], float ts, uint32_t& sc) {
  const float yts = __frcp_rn(ts);
  const unsigned long long ts2 = pair(ts, ts), myts2 = pair(-yts, -yts);
  const bool plain = ts > 1e-18f && ts < 1e18f;
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) amax = fmaxf(amax, fabsf(x[j]));
  const bool whole = ts == 1.f;
  if (!whole) {  // x becomes -x / ts
    if (plain && amax < 1e18f) {  // (smaller quotients than normal ones leave codes of 0)
#pragma unroll
      for (int j = 0; j < 16; j += 2) minus_quotients(x[j], x[j + 1], ts2, myts2);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = __fdiv_rn(x[j], -ts);
    }
    amax = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) amax = fmaxf(amax, fabsf(x[j]));
  }
  // amax / 6 (what is beyond 448 saturates)
  const float y6 = 1.f / 6.f, am = fminf(amax, 1e6f), q6 = am * y6;
  sc = f32_to_e4m3(fmaf(fmaf(-q6, 6.f, am), y6, q6));
  const float dec = e4m3_to_f32(sc);
  uint32_t c[2] = {0u, 0u};
  if (amax > 2688.f) {  // saturates, with infinities perhaps
    const float d = whole ? dec : -dec;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      c[j >> 2] |= f32x2_to_e2m1x2(__fdiv_rn(x[2 * j], d), __fdiv_rn(x[2 * j + 1], d)) << (8 * (j & 3));
  } else if (dec > 0.f) {
    const float y = __frcp_rn(dec);
    auto codes = [&](auto negate) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float u = x[2 * j], v = x[2 * j + 1];
        minus_quotients(u, v, pair(dec, dec), pair(-y, -y));
        c[j >> 2] |= (negate() ? f32x2_to_e2m1x2(-u, -v) : f32x2_to_e2m1x2(u, v)) << (8 * (j & 3));
      }
    };
    if (whole) codes(std::true_type());
    else codes(std::false_type());  // (two negative quotients)
  }
  return make_uint2(c[0], c[1]);
}

}  // namespace msk
