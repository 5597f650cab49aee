// fp32 values as bf16 operands of the tensor cores, without loss: a value is the
// exact sum of its top 8 significand bits, the next 8 and the last 8.
#pragma once

#include <stdint.h>

namespace area {
namespace {

// The order of the six terms: parts of the first and of the second factor.
__device__ __forceinline__ constexpr uint32_t part_a(int t) { return 0x102010u >> (4 * (5 - t)) & 3u; }
__device__ __forceinline__ constexpr uint32_t part_b(int t) { return 0x120100u >> (4 * (5 - t)) & 3u; }

// The top parts of two values, packed (a in the low half); what is left of the
// values takes their place.
__device__ __forceinline__ uint32_t cut2(float& a, float& b) {
  const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
  a -= __uint_as_float(x & 0xffff0000u);
  b -= __uint_as_float(y & 0xffff0000u);
  return __byte_perm(x, y, 0x7632);
}

__device__ __forceinline__ void st_shared16(uint32_t at, const uint32_t (&w)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3])
               : "memory");
}

// Eight values of a row in registers, as the operand's 16-byte pieces: part t
// at t * term.
__device__ __forceinline__ void put8(uint32_t at, int term, float (&f)[8]) {
#pragma unroll
  for (int t = 0; t < 3; ++t) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = cut2(f[2 * i], f[2 * i + 1]);
    st_shared16(at + t * term, w);
  }
}
// Eight values of a row, or zeros.
__device__ __forceinline__ void get8(const float* p, bool in, float (&f)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in) x = __ldg(reinterpret_cast<const float4*>(p) + h);
    f[4 * h] = x.x, f[4 * h + 1] = x.y, f[4 * h + 2] = x.z, f[4 * h + 3] = x.w;
  }
}

// Four values of a row, or zeros, that no other block of the SM will read.
__device__ __forceinline__ void get4(const float* p, bool in, float (&f)[4]) {
  f[0] = f[1] = f[2] = f[3] = 0.f;
  if (in)
    asm volatile("ld.global.nc.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3])
                 : "l"(p));
}
// Four values as the operand's 8-byte pieces: part t at t * term.
__device__ __forceinline__ void put4(uint32_t at, int term, float (&f)[4]) {
#pragma unroll
  for (int t = 0; t < 3; ++t) {
    const uint32_t x = cut2(f[0], f[1]), y = cut2(f[2], f[3]);
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at + t * term), "r"(x), "r"(y) : "memory");
  }
}

}  // namespace
}  // namespace area
