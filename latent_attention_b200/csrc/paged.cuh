// e4m3 values and power-of-two block scales of the paged latent cache.
#pragma once
#include <cstdint>

#include "internal.h"

namespace mla {
namespace paged {

// Smallest exponent of a block's scale: a block of zeros has 2^-64.  (The
// largest that fp32 rows can need is 2^120.)
constexpr int kMinExp = -64;

// Two floats -> two e4m3 bytes (lo in the low byte), nearest even, +-448 at
// the ends; NaN stays NaN.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  return to_e4m3x2(a, b) | (to_e4m3x2(c, d) << 16);
}
// Two e4m3 bytes -> an fp16 pair (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)v));
  return r;
}
__device__ __forceinline__ void from_e4m3x4(uint32_t v, float (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t h = e4m3x2_to_f16x2(v >> (16 * i));
    asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\t"
        "cvt.f32.f16 %1, h;\n\t}"
        : "=f"(f[2 * i]), "=f"(f[2 * i + 1])
        : "r"(h));
  }
}

// (d0, d1) *= (a0, a1) in one packed instruction.
__device__ __forceinline__ void mul2(float& d0, float& d1, float a0, float a1) {
  asm("{\n\t.reg .b64 a, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 d, {%0, %1};\n\t"
      "mul.rn.f32x2 d, d, a;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "+f"(d0), "+f"(d1)
      : "f"(a0), "f"(a1));
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// 2^e for e in [-126, 127]; 0 below, 2^127 above.
__device__ __forceinline__ float pow2(int e) {
  return e < -126 ? 0.f : __int_as_float((min(e, 127) + 127) << 23);
}

// Smallest e >= kMinExp with amax <= 448 * 2^e, for the bits of a finite
// amax = m 2^k, 1 <= m < 2: 448 = 1.75 * 2^8, so e is k - 8 while m <= 1.75
// and k - 7 above.
__device__ __forceinline__ int scale_exp(uint32_t amax_bits) {
  const int k = (int)(amax_bits >> 23) - 127;
  return max(k - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0), kMinExp);
}

// Exponent of a block's stored scale; false unless it is a power of two that
// the append writes (2^-64 .. 2^120).
__device__ __forceinline__ bool stored_exp(float scale, int* e) {
  const uint32_t b = __float_as_uint(scale);
  *e = (int)(b >> 23) - 127;
  return (b & 0x807fffffu) == 0 && *e >= kMinExp && *e <= 120;
}
// A stored scale to read values with: 1, reported, for one that the append does
// not write.
__device__ __forceinline__ float read_scale(float scale, uint32_t* status) {
  int e;
  if (stored_exp(scale, &e)) return scale;
  atomicOr(status, kStatusBadPage);
  return 1.f;
}

// 32 bytes at a 32-byte aligned address in one access: a warp's whole sectors,
// where two accesses of 16 bytes would each touch half of every sector.
__device__ __forceinline__ void load32(const void* p, uint32_t* w) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                 "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}
__device__ __forceinline__ void store32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ bool aligned32(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 31u) == 0;
}

// 16 elements of a row as they lie in memory, 32 or 64 bytes.  wide: the
// address is 32-byte aligned.
template <typename T> struct Piece;
template <> struct Piece<__nv_bfloat16> { static constexpr int N = 8; uint32_t w[8]; };
template <> struct Piece<float> { static constexpr int N = 16; uint32_t w[16]; };

template <typename T>
__device__ __forceinline__ void load_piece(const T* p, bool wide, Piece<T>& x) {
  if (wide) {
#pragma unroll
    for (int i = 0; i < Piece<T>::N; i += 8) load32(reinterpret_cast<const uint32_t*>(p) + i, x.w + i);
  } else {
#pragma unroll
    for (int i = 0; i < Piece<T>::N; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p) + i);
      x.w[i] = v.x; x.w[i + 1] = v.y; x.w[i + 2] = v.z; x.w[i + 3] = v.w;
    }
  }
}
template <typename T>
__device__ __forceinline__ void store_piece(T* p, bool wide, const Piece<T>& x) {
  if (wide) {
#pragma unroll
    for (int i = 0; i < Piece<T>::N; i += 8) store32(reinterpret_cast<uint32_t*>(p) + i, x.w + i);
  } else {
#pragma unroll
    for (int i = 0; i < Piece<T>::N; i += 4)
      *reinterpret_cast<uint4*>(reinterpret_cast<uint32_t*>(p) + i) =
          make_uint4(x.w[i], x.w[i + 1], x.w[i + 2], x.w[i + 3]);
  }
}
__device__ __forceinline__ void values(const Piece<float>& x, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(x.w[i]);
}
__device__ __forceinline__ void values(const Piece<__nv_bfloat16>& x, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = __uint_as_float(x.w[i] << 16);
    v[2 * i + 1] = __uint_as_float(x.w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void piece_of(const float (&v)[16], Piece<float>& x) {
#pragma unroll
  for (int i = 0; i < 16; ++i) x.w[i] = __float_as_uint(v[i]);
}
__device__ __forceinline__ void piece_of(const float (&v)[16], Piece<__nv_bfloat16>& x) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    x.w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
}

// 16 e4m3 bytes times a scale.
__device__ __forceinline__ void dequant16(uint4 c, float s, float (&v)[16]) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[4];
    from_e4m3x4(w[i], f);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[4 * i + k] = f[k] * s;
  }
}

// First index in [0, n) whose inclusive prefix sum `ends` exceeds i.
__device__ __forceinline__ int request_of(const int32_t* ends, int n, int i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] <= i) lo = mid + 1; else hi = mid;
  }
  return lo;
}

}  // namespace paged
}  // namespace mla
