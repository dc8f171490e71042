// 8-bit checkpoints of activations: groups of 32 consecutive values of a row with a
// power-of-two scale 2^k, the smallest with max|v| <= Q 2^k and k >= -126 (Q = 127 for int8
// codes, 448 for E4M3), so that v / 2^k is exact, a code never saturates, and code * 2^k is
// exact in bf16.  Scale byte = k + 127; 255 marks a group that held an infinity or NaN.
// Also the loads and stores of 16- and 32-bit activations shared by the training kernels.
#pragma once

#include "common.cuh"

namespace moe {

// Formats of an activation (the values of moe_format_t).
constexpr int kFmtBf16 = 0, kFmtF16 = 1, kFmtF32 = 2, kFmtInt8 = 3, kFmtE4m3 = 4;
constexpr int kGroup8 = 32;       // values that share a scale
constexpr int kBadScale = 255;    // scale byte of a group with an infinity or NaN

__host__ __device__ constexpr int fmt_bytes(int fmt) {
  return fmt == kFmtF32 ? 4 : fmt >= kFmtInt8 ? 1 : 2;
}

// Scale byte of a group from the bits of its max|v| (the integer maximum of the absolute
// values' bits, which orders infinities and NaN above every finite value).
// |v|max = 1.m 2^(e-127): int8 allows 1.m <= 127/64 at k = e - 133, E4M3 1.m <= 1.75 at
// k = e - 135, and one more otherwise, which the addition below carries into e.
template <bool INT8>
__device__ __forceinline__ int scale_byte(uint32_t amax_bits) {
  const int e = static_cast<int>((amax_bits + (INT8 ? 0x0001FFFFu : 0x001FFFFFu)) >> 23);
  const int b = max(e - (INT8 ? 6 : 8), 1);
  return amax_bits >= 0x7F800000u ? kBadScale : b;
}

// 2^k and 2^-k of a scale byte (k + 127 in 1..249, so both are normal); NaN of a bad one.
__device__ __forceinline__ float scale_value(int byte) {
  return byte == kBadScale ? __uint_as_float(0x7FC00000u)
                           : __uint_as_float(static_cast<uint32_t>(byte) << 23);
}
__device__ __forceinline__ float scale_inverse(int byte) {
  return byte == kBadScale ? 0.f : __uint_as_float(static_cast<uint32_t>(254 - byte) << 23);
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void of_pair(uint64_t p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// max(m, |a|, |b|), NaN if one is: its bits order as scale_byte wants them.
__device__ __forceinline__ float amax3(float m, float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}
template <int N>
__device__ __forceinline__ uint32_t amax_bits(const float (&f)[N]) {
  float m = fabsf(f[0]);
  if constexpr (N % 2 == 0) m = amax3(m, f[1], f[1]);
#pragma unroll
  for (int i = N % 2 == 0 ? 2 : 1; i + 1 < N; i += 2) m = amax3(m, f[i], f[i + 1]);
  return __float_as_uint(m);
}

// Codes; inv = scale_inverse of the group (0 for a bad group, whose codes are set to 0 a word
// at a time, whatever its values gave).
// int8: adding 1.5 2^23 rounds a value of at most 127 to an integer (nearest even) and leaves
// its two's complement code in the low byte; the product with a power of two being exact, one
// fma does both, where the conversion instruction runs at a quarter of the rate.
constexpr float kRound8 = 12582912.f;
__device__ __forceinline__ uint32_t int8_bits(float v, float inv) {
  return __float_as_uint(fmaf(v, inv, kRound8));
}
__device__ __forceinline__ uint32_t int8x2(float a, float b, float inv) {  // in the low bytes
  float x, y;
  of_pair(fma2(pair_of(a, b), pair_of(inv, inv), pair_of(kRound8, kRound8)), x, y);
  return __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x0040);
}
__device__ __forceinline__ uint32_t e4m3x2(float a, float b, float inv) {
  float2 p;
  of_pair(mul2(pair_of(a, b), pair_of(inv, inv)), p.x, p.y);
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(p, __NV_SATFINITE, __NV_E4M3));
}

// INT8 is a template parameter because both forms are short: as a run-time choice they would
// both be computed for every value.
template <bool INT8>
__device__ __forceinline__ uint32_t encode1(float v, float inv) {
  return inv == 0.f ? 0u : (INT8 ? int8_bits(v, inv) : e4m3x2(v, 0.f, inv)) & 0xFFu;
}

template <bool INT8>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float inv) {
  const uint32_t w = INT8 ? __byte_perm(int8x2(a, b, inv), int8x2(c, d, inv), 0x5410)
                          : __byte_perm(e4m3x2(a, b, inv), e4m3x2(c, d, inv), 0x5410);
  return inv == 0.f ? 0u : w;
}

template <bool INT8>
__device__ __forceinline__ uint2 encode8(const float (&f)[8], float inv) {
  return make_uint2(encode4<INT8>(f[0], f[1], f[2], f[3], inv),
                    encode4<INT8>(f[4], f[5], f[6], f[7], inv));
}

template <bool INT8>
__device__ __forceinline__ float decode1(uint32_t code, float scale) {
  if (INT8) return static_cast<float>(static_cast<int8_t>(code)) * scale;
  const __half_raw h =
      __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3);  // exact
  return __half2float(__half(h)) * scale;
}

// int8: code + 128 in the low mantissa byte of 2^23, from which 2^23 + 128 is taken again (in
// an operation of its own: 2^23 times the scale may overflow).
template <bool INT8>
__device__ __forceinline__ void decode4(uint32_t w, float scale, float* f) {
  const uint32_t u = w ^ 0x80808080u;
  const uint64_t s2 = pair_of(scale, scale);
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    if (INT8) {
      const uint64_t p = pair_of(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 + i)),
                                 __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441 + i)));
      of_pair(mul2(add2(p, pair_of(-8388736.f, -8388736.f)), s2), f[i], f[i + 1]);
    } else {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
          static_cast<__nv_fp8x2_storage_t>(w >> (8 * i)), __NV_E4M3);
      const float2 p = __half22float2(__half2(h));
      of_pair(mul2(pair_of(p.x, p.y), s2), f[i], f[i + 1]);
    }
  }
}

template <bool INT8>
__device__ __forceinline__ void decode8(uint2 w, float scale, float (&f)[8]) {
  decode4<INT8>(w.x, scale, f);
  decode4<INT8>(w.y, scale, f + 4);
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// ------------------------------------------------------------ 16- and 32-bit elements
__device__ __forceinline__ uint32_t pack2_f16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint4 pack8_f16(const float (&f)[8]) {
  return make_uint4(pack2_f16(f[0], f[1]), pack2_f16(f[2], f[3]), pack2_f16(f[4], f[5]),
                    pack2_f16(f[6], f[7]));
}

// Eight consecutive elements as they lie in memory (16 bytes, or 32 of fp32).
template <int FMT>
struct Raw8 {
  uint4 a;
};
template <>
struct Raw8<kFmtF32> {
  uint4 a, b;
};

template <int FMT>
__device__ __forceinline__ Raw8<FMT> load_raw8(const void* base, int64_t i) {
  Raw8<FMT> r;
  if constexpr (FMT == kFmtF32) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + i);
    r.a = p[0];
    r.b = p[1];
  } else {
    r.a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i);
  }
  return r;
}

template <int FMT>
__device__ __forceinline__ void widen8(const Raw8<FMT>& r, float (&f)[8]) {
  if constexpr (FMT == kFmtF32) {
    const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
  } else if constexpr (FMT == kFmtF16) {
    unpack8_f16(r.a, f);
  } else {
    unpack8(r.a, f);
  }
}

template <int FMT>
__device__ __forceinline__ void store8(void* base, int64_t i, const float (&f)[8]) {
  if constexpr (FMT == kFmtF32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
    p[0] = make_float4(f[0], f[1], f[2], f[3]);
    p[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + i) =
        FMT == kFmtF16 ? pack8_f16(f) : pack8(f);
  }
}

template <int FMT>
__device__ __forceinline__ float load1(const void* base, int64_t i) {
  if constexpr (FMT == kFmtF32) return static_cast<const float*>(base)[i];
  const uint16_t v = static_cast<const uint16_t*>(base)[i];
  if constexpr (FMT == kFmtF16) return __half2float(*reinterpret_cast<const __half*>(&v));
  return __uint_as_float(static_cast<uint32_t>(v) << 16);
}

template <int FMT>
__device__ __forceinline__ void store1(void* base, int64_t i, float f) {
  if constexpr (FMT == kFmtF32) {
    static_cast<float*>(base)[i] = f;
  } else if constexpr (FMT == kFmtF16) {
    static_cast<uint16_t*>(base)[i] = f16_bits(f);
  } else {
    static_cast<uint16_t*>(base)[i] = bf16_bits(f);
  }
}

// The same with the format known at run time (parameters: small, read once per CTA).
__device__ __forceinline__ float load1_any(const void* base, int64_t i, int fmt) {
  return fmt == kFmtF32 ? load1<kFmtF32>(base, i)
                        : fmt == kFmtF16 ? load1<kFmtF16>(base, i) : load1<kFmtBf16>(base, i);
}

}  // namespace moe
