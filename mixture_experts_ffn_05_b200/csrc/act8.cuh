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

// 2^k and 2^-k of a scale byte (k + 127 in 1..248, so both are normal); NaN of a bad one.
__device__ __forceinline__ float scale_value(int byte) {
  return byte == kBadScale ? __uint_as_float(0x7FC00000u)
                           : __uint_as_float(static_cast<uint32_t>(byte) << 23);
}
__device__ __forceinline__ float scale_inverse(int byte) {
  return byte == kBadScale ? 0.f : __uint_as_float(static_cast<uint32_t>(254 - byte) << 23);
}

// Codes; inv = scale_inverse of the group (0 for a bad group, whose codes are set to 0 a word
// at a time, whatever its values gave).
// int8: adding 1.5 2^23 rounds a value of at most 127 to an integer (nearest even) and leaves
// its two's complement code in the low byte: one addition, where the conversion instruction
// runs at a quarter of the rate.
__device__ __forceinline__ uint32_t int8_bits(float v, float inv) {
  return __float_as_uint(__fadd_rn(__fmul_rn(v, inv), 12582912.f));
}
__device__ __forceinline__ uint32_t e4m3x2(float a, float b, float inv) {
  return static_cast<uint32_t>(
      __nv_cvt_float2_to_fp8x2(make_float2(a * inv, b * inv), __NV_SATFINITE, __NV_E4M3));
}

// INT8 is a template parameter because both forms are short: as a run-time choice they would
// both be computed for every value.
template <bool INT8>
__device__ __forceinline__ uint32_t encode1(float v, float inv) {
  return inv == 0.f ? 0u : (INT8 ? int8_bits(v, inv) : e4m3x2(v, 0.f, inv)) & 0xFFu;
}

template <bool INT8>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float inv) {
  const uint32_t w =
      INT8 ? __byte_perm(__byte_perm(int8_bits(a, inv), int8_bits(b, inv), 0x0040),
                         __byte_perm(int8_bits(c, inv), int8_bits(d, inv), 0x0040), 0x5410)
           : e4m3x2(a, b, inv) | (e4m3x2(c, d, inv) << 16);
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

// int8: code + 128 in the low mantissa byte of 2^23, from which 2^23 + 128 is taken again.
template <bool INT8>
__device__ __forceinline__ void decode4(uint32_t w, float scale, float* f) {
  if (INT8) {
    const uint32_t u = w ^ 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[i] = (__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 + i)) - 8388736.f) * scale;
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
          static_cast<__nv_fp8x2_storage_t>(w >> (16 * i)), __NV_E4M3);
      const float2 p = __half22float2(__half2(h));
      f[2 * i] = p.x * scale;
      f[2 * i + 1] = p.y * scale;
    }
  }
}

template <bool INT8>
__device__ __forceinline__ void decode8(uint2 w, float scale, float (&f)[8]) {
  decode4<INT8>(w.x, scale, f);
  decode4<INT8>(w.y, scale, f + 4);
}

// The integer maximum of |v| bits over the 32 lanes, and over groups of 4 lanes.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t max4_lanes(uint32_t a) {
  a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
  return max(a, __shfl_xor_sync(0xffffffffu, a, 2));
}

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
