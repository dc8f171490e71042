// Pieces that the gated MLP's product kernels share: the MN-major operand descriptor, the 3-D
// bulk copy and the activation.
#pragma once

#include "act8.cuh"

namespace moe {

// True in one lane of a converged warp.  The loops that issue bulk copies and MMAs run under it
// and not under `lane == 0`: the compiler then knows that one thread is active and keeps these
// instructions' operands in uniform registers.  Under `lane == 0` a K step took 810 cycles to
// issue, under this 510, which is the tensor cores' own rate for a pair's 256 x 256 x 64.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Shared-memory descriptor of an MN-major tile laid out by TMA boxes of 64 (M or N) elements x
// 64 K rows with 128-byte swizzling: a box is 8 KB, the next 64 elements follow it (leading
// byte offset), 8 K rows are 1024 bytes apart (stride byte offset).
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(8192 >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t c0, int32_t c1, int32_t c2, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2),
      "l"(policy)
      : "memory");
}

// Eight values in 16 bits.  The format is a template parameter: as a run-time choice both
// conversions would be computed for every value.
template <bool F16>
__device__ __forceinline__ uint32_t pack_two(float a, float b) {
  return F16 ? pack2_f16(a, b) : pack2(a, b);
}
template <bool F16>
__device__ __forceinline__ uint4 pack16(const float* v) {
  return make_uint4(pack_two<F16>(v[0], v[1]), pack_two<F16>(v[2], v[3]),
                    pack_two<F16>(v[4], v[5]), pack_two<F16>(v[6], v[7]));
}
template <bool F16>
__device__ __forceinline__ void unpack16(const uint4& u, float* v) {
  float t[8];
  if (F16)
    unpack8_f16(u, t);
  else
    unpack8(u, t);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = t[e];
}

// ---------------------------------------------------------------- the activation
// Both are a = g L(z) with the logistic L(z) = 1 / (1 + exp(-z)): z = g (silu) or
// 2 sqrt(2/pi) (g + 0.044715 g^3) (gelu_tanh, since (1 + tanh w) / 2 = L(2w)).  Then
// a' = L + g L (1 - L) z'.  For gelu_tanh z' is taken at g^2 <= 256: beyond, L (1 - L) is 0 in
// fp32 and an unbounded z' would turn it into NaN.  Two values at a time.
__device__ __forceinline__ uint64_t both(float v) { return pair_of(v, v); }
struct Gate2 {
  uint64_t a, da;
};
template <bool WITH_D, bool SILU>
__device__ __forceinline__ Gate2 gate_of(uint64_t g) {
  constexpr float kLog2e = 1.4426950408889634f, kC0 = 1.5957691216057308f, kC1 = 0.044715f;
  const uint64_t g2 = mul2(g, g);
  uint64_t w = mul2(g, both(SILU ? -kLog2e : -kC0 * kLog2e));  // exp(-z) = 2^w
  if (!SILU) w = mul2(w, fma2(g2, both(kC1), both(1.f)));
  float w0, w1, l0, l1;
  of_pair(w, w0, w1);
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w0) : "f"(w0));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w1) : "f"(w1));
  of_pair(add2(pair_of(w0, w1), both(1.f)), w0, w1);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(l0) : "f"(w0));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(l1) : "f"(w1));
  const uint64_t l = pair_of(l0, l1);
  Gate2 r;
  r.a = mul2(g, l);
  r.da = 0;
  if (WITH_D) {
    uint64_t t = mul2(r.a, fma2(l, both(-1.f), both(1.f)));
    if (!SILU) {
      float q0, q1;
      of_pair(g2, q0, q1);
      t = mul2(t, fma2(pair_of(fminf(q0, 256.f), fminf(q1, 256.f)), both(3.f * kC1 * kC0), both(kC0)));
    }
    r.da = add2(t, l);
  }
  return r;
}

}  // namespace moe
