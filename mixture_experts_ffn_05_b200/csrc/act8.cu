// 8-bit activation checkpoints: write and read (see act8.cuh for the format).  Both are one
// pass over the data and bound by HBM: bf16 moves 2 + 1 + 1/32 bytes per value each way.
//
// A warp takes chunks of 256 columns of a row.  Wide form (every row starts on a 16-byte
// boundary and holds whole 8-element pieces): lane l owns columns 8l..8l+7 of the chunk, so a
// group of 32 is four neighbouring lanes.  Narrow form (any column count or stride): lane l
// owns columns l, l + 32, ..., so each access of the warp is one group of 32 consecutive
// elements.  Groups never cross a row.
#include "act8.cuh"
#include "train_internal.h"

namespace moe {

constexpr int kChunk8 = 256;
constexpr int kActWarps = 8;

template <int FMT, bool WIDE>
__global__ void __launch_bounds__(32 * kActWarps) act_encode_kernel(Act8Args a) {
  const int lane = threadIdx.x & 31;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kActWarps;
  const int64_t items = a.rows * a.chunks;
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * kActWarps + (threadIdx.x >> 5); it < items;
       it += stride) {
    const int64_t r = it / a.chunks;
    const int64_t c0 = (it - r * a.chunks) * kChunk8;
    uint8_t* codes = a.codes + r * a.ld_codes;
    uint8_t* scales = a.scales + r * a.groups;
    if constexpr (WIDE) {
      const int64_t c = c0 + 8 * lane;
      float f[8] = {};
      if (c < a.cols) widen8<FMT>(load_raw8<FMT>(a.vals, r * a.ld_vals + c), f);
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, abs_bits(f[i]));
      const int b = scale_byte(max4_lanes(m), a.int8);
      if (c < a.cols) {
        if ((lane & 3) == 0) scales[c / kGroup8] = static_cast<uint8_t>(b);
        *reinterpret_cast<uint2*>(codes + c) = encode8(f, scale_inverse(b), a.int8);
      }
    } else {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t c = c0 + 32 * i + lane;
        f[i] = c < a.cols ? load1<FMT>(a.vals, r * a.ld_vals + c) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t c = c0 + 32 * i + lane;
        const int b = scale_byte(__reduce_max_sync(0xffffffffu, abs_bits(f[i])), a.int8);
        if (c < a.cols) {
          if (lane == 0) scales[c / kGroup8] = static_cast<uint8_t>(b);
          codes[c] = static_cast<uint8_t>(encode1(f[i], scale_inverse(b), a.int8));
        }
      }
    }
  }
}

template <int FMT, bool WIDE>
__global__ void __launch_bounds__(32 * kActWarps) act_decode_kernel(Act8Args a) {
  const int lane = threadIdx.x & 31;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kActWarps;
  const int64_t items = a.rows * a.chunks;
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * kActWarps + (threadIdx.x >> 5); it < items;
       it += stride) {
    const int64_t r = it / a.chunks;
    const int64_t c0 = (it - r * a.chunks) * kChunk8;
    const uint8_t* codes = a.codes + r * a.ld_codes;
    const uint8_t* scales = a.scales + r * a.groups;
    if constexpr (WIDE) {
      const int64_t c = c0 + 8 * lane;
      if (c < a.cols) {
        float f[8];
        decode8(*reinterpret_cast<const uint2*>(codes + c), scale_value(scales[c / kGroup8]),
                a.int8, f);
        store8<FMT>(a.vals, r * a.ld_vals + c, f);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t c = c0 + 32 * i + lane;
        if (c < a.cols)
          store1<FMT>(a.vals, r * a.ld_vals + c,
                      decode1(codes[c], scale_value(scales[c / kGroup8]), a.int8));
      }
    }
  }
}

template <int FMT>
static cudaError_t launch_act(const Act8Args& a, bool encode, bool wide, int grid,
                              cudaStream_t s) {
  auto k = encode ? (wide ? act_encode_kernel<FMT, true> : act_encode_kernel<FMT, false>)
                  : (wide ? act_decode_kernel<FMT, true> : act_decode_kernel<FMT, false>);
  k<<<grid, 32 * kActWarps, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_act8(Act8Args a, int fmt, bool encode, cudaStream_t s) {
  const int es = fmt_bytes(fmt);
  const bool wide = a.cols % 8 == 0 && (a.rows == 1 || (a.ld_vals * es % 16 == 0 && a.ld_codes % 8 == 0));
  if (wide && a.cols % kGroup8 == 0 && a.ld_vals == a.cols && a.ld_codes == a.cols) {
    // rows back to back and whole groups: one long row, so that no chunk is cut short
    a.cols *= a.rows;
    a.groups = a.cols / kGroup8;
    a.rows = 1;
    a.ld_vals = a.ld_codes = a.cols;
  }
  a.chunks = (a.cols + kChunk8 - 1) / kChunk8;
  const int64_t ctas = (a.rows * a.chunks + kActWarps - 1) / kActWarps;
  const int grid = static_cast<int>(ctas < 148 * 8 ? ctas : 148 * 8);
  switch (fmt) {
    case kFmtBf16: return launch_act<kFmtBf16>(a, encode, wide, grid, s);
    case kFmtF16: return launch_act<kFmtF16>(a, encode, wide, grid, s);
    case kFmtF32: return launch_act<kFmtF32>(a, encode, wide, grid, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace moe
