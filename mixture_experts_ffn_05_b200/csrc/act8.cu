// 8-bit activation checkpoints: write and read (see act8.cuh for the format).  Both are one
// pass over the data and bound by HBM: bf16 moves 2 + 1 + 1/32 bytes per value each way.
//
// A warp takes chunks of 256 columns of a row, four at a time, so that a thread has four loads
// under way (at 32 warps an SM 64 KB of 16-bit values, with which reads keep HBM busy).  Wide
// form (every row starts on a 16-byte boundary and holds whole 8-element pieces): lane l owns
// columns 8l..8l+7 of the chunk, so a group of 32 is four neighbouring lanes.  Narrow form (any
// column count or stride): lane l owns columns l, l + 32, ..., so each access of the warp is
// one group of 32 consecutive elements.  Groups never cross a row.
#include "act8.cuh"
#include "train_internal.h"

namespace moe {

constexpr int kChunk8 = 256;
constexpr int kActWarps = 8;
constexpr int kActBatch = 4;   // chunks of a warp under way
constexpr int kActCtas = 4;    // per SM

// A warp's chunks: every `stride`-th one of all rows' chunks, as row and first column.
struct Chunks {
  int64_t left, row, at;      // chunks left; the next one's row and place in it
  int64_t rows_on, at_on, per_row;
  __device__ __forceinline__ Chunks(const Act8Args& a) {
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kActWarps + (threadIdx.x >> 5);
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kActWarps;
    const int64_t items = a.rows * a.chunks;
    per_row = a.chunks;
    left = first < items ? (items - 1 - first) / stride + 1 : 0;
    row = first / per_row;
    at = first - row * per_row;
    rows_on = stride / per_row;
    at_on = stride - rows_on * per_row;
  }
  __device__ __forceinline__ bool take(int64_t& r, int64_t& c0) {
    r = row;
    c0 = at * kChunk8;
    row += rows_on;
    at += at_on;
    if (at >= per_row) {
      at -= per_row;
      ++row;
    }
    return left-- > 0;
  }
};

template <int FMT, bool WIDE, bool INT8>
__global__ void __launch_bounds__(32 * kActWarps, kActCtas) act_encode_kernel(Act8Args a) {
  const int lane = threadIdx.x & 31;
  Chunks ch(a);
  if constexpr (WIDE) {
    while (ch.left > 0) {
      Raw8<FMT> raw[kActBatch];
      int64_t row[kActBatch], col[kActBatch];
#pragma unroll
      for (int b = 0; b < kActBatch; ++b) {
        const bool in = ch.take(row[b], col[b]);
        col[b] += 8 * lane;
        if (!in) col[b] = a.cols;
        raw[b] = Raw8<FMT>{};
        if (col[b] < a.cols) raw[b] = load_raw8<FMT>(a.vals, row[b] * a.ld_vals + col[b]);
      }
#pragma unroll
      for (int b = 0; b < kActBatch; ++b) {
        float f[8];
        widen8<FMT>(raw[b], f);
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, abs_bits(f[i]));
        const int s = scale_byte<INT8>(max4_lanes(m));
        if (col[b] < a.cols) {
          if ((lane & 3) == 0)
            a.scales[row[b] * a.groups + col[b] / kGroup8] = static_cast<uint8_t>(s);
          *reinterpret_cast<uint2*>(a.codes + row[b] * a.ld_codes + col[b]) =
              encode8<INT8>(f, scale_inverse(s));
        }
      }
    }
  } else {
    int64_t r, c0;
    while (ch.take(r, c0)) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t c = c0 + 32 * i + lane;
        f[i] = c < a.cols ? load1<FMT>(a.vals, r * a.ld_vals + c) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t c = c0 + 32 * i + lane;
        const int b = scale_byte<INT8>(__reduce_max_sync(0xffffffffu, abs_bits(f[i])));
        if (c < a.cols) {
          if (lane == 0) a.scales[r * a.groups + c / kGroup8] = static_cast<uint8_t>(b);
          a.codes[r * a.ld_codes + c] = static_cast<uint8_t>(encode1<INT8>(f[i], scale_inverse(b)));
        }
      }
    }
  }
}

template <int FMT, bool WIDE, bool INT8>
__global__ void __launch_bounds__(32 * kActWarps, kActCtas) act_decode_kernel(Act8Args a) {
  const int lane = threadIdx.x & 31;
  Chunks ch(a);
  if constexpr (WIDE) {
    while (ch.left > 0) {
      uint2 w[kActBatch];
      int s[kActBatch];
      int64_t row[kActBatch], col[kActBatch];
#pragma unroll
      for (int b = 0; b < kActBatch; ++b) {
        const bool in = ch.take(row[b], col[b]);
        col[b] += 8 * lane;
        if (!in) col[b] = a.cols;
        w[b] = make_uint2(0u, 0u);
        s[b] = 1;
        if (col[b] < a.cols) {
          w[b] = *reinterpret_cast<const uint2*>(a.codes + row[b] * a.ld_codes + col[b]);
          s[b] = a.scales[row[b] * a.groups + col[b] / kGroup8];
        }
      }
#pragma unroll
      for (int b = 0; b < kActBatch; ++b) {
        float f[8];
        decode8<INT8>(w[b], scale_value(s[b]), f);
        if (col[b] < a.cols) store8<FMT>(a.vals, row[b] * a.ld_vals + col[b], f);
      }
    }
  } else {
    int64_t r, c0;
    while (ch.take(r, c0)) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t c = c0 + 32 * i + lane;
        f[i] = 0.f;
        if (c < a.cols)
          f[i] = decode1<INT8>(a.codes[r * a.ld_codes + c],
                               scale_value(a.scales[r * a.groups + c / kGroup8]));
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t c = c0 + 32 * i + lane;
        if (c < a.cols) store1<FMT>(a.vals, r * a.ld_vals + c, f[i]);
      }
    }
  }
}

template <int FMT, bool INT8>
static cudaError_t launch_act(const Act8Args& a, bool encode, bool wide, int grid,
                              cudaStream_t s) {
  auto k = encode ? (wide ? act_encode_kernel<FMT, true, INT8> : act_encode_kernel<FMT, false, INT8>)
                  : (wide ? act_decode_kernel<FMT, true, INT8> : act_decode_kernel<FMT, false, INT8>);
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
  const int most = kB200Sms * kActCtas;
  const int grid = static_cast<int>(ctas < most ? ctas : most);
  switch (fmt) {
    case kFmtBf16:
      return a.int8 ? launch_act<kFmtBf16, true>(a, encode, wide, grid, s)
                    : launch_act<kFmtBf16, false>(a, encode, wide, grid, s);
    case kFmtF16:
      return a.int8 ? launch_act<kFmtF16, true>(a, encode, wide, grid, s)
                    : launch_act<kFmtF16, false>(a, encode, wide, grid, s);
    case kFmtF32:
      return a.int8 ? launch_act<kFmtF32, true>(a, encode, wide, grid, s)
                    : launch_act<kFmtF32, false>(a, encode, wide, grid, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace moe
