// 8-bit activation checkpoints: write and read (see act8.cuh for the format).  Both are one
// pass over the data and bound by HBM: bf16 moves 2 + 1 + 1/32 bytes per value each way.
//
// Wide form (every row starts on a 16-byte boundary and holds whole 8-element pieces): a group
// of 32 columns is two neighbouring threads' two pieces each (a pair's accesses fill 32-byte
// sectors), and the groups of all rows are dealt to the thread pairs in turn, so that short
// rows leave no thread idle.  A thread keeps two groups' loads under way (with four 8-warp CTAs an SM 64 KB of 16-bit values, which keeps HBM busy)
// and walks its groups by adding to pointers: at 15 instructions a value, as with a division
// and eight values a thread, the instruction slots and not HBM were the bound.
// Narrow form (any column count or stride): a warp takes chunks of 256 columns of a row, lane l
// columns l, l + 32, ..., so each access of the warp is one group.
#include "act8.cuh"
#include "train_internal.h"

namespace moe {

constexpr int kChunk8 = 256;
constexpr int kActWarps = 8;
constexpr int kEncBatch = 2, kDecBatch = 4;  // groups of a thread under way
constexpr int kActCtas = 4;    // per SM

// A thread pair's groups: every `stride`-th one of all rows' groups.
template <int ES>
struct Groups {
  uint8_t *vals, *codes, *scales;  // the next group's
  int at, groups, at_on;           // its place in the row
  int64_t vals_on, codes_on, stride, left;
  int64_t vals_wrap, codes_wrap;   // added where the place passes the row's end
  __device__ __forceinline__ Groups(const Act8Args& a) {
    stride = static_cast<int64_t>(gridDim.x) * (kActWarps * 16);
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (kActWarps * 16) + (threadIdx.x >> 1);
    const int64_t total = a.rows * a.groups;
    left = first < total ? (total - 1 - first) / stride + 1 : 0;
    groups = static_cast<int>(a.groups);
    const int64_t row = first / a.groups, rows_on = stride / a.groups;
    at = static_cast<int>(first - row * a.groups);
    at_on = static_cast<int>(stride - rows_on * a.groups);
    vals = static_cast<uint8_t*>(a.vals) + (row * a.ld_vals + at * kGroup8) * ES;
    codes = a.codes + row * a.ld_codes + at * kGroup8;
    scales = a.scales + first;
    vals_on = (rows_on * a.ld_vals + at_on * kGroup8) * ES;
    codes_on = rows_on * a.ld_codes + at_on * kGroup8;
    vals_wrap = (a.ld_vals - a.groups * kGroup8) * ES;
    codes_wrap = a.ld_codes - a.groups * kGroup8;
  }
  __device__ __forceinline__ void next() {
    --left;
    at += at_on;
    vals += vals_on;
    codes += codes_on;
    scales += stride;
    if (at >= groups) {
      at -= groups;
      vals += vals_wrap;
      codes += codes_wrap;
    }
  }
};

// Narrow form: a warp's chunks, every `stride`-th one of all rows' chunks, as row and first
// column.
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
  if constexpr (WIDE) {
    constexpr int ES = fmt_bytes(FMT);
    const int mine = 8 * (lane & 1);  // the thread's first column of a group, the other 16 on
    Groups<ES> g(a);
    // the warp's first thread has the most groups; the sums of a pair want the whole warp
    for (int64_t n = __shfl_sync(0xffffffffu, g.left, 0); n > 0; n -= kEncBatch) {
      Raw8<FMT> raw[kEncBatch][2];
      uint8_t *codes[kEncBatch], *scales[kEncBatch];
      int room[kEncBatch];  // columns left from the thread's first
#pragma unroll
      for (int b = 0; b < kEncBatch; ++b) {
        room[b] = g.left > 0 ? static_cast<int>(a.cols) - g.at * kGroup8 - mine : 0;
        codes[b] = g.codes + mine;
        scales[b] = g.scales;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          raw[b][i] = Raw8<FMT>{};
          if (room[b] > 16 * i) raw[b][i] = load_raw8<FMT>(g.vals + mine * ES, 16 * i);
        }
        g.next();
      }
#pragma unroll
      for (int b = 0; b < kEncBatch; ++b) {
        float f[2][8];
        widen8<FMT>(raw[b][0], f[0]);
        widen8<FMT>(raw[b][1], f[1]);
        uint32_t m = max(amax_bits(f[0]), amax_bits(f[1]));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        const int s = scale_byte<INT8>(m);
        const float inv = scale_inverse(s);
        if (room[b] > 0) {
          if (mine == 0) *scales[b] = static_cast<uint8_t>(s);
          *reinterpret_cast<uint2*>(codes[b]) = encode8<INT8>(f[0], inv);
        }
        if (room[b] > 16) *reinterpret_cast<uint2*>(codes[b] + 16) = encode8<INT8>(f[1], inv);
      }
    }
  } else {
    Chunks ch(a);
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

// Values read back, rounded to nearest even.  A code times its scale may be a rounding above
// the format's largest finite value (fp16: 65504 is kept as 64 2^10): 16-bit formats take that
// largest value for anything past it, so that what was finite stays finite.  NaN stays NaN.
template <int FMT>
__device__ __forceinline__ uint32_t pack2_finite(float a, float b) {
  uint32_t r;
  if constexpr (FMT == kFmtF16)
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  else
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
template <int FMT>
__device__ __forceinline__ void store8_finite(void* base, int64_t i, const float (&f)[8]) {
  if constexpr (FMT == kFmtF32)
    store8<FMT>(base, i, f);
  else
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + i) =
        make_uint4(pack2_finite<FMT>(f[0], f[1]), pack2_finite<FMT>(f[2], f[3]),
                   pack2_finite<FMT>(f[4], f[5]), pack2_finite<FMT>(f[6], f[7]));
}
template <int FMT>
__device__ __forceinline__ void store1_finite(void* base, int64_t i, float f) {
  if constexpr (FMT == kFmtF32)
    store1<FMT>(base, i, f);
  else
    static_cast<uint16_t*>(base)[i] = static_cast<uint16_t>(pack2_finite<FMT>(f, 0.f));
}

template <int FMT, bool WIDE, bool INT8>
__global__ void __launch_bounds__(32 * kActWarps, kActCtas) act_decode_kernel(Act8Args a) {
  const int lane = threadIdx.x & 31;
  if constexpr (WIDE) {
    constexpr int ES = fmt_bytes(FMT);
    const int mine = 8 * (lane & 1);  // the thread's first column of a group, the other 16 on
    Groups<ES> g(a);
    while (g.left > 0) {
      uint2 w[kDecBatch][2];
      uint8_t* vals[kDecBatch];
      int room[kDecBatch], s[kDecBatch];
#pragma unroll
      for (int b = 0; b < kDecBatch; ++b) {
        room[b] = g.left > 0 ? static_cast<int>(a.cols) - g.at * kGroup8 - mine : 0;
        vals[b] = g.vals + mine * ES;
        s[b] = room[b] > 0 ? *g.scales : 1;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          w[b][i] = room[b] > 16 * i ? *reinterpret_cast<const uint2*>(g.codes + mine + 16 * i)
                                    : make_uint2(0u, 0u);
        g.next();
      }
#pragma unroll
      for (int b = 0; b < kDecBatch; ++b) {
        const float scale = scale_value(s[b]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float f[8];
          decode8<INT8>(w[b][i], scale, f);
          if (room[b] > 16 * i) store8_finite<FMT>(vals[b], 16 * i, f);
        }
      }
    }
  } else {
    Chunks ch(a);
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
        if (c < a.cols) store1_finite<FMT>(a.vals, r * a.ld_vals + c, f[i]);
      }
    }
  }
}

template <int FMT, bool INT8>
static cudaError_t launch_act(const Act8Args& a, bool encode, bool wide, int grid,
                              cudaStream_t s) {
  auto k = encode ? (wide ? act_encode_kernel<FMT, true, INT8> : act_encode_kernel<FMT, false, INT8>)
                  : (wide ? act_decode_kernel<FMT, true, INT8> : act_decode_kernel<FMT, false, INT8>);
  return launch_k(k, dim3(static_cast<unsigned>(grid)), dim3(32 * kActWarps), 0, s, false, a);
}

cudaError_t launch_act8(Act8Args a, int fmt, bool encode, cudaStream_t s) {
  const int es = fmt_bytes(fmt);
  const bool wide = a.cols % 8 == 0 && (a.rows == 1 || (a.ld_vals * es % 16 == 0 && a.ld_codes % 8 == 0));
  if (a.rows == 1) a.ld_vals = a.ld_codes = a.cols;
  a.chunks = (a.cols + kChunk8 - 1) / kChunk8;
  const int64_t ctas = wide ? (a.rows * a.groups + kActWarps * 16 - 1) / (kActWarps * 16)
                            : (a.rows * a.chunks + kActWarps - 1) / kActWarps;
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
