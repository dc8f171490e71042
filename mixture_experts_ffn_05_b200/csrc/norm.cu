// RMS norm and layer norm over rows, forward and backward, with the 8-bit checkpoint of the
// input written or read in the same pass.
//
// A team of TPR threads (whole warps) holds one row in registers, NV pieces of 8 elements a
// thread, so x is read once although the statistics need it twice; R = 4 / NV rows are in
// flight per team and share one round of reductions.  The kernels are bound by HBM: forward
// reads x and writes y, backward reads x (2, 4 or 1 + 1/32 bytes) and dy and writes dx.
// Wide form: thread t's piece i is columns 8 (t + i TPR) ... + 7.  Narrow form (columns,
// strides that no 16-byte access fits): element e of piece i is column t + (8 i + e) TPR, so
// a warp's accesses stay contiguous.  In both a group of 32 columns lies in 4 lanes or in one
// warp, where the checkpoint's scale is formed.
//
// The gradients of gain and bias are sums over all rows: a thread owns its columns for the
// whole kernel and adds its rows in registers, the teams of a CTA meet in shared memory, each
// CTA writes one row of partial sums, and a second small launch adds those in CTA order
// (deterministic; a single CTA writes the result itself).
#include "act8.cuh"
#include "train_internal.h"

namespace moe {

struct NormShape {
  int nv, tpr, teams;
};

// Pieces a thread, threads a row, rows side by side in a CTA.
static NormShape norm_shape(int cols) {
  const int pieces = (cols + 7) / 8;
  NormShape s;
  s.nv = pieces <= 512 ? 1 : pieces <= 1024 ? 2 : 4;
  s.tpr = ((pieces + s.nv - 1) / s.nv + 31) / 32 * 32;
  s.teams = s.tpr >= 256 ? 1 : 256 / s.tpr;
  return s;
}

// Sums of N values over a team; every thread of the CTA calls it.  buf: two halves of
// [warps][N] floats used in turn, so that one barrier per call is enough.
template <int N>
__device__ __forceinline__ void team_sum(float (&v)[N], float* buf, int tpr, int team) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (tpr == 32) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) buf[warp * N + i] = v[i];
  }
  __syncthreads();
  const int w0 = team * (tpr >> 5), nw = tpr >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
  for (int w = 0; w < nw; ++w) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += buf[(w0 + w) * N + i];
  }
}

constexpr int kNormMaxWarps = 16;

// Where a thread's elements lie.
template <bool WIDE>
struct Cols {
  int t, tpr;
  __device__ __forceinline__ int first(int i) const {  // wide: the piece's first column
    return 8 * (t + i * tpr);
  }
  __device__ __forceinline__ int at(int i, int e) const {
    return WIDE ? 8 * (t + i * tpr) + e : t + (8 * i + e) * tpr;
  }
};

template <int FMT, bool WIDE>
struct Piece {
  Raw8<FMT> raw;
};
template <int FMT>
struct Piece<FMT, false> {
  float f[8];
};

template <int FMT, bool WIDE>
__device__ __forceinline__ void load_piece(Piece<FMT, WIDE>& p, const void* base, int64_t row0,
                                           const Cols<WIDE>& c, int i, int cols, bool live) {
  if constexpr (WIDE) {
    p.raw = Raw8<FMT>{};
    if (live && c.first(i) < cols) p.raw = load_raw8<FMT>(base, row0 + c.first(i));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      p.f[e] = live && c.at(i, e) < cols ? load1<FMT>(base, row0 + c.at(i, e)) : 0.f;
  }
}

template <int FMT, bool WIDE>
__device__ __forceinline__ void widen_piece(const Piece<FMT, WIDE>& p, float (&f)[8]) {
  if constexpr (WIDE) {
    widen8<FMT>(p.raw, f);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = p.f[e];
  }
}

template <int FMT, bool WIDE>
__device__ __forceinline__ void store_piece(void* base, int64_t row0, const Cols<WIDE>& c, int i,
                                            int cols, const float (&f)[8]) {
  if constexpr (WIDE) {
    if (c.first(i) < cols) store8<FMT>(base, row0 + c.first(i), f);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c.at(i, e) < cols) store1<FMT>(base, row0 + c.at(i, e), f[e]);
  }
}

template <bool WIDE>
__device__ __forceinline__ void load_param(float (&f)[8], const void* p, int fmt,
                                           const Cols<WIDE>& c, int i, int cols, float absent) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    f[e] = p != nullptr && c.at(i, e) < cols ? load1_any(p, c.at(i, e), fmt) : absent;
}

// ---------------------------------------------------------------- forward
template <int FMT, int NV, bool WIDE, bool LAYER>
__global__ void __launch_bounds__(512) norm_forward_kernel(NormArgs a, int tpr, int teams) {
  constexpr int R = 4 / NV;
  __shared__ float red[4][kNormMaxWarps * R];
  const int team = threadIdx.x / tpr;
  const Cols<WIDE> c{static_cast<int>(threadIdx.x) - team * tpr, tpr};
  const int cols = a.cols;
  const float inv_n = 1.f / static_cast<float>(cols);
  const int64_t groups = (cols + kGroup8 - 1) / kGroup8;
  const int lane = threadIdx.x & 31;
  float g[NV][8], b[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load_param<WIDE>(g[i], a.gain, a.pfmt, c, i, cols, 1.f);
    load_param<WIDE>(b[i], a.bias, a.pfmt, c, i, cols, 0.f);
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * teams * R;
  int turn = 0;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * teams * R; base < a.T; base += step) {
    const int64_t r0 = base + team * R;
    Piece<FMT, WIDE> raw[R][NV];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < NV; ++i)
        load_piece(raw[r][i], a.x, (r0 + r) * a.ldx, c, i, cols, r0 + r < a.T);
    float mean[R] = {}, var[R] = {};
    if (LAYER) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          float f[8];
          widen_piece(raw[r][i], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) mean[r] += f[e];
        }
      team_sum<R>(mean, red[turn], tpr, team);
#pragma unroll
      for (int r = 0; r < R; ++r) mean[r] *= inv_n;
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float f[8];
        widen_piece(raw[r][i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float d = LAYER ? (c.at(i, e) < cols ? f[e] - mean[r] : 0.f) : f[e];
          var[r] = fmaf(d, d, var[r]);
        }
      }
    team_sum<R>(var, red[2 + turn], tpr, team);
    turn ^= 1;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = r0 + r;
      const bool live = row < a.T;
      const float rstd = 1.f / sqrtf(fmaf(var[r], inv_n, a.eps));
      if (live && c.t == 0) {
        a.rstd[row] = rstd;
        if (LAYER) a.mean[row] = mean[r];
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float f[8], y[8];
        widen_piece(raw[r][i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float z = (LAYER ? f[e] - mean[r] : f[e]) * rstd;
          y[e] = LAYER ? fmaf(z, g[i][e], b[i][e]) : z * g[i][e];
        }
        if (a.codes != nullptr) {  // uniform; every lane takes part in the groups' maxima
          if constexpr (WIDE) {
            uint32_t m = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) m = max(m, abs_bits(f[e]));
            const int sb = scale_byte(max4_lanes(m), a.int8);
            const int col = c.first(i);
            if (live && col < cols) {
              if ((lane & 3) == 0) a.code_scales[row * groups + col / kGroup8] = static_cast<uint8_t>(sb);
              *reinterpret_cast<uint2*>(a.codes + row * a.ld_codes + col) =
                  encode8(f, scale_inverse(sb), a.int8);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int sb = scale_byte(__reduce_max_sync(0xffffffffu, abs_bits(f[e])), a.int8);
              const int col = c.at(i, e);
              if (live && col < cols) {
                if (lane == 0) a.code_scales[row * groups + col / kGroup8] = static_cast<uint8_t>(sb);
                a.codes[row * a.ld_codes + col] =
                    static_cast<uint8_t>(encode1(f[e], scale_inverse(sb), a.int8));
              }
            }
          }
        }
        if (live) store_piece<FMT, WIDE>(a.out, row * a.ldo, c, i, cols, y);
      }
    }
  }
}

// ---------------------------------------------------------------- backward
// One row's x pieces as loaded: the activation's format or 8-bit codes with their scale.
template <int FMT, bool WIDE, bool X8>
struct XPiece {
  Piece<FMT, WIDE> p;
};
template <int FMT>
struct XPiece<FMT, true, true> {
  uint2 codes;
  int byte;
};

template <int FMT, int NV, bool WIDE, bool LAYER, bool X8>
__global__ void __launch_bounds__(512) norm_backward_kernel(NormArgs a, int tpr, int teams) {
  constexpr int R = NV == 1 ? 2 : 1;
  __shared__ float red[2][kNormMaxWarps * 2 * R];
  extern __shared__ float teamsum[];  // [teams][cols], teams > 1 only
  pdl_trigger();
  const int team = threadIdx.x / tpr;
  const Cols<WIDE> c{static_cast<int>(threadIdx.x) - team * tpr, tpr};
  const int cols = a.cols;
  const float inv_n = 1.f / static_cast<float>(cols);
  const int64_t groups = (cols + kGroup8 - 1) / kGroup8;
  float g[NV][8], dg[NV][8], db[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load_param<WIDE>(g[i], a.gain, a.pfmt, c, i, cols, 1.f);
#pragma unroll
    for (int e = 0; e < 8; ++e) dg[i][e] = db[i][e] = 0.f;
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * teams * R;
  int turn = 0;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * teams * R; base < a.T; base += step) {
    const int64_t r0 = base + team * R;
    XPiece<FMT, WIDE, X8> xr[R][NV];
    Piece<FMT, WIDE> dyr[R][NV];
    float mean[R], rstd[R], s[2 * R] = {};
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = r0 + r;
      const bool live = row < a.T;
      mean[r] = LAYER && live ? a.mean[row] : 0.f;
      rstd[r] = live ? a.rstd[row] : 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        load_piece(dyr[r][i], a.dy, row * a.lddy, c, i, cols, live);
        if constexpr (!X8) {
          load_piece(xr[r][i].p, a.x, row * a.ldx, c, i, cols, live);
        } else if constexpr (WIDE) {
          xr[r][i].codes = make_uint2(0u, 0u);
          xr[r][i].byte = 1;
          if (live && c.first(i) < cols) {
            xr[r][i].codes = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.x) +
                                                             row * a.ldx + c.first(i));
            xr[r][i].byte = a.x_scales[row * groups + c.first(i) / kGroup8];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int col = c.at(i, e);
            xr[r][i].p.f[e] =
                live && col < cols
                    ? decode1(static_cast<const uint8_t*>(a.x)[row * a.ldx + col],
                              scale_value(a.x_scales[row * groups + col / kGroup8]), a.int8)
                    : 0.f;
          }
        }
      }
    }
    auto x_of = [&](int r, int i, float (&f)[8]) {
      if constexpr (X8 && WIDE)
        decode8(xr[r][i].codes, scale_value(xr[r][i].byte), a.int8, f);
      else
        widen_piece(xr[r][i].p, f);
    };
    // sums of a z and (layer) of a, and this thread's share of the parameter gradients:
    // dead rows and columns have dy = 0 and, rstd being 0 or x finite, add nothing
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float xf[8], df[8];
        x_of(r, i, xf);
        widen_piece(dyr[r][i], df);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float z = (xf[e] - mean[r]) * rstd[r];
          const float av = df[e] * g[i][e];
          s[2 * r] = fmaf(av, z, s[2 * r]);
          if (LAYER) {
            s[2 * r + 1] += av;
            db[i][e] += df[e];
          }
          dg[i][e] = fmaf(df[e], z, dg[i][e]);
        }
      }
    team_sum<2 * R>(s, red[turn], tpr, team);
    turn ^= 1;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = r0 + r;
      if (row >= a.T) continue;
      const float c1 = s[2 * r] * inv_n, c2 = LAYER ? s[2 * r + 1] * inv_n : 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float xf[8], df[8], o[8];
        x_of(r, i, xf);
        widen_piece(dyr[r][i], df);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float z = (xf[e] - mean[r]) * rstd[r];
          o[e] = rstd[r] * (df[e] * g[i][e] - c2 - z * c1);
        }
        store_piece<FMT, WIDE>(a.out, row * a.ldo, c, i, cols, o);
      }
    }
  }
  // ---- the CTA's sums of the parameter gradients
  const bool single = gridDim.x == 1;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* fin = which == 0 ? a.d_gain : a.d_bias;
    if (fin == nullptr) continue;  // uniform
    float* dst = single ? fin
                        : a.partials + (static_cast<int64_t>(blockIdx.x) * 2 + which) * cols;
    const bool add = single && a.accumulate;
    if (teams > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c.at(i, e) < cols) teamsum[team * cols + c.at(i, e)] = which == 0 ? dg[i][e] : db[i][e];
      __syncthreads();
      for (int col = threadIdx.x; col < cols; col += blockDim.x) {
        float v = add ? dst[col] : 0.f;
        for (int k = 0; k < teams; ++k) v += teamsum[k * cols + col];
        dst[col] = v;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int col = c.at(i, e);
          if (col < cols) dst[col] = (which == 0 ? dg[i][e] : db[i][e]) + (add ? dst[col] : 0.f);
        }
    }
  }
}

// out[col] (+)= the sum of the partial rows, in row order per lane and then over 16 lanes.
constexpr int kRedCols = 32, kRedLanes = 16;
__global__ void __launch_bounds__(kRedCols * kRedLanes) norm_reduce_kernel(
    const float* __restrict__ partials, int rows, int cols, float* d_gain, float* d_bias,
    int accumulate) {
  __shared__ float s[kRedLanes][kRedCols];
  pdl_wait();
  const int which = blockIdx.y;
  float* out = which == 0 ? d_gain : d_bias;
  if (out == nullptr) return;
  const int cx = threadIdx.x % kRedCols, ly = threadIdx.x / kRedCols;
  const int col = blockIdx.x * kRedCols + cx;
  float v = 0.f;
  if (col < cols)
    for (int r = ly; r < rows; r += kRedLanes)
      v += partials[(static_cast<int64_t>(r) * 2 + which) * cols + col];
  s[ly][cx] = v;
  __syncthreads();
  if (ly == 0 && col < cols) {
    v = accumulate ? out[col] : 0.f;
#pragma unroll
    for (int k = 0; k < kRedLanes; ++k) v += s[k][cx];
    out[col] = v;
  }
}

// ---------------------------------------------------------------- launches
static int norm_rows_per_cta(const NormShape& sh, int rows_per_team) {
  return sh.teams * rows_per_team;
}

// About 1024 threads an SM: enough bytes in flight, and few partial rows.
static int norm_ctas_per_sm(const NormShape& sh) {
  const int threads = sh.tpr * sh.teams;
  return threads >= 1024 ? 1 : 1024 / threads;
}

int norm_backward_ctas(int T, int cols) {
  const NormShape sh = norm_shape(cols);
  const int64_t rows = norm_rows_per_cta(sh, sh.nv == 1 ? 2 : 1);
  const int64_t need = (static_cast<int64_t>(T) + rows - 1) / rows;
  const int64_t most = static_cast<int64_t>(kB200Sms) * norm_ctas_per_sm(sh);
  return static_cast<int>(need < most ? need : most);
}

template <int FMT, bool WIDE, bool LAYER>
static cudaError_t forward_nv(const NormArgs& a, const NormShape& sh, cudaStream_t s) {
  const int64_t rows = norm_rows_per_cta(sh, 4 / sh.nv);
  const int64_t need = (static_cast<int64_t>(a.T) + rows - 1) / rows;
  const int64_t most = static_cast<int64_t>(kB200Sms) * 2 * norm_ctas_per_sm(sh);
  const int grid = static_cast<int>(need < most ? need : most);
  auto k = sh.nv == 1   ? norm_forward_kernel<FMT, 1, WIDE, LAYER>
           : sh.nv == 2 ? norm_forward_kernel<FMT, 2, WIDE, LAYER>
                        : norm_forward_kernel<FMT, 4, WIDE, LAYER>;
  return launch_k(k, dim3(grid), dim3(sh.tpr * sh.teams), 0, s, false, a, sh.tpr, sh.teams);
}

template <int FMT>
static cudaError_t forward_fmt(const NormArgs& a, cudaStream_t s) {
  const NormShape sh = norm_shape(a.cols);
  const int es = fmt_bytes(FMT);
  const bool wide = a.cols % 8 == 0 && a.ldx * es % 16 == 0 && a.ldo * es % 16 == 0 &&
                    (a.codes == nullptr || a.ld_codes % 8 == 0);
  if (a.layer)
    return wide ? forward_nv<FMT, true, true>(a, sh, s) : forward_nv<FMT, false, true>(a, sh, s);
  return wide ? forward_nv<FMT, true, false>(a, sh, s) : forward_nv<FMT, false, false>(a, sh, s);
}

cudaError_t launch_norm_forward(const NormArgs& a, int fmt, cudaStream_t s) {
  switch (fmt) {
    case kFmtBf16: return forward_fmt<kFmtBf16>(a, s);
    case kFmtF16: return forward_fmt<kFmtF16>(a, s);
    case kFmtF32: return forward_fmt<kFmtF32>(a, s);
  }
  return cudaErrorInvalidValue;
}

template <int FMT, bool WIDE, bool LAYER, bool X8>
static cudaError_t backward_nv(const NormArgs& a, const NormShape& sh, cudaStream_t s) {
  const int grid = norm_backward_ctas(a.T, a.cols);
  const size_t smem = sh.teams > 1 ? static_cast<size_t>(sh.teams) * a.cols * sizeof(float) : 0;
  auto k = sh.nv == 1   ? norm_backward_kernel<FMT, 1, WIDE, LAYER, X8>
           : sh.nv == 2 ? norm_backward_kernel<FMT, 2, WIDE, LAYER, X8>
                        : norm_backward_kernel<FMT, 4, WIDE, LAYER, X8>;
  cudaError_t e =
      launch_k(k, dim3(grid), dim3(sh.tpr * sh.teams), smem, s, false, a, sh.tpr, sh.teams);
  if (e != cudaSuccess || grid == 1 || (a.d_gain == nullptr && a.d_bias == nullptr)) return e;
  return launch_k(norm_reduce_kernel,
                  dim3((a.cols + kRedCols - 1) / kRedCols, a.d_bias != nullptr ? 2 : 1),
                  dim3(kRedCols * kRedLanes), 0, s, true, a.partials, grid, a.cols, a.d_gain,
                  a.d_bias, a.accumulate);
}

template <int FMT, bool X8>
static cudaError_t backward_fmt(const NormArgs& a, cudaStream_t s) {
  const NormShape sh = norm_shape(a.cols);
  const int es = fmt_bytes(FMT);
  const bool wide = a.cols % 8 == 0 && (X8 ? a.ldx % 8 == 0 : a.ldx * es % 16 == 0) &&
                    a.ldo * es % 16 == 0 && a.lddy * es % 16 == 0;
  if (a.layer)
    return wide ? backward_nv<FMT, true, true, X8>(a, sh, s)
                : backward_nv<FMT, false, true, X8>(a, sh, s);
  return wide ? backward_nv<FMT, true, false, X8>(a, sh, s)
              : backward_nv<FMT, false, false, X8>(a, sh, s);
}

cudaError_t launch_norm_backward(const NormArgs& a, int fmt, int xfmt, cudaStream_t s) {
  const bool x8 = xfmt == kFmtInt8 || xfmt == kFmtE4m3;
  switch (fmt) {
    case kFmtBf16: return x8 ? backward_fmt<kFmtBf16, true>(a, s) : backward_fmt<kFmtBf16, false>(a, s);
    case kFmtF16: return x8 ? backward_fmt<kFmtF16, true>(a, s) : backward_fmt<kFmtF16, false>(a, s);
    case kFmtF32: return x8 ? backward_fmt<kFmtF32, true>(a, s) : backward_fmt<kFmtF32, false>(a, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace moe
