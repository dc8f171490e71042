// RMS norm and layer norm over rows, forward and backward, with the 8-bit checkpoint of the
// input written or read in the same pass.
//
// A team of W warps holds one row, NV times 8 elements a thread, so x is read from memory once
// although the statistics need it twice.  The teams of a CTA work on rows of their own and
// meet at named barriers of their own.  The kernels are bound by HBM: forward reads x and
// writes y, backward reads x (2, 4 or 1 + 1/32 bytes) and dy and writes dx.  Rows come through
// a ring in shared memory that cp.async fills up to four rows ahead, which keeps 50 to 200 KB
// of loads in flight per SM without registers and whatever phase the teams are in.
//
// Wide form (columns, strides and bases that 16-byte accesses fit): a thread owns units of 16
// bytes of the activation's format, U = 8 or 4 columns, unit u at column U (t + 32 W u); it
// reads back only the units that it copied itself, so the ring needs no barrier.  Narrow form
// (any other): the row is copied as the aligned 16-byte chunks that cover it, and element j is
// column t + 32 W j, so that a warp's accesses stay contiguous.  In both a group of 32 columns
// lies within one warp, where the checkpoint's scale is formed.
//
// The gradients of gain and bias are sums over all rows: a thread owns its columns for the
// whole kernel and adds its rows in registers, the teams of a CTA meet in shared memory, each
// CTA writes one row of partial sums, and a second small launch adds those in a fixed order
// (deterministic; a single CTA writes the result itself).
#include "act8.cuh"
#include "train_internal.h"

namespace moe {

// Rows of up to 12 warps of 8 (16) elements a thread; longer ones take 32 elements a thread of
// 16 warps, where 128 registers hold no more (the sums of the gradients spill there).
__host__ __device__ constexpr int norm_threads(int nv) { return nv == 4 ? 512 : 384; }
__host__ __device__ constexpr int norm_ctas_per_sm(int nv) { return nv == 1 ? 2 : 1; }
constexpr int kNormMaxWarps = 16;
constexpr int kNormRingBytes = 200 * 1024;  // per SM

struct NormShape {
  int nv, warps, teams;  // 8-element pieces a thread, warps a row, rows side by side in a CTA
};

static NormShape norm_shape(int cols, int64_t T) {
  const int w1 = (cols + 255) / 256;  // warps of 8 elements a thread
  NormShape s;
  s.nv = w1 <= 12 ? 1 : w1 <= 24 ? 2 : 4;
  s.warps = (w1 + s.nv - 1) / s.nv;
  s.teams = norm_threads(s.nv) / 32 / s.warps;
  const int64_t ctas = static_cast<int64_t>(kB200Sms) * norm_ctas_per_sm(s.nv);
  const int64_t need = (T + ctas - 1) / ctas;  // few rows: spread over the SMs first
  if (need < s.teams) s.teams = static_cast<int>(need);
  return s;
}

// Ring bytes that a row's slot takes (16 more than the row: the narrow form's shift).
__host__ __device__ constexpr int norm_slot(int cols, int es) {
  return (cols * es + 15) / 16 * 16 + 16;
}
// Ring depth in rows: at most 4, and what the SM's shared memory holds.
__host__ __device__ constexpr int norm_stages(int nv, int bytes) {
  const int row = norm_threads(nv) * nv * 8 * bytes * norm_ctas_per_sm(nv);
  const int n = kNormRingBytes / row;
  return n > 4 ? 4 : n < 1 ? 1 : n;
}

// ---- asynchronous copies of 4, 8 or 16 bytes into shared memory
template <int BYTES>
__device__ __forceinline__ void cp_async(void* dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES)
                 : "memory");
}
// The first n of 16 bytes, the rest as zeros.
__device__ __forceinline__ void cp_async_part(void* dst, const void* src, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int FMT, int NV, bool WIDE>
struct NormThread {
  static constexpr int E = 8 * NV;              // elements a thread
  static constexpr int ES = fmt_bytes(FMT);
  static constexpr int U = WIDE ? 16 / ES : 1;  // columns of a unit
  static constexpr int NU = E / U;
  int t, tpr, warps, wt, lane, team, cols;
  float* red;  // the team's two buffers of a warp's sums
  int turn;

  __device__ __forceinline__ NormThread(int w, int n, float* buf) {
    tpr = 32 * w;
    warps = w;
    team = static_cast<int>(threadIdx.x) / tpr;
    t = static_cast<int>(threadIdx.x) - team * tpr;
    wt = t >> 5;
    lane = t & 31;
    cols = n;
    red = buf + team * w * 2;
    turn = 0;
  }
  __device__ __forceinline__ int unit(int u) const { return U * (t + u * tpr); }
  __device__ __forceinline__ int col(int j) const { return unit(j / U) + j % U; }

  __device__ __forceinline__ void sync() const {
    if (warps == 1)
      __syncwarp();
    else
      named_sync(1 + team, tpr);
  }

  // Sums of N <= 2 values over the team.  The buffers alternate: one is written again only
  // after the barrier of the sum in between.
  template <int N>
  __device__ __forceinline__ void sum(float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
    if (warps == 1) return;
    float* buf = red + turn * (kNormMaxWarps * 2);
    turn ^= 1;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) buf[wt * N + i] = v[i];
    }
    sync();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
    for (int w = 0; w < warps; ++w)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += buf[w * N + i];
  }

  // Gain or bias, `absent` without one.
  __device__ __forceinline__ void param(float (&f)[E], const void* p, int fmt, float absent) const {
#pragma unroll
    for (int j = 0; j < E; ++j) f[j] = p != nullptr && col(j) < cols ? load1_any(p, col(j), fmt) : absent;
  }

  __device__ __forceinline__ void store(void* base, int64_t row0, const float (&f)[E]) const {
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      if (unit(u) >= cols) continue;
      if constexpr (!WIDE) {
        store1<FMT>(base, row0 + unit(u), f[u]);
      } else if constexpr (FMT == kFmtF32) {
        *reinterpret_cast<float4*>(static_cast<float*>(base) + row0 + unit(u)) =
            make_float4(f[4 * u], f[4 * u + 1], f[4 * u + 2], f[4 * u + 3]);
      } else {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = f[8 * u + e];
        store8<FMT>(base, row0 + unit(u), v);
      }
    }
  }

  // ---- the ring.  XF: the format in memory, FMT or 8-bit codes.
  template <int XF>
  __device__ __forceinline__ void request(uint8_t* slot, const void* base, int64_t row0) const {
    constexpr int XS = fmt_bytes(XF);
    const uint8_t* src = static_cast<const uint8_t*>(base) + row0 * XS;
    if constexpr (WIDE) {
#pragma unroll
      for (int u = 0; u < NU; ++u)
        if (unit(u) < cols) cp_async<U * XS>(slot + unit(u) * XS, src + unit(u) * XS);
    } else {
      const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15);
      const int end = shift + cols * XS;  // nothing behind the row is read
      for (int c = 16 * t; c < end; c += 16 * tpr) cp_async_part(slot + c, src - shift + c, min(16, end - c));
    }
  }

  // The row in the slot, its columns past the end as zeros.  8-bit codes: `byte` holds the
  // scale bytes of the warp's E groups, one a lane (see scale_bytes).
  template <int XF>
  __device__ __forceinline__ void read(float (&f)[E], const uint8_t* slot, const void* base,
                                       int64_t row0, int byte, bool int8) const {
    constexpr int XS = fmt_bytes(XF);
    if constexpr (!WIDE)
      slot += reinterpret_cast<uintptr_t>(static_cast<const uint8_t*>(base) + row0 * XS) & 15;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const bool in = unit(u) < cols;
      float scale = 0.f;
      if constexpr (XS == 1)
        scale = scale_value(__shfl_sync(0xffffffffu, byte, WIDE ? u * U + lane * U / 32 : u));
#pragma unroll
      for (int e = 0; e < U; ++e) f[U * u + e] = 0.f;
      if (!in) continue;
      const uint8_t* at = slot + unit(u) * XS;
      if constexpr (!WIDE) {
        if constexpr (XS == 1)
          f[u] = decode1(*at, scale, int8);
        else
          f[u] = load1<XF>(at, 0);
      } else if constexpr (XS == 1) {
#pragma unroll
        for (int k = 0; k < U / 4; ++k)
          decode4(*reinterpret_cast<const uint32_t*>(at + 4 * k), scale, int8, f + U * u + 4 * k);
      } else if constexpr (XF == kFmtF32) {
        const float4 v = *reinterpret_cast<const float4*>(at);
        f[4 * u] = v.x; f[4 * u + 1] = v.y; f[4 * u + 2] = v.z; f[4 * u + 3] = v.w;
      } else {
        Raw8<XF> r;
        float v[8];
        r.a = *reinterpret_cast<const uint4*>(at);
        widen8<XF>(r, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[8 * u + e] = v[e];
      }
    }
  }

  // Lane l's scale byte: the l-th of the E groups that this warp's columns form.
  __device__ __forceinline__ int scale_bytes(const uint8_t* row) const {
    const int g = WIDE ? U * (wt + lane / U * warps) + lane % U : wt + lane * warps;
    return lane < E && g * kGroup8 < cols ? row[g] : 1;
  }

  // The row's 8-bit checkpoint.  Every lane takes part in the maxima.
  __device__ __forceinline__ void keep(const float (&f)[E], uint8_t* codes, uint8_t* scales,
                                       bool int8) const {
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int c = unit(u);
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < U; ++e) m = max(m, abs_bits(f[U * u + e]));
      if constexpr (WIDE) {
#pragma unroll
        for (int o = 1; o < 32 / U; o *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      } else {
        m = __reduce_max_sync(0xffffffffu, m);
      }
      if (c >= cols) continue;
      const int sb = scale_byte(m, int8);
      const float inv = scale_inverse(sb);
      if (c % kGroup8 == 0) scales[c / kGroup8] = static_cast<uint8_t>(sb);
      if constexpr (!WIDE) {
        codes[c] = static_cast<uint8_t>(encode1(f[u], inv, int8));
      } else {
        uint32_t w[U / 4];
#pragma unroll
        for (int k = 0; k < U / 4; ++k) {
          const float* v = f + U * u + 4 * k;
          w[k] = encode4(v[0], v[1], v[2], v[3], inv, int8);
        }
        if constexpr (U == 8)
          *reinterpret_cast<uint2*>(codes + c) = make_uint2(w[0], w[1]);
        else
          *reinterpret_cast<uint32_t*>(codes + c) = w[0];
      }
    }
  }
};

// ---------------------------------------------------------------- forward
template <int FMT, int NV, bool WIDE, bool LAYER>
__global__ void __launch_bounds__(norm_threads(NV), norm_ctas_per_sm(NV))
    norm_forward_kernel(NormArgs a, int warps, int teams) {
  using Th = NormThread<FMT, NV, WIDE>;
  constexpr int E = Th::E, S = norm_stages(NV, fmt_bytes(FMT));
  __shared__ float red[2 * kNormMaxWarps * 2];
  extern __shared__ uint4 ring4[];
  Th th(warps, a.cols, red);
  const float inv_n = 1.f / static_cast<float>(a.cols);
  const int64_t groups = (a.cols + kGroup8 - 1) / kGroup8;
  const int slot = norm_slot(a.cols, fmt_bytes(FMT));
  uint8_t* ring = reinterpret_cast<uint8_t*>(ring4) + th.team * S * slot;
  const int64_t step = static_cast<int64_t>(gridDim.x) * teams;
  int64_t row = blockIdx.x + static_cast<int64_t>(gridDim.x) * th.team;
  auto request = [&](int64_t r, int s) {
    if (r < a.T) th.template request<FMT>(ring + s * slot, a.x, r * a.ldx);
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < S; ++s) request(row + s * step, s);
  float g[E], b[E];
  if (NV < 4) {
    th.param(g, a.gain, a.pfmt, 1.f);
    if (LAYER) th.param(b, a.bias, a.pfmt, 0.f);
  }
  for (int s = 0; row < a.T; row += step) {
    float x[E], mean[1] = {0.f}, var[1] = {0.f};
    cp_async_wait<S - 1>();
    if (!WIDE) th.sync();  // the others' chunks
    th.template read<FMT>(x, ring + s * slot, a.x, row * a.ldx, 0, false);
    if (LAYER) {
#pragma unroll
      for (int j = 0; j < E; ++j) mean[0] += x[j];
      th.sum(mean);
      mean[0] *= inv_n;
    }
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float d = LAYER ? (th.col(j) < a.cols ? x[j] - mean[0] : 0.f) : x[j];
      var[0] = fmaf(d, d, var[0]);
    }
    th.sum(var);
    if (!WIDE && warps == 1) th.sync();
    request(row + S * step, s);  // every thread of the team holds its part of the row
    if (++s == S) s = 0;
    const float rstd = 1.f / sqrtf(fmaf(var[0], inv_n, a.eps));
    if (th.t == 0) {
      a.rstd[row] = rstd;
      if (LAYER) a.mean[row] = mean[0];
    }
    if (NV == 4) {
      th.param(g, a.gain, a.pfmt, 1.f);
      if (LAYER) th.param(b, a.bias, a.pfmt, 0.f);
    }
    if (a.codes != nullptr)
      th.keep(x, a.codes + row * a.ld_codes, a.code_scales + row * groups, a.int8);
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float z = (LAYER ? x[j] - mean[0] : x[j]) * rstd;
      x[j] = LAYER ? fmaf(z, g[j], b[j]) : z * g[j];
    }
    th.store(a.out, row * a.ldo, x);
  }
  cp_async_wait<0>();
}

// ---------------------------------------------------------------- backward
template <int FMT, int NV, bool WIDE, bool LAYER, bool X8>
__global__ void __launch_bounds__(norm_threads(NV), norm_ctas_per_sm(NV))
    norm_backward_kernel(NormArgs a, int warps, int teams) {
  using Th = NormThread<FMT, NV, WIDE>;
  constexpr int XF = X8 ? kFmtInt8 : FMT;  // of x in the ring
  constexpr int E = Th::E, S = norm_stages(NV, fmt_bytes(XF) + fmt_bytes(FMT));
  __shared__ float red[2 * kNormMaxWarps * 2];
  extern __shared__ uint4 ring4[];  // at the end the teams' sums [teams][cols]
  pdl_trigger();
  Th th(warps, a.cols, red);
  const float inv_n = 1.f / static_cast<float>(a.cols);
  const int64_t groups = (a.cols + kGroup8 - 1) / kGroup8;
  const int slot_x = norm_slot(a.cols, fmt_bytes(XF));
  const int slot = slot_x + norm_slot(a.cols, fmt_bytes(FMT));
  uint8_t* ring = reinterpret_cast<uint8_t*>(ring4) + th.team * S * slot;
  const int64_t step = static_cast<int64_t>(gridDim.x) * teams;
  int64_t row = blockIdx.x + static_cast<int64_t>(gridDim.x) * th.team;
  auto request = [&](int64_t r, int s) {
    if (r < a.T) {
      th.template request<XF>(ring + s * slot, a.x, r * a.ldx);
      th.template request<FMT>(ring + s * slot + slot_x, a.dy, r * a.lddy);
    }
    cp_async_commit();
  };
  // the row's statistics and scale bytes, one row ahead
  float mean_n = 0.f, rstd_n = 0.f;
  int byte_n = 1;
  auto small = [&](int64_t r) {
    if (r >= a.T) return;
    if (LAYER) mean_n = a.mean[r];
    rstd_n = a.rstd[r];
    if (X8) byte_n = th.scale_bytes(a.x_scales + r * groups);
  };
#pragma unroll
  for (int s = 0; s < S; ++s) request(row + s * step, s);
  small(row);
  float g[E], dg[E], db[E];
  if (NV < 4) th.param(g, a.gain, a.pfmt, 1.f);
#pragma unroll
  for (int j = 0; j < E; ++j) dg[j] = db[j] = 0.f;
  for (int s = 0; row < a.T; row += step) {
    const float mean = mean_n, rstd = rstd_n;
    const int byte = byte_n;
    small(row + step);
    float z[E], d[E];  // z, and dy then a = dy gain
    float sums[LAYER ? 2 : 1] = {};
    if (NV == 4) th.param(g, a.gain, a.pfmt, 1.f);
    cp_async_wait<S - 1>();
    if (!WIDE) th.sync();
    th.template read<XF>(z, ring + s * slot, a.x, row * a.ldx, byte, a.int8);
    th.template read<FMT>(d, ring + s * slot + slot_x, a.dy, row * a.lddy, 0, false);
    // sums of a z and (layer) of a, and this thread's share of the parameter gradients;
    // columns past the end have dy = 0 and add nothing
#pragma unroll
    for (int j = 0; j < E; ++j) {
      z[j] = (z[j] - mean) * rstd;
      if (LAYER) db[j] += d[j];
      dg[j] = fmaf(d[j], z[j], dg[j]);
      d[j] *= g[j];
      sums[0] = fmaf(d[j], z[j], sums[0]);
      if (LAYER) sums[LAYER] += d[j];
    }
    th.sum(sums);
    if (!WIDE && warps == 1) th.sync();
    request(row + S * step, s);
    if (++s == S) s = 0;
    const float c1 = sums[0] * inv_n, c2 = LAYER ? sums[LAYER] * inv_n : 0.f;
#pragma unroll
    for (int j = 0; j < E; ++j) d[j] = rstd * (d[j] - c2 - z[j] * c1);
    th.store(a.out, row * a.ldo, d);
  }
  cp_async_wait<0>();
  // ---- the CTA's sums of the parameter gradients
  const bool single = gridDim.x == 1;
  float* teamsum = reinterpret_cast<float*>(ring4);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* fin = which == 0 ? a.d_gain : a.d_bias;
    if (fin == nullptr) continue;  // uniform
    float* dst = single ? fin
                        : a.partials + (static_cast<int64_t>(blockIdx.x) * 2 + which) * a.cols;
    const bool add = single && a.accumulate;
    if (teams > 1) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (th.col(j) < a.cols)
          teamsum[th.team * a.cols + th.col(j)] = which == 0 ? dg[j] : db[j];
      __syncthreads();
      for (int col = threadIdx.x; col < a.cols; col += blockDim.x) {
        float v = add ? dst[col] : 0.f;
        for (int k = 0; k < teams; ++k) v += teamsum[k * a.cols + col];
        dst[col] = v;
      }
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const int col = th.col(j);
        if (col < a.cols) dst[col] = (which == 0 ? dg[j] : db[j]) + (add ? dst[col] : 0.f);
      }
    }
  }
}

// out[col] (+)= the sum of the partial rows: 32 lanes of rows, each in row order, then the
// lanes in order.
constexpr int kRedCols = 32, kRedLanes = 32;
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
  if (col < cols) {
#pragma unroll 4
    for (int r = ly; r < rows; r += kRedLanes)
      v += partials[(static_cast<int64_t>(r) * 2 + which) * cols + col];
  }
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
int norm_backward_max_ctas(int T) { return T < 2 * kB200Sms ? T : 2 * kB200Sms; }

// CTAs for T rows: as many as are resident at once.
static int norm_grid(int64_t T, const NormShape& sh) {
  const int64_t most = static_cast<int64_t>(kB200Sms) * norm_ctas_per_sm(sh.nv);
  return static_cast<int>(T < most ? T : most);
}

template <typename K>
static cudaError_t norm_launch(K kernel, const NormShape& sh, size_t smem, const NormArgs& a,
                               cudaStream_t s) {
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  return launch_k(kernel, dim3(norm_grid(a.T, sh)), dim3(32 * sh.warps * sh.teams), smem, s, false,
                  a, sh.warps, sh.teams);
}

template <int FMT, int NV, bool WIDE, bool LAYER>
static cudaError_t forward_nv(const NormArgs& a, const NormShape& sh, cudaStream_t s) {
  constexpr int ES = fmt_bytes(FMT);
  const size_t smem = static_cast<size_t>(sh.teams) * norm_stages(NV, ES) * norm_slot(a.cols, ES);
  return norm_launch(norm_forward_kernel<FMT, NV, WIDE, LAYER>, sh, smem, a, s);
}

template <int FMT, bool WIDE, bool LAYER>
static cudaError_t forward_shape(const NormArgs& a, cudaStream_t s) {
  const NormShape sh = norm_shape(a.cols, a.T);
  switch (sh.nv) {
    case 1: return forward_nv<FMT, 1, WIDE, LAYER>(a, sh, s);
    case 2: return forward_nv<FMT, 2, WIDE, LAYER>(a, sh, s);
    default: return forward_nv<FMT, 4, WIDE, LAYER>(a, sh, s);
  }
}

template <int FMT>
static cudaError_t forward_fmt(const NormArgs& a, cudaStream_t s) {
  constexpr int es = fmt_bytes(FMT), u = 16 / es;
  const bool wide = a.cols % u == 0 && a.ldx % u == 0 && a.ldo % u == 0 &&
                    (a.codes == nullptr || a.ld_codes % u == 0);
  if (a.layer)
    return wide ? forward_shape<FMT, true, true>(a, s) : forward_shape<FMT, false, true>(a, s);
  return wide ? forward_shape<FMT, true, false>(a, s) : forward_shape<FMT, false, false>(a, s);
}

cudaError_t launch_norm_forward(const NormArgs& a, int fmt, cudaStream_t s) {
  switch (fmt) {
    case kFmtBf16: return forward_fmt<kFmtBf16>(a, s);
    case kFmtF16: return forward_fmt<kFmtF16>(a, s);
    case kFmtF32: return forward_fmt<kFmtF32>(a, s);
  }
  return cudaErrorInvalidValue;
}

template <int FMT, int NV, bool WIDE, bool LAYER, bool X8>
static cudaError_t backward_nv(const NormArgs& a, const NormShape& sh, cudaStream_t s) {
  constexpr int ES = fmt_bytes(FMT), XS = X8 ? 1 : ES;
  size_t smem = static_cast<size_t>(sh.teams) * norm_stages(NV, XS + ES) *
                (norm_slot(a.cols, XS) + norm_slot(a.cols, ES));
  const size_t sums = sh.teams > 1 ? static_cast<size_t>(sh.teams) * a.cols * sizeof(float) : 0;
  if (sums > smem) smem = sums;
  const cudaError_t e =
      norm_launch(norm_backward_kernel<FMT, NV, WIDE, LAYER, X8>, sh, smem, a, s);
  const int grid = norm_grid(a.T, sh);
  if (e != cudaSuccess || grid == 1 || (a.d_gain == nullptr && a.d_bias == nullptr)) return e;
  return launch_k(norm_reduce_kernel,
                  dim3((a.cols + kRedCols - 1) / kRedCols, a.d_bias != nullptr ? 2 : 1),
                  dim3(kRedCols * kRedLanes), 0, s, true, a.partials, grid, a.cols, a.d_gain,
                  a.d_bias, a.accumulate);
}

template <int FMT, bool WIDE, bool LAYER, bool X8>
static cudaError_t backward_shape(const NormArgs& a, cudaStream_t s) {
  const NormShape sh = norm_shape(a.cols, a.T);
  switch (sh.nv) {
    case 1: return backward_nv<FMT, 1, WIDE, LAYER, X8>(a, sh, s);
    case 2: return backward_nv<FMT, 2, WIDE, LAYER, X8>(a, sh, s);
    default: return backward_nv<FMT, 4, WIDE, LAYER, X8>(a, sh, s);
  }
}

template <int FMT, bool X8>
static cudaError_t backward_fmt(const NormArgs& a, cudaStream_t s) {
  constexpr int u = 16 / fmt_bytes(FMT);
  const bool wide = a.cols % u == 0 && a.ldx % u == 0 && a.ldo % u == 0 && a.lddy % u == 0;
  if (a.layer)
    return wide ? backward_shape<FMT, true, true, X8>(a, s)
                : backward_shape<FMT, false, true, X8>(a, s);
  return wide ? backward_shape<FMT, true, false, X8>(a, s)
              : backward_shape<FMT, false, false, X8>(a, s);
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
