// RMS norm and layer norm over rows, forward and backward, with the 8-bit checkpoint of the
// input written or read in the same pass.
//
// A team of W warps holds one row, NV times 8 elements a thread, so x is read from memory once
// although the statistics need it twice.  The teams of a CTA (one per SM) work on rows of their
// own and meet at named barriers of their own.  The kernels are bound by HBM: forward reads x
// and writes y, backward reads x (2, 4 or 1 + 1/32 bytes) and dy and writes dx.  Rows come
// through a ring in shared memory that cp.async fills up to four rows ahead, which keeps
// 50 to 200 KB of loads in flight per SM without registers and whatever phase the teams are
// in.  Gain and bias lie in shared memory in fp32.
//
// Beside HBM a row's instructions and the latency of its sums decide (2.3 to 2.6 instructions a
// cycle of 4 at 16384 x 2816): a row costs a warp about 8 NV + 9 tens of instructions (the sums
// over lanes and warps, the ring, the row's addresses), so NV is what makes W (8 NV + 9)
// smallest: 2816 columns take 4 warps of 24 elements.
//
// Wide form (columns, strides and bases that 16-byte accesses fit): a thread owns units of 16
// bytes of the activation's format, U = 8 or 4 columns; it reads back only the units that it
// copied itself, so the ring needs no barrier.  Narrow form (any other): the row is copied as
// the aligned 16-byte chunks that cover it, and U is 1.  In both warp w's unit u of lane l is at
// column 256 NV w + 32 U u + U l: accesses are contiguous over a warp, differ by constants from
// unit to unit, and a group of 32 columns lies within one warp, where the checkpoint's scale
// is formed.
//
// The gradients of gain and bias are sums over all rows: a thread owns its columns for the
// whole kernel and adds its rows in registers, the teams of a CTA meet in shared memory, each
// CTA writes one row of partial sums, and a second small launch adds those in a fixed order
// (deterministic; a single CTA writes the result itself).
#include "act8.cuh"
#include "train_internal.h"

namespace moe {

constexpr int kNormMaxWarps = 16;             // of a row
constexpr int kNormSmem = 226 * 1024;         // of a CTA
constexpr int kNormMaxStages = 4;
constexpr int kNormRed = 2 * 768 / 32;         // floats of a round of sums: two a warp

// Threads of a CTA: as many as the registers of 8 NV elements allow with next to no spills
// (which, the ring leaving little of L1, would go to L2): 20 bytes at most up to NV = 3 (narrow
// layer norm forward at NV = 2, fp32 RMS backward at NV = 3).  NV = 4 only serves rows of more
// than 12288 columns (layer norm's backward: 9216) and spills in backward, 16 to 130 bytes for
// RMS and 350 to 390 for layer norm: 4096 x 16384 in bf16 takes 122 and 185 us there, 62 at the
// copy's rate, and layer norm's 4096 x 12288 161 us where 9216 columns at NV = 3 take 68.
__host__ __device__ constexpr int norm_forward_threads(int nv) {
  return nv <= 2 ? 768 : nv == 3 ? 640 : 512;
}
__host__ __device__ constexpr int norm_backward_threads(int nv, bool layer) {
  return nv == 1 ? 768 : nv == 3 && layer ? 384 : 512;
}

struct NormShape {
  int nv, warps, teams;  // 8-element pieces a thread, warps a row, rows side by side in a CTA
  int stages;            // of the ring
  int grid;
  size_t smem;
};

// Shared bytes that a row of `cols` elements takes in the ring (16 more: the narrow form's
// shift), and a parameter.
__host__ __device__ constexpr int norm_slot(int cols, int es) {
  return (cols * es + 15) / 16 * 16 + 16;
}
__host__ __device__ constexpr int norm_param(int cols) { return (cols + 7) / 8 * 32; }

// row: ring bytes of a row, params: shared bytes of gain and bias.  At most a row per SM: the
// fewest elements a thread, which is the shortest way through it (a 2816-column row of one
// token takes 2.6 us forward so, 7 us with 32 a thread).  Else the least instructions; fp32 has
// half the elements per byte and takes NV <= 2, with more warps to overlap.
template <typename Threads>
static NormShape norm_shape(int cols, int64_t T, int es, int row, int params, Threads threads) {
  NormShape s{};
  int best = 0;
  for (int nv = 1; nv <= 4; ++nv) {
    const int w = (cols + 256 * nv - 1) / (256 * nv);
    if (w > kNormMaxWarps || w * 32 > threads(nv)) continue;
    if (s.nv != 0 && (T <= kB200Sms || nv == 4 || (nv == 3 && es == 4))) break;
    const int cost = w * (8 * nv + 9);
    if (s.nv == 0 || cost < best) {
      best = cost;
      s.nv = nv;
      s.warps = w;
    }
  }
  const int64_t need = (T + kB200Sms - 1) / kB200Sms;  // few rows: spread over the SMs first
  const int most = threads(s.nv) / 32 / s.warps;
  s.teams = static_cast<int>(need < most ? need : most);
  // at least two rows ahead, but for rows so long that one team cannot have them
  while (s.teams > 1 && params + 2 * s.teams * row > kNormSmem) --s.teams;
  s.stages = (kNormSmem - params) / (s.teams * row);
  s.stages = s.stages > kNormMaxStages ? kNormMaxStages : s.stages;
  s.grid = static_cast<int>(T < kB200Sms ? T : kB200Sms);
  s.smem = static_cast<size_t>(params) + static_cast<size_t>(s.stages) * s.teams * row;
  return s;
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

// All groups but the newest `behind` are complete.
__device__ __forceinline__ void cp_async_wait_all_but(int behind) {
  if (behind >= 3)
    cp_async_wait<3>();
  else if (behind == 2)
    cp_async_wait<2>();
  else if (behind == 1)
    cp_async_wait<1>();
  else
    cp_async_wait<0>();
}

// A team's rows of a tensor, one after another.
struct Rows {
  uint8_t* p;
  int64_t ahead;
  __device__ __forceinline__ Rows(const void* base, int64_t row0, int64_t bytes, int64_t step)
      : p(static_cast<uint8_t*>(const_cast<void*>(base)) + row0 * bytes), ahead(step * bytes) {}
  __device__ __forceinline__ uint8_t* take() {
    uint8_t* r = p;
    p += ahead;
    return r;
  }
};

__device__ __forceinline__ float sum_of(uint64_t p) {
  float a, b;
  of_pair(p, a, b);
  return a + b;
}

template <int FMT, int NV, bool WIDE>
struct NormThread {
  static constexpr int E = 8 * NV;              // elements a thread
  static constexpr int ES = fmt_bytes(FMT);
  static constexpr int U = WIDE ? 16 / ES : 1;  // columns of a unit
  static constexpr int NU = E / U;
  int t, tpr, warps, wt, lane, team, cols;
  int c0, room;  // the thread's first column, columns from there
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
    c0 = wt * 32 * E + U * lane;
    room = n - c0;
    red = buf + team * w * 2;  // one warp a row: unused
    turn = 0;
  }
  __device__ __forceinline__ static constexpr int off(int u) { return 32 * U * u; }
  __device__ __forceinline__ bool in(int u) const { return off(u) < room; }
  __device__ __forceinline__ int col(int j) const { return c0 + off(j / U) + j % U; }

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
    float* buf = red + turn * (kNormRed);
    turn ^= 1;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) buf[wt * N + i] = v[i];
    }
    sync();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = lane < warps ? buf[lane * N + i] : 0.f;
#pragma unroll
      for (int o = kNormMaxWarps / 2; o > 0; o /= 2) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
      v[i] = __shfl_sync(0xffffffffu, v[i], 0);
    }
  }

  // Gain or bias as fp32 in shared memory, `absent` without one.  Wide 16-bit formats: the
  // first four of every eight columns lie together, then the others, so that neighbouring
  // threads' 16-byte reads are neighbours.
  __device__ __forceinline__ static int place(int c, int cols) {
    if constexpr (U != 8) return c;
    return (c >> 3) * 4 + (c & 3) + (c & 4) * ((cols + 7) / 8);
  }
  // Team 0 fills, each thread its own columns, all loads under way at once.
  __device__ __forceinline__ void fill(float* dst, const void* p, int fmt, float absent) const {
    if (team != 0) return;
    float f[E];
#pragma unroll
    for (int j = 0; j < E; ++j)
      f[j] = p != nullptr && col(j) < cols ? load1_any(p, col(j), fmt) : absent;
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (col(j) < cols) dst[place(col(j), cols)] = f[j];
  }
  __device__ __forceinline__ void param(float (&f)[U], const float* p, int u) const {
#pragma unroll
    for (int e = 0; e < U; ++e) f[e] = 0.f;
    if (!in(u)) return;
    if constexpr (U == 1) {
      f[0] = p[c0 + off(u)];
    } else {
#pragma unroll
      for (int k = 0; k < U / 4; ++k) {
        const float4 v = *reinterpret_cast<const float4*>(
            p + place(c0 + 4 * k, cols) + off(u) * 4 / U);
        f[4 * k] = v.x; f[4 * k + 1] = v.y; f[4 * k + 2] = v.z; f[4 * k + 3] = v.w;
      }
    }
  }

  // The parameters of UP elements: a unit's, or in the narrow form two units'.
  static constexpr int UP = U == 1 ? 2 : U;
  __device__ __forceinline__ void params(float (&f)[UP], const float* p, int u) const {
    if constexpr (U == 1) {
      float a[1], b[1];
      param(a, p, 2 * u);
      param(b, p, 2 * u + 1);
      f[0] = a[0];
      f[1] = b[0];
    } else {
      param(f, p, u);
    }
  }

  __device__ __forceinline__ void store(uint8_t* row, const float (&f)[E]) const {
    row += c0 * ES;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      if (!in(u)) continue;
      if constexpr (!WIDE) {
        store1<FMT>(row, off(u), f[u]);
      } else if constexpr (FMT == kFmtF32) {
        *reinterpret_cast<float4*>(row + off(u) * ES) =
            make_float4(f[4 * u], f[4 * u + 1], f[4 * u + 2], f[4 * u + 3]);
      } else {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = f[8 * u + e];
        store8<FMT>(row, off(u), v);
      }
    }
  }

  // ---- the ring.  XF: the format in memory, FMT or 8-bit codes.
  template <int XF>
  __device__ __forceinline__ void request(uint8_t* slot, const uint8_t* src) const {
    constexpr int XS = fmt_bytes(XF);
    if constexpr (WIDE) {
      slot += c0 * XS;
      src += c0 * XS;
#pragma unroll
      for (int u = 0; u < NU; ++u)
        if (in(u)) cp_async<U * XS>(slot + off(u) * XS, src + off(u) * XS);
    } else {
      const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15);
      const int end = shift + cols * XS;  // nothing behind the row is read
      for (int c = 16 * t; c < end; c += 16 * tpr) cp_async_part(slot + c, src - shift + c, min(16, end - c));
    }
  }

  // The row in the slot, its columns past the end as zeros.  8-bit codes: `byte` holds the
  // scale bytes of the warp's E groups, one a lane (see scale_bytes).
  template <int XF>
  __device__ __forceinline__ void read(float (&f)[E], const uint8_t* slot, const uint8_t* src,
                                       int byte) const {
    constexpr int XS = fmt_bytes(XF);
    constexpr bool I8 = XF == kFmtInt8;
    if constexpr (!WIDE) slot += reinterpret_cast<uintptr_t>(src) & 15;
    slot += c0 * XS;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      float scale = 0.f;
      if constexpr (XS == 1)
        scale = scale_value(__shfl_sync(0xffffffffu, byte, u * U + lane * U / 32));
#pragma unroll
      for (int e = 0; e < U; ++e) f[U * u + e] = 0.f;
      if (!in(u)) continue;
      const uint8_t* at = slot + off(u) * XS;
      if constexpr (!WIDE) {
        if constexpr (XS == 1)
          f[u] = decode1<I8>(*at, scale);
        else
          f[u] = load1<XF>(at, 0);
      } else if constexpr (XS == 1) {
#pragma unroll
        for (int k = 0; k < U / 4; ++k)
          decode4<I8>(*reinterpret_cast<const uint32_t*>(at + 4 * k), scale, f + U * u + 4 * k);
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
    const int g = wt * E + lane;
    return lane < E && g * kGroup8 < cols ? row[g] : 1;
  }

  // The row's 8-bit checkpoint.  Every lane takes part in the maxima.
  template <bool INT8>
  __device__ __forceinline__ void keep(const float (&f)[E], uint8_t* codes,
                                       uint8_t* scales) const {
    codes += c0;
    scales += c0 / kGroup8;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      float own[U];
#pragma unroll
      for (int e = 0; e < U; ++e) own[e] = f[U * u + e];
      uint32_t m = amax_bits(own);
      if constexpr (WIDE) {
#pragma unroll
        for (int o = 1; o < 32 / U; o *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      } else {
        m = __reduce_max_sync(0xffffffffu, m);
      }
      if (!in(u)) continue;
      const int sb = scale_byte<INT8>(m);
      const float inv = scale_inverse(sb);
      if (U * lane % kGroup8 == 0) scales[U * u] = static_cast<uint8_t>(sb);
      if constexpr (!WIDE) {
        codes[off(u)] = static_cast<uint8_t>(encode1<INT8>(f[u], inv));
      } else {
        uint32_t w[U / 4];
#pragma unroll
        for (int k = 0; k < U / 4; ++k) {
          const float* v = f + U * u + 4 * k;
          w[k] = encode4<INT8>(v[0], v[1], v[2], v[3], inv);
        }
        if constexpr (U == 8)
          *reinterpret_cast<uint2*>(codes + off(u)) = make_uint2(w[0], w[1]);
        else
          *reinterpret_cast<uint32_t*>(codes + off(u)) = w[0];
      }
    }
  }
};

// ---------------------------------------------------------------- forward
template <int FMT, int NV, bool WIDE, bool LAYER>
__global__ void __launch_bounds__(norm_forward_threads(NV), 1)
    norm_forward_kernel(NormArgs a, int warps, int teams, int stages) {
  using Th = NormThread<FMT, NV, WIDE>;
  constexpr int E = Th::E, U = Th::U, UP = Th::UP;
  __shared__ float red[2 * kNormRed];
  extern __shared__ uint4 ring4[];
  Th th(warps, a.cols, red);
  const float inv_n = 1.f / static_cast<float>(a.cols);
  const int64_t groups = (a.cols + kGroup8 - 1) / kGroup8;
  const int slot = norm_slot(a.cols, fmt_bytes(FMT));
  float* gain = reinterpret_cast<float*>(ring4);
  float* bias = gain + norm_param(a.cols) / 4;  // LAYER
  uint8_t* ring = reinterpret_cast<uint8_t*>(LAYER ? bias + norm_param(a.cols) / 4 : bias) +
                  th.team * stages * slot;
  const int64_t step = static_cast<int64_t>(gridDim.x) * teams;
  const int64_t row0 = blockIdx.x + static_cast<int64_t>(gridDim.x) * th.team;
  int rows = static_cast<int>((a.T - row0 + step - 1) / step);  // <= 0: none
  int asked = rows;
  const Rows px(a.x, row0, a.ldx * Th::ES, step);
  Rows next = px, now = px, out(a.out, row0, a.ldo * Th::ES, step);
  Rows codes(a.codes, row0, a.ld_codes, step), scales(a.code_scales, row0, groups, step);
  int64_t row = row0;
  auto request = [&](int s) {
    if (asked-- > 0) th.template request<FMT>(ring + s * slot, next.take());
    cp_async_commit();
  };
  for (int s = 0; s < stages; ++s) request(s);
  th.fill(gain, a.gain, a.pfmt, 1.f);
  if (LAYER) th.fill(bias, a.bias, a.pfmt, 0.f);
  __syncthreads();
  for (int s = 0; rows > 0; --rows, row += step) {
    float x[E], mean[1] = {0.f}, var[1];
    cp_async_wait_all_but(stages - 1);
    if (!WIDE) th.sync();  // the others' chunks
    th.template read<FMT>(x, ring + s * slot, now.take(), 0);
    if (LAYER) {
      uint64_t m2 = 0;
#pragma unroll
      for (int j = 0; j < E; j += 2) m2 = add2(m2, pair_of(x[j], x[j + 1]));
      mean[0] = sum_of(m2);
      th.sum(mean);
      mean[0] *= inv_n;
    }
    const uint64_t less = pair_of(-mean[0], -mean[0]);
    uint64_t v2 = 0;
#pragma unroll
    for (int j = 0; j < E; j += 2) {
      uint64_t d = pair_of(x[j], x[j + 1]);
      if (LAYER) {  // columns past the end add nothing
        d = add2(d, less);
        if (U == 1) {
          float d0, d1;
          of_pair(d, d0, d1);
          d = pair_of(th.in(j) ? d0 : 0.f, th.in(j + 1) ? d1 : 0.f);
        } else if (!th.in(j / U)) {
          d = 0;
        }
      }
      v2 = fma2(d, d, v2);
    }
    var[0] = sum_of(v2);
    th.sum(var);
    if (!WIDE && warps == 1) th.sync();
    request(s);  // every thread of the team holds its part of the row
    if (++s == stages) s = 0;
    const float rstd = rsqrtf(fmaf(var[0], inv_n, a.eps));  // within 2 ulp
    if (th.t == 0) {
      a.rstd[row] = rstd;
      if (LAYER) a.mean[row] = mean[0];
    }
    if (a.codes != nullptr) {
      if (a.int8)
        th.template keep<true>(x, codes.take(), scales.take());
      else
        th.template keep<false>(x, codes.take(), scales.take());
    }
    const uint64_t rstd2 = pair_of(rstd, rstd);
#pragma unroll
    for (int u = 0; u < E / UP; ++u) {
      float g[UP], b[UP];
      th.params(g, gain, u);
      if (LAYER) th.params(b, bias, u);
#pragma unroll
      for (int e = 0; e < UP; e += 2) {
        float *v = x + UP * u + e;
        uint64_t z = pair_of(v[0], v[1]);
        if (LAYER) z = add2(z, less);
        z = mul2(z, rstd2);
        const uint64_t g2 = pair_of(g[e], g[e + 1]);
        of_pair(LAYER ? fma2(z, g2, pair_of(b[e], b[e + 1])) : mul2(z, g2), v[0], v[1]);
      }
    }
    th.store(out.take(), x);
  }
  cp_async_wait<0>();
}

// ---------------------------------------------------------------- backward
// XF: the format of x, FMT or an 8-bit checkpoint.
template <int FMT, int NV, bool WIDE, bool LAYER, int XF>
__global__ void __launch_bounds__(norm_backward_threads(NV, LAYER), 1)
    norm_backward_kernel(NormArgs a, int warps, int teams, int stages) {
  using Th = NormThread<FMT, NV, WIDE>;
  constexpr bool X8 = fmt_bytes(XF) == 1;
  constexpr int E = Th::E, UP = Th::UP;
  __shared__ float red[2 * kNormRed];
  extern __shared__ uint4 ring4[];  // gain, ring; at the end gain, the teams' sums [teams][cols]
  pdl_trigger();
  Th th(warps, a.cols, red);
  const float inv_n = 1.f / static_cast<float>(a.cols);
  const int64_t groups = (a.cols + kGroup8 - 1) / kGroup8;
  const int slot_x = norm_slot(a.cols, fmt_bytes(XF));
  const int slot = slot_x + norm_slot(a.cols, fmt_bytes(FMT));
  float* gain = reinterpret_cast<float*>(ring4);
  float* teamsum = gain + norm_param(a.cols) / 4;
  uint8_t* ring = reinterpret_cast<uint8_t*>(teamsum) + th.team * stages * slot;
  const int64_t step = static_cast<int64_t>(gridDim.x) * teams;
  const int64_t row0 = blockIdx.x + static_cast<int64_t>(gridDim.x) * th.team;
  int rows = static_cast<int>((a.T - row0 + step - 1) / step);  // <= 0: none
  int asked = rows, told = rows;
  const Rows px(a.x, row0, a.ldx * fmt_bytes(XF), step);
  const Rows pdy(a.dy, row0, a.lddy * Th::ES, step);
  Rows next_x = px, now_x = px, next_dy = pdy, now_dy = pdy;
  Rows out(a.out, row0, a.ldo * Th::ES, step), scales(a.x_scales, row0, groups, step);
  Rows means(a.mean, row0, sizeof(float), step), rstds(a.rstd, row0, sizeof(float), step);
  auto request = [&](int s) {
    if (asked-- > 0) {
      th.template request<XF>(ring + s * slot, next_x.take());
      th.template request<FMT>(ring + s * slot + slot_x, next_dy.take());
    }
    cp_async_commit();
  };
  // the row's statistics and scale bytes, one row ahead
  float mean_n = 0.f, rstd_n = 0.f;
  int byte_n = 1;
  auto small = [&] {
    if (told-- <= 0) return;
    if (LAYER) mean_n = *reinterpret_cast<const float*>(means.take());
    rstd_n = *reinterpret_cast<const float*>(rstds.take());
    if (X8) byte_n = th.scale_bytes(scales.take());
  };
  for (int s = 0; s < stages; ++s) request(s);
  small();
  th.fill(gain, a.gain, a.pfmt, 1.f);
  __syncthreads();
  float dg[E], db[E];
#pragma unroll
  for (int j = 0; j < E; ++j) dg[j] = db[j] = 0.f;
  for (int s = 0; rows > 0; --rows) {
    const float mean = mean_n, rstd = rstd_n;
    const int byte = byte_n;
    small();
    float z[E], d[E];  // z, and dy then a = dy gain
    float sums[LAYER ? 2 : 1];
    cp_async_wait_all_but(stages - 1);
    if (!WIDE) th.sync();
    th.template read<XF>(z, ring + s * slot, now_x.take(), byte);
    th.template read<FMT>(d, ring + s * slot + slot_x, now_dy.take(), 0);
    // sums of a z and (layer) of a, and this thread's share of the parameter gradients;
    // columns past the end have dy = 0 and add nothing
    const uint64_t less = pair_of(-mean, -mean), rstd2 = pair_of(rstd, rstd);
    uint64_t az = 0, as = 0;
#pragma unroll
    for (int u = 0; u < E / UP; ++u) {
      float g[UP];
      th.params(g, gain, u);
#pragma unroll
      for (int e = 0; e < UP; e += 2) {
        const int j = UP * u + e;
        uint64_t zz = pair_of(z[j], z[j + 1]), dd = pair_of(d[j], d[j + 1]);
        if (LAYER) {
          zz = add2(zz, less);
          of_pair(add2(pair_of(db[j], db[j + 1]), dd), db[j], db[j + 1]);
        }
        zz = mul2(zz, rstd2);
        of_pair(fma2(dd, zz, pair_of(dg[j], dg[j + 1])), dg[j], dg[j + 1]);
        dd = mul2(dd, pair_of(g[e], g[e + 1]));
        az = fma2(dd, zz, az);
        if (LAYER) as = add2(as, dd);
        of_pair(zz, z[j], z[j + 1]);
        of_pair(dd, d[j], d[j + 1]);
      }
    }
    sums[0] = sum_of(az);
    if (LAYER) sums[LAYER] = sum_of(as);
    th.sum(sums);
    if (!WIDE && warps == 1) th.sync();
    request(s);
    if (++s == stages) s = 0;
    // dx = rstd (a - mean(a)) - z rstd mean(a z)
    const float c1 = -rstd * (sums[0] * inv_n), c2 = LAYER ? -rstd * (sums[LAYER] * inv_n) : 0.f;
#pragma unroll
    for (int j = 0; j < E; j += 2) {
      uint64_t dd = pair_of(d[j], d[j + 1]);
      dd = LAYER ? fma2(dd, rstd2, pair_of(c2, c2)) : mul2(dd, rstd2);
      of_pair(fma2(pair_of(z[j], z[j + 1]), pair_of(c1, c1), dd), d[j], d[j + 1]);
    }
    th.store(out.take(), d);
  }
  cp_async_wait<0>();
  // ---- the CTA's sums of the parameter gradients
  const bool single = gridDim.x == 1;
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
int norm_backward_max_ctas(int T) { return T < kB200Sms ? T : kB200Sms; }

template <typename K>
static cudaError_t norm_launch(K kernel, const NormShape& sh, const NormArgs& a, cudaStream_t s) {
  if (sh.smem > 40 * 1024) {
    // the limit belongs to the kernel and not to this call: always the same, so that a call
    // on another host thread cannot lower it between here and the launch
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormSmem);
    if (e != cudaSuccess) return e;
  }
  return launch_k(kernel, dim3(sh.grid), dim3(32 * sh.warps * sh.teams), sh.smem, s, false, a,
                  sh.warps, sh.teams, sh.stages);
}

template <int FMT, bool WIDE, bool LAYER>
static cudaError_t forward_shape(const NormArgs& a, cudaStream_t s) {
  constexpr int ES = fmt_bytes(FMT);
  const NormShape sh = norm_shape(a.cols, a.T, ES, norm_slot(a.cols, ES),
                                  (LAYER ? 2 : 1) * norm_param(a.cols), norm_forward_threads);
  switch (sh.nv) {
    case 1: return norm_launch(norm_forward_kernel<FMT, 1, WIDE, LAYER>, sh, a, s);
    case 2: return norm_launch(norm_forward_kernel<FMT, 2, WIDE, LAYER>, sh, a, s);
    case 3: return norm_launch(norm_forward_kernel<FMT, 3, WIDE, LAYER>, sh, a, s);
    default: return norm_launch(norm_forward_kernel<FMT, 4, WIDE, LAYER>, sh, a, s);
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

template <int FMT, bool WIDE, bool LAYER, int XF>
static cudaError_t backward_shape(const NormArgs& a, cudaStream_t s) {
  constexpr int ES = fmt_bytes(FMT), XS = fmt_bytes(XF);
  NormShape sh = norm_shape(a.cols, a.T, ES, norm_slot(a.cols, XS) + norm_slot(a.cols, ES),
                            norm_param(a.cols),
                            [](int nv) { return norm_backward_threads(nv, LAYER); });
  if (sh.teams > 1) {  // the teams' sums at the end
    // (two rows a team fit, and a row is at least 3 bytes a column: so do these 4)
    const size_t sums = norm_param(a.cols) + static_cast<size_t>(sh.teams) * a.cols * sizeof(float);
    if (sums > sh.smem) sh.smem = sums;
  }
  cudaError_t e;
  switch (sh.nv) {
    case 1: e = norm_launch(norm_backward_kernel<FMT, 1, WIDE, LAYER, XF>, sh, a, s); break;
    case 2: e = norm_launch(norm_backward_kernel<FMT, 2, WIDE, LAYER, XF>, sh, a, s); break;
    case 3: e = norm_launch(norm_backward_kernel<FMT, 3, WIDE, LAYER, XF>, sh, a, s); break;
    default: e = norm_launch(norm_backward_kernel<FMT, 4, WIDE, LAYER, XF>, sh, a, s); break;
  }
  if (e != cudaSuccess || sh.grid == 1 || (a.d_gain == nullptr && a.d_bias == nullptr)) return e;
  return launch_k(norm_reduce_kernel,
                  dim3((a.cols + kRedCols - 1) / kRedCols, a.d_bias != nullptr ? 2 : 1),
                  dim3(kRedCols * kRedLanes), 0, s, true, a.partials, sh.grid, a.cols, a.d_gain,
                  a.d_bias, a.accumulate);
}

template <int FMT, int XF>
static cudaError_t backward_fmt(const NormArgs& a, cudaStream_t s) {
  constexpr int u = 16 / fmt_bytes(FMT);
  const bool wide = a.cols % u == 0 && a.ldx % u == 0 && a.ldo % u == 0 && a.lddy % u == 0;
  if (a.layer)
    return wide ? backward_shape<FMT, true, true, XF>(a, s)
                : backward_shape<FMT, false, true, XF>(a, s);
  return wide ? backward_shape<FMT, true, false, XF>(a, s)
              : backward_shape<FMT, false, false, XF>(a, s);
}

template <int FMT>
static cudaError_t backward_x(const NormArgs& a, int xfmt, cudaStream_t s) {
  if (xfmt == kFmtInt8) return backward_fmt<FMT, kFmtInt8>(a, s);
  if (xfmt == kFmtE4m3) return backward_fmt<FMT, kFmtE4m3>(a, s);
  return backward_fmt<FMT, FMT>(a, s);
}

cudaError_t launch_norm_backward(const NormArgs& a, int fmt, int xfmt, cudaStream_t s) {
  switch (fmt) {
    case kFmtBf16: return backward_x<kFmtBf16>(a, xfmt, s);
    case kFmtF16: return backward_x<kFmtF16>(a, xfmt, s);
    case kFmtF32: return backward_x<kFmtF32>(a, xfmt, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace moe
