// Host-side declarations shared by the training kernels and their C interface (train.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace moe {

constexpr int kB200Sms = 148;  // sizes grids and workspaces; other counts only shift balance

// ---------------------------------------------------------------- 8-bit checkpoints
struct Act8Args {
  void* vals;         // [rows][cols], ld_vals apart: read by encode, written by decode
  uint8_t* codes;     // [rows][cols], ld_codes apart
  uint8_t* scales;    // [rows][groups]
  int64_t rows, cols, ld_vals, ld_codes, groups;
  int64_t chunks;     // warp chunks per row (set by the launcher)
  int int8;
};
// fmt: kFmtBf16, kFmtF16 or kFmtF32.
cudaError_t launch_act8(Act8Args a, int fmt, bool encode, cudaStream_t s);

// ---------------------------------------------------------------- norms
struct NormArgs {
  int T, cols;
  int layer;          // layer norm, else RMS norm
  float eps;
  const void* x;      // forward: format fmt; backward: xfmt (fmt or an 8-bit checkpoint)
  int64_t ldx;
  const uint8_t* x_scales;
  const void* gain;   // or NULL
  const void* bias;   // forward only; or NULL
  int pfmt;           // format of gain and bias
  void* out;          // forward: y; backward: dx
  int64_t ldo;
  const void* dy;     // backward
  int64_t lddy;
  float* mean;        // written by forward, read by backward; NULL for RMS
  float* rstd;
  uint8_t* codes;     // forward: 8-bit checkpoint of x, or NULL
  uint8_t* code_scales;
  int64_t ld_codes;
  int int8;           // of codes (forward) or of x (backward)
  float* d_gain;      // backward: or NULL
  float* d_bias;      // backward: or NULL
  int accumulate;
  float* partials;    // backward: [CTA][d_gain | d_bias][cols]
};
// The most CTAs of a backward pass over T rows, and so rows of its partial sums.
int norm_backward_max_ctas(int T);
cudaError_t launch_norm_forward(const NormArgs& a, int fmt, cudaStream_t s);
cudaError_t launch_norm_backward(const NormArgs& a, int fmt, int xfmt, cudaStream_t s);

// ---------------------------------------------------------------- the gated MLP's products
// Epilogues of a product's 128 x BN (or, on CTA pairs, 256 x 256) fp32 tiles.
//   kTgStore:  C in 16 bits or fp32, optionally added to what is there
//   kTgGluFwd: columns are features; the tile holds gate and up sums: h = act(g) u, and the
//              pre-activations kept in 16 or 8 bits on request
//   kTgGluBwd: the tile holds dh: dg, du and h from the kept pre-activations
constexpr int kTgStore = 0, kTgGluFwd = 1, kTgGluBwd = 2;

struct TgProblem {
  int m, n;           // rows and columns of the output (GLU: n = D features)
  int k_steps;        // ceil(K / 64)
  int m_tiles, n_tiles;
  int a_mn, b_mn;     // operand's rows run along K in memory (M or N contiguous)
  void* out;          // kTgStore: C; GLU: h [m][n] in 16 bits (kTgGluBwd: or NULL)
  int64_t ld_out;
  int out_f32, accumulate;
};

struct TgParams {
  TgProblem prob[3];
  int nprob;
  int kind;
  int f16;            // 16-bit format: fp16, else bf16
  int silu;
  void* gu;           // kept pre-activations (kTgGluFwd writes, kTgGluBwd reads); or NULL
  uint8_t* gu_scales;
  int64_t ld_gu;
  int gu_fmt;
  void* dgu;          // kTgGluBwd: [m][2n] in 16 bits
  int64_t ld_dgu;
  unsigned* status;
  uint64_t timeout_ns;
};

struct TgMaps {
  CUtensorMap a[3], b[3];
};

// Tile shapes: CTA pairs on 256 x 256, single CTAs on 128 x 128 or 128 x 64.
enum TgShape { kTgPair256 = 0, kTgOne128 = 1, kTgOne64 = 2 };
constexpr int tg_tile_m(TgShape s) { return s == kTgPair256 ? 256 : 128; }
constexpr int tg_tile_n(TgShape s) { return s == kTgPair256 ? 256 : s == kTgOne128 ? 128 : 64; }
cudaError_t launch_train_gemm(TgShape shape, const TgMaps& maps, const TgParams& p, int sms,
                              cudaStream_t s, bool pdl);

// The same for few tokens (prob[0] alone): tiles of 128 features (GLU forward: 64, gate and up)
// by nt tokens, nt a multiple of 16 up to 128, their K steps split over a cluster of 1, 2, 4 or
// 8 CTAs, all of them on the GPU at one time.
constexpr int ts_tokens(int64_t T) { return T >= 128 ? 128 : static_cast<int>((T + 15) / 16 * 16); }
// The most CTAs: above 64 tokens a CTA fills an SM, and a cluster's SMs lie in one of the GPU's
// processor clusters, which then hold no more than 32 clusters of 4 or 14 of 8 (at 34 of 4 the
// launch took two turns).
constexpr int ts_most_ctas(int splits, int nt) {
  return nt <= 64 || splits <= 2 ? kB200Sms : splits == 4 ? 128 : 112;
}
cudaError_t launch_train_small(const TgMaps& maps, const TgParams& p, int nt, int splits,
                               cudaStream_t s, bool pdl);

}  // namespace moe
