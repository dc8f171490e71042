// C interface of the training operators: argument checks, workspace layout, tensor maps and
// launch sequences.  See include/moe_train.h for the contract.
#include <stdint.h>

#include <algorithm>

#include "act8.cuh"
#include "moe_train.h"
#include "train_internal.h"

using namespace moe;

namespace {

constexpr uint64_t kWaitTimeoutNs = 2000000000ull;  // bound of every device wait: 2 s
constexpr size_t kAlign = 1024;
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 512;
constexpr int64_t kMaxLd = int64_t(1) << 32;  // elements; keeps TMA strides below 2^40 bytes

size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool tensor_ok(const void* p) { return p != nullptr && aligned16(p); }
moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

bool wide_format(int f) { return f == kFmtBf16 || f == kFmtF16 || f == kFmtF32; }
bool eight_bits(int f) { return f == kFmtInt8 || f == kFmtE4m3; }

// An activation of `cols` columns in `format`, or (allow8) an 8-bit checkpoint.
bool act_ok(const moe_act_t* a, int64_t cols, int format, bool allow8) {
  if (a == nullptr || !tensor_ok(a->data) || a->ld < cols || a->ld > kMaxLd) return false;
  if (allow8 && eight_bits(a->format)) return a->scales != nullptr;
  return a->format == format && a->scales == nullptr;
}

bool ws_ok(const void* ws, size_t bytes, size_t need) {
  return ws != nullptr && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0 && bytes >= need;
}

moe_status_t act8_call(int64_t rows, int32_t cols, const moe_act_t* vals, const moe_act_t* codes,
                       bool encode, void* stream) {
  if (rows < 0 || cols < 1 || vals == nullptr || codes == nullptr) return MOE_ERR_INVALID_ARG;
  if (cols > 65536 || rows >= (int64_t(1) << 46) / cols) return MOE_ERR_UNSUPPORTED;
  if (!wide_format(vals->format) || !eight_bits(codes->format)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!act_ok(vals, cols, vals->format, false) || !act_ok(codes, cols, codes->format, true))
    return MOE_ERR_INVALID_ARG;
  Act8Args a{};
  a.vals = vals->data;
  a.codes = static_cast<uint8_t*>(codes->data);
  a.scales = codes->scales;
  a.rows = rows;
  a.cols = cols;
  a.ld_vals = vals->ld;
  a.ld_codes = codes->ld;
  a.groups = ceil_div(cols, kGroup8);
  a.int8 = codes->format == kFmtInt8;
  return cuda_status(launch_act8(a, vals->format, encode, static_cast<cudaStream_t>(stream)));
}

// ---------------------------------------------------------------- norms
moe_status_t check_norm(const moe_norm_config_t* c, int32_t T) {
  if (c == nullptr || T < 0) return MOE_ERR_INVALID_ARG;
  if (c->kind != MOE_NORM_RMS && c->kind != MOE_NORM_LAYER) return MOE_ERR_INVALID_ARG;
  if (!(c->eps > 0.f) || !(c->eps < 1e30f)) return MOE_ERR_INVALID_ARG;
  if (!wide_format(c->format) || !wide_format(c->param_format)) return MOE_ERR_INVALID_ARG;
  if (c->cols < 1 || c->cols > 16384 || T > kMaxRows) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool optional_ok(const void* p) { return p == nullptr || aligned16(p); }

NormArgs norm_args(const moe_norm_config_t* c, int32_t T, const moe_act_t* x) {
  NormArgs a{};
  a.T = T;
  a.cols = c->cols;
  a.layer = c->kind == MOE_NORM_LAYER;
  a.eps = c->eps;
  a.x = x->data;
  a.ldx = x->ld;
  a.x_scales = x->scales;
  a.pfmt = c->param_format;
  return a;
}

// ---------------------------------------------------------------- the gated MLP
moe_status_t check_mlp(const moe_mlp_config_t* c, int32_t T) {
  if (c == nullptr || T < 0) return MOE_ERR_INVALID_ARG;
  if (c->act != MOE_ACT_GELU_TANH && c->act != MOE_ACT_SILU) return MOE_ERR_INVALID_ARG;
  if (c->format != MOE_F_BF16 && c->format != MOE_F_F16) return MOE_ERR_INVALID_ARG;
  for (int32_t v : {c->hidden, c->inter})
    if (v < 8 || v > 16384 || v % 8) return MOE_ERR_UNSUPPORTED;
  return T > kMaxRows ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

struct MlpLayout {
  size_t h, dgu, x16, total;
  int64_t ld_h, ld_dgu, ld_x; // rows start on 128-byte lines, as the copies like them best
};

MlpLayout mlp_layout(const moe_mlp_config_t* c, int32_t T) {
  const size_t t = static_cast<size_t>(T), H = c->hidden, D = c->inter;
  MlpLayout L;
  L.ld_h = static_cast<int64_t>((D + 63) / 64 * 64);
  L.ld_dgu = static_cast<int64_t>((2 * D + 63) / 64 * 64);
  L.ld_x = static_cast<int64_t>((H + 63) / 64 * 64);
  L.h = kWsData;
  L.dgu = L.h + align_up(t * L.ld_h * 2);
  L.x16 = L.dgu + align_up(t * L.ld_dgu * 2);
  L.total = L.x16 + align_up(t * L.ld_x * 2);
  return L;
}

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off);
}

// 16-bit matrix of `rows` rows of `cols` elements, ld apart, in boxes of 64 columns x box_rows,
// swizzled as the tensor core reads them.
bool map_2d(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t ld,
            int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Gate and up rows [2][D][H] as a third dimension, so that a tile past the last gate row
// reads zeros and not the first up rows.
bool map_gate_up(CUtensorMap* m, const void* base, int64_t D, int64_t H, int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
  if (fn == nullptr) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(D), 2};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(H) * 2, static_cast<cuuint64_t>(D * H) * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An operand: `rows` (M or N) by K.  mn: the rows lie along memory (K rows of `rows` elements).
struct Operand {
  const void* p;
  int64_t ld;
  bool mn;
};

bool map_operand(CUtensorMap* m, const Operand& o, int64_t rows, int64_t K, int tile_rows) {
  return o.mn ? map_2d(m, o.p, K, rows, o.ld, 64) : map_2d(m, o.p, rows, K, o.ld, tile_rows);
}

struct Product {
  int64_t m, n, k;  // GLU forward: n = features
  Operand a, b;     // GLU forward: b is the stacked gate and up weights
  void* out;
  int64_t ld_out;
  int out_f32, accumulate;
};

// How a launch is tiled: by the least time that these estimates give, in ns, fitted to launches
// of every form at 2816 x 2112, 2048 x 1024, 1000 x 1352 and 512 x 384 with 4 to 4096 tokens.
// A tile's time is its K steps or its epilogue, whichever is longer, and the last epilogue is
// not overlapped; tiles of 256 x 256 on CTA pairs move the fewest bytes a FLOP but leave most
// SMs idle when they are few.  At 2816 x 2112 (k = 44 steps) the gate_up product of 1001
// tokens takes 23.8 us on pairs, 26.2 on 128 x 128 and 36.7 on 128 x 64; of 512 tokens 22.4,
// 15.5 and 21.4; of 256 tokens 21.5, 14.7 and 13.2; of 64 tokens 12.4 on 128 x 64 and 9.3 on
// few-token tiles split 4 ways.  Rows of 1000 elements, whose pieces of 128 bytes lie in two
// lines, shift that: of 4096 tokens 32.7, 42.9 and 56.4 (1000 x 1352, k = 16).
struct TileCost {
  int step, step_off;   // a K step of 64; with rows that start off a 128-byte line
  int fixed, fixed_bwd; // launch, setup, last epilogue; that of dh
  int least;            // a tile's epilogue
};
constexpr TileCost kTileCost[3] = {{320, 515, 8000, 14500, 2200}, {222, 480, 4500, 7500, 2400},
                                   {180, 326, 4200, 5600, 1360}};

struct Plan {
  bool small;  // train_small.cu; else `shape`
  TgShape shape;
  int splits;  // small: CTAs that share a tile
  int64_t ns;
};

Plan plan_products(const Product* pr, int n, int kind) {
  const bool glu_fwd = kind == kTgGluFwd, glu_bwd = kind == kTgGluBwd;
  Plan best{};
  for (TgShape s : {kTgPair256, kTgOne128, kTgOne64}) {
    const TileCost& tc = kTileCost[s];
    const int64_t ctas = s == kTgPair256 ? kB200Sms / 2 : kB200Sms;
    int64_t tiles = 0, longest = tc.least;
    for (int i = 0; i < n; ++i) {
      const bool off = pr[i].a.ld % 64 != 0 || pr[i].b.ld % 64 != 0;
      tiles += ceil_div(pr[i].m, tg_tile_m(s)) * ceil_div((glu_fwd ? 2 : 1) * pr[i].n, tg_tile_n(s));
      longest = std::max(longest, ceil_div(pr[i].k, 64) * (off ? tc.step_off : tc.step));
    }
    const int64_t ns = (glu_bwd ? tc.fixed_bwd : tc.fixed) + ceil_div(tiles, ctas) * longest;
    if (best.ns == 0 || ns < best.ns) best = Plan{false, s, 1, ns};
  }
  if (n == 1 && !pr[0].a.mn && !pr[0].out_f32 && !pr[0].accumulate) {
    const int nt = ts_tokens(pr[0].m);
    const int64_t tiles = ceil_div(pr[0].m, nt) * ceil_div(pr[0].n, glu_fwd ? 64 : 128);
    const int64_t k = ceil_div(pr[0].k, 64);
    for (int splits = 1; splits <= 8 && k >= 2 * splits; splits *= 2) {
      if (tiles * splits > ts_most_ctas(splits, nt)) break;
      const int64_t ns = 5000 + 8 * nt + ceil_div(k, splits) * (180 + nt * 6 / 10) +
                         nt * (glu_bwd ? 80 : 25) / splits;
      if (ns < best.ns) best = Plan{true, kTgOne128, splits, ns};
    }
  }
  return best;
}

// The products of either pass; p points at what the call was given (NULL where only the sizes
// matter).
struct MlpTensors {
  const void *x, *w_gate_up, *w_down, *dy;
  int64_t ld_x, ld_dy;
  void *h, *dgu;
};
Product up_product(const moe_mlp_config_t* c, int32_t T, const MlpLayout& L, const MlpTensors& p) {
  const int64_t H = c->hidden, D = c->inter;
  return Product{T, D, H, {p.x, p.ld_x, false}, {p.w_gate_up, H, false}, p.h, L.ld_h, 0, 0};
}
Product down_product(const moe_mlp_config_t* c, int32_t T, const MlpLayout& L, const MlpTensors& p,
                     void* y, int64_t ld_y) {
  const int64_t H = c->hidden, D = c->inter;
  return Product{T, H, D, {p.h, L.ld_h, false}, {p.w_down, D, false}, y, ld_y, 0, 0};
}
Product dh_product(const moe_mlp_config_t* c, int32_t T, const MlpLayout& L, const MlpTensors& p,
                   bool keep_h) {
  const int64_t H = c->hidden, D = c->inter;
  return Product{T, D, H, {p.dy, p.ld_dy, false}, {p.w_down, D, true}, keep_h ? p.h : nullptr,
                 L.ld_h, 0, 0};
}
Product dx_product(const moe_mlp_config_t* c, int32_t T, const MlpLayout& L, const MlpTensors& p,
                   void* dx, int64_t ld_dx) {
  const int64_t H = c->hidden, D = c->inter;
  return Product{T, H, 2 * D, {p.dgu, L.ld_dgu, false}, {p.w_gate_up, H, true}, dx, ld_dx, 0, 0};
}
Product dw_gate_up_product(const moe_mlp_config_t* c, int32_t T, const MlpLayout& L,
                           const MlpTensors& p, void* dw, int f32, int acc) {
  const int64_t H = c->hidden, D = c->inter;
  return Product{2 * D, H, T, {p.dgu, L.ld_dgu, true}, {p.x, p.ld_x, true}, dw, H, f32, acc};
}
Product dw_down_product(const moe_mlp_config_t* c, int32_t T, const MlpLayout& L,
                        const MlpTensors& p, void* dw, int f32, int acc) {
  const int64_t H = c->hidden, D = c->inter;
  return Product{H, D, T, {p.dy, p.ld_dy, true}, {p.h, L.ld_h, true}, dw, D, f32, acc};
}

moe_status_t run_products(const Product* pr, int n, TgParams p, cudaStream_t s, bool pdl) {
  const int sms = device_sm_count();
  if (sms <= 0) return MOE_ERR_CUDA;
  const bool glu_fwd = p.kind == kTgGluFwd;
  const Plan plan = plan_products(pr, n, p.kind);
  const bool small = plan.small;
  const TgShape shape = plan.shape;
  const int nt = ts_tokens(pr[0].m);
  const int tm = small ? nt : tg_tile_m(shape), tn = tg_tile_n(shape);
  const int b_rows = shape == kTgPair256 ? 128 : tn;  // B rows that one CTA loads
  TgMaps maps{};
  for (int i = 0; i < n; ++i) {
    TgProblem& q = p.prob[i];
    q = TgProblem{};
    q.m = static_cast<int>(pr[i].m);
    q.n = static_cast<int>(pr[i].n);
    q.k_steps = static_cast<int>(ceil_div(pr[i].k, 64));
    q.m_tiles = static_cast<int>(ceil_div(pr[i].m, tm));
    q.n_tiles = static_cast<int>(ceil_div((glu_fwd ? 2 : 1) * pr[i].n, tn));
    q.a_mn = pr[i].a.mn;
    q.b_mn = pr[i].b.mn;
    q.out = pr[i].out;
    q.ld_out = pr[i].ld_out;
    q.out_f32 = pr[i].out_f32;
    q.accumulate = pr[i].accumulate;
    if (!map_operand(&maps.a[i], pr[i].a, pr[i].m, pr[i].k, small ? nt : 128)) return MOE_ERR_CUDA;
    const bool ok = glu_fwd ? map_gate_up(&maps.b[i], pr[i].b.p, pr[i].n, pr[i].k,
                                          shape == kTgPair256 ? 128 : tn / 2)
                            : map_operand(&maps.b[i], pr[i].b, pr[i].n, pr[i].k, b_rows);
    if (!ok) return MOE_ERR_CUDA;
  }
  for (int i = n; i < 3; ++i) {  // unused sets: valid copies of the first
    maps.a[i] = maps.a[0];
    maps.b[i] = maps.b[0];
  }
  p.nprob = n;
  if (small) return cuda_status(launch_train_small(maps, p, nt, plan.splits, s, pdl));
  return cuda_status(launch_train_gemm(shape, maps, p, sms, s, pdl));
}

// Kept pre-activations: cfg's format, or 8-bit checkpoints of the two halves.
bool gu_ok(const moe_act_t* gu, const moe_mlp_config_t* c) {
  return act_ok(gu, 2 * static_cast<int64_t>(c->inter), c->format, true) && gu->ld % 8 == 0;
}

// dx in a launch of its own, whose K loop is split, and not with the weight gradients.
bool dx_alone(const Product& dx) { return plan_products(&dx, 1, kTgStore).small; }

TgParams mlp_params(const moe_mlp_config_t* c, int kind, const moe_act_t* gu, void* ws) {
  TgParams p{};
  p.kind = kind;
  p.f16 = c->format == MOE_F_F16;
  p.silu = c->act == MOE_ACT_SILU;
  if (gu != nullptr) {
    p.gu = gu->data;
    p.gu_scales = gu->scales;
    p.ld_gu = gu->ld;
    p.gu_fmt = gu->format;
  }
  p.status = at<unsigned>(ws, 0);
  p.timeout_ns = kWaitTimeoutNs;
  return p;
}

}  // namespace

extern "C" {

moe_status_t moe_act_encode(int64_t rows, int32_t cols, const moe_act_t* src,
                            const moe_act_t* dst, void* stream) {
  return act8_call(rows, cols, src, dst, true, stream);
}

moe_status_t moe_act_decode(int64_t rows, int32_t cols, const moe_act_t* src,
                            const moe_act_t* dst, void* stream) {
  return act8_call(rows, cols, dst, src, false, stream);
}

moe_status_t moe_norm_forward(const moe_norm_config_t* cfg, int32_t T, const moe_act_t* x,
                              const void* gain, const void* bias, const moe_act_t* y,
                              float* mean, float* rstd, const moe_act_t* kept, void* stream) {
  moe_status_t st = check_norm(cfg, T);
  if (st != MOE_OK) return st;
  const bool layer = cfg->kind == MOE_NORM_LAYER;
  if (!layer && (bias != nullptr || mean != nullptr)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!act_ok(x, cfg->cols, cfg->format, false) || !act_ok(y, cfg->cols, cfg->format, false) ||
      !optional_ok(gain) || !optional_ok(bias) || !tensor_ok(rstd) || (layer && !tensor_ok(mean)))
    return MOE_ERR_INVALID_ARG;
  if (y->data == x->data && y->ld != x->ld) return MOE_ERR_INVALID_ARG;
  if (kept != nullptr && (!eight_bits(kept->format) || !act_ok(kept, cfg->cols, -1, true)))
    return MOE_ERR_INVALID_ARG;
  NormArgs a = norm_args(cfg, T, x);
  a.gain = gain;
  a.bias = bias;
  a.out = y->data;
  a.ldo = y->ld;
  a.mean = mean;
  a.rstd = rstd;
  if (kept != nullptr) {
    a.codes = static_cast<uint8_t*>(kept->data);
    a.code_scales = kept->scales;
    a.ld_codes = kept->ld;
    a.int8 = kept->format == kFmtInt8;
  }
  return cuda_status(launch_norm_forward(a, cfg->format, static_cast<cudaStream_t>(stream)));
}

size_t moe_norm_workspace_size(const moe_norm_config_t* cfg, int32_t T) {
  if (check_norm(cfg, T) != MOE_OK) return 0;
  const size_t rows = norm_backward_max_ctas(T);
  return kWsData + align_up(rows * 2 * cfg->cols * sizeof(float));
}

moe_status_t moe_norm_backward(const moe_norm_config_t* cfg, int32_t T, const moe_act_t* x,
                               const void* gain, const float* mean, const float* rstd,
                               const moe_act_t* dy, const moe_act_t* dx, float* d_gain,
                               float* d_bias, int32_t accumulate, void* ws, size_t ws_bytes,
                               void* stream) {
  moe_status_t st = check_norm(cfg, T);
  if (st != MOE_OK) return st;
  const bool layer = cfg->kind == MOE_NORM_LAYER;
  if (!layer && (d_bias != nullptr || mean != nullptr)) return MOE_ERR_INVALID_ARG;
  if (!optional_ok(d_gain) || !optional_ok(d_bias)) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {  // sums over no rows
    const size_t n = static_cast<size_t>(cfg->cols) * sizeof(float);
    for (float* g : {d_gain, d_bias})
      if (g != nullptr && !accumulate && (st = cuda_status(cudaMemsetAsync(g, 0, n, s))) != MOE_OK)
        return st;
    return MOE_OK;
  }
  if (!act_ok(x, cfg->cols, cfg->format, true) || !act_ok(dy, cfg->cols, cfg->format, false) ||
      !act_ok(dx, cfg->cols, cfg->format, false) || !optional_ok(gain) || !tensor_ok(rstd) ||
      (layer && !tensor_ok(mean)))
    return MOE_ERR_INVALID_ARG;
  if (dx->data == dy->data && dx->ld != dy->ld) return MOE_ERR_INVALID_ARG;
  if (!ws_ok(ws, ws_bytes, moe_norm_workspace_size(cfg, T))) return MOE_ERR_WORKSPACE;
  NormArgs a = norm_args(cfg, T, x);
  a.gain = gain;
  a.out = dx->data;
  a.ldo = dx->ld;
  a.dy = dy->data;
  a.lddy = dy->ld;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.int8 = x->format == kFmtInt8;
  a.d_gain = d_gain;
  a.d_bias = d_bias;
  a.accumulate = accumulate != 0;
  a.partials = at<float>(ws, kWsData);
  return cuda_status(launch_norm_backward(a, cfg->format, x->format, s));
}

size_t moe_mlp_workspace_size(const moe_mlp_config_t* cfg, int32_t T) {
  return check_mlp(cfg, T) == MOE_OK ? mlp_layout(cfg, T).total : 0;
}

moe_status_t moe_mlp_forward(const moe_mlp_config_t* cfg, int32_t T, const moe_act_t* x,
                             const void* w_gate_up, const void* w_down, const moe_act_t* y,
                             const moe_act_t* kept_gu, void* ws, size_t ws_bytes, void* stream) {
  moe_status_t st = check_mlp(cfg, T);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  const int64_t H = cfg->hidden;
  if (!act_ok(x, H, cfg->format, false) || !act_ok(y, H, cfg->format, false) || x->ld % 8 ||
      y->ld % 8 || !tensor_ok(w_gate_up) || !tensor_ok(w_down) ||
      (kept_gu != nullptr && !gu_ok(kept_gu, cfg)))
    return MOE_ERR_INVALID_ARG;
  const MlpLayout L = mlp_layout(cfg, T);
  if (!ws_ok(ws, ws_bytes, L.total)) return MOE_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const MlpTensors p{x->data, w_gate_up, w_down, nullptr, x->ld, 0, at<void>(ws, L.h), nullptr};
  const Product up = up_product(cfg, T, L, p);
  if ((st = run_products(&up, 1, mlp_params(cfg, kTgGluFwd, kept_gu, ws), s, false)) != MOE_OK)
    return st;
  const Product down = down_product(cfg, T, L, p, y->data, y->ld);
  return run_products(&down, 1, mlp_params(cfg, kTgStore, nullptr, ws), s, true);
}

moe_status_t moe_mlp_backward(const moe_mlp_config_t* cfg, int32_t T, const moe_act_t* x,
                              const moe_act_t* gu, const void* w_gate_up, const void* w_down,
                              const moe_act_t* dy, const moe_act_t* dx, void* dw_gate_up,
                              void* dw_down, int32_t grad_format, int32_t accumulate, void* ws,
                              size_t ws_bytes, void* stream) {
  moe_status_t st = check_mlp(cfg, T);
  if (st != MOE_OK) return st;
  if (grad_format != cfg->format && grad_format != MOE_F_F32) return MOE_ERR_INVALID_ARG;
  if (!optional_ok(dw_gate_up) || !optional_ok(dw_down)) return MOE_ERR_INVALID_ARG;
  const int64_t H = cfg->hidden, D = cfg->inter;
  const int f32 = grad_format == MOE_F_F32, acc = accumulate != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {  // sums over no rows
    const size_t n = static_cast<size_t>(H * D) * (f32 ? 4 : 2);
    if (dw_gate_up != nullptr && !acc && cudaMemsetAsync(dw_gate_up, 0, 2 * n, s) != cudaSuccess)
      return MOE_ERR_CUDA;
    if (dw_down != nullptr && !acc && cudaMemsetAsync(dw_down, 0, n, s) != cudaSuccess)
      return MOE_ERR_CUDA;
    return MOE_OK;
  }
  if (!gu_ok(gu, cfg) || !act_ok(dy, H, cfg->format, false) || dy->ld % 8 ||
      !tensor_ok(w_down))
    return MOE_ERR_INVALID_ARG;
  if (dx != nullptr && (!act_ok(dx, H, cfg->format, false) || dx->ld % 8 || !tensor_ok(w_gate_up)))
    return MOE_ERR_INVALID_ARG;
  if (dw_gate_up != nullptr && (!act_ok(x, H, cfg->format, true) || x->ld % 8))
    return MOE_ERR_INVALID_ARG;
  const MlpLayout L = mlp_layout(cfg, T);
  if (!ws_ok(ws, ws_bytes, L.total)) return MOE_ERR_WORKSPACE;
  if (dx == nullptr && dw_gate_up == nullptr && dw_down == nullptr) return MOE_OK;
  MlpTensors t{x != nullptr ? x->data : nullptr, w_gate_up, w_down, dy->data,
               x != nullptr ? x->ld : 0, dy->ld, at<void>(ws, L.h), at<void>(ws, L.dgu)};
  if (dw_gate_up != nullptr && eight_bits(x->format)) {  // exact in bf16: operands as they were kept
    const moe_act_t wide{at<void>(ws, L.x16), nullptr, L.ld_x, cfg->format};
    if ((st = act8_call(T, cfg->hidden, &wide, x, false, stream)) != MOE_OK) return st;
    t.x = wide.data;
    t.ld_x = L.ld_x;
  }
  TgParams p = mlp_params(cfg, kTgGluBwd, gu, ws);
  p.dgu = t.dgu;
  p.ld_dgu = L.ld_dgu;
  const Product dh = dh_product(cfg, T, L, t, dw_down != nullptr);
  if ((st = run_products(&dh, 1, p, s, false)) != MOE_OK) return st;
  Product out[3];
  int n = 0;
  if (dx != nullptr) {
    out[n++] = dx_product(cfg, T, L, t, dx->data, dx->ld);
    if (dx_alone(out[0])) {
      if ((st = run_products(out, 1, mlp_params(cfg, kTgStore, nullptr, ws), s, true)) != MOE_OK)
        return st;
      n = 0;
    }
  }
  if (dw_gate_up != nullptr) out[n++] = dw_gate_up_product(cfg, T, L, t, dw_gate_up, f32, acc);
  if (dw_down != nullptr) out[n++] = dw_down_product(cfg, T, L, t, dw_down, f32, acc);
  if (n == 0) return MOE_OK;
  return run_products(out, n, mlp_params(cfg, kTgStore, nullptr, ws), s, true);
}

// Not part of the interface: how the launches of a call with contiguous 16-bit activations are
// tiled, for the tests that cover every form.  forms: gate_up, down, dh, dx (-1: with the weight
// gradients), the weight gradients (with dx: when it is); a form is a TgShape, or 10 + the CTAs
// that share a tile of few tokens.  Returns 0 if cfg or T is invalid.
int32_t moe_mlp_tilings(const moe_mlp_config_t* cfg, int32_t T, int32_t with_dx, int32_t* forms) {
  if (check_mlp(cfg, T) != MOE_OK || T == 0) return 0;
  const MlpLayout L = mlp_layout(cfg, T);
  const MlpTensors t{nullptr, nullptr, nullptr, nullptr, cfg->hidden, cfg->hidden, nullptr, nullptr};
  auto form = [](const Product* pr, int n, int kind) {
    const Plan p = plan_products(pr, n, kind);
    return p.small ? 10 + p.splits : static_cast<int32_t>(p.shape);
  };
  const Product up = up_product(cfg, T, L, t), down = down_product(cfg, T, L, t, nullptr, cfg->hidden);
  const Product dh = dh_product(cfg, T, L, t, true);
  Product out[3] = {dx_product(cfg, T, L, t, nullptr, cfg->hidden),
                    dw_gate_up_product(cfg, T, L, t, nullptr, 0, 0),
                    dw_down_product(cfg, T, L, t, nullptr, 0, 0)};
  const bool alone = !with_dx || dx_alone(out[0]);
  forms[0] = form(&up, 1, kTgGluFwd);
  forms[1] = form(&down, 1, kTgStore);
  forms[2] = form(&dh, 1, kTgGluBwd);
  forms[3] = with_dx && alone ? form(out, 1, kTgStore) : -1;
  forms[4] = alone ? form(out + 1, 2, kTgStore) : form(out, 3, kTgStore);
  return 1;
}

}  // extern "C"
