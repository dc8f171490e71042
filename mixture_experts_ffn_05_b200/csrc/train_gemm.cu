// The products of the gated MLP's forward and backward passes on the 5th-generation tensor
// cores: C[m][n] = sum_k A[m][k] B[n][k] with 16-bit operands and fp32 sums in tensor memory.
//
//   forward   gate_up  A = x [T][H],       B = Wg, Wu rows     epilogue h = act(g) u, keeps g, u
//             down     A = h [T][D],       B = Wd [H][D]       y
//   backward  dh       A = dy [T][H],      B = Wd as [D][H]^T  epilogue dg, du, h from g, u
//             dx       A = dgu [T][2D],    B = Wgu as [H][2D]^T
//             dWgu     A = dgu^T [2D][T],  B = x^T [H][T]
//             dWd      A = dy^T [H][T],    B = h^T [D][T]
//
// Every operand is read where it lies: one whose rows run along K is a K-major tile, one whose
// rows run along M or N an MN-major tile (the descriptors' major bits), so no transpose is
// ever written.  Rows, columns and K past the end come from TMA as zeros.
//
// A CTA runs a TMA producer warp, an MMA warp and eight epilogue warps (two per quarter of
// the 128 accumulator rows, which take alternate 32-column chunks).  A K step is 64 elements,
// 128 bytes of a 128-byte-swizzled row.  Two accumulators alternate in tensor memory, so a
// tile's epilogue overlaps the next tile's products.  The grid is persistent and the tiles
// are dealt round-robin.
#include "act8.cuh"
#include "train_internal.h"

namespace moe {

constexpr int kTgThreads = 320;  // producer, MMA, 8 epilogue warps
constexpr int kTgEpiWarps = 8;

template <bool PAIR, int BN>
struct TgCfg {
  static constexpr int kBRows = PAIR ? 128 : BN;       // B rows in this CTA's shared memory
  static constexpr int kABytes = 128 * 128;
  static constexpr int kBBytes = kBRows * 128;
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr int kStages = kStage >= 32768 ? 6 : 8;
  static constexpr int kTileM = PAIR ? 256 : 128;      // rows of an item (both CTAs of a pair)
  static constexpr int kAccCols = PAIR ? 256 : BN;     // columns of an accumulator
  static constexpr int kTmemCols = 2 * kAccCols;
  static constexpr int kSmem = 1024 + kStages * kStage + 256;
};

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

__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map,
                                                 uint32_t cluster_bar, int32_t c0, int32_t c1,
                                                 int32_t c2, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(c0), "r"(c1), "r"(c2),
      "l"(policy)
      : "memory");
}

// Each thread of the warp reads 32 consecutive fp32 columns of its TMEM lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  __syncwarp();  // the instruction wants the whole warp; rows past the end left a branch early
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
  // the wait takes the registers as operands so that no use is scheduled before it
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
  asm volatile(""
               : "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]),
                 "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// ---------------------------------------------------------------- the activation
// Both are a = g L(z) with the logistic L(z) = 1 / (1 + exp(-z)): z = g (silu) or
// 2 sqrt(2/pi) (g + 0.044715 g^3) (gelu_tanh, since (1 + tanh w) / 2 = L(2w)).  Then
// a' = L + g L (1 - L) z'.  For gelu_tanh z' is taken at |g| <= 16: beyond, L (1 - L) is 0 in
// fp32 and an unbounded z' would turn it into NaN.
struct Gate {
  float a, da;
};
template <bool WITH_D>
__device__ __forceinline__ Gate gate_of(float g, bool silu) {
  const float c0 = 1.5957691216057308f, c1 = 0.044715f;  // 2 sqrt(2/pi)
  const float z = silu ? g : c0 * fmaf(c1 * g, g * g, g);
  const float l = __fdividef(1.0f, 1.0f + __expf(-z));
  Gate r;
  r.a = g * l;
  r.da = 0.f;
  if (WITH_D) {
    const float gc = fminf(fmaxf(g, -16.f), 16.f);
    const float dz = silu ? 1.f : c0 * fmaf(3.f * c1 * gc, gc, 1.f);
    r.da = fmaf(r.a * (1.f - l), dz, l);
  }
  return r;
}

// ---------------------------------------------------------------- tiles
struct TgTile {
  int p, m, n;
};

// Tiles of a problem in bands of 8 M tiles, M fastest: what runs at one time shares few
// distinct rows of A and of B, which then stay in L2.
constexpr int kBand = 8;
__device__ __forceinline__ TgTile tg_tile(int t, const TgParams& P) {
  TgTile r{0, 0, 0};
  for (; r.p < P.nprob - 1; ++r.p) {
    const int cnt = P.prob[r.p].m_tiles * P.prob[r.p].n_tiles;
    if (t < cnt) break;
    t -= cnt;
  }
  const TgProblem& pr = P.prob[r.p];
  const int band = t / (kBand * pr.n_tiles);
  const int rows = min(kBand, pr.m_tiles - band * kBand);
  const int in = t - band * kBand * pr.n_tiles;
  r.n = in / rows;
  r.m = band * kBand + in - r.n * rows;
  return r;
}

// Stores 8 values as 16 bits.
__device__ __forceinline__ void put8(void* base, int64_t i, const float* f, bool f16) {
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = f[e];
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + i) = f16 ? pack8_f16(v) : pack8(v);
}
__device__ __forceinline__ void get8(const void* base, int64_t i, float* f, bool f16) {
  float v[8];
  const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i);
  if (f16)
    unpack8_f16(u, v);
  else
    unpack8(u, v);
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = v[e];
}

// Kept pre-activations of 32 consecutive features of one half (gate: half 0) of a row.
template <bool INT8>
__device__ __forceinline__ void keep32_8(const TgParams& P, int64_t row, int d, int half, int n,
                                         const float (&v)[32]) {
  const int64_t at = row * P.ld_gu + static_cast<int64_t>(half) * n + d;
  const int b = scale_byte<INT8>(amax_bits(v));  // past n the sums are zero
  const float inv = scale_inverse(b);
  const int groups = (n + kGroup8 - 1) / kGroup8;
  P.gu_scales[row * 2 * groups + half * groups + d / kGroup8] = static_cast<uint8_t>(b);
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (d + 8 * c < n)
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(P.gu) + at + 8 * c) =
          make_uint2(encode4<INT8>(v[8 * c], v[8 * c + 1], v[8 * c + 2], v[8 * c + 3], inv),
                     encode4<INT8>(v[8 * c + 4], v[8 * c + 5], v[8 * c + 6], v[8 * c + 7], inv));
}
__device__ __forceinline__ void keep32(const TgParams& P, int64_t row, int d, int half, int n,
                                       const float (&v)[32]) {
  if (P.gu_fmt == kFmtInt8) {
    keep32_8<true>(P, row, d, half, n, v);
  } else if (P.gu_fmt == kFmtE4m3) {
    keep32_8<false>(P, row, d, half, n, v);
  } else {
    const int64_t at = row * P.ld_gu + static_cast<int64_t>(half) * n + d;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (d + 8 * c < n) put8(P.gu, at + 8 * c, v + 8 * c, P.f16);
  }
}

template <bool INT8>
__device__ __forceinline__ void kept32_8(const TgParams& P, int64_t row, int d, int half, int n,
                                         float (&v)[32]) {
  const int64_t at = row * P.ld_gu + static_cast<int64_t>(half) * n + d;
  const int groups = (n + kGroup8 - 1) / kGroup8;
  const float s = scale_value(P.gu_scales[row * 2 * groups + half * groups + d / kGroup8]);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint2 w = make_uint2(0u, 0u);
    if (d + 8 * c < n)
      w = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(P.gu) + at + 8 * c);
    decode4<INT8>(w.x, s, v + 8 * c);
    decode4<INT8>(w.y, s, v + 8 * c + 4);
  }
}
__device__ __forceinline__ void kept32(const TgParams& P, int64_t row, int d, int half, int n,
                                       float (&v)[32]) {
  if (P.gu_fmt == kFmtInt8) {
    kept32_8<true>(P, row, d, half, n, v);
  } else if (P.gu_fmt == kFmtE4m3) {
    kept32_8<false>(P, row, d, half, n, v);
  } else {
    const int64_t at = row * P.ld_gu + static_cast<int64_t>(half) * n + d;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[8 * c + e] = 0.f;
      if (d + 8 * c < n) get8(P.gu, at + 8 * c, v + 8 * c, P.f16);
    }
  }
}

// ---------------------------------------------------------------- the kernel
template <bool PAIR, int BN, int KIND>
__global__ void __launch_bounds__(kTgThreads, 1)
    train_gemm_kernel(const __grid_constant__ TgMaps maps, const __grid_constant__ TgParams P) {
  using C = TgCfg<PAIR, BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStage);
  uint64_t* empty = full + C::kStages;
  uint64_t* acc_full = empty + C::kStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  const int first = PAIR ? static_cast<int>(blockIdx.x >> 1) : static_cast<int>(blockIdx.x);
  const int stride = PAIR ? static_cast<int>(gridDim.x >> 1) : static_cast<int>(gridDim.x);
  int total = 0;
  for (int i = 0; i < P.nprob; ++i) total += P.prob[i].m_tiles * P.prob[i].n_tiles;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], (PAIR ? 2 : 1) * kTgEpiWarps);  // both CTAs' epilogues
    }
    mbar_init(drain, 1);
    mbar_fence_init();
    *abort_flag = 0;
    for (int i = 0; i < P.nprob; ++i) {
      tma_prefetch_map(&maps.a[i]);
      tma_prefetch_map(&maps.b[i]);
    }
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(tmem_slot, C::kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, C::kTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();  // the peer's barriers are ready before either CTA signals them
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint64_t tmo = P.timeout_ns;
  // Setup overlaps the previous kernel's tail; nothing of its results is touched before.
  pdl_wait();
  pdl_trigger();

  if (warp == 0) {
    // ================= TMA producer =================
    if (lane == 0) {
      const uint64_t pol = policy_evict_last();
      int stage = 0;
      uint32_t phase = 0;
      int armed[C::kStages];
      for (int i = 0; i < C::kStages; ++i) armed[i] = -1;
      bool ok = true;
      for (int t = first; t < total && ok; t += stride) {
        const TgTile tl = tg_tile(t, P);
        const TgProblem& pr = P.prob[tl.p];
        const CUtensorMap* ma = &maps.a[tl.p];
        const CUtensorMap* mb = &maps.b[tl.p];
        const int m0 = tl.m * C::kTileM + static_cast<int>(rank) * 128;
        // GLU forward: the tile's columns are BN / 2 features, gate and up rows of each
        const int n0 = KIND == kTgGluFwd ? tl.n * (BN / 2)
                                         : tl.n * BN + (PAIR ? static_cast<int>(rank) * 128 : 0);
        for (int ks = 0; ks < pr.k_steps; ++ks) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, tmo, abort_flag)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + stage * C::kStage;
          uint8_t* sb = sa + C::kABytes;
          const int k0 = ks * 64;
          if (!PAIR || leader) mbar_arrive_expect_tx(&full[stage], (PAIR ? 2 : 1) * C::kStage);
          const uint32_t fb = PAIR ? cluster_addr(&full[stage], 0) : 0u;
          auto load2 = [&](uint8_t* dst, const CUtensorMap* m, int c0, int c1) {
            if (PAIR)
              tma_load_2d_pair(dst, m, fb, c0, c1, pol);
            else
              tma_load_2d(dst, m, &full[stage], c0, c1, pol);
          };
          if (pr.a_mn) {
#pragma unroll
            for (int j = 0; j < 2; ++j) load2(sa + j * 8192, ma, m0 + 64 * j, k0);
          } else {
            load2(sa, ma, k0, m0);
          }
          if constexpr (KIND == kTgGluFwd) {
            if (PAIR) {  // this CTA's half of B: gate rows in the leader, up rows in its peer
              tma_load_3d_pair(sb, mb, fb, k0, n0, static_cast<int>(rank), pol);
            } else {
              tma_load_3d(sb, mb, &full[stage], k0, n0, 0, pol);
              tma_load_3d(sb + C::kBBytes / 2, mb, &full[stage], k0, n0, 1, pol);
            }
          } else if (pr.b_mn) {
#pragma unroll
            for (int j = 0; j < C::kBRows / 64; ++j) load2(sb + j * 8192, mb, n0 + 64 * j, k0);
          } else {
            load2(sb, mb, k0, n0);
          }
          armed[stage] = static_cast<int>(phase);
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        record_status(P.status, kStatusTimeout);
        *abort_flag = 1;
        // every copy already issued lands before the CTA winds down (PAIR: the leader's
        // barriers count both CTAs' copies)
        if (!PAIR || leader)
          for (int i = 0; i < C::kStages; ++i)
            if (armed[i] >= 0) mbar_wait(&full[i], static_cast<uint32_t>(armed[i]), tmo, nullptr);
      }
    }
  } else if (warp == 1) {
    // ================= MMA issuer (PAIR: the leader's, for both CTAs) =================
    if (lane == 0 && leader) {
      int stage = 0;
      uint32_t phase = 0;
      int ab = 0;
      uint32_t aph = 0;
      bool ok = true, issued = false;
      const uint32_t peer_empty0 = PAIR ? cluster_addr(&empty[0], 1) : 0u;
      const uint32_t peer_acc0 = PAIR ? cluster_addr(&acc_full[0], 1) : 0u;
      for (int t = first; t < total && ok; t += stride) {
        const TgTile tl = tg_tile(t, P);
        const TgProblem& pr = P.prob[tl.p];
        const uint32_t idesc = (P.f16 ? idesc_f16_f32(C::kTileM, BN) : idesc_bf16_f32(C::kTileM, BN)) |
                               (pr.a_mn ? 1u << 15 : 0u) | (pr.b_mn ? 1u << 16 : 0u);
        // 16 K elements: 32 bytes along a K-major row, 16 rows of 128 bytes MN-major
        const uint64_t astep = pr.a_mn ? 2048 >> 4 : 32 >> 4;
        const uint64_t bstep = pr.b_mn ? 2048 >> 4 : 32 >> 4;
        if (!mbar_wait(&acc_empty[ab], aph ^ 1u, tmo, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + static_cast<uint32_t>(ab * C::kAccCols);
        for (int ks = 0; ks < pr.k_steps; ++ks) {
          if (!mbar_wait(&full[stage], phase, tmo, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + stage * C::kStage);
          uint64_t ad = pr.a_mn ? sdesc_mn_sw128(sa) : sdesc_k_sw128(sa);
          uint64_t bd = pr.b_mn ? sdesc_mn_sw128(sa + C::kABytes) : sdesc_k_sw128(sa + C::kABytes);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint32_t acc = (ks > 0 || kk > 0) ? 1u : 0u;
            if (PAIR)
              umma_bf16_pair(d, ad, bd, idesc, acc);
            else
              umma_bf16(d, ad, bd, idesc, acc);
            ad += astep;
            bd += bstep;
          }
          if (PAIR) {
            umma_commit_pair(smem_u32(&empty[stage]));
            umma_commit_pair(peer_empty0 + stage * 8);
          } else {
            umma_commit(&empty[stage]);
          }
          issued = true;
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (PAIR) {
          umma_commit_pair(smem_u32(&acc_full[ab]));
          umma_commit_pair(peer_acc0 + ab * 8);
        } else {
          umma_commit(&acc_full[ab]);
        }
        ab ^= 1;
        if (ab == 0) aph ^= 1u;
      }
      if (!ok) {
        record_status(P.status, kStatusTimeout);
        *abort_flag = 1;
        if (issued) {  // the MMAs in flight end before TMEM is released
          if (PAIR)
            umma_commit_pair(smem_u32(drain));
          else
            umma_commit(drain);
          mbar_wait(drain, 0, tmo, nullptr);
        }
      }
    }
  } else {
    // ================= epilogue =================
    const int grp = (warp - 2) >> 2;  // takes chunks grp, grp + 2, ...
    const int q = warp & 3;           // TMEM lane quarter
    int ab = 0;
    uint32_t aph = 0;
    for (int t = first; t < total; t += stride) {
      const TgTile tl = tg_tile(t, P);
      const TgProblem& pr = P.prob[tl.p];
      int good = 1;
      if (lane == 0) good = mbar_wait(&acc_full[ab], aph, tmo, abort_flag) ? 1 : 0;
      good = __shfl_sync(0xffffffffu, good, 0);
      if (!good) {
        if (lane == 0) {
          record_status(P.status, kStatusTimeout);
          *abort_flag = 1;
        }
        break;
      }
      tc_fence_after();
      const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                             static_cast<uint32_t>(ab * C::kAccCols);
      const int row = tl.m * C::kTileM + static_cast<int>(rank) * 128 + q * 32 + lane;
      const bool live = row < pr.m;
      if constexpr (KIND == kTgGluFwd) {
        for (int c = grp; c < BN / 64; c += 2) {
          const int d = tl.n * (BN / 2) + 32 * c;  // first feature of the chunk
          if (d >= pr.n) break;
          float g[32], u[32];
          tmem_ld32(tbase + 32 * c, g);
          tmem_ld32(tbase + BN / 2 + 32 * c, u);
          if (!live) continue;
          if (P.gu != nullptr) {
            keep32(P, row, d, 0, pr.n, g);
            keep32(P, row, d, 1, pr.n, u);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) g[e] = gate_of<false>(g[e], P.silu).a * u[e];
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (d + 8 * v < pr.n) put8(pr.out, row * pr.ld_out + d + 8 * v, g + 8 * v, P.f16);
        }
      } else if constexpr (KIND == kTgGluBwd) {
        for (int c = grp; c < BN / 32; c += 2) {
          const int d = tl.n * BN + 32 * c;
          if (d >= pr.n) break;
          float dh[32];
          tmem_ld32(tbase + 32 * c, dh);
          if (!live) continue;
          float g[32], u[32];
          kept32(P, row, d, 0, pr.n, g);
          kept32(P, row, d, 1, pr.n, u);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const Gate ga = gate_of<true>(g[e], P.silu);
            const float uu = u[e];
            g[e] = dh[e] * uu * ga.da;  // dg
            u[e] = dh[e] * ga.a;        // du
            dh[e] = ga.a * uu;          // h
          }
          const int64_t at = static_cast<int64_t>(row) * 2 * pr.n + d;
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (d + 8 * v < pr.n) {
              put8(P.dgu, at + 8 * v, g + 8 * v, P.f16);
              put8(P.dgu, at + pr.n + 8 * v, u + 8 * v, P.f16);
              if (pr.out != nullptr) put8(pr.out, row * pr.ld_out + d + 8 * v, dh + 8 * v, P.f16);
            }
        }
      } else {
        for (int c = grp; c < BN / 32; c += 2) {
          const int n = tl.n * BN + 32 * c;
          if (n >= pr.n) break;
          float v[32];
          tmem_ld32(tbase + 32 * c, v);
          if (!live) continue;
          const int64_t at = row * pr.ld_out + n;
          if (pr.out_f32) {
            float* o = static_cast<float*>(pr.out) + at;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (n + 4 * k < pr.n) {
                float4 w = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                if (pr.accumulate) {
                  const float4 old = *reinterpret_cast<const float4*>(o + 4 * k);
                  w.x += old.x; w.y += old.y; w.z += old.z; w.w += old.w;
                }
                *reinterpret_cast<float4*>(o + 4 * k) = w;
              }
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (n + 8 * k < pr.n) {
                if (pr.accumulate) {
                  float old[8];
                  get8(pr.out, at + 8 * k, old, P.f16);
#pragma unroll
                  for (int e = 0; e < 8; ++e) v[8 * k + e] += old[e];
                }
                put8(pr.out, at + 8 * k, v + 8 * k, P.f16);
              }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR)
          mbar_arrive_cluster(cluster_addr(&acc_empty[ab], 0));  // the leader's MMA waits
        else
          mbar_arrive(&acc_empty[ab]);
      }
      ab ^= 1;
      if (ab == 0) aph ^= 1u;
    }
  }

  // ---- teardown: neither CTA of a pair releases TMEM or exits while its peer may still
  // signal it or read its shared memory
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    if (PAIR)
      tmem_dealloc_pair(tmem_base, C::kTmemCols);
    else
      tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

template <bool PAIR, int BN, int KIND>
static cudaError_t launch_tg(const TgMaps& maps, const TgParams& p, int sms, cudaStream_t s,
                             bool pdl) {
  using C = TgCfg<PAIR, BN>;
  auto kernel = train_gemm_kernel<PAIR, BN, KIND>;
  cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  int64_t tiles = 0;
  for (int i = 0; i < p.nprob; ++i)
    tiles += static_cast<int64_t>(p.prob[i].m_tiles) * p.prob[i].n_tiles;
  const int64_t ctas = PAIR ? 2 * tiles : tiles;
  int grid = static_cast<int>(ctas < sms ? ctas : sms);
  if (!PAIR) return launch_k(kernel, dim3(grid), dim3(kTgThreads), C::kSmem, s, pdl, maps, p);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid & ~1);
  cfg.blockDim = dim3(kTgThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, maps, p);
}

template <int KIND>
static cudaError_t launch_kind(TgShape shape, const TgMaps& maps, const TgParams& p, int sms,
                               cudaStream_t s, bool pdl) {
  switch (shape) {
    case kTgPair256: return launch_tg<true, 256, KIND>(maps, p, sms, s, pdl);
    case kTgOne128: return launch_tg<false, 128, KIND>(maps, p, sms, s, pdl);
    case kTgOne64: return launch_tg<false, 64, KIND>(maps, p, sms, s, pdl);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_train_gemm(TgShape shape, const TgMaps& maps, const TgParams& p, int sms,
                              cudaStream_t s, bool pdl) {
  switch (p.kind) {
    case kTgStore: return launch_kind<kTgStore>(shape, maps, p, sms, s, pdl);
    case kTgGluFwd: return launch_kind<kTgGluFwd>(shape, maps, p, sms, s, pdl);
    case kTgGluBwd: return launch_kind<kTgGluBwd>(shape, maps, p, sms, s, pdl);
  }
  return cudaErrorInvalidValue;
}

}  // namespace moe
