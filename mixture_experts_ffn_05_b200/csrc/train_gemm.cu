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
#include "train_internal.h"
#include "train_tile.cuh"

namespace moe {

constexpr int kTgThreads = 320;  // producer, MMA, 8 epilogue warps
constexpr int kTgEpiWarps = 8;
constexpr int kTgWarpStage = 4096;  // bytes in which an epilogue warp turns its chunk around

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
  static constexpr int kSmem = 1024 + kStages * kStage + kTgEpiWarps * kTgWarpStage + 256;
};

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

// Arrival that orders no memory: a released accumulator was read with tcgen05.ld and its wait,
// while a releasing arrival would first wait for the tile's global stores (2 to 3 K cycles).
__device__ __forceinline__ void mbar_arrive_relaxed(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
               : "memory");
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

// ---------------------------------------------------------------- an epilogue warp's chunk
// A warp holds 32 rows x 32 columns of an accumulator, one row a lane.  Global memory is read
// and written through a stage of the warp's own in shared memory, so that neighbouring lanes
// touch neighbouring bytes: 8 rows of 64 bytes an instruction for 16-bit values.  (With each
// lane on its own row an instruction touched 32 lines by half a sector, and the epilogue of
// the dh product took 54 K cycles a tile against 32 K of the tile's MMAs.)
// 16-byte pieces of a row are exchanged by a few bits of the row so that both sides are free
// of bank conflicts.
__device__ __forceinline__ int stage16(int row, int piece) { return row * 4 + (piece ^ ((row >> 1) & 3)); }
__device__ __forceinline__ int stage32(int row, int piece) { return row * 8 + (piece ^ (row & 7)); }

struct Chunk {
  int lane, row0, m, col, n;  // first row, rows of the output; first column, columns
  // the place of access k (of 4) in a chunk of four pieces a row
  __device__ __forceinline__ int row(int k) const { return 8 * k + (lane >> 2); }
  __device__ __forceinline__ int piece() const { return lane & 3; }
  __device__ __forceinline__ bool in(int k) const {
    return row0 + row(k) < m && col + 8 * piece() < n;
  }
  // of access 0, in elements; each next one is 8 rows on
  __device__ __forceinline__ int64_t first(int64_t ld) const {
    return static_cast<int64_t>(row0 + (lane >> 2)) * ld + col + 8 * piece();
  }
};

// base: the output's column 0; ld elements.
template <bool F16>
__device__ __forceinline__ void put16(uint4* stage, const Chunk& c, void* base, int64_t ld,
                                      const float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) stage[stage16(c.lane, i)] = pack16<F16>(v + 8 * i);
  __syncwarp();
  uint16_t* out = static_cast<uint16_t*>(base) + c.first(ld);
  uint4 w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = stage[stage16(c.row(k), c.piece())];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (c.in(k)) *reinterpret_cast<uint4*>(out) = w[k];
    out += 8 * ld;
  }
  __syncwarp();
}

// fp32 outputs, and sums to 16- or 32-bit ones (rounded once).
template <bool F16>
__device__ __forceinline__ void put32(uint4* stage, const Chunk& c, void* base, int64_t ld,
                                      const float (&v)[32], bool f32, bool add) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<float4*>(stage + stage32(c.lane, i)) =
        make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  __syncwarp();
  const int piece = c.lane & 7;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int r = 4 * k + (c.lane >> 3);
    if (c.row0 + r >= c.m || c.col + 4 * piece >= c.n) continue;
    float4 w = *reinterpret_cast<const float4*>(stage + stage32(r, piece));
    const int64_t at = static_cast<int64_t>(c.row0 + r) * ld + c.col + 4 * piece;
    if (f32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
      if (add) {
        const float4 old = *o;
        w.x += old.x; w.y += old.y; w.z += old.z; w.w += old.w;
      }
      *o = w;
    } else {
      uint2* o = reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + at);
      const uint2 old = *o;
      float t[8];
      unpack16<F16>(make_uint4(old.x, old.y, 0u, 0u), t);
      w.x += t[0]; w.y += t[1]; w.z += t[2]; w.w += t[3];
      *o = make_uint2(pack_two<F16>(w.x, w.y), pack_two<F16>(w.z, w.w));
    }
  }
  __syncwarp();
}

// Kept pre-activations of one half (gate: 0, up: 1): columns col.. of n.
template <bool INT8>
__device__ __forceinline__ void keep8(const TgParams& P, uint4* stage4, const Chunk& c, int half,
                                      const float (&v)[32]) {
  uint2* stage = reinterpret_cast<uint2*>(stage4);
  const int b = scale_byte<INT8>(amax_bits(v));  // past n the sums are zero
  const float inv = scale_inverse(b);
  const int groups = (c.n + kGroup8 - 1) / kGroup8;
  if (c.row0 + c.lane < c.m)
    P.gu_scales[(static_cast<int64_t>(c.row0 + c.lane) * 2 + half) * groups + c.col / kGroup8] =
        static_cast<uint8_t>(b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float* f = v + 8 * i;
    stage[stage16(c.lane, i)] = make_uint2(encode4<INT8>(f[0], f[1], f[2], f[3], inv),
                                           encode4<INT8>(f[4], f[5], f[6], f[7], inv));
  }
  __syncwarp();
  uint8_t* out = static_cast<uint8_t*>(P.gu) + c.first(P.ld_gu) + static_cast<int64_t>(half) * c.n;
  uint2 w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = stage[stage16(c.row(k), c.piece())];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (c.in(k)) *reinterpret_cast<uint2*>(out) = w[k];
    out += 8 * P.ld_gu;
  }
  __syncwarp();
}
template <bool F16>
__device__ __forceinline__ void keep(const TgParams& P, uint4* stage, const Chunk& c, int half,
                                     const float (&v)[32]) {
  if (P.gu_fmt == kFmtInt8)
    keep8<true>(P, stage, c, half, v);
  else if (P.gu_fmt == kFmtE4m3)
    keep8<false>(P, stage, c, half, v);
  else
    put16<F16>(stage, c, static_cast<uint16_t*>(P.gu) + static_cast<int64_t>(half) * c.n, P.ld_gu, v);
}

// The same read back: requested (early, into registers) and turned into rows.
struct Kept {
  uint4 p[4];  // 8-bit formats: the low halves
  int scale;
};
__device__ __forceinline__ Kept request_kept(const TgParams& P, const Chunk& c, int half) {
  Kept r;
  const int64_t at = c.first(P.ld_gu) + static_cast<int64_t>(half) * c.n, step = 8 * P.ld_gu;
  r.scale = 1;
  if (fmt_bytes(P.gu_fmt) == 1) {
    const uint8_t* p = static_cast<const uint8_t*>(P.gu) + at;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint2 w = c.in(k) ? *reinterpret_cast<const uint2*>(p) : make_uint2(0u, 0u);
      r.p[k] = make_uint4(w.x, w.y, 0u, 0u);
      p += step;
    }
    const int groups = (c.n + kGroup8 - 1) / kGroup8;
    if (c.row0 + c.lane < c.m)
      r.scale = P.gu_scales[(static_cast<int64_t>(c.row0 + c.lane) * 2 + half) * groups +
                            c.col / kGroup8];
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(P.gu) + at;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      r.p[k] = c.in(k) ? *reinterpret_cast<const uint4*>(p) : make_uint4(0u, 0u, 0u, 0u);
      p += step;
    }
  }
  return r;
}
template <bool F16>
__device__ __forceinline__ void read_kept(const TgParams& P, uint4* stage, const Chunk& c,
                                          const Kept& r, float (&v)[32]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) stage[stage16(c.row(k), c.piece())] = r.p[k];
  __syncwarp();
  uint4 w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = stage[stage16(c.lane, i)];
  __syncwarp();
  if (fmt_bytes(P.gu_fmt) != 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack16<F16>(w[i], v + 8 * i);
    return;
  }
  const float s = scale_value(r.scale);
  if (P.gu_fmt == kFmtInt8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      decode4<true>(w[i].x, s, v + 8 * i);
      decode4<true>(w[i].y, s, v + 8 * i + 4);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      decode4<false>(w[i].x, s, v + 8 * i);
      decode4<false>(w[i].y, s, v + 8 * i + 4);
    }
  }
}

// The epilogues hold 32 columns of up to three matrices; that of dh spills 12 bytes a thread.
// h = act(g) u, over g.
template <bool SILU>
__device__ __forceinline__ void glu_forward(float (&g)[32], const float (&u)[32]) {
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const Gate2 ga = gate_of<false, SILU>(pair_of(g[e], g[e + 1]));
    of_pair(mul2(ga.a, pair_of(u[e], u[e + 1])), g[e], g[e + 1]);
  }
}
// dg, du and h over g, u and dh.
template <bool SILU>
__device__ __forceinline__ void glu_backward(float (&dh)[32], float (&g)[32], float (&u)[32]) {
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const Gate2 ga = gate_of<true, SILU>(pair_of(g[e], g[e + 1]));
    const uint64_t d = pair_of(dh[e], dh[e + 1]), uu = pair_of(u[e], u[e + 1]);
    of_pair(mul2(mul2(d, uu), ga.da), g[e], g[e + 1]);
    of_pair(mul2(d, ga.a), u[e], u[e + 1]);
    of_pair(mul2(ga.a, uu), dh[e], dh[e + 1]);
  }
}

// ---------------------------------------------------------------- the kernel
template <bool PAIR, int BN, int KIND, bool F16>
__global__ void __launch_bounds__(kTgThreads, 1)
    train_gemm_kernel(const __grid_constant__ TgMaps maps, const __grid_constant__ TgParams P) {
  using C = TgCfg<PAIR, BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStage +
                                               kTgEpiWarps * kTgWarpStage);
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
    if (elect_one()) {
      const uint64_t pol = policy_evict_last();
      int stage = 0;
      uint32_t phase = 0;
      int64_t fills = 0;
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
        const int k_steps = pr.k_steps;
        const bool a_mn = pr.a_mn, b_mn = pr.b_mn;
        for (int ks = 0; ks < k_steps; ++ks) {
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
          if (a_mn) {
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
          } else if (b_mn) {
#pragma unroll
            for (int j = 0; j < C::kBRows / 64; ++j) load2(sb + j * 8192, mb, n0 + 64 * j, k0);
          } else {
            load2(sb, mb, k0, n0);
          }
          ++fills;
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
          for (int64_t i = fills > C::kStages ? fills - C::kStages : 0; i < fills; ++i)
            mbar_wait(&full[i % C::kStages], static_cast<uint32_t>(i / C::kStages) & 1u, tmo, nullptr);
      }
    }
  } else if (warp == 1) {
    // ================= MMA issuer (PAIR: the leader's, for both CTAs) =================
    if (leader && elect_one()) {
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
        const int k_steps = pr.k_steps;
        const bool a_mn = pr.a_mn, b_mn = pr.b_mn;
        const uint32_t idesc = (F16 ? idesc_f16_f32(C::kTileM, BN) : idesc_bf16_f32(C::kTileM, BN)) |
                               (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
        // 16 K elements: 32 bytes along a K-major row, 16 rows of 128 bytes MN-major
        const uint64_t astep = a_mn ? 2048 >> 4 : 32 >> 4;
        const uint64_t bstep = b_mn ? 2048 >> 4 : 32 >> 4;
        if (!mbar_wait(&acc_empty[ab], aph ^ 1u, tmo, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + static_cast<uint32_t>(ab * C::kAccCols);
        for (int ks = 0; ks < k_steps; ++ks) {
          if (!mbar_wait(&full[stage], phase, tmo, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + stage * C::kStage);
          uint64_t ad = a_mn ? sdesc_mn_sw128(sa) : sdesc_k_sw128(sa);
          uint64_t bd = b_mn ? sdesc_mn_sw128(sa + C::kABytes) : sdesc_k_sw128(sa + C::kABytes);
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
    uint4* stage = reinterpret_cast<uint4*>(smem + C::kStages * C::kStage +
                                            (warp - 2) * kTgWarpStage);
    int ab = 0;
    uint32_t aph = 0;
    for (int t = first; t < total; t += stride) {
      const TgTile tl = tg_tile(t, P);
      const TgProblem& pr = P.prob[tl.p];
      const int row0 = tl.m * C::kTileM + static_cast<int>(rank) * 128 + q * 32;
      const int n0 = tl.n * (KIND == kTgGluFwd ? BN / 2 : BN);
      const int chunks = row0 < pr.m ? min(KIND == kTgGluFwd ? BN / 64 : BN / 32, (pr.n - n0 + 31) / 32) : 0;
      Kept kg, ku;
      if constexpr (KIND == kTgGluBwd) {  // under way while the tile's products end
        if (grp < chunks) {
          const Chunk c{lane, row0, pr.m, n0 + 32 * grp, pr.n};
          kg = request_kept(P, c, 0);
          ku = request_kept(P, c, 1);
        }
      }
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
      // the leader's MMA waits for all epilogue warps of both CTAs; each releases the accumulator
      // when it has read its last chunk, before it stores it
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed(cluster_addr(&acc_empty[ab], 0));
      };
      for (int i = grp; i < chunks; i += 2) {
        const bool last = i + 2 >= chunks;
        const Chunk c{lane, row0, pr.m, n0 + 32 * i, pr.n};
        if constexpr (KIND == kTgGluFwd) {
          float g[32], u[32];
          tmem_ld32(tbase + 32 * i, g);
          tmem_ld32(tbase + BN / 2 + 32 * i, u);
          if (last) release();
          if (P.gu != nullptr) {
            keep<F16>(P, stage, c, 0, g);
            keep<F16>(P, stage, c, 1, u);
          }
          if (P.silu)
            glu_forward<true>(g, u);
          else
            glu_forward<false>(g, u);
          put16<F16>(stage, c, pr.out, pr.ld_out, g);
        } else if constexpr (KIND == kTgGluBwd) {
          float dh[32], g[32], u[32];
          read_kept<F16>(P, stage, c, kg, g);
          read_kept<F16>(P, stage, c, ku, u);
          if (!last) {
            const Chunk next{lane, row0, pr.m, c.col + 64, pr.n};
            kg = request_kept(P, next, 0);
            ku = request_kept(P, next, 1);
          }
          tmem_ld32(tbase + 32 * i, dh);
          if (last) release();
          if (P.silu)
            glu_backward<true>(dh, g, u);
          else
            glu_backward<false>(dh, g, u);
          put16<F16>(stage, c, P.dgu, P.ld_dgu, g);
          put16<F16>(stage, c, static_cast<uint16_t*>(P.dgu) + pr.n, P.ld_dgu, u);
          if (pr.out != nullptr) put16<F16>(stage, c, pr.out, pr.ld_out, dh);
        } else {
          float v[32];
          tmem_ld32(tbase + 32 * i, v);
          if (last) release();
          if (pr.out_f32 || pr.accumulate)
            put32<F16>(stage, c, pr.out, pr.ld_out, v, pr.out_f32, pr.accumulate);
          else
            put16<F16>(stage, c, pr.out, pr.ld_out, v);
        }
      }
      if (grp >= chunks) release();
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

template <bool PAIR, int BN, int KIND, bool F16>
static cudaError_t launch_tg(const TgMaps& maps, const TgParams& p, int sms, cudaStream_t s,
                             bool pdl) {
  using C = TgCfg<PAIR, BN>;
  auto kernel = train_gemm_kernel<PAIR, BN, KIND, F16>;
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

template <int KIND, bool F16>
static cudaError_t launch_shape(TgShape shape, const TgMaps& maps, const TgParams& p, int sms,
                               cudaStream_t s, bool pdl) {
  switch (shape) {
    case kTgPair256: return launch_tg<true, 256, KIND, F16>(maps, p, sms, s, pdl);
    case kTgOne128: return launch_tg<false, 128, KIND, F16>(maps, p, sms, s, pdl);
    case kTgOne64: return launch_tg<false, 64, KIND, F16>(maps, p, sms, s, pdl);
  }
  return cudaErrorInvalidValue;
}

template <int KIND>
static cudaError_t launch_kind(TgShape shape, const TgMaps& maps, const TgParams& p, int sms,
                               cudaStream_t s, bool pdl) {
  return p.f16 ? launch_shape<KIND, true>(shape, maps, p, sms, s, pdl)
               : launch_shape<KIND, false>(shape, maps, p, sms, s, pdl);
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
