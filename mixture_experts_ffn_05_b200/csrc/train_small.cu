// The products of the gated MLP for few tokens, where the weights' bytes and the latency of the
// K loop bind and not the tensor cores: C[t][f] = sum_k X[t][k] W[f][k] with the weights as the
// M operand (128 features a tile, every TMEM lane in use) and up to 128 tokens as N.
//
// A cluster of 1, 2, 4 or 8 CTAs shares a tile and splits its K steps, so that the weights of
// one product stream through all SMs at once; with whole K loops 66 CTAs of 44 steps took 21 us
// for the 24 MB of a gate_up product at 8 tokens.  Each CTA leaves its fp32 sums in its own
// shared memory as [token][128 features]; the CTAs then take tokens in turn, add the partial
// sums in a fixed order through distributed shared memory and apply the epilogue,
// four neighbouring features a lane, so that a warp writes 128 to 256 contiguous bytes.
//
// Weights do not depend on the kernel before: the first ring fill requests them before the
// dependency wait.
#include "train_internal.h"
#include "train_tile.cuh"

namespace moe {

constexpr int kTsThreads = 320;        // producer, MMA, 8 epilogue warps
constexpr int kTsWeightBytes = 16384;  // 128 features x 64 K elements
// Ring bytes: up to 64 tokens two CTAs fit an SM, so that the next product's weights come in
// while this one runs; above, the tokens' bytes count as much as the weights' and a deep ring
// more (256 tokens, 2816 x 2112, forward: 23.4 us, 27.0 us with half of it).
constexpr int ts_ring(int nt) { return (nt <= 64 ? 108 : 192) * 1024; }

// The cluster barrier in two parts, for a thread at a time.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
constexpr int kTsMaxStages = 8;

// N tokens' sums of four neighbouring features over the cluster's CTAs; `mine` + i * `step`
// floats is token i's place.  All loads are under way at once, and each CTA begins with its own
// sums, so that the cluster does not read one CTA's memory all at a time (in rank order the
// sums of 64 tokens over 8 CTAs took 7 us).  A token is always summed by the same rank, so the
// order is fixed.
template <int SPLITS, int N>
__device__ __forceinline__ void cluster_sums(float (&v)[N][4], const float* mine, int step,
                                             int count, uint32_t rank) {
  float p[SPLITS][N][4];
#pragma unroll
  for (int c = 0; c < SPLITS; ++c) {
    const uint32_t from = cluster_addr(mine, (rank + c) % SPLITS);
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) p[c][i][e] = 0.f;
      if (i < count)
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(p[c][i][0]), "=f"(p[c][i][1]), "=f"(p[c][i][2]), "=f"(p[c][i][3])
                     : "r"(from + static_cast<uint32_t>(i * step * 4))
                     : "memory");
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[i][e] = p[0][i][e];
#pragma unroll
      for (int c = 1; c < SPLITS; ++c) v[i][e] += p[c][i][e];
    }
}

__device__ __forceinline__ void put4(void* base, int64_t i, const float (&v)[4], bool f16) {
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + i) =
      f16 ? make_uint2(pack2_f16(v[0], v[1]), pack2_f16(v[2], v[3]))
          : make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
}

__device__ __forceinline__ uint64_t gate_act(uint64_t g, bool silu) {
  return silu ? gate_of<false, true>(g).a : gate_of<false, false>(g).a;
}

// A group of 32 features is eight lanes' four values; every lane takes part.
template <bool INT8>
__device__ __forceinline__ void keep4(const TgParams& P, const float (&v)[4], int64_t row, int half,
                                      int f, int n, bool live) {
  uint32_t m = amax_bits(v);
#pragma unroll
  for (int o = 1; o < 8; o *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  const int b = scale_byte<INT8>(m);
  if (!live) return;
  const int groups = (n + kGroup8 - 1) / kGroup8;
  if (f % kGroup8 == 0)
    P.gu_scales[(row * 2 + half) * groups + f / kGroup8] = static_cast<uint8_t>(b);
  *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(P.gu) + row * P.ld_gu +
                               static_cast<int64_t>(half) * n + f) =
      encode4<INT8>(v[0], v[1], v[2], v[3], scale_inverse(b));
}

__device__ __forceinline__ void kept4(const TgParams& P, float (&v)[4], int64_t row, int half, int f,
                                      int n) {
  const int64_t at = row * P.ld_gu + static_cast<int64_t>(half) * n + f;
  if (fmt_bytes(P.gu_fmt) == 1) {
    const int groups = (n + kGroup8 - 1) / kGroup8;
    const float s = scale_value(P.gu_scales[(row * 2 + half) * groups + f / kGroup8]);
    const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(P.gu) + at);
    if (P.gu_fmt == kFmtInt8)
      decode4<true>(w, s, v);
    else
      decode4<false>(w, s, v);
    return;
  }
  const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(P.gu) + at);
  float t[8];
  if (P.f16)
    unpack8_f16(make_uint4(w.x, w.y, 0u, 0u), t);
  else
    unpack8(make_uint4(w.x, w.y, 0u, 0u), t);
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = t[e];
}

template <int KIND, int SPLITS>
__global__ void __launch_bounds__(kTsThreads, 2)
    train_small_kernel(const __grid_constant__ TgMaps maps, const __grid_constant__ TgParams P,
                       int nt, int stages) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ uint64_t full[kTsMaxStages], empty[kTsMaxStages], done[1];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const TgProblem& pr = P.prob[0];
  const int stage_bytes = kTsWeightBytes + nt * 128;
  constexpr int kBatch = SPLITS >= 4 ? 2 : 4;  // tokens a warp sums at a time
  const uint32_t rank = cluster_ctarank();
  const int tile = static_cast<int>(blockIdx.x / SPLITS);
  const int fb = tile % pr.n_tiles, tb = tile / pr.n_tiles;  // feature and token tile
  const int k_first = pr.k_steps * static_cast<int>(rank) / SPLITS;
  const int k_end = pr.k_steps * static_cast<int>(rank + 1) / SPLITS;
  const int steps = k_end - k_first;
  const uint32_t cols = nt <= 32 ? 32 : nt <= 64 ? 64 : 128;  // TMEM columns

  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(done, 1);
    mbar_fence_init();
    abort_flag = 0;
    tma_prefetch_map(&maps.a[0]);
    tma_prefetch_map(&maps.b[0]);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  const uint64_t tmo = P.timeout_ns;
  pdl_trigger();

  if (warp == 0) {
    // ================= TMA producer =================
    if (elect_one()) {
      const uint64_t keep_w = policy_evict_first(), keep_x = policy_evict_last();
      const bool w_mn = pr.b_mn;
      auto weights = [&](int k, int s) {
        uint8_t* dst = smem + s * stage_bytes;
        const int k0 = (k_first + k) * 64;
        mbar_arrive_expect_tx(&full[s], stage_bytes);
        if constexpr (KIND == kTgGluFwd) {
          tma_load_3d(dst, &maps.b[0], &full[s], k0, fb * 64, 0, keep_w);
          tma_load_3d(dst + kTsWeightBytes / 2, &maps.b[0], &full[s], k0, fb * 64, 1, keep_w);
        } else if (w_mn) {
          tma_load_2d(dst, &maps.b[0], &full[s], fb * 128, k0, keep_w);
          tma_load_2d(dst + kTsWeightBytes / 2, &maps.b[0], &full[s], fb * 128 + 64, k0, keep_w);
        } else {
          tma_load_2d(dst, &maps.b[0], &full[s], k0, fb * 128, keep_w);
        }
      };
      auto tokens = [&](int k, int s) {
        tma_load_2d(smem + s * stage_bytes + kTsWeightBytes, &maps.a[0], &full[s],
                    (k_first + k) * 64, tb * nt, keep_x);
      };
      const int ahead = steps < stages ? steps : stages;
      for (int k = 0; k < ahead; ++k) weights(k, k);
      pdl_wait();
      for (int k = 0; k < ahead; ++k) tokens(k, k);
      int s = 0, last = ahead;
      uint32_t phase = 0;
      for (int k = ahead; k < steps; ++k) {
        if (!mbar_wait(&empty[s], phase, tmo, &abort_flag)) {
          record_status(P.status, kStatusTimeout);
          abort_flag = 1;
          break;
        }
        weights(k, s);
        tokens(k, s);
        last = k + 1;
        if (++s == stages) {
          s = 0;
          phase ^= 1u;
        }
      }
      // every copy lands before the CTA winds down, whatever else happened
      for (int k = last > stages ? last - stages : 0; k < last; ++k)
        mbar_wait(&full[k % stages], static_cast<uint32_t>(k / stages) & 1u, tmo, nullptr);
    }
  } else if (warp == 1) {
    // ================= MMA issuer =================
    if (elect_one()) {
      const bool w_mn = pr.b_mn;
      const uint32_t idesc = (P.f16 ? idesc_f16_f32(128, nt) : idesc_bf16_f32(128, nt)) |
                             (w_mn ? 1u << 15 : 0u);
      const uint64_t wstep = w_mn ? 2048 >> 4 : 32 >> 4;
      int s = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int k = 0; k < steps; ++k) {
        if (!mbar_wait(&full[s], phase, tmo, &abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sw = smem_u32(smem + s * stage_bytes);
        uint64_t wd = w_mn ? sdesc_mn_sw128(sw) : sdesc_k_sw128(sw);
        uint64_t xd = sdesc_k_sw128(sw + kTsWeightBytes);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          umma_bf16(tmem_base, wd, xd, idesc, k > 0 || kk > 0 ? 1u : 0u);
          wd += wstep;
          xd += 32 >> 4;
        }
        umma_commit(&empty[s]);
        if (++s == stages) {
          s = 0;
          phase ^= 1u;
        }
      }
      if (!ok) {
        record_status(P.status, kStatusTimeout);
        abort_flag = 1;
      }
      umma_commit(done);  // also after a timeout: what was issued ends before TMEM is released
    }
  } else {
    // ================= sums to shared memory =================
    pdl_wait();  // the epilogue below reads and overwrites what the kernel before uses
    int good = 1;
    if (lane == 0) good = mbar_wait(done, 0, tmo, nullptr) ? 1 : 0;
    good = __shfl_sync(0xffffffffu, good, 0);
    if (!good) {
      if (lane == 0) {
        record_status(P.status, kStatusTimeout);
        abort_flag = 1;
      }
    } else {
      // every copy has landed and every MMA has read it: the ring is free
      tc_fence_after();
      const int q = warp & 3;
      float* part = reinterpret_cast<float*>(smem) + q * 32 + lane;
      for (int c = (warp - 2) >> 2; 16 * c < nt; c += 2) {
        float v[16];
        tmem_ld16(tmem_base + (static_cast<uint32_t>(q * 32) << 16) + 16 * c, v);
#pragma unroll
        for (int j = 0; j < 16; ++j) part[(16 * c + j) * 128] = v[j];
      }
      tc_fence_before();
    }
  }
  __syncwarp();
  cluster_sync();  // all CTAs' sums are in place, and tensor memory is read
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, cols);
  }

  bool arrived = false;
  if (warp >= 2 && !abort_flag) {
    const int f0 = KIND == kTgGluFwd ? fb * 64 + 4 * (lane & 15) : fb * 128 + 4 * lane;
    const int tokens = min(nt, pr.m - tb * nt);
    const bool live = f0 < pr.n;  // n is a multiple of 8
    constexpr int step = 8 * SPLITS;
    for (int t0 = static_cast<int>(rank) + SPLITS * (warp - 2); t0 < tokens;
         t0 += kBatch * step) {
      const int64_t row0 = static_cast<int64_t>(tb) * nt + t0;
      const int count = min(kBatch, (tokens - t0 + step - 1) / step);
      float v[kBatch][4];
      float g[KIND == kTgGluBwd ? kBatch : 1][4], u[KIND == kTgGluBwd ? kBatch : 1][4];
      if constexpr (KIND == kTgGluBwd) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (i < count && live) {
            kept4(P, g[i], row0 + i * step, 0, f0, pr.n);
            kept4(P, u[i], row0 + i * step, 1, f0, pr.n);
          }
      }
      cluster_sums<SPLITS>(v, reinterpret_cast<const float*>(smem) + t0 * 128 + 4 * lane,
                           step * 128, count, rank);
      if (t0 + kBatch * step >= tokens) {  // the last reads of the peers' sums
        cluster_arrive();  // before the stores, which a release after them would wait for
        arrived = true;
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (i >= count) break;
        const int64_t row = row0 + i * step;
        if constexpr (KIND == kTgGluFwd) {  // lanes 0-15 hold gate, 16-31 up
          const int half = lane >> 4;
          if (P.gu != nullptr) {
            if (P.gu_fmt == kFmtInt8)
              keep4<true>(P, v[i], row, half, f0, pr.n, live);
            else if (P.gu_fmt == kFmtE4m3)
              keep4<false>(P, v[i], row, half, f0, pr.n, live);
            else if (live)
              put4(P.gu, row * P.ld_gu + static_cast<int64_t>(half) * pr.n + f0, v[i], P.f16);
          }
          float up[4], h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) up[e] = __shfl_xor_sync(0xffffffffu, v[i][e], 16);
#pragma unroll
          for (int e = 0; e < 4; e += 2)
            of_pair(mul2(gate_act(pair_of(v[i][e], v[i][e + 1]), P.silu),
                         pair_of(up[e], up[e + 1])),
                    h[e], h[e + 1]);
          if (live && half == 0) put4(pr.out, row * pr.ld_out + f0, h, P.f16);
        } else if (live) {
          if constexpr (KIND == kTgGluBwd) {
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const uint64_t gg = pair_of(g[i][e], g[i][e + 1]);
              const Gate2 ga = P.silu ? gate_of<true, true>(gg) : gate_of<true, false>(gg);
              const uint64_t d = pair_of(v[i][e], v[i][e + 1]), uu = pair_of(u[i][e], u[i][e + 1]);
              of_pair(mul2(mul2(d, uu), ga.da), g[i][e], g[i][e + 1]);
              of_pair(mul2(d, ga.a), u[i][e], u[i][e + 1]);
              of_pair(mul2(ga.a, uu), v[i][e], v[i][e + 1]);
            }
            const int64_t at = row * P.ld_dgu + f0;
            put4(P.dgu, at, g[i], P.f16);
            put4(P.dgu, at + pr.n, u[i], P.f16);
            if (pr.out != nullptr) put4(pr.out, row * pr.ld_out + f0, v[i], P.f16);
          } else {
            put4(pr.out, row * pr.ld_out + f0, v[i], P.f16);
          }
        }
      }
    }
  }
  // ---- no CTA exits while its peers may still read its sums
  if (!arrived) cluster_arrive();
  cluster_wait();
}

template <int KIND, int SPLITS>
static cudaError_t launch_ts(const TgMaps& maps, const TgParams& p, int nt, cudaStream_t s,
                             bool pdl) {
  const int stage = kTsWeightBytes + nt * 128;
  const int fit = ts_ring(nt) / stage;
  const int stages = fit < kTsMaxStages ? fit : kTsMaxStages;
  const int smem = 1024 + ts_ring(nt);
  auto kernel = train_small_kernel<KIND, SPLITS>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 1024 + ts_ring(128));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.prob[0].m_tiles * p.prob[0].n_tiles * SPLITS));
  cfg.blockDim = dim3(kTsThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = SPLITS;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, maps, p, nt, stages);
}

template <int KIND>
static cudaError_t launch_kind(const TgMaps& maps, const TgParams& p, int nt, int splits,
                               cudaStream_t s, bool pdl) {
  switch (splits) {
    case 1: return launch_ts<KIND, 1>(maps, p, nt, s, pdl);
    case 2: return launch_ts<KIND, 2>(maps, p, nt, s, pdl);
    case 4: return launch_ts<KIND, 4>(maps, p, nt, s, pdl);
    default: return launch_ts<KIND, 8>(maps, p, nt, s, pdl);
  }
}

cudaError_t launch_train_small(const TgMaps& maps, const TgParams& p, int nt, int splits,
                               cudaStream_t s, bool pdl) {
  switch (p.kind) {
    case kTgStore: return launch_kind<kTgStore>(maps, p, nt, splits, s, pdl);
    case kTgGluFwd: return launch_kind<kTgGluFwd>(maps, p, nt, splits, s, pdl);
    case kTgGluBwd: return launch_kind<kTgGluBwd>(maps, p, nt, splits, s, pdl);
  }
  return cudaErrorInvalidValue;
}

}  // namespace moe
