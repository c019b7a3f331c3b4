// The FP8 forward with an epilogue (falqon_linear_fwd_epilogue) for few rows
// of X, where 256 x 256 tiles would leave most SMs without work: one token of
// a model that is sampled from, a short batch, a narrow layer.
//
//   Z = Xq . Wq^T / (s_X s_W) + bias,   Y = act(Z) + residual
//
// At M = 1 the weight is the work: N K bytes are read once and the tensor
// cores idle.  So the product runs transposed, Wq's rows as the M = 128 side
// of the UMMA and kT rows of X (16 to 128) as its N
// side, which costs nothing for the rows that X does not have, and K is split
// over a cluster of up to eight CTAs so that every SM streams its share.  The
// CTAs of a cluster leave their float32 tiles in shared memory and each sums
// and finishes a slice of the outputs out of the others' (in rank order: the
// result does not depend on the schedule).
//
// Measured on a B200 (us; in brackets the floor at 6.55 TB/s): one token, N x K
// 4096 x 4096: 8.2 with the weight from memory (2.6), 6.4 from the L2, where
// pairs of SMs took 18.4; 11008 x 4096: 12.1 (6.9).  What is left is the launch,
// the cluster's start and its two barriers.  Asking for the weight into the L2
// before the previous kernel has ended took 7.8, but 9.8 against 9.3 at 64
// tokens.
//
// Roles: warp 0 TMA producer, warp 1 UMMA issuer (one lane each), warp 2 MMA
// waiter; all eight warps drain the accumulator, [token][feature] in shared
// memory, and write the outputs, a token a warp.  Every wait is bounded
// (FALQON_DEV_TIMEOUT).
#include "act.cuh"
#include "elem.cuh"
#include "internal.h"
#include "tc_common.cuh"

namespace falqon {
namespace {

constexpr int kFewMmaBar = 1;  // named barrier between the issuer and its waiter

struct FewArgs {
  int32_t n_tiles, kb_total, kb_per_split, splits;
  int64_t M, N;
  __nv_bfloat16* y;
  const float* s_x;
  const float* s_w;
  LinearEpilogue epi;
  int32_t* dev_status;
};

template <int kT, int kStages, int kMinBlocks>
struct FewCfg {
  static constexpr int T = kT;  // rows of X in a tile
  static constexpr int Stages = kStages;
  static constexpr int MinBlocks = kMinBlocks;
  static constexpr int BK = kRowBytes;
  static constexpr int ABytes = kBM * kRowBytes;
  static constexpr int BBytes = kT * kRowBytes;
  static constexpr int StageBytes = ABytes + BBytes;
  static constexpr int Threads = 256;
  static constexpr uint32_t TmemCols = kT < 32 ? 32 : kT;
  static constexpr int RedStride = kBM + 4;  // float32 words of one token's row of the reduction tile
  static constexpr int SmemBytes = kStages * StageBytes + 8 * (2 * kStages + 2) + 16 + 1024;
  static constexpr uint32_t IDesc = idesc_f32acc(0u, 0u, 0u, 0u, kBM, kT);
  static_assert(kT * RedStride * 4 <= kStages * StageBytes, "reduction tile");
  static_assert(kMinBlocks * (SmemBytes + 1024) <= 233472, "shared memory per SM");
  static_assert(kMinBlocks * TmemCols <= 512, "tensor memory per SM");
};

template <int kAct>
__device__ __forceinline__ void act4(float2 (&v)[2]) {
  v[0] = act_value2<kAct>(v[0]);
  v[1] = act_value2<kAct>(v[1]);
}

__device__ __forceinline__ void act4(falqon_act act, float2 (&v)[2]) {
  switch (act) {
    case FALQON_ACT_NONE: break;
    case FALQON_ACT_RELU: act4<FALQON_ACT_RELU>(v); break;
    case FALQON_ACT_GELU_ERF: act4<FALQON_ACT_GELU_ERF>(v); break;
    case FALQON_ACT_GELU_TANH: act4<FALQON_ACT_GELU_TANH>(v); break;
    case FALQON_ACT_SILU: act4<FALQON_ACT_SILU>(v); break;
  }
}

template <class C>
__global__ void __launch_bounds__(C::Threads, C::MinBlocks)
    tc_gemm_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                       const FewArgs g) {
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::Stages * C::StageBytes);  // [Stages] landed
  uint64_t* empty = full + C::Stages;                                              // [Stages] MMAs done
  uint64_t* acc_full = empty + C::Stages;
  uint64_t* drain = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the CTAs of a cluster are the K splits of one tile
  const int split = static_cast<int>(blockIdx.x) % g.splits;
  const int tile = static_cast<int>(blockIdx.x) / g.splits;
  const int n0 = tile % g.n_tiles * kBM, m0 = tile / g.n_tiles * C::T;
  const int kb0 = split * g.kb_per_split;
  const int nkb = min(g.kb_total, kb0 + g.kb_per_split) - kb0;  // no split is empty (few_split)

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::Stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::TmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_trigger();  // the next kernel may start launching; it waits for this one
  pdl_wait();     // the previous kernel's results are complete and visible

  auto fail = [&]() {
    *abort_flag = 1;
    raise_status(g.dev_status, kDevTimeout);
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      uint32_t issued = 0, issued_parity = 0;
      for (int i = 0; i < nkb; ++i) {
        const int s = i % C::Stages;
        const uint32_t phase = static_cast<uint32_t>(i / C::Stages) & 1u;
        if (!mbar_wait(&empty[s], phase ^ 1, abort_flag)) { fail(); break; }
        uint8_t* sA = smem + s * C::StageBytes;
        mbar_arrive_expect_tx(&full[s], C::StageBytes);
        issued |= 1u << s;
        issued_parity = (issued_parity & ~(1u << s)) | (phase << s);
        tma_load_2d(sA, &tmW, &full[s], (kb0 + i) * C::BK, n0);
        tma_load_2d(sA + C::ABytes, &tmX, &full[s], (kb0 + i) * C::BK, m0);
      }
      // every load issued must land before shared memory is reused or released
      for (int s = 0; s < C::Stages; ++s)
        if (issued & (1u << s)) mbar_wait_budget(&full[s], (issued_parity >> s) & 1u);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ UMMA issuer
    // Released once per K block by the waiter (an mbarrier wait in the issuing
    // thread would hold back its MMA stream).
    bool ok = true;
    for (int i = 0; i < nkb; ++i) {
      if (bar_red_or(kFewMmaBar, 64, false)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (lane == 0) {
        const int s = i % C::Stages;
        const uint32_t a_base = smem_u32(smem + s * C::StageBytes);
        const uint32_t b_base = a_base + C::ABytes;
#pragma unroll
        for (int ks = 0; ks < kRowBytes / 32; ++ks)
          umma_f8(tmem_base, operand_desc<false, 1, C::BK>(a_base, ks), operand_desc<false, 1, C::BK>(b_base, ks),
                  C::IDesc, (i > 0 || ks > 0) ? 1u : 0u);
        umma_commit(&empty[s]);
      }
      __syncwarp();
    }
    if (lane == 0) {
      if (ok) umma_commit(acc_full);
      umma_commit(drain);
      mbar_wait_budget(drain, 0);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------ MMA waiter
    for (int i = 0; i < nkb; ++i) {
      const bool ok = warp_wait(&full[i % C::Stages], static_cast<uint32_t>(i / C::Stages) & 1u, abort_flag);
      if (!ok && lane == 0) fail();
      __syncwarp();
      if (bar_red_or(kFewMmaBar, 64, !ok)) break;
    }
  }
  __syncwarp();

  // ---------------------------------------------------------------- accumulator -> shared memory
  // The ring is idle once every MMA has completed.  Warp w reads TMEM lane
  // quarter w % 4 (features), the two warps of a quarter every other 16 tokens.
  float* red = reinterpret_cast<float*>(smem);
  {
    const int q = warp & 3;
    if (warp_wait(acc_full, 0, abort_flag)) {
      tc_fence_after();
#pragma unroll 1
      for (int c = warp >> 2; c < C::T / 16; c += 2) {
        uint32_t r[16];
        tmem_ld_16cols(tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(c * 16), r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j)
          red[(c * 16 + j) * C::RedStride + q * 32 + lane] = __uint_as_float(r[j]);
      }
    } else if (lane == 0) {
      fail();
    }
    tc_fence_before();
  }
  __syncthreads();
  if (g.splits > 1) cluster_sync_all();

  // ---------------------------------------------------------------- sums over the cluster, epilogue
  {
    float alpha = 1.0f;
    {
      double den = static_cast<double>(*g.s_x) * static_cast<double>(*g.s_w);
      alpha = static_cast<float>(1.0 / den);
    }
    // this CTA's tokens, one a warp in turn; four features a lane (N is a multiple of 16)
    const int tokens = static_cast<int>(g.M - m0 < C::T ? g.M - m0 : C::T);
    const int t_end = tokens * (split + 1) / g.splits;
    const int f = lane * 4;
    if (n0 + f < g.N) {
      float2 bias[2] = {both(0.0f), both(0.0f)};
      if (g.epi.bias) {
        bias[0] = make_float2(load_param(g.epi.bias, g.epi.bias_bf16, n0 + f, 0.0f),
                              load_param(g.epi.bias, g.epi.bias_bf16, n0 + f + 1, 0.0f));
        bias[1] = make_float2(load_param(g.epi.bias, g.epi.bias_bf16, n0 + f + 2, 0.0f),
                              load_param(g.epi.bias, g.epi.bias_bf16, n0 + f + 3, 0.0f));
      }
      const __nv_bfloat16* residual = static_cast<const __nv_bfloat16*>(g.epi.residual);
      __nv_bfloat16* z = static_cast<__nv_bfloat16*>(g.epi.z);
      constexpr int kStep = C::Threads / 32, kBatch = 4;
      for (int t0 = tokens * split / g.splits + warp; t0 < t_end; t0 += kBatch * kStep) {
        // the residuals of four tokens on their way together: a load in turn
        // with the stores would wait for memory once a token
        uint2 res[kBatch];
        if (residual) {
#pragma unroll
          for (int k = 0; k < kBatch; ++k)
            if (t0 + k * kStep < t_end)
              res[k] = *reinterpret_cast<const uint2*>(residual + (m0 + t0 + k * kStep) * g.N + n0 + f);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int t = t0 + k * kStep;
          if (t >= t_end) break;
          const int64_t at = (m0 + t) * g.N + n0 + f;
          const float* own = red + t * C::RedStride + f;
          float2 v[2] = {both(0.0f), both(0.0f)};
          if (g.splits == 1) {
            const float4 a = *reinterpret_cast<const float4*>(own);
            v[0] = make_float2(a.x, a.y);
            v[1] = make_float2(a.z, a.w);
          } else {
            float4 a[kMaxSplits];
#pragma unroll
            for (int s = 0; s < kMaxSplits; ++s)
              if (s < g.splits) a[s] = dsmem_load_f32x4(dsmem_addr(own, s));
#pragma unroll
            for (int s = 0; s < kMaxSplits; ++s) {
              if (s < g.splits) {
                v[0] = add2(v[0], make_float2(a[s].x, a[s].y));
                v[1] = add2(v[1], make_float2(a[s].z, a[s].w));
              }
            }
          }
          v[0] = fma2(v[0], both(alpha), bias[0]);
          v[1] = fma2(v[1], both(alpha), bias[1]);
          if (z) *reinterpret_cast<uint2*>(z + at) = make_uint2(pack2(v[0].x, v[0].y), pack2(v[1].x, v[1].y));
          act4(g.epi.act, v);
          if (residual) {
            v[0] = add2(v[0], make_float2(__uint_as_float(res[k].x << 16), __uint_as_float(res[k].x & 0xFFFF0000u)));
            v[1] = add2(v[1], make_float2(__uint_as_float(res[k].y << 16), __uint_as_float(res[k].y & 0xFFFF0000u)));
          }
          *reinterpret_cast<uint2*>(g.y + at) = make_uint2(pack2(v[0].x, v[0].y), pack2(v[1].x, v[1].y));
        }
      }
    }
  }

  if (g.splits > 1) cluster_sync_all();  // the others are done with this CTA's tile
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TmemCols);
  }
}

// ---------------------------------------------------------------- host side
// Up to 64 rows two CTAs share an SM; above, a tile takes the whole of it.
using Few16 = FewCfg<16, 6, 2>;
using Few32 = FewCfg<32, 5, 2>;
using Few64 = FewCfg<64, 4, 2>;
using Few128 = FewCfg<128, 6, 1>;

// Clusters of `splits` CTAs that the device keeps resident at once (cached per
// device, with the kernel's attributes set).  A GPC holds whole clusters only:
// 48 clusters of six CTAs take two waves on 148 SMs although 288 CTAs fit.
// The occupancy query counts one CTA of a cluster per SM; where two fit, a
// cluster of 2 s takes the SMs of one of s.
template <class C>
cudaError_t few_resident(const DeviceInfo* di, int splits, int* clusters) {
  static int cached[32][kMaxSplits + 1] = {};
  const int dev = di->device;
  if (dev < 32) {
    *clusters = __atomic_load_n(&cached[dev][splits], __ATOMIC_ACQUIRE);
    if (*clusters > 0) return cudaSuccess;
  }
  cudaError_t e = cudaFuncSetAttribute(tc_gemm_few_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SmemBytes);
  if (e != cudaSuccess) return e;
  const bool halve = C::MinBlocks == 2 && splits % 2 == 0;
  const int size = halve ? splits / 2 : splits;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(size);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(di->sm_count / size * size));
  cfg.blockDim = dim3(C::Threads);
  cfg.dynamicSmemBytes = C::SmemBytes;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, tc_gemm_few_kernel<C>, &cfg) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    n = di->sm_count / size;
  }
  if (n > di->sm_count / size) n = di->sm_count / size;
  if (n < 1) n = 1;
  if (C::MinBlocks == 2 && !halve) n *= 2;
  if (dev < 32) __atomic_store_n(&cached[dev][splits], n, __ATOMIC_RELEASE);
  *clusters = n;
  return cudaSuccess;
}

// How a product is split: the tile's rows of X, the K splits, and the waves of
// clusters that this takes.
struct FewPlan {
  int rows, tiles, splits, per_split, waves;
};

// The most splits (up to kMaxSplits, none empty) that leave all tiles in one wave.
template <class C>
cudaError_t few_split(const DeviceInfo* di, int64_t M, int64_t N, int64_t K, FewPlan* p) {
  const int kb = ceil_div(K, C::BK);
  p->rows = C::T;
  p->tiles = ceil_div(N, kBM) * ceil_div(M, C::T);
  int resident = 1;
  for (int s = kb < kMaxSplits ? kb : kMaxSplits; s >= 1; --s) {
    p->per_split = ceil_div(kb, s);
    if (ceil_div(kb, p->per_split) != s) continue;  // a split would be empty
    p->splits = s;
    cudaError_t e = few_resident<C>(di, s, &resident);
    if (e != cudaSuccess) return e;
    if (p->tiles <= resident) break;
  }
  p->waves = ceil_div(p->tiles, resident);
  return cudaSuccess;
}

// The tile's rows of X.  A wider tile re-reads Wq less often, a narrower one
// finishes sooner and leaves more CTAs to split K over.  Measured in us for
// 16 / 32 / 64 / 128 rows: M = 64, N x K = 4096 x 256: 5.0 / 5.5 / 6.5 / 6.5
// (K short: what counts is the end); 64, 4096 x 4096: - / 8.1 / 8.7 / 8.4;
// 128, 4096 x 4096: - / 10.5 / 9.4 / 9.6; 64, 11008 x 4096: - / 17.0 / 14.6 / 18.9.
cudaError_t few_plan(const DeviceInfo* di, int64_t M, int64_t N, int64_t K, FewPlan* p) {
  const int sms = di->sm_count;
  const int64_t n_tiles = (N + kBM - 1) / kBM;
  auto tiles = [&](int64_t rows) { return n_tiles * ((M + rows - 1) / rows); };
  if (M <= 16 || (K <= 512 && tiles(16) <= 2 * sms)) return few_split<Few16>(di, M, N, K, p);
  if (M <= 32 || tiles(32) <= sms / 2) return few_split<Few32>(di, M, N, K, p);
  if (tiles(64) <= 2 * sms) return few_split<Few64>(di, M, N, K, p);
  return few_split<Few128>(di, M, N, K, p);
}

template <class C>
cudaError_t few_gemm(const FewPlan& p, const uint8_t* xq, const float* s_x, const uint8_t* wq, const float* s_w,
                     int64_t M, int64_t N, int64_t K, const LinearEpilogue& epi, void* y, int32_t* dev_status,
                     cudaStream_t stream) {
  CUtensorMap tW, tX;
  const auto U8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  if (!make_tmap_2d(&tW, U8, 1, wq, K, N, C::BK, kBM, true)) return cudaErrorInvalidValue;
  if (!make_tmap_2d(&tX, U8, 1, xq, K, M, C::BK, C::T, true)) return cudaErrorInvalidValue;
  FewArgs g{};
  g.n_tiles = ceil_div(N, kBM);
  g.kb_total = ceil_div(K, C::BK);
  g.kb_per_split = p.per_split;
  g.splits = p.splits;
  g.M = M;
  g.N = N;
  g.y = static_cast<__nv_bfloat16*>(y);
  g.s_x = s_x;
  g.s_w = s_w;
  g.epi = epi;
  g.dev_status = dev_status;
  return launch_pdl(tc_gemm_few_kernel<C>, dim3(static_cast<unsigned>(p.tiles * p.splits)), dim3(C::Threads),
                    C::SmemBytes, stream, static_cast<unsigned>(p.splits), tW, tX, g);
}

}  // namespace

cudaError_t launch_fp8_gemm_fwd_few(const uint8_t* xq, const float* s_x, const uint8_t* wq, const float* s_w,
                                    int64_t M, int64_t N, int64_t K, const LinearEpilogue& epi, void* y,
                                    int32_t* dev_status, cudaStream_t stream, bool* taken) {
  *taken = false;
  const DeviceInfo* di = current_device_info();
  if (!di) return cudaErrorInvalidDevice;
  // more than twice as many of the widest tiles as SMs are the other kernel's anyway
  if ((N + kBM - 1) / kBM * ((M + 127) / 128) > 2 * int64_t(di->sm_count)) return cudaSuccess;
  FewPlan p{};
  cudaError_t e = few_plan(di, M, N, K, &p);
  if (e != cudaSuccess) return e;
  // Both kernels' times in ns, fitted to 200 measured sizes (M from 1 to 8192,
  // N and K from 16 to 11008), where the one expected to be faster was within
  // 3 % of the faster one in the mean.
  // Few rows: 3.2 us for the launch and the ends, and per wave of CTAs 30 ns a
  // row of the tile and 0.5 us (0.6 where a tile has 128 rows) a K block.
  const int64_t few = 3200 + static_cast<int64_t>(p.waves) * (30 * p.rows + (p.rows <= 64 ? 500 : 600) * p.per_split);
  // 256 x 256 tiles on pairs of SMs: 10 us for the launch and the ends, 0.37
  // us a K block, and every further wave at least the 6 us of its epilogue.
  const int64_t kb = (K + kRowBytes - 1) / kRowBytes;
  const int64_t pair_tiles = (M + 255) / 256 * ((N + 255) / 256);
  const int64_t pair_waves = (pair_tiles + di->sm_count / 2 - 1) / (di->sm_count / 2);
  const int64_t pair = 10000 + 370 * kb + (pair_waves - 1) * (370 * kb > 6000 ? 370 * kb : 6000);
  if (few >= pair) return cudaSuccess;
  *taken = true;
  auto fn = p.rows == 16   ? few_gemm<Few16>
            : p.rows == 32 ? few_gemm<Few32>
            : p.rows == 64 ? few_gemm<Few64>
                           : few_gemm<Few128>;
  return fn(p, xq, s_x, wq, s_w, M, N, K, epi, y, dev_status, stream);
}

}  // namespace falqon
