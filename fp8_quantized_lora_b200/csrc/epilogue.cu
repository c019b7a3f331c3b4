// Backward of the linear layer's epilogue: the activation's derivative and
// the bias gradient.
//
//   dZ = dY act'(Z)   (bf16, rounded once)      dbias[n] = sum over m of dZ[m, n]
// (the sum is of the float32 products, before their rounding).
//
// Bound by HBM: dY and Z read, dZ written, 6 bytes per element (and, with a
// sigmoid, close to the special function unit: two results an element).  A
// block owns a strip of up to 256 columns and a range of rows, its warps take
// the rows in turn, two at a time so that four loads are on their way, and
// every lane keeps the sums of its eight columns in registers.  A narrow
// matrix gives a warp several rows at once.  The blocks' sums are joined in a
// fixed order by a second kernel, so the gradients do not depend on the
// schedule.
//
// Measured on a B200 (us; in brackets the floor at 6.55 TB/s), GELU: 8192 x
// 11008 86.7 (82.6), 4096 x 4096 19.8 (tanh), 20.4 (erf) (15.4); SiLU, 200 x 272: 3.2 (0.05;
// two launches).
#include "act.cuh"
#include "elem.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace falqon {
namespace {

constexpr int kStripWarps = 8;
constexpr int kStripBlocks = 4;  // per SM

// dz (or dy itself) of one vector; adds it to the sums.
template <int kAct>
__device__ __forceinline__ uint4 epilogue_vec(const uint4& dq, const uint4& zq, float2 (&acc)[4]) {
  float d[8];
  unpack16<true>(dq, d);
  float2 v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = make_float2(d[2 * j], d[2 * j + 1]);
  if constexpr (kAct != FALQON_ACT_NONE) {
    unpack16<true>(zq, d);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = mul2(v[j], act_slope2<kAct>(make_float2(d[2 * j], d[2 * j + 1])));
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = add2(acc[j], v[j]);
  return make_uint4(pack2(v[0].x, v[0].y), pack2(v[1].x, v[1].y), pack2(v[2].x, v[2].y), pack2(v[3].x, v[3].y));
}

// lanes: lanes that share a row of the strip (8 columns each); a warp holds 32 / lanes rows.
template <int kAct>
__global__ void __launch_bounds__(32 * kStripWarps, kStripBlocks)
    epilogue_bwd_kernel(const uint4* __restrict__ dy, const uint4* __restrict__ z, int64_t M, int64_t N, int lanes,
                        uint4* __restrict__ dz, float* __restrict__ part) {
  pdl_trigger();
  pdl_wait();
  __shared__ float sums[32 * kStripWarps * 8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows_warp = 32 / lanes, strip = lanes * 8;
  const int64_t vecs = N / 8;  // of a row
  const int64_t vec = static_cast<int64_t>(blockIdx.x) * lanes + lane % lanes;
  const int64_t m0 = M * blockIdx.y / gridDim.y, m1 = M * (blockIdx.y + 1) / gridDim.y;
  const int64_t step = kStripWarps * rows_warp;
  float2 acc[4] = {};
  if (vec < vecs) {
    int64_t m = m0 + warp * rows_warp + lane / lanes;
    for (; m + step < m1; m += 2 * step) {
      const int64_t a = m * vecs + vec, b = a + step * vecs;
      const uint4 da = dy[a], db = dy[b];
      uint4 za = {}, zb = {};
      if constexpr (kAct != FALQON_ACT_NONE) {
        za = z[a];
        zb = z[b];
      }
      const uint4 ra = epilogue_vec<kAct>(da, za, acc), rb = epilogue_vec<kAct>(db, zb, acc);
      if (dz) {
        dz[a] = ra;
        dz[b] = rb;
      }
    }
    if (m < m1) {
      const int64_t a = m * vecs + vec;
      uint4 za = {};
      if constexpr (kAct != FALQON_ACT_NONE) za = z[a];
      const uint4 ra = epilogue_vec<kAct>(dy[a], za, acc);
      if (dz) dz[a] = ra;
    }
  }
  if (!part) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) *reinterpret_cast<float2*>(&sums[(threadIdx.x * 4 + j) * 2]) = acc[j];
  __syncthreads();
  const int64_t c = static_cast<int64_t>(blockIdx.x) * strip + threadIdx.x;
  if (static_cast<int>(threadIdx.x) < strip && c < N) {
    float s = 0.0f;
    for (int r = 0; r < kStripWarps * rows_warp; ++r) s += sums[r * strip + threadIdx.x];
    part[static_cast<int64_t>(blockIdx.y) * N + c] = s;
  }
}

// out[c] = sum over p of part[p][c], for up to two sums (blockIdx.y).  A block
// takes 32 columns; its 16 warps each add every sixteenth partial row, and the
// first joins the sixteen.
constexpr int kSumWarps = 16;

__global__ void __launch_bounds__(32 * kSumWarps)
    column_sums_kernel(const float* __restrict__ p0, float* __restrict__ o0, const float* __restrict__ p1,
                       float* __restrict__ o1, int parts, int64_t cols) {
  pdl_trigger();
  pdl_wait();
  __shared__ float sums[kSumWarps][33];
  const float* p = blockIdx.y ? p1 : p0;
  float* o = blockIdx.y ? o1 : o0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int64_t c0 = static_cast<int64_t>(blockIdx.x) * 32; c0 < cols; c0 += static_cast<int64_t>(gridDim.x) * 32) {
    const int64_t c = c0 + lane;
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 8
      for (int i = warp; i < parts; i += kSumWarps) s += p[static_cast<int64_t>(i) * cols + c];
    }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < cols) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kSumWarps; ++w) v += sums[w][lane];
      o[c] = v;
    }
    __syncthreads();
  }
}

// Lanes of a row, strips, and row ranges: one wave of blocks on the 148 SMs of
// a B200 (1.6 waves cost a fifth at 8192 x 11008), each of at least two steps;
// up to 64 rows a single range, which needs no second kernel.
struct EpilogueShape {
  int lanes;
  int64_t strips, parts;
};

EpilogueShape epilogue_shape(int64_t M, int64_t N) {
  EpilogueShape s{32, 0, 1};
  while (s.lanes > 2 && s.lanes * 4 >= N) s.lanes /= 2;
  s.strips = (N + s.lanes * 8 - 1) / (s.lanes * 8);
  if (M > 64) {
    const int64_t most = (M + 2 * kStripWarps * (32 / s.lanes) - 1) / (2 * kStripWarps * (32 / s.lanes));
    s.parts = 148 * kStripBlocks / s.strips;
    if (s.parts > most) s.parts = most;
    if (s.parts < 1) s.parts = 1;
  }
  return s;
}

template <int kAct>
cudaError_t epilogue_bwd_t(const void* dy, const void* z, int64_t M, int64_t N, void* dz, float* dbias, float* ws,
                           cudaStream_t stream) {
  const EpilogueShape s = epilogue_shape(M, N);
  cudaError_t e = launch_pdl(epilogue_bwd_kernel<kAct>,
                             dim3(static_cast<unsigned>(s.strips), static_cast<unsigned>(s.parts)),
                             dim3(32 * kStripWarps), 0, stream, 1u, static_cast<const uint4*>(dy),
                             static_cast<const uint4*>(z), M, N, s.lanes, static_cast<uint4*>(dz),
                             dbias ? (s.parts == 1 ? dbias : ws) : static_cast<float*>(nullptr));
  if (e != cudaSuccess || !dbias || s.parts == 1) return e;
  return launch_column_sums(ws, dbias, nullptr, nullptr, static_cast<int>(s.parts), N, stream);
}

}  // namespace

size_t epilogue_bwd_workspace_bytes(int64_t M, int64_t N) {
  return align_up(static_cast<size_t>(epilogue_shape(M, N).parts) * static_cast<size_t>(N) * sizeof(float), 256);
}

cudaError_t launch_column_sums(const float* part0, float* out0, const float* part1, float* out1, int parts,
                               int64_t cols, cudaStream_t stream) {
  const int64_t blocks = (cols + 31) / 32;
  return launch_pdl(column_sums_kernel, dim3(static_cast<unsigned>(blocks < 65535 ? blocks : 65535), out1 ? 2u : 1u),
                    dim3(32 * kSumWarps), 0, stream, 1u, part0, out0, part1, out1, parts, cols);
}

cudaError_t launch_epilogue_bwd(const void* dy, const void* z, falqon_act act, int64_t M, int64_t N, void* dz,
                                float* dbias, void* workspace, cudaStream_t stream) {
  float* ws = static_cast<float*>(workspace);
  switch (act) {
    case FALQON_ACT_NONE: return epilogue_bwd_t<FALQON_ACT_NONE>(dy, z, M, N, dz, dbias, ws, stream);
    case FALQON_ACT_RELU: return epilogue_bwd_t<FALQON_ACT_RELU>(dy, z, M, N, dz, dbias, ws, stream);
    case FALQON_ACT_GELU_ERF: return epilogue_bwd_t<FALQON_ACT_GELU_ERF>(dy, z, M, N, dz, dbias, ws, stream);
    case FALQON_ACT_GELU_TANH: return epilogue_bwd_t<FALQON_ACT_GELU_TANH>(dy, z, M, N, dz, dbias, ws, stream);
    case FALQON_ACT_SILU: return epilogue_bwd_t<FALQON_ACT_SILU>(dy, z, M, N, dz, dbias, ws, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace falqon
