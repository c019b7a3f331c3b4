// Backward of the linear layer's epilogue: the activation's derivative and
// the bias gradient.
//
//   dZ = dY act'(Z)   (bf16, rounded once)      dbias[n] = sum over m of dZ[m, n]
// (the sum is of the float32 products, before their rounding).
//
// Bound by HBM: dY and Z read, dZ written, 6 bytes per element.  A block owns
// a strip of 256 columns (32 lanes x 16 bytes) and a range of rows, its warps
// take the rows in turn, and every lane keeps the sums of its eight columns
// in registers.  The blocks' sums are joined in a fixed order by a second
// kernel, so the gradients do not depend on the schedule.
#include "act.cuh"
#include "elem.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace falqon {
namespace {

constexpr int kStripCols = 256;
constexpr int kStripWarps = 8;

template <int kAct>
__global__ void __launch_bounds__(32 * kStripWarps)
    epilogue_bwd_kernel(const void* __restrict__ dy, const void* __restrict__ z, int64_t M, int64_t N,
                        void* __restrict__ dz, float* __restrict__ part) {
  pdl_trigger();
  pdl_wait();
  __shared__ float sums[kStripWarps][kStripCols];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * kStripCols + lane * 8;
  const int64_t m0 = M * blockIdx.y / gridDim.y, m1 = M * (blockIdx.y + 1) / gridDim.y;
  float acc[8] = {};
  if (col < N) {  // N is a multiple of 16: eight columns in or out together
    for (int64_t m = m0 + warp; m < m1; m += kStripWarps) {
      const int64_t at = (m * N + col) / 8;
      float d[8];
      unpack16<true>(static_cast<const uint4*>(dy)[at], d);
      if constexpr (kAct != FALQON_ACT_NONE) {
        float v[8];
        unpack16<true>(static_cast<const uint4*>(z)[at], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] *= act_slope<kAct>(v[j]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += d[j];
      if (dz) static_cast<uint4*>(dz)[at] = pack16<true>(d);
    }
  }
  if (!part) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) sums[warp][lane * 8 + j] = acc[j];
  __syncthreads();
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kStripCols + threadIdx.x;
  if (c < N) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kStripWarps; ++w) s += sums[w][threadIdx.x];
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

// Row ranges: enough blocks for eight per SM of a B200 over all strips, each
// of at least one row per warp.
int epilogue_parts(int64_t M, int64_t N) {
  const int64_t strips = (N + kStripCols - 1) / kStripCols;
  int64_t p = (148 * 8 + strips - 1) / strips;
  const int64_t most = (M + kStripWarps - 1) / kStripWarps;
  if (p > most) p = most;
  return static_cast<int>(p);
}

template <int kAct>
cudaError_t epilogue_bwd_t(const void* dy, const void* z, int64_t M, int64_t N, void* dz, float* dbias, float* ws,
                           cudaStream_t stream) {
  const int parts = epilogue_parts(M, N);
  const unsigned strips = static_cast<unsigned>((N + kStripCols - 1) / kStripCols);
  cudaError_t e = launch_pdl(epilogue_bwd_kernel<kAct>, dim3(strips, static_cast<unsigned>(parts)),
                             dim3(32 * kStripWarps), 0, stream, 1u, dy, z, M, N, dz,
                             dbias ? (parts == 1 ? dbias : ws) : static_cast<float*>(nullptr));
  if (e != cudaSuccess || !dbias || parts == 1) return e;
  return launch_column_sums(ws, dbias, nullptr, nullptr, parts, N, stream);
}

}  // namespace

size_t epilogue_bwd_workspace_bytes(int64_t M, int64_t N) {
  return align_up(static_cast<size_t>(epilogue_parts(M, N)) * static_cast<size_t>(N) * sizeof(float), 256);
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
