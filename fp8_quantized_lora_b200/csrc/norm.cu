// Layer norm and RMS norm over the rows of a matrix, forward and backward.
//
//   layer  mu = mean(x), rstd = 1 / sqrt(mean((x - mu)^2) + eps), xh = (x - mu) rstd
//   rms    rstd = 1 / sqrt(mean(x^2) + eps),                      xh = x rstd
//   y  = xh gamma + beta
//   g  = dy gamma,  c1 = mean(g) (0 for rms),  c2 = mean(g xh)
//   dx = rstd (g - c1 - xh c2) + dres
//   dgamma = sum over rows of dy xh,  dbeta = sum over rows of dy
//
// Both directions are bound by HBM: 2 (forward) or 3 to 4 (backward) elements
// of the matrix per element.  The variance is taken about the mean, not as
// the difference of two moments, so a large common offset costs no digits.
// Statistics, sums and the parameter gradients are float32; one rounding per
// output element.
#include "elem.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace falqon {
namespace {

constexpr int kRowThreads = 256;

// One row per block iteration; three passes over the row (the second and
// third out of L1 / L2).
template <bool kBF16, bool kRms>
__global__ void __launch_bounds__(kRowThreads)
    norm_fwd_kernel(const void* __restrict__ x, const void* __restrict__ gamma, const void* __restrict__ beta,
                    bool param_bf16, int64_t rows, int64_t cols, float eps, void* __restrict__ y,
                    float* __restrict__ mean, float* __restrict__ rstd, int32_t* __restrict__ dev_status) {
  pdl_trigger();
  pdl_wait();
  __shared__ float red[32];
  const float inv = 1.0f / static_cast<float>(cols);
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int64_t base = row * cols;
    float mu = 0.0f;
    if constexpr (!kRms) {
      float s = 0.0f;
      for (int64_t c = threadIdx.x; c < cols; c += kRowThreads) s += load_elem<kBF16>(x, base + c);
      mu = block_sum(s, red) * inv;
    }
    float s2 = 0.0f;
    for (int64_t c = threadIdx.x; c < cols; c += kRowThreads) {
      const float d = load_elem<kBF16>(x, base + c) - mu;
      s2 = fmaf(d, d, s2);
    }
    const float rs = 1.0f / sqrtf(block_sum(s2, red) * inv + eps);
    if (threadIdx.x == 0) {
      if (mean && !kRms) mean[row] = mu;
      if (rstd) rstd[row] = rs;
      // a NaN or infinity in the row, or sums past float32: rs is then 0 or NaN (infinite: eps = 0, constant row)
      if (dev_status && !(rs > 0.0f && isfinite(rs) && isfinite(mu))) atomicOr(dev_status, kDevNonfinite);
    }
    for (int64_t c = threadIdx.x; c < cols; c += kRowThreads) {
      const float xh = (load_elem<kBF16>(x, base + c) - mu) * rs;
      store_elem<kBF16>(y, base + c,
                        fmaf(xh, load_param(gamma, param_bf16, c, 1.0f), load_param(beta, param_bf16, c, 0.0f)));
    }
  }
}

// Block b owns the rows [b rows / grid, (b + 1) rows / grid) and one row of
// each partial sum; a thread owns its columns of them.
template <bool kBF16, bool kRms>
__global__ void __launch_bounds__(kRowThreads)
    norm_bwd_kernel(const void* __restrict__ dy, const void* __restrict__ x, const void* __restrict__ gamma,
                    bool param_bf16, const float* __restrict__ mean, const float* __restrict__ rstd,
                    const void* __restrict__ dres, int64_t rows, int64_t cols, void* __restrict__ dx,
                    float* __restrict__ part_g, float* __restrict__ part_b) {
  pdl_trigger();
  pdl_wait();
  __shared__ float red[32];
  const float inv = 1.0f / static_cast<float>(cols);
  const int64_t r0 = rows * blockIdx.x / gridDim.x, r1 = rows * (blockIdx.x + 1) / gridDim.x;
  const int64_t pbase = static_cast<int64_t>(blockIdx.x) * cols;
  for (int64_t row = r0; row < r1; ++row) {
    const int64_t base = row * cols;
    const float mu = kRms ? 0.0f : mean[row];
    const float rs = rstd[row];
    float c1 = 0.0f, c2 = 0.0f;
    for (int64_t c = threadIdx.x; c < cols; c += kRowThreads) {
      const float d = load_elem<kBF16>(dy, base + c);
      const float xh = (load_elem<kBF16>(x, base + c) - mu) * rs;
      const float gv = d * load_param(gamma, param_bf16, c, 1.0f);
      c1 += gv;
      c2 = fmaf(gv, xh, c2);
      if (part_g) part_g[pbase + c] = row == r0 ? d * xh : fmaf(d, xh, part_g[pbase + c]);
      if (part_b) part_b[pbase + c] = row == r0 ? d : part_b[pbase + c] + d;
    }
    if (!dx) continue;
    c1 = kRms ? 0.0f : block_sum(c1, red) * inv;
    c2 = block_sum(c2, red) * inv;
    for (int64_t c = threadIdx.x; c < cols; c += kRowThreads) {
      const float xh = (load_elem<kBF16>(x, base + c) - mu) * rs;
      const float gv = load_elem<kBF16>(dy, base + c) * load_param(gamma, param_bf16, c, 1.0f);
      float v = (gv - c1 - xh * c2) * rs;
      if (dres) v += load_elem<kBF16>(dres, base + c);
      store_elem<kBF16>(dx, base + c, v);
    }
  }
}

// Blocks of the backward, each with one partial row of dgamma and dbeta:
// two per SM of a B200, never more than rows.
constexpr int64_t kNormParts = 296;

int norm_parts(int64_t rows) { return static_cast<int>(rows < kNormParts ? rows : kNormParts); }

template <bool kBF16, bool kRms>
cudaError_t norm_fwd_t(const void* x, const void* gamma, const void* beta, bool pbf, int64_t rows, int64_t cols,
                       float eps, void* y, float* mean, float* rstd, int32_t* dev_status, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(rows < (1 << 20) ? rows : (1 << 20));
  return launch_pdl(norm_fwd_kernel<kBF16, kRms>, dim3(grid), dim3(kRowThreads), 0, stream, 1u, x, gamma, beta, pbf,
                    rows, cols, eps, y, mean, rstd, dev_status);
}

template <bool kBF16, bool kRms>
cudaError_t norm_bwd_t(const void* dy, const void* x, const void* gamma, bool pbf, const float* mean,
                       const float* rstd, const void* dres, int64_t rows, int64_t cols, void* dx, float* part_g,
                       float* part_b, cudaStream_t stream) {
  return launch_pdl(norm_bwd_kernel<kBF16, kRms>, dim3(norm_parts(rows)), dim3(kRowThreads), 0, stream, 1u, dy, x,
                    gamma, pbf, mean, rstd, dres, rows, cols, dx, part_g, part_b);
}

}  // namespace

size_t norm_bwd_workspace_bytes(int64_t rows, int64_t cols) {
  return 2 * align_up(static_cast<size_t>(norm_parts(rows)) * static_cast<size_t>(cols) * sizeof(float), 256);
}

cudaError_t launch_norm_fwd(const void* x, bool bf16, const void* gamma, const void* beta, bool param_bf16, bool rms,
                            int64_t rows, int64_t cols, float eps, void* y, float* mean, float* rstd,
                            int32_t* dev_status, cudaStream_t stream) {
  auto fn = bf16 ? (rms ? norm_fwd_t<true, true> : norm_fwd_t<true, false>)
                 : (rms ? norm_fwd_t<false, true> : norm_fwd_t<false, false>);
  return fn(x, gamma, beta, param_bf16, rows, cols, eps, y, mean, rstd, dev_status, stream);
}

cudaError_t launch_norm_bwd(const void* dy, const void* x, bool bf16, const void* gamma, bool param_bf16, bool rms,
                            const float* mean, const float* rstd, const void* dres, int64_t rows, int64_t cols,
                            void* dx, float* dgamma, float* dbeta, void* workspace, cudaStream_t stream) {
  float* pg = static_cast<float*>(workspace);
  float* pb = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + norm_bwd_workspace_bytes(rows, cols) / 2);
  auto fn = bf16 ? (rms ? norm_bwd_t<true, true> : norm_bwd_t<true, false>)
                 : (rms ? norm_bwd_t<false, true> : norm_bwd_t<false, false>);
  cudaError_t e = fn(dy, x, gamma, param_bf16, mean, rstd, dres, rows, cols, dx, dgamma ? pg : nullptr,
                     dbeta ? pb : nullptr, stream);
  if (e != cudaSuccess || (!dgamma && !dbeta)) return e;
  return launch_column_sums(dgamma ? pg : nullptr, dgamma, dbeta ? pb : nullptr, dbeta, norm_parts(rows), cols,
                            stream);
}

}  // namespace falqon
