// Layer norm and RMS norm over the rows of a matrix, forward and backward.
//
//   layer  mu = mean(x), rstd = 1 / sqrt(mean((x - mu)^2) + eps), xh = (x - mu) rstd
//   rms    rstd = 1 / sqrt(mean(x^2) + eps),                      xh = x rstd
//   y  = xh gamma + beta
//   g  = dy gamma,  c1 = mean(g) (0 for rms),  c2 = mean(g xh)
//   dx = rstd (g - c1 - xh c2) + dres
//   dgamma = sum over rows of dy xh,  dbeta = sum over rows of dy
//
// The variance is taken about the mean, not as the difference of two moments,
// so a large common offset costs no digits.  Statistics, sums and the parameter
// gradients are float32; one rounding per output element.
//
// What cannot be done without is HBM traffic: 2 (forward) or 3 to 4 (backward)
// elements of the matrix per element.  A row stays in registers between its
// sums and its outputs, so it is read once; the threads that share it meet at
// one barrier for each sum that the next step waits for.  Measured on a B200
// (us, floor at 6.55 TB/s in brackets):
//   forward   4096 x 4096 bf16   RMS 12.8, layer 14.7 (10.2)
//             4096 x 4096 fp32   RMS 23.4, layer 24.4 (20.5)
//             8192 x 1537 bf16   RMS 12.1, layer 18.7 (7.7)
//   backward  8192 x 4096 bf16 + dres   RMS 44.9, layer 48.0 (41.0)
//             4096 x 4096 bf16   RMS 21.4, layer 25.4 (15.4)
//             4096 x 4096 fp32   RMS 34.4, layer 36.9 (30.7)
//             8192 x 1537 bf16   RMS 24.9, layer 33.6 (11.5)
//              300 x 4096 bf16   RMS 6.0, layer 7.3 (1.1)
// (the backward with its second kernel, which joins the blocks' sums over the
// rows: about 2.5 us).  float32 is near its bound; in bf16 the backward's
// instructions and their latency bound it: a bf16 value costs an instruction
// to widen, and 128 registers a thread leave 16 warps an SM.
#include <algorithm>

#include "elem.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace falqon {
namespace {

constexpr int kRowThreads = 256;

// Rows of more than 16384 columns: one row per block iteration, three passes
// over it (the second and third out of L1 / L2).
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

// Sum of a row of kWarps per-warp values, zeros past the last (a multiple of four are read).
template <int kWarps>
__device__ __forceinline__ float sum_warps(const float* r) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kWarps; i += 4) {
    const float4 v = *reinterpret_cast<const float4*>(r + i);
    s += (v.x + v.y) + (v.z + v.w);
  }
  return s;
}

// Asks for [p, p + bytes) of a matrix that ends at `end` to come into L2 (whole
// 16-byte units; one thread).
__device__ __forceinline__ void prefetch_l2(const uint8_t* p, int64_t bytes, const uint8_t* end) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p) & ~static_cast<uintptr_t>(15);
  uintptr_t b = (reinterpret_cast<uintptr_t>(p) + bytes + 15) & ~static_cast<uintptr_t>(15);
  const uintptr_t last = reinterpret_cast<uintptr_t>(end) & ~static_cast<uintptr_t>(15);
  if (b > last) b = last;
  if (b > a)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a), "r"(static_cast<uint32_t>(b - a)) : "memory");
}

// Sum over the threads that share a row (a warp, or the block), in every
// thread, in an order that depends on their number alone.  Calls of a block
// alternate between two buffers: a thread that writes one again has passed the
// barrier of the call between, which every thread reaches after its reads.
template <bool kWarp, int kWarps>
__device__ __forceinline__ float row_sum(float v, float (*red)[32], uint32_t& turn) {
  v = warp_sum(v);
  if constexpr (!kWarp) {
    const int lane = threadIdx.x & 31;
    float* r = red[turn & 1u];
    ++turn;
    if (lane == 0) r[threadIdx.x >> 5] = v;
    __syncthreads();
    v = sum_warps<kWarps>(r);
  }
  return v;
}

// A thread's columns lie in 16-byte units of memory, whatever the row length: a
// row whose first element is `shift` elements into a unit (kShift; shift is 0
// without it) has unit i hold the columns i V - shift .. + V, of which the
// first and last unit hold some.  Rows a multiple of V apart have the same
// shift, so a block that takes such rows keeps its columns, their parameters
// and their sums in registers all the same.
template <bool kBF16, bool kShift>
struct Unit {
  static constexpr int V = kVec<kBF16>;
  static constexpr int Pairs = V / 2;
  static constexpr int Elem = kBF16 ? 2 : 4;
  uint4 q;

  __device__ static __forceinline__ int column(int unit, int shift) { return unit * V - (kShift ? shift : 0); }
  // whether every column of the unit at c exists (some do where c < cols)
  __device__ static __forceinline__ bool whole(int c, int cols) { return !kShift || (c >= 0 && c + V <= cols); }
  __device__ static __forceinline__ bool has(int c, int j, int cols) { return !kShift || (c + j >= 0 && c + j < cols); }

  // row: the row's first element; end: the matrix's.  A unit that the row
  // shares with its neighbours is read whole where it lies in the matrix.
  __device__ __forceinline__ void load(const uint8_t* row, int c, const uint8_t* end) {
    const uint8_t* p = row + static_cast<int64_t>(c) * Elem;
    if (!kShift || p + 16 <= end) {
      q = *reinterpret_cast<const uint4*>(p);
    } else {  // the matrix's last unit, not a whole one
      float v[V];
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = p + (j + 1) * Elem <= end ? load_elem<kBF16>(p, j) : 0.0f;
      q = pack16<kBF16>(v);
    }
  }
  // a unit as loaded, with the columns that are not the row's set to 0 (at its
  // use: doing it at once would wait for the load)
  __device__ __forceinline__ Unit trimmed(int c, int cols) const {
    Unit r = *this;
    if (!whole(c, cols)) {
      const uint4 m = mask(c, cols);
      r.q = make_uint4(q.x & m.x, q.y & m.y, q.z & m.z, q.w & m.w);
    }
    return r;
  }
  // ones where the unit's columns exist
  __device__ static __forceinline__ uint4 mask(int c, int cols) {
    const int low = c < 0 ? -c * 8 * Elem : 0, high = c + V > cols ? (c + V - cols) * 8 * Elem : 0;  // bits
    uint64_t a = ~0ull, b = ~0ull;  // low, high half
    a = low >= 64 ? 0ull : a << low;
    b = low > 64 ? b << (low - 64) : b;
    b = high >= 64 ? 0ull : b & (~0ull >> high);
    a = high > 64 ? a & (~0ull >> (high - 64)) : a;
    return make_uint4(static_cast<uint32_t>(a), static_cast<uint32_t>(a >> 32), static_cast<uint32_t>(b),
                      static_cast<uint32_t>(b >> 32));
  }
  __device__ __forceinline__ void pairs(float2 (&out)[Pairs]) const {
    float v[V];
    unpack16<kBF16>(q, v);
#pragma unroll
    for (int j = 0; j < Pairs; ++j) out[j] = make_float2(v[2 * j], v[2 * j + 1]);
  }
  __device__ static __forceinline__ void store(uint8_t* row, int c, int cols, const float2 (&p)[Pairs]) {
    float v[V];
#pragma unroll
    for (int j = 0; j < Pairs; ++j) {
      v[2 * j] = p[j].x;
      v[2 * j + 1] = p[j].y;
    }
    const uint4 r = pack16<kBF16>(v);
    uint8_t* to = row + static_cast<int64_t>(c) * Elem;
    if (whole(c, cols)) {
      *reinterpret_cast<uint4*>(to) = r;
    } else {
      const uint4 m = mask(c, cols);
      store_masked(to, r.x, m.x);
      store_masked(to + 4, r.y, m.y);
      store_masked(to + 8, r.z, m.z);
      store_masked(to + 12, r.w, m.w);
    }
  }
  __device__ static __forceinline__ void store_masked(uint8_t* p, uint32_t v, uint32_t m) {
    if (m == 0xFFFFFFFFu) *reinterpret_cast<uint32_t*>(p) = v;
    else if (m == 0x0000FFFFu) *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(v);
    else if (m == 0xFFFF0000u) *reinterpret_cast<uint16_t*>(p + 2) = static_cast<uint16_t>(v >> 16);
  }
  // values where there is no column become 0
  __device__ static __forceinline__ void clip(int c, int cols, float2 (&p)[Pairs]) {
    if (!whole(c, cols)) {
#pragma unroll
      for (int j = 0; j < Pairs; ++j) {
        if (!has(c, 2 * j, cols)) p[j].x = 0.0f;
        if (!has(c, 2 * j + 1, cols)) p[j].y = 0.0f;
      }
    }
  }
  __device__ static __forceinline__ void params(const void* v, bool bf16, int c, int cols, float none,
                                                float2 (&out)[Pairs]) {
    float a[V];
    if constexpr (!kShift) {
      load_params(v, bf16, c, none, a);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) a[j] = has(c, j, cols) ? load_param(v, bf16, c + j, none) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < Pairs; ++j) out[j] = make_float2(a[2 * j], a[2 * j + 1]);
  }
};

// (0 blocks: no bound on the registers; a bound of one lets it take more than
// four blocks of 256 threads an SM leave)
template <bool kBF16, bool kRms, bool kShift, int kCols, bool kWarp, int kThreads>
__global__ void __launch_bounds__(kThreads, kShift && !kRms && !kWarp ? 1024 / kThreads : 0)
    norm_fwd_row_kernel(const void* __restrict__ x, const void* __restrict__ gamma, const void* __restrict__ beta,
                        bool param_bf16, int64_t rows, int64_t cols, float eps, void* __restrict__ y,
                        float* __restrict__ mean, float* __restrict__ rstd, int32_t* __restrict__ dev_status) {
  using U = Unit<kBF16, kShift>;
  constexpr int kN = kCols / U::V, kPairs = U::Pairs;
  __shared__ __align__(16) float red[2][32];
  if (!kWarp && threadIdx.x < 64) red[threadIdx.x >> 5][threadIdx.x & 31] = 0.0f;
  if (!kWarp) __syncthreads();
  pdl_trigger();
  pdl_wait();
  const float inv = 1.0f / static_cast<float>(cols);
  const int ncols = static_cast<int>(cols);
  const int tpr = kWarp ? 32 : static_cast<int>(blockDim.x);
  const int t = kWarp ? static_cast<int>(threadIdx.x) & 31 : static_cast<int>(threadIdx.x);
  const int64_t first = kWarp ? static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32 : blockIdx.x;
  const int64_t step = kWarp ? static_cast<int64_t>(gridDim.x) * (blockDim.x / 32) : gridDim.x;
  const int64_t rb = cols * U::Elem;
  const int shift = kShift ? static_cast<int>(first * cols % U::V) : 0;  // step * cols is a multiple of V
  uint32_t turn = 0;

  const uint8_t* x_end = static_cast<const uint8_t*>(x) + rows * rb;
  U w[kN], next[kN];
  auto fetch = [&](int64_t row) {
    const uint8_t* xr = static_cast<const uint8_t*>(x) + row * rb;
#pragma unroll
    for (int k = 0; k < kN; ++k)
      if (U::column(t + k * tpr, shift) < ncols) next[k].load(xr, U::column(t + k * tpr, shift), x_end);
  };
  if (first < rows) fetch(first);
  float2 ga[kN][kPairs], be[kRms ? 1 : kN][kPairs];
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    const int c = U::column(t + k * tpr, shift);
    if (c < ncols) {
      U::params(gamma, param_bf16, c, ncols, 1.0f, ga[k]);
      if constexpr (!kRms) U::params(beta, param_bf16, c, ncols, 0.0f, be[k]);
    }
  }
  for (int64_t row = first; row < rows; row += step) {
#pragma unroll
    for (int k = 0; k < kN; ++k) w[k] = next[k].trimmed(U::column(t + k * tpr, shift), ncols);
    if (row + step < rows) fetch(row + step);
    float mu = 0.0f;
    if constexpr (!kRms) {
      float2 s = both(0.0f);
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        if (U::column(t + k * tpr, shift) < ncols) {
          float2 v[kPairs];
          w[k].pairs(v);
#pragma unroll
          for (int j = 0; j < kPairs; ++j) s = add2(s, v[j]);
        }
      }
      mu = row_sum<kWarp, kThreads / 32>(s.x + s.y, red, turn) * inv;
    }
    float2 q = both(0.0f);
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const int c = U::column(t + k * tpr, shift);
      if (c < ncols) {
        float2 v[kPairs];
        w[k].pairs(v);
#pragma unroll
        for (int j = 0; j < kPairs; ++j)
          if constexpr (!kRms) v[j] = add2(v[j], both(-mu));
        if constexpr (!kRms) U::clip(c, ncols, v);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) q = fma2(v[j], v[j], q);
      }
    }
    const float rs = 1.0f / sqrtf(row_sum<kWarp, kThreads / 32>(q.x + q.y, red, turn) * inv + eps);
    if (t == 0) {
      if (mean && !kRms) mean[row] = mu;
      if (rstd) rstd[row] = rs;
      // a NaN or infinity in the row, or sums past float32: rs is then 0 or NaN (infinite: eps = 0, constant row)
      if (dev_status && !(rs > 0.0f && isfinite(rs) && isfinite(mu))) atomicOr(dev_status, kDevNonfinite);
    }
    uint8_t* yr = static_cast<uint8_t*>(y) + row * rb;
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const int c = U::column(t + k * tpr, shift);
      if (c < ncols) {
        float2 v[kPairs];
        w[k].pairs(v);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          if constexpr (!kRms) v[j] = add2(v[j], both(-mu));
          v[j] = mul2(v[j], both(rs));
          if constexpr (kRms) v[j] = mul2(v[j], ga[k][j]);
          else v[j] = fma2(v[j], ga[k][j], be[k][j]);
        }
        U::store(yr, c, ncols, v);
      }
    }
  }
}

// Rows of more than 16384 columns: block b owns the rows [b rows / grid,
// (b + 1) rows / grid) and one row of each partial sum, in memory; a thread
// owns its columns of them.
template <bool kBF16, bool kRms>
__global__ void __launch_bounds__(kRowThreads)
    norm_bwd_kernel(const void* __restrict__ dy, const void* __restrict__ x, const void* __restrict__ gamma,
                    bool param_bf16, const float* __restrict__ mean, const float* __restrict__ rstd,
                    const void* __restrict__ dres, int64_t rows, int64_t cols, void* __restrict__ dx,
                    float* __restrict__ part_g, float* __restrict__ part_b, int32_t* __restrict__ dev_status) {
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
    if (threadIdx.x == 0 && dev_status && !isfinite((c1 + c2) * rs)) atomicOr(dev_status, kDevNonfinite);
    for (int64_t c = threadIdx.x; c < cols; c += kRowThreads) {
      const float xh = (load_elem<kBF16>(x, base + c) - mu) * rs;
      const float gv = load_elem<kBF16>(dy, base + c) * load_param(gamma, param_bf16, c, 1.0f);
      float v = (gv - c1 - xh * c2) * rs;
      if (dres) v += load_elem<kBF16>(dres, base + c);
      store_elem<kBF16>(dx, base + c, v);
    }
  }
}

// ---------------------------------------------------------------- backward: rows in registers
// A group of threads takes a row at a time: its columns' parts of dgamma and
// dbeta stay in a thread's registers over all the rows that the group takes,
// and the next row of x and dy is on its way while this one is worked on
// (kAhead); the row after that is asked for into L2 (float32 39.6 -> 34.3 us).
//
// Columns a thread: what a row costs beside its columns (two sums over the
// group, a barrier, addresses) is paid by every warp of it, so 16 columns
// instead of 8 take bf16 layer norm from 29.9 to 25.2 us at 4096 x 4096, two
// blocks of 256 threads an SM; float32, whose columns take twice the registers in
// flight, stays at 8.  The rows streamed through a ring in shared memory by
// bulk copies instead took 26.6 (RMS) and 36.1 us (layer).
//
// kMode: a block takes a row (0), a group of kTpr threads (1) or a warp (2);
// where a block holds several groups it joins their sums at the end.
constexpr int kMaxGroups = 15;  // a named barrier each beside the block's
constexpr int kL2Rows = 2;      // rows ahead that are asked for into L2

// Two sums over a warp with the shuffles of one: after the first exchange the
// lower lanes hold the first value's parts and the upper ones the second's.
// Lane 0 gets the first sum, lane 16 the second.
__device__ __forceinline__ float warp_sum2(float a, float b, int lane) {
  const bool up = lane & 16;
  float v = (up ? b : a) + __shfl_xor_sync(0xFFFFFFFFu, up ? a : b, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

template <bool kBF16, bool kRms, bool kShift, int kCols, int kMode, int kThreads, int kBlocks, bool kAhead, int kTpr>
__global__ void __launch_bounds__(kThreads, kBlocks)
    norm_bwd_row_kernel(const void* __restrict__ dy, const void* __restrict__ x, const void* __restrict__ gamma,
                        bool param_bf16, const float* __restrict__ mean, const float* __restrict__ rstd,
                        const void* __restrict__ dres, int64_t rows, int64_t cols, void* __restrict__ dx,
                            float* __restrict__ part_g, float* __restrict__ part_b, int32_t* __restrict__ dev_status) {
  using U = Unit<kBF16, kShift>;
  constexpr int kN = kCols / U::V, kPairs = U::Pairs;
  constexpr bool kKeep = kAhead;           // gamma in registers
  // and, from the sums to dx, xh and g = dy gamma instead of x and dy: in bf16
  // that takes 32 registers for 16 (16 columns), which layer norm does not have
  constexpr bool kHold = kThreads <= 512 && (kRms || !kBF16 || (kMode == 0 && kCols == 8));
  constexpr bool kJoin = kMode != 0;
  // [call][sum][group][warp]: a block's 32 warps, or 16 of each group, zeros past the last
  constexpr int kRow = kMode == 0 ? 32 : 16 * (kMaxGroups + 1);
  __shared__ __align__(16) float red[2][2][kRow];
  __shared__ __align__(16) float merge[kJoin ? kThreads * kCols : 1];
  if constexpr (kMode != 2) {
    for (int i = static_cast<int>(threadIdx.x); i < 4 * kRow; i += static_cast<int>(blockDim.x))
      (&red[0][0][0])[i] = 0.0f;
    __syncthreads();
  }
  pdl_trigger();
  pdl_wait();
  const float inv = 1.0f / static_cast<float>(cols);
  const int lane = threadIdx.x & 31;
  const int tpr = kMode == 2 ? 32 : kMode == 1 ? kTpr : static_cast<int>(blockDim.x);
  const int groups = kMode == 0 ? 1 : static_cast<int>(blockDim.x) / tpr;
  const int group = kMode == 0 ? 0 : static_cast<int>(threadIdx.x) / tpr;
  const int t = static_cast<int>(threadIdx.x) - group * tpr, warp = t >> 5;
  const int step = static_cast<int>(gridDim.x) * groups;
  const int ncols = static_cast<int>(cols);
  const int64_t rb = cols * U::Elem;
  int64_t row = static_cast<int64_t>(blockIdx.x) * groups + group;
  int64_t at = row * rb;
  const int shift = kShift ? static_cast<int>(row * cols % U::V) : 0;  // step * cols is a multiple of V
  uint32_t turn = 0;

  U wx[kHold ? 1 : kN], wd[kHold ? 1 : kN], nx[kN], nd[kN];
  float nmu = 0.0f, nrs = 0.0f;
  auto fetch = [&](int64_t r, int64_t from) {
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const int c = U::column(t + k * tpr, shift);
      if (c < ncols) {
        nx[k].load(static_cast<const uint8_t*>(x) + from, c, static_cast<const uint8_t*>(x) + rows * rb);
        nd[k].load(static_cast<const uint8_t*>(dy) + from, c, static_cast<const uint8_t*>(dy) + rows * rb);
      }
    }
    if constexpr (!kRms) nmu = mean[r];
    nrs = rstd[r];
  };
  if (row < rows) fetch(row, at);
  float2 ga[kKeep ? kN : 1][kPairs];
  float2 ag[kN][kPairs], ab[kRms ? 1 : kN][kPairs];
#pragma unroll
  for (int k = 0; k < kN; ++k) {
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      ag[k][j] = both(0.0f);
      if constexpr (!kRms) ab[k][j] = both(0.0f);
    }
    const int c = U::column(t + k * tpr, shift);
    if constexpr (kKeep)
      if (c < ncols) U::params(gamma, param_bf16, c, ncols, 1.0f, ga[k]);
  }
  for (; row < rows; row += step, at += step * rb) {
    const float mu = nmu, rs = nrs;
    float2 xc[kHold ? kN : 1][kPairs], gd[kHold ? kN : 1][kPairs];  // x and dy, then xh and g
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      if constexpr (kHold) {
        nx[k].trimmed(U::column(t + k * tpr, shift), ncols).pairs(xc[k]);
        nd[k].trimmed(U::column(t + k * tpr, shift), ncols).pairs(gd[k]);
      } else {
        wx[k] = nx[k].trimmed(U::column(t + k * tpr, shift), ncols);
        wd[k] = nd[k].trimmed(U::column(t + k * tpr, shift), ncols);
      }
    }
    if constexpr (kAhead)
      if (row + step < rows) fetch(row + step, at + step * rb);
    if (t == 0 && row + kL2Rows * step < rows) {
      const int64_t far = (row + kL2Rows * step) * rb, all = rows * rb;
      prefetch_l2(static_cast<const uint8_t*>(x) + far, rb, static_cast<const uint8_t*>(x) + all);
      prefetch_l2(static_cast<const uint8_t*>(dy) + far, rb, static_cast<const uint8_t*>(dy) + all);
      if (dres) prefetch_l2(static_cast<const uint8_t*>(dres) + far, rb, static_cast<const uint8_t*>(dres) + all);
    }
    float2 s1 = both(0.0f), s2 = both(0.0f);
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const int c = U::column(t + k * tpr, shift);
      if (c < ncols) {
        float2 xv[kPairs], dv[kPairs], g[kPairs];
        if constexpr (kHold) {
#pragma unroll
          for (int j = 0; j < kPairs; ++j) {
            xv[j] = xc[k][j];
            dv[j] = gd[k][j];
          }
        } else {
          wx[k].pairs(xv);
          wd[k].pairs(dv);
        }
        if constexpr (!kKeep) U::params(gamma, param_bf16, c, ncols, 1.0f, g);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          if constexpr (kKeep) g[j] = ga[k][j];
          if constexpr (!kRms) xv[j] = add2(xv[j], both(-mu));
          xv[j] = mul2(xv[j], both(rs));
          // dy xh once for both sums: g xh from g costs layer norm 31.7 us
          // against 27.0 at 2048 x 8192 bf16
          const float2 dxh = mul2(dv[j], xv[j]);
          ag[k][j] = add2(ag[k][j], dxh);
          s2 = fma2(g[j], dxh, s2);
          const float2 gv = mul2(g[j], dv[j]);
          if constexpr (!kRms) {
            ab[k][j] = add2(ab[k][j], dv[j]);
            s1 = add2(s1, gv);
          }
          if constexpr (kHold) {
            xc[k][j] = xv[j];
            gd[k][j] = gv;
          }
        }
      }
    }
    if (dx) {
      U wr[kN];
      if (dres) {
#pragma unroll
        for (int k = 0; k < kN; ++k)
          if (U::column(t + k * tpr, shift) < ncols)
            wr[k].load(static_cast<const uint8_t*>(dres) + at, U::column(t + k * tpr, shift),
                       static_cast<const uint8_t*>(dres) + rows * rb);
      }
      float c1 = 0.0f, c2;
      if constexpr (kRms) {
        c2 = warp_sum(s2.x + s2.y);
      } else {
        c2 = warp_sum2(s2.x + s2.y, s1.x + s1.y, lane);
        if constexpr (kMode == 2) {
          c1 = __shfl_sync(0xFFFFFFFFu, c2, 16);
          c2 = __shfl_sync(0xFFFFFFFFu, c2, 0);
        }
      }
      if constexpr (kMode != 2) {
        // One barrier a row: calls alternate between two buffers, so that a
        // thread that writes one again has passed the barrier of the call
        // between, which every thread reaches after its reads.
        float* r = red[turn & 1u][0] + (kMode == 0 ? 0 : 16 * group);
        ++turn;
        if (lane == 0) r[warp] = c2;
        if constexpr (!kRms)
          if (lane == 16) r[kRow + warp] = c2;
        if constexpr (kMode == 0) __syncthreads();
        else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(tpr) : "memory");
        constexpr int kWarps = kMode == 1 ? (kTpr + 127) / 128 * 4 : kThreads / 32;  // a multiple of four
        c2 = sum_warps<kWarps>(r);
        if constexpr (!kRms) c1 = sum_warps<kWarps>(r + kRow);
      }
      // dx = g rs + xh a + b: the factors are of the size of the formula's own
      // terms.  (x - mu) times c2 rs^2 would spare RMS norms a product, but
      // rs^2 leaves float32 where rs is 1e-19 or 1e19; times are within 4 %.
      const float a = -c2 * inv * rs, b = -c1 * inv * rs;
      // a NaN or infinity in the row or its statistics, or sums past float32
      if (t == 0 && dev_status && !isfinite(a + b)) atomicOr(dev_status, kDevNonfinite);
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const int c = U::column(t + k * tpr, shift);
        if (c < ncols) {
          float2 xv[kPairs], dv[kPairs], g[kPairs];
          if constexpr (kHold) {
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
              xv[j] = xc[k][j];
              dv[j] = gd[k][j];
            }
          } else {
            wx[k].pairs(xv);
            wd[k].pairs(dv);
            if constexpr (!kKeep) U::params(gamma, param_bf16, c, ncols, 1.0f, g);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
              if constexpr (kKeep) g[j] = ga[k][j];
              if constexpr (!kRms) xv[j] = add2(xv[j], both(-mu));
              xv[j] = mul2(xv[j], both(rs));
              dv[j] = mul2(g[j], dv[j]);
            }
          }
#pragma unroll
          for (int j = 0; j < kPairs; ++j) {
            if constexpr (kRms) xv[j] = mul2(xv[j], both(a));
            else xv[j] = fma2(xv[j], both(a), both(b));
            dv[j] = fma2(dv[j], both(rs), xv[j]);
          }
          if (dres) {
            wr[k].pairs(xv);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) dv[j] = add2(dv[j], xv[j]);
          }
          U::store(static_cast<uint8_t*>(dx) + at, c, ncols, dv);
        }
      }
    }
    if constexpr (!kAhead)
      if (row + step < rows) fetch(row + step, at + step * rb);
  }
  // this block's row of the partial sums
  auto put = [&](float* part, const float2(*acc)[kPairs]) {
    float* to = part + static_cast<int64_t>(blockIdx.x) * cols;
    float* into = kJoin ? merge + group * static_cast<int>(cols) : to;  // groups * cols <= threads * kCols
    if (kJoin) __syncthreads();                                        // the sum before this one is read
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const int c = U::column(t + k * tpr, shift);
      if (c < ncols) {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          if constexpr (kShift) {
            if (U::has(c, 2 * j, ncols)) into[c + 2 * j] = acc[k][j].x;
            if (U::has(c, 2 * j + 1, ncols)) into[c + 2 * j + 1] = acc[k][j].y;
          } else if (j % 2 == 0) {  // whole units begin on 16 bytes of the sums too
            *reinterpret_cast<float4*>(into + c + 2 * j) =
                make_float4(acc[k][j].x, acc[k][j].y, acc[k][(j + 1) % kPairs].x, acc[k][(j + 1) % kPairs].y);
          }
        }
      }
    }
    if (kJoin) {
      __syncthreads();
      for (int c = static_cast<int>(threadIdx.x); c < cols; c += static_cast<int>(blockDim.x)) {
        float s = 0.0f;
        for (int g = 0; g < groups; ++g) s += merge[g * static_cast<int>(cols) + c];
        to[c] = s;
      }
    }
  };
  if (part_g) put(part_g, ag);
  if constexpr (!kRms)
    if (part_b) put(part_b, ab);
}

// Blocks of the backward, each with one partial row of dgamma and dbeta: at
// most three per SM of a B200, never more than rows.
constexpr int64_t kNormParts = 444;

int norm_parts(int64_t rows) { return static_cast<int>(rows < kNormParts ? rows : kNormParts); }

struct FwdArgs {
  const void *x, *gamma, *beta;
  bool param_bf16;
  int64_t rows, cols;
  float eps;
  void* y;
  float *mean, *rstd;
  int32_t* dev_status;
  cudaStream_t stream;
};

// Resident blocks per SM of a kernel at so many threads (at most 1024; cached:
// every device of a process is taken to be alike).
template <class Kernel>
cudaError_t resident_blocks(Kernel kernel, int threads, int (&cache)[33], int* blocks) {
  int& slot = cache[threads / 32];
  *blocks = __atomic_load_n(&slot, __ATOMIC_RELAXED);
  if (*blocks > 0) return cudaSuccess;
  cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks, kernel, threads, 0);
  if (e != cudaSuccess) return e;
  if (*blocks < 1) *blocks = 1;
  __atomic_store_n(&slot, *blocks, __ATOMIC_RELAXED);
  return cudaSuccess;
}

// Threads that hold `cols` columns, kCols each, at any shift.
template <bool kBF16, bool kShift>
int row_threads(int64_t cols, int per_thread) {
  const int64_t held = cols + (kShift ? kVec<kBF16> - 1 : 0);
  return static_cast<int>((held + 32 * per_thread - 1) / (32 * per_thread) * 32);
}

// Blocks, such that the rows of a group are a multiple of V apart where it
// takes more than one (kShift): as many as fit at once.
template <bool kBF16, bool kShift>
int64_t row_blocks(int64_t rows, int64_t groups, int64_t resident) {
  const int64_t blocks = (rows + groups - 1) / groups;
  if (blocks <= resident) return blocks;
  return kShift ? std::max<int64_t>(resident / kVec<kBF16> * kVec<kBF16>, kVec<kBF16>) : resident;
}

template <bool kBF16, bool kRms, bool kShift, int kCols, bool kWarp, int kThreads>
cudaError_t norm_fwd_row(const DeviceInfo* di, const FwdArgs& a, int threads) {
  auto kernel = norm_fwd_row_kernel<kBF16, kRms, kShift, kCols, kWarp, kThreads>;
  static int cache[33] = {};
  int per_sm = 1;
  cudaError_t e = resident_blocks(kernel, threads, cache, &per_sm);
  if (e != cudaSuccess) return e;
  const int64_t blocks =
      row_blocks<kBF16, kShift>(a.rows, kWarp ? 4 : 1, static_cast<int64_t>(di->sm_count) * per_sm);
  return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(threads), 0, a.stream, 1u, a.x, a.gamma, a.beta,
                    a.param_bf16, a.rows, a.cols, a.eps, a.y, a.mean, a.rstd, a.dev_status);
}

template <bool kBF16, bool kRms, bool kShift>
cudaError_t norm_fwd_rows(const DeviceInfo* di, const FwdArgs& a, bool* taken) {
  constexpr int kSlack = kShift ? kVec<kBF16> - 1 : 0;
  *taken = true;
  if (a.cols + kSlack <= 256) return norm_fwd_row<kBF16, kRms, kShift, 8, true, 128>(di, a, 128);
  if (a.cols + kSlack <= 512) return norm_fwd_row<kBF16, kRms, kShift, 16, true, 128>(di, a, 128);
  // 16 columns a thread where they and their parameters fit 64 registers
  // (bf16), else 8: 4096 x 4096 bf16 layer 15.5 against 20.3 us, but float32
  // 32.1 against 24.1.  Compiled for at most so many threads, whose sums are
  // then read without a loop (4096 x 4096 bf16 layer 15.4 -> 14.7); layer norms
  // off their 16 bytes are held to 64 registers (8192 x 2050 25.5 -> 23.5).
  auto threads = [&](int c) { return row_threads<kBF16, kShift>(a.cols, c); };
  if constexpr (!kBF16) {
    if (threads(8) <= 256) return norm_fwd_row<kBF16, kRms, kShift, 8, false, 256>(di, a, threads(8));
    if (threads(8) <= 512) return norm_fwd_row<kBF16, kRms, kShift, 8, false, 512>(di, a, threads(8));
    if (threads(8) <= 1024) return norm_fwd_row<kBF16, kRms, kShift, 8, false, 1024>(di, a, threads(8));
  } else {
    if (threads(16) <= 128) return norm_fwd_row<kBF16, kRms, kShift, 16, false, 128>(di, a, threads(16));
    if (threads(16) <= 256) return norm_fwd_row<kBF16, kRms, kShift, 16, false, 256>(di, a, threads(16));
    if (threads(16) <= 512) return norm_fwd_row<kBF16, kRms, kShift, 16, false, 512>(di, a, threads(16));
  }
  if (threads(16) <= 1024) return norm_fwd_row<kBF16, kRms, kShift, 16, false, 1024>(di, a, threads(16));
  *taken = false;
  return cudaSuccess;
}

template <bool kBF16, bool kRms>
cudaError_t norm_fwd_t(const FwdArgs& a) {
  const DeviceInfo* di = current_device_info();
  if (!di) return cudaErrorInvalidDevice;
  bool taken = false;
  cudaError_t e = a.cols % kVec<kBF16> == 0 ? norm_fwd_rows<kBF16, kRms, false>(di, a, &taken)
                                            : norm_fwd_rows<kBF16, kRms, true>(di, a, &taken);
  if (e != cudaSuccess || taken) return e;
  const unsigned grid = static_cast<unsigned>(a.rows < (1 << 20) ? a.rows : (1 << 20));
  return launch_pdl(norm_fwd_kernel<kBF16, kRms>, dim3(grid), dim3(kRowThreads), 0, a.stream, 1u, a.x, a.gamma, a.beta,
                    a.param_bf16, a.rows, a.cols, a.eps, a.y, a.mean, a.rstd, a.dev_status);
}

struct BwdArgs {
  const void *dy, *x, *gamma;
  bool param_bf16;
  const float *mean, *rstd;
  const void* dres;
  int64_t rows, cols;
  void* dx;
  float *dgamma, *dbeta;
  float *part_g, *part_b;  // null where dgamma, dbeta are
  int32_t* dev_status;
  cudaStream_t stream;
};

// Rows' partial sums, or, from a single block, the sums themselves.
void norm_bwd_outputs(BwdArgs& a, int parts) {
  if (parts == 1) {
    a.part_g = a.dgamma;
    a.part_b = a.dbeta;
  }
}

template <bool kBF16, bool kRms, bool kShift, int kCols, int kMode, int kThreads, int kBlocks, bool kAhead, int kTpr = 0>
cudaError_t norm_bwd_row(const DeviceInfo* di, BwdArgs a, int* parts) {
  auto kernel = norm_bwd_row_kernel<kBF16, kRms, kShift, kCols, kMode, kThreads, kBlocks, kAhead, kTpr>;
  const int tpr = kTpr ? kTpr : kMode == 2 ? 32 : row_threads<kBF16, kShift>(a.cols, kCols);
  int groups = kMode == 0 ? 1 : std::min(kThreads / tpr, kMaxGroups);
  // few rows: one a group
  const int64_t sms = di->sm_count;
  if (a.rows < groups * sms) groups = static_cast<int>(std::max<int64_t>(1, (a.rows + sms - 1) / sms));
  static int cache[33] = {};
  int per_sm = 1;
  cudaError_t e = resident_blocks(kernel, groups * tpr, cache, &per_sm);
  if (e != cudaSuccess) return e;
  const int64_t blocks = row_blocks<kBF16, kShift>(
      a.rows, groups, std::min<int64_t>(sms * std::min(per_sm, 3), norm_parts(a.rows)));
  *parts = static_cast<int>(blocks);
  norm_bwd_outputs(a, *parts);
  return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(groups * tpr), 0, a.stream, 1u, a.dy, a.x,
                    a.gamma, a.param_bf16, a.mean, a.rstd, a.dres, a.rows, a.cols, a.dx, a.part_g, a.part_b, a.dev_status);
}

template <bool kBF16, bool kRms, bool kShift>
cudaError_t norm_bwd_rows(const DeviceInfo* di, BwdArgs a, int* parts) {
  constexpr int kSlack = kShift ? kVec<kBF16> - 1 : 0;
  const int64_t held = a.cols + kSlack;
  if constexpr (kBF16) {
    if (held <= 256) return norm_bwd_row<kBF16, kRms, kShift, 8, 2, 256, 1, true>(di, a, parts);
    // A block a row and 8 columns a thread: few rows, since the code is shorter
    // to fetch and run once (layer norms, us: 148 x 2048 9.9 -> 5.7, 300 x 4096
    // 8.9 -> 7.3, 1700 x 4096 15.9 -> 15.6, 300 x 1024 6.3 -> 5.8; it loses where
    // narrow rows are many, 700 x 1024 7.1 -> 7.5, and on long runs); the widths
    // whose groups of 16 columns a thread are two a block, at any count (8192 x
    // 2048 28.6 -> 27.4, 8192 x 1792 28.4 -> 26.2); and rows off their 16 bytes,
    // whose masks cost registers that 16 columns do not leave (8192 x 1537
    // 38.3 -> 33.6; 4096 x 2049 27.9 -> 31.3, but RMS 20.5 -> 19.1).
    const bool few = a.rows <= (held <= 1024 ? 3 : 12) * static_cast<int64_t>(di->sm_count);
    if (held <= 4096 && (few || (held > 1536 && held <= 2048) || (kShift && held > 1024)))
      return norm_bwd_row<kBF16, kRms, kShift, 8, 0, 512, 1, true>(di, a, parts);
    if (held <= 512) return norm_bwd_row<kBF16, kRms, kShift, 16, 2, 256, 2, true>(di, a, parts);
    // groups of a size known when compiled (layer 8192 x 1536 25.4 -> 23.1 us,
    // 16384 x 1000 27.6 -> 25.9), and one a block where a block has no room for
    // two (4096 x 4096 31.0 -> 25.2)
    if (held <= 1024) return norm_bwd_row<kBF16, kRms, kShift, 16, 1, 256, 2, true, 64>(di, a, parts);
    if (held <= 1536) return norm_bwd_row<kBF16, kRms, kShift, 16, 1, 192, 2, true, 96>(di, a, parts);
    if (held <= 4096) return norm_bwd_row<kBF16, kRms, kShift, 16, 0, 256, 2, true>(di, a, parts);
    if (held <= 8192) return norm_bwd_row<kBF16, kRms, kShift, 16, 0, 512, 1, true>(di, a, parts);
  } else {
    if (held <= 256) return norm_bwd_row<kBF16, kRms, kShift, 8, 2, 512, 1, true>(di, a, parts);
    if (held <= 512) return norm_bwd_row<kBF16, kRms, kShift, 8, 1, 512, 1, true, 64>(di, a, parts);
    if (held <= 768) return norm_bwd_row<kBF16, kRms, kShift, 8, 1, 480, 1, true, 96>(di, a, parts);
    if (held <= 1024) return norm_bwd_row<kBF16, kRms, kShift, 8, 1, 512, 1, true, 128>(di, a, parts);
    if (held <= 1536) return norm_bwd_row<kBF16, kRms, kShift, 8, 1, 384, 1, true, 192>(di, a, parts);
    if (held <= 2048) return norm_bwd_row<kBF16, kRms, kShift, 8, 1, 512, 1, true, 256>(di, a, parts);
    if (held <= 4096) return norm_bwd_row<kBF16, kRms, kShift, 8, 0, 512, 1, true>(di, a, parts);
    if (held <= 8192) return norm_bwd_row<kBF16, kRms, kShift, 8, 0, 1024, 1, true>(di, a, parts);
  }
  if (held <= 16384) return norm_bwd_row<kBF16, kRms, kShift, 16, 0, 1024, 1, false>(di, a, parts);
  *parts = norm_parts(a.rows);
  norm_bwd_outputs(a, *parts);
  return launch_pdl(norm_bwd_kernel<kBF16, kRms>, dim3(*parts), dim3(kRowThreads), 0, a.stream, 1u, a.dy, a.x, a.gamma,
                    a.param_bf16, a.mean, a.rstd, a.dres, a.rows, a.cols, a.dx, a.part_g, a.part_b, a.dev_status);
}

template <bool kBF16, bool kRms>
cudaError_t norm_bwd_t(const BwdArgs& a, int* parts) {
  const DeviceInfo* di = current_device_info();
  if (!di) return cudaErrorInvalidDevice;
  return a.cols % kVec<kBF16> == 0 ? norm_bwd_rows<kBF16, kRms, false>(di, a, parts)
                                   : norm_bwd_rows<kBF16, kRms, true>(di, a, parts);
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
  return fn(FwdArgs{x, gamma, beta, param_bf16, rows, cols, eps, y, mean, rstd, dev_status, stream});
}

cudaError_t launch_norm_bwd(const void* dy, const void* x, bool bf16, const void* gamma, bool param_bf16, bool rms,
                            const float* mean, const float* rstd, const void* dres, int64_t rows, int64_t cols,
                            void* dx, float* dgamma, float* dbeta, int32_t* dev_status, void* workspace,
                            cudaStream_t stream) {
  float* pg = static_cast<float*>(workspace);
  float* pb = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + norm_bwd_workspace_bytes(rows, cols) / 2);
  auto fn = bf16 ? (rms ? norm_bwd_t<true, true> : norm_bwd_t<true, false>)
                 : (rms ? norm_bwd_t<false, true> : norm_bwd_t<false, false>);
  int parts = 0;
  cudaError_t e = fn(BwdArgs{dy, x, gamma, param_bf16, mean, rstd, dres, rows, cols, dx, dgamma, dbeta,
                             dgamma ? pg : nullptr, dbeta ? pb : nullptr, dev_status, stream},
                     &parts);
  if (e != cudaSuccess || (!dgamma && !dbeta) || parts == 1) return e;
  if (!dgamma) return launch_column_sums(pb, dbeta, nullptr, nullptr, parts, cols, stream);
  return launch_column_sums(pg, dgamma, dbeta ? pb : nullptr, dbeta, parts, cols, stream);
}

}  // namespace falqon
