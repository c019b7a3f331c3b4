// The global norm of many gradient tensors, and clipping by it.
//
//   norm = sqrt(sum of g^2 over every element of every tensor)
//   coef = max_norm / norm where norm > max_norm, else 1
//   out  = g (factor coef), rounded once to g's type
//
// Bound by HBM: every gradient is read for the norm, read again for the
// scaling and written.  The tensors are cut into chunks of 16 KB; a block takes
// a run of them, the same one in both kernels, and scales it from its end
// backwards, so that what the L2 still holds of it is not read from memory
// again.  A table of the tensors travels in the kernel's parameters, so a call
// copies nothing to the device and can be captured.
//
// Measured on a B200 (us; in brackets the floor at 6.55 TB/s with one read):
// the 448 adapter gradients of a stack of 32 blocks at rank 64, 320 MB: 160 (98;
// 147 with both reads from memory); at rank 16: 39 (24); the four of one layer:
// 5.4 (0.3; two launches).
//
// Sums: eight (bf16) or four (float32) squares are added in float32, which is
// exact enough while the sum stays away from the ends of float32's range, and
// in float64 otherwise; everything above one 16-byte vector is float64.  So
// neither gradients near 1e-30 nor near 1e30 spoil the norm.  The blocks'
// sums are joined in a fixed order: the result does not depend on the
// schedule.
#include <algorithm>

#include "elem.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace falqon {
namespace {

constexpr int kClipThreads = 256;
constexpr int kClipVecs = 4;        // 16-byte vectors of a thread in a chunk
constexpr int kClipChunk = kClipThreads * kClipVecs * 16;  // bytes
constexpr int kClipTensors = 512;   // tensors of one launch
constexpr int kClipFew = 32;        // the table of a launch of few tensors: its parameters take less time to arrive
// Blocks an SM (of a B200's 148): five for long runs (48 registers); four, and
// the registers that the norm asks for, where a block has no more than four
// chunks, which also lets the second kernel's blocks in beside the first's (14
// tensors of rank 16: 5.7 us against 7.8).
constexpr int kClipMany = 5, kClipFewer = 4, kClipSms = 148;
constexpr int kClipBlocks = kClipMany * kClipSms;
// The last chunks of a block's run that the norm leaves in the L2 for the
// scaling, 6 x 740 x 16 KB = 73 MB in all, of which it then finds 57 to 59;
// what it reads before them gives way first (with the fifth block, 448 tensors of rank 64: 172 -> 160 us).
constexpr uint32_t kClipKeep = 6;

template <int kTensors>
struct ClipTable {
  const void* in[kTensors];
  void* out[kTensors];
  int64_t numel[kTensors];
  uint32_t end[kTensors];  // chunks up to and including tensor i
  uint8_t bf16[kTensors];
  int32_t n;
  uint32_t chunks;
};
static_assert(sizeof(ClipTable<kClipTensors>) <= 32000, "kernel parameters");

// The tensor that chunk c belongs to: the first whose end is past c.
template <int kTensors>
__device__ __forceinline__ int clip_tensor(const ClipTable<kTensors>& t, uint32_t c) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (t.end[mid] > c) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// This block's run of chunks.
template <int kTensors>
__device__ __forceinline__ void clip_run(const ClipTable<kTensors>& t, uint32_t& c0, uint32_t& c1) {
  c0 = static_cast<uint32_t>(static_cast<uint64_t>(t.chunks) * blockIdx.x / gridDim.x);
  c1 = static_cast<uint32_t>(static_cast<uint64_t>(t.chunks) * (blockIdx.x + 1) / gridDim.x);
}

// Sum of the squares of one vector: float32 while the sum is in
// [2^-60, 2^120] (a square below 2^-126 is then nothing beside it, and none
// overflowed), else float64.
template <int kN>
__device__ __forceinline__ double square_sum(const float (&v)[kN]) {
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < kN; ++j) s = fmaf(v[j], v[j], s);
  if (s >= 8.673617e-19f && s <= 1.329228e36f) return static_cast<double>(s);
  double d = 0.0;
#pragma unroll
  for (int j = 0; j < kN; ++j) d = fma(static_cast<double>(v[j]), static_cast<double>(v[j]), d);
  return d;
}

// Elements [e0, e1) of a tensor, at most a chunk.
template <bool kBF16>
__device__ __forceinline__ double chunk_square_sum(const void* p, int64_t e0, int64_t e1, bool keep) {
  constexpr int kV = kVec<kBF16>;
  const uint4* v = static_cast<const uint4*>(p) + e0 / kV;  // chunks begin on whole vectors
  const int n = static_cast<int>(e1 - e0), whole = n / kV;
  double acc = 0.0;
  uint4 q[kClipVecs];
#pragma unroll
  for (int k = 0; k < kClipVecs; ++k)
    if (static_cast<int>(threadIdx.x) + k * kClipThreads < whole)
      q[k] = keep ? v[threadIdx.x + k * kClipThreads] : __ldcs(v + threadIdx.x + k * kClipThreads);
#pragma unroll
  for (int k = 0; k < kClipVecs; ++k) {
    if (static_cast<int>(threadIdx.x) + k * kClipThreads < whole) {
      float f[kV];
      unpack16<kBF16>(q[k], f);
      acc += square_sum(f);
    }
  }
  const int tail = whole * kV + static_cast<int>(threadIdx.x);
  if (tail < n) {
    const double x = load_elem<kBF16>(p, e0 + tail);
    acc = fma(x, x, acc);
  }
  return acc;
}

template <bool kBF16>
__device__ __forceinline__ void scale_chunk(const void* p, void* o, int64_t e0, int64_t e1, float by, bool zero) {
  constexpr int kV = kVec<kBF16>;
  const uint4* v = static_cast<const uint4*>(p) + e0 / kV;
  uint4* to = static_cast<uint4*>(o) + e0 / kV;
  const int n = static_cast<int>(e1 - e0), whole = n / kV;
  uint4 q[kClipVecs];
#pragma unroll
  for (int k = 0; k < kClipVecs; ++k)  // read and written for the last time here
    if (static_cast<int>(threadIdx.x) + k * kClipThreads < whole) q[k] = __ldcs(v + threadIdx.x + k * kClipThreads);
#pragma unroll
  for (int k = 0; k < kClipVecs; ++k) {
    if (static_cast<int>(threadIdx.x) + k * kClipThreads < whole) {
      float f[kV];
      unpack16<kBF16>(q[k], f);
#pragma unroll
      for (int j = 0; j < kV; ++j) f[j] = zero ? 0.0f : f[j] * by;
      __stcs(to + threadIdx.x + k * kClipThreads, pack16<kBF16>(f));
    }
  }
  const int tail = whole * kV + static_cast<int>(threadIdx.x);
  if (tail < n) store_elem<kBF16>(o, e0 + tail, zero ? 0.0f : load_elem<kBF16>(p, e0 + tail) * by);
}

// Chunk c of tensor i: its elements.
template <int kTensors>
__device__ __forceinline__ void chunk_elements(const ClipTable<kTensors>& t, int i, uint32_t c, int64_t& e0, int64_t& e1) {
  const int64_t size = kClipChunk / (t.bf16[i] ? 2 : 4);
  e0 = static_cast<int64_t>(c - (i ? t.end[i - 1] : 0u)) * size;
  e1 = e0 + size < t.numel[i] ? e0 + size : t.numel[i];
}

// part[b] = this block's share (added to what an earlier launch of the call
// left there when `add`).
template <int kTensors, int kMinBlocks>
__global__ void __launch_bounds__(kClipThreads, kMinBlocks)
    clip_norm_kernel(const __grid_constant__ ClipTable<kTensors> t, double* __restrict__ part, bool add) {
  pdl_trigger();
  pdl_wait();
  __shared__ double red[32];
  double acc = 0.0;
  uint32_t c0, c1;
  clip_run(t, c0, c1);
  if (c0 < c1) {
    int i = clip_tensor(t, c0);
    for (uint32_t c = c0; c < c1; ++c) {
      while (t.end[i] <= c) ++i;
      int64_t e0, e1;
      chunk_elements(t, i, c, e0, e1);
      const bool keep = c + kClipKeep >= c1;
      acc += t.bf16[i] ? chunk_square_sum<true>(t.in[i], e0, e1, keep) : chunk_square_sum<false>(t.in[i], e0, e1, keep);
    }
  }
  acc = block_sum(acc, red);
  if (threadIdx.x == 0) part[blockIdx.x] = add ? part[blockIdx.x] + acc : acc;
}

// Every block joins the partial sums (in the same order) and scales its
// chunks; block 0 of the call's first launch publishes the results.
template <int kTensors>
__global__ void __launch_bounds__(kClipThreads)
    clip_scale_kernel(const __grid_constant__ ClipTable<kTensors> t, const double* __restrict__ part, int parts,
                      float max_norm, float factor, bool scale, float* __restrict__ norm, float* __restrict__ coef,
                      int32_t* __restrict__ dev_status) {
  pdl_trigger();
  pdl_wait();
  __shared__ double red[32];
  double acc = 0.0;
  for (int i = threadIdx.x; i < parts; i += kClipThreads) acc += part[i];
  acc = block_sum(acc, red);
  const bool finite = isfinite(acc);  // squares of finite float32 values cannot overflow float64 sums
  const double n = sqrt(acc);
  const double c = !finite ? 0.0 : (n > static_cast<double>(max_norm) ? static_cast<double>(max_norm) / n : 1.0);
  if (blockIdx.x == 0 && threadIdx.x == 0 && norm) {
    *norm = static_cast<float>(n);
    if (coef) *coef = static_cast<float>(c);
    if (!finite && dev_status) atomicOr(dev_status, kDevNonfinite);
  }
  if (!scale) return;
  const float by = static_cast<float>(static_cast<double>(factor) * c);
  uint32_t c0, c1;
  clip_run(t, c0, c1);
  if (c0 >= c1) return;
  int i = clip_tensor(t, c1 - 1);
  for (uint32_t k = c1; k-- > c0;) {
    while (i > 0 && t.end[i - 1] > k) --i;
    int64_t e0, e1;
    chunk_elements(t, i, k, e0, e1);
    if (t.bf16[i]) scale_chunk<true>(t.in[i], t.out[i], e0, e1, by, !finite);
    else scale_chunk<false>(t.in[i], t.out[i], e0, e1, by, !finite);
  }
}

// Fills `t` from tensor `i` on; returns the next tensor.  A launch takes up to
// kTensors tensors that hold elements.
template <int kTensors>
int clip_table(ClipTable<kTensors>& t, int i, int n, const void* const* grads, void* const* outs,
               const falqon_dtype* dtypes, const int64_t* numel) {
  t.n = 0;
  t.chunks = 0;
  for (; i < n && t.n < kTensors; ++i) {
    if (numel[i] == 0) continue;
    const bool bf16 = dtypes[i] == FALQON_DTYPE_BF16;
    const int64_t size = kClipChunk / (bf16 ? 2 : 4);
    t.in[t.n] = grads[i];
    t.out[t.n] = outs ? outs[i] : nullptr;
    t.numel[t.n] = numel[i];
    t.bf16[t.n] = bf16;
    t.chunks += static_cast<uint32_t>((numel[i] + size - 1) / size);
    t.end[t.n] = t.chunks;
    ++t.n;
  }
  return i;
}

template <int kTensors>
cudaError_t clip_grads_t(int n, const void* const* grads, const falqon_dtype* dtypes, const int64_t* numel,
                         float max_norm, float factor, void* const* outs, float* norm, float* coef,
                         int32_t* dev_status, double* part, cudaStream_t stream) {
  ClipTable<kTensors> t;
  auto many = [&]() { return t.chunks > 4u * kClipBlocks; };
  auto grid_of = [&]() -> unsigned {
    return many() ? kClipBlocks : std::min<unsigned>(std::max(t.chunks, 1u), kClipFewer * kClipSms);
  };
  int parts = 0;
  for (int i = 0; i < n || parts == 0;) {  // at least one launch: no elements at all give norm 0
    i = clip_table(t, i, n, grads, outs, dtypes, numel);
    // the first launch sets how many sums there are; later ones add to them
    const unsigned grid = parts ? static_cast<unsigned>(parts) : (i < n ? kClipBlocks : grid_of());
    auto kernel = many() ? clip_norm_kernel<kTensors, kClipMany> : clip_norm_kernel<kTensors, 1>;
    cudaError_t e = launch_pdl(kernel, dim3(grid), dim3(kClipThreads), 0, stream, 1u, t, part, parts != 0);
    if (e != cudaSuccess) return e;
    parts = static_cast<int>(grid);
  }
  bool first = true;
  for (int i = 0; i < n || first;) {
    i = clip_table(t, i, n, grads, outs, dtypes, numel);
    cudaError_t e = launch_pdl(clip_scale_kernel<kTensors>, dim3(outs ? grid_of() : 1u), dim3(kClipThreads), 0, stream, 1u, t, part, parts,
                               max_norm, factor, outs != nullptr, first ? norm : nullptr, coef, dev_status);
    if (e != cudaSuccess) return e;
    first = false;
    if (!outs) break;
  }
  return cudaSuccess;
}

}  // namespace

int64_t clip_chunk_elements() { return kClipChunk / 4; }

size_t clip_workspace_bytes() { return align_up(kClipBlocks * sizeof(double), 256); }

cudaError_t launch_clip_grads(int n, const void* const* grads, const falqon_dtype* dtypes, const int64_t* numel,
                              float max_norm, float factor, void* const* outs, float* norm, float* coef,
                              int32_t* dev_status, void* workspace, cudaStream_t stream) {
  auto fn = n <= kClipFew ? clip_grads_t<kClipFew> : clip_grads_t<kClipTensors>;
  return fn(n, grads, dtypes, numel, max_norm, factor, outs, norm, coef, dev_status, static_cast<double*>(workspace),
            stream);
}

}  // namespace falqon
