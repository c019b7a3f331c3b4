// Element helpers of the bandwidth-bound kernels (norm.cu, epilogue.cu,
// clip.cu): 16-byte vectors of bf16 or float32 as float32 values, one
// parameter of either type, and block reductions in a fixed order.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>
#include <cstring>

namespace falqon {

// Elements of one 16-byte vector.
template <bool kBF16>
constexpr int kVec = kBF16 ? 8 : 4;

template <bool kBF16>
__device__ __forceinline__ void unpack16(const uint4& q, float (&v)[kVec<kBF16>]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (kBF16) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    } else {
      v[j] = __uint_as_float(w[j]);
    }
  }
}

// Two values rounded to bf16, the first in the low half.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  uint32_t w;
  memcpy(&w, &b, 4);
  return w;
}

// Rounded once, to nearest even (bf16), or kept (float32).
template <bool kBF16>
__device__ __forceinline__ uint4 pack16(const float (&v)[kVec<kBF16>]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (kBF16) {
      w[j] = pack2(v[2 * j], v[2 * j + 1]);
    } else {
      w[j] = __float_as_uint(v[j]);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool kBF16>
__device__ __forceinline__ float load_elem(const void* p, int64_t i) {
  if constexpr (kBF16)
    return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
  else
    return static_cast<const float*>(p)[i];
}

template <bool kBF16>
__device__ __forceinline__ void store_elem(void* p, int64_t i, float v) {
  if constexpr (kBF16)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(p)[i] = v;
}

// A parameter vector of either type; `none` where there is no vector.
__device__ __forceinline__ float load_param(const void* p, bool bf16, int64_t i, float none) {
  if (!p) return none;
  return bf16 ? load_elem<true>(p, i) : load_elem<false>(p, i);
}

template <class T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Sum over the block, in every thread, in an order that depends on the block
// size alone.  `red` holds 32 values; the barriers let it be reused at once.
template <class T>
__device__ __forceinline__ T block_sum(T v, T* red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int warps = static_cast<int>(blockDim.x) >> 5;
  v = warp_sum(v);
  if (lane == 0) red[warp] = v;
  __syncthreads();
  v = warp_sum(lane < warps ? red[lane] : T(0));
  __syncthreads();
  return v;
}

}  // namespace falqon
