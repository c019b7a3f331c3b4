// Element helpers of the bandwidth-bound kernels (norm.cu, epilogue.cu,
// clip.cu): 16-byte vectors of bf16 or float32 as float32 values, one
// parameter of either type, and block reductions in a fixed order.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>
#include <cstring>

namespace falqon {

// Two float32 operations in one instruction (each rounded as its scalar form).
__device__ __forceinline__ uint64_t f2_bits(float2 a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ float2 f2_of(uint64_t a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)), "l"(f2_bits(c)));
  return f2_of(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)));
  return f2_of(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)));
  return f2_of(r);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

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

// kBytes (2, 4, 8 or 16) of a row: its words, and the values they hold.
template <int kBytes>
struct Words {
  static constexpr int N = kBytes < 4 ? 1 : kBytes / 4;
  uint32_t w[N];
};

template <int kBytes>
__device__ __forceinline__ Words<kBytes> load_words(const void* p) {
  Words<kBytes> r;
  if constexpr (kBytes == 16) {
    const uint4 q = *static_cast<const uint4*>(p);
    r.w[0] = q.x; r.w[1] = q.y; r.w[2] = q.z; r.w[3] = q.w;
  } else if constexpr (kBytes == 8) {
    const uint2 q = *static_cast<const uint2*>(p);
    r.w[0] = q.x; r.w[1] = q.y;
  } else if constexpr (kBytes == 4) {
    r.w[0] = *static_cast<const uint32_t*>(p);
  } else {
    r.w[0] = *static_cast<const uint16_t*>(p);
  }
  return r;
}

// Values in kBytes of bf16 or float32.
template <bool kBF16, int kBytes>
constexpr int kValues = kBytes / (kBF16 ? 2 : 4);

template <bool kBF16, int kBytes>
__device__ __forceinline__ void values_of(const Words<kBytes>& r, float (&v)[kValues<kBF16, kBytes>]) {
#pragma unroll
  for (int j = 0; j < kValues<kBF16, kBytes>; ++j) {
    if constexpr (!kBF16) v[j] = __uint_as_float(r.w[j]);
    else v[j] = __uint_as_float(j & 1 ? r.w[j / 2] & 0xFFFF0000u : r.w[j / 2] << 16);
  }
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

// kN consecutive parameters from element i on (a multiple of kN; the vector is
// 16-byte aligned).
template <int kN>
__device__ __forceinline__ void load_params(const void* p, bool bf16, int64_t i, float none, float (&v)[kN]) {
  if (!p) {
#pragma unroll
    for (int j = 0; j < kN; ++j) v[j] = none;
  } else if (bf16) {
    values_of<true, 2 * kN>(load_words<2 * kN>(static_cast<const uint16_t*>(p) + i), v);
  } else if constexpr (kN == 8) {
    float a[4], b[4];
    values_of<false, 16>(load_words<16>(static_cast<const float*>(p) + i), a);
    values_of<false, 16>(load_words<16>(static_cast<const float*>(p) + i + 4), b);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = a[j];
      v[j + 4] = b[j];
    }
  } else {
    values_of<false, 4 * kN>(load_words<4 * kN>(static_cast<const float*>(p) + i), v);
  }
}

// Half of one lane's 64-byte row: one 256-bit access where `wide` (the address
// is then a multiple of 32), else two of 128 bits.
__device__ __forceinline__ void load_global_32B(const void* p, bool wide, uint32_t (&v)[8]) {
  if (wide) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "l"(p));
  } else {
    const uint4 a = static_cast<const uint4*>(p)[0], b = static_cast<const uint4*>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

__device__ __forceinline__ void store_global_32B(void* p, bool wide, const uint32_t (&v)[8]) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    static_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
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
