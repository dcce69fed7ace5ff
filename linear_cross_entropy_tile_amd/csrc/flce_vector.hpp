// Vectors of bf16 and fp32 values in registers, shared by the kernels of the
// operators beside the head.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace flce {

typedef uint32_t eu32x4 __attribute__((ext_vector_type(4)));
typedef float ef32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 ebf16x2 __attribute__((ext_vector_type(2)));
typedef float ef32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) {
  return __builtin_bit_cast(float, w & 0xFFFF0000u);
}
// Two floats to a bf16 pair, nearest even.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((ef32x2{lo, hi}), ebf16x2));
}
__device__ __forceinline__ void unpack8(const eu32x4& w, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ eu32x4 pack8(const float (&v)[8]) {
  return eu32x4{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]),
                bf16_pair(v[6], v[7])};
}

// A value of T at any address its elements may have: global memory takes vector
// accesses at every byte, only slower where they cross a cache line.
template <class T>
__device__ __forceinline__ T load_any(const void* p) {
  T v;
  __builtin_memcpy(&v, p, sizeof(T));
  return v;
}
template <class T>
__device__ __forceinline__ void store_any(void* p, const T& v) {
  __builtin_memcpy(p, &v, sizeof(T));
}

// The same past the caches (nontemporal).
template <class T>
__device__ __forceinline__ void stream_any(void* p, const T& v) {
  typedef T loose __attribute__((aligned(2)));
  __builtin_nontemporal_store(v, static_cast<loose*>(p));
}

// Eight consecutive values of an array of bf16 or fp32 from element i on, at any
// address; the first `n` of them where n < 8 (the others read as 0 or stay).
template <bool F32>
__device__ __forceinline__ void load8(const void* p, int64_t i, int n, float (&v)[8]) {
  if (n >= 8) {
    if constexpr (F32) {
      const float* q = static_cast<const float*>(p) + i;
      const ef32x4 a = load_any<ef32x4>(q), b = load_any<ef32x4>(q + 4);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[k] = a[k];
        v[4 + k] = b[k];
      }
    } else {
      unpack8(load_any<eu32x4>(static_cast<const uint16_t*>(p) + i), v);
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    v[k] = 0.f;
    if (k < n) {
      if constexpr (F32)
        v[k] = static_cast<const float*>(p)[i + k];
      else
        v[k] = bf16_lo(static_cast<const uint16_t*>(p)[i + k]);
    }
  }
}
template <bool F32>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
  if constexpr (F32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<uint16_t*>(p)[i] = (uint16_t)bf16_pair(v, 0.f);
}
template <bool F32, bool STREAM = false>
__device__ __forceinline__ void store8(void* p, int64_t i, int n, const float (&v)[8]) {
  if constexpr (F32) {
    float* q = static_cast<float*>(p) + i;
    if (n >= 8) {
      const ef32x4 a{v[0], v[1], v[2], v[3]}, b{v[4], v[5], v[6], v[7]};
      if constexpr (STREAM) {
        stream_any(q, a);
        stream_any(q + 4, b);
      } else {
        store_any(q, a);
        store_any(q + 4, b);
      }
      return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) q[k] = v[k];
  } else {
    uint16_t* q = static_cast<uint16_t*>(p) + i;
    const eu32x4 w = pack8(v);
    if (n >= 8) {
      if constexpr (STREAM)
        stream_any(q, w);
      else
        store_any(q, w);
      return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) q[k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
  }
}

}  // namespace flce
