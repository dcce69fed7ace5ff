// Kernels of the gradients' norm and of the AdamW update over many tensors (gfx950).
//
// A launch takes up to a table's length of tensors, which is a kernel argument: a
// captured launch keeps it, and nothing is copied to the device. Blocks are numbered
// over the tensors' chunks; each finds its tensor in the table.
//
// Norm: each block writes the float64 sum of its chunk's squares, one block adds
// those up. Update: one block first turns the device's step count into the step's
// constants and raises it; then each value is read, updated and written once. States
// in 8 bits take 16 values a lane, so that the 256 values that share a scale lie in a
// row of 16 lanes and their largest magnitude takes four exchanges within it.
//
// What bounds them: the bytes; with 8-bit states also the instructions. A bf16 weight of
// 590 M values with fp32 states takes 2.44 ms (22 bytes a value, 5.3 TB/s), with 8-bit
// ones 1.2 ms (10 bytes, 4.9 TB/s), 356 M values in 97 tensors with fp32 copies 1.88 ms
// (28 bytes, 5.3 TB/s).
// The norm of 590 M bf16 values takes 200 us by itself (5.9 TB/s) and 245 behind an update
// that leaves its own values in the caches. The bytes bound it: sums in fp32 take the same
// 200 us, and more or smaller chunks, or two loads in flight instead of four, more.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "flce_step_plan.hpp"
#include "flce_vector.hpp"

namespace flce {

// ---- norm ----------------------------------------------------------------------------

struct NormTable {
  const void* grad[kNormTensors];
  int64_t size[kNormTensors];
  int32_t first[kNormTensors];   // first block, within the launch
  uint8_t f32[kNormTensors];
  int count;
};
struct NormArgs {
  NormTable t;
  int64_t chunk;
  double* parts;                 // of the launch's first block
};

// Largest k with first[k] <= b.
template <class First>
__device__ __forceinline__ int table_find(const First& first, int count, int b) {
  int lo = 0, hi = count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= b)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Four loads a thread are in flight.
template <bool F32>
__device__ __forceinline__ double norm_chunk_sum(const void* p, int64_t i0, int64_t i1) {
  constexpr int U = 4, kStride = 8 * kNormThreads;
  double s[U] = {0.0, 0.0, 0.0, 0.0};
  int64_t i = i0 + threadIdx.x * 8;
  for (; i + (U - 1) * kStride + 8 <= i1; i += U * kStride) {
    float v[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) load8<F32>(p, i + u * kStride, 8, v[u]);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < 8; ++k) s[u] += (double)v[u][k] * (double)v[u][k];
  }
  for (; i < i1; i += kStride) {
    const int64_t left = i1 - i;
    float v[8];
    load8<F32>(p, i, left < 8 ? (int)left : 8, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) s[0] += (double)v[k] * (double)v[k];
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

template <int WAVES>
__device__ __forceinline__ double block_sum_f64(double s, double* sh) {
  for (int d = 32; d > 0; d >>= 1) s += __shfl_down(s, d, 64);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = s;
  __syncthreads();
  double t = sh[0];
  for (int w = 1; w < WAVES; ++w) t += sh[w];
  return t;
}

__global__ void __launch_bounds__(kNormThreads) norm_parts_kernel(NormArgs a) {
  __shared__ double sh[kNormThreads / 64];
  const int b = blockIdx.x;
  const int k = table_find(a.t.first, a.t.count, b);
  const int64_t i0 = (int64_t)(b - a.t.first[k]) * a.chunk;
  const int64_t end = i0 + a.chunk < a.t.size[k] ? i0 + a.chunk : a.t.size[k];
  const double s = a.t.f32[k] ? norm_chunk_sum<true>(a.t.grad[k], i0, end)
                              : norm_chunk_sum<false>(a.t.grad[k], i0, end);
  const double t = block_sum_f64<kNormThreads / 64>(s, sh);
  if (threadIdx.x == 0) a.parts[b] = t;
}

__global__ void __launch_bounds__(1024) norm_total_kernel(const double* parts, int64_t n,
                                                          double max_norm, float* norm,
                                                          float* scale, int32_t* header) {
  __shared__ double sh[16];
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += 1024) s += parts[i];
  const double t = block_sum_f64<16>(s, sh);
  if (threadIdx.x != 0) return;
  const double r = sqrt(t);
  *norm = (float)r;
  if (scale != nullptr) {
    double c = 1.0;
    if (max_norm > 0.0 && r > max_norm) c = max_norm / r;
    if (!(r < INFINITY)) c = NAN;
    *scale = (float)c;
  }
  header[0] = header[1] = 0;
}

// ---- AdamW ---------------------------------------------------------------------------

// The step's constants, the same for every value.
struct AdamCoef {
  float scale, keep;       // of the gradient; 1 - lr weight_decay
  float b1, a1, b2, a2;    // betas and 1 - betas
  float rise, root, eps;   // lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  int live;                // 0: the step is skipped
  uint32_t key;            // of the random bits
};

// A hash of 32 bits: every output bit depends on every input bit. The constants are
// the leading fraction bits of the golden ratio and of sqrt(3), made odd.
__host__ __device__ __forceinline__ uint32_t hash32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x9E3779B1u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}

__device__ __forceinline__ double power(double b, int64_t t) {
  double r = 1.0;
  for (; t > 0; t >>= 1) {
    if (t & 1) r *= b;
    b *= b;
  }
  return r;
}

struct AdamCoefArgs {
  double lr, beta1, beta2, eps, weight_decay;
  uint64_t seed;
  const float* lr_device;
  const float* grad_scale;
  int64_t* step;
  int32_t* header;
  AdamCoef* coef;
};
__global__ void __launch_bounds__(64) adamw_coef_kernel(AdamCoefArgs a) {
  if (threadIdx.x != 0) return;
  const float s = a.grad_scale != nullptr ? *a.grad_scale : 1.f;
  const double lr = a.lr_device != nullptr ? (double)*a.lr_device : a.lr;
  const int64_t t = *a.step + 1;
  AdamCoef c;
  c.live = fabsf(s) < INFINITY ? 1 : 0;
  c.scale = s;
  c.keep = (float)(1.0 - lr * a.weight_decay);
  c.b1 = (float)a.beta1;
  c.a1 = (float)(1.0 - a.beta1);
  c.b2 = (float)a.beta2;
  c.a2 = (float)(1.0 - a.beta2);
  c.rise = (float)(lr / (1.0 - power(a.beta1, t)));
  c.root = (float)(1.0 / sqrt(1.0 - power(a.beta2, t)));
  c.eps = (float)a.eps;
  c.key = hash32(hash32((uint32_t)a.seed ^ hash32((uint32_t)(a.seed >> 32))) ^ (uint32_t)t);
  *a.coef = c;
  if (c.live) *a.step = t;
  a.header[0] = a.header[1] = 0;
}

struct AdamEntry {
  void* param;
  const void* grad;
  float* master;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t size;
};
enum { ADAM_PARAM_F32 = 1, ADAM_GRAD_F32 = 2 };
struct AdamTable {
  AdamEntry e[kAdamTensors];
  int32_t first[kAdamTensors];   // first block, within the launch
  int32_t number[kAdamTensors];  // in the call's list
  uint8_t kind[kAdamTensors];
  int count;
};
struct AdamArgs {
  AdamTable t;
  const AdamCoef* coef;
};

// Random bits of value i of a tensor of key k: 16 for the weight; in `moments` the
// upper 16 for the first and the lower 16 for the second.
struct AdamBits {
  uint32_t p, moments;
};
__device__ __forceinline__ AdamBits adam_bits(uint32_t key, uint32_t i) {
  const uint32_t h = hash32(i ^ key);
  uint32_t g = (h ^ 0x6A09E667u) * 0x9E3779B1u;
  g ^= g >> 16;
  return {h >> 16, g};
}

// fp32 bits of x rounded to bf16, up with the probability of the part cut off.
__device__ __forceinline__ float bf16_stochastic(float x, uint32_t bits) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x);
  const uint32_t up = (b + bits) & 0xFFFF0000u;
  return (b & 0x7F800000u) == 0x7F800000u ? x : __builtin_bit_cast(float, up);
}

// The gradient scaled, and both moments.
__device__ __forceinline__ void adam_moments(const AdamCoef& c, float g, float& m, float& v) {
#pragma clang fp contract(off)
  g = g * c.scale;
  m = m * c.b1 + g * c.a1;
  v = v * c.b2 + (g * g) * c.a2;
}
// The weight, from the root r of the second moment. The quotient's reciprocal is the
// hardware's (1 ulp): the update is far below the weight.
__device__ __forceinline__ float adam_weight(const AdamCoef& c, float p, float m, float r) {
#pragma clang fp contract(off)
  return p * c.keep - c.rise * (m * __builtin_amdgcn_rcpf(r * c.root + c.eps));
}

// Root within 1 ulp. The instruction flushes denormals, which a scale of 2^32 takes out
// of them.
__device__ __forceinline__ float root_near(float v) {
  const bool tiny = v < 0x1p-96f;
  const float r = __builtin_amdgcn_sqrtf(tiny ? v * 0x1p32f : v);
  return tiny ? r * 0x1p-16f : r;
}
// Roots rounded to the nearest: the last bit of a root that is kept in 8 bits can decide
// a code, and with it a block's scale. One Newton step from the reciprocal root on x and
// on 1 / (2 x), then the remainder, in 11 instruction slots a value against sqrtf's 20
// (equal to it for every mantissa); values that it does not hold for (0, below 2^-96,
// infinities, NaN) take sqrtf. Returns infinity if there is a NaN, else 0.
__device__ __forceinline__ float roots16(const float (&v)[16], float (&r)[16]) {
  bool odd = false;
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const float y = __builtin_amdgcn_rsqf(v[k]);
    float x = v[k] * y, h = 0.5f * y;
    const float e = __builtin_fmaf(-h, x, 0.5f);
    x = __builtin_fmaf(x, e, x);
    h = __builtin_fmaf(h, e, h);
    r[k] = __builtin_fmaf(__builtin_fmaf(-x, x, v[k]), h, x);
    odd = odd || !(v[k] >= 0x1p-96f && v[k] < INFINITY);
  }
  if (odd) {
#pragma unroll
    for (int k = 0; k < 16; ++k) r[k] = sqrtf(v[k]);
#pragma unroll
    for (int k = 0; k < 16; ++k) sum += r[k];
  }
  return sum != sum ? INFINITY : 0.f;
}

// W values of an update with fp32 states, from element i on (n of them).
template <bool P32, bool G32, bool MASTER, bool SR>
__device__ __forceinline__ void adam_f32(const AdamEntry& e, const AdamCoef& c, uint32_t key,
                                         int64_t i, int n) {
  float p[8], g[8], m[8], v[8];
  if constexpr (MASTER)
    load8<true>(e.master, i, n, p);
  else
    load8<P32>(e.param, i, n, p);
  load8<G32>(e.grad, i, n, g);
  load8<true>(e.m, i, n, m);
  load8<true>(e.v, i, n, v);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    adam_moments(c, g[k], m[k], v[k]);
    p[k] = adam_weight(c, p[k], m[k], root_near(v[k]));
  }
  store8<true>(e.m, i, n, m);
  store8<true>(e.v, i, n, v);
  if constexpr (MASTER) store8<true>(e.master, i, n, p);
  if constexpr (SR && !P32 && !MASTER) {
    const uint32_t k0 = hash32(key ^ (uint32_t)((uint64_t)i >> 32));
#pragma unroll
    for (int k = 0; k < 8; ++k) p[k] = bf16_stochastic(p[k], adam_bits(k0, (uint32_t)i + k).p);
  }
  store8<P32>(e.param, i, n, p);
}

// 16 codes in four words, from element i on (n of them).
__device__ __forceinline__ void load_codes(const void* p, int64_t i, int n, uint32_t (&w)[4]) {
  const uint8_t* q = static_cast<const uint8_t*>(p) + i;
  if (n >= 16) {
    const eu32x4 x = load_any<eu32x4>(q);
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = x[k];
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = 0;
#pragma unroll
  for (int k = 0; k < 16; ++k)
    if (k < n) w[k >> 2] |= (uint32_t)q[k] << (8 * (k & 3));
}
__device__ __forceinline__ void store_codes(void* p, int64_t i, int n, const uint32_t (&w)[4]) {
  uint8_t* q = static_cast<uint8_t*>(p) + i;
  if (n >= 16) {
    store_any(q, eu32x4{w[0], w[1], w[2], w[3]});
    return;
  }
#pragma unroll
  for (int k = 0; k < 16; ++k)
    if (k < n) q[k] = (uint8_t)(w[k >> 2] >> (8 * (k & 3)));
}
template <bool F32>
__device__ __forceinline__ void load16(const void* p, int64_t i, int n, float (&v)[16]) {
  float a[8], b[8];
  load8<F32>(p, i, n, a);
  load8<F32>(p, i + 8, n - 8, b);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    v[k] = a[k];
    v[8 + k] = b[k];
  }
}
template <bool F32>
__device__ __forceinline__ void store16(void* p, int64_t i, int n, const float (&v)[16]) {
  float a[8], b[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    a[k] = v[k];
    b[k] = v[8 + k];
  }
  store8<F32>(p, i, n, a);
  store8<F32>(p, i + 8, n - 8, b);
}

// The largest of a row of 16 lanes, in all of them.
template <int CTRL>
__device__ __forceinline__ float row_rotated(float v) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ float row16_max(float v) {
  v = fmaxf(v, row_rotated<0x128>(v));  // row_ror:8
  v = fmaxf(v, row_rotated<0x124>(v));  // row_ror:4
  v = fmaxf(v, row_rotated<0x122>(v));  // row_ror:2
  return fmaxf(v, row_rotated<0x121>(v));
}

constexpr float kTinyBlock = 0x1p-100f;

// Codes of 16 values whose block of 256 lies in the row of 16 lanes; returns the
// block's scale. POSITIVE: values >= 0, of which those above 0 get a code above 0. SR:
// stochastic rounding by the upper 16 of `bits` (the others 0), which the conversion adds
// to the part that it cuts off. top: 0, or infinity if the lane has a NaN, which the
// maximum passes over: the block then reads as NaN, as it does with an infinity among its
// values, whose scale is infinite and every code 0 or NaN.
template <bool SR, bool POSITIVE>
__device__ __forceinline__ float encode16(const float (&x)[16], float top,
                                          const uint32_t (&bits)[16], uint32_t (&w)[4]) {
#pragma clang fp contract(off)
#pragma unroll
  for (int k = 0; k < 16; ++k) top = fmaxf(top, fabsf(x[k]));
  top = row16_max(top);
  const bool live = top >= kTinyBlock;
  const float up = live ? 448.f * (1.f / top) : 0.f;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      y[k] = x[4 * q + k] * up;
      if constexpr (POSITIVE) y[k] = y[k] > 0.f ? fmaxf(y[k], 0x1p-9f) : y[k];
    }
    int word = 0;
    if constexpr (SR) {
      word = __builtin_amdgcn_cvt_sr_fp8_f32(y[0], (int)bits[4 * q], word, 0);
      word = __builtin_amdgcn_cvt_sr_fp8_f32(y[1], (int)bits[4 * q + 1], word, 1);
      word = __builtin_amdgcn_cvt_sr_fp8_f32(y[2], (int)bits[4 * q + 2], word, 2);
      word = __builtin_amdgcn_cvt_sr_fp8_f32(y[3], (int)bits[4 * q + 3], word, 3);
    } else {
      word = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], word, false);
      word = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], word, true);
    }
    w[q] = (uint32_t)word;
  }
  return live ? top * (1.f / 448.f) : 0.f;
}
__device__ __forceinline__ void decode16(const uint32_t (&w)[4], float (&x)[16]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const ef32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[q], false);
    const ef32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[q], true);
    x[4 * q] = a[0];
    x[4 * q + 1] = a[1];
    x[4 * q + 2] = b[0];
    x[4 * q + 3] = b[1];
  }
}

// 16 values of an update with 8-bit states, from element i on (n of them, none for
// lanes past the tensor, which still take part in their row's maximum).
template <bool P32, bool G32, bool MASTER, bool SR>
__device__ __forceinline__ void adam_8bit(const AdamEntry& e, const AdamCoef& c, uint32_t key,
                                          int64_t i, int n) {
#pragma clang fp contract(off)
  float p[16], g[16], m[16], v[16];
  uint32_t mw[4], vw[4], mb[16], vb[16];
  if constexpr (MASTER)
    load16<true>(e.master, i, n, p);
  else
    load16<P32>(e.param, i, n, p);
  load16<G32>(e.grad, i, n, g);
  load_codes(e.m, i, n, mw);
  load_codes(e.v, i, n, vw);
  const int64_t block = i / kStateBlock;
  const float ms = n > 0 ? e.m_scale[block] : 0.f, vs = n > 0 ? e.v_scale[block] : 0.f;
  decode16(mw, m);
  decode16(vw, v);
  const uint32_t k0 = SR ? hash32(key ^ (uint32_t)((uint64_t)i >> 32)) : 0;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const float q = v[k] * vs;
    m[k] = m[k] * ms;
    v[k] = q * q;
    adam_moments(c, g[k], m[k], v[k]);
  }
  // A NaN of the gradient or of the states is one of the second moment too.
  float r[16];
  const float lost = roots16(v, r);
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    p[k] = adam_weight(c, p[k], m[k], r[k]);
    if constexpr (SR) {
      const AdamBits b = adam_bits(k0, (uint32_t)i + k);
      mb[k] = b.moments & 0xFFFF0000u;
      vb[k] = b.moments << 16;
      if constexpr (!P32 && !MASTER) p[k] = bf16_stochastic(p[k], b.p);
    }
  }
  // Lanes and values past the end: a gradient, weight and moments of 0 give 0.
  const float ms1 = encode16<SR, false>(m, lost, mb, mw);
  const float vs1 = encode16<SR, true>(r, lost, vb, vw);
  if (n <= 0) return;
  store_codes(e.m, i, n, mw);
  store_codes(e.v, i, n, vw);
  if ((threadIdx.x & 15) == 0) {
    e.m_scale[block] = ms1;
    e.v_scale[block] = vs1;
  }
  if constexpr (MASTER) store16<true>(e.master, i, n, p);
  store16<P32>(e.param, i, n, p);
}

template <bool P32, bool G32, bool MASTER, bool EIGHT, bool SR>
__device__ __forceinline__ void adam_chunk(const AdamEntry& e, const AdamCoef& c, uint32_t key,
                                           int64_t i0) {
  if constexpr (EIGHT) {
    const int64_t i = i0 + threadIdx.x * 16, left = e.size - i;
    adam_8bit<P32, G32, MASTER, SR>(e, c, key, i, left > 16 ? 16 : (left > 0 ? (int)left : 0));
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t i = i0 + (h * kAdamThreads + threadIdx.x) * 8, left = e.size - i;
      if (left > 0) adam_f32<P32, G32, MASTER, SR>(e, c, key, i, left > 8 ? 8 : (int)left);
    }
  }
}

template <bool EIGHT, bool SR>
__global__ void __launch_bounds__(kAdamThreads) adamw_kernel(AdamArgs a) {
  const AdamCoef c = *a.coef;
  if (!c.live) return;
  const int k = table_find(a.t.first, a.t.count, blockIdx.x);
  const AdamEntry& e = a.t.e[k];
  const int64_t i0 = (int64_t)((int)blockIdx.x - a.t.first[k]) * kAdamChunk;
  const uint32_t key = hash32(c.key + (uint32_t)a.t.number[k] * 0x6A09E667u);
  const int kind = a.t.kind[k];
  const bool g32 = (kind & ADAM_GRAD_F32) != 0;
  if (kind & ADAM_PARAM_F32) {
    if (g32)
      adam_chunk<true, true, false, EIGHT, SR>(e, c, key, i0);
    else
      adam_chunk<true, false, false, EIGHT, SR>(e, c, key, i0);
  } else if (e.master != nullptr) {
    if (g32)
      adam_chunk<false, true, true, EIGHT, SR>(e, c, key, i0);
    else
      adam_chunk<false, false, true, EIGHT, SR>(e, c, key, i0);
  } else {
    if (g32)
      adam_chunk<false, true, false, EIGHT, SR>(e, c, key, i0);
    else
      adam_chunk<false, false, false, EIGHT, SR>(e, c, key, i0);
  }
}

}  // namespace flce
