// Kernels of the logits of some rows (gfx950): out = cap(hidden weight + bias).
//
// With few rows the product is bound by the one pass over the weight, so the weight
// goes from memory straight into registers (logits_kernel). A wave takes a strip of
// 128 vocabulary columns and part of the hidden dimension in steps of 32: lane (c, g)
// = (l % 16, l / 16) loads 16 bytes, the columns 8c .. 8c+7, of each of the eight
// weight rows 8g .. 8g+7 of a step. v_mfma_f32_16x16x32_bf16 wants eight consecutive k
// of one column in a lane: a byte permute of two rows' words pairs their values of one
// column, so the eight loads hold the A operands of eight products, the j-th of
// which takes the 16 columns 8c + j. The B operand are 16 tokens, 16 bytes of a
// hidden row a lane. A lane then holds, for one token, eight consecutive columns:
// 32 or 16 bytes of the output. The waves of a block share the hidden dimension (step
// by step in turn) and add up their sums in LDS in a fixed order. No weight row has to
// be aligned, so any vocabulary is read in place.
//
// With many rows the matrix units bound it, and the head's block tile of 256 columns
// by 256 tokens takes it (logits_tile_kernel), or, where rows of the weight are not
// aligned, logits_wide_kernel. make_logits_plan says which and why.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "flce_gemm.hpp"
#include "flce_step_plan.hpp"
#include "flce_vector.hpp"

namespace flce {

typedef __bf16 lbf16x8 __attribute__((ext_vector_type(8)));
typedef float lf32x4 __attribute__((ext_vector_type(4)));

struct LogitsArgs {
  const uint16_t* hidden;
  const uint16_t* weight;
  const float* bias;
  int64_t N, H, V;
  float cap, inv_cap;  // cap 0: none
  void* out;
  int64_t ld_out;
  int passes;          // logits_kernel: groups of 16 MT tokens
  int split_steps;     // steps of the hidden dimension a block row (blockIdx.y) takes
  float* parts;        // sums of the splits [splits, N, V], where there are several
  // logits_tile_kernel
  uint16_t* image;     // blocked hidden: strips of 256 tokens
  int hkb, VT, TB;     // K blocks a strip; vocabulary and token tiles
};

// c tanh(z / c), within 2^-23 c of it and exact to fp32 for small z.
__device__ __forceinline__ float soft_cap(float z, float c, float inv_c) {
  const float x = z * inv_c, q = x * x;
  const float t = __builtin_amdgcn_exp2f(-2.f * kLog2e * fabsf(x));
  const float far = copysignf((1.f - t) * __builtin_amdgcn_rcpf(1.f + t), x);
  const float near = x * (1.f + q * (q * (2.f / 15.f) - 1.f / 3.f));
  return c * (fabsf(x) < 0.04f ? near : far);
}

// LDS traffic of the block is complete; loads from memory may still be on their way.
__device__ __forceinline__ void lds_barrier() {
  wait_lgkmcnt0();
  block_barrier();
}

// Bias and cap of the eight (n) columns from col on.
__device__ __forceinline__ void logits_finish(const LogitsArgs& a, int64_t col, int n,
                                              float (&z)[8]) {
  if (a.bias != nullptr) {
    float b[8];
    load8<true>(a.bias, col, n, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] += b[j];
  }
  if (a.cap > 0.f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = soft_cap(z[j], a.cap, a.inv_cap);
  }
}

// The lane's eight columns of eight weight rows.
struct WeightStep {
  eu32x4 w[8];
};
// p: the same for all lanes, `off` the lane's bytes from there, so that a load takes
// its address from scalar registers and one vector register.
__device__ __forceinline__ void load_weight(const uint16_t* p, uint32_t off, int64_t V,
                                            WeightStep& s) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    s.w[i] = load_any<eu32x4>(reinterpret_cast<const char*>(p + i * V) + off);
}
// In a vocabulary of less than eight ids: the first `cols` columns.
__device__ __forceinline__ void load_weight_few(const uint16_t* p, uint32_t off, int64_t V,
                                                int cols, WeightStep& s) {
  for (int i = 0; i < 8; ++i) {
    const uint16_t* q = p + i * V + off / 2;
    eu32x4 x{0, 0, 0, 0};
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < cols) x[c >> 1] |= (uint32_t)q[c] << (16 * (c & 1));
    s.w[i] = x;
  }
}
// A operand of column j: its eight k values.
__device__ __forceinline__ lbf16x8 weight_column(const WeightStep& s, int j) {
  // Byte selectors: the low or the high halves of two words.
  const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
  eu32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = __builtin_amdgcn_perm(s.w[2 * i + 1][j >> 1], s.w[2 * i][j >> 1], sel);
  return __builtin_bit_cast(lbf16x8, r);
}

// MT: groups of 16 tokens a block takes, W: its waves. Blocks that read the same strip
// for other tokens are eight apart in number, so that they run on one XCD at about the
// same time and all but the first find the strip in its L2.
template <int MT, int W, bool OUT32>
__global__ void __launch_bounds__(64 * W, MT >= 2 ? (MT >= 4 ? 2 : 3) : 4)
logits_kernel(LogitsArgs a) {
  __shared__ float sh[W][8][4][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int c = lane & 15, g = lane >> 4;
  const int group = (int)blockIdx.x / (8 * a.passes), in = (int)blockIdx.x % (8 * a.passes);
  const int64_t v0 = (int64_t)(group * 8 + (in & 7)) * kLogitStrip;
  if (v0 >= a.V) return;
  const int64_t t0 = (int64_t)(in >> 3) * (16 * MT);
  // Lane c's columns start at 8c of the strip; where the vocabulary ends, at its last
  // eight, and those that belong to a lane before are not stored again.
  const int64_t last = a.V >= 8 ? a.V - 8 : 0;
  // Rows past the last token read the first one's values; their results are dropped.
  uint32_t hoff[MT];  // bytes, below 2^31
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int64_t t = t0 + 16 * m + c;
    hoff[m] = (uint32_t)(2 * ((t < a.N ? t : 0) * a.H + 8 * g));
  }
  lf32x4 acc[MT][8];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[m][j] = lf32x4{0.f, 0.f, 0.f, 0.f};

  auto hidden_step = [&](int64_t k, eu32x4 (&h)[MT]) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
      h[m] = *reinterpret_cast<const eu32x4*>(reinterpret_cast<const char*>(a.hidden + k) +
                                              hoff[m]);
  };
  auto multiply = [&](WeightStep& s, const eu32x4 (&h)[MT]) {
    // Here and no earlier: the compiler would pair the words of a step in flight
    // before the products of the step at hand, and wait for them.
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 8; ++i) __asm__ volatile("" : "+v"(s.w[i]));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const lbf16x8 w = weight_column(s, j);
#pragma unroll
      for (int m = 0; m < MT; ++m)
        acc[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            w, __builtin_bit_cast(lbf16x8, h[m]), acc[m][j], 0, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  const int first = (int)blockIdx.y * a.split_steps;
  const int whole = (int)(a.H / 32);  // full steps
  const int steps = whole < first + a.split_steps ? whole : first + a.split_steps;
  const int64_t base = v0 < last ? v0 : last;
  const int64_t v = v0 + 8 * c < last ? v0 + 8 * c : last;
  const uint32_t woff = (uint32_t)(2 * (8 * g * a.V + (v - base)));
  const uint16_t* strip = a.weight + base;
  const int cols = a.V < 8 ? (int)a.V : 8;
  if (first + wave < steps) {
    if (a.V >= 8) {
      // The next step's loads are in flight while one is multiplied (the last step's
      // are repeated, for nothing).
      WeightStep s0, s1;
      eu32x4 h0[MT], h1[MT];
      auto load = [&](int step, WeightStep& s, eu32x4 (&h)[MT]) {
        const int64_t k = 32 * (int64_t)(step < steps ? step : steps - 1);
        load_weight(strip + k * a.V, woff, a.V, s);
        hidden_step(k, h);
      };
      int step = first + wave;
      load(step, s0, h0);
      while (true) {
        load(step + W, s1, h1);
        multiply(s0, h0);
        step += W;
        if (step >= steps) break;
        load(step + W, s0, h0);
        multiply(s1, h1);
        step += W;
        if (step >= steps) break;
      }
    } else {
      for (int step = first + wave; step < steps; step += W) {
        WeightStep s;
        eu32x4 h[MT];
        load_weight_few(strip + 32 * (int64_t)step * a.V, woff, a.V, cols, s);
        hidden_step(32 * (int64_t)step, h);
        multiply(s, h);
      }
    }
  }
  // What is left of the hidden dimension, in groups of eight.
  const int64_t k = 32 * (int64_t)whole;
  if (k < a.H && blockIdx.y == gridDim.y - 1 && wave == (whole - first) % W) {
    WeightStep s;
    eu32x4 h[MT];
#pragma unroll
    for (int i = 0; i < 8; ++i) s.w[i] = eu32x4{0, 0, 0, 0};
#pragma unroll
    for (int m = 0; m < MT; ++m) h[m] = eu32x4{0, 0, 0, 0};
    if (k + 8 * g < a.H) {
      if (a.V >= 8)
        load_weight(strip + k * a.V, woff, a.V, s);
      else
        load_weight_few(strip + k * a.V, woff, a.V, cols, s);
      hidden_step(k, h);
    }
    multiply(s, h);
  }

  // Sum over the waves. Wave w < 4 finishes row i = w of the lanes' four rows of the
  // products: of lane (c, g) the columns 8 (4 g + w) on.
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) sh[wave][j][i][lane] = acc[m][j][i];
    __syncthreads();
    const int64_t t = t0 + 16 * m + c;
    const int64_t want = v0 + 8 * (4 * g + wave);
    const int64_t col = want < last ? want : last;
    const int skip = (int)(want - col);  // columns of a lane before
    if (wave < 4 && t < a.N && want < a.V) {
      float z[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        z[j] = sh[0][j][wave][lane];
#pragma unroll
        for (int w = 1; w < W; ++w) z[j] += sh[w][j][wave][lane];
      }
      if (gridDim.y > 1) {
        // Columns of a lane before get the same sums again.
        store8<true>(a.parts, ((int64_t)blockIdx.y * a.N + t) * a.V + col, cols, z);
        continue;
      }
      logits_finish(a, col, cols, z);
      if (skip == 0) {
        store8<OUT32>(a.out, t * a.ld_out + col, cols, z);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j >= skip) store1<OUT32>(a.out, t * a.ld_out + col + j, z[j]);
      }
    }
  }
}

// Adds up the splits of eight columns a thread, in order; the parts come from the caches.
template <bool OUT32>
__global__ void __launch_bounds__(256) logits_sum_kernel(LogitsArgs a, int splits) {
  const int64_t col = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  const int64_t t = blockIdx.y;
  if (col >= a.V) return;
  const int n = a.V - col < 8 ? (int)(a.V - col) : 8;
  float z[8], x[8];
  load8<true>(a.parts, t * a.V + col, n, z);
  for (int s = 1; s < splits; ++s) {
    load8<true>(a.parts, ((int64_t)s * a.N + t) * a.V + col, n, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] += x[j];
  }
  logits_finish(a, col, n, z);
  store8<OUT32>(a.out, t * a.ld_out + col, n, z);
}

// Up to 64 WM tokens at once for more than 64 of them, in any vocabulary of 128 ids or
// more. The waves share the strip's weight rows, of which each thread brings 128 / WM
// bytes a step to LDS, some steps ahead in registers and one in LDS; wave w takes the
// tokens 64 w .. 64 w + 63 of the pass, reads the strip's eight rows of its lanes from
// LDS and goes on like logits_kernel. One barrier a step. With one wave a SIMD and 254
// registers the wait for LDS before the products is what bounds it: 200 tokens of hidden
// size 4096 and 50257 ids take 192 us (430 TFLOP/s, 2.4 TB/s), 1024 take 650 us (648
// TFLOP/s).
template <int WM, bool OUT32>
__global__ void __launch_bounds__(64 * WM, 2) logits_wide_kernel(LogitsArgs a) {
  constexpr int kPieces = 8 / WM;           // 16-byte pieces a thread and step
  constexpr int kAhead = 8 / kPieces;       // steps in registers
  __shared__ __attribute__((aligned(16))) char sh[2][32 * 2 * kLogitStrip];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int group = (int)blockIdx.x / (8 * a.passes), in = (int)blockIdx.x % (8 * a.passes);
  const int64_t v0 = (int64_t)(group * 8 + (in & 7)) * kLogitStrip;
  if (v0 >= a.V) return;
  // The last strip starts where it ends with the vocabulary; ids below v0 are not stored
  // again.
  const int64_t base = v0 < a.V - kLogitStrip ? v0 : a.V - kLogitStrip;
  const int64_t t0 = (int64_t)(in >> 3) * (64 * WM) + 64 * wave;
  const bool idle = t0 >= a.N;
  const int whole = (int)(a.H / 32);  // steps
  const uint16_t* strip = a.weight + base;

  uint32_t hoff[4];  // bytes, at most 2^31; rows past the last token read the first one's
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const int64_t t = t0 + 16 * m + c;
    hoff[m] = (uint32_t)(2 * ((t < a.N ? t : 0) * a.H + 8 * g));
  }
  lf32x4 acc[4][8];
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[m][j] = lf32x4{0.f, 0.f, 0.f, 0.f};

  // Piece p of thread tid: row (p * 64 WM + tid) / 16 of the step, columns 8 (tid % 16).
  const uint32_t poff = (uint32_t)(2 * ((tid >> 4) * a.V + 8 * (tid & 15)));
  auto fetch = [&](int step, eu32x4 (&r)[kPieces]) {
#pragma unroll
    for (int p = 0; p < kPieces; ++p)
      r[p] = load_any<eu32x4>(reinterpret_cast<const char*>(
                                  strip + (32 * (int64_t)step + p * (4 * WM)) * a.V) + poff);
  };
  auto put = [&](int buffer, const eu32x4 (&r)[kPieces]) {
#pragma unroll
    for (int p = 0; p < kPieces; ++p)
      *reinterpret_cast<eu32x4*>(&sh[buffer][(p * (64 * WM) + tid) * 16]) = r[p];
  };
  auto hidden_step = [&](int step, eu32x4 (&h)[4]) {
    const char* src = reinterpret_cast<const char*>(a.hidden + 32 * (int64_t)step);
#pragma unroll
    for (int m = 0; m < 4; ++m) h[m] = *reinterpret_cast<const eu32x4*>(src + hoff[m]);
  };
  auto multiply = [&](int buffer, const eu32x4 (&h)[4]) {
    WeightStep w;
    const char* src = &sh[buffer][(8 * g * 16 + c) * 16];
#pragma unroll
    for (int i = 0; i < 8; ++i) w.w[i] = *reinterpret_cast<const eu32x4*>(src + i * 256);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const lbf16x8 x = weight_column(w, j);
#pragma unroll
      for (int m = 0; m < 4; ++m)
        acc[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            x, __builtin_bit_cast(lbf16x8, h[m]), acc[m][j], 0, 0, 0);
    }
  };
  if (whole > 0) {
    // Steps past the last whole one are fetched as that one, for nothing: without a
    // branch around them the loads' waits stay exact.
    const int end = whole - 1;
    eu32x4 ahead[kAhead][kPieces], h[2][4];
#pragma unroll
    for (int s = 0; s < kAhead; ++s) fetch(s < end ? s : end, ahead[s]);
    hidden_step(0, h[0]);
    put(0, ahead[0]);
    lds_barrier();
    // S: the step's number modulo four, so that registers and buffers are known.
    auto one = [&](int step, auto S) {
      constexpr int s = decltype(S)::value;
      fetch(step + kAhead < end ? step + kAhead : end, ahead[s % kAhead]);
      hidden_step(step + 1 < end ? step + 1 : end, h[(s + 1) & 1]);
      __builtin_amdgcn_sched_barrier(0);
      multiply(s & 1, h[s & 1]);
      __builtin_amdgcn_sched_barrier(0);
      put((s + 1) & 1, ahead[(s + 1) % kAhead]);
      lds_barrier();
    };
    int step = 0;
    for (; step + 4 <= whole; step += 4) {
      one(step, std::integral_constant<int, 0>{});
      one(step + 1, std::integral_constant<int, 1>{});
      one(step + 2, std::integral_constant<int, 2>{});
      one(step + 3, std::integral_constant<int, 3>{});
    }
    if (step < whole) one(step, std::integral_constant<int, 0>{});
    if (step + 1 < whole) one(step + 1, std::integral_constant<int, 1>{});
    if (step + 2 < whole) one(step + 2, std::integral_constant<int, 2>{});
  }
  if (32 * (int64_t)whole < a.H) {
    // What is left of the hidden dimension, in groups of eight.
    const int64_t k = 32 * (int64_t)whole;
    eu32x4 r[kPieces], h[4];
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
      r[p] = eu32x4{0, 0, 0, 0};
      if (k + p * (4 * WM) + (tid >> 4) < a.H)
        r[p] = load_any<eu32x4>(
            reinterpret_cast<const char*>(strip + (k + p * (4 * WM)) * a.V) + poff);
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      h[m] = eu32x4{0, 0, 0, 0};
      if (k + 8 * g < a.H)
        h[m] = *reinterpret_cast<const eu32x4*>(reinterpret_cast<const char*>(a.hidden + k) +
                                                hoff[m]);
    }
    put(0, r);
    lds_barrier();
    multiply(0, h);
  }
  if (idle) return;
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const int64_t t = t0 + 16 * m + c;
    if (t >= a.N) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t col = base + 8 * (4 * g + i);
      if (col + 8 <= v0) continue;
      float z[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) z[j] = acc[m][j][i];
      logits_finish(a, col, 8, z);
      const int skip = v0 > col ? (int)(v0 - col) : 0;
      if (skip == 0) {
        store8<OUT32>(a.out, t * a.ld_out + col, 8, z);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j >= skip) store1<OUT32>(a.out, t * a.ld_out + col + j, z[j]);
      }
    }
  }
}

// The hidden rows as the tile's B operand: strips of 256 tokens (zeros past the last
// one), K blocks of 32. A block fills two consecutive K blocks of one strip with all of
// its loads at once (256 rows of 5120: 9 us; eight K blocks, four loads at once: 20).
constexpr int kPackBlocks = 2;
__global__ void __launch_bounds__(256) logits_pack_kernel(LogitsArgs a) {
  constexpr int kPieces = kPackBlocks * 4;  // 16 bytes of a row
  const int strip = blockIdx.y;
  eu32x4 v[kPieces];
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const int i = p * 256 + threadIdx.x, r = i / kPieces, c = i % kPieces;
    const int64_t row = (int64_t)strip * kTile + r;
    const int64_t k = (int64_t)blockIdx.x * kPackBlocks * kBK + c * 8;
    v[p] = eu32x4{0, 0, 0, 0};
    if (row < a.N && k < a.H) v[p] = *reinterpret_cast<const eu32x4*>(a.hidden + row * a.H + k);
  }
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const int i = p * 256 + threadIdx.x, r = i / kPieces, c = i % kPieces;
    const int kb = blockIdx.x * kPackBlocks + (c >> 2);
    if (kb >= a.hkb) continue;
    char* block = reinterpret_cast<char*>(a.image) +
                  ((int64_t)strip * a.hkb + kb) * (int64_t)kBlockBytes;
    *reinterpret_cast<eu32x4*>(block + blk_byte(r, (c & 3) * 8)) = v[p];
  }
}

// Tokens [256 tb, +256) against vocabulary [256 vt, +256), rows of the tile the
// vocabulary (the weight read row-contiguous, V a multiple of 8) and its columns the
// tokens, as in the head's forward: a lane holds 64 logits of each of two tokens, four
// consecutive ids at a time. 1024 tokens of hidden size 4096 and 128256 ids take 978 us
// (1100 TFLOP/s, bound by the matrix units), 256 of 5120 and 152064 412 us: 594 tiles on
// 256 CUs, 4.7 TB/s of weight in a full round.
template <bool OUT32>
__global__ void __attribute__((amdgpu_flat_work_group_size(kThreads, kThreads),
                               amdgpu_waves_per_eu(2, 2)))
logits_tile_kernel(LogitsArgs a) {
  FLCE_DECLARE_STAGES(sa, sb);
  int tb, vt;
  group_map(xcd_remap(blockIdx.x, a.VT * a.TB), a.TB, a.VT, a.TB, tb, vt);
  const int lane = threadIdx.x & 63;
  const int wave = wave_id(), wm = wave & 1, wn = wave >> 1;
  Acc acc;
  {
    MainloopRowA ml;
    RowA A;
    A.init(a.weight, a.V, a.V, (int64_t)vt * kTile, 0, a.H);
    const Strip B{a.image + (int64_t)tb * a.hkb * kBlockElems, a.hkb};
    ml.run(sa, sb, A, B, 0, a.hkb, acc);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t t = (int64_t)tb * kTile + acc_col(wn, j, lane);
    if (t >= a.N) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t v = (int64_t)vt * kTile + acc_row(wm, i, 4 * q, lane);
        if (v >= a.V) continue;
        float z[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          z[k] = acc[i][j][4 * q + k];
          if (a.bias != nullptr) z[k] += a.bias[v + k];
          if (a.cap > 0.f) z[k] = soft_cap(z[k], a.cap, a.inv_cap);
        }
        const int64_t at = t * a.ld_out + v;
        if constexpr (OUT32)
          store_any(static_cast<float*>(a.out) + at, ef32x4{z[0], z[1], z[2], z[3]});
        else
          store_any(static_cast<uint16_t*>(a.out) + at,
                    u32x2_t{bf16_pair(z[0], z[1]), bf16_pair(z[2], z[3])});
      }
  }
}

}  // namespace flce
