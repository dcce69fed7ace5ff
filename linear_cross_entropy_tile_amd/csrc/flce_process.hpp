// Kernels of the processing of logits before sampling (gfx950): penalties for the
// tokens of a row's history, biases, temperature and mask, with the logsumexp,
// entropy and first largest id of the result, and the gradient.
//
// A row's ids are cut into slices, a block each. The block counts the history's
// tokens that fall into its slice in LDS (integer atomics: the order does not
// matter), adds up the slice's listed biases there in the list's order, and then
// streams the slice once, eight ids a thread and step, keeping per thread the
// running maximum m, s = sum exp(x - m), u = sum exp(x - m) (x - m) and the first
// id of the maximum. The slices' states are merged by a wave a row in a second
// launch. lse = m + ln s, entropy = ln s - u / s.
//
// Contraction of a product and a sum into one rounding is off: the value of a
// logit is the header's sequence of fp32 operations, whatever the compiler picks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "flce_gemm.hpp"
#include "flce_step_plan.hpp"
#include "flce_vector.hpp"

namespace flce {

struct ProcArgs {
  const void* in;
  void* out;
  int64_t ld, ld_out;
  int64_t N, V;
  int64_t row0;       // of the launch
  int slice;
  int64_t slices;
  flce_process_options_t o;
  float4* parts;      // [N, slices]: m, s, u, bits of the first id
  int32_t* invalid;   // [N]
  int32_t* header;
  float* lse;
  float* entropy;
  int64_t* greedy;
  // Backward: the upstream gradients, and the gradient. in: the logits.
  flce_process_grads_t g;
  void* grad;
  int64_t ld_grad;
};

constexpr float kMostNegative = -3.402823466e38f;

// A row's history and listed biases: [begin, end) of its tokens, the first `prompt`
// of which are the prompt.
struct ProcRow {
  int64_t begin, end, generated;
  int64_t bias_begin, bias_end;
  bool bad;
};
__device__ __forceinline__ ProcRow proc_row(const ProcArgs& a, int64_t row) {
  ProcRow r{0, 0, 0, 0, 0, false};
  const flce_process_options_t& o = a.o;
  if (o.tokens != nullptr) {
    if (o.tokens_stride > 0) {
      const int64_t n = o.offsets[row];
      r.bad = n < 0 || n > o.tokens_stride;
      r.begin = row * o.tokens_stride;
      r.end = r.begin + n;
    } else {
      r.begin = o.offsets[row];
      r.end = o.offsets[row + 1];
      r.bad = r.begin < 0 || r.end < r.begin || r.end > o.tokens_size;
    }
    const int64_t p = o.prompt_lengths != nullptr ? o.prompt_lengths[row] : 0;
    r.generated = p <= 0 ? r.begin : (p < r.end - r.begin ? r.begin + p : r.end);
  }
  if (o.bias_offsets != nullptr) {
    r.bias_begin = o.bias_offsets[row];
    r.bias_end = o.bias_offsets[row + 1];
    r.bad = r.bad || r.bias_begin < 0 || r.bias_end < r.bias_begin || r.bias_end > o.bias_count;
  }
  if (r.bad) r.begin = r.end = r.generated = r.bias_begin = r.bias_end = 0;
  return r;
}

// The row's penalties.
struct ProcScale {
  float r, inv_r, presence, frequency, inv_t;
};
__device__ __forceinline__ ProcScale proc_scale(const ProcArgs& a, int64_t row) {
  const flce_process_options_t& o = a.o;
  ProcScale s;
  s.r = o.repetition != nullptr ? o.repetition[row] : (float)o.repetition_penalty;
  s.inv_r = 1.f / s.r;
  s.presence = o.presence != nullptr ? o.presence[row] : (float)o.presence_penalty;
  s.frequency = o.frequency != nullptr ? o.frequency[row] : (float)o.frequency_penalty;
  const float t = o.temperatures != nullptr ? o.temperatures[row] : (float)o.temperature;
  s.inv_t = t == 0.f ? 1.f : 1.f / t;
  return s;
}

// Bits of ids base .. base + 7 (base a multiple of 8) of the row's mask; ids past V
// are not looked at by the caller, and words past the row are not read.
__device__ __forceinline__ uint32_t mask_bits(const ProcArgs& a, int64_t row, int64_t base) {
  if (a.o.allowed == nullptr) return 0xFFu;
  const uint8_t* p = reinterpret_cast<const uint8_t*>(a.o.allowed + row * a.o.allowed_stride);
  return p[base >> 3];
}

constexpr uint32_t kSeenPrompt = 0x80000000u;  // a count's flag: seen in the prompt

// Counts the row's tokens of [lo, lo + n) into count (cleared by the caller);
// COUNT: occurrences among the generated ones and kSeenPrompt, else bits. Returns
// the thread's number of tokens that are no ids of the vocabulary.
template <int HIST>
__device__ __forceinline__ int proc_history_slice(const ProcArgs& a, const ProcRow& r, int64_t lo,
                                                  int n, uint32_t* count) {
  constexpr int U = 8;
  int invalid = 0;
  for (int64_t i0 = r.begin + threadIdx.x; i0 < r.end; i0 += U * kProcThreads) {
    int64_t t[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = i0 + u * kProcThreads;
      t[u] = i < r.end ? a.o.tokens[i] : a.o.ignore_index;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t x = t[u];
      if (x == a.o.ignore_index) continue;
      invalid += x < 0 || x >= a.V ? 1 : 0;
      const int64_t d = x - lo;
      if (d < 0 || d >= n || x >= a.V) continue;
      if constexpr (HIST == HIST_COUNT) {
        if (i0 + u * kProcThreads < r.generated)
          atomicOr(&count[d], kSeenPrompt);
        else
          atomicAdd(&count[d], 1u);
      } else {
        atomicOr(&count[d >> 5], 1u << (d & 31));
      }
    }
  }
  return invalid;
}

// One wave adds the row's listed biases of [lo, lo + n) to sum (cleared by the
// caller) in the list's order: of the lanes that have the same id, the first one
// goes first. `tag` holds one word an id. Returns the lane's number of ids outside
// the vocabulary.
__device__ __forceinline__ int proc_bias_slice(const ProcArgs& a, const ProcRow& r, int64_t lo,
                                               int n, volatile float* sum, uint32_t* tag) {
  const int lane = threadIdx.x & 63;
  int invalid = 0;
  for (int64_t i0 = r.bias_begin; i0 < r.bias_end; i0 += 64) {
    const int64_t i = i0 + lane;
    bool on = i < r.bias_end;
    int64_t d = 0;
    float value = 0.f;
    if (on) {
      const int64_t x = a.o.bias_tokens[i];
      invalid += x != a.o.ignore_index && (x < 0 || x >= a.V) ? 1 : 0;
      d = x - lo;
      on = x != a.o.ignore_index && d >= 0 && d < n && x < a.V;
      if (on) value = a.o.bias_values[i];
    }
    while (__builtin_amdgcn_ballot_w64(on) != 0) {
      if (on) tag[d] = 64u;
      __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
      if (on) atomicMin(&tag[d], (uint32_t)lane);
      __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
      if (on && *(volatile uint32_t*)&tag[d] == (uint32_t)lane) {
        sum[d] = sum[d] + value;
        on = false;
      }
      __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    }
  }
  return invalid;
}

// Softmax state of part of a row; id: of the first largest value, -1 when there is
// none. A NaN makes m NaN and id its place.
struct ProcState {
  float m, s, u;
  int id;
};
__device__ __forceinline__ ProcState proc_merge(const ProcState& a, const ProcState& b) {
  const bool an = a.m != a.m, bn = b.m != b.m;
  if (an || bn) {
    if (an && bn) return a.id < b.id ? a : b;
    return an ? a : b;
  }
  if (b.m == -INFINITY) return a;
  if (a.m == -INFINITY) return b;
  const float m = fmaxf(a.m, b.m);
  const float da = fmaxf(a.m - m, kMostNegative), db = fmaxf(b.m - m, kMostNegative);
  const float fa = a.m == m ? 1.f : __builtin_amdgcn_exp2f(da * kLog2e);
  const float fb = b.m == m ? 1.f : __builtin_amdgcn_exp2f(db * kLog2e);
  ProcState r;
  r.m = m;
  r.s = fa * a.s + fb * b.s;
  // A part that vanishes beside the other has no share, however far down it is.
  r.u = (a.m == m ? a.u : (fa > 0.f ? fa * (a.u + a.s * da) : 0.f)) +
        (b.m == m ? b.u : (fb > 0.f ? fb * (b.u + b.s * db) : 0.f));
  r.id = a.m > b.m ? a.id : (b.m > a.m ? b.id : (a.id < b.id ? a.id : b.id));
  return r;
}
__device__ __forceinline__ ProcState proc_wave_merge(ProcState v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    ProcState w;
    w.m = __shfl_xor(v.m, d, 64);
    w.s = __shfl_xor(v.s, d, 64);
    w.u = __shfl_xor(v.u, d, 64);
    w.id = __shfl_xor(v.id, d, 64);
    // The same operand order in both lanes.
    v = (threadIdx.x & d) == 0 ? proc_merge(v, w) : proc_merge(w, v);
  }
  return v;
}

// Adds eight values (the first `n`) of ids id0 .. to the thread's state, in ids'
// order. NaN: s becomes NaN.
__device__ __forceinline__ void proc_accumulate(ProcState& st, const float (&x)[8], int n, int id0) {
  float top = -INFINITY;
#pragma unroll
  for (int k = 0; k < 8; ++k) top = fmaxf(top, k < n ? x[k] : -INFINITY);
  if (top > st.m) {
    const float d = fmaxf(st.m - top, kMostNegative);
    const float f = __builtin_amdgcn_exp2f(d * kLog2e);
    st.u = f > 0.f ? f * (st.u + st.s * d) : 0.f;
    st.s = f * st.s;
    st.m = top;
#pragma unroll
    for (int k = 7; k >= 0; --k)
      if (k < n && x[k] == top) st.id = id0 + k;
  }
  const float m = st.m == -INFINITY ? 0.f : st.m;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (k < n) {
      const float d = x[k] - m;
      const float e = __builtin_amdgcn_exp2f(d * kLog2e);
      st.s += e;
      st.u += e * fmaxf(d, kMostNegative);
    }
  }
}

// Block (row, slice): see the head of the file. LIST: there are listed biases.
template <int HIST, bool LIST, bool IN32, bool OUT32>
__global__ void __launch_bounds__(kProcThreads) process_kernel(ProcArgs a) {
#pragma clang fp contract(off)
  extern __shared__ uint32_t sh[];
  __shared__ ProcState wave_state[kProcThreads / 64];
  __shared__ int wave_invalid[kProcThreads / 64];
  const int64_t slice = blockIdx.x % (uint32_t)a.slices;
  const int64_t row = a.row0 + blockIdx.x / (uint32_t)a.slices;
  const int64_t lo = slice * a.slice;
  const int n = (int)(a.V - lo < a.slice ? a.V - lo : a.slice);
  const int tid = threadIdx.x;
  const ProcRow r = proc_row(a, row);
  const ProcScale sc = proc_scale(a, row);
  uint32_t* count = sh;
  const int words = HIST == HIST_COUNT ? a.slice : (HIST == HIST_SEEN ? a.slice / 32 : 0);
  float* sum = reinterpret_cast<float*>(sh + words);
  uint32_t* tag = sh + words + a.slice;
  if constexpr (HIST != HIST_NONE || LIST) {
    const int clear = words + (LIST ? a.slice : 0);
    for (int i = tid; i < clear; i += kProcThreads) sh[i] = 0;
    __syncthreads();
    int invalid = 0;
    if constexpr (HIST != HIST_NONE) invalid = proc_history_slice<HIST>(a, r, lo, n, count);
    if constexpr (LIST)
      if (tid < 64) invalid += proc_bias_slice(a, r, lo, n, sum, tag);
    if (slice == 0) {
      for (int d = 32; d > 0; d >>= 1) invalid += __shfl_down(invalid, d, 64);
      if ((tid & 63) == 0) wave_invalid[tid >> 6] = invalid;
    }
    __syncthreads();
  }
  if (slice == 0 && tid == 0) {
    int invalid = r.bad ? 1 : 0;
    if constexpr (HIST != HIST_NONE || LIST)
      for (int w = 0; w < kProcThreads / 64; ++w) invalid += wave_invalid[w];
    a.invalid[row] = invalid;
  }
  ProcState st{-INFINITY, 0.f, 0.f, -1};
  for (int v = tid * 8; v < n; v += kProcStep) {
    const int left = n - v;
    float x[8];
    load8<IN32>(a.in, row * a.ld + lo + v, left, x);
    if constexpr (HIST == HIST_COUNT) {
      uint32_t c[8], any = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        c[k] = count[v + k];
        any |= c[k];
      }
      if (any != 0) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float times = (float)(c[k] & ~kSeenPrompt);
          if (c[k] != 0) x[k] = x[k] * (x[k] > 0.f ? sc.inv_r : sc.r);
          if (times > 0.f) x[k] = (x[k] - sc.frequency * times) - sc.presence;
        }
      }
    } else if constexpr (HIST == HIST_SEEN) {
      const uint32_t bits = (count[v >> 5] >> (v & 31)) & 0xFFu;
      if (bits != 0) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if ((bits >> k) & 1) x[k] = x[k] * (x[k] > 0.f ? sc.inv_r : sc.r);
      }
    }
    if (a.o.bias != nullptr) {
      float b[8];
      load8<true>(a.o.bias, row * a.o.bias_stride + lo + v, left, b);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = x[k] + b[k];
    }
    if constexpr (LIST) {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = x[k] + sum[v + k];
    }
    const uint32_t allowed = mask_bits(a, row, lo + v);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[k] = x[k] * sc.inv_t;
      x[k] = (allowed >> k) & 1 ? x[k] : -INFINITY;
      if (r.bad) x[k] = NAN;
    }
    store8<OUT32>(a.out, row * a.ld_out + lo + v, left, x);
    // The statistics are those of the values as they are returned.
    if constexpr (!OUT32) unpack8(pack8(x), x);
    proc_accumulate(st, x, left, (int)lo + v);
  }
  if (!r.bad && st.s != st.s) {
    // A NaN among this thread's values (or infinity - infinity): find it.
    for (int v = tid * 8; v < n; v += kProcStep) {
      float x[8];
      load8<OUT32>(a.out, row * a.ld_out + lo + v, n - v, x);
      for (int k = 0; k < 8 && v + k < n; ++k)
        if (x[k] != x[k] && st.m == st.m) {
          st.m = NAN;
          st.id = (int)lo + v + k;
        }
    }
  }
  if (r.bad) st = ProcState{NAN, NAN, NAN, -1};
  st = proc_wave_merge(st);
  if ((tid & 63) == 0) wave_state[tid >> 6] = st;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kProcThreads / 64; ++w) st = proc_merge(st, wave_state[w]);
    a.parts[row * a.slices + slice] = make_float4(st.m, st.s, st.u, __int_as_float(st.id));
  }
}

// One block: the header's count of invalid tokens from those of the rows.
__device__ __forceinline__ void proc_status(const ProcArgs& a) {
  __shared__ int sh[4];
  int64_t all = 0;
  for (int64_t i = threadIdx.x; i < a.N; i += 256) all += a.invalid[i];
  int64_t t = all;
  for (int d = 32; d > 0; d >>= 1) t += __shfl_down((long long)t, d, 64);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = t > 0xFFFFFFF ? 0xFFFFFFF : (int)t;
  __syncthreads();
  if (threadIdx.x == 0) {
    a.header[0] = sh[0] + sh[1] + sh[2] + sh[3];
    a.header[1] = 0;
  }
}
__global__ void __launch_bounds__(256) process_status_kernel(ProcArgs a) { proc_status(a); }

// A wave a row merges its slices; one more block adds up the rows' invalid tokens.
__global__ void __launch_bounds__(256) process_rows_kernel(ProcArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (blockIdx.x == gridDim.x - 1) {
    proc_status(a);
    return;
  }
  const int64_t row = (int64_t)blockIdx.x * 4 + wave;
  if (row >= a.N) return;
  ProcState st{-INFINITY, 0.f, 0.f, -1};
  for (int64_t i = lane; i < a.slices; i += 64) {
    const float4 p = a.parts[row * a.slices + i];
    st = proc_merge(st, ProcState{p.x, p.y, p.z, __float_as_int(p.w)});
  }
  st = proc_wave_merge(st);
  if (lane != 0) return;
  float lse, entropy;
  if (st.m != st.m) {
    lse = entropy = NAN;
  } else if (st.m == -INFINITY) {
    lse = -INFINITY;
    entropy = 0.f;
  } else if (st.m == INFINITY) {
    lse = INFINITY;
    entropy = NAN;
  } else {
    const float ln_s = logf(st.s);
    lse = st.m + ln_s;
    entropy = ln_s - st.u / st.s;
  }
  if (a.lse != nullptr) a.lse[row] = lse;
  if (a.entropy != nullptr) a.entropy[row] = entropy;
  if (a.greedy != nullptr) a.greedy[row] = st.id;
}

// Gradient of a slice of a row. STATS: with the gradients of lse and entropy.
template <bool SEEN, bool STATS, bool IN32, bool OUT32>
__global__ void __launch_bounds__(kProcThreads) process_grad_kernel(ProcArgs a) {
#pragma clang fp contract(off)
  extern __shared__ uint32_t sh[];
  __shared__ int wave_invalid[kProcThreads / 64];
  const int64_t slice = blockIdx.x % (uint32_t)a.slices;
  const int64_t row = a.row0 + blockIdx.x / (uint32_t)a.slices;
  const int64_t lo = slice * a.slice;
  const int n = (int)(a.V - lo < a.slice ? a.V - lo : a.slice);
  const int tid = threadIdx.x;
  const ProcRow r = proc_row(a, row);
  const ProcScale sc = proc_scale(a, row);
  float lse = 0.f, entropy = 0.f, g_lse = 0.f, g_entropy = 0.f;
  if constexpr (STATS) {
    lse = a.g.lse[row];
    if (a.g.grad_lse != nullptr) g_lse = a.g.grad_lse[row];
    if (a.g.grad_entropy != nullptr) {
      g_entropy = a.g.grad_entropy[row];
      entropy = a.g.entropy[row];
    }
  }
  int invalid = 0;
  if constexpr (SEEN) {
    for (int i = tid; i < a.slice / 32; i += kProcThreads) sh[i] = 0;
    __syncthreads();
    invalid = proc_history_slice<HIST_SEEN>(a, r, lo, n, sh);
  }
  if (slice == 0) {
    for (int d = 32; d > 0; d >>= 1) invalid += __shfl_down(invalid, d, 64);
    if ((tid & 63) == 0) wave_invalid[tid >> 6] = invalid;
  }
  __syncthreads();
  if (slice == 0 && tid == 0) {
    for (int w = 1; w < kProcThreads / 64; ++w) invalid += wave_invalid[w];
    a.invalid[row] = invalid + (r.bad ? 1 : 0);
  }
  for (int v = tid * 8; v < n; v += kProcStep) {
    const int left = n - v;
    float g[8];
    if (a.g.grad_out != nullptr) {
      load8<OUT32>(a.g.grad_out, row * a.g.ld_grad_out + lo + v, left, g);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) g[k] = 0.f;
    }
    if constexpr (STATS) {
      float y[8];
      load8<OUT32>(a.g.out, row * a.g.ld_out + lo + v, left, y);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float d = y[k] - lse;
        const float p = __builtin_amdgcn_exp2f(d * kLog2e);
        // Nothing is allowed: lse is -inf and so is y.
        const float more = p * (g_lse - g_entropy * (d + entropy));
        if (lse != -INFINITY && p != 0.f) g[k] = g[k] + more;
      }
    }
    if constexpr (SEEN) {
      const uint32_t bits = (sh[v >> 5] >> (v & 31)) & 0xFFu;
      if (bits != 0) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (((bits >> k) & 1) && k < left) {
            const int64_t i = row * a.ld + lo + v + k;
            float x;
            if constexpr (IN32)
              x = static_cast<const float*>(a.in)[i];
            else
              x = bf16_lo(static_cast<const uint16_t*>(a.in)[i]);
            g[k] = g[k] * (x > 0.f ? sc.inv_r : sc.r);
          }
      }
    }
    const uint32_t allowed = mask_bits(a, row, lo + v);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      g[k] = g[k] * sc.inv_t;
      g[k] = (allowed >> k) & 1 ? g[k] : 0.f;
      if (r.bad) g[k] = NAN;
    }
    store8<IN32>(a.grad, row * a.ld_grad + lo + v, left, g);
  }
}

}  // namespace flce
