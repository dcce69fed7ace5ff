// Kernels of the processing of logits before sampling (gfx950): penalties for the
// tokens of a row's history, biases, temperature and mask, with the logsumexp,
// entropy and first largest id of the result, and the gradient.
//
// A row's ids are cut into slices, a block each, of which a thread holds eight
// consecutive ids a step in registers. The logits are asked for first; while they
// come, the block counts the history's tokens that fall into its slice in LDS
// (integer atomics: the order does not matter) and then, once the penalties have been
// applied, adds up the slice's listed biases there in the list's order. The values are
// formed and stored, and from the block's maximum m come s = sum exp(x - m) and
// u = sum exp(x - m) (x - m). The slices' states are merged by a wave a row in a second
// launch. lse = m + ln s, entropy = ln s - u / s.
//
// 512 rows of 152064 bf16 logits take 57 us without a history (5.4 TB/s, bound by the
// bytes) and 89 to 96 with up to 2048 tokens a row and a mask: then a block's chain of
// offsets, tokens, counts and statistics shows, at eight blocks a CU. Sorting the
// histories by slice in a launch before saves 5 us and costs 9. 64 rows of 128256 fp32
// logits, up to 4096 tokens and 100 listed biases a row, take 24 us and 5 to 8 of the
// merge. The gradient of 300 rows of 50257 fp32 takes 36 us (4.9 TB/s with the logits that
// it reads of seen ids), and with the gradients of lse and entropy, for which it reads the
// returned logits too, 45 us; of 512 rows of 152064 bf16 without a history 59 and 91 us
// (5.2 TB/s), with 1000 tokens a row 99 and 121 us.
//
// Contraction of a product and a sum into one rounding is off: the value of a
// logit is the header's sequence of fp32 operations, whatever the compiler picks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "flce_gemm.hpp"
#include "flce_logits.hpp"
#include "flce_step_plan.hpp"
#include "flce_vector.hpp"

namespace flce {

struct ProcArgs {
  const void* in;
  void* out;
  int64_t ld, ld_out;
  int64_t N, V;
  int64_t row0;       // of the launch
  int slice;          // of the gradient; a multiple of kProcStep
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
      r.bad = n < 0 || n > o.tokens_stride || n > kMostHistory;
      r.begin = row * o.tokens_stride;
      r.end = r.begin + n;
    } else {
      r.begin = o.offsets[row];
      r.end = o.offsets[row + 1];
      r.bad = r.begin < 0 || r.end < r.begin || r.end > o.tokens_size ||
              r.end - r.begin > kMostHistory;
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

// Counts of generated tokens in 16 bits, two ids a word, with a flag for those seen in
// the prompt; rows of more than kLongHistory tokens take 32 bits.
constexpr uint32_t kSeenPrompt = 0x8000u, kSeenPromptWide = 0x80000000u;

// Counts the row's tokens of [lo, lo + n) into count (cleared by the caller): under
// HIST_SEEN bits, under HIST_COUNT occurrences among the generated ones and the flag, a
// word an id if WIDE. Returns the thread's number of tokens that are no ids of the
// vocabulary.
template <int HIST, bool WIDE>
__device__ __forceinline__ int proc_history_slice(const ProcArgs& a, const ProcRow& r, int64_t lo,
                                                  uint32_t n, uint32_t* count) {
  constexpr int U = 4;
  // Only a row's first slice counts what is no id, and the id to pass over is mostly
  // none of the slice's: elsewhere a token costs a subtraction and a comparison.
  const bool all = lo == 0;
  const uint64_t skip = proc_place(a.o.ignore_index, lo);
  int invalid = 0;
  for (int64_t i0 = r.begin + threadIdx.x; i0 < r.end; i0 += U * kProcThreads) {
    int64_t t[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = i0 + u * kProcThreads;
      t[u] = i < r.end ? a.o.tokens[i] : a.o.ignore_index;
    }
    if (all) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        invalid += t[u] != a.o.ignore_index && (uint64_t)t[u] >= (uint64_t)a.V ? 1 : 0;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint64_t x = proc_place(t[u], lo);
      if (x >= n || x == skip) continue;
      const int d = (int)x;
      if constexpr (HIST == HIST_COUNT) {
        const bool made = i0 + u * kProcThreads >= r.generated;
        const int shift = WIDE ? 0 : 16 * (d & 1);
        uint32_t* word = &count[WIDE ? d : d >> 1];
        if (made)
          atomicAdd(word, 1u << shift);
        else
          atomicOr(word, (WIDE ? kSeenPromptWide : kSeenPrompt) << shift);
      } else {
        atomicOr(&count[d >> 5], 1u << (d & 31));
      }
    }
  }
  return invalid;
}

// Listed bias i of the row for a lane, as far as there is one.
struct ProcListed {
  int64_t id;
  float value;
};
__device__ __forceinline__ ProcListed proc_listed(const ProcArgs& a, const ProcRow& r, int64_t i) {
  ProcListed p{a.o.ignore_index, 0.f};
  if (i < r.bias_end) {
    p.id = a.o.bias_tokens[i];
    p.value = a.o.bias_values[i];
  }
  return p;
}

// One wave adds the row's listed biases of [lo, lo + n) to sum (cleared by the
// caller) in the list's order: of the lanes that have the same id, the first one
// goes first. `tag` holds kProcTags words; ids that share one wait for each other.
// next: the lane's first one, which has been asked for before. Returns the lane's
// number of ids outside the vocabulary.
__device__ __forceinline__ int proc_bias_slice(const ProcArgs& a, const ProcRow& r, int64_t lo,
                                               uint32_t n, ProcListed next, volatile float* sum,
                                               uint32_t* tag) {
  const int lane = threadIdx.x & 63;
  int invalid = 0;
  for (int64_t i0 = r.bias_begin; i0 < r.bias_end; i0 += 64) {
    const ProcListed p = next;
    next = proc_listed(a, r, i0 + 64 + lane);
    invalid += p.id != a.o.ignore_index && (p.id < 0 || p.id >= a.V) ? 1 : 0;
    const uint64_t d = proc_place(p.id, lo);
    bool on = p.id != a.o.ignore_index && d < n;
    while (__builtin_amdgcn_ballot_w64(on) != 0) {
      uint32_t* slot = &tag[d & (kProcTags - 1)];
      if (on) *slot = 64u;
      __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
      if (on) atomicMin(slot, (uint32_t)lane);
      __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
      if (on && *(volatile uint32_t*)slot == (uint32_t)lane) {
        sum[d] = sum[d] + p.value;
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

// A wave's result of `op` over its lanes, in all of them, in a fixed order: within the
// rows of 16 lanes, then over the four rows.
template <int CTRL>
__device__ __forceinline__ float dpp_rotated(float v) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}
template <class Op>
__device__ __forceinline__ float wave_all(float v, Op op) {
  v = op(v, dpp_rotated<0x128>(v));  // row_ror:8
  v = op(v, dpp_rotated<0x124>(v));
  v = op(v, dpp_rotated<0x122>(v));
  v = op(v, dpp_rotated<0x121>(v));
  float r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = __builtin_bit_cast(
        float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 16 * i));
  return op(op(r[0], r[1]), op(r[2], r[3]));
}
struct MaxOp {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct SumOp {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};

// Eight values as they lie in memory.
template <bool F32>
struct Raw8 {
  eu32x4 w[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ void load_raw8(const void* p, int64_t i, int n, Raw8<F32>& r) {
  if (n >= 8) {
    const char* q = static_cast<const char*>(p) + i * (F32 ? 4 : 2);
    r.w[0] = load_any<eu32x4>(q);
    if constexpr (F32) r.w[1] = load_any<eu32x4>(q + 16);
    return;
  }
  float v[8];
  load8<F32>(p, i, n, v);
  if constexpr (F32) {
#pragma unroll
    for (int k = 0; k < 8; ++k) r.w[k >> 2][k & 3] = __builtin_bit_cast(uint32_t, v[k]);
  } else {
    r.w[0] = pack8(v);
  }
}
template <bool F32>
__device__ __forceinline__ void unpack_raw8(const Raw8<F32>& r, float (&v)[8]) {
  if constexpr (F32) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t word = r.w[k >> 2][k & 3];  // a bit cast of a vector's element takes its first
      v[k] = __builtin_bit_cast(float, word);
    }
  } else {
    unpack8(r.w[0], v);
  }
}

// x where bit k of `bits` is set, else `other`.
__device__ __forceinline__ float select_bit(uint32_t bits, int k, float x, float other) {
  const uint32_t m = (uint32_t)((int)(bits << (31 - k)) >> 31);
  return __builtin_bit_cast(float, (m & __builtin_bit_cast(uint32_t, x)) |
                                       (~m & __builtin_bit_cast(uint32_t, other)));
}

// The penalties of the eight ids from v on of the slice.
template <int HIST, bool WIDE>
__device__ __forceinline__ void proc_penalise(const uint32_t* count, int v, const ProcScale& sc,
                                              float (&x)[8]) {
#pragma clang fp contract(off)
  if constexpr (HIST == HIST_SEEN) {
    const uint32_t bits = (count[v >> 5] >> (v & 31)) & 0xFFu;
    if (bits != 0) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if ((bits >> k) & 1) x[k] = x[k] * (x[k] > 0.f ? sc.inv_r : sc.r);
    }
  } else if constexpr (HIST == HIST_COUNT) {
    uint32_t c[8], any = 0;
    if constexpr (WIDE) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        c[k] = count[v + k];
        any |= c[k];
      }
    } else {
      const eu32x4 w = *reinterpret_cast<const eu32x4*>(count + (v >> 1));
      any = w[0] | w[1] | w[2] | w[3];
#pragma unroll
      for (int k = 0; k < 8; ++k) c[k] = (w[k >> 1] >> (16 * (k & 1))) & 0xFFFFu;
    }
    if (any == 0) return;
    const uint32_t flag = WIDE ? kSeenPromptWide : kSeenPrompt;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float times = (float)(c[k] & ~flag);
      if (c[k] != 0) x[k] = x[k] * (x[k] > 0.f ? sc.inv_r : sc.r);
      if (times > 0.f) x[k] = (x[k] - sc.frequency * times) - sc.presence;
    }
  }
}

__device__ __forceinline__ void lds_clear(uint32_t* p, int words) {  // a multiple of 4
  for (int i = threadIdx.x * 4; i < words; i += 4 * kProcThreads)
    *reinterpret_cast<eu32x4*>(p + i) = eu32x4{0, 0, 0, 0};
}

// Block (row, slice): see the head of the file. LIST: there are listed biases. A slice
// has STEPS steps of eight ids a thread.
template <int HIST, bool LIST, int STEPS, bool IN32, bool OUT32>
__global__ void __launch_bounds__(kProcThreads) process_kernel(ProcArgs a) {
#pragma clang fp contract(off)
  constexpr int kSlice = STEPS * kProcStep, kWaves = kProcThreads / 64;
  __shared__ __attribute__((aligned(16))) uint32_t sh[proc_lds_words(HIST, LIST, kSlice) + 4];
  __shared__ float wave_max[kWaves], wave_s[kWaves], wave_u[kWaves];
  __shared__ int wave_invalid[kWaves], first_id, first_nan;
  const int64_t slice = blockIdx.x % (uint32_t)a.slices;
  const int64_t row = a.row0 + blockIdx.x / (uint32_t)a.slices;
  const int64_t lo = slice * kSlice;
  const int n = (int)(a.V - lo < kSlice ? a.V - lo : kSlice);
  const int tid = threadIdx.x;
  Raw8<IN32> raw[STEPS];
  uint32_t allowed[STEPS];
#pragma unroll
  for (int j = 0; j < STEPS; ++j) {
    const int v = j * kProcStep + tid * 8;
    if (v < n) {
      load_raw8<IN32>(a.in, row * a.ld + lo + v, n - v, raw[j]);
      allowed[j] = mask_bits(a, row, lo + v);
    }
  }
  const ProcRow r = proc_row(a, row);
  const ProcScale sc = proc_scale(a, row);
  uint32_t* count = sh;
  float* sum = reinterpret_cast<float*>(sh);
  const bool wide = HIST == HIST_COUNT && r.end - r.begin > kLongHistory;
  if (tid == 0) {
    first_id = 0x7FFFFFFF;
    first_nan = 0x7FFFFFFF;
  }
  int invalid = 0;
  ProcListed listed{0, 0.f};
  if constexpr (LIST)
    if (tid < 64) listed = proc_listed(a, r, r.bias_begin + tid);
  if constexpr (HIST != HIST_NONE) {
    lds_clear(sh, proc_count_words(HIST, kSlice));
    lds_barrier();
    if (!wide) invalid = proc_history_slice<HIST, false>(a, r, lo, n, count);
  }
  lds_barrier();
  float x[STEPS][8];
#pragma unroll
  for (int j = 0; j < STEPS; ++j) {
    const int v = j * kProcStep + tid * 8;
    if (v < n) {
      unpack_raw8<IN32>(raw[j], x[j]);
      if (!wide) proc_penalise<HIST, false>(count, v, sc, x[j]);
    }
  }
  if constexpr (HIST == HIST_COUNT) {
    // Half the slice at a time has room for counts of 32 bits. A row's last slice may end
    // within the first half: there is nothing to count in the second one then. (The break
    // stands behind the clearing since a loop of one or two halves costs every row four
    // registers more, and 512 rows of 152064 bf16 logits 96 us instead of 89.)
    for (int half = 0; wide && half < 2; ++half) {
      lds_barrier();
      lds_clear(count, kSlice / 2);
      lds_barrier();
      const int from = half * (kSlice / 2);
      const uint32_t ids = proc_part(n, from, kSlice / 2);
      if (ids == 0) break;
      const int found = proc_history_slice<HIST, true>(a, r, lo + from, ids, count);
      if (half == 0) invalid += found;
      lds_barrier();
#pragma unroll
      for (int j = 0; j < STEPS; ++j) {
        const int v = j * kProcStep + tid * 8 - from;
        if (v >= 0 && v < (int)ids) proc_penalise<HIST, true>(count, v, sc, x[j]);
      }
    }
  }
  if constexpr (LIST) {
    // The counts have been read: their LDS and more holds the sums, so that eight blocks
    // fit a CU and not six (64 rows of 128256 fp32 logits with up to 100 biases 29.5 -> 27.7
    // us, 256 rows of bf16 ones with 300 64 -> 56).
    if constexpr (HIST != HIST_NONE) lds_barrier();
    lds_clear(sh, kSlice);
    lds_barrier();
    if (tid < 64) invalid += proc_bias_slice(a, r, lo, n, listed, sum, sh + kSlice);
    lds_barrier();
  }
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < STEPS; ++j) {
    const int v = j * kProcStep + tid * 8, left = n - v;
    if (left > 0) {
      if (a.o.bias != nullptr) {
        float b[8];
        load8<true>(a.o.bias, row * a.o.bias_stride + lo + v, left, b);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[j][k] = x[j][k] + b[k];
      }
      if constexpr (LIST) {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[j][k] = x[j][k] + sum[v + k];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k)
        x[j][k] = select_bit(allowed[j], k, x[j][k] * sc.inv_t, -INFINITY);
      if (r.bad) {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[j][k] = NAN;
      }
      // Slices of two steps, which are batches of 1024 blocks or more, are streamed past the
      // caches. The call alone: 512 rows of 152064 bf16 logits with histories 91 us against
      // 102 through the caches, 64 rows of 128256 fp32 ones 28.3 against 29.3. A pass over
      // the result right behind it then finds nothing in the last cache; call and sum over
      // the rows take 131 and 133 us of the former, but 61 and 50 of the latter.
      store8<OUT32, (STEPS > 1)>(a.out, row * a.ld_out + lo + v, left, x[j]);
      // The statistics are those of the values as they are returned.
      if constexpr (!OUT32) unpack8(pack8(x[j]), x[j]);
      if (left < 8) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k >= left) x[j][k] = -INFINITY;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[j][k] = -INFINITY;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) top = fmaxf(top, x[j][k]);
  }
  const float wmax = wave_all(top, MaxOp{});
  if constexpr (HIST != HIST_NONE || LIST) {
    if (slice == 0)
      for (int d = 32; d > 0; d >>= 1) invalid += __shfl_down(invalid, d, 64);
  }
  if ((tid & 63) == 0) {
    wave_max[tid >> 6] = wmax;
    wave_invalid[tid >> 6] = invalid;
  }
  lds_barrier();
  float m = wave_max[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) m = fmaxf(m, wave_max[w]);
  // Nothing is allowed: every term is exp(-inf).
  const float base = m == -INFINITY ? 0.f : m;
  float s = 0.f, u = 0.f;
#pragma unroll
  for (int j = 0; j < STEPS; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float d = x[j][k] - base;
      const float e = __builtin_amdgcn_exp2f(d * kLog2e);
      s = s + e;
      u = __builtin_fmaf(e, fmaxf(d, kMostNegative), u);
    }
  if (top == m && m != -INFINITY) {
    int id = 0x7FFFFFFF;
#pragma unroll
    for (int j = STEPS - 1; j >= 0; --j)
#pragma unroll
      for (int k = 7; k >= 0; --k)
        if (x[j][k] == m) id = (int)lo + j * kProcStep + tid * 8 + k;
    atomicMin(&first_id, id);
  }
  if (s != s) {
    // A NaN among the thread's values, or infinity - infinity.
#pragma unroll
    for (int j = STEPS - 1; j >= 0; --j)
#pragma unroll
      for (int k = 7; k >= 0; --k)
        if (x[j][k] != x[j][k]) atomicMin(&first_nan, (int)lo + j * kProcStep + tid * 8 + k);
  }
  s = wave_all(s, SumOp{});
  u = wave_all(u, SumOp{});
  if ((tid & 63) == 0) {
    wave_s[tid >> 6] = s;
    wave_u[tid >> 6] = u;
  }
  lds_barrier();
  if (tid == 0) {
#pragma unroll
    for (int w = 1; w < kWaves; ++w) {
      s += wave_s[w];
      u += wave_u[w];
      invalid += wave_invalid[w];
    }
    int id = m == -INFINITY ? -1 : first_id;
    if (first_nan != 0x7FFFFFFF) {
      m = NAN;
      id = r.bad ? -1 : first_nan;
    }
    a.parts[row * a.slices + slice] = make_float4(m, s, u, __int_as_float(id));
    if (slice == 0) a.invalid[row] = invalid + (r.bad ? 1 : 0);
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
    invalid = proc_history_slice<HIST_SEEN, false>(a, r, lo, n, sh);
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
