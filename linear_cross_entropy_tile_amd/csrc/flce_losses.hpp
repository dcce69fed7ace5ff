// Kernels of the losses on the head's per-token outputs (gfx950): the clipped
// policy loss with a KL term and the paired preference loss.
//
// Both are sums over ragged sequences of a packed batch, then a small formula a
// sequence (or pair), then one gradient value a token:
//   parts      every 64-lane wave takes a tile of consecutive tokens, forms
//              the per-token terms and sums them over each sequence's share of
//              the tile. The share of sequence s in tile t goes to parts[s + t]:
//              walking the batch, either s or t grows by one from a share to the
//              next, so s + t names it uniquely and B + T slots hold them all,
//              however the lengths are mixed.
//   sequences  adds the shares of each sequence, forms its ratio / its pair's
//              loss and gradient coefficient, and adds up the batch.
//   gradients  one pass over the tokens with the coefficients.
// Tiles and trees depend on the sizes alone and no atomics are used, so equal
// inputs give equal bits. Terms and sums are float64: a difference of two
// log-probabilities is exact there, a ratio next to a clip bound falls on the
// side the definition gives (bounds are compared as logarithms), exp(-x) + x - 1
// keeps its digits at small x, and sums over 2^21 tokens lose nothing. Each
// output is rounded once, to fp32.
//
// What bounds them: below some 10^5 tokens the launches and each kernel's chain of
// dependent loads (hence one launch for everything in small batches, three
// otherwise); at 2^21 tokens the bytes, read twice because the batch's divisor is
// not known before the last token, and the float64 exponentials. Measured on an
// MI355X, policy loss with k3 KL, entropy and gradients: 413 tokens 8.1 us, 32768
// tokens 14.4 us, 2.07 M tokens 50 us (75 MB of distinct inputs and outputs); pairs
// without a reference, 2.07 M tokens, 24 us (33 MB).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "flce_ops_plan.hpp"

namespace flce {

// ---- sequences ------------------------------------------------------------------

// Number of entries <= x among the n entries of the sorted array a, found by a
// whole wave: 64 probes a step. For an array that is not sorted the result is
// meaningless but lies in [0, n], and the loop ends (m shrinks every step).
__device__ __forceinline__ int64_t wave_count_le(const int64_t* a, int64_t n, int64_t x) {
  const int lane = threadIdx.x & 63;
  int64_t lo = 0, m = n;
  while (m > 0) {
    const int64_t step = (m + 63) >> 6;
    const int64_t p = lane * step + step - 1;
    const bool le = p < m && a[lo + p] <= x;
    const int64_t c = __popcll(__builtin_amdgcn_ballot_w64(le));
    lo += c * step;
    m = m - c * step < step - 1 ? m - c * step : step - 1;
  }
  return lo;
}

// The sequences that a tile of tokens [t0, t1) can belong to: ns of them from s0
// (none when all the tokens lie before the first or behind the last sequence).
// Lane k has off, where sequence s0 + k begins, counted from t0 and clamped to
// [0, kLossTile]; lane ns has the last one's end. Tiles of up to kOffSeqs sequences
// need no other load of the offsets.
constexpr int kOffSeqs = 62;
struct TileSeqs {
  int64_t s0, ns;
  int off;
};
__device__ __forceinline__ TileSeqs tile_sequences(const int64_t* cu, int64_t B, int64_t N,
                                                   int64_t t0, int64_t t1) {
  const int lane = threadIdx.x & 63;
  if (cu == nullptr) return {0, 1, lane == 0 ? 0 : kLossTile};
  // Lengths of one batch are of one order, so the tile's offsets are nearly always
  // among the 64 around its share of the batch: one load. Otherwise a search.
  const int64_t n = B + 1;
  const int64_t guess = (int64_t)((float)t0 / (float)N * (float)B) - 31;
  const int64_t w0 = guess < 0 || n <= 64 ? 0 : (guess < n - 64 ? guess : n - 64);
  int64_t s0, c1, v = cu[w0 + lane < n ? w0 + lane : n - 1];
  const uint64_t in = __builtin_amdgcn_ballot_w64(w0 + lane < n);
  const uint64_t m0 = __builtin_amdgcn_ballot_w64(v <= t0) & in;
  const uint64_t m1 = __builtin_amdgcn_ballot_w64(v <= t1 - 1) & in;
  if ((w0 == 0 || (m0 & 1) != 0) && (w0 + 64 >= n || (m1 >> 63) == 0)) {
    const int c0 = __popcll(m0);
    c1 = w0 + __popcll(m1);
    const int from = c0 > 0 ? c0 - 1 : 0;
    s0 = w0 + from;
    const int last = n - w0 < 64 ? (int)(n - w0) - 1 : 63;
    v = (int64_t)__shfl((long long)v, from + lane < last ? from + lane : last, 64);
  } else {
    const int64_t c0 = wave_count_le(cu, n, t0);
    s0 = c0 > 0 ? c0 - 1 : 0;
    v = cu[s0 + lane < n ? s0 + lane : n - 1];
    const int c = __popcll(__builtin_amdgcn_ballot_w64(s0 + lane < n && v <= t1 - 1));
    c1 = c < 64 ? s0 + c : wave_count_le(cu, n, t1 - 1);
  }
  const int64_t s1 = c1 - 1 < B - 1 ? c1 - 1 : B - 1;
  const int64_t d = v < t0 ? 0 : (v < t1 ? v - t0 : kLossTile);
  return {s0, s1 - s0 + 1, (int)d};
}

// Rank (sequence - s0) of the tile's token tl, or -1 when it lies in none. All
// lanes of the wave take part.
__device__ __forceinline__ int token_rank(const int64_t* cu, const TileSeqs& r, int64_t t0,
                                          int tl) {
  if (r.ns <= 0) return -1;
  int lo = 0;
  bool in;
  if (r.ns <= kOffSeqs) {
    const int ns = (int)r.ns;
    for (int k = 1; k < ns; ++k) lo += __builtin_amdgcn_readlane(r.off, k) <= tl ? 1 : 0;
    in = __builtin_amdgcn_readlane(r.off, 0) <= tl && tl < __builtin_amdgcn_readlane(r.off, ns);
  } else {
    const int64_t* c = cu + r.s0;
    int hi = (int)r.ns - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (c[mid] <= t0 + tl)
        lo = mid;
      else
        hi = mid - 1;
    }
    in = c[lo] <= t0 + tl && t0 + tl < c[lo + 1];
  }
  return in ? lo : -1;
}

// Whether the tile's token tl, of rank k >= 0, is the last of its sequence.
__device__ __forceinline__ bool ends_sequence(const int64_t* cu, const TileSeqs& r, int64_t t0,
                                              int tl, int k) {
  if (r.ns <= kOffSeqs) return __shfl(r.off, k + 1, 64) == tl + 1;
  return cu[r.s0 + k + 1] == t0 + tl + 1;
}

__device__ __forceinline__ int64_t seq_begin(const int64_t* cu, int64_t s) {
  return cu == nullptr ? 0 : cu[s];
}
__device__ __forceinline__ int64_t seq_end(const int64_t* cu, int64_t s, int64_t N) {
  return cu == nullptr ? N : cu[s + 1];
}

__device__ __forceinline__ bool label_valid(int64_t y, int64_t ignore_index, int64_t V) {
  return y != ignore_index && y >= 0 && y < V;
}

// ---- wave and block sums --------------------------------------------------------

// The counts of one tile's tokens in one word (at most kLossTile = 256 each).
constexpr int kCountValid = 1, kCountClipped = 1 << 10, kCountInvalid = 1 << 20;

// Sums over the wave in lane 63: within rows of 16 lanes by shifts of 1, 2, 4 and
// 8, then row 0 into 1 and 2 into 3, then 1 into 3.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_or_0(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_or_0(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)dpp_or_0<CTRL, ROWS>((int)(uint32_t)u);
  const uint32_t hi = (uint32_t)dpp_or_0<CTRL, ROWS>((int)(uint32_t)(u >> 32));
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
template <class T>
__device__ __forceinline__ T wave_sum_dpp(T v) {
  v += dpp_or_0<0x111, 0xf>(v);  // row_shr:1
  v += dpp_or_0<0x112, 0xf>(v);  // row_shr:2
  v += dpp_or_0<0x114, 0xf>(v);  // row_shr:4
  v += dpp_or_0<0x118, 0xf>(v);  // row_shr:8
  v += dpp_or_0<0x142, 0xa>(v);  // row_bcast:15 into rows 1 and 3
  v += dpp_or_0<0x143, 0xc>(v);  // row_bcast:31 into rows 2 and 3
  return v;
}

// What a share of a sequence, a sequence, and the batch sum up to: the loss's
// own terms x[]; n valid tokens; c clipped tokens (of the batch: sequences with
// a valid token); inv labels outside [0, V); bad offsets.
template <int K>
struct LossSum {
  double x[K];
  int n, c, inv, bad;
  __device__ void clear() {
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] = 0.0;
    n = c = inv = bad = 0;
  }
  __device__ void add(const LossSum& o) {
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] += o.x[k];
    n += o.n;
    c += o.c;
    inv += o.inv;
    bad += o.bad;
  }
  // Sum over the wave, in lane 63.
  __device__ void wave_sum() {
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] = wave_sum_dpp(x[k]);
    n = wave_sum_dpp(n);
    c = wave_sum_dpp(c);
    inv = wave_sum_dpp(inv);
    bad = wave_sum_dpp(bad);
  }
  // Sum over each group of g lanes (a power of two), in its first lane.
  __device__ void group_sum(int g) {
#pragma unroll 1
    for (int d = g >> 1; d > 0; d >>= 1) {
#pragma unroll
      for (int k = 0; k < K; ++k) x[k] += __shfl_down(x[k], d, 64);
      n += __shfl_down(n, d, 64);
      c += __shfl_down(c, d, 64);
      inv += __shfl_down(inv, d, 64);
      bad += __shfl_down(bad, d, 64);
    }
  }
};

// The terms of a token, or of several of one tile.
template <int K>
struct Terms {
  double x[K];
  int counts;
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] = 0.0;
    counts = 0;
  }
  __device__ __forceinline__ void add(const Terms& o) {
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] += o.x[k];
    counts += o.counts;
  }
  __device__ __forceinline__ Terms up(int d) const {
    Terms o;
#pragma unroll
    for (int k = 0; k < K; ++k) o.x[k] = __shfl_up(x[k], d, 64);
    o.counts = __shfl_up(counts, d, 64);
    return o;
  }
  __device__ __forceinline__ Terms from(int l) const {
    Terms o;
#pragma unroll
    for (int k = 0; k < K; ++k) o.x[k] = __shfl(x[k], l, 64);
    o.counts = __shfl(counts, l, 64);
    return o;
  }
  // Sum over the wave, in lane 63.
  __device__ __forceinline__ void wave_sum() {
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] = wave_sum_dpp(x[k]);
    counts = wave_sum_dpp(counts);
  }
  __device__ __forceinline__ LossSum<K> share() const {
    LossSum<K> s;
#pragma unroll
    for (int k = 0; k < K; ++k) s.x[k] = x[k];
    s.n = counts & 1023;
    s.c = (counts >> 10) & 1023;
    s.inv = counts >> 20;
    s.bad = 0;
    return s;
  }
};

// Sum of the first `used` waves over the block, waves in order, in thread 0. sh:
// one entry a wave.
template <class S>
__device__ __forceinline__ S block_total(S v, int used, S* sh) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  if (w < used) {
    v.wave_sum();
    if (lane == 63) sh[w] = v;
  }
  __syncthreads();
  S r;
  r.clear();
  if (threadIdx.x == 0)
    for (int k = 0; k < used; ++k) r.add(sh[k]);
  __syncthreads();
  return r;
}

// Everything the kernels of one call share; Loss is PolicyLoss or PreferenceLoss.
template <class Loss>
struct LossArgs {
  typename Loss::In in;
  typename Loss::Out out;
  const int64_t* labels;
  const int64_t* cu;            // [B+1], or null: one sequence of all tokens
  int64_t N, B, V, ignore_index;
  int64_t items;                // sequences, or pairs
  int64_t tiles;
  int rows;                     // of 64 tokens a tile: 1 or kLossRows
  int deferred;                 // blocks whose totals the gradients kernel adds up; 0: the
                                // batch is finished before it
  typename Loss::Share* parts;    // [B + tiles]
  typename Loss::Share* seq_sum;  // [B]
  typename Loss::Total* totals;   // [blocks of the sequences kernel]
  int32_t* header;                // [0] invalid labels and offsets, [2] blocks that are done
  double* state;                  // see Loss
};

// exp(x) - 1, or exp(x): x = n ln 2 + f with |f| <= ln 2 / 2, Taylor's series of
// exp(f) - 1 to f^11 (the rest is below 10^-13 of it; the rounding of ln 2 adds
// at most 10^-16 |x|), and 2^n. Near 0 n is 0 and the difference with 1 is never
// formed. That is far below the fp32 rounding of every output; the library's
// functions, exact to the last bit, took 3 us more of the 26 of a parts step over
// 2^21 tokens.
template <bool MINUS_1>
__device__ __forceinline__ double exp_f64(double x) {
  x = x > 1000.0 ? 1000.0 : x;  // keeps NaN
  x = x < -1000.0 ? -1000.0 : x;
  const double n = __builtin_rint(x * 1.4426950408889634);
  const double f = fma(n, -0.6931471805599453, x);
  double p = 1.0 / 39916800.0;
  p = fma(p, f, 1.0 / 3628800.0);
  p = fma(p, f, 1.0 / 362880.0);
  p = fma(p, f, 1.0 / 40320.0);
  p = fma(p, f, 1.0 / 5040.0);
  p = fma(p, f, 1.0 / 720.0);
  p = fma(p, f, 1.0 / 120.0);
  p = fma(p, f, 1.0 / 24.0);
  p = fma(p, f, 1.0 / 6.0);
  p = fma(p, f, 0.5);
  p = fma(p * f, f, f);
  const double e = ldexp(1.0 + p, (int)n);
  if (!MINUS_1) return e;
  return n == 0.0 ? p : e - 1.0;
}

// ---- the clipped policy loss --------------------------------------------------------

struct PolicyLoss {
  struct In {
    const float *logprob, *old_logprob, *ref_logprob, *entropy, *advantages;
    double over, under, dual;              // ratio bounds 1 + clip_high, 1 - clip_low, dual_clip
    double log_over, log_under, log_dual;  // their logarithms (+-infinity where off)
    double kl_coef, ent_coef;
    int kl, by_sequence, adv_seq, reduction;
  };
  struct Out {
    float* loss;             // [1] or null
    float* stats;            // [8]
    const float* grad_loss;  // [1] or null
    float* grad_logprob;
    float* grad_entropy;     // or null
  };
  static __host__ __device__ constexpr int state_size(int B) { return 2 * (B + 1); }
  static constexpr bool kGradReads = true;  // the gradient needs the per-token inputs
  // state[2 s]: token weight of sequence s before the batch's factor;
  // state[2 s + 1]: derivative of the policy term by the mean of d (sequence
  // level); state[2 B]: the batch's factor.
  using Share = LossSum<4>;  // d, policy, kl, entropy
  using Token = Terms<4>;
  using Total = LossSum<5>;  // weighted: d, policy, kl, entropy, clipped
  static constexpr int kSides = 1;

  struct Raw {
    float lp, old, ref, ent;
  };
  __device__ static Raw load(const LossArgs<PolicyLoss>& a, int64_t t) {
    const In& in = a.in;
    return {in.logprob[t], in.old_logprob[t], in.ref_logprob != nullptr ? in.ref_logprob[t] : 0.f,
            in.entropy != nullptr ? in.entropy[t] : 0.f};
  }
  // Policy term f and its derivative df by the log ratio d, for advantage A.
  __device__ static void clipped(const In& in, double d, double A, double& f, double& df,
                                 bool& clip) {
    double bound = 0.0;
    clip = true;
    if (A > 0.0 && d > in.log_over)
      bound = in.over;
    else if (A < 0.0 && d < in.log_under)
      bound = in.under;
    else if (A < 0.0 && d > in.log_dual)
      bound = in.dual;
    else
      clip = false;
    f = clip ? -bound * A : (A == 0.0 ? 0.0 : -exp_f64<false>(d) * A);  // A = 0: 0 for any ratio
    df = clip ? 0.0 : f;
  }
  __device__ static void kl_term(const In& in, double x, double& f, double& df) {
    if (in.kl == FLCE_KL_K1) {
      f = x;
      df = 1.0;
    } else if (in.kl == FLCE_KL_K2) {
      f = 0.5 * x * x;
      df = x;
    } else {
      const double e = exp_f64<true>(-x);
      f = e + x;
      df = -e;
    }
  }
  // The terms of valid token t of sequence s.
  __device__ static void token(const LossArgs<PolicyLoss>& a, const Raw& r, int64_t t, int64_t s,
                               Token& v) {
    const In& in = a.in;
    const double d = (double)r.lp - (double)r.old;
    double df;
    v.counts = kCountValid;
    v.x[0] = d;
    if (!in.by_sequence) {
      bool clip;
      clipped(in, d, in.advantages[in.adv_seq ? s : t], v.x[1], df, clip);
      v.counts += clip ? kCountClipped : 0;
    }
    if (in.ref_logprob != nullptr) kl_term(in, (double)r.lp - (double)r.ref, v.x[2], df);
    v.x[3] = r.ent;
  }
  // Sequence s from its sums: its state, and its share of the batch's.
  __device__ static void item(const LossArgs<PolicyLoss>& a, int64_t s, Total& tot) {
    const In& in = a.in;
    Share v = a.seq_sum[s];
    double df = 0.0;
    if (in.by_sequence && v.n > 0) {
      bool clip;
      double f;
      clipped(in, v.x[0] / v.n, in.advantages[s], f, df, clip);
      v.x[1] = f * v.n;
      v.c = clip ? v.n : 0;
    }
    double w = 1.0;
    if (in.reduction == FLCE_REDUCTION_SEQUENCE_MEAN) w = v.n > 0 ? 1.0 / v.n : 0.0;
    a.state[2 * s] = w;
    a.state[2 * s + 1] = df;
#pragma unroll
    for (int k = 0; k < 4; ++k) tot.x[k] += w * v.x[k];
    tot.x[4] += w * v.c;
    tot.n += v.n;
    tot.c += v.n > 0 ? 1 : 0;
    tot.inv += v.inv;
    tot.bad += v.bad;
  }
  // The batch's factor, from its counts.
  __device__ static double factor(const LossArgs<PolicyLoss>& a, int n, int c, int bad) {
    double k = 1.0;
    if (a.in.reduction == FLCE_REDUCTION_MEAN) k = n > 0 ? 1.0 / n : 0.0;
    if (a.in.reduction == FLCE_REDUCTION_SEQUENCE_MEAN) k = c > 0 ? 1.0 / c : 0.0;
    return bad != 0 ? __builtin_nan("") : k;
  }
  __device__ static void finish(const LossArgs<PolicyLoss>& a, const Total& v) {
    const In& in = a.in;
    const double k = factor(a, v.n, v.c, v.bad);
    a.state[2 * a.B] = k;
    a.state[2 * a.B + 1] = 0.0;
    float* s = a.out.stats;
    // A term whose coefficient is 0 is absent, whatever its value.
    const double kl = in.kl_coef != 0.0 ? in.kl_coef * v.x[2] : 0.0;
    const double ent = in.ent_coef != 0.0 ? in.ent_coef * v.x[3] : 0.0;
    s[0] = (float)(k * (v.x[1] + kl - ent));
    if (a.out.loss != nullptr) a.out.loss[0] = s[0];
    s[1] = (float)(k * v.x[1]);
    s[2] = (float)(k * v.x[2]);
    s[3] = (float)(k * v.x[3]);
    s[4] = (float)(k * v.x[4]);
    s[5] = (float)(0.0 - k * v.x[0]);
    // The counts are of shares that are undefined after bad offsets.
    s[6] = v.bad != 0 ? __builtin_nanf("") : (float)v.n;
    s[7] = v.bad != 0 ? __builtin_nanf("") : (float)v.c;
  }
  __device__ static double state_factor(const LossArgs<PolicyLoss>& a) { return a.state[2 * a.B]; }
  // The reduced loss's upstream gradient.
  __device__ static double upstream(const LossArgs<PolicyLoss>& a) {
    return a.out.grad_loss != nullptr ? (double)a.out.grad_loss[0] : 1.0;
  }
  __device__ static void grad(const LossArgs<PolicyLoss>& a, const Raw& r, double scale, int64_t t,
                              int64_t s) {
    const In& in = a.in;
    float glp = 0.f, gent = 0.f;
    if (s >= 0) {
      double df, f;
      if (in.by_sequence) {
        df = a.state[2 * s + 1];
      } else {
        bool clip;
        clipped(in, (double)r.lp - (double)r.old, in.advantages[in.adv_seq ? s : t], f, df, clip);
      }
      if (in.kl_coef != 0.0) {
        double dk;
        kl_term(in, (double)r.lp - (double)r.ref, f, dk);
        df += in.kl_coef * dk;
      }
      const double w = scale * a.state[2 * s];
      glp = (float)(w * df);
      gent = (float)(0.0 - w * in.ent_coef);
    }
    a.out.grad_logprob[t] = glp;
    if (a.out.grad_entropy != nullptr) a.out.grad_entropy[t] = gent;
  }
};

// ---- the preference loss --------------------------------------------------------------

struct PreferenceLoss {
  struct In {
    const float *logprob, *ref_logprob;
    double beta, eps, margin, half_inv_beta;
    int kind, normalize, reduction;
  };
  struct Out {
    float *loss, *pair_loss, *chosen, *rejected;
    const float* grad_loss;  // [P] under NONE, else [1]; or null
    float* grad_logprob;
  };
  static __host__ __device__ constexpr int state_size(int B) { return B + 1; }
  static constexpr bool kGradReads = false;
  // state[s]: gradient of the reduced loss by a valid token's logprob of
  // sequence s; state[B] = 1, or NaN after bad offsets.
  using Share = LossSum<1>;  // logprob - ref_logprob
  using Token = Terms<1>;
  using Total = LossSum<1>;  // the pairs' losses
  static constexpr int kSides = 2;

  struct Raw {
    float lp, ref;
  };
  __device__ static Raw load(const LossArgs<PreferenceLoss>& a, int64_t t) {
    return {a.in.logprob[t], a.in.ref_logprob != nullptr ? a.in.ref_logprob[t] : 0.f};
  }
  __device__ static void token(const LossArgs<PreferenceLoss>&, const Raw& r, int64_t, int64_t,
                               Token& v) {
    v.counts = kCountValid;
    v.x[0] = (double)r.lp - (double)r.ref;
  }
  __device__ static void item(const LossArgs<PreferenceLoss>& a, int64_t i, Total& tot) {
    const In& in = a.in;
    const int64_t P = a.items;
    const Share c = a.seq_sum[i], r = a.seq_sum[P + i];
    const double ic = in.normalize && c.n > 0 ? 1.0 / c.n : 1.0;
    const double ir = in.normalize && r.n > 0 ? 1.0 / r.n : 1.0;
    // Bad offsets on either side take the whole pair.
    const bool bad = c.bad != 0 || r.bad != 0;
    const double rc = bad ? __builtin_nan("") : c.x[0] * ic;
    const double rr = bad ? __builtin_nan("") : r.x[0] * ir;
    const double diff = rc - rr;
    double loss, slope;  // slope: derivative by diff
    if (in.kind == FLCE_PREFERENCE_IPO) {
      const double u = diff - in.half_inv_beta;
      loss = u * u;
      slope = 2.0 * u;
    } else {
      const double x = in.beta * diff - in.margin;
      if (in.kind == FLCE_PREFERENCE_HINGE) {
        loss = x < 1.0 ? 1.0 - x : (x >= 1.0 ? 0.0 : x);  // the last keeps NaN
        slope = x < 1.0 ? -in.beta : (x >= 1.0 ? 0.0 : x);
      } else {
        // -log sigmoid(x) = log1p(exp(-|x|)) + max(-x, 0); neither it nor the
        // sigmoids overflow.
        const double e = exp(-fabs(x)), tail = log1p(e);
        const double pos = x >= 0.0 ? 1.0 / (1.0 + e) : e / (1.0 + e);  // sigmoid(x)
        const double neg = x >= 0.0 ? e / (1.0 + e) : 1.0 / (1.0 + e);  // sigmoid(-x)
        const double lpos = tail + (x < 0.0 ? -x : 0.0), lneg = tail + (x > 0.0 ? x : 0.0);
        loss = (1.0 - in.eps) * lpos;
        if (in.eps != 0.0) loss += in.eps * lneg;  // lneg may be infinite
        slope = in.beta * (in.eps * pos - (1.0 - in.eps) * neg);
      }
    }
    const double k = in.reduction == FLCE_REDUCTION_MEAN ? 1.0 / (double)P : 1.0;
    a.state[i] = k * slope * ic;
    a.state[P + i] = -k * slope * ir;
    a.out.pair_loss[i] = (float)loss;
    a.out.chosen[i] = (float)(in.beta * rc);
    a.out.rejected[i] = (float)(in.beta * rr);
    tot.x[0] += loss;
    tot.inv += c.inv + r.inv;
    tot.bad += c.bad + r.bad;
  }
  __device__ static double factor(const LossArgs<PreferenceLoss>&, int, int, int bad) {
    return bad != 0 ? __builtin_nan("") : 1.0;
  }
  __device__ static void finish(const LossArgs<PreferenceLoss>& a, const Total& v) {
    a.state[a.B] = factor(a, v.n, v.c, v.bad);
    if (a.in.reduction != FLCE_REDUCTION_NONE) {
      const double k = a.in.reduction == FLCE_REDUCTION_MEAN && a.items > 0
                           ? 1.0 / (double)a.items : 1.0;
      a.out.loss[0] = (float)(k * v.x[0]);
    }
  }
  __device__ static double state_factor(const LossArgs<PreferenceLoss>& a) { return a.state[a.B]; }
  __device__ static double upstream(const LossArgs<PreferenceLoss>& a) {
    const bool one = a.in.reduction != FLCE_REDUCTION_NONE && a.out.grad_loss != nullptr;
    return one ? (double)a.out.grad_loss[0] : 1.0;
  }
  __device__ static void grad(const LossArgs<PreferenceLoss>& a, const Raw&, double scale,
                              int64_t t, int64_t s) {
    double g = 0.0;
    if (s >= 0) {
      g = scale * a.state[s];
      if (a.in.reduction == FLCE_REDUCTION_NONE && a.out.grad_loss != nullptr)
        g *= (double)a.out.grad_loss[s < a.items ? s : s - a.items];
    }
    a.out.grad_logprob[t] = (float)g;
  }
};

// ---- the three steps ----------------------------------------------------------------

// A tile's inputs, lane l having the tokens t0 + 64 j + l. The loads are not all in
// flight at once: those of an optional input sit in branches that wait for it (in the
// policy loss two waits a row, reference and entropy, before the offsets are asked
// for), and a token-level advantage is loaded with the token's terms.
template <class Loss, int ROWS, bool READ>
struct TileRows {
  typename Loss::Raw raw[ROWS];
  int64_t y[ROWS];
  __device__ __forceinline__ void load(const LossArgs<Loss>& a, int64_t t0) {
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const int64_t t = t0 + j * 64 + (threadIdx.x & 63);
      const int64_t tc = t < a.N ? t : a.N - 1;
      y[j] = a.labels[tc];
      if constexpr (READ) raw[j] = Loss::load(a, tc);
    }
  }
};

// Step 1, one wave, one tile of ROWS rows of 64 tokens. A tile in one or two
// sequences, the usual case, adds each lane's tokens and reduces them over the
// wave once a sequence. With more, each row is scanned with the sequences as
// segments, the open segment carried to the next row, and the lane with a
// sequence's last token in the tile has its share. No LDS either way, so the
// occupancy is the registers'; token terms in LDS and sums over them took 36 us where
// this takes 24 (policy loss, 2.07 M tokens in 1000 sequences: 58 MB, 2.4 TB/s), which
// its chain of loads and waits bounds rather than the memory. 32768 tokens take 4.6 us.
template <class Loss, int ROWS>
__device__ __forceinline__ void tile_parts(const LossArgs<Loss>& a, int64_t tile) {
  using Token = typename Loss::Token;
  const int lane = threadIdx.x & 63;
  const int64_t t0 = tile * (ROWS * 64);
  const int64_t t1 = a.N - t0 < ROWS * 64 ? a.N : t0 + ROWS * 64;
  TileRows<Loss, ROWS, true> in;
  in.load(a, t0);
  const TileSeqs r = tile_sequences(a.cu, a.B, a.N, t0, t1);
  if (r.ns <= 0) return;
  Token v0, v1;  // up to two sequences: their sums; more: v0 is the carried segment's
  v0.clear();
  v1.clear();
  int rank0 = -1;        // the carried segment
  bool any0 = false, any1 = false;
#pragma unroll
  for (int j = 0; j < ROWS; ++j) {
    const int tl = j * 64 + lane;
    const int64_t t = t0 + tl;
    int rank = token_rank(a.cu, r, t0, tl);
    if (t >= a.N) rank = -1;
    Token v;
    v.clear();
    if (rank >= 0) {
      if (label_valid(in.y[j], a.ignore_index, a.V))
        Loss::token(a, in.raw[j], t, r.s0 + rank, v);
      else if (in.y[j] != a.ignore_index)
        v.counts = kCountInvalid;
    }
    if (r.ns <= 2) {
      if (rank == 0) {
        v0.add(v);
        any0 = true;
      } else if (rank == 1) {
        v1.add(v);
        any1 = true;
      }
      continue;
    }
    const int before = __shfl_up(rank, 1, 64);
    const uint64_t heads = __builtin_amdgcn_ballot_w64(lane == 0 || before != rank);
    // This lane's segment starts at the last head at or below it.
    const int head = 63 - __builtin_clzll(heads & (~(uint64_t)0 >> (63 - lane)));
#pragma unroll 1
    for (int d = 1; d < 64; d <<= 1) {
      const Token o = v.up(d);
      if (lane - d >= head) v.add(o);
    }
    if (rank == rank0 && rank >= 0) v.add(v0);  // only the first segment can match
    const bool ends = ends_sequence(a.cu, r, t0, tl, rank < 0 ? 0 : rank);
    if (rank >= 0 && (ends || t + 1 == t1)) a.parts[r.s0 + rank + tile] = v.share();
    if (j + 1 < ROWS) {
      v0 = v.from(63);
      rank0 = __shfl(rank, 63, 64);
    }
  }
  if (r.ns > 2) return;
  if (__builtin_amdgcn_ballot_w64(any0) != 0) {
    v0.wave_sum();
    if (lane == 63) a.parts[r.s0 + tile] = v0.share();
  }
  if (__builtin_amdgcn_ballot_w64(any1) != 0) {
    v1.wave_sum();
    if (lane == 63) a.parts[r.s0 + 1 + tile] = v1.share();
  }
}

// Shares of sequence s: tiles [p0, p0 + count); a sequence with bad offsets has
// none.
struct SeqParts {
  int64_t p0, count;
  bool bad;
};
__device__ __forceinline__ SeqParts seq_parts(const int64_t* cu, int64_t N, int rows, int64_t s) {
  const int64_t b = seq_begin(cu, s), e = seq_end(cu, s, N);
  if (b < 0 || e < b || e > N) return {0, 0, true};
  if (b == e) return {0, 0, false};
  const int sh = 5 + __builtin_ffs(rows);  // log2 of the tile: rows is a power of two
  return {b >> sh, ((e - 1) >> sh) - (b >> sh) + 1, false};
}

// Step 2, one block, items [i0, i1): adds up the sequences' shares, then the
// items (5.7 us for 1000 sequences in 16 blocks; 45 us in one block). Groups of
// lanes take a sequence each, sized by the average number of shares; a sequence
// with far more than that is added by the whole block.
template <class Loss>
__device__ __forceinline__ typename Loss::Total sum_sequences(const LossArgs<Loss>& a, int64_t i0,
                                                              int64_t i1) {
  using Share = typename Loss::Share;
  using Total = typename Loss::Total;
  __shared__ Share sh_share[16];
  __shared__ Total sh_total[16];
  const int64_t m = i1 - i0, local = m * Loss::kSides;
  auto seq = [&](int64_t j) { return j < m ? i0 + j : a.items + i0 + (j - m); };
  const int g = lanes_per_sequence(a.B, a.tiles);
  const int64_t longest = (int64_t)g * 16;
  const int groups = (int)blockDim.x / g, k = threadIdx.x & (g - 1);
  bool any_long = false;
  for (int64_t jb = 0; jb < local; jb += groups) {
    const int64_t j = jb + threadIdx.x / g;
    Share v;
    v.clear();
    bool mine = j < local;
    int64_t s = 0;
    if (mine) {
      s = seq(j);
      const SeqParts p = seq_parts(a.cu, a.N, a.rows, s);
      if (p.count > longest) {
        any_long = true;
        mine = false;
      } else {
        for (int64_t q = k; q < p.count; q += g) v.add(a.parts[s + p.p0 + q]);
        v.bad = p.bad && k == 0 ? 1 : 0;
        if (v.bad != 0) v.x[0] = __builtin_nan("");
      }
    }
    v.group_sum(g);
    if (mine && k == 0) a.seq_sum[s] = v;
  }
  if (__syncthreads_or(any_long ? 1 : 0)) {
    for (int64_t jb = 0; jb < local; jb += 64) {
      const int64_t jl = jb + (threadIdx.x & 63);
      const bool lg = jl < local && seq_parts(a.cu, a.N, a.rows, seq(jl)).count > longest;
      uint64_t bits = __builtin_amdgcn_ballot_w64(lg);  // the same in every wave
      while (bits != 0) {
        const int64_t s = seq(jb + __builtin_ctzll(bits));
        bits &= bits - 1;
        const SeqParts p = seq_parts(a.cu, a.N, a.rows, s);
        Share v;
        v.clear();
        for (int64_t q = threadIdx.x; q < p.count; q += blockDim.x) v.add(a.parts[s + p.p0 + q]);
        v = block_total(v, (int)(blockDim.x >> 6), sh_share);
        v.bad = 0;  // its own offsets are good; shares that no tile wrote hold anything
        if (threadIdx.x == 0) a.seq_sum[s] = v;
      }
    }
    __syncthreads();
  }
  Total t;
  t.clear();
  for (int64_t i = i0 + threadIdx.x; i < i1; i += blockDim.x) Loss::item(a, i, t);
  const int64_t waves = (m + 63) >> 6, nw = blockDim.x >> 6;
  return block_total(t, (int)(waves < nw ? waves : nw), sh_total);
}

template <class Loss>
__device__ __forceinline__ void finish_batch(const LossArgs<Loss>& a,
                                             const typename Loss::Total& t) {
  if (threadIdx.x == 0) {
    a.header[0] = t.bad != 0 ? t.bad : t.inv;  // shares are undefined beside bad offsets
    a.header[1] = t.n;
    Loss::finish(a, t);
  }
}

// The batch's factor for the gradients, in every lane: from the state, or from the
// counts of the blocks that step 2 left unadded (at most 64, one a lane).
template <class Loss>
__device__ __forceinline__ double batch_factor(const LossArgs<Loss>& a) {
  if (a.deferred == 0) return Loss::state_factor(a);
  const int lane = threadIdx.x & 63;
  int n = 0, c = 0, bad = 0;
  if (lane < a.deferred) {
    n = a.totals[lane].n;
    c = a.totals[lane].c;
    bad = a.totals[lane].bad;
  }
  n = __builtin_amdgcn_readlane(wave_sum_dpp(n), 63);
  c = __builtin_amdgcn_readlane(wave_sum_dpp(c), 63);
  bad = __builtin_amdgcn_readlane(wave_sum_dpp(bad), 63);
  return Loss::factor(a, n, c, bad);
}

// Step 3, one wave, one tile: the inputs again, now out of the MALL for most batches
// (policy loss, 2.07 M tokens: 75 MB in 19 us, 3.9 TB/s).
template <class Loss, int ROWS>
__device__ __forceinline__ void tile_grads(const LossArgs<Loss>& a, int64_t tile) {
  const int64_t t0 = tile * (ROWS * 64);
  const int64_t t1 = a.N - t0 < ROWS * 64 ? a.N : t0 + ROWS * 64;
  TileRows<Loss, ROWS, Loss::kGradReads> in;
  in.load(a, t0);
  const TileSeqs r = tile_sequences(a.cu, a.B, a.N, t0, t1);
  const double factor = batch_factor(a);
  const double scale = Loss::upstream(a) * factor;
  // The factor is NaN after bad offsets, and only then. A valid token may lie in no
  // sequence there; it goes with the first, and so has a NaN gradient as all others.
  const int64_t none = factor != factor ? 0 : -1;
#pragma unroll
  for (int j = 0; j < ROWS; ++j) {
    const int tl = j * 64 + (threadIdx.x & 63);
    const int rank = token_rank(a.cu, r, t0, tl);
    const int64_t t = t0 + tl;
    if (t >= a.N) continue;
    const int64_t s = rank >= 0 ? r.s0 + rank : none;
    const bool valid = s >= 0 && label_valid(in.y[j], a.ignore_index, a.V);
    Loss::grad(a, in.raw[j], scale, t, valid ? s : -1);
  }
}

template <class Loss, int ROWS>
__global__ void __launch_bounds__(64 * kLossWaves) loss_parts_kernel(LossArgs<Loss> a) {
  if (blockIdx.x == 0 && threadIdx.x == 0) a.header[2] = 0;  // for the next kernel's count
  const int64_t tile = (int64_t)blockIdx.x * kLossWaves + (threadIdx.x >> 6);
  if (tile < a.tiles) tile_parts<Loss, ROWS>(a, tile);
}

// Adds up the totals of `blocks` blocks, in block order, and finishes the batch.
template <class Loss>
__device__ __forceinline__ void finish_blocks(const LossArgs<Loss>& a, int blocks,
                                              typename Loss::Total* sh) {
  typename Loss::Total t;
  t.clear();
  for (int b = threadIdx.x; b < blocks; b += blockDim.x) t.add(a.totals[b]);
  t = block_total(t, (int)(blockDim.x >> 6), sh);
  finish_batch(a, t);
}

// A block takes `per` items. With several blocks the one that is done last finishes
// the batch, or the next kernel if that is there: passing on what other blocks
// wrote within a launch costs 5 us of fences and round trips.
template <class Loss>
__global__ void __launch_bounds__(kSeqThreads) loss_sequences_kernel(LossArgs<Loss> a,
                                                                     int64_t per) {
  using Total = typename Loss::Total;
  __shared__ Total sh[kSeqThreads / 64];
  __shared__ int last;
  const int64_t i0 = (int64_t)blockIdx.x * per;
  const int64_t i1 = a.items - i0 < per ? a.items : i0 + per;
  Total t = sum_sequences(a, i0, i1);
  if (gridDim.x > 1) {
    if (a.deferred != 0) {
      if (threadIdx.x == 0) a.totals[blockIdx.x] = t;
      return;
    }
    if (threadIdx.x == 0) {
      a.totals[blockIdx.x] = t;
      __threadfence();
      const int done = __hip_atomic_fetch_add(&a.header[2], 1, __ATOMIC_ACQ_REL,
                                              __HIP_MEMORY_SCOPE_AGENT);
      last = done == (int)gridDim.x - 1 ? 1 : 0;
    }
    __syncthreads();
    if (last == 0) return;
    __threadfence();
    finish_blocks(a, (int)gridDim.x, sh);
    return;
  }
  finish_batch(a, t);
}

template <class Loss, int ROWS>
__global__ void __launch_bounds__(64 * kLossWaves) loss_grads_kernel(LossArgs<Loss> a) {
  __shared__ typename Loss::Total sh[kLossWaves];
  const int64_t tile = (int64_t)blockIdx.x * kLossWaves + (threadIdx.x >> 6);
  if (tile < a.tiles) tile_grads<Loss, ROWS>(a, tile);
  if (a.deferred != 0 && blockIdx.x == 0) finish_blocks(a, a.deferred, sh);
}

// All three steps in one block, for small batches; the steps exchange their sums
// through LDS. Bound by latency: 8.1 us for 413 tokens, half of it the loads and
// exponentials of the two token steps.
template <class Loss, bool GRADS>
__global__ void __launch_bounds__(64 * kSmallWaves) loss_small_kernel(LossArgs<Loss> a) {
  __shared__ typename Loss::Share parts[kSmallSequences + kSmallTokens / 64];
  __shared__ typename Loss::Share seq_sum[kSmallSequences];
  __shared__ double state[2 * kSmallSequences + 2];
  double* const out_state = a.state;  // the caller's, or null
  a.parts = parts;
  a.seq_sum = seq_sum;
  a.state = state;
  const int w = threadIdx.x >> 6;
  for (int64_t tile = w; tile < a.tiles; tile += kSmallWaves) tile_parts<Loss, 1>(a, tile);
  __syncthreads();
  finish_batch(a, sum_sequences(a, 0, a.items));
  __syncthreads();
  if (out_state != nullptr)
    for (int i = threadIdx.x; i < Loss::state_size((int)a.B); i += blockDim.x)
      out_state[i] = state[i];
  if constexpr (GRADS)
    for (int64_t tile = w; tile < a.tiles; tile += kSmallWaves) tile_grads<Loss, 1>(a, tile);
}

}  // namespace flce
