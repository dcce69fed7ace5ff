// Kernels of the embedding lookup and its gradient (gfx950).
//
//   hidden_i = scale * E[x_i]                E[v]: row v of a [V,H] table, or
//   dE[v] = scale * sum_{x_i = v} g_i        column v of the head's [H,V] weight
//
// Lookup: a table's rows are copied 16 bytes a lane. A column of [H,V] touches a
// cache line of 64 columns for every one of its H values; with the tokens
// sorted, lanes, waves and blocks that run together ask for the same lines, and
// each line comes from memory about once however many of its columns are used.
//
// Gradient: a stable radix sort puts equal tokens side by side (a token's
// positions stay in order, so every sum has one fixed order and no atomics are
// needed), then each row of dE sums its run of gradient rows and is written
// once, zeros included. A frequent token's run can be a large part of the batch:
// runs longer than kPiece positions are cut at multiples of kPiece, the pieces
// summed in parallel to fp32 rows, and those summed in order by the row's owner.
// At most two split runs overlap a piece (the one that comes in and the one that
// goes out), so 2 rows a piece hold them.
//
// What bounds them: the bytes (the lookup its output and the distinct rows, the
// gradient the write of all of dE), and for small batches the sort's latency.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "flce_ops_plan.hpp"

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

// Eight consecutive values (16 or 32 bytes, 16-byte aligned) from an array of
// bf16 or fp32.
template <bool F32>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[8]) {
  if constexpr (F32) {
    const ef32x4* q = reinterpret_cast<const ef32x4*>(static_cast<const float*>(p) + i);
    const ef32x4 a = q[0], b = q[1];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = a[k];
      v[4 + k] = b[k];
    }
  } else {
    unpack8(*reinterpret_cast<const eu32x4*>(static_cast<const uint16_t*>(p) + i), v);
  }
}
template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&v)[8]) {
  if constexpr (F32) {
    ef32x4* q = reinterpret_cast<ef32x4*>(static_cast<float*>(p) + i);
    q[0] = ef32x4{v[0], v[1], v[2], v[3]};
    q[1] = ef32x4{v[4], v[5], v[6], v[7]};
  } else {
    *reinterpret_cast<eu32x4*>(static_cast<uint16_t*>(p) + i) = pack8(v);
  }
}

// ---- tokens -> keys ---------------------------------------------------------------

struct TokenArgs {
  const int64_t* tokens;
  int64_t N, Vs, v_begin, V_total, ignore_index;
  int32_t* header;  // [0] tokens outside [0, V_total), [1] tokens of the slice
};

// Row of token x in the slice, or Vs when it takes no part.
__device__ __forceinline__ int32_t token_key(const TokenArgs& a, int64_t x, bool& invalid) {
  invalid = x != a.ignore_index && (x < 0 || x >= a.V_total);
  const bool in = x != a.ignore_index && x >= 0 && x < a.V_total && x >= a.v_begin &&
                  x < a.v_begin + a.Vs;
  return in ? (int32_t)(x - a.v_begin) : (int32_t)a.Vs;
}

__device__ __forceinline__ int block_sum_int(int v, int* sh) {
  for (int d = 32; d > 0; d >>= 1) v += __shfl_down(v, d, 64);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  int r = 0;
  for (int w = 0; w < (int)(blockDim.x >> 6); ++w) r += sh[w];
  __syncthreads();
  return r;
}

// One block: the header's counts.
__device__ __forceinline__ void count_tokens(const TokenArgs& a, int* sh) {
  int inv = 0, n = 0;
  for (int64_t i = threadIdx.x; i < a.N; i += blockDim.x) {
    bool bad;
    n += token_key(a, a.tokens[i], bad) < a.Vs ? 1 : 0;
    inv += bad ? 1 : 0;
  }
  inv = block_sum_int(inv, sh);
  n = block_sum_int(n, sh);
  if (threadIdx.x == 0) {
    a.header[0] = inv;
    a.header[1] = n;
  }
}

__global__ void __launch_bounds__(64) embed_clear_kernel(int32_t* header) {
  if (threadIdx.x < 2) header[threadIdx.x] = 0;
}

// ---- stable sort by key -------------------------------------------------------------

// Lanes whose digit (bits wide) equals this lane's.
__device__ __forceinline__ uint64_t match_digit(uint32_t d, int bits) {
  uint64_t m = ~(uint64_t)0;
  for (int b = 0; b < bits; ++b) {
    const bool set = (d >> b) & 1u;
    const uint64_t bal = __builtin_amdgcn_ballot_w64(set);
    m &= set ? bal : ~bal;
  }
  return m;
}

__device__ __forceinline__ int lanes_below(uint64_t m) {
  return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32),
                                        __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u));
}

// Ranks the wave's next item among the wave's earlier items of its digit, using
// and updating the wave's counters cnt[digit].
__device__ __forceinline__ int wave_rank(uint32_t d, int bits, uint16_t* cnt) {
  const uint64_t m = match_digit(d, bits);
  const int below = lanes_below(m);
  const int base = cnt[d];
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  if (below == 0) cnt[d] = (uint16_t)(base + __popcll(m));
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  return base + below;
}

// Exclusive scan over the block's threads; sh: one int a wave.
__device__ __forceinline__ int block_exclusive(int v, int* sh) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int x = v;
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d, 64);
    if (lane >= d) x += y;
  }
  if (lane == 63) sh[w] = x;
  __syncthreads();
  int off = 0;
  for (int k = 0; k < (int)(blockDim.x >> 6); ++k) off += k < w ? sh[k] : 0;
  __syncthreads();
  return off + x - v;
}

constexpr int kSortWaves = 16;
constexpr int kSortDigits = 512;

// All passes in one block with the keys in LDS: 1024 * ITEMS items. Item order is
// wave, then round, then lane, so ranks by (wave, round, lane) keep it.
template <int ITEMS>
__global__ void __launch_bounds__(64 * kSortWaves) embed_sort_block_kernel(TokenArgs a, int passes,
                                                                           int bits, int32_t* key,
                                                                           int32_t* perm) {
  constexpr int kCap = 64 * kSortWaves * ITEMS;
  __shared__ uint32_t skey[kCap];
  __shared__ uint32_t sperm[kCap];
  __shared__ uint16_t cnt[kSortWaves][kSortDigits];
  __shared__ int base[kSortDigits];
  __shared__ int sh[kSortWaves];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int nd = 1 << bits;
  const uint32_t last = (uint32_t)(((uint64_t)1 << (passes * bits)) - 1);  // >= every key
  uint32_t k[ITEMS], p[ITEMS];
  int rank[ITEMS];
  int inv = 0, n = 0;
#pragma unroll
  for (int j = 0; j < ITEMS; ++j) {
    const int i = (w * ITEMS + j) * 64 + lane;
    k[j] = last;
    p[j] = (uint32_t)i;
    if (i < a.N) {
      bool bad;
      k[j] = (uint32_t)token_key(a, a.tokens[i], bad);
      n += k[j] < (uint32_t)a.Vs ? 1 : 0;
      inv += bad ? 1 : 0;
    }
  }
  inv = block_sum_int(inv, sh);
  n = block_sum_int(n, sh);
  if (threadIdx.x == 0) {
    a.header[0] = inv;
    a.header[1] = n;
  }
  for (int pass = 0; pass < passes; ++pass) {
    const int shift = pass * bits;
    for (int i = threadIdx.x; i < kSortWaves * nd; i += 64 * kSortWaves) {
      const int cw = i >> bits;
      cnt[cw][i & (nd - 1)] = 0;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < ITEMS; ++j)
      rank[j] = wave_rank((k[j] >> shift) & (uint32_t)(nd - 1), bits, cnt[w]);
    __syncthreads();
    int total = 0;
    if ((int)threadIdx.x < nd) {
      for (int v = 0; v < kSortWaves; ++v) {
        const int c = cnt[v][threadIdx.x];
        cnt[v][threadIdx.x] = (uint16_t)total;  // <= 16384 - 1 where an item follows
        total += c;
      }
    }
    const int off = block_exclusive(total, sh);
    if ((int)threadIdx.x < nd) base[threadIdx.x] = off;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
      const uint32_t d = (k[j] >> shift) & (uint32_t)(nd - 1);
      const int q = base[d] + cnt[w][d] + rank[j];
      skey[q] = k[j];
      sperm[q] = p[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
      const int i = (w * ITEMS + j) * 64 + lane;
      k[j] = skey[i];
      p[j] = sperm[i];
    }
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < ITEMS; ++j) {
    const int i = (w * ITEMS + j) * 64 + lane;
    if (i < a.N) {
      key[i] = (int32_t)k[j];
      perm[i] = (int32_t)p[j];
    }
  }
}

// The larger sort, a pass: digit counts of every tile of kSortTile items, the
// counts' prefix over the tiles (a wave a digit), and the move. Pass 0 reads the
// tokens, later ones the previous pass's keys.
struct SortArgs {
  TokenArgs t;
  const int32_t *key_in, *perm_in;  // null: from the tokens
  int32_t *key_out, *perm_out;
  int32_t* counts;                  // [digit][tile]
  int64_t tiles;
  int shift, bits;
};

constexpr int kSortMoveWaves = 4;
constexpr int kSortRounds = kSortTile / (64 * kSortMoveWaves);

__device__ __forceinline__ uint32_t sort_key(const SortArgs& a, int64_t i, bool& bad) {
  bad = false;
  return a.key_in != nullptr ? (uint32_t)a.key_in[i] : (uint32_t)token_key(a.t, a.t.tokens[i], bad);
}

__global__ void __launch_bounds__(256) embed_sort_count_kernel(SortArgs a) {
  __shared__ int hist[1 << kMaxDigitBits];
  __shared__ int sh[4];
  const int nd = 1 << a.bits;
  for (int d = threadIdx.x; d < nd; d += 256) hist[d] = 0;
  __syncthreads();
  int inv = 0, n = 0;
  const int64_t i0 = (int64_t)blockIdx.x * kSortTile;
  for (int j = 0; j < kSortTile / 256; ++j) {
    const int64_t i = i0 + j * 256 + threadIdx.x;
    if (i < a.t.N) {
      bool bad;
      const uint32_t k = sort_key(a, i, bad);
      inv += bad ? 1 : 0;
      n += k < (uint32_t)a.t.Vs ? 1 : 0;
      atomicAdd(&hist[(k >> a.shift) & (uint32_t)(nd - 1)], 1);  // counts: any order is the same
    }
  }
  __syncthreads();
  for (int d = threadIdx.x; d < nd; d += 256) a.counts[d * a.tiles + blockIdx.x] = hist[d];
  if (a.key_in == nullptr) {
    inv = block_sum_int(inv, sh);
    n = block_sum_int(n, sh);
    if (threadIdx.x == 0) {
      if (inv != 0) atomicAdd(&a.t.header[0], inv);
      if (n != 0) atomicAdd(&a.t.header[1], n);
    }
  }
}

// A wave a digit: counts[d][*] becomes its exclusive prefix over the tiles, the
// digit's total goes to totals[d].
__global__ void __launch_bounds__(256) embed_sort_scan_kernel(int32_t* counts, int64_t tiles,
                                                              int nd, int32_t* totals) {
  const int lane = threadIdx.x & 63;
  const int d = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (d >= nd) return;
  int32_t* c = counts + d * tiles;
  int run = 0;
  for (int64_t t0 = 0; t0 < tiles; t0 += 64) {
    const int64_t t = t0 + lane;
    const int v = t < tiles ? c[t] : 0;
    int x = v;
    for (int s = 1; s < 64; s <<= 1) {
      const int y = __shfl_up(x, s, 64);
      if (lane >= s) x += y;
    }
    if (t < tiles) c[t] = run + x - v;
    run += __shfl(x, 63, 64);
  }
  if (lane == 0) totals[d] = run;
}

__global__ void __launch_bounds__(64 * kSortMoveWaves) embed_sort_move_kernel(SortArgs a,
                                                                              const int32_t* totals) {
  __shared__ uint16_t cnt[kSortMoveWaves][1 << kMaxDigitBits];
  __shared__ int base[1 << kMaxDigitBits];
  __shared__ int sh[kSortMoveWaves];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int nd = 1 << a.bits;
  const int64_t i0 = (int64_t)blockIdx.x * kSortTile + w * (kSortTile / kSortMoveWaves);
  for (int i = threadIdx.x; i < kSortMoveWaves * nd; i += 256) cnt[i >> a.bits][i & (nd - 1)] = 0;
  // Each thread owns 8 consecutive digits of the scan over the totals.
  constexpr int kPer = (1 << kMaxDigitBits) / 256;
  int t[kPer], sum = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int d = threadIdx.x * kPer + q;
    t[q] = d < nd ? totals[d] : 0;
    sum += t[q];
  }
  int off = block_exclusive(sum, sh);
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int d = threadIdx.x * kPer + q;
    if (d < nd) base[d] = off + a.counts[d * a.tiles + blockIdx.x];
    off += t[q];
  }
  __syncthreads();
  uint32_t k[kSortRounds];
  int rank[kSortRounds];
#pragma unroll
  for (int j = 0; j < kSortRounds; ++j) {
    const int64_t i = i0 + j * 64 + lane;
    bool bad;
    // Past the end: the largest digit, behind every item.
    k[j] = i < a.t.N ? sort_key(a, i, bad) : 0xFFFFFFFFu;
    rank[j] = wave_rank((k[j] >> a.shift) & (uint32_t)(nd - 1), a.bits, cnt[w]);
  }
  __syncthreads();
  for (int d = threadIdx.x; d < nd; d += 256) {
    int run = 0;
    for (int v = 0; v < kSortMoveWaves; ++v) {
      const int c = cnt[v][d];
      cnt[v][d] = (uint16_t)run;
      run += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kSortRounds; ++j) {
    const int64_t i = i0 + j * 64 + lane;
    if (i < a.t.N) {
      const uint32_t d = (k[j] >> a.shift) & (uint32_t)(nd - 1);
      const int64_t q = (int64_t)base[d] + cnt[w][d] + rank[j];
      a.key_out[q] = (int32_t)k[j];
      a.perm_out[q] = a.perm_in != nullptr ? a.perm_in[i] : (int32_t)i;
    }
  }
}

// ---- lookup ---------------------------------------------------------------------------

struct GatherArgs {
  TokenArgs t;
  const uint16_t* weight;
  const int32_t *key, *perm;  // sorted order, or null: token order
  int64_t H;
  float scale;
  uint16_t* out;
  int count_block;            // 1: the last block of grid.x fills the header
  int tpr;                    // threads a row (table lookup)
};

constexpr int kGatherRows = 4;  // rows a thread has in flight

// Rows of a table [Vs,H]: tpr threads a row, 8 values each.
__global__ void __launch_bounds__(256) embed_gather_rows_kernel(GatherArgs a) {
  __shared__ int sh[4];
  if (a.count_block != 0 && blockIdx.x == gridDim.x - 1) {
    if (blockIdx.y == 0) count_tokens(a.t, sh);
    return;
  }
  const int per = 256 / a.tpr;  // rows side by side
  const int64_t h = ((int64_t)blockIdx.y * a.tpr + threadIdx.x % a.tpr) * 8;
  const int64_t r0 = (int64_t)blockIdx.x * per * kGatherRows + threadIdx.x / a.tpr;
  int32_t key[kGatherRows];
  int inv = 0, n = 0;
#pragma unroll
  for (int j = 0; j < kGatherRows; ++j) {
    const int64_t i = r0 + j * per;
    bool bad = false;
    key[j] = i < a.t.N ? token_key(a.t, a.t.tokens[i], bad) : (int32_t)a.t.Vs;
    inv += bad ? 1 : 0;
    n += key[j] < a.t.Vs ? 1 : 0;
  }
  if (a.count_block == 0 && blockIdx.y == 0) {
    // One thread a row counts.
    inv = block_sum_int(threadIdx.x % a.tpr == 0 ? inv : 0, sh);
    n = block_sum_int(threadIdx.x % a.tpr == 0 ? n : 0, sh);
    if (threadIdx.x == 0) {
      if (inv != 0) atomicAdd(&a.t.header[0], inv);
      if (n != 0) atomicAdd(&a.t.header[1], n);
    }
  }
  if (h >= a.H) return;
  eu32x4 w[kGatherRows];
#pragma unroll
  for (int j = 0; j < kGatherRows; ++j) {
    w[j] = eu32x4{0u, 0u, 0u, 0u};
    if (key[j] < a.t.Vs)
      w[j] = *reinterpret_cast<const eu32x4*>(a.weight + (int64_t)key[j] * a.H + h);
  }
#pragma unroll
  for (int j = 0; j < kGatherRows; ++j) {
    const int64_t i = r0 + j * per;
    if (i >= a.t.N) continue;
    eu32x4 o = w[j];
    if (a.scale != 1.f && key[j] < a.t.Vs) {
      float v[8];
      unpack8(w[j], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= a.scale;
      o = pack8(v);
    }
    *reinterpret_cast<eu32x4*>(a.out + i * a.H + h) = o;
  }
}

// Columns of a weight [H,Vs]: a wave takes 8 consecutive (sorted) tokens and 64
// hidden values; lane (t, g) gathers 8 values of token t down the rows 8 g .. and
// stores them as 16 bytes, 128 contiguous bytes a token.
constexpr int kGatherTokens = 32;  // tokens a block

__global__ void __launch_bounds__(256) embed_gather_cols_kernel(GatherArgs a) {
  __shared__ int sh[4];
  if (a.count_block != 0 && blockIdx.x == gridDim.x - 1) {
    if (blockIdx.y == 0) count_tokens(a.t, sh);
    return;
  }
  const int lane = threadIdx.x & 63;
  const int64_t i = (int64_t)blockIdx.x * kGatherTokens + (threadIdx.x >> 6) * 8 + (lane & 7);
  const int64_t h = (int64_t)blockIdx.y * 64 + (lane >> 3) * 8;
  if (i >= a.t.N || h >= a.H) return;
  bool bad;
  const int32_t key = a.key != nullptr ? a.key[i] : token_key(a.t, a.t.tokens[i], bad);
  const int64_t row = a.perm != nullptr ? a.perm[i] : i;
  eu32x4 o = eu32x4{0u, 0u, 0u, 0u};
  if (key < a.t.Vs) {
    const uint16_t* src = a.weight + h * a.t.Vs + key;
    uint32_t u[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = src[e * a.t.Vs];
    if (a.scale == 1.f) {
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = u[2 * e] | (u[2 * e + 1] << 16);
    } else {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = bf16_lo(u[e]) * a.scale;
      o = pack8(v);
    }
  }
  *reinterpret_cast<eu32x4*>(a.out + row * a.H + h) = o;
}

// ---- gradient ------------------------------------------------------------------------

struct GradArgs {
  const void* grad;           // [N,H]
  const int32_t *key, *perm;  // sorted
  const int32_t* header;      // [1] tokens of the slice: the sorted positions that count
  int32_t* starts;            // [Vs + 1]
  float* part;                // [2 * pieces][H]
  int64_t N, H, Vs;
  float scale;
  void* out;
  int start_blocks;           // blocks of the segments kernel that fill starts
  int chunks;                 // column chunks a piece
  int tpr;                    // threads a row (table layout)
};

// acc += gradient rows of the sorted positions [b, e), in order.
template <bool HF32>
__device__ __forceinline__ void add_rows(const GradArgs& a, int64_t b, int64_t e, int64_t h,
                                         float (&acc)[8]) {
  int64_t i = b;
  for (; i + 4 <= e; i += 4) {
    float v[4][8];
#pragma unroll
    for (int j = 0; j < 4; ++j) load8<HF32>(a.grad, (int64_t)a.perm[i + j] * a.H + h, v[j]);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[c] += v[j][c];
  }
  for (; i < e; ++i) {
    float v[8];
    load8<HF32>(a.grad, (int64_t)a.perm[i] * a.H + h, v);
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] += v[c];
  }
}

// The sum of the run [b, e): directly, or from its pieces' sums.
template <bool HF32>
__device__ __forceinline__ void run_sum(const GradArgs& a, int64_t b, int64_t e, int64_t h,
                                        float (&acc)[8]) {
#pragma unroll
  for (int c = 0; c < 8; ++c) acc[c] = 0.f;
  if (e - b <= kPiece) {
    add_rows<HF32>(a, b, e, h, acc);
    return;
  }
  const int64_t p0 = b / kPiece, p1 = (e - 1) / kPiece;
  int64_t p = p0;
  if (b > p0 * kPiece) {  // starts inside its first piece
    load8<true>(a.part, (2 * p0 + 1) * a.H + h, acc);
    ++p;
  }
  for (; p + 4 <= p1 + 1; p += 4) {
    float v[4][8];
#pragma unroll
    for (int j = 0; j < 4; ++j) load8<true>(a.part, 2 * (p + j) * a.H + h, v[j]);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[c] += v[j][c];
  }
  for (; p <= p1; ++p) {
    float v[8];
    load8<true>(a.part, 2 * p * a.H + h, v);
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] += v[c];
  }
}

// First blocks: starts[v], the first sorted position with key >= v. The others:
// one piece and column chunk each, summing the split runs that overlap it.
template <bool HF32>
__global__ void __launch_bounds__(256) embed_segments_kernel(GradArgs a) {
  const int64_t n = a.header[1];
  if ((int)blockIdx.x < a.start_blocks) {
    const int64_t v = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (v > a.Vs) return;
    int64_t lo = 0, hi = n;
    while (lo < hi) {
      const int64_t mid = (lo + hi) >> 1;
      if (a.key[mid] < v)
        lo = mid + 1;
      else
        hi = mid;
    }
    a.starts[v] = (int32_t)lo;
    return;
  }
  const int64_t id = (int64_t)blockIdx.x - a.start_blocks;
  const int64_t piece = id / a.chunks;
  const int64_t q0 = piece * kPiece;
  if (q0 >= n) return;
  const int64_t h = ((id % a.chunks) * blockDim.x + threadIdx.x) * 8;
  // Keys around the piece: positions q0 - 32 .. q0 + 31 and q0 + 32 .. q0 + 95;
  // -1 (no key) outside the slice's tokens.
  const int lane = threadIdx.x & 63;
  const int64_t i0 = q0 - kPiece + lane, i1 = q0 + kPiece + lane;
  const int32_t x0 = i0 >= 0 && i0 < n ? a.key[i0] : -1;
  const int32_t x1 = i1 < n ? a.key[i1] : -1;
  const int64_t qe = q0 + kPiece < n ? q0 + kPiece : n;  // the piece's end
  const int in = (int)(qe - q0);
  const int32_t first = __shfl(x0, kPiece, 64);
  const int32_t last = __shfl(x0, kPiece + in - 1, 64);
  // Equal keys are consecutive, so counts are lengths.
  const uint64_t f0 = __builtin_amdgcn_ballot_w64(x0 == first);
  const uint64_t f1 = __builtin_amdgcn_ballot_w64(x1 == first);
  const uint64_t l0 = __builtin_amdgcn_ballot_w64(x0 == last);
  const uint64_t l1 = __builtin_amdgcn_ballot_w64(x1 == last);
  const int head = __popcll(f0 >> kPiece);          // of `first`, within the piece
  const int tail = __popcll(l0 >> kPiece);          // of `last`, within the piece
  const bool split_first = __popcll(f0) + __popcll(f1) > kPiece;
  const bool split_last = last != first && tail + __popcll(l1) > kPiece;
  if (h >= a.H) return;
  if (split_first) {
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    add_rows<HF32>(a, q0, q0 + head, h, acc);
    store8<true>(a.part, 2 * piece * a.H + h, acc);
  }
  if (split_last) {
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    add_rows<HF32>(a, qe - tail, qe, h, acc);
    store8<true>(a.part, (2 * piece + 1) * a.H + h, acc);
  }
}

constexpr int kGradRows = 8;  // rows a thread takes one after another

// Rows of a table gradient [Vs,H].
template <bool HF32, bool GF32, bool ACC>
__global__ void __launch_bounds__(256) embed_grad_rows_kernel(GradArgs a) {
  const int per = 256 / a.tpr;
  const int64_t h = ((int64_t)blockIdx.y * a.tpr + threadIdx.x % a.tpr) * 8;
  const int64_t v0 = (int64_t)blockIdx.x * per * kGradRows + threadIdx.x / a.tpr;
  if (h >= a.H) return;
#pragma unroll 2
  for (int j = 0; j < kGradRows; ++j) {
    const int64_t v = v0 + j * per;
    if (v >= a.Vs) return;
    const int64_t b = a.starts[v], e = a.starts[v + 1];
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (b == e) {
      if constexpr (!ACC) store8<GF32>(a.out, v * a.H + h, acc);
      continue;
    }
    run_sum<HF32>(a, b, e, h, acc);
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] *= a.scale;
    if constexpr (ACC) {
      float old[8];
      load8<GF32>(a.out, v * a.H + h, old);
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[c] += old[c];
    }
    store8<GF32>(a.out, v * a.H + h, acc);
  }
}

// Columns of a weight gradient [H,Vs]: a block takes a strip of 64 columns and
// 128 hidden values, sums the strip's runs to an LDS tile (16 lanes a run, 8
// values each) and writes the tile's rows, 128 (bf16) or 256 bytes each. VEC:
// rows start 16-byte aligned (Vs a multiple of 8), eight columns a thread;
// otherwise one column a thread.
constexpr int kStrip = 64;
constexpr int kStripH = 128;

template <bool HF32, bool GF32, bool ACC, bool VEC>
__global__ void __launch_bounds__(256) embed_grad_cols_kernel(GradArgs a) {
  __shared__ float tile[kStripH][kStrip + 1];
  __shared__ int32_t st[kStrip + 1];
  const int tid = threadIdx.x;
  const int64_t v0 = (int64_t)blockIdx.x * kStrip;
  const int64_t h0 = (int64_t)blockIdx.y * kStripH;
  const int nv = a.Vs - v0 < kStrip ? (int)(a.Vs - v0) : kStrip;
  const int nh = a.H - h0 < kStripH ? (int)(a.H - h0) : kStripH;
  if (tid <= kStrip) st[tid] = a.starts[v0 + (tid < nv ? tid : nv)];
  __syncthreads();
  const bool empty = st[0] == st[kStrip];
  if (empty && ACC) return;
  if (!empty) {
    const int hl = (tid & 15) * 8;
    for (int r = tid >> 4; r < kStrip; r += 16) {
      const int64_t b = st[r], e = st[r + 1];
      float acc[8];
      if (b < e && hl < nh) {
        run_sum<HF32>(a, b, e, h0 + hl, acc);
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] *= a.scale;
      } else {
        // Added to what is there, -0 changes nothing, the sign of a zero included.
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] = ACC ? -0.f : 0.f;
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) tile[hl + c][r] = acc[c];
    }
    __syncthreads();
  }
  if constexpr (VEC) {
    const int c0 = (tid & 7) * 8;
    if (c0 >= nv) return;
    for (int r = tid >> 3; r < nh; r += 32) {
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (!empty) {
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = tile[r][c0 + c];
      }
      const int64_t at = (h0 + r) * a.Vs + v0 + c0;
      if constexpr (ACC) {
        float old[8];
        load8<GF32>(a.out, at, old);
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] += old[c];
      }
      store8<GF32>(a.out, at, v);
    }
  } else {
    const int c = tid & 63;
    if (c >= nv) return;
    for (int r = tid >> 6; r < nh; r += 4) {
      float v = empty ? 0.f : tile[r][c];
      const int64_t at = (h0 + r) * a.Vs + v0 + c;
      if constexpr (GF32) {
        float* o = static_cast<float*>(a.out) + at;
        *o = ACC ? v + *o : v;
      } else {
        uint16_t* o = static_cast<uint16_t*>(a.out) + at;
        if constexpr (ACC) v += bf16_lo(*o);
        *o = (uint16_t)(bf16_pair(v, 0.f) & 0xFFFFu);
      }
    }
  }
}

}  // namespace flce
