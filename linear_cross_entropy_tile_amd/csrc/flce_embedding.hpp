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
// goes out), so 2 rows a piece hold them. In large batches the sums of kPieces2
// consecutive pieces inside one run are added up once more.
//
// What bounds them: the bytes (a table's lookup its output and the distinct rows, a
// weight's the cache lines of its columns, the gradient the write of all of dE),
// and for small batches the launches. The figures at the kernels are an MI355X's, on
// which a large copy reaches 5.1 TB/s and a fill 6.8.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "flce_ops_plan.hpp"
#include "flce_vector.hpp"

namespace flce {

// W = 4 or 8 consecutive values of an array of bf16 or fp32, aligned to their
// bytes or to 16.
template <bool F32, int W>
__device__ __forceinline__ void load_w(const void* p, int64_t i, float (&v)[W]) {
  if constexpr (F32) {
    const ef32x4* q = reinterpret_cast<const ef32x4*>(static_cast<const float*>(p) + i);
#pragma unroll
    for (int j = 0; j < W / 4; ++j) {
      const ef32x4 x = q[j];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[4 * j + k] = x[k];
    }
  } else {
    typedef uint32_t words __attribute__((ext_vector_type(W / 2)));
    const words x = *reinterpret_cast<const words*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int j = 0; j < W / 2; ++j) {
      v[2 * j] = bf16_lo(x[j]);
      v[2 * j + 1] = bf16_hi(x[j]);
    }
  }
}
// Outputs are streamed past the caches (nontemporal): they are larger than the
// caches and would push out the inputs. A lookup of 32768 rows of 4096 values took
// 77 us without and takes 54 us; an fp32 gradient of [32000, 4096] 125 and 107 us.
template <class T>
__device__ __forceinline__ void stream(T* p, const T& v) {
  __builtin_nontemporal_store(v, p);
}
template <bool F32, int W>
__device__ __forceinline__ void store_w(void* p, int64_t i, const float (&v)[W]) {
  if constexpr (F32) {
    ef32x4* q = reinterpret_cast<ef32x4*>(static_cast<float*>(p) + i);
#pragma unroll
    for (int j = 0; j < W / 4; ++j)
      stream(q + j, ef32x4{v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]});
  } else {
    typedef uint32_t words __attribute__((ext_vector_type(W / 2)));
    words x;
#pragma unroll
    for (int j = 0; j < W / 2; ++j) x[j] = bf16_pair(v[2 * j], v[2 * j + 1]);
    stream(reinterpret_cast<words*>(static_cast<uint16_t*>(p) + i), x);
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

// One block: the header's count of invalid tokens.
__device__ __forceinline__ void count_tokens(const TokenArgs& a, int* sh) {
  int inv = 0;
  for (int64_t i0 = threadIdx.x; i0 < a.N; i0 += 8 * blockDim.x) {
    int64_t x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t i = i0 + (int64_t)j * blockDim.x;
      x[j] = i < a.N ? a.tokens[i] : a.ignore_index;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      bool bad;
      (void)token_key(a, x[j], bad);
      inv += bad ? 1 : 0;
    }
  }
  inv = block_sum_int(inv, sh);
  if (threadIdx.x == 0) a.header[0] = inv;
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

// Up to kRankTokens tokens: every item's place is counted, N compares an item
// spread over the whole GPU, in one launch and without a dependence on any other
// item's place. 32 items a block; thread (part, item) compares the item with every
// 32nd group of 32 keys, four keys a (broadcast) LDS read. Equal keys keep their
// order: earlier groups count keys <= the item's, later ones keys < it, and the
// item's own group goes by the position. Keys stay below 2^23, so x < t is the sign
// of x - t: three VALU operations a compare, no condition codes (whose hazards cost
// as much again). 8192 tokens take 11 us, 300 take 3.8 (one block sorting in LDS by
// digits: 39 and 6.9); 16384 take 28, seven launches of the larger sort 40.
constexpr int kRankItems = 32;
constexpr int kRankThreads = 1024;

// -1 if x < t, else 0.
__device__ __forceinline__ int minus_less(uint32_t x, uint32_t t) {
  return (int)(x - t) >> 31;
}

__global__ void __launch_bounds__(kRankThreads) embed_rank_kernel(TokenArgs a, int32_t* key_out,
                                                                  int32_t* perm_out) {
  extern __shared__ uint32_t keys[];  // N, rounded up to groups
  __shared__ int count[kRankItems];
  __shared__ int sh[kRankThreads / 64];
  const int tid = threadIdx.x;
  const int N = (int)a.N, groups = (N + kRankItems - 1) / kRankItems;
  int inv = 0, n = 0;
  for (int i = tid; i < groups * kRankItems; i += kRankThreads) {
    uint32_t k = 1u << 24;  // past the end: above every bound
    if (i < N) {
      bool bad;
      k = (uint32_t)token_key(a, a.tokens[i], bad);
      n += k < (uint32_t)a.Vs ? 1 : 0;
      inv += bad ? 1 : 0;
    }
    keys[i] = k;
  }
  if (tid < kRankItems) count[tid] = 0;
  if (blockIdx.x == 0) {
    inv = block_sum_int(inv, sh);
    n = block_sum_int(n, sh);
    if (tid == 0) {
      a.header[0] = inv;
      a.header[1] = n;
    }
  }
  __syncthreads();
  const int item = tid & (kRankItems - 1), part = tid / kRankItems;
  const int own = (int)blockIdx.x;  // the block's group of items
  if (own >= groups) return;        // no tokens at all
  const uint32_t k = keys[own * kRankItems + item];
  int c = 0;
  for (int g = part; g < groups; g += kRankThreads / kRankItems) {
    const eu32x4* q = reinterpret_cast<const eu32x4*>(keys + g * kRankItems);
    const uint32_t t = g < own ? k + 1 : k;
    const int tie = g == own ? item : 0;  // own group: equal keys before the item count too
#pragma unroll
    for (int j = 0; j < kRankItems / 4; ++j) {
      const eu32x4 x = q[j];
      c += minus_less(x[0], t) + minus_less(x[1], t);
      c += minus_less(x[2], t) + minus_less(x[3], t);
    }
    for (int e = 0; e < tie; ++e) c -= keys[g * kRankItems + e] == k ? 1 : 0;
  }
  atomicAdd(&count[item], -c);  // of whole numbers: the order does not matter
  __syncthreads();
  const int i = own * kRankItems + item;
  if (tid >= kRankItems || i >= N) return;
  key_out[count[item]] = (int32_t)k;
  perm_out[count[item]] = i;
}

// The larger sort, a pass: digit counts of every tile of kSortTile items, the
// counts' prefix over the tiles (a wave a digit), and the move. Pass 0 reads the
// tokens, later ones the previous pass's keys.
struct SortArgs {
  TokenArgs t;
  const int32_t *key_in, *perm_in;  // null: from the tokens
  int32_t *key_out, *perm_out;
  int32_t* counts;                  // [digit][tile], rows `pitch` apart
  int64_t pitch;
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
  for (int d = threadIdx.x; d < nd; d += 256) a.counts[d * a.pitch + blockIdx.x] = hist[d];
  if (a.key_in == nullptr) {
    inv = block_sum_int(inv, sh);
    n = block_sum_int(n, sh);
    if (threadIdx.x == 0) {
      if (inv != 0) atomicAdd(&a.t.header[0], inv);
      if (n != 0) atomicAdd(&a.t.header[1], n);
    }
  }
}

// A wave a digit, four tiles a lane: counts[d][*] becomes its exclusive prefix over
// the tiles, the digit's total goes to totals[d]. Rows are padded to four tiles.
__global__ void __launch_bounds__(256) embed_sort_scan_kernel(int32_t* counts, int64_t tiles,
                                                              int64_t pitch, int nd,
                                                              int32_t* totals) {
  typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
  const int lane = threadIdx.x & 63;
  const int d = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (d >= nd) return;
  int run = 0;
  for (int64_t t0 = 0; t0 < tiles; t0 += 256) {
    const int64_t t = t0 + lane * 4;
    i32x4* c = reinterpret_cast<i32x4*>(counts + d * pitch + t);
    i32x4 v = {0, 0, 0, 0};
    if (t < tiles) v = *c;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = t + k < tiles ? v[k] : 0;
    const int sum = v[0] + v[1] + v[2] + v[3];
    int x = sum;
    for (int s = 1; s < 64; s <<= 1) {
      const int y = __shfl_up(x, s, 64);
      if (lane >= s) x += y;
    }
    const int before = run + x - sum;
    if (t < tiles)
      *c = i32x4{before, before + v[0], before + v[0] + v[1], before + v[0] + v[1] + v[2]};
    run += __shfl(x, 63, 64);
  }
  if (lane == 0) totals[d] = run;
}

__global__ void __launch_bounds__(64 * kSortMoveWaves)
embed_sort_move_kernel(SortArgs a, const int32_t* totals) {
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
    if (d < nd) base[d] = off + a.counts[d * a.pitch + blockIdx.x];
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
  int count_block;            // 1: one more block counts the invalid tokens
  int lanes;                  // lanes a row (table lookup): a power of two, 8 to 64
};

// Rows of a table [Vs,H], eight values a lane. Wide rows: a wave takes a row and a
// chunk of kGatherLoads * 512 of its values, all loads in flight before the first
// store. Narrow ones (lanes < 64): a wave takes 64 / lanes rows at a time. 32768
// tokens of 5120 values (419 MB) take 90 us, 4.6 TB/s. Of 2, 4, 5, 8 and 10 loads five
// is within 2.5 % of the best at every row length tried (the same 32768 tokens again
// and again, rows of 2304, 4096, 5120 and 7168 values: 32.0, 55.2, 69.3 and 94.8 us);
// two lose 5 % at 2304 and 4096, ten 2.5 to 5 % at 5120 and 7168.
constexpr int kGatherLoads = 5;

__device__ __forceinline__ eu32x4 scaled8(const eu32x4& w, float scale) {
  if (scale == 1.f) return w;
  float v[8];
  unpack8(w, v);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] *= scale;
  return pack8(v);
}

__global__ void __launch_bounds__(256) embed_gather_rows_kernel(GatherArgs a) {
  __shared__ int sh[4];
  if (a.count_block != 0 && blockIdx.x == 0) {
    if (blockIdx.y == 0) count_tokens(a.t, sh);
    return;
  }
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int side = 64 / a.lanes;  // rows a wave takes side by side
  const int64_t i = ((int64_t)(blockIdx.x - a.count_block) * 4 + w) * side + lane / a.lanes;
  const int k = lane & (a.lanes - 1);
  bool bad = false;
  const bool on = i < a.t.N;
  const int32_t key = on ? token_key(a.t, a.t.tokens[i], bad) : (int32_t)a.t.Vs;
  if (a.count_block == 0 && blockIdx.y == 0) {
    // Invalid tokens only: an atomic a block on one address would take longer than
    // the copy.
    const uint64_t inv = __builtin_amdgcn_ballot_w64(k == 0 && bad);
    if (inv != 0 && lane == 0) atomicAdd(&a.t.header[0], __popcll(inv));
  }
  if (!on) return;
  const int64_t h0 = ((int64_t)blockIdx.y * kGatherLoads * a.lanes + k) * 8;
  const uint16_t* src = a.weight + (int64_t)key * a.H;
  uint16_t* dst = a.out + i * a.H;
  const float scale = key < a.t.Vs ? a.scale : 1.f;  // zero rows are +0 for every scale
  eu32x4 v[kGatherLoads];
#pragma unroll
  for (int j = 0; j < kGatherLoads; ++j) {
    const int64_t h = h0 + (int64_t)j * a.lanes * 8;
    v[j] = eu32x4{0u, 0u, 0u, 0u};
    if (key < a.t.Vs && h < a.H) v[j] = *reinterpret_cast<const eu32x4*>(src + h);
  }
#pragma unroll
  for (int j = 0; j < kGatherLoads; ++j) {
    const int64_t h = h0 + (int64_t)j * a.lanes * 8;
    if (h < a.H) stream(reinterpret_cast<eu32x4*>(dst + h), scaled8(v[j], scale));
  }
}

// Columns of a weight [H,Vs]: a wave takes 8 consecutive (sorted) tokens and 64
// hidden values; lane (t, g) gathers 8 values of token t down the rows 8 g .. and
// stores them as 16 bytes, 128 contiguous bytes a token. Bound by the lines: 8192
// tokens (2861 different, in 986 lines of each of 2304 rows, 291 MB) of 256000 take
// 82 us, all different (3800 lines, nearly the whole 1.18 GB) 218 us; a decoding
// step of 16 takes 3.3 us.
constexpr int kGatherTokens = 32;  // tokens a block

__global__ void __launch_bounds__(256) embed_gather_cols_kernel(GatherArgs a) {
  __shared__ int sh[4];
  if (a.count_block != 0 && blockIdx.x >= gridDim.x - 8) {
    if (blockIdx.x == gridDim.x - 8 && blockIdx.y == 0) count_tokens(a.t, sh);
    return;
  }
  const int lane = threadIdx.x & 63;
  // Blocks go to the 8 XCDs in turn, each with an L2 of its own. grid.x is a multiple
  // of 8, so a chunk of 64 rows of the weight stays with one XCD, and the tokens of
  // a line, neighbours in the sorted order, find it in that L2; a chunk's tokens run
  // one after another, within the same 64 rows' pages.
  const int64_t i0 = (int64_t)(blockIdx.x >> 3) * kGatherTokens;
  const int64_t i = i0 + (threadIdx.x >> 6) * 8 + (lane & 7);
  const int64_t h = ((int64_t)blockIdx.y * 8 + (blockIdx.x & 7)) * 64 + (lane >> 3) * 8;
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
  int32_t* strips;            // [strips + 1] first sorted position of every strip of 64 rows
  float* part;                // [2 * pieces][H]
  float* part2;               // [large pieces][H], or null
  int64_t N, H, Vs;
  float scale;
  void* out;
  int strip_blocks;           // blocks of the segments kernel that fill strips
  int chunks;                 // column chunks a piece
  int lanes;                  // lanes a row, eight values each: a power of two, 8 to 64
  int64_t range;              // hidden values a block takes
};

// acc += gradient rows of the sorted positions [b, e), in order. All `lanes` lanes of
// a group call it with the same range, lane k of them holding W columns from each of
// h[0 .. U); a lane reads one position's row number for the group at a time. DEEP
// rows are in flight at once.
template <bool HF32, int W, int U, int DEEP>
__device__ __forceinline__ void add_rows(const GradArgs& a, int64_t b, int64_t e, int lanes, int k,
                                         const int64_t (&h)[U], float (&acc)[U][W]) {
  const int first = (threadIdx.x & 63) - k;
  for (int64_t c = b; c < e; c += lanes) {
    const int32_t row = c + k < e ? a.perm[c + k] : 0;
    const int m = e - c < lanes ? (int)(e - c) : lanes;
    int j = 0;
    for (; j + DEEP <= m; j += DEEP) {
      float v[DEEP][U][W];
#pragma unroll
      for (int d = 0; d < DEEP; ++d) {
        const int64_t at = (int64_t)__shfl(row, first + j + d, 64) * a.H;
#pragma unroll
        for (int u = 0; u < U; ++u) load_w<HF32, W>(a.grad, at + h[u], v[d][u]);
      }
#pragma unroll
      for (int d = 0; d < DEEP; ++d)
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int q = 0; q < W; ++q) acc[u][q] += v[d][u][q];
    }
    for (; j < m; ++j) {
      const int64_t at = (int64_t)__shfl(row, first + j, 64) * a.H;
      float v[U][W];
#pragma unroll
      for (int u = 0; u < U; ++u) load_w<HF32, W>(a.grad, at + h[u], v[u]);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int q = 0; q < W; ++q) acc[u][q] += v[u][q];
    }
  }
}

// Whether the run [b, e) has a sum of the kPieces2 pieces from p on.
__device__ __forceinline__ bool large_piece(const GradArgs& a, int64_t p, int64_t b, int64_t e) {
  return a.part2 != nullptr && p % kPieces2 == 0 && p * kPiece >= b &&
         (p + kPieces2) * kPiece <= e;
}

// The sum of the run [b, e): directly, or from its pieces' sums.
template <bool HF32, int W, int U, int DEEP>
__device__ __forceinline__ void run_sum(const GradArgs& a, int64_t b, int64_t e, int lanes, int k,
                                        const int64_t (&h)[U], float (&acc)[U][W]) {
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int q = 0; q < W; ++q) acc[u][q] = 0.f;
  if (e - b <= kPiece) {
    add_rows<HF32, W, U, DEEP>(a, b, e, lanes, k, h, acc);
    return;
  }
  const int64_t p1 = (e - 1) / kPiece;
  int64_t p = b / kPiece;
  if (b > p * kPiece) {  // starts inside its first piece
#pragma unroll
    for (int u = 0; u < U; ++u) load_w<true, W>(a.part, (2 * p + 1) * a.H + h[u], acc[u]);
    ++p;
  }
  while (p <= p1) {
    // The next DEEP rows, large or small.
    float v[DEEP][U][W];
#pragma unroll
    for (int d = 0; d < DEEP; ++d) {
      if (p > p1) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int q = 0; q < W; ++q) v[d][u][q] = 0.f;
        continue;
      }
      const bool large = large_piece(a, p, b, e);
      const float* row = large ? a.part2 + p / kPieces2 * a.H : a.part + 2 * p * a.H;
#pragma unroll
      for (int u = 0; u < U; ++u) load_w<true, W>(row, h[u], v[d][u]);
      p += large ? kPieces2 : 1;
    }
#pragma unroll
    for (int d = 0; d < DEEP; ++d)
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int q = 0; q < W; ++q) acc[u][q] += v[d][u][q];
  }
}

__device__ __forceinline__ int64_t lower_bound(const int32_t* key, int64_t lo, int64_t hi,
                                               int64_t v) {
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (key[mid] < v)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ void store_part(const GradArgs& a, int64_t slot, int64_t h,
                                           const float (&v)[4]) {
  *reinterpret_cast<ef32x4*>(a.part + slot * a.H + h) = ef32x4{v[0], v[1], v[2], v[3]};
}

// First blocks: the strips. The others: one piece and column chunk each, summing the
// split runs that overlap it, 16 rows in flight. Bound by latency: 11 us for 8192
// tokens of 2304 values of which 3647 lie in split runs.
template <bool HF32>
__global__ void __launch_bounds__(256) embed_segments_kernel(GradArgs a) {
  const int64_t n = a.header[1];
  if ((int)blockIdx.x < a.strip_blocks) {
    const int64_t s = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t v = s * kStrip < a.Vs ? s * kStrip : a.Vs;
    if (s * kStrip < a.Vs + kStrip) a.strips[s] = (int32_t)lower_bound(a.key, 0, n, v);
    return;
  }
  const int64_t id = (int64_t)blockIdx.x - a.strip_blocks;
  const int64_t piece = id / a.chunks;
  const int64_t q0 = piece * kPiece;
  if (q0 >= n) return;
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
  const int64_t h = ((id % a.chunks) * blockDim.x + threadIdx.x) * 4;
  const bool on = h < a.H;           // the whole wave takes part in the row numbers' exchange
  const int64_t hc[1] = {on ? h : a.H - 4};
  if (split_first) {
    float acc[1][4] = {};
    add_rows<HF32, 4, 1, 16>(a, q0, q0 + head, 64, lane, hc, acc);
    if (on) store_part(a, 2 * piece, h, acc[0]);
  }
  if (split_last) {
    float acc[1][4] = {};
    add_rows<HF32, 4, 1, 16>(a, qe - tail, qe, 64, lane, hc, acc);
    if (on) store_part(a, 2 * piece + 1, h, acc[0]);
  }
}

// One large piece and column chunk a block, if it lies inside one run: the pieces'
// sums in order, 16 in flight.
__global__ void __launch_bounds__(256) embed_large_pieces_kernel(GradArgs a) {
  const int64_t n = a.header[1];
  const int64_t q = blockIdx.x / a.chunks, p0 = q * kPieces2;
  const int64_t b = p0 * kPiece, e = b + kPieces2 * kPiece;
  const int64_t h = ((int64_t)(blockIdx.x % a.chunks) * blockDim.x + threadIdx.x) * 4;
  if (e > n || a.key[b] != a.key[e - 1] || h >= a.H) return;
  float acc[4] = {};
#pragma unroll
  for (int c = 0; c < kPieces2; c += 16) {
    float v[16][4];
#pragma unroll
    for (int d = 0; d < 16; ++d) load_w<true, 4>(a.part, 2 * (p0 + c + d) * a.H + h, v[d]);
#pragma unroll
    for (int d = 0; d < 16; ++d)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[k] += v[d][k];
  }
  *reinterpret_cast<ef32x4*>(a.part2 + q * a.H + h) = ef32x4{acc[0], acc[1], acc[2], acc[3]};
}

// Rows of a table gradient [Vs,H]: a block takes kGradRows consecutive rows, whole
// or in column ranges, W values (16 bytes of output) a lane, so that what the GPU
// writes at a time is close together and every store instruction writes whole
// lines. Bound by the write: [32000, 4096] fp32 from 4096 tokens 101 us (5.5 TB/s),
// [256000, 2304] bf16 from 8192 tokens 215 us (5.6 TB/s); 64 rows a block 30 to 60 %
// more where frequent ids crowd into few blocks.
constexpr int kGradRows = 4;
constexpr int kGradSteps = 4;  // column steps in flight

template <bool HF32, bool GF32, bool ACC>
__global__ void __launch_bounds__(256) embed_grad_rows_kernel(GradArgs a) {
  constexpr int W = GF32 ? 4 : 8;
  __shared__ int32_t st[kGradRows + 1];
  const int64_t v0 = (int64_t)blockIdx.x * kGradRows;
  const int64_t b0 = a.strips[v0 / kStrip], e0 = a.strips[v0 / kStrip + 1];
  if (ACC && b0 == e0) return;
  if (b0 < e0) {
    if (threadIdx.x <= kGradRows)
      st[threadIdx.x] = (int32_t)lower_bound(a.key, b0, e0, v0 + threadIdx.x);
    __syncthreads();
  }
  const int nv = a.Vs - v0 < kGradRows ? (int)(a.Vs - v0) : kGradRows;
  const int k = threadIdx.x & (a.lanes - 1);
  const int64_t h0 = (int64_t)blockIdx.y * a.range;
  const int64_t h1 = h0 + a.range < a.H ? h0 + a.range : a.H;
  for (int r = threadIdx.x / a.lanes; r < nv; r += 256 / a.lanes) {
    const int64_t b = b0 < e0 ? st[r] : 0, e = b0 < e0 ? st[r + 1] : 0;
    if (b == e) {
      if constexpr (!ACC) {
        const float zero[W] = {};
        for (int64_t h = h0 + k * W; h < h1; h += a.lanes * W)
          store_w<GF32, W>(a.out, (v0 + r) * a.H + h, zero);
      }
      continue;
    }
    for (int64_t hs = h0; hs < h1; hs += a.lanes * W * kGradSteps) {
      int64_t h[kGradSteps];
      float acc[kGradSteps][W];
#pragma unroll
      for (int u = 0; u < kGradSteps; ++u) {
        h[u] = hs + ((int64_t)u * a.lanes + k) * W;
        if (h[u] >= h1) h[u] = h1 - W;  // the same values as the range's last lane
      }
      run_sum<HF32, W, kGradSteps, 2>(a, b, e, a.lanes, k, h, acc);
#pragma unroll
      for (int u = 0; u < kGradSteps; ++u) {
        if (hs + ((int64_t)u * a.lanes + k) * W >= h1) continue;
#pragma unroll
        for (int q = 0; q < W; ++q) acc[u][q] *= a.scale;
        const int64_t at = (v0 + r) * a.H + h[u];
        if constexpr (ACC) {
          float old[W];
          load_w<GF32, W>(a.out, at, old);
#pragma unroll
          for (int q = 0; q < W; ++q) acc[u][q] += old[q];
        }
        store_w<GF32, W>(a.out, at, acc[u]);
      }
    }
  }
}

// Columns of a weight gradient [H,Vs]: a block takes a strip of 64 columns and 128
// hidden values, sums the runs of the columns that have one to an LDS tile (16 lanes
// a run, 8 values each; the other columns stay as the tile was cleared) and writes
// the tile's rows, 128 (bf16) or 256 bytes each. Neighbouring strips run together,
// so that the GPU's writes of a row lie together; taking a strip's hidden values
// together instead, or 256 or 512 of them a block, was 3 to 30 % slower; strips of
// 128 columns and 64 hidden values were 6 % faster where few ids occur and 7 to 11 %
// slower where most do. Bound by the write: [2304, 256000] bf16 from 8192 tokens
// 232 us (5.2 TB/s; zeros alone in this pattern take 210 to 230).
// The tile holds what is stored, bf16 or fp32, so twice as many blocks fit where
// that is bf16; sums that are added to what is there stay fp32 until then. VEC:
// rows start 16-byte aligned (Vs a multiple of 8), 16 bytes of a row a thread;
// otherwise one column a thread. When added to what is there, columns without a run
// are not written, since another stream may be adding to them: a thread reads 16
// bytes and stores the values that have a run. Against writing all 64 columns of a
// strip, a call takes 242 us (251) for 8192 Zipf-distributed tokens into [2304, 256000]
// bf16 and 292 (357) into fp32, and 105 (86) and 113 (99) for 32768 tokens into [1024,
// 32000], where most columns have a run; the columns' stores gathered through LDS
// took 260, 308, 95 and 104.
constexpr int kStripH = 128;
static_assert(kStrip == 64, "a strip's columns are the bits of one word");

// One value of an array of bf16 or fp32.
template <bool F32>
__device__ __forceinline__ void store_one(void* p, int64_t i, float v) {
  if constexpr (F32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<uint16_t*>(p)[i] = (uint16_t)(bf16_pair(v, 0.f) & 0xFFFFu);
}

template <bool HF32, bool GF32, bool ACC, bool VEC>
__global__ void __launch_bounds__(256) embed_grad_cols_kernel(GradArgs a) {
  constexpr bool TF32 = GF32 || ACC;
  using T = std::conditional_t<TF32, float, uint16_t>;
  constexpr int kPitch = TF32 ? kStrip + 1 : kStrip + 2;
  __shared__ __attribute__((aligned(16))) T tile[kStripH * kPitch];
  __shared__ int32_t st[kStrip + 1];
  __shared__ uint8_t used[kStrip];
  const int tid = threadIdx.x;
  const int64_t v0 = (int64_t)blockIdx.x * kStrip;
  const int nv = a.Vs - v0 < kStrip ? (int)(a.Vs - v0) : kStrip;
  const int64_t b0 = a.strips[blockIdx.x], e0 = a.strips[blockIdx.x + 1];
  const bool any = b0 < e0;
  if (ACC && !any) return;
  int nu = 0;
  uint64_t cols = 0;  // the columns with a run
  if (any) {
    if (tid <= kStrip) st[tid] = (int32_t)lower_bound(a.key, b0, e0, v0 + tid);
    if constexpr (!ACC)
      for (int i = tid; i < kStripH * kPitch; i += 256) tile[i] = (T)0;
    __syncthreads();
    const int lane = tid & 63;
    cols = __builtin_amdgcn_ballot_w64(st[lane] < st[lane + 1]);
    if (tid < 64 && ((cols >> lane) & 1) != 0) used[lanes_below(cols)] = (uint8_t)lane;
    nu = __popcll(cols);
    __syncthreads();
  }
  const int64_t h0 = (int64_t)blockIdx.y * kStripH;
  const int nh = a.H - h0 < kStripH ? (int)(a.H - h0) : kStripH;
  if (any) {
    constexpr int kLanes = kStripH / 8;  // lanes a run
    const int k = tid % kLanes, hl = k * 8;
    for (int u = tid / kLanes; u < nu; u += 256 / kLanes) {
      const int r = used[u];
      const int64_t h[1] = {hl < nh ? h0 + hl : a.H - 8};
      float sum[1][8];
      run_sum<HF32, 8, 1, 4>(a, st[r], st[r + 1], kLanes, k, h, sum);
      float acc[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[c] = sum[0][c] * a.scale;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if constexpr (TF32)
          tile[(hl + c) * kPitch + r] = acc[c];
        else
          tile[(hl + c) * kPitch + r] = (uint16_t)(bf16_pair(acc[c], 0.f) & 0xFFFFu);
      }
    }
    __syncthreads();
  }
  if constexpr (VEC) {
    constexpr int W = GF32 ? 4 : 8, kPer = kStrip / W;  // values a thread, threads a row
    const int c0 = tid % kPer * W;
    const uint32_t all = (1u << W) - 1, mine = ACC ? (uint32_t)(cols >> c0) & all : all;
    if (c0 < nv && mine != 0) {
      for (int r = tid / kPer; r < nh; r += 256 / kPer) {
        const int64_t at = (h0 + r) * a.Vs + v0 + c0;
        if constexpr (TF32) {
          float v[W] = {};
          if (any) {
#pragma unroll
            for (int c = 0; c < W; ++c) v[c] = tile[r * kPitch + c0 + c];
          }
          if constexpr (ACC) {
            float old[W];
            load_w<GF32, W>(a.out, at, old);
#pragma unroll
            for (int c = 0; c < W; ++c) v[c] += old[c];
          }
          if (mine == all) {
            store_w<GF32, W>(a.out, at, v);
          } else {
#pragma unroll
            for (int c = 0; c < W; ++c)
              if (((mine >> c) & 1) != 0) store_one<GF32>(a.out, at + c, v[c]);
          }
        } else {
          eu32x4 v = eu32x4{0u, 0u, 0u, 0u};
          if (any) {
            const uint32_t* q = reinterpret_cast<const uint32_t*>(tile + r * kPitch + c0);
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] = q[c];
          }
          stream(reinterpret_cast<eu32x4*>(static_cast<uint16_t*>(a.out) + at), v);
        }
      }
    }
  } else {
    const int c = tid % kStrip;
    if (c < nv && (!ACC || ((cols >> c) & 1) != 0)) {
      for (int r = tid / kStrip; r < nh; r += 256 / kStrip) {
        const int64_t at = (h0 + r) * a.Vs + v0 + c;
        const T v = any ? tile[r * kPitch + c] : (T)0;
        if constexpr (ACC && GF32)
          static_cast<float*>(a.out)[at] += v;
        else if constexpr (ACC)
          store_one<false>(a.out, at, v + bf16_lo(static_cast<const uint16_t*>(a.out)[at]));
        else
          static_cast<T*>(a.out)[at] = v;
      }
    }
  }
}

}  // namespace flce
