// Host planner of the embedding and loss operators: limits, argument checks
// and workspace layouts. Host-only C++ without HIP, so that it also builds on
// its own for sanitizer checks of the layout arithmetic.
#pragma once

#include <cmath>
#include <cstddef>
#include <cstdint>

#include "flce.h"
#include "flce_plan.hpp"

// Also called in kernels.
#ifdef __HIPCC__
#define FLCE_HD __host__ __device__
#else
#define FLCE_HD
#endif

namespace flce {

// ---- losses ----------------------------------------------------------------------

constexpr int kLossTile = 256;        // tokens a wave takes at most
constexpr int kLossRows = kLossTile / 64;
constexpr int kLossWaves = 4;         // waves a block, parts and gradients kernels
constexpr int kSmallWaves = 16;       // waves of the one-block kernel
constexpr int kSeqThreads = 1024;     // threads a block, sequences kernel
constexpr int64_t kMaxSeqBlocks = 512;
// Batches up to these sizes take the one-block kernel, at most two rounds of its 16
// waves. Policy loss with gradients, kernels back to back: 512 tokens 7.8 us against
// 11.2 in three launches, 1024 9.5 against 11.7; by itself, as such batches mostly
// run, each launch has 3 to 5 us more (cold caches) and 2.5 us on the host. With
// more tokens or sequences one block is too slow: 4000 tokens 33 us against 14.
constexpr int64_t kSmallTokens = 2048;
constexpr int64_t kSmallSequences = 256;
constexpr int64_t kMaxSequences = (int64_t)1 << 21;

// Workspace: header, shares [B + tiles], sequence sums [B], block totals, and
// the state of the calls that return gradients at once.
struct LossPlan {
  int rows;             // rows of 64 tokens a tile
  int64_t tiles;
  int64_t seq_items;    // items a block of the sequences kernel takes
  int seq_blocks;
  bool small;
  size_t parts, seq_sum, totals, state, total;
};

// Lanes that add up one sequence's shares: its average number of shares, as a
// power of two up to a wave.
FLCE_HD inline int lanes_per_sequence(int64_t B, int64_t tiles) {
  int g = 1;
  while (g < 64 && g * B < tiles) g <<= 1;
  return g;
}

// Rows a tile: one while that gives the GPU's 1024 SIMDs four waves or fewer each,
// so that a wave's chain of dependent loads is short; then kLossRows, for fewer
// shares and more loads in flight a wave.
inline int loss_rows(int64_t N) { return ceil_div(N, 64) <= 4096 ? 1 : kLossRows; }

inline LossPlan make_loss_plan(int64_t N, int64_t B, int64_t items, size_t share_bytes,
                               size_t total_bytes, int64_t state_doubles) {
  LossPlan p{};
  p.small = N <= kSmallTokens && B <= kSmallSequences;
  p.rows = loss_rows(N);
  p.tiles = ceil_div(N, 64 * p.rows);
  // One round of a block's lane groups, or more when that makes too many blocks.
  const int64_t round = kSeqThreads / lanes_per_sequence(B, p.tiles) / (B / items);
  p.seq_items = round * ceil_div(ceil_div(items, round), kMaxSeqBlocks);
  p.seq_blocks = (int)ceil_div(items, p.seq_items);
  size_t off = kHeaderBytes;
  auto take = [&](size_t& field, size_t bytes) {
    field = off;
    off = align_up(off + bytes);
  };
  take(p.parts, share_bytes * (size_t)(B + p.tiles));
  take(p.seq_sum, share_bytes * (size_t)B);
  take(p.totals, total_bytes * (size_t)p.seq_blocks);
  take(p.state, 8 * (size_t)state_doubles);
  p.total = off;
  return p;
}

// Bytes of the kernels' sums: K doubles and four counts (checked where the
// kernels' types are known).
constexpr size_t sum_bytes(int k) { return 8 * (size_t)k + 16; }

inline LossPlan policy_plan(int64_t N, int64_t B) {
  return make_loss_plan(N, B, B, sum_bytes(4), sum_bytes(5), 2 * (B + 1));
}
inline LossPlan preference_plan(int64_t N, int64_t P) {
  return make_loss_plan(N, 2 * P, P, sum_bytes(1), sum_bytes(1), 2 * P + 1);
}

inline flce_status_t check_policy(int64_t N, int64_t B, int64_t V, bool has_cu,
                                  const flce_policy_options_t* o) {
  if (N < 0 || N > kMaxN || B < 1 || B > kMaxSequences || V < 1 || V > kMaxV)
    return FLCE_ERR_BAD_SHAPE;
  if (!has_cu && B != 1) return FLCE_ERR_BAD_SHAPE;
  if (o == nullptr) return FLCE_ERR_NULL_POINTER;
  if (o->reduction != FLCE_REDUCTION_MEAN && o->reduction != FLCE_REDUCTION_SUM &&
      o->reduction != FLCE_REDUCTION_SEQUENCE_MEAN)
    return FLCE_ERR_BAD_REDUCTION;
  if (!(o->clip_low >= 0.0 && o->clip_low <= 1.0)) return FLCE_ERR_BAD_OPTION;
  if (!(o->clip_high >= 0.0 && std::isfinite(o->clip_high))) return FLCE_ERR_BAD_OPTION;
  if (!(o->dual_clip == 0.0 || (o->dual_clip > 1.0 && std::isfinite(o->dual_clip))))
    return FLCE_ERR_BAD_OPTION;
  if (!std::isfinite(o->kl_coef) || !std::isfinite(o->entropy_coef)) return FLCE_ERR_BAD_OPTION;
  if (o->kl_estimator < FLCE_KL_K1 || o->kl_estimator > FLCE_KL_K3) return FLCE_ERR_BAD_OPTION;
  if (o->level != FLCE_RATIO_TOKEN && o->level != FLCE_RATIO_SEQUENCE) return FLCE_ERR_BAD_OPTION;
  if (o->advantages_per_sequence != 0 && o->advantages_per_sequence != 1)
    return FLCE_ERR_BAD_OPTION;
  if (o->level == FLCE_RATIO_SEQUENCE && (!has_cu || o->advantages_per_sequence != 1))
    return FLCE_ERR_BAD_OPTION;
  return FLCE_OK;
}

inline flce_status_t check_preference(int64_t N, int64_t P, int64_t V,
                                      const flce_preference_options_t* o) {
  if (N < 0 || N > kMaxN || P < 1 || P > kMaxSequences / 2 || V < 1 || V > kMaxV)
    return FLCE_ERR_BAD_SHAPE;
  if (o == nullptr) return FLCE_ERR_NULL_POINTER;
  if (!valid_reduction(o->reduction)) return FLCE_ERR_BAD_REDUCTION;
  if (!(o->beta > 0.0 && std::isfinite(o->beta)) || !std::isfinite(o->margin))
    return FLCE_ERR_BAD_OPTION;
  if (!(o->label_smoothing >= 0.0 && o->label_smoothing <= 0.5)) return FLCE_ERR_BAD_OPTION;
  if (o->kind < FLCE_PREFERENCE_SIGMOID || o->kind > FLCE_PREFERENCE_IPO)
    return FLCE_ERR_BAD_OPTION;
  if (o->kind != FLCE_PREFERENCE_SIGMOID && o->label_smoothing != 0.0) return FLCE_ERR_BAD_OPTION;
  if (o->kind == FLCE_PREFERENCE_IPO && o->margin != 0.0) return FLCE_ERR_BAD_OPTION;
  if (o->length_normalize != 0 && o->length_normalize != 1) return FLCE_ERR_BAD_OPTION;
  return FLCE_OK;
}

inline bool aligned_to(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// ---- embedding --------------------------------------------------------------------

constexpr int kPiece = 32;                    // sorted positions a piece; longer runs are split
// Batches sorted by digits sum this many consecutive pieces of one run once more
// (a launch of 4 us; a run of 10 % of 2^21 tokens has 6500 pieces).
constexpr int kPieces2 = 32;
constexpr int kStrip = 64;                    // rows (ids) a block of the gradient takes
constexpr int64_t kRankTokens = 16384;        // tokens sorted by counting every place
constexpr int kSortTile = 1024;               // tokens a block of the larger sort takes
constexpr int kMaxDigitBits = 11;

// The sort: keys are the token's row in the slice, or Vs for a token that takes
// no part, so that these come last.
struct SortPlan {
  int passes, bits;     // digit passes of `bits` bits each
  int64_t tiles, pitch; // blocks of the larger sort, and their counts' row length
  bool by_rank;
};
inline SortPlan make_sort_plan(int64_t N, int64_t Vs) {
  SortPlan s{};
  int total = 1;
  while (((int64_t)1 << total) <= Vs) ++total;  // the keys 0 .. Vs
  s.by_rank = N <= kRankTokens;
  s.passes = (total + kMaxDigitBits - 1) / kMaxDigitBits;
  s.bits = (total + s.passes - 1) / s.passes;
  s.tiles = ceil_div(N, kSortTile);
  s.pitch = ceil_div(s.tiles, 4) * 4;
  return s;
}

struct EmbedPlan {
  SortPlan sort;
  bool sorted;          // the forward gathers in sorted order
  size_t key, perm, key2, perm2, counts, totals;  // sort
  size_t strips;        // backward: first sorted position of every strip, [strips + 1]
  size_t part;          // backward: sums of split runs, [2 * pieces, H] fp32
  int64_t large_pieces; // and of whole groups of kPieces2 pieces, [large_pieces, H]
  size_t part2;
  size_t f_total, b_total;
};

// Lookups from a table of up to this many tokens, or of rows this long, count the
// invalid tokens in one block: it takes 0.8 ns a token, the copy 1.6 ns or more a
// token from this row length on.
constexpr int64_t kCountBlockTokens = 8192;
constexpr int64_t kCountBlockHidden = 2048;
// Lookups of fewer tokens from an [H,V] weight gather in token order: a sort and a
// sorted gather of 2048 tokens took 37 us (frequent ids) and 102 us (all different)
// at H = 2304, V = 256000, the gather alone 34 and 104; of 4096, 61 and 165 against
// 63 and 201; of 1024, 19 and 59 against 17 and 55.
constexpr int64_t kGatherSorted = 2048;

inline EmbedPlan make_embed_plan(int64_t N, int64_t H, int64_t Vs, int layout) {
  EmbedPlan p{};
  p.sort = make_sort_plan(N, Vs);
  p.sorted = layout == FLCE_EMBED_HV && N >= kGatherSorted;
  size_t off = kHeaderBytes;
  auto take = [&](size_t& field, size_t bytes) {
    field = off;
    off = align_up(off + bytes);
  };
  take(p.key, 4 * (size_t)N);
  take(p.perm, 4 * (size_t)N);
  if (!p.sort.by_rank) {
    take(p.key2, 4 * (size_t)N);
    take(p.perm2, 4 * (size_t)N);
    take(p.counts, 4 * ((size_t)p.sort.pitch << p.sort.bits));
    take(p.totals, (size_t)4 << p.sort.bits);
  }
  p.f_total = p.sorted ? off : kHeaderBytes;
  take(p.strips, 4 * ((size_t)ceil_div(Vs, kStrip) + 1));
  take(p.part, 4 * 2 * (size_t)ceil_div(N, kPiece) * (size_t)H);
  p.large_pieces = p.sort.by_rank ? 0 : N / (kPiece * kPieces2);
  take(p.part2, 4 * (size_t)p.large_pieces * (size_t)H);
  p.b_total = off;
  return p;
}

inline flce_status_t check_embedding(int64_t N, int64_t H, int64_t Vs, int64_t v_begin,
                                     int64_t V_total, const flce_embedding_options_t* o) {
  const flce_status_t s = check_shape(N, H, Vs);
  if (s != FLCE_OK) return s;
  if (V_total < 1 || V_total > kMaxV || v_begin < 0 || Vs > V_total ||
      v_begin > V_total - Vs)
    return FLCE_ERR_BAD_SHAPE;
  if (o == nullptr) return FLCE_ERR_NULL_POINTER;
  if (!std::isfinite(o->scale) || !std::isfinite((float)o->scale)) return FLCE_ERR_BAD_OPTION;
  if (o->layout != FLCE_EMBED_VH && o->layout != FLCE_EMBED_HV) return FLCE_ERR_BAD_OPTION;
  if (o->hidden_dtype != FLCE_GRAD_BF16 && o->hidden_dtype != FLCE_GRAD_F32)
    return FLCE_ERR_BAD_OPTION;
  if (o->grad_dtype != FLCE_GRAD_BF16 && o->grad_dtype != FLCE_GRAD_F32)
    return FLCE_ERR_BAD_OPTION;
  if (o->accumulate != 0 && o->accumulate != 1) return FLCE_ERR_BAD_OPTION;
  return FLCE_OK;
}

}  // namespace flce
