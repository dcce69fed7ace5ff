// Host-only check of the operators' planner (flce_ops_plan.hpp): over a sweep of
// sizes up to the library's limits, every workspace region is 256-byte aligned and
// inside the total, regions follow one another without overlap, the sort's digits
// cover every key, and the losses' blocks cover every sequence. Built with
// AddressSanitizer and UndefinedBehaviorSanitizer by tests/test_plan_sanitizers_ops.py.
#include <cstdio>
#include <cstdlib>

#include "flce_ops_plan.hpp"

using namespace flce;

static int failures = 0;
#define CHECK(cond)                                                  \
  do {                                                               \
    if (!(cond)) {                                                   \
      std::fprintf(stderr, "FAIL line %d: %s\n", __LINE__, #cond);   \
      if (++failures > 20) std::exit(1);                             \
    }                                                                \
  } while (0)

static void check_embed(int64_t N, int64_t H, int64_t V, int layout) {
  const EmbedPlan p = make_embed_plan(N, H, V, layout);
  const SortPlan& s = p.sort;
  CHECK(s.passes >= 1 && s.bits >= 1 && s.bits <= kMaxDigitBits && s.passes * s.bits <= 32);
  CHECK(((int64_t)1 << (s.passes * s.bits)) > V);  // the keys 0 .. V
  CHECK(s.by_rank == (N <= kRankTokens));
  CHECK(s.tiles * kSortTile >= N && s.pitch >= s.tiles && s.pitch % 4 == 0);
  size_t end = kHeaderBytes;
  auto region = [&](size_t off, size_t bytes) {
    CHECK(off % kAlign == 0);
    CHECK(off >= end);
    CHECK(off + bytes >= off);
    end = off + bytes;
  };
  region(p.key, 4 * (size_t)N);
  region(p.perm, 4 * (size_t)N);
  if (!s.by_rank) {
    region(p.key2, 4 * (size_t)N);
    region(p.perm2, 4 * (size_t)N);
    region(p.counts, 4 * ((size_t)s.pitch << s.bits));
    region(p.totals, (size_t)4 << s.bits);
  }
  CHECK(p.sorted ? end <= p.f_total : p.f_total == kHeaderBytes);
  region(p.strips, 4 * ((size_t)((V + kStrip - 1) / kStrip) + 1));
  region(p.part, 8 * (size_t)((N + kPiece - 1) / kPiece) * (size_t)H);
  CHECK(p.large_pieces * kPieces2 * kPiece <= N);
  CHECK(s.by_rank ? p.large_pieces == 0
                  : (p.large_pieces + 1) * kPieces2 * kPiece > N);
  region(p.part2, 4 * (size_t)p.large_pieces * (size_t)H);
  CHECK(end <= p.b_total);
}

static void check_loss(const LossPlan& p, int64_t N, int64_t B, int64_t items, size_t share,
                       size_t total, int64_t state) {
  CHECK(p.rows == 1 || p.rows == kLossRows);
  CHECK(p.tiles * 64 * p.rows >= N);
  CHECK(p.seq_items >= 1 && p.seq_blocks >= 1 && p.seq_blocks <= kMaxSeqBlocks);
  CHECK(p.seq_blocks * p.seq_items >= items && (p.seq_blocks - 1) * p.seq_items < items);
  CHECK(!p.small || (N <= kSmallTokens && B <= kSmallSequences && p.rows == 1 &&
                     p.tiles <= kSmallTokens / 64));
  size_t end = kHeaderBytes;
  auto region = [&](size_t off, size_t bytes) {
    CHECK(off % kAlign == 0);
    CHECK(off >= end);
    end = off + bytes;
  };
  region(p.parts, share * (size_t)(B + p.tiles));
  region(p.seq_sum, share * (size_t)B);
  region(p.totals, total * (size_t)p.seq_blocks);
  region(p.state, 8 * (size_t)state);
  CHECK(end <= p.total);
}

int main() {
  const int64_t ns[] = {0, 1, 31, 32, 33, 300, 511, 2047, 2048, 4096, 4097, 8192, 16384, 16385,
                        20000, 262144, 262145, 1000003, kMaxN};
  const int64_t vs[] = {1, 2, 63, 64, 65, 127, 128, 511, 512, 1001, 32000, 131071, 131072, 256000,
                        (1 << 21) + 5, kMaxV};
  const int64_t hs[] = {8, 64, 520, 4096, kMaxH};
  for (int64_t N : ns)
    for (int64_t V : vs)
      for (int64_t H : hs)
        for (int layout = FLCE_EMBED_VH; layout <= FLCE_EMBED_HV; ++layout)
          check_embed(N, H, V, layout);
  const int64_t bs[] = {1, 2, 3, 17, 64, 65, 1000, 1023, 1024, 1025, 4096, 70000, 1 << 20,
                        kMaxSequences};
  for (int64_t N : ns)
    for (int64_t B : bs) {
      check_loss(policy_plan(N, B), N, B, B, sum_bytes(4), sum_bytes(5), 2 * (B + 1));
      if (B <= kMaxSequences / 2)
        check_loss(preference_plan(N, B), N, 2 * B, B, sum_bytes(1), sum_bytes(1), 2 * B + 1);
    }
  std::printf("failures: %d\n", failures);
  return failures != 0;
}
