// Host-only check of where the processing of logits counts a token (flce_step_plan.hpp):
// over vocabularies on both sides of every border of a slice and of half a slice, each
// id is counted once, at a place inside the block's LDS, also where a long history is
// counted in two parts and the last slice ends within the first one, and no other int64
// is counted at all. Built with AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/test_process_places.py.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "flce_step_plan.hpp"

using namespace flce;

static int failures = 0;
#define CHECK(cond)                                                            \
  do {                                                                         \
    if (!(cond)) {                                                             \
      std::fprintf(stderr, "FAIL line %d: %s\n", __LINE__, #cond);             \
      if (++failures > 20) std::exit(1);                                       \
    }                                                                          \
  } while (0)

// The places that a token gets over all slices and parts; 16-bit counts lie two a word.
static int places(int64_t token, int64_t V, int slice, int hist, bool wide) {
  const int words = proc_count_words(hist, slice);
  CHECK(words <= proc_lds_words(hist, true, slice) && words % 4 == 0);
  int found = 0;
  for (int64_t lo = 0; lo < V; lo += slice) {
    const int n = (int)(V - lo < slice ? V - lo : slice);
    const int part = wide ? slice / 2 : slice;
    for (int from = 0; from < slice; from += part) {
      const uint32_t ids = wide ? proc_part(n, from, part) : (uint32_t)n;
      CHECK(ids <= (uint32_t)part && (from > 0 || ids > 0));
      const uint64_t x = proc_place(token, lo + from);
      if (x >= ids) continue;
      const int d = (int)x, word = hist == HIST_SEEN ? d >> 5 : (wide ? d : d >> 1);
      CHECK(word < words && lo + from + d == token);
      ++found;
    }
  }
  return found;
}

static void check_vocabulary(int64_t V, int slice) {
  const int64_t others[] = {-1, -100, V, V + 1, V + 20, V + slice / 2, V + slice, V + 2 * slice,
                            (int64_t)1 << 31, (int64_t)1 << 32, ((int64_t)1 << 32) + 3,
                            (int64_t)1 << 40, -((int64_t)1 << 32), -((int64_t)1 << 40), INT64_MIN,
                            INT64_MIN + V, INT64_MIN + slice, INT64_MAX, INT64_MAX - 1};
  for (int hist : {(int)HIST_SEEN, (int)HIST_COUNT})
    for (bool wide : {false, true}) {
      if (wide && hist != HIST_COUNT) continue;
      for (int64_t t : others) CHECK(places(t, V, slice, hist, wide) == 0);
      for (int64_t t = 0; t < V; t += t < 5000 || V - t < 5000 ? 1 : 997)
        CHECK(places(t, V, slice, hist, wide) == 1);
    }
  // Every id is taken from the part that counted it: eight a thread, from the first of a
  // step on, and never past the counts.
  std::vector<int> read(V < 20000 ? V : 0);
  for (int64_t lo = 0; lo < (int64_t)read.size(); lo += slice) {
    const int n = (int)(V - lo < slice ? V - lo : slice);
    for (int from = 0; from < slice; from += slice / 2) {
      const int ids = (int)proc_part(n, from, slice / 2);
      for (int at = 0; at < slice; at += 8) {
        const int v = at - from;
        if (v < 0 || v >= ids) continue;
        CHECK(v + 8 <= slice / 2);
        for (int k = 0; k < 8 && at + k < n; ++k) ++read[lo + at + k];
      }
    }
  }
  for (int r : read) CHECK(r == 1);
}

int main() {
  // A part behind the slice's end has no ids.
  for (int part : {kProcStep / 2, kProcStep})
    for (int n : {1, 2, 1000, part - 1, part}) CHECK(proc_part(n, part, part) == 0);
  for (int steps = 1; steps <= kProcSteps; ++steps) {
    const int slice = steps * kProcStep;
    for (int64_t V : {1, 2, 7, 8, 9, 1000, 1023, 1024, 1025, 1500, 2047, 2048, 2049, 3001, 4095,
                      4096, 4097, 5119, 5120, 5121, 6143, 6145, 10239, 10241, 50257, 128256,
                      152064})
      check_vocabulary(V, slice);
    check_vocabulary(kMaxV, slice);
  }
  std::printf("failures: %d\n", failures);
  return failures != 0;
}
