// Host-only check of the planner of the operators at the ends of a training step
// (flce_step_plan.hpp): over a sweep of sizes up to the library's limits, the blocks
// cover the work, grids and LDS stay within the GPU's limits, and every workspace
// region is aligned and inside the total. Built with AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_step_abi.py.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "flce_step_plan.hpp"

using namespace flce;

static int failures = 0;
#define CHECK(cond)                                                  \
  do {                                                               \
    if (!(cond)) {                                                   \
      std::fprintf(stderr, "FAIL line %d: %s\n", __LINE__, #cond);   \
      if (++failures > 20) std::exit(1);                             \
    }                                                                \
  } while (0)

static void check_logits_plan(int64_t N, int64_t H, int64_t V) {
  const LogitsPlan p = make_logits_plan(N, H, V);
  CHECK(p.total >= kHeaderBytes && p.total % kAlign == 0);
  if (N == 0) return;
  if (p.wide > 0) {
    CHECK((p.wide == 2 || p.wide == 4) && V >= kLogitStrip && p.strips * kLogitStrip >= V);
    CHECK((int64_t)p.passes * p.wide * 64 >= N);
    CHECK((p.strips + 7) / 8 * 8 * p.passes * p.wide * 64 < ((int64_t)1 << 32));
    return;
  }
  if (p.mt == 0) {
    CHECK(V % 8 == 0);
    CHECK((int64_t)p.hkb * kBK >= H && (int64_t)p.vt * kTile >= V && (int64_t)p.tb * kTile >= N);
    CHECK(p.image >= kHeaderBytes && p.image % 16 == 0);
    CHECK(p.image + (size_t)p.tb * p.hkb * kBlockBytes <= p.total);
    CHECK((int64_t)p.vt * p.tb * 512 < ((int64_t)1 << 32));
    return;
  }
  CHECK(p.mt == 1 || p.mt == 2 || p.mt == 4);
  CHECK(p.waves == 4 || p.waves == 8 || (p.waves == 16 && p.mt == 1));
  CHECK(p.mt != 4 || p.waves == 4);
  CHECK((int64_t)p.passes * p.mt * 16 >= N && p.strips * kLogitStrip >= V);
  const int64_t steps = ceil_div(H, 32);
  CHECK(p.splits >= 1 && p.splits <= 65535 && (int64_t)p.splits * p.split_steps >= steps);
  CHECK((int64_t)(p.splits - 1) * p.split_steps < steps);
  CHECK((p.strips + 7) / 8 * 8 * p.passes * p.waves * 64 < ((int64_t)1 << 32));
  if (p.splits > 1)
    CHECK(p.parts % 16 == 0 && p.parts + 4 * (size_t)p.splits * N * V <= p.total);
}

static void check_proc_plan(int64_t N, int64_t V) {
  const ProcPlan p = make_proc_plan(N, V);
  CHECK(p.slices >= 1 && p.slices * p.slice >= V && (p.slices - 1) * p.slice < V);
  CHECK(p.slices <= kMaxGrid);
  // One of the kernel's slices.
  CHECK(p.slice == kProcStep || p.slice == kProcSteps * kProcStep);
  CHECK(p.parts % 16 == 0 && p.parts + 16 * (size_t)N * p.slices <= p.invalid);
  CHECK(p.invalid + 4 * (size_t)N <= p.total);
}

static void check_norm_plan(const std::vector<int64_t>& sizes) {
  NormPlan p;
  CHECK(make_norm_plan(sizes.data(), (int64_t)sizes.size(), &p) == FLCE_OK);
  int64_t blocks = 0;
  for (int64_t n : sizes) blocks += ceil_div(n, p.chunk);
  CHECK(p.chunk % kNormStep == 0 && p.blocks == blocks);
  CHECK(blocks <= 4096 + (int64_t)sizes.size() && blocks * kNormThreads < ((int64_t)1 << 32));
  CHECK(p.parts % 8 == 0 && p.parts + 8 * (size_t)blocks <= p.total);
}

int main() {
  const int64_t ns[] = {0, 1, 2, 15, 16, 17, 32, 33, 64, 65, 128, 256, 257, 1000, kMaxLogitRows};
  const int64_t vs[] = {1, 2, 7, 8, 9, 127, 128, 129, 1000, 1001, 2410, 32000, 50257, 131072,
                        256000, (1 << 21) + 5, kMaxV};
  const int64_t hs[] = {8, 24, 32, 64, 520, 1024, 2304, 4096, 5120, 65536, kMaxH};
  for (int64_t N : ns)
    for (int64_t V : vs)
      for (int64_t H : hs) check_logits_plan(N, H, V);
  const int64_t rows[] = {0, 1, 3, 64, 255, 512, 1000, 300000, kMaxN};
  for (int64_t N : rows)
    for (int64_t V : vs) check_proc_plan(N, V);
  check_norm_plan({});
  check_norm_plan({0});
  check_norm_plan({1, 4095, 4096, 4097, 0, 7});
  check_norm_plan({kMaxTensorSize, 5, kMaxTensorSize});
  check_norm_plan(std::vector<int64_t>(1000, 590000));
  check_norm_plan(std::vector<int64_t>(kMaxTensors, 1));
  NormPlan p;
  const int64_t bad[] = {-1}, large[] = {kMaxTensorSize + 1};
  CHECK(make_norm_plan(bad, 1, &p) == FLCE_ERR_BAD_SHAPE);
  CHECK(make_norm_plan(large, 1, &p) == FLCE_ERR_BAD_SHAPE);
  CHECK(make_norm_plan(nullptr, 1, &p) == FLCE_ERR_NULL_POINTER);
  CHECK(make_norm_plan(bad, kMaxTensors + 1, &p) == FLCE_ERR_BAD_SHAPE);
  CHECK(ceil_div(kMaxTensorSize, kAdamChunk) * kAdamThreads < ((int64_t)1 << 32));
  std::printf("failures: %d\n", failures);
  return failures != 0;
}
