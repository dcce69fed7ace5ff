// Host-only check of the launch hooks (flce_launch.hpp): no C++ exception leaves
// them when memory runs out while kernel timing is on; the launch itself goes
// ahead and only its sample is dropped. The HIP event calls are stand-ins here,
// which also count the events that are alive.
#include <cstdio>
#include <cstdlib>
#include <new>

#include "flce_launch.hpp"

static bool g_full = false;
static int g_events = 0;

void* operator new(size_t n) {
  if (g_full) throw std::bad_alloc();
  void* p = std::malloc(n ? n : 1);
  if (p == nullptr) throw std::bad_alloc();
  return p;
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, size_t) noexcept { std::free(p); }

extern "C" {
hipError_t hipEventCreate(hipEvent_t* e) {
  *e = reinterpret_cast<hipEvent_t>(std::malloc(1));
  ++g_events;
  return hipSuccess;
}
hipError_t hipEventDestroy(hipEvent_t e) {
  std::free(e);
  --g_events;
  return hipSuccess;
}
hipError_t hipEventRecord(hipEvent_t, hipStream_t) { return hipSuccess; }
hipError_t hipEventSynchronize(hipEvent_t) { return hipSuccess; }
hipError_t hipEventElapsedTime(float* t, hipEvent_t, hipEvent_t) {
  *t = 1.f;
  return hipSuccess;
}
static hipError_t g_error = hipSuccess;
hipError_t hipGetLastError(void) { return g_error; }
}

static int failures = 0;
#define CHECK(cond)                                                  \
  do {                                                               \
    if (!(cond)) {                                                   \
      std::fprintf(stderr, "FAIL line %d: %s\n", __LINE__, #cond);   \
      ++failures;                                                    \
    }                                                                \
  } while (0)

int main() {
  using namespace flce;
  Profiler& P = prof();
  int ran = 0;
  auto fn = [&] { ++ran; };
  CHECK(launch(K_FILL, nullptr, fn) == FLCE_OK && ran == 1 && g_events == 0);
  P.on = true;
  try {
    g_full = true;
    CHECK(launch(K_FILL, nullptr, fn) == FLCE_OK && ran == 2);
    g_full = false;
    CHECK(P.pending.empty());
    const size_t pooled = P.pool.size();
    CHECK((size_t)g_events == pooled);  // none is lost
    CHECK(launch(K_FILL, nullptr, fn) == FLCE_OK && ran == 3);
    CHECK(P.pending.size() == 1);
    g_full = true;
    P.drain();
    g_full = false;
    CHECK(P.pending.empty() && P.launches[K_FILL] == 1 && P.ms[K_FILL] == 1.0);
    CHECK((size_t)g_events == P.pool.size());
    g_error = hipErrorInvalidConfiguration;  // a failed launch keeps its events
    CHECK(launch(K_FILL, nullptr, fn) == FLCE_ERR_HIP);
    g_error = hipSuccess;
    CHECK(P.pending.empty() && (size_t)g_events == P.pool.size());
  } catch (...) {
    g_full = false;
    std::fprintf(stderr, "FAIL: an exception left the hooks\n");
    ++failures;
  }
  std::printf("failures: %d\n", failures);
  return failures != 0;
}
