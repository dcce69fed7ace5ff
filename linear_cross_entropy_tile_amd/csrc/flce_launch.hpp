// Kernel launches of libflce with the optional per-kernel event timing, shared
// by its translation units.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <mutex>
#include <vector>

#include "flce.h"

namespace flce {

// ---- kernel timing hooks --------------------------------------------------------
// flce_profile_read reports per kind in this order. K_PACK_WEIGHT no longer
// launches (the weight's dH image is written by the logit tiles themselves);
// its slot stays so that the indices of the later kinds do not move.
enum Kind {
  K_FWD_PREP, K_FWD_TILE, K_FWD_COMBINE, K_FWD_REDUCE, K_BWD_PREP, K_BWD_DLOGITS, K_BWD_DX,
  K_BWD_DW, K_DW_REDUCE, K_FILL, K_PACK_WEIGHT, K_PACK_HIDDEN, K_DX_FINALIZE, K_FUSED_TILE,
  K_FUSED_DLOGITS, K_BWD_DXDW, K_EMBED_SORT, K_EMBED_GATHER, K_EMBED_SEGMENTS, K_EMBED_GRAD,
  K_LOSS_PARTS, K_LOSS_SEQUENCES, K_LOSS_GRADS, K_LOSS_SMALL, K_NUM
};
inline const char* const kKindNames[K_NUM] = {
    "fwd_prep", "fwd_tile", "fwd_combine", "fwd_reduce", "bwd_prep", "bwd_dlogits", "bwd_dx",
    "bwd_dw", "dw_reduce", "fill_zero", "pack_weight", "pack_hidden", "dx_finalize", "fused_tile",
    "fused_dlogits", "bwd_dxdw", "embed_sort", "embed_gather", "embed_segments", "embed_grad",
    "loss_parts", "loss_sequences", "loss_grads", "loss_small"};

struct Pending {
  int kind;
  hipEvent_t a, b;
};
struct Profiler {
  std::mutex mu;
  bool on = false;
  std::vector<Pending> pending;
  std::vector<hipEvent_t> pool;
  int64_t launches[K_NUM] = {};
  double ms[K_NUM] = {};
  hipEvent_t get() {
    if (!pool.empty()) {
      hipEvent_t e = pool.back();
      pool.pop_back();
      return e;
    }
    hipEvent_t e = nullptr;
    if (hipEventCreate(&e) != hipSuccess) return nullptr;
    return e;
  }
  // Back into the pool; destroyed when there is no memory for that.
  void give(hipEvent_t e) {
    if (e == nullptr) return;
    try {
      pool.push_back(e);
    } catch (...) {
      (void)hipEventDestroy(e);
    }
  }
  void drain() {
    for (auto& p : pending) {
      float t = 0.f;
      if (hipEventSynchronize(p.b) == hipSuccess && hipEventElapsedTime(&t, p.a, p.b) == hipSuccess) {
        launches[p.kind] += 1;
        ms[p.kind] += t;
      }
      give(p.a);
      give(p.b);
    }
    pending.clear();
  }
};
inline Profiler& prof() {
  static Profiler* p = new Profiler();
  return *p;
}

// Launches through `fn` on `st`, bracketed by events when timing is on. A sample
// that there is no memory for is dropped: no exception leaves the C entry points.
template <class F>
flce_status_t launch(int kind, hipStream_t st, F fn) {
  Profiler& P = prof();
  hipEvent_t a = nullptr, b = nullptr;
  const bool timed = P.on;
  if (timed) {
    std::lock_guard<std::mutex> g(P.mu);
    a = P.get();
    b = P.get();
    if (a != nullptr) (void)hipEventRecord(a, st);
  }
  fn();
  const bool ok = hipGetLastError() == hipSuccess;
  if (timed) {
    bool kept = ok && a != nullptr && b != nullptr;
    if (kept) (void)hipEventRecord(b, st);
    std::lock_guard<std::mutex> g(P.mu);
    try {
      if (kept) P.pending.push_back({kind, a, b});
    } catch (...) {
      kept = false;
    }
    if (!kept) {
      P.give(a);
      P.give(b);
    }
  }
  return ok ? FLCE_OK : FLCE_ERR_HIP;
}

#define FLCE_TRY(x)                    \
  do {                                 \
    const flce_status_t _s = (x);      \
    if (_s != FLCE_OK) return _s;      \
  } while (0)

inline char* wsp(void* ws, size_t off) { return static_cast<char*>(ws) + off; }

}  // namespace flce
