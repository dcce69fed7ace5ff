// Host side of the operators at the two ends of a training step: argument checks,
// workspace layouts and kernel launches. Declarations and their documentation:
// include/flce.h.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "flce.h"
#include "flce_adamw.hpp"
#include "flce_launch.hpp"
#include "flce_logits.hpp"
#include "flce_process.hpp"
#include "flce_step_plan.hpp"

namespace {

using namespace flce;

template <int MT, int W>
void launch_logits(const LogitsArgs& a, bool f32, dim3 grid, hipStream_t st) {
  if (f32)
    logits_kernel<MT, W, true><<<grid, 64 * W, 0, st>>>(a);
  else
    logits_kernel<MT, W, false><<<grid, 64 * W, 0, st>>>(a);
}

// ---- processing of logits ----------------------------------------------------------

template <int HIST, bool LIST, int STEPS>
void launch_process_types(const ProcArgs& a, unsigned grid, hipStream_t st) {
  const bool i = a.o.logits_dtype == FLCE_GRAD_F32, o = a.o.out_dtype == FLCE_GRAD_F32;
  if (i && o)
    process_kernel<HIST, LIST, STEPS, true, true><<<grid, kProcThreads, 0, st>>>(a);
  else if (i)
    process_kernel<HIST, LIST, STEPS, true, false><<<grid, kProcThreads, 0, st>>>(a);
  else if (o)
    process_kernel<HIST, LIST, STEPS, false, true><<<grid, kProcThreads, 0, st>>>(a);
  else
    process_kernel<HIST, LIST, STEPS, false, false><<<grid, kProcThreads, 0, st>>>(a);
}
template <int HIST, bool LIST>
void launch_process(const ProcArgs& a, unsigned grid, hipStream_t st) {
  if (a.slice == kProcStep)
    launch_process_types<HIST, LIST, 1>(a, grid, st);
  else
    launch_process_types<HIST, LIST, kProcSteps>(a, grid, st);
}

template <bool SEEN, bool STATS>
void launch_process_grad(const ProcArgs& a, unsigned grid, hipStream_t st) {
  const size_t lds = SEEN ? (size_t)a.slice / 8 : 0;
  const bool i = a.o.logits_dtype == FLCE_GRAD_F32, o = a.o.out_dtype == FLCE_GRAD_F32;
  if (i && o)
    process_grad_kernel<SEEN, STATS, true, true><<<grid, kProcThreads, lds, st>>>(a);
  else if (i)
    process_grad_kernel<SEEN, STATS, true, false><<<grid, kProcThreads, lds, st>>>(a);
  else if (o)
    process_grad_kernel<SEEN, STATS, false, true><<<grid, kProcThreads, lds, st>>>(a);
  else
    process_grad_kernel<SEEN, STATS, false, false><<<grid, kProcThreads, lds, st>>>(a);
}

// `fn(args, grid)` for all rows, in launches of at most kMaxGrid blocks.
template <class F>
flce_status_t over_rows(ProcArgs a, int kind, hipStream_t st, F fn) {
  const int64_t most = kMaxGrid / a.slices;
  for (int64_t r = 0; r < a.N; r += most) {
    a.row0 = r;
    const int64_t rows = a.N - r < most ? a.N - r : most;
    FLCE_TRY(launch(kind, st, [&] { fn(a, (unsigned)(rows * a.slices)); }));
  }
  return FLCE_OK;
}

ProcArgs process_args(int64_t N, int64_t V, const flce_process_options_t& o, const ProcPlan& p,
                      void* ws) {
  ProcArgs a{};
  a.N = N;
  a.V = V;
  a.slice = p.slice;
  a.slices = p.slices;
  a.o = o;
  a.parts = reinterpret_cast<float4*>(wsp(ws, p.parts));
  a.invalid = reinterpret_cast<int32_t*>(wsp(ws, p.invalid));
  a.header = reinterpret_cast<int32_t*>(ws);
  return a;
}

bool good_ld(int64_t ld, int64_t V) { return ld >= V && ld <= ((int64_t)1 << 40); }

}  // namespace

extern "C" {

// ---- logits --------------------------------------------------------------------------

flce_status_t flce_logits_workspace_size(int64_t N, int64_t H, int64_t V, size_t* bytes) {
  FLCE_TRY(check_logits(N, H, V, 0.f, FLCE_GRAD_F32, V));
  if (bytes) *bytes = make_logits_plan(N, H, V).total;
  return FLCE_OK;
}

flce_status_t flce_logits(const void* hidden, const void* weight, const float* bias, int64_t N,
                          int64_t H, int64_t V, float softcap, int out_dtype, void* out,
                          int64_t ld_out, void* workspace, size_t workspace_bytes, void* stream) {
  FLCE_TRY(check_logits(N, H, V, softcap, out_dtype, ld_out));
  if (workspace == nullptr) return FLCE_ERR_NULL_POINTER;
  if (N > 0 && (hidden == nullptr || weight == nullptr || out == nullptr))
    return FLCE_ERR_NULL_POINTER;
  if (!aligned16(hidden) || !aligned16(weight) || !aligned16(workspace) || !at_multiple(bias, 4) ||
      !at_multiple(out, dtype_bytes(out_dtype)))
    return FLCE_ERR_MISALIGNED;
  const LogitsPlan p = make_logits_plan(N, H, V);
  if (workspace_bytes < p.total) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  if (N == 0) return FLCE_OK;
  LogitsArgs a{};
  a.hidden = static_cast<const uint16_t*>(hidden);
  a.weight = static_cast<const uint16_t*>(weight);
  a.bias = bias;
  a.N = N;
  a.H = H;
  a.V = V;
  a.cap = softcap > 0.f ? softcap : 0.f;
  a.inv_cap = softcap > 0.f ? 1.f / softcap : 0.f;
  a.out = out;
  a.ld_out = ld_out;
  const bool f32 = out_dtype == FLCE_GRAD_F32;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (p.wide > 0) {
    a.passes = p.passes;
    const unsigned grid = (unsigned)(ceil_div(p.strips, 8) * 8 * p.passes);
    return launch(K_LOGITS, st, [&] {
      switch (p.wide * 2 + (f32 ? 1 : 0)) {
        case 4: logits_wide_kernel<2, false><<<grid, 128, 0, st>>>(a); break;
        case 5: logits_wide_kernel<2, true><<<grid, 128, 0, st>>>(a); break;
        case 8: logits_wide_kernel<4, false><<<grid, 256, 0, st>>>(a); break;
        default: logits_wide_kernel<4, true><<<grid, 256, 0, st>>>(a); break;
      }
    });
  }
  if (p.mt == 0) {
    a.image = reinterpret_cast<uint16_t*>(wsp(workspace, p.image));
    a.hkb = p.hkb;
    a.VT = p.vt;
    a.TB = p.tb;
    const dim3 pack((unsigned)ceil_div(p.hkb, kPackBlocks), (unsigned)p.tb);
    FLCE_TRY(launch(K_LOGITS, st, [&] { logits_pack_kernel<<<pack, 256, 0, st>>>(a); }));
    return launch(K_LOGITS, st, [&] {
      const unsigned grid = (unsigned)(p.vt * p.tb);
      if (f32)
        logits_tile_kernel<true><<<grid, kThreads, 0, st>>>(a);
      else
        logits_tile_kernel<false><<<grid, kThreads, 0, st>>>(a);
    });
  }
  a.passes = p.passes;
  a.split_steps = p.split_steps;
  a.parts = reinterpret_cast<float*>(wsp(workspace, p.parts));
  const dim3 grid((unsigned)(ceil_div(p.strips, 8) * 8 * p.passes), (unsigned)p.splits);
  FLCE_TRY(launch(K_LOGITS, st, [&] {
    switch (p.mt * 100 + p.waves) {
      case 104: launch_logits<1, 4>(a, f32, grid, st); break;
      case 108: launch_logits<1, 8>(a, f32, grid, st); break;
      case 116: launch_logits<1, 16>(a, f32, grid, st); break;
      case 204: launch_logits<2, 4>(a, f32, grid, st); break;
      case 208: launch_logits<2, 8>(a, f32, grid, st); break;
      default: launch_logits<4, 4>(a, f32, grid, st); break;
    }
  }));
  if (p.splits == 1) return FLCE_OK;
  const dim3 sums((unsigned)ceil_div(V, 8 * 256), (unsigned)N);
  return launch(K_LOGITS, st, [&] {
    if (f32)
      logits_sum_kernel<true><<<sums, 256, 0, st>>>(a, p.splits);
    else
      logits_sum_kernel<false><<<sums, 256, 0, st>>>(a, p.splits);
  });
}

// ---- processing of logits ------------------------------------------------------------

flce_status_t flce_process_workspace_size(int64_t N, int64_t V, size_t* bytes) {
  if (N < 0 || N > kMaxN || V < 1 || V > kMaxV) return FLCE_ERR_BAD_SHAPE;
  if (bytes) *bytes = make_proc_plan(N, V).total;
  return FLCE_OK;
}

flce_status_t flce_process_logits(const void* logits, int64_t ld, int64_t N, int64_t V,
                                  const flce_process_options_t* opt, void* out, int64_t ld_out,
                                  float* lse, float* entropy, int64_t* greedy, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  FLCE_TRY(check_process(N, V, opt));
  if (!good_ld(ld, V) || !good_ld(ld_out, V)) return FLCE_ERR_BAD_SHAPE;
  if (workspace == nullptr) return FLCE_ERR_NULL_POINTER;
  if (N > 0 && (logits == nullptr || out == nullptr)) return FLCE_ERR_NULL_POINTER;
  if (!at_multiple(logits, dtype_bytes(opt->logits_dtype)) ||
      !at_multiple(out, dtype_bytes(opt->out_dtype)) || !at_multiple(lse, 4) ||
      !at_multiple(entropy, 4) || !at_multiple(greedy, 8) || !aligned16(workspace))
    return FLCE_ERR_MISALIGNED;
  if (N > 0 && logits == out && (opt->logits_dtype != opt->out_dtype || ld != ld_out))
    return FLCE_ERR_BAD_OPTION;
  const bool list = opt->bias_offsets != nullptr;
  const int hist = proc_history(*opt, false);
  const ProcPlan p = make_proc_plan(N, V);
  if (workspace_bytes < p.total) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  hipStream_t st = static_cast<hipStream_t>(stream);
  ProcArgs a = process_args(N, V, *opt, p, workspace);
  a.in = logits;
  a.ld = ld;
  a.out = out;
  a.ld_out = ld_out;
  a.lse = lse;
  a.entropy = entropy;
  a.greedy = greedy;
  FLCE_TRY(over_rows(a, K_PROCESS, st, [&](const ProcArgs& b, unsigned grid) {
    switch (hist * 2 + (list ? 1 : 0)) {
      case 0: launch_process<HIST_NONE, false>(b, grid, st); break;
      case 1: launch_process<HIST_NONE, true>(b, grid, st); break;
      case 2: launch_process<HIST_SEEN, false>(b, grid, st); break;
      case 3: launch_process<HIST_SEEN, true>(b, grid, st); break;
      case 4: launch_process<HIST_COUNT, false>(b, grid, st); break;
      default: launch_process<HIST_COUNT, true>(b, grid, st); break;
    }
  }));
  const unsigned rows = (unsigned)ceil_div(N, 4) + 1;
  return launch(K_PROCESS_ROWS, st, [&] { process_rows_kernel<<<rows, 256, 0, st>>>(a); });
}

flce_status_t flce_process_logits_backward(const flce_process_grads_t* grads, const void* logits,
                                           int64_t ld, int64_t N, int64_t V,
                                           const flce_process_options_t* opt, void* grad_logits,
                                           int64_t ld_grad, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  FLCE_TRY(check_process(N, V, opt));
  if (grads == nullptr || workspace == nullptr) return FLCE_ERR_NULL_POINTER;
  const flce_process_grads_t& g = *grads;
  const bool stats = g.grad_lse != nullptr || g.grad_entropy != nullptr;
  if (!good_ld(ld, V) || !good_ld(ld_grad, V) ||
      (g.grad_out != nullptr && !good_ld(g.ld_grad_out, V)) || (stats && !good_ld(g.ld_out, V)))
    return FLCE_ERR_BAD_SHAPE;
  if (N > 0 && (logits == nullptr || grad_logits == nullptr ||
                (stats && (g.out == nullptr || g.lse == nullptr)) ||
                (g.grad_entropy != nullptr && g.entropy == nullptr)))
    return FLCE_ERR_NULL_POINTER;
  const size_t out_bytes = dtype_bytes(opt->out_dtype), in_bytes = dtype_bytes(opt->logits_dtype);
  if (!at_multiple(logits, in_bytes) || !at_multiple(grad_logits, in_bytes) ||
      !at_multiple(g.grad_out, out_bytes) || !at_multiple(g.out, out_bytes) ||
      !at_multiple(g.grad_lse, 4) || !at_multiple(g.grad_entropy, 4) || !at_multiple(g.lse, 4) ||
      !at_multiple(g.entropy, 4) || !aligned16(workspace))
    return FLCE_ERR_MISALIGNED;
  if (N > 0 && g.grad_out == grad_logits &&
      (opt->logits_dtype != opt->out_dtype || g.ld_grad_out != ld_grad))
    return FLCE_ERR_BAD_OPTION;
  const ProcPlan p = make_proc_plan(N, V);
  if (workspace_bytes < p.total) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  hipStream_t st = static_cast<hipStream_t>(stream);
  ProcArgs a = process_args(N, V, *opt, p, workspace);
  a.in = logits;
  a.ld = ld;
  a.g = g;
  a.grad = grad_logits;
  a.ld_grad = ld_grad;
  // The lists have no part in the gradient.
  a.o.bias_offsets = nullptr;
  const bool seen = proc_history(*opt, true) == HIST_SEEN;
  FLCE_TRY(over_rows(a, K_PROCESS_GRAD, st, [&](const ProcArgs& b, unsigned grid) {
    switch ((seen ? 2 : 0) + (stats ? 1 : 0)) {
      case 0: launch_process_grad<false, false>(b, grid, st); break;
      case 1: launch_process_grad<false, true>(b, grid, st); break;
      case 2: launch_process_grad<true, false>(b, grid, st); break;
      default: launch_process_grad<true, true>(b, grid, st); break;
    }
  }));
  return launch(K_PROCESS_ROWS, st, [&] { process_status_kernel<<<1, 256, 0, st>>>(a); });
}

// ---- norm of the gradients, AdamW ------------------------------------------------------

flce_status_t flce_grad_norm_workspace_size(const int64_t* sizes, int64_t count, size_t* bytes) {
  NormPlan p;
  FLCE_TRY(make_norm_plan(sizes, count, &p));
  if (bytes) *bytes = p.total;
  return FLCE_OK;
}

flce_status_t flce_grad_norm(const void* const* grads, const int64_t* sizes, const int* dtypes,
                             int64_t count, double max_norm, float* norm, float* scale,
                             void* workspace, size_t workspace_bytes, void* stream) {
  NormPlan p;
  FLCE_TRY(make_norm_plan(sizes, count, &p));
  if (norm == nullptr || workspace == nullptr ||
      (count > 0 && (grads == nullptr || dtypes == nullptr)))
    return FLCE_ERR_NULL_POINTER;
  if (!(max_norm >= 0.0 && std::isfinite(max_norm))) return FLCE_ERR_BAD_OPTION;
  for (int64_t i = 0; i < count; ++i) {
    if (!known_dtype(dtypes[i])) return FLCE_ERR_BAD_OPTION;
    if (sizes[i] > 0 && grads[i] == nullptr) return FLCE_ERR_NULL_POINTER;
    if (sizes[i] > 0 && !at_multiple(grads[i], dtype_bytes(dtypes[i]))) return FLCE_ERR_MISALIGNED;
  }
  if (!at_multiple(norm, 4) || !at_multiple(scale, 4) || !aligned16(workspace))
    return FLCE_ERR_MISALIGNED;
  if (workspace_bytes < p.total) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  hipStream_t st = static_cast<hipStream_t>(stream);
  double* parts = reinterpret_cast<double*>(wsp(workspace, p.parts));
  NormArgs a{};
  a.chunk = p.chunk;
  a.parts = parts;
  int64_t blocks = 0;  // of the launch being collected
  auto flush = [&]() -> flce_status_t {
    if (blocks == 0) return FLCE_OK;
    FLCE_TRY(launch(K_GRAD_NORM, st, [&] {
      norm_parts_kernel<<<(unsigned)blocks, kNormThreads, 0, st>>>(a);
    }));
    a.parts += blocks;
    a.t.count = 0;
    blocks = 0;
    return FLCE_OK;
  };
  for (int64_t i = 0; i < count; ++i) {
    if (sizes[i] == 0) continue;
    if (a.t.count == kNormTensors) FLCE_TRY(flush());
    const int k = a.t.count++;
    a.t.grad[k] = grads[i];
    a.t.size[k] = sizes[i];
    a.t.f32[k] = dtypes[i] == FLCE_GRAD_F32 ? 1 : 0;
    a.t.first[k] = (int32_t)blocks;
    blocks += ceil_div(sizes[i], p.chunk);
  }
  FLCE_TRY(flush());
  return launch(K_GRAD_NORM, st, [&] {
    norm_total_kernel<<<1, 1024, 0, st>>>(parts, p.blocks, max_norm, norm, scale,
                                          reinterpret_cast<int32_t*>(workspace));
  });
}

size_t flce_adamw_workspace_size(void) { return 2 * kHeaderBytes; }

flce_status_t flce_adamw_step(const flce_adamw_list_t* list, const flce_adamw_options_t* opt,
                              const float* lr_device, const float* grad_scale, int64_t* step,
                              void* workspace, size_t workspace_bytes, void* stream) {
  FLCE_TRY(check_adamw(list, opt));
  if (step == nullptr || workspace == nullptr) return FLCE_ERR_NULL_POINTER;
  if (!at_multiple(lr_device, 4) || !at_multiple(grad_scale, 4) || !at_multiple(step, 8) ||
      !aligned16(workspace))
    return FLCE_ERR_MISALIGNED;
  if (workspace_bytes < flce_adamw_workspace_size()) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  static_assert(sizeof(AdamCoef) <= kHeaderBytes, "workspace layout");
  static_assert(sizeof(AdamArgs) <= 4096 && sizeof(NormArgs) <= 4096, "kernel arguments");
  hipStream_t st = static_cast<hipStream_t>(stream);
  AdamCoef* coef = reinterpret_cast<AdamCoef*>(wsp(workspace, kHeaderBytes));
  const AdamCoefArgs ca{opt->lr, opt->beta1, opt->beta2, opt->eps, opt->weight_decay, opt->seed,
                        lr_device, grad_scale, step, reinterpret_cast<int32_t*>(workspace), coef};
  FLCE_TRY(launch(K_ADAMW, st, [&] { adamw_coef_kernel<<<1, 64, 0, st>>>(ca); }));
  const bool eight = opt->state_dtype == FLCE_STATE_8BIT;
  const bool stochastic = opt->rounding == FLCE_ROUND_STOCHASTIC;
  AdamArgs a{};
  a.coef = coef;
  int64_t blocks = 0;
  auto flush = [&]() -> flce_status_t {
    if (blocks == 0) return FLCE_OK;
    FLCE_TRY(launch(K_ADAMW, st, [&] {
      const unsigned grid = (unsigned)blocks;
      if (eight && stochastic)
        adamw_kernel<true, true><<<grid, kAdamThreads, 0, st>>>(a);
      else if (eight)
        adamw_kernel<true, false><<<grid, kAdamThreads, 0, st>>>(a);
      else if (stochastic)
        adamw_kernel<false, true><<<grid, kAdamThreads, 0, st>>>(a);
      else
        adamw_kernel<false, false><<<grid, kAdamThreads, 0, st>>>(a);
    }));
    a.t.count = 0;
    blocks = 0;
    return FLCE_OK;
  };
  const flce_adamw_list_t& l = *list;
  for (int64_t i = 0; i < l.count; ++i) {
    if (l.sizes[i] == 0) continue;
    const int64_t n = ceil_div(l.sizes[i], kAdamChunk);
    if (a.t.count == kAdamTensors || blocks + n > kMaxGrid) FLCE_TRY(flush());
    const int k = a.t.count++;
    AdamEntry& e = a.t.e[k];
    e.param = l.params[i];
    e.grad = l.grads[i];
    e.master = l.masters != nullptr ? static_cast<float*>(l.masters[i]) : nullptr;
    e.m = l.exp_avgs[i];
    e.v = l.exp_avg_sqs[i];
    e.m_scale = eight ? static_cast<float*>(l.exp_avg_scales[i]) : nullptr;
    e.v_scale = eight ? static_cast<float*>(l.exp_avg_sq_scales[i]) : nullptr;
    e.size = l.sizes[i];
    a.t.kind[k] = (uint8_t)((l.param_dtypes[i] == FLCE_GRAD_F32 ? ADAM_PARAM_F32 : 0) |
                            (l.grad_dtypes[i] == FLCE_GRAD_F32 ? ADAM_GRAD_F32 : 0));
    a.t.number[k] = (int32_t)i;
    a.t.first[k] = (int32_t)blocks;
    blocks += n;
  }
  return flush();
}

}  // extern "C"
