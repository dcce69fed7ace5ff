/*
 * The operators at the two ends of a training step from plain C99: device buffers from
 * the HIP runtime, one stream, checked against the definitions computed here.
 *
 *   - logits: whole numbers, every sum exact, with a bias, in a wider output;
 *   - processing: penalties, a listed bias and a mask, bit for bit, statistics, the
 *     invalid-token count and the gradient;
 *   - norm of two tensors and an AdamW step of fp32 and 8-bit states, a skipped step;
 *   - host-side argument errors, after which nothing is launched.
 *
 * Prints "flce_step_check ok" and returns 0 on success, 1 on the first failure.
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <hip/hip_runtime_api.h>

#include "flce.h"

#define N 3
#define H 40
#define V 37
#define LD 41

#define CHECK(cond, ...)                 \
  do {                                   \
    if (!(cond)) {                       \
      printf("FAIL: " __VA_ARGS__);      \
      printf("\n");                      \
      return 1;                          \
    }                                    \
  } while (0)
#define HIPCK(x) CHECK((x) == hipSuccess, "HIP call %s", #x)
#define FLCK(x) CHECK((x) == FLCE_OK, "%s -> %s", #x, flce_status_string(x))
#define UP(d, h)                                                   \
  do {                                                             \
    HIPCK(hipMalloc((void**)&(d), sizeof(h)));                     \
    HIPCK(hipMemcpy((d), (h), sizeof(h), hipMemcpyHostToDevice));  \
  } while (0)
#define DOWN(h, d)                                                 \
  do {                                                             \
    HIPCK(hipStreamSynchronize(st));                               \
    HIPCK(hipMemcpy((h), (d), sizeof(h), hipMemcpyDeviceToHost));  \
  } while (0)

static uint32_t lcg = 777u;
static uint32_t next(void) {
  lcg = lcg * 1664525u + 1013904223u;
  return lcg >> 8;
}
static float small(void) { return (float)((int)(next() % 17) - 8); } /* whole, exact in bf16 */
static uint16_t bf16(float f) { /* f exact in bf16 */
  uint32_t u;
  memcpy(&u, &f, 4);
  return (uint16_t)(u >> 16);
}
static int close_to(float got, double want) {
  return fabs((double)got - want) <= ldexp(fabs(want) + 1.0, -20);
}

static int logits(hipStream_t st) {
  static uint16_t hh[N * H], hw[H * V];
  static float fh[N * H], fw[H * V], hb[V], out[N * LD];
  for (int i = 0; i < N * H; ++i) hh[i] = bf16(fh[i] = small());
  for (int i = 0; i < H * V; ++i) hw[i] = bf16(fw[i] = small());
  for (int i = 0; i < V; ++i) hb[i] = small();
  for (int i = 0; i < N * LD; ++i) out[i] = 5.0f;
  void *dh, *dw, *ws;
  float *db, *dout;
  UP(dh, hh);
  UP(dw, hw);
  UP(db, hb);
  UP(dout, out);
  size_t wsb = 0;
  FLCK(flce_logits_workspace_size(N, H, V, &wsb));
  HIPCK(hipMalloc(&ws, wsb));
  CHECK(flce_logits(dh, dw, db, N, H, V, 0.0f, FLCE_GRAD_F32, dout, V - 1, ws, wsb, st) ==
            FLCE_ERR_BAD_SHAPE, "short rows");
  CHECK(flce_logits(dh, dw, db, N, H, V, 0.0f, FLCE_GRAD_F32, dout, LD, ws, wsb - 1, st) ==
            FLCE_ERR_WORKSPACE_TOO_SMALL, "short workspace");
  FLCK(flce_logits(dh, dw, db, N, H, V, 0.0f, FLCE_GRAD_F32, dout, LD, ws, wsb, st));
  DOWN(out, dout);
  for (int i = 0; i < N; ++i)
    for (int v = 0; v < LD; ++v) {
      float want = v < V ? hb[v] : 5.0f;
      for (int h = 0; v < V && h < H; ++h) want += fh[i * H + h] * fw[h * V + v];
      CHECK(out[i * LD + v] == want, "logit %d %d: %g, not %g", i, v, out[i * LD + v], want);
    }
  return 0;
}

static int process(hipStream_t st) {
  static float x[N * V], out[N * V], g[N * V], want[N * V], slope[N * V];
  static float lse[N], ent[N];
  static int64_t top[N];
  /* Histories: {1, 2 | 2, 2, V}, {} and {0 |}. */
  static int64_t tokens[6] = {1, 2, 2, 2, V, 0}, cu[N + 1] = {0, 5, 5, 6}, prompt[N] = {2, 0, 9};
  static int64_t bt[2] = {3, 3}, bcu[N + 1] = {0, 0, 2, 2};
  static float bv[2] = {0.5f, 0.25f};
  static int32_t allowed[2] = {~1, -1}; /* all but id 0 */
  for (int i = 0; i < N * V; ++i) {
    x[i] = small();
    g[i] = small();
  }
  for (int i = 0; i < N; ++i)
    for (int v = 0; v < V; ++v) {
      float y = x[i * V + v], s = 1.0f;
      const int seen = (i == 0 && (v == 1 || v == 2)) || (i == 2 && v == 0);
      if (seen) s = y > 0 ? 1.0f / 2.0f : 2.0f;
      y *= s;
      if (i == 0 && v == 2) y = (y - 0.5f * 2) - 0.25f;
      if (i == 1 && v == 3) y += 0.5f + 0.25f;
      want[i * V + v] = v == 0 ? -INFINITY : y * 4.0f;
      slope[i * V + v] = v == 0 ? 0.0f : s * 4.0f;
    }
  float *dx, *dout, *dg, *dlse, *dent, *dbv;
  int64_t *dtop, *dt, *dcu, *dp, *dbt, *dbcu;
  int32_t* da;
  void* ws;
  UP(dx, x);
  UP(dout, out);
  UP(dg, g);
  UP(dlse, lse);
  UP(dent, ent);
  UP(dtop, top);
  UP(dt, tokens);
  UP(dcu, cu);
  UP(dp, prompt);
  UP(dbt, bt);
  UP(dbv, bv);
  UP(dbcu, bcu);
  UP(da, allowed);
  flce_process_options_t o;
  memset(&o, 0, sizeof o);
  o.ignore_index = -100;
  o.tokens = dt;
  o.tokens_size = 6;
  o.offsets = dcu;
  o.prompt_lengths = dp;
  o.repetition_penalty = 2.0;
  o.presence_penalty = 0.25;
  o.frequency_penalty = 0.5;
  o.temperature = 0.25;
  o.bias_tokens = dbt;
  o.bias_values = dbv;
  o.bias_count = 2;
  o.bias_offsets = dbcu;
  o.allowed = da;
  o.logits_dtype = o.out_dtype = FLCE_GRAD_F32;
  size_t wsb = 0;
  FLCK(flce_process_workspace_size(N, V, &wsb));
  HIPCK(hipMalloc(&ws, wsb));
  o.temperature = -1.0;
  CHECK(flce_process_logits(dx, V, N, V, &o, dout, V, dlse, dent, dtop, ws, wsb, st) ==
            FLCE_ERR_BAD_OPTION, "negative temperature");
  o.temperature = 0.25;
  FLCK(flce_process_logits(dx, V, N, V, &o, dout, V, dlse, dent, dtop, ws, wsb, st));
  int64_t invalid = -1;
  CHECK(flce_get_status(ws, &invalid, st) == FLCE_ERR_INVALID_LABEL && invalid == 1,
        "invalid tokens %lld", (long long)invalid);
  DOWN(out, dout);
  DOWN(lse, dlse);
  DOWN(ent, dent);
  DOWN(top, dtop);
  for (int i = 0; i < N; ++i) {
    double m = -INFINITY, s = 0, u = 0;
    int best = -1;
    for (int v = 0; v < V; ++v) {
      CHECK(out[i * V + v] == want[i * V + v], "row %d id %d: %g, not %g", i, v, out[i * V + v],
            want[i * V + v]);
      if (want[i * V + v] > m) {
        m = want[i * V + v];
        best = v;
      }
    }
    for (int v = 1; v < V; ++v) {
      s += exp(want[i * V + v] - m);
      u += exp(want[i * V + v] - m) * (want[i * V + v] - m);
    }
    CHECK(close_to(lse[i], m + log(s)) && close_to(ent[i], log(s) - u / s) && top[i] == best,
          "statistics of row %d", i);
  }
  flce_process_grads_t up;
  memset(&up, 0, sizeof up);
  up.grad_out = dg;
  up.ld_grad_out = V;
  FLCK(flce_process_logits_backward(&up, dx, V, N, V, &o, dout, V, ws, wsb, st));
  DOWN(out, dout);
  for (int i = 0; i < N * V; ++i)
    CHECK(out[i] == g[i] * slope[i], "gradient %d: %g, not %g", i, out[i], g[i] * slope[i]);
  return 0;
}

static int update(int state, hipStream_t st) {
  enum { A = 300, B = 5 };
  static float pa[A], ga[A], m[A], v[A], sc[2], na[1], ns[1];
  static uint16_t pb[B], gb[B];
  static int64_t step[1];
  double sum = 0;
  for (int i = 0; i < A; ++i) {
    pa[i] = small();
    ga[i] = small();
    m[i] = v[i] = 0;
    sum += (double)ga[i] * ga[i];
  }
  for (int i = 0; i < B; ++i) {
    pb[i] = bf16(small());
    gb[i] = bf16(2.0f);
    sum += 4.0;
  }
  step[0] = 0;
  float *dpa, *dga, *dn, *ds, *dsc[4];
  uint16_t *dpb, *dgb;
  void *dm[2], *dv[2], *ws;
  int64_t* dstep;
  UP(dpa, pa);
  UP(dga, ga);
  UP(dpb, pb);
  UP(dgb, gb);
  UP(dn, na);
  UP(ds, ns);
  UP(dstep, step);
  sc[0] = sc[1] = 0;
  for (int k = 0; k < 4; ++k) UP(dsc[k], sc);
  for (int k = 0; k < 2; ++k) {
    UP(dm[k], m);
    UP(dv[k], v);
  }
  const void* grads[2] = {dga, dgb};
  const int64_t sizes[2] = {A, B};
  const int dtypes[2] = {FLCE_GRAD_F32, FLCE_GRAD_BF16};
  size_t wsb = 0;
  FLCK(flce_grad_norm_workspace_size(sizes, 2, &wsb));
  if (wsb < flce_adamw_workspace_size()) wsb = flce_adamw_workspace_size();
  HIPCK(hipMalloc(&ws, wsb));
  CHECK(flce_grad_norm(grads, sizes, dtypes, 2, -1.0, dn, ds, ws, wsb, st) ==
            FLCE_ERR_BAD_OPTION, "negative norm");
  FLCK(flce_grad_norm(grads, sizes, dtypes, 2, 1.0, dn, ds, ws, wsb, st));
  DOWN(na, dn);
  DOWN(ns, ds);
  CHECK(na[0] == (float)sqrt(sum) && close_to(ns[0], 1.0 / sqrt(sum)), "norm %g", na[0]);

  void* params[2] = {dpa, dpb};
  void* ms[2] = {dsc[0], dsc[1]};
  void* vs[2] = {dsc[2], dsc[3]};
  flce_adamw_list_t l;
  memset(&l, 0, sizeof l);
  l.count = 2;
  l.sizes = sizes;
  l.params = params;
  l.grads = grads;
  l.exp_avgs = dm;
  l.exp_avg_sqs = dv;
  l.exp_avg_scales = ms;
  l.exp_avg_sq_scales = vs;
  l.param_dtypes = l.grad_dtypes = dtypes;
  flce_adamw_options_t o;
  memset(&o, 0, sizeof o);
  o.lr = 0.5;
  o.beta1 = 0.9;
  o.beta2 = 0.99;
  o.eps = 1e-8;
  o.state_dtype = state;
  o.rounding = FLCE_ROUND_NEAREST;
  o.beta1 = 1.0;
  CHECK(flce_adamw_step(&l, &o, NULL, ds, dstep, ws, wsb, st) == FLCE_ERR_BAD_OPTION, "beta 1");
  o.beta1 = 0.9;
  /* Bias correction makes the first update lr times the gradient's sign. */
  FLCK(flce_adamw_step(&l, &o, NULL, ds, dstep, ws, wsb, st));
  static float got[A];
  static uint16_t gotb[B];
  DOWN(got, dpa);
  DOWN(gotb, dpb);
  DOWN(step, dstep);
  CHECK(step[0] == 1, "step %lld", (long long)step[0]);
  for (int i = 0; i < A; ++i) {
    const double want = pa[i] - (ga[i] > 0 ? 0.5 : (ga[i] < 0 ? -0.5 : 0.0));
    CHECK(fabs(got[i] - want) < 1e-5, "weight %d: %g, not %g", i, got[i], want);
  }
  for (int i = 0; i < B; ++i) {
    uint32_t u = (uint32_t)pb[i] << 16;
    float f;
    memcpy(&f, &u, 4);
    CHECK(gotb[i] == bf16(f - 0.5f), "bf16 weight %d", i);
  }
  /* A factor that is not finite: nothing changes. */
  ns[0] = NAN;
  HIPCK(hipMemcpy(ds, ns, sizeof ns, hipMemcpyHostToDevice));
  FLCK(flce_adamw_step(&l, &o, NULL, ds, dstep, ws, wsb, st));
  static float again[A];
  DOWN(again, dpa);
  DOWN(step, dstep);
  CHECK(step[0] == 1 && memcmp(again, got, sizeof got) == 0, "a skipped step");
  return 0;
}

int main(void) {
  hipStream_t st;
  HIPCK(hipStreamCreate(&st));
  if (logits(st) || process(st) || update(FLCE_STATE_F32, st) || update(FLCE_STATE_8BIT, st))
    return 1;
  printf("flce_step_check ok\n");
  return 0;
}
