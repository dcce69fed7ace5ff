/*
 * The operators beside the head from plain C99: device buffers from the HIP
 * runtime, one stream, checked against the definitions computed here in double.
 *
 *   - embedding: lookup from a table [V,H] and from a weight [H,V], bit for bit
 *     (scale 2: exact), the invalid-token count, and the gradient of both layouts,
 *     written fresh and added (whole numbers: every sum exact);
 *   - policy loss: mean over tokens with k2 KL and an entropy bonus, the statistics
 *     and gradients, in one call and in two;
 *   - preference loss: the sigmoid loss of two pairs, rewards and gradient;
 *   - host-side argument errors, after which nothing is launched.
 *
 * Prints "flce_ops_check ok" and returns 0 on success, 1 on the first failure.
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <hip/hip_runtime_api.h>

#include "flce.h"

#define N 200
#define H 16
#define V 37
#define B 4

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
static float urand(void) { return (float)next() / 16777216.0f; } /* [0, 1) */
static float small(void) { return (float)((int)(next() % 17) - 8); } /* whole, exact in bf16 */
static uint16_t bf16(float f) { /* f exact in bf16 */
  uint32_t u;
  memcpy(&u, &f, 4);
  return (uint16_t)(u >> 16);
}
static float from_bf16(uint16_t b) {
  uint32_t u = (uint32_t)b << 16;
  float f;
  memcpy(&f, &u, 4);
  return f;
}
static int close_to(float got, double want) {
  return fabs((double)got - want) <= ldexp(fabs(want), -23) + 1e-12;
}

static int embedding(int layout, hipStream_t st) {
  static uint16_t hw[V * H], hout[N * H], hg[N * H];
  static float hgw[V * H], hbase[V * H];
  static int64_t ht[N];
  for (int i = 0; i < V * H; ++i) hw[i] = bf16(small());
  for (int i = 0; i < V * H; ++i) hbase[i] = small();
  for (int i = 0; i < N * H; ++i) hg[i] = bf16(small());
  for (int i = 0; i < N; ++i) ht[i] = (int64_t)(next() % V);
  ht[3] = -100;
  ht[4] = V;
  void *dw, *dg, *ws;
  uint16_t* dout;
  float* dgw;
  int64_t* dt;
  UP(dw, hw);
  UP(dg, hg);
  UP(dt, ht);
  UP(dout, hout);
  UP(dgw, hbase);
  flce_embedding_options_t o;
  memset(&o, 0, sizeof o);
  o.ignore_index = -100;
  o.scale = 2.0;
  o.layout = layout;
  o.hidden_dtype = FLCE_GRAD_BF16;
  o.grad_dtype = FLCE_GRAD_F32;
  size_t fb = 0, bb = 0;
  FLCK(flce_embedding_workspace_size(N, H, V, &o, &fb, &bb));
  const size_t wsb = fb > bb ? fb : bb;
  HIPCK(hipMalloc(&ws, wsb));
  CHECK(flce_embedding_forward((char*)dw + 2, dt, N, H, V, 0, V, &o, dout, ws, wsb, st) ==
            FLCE_ERR_MISALIGNED, "misaligned weight");
  CHECK(flce_embedding_backward(dg, dt, N, H, V, 2, V, &o, dgw, ws, wsb, st) ==
            FLCE_ERR_BAD_SHAPE, "slice outside the vocabulary");
  FLCK(flce_embedding_forward(dw, dt, N, H, V, 0, V, &o, dout, ws, wsb, st));
  int64_t invalid = -1;
  CHECK(flce_get_status(ws, &invalid, st) == FLCE_ERR_INVALID_LABEL && invalid == 1,
        "invalid tokens %lld", (long long)invalid);
  DOWN(hout, dout);
  for (int i = 0; i < N; ++i)
    for (int h = 0; h < H; ++h) {
      const int64_t v = ht[i];
      const int on = v >= 0 && v < V;
      const float want =
          on ? 2.0f * from_bf16(hw[layout == FLCE_EMBED_VH ? v * H + h : h * V + v]) : 0.0f;
      CHECK(from_bf16(hout[i * H + h]) == want, "layout %d hidden %d %d", layout, i, h);
    }
  for (int acc = 1; acc >= 0; --acc) { /* added first: the buffer holds hbase */
    o.accumulate = acc;
    FLCK(flce_embedding_backward(dg, dt, N, H, V, 0, V, &o, dgw, ws, wsb, st));
    DOWN(hgw, dgw);
    for (int v = 0; v < V; ++v)
      for (int h = 0; h < H; ++h) {
        const int at = layout == FLCE_EMBED_VH ? v * H + h : h * V + v;
        double want = acc ? hbase[at] : 0.0;
        for (int i = 0; i < N; ++i)
          if (ht[i] == v) want += 2.0 * from_bf16(hg[i * H + h]);
        CHECK((double)hgw[at] == want, "layout %d acc %d gradient %d %d", layout, acc, v, h);
      }
  }
  (void)hipFree(dw);
  (void)hipFree(dg);
  (void)hipFree(dt);
  (void)hipFree(dout);
  (void)hipFree(dgw);
  (void)hipFree(ws);
  return 0;
}

static int losses(hipStream_t st) {
  static float lp[N], old[N], ref[N], ent[N], adv[N], glp[N], gent[N], stats[8], loss[1];
  static int64_t lab[N];
  static const int64_t cu[B + 1] = {0, 60, 61, 61, 190}; /* one token, none; padding behind */
  float up[1] = {0.5f};
  double state_init[2 * (B + 1)] = {0};
  for (int i = 0; i < N; ++i) {
    lp[i] = -urand();
    old[i] = lp[i] + 0.6f * (urand() - 0.5f);
    ref[i] = lp[i] + 0.4f * (urand() - 0.5f);
    ent[i] = urand();
    adv[i] = urand() - 0.5f;
    lab[i] = next() % 5 == 0 ? -100 : (int64_t)(next() % V);
  }
  lab[60] = 5; /* the sequence of one token */
  float *dlp, *dold, *dref, *dent, *dadv, *dglp, *dgent, *dstats, *dloss, *dup;
  int64_t *dlab, *dcu;
  double* dstate;
  void* ws;
  UP(dlp, lp);
  UP(dold, old);
  UP(dref, ref);
  UP(dent, ent);
  UP(dadv, adv);
  UP(dlab, lab);
  UP(dcu, cu);
  UP(dglp, glp);
  UP(dgent, gent);
  UP(dstats, stats);
  UP(dloss, loss);
  UP(dup, up);
  UP(dstate, state_init);
  size_t pb = 0, qb = 0;
  FLCK(flce_policy_workspace_size(N, B, &pb));
  FLCK(flce_preference_workspace_size(N, B / 2, &qb));
  HIPCK(hipMalloc(&ws, pb > qb ? pb : qb));

  flce_policy_options_t p;
  memset(&p, 0, sizeof p);
  p.ignore_index = -100;
  p.clip_low = 0.125;
  p.clip_high = 0.25;
  p.kl_coef = 0.1;
  p.entropy_coef = 0.01;
  p.kl_estimator = FLCE_KL_K2;
  p.level = FLCE_RATIO_TOKEN;
  p.reduction = FLCE_REDUCTION_MEAN;
  double want[6] = {0}, count = 0;
  for (int i = 0; i < cu[B]; ++i) count += lab[i] >= 0;
  for (int i = 0; i < cu[B]; ++i) {
    if (lab[i] < 0) continue;
    const double r = exp((double)lp[i] - old[i]), x = (double)lp[i] - ref[i], A = adv[i];
    const double c = r < 0.875 ? 0.875 : (r > 1.25 ? 1.25 : r);
    const double f = -(r * A < c * A ? r * A : c * A);
    want[0] += (f + 0.1 * 0.5 * x * x - 0.01 * ent[i]) / count;
    want[1] += f / count;
    want[2] += 0.5 * x * x / count;
    want[3] += ent[i] / count;
    want[4] += (f != -r * A) / count;
    want[5] -= ((double)lp[i] - old[i]) / count;
  }
  CHECK(flce_policy_loss_forward(dlp, dent, dold, NULL, dadv, dlab, dcu, N, B, V, &p, dloss,
                                 dstats, dstate, ws, pb, st) == FLCE_ERR_NULL_POINTER,
        "KL without a reference");
  p.clip_low = 2.0;
  CHECK(flce_policy_loss_forward(dlp, dent, dold, dref, dadv, dlab, dcu, N, B, V, &p, dloss,
                                 dstats, dstate, ws, pb, st) == FLCE_ERR_BAD_OPTION, "clip_low");
  p.clip_low = 0.125;
  for (int both = 0; both < 2; ++both) {
    if (both) {
      FLCK(flce_policy_loss_forward_backward(dlp, dent, dold, dref, dadv, dlab, dcu, N, B, V, &p,
                                             dup, dloss, dstats, dglp, dgent, ws, pb, st));
    } else {
      FLCK(flce_policy_loss_forward(dlp, dent, dold, dref, dadv, dlab, dcu, N, B, V, &p, dloss,
                                    dstats, dstate, ws, pb, st));
      FLCK(flce_policy_loss_backward(dlp, dold, dref, dadv, dlab, dcu, N, B, V, &p, dstate, dup,
                                     dglp, dgent, st));
    }
    FLCK(flce_get_status(ws, NULL, st));
    DOWN(stats, dstats);
    DOWN(loss, dloss);
    DOWN(glp, dglp);
    DOWN(gent, dgent);
    for (int k = 0; k < 6; ++k)
      CHECK(close_to(stats[k], want[k]), "statistic %d: %g, %g", k, stats[k], want[k]);
    CHECK(loss[0] == stats[0] && stats[6] == count && stats[7] == 3.0, "loss and counts");
    for (int i = 0; i < N; ++i) {
      double g = 0.0, e = 0.0;
      if (i < cu[B] && lab[i] >= 0) {
        const double r = exp((double)lp[i] - old[i]), x = (double)lp[i] - ref[i], A = adv[i];
        const int clip = A > 0 ? r > 1.25 : r < 0.875;
        g = 0.5 * ((clip ? 0.0 : -r * A) + 0.1 * x) / count;
        e = -0.5 * 0.01 / count;
      }
      CHECK(close_to(glp[i], g) && close_to(gent[i], e), "policy gradient %d", i);
    }
  }

  flce_preference_options_t q;
  memset(&q, 0, sizeof q);
  q.ignore_index = -100;
  q.beta = 0.3;
  q.margin = 0.1;
  q.kind = FLCE_PREFERENCE_SIGMOID;
  q.reduction = FLCE_REDUCTION_SUM;
  float pair[B / 2], chosen[B / 2], rejected[B / 2];
  float *dpair, *dchosen, *drejected;
  UP(dpair, pair);
  UP(dchosen, chosen);
  UP(drejected, rejected);
  FLCK(flce_preference_loss_forward_backward(dlp, dref, dlab, dcu, N, B / 2, V, &q, dup, dloss,
                                             dpair, dchosen, drejected, dglp, ws, qb, st));
  DOWN(loss, dloss);
  DOWN(pair, dpair);
  DOWN(chosen, dchosen);
  DOWN(rejected, drejected);
  DOWN(glp, dglp);
  double R[B] = {0}, total = 0.0, slope[B];
  for (int s = 0; s < B; ++s)
    for (int i = (int)cu[s]; i < cu[s + 1]; ++i)
      if (lab[i] >= 0) R[s] += (double)lp[i] - ref[i];
  for (int i = 0; i < B / 2; ++i) {
    const double x = 0.3 * (R[i] - R[B / 2 + i]) - 0.1, l = log1p(exp(-x));
    slope[i] = -0.3 / (1.0 + exp(x));
    slope[B / 2 + i] = -slope[i];
    total += l;
    CHECK(close_to(pair[i], l) && close_to(chosen[i], 0.3 * R[i]) &&
              close_to(rejected[i], 0.3 * R[B / 2 + i]), "pair %d", i);
  }
  CHECK(close_to(loss[0], total), "preference loss");
  for (int s = 0, i = 0; i < N; ++i) {
    while (s < B && i >= cu[s + 1]) ++s;
    CHECK(close_to(glp[i], s < B && lab[i] >= 0 ? 0.5 * slope[s] : 0.0), "gradient %d", i);
  }
  FLCK(flce_preference_loss_forward(dlp, dref, dlab, dcu, N, B / 2, V, &q, dloss, dpair, dchosen,
                                    drejected, dstate, ws, qb, st));
  HIPCK(hipMemsetAsync(dglp, 0xff, sizeof glp, st));
  FLCK(flce_preference_loss_backward(dlab, dcu, N, B / 2, V, &q, dstate, dup, dglp, st));
  static float again[N];
  DOWN(again, dglp);
  CHECK(memcmp(again, glp, sizeof glp) == 0, "two calls and one differ");
  return 0;
}

int main(void) {
  hipStream_t st;
  HIPCK(hipStreamCreate(&st));
  if (embedding(FLCE_EMBED_VH, st) || embedding(FLCE_EMBED_HV, st) || losses(st)) return 1;
  printf("flce_ops_check ok\n");
  return 0;
}
