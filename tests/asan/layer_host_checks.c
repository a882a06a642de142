/* Host-side argument checks of the operators around the routed experts, built with AddressSanitizer
 * on the host code of the library (as abi_host_checks.c): every call must be rejected, or finish as
 * a no-op, on the host; the parameter structs are heap blocks of exactly their size, so a read past
 * them in the library is reported.  Exit status 0 when every status code matches, 1 otherwise. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "moe_mi355x.h"

static void *const P = (void *)0x100000; /* placeholder device pointer */
static int failures = 0;

#define EXPECT(call, want)                                                                   \
  do {                                                                                       \
    const int got_ = (int)(call);                                                            \
    if (got_ != (int)(want)) {                                                               \
      fprintf(stderr, "%s:%d: %s -> %d, expected %d\n", __FILE__, __LINE__, #call, got_,     \
              (int)(want));                                                                  \
      ++failures;                                                                            \
    }                                                                                        \
  } while (0)

static moe_block_norm_t *norm(void) {
  moe_block_norm_t *p = (moe_block_norm_t *)calloc(1, sizeof(*p));
  p->x = P; p->y = P; p->w_post = P; p->w_pre = P; p->h = P; p->n = P; p->rstd = P;
  p->tokens = 4; p->dim = 64; p->scale = 1.f; p->eps = 1e-6f;
  return p;
}

static void norm_checks(void) {
  moe_block_norm_t *p = norm();
  EXPECT(moe_block_norm(NULL, NULL), MOE_ERR_INVALID_ARG);
  p->eps = -1.f;
  EXPECT(moe_block_norm(p, NULL), MOE_ERR_INVALID_ARG);
  p->eps = 1e-6f; p->gate_kind = MOE_GATE_TOKEN;
  EXPECT(moe_block_norm(p, NULL), MOE_ERR_INVALID_ARG);
  p->gate_kind = 0; p->dim = MOE_NORM_MAX_DIM + 1;
  EXPECT(moe_block_norm(p, NULL), MOE_ERR_UNSUPPORTED);
  p->dim = 64; p->tokens = 0;
  EXPECT(moe_block_norm(p, NULL), MOE_OK);
  p->tokens = 4;
  moe_block_norm_grads_t *d = (moe_block_norm_grads_t *)calloc(1, sizeof(*d));
  EXPECT(moe_block_norm_backward(p, NULL, P, 1 << 20, NULL), MOE_ERR_INVALID_ARG);
  EXPECT(moe_block_norm_backward(p, d, P, 1 << 20, NULL), MOE_ERR_INVALID_ARG);
  d->dh = P; d->dx = P; d->dy = P; d->dw_post = P;
  EXPECT(moe_block_norm_backward(p, d, P, 16, NULL), MOE_ERR_WORKSPACE);
  EXPECT(moe_block_norm_backward(p, d, NULL, 1 << 20, NULL), MOE_ERR_INVALID_ARG);
  EXPECT(moe_block_norm_backward(p, d, (char *)P + 2, 1 << 20, NULL), MOE_ERR_INVALID_ARG);
  free(d); free(p);
}

static void router_checks(void) {
  moe_router_t *r = (moe_router_t *)calloc(1, sizeof(*r));
  moe_balance_t *b = (moe_balance_t *)calloc(1, sizeof(*b));
  r->logits = P; r->topk_ids = P; r->topk_w = P;
  r->tokens = 4; r->num_experts = 8; r->topk = 2; r->scale = 1.f;
  EXPECT(moe_router(NULL, NULL, NULL, 0, NULL), MOE_ERR_INVALID_ARG);
  r->score = 7;
  EXPECT(moe_router(r, NULL, NULL, 0, NULL), MOE_ERR_INVALID_ARG);
  r->score = 0; r->topk = 9;
  EXPECT(moe_router(r, NULL, NULL, 0, NULL), MOE_ERR_UNSUPPORTED);
  r->topk = 2;
  EXPECT(moe_router(r, b, P, 1 << 20, NULL), MOE_ERR_INVALID_ARG);
  b->counts = P; b->mean_prob = P; b->loss = P; b->num_valid = P;
  EXPECT(moe_router(r, b, P, 16, NULL), MOE_ERR_WORKSPACE);
  EXPECT(moe_router(r, b, (char *)P + 1, 1 << 20, NULL), MOE_ERR_INVALID_ARG);
  EXPECT(moe_router_backward(r, NULL, NULL, NULL, P, NULL), MOE_ERR_INVALID_ARG);
  EXPECT(moe_router_backward(r, b, P, NULL, NULL, NULL), MOE_ERR_INVALID_ARG);
  r->tokens = 0;
  EXPECT(moe_router(r, NULL, NULL, 0, NULL), MOE_OK);
  EXPECT(moe_router_backward(r, b, P, NULL, NULL, NULL), MOE_OK);
  free(b); free(r);
}

static void int8_checks(void) {
  moe_act_params_t *a = (moe_act_params_t *)calloc(1, sizeof(*a));
  a->act = MOE_ACT_SITUV2; a->beta = 4.f; a->linear_beta = NAN;
  EXPECT(moe_quant_i8(P, 4, 24, P, P, NULL), MOE_ERR_INVALID_ARG);
  EXPECT(moe_quant_i8(P, 0, 32, P, P, NULL), MOE_OK);
  EXPECT(moe_pack_i8(P, 16, 72, (int8_t *)P + (1 << 20), NULL), MOE_ERR_UNSUPPORTED);
  EXPECT(moe_pack_i8(P, 16, 64, P, NULL), MOE_ERR_INVALID_ARG);
  EXPECT(moe_gemm_i8(P, P, P, P, 4, 64, 64, a, NULL, P, NULL), MOE_ERR_INVALID_ARG);
  a->linear_beta = 25.f;
  EXPECT(moe_gemm_i8(P, P, P, P, 4, 48, 64, a, NULL, P, NULL), MOE_ERR_UNSUPPORTED);
  EXPECT(moe_gemm_i8(P, P, P, P, 4, 64, 24, a, NULL, P, NULL), MOE_ERR_UNSUPPORTED);
  EXPECT(moe_gemm_i8(NULL, P, P, P, 0, 64, 64, a, NULL, P, NULL), MOE_OK);
  free(a);
}

int main(void) {
  norm_checks();
  router_checks();
  int8_checks();
  if (failures) return 1;
  printf("all passed\n");
  return 0;
}
