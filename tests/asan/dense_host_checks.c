/* Host-side argument checks of layer norm, the microscaled matrices and the routed layer of a few tokens, built with AddressSanitizer on
 * the host code of the library (as layer_host_checks.c): every call must be rejected, or finish as a
 * no-op, on the host; the parameter structs are heap blocks of exactly their size. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

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

static void norm_checks(void) {
  moe_layer_norm_t *p = (moe_layer_norm_t *)calloc(1, sizeof(*p));
  moe_layer_norm_grads_t *d = (moe_layer_norm_grads_t *)calloc(1, sizeof(*d));
  p->x = P; p->n = P; p->stats = P; p->tokens = 4; p->dim = 64; p->eps = NAN;
  EXPECT(moe_layer_norm(NULL, NULL), MOE_ERR_INVALID_ARG);
  EXPECT(moe_layer_norm(p, NULL), MOE_ERR_INVALID_ARG);
  p->eps = 1e-5f; p->dim = MOE_NORM_MAX_DIM + 1;
  EXPECT(moe_layer_norm(p, NULL), MOE_ERR_UNSUPPORTED);
  p->dim = 64;
  EXPECT(moe_layer_norm_backward(p, NULL, P, 1 << 20, NULL), MOE_ERR_INVALID_ARG);
  EXPECT(moe_layer_norm_backward(p, d, P, 1 << 20, NULL), MOE_ERR_INVALID_ARG);
  d->dn = P; d->dx = P;
  EXPECT(moe_layer_norm_backward(p, d, P, 16, NULL), MOE_ERR_WORKSPACE);
  EXPECT(moe_layer_norm_backward(p, d, (char *)P + 2, 1 << 20, NULL), MOE_ERR_INVALID_ARG);
  p->tokens = 0;
  EXPECT(moe_layer_norm(p, NULL), MOE_OK);
  free(d); free(p);
}

static void mx_checks(void) {
  moe_quant_mx_t *p = (moe_quant_mx_t *)calloc(1, sizeof(*p));
  moe_act_params_t *a = (moe_act_params_t *)calloc(1, sizeof(*a));
  EXPECT(moe_quant_mx(NULL, NULL), MOE_ERR_INVALID_ARG);
  p->x = P; p->q = P; p->rows = 4; p->cols = 32; p->q_dt = MOE_DT_FP8_E4M3;
  EXPECT(moe_quant_mx(p, NULL), MOE_ERR_INVALID_ARG);
  p->q_scale = P; p->q_layout = MOE_MX_PACKED;
  EXPECT(moe_quant_mx(p, NULL), MOE_ERR_UNSUPPORTED);
  p->q_layout = MOE_MX_ROWS; p->rows = 0;
  EXPECT(moe_quant_mx(p, NULL), MOE_OK);
  EXPECT(moe_pack_mx(P, P, 16, 40, (uint8_t *)P + (1 << 20), (uint8_t *)P + (1 << 21), NULL), MOE_ERR_UNSUPPORTED);
  EXPECT(moe_pack_mx(P, (uint8_t *)P + (1 << 20), 16, 64, P, (uint8_t *)P + (1 << 21), NULL), MOE_ERR_INVALID_ARG);
  a->act = MOE_ACT_SITUV2; a->beta = 4.f; a->linear_beta = NAN;
  EXPECT(moe_gemm_mx(P, P, MOE_DT_FP4_E2M1, P, P, 4, 64, 128, a, NULL, P, MOE_DT_BF16, NULL), MOE_ERR_INVALID_ARG);
  a->linear_beta = 25.f;
  EXPECT(moe_gemm_mx(P, P, MOE_DT_FP4_E2M1, P, P, 4, 48, 128, a, NULL, P, MOE_DT_BF16, NULL), MOE_ERR_UNSUPPORTED);
  EXPECT(moe_gemm_mx(P, P, MOE_DT_FP4_E2M1, P, P, 4, 64, 96, a, NULL, P, MOE_DT_F32, NULL), MOE_ERR_UNSUPPORTED);
  EXPECT(moe_gemm_mx(NULL, NULL, MOE_DT_FP8_E4M3, P, P, 0, 64, 128, NULL, NULL, P, MOE_DT_F32, NULL), MOE_OK);
  free(a); free(p);
}

static void few_checks(void) {
  moe_router_t *r = (moe_router_t *)calloc(1, sizeof(*r));
  moe_act_params_t *a = (moe_act_params_t *)calloc(1, sizeof(*a));
  r->logits = P; r->topk_ids = P; r->topk_w = P;
  r->tokens = 4; r->num_experts = 8; r->topk = 2; r->scale = 1.f;
  a->act = MOE_ACT_SILU;
  EXPECT(moe_routed_few(NULL, P, NULL, MOE_DT_BF16, P, P, P, P, 0, 8, 128, 128, a, P, P, 1 << 30, NULL), MOE_ERR_INVALID_ARG);
  EXPECT(moe_routed_few(r, P, NULL, MOE_DT_BF16, P, P, P, P, 0, 8, 128, 128, NULL, P, P, 1 << 30, NULL), MOE_ERR_INVALID_ARG);
  EXPECT(moe_routed_few(r, P, NULL, MOE_DT_BF16, P, P, P, P, 0, 8, 128, 128, a, P, P, 64, NULL), MOE_ERR_WORKSPACE);
  EXPECT(moe_routed_few(r, P, NULL, MOE_DT_BF16, P, P, P, P, 0, 8, 130, 128, a, P, P, 1 << 30, NULL), MOE_ERR_UNSUPPORTED);
  r->tokens = MOE_FEW_MAX_TOKENS + 1;
  EXPECT(moe_routed_few(r, P, NULL, MOE_DT_BF16, P, P, P, P, 0, 8, 128, 128, a, P, P, 1 << 30, NULL), MOE_ERR_UNSUPPORTED);
  r->tokens = 0;
  EXPECT(moe_routed_few(r, P, NULL, MOE_DT_BF16, P, P, P, P, 0, 8, 128, 128, a, P, P, 1 << 30, NULL), MOE_OK);
  free(a); free(r);
}

int main(void) {
  norm_checks();
  few_checks();
  mx_checks();
  if (failures) return 1;
  printf("all passed\n");
  return 0;
}
