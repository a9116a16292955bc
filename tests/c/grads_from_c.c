/* A plain C caller of the gradient norm, clipping, all-reduce with norm and
 * AdamW entry points: workspace sizes and refusals, with no GPU work (every
 * call below returns before any launch; the addresses are never
 * dereferenced).  Built and run by tests/test_c_grads.py; prints one line per
 * check and exits non-zero on the first failure. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "ddp_allreduce.h"

#define CHECK(cond, what)                                              \
    do {                                                               \
        if (!(cond)) {                                                 \
            printf("FAIL %s (last error: %s)\n", what, ddp_last_error()); \
            return 1;                                                  \
        }                                                              \
        printf("ok %s\n", what);                                       \
    } while (0)

#define AT(k) ((void*)(0x7f0000000000ull + ((uint64_t)(k) << 24)))

int main(void) {
    const int64_t numels[2] = {1000000, 7};
    const int32_t types[2] = {DDP_BF16, DDP_F32};
    const void* g[2] = {AT(0), AT(1)};
    void* out[2] = {AT(2), AT(3)};
    void* same[2] = {AT(0), AT(0)};
    void* ws = AT(20);
    float* norm = AT(21);
    int64_t bytes = -1;

    CHECK(grad_norm_workspace_bytes(2, numels, g, types, &bytes) == DDP_OK && bytes == DDP_NORM_WORKSPACE_BYTES,
          "workspace of a large set");
    CHECK(grad_norm_workspace_bytes(1, numels + 1, g + 1, types + 1, &bytes) == DDP_OK && bytes == 0,
          "no workspace for a small one");
    CHECK(grad_norm_multi(2, numels, g, types, NULL, 0, norm, NULL) == DDP_E_ARG &&
              strstr(ddp_last_error(), "workspace") != NULL, "norm without its workspace");
    CHECK(grad_norm_multi(2, numels, g, types, ws, 16, norm, NULL) == DDP_E_ARG, "norm with a short workspace");
    CHECK(grad_norm_multi(2, numels, g, types, ws, bytes = 1 << 20, NULL, NULL) == DDP_E_ARG, "norm without a result");
    CHECK(grad_norm_multi(0, numels, g, types, ws, bytes, norm, NULL) == DDP_E_ARG, "no tensor");
    CHECK(grad_clip_multi(2, numels, g, types, same, 1.0, 0, norm, ws, bytes, NULL) == DDP_E_OVERLAP,
          "two outputs in one place");
    CHECK(grad_clip_multi(2, numels, g, types, out, -1.0, 0, norm, ws, bytes, NULL) == DDP_E_ARG, "negative limit");
    CHECK(grad_clip_multi(2, numels, g, types, out, NAN, 1, norm, NULL, 0, NULL) == DDP_E_ARG, "limit not a number");
    CHECK(grad_clip_multi(2, numels, g, types, NULL, 1.0, 0, norm, ws, bytes, NULL) == DDP_E_ARG, "no outputs");

    CHECK(allreduce_norm_workspace_bytes(8, 8, DDP_F32, DDP_F32, 256 * 1000, 0, &bytes) == DDP_OK && bytes == 8000,
          "a partial sum per workgroup");
    CHECK(allreduce_norm_workspace_bytes(17, 8, DDP_F32, DDP_F32, 256, 0, &bytes) == DDP_E_ARG, "17 ranks");
    const void* in[2] = {AT(0), AT(1)};
    CHECK(allreduce_ring_norm(DDP_MEAN, 2, 2, in, DDP_F32, 3, out, DDP_F32, 1000, norm, ws, 1 << 20, NULL) == DDP_E_ARG,
          "three results of two ranks");
    CHECK(allreduce_ring_norm(DDP_MEAN, 2, 2, in, DDP_F32, 1, out, DDP_F32, 1000, norm, AT(0), 1 << 20, NULL) ==
              DDP_E_OVERLAP, "workspace over an input");
    CHECK(allreduce_ring_norm_buckets(DDP_MEAN, 2, 2, in, DDP_F32, 2, out, DDP_F32, 1000, 0, norm, ws, 1 << 20,
                                      NULL) == DDP_E_ARG, "buckets of nothing");

    float* w[2] = {AT(4), AT(5)};
    float* m[2] = {AT(6), AT(7)};
    float* v[2] = {AT(8), AT(9)};
    CHECK(adamw_step_multi(2, numels, g, DDP_BF16, w, m, m, NULL, DDP_BF16, 1e-3, 0.9, 0.999, 1e-8, 0.01, 1, NULL,
                           NULL, 0.0, NULL) == DDP_E_OVERLAP, "one buffer for both moments");
    CHECK(adamw_step_multi(2, numels, g, DDP_BF16, w, m, v, NULL, DDP_BF16, 1e-3, 0.9, 1.0, 1e-8, 0.01, 1, NULL,
                           NULL, 0.0, NULL) == DDP_E_ARG, "beta2 = 1");
    CHECK(adamw_step_multi(2, numels, g, DDP_BF16, w, m, v, NULL, DDP_BF16, 1e-3, 0.9, 0.999, 1e-8, 0.01, 0, NULL,
                           NULL, 0.0, NULL) == DDP_E_ARG, "step 0");
    printf("all checks passed\n");
    return 0;
}
