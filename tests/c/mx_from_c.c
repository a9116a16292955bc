/* A plain C caller of the 4-bit gradient and 8-bit moment entry points:
 * workspace sizes and refusals, with no GPU work (every call below returns
 * before any launch; the addresses are never dereferenced).  Built and run by
 * tests/test_c_mx.py; prints one line per check and exits non-zero on the
 * first failure. */
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
    const void* in[2] = {AT(0), AT(1)};
    void* left[2] = {AT(2), AT(3)};
    uint8_t* codes[2] = {AT(4), AT(5)};
    uint8_t* scales[2] = {AT(6), AT(7)};
    const uint8_t* const rcodes[2] = {AT(4), AT(5)};
    const uint8_t* const rscales[2] = {AT(6), AT(7)};
    uint8_t* same[2] = {AT(4), AT(4)};
    uint8_t* odd[2] = {(uint8_t*)AT(4) + 8, AT(5)};
    void* out[2] = {AT(8), AT(9)};
    const int64_t n = 1000;
    int64_t bytes = -1;

    CHECK(DDP_MX_BLOCK == 32, "block size");
    CHECK(mx4_quantize(2, in, DDP_BF16, 0, NULL, DDP_F32, NULL, NULL, NULL) == DDP_OK, "nothing to quantise");
    CHECK(mx4_quantize(2, in, DDP_BF16, n, left, DDP_F32, same, scales, NULL) == DDP_E_OVERLAP, "codes of two ranks in one place");
    CHECK(mx4_quantize(2, in, DDP_BF16, n, left, DDP_F32, odd, scales, NULL) == DDP_E_ALIGN, "codes off a 16-byte line");
    CHECK(mx4_quantize(17, in, DDP_BF16, n, left, DDP_F32, codes, scales, NULL) == DDP_E_ARG, "17 ranks");
    CHECK(mx4_dequantize(2, rcodes, rscales, n, NULL, DDP_F32, NULL) == DDP_E_ARG &&
              strstr(ddp_last_error(), "rank_out") != NULL, "no outputs");

    CHECK(allreduce_mx4_workspace_bytes(2048 * 1000, &bytes) == DDP_OK && bytes == 8000, "a partial sum per workgroup");
    CHECK(allreduce_mx4_workspace_bytes(-1, &bytes) == DDP_E_ARG, "negative length");
    CHECK(allreduce_mx4(DDP_MEAN, 2, rcodes, rscales, n, 2, out, DDP_F32, AT(20), AT(21), 4, NULL) == DDP_E_ARG &&
              strstr(ddp_last_error(), "workspace") != NULL, "a short workspace");
    CHECK(allreduce_mx4(DDP_MEAN, 2, rcodes, rscales, n, 3, out, DDP_F32, NULL, NULL, 0, NULL) == DDP_E_ARG, "three results of two ranks");
    CHECK(allreduce_mx4_coded(DDP_MEAN, 2, rcodes, rscales, n, 1, codes, scales, AT(4), DDP_F32, NULL, NULL, 0, NULL) ==
              DDP_E_OVERLAP, "residual over codes");
    CHECK(allreduce_mx4_coded(DDP_MEAN, 2, rcodes, rscales, n, 1, odd, scales, NULL, DDP_F32, NULL, NULL, 0, NULL) ==
              DDP_E_ALIGN, "codes half over codes");

    const int64_t numels[2] = {1000000, 7};
    float* w[2] = {AT(10), AT(11)};
    uint8_t* m[2] = {AT(12), AT(13)};
    uint8_t* v[2] = {AT(14), AT(15)};
    uint8_t* s[2] = {AT(16), AT(17)};
    CHECK(adamw8_step_multi(2, numels, in, DDP_BF16, w, m, m, s, NULL, DDP_BF16, 1e-3, 0.9, 0.999, 1e-8, 0.01, 1, NULL, 0,
                            NULL, 0.0, NULL) == DDP_E_OVERLAP, "one buffer for both moments");
    CHECK(adamw8_step_multi(2, numels, in, DDP_BF16, w, m, v, NULL, NULL, DDP_BF16, 1e-3, 0.9, 0.999, 1e-8, 0.01, 1, NULL,
                            0, NULL, 0.0, NULL) == DDP_E_ARG, "no scales");
    CHECK(adamw8_read_multi(2, numels, rcodes, rcodes, rscales, out, out, DDP_F32, NULL) == DDP_E_OVERLAP,
          "both moments read into one place");
    printf("all checks passed\n");
    return 0;
}
