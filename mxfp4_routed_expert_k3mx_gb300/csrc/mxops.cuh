// mxops.cuh - launchers of the microscaled operators of any shape (mxfmt.cu:
// the formats and the norm, mxprod.cu: the products).
#pragma once

#include "common.cuh"
#include "k3mx_mx.h"

namespace k3mx {

cudaError_t launch_mx_quantize(const Ctx &c, uint8_t *codes, uint8_t *scales, const void *x, int x_bf16, int rows,
                               int cols, int64_t ldx, int format);
cudaError_t launch_mx_dequantize(const Ctx &c, void *y, int y_bf16, const uint8_t *codes, const uint8_t *scales,
                                 int rows, int cols, int format);

struct NormArgs {
    uint8_t *codes, *scales;
    void *sum;                 // or nullptr (no residual)
    uint16_t *normed;          // or nullptr
    const void *x;
    int64_t ldx;
    const void *residual;      // or nullptr
    const uint16_t *g;
    float eps;
    int n_tokens, width;
};
cudaError_t launch_rmsnorm_mx(const Ctx &c, const NormArgs &a, int bf16);

// offsets == nullptr: one group of all rows
struct ProdArgs {
    void *y;
    const uint8_t *codes, *scales;
    const uint8_t *packed, *wscales;
    const int32_t *offsets;
    int n_groups, n_rows, in, out;
    int *status;
};
cudaError_t launch_mx_product(const Ctx &c, const ProdArgs &a, int y_bf16);

}  // namespace k3mx
