// blockops.cuh - launchers of the steps between an expert block's products
// (block.cu: pairs by expert, rows there and back; situ.cu: the activation
// and the norm's gradient).
#pragma once

#include "common.cuh"
#include "k3mx_block.h"

namespace k3mx {

size_t sort_scratch_bytes(int n_pairs, int n_experts);
cudaError_t launch_sort(const Ctx &c, int32_t *offsets, int32_t *perm, int32_t *place, const int32_t *idx, int n_pairs,
                        int n_experts, void *scratch);

struct DispatchArgs {
    void *rows;
    uint8_t *scales;           // or nullptr
    const void *x;
    const uint8_t *x_scales;   // or nullptr
    int64_t ldx;               // elements
    int elem;                  // bytes of one
    const int32_t *place;
    int n_tokens, topk, n_rows, width;
    int *status;
};
cudaError_t launch_dispatch(const Ctx &c, const DispatchArgs &a);

struct CombineArgs {
    void *y;
    const void *rows;
    const int32_t *place;
    const float *w;            // or nullptr
    const void *base;          // or nullptr
    int n_tokens, topk, n_rows, width;
    int *status;
};
cudaError_t launch_combine(const Ctx &c, const CombineArgs &a, int y_bf16, int rows_bf16);

struct CombineGradArgs {
    void *drows;
    float *dw;
    const void *dy;
    int64_t lddy;
    const void *rows;
    const int32_t *place;
    const float *w;
    int n_tokens, topk, n_rows, width;
    int *status;
};
cudaError_t launch_combine_grad(const Ctx &c, const CombineGradArgs &a, int dy_bf16, int rows_bf16);

struct SituArgs {
    uint8_t *codes, *scales;
    uint8_t *saved, *saved_scales;     // or nullptr
    const void *gu;
    int64_t ldgu;
    int rows, inter;
};
cudaError_t launch_situ(const Ctx &c, const SituArgs &a, int bf16);

struct SituGradArgs {
    void *dgu;
    const void *dh;
    int64_t lddh;
    const uint8_t *saved, *saved_scales;
    int rows, inter;
};
cudaError_t launch_situ_grad(const Ctx &c, const SituGradArgs &a, int bf16);

struct NormGradArgs {
    void *dx;
    float *dweight, *part;
    const void *dn;
    int64_t lddn;
    const void *dres;          // or nullptr
    const uint8_t *saved, *saved_scales;
    const uint16_t *g;
    float eps;
    int n_tokens, width;
};
size_t norm_grad_scratch_bytes(int n_tokens, int width);
cudaError_t launch_norm_grad(const Ctx &c, const NormGradArgs &a, int bf16);

}  // namespace k3mx
