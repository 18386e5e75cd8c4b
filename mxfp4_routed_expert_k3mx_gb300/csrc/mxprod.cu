// mxprod.cu - products of MXFP8 activations with MXFP4 weights of any shape,
// dense or by groups of rows with a weight matrix each.
#include "mxops.cuh"

namespace k3mx {
namespace {

constexpr int kRows = 8;                  // rows of a unit
constexpr int kWarps = 8;                 // outputs of a CTA

// One warp per (unit, output): lane l takes the 32-column blocks l, l + 32,
// ... for all rows of the unit; the warp's sums meet in shuffles.  Unit u is
// the u-th run of at most kRows rows counting group by group.
template <bool BF16>
__global__ void __launch_bounds__(kWarps * 32) k_mx_product(const ProdArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int tiles = (a.out + kWarps - 1) / kWarps;
    int g = 0, r0 = 0, r1 = 0, u = (int)(blockIdx.x / tiles);
    if (blockIdx.x == 0 && a.offsets)
        for (int k = threadIdx.x; k < a.n_groups; k += kWarps * 32)
            if (a.offsets[k] < 0 || a.offsets[k + 1] < a.offsets[k] || a.offsets[k + 1] > a.n_rows)
                report_status(a.status, kStatusBadIndex, k);
    for (; g < a.n_groups; g++) {
        const int lo = a.offsets ? a.offsets[g] : 0, hi = a.offsets ? a.offsets[g + 1] : a.n_rows;
        if (lo < 0 || hi < lo || hi > a.n_rows) continue;
        const int n = (hi - lo + kRows - 1) / kRows;
        if (u < n) {
            r0 = lo + u * kRows;
            r1 = min(hi, r0 + kRows);
            break;
        }
        u -= n;
    }
    const int o = (int)(blockIdx.x % tiles) * kWarps + (threadIdx.x >> 5);
    if (g == a.n_groups || o >= a.out) return;
    const int G = a.in / 32;
    const uint8_t *w = a.packed + ((size_t)g * a.out + o) * (a.in / 2);
    const uint8_t *ws = a.wscales + ((size_t)g * a.out + o) * G;
    float acc[kRows] = {};
    for (int b = lane; b < G; b += 32) {
        // a dropped block's codes count as zeros, so a NaN in x still shows
        uint4 q = *reinterpret_cast<const uint4 *>(w + (size_t)b * 16);
        const uint32_t s = ws[b];
        if (s == 255u) q = make_uint4(0u, 0u, 0u, 0u);
        const float k = s == 255u ? 1.f : e8m0_to_f32(s);
        for (int r = r0; r < r1; r++) {
            const uint8_t *xc = a.codes + (size_t)r * a.in + (size_t)b * 32;
            const uint32_t sx = a.scales[(size_t)r * G + b];
            float2 x[16];
#pragma unroll
            for (int j = 0; j < 16; j++) {
                uint32_t h2;
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(reinterpret_cast<const uint16_t *>(xc)[j]));
                x[j] = h2_to_f2(h2);
            }
            const float up = sx == 255u ? __uint_as_float(0x7FC00000u) : e8m0_to_f32(sx);
            acc[r - r0] += group_dot(q, x) * k * up;
        }
    }
    for (int r = r0; r < r1; r++) {
        float v = acc[r - r0];
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
        if (lane == 0) {
            if (BF16) static_cast<__nv_bfloat16 *>(a.y)[(size_t)r * a.out + o] = __float2bfloat16_rn(v);
            else static_cast<float *>(a.y)[(size_t)r * a.out + o] = v;
        }
    }
}

}  // namespace

cudaError_t launch_mx_product(const Ctx &c, const ProdArgs &a, int y_bf16) {
    const int64_t ctas = (int64_t)(a.n_rows / kRows + a.n_groups) * ((a.out + kWarps - 1) / kWarps);
    if (ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)ctas);
    return y_bf16 ? launch_pdl(k_mx_product<true>, grid, dim3(kWarps * 32), 0, c.stream, a)
                  : launch_pdl(k_mx_product<false>, grid, dim3(kWarps * 32), 0, c.stream, a);
}

}  // namespace k3mx
