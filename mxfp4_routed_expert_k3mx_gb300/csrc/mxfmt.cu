// mxfmt.cu - the microscaled formats: fp32 or bf16 rows to MXFP4 or MXFP8
// codes and scales and back, and the RMSNorm that adds the residual and
// writes MXFP8.
//
// A block of 32 columns is four neighbouring lanes of 8 values, so its
// largest magnitude is 8 compares and two shuffles, and every load and store
// is a whole vector.  All three kernels make one pass over the input and one
// over each output.  Measured (repeated calls, inputs larger than L2, of a
// measured copy of 6.77 TB/s):
//   quantise 12288 x 7168 fp32 to MXFP4    56.9 us, 7.0 TB/s; back 58.7 us, 6.8
//   quantise 4096 x 7168 bf16 to MXFP8     14.8 us, 6.0 TB/s; back 15.0 us, 5.9
//   norm 4096 x 7168 fp32, no normed       60.2 us, 6.4 TB/s
//   norm 4096 x 7168 bf16, with normed     49.6 us, 5.3 TB/s; without 45.2, 4.6
//   one row of 7168 bf16: quantise 1.3 us, back 1.2, norm 2.9 (launch and one
//   or two memory latencies)
// The large fp32 calls are bound by HBM.  The bf16 norm has half the bytes for
// the same values, and the latencies of a row (load, sum, weights, stores) are
// not all hidden by the rows beside it: rows streamed through shared memory
// by bulk copies took 36.5 us without normed where this form took 42.7 at the
// time, but 46.8 and 47.1 with it, 63.8 and 59.1 in fp32, and 31 and 26.4 for
// 8192 x 2048.
#include "mxcode.cuh"
#include "mxops.cuh"

namespace k3mx {
namespace {

// U runs of eight values a lane, a CTA's threads apart: U loads in flight.
constexpr int kFmtThreads = 256;

// FLAT: ldx = cols, the matrix is one line of n8 runs.  Else the grid's y
// walks the rows and its x a row's per_row = cols / 8 runs, so that a run's
// place takes no division (35 us a call with one, 26 without, for 4096 rows of
// 7168 bf16 to MXFP8 and back).
template <int FMT, bool BF16, bool VEC, bool FLAT, int U>
__global__ void __launch_bounds__(kFmtThreads)
k_mx_quantize(uint8_t *codes, uint8_t *scales, const void *x, int64_t n8, int per_row, int64_t ldx, int rows, int *status) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t c0 = (int64_t)blockIdx.x * (kFmtThreads * U) + threadIdx.x;
    int row = FLAT ? 0 : blockIdx.y;
    do {
        const int64_t from = FLAT ? 0 : row * ldx, to = FLAT ? 0 : (int64_t)row * per_row;
        float v[U][8];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int64_t c = c0 + u * kFmtThreads;       // whole blocks: the line is a multiple of 4 runs
#pragma unroll
            for (int j = 0; j < 8; j++) v[u][j] = 0.f;
            if (c < n8) load8<BF16, VEC>(x, from + 8 * c, v[u]);
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int64_t c = c0 + u * kFmtThreads;
            const uint32_t s = encode8<FMT>(v[u], codes, scales, to + c, c < n8);
            if (FMT == K3MX_MXFP4 && s == 255u && c < n8)
                report_status(status, kStatusBadIndex, FLAT ? (int)(c / per_row) : row);
        }
        row += gridDim.y;
    } while (!FLAT && row < rows);
}

template <int FMT, bool BF16, int U>
__global__ void __launch_bounds__(kFmtThreads)
k_mx_dequantize(void *y, const uint8_t *codes, const uint8_t *scales, int64_t n8) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t i0 = (int64_t)blockIdx.x * (kFmtThreads * U) + threadIdx.x;
    uint2 q[U];
    uint32_t s[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int64_t i = i0 + u * kFmtThreads;
        q[u] = make_uint2(0u, 0u);
        s[u] = 0;
        if (i < n8) {
            if (FMT == K3MX_MXFP4) q[u].x = reinterpret_cast<const uint32_t *>(codes)[i];
            else q[u] = reinterpret_cast<const uint2 *>(codes)[i];
            s[u] = scales[i >> 2];
        }
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int64_t i = i0 + u * kFmtThreads;
        float v[8];
        if (FMT == K3MX_MXFP4) {
            uint32_t h[4];
            e2m1x8_to_h2x4(q[u].x, h);
            const float up = s[u] == 255u ? 0.f : e8m0_to_f32(s[u]);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const float2 f = h2_to_f2(h[j]);
                v[2 * j] = f.x * up;
                v[2 * j + 1] = f.y * up;
            }
        } else {
            const float up = s[u] == 255u ? __uint_as_float(0x7FC00000u) : e8m0_to_f32(s[u]);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const uint32_t pair = (j < 2 ? q[u].x : q[u].y) >> (16 * (j & 1));
                uint32_t h2;
                asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h2) : "r"(pair));
                const float2 f = h2_to_f2(h2);
                v[2 * j] = f.x * up;
                v[2 * j + 1] = f.y * up;
            }
        }
        store8<BF16>(y, 8 * i, v, i < n8);
    }
}

// ------------------------------------------------------------------ norm --

// A sum as s + l, l what s was rounded by.
__device__ __forceinline__ void two_sum(float &s, float &l, float a) {
    const float t = s + a, b = t - s;
    l += (s - (t - b)) + (a - b);
    s = t;
}
// s + l of all lanes, or of every `lanes` of them (a power of two), in the same
// order on each
__device__ __forceinline__ void warp_two_sum(float &s, float &l, int lanes) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < lanes) {
            const float s2 = __shfl_xor_sync(0xffffffffu, s, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
            l += l2;
            two_sum(s, l, s2);
        }
}

// The factor of a row whose squares sum to ss + sl: 1 / sqrt(sum / width + eps)
// as k + kl.
__device__ __forceinline__ void norm_factor(float ss, float sl, int width, float eps, float &k, float &kl) {
    const float w = (float)width, q = ss / w, m = q + eps, b = m - q;
    const float ml = ((q - (m - b)) + (eps - b)) + (fmaf(-q, w, ss) + sl) / w;      // what q and m were rounded by
    k = rsqrtf(m);
    const float k2 = k * k;
    kl = 0.5f * k * (fmaf(-m, k2, 1.0f) - m * fmaf(k, k, -k2) - ml * k2);
    if (!(m > 0.f && m < INFINITY)) kl = 0.f;
}

// Eight values times g (k + kl), so that rounding them on to e4m3 or bf16
// rounds the exact products: k's upper 16 bits times g are exact, the rest is
// added in the one rounding, and that goes to the odd one of the two fp32
// neighbours (where the product is none itself), which is never the middle of
// two codes (two directed roundings and a choice: 4096 x 7168 bf16 in 49.9 us,
// 48.3 rounded to the nearest; finding the few doubtful products and mending
// them in a branch took 60).
__device__ __forceinline__ void scale8(float (&v)[8], uint4 g, float k, float kl) {
    const uint32_t gw[4] = {g.x, g.y, g.z, g.w};
    const float kh = __uint_as_float(__float_as_uint(k) & 0xFFFFFF00u);
    kl += k - kh;
    k = kh;
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const float gj = __uint_as_float(j & 1 ? gw[j >> 1] & 0xFFFF0000u : gw[j >> 1] << 16);
        const float gk = gj * k, rest = v[j] * (gj * kl);
        const float down = __fmaf_rd(v[j], gk, rest), up = __fmaf_ru(v[j], gk, rest);
        v[j] = __float_as_uint(down) & 1u ? down : up;
    }
}

// V runs of 8 values a thread, the row in registers between its two uses (the
// sum of squares, then the scaled values): every input is read once, all
// loads of a row at the start.  WARP: a row to a warp, four rows to a CTA of
// 128 threads, no barrier; else a row to a CTA of as many warps as its runs
// need.  EARLY: the weights are loaded with the row, not after its sum.  For
// few rows (to four an SM) that is one latency less (1 row of 7168 2.9 to
// 2.8 us, 300 rows 5.2 to 4.1); many rows all reading the same lines then hold
// up each other's (4096 rows 43 to 51 us).
template <bool WARP, int V, bool BF16, bool EARLY>
__global__ void __launch_bounds__(WARP ? 128 : V == 1 ? 1024 : V == 2 ? 512 : 1024) k_rmsnorm_mx(const NormArgs a) {
    __shared__ float part[32];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, P = WARP ? 32 : blockDim.x;
    const int64_t t = WARP ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
    const int i0 = WARP ? lane : threadIdx.x, per_row = t < a.n_tokens ? a.width / 8 : 0;
    float v[V][8];
#pragma unroll
    for (int p = 0; p < V; p++) {
#pragma unroll
        for (int j = 0; j < 8; j++) v[p][j] = 0.f;
        if (p * P + i0 < per_row) load8<BF16, true>(a.x, t * a.ldx + 8 * (p * P + i0), v[p]);
    }
    uint4 gq[V];
    auto weights = [&](int p) {
        gq[p] = p * P + i0 < per_row ? reinterpret_cast<const uint4 *>(a.g)[p * P + i0] : make_uint4(0u, 0u, 0u, 0u);
    };
    if (EARLY) {
#pragma unroll
        for (int p = 0; p < V; p++) weights(p);
    }
    if (a.residual != nullptr) {
        float r[V][8];
#pragma unroll
        for (int p = 0; p < V; p++) {
#pragma unroll
            for (int j = 0; j < 8; j++) r[p][j] = 0.f;
            if (p * P + i0 < per_row) load8<BF16, true>(a.residual, t * a.width + 8 * (p * P + i0), r[p]);
        }
#pragma unroll
        for (int p = 0; p < V; p++) {
#pragma unroll
            for (int j = 0; j < 8; j++) v[p][j] += r[p][j];
            store8<BF16>(a.sum, t * a.width + 8 * (p * P + i0), v[p], p * P + i0 < per_row);
        }
    }
    // Where many roundings average out (a thread's four parts, a warp's lanes)
    // the sum is plain fp32; where each would be the whole sum's, the low half
    // is kept.
    float ss, sl;
    auto sum_squares = [&](float by) {
        float sq[4] = {};
#pragma unroll
        for (int p = 0; p < V; p++)
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float u = v[p][j] * by;
                sq[j & 3] = fmaf(u, u, sq[j & 3]);
            }
        ss = (sq[0] + sq[1]) + (sq[2] + sq[3]), sl = 0.f;
        if (WARP) {
            warp_two_sum(ss, sl, 32);
        } else {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (lane == 0) part[threadIdx.x >> 5] = ss;
            __syncthreads();
            const int nw = blockDim.x >> 5, lanes = nw == 1 ? 1 : 1 << (32 - __clz(nw - 1));
            ss = (lane & (lanes - 1)) < nw ? part[lane & (lanes - 1)] : 0.f;
            warp_two_sum(ss, sl, lanes);
        }
    };
    sum_squares(1.f);
    float k, kl;
    if (ss + a.eps < INFINITY) {
        norm_factor(ss, sl, a.width, a.eps, k, kl);
    } else {                              // (a branch that costs 4096 x 7168 bf16 0.8 us)
        // The squares' sum leaves fp32 (values from 2^56 on do, in wide rows): it
        // is formed again of 2^-72 times the values, below 2^128 for any finite
        // ones, and what is lost at its lower end is below 2^-90 of it.  The
        // same for every thread of the row.
        if (!WARP) __syncthreads();                       // part[] has been read
        sum_squares(0x1p-72f);
        norm_factor(ss, sl, a.width, a.eps * 0x1p-144f, k, kl);
        k *= 0x1p-72f, kl *= 0x1p-72f;
    }
#pragma unroll
    for (int p = 0; p < V; p++) {
        const int i = p * P + i0;
        const bool live = i < per_row;
        if (!EARLY) weights(p);
        if (live) {
            scale8(v[p], gq[p], k, kl);
            if (a.normed != nullptr) store8<true>(a.normed, t * a.width + 8 * i, v[p], true);
        }
        encode8<K3MX_MXFP8>(v[p], a.codes, a.scales, t * per_row + i, live);
    }
}

template <bool WARP, int V>
cudaError_t norm_t(const Ctx &c, const NormArgs &a, int bf16) {
    const int warps = WARP ? 4 : (a.width / 8 + 32 * V - 1) / (32 * V);
    const dim3 grid((unsigned)(WARP ? (a.n_tokens + 3) / 4 : a.n_tokens)), block(32 * warps);
    auto go = [&](auto kernel) { return launch_pdl(kernel, grid, block, 0, c.stream, a); };
    constexpr bool kFewRows = !WARP && V == 1, kWide = !WARP && V == 4;       // (kWide has no registers left for it)
    if constexpr (!kWide)
        if (kFewRows || a.n_tokens <= 4 * c.num_sms)
            return bf16 ? go(k_rmsnorm_mx<WARP, V, true, true>) : go(k_rmsnorm_mx<WARP, V, false, true>);
    if constexpr (!kFewRows)
        return bf16 ? go(k_rmsnorm_mx<WARP, V, true, false>) : go(k_rmsnorm_mx<WARP, V, false, false>);
}

}  // namespace

// Runs a lane: four where that still fills the device several times over.
static bool many_runs(const Ctx &c, int64_t n8) { return n8 >= (int64_t)c.num_sms * 8 * kFmtThreads * 4; }

template <int FMT, bool BF16>
static cudaError_t quantize_t(const Ctx &c, uint8_t *codes, uint8_t *scales, const void *x, int rows, int cols,
                              int64_t ldx) {
    const int64_t n8 = (int64_t)rows * cols / 8;
    const bool vec = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && (ldx * (BF16 ? 2 : 4)) % 16 == 0;
    // a line of `n` runs, `lines` of them
    auto go = [&](auto kernel, int U, int64_t n, int lines) {
        const dim3 grid((unsigned)((n + kFmtThreads * U - 1) / (kFmtThreads * U)), (unsigned)(lines < 65535 ? lines : 65535));
        return launch_pdl(kernel, grid, dim3(kFmtThreads), 0, c.stream, codes, scales, x, n, cols / 8, ldx, lines, c.status);
    };
    if (!vec) return go(k_mx_quantize<FMT, BF16, false, false, 1>, 1, cols / 8, rows);
    if (ldx != cols)
        return cols / 8 > kFmtThreads && many_runs(c, n8) ? go(k_mx_quantize<FMT, BF16, true, false, 4>, 4, cols / 8, rows)
                                                          : go(k_mx_quantize<FMT, BF16, true, false, 1>, 1, cols / 8, rows);
    return many_runs(c, n8) ? go(k_mx_quantize<FMT, BF16, true, true, 4>, 4, n8, 1)
                            : go(k_mx_quantize<FMT, BF16, true, true, 1>, 1, n8, 1);
}

cudaError_t launch_mx_quantize(const Ctx &c, uint8_t *codes, uint8_t *scales, const void *x, int x_bf16, int rows,
                               int cols, int64_t ldx, int format) {
    if (format == K3MX_MXFP4)
        return x_bf16 ? quantize_t<K3MX_MXFP4, true>(c, codes, scales, x, rows, cols, ldx)
                      : quantize_t<K3MX_MXFP4, false>(c, codes, scales, x, rows, cols, ldx);
    return x_bf16 ? quantize_t<K3MX_MXFP8, true>(c, codes, scales, x, rows, cols, ldx)
                  : quantize_t<K3MX_MXFP8, false>(c, codes, scales, x, rows, cols, ldx);
}

template <int FMT, bool BF16>
static cudaError_t dequantize_t(const Ctx &c, void *y, const uint8_t *codes, const uint8_t *scales, int rows, int cols) {
    const int64_t n8 = (int64_t)rows * cols / 8;
    auto go = [&](auto kernel, int U) {
        const dim3 grid((unsigned)((n8 + kFmtThreads * U - 1) / (kFmtThreads * U)));
        return launch_pdl(kernel, grid, dim3(kFmtThreads), 0, c.stream, y, codes, scales, n8);
    };
    return many_runs(c, n8) ? go(k_mx_dequantize<FMT, BF16, 4>, 4) : go(k_mx_dequantize<FMT, BF16, 1>, 1);
}

cudaError_t launch_mx_dequantize(const Ctx &c, void *y, int y_bf16, const uint8_t *codes, const uint8_t *scales,
                                 int rows, int cols, int format) {
    if (format == K3MX_MXFP4)
        return y_bf16 ? dequantize_t<K3MX_MXFP4, true>(c, y, codes, scales, rows, cols)
                      : dequantize_t<K3MX_MXFP4, false>(c, y, codes, scales, rows, cols);
    return y_bf16 ? dequantize_t<K3MX_MXFP8, true>(c, y, codes, scales, rows, cols)
                  : dequantize_t<K3MX_MXFP8, false>(c, y, codes, scales, rows, cols);
}

cudaError_t launch_rmsnorm_mx(const Ctx &c, const NormArgs &a, int bf16) {
    const int n8 = a.width / 8;
    if (n8 <= 32) return norm_t<true, 1>(c, a, bf16);
    if (n8 <= 128) return norm_t<true, 4>(c, a, bf16);
    // few rows: the fewest values a thread; many: two runs a thread, so that
    // several rows share an SM
    if (n8 <= 1024) return a.n_tokens <= c.num_sms ? norm_t<false, 1>(c, a, bf16) : norm_t<false, 2>(c, a, bf16);
    return norm_t<false, 4>(c, a, bf16);
}

}  // namespace k3mx
