// mxfmt.cu - the microscaled formats: fp32 or bf16 rows to MXFP4 or MXFP8
// codes and scales and back, and the RMSNorm that adds the residual and
// writes MXFP8.
//
// A block of 32 columns is four neighbouring lanes of 8 values, so its
// largest magnitude is 8 compares and two shuffles, and every load and store
// is a whole vector.  All three kernels are bound by HBM: one pass over the
// input, one over each output.
#include "mxops.cuh"
#include "pieces.cuh"

namespace k3mx {
namespace {

// ------------------------------------------------------------ loads, stores --

// 8 consecutive values; VEC: the address is a multiple of 16 bytes
template <bool BF16, bool VEC>
__device__ __forceinline__ void load8(const void *base, int64_t i, float (&v)[8]) {
    if (BF16) {
        const uint16_t *p = static_cast<const uint16_t *>(base) + i;
        if (VEC) {
            const uint4 q = *reinterpret_cast<const uint4 *>(p);
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < 4; j++) {
                v[2 * j] = __uint_as_float(w[j] << 16);
                v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] = __uint_as_float((uint32_t)p[j] << 16);
        }
    } else {
        const float *p = static_cast<const float *>(base) + i;
        if (VEC) {
            const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
            v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] = p[j];
        }
    }
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <bool BF16>
__device__ __forceinline__ void store8(void *base, int64_t i, const float (&v)[8]) {
    if (BF16) {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + i) =
            make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
    } else {
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + i);
        p[0] = make_float4(v[0], v[1], v[2], v[3]);
        p[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}

// ------------------------------------------------------------- one block --

// The ue8m0 byte of a block whose largest magnitude has bits mb: the smallest
// e >= -127 with max <= TOP * 2^e, TOP = 1.5 * 2^2 (e2m1) or 1.75 * 2^8
// (e4m3); 255 for Inf and NaN, 0 for an all-zero block.  `down` is 2^-e.
// A subnormal maximum is below 2^-126 <= TOP * 2^-127: e = -127.
template <int FMT>
__device__ __forceinline__ uint32_t block_scale(uint32_t mb, float &down) {
    constexpr uint32_t kTopMant = FMT == K3MX_MXFP4 ? 0x400000u : 0x600000u;
    constexpr int kTopExp = FMT == K3MX_MXFP4 ? 2 : 8;
    const int E = (int)(mb >> 23) - 127;
    if (E == 128) {
        down = 0.f;
        return 255u;
    }
    const int e = mb == 0 ? -127 : max((mb & 0x7FFFFFu) <= kTopMant ? E - kTopExp : E - kTopExp + 1, -127);
    down = exp2i(-e);                       // -e is in -125 .. 127
    return (uint32_t)(e + 127);
}

// 8 values of a block already divided by its scale -> 8 e4m3 bytes
__device__ __forceinline__ uint2 to_e4m3x8(const float (&v)[8]) {
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; k++)
        asm("{\n\t.reg .b16 a, b;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
            "mov.b32 %0, {a, b};\n\t}"
            : "=r"(w[k])
            : "f"(v[4 * k]), "f"(v[4 * k + 1]), "f"(v[4 * k + 2]), "f"(v[4 * k + 3]));
    return make_uint2(w[0], w[1]);
}
// the same -> 8 e2m1 codes (the low nibble of byte j is value 2 j)
__device__ __forceinline__ uint32_t to_e2m1x8(const float (&v)[8]) {
    uint32_t w;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return w;
}

// largest |v| of the block (four lanes x 8 values) as fp32 bits: non-negative
// floats order as their bit patterns, Inf and NaN above every finite value
__device__ __forceinline__ uint32_t block_max(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; j++) m = max(m, __float_as_uint(fabsf(v[j])));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// One lane's 8 values (quarter q8 of the matrix in row-major order) into the
// codes, the block's byte by its first lane; whole warps.
template <int FMT>
__device__ __forceinline__ uint32_t encode8(float (&v)[8], uint8_t *codes, uint8_t *scales, int64_t q8, bool live) {
    float down;
    const uint32_t s = block_scale<FMT>(block_max(v), down);
    // 2^-e times a value is exact (or, for the smallest values, below half
    // the smallest code); a dropped block's codes are zero
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = s == 255u ? 0.f : v[j] * down;
    if (live) {
        if (FMT == K3MX_MXFP4) reinterpret_cast<uint32_t *>(codes)[q8] = to_e2m1x8(v);
        else reinterpret_cast<uint2 *>(codes)[q8] = to_e4m3x8(v);
        if ((q8 & 3) == 0) scales[q8 >> 2] = (uint8_t)s;
    }
    return s;
}

constexpr int kFmtThreads = 256;

// Eight values a lane.  x rows ldx apart; `per_row` = cols / 8 lanes to a row.
template <int FMT, bool BF16, bool VEC>
__global__ void __launch_bounds__(kFmtThreads)
k_mx_quantize(uint8_t *codes, uint8_t *scales, const void *x, int64_t n8, int per_row, int64_t ldx, int *status) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t i = (int64_t)blockIdx.x * kFmtThreads + threadIdx.x;
    const bool live = i < n8;               // whole blocks: n8 is a multiple of 4
    const int64_t row = live ? i / per_row : 0;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (live) load8<BF16, VEC>(x, row * ldx + (i - row * per_row) * 8, v);
    const uint32_t s = encode8<FMT>(v, codes, scales, i, live);
    if (FMT == K3MX_MXFP4 && live && s == 255u) report_status(status, kStatusBadIndex, (int)row);
}

template <int FMT, bool BF16>
__global__ void __launch_bounds__(kFmtThreads)
k_mx_dequantize(void *y, const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int64_t n8) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t i = (int64_t)blockIdx.x * kFmtThreads + threadIdx.x;
    if (i >= n8) return;
    const uint32_t s = scales[i >> 2];
    float v[8];
    if (FMT == K3MX_MXFP4) {
        uint32_t h[4];
        e2m1x8_to_h2x4(reinterpret_cast<const uint32_t *>(codes)[i], h);
        const float up = s == 255u ? 0.f : e8m0_to_f32(s);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const float2 f = h2_to_f2(h[j]);
            v[2 * j] = f.x * up;
            v[2 * j + 1] = f.y * up;
        }
    } else {
        const uint2 q = reinterpret_cast<const uint2 *>(codes)[i];
        const float up = s == 255u ? __uint_as_float(0x7FC00000u) : e8m0_to_f32(s);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint32_t pair = (j < 2 ? q.x : q.y) >> (16 * (j & 1));
            uint32_t h2;
            asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h2) : "r"(pair));
            const float2 f = h2_to_f2(h2);
            v[2 * j] = f.x * up;
            v[2 * j + 1] = f.y * up;
        }
    }
    store8<BF16>(y, 8 * i, v);
}

// ------------------------------------------------------------------ norm --

// One row per CTA of 1024 threads, the row in registers (8 values a lane and
// pass, up to 4 passes).
constexpr int kNormThreads = 1024, kNormVec = 4;

template <bool BF16>
__global__ void __launch_bounds__(kNormThreads) k_rmsnorm_mx(const NormArgs a) {
    __shared__ float part[kNormThreads / 32];
    pdl_launch_dependents();
    pdl_wait();
    const int64_t t = blockIdx.x;
    const int per_row = a.width / 8;
    float v[kNormVec][8];
    float ss = 0.f;
#pragma unroll
    for (int p = 0; p < kNormVec; p++) {
        const int i = p * kNormThreads + threadIdx.x;
#pragma unroll
        for (int j = 0; j < 8; j++) v[p][j] = 0.f;
        if (i < per_row) {
            load8<BF16, true>(a.x, t * a.ldx + 8 * i, v[p]);
            if (a.residual != nullptr) {
                float r[8];
                load8<BF16, true>(a.residual, t * a.width + 8 * i, r);
#pragma unroll
                for (int j = 0; j < 8; j++) v[p][j] += r[j];
                store8<BF16>(a.sum, t * a.width + 8 * i, v[p]);
            }
#pragma unroll
            for (int j = 0; j < 8; j++) ss = fmaf(v[p][j], v[p][j], ss);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ss;
    __syncthreads();
    ss = 0.f;
#pragma unroll
    for (int w = 0; w < kNormThreads / 32; w++) ss += part[w];
    const float k = 1.0f / sqrtf(ss / (float)a.width + a.eps);
#pragma unroll
    for (int p = 0; p < kNormVec; p++) {
        const int i = p * kNormThreads + threadIdx.x;
        if (p * kNormThreads >= per_row) break;
        const bool live = i < per_row;
        if (live) {
            float g[8];
            load8<true, true>(a.g, 8 * i, g);
#pragma unroll
            for (int j = 0; j < 8; j++) v[p][j] = v[p][j] * k * g[j];
            if (a.normed != nullptr) store8<true>(a.normed, t * a.width + 8 * i, v[p]);
        }
        encode8<K3MX_MXFP8>(v[p], a.codes, a.scales, t * per_row + i, live);
    }
}

}  // namespace

cudaError_t launch_mx_quantize(const Ctx &c, uint8_t *codes, uint8_t *scales, const void *x, int x_bf16, int rows,
                               int cols, int64_t ldx, int format) {
    const int64_t n8 = (int64_t)rows * cols / 8;
    const dim3 grid((unsigned)((n8 + kFmtThreads - 1) / kFmtThreads));
    const bool vec = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && (ldx * (x_bf16 ? 2 : 4)) % 16 == 0;
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, grid, dim3(kFmtThreads), 0, c.stream, codes, scales, x, n8, cols / 8, ldx, c.status);
    };
    if (format == K3MX_MXFP4) {
        if (x_bf16) return vec ? go(k_mx_quantize<K3MX_MXFP4, true, true>) : go(k_mx_quantize<K3MX_MXFP4, true, false>);
        return vec ? go(k_mx_quantize<K3MX_MXFP4, false, true>) : go(k_mx_quantize<K3MX_MXFP4, false, false>);
    }
    if (x_bf16) return vec ? go(k_mx_quantize<K3MX_MXFP8, true, true>) : go(k_mx_quantize<K3MX_MXFP8, true, false>);
    return vec ? go(k_mx_quantize<K3MX_MXFP8, false, true>) : go(k_mx_quantize<K3MX_MXFP8, false, false>);
}

cudaError_t launch_mx_dequantize(const Ctx &c, void *y, int y_bf16, const uint8_t *codes, const uint8_t *scales,
                                 int rows, int cols, int format) {
    const int64_t n8 = (int64_t)rows * cols / 8;
    const dim3 grid((unsigned)((n8 + kFmtThreads - 1) / kFmtThreads));
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, grid, dim3(kFmtThreads), 0, c.stream, y, codes, scales, n8);
    };
    if (format == K3MX_MXFP4) return y_bf16 ? go(k_mx_dequantize<K3MX_MXFP4, true>) : go(k_mx_dequantize<K3MX_MXFP4, false>);
    return y_bf16 ? go(k_mx_dequantize<K3MX_MXFP8, true>) : go(k_mx_dequantize<K3MX_MXFP8, false>);
}

cudaError_t launch_rmsnorm_mx(const Ctx &c, const NormArgs &a, int bf16) {
    const dim3 grid((unsigned)a.n_tokens);
    return bf16 ? launch_pdl(k_rmsnorm_mx<true>, grid, dim3(kNormThreads), 0, c.stream, a)
                : launch_pdl(k_rmsnorm_mx<false>, grid, dim3(kNormThreads), 0, c.stream, a);
}

}  // namespace k3mx
