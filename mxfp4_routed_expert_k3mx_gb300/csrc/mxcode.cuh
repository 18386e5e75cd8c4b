// mxcode.cuh - eight values a lane, four lanes a block of 32 columns: loads,
// stores and the conversion to the microscaled formats (mxfmt.cu and the steps
// of an expert block).
#pragma once

#include "mxops.cuh"
#include "pieces.cuh"

namespace k3mx {

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
// 8 consecutive values a lane, neighbouring lanes neighbouring runs, both of a
// pair live or neither; whole warps.  fp32: the lanes of a pair swap halves,
// so that each store instruction writes whole 32-byte sectors.
template <bool BF16>
__device__ __forceinline__ void store8(void *base, int64_t i, const float (&v)[8], bool live) {
    if (BF16) {
        if (live) *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + i) =
            make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
    } else {
        const bool odd = threadIdx.x & 1;
        float4 t;
        t.x = __shfl_xor_sync(0xffffffffu, odd ? v[0] : v[4], 1);
        t.y = __shfl_xor_sync(0xffffffffu, odd ? v[1] : v[5], 1);
        t.z = __shfl_xor_sync(0xffffffffu, odd ? v[2] : v[6], 1);
        t.w = __shfl_xor_sync(0xffffffffu, odd ? v[3] : v[7], 1);
        // even: own first half and the neighbour's, odd: the neighbour's second half and its own
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + (odd ? i - 8 : i));
        if (live) {
            p[odd ? 1 : 0] = odd ? t : make_float4(v[0], v[1], v[2], v[3]);
            p[odd ? 3 : 2] = odd ? make_float4(v[4], v[5], v[6], v[7]) : t;
        }
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

// largest of three magnitudes, NaN if one is
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
    float m;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}
// largest |v| of the block (four lanes x 8 values) as fp32 bits: non-negative
// floats order as their bit patterns, Inf and NaN above every finite value
__device__ __forceinline__ uint32_t block_max(const float (&v)[8]) {
    const float a = max_abs3(v[0], v[1], v[2]), b = max_abs3(v[3], v[4], v[5]);
    uint32_t m = __float_as_uint(max_abs3(a, b, max_abs3(v[6], v[7], v[7]))) & 0x7FFFFFFFu;
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
    const uint32_t keep = s == 255u ? 0u : 0xFFFFFFFFu;
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] *= down;
    if (live) {
        if (FMT == K3MX_MXFP4) {
            reinterpret_cast<uint32_t *>(codes)[q8] = to_e2m1x8(v) & keep;
        } else {
            const uint2 w = to_e4m3x8(v);
            reinterpret_cast<uint2 *>(codes)[q8] = make_uint2(w.x & keep, w.y & keep);
        }
        if ((q8 & 3) == 0) scales[q8 >> 2] = (uint8_t)s;
    }
    return s;
}

__device__ __forceinline__ float at_least(float x, float least) {        // NaN stays NaN
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(least));
    return y;
}
// Eight values as they lie in memory
template <bool BF16> struct Raw {
    uint4 q[BF16 ? 1 : 2];
    __device__ __forceinline__ void load(const void *base, int64_t i) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(base) + i * (BF16 ? 2 : 4));
        q[0] = p[0];
        if (!BF16) q[BF16 ? 0 : 1] = p[1];
    }
    __device__ __forceinline__ void zero() { q[0] = q[BF16 ? 0 : 1] = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void minus_zero() {
        constexpr uint32_t z = BF16 ? 0x80008000u : 0x80000000u;
        q[0] = q[BF16 ? 0 : 1] = make_uint4(z, z, z, z);
    }
    __device__ __forceinline__ void values(float (&v)[8]) const {
        const uint32_t w[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[BF16 ? 0 : 1].x, q[BF16 ? 0 : 1].y, q[BF16 ? 0 : 1].z, q[BF16 ? 0 : 1].w};
#pragma unroll
        for (int j = 0; j < 8; j++)
            v[j] = __uint_as_float(!BF16 ? w[j] : j & 1 ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
    }
    // the values, but not below `least` (a value that bf16 has; NaN stays)
    __device__ __forceinline__ void at_least_values(float least, float (&v)[8]) const {
        if (BF16) {
            Raw r;
            const uint32_t l = bf16x2(least, least), w[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
            uint32_t m[4];
#pragma unroll
            for (int j = 0; j < 4; j++) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m[j]) : "r"(w[j]), "r"(l));
            r.q[0] = make_uint4(m[0], m[1], m[2], m[3]);
            r.values(v);
        } else {
            values(v);
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] = at_least(v[j], least);
        }
    }
};

}  // namespace k3mx
