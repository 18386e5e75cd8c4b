// situ.cu - the SiTU-GLU between an expert block's products, with its inputs
// saved in MXFP8, and the backward passes that read activations saved so: its
// own and the RMSNorm's.
//
// Measured (repeated calls, inputs larger than L2; a copy reaches 6.78 TB/s):
//   SiTU 65536 x 2048 bf16, saved       242 us, 3.9 TB/s; not saved 177 us
//   SiTU 32768 x 2048 fp32, saved       139 us, 5.4 TB/s
//   its gradient, 65536 x 2048 bf16     173 us, 6.3 TB/s; 32768 fp32 150 us, 6.3
//   norm's gradient, 4096 x 7168 bf16   39 us, 5.3 TB/s; fp32 88 us, 4.3
//   16 x 2048: SiTU 2.3 us; 64 x 7168: norm's gradient 4.8 us (two kernels)
// bf16 SiTU is bound by the integer pipe (80 % busy: bits to places, values to
// codes), the gradients by HBM, the norm's by what its 14 warps an SM leave idle
// around a row's barrier (51 % of the issue slots used) and, in fp32, by shared
// memory's traffic.
#include "blockops.cuh"
#include "mxcode.cuh"

namespace k3mx {
namespace {

constexpr int kThreads = 256;

// CTAs of k_situ an SM holds, and the rounds of them in its grid (8.4 M runs of
// fp32, saved: 139 us, by two CTAs 148, four 151; in one round 142, two 139,
// sixteen 144; 0.5 M of bf16 13.7, 14.5, 15.3; 12.5, 12.4, 15.4)
constexpr int kSituCtas = 3, kSituWaves = 4;

// 8 e4m3 codes -> their values times `up`
__device__ __forceinline__ void from_e4m3x8(uint2 q, float up, float (&v)[8]) {
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
// the factor of a block of MXFP8
__device__ __forceinline__ float up_scale(uint32_t s) {
    return s == 255u ? __uint_as_float(0x7FC00000u) : e8m0_to_f32(s);
}

// ------------------------------------------------------------ activation --
//
// a(g) = 4 tanh(g/4) sigma(g) and b(u) = 25 tanh(u/25), h = a b.  With E =
// exp(-g/2) and F = exp(-2u/25):
//   h = 4 (1 - E) / (1 + E) / (1 + E^2) * 25 (1 - F) / (1 + F),
// two exponentials and two reciprocals, for either sign.  g and u are taken for
// no less than -110 and -288 first: E is below 2^80 and F below 2^34 then, so
// that the two numerators' product, 2^121 at most, and that of the denominators
// stay finite (E^2 is infinite below g = -88.7: its reciprocal is the limit, 0;
// b(-288) is its limit to 2^-32).  Where 1 - E cancels (|g| < 1/2, |u| < 25/8)
// tanh is its series at 0 instead, times the 1 + E that the reciprocal divides by.

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float reciprocal(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 pair(const float (&v)[8], int j) { return make_float2(v[j], v[j + 1]); }
__device__ __forceinline__ void put(float (&v)[8], int j, float2 f) { v[j] = f.x, v[j + 1] = f.y; }
__device__ __forceinline__ float2 exp2_approx(float2 x) { return make_float2(exp2_approx(x.x), exp2_approx(x.y)); }
__device__ __forceinline__ float2 reciprocal(float2 x) { return make_float2(reciprocal(x.x), reciprocal(x.y)); }

constexpr double kLog2e = 1.4426950408889634;
constexpr float kLeastG = -110.f, kLeastU = -288.f;
// x P(x^2) = tanh(x/C) up to x = C/8: y (1 - y^2/3 + 2y^4/15 - ..), what
// follows is below 3.5 units of 2^-24
template <int C> __device__ __forceinline__ float2 tanh_series(float2 x, double scale) {
    constexpr double k = 1.0 / C;
    const float2 z = __fmul2_rn(x, x);
    const float2 p = __ffma2_rn(z, both((float)(scale * k * k * k * k * k * 2 / 15)), both((float)(-scale * k * k * k / 3)));
    return __fmul2_rn(x, __ffma2_rn(z, p, both((float)(scale * k))));
}

// Two values of h (1 + bias), g and u not below kLeastG and kLeastU.  Without
// the bias each is within (64 + 1.5 |g|) units of 2^-24 of h for g >= -87,
// where 1 + E^2 has a normal reciprocal: an exponential is off by 4 units and
// by 0.75 |g| of its argument's rounding, its square by twice that, of which
// 1 + E^2 has at most all (9 + 1.5 |g| rounded); (1 - E) / (1 + E) by four times
// an exponential's error at |g| = 1/2, and two roundings, 20, and 19 for F; the
// two reciprocals by 4, products and constants by 5.
__device__ __forceinline__ float2 situ2(float2 g, float2 u, double bias) {
    const double scale = 100.0 * (1.0 + bias);
    const float2 E = exp2_approx(__fmul2_rn(g, both((float)(-0.5 * kLog2e))));
    const float2 F = exp2_approx(__fmul2_rn(u, both((float)(-0.08 * kLog2e))));
    const float2 e1 = __fadd2_rn(E, both(1.f)), f1 = __fadd2_rn(F, both(1.f));
    const float2 sg = __fmul2_rn(tanh_series<4>(g, 1.0), e1), su = __fmul2_rn(tanh_series<25>(u, scale), f1);
    const float2 lg = __ffma2_rn(E, both(-1.f), both(1.f)), lu = __ffma2_rn(F, both((float)-scale), both((float)scale));
    const float2 ng = make_float2(fabsf(g.x) < 0.5f ? sg.x : lg.x, fabsf(g.y) < 0.5f ? sg.y : lg.y);
    const float2 nu = make_float2(fabsf(u.x) < 3.125f ? su.x : lu.x, fabsf(u.y) < 3.125f ? su.y : lu.y);
    const float2 rc = reciprocal(__ffma2_rn(E, E, both(1.f))), rd = reciprocal(__fmul2_rn(e1, f1));
    return __fmul2_rn(__fmul2_rn(__fmul2_rn(ng, nu), rd), rc);
}
// The same to 2^-29 (relative, where h is above 2^-96), in sums of two floats:
// Knuth's error-free sum of two numbers, products whose error a fused product
// and sum gives exactly, and Cody and Waite's reduction of an exponential's
// argument, by the first bits of ln 2 and the rest of it.
struct Two {
    float h, l;
};
__device__ __forceinline__ Two two(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two plus_low(Two a, float l) {
    l = __fadd_rn(l, a.l);
    const float s = __fadd_rn(a.h, l);
    return {s, __fsub_rn(l, __fsub_rn(s, a.h))};
}
__device__ __forceinline__ Two times(Two a, Two b) {
    const float p = __fmul_rn(a.h, b.h), e = fmaf(a.h, b.l, fmaf(a.l, b.h, fmaf(a.h, b.h, -p))), s = __fadd_rn(p, e);
    return {s, __fsub_rn(e, __fsub_rn(s, p))};
}
__device__ __forceinline__ Two over(Two a, Two b) {
    const float r = 1.f / b.h, q = __fmul_rn(a.h, r);
    return {q, __fmul_rn(fmaf(-q, b.h, a.h) + fmaf(-q, b.l, a.l), r)};
}
// e^x, 1 - e^x and 1 + e^x of x = xh + xl: 2^n times the series of what is left
__device__ void exp_two(float xh, float xl, Two &E, Two &less, Two &more) {
    constexpr double kLn2 = 0.6931471805599453;
    constexpr double kBits = (int)(kLn2 * 32768) / 32768.0;                      // ln 2 to 15 bits: n kHigh is exact
    constexpr float kHigh = (float)kBits, kLow = (float)(kLn2 - kBits);
    constexpr float kSixth = (float)(1.0 / 6);
    const float n = rintf(__fmul_rn(xh, (float)kLog2e)), p = __fmul_rn(n, kLow);
    const Two r = plus_low(two(fmaf(n, -kHigh, xh), -p), __fsub_rn(xl, fmaf(n, kLow, -p)));
    float q = fmaf(r.h, (float)(1.0 / 362880), (float)(1.0 / 40320));
    q = fmaf(r.h, fmaf(r.h, fmaf(r.h, fmaf(r.h, q, (float)(1.0 / 5040)), (float)(1.0 / 720)), (float)(1.0 / 120)), (float)(1.0 / 24));
    const float s = __fmul_rn(r.h, r.h), sl = fmaf(r.h, r.h, -s) + 2.f * r.h * r.l;
    const float c = __fmul_rn(s, r.h), cl = fmaf(s, r.h, -c) + sl * r.h;
    const float t = __fmul_rn(c, kSixth), tl = fmaf(c, kSixth, -t) + fmaf(cl, kSixth, c * (float)(1.0 / 6 - (double)kSixth));
    const Two m1 = two(r.h, 0.5f * s), m2 = two(m1.h, t);
    const Two m = plus_low(m2, __fadd_rn(m1.l, __fadd_rn(r.l, fmaf(0.5f, sl, tl) + s * s * q)));    // e^r - 1
    E = plus_low(two(1.f, m.h), m.l);
    const float k = ldexpf(1.f, (int)n);
    E.h *= k, E.l *= k;
    more = plus_low(two(1.f, E.h), E.l);
    less = plus_low(two(1.f, -E.h), -E.l);
    if (n == 0.f) less = {-m.h, -m.l};
}
// a(g) and b(u) (for g <= 100 and |u| <= 700, where they have their limits to
// 2^-48); a is taken for 0 where E^2 leaves fp32
__device__ __forceinline__ Two situ_a(float g) {
    if (g < -87.f) return {-0.f, 0.f};
    Two E, n, d;
    exp_two(-0.5f * g, 0.f, E, n, d);
    const Two E2 = times(E, E), c = plus_low(two(1.f, E2.h), E2.l);
    return times(over(n, d), over(Two{4.f, 0.f}, c));
}
__device__ __forceinline__ Two situ_b(float u) {
    Two F, n, d;
    constexpr float k = -0.08f;
    const float xh = __fmul_rn(u, k);
    exp_two(xh, fmaf(u, k, -xh) + u * (float)(-0.08 - (double)k), F, n, d);
    return times(over(n, d), Two{25.f, 0.f});
}
// h of g and u that are not NaN, rounded to the odd one of its two fp32
// neighbours, so that rounding it on to a code rounds h itself
__device__ __noinline__ float situ_odd(float g, float u) {
    const Two h = times(situ_a(fminf(g, 100.f)), situ_b(fminf(fmaxf(u, -700.f), 700.f)));
    const uint32_t bits = __float_as_uint(h.h);
    if (h.l == 0.f || (bits & 1u)) return h.h;
    return __uint_as_float((h.l < 0.f) == (h.h < 0.f) ? bits + 1 : bits - 1);
}

// Eight values of h of a lane into codes.  They are the codes of h itself: the
// fp32 values are biased upwards by what they may be off, so that h lies between
// them and what is 2 NEAR units less; where these two have other codes (2 in
// 10 000 values), or a block's largest is as near to where its scale changes, h
// is formed again.  (Where g < -16 the value may be further off: there a code may
// be the other of two neighbours.)
constexpr uint32_t kNear = 88;        // units of 2^-24: 64 + 1.5 * 16
constexpr double bias_of(uint32_t units) { return units / 16777216.0; }
// NEAR: the units of h's bias; g, u: the values by place, for those formed again
template <uint32_t NEAR, typename G, typename U>
__device__ __forceinline__ void encode_situ(float (&h)[8], G g, U u, uint8_t *codes, uint8_t *scales, int64_t i, bool live) {
    uint32_t mb = block_max(h);
    const bool scale_near = ((mb ^ 0x600000u) & 0x7FFFFFu) <= 2 * NEAR && mb < 0x7F800000u;
    if (__any_sync(0xffffffffu, scale_near)) {
        if (scale_near) {
#pragma unroll
            for (int j = 0; j < 8; j++) h[j] = situ_odd(g(j), u(j));
        }
        mb = block_max(h);
    }
    float down;
    const uint32_t s = block_scale<K3MX_MXFP8>(mb, down);
    float less[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        put(h, j, __fmul2_rn(pair(h, j), both(down)));
        put(less, j, __fmul2_rn(pair(h, j), both((float)(1.0 - bias_of(2 * NEAR + 2)))));
    }
    uint2 w = to_e4m3x8(h);
    const uint2 l = to_e4m3x8(less);
    if (((w.x ^ l.x) | (w.y ^ l.y)) != 0 && s != 255u) {
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (((j < 4 ? w.x ^ l.x : w.y ^ l.y) >> 8 * (j & 3) & 255u) != 0) h[j] = situ_odd(g(j), u(j)) * down;
        w = to_e4m3x8(h);
    }
    const uint32_t keep = s == 255u ? 0u : 0xFFFFFFFFu;
    if (live) {
        reinterpret_cast<uint2 *>(codes)[i] = make_uint2(w.x & keep, w.y & keep);
        if ((i & 3) == 0) scales[i >> 2] = (uint8_t)s;
    }
}

// A place in a matrix of `runs` runs a row, walked with a fixed stride
struct Walk {
    int r, c, dr, dc, runs;
    __device__ __forceinline__ Walk(int64_t i, int64_t stride, int runs) : runs(runs) {
        r = (int)(i / runs), c = (int)(i - (int64_t)r * runs);
        dr = (int)(stride / runs), dc = (int)(stride - (int64_t)dr * runs);
    }
    __device__ __forceinline__ void next() {
        r += dr, c += dc;
        if (c >= runs) c -= runs, r++;
    }
};

template <bool BF16, bool SAVE>
__global__ void __launch_bounds__(kThreads, kSituCtas) k_situ(const SituArgs a, int64_t n8, int runs) {
    pdl_wait();
    pdl_launch_dependents();
    int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;             // whole blocks: runs is a multiple of 4
    const int64_t stride = (int64_t)gridDim.x * kThreads;
    Walk at(i, stride, runs);
    Raw<BF16> ng, nu;
    auto fetch = [&] {
        ng.zero(), nu.zero();
        if (i < n8) {
            ng.load(a.gu, at.r * a.ldgu + 8 * at.c);
            nu.load(a.gu, at.r * a.ldgu + 8 * (at.c + runs));
        }
    };
    fetch();
    for (; i - threadIdx.x < n8;) {
        const Raw<BF16> rg = ng, ru = nu;
        const int64_t k = i;
        const bool live = k < n8;
        const int64_t sg = (int64_t)at.r * 2 * runs + at.c;
        i += stride;
        at.next();
        fetch();
        float g[8], u[8];
        rg.at_least_values(kLeastG, g);
        ru.at_least_values(kLeastU, u);
        float h[8];
#pragma unroll
        for (int j = 0; j < 8; j += 2) put(h, j, situ2(pair(g, j), pair(u, j), bias_of(kNear)));
        encode_situ<kNear>(h, [&](int j) { return g[j]; }, [&](int j) { return u[j]; }, a.codes, a.scales, k, live);
        if (SAVE) {
            rg.values(g);
            ru.values(u);
            encode8<K3MX_MXFP8>(g, a.saved, a.saved_scales, sg, live);
            encode8<K3MX_MXFP8>(u, a.saved, a.saved_scales, sg + runs, live);
        }
    }
}

// Many runs of bf16.  bf16 has 128 values a binade, so a(g) for 2^-14 <= |g| < 2^7
// and b(u) for 2^-13 <= |u| < 2^9 are tables of fp32 values in shared memory,
// each rounded once, looked up by the value's bits; h is their product, within 4
// units of 2^-24 of itself, and hardly any value has to be formed again.  Places
// are clamped to the tables; a value that this changed (zeros, Inf and NaN among
// them) is worked out by itself.  The codes are h's for any g here.  By tables and
// without, us: 16.8 M runs, saved, 242 and 258, 8.4 M 126 and 132, 4.2 M 68 and 70, 2.1 M
// 39.7 and 38.1, 1 M 24.3 and 22.2, 0.5 M 17.5 and 13.7; not saved 177 and 194, 94 and
// 101, 53 and 55, 31.3 and 30.6, 20.1 and 18.7, 15.0 and 11.4: from 4 M runs on they
// are faster.
constexpr int kLowG = (127 - 14) * 128, kCountG = 21 * 128, kLowU = (127 - 13) * 128, kCountU = 22 * 128;
constexpr uint32_t kNearTable = 6;
constexpr int kSituTableThreads = 1024;       // (two CTAs of 512, with a table each, take 5 % more)
constexpr int64_t kSituTableRuns = 1 << 20;

__device__ __noinline__ float situ_apart(float g, float u) {
    if (g != g || u != u) return __uint_as_float(0x7FC00000u);
    const float zero = __uint_as_float((__float_as_uint(g) ^ __float_as_uint(u)) & 0x80000000u);
    return g == 0.f || u == 0.f ? zero : situ_odd(g, u);
}

template <bool SAVE>
__global__ void __launch_bounds__(kSituTableThreads, 1024 / kSituTableThreads) k_situ_table(const SituArgs a, int64_t n8, int runs) {
    __shared__ float ta[2 * kCountG], tb[kCountU];        // ta: g > 0, then g < 0
    pdl_wait();
    pdl_launch_dependents();
    int64_t i = (int64_t)blockIdx.x * kSituTableThreads + threadIdx.x;
    const int64_t stride = (int64_t)gridDim.x * kSituTableThreads;
    Walk at(i, stride, runs);
    Raw<true> ng, nu;
    auto fetch = [&] {
        ng.zero(), nu.zero();
        if (i < n8) {
            ng.load(a.gu, at.r * a.ldgu + 8 * at.c);
            nu.load(a.gu, at.r * a.ldgu + 8 * (at.c + runs));
        }
    };
    fetch();
    for (int e = threadIdx.x; e < 2 * kCountG + kCountU; e += kSituTableThreads) {
        if (e < 2 * kCountG) {
            const float v = __uint_as_float((uint32_t)(kLowG + (e < kCountG ? e : e - kCountG)) << 16);
            ta[e] = situ_a(e < kCountG ? v : -v).h;
        } else {
            const float v = __uint_as_float((uint32_t)(kLowU + e - 2 * kCountG) << 16);
            tb[e - 2 * kCountG] = situ_b(v).h * (float)(1.0 + bias_of(kNearTable));
        }
    }
    __syncthreads();
    for (; i - threadIdx.x < n8;) {
        const Raw<true> rg = ng, ru = nu;
        const int64_t k = i;
        const bool live = k < n8;
        const int64_t sg = (int64_t)at.r * 2 * runs + at.c;
        i += stride;
        at.next();
        fetch();
        const uint32_t wg[4] = {rg.q[0].x, rg.q[0].y, rg.q[0].z, rg.q[0].w}, wu[4] = {ru.q[0].x, ru.q[0].y, ru.q[0].z, ru.q[0].w};
        auto value = [](const uint32_t (&w)[4], int j) {
            return __uint_as_float(j & 1 ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
        };
        float h[8];
        uint32_t out = 0;                              // differs from 0 where a place was clamped
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint32_t mg = wg[j] & 0x7FFF7FFFu, mu = wu[j] & 0x7FFF7FFFu;
            // the place, clamped, and that of the bits as they are
            const uint32_t cg = __viaddmin_s16x2_relu(mg, (65536u - kLowG) * 0x10001u, (kCountG - 1) * 0x10001u);
            const uint32_t cu = __viaddmin_s16x2_relu(mu, (65536u - kLowU) * 0x10001u, (kCountU - 1) * 0x10001u);
            out |= (cg ^ (mg - kLowG * 0x10001u)) | (cu ^ (mu - kLowU * 0x10001u));
            // byte offsets, two to a word; the negative g's are behind the others
            const uint32_t og = cg * 4u + ((wg[j] >> 15) & 0x10001u) * (4u * kCountG), ou = cu * 4u;
            auto at = [](const float *t, uint32_t o) { return *reinterpret_cast<const float *>(reinterpret_cast<const char *>(t) + o); };
            h[2 * j] = at(ta, og & 0xFFFFu) * __uint_as_float(__float_as_uint(at(tb, ou & 0xFFFFu)) ^ (wu[j] << 16 & 0x80000000u));
            h[2 * j + 1] = at(ta, og >> 16) * __uint_as_float(__float_as_uint(at(tb, ou >> 16)) ^ (wu[j] & 0x80000000u));
        }
        if (out != 0) {
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const uint32_t mg = (j & 1 ? wg[j >> 1] >> 16 : wg[j >> 1]) & 0x7FFFu, mu = (j & 1 ? wu[j >> 1] >> 16 : wu[j >> 1]) & 0x7FFFu;
                if (mg - kLowG >= kCountG || mu - kLowU >= kCountU) h[j] = situ_apart(value(wg, j), value(wu, j));
            }
        }
        __syncwarp();
        encode_situ<kNearTable>(h, [&](int j) { return value(wg, j); }, [&](int j) { return value(wu, j); }, a.codes, a.scales, k, live);
        if (SAVE) {
            float g[8], u[8];
            rg.values(g);
            ru.values(u);
            encode8<K3MX_MXFP8>(g, a.saved, a.saved_scales, sg, live);
            encode8<K3MX_MXFP8>(u, a.saved, a.saved_scales, sg + runs, live);
        }
    }
}

// The gradient's factors, from E = exp(-|g|/2) and F = exp(-2|u|/25):
// sech^2(g/4) = 4 E / (1 + E)^2, sigma(|g|) = 1 / (1 + E^2),
// a(g)/g = sigma(g) tanh(|g|/4) / (|g|/4), and
// da/dg = sigma(g) (sech^2(g/4) + 4 tanh(g/4) sigma(-g)).  Below 2^-23 they are
// those at 0 to a rounding.
__device__ __forceinline__ float tanh_ratio(float y, float E, float r) {      // tanh(y)/y, E = exp(-2y), r = 1/(1 + E)
    const float z = y * y;
    const float p = fmaf(z, fmaf(z, fmaf(z, (float)(62.0 / 2835), (float)(-17.0 / 315)), (float)(2.0 / 15)), (float)(-1.0 / 3));
    return y < 0.25f ? fmaf(z, p, 1.f) : (1.f - E) * r * reciprocal(y);
}
__device__ __forceinline__ float2 slope_g(float g) {         // a(g)/g, da/dg
    const float m = fabsf(g) < 0x1p-23f ? 0.f : fabsf(g), E = exp2_approx(m * (float)(-0.5 * kLog2e));
    const float r = reciprocal(1.f + E), q = reciprocal(fmaf(E, E, 1.f)), ratio = tanh_ratio(0.25f * m, E, r);
    const float s = g < 0.f ? E * E * q : q, n = g < 0.f ? q : E * E * q;
    return make_float2(s * ratio, s * fmaf(copysignf(m, g) * ratio, n, 4.f * E * r * r));
}
__device__ __forceinline__ float2 slope_u(float u) {         // b(u)/u, db/du
    const float m = fabsf(u) < 0x1p-23f ? 0.f : fabsf(u), F = exp2_approx(m * (float)(-0.08 * kLog2e));
    const float r = reciprocal(1.f + F);
    return make_float2(tanh_ratio(0.04f * m, F, r), 4.f * F * r * r);
}
__device__ __forceinline__ float2 situ_grad(float g, float u, float d) {      // dg, du
    const bool nan = g != g || u != u;
    g = fminf(fmaxf(g, -0x1p100f), 0x1p100f), u = fminf(fmaxf(u, -0x1p100f), 0x1p100f);      // (limits, not 0 * Inf)
    const float2 p = slope_g(g), q = slope_u(u);
    return nan ? both(__uint_as_float(0x7FC00000u)) : make_float2((d * p.y) * (u * q.x), (d * q.y) * (g * p.x));
}
__device__ __noinline__ float2 situ_grad_apart(float g, float u, float d) { return situ_grad(g, u, d); }

// What a thread reads of one run of eight: the codes, their blocks' bytes, dh
template <bool BF16> struct GradRun {
    uint2 g, u;
    uint32_t sg, su;
    Raw<BF16> d;
    __device__ __forceinline__ void load(const SituGradArgs &a, const Walk &at, bool live) {
        g = u = make_uint2(0u, 0u), sg = su = 0u;
        d.zero();
        if (live) {
            const int64_t i = (int64_t)at.r * 2 * at.runs + at.c;
            g = reinterpret_cast<const uint2 *>(a.saved)[i];
            u = reinterpret_cast<const uint2 *>(a.saved)[i + at.runs];
            sg = a.saved_scales[i >> 2];
            su = a.saved_scales[(i + at.runs) >> 2];
            d.load(a.dh, at.r * a.lddh + 8 * at.c);
        }
    }
};

// Few runs: each value's factors are worked out where they are needed.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_situ_grad(const SituGradArgs a, int64_t n8, int runs) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const bool live = i < n8;
    const Walk at(live ? i : 0, 0, runs);
    GradRun<BF16> x;
    x.load(a, at, live);
    float g[8], u[8], d[8];
    from_e4m3x8(x.g, up_scale(x.sg), g);
    from_e4m3x8(x.u, up_scale(x.su), u);
    x.d.values(d);
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const float2 r = situ_grad(g[j], u[j], d[j]);
        g[j] = r.x, u[j] = r.y;
    }
    const int64_t to = ((int64_t)at.r * 2 * runs + at.c) * 8;
    store8<BF16>(a.dgu, to, g, live);
    store8<BF16>(a.dgu, to + 8 * runs, u, live);
}

// Many runs.  A saved value has three mantissa bits, so within 2^-24 .. 2^8
// there are 256 of each sign, and their factors are a table in shared memory:
// the value times 2^-7 has its place in eight bits of its fp32 pattern (bits
// 20..27: 2^-31 at 0; a zero has 0 there too, whose factors are the same).
// Sixteen copies, one for each lane of a half warp, so that no two lanes of a
// read meet in a bank.  A block whose scale allows values outside that range is
// worked out as above.  The places of 1.875 * 2^7 are free (no code under such
// a scale has that value) and are where a NaN code looks: they hold NaN.
// Measured, with the table and without: 1 M runs of bf16 18.3 and 23.5 us,
// 0.5 M 12.8 and 12.9, 0.25 M 10.4 and 8.1; of fp32 24.7 and 25.6, 16.3 and 14.1.
constexpr int64_t kTableRuns = 1 << 19, kRoundsRuns = 1 << 23;
constexpr int kTableThreads = 512, kTableRow = 128, kTableBytes = 3 * 256 * kTableRow;     // g >= 0, g < 0, |u|
constexpr uint32_t kTableLow = 112, kTableHigh = 126;        // scale bytes that it serves

template <bool BF16>
__global__ void __launch_bounds__(kTableThreads, 2) k_situ_grad_table(const SituGradArgs a, int64_t n8, int runs) {
    extern __shared__ __align__(16) uint8_t table[];
    pdl_wait();
    pdl_launch_dependents();
    int64_t i = (int64_t)blockIdx.x * kTableThreads + threadIdx.x;
    const int64_t stride = (int64_t)gridDim.x * kTableThreads;
    Walk at(i, stride, runs);
    GradRun<BF16> next;
    next.load(a, at, i < n8);
    for (int e = threadIdx.x; e < 3 * 256; e += kTableThreads) {
        // entry e & 255: the value of 2^7 times the pattern with these bits
        float v = __uint_as_float((uint32_t)((e & 255) + 768) << 20) * 128.f;
        float2 f = e >= 512 ? slope_u(v) : slope_g(e >= 256 ? -v : v);
        f.x *= 128.f;
        if ((e & 255) == 255) f.x = f.y = __uint_as_float(0x7FC00000u);
        float4 *to = reinterpret_cast<float4 *>(table + e * kTableRow);
#pragma unroll
        for (int k = 0; k < kTableRow / 16; k++) to[k] = make_float4(f.x, f.y, f.x, f.y);
    }
    __syncthreads();
    const uint32_t lane = (threadIdx.x & 15) * 8;
    for (; i - threadIdx.x < n8;) {
        const GradRun<BF16> x = next;
        const bool live = i < n8;
        const int64_t to = ((int64_t)at.r * 2 * runs + at.c) * 8;
        i += stride;
        at.next();
        next.load(a, at, i < n8);
        float g[8], u[8], d[8];
        x.d.values(d);
        const bool in_table = x.sg - kTableLow <= kTableHigh - kTableLow && x.su - kTableLow <= kTableHigh - kTableLow;
        if (in_table) {
            from_e4m3x8(x.g, __uint_as_float((x.sg - 7u) << 23), g);
            from_e4m3x8(x.u, __uint_as_float((x.su - 7u) << 23), u);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const uint32_t bg = __float_as_uint(g[j]), bu = __float_as_uint(u[j]);
                const float2 p = *reinterpret_cast<const float2 *>(table + ((bg >> 13 & 0x7F80u) | lane | (bg >> 16 & 0x8000u)));
                const float2 q = *reinterpret_cast<const float2 *>(table + 512 * kTableRow + ((bu >> 13 & 0x7F80u) | lane));
                const float dg = (d[j] * p.y) * (u[j] * q.x), du = (d[j] * q.y) * (g[j] * p.x);
                g[j] = dg, u[j] = du;
            }
        } else {
            from_e4m3x8(x.g, up_scale(x.sg), g);
            from_e4m3x8(x.u, up_scale(x.su), u);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float2 r = situ_grad_apart(g[j], u[j], d[j]);
                g[j] = r.x, u[j] = r.y;
            }
        }
        __syncwarp();
        store8<BF16>(a.dgu, to, g, live);
        store8<BF16>(a.dgu, to + 8 * runs, u, live);
    }
}

// ------------------------------------------------------ the norm's gradient --
//
// With k = 1 / sqrt(mean(s^2) + eps), n = s k and a = g dn: dx = k (a - n q),
// q = mean(a n) = k mean(a s), so one pass over a row gives both sums.  A CTA
// (or a warp, for narrow rows) keeps its columns of the weight and of its rows'
// sum of dn n in registers and walks the rows part by part; the parts are
// added by a second kernel in their order.
//
// A thread has the same runs of every row, so what it needs of the next rows it
// copies ahead into shared memory for itself (cp.async, D rows deep, no
// barrier).  D = 0: they come from global memory, for a CTA's only row (64 rows
// of 7168 fp32: 4.8 us, by way of shared memory 6.5) and for rows that shared
// memory does not hold: those are read before the sums and from L2 once more
// after them (KEEP false), and the sums of dn n have the shared memory.

constexpr int kNormSms = 152;         // parts are a multiple of it (a constant: results do not depend on the device)
constexpr int kRowsOfPart = 1024;     // rows that one thread adds, at most
constexpr int kNormSmem = 220 << 10;
// rows copied ahead (4096 x 7168: of bf16 39.2 us, three 39.9, four 40.5, one
// 57.7; of fp32 85.2, three 85.7, one 113; 8192 x 512 bf16 10.4, three 10.6, one
// 12.7)
constexpr int kNormRing = 2;

struct NormShape {
    bool warp;         // a row to a warp, eight a CTA
    bool few;          // one row a CTA
    int v, threads, parts;
};
// A warp a row up to 128 runs (8192 x 1024 bf16 15.5 us, fp32 30.4; by a CTA a row
// 18.0 and 33.5); two runs a thread of a CTA (4096 x 7168 bf16: 41 us with four
// rows ahead, one 59), four where 1024 threads do not reach otherwise.
NormShape norm_shape(int n_tokens, int width) {
    const int runs = width / 8;
    NormShape s;
    s.warp = runs <= 128;
    s.few = !s.warp && runs <= 1024 && n_tokens <= kNormSms;
    s.v = s.warp ? (runs <= 32 ? 1 : runs <= 64 ? 2 : 4) : s.few ? 1 : runs <= 2048 ? 2 : 4;
    s.threads = s.warp ? kThreads : (runs + 32 * s.v - 1) / (32 * s.v) * 32;
    const int at_once = s.warp ? kThreads / 32 : 1, full = (n_tokens + at_once - 1) / at_once;
    const int least = (full + kRowsOfPart - 1) / kRowsOfPart;
    const int most = kNormSms * (s.warp ? 1 : s.threads <= 128 ? 4 : s.threads <= 256 ? 2 : 1);
    // (two rows, or rounds of eight, in one part: 16 x 128 2.6 us a call, 4.0 with a
    // second kernel; 2 x 2048 3.0 and 4.0; three rows of 7168 5.8 and 4.5)
    s.parts = full <= 2 ? 1 : full < most ? full : least > most ? least : most;
    return s;
}
// bytes that a thread keeps of a run: dn, dres, codes
constexpr int run_bytes(bool bf16) { return 8 + 2 * (bf16 ? 16 : 32); }
static_assert(kNormRing * 512 * 2 * run_bytes(false) <= kNormSmem, "the rows of 1024 runs have to fit");

__device__ __forceinline__ void copy16(uint32_t to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t to, const void *from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_end_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// The sums of a and b over a warp, to all its lanes: one half of it adds a, the
// other b.
__device__ __forceinline__ float half_sums(float a, float b) {
    const bool high = threadIdx.x & 16;
    float v = (high ? b : a) + __shfl_xor_sync(0xffffffffu, high ? a : b, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <bool WARP, int V, bool BF16, int D, bool KEEP>
__global__ void __launch_bounds__(WARP ? kThreads : D > 0 ? 512 : 1024, 1)
k_norm_grad(const NormGradArgs a) {
    extern __shared__ __align__(16) uint8_t ring[];       // D > 0: [D][V] of dn, dres, codes of the CTA's threads; !KEEP: the sums
    __shared__ float sums[2][2][32];
    constexpr int kQ = BF16 ? 1 : 2, kElem = BF16 ? 2 : 4;        // kQ: 16 bytes of a run's dn
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, P = WARP ? 32 : blockDim.x;
    const int i0 = WARP ? lane : threadIdx.x, runs = a.width / 8;
    const int step = gridDim.x * (WARP ? kThreads / 32 : 1);
    int t = WARP ? blockIdx.x * (kThreads / 32) + warp : blockIdx.x;
    const int P16 = blockDim.x * 16, slot = (int)blockDim.x * run_bytes(BF16), me = threadIdx.x * 16;
    // run p of a row: whether it is there; the rest of the row is at 8 P columns' distance
    auto there = [&](int p) { return p * P + i0 < runs; };
    const bool res = a.dres != nullptr;

    // the row to be copied ahead
    int ahead = t;
    const int64_t first = (int64_t)t * a.width + 8 * i0, pitch = (int64_t)step * a.width, dn_pitch = (int64_t)step * a.lddn * kElem;
    const uint8_t *from_dn = static_cast<const uint8_t *>(a.dn) + (t * a.lddn + 8 * i0) * kElem;
    const uint8_t *from_res = static_cast<const uint8_t *>(a.dres) + first * kElem;
    const uint8_t *from_codes = a.saved + first;
    auto fetch = [&](uint32_t to) {
        if (ahead < a.n_tokens) {
#pragma unroll
            for (int p = 0; p < V; p++)
                if (there(p)) {
                    const uint32_t at = to + p * slot;
#pragma unroll
                    for (int q = 0; q < kQ; q++) copy16(at + me + q * P16, from_dn + 8 * p * P * kElem + 16 * q);
                    if (res) {
#pragma unroll
                        for (int q = 0; q < kQ; q++) copy16(at + me + (kQ + q) * P16, from_res + 8 * p * P * kElem + 16 * q);
                    }
                    copy8(at + me / 2 + 2 * kQ * P16, from_codes + 8 * p * P);
                }
            ahead += step;
            from_dn += dn_pitch, from_res += pitch * kElem, from_codes += pitch;
        }
        copies_end_group();
    };
    const uint32_t base = D > 0 ? smem_addr(ring) : 0u;
    if (D > 0) {
#pragma unroll
        for (int d = 0; d < D; d++) fetch(base + d * V * slot);
    }
    const uint8_t *from_scales = a.saved_scales + (first >> 5);
    auto scales = [&](int t, uint32_t (&s)[V]) {
#pragma unroll
        for (int p = 0; p < V; p++) s[p] = there(p) && t < a.n_tokens ? from_scales[p * P / 4] : 0u;
        from_scales += pitch >> 5;
    };
    uint32_t scale[V];
    scales(t, scale);
    uint8_t *to_dx = static_cast<uint8_t *>(a.dx) + first * kElem;
    float weight[KEEP ? V : 1][8], acc[KEEP ? V : 1][8];
    auto load_weight = [&](int p, float (&g)[8]) {
        Raw<true> r;
        r.zero();
        if (there(p)) r.load(a.g, 8 * (p * P + i0));
        r.values(g);
    };
    auto parked = [&](int p, int h) { return reinterpret_cast<float4 *>(ring) + (2 * p + h) * blockDim.x + threadIdx.x; };
#pragma unroll
    for (int p = 0; p < V; p++) {
        if (KEEP) {
            load_weight(p, weight[KEEP ? p : 0]);
#pragma unroll
            for (int j = 0; j < 8; j++) acc[KEEP ? p : 0][j] = 0.f;
        } else {
            *parked(p, 0) = *parked(p, 1) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    const float inverse = 1.f / (float)a.width;
    int flip = 0, d = 0;
    for (; t < a.n_tokens; t += step) {
        uint32_t next[V];
        scales(t + step, next);
        if (D > 0) copies_wait<D - 1>();
        const uint8_t *at = ring + d * V * slot;
        auto values = [&](int p, float (&x)[8]) {
            uint2 q = make_uint2(0u, 0u);
            if (there(p))
                q = D > 0 ? *reinterpret_cast<const uint2 *>(at + p * slot + 2 * kQ * P16 + me / 2)
                          : reinterpret_cast<const uint2 *>(a.saved)[(int64_t)t * runs + p * P + i0];
            from_e4m3x8(q, up_scale(scale[p]), x);
        };
        auto grads = [&](int p, int part, float (&v)[8]) {            // part 0: dn, 1: dres
            Raw<BF16> r;
            r.zero();
            if (there(p)) {
                if (D > 0) {
#pragma unroll
                    for (int q = 0; q < kQ; q++) r.q[q] = *reinterpret_cast<const uint4 *>(at + p * slot + (part * kQ + q) * P16 + me);
                } else if (part == 0) {
                    r.load(a.dn, t * a.lddn + 8 * (p * P + i0));
                } else {
                    r.load(a.dres, (int64_t)t * a.width + 8 * (p * P + i0));
                }
            }
            r.values(v);
        };
        float x[KEEP ? V : 1][8], dn[KEEP ? V : 1][8];
        if (KEEP) {
#pragma unroll
            for (int p = 0; p < V; p++) values(p, x[KEEP ? p : 0]), grads(p, 0, dn[KEEP ? p : 0]);
        }
        // g bd; beside an s of 0, where the product is 0, not an infinite one
        auto up = [](float g, float bd, float s) { return bd > 1.f && s == 0.f ? 0.f : g * bd; };
        auto scaled_again = [&](float by, float bd) {                 // s by, dn bd
            if (KEEP) {
#pragma unroll
                for (int p = 0; p < V; p++) {
                    values(p, x[KEEP ? p : 0]), grads(p, 0, dn[KEEP ? p : 0]);
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        float &s = x[KEEP ? p : 0][j], &g = dn[KEEP ? p : 0][j];
                        s *= by, g = up(g, bd, s);
                    }
                }
            }
        };
        // a run's s, dn and weight: kept in registers, or fetched again
        auto run = [&](int p, float (&rx)[8], float (&rd)[8], float (&rw)[8]) {
            if (KEEP) {
#pragma unroll
                for (int j = 0; j < 8; j++) rx[j] = x[KEEP ? p : 0][j], rd[j] = dn[KEEP ? p : 0][j], rw[j] = weight[KEEP ? p : 0][j];
            } else {
                values(p, rx), grads(p, 0, rd), load_weight(p, rw);
            }
        };
        constexpr bool kEarly = KEEP && D == 0;              // dres with the rest, not after the sums
        float early[8] = {};
        if (kEarly && res) grads(0, 1, early);
        float ss, sx;
        auto sum = [&](float by, float bd) {                 // the sums of s^2 and a s (KEEP: of what the registers hold)
            float2 s2 = both(0.f), x2 = both(0.f);
#pragma unroll
            for (int p = 0; p < V; p++) {
                float rx[8], rd[8], rw[8];
                run(p, rx, rd, rw);
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const float2 v = KEEP ? pair(rx, j) : __fmul2_rn(pair(rx, j), both(by));
                    const float2 g = KEEP ? pair(rd, j) : make_float2(up(rd[j], bd, v.x), up(rd[j + 1], bd, v.y));
                    s2 = __ffma2_rn(v, v, s2);
                    x2 = __ffma2_rn(__fmul2_rn(pair(rw, j), g), v, x2);
                }
            }
            float v = half_sums(s2.x + s2.y, x2.x + x2.y);
            if (!WARP) {
                if ((lane & 15) == 0) sums[flip][lane >> 4][warp] = v;
                __syncthreads();
                const int nw = blockDim.x >> 5, l = lane & 15;
                const float *row = sums[flip][lane >> 4];
                v = (l < nw ? row[l] : 0.f) + (l + 16 < nw ? row[l + 16] : 0.f);
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                flip ^= 1;
            }
            ss = __shfl_sync(0xffffffffu, v, 0), sx = __shfl_sync(0xffffffffu, v, 16);
        };
        sum(1.f, 1.f);
        float m = fmaf(ss, inverse, a.eps), by = 1.f, undo = 1.f;
        // (the same for every thread of the row)
        if (!(m >= 0x1p-100f && m < INFINITY && fabsf(sx) < INFINITY && (fabsf(sx) >= 0x1p-90f || m >= 0x1p-24f))) {
            // A sum leaves fp32, or its normal numbers: both again, of s and dn by a power of two each.  Squares above
            // it: s by 2^-72, whose squares add up to 2^127 at most.  A mean below 2^-100, of which subnormal squares
            // (each off by 2^-150) may be much: s by 2^64.  Products above it: dn by 2^-72 (they add up to sqrt(width)
            // |a| times the root of the squares' sum, below 2^128 then).  Products that may be subnormal, where k^2 |n|
            // times 2^-150 may be much, or that add up to 0: dn by 2^100, or as it is where that is too large.
            by = !(m < INFINITY) ? 0x1p-72f : m < 0x1p-100f ? 0x1p64f : 1.f;
            float bd = !(fabsf(sx) < INFINITY) ? 0x1p-72f : fabsf(sx) < 0x1p-90f && m < 0x1p-24f ? 0x1p100f : 1.f;
            undo = bd < 1.f ? 0x1p72f : bd > 1.f ? 0x1p-100f : 1.f;
            for (;;) {
                scaled_again(by, bd);
                sum(by, bd);
                if (bd <= 1.f || fabsf(sx) < INFINITY) break;
                bd = undo = 1.f;
            }
            m = fmaf(ss, inverse, a.eps * by * by);
            scaled_again(1.f, 1.f);
        }
        // k by: the factor of the values themselves, kq: dx = k a - n kq
        const float k0 = rsqrtf(m), k = m == 0.f ? k0 : k0 * fmaf(-0.5f, fmaf(m * k0, k0, -1.f), 1.f);
        const float kx = k * by, kq = kx * (k * (sx * inverse) * undo);
#pragma unroll
        for (int p = 0; p < V; p++) {
            float rx[8], rd[8], rw[8], r[8] = {};
            run(p, rx, rd, rw);
            if (kEarly) {
#pragma unroll
                for (int j = 0; j < 8; j++) r[j] = early[j];
            } else if (res) {
                grads(p, 1, r);
            }
            if (!KEEP) {
                const float4 f = *parked(p, 0), g = *parked(p, 1);
                acc[0][0] = f.x, acc[0][1] = f.y, acc[0][2] = f.z, acc[0][3] = f.w;
                acc[0][4] = g.x, acc[0][5] = g.y, acc[0][6] = g.z, acc[0][7] = g.w;
            }
            float (&sum)[8] = acc[KEEP ? p : 0];
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float2 n = __fmul2_rn(pair(rx, j), both(kx));
                put(sum, j, __ffma2_rn(pair(rd, j), n, pair(sum, j)));
                put(r, j, __ffma2_rn(n, both(-kq), __ffma2_rn(__fmul2_rn(pair(rw, j), pair(rd, j)), both(kx), pair(r, j))));
            }
            if (!KEEP) {
                *parked(p, 0) = make_float4(sum[0], sum[1], sum[2], sum[3]);
                *parked(p, 1) = make_float4(sum[4], sum[5], sum[6], sum[7]);
            }
            store8<BF16>(to_dx, 8 * p * P, r, there(p));
        }
        to_dx += pitch * kElem;
        if (D > 0) {
            // (what was read of the slot has gone into the stores above)
            fetch(base + d * V * slot);
            d = d + 1 == D ? 0 : d + 1;
        }
#pragma unroll
        for (int p = 0; p < V; p++) scale[p] = next[p];
    }
    float *to = gridDim.x == 1 ? a.dweight : a.part + (int64_t)blockIdx.x * a.width;
    if (D > 0) copies_wait<0>();
    if (WARP) {
        // the eight warps' columns, added in their order
        float *cols = reinterpret_cast<float *>(ring);
        __syncthreads();
#pragma unroll
        for (int p = 0; p < V; p++)
#pragma unroll
            for (int j = 0; j < 8; j++) cols[warp * 256 * V + 8 * (p * 32 + lane) + j] = acc[KEEP ? p : 0][j];
        __syncthreads();
        for (int c = threadIdx.x; c < a.width; c += kThreads) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kThreads / 32; w++) s += cols[w * 256 * V + c];
            to[c] = s;
        }
    } else {
#pragma unroll
        for (int p = 0; p < V; p++) {
            if (!KEEP) {
                const float4 f = *parked(p, 0), g = *parked(p, 1);
                acc[0][0] = f.x, acc[0][1] = f.y, acc[0][2] = f.z, acc[0][3] = f.w;
                acc[0][4] = g.x, acc[0][5] = g.y, acc[0][6] = g.z, acc[0][7] = g.w;
            }
            store8<false>(to, 8 * (p * P + i0), acc[KEEP ? p : 0], there(p));
        }
    }
}

// dweight[c] = sum over the parts: 32 columns a CTA, a share of the parts a warp
__global__ void __launch_bounds__(1024) k_norm_grad_sum(float *dweight, const float *part, int parts, int width) {
    __shared__ float sums[32][32];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, c = blockIdx.x * 32 + lane;
    float s = 0.f;
    for (int p0 = warp; p0 < parts; p0 += 8 * warps) {
        float v[8];                   // loads at once, the last ones of the last part again
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = part[(int64_t)min(p0 + j * warps, parts - 1) * width + c];      // width: whole blocks of 32
#pragma unroll
        for (int j = 0; j < 8; j++) s += p0 + j * warps < parts ? v[j] : 0.f;
    }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0) {
        s = 0.f;
#pragma unroll 8
        for (int w = 0; w < warps; w++) s += sums[w][lane];
        dweight[c] = s;
    }
}

}  // namespace

cudaError_t launch_situ(const Ctx &c, const SituArgs &a, int bf16) {
    const int runs = a.inter / 8;
    const int64_t n8 = (int64_t)a.rows * runs, ctas = (n8 + kThreads - 1) / kThreads, most = (int64_t)c.num_sms * kSituCtas * kSituWaves;
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, dim3((unsigned)(ctas < most ? ctas : most)), dim3(kThreads), 0, c.stream, a, n8, runs);
    };
    if (bf16 && n8 >= kSituTableRuns) {
        const int64_t per = kSituTableThreads, all = (n8 + per - 1) / per, fit = (int64_t)c.num_sms * (1024 / per);
        auto table = [&](auto kernel) {
            return launch_pdl(kernel, dim3((unsigned)(all < fit ? all : fit)), dim3(kSituTableThreads), 0, c.stream, a, n8, runs);
        };
        return a.saved != nullptr ? table(k_situ_table<true>) : table(k_situ_table<false>);
    }
    if (a.saved != nullptr) return bf16 ? go(k_situ<true, true>) : go(k_situ<false, true>);
    return bf16 ? go(k_situ<true, false>) : go(k_situ<false, false>);
}

cudaError_t launch_situ_grad(const Ctx &c, const SituGradArgs &a, int bf16) {
    const int runs = a.inter / 8;
    const int64_t n8 = (int64_t)a.rows * runs;
    if (n8 < kTableRuns) {
        auto go = [&](auto kernel) {
            return launch_pdl(kernel, dim3((unsigned)((n8 + kThreads - 1) / kThreads)), dim3(kThreads), 0, c.stream, a, n8, runs);
        };
        return bf16 ? go(k_situ_grad<true>) : go(k_situ_grad<false>);
    }
    // two CTAs an SM; fp32 gradients of very many runs in four rounds of them
    // (8.4 M runs 165 to 150 us, 4.2 M 85 either way, 1 M 25 to 43; bf16: 16.8 M runs 173 to 186)
    const int64_t ctas = (n8 + kTableThreads - 1) / kTableThreads;
    const int64_t most = (int64_t)c.num_sms * (!bf16 && n8 >= kRoundsRuns ? 8 : 2);
    auto go = [&](auto kernel, std::atomic<uint64_t> &done) {
        const cudaError_t e = ensure_smem((const void *)kernel, kTableBytes, done);
        if (e != cudaSuccess) return e;
        return launch_pdl(kernel, dim3((unsigned)(ctas < most ? ctas : most)), dim3(kTableThreads), kTableBytes, c.stream, a, n8, runs);
    };
    static std::atomic<uint64_t> done_f32{0}, done_bf16{0};
    return bf16 ? go(k_situ_grad_table<true>, done_bf16) : go(k_situ_grad_table<false>, done_f32);
}

size_t norm_grad_scratch_bytes(int n_tokens, int width) {
    return (size_t)norm_shape(n_tokens, width).parts * width * sizeof(float);
}

template <bool WARP, int V, int D, bool KEEP>
static cudaError_t norm_grad_t(const Ctx &c, const NormGradArgs &a, const NormShape &s, int bf16) {
    auto go = [&](auto kernel, std::atomic<uint64_t> &done) {
        const int slots = D * V * run_bytes(bf16) * s.threads, sum = WARP || !KEEP ? s.threads * 8 * V * (int)sizeof(float) : 0;
        const cudaError_t e = ensure_smem((const void *)kernel, kNormSmem, done);
        if (e != cudaSuccess) return e;
        return launch_pdl(kernel, dim3(s.parts), dim3(s.threads), slots > sum ? slots : sum, c.stream, a);
    };
    static std::atomic<uint64_t> done_f32{0}, done_bf16{0};
    return bf16 ? go(k_norm_grad<WARP, V, true, D, KEEP>, done_bf16) : go(k_norm_grad<WARP, V, false, D, KEEP>, done_f32);
}

cudaError_t launch_norm_grad(const Ctx &c, const NormGradArgs &a, int bf16) {
    const NormShape s = norm_shape(a.n_tokens, a.width);
    auto go = [&] {
        if (s.warp)
            return s.v == 1   ? norm_grad_t<true, 1, kNormRing, true>(c, a, s, bf16)
                   : s.v == 2 ? norm_grad_t<true, 2, kNormRing, true>(c, a, s, bf16)
                              : norm_grad_t<true, 4, kNormRing, true>(c, a, s, bf16);
        if (s.few) return norm_grad_t<false, 1, 0, true>(c, a, s, bf16);
        if (s.threads <= 512) return norm_grad_t<false, 2, kNormRing, true>(c, a, s, bf16);
        return s.v == 2 ? norm_grad_t<false, 2, 0, false>(c, a, s, bf16) : norm_grad_t<false, 4, 0, false>(c, a, s, bf16);
    };
    const cudaError_t e = go();
    if (e != cudaSuccess || s.parts == 1) return e;
    return launch_pdl(k_norm_grad_sum, dim3(a.width / 32), dim3(s.parts <= 64 ? 256 : 1024), 0, c.stream, a.dweight, (const float *)a.part,
                      s.parts, a.width);
}

}  // namespace k3mx
