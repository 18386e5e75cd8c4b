// situ.cu - the SiTU-GLU between an expert block's products, with its inputs
// saved in MXFP8, and the backward passes that read activations saved so: its
// own and the RMSNorm's.
#include "blockops.cuh"
#include "mxcode.cuh"

namespace k3mx {
namespace {

constexpr int kThreads = 256;

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
// a(g) = 4 tanh(g/4) sigma(g) and b(u) = 25 tanh(u/25), h = a b.  With
// E = exp(-|g|/2): tanh(|g|/4) = (1 - E) / (1 + E), sigma(|g|) = 1 / (1 + E^2)
// and sigma(-|g|) = E^2 / (1 + E^2), so one exponential serves both factors,
// and no intermediate overflows.  Where 1 - E would cancel (|g| < 1) tanh is
// its series at 0.

// tanh(|x|/c) from E = exp(-2|x|/c) and r = 1/(1 + E); y = |x|/c
__device__ __forceinline__ float tanh_of(float y, float E, float r) {
    const float z = y * y;
    const float series = y * fmaf(z, fmaf(z, fmaf(z, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.f);
    return y < 0.25f ? series : (1.f - E) * r;
}

__device__ __forceinline__ float situ(float g, float u) {
    const float ag = fabsf(g), au = fabsf(u);
    const float E = __expf(-0.5f * ag), F = __expf(-0.08f * au), E2 = E * E;
    const float re = __fdividef(1.f, 1.f + E), rs = __fdividef(1.f, 1.f + E2), rf = __fdividef(1.f, 1.f + F);
    const float t = tanh_of(0.25f * ag, E, re), v = tanh_of(0.04f * au, F, rf);
    const float h = 100.f * (t * v) * ((g < 0.f ? E2 : 1.f) * rs);
    const uint32_t sign = (__float_as_uint(g) ^ __float_as_uint(u)) & 0x80000000u;
    return __uint_as_float(__float_as_uint(h) ^ sign);
}

template <bool BF16, bool SAVE>
__global__ void __launch_bounds__(kThreads) k_situ(const SituArgs a, int64_t n8, int runs) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;       // whole blocks: runs is a multiple of 4
    const bool live = i < n8;
    const int64_t r = live ? i / runs : 0;
    const int c = (int)(i - r * runs);
    float g[8] = {}, u[8] = {}, h[8];
    if (live) {
        load8<BF16, true>(a.gu, r * a.ldgu + 8 * c, g);
        load8<BF16, true>(a.gu, r * a.ldgu + 8 * (c + runs), u);
    }
#pragma unroll
    for (int j = 0; j < 8; j++) h[j] = situ(g[j], u[j]);
    encode8<K3MX_MXFP8>(h, a.codes, a.scales, i, live);
    if (SAVE) {
        encode8<K3MX_MXFP8>(g, a.saved, a.saved_scales, r * 2 * runs + c, live);
        encode8<K3MX_MXFP8>(u, a.saved, a.saved_scales, r * 2 * runs + runs + c, live);
    }
}

// da/dg = s (sech^2(g/4) + 4 tanh(g/4) (1 - s)), s = sigma(g), sech^2(g/4) =
// 4 E / (1 + E)^2; db/du = sech^2(u/25)
__device__ __forceinline__ void situ_grad(float g, float u, float dh, float &dg, float &du) {
    const float ag = fabsf(g), au = fabsf(u);
    const float E = __expf(-0.5f * ag), F = __expf(-0.08f * au), E2 = E * E;
    const float re = __fdividef(1.f, 1.f + E), rs = __fdividef(1.f, 1.f + E2), rf = __fdividef(1.f, 1.f + F);
    const float t = copysignf(tanh_of(0.25f * ag, E, re), g), v = copysignf(tanh_of(0.04f * au, F, rf), u);
    const float s = (g < 0.f ? E2 : 1.f) * rs, n = (g < 0.f ? 1.f : E2) * rs;
    const float slope = 4.f * s * fmaf(t, n, E * re * re);
    dg = dh * (25.f * v) * slope;
    du = dh * (4.f * t * s) * (4.f * F * rf * rf);
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_situ_grad(const SituGradArgs a, int64_t n8, int runs) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const bool live = i < n8;
    const int64_t r = live ? i / runs : 0;
    const int c = (int)(i - r * runs);
    const int64_t ig = r * 2 * runs + c, iu = ig + runs;
    uint2 qg = make_uint2(0u, 0u), qu = qg;
    float g[8], u[8], d[8] = {}, sg = 0.f, su = 0.f;
    if (live) {
        qg = reinterpret_cast<const uint2 *>(a.saved)[ig];
        qu = reinterpret_cast<const uint2 *>(a.saved)[iu];
        sg = up_scale(a.saved_scales[ig >> 2]);
        su = up_scale(a.saved_scales[iu >> 2]);
        load8<BF16, true>(a.dh, r * a.lddh + 8 * c, d);
    }
    from_e4m3x8(qg, sg, g);
    from_e4m3x8(qu, su, u);
#pragma unroll
    for (int j = 0; j < 8; j++) situ_grad(g[j], u[j], d[j], g[j], u[j]);
    store8<BF16>(a.dgu, 8 * ig, g, live);
    store8<BF16>(a.dgu, 8 * iu, u, live);
}

// ------------------------------------------------------ the norm's gradient --
//
// With k = 1 / sqrt(mean(s^2) + eps), n = s k and a = g dn: dx = k (a - n q),
// q = mean(a n) = k mean(a s), so one pass over a row gives both sums.  A CTA
// (or a warp, for narrow rows) keeps its columns of the weight and of its rows'
// sum of dn n in registers and walks the rows part by part; the parts are
// added by a second kernel in their order.

constexpr int kNormParts = 608;       // parts at most, but for the next line
constexpr int kRowsOfPart = 1024;     // rows that one thread adds, at most

struct NormShape {
    bool warp;         // a row to a warp, eight a CTA
    int v, threads, parts;
};
NormShape norm_shape(int n_tokens, int width) {
    const int runs = width / 8;
    NormShape s;
    s.warp = runs <= 128;
    s.v = s.warp ? (runs <= 32 ? 1 : 4) : runs <= 1024 ? 1 : runs <= 2048 ? 2 : 4;
    s.threads = s.warp ? kThreads : (runs + 32 * s.v - 1) / (32 * s.v) * 32;
    const int at_once = s.warp ? kThreads / 32 : 1, full = (n_tokens + at_once - 1) / at_once;
    const int least = (full + kRowsOfPart - 1) / kRowsOfPart;
    s.parts = full < kNormParts ? full : least > kNormParts ? least : kNormParts;
    return s;
}

template <bool WARP, int V, bool BF16>
__global__ void __launch_bounds__(WARP ? kThreads : 1024) k_norm_grad(const NormGradArgs a) {
    __shared__ float2 sums[2][32];
    __shared__ float cols[WARP ? kThreads / 32 * 256 * V : 1];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, P = WARP ? 32 : blockDim.x;
    const int i0 = WARP ? lane : threadIdx.x, runs = a.width / 8;
    const int step = gridDim.x * (WARP ? kThreads / 32 : 1);
    uint4 gq[V];
    float acc[V][8] = {};
#pragma unroll
    for (int p = 0; p < V; p++)
        gq[p] = p * P + i0 < runs ? reinterpret_cast<const uint4 *>(a.g)[p * P + i0] : make_uint4(0u, 0u, 0u, 0u);
    int flip = 0;
    for (int64_t t = WARP ? blockIdx.x * (kThreads / 32) + warp : blockIdx.x; t < a.n_tokens; t += step) {
        float x[V][8], d[V][8];
#pragma unroll
        for (int p = 0; p < V; p++) {
            const int c = p * P + i0;
#pragma unroll
            for (int j = 0; j < 8; j++) x[p][j] = d[p][j] = 0.f;
            if (c < runs) {
                const int64_t i = t * runs + c;
                from_e4m3x8(reinterpret_cast<const uint2 *>(a.saved)[i], up_scale(a.saved_scales[i >> 2]), x[p]);
                load8<BF16, true>(a.dn, t * a.lddn + 8 * c, d[p]);
            }
        }
        float ss, sx;
        auto sum = [&](float by) {
            ss = sx = 0.f;
#pragma unroll
            for (int p = 0; p < V; p++) {
                const uint32_t gw[4] = {gq[p].x, gq[p].y, gq[p].z, gq[p].w};
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const float gj = __uint_as_float(j & 1 ? gw[j >> 1] & 0xFFFF0000u : gw[j >> 1] << 16);
                    const float v = x[p][j] * by;
                    ss = fmaf(v, v, ss);
                    sx = fmaf(gj * d[p][j], v, sx);
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                ss += __shfl_xor_sync(0xffffffffu, ss, o);
                sx += __shfl_xor_sync(0xffffffffu, sx, o);
            }
            if (!WARP) {
                if (lane == 0) sums[flip][warp] = make_float2(ss, sx);
                __syncthreads();
                const int nw = blockDim.x >> 5;
                const float2 f = lane < nw ? sums[flip][lane] : make_float2(0.f, 0.f);
                ss = f.x, sx = f.y;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    sx += __shfl_xor_sync(0xffffffffu, sx, o);
                }
                flip ^= 1;
            }
        };
        sum(1.f);
        float by = 1.f, eps = a.eps;
        if (!(ss + eps < INFINITY && fabsf(sx) < INFINITY)) {   // the same for every thread of the row
            // sums of large values leave fp32: again of 2^-72 times the values
            by = 0x1p-72f, eps *= 0x1p-144f;
            sum(by);
        }
        // k: the factor of the values times `by`
        const float k = 1.f / sqrtf(ss / (float)a.width + eps);
        const float q = k * (sx / (float)a.width), kx = k * by;
#pragma unroll
        for (int p = 0; p < V; p++) {
            const int c = p * P + i0;
            const uint32_t gw[4] = {gq[p].x, gq[p].y, gq[p].z, gq[p].w};
            float r[8] = {};
            if (a.dres != nullptr && c < runs) load8<BF16, true>(a.dres, t * a.width + 8 * c, r);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float gj = __uint_as_float(j & 1 ? gw[j >> 1] & 0xFFFF0000u : gw[j >> 1] << 16);
                const float n = x[p][j] * by * k;
                acc[p][j] = fmaf(d[p][j], n, acc[p][j]);
                r[j] = fmaf(kx, fmaf(-n, q, gj * d[p][j]), r[j]);
            }
            store8<BF16>(a.dx, t * a.width + 8 * c, r, c < runs);
        }
    }
    float *to = gridDim.x == 1 ? a.dweight : a.part + (int64_t)blockIdx.x * a.width;
    if (WARP) {
        // the eight warps' columns, added in their order
#pragma unroll
        for (int p = 0; p < V; p++)
#pragma unroll
            for (int j = 0; j < 8; j++) cols[warp * 256 * V + 8 * (p * 32 + lane) + j] = acc[p][j];
        __syncthreads();
        for (int c = threadIdx.x; c < a.width; c += kThreads) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kThreads / 32; w++) s += cols[w * 256 * V + c];
            to[c] = s;
        }
    } else {
#pragma unroll
        for (int p = 0; p < V; p++) store8<false>(to, 8 * (p * P + i0), acc[p], p * P + i0 < runs);
    }
}

// dweight[c] = sum over the parts: 32 columns a CTA, a share of the parts a warp
__global__ void __launch_bounds__(kThreads) k_norm_grad_sum(float *dweight, const float *part, int parts, int width) {
    __shared__ float sums[kThreads / 32][32];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float s = 0.f;
#pragma unroll 8
    for (int p = warp; p < parts; p += kThreads / 32) s += part[(int64_t)p * width + c];      // width: whole blocks of 32
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0) {
        s = 0.f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; w++) s += sums[w][lane];
        dweight[c] = s;
    }
}

}  // namespace

cudaError_t launch_situ(const Ctx &c, const SituArgs &a, int bf16) {
    const int runs = a.inter / 8;
    const int64_t n8 = (int64_t)a.rows * runs;
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, dim3((unsigned)((n8 + kThreads - 1) / kThreads)), dim3(kThreads), 0, c.stream, a, n8, runs);
    };
    if (a.saved != nullptr) return bf16 ? go(k_situ<true, true>) : go(k_situ<false, true>);
    return bf16 ? go(k_situ<true, false>) : go(k_situ<false, false>);
}

cudaError_t launch_situ_grad(const Ctx &c, const SituGradArgs &a, int bf16) {
    const int runs = a.inter / 8;
    const int64_t n8 = (int64_t)a.rows * runs;
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, dim3((unsigned)((n8 + kThreads - 1) / kThreads)), dim3(kThreads), 0, c.stream, a, n8, runs);
    };
    return bf16 ? go(k_situ_grad<true>) : go(k_situ_grad<false>);
}

size_t norm_grad_scratch_bytes(int n_tokens, int width) {
    return (size_t)norm_shape(n_tokens, width).parts * width * sizeof(float);
}

template <bool WARP, int V> static cudaError_t norm_grad_t(const Ctx &c, const NormGradArgs &a, const NormShape &s, int bf16) {
    auto go = [&](auto kernel) { return launch_pdl(kernel, dim3(s.parts), dim3(s.threads), 0, c.stream, a); };
    return bf16 ? go(k_norm_grad<WARP, V, true>) : go(k_norm_grad<WARP, V, false>);
}

cudaError_t launch_norm_grad(const Ctx &c, const NormGradArgs &a, int bf16) {
    const NormShape s = norm_shape(a.n_tokens, a.width);
    cudaError_t e;
    if (s.warp) e = s.v == 1 ? norm_grad_t<true, 1>(c, a, s, bf16) : norm_grad_t<true, 4>(c, a, s, bf16);
    else e = s.v == 1 ? norm_grad_t<false, 1>(c, a, s, bf16) : s.v == 2 ? norm_grad_t<false, 2>(c, a, s, bf16)
                                                                         : norm_grad_t<false, 4>(c, a, s, bf16);
    if (e != cudaSuccess || s.parts == 1) return e;
    return launch_pdl(k_norm_grad_sum, dim3(a.width / 32), dim3(kThreads), 0, c.stream, a.dweight, (const float *)a.part,
                      s.parts, a.width);
}

}  // namespace k3mx
