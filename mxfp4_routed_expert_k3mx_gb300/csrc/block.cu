// block.cu - pairs (a token and one of its choices) in the order of their
// experts, tokens' rows taken to their pairs' places, and back with weights.
#include "blockops.cuh"
#include "mxcode.cuh"

namespace k3mx {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------- sort --
//
// A stable counting sort: the place of a pair is the number of pairs of lower
// experts, plus those of its own expert before it.  A warp owns a run of
// pairs and counts them by expert in shared memory; running sums over the
// experts, and for one expert over the warps, give each warp where its first
// pair of an expert goes; then it walks its run again, 32 pairs at a time, and
// the pairs of one expert among them rank themselves by lane.
// One CTA takes all pairs where there are few (kOneCta); else a CTA takes a
// segment, with a second kernel for the sums over the segments.

constexpr int kOneCta = 8192;         // pairs up to which one CTA takes all
constexpr int kSortWarps = 8;         // warps of a segment's CTA
constexpr int kMaxExperts = K3MX_MX_MAX_GROUPS;

// pairs of a segment
inline int segment_pairs(int n_pairs) { return n_pairs <= (1 << 18) ? 1024 : 4096; }

__device__ __forceinline__ int expert_of(const int32_t *idx, int p, int end, int n_experts, int *status) {
    if (p >= end) return -1;
    const int e = idx[p];
    if ((unsigned)e < (unsigned)n_experts) return e;
    if (e != -1 && status != nullptr) report_status(status, kStatusBadIndex, p);
    return -1;
}

// counts[e] += pairs first..end-1 of expert e (a warp and its own counts)
__device__ void count_run(uint16_t *counts, const int32_t *idx, int first, int end, int n_experts, int *status) {
    const int lane = threadIdx.x & 31;
    for (int p = first; p < end; p += 32) {
        const int e = expert_of(idx, p + lane, end, n_experts, status);
        const unsigned peers = __match_any_sync(0xffffffffu, e);
        if (e >= 0 && lane == __ffs(peers) - 1) counts[e] += (uint16_t)__popc(peers);
        __syncwarp();
    }
}
// the pairs' places: base[e] + counts[e], which moves on
__device__ void place_run(const int *base, uint16_t *counts, const int32_t *idx, int first, int end, int n_experts,
                          int32_t *perm, int32_t *place) {
    const int lane = threadIdx.x & 31;
    for (int p = first; p < end; p += 32) {
        const int e = expert_of(idx, p + lane, end, n_experts, nullptr);
        const unsigned peers = __match_any_sync(0xffffffffu, e);
        int at = -1;
        if (e >= 0) {
            at = base[e] + counts[e] + __popc(peers & ((1u << lane) - 1u));
            if (perm != nullptr) perm[at] = p + lane;
        }
        if (p + lane < end) place[p + lane] = at;
        __syncwarp();
        if (e >= 0 && lane == __ffs(peers) - 1) counts[e] += (uint16_t)__popc(peers);
        __syncwarp();
    }
}

// Exclusive sums over the experts of n[e], e = threadIdx.x + j * blockDim.x
// with J values a thread held in blocked order (thread t: t J .. t J + J - 1);
// returns the sum of all.  tmp: 33 ints.
template <int J> __device__ int exclusive_sums(int (&n)[J], int *tmp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    int mine = 0;
#pragma unroll
    for (int j = 0; j < J; j++) mine += n[j];
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) tmp[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        int v = lane < nw ? tmp[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += up;
        }
        tmp[lane] = v;
    }
    __syncthreads();
    int at = (warp > 0 ? tmp[warp - 1] : 0) + incl - mine;
#pragma unroll
    for (int j = 0; j < J; j++) {
        const int v = n[j];
        n[j] = at;
        at += v;
    }
    return tmp[nw - 1];
}

// all pairs in one CTA of 1024 threads; warps: those that get pairs
__global__ void __launch_bounds__(1024) k_sort_one(int32_t *offsets, int32_t *perm, int32_t *place, const int32_t *idx,
                                                   int n_pairs, int n_experts, int warps, int run, int *status) {
    extern __shared__ uint16_t counts[];             // [warps][n_experts]
    __shared__ int base[kMaxExperts];
    __shared__ int tmp[33];
    const int warp = threadIdx.x >> 5, e = threadIdx.x;
    for (int i = threadIdx.x; i < warps * n_experts; i += 1024) counts[i] = 0;
    pdl_wait();
    pdl_launch_dependents();
    __syncthreads();
    const int first = warp * run, end = min(first + run, n_pairs);
    if (warp < warps) count_run(counts + warp * n_experts, idx, first, end, n_experts, status);
    __syncthreads();
    int n[1] = {0};
    if (e < n_experts)
        for (int w = 0; w < warps; w++) {
            const int v = counts[w * n_experts + e];
            counts[w * n_experts + e] = (uint16_t)n[0];
            n[0] += v;
        }
    const int all = exclusive_sums(n, tmp);
    if (e < n_experts) base[e] = offsets[e] = n[0];
    if (e == 0) offsets[n_experts] = all;
    __syncthreads();
    if (warp < warps) place_run(base, counts + warp * n_experts, idx, first, end, n_experts, perm, place);
}

// hist[segment][e]: a segment's pairs by expert
__global__ void __launch_bounds__(kThreads)
k_sort_count(int *hist, const int32_t *idx, int n_pairs, int n_experts, int segment, int *status) {
    __shared__ int counts[kMaxExperts];
    for (int e = threadIdx.x; e < n_experts; e += kThreads) counts[e] = 0;
    pdl_wait();
    pdl_launch_dependents();
    __syncthreads();
    const int first = blockIdx.x * segment, end = min(first + segment, n_pairs);
    for (int p = first + threadIdx.x; p < end; p += kThreads) {
        const int e = expert_of(idx, p, end, n_experts, status);
        if (e >= 0) atomicAdd(&counts[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < n_experts; e += kThreads) hist[(int64_t)blockIdx.x * n_experts + e] = counts[e];
}

// hist[s][e] -> the sum over the segments before s, total[e] over all; a CTA
// has 32 experts, its 32 warps a share of the segments each
__global__ void __launch_bounds__(1024) k_sort_sums(int *hist, int *total, int segments, int n_experts) {
    __shared__ int sum[32][33];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
    const int share = (segments + 31) / 32, s0 = warp * share, s1 = min(s0 + share, segments);
    int n = 0;
    if (e < n_experts) {
#pragma unroll 8
        for (int s = s0; s < s1; s++) n += hist[(int64_t)s * n_experts + e];
    }
    sum[warp][lane] = n;
    __syncthreads();
    n = 0;
#pragma unroll
    for (int w = 0; w < 32; w++) n += w < warp ? sum[w][lane] : 0;
    if (e < n_experts) {
        for (int s = s0; s < s1; s++) {
            int *at = hist + (int64_t)s * n_experts + e;
            const int v = *at;
            *at = n;
            n += v;
        }
        if (warp == 31) total[e] = n;
    }
}

__global__ void __launch_bounds__(kThreads)
k_sort_place(int32_t *offsets, int32_t *perm, int32_t *place, const int32_t *idx, const int *hist, const int *total,
             int n_pairs, int n_experts, int segment) {
    __shared__ uint16_t counts[kSortWarps][kMaxExperts];
    __shared__ int base[kMaxExperts];
    __shared__ int tmp[33];
    constexpr int J = kMaxExperts / kThreads;
    const int warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < kSortWarps * kMaxExperts; i += kThreads) (&counts[0][0])[i] = 0;
    pdl_wait();
    pdl_launch_dependents();
    __syncthreads();
    const int run = segment / kSortWarps, first = blockIdx.x * segment + warp * run;
    const int end = min(first + run, n_pairs);
    count_run(counts[warp], idx, first, end, n_experts, nullptr);
    int n[J];
#pragma unroll
    for (int j = 0; j < J; j++) {
        const int e = threadIdx.x * J + j;
        n[j] = e < n_experts ? total[e] : 0;
    }
    const int all = exclusive_sums(n, tmp);          // (its barriers end the counting too)
#pragma unroll
    for (int j = 0; j < J; j++) {
        const int e = threadIdx.x * J + j;
        if (e < n_experts) {
            base[e] = n[j] + hist[(int64_t)blockIdx.x * n_experts + e];
            if (blockIdx.x == 0) offsets[e] = n[j];
            int before = 0;
#pragma unroll
            for (int w = 0; w < kSortWarps; w++) {
                const int v = counts[w][e];
                counts[w][e] = (uint16_t)before;
                before += v;
            }
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) offsets[n_experts] = all;
    __syncthreads();
    place_run(base, counts[warp], idx, first, end, n_experts, perm, place);
}

// --------------------------------------------------------- rows, by pairs --

// a pair's row, or -1 (none, or not one of n_rows: reported by `report`)
__device__ __forceinline__ int row_of(int at, int n_rows, bool report, int pair, int *status) {
    if ((unsigned)at < (unsigned)n_rows) return at;
    if (at != -1 && report) report_status(status, kStatusBadIndex, pair);
    return -1;
}

// One unit (16 bytes, or an element where rows do not begin at multiples of
// 16) of a token's row a thread: one load, a store for each of its pairs.  The
// units of the scale bytes follow those of the row.
template <typename T, typename S>
__global__ void __launch_bounds__(kThreads)
k_dispatch(T *rows, S *scales, const T *x, const S *x_scales, int64_t ldx, const int32_t *place, int n_tokens, int topk,
           int n_rows, int units, int scale_units, int *status) {
    pdl_wait();
    pdl_launch_dependents();
    const int all = units + scale_units;
    const int64_t i0 = (int64_t)blockIdx.x * kThreads, t0 = i0 / all;
    const int v = (int)(i0 - t0 * all) + threadIdx.x, u = v % all;
    const int64_t t = t0 + v / all;
    if (t >= n_tokens) return;
    const int32_t *at = place + t * topk;
    if (u < units) {
        const T q = x[t * ldx + u];
        for (int k = 0; k < topk; k++) {
            const int r = row_of(at[k], n_rows, u == 0, (int)t * topk + k, status);
            if (r >= 0) rows[(int64_t)r * units + u] = q;
        }
    } else {
        const S q = x_scales[t * scale_units + (u - units)];
        for (int k = 0; k < topk; k++) {
            const int r = row_of(at[k], n_rows, false, 0, status);
            if (r >= 0) scales[(int64_t)r * scale_units + (u - units)] = q;
        }
    }
}

// V consecutive values; V 8: whole vectors
template <bool BF16, int V> __device__ __forceinline__ void load_run(const void *base, int64_t i, float (&v)[V]) {
    if constexpr (V == 8) {
        load8<BF16, true>(base, i, v);
    } else {
#pragma unroll
        for (int j = 0; j < V; j++)
            v[j] = BF16 ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(base)[i + j] << 16)
                        : static_cast<const float *>(base)[i + j];
    }
}
template <bool BF16, int V> __device__ __forceinline__ void store_run(void *base, int64_t i, const float (&v)[V]) {
    if constexpr (V == 8) {
        if (BF16) {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + i) =
                make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
        } else {
            float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + i);
            p[0] = make_float4(v[0], v[1], v[2], v[3]);
            p[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; j++) {
            if (BF16) static_cast<uint16_t *>(base)[i + j] = __bfloat16_as_ushort(__float2bfloat16_rn(v[j]));
            else static_cast<float *>(base)[i + j] = v[j];
        }
    }
}

// A run of V columns of a token a thread, its pairs' rows U at a time.
template <bool RB, bool YB, int V>
__global__ void __launch_bounds__(kThreads) k_combine(const CombineArgs a, int runs) {
    constexpr int U = 4;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t i0 = (int64_t)blockIdx.x * kThreads, t0 = i0 / runs;
    const int v0 = (int)(i0 - t0 * runs) + threadIdx.x, u = v0 % runs;
    const int64_t t = t0 + v0 / runs;
    if (t >= a.n_tokens) return;
    const int c = u * V;
    float acc[V] = {};
    for (int k0 = 0; k0 < a.topk; k0 += U) {
        int r[U];
        float w[U], v[U][V];
#pragma unroll
        for (int j = 0; j < U; j++) {
            const int64_t p = t * a.topk + k0 + j;
            r[j] = k0 + j < a.topk ? row_of(a.place[p], a.n_rows, u == 0, (int)p, a.status) : -1;
            w[j] = r[j] >= 0 && a.w != nullptr ? a.w[p] : 1.f;
        }
#pragma unroll
        for (int j = 0; j < U; j++)
            if (r[j] >= 0) load_run<RB, V>(a.rows, (int64_t)r[j] * a.width + c, v[j]);
#pragma unroll
        for (int j = 0; j < U; j++)
            if (r[j] >= 0) {
#pragma unroll
                for (int q = 0; q < V; q++) acc[q] = fmaf(w[j], v[j][q], acc[q]);
            }
    }
    if (a.base != nullptr) {
        float b[V];
        load_run<YB, V>(a.base, t * a.width + c, b);
#pragma unroll
        for (int q = 0; q < V; q++) acc[q] += b[q];
    }
    store_run<YB, V>(a.y, t * a.width + c, acc);
}

// W warps a pair: its row and its token's gradient read once (pairs of a token
// are neighbours, so the gradient comes from L1 for all but the first), the
// row's gradient written, their product summed.
template <bool RB, bool DB, int V, int W>
__global__ void __launch_bounds__(kThreads) k_combine_grad(const CombineGradArgs a, int n_pairs) {
    __shared__ float part[kThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t p = (int64_t)blockIdx.x * (kThreads / 32 / W) + warp / W;
    const int l = (warp % W) * 32 + lane;
    float dot = 0.f;
    if (p < n_pairs) {
        const int r = row_of(a.place[p], a.n_rows, l == 0, (int)p, a.status);
        if (r >= 0) {
            const float w = a.w[p];
            const int64_t from = (int64_t)r * a.width, dfrom = p / a.topk * a.lddy;
            float acc[4] = {};
#pragma unroll 4
            for (int c = l * V; c < a.width; c += 32 * W * V) {
                float x[V], d[V];
                load_run<RB, V>(a.rows, from + c, x);
                load_run<DB, V>(a.dy, dfrom + c, d);
#pragma unroll
                for (int j = 0; j < V; j++) {
                    acc[j & 3] = fmaf(x[j], d[j], acc[j & 3]);
                    d[j] *= w;
                }
                store_run<RB, V>(a.drows, from + c, d);
            }
            dot = (acc[0] + acc[1]) + (acc[2] + acc[3]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    }
    if (W > 1) {
        if (lane == 0) part[warp] = dot;
        __syncthreads();
        dot = 0.f;
#pragma unroll
        for (int i = 0; i < W; i++) dot += part[warp / W * W + i];
    }
    if (p < n_pairs && l == 0) a.dw[p] = dot;
}

bool multiple16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename T, typename S>
cudaError_t dispatch_t(const Ctx &c, const DispatchArgs &a, int units, int64_t ld, int scale_units) {
    const int64_t n = (int64_t)a.n_tokens * (units + scale_units);
    return launch_pdl(k_dispatch<T, S>, dim3((unsigned)((n + kThreads - 1) / kThreads)), dim3(kThreads), 0, c.stream,
                      static_cast<T *>(a.rows), reinterpret_cast<S *>(a.scales), static_cast<const T *>(a.x),
                      reinterpret_cast<const S *>(a.x_scales), ld, a.place, a.n_tokens, a.topk, a.n_rows, units,
                      scale_units, a.status);
}

}  // namespace

size_t sort_scratch_bytes(int n_pairs, int n_experts) {
    if (n_pairs <= kOneCta) return 0;
    const int segment = segment_pairs(n_pairs);
    return ((size_t)(n_pairs + segment - 1) / segment + 1) * n_experts * sizeof(int);
}

cudaError_t launch_sort(const Ctx &c, int32_t *offsets, int32_t *perm, int32_t *place, const int32_t *idx, int n_pairs,
                        int n_experts, void *scratch) {
    if (n_pairs <= kOneCta) {
        const int run = (n_pairs + 1023) / 1024 * 32, warps = (n_pairs + run - 1) / run;
        constexpr int kMost = 32 * kMaxExperts * (int)sizeof(uint16_t);
        static std::atomic<uint64_t> done{0};
        const cudaError_t e = ensure_smem((const void *)k_sort_one, kMost, done);
        if (e != cudaSuccess) return e;
        return launch_pdl(k_sort_one, dim3(1), dim3(1024), (size_t)warps * n_experts * sizeof(uint16_t), c.stream, offsets,
                          perm, place, idx, n_pairs, n_experts, warps, run, c.status);
    }
    const int segment = segment_pairs(n_pairs), segments = (n_pairs + segment - 1) / segment;
    int *hist = static_cast<int *>(scratch), *total = hist + (size_t)segments * n_experts;
    cudaError_t e = launch_pdl(k_sort_count, dim3(segments), dim3(kThreads), 0, c.stream, hist, idx, n_pairs, n_experts,
                               segment, c.status);
    if (e != cudaSuccess) return e;
    e = launch_pdl(k_sort_sums, dim3((n_experts + 31) / 32), dim3(1024), 0, c.stream, hist, total, segments, n_experts);
    if (e != cudaSuccess) return e;
    return launch_pdl(k_sort_place, dim3(segments), dim3(kThreads), 0, c.stream, offsets, perm, place, idx,
                      (const int *)hist, (const int *)total, n_pairs, n_experts, segment);
}

cudaError_t launch_dispatch(const Ctx &c, const DispatchArgs &a) {
    const int64_t bytes = (int64_t)a.width * a.elem;
    const int sb = a.x_scales != nullptr ? a.width / 32 : 0;
    const bool wide = multiple16(a.rows) && multiple16(a.x) && bytes % 16 == 0 && a.ldx * a.elem % 16 == 0;
    const bool words = sb % 4 == 0 && ((reinterpret_cast<uintptr_t>(a.scales) | reinterpret_cast<uintptr_t>(a.x_scales)) & 3u) == 0;
    if (wide)
        return words ? dispatch_t<uint4, uint32_t>(c, a, (int)(bytes / 16), a.ldx * a.elem / 16, sb / 4)
                     : dispatch_t<uint4, uint8_t>(c, a, (int)(bytes / 16), a.ldx * a.elem / 16, sb);
    if (a.elem == 4) return dispatch_t<uint32_t, uint8_t>(c, a, a.width, a.ldx, sb);
    if (a.elem == 2) return dispatch_t<uint16_t, uint8_t>(c, a, a.width, a.ldx, sb);
    return dispatch_t<uint8_t, uint8_t>(c, a, a.width, a.ldx, sb);
}

cudaError_t launch_combine(const Ctx &c, const CombineArgs &a, int y_bf16, int rows_bf16) {
    const bool wide = a.width % 8 == 0 && multiple16(a.rows) && multiple16(a.y) && multiple16(a.base);
    const int runs = wide ? a.width / 8 : a.width;
    const int64_t n = (int64_t)a.n_tokens * runs;
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, dim3((unsigned)((n + kThreads - 1) / kThreads)), dim3(kThreads), 0, c.stream, a, runs);
    };
    if (wide)
        return rows_bf16 ? (y_bf16 ? go(k_combine<true, true, 8>) : go(k_combine<true, false, 8>))
                         : (y_bf16 ? go(k_combine<false, true, 8>) : go(k_combine<false, false, 8>));
    return rows_bf16 ? (y_bf16 ? go(k_combine<true, true, 1>) : go(k_combine<true, false, 1>))
                     : (y_bf16 ? go(k_combine<false, true, 1>) : go(k_combine<false, false, 1>));
}

template <int V, int W>
static cudaError_t combine_grad_t(const Ctx &c, const CombineGradArgs &a, int dy_bf16, int rows_bf16) {
    const int n = a.n_tokens * a.topk, per = kThreads / 32 / W;
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, dim3((unsigned)((n + per - 1) / per)), dim3(kThreads), 0, c.stream, a, n);
    };
    return rows_bf16 ? (dy_bf16 ? go(k_combine_grad<true, true, V, W>) : go(k_combine_grad<true, false, V, W>))
                     : (dy_bf16 ? go(k_combine_grad<false, true, V, W>) : go(k_combine_grad<false, false, V, W>));
}

cudaError_t launch_combine_grad(const Ctx &c, const CombineGradArgs &a, int dy_bf16, int rows_bf16) {
    const bool wide = a.width % 8 == 0 && a.lddy % 8 == 0 && multiple16(a.rows) && multiple16(a.drows) && multiple16(a.dy);
    const bool few = (int64_t)a.n_tokens * a.topk <= 4 * c.num_sms;
    if (wide) return few ? combine_grad_t<8, 8>(c, a, dy_bf16, rows_bf16) : combine_grad_t<8, 1>(c, a, dy_bf16, rows_bf16);
    return few ? combine_grad_t<1, 8>(c, a, dy_bf16, rows_bf16) : combine_grad_t<1, 1>(c, a, dy_bf16, rows_bf16);
}

}  // namespace k3mx
