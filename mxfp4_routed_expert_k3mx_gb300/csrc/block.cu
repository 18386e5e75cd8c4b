// block.cu - pairs (a token and one of its choices) in the order of their
// experts, tokens' rows taken to their pairs' places, and back with weights.
//
// All of it moves data: what counts is that each row is read and written once,
// in whole vectors, with enough of them on their way, and for few tokens that
// a call is one latency after another as seldom as can be.  Measured (repeated
// calls, inputs larger than L2; a copy reaches 6.78 TB/s):
//   dispatch 4096 tokens x 16, 3584 MXFP8      41 us, 6.3 TB/s; 1 token 1.6 us
//   combine 65536 rows of 3584 fp32            141 us, 7.1 TB/s; bf16 75 us, 6.6
//   combine 1 token, 16 rows of 7168 bf16      1.5 us
//   its gradient, 65536 rows of 3584 bf16      155 us, 6.3 TB/s; 1 token 2.2 us
// Rows that do not begin at multiples of 16 bytes (an odd width) are put together
// from whole vectors by dispatch and, of bf16, by combine (32768 rows of 3001 in 83
// us, 136 an element at a time, 36 by their bytes) and its gradient (77 us, 100,
// 62); fp32 rows (16384 of 3001 combined in 50 us, 36 by their bytes) and other
// types take an element at a time.
#include <type_traits>

#include "blockops.cuh"
#include "mxcode.cuh"

namespace k3mx {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------- sort --
//
// A stable counting sort: the place of a pair is the number of pairs of lower
// experts, plus those of its own expert before it.  A warp owns a run of pairs,
// 32 of them at a time, and counts them by expert in shared memory; what was
// there before its 32, and the lanes below of the same expert, are a pair's
// rank in the run, kept with its expert in a register.  Sums over the experts,
// and for one expert over the warps, then give each run its places.
// Measured (16 choices of 896, on the device): one CTA up to 2048 pairs (16 pairs
// 1.9 us, 1024 3.8, 2048 4.5; 4096 6.7, 16384 19.6); to 65536 a CTA for each
// 1024, after a kernel that counts them, which adds up the counts of all for
// itself (2048 pairs 5.1 us, 4112 5.6, 65536 7.9; by three kernels 7.7); beyond,
// one more kernel adds them up (131072 9.3, by two 18; 1 M 24.6).  An SM's
// scattered stores bound it: four bytes cost as much as a sector's 32.

constexpr int kOneCta = 2048, kTwoKernels = 65536;       // pairs up to which
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
// pairs of a CTA: one a thread, or two
inline int segment_pairs(int n_pairs) { return n_pairs <= kTwoKernels ? kSortThreads : 2 * kSortThreads; }
constexpr int kMaxExperts = K3MX_MX_MAX_GROUPS;

__device__ __forceinline__ int expert_of(const int32_t *idx, int p, int end, int n_experts, int *status) {
    if (p >= end) return -1;
    const int e = idx[p];
    if ((unsigned)e < (unsigned)n_experts) return e;
    if (e != -1 && status != nullptr) report_status(status, kStatusBadIndex, p);
    return -1;
}

// A warp's run: pairs first + 32 i + lane, i < N.  rank[i]: expert << 16 | rank
// in the run, or -1; counts[e]: the run's.
template <int N>
__device__ __forceinline__ void rank_run(uint16_t *counts, int (&rank)[N], const int32_t *idx, int first, int end,
                                         int n_experts, int *status) {
    const int lane = threadIdx.x & 31, bits = 32 - __clz(n_experts - 1);
#pragma unroll
    for (int i = 0; i < N; i++) rank[i] = expert_of(idx, first + 32 * i + lane, end, n_experts, status);
#pragma unroll
    for (int i = 0; i < N; i++) {
        if (first + 32 * i >= end) break;
        const int e = rank[i];
        // the lanes of the same expert, a vote a bit
        unsigned peers = __ballot_sync(0xffffffffu, e >= 0);
        for (int b = 0; b < bits; b++) {
            const bool set = e >> b & 1;
            const unsigned m = __ballot_sync(0xffffffffu, set);
            peers &= set ? m : ~m;
        }
        int before = 0;
        if (e >= 0) before = counts[e];
        __syncwarp();
        if (e >= 0) {
            if (lane == __ffs(peers) - 1) counts[e] = (uint16_t)(before + __popc(peers));
            rank[i] = e << 16 | (before + __popc(peers & ((1u << lane) - 1u)));
        }
        __syncwarp();
    }
}
// The same pairs' places: base[e] + counts[e], which by now are the pairs of e
// in the warps before, + rank
template <int N>
__device__ __forceinline__ void place_run(const int *base, const uint16_t *counts, const int (&rank)[N], int first, int end,
                                          int32_t *perm, int32_t *place) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < N; i++) {
        const int p = first + 32 * i + lane;
        if (p >= end) break;
        int at = -1;
        if (rank[i] >= 0) {
            const int e = rank[i] >> 16;
            at = base[e] + counts[e] + (rank[i] & 0xFFFF);
            if (perm != nullptr) perm[at] = p;
        }
        place[p] = at;
    }
}
// counts[w][e] -> those of the warps before w; returns the sum over all
__device__ __forceinline__ int before_warps(uint16_t *counts, int e, int warps, int n_experts) {
    int n = 0;
#pragma unroll 4
    for (int w = 0; w < warps; w++) {
        const int v = counts[w * n_experts + e];
        counts[w * n_experts + e] = (uint16_t)n;
        n += v;
    }
    return n;
}

// The sum of n over the threads before this one; `all`: over all 1024.  tmp: 33
// ints.
__device__ int exclusive_sum(int n, int *tmp, int &all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) tmp[warp] = incl;
    __syncthreads();
    int v = tmp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += up;
    }
    all = __shfl_sync(0xffffffffu, v, 31);
    const int below = __shfl_sync(0xffffffffu, v, (warp + 31) & 31);
    return (warp > 0 ? below : 0) + incl - n;
}

// all pairs in one CTA; warps: those that get pairs, N 32s each
template <int N>
__global__ void __launch_bounds__(kSortThreads) k_sort_one(int32_t *offsets, int32_t *perm, int32_t *place, const int32_t *idx,
                                                           int n_pairs, int n_experts, int warps, int *status) {
    extern __shared__ int sorted[];                  // [n_pairs], for perm: a store of a sector's four bytes from here
    uint16_t *counts = reinterpret_cast<uint16_t *>(sorted + n_pairs);     // costs as much as of all 32; [warps][n_experts]
    __shared__ int base[kMaxExperts];
    __shared__ int tmp[33];
    const int warp = threadIdx.x >> 5, e = threadIdx.x;
    for (int i = threadIdx.x; i < warps * n_experts; i += kSortThreads) counts[i] = 0;
    pdl_wait();
    pdl_launch_dependents();
    __syncthreads();
    int rank[N];
    const int first = warp * N * 32;
    if (warp < warps) rank_run(counts + warp * n_experts, rank, idx, first, n_pairs, n_experts, status);
    __syncthreads();
    int all;
    const int at = exclusive_sum(e < n_experts ? before_warps(counts, e, warps, n_experts) : 0, tmp, all);
    if (e < n_experts) base[e] = offsets[e] = at;
    if (e == 0) offsets[n_experts] = all;
    __syncthreads();
    if (warp < warps) place_run(base, counts + warp * n_experts, rank, first, n_pairs, perm != nullptr ? sorted : nullptr, place);
    if (perm != nullptr) {
        __syncthreads();
        for (int i = threadIdx.x; i < all; i += kSortThreads) perm[i] = sorted[i];
    }
}

// hist[segment][e]: a segment's pairs by expert
__global__ void __launch_bounds__(kSortThreads)
k_sort_count(int *hist, const int32_t *idx, int n_pairs, int n_experts, int segment, int *status) {
    __shared__ int counts[kMaxExperts];
    counts[threadIdx.x] = 0;
    pdl_wait();
    pdl_launch_dependents();
    __syncthreads();
    const int first = blockIdx.x * segment, end = min(first + segment, n_pairs);
    for (int p = first + threadIdx.x; p < end; p += kSortThreads) {
        const int e = expert_of(idx, p, end, n_experts, status);
        if (e >= 0) atomicAdd(&counts[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < n_experts; e += kSortThreads) hist[(int64_t)blockIdx.x * n_experts + e] = counts[e];
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
        constexpr int B = 8;                         // loads before the stores to the same places
        for (int s = s0; s < s1; s += B) {
            int v[B];
#pragma unroll
            for (int j = 0; j < B; j++) v[j] = s + j < s1 ? hist[(int64_t)(s + j) * n_experts + e] : 0;
#pragma unroll
            for (int j = 0; j < B; j++)
                if (s + j < s1) {
                    hist[(int64_t)(s + j) * n_experts + e] = n;
                    n += v[j];
                }
        }
        if (warp == 31) total[e] = n;
    }
}

// N pairs a thread.  ALONE: hist holds the segments' counts, else the sums of
// k_sort_sums
template <int N, bool ALONE>
__global__ void __launch_bounds__(kSortThreads)
k_sort_place(int32_t *offsets, int32_t *perm, int32_t *place, const int32_t *idx, const int *hist, const int *total,
             int n_pairs, int n_experts, int segments) {
    extern __shared__ uint16_t counts[];             // [kSortWarps][n_experts]
    __shared__ int base[kMaxExperts];
    __shared__ int tmp[33];
    const int warp = threadIdx.x >> 5, e = threadIdx.x;
    for (int i = threadIdx.x; i < kSortWarps * n_experts; i += kSortThreads) counts[i] = 0;
    pdl_wait();
    pdl_launch_dependents();
    __syncthreads();
    int mine = 0, before = 0;
    if (e < n_experts) {
        if (ALONE) {
            // 32 loads at a time, then 8, the last ones some of them twice
            const int *h = hist + e;
            int s = 0;
            for (; s + 32 <= segments; s += 32, h += 32 * n_experts) {
                int v[32];
#pragma unroll
                for (int j = 0; j < 32; j++) v[j] = h[j * n_experts];
#pragma unroll
                for (int j = 0; j < 32; j++) {
                    mine += v[j];
                    before += s + j < (int)blockIdx.x ? v[j] : 0;
                }
            }
            for (; s < segments; s += 8, h += 8 * n_experts) {
                int v[8];
#pragma unroll
                for (int j = 0; j < 8; j++) v[j] = h[min(j, segments - 1 - s) * n_experts];
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    mine += s + j < segments ? v[j] : 0;
                    before += s + j < (int)blockIdx.x ? v[j] : 0;
                }
            }
        } else {
            mine = total[e];
            before = hist[(int64_t)blockIdx.x * n_experts + e];
        }
    }
    int rank[N];
    const int first = (blockIdx.x * kSortWarps + warp) * N * 32, end = min((int)(blockIdx.x + 1) * N * kSortThreads, n_pairs);
    rank_run(counts + warp * n_experts, rank, idx, first, end, n_experts, nullptr);
    int all;
    const int at = exclusive_sum(mine, tmp, all);        // (its barrier ends the counting too)
    if (e < n_experts) {
        before_warps(counts, e, kSortWarps, n_experts);
        base[e] = at + before;
        if (blockIdx.x == 0) offsets[e] = at;
    }
    if (blockIdx.x == 0 && e == 0) offsets[n_experts] = all;
    __syncthreads();
    place_run(base, counts + warp * n_experts, rank, first, end, perm, place);
}

// --------------------------------------------------------- rows, by pairs --

// a pair's row, or -1 (none, or not one of n_rows: reported by `report`)
__device__ __forceinline__ int row_of(int at, int n_rows, bool report, int pair, int *status) {
    if ((unsigned)at < (unsigned)n_rows) return at;
    if (at != -1 && report) report_status(status, kStatusBadIndex, pair);
    return -1;
}

// A CTA is by tokens of bx threads.  The rows that a token's pairs name are
// listed in shared memory first; then a thread loads a unit of 16 bytes of its
// row and stores it to each of them.  The units of the scale bytes follow those
// of the row.
constexpr int kListed = 32;           // pairs of a token listed at a time

// The first warp of a token's threads lists its pairs k0.. that name a row;
// the entry is make(row, pair).
template <typename E, typename F>
__device__ __forceinline__ void list_rows(E *list, int *listed, const int32_t *place, int64_t t, bool live, int topk, int n_rows,
                                          int k0, bool report, int *status, F make) {
    const int k = k0 + threadIdx.x;
    const int64_t p = t * topk + k;
    const int r = live && k < topk ? row_of(place[p], n_rows, report, (int)p, status) : -1;
    const unsigned some = __ballot_sync(0xffffffffu, r >= 0);
    if (r >= 0) list[__popc(some & ((1u << threadIdx.x) - 1u))] = make(r, p);
    if (threadIdx.x == 0) *listed = __popc(some);
}

template <typename S>
__global__ void __launch_bounds__(kThreads)
k_dispatch(uint4 *rows, S *scales, const uint4 *x, const S *x_scales, int64_t ldx, const int32_t *place, int n_tokens, int topk,
           int n_rows, int units, int scale_units, int chunks, int *status) {
    __shared__ int list[kThreads / 32][kListed], listed[kThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int tile = blockIdx.x / chunks, chunk = blockIdx.x - tile * chunks, u = chunk * blockDim.x + threadIdx.x;
    const int64_t t = (int64_t)tile * blockDim.y + threadIdx.y;
    const bool live = t < n_tokens, row = live && u < units, scale = live && u >= units && u < units + scale_units;
    uint4 q = make_uint4(0u, 0u, 0u, 0u);
    S b = 0;
    if (row) q = x[t * ldx + u];
    if (scale) b = x_scales[t * scale_units + (u - units)];
    for (int k0 = 0; k0 < topk; k0 += kListed) {
        if (k0 > 0) __syncthreads();
        if (threadIdx.x < 32)
            list_rows(list[threadIdx.y], &listed[threadIdx.y], place, t, live, topk, n_rows, k0, chunk == 0, status,
                      [](int r, int64_t) { return r; });
        __syncthreads();
        const int n = listed[threadIdx.y];
        const int *mine = list[threadIdx.y];
        if (row) {
#pragma unroll 4
            for (int j = 0; j < n; j++) rows[(int64_t)mine[j] * units + u] = q;
        } else if (scale) {
#pragma unroll 4
            for (int j = 0; j < n; j++) scales[(int64_t)mine[j] * scale_units + (u - units)] = b;
        }
    }
}

// Rows that begin anywhere.  A CTA has 4096 bytes of a token's row in shared
// memory and writes them to each pair's row as that one lies: whole 16 bytes,
// put together from two of the row's by one shift for all, and elements at both
// ends.  (An element a thread, 16384 rows of 3001 bf16 took 46.6 us, so 22.5.)
template <typename T>
__global__ void __launch_bounds__(kThreads)
k_dispatch_odd(T *rows, uint8_t *scales, const T *x, const uint8_t *x_scales, int64_t ldx, const int32_t *place, int n_tokens,
               int topk, int n_rows, int width, int scale_units, int chunks, int *status) {
    constexpr int kBytes = 16 * kThreads, kElems = kBytes / sizeof(T), kVec = 16 / sizeof(T);
    __shared__ uint4 buffer[kThreads + 2];
    __shared__ int list[1][kListed], listed;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t = blockIdx.x / chunks;
    const int chunk = (int)(blockIdx.x - t * chunks), c0 = chunk * kElems, n = min(kElems, width - c0);
    T *mine = reinterpret_cast<T *>(buffer);
    for (int i = threadIdx.x; i < n; i += kThreads) mine[i] = x[t * ldx + c0 + i];
    for (int k0 = 0; k0 < topk; k0 += kListed) {
        __syncthreads();
        if (threadIdx.x < 32)
            list_rows(list[0], &listed, place, t, true, topk, n_rows, k0, chunk == 0, status, [](int r, int64_t) { return r; });
        __syncthreads();
        for (int j = 0; j < listed; j++) {
            T *to = rows + (int64_t)list[0][j] * width + c0;
            // elements before the first 16-byte boundary, vectors from it on
            const int head = min(n, (int)((16u - (reinterpret_cast<uintptr_t>(to) & 15u)) & 15u) / (int)sizeof(T));
            const int vectors = (n - head) / kVec, tail = head + vectors * kVec;
            if ((int)threadIdx.x < vectors) {
                const int from = head * sizeof(T);          // bytes, below 16, the same for all
                const uint4 a = buffer[threadIdx.x], b = buffer[threadIdx.x + 1];
                const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                const uint32_t sel = 0x3210u + 0x1111u * (from & 3);
                uint32_t o[4];
                auto shift = [&](auto q) {
#pragma unroll
                    for (int i = 0; i < 4; i++) o[i] = __byte_perm(w[q.value + i], w[(q.value + i + 1) & 7], sel);
                };
                switch (from >> 2) {
                case 0: shift(std::integral_constant<int, 0>()); break;
                case 1: shift(std::integral_constant<int, 1>()); break;
                case 2: shift(std::integral_constant<int, 2>()); break;
                default: shift(std::integral_constant<int, 3>()); break;
                }
                reinterpret_cast<uint4 *>(to + head)[threadIdx.x] = make_uint4(o[0], o[1], o[2], o[3]);
            }
            if ((int)threadIdx.x < head) to[threadIdx.x] = mine[threadIdx.x];
            if ((int)threadIdx.x < n - tail) to[tail + threadIdx.x] = mine[tail + threadIdx.x];
        }
        if (chunk == 0 && scale_units > 0)
            for (int j = 0; j < listed; j++)
                for (int i = threadIdx.x; i < scale_units; i += kThreads)
                    scales[(int64_t)list[0][j] * scale_units + i] = x_scales[t * scale_units + i];
    }
}

// V consecutive values; V 8: whole vectors, 2: whole pairs
template <bool BF16, int V> __device__ __forceinline__ void load_run(const void *base, int64_t i, float (&v)[V]) {
    if constexpr (V == 8) {
        load8<BF16, true>(base, i, v);
    } else if constexpr (V == 2) {
        if (BF16) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(base) + i);
            v[0] = __uint_as_float(w << 16), v[1] = __uint_as_float(w & 0xFFFF0000u);
        } else {
            const float2 w = *reinterpret_cast<const float2 *>(static_cast<const float *>(base) + i);
            v[0] = w.x, v[1] = w.y;
        }
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
    } else if constexpr (V == 2) {
        if (BF16) *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(base) + i) = bf16x2(v[0], v[1]);
        else *reinterpret_cast<float2 *>(static_cast<float *>(base) + i) = make_float2(v[0], v[1]);
    } else {
#pragma unroll
        for (int j = 0; j < V; j++) {
            if (BF16) static_cast<uint16_t *>(base)[i + j] = __bfloat16_as_ushort(__float2bfloat16_rn(v[j]));
            else static_cast<float *>(base)[i + j] = v[j];
        }
    }
}

// Combine.  A CTA is by tokens of bx threads; a thread has R runs of eight
// columns, bx runs apart.  The tokens' pairs that name a row are listed in
// shared memory first (where the row begins, the weight), so that what is left
// a row and run is its load, the conversion and eight products: with the places
// looked up, checked and multiplied by every thread, 4096 x 16 rows of 3584 bf16
// took 115 us where the bytes take 74.
struct Listed {
    int64_t at;        // elements
    float w;
};
template <bool RB, bool YB, int R, int U>
__global__ void __launch_bounds__(kThreads, 4) k_combine(const CombineArgs a, int runs, int chunks) {
    __shared__ Listed list[kThreads / 32][kListed];
    __shared__ int listed[kThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int tile = blockIdx.x / chunks, chunk = blockIdx.x - tile * chunks;
    const int64_t t = (int64_t)tile * blockDim.y + threadIdx.y;
    const int u0 = chunk * blockDim.x * R + threadIdx.x, bx = blockDim.x;
    const bool live = t < a.n_tokens;
    constexpr bool kEarly = U == 2;                // few rows: base is on its way with them
    Raw<YB> base[R];
    float acc[R][8] = {};
    auto load_base = [&](int q) {
        base[q].zero();
        if (a.base != nullptr && live && u0 + q * bx < runs) base[q].load(a.base, t * a.width + 8 * (u0 + q * bx));
    };
    if (kEarly) {
#pragma unroll
        for (int q = 0; q < R; q++) load_base(q);
    }
    const Listed *mine = list[threadIdx.y];
    for (int k0 = 0; k0 < a.topk; k0 += kListed) {
        if (k0 > 0) __syncthreads();
        if (threadIdx.x < 32)
            list_rows(list[threadIdx.y], &listed[threadIdx.y], a.place, t, live, a.topk, a.n_rows, k0, chunk == 0, a.status,
                      [&](int r, int64_t p) { return Listed{(int64_t)r * a.width, a.w != nullptr ? a.w[p] : 1.f}; });
        __syncthreads();
        const int n = listed[threadIdx.y];
        for (int j0 = 0; j0 < n; j0 += U) {
            Raw<RB> v[U][R];
            float w[U];
#pragma unroll
            for (int j = 0; j < U; j++)
                if (j0 + j < n) {
                    const Listed l = mine[j0 + j];
                    w[j] = l.w;
#pragma unroll
                    for (int q = 0; q < R; q++)
                        if (u0 + q * bx < runs) v[j][q].load(a.rows, l.at + 8 * (u0 + q * bx));
                }
#pragma unroll
            for (int j = 0; j < U; j++)
                if (j0 + j < n) {
#pragma unroll
                    for (int q = 0; q < R; q++) {
                        float x[8];
                        v[j][q].values(x);
#pragma unroll
                        for (int e = 0; e < 8; e++) acc[q][e] = fmaf(w[j], x[e], acc[q][e]);
                    }
                }
        }
    }
    if (!live) return;
#pragma unroll
    for (int q = 0; q < R; q++)
        if (u0 + q * bx < runs) {
            if (a.base != nullptr) {
                float b[8];
                if (!kEarly) load_base(q);
                base[q].values(b);
#pragma unroll
                for (int e = 0; e < 8; e++) acc[q][e] += b[e];
            }
            store_run<YB, 8>(a.y, t * a.width + 8 * (u0 + q * bx), acc[q]);
        }
}

// Few tokens: a CTA has 256 / K runs of one token and brings them of K choices at
// a time to shared memory, a run a thread; the first 1024 / K threads then add
// two columns each, k rising as in k_combine, so that a token's bits do not depend
// on how many others the call has.  (Device time, here and by k_combine: 1 token,
// 16 rows of 7168 bf16 1.5 and 4.4 us, 8 x 3584 1.8 and 3.1, 36 x 7168 3.8 and
// 5.0, 500 x 512, 8 rows each, 2.5 and 3.5; 64 x 7168, 8 rows each, 3.75 and 3.6.)
constexpr int64_t kCombineFew = 1 << 15;      // runs of all tokens
// Eight choices at a time, not sixteen: few CTAs wait for the second eight, many
// are half as many then (1 token, 16 rows: 1.95 and 1.54 us, 8 2.15 and 1.84; 16 x
// 7168 2.26 and 2.46, 36 3.81 and 4.00).
constexpr int64_t kCombineEights = 1 << 13;   // runs of all tokens above which
template <bool RB, bool YB, int K>
__global__ void __launch_bounds__(kThreads) k_combine_few(const CombineArgs a, int chunks) {
    constexpr int kRuns = kThreads / K;
    __shared__ Raw<RB> part[K][kRuns];
    __shared__ __align__(16) float weight[K];
    pdl_wait();
    pdl_launch_dependents();
    const int u = threadIdx.x % kRuns, i = threadIdx.x / kRuns;
    const int64_t t = blockIdx.x / chunks;
    const int c0 = (int)(blockIdx.x - t * chunks) * 8 * kRuns, c = c0 + 8 * u, mine = c0 + 2 * threadIdx.x;
    const bool adds = threadIdx.x < 4 * kRuns && mine < a.width;
    float base[2] = {0.f, 0.f}, acc[2] = {0.f, 0.f};
    if (a.base != nullptr && adds) load_run<YB, 2>(a.base, t * a.width + mine, base);
    for (int k0 = 0; k0 < a.topk; k0 += K) {
        const int k = k0 + i;
        const int64_t p = t * a.topk + k;
        const int r = k < a.topk ? row_of(a.place[p], a.n_rows, c == 0, (int)p, a.status) : -1;
        const float w = r < 0 ? 0.f : a.w != nullptr ? a.w[p] : 1.f;
        Raw<RB> v;
        v.minus_zero();                            // (0 times -0 leaves any sum as it is)
        if (r >= 0 && c < a.width) v.load(a.rows, (int64_t)r * a.width + c);
        if (k0 > 0) __syncthreads();
        if (u == 0) weight[i] = w;
        part[i][u] = v;
        __syncthreads();
        if (adds) {
#pragma unroll
            for (int j = 0; j < K; j++) {
                float x[2];
                load_run<RB, 2>(part[j], 2 * threadIdx.x, x);
                acc[0] = fmaf(weight[j], x[0], acc[0]);
                acc[1] = fmaf(weight[j], x[1], acc[1]);
            }
        }
    }
    if (adds) {
        acc[0] += base[0], acc[1] += base[1];
        store_run<YB, 2>(a.y, t * a.width + mine, acc);
    }
}

// Vector i of an array of 16-bit elements that begins at 16 bytes and has `end`
// of them, zeros behind it
__device__ __forceinline__ uint4 vector_of(const void *base, int64_t i, int64_t end) {
    if (8 * (i + 1) <= end) return static_cast<const uint4 *>(base)[i];
    uint32_t w[4] = {};
    for (int e = 0; e < 8 && 8 * i + e < end; e++) w[e >> 1] |= (uint32_t)static_cast<const uint16_t *>(base)[8 * i + e] << 16 * (e & 1);
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// eight elements from the one `from` (0..7) of two neighbouring vectors on, two to a word
__device__ __forceinline__ void shifted(uint4 lo, uint4 hi, int from, uint32_t (&b)[4]) {
    uint32_t q[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    const uint32_t sel = from & 1 ? 0x5432u : 0x3210u;
#pragma unroll
    for (int i = 0; i < 6; i++) q[i] = from & 4 ? q[i + 2] : q[i];
#pragma unroll
    for (int i = 0; i < 5; i++) q[i] = from & 2 ? q[i + 1] : q[i];
#pragma unroll
    for (int i = 0; i < 4; i++) b[i] = __byte_perm(q[i], q[i + 1], sel);
}

// Rows of bf16 that begin anywhere, in an array that begins at 16 bytes: a
// thread's eight columns are put together from two of the array's vectors by one
// shift for all of a row (its second vector is the next thread's first, and
// comes from L1).  What a CTA has summed goes through shared memory, so that y,
// which may begin anywhere too, is written by neighbouring threads.
template <bool YB>
__global__ void __launch_bounds__(128) k_combine_shift(const CombineArgs a, int chunks) {
    constexpr int U = 4;
    __shared__ Listed list[kListed];
    __shared__ int listed;
    __shared__ float4 out[256];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t = blockIdx.x / chunks, end = (int64_t)a.n_rows * a.width;       // elements of rows
    const int chunk = (int)(blockIdx.x - t * chunks), c0 = chunk * 8 * blockDim.x, c = c0 + 8 * threadIdx.x;
    float acc[8] = {};
    for (int k0 = 0; k0 < a.topk; k0 += kListed) {
        if (k0 > 0) __syncthreads();
        if (threadIdx.x < 32)
            list_rows(list, &listed, a.place, t, true, a.topk, a.n_rows, k0, chunk == 0, a.status,
                      [&](int r, int64_t p) { return Listed{(int64_t)r * a.width, a.w != nullptr ? a.w[p] : 1.f}; });
        __syncthreads();
        const int n = c < a.width ? listed : 0;
        for (int j0 = 0; j0 < n; j0 += U) {
            uint4 lo[U], hi[U];
#pragma unroll
            for (int j = 0; j < U; j++)
                if (j0 + j < n) {
                    const int64_t v = (list[j0 + j].at + c) >> 3;                   // the first vector with a column of ours
                    lo[j] = vector_of(a.rows, v, end);
                    hi[j] = vector_of(a.rows, v + 1, end);
                }
#pragma unroll
            for (int j = 0; j < U; j++)
                if (j0 + j < n) {
                    const int from = (int)list[j0 + j].at & 7;                     // elements
                    const float w = list[j0 + j].w;
                    uint32_t b[4];
                    shifted(lo[j], hi[j], from, b);
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        acc[2 * i] = fmaf(w, __uint_as_float(b[i] << 16), acc[2 * i]);
                        acc[2 * i + 1] = fmaf(w, __uint_as_float(b[i] & 0xFFFF0000u), acc[2 * i + 1]);
                    }
                }
        }
    }
    out[2 * threadIdx.x] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    out[2 * threadIdx.x + 1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    __syncthreads();
    for (int i = threadIdx.x; i < 8 * (int)blockDim.x && c0 + i < a.width; i += blockDim.x) {
        float s[1] = {reinterpret_cast<const float *>(out)[i]}, b[1] = {0.f};
        if (a.base != nullptr) load_run<YB, 1>(a.base, t * a.width + c0 + i, b);
        s[0] += b[0];
        store_run<YB, 1>(a.y, t * a.width + c0 + i, s);
    }
}

// Rows that begin anywhere: four columns a thread, a CTA's threads apart, so
// that a row's address is worked out once for the four.
template <bool RB, bool YB>
__global__ void __launch_bounds__(kThreads) k_combine_odd(const CombineArgs a, int chunks) {
    constexpr int U = 4, C = 4;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t = blockIdx.x / chunks;
    const int c0 = (int)(blockIdx.x - t * chunks) * C * blockDim.x + threadIdx.x, B = blockDim.x;
    float acc[C] = {};
    for (int k0 = 0; k0 < a.topk; k0 += U) {
        float v[U][C], w[U];
#pragma unroll
        for (int j = 0; j < U; j++) {
            const int64_t p = t * a.topk + k0 + j;
            const int r = k0 + j < a.topk ? row_of(a.place[p], a.n_rows, c0 == 0, (int)p, a.status) : -1;
            w[j] = r >= 0 && a.w != nullptr ? a.w[p] : 1.f;
#pragma unroll
            for (int q = 0; q < C; q++) {
                float x[1] = {0.f};
                if (r >= 0 && c0 + q * B < a.width) load_run<RB, 1>(a.rows, (int64_t)r * a.width + c0 + q * B, x);
                v[j][q] = x[0];
            }
            if (r < 0) w[j] = 0.f;                 // (0 times the zeros in its place)
        }
#pragma unroll
        for (int j = 0; j < U; j++)
#pragma unroll
            for (int q = 0; q < C; q++) acc[q] = fmaf(w[j], v[j][q], acc[q]);
    }
#pragma unroll
    for (int q = 0; q < C; q++)
        if (c0 + q * B < a.width) {
            float s[1] = {acc[q]}, b[1] = {0.f};
            if (a.base != nullptr) load_run<YB, 1>(a.base, t * a.width + c0 + q * B, b);
            s[0] += b[0];
            store_run<YB, 1>(a.y, t * a.width + c0 + q * B, s);
        }
}

// W warps a pair: its row and its token's gradient read once (pairs of a token
// are neighbours, so the gradient comes from L1 for all but the first), the
// row's gradient written, their product summed.  W = 1: a warp walks pairs, the
// next one's place and weight on their way while it works on a row.  U runs of
// both are loaded at a time: the stores, which may be to where the rows are,
// keep the compiler from loading ahead.
template <bool RB, bool DB, int V, int W, int U, int M>
__global__ void __launch_bounds__(kThreads, M) k_combine_grad(const CombineGradArgs a, int n_pairs) {
    __shared__ float part[kThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    constexpr int kAtOnce = kThreads / 32 / W, S = 32 * W * V;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = (warp % W) * 32 + lane;
    int p = blockIdx.x * kAtOnce + warp / W;
    int at = -1;
    float w = 0.f;
    auto look = [&](int p) {
        at = p < n_pairs ? a.place[p] : -1;
        w = p < n_pairs ? a.w[p] : 0.f;
    };
    look(p);
    for (; W > 1 ? p < n_pairs : p - warp < n_pairs; p += gridDim.x * kAtOnce) {
        const int r = row_of(at, a.n_rows, l == 0, p, a.status);
        const float wp = w;
        look(p + gridDim.x * kAtOnce);
        float acc[4] = {};
        if (r >= 0) {
            const int64_t from = (int64_t)r * a.width, dfrom = (int64_t)(p / a.topk) * a.lddy;
            for (int c0 = l * V; c0 < a.width; c0 += U * S) {
                float x[U][V], d[U][V];
#pragma unroll
                for (int k = 0; k < U; k++)
                    if (c0 + k * S < a.width) {
                        load_run<RB, V>(a.rows, from + c0 + k * S, x[k]);
                        load_run<DB, V>(a.dy, dfrom + c0 + k * S, d[k]);
                    }
#pragma unroll
                for (int k = 0; k < U; k++)
                    if (c0 + k * S < a.width) {
#pragma unroll
                        for (int j = 0; j < V; j++) {
                            acc[(k * V + j) & 3] = fmaf(x[k][j], d[k][j], acc[(k * V + j) & 3]);
                            d[k][j] *= wp;
                        }
                        store_run<RB, V>(a.drows, from + c0 + k * S, d[k]);
                    }
            }
        }
        float dot = (acc[0] + acc[1]) + (acc[2] + acc[3]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (W > 1) {
            if (lane == 0) part[warp] = dot;
            __syncthreads();
            dot = 0.f;
#pragma unroll
            for (int i = 0; i < W; i++) dot += part[warp / W * W + i];
            __syncthreads();
        }
        if (p < n_pairs && l == 0) a.dw[p] = dot;
    }
}

// The same for bf16 rows that begin anywhere in arrays that begin at 16 bytes: a
// row and its gradient have whole vectors at the same places, and elements at
// both ends; the token's gradient is put together by one shift for all.  (32768
// rows of 3001: 77 us, 100 an element at a time, 92 with registers for four CTAs
// an SM and not six.)
__global__ void __launch_bounds__(kThreads, 6) k_combine_grad_shift(const CombineGradArgs a, int n_pairs) {
    pdl_wait();
    pdl_launch_dependents();
    constexpr int kAtOnce = kThreads / 32;
    const int lane = threadIdx.x & 31;
    int p = blockIdx.x * kAtOnce + (threadIdx.x >> 5);
    const int64_t dend = (int64_t)(a.n_tokens - 1) * a.lddy + a.width;
    int at = -1;
    float w = 0.f;
    auto look = [&](int p) {
        at = p < n_pairs ? a.place[p] : -1;
        w = p < n_pairs ? a.w[p] : 0.f;
    };
    look(p);
    for (; p < n_pairs; p += gridDim.x * kAtOnce) {
        const int r = row_of(at, a.n_rows, lane == 0, p, a.status);
        const float wp = w;
        look(p + gridDim.x * kAtOnce);
        float acc[2] = {};
        if (r >= 0) {
            const int64_t from = (int64_t)r * a.width, dfrom = (int64_t)(p / a.topk) * a.lddy;
            const int head = min(a.width, (int)(-from & 7)), vectors = (a.width - head) / 8, tail = head + 8 * vectors;
            const uint4 *rows = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.rows) + from + head);
            uint4 *drows = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.drows) + from + head);
            const int64_t d0 = (dfrom + head) >> 3;
            const int shift = (int)(dfrom + head) & 7;
#pragma unroll 1
            for (int v = lane; v < vectors; v += 32) {
                const uint4 x = rows[v], lo = vector_of(a.dy, d0 + v, dend), hi = vector_of(a.dy, d0 + v + 1, dend);
                uint32_t b[4], o[4];
                shifted(lo, hi, shift, b);
                const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float d0 = __uint_as_float(b[i] << 16), d1 = __uint_as_float(b[i] & 0xFFFF0000u);
                    acc[0] = fmaf(__uint_as_float(xw[i] << 16), d0, acc[0]);
                    acc[1] = fmaf(__uint_as_float(xw[i] & 0xFFFF0000u), d1, acc[1]);
                    o[i] = bf16x2(wp * d0, wp * d1);
                }
                drows[v] = make_uint4(o[0], o[1], o[2], o[3]);
            }
            // the elements before and behind, at most seven each
            const int c = lane < 8 ? lane : tail + lane - 8;
            if (lane < 8 ? c < head : lane < 16 && c < a.width) {
                float x[1], d[1];
                load_run<true, 1>(a.rows, from + c, x);
                load_run<true, 1>(a.dy, dfrom + c, d);
                acc[0] = fmaf(x[0], d[0], acc[0]);
                d[0] *= wp;
                store_run<true, 1>(a.drows, from + c, d);
            }
        }
        float dot = acc[0] + acc[1];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (lane == 0) a.dw[p] = dot;
    }
}

bool multiple16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename S> cudaError_t dispatch_t(const Ctx &c, const DispatchArgs &a, int units, int64_t ld, int scale_units) {
    // threads of a token, in CTAs of 128 and less, or sharing one with other tokens
    const int all = units + scale_units, chunks = (all + 127) / 128, bx = ((all + chunks - 1) / chunks + 31) / 32 * 32;
    const int by = chunks > 1 ? 1 : kThreads / bx;
    const int64_t tiles = (a.n_tokens + by - 1) / by;
    return launch_pdl(k_dispatch<S>, dim3((unsigned)(tiles * chunks)), dim3(bx, by), 0, c.stream, static_cast<uint4 *>(a.rows),
                      reinterpret_cast<S *>(a.scales), static_cast<const uint4 *>(a.x), reinterpret_cast<const S *>(a.x_scales),
                      ld, a.place, a.n_tokens, a.topk, a.n_rows, units, scale_units, chunks, a.status);
}
template <typename T> cudaError_t dispatch_odd_t(const Ctx &c, const DispatchArgs &a, int scale_units) {
    const int chunks = (int)(((int64_t)a.width * sizeof(T) + 16 * kThreads - 1) / (16 * kThreads));
    return launch_pdl(k_dispatch_odd<T>, dim3((unsigned)((int64_t)a.n_tokens * chunks)), dim3(kThreads), 0, c.stream,
                      static_cast<T *>(a.rows), a.scales, static_cast<const T *>(a.x), a.x_scales, a.ldx, a.place, a.n_tokens,
                      a.topk, a.n_rows, a.width, scale_units, chunks, a.status);
}

}  // namespace

size_t sort_scratch_bytes(int n_pairs, int n_experts) {
    if (n_pairs <= kOneCta) return 0;
    const int segment = segment_pairs(n_pairs);
    return ((size_t)(n_pairs + segment - 1) / segment + 1) * n_experts * sizeof(int);
}

cudaError_t launch_sort(const Ctx &c, int32_t *offsets, int32_t *perm, int32_t *place, const int32_t *idx, int n_pairs,
                        int n_experts, void *scratch) {
    constexpr int kMost = kSortWarps * kMaxExperts * (int)sizeof(uint16_t);
    if (n_pairs <= kOneCta) {
        auto go = [&](auto kernel, int n, std::atomic<uint64_t> &done) {
            const int warps = (n_pairs + 32 * n - 1) / (32 * n);
            const cudaError_t e = ensure_smem((const void *)kernel, kMost + kOneCta * (int)sizeof(int), done);
            if (e != cudaSuccess) return e;
            return launch_pdl(kernel, dim3(1), dim3(kSortThreads),
                              n_pairs * sizeof(int) + (size_t)warps * n_experts * sizeof(uint16_t), c.stream, offsets, perm,
                              place, idx, n_pairs, n_experts, warps, c.status);
        };
        static std::atomic<uint64_t> done1{0}, done4{0};
        return n_pairs <= 256 ? go(k_sort_one<1>, 1, done1) : go(k_sort_one<4>, 4, done4);
    }
    const int segment = segment_pairs(n_pairs), segments = (n_pairs + segment - 1) / segment;
    int *hist = static_cast<int *>(scratch), *total = hist + (size_t)segments * n_experts;
    cudaError_t e = launch_pdl(k_sort_count, dim3(segments), dim3(kSortThreads), 0, c.stream, hist, idx, n_pairs, n_experts,
                               segment, c.status);
    if (e != cudaSuccess) return e;
    auto place_all = [&](auto kernel, std::atomic<uint64_t> &done) {
        const cudaError_t e = ensure_smem((const void *)kernel, kMost, done);
        if (e != cudaSuccess) return e;
        return launch_pdl(kernel, dim3(segments), dim3(kSortThreads), (size_t)kSortWarps * n_experts * sizeof(uint16_t), c.stream,
                          offsets, perm, place, idx, (const int *)hist, (const int *)total, n_pairs, n_experts, segments);
    };
    static std::atomic<uint64_t> done_two{0}, done_three{0};
    if (n_pairs <= kTwoKernels) return place_all(k_sort_place<1, true>, done_two);
    e = launch_pdl(k_sort_sums, dim3((n_experts + 31) / 32), dim3(1024), 0, c.stream, hist, total, segments, n_experts);
    if (e != cudaSuccess) return e;
    return place_all(k_sort_place<2, false>, done_three);
}

cudaError_t launch_dispatch(const Ctx &c, const DispatchArgs &a) {
    const int64_t bytes = (int64_t)a.width * a.elem;
    const int sb = a.x_scales != nullptr ? a.width / 32 : 0;
    const bool wide = multiple16(a.rows) && multiple16(a.x) && bytes % 16 == 0 && a.ldx * a.elem % 16 == 0;
    const bool words = sb % 4 == 0 && ((reinterpret_cast<uintptr_t>(a.scales) | reinterpret_cast<uintptr_t>(a.x_scales)) & 3u) == 0;
    if (wide)
        return words ? dispatch_t<uint32_t>(c, a, (int)(bytes / 16), a.ldx * a.elem / 16, sb / 4)
                     : dispatch_t<uint8_t>(c, a, (int)(bytes / 16), a.ldx * a.elem / 16, sb);
    if (a.elem == 4) return dispatch_odd_t<uint32_t>(c, a, sb);
    if (a.elem == 2) return dispatch_odd_t<uint16_t>(c, a, sb);
    return dispatch_odd_t<uint8_t>(c, a, sb);
}

template <bool RB, bool YB> static cudaError_t combine_t(const Ctx &c, const CombineArgs &a) {
    if (a.width % 8 != 0 || !multiple16(a.rows) || !multiple16(a.y) || !multiple16(a.base)) {
        if constexpr (RB)
            if (multiple16(a.rows)) {
                const int runs = (a.width + 7) / 8, chunks = (runs + 63) / 64, threads = ((runs + chunks - 1) / chunks + 31) / 32 * 32;
                return launch_pdl(k_combine_shift<YB>, dim3((unsigned)((int64_t)a.n_tokens * chunks)), dim3(threads), 0, c.stream, a,
                                  chunks);
            }
        int threads = (a.width + 3) / 4;
        threads = threads < kThreads ? (threads + 31) / 32 * 32 : kThreads;
        const int chunks = (a.width + 4 * threads - 1) / (4 * threads);
        return launch_pdl(k_combine_odd<RB, YB>, dim3((unsigned)((int64_t)a.n_tokens * chunks)), dim3(threads), 0, c.stream, a, chunks);
    }
    const int runs = a.width / 8;
    if ((int64_t)a.n_tokens * runs <= kCombineFew && a.topk > 2) {
        auto few = [&](auto kernel, int per) {
            const int chunks = (runs + per - 1) / per;
            return launch_pdl(kernel, dim3((unsigned)(a.n_tokens * chunks)), dim3(kThreads), 0, c.stream, a, chunks);
        };
        return a.topk <= 8 || (int64_t)a.n_tokens * runs > kCombineEights ? few(k_combine_few<RB, YB, 8>, kThreads / 8)
                                                                          : few(k_combine_few<RB, YB, 16>, kThreads / 16);
    }
    auto go = [&](auto kernel, int per) {
        // (CTAs of 64 threads, or of 256 that share 4 tokens and more)
        const int threads = (runs + per - 1) / per, parts = (threads + 63) / 64;
        const int bx = ((threads + parts - 1) / parts + 31) / 32 * 32, by = parts > 1 ? 1 : kThreads / bx;
        const int64_t tiles = (a.n_tokens + by - 1) / by;
        return launch_pdl(kernel, dim3((unsigned)(tiles * parts)), dim3(bx, by), 0, c.stream, a, runs, parts);
    };
    // two runs a thread of bf16 rows (65536 of 3584 75 us, one 79, four 167; 2 x 8192
    // of 7168 84, 117, 122), one of fp32 (141, two 311); two choices at a time where
    // there are no more (2 x 8192 of 7168 bf16 84 us, four 98; 1 x 16384 147 and 176)
    constexpr int R = RB ? 2 : 1;
    return a.topk <= 2 ? go(k_combine<RB, YB, R, 2>, R) : go(k_combine<RB, YB, R, 4>, R);
}

cudaError_t launch_combine(const Ctx &c, const CombineArgs &a, int y_bf16, int rows_bf16) {
    return rows_bf16 ? (y_bf16 ? combine_t<true, true>(c, a) : combine_t<true, false>(c, a))
                     : (y_bf16 ? combine_t<false, true>(c, a) : combine_t<false, false>(c, a));
}

template <bool RB, bool DB> static cudaError_t combine_grad_t(const Ctx &c, const CombineGradArgs &a) {
    const int n = a.n_tokens * a.topk;
    // pairs a CTA has at once, and CTAs an SM at most (0: one for each)
    auto go = [&](auto kernel, int per, int most) {
        const int ctas = (n + per - 1) / per;
        return launch_pdl(kernel, dim3((unsigned)(most == 0 || ctas < most * c.num_sms ? ctas : most * c.num_sms)), dim3(kThreads),
                          0, c.stream, a, n);
    };
    const bool wide = a.width % 8 == 0 && a.lddy % 8 == 0 && multiple16(a.rows) && multiple16(a.drows) && multiple16(a.dy);
    const bool few = n <= 4 * c.num_sms;                  // (16 pairs of 7168 bf16: 2.2 us, 4 by a warp each)
    if constexpr (RB && DB)
        if (!wide && !few && multiple16(a.rows) && multiple16(a.drows) && multiple16(a.dy)) return go(k_combine_grad_shift, 8, 6);
    if (!wide) return few ? go(k_combine_grad<RB, DB, 1, 8, 4, 4>, 1, 0) : go(k_combine_grad<RB, DB, 1, 1, 8, 4>, 8, 4);
    if (few) return go(k_combine_grad<RB, DB, 8, 8, 2, 4>, 1, 0);
    // bf16: many warps with a run each in flight (65536 x 3584 155 us, 182 with
    // two runs; 131072 x 512 50 and 69); fp32: two, and a CTA for each eight
    // pairs (32768 x 3584 149 us, 190 walked)
    if constexpr (RB) return go(k_combine_grad<RB, DB, 8, 1, 1, 6>, 8, 6);
    else return go(k_combine_grad<RB, DB, 8, 1, 2, 4>, 8, 0);
}

cudaError_t launch_combine_grad(const Ctx &c, const CombineGradArgs &a, int dy_bf16, int rows_bf16) {
    return rows_bf16 ? (dy_bf16 ? combine_grad_t<true, true>(c, a) : combine_grad_t<true, false>(c, a))
                     : (dy_bf16 ? combine_grad_t<false, true>(c, a) : combine_grad_t<false, false>(c, a));
}

}  // namespace k3mx
