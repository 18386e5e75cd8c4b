// mxprod.cu - products of MXFP8 activations with MXFP4 weights of any shape,
// dense or by groups of rows with a weight matrix each:
//   y[t][n] = sum_b 2^(sx[t][b] + sw[n][b] - 254) sum_{i<32} x[t][32b+i] w[n][32b+i]
// on the block-scaled 5th-generation tensor cores (tcgen05 kind::mxf8f6f4:
// e2m1 x e4m3, one ue8m0 scale per 32 columns on either side), which
// multiply the codes as they lie in memory exactly and add in fp32.
//
// Work.  A unit is at most NT rows of one group, an item a unit and a tile of
// 128 outputs; weights are the MMA's A (M = 128 outputs), activations its B
// (N = the unit's rows), so one row costs 16 columns and not 128.  A cluster
// of S CTAs shares an item: CTA r multiplies the r-th part of its inner
// width, and the parts meet in shared memory (each CTA adds and stores 128 / S
// of the outputs, in rank order, so results do not depend on timing).
// Clusters take items round robin.  Per CTA, the inner width streams in
// stages of 128 columns:
//   warp 0      copies: TMA of the weight tile (128 rows x 128 codes, 64 B a
//               row in memory, spread to 128 B in shared memory, 128-byte
//               swizzle) and of the unit's rows (boxes of 64 and 16 rows)
//   warp 1      the tile's scales: four bytes a row and stage, loaded some
//               stages ahead into registers, stored as the 32-line source of
//               tcgen05.cp; a block of scale 255 gets scale 0 and its codes
//               are zeroed once the tile landed, so it adds exactly 0
//   warp 2      owns TMEM; lane 0 copies scales to TMEM and issues the MMAs
//   warp 3      the rows' scales, as warp 1's
//   warps 4-11  epilogue: two warps to a lane quarter, half the rows each
// Every wait is bounded; one that gives up is reported on the device status
// word and every role leaves its loop.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "mxops.cuh"
#include "tc.cuh"
#include "tmaps.cuh"

namespace k3mx {
namespace {

constexpr int kStageCols = 128;
constexpr int kWTile = 128 * 128;          // weight tile in shared memory (spread codes)
constexpr int kWTileTx = 128 * 64;         // bytes its copy moves
constexpr int kAtom = 512;                 // scales of 128 rows and a stage
constexpr int kThreads = 12 * 32, kEpi0 = 4, kEpiThreads = 8 * 32;

// outputs of an item that one CTA of a cluster of S adds and stores
__host__ __device__ constexpr int split_rows(int S) { return S == 3 ? 48 : 128 / S; }

template <int NT_> struct Shape {
    static constexpr int NT = NT_;                                   // rows of a unit
    static constexpr int ATOMS = (NT + 127) / 128;
    static constexpr int STAGE = kWTile + NT * 128 + (NT == 256 ? 4 : 2) * kAtom;
    static constexpr int SA = NT == 32 ? 9 : NT == 64 ? 7 : 4;       // stages
    static constexpr int NBUF = NT == 256 ? 1 : 2;                   // accumulators
    static constexpr bool SPLIT = NT < 256;
    // parts of the outputs this CTA adds: [S][NT][split_rows(S)] fp32 (largest at S = 3)
    static constexpr int RED = SPLIT ? NT * 3 * 48 * 4 : 0;
    static constexpr int TABLES = 2 * (K3MX_MX_MAX_GROUPS + 8) * 4;
    static constexpr int SMEM = 1024 + 1024 + SA * STAGE + RED + TABLES;
    static constexpr int SF_COL = NBUF * NT, SF_STEP = 4 + 4 * ATOMS;  // TMEM columns: accumulators, then scales
    static constexpr int TMEM_COLS = 512;
    static_assert(STAGE % 1024 == 0 && SMEM <= 227 * 1024, "shared memory");
    static_assert(SF_COL + SA * SF_STEP <= TMEM_COLS, "TMEM");
};

struct Maps {
    CUtensorMap w, x64, x16;
};

struct Hdr {
    uint64_t tfull[16], sfull[16], empty[16], accf[2], acce[2], done, redfull, redfree;
    uint32_t tmem;
    int abort;
    int part[kThreads / 32];
};

struct Item {
    int g, mt, off, ntok;
};

__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity) {
    const uint32_t lim = wait_polls();
    for (uint32_t i = 0; i < lim; i++) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity), "r"(kWaitSuspendNs)
            : "memory");
        if (ok) return true;
    }
    return false;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// Scale words of a stream of stages: lane l loads the words of rows l, l + 32,
// ... (R of them) D stages ahead.  begin(i) gives item i's address for the
// lane's first row and the mask of its rows that exist; use(p, words) takes
// stage p's.
template <int R, int D, typename Begin, typename Use>
__device__ __forceinline__ bool stage_words(int total, int per_item, size_t row_step, Begin begin, Use use) {
    uint32_t q[D][R];
    const uint8_t *base = nullptr;
    uint32_t live = 0;
    int loaded = 0, c = 0, i = 0;
    auto load = [&](uint32_t (&d)[R]) {
        if (loaded >= total) return;
        if (c == 0) begin(i, base, live);
#pragma unroll
        for (int r = 0; r < R; r++)
            d[r] = (live >> r) & 1 ? __ldg(reinterpret_cast<const uint32_t *>(base + r * row_step + 4 * c)) : 0u;
        loaded++;
        if (++c == per_item) {
            c = 0;
            i++;
        }
    };
#pragma unroll
    for (int d = 0; d < D; d++) load(q[d]);
    for (int p = 0; p < total; p += D) {
#pragma unroll
        for (int d = 0; d < D; d++)
            if (p + d < total) {
                if (!use(p + d, q[d])) return false;
                load(q[d]);
            }
    }
    return true;
}

template <int NT>
__global__ void __launch_bounds__(kThreads, 1)
k_mx_product(const ProdArgs a, const int y_bf16, const int S, const __grid_constant__ Maps maps) {
    using Sh = Shape<NT>;
    constexpr int SA = Sh::SA, NBUF = Sh::NBUF;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Hdr *hd = reinterpret_cast<Hdr *>(smem);
    const uint32_t ring = smem_addr(smem) + 1024;
    float *red = reinterpret_cast<float *>(smem + 1024 + SA * Sh::STAGE);
    int *ustart = reinterpret_cast<int *>(smem + 1024 + SA * Sh::STAGE + Sh::RED);   // first unit of each group
    int *goff = ustart + K3MX_MX_MAX_GROUPS + 8;                                     // first row of each group
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t tfull0 = smem_addr(hd->tfull), sfull0 = smem_addr(hd->sfull), empty0 = smem_addr(hd->empty);
    const uint32_t accf0 = smem_addr(hd->accf), acce0 = smem_addr(hd->acce), done = smem_addr(&hd->done);
    const uint32_t redfull = smem_addr(&hd->redfull), redfree = smem_addr(&hd->redfree);
    const int rank = S > 1 ? (int)(blockIdx.x % S) : 0;       // %cluster_ctarank of a 1-D cluster

    if (tid == 0) {
        for (int i = 0; i < SA; i++) {
            mbar_init(tfull0 + 8 * i, 1);
            mbar_init(sfull0 + 8 * i, 64);
            mbar_init(empty0 + 8 * i, 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(accf0 + 8 * i, 1);
            mbar_init(acce0 + 8 * i, kEpiThreads);
        }
        mbar_init(done, 1);
        mbar_init(redfull, S * (kEpiThreads / 32));
        mbar_init(redfree, S * (kEpiThreads / 32));
        hd->abort = 0;
        fence_mbar_init();
    }
    if (warp == 2) tmem_alloc(smem_addr(&hd->tmem), Sh::TMEM_COLS);
    pdl_wait();
    pdl_launch_dependents();

    // units of every group (0 for one whose offsets are unusable)
    constexpr int GPT = (K3MX_MX_MAX_GROUPS + kThreads - 1) / kThreads;
    int nu[GPT], mine = 0;
#pragma unroll
    for (int k = 0; k < GPT; k++) {
        const int g = tid * GPT + k;
        nu[k] = 0;
        if (g < a.n_groups) {
            const int lo = a.offsets ? __ldg(a.offsets + g) : 0, hi = a.offsets ? __ldg(a.offsets + g + 1) : a.n_rows;
            if (lo < 0 || hi < lo || hi > a.n_rows) {
                if (blockIdx.x == 0) report_status(a.status, kStatusBadIndex, g);
            } else {
                nu[k] = (hi - lo + NT - 1) / NT;
            }
            goff[g] = lo;
            if (g == a.n_groups - 1) goff[a.n_groups] = hi;
        }
        mine += nu[k];
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) hd->part[warp] = incl;
    __syncthreads();
    int at = incl - mine;
    for (int w = 0; w < warp; w++) at += hd->part[w];
#pragma unroll
    for (int k = 0; k < GPT; k++) {
        const int g = tid * GPT + k;
        if (g < a.n_groups) ustart[g] = at;
        at += nu[k];
        if (g == a.n_groups - 1) ustart[a.n_groups] = at;
    }
    tc_fence_before();
    if (S > 1) cluster_sync();               // also: every CTA's barriers are initialised
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = hd->tmem;
    volatile int *abort_flag = &hd->abort;

    const int MT = (a.out + 127) / 128, KC = a.in / kStageCols, G = a.in / 32;
    const int c0 = KC * rank / S, kcs = KC * (rank + 1) / S - c0;      // this CTA's stages of every item
    const int first = blockIdx.x / S, step = gridDim.x / S;
    const int items = ustart[a.n_groups] * MT;
    const int n_items = items > first ? (items - first + step - 1) / step : 0;
    const int total = n_items * kcs;

    // item `first + k * step`: groups in order, in a group tile by tile, a
    // tile's units together (they share its weights in L2)
    auto item_at = [&](int k) {
        const int it = first + k * step, q = it / MT;
        int lo = 0, hi = a.n_groups - 1;                    // last group with ustart <= q
        while (lo < hi) {
            const int m = (lo + hi + 1) >> 1;
            if (ustart[m] <= q) lo = m;
            else hi = m - 1;
        }
        const int u0 = ustart[lo], ug = ustart[lo + 1] - u0, l = it - u0 * MT;
        const int mt = l / ug, u = l - mt * ug;
        const long long cnt = goff[lo + 1] - goff[lo];
        const int r0 = (int)(cnt * u / ug), r1 = (int)(cnt * (u + 1) / ug);
        return Item{lo, mt, goff[lo] + r0, r1 - r0};
    };
    auto fail = [&](int detail) {
        report_status(a.status, kStatusWaitTimeout, detail);
        *abort_flag = 1;
    };

    if (warp == 0) {
        // ---------------------------------------------------- copies --
        if (lane == 0) {
            const uint64_t wpol = l2_evict_first_policy(), xpol = l2_evict_last_policy();
            int p = 0;
            for (int k = 0; k < n_items && !*abort_flag; k++) {
                const Item it = item_at(k);
                const int rows = (it.ntok + 15) & ~15, wy = it.g * a.out + it.mt * 128;
                bool ok = true;
                for (int c = c0; c < c0 + kcs; c++, p++) {
                    const int s = p % SA;
                    if (!mbar_wait(empty0 + 8 * s, ((p / SA) & 1) ^ 1)) {
                        fail(400);
                        ok = false;
                        break;
                    }
                    const uint32_t st = ring + s * Sh::STAGE, bar = tfull0 + 8 * s;
                    mbar_arrive_expect_tx(bar, kWTileTx + rows * 128);
                    tma_2d(st, &maps.w, c * kStageCols, wy, bar, wpol);
                    int r = 0;
                    if (NT >= 64)
                        for (; r + 64 <= rows; r += 64)
                            tma_2d(st + kWTile + r * 128, &maps.x64, c * kStageCols, it.off + r, bar, xpol);
                    for (; r < rows; r += 16)
                        tma_2d(st + kWTile + r * 128, &maps.x16, c * kStageCols, it.off + r, bar, xpol);
                }
                if (!ok) break;
            }
            // copies still in flight (after a wait gave up) land before the CTA leaves
            if (!drain_ring(tfull0, SA, p)) report_status(a.status, kStatusWaitTimeout, 401);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------- the tile's scales --
        auto begin = [&](int k, const uint8_t *&base, uint32_t &live) {
            const Item it = item_at(k);
            const int row = it.mt * 128 + lane;
            base = a.wscales + ((size_t)it.g * a.out + row) * G + 4 * c0;
            live = 0;
#pragma unroll
            for (int r = 0; r < 4; r++) live |= (row + 32 * r < a.out ? 1u : 0u) << r;
        };
        auto use = [&](int p, const uint32_t (&w)[4]) {
            const int s = p % SA;
            if (*abort_flag || !mbar_wait(empty0 + 8 * s, ((p / SA) & 1) ^ 1)) {
                if (lane == 0) fail(410);
                return false;
            }
            const uint32_t st = ring + s * Sh::STAGE;
            const uint32_t nan = nan_scale_mask(w[0]) | nan_scale_mask(w[1]) | nan_scale_mask(w[2]) | nan_scale_mask(w[3]);
            if (__any_sync(0xffffffffu, nan != 0)) {        // rare
                if (!mbar_wait(tfull0 + 8 * s, (p / SA) & 1)) {
                    if (lane == 0) fail(411);
                    return false;
                }
#pragma unroll
                for (int r = 0; r < 4; r++) zero_nan_groups_x128(st, lane + 32 * r, w[r]);
            }
            sts128(st + kWTile + NT * 128 + 16 * lane, drop_nan_scales(w[0]), drop_nan_scales(w[1]),
                   drop_nan_scales(w[2]), drop_nan_scales(w[3]));
            fence_async_smem();
            mbar_arrive(sfull0 + 8 * s);
            return true;
        };
        stage_words<4, 8>(total, kcs, (size_t)32 * G, begin, use);
    } else if (warp == 3) {
        // -------------------------------------------- the rows' scales --
        constexpr int R = NT / 32;
        auto begin = [&](int k, const uint8_t *&base, uint32_t &live) {
            const Item it = item_at(k);
            base = a.scales + ((size_t)it.off + lane) * G + 4 * c0;
            live = 0;
#pragma unroll
            for (int r = 0; r < R; r++) live |= (lane + 32 * r < it.ntok ? 1u : 0u) << r;
        };
        auto use = [&](int p, const uint32_t (&w)[R]) {
            const int s = p % SA;
            if (*abort_flag || !mbar_wait(empty0 + 8 * s, ((p / SA) & 1) ^ 1)) {
                if (lane == 0) fail(420);
                return false;
            }
            const uint32_t at = ring + s * Sh::STAGE + kWTile + NT * 128 + kAtom + 16 * lane;
#pragma unroll
            for (int r = 0; r < R; r += 4)
                sts128(at + (r >> 2) * kAtom, w[r], r + 1 < R ? w[r + 1 < R ? r + 1 : 0] : 0u,
                       r + 2 < R ? w[r + 2 < R ? r + 2 : 0] : 0u, r + 3 < R ? w[r + 3 < R ? r + 3 : 0] : 0u);
            fence_async_smem();
            mbar_arrive(sfull0 + 8 * s);
            return true;
        };
        stage_words<R, NT == 256 ? 4 : 8>(total, kcs, (size_t)32 * G, begin, use);
    } else if (warp == 2) {
        // ------------------------------------------------ MMA issuer --
        if (lane == 0) {
            int p = 0, itn = 0;
            bool run = true, ready = false;
            for (int k = 0; k < n_items && run && !*abort_flag; k++, itn++) {
                const Item it = item_at(k);
                const int n = (it.ntok + 15) & ~15, b = itn % NBUF;
                uint32_t idk[4];
#pragma unroll
                for (int ks = 0; ks < 4; ks++) idk[ks] = idesc_e2m1_e4m3(n, ks);
                if (!mbar_wait(acce0 + 8 * b, ((itn / NBUF) & 1) ^ 1)) {
                    fail(430);
                    break;
                }
                tc_fence_after();
                for (int c = 0; c < kcs; c++, p++) {
                    const int s = p % SA, ph = (p / SA) & 1;
                    if (!ready && (!mbar_wait(tfull0 + 8 * s, ph) || !mbar_wait(sfull0 + 8 * s, ph))) {
                        fail(431);
                        run = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t st = ring + s * Sh::STAGE, xt = st + kWTile, sf = xt + NT * 128;
                    const uint32_t sfa = tmem + Sh::SF_COL + s * Sh::SF_STEP, sfb = sfa + 4;
                    tmem_cp_atom(sfa, desc_atom(sf, 128));
                    tmem_cp_atom(sfb, desc_atom(sf + kAtom, 128));
                    if (Sh::ATOMS == 2 && n > 128) tmem_cp_atom(sfb + 4, desc_atom(sf + 2 * kAtom, 128));
                    const uint32_t d = tmem + b * NT;
#pragma unroll
                    for (int ks = 0; ks < 4; ks++) {
                        const uint64_t ad = umma_desc_sw128(st + 32 * ks), bd = umma_desc_sw128(xt + 32 * ks);
                        const uint32_t acc = (c | ks) != 0 ? 1u : 0u;
                        if (ks == 3) {
                            // the barriers of the next stage, polled beside the last MMA
                            const int s2 = (p + 1) % SA, ph2 = ((p + 1) / SA) & 1;
                            ready = mma_mxf8f6f4_poll3(d, ad, bd, idk[ks], sfa, sfb, acc, tfull0 + 8 * s2, ph2,
                                                       sfull0 + 8 * s2, ph2, sfull0 + 8 * s2, ph2);
                        } else {
                            mma_mxf8f6f4(d, ad, bd, idk[ks], sfa, sfb, acc);
                        }
                    }
                    umma_commit(empty0 + 8 * s);
                }
                if (run) umma_commit(accf0 + 8 * b);
            }
            umma_commit(done);
        }
        __syncwarp();
    } else {
        // -------------------------------------------------- epilogue --
        constexpr int HC = NT / 2;                            // rows of the unit to a warp
        const int q4 = warp & 3, half = (warp - kEpi0) >> 2;
        const int o = 32 * q4 + lane;                         // output within the tile
        const uint32_t quarter = (uint32_t)(32 * q4) << 16;
        const int RS = split_rows(S);
        for (int k = 0; k < n_items && !*abort_flag; k++) {
            const Item it = item_at(k);
            const int b = k % NBUF, n0 = half * HC, n1 = min(it.ntok, n0 + HC);
            if (!mbar_wait(accf0 + 8 * b, (k / NBUF) & 1)) {
                if (lane == 0) fail(440);
                break;
            }
            tc_fence_after();
            float v[HC];
#pragma unroll
            for (int j = 0; j < HC; j += 16)
                if (n0 + j < n1) {
                    uint32_t u[16];
                    tmem_ld16(tmem + quarter + b * NT + n0 + j, u);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; i++) v[j + i] = __uint_as_float(u[i]);
                }
            tc_fence_before();
            mbar_arrive(acce0 + 8 * b);
            auto store = [&](int out, int n, float val) {
                const size_t at = (size_t)(it.off + n) * a.out + out;
                if (y_bf16) static_cast<__nv_bfloat16 *>(a.y)[at] = __float2bfloat16_rn(val);
                else static_cast<float *>(a.y)[at] = val;
            };
            if (!Sh::SPLIT || S == 1) {
                const int out = it.mt * 128 + o;
                if (out < a.out)
#pragma unroll
                    for (int j = 0; j < HC; j++)
                        if (n0 + j < n1) store(out, n0 + j, v[j]);
                continue;
            }
            // this CTA's parts to the CTAs that add them, once those are done
            // with the item before
            if (k > 0 && !wait_cluster(redfree, (k - 1) & 1)) {
                if (lane == 0) fail(441);
                break;
            }
            {
                const int own = o / RS;
                const uint32_t to = map_rank(smem_addr(red) + ((rank * NT + n0) * RS + o - own * RS) * 4, own);
#pragma unroll
                for (int j = 0; j < HC; j++)
                    if (n0 + j < n1) st_cluster(to + j * RS * 4, v[j]);
            }
            __syncwarp();
            if (lane < S) arrive_cluster(map_rank(redfull, lane));
            if (!wait_cluster(redfull, k & 1)) {
                if (lane == 0) fail(442);
                break;
            }
            const int cnt = min(RS, 128 - rank * RS);
            for (int i = tid - kEpi0 * 32; i < cnt * it.ntok; i += kEpiThreads) {
                const int n = i / cnt, r = i - n * cnt, out = it.mt * 128 + rank * RS + r;
                float sum = 0.f;
                for (int s = 0; s < S; s++) sum += red[(s * NT + n) * RS + r];
                if (out < a.out) store(out, n, sum);
            }
            __syncwarp();
            if (lane < S) arrive_cluster(map_rank(redfree, lane));
        }
    }

    __syncthreads();
    if (warp == 2) {
        // no MMA may still be running when TMEM is released
        if (!mbar_wait_drain(done, 0) && lane == 0) report_status(a.status, kStatusWaitTimeout, 450);
        tc_fence_after();
        tmem_dealloc(tmem, Sh::TMEM_COLS);
    }
    if (S > 1) cluster_sync();               // no CTA leaves while another may write to its shared memory
}

// ------------------------------------------------------------- launchers --

// packed e2m1 rows: boxes of 128 rows x 128 codes, each 16 packed codes (8
// bytes) spread over 16 bytes of shared memory
bool encode_weights(CUtensorMap &m, const void *base, uint64_t cols, uint64_t rows) {
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {cols / 2};
    const cuuint32_t box[2] = {kStageCols, 128}, es[2] = {1, 1};
    return tensor_map_encoder()(&m, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 2, const_cast<void *>(base), dims, strides,
                                box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// e4m3 rows: boxes of box_rows rows x 128 columns
bool encode_states(CUtensorMap &m, const void *base, uint64_t cols, uint64_t rows, uint32_t box_rows) {
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {cols};
    const cuuint32_t box[2] = {kStageCols, box_rows}, es[2] = {1, 1};
    return tensor_map_encoder()(&m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, es,
                                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT>
cudaError_t launch_t(const Ctx &c, const ProdArgs &a, int y_bf16, int S, int clusters, const Maps &maps) {
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = ensure_smem((const void *)k_mx_product<NT>, Shape<NT>::SMEM, configured);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(clusters * S));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Shape<NT>::SMEM;
    cfg.stream = c.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)S;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = S > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k_mx_product<NT>, a, y_bf16, S, maps);
}

struct Plan {
    int NT, S, clusters;
};

// Rows of a unit and CTAs of a cluster.
Plan choose(const Ctx &c, const ProdArgs &a) {
    const int groups = a.n_groups < a.n_rows ? a.n_groups : a.n_rows;
    const int mean = (a.n_rows + groups - 1) / groups;       // rows of a group, were they even
    const int MT = (a.out + 127) / 128, KC = a.in / kStageCols;
    Plan best{};
    double least = 0;
    for (int NT : {32, 64, 128, 256}) {
        const long long items = (long long)groups * ((mean + NT - 1) / NT) * MT;
        for (int S : {1, 2, 3, 4, 8}) {
            if (S > KC || (S > 1 && NT == 256)) continue;
            long long clusters = c.num_sms / S;
            if (clusters > items) clusters = items;
            const long long waves = (items + clusters - 1) / clusters;
            const int n = mean < NT ? (mean + 15) & ~15 : NT;
            const double mma = 2.0 * (n < 64 ? 64 : n) + 60, mem = 8192.0 / (3400.0 / (double)(clusters * S) < 60 ? 3400.0 / (double)(clusters * S) : 60);
            const double t = (double)waves * (((KC + S - 1) / S) * (mma > mem ? mma : mem) + 1000.0 + (S > 1 ? 500 : 0));
            if (best.NT == 0 || t < least) {
                least = t;
                best = Plan{NT, S, (int)clusters};
            }
        }
    }
    return best;
}

}  // namespace

cudaError_t set_wait_polls_mxprod(uint32_t polls) { return set_wait_polls_here(polls); }

cudaError_t launch_mx_product(const Ctx &c, const ProdArgs &a, int y_bf16) {
    if (tensor_map_encoder() == nullptr) return cudaErrorNotSupported;
    const long long units = a.n_rows / 32 + (long long)a.n_groups;
    if (units * ((a.out + 127) / 128) > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    Maps maps;
    if (!encode_weights(maps.w, a.packed, a.in, (uint64_t)a.n_groups * a.out) ||
        !encode_states(maps.x64, a.codes, a.in, a.n_rows, 64) || !encode_states(maps.x16, a.codes, a.in, a.n_rows, 16))
        return cudaErrorInvalidValue;
    const Plan p = choose(c, a);
    if (p.NT == 32) return launch_t<32>(c, a, y_bf16, p.S, p.clusters, maps);
    if (p.NT == 64) return launch_t<64>(c, a, y_bf16, p.S, p.clusters, maps);
    if (p.NT == 128) return launch_t<128>(c, a, y_bf16, p.S, p.clusters, maps);
    return launch_t<256>(c, a, y_bf16, p.S, p.clusters, maps);
}

}  // namespace k3mx
