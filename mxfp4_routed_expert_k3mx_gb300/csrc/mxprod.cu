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
// tiles of 128 columns, KS tiles to a stage of the ring:
//   warp 0      copies: one TMA of the stage's weight tiles (128 rows x 128
//               codes each, 64 B a row in memory, spread to 128 B in shared
//               memory, 128-byte swizzle), one or a few of the unit's rows
//   warp 1      the weights' scales, four tiles (16 bytes a row) at a time:
//               loaded some groups ahead into registers, stored as the 32-line
//               sources of tcgen05.cp, one fence and one barrier per group; a
//               block of scale 255 gets scale 0 and its codes are zeroed once
//               the group before is multiplied and the tile landed, so it
//               adds exactly 0
//   warp 2      owns TMEM; one elected lane copies scales to TMEM and issues the
//               MMAs (the whole warp walks the loop, so that addresses and
//               descriptors stay in uniform registers: with one lane in the
//               loop, a tile took 1200 clocks to issue whatever its size)
//   warp 3      the rows' scales, as warp 1's
//   warps 4-11  epilogue: two warps to a lane quarter, half the rows each
// Every wait is bounded; one that gives up is reported on the device status
// word and every role leaves its loop (the epilogue after the exchanges that its
// cluster still has).
//
// Measured (calls repeated in a graph, in a burst; of a measured copy of 6.77 TB/s
// and library bf16 of 1957 TFLOP/s):
//   1 x 3584 x 7168 bf16 (rows, out, in)      7.4 us, 1.8 TB/s of weights and scales
//   1 x 12288 x 7168 bf16                    13.1 us, 3.6 TB/s; 1 x 19456 x 7168 14.4, 5.1
//   16 rows of 64 groups, 2048 x 3584 bf16   16.2 us, 3.6 TB/s
//   64 x 12288 x 7168 fp32                   15.9 us, 3.2 TB/s, 710 TFLOP/s
//   4096 x 12288 x 7168 bf16                 213 us, 3390 TFLOP/s; called without pause,
//                                            where the power limit holds the clock near
//                                            1.6 GHz, 256 us, 2820
//   16384 rows of 64 groups, 4096 x 3584     even groups 176 us, 2730 TFLOP/s; uneven ones
//                                            called without pause 229-235 us, 2050-2100
// Few rows: about 3 us pass before the first and after the last tile (launch,
// set-up, one latency, the MMA's, the epilogue), an exchange of a cluster takes
// one more, and a tile 0.18 us however few rows it has: the copy writes its
// 16 KB of spread codes into shared memory and the MMAs read them once, 256 of
// some 350 clocks (half the MMAs: 13.2 to 11.6 us for 1 x 12288 x 7168; no scale
// copies: 12.75; weights from L2: 12.5; no scale loads: no change).  HBM is
// only reached where every SM has many tiles.  Many rows: an SM takes a tile's 8 KB of weights and 32 KB of rows
// from L2 in about 0.33 us (64 bytes a clock), its MMAs take 0.27, and the
// accumulator changes hands once an item.  Without the MMAs the kernel takes
// 183 of 216 us, with half of them 191, with a sixteenth of the rows' copies
// 204, without stores 200.  Units of 192 rows with two accumulators and a
// fifth stage take 222 (0.28 us a tile, but a third more tiles).
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
constexpr int kAtom = 512;                 // scales of 128 rows and a tile: 32 lines of 16 bytes
constexpr int kThreads = 12 * 32, kEpi0 = 4, kEpiThreads = 8 * 32;

constexpr int kMaxSplit = 8;               // CTAs of a cluster: 1, 2, 4 or 8

// One exchange of a cluster: kExCols rows of the unit, every CTA's parts of
// this CTA's 128 / S outputs, [part][output][row] fp32.  Outputs lie kExPitch
// apart, so that 16-byte accesses of neighbouring outputs hit different banks.
constexpr int kExCols = 32, kExPitch = kExCols + 4;
constexpr int kExBytes = 128 * kExPitch * 4;

constexpr int kGroup = 4;                  // tiles whose scales travel together

template <int NT_> struct Shape {
    static constexpr int NT = NT_;                                   // rows of a unit
    static constexpr int ATOMS = NT == 256 ? 2 : 1;                  // the rows' scales of a tile
    // Tiles of a stage: two where a unit has few rows, so that what a stage
    // costs to copy, wait for and issue is spent half as often.
    static constexpr int KS = NT <= 64 ? 2 : 1;
    static constexpr int STAGE = KS * (kWTile + NT * 128);
    static constexpr int SA = NT == 64 ? 3 : NT == 128 ? 6 : 4;      // stages
    static constexpr int SG = 3;                                     // scale groups
    static constexpr int GROUP = kGroup * (1 + ATOMS) * kAtom;       // weights' atoms, then the rows'
    static constexpr int NBUF = NT == 256 ? 1 : 2;                   // accumulators
    static constexpr bool SPLIT = NT <= 64;                          // clusters of more than one CTA
    static constexpr int RED = SPLIT ? 2 * kExBytes : 0;
    static constexpr int TABLES = 2 * (K3MX_MX_MAX_GROUPS + 8) * 4;
    static constexpr int SMEM = 1024 + 1024 + SA * STAGE + SG * GROUP + RED + TABLES;
    // TMEM columns: accumulators, then every tile's scales (addresses the MMA
    // reads scales from are multiples of four columns)
    static constexpr int SF_COL = NBUF * NT, SF_STEP = 4 + 4 * ATOMS;
    static constexpr int TMEM_COLS = 512;
    static_assert(STAGE % 1024 == 0 && SMEM <= 227 * 1024, "shared memory");
    static_assert(SF_COL + SG * kGroup * SF_STEP <= TMEM_COLS, "TMEM");
    static_assert(SF_COL % 4 == 0 && SF_STEP % 4 == 0, "addresses the MMA reads scales from");
    static_assert(SA * KS >= kGroup, "a group's weight tiles fit the ring together: its dropped blocks are zeroed with "
                                     "the group before consumed and none of its own");
};

// weights, and the rows in boxes of 16, 32 and 64
struct Maps {
    CUtensorMap w, x16, x32, x64;
};

struct Hdr {
    uint64_t tfull[8], empty[8], gfull[4], gempty[4], accf[2], acce[2], done, exfull[2];
    uint32_t tmem;
    int abort;
    int part[16];
};

struct Item {
    int g, mt, off, ntok;
};

__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// 16 bytes into another CTA's shared memory; the bytes count on its barrier
__device__ __forceinline__ void st_async4(uint32_t addr, float a, float b, float c, float d, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
                 "f"(a), "f"(b), "f"(c), "f"(d), "r"(bar)
                 : "memory");
}
// An exchange's wait.  Its limit is not the one that callers set: after another
// wait gave up the cluster's CTAs still go through every exchange in step (the
// parts are worthless and y is not written), so that each barrier is armed once a
// phase and no part is under way when a CTA leaves.  Twice the limit of the
// others, which a peer may wait out first.
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity) {
    for (uint32_t i = 0; i < 2 * kWaitLimit; i++) {
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

// 16 TMEM columns of this warp's lanes; the values are there after tmem_ld_wait
__device__ __forceinline__ void tmem_ld16f(uint32_t taddr, float *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr));
}
// tmem_ld_wait for the values `v`.  Their uses are register arithmetic, which a
// wait that does not name them would not hold back: it hands them on.
template <int N>
__device__ __forceinline__ void tmem_ld_wait_for(float (&v)[N]) {
    static_assert(N % 16 == 0, "whole loads");
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < N; j += 16)
        asm volatile(""
                     : "+f"(v[j]), "+f"(v[j + 1]), "+f"(v[j + 2]), "+f"(v[j + 3]), "+f"(v[j + 4]), "+f"(v[j + 5]),
                       "+f"(v[j + 6]), "+f"(v[j + 7]), "+f"(v[j + 8]), "+f"(v[j + 9]), "+f"(v[j + 10]), "+f"(v[j + 11]),
                       "+f"(v[j + 12]), "+f"(v[j + 13]), "+f"(v[j + 14]), "+f"(v[j + 15]));
}
// one lane of the (converged) warp
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void prefetch_l2(const void *p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}
// whether the phase has completed, without waiting
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// a place in a ring of N slots and the parity of its current use
template <int N> struct Slot {
    uint32_t i = 0, ph = 0;
    __device__ __forceinline__ void next() {
        if (++i == N) {
            i = 0;
            ph ^= 1;
        }
    }
};

// Loads that happen or leave their registers alone (a predicate and no branch).
// Not through the read-only path, as no load of this kernel's inputs: they may be
// the kernel's before, which this one overlaps until its dependency wait, and
// that path is for what nothing writes while a kernel lasts.
__device__ __forceinline__ void ldg_if(uint32_t &v, const uint8_t *p, bool live) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t@q ld.global.u32 %0, [%1];\n\t}" : "+r"(v) : "l"(p), "r"((uint32_t)live));
}
__device__ __forceinline__ void ldg2_if(uint32_t &v, uint32_t &w, const uint8_t *p, bool live) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %3, 0;\n\t@q ld.global.v2.u32 {%0, %1}, [%2];\n\t}"
                 : "+r"(v), "+r"(w) : "l"(p), "r"((uint32_t)live));
}

// Scale words of a stream of items, kcs tiles (words of a row) each, in
// groups of four tiles: lane l loads the words of rows l, l + 32, ... (R of
// them), W bytes at a time, a group ahead of its use (two or three ahead cost
// more, in code to fetch and in loads before the first use, than they hid:
// 1 x 3584 x 7168 8.0 us, 8.5 and 10.0).  begin(i, base) gives item i's first
// words of the lane's R rows (rows that do not exist repeat one that does);
// use(n, i, c, words) takes the n-th group: tiles c .. c + 3 of item i (words
// past the item's last tile are any that were loaded before).  A load has one
// width and no alternative, so that it is not waited for before its use: with
// a branch between widths, the moves at its end waited for each.
template <int R, int W, typename Begin, typename Use>
__device__ __forceinline__ void scale_groups_w(int n_items, int kcs, Begin begin, Use use) {
    uint32_t q[R][kGroup];
    const uint8_t *base[R];
    auto load = [&](int i, int c) {
        if (c == 0) begin(i, base);
#pragma unroll
        for (int r = 0; r < R; r++) {
            const uint8_t *at = base[r] + 4 * c;
            if (W == 16) {
                const uint4 v = *reinterpret_cast<const uint4 *>(at);
                q[r][0] = v.x, q[r][1] = v.y, q[r][2] = v.z, q[r][3] = v.w;
            } else if (W == 8) {
                const uint2 v = *reinterpret_cast<const uint2 *>(at);
                q[r][0] = v.x, q[r][1] = v.y;
                ldg2_if(q[r][2], q[r][3], at + 8, c + 2 < kcs);
            } else {
#pragma unroll
                for (int j = 0; j < kGroup; j++) ldg_if(q[r][j], at + 4 * j, c + j < kcs);
            }
        }
    };
#pragma unroll
    for (int r = 0; r < R; r++)
#pragma unroll
        for (int j = 0; j < kGroup; j++) q[r][j] = 0u;
    int n = 0, i = 0, c = 0;
    if (n_items > 0) load(0, 0);
#pragma unroll 1
    while (i < n_items) {
        if (!use(n, i, c, q)) return;
        n++;
        c += kGroup;
        if (c >= kcs) {
            c = 0;
            i++;
        }
        if (i < n_items) load(i, c);
    }
}
// W by what the first words' addresses (`bits`: their low bits) and the
// items' length allow
template <int R, typename Begin, typename Use>
__device__ __forceinline__ void scale_groups(int n_items, int kcs, uint32_t bits, Begin begin, Use use) {
    if ((bits & 15) == 0 && kcs % 4 == 0) scale_groups_w<R, 16>(n_items, kcs, begin, use);
    else if ((bits & 7) == 0 && kcs % 2 == 0) scale_groups_w<R, 8>(n_items, kcs, begin, use);
    else scale_groups_w<R, 4>(n_items, kcs, begin, use);
}

// Every role fetches its own code when a call starts, and beside other kernels
// it is rarely still in an SM's instruction cache: a one-row and a 64-row
// product in turn take 19.2 us where each repeated takes 18.5, 22.4 with the
// three functions below inlined and the loops unrolled (108 to 151 KB of code
// a kernel, 69 to 115 so).  So what few calls reach is out of line: later
// items, a wait's polls after the first, dropped blocks.

// Item `it`: groups in order, in a group tile by tile, a tile's units together
// (they share its weights in L2)
__device__ __noinline__ Item item_of(const int *ustart, const int *goff, uint32_t it, uint32_t MT, int n_groups) {
    const uint32_t q = it / MT;
    int lo = 0, hi = n_groups - 1;                    // last group with ustart <= q
#pragma unroll 1
    while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (ustart[m] <= (int)q) lo = m;
        else hi = m - 1;
    }
    const uint32_t u0 = ustart[lo], ug = ustart[lo + 1] - u0, l = it - u0 * MT;
    const uint32_t mt = l / ug, u = l - mt * ug;
    // the group's rows in ug units, the first ones a row longer
    const uint32_t cnt = goff[lo + 1] - goff[lo], each = cnt / ug, more = cnt - each * ug;
    return Item{lo, (int)mt, goff[lo] + (int)(each * u + min(u, more)), (int)(each + (u < more ? 1 : 0))};
}

__device__ __noinline__ bool wait_more(uint32_t bar, uint32_t parity) {
    const uint32_t lim = wait_polls();
    for (uint32_t i = 1; i < lim; i++)
        if (mbar_try_wait(bar, parity)) return true;
    return false;
}
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity) {
    return mbar_try_wait(bar, parity) || wait_more(bar, parity);
}

// The blocks of scale 255 of a group of `n` tiles, v[4][kGroup] the scale words
// of this lane's rows: codes zeroed once each tile has landed, scales too.
// False if a wait gave up.
// First the MMAs of the group before are waited for.  The scales' warp runs up
// to SG groups ahead of them, which is further than the ring is long, and a
// barrier whose use before the one meant is still open has the parity that is
// waited for: the zeros went into the slot's earlier tile, where a group with a
// dropped block followed groups without one.  With the group before consumed,
// every stage before this group's has landed, the next use of each of its slots
// is its own, and (the static_assert above) the group's own stages fit the
// ring; nothing of the group before waits for this one.
struct DropAt {
    uint32_t before, parity;            // the barrier of the MMAs of the group before
    uint32_t tfull0, ring, stage;
    int KS, SA, first, c, n;            // the item's first stage, the group's first tile in it
};
__device__ __noinline__ bool drop_blocks(const DropAt d, uint32_t *v, int lane) {
    if (!mbar_wait(d.before, d.parity)) return false;
#pragma unroll 1
    for (int j = 0; j < kGroup && j < d.n; j++) {
        const int f = d.first + (d.c + j) / d.KS, s = f % d.SA;
        if (!mbar_wait(d.tfull0 + 8 * s, (f / d.SA) & 1)) return false;
#pragma unroll 1
        for (int r = 0; r < 4; r++) {
            zero_nan_groups_x128(d.ring + s * d.stage + (d.c + j) % d.KS * kWTile, lane + 32 * r, v[r * kGroup + j]);
            v[r * kGroup + j] = drop_nan_scales(v[r * kGroup + j]);
        }
    }
    return true;
}

template <int NT>
__global__ void __launch_bounds__(kThreads, 1)
k_mx_product(const ProdArgs a, const int y_bf16, const int S, const int seg, const __grid_constant__ Maps maps) {
    using Sh = Shape<NT>;
    constexpr int SA = Sh::SA, SG = Sh::SG, NBUF = Sh::NBUF, KS = Sh::KS;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Hdr *hd = reinterpret_cast<Hdr *>(smem);
    const uint32_t ring = smem_addr(smem) + 1024;
    const uint32_t sgroups = ring + SA * Sh::STAGE;
    uint8_t *red = smem + 1024 + SA * Sh::STAGE + SG * Sh::GROUP;
    int *ustart = reinterpret_cast<int *>(smem + Sh::SMEM - 1024 - Sh::TABLES);      // first unit of each group
    int *goff = ustart + K3MX_MX_MAX_GROUPS + 8;                                     // first row of each group
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t tfull0 = smem_addr(hd->tfull), empty0 = smem_addr(hd->empty);
    const uint32_t gfull0 = smem_addr(hd->gfull), gempty0 = smem_addr(hd->gempty);
    const uint32_t accf0 = smem_addr(hd->accf), acce0 = smem_addr(hd->acce), done = smem_addr(&hd->done);
    const uint32_t exfull0 = smem_addr(hd->exfull);
    const int rank = S > 1 ? (int)(blockIdx.x % S) : 0;       // %cluster_ctarank of a 1-D cluster

    if (tid == 0) {
        for (int i = 0; i < SA; i++) {
            mbar_init(tfull0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, 1);
        }
        for (int i = 0; i < SG; i++) {
            mbar_init(gfull0 + 8 * i, 64);
            mbar_init(gempty0 + 8 * i, 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(accf0 + 8 * i, 1);
            mbar_init(acce0 + 8 * i, kEpiThreads);
        }
        mbar_init(done, 1);
        mbar_init(exfull0, 1);
        mbar_init(exfull0 + 8, 1);
        hd->abort = 0;
        fence_mbar_init();
    }
    if (warp == 2) tmem_alloc(smem_addr(&hd->tmem), Sh::TMEM_COLS);
    if (tid < 2)
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<const char *>(&maps) + 128 * tid) : "memory");
    const int MT = (a.out + 127) / 128, KC = a.in / kStageCols, G = a.in / 32;
    // this CTA's tiles of every item, whole stages of them
    const int KF = (KC + KS - 1) / KS, f0 = KF * rank / S, f1 = KF * (rank + 1) / S;
    const int c0 = f0 * KS, kcs = min(f1 * KS, KC) - c0, fts = f1 - f0;
    const int first = blockIdx.x / S, step = gridDim.x / S;
    if (a.offsets == nullptr) {
        // One group of all rows: everything up to the copies is ready before
        // the kernel before this one ends, and the first weights are on their
        // way into L2 (they may be that kernel's output: L2 is where it writes).
        if (tid == 0) {
            ustart[0] = goff[0] = 0;
            ustart[1] = (a.n_rows + NT - 1) / NT;
            goff[1] = a.n_rows;
        }
        const int mt = first / ((a.n_rows + NT - 1) / NT), row = mt * 128 + (tid & 127);
        if (row < a.out) {
            // the first SA stages' codes (64 bytes a tile) and their scales
            const uint8_t *w = a.packed + (size_t)row * (a.in / 2);
            const int t = (tid >> 7) * 2;                             // three lines of 128 bytes
            if (t < min(kcs, SA * KS)) prefetch_l2(w + (size_t)(c0 + t) * (kStageCols / 2));
            if (tid < 128) prefetch_l2(a.wscales + (size_t)row * G + 4 * c0);
        }
    } else {
        pdl_wait();
        // units of every group (0 for one whose offsets are unusable)
        constexpr int GPT = (K3MX_MX_MAX_GROUPS + kThreads - 1) / kThreads;
        int nu[GPT], mine = 0;
#pragma unroll
        for (int k = 0; k < GPT; k++) {
            const int g = tid * GPT + k;
            nu[k] = 0;
            if (g < a.n_groups) {
                const int lo = a.offsets[g], hi = a.offsets[g + 1];
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
        int before = lane < warp ? hd->part[lane] : 0;                 // (12 warps)
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
        int at = __shfl_sync(0xffffffffu, before, 0) + incl - mine;
#pragma unroll
        for (int k = 0; k < GPT; k++) {
            const int g = tid * GPT + k;
            if (g < a.n_groups) ustart[g] = at;
            at += nu[k];
            if (g == a.n_groups - 1) ustart[a.n_groups] = at;
        }
    }
    tc_fence_before();
    if (S > 1) cluster_sync();               // also: every CTA's barriers are initialised
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, hd->tmem, 0);
    volatile int *abort_flag = &hd->abort;

    const int items = ustart[a.n_groups] * MT;
    const int n_items = items > first ? (items - first + step - 1) / step : 0;
    const int groups = (kcs + kGroup - 1) / kGroup, n_seg = (groups + seg - 1) / seg;   // accumulations of an item

    auto item_at = [&](int k) { return item_of(ustart, goff, first + k * step, MT, a.n_groups); };
    // The first item, which is the only one of most short calls, is worked out
    // here and not by every role: the code of the rest is then never fetched.
    const Item item0 = n_items > 0 ? item_at(0) : Item{};
    auto next_item = [&](int k) { return k == 0 ? item0 : item_at(k); };
    if (a.offsets == nullptr) pdl_wait();
    pdl_launch_dependents();
    auto fail = [&](int detail) {
        report_status(a.status, kStatusWaitTimeout, detail);
        *abort_flag = 1;
    };
    uint32_t late = 0;                        // exchanges given up (the epilogue's)

    if (warp == 0) {
        // ---------------------------------------------------- copies --
        const bool leader = elect_one();
        const uint64_t wpol = l2_evict_first_policy(), xpol = l2_evict_last_policy();
        Slot<SA> sl;
        int issued = 0;
        bool alive = true;                    // as the MMA warp's
#pragma unroll 1
        for (int k = 0; k < n_items; k++) {
            const Item it = next_item(k);
            const int rows = (it.ntok + 15) & ~15, wy = it.g * a.out + it.mt * 128;
            const int box = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;          // of the KS = 2 forms
            const CUtensorMap *xmap = rows <= 16 ? &maps.x16 : rows <= 32 ? &maps.x32 : &maps.x64;
#pragma unroll 1
            for (int c = c0; c < c0 + kcs; c += KS, sl.next()) {
                const uint32_t bar = tfull0 + 8 * sl.i, st = ring + sl.i * Sh::STAGE, xt = st + KS * kWTile;
                alive = alive && wait_for(empty0 + 8 * sl.i, sl.ph ^ 1);
                if (leader && alive) {
                    if (KS == 2) {
                        mbar_arrive_expect_tx(bar, 2 * (kWTileTx + box * 128));
                        tma_3d(st, &maps.w, 0, wy, c, bar, wpol);
                        tma_3d(xt, xmap, 0, it.off, c, bar, xpol);
                    } else {
                        mbar_arrive_expect_tx(bar, kWTileTx + rows * 128);
                        tma_3d(st, &maps.w, 0, wy, c, bar, wpol);
                        int r = 0;
#pragma unroll 1
                        for (; r + 64 <= rows; r += 64) tma_3d(xt + r * 128, &maps.x64, 0, it.off + r, c, bar, xpol);
#pragma unroll 1
                        for (; r < rows; r += 16) tma_3d(xt + r * 128, &maps.x16, 0, it.off + r, c, bar, xpol);
                    }
                    issued++;
                }
                __syncwarp();
            }
            if (*abort_flag) alive = false;
        }
        if (leader && !alive) fail(400);
        // copies still in flight (after a wait gave up) land before the CTA leaves
        if (leader && !drain_ring(tfull0, SA, issued)) report_status(a.status, kStatusWaitTimeout, 401);
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------- the tile's scales --
        auto begin = [&](int k, const uint8_t *(&base)[4]) {
            const Item it = next_item(k);
#pragma unroll
            for (int r = 0; r < 4; r++)
                base[r] = a.wscales + ((size_t)it.g * a.out + min(it.mt * 128 + lane + 32 * r, a.out - 1)) * G + 4 * c0;
        };
        auto use = [&](int n, int i, int c, const uint32_t (&w)[4][kGroup]) {
            const int gs = n % SG;
            // (lanes poll for themselves: they leave together, for the votes below)
            if (!__all_sync(0xffffffffu, !*abort_flag && wait_for(gempty0 + 8 * gs, ((n / SG) & 1) ^ 1))) {
                if (lane == 0) fail(410);
                return false;
            }
            uint32_t v[4][kGroup], nan = 0;
#pragma unroll
            for (int r = 0; r < 4; r++)
#pragma unroll
                for (int j = 0; j < kGroup; j++) {
                    v[r][j] = w[r][j];
                    nan |= (~v[r][j] - 0x01010101u) & v[r][j] & 0x80808080u;      // a byte of ~v is 0
                }
            if (__any_sync(0xffffffffu, nan != 0)) {
                // (before the first group: the last slot's barrier, free from the start)
                const int b = n + SG - 1;
                const DropAt at{gempty0 + 8 * (b % SG), (uint32_t)(((b / SG) & 1) ^ 1), tfull0, ring, Sh::STAGE,
                                KS,                     SA,                             i * fts, c,  kcs - c};
                uint32_t u[4 * kGroup];
#pragma unroll
                for (int t = 0; t < 4 * kGroup; t++) u[t] = v[t / kGroup][t % kGroup];
                if (!__all_sync(0xffffffffu, drop_blocks(at, u, lane))) {
                    if (lane == 0) fail(411);
                    return false;
                }
#pragma unroll
                for (int t = 0; t < 4 * kGroup; t++) v[t / kGroup][t % kGroup] = u[t];
            }
#pragma unroll
            for (int j = 0; j < kGroup; j++)
                sts128(sgroups + gs * Sh::GROUP + j * kAtom + 16 * lane, v[0][j], v[1][j], v[2][j], v[3][j]);
            fence_async_smem();
            mbar_arrive(gfull0 + 8 * gs);
            return true;
        };
        scale_groups<4>(n_items, kcs, (uint32_t)reinterpret_cast<uintptr_t>(a.wscales) | G | 4 * c0, begin, use);
    } else if (warp == 3) {
        // -------------------------------------------- the rows' scales --
        constexpr int R = NT / 32;
        auto begin = [&](int k, const uint8_t *(&base)[R]) {
            const Item it = next_item(k);
#pragma unroll
            for (int r = 0; r < R; r++)
                base[r] = a.scales + ((size_t)it.off + min(lane + 32 * r, it.ntok - 1)) * G + 4 * c0;
        };
        auto use = [&](int n, int, int, const uint32_t (&w)[R][kGroup]) {
            const int gs = n % SG;
            if (!__all_sync(0xffffffffu, !*abort_flag && wait_for(gempty0 + 8 * gs, ((n / SG) & 1) ^ 1))) {
                if (lane == 0) fail(420);
                return false;
            }
            const uint32_t at = sgroups + gs * Sh::GROUP + kGroup * kAtom + 16 * lane;
            auto word = [&](int r, int j) { return r < R ? w[r < R ? r : 0][j] : 0u; };
#pragma unroll
            for (int j = 0; j < kGroup; j++)
#pragma unroll
                for (int r = 0; r < R; r += 4)
                    sts128(at + (j * Sh::ATOMS + (r >> 2)) * kAtom, w[r][j], word(r + 1, j), word(r + 2, j), word(r + 3, j));
            fence_async_smem();
            mbar_arrive(gfull0 + 8 * gs);
            return true;
        };
        scale_groups<R>(n_items, kcs, (uint32_t)reinterpret_cast<uintptr_t>(a.scales) | G | 4 * c0,
                                                           begin, use);
    } else if (warp == 2) {
        // ------------------------------------------------ MMA issuer --
        const bool leader = elect_one();
        Slot<SA> sl;
        Slot<SG> sg;
        Slot<NBUF> sb;
        // `alive` turns false when a wait gave up.  The loops run on to their
        // ends all the same (doing nothing): an exit on a loaded value would
        // take every address in them out of the uniform registers.
        bool alive = true, ready = false;              // ready: the next stage's tiles have landed
        const uint32_t tile_hi = (uint32_t)(umma_desc_sw128(0) >> 32), tile_lo = (uint32_t)umma_desc_sw128(0);
        const uint32_t atom_hi = (uint32_t)(desc_atom(0, 128) >> 32), atom_lo = (uint32_t)desc_atom(0, 128);
        auto atom = [&](uint32_t addr16) { return (uint64_t)atom_hi << 32 | (atom_lo + addr16); };
        auto desc = [&](uint32_t addr16) { return (uint64_t)tile_hi << 32 | (tile_lo + addr16); };
#pragma unroll 1
        for (int k = 0; k < n_items; k++) {
            const int rows = __shfl_sync(0xffffffffu, (next_item(k).ntok + 15) & ~15, 0);
            const uint32_t xstep = KS == 1 ? 0 : rows <= 16 ? 16 * 128 : rows <= 32 ? 32 * 128 : 64 * 128;
            uint32_t id[4];
#pragma unroll
            for (int ks = 0; ks < 4; ks++) id[ks] = idesc_e2m1_e4m3(rows, ks);
            int in_seg = 0;
#pragma unroll 1
            for (int c = 0; c < kcs; c += kGroup) {
                if (in_seg == 0) alive = alive && wait_for(acce0 + 8 * sb.i, sb.ph ^ 1);
                alive = alive && wait_for(gfull0 + 8 * sg.i, sg.ph);
                const bool last = c + kGroup >= kcs, seg_end = last || in_seg + 1 == seg;
                const uint32_t d = tmem + sb.i * NT;
                const uint32_t sf = tmem + Sh::SF_COL + sg.i * (kGroup * Sh::SF_STEP);
                const uint32_t src = (sgroups + sg.i * Sh::GROUP) >> 4;
#pragma unroll
                for (int j = 0; j < kGroup; j += KS) {
                    if (c + j < kcs) {
                        alive = alive && (ready || wait_for(tfull0 + 8 * sl.i, sl.ph));
                        const uint32_t slot = sl.i;
                        sl.next();
                        ready = mbar_test(tfull0 + 8 * sl.i, sl.ph);
                        const uint32_t wt = (ring + slot * Sh::STAGE) >> 4;
                        tc_fence_after();
                        if (leader && alive) {
#pragma unroll
                            for (int t = 0; t < KS; t++)
                                if (t == 0 || c + j + t < kcs) {
                                    const uint32_t sfa = sf + (j + t) * Sh::SF_STEP, sfb = sfa + 4;
                                    tmem_cp_atom(sfa, atom(src + (j + t) * (kAtom >> 4)));
                                    tmem_cp_atom(sfb, atom(src + (kGroup + (j + t) * Sh::ATOMS) * (kAtom >> 4)));
                                    if (Sh::ATOMS == 2 && rows > 128)
                                        tmem_cp_atom(sfb + 4, atom(src + (kGroup + (j + t) * Sh::ATOMS + 1) * (kAtom >> 4)));
                                    const uint32_t ad = wt + t * (kWTile >> 4), bd = wt + ((KS * kWTile + t * xstep) >> 4);
#pragma unroll
                                    for (int ks = 0; ks < 4; ks++)
                                        mma_mxf8f6f4(d, desc(ad + 2 * ks), desc(bd + 2 * ks), id[ks], sfa, sfb,
                                                     (in_seg | j | t | ks) != 0 ? 1u : 0u);
                                }
                            umma_commit(empty0 + 8 * slot);
                        }
                        __syncwarp();
                    }
                }
                if (leader && alive) {
                    umma_commit(gempty0 + 8 * sg.i);
                    if (seg_end) umma_commit(accf0 + 8 * sb.i);
                }
                __syncwarp();
                sg.next();
                in_seg++;
                if (seg_end) {
                    in_seg = 0;
                    sb.next();
                }
            }
            if (*abort_flag) alive = false;
        }
        if (leader && !alive) fail(430);
        if (leader) umma_commit(done);
        __syncwarp();
    } else {
        // -------------------------------------------------- epilogue --
        constexpr int HC = NT / 2;                            // rows of the unit to a warp
        const int q4 = warp & 3, half = (warp - kEpi0) >> 2;
        const int o = 32 * q4 + lane;                         // output within the tile
        const uint32_t quarter = (uint32_t)(32 * q4) << 16;
        const int RS = 128 / S;                               // outputs this CTA adds
        Slot<NBUF> sb;
        Slot<2> ex;
        // `alive` as in the MMA warp: the loops run to their ends, so the named
        // barrier below always has all its warps.  `missed` counts the exchanges
        // from the first whose own wait gave up.  From then on nothing is sent
        // (the peers' waits give up in turn), and only the one after it is still
        // armed: its barrier's phase before was seen complete, a later one's was
        // not.  Peers may have sent to these two, not to any later one, for which
        // they would have to have this CTA's parts of the second.
        bool alive = true;
        uint32_t missed = 0;
#pragma unroll 1
        for (int k = 0; k < n_items; k++) {
            const Item it = next_item(k);
            const int n0 = half * HC, n1 = min(it.ntok, n0 + HC);
            // The item's accumulations, added in fp32.  The first is loaded
            // whole (rows past the unit's hold whatever was there) and waited
            // for once.
            float v[HC];
            alive = alive && wait_for(accf0 + 8 * sb.i, sb.ph);
            __syncwarp();                       // (each lane polls for itself; the loads are the whole warp's)
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < HC; j += 16) tmem_ld16f(tmem + quarter + sb.i * NT + n0 + j, v + j);
            tmem_ld_wait_for(v);
            tc_fence_before();
            mbar_arrive(acce0 + 8 * sb.i);
            sb.next();
#pragma unroll 1
            for (int sg = 1; sg < n_seg; sg++, sb.next()) {
                alive = alive && wait_for(accf0 + 8 * sb.i, sb.ph);
                __syncwarp();
                tc_fence_after();
#pragma unroll
                for (int j = 0; j < HC; j += 16)
                    if (n0 + j < n1) {
                        float u[16];
                        tmem_ld16f(tmem + quarter + sb.i * NT + n0 + j, u);
                        tmem_ld_wait_for(u);
#pragma unroll
                        for (int i = 0; i < 16; i++) v[j + i] += u[i];
                    }
                tc_fence_before();
                mbar_arrive(acce0 + 8 * sb.i);
            }
            if (!Sh::SPLIT || S == 1) {
                const int out = it.mt * 128 + o;
                const bool ok = out < a.out && alive;
                if (y_bf16 && (a.out & 1) == 0) {
                    // two outputs of a row to a store: the lanes of a pair swap, the
                    // even one stores the first of two rows, the odd one the second
                    // (grouped prefill 221 to 213 us)
                    const int odd = lane & 1;
                    uint32_t *y = reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(a.y) +
                                                               (size_t)(it.off + n0 + odd) * a.out + (out - odd));
#pragma unroll
                    for (int j = 0; j < HC; j += 2, y += a.out) {
                        const float got = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
                        const __nv_bfloat162 h = odd ? __floats2bfloat162_rn(got, v[j + 1]) : __floats2bfloat162_rn(v[j], got);
                        if (ok && n0 + j + odd < n1) *y = *reinterpret_cast<const uint32_t *>(&h);
                    }
                } else if (ok && y_bf16) {
                    __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(a.y) + (size_t)(it.off + n0) * a.out + out;
#pragma unroll
                    for (int j = 0; j < HC; j++, y += a.out)
                        if (n0 + j < n1) *y = __float2bfloat16_rn(v[j]);
                } else if (ok) {
                    float *y = static_cast<float *>(a.y) + (size_t)(it.off + n0) * a.out + out;
#pragma unroll
                    for (int j = 0; j < HC; j++, y += a.out)
                        if (n0 + j < n1) *y = v[j];
                }
            } else {
                // Exchanges of kExCols rows.  Every CTA sends its parts of all
                // outputs to the CTAs that add them.  A buffer is used again two
                // exchanges later: by then this CTA has all parts of the exchange
                // between, and no CTA sends those before all its warps (the
                // named barrier) are done with the one before.
                const int own = o / RS;
#pragma unroll
                for (int x = 0; x < NT / kExCols; x++) {
                    if (x * kExCols >= it.ntok) break;
                    const int cols = (min(kExCols, it.ntok - x * kExCols) + 3) & ~3;
                    const uint32_t buf = smem_addr(red) + ex.i * kExBytes, bar = exfull0 + 8 * ex.i;
                    __syncwarp();
                    named_sync(1, kEpiThreads);
                    if (warp == kEpi0 && lane == 0 && missed < 2) mbar_arrive_expect_tx(bar, S * RS * cols * 16 / 4);
                    const uint32_t to = map_rank(buf + (rank * RS + o - own * RS) * (kExPitch * 4), own), tobar = map_rank(bar, own);
                    constexpr int PER = HC < kExCols ? HC : kExCols;             // this warp's rows of an exchange
                    if (HC < kExCols || x / (HC / PER) == half) {
#pragma unroll
                        for (int j = 0; j < PER; j += 4) {
                            const int jj = HC < kExCols ? j : (x % (HC / PER)) * PER + j;      // in v
                            const int n = HC < kExCols ? n0 + j : j;                           // of the exchange
                            if (n < cols && missed == 0) st_async4(to + n * 4, v[jj], v[jj + 1], v[jj + 2], v[jj + 3], tobar);
                        }
                    }
                    if (missed != 0 || !wait_cluster(bar, ex.ph)) {
                        if (missed < 2) late |= (2u | ex.ph) << (2 * ex.i);
                        missed++;
                        alive = false;
                    }
                    __syncwarp();
                    const float *src = reinterpret_cast<const float *>(red + ex.i * kExBytes);
#pragma unroll 1
                    for (int i = tid - kEpi0 * 32; i < RS * (cols / 4); i += kEpiThreads) {
                        const int n = i / RS * 4, r = i % RS, out = it.mt * 128 + rank * RS + r;
                        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
                        for (int s = 0; s < S; s++) {
                            const float4 q = *reinterpret_cast<const float4 *>(src + (s * RS + r) * kExPitch + n);
                            sum.x += q.x, sum.y += q.y, sum.z += q.z, sum.w += q.w;
                        }
                        const float f[4] = {sum.x, sum.y, sum.z, sum.w};
                        const int left = it.ntok - x * kExCols - n;
                        if (out < a.out && alive) {
                            const size_t at = (size_t)(it.off + x * kExCols + n) * a.out + out;
                            if (y_bf16) {
#pragma unroll
                                for (int j = 0; j < 4; j++)
                                    if (j < left) static_cast<__nv_bfloat16 *>(a.y)[at + (size_t)j * a.out] = __float2bfloat16_rn(f[j]);
                            } else {
#pragma unroll
                                for (int j = 0; j < 4; j++)
                                    if (j < left) static_cast<float *>(a.y)[at + (size_t)j * a.out] = f[j];
                            }
                        }
                    }
                    ex.next();
                }
            }
            if (*abort_flag) alive = false;
        }
        if (__any_sync(0xffffffffu, !alive) && lane == 0) fail(440);
    }

    __syncthreads();
    if (warp == 2) {
        // no MMA may still be running when TMEM is released
        if (!mbar_wait_drain(done, 0) && lane == 0) report_status(a.status, kStatusWaitTimeout, 450);
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, Sh::TMEM_COLS);
    }
    if (S > 1) {
        cluster_sync();                      // no CTA leaves while another may write to its shared memory
        // nor while parts are under way to it: all are sent by now, and those of
        // an exchange that was given up (armed by this thread) land first
        if (tid == kEpi0 * 32)
            for (int i = 0; i < 2; i++)
                if ((late >> (2 * i) & 2u) && !mbar_wait_drain(exfull0 + 8 * i, late >> (2 * i) & 1u))
                    report_status(a.status, kStatusWaitTimeout, 451);
    }
}

// ------------------------------------------------------------- launchers --

// Matrices as [tile of 128 columns][row][column]: one copy brings a box of
// rows of ks neighbouring tiles, each a K-major operand of 128-byte rows.
bool encode(CUtensorMap &m, CUtensorMapDataType type, const void *base, int in, uint64_t rows, uint64_t pitch,
            uint64_t tile, uint32_t box_rows, uint32_t ks) {
    const cuuint64_t dims[3] = {kStageCols, rows, (cuuint64_t)(in / kStageCols)}, strides[2] = {pitch, tile};
    const cuuint32_t box[3] = {kStageCols, box_rows, ks}, es[3] = {1, 1, 1};
    return tensor_map_encoder()(&m, type, 3, const_cast<void *>(base), dims, strides, box, es,
                                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// packed e2m1 rows, each 16 packed codes (8 bytes) spread over 16 bytes of
// shared memory
bool encode_weights(CUtensorMap &m, const ProdArgs &a, int ks) {
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, a.packed, a.in, (uint64_t)a.n_groups * a.out, a.in / 2,
                  kStageCols / 2, 128, ks);
}
// e4m3 rows
bool encode_states(CUtensorMap &m, const ProdArgs &a, int box_rows, int ks) {
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.codes, a.in, a.n_rows, a.in, kStageCols, box_rows, ks);
}

// Scale groups (512 columns) of one accumulation, by the result's type.  Of an
// MMA's 32 products and the sum so far the tensor cores keep what lies within 2^-25
// of the largest one's power of two, of their sum fp32's 24 bits, both cut
// towards zero (measured: 1 + 2^-26 + ... stays 1 however many follow), so that
// where a large term comes first an accumulation of n columns loses up to
// n 2^-25 + n / 32 (2^-23 + 2^-25) of sum |x w|: 3.6e-5 for 1024 columns, 2.8e-4
// for 8192, 2.3e-3 for 65536.  fp32 results are added in fp32 from accumulations
// of 1024 (random codes, in = 7168: 2.1e-7 off, 2-norm; fp32 sums 3.0e-7, one
// accumulation of all 1.5e-6).  bf16 ones, whose rounding is 2e-3, from 8192: no
// more hand-overs of the accumulator up to that width.
constexpr int kSegF32 = 2, kSegBf16 = 16;

template <int NT>
cudaError_t launch_t(const Ctx &c, const ProdArgs &a, int y_bf16, int S, int clusters) {
    constexpr int KS = Shape<NT>::KS;
    Maps maps;
    if (!encode_weights(maps.w, a, KS) || !encode_states(maps.x16, a, 16, KS) ||
        (NT <= 64 && !encode_states(maps.x32, a, 32, KS)) || (NT >= 64 && !encode_states(maps.x64, a, 64, KS)))
        return cudaErrorInvalidValue;
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
    return cudaLaunchKernelEx(&cfg, k_mx_product<NT>, a, y_bf16, S, y_bf16 ? kSegBf16 : kSegF32, maps);
}

// Clusters of S CTAs (one CTA an SM) that the device runs at once: an SM's
// neighbours limit the larger ones.  Asked once per device.
int resident_clusters(const Ctx &c, int S) {
    static std::atomic<int> known[64][kMaxSplit + 1];
    int dev = 0;
    if (S == 1 || cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return c.num_sms / S;
    int n = known[dev][S].load(std::memory_order_relaxed);
    if (n == 0) {
        static std::atomic<uint64_t> configured{0};
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)(c.num_sms / S * S));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = Shape<32>::SMEM;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)S;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (ensure_smem((const void *)k_mx_product<32>, Shape<32>::SMEM, configured) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, k_mx_product<32>, &cfg) != cudaSuccess || n < 1)
            return 1;
        known[dev][S].store(n, std::memory_order_relaxed);
    }
    return n;
}

struct Plan {
    int NT, S, clusters;
};

// Rows of a unit and CTAs of a cluster: the form whose estimate is least.  Over
// 67 shapes (rows 1-10587, groups 1-64, out 36-12288, in 128-7168) its choice
// took 1.7 % longer on the mean than the best of all forms, run-to-run noise
// included; at the corners 1 x 3584 x 7168 takes 12.7 us with clusters of 1, 8.1
// with 4 and 9.3 with 8; 64 x 12288 x 7168 16 us in units of 64 rows, 24 in units of
// 32; 4768 rows of 25 groups (613 x 1664) 10.9 us in units of 256, 13.3 of 128
// and 23.5 of 32; 926 x 56 x 1280 4.7 us where units of 128 take 5.4.
Plan choose(const Ctx &c, const ProdArgs &a, int y_bf16) {
    const int groups = a.n_groups < a.n_rows ? a.n_groups : a.n_rows;
    const int mean = (a.n_rows + groups - 1) / groups;       // rows of a group, were they even
    const int MT = (a.out + 127) / 128, KC = a.in / kStageCols;
    Plan best{};
    double least = 0;
    for (int NT : {32, 64, 128, 256}) {
        const int KS = NT <= 64 ? 2 : 1;
        const long long items = (long long)groups * ((mean + NT - 1) / NT) * MT;
        for (int S : {1, 2, 4, 8}) {
            // (NT = 256 has one accumulator: reading it several times an item would
            // stall the MMAs)
            if (S > (KC + KS - 1) / KS) continue;
            if ((S > 1 && NT > 64) || (NT == 256 && !y_bf16 && KC > kGroup * kSegF32)) continue;
            long long clusters = resident_clusters(c, S);
            if (clusters > items) clusters = items;
            const long long waves = (items + clusters - 1) / clusters;
            // us, fitted to a sweep of 24 shapes (rows 1-4096, out 1000-12288, in 1024-7168)
            const int n = mean < NT ? mean : NT, tiles = ((KC + KS - 1) / KS + S - 1) / S * KS;
            const double tile = NT == 32 ? 0.23 : NT == 64 ? 0.26 : NT == 128 ? 0.32 : 0.39;
            const double t = (double)waves * (tiles * tile + (S == 1 ? 0.5 + 0.006 * n : 2.0 + 0.05 * n));
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
    const Plan p = choose(c, a, y_bf16);
    if (p.NT == 32) return launch_t<32>(c, a, y_bf16, p.S, p.clusters);
    if (p.NT == 64) return launch_t<64>(c, a, y_bf16, p.S, p.clusters);
    if (p.NT == 128) return launch_t<128>(c, a, y_bf16, p.S, p.clusters);
    return launch_t<256>(c, a, y_bf16, p.S, p.clusters);
}

}  // namespace k3mx
