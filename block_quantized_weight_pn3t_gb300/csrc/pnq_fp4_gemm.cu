// pnq_fp4_gemm.cu -- products of 4-bit microscaled operands on the fifth-generation tensor cores
// (tcgen05, block-scaled kinds), sm_103a: Y[m][n] = alpha * sum_k X[m][k] W[n][k], dense or by experts.
//
// The tensor core takes the packed codes and the scale words as they are stored and accumulates in fp32:
//   NVFP4: kind::mxf4nvf4, scale_vec::4X (one E4M3 word per 16 of K);
//   MXFP4: kind::mxf4, scale_vec::2X (one power of two per 32).
// A product of two codes and two scales is exact; the global multipliers go into the epilogue.
//
// Layout. The weight rows are the MMA's M axis (128 lanes of tensor memory per CTA), the activation rows its N axis
// (32 .. 256 columns): a few activation rows then waste no weight traffic, an expert's ragged rows waste columns
// only, and a warp's store covers consecutive n of one Y row.
//
// Roles. Persistent CTAs walk the tiles. One lane of warp 0 fills a ring of stages by tensor-map copies: a stage is
// K = 256 of a tile (128-byte rows of codes, 128-byte swizzle) and its 512-byte scale tiles. One lane of warp 1 copies
// the stage's scale tiles to tensor memory (tcgen05.cp, 32 rows x 16 bytes, repeated over the four lane quarters) and
// issues one MMA per K = 64. Warps 2..9 take the accumulator to registers, one weight row per lane, and store it while
// the next tile is multiplied. Up to 128 columns two accumulators alternate; 256 columns leave room for one beside
// the scale columns.
//
// What bounds it (GB300, times of 8192 x 17408 x 5120 NVFP4 to bf16 unless said otherwise; in short runs, in runs of
// seconds the power limit holds it at 250 us).
//   - Many rows: the tensor pipe. 256 x 256 tiles by CTA pairs (cta_group::2: each CTA holds half of the activation
//     rows, so a stage is 38 KB for the work that takes one CTA 54 KB) 230 us = 6.4 PFLOP/s, single CTAs of 128 x 256
//     248 us, of 128 x 128 290 us. ncu: the tensor pipe is busy 68 percent of the cycles. A stage in the run of a tile
//     takes 0.30 us, 0.27 of it the MMAs; a change of tiles costs some 1.9 us, the way from the last MMA through the
//     accumulator's release to the first (beside the scale columns that each stage has for itself there is no room for a
//     second one) and the stores. 192 columns with two accumulators took longer a stage than 256 (279 us).
//   - Few rows: HBM. One row of 17408 x 5120 takes 11.0 us (50.1 MB: 7.4 us at the copy rate; a product of 1/20 of the
//     bytes, 17408 x 256, takes 3.4). K is split over a cluster where there are fewer tiles than SMs (13 rows of 5120 x 17408:
//     20.7 -> 12.3 us with three CTAs per tile); the partial tiles meet in distributed shared memory, in CTA order.
//   - Between them: a stage's turn through one thread's waits and instructions. Waits by one lane (32 lanes probe the
//     barrier 32 times), bounded by the SM's clock (a read of the global timer costs 0.4 us), one wait per stage (its
//     scale columns are its own), and the next stage probed ahead brought a 128-column stage from 0.42 to 0.21 us.
//
// Every wait is bounded; a wait that gives up records its site in the device error word and ends the role, and
// tensor memory is released whatever the outcome.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <map>
#include <mutex>
#include <tuple>
#include <utility>

#include "pnq_device.cuh"
#include "pnq_internal.h"

namespace pnq {
namespace {

constexpr int kRows = 128;                     // weight rows per tile (MMA M)
constexpr int kStageK = 256;                   // K per stage: 128 bytes of codes per row
constexpr int kStageWords = kStageK / 8;       // the same in u32 words
constexpr int kCodesA = kRows * kStageK / 2;   // 16 KB
constexpr int kScaleTile = 512;                // 128 rows x 4 groups
constexpr int kEpilogueWarps = 8;              // two per lane quarter of tensor memory
constexpr int kEpilogueThreads = 32 * kEpilogueWarps;
constexpr int kThreads = 64 + kEpilogueThreads;  // producer, MMA, epilogue
constexpr int kMaxExperts = 1024;
constexpr int kMaxStages = 10;
constexpr int kMaxSplit = 8;                   // CTAs of a cluster that share a tile's K
constexpr int kSmemLimit = 227 * 1024;
constexpr int kStaticSmem = 9 * 1024;          // barriers, first rows and tiles of the experts (rounded up)

constexpr int imin(int a, int b) { return a < b ? a : b; }

struct GemmArgs {
    void* Y;
    int* err;
    PlanView p;              // experts == 0: dense
    const float* w_global;   // per expert, or null
    float alpha;
    int M, N, K;             // activation rows, weight rows of a matrix, K
    int chunks;              // scale tiles along K per 128-row block
    int weights_once;        // every weight row is read by one tile only
    int static_weights;      // dense: no earlier kernel in flight writes the weights
    int ks;                  // CTAs of a cluster that share a tile's K (1: none)
    int xbox;                // activation rows of a copy: as many copies as a tile's rows need
};

template <bool MX, int BN, int CG>
struct Plan {
    static constexpr int kTiles = MX ? 2 : 4;                    // scale tiles per stage and 128-row block
    static constexpr int kScalesA = kTiles * kScaleTile;
    static constexpr int kBlocksB = BN > 128 ? 2 : 1;            // 128-row blocks of activation scales
    static constexpr int kCodesB = BN / CG * kStageK / 2;         // a pair's CTAs hold half of the activation rows each
    static constexpr int kStage = kCodesA + kCodesB + kScalesA * (1 + kBlocksB);
    static constexpr int kAcc = BN <= 128 ? 2 : 1;               // accumulators
    // tensor-memory columns: accumulators, then a set of scale columns for every stage (A: 4 per tile, B: 4 per tile and
    // block): a stage that is full again has its scale columns free too, so the MMA thread waits once per stage
    static constexpr int kSetCols = 4 * kTiles * (1 + kBlocksB);
    static constexpr int kStages = imin(kMaxStages, imin((kSmemLimit - 1024 - kStaticSmem) / kStage, (512 - kAcc * BN) / kSetCols));
    static_assert(kStages >= 3, "three stages at least");
    static constexpr int kUsed = kAcc * BN + kStages * kSetCols;
    static constexpr int kCols = kUsed <= 64 ? 64 : kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
    // E2M1 operands, scale type, N, M = 128 per CTA
    static constexpr uint32_t kIdesc = (1u << 7) | (1u << 10) | (static_cast<uint32_t>(BN >> 3) << 17) |
                                       ((MX ? 1u : 0u) << 23) | (static_cast<uint32_t>(CG * kRows >> 4) << 24);
};

// Shared-memory descriptors: K-major 128-byte swizzled code rows (8-row groups 1024 bytes apart), and unswizzled
// scale tiles (8 rows of 16 bytes = 128 contiguous bytes).
__device__ __forceinline__ uint64_t desc_codes(uint32_t addr) {
    return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (1ull << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_scales(uint32_t addr) {
    return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(128 >> 4) << 32) | (1ull << 46);
}

// One scale tile (32 rows x 16 bytes) -> four columns of tensor memory, in all four lane quarters (a pair: in both
// CTAs, each from its own shared memory).
template <int CG>
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint64_t desc) {
    if constexpr (CG == 2)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

#define PNQ_MMA_FP4(GROUP, KIND)                                                                                   \
    asm volatile(                                                                                                  \
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                                                          \
        "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),          \
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)                                            \
        : "memory")

template <bool MX, int CG>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
    if constexpr (MX && CG == 1) PNQ_MMA_FP4("1", "mxf4.block_scale.scale_vec::2X");
    if constexpr (MX && CG == 2) PNQ_MMA_FP4("2", "mxf4.block_scale.scale_vec::2X");
    if constexpr (!MX && CG == 1) PNQ_MMA_FP4("1", "mxf4nvf4.block_scale.scale_vec::4X");
    if constexpr (!MX && CG == 2) PNQ_MMA_FP4("2", "mxf4nvf4.block_scale.scale_vec::4X");
}
#undef PNQ_MMA_FP4

// A tile: 128 weight rows (a pair: 256) from n0 of matrix e, up to BN activation rows.
struct Tile {
    int e;        // matrix (0 when dense)
    int row0;     // first activation row (global)
    int rows;     // activation rows in the tile
    int n0;       // first weight row within the matrix
    int sblock;   // 128-row scale block of row0 within the matrix
    int srow;     // row0's row within that block (a multiple of 64)
};

// Walks the tiles number first, first + step, ..: all roles of a CTA see the same sequence. Dense: bands of 16 weight
// tiles, row tile by row tile (the CTAs at work share a few operand rows in L2). By experts: `starts[e]` and `firsts[e]`
// (shared memory) are the tiles and the rows before expert e. Steps by addition: a division or two per tile stood in the way of the threads
// that issue copies and MMAs.
template <int BN, int CG>
struct Walk {
    static constexpr int kTileN = CG * kRows, kBand = 16;
    const GemmArgs& a;
    const int *starts, *firsts;
    int at, step, nt, mt;   // dense: `at` counts from (m, 0) of the band
    int m, band, width;     // row tile; first weight tile of the band and its tiles
    int e;                  // expert
    __device__ Walk(const GemmArgs& args, const int* tile_starts, const int* first_rows)
        : a(args), starts(tile_starts), firsts(first_rows), at(static_cast<int>(blockIdx.x) / CG), step(static_cast<int>(gridDim.x) / CG),
          nt((args.N + kTileN - 1) / kTileN), mt((args.M + BN - 1) / BN), m(0), band(0), width(min(kBand, nt)), e(0) {}
    __device__ bool next(Tile& o) {
        if (a.p.experts == 0) {
            while (at >= width) {
                at -= width;
                if (++m == mt) {
                    m = 0;
                    band += kBand;
                    width = min(kBand, nt - band);
                    if (width <= 0) {
                        width = 0x7fffffff;  // past the end: no further tile
                        band = nt;
                        mt = 0x7fffffff;
                    }
                }
            }
            if (band >= nt) return false;
            o = Tile{0, m * BN, min(BN, a.M - m * BN), (band + at) * kTileN, m * BN / 128, m * BN % 128};
        } else {
            if (at >= starts[a.p.experts]) return false;
            while (at >= starts[e + 1]) ++e;
            const int first = firsts[e], count = firsts[e + 1] - first;
            const int tiles = (count + BN - 1) / BN, r = at - starts[e], n = r / tiles, i = r - n * tiles;
            o = Tile{e, first + i * BN, min(BN, count - i * BN), n * kTileN, i * BN / 128, i * BN % 128};
        }
        at += step;
        return true;
    }
};

// f * scale of one accumulator column -> y, n consecutive across the warp.
template <class T>
__device__ __forceinline__ void store_y(T* y, float f) {
    if constexpr (sizeof(T) == 4) *y = f;
    else *y = __float2bfloat16_rn(f);
}

template <bool MX, int BN, int CG, class T>
__global__ void __launch_bounds__(kThreads, 1) fp4_gemm_kernel(const __grid_constant__ CUtensorMap map_w,
                                                               const __grid_constant__ CUtensorMap map_ws,
                                                               const __grid_constant__ CUtensorMap map_x,
                                                               const __grid_constant__ CUtensorMap map_xs,
                                                               const GemmArgs a) {
    using P = Plan<MX, BN, CG>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 5];
    __shared__ uint32_t tmem_slot;
    __shared__ int starts[kMaxExperts + 1], firsts[kMaxExperts + 1];
    __shared__ int warp_sums[kThreads / 32];
    const uint32_t b0 = smem_addr(bars);
    auto full = [&](int s) { return b0 + 8u * s; };
    auto empty = [&](int s) { return b0 + 8u * (kMaxStages + s); };
    auto acc_full = [&](int i) { return b0 + 8u * (2 * kMaxStages + i); };
    auto acc_empty = [&](int i) { return b0 + 8u * (2 * kMaxStages + 2 + i); };
    const uint32_t finished = b0 + 8u * (2 * kMaxStages + 4);
    constexpr int S = P::kStages;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t sbase = smem_addr(base);
    // pair: CTA 0 leads (its barriers count both CTAs' copies, its thread issues the MMAs of both)
    const uint32_t rank = CG == 2 ? blockIdx.x & 1u : 0u;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full(i), 1);
            mbar_init(acc_empty(i), CG * kEpilogueWarps);
        }
        mbar_init(finished, 1);
        mbar_fence_init();
        prefetch_tensor_map(&map_w);
        prefetch_tensor_map(&map_ws);
        prefetch_tensor_map(&map_x);
        prefetch_tensor_map(&map_xs);
    }
    if constexpr (CG == 2) {
        cluster_sync();  // the pair's barriers exist before either CTA signals them
        if (warp == 1) tmem_alloc_pair(smem_addr(&tmem_slot), P::kCols);
    } else {
        if (warp == 1) tmem_alloc(smem_addr(&tmem_slot), P::kCols);
    }
    // nothing above reads what an earlier kernel wrote; static weights: nor do the first copies below, and their thread
    // waits after them
    const bool early = a.static_weights && a.p.experts == 0;
    if (!early || warp != 0) griddep_wait();
    if (a.p.experts > 0) {
        // tiles before each expert: a block scan, each thread over consecutive experts
        const int E = a.p.experts, nt = (a.N + CG * kRows - 1) / (CG * kRows), per = (E + kThreads - 1) / kThreads;
        const int e0 = min(E, static_cast<int>(threadIdx.x) * per), e1 = min(E, e0 + per);
        int sum = 0, first = ld_l2(a.p.offsets + e0);
        bool wrong = first < 0 || first > a.M;  // not the offsets of a sorted plan of these sizes
        for (int e = e0; e < e1; ++e) {
            const int next = ld_l2(a.p.offsets + e + 1);
            wrong |= next < first || next > a.M;
            firsts[e] = first;
            starts[e] = wrong ? 0 : (next - first + BN - 1) / BN * nt;
            sum += starts[e];
            first = next;
        }
        if (__syncthreads_or(wrong)) {  // no tile and no row in use
            sum = first = 0;
            for (int e = e0; e < e1; ++e) starts[e] = 0;
        }
        if (e1 == E) firsts[E] = first;
        int incl = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += u;
        }
        if (lane == 31) warp_sums[warp] = incl;
        __syncthreads();
        int at = incl - sum;
        for (int w = 0; w < warp; ++w) at += warp_sums[w];
        for (int e = e0; e < e1; ++e) {
            const int tiles = starts[e];
            starts[e] = at;
            at += tiles;
        }
        if (e1 == E && e0 < E) starts[E] = at;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_launch_dependents();
    const uint32_t tmem = tmem_slot;
    // this CTA's share of the stages along K: [kt0, kt1)
    const int nk = (a.K + kStageK - 1) / kStageK, kz = static_cast<int>(blockIdx.y);
    const int kt0 = kz * nk / a.ks, kt1 = (kz + 1) * nk / a.ks;
    Walk<BN, CG> walk(a, starts, firsts);
    Tile tile{};

    // Warps 0 and 1 run their loops in one elected lane: a wait by 32 lanes is 32 probes of the barrier, one after
    // the other (a stage's turn took 0.25 us that way with nothing else in it).
    if (warp == 0) {
        if (elect_one()) {
            // weights that no other tile reads leave L2 first
            const uint64_t pol_x = l2_policy_evict_last(), pol_w = a.weights_once ? l2_policy_evict_first() : pol_x;
            const int blocks_w = (a.N + 127) / 128;
            bool ok = true;
            int s = 0, issued = 0;
            uint32_t phase = 1;  // the first wait for each free stage passes
            auto load = [&](uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar, uint64_t pol) {
                if constexpr (CG == 2) tma_load_2d_pair(dst, map, x, y, bar, pol);
                else tma_load_2d(dst, map, x, y, bar, pol);
            };
            // of the tile in turn: coordinates at K = 0, copies and bytes of a stage. All of it outside the loop over K: this
            // one thread's instructions are a stage's turn where a tile is small.
            int wrow = 0, wsc = 0, xrow = 0, xsc = 0, xcopies = 0;
            uint32_t bytes = 0;
            auto take = [&] {
                const int n0 = tile.n0 + static_cast<int>(rank) * kRows;
                wrow = tile.e * a.N + n0;
                wsc = (tile.e * blocks_w + n0 / 128) * a.chunks;
                xrow = tile.row0 + static_cast<int>(rank) * (BN / CG);
                xsc = ((a.p.experts ? max(0, plan_index(ld_l2(a.p.block_start + tile.e), a.p.tiled)) : 0) + tile.sblock) * a.chunks;
                // rows past the tile's activations are not copied: their columns are not stored (and a copy's rows past
                // the end of the matrix, filled with zeros, take longer than rows that are there)
                xcopies = CG == 2 ? 1 : (tile.rows + a.xbox - 1) / a.xbox;  // a pair's CTAs copy one half each
                bytes = static_cast<uint32_t>(CG * (P::kStage - P::kCodesB + xcopies * a.xbox * (kStageK / 2)));
            };
            auto load_weights = [&](int i, int kt) {
                const uint32_t st = sbase + static_cast<uint32_t>(i * P::kStage), bar = CG == 2 ? cluster_addr(full(i), 0) : full(i);
                if (rank == 0) mbar_arrive_expect_tx(full(i), bytes);
                load(st, &map_w, kt * kStageWords, wrow, bar, pol_w);
                load(st + kCodesA + P::kCodesB, &map_ws, 0, wsc + kt * P::kTiles, bar, pol_w);
            };
            int ahead = 0;  // stages of the first tile whose weights are under way
            if (early) {
                Walk<BN, CG> first(a, starts, firsts);
                if (first.next(tile)) {
                    take();
                    for (; ahead < min(S, kt1 - kt0); ++ahead) load_weights(ahead, kt0 + ahead);
                }
                griddep_wait();
            }
            while (ok && walk.next(tile)) {
                take();
                for (int kt = kt0; kt < kt1; ++kt) {
                    if (issued >= ahead) {
                        if (!mbar_wait_cycles(empty(s), phase)) {
                            ok = false;
                            break;
                        }
                        load_weights(s, kt);
                    }
                    const uint32_t st = sbase + static_cast<uint32_t>(s * P::kStage), bar = CG == 2 ? cluster_addr(full(s), 0) : full(s);
                    load(st + kCodesA, &map_x, kt * kStageWords, xrow, bar, pol_x);
#pragma unroll 1
                    for (int c = 1; c < xcopies; ++c)
                        load(st + kCodesA + static_cast<uint32_t>(c * a.xbox * (kStageK / 2)), &map_x, kt * kStageWords,
                             xrow + c * a.xbox, bar, pol_x);
#pragma unroll
                    for (int b = 0; b < P::kBlocksB; ++b)
                        load(st + kCodesA + P::kCodesB + P::kScalesA * (1 + b), &map_xs, 0, xsc + b * a.chunks + kt * P::kTiles, bar,
                             pol_x);
                    ++issued;
                    if (++s == S) s = 0, phase ^= 1;
                }
            }
            if (!ok) record_error(a.err, kErrEmptyWait);
            // every copy issued has landed before the CTA may exit; a pair's are all counted in CTA 0, and CTA 1 waits
            // until its last stages are reported free (no signal to its barriers is under way when it exits)
            bool drained = true;
            for (int g = max(0, issued - S); drained && g < issued; ++g)
                drained = mbar_wait_cycles(rank == 0 ? full(g % S) : empty(g % S), (g / S) & 1);
            if (!drained) record_error(a.err, kErrDrainWait);
        }
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            auto commit = [](uint32_t bar) {
                if constexpr (CG == 2) tc_commit_pair(bar);
                else tc_commit(bar);
            };
            bool ok = true;
            int s = 0, buf = 0;
            uint32_t phase = 0, acc_phase = 1;
            bool peek = false;  // the stage in turn was seen full
            while (ok && walk.next(tile)) {
                const uint32_t acc = tmem + static_cast<uint32_t>(buf * BN);
                const uint32_t sfb_row = static_cast<uint32_t>(tile.srow >> 5);
                for (int kt = kt0; kt < kt1; ++kt) {
                    if (!peek && !mbar_wait_cycles(full(s), phase)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t st = sbase + static_cast<uint32_t>(s * P::kStage), sc = st + kCodesA + P::kCodesB;
                    const uint32_t sfa = tmem + P::kAcc * BN + static_cast<uint32_t>(s * P::kSetCols);
                    const uint32_t sfb = sfa + 4 * P::kTiles;
                    const uint64_t da = desc_codes(st), db = desc_codes(st + kCodesA), ds = desc_scales(sc);
                    const int steps = min(4, (a.K - kt * kStageK + 63) / 64);  // K past the end: no MMA
                    const int now = s;
                    if (++s == S) s = 0, phase ^= 1;
                    peek = mbar_test(full(s), phase);  // a probe takes some 100 cycles: over before the next stage's turn
#pragma unroll
                    for (int j = 0; j < P::kTiles; ++j) {
                        tmem_copy_scales<CG>(sfa + 4 * j, ds + (j * kScaleTile >> 4));
#pragma unroll
                        for (int b = 0; b < P::kBlocksB; ++b)
                            tmem_copy_scales<CG>(sfb + 4 * (j * P::kBlocksB + b),
                                                 ds + ((P::kScalesA * (1 + b) + j * kScaleTile) >> 4));
                    }
                    if (kt == kt0) {  // the accumulator: asked for once the first scales are on their way
                        if (!mbar_wait_cycles(acc_empty(buf), acc_phase)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        constexpr int kPerTile = MX ? 2 : 1;
                        const int q = j / kPerTile;
                        // MXFP4: two K steps share a tile; the descriptor says which half of its words
                        const uint32_t half = MX ? 2u * (j & 1) : 0u;
                        if (j < steps)
                            mma_fp4<MX, CG>(acc, da + 2 * j, db + 2 * j, P::kIdesc | (half << 4) | (half << 29), sfa + 4 * q,
                                            sfb + 4 * q * P::kBlocksB + sfb_row, (kt > kt0 || j > 0) ? 1u : 0u);
                    }
                    commit(empty(now));  // the stage and its scale columns are free once these MMAs have read them
                    if (kt == kt1 - 1) commit(acc_full(buf));
                }
                if (++buf == P::kAcc) buf = 0, acc_phase ^= 1;
            }
            if (!ok) record_error(a.err, kErrFullWait);
            // no MMA is in flight when tensor memory is released
            if constexpr (CG == 2) tc_commit_pair_own(finished);
            else tc_commit(finished);
            if (!mbar_wait_cycles(finished, 0)) record_error(a.err, kErrDrainWait);
        }
    } else {
        const int q = warp & 3, half = (warp - 2) >> 2;  // lanes 32 q .. of tensor memory, half of the columns
        constexpr int kHalf = BN / 2;
        constexpr int kChunk = kHalf < 32 ? kHalf : 32;
        T* Y = static_cast<T*>(a.Y);
        float* red = reinterpret_cast<float*>(base);
        bool ok = true;
        int buf = 0;
        uint32_t acc_phase = 0;
        while (walk.next(tile)) {
            if (lane == 0) ok = mbar_wait_cycles(acc_full(buf), acc_phase);
            ok = __shfl_sync(0xffffffffu, ok, 0);  // tcgen05.ld is .aligned: the warp goes on or stops as one
            if (!ok) break;
            tc_fence_after();
            const uint32_t acc = tmem + static_cast<uint32_t>(buf * BN + half * kHalf) + (static_cast<uint32_t>(32 * q) << 16);
            const int r = tile.n0 + static_cast<int>(rank) * kRows + 32 * q + lane, cols = tile.rows - half * kHalf;
            // the accumulator goes to registers at once: the next tile's MMAs wait for nothing more
            uint32_t v[kHalf / kChunk][kChunk];
#pragma unroll
            for (int c = 0; c < kHalf / kChunk; ++c)
                if (c * kChunk < cols) tmem_ld<kChunk>(acc + c * kChunk, v[c]);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (CG == 2) mbar_arrive_cluster(cluster_addr(acc_empty(buf), 0));
                else mbar_arrive(acc_empty(buf));
            }
            if (a.ks > 1) {
                // the partial tile to shared memory, [column][128 rows]; every copy and MMA of the one tile is done
#pragma unroll
                for (int c = 0; c < kHalf / kChunk; ++c)
#pragma unroll
                    for (int j = 0; j < kChunk; ++j)
                        if (c * kChunk + j < cols)
                            red[(half * kHalf + c * kChunk + j) * kRows + 32 * q + lane] = __uint_as_float(v[c][j]);
            } else if (r < a.N) {
                const float scale = a.w_global ? a.alpha * ld_l2(a.w_global + tile.e) : a.alpha;
                T* y = Y + static_cast<int64_t>(tile.row0 + half * kHalf) * a.N + r;
#pragma unroll
                for (int c = 0; c < kHalf / kChunk; ++c)
#pragma unroll
                    for (int j = 0; j < kChunk; ++j) {
                        if (c * kChunk + j < cols) store_y(y, __uint_as_float(v[c][j]) * scale);
                        y += a.N;
                    }
            }
            if (++buf == P::kAcc) buf = 0, acc_phase ^= 1;
        }
        if (!ok && lane == 0) record_error(a.err, kErrFullWait);
        if (a.p.experts > 0) {  // rows past the rows in use
            const int64_t used = firsts[a.p.experts], count = (static_cast<int64_t>(a.M) - used) * a.N;
            const int64_t cta = blockIdx.y * static_cast<int64_t>(gridDim.x) + blockIdx.x;
            const int64_t step = static_cast<int64_t>(gridDim.x) * gridDim.y * kEpilogueThreads;
            for (int64_t j = cta * kEpilogueThreads + static_cast<int>(threadIdx.x) - 64; j < count; j += step)
                Y[used * a.N + j] = T(0.0f);
        }
        tc_fence_before();
    }
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();  // both CTAs' copies have landed, both accumulators are read
    if (CG == 1 && a.ks > 1) {
        // CTA kz of the cluster sums its share of the tile's columns over the ks partial tiles, in CTA order
        // (distributed shared memory), and writes them
        cluster_sync();
        Walk<BN, CG> again(a, starts, firsts);
        if (again.next(tile)) {
            T* Y = static_cast<T*>(a.Y);
            const float scale = a.w_global ? a.alpha * ld_l2(a.w_global + tile.e) : a.alpha;
            // a thread sums four rows of a column: its loads from all the CTAs are in flight together
            const int c0 = kz * tile.rows / a.ks, c1 = (kz + 1) * tile.rows / a.ks;
            for (int e = static_cast<int>(threadIdx.x); e < (c1 - c0) * (kRows / 4); e += kThreads) {
                const int c = c0 + e / (kRows / 4), r = 4 * (e % (kRows / 4));
                const uint32_t at = sbase + 4u * static_cast<uint32_t>(c * kRows + r);
                float4 v[kMaxSplit];
#pragma unroll
                for (int z = 0; z < kMaxSplit; ++z)
                    if (z < a.ks) v[z] = ld_dsmem_f32x4(cluster_addr(at, static_cast<uint32_t>(z)));
                float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int z = 0; z < kMaxSplit; ++z)
                    if (z < a.ks) f[0] += v[z].x, f[1] += v[z].y, f[2] += v[z].z, f[3] += v[z].w;
                T* y = Y + static_cast<int64_t>(tile.row0 + c) * a.N + tile.n0 + r;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (tile.n0 + r + i < a.N) store_y(y + i, f[i] * scale);
            }
        }
        cluster_sync();  // no CTA leaves while another still reads its tile
    }
    if (warp == 1) {
        tc_fence_after();
        if constexpr (CG == 2) tmem_dealloc_pair(tmem, P::kCols);
        else tmem_dealloc(tmem, P::kCols);
    }
}

// Clusters of x by y CTAs of a kernel that the current device holds at once (not every group of SMs divides evenly).
cudaError_t resident_clusters(const void* kernel, int smem, int x, int y, int* clusters) {
    static std::mutex mu;
    static std::map<std::tuple<const void*, int, int, int>, int> known;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    int& n = known[{kernel, dev, x, y}];
    if (n == 0) {
        e = opt_in_smem(kernel, smem);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t lc{};
        lc.gridDim = dim3(static_cast<unsigned>(x * device_sm_count()), static_cast<unsigned>(y));
        lc.blockDim = dim3(kThreads);
        lc.dynamicSmemBytes = static_cast<size_t>(smem);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(x);
        attr[0].val.clusterDim.y = static_cast<unsigned>(y);
        attr[0].val.clusterDim.z = 1;
        lc.attrs = attr;
        lc.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&n, kernel, &lc);
        if (e != cudaSuccess) return e;
        n = std::max(n, 1);
    }
    *clusters = n;
    return cudaSuccess;
}

template <bool MX, int BN, int CG>
constexpr int gemm_smem() {
    return Plan<MX, BN, CG>::kStages * Plan<MX, BN, CG>::kStage + 1024;
}

template <bool MX, int BN, int CG, class T>
cudaError_t run_gemm(const CUtensorMap (&maps)[4], const GemmArgs& a, int64_t tiles, cudaStream_t stream) {
    using P = Plan<MX, BN, CG>;
    static_assert(P::kStages * P::kStage >= BN * kRows * 4, "a partial tile fits the stages");
    constexpr int smem = gemm_smem<MX, BN, CG>();
    auto kern = fp4_gemm_kernel<MX, BN, CG, T>;
    cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t lc{};
    lc.blockDim = dim3(kThreads);
    lc.dynamicSmemBytes = static_cast<size_t>(smem);
    lc.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CG;
    attr[0].val.clusterDim.y = static_cast<unsigned>(a.ks);
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 2;
    // K split: one tile per cluster; otherwise as many persistent CTAs (pairs) as the device holds at once
    if (a.ks > 1) {
        lc.gridDim = dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(a.ks));
    } else if (CG == 1) {
        lc.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(tiles, device_sm_count())));
    } else {
        int pairs = 0;
        e = resident_clusters(reinterpret_cast<const void*>(kern), smem, CG, 1, &pairs);
        if (e != cudaSuccess) return e;
        lc.gridDim = dim3(static_cast<unsigned>(CG * std::min<int64_t>(tiles, pairs)));
    }
    return cudaLaunchKernelEx(&lc, kern, maps[0], maps[1], maps[2], maps[3], a);
}

template <bool MX, int BN, int CG = 1>
cudaError_t run_out(bool bf16, const Fp4View& x, const Fp4View& w, int64_t K, GemmArgs a, int64_t tiles,
                    cudaStream_t stream) {
    using P = Plan<MX, BN, CG>;
    // the tile's rows in one copy; by experts, with few rows each, in copies of 32 (full tiles of 128 in copies of 32 took
    // 12 percent longer)
    a.xbox = static_cast<int>(std::min<int64_t>(BN / CG, a.p.experts && x.rows < 32ll * a.p.experts ? 32 : x.rows));
    if (CG == 2) a.xbox = BN / CG;
    const int64_t nt = (w.rows + kRows - 1) / kRows;  // 128-row scale blocks of a matrix
    // 128-row scale blocks that a copy may touch: by experts the operand has room for any distribution
    const int64_t xblocks = a.p.experts ? (x.rows + 127 * std::min<int64_t>(a.p.experts, x.rows)) / 128 : (x.rows + 127) / 128;
    CUtensorMap maps[4];
    if (!encode_u32_map_pitch(&maps[0], w.codes, w.rows * w.matrices, K / 8, fp4_pitch(K), kStageWords, kRows, true) ||
        !encode_u32_map(&maps[1], w.scales, nt * w.matrices * a.chunks, 128, 128, P::kTiles) ||
        !encode_u32_map_pitch(&maps[2], x.codes, x.rows, K / 8, fp4_pitch(K), kStageWords, a.xbox, true) ||
        !encode_u32_map(&maps[3], x.scales, xblocks * a.chunks, 128, 128, P::kTiles))
        return cudaErrorInvalidValue;
    return bf16 ? run_gemm<MX, BN, CG, __nv_bfloat16>(maps, a, tiles, stream)
                : run_gemm<MX, BN, CG, float>(maps, a, tiles, stream);
}

// A tile shape: columns, CTAs per tile, and what a stage of K, a further tile of a CTA, and the last one cost beyond
// its stages (us; the first two over long sums and many tiles on products of 17408 rows, the third as the difference
// of one-tile products; a tile's cost is what its stores and the change of accumulators leave uncovered).
struct Shape {
    int bn, cg;
    double stage, tile, last;
};
constexpr Shape kShapes[] = {{32, 1, 0.25, 0.6, 0.0}, {64, 1, 0.25, 0.7, 0.3}, {128, 1, 0.21, 1.0, 0.8}, {256, 2, 0.30, 1.9, 2.4}};
constexpr Shape kExpertShapes[] = {{64, 1, 0, 0, 0}, {128, 1, 0, 0, 0}, {256, 1, 0, 0, 0}, {256, 2, 0, 0, 0}};

// Tiles of a dense product of M by N rows.
int64_t dense_tiles(const Shape& s, int64_t M, int64_t N) {
    return (N + s.cg * kRows - 1) / (s.cg * kRows) * ((M + s.bn - 1) / s.bn);
}

// The shape of a dense product's tiles, and the CTAs that share a tile's K, whose estimate is least.
cudaError_t choose_dense(int64_t M, int64_t N, int64_t K, Shape* best, int* split) {
    const int64_t nk = (K + kStageK - 1) / kStageK;
    double least = 0.0;
    for (const Shape& s : kShapes) {
        if (s.bn == 32 && M > 32) continue;
        const int64_t tiles = dense_tiles(s, M, N);
        for (int ks = 1; ks <= (s.cg == 1 ? kMaxSplit : 1) && (ks == 1 || nk >= 3 * ks); ++ks) {
            int slots = device_sm_count() / s.cg;
            if (ks > 1) {
                // clusters of any shape hold one CTA per SM: the 64-column kernel answers for all
                const cudaError_t e = resident_clusters(reinterpret_cast<const void*>(fp4_gemm_kernel<false, 64, 1, float>),
                                                        gemm_smem<false, 64, 1>(), 1, ks, &slots);
                if (e != cudaSuccess) return e;
                if (tiles > slots) break;  // one tile per cluster, all at once
            }
            const double waves = static_cast<double>((tiles + slots - 1) / slots);
            const double stages = static_cast<double>((nk + ks - 1) / ks);
            double t = waves * stages * s.stage + (waves - 1.0) * s.tile + s.last;
            if (ks > 1) t += 1.6 + 0.01 * static_cast<double>(std::min<int64_t>(s.bn, M));  // the cluster's sum
            if (least == 0.0 || t < least) least = t, *best = s, *split = ks;
        }
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t fp4_gemm_shape(int64_t M, int64_t N, int64_t K, int* columns, int* ctas, int* split) {
    Shape s{};
    const cudaError_t e = choose_dense(M, N, K, &s, split);
    *columns = s.bn;
    *ctas = s.cg;
    return e;
}

cudaError_t launch_fp4_gemm(bool mx, const Fp4View& x, const Fp4View& w, int64_t K, const PlanView& p, float alpha,
                            const float* w_global, bool bf16, void* Y, int* err, bool static_weights,
                            cudaStream_t stream) {
    GemmArgs a{};
    a.Y = Y;
    a.err = err;
    a.p = p;
    a.w_global = w_global;
    a.alpha = alpha;
    a.M = static_cast<int>(x.rows);
    a.N = static_cast<int>(w.rows);
    a.K = static_cast<int>(K);
    a.chunks = static_cast<int>(fp4_chunks(mx, K));
    a.static_weights = static_weights;
    a.ks = 1;
    Shape best{};
    int64_t tiles = 0;
    if (p.experts) {
        // the experts' loads are not known here: by the rows in all, and by the average. 64 columns where no expert can
        // have more (one token, 8 of 64 experts of 1408 x 2048: 8.2 us, 8.5 with 128); 256 from 160 rows an expert on
        // (64 experts of 1408 x 2048, 100 rows each: 23.1 us with 128, 27.4 with 256; 192 each: 34.6 and 29.2), by pairs
        // where K outweighs their dearer change of tiles (8 experts of 4096 x 4096, 1000 rows each: 54.6 us and 51.3 by
        // pairs; 64 of 1408 x 2048: 87.3 and 95.4). The rule looks at neither N nor the number of SMs: few experts with few
        // weight rows leave SMs without a tile (8 experts of 512 x 2048, 200 rows each: 7.9 us, 6.6 with 128 columns; of
        // 512 x 4096: 10.6 by pairs, 8.3 with 128)
        best = kExpertShapes[x.rows <= 64 ? 0 : x.rows < 160ll * p.experts ? 1 : K < 4096 ? 2 : 3];
        a.weights_once = best.bn < 256;
        // the most that any distribution of the rows makes
        tiles = (w.rows + best.cg * kRows - 1) / (best.cg * kRows) *
                std::min<int64_t>(x.rows, x.rows / best.bn + std::min<int64_t>(p.experts, x.rows));
    } else {
        const cudaError_t e = choose_dense(x.rows, w.rows, K, &best, &a.ks);
        if (e != cudaSuccess) return e;
        tiles = dense_tiles(best, x.rows, w.rows);
        a.weights_once = x.rows <= best.bn;
    }
    auto go = [&](auto m) {
        constexpr bool MX = decltype(m)::value;
        switch (best.bn) {
            case 32: return run_out<MX, 32>(bf16, x, w, K, a, tiles, stream);
            case 64: return run_out<MX, 64>(bf16, x, w, K, a, tiles, stream);
            case 128: return run_out<MX, 128>(bf16, x, w, K, a, tiles, stream);
            default: return best.cg == 2 ? run_out<MX, 256, 2>(bf16, x, w, K, a, tiles, stream)
                                         : run_out<MX, 256>(bf16, x, w, K, a, tiles, stream);
        }
    };
    return mx ? go(std::true_type{}) : go(std::false_type{});
}

}  // namespace pnq
