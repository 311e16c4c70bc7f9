// pnq_int8_mma.cu -- products of 8-bit integer matrices on the fifth-generation tensor cores (tcgen05), sm_103a, for more rows than
// pnq_int8_gemm.cu takes through registers.
//
// The chip has no fast 8-bit integer MMA. Every code is exact in fp16 (11 significant bits) and a product of two is a whole number up to 2^14, so
// the 16-bit MMA with fp32 accumulators sums 1024 of them exactly: no partial sum passes 2^24. After each 1024 of K the accumulator is
// taken out, turned into whole numbers and added to 32-bit sums in registers, while the next 1024 go to a second accumulator.
// That makes the result independent of tile shapes and of how K is split.
//
// Layout. The weight rows are the MMA's M axis (128 lanes of tensor memory per CTA), the activation rows its N axis. The weights stay 8-bit until
// they are on the SM: four warps (or eight, in turn) read a stage's codes from shared memory, one row a thread, widen them (a byte b xor 128
// beside the byte 0x64 is the fp16 number 1024 + 128 + b, less 1152) and write them to tensor memory, where the MMA takes its A operand
// from. Weight bytes cross HBM, L2 and shared memory as they are. x is widened once, in a pass of its own, to scratch (1.2 to 2.8 us), or, for
// products of few stages, by the same warps from a stage's codes to shared memory.
//
// What bounds it. Many rows: the tensor pipe (8192 x 17408 x 5120 745 us in short runs, 1.96 PFLOP/s; 842 in long ones, at the power limit;
// counters of 2048 rows: 85 % busy). A stage of 128 of K with 192 rows moves 137 bytes of shared memory a cycle of its MMAs, where 128 is
// the limit: so activations are not widened there. Few rows: HBM for the weights' bytes (16 x 17408 x 5120 20.7 us for 89 MB), and what
// stands before and after it: launch, the first copies, the sum over a cluster (100 x 256 with 64 rows: 4.8 us).
// What it took (8192 x 17408 x 5120): signals within a pair that do not release memory (2718 us to 1125: a release at cluster scope held each warp up
// by 0.5 us a stage), stages of 128 of K (943), waits by whole warps (792), a row widened before its slot is waited for (781), accumulators of a tile's
// end taken out under the next (745).
//
// Roles of the warps of a CTA: 0..3 (0..7) widen, the next 8 take accumulators out (two per lane quarter, half of the columns each), then one that
// copies (one lane) and one that issues MMAs (one lane). Pairs (CG = 2): two CTAs work on one tile of 256 weight rows (cta_group::2), each with
// its own 128 and half of the activation rows; the first one's thread issues for both.
//
// Every wait is bounded; a wait that gives up records its site in the device error word and ends the role, and tensor memory is
// released whatever the outcome.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <map>
#include <mutex>
#include <utility>

#include "pnq_device.cuh"
#include "pnq_internal.h"

namespace pnq {
namespace {

constexpr int kRows = 128;          // weight rows per CTA and tile (MMA M)
constexpr int KS = 128;             // K of a stage: one row of shared memory for the weights, two for the activations
constexpr int kChunkK = 1024;       // K of an accumulator: 1024 * 2^14 = 2^24
constexpr int kDrainWarps = 8;
constexpr int kMaxStages = 8;
constexpr int kMaxSlots = 4;
constexpr int kBand = 16;           // weight tiles of a band
constexpr int kSmemLimit = 227 * 1024;
constexpr int kCodes = kRows * KS;  // bytes of a stage's weights
constexpr int kSlotCols = KS / 2;   // tensor-memory columns of a widened stage
constexpr int kChunkStages = kChunkK / KS;

struct MmaArgs {
    const float *x_scales, *w_scales;
    void* Y;
    int* err;
    int M, N, K;
    int bn;            // activation rows of a tile
    int ks;            // CTAs (pairs) of a cluster that share a tile's K (1: none)
    int stages, slots; // of the rings in shared and in tensor memory
    int xbox;          // activation rows of a copy
    int weights_once;  // every weight row is read by one tile only
    int early;         // the weights are the caller's: no kernel in flight writes them
};

// Tiles of at most BN activation rows, by CG CTAs with SETS sets of four warps that widen the weights, and with WX the activations too.
template <int BN, int CG, int SETS, bool WX>
struct Plan {
    static constexpr int kCtas = BN <= 64 ? 2 : 1;             // CTAs of an SM
    static constexpr int kCopyWarp = 4 * SETS + kDrainWarps, kMmaWarp = kCopyWarp + 1, kThreads = 32 * (kMmaWarp + 1);
    static constexpr int kBound = kCtas == 2 ? 512 : kThreads; // two CTAs of 14 warps share an SM's four register files as two of 16 do
    static constexpr int kStep = 16 * CG;                      // a tile's activation rows are a multiple of it
    static constexpr int kCols = kCtas == 2 ? 256 : 512;       // tensor-memory columns: two accumulators, and the slots
    static constexpr int kSplit = 8 / CG;                      // the most that share a tile's K: clusters of 8 CTAs
    static constexpr bool kWidenX = WX;                        // a stage holds x's codes; beside every slot of tensor memory there is one of x
    static constexpr int slot(int bn) { return kWidenX ? bn * KS * 2 : 0; }
    static constexpr int stage(int bn) { return kCodes + (kWidenX ? bn * KS : bn / CG * KS * 2); }
    static constexpr int slots(int bn) { return std::min(kMaxSlots, (kCols - 2 * bn) / kSlotCols); }
    static constexpr int stages(int bn) { return std::min(kMaxStages, (kSmemLimit / kCtas - 3 * 1024 - slots(bn) * slot(bn)) / stage(bn)); }
    static constexpr int smem(int bn) { return stages(bn) * stage(bn) + slots(bn) * slot(bn) + 1024; }
    static constexpr int largest_smem() {
        int most = 0;
        for (int bn = kStep; bn <= BN; bn += kStep) most = std::max(most, smem(bn));
        return most;
    }
    // kCtas of them share an SM whatever bn is (1 KB of each CTA is the system's, and the barriers are static)
    static_assert(kCtas * (largest_smem() + 2048) <= 228 * 1024, "the rings leave no room for the CTAs of an SM");
    // fp32 accumulators, fp16 operands, N, M = 128 per CTA
    static __device__ uint32_t idesc(int bn) {
        return (1u << 4) | (static_cast<uint32_t>(bn >> 3) << 17) | (static_cast<uint32_t>(CG * kRows >> 4) << 24);
    }
};

// Shared-memory descriptor: K-major rows of 128 bytes, 128-byte swizzle, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_rows(uint32_t addr) {
    return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (1ull << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// D += A B^T, A (M x 16, fp16) in tensor memory, B (N x 16) in shared memory.
template <int CG>
__device__ __forceinline__ void mma_f16(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if constexpr (CG == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
            "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
            "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
}

// The first CTA of this CTA's pair, by its rank in the cluster (pairs lie along x, the parts of a tile's K along y).
__device__ __forceinline__ uint32_t pair_leader() { return 2u * blockIdx.y; }

// Arrives on the barrier at this offset in both CTAs of the pair whose first has the given rank, when the pair's MMAs are done.
__device__ __forceinline__ void tc_commit_pair_of(uint32_t bar, uint32_t leader) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3u << leader))
        : "memory");
}

// The sum as fp32 (one rounding), times both scales in turn.
__device__ __forceinline__ float scaled(int sum, float x_scale, float w_scale) {
    return __fmul_rn(__fmul_rn(__int2float_rn(sum), x_scale), w_scale);
}
__device__ __forceinline__ void store_product(float* y, float f) { *y = f; }
__device__ __forceinline__ void store_product(__nv_bfloat16* y, float f) { *y = __float2bfloat16_rn(f); }

// Walks the tiles number first, first + step, ..: all roles of a CTA see the same sequence. Bands of 16 weight tiles, row tile by row
// tile: the CTAs at work share a few operand rows in L2.
struct Tile {
    int row0, rows, n0;
};
template <int CG>
struct Walk {
    static constexpr int kTileN = CG * kRows;
    const MmaArgs& a;
    int at, step, nt, mt, m, band, width;
    __device__ explicit Walk(const MmaArgs& args)
        : a(args), at(static_cast<int>(blockIdx.x) / CG), step(static_cast<int>(gridDim.x) / CG), nt((args.N + kTileN - 1) / kTileN),
          mt((args.M + args.bn - 1) / args.bn), m(0), band(0), width(min(kBand, nt)) {}
    __device__ bool next(Tile& o) {
        while (band < nt && at >= width) {
            at -= width;
            if (++m == mt) m = 0, band += kBand, width = min(kBand, nt - band);
        }
        if (band >= nt) return false;
        o = Tile{m * a.bn, min(a.bn, a.M - m * a.bn), (band + at) * kTileN};
        at += step;
        return true;
    }
};

template <int BN, int CG, int SETS, bool WX, class T>
__global__ void __launch_bounds__(Plan<BN, CG, SETS, WX>::kBound, Plan<BN, CG, SETS, WX>::kCtas) int8_mma_kernel(const __grid_constant__ CUtensorMap map_w,
                                                                                             const __grid_constant__ CUtensorMap map_x,
                                                                                             const MmaArgs a) {
    using P = Plan<BN, CG, SETS, WX>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    __shared__ __align__(8) uint64_t bars[3 * kMaxStages + kMaxSlots + 5];
    __shared__ uint32_t tmem_slot;
    const uint32_t b0 = smem_addr(bars), sbase = smem_addr(base);
    auto full_w = [&](int s) { return b0 + 8u * s; };                                // the weights of a stage, this CTA's
    auto full_x = [&](int s) { return b0 + 8u * (kMaxStages + s); };                 // the activations, both CTAs', at the first
    auto slot_done = full_x;                                                          // widened here: a slot's MMAs are done
    auto empty = [&](int s) { return b0 + 8u * (2 * kMaxStages + s); };              // the stage's MMAs are done; widened here: its codes are read
    auto wide = [&](int i) { return b0 + 8u * (3 * kMaxStages + i); };               // a slot is written, by both CTAs, at the first
    auto acc_full = [&](int i) { return b0 + 8u * (3 * kMaxStages + kMaxSlots + i); };
    auto acc_empty = [&](int i) { return b0 + 8u * (3 * kMaxStages + kMaxSlots + 2 + i); };
    const uint32_t finished = b0 + 8u * (3 * kMaxStages + kMaxSlots + 4);
    const int S = a.stages, A = a.slots, bn = a.bn;
    const uint32_t box = static_cast<uint32_t>(bn / CG) * 128;  // bytes of 64 of K of this CTA's activations as fp16, of 128 as codes
    const uint32_t x_bytes = P::kWidenX ? box : 2 * box, stage = kCodes + x_bytes;
    const uint32_t xslots = sbase + static_cast<uint32_t>(S) * stage;  // widened here: activations beside the slots of tensor memory
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? blockIdx.x & 1u : 0u;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_w(s), 1);
            mbar_init(full_x(s), 1);
            mbar_init(empty(s), P::kWidenX ? 4 : 1);
        }
        for (int i = 0; i < A; ++i) mbar_init(wide(i), CG * 4);
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full(i), 1);
            mbar_init(acc_empty(i), CG * kDrainWarps);
        }
        mbar_init(finished, 1);
        mbar_fence_init();
        prefetch_tensor_map(&map_w);
        prefetch_tensor_map(&map_x);
    }
    if constexpr (CG == 2) {
        cluster_sync();  // the pair's barriers exist before either CTA signals them
        if (warp == P::kMmaWarp) tmem_alloc_pair(smem_addr(&tmem_slot), P::kCols);
    } else {
        if (warp == P::kMmaWarp) tmem_alloc(smem_addr(&tmem_slot), P::kCols);
    }
    // nothing above reads what an earlier kernel wrote. Nor do the first copies of the weights below, where they are the caller's own: the
    // pass that widened x has waited for all that came before it, and this kernel begins after that
    if (!a.early || warp != P::kCopyWarp) griddep_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_launch_dependents();
    const uint32_t tmem = tmem_slot, slots = tmem + static_cast<uint32_t>(2 * bn);
    const int nk = (a.K + KS - 1) / KS, kz = static_cast<int>(blockIdx.y);
    const int kt0 = kz * nk / a.ks, kt1 = (kz + 1) * nk / a.ks, chunks = (kt1 - kt0 + kChunkStages - 1) / kChunkStages;
    Walk<CG> walk(a);
    Tile tile{};

    if (warp == P::kCopyWarp) {
        if (elect_one()) {
            const uint64_t pol_x = l2_policy_evict_last(), pol_w = a.weights_once ? l2_policy_evict_first() : pol_x;
            bool ok = true;
            int s = 0, issued = 0, ahead = 0;  // ahead: stages of the first tile whose weights are under way
            uint32_t phase = 1;                // the first wait for each free stage passes
            const uint32_t x_box = static_cast<uint32_t>(a.xbox * KS);
            auto load_weights = [&](int i, int kt) {
                mbar_arrive_expect_tx(full_w(i), kCodes + (P::kWidenX ? x_box : 0u));
                tma_load_2d(sbase + static_cast<uint32_t>(i) * stage + x_bytes, &map_w, kt * KS, tile.n0 + static_cast<int>(rank) * kRows,
                            full_w(i), pol_w);
            };
            if (a.early) {
                Walk<CG> first(a);
                if (first.next(tile))
                    for (; ahead < min(S, kt1 - kt0); ++ahead) load_weights(ahead, kt0 + ahead);
                griddep_wait();
            }
            while (ok && walk.next(tile)) {
                const int xrow = tile.row0 + static_cast<int>(rank) * (bn / CG);
                for (int kt = kt0; kt < kt1; ++kt) {
                    if (issued >= ahead) {
                        if (!mbar_wait_cycles(empty(s), phase)) {
                            ok = false;
                            break;
                        }
                        load_weights(s, kt);
                    }
                    const uint32_t st = sbase + static_cast<uint32_t>(s) * stage;
                    if constexpr (P::kWidenX) {
                        tma_load_2d(st, &map_x, kt * KS, xrow, full_w(s), pol_x);
                    } else {
                        if (rank == 0) mbar_arrive_expect_tx(full_x(s), CG * 2 * x_box);
                        const uint32_t bar = CG == 2 ? cluster_addr(full_x(s), pair_leader()) : full_x(s);
#pragma unroll
                        for (int h = 0; h < KS / 64; ++h) {
                            if constexpr (CG == 2) tma_load_2d_pair(st + h * box, &map_x, kt * KS + 64 * h, xrow, bar, pol_x);
                            else tma_load_2d(st + h * box, &map_x, kt * KS + 64 * h, xrow, bar, pol_x);
                        }
                    }
                    ++issued;
                    if (++s == S) s = 0, phase ^= 1;
                }
            }
            if (!ok) record_error(a.err, kErrEmptyWait);
            // every copy issued has landed before the CTA may exit; a pair's activations are all counted in its first CTA, and the second waits until
            // its last stages are reported free (no signal to its barriers is under way when it exits)
            bool drained = true;
            for (int g = max(0, issued - S); drained && g < issued; ++g) {
                drained = mbar_wait_cycles(full_w(g % S), (g / S) & 1);
                if constexpr (!P::kWidenX) drained = drained && mbar_wait_cycles(rank == 0 ? full_x(g % S) : empty(g % S), (g / S) & 1);
            }
            if (!drained) record_error(a.err, kErrDrainWait);
        }
    } else if (warp == P::kMmaWarp) {
        if (rank == 0 && elect_one()) {
            auto commit = [&](uint32_t bar) {
                if constexpr (CG == 2) tc_commit_pair_of(bar, pair_leader());
                else tc_commit(bar);
            };
            const uint32_t idesc = P::idesc(bn);
            bool ok = true;
            int s = 0, slot = 0, buf = 0;
            uint32_t phase = 0, slot_phase = 0, acc_phase = 1;
            while (ok && walk.next(tile)) {
                for (int kt = kt0, in_chunk = 0; kt < kt1; ++kt) {
                    if (in_chunk == 0 && !mbar_wait_cycles(acc_empty(buf), acc_phase)) {
                        ok = false;
                        break;
                    }
                    if ((!P::kWidenX && !mbar_wait_cycles(full_x(s), phase)) || !mbar_wait_cycles(wide(slot), slot_phase)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t acc = tmem + static_cast<uint32_t>(buf * bn), from = slots + static_cast<uint32_t>(slot * kSlotCols);
                    const uint32_t st = P::kWidenX ? xslots + static_cast<uint32_t>(slot) * 2 * box : sbase + static_cast<uint32_t>(s) * stage;
                    const uint64_t x0 = desc_rows(st), x1 = desc_rows(st + box);
#pragma unroll
                    for (int j = 0; j < KS / 16; ++j)
                        mma_f16<CG>(acc, from + 8 * j, (j < 4 ? x0 : x1) + 2 * (j % 4), idesc, (in_chunk > 0 || j > 0) ? 1u : 0u);
                    commit(P::kWidenX ? slot_done(slot) : empty(s));  // the slot is free, and where it holds activations the stage
                    if (++s == S) s = 0, phase ^= 1;
                    if (++slot == A) slot = 0, slot_phase ^= 1;
                    if (++in_chunk == kChunkStages || kt == kt1 - 1) {
                        commit(acc_full(buf));
                        in_chunk = 0;
                        if (++buf == 2) buf = 0, acc_phase ^= 1;
                    }
                }
            }
            if (!ok) record_error(a.err, kErrFullWait);
            // no MMA is in flight when tensor memory is released
            if constexpr (CG == 2) tc_commit_pair_own(finished);
            else tc_commit(finished);
            if (!mbar_wait_cycles(finished, 0)) record_error(a.err, kErrDrainWait);
        }
    } else if (warp < 4 * SETS) {
        const int row = 32 * (warp & 3) + lane, set = warp >> 2;  // the sets take the stages in turn
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        bool ok = true;
        int i = 0, s = 0, slot = 0, es = 0;   // es, ephase: the stage whose MMAs were the slot's last, A stages before
        uint32_t phase = 0, ephase = 0, sphase = 1;
        auto step = [&] {
            if (++s == S) s = 0, phase ^= 1;
            if (++slot == A) slot = 0, sphase ^= 1;
            if (i++ >= A && ++es == S) es = 0, ephase ^= 1;
        };
        while (ok && walk.next(tile)) {
            for (int kt = kt0; kt < kt1; ++kt, step()) {
                if (SETS == 2 && (i & 1) != set) continue;
                ok = mbar_wait_cycles_warp(full_w(s), phase);
                if (!ok) break;
                const uint32_t src = sbase + static_cast<uint32_t>(s) * stage + x_bytes + static_cast<uint32_t>(row * KS);
                auto widen = [&](int h, uint32_t (&v)[16]) {  // 32 codes of the row: 16-byte chunks 2 h and 2 h + 1, where the swizzle put them
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint4 w = ld_shared_v4<0>(src + 16 * ((2 * h + c) ^ (row & 7)));
                        int8x4_to_f16x2(w.x, v[8 * c], v[8 * c + 1]);
                        int8x4_to_f16x2(w.y, v[8 * c + 2], v[8 * c + 3]);
                        int8x4_to_f16x2(w.z, v[8 * c + 4], v[8 * c + 5]);
                        int8x4_to_f16x2(w.w, v[8 * c + 6], v[8 * c + 7]);
                    }
                };
                auto slot_free = [&] { return i < A || mbar_wait_cycles_warp(empty(es), ephase); };
                auto slot_at = [&](int h) { return slots + static_cast<uint32_t>(slot * kSlotCols + 16 * h) + lanes; };
                if constexpr (P::kCtas == 1) {  // the whole row in registers while the slot is waited for
                    uint32_t v[KS / 32][16];
#pragma unroll
                    for (int h = 0; h < KS / 32; ++h) widen(h, v[h]);
                    ok = slot_free();
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int h = 0; h < KS / 32; ++h) tmem_st16(slot_at(h), v[h]);
                } else {
                    ok = P::kWidenX ? mbar_wait_cycles_warp(slot_done(slot), sphase) : slot_free();
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int h = 0; h < KS / 32; ++h) {
                        uint32_t v[16];
                        widen(h, v);
                        tmem_st16(slot_at(h), v);
                    }
                }
                if constexpr (P::kWidenX) {
                    // the activations, 16 codes a thread and turn: 32 bytes in the row's half of K, where the swizzle of 128 bytes puts them (lanes
                    // of the two halves write theirs in opposite orders, so that they do not meet in a bank)
                    const uint32_t from = sbase + static_cast<uint32_t>(s) * stage, to = xslots + static_cast<uint32_t>(slot) * 2 * box;
                    const int c = row & 7, first = 2 * (c & 3) + (c >> 2);
                    for (int r = row >> 3; r < bn; r += 16) {
                        const uint4 w = ld_shared_v4<0>(from + static_cast<uint32_t>(r * KS + 16 * (c ^ (r & 7))));
                        uint4 u, v;
                        int8x4_to_f16x2(w.x, u.x, u.y);
                        int8x4_to_f16x2(w.y, u.z, u.w);
                        int8x4_to_f16x2(w.z, v.x, v.y);
                        int8x4_to_f16x2(w.w, v.z, v.w);
                        const uint32_t row_at = to + static_cast<uint32_t>(c >> 2) * box + static_cast<uint32_t>(r * 128);
                        st_shared_v4(row_at + 16 * (first ^ (r & 7)), c < 4 ? u : v);
                        st_shared_v4(row_at + 16 * (first ^ 1 ^ (r & 7)), c < 4 ? v : u);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(empty(s));
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CG == 2) mbar_arrive_cluster_relaxed(cluster_addr(wide(slot), pair_leader()));
                    else mbar_arrive(wide(slot));
                }
            }
        }
        if (!ok && lane == 0) record_error(a.err, kErrOperandWait);
        tc_fence_before();
    } else {
        const int q = warp & 3, half = (warp - 4 * SETS) >> 2;  // lanes 32 q .. of tensor memory, half of the columns
        constexpr int kHalf = BN / 2, kLoad = P::kStep / 2;
        const int columns = bn / 2;  // a multiple of kLoad
        T* Y = static_cast<T*>(a.Y);
        int* red = reinterpret_cast<int*>(base);
        bool ok = true;
        int buf = 0;
        uint32_t acc_phase = 0;
        while (walk.next(tile)) {
            const int cols = min(columns, tile.rows - half * columns), m0 = tile.row0 + half * columns;
            const int n = tile.n0 + static_cast<int>(rank) * kRows + 32 * q + lane;
            // the scales, under way while the sums are: this lane's weight row's, and of 32 columns at a time one a lane
            const float ws = a.ks == 1 && n < a.N ? ld_l2(a.w_scales + n) : 0.0f;
            float xs[(kHalf + 31) / 32];
#pragma unroll
            for (int p = 0; p < (kHalf + 31) / 32; ++p) xs[p] = a.ks == 1 && 32 * p + lane < cols ? ld_l2(a.x_scales + m0 + 32 * p + lane) : 0.0f;
            int sum[kHalf];
#pragma unroll
            for (int j = 0; j < kHalf; ++j) sum[j] = 0;
            for (int c = 0; c < chunks; ++c) {
                ok = mbar_wait_cycles_warp(acc_full(buf), acc_phase);
                if (!ok) break;
                tc_fence_after();
                const uint32_t acc = tmem + static_cast<uint32_t>(buf * bn + half * columns) + (static_cast<uint32_t>(32 * q) << 16);
#pragma unroll
                for (int p = 0; p < kHalf / kLoad; ++p) {
                    if (p * kLoad >= cols) continue;
                    uint32_t v[kLoad];
                    tmem_ld<kLoad>(acc + p * kLoad, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < kLoad; ++j) sum[p * kLoad + j] += __float2int_rn(__uint_as_float(v[j]));
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CG == 2) mbar_arrive_cluster_relaxed(cluster_addr(acc_empty(buf), pair_leader()));
                    else mbar_arrive(acc_empty(buf));
                }
                if (++buf == 2) buf = 0, acc_phase ^= 1;
            }
            if (!ok) break;
            if (a.ks > 1) {
                // the partial sums to shared memory, [column][128 rows]; every copy and MMA of the one tile is done
#pragma unroll
                for (int j = 0; j < kHalf; ++j)
                    if (j < cols) red[(half * columns + j) * kRows + 32 * q + lane] = sum[j];
            } else {
                T* y = Y + static_cast<int64_t>(m0) * a.N + n;
#pragma unroll
                for (int p = 0; p < (kHalf + 31) / 32; ++p) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const float x_scale = __shfl_sync(0xffffffffu, xs[p], j);
                        if (32 * p + j < cols && n < a.N) store_product(y, scaled(sum[32 * p + j], x_scale, ws));
                        y += a.N;
                    }
                }
            }
        }
        if (!ok && lane == 0) record_error(a.err, kErrFullWait);
        tc_fence_before();
    }
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();  // both CTAs' copies have landed, both accumulators are read
    if (a.ks > 1) {
        // CTA kz of the cluster adds up its share of the tile's columns over the ks partial tiles (distributed shared memory), and writes them
        Walk<CG> again(a);
        again.next(tile);
        const int c0 = kz * tile.rows / a.ks, c1 = (kz + 1) * tile.rows / a.ks;
        // a thread sums four rows of a column, always the same rows: their scales while the cluster meets
        constexpr int kEach = kRows / 4;
        const int r = 4 * (static_cast<int>(threadIdx.x) % kEach), n = tile.n0 + static_cast<int>(rank) * kRows + r;
        float ws[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) ws[i] = n + i < a.N ? ld_l2(a.w_scales + n + i) : 0.0f;
        if constexpr (CG == 1) cluster_sync();
        T* Y = static_cast<T*>(a.Y);
#pragma unroll 2
        for (int c = c0 + static_cast<int>(threadIdx.x) / kEach; c < c1; c += P::kThreads / kEach) {
            const uint32_t at = sbase + 4u * static_cast<uint32_t>(c * kRows + r);
            const float xs = ld_l2(a.x_scales + tile.row0 + c);
            float4 v[P::kSplit];
#pragma unroll
            for (int z = 0; z < P::kSplit; ++z)
                if (z < a.ks) v[z] = ld_dsmem_f32x4(cluster_addr(at, rank + static_cast<uint32_t>(CG * z)));
            int f[4] = {0, 0, 0, 0};
#pragma unroll
            for (int z = 0; z < P::kSplit; ++z)
                if (z < a.ks) {
                    f[0] += __float_as_int(v[z].x), f[1] += __float_as_int(v[z].y);
                    f[2] += __float_as_int(v[z].z), f[3] += __float_as_int(v[z].w);
                }
            T* y = Y + static_cast<int64_t>(tile.row0 + c) * a.N + n;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < a.N) store_product(y + i, scaled(f[i], xs, ws[i]));
        }
        cluster_sync();  // no CTA leaves while another still reads its tile
    }
    if (warp == P::kMmaWarp) {
        tc_fence_after();
        if constexpr (CG == 2) tmem_dealloc_pair(tmem, P::kCols);
        else tmem_dealloc(tmem, P::kCols);
    }
}

// ---- x widened, and rows of weights laid out on 16 bytes -------------------------------------------------

// 16 bytes of a row from `at` on, bytes from K on as zeros.
template <bool ALIGNED>
__device__ __forceinline__ uint4 load16(const int8_t* row, int at, int K) {
    if (ALIGNED && at + 16 <= K) return ld_l2(reinterpret_cast<const uint4*>(row + at));
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (at + i < K) w[i / 4] |= ld_l2(reinterpret_cast<const uint8_t*>(row + at + i)) << (8 * (i % 4));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Rows of K codes -> rows of `per` pieces of 16: as fp16, or as they are.
template <bool ALIGNED, bool WIDEN>
__global__ void __launch_bounds__(256) int8_rows_copy_kernel(const int8_t* X, int64_t ld, int64_t rows, int K, int per, uint4* out) {
    griddep_begin();
    const int64_t total = rows * per;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; u < total; u += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t r = u / per;
        const int c = static_cast<int>(u - r * per);
        const uint4 w = load16<ALIGNED>(X + r * ld, 16 * c, K);
        if constexpr (WIDEN) {
            uint4 a, b;
            int8x4_to_f16x2(w.x, a.x, a.y);
            int8x4_to_f16x2(w.y, a.z, a.w);
            int8x4_to_f16x2(w.z, b.x, b.y);
            int8x4_to_f16x2(w.w, b.z, b.w);
            out[2 * u] = a;
            out[2 * u + 1] = b;
        } else {
            out[u] = w;
        }
    }
}

template <bool WIDEN>
cudaError_t copy_rows(const int8_t* X, int64_t ld, int64_t rows, int64_t K, void* out, cudaStream_t stream) {
    const bool aligned = reinterpret_cast<uintptr_t>(X) % 16 == 0 && ld % 16 == 0;
    const int64_t per = (K + 15) / 16;
    const int grid = static_cast<int>(std::min<int64_t>((rows * per + 255) / 256, static_cast<int64_t>(device_sm_count()) * 32));
    return launch_dependent(aligned ? int8_rows_copy_kernel<true, WIDEN> : int8_rows_copy_kernel<false, WIDEN>, grid, 256, stream, X, ld, rows,
                            static_cast<int>(K), static_cast<int>(per), static_cast<uint4*>(out));
}

// ---- launches ------------------------------------------------------------------------------------------

// How a product is cut: tiles of bn activation rows, and the CTAs (pairs) that share a tile's K.
struct Cut {
    int bn, ks;
    int64_t tiles, stages;  // stages: one after the other
};

// Clusters of CG by ks CTAs of a kernel that the current device holds at once (not every group of SMs divides evenly), asked for with the largest
// tile's shared memory, so that the answer is one for all of them. The runtime counts one CTA an SM for kernels that allocate tensor memory; two fit where
// theirs is half of it. The kernel that widens x too has the same threads, tensor memory and CTAs an SM, and goes by the same count.
template <int BN, int CG, int SETS, bool WX>
cudaError_t resident(int ks, int* clusters) {
    using P = Plan<BN, CG, SETS, WX>;
    constexpr int smem = P::largest_smem();
    static std::mutex mu;
    static std::map<std::pair<int, int>, int> known;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    int& n = known[{dev, ks}];
    if (n == 0) {
        const void* kernel = reinterpret_cast<const void*>(int8_mma_kernel<BN, CG, SETS, WX, float>);
        e = opt_in_smem(kernel, smem);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t lc{};
        lc.gridDim = dim3(static_cast<unsigned>(CG * device_sm_count()), static_cast<unsigned>(ks));
        lc.blockDim = dim3(P::kThreads);
        lc.dynamicSmemBytes = static_cast<size_t>(smem);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = CG;
        attr[0].val.clusterDim.y = static_cast<unsigned>(ks);
        attr[0].val.clusterDim.z = 1;
        lc.attrs = attr;
        lc.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&n, kernel, &lc);
        if (e != cudaSuccess) return e;
        n = std::max(n, 1);
    }
    *clusters = n * P::kCtas;
    return cudaSuccess;
}

// The tiles of a product, and over how many CTAs (pairs) K is split: so that the fewest stages come one after the other, with a cluster's sum
// counted as three. K is split only where all clusters run at once: a second round of them costs more than a split gains.
template <int BN, int CG, int SETS, bool WX>
cudaError_t cut_by(int64_t M, int64_t N, int64_t K, Cut* c) {
    using P = Plan<BN, CG, SETS, WX>;
    const int64_t mt = (M + BN - 1) / BN, nk = (K + KS - 1) / KS;
    c->bn = static_cast<int>(((M + mt - 1) / mt + P::kStep - 1) / P::kStep * P::kStep);
    c->tiles = (N + CG * kRows - 1) / (CG * kRows) * mt;
    c->ks = 1;
    c->stages = (c->tiles * CG + P::kCtas * device_sm_count() - 1) / (P::kCtas * device_sm_count()) * nk;
    for (int ks = 2; ks <= P::kSplit && nk >= 2 * ks; ++ks) {
        int clusters = 0;
        const cudaError_t e = resident<BN, CG, SETS, WX>(ks, &clusters);
        if (e != cudaSuccess) return e;
        const int64_t stages = (nk + ks - 1) / ks + 3;
        if (c->tiles <= clusters && stages < c->stages) c->stages = stages, c->ks = ks;
    }
    return cudaSuccess;
}

template <int BN, int CG, int SETS, bool WX, class T>
cudaError_t run_mma(const CUtensorMap& map_w, const CUtensorMap& map_x, const MmaArgs& a, int64_t tiles, cudaStream_t stream) {
    using P = Plan<BN, CG, SETS, WX>;
    const int smem = P::smem(a.bn);
    auto kern = int8_mma_kernel<BN, CG, SETS, WX, T>;
    const cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t lc{};
    // K split: one tile a cluster; otherwise as many CTAs as the device holds at once, each over its tiles
    const int64_t units = static_cast<int64_t>(P::kCtas) * device_sm_count() / CG;
    lc.gridDim = dim3(static_cast<unsigned>(CG * (a.ks > 1 ? tiles : std::min(tiles, units))), static_cast<unsigned>(a.ks));
    lc.blockDim = dim3(P::kThreads);
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
    return cudaLaunchKernelEx(&lc, kern, map_w, map_x, a);
}

template <int BN, int CG, int SETS, bool WX>
cudaError_t run_cut(const Cut& c, bool bf16, const void* x, int64_t ldx, const int8_t* w, int64_t ldw, MmaArgs a, cudaStream_t stream) {
    using P = Plan<BN, CG, SETS, WX>;
    const int64_t M = a.M, N = a.N, K = a.K;
    a.bn = c.bn, a.ks = c.ks;
    a.stages = P::stages(c.bn), a.slots = P::slots(c.bn);
    a.xbox = CG == 2 ? c.bn / CG : static_cast<int>(std::min<int64_t>(c.bn, M));
    a.weights_once = M <= c.bn;
    CUtensorMap map_w, map_x;
    const bool mapped = P::kWidenX ? encode_rows_map(&map_x, x, M, K, 1, ldx, KS, a.xbox)
                                   : encode_rows_map(&map_x, x, M, K, 2, (K + 15) / 16 * 32, 64, a.xbox);
    if (!mapped || !encode_rows_map(&map_w, w, N, K, 1, ldw, KS, kRows)) return cudaErrorInvalidValue;
    return bf16 ? run_mma<BN, CG, SETS, WX, __nv_bfloat16>(map_w, map_x, a, c.tiles, stream)
                : run_mma<BN, CG, SETS, WX, float>(map_w, map_x, a, c.tiles, stream);
}

bool on_16(const Int8View& w) { return reinterpret_cast<uintptr_t>(w.codes) % 16 == 0 && w.ld % 16 == 0; }

}  // namespace

// x as fp16 (or its codes where their rows are not on 16 bytes), and the weights' codes where their rows are not on 16 bytes.
uint64_t int8_mma_scratch(int64_t M, const Int8View& w, int64_t K) {
    const uint64_t per = static_cast<uint64_t>((K + 15) / 16);
    return static_cast<uint64_t>(M) * per * 32 + (on_16(w) ? 0 : static_cast<uint64_t>(w.rows) * per * 16);
}

cudaError_t launch_int8_mma(const Int8View& x, const Int8View& w, int64_t K, bool bf16, void* Y, void* scratch, int* err,
                            cudaStream_t stream) {
    const int64_t per = (K + 15) / 16;
    MmaArgs a{};
    a.x_scales = x.scales, a.w_scales = w.scales, a.Y = Y, a.err = err;
    a.M = static_cast<int>(x.rows), a.N = static_cast<int>(w.rows), a.K = static_cast<int>(K);
    // up to 64 rows a CTA a tile; above, pairs: tiles of at most 128 rows, widened by eight warps, or of at most 192 by four (more would not leave
    // registers for 192 rows' sums), by the stages that come one after the other and what one takes, 0.22 us and 0.00122 for each row
    // (fitted on 17408 x 5120, 5120 x 17408 and 4096 x 4096, 65 to 2048 rows)
    Cut small{}, few{}, many{};
    cudaError_t e = cut_by<64, 1, 1, false>(a.M, a.N, a.K, &small);
    if (e == cudaSuccess && a.M > 64) e = cut_by<128, 2, 2, false>(a.M, a.N, a.K, &few);
    if (e == cudaSuccess && a.M > 64) e = cut_by<192, 2, 1, false>(a.M, a.N, a.K, &many);
    if (e != cudaSuccess) return e;
    auto time = [](const Cut& c) { return static_cast<double>(c.stages) * (0.22 + 0.00122 * c.bn); };
    // A kernel that widens x itself saves the pass that does it, some 1.2 us, and takes 0.0028 us more for each row of each stage: for few stages (64 x
    // 1001 x 2063 7.9 us instead of 8.4, 64 x 4096 x 4096 13.6 and 14.2, but 33 x 17408 x 5120 23.8 and 22.7). Of few tiles a CTA an SM, each with
    // few stages, is then faster than pairs are, too (128 x 1001 x 2063 8.1 and 10.7, 333 x 384 x 7168 13.4 and 14.9; two CTAs an SM lose: 192 x 1001 x
    // 2063 10.6 and 10.2).
    const int64_t work = (small.ks == 1 ? small.stages : ((K + KS - 1) / KS + small.ks - 1) / small.ks) * small.bn;
    const bool wide_x = a.M <= 64 ? work <= 300 : small.tiles * small.ks <= device_sm_count() && work <= 512;
    const bool own_x = wide_x && on_16(x), own = on_16(w);
    const void* xs = own_x ? static_cast<const void*>(x.codes) : scratch;
    const int64_t ldx = own_x ? x.ld : per * 16;
    if (!own_x) {
        e = wide_x ? copy_rows<false>(x.codes, x.ld, x.rows, K, scratch, stream) : copy_rows<true>(x.codes, x.ld, x.rows, K, scratch, stream);
        if (e != cudaSuccess) return e;
    }
    const int8_t* codes = w.codes;
    int64_t ldw = w.ld;
    if (!own) {
        int8_t* copy = static_cast<int8_t*>(scratch) + x.rows * per * 32;
        e = copy_rows<false>(w.codes, w.ld, w.rows, K, copy, stream);
        if (e != cudaSuccess) return e;
        codes = copy, ldw = per * 16;
    }
    a.early = own && !own_x;
    if (wide_x) return run_cut<64, 1, 1, true>(small, bf16, xs, ldx, codes, ldw, a, stream);
    if (a.M <= 64) return run_cut<64, 1, 1, false>(small, bf16, xs, ldx, codes, ldw, a, stream);
    return time(few) <= time(many) ? run_cut<128, 2, 2, false>(few, bf16, xs, ldx, codes, ldw, a, stream)
                                   : run_cut<192, 2, 1, false>(many, bf16, xs, ldx, codes, ldw, a, stream);
}

}  // namespace pnq
