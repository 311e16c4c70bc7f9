// pnq_fp4_gemm.cu -- products of 4-bit microscaled operands on the fifth-generation tensor cores
// (tcgen05, block-scaled kinds), sm_103a: Y[m][n] = alpha * sum_k X[m][k] W[n][k], dense or by experts.
//
// The tensor core takes the packed codes and the scale words as they are stored and accumulates in fp32:
//   NVFP4: kind::mxf4nvf4, scale_vec::4X (one E4M3 word per 16 of K);
//   MXFP4: kind::mxf4, scale_vec::2X (one power of two per 32).
// A product of two codes and two scales is exact; the global multipliers go into the epilogue.
//
// Roles. The weight rows are the MMA's M axis (128 lanes), the activation rows its N axis (BN columns): a few
// activation rows then waste no weight traffic, and a warp's store covers consecutive n of one Y row.
// Persistent CTAs walk the tiles. Warp 0 (one thread) fills a ring of stages by tensor-map copies: a stage is
// K = 256 of a tile (128-byte rows of codes, 128-byte swizzle) and its 512-byte scale tiles. Warp 1 (one
// thread) copies the stage's scale tiles to tensor memory (tcgen05.cp, 32 rows x 16 bytes, repeated over the
// four lane quarters) and issues one MMA per K = 64. Warps 2..5 read the accumulator back, one weight row per
// thread, and store. With BN <= 128 two accumulators alternate, so a tile's stores overlap the next tile's MMAs.
//
// Every wait is bounded; a wait that gives up records its site in the device error word and ends the role, and
// tensor memory is released whatever the outcome.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "pnq_device.cuh"
#include "pnq_internal.h"

namespace pnq {
namespace {

constexpr int kRows = 128;                     // weight rows per tile (MMA M)
constexpr int kStageK = 256;                   // K per stage: 128 bytes of codes per row
constexpr int kStageWords = kStageK / 8;       // the same in u32 words
constexpr int kCodesA = kRows * kStageK / 2;   // 16 KB
constexpr int kScaleTile = 512;                // 128 rows x 4 groups
constexpr int kThreads = 192;                  // producer, MMA, four epilogue warps
constexpr int kEpilogueThreads = 128;
constexpr int kMaxExperts = 1024;
constexpr int kMaxStages = 10;
constexpr int kSmemLimit = 227 * 1024;

struct GemmArgs {
    void* Y;
    int* err;
    PlanView p;              // experts == 0: dense
    const float* w_global;   // per expert, or null
    float alpha;
    int M, N, K;             // activation rows, weight rows of a matrix, K
    int chunks;              // scale tiles along K per 128-row block
    int S;                   // stages
};

template <bool MX, int BN>
struct Plan {
    static constexpr int kTiles = MX ? 2 : 4;                    // scale tiles per stage and 128-row block
    static constexpr int kScalesA = kTiles * kScaleTile;
    static constexpr int kBlocksB = BN > 128 ? 2 : 1;            // 128-row blocks of activation scales
    static constexpr int kCodesB = BN * kStageK / 2;
    static constexpr int kStage = kCodesA + kCodesB + kScalesA * (1 + kBlocksB);
    static constexpr int kAcc = BN <= 128 ? 2 : 1;               // accumulators
    // tensor-memory columns: accumulators, then two sets of scale columns (A: 4 per tile, B: 4 per tile and block)
    static constexpr int kSetCols = 4 * kTiles * (1 + kBlocksB);
    static constexpr int kUsed = kAcc * BN + 2 * kSetCols;
    static constexpr int kCols = kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
    // E2M1 operands, scale type, N, M = 128
    static constexpr uint32_t kIdesc = (1u << 7) | (1u << 10) | (static_cast<uint32_t>(BN >> 3) << 17) |
                                       ((MX ? 1u : 0u) << 23) | (static_cast<uint32_t>(kRows >> 4) << 24);
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

// One scale tile (32 rows x 16 bytes) -> four columns of tensor memory, in all four lane quarters.
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

template <bool MX>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
    if constexpr (MX)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
}

// A tile: 128 weight rows from n0 of matrix e, up to BN activation rows from m0 of the matrix's rows.
struct Tile {
    int e;        // matrix (0 when dense)
    int row0;     // first activation row (global)
    int rows;     // activation rows in the tile
    int n0;       // first weight row within the matrix
    int sblock;   // 128-row scale block of row0
    int srow;     // row0's row within that block (a multiple of 64)
};

// Walks the tiles t = first, first + step, ..: all roles of a CTA see the same sequence. By experts: `starts[e]`
// (shared memory) is the number of tiles before expert e.
template <int BN>
struct Walk {
    const GemmArgs& a;
    const int* starts;
    int t, step, nt, e;
    __device__ Walk(const GemmArgs& args, const int* tile_starts)
        : a(args), starts(tile_starts), t(static_cast<int>(blockIdx.x)), step(static_cast<int>(gridDim.x)),
          nt((args.N + kRows - 1) / kRows), e(0) {}
    __device__ bool next(Tile& o) {
        int m;
        if (a.p.experts == 0) {
            const int mt = (a.M + BN - 1) / BN;
            if (t >= nt * mt) return false;
            // bands of 16 weight tiles: the CTAs at work share a few operand rows in L2
            const int band = t / (16 * mt), r = t - band * 16 * mt;
            const int width = min(16, nt - 16 * band);
            m = r / width;
            o = Tile{0, m * BN, min(BN, a.M - m * BN), (16 * band + r - m * width) * kRows, m * BN / 128, m * BN % 128};
        } else {
            if (t >= starts[a.p.experts]) return false;
            while (t >= starts[e + 1]) ++e;
            const int first = __ldg(a.p.offsets + e), count = __ldg(a.p.offsets + e + 1) - first;
            const int mt = (count + BN - 1) / BN, r = t - starts[e];
            m = r % mt;
            o = Tile{e, first + m * BN, min(BN, count - m * BN), r / mt * kRows,
                     __ldg(a.p.block_start + e) + m * BN / 128, m * BN % 128};
        }
        t += step;
        return true;
    }
};

template <bool MX, int BN, class T>
__global__ void __launch_bounds__(kThreads, 1) fp4_gemm_kernel(const __grid_constant__ CUtensorMap map_w,
                                                               const __grid_constant__ CUtensorMap map_ws,
                                                               const __grid_constant__ CUtensorMap map_x,
                                                               const __grid_constant__ CUtensorMap map_xs,
                                                               const GemmArgs a) {
    using P = Plan<MX, BN>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 5];
    __shared__ uint32_t tmem_slot;
    __shared__ int starts[kMaxExperts + 1];
    __shared__ int warp_sums[kThreads / 32];
    const uint32_t b0 = smem_addr(bars);
    auto full = [&](int s) { return b0 + 8u * s; };
    auto empty = [&](int s) { return b0 + 8u * (kMaxStages + s); };
    auto acc_full = [&](int i) { return b0 + 8u * (2 * kMaxStages + i); };
    auto acc_empty = [&](int i) { return b0 + 8u * (2 * kMaxStages + 2 + i); };
    const uint32_t finished = b0 + 8u * (2 * kMaxStages + 4);
    const int S = a.S, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto stage = [&](int s) { return smem_addr(base) + static_cast<uint32_t>(s * P::kStage); };

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full(i), 1);
            mbar_init(acc_empty(i), kEpilogueThreads / 32);
        }
        mbar_init(finished, 1);
        mbar_fence_init();
    }
    if (warp == 1) tmem_alloc(smem_addr(&tmem_slot), P::kCols);
    if (a.p.experts > 0) {
        // tiles before each expert: a block scan, each thread over consecutive experts
        const int E = a.p.experts, nt = (a.N + kRows - 1) / kRows, per = (E + kThreads - 1) / kThreads;
        const int e0 = min(E, static_cast<int>(threadIdx.x) * per), e1 = min(E, e0 + per);
        int sum = 0;
        for (int e = e0; e < e1; ++e) sum += (__ldg(a.p.offsets + e + 1) - __ldg(a.p.offsets + e) + BN - 1) / BN * nt;
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
            starts[e] = at;
            at += (__ldg(a.p.offsets + e + 1) - __ldg(a.p.offsets + e) + BN - 1) / BN * nt;
        }
        if (e1 == E && e0 < E) starts[E] = at;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const int nk = (a.K + kStageK - 1) / kStageK;
    Walk<BN> walk(a, starts);
    Tile tile;

    if (warp == 0) {
        if (lane == 0) {
            // one pass over the weights of a tile row: keep the activations in L2, let the weights go first
            const uint64_t pol_w = l2_policy_evict_first(), pol_x = l2_policy_evict_last();
            const int blocks_w = (a.N + 127) / 128;
            bool ok = true;
            int i = 0;
            while (ok && walk.next(tile)) {
                const int wrow = tile.e * a.N + tile.n0;
                const int wsc = (tile.e * blocks_w + tile.n0 / 128) * a.chunks, xsc = tile.sblock * a.chunks;
                for (int kt = 0; kt < nk; ++kt, ++i) {
                    const int s = i % S;
                    if (i >= S && !mbar_wait_bounded(empty(s), ((i / S) - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    const uint32_t st = stage(s), sc = st + kCodesA + P::kCodesB;
                    mbar_arrive_expect_tx(full(s), P::kStage);
                    tma_load_2d(st, &map_w, kt * kStageWords, wrow, full(s), pol_w);
                    tma_load_2d(sc, &map_ws, 0, wsc + kt * P::kTiles, full(s), pol_w);
                    tma_load_2d(st + kCodesA, &map_x, kt * kStageWords, tile.row0, full(s), pol_x);
#pragma unroll
                    for (int b = 0; b < P::kBlocksB; ++b)
                        tma_load_2d(sc + P::kScalesA * (1 + b), &map_xs, 0, xsc + b * a.chunks + kt * P::kTiles, full(s), pol_x);
                }
            }
            if (!ok) record_error(a.err, kErrEmptyWait);
            bool drained = true;  // every copy issued has landed before the CTA may exit
            for (int g = max(0, i - S); drained && g < i; ++g) drained = mbar_wait_bounded(full(g % S), (g / S) & 1);
            if (!drained) record_error(a.err, kErrDrainWait);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            bool ok = true;
            int i = 0, n = 0;
            while (ok && walk.next(tile)) {
                const int buf = n % P::kAcc;
                if (n >= P::kAcc && !mbar_wait_bounded(acc_empty(buf), ((n / P::kAcc) - 1) & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t acc = tmem + static_cast<uint32_t>(buf * BN);
                for (int kt = 0; kt < nk; ++kt, ++i) {
                    const int s = i % S;
                    if (!mbar_wait_bounded(full(s), (i / S) & 1)) {
                        ok = false;
                        break;
                    }
                    // the scale columns of stage i - 2 are written again: its MMAs have to be done
                    if (i >= 2 && !mbar_wait_bounded(empty((i - 2) % S), ((i - 2) / S) & 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t st = stage(s), sc = st + kCodesA + P::kCodesB;
                    const uint32_t sfa = tmem + P::kAcc * BN + static_cast<uint32_t>((i & 1) * P::kSetCols);
                    const uint32_t sfb = sfa + 4 * P::kTiles;
#pragma unroll
                    for (int j = 0; j < P::kTiles; ++j) {
                        tmem_copy_scales(sfa + 4 * j, desc_scales(sc + j * kScaleTile));
#pragma unroll
                        for (int b = 0; b < P::kBlocksB; ++b)
                            tmem_copy_scales(sfb + 4 * (j * P::kBlocksB + b),
                                             desc_scales(sc + P::kScalesA * (1 + b) + j * kScaleTile));
                    }
                    const int steps = min(4, (a.K - kt * kStageK + 63) / 64);  // K past the end: no MMA
                    for (int j = 0; j < steps; ++j) {
                        const int q = MX ? j >> 1 : j;
                        // MXFP4: two K steps share a tile; the descriptor says which half of its words
                        const uint32_t half = MX ? 2u * (j & 1) : 0u;
                        mma_fp4<MX>(acc, desc_codes(st + 32 * j), desc_codes(st + kCodesA + 32 * j),
                                    P::kIdesc | (half << 4) | (half << 29), sfa + 4 * q,
                                    sfb + 4 * q * P::kBlocksB + (tile.srow >> 5), (kt > 0 || j > 0) ? 1u : 0u);
                    }
                    tc_commit(empty(s));  // the stage and its scale columns are free once these MMAs have read them
                }
                if (!ok) break;
                tc_commit(acc_full(buf));
                ++n;
            }
            if (!ok) record_error(a.err, kErrFullWait);
            tc_commit(finished);  // no MMA is in flight when tensor memory is released
            if (!mbar_wait_bounded(finished, 0)) record_error(a.err, kErrDrainWait);
        }
        __syncwarp();
    } else {
        const int q = warp & 3;  // lanes 32 q .. of tensor memory
        T* Y = static_cast<T*>(a.Y);
        bool ok = true;
        int n = 0;
        while (walk.next(tile)) {
            const int buf = n % P::kAcc;
            ok = mbar_wait_warp(acc_full(buf), (n / P::kAcc) & 1);  // warp-uniform: tcgen05.ld is .aligned
            if (!ok) break;
            tc_fence_after();
            const uint32_t acc = tmem + static_cast<uint32_t>(buf * BN) + (static_cast<uint32_t>(32 * q) << 16);
            const int r = tile.n0 + 32 * q + lane;
            const float scale = a.w_global ? a.alpha * __ldg(a.w_global + tile.e) : a.alpha;
            T* y = Y + static_cast<int64_t>(tile.row0) * a.N + r;
#pragma unroll 1
            for (int c0 = 0; c0 < BN && c0 < tile.rows; c0 += 16) {
                uint32_t v[16];
                tmem_ld<16>(acc + static_cast<uint32_t>(c0), v);
                tmem_wait_ld();
                if (r < a.N) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (c0 + j < tile.rows) {
                            const float f = __uint_as_float(v[j]) * scale;
                            if constexpr (sizeof(T) == 4) y[static_cast<int64_t>(c0 + j) * a.N] = f;
                            else y[static_cast<int64_t>(c0 + j) * a.N] = __float2bfloat16_rn(f);
                        }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty(buf));
            ++n;
        }
        if (!ok && lane == 0) record_error(a.err, kErrFullWait);
        if (a.p.experts > 0) {  // rows past the rows in use
            const int64_t used = __ldg(a.p.offsets + a.p.experts), count = (static_cast<int64_t>(a.M) - used) * a.N;
            const int tid = static_cast<int>(threadIdx.x) - (kThreads - kEpilogueThreads);
            for (int64_t j = static_cast<int64_t>(blockIdx.x) * kEpilogueThreads + tid; j < count;
                 j += static_cast<int64_t>(gridDim.x) * kEpilogueThreads)
                Y[used * a.N + j] = T(0.0f);
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, P::kCols);
    }
}

template <bool MX, int BN, class T>
cudaError_t run_gemm(const CUtensorMap (&maps)[4], GemmArgs a, int64_t tiles, cudaStream_t stream) {
    using P = Plan<MX, BN>;
    constexpr int kStatic = 8 * 1024;  // barriers, expert tiles (rounded up)
    a.S = std::min(kMaxStages, (kSmemLimit - 1024 - kStatic) / P::kStage);
    static_assert((kSmemLimit - 1024 - kStatic) / P::kStage >= 3, "three stages at least");
    const int smem = a.S * P::kStage + 1024;
    auto kern = fp4_gemm_kernel<MX, BN, T>;
    const cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return e;
    const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(tiles, device_sm_count())));
    kern<<<grid, kThreads, smem, stream>>>(maps[0], maps[1], maps[2], maps[3], a);
    return cudaGetLastError();
}

template <bool MX, int BN>
cudaError_t run_out(bool bf16, const Fp4View& x, const Fp4View& w, int64_t K, const GemmArgs& a, cudaStream_t stream) {
    using P = Plan<MX, BN>;
    const int64_t nt = (w.rows + kRows - 1) / kRows;
    // 128-row scale blocks that a copy may touch: by experts the operand has room for any distribution
    const int64_t xblocks = a.p.experts ? (x.rows + 127 * std::min<int64_t>(a.p.experts, x.rows)) / 128 : (x.rows + 127) / 128;
    const int64_t mt = a.p.experts ? std::min<int64_t>(x.rows, x.rows / BN + std::min<int64_t>(a.p.experts, x.rows))
                                   : (x.rows + BN - 1) / BN;
    CUtensorMap maps[4];
    if (!encode_u32_map_pitch(&maps[0], w.codes, w.rows * w.matrices, K / 8, fp4_pitch(K), kStageWords, kRows, true) ||
        !encode_u32_map(&maps[1], w.scales, nt * w.matrices * a.chunks, 128, 128, P::kTiles) ||
        !encode_u32_map_pitch(&maps[2], x.codes, x.rows, K / 8, fp4_pitch(K), kStageWords, BN, true) ||
        !encode_u32_map(&maps[3], x.scales, xblocks * a.chunks, 128, 128, P::kTiles))
        return cudaErrorInvalidValue;
    return bf16 ? run_gemm<MX, BN, __nv_bfloat16>(maps, a, nt * mt, stream)
                : run_gemm<MX, BN, float>(maps, a, nt * mt, stream);
}

}  // namespace

cudaError_t launch_fp4_gemm(bool mx, const Fp4View& x, const Fp4View& w, int64_t K, const PlanView& p, float alpha,
                            const float* w_global, bool bf16, void* Y, int* err, bool /*static_weights*/,
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
    // activation rows of a tile: of the matrix, or of an expert on average
    const int64_t rows = p.experts ? (x.rows + p.experts - 1) / p.experts : x.rows;
    auto go = [&](auto m) {
        constexpr bool MX = decltype(m)::value;
        if (rows <= 64) return run_out<MX, 64>(bf16, x, w, K, a, stream);
        if (rows <= 128) return run_out<MX, 128>(bf16, x, w, K, a, stream);
        return run_out<MX, 256>(bf16, x, w, K, a, stream);
    };
    return mx ? go(std::true_type{}) : go(std::false_type{});
}

}  // namespace pnq
