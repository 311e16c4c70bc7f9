// pnq_experts.cu -- tokens sorted by expert and back: the plan (a stable counting sort), the gather of
// token rows into expert order, the weighted sum back, and the gradients of both.
//
// Every row kernel runs token by token: a token's row is read once and written to (or summed from) the
// sorted rows of its slots, so the bytes moved are the least possible: T rows on one side, T * k on
// the other. All of them are bound by HBM. Sums over slots run in slot order in fp32: rows do not depend on
// the launch. The weights' gradients are sums over D in fp32, split over a warp's or a CTA's threads: in which pieces goes by the
// number of tokens and the alignment of the rows, so the same token's may differ in the last bits between batches
// (never between two calls with the same tensors). A thread adds D / 32 (a warp per token) or D / 256 terms (a CTA), then the
// threads' sums meet in 5 or 13 additions.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "pnq_device.cuh"
#include "pnq_internal.h"

namespace pnq {
namespace {

// ---- the plan -----------------------------------------------------------------------------------
//
// Counting sort of n expert ids by a cluster of C CTAs (C = 1..16) of W warps each:
//   1. every warp counts the experts of its own run of consecutive slots (shared-memory histogram per
//      warp);
//   2. a prefix over the CTA's warps, then over the cluster's CTAs (distributed shared memory), then
//      over the experts, turns the counts into each warp's first sorted row per expert;
//   3. every warp walks its run again, 32 slots at a time: lanes with the same expert rank themselves by
//      lane, so equal experts keep the order of their slots. The lanes with the same expert are found by a
//      ballot for each bit of its number (a match instruction costs an SM some 64 cycles: 131072 slots over 128
//      experts took 21 us with it).
// Many slots (C > 1): the sorted side's words (order, scale_row) are written by a second kernel on the whole device,
// from position: they scatter, one sector a word, and eight SMs would take longer over those stores than over all
// the rest (131072 slots over 128 experts: 20.5 us in one launch).
// The work is a chain of latencies, not bytes: a warp's ids are loaded kSortAhead batches at a time and, where one
// such load holds its whole run, once for both passes.
constexpr int kSortThreads = 1024;
constexpr int kSortAhead = 8;
constexpr int kSortCluster = 16;  // the largest a device may run; not a portable size, this is one device's code

__device__ __forceinline__ int ld_dsmem_s32(uint32_t local_addr, uint32_t rank) {
    return __float_as_int(ld_dsmem_f32(local_addr, rank));
}

// Exclusive prefix sum of v over the block's threads (all take part; warp_sums: one value per warp).
__device__ __forceinline__ unsigned long long block_exclusive_scan(unsigned long long v, unsigned long long* warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    unsigned long long s = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned long long u = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += u;
    }
    if (lane == 31) warp_sums[warp] = s;
    __syncthreads();
    unsigned long long before = lane < warp && lane < warps ? warp_sums[lane] : 0;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) before += __shfl_xor_sync(0xffffffffu, before, d);
    return before + s - v;
}

template <bool MANY>
__global__ void __launch_bounds__(kSortThreads, 1) expert_sort_kernel(const int32_t* __restrict__ ids, int n, PlanView p,
                                                                     int C, int per, int bits) {
    extern __shared__ int sort_smem[];
    griddep_begin();
    const int E = p.experts, W = static_cast<int>(blockDim.x) >> 5;
    int* hist = sort_smem;        // [W][E]
    int* total = hist + W * E;    // [E] counts of this CTA
    int* first = total + E;       // [E] first sorted row of the expert
    int* block0 = first + E;      // [E] first scale block of the expert
    int* base = block0 + E;       // [E] first sorted row of the expert's slots in this CTA
    __shared__ unsigned long long warp_sums[32];
    __shared__ int used_rows;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = static_cast<int>(blockDim.x);
    const int rank = static_cast<int>(blockIdx.x);
    // this warp's run of slots: `per` whole batches of 32
    const int batches = (n + 31) / 32;
    const int b0 = min(batches, (rank * W + warp) * per), b1 = min(batches, b0 + per);

    int e[kSortAhead];
    auto load = [&](int b) {  // the experts of batches b .. b + kSortAhead - 1, -1 where there is none
#pragma unroll
        for (int j = 0; j < kSortAhead; ++j) {
            const int i = 32 * (b + j) + lane;
            e[j] = b + j < b1 && i < n ? ld_l2(ids + i) : -1;
        }
#pragma unroll
        for (int j = 0; j < kSortAhead; ++j)
            if (static_cast<unsigned>(e[j]) >= static_cast<unsigned>(E)) e[j] = -1;
    };
    load(b0);
    for (int i = tid; i < W * E; i += threads) hist[i] = 0;
    __syncthreads();
    int* mine = hist + warp * E;
    for (int b = b0; b < b1; b += kSortAhead) {
        if (b > b0) load(b);
#pragma unroll
        for (int j = 0; j < kSortAhead; ++j)
            if (e[j] >= 0) atomicAdd(mine + e[j], 1);
    }
    __syncthreads();
    int count = 0;  // of expert `tid` in this CTA (E <= threads)
    if (tid < E) {
#pragma unroll 8
        for (int w = 0; w < W; ++w) {
            const int c = hist[w * E + tid];
            hist[w * E + tid] = count;
            count += c;
        }
        total[tid] = count;
    }
    int before = 0, all = count;
    if (MANY) {
        cluster_sync();
        if (tid < E) {
            all = 0;
            int v[kSortCluster];  // all the loads in flight together: one takes some 0.25 us
#pragma unroll
            for (int c = 0; c < kSortCluster; ++c) v[c] = c < C ? ld_dsmem_s32(smem_addr(total + tid), static_cast<uint32_t>(c)) : 0;
#pragma unroll
            for (int c = 0; c < kSortCluster; ++c) {
                if (c < rank) before += v[c];
                all += v[c];
            }
        }
    }
    if (MANY) cluster_arrive();  // this CTA has read the counts (cluster_wait at the end: no CTA leaves before all have)
    // rows and 128-row blocks before expert tid, in one scan
    const unsigned long long pre =
        block_exclusive_scan((static_cast<unsigned long long>((all + 127) / 128) << 32) | static_cast<unsigned>(all), warp_sums);
    const int off = static_cast<int>(pre & 0xffffffffu), blk = static_cast<int>(pre >> 32);
    if (tid < E) {
        base[tid] = off + before;  // this CTA's first sorted row of the expert
        first[tid] = off;
        block0[tid] = blk;
        if (rank == 0) {
            p.offsets[tid] = off;
            p.block_start[tid] = blk;
            if (tid == E - 1) {
                p.offsets[E] = off + all;
                p.block_start[E] = blk + (all + 127) / 128;
            }
        }
        if (tid == E - 1) used_rows = off + all;
    }
    __syncthreads();
    if (b1 - b0 > kSortAhead) load(b0);
    for (int b = b0; b < b1; b += kSortAhead) {
        if (b > b0) load(b);
        const int most = min(kSortAhead, b1 - b);
#pragma unroll
        for (int j = 0; j < kSortAhead; ++j) {
            if (j >= most) break;
            const int i = 32 * (b + j) + lane;
            const uint32_t key = e[j] >= 0 ? static_cast<uint32_t>(e[j]) : static_cast<uint32_t>(E);
            uint32_t same = 0xffffffffu;
            for (int q = 0; q < bits; ++q) {
                const bool one = (key >> q) & 1u;
                const uint32_t ones = __ballot_sync(0xffffffffu, one);
                same &= one ? ones : ~ones;
            }
            const int r = __popc(same & ((1u << lane) - 1u));
            const int at = e[j] >= 0 ? mine[e[j]] + base[e[j]] + r : -1;
            __syncwarp();
            if (e[j] >= 0 && r == 0) mine[e[j]] += __popc(same);
            __syncwarp();
            if (i < n) p.position[i] = at;
            if (!MANY && at >= 0) {
                p.order[at] = i;
                p.scale_row[at] = 128 * block0[e[j]] + at - first[e[j]];
            }
        }
    }
    if (!MANY)
        for (int i = used_rows + tid; i < n; i += threads) {
            p.order[i] = -1;
            p.scale_row[i] = -1;
        }
    if (MANY) cluster_wait();
}

// order and scale_row from position (many slots).
__global__ void __launch_bounds__(256) expert_order_kernel(const int32_t* __restrict__ ids, int n, PlanView p) {
    __shared__ int shift[1024];  // of each expert: from sorted row to row in the tiled scales
    griddep_begin();
    for (int e = threadIdx.x; e < p.experts; e += 256) shift[e] = 128 * ld_l2(p.block_start + e) - ld_l2(p.offsets + e);
    __syncthreads();
    const int used = ld_l2(p.offsets + p.experts);
    for (int i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) {
        const int at = ld_l2(p.position + i);
        if (at >= 0) {
            const int e = ld_l2(ids + i);
            p.order[at] = i;
            p.scale_row[at] = at + shift[e];
        }
        if (i >= used) {
            p.order[i] = -1;
            p.scale_row[i] = -1;
        }
    }
}

// ---- rows ---------------------------------------------------------------------------------------

// V consecutive elements of T in one access of 16 bytes, or of the 8, 4 or 2 that the rows' alignment allows; kSteps
// such accesses a thread are in flight together, so that rows of any length keep the loads' bytes up.
template <int BYTES> struct RawOf;
template <> struct RawOf<16> { using type = uint4; };
template <> struct RawOf<8> { using type = uint2; };
template <> struct RawOf<4> { using type = uint32_t; };
template <> struct RawOf<2> { using type = uint16_t; };

template <class T, int V>
struct Vec {
    static constexpr int kBytes = V * static_cast<int>(sizeof(T)), kWords = kBytes < 4 ? 1 : kBytes / 4;
    static constexpr int kSteps = kBytes == 16 ? 1 : kBytes == 8 ? 2 : 4;
    using Raw = typename RawOf<kBytes>::type;
    static __device__ __forceinline__ void words(const Raw& r, uint32_t (&w)[kWords]) {
        if constexpr (kBytes == 16) w[0] = r.x, w[1] = r.y, w[2] = r.z, w[3] = r.w;
        else if constexpr (kBytes == 8) w[0] = r.x, w[1] = r.y;
        else w[0] = r;
    }
    static __device__ __forceinline__ void to_f32(const Raw& r, float (&f)[V]) {
        uint32_t w[kWords];
        words(r, w);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (sizeof(T) == 4) f[i] = __uint_as_float(w[i]);
            else f[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
        }
    }
    static __device__ __forceinline__ Raw from_f32(const float (&f)[V]) {
        uint32_t w[kWords];
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < V; ++i) w[i] = __float_as_uint(f[i]);
        } else if constexpr (V == 1) {
            w[0] = f32x2_to_bf16x2(f[0], 0.0f);
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) w[i] = f32x2_to_bf16x2(f[2 * i], f[2 * i + 1]);
        }
        if constexpr (kBytes == 16) return make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (kBytes == 8) return make_uint2(w[0], w[1]);
        else return static_cast<Raw>(w[0]);
    }
};

// Zero rows [used, n) of out, shared by all CTAs.
template <class Raw>
__device__ __forceinline__ void zero_tail(Raw* out, const PlanView& p, int64_t n, int64_t vecs) {
    const int64_t used = max(0, ld_l2(p.offsets + p.experts));
    const int64_t count = (n - used) * vecs;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < count;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x)
        out[used * vecs + i] = Raw{};
}

// A team of TEAM threads takes a token: a warp where there are many tokens (no block-wide step, and the loads of many
// tokens in flight), a CTA where there are few.
constexpr int kRowThreads = 256;
constexpr int kSlotBatch = 8;  // slots whose rows are in flight together

template <int TEAM>
struct Team {
    static constexpr int kPerCta = kRowThreads / TEAM;
    static __device__ __forceinline__ int thread() { return static_cast<int>(threadIdx.x) % TEAM; }
    static __device__ __forceinline__ int64_t first() {
        return static_cast<int64_t>(blockIdx.x) * kPerCta + static_cast<int>(threadIdx.x) / TEAM;
    }
    static __device__ __forceinline__ int64_t step() { return static_cast<int64_t>(gridDim.x) * kPerCta; }
};

// Sorted rows and weights (or ones) of slots j0 .. j0 + kSlotBatch - 1 of token t, in every lane of the warp; -1 where there is
// none. Lane j loads slot j's: one request for all of them.
__device__ __forceinline__ void load_slots(const PlanView& p, const float* weights, int64_t t, int j0, int (&at)[kSlotBatch],
                                           float (&w)[kSlotBatch]) {
    const int k = p.slots, j = j0 + (static_cast<int>(threadIdx.x) & 31);
    int mine = -1;
    float weight = 1.0f;
    if (j < min(k, j0 + kSlotBatch)) {
        mine = plan_index(ld_l2(p.position + t * k + j), p.rows);
        if (weights) weight = ld_l2(weights + t * k + j);
    }
#pragma unroll
    for (int i = 0; i < kSlotBatch; ++i) {
        at[i] = __shfl_sync(0xffffffffu, mine, i);
        w[i] = __shfl_sync(0xffffffffu, weight, i);
    }
}

// XS[position of each slot of t] = X[t].
template <class T, int V, int TEAM>
__global__ void __launch_bounds__(kRowThreads) expert_gather_kernel(const typename Vec<T, V>::Raw* __restrict__ X,
                                                                    int64_t vecs, PlanView p,
                                                                    typename Vec<T, V>::Raw* __restrict__ XS) {
    constexpr int U = Vec<T, V>::kSteps;
    griddep_begin();
    for (int64_t t = Team<TEAM>::first(); t < p.tokens; t += Team<TEAM>::step()) {
        for (int j0 = 0; j0 < p.slots; j0 += kSlotBatch) {
            int at[kSlotBatch];
            float w[kSlotBatch];
            load_slots(p, nullptr, t, j0, at, w);
            for (int64_t c = Team<TEAM>::thread(); c < vecs; c += TEAM * U) {
                typename Vec<T, V>::Raw v[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c + u * TEAM < vecs) v[u] = ld_l2(X + t * vecs + c + u * TEAM);
#pragma unroll
                for (int j = 0; j < kSlotBatch; ++j) {
                    if (at[j] < 0) continue;
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (c + u * TEAM < vecs) XS[at[j] * vecs + c + u * TEAM] = v[u];
                }
            }
        }
    }
    zero_tail(XS, p, p.tokens * p.slots, vecs);
}

// Y[t] = sum over slots of (weights, or 1 where they are null) * YS[position].
// bf16 by 16 bytes: 3 CTAs an SM, which its 80 registers give and 85 would not.
template <class T, int V, int TEAM>
__global__ void __launch_bounds__(kRowThreads, sizeof(T) == 2 && V == 8 ? 3 : 0) expert_combine_kernel(const typename Vec<T, V>::Raw* __restrict__ YS,
                                                                     int64_t vecs, PlanView p,
                                                                     const float* __restrict__ weights,
                                                                     typename Vec<T, V>::Raw* __restrict__ Y) {
    using Raw = typename Vec<T, V>::Raw;
    constexpr int U = Vec<T, V>::kSteps;
    const int k = p.slots;
    griddep_begin();
    for (int64_t t = Team<TEAM>::first(); t < p.tokens; t += Team<TEAM>::step()) {
        int at[kSlotBatch];
        float w[kSlotBatch];
        load_slots(p, weights, t, 0, at, w);
        // whole warps take the columns' steps together (the slots are loaded again in each where there are over kSlotBatch)
        for (int64_t c0 = Team<TEAM>::thread() & ~31; c0 < vecs; c0 += TEAM * U) {
            const int64_t c = c0 + (static_cast<int>(threadIdx.x) & 31);
            float acc[U][V];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < V; ++i) acc[u][i] = 0.0f;
            for (int j0 = 0; j0 < k; j0 += kSlotBatch) {
                if (k > kSlotBatch) load_slots(p, weights, t, j0, at, w);
                Raw r[kSlotBatch][U];
#pragma unroll
                for (int j = 0; j < kSlotBatch; ++j)
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (at[j] >= 0 && c + u * TEAM < vecs) r[j][u] = ld_l2(YS + at[j] * vecs + c + u * TEAM);
#pragma unroll
                for (int j = 0; j < kSlotBatch; ++j) {
                    if (at[j] < 0) continue;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        if (c + u * TEAM >= vecs) continue;
                        float f[V];
                        Vec<T, V>::to_f32(r[j][u], f);
#pragma unroll
                        for (int i = 0; i < V; ++i) acc[u][i] = fmaf(w[j], f[i], acc[u][i]);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c + u * TEAM < vecs) Y[t * vecs + c + u * TEAM] = Vec<T, V>::from_f32(acc[u]);
        }
    }
}

// dYS[position] = weights * dY[t], dWeights[t][j] = <dY[t], YS[position]>. 2 CTAs an SM: 128 registers, and 28 to 68 bytes a
// thread spilled (16384 x 8 rows of 2048 bf16, 40 bytes: 183 us = 6.2 TB/s all the same).
template <class T, int V, int TEAM>
__global__ void __launch_bounds__(kRowThreads, 2) expert_combine_backward_kernel(
    const typename Vec<T, V>::Raw* __restrict__ dY, const typename Vec<T, V>::Raw* __restrict__ YS, int64_t vecs,
    PlanView p, const float* __restrict__ weights, typename Vec<T, V>::Raw* __restrict__ dYS,
    float* __restrict__ dWeights) {
    using Raw = typename Vec<T, V>::Raw;
    constexpr int U = Vec<T, V>::kSteps;
    __shared__ float part[kRowThreads / 32][kSlotBatch];
    const int k = p.slots, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    griddep_begin();
    for (int64_t t = Team<TEAM>::first(); t < p.tokens; t += Team<TEAM>::step()) {
        for (int j0 = 0; j0 < k; j0 += kSlotBatch) {
            int at[kSlotBatch];
            float w[kSlotBatch], dot[kSlotBatch];
            load_slots(p, weights, t, j0, at, w);
#pragma unroll
            for (int j = 0; j < kSlotBatch; ++j) dot[j] = 0.0f;
            for (int64_t c = Team<TEAM>::thread(); c < vecs; c += TEAM * U) {
                Raw gr[U], r[kSlotBatch][U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c + u * TEAM < vecs) gr[u] = ld_l2(dY + t * vecs + c + u * TEAM);
                if (dWeights) {
#pragma unroll
                    for (int j = 0; j < kSlotBatch; ++j)
#pragma unroll
                        for (int u = 0; u < U; ++u)
                            if (at[j] >= 0 && c + u * TEAM < vecs) r[j][u] = ld_l2(YS + at[j] * vecs + c + u * TEAM);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (c + u * TEAM >= vecs) continue;
                    float g[V];
                    Vec<T, V>::to_f32(gr[u], g);
#pragma unroll
                    for (int j = 0; j < kSlotBatch; ++j) {
                        if (at[j] < 0) continue;
                        float f[V];
#pragma unroll
                        for (int i = 0; i < V; ++i) f[i] = w[j] * g[i];
                        dYS[at[j] * vecs + c + u * TEAM] = Vec<T, V>::from_f32(f);
                        if (dWeights) {
                            Vec<T, V>::to_f32(r[j][u], f);
#pragma unroll
                            for (int i = 0; i < V; ++i) dot[j] = fmaf(g[i], f[i], dot[j]);
                        }
                    }
                }
            }
            if (dWeights) {
                float mine = 0.0f;  // lane j: the warp's sum of slot j0 + j
#pragma unroll
                for (int j = 0; j < kSlotBatch; ++j) {
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], d);
                    if (lane == j) mine = dot[j];
                }
                if (TEAM == 32) {
                    if (lane < kSlotBatch && j0 + lane < k) dWeights[t * k + j0 + lane] = mine;
                } else {
                    if (lane < kSlotBatch) part[warp][lane] = mine;
                    __syncthreads();
                    if (threadIdx.x < kSlotBatch && j0 + static_cast<int>(threadIdx.x) < k) {
                        float s = 0.0f;
                        for (int q = 0; q < TEAM / 32; ++q) s += part[q][threadIdx.x];
                        dWeights[t * k + j0 + threadIdx.x] = s;
                    }
                    __syncthreads();
                }
            }
        }
    }
    zero_tail(dYS, p, p.tokens * k, vecs);
}

// Bytes of the widest access that the tensors' addresses and the rows' length allow (16 at most).
int access_bytes(const void* a, const void* b, const void* c, int64_t row_bytes) {
    const uintptr_t all = reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) | reinterpret_cast<uintptr_t>(c) |
                          static_cast<uintptr_t>(row_bytes) | 16u;
    return static_cast<int>(all & (~all + 1));
}

template <class T, int V>
const typename Vec<T, V>::Raw* raw(const void* p) {
    return static_cast<const typename Vec<T, V>::Raw*>(p);
}
template <class T, int V>
typename Vec<T, V>::Raw* raw(void* p) {
    return static_cast<typename Vec<T, V>::Raw*>(p);
}

template <class T, int V, int TEAM>
cudaError_t run_rows(ExpertOp op, const void* a, const void* b, int64_t D, const PlanView& p, const float* weights,
                     void* out, float* dw, cudaStream_t stream) {
    const int64_t vecs = D / V, per = Team<TEAM>::kPerCta;
    // enough CTAs to fill the device several times over; each then walks tokens with that stride
    const int grid = static_cast<int>(
        std::max<int64_t>(1, std::min<int64_t>((p.tokens + per - 1) / per, int64_t(device_sm_count()) * 32)));
    if (op == ExpertOp::CombineBackward)
        return launch_dependent(expert_combine_backward_kernel<T, V, TEAM>, grid, kRowThreads, stream, raw<T, V>(a), raw<T, V>(b), vecs,
                                p, weights, raw<T, V>(out), dw);
    if (op == ExpertOp::Gather)
        return launch_dependent(expert_gather_kernel<T, V, TEAM>, grid, kRowThreads, stream, raw<T, V>(a), vecs, p, raw<T, V>(out));
    return launch_dependent(expert_combine_kernel<T, V, TEAM>, grid, kRowThreads, stream, raw<T, V>(a), vecs, p, weights,
                            raw<T, V>(out));
}

template <class T, int V>
cudaError_t run_rows(ExpertOp op, const void* a, const void* b, int64_t D, const PlanView& p, const float* weights,
                     void* out, float* dw, cudaStream_t stream) {
    // A warp per token where the tokens give every SM 16 warps (16384 tokens of 2048 bf16, 8 slots: combine 94 us = 6.4 TB/s,
    // its gradients 183 = 6.2 TB/s; a CTA per token took 13 to 15 percent longer), a CTA where they are few (5 tokens of 2048
    // fp32, 4 slots: combine 8.1 us by warps and 2.0 by CTAs). The gather of rows of 4096 bytes or more keeps the CTA (93 us
    // against 96).
    // Between them, rounds of the device times the steps of a token in each (a step is about half of what a round costs
    // besides), with the 2 CTAs of 256 per SM that the gradients have room for and the 3 of the others. By warps and by CTAs,
    // 2300 tokens of 101 bf16, 4 slots: gather 2.4 and 6.5 us, combine 2.2 and 11.5, gradients 3.7 and 17.8; 400 of 2048,
    // 8 slots: 5.9 and 3.9, 7.1 and 2.8, 11.9 and 7.4.
    // Larger CTAs for few tokens give nothing now that a thread has several narrow accesses in flight (7 tokens of 1999 fp32 by
    // 256 threads: combine 2.8 us, gradients 3.9; by 1024 and 512: 2.9 and 3.8; 300 of 5120 bf16: 5.5 and 11, 9 and 14).
    // Rows that are not on 16 bytes (D = 3924 bf16, 3194 tokens, 4 slots): gather 25.6 us, combine 40; 34 and 77 where D
    // is odd and an access two bytes; with one access of one element a thread the two took some three times as long. Accesses
    // of 16 bytes shifted into place by shuffles and funnel shifts are no better: 73 and 76 us at any D.
    const int64_t vecs = D / V, sms = device_sm_count();
    const int64_t round = sms * (op == ExpertOp::CombineBackward ? 2 : 3);  // CTAs that run at a time
    auto rounds = [&](int64_t per_cta, int64_t threads) {
        const int64_t step = threads * Vec<T, V>::kSteps;
        return (p.tokens + round * per_cta - 1) / (round * per_cta) * (2 + (vecs + step - 1) / step);
    };
    const bool warps = p.tokens >= sms * 16 || (p.tokens > sms * 2 && rounds(kRowThreads / 32, 32) <= rounds(1, kRowThreads));
    if (warps && (op != ExpertOp::Gather || vecs * Vec<T, V>::kBytes < 4096))
        return run_rows<T, V, 32>(op, a, b, D, p, weights, out, dw, stream);
    return run_rows<T, V, kRowThreads>(op, a, b, D, p, weights, out, dw, stream);
}

}  // namespace

cudaError_t launch_expert_rows(ExpertOp op, bool bf16, const void* a, const void* b, int64_t D, const PlanView& p,
                               const float* weights, void* out, float* dweights, cudaStream_t stream) {
    switch (access_bytes(a, b, out, D * (bf16 ? 2 : 4))) {
        case 16:
            return bf16 ? run_rows<__nv_bfloat16, 8>(op, a, b, D, p, weights, out, dweights, stream)
                        : run_rows<float, 4>(op, a, b, D, p, weights, out, dweights, stream);
        case 8:
            return bf16 ? run_rows<__nv_bfloat16, 4>(op, a, b, D, p, weights, out, dweights, stream)
                        : run_rows<float, 2>(op, a, b, D, p, weights, out, dweights, stream);
        case 4:
            return bf16 ? run_rows<__nv_bfloat16, 2>(op, a, b, D, p, weights, out, dweights, stream)
                        : run_rows<float, 1>(op, a, b, D, p, weights, out, dweights, stream);
        default:
            return run_rows<__nv_bfloat16, 1>(op, a, b, D, p, weights, out, dweights, stream);
    }
}

cudaError_t launch_expert_sort(const int32_t* ids, const PlanView& p, cudaStream_t stream) {
    const int n = static_cast<int>(p.tokens * p.slots), batches = (n + 31) / 32;
    // Few slots: one warp per batch of 32 and a thread per expert. Many: CTAs of 32 warps, up to the largest cluster,
    // before a warp takes a second batch.
    const int C = std::max(1, std::min(kSortCluster, (batches + 31) / 32));
    const int warps = C > 1 ? 32 : std::max({1, batches, (p.experts + 31) / 32});
    const int per = std::max(1, (batches + C * warps - 1) / (C * warps));
    const int smem = (warps + 4) * p.experts * static_cast<int>(sizeof(int));
    const auto kern = C > 1 ? expert_sort_kernel<true> : expert_sort_kernel<false>;
    // opt in to the most any number of experts needs (1024: 147,456 bytes), once per device
    cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(kern), (kSortThreads / 32 + 4) * 1024 * 4);
    if (e == cudaSuccess && C > 8) e = opt_in_cluster(reinterpret_cast<const void*>(kern));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3(C);
    lc.blockDim = dim3(32 * warps);
    lc.dynamicSmemBytes = smem;
    lc.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(C);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 2;
    int bits = 1;  // of the numbers 0 .. experts (the last: a dropped slot)
    while ((p.experts >> bits) != 0) ++bits;
    e = cudaLaunchKernelEx(&lc, kern, ids, n, p, C, per, bits);
    if (e != cudaSuccess || C == 1) return e;
    const int grid = std::min((n + 255) / 256, device_sm_count() * 8);
    return launch_dependent(expert_order_kernel, grid, 256, stream, ids, n, p);
}

}  // namespace pnq
