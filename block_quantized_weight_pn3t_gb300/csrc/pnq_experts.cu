// pnq_experts.cu -- tokens sorted by expert and back: the plan (a stable counting sort), the gather of
// token rows into expert order, the weighted sum back, and the gradients of both.
//
// Every row kernel runs token by token: a token's row is read once and written to (or summed from) the
// sorted rows of its slots, so the bytes moved are the least possible: T rows on one side, T * k on
// the other. All of them are bound by HBM. Sums run in slot order in fp32: results do not depend on
// the launch.
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
// Counting sort of n expert ids by a cluster of C CTAs (C = 1..8), one launch:
//   1. every warp counts the experts of its own run of consecutive slots (shared-memory histogram per
//      warp);
//   2. a prefix over the CTA's warps, then over the cluster's CTAs (distributed shared memory), then
//      over the experts, turns the counts into each warp's first sorted row per expert;
//   3. every warp walks its run again, 32 slots at a time: lanes with the same expert rank themselves by
//      lane (match), so equal experts keep the order of their slots.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;

__device__ __forceinline__ int ld_dsmem_s32(uint32_t local_addr, uint32_t rank) {
    return __float_as_int(ld_dsmem_f32(local_addr, rank));
}

// Exclusive prefix sum of v over the block's threads (all kSortThreads take part).
__device__ __forceinline__ int block_exclusive_scan(int v, int* warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += u;
    }
    if (lane == 31) warp_sums[warp] = s;
    __syncthreads();
    if (warp == 0) {
        const int own = warp_sums[lane];
        int t = own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, t, d);
            if (lane >= d) t += u;
        }
        warp_sums[lane] = t - own;
    }
    __syncthreads();
    const int r = warp_sums[warp] + s - v;
    __syncthreads();
    return r;
}

__global__ void __launch_bounds__(kSortThreads, 1) expert_sort_kernel(const int32_t* __restrict__ ids, int n, PlanView p,
                                                                     int C) {
    extern __shared__ int sort_smem[];
    const int E = p.experts;
    int* hist = sort_smem;                 // [warps][E]
    int* total = hist + kSortWarps * E;    // [E] counts of this CTA
    int* first = total + E;                // [E] first sorted row of the expert
    int* block0 = first + E;               // [E] first scale block of the expert
    __shared__ int warp_sums[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = static_cast<int>(blockIdx.x);
    // this warp's run of slots: whole batches of 32, the same number for every warp of the cluster
    const int batches = (n + 31) / 32, per = (batches + C * kSortWarps - 1) / (C * kSortWarps);
    const int b0 = (rank * kSortWarps + warp) * per, b1 = min(batches, b0 + per);

    for (int i = tid; i < kSortWarps * E; i += kSortThreads) hist[i] = 0;
    __syncthreads();
    int* mine = hist + warp * E;
    for (int b = b0; b < b1; ++b) {
        const int i = 32 * b + lane;
        const int e = i < n ? __ldg(ids + i) : -1;
        if (e >= 0 && e < E) atomicAdd(mine + e, 1);
    }
    __syncthreads();
    int count = 0;  // of expert `tid` in this CTA (E <= kSortThreads)
    if (tid < E) {
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = hist[w * E + tid];
            hist[w * E + tid] = count;
            count += c;
        }
        total[tid] = count;
    }
    int before = 0, all = count;
    if (C > 1) {
        cluster_sync();
        if (tid < E) {
            all = 0;
            for (int c = 0; c < C; ++c) {
                const int v = ld_dsmem_s32(smem_addr(total + tid), static_cast<uint32_t>(c));
                if (c < rank) before += v;
                all += v;
            }
        }
    }
    const int off = block_exclusive_scan(all, warp_sums);
    const int blk = block_exclusive_scan((all + 127) / 128, warp_sums);
    if (tid < E) {
        first[tid] = off;
        block0[tid] = blk;
        for (int w = 0; w < kSortWarps; ++w) hist[w * E + tid] += off + before;
        if (rank == 0) {
            p.offsets[tid] = off;
            p.block_start[tid] = blk;
            if (tid == E - 1) {
                p.offsets[E] = off + all;
                p.block_start[E] = blk + (all + 127) / 128;
            }
        }
        if (tid == E - 1) warp_sums[0] = off + all;
    }
    __syncthreads();
    const int used = warp_sums[0];
    for (int b = b0; b < b1; ++b) {
        const int i = 32 * b + lane;
        int e = i < n ? __ldg(ids + i) : -1;
        if (e < 0 || e >= E) e = -1;
        const uint32_t same = __match_any_sync(0xffffffffu, e);
        const int r = __popc(same & ((1u << lane) - 1u));
        const int at = e >= 0 ? mine[e] + r : -1;
        __syncwarp();
        if (e >= 0 && r == 0) mine[e] += __popc(same);
        __syncwarp();
        if (i < n) p.position[i] = at;
        if (at >= 0) {
            p.order[at] = i;
            p.scale_row[at] = 128 * block0[e] + at - first[e];
        }
    }
    for (int i = used + rank * kSortThreads + tid; i < n; i += C * kSortThreads) {
        p.order[i] = -1;
        p.scale_row[i] = -1;
    }
    if (C > 1) cluster_sync();  // no CTA leaves while another still reads its counts
}

// ---- rows ---------------------------------------------------------------------------------------

// V consecutive elements of T: 16 bytes (or one element, for rows that are not 16-byte aligned).
template <class T, int V> struct Vec;
template <> struct Vec<float, 4> {
    using Raw = uint4;
    static __device__ __forceinline__ void to_f32(const uint4& r, float (&f)[4]) {
        f[0] = __uint_as_float(r.x), f[1] = __uint_as_float(r.y), f[2] = __uint_as_float(r.z), f[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ uint4 from_f32(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};
template <> struct Vec<float, 1> {
    using Raw = uint32_t;
    static __device__ __forceinline__ void to_f32(const uint32_t& r, float (&f)[1]) { f[0] = __uint_as_float(r); }
    static __device__ __forceinline__ uint32_t from_f32(const float (&f)[1]) { return __float_as_uint(f[0]); }
};
template <> struct Vec<__nv_bfloat16, 8> {
    using Raw = uint4;
    static __device__ __forceinline__ void to_f32(const uint4& r, float (&f)[8]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ uint4 from_f32(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = f32x2_to_bf16x2(f[2 * i], f[2 * i + 1]);
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <> struct Vec<__nv_bfloat16, 1> {
    using Raw = uint16_t;
    static __device__ __forceinline__ void to_f32(const uint16_t& r, float (&f)[1]) {
        f[0] = __uint_as_float(static_cast<uint32_t>(r) << 16);
    }
    static __device__ __forceinline__ uint16_t from_f32(const float (&f)[1]) {
        return static_cast<uint16_t>(f32x2_to_bf16x2(f[0], 0.0f));
    }
};

// Zero rows [used, n) of out, shared by all CTAs.
template <class Raw>
__device__ __forceinline__ void zero_tail(Raw* out, const PlanView& p, int64_t n, int64_t vecs) {
    const int64_t used = __ldg(p.offsets + p.experts);
    const int64_t count = (n - used) * vecs;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < count;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x)
        out[used * vecs + i] = Raw{};
}

constexpr int kRowThreads = 256;
constexpr int kSlotBatch = 8;  // slots whose rows are in flight together

// XS[position of each slot of t] = X[t].
template <class T, int V>
__global__ void __launch_bounds__(kRowThreads) expert_gather_kernel(const typename Vec<T, V>::Raw* __restrict__ X,
                                                                    int64_t vecs, PlanView p,
                                                                    typename Vec<T, V>::Raw* __restrict__ XS) {
    const int k = p.slots;
    for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
        const int32_t* pos = p.position + t * k;
        for (int64_t c = threadIdx.x; c < vecs; c += kRowThreads) {
            const auto v = __ldg(X + t * vecs + c);
            for (int j = 0; j < k; ++j) {
                const int64_t at = __ldg(pos + j);
                if (at >= 0) XS[at * vecs + c] = v;
            }
        }
    }
    zero_tail(XS, p, p.tokens * k, vecs);
}

// Y[t] = sum over slots of (weights or 1) * YS[position].
template <class T, int V, bool WEIGHTED>
__global__ void __launch_bounds__(kRowThreads) expert_combine_kernel(const typename Vec<T, V>::Raw* __restrict__ YS,
                                                                     int64_t vecs, PlanView p,
                                                                     const float* __restrict__ weights,
                                                                     typename Vec<T, V>::Raw* __restrict__ Y) {
    using Raw = typename Vec<T, V>::Raw;
    const int k = p.slots;
    for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
        const int32_t* pos = p.position + t * k;
        const float* wt = weights + t * k;
        for (int64_t c = threadIdx.x; c < vecs; c += kRowThreads) {
            float acc[V];
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = 0.0f;
            for (int j0 = 0; j0 < k; j0 += kSlotBatch) {
                Raw r[kSlotBatch];
                int64_t at[kSlotBatch];
#pragma unroll
                for (int j = 0; j < kSlotBatch; ++j) at[j] = j0 + j < k ? __ldg(pos + j0 + j) : -1;
#pragma unroll
                for (int j = 0; j < kSlotBatch; ++j)
                    if (at[j] >= 0) r[j] = __ldg(YS + at[j] * vecs + c);
#pragma unroll
                for (int j = 0; j < kSlotBatch; ++j) {
                    if (at[j] < 0) continue;
                    const float w = WEIGHTED ? __ldg(wt + j0 + j) : 1.0f;
                    float f[V];
                    Vec<T, V>::to_f32(r[j], f);
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[i] = WEIGHTED ? fmaf(w, f[i], acc[i]) : acc[i] + f[i];
                }
            }
            Y[t * vecs + c] = Vec<T, V>::from_f32(acc);
        }
    }
}

// dYS[position] = weights * dY[t], dWeights[t][j] = <dY[t], YS[position]>.
template <class T, int V>
__global__ void __launch_bounds__(kRowThreads) expert_combine_backward_kernel(
    const typename Vec<T, V>::Raw* __restrict__ dY, const typename Vec<T, V>::Raw* __restrict__ YS, int64_t vecs,
    PlanView p, const float* __restrict__ weights, typename Vec<T, V>::Raw* __restrict__ dYS,
    float* __restrict__ dWeights) {
    using Raw = typename Vec<T, V>::Raw;
    __shared__ float part[kRowThreads / 32][kSlotBatch];
    const int k = p.slots, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
        const int32_t* pos = p.position + t * k;
        for (int j0 = 0; j0 < k; j0 += kSlotBatch) {
            int64_t at[kSlotBatch];
            float w[kSlotBatch], dot[kSlotBatch];
#pragma unroll
            for (int j = 0; j < kSlotBatch; ++j) {
                at[j] = j0 + j < k ? __ldg(pos + j0 + j) : -1;
                w[j] = at[j] >= 0 ? __ldg(weights + t * k + j0 + j) : 0.0f;
                dot[j] = 0.0f;
            }
            for (int64_t c = threadIdx.x; c < vecs; c += kRowThreads) {
                float g[V];
                Vec<T, V>::to_f32(__ldg(dY + t * vecs + c), g);
                Raw r[kSlotBatch];
                if (dWeights) {
#pragma unroll
                    for (int j = 0; j < kSlotBatch; ++j)
                        if (at[j] >= 0) r[j] = __ldg(YS + at[j] * vecs + c);
                }
#pragma unroll
                for (int j = 0; j < kSlotBatch; ++j) {
                    if (at[j] < 0) continue;
                    float f[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) f[i] = w[j] * g[i];
                    dYS[at[j] * vecs + c] = Vec<T, V>::from_f32(f);
                    if (dWeights) {
                        Vec<T, V>::to_f32(r[j], f);
#pragma unroll
                        for (int i = 0; i < V; ++i) dot[j] = fmaf(g[i], f[i], dot[j]);
                    }
                }
            }
            if (dWeights) {
#pragma unroll
                for (int j = 0; j < kSlotBatch; ++j) {
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], d);
                    if (lane == 0) part[warp][j] = dot[j];
                }
                __syncthreads();
                if (threadIdx.x < kSlotBatch && j0 + static_cast<int>(threadIdx.x) < k) {
                    float s = 0.0f;
                    for (int q = 0; q < kRowThreads / 32; ++q) s += part[q][threadIdx.x];
                    dWeights[t * k + j0 + threadIdx.x] = s;
                }
                __syncthreads();
            }
        }
    }
    zero_tail(dYS, p, p.tokens * k, vecs);
}

int row_grid(int64_t tokens) {
    // enough CTAs to fill the device several times over; each then walks tokens with that stride
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(tokens, int64_t(device_sm_count()) * 32)));
}

bool vectorised(const void* a, const void* b, const void* c, int64_t row_bytes) {
    return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) | reinterpret_cast<uintptr_t>(c)) % 16 == 0) &&
           row_bytes % 16 == 0;
}

template <class T, int V>
const typename Vec<T, V>::Raw* raw(const void* p) {
    return static_cast<const typename Vec<T, V>::Raw*>(p);
}
template <class T, int V>
typename Vec<T, V>::Raw* raw(void* p) {
    return static_cast<typename Vec<T, V>::Raw*>(p);
}

template <class T, int V>
cudaError_t run_rows(ExpertOp op, const void* a, const void* b, int64_t D, const PlanView& p, const float* weights,
                     void* out, float* dw, cudaStream_t stream) {
    const int64_t vecs = D / V;
    const int grid = row_grid(p.tokens);
    switch (op) {
        case ExpertOp::Gather:
            expert_gather_kernel<T, V><<<grid, kRowThreads, 0, stream>>>(raw<T, V>(a), vecs, p, raw<T, V>(out));
            break;
        case ExpertOp::GatherBackward:
            expert_combine_kernel<T, V, false><<<grid, kRowThreads, 0, stream>>>(raw<T, V>(a), vecs, p, nullptr,
                                                                                 raw<T, V>(out));
            break;
        case ExpertOp::Combine:
            expert_combine_kernel<T, V, true><<<grid, kRowThreads, 0, stream>>>(raw<T, V>(a), vecs, p, weights,
                                                                                raw<T, V>(out));
            break;
        case ExpertOp::CombineBackward:
            expert_combine_backward_kernel<T, V><<<grid, kRowThreads, 0, stream>>>(raw<T, V>(a), raw<T, V>(b), vecs, p,
                                                                                   weights, raw<T, V>(out), dw);
            break;
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_expert_rows(ExpertOp op, bool bf16, const void* a, const void* b, int64_t D, const PlanView& p,
                               const float* weights, void* out, float* dweights, cudaStream_t stream) {
    if (bf16) {
        if (vectorised(a, b, out, D * 2)) return run_rows<__nv_bfloat16, 8>(op, a, b, D, p, weights, out, dweights, stream);
        return run_rows<__nv_bfloat16, 1>(op, a, b, D, p, weights, out, dweights, stream);
    }
    if (vectorised(a, b, out, D * 4)) return run_rows<float, 4>(op, a, b, D, p, weights, out, dweights, stream);
    return run_rows<float, 1>(op, a, b, D, p, weights, out, dweights, stream);
}

cudaError_t launch_expert_sort(const int32_t* ids, const PlanView& p, cudaStream_t stream) {
    const int n = static_cast<int>(p.tokens * p.slots);
    const int smem = (kSortWarps + 3) * p.experts * static_cast<int>(sizeof(int));
    // opt in to the most any number of experts needs (1024: 143,360 bytes), once per device
    cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(expert_sort_kernel), (kSortWarps + 3) * 1024 * 4);
    if (e != cudaSuccess) return e;
    // one CTA per 8192 slots, at most a portable cluster
    const int C = std::max(1, std::min(8, (n + 8191) / 8192));
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3(C);
    lc.blockDim = dim3(kSortThreads);
    lc.dynamicSmemBytes = smem;
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(C);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, expert_sort_kernel, ids, n, p, C);
}

}  // namespace pnq
