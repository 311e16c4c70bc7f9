// pnq_int8_gemm.cu -- products of 8-bit integer matrices with a scale per activation row and per weight row, sm_103a:
//   Y[m][n] = (sum_k X[m][k] W[n][k]) x_scale[m] w_scale[n]
// The sum is exact (32-bit integers), whatever kernel takes a call: results do not hang on the number of rows.
//
// pnq_int8_mma.cu takes more than eight activation rows; here are the fewer ones.
//
// Few rows (int8_rows_kernel): bound by HBM. The weights stream through registers, 512 contiguous bytes of a row at a time, and are multiplied by
// __dp4a (two multiply-adds of 2 x 16 bits or four of 8 are what the CUDA cores do on integers in one instruction); x waits in shared memory. One row
// of 17408 x 5120 takes 16.3 us (89 MB: 13.1 us at the copy rate), of 5120 x 17408 16.2 us; eight rows 22.8 and 24.8, where the
// multiplications begin to count. (Through mma.sync on codes widened to fp16, whose fragments want 16 rows of 64 bytes an
// access: 20.7 and 25.7 us for one row. Through the tensor cores of pnq_int8_mma.cu: 20.8 and 29.9.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "pnq_device.cuh"
#include "pnq_internal.h"

namespace pnq {
namespace {

constexpr int kRowThreads = 1024;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kGroup = 2;                 // weight rows that a warp takes together: a piece of x serves them all
constexpr int kBlockRows = 256;           // weight rows of a CTA whose sums are in shared memory at a time
constexpr int kRowSmem = 200 * 1024;      // x

struct RowArgs {
    const int8_t *X, *W;
    const float *x_scales, *w_scales;
    void* Y;
    int64_t ldx, ldw;
    int M, N, K;
};

__device__ __forceinline__ void store_product(float* y, float f) { *y = f; }
__device__ __forceinline__ void store_product(__nv_bfloat16* y, float f) { *y = __float2bfloat16_rn(f); }

// The sum as fp32 (one rounding), times both scales in turn.
__device__ __forceinline__ float scaled(int sum, float x_scale, float w_scale) {
    return __fmul_rn(__fmul_rn(__int2float_rn(sum), x_scale), w_scale);
}

// 16 bytes of a row from `at` on, bytes from K on as zeros. ALIGNED: rows start on 16 bytes.
template <bool ALIGNED>
__device__ __forceinline__ uint4 load16(const int8_t* row, int at, int K) {
    if (ALIGNED && at + 16 <= K) return ld_l2(reinterpret_cast<const uint4*>(row + at));
    if (at >= K) return make_uint4(0, 0, 0, 0);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (at + i < K) w[i / 4] |= ld_l2(reinterpret_cast<const uint8_t*>(row + at + i)) << (8 * (i % 4));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ int dot16(uint4 a, uint4 b, int c) {
    c = __dp4a(static_cast<int>(a.x), static_cast<int>(b.x), c);
    c = __dp4a(static_cast<int>(a.y), static_cast<int>(b.y), c);
    c = __dp4a(static_cast<int>(a.z), static_cast<int>(b.z), c);
    return __dp4a(static_cast<int>(a.w), static_cast<int>(b.w), c);
}

// CTA b: weight rows [N b / grid, N (b + 1) / grid) in groups of kGroup, all of x (MT rows at most). A step is 512 bytes of a group's rows, 16 a
// lane; the steps of all groups, one after the other, are dealt to the warps in equal runs, and a warp has kAhead of its steps in
// flight, across the groups' ends. A group's sums go into the CTA's by integer additions in shared memory.
template <int MT, bool ALIGNED, class T>
__global__ void __launch_bounds__(kRowThreads, 1) int8_rows_kernel(const RowArgs a) {
    extern __shared__ __align__(16) uint8_t xs[];
    __shared__ int sums[kBlockRows][MT];
    constexpr int kAhead = MT == 8 ? 2 : 4;  // 64 registers a thread: with eight rows' sums, fewer steps
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int K = a.K, per = (K + 511) / 512, pitch = per * 512;
    const int64_t N = a.N, b = blockIdx.x, g = gridDim.x;
    const int first = static_cast<int>(N * b / g), last = static_cast<int>(N * (b + 1) / g);
    griddep_begin();
    for (int r0 = first; r0 < last; r0 += kBlockRows) {
        const int rows = min(kBlockRows, last - r0), groups = (rows + kGroup - 1) / kGroup, steps = groups * per;
        const int s0 = steps * warp / kRowWarps, s1 = steps * (warp + 1) / kRowWarps;
        uint4 v[kAhead][kGroup];
        int next = s0, next_group = s0 / per, next_at = (s0 - next_group * per) * 512 + lane * 16;  // of the step to load
        auto load = [&](uint4 (&to)[kGroup]) {
            if (next < s1) {
#pragma unroll
                for (int r = 0; r < kGroup; ++r)
                    to[r] = load16<ALIGNED>(a.W + min(r0 + next_group * kGroup + r, last - 1) * a.ldw, next_at, K);
                ++next;
                next_at += 512;
                if (next_at >= pitch) next_at -= pitch, ++next_group;
            }
        };
#pragma unroll
        for (int p = 0; p < kAhead; ++p) load(v[p]);
        if (r0 == first) {
            const bool on16 = (reinterpret_cast<uintptr_t>(a.X) | static_cast<uintptr_t>(a.ldx)) % 16 == 0;
            for (int i = threadIdx.x; i < MT * (pitch / 16); i += kRowThreads) {
                const int m = i / (pitch / 16), at = (i - m * (pitch / 16)) * 16;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (m < a.M) v = on16 ? load16<true>(a.X + m * a.ldx, at, K) : load16<false>(a.X + m * a.ldx, at, K);
                *reinterpret_cast<uint4*>(xs + static_cast<int64_t>(m) * pitch + at) = v;
            }
        }
        for (int i = threadIdx.x; i < rows * MT; i += kRowThreads) (&sums[0][0])[i] = 0;
        __syncthreads();
        int group = s0 / per, at = (s0 - group * per) * 512 + lane * 16;
        int acc[kGroup][MT] = {};
        for (int s = s0; s < s1; s += kAhead) {
#pragma unroll
            for (int p = 0; p < kAhead; ++p) {
                if (s + p >= s1) break;
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const uint4 x = *reinterpret_cast<const uint4*>(xs + static_cast<int64_t>(m) * pitch + at);
#pragma unroll
                    for (int r = 0; r < kGroup; ++r) acc[r][m] = dot16(v[p][r], x, acc[r][m]);
                }
                load(v[p]);
                at += 512;
                if (at >= pitch || s + p + 1 == s1) {
#pragma unroll
                    for (int r = 0; r < kGroup; ++r)
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const int sum = __reduce_add_sync(0xffffffffu, acc[r][m]);
                            acc[r][m] = 0;
                            if (lane == 0 && group * kGroup + r < rows) atomicAdd(&sums[group * kGroup + r][m], sum);
                        }
                    if (at >= pitch) at -= pitch, ++group;
                }
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < rows * a.M; i += kRowThreads) {
            const int m = i / rows, r = i - m * rows, n = r0 + r;
            store_product(static_cast<T*>(a.Y) + static_cast<int64_t>(m) * a.N + n,
                          scaled(sums[r][m], ld_l2(a.x_scales + m), ld_l2(a.w_scales + n)));
        }
        __syncthreads();
    }
}

template <int MT, class T>
cudaError_t run_rows(const RowArgs& a, cudaStream_t stream) {
    const bool aligned = reinterpret_cast<uintptr_t>(a.W) % 16 == 0 && a.ldw % 16 == 0;
    auto kernel = aligned ? int8_rows_kernel<MT, true, T> : int8_rows_kernel<MT, false, T>;
    const int smem = MT * ((a.K + 511) / 512 * 512);
    const cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(kernel), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3(static_cast<unsigned>(std::min(device_sm_count(), (a.N + 3) / 4)));
    lc.blockDim = dim3(kRowThreads);
    lc.dynamicSmemBytes = static_cast<size_t>(smem);
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kernel, a);
}

template <class T>
cudaError_t run_rows(RowArgs a, int mt, cudaStream_t stream) {
    switch (mt) {
        case 8: return run_rows<8, T>(a, stream);
        case 4: return run_rows<4, T>(a, stream);
        case 2: return run_rows<2, T>(a, stream);
        default: return run_rows<1, T>(a, stream);
    }
}

// The activation rows (1, 2, 4 or 8) of the kernel that takes M of them with its x in shared memory; 0 where none does.
int row_tile(int64_t M, int64_t K) {
    for (int mt = 1; mt <= 8; mt *= 2)
        if (M <= mt) return mt * ((K + 511) / 512 * 512) <= kRowSmem ? mt : 0;
    return 0;
}

}  // namespace

uint64_t int8_gemm_scratch(int64_t M, const Int8View& w, int64_t K) { return M == 0 || row_tile(M, K) > 0 ? 0 : int8_mma_scratch(M, w, K); }

cudaError_t launch_int8_gemm(const Int8View& x, const Int8View& w, int64_t K, bool bf16, void* Y, void* scratch, int* err,
                             cudaStream_t stream) {
    const int mt = row_tile(x.rows, K);
    if (mt == 0) return launch_int8_mma(x, w, K, bf16, Y, scratch, err, stream);
    RowArgs a{};
    a.X = x.codes, a.ldx = x.ld, a.x_scales = x.scales;
    a.W = w.codes, a.ldw = w.ld, a.w_scales = w.scales;
    a.Y = Y;
    a.M = static_cast<int>(x.rows), a.N = static_cast<int>(w.rows), a.K = static_cast<int>(K);
    return bf16 ? run_rows<__nv_bfloat16>(a, mt, stream) : run_rows<float>(a, mt, stream);
}

}  // namespace pnq
