// pnq_fp4_quantize.cu -- 4-bit microscaled operands: encode, decode, and the one-time layout of row-major
// weights (NVFP4: groups of 16 with E4M3 scales, MXFP4: groups of 32 with power-of-two scales; layout and
// definitions in include/pnq.h).
//
// All three are elementwise over K with a maximum per group: bound by HBM. A warp takes 256 consecutive
// elements of a row, 8 per lane (one 16-byte load of bf16); the lanes of a group take its maximum by
// shuffles, and each lane writes its 8 codes as one word. The scale words of four groups meet in one lane
// and leave as one word (they are neighbours in the tiled layout).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "pnq_device.cuh"
#include "pnq_internal.h"

namespace pnq {
namespace {

constexpr int kQThreads = 256;
constexpr int kItemElems = 256;  // elements of a row per warp and item

// Byte offset of the word of four groups (chunk c) of tiled row r.
__device__ __forceinline__ int64_t scale_word(int64_t r, int64_t c, int64_t chunks) {
    return ((r >> 7) * chunks + c) * 512 + ((r & 31) << 4) + (((r >> 5) & 3) << 2);
}

// Tiled row of row r (of all matrices' rows): every matrix of `rows` rows starts a 128-row block.
__device__ __forceinline__ int64_t tiled_row(int64_t r, int64_t rows, int64_t matrices) {
    if (matrices == 1) return r;
    const int64_t m = r / rows;
    return m * ((rows + 127) / 128 * 128) + (r - m * rows);
}

// Eight floats -> eight E2M1 codes, low nibble first: nearest, ties to even, saturating at 6.
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float (&t)[8]) {
    uint32_t d;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(d)
        : "f"(t[0]), "f"(t[1]), "f"(t[2]), "f"(t[3]), "f"(t[4]), "f"(t[5]), "f"(t[6]), "f"(t[7]));
    return d;
}

// The E4M3FN word nearest to v >= 0, ties to even, saturating at 448.
__device__ __forceinline__ uint32_t f32_to_e4m3(float v) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(0.0f), "f"(v));
    return d & 0xFFu;
}

template <class T, bool VEC>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
    if constexpr (sizeof(T) == 4) {
        if constexpr (VEC) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
            x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __ldg(p + i);
        }
    } else {
        uint32_t w[4];
        if constexpr (VEC) {
            const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
            w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
        } else {
            const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __ldg(h + 2 * i) | (static_cast<uint32_t>(__ldg(h + 2 * i + 1)) << 16);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

// Encodes this lane's 8 elements (live: the lane is inside the row): its scale word and its 8 codes. The
// group's lanes (2 for NVFP4, 4 for MXFP4) are neighbours.
template <bool MX>
__device__ __forceinline__ void encode8(float (&x)[8], bool live, float inv_g, uint32_t& word, uint32_t& codes) {
    uint32_t top = 0;  // largest |y| as bits: infinities and NaN sort above every finite value
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = live ? __fmul_rn(x[i], inv_g) : 0.0f;
        top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    if (MX) top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const bool finite = top < 0x7F800000u;
    const float amax = __uint_as_float(top);
    float t[8];
    bool zero = !finite;
    if (MX) {
        // floor(log2 amax) - 2 in the biased exponent; amax below 2^-125 (zero too) takes the least, 2^-127
        const int b = max(static_cast<int>(top >> 23) - 2, 0);
        word = finite ? static_cast<uint32_t>(b) : 255u;
        const float inv = __uint_as_float(static_cast<uint32_t>(254 - b) << 23);  // 2^(127 - b), exact
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = x[i] * inv;
    } else {
        word = finite ? f32_to_e4m3(__fdiv_rn(amax, 6.0f)) : 0x7Fu;
        zero |= word == 0;
        const float s = zero ? 1.0f : e4m3_to_f32(word);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = __fdiv_rn(x[i], s);
    }
    codes = zero ? 0u : f32x8_to_e2m1(t);
    if (!live) word = 0;
}

template <bool MX, class T, bool VEC, bool PLAN>
__global__ void __launch_bounds__(kQThreads) fp4_quantize_kernel(const T* __restrict__ X, int64_t ldx, int64_t rows,
                                                                 int64_t matrices, int K, float inv_g, PlanView p,
                                                                 uint8_t* __restrict__ codes, int64_t pitch,
                                                                 uint8_t* __restrict__ scales, int64_t chunks) {
    constexpr int kGroupLanes = MX ? 4 : 2;
    const int lane = threadIdx.x & 31;
    const int64_t per_row = (K + kItemElems - 1) / kItemElems, items = rows * matrices * per_row;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kQThreads / 32);
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * (kQThreads / 32) + (threadIdx.x >> 5); it < items; it += step) {
        const int64_t r = it / per_row;
        const int k = static_cast<int>(it - r * per_row) * kItemElems + 8 * lane;
        const bool live = k < K;
        float x[8];
        if (live) load8<T, VEC>(X + r * ldx + k, x);
        uint32_t word, c;
        encode8<MX>(x, live, inv_g, word, c);
        // the words of four groups in one, in every lane of the four
        word = lane % kGroupLanes == 0 ? word << (8 * (lane / kGroupLanes % 4)) : 0u;
        word |= __shfl_xor_sync(0xffffffffu, word, kGroupLanes);
        word |= __shfl_xor_sync(0xffffffffu, word, 2 * kGroupLanes);
        const int64_t chunk = k / (MX ? 128 : 64);
        const bool leads = lane % (4 * kGroupLanes) == 0 && chunk < chunks;
        if (!PLAN) {
            if (live) *reinterpret_cast<uint32_t*>(codes + r * pitch + k / 2) = c;
            if (leads) *reinterpret_cast<uint32_t*>(scales + scale_word(tiled_row(r, rows, matrices), chunk, chunks)) = word;
        } else {
            for (int j = 0; j < p.slots; ++j) {
                const int64_t at = __ldg(p.position + r * p.slots + j);
                if (at < 0) continue;
                if (live) *reinterpret_cast<uint32_t*>(codes + at * pitch + k / 2) = c;
                if (leads)
                    *reinterpret_cast<uint32_t*>(scales + scale_word(__ldg(p.scale_row + at), chunk, chunks)) = word;
            }
        }
    }
}

// A lane decodes 8 codes: out = fp32(e2m1 * s * g), the first product exact.
template <bool MX, class T, bool VEC>
__global__ void __launch_bounds__(kQThreads) fp4_dequantize_kernel(const uint8_t* __restrict__ codes, int64_t pitch,
                                                                   const uint8_t* __restrict__ scales, int64_t chunks,
                                                                   int64_t rows, int64_t matrices, int K, float g,
                                                                   const int32_t* __restrict__ scale_row,
                                                                   T* __restrict__ out) {
    const int64_t per_row = K / 8, items = rows * matrices * per_row;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kQThreads;
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * kQThreads + threadIdx.x; it < items; it += step) {
        const int64_t r = it / per_row;
        const int k = static_cast<int>(it - r * per_row) * 8;
        const int64_t sr = scale_row ? __ldg(scale_row + r) : tiled_row(r, rows, matrices);
        float v[8];
        if (sr >= 0) {
            const uint32_t c = __ldg(reinterpret_cast<const uint32_t*>(codes + r * pitch + k / 2));
            const int group = k / (MX ? 32 : 16);
            const uint32_t word = __ldg(scales + scale_word(sr, group >> 2, chunks) + (group & 3));
            const float s = !MX ? e4m3_to_f32(word)
                            : word == 255u ? __uint_as_float(0x7FC00000u)
                            : word == 0u   ? __uint_as_float(0x00400000u)  // 2^-127
                                           : __uint_as_float(word << 23);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(__fmul_rn(e2m1_to_f32((c >> (4 * i)) & 15u), s), g);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.0f;
        }
        T* o = out + r * static_cast<int64_t>(K) + k;
        if constexpr (sizeof(T) == 4) {
            if constexpr (VEC) {
                reinterpret_cast<float4*>(o)[0] = make_float4(v[0], v[1], v[2], v[3]);
                reinterpret_cast<float4*>(o)[1] = make_float4(v[4], v[5], v[6], v[7]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = v[i];
            }
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = f32x2_to_bf16x2(v[2 * i], v[2 * i + 1]);
            if constexpr (VEC) {
                *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
                uint16_t* h = reinterpret_cast<uint16_t*>(o);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
            }
        }
    }
}

// Row-major scale words -> tiles: a thread writes the word of four groups of one tiled row (rows and groups
// past the matrix: zeros).
__global__ void __launch_bounds__(kQThreads) fp4_tile_scales_kernel(const uint8_t* __restrict__ in, int64_t rows,
                                                                    int64_t matrices, int64_t groups, int64_t chunks,
                                                                    uint8_t* __restrict__ out) {
    const int64_t padded = (rows + 127) / 128 * 128, items = matrices * padded * chunks;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kQThreads;
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * kQThreads + threadIdx.x; it < items; it += step) {
        const int64_t r = it / chunks, c = it - r * chunks, m = r / padded, rr = r - m * padded;
        uint32_t word = 0;
        if (rr < rows) {
            const uint8_t* src = in + (m * rows + rr) * groups + 4 * c;
            const int64_t left = groups - 4 * c;
            for (int j = 0; j < 4; ++j)
                if (j < left) word |= static_cast<uint32_t>(__ldg(src + j)) << (8 * j);
        }
        *reinterpret_cast<uint32_t*>(out + scale_word(r, c, chunks)) = word;
    }
}

// Code rows of half bytes each -> rows of `pitch` bytes (K % 16 == 0: whole 8-byte words; the rows may start
// on any byte).
__global__ void __launch_bounds__(kQThreads) fp4_pitch_codes_kernel(const uint8_t* __restrict__ in, int64_t rows,
                                                                    int64_t half, int64_t pitch, uint8_t* __restrict__ out) {
    const int64_t words = pitch / 8, items = rows * words;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kQThreads;
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * kQThreads + threadIdx.x; it < items; it += step) {
        const int64_t r = it / words, b = 8 * (it - r * words);
        uint32_t lo = 0, hi = 0;
        if (b < half) {
            const uint8_t* src = in + r * half + b;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                lo |= static_cast<uint32_t>(__ldg(src + j)) << (8 * j);
                hi |= static_cast<uint32_t>(__ldg(src + 4 + j)) << (8 * j);
            }
        }
        *reinterpret_cast<uint2*>(out + r * pitch + b) = make_uint2(lo, hi);
    }
}

int item_grid(int64_t items, int per_cta) {
    return static_cast<int>(
        std::max<int64_t>(1, std::min<int64_t>((items + per_cta - 1) / per_cta, int64_t(device_sm_count()) * 8)));
}

template <bool MX, class T, bool VEC>
void run_quantize(const void* X, int64_t ldx, int64_t rows, int64_t K, int64_t matrices, float inv_g, const PlanView& p,
                  uint8_t* codes, uint8_t* scales, cudaStream_t stream) {
    const int64_t items = rows * matrices * ((K + kItemElems - 1) / kItemElems);
    const int grid = item_grid(items, kQThreads / 32);
    const int64_t pitch = fp4_pitch(K), chunks = fp4_chunks(MX, K);
    const T* x = static_cast<const T*>(X);
    if (p.experts)
        fp4_quantize_kernel<MX, T, VEC, true><<<grid, kQThreads, 0, stream>>>(x, ldx, rows, matrices, static_cast<int>(K),
                                                                              inv_g, p, codes, pitch, scales, chunks);
    else
        fp4_quantize_kernel<MX, T, VEC, false><<<grid, kQThreads, 0, stream>>>(x, ldx, rows, matrices, static_cast<int>(K),
                                                                               inv_g, p, codes, pitch, scales, chunks);
}

template <bool MX, class T>
void run_dequantize(const Fp4View& v, int64_t K, float g, const PlanView& p, void* out, cudaStream_t stream) {
    const int grid = item_grid(v.rows * v.matrices * (K / 8), kQThreads);
    const int64_t pitch = fp4_pitch(K), chunks = fp4_chunks(MX, K);
    const int32_t* sr = p.experts ? p.scale_row : nullptr;
    T* o = static_cast<T*>(out);
    // rows of K elements (a multiple of 8) keep the base's 16-byte alignment
    if (reinterpret_cast<uintptr_t>(out) % 16 == 0)
        fp4_dequantize_kernel<MX, T, true><<<grid, kQThreads, 0, stream>>>(v.codes, pitch, v.scales, chunks, v.rows,
                                                                           v.matrices, static_cast<int>(K), g, sr, o);
    else
        fp4_dequantize_kernel<MX, T, false><<<grid, kQThreads, 0, stream>>>(v.codes, pitch, v.scales, chunks, v.rows,
                                                                            v.matrices, static_cast<int>(K), g, sr, o);
}

}  // namespace

cudaError_t launch_fp4_quantize(bool mx, bool bf16, const void* X, int64_t ldx, int64_t rows, int64_t K,
                                int64_t matrices, float inv_g, const PlanView& p, uint8_t* codes, uint8_t* scales,
                                cudaStream_t stream) {
    const bool vec = reinterpret_cast<uintptr_t>(X) % 16 == 0 && ldx * (bf16 ? 2 : 4) % 16 == 0;
    auto go = [&](auto m) {
        constexpr bool MX = decltype(m)::value;
        if (bf16) {
            if (vec) run_quantize<MX, __nv_bfloat16, true>(X, ldx, rows, K, matrices, inv_g, p, codes, scales, stream);
            else run_quantize<MX, __nv_bfloat16, false>(X, ldx, rows, K, matrices, inv_g, p, codes, scales, stream);
        } else {
            if (vec) run_quantize<MX, float, true>(X, ldx, rows, K, matrices, inv_g, p, codes, scales, stream);
            else run_quantize<MX, float, false>(X, ldx, rows, K, matrices, inv_g, p, codes, scales, stream);
        }
    };
    if (mx) go(std::true_type{});
    else go(std::false_type{});
    return cudaGetLastError();
}

cudaError_t launch_fp4_dequantize(bool mx, const Fp4View& v, int64_t K, float g, const PlanView& p, bool bf16, void* out,
                                  cudaStream_t stream) {
    if (mx) {
        if (bf16) run_dequantize<true, __nv_bfloat16>(v, K, g, p, out, stream);
        else run_dequantize<true, float>(v, K, g, p, out, stream);
    } else {
        if (bf16) run_dequantize<false, __nv_bfloat16>(v, K, g, p, out, stream);
        else run_dequantize<false, float>(v, K, g, p, out, stream);
    }
    return cudaGetLastError();
}

cudaError_t launch_fp4_pack(bool mx, const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K,
                            int64_t matrices, uint8_t* codes_out, uint8_t* scales_out, cudaStream_t stream) {
    const int64_t chunks = fp4_chunks(mx, K), padded = (rows + 127) / 128 * 128;
    fp4_tile_scales_kernel<<<item_grid(matrices * padded * chunks, kQThreads), kQThreads, 0, stream>>>(
        scales, rows, matrices, K / (mx ? 32 : 16), chunks, scales_out);
    if (codes_out != codes) {
        const int64_t pitch = fp4_pitch(K);
        fp4_pitch_codes_kernel<<<item_grid(matrices * rows * (pitch / 8), kQThreads), kQThreads, 0, stream>>>(
            codes, matrices * rows, K / 2, pitch, codes_out);
    }
    return cudaGetLastError();
}

}  // namespace pnq
