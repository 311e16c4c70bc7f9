// pnq_fp4_quantize.cu -- 4-bit microscaled operands: encode, decode, and the one-time layout of row-major
// weights (NVFP4: groups of 16 with E4M3 scales, MXFP4: groups of 32 with power-of-two scales; layout and
// definitions in include/pnq.h).
//
// All three are elementwise over K with a maximum per group: bound by HBM. A warp takes 1024 consecutive
// elements of a row in four steps of 256, all four loads in flight at once (few rows: one step per warp, so
// that more warps share them).
//   encode: 8 elements per lane (one 16-byte load of bf16); the lanes of a group take its maximum by shuffles; with four
//           steps the lanes of a four exchange their codes and write 16 bytes each; the scale words of four groups are
//           neighbours in the tiled layout and leave as one word.
//   decode: a lane loads the word of 8 codes, which is a store of 16 bytes of bf16. For fp32 the warp exchanges the words so
//           that lane l writes elements 4 l .. 4 l + 3 of 128: every store covers 512 contiguous bytes (with a quarter of the CTAs
//           that a launch has now, 8191 x 5152 took 34.3 us so and 36.7 by lanes that wrote 32 bytes each; now 29.9), and
//           for a bf16 output that is not on 16 bytes too.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "pnq_device.cuh"
#include "pnq_internal.h"

namespace pnq {
namespace {

constexpr int kQThreads = 128;

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

__device__ __forceinline__ __half2 u32_as_half2(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }

// Value of an E4M3FN word with its sign bit clear (a positive scale, or NaN).
__device__ __forceinline__ float e4m3_bits_to_f32(uint32_t word) {
    return __low2float(u32_as_half2(e4m3x2_to_f16x2(word)));
}

// Eight consecutive elements as loaded: four words of two bf16, or eight floats.
template <class T>
struct Eight {
    static constexpr int kWords = 2 * static_cast<int>(sizeof(T));
    uint32_t w[kWords];
};

// By one load, 8 * sizeof(T) bytes aligned.
template <class T>
__device__ __forceinline__ void load8(const T* p, Eight<T>& x) {
    if constexpr (sizeof(T) == 4) {
        float f[8];
        ld_l2_f32x8(p, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) x.w[i] = __float_as_uint(f[i]);
    } else {
        const uint4 a = ld_l2(reinterpret_cast<const uint4*>(p));
        x.w[0] = a.x, x.w[1] = a.y, x.w[2] = a.z, x.w[3] = a.w;
    }
}

// Rows of any other alignment: a lane loads elements lane + 32 i, so that a load of the warp reads one run of addresses and
// not 32 (8191 x 5152 fp32 to NVFP4, row stride 5153: 72.5 us by lanes of eight elements each, 35.4 so; bf16 41.1 and 34.2), and
// the warp turns them through shared memory.
__device__ __forceinline__ void pack8(const uint32_t (&e)[8], Eight<float>& x) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x.w[i] = e[i];
}
__device__ __forceinline__ void pack8(const uint16_t (&e)[8], Eight<__nv_bfloat16>& x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x.w[i] = e[2 * i] | (static_cast<uint32_t>(e[2 * i + 1]) << 16);
}
__device__ __forceinline__ void turn8(Eight<float>& x, uint32_t* warp, int lane) {
#pragma unroll
    for (int i = 0; i < 8; ++i) warp[32 * i + lane] = x.w[i];
    __syncwarp();
    const uint4 a = reinterpret_cast<const uint4*>(warp)[2 * lane], b = reinterpret_cast<const uint4*>(warp)[2 * lane + 1];
    __syncwarp();
    x.w[0] = a.x, x.w[1] = a.y, x.w[2] = a.z, x.w[3] = a.w;
    x.w[4] = b.x, x.w[5] = b.y, x.w[6] = b.z, x.w[7] = b.w;
}
__device__ __forceinline__ void turn8(Eight<__nv_bfloat16>& x, uint16_t* warp, int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        warp[64 * i + lane] = static_cast<uint16_t>(x.w[i]);
        warp[64 * i + 32 + lane] = static_cast<uint16_t>(x.w[i] >> 16);
    }
    __syncwarp();
    const uint4 a = reinterpret_cast<const uint4*>(warp)[lane];
    __syncwarp();
    x.w[0] = a.x, x.w[1] = a.y, x.w[2] = a.z, x.w[3] = a.w;
}

// Largest magnitude of the eight; NaN where one of them is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
template <class T>
__device__ __forceinline__ float magnitude(const Eight<T>& x) {
    if constexpr (sizeof(T) == 4) {
        float m = fabsf(__uint_as_float(x.w[0]));
#pragma unroll
        for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(__uint_as_float(x.w[i])));
        return m;
    } else {
        uint32_t m = x.w[0] & 0x7FFF7FFFu;
#pragma unroll
        for (int i = 1; i < 4; ++i) m = max_nan_bf16x2(m, x.w[i] & 0x7FFF7FFFu);
        m = max_nan_bf16x2(m, m >> 16);  // the low half: both halves' largest
        return __uint_as_float(m << 16);
    }
}
// Elements 2 i and 2 i + 1 as packed floats.
template <class T>
__device__ __forceinline__ uint64_t pair_of(const Eight<T>& x, int i) {
    if constexpr (sizeof(T) == 4) return f32x2_pack(__uint_as_float(x.w[2 * i]), __uint_as_float(x.w[2 * i + 1]));
    else return f32x2_pack(__uint_as_float(x.w[i] << 16), __uint_as_float(x.w[i] & 0xFFFF0000u));
}

// v / 6 rounded to nearest (see encode8).
__device__ __forceinline__ float sixth(float v) {
    const float q = v * (1.0f / 6.0f);
    return fmaf(fmaf(-q, 6.0f, v), 1.0f / 6.0f, q);
}

// 1 / s rounded to nearest for an E4M3 value s > 0: an approximation one unit off at most, and one Newton step (the same
// paper), which leaves 2^-46 of 1 / s before its own rounding. s is 8 .. 15 or 1 .. 7 times a power of two: 1 / s is such a
// power itself or has binary digits of a period of 12 at most, so no midpoint of two floats is that near. All 126 values are
// tested through the codes on both sides of every threshold.
__device__ __forceinline__ float reciprocal(float s) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(s));
    return fmaf(fmaf(-r, s, 1.0f), r, r);
}

// Encodes this lane's 8 elements (zeros where the lane is past the row): its scale word and its 8 codes. The group's lanes
// (2 for NVFP4, 4 for MXFP4) are neighbours. Instructions, not HBM, bound the encode of bf16 (of NVFP4 the issue slots are
// busy 79 percent of the cycles, DRAM 39), so two elements go through each packed one, and the largest |y| is made from
// the largest |x| (the product's rounding keeps their order). 8191 x 5152 with an instruction an element took 36 us to
// NVFP4 from either type and 31 to MXFP4; now 25.4 from bf16 and 29.6 from fp32, and 21.6 and 28.4.
//
// y / s is rounded to nearest, from r = 1 / s rounded to nearest, by two fused steps after the first estimate (P. W.
// Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor", 1990):
// q = y r, y / s = q - (q s - y) r. Written with -y and -r the signs of zeros come out right. Where the remainder
// underflows the quotient is far below the least nonzero code's threshold.
template <bool MX, class T>
__device__ __forceinline__ void encode8(const Eight<T>& x, float inv_g, uint32_t& word, uint32_t& codes) {
    float amax = magnitude(x);
    amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    if (MX) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    amax = __fmul_rn(amax, inv_g);
    const bool finite = __float_as_uint(amax) < 0x7F800000u;
    bool zero = !finite;
    const uint64_t ng = f32x2_pack(-inv_g, -inv_g);
    float t[8];
    if (MX) {
        // floor(log2 amax) - 2 in the biased exponent; amax below 2^-125 (zero too) takes the least, 2^-127
        const int b = max(static_cast<int>(__float_as_uint(amax) >> 23) - 2, 0);
        word = finite ? static_cast<uint32_t>(b) : 255u;
        const float inv = __uint_as_float(static_cast<uint32_t>(254 - b) << 23);  // 2^(127 - b), exact
        const uint64_t ni = f32x2_pack(-inv, -inv);
#pragma unroll
        for (int i = 0; i < 4; ++i) f32x2_unpack(f32x2_mul(f32x2_mul(pair_of(x, i), ng), ni), t[2 * i], t[2 * i + 1]);
    } else {
        word = finite ? f32_to_e4m3(sixth(amax)) : 0x7Fu;
        zero |= word == 0;
        const float s = zero ? 1.0f : e4m3_bits_to_f32(word), r = reciprocal(s);
        const uint64_t ss = f32x2_pack(s, s), nr = f32x2_pack(-r, -r);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint64_t ny = f32x2_mul(pair_of(x, i), ng), q = f32x2_mul(ny, nr);
            f32x2_unpack(f32x2_fma(f32x2_fma(q, ss, ny), nr, q), t[2 * i], t[2 * i + 1]);
        }
    }
    codes = zero ? 0u : f32x8_to_e2m1(t);
}

// Where the encoded rows go: row r to row r; a plan's token to the sorted rows of its slots; a plan's sorted row to its place.
enum class Rows { Plain, Tokens, Sorted };

// STEPS steps of 256 elements per warp and item. 64 registers, and 48 for bf16, which holds half as many words: without the
// bounds 8191 x 5152 took 8 percent longer from fp32 and 6 from bf16. CTAs of 128 threads rather than 256: 4096 tokens x 8 slots
// of 2048 to MXFP4 13.8 -> 12.6 us (1.7 rounds of CTAs, the second not full; its issue slots are busy 42 percent of
// the cycles and DRAM 15: latency bounds it, not either of them).
template <bool MX, class T, bool VEC, Rows ROWS, int STEPS>
__global__ void __launch_bounds__(kQThreads, sizeof(T) == 2 ? 10 : 8) fp4_quantize_kernel(const T* __restrict__ X, int64_t ldx, int64_t rows,
                                                                 int64_t matrices, int K, float inv_g, PlanView p,
                                                                 uint8_t* __restrict__ codes, int64_t pitch,
                                                                 uint8_t* __restrict__ scales, int chunks) {
    constexpr int kGroupLanes = MX ? 4 : 2, kChunkElems = MX ? 128 : 64;
    const int lane = threadIdx.x & 31;
    const int per_row = (K + STEPS * 256 - 1) / (STEPS * 256);
    int64_t items = rows * matrices * per_row;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kQThreads / 32);
    using Bits = std::conditional_t<sizeof(T) == 4, uint32_t, uint16_t>;
    __shared__ alignas(16) Bits turned[VEC ? 1 : kQThreads / 32][256];  // unaligned rows: a step of each warp's
    griddep_begin();
    // sorted rows: those past the rows in use are not read (the caller's buffer may end before them)
    if constexpr (ROWS == Rows::Sorted) items = min(items, static_cast<int64_t>(ld_l2(p.offsets + p.experts)) * per_row);
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * (kQThreads / 32) + (threadIdx.x >> 5); it < items; it += step) {
        const int64_t r = items <= INT32_MAX ? static_cast<int32_t>(it) / per_row : it / per_row;
        const int k0 = static_cast<int>(it - r * per_row) * (STEPS * 256) + 8 * lane;
        int tiled = -1;
        if constexpr (ROWS == Rows::Sorted) tiled = plan_index(ld_l2(p.scale_row + r), p.tiled);
        Eight<T> x[STEPS];
#pragma unroll
        for (int u = 0; u < STEPS; ++u) {
            x[u] = Eight<T>{};
            if constexpr (VEC) {
                if (k0 + 256 * u < K) load8(X + r * ldx + k0 + 256 * u, x[u]);
            } else {
                const int k = k0 - 8 * lane + 256 * u + lane;
                const Bits* p = reinterpret_cast<const Bits*>(X + r * ldx + k);
                Bits e[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) e[i] = k + 32 * i < K ? ld_l2(p + 32 * i) : Bits{0};
                pack8(e, x[u]);
            }
        }
        if constexpr (!VEC) {
#pragma unroll
            for (int u = 0; u < STEPS; ++u) turn8(x[u], turned[threadIdx.x >> 5], lane);
        }
        // with a plan: where the row goes, lane j holding slot j's places (checked where they are used: a check here, in the way of
        // the loads, cost 96 rows of 2048 a tenth, 2.4 -> 2.6 us)
        int at = -1, srow = -1;
        if (ROWS == Rows::Tokens && lane < p.slots) {
            at = ld_l2(p.position + r * p.slots + lane);
            if (plan_index(at, p.rows) >= 0) srow = ld_l2(p.scale_row + at);
        }
        uint32_t c[STEPS], words = 0;  // words: a byte of each step, the same in a group's lanes; groups past K: zero
#pragma unroll
        for (int u = 0; u < STEPS; ++u) {
            uint32_t word;
            encode8<MX>(x[u], inv_g, word, c[u]);
            if (k0 + 256 * u < K) words |= word << (8 * u);
        }
        // Four groups are a scale word. Four steps: the groups transpose their four bytes, so that group i holds the word of
        // step i; one step: every group gathers the word.
        const int group = lane / kGroupLanes % 4;  // within the four
        if constexpr (STEPS == 4) {
            uint32_t got = __shfl_xor_sync(0xffffffffu, words, kGroupLanes);
            words = group & 1 ? prmt(words, got, 0x3715) : prmt(words, got, 0x6240);
            got = __shfl_xor_sync(0xffffffffu, words, 2 * kGroupLanes);
            words = group & 2 ? prmt(words, got, 0x3276) : prmt(words, got, 0x5410);
        } else {
            words <<= 8 * group;
            words |= __shfl_xor_sync(0xffffffffu, words, kGroupLanes);
            words |= __shfl_xor_sync(0xffffffffu, words, 2 * kGroupLanes);
        }
        // Codes of row `row`: where there are four steps the lanes of a four exchange them so that each writes 16 bytes of
        // one step (a store instruction per row instead of four).
        const int quad = lane & 3;
        if constexpr (STEPS == 4) {
#pragma unroll
            for (int d = 1; d < 4; d <<= 1) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (u & d) continue;
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, quad & d ? c[u] : c[u + d], d);
                    if (quad & d) c[u] = got;
                    else c[u + d] = got;
                }
            }
        }
        auto put_codes = [&](int64_t row) {
            uint8_t* cp = codes + row * pitch + (k0 - 8 * lane) / 2;
            if constexpr (STEPS == 4) {
                const int k = 256 * quad + 32 * (lane >> 2);  // within the item; the bytes up to the pitch are the row's own
                if (k0 - 8 * lane + k < K) *reinterpret_cast<uint4*>(cp + k / 2) = make_uint4(c[0], c[1], c[2], c[3]);
            } else {
                if (k0 < K) *reinterpret_cast<uint32_t*>(cp + 4 * lane) = c[0];
            }
        };
        // Scale words: a lane of each group writes the group's step (one step: of the first group); with a plan the group's
        // kSub lanes write for kSub slots at once.
        constexpr int kSub = kGroupLanes, kChunkLanes = 4 * kGroupLanes, kChunksStep = 32 / kChunkLanes;
        const int sub = lane % kGroupLanes;
        const int chunk = (k0 - 8 * lane) / kChunkElems + (STEPS == 4 ? group * kChunksStep : 0) + lane / kChunkLanes;
        const bool has = chunk < chunks && (STEPS == 4 || group == 0);
        auto put_scales = [&](int64_t tiled) {
            *reinterpret_cast<uint32_t*>(scales + scale_word(tiled, chunk, chunks)) = words;
        };
        if (ROWS == Rows::Plain) {
            put_codes(r);
            if (has && sub == 0) put_scales(tiled_row(r, rows, matrices));
        } else if (ROWS == Rows::Sorted) {
            if (tiled >= 0) {
                put_codes(r);
                if (has && sub == 0) put_scales(tiled);
            }
        } else {
            for (int j0 = 0; j0 < p.slots; j0 += 32) {
                if (j0) {
                    at = srow = -1;
                    if (j0 + lane < p.slots) at = ld_l2(p.position + r * p.slots + j0 + lane);
                    if (plan_index(at, p.rows) >= 0) srow = ld_l2(p.scale_row + at);
                }
                const int most = min(32, p.slots - j0);
                for (int j = 0; j < most; ++j) {
                    const int row = plan_index(__shfl_sync(0xffffffffu, at, j), p.rows);
                    if (row >= 0) put_codes(row);
                }
                for (int j = 0; j < most; j += kSub) {  // lanes past the slots hold -1
                    const int tiled = plan_index(__shfl_sync(0xffffffffu, srow, (j + sub) & 31), p.tiled);
                    if (has && tiled >= 0 && j + sub < most) put_scales(tiled);
                }
            }
        }
    }
}

// E consecutive elements -> out at o: by one store of 16 bytes, or of an element each.
template <class T, bool VEC, int E>
__device__ __forceinline__ void store(T* o, const float (&v)[E]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4 && i < E; ++i) {
        if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(v[i]);
        else if (2 * i < E) w[i] = f32x2_to_bf16x2(v[2 * i], v[2 * i + 1]);
    }
    if constexpr (VEC) {
        *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if constexpr (sizeof(T) == 4) o[i] = v[i];
            else reinterpret_cast<uint16_t*>(o)[i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i % 2)));
        }
    }
}

// out = fp32(e2m1 * s * g), the first product exact. A kernel of its own for a plan's rows: the check of scale_row in one for
// both cost 1000 x 5120 of no plan a tenth (3.8 -> 4.2 us to bf16).
template <bool MX, class T, bool VEC, int STEPS, bool PLAN>
__global__ void __launch_bounds__(kQThreads) fp4_dequantize_kernel(const uint8_t* __restrict__ codes, int64_t pitch,
                                                                   const uint8_t* __restrict__ scales, int chunks,
                                                                   int64_t rows, int64_t matrices, int K, float g,
                                                                   const int32_t* __restrict__ scale_row, int tiled,
                                                                   T* __restrict__ out) {
    constexpr int kChunkElems = MX ? 128 : 64, kChunksStep = 256 / kChunkElems;
    constexpr int E = VEC && sizeof(T) == 2 ? 8 : 4;  // elements a lane writes at a time
    const int lane = threadIdx.x & 31;
    const int per_row = (K + STEPS * 256 - 1) / (STEPS * 256);
    const int64_t items = rows * matrices * per_row;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kQThreads / 32);
    griddep_begin();
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * (kQThreads / 32) + (threadIdx.x >> 5); it < items; it += step) {
        const int64_t r = items <= INT32_MAX ? static_cast<int32_t>(it) / per_row : it / per_row;
        const int k0 = static_cast<int>(it - r * per_row) * (STEPS * 256);
        const int64_t sr = PLAN ? plan_index(ld_l2(scale_row + r), tiled) : tiled_row(r, rows, matrices);  // -1: a row not in use
        uint32_t c[STEPS], w = 0;
#pragma unroll
        for (int u = 0; u < STEPS; ++u) {
            const int k = k0 + 256 * u + 8 * lane;
            c[u] = sr >= 0 && k < K ? ld_l2(reinterpret_cast<const uint32_t*>(codes + r * pitch + k / 2)) : 0u;
        }
        // lane j holds the scale words of the item's chunk j
        const int chunk = k0 / kChunkElems + lane;
        if (sr >= 0 && lane < STEPS * kChunksStep && chunk < chunks)
            w = ld_l2(reinterpret_cast<const uint32_t*>(scales + scale_word(sr, chunk, chunks)));
#pragma unroll
        for (int u = 0; u < STEPS; ++u) {
            if (k0 + 256 * u >= K) break;
#pragma unroll
            for (int h = 0; h < 8 / E; ++h) {  // lane l: elements E l .. E l + E - 1 of this part of the step
                const int at = 32 * E * h + E * lane;
                const uint32_t mine = E == 8 ? c[u] : __shfl_sync(0xffffffffu, c[u], 16 * h + (lane >> 1)) >> (16 * (lane & 1));
                const int group = at / (kChunkElems / 4);  // within the step
                const uint32_t word = __shfl_sync(0xffffffffu, w, u * kChunksStep + (group >> 2)) >> (8 * (group & 3)) & 255u;
                float s = MX ? (word == 255u ? __uint_as_float(0x7FC00000u)
                                : word == 0u ? __uint_as_float(0x00400000u)  // 2^-127
                                             : __uint_as_float(word << 23))
                             : e4m3_bits_to_f32(word);
                if (sr < 0) s = 0.0f;
                float v[E];
#pragma unroll
                for (int i = 0; i < E / 2; ++i) {
                    const float2 e = __half22float2(u32_as_half2(e2m1x2_to_f16x2<0>(mine >> (8 * i))));
                    f32x2_unpack(f32x2_mul(f32x2_mul(f32x2_pack(e.x, e.y), f32x2_pack(s, s)), f32x2_pack(g, g)), v[2 * i], v[2 * i + 1]);
                }
                const int k = k0 + 256 * u + at;
                if (k < K) store<T, VEC, E>(out + r * static_cast<int64_t>(K) + k, v);
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
    griddep_begin();
    const int64_t step = static_cast<int64_t>(gridDim.x) * kQThreads;
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * kQThreads + threadIdx.x; it < items; it += step) {
        const int64_t r = it / chunks, c = it - r * chunks, m = r / padded, rr = r - m * padded;
        uint32_t word = 0;
        if (rr < rows) {
            const uint8_t* src = in + (m * rows + rr) * groups + 4 * c;
            const int64_t left = groups - 4 * c;
            for (int j = 0; j < 4; ++j)
                if (j < left) word |= static_cast<uint32_t>(ld_l2(src + j)) << (8 * j);
        }
        *reinterpret_cast<uint32_t*>(out + scale_word(r, c, chunks)) = word;
    }
}

// Code rows of half bytes each -> rows of `pitch` bytes (K % 16 == 0: whole 8-byte words; the rows may start
// on any byte).
__global__ void __launch_bounds__(kQThreads) fp4_pitch_codes_kernel(const uint8_t* __restrict__ in, int64_t rows,
                                                                    int64_t half, int64_t pitch, uint8_t* __restrict__ out) {
    const int64_t words = pitch / 8, items = rows * words;
    griddep_begin();
    const int64_t step = static_cast<int64_t>(gridDim.x) * kQThreads;
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * kQThreads + threadIdx.x; it < items; it += step) {
        const int64_t r = it / words, b = 8 * (it - r * words);
        uint32_t lo = 0, hi = 0;
        if (b < half) {
            const uint8_t* src = in + r * half + b;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                lo |= static_cast<uint32_t>(ld_l2(src + j)) << (8 * j);
                hi |= static_cast<uint32_t>(ld_l2(src + 4 + j)) << (8 * j);
            }
        }
        *reinterpret_cast<uint2*>(out + r * pitch + b) = make_uint2(lo, hi);
    }
}

// CTAs of a grid, each of which walks its items with that stride. Several rounds of them: a CTA that comes in loads while its
// neighbours compute (8191 x 5152 with 64 per SM rather than 16: decode 34.1 -> 29.9 us, 19.8 -> 18.2 to bf16, encode of fp32 30.6
// -> 29.6; with 256 the unaligned outputs take a fifth longer).
int item_grid(int64_t items, int per_cta) {
    return static_cast<int>(
        std::max<int64_t>(1, std::min<int64_t>((items + per_cta - 1) / per_cta, int64_t(device_sm_count()) * 64)));
}

// Whether the rows fill the device's warps with items of 1024 elements; otherwise items of 256.
bool many_items(int64_t rows, int64_t K) { return rows * ((K + 1023) / 1024) >= int64_t(device_sm_count()) * 16; }

template <bool MX, class T, bool VEC, Rows ROWS, int STEPS>
cudaError_t run_quantize(const T* x, int64_t ldx, int64_t rows, int64_t K, int64_t matrices, float inv_g, const PlanView& p,
                  uint8_t* codes, uint8_t* scales, cudaStream_t stream) {
    const int64_t items = rows * matrices * ((K + STEPS * 256 - 1) / (STEPS * 256));
    return launch_dependent(fp4_quantize_kernel<MX, T, VEC, ROWS, STEPS>, item_grid(items, kQThreads / 32), kQThreads, stream, x,
                            ldx, rows, matrices, K, inv_g, p, codes, fp4_pitch(K), scales, fp4_chunks(MX, K));
}

template <bool MX, class T, bool VEC>
cudaError_t run_quantize(const void* X, int64_t ldx, int64_t rows, int64_t K, int64_t matrices, float inv_g, const PlanView& p,
                         bool sorted, uint8_t* codes, uint8_t* scales, cudaStream_t stream) {
    const T* x = static_cast<const T*>(X);
    const bool many = many_items(rows * matrices, K);
    auto go = [&](auto r) {
        constexpr Rows ROWS = decltype(r)::value;
        return many ? run_quantize<MX, T, VEC, ROWS, 4>(x, ldx, rows, K, matrices, inv_g, p, codes, scales, stream)
                    : run_quantize<MX, T, VEC, ROWS, 1>(x, ldx, rows, K, matrices, inv_g, p, codes, scales, stream);
    };
    if (!p.experts) return go(std::integral_constant<Rows, Rows::Plain>{});
    return sorted ? go(std::integral_constant<Rows, Rows::Sorted>{}) : go(std::integral_constant<Rows, Rows::Tokens>{});
}

template <bool MX, class T, bool VEC, int STEPS>
cudaError_t run_dequantize(const Fp4View& v, int64_t K, float g, const PlanView& p, T* out, cudaStream_t stream) {
    const int64_t items = v.rows * v.matrices * ((K + STEPS * 256 - 1) / (STEPS * 256));
    const auto kern = p.experts ? fp4_dequantize_kernel<MX, T, VEC, STEPS, true> : fp4_dequantize_kernel<MX, T, VEC, STEPS, false>;
    return launch_dependent(kern, item_grid(items, kQThreads / 32), kQThreads, stream, v.codes, fp4_pitch(K), v.scales,
                            fp4_chunks(MX, K), v.rows, v.matrices, K, g, p.scale_row, p.tiled, out);
}

template <bool MX, class T>
cudaError_t run_dequantize(const Fp4View& v, int64_t K, float g, const PlanView& p, void* out, cudaStream_t stream) {
    T* o = static_cast<T*>(out);
    const bool many = many_items(v.rows * v.matrices, K);
    // rows of K elements (a multiple of 16) keep the base's 16-byte alignment
    if (reinterpret_cast<uintptr_t>(out) % 16 == 0) {
        if (many) return run_dequantize<MX, T, true, 4>(v, K, g, p, o, stream);
        else return run_dequantize<MX, T, true, 1>(v, K, g, p, o, stream);
    } else {
        return run_dequantize<MX, T, false, 1>(v, K, g, p, o, stream);
    }
}

}  // namespace

cudaError_t launch_fp4_quantize(bool mx, bool bf16, const void* X, int64_t ldx, int64_t rows, int64_t K,
                                int64_t matrices, float inv_g, const PlanView& p, bool sorted, uint8_t* codes,
                                uint8_t* scales, cudaStream_t stream) {
    const int64_t bytes = bf16 ? 16 : 32;  // of eight elements
    const bool vec = reinterpret_cast<uintptr_t>(X) % bytes == 0 && ldx * (bytes / 8) % bytes == 0;
    auto go = [&](auto m) {
        constexpr bool MX = decltype(m)::value;
        if (bf16) {
            if (vec) return run_quantize<MX, __nv_bfloat16, true>(X, ldx, rows, K, matrices, inv_g, p, sorted, codes, scales, stream);
            else return run_quantize<MX, __nv_bfloat16, false>(X, ldx, rows, K, matrices, inv_g, p, sorted, codes, scales, stream);
        } else {
            if (vec) return run_quantize<MX, float, true>(X, ldx, rows, K, matrices, inv_g, p, sorted, codes, scales, stream);
            else return run_quantize<MX, float, false>(X, ldx, rows, K, matrices, inv_g, p, sorted, codes, scales, stream);
        }
    };
    return mx ? go(std::true_type{}) : go(std::false_type{});
}

cudaError_t launch_fp4_dequantize(bool mx, const Fp4View& v, int64_t K, float g, const PlanView& p, bool bf16, void* out,
                                  cudaStream_t stream) {
    if (mx)
        return bf16 ? run_dequantize<true, __nv_bfloat16>(v, K, g, p, out, stream) : run_dequantize<true, float>(v, K, g, p, out, stream);
    return bf16 ? run_dequantize<false, __nv_bfloat16>(v, K, g, p, out, stream) : run_dequantize<false, float>(v, K, g, p, out, stream);
}

cudaError_t launch_fp4_pack(bool mx, const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K,
                            int64_t matrices, uint8_t* codes_out, uint8_t* scales_out, cudaStream_t stream) {
    const int64_t chunks = fp4_chunks(mx, K), padded = (rows + 127) / 128 * 128;
    cudaError_t e = launch_dependent(fp4_tile_scales_kernel, item_grid(matrices * padded * chunks, kQThreads), kQThreads, stream, scales,
                                     rows, matrices, K / (mx ? 32 : 16), chunks, scales_out);
    if (e != cudaSuccess || codes_out == codes) return e;
    const int64_t pitch = fp4_pitch(K);
    return launch_dependent(fp4_pitch_codes_kernel, item_grid(matrices * rows * (pitch / 8), kQThreads), kQThreads, stream, codes,
                            matrices * rows, K / 2, pitch, codes_out);
}

}  // namespace pnq
