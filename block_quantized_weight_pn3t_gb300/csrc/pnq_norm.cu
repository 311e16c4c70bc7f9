// pnq_norm.cu -- root-mean-square norm with the residual's addition, its gradients, and rows of 8-bit codes with one scale
// each (of a norm, or of rows as they are); definitions in include/pnq.h.
//
//   t = x + residual (rounded to the rows' type), r = 1 / sqrt(mean(t^2) + eps), y = t r w
//   codes: p = fp32(t w), code = rne(127 p / max|p|), scale = max|p| r / 127. The row's factor r cancels in the codes, so they hang on
//   no rounded sum, and the sum of squares and the maximum go through one reduction.
//   gradients: n = t r, g = dy w: dx = r (g - n mean(g n)) + dtotal, dw = sum over rows of dy n.
//
// All of it is bound by HBM: every input is read once and held in registers (a row by a warp or by a CTA) until it is written.
// Sums, maxima and products are fp32; each result is rounded once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "pnq_device.cuh"
#include "pnq_internal.h"

namespace pnq {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kWarpRows = 4;      // rows (warps) of a CTA where a warp takes a row
constexpr uint32_t kInf = 0x7f800000u;

// V consecutive elements as they are in memory (`Raw` words) and as fp32. V = 8: 16-byte accesses; V = 2: one access of two elements.
template <class T, int V>
struct Io;
template <int V>
struct Io<float, V> {
    struct Raw {
        uint32_t w[V];
    };
    static __device__ __forceinline__ Raw raw(const float* p) {
        if constexpr (V == 8) {
            const uint4 a = ld_l2(reinterpret_cast<const uint4*>(p)), b = ld_l2(reinterpret_cast<const uint4*>(p) + 1);
            return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
        } else if constexpr (V == 2) {
            const uint2 a = ld_l2(reinterpret_cast<const uint2*>(p));
            return {{a.x, a.y}};
        } else {
            return {{__float_as_uint(ld_l2(p))}};
        }
    }
    static __device__ __forceinline__ void value(const Raw& r, float (&f)[V]) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = __uint_as_float(r.w[i]);
    }
    static __device__ __forceinline__ void store(float* p, const float (&f)[V]) {
        if constexpr (V == 8) {
            reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
            reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else if constexpr (V == 2) {
            *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
        } else {
            *p = f[0];
        }
    }
    static __device__ __forceinline__ void store(float* p, const Raw& r) {
        float f[V];
        value(r, f);
        store(p, f);
    }
    static __device__ __forceinline__ Raw sum(const Raw& a, const Raw& b) {
        Raw r;
#pragma unroll
        for (int i = 0; i < V; ++i) r.w[i] = __float_as_uint(__fadd_rn(__uint_as_float(a.w[i]), __uint_as_float(b.w[i])));
        return r;
    }
};
template <int V>
struct Io<__nv_bfloat16, V> {
    struct Raw {
        uint32_t w[(V + 1) / 2];
    };
    static __device__ __forceinline__ Raw raw(const __nv_bfloat16* p) {
        if constexpr (V == 8) {
            const uint4 a = ld_l2(reinterpret_cast<const uint4*>(p));
            return {{a.x, a.y, a.z, a.w}};
        } else if constexpr (V == 2) {
            return {{ld_l2(reinterpret_cast<const uint32_t*>(p))}};
        } else {
            return {{static_cast<uint32_t>(ld_l2(reinterpret_cast<const uint16_t*>(p)))}};
        }
    }
    static __device__ __forceinline__ void value(const Raw& r, float (&f)[V]) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = __uint_as_float(i % 2 ? r.w[i / 2] & 0xffff0000u : r.w[i / 2] << 16);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&f)[V]) {
        if constexpr (V == 8) {
            *reinterpret_cast<uint4*>(p) = make_uint4(f32x2_to_bf16x2(f[0], f[1]), f32x2_to_bf16x2(f[2], f[3]),
                                                      f32x2_to_bf16x2(f[4], f[5]), f32x2_to_bf16x2(f[6], f[7]));
        } else if constexpr (V == 2) {
            *reinterpret_cast<uint32_t*>(p) = f32x2_to_bf16x2(f[0], f[1]);
        } else {
            *p = __float2bfloat16_rn(f[0]);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const Raw& r) {
        if constexpr (V == 8) *reinterpret_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
        else if constexpr (V == 2) *reinterpret_cast<uint32_t*>(p) = r.w[0];
        else *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(r.w[0]);
    }
    // Rounded once, which is what the fp32 sum rounded again is: where two numbers of 8 bits have no exact sum of 24, one is below 2^-16 of the other,
    // and the sum is not near the middle of two bf16 numbers.
    static __device__ __forceinline__ Raw sum(const Raw& a, const Raw& b) {
        Raw r;
#pragma unroll
        for (int i = 0; i < (V + 1) / 2; ++i) asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r.w[i]) : "r"(a.w[i]), "r"(b.w[i]));
        return r;
    }
};
template <class T, int V>
__device__ __forceinline__ void load(const T* p, float (&f)[V]) {
    Io<T, V>::value(Io<T, V>::raw(p), f);
}

template <int V>
__device__ __forceinline__ void load_weight(const void* w, bool bf16, int at, float (&f)[V]) {
    if (bf16) load<__nv_bfloat16, V>(static_cast<const __nv_bfloat16*>(w) + at, f);
    else load<float, V>(static_cast<const float*>(w) + at, f);
}

// The codes of p against inv = 127 / top: p inv, rounded once to a whole number, is the code unless it is near the middle of two (inv's
// rounding moves it by 127 * 2^-24 at most, and what is left of it is computed to 2^-25). There the sign of 127 p - middle top decides, ties to
// even: both products as unevaluated sums of two floats (T. J. Dekker 1971), whose difference is exact (31 and 33 bits, near to each other). bf16 rows, whose
// quotients often are ties, need that for one element in a hundred. (In doubles, which run at 1/64 of the rate, it took 70 of 100 us.)
struct Encoder {
    float f, inv, top;  // f lifts rows of tiny values, and lowers rows of huge ones, so that no step leaves the normal numbers
    __device__ __forceinline__ explicit Encoder(float t) {
        f = t < 0x1p-60f ? 0x1p100f : t > 0x1p100f ? 0x1p-100f : 1.0f;
        top = t * f;
        inv = t > 0.0f ? 127.0f / top : 0.0f;
    }
    static constexpr float kWhole = 12582912.0f;  // 1.5 * 2^23: a sum's low bits are the whole number
    template <int V>
    __device__ __forceinline__ void operator()(const float (&v)[V], uint32_t (&c)[V]) const {
        float p[V], away[V];
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = v[i];
        if (f != 1.0f) {
#pragma unroll
            for (int i = 0; i < V; ++i) p[i] *= f;
        }
        bool near = false;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float s = fmaf(p[i], inv, kWhole);
            away[i] = fmaf(p[i], inv, -__fsub_rn(s, kWhole));
            near |= fabsf(away[i]) > 0.5f - 0x1p-16f;
            c[i] = __float_as_uint(s);
        }
        if (near) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (fabsf(away[i]) > 0.5f - 0x1p-16f) c[i] = decide(p[i], c[i], away[i] > 0.0f ? 1.0f : -1.0f);
        }
    }
    // The code of p, which lies near the middle of the whole number (in c's low bits) and the next to `side`.
    __device__ __forceinline__ uint32_t decide(float p, uint32_t c, float side) const {
        const float middle = fmaf(0.5f, side, __fsub_rn(__uint_as_float(c), kWhole)), a = __fmul_rn(127.0f, p), b = __fmul_rn(middle, top);
        const float d = side * __fadd_rn(__fsub_rn(a, b), __fsub_rn(fmaf(127.0f, p, -a), fmaf(middle, top, -b)));
        // beyond the middle, or on it with an odd whole number (its lowest bit is the sum's)
        return d > 0.0f || (d == 0.0f && (c & 1)) ? c + (side > 0.0f ? 1u : ~0u) : c;
    }
};

template <int V>
__device__ __forceinline__ void store_codes(int8_t* at, const Encoder& e, const float (&p)[V]) {
    uint32_t c[V];
    e(p, c);
    if constexpr (V == 8) {
        *reinterpret_cast<uint2*>(at) = make_uint2(prmt(prmt(c[0], c[1], 0x0040), prmt(c[2], c[3], 0x0040), 0x5410),
                                                   prmt(prmt(c[4], c[5], 0x0040), prmt(c[6], c[7], 0x0040), 0x5410));
    } else if constexpr (V == 2) {
        *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(prmt(c[0], c[1], 0x0040));
    } else {
        *at = static_cast<int8_t>(c[0]);
    }
}

// The larger of top and the magnitudes of a row's values, NaN if there is one.
template <int V>
__device__ __forceinline__ float largest(float top, const float (&p)[V]) {
    if constexpr (V == 1) {
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(fabsf(p[0])));
    } else {
#pragma unroll
        for (int j = 0; j < V; j += 2) asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(top) : "f"(p[j]), "f"(p[j + 1]));
    }
    return top;
}

__device__ __forceinline__ float warp_total(float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// Sum and largest word over a team (a warp, or the CTA through `part`), the same in every thread and from call to call.
template <bool WARP>
__device__ __forceinline__ void reduce(float& sum, uint32_t& top, float2* part) {
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    top = __reduce_max_sync(0xffffffffu, top);
    if constexpr (!WARP) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
        if (warps == 1) return;
        if (lane == 0) part[warp] = make_float2(sum, __uint_as_float(top));
        __syncthreads();
        const float2 v = lane < warps ? part[lane] : make_float2(0.0f, 0.0f);
        sum = v.x;
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        top = __reduce_max_sync(0xffffffffu, __float_as_uint(v.y));
    }
}

struct NormArgs {
    const void *x, *residual, *weight;  // residual, weight: null where there is none
    void *total, *y;                    // null where not wanted
    float* rstd;
    int8_t* codes;
    float* scales;
    int64_t ldx, ldr, pitch, rows;
    float eps;
    int D;
    bool weight_bf16, norm;             // norm: not an encode of the rows as they are
};

// What a row's sum of squares and largest |p| come to: rstd, and the scale of its codes.
__device__ __forceinline__ float row_rstd(const NormArgs& a, float sum) {
    return a.norm ? 1.0f / sqrtf(sum / static_cast<float>(a.D) + a.eps) : 1.0f;
}
// A row that holds a NaN or an infinity (or whose p do) has the scale NaN and codes of zero.
__device__ __forceinline__ float row_scale(uint32_t top, float rstd) {
    return top >= kInf ? __uint_as_float(0x7fc00000u) : __uint_as_float(top) * rstd / 127.0f;
}

template <class T, int V>
__device__ __forceinline__ typename Io<T, V>::Raw load_total(const NormArgs& a, int64_t row, int at) {
    const auto x = Io<T, V>::raw(static_cast<const T*>(a.x) + row * a.ldx + at);
    return a.residual ? Io<T, V>::sum(x, Io<T, V>::raw(static_cast<const T*>(a.residual) + row * a.ldr + at)) : x;
}

// A row by a warp or a CTA, N accesses of V elements a thread, all in flight at once; row after row. With eight elements a thread the weight
// stays in registers and the next row is loaded before the present one's sum is known. Few rows, and rows not on 16 bytes, go here.
template <class T, int V, int N, bool WARP, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) norm_kernel(const NormArgs a) {
    constexpr bool kAhead = V * N == 8;
    using X = Io<T, V>;
    __shared__ float2 part[2][32];
    const int team = WARP ? 32 : static_cast<int>(blockDim.x), tid = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (WARP ? kWarpRows : 1);
    int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    griddep_begin();
    const int D = a.D;
    const bool added = a.residual != nullptr;
    typename X::Raw x[N] = {}, r[N] = {};
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = (tid + i * team) * V;
            if (at < D) {
                x[i] = X::raw(static_cast<const T*>(a.x) + row * a.ldx + at);
                if (added) r[i] = X::raw(static_cast<const T*>(a.residual) + row * a.ldr + at);
            }
        }
    };
    float w[kAhead ? N : 1][V];
    if (row < a.rows) fetch(row);
    if (kAhead && a.norm) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if ((tid + i * team) * V < D) load_weight<V>(a.weight, a.weight_bf16, (tid + i * team) * V, w[kAhead ? i : 0]);
    }
    for (int turn = 0; row < a.rows; turn ^= 1) {
        float p[N][V], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (added) {
                x[i] = X::sum(x[i], r[i]);
                if (a.total && (tid + i * team) * V < D) X::store(static_cast<T*>(a.total) + row * D + (tid + i * team) * V, x[i]);
            }
            X::value(x[i], p[i]);
        }
        const int64_t now = row;
        row += step;
        if (kAhead && row < a.rows) fetch(row);
        if (a.norm) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int at = (tid + i * team) * V;
#pragma unroll
                for (int j = 0; j < V; ++j) sum = fmaf(p[i][j], p[i][j], sum);
                if (at < D) {
                    if (a.total && !added) X::store(static_cast<T*>(a.total) + now * D + at, p[i]);
                    if constexpr (!kAhead) load_weight<V>(a.weight, a.weight_bf16, at, w[0]);
#pragma unroll
                    for (int j = 0; j < V; ++j) p[i][j] = __fmul_rn(p[i][j], w[kAhead ? i : 0][j]);
                }
            }
        }
        float most = 0.0f;
        if (a.codes) {
#pragma unroll
            for (int i = 0; i < N; ++i) most = largest(most, p[i]);
        }
        uint32_t top = __float_as_uint(most) & 0x7fffffffu;
        reduce<WARP>(sum, top, part[turn]);
        const float rstd = row_rstd(a, sum);
        if (tid == 0) {
            if (a.rstd) a.rstd[now] = rstd;
            if (a.codes) a.scales[now] = row_scale(top, rstd);
        }
        if (a.codes) {
            const Encoder e(top >= kInf ? 0.0f : __uint_as_float(top));
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int at = (tid + i * team) * V;
                if (at >= D) continue;
                if (top >= kInf) {
                    const float none[V] = {};
                    store_codes<V>(a.codes + now * a.pitch + at, e, none);
                } else {
                    store_codes<V>(a.codes + now * a.pitch + at, e, p[i]);
                }
            }
        }
        if (a.y) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int at = (tid + i * team) * V;
                if (at >= D) continue;
#pragma unroll
                for (int j = 0; j < V; ++j) p[i][j] *= rstd;
                X::store(static_cast<T*>(a.y) + now * D + at, p[i]);
            }
        }
        if (!kAhead && row < a.rows) {
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = r[i] = {};
            fetch(row);
        }
    }
}

// The same for many rows on 16 bytes: `teams` rows at a time in a CTA, each by `warps` warps, N accesses of eight elements a lane. What a row costs
// besides its elements (sums through the warps, two divisions, addresses) is some 150 instructions a thread, more than eight elements do: 8192 x 5120
// bf16 with eight a thread executed 35 instructions an element and took 64 us (74 to codes); this takes 55 (55), 6.1 (5.3) TB/s. The weight waits
// in shared memory. Encoding rows as they are (not NORM) leaves registers: bf16 rows are loaded one ahead (65536 x 256 21.0 us, 26.9 without; fp32 rows of 5120
// spill, 99 and 81).
template <class T, bool NORM, int N, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) norm_teams_kernel(const NormArgs a, int warps, int teams) {
    using X = Io<T, 8>;
    constexpr bool kAhead = !NORM && sizeof(T) == 2;
    const bool norm = NORM && (sizeof(T) == 2 || a.norm);  // always NORM: taken as known, it makes fp32 rows spill (17408 x 5120 with residual 236 us, 225)
    extern __shared__ __align__(16) float weight[];  // [D] fp32
    __shared__ float2 part[2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mine = warp / warps, first = mine * warps, team = 32 * warps;
    const int tid = static_cast<int>(threadIdx.x) - 32 * first, D = a.D;
    griddep_begin();
    if (norm) {
        for (int at = static_cast<int>(threadIdx.x) * 8; at < D; at += static_cast<int>(blockDim.x) * 8) {
            float w[8];
            load_weight<8>(a.weight, a.weight_bf16, at, w);
            Io<float, 8>::store(weight + at, w);
        }
        __syncthreads();
    }
    const bool added = a.residual != nullptr;
    const int64_t step = static_cast<int64_t>(gridDim.x) * teams;
    int64_t row = static_cast<int64_t>(blockIdx.x) * teams + mine;
    auto fetch = [&](int64_t row, typename X::Raw(&x)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            x[i] = {};
            if ((tid + i * team) * 8 < D) x[i] = X::raw(static_cast<const T*>(a.x) + row * a.ldx + (tid + i * team) * 8);
        }
    };
    typename X::Raw ahead[N];
    if (kAhead && row < a.rows) fetch(row, ahead);
    for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
        typename X::Raw x[N];
        if constexpr (kAhead) {
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = ahead[i];
        } else {
            fetch(row, x);
        }
        if (NORM && added) {
            typename X::Raw r[N] = {};
#pragma unroll
            for (int i = 0; i < N; ++i)
                if ((tid + i * team) * 8 < D) r[i] = X::raw(static_cast<const T*>(a.residual) + row * a.ldr + (tid + i * team) * 8);
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = X::sum(x[i], r[i]);
        }
        float p[N][8], sum = 0.0f, most = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = (tid + i * team) * 8;
            X::value(x[i], p[i]);
            if (at >= D) continue;
            if (norm) {
                if (a.total) X::store(static_cast<T*>(a.total) + row * D + at, x[i]);
                float w[8];
                const float4 u = *reinterpret_cast<const float4*>(weight + at), v = *reinterpret_cast<const float4*>(weight + at + 4);
                w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w, w[4] = v.x, w[5] = v.y, w[6] = v.z, w[7] = v.w;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    sum = fmaf(p[i][j], p[i][j], sum);
                    p[i][j] = __fmul_rn(p[i][j], w[j]);
                }
            }
            if (a.codes) most = largest(most, p[i]);
        }
        if (kAhead && row + step < a.rows) fetch(row + step, ahead);
        uint32_t top = __float_as_uint(most) & 0x7fffffffu;
        sum = warp_total(sum);
        top = __reduce_max_sync(0xffffffffu, top);
        if (warps > 1) {
            if (lane == 0) part[turn][warp] = make_float2(sum, __uint_as_float(top));
            named_sync(static_cast<uint32_t>(1 + mine), static_cast<uint32_t>(team));
            sum = 0.0f, top = 0;
            for (int w = first; w < first + warps; ++w) {
                const float2 v = part[turn][w];
                sum += v.x;
                top = max(top, __float_as_uint(v.y));
            }
        }
        const float rstd = row_rstd(a, sum);
        if (tid == 0) {
            if (a.rstd) a.rstd[row] = rstd;
            if (a.codes) a.scales[row] = row_scale(top, rstd);
        }
        if (a.codes) {
            const Encoder e(top >= kInf ? 0.0f : __uint_as_float(top));
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int at = (tid + i * team) * 8;
                if (at >= D) continue;
                int8_t* to = a.codes + row * a.pitch + at;
                if (top >= kInf) *reinterpret_cast<uint2*>(to) = make_uint2(0, 0);
                else store_codes<8>(to, e, p[i]);
            }
        }
        if (a.y) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int at = (tid + i * team) * 8;
                if (at >= D) continue;
#pragma unroll
                for (int j = 0; j < 8; ++j) p[i][j] *= rstd;
                X::store(static_cast<T*>(a.y) + row * D + at, p[i]);
            }
        }
    }
}

// Rows too long for registers: read twice, the second time from L2 as far as it goes. A thread reads and writes the same
// elements in both passes, so that y or total may be x or residual here too.
template <class T, int V>
__global__ void __launch_bounds__(kMaxThreads) norm_long_kernel(const NormArgs a) {
    __shared__ float2 part[32];
    const int64_t row = blockIdx.x;
    const int64_t D = a.D, step = static_cast<int64_t>(kMaxThreads) * V, first = static_cast<int64_t>(threadIdx.x) * V;
    griddep_begin();
    float sum = 0.0f, most = 0.0f, p[V], w[V];
    for (int64_t at = first; at < D; at += step) {
        const auto t = load_total<T, V>(a, row, static_cast<int>(at));
        Io<T, V>::value(t, p);
        if (a.norm) {
#pragma unroll
            for (int j = 0; j < V; ++j) sum = fmaf(p[j], p[j], sum);
            if (a.total) Io<T, V>::store(static_cast<T*>(a.total) + row * D + at, t);
            load_weight<V>(a.weight, a.weight_bf16, static_cast<int>(at), w);
#pragma unroll
            for (int j = 0; j < V; ++j) p[j] = __fmul_rn(p[j], w[j]);
        }
        most = largest(most, p);
    }
    uint32_t top = __float_as_uint(most) & 0x7fffffffu;
    reduce<false>(sum, top, part);
    const float rstd = row_rstd(a, sum);
    if (threadIdx.x == 0) {
        if (a.rstd) a.rstd[row] = rstd;
        if (a.codes) a.scales[row] = row_scale(top, rstd);
    }
    const Encoder e(top >= kInf ? 0.0f : __uint_as_float(top));
    for (int64_t at = first; at < D; at += step) {
        if (a.norm && a.total) load<T, V>(static_cast<const T*>(a.total) + row * D + at, p);
        else Io<T, V>::value(load_total<T, V>(a, row, static_cast<int>(at)), p);
        if (a.norm) {
            load_weight<V>(a.weight, a.weight_bf16, static_cast<int>(at), w);
#pragma unroll
            for (int j = 0; j < V; ++j) p[j] = __fmul_rn(p[j], w[j]);
        }
        if (a.codes) {
            if (top >= kInf) {
                const float none[V] = {};
                store_codes<V>(a.codes + row * a.pitch + at, e, none);
            } else {
                store_codes<V>(a.codes + row * a.pitch + at, e, p);
            }
        }
        if (a.y) {
#pragma unroll
            for (int j = 0; j < V; ++j) p[j] *= rstd;
            Io<T, V>::store(static_cast<T*>(a.y) + row * D + at, p);
        }
    }
}

// ---- gradients ------------------------------------------------------------------------------------

struct NormBackwardArgs {
    const void *dy, *total, *weight, *dtotal;  // dtotal: null where there is none
    const float* rstd;
    void* dx;
    float* partial;  // [grid][D] sums of dy n over a CTA's rows, or null
    float* dweight;  // written by the columns' CTAs
    int64_t ldy, ldt, ldd, rows;
    int D, columns;  // columns: CTAs that take kColumns of them each, before those of the rows
    bool weight_bf16;
};

// dw[c] of kColumns columns by a CTA: kColumns lanes to a row, `slots` rows at a time, then the slots in order. value(r, c): row r's part.
constexpr int kColumns = 16;
template <class Value>
__device__ __forceinline__ void sum_columns(int64_t rows, int D, int block, float* dw, Value&& value) {
    __shared__ float part[kMaxThreads / kColumns][kColumns + 1];
    const int lane = static_cast<int>(threadIdx.x) % kColumns, slot = static_cast<int>(threadIdx.x) / kColumns;
    const int slots = static_cast<int>(blockDim.x) / kColumns, c = block * kColumns + lane;
    float sum = 0.0f;
    if (c < D) {
#pragma unroll 8
        for (int64_t r = slot; r < rows; r += slots) sum += value(r, c);
    }
    part[slot][lane] = sum;
    __syncthreads();
    if (slot == 0 && c < D) {
        sum = 0.0f;
#pragma unroll 8
        for (int s = 0; s < slots; ++s) sum += part[s][lane];
        dw[c] = sum;
    }
}

// CTA b takes rows b, b + grid, ..: the weight and its gradient's sums stay in registers from row to row, the next row is loaded
// before the present one's sum is known, and the sums leave once, to the CTA's row of `partial`.
// COLUMNS, for few elements: the weight's gradient has CTAs of its own, before those of the rows, which read dy and the total a second time, out of
// L2 (333 x 2048 fp32 8.1 us, 64 x 4096 bf16 4.6; with a kernel for it 10.2 and 6.1).
template <class T, int V, int N, bool COLUMNS>
__global__ void __launch_bounds__(kMaxThreads) norm_backward_kernel(const NormBackwardArgs a) {
    __shared__ float part[2][32];
    const int tid = threadIdx.x, team = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = team >> 5, D = a.D;
    griddep_begin();
    float w[N][V], dw[N][V];
    typename Io<T, V>::Raw t[N], g[N], d[N] = {};
    if (COLUMNS && static_cast<int>(blockIdx.x) < a.columns) {
        auto value = [&](int64_t r, int c) {
            float t[1], g[1];
            load<T, 1>(static_cast<const T*>(a.total) + r * a.ldt + c, t);
            load<T, 1>(static_cast<const T*>(a.dy) + r * a.ldy + c, g);
            return g[0] * (t[0] * ld_l2(a.rstd + r));
        };
        return sum_columns(a.rows, D, static_cast<int>(blockIdx.x), a.dweight, value);
    }
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = (tid + i * team) * V;
            if (at < D) {
                t[i] = Io<T, V>::raw(static_cast<const T*>(a.total) + row * a.ldt + at);
                g[i] = Io<T, V>::raw(static_cast<const T*>(a.dy) + row * a.ldy + at);
                if (a.dtotal) d[i] = Io<T, V>::raw(static_cast<const T*>(a.dtotal) + row * a.ldd + at);
            } else {
                t[i] = g[i] = {};
            }
        }
    };
    int64_t row = COLUMNS ? blockIdx.x - a.columns : blockIdx.x;
    fetch(row);
    float rstd = ld_l2(a.rstd + row);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int at = (tid + i * team) * V;
#pragma unroll
        for (int j = 0; j < V; ++j) w[i][j] = dw[i][j] = 0.0f;
        if (at < D) load_weight<V>(a.weight, a.weight_bf16, at, w[i]);
    }
    for (int turn = 0; row < a.rows; turn ^= 1) {
        float dot = 0.0f, n[N][V], h[N][V];
        typename Io<T, V>::Raw more[N];
        const float r = rstd;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            Io<T, V>::value(t[i], n[i]);
            Io<T, V>::value(g[i], h[i]);
            more[i] = d[i];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                n[i][j] *= r;
                dw[i][j] = fmaf(h[i][j], n[i][j], dw[i][j]);
                h[i][j] *= w[i][j];
                dot = fmaf(h[i][j], n[i][j], dot);
            }
        }
        const int64_t now = row;
        row += COLUMNS ? gridDim.x - a.columns : gridDim.x;
        if (row < a.rows) {
            fetch(row);
            rstd = ld_l2(a.rstd + row);
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
        if (warps > 1) {
            if (lane == 0) part[turn][warp] = dot;
            __syncthreads();
            dot = lane < warps ? part[turn][lane] : 0.0f;
#pragma unroll
            for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
        }
        const float mean = dot / static_cast<float>(D);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = (tid + i * team) * V;
            if (at >= D) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) h[i][j] = r * (h[i][j] - n[i][j] * mean);
            if (a.dtotal) {
                float e[V];
                Io<T, V>::value(more[i], e);
#pragma unroll
                for (int j = 0; j < V; ++j) h[i][j] += e[j];
            }
            Io<T, V>::store(static_cast<T*>(a.dx) + now * D + at, h[i]);
        }
    }
    if (a.partial) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = (tid + i * team) * V;
            if (at >= D) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) a.partial[static_cast<int64_t>(blockIdx.x) * D + at + j] = dw[i][j];
        }
    }
}

// The same for rows too long for registers: each row twice, and the weight's sums kept in the CTA's row of `partial`.
template <class T, int V>
__global__ void __launch_bounds__(kMaxThreads) norm_backward_long_kernel(const NormBackwardArgs a) {
    __shared__ float2 part[32];
    griddep_begin();
    const int64_t D = a.D, first = static_cast<int64_t>(threadIdx.x) * V, step = static_cast<int64_t>(kMaxThreads) * V;
    float* dw = a.partial ? a.partial + static_cast<int64_t>(blockIdx.x) * D : nullptr;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float r = ld_l2(a.rstd + row);
        const T *t = static_cast<const T*>(a.total) + row * a.ldt, *dy = static_cast<const T*>(a.dy) + row * a.ldy;
        float dot = 0.0f, w[V], n[V], g[V];
        uint32_t none = 0;
        for (int64_t at = first; at < D; at += step) {
            load<T, V>(t + at, n);
            load<T, V>(dy + at, g);
            load_weight<V>(a.weight, a.weight_bf16, static_cast<int>(at), w);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                n[j] *= r;
                if (dw) dw[at + j] = fmaf(g[j], n[j], row == blockIdx.x ? 0.0f : dw[at + j]);
                dot = fmaf(g[j] * w[j], n[j], dot);
            }
        }
        __syncthreads();  // the last row's sums have been read
        reduce<false>(dot, none, part);
        const float mean = dot / static_cast<float>(D);
        for (int64_t at = first; at < D; at += step) {
            load<T, V>(t + at, n);
            load<T, V>(dy + at, g);
            load_weight<V>(a.weight, a.weight_bf16, static_cast<int>(at), w);
#pragma unroll
            for (int j = 0; j < V; ++j) n[j] = r * (g[j] * w[j] - n[j] * r * mean);
            if (a.dtotal) {
                load<T, V>(static_cast<const T*>(a.dtotal) + row * a.ldd + at, g);
#pragma unroll
                for (int j = 0; j < V; ++j) n[j] += g[j];
            }
            Io<T, V>::store(static_cast<T*>(a.dx) + row * D + at, n);
        }
    }
}

// dw[c] = sum over the CTAs' partial rows, in an order that goes by their number alone: 32 columns a CTA, a warp over
// every 32nd row, then the warps in order.
__global__ void __launch_bounds__(1024) norm_weight_kernel(const float* partial, int rows, int D, float* dw) {
    __shared__ float part[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = static_cast<int>(blockIdx.x) * 32 + lane;
    griddep_begin();
    float sum = 0.0f;
    if (c < D) {
        for (int r0 = warp; r0 < rows; r0 += 8 * 32) {  // eight under way at once, the last ones too
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = r0 + 32 * i < rows ? ld_l2(partial + static_cast<int64_t>(r0 + 32 * i) * D + c) : 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += v[i];
        }
    }
    part[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && c < D) {
        sum = 0.0f;
#pragma unroll
        for (int w = 0; w < 32; ++w) sum += part[w][lane];
        dw[c] = sum;
    }
}

// ---- codes back to values -----------------------------------------------------------------------------

// out[r][k] = codes[r][k] * scales[r]: four consecutive elements a thread and step; the rows' pieces of four (`per` a row) one after the other, so
// that short rows fill CTAs too. Many pieces: eight steps, all loads under way at once (17408 x 5120 to fp32 72.6 us, to bf16 57.7; four 75.3 and
// 61.3, sixteen 79.9 and 68.0). Fewer than some sixteen such CTAs an SM: four, for more CTAs (13 x 17408 1.9 us, with eight 2.3).
constexpr int kDecodeThreads = 128;
template <class T, int STEPS>
__global__ void __launch_bounds__(kDecodeThreads) int8_dequantize_kernel(const int8_t* codes, int64_t pitch, const float* scales, int64_t rows,
                                                                         int per, T* out) {
    griddep_begin();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (STEPS * kDecodeThreads), row0 = first / per;
    const int in0 = static_cast<int>(first - row0 * per);  // of the CTA's first piece within its row
    uint32_t word[STEPS];
    float scale[STEPS];
    int64_t row[STEPS];
    int at[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const uint32_t u = static_cast<uint32_t>(in0) + i * kDecodeThreads + threadIdx.x, r = u / static_cast<uint32_t>(per);
        row[i] = row0 + r;
        at[i] = static_cast<int>(u - r * per);
        if (row[i] < rows) {
            word[i] = ld_l2(reinterpret_cast<const uint32_t*>(codes + row[i] * pitch) + at[i]);
            scale[i] = ld_l2(scales + row[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        if (row[i] >= rows) continue;
        float f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = static_cast<float>(static_cast<int8_t>(word[i] >> (8 * j))) * scale[i];
        T* o = out + (row[i] * per + at[i]) * 4;
        if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(o) = make_float4(f[0], f[1], f[2], f[3]);
        else *reinterpret_cast<uint2*>(o) = make_uint2(f32x2_to_bf16x2(f[0], f[1]), f32x2_to_bf16x2(f[2], f[3]));
    }
}

// The same for rows of any length and alignment: pieces of 128 elements of a row (`per` a row), two a warp, of each four elements a lane, 32 apart.
template <class T>
__global__ void __launch_bounds__(kDecodeThreads) int8_dequantize_any_kernel(const int8_t* codes, int64_t pitch, const float* scales, int64_t rows,
                                                                             int K, int per, T* out) {
    griddep_begin();
    const int lane = threadIdx.x & 31;
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * (kDecodeThreads / 32) + (threadIdx.x >> 5)) * 2;
    uint8_t code[2][4];
    float scale[2];
    int64_t row[2];
    int at[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        row[i] = (first + i) / per;
        at[i] = static_cast<int>(first + i - row[i] * per) * 128 + lane;
        if (row[i] >= rows) continue;
        scale[i] = ld_l2(scales + row[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (at[i] + 32 * j < K) code[i][j] = ld_l2(reinterpret_cast<const uint8_t*>(codes + row[i] * pitch + at[i] + 32 * j));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (row[i] >= rows) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (at[i] + 32 * j < K) out[row[i] * K + at[i] + 32 * j] = T(static_cast<float>(static_cast<int8_t>(code[i][j])) * scale[i]);
    }
}

// ---- launches -------------------------------------------------------------------------------------------

// The widest access (8, 2 or 1 elements) that rows of D elements at every `ld` elements of these buffers allow.
struct Rows {
    const void* p;
    int64_t ld;
    int bytes;  // of an element
};
template <size_t M>
int widest(const Rows (&rows)[M], int64_t D) {
    for (int v : {8, 2}) {
        bool fits = D % v == 0;
        for (const Rows& r : rows) {
            const int64_t a = std::min<int64_t>(16, static_cast<int64_t>(v) * r.bytes);
            fits = fits && (!r.p || (reinterpret_cast<uintptr_t>(r.p) % a == 0 && r.ld * r.bytes % a == 0));
        }
        if (fits) return v;
    }
    return 1;
}

int threads_for(int64_t D, int per) {
    return static_cast<int>(std::max<int64_t>(32, ((D + per - 1) / per + 31) / 32 * 32));
}

template <class T, int N, int THREADS, int CTAS>
cudaError_t run_teams(const NormArgs& a, cudaStream_t stream) {
    const int warps = static_cast<int>((a.D + 256 * N - 1) / (256 * N)), teams = std::max(1, THREADS / 32 / warps), smem = a.norm ? 4 * a.D : 0;
    auto kernel = a.norm ? norm_teams_kernel<T, true, N, THREADS, CTAS> : norm_teams_kernel<T, false, N, THREADS, CTAS>;
    const cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(kernel), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>((a.rows + teams - 1) / teams, CTAS * device_sm_count())));
    lc.blockDim = dim3(static_cast<unsigned>(32 * warps * teams));
    lc.dynamicSmemBytes = static_cast<size_t>(smem);
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kernel, a, warps, teams);
}

template <class T, int V>
cudaError_t run_norm(const NormArgs& a, cudaStream_t stream) {
    const int64_t D = a.D, sms = device_sm_count();
    if constexpr (V == 8) {
        // Many rows: rows together in a CTA, 32 elements a lane (16: 67 us for 8192 x 5120 bf16, 64: 63, 32: 55), by few warps a row
        if (a.rows > 4 * sms && D <= 20 * kMaxThreads) {
            if (D <= 256) return run_teams<T, 1, 320, 4>(a, stream);
            if (D <= 512) return run_teams<T, 2, 320, 3>(a, stream);
            if (D <= 10 * kMaxThreads) return run_teams<T, 4, 320, 2>(a, stream);
            return run_teams<T, 4, 640, 1>(a, stream);
        }
    }
    auto block = [&](auto n, auto most, auto per_sm) {
        constexpr int N = decltype(n)::value;
        const int threads = threads_for(D, V * N);
        const int64_t ctas = std::min(a.rows, sms * std::max(1, 1536 / threads));
        return launch_dependent(norm_kernel<T, V, N, false, decltype(most)::value, decltype(per_sm)::value>, static_cast<int>(ctas), threads, stream, a);
    };
    if (D <= 256) {
        const int64_t ctas = std::min((a.rows + kWarpRows - 1) / kWarpRows, sms * 12);
        return launch_dependent(norm_kernel<T, V, 8 / V, true, 32 * kWarpRows, 1>, static_cast<int>(ctas), 32 * kWarpRows, stream, a);
    }
    using One = std::integral_constant<int, 1>;
    using Two = std::integral_constant<int, 2>;
    using All = std::integral_constant<int, kMaxThreads>;
    if (D <= 5120) return block(std::integral_constant<int, 8 / V>{}, std::integral_constant<int, 640>{}, Two{});
    if (D <= 8 * kMaxThreads) return block(std::integral_constant<int, 8 / V>{}, All{}, One{});
    if (D <= 16 * kMaxThreads) return block(std::integral_constant<int, 16 / V>{}, All{}, One{});
    if (D <= 32 * kMaxThreads) return block(std::integral_constant<int, 32 / V>{}, All{}, One{});
    return launch_dependent(norm_long_kernel<T, V>, static_cast<int>(a.rows), kMaxThreads, stream, a);
}

template <class T>
cudaError_t run_norm(const NormArgs& a, int v, cudaStream_t stream) {
    return v == 8 ? run_norm<T, 8>(a, stream) : v == 2 ? run_norm<T, 2>(a, stream) : run_norm<T, 1>(a, stream);
}

cudaError_t run_norm(bool bf16, const NormArgs& a, cudaStream_t stream) {
    const int b = bf16 ? 2 : 4, wb = a.weight_bf16 ? 2 : 4;
    const Rows rows[] = {{a.x, a.ldx, b}, {a.residual, a.ldr, b}, {a.weight, 0, wb}, {a.total, a.D, b}, {a.y, a.D, b}};
    const int v = widest(rows, a.D);
    return bf16 ? run_norm<__nv_bfloat16>(a, v, stream) : run_norm<float>(a, v, stream);
}

// CTAs of the backward pass: as many as fill the device with threads, at most one for each row.
constexpr int64_t kBackwardRegs = 8 * kMaxThreads;  // longest row that stays in registers
// Whether the weight's gradient has CTAs of its own: few elements (500 x 4096 12.5 us so, 11.8 with a kernel for it), and few rows one after the other.
bool by_columns(int64_t rows, int64_t D) {
    return D <= kBackwardRegs && rows * D <= 1 << 20 && rows <= 24 * (threads_for(D, 8) / kColumns);
}
int64_t backward_ctas(int64_t rows, int64_t D) {
    const int threads = D <= kBackwardRegs ? threads_for(D, 8) : kMaxThreads;
    return std::min<int64_t>(rows, static_cast<int64_t>(device_sm_count()) * std::max(1, std::min(16, kMaxThreads / threads)));
}

template <class T, int V>
cudaError_t run_backward(const NormBackwardArgs& a, int ctas, cudaStream_t stream) {
    if (a.D > kBackwardRegs) return launch_dependent(norm_backward_long_kernel<T, V>, ctas, kMaxThreads, stream, a);
    return launch_dependent(a.columns ? norm_backward_kernel<T, V, 8 / V, true> : norm_backward_kernel<T, V, 8 / V, false>, ctas + a.columns,
                            threads_for(a.D, 8), stream, a);
}

template <class T>
cudaError_t run_backward(const NormBackwardArgs& a, int v, int ctas, cudaStream_t stream) {
    return v == 8   ? run_backward<T, 8>(a, ctas, stream)
           : v == 2 ? run_backward<T, 2>(a, ctas, stream)
                    : run_backward<T, 1>(a, ctas, stream);
}

}  // namespace

cudaError_t launch_rms_norm(bool bf16, const RowsView& x, const RowsView& residual, bool weight_bf16, const void* weight, float eps,
                            int64_t rows, int64_t D, void* total, void* y, float* rstd, int8_t* codes, int64_t pitch, float* scales,
                            cudaStream_t stream) {
    NormArgs a{};
    a.x = x.p, a.ldx = x.ld;
    a.residual = residual.p, a.ldr = residual.ld;
    a.weight = weight, a.weight_bf16 = weight_bf16;
    a.total = total, a.y = y, a.rstd = rstd;
    a.codes = codes, a.pitch = pitch, a.scales = scales;
    a.rows = rows, a.D = static_cast<int>(D), a.eps = eps, a.norm = true;
    return run_norm(bf16, a, stream);
}

cudaError_t launch_int8_quantize(bool bf16, const RowsView& x, int64_t rows, int64_t K, int8_t* codes, int64_t pitch, float* scales,
                                 cudaStream_t stream) {
    NormArgs a{};
    a.x = x.p, a.ldx = x.ld;
    a.codes = codes, a.pitch = pitch, a.scales = scales;
    a.rows = rows, a.D = static_cast<int>(K);
    return run_norm(bf16, a, stream);
}

int64_t rms_norm_backward_rows(int64_t rows, int64_t D) { return backward_ctas(rows, D); }

cudaError_t launch_rms_norm_backward(bool bf16, const RowsView& dy, const RowsView& total, bool weight_bf16, const void* weight,
                                     const float* rstd, const RowsView& dtotal, int64_t rows, int64_t D, void* dx, float* dweight,
                                     float* partial, cudaStream_t stream) {
    NormBackwardArgs a{};
    a.dy = dy.p, a.ldy = dy.ld;
    a.total = total.p, a.ldt = total.ld;
    a.dtotal = dtotal.p, a.ldd = dtotal.ld;
    a.weight = weight, a.weight_bf16 = weight_bf16, a.rstd = rstd;
    const bool columns = dweight && by_columns(rows, D);
    a.dx = dx, a.partial = dweight && !columns ? partial : nullptr;
    a.dweight = dweight, a.columns = columns ? static_cast<int>((D + kColumns - 1) / kColumns) : 0;
    a.rows = rows, a.D = static_cast<int>(D);
    const int b = bf16 ? 2 : 4;
    const Rows views[] = {{dy.p, dy.ld, b}, {total.p, total.ld, b}, {dtotal.p, dtotal.ld, b}, {weight, 0, weight_bf16 ? 2 : 4}, {dx, D, b}};
    const int v = widest(views, D), ctas = static_cast<int>(backward_ctas(rows, D));
    cudaError_t e = cudaSuccess;
    if (ctas > 0) e = bf16 ? run_backward<__nv_bfloat16>(a, v, ctas, stream) : run_backward<float>(a, v, ctas, stream);
    if (e != cudaSuccess || !dweight || (columns && rows > 0)) return e;
    return launch_dependent(norm_weight_kernel, static_cast<int>((D + 31) / 32), 1024, stream, partial, ctas, static_cast<int>(D), dweight);
}

cudaError_t launch_int8_dequantize(const int8_t* codes, int64_t pitch, const float* scales, int64_t rows, int64_t K, bool bf16, void* out,
                                   cudaStream_t stream) {
    const bool wide = K % 4 == 0 && pitch % 4 == 0 && reinterpret_cast<uintptr_t>(codes) % 4 == 0 &&
                      reinterpret_cast<uintptr_t>(out) % (bf16 ? 8 : 16) == 0;
    // threads of the kernels' first kind and warps of the second, at one step each
    const int64_t per = wide ? K / 4 : (K + 127) / 128, each = wide ? kDecodeThreads : kDecodeThreads / 32, ctas = (rows * per + each - 1) / each;
    if (ctas > INT32_MAX) return cudaErrorInvalidValue;
    auto go = [&](auto* o) {
        using T = std::remove_pointer_t<decltype(o)>;
        auto steps = [&](auto s) {
            constexpr int S = decltype(s)::value;
            return launch_dependent(int8_dequantize_kernel<T, S>, static_cast<int>((ctas + S - 1) / S), kDecodeThreads, stream, codes, pitch, scales,
                                    rows, static_cast<int>(per), o);
        };
        if (!wide)
            return launch_dependent(int8_dequantize_any_kernel<T>, static_cast<int>((ctas + 1) / 2), kDecodeThreads, stream, codes, pitch, scales, rows,
                                    static_cast<int>(K), static_cast<int>(per), o);
        return ctas > 8 * 16 * static_cast<int64_t>(device_sm_count()) ? steps(std::integral_constant<int, 8>{}) : steps(std::integral_constant<int, 4>{});
    };
    return bf16 ? go(static_cast<__nv_bfloat16*>(out)) : go(static_cast<float*>(out));
}

}  // namespace pnq
