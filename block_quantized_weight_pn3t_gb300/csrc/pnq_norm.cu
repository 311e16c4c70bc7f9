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

#include "pnq_device.cuh"
#include "pnq_internal.h"

namespace pnq {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kWarpRows = 4;      // rows (warps) of a CTA where a warp takes a row
constexpr uint32_t kInf = 0x7f800000u;

// V consecutive elements <-> fp32. V = 8: 16-byte accesses; V = 2: one access of two elements.
template <class T, int V>
struct Io;
template <int V>
struct Io<float, V> {
    static __device__ __forceinline__ void load(const float* p, float (&f)[V]) {
        if constexpr (V == 8) {
            const uint4 a = ld_l2(reinterpret_cast<const uint4*>(p)), b = ld_l2(reinterpret_cast<const uint4*>(p) + 1);
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
        } else if constexpr (V == 2) {
            const uint2 a = ld_l2(reinterpret_cast<const uint2*>(p));
            f[0] = __uint_as_float(a.x), f[1] = __uint_as_float(a.y);
        } else {
            f[0] = ld_l2(p);
        }
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
    static __device__ __forceinline__ float round(float f) { return f; }
};
template <int V>
struct Io<__nv_bfloat16, V> {
    static __device__ __forceinline__ void load(const __nv_bfloat16* p, float (&f)[V]) {
        if constexpr (V == 8) {
            const uint4 a = ld_l2(reinterpret_cast<const uint4*>(p));
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        } else if constexpr (V == 2) {
            const uint32_t a = ld_l2(reinterpret_cast<const uint32_t*>(p));
            f[0] = __uint_as_float(a << 16), f[1] = __uint_as_float(a & 0xffff0000u);
        } else {
            f[0] = __uint_as_float(static_cast<uint32_t>(ld_l2(reinterpret_cast<const uint16_t*>(p))) << 16);
        }
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
    static __device__ __forceinline__ float round(float f) { return __bfloat162float(__float2bfloat16_rn(f)); }
};

template <int V>
__device__ __forceinline__ void load_weight(const void* w, bool bf16, int at, float (&f)[V]) {
    if (bf16) Io<__nv_bfloat16, V>::load(static_cast<const __nv_bfloat16*>(w) + at, f);
    else Io<float, V>::load(static_cast<const float*>(w) + at, f);
}

// The codes of p against inv = 127 / top: t = p inv is within 127 * 2^-23 of 127 p / top (two roundings), so the whole number
// nearest to it is the code unless t is near a border; there the two sides of the border are compared exactly (254 |p| and an odd
// number up to 253 times top have 32 bits each), ties to even.
struct Encoder {
    float f, inv;   // p f inv: f lifts rows whose 127 / top would not be finite
    double top;
    __device__ __forceinline__ explicit Encoder(float t) {
        f = t < 0x1p-60f ? 0x1p100f : 1.0f;
        inv = t > 0.0f ? 127.0f / (t * f) : 0.0f;
        top = static_cast<double>(t);
    }
    __device__ __forceinline__ uint32_t operator()(float p) const {
        constexpr float kWhole = 12582912.0f;  // 1.5 * 2^23: the sum's low bits are the whole number
        const float t = p * f * inv, s = __fadd_rn(t, kWhole), away = __fsub_rn(t, __fsub_rn(s, kWhole));
        uint32_t code = __float_as_uint(s);
        if (fabsf(away) > 0.5f - 0x1p-14f) {
            const int low = static_cast<int>(floorf(fabsf(t)));
            const double twice = 254.0 * fabs(static_cast<double>(p)), middle = (2 * low + 1) * top;
            const int q = low + ((twice > middle || (twice == middle && (low & 1))) ? 1 : 0);
            code = static_cast<uint32_t>(p < 0.0f ? -q : q);
        }
        return code & 0xffu;
    }
};

template <int V>
__device__ __forceinline__ void store_codes(int8_t* at, const Encoder& e, const float (&p)[V]) {
    uint32_t c[V];
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = e(p[i]);
    if constexpr (V == 8) {
        *reinterpret_cast<uint2*>(at) = make_uint2(c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24, c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24);
    } else if constexpr (V == 2) {
        *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(c[0] | c[1] << 8);
    } else {
        *at = static_cast<int8_t>(c[0]);
    }
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
__device__ __forceinline__ void load_total(const NormArgs& a, int64_t row, int at, float (&f)[V]) {
    Io<T, V>::load(static_cast<const T*>(a.x) + row * a.ldx + at, f);
    if (a.residual) {
        float r[V];
        Io<T, V>::load(static_cast<const T*>(a.residual) + row * a.ldr + at, r);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = Io<T, V>::round(f[i] + r[i]);
    }
}

// A row by a warp or a CTA, N accesses of V elements a thread, all in flight at once.
template <class T, int V, int N, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kWarpRows : kMaxThreads) norm_kernel(const NormArgs a) {
    __shared__ float2 part[32];
    const int team = WARP ? 32 : static_cast<int>(blockDim.x), tid = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    griddep_begin();
    if (WARP && row >= a.rows) return;
    const int D = a.D;
    float p[N][V];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int at = (tid + i * team) * V;
        if (at < D) load_total<T, V>(a, row, at, p[i]);
        else
#pragma unroll
            for (int j = 0; j < V; ++j) p[i][j] = 0.0f;
    }
    float sum = 0.0f;
    if (a.norm) {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) sum = fmaf(p[i][j], p[i][j], sum);
        if (a.total) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int at = (tid + i * team) * V;
                if (at < D) Io<T, V>::store(static_cast<T*>(a.total) + row * D + at, p[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = (tid + i * team) * V;
            if (at < D) {
                float w[V];
                load_weight<V>(a.weight, a.weight_bf16, at, w);
#pragma unroll
                for (int j = 0; j < V; ++j) p[i][j] = __fmul_rn(p[i][j], w[j]);
            }
        }
    }
    uint32_t top = 0;
    if (a.codes) {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) top = max(top, __float_as_uint(p[i][j]) & 0x7fffffffu);
    }
    reduce<WARP>(sum, top, part);
    const float rstd = row_rstd(a, sum);
    if (tid == 0) {
        if (a.rstd) a.rstd[row] = rstd;
        if (a.codes) a.scales[row] = row_scale(top, rstd);
    }
    if (a.codes) {
        const Encoder e(top >= kInf ? 0.0f : __uint_as_float(top));
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = (tid + i * team) * V;
            if (at >= D) continue;
            if (top >= kInf) {
                const float none[V] = {};
                store_codes<V>(a.codes + row * a.pitch + at, e, none);
            } else {
                store_codes<V>(a.codes + row * a.pitch + at, e, p[i]);
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
            Io<T, V>::store(static_cast<T*>(a.y) + row * D + at, p[i]);
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
    float sum = 0.0f, p[V], w[V];
    uint32_t top = 0;
    for (int64_t at = first; at < D; at += step) {
        load_total<T, V>(a, row, static_cast<int>(at), p);
        if (a.norm) {
#pragma unroll
            for (int j = 0; j < V; ++j) sum = fmaf(p[j], p[j], sum);
            if (a.total) Io<T, V>::store(static_cast<T*>(a.total) + row * D + at, p);
            load_weight<V>(a.weight, a.weight_bf16, static_cast<int>(at), w);
#pragma unroll
            for (int j = 0; j < V; ++j) p[j] = __fmul_rn(p[j], w[j]);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) top = max(top, __float_as_uint(p[j]) & 0x7fffffffu);
    }
    reduce<false>(sum, top, part);
    const float rstd = row_rstd(a, sum);
    if (threadIdx.x == 0) {
        if (a.rstd) a.rstd[row] = rstd;
        if (a.codes) a.scales[row] = row_scale(top, rstd);
    }
    const Encoder e(top >= kInf ? 0.0f : __uint_as_float(top));
    for (int64_t at = first; at < D; at += step) {
        if (a.norm && a.total) Io<T, V>::load(static_cast<const T*>(a.total) + row * D + at, p);
        else load_total<T, V>(a, row, static_cast<int>(at), p);
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
    int64_t ldy, ldt, ldd, rows;
    int D;
    bool weight_bf16;
};

// CTA b takes rows b, b + grid, ..: the weight and its gradient's sums stay in registers from row to row, the next row is loaded
// before the present one's sum is known, and the sums leave once, to the CTA's row of `partial`.
template <class T, int V, int N>
__global__ void __launch_bounds__(kMaxThreads) norm_backward_kernel(const NormBackwardArgs a) {
    __shared__ float part[2][32];
    const int tid = threadIdx.x, team = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = team >> 5, D = a.D;
    griddep_begin();
    float w[N][V], dw[N][V], t[N][V], g[N][V];
    auto load = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = (tid + i * team) * V;
            if (at < D) {
                Io<T, V>::load(static_cast<const T*>(a.total) + row * a.ldt + at, t[i]);
                Io<T, V>::load(static_cast<const T*>(a.dy) + row * a.ldy + at, g[i]);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) t[i][j] = g[i][j] = 0.0f;
            }
        }
    };
    int64_t row = blockIdx.x;
    load(row);
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
        const float r = rstd;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                n[i][j] = t[i][j] * r;
                dw[i][j] = fmaf(g[i][j], n[i][j], dw[i][j]);
                h[i][j] = g[i][j] * w[i][j];
                dot = fmaf(h[i][j], n[i][j], dot);
            }
        const int64_t now = row;
        row += gridDim.x;
        if (row < a.rows) {
            load(row);
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
                float d[V];
                Io<T, V>::load(static_cast<const T*>(a.dtotal) + now * a.ldd + at, d);
#pragma unroll
                for (int j = 0; j < V; ++j) h[i][j] += d[j];
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
            Io<T, V>::load(t + at, n);
            Io<T, V>::load(dy + at, g);
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
            Io<T, V>::load(t + at, n);
            Io<T, V>::load(dy + at, g);
            load_weight<V>(a.weight, a.weight_bf16, static_cast<int>(at), w);
#pragma unroll
            for (int j = 0; j < V; ++j) n[j] = r * (g[j] * w[j] - n[j] * r * mean);
            if (a.dtotal) {
                Io<T, V>::load(static_cast<const T*>(a.dtotal) + row * a.ldd + at, g);
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
#pragma unroll 4
        for (int r = warp; r < rows; r += 32) sum += ld_l2(partial + static_cast<int64_t>(r) * D + c);
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

// out[r][k] = codes[r][k] * scales[r]: V consecutive elements a thread and step.
template <class T, int V>
__global__ void __launch_bounds__(256) int8_dequantize_kernel(const int8_t* codes, int64_t pitch, const float* scales, int64_t rows,
                                                              int K, T* out) {
    constexpr int kSteps = 4;
    griddep_begin();
    const int first = (static_cast<int>(blockIdx.x) * kSteps * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * V;
    const int step = static_cast<int>(blockDim.x) * V;
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
        const uint8_t* c = reinterpret_cast<const uint8_t*>(codes) + row * pitch;
        uint32_t word[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int at = first + i * step;
            if (at < K) {
                if constexpr (V == 4) word[i] = ld_l2(reinterpret_cast<const uint32_t*>(c + at));
                else word[i] = ld_l2(c + at);
            }
        }
        const float scale = ld_l2(scales + row);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int at = first + i * step;
            if (at >= K) continue;
            float f[4];
#pragma unroll
            for (int j = 0; j < V; ++j) f[j] = static_cast<float>(static_cast<int8_t>(word[i] >> (8 * j))) * scale;
            T* o = out + row * K + at;
            if constexpr (V == 4 && sizeof(T) == 4) *reinterpret_cast<float4*>(o) = make_float4(f[0], f[1], f[2], f[3]);
            else if constexpr (V == 4) *reinterpret_cast<uint2*>(o) = make_uint2(f32x2_to_bf16x2(f[0], f[1]), f32x2_to_bf16x2(f[2], f[3]));
            else *o = T(f[0]);
        }
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

template <class T, int V>
cudaError_t run_norm(const NormArgs& a, cudaStream_t stream) {
    const int64_t D = a.D;
    auto block = [&](auto n) {
        constexpr int N = decltype(n)::value;
        return launch_dependent(norm_kernel<T, V, N, false>, static_cast<int>(a.rows), threads_for(D, V * N), stream, a);
    };
    if (D <= 256)
        return launch_dependent(norm_kernel<T, V, 8 / V, true>, static_cast<int>((a.rows + kWarpRows - 1) / kWarpRows), 32 * kWarpRows, stream, a);
    if (D <= 8 * kMaxThreads) return block(std::integral_constant<int, 8 / V>{});
    if (D <= 32 * kMaxThreads) return block(std::integral_constant<int, 32 / V>{});
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
int64_t backward_ctas(int64_t rows, int64_t D) {
    const int threads = D <= kBackwardRegs ? threads_for(D, 8) : kMaxThreads;
    return std::min<int64_t>(rows, static_cast<int64_t>(device_sm_count()) * std::max(1, std::min(16, kMaxThreads / threads)));
}

template <class T, int V>
cudaError_t run_backward(const NormBackwardArgs& a, int ctas, cudaStream_t stream) {
    if (a.D > kBackwardRegs) return launch_dependent(norm_backward_long_kernel<T, V>, ctas, kMaxThreads, stream, a);
    return launch_dependent(norm_backward_kernel<T, V, 8 / V>, ctas, threads_for(a.D, 8), stream, a);
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
    a.dx = dx, a.partial = dweight ? partial : nullptr;
    a.rows = rows, a.D = static_cast<int>(D);
    const int b = bf16 ? 2 : 4;
    const Rows views[] = {{dy.p, dy.ld, b}, {total.p, total.ld, b}, {dtotal.p, dtotal.ld, b}, {weight, 0, weight_bf16 ? 2 : 4}, {dx, D, b}};
    const int v = widest(views, D), ctas = static_cast<int>(backward_ctas(rows, D));
    cudaError_t e = cudaSuccess;
    if (ctas > 0) e = bf16 ? run_backward<__nv_bfloat16>(a, v, ctas, stream) : run_backward<float>(a, v, ctas, stream);
    if (e != cudaSuccess || !dweight) return e;
    return launch_dependent(norm_weight_kernel, static_cast<int>((D + 31) / 32), 1024, stream, partial, ctas, static_cast<int>(D), dweight);
}

cudaError_t launch_int8_dequantize(const int8_t* codes, int64_t pitch, const float* scales, int64_t rows, int64_t K, bool bf16, void* out,
                                   cudaStream_t stream) {
    const bool wide = K % 4 == 0 && pitch % 4 == 0 && reinterpret_cast<uintptr_t>(codes) % 4 == 0 &&
                      reinterpret_cast<uintptr_t>(out) % (bf16 ? 8 : 16) == 0;
    const int V = wide ? 4 : 1;
    const int threads = std::min(256, threads_for(K, V));
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3(static_cast<unsigned>((K + 4ll * threads * V - 1) / (4ll * threads * V)), static_cast<unsigned>(std::min<int64_t>(rows, 65535)));
    lc.blockDim = dim3(static_cast<unsigned>(threads));
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    const int k = static_cast<int>(K);
    if (bf16) {
        auto* o = static_cast<__nv_bfloat16*>(out);
        return wide ? cudaLaunchKernelEx(&lc, int8_dequantize_kernel<__nv_bfloat16, 4>, codes, pitch, scales, rows, k, o)
                    : cudaLaunchKernelEx(&lc, int8_dequantize_kernel<__nv_bfloat16, 1>, codes, pitch, scales, rows, k, o);
    }
    auto* o = static_cast<float*>(out);
    return wide ? cudaLaunchKernelEx(&lc, int8_dequantize_kernel<float, 4>, codes, pitch, scales, rows, k, o)
                : cudaLaunchKernelEx(&lc, int8_dequantize_kernel<float, 1>, codes, pitch, scales, rows, k, o);
}

}  // namespace pnq
