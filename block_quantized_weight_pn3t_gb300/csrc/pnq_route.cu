// pnq_route.cu -- routing to experts: scores of a token's logits, its experts in order, their weights, and the gradient of the
// logits (definitions in include/pnq.h). A warp takes a token; its scores stay in registers.
//
//   s = softmax(x) or 1 / (1 + exp(-x)), c = s + bias; of groups of experts the best by the sum of their largest c; then the
//   largest c in turn, ties to the lowest index; weights s, over their sum where renormalised, times a scale.
//
// Which of two scores is the larger must not hang on a rounding. Without bias and groups the logits themselves are compared. Otherwise
// c is computed in fp32 with a bound on its error (route_kernel), and a row in which two scores that decide anything are nearer than that,
// and are not of equal logits and equal biases, is done again with scores of some 2^-44 (four tokens in ten thousand of 256 experts with normal logits).
// Groups near each other are done again even where they are equal: a batch whose logits are all the same, with groups, goes there whole (route_kernel).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "pnq_device.cuh"
#include "pnq_internal.h"

namespace pnq {
namespace {

constexpr int kWarps = 4;          // of a CTA
constexpr int kCtas = 16;          // of an SM at most
constexpr int kScan = 32;          // tokens that a CTA of the second kernel looks through, one a lane of its first warp
constexpr int32_t kAgain = INT32_MIN;  // the first id of a token that the second kernel is to do
constexpr uint32_t kAll = 0xffffffffu;
constexpr float kNone = -INFINITY;  // the score of an expert that is out

struct RouteArgs {
    const void* logits;
    const float* bias;  // null: none
    int32_t* ids;
    float* weights;
    int64_t ld, tokens;
    int E, k, groups, per, top_groups, best;
    uint32_t per_magic;  // e / per = e * per_magic >> 20 for e < 1024
    float scale;
    bool sigmoid, renormalize;
};

// Elements e(i) of a lane: V consecutive ones of every run of 32 V.
template <int V>
__device__ __forceinline__ int element(int i, int lane) {
    return i / V * 32 * V + lane * V + i % V;
}

template <class T>
__device__ __forceinline__ float load_one(const T* p);
template <>
__device__ __forceinline__ float load_one(const float* p) { return ld_l2(p); }
template <>
__device__ __forceinline__ float load_one(const __nv_bfloat16* p) {
    return __uint_as_float(static_cast<uint32_t>(ld_l2(reinterpret_cast<const uint16_t*>(p))) << 16);
}

// Row x of E logits: what lies past E counts as -infinity.
template <class T, int NE, int V>
__device__ __forceinline__ void load_row(const T* row, int E, int lane, float (&x)[NE]) {
#pragma unroll
    for (int i = 0; i < NE; i += V) {
        const int e = element<V>(i, lane);
        if constexpr (V == 1) {
            x[i] = e < E ? load_one(row + e) : kNone;
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) x[i + j] = kNone;
            if (e < E) {
                if constexpr (sizeof(T) == 4) {
                    const uint4 w = ld_l2(reinterpret_cast<const uint4*>(row + e));
                    x[i] = __uint_as_float(w.x), x[i + 1] = __uint_as_float(w.y), x[i + 2] = __uint_as_float(w.z), x[i + 3] = __uint_as_float(w.w);
                } else {
                    const uint2 w = ld_l2(reinterpret_cast<const uint2*>(row + e));
                    x[i] = __uint_as_float(w.x << 16), x[i + 1] = __uint_as_float(w.x & 0xffff0000u);
                    x[i + 2] = __uint_as_float(w.y << 16), x[i + 3] = __uint_as_float(w.y & 0xffff0000u);
                }
            }
        }
    }
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}
// The largest of a warp's values in one instruction (no NaN among them). Volatile: all lanes have to meet in it where it stands.
__device__ __forceinline__ float redux_max(float v) {
    float d;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(v));
    return d;
}

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// ---- scores to some 2^-44, as unevaluated sums of two floats (T. J. Dekker 1971, D. E. Knuth) ---------------
// (64-bit arithmetic runs at 1/64 of the rate of 32-bit here: the same row took 15 us in doubles.)

struct Two {
    float hi, lo;  // |lo| <= half an ulp of hi
};
__device__ __forceinline__ Two two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two fast_sum(float a, float b) {  // |a| >= |b|
    const float s = __fadd_rn(a, b);
    return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
    const Two s = two_sum(a.hi, b.hi), t = two_sum(a.lo, b.lo), u = fast_sum(s.hi, __fadd_rn(s.lo, t.hi));
    return fast_sum(u.hi, __fadd_rn(u.lo, t.lo));
}
__device__ __forceinline__ Two operator*(Two a, Two b) {
    const float p = __fmul_rn(a.hi, b.hi);
    return fast_sum(p, fmaf(a.hi, b.lo, fmaf(a.lo, b.hi, fmaf(a.hi, b.hi, -p))));
}
__device__ __forceinline__ Two inverse(Two a) {  // Newton's step, 2 - a q, from the fp32 quotient
    const float q = __fdiv_rn(1.0f, a.hi), e = fmaf(-a.lo, q, fmaf(-a.hi, q, 1.0f));
    return fast_sum(q, __fmul_rn(q, e));
}

// log 2 in three parts (the reduction of W. J. Cody and W. Waite 1980): its first 17 bits, of which n times (7 bits) is exact, and what is left
// of it in two floats. kLog2Rest: log 2 less the double kLog2.
constexpr double kLog2 = 0.6931471805599453094, kLog2Rest = 2.3190468138462996e-17;
constexpr float kLog2High = static_cast<float>(static_cast<int>(kLog2 * 131072.0) / 131072.0);
constexpr float kLog2Middle = static_cast<float>(kLog2 - static_cast<double>(kLog2High));
constexpr float kLog2Low = static_cast<float>(kLog2 - static_cast<double>(kLog2High) - static_cast<double>(kLog2Middle) + kLog2Rest);

// exp(d) for d <= 0: d = n log 2 + r, the series of exp(r) (|r| <= 0.35; terms from r^8 / 8! on weigh below 2^-27, in fp32), times 2^n. Below
// 2^-125: zero.
__device__ __forceinline__ Two exp_two(Two d) {
    const bool none = !(d.hi > -86.6f);
    if (none) d = {0.0f, 0.0f};
    const float n = rintf(d.hi * 1.44269504f);
    const Two t = two_sum(d.hi, -n * kLog2High);
    const float p = __fmul_rn(n, kLog2Middle), e = fmaf(n, kLog2Middle, -p);
    const Two r = t + Two{-p, -e} + Two{d.lo, n * -kLog2Low};
    constexpr double kInverse[] = {1.0, 1.0, 1.0 / 2, 1.0 / 6, 1.0 / 24, 1.0 / 120, 1.0 / 720, 1.0 / 5040};  // 1 / k!
    const float x = r.hi;
    float high = 1.0f / 479001600;  // r^8 (1 / 8! + r / 9! + r^2 / 10! + r^3 / 11! + r^4 / 12!)
    high = fmaf(high, x, 1.0f / 39916800);
    high = fmaf(high, x, 1.0f / 3628800);
    high = fmaf(high, x, 1.0f / 362880);
    high = fmaf(high, x, 1.0f / 40320);
    Two sum{__fmul_rn(high, x), 0.0f};
#pragma unroll
    for (int k = 7; k >= 0; --k) {
        const float c = static_cast<float>(kInverse[k]), l = static_cast<float>(kInverse[k] - static_cast<double>(c));
        sum = sum + Two{c, l};
        if (k > 0) sum = sum * r;
    }
    const float scale = exp2i(static_cast<int>(n));  // n >= -125
    return {none ? 0.0f : sum.hi * scale, none ? 0.0f : sum.lo * scale};
}

// Whole numbers in the order of the values (-0 as +0).
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ uint64_t order_key(Two v) { return static_cast<uint64_t>(order_key(v.hi)) << 32 | order_key(v.lo); }
__device__ __forceinline__ Two key_value(uint64_t key) {
    auto value = [](uint32_t k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu)); };
    return {value(static_cast<uint32_t>(key >> 32)), value(static_cast<uint32_t>(key))};
}

// The weights of token t's experts, slots lane and lane + 32 of them in id, from its logits x in shared memory; m, sum: softmax's largest logit and
// divisor. Renormalised by the chosen experts alone, by their largest logit (so that no sum of theirs is too small to divide by).
__device__ __forceinline__ void write_weights(const RouteArgs& a, int64_t t, int (&id)[2], const float* x, float m, float sum, bool bad, int lane) {
    const int halves = a.k > 32 ? 2 : 1;
    float w[2] = {0.0f, 0.0f}, z[2], mc = kNone, total = 0.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (h >= halves) break;
        if (32 * h + lane >= a.k) id[h] = -1;
        z[h] = id[h] >= 0 ? x[id[h]] : kNone;
        mc = fmaxf(mc, z[h]);
    }
    if (a.renormalize) mc = redux_max(mc);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (h >= halves) break;
        if (id[h] >= 0) {
            if (a.sigmoid) w[h] = a.renormalize && mc < -60.0f ? expf(z[h] - mc) : sigmoid(z[h]);
            else w[h] = a.renormalize ? expf(z[h] - mc) : expf(z[h] - m) / sum;
        }
        total += w[h];
    }
    if (a.renormalize) total = warp_sum(total);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (32 * h + lane >= a.k) continue;
        const int64_t at = t * a.k + 32 * h + lane;
        float v = a.scale * w[h];
        if (a.renormalize && id[h] >= 0) v /= total;
        a.ids[at] = id[h];
        a.weights[at] = bad ? __uint_as_float(0x7fc00000u) : v;
    }
}

// Token t with such scores, by a whole CTA. c: E keys of shared memory (0: an expert that is out); x: the row's logits there. Equal
// scores go by the logits, then by the index.
__device__ __noinline__ void route_exact(const RouteArgs& a, int64_t t, const float* x, const float* bias, uint64_t* c) {
    __shared__ Two part[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Two scale{1.0f, 0.0f}, sum{1.0f, 0.0f};
    float top = kNone;
    if (!a.sigmoid) {
        for (int e = lane; e < a.E; e += 32) top = fmaxf(top, x[e]);
        top = redux_max(top);
        Two mine{0.0f, 0.0f};
        for (int e = tid; e < a.E; e += 32 * kWarps) {
            const Two z = exp_two(two_sum(fmaxf(x[e], -3e38f), -top));
            c[e] = static_cast<uint64_t>(__float_as_uint(z.hi)) << 32 | __float_as_uint(z.lo);
            mine = mine + z;
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) mine = mine + Two{__shfl_xor_sync(kAll, mine.hi, d), __shfl_xor_sync(kAll, mine.lo, d)};
        if (lane == 0) part[warp] = mine;
        __syncthreads();
        sum = (part[0] + part[1]) + (part[2] + part[3]);
        scale = inverse(sum);
    }
#pragma unroll 2
    for (int e = tid; e < a.E; e += 32 * kWarps) {  // two at a time, without branches: a score is some 200 instructions, one after the other
        const float b = a.bias ? bias[e] : 0.0f;
        Two s;
        if (a.sigmoid) {
            const float v = fmaxf(x[e], -3e38f);
            const Two z = exp_two({-fabsf(v), 0.0f}), w = inverse(z + Two{1.0f, 0.0f}), u = w * z;
            s = {v >= 0.0f ? w.hi : u.hi, v >= 0.0f ? w.lo : u.lo};
        } else {
            s = Two{__uint_as_float(static_cast<uint32_t>(c[e] >> 32)), __uint_as_float(static_cast<uint32_t>(c[e]))} * scale;
        }
        c[e] = x[e] == kNone || b == kNone ? 0 : order_key(s + Two{b, 0.0f});
    }
    __syncthreads();
    if (warp > 0) return;
    if (a.groups > 1) {
        // the largest power of two of lanes that a group can have: its best two by them
        const int lanes = 1 << (31 - __clz(32 / a.groups)), g = lane / lanes;
        uint64_t b1 = 0, b2 = 0;
        auto take = [&](uint64_t v) {
            if (v > b1) b2 = b1, b1 = v;
            else if (v > b2) b2 = v;
        };
        if (g < a.groups) {
            for (int j = lane & (lanes - 1); j < a.per; j += lanes) take(c[g * a.per + j]);
        }
        for (int d = lanes >> 1; d; d >>= 1) {
            const uint64_t o1 = __shfl_xor_sync(kAll, b1, d), o2 = __shfl_xor_sync(kAll, b2, d);
            take(o1);
            take(o2);
        }
        const uint64_t score = a.best == 2 && b2 ? order_key(key_value(b1) + key_value(b2)) : b1;
        int rank = 0;
        for (int h = 0; h < a.groups; ++h) {
            const uint64_t other = __shfl_sync(kAll, score, h * lanes);
            rank += other > score || (other == score && h < g);
        }
        const uint32_t kept = __ballot_sync(kAll, g < a.groups && rank < a.top_groups);
        for (int e = lane; e < a.E; e += 32)
            if (!(kept >> (e / a.per * lanes) & 1)) c[e] = 0;
        __syncwarp();
    }
    // each lane's best of its own (lane, lane + 32, ..); the winner's next is found by all lanes together, one of its experts each
    struct Best {
        uint32_t hi, lo, tie;  // the score in order, and the logit
        int at;
    };
    auto of = [&](int e) -> Best {
        const uint64_t key = e < a.E ? c[e] : 0;
        return {static_cast<uint32_t>(key >> 32), static_cast<uint32_t>(key), key ? order_key(x[e]) : 0, key ? e : 1 << 30};
    };
    auto largest = [&](Best b) -> Best {  // of the warp; at = 1 << 30 where none is left
        const uint32_t hi = __reduce_max_sync(kAll, b.hi), first = __ballot_sync(kAll, b.hi == hi);
        if ((first & (first - 1)) == 0) {
            const int from = __ffs(first) - 1;
            return {hi, __shfl_sync(kAll, b.lo, from), __shfl_sync(kAll, b.tie, from), __shfl_sync(kAll, b.at, from)};
        }
        bool in = b.hi == hi;
        const uint32_t lo = __reduce_max_sync(kAll, in ? b.lo : 0);
        in = in && b.lo == lo;
        const uint32_t tie = __reduce_max_sync(kAll, in ? b.tie : 0);
        in = in && b.tie == tie;
        return {hi, lo, tie, static_cast<int>(__reduce_min_sync(kAll, in ? static_cast<uint32_t>(b.at) : 1u << 30))};
    };
    Best mine = of(lane);
    for (int e = lane + 32; e < a.E; e += 32) {
        const Best b = of(e);
        if (b.hi > mine.hi || (b.hi == mine.hi && (b.lo > mine.lo || (b.lo == mine.lo && b.tie > mine.tie)))) mine = b;
    }
    int id[2] = {-1, -1};
    for (int j = 0; j < a.k; ++j) {
        const Best won = largest(mine);
        if (won.at >= a.E) break;  // no expert is left
        if (lane == j) id[0] = won.at;
        if (lane + 32 == j) id[1] = won.at;
        const int w = won.at & 31;
        if (lane == w) c[won.at] = 0;
        __syncwarp();
        const Best next = largest(of(w + 32 * lane));
        if (lane == w) mine = next;
    }
    write_weights(a, t, id, x, top, sum.hi, false, lane);
}

// The same with the row's logits loaded; x: shared memory of route_floats(E).
template <class T>
__device__ __forceinline__ void route_again(const RouteArgs& a, int64_t t, const float* bias, float* x) {
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    for (int e = threadIdx.x; e < a.E; e += 32 * kWarps) x[e] = load_one(row + e);
    __syncthreads();
    route_exact(a, t, x, bias, reinterpret_cast<uint64_t*>(x + (a.E + 3) / 4 * 4));
    __syncthreads();
}

// Shared memory of a warp: the row's logits, and behind them the groups' scores (each group on an odd pitch) or the keys above.
__host__ __device__ inline int route_floats(int E) { return (E + 3) / 4 * 4 * 3 + 32; }

// A warp takes token after token. Tokens with near scores (six of 16384 with normal logits) are done again by a whole CTA: HERE, where a warp has one token at
// most, at this kernel's end, otherwise by the kernel below. In the loop, by the warp that met them, the code for it alone cost every call 2 to 4
// us: 16384 x 256 sigmoid by the logits 18.1 us, now 15.6, 4096 x 256 with bias and 8 groups 16.2 and 13.6; 16384 of those 36.9 and 35.0, of which
// the second kernel is 9 (with 64 experts it takes 1.7 more than it saves). Where every token is near it takes most of the time: 16384 x 256 equal logits in 8
// groups 266 us, 4096 of them 46, 12 of 128 experts 28 (random ones 34, 16 and 5; equal logits without groups are ties, not near: 24, 10 and 5). The bias is read once a CTA: by every warp for every token, out of the
// same few lines of L2, it took more time than all the rest (25 of 45 us then).
// (Registers for eight CTAs an SM up to 256 experts: a token is a chain of some 3 us. With four CTAs fewer it took 4 to 12 percent longer.)
template <class T, int NE, int V, bool HERE>
__global__ void __launch_bounds__(32 * kWarps, NE <= 8 ? 8 : 4) route_kernel(const RouteArgs a) {
    extern __shared__ __align__(16) float shared[];
    __shared__ int64_t again[kWarps];  // HERE: a warp's token if it is to be done again, else -1
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* bs = shared;  // [E] bias, in whole 16 bytes
    float* xs = shared + (a.E + 3) / 4 * 4 + warp * route_floats(a.E);
    float* cs = xs + (a.E + 3) / 4 * 4;
    griddep_begin();
    int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
    const T* logits = static_cast<const T*>(a.logits);
    if (a.bias) {
        for (int e = threadIdx.x; e < a.E; e += 32 * kWarps) bs[e] = ld_l2(a.bias + e);
    }
    __syncthreads();
    const bool by_logit = !a.bias && a.groups == 1;
    float bmax = 0.0f;  // the largest finite |bias|
    if (a.bias) {
        for (int e = lane; e < a.E; e += 32)
            if (fabsf(bs[e]) < INFINITY) bmax = fmaxf(bmax, fabsf(bs[e]));
        bmax = redux_max(bmax);
    }
    const int pitch = a.per | 1;  // of a group in shared memory
    auto group = [&](int e) { return static_cast<int>(e * a.per_magic >> 20); };
    // a row's values to shared memory, in the experts' order
    auto keep = [&](float* to, const float (&v)[NE]) {
#pragma unroll
        for (int i = 0; i < NE; i += V) {
            const int e = element<V>(i, lane);
            if (e >= a.E) continue;
            if constexpr (V == 4) *reinterpret_cast<float4*>(to + e) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            else to[e] = v[i];
        }
    };
    if (HERE && lane == 0) again[warp] = -1;
    for (; t < a.tokens; t += step) {
        float x[NE];
        load_row<T, NE, V>(logits + t * a.ld, a.E, lane, x);
        __syncwarp();  // the last token's scores have been read
        keep(xs, x);

        // scores c; a NaN, or an infinity that is not an expert taken out, makes the whole row NaN
        float m = kNone, sum = 0.0f, smax = 1.0f, c[NE];
        bool bad = false;
        if (!a.sigmoid) {
#pragma unroll
            for (int i = 0; i < NE; ++i) m = fmaxf(m, x[i]);
            m = redux_max(m);
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                bad |= !(x[i] < INFINITY);
                c[i] = x[i] == kNone ? 0.0f : expf(x[i] - m);
                sum += c[i];
            }
            sum = warp_sum(sum);
            smax = sum > 0.0f ? 1.0f / sum : 0.0f;  // the score of the largest logit, if any expert is in
        } else {
#pragma unroll
            for (int i = 0; i < NE; ++i) bad |= isnan(x[i]);
        }
        if (by_logit) {
#pragma unroll
            for (int i = 0; i < NE; ++i) c[i] = x[i];
        } else {
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int e = element<V>(i, lane);
                float s = a.sigmoid ? __fdividef(1.0f, 1.0f + __expf(-x[i])) : c[i] * smax;  // 0 from a divisor of 2^126 on
                if (a.bias && e < a.E) s += bs[e];
                bad |= !(s < INFINITY);
                c[i] = x[i] == kNone ? kNone : s;
            }
        }
        bad = __any_sync(kAll, bad);

        int id[2] = {-1, -1};
        if (bad) {
            id[0] = lane, id[1] = lane + 32;
        } else {
            // How far two computed scores of different order may be apart. Sigmoid, in units of 2^-23: __expf is within (2 + 1.18 |x|) ulp, which moves s by
            // s (1 - s) (2 + 1.18 |x|) <= 0.63 (largest at |x| = 0.84); the sum with 1 rounds by half an ulp, 0.5 at most; the quotient is within 2 ulp, 1 where it is
            // below 1: s within 2.13, two of them 4.26, and the tolerance is 5.5. Softmax: an exponential is within 2^-22 of itself
            // and its argument's rounding adds (m - x) 2^-24; the sum, E / 32 + 5 additions of such, is within 1.5 * 2^-19 and moves a difference by
            // that times the larger score. The addition of the bias rounds by half an ulp of c.
            const float cmax = smax + bmax;
            const float tol = (a.sigmoid ? 0x1.6p-21f : 0x1p-18f * smax + 0x1p-24f) + 0x1p-23f * cmax;
            bool near = false;
            if (a.groups > 1) {
#pragma unroll
                for (int i = 0; i < NE; ++i) {
                    const int e = element<V>(i, lane);
                    if (e < a.E) cs[group(e) * (pitch - a.per) + e] = c[i];
                }
                __syncwarp();
                // the largest power of two of lanes that a group can have: its best two by them
                const int lanes = 1 << (31 - __clz(32 / a.groups)), g = lane / lanes;
                float b1 = kNone, b2 = kNone;
                if (g < a.groups) {
                    for (int j = lane & (lanes - 1); j < a.per; j += lanes) {
                        const float v = cs[g * pitch + j];
                        b2 = fmaxf(b2, fminf(b1, v));
                        b1 = fmaxf(b1, v);
                    }
                }
                for (int d = lanes >> 1; d; d >>= 1) {
                    const float o1 = __shfl_xor_sync(kAll, b1, d), o2 = __shfl_xor_sync(kAll, b2, d);
                    b2 = fmaxf(fmaxf(b2, o2), fminf(b1, o1));
                    b1 = fmaxf(b1, o1);
                }
                const float score = a.best == 2 && b2 != kNone ? b1 + b2 : b1;
                int rank = 0;
                for (int h = 0; h < a.groups; ++h) {
                    const float other = __shfl_sync(kAll, score, h * lanes);
                    rank += other > score || (other == score && h < g);
                }
                const bool stays = g < a.groups && rank < a.top_groups;
                const uint32_t kept = __ballot_sync(kAll, stays);
                const float least = -redux_max(stays ? -score : kNone), most = redux_max(g < a.groups && !stays ? score : kNone);
                near |= most != kNone && least - most <= 2.0f * tol + 0x1p-22f * cmax;
#pragma unroll
                for (int i = 0; i < NE; ++i) {
                    const int e = element<V>(i, lane);
                    if (e < a.E && !(kept >> (group(e) * lanes) & 1)) c[i] = kNone;
                }
                __syncwarp();  // the groups' scores have been read
            }
            // each lane's best and where it is. The winner's lane loses it, and its next is found by all lanes together, one of its experts each (by
            // that lane alone, the others waiting, selection took twice the instructions)
            keep(cs, c);
            float mine = kNone, won[2] = {kNone, kNone};
            int mine_at = a.E;
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (c[i] > mine) mine = c[i], mine_at = element<V>(i, lane);
            __syncwarp();
            for (int j = 0; j < a.k; ++j) {
                const float most = redux_max(mine);
                if (!(most > kNone)) break;  // no expert is left
                const uint32_t ties = __ballot_sync(kAll, mine == most);
                int e = __shfl_sync(kAll, mine_at, __ffs(ties) - 1);
                if (ties & (ties - 1)) e = static_cast<int>(__reduce_min_sync(kAll, mine == most ? static_cast<uint32_t>(mine_at) : 0xffffffffu));
                const int owner = e / V & 31, own = element<V>(lane, owner);
                if (lane == owner) cs[e] = kNone;
                __syncwarp();
                const float v = lane < NE && own < a.E ? cs[own] : kNone, next = redux_max(v);
                const int next_at = element<V>(__ffs(__ballot_sync(kAll, v == next)) - 1, owner);
                if (lane == owner) mine = next, mine_at = next_at;
                if (lane == j) id[0] = e, won[0] = most;
                if (lane + 32 == j) id[1] = e, won[1] = most;
            }
            if (!by_logit) {
                // neighbours in order, and the last against what is left: near, and not the same logit with the same bias
                const float left = redux_max(mine);
                auto same = [&](int e, int f) { return xs[e] == xs[f] && (!a.bias || bs[e] == bs[f]); };
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int j = 32 * h + lane;
                    const float next = __shfl_sync(kAll, h == 0 && lane == 0 ? won[1] : won[h], (lane + 1) & 31);
                    const int next_id = __shfl_sync(kAll, h == 0 && lane == 0 ? id[1] : id[h], (lane + 1) & 31);
                    if (j + 1 < a.k && next != kNone && won[h] - next <= tol) near |= !same(id[h], next_id);
                }
                const int last = a.k - 1;
                const float final_won = __shfl_sync(kAll, last < 32 ? won[0] : won[1], last & 31);
                const int final_id = __shfl_sync(kAll, last < 32 ? id[0] : id[1], last & 31);
                if (final_won != kNone && left != kNone && final_won - left <= tol) {
                    for (int e = lane; e < a.E; e += 32)
                        if (cs[e] != kNone && final_won - cs[e] <= tol) near |= !same(e, final_id);
                }
                if (__any_sync(kAll, near)) {
                    if (lane == 0) {
                        if constexpr (HERE) again[warp] = t;
                        else a.ids[t * a.k] = kAgain;
                    }
                    continue;
                }
            }
        }

        __syncwarp();
        write_weights(a, t, id, xs, m, sum, bad, lane);
    }
    if constexpr (HERE) {
        __syncthreads();
        for (int w = 0; w < kWarps; ++w)
            if (again[w] >= 0) route_again<T>(a, again[w], bs, shared + (a.E + 3) / 4 * 4);
    }
}

// The tokens that the kernel above left: a CTA looks through kScan of them at a time.
template <class T>
__global__ void __launch_bounds__(32 * kWarps) route_again_kernel(const RouteArgs a) {
    extern __shared__ __align__(16) float shared[];
    __shared__ uint32_t marked;
    bool bias = false;
    griddep_begin();
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kScan; t0 < a.tokens; t0 += static_cast<int64_t>(gridDim.x) * kScan) {
        if (threadIdx.x < 32) {
            const int64_t t = t0 + threadIdx.x;
            const uint32_t mask = __ballot_sync(kAll, t < a.tokens && ld_l2(a.ids + t * a.k) == kAgain);
            if (threadIdx.x == 0) marked = mask;
        }
        __syncthreads();
        uint32_t mask = marked;
        if (mask && a.bias && !bias) {
            for (int e = threadIdx.x; e < a.E; e += 32 * kWarps) shared[e] = ld_l2(a.bias + e);
            bias = true;
        }
        for (; mask; mask &= mask - 1) route_again<T>(a, t0 + __ffs(mask) - 1, shared, shared + (a.E + 3) / 4 * 4);
        __syncthreads();  // marked has been read
    }
}

// ---- gradient -------------------------------------------------------------------------------------------

struct RouteBackwardArgs {
    const float* dweights;
    const void* logits;
    const int32_t* ids;
    void* dlogits;
    int64_t ld, tokens;
    int E, k;
    float scale;
    bool sigmoid, renormalize;
};

// dlogits of a token by a warp. Renormalised weights hang on the chosen logits alone: r = their shares, softmax scale r (dw - <dw, r>),
// sigmoid times 1 - s besides; the rest is zeros. Sigmoid: scale dw s (1 - s). Softmax: s (g - <g, s>) over the row, g = scale dw at the
// chosen. An expert named twice gets both, in slot order.
template <class T, int NE, int V>
__global__ void __launch_bounds__(32 * kWarps) route_backward_kernel(const RouteBackwardArgs a) {
    extern __shared__ __align__(16) float shared[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* g = shared + warp * a.E;
    griddep_begin();
    const bool whole = !a.sigmoid && !a.renormalize;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < a.tokens; t += static_cast<int64_t>(gridDim.x) * kWarps) {
        const T* row = static_cast<const T*>(a.logits) + t * a.ld;
        float x[NE];
        if (whole) load_row<T, NE, V>(row, a.E, lane, x);
        int id[2];
        float dw[2], z[2], q[2], mc = kNone;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = 32 * h + lane;
            id[h] = j < a.k ? plan_index(ld_l2(a.ids + t * a.k + j), a.E) : -1;
            dw[h] = id[h] >= 0 ? ld_l2(a.dweights + t * a.k + j) : 0.0f;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            z[h] = id[h] >= 0 ? load_one(row + id[h]) : kNone;
            mc = fmaxf(mc, z[h]);
        }
        for (int e = lane; e < a.E; e += 32) g[e] = 0.0f;
        __syncwarp();
        if (a.renormalize) {
            mc = warp_max(mc);
            float total = 0.0f, dot = 0.0f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                q[h] = 0.0f;
                if (id[h] >= 0) q[h] = a.sigmoid && !(mc < -60.0f) ? sigmoid(z[h]) : expf(z[h] - mc);
                total += q[h];
            }
            total = warp_sum(total);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (id[h] >= 0) q[h] /= total;
                dot = fmaf(q[h], dw[h], dot);
            }
            dot = warp_sum(dot);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                q[h] = a.scale * q[h] * (dw[h] - dot);
                if (a.sigmoid && id[h] >= 0) q[h] *= sigmoid(-z[h]);
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                q[h] = a.scale * dw[h];
                if (a.sigmoid && id[h] >= 0) q[h] *= sigmoid(z[h]) * sigmoid(-z[h]);
            }
        }
        for (int j = 0; j < a.k; ++j) {
            const int e = __shfl_sync(kAll, j < 32 ? id[0] : id[1], j & 31);
            const float v = __shfl_sync(kAll, j < 32 ? q[0] : q[1], j & 31);
            if (e >= 0 && lane == (e & 31)) g[e] += v;
        }
        __syncwarp();
        float out[NE];
        if (whole) {
            float m = kNone, sum = 0.0f, dot = 0.0f;
#pragma unroll
            for (int i = 0; i < NE; ++i) m = fmaxf(m, x[i]);
            m = warp_max(m);
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                x[i] = x[i] == kNone ? 0.0f : expf(x[i] - m);
                sum += x[i];
            }
            sum = warp_sum(sum);
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int e = element<V>(i, lane);
                x[i] = m == kNone ? 0.0f : x[i] / sum;  // no expert at all: zeros
                out[i] = e < a.E ? g[e] : 0.0f;
                dot = fmaf(x[i], out[i], dot);
            }
            dot = warp_sum(dot);
#pragma unroll
            for (int i = 0; i < NE; ++i) out[i] = x[i] * (out[i] - dot);
        } else {
#pragma unroll
            for (int i = 0; i < NE; ++i) out[i] = element<V>(i, lane) < a.E ? g[element<V>(i, lane)] : 0.0f;
        }
        T* to = static_cast<T*>(a.dlogits) + t * a.E;
#pragma unroll
        for (int i = 0; i < NE; i += V) {
            const int e = element<V>(i, lane);
            if (e >= a.E) continue;
            if constexpr (V == 1) to[e] = T(out[i]);
            else if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(to + e) = make_float4(out[i], out[i + 1], out[i + 2], out[i + 3]);
            else *reinterpret_cast<uint2*>(to + e) = make_uint2(f32x2_to_bf16x2(out[i], out[i + 1]), f32x2_to_bf16x2(out[i + 2], out[i + 3]));
        }
        __syncwarp();  // the row's sums have been read
    }
}

// `floats` of shared memory, `tokens` to a CTA at a time. As many CTAs as keep the SMs full (and no more than there are tokens for).
template <class Kernel, class Args>
cudaError_t launch_rows(Kernel kernel, const Args& a, int floats, int tokens, cudaStream_t stream) {
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>((a.tokens + tokens - 1) / tokens, static_cast<int64_t>(device_sm_count()) * kCtas)));
    lc.blockDim = dim3(32 * kWarps);
    lc.dynamicSmemBytes = static_cast<size_t>(floats) * 4;
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    if (lc.dynamicSmemBytes > 48 * 1024) {
        const cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(kernel), static_cast<int>(lc.dynamicSmemBytes));
        if (e != cudaSuccess) return e;
    }
    return cudaLaunchKernelEx(&lc, kernel, a);
}

// go(elements a lane, elements an access) with both as types: the fewest registers that hold a row.
template <class F>
cudaError_t by_experts(int E, bool wide, F&& go) {
    auto with = [&](auto v) {
        if (E <= 128) return go(std::integral_constant<int, 4>{}, v);
        if (E <= 256) return go(std::integral_constant<int, 8>{}, v);
        if (E <= 512) return go(std::integral_constant<int, 16>{}, v);
        return go(std::integral_constant<int, 32>{}, v);
    };
    return wide ? with(std::integral_constant<int, 4>{}) : with(std::integral_constant<int, 1>{});
}

bool aligned4(const void* p, int64_t ld, int E, bool bf16) {
    return E % 4 == 0 && ld % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (bf16 ? 8 : 16) == 0;
}

}  // namespace

cudaError_t launch_expert_route(bool bf16, const RowsView& logits, int64_t tokens, const RouteRule& rule, const float* bias, int32_t* ids,
                                float* weights, cudaStream_t stream) {
    RouteArgs a{};
    a.logits = logits.p, a.ld = logits.ld, a.tokens = tokens;
    a.bias = bias, a.ids = ids, a.weights = weights;
    a.E = rule.experts, a.k = rule.slots, a.groups = rule.groups, a.per = rule.experts / rule.groups;
    a.top_groups = rule.top_groups, a.best = rule.best;
    a.per_magic = static_cast<uint32_t>(((1 << 20) + a.per - 1) / a.per);
    a.scale = rule.scale, a.sigmoid = rule.sigmoid, a.renormalize = rule.renormalize;
    // by the logits alone no token is done again; few tokens, one a warp, end in one launch
    const bool by_logit = !bias && rule.groups == 1, here = !by_logit && tokens <= std::min(4096, kWarps * kCtas * device_sm_count());
    const int whole = (a.E + 3) / 4 * 4;
    const cudaError_t e = by_experts(a.E, aligned4(logits.p, logits.ld, a.E, bf16), [&](auto n, auto v) {
        constexpr int NE = decltype(n)::value, V = decltype(v)::value;
        const int floats = whole + kWarps * route_floats(a.E);
        if (here) return launch_rows(bf16 ? route_kernel<__nv_bfloat16, NE, V, true> : route_kernel<float, NE, V, true>, a, floats, kWarps, stream);
        return launch_rows(bf16 ? route_kernel<__nv_bfloat16, NE, V, false> : route_kernel<float, NE, V, false>, a, floats, kWarps, stream);
    });
    if (e != cudaSuccess || here || by_logit) return e;
    return launch_rows(bf16 ? route_again_kernel<__nv_bfloat16> : route_again_kernel<float>, a, whole + route_floats(a.E), kScan, stream);
}

cudaError_t launch_expert_route_backward(bool bf16, const float* dweights, const RowsView& logits, const int32_t* ids, int64_t tokens,
                                         const RouteRule& rule, void* dlogits, cudaStream_t stream) {
    RouteBackwardArgs a{};
    a.dweights = dweights, a.logits = logits.p, a.ld = logits.ld, a.ids = ids, a.dlogits = dlogits, a.tokens = tokens;
    a.E = rule.experts, a.k = rule.slots;
    a.scale = rule.scale, a.sigmoid = rule.sigmoid, a.renormalize = rule.renormalize;
    const bool wide = aligned4(logits.p, logits.ld, a.E, bf16) && aligned4(dlogits, a.E, a.E, bf16);
    return by_experts(a.E, wide, [&](auto n, auto v) {
        constexpr int NE = decltype(n)::value, V = decltype(v)::value;
        return launch_rows(bf16 ? route_backward_kernel<__nv_bfloat16, NE, V> : route_backward_kernel<float, NE, V>, a, kWarps * a.E, kWarps, stream);
    });
}

}  // namespace pnq
