// pnq_fp4_api.cu -- the C ABI of the 4-bit microscaled operands and the expert layer (include/pnq.h):
// argument checks and status codes. Everything is checked before anything is launched.
#include "pnq.h"
#include "pnq_internal.h"

#include <cmath>
#include <cstdint>

using namespace pnq;

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 30;  // rows, expert rows and scale tiles are 32-bit in the kernels

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// The status of a launch. The launches keep what they asked of the device in maps under a mutex, which may throw where the host has
// no memory left: no exception leaves a C entry.
template <class F>
int launched(F&& launch) {
    try {
        return launch() == cudaSuccess ? PNQ_OK : PNQ_ERR_CUDA;
    } catch (...) {
        return PNQ_ERR_CUDA;
    }
}

bool is_fp4(int type) { return type == PNQ_NVFP4 || type == PNQ_MXFP4; }
bool is_float(int type) { return type == PNQ_F32 || type == PNQ_BF16; }
int group(int type) { return type == PNQ_MXFP4 ? 32 : 16; }

// Shape of `matrices` matrices of rows x K, and their scale blocks within the kernels' index range.
int check_shape(int type, int64_t rows, int64_t K, int64_t matrices) {
    if (!is_fp4(type)) return PNQ_ERR_TYPE;
    if (rows < 0 || matrices < 1 || K <= 0 || K > kMaxRows || K % group(type) != 0) return PNQ_ERR_SHAPE;
    if (rows > kMaxRows || matrices > kMaxRows || (rows + 127) / 128 * 128 > kMaxRows / matrices) return PNQ_ERR_SHAPE;
    if ((rows + 127) / 128 * matrices > kMaxRows / fp4_chunks(type == PNQ_MXFP4, K)) return PNQ_ERR_SHAPE;
    return PNQ_OK;
}

// Most 128-row blocks that n rows of `experts` experts take.
int64_t plan_blocks(int64_t n, int64_t experts) { return (n + 127 * (n < experts ? n : experts)) / 128; }

int check_plan(const pnq_expert_plan* d, PlanView* p) {
    if (!d) return PNQ_ERR_NULL;
    if (d->slots < 1 || d->slots > 64 || d->experts < 1 || d->experts > 1024 || d->tokens < 0 ||
        d->tokens > kMaxRows / d->slots)
        return PNQ_ERR_SHAPE;
    if (!d->offsets || !d->block_start) return PNQ_ERR_NULL;
    if (d->tokens > 0 && (!d->order || !d->position || !d->scale_row)) return PNQ_ERR_NULL;
    if (!aligned(d->offsets, 4) || !aligned(d->block_start, 4) || !aligned(d->order, 4) || !aligned(d->position, 4) ||
        !aligned(d->scale_row, 4))
        return PNQ_ERR_ALIGN;
    p->offsets = d->offsets;
    p->block_start = d->block_start;
    p->order = d->order;
    p->position = d->position;
    p->scale_row = d->scale_row;
    p->tokens = d->tokens;
    p->slots = d->slots;
    p->experts = d->experts;
    p->rows = static_cast<int>(d->tokens * d->slots);
    p->tiled = static_cast<int>(128 * plan_blocks(p->rows, d->experts));
    return PNQ_OK;
}

// The plan's rows as an operand's: their scale tiles within the kernels' index range.
int check_plan_rows(int type, const PlanView& p, int64_t K) {
    const int64_t n = p.tokens * p.slots;
    return plan_blocks(n, p.experts) > kMaxRows / fp4_chunks(type == PNQ_MXFP4, K) ? PNQ_ERR_SHAPE : PNQ_OK;
}

int check_operand(const void* codes, const void* scales) {
    if (!codes || !scales) return PNQ_ERR_NULL;
    return aligned(codes, 16) && aligned(scales, 16) ? PNQ_OK : PNQ_ERR_ALIGN;
}

int check_rows(int type, int64_t D, const pnq_expert_plan* plan, PlanView* p) {
    if (!is_float(type)) return PNQ_ERR_TYPE;
    const int rc = check_plan(plan, p);
    if (rc != PNQ_OK) return rc;
    return D < 1 || D > kMaxRows ? PNQ_ERR_SHAPE : PNQ_OK;
}

int check_elements(int type, std::initializer_list<const void*> ptrs) {
    for (const void* q : ptrs)
        if (!q) return PNQ_ERR_NULL;
    for (const void* q : ptrs)
        if (!aligned(q, type == PNQ_BF16 ? 2 : 4)) return PNQ_ERR_ALIGN;
    return PNQ_OK;
}

}  // namespace

extern "C" int pnq_fp4_layout(int type, int64_t rows, int64_t K, int64_t matrices, int64_t plan_experts,
                              uint64_t* pitch, uint64_t* scale_bytes) {
    const int rc = check_shape(type, rows, K, matrices);
    if (rc != PNQ_OK) return rc;
    if (plan_experts < 0 || plan_experts > 1024 || (plan_experts > 0 && matrices != 1)) return PNQ_ERR_SHAPE;
    if (!pitch || !scale_bytes) return PNQ_ERR_NULL;
    const int64_t blocks = plan_experts ? plan_blocks(rows, plan_experts) : (rows + 127) / 128 * matrices;
    *pitch = static_cast<uint64_t>(fp4_pitch(K));
    *scale_bytes = static_cast<uint64_t>(blocks * fp4_chunks(type == PNQ_MXFP4, K) * 512);
    return PNQ_OK;
}

extern "C" int pnq_fp4_quantize(int type, int x_type, const void* X, int64_t ldx, int64_t rows, int64_t K,
                                int64_t matrices, float global_scale, const pnq_expert_plan* plan, unsigned int flags,
                                uint8_t* codes, uint8_t* scales, cudaStream_t stream) {
    int rc = check_shape(type, rows, K, matrices);
    if (rc != PNQ_OK) return rc;
    if (!is_float(x_type)) return PNQ_ERR_TYPE;
    const bool sorted = (flags & PNQ_FP4_SORTED) != 0;
    if ((flags & ~static_cast<unsigned int>(PNQ_FP4_SORTED)) != 0 || (sorted && !plan)) return PNQ_ERR_FLAGS;
    if (ldx < K || ldx > INT64_MAX / 8 / (rows * matrices + 1)) return PNQ_ERR_SHAPE;
    const float inv_g = 1.0f / global_scale;
    if (!(global_scale > 0.0f) || !std::isfinite(global_scale) || !std::isfinite(inv_g)) return PNQ_ERR_VALUE;
    PlanView p{};
    if (plan) {
        rc = check_plan(plan, &p);
        if (rc != PNQ_OK) return rc;
        if (matrices != 1 || rows != (sorted ? p.tokens * p.slots : p.tokens)) return PNQ_ERR_SHAPE;
        rc = check_plan_rows(type, p, K);
        if (rc != PNQ_OK) return rc;
    }
    if (rows == 0) return PNQ_OK;
    if (!X) return PNQ_ERR_NULL;
    if (!aligned(X, x_type == PNQ_BF16 ? 2 : 4)) return PNQ_ERR_ALIGN;
    rc = check_operand(codes, scales);
    if (rc != PNQ_OK) return rc;
    return launched([&] {
        return launch_fp4_quantize(type == PNQ_MXFP4, x_type == PNQ_BF16, X, ldx, rows, K, matrices, inv_g, p, sorted, codes,
                                   scales, stream);
    });
}

extern "C" int pnq_fp4_dequantize(int type, const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K,
                                  int64_t matrices, float global_scale, const pnq_expert_plan* plan, int out_type,
                                  void* out, cudaStream_t stream) {
    int rc = check_shape(type, rows, K, matrices);
    if (rc != PNQ_OK) return rc;
    if (!is_float(out_type)) return PNQ_ERR_TYPE;
    PlanView p{};
    if (plan) {
        rc = check_plan(plan, &p);
        if (rc != PNQ_OK) return rc;
        if (matrices != 1 || rows != p.tokens * p.slots) return PNQ_ERR_SHAPE;
        rc = check_plan_rows(type, p, K);
        if (rc != PNQ_OK) return rc;
    }
    if (rows == 0) return PNQ_OK;
    rc = check_operand(codes, scales);
    if (rc != PNQ_OK) return rc;
    if (!out) return PNQ_ERR_NULL;
    if (!aligned(out, out_type == PNQ_BF16 ? 2 : 4)) return PNQ_ERR_ALIGN;
    return launched([&] {
        return launch_fp4_dequantize(type == PNQ_MXFP4, Fp4View{codes, scales, rows, matrices}, K, global_scale, p,
                                     out_type == PNQ_BF16, out, stream);
    });
}

extern "C" int pnq_fp4_pack(int type, const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K,
                            int64_t matrices, uint8_t* codes_out, uint8_t* scales_out, cudaStream_t stream) {
    int rc = check_shape(type, rows, K, matrices);
    if (rc != PNQ_OK) return rc;
    if (rows == 0) return PNQ_OK;
    if (!codes || !scales) return PNQ_ERR_NULL;
    if (codes_out == codes && K % 32 != 0) return PNQ_ERR_SHAPE;  // the rows' pitch changes: not in place
    rc = check_operand(codes_out, scales_out);
    if (rc != PNQ_OK) return rc;
    return launched([&] {
        return launch_fp4_pack(type == PNQ_MXFP4, codes, scales, rows, K, matrices, codes_out, scales_out, stream);
    });
}

extern "C" int pnq_fp4_gemm(int type, const uint8_t* x_codes, const uint8_t* x_scales, int64_t M, const uint8_t* w_codes,
                            const uint8_t* w_scales, int64_t N, int64_t K, float alpha, int y_type, void* Y,
                            unsigned int flags, cudaStream_t stream) {
    int rc = check_shape(type, M, K, 1);
    if (rc != PNQ_OK) return rc;
    rc = check_shape(type, N, K, 1);
    if (rc != PNQ_OK) return rc;
    if (!is_float(y_type)) return PNQ_ERR_TYPE;
    if ((flags & ~static_cast<unsigned int>(PNQ_GEMV_STATIC_WEIGHTS)) != 0) return PNQ_ERR_FLAGS;
    // the tiles of the launch are counted in 32 bits (64 x 128 the smallest)
    if (((M + 63) / 64) * ((N + 127) / 128) > kMaxRows) return PNQ_ERR_SHAPE;
    if (M == 0 || N == 0) return PNQ_OK;
    rc = check_operand(x_codes, x_scales);
    if (rc != PNQ_OK) return rc;
    rc = check_operand(w_codes, w_scales);
    if (rc != PNQ_OK) return rc;
    if (!Y) return PNQ_ERR_NULL;
    if (!aligned(Y, y_type == PNQ_BF16 ? 2 : 4)) return PNQ_ERR_ALIGN;
    return launched([&] {
        return launch_fp4_gemm(type == PNQ_MXFP4, Fp4View{x_codes, x_scales, M, 1}, Fp4View{w_codes, w_scales, N, 1}, K,
                               PlanView{}, alpha, nullptr, y_type == PNQ_BF16, Y, device_error_word(),
                               (flags & PNQ_GEMV_STATIC_WEIGHTS) != 0, stream);
    });
}

extern "C" int pnq_fp4_gemm_shape(int type, int64_t M, int64_t N, int64_t K, int32_t* columns, int32_t* ctas, int32_t* split) {
    int rc = check_shape(type, M, K, 1);
    if (rc != PNQ_OK) return rc;
    rc = check_shape(type, N, K, 1);
    if (rc != PNQ_OK) return rc;
    if (M == 0 || N == 0 || ((M + 63) / 64) * ((N + 127) / 128) > kMaxRows) return PNQ_ERR_SHAPE;
    if (!columns || !ctas || !split) return PNQ_ERR_NULL;
    return launched([&] { return fp4_gemm_shape(M, N, K, columns, ctas, split); });
}

extern "C" int pnq_fp4_gemm_experts(int type, const uint8_t* x_codes, const uint8_t* x_scales,
                                    const pnq_expert_plan* plan, const uint8_t* w_codes, const uint8_t* w_scales,
                                    int64_t N, int64_t K, float alpha, const float* w_global, int y_type, void* Y,
                                    unsigned int flags, cudaStream_t stream) {
    if (!is_fp4(type)) return PNQ_ERR_TYPE;
    PlanView p{};
    int rc = check_plan(plan, &p);
    if (rc != PNQ_OK) return rc;
    const int64_t n = p.tokens * p.slots;
    rc = check_shape(type, N, K, p.experts);
    if (rc != PNQ_OK) return rc;
    rc = check_plan_rows(type, p, K);
    if (rc != PNQ_OK) return rc;
    if (!is_float(y_type)) return PNQ_ERR_TYPE;
    if ((flags & ~static_cast<unsigned int>(PNQ_GEMV_STATIC_WEIGHTS)) != 0) return PNQ_ERR_FLAGS;
    if ((n / 64 + p.experts) * ((N + 127) / 128) > kMaxRows) return PNQ_ERR_SHAPE;
    if (n == 0 || N == 0) return PNQ_OK;
    rc = check_operand(x_codes, x_scales);
    if (rc != PNQ_OK) return rc;
    rc = check_operand(w_codes, w_scales);
    if (rc != PNQ_OK) return rc;
    if (!Y) return PNQ_ERR_NULL;
    if (!aligned(Y, y_type == PNQ_BF16 ? 2 : 4) || !aligned(w_global, 4)) return PNQ_ERR_ALIGN;
    return launched([&] {
        return launch_fp4_gemm(type == PNQ_MXFP4, Fp4View{x_codes, x_scales, n, 1}, Fp4View{w_codes, w_scales, N, p.experts},
                               K, p, alpha, w_global, y_type == PNQ_BF16, Y, device_error_word(),
                               (flags & PNQ_GEMV_STATIC_WEIGHTS) != 0, stream);
    });
}

extern "C" int pnq_expert_sort(const int32_t* ids, const pnq_expert_plan* plan, cudaStream_t stream) {
    PlanView p{};
    const int rc = check_plan(plan, &p);
    if (rc != PNQ_OK) return rc;
    if (p.tokens > 0 && !ids) return PNQ_ERR_NULL;
    if (!aligned(ids, 4)) return PNQ_ERR_ALIGN;
    return launched([&] { return launch_expert_sort(ids, p, stream); });
}

extern "C" int pnq_expert_gather(int type, const void* X, int64_t D, const pnq_expert_plan* plan, void* XS,
                                 cudaStream_t stream) {
    PlanView p{};
    int rc = check_rows(type, D, plan, &p);
    if (rc != PNQ_OK || p.tokens == 0) return rc;
    rc = check_elements(type, {X, XS});
    if (rc != PNQ_OK) return rc;
    return launched([&] {
        return launch_expert_rows(ExpertOp::Gather, type == PNQ_BF16, X, nullptr, D, p, nullptr, XS, nullptr, stream);
    });
}

extern "C" int pnq_expert_gather_backward(int type, const void* dXS, int64_t D, const pnq_expert_plan* plan, void* dX,
                                          cudaStream_t stream) {
    PlanView p{};
    int rc = check_rows(type, D, plan, &p);
    if (rc != PNQ_OK || p.tokens == 0) return rc;
    rc = check_elements(type, {dXS, dX});
    if (rc != PNQ_OK) return rc;
    return launched([&] {
        return launch_expert_rows(ExpertOp::GatherBackward, type == PNQ_BF16, dXS, nullptr, D, p, nullptr, dX, nullptr,
                                  stream);
    });
}

extern "C" int pnq_expert_combine(int type, const void* YS, int64_t D, const pnq_expert_plan* plan, const float* weights,
                                  void* Y, cudaStream_t stream) {
    PlanView p{};
    int rc = check_rows(type, D, plan, &p);
    if (rc != PNQ_OK || p.tokens == 0) return rc;
    rc = check_elements(type, {YS, Y, weights});
    if (rc != PNQ_OK) return rc;
    if (!aligned(weights, 4)) return PNQ_ERR_ALIGN;
    return launched([&] {
        return launch_expert_rows(ExpertOp::Combine, type == PNQ_BF16, YS, nullptr, D, p, weights, Y, nullptr, stream);
    });
}

extern "C" int pnq_expert_combine_backward(int type, const void* dY, const void* YS, int64_t D,
                                           const pnq_expert_plan* plan, const float* weights, void* dYS, float* dWeights,
                                           cudaStream_t stream) {
    PlanView p{};
    int rc = check_rows(type, D, plan, &p);
    if (rc != PNQ_OK || p.tokens == 0) return rc;
    rc = check_elements(type, {dY, YS, dYS, weights});
    if (rc != PNQ_OK) return rc;
    if (!aligned(weights, 4) || !aligned(dWeights, 4)) return PNQ_ERR_ALIGN;
    return launched([&] {
        return launch_expert_rows(ExpertOp::CombineBackward, type == PNQ_BF16, dY, YS, D, p, weights, dYS, dWeights,
                                  stream);
    });
}
