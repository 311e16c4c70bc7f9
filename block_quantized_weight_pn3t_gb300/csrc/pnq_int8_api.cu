// pnq_int8_api.cu -- the C ABI of the norms, the 8-bit rows and their products, and the routing to experts (include/pnq.h):
// argument checks and status codes. Everything is checked before anything is launched.
#include "pnq.h"
#include "pnq_internal.h"

#include <cmath>
#include <cstdint>
#include <initializer_list>

using namespace pnq;

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 30;  // rows, columns and tiles are 32-bit in the kernels
constexpr int64_t kMaxK = 131071;               // K 2^14 stays below 2^31

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool is_float(int type) { return type == PNQ_F32 || type == PNQ_BF16; }
uintptr_t size_of(int type) { return type == PNQ_BF16 ? 2 : 4; }

// The status of a launch: no exception leaves a C entry (what was asked of the device is kept in maps, which may throw).
template <class F>
int launched(F&& launch) {
    try {
        return launch() == cudaSuccess ? PNQ_OK : PNQ_ERR_CUDA;
    } catch (...) {
        return PNQ_ERR_CUDA;
    }
}

// rows x D elements, rows `ld` apart: offsets stay within 64 bits.
bool fits(int64_t rows, int64_t D, int64_t ld) {
    return rows >= 0 && rows <= kMaxRows && D >= 1 && D <= kMaxRows && ld >= D && ld <= INT64_MAX / 8 / (rows + 1);
}

// Whether a contiguous [rows][D] result may stand where rows of an operand do: in their own place, row for row, or apart from them.
bool apart(const void* out, const RowsView& in, int64_t rows, int64_t D, uintptr_t bytes) {
    if (!out || !in.p) return true;
    const uintptr_t o = reinterpret_cast<uintptr_t>(out), i = reinterpret_cast<uintptr_t>(in.p);
    const uintptr_t length = static_cast<uintptr_t>(D) * bytes, step = static_cast<uintptr_t>(in.ld) * bytes, n = static_cast<uintptr_t>(rows);
    const uintptr_t r = i + length > o ? 0 : (o - i - length) / step + 1;  // the operand's first row that ends behind the result's start
    return r >= n || i + r * step >= o + n * length;
}
bool in_place_or_apart(const void* out, const RowsView& in, int64_t rows, int64_t D, uintptr_t bytes) {
    return (out == in.p && (in.ld == D || rows == 1)) || apart(out, in, rows, D, bytes);
}

int check_rule(const pnq_route_rule* r, int64_t tokens, RouteRule* out) {
    if (!r) return PNQ_ERR_NULL;
    if (r->score != PNQ_SOFTMAX && r->score != PNQ_SIGMOID) return PNQ_ERR_TYPE;
    if (r->experts < 1 || r->experts > 1024 || r->groups < 1 || r->groups > 32 || r->experts % r->groups != 0 || r->top_groups < 1 ||
        r->top_groups > r->groups || r->best < 1 || r->best > 2 || r->slots < 1 || r->slots > 64 ||
        r->slots > r->experts / r->groups * r->top_groups || tokens < 0 || tokens > kMaxRows / r->slots)
        return PNQ_ERR_SHAPE;
    if (!std::isfinite(r->scale)) return PNQ_ERR_VALUE;
    *out = RouteRule{r->experts, r->slots, r->groups, r->top_groups, r->best, r->score == PNQ_SIGMOID, r->renormalize != 0, r->scale};
    return PNQ_OK;
}

}  // namespace

extern "C" int pnq_expert_route(int type, const void* logits, int64_t ld, int64_t tokens, const pnq_route_rule* rule, const float* bias,
                                int32_t* ids, float* weights, cudaStream_t stream) {
    if (!is_float(type)) return PNQ_ERR_TYPE;
    RouteRule r{};
    const int rc = check_rule(rule, tokens, &r);
    if (rc != PNQ_OK) return rc;
    if (!fits(tokens, r.experts, ld)) return PNQ_ERR_SHAPE;
    if (tokens == 0) return PNQ_OK;
    if (!logits || !ids || !weights) return PNQ_ERR_NULL;
    if (!aligned(logits, size_of(type)) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4)) return PNQ_ERR_ALIGN;
    return launched([&] { return launch_expert_route(type == PNQ_BF16, RowsView{logits, ld}, tokens, r, bias, ids, weights, stream); });
}

extern "C" int pnq_expert_route_backward(int type, const float* dweights, const void* logits, int64_t ld, const int32_t* ids,
                                         int64_t tokens, const pnq_route_rule* rule, void* dlogits, cudaStream_t stream) {
    if (!is_float(type)) return PNQ_ERR_TYPE;
    RouteRule r{};
    const int rc = check_rule(rule, tokens, &r);
    if (rc != PNQ_OK) return rc;
    if (!fits(tokens, r.experts, ld)) return PNQ_ERR_SHAPE;
    if (tokens == 0) return PNQ_OK;
    if (!dweights || !logits || !ids || !dlogits) return PNQ_ERR_NULL;
    if (!aligned(logits, size_of(type)) || !aligned(dlogits, size_of(type)) || !aligned(ids, 4) || !aligned(dweights, 4)) return PNQ_ERR_ALIGN;
    if (!in_place_or_apart(dlogits, RowsView{logits, ld}, tokens, r.experts, size_of(type))) return PNQ_ERR_VALUE;
    return launched(
        [&] { return launch_expert_route_backward(type == PNQ_BF16, dweights, RowsView{logits, ld}, ids, tokens, r, dlogits, stream); });
}

extern "C" int pnq_rms_norm(int type, const void* X, int64_t ldx, const void* residual, int64_t ldr, int64_t rows, int64_t D,
                            int weight_type, const void* weight, float eps, void* total, void* y, float* rstd, int8_t* codes,
                            int64_t pitch, float* scales, cudaStream_t stream) {
    if (!is_float(type) || !is_float(weight_type)) return PNQ_ERR_TYPE;
    if (!fits(rows, D, ldx) || (residual && !fits(rows, D, ldr))) return PNQ_ERR_SHAPE;
    if (codes && (!fits(rows, D, pitch) || pitch % 16 != 0)) return PNQ_ERR_SHAPE;
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return PNQ_ERR_VALUE;
    if (rows == 0) return PNQ_OK;
    if (!X || !weight || (codes == nullptr) != (scales == nullptr) || (!total && !y && !rstd && !codes)) return PNQ_ERR_NULL;
    const uintptr_t b = size_of(type);
    if (!aligned(X, b) || !aligned(residual, b) || !aligned(total, b) || !aligned(y, b) || !aligned(weight, size_of(weight_type)) ||
        !aligned(rstd, 4) || !aligned(scales, 4) || !aligned(codes, 16))
        return PNQ_ERR_ALIGN;
    for (const void* out : {total, y})
        if (!in_place_or_apart(out, RowsView{X, ldx}, rows, D, b) || !in_place_or_apart(out, RowsView{residual, ldr}, rows, D, b)) return PNQ_ERR_VALUE;
    if (!apart(total, RowsView{y, D}, rows, D, b)) return PNQ_ERR_VALUE;
    return launched([&] {
        return launch_rms_norm(type == PNQ_BF16, RowsView{X, ldx}, RowsView{residual, ldr}, weight_type == PNQ_BF16, weight, eps, rows, D,
                               total, y, rstd, codes, pitch, scales, stream);
    });
}

extern "C" int pnq_rms_norm_backward_scratch_bytes(int64_t rows, int64_t D, uint64_t* bytes) {
    if (!fits(rows, D, D)) return PNQ_ERR_SHAPE;
    if (!bytes) return PNQ_ERR_NULL;
    *bytes = static_cast<uint64_t>(rms_norm_backward_rows(rows, D)) * static_cast<uint64_t>(D) * 4;
    return PNQ_OK;
}

extern "C" int pnq_rms_norm_backward(int type, const void* dY, int64_t ldy, const void* total, int64_t ldt, int weight_type,
                                     const void* weight, const float* rstd, const void* dtotal, int64_t ldd, int64_t rows, int64_t D,
                                     void* dX, float* dweight, void* scratch, uint64_t scratch_bytes, cudaStream_t stream) {
    if (!is_float(type) || !is_float(weight_type)) return PNQ_ERR_TYPE;
    if (!fits(rows, D, ldy) || !fits(rows, D, ldt) || (dtotal && !fits(rows, D, ldd))) return PNQ_ERR_SHAPE;
    if (rows == 0 && !dweight) return PNQ_OK;
    if (rows > 0 && (!dY || !total || !weight || !rstd || !dX || (dweight && !scratch))) return PNQ_ERR_NULL;
    const uintptr_t b = size_of(type);
    if (!aligned(dY, b) || !aligned(total, b) || !aligned(dtotal, b) || !aligned(dX, b) || !aligned(weight, size_of(weight_type)) ||
        !aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(scratch, 4))
        return PNQ_ERR_ALIGN;
    uint64_t need = 0;
    const int rc = pnq_rms_norm_backward_scratch_bytes(rows, D, &need);
    if (rc != PNQ_OK) return rc;
    if (dweight && scratch_bytes < need) return PNQ_ERR_SCRATCH;
    // the weight's gradient may be summed from rows whose dX is written
    if (rows > 0 && (!apart(dX, RowsView{dY, ldy}, rows, D, b) || !apart(dX, RowsView{total, ldt}, rows, D, b) ||
                     !in_place_or_apart(dX, RowsView{dtotal, ldd}, rows, D, b)))
        return PNQ_ERR_VALUE;
    return launched([&] {
        return launch_rms_norm_backward(type == PNQ_BF16, RowsView{dY, ldy}, RowsView{total, ldt}, weight_type == PNQ_BF16, weight, rstd,
                                        RowsView{dtotal, ldd}, rows, D, dX, dweight, static_cast<float*>(scratch), stream);
    });
}

extern "C" int pnq_int8_quantize(int type, const void* X, int64_t ldx, int64_t rows, int64_t K, int8_t* codes, int64_t pitch,
                                 float* scales, cudaStream_t stream) {
    if (!is_float(type)) return PNQ_ERR_TYPE;
    if (!fits(rows, K, ldx) || !fits(rows, K, pitch) || pitch % 16 != 0) return PNQ_ERR_SHAPE;
    if (rows == 0) return PNQ_OK;
    if (!X || !codes || !scales) return PNQ_ERR_NULL;
    if (!aligned(X, size_of(type)) || !aligned(codes, 16) || !aligned(scales, 4)) return PNQ_ERR_ALIGN;
    return launched([&] { return launch_int8_quantize(type == PNQ_BF16, RowsView{X, ldx}, rows, K, codes, pitch, scales, stream); });
}

extern "C" int pnq_int8_dequantize(const int8_t* codes, int64_t pitch, const float* scales, int64_t rows, int64_t K, int out_type,
                                   void* out, cudaStream_t stream) {
    if (!is_float(out_type)) return PNQ_ERR_TYPE;
    if (!fits(rows, K, pitch)) return PNQ_ERR_SHAPE;
    if (rows == 0) return PNQ_OK;
    if (!codes || !scales || !out) return PNQ_ERR_NULL;
    if (!aligned(scales, 4) || !aligned(out, size_of(out_type))) return PNQ_ERR_ALIGN;
    return launched([&] { return launch_int8_dequantize(codes, pitch, scales, rows, K, out_type == PNQ_BF16, out, stream); });
}

extern "C" int pnq_int8_gemm_scratch_bytes(int64_t M, const int8_t* W, int64_t ldw, int64_t N, int64_t K, uint64_t* bytes) {
    if (K > kMaxK || !fits(M, K, K) || !fits(N, K, ldw)) return PNQ_ERR_SHAPE;
    if (!bytes) return PNQ_ERR_NULL;
    *bytes = int8_gemm_scratch(M, Int8View{W, ldw, nullptr, N}, K);
    return PNQ_OK;
}

extern "C" int pnq_int8_gemm(const int8_t* X, int64_t ldx, const float* x_scales, int64_t M, const int8_t* W, int64_t ldw,
                             const float* w_scales, int64_t N, int64_t K, int y_type, void* Y, void* scratch, uint64_t scratch_bytes,
                             cudaStream_t stream) {
    if (!is_float(y_type)) return PNQ_ERR_TYPE;
    if (K > kMaxK || !fits(M, K, ldx) || !fits(N, K, ldw)) return PNQ_ERR_SHAPE;
    if ((M + 15) / 16 * ((N + 127) / 128) > kMaxRows) return PNQ_ERR_SHAPE;  // tiles are counted in 32 bits (16 x 128 the smallest)
    if (M == 0 || N == 0) return PNQ_OK;
    if (!X || !x_scales || !W || !w_scales || !Y) return PNQ_ERR_NULL;
    if (!aligned(x_scales, 4) || !aligned(w_scales, 4) || !aligned(Y, size_of(y_type))) return PNQ_ERR_ALIGN;
    const uint64_t need = int8_gemm_scratch(M, Int8View{W, ldw, w_scales, N}, K);
    if (need > 0 && !scratch) return PNQ_ERR_NULL;
    if (need > 0 && !aligned(scratch, 16)) return PNQ_ERR_ALIGN;
    if (scratch_bytes < need) return PNQ_ERR_SCRATCH;
    return launched([&] {
        return launch_int8_gemm(Int8View{X, ldx, x_scales, M}, Int8View{W, ldw, w_scales, N}, K, y_type == PNQ_BF16, Y, scratch,
                                device_error_word(), stream);
    });
}
