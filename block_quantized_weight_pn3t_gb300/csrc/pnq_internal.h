// pnq_internal.h -- host-side launchers shared by the translation units of libpnq.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace pnq {

struct Nvfp4View {
    const uint8_t* codes;   // device [N][K/2], low nibble = even k
    const uint8_t* scales;  // device [N][K/16] E4M3FN
    float g;                // global multiplier (div: the global divisor d_w)
    bool div = false;       // the weight is e2m1 * e4m3 / g
};

// Planes of a grouped signed-integer matrix (pnq_grouped.cu states the layout).
struct GroupedView {
    const uint8_t* lo;
    const uint8_t* hi;
    const uint16_t* scales;
};
struct GroupedOut {
    uint8_t* lo;
    uint8_t* hi;
    uint16_t* scales;
};

int device_sm_count();

// Device address of the library's error word on the current device (pnq_device_error reads it).
int* device_error_word();

// Raises a kernel's dynamic shared memory limit to `bytes`, once per (kernel, device).
cudaError_t opt_in_smem(const void* kernel, int bytes);

// Allows a kernel clusters of more than 8 CTAs, once per (kernel, device).
cudaError_t opt_in_cluster(const void* kernel);

// 2-D tensor map over a row-major u32 matrix [rows][row_u32] (row pitch a multiple of 16
// bytes) with box {box_x, box_y}; rows past the end read as zeros. swizzle_128b: the copy
// stores 16-byte chunk c of box row r at chunk c ^ (r % 8) of that row (box rows of 128 bytes,
// shared destination 1024-byte aligned). False when the driver entry point is missing or the
// encoder rejects the arguments.
bool encode_u32_map(CUtensorMap* map, const void* base, int64_t rows, int64_t row_u32, int box_x, int box_y,
                    bool swizzle_128b = false);

// The same for rows of row_u32 words that start every pitch_bytes bytes (a multiple of 16).
bool encode_u32_map_pitch(CUtensorMap* map, const void* base, int64_t rows, int64_t row_u32, int64_t pitch_bytes,
                          int box_x, int box_y, bool swizzle_128b);

cudaError_t launch_pn_dequant(int type, const uint8_t* W, int64_t n_rows, int64_t K, float* out,
                              cudaStream_t stream);
cudaError_t launch_nvfp4_dequant(const Nvfp4View& w, int64_t n_rows, int64_t K, float* out,
                                 cudaStream_t stream);
cudaError_t launch_pn_validate(int type, const uint8_t* W, int64_t n_rows, int64_t K, int32_t* flags,
                               cudaStream_t stream);
cudaError_t launch_nvfp4_validate(const Nvfp4View& w, int64_t n_rows, int64_t K, int32_t* flags,
                                  cudaStream_t stream);

// Grouped signed-integer formats (type = kTypeQ4G64 ..): bit-exact dequantize, validate, GEMV on
// the CUDA cores (X fp32), and the canonical encoder MAXABS_F16_RECIP_RNE_V1 (status[r] = 1 for
// a row with a non-finite weight or a scale that overflows binary16; zeroed first).
cudaError_t launch_grouped_dequant(int type, const GroupedView& v, int64_t n_rows, int64_t K, float* out,
                                   cudaStream_t stream);
cudaError_t launch_grouped_validate(int type, const GroupedView& v, int64_t n_rows, int64_t K, int32_t* flags,
                                    cudaStream_t stream);
cudaError_t launch_grouped_gemv(int type, const GroupedView& v, int64_t N, int64_t K, const float* X, int M,
                                float* Y, cudaStream_t stream);
cudaError_t launch_grouped_quantize(int type, const float* w, int64_t n_rows, int64_t K, const GroupedOut& out,
                                    int32_t* status, cudaStream_t stream);

// PN reference quantizer, bit-exact with the CPU reference (status[r] = 1 for a row with a
// non-finite weight; zeroed first).
cudaError_t launch_pn_quantize(int type, const float* w, int64_t n_rows, int64_t K, uint8_t* out, int32_t* status,
                               cudaStream_t stream);

// NVFP4 clip search (TandemLLM "Quantisation and profiles"), bit-exact with the CPU reference;
// status[r] = 1 for a row with a non-finite weight (zeroed first).
cudaError_t launch_nvfp4_clip(const float* w, const float* act_ms, float g, int64_t n_rows, int64_t K, uint8_t* codes,
                              uint8_t* scales, int32_t* status, cudaStream_t stream);

// PN products for any M on the tcgen05 tensor cores (prefill): x split into two tf32 planes, the
// weights decoded slice by slice into two tf32 planes, three tf32 MMAs per K step (pnq_prefill.cu).
// scratch: 8 * M * K bytes for x plus 8 * K bytes per weight row of a slice (slices of a multiple
// of 128 rows); cudaErrorMemoryAllocation when it holds less than one 128-row slice.
int64_t prefill_slice_rows(int64_t N, int64_t K, int64_t M, size_t scratch_bytes);
cudaError_t launch_pn_prefill(int type, const uint8_t* W, int64_t N, int64_t K, const float* X, int64_t M, float* Y,
                              int* err, void* scratch, size_t scratch_bytes, cudaStream_t stream);

// Generic path: any 2-byte aligned PN buffer / any NVFP4 layout, CUDA-core FMA.
cudaError_t launch_pn_gemv_simt(int type, const uint8_t* W, int64_t N, int64_t K, const float* X, int M,
                                float* Y, cudaStream_t stream);
cudaError_t launch_nvfp4_gemv_simt(const Nvfp4View& w, int64_t N, int64_t K, const uint16_t* X, int M,
                                   float* Y, cudaStream_t stream);

// Fast path: 16-byte aligned weights and x, (K / block) a multiple of 8; clusters of one or two
// CTAs own disjoint row ranges and sum their partials on chip (no workspace). static_weights: the
// weights are not written by work queued earlier in the stream, so they may be streamed before
// the previous grid completes. cluster / stages > 0 force the plan (tests); 0 = automatic.
// Returns cudaErrorNotSupported when the shape is outside the fast path's range (the caller then
// uses the generic path).
cudaError_t launch_pn_gemv_mma(int type, const uint8_t* W, int64_t N, int64_t K, const float* X, int M,
                               float* Y, int* err, int cluster, int stages, bool static_weights,
                               cudaStream_t stream);
// Same pipeline for NVFP4: codes, scales and x 16-byte aligned, K % 256 == 0.
cudaError_t launch_nvfp4_gemv_mma(const Nvfp4View& w, int64_t N, int64_t K, const uint16_t* X, int M,
                                  float* Y, int* err, int cluster, int stages, bool static_weights,
                                  cudaStream_t stream);

// Launches a kernel that begins with griddep_wait() so that its launch and first instructions overlap the end of the
// kernel before it on the stream (programmatic dependent launch).
template <class... Params, class... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), int grid, int block, cudaStream_t stream, const Args&... args) {
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3(static_cast<unsigned>(grid));
    lc.blockDim = dim3(static_cast<unsigned>(block));
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kernel, static_cast<Params>(args)...);
}

// ---- expert layer (pnq_experts.cu) ------------------------------------------------------------

// pnq_expert_plan of the C ABI (all pointers device); no plan: tokens = rows, experts = 0.
struct PlanView {
    int32_t* offsets = nullptr;
    int32_t* block_start = nullptr;
    int32_t* order = nullptr;
    int32_t* position = nullptr;
    int32_t* scale_row = nullptr;
    int64_t tokens = 0;
    int slots = 1;
    int experts = 0;
    int rows = 0;   // tokens * slots
    int tiled = 0;  // rows that the tiled scales of an operand of the plan's rows have
};

// Entry v of a plan's arrays as an index below `limit`, or -1. The arrays are the caller's memory: one that was never sorted, or
// sorted for other sizes, leads to no access outside the buffers of a call.
__host__ __device__ inline int plan_index(int v, int limit) {
    return static_cast<unsigned>(v) < static_cast<unsigned>(limit) ? v : -1;
}

enum class ExpertOp { Gather, GatherBackward, Combine, CombineBackward };

cudaError_t launch_expert_sort(const int32_t* ids, const PlanView& p, cudaStream_t stream);
// a, b: input rows (b: CombineBackward's YS); weights, dweights where the operator has them.
cudaError_t launch_expert_rows(ExpertOp op, bool bf16, const void* a, const void* b, int64_t D, const PlanView& p,
                               const float* weights, void* out, float* dweights, cudaStream_t stream);

// ---- 4-bit microscaled operands (layout: include/pnq.h) -----------------------------------------

struct Fp4View {
    const uint8_t* codes;
    const uint8_t* scales;
    int64_t rows;      // of one matrix
    int64_t matrices;
};

inline int64_t fp4_pitch(int64_t K) { return (K / 2 + 15) / 16 * 16; }
inline int64_t fp4_chunks(bool mx, int64_t K) { return mx ? (K + 127) / 128 : (K + 63) / 64; }

cudaError_t launch_fp4_quantize(bool mx, bool bf16, const void* X, int64_t ldx, int64_t rows, int64_t K,
                                int64_t matrices, float inv_g, const PlanView& p, bool sorted, uint8_t* codes,
                                uint8_t* scales, cudaStream_t stream);
cudaError_t launch_fp4_dequantize(bool mx, const Fp4View& v, int64_t K, float g, const PlanView& p, bool bf16, void* out,
                                  cudaStream_t stream);
cudaError_t launch_fp4_pack(bool mx, const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K,
                            int64_t matrices, uint8_t* codes_out, uint8_t* scales_out, cudaStream_t stream);

// How launch_fp4_gemm tiles a dense product: activation rows of a tile, CTAs of a tile, CTAs that share a tile's K.
cudaError_t fp4_gemm_shape(int64_t M, int64_t N, int64_t K, int* columns, int* ctas, int* split);

// Y = alpha X W^T (p.experts == 0), or by experts with p (x: its sorted rows).
cudaError_t launch_fp4_gemm(bool mx, const Fp4View& x, const Fp4View& w, int64_t K, const PlanView& p, float alpha,
                            const float* w_global, bool bf16, void* Y, int* err, bool static_weights,
                            cudaStream_t stream);

}  // namespace pnq
