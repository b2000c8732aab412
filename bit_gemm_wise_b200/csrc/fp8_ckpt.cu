// The 8-bit activation checkpoint (fp8_ckpt_save, fp8_ckpt_load) and the weight gradient from it
// (fp8_ckpt_wgrad).
//
// First form of the checkpoint: one thread per block of 32 columns. The weight gradient is a
// product of w4_expand_gemm.cuh.
#include "w4_common.cuh"
#include "w4_expand_gemm.cuh"

#include <cuda_fp8.h>

namespace w4 {
namespace ckpt {

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // e in [-126, 127]

// 2^e of a scale byte; 255 is NaN
__device__ __forceinline__ float scale_of(uint8_t b) { return b == 255 ? __int_as_float(0x7fffffff) : pow2((int)b - 127); }

__device__ __forceinline__ float e4m3(uint8_t v) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(v, __NV_E4M3);
    return __half2float(__half(h));
}

// e of the block maximum `amax` (finite): the smallest e >= -124 with amax <= 448 * 2^e. 448 is
// 1.75 * 2^8, so e is the exponent of amax less 8, and one more where its mantissa is over 1.75.
__device__ __forceinline__ int exponent_of(float amax) {
    const int e = (int)((__float_as_uint(amax) + 0x1FFFFFu) >> 23) - 127 - 8;
    return e < -124 ? -124 : e;
}

__global__ void save_kernel(const __nv_bfloat16 *x, int64_t n, uint8_t *x8, uint8_t *scale) {
    for (int64_t b = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; b < n; b += (int64_t)gridDim.x * blockDim.x) {
        float amax = 0.0f;
        bool bad = false;
        for (int i = 0; i < 32; ++i) {
            const float v = fabsf(__bfloat162float(x[b * 32 + i]));
            bad = bad || !(v <= 3.4e38f);
            amax = fmaxf(amax, v);
        }
        const int e = bad ? 0 : exponent_of(amax);
        const float top = e == 120 ? 240.0f : 448.0f;  // 256 * 2^120 would leave bf16's range
        for (int i = 0; i < 32; ++i)
            x8[b * 32 + i] = bad ? 0x7F
                                 : (uint8_t)__nv_cvt_float_to_fp8(
                                       fminf(fmaxf(__bfloat162float(x[b * 32 + i]) * pow2(-e), -top), top),
                                       __NV_SATFINITE, __NV_E4M3);
        scale[b] = bad ? 255 : (uint8_t)(e + 127);
    }
}

__global__ void load_kernel(const uint8_t *x8, const uint8_t *scale, int64_t n, __nv_bfloat16 *x) {
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x)
        x[i] = __float2bfloat16_rn(e4m3(x8[i]) * scale_of(scale[i >> 5]));
}

}  // namespace ckpt
}  // namespace w4

using namespace w4;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 24;

bool ckpt_shape_ok(int64_t M, int64_t K) {
    return M >= 1 && M <= kMaxRows && K >= 32 && K <= kMaxRows && K % 32 == 0;
}

unsigned blocks_for(int64_t n) {
    const int64_t b = (n + 255) / 256;
    return (unsigned)(b < 65536 ? b : 65536);
}

}  // namespace

W4_API w4_status fp8_ckpt_save(const void *X_bf16, int64_t M, int64_t K, uint8_t *X_e4m3, uint8_t *X_scale,
                               cudaStream_t stream) {
    if (!X_bf16 || !X_e4m3 || !X_scale) return W4_ERR_NULL;
    if (!ckpt_shape_ok(M, K)) return W4_ERR_SHAPE;
    if (!aligned16(X_bf16) || !aligned16(X_e4m3) || !aligned16(X_scale)) return W4_ERR_ALIGN;
    const int64_t n = M * (K / 32);
    ckpt::save_kernel<<<blocks_for(n), 256, 0, stream>>>((const __nv_bfloat16 *)X_bf16, n, X_e4m3, X_scale);
    return launch_status();
}

W4_API w4_status fp8_ckpt_load(const uint8_t *X_e4m3, const uint8_t *X_scale, int64_t M, int64_t K, void *X_bf16,
                               cudaStream_t stream) {
    if (!X_bf16 || !X_e4m3 || !X_scale) return W4_ERR_NULL;
    if (!ckpt_shape_ok(M, K)) return W4_ERR_SHAPE;
    if (!aligned16(X_bf16) || !aligned16(X_e4m3) || !aligned16(X_scale)) return W4_ERR_ALIGN;
    ckpt::load_kernel<<<blocks_for(M * K), 256, 0, stream>>>(X_e4m3, X_scale, M * K, (__nv_bfloat16 *)X_bf16);
    return launch_status();
}

// fp32 sums of the tensor cores truncate: against a 64-bit product, bf16 operands of N(0, 1) gave a
// relative error of 4e-7 over 910 rows, 2e-6 over 2048 and 9e-6 over 8192. An fp32 gradient is
// therefore added up outside them every 2048 rows; a bf16 one rounds far above that.
static xg::Plan wgrad_plan(int64_t M, int64_t N, int64_t K, bool fp32, int sms) {
    return xg::make_plan(xg::WGRAD, K, N, M, 1, fp32 ? 2048 : 0, sms);
}

W4_API size_t fp8_ckpt_wgrad_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (!ckpt_shape_ok(M, K) || N < 1 || N > kMaxRows || N % 8 != 0) return 0;
    return wgrad_plan(M, N, K, false, num_sms()).bytes;
}

W4_API w4_status fp8_ckpt_wgrad(const void *dY_bf16, const uint8_t *X_e4m3, const uint8_t *X_scale, int64_t M, int64_t N,
                                int64_t K, void *dW, int flags, void *workspace, size_t workspace_bytes,
                                cudaStream_t stream) {
    if (!dY_bf16 || !X_e4m3 || !X_scale || !dW) return W4_ERR_NULL;
    if (!ckpt_shape_ok(M, K) || N < 1 || N > kMaxRows || N % 8 != 0) return W4_ERR_SHAPE;
    if ((flags & ~W4_OUT_FP32) != 0) return W4_ERR_ARG;
    for (const void *p : {dY_bf16, (const void *)X_e4m3, (const void *)X_scale, (const void *)dW, (const void *)workspace})
        if (p && !aligned16(p)) return W4_ERR_ALIGN;
    const int sms = num_sms();
    const bool fp32 = (flags & W4_OUT_FP32) != 0;
    const xg::Plan p = wgrad_plan(M, N, K, fp32, sms);
    if (p.bytes && (!workspace || workspace_bytes < p.bytes)) return W4_ERR_WORKSPACE;
    xg::Maps tm;
    if (!xg::make_map(&tm.b[0], dY_bf16, M, N, xg::BK)) return W4_ERR_CUDA;
    tm.b[1] = tm.b[0];
    xg::Args a = {};
    a.x8 = X_e4m3;
    a.xs = X_scale;
    a.out = dW;
    a.rows = M;
    a.K = K;
    a.cols = N;
    a.out_fp32 = fp32 ? 1 : 0;
    return xg::launch<xg::WGRAD, false>(p, tm, a, workspace, sms, stream);
}
