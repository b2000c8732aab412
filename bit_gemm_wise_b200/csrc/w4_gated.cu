// The gated feed-forward block over canonical 4-bit weights (w4a16_gated), its backward pass
// (w4a16_gated_bwd) and the input gradient of a 4-bit layer (w4a16_dgrad).
//
// First form: one thread per output, the weight dequantized to fp32 as it is read.
#include "w4_common.cuh"

namespace w4 {
namespace gated {

struct Weight {
    const uint8_t *codes;     // [N, K/2]
    const uint16_t *scales;   // [N, K/g] fp16 bits
    const int16_t *zeros;     // [N, K/g], NULL for symmetric weights (z = 8)
};

__device__ __forceinline__ float weight_at(const Weight &w, int64_t n, int64_t k, int64_t K, int gshift) {
    const int q = (w.codes[n * (K / 2) + (k >> 1)] >> (4 * (k & 1))) & 15;
    const int64_t j = n * (K >> gshift) + (k >> gshift);
    const int z = w.zeros ? w.zeros[j] : 8;
    return (float)(q - z) * __half2float(__ushort_as_half(w.scales[j]));
}

__device__ __forceinline__ float act_of(float g, int act) {
    if (act == W4_ACT_SILU) return g / (1.0f + expf(-g));
    const float t = tanhf(0.7978845608028654f * (g + 0.044715f * g * g * g));
    return 0.5f * g * (1.0f + t);
}

__device__ __forceinline__ float slope_of(float g, int act) {
    if (act == W4_ACT_SILU) {
        const float s = 1.0f / (1.0f + expf(-g));
        return s * (1.0f + g * (1.0f - s));
    }
    const float t = tanhf(0.7978845608028654f * (g + 0.044715f * g * g * g));
    return 0.5f * (1.0f + t) + 0.5f * g * (1.0f - t * t) * 0.7978845608028654f * (1.0f + 3.0f * 0.044715f * g * g);
}

// act(g) u, or with dh the gradients dG and dU
__global__ void gated_kernel(const __nv_bfloat16 *x, int64_t M, Weight wg, Weight wu, int64_t H, int64_t K, int gshift,
                             int act, const __nv_bfloat16 *dh, __nv_bfloat16 *y, __nv_bfloat16 *dg, __nv_bfloat16 *du) {
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < M * H; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t m = i / H, h = i % H;
        float g = 0.0f, u = 0.0f;
        for (int64_t k = 0; k < K; ++k) {
            const float xv = __bfloat162float(x[m * K + k]);
            g = fmaf(xv, weight_at(wg, h, k, K, gshift), g);
            u = fmaf(xv, weight_at(wu, h, k, K, gshift), u);
        }
        if (!dh) {
            y[i] = __float2bfloat16_rn(act_of(g, act) * u);
        } else {
            const float d = __bfloat162float(dh[i]);
            dg[i] = __float2bfloat16_rn(d * u * slope_of(g, act));
            du[i] = __float2bfloat16_rn(d * act_of(g, act));
        }
    }
}

// dX = dA Wa (+ dB Wb)
__global__ void dgrad_kernel(const __nv_bfloat16 *da, Weight wa, const __nv_bfloat16 *db, Weight wb, int64_t M, int64_t N,
                             int64_t K, int gshift, __nv_bfloat16 *dx) {
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < M * K; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t m = i / K, k = i % K;
        float s = 0.0f;
        for (int64_t n = 0; n < N; ++n) s = fmaf(__bfloat162float(da[m * N + n]), weight_at(wa, n, k, K, gshift), s);
        if (db)
            for (int64_t n = 0; n < N; ++n) s = fmaf(__bfloat162float(db[m * N + n]), weight_at(wb, n, k, K, gshift), s);
        dx[i] = __float2bfloat16_rn(s);
    }
}

}  // namespace gated
}  // namespace w4

using namespace w4;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 24;

bool gated_shape_ok(int64_t M, int64_t N, int64_t K) {
    return M >= 1 && M <= kMaxRows && N >= 1 && N <= kMaxRows && K >= 32 && K <= kMaxRows && K % 32 == 0;
}

int group_shift(int g) { return g == 32 ? 5 : g == 64 ? 6 : g == 128 ? 7 : 8; }

// Checks shared by the entry points that take canonical weights.
w4_status weight_ok(const uint8_t *codes, const uint16_t *scales, const int16_t *zeros, int mode) {
    if (!codes || !scales) return W4_ERR_NULL;
    if (mode == W4_ASYM && !zeros) return W4_ERR_NULL;
    if (mode == W4_SYM && zeros) return W4_ERR_ARG;
    if (!aligned16(codes) || !aligned16(scales) || (zeros && !aligned16(zeros))) return W4_ERR_ALIGN;
    return W4_OK;
}

unsigned blocks_for(int64_t n) {
    const int64_t b = (n + 255) / 256;
    return (unsigned)(b < 65536 ? b : 65536);
}

}  // namespace

W4_API size_t w4a16_gated_workspace_bytes(int64_t M, int64_t H, int64_t K, int group) { return 0; }

W4_API w4_status w4a16_gated(const void *X_bf16, int64_t M, const uint8_t *codes_gate, const uint16_t *scales_gate,
                             const int16_t *zeros_gate, const uint8_t *codes_up, const uint16_t *scales_up,
                             const int16_t *zeros_up, int64_t H, int64_t K, int group, int mode, int act, void *Y_bf16,
                             void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (!X_bf16 || !Y_bf16) return W4_ERR_NULL;
    if (!gated_shape_ok(M, H, K)) return W4_ERR_SHAPE;
    if (!valid_group(group) || K % group != 0) return W4_ERR_GROUP;
    if (!valid_mode(mode) || (act != W4_ACT_SILU && act != W4_ACT_GELU_TANH)) return W4_ERR_ARG;
    w4_status st = weight_ok(codes_gate, scales_gate, zeros_gate, mode);
    if (st == W4_OK) st = weight_ok(codes_up, scales_up, zeros_up, mode);
    if (st != W4_OK) return st;
    if (!aligned16(X_bf16) || !aligned16(Y_bf16) || (workspace && !aligned16(workspace))) return W4_ERR_ALIGN;
    if (workspace_bytes < w4a16_gated_workspace_bytes(M, H, K, group)) return W4_ERR_WORKSPACE;
    gated::gated_kernel<<<blocks_for(M * H), 256, 0, stream>>>(
        (const __nv_bfloat16 *)X_bf16, M, {codes_gate, scales_gate, zeros_gate}, {codes_up, scales_up, zeros_up}, H, K,
        group_shift(group), act, nullptr, (__nv_bfloat16 *)Y_bf16, nullptr, nullptr);
    return launch_status();
}

W4_API size_t w4a16_gated_bwd_workspace_bytes(int64_t M, int64_t H, int64_t K, int group, int from_ckpt) {
    if (!gated_shape_ok(M, H, K) || H % 8 != 0 || !valid_group(group) || K % group != 0) return 0;
    return from_ckpt ? (size_t)M * K * 2 : 0;
}

W4_API w4_status w4a16_gated_bwd(const void *dH_bf16, const void *X_bf16, const uint8_t *X_e4m3, const uint8_t *X_scale,
                                 int64_t M, const uint8_t *codes_gate, const uint16_t *scales_gate,
                                 const int16_t *zeros_gate, const uint8_t *codes_up, const uint16_t *scales_up,
                                 const int16_t *zeros_up, int64_t H, int64_t K, int group, int mode, int act,
                                 void *dG_bf16, void *dU_bf16, void *dX_bf16, void *workspace, size_t workspace_bytes,
                                 cudaStream_t stream) {
    const bool ckpt = X_bf16 == nullptr;
    if (!dH_bf16 || !dG_bf16 || !dU_bf16 || (ckpt && (!X_e4m3 || !X_scale))) return W4_ERR_NULL;
    if (!ckpt && (X_e4m3 || X_scale)) return W4_ERR_ARG;
    if (!gated_shape_ok(M, H, K) || H % 8 != 0) return W4_ERR_SHAPE;
    if (!valid_group(group) || K % group != 0) return W4_ERR_GROUP;
    if (!valid_mode(mode) || (act != W4_ACT_SILU && act != W4_ACT_GELU_TANH)) return W4_ERR_ARG;
    w4_status st = weight_ok(codes_gate, scales_gate, zeros_gate, mode);
    if (st == W4_OK) st = weight_ok(codes_up, scales_up, zeros_up, mode);
    if (st != W4_OK) return st;
    for (const void *p : {dH_bf16, X_bf16, (const void *)X_e4m3, (const void *)X_scale, (const void *)dG_bf16,
                          (const void *)dU_bf16, (const void *)dX_bf16, (const void *)workspace})
        if (p && !aligned16(p)) return W4_ERR_ALIGN;
    const size_t need = w4a16_gated_bwd_workspace_bytes(M, H, K, group, ckpt ? 1 : 0);
    if (need && (!workspace || workspace_bytes < need)) return W4_ERR_WORKSPACE;
    if (ckpt) {
        st = fp8_ckpt_load(X_e4m3, X_scale, M, K, workspace, stream);
        if (st != W4_OK) return st;
        X_bf16 = workspace;
    }
    const gated::Weight wg = {codes_gate, scales_gate, zeros_gate}, wu = {codes_up, scales_up, zeros_up};
    gated::gated_kernel<<<blocks_for(M * H), 256, 0, stream>>>(
        (const __nv_bfloat16 *)X_bf16, M, wg, wu, H, K, group_shift(group), act, (const __nv_bfloat16 *)dH_bf16, nullptr,
        (__nv_bfloat16 *)dG_bf16, (__nv_bfloat16 *)dU_bf16);
    if (dX_bf16)
        gated::dgrad_kernel<<<blocks_for(M * K), 256, 0, stream>>>((const __nv_bfloat16 *)dG_bf16, wg,
                                                                   (const __nv_bfloat16 *)dU_bf16, wu, M, H, K,
                                                                   group_shift(group), (__nv_bfloat16 *)dX_bf16);
    return launch_status();
}

W4_API size_t w4a16_dgrad_workspace_bytes(int64_t M, int64_t N, int64_t K, int group) { return 0; }

W4_API w4_status w4a16_dgrad(const void *dY_bf16, int64_t M, const uint8_t *codes, const uint16_t *scales,
                             const int16_t *zeros, int64_t N, int64_t K, int group, int mode, void *dX_bf16,
                             void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (!dY_bf16 || !dX_bf16) return W4_ERR_NULL;
    if (!gated_shape_ok(M, N, K) || N % 8 != 0) return W4_ERR_SHAPE;
    if (!valid_group(group) || K % group != 0) return W4_ERR_GROUP;
    if (!valid_mode(mode)) return W4_ERR_ARG;
    w4_status st = weight_ok(codes, scales, zeros, mode);
    if (st != W4_OK) return st;
    if (!aligned16(dY_bf16) || !aligned16(dX_bf16) || (workspace && !aligned16(workspace))) return W4_ERR_ALIGN;
    if (workspace_bytes < w4a16_dgrad_workspace_bytes(M, N, K, group)) return W4_ERR_WORKSPACE;
    gated::dgrad_kernel<<<blocks_for(M * K), 256, 0, stream>>>((const __nv_bfloat16 *)dY_bf16, {codes, scales, zeros},
                                                               nullptr, {}, M, N, K, group_shift(group),
                                                               (__nv_bfloat16 *)dX_bf16);
    return launch_status();
}
