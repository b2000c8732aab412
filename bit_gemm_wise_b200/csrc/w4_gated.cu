// The gated feed-forward block over canonical 4-bit weights (w4a16_gated), its backward pass
// (w4a16_gated_bwd) and the input gradient of a 4-bit layer (w4a16_dgrad).
//
// The products of many rows are those of w4_expand_gemm.cuh; for up to 16 rows w4a16_gated has one
// thread per output, the weight dequantized to fp32 as it is read.
#include "w4_common.cuh"
#include "w4_expand_gemm.cuh"

namespace w4 {
namespace gated {

using xg::Weight;
using xg::act_of;

__device__ __forceinline__ float weight_at(const Weight &w, int64_t n, int64_t k, int64_t K, int gshift) {
    const int q = (w.codes[n * (K / 2) + (k >> 1)] >> (4 * (k & 1))) & 15;
    const int64_t j = n * (K >> gshift) + (k >> gshift);
    const int z = w.zeros ? w.zeros[j] : 8;
    return (float)(q - z) * __half2float(__ushort_as_half(w.scales[j]));
}

__global__ void gated_kernel(const __nv_bfloat16 *x, int64_t M, Weight wg, Weight wu, int64_t H, int64_t K, int gshift,
                             int act, __nv_bfloat16 *y) {
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < M * H; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t m = i / H, h = i % H;
        float g = 0.0f, u = 0.0f;
        for (int64_t k = 0; k < K; ++k) {
            const float xv = __bfloat162float(x[m * K + k]);
            g = fmaf(xv, weight_at(wg, h, k, K, gshift), g);
            u = fmaf(xv, weight_at(wu, h, k, K, gshift), u);
        }
        y[i] = __float2bfloat16_rn(act_of(g, act).value * u);
    }
}

}  // namespace gated
}  // namespace w4

using namespace w4;

namespace {

constexpr int64_t kFewRows = 16;  // up to here w4a16_gated reads the weights as a decode step does
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

W4_API size_t w4a16_gated_workspace_bytes(int64_t M, int64_t H, int64_t K, int group) {
    if (!gated_shape_ok(M, H, K) || !valid_group(group) || K % group != 0 || M <= kFewRows) return 0;
    return xg::place_prep(xg::make_plan(xg::FWD, H, M, K, 1, 0, num_sms()).bytes, M * K, M).end;
}

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
    if (M <= kFewRows) {
        gated::gated_kernel<<<blocks_for(M * H), 256, 0, stream>>>(
            (const __nv_bfloat16 *)X_bf16, M, {codes_gate, scales_gate, zeros_gate}, {codes_up, scales_up, zeros_up}, H,
            K, group_shift(group), act, (__nv_bfloat16 *)Y_bf16);
        return launch_status();
    }
    const int sms = num_sms();
    const xg::Plan p = xg::make_plan(xg::FWD, H, M, K, 1, 0, sms);
    const xg::PrepPlace q = xg::place_prep(p.bytes, M * K, M);
    if (!workspace || workspace_bytes < q.end) return W4_ERR_WORKSPACE;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    xg::Maps tm;
    if (!xg::make_map(&tm.b[0], ws + q.y, M, K, p.NT)) return W4_ERR_CUDA;
    tm.b[1] = tm.b[0];
    xg::Prep prep = {};
    prep.x[0] = static_cast<const __nv_bfloat16 *>(X_bf16);
    prep.y[0] = reinterpret_cast<__half *>(ws + q.y);
    prep.row_pow = reinterpret_cast<float *>(ws + q.row_pow);
    prep.M = M;
    prep.K = K;
    prep.tensors = 1;
    prep.pairs = 1;
    st = xg::launch_prep(prep, stream);
    if (st != W4_OK) return st;
    xg::Args a = {};
    a.row_pow = prep.row_pow;
    a.w[0] = {codes_gate, scales_gate, zeros_gate};
    a.w[1] = {codes_up, scales_up, zeros_up};
    a.out = Y_bf16;
    a.rows = H;
    a.K = K;
    a.cols = M;
    a.gshift = group_shift(group);
    a.act = act;
    return xg::launch<xg::FWD, false>(p, tm, a, workspace, sms, stream);
}

namespace {

// Workspace of the backward pass: counters and partial sums of its two products, then the fp16 rows
// that each multiplies (X, and after it dG and dU), each time in the same place.
struct BwdLayout {
    xg::Plan grads, dx;
    xg::PrepPlace q;
};
BwdLayout bwd_layout(int64_t M, int64_t H, int64_t K, int sms) {
    BwdLayout l;
    l.grads = xg::make_plan(xg::FWD, H, M, K, 1, 0, sms);
    l.dx = xg::make_plan(xg::DGRAD, K, M, H, 2, 0, sms);
    l.q = xg::place_prep(l.grads.bytes > l.dx.bytes ? l.grads.bytes : l.dx.bytes, M * (K > 2 * H ? K : 2 * H), M);
    return l;
}

}  // namespace

W4_API size_t w4a16_gated_bwd_workspace_bytes(int64_t M, int64_t H, int64_t K, int group, int from_ckpt) {
    if (!gated_shape_ok(M, H, K) || H % 8 != 0 || !valid_group(group) || K % group != 0) return 0;
    (void)from_ckpt;  // both sources become the same fp16 rows
    return bwd_layout(M, H, K, num_sms()).q.end;
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
    const int sms = num_sms();
    const BwdLayout l = bwd_layout(M, H, K, sms);
    if (!workspace || workspace_bytes < l.q.end) return W4_ERR_WORKSPACE;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    xg::Prep prep = {};
    prep.x[0] = static_cast<const __nv_bfloat16 *>(X_bf16);
    prep.x8 = X_e4m3;
    prep.xs = X_scale;
    prep.y[0] = reinterpret_cast<__half *>(ws + l.q.y);
    prep.row_pow = reinterpret_cast<float *>(ws + l.q.row_pow);
    prep.M = M;
    prep.K = K;
    prep.tensors = 1;
    prep.pairs = 1;
    st = xg::launch_prep(prep, stream);
    if (st != W4_OK) return st;
    xg::Maps tm;
    xg::Args a = {};
    a.w[0] = {codes_gate, scales_gate, zeros_gate};
    a.w[1] = {codes_up, scales_up, zeros_up};
    a.rows = H;
    a.K = K;
    a.cols = M;
    a.gshift = group_shift(group);
    a.act = act;
    a.dh = static_cast<const __nv_bfloat16 *>(dH_bf16);
    a.out = dG_bf16;
    a.out2 = static_cast<__nv_bfloat16 *>(dU_bf16);
    a.row_pow = prep.row_pow;
    if (!xg::make_map(&tm.b[0], prep.y[0], M, K, l.grads.NT)) return W4_ERR_CUDA;
    tm.b[1] = tm.b[0];
    st = xg::launch<xg::FWD, true>(l.grads, tm, a, workspace, sms, stream);
    if (st != W4_OK || !dX_bf16) return st;
    prep.x[0] = static_cast<const __nv_bfloat16 *>(dG_bf16);
    prep.x[1] = static_cast<const __nv_bfloat16 *>(dU_bf16);
    prep.x8 = prep.xs = nullptr;
    prep.y[1] = prep.y[0] + M * H;
    prep.K = H;
    prep.tensors = 2;
    prep.pairs = 0;
    st = xg::launch_prep(prep, stream);
    if (st != W4_OK) return st;
    if (!xg::make_map(&tm.b[0], prep.y[0], M, H, l.dx.NT) || !xg::make_map(&tm.b[1], prep.y[1], M, H, l.dx.NT))
        return W4_ERR_CUDA;
    a.dh = nullptr;
    a.out = dX_bf16;
    a.out2 = nullptr;
    return xg::launch<xg::DGRAD, false>(l.dx, tm, a, workspace, sms, stream);
}

W4_API size_t w4a16_dgrad_workspace_bytes(int64_t M, int64_t N, int64_t K, int group) {
    if (!gated_shape_ok(M, N, K) || N % 8 != 0 || !valid_group(group) || K % group != 0) return 0;
    return xg::place_prep(xg::make_plan(xg::DGRAD, K, M, N, 1, 0, num_sms()).bytes, M * N, M).end;
}

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
    const int sms = num_sms();
    const xg::Plan p = xg::make_plan(xg::DGRAD, K, M, N, 1, 0, sms);
    const xg::PrepPlace q = xg::place_prep(p.bytes, M * N, M);
    if (!workspace || workspace_bytes < q.end) return W4_ERR_WORKSPACE;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    xg::Maps tm;
    if (!xg::make_map(&tm.b[0], ws + q.y, M, N, p.NT)) return W4_ERR_CUDA;
    tm.b[1] = tm.b[0];
    xg::Prep prep = {};
    prep.x[0] = static_cast<const __nv_bfloat16 *>(dY_bf16);
    prep.y[0] = reinterpret_cast<__half *>(ws + q.y);
    prep.row_pow = reinterpret_cast<float *>(ws + q.row_pow);
    prep.M = M;
    prep.K = N;
    prep.tensors = 1;
    st = xg::launch_prep(prep, stream);
    if (st != W4_OK) return st;
    xg::Args a = {};
    a.row_pow = prep.row_pow;
    a.w[0] = a.w[1] = {codes, scales, zeros};
    a.out = dX_bf16;
    a.rows = N;
    a.K = K;
    a.cols = M;
    a.gshift = group_shift(group);
    return xg::launch<xg::DGRAD, false>(p, tm, a, workspace, sms, stream);
}
