// The gated feed-forward block over canonical 4-bit weights (w4a16_gated), its backward pass
// (w4a16_gated_bwd) and the input gradient of a 4-bit layer (w4a16_dgrad).
//
// The products of many rows are those of w4_expand_gemm.cuh. Up to 16 rows w4a16_gated is a decode
// step, which reads every weight once for a handful of products, so the kernel below is built around
// the weight stream:
//   - a warp takes 16 features (the 16 gate rows and the 16 up rows of a matrix fragment each) and
//     every W-th block of 128 columns; its codes go from memory straight into registers (16 bytes a
//     lane and row where the group allows), a block ahead, and are there the A operand of
//     mma.m16n8k16, which may sum its 16 columns in any order: lane t of a row's four holds a quarter
//     of each group. The M <= 8 (16) tokens are the N = 8 columns of one (two) products;
//   - two shifts' worth of work per weight: a nibble OR-ed into the mantissa of bf16 128.0 is 128 + q,
//     exactly; the products with bf16 activations are exact too, and
//         y += s (sum (128 + q) x - (128 + z) sum x)
//     in fp32 after each group, with sum x from a product with a matrix of ones. (The legacy mma is
//     no bottleneck here: 24 products for 4096 weights; a tcgen05 tile would spend its time loading
//     TMEM.)
//   - the W warps' sums meet in shared memory, in order; the activation and the product follow there.
#include "w4_common.cuh"
#include "w4_expand_gemm.cuh"

namespace w4 {
namespace gated {

using xg::Weight;
using xg::act_of;

constexpr int WARPS = 8;          // of a block: they share its features' columns
constexpr int SCALE_WORDS = 6144;  // of shared memory for a run of groups (24 KB; 18 KB hold the sums)

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// codes i and i + 4 of eight as the bf16 pair 128 + q
__device__ __forceinline__ uint32_t codes_pair(uint32_t w, int i) { return ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u; }

struct FewArgs {
    const __nv_bfloat16 *x;   // [M, K]
    Weight w[2];              // gate, up
    __nv_bfloat16 *y;         // [M, H]
    int64_t H, K;
    int M, gshift, act;
    int run;                  // groups whose scales are in shared memory at a time
};

// A lane's codes of one block of 128 columns: rows r and r + 8 of the gate's and the up's fragment,
// 16 bytes each. GB is the group, or 128 for groups of 256 (whose halves share a scale): lane t has
// bytes [GB/8 t, GB/8 (t + 1)) of each group's GB/2.
template <int GB> struct Codes {
    uint32_t w[2][2][4];
    __device__ __forceinline__ void load(const uint8_t *const (&p)[2][2], int64_t k0, int64_t K, int t) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint8_t *q = p[m][h] + (k0 >> 1) + t * (GB / 8);
                if (GB == 128) {
                    const uint4 v = ldg_stream(q);
                    w[m][h][0] = v.x; w[m][h][1] = v.y; w[m][h][2] = v.z; w[m][h][3] = v.w;
                } else {
#pragma unroll
                    for (int g = 0; g < 128 / GB; ++g) {
                        const bool in = k0 + g * GB < K;  // the last block may be cut at a group
                        if (GB == 64) {
                            const uint2 v = in ? __ldg(reinterpret_cast<const uint2 *>(q + 32 * g)) : make_uint2(0, 0);
                            w[m][h][(2 * g) & 3] = v.x;
                            w[m][h][(2 * g + 1) & 3] = v.y;
                        } else {
                            w[m][h][g & 3] = in ? __ldg(reinterpret_cast<const uint32_t *>(q + 16 * g)) : 0u;
                        }
                    }
                }
            }
    }
};

template <int GB, int NB>
__global__ void __launch_bounds__(WARPS * 32) gated_few_kernel(const FewArgs a) {
    extern __shared__ uint32_t sc[];                         // [group of the run][32 rows]: s | z << 16
    __shared__ float sums[WARPS][NB][32][9];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
    const int64_t h0 = (int64_t)blockIdx.x * 16, J = a.K >> a.gshift;
    const uint8_t *p[2][2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t row = h0 + r + 8 * h;
            p[m][h] = a.w[m].codes + (row < a.H ? row : a.H - 1) * (a.K >> 1);
        }
    const __nv_bfloat16 *xp[NB];
    bool tok[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        tok[n] = r + 8 * n < a.M;
        xp[n] = a.x + (int64_t)(tok[n] ? r + 8 * n : 0) * a.K;
    }
    float acc[2][NB][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;

    const int64_t blocks = (a.K + 127) / 128, per_run = ((int64_t)a.run << a.gshift) / 128;
    Codes<GB> next;
    int64_t b = warp;
    if (b < blocks) next.load(p, b * 128, a.K, t);
    for (int64_t run0 = 0; run0 < blocks; run0 += per_run) {
        const int64_t run1 = run0 + per_run < blocks ? run0 + per_run : blocks;
        const int64_t j0 = (run0 * 128) >> a.gshift, j1 = j0 + a.run < J ? j0 + a.run : J;
        __syncthreads();  // the previous run's readers
        for (int row = warp; row < 32; row += WARPS) {
            const Weight &w = a.w[row >> 4];
            const int64_t h = h0 + (row & 15) < a.H ? h0 + (row & 15) : a.H - 1;
            for (int64_t j = j0 + lane; j < j1; j += 32) {
                const uint32_t s = __ldg(w.scales + h * J + j);
                const uint32_t z = w.zeros ? (uint32_t)(uint16_t)__ldg(w.zeros + h * J + j) : 8u;
                sc[(j - j0) * 32 + row] = s | (z << 16);
            }
        }
        __syncthreads();
        for (; b < run1; b += WARPS) {
            const Codes<GB> c = next;
            if (b + WARPS < blocks) next.load(p, (b + WARPS) * 128, a.K, t);
            const int64_t k0 = b * 128;
#pragma unroll
            for (int g = 0; g < 128 / GB; ++g) {
                if (k0 + g * GB >= a.K) break;
                float P[2][NB][4], X[NB][4];
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) P[0][n][i] = P[1][n][i] = X[n][i] = 0.0f;
#pragma unroll
                for (int i = 0; i < GB / 32; ++i) {
                    const int wi = (GB / 32) * g + i;
                    uint32_t xb[NB][4];
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (tok[n]) v = __ldg(reinterpret_cast<const uint4 *>(xp[n] + k0 + g * GB + (GB / 4) * t + 8 * i));
                        xb[n][0] = __byte_perm(v.x, v.z, 0x5410);
                        xb[n][1] = __byte_perm(v.x, v.z, 0x7632);
                        xb[n][2] = __byte_perm(v.y, v.w, 0x5410);
                        xb[n][3] = __byte_perm(v.y, v.w, 0x7632);
                    }
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            const uint32_t a0 = codes_pair(c.w[m][0][wi], 2 * s), a1 = codes_pair(c.w[m][1][wi], 2 * s);
                            const uint32_t a2 = codes_pair(c.w[m][0][wi], 2 * s + 1), a3 = codes_pair(c.w[m][1][wi], 2 * s + 1);
#pragma unroll
                            for (int n = 0; n < NB; ++n) mma16816(P[m][n], a0, a1, a2, a3, xb[n][2 * s], xb[n][2 * s + 1]);
                        }
#pragma unroll
                        for (int n = 0; n < NB; ++n)
                            mma16816(X[n], 0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u, xb[n][2 * s], xb[n][2 * s + 1]);
                    }
                }
                const uint32_t *sg = sc + (((k0 + g * GB) >> a.gshift) - j0) * 32;
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t sz = sg[16 * m + r + 8 * h];
                        const float s = __half2float(__ushort_as_half((unsigned short)(sz & 0xFFFFu)));
                        const float z = (float)(128 + (int)(int16_t)(sz >> 16));
#pragma unroll
                        for (int n = 0; n < NB; ++n)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                acc[m][n][2 * h + i] = fmaf(s, fmaf(-z, X[n][i], P[m][n][2 * h + i]), acc[m][n][2 * h + i]);
                    }
            }
        }
    }
    // rows r and r + 8 of each fragment, tokens 2 t and 2 t + 1
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) sums[warp][n][16 * m + r + 8 * (i >> 1)][2 * t + (i & 1)] = acc[m][n][i];
    __syncthreads();
    for (int i = threadIdx.x; i < NB * 128; i += WARPS * 32) {
        const int f = i & 15, c = (i >> 4) & 7, n = i >> 7;
        float g = 0.0f, u = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            g += sums[w][n][f][c];
            u += sums[w][n][16 + f][c];
        }
        if (h0 + f < a.H && 8 * n + c < a.M)
            a.y[(int64_t)(8 * n + c) * a.H + h0 + f] = __float2bfloat16_rn(act_of(g, a.act).value * u);
    }
}

template <int GB> w4_status launch_few(const FewArgs &a, cudaStream_t stream) {
    const unsigned grid = (unsigned)((a.H + 15) / 16);
    const size_t smem = (size_t)a.run * 32 * sizeof(uint32_t);
    if (a.M <= 8)
        gated_few_kernel<GB, 1><<<grid, WARPS * 32, smem, stream>>>(a);
    else
        gated_few_kernel<GB, 2><<<grid, WARPS * 32, smem, stream>>>(a);
    return launch_status();
}

inline w4_status gated_few(FewArgs a, int group, cudaStream_t stream) {
    // a run holds whole blocks of 128 columns and of the group
    const int64_t J = a.K >> a.gshift;
    a.run = SCALE_WORDS / 32;
    if (J < a.run) a.run = (int)((J + 3) / 4 * 4);
    return group == 32 ? launch_few<32>(a, stream) : group == 64 ? launch_few<64>(a, stream) : launch_few<128>(a, stream);
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
        gated::FewArgs f = {};
        f.x = static_cast<const __nv_bfloat16 *>(X_bf16);
        f.w[0] = {codes_gate, scales_gate, zeros_gate};
        f.w[1] = {codes_up, scales_up, zeros_up};
        f.y = static_cast<__nv_bfloat16 *>(Y_bf16);
        f.H = H;
        f.K = K;
        f.M = (int)M;
        f.gshift = group_shift(group);
        f.act = act;
        return gated::gated_few(f, group, stream);
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
