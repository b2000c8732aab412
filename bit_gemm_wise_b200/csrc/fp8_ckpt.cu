// The 8-bit activation checkpoint (fp8_ckpt_save, fp8_ckpt_load) and the weight gradient from it
// (fp8_ckpt_wgrad).
//
// Save and load are bound by memory traffic: 2 bytes read (written) and 1 + 1/32 written (read) a
// value. A thread of the save takes 8 values, four threads a block of 32 (two shuffles for its
// maximum); a thread of the load 16 values. Four such pieces of a block's range are in flight per
// thread. The weight gradient is a product of w4_expand_gemm.cuh.
#include "w4_common.cuh"
#include "w4_expand_gemm.cuh"

#include <cuda_fp8.h>

namespace w4 {
namespace ckpt {

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // e in [-126, 127]

// e of the block maximum `amax` (finite): the smallest e >= -124 with amax <= 448 * 2^e. 448 is
// 1.75 * 2^8, so e is the exponent of amax less 8, and one more where its mantissa is over 1.75.
__device__ __forceinline__ int exponent_of(float amax) {
    const int e = (int)((__float_as_uint(amax) + 0x1FFFFFu) >> 23) - 127 - 8;
    return e < -124 ? -124 : e;
}

constexpr int THREADS = 256, PIECES = 4;  // pieces of THREADS x 8 (save) or 16 (load) values

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {  // two values, round to nearest even
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// n: blocks of 32 values
__global__ void __launch_bounds__(THREADS) save_kernel(const uint4 *__restrict__ x, int64_t n, uint2 *__restrict__ x8,
                                                       uint8_t *__restrict__ scale) {
    const int64_t i0 = (int64_t)blockIdx.x * (THREADS * PIECES) + threadIdx.x, end = 4 * n;
    uint4 v[PIECES];
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
        const int64_t i = i0 + p * THREADS;
        v[p] = i < end ? ldg_stream(x + i) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
        const int64_t i = i0 + p * THREADS;
        const uint32_t w[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
        // the largest magnitude, by its bits (a block that is not finite has 0x7F80 or more)
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) top = __vmaxu2(top, w[j] & 0x7FFF7FFFu);
        top = __vmaxu2(top, __shfl_xor_sync(FULL, top, 1));
        top = __vmaxu2(top, __shfl_xor_sync(FULL, top, 2));
        const uint32_t mx = max(top & 0xFFFFu, top >> 16);
        const bool bad = mx >= 0x7F80u;
        const int e = bad ? 0 : exponent_of(__uint_as_float(mx << 16));
        const float f = pow2(-e);
        // x 2^-e is exact; at e = 120 values stop at 240: 256 * 2^120 would leave bf16's range
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float lo = bf16_lo(w[j]) * f, hi = bf16_hi(w[j]) * f;
            if (e == 120) {
                lo = fminf(fmaxf(lo, -240.0f), 240.0f);
                hi = fminf(fmaxf(hi, -240.0f), 240.0f);
            }
            o[j] = bad ? 0x7F7Fu : e4m3x2(lo, hi);
        }
        if (i < end) {
            x8[i] = make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
            if ((threadIdx.x & 3) == 0) scale[i >> 2] = bad ? 255 : (uint8_t)(e + 127);
        }
    }
}

// n: pieces of 16 values
__global__ void __launch_bounds__(THREADS) load_kernel(const uint4 *__restrict__ x8, const uint8_t *__restrict__ scale,
                                                       int64_t n, uint4 *__restrict__ x) {
    const int64_t i0 = (int64_t)blockIdx.x * (THREADS * PIECES) + threadIdx.x;
    uint4 v[PIECES];
    uint32_t b[PIECES];
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
        const int64_t i = i0 + p * THREADS;
        v[p] = i < n ? ldg_stream(x8 + i) : make_uint4(0, 0, 0, 0);
        b[p] = i < n ? __ldg(scale + (i >> 1)) : 127u;
    }
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
        const int64_t i = i0 + p * THREADS;
        const uint32_t w[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t even, odd;
            xg::expand4_any(w[j], b[p], even, odd);
            o[2 * j] = __byte_perm(even, odd, 0x5410);
            o[2 * j + 1] = __byte_perm(even, odd, 0x7632);
        }
        if (i < n) {
            x[2 * i] = make_uint4(o[0], o[1], o[2], o[3]);
            x[2 * i + 1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
}

}  // namespace ckpt
}  // namespace w4

using namespace w4;

namespace {

// blocks of THREADS threads with PIECES pieces each (of 2^37 at most: shape_ok)
unsigned blocks_for(int64_t pieces) {
    return (unsigned)((pieces + ckpt::THREADS * ckpt::PIECES - 1) / (ckpt::THREADS * ckpt::PIECES));
}

}  // namespace

W4_API w4_status fp8_ckpt_save(const void *X_bf16, int64_t M, int64_t K, uint8_t *X_e4m3, uint8_t *X_scale,
                               cudaStream_t stream) {
    if (!X_bf16 || !X_e4m3 || !X_scale) return W4_ERR_NULL;
    if (!xg::shape_ok(M, 1, K)) return W4_ERR_SHAPE;
    if (!aligned16(X_bf16) || !aligned16(X_e4m3) || !aligned16(X_scale)) return W4_ERR_ALIGN;
    const int64_t n = M * (K / 32);
    const unsigned grid = blocks_for(4 * n);
    ckpt::save_kernel<<<grid, ckpt::THREADS, 0, stream>>>(static_cast<const uint4 *>(X_bf16), n,
                                                          reinterpret_cast<uint2 *>(X_e4m3), X_scale);
    return launch_status();
}

W4_API w4_status fp8_ckpt_load(const uint8_t *X_e4m3, const uint8_t *X_scale, int64_t M, int64_t K, void *X_bf16,
                               cudaStream_t stream) {
    if (!X_bf16 || !X_e4m3 || !X_scale) return W4_ERR_NULL;
    if (!xg::shape_ok(M, 1, K)) return W4_ERR_SHAPE;
    if (!aligned16(X_bf16) || !aligned16(X_e4m3) || !aligned16(X_scale)) return W4_ERR_ALIGN;
    const int64_t n = M * (K / 16);
    const unsigned grid = blocks_for(n);
    ckpt::load_kernel<<<grid, ckpt::THREADS, 0, stream>>>(reinterpret_cast<const uint4 *>(X_e4m3), X_scale, n,
                                                          static_cast<uint4 *>(X_bf16));
    return launch_status();
}

W4_API size_t fp8_ckpt_wgrad_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (!xg::shape_ok(M, N, K) || N % 8 != 0) return 0;
    // results in fp32 ask for no more: their plan differs only in where long sums are added up
    return xg::make_plan(xg::WGRAD, K, N, M, 1, num_sms()).bytes;
}

W4_API w4_status fp8_ckpt_wgrad_schedule(int64_t M, int64_t N, int64_t K, int flags, int sms, int64_t *out) {
    if (!out) return W4_ERR_NULL;
    if (!xg::shape_ok(M, N, K) || N % 8 != 0 || sms < 1 || sms > 4096) return W4_ERR_SHAPE;
    if ((flags & ~W4_OUT_FP32) != 0) return W4_ERR_ARG;
    xg::describe(xg::make_plan(xg::WGRAD, K, N, M, 1, sms, false, (flags & W4_OUT_FP32) != 0), sms, out);
    return W4_OK;
}

W4_API w4_status fp8_ckpt_wgrad(const void *dY_bf16, const uint8_t *X_e4m3, const uint8_t *X_scale, int64_t M, int64_t N,
                                int64_t K, void *dW, int flags, void *workspace, size_t workspace_bytes,
                                cudaStream_t stream) {
    if (!dY_bf16 || !X_e4m3 || !X_scale || !dW) return W4_ERR_NULL;
    if (!xg::shape_ok(M, N, K) || N % 8 != 0) return W4_ERR_SHAPE;
    if ((flags & ~W4_OUT_FP32) != 0) return W4_ERR_ARG;
    for (const void *p : {dY_bf16, (const void *)X_e4m3, (const void *)X_scale, (const void *)dW, (const void *)workspace})
        if (p && !aligned16(p)) return W4_ERR_ALIGN;
    const int sms = num_sms();
    const bool fp32 = (flags & W4_OUT_FP32) != 0;
    const xg::Plan p = xg::make_plan(xg::WGRAD, K, N, M, 1, sms, false, fp32);
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
    return xg::launch<xg::WGRAD, false, false>(p, tm, a, workspace, sms, stream);
}
