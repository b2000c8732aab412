// The gated feed-forward block over canonical 4-bit weights (w4a16_gated), its backward pass
// (w4a16_gated_bwd) and the input gradient of a 4-bit layer (w4a16_dgrad).
//
// The products of many rows are those of w4_expand_gemm.cuh. Up to 16 rows w4a16_gated is a decode
// step, which reads every weight once for a handful of products, so the two kernels below are built
// around the weight stream. In both a warp takes 16 features (the 16 gate rows and the 16 up rows of a
// matrix fragment each) and every W-th block of 128 columns, and its codes are in registers the A
// operand of a warp-level product, which may sum its columns in any order: lane t of a row's four holds
// a quarter of each group. The W warps' sums meet in shared memory, in order; the activation and the
// product follow there. (The warp-level products are no bottleneck: 2 cycles an SM each, 24 or 8 of
// them for 4096 weights, of which HBM brings 46 a cycle and SM. A tcgen05 tile would spend its time
// filling TMEM.)
//
// gated_few_kernel, one launch: a nibble OR-ed into the mantissa of bf16 128.0 is 128 + q, exactly (a
// shift and a mask for two of them); the products with bf16 activations are exact too, and
//     y += s (sum (128 + q) x - (128 + z) sum x)
// in fp32 after each group, with sum x from a product with a matrix of ones. M <= 8 (16) tokens are the
// N = 8 columns of one (two) products. It is bound by instructions, about 400 a block of 4096 weights.
//
// gated_bytes_kernel, for one or two tokens of large layers: the activations become integers once, in a
// small kernel before it. Each slice of a token (a group's columns) is divided by a power of two so that
// its largest magnitude is under 2^22, rounded (exact for bf16 values within 2^14 of the largest, else
// off by 2^-22 of it) and split in three signed bytes, a column each: x = (c0 + 2^8 c1 + 2^16 c2) 2^e.
// Three instructions then make a word of eight codes two A registers of mma.m16n8k32 on unsigned and
// signed bytes, and after each group, exact until then,
//     y_c += (s f_c) (sum q c - z sum c),   f_c = 2^(e + 8 i),
// in fp32 for each byte column; a token's three meet at the end. 277 instructions a block.
//
// Which one: one token through 14336 x 4096 takes 27.7 us with the first and 19.6 us with the second;
// 5632 x 2048 takes 10.1 and 11.4 us, and small layers lose the second launch's 2 us. The bytes start at
// 2^25 weights a matrix. Four tokens take 28 us either way, eight 29 and 34 us: more than two stay with
// the first.
#include "w4_common.cuh"
#include "w4_expand_gemm.cuh"

namespace w4 {
namespace gated {

using xg::Weight;
using xg::act_of;

constexpr int WARPS = 8;           // of a block of gated_few_kernel
constexpr int B_WARPS = 4;         // of gated_bytes_kernel: with two blocks ahead a warp, 96 KB an SM in flight
constexpr int AHEAD = 2;           // column blocks of a warp in flight there (3: 20.2 us, 4: 30.5 us)
constexpr int BLOCK_BYTES = 2048;  // codes of 32 rows and 128 columns
constexpr int MAX_RUN = 192;       // groups whose scales are in shared memory at a time: 24 KB

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// codes i and i + 4 of eight as the bf16 pair 128 + q
__device__ __forceinline__ uint32_t codes_pair(uint32_t w, int i) { return ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u; }

__device__ __forceinline__ void mma16832(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The activations as bytes: column c = 3 m + i holds byte i of token m, each eight of its K values in
// the order 0, 2, 4, 6, 1, 3, 5, 7 (the order in which a code word falls apart).
struct Bytes {
    int8_t *x;                // [3 M][K]
    float *f;                 // [slice][columns] 2^(e + 8 i); columns are padded to whole products
    int *sum;                 // [slice][columns] sum of the bytes
};
struct FewArgs {
    const __nv_bfloat16 *x;   // [M, K]
    Bytes v;                  // gated_bytes_kernel
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
            a.y[(int64_t)(8 * n + c) * a.H + h0 + f] = __float2bfloat16_rn(act_of(g, a.act == W4_ACT_GELU_TANH).value * u);
    }
}

// One warp per token and slice of GB columns.
template <int GB> __global__ void __launch_bounds__(128) bytes_prep_kernel(const FewArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int64_t slices = a.K / GB, i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (i >= slices * a.M) return;
    const int64_t slice = i % slices;
    const int m = (int)(i / slices);
    const __nv_bfloat16 *x = a.x + (int64_t)m * a.K + slice * GB;
    constexpr int N = GB / 32;
    float v[N], top = 0.0f;
    bool bad = false;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        v[j] = __bfloat162float(x[lane + 32 * j]);
        bad = bad || !(fabsf(v[j]) <= 3.4e38f);
        top = fmaxf(top, fabsf(v[j]));
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, o));
    bad = __any_sync(FULL, bad);
    int e = (int)(__float_as_uint(top) >> 23) - 127;  // 2^e <= top < 2^(e + 1)
    e = e < -100 ? -100 : e;
    const float scale = __uint_as_float((uint32_t)(21 - e + 127) << 23);
    int sums[3] = {0, 0, 0};
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int k = lane + 32 * j, at = (k & ~7) + ((k & 1) << 2) + ((k & 7) >> 1);
        const int q = bad ? 0 : __float2int_rn(v[j] * scale);  // under 2^22 in magnitude
        const int c0 = (int)(int8_t)q, r1 = (q - c0) >> 8, c1 = (int)(int8_t)r1, c2 = (r1 - c1) >> 8;
        int8_t *o = a.v.x + (int64_t)(3 * m) * a.K + slice * GB + at;
        o[0] = (int8_t)c0;
        o[a.K] = (int8_t)c1;
        o[2 * a.K] = (int8_t)c2;
        sums[0] += c0;
        sums[1] += c1;
        sums[2] += c2;
    }
#pragma unroll
    for (int c = 0; c < 3; ++c) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) sums[c] += __shfl_xor_sync(FULL, sums[c], o);
        if (lane == 0) {
            const int ec = e - 21 + 8 * c;  // from -121; a slice that is not finite gives NaN
            a.v.f[slice * 8 + 3 * m + c] = bad ? __int_as_float(0x7fffffff) : __uint_as_float((uint32_t)(ec + 127) << 23);
            a.v.sum[slice * 8 + 3 * m + c] = sums[c];
        }
    }
}

// 16 bytes from global to shared memory, or 16 zero bytes
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Codes of one column block in a warp's shared memory: for the gate's and the up's fragment (m) and
// rows r and r + 8 (h), 64 bytes a row, rows one after the other. GB is the group, or 128 for groups
// of 256 (whose halves share a scale): lane t of a row takes bytes [GB/8 t, GB/8 (t + 1)) of each
// group's GB/2 as words (GB/32) g + i.
template <int GB> __device__ __forceinline__ void block_words(uint32_t at, int r, int t, uint32_t (&w)[2][2][4]) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t row = at + (uint32_t)((2 * m + h) * 512 + r * 64);
            if (GB == 128) {
                const uint4 v = xg::lds128(row + (uint32_t)t * 16u);
                w[m][h][0] = v.x; w[m][h][1] = v.y; w[m][h][2] = v.z; w[m][h][3] = v.w;
            } else if (GB == 64) {
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const uint2 v = xg::lds64(row + (uint32_t)(32 * g + 8 * t));
                    w[m][h][2 * g] = v.x;
                    w[m][h][2 * g + 1] = v.y;
                }
            } else {
#pragma unroll
                for (int g = 0; g < 4; ++g) w[m][h][g] = xg::lds32(row + (uint32_t)(16 * g + 4 * t));
            }
        }
}

template <int GB> __global__ void __launch_bounds__(B_WARPS * 32, 8) gated_bytes_kernel(const FewArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    // [warp][AHEAD] column blocks, later the warps' sums; then [group of the run][32 rows] s | z << 16
    uint32_t *sc = reinterpret_cast<uint32_t *>(smem + B_WARPS * AHEAD * BLOCK_BYTES);
    float(*sums)[32][9] = reinterpret_cast<float(*)[32][9]>(smem);
    static_assert(sizeof(float) * 32 * 9 <= AHEAD * BLOCK_BYTES, "sums of one warp");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
    const int64_t h0 = (int64_t)blockIdx.x * 16, J = a.K >> a.gshift;
    const int blocks = (int)((a.K + 127) / 128), per_run = (int)(((int64_t)a.run << a.gshift) / 128);
    const uint32_t ring = smem_addr(smem) + (uint32_t)(warp * AHEAD * BLOCK_BYTES);

    const uint8_t *p[2][2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t row = h0 + r + 8 * h;
            p[m][h] = a.w[m].codes + (row < a.H ? row : a.H - 1) * (a.K >> 1) + 16 * t;
        }
    auto fetch = [&](int b, int slot) {
        if (b < blocks) {
            const bool in = GB == 128 || (int64_t)b * 128 + 32 * t < a.K;  // the last block may be cut at a group
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    copy16(ring + (uint32_t)(slot * BLOCK_BYTES + (2 * m + h) * 512 + lane * 16),
                           in ? p[m][h] + (int64_t)b * 64 : a.w[m].codes, in);
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) fetch(warp + i * B_WARPS, i);

    // this lane's byte column of each product (one that does not exist repeats the last: its sums are
    // not used)
    const int8_t *xp = a.v.x + (int64_t)(r < 3 * a.M ? r : 3 * a.M - 1) * a.K + (GB / 4) * t;
    float acc[2][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][i] = 0.0f;

    int b = warp, slot = 0;
    for (int run0 = 0; run0 < blocks; run0 += per_run) {
        const int run1 = run0 + per_run < blocks ? run0 + per_run : blocks;
        const int j0 = (int)(((int64_t)run0 * 128) >> a.gshift), j1 = j0 + a.run < J ? j0 + a.run : (int)J;
        if (run0 > 0) __syncthreads();  // the previous run's readers
        for (int row = warp; row < 32; row += B_WARPS) {
            const Weight &w = a.w[row >> 4];
            const int64_t h = (h0 + (row & 15) < a.H ? h0 + (row & 15) : a.H - 1) * J;
            for (int j = j0 + lane; j < j1; j += 32) {
                const uint32_t s = __ldg(w.scales + h + j);
                const uint32_t z = w.zeros ? (uint32_t)(uint16_t)__ldg(w.zeros + h + j) : 8u;
                sc[(j - j0) * 32 + row] = s | (z << 16);
            }
        }
        __syncthreads();
        if (run0 == 0) asm volatile("griddepcontrol.wait;" ::: "memory");  // the bytes are bytes_prep_kernel's
        for (; b < run1; b += B_WARPS) {
            const int k0 = b * 128;
            copy_wait<AHEAD - 1>();
            __syncwarp();
            uint32_t w[2][2][4];
            block_words<GB>(ring + (uint32_t)(slot * BLOCK_BYTES), r, t, w);
            __syncwarp();
            fetch(b + AHEAD * B_WARPS, slot);
            slot = slot + 1 == AHEAD ? 0 : slot + 1;
#pragma unroll
            for (int g = 0; g < 128 / GB; ++g) {
                if (GB != 128 && k0 + g * GB >= a.K) break;
                const int slice = (k0 + g * GB) / GB;
                const uint32_t *sg = sc + (((k0 + g * GB) >> a.gshift) - j0) * 32;
                float s[2][2];
                int z[2][2];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t sz = sg[16 * m + r + 8 * h];
                        s[m][h] = __half2float(__ushort_as_half((unsigned short)(sz & 0xFFFFu)));
                        z[m][h] = (int)(int16_t)(sz >> 16);
                    }
                // eight bytes of this lane's column for each of the group's words
                uint32_t x[8];
                const int8_t *q = xp + k0 + g * GB;
                if (GB >= 64) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(q);
                    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
                } else {
                    const uint2 u = *reinterpret_cast<const uint2 *>(q);
                    x[0] = u.x; x[1] = u.y;
                }
                if (GB == 128) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(q + 16);
                    x[4] = u.x; x[5] = u.y; x[6] = u.z; x[7] = u.w;
                }
                const float2 f = *reinterpret_cast<const float2 *>(a.v.f + (int64_t)slice * 8 + 2 * t);
                const int2 d = *reinterpret_cast<const int2 *>(a.v.sum + (int64_t)slice * 8 + 2 * t);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    int P[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int i = 0; i < GB / 32; ++i) {
                        const uint32_t lo = w[m][0][(GB / 32) * g + i], hi = w[m][1][(GB / 32) * g + i];
                        mma16832(P, lo & 0x0F0F0F0Fu, hi & 0x0F0F0F0Fu, (lo >> 4) & 0x0F0F0F0Fu, (hi >> 4) & 0x0F0F0F0Fu,
                                 x[2 * i], x[2 * i + 1]);
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        acc[m][2 * h] = fmaf(s[m][h] * f.x, (float)(P[2 * h] - z[m][h] * d.x), acc[m][2 * h]);
                        acc[m][2 * h + 1] = fmaf(s[m][h] * f.y, (float)(P[2 * h + 1] - z[m][h] * d.y), acc[m][2 * h + 1]);
                    }
                }
            }
        }
    }
    // the warps' sums take the place of the codes: rows r and r + 8 of each fragment, columns 2 t and
    // 2 t + 1
    copy_wait<0>();
    __syncthreads();
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) sums[warp][16 * m + r + 8 * (i >> 1)][2 * t + (i & 1)] = acc[m][i];
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * a.M; i += B_WARPS * 32) {
        const int f = i & 15, c = 3 * (i >> 4);
        float g = 0.0f, u = 0.0f;
#pragma unroll
        for (int k = 2; k >= 0; --k)  // the large bytes first
#pragma unroll
            for (int w = 0; w < B_WARPS; ++w) {
                g += sums[w][f][c + k];
                u += sums[w][16 + f][c + k];
            }
        if (h0 + f < a.H) a.y[(int64_t)(i >> 4) * a.H + h0 + f] = __float2bfloat16_rn(act_of(g, a.act == W4_ACT_GELU_TANH).value * u);
    }
}

// The kernel of the bytes, and its workspace (behind the arrival counters of the other shapes' calls,
// which stay zero).
inline bool by_bytes(int64_t M, int64_t H, int64_t K) { return M <= 2 && H * K >= ((int64_t)1 << 25); }

struct BytesPlace {
    size_t x, f, sum, end;
};
inline BytesPlace bytes_place(int64_t M, int64_t K, int group) {
    const size_t slices = (size_t)(K / (group < 128 ? group : 128));
    BytesPlace q;
    q.x = xg::CNT_BYTES;
    q.f = (q.x + (size_t)(3 * M * K) + 255) / 256 * 256;
    q.sum = (q.f + slices * 8 * 4 + 255) / 256 * 256;
    q.end = (q.sum + slices * 8 * 4 + 255) / 256 * 256;
    return q;
}

template <int GB> w4_status launch_few(const FewArgs &a, cudaStream_t stream) {
    const unsigned grid = (unsigned)((a.H + 15) / 16);
    const size_t scales = (size_t)a.run * 32 * sizeof(uint32_t);
    if (by_bytes(a.M, a.H, a.K)) {
        const int64_t warps = a.K / GB * a.M;
        bytes_prep_kernel<GB><<<(unsigned)((warps + 3) / 4), 128, 0, stream>>>(a);
        const w4_status st = launch_status();
        return st != W4_OK ? st : xg::launch_behind(gated_bytes_kernel<GB>, grid, B_WARPS * 32,
                                                    (size_t)(B_WARPS * AHEAD * BLOCK_BYTES) + scales, stream, 1, 1, a);
    }
    if (a.M <= 8)
        gated_few_kernel<GB, 1><<<grid, WARPS * 32, scales, stream>>>(a);
    else
        gated_few_kernel<GB, 2><<<grid, WARPS * 32, scales, stream>>>(a);
    return launch_status();
}
static_assert(B_WARPS * AHEAD * BLOCK_BYTES + MAX_RUN * 128 <= 48 * 1024, "no opt-in to more shared memory");

inline w4_status gated_few(FewArgs a, int group, cudaStream_t stream) {
    // a run holds whole blocks of 128 columns and of the group
    const int64_t J = a.K >> a.gshift;
    a.run = J < MAX_RUN ? (int)((J + 3) / 4 * 4) : MAX_RUN;
    return group == 32 ? launch_few<32>(a, stream) : group == 64 ? launch_few<64>(a, stream) : launch_few<128>(a, stream);
}

}  // namespace gated
}  // namespace w4

using namespace w4;

namespace {

constexpr int64_t kFewRows = 16;  // up to here w4a16_gated reads the weights as a decode step does

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
    if (!xg::shape_ok(M, H, K) || !valid_group(group) || K % group != 0) return 0;
    if (M <= kFewRows) return gated::by_bytes(M, H, K) ? gated::bytes_place(M, K, group).end : 0;
    return xg::place_prep(xg::make_plan(xg::FWD, H, M, K, 1, num_sms()).bytes, M * K, M).end;
}

W4_API w4_status w4a16_gated_schedule(int64_t M, int64_t H, int64_t K, int group, int sms, int64_t *out) {
    if (!out) return W4_ERR_NULL;
    if (!xg::shape_ok(M, H, K) || sms < 1 || sms > 4096) return W4_ERR_SHAPE;
    if (!valid_group(group) || K % group != 0) return W4_ERR_GROUP;
    for (int i = 0; i < 8; ++i) out[i] = 0;
    if (M > kFewRows) xg::describe(xg::make_plan(xg::FWD, H, M, K, 1, sms), sms, out);
    return W4_OK;
}

W4_API w4_status w4a16_gated(const void *X_bf16, int64_t M, const uint8_t *codes_gate, const uint16_t *scales_gate,
                             const int16_t *zeros_gate, const uint8_t *codes_up, const uint16_t *scales_up,
                             const int16_t *zeros_up, int64_t H, int64_t K, int group, int mode, int act, void *Y_bf16,
                             void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (!X_bf16 || !Y_bf16) return W4_ERR_NULL;
    if (!xg::shape_ok(M, H, K)) return W4_ERR_SHAPE;
    if (!valid_group(group) || K % group != 0) return W4_ERR_GROUP;
    if (!valid_mode(mode) || (act != W4_ACT_SILU && act != W4_ACT_GELU_TANH)) return W4_ERR_ARG;
    w4_status st = weight_ok(codes_gate, scales_gate, zeros_gate, mode);
    if (st == W4_OK) st = weight_ok(codes_up, scales_up, zeros_up, mode);
    if (st != W4_OK) return st;
    if (!aligned16(X_bf16) || !aligned16(Y_bf16) || (workspace && !aligned16(workspace))) return W4_ERR_ALIGN;
    if (M <= kFewRows) {
        gated::FewArgs f = {};
        if (gated::by_bytes(M, H, K)) {
            const gated::BytesPlace q = gated::bytes_place(M, K, group);
            if (!workspace || workspace_bytes < q.end) return W4_ERR_WORKSPACE;
            uint8_t *ws = static_cast<uint8_t *>(workspace);
            f.v.x = reinterpret_cast<int8_t *>(ws + q.x);
            f.v.f = reinterpret_cast<float *>(ws + q.f);
            f.v.sum = reinterpret_cast<int *>(ws + q.sum);
        }
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
    const xg::Plan p = xg::make_plan(xg::FWD, H, M, K, 1, sms);
    const xg::PrepPlace q = xg::place_prep(p.bytes, M * K, M);
    if (!workspace || workspace_bytes < q.end) return W4_ERR_WORKSPACE;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    xg::Maps tm;
    if (!xg::make_map(&tm.b[0], ws + q.y, M, K, p.box)) return W4_ERR_CUDA;
    tm.b[1] = tm.b[0];
    xg::Prep prep = {};
    prep.x[0] = static_cast<const __nv_bfloat16 *>(X_bf16);
    prep.y[0] = reinterpret_cast<__half *>(ws + q.y);
    prep.row_pow = reinterpret_cast<float *>(ws + q.row_pow);
    prep.M = M;
    prep.K = K;
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
    return act == W4_ACT_SILU ? xg::launch<xg::FWD, false, false>(p, tm, a, workspace, sms, stream)
                              : xg::launch<xg::FWD, false, true>(p, tm, a, workspace, sms, stream);
}

namespace {

// Workspace of the backward pass: counters and partial sums of its two products, then the fp16 rows
// that each multiplies (X, and after it dG and dU), each time in the same place, and the rests of dG
// and dU.
struct BwdLayout {
    xg::Plan grads, dx;
    xg::PrepPlace q;
    size_t end;
};
BwdLayout bwd_layout(int64_t M, int64_t H, int64_t K, int sms) {
    BwdLayout l;
    l.grads = xg::make_plan(xg::FWD, H, M, K, 1, sms, true);
    l.dx = xg::make_plan(xg::DGRAD, K, M, H, 2, sms);
    l.q = xg::place_prep(l.grads.bytes > l.dx.bytes ? l.grads.bytes : l.dx.bytes, M * (K > 2 * H ? K : 2 * H), M);
    l.end = (l.q.end + (size_t)(M * H) * 2 + 255) / 256 * 256;
    return l;
}

}  // namespace

W4_API size_t w4a16_gated_bwd_workspace_bytes(int64_t M, int64_t H, int64_t K, int group, int from_ckpt) {
    if (!xg::shape_ok(M, H, K) || H % 8 != 0 || !valid_group(group) || K % group != 0) return 0;
    (void)from_ckpt;  // both sources become the same fp16 rows
    return bwd_layout(M, H, K, num_sms()).end;
}

W4_API w4_status w4a16_gated_bwd_schedule(int64_t M, int64_t H, int64_t K, int group, int sms, int64_t *out) {
    if (!out) return W4_ERR_NULL;
    if (!xg::shape_ok(M, H, K) || H % 8 != 0 || sms < 1 || sms > 4096) return W4_ERR_SHAPE;
    if (!valid_group(group) || K % group != 0) return W4_ERR_GROUP;
    const BwdLayout l = bwd_layout(M, H, K, sms);
    xg::describe(l.grads, sms, out);
    xg::describe(l.dx, sms, out + 8);
    return W4_OK;
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
    if (!xg::shape_ok(M, H, K) || H % 8 != 0) return W4_ERR_SHAPE;
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
    if (!workspace || workspace_bytes < l.end) return W4_ERR_WORKSPACE;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    xg::Prep prep = {};
    prep.x[0] = static_cast<const __nv_bfloat16 *>(X_bf16);
    prep.x8 = X_e4m3;
    prep.xs = X_scale;
    prep.y[0] = reinterpret_cast<__half *>(ws + l.q.y);
    prep.row_pow = reinterpret_cast<float *>(ws + l.q.row_pow);
    prep.M = M;
    prep.K = K;
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
    a.dh = static_cast<const __nv_bfloat16 *>(dH_bf16);
    a.out = dG_bf16;
    a.out2 = static_cast<__nv_bfloat16 *>(dU_bf16);
    a.rest = dX_bf16 ? reinterpret_cast<uint16_t *>(ws + l.q.end) : nullptr;
    a.row_pow = prep.row_pow;
    if (!xg::make_map(&tm.b[0], prep.y[0], M, K, l.grads.box)) return W4_ERR_CUDA;
    tm.b[1] = tm.b[0];
    st = act == W4_ACT_SILU ? xg::launch<xg::FWD, true, false>(l.grads, tm, a, workspace, sms, stream)
                            : xg::launch<xg::FWD, true, true>(l.grads, tm, a, workspace, sms, stream);
    if (st != W4_OK || !dX_bf16) return st;
    prep.x[0] = static_cast<const __nv_bfloat16 *>(dG_bf16);
    prep.x[1] = static_cast<const __nv_bfloat16 *>(dU_bf16);
    prep.rest = a.rest;
    prep.x8 = prep.xs = nullptr;
    prep.y[1] = prep.y[0] + M * H;
    prep.K = H;
    st = xg::launch_prep(prep, stream);
    if (st != W4_OK) return st;
    if (!xg::make_map(&tm.b[0], prep.y[0], M, H, l.dx.box) || !xg::make_map(&tm.b[1], prep.y[1], M, H, l.dx.box))
        return W4_ERR_CUDA;
    a.dh = nullptr;
    a.out = dX_bf16;
    a.out2 = nullptr;
    a.rest = nullptr;
    return xg::launch<xg::DGRAD, false, false>(l.dx, tm, a, workspace, sms, stream);
}

W4_API size_t w4a16_dgrad_workspace_bytes(int64_t M, int64_t N, int64_t K, int group) {
    if (!xg::shape_ok(M, N, K) || N % 8 != 0 || !valid_group(group) || K % group != 0) return 0;
    return xg::place_prep(xg::make_plan(xg::DGRAD, K, M, N, 1, num_sms()).bytes, M * N, M).end;
}

W4_API w4_status w4a16_dgrad_schedule(int64_t M, int64_t N, int64_t K, int group, int sms, int64_t *out) {
    if (!out) return W4_ERR_NULL;
    if (!xg::shape_ok(M, N, K) || N % 8 != 0 || sms < 1 || sms > 4096) return W4_ERR_SHAPE;
    if (!valid_group(group) || K % group != 0) return W4_ERR_GROUP;
    xg::describe(xg::make_plan(xg::DGRAD, K, M, N, 1, sms), sms, out);
    return W4_OK;
}

W4_API w4_status w4a16_dgrad(const void *dY_bf16, int64_t M, const uint8_t *codes, const uint16_t *scales,
                             const int16_t *zeros, int64_t N, int64_t K, int group, int mode, void *dX_bf16,
                             void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (!dY_bf16 || !dX_bf16) return W4_ERR_NULL;
    if (!xg::shape_ok(M, N, K) || N % 8 != 0) return W4_ERR_SHAPE;
    if (!valid_group(group) || K % group != 0) return W4_ERR_GROUP;
    if (!valid_mode(mode)) return W4_ERR_ARG;
    w4_status st = weight_ok(codes, scales, zeros, mode);
    if (st != W4_OK) return st;
    if (!aligned16(dY_bf16) || !aligned16(dX_bf16) || (workspace && !aligned16(workspace))) return W4_ERR_ALIGN;
    const int sms = num_sms();
    const xg::Plan p = xg::make_plan(xg::DGRAD, K, M, N, 1, sms);
    const xg::PrepPlace q = xg::place_prep(p.bytes, M * N, M);
    if (!workspace || workspace_bytes < q.end) return W4_ERR_WORKSPACE;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    xg::Maps tm;
    if (!xg::make_map(&tm.b[0], ws + q.y, M, N, p.box)) return W4_ERR_CUDA;
    tm.b[1] = tm.b[0];
    xg::Prep prep = {};
    prep.x[0] = static_cast<const __nv_bfloat16 *>(dY_bf16);
    prep.y[0] = reinterpret_cast<__half *>(ws + q.y);
    prep.row_pow = reinterpret_cast<float *>(ws + q.row_pow);
    prep.M = M;
    prep.K = N;
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
    return xg::launch<xg::DGRAD, false, false>(p, tm, a, workspace, sms, stream);
}
