// Matrix products with one operand expanded inside the kernel, on the sm_100a tensor cores:
// the gated feed-forward block over 4-bit weights, its backward pass, the input gradient of a
// 4-bit layer and the weight gradient from an 8-bit checkpoint are all
//     D[i, c] = sum_r A[i, r] B[c, r],     i: 128 lanes of a tile, c: up to 256 columns
// with A expanded to 16 bits by the kernel's own warps and B 16-bit in memory:
//   FWD    A = 64 gate rows and 64 up rows of the weights, r = their K columns; B = X [token, K]
//   DGRAD  A = 128 columns k of the weight(s), r = weight rows n;               B = dY [token, N]
//   WGRAD  A = 128 columns k of the checkpoint, r = tokens;                      B = dY^T (c = n)
// FWD and DGRAD multiply in fp16: a weight (q - z) s then takes one rounding of 2^-11, an eighth of
// bf16's, and bf16 activations are exact in fp16 once each token's row is divided by a power of
// two (row_prep_kernel writes that copy; the epilogue multiplies the power back). WGRAD multiplies
// in bf16, in which both operands are exact.
// In FWD a row of A is contiguous along r (K-major); in DGRAD and WGRAD it is contiguous along i
// (MN-major, which the MMA reads as it stands), so the expansion writes the same bytes either way:
// 16-byte chunks of eight k, at the place that the 128-byte swizzle gives them.
//
// One persistent CTA per SM takes units (tile, part of the reduction). Warps 0-7 expand A: thread
// t takes 32 consecutive values a stage (a row's half block of 64 columns, or a quarter of a row
// of 128), loaded straight into registers LOOKAHEAD stages ahead, so that every value's group
// scale is a single one. Warp 12 loads B by TMA, warp 13 issues the MMAs (M = 128, N = the token
// tile, K = 16), warps 8-11 read the fp32 accumulators (two buffers in TMEM, so that a tile's
// results leave while the next one is multiplied). Lanes are weights and columns are tokens: a
// small batch takes a small N and the MMAs shrink with it, while the expansion is shared by all
// tokens of a tile.
//
// Where the tiles are too few for the SMs, the reduction is cut into S parts: each part's fp32 sums
// go to the workspace and the last part to finish adds them in order, so results do not depend on
// timing. Every wait is bounded (W4_ERR_TIMEOUT in the device status).
#pragma once

#include "w4_common.cuh"

#include <cuda.h>

#include <atomic>

namespace w4 {
namespace xg {

enum Kind { FWD = 0, DGRAD = 1, WGRAD = 2 };

constexpr int THREADS = 448;
constexpr int EXPAND_WARPS = 8;
constexpr int BK = 64;                        // reduction per stage
constexpr uint32_t A_BYTES = 128 * BK * 2;    // an expanded stage
constexpr int MAX_STAGES = 8;
constexpr uint32_t SMEM_RING = 200 * 1024;
constexpr int LOOKAHEAD = 4;                  // stages whose codes are on their way to registers
constexpr uint64_t kWaitNs = 2000000000ull;

struct Smem {
    uint64_t full[MAX_STAGES];    // B landed (TMA bytes) and A expanded (one arrival per warp)
    uint64_t empty[MAX_STAGES];   // the stage's MMAs completed (commit)
    uint64_t accf[2];             // an accumulator is complete (commit)
    uint64_t acce[2];             // its columns were read (one arrival per warp)
    uint32_t tmem_base;
    int abort;
};
static_assert(sizeof(Smem) <= 1024, "control block");

struct Weight {
    const uint8_t *codes;     // [N, K/2]
    const uint16_t *scales;   // [N, K/g] fp16 bits
    const int16_t *zeros;     // [N, K/g], NULL for symmetric weights (z = 8)
};

struct Args {
    Weight w[2];              // FWD: gate, up; DGRAD: one or two sources
    const uint8_t *x8, *xs;   // WGRAD: checkpoint values [rows, K] and scale bytes [rows, K/32]
    const __nv_bfloat16 *dh;  // FWD: NULL, or [cols, rows]: write the gradients of both projections
    void *out;                // FWD: Y or dG [cols, rows]; DGRAD: dX [cols, K]; WGRAD: dW [cols, K]
    __nv_bfloat16 *out2;      // FWD with dh: dU
    const float *row_pow;     // FWD, DGRAD: the power of two that each token's row was divided by
    float *part;              // partial sums [tile][part][column][lane]
    uint32_t *cnt;            // arrival counters [tile][4], zero between calls
    int *status;
    int64_t rows;             // weight rows (FWD, DGRAD: of one source) or tokens (WGRAD)
    int64_t K;                // columns of the expanded matrix
    int64_t cols;             // tokens, or dY's columns (WGRAD)
    int64_t units;            // Tw * Tn * S
    int Tw, S;                // lane tiles, parts of the reduction
    int KB, KB0;              // stages of the whole reduction, and of the first source
    int seg;                  // stages that one fp32 accumulator sums at most
    int NT;                   // columns per tile, a multiple of 16
    int stages;
    uint32_t stage_bytes;
    int gshift, act, out_fp32;
};

__device__ __forceinline__ void mma(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
    // descriptor high word: 1024 bytes between groups of eight rows, version 1, 128-byte swizzle
    constexpr uint32_t hi = 64u | (1u << 14) | (2u << 29);
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.b32 p, %4, 0;\n mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(hi));
}
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ uint32_t hsub(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t hadd(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t hmul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t hfma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t bmul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t hpair(float v) {  // v, rounded to fp16, in both halves
    const uint32_t b = __half_as_ushort(__float2half_rn(v));
    return b | (b << 16);
}

// The scale and zero point of 32 values, as the constants of their expansion. A weight is
// (q - z) s rounded once to fp16: q enters the mantissa of 1024.0 (1024 + q, exact), less 1024 + z
// is q - z (exact for |z| <= 1024), times the fp16 scale as it is. Zero points beyond that
// (groups of one sign far from zero) take ((q - 8) s + c_lo) + c_hi with (8 - z) s = c_hi + c_lo,
// of which again only the last operation rounds at the weight's size.
struct Scale {
    uint32_t s, zc;        // s, 1024 + z
    uint32_t ch, cl;       // (8 - z) s, split
    bool far;
};
__device__ __forceinline__ Scale scale_of(uint32_t sz) {
    Scale c;
    c.s = __byte_perm(sz, 0, 0x1010);
    const int z = (int)(int16_t)(sz >> 16);
    c.far = z > 1024 || z < -1024;
    c.zc = hpair((float)(1024 + z));
    c.ch = c.cl = 0u;
    if (c.far) {
        const float k = (float)(8 - z) * __half2float(__ushort_as_half((unsigned short)(sz & 0xFFFFu)));
        c.ch = hpair(k);
        c.cl = hpair(k - __half2float(__ushort_as_half((unsigned short)(c.ch & 0xFFFFu))));
    }
    return c;
}
// eight codes (nibble i is value i) as fp16, in order
__device__ __forceinline__ void expand8(uint32_t w, const Scale &c, uint32_t (&o)[4]) {
    uint32_t p[4];  // pairs (i, i + 4)
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = ((w >> (4 * i)) & 0x000F000Fu) | 0x64006400u;
    if (!c.far) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = hmul(hsub(p[i], c.zc), c.s);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = hadd(hfma(hsub(p[i], 0x64086408u), c.s, c.cl), c.ch);
    }
    o[0] = __byte_perm(p[0], p[1], 0x5410);
    o[1] = __byte_perm(p[2], p[3], 0x5410);
    o[2] = __byte_perm(p[0], p[1], 0x7632);
    o[3] = __byte_perm(p[2], p[3], 0x7632);
}
// four E4M3 bytes as bf16 pairs, times 2^e: the value's seven exponent and mantissa bits under
// bf16's exponent read as the value times 2^-120 (subnormals too), so one multiplication by
// 2^(120 + e) restores it exactly; two where that power is past bf16's range.
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t t) {  // bytes in the high halves' places
    return ((t >> 4) & 0x07F007F0u) | (t & 0x80008000u);
}
struct Pow2 {
    uint32_t f1, f2;
    bool two;
};
__device__ __forceinline__ Pow2 pow2_of(uint32_t b) {  // scale byte e + 127; 255 is NaN
    Pow2 p;
    p.two = b > 134u;
    const uint32_t one = p.two ? 0x7B80u : (120u + b) << 7;        // 2^120, or 2^(120 + e)
    const uint32_t two = b == 255u ? 0x7FC0u : b << 7;
    p.f1 = b == 0u ? 0u : one | (one << 16);
    p.f2 = two | (two << 16);
    return p;
}
__device__ __forceinline__ void expand4(uint32_t w, const Pow2 &p, uint32_t &o0, uint32_t &o1) {
    o0 = bmul(e4m3_pair(__byte_perm(w, 0, 0x1404)), p.f1);
    o1 = bmul(e4m3_pair(__byte_perm(w, 0, 0x3424)), p.f1);
    if (p.two) {
        o0 = bmul(o0, p.f2);
        o1 = bmul(o1, p.f2);
    }
}

__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, Smem *sm, int *status) {
    bool r = true;
    if ((threadIdx.x & 31) == 0) r = mbar_wait_abortable(bar, parity, &sm->abort, status, kWaitNs);
    r = __shfl_sync(FULL, r ? 1 : 0, 0) != 0;
    __syncwarp();
    return r;
}
__device__ __forceinline__ bool wait1(uint64_t *bar, uint32_t parity, Smem *sm, int *status) {
    return mbar_wait_abortable<true>(bar, parity, &sm->abort, status, kWaitNs);
}

// act(g) and act'(g)
__device__ __forceinline__ float act_of(float g, int act) {
    if (act == W4_ACT_SILU) return g / (1.0f + __expf(-g));
    const float t = tanhf(0.7978845608028654f * (g + 0.044715f * g * g * g));
    return 0.5f * g * (1.0f + t);
}
__device__ __forceinline__ float slope_of(float g, int act) {
    if (act == W4_ACT_SILU) {
        const float s = 1.0f / (1.0f + __expf(-g));
        return s * (1.0f + g * (1.0f - s));
    }
    const float t = tanhf(0.7978845608028654f * (g + 0.044715f * g * g * g));
    return 0.5f * (1.0f + t) + 0.5f * g * (1.0f - t * t) * 0.7978845608028654f * (1.0f + 3.0f * 0.044715f * g * g);
}

// A unit: its tile, its part of the reduction (stages [b0, b1)) and its place in the partial sums.
struct Unit {
    int64_t tile, tw, tn, s;
    int b0, b1;
};
__device__ __forceinline__ Unit unit_of(const Args &a, int64_t u) {
    Unit t;
    t.tw = u % a.Tw;
    const int64_t r = u / a.Tw;
    t.s = r % a.S;
    t.tn = r / a.S;
    t.tile = t.tn * a.Tw + t.tw;
    t.b0 = (int)(t.s * a.KB / a.S);
    t.b1 = (int)((t.s + 1) * a.KB / a.S);
    return t;
}

// The values that one thread expands in one stage, and where they come from.
template <int KIND> struct Chunk {
    uint4 q[KIND == WGRAD ? 2 : 1];
    uint32_t s;               // scale and zero point, or the scale byte
};

template <int KIND> struct Loader {
    int64_t u;
    int kb, b1;
    bool ok;                  // this thread's row or columns exist
    const uint8_t *q;         // its values in stage kb
    const uint16_t *sc;
    const int16_t *zp;
    int64_t k, row;           // its column (in stage 0 for FWD) and row

    __device__ __forceinline__ void begin(const Args &a, int t) {
        const Unit un = unit_of(a, u);
        kb = un.b0;
        b1 = un.b1;
        if (KIND == FWD) {
            const int r = t >> 1;
            const int i = r & 31;
            row = un.tw * 64 + 16 * (r >> 5) + (i & 15);
            const Weight &w = a.w[i >> 4];
            ok = row < a.rows;
            k = 32 * (t & 1);
            q = w.codes + row * (a.K >> 1) + (k >> 1);
            sc = w.scales + row * (a.K >> a.gshift);
            zp = w.zeros ? w.zeros + row * (a.K >> a.gshift) : nullptr;
        } else {
            k = un.tw * 128 + 32 * (t & 3);
            ok = k < a.K;
        }
    }
    __device__ __forceinline__ void load(const Args &a, int t, Chunk<KIND> &c) {
        if (KIND == FWD) {
            const int64_t kk = (int64_t)kb * BK + k;
            if (ok && kk < a.K) {
                c.q[0] = ldg_stream(q + (int64_t)kb * (BK / 2));
                const int64_t j = kk >> a.gshift;
                c.s = (uint32_t)__ldg(sc + j) | ((zp ? (uint32_t)(uint16_t)__ldg(zp + j) : 8u) << 16);
            } else {
                c.q[0] = make_uint4(0, 0, 0, 0);
                c.s = 8u << 16;
            }
        } else if (KIND == DGRAD) {
            const int src = kb >= a.KB0 ? 1 : 0;
            const int64_t n = (int64_t)(kb - (src ? a.KB0 : 0)) * BK + (t >> 2);
            if (ok && n < a.rows) {
                const Weight &w = a.w[src];
                c.q[0] = ldg_stream(w.codes + n * (a.K >> 1) + (k >> 1));
                const int64_t j = n * (a.K >> a.gshift) + (k >> a.gshift);
                c.s = (uint32_t)__ldg(w.scales + j) | ((w.zeros ? (uint32_t)(uint16_t)__ldg(w.zeros + j) : 8u) << 16);
            } else {
                c.q[0] = make_uint4(0, 0, 0, 0);
                c.s = 8u << 16;
            }
        } else {
            const int64_t m = (int64_t)kb * BK + (t >> 2);
            if (ok && m < a.rows) {
                const uint8_t *p = a.x8 + m * a.K + k;
                c.q[0] = ldg_stream(p);
                c.q[KIND == WGRAD ? 1 : 0] = ldg_stream(p + 16);
                c.s = __ldg(a.xs + m * (a.K >> 5) + (k >> 5));
            } else {
                c.q[0] = c.q[KIND == WGRAD ? 1 : 0] = make_uint4(0, 0, 0, 0);
                c.s = 127u;
            }
        }
        if (++kb == b1) {
            u += gridDim.x;
            if (u < a.units) begin(a, t);
        }
    }
};

// thread t's chunk into the A tile at `base`
template <int KIND> __device__ __forceinline__ void expand_store(const Chunk<KIND> &c, uint32_t base, int t) {
    if (KIND == WGRAD) {
        const int row = t >> 2, x = row & 7, c0 = 4 * (t & 1);
        const uint32_t at = base + (uint32_t)((t >> 1) & 1) * 8192u + (uint32_t)row * 128u;
        const Pow2 p = pow2_of(c.s);
        const bool f = (t & 2) != 0;  // chunk order as for DGRAD below
        const uint4 q0 = c.q[0], q1 = c.q[KIND == WGRAD ? 1 : 0];
        const uint4 v[2] = {f ? q1 : q0, f ? q0 : q1};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t o[4];
            expand4(i & 1 ? v[i >> 1].z : v[i >> 1].x, p, o[0], o[1]);
            expand4(i & 1 ? v[i >> 1].w : v[i >> 1].y, p, o[2], o[3]);
            sts128(at + (uint32_t)(((c0 + (f ? i ^ 2 : i)) ^ x) << 4), o[0], o[1], o[2], o[3]);
        }
        return;
    }
    const Scale s = scale_of(c.s);
    const uint4 v = c.q[0];
    if (KIND == FWD) {
        const int row = t >> 1, x = row & 7, c0 = 4 * (t & 1);
        const uint32_t at = base + (uint32_t)row * 128u;
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t o[4];
            expand8(w[i], s, o);
            sts128(at + (uint32_t)(((c0 + i) ^ x) << 4), o[0], o[1], o[2], o[3]);
        }
    } else {
        const int row = t >> 2, x = row & 7, c0 = 4 * (t & 1);
        const uint32_t at = base + (uint32_t)((t >> 1) & 1) * 8192u + (uint32_t)row * 128u;
        // the threads of the second 64 columns write their chunks in the order 2, 3, 0, 1: the
        // eight threads of a quarter warp then write eight different 16-byte bank groups
        const bool f = (t & 2) != 0;
        const uint32_t w[4] = {f ? v.z : v.x, f ? v.w : v.y, f ? v.x : v.z, f ? v.y : v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t o[4];
            expand8(w[i], s, o);
            sts128(at + (uint32_t)(((c0 + (f ? i ^ 2 : i)) ^ x) << 4), o[0], o[1], o[2], o[3]);
        }
    }
}

// Results of columns [c, c + 16) of a tile for this thread's lane.
template <int KIND, bool GRADS>
__device__ __forceinline__ void emit(const Args &a, const Unit &un, int q4, int lane, int c, int ncols,
                                     const float (&v)[16], bool add) {
    if (KIND == FWD) {
        // lanes 0-15 of a warp hold gate rows, lanes 16-31 the same features' up rows: of each pair
        // of tokens the lower half takes the even one and the upper half the odd one
        const bool up = lane >= 16;
        const int64_t h = un.tw * 64 + 16 * q4 + (lane & 15);
        const int64_t tok0 = un.tn * a.NT + c + (up ? 1 : 0);
        float d[8];
        if (GRADS) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                d[i] = (h < a.rows && c + 2 * i + (up ? 1 : 0) < ncols) ? __bfloat162float(a.dh[(tok0 + 2 * i) * a.rows + h])
                                                                        : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float got = __shfl_xor_sync(FULL, up ? v[2 * i] : v[2 * i + 1], 16);
            const float f = a.row_pow[tok0 + 2 * i];
            const float g = f * (up ? got : v[2 * i]), u = f * (up ? v[2 * i + 1] : got);
            if (h < a.rows && c + 2 * i + (up ? 1 : 0) < ncols) {
                const int64_t at = (tok0 + 2 * i) * a.rows + h;
                if (GRADS) {
                    static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(d[i] * u * slope_of(g, a.act));
                    a.out2[at] = __float2bfloat16_rn(d[i] * act_of(g, a.act));
                } else {
                    static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(act_of(g, a.act) * u);
                }
            }
        }
    } else {
        const int64_t k = un.tw * 128 + 32 * q4 + lane;
        if (k >= a.K) return;
        const int64_t at = (un.tn * a.NT + c) * a.K + k;
        if (KIND == WGRAD && a.out_fp32) {
            float *o = static_cast<float *>(a.out) + at;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (c + i < ncols) o[i * a.K] = add ? o[i * a.K] + v[i] : v[i];
        } else {
            __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.out) + at;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (c + i < ncols)
                    o[i * a.K] = __float2bfloat16_rn(KIND == DGRAD ? v[i] * a.row_pow[un.tn * a.NT + c + i] : v[i]);
        }
    }
}

template <int KIND, bool GRADS>
__global__ void __launch_bounds__(THREADS, 1) expand_gemm_kernel(const __grid_constant__ CUtensorMap tm0,
                                                                 const __grid_constant__ CUtensorMap tm1,
                                                                 const __grid_constant__ Args a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Smem *sm = reinterpret_cast<Smem *>(base + (size_t)a.stages * a.stage_bytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int NS = a.stages;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&sm->full[s], 1 + EXPAND_WARPS);
            mbar_init(&sm->empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sm->accf[b], 1);
            mbar_init(&sm->acce[b], 4);
        }
        sm->abort = 0;
        fence_mbar_init();
    }
    if (warp == 13) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sm->tmem_base)),
                     "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm->tmem_base;

    if (warp < EXPAND_WARPS) {
        // ------------------------------------------------ expansion of A
        const int t = threadIdx.x;
        int total = 0;
        for (int64_t u = blockIdx.x; u < a.units; u += gridDim.x) {
            const Unit un = unit_of(a, u);
            total += un.b1 - un.b0;
        }
        Loader<KIND> ld;
        ld.u = blockIdx.x;
        ld.begin(a, t);
        Chunk<KIND> ch[LOOKAHEAD];
#pragma unroll
        for (int j = 0; j < LOOKAHEAD; ++j)
            if (j < total) ld.load(a, t, ch[j]);
        int slot = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int i = 0; i < total && ok; i += LOOKAHEAD) {
#pragma unroll
            for (int j = 0; j < LOOKAHEAD; ++j) {
                if (i + j >= total) break;
                if (!warp_wait(&sm->empty[slot], phase ^ 1u, sm, a.status)) { ok = false; break; }
                expand_store<KIND>(ch[j], smem_addr(base + (size_t)slot * a.stage_bytes), t);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the MMA reads them
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->full[slot]);
                if (i + j + LOOKAHEAD < total) ld.load(a, t, ch[j]);
                if (++slot == NS) { slot = 0; phase ^= 1u; }
            }
        }
    } else if (warp == 12) {
        // ------------------------------------------------ B by TMA
        if (lane == 0) {
            if (KIND != WGRAD) asm volatile("griddepcontrol.wait;" ::: "memory");  // B is row_prep_kernel's
            int slot = 0, issued = 0;
            uint32_t phase = 0;
            bool ok = true;
            const uint32_t bytes = a.stage_bytes - A_BYTES;
            for (int64_t u = blockIdx.x; u < a.units && ok; u += gridDim.x) {
                const Unit un = unit_of(a, u);
                const int c0 = (int)(un.tn * a.NT);
                for (int kb = un.b0; kb < un.b1; ++kb) {
                    if (!wait1(&sm->empty[slot], phase ^ 1u, sm, a.status)) { ok = false; break; }
                    uint8_t *dst = base + (size_t)slot * a.stage_bytes + A_BYTES;
                    mbar_arrive_expect_tx(&sm->full[slot], bytes);
                    if (KIND == WGRAD) {
                        for (uint32_t o = 0; o < bytes; o += 8192u)  // 64 columns of dY a box
                            tma_load_2d(dst + o, &tm0, c0 + (int)(o >> 7), kb * BK, &sm->full[slot]);
                    } else if (KIND == DGRAD && kb >= a.KB0) {
                        tma_load_2d(dst, &tm1, (kb - a.KB0) * BK, c0, &sm->full[slot]);
                    } else {
                        tma_load_2d(dst, &tm0, kb * BK, c0, &sm->full[slot]);
                    }
                    ++issued;
                    if (++slot == NS) { slot = 0; phase ^= 1u; }
                }
            }
            // no copy may land after the CTA exits
            for (int i = issued > NS ? issued - NS : 0; i < issued; ++i)
                (void)mbar_wait_bounded(&sm->full[i % NS], (uint32_t)(i / NS) & 1u, a.status);
        }
        __syncwarp();
    } else if (warp == 13) {
        // ------------------------------------------------ MMA issue
        if (lane == 0) {
            // D fp32, A and B fp16 (0) or bf16 (1), M = 128, N = NT; A (and B in WGRAD) contiguous
            // along M (N)
            const uint32_t idesc = (1u << 4) | (KIND == WGRAD ? (1u << 7) | (1u << 10) : 0u) | (KIND != FWD ? 1u << 15 : 0u) |
                                   (KIND == WGRAD ? 1u << 16 : 0u) | ((uint32_t)(a.NT >> 3) << 17) | (8u << 24);
            // low word: address / 16 | leading offset / 16 (K-major: unused; MN-major: 8192 bytes
            // between the 64-element atoms); a K step of 16 is 32 bytes, or 16 rows of 128
            constexpr uint32_t alead = KIND == FWD ? 1u << 16 : 512u << 16, astep = KIND == FWD ? 2u : 128u;
            constexpr uint32_t blead = KIND == WGRAD ? 512u << 16 : 1u << 16, bstep = KIND == WGRAD ? 128u : 2u;
            int slot = 0, done = 0, n = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int64_t u = blockIdx.x; u < a.units && ok; u += gridDim.x) {
                const Unit un = unit_of(a, u);
                for (int s0 = un.b0; s0 < un.b1 && ok; s0 += a.seg, ++n) {
                    const int s1 = un.b1 - s0 < a.seg ? un.b1 : s0 + a.seg;
                    const int buf = n & 1;
                    if (!wait1(&sm->acce[buf], ((uint32_t)(n >> 1) & 1u) ^ 1u, sm, a.status)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t d = tmem + (uint32_t)(buf * 256);
                    for (int kb = s0; kb < s1; ++kb) {
                        if (!wait1(&sm->full[slot], phase, sm, a.status)) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t sa = smem_addr(base + (size_t)slot * a.stage_bytes);
                        const uint32_t alo = (sa >> 4) | alead, blo = ((sa + A_BYTES) >> 4) | blead;
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk)
                            mma(d, alo + kk * astep, blo + kk * bstep, idesc, kb > s0 || kk > 0 ? 1u : 0u);
                        mma_commit(&sm->empty[slot]);
                        ++done;
                        if (++slot == NS) { slot = 0; phase ^= 1u; }
                    }
                    if (ok) mma_commit(&sm->accf[buf]);
                }
            }
            // no commit may arrive after the CTA exits
            for (int i = done > NS ? done - NS : 0; i < done; ++i)
                (void)mbar_wait_bounded(&sm->empty[i % NS], (uint32_t)(i / NS) & 1u, a.status);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ results (lane 32 q4 + lane of the tile)
        const int q4 = warp & 3, r = q4 * 32 + lane;
        const uint32_t tl = tmem + ((uint32_t)(q4 * 32) << 16);
        if (KIND != WGRAD) asm volatile("griddepcontrol.wait;" ::: "memory");  // row_pow too
        int n = 0;
        bool ok = true;
        for (int64_t u = blockIdx.x; u < a.units && ok; u += gridDim.x) {
            const Unit un = unit_of(a, u);
            const int64_t left = a.cols - un.tn * a.NT;
            const int ncols = left < a.NT ? (int)left : a.NT;
            float *part = a.S > 1 ? a.part + ((size_t)(un.tile * a.S + un.s) * a.NT) * 128 + r : nullptr;
            for (int s0 = un.b0; s0 < un.b1; s0 += a.seg, ++n) {
                const int buf = n & 1;
                if (!warp_wait(&sm->accf[buf], (uint32_t)(n >> 1) & 1u, sm, a.status)) { ok = false; break; }
                tc_fence_after();
                for (int c = 0; c < ncols; c += 16) {
                    uint32_t raw[16];
                    tmem_ld16(tl + (uint32_t)(buf * 256 + c), raw);
                    tmem_wait_ld(raw);
                    float v[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(raw[i]);
                    if (a.S > 1) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float *p = part + (size_t)(c + i) * 128;
                            *p = s0 > un.b0 ? *p + v[i] : v[i];
                        }
                    } else {
                        emit<KIND, GRADS>(a, un, q4, lane, c, ncols, v, s0 > un.b0);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->acce[buf]);
            }
            if (!ok || a.S == 1) continue;
            __threadfence();
            __syncwarp();
            uint32_t old = 0;
            if (lane == 0) old = atomicAdd(a.cnt + un.tile * 4 + q4, 1u);
            old = __shfl_sync(FULL, old, 0);
            if (old != (uint32_t)(a.S - 1)) continue;
            // the last part of this tile's 32 lanes: add all parts in order
            __threadfence();
            const float *p0 = a.part + ((size_t)(un.tile * a.S) * a.NT) * 128 + r;
            for (int c = 0; c < ncols; c += 16) {
                float v[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = __ldcg(p0 + (size_t)(c + i) * 128);
                for (int s = 1; s < a.S; ++s) {
                    const float *p = p0 + (size_t)s * a.NT * 128;
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] += __ldcg(p + (size_t)(c + i) * 128);
                }
                emit<KIND, GRADS>(a, un, q4, lane, c, ncols, v, false);
            }
            if (lane == 0) a.cnt[un.tile * 4 + q4] = 0u;  // ready for the next call
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 13)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

// ------------------------------------------------------------------ activations as fp16 rows

// The fp16 copy of bf16 rows that the products above multiply: row m divided by the power of two
// that brings its largest finite value into [2^14, 2^15). A bf16 value within 2^-31 of the
// largest is exact in it; what is smaller is off by 2^-40 of the largest at most. One or two
// tensors of the same rows (the two gradients, which one accumulator sums) share a power; the 8-bit
// checkpoint is restored on the way. One block per row, which it reads twice (the second time from
// L1 or L2); bound by the memory traffic of reading 2 (1) and writing 2 bytes a value.
struct Prep {
    const __nv_bfloat16 *x[2];    // [M, K] each; NULL for the checkpoint
    const uint8_t *x8, *xs;       // checkpoint values [M, K] and scale bytes [M, K/32]
    __half *y[2];                 // [M, K] each
    float *row_pow;               // [M]
    int64_t M, K;
    int tensors;
};

// a non-finite value takes no part in the maximum
__device__ __forceinline__ float finite_abs(float v) {
    const float f = fabsf(v);
    return f <= 3.4e38f ? f : 0.0f;
}

template <bool CKPT> __device__ __forceinline__ void prep_read(const Prep &p, int t, int64_t m, int64_t i, float (&v)[8]) {
    if (CKPT) {
        const uint2 w = __ldg(reinterpret_cast<const uint2 *>(p.x8 + m * p.K) + i);
        const Pow2 f = pow2_of(__ldg(p.xs + m * (p.K >> 5) + (i >> 2)));
        uint32_t o[4];
        expand4(w.x, f, o[0], o[1]);
        expand4(w.y, f, o[2], o[3]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = bf16_lo(o[j]);
            v[2 * j + 1] = bf16_hi(o[j]);
        }
    } else {
        const uint4 w = __ldg(reinterpret_cast<const uint4 *>(p.x[t] + m * p.K) + i);
        const uint32_t o[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = bf16_lo(o[j]);
            v[2 * j + 1] = bf16_hi(o[j]);
        }
    }
}

template <bool CKPT> __global__ void __launch_bounds__(256) row_prep_kernel(const Prep p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ float top[8];
    const int64_t chunks = p.K >> 3;
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
        float mx = 0.0f;
        for (int t = 0; t < p.tensors; ++t)
            for (int64_t i = threadIdx.x; i < chunks; i += 256) {
                float v[8];
                prep_read<CKPT>(p, t, m, i, v);
#pragma unroll
                for (int j = 0; j < 8; ++j) mx = fmaxf(mx, finite_abs(v[j]));
            }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, o));
        __syncthreads();  // the previous row's readers of top
        if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = mx;
        __syncthreads();
        mx = fmaxf(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), fmaxf(fmaxf(top[4], top[5]), fmaxf(top[6], top[7])));
        int e = (int)(__float_as_uint(mx) >> 23);  // the exponent, biased by 127
        if (e < 15) e = mx == 0.0f ? 141 : 15;      // factors stay finite; a row of zeros has factor 1
        const float f = __uint_as_float((uint32_t)(268 - e) << 23);  // 2^(14 - (e - 127))
        if (threadIdx.x == 0) p.row_pow[m] = __uint_as_float((uint32_t)(e - 14) << 23);
        for (int t = 0; t < p.tensors; ++t)
            for (int64_t i = threadIdx.x; i < chunks; i += 256) {
                float v[8];
                prep_read<CKPT>(p, t, m, i, v);
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const __half2 h = __floats2half2_rn(v[2 * j] * f, v[2 * j + 1] * f);
                    o[j] = *reinterpret_cast<const uint32_t *>(&h);
                }
                reinterpret_cast<uint4 *>(p.y[t] + m * p.K)[i] = make_uint4(o[0], o[1], o[2], o[3]);
            }
    }
}

// Place of the fp16 copy (of `values` in all) and of its powers (M of them, and room for the rest
// of a column group, which the epilogue may read beside them) behind the first `at` bytes.
struct PrepPlace {
    size_t y, row_pow, end;
};
inline PrepPlace place_prep(size_t at, int64_t values, int64_t M) {
    PrepPlace q;
    q.y = (at + 255) / 256 * 256;
    q.row_pow = (q.y + (size_t)values * 2 + 255) / 256 * 256;
    q.end = (q.row_pow + ((size_t)M + 16) * sizeof(float) + 255) / 256 * 256;
    return q;
}

inline w4_status launch_prep(const Prep &p, cudaStream_t stream) {
    const unsigned grid = (unsigned)(p.M < (1 << 20) ? p.M : (1 << 20));
    if (p.x8)
        row_prep_kernel<true><<<grid, 256, 0, stream>>>(p);
    else
        row_prep_kernel<false><<<grid, 256, 0, stream>>>(p);
    return launch_status();
}

// ------------------------------------------------------------------ host side

struct Plan {
    int64_t Tw, Tn, units;
    int NT, S, KB, KB0, seg, stages;
    uint32_t stage_bytes;
    size_t bytes;                   // of the workspace, 0 where S is 1
};

// The workspace starts with the arrival counters, in a region of one size for all shapes (what
// one call leaves as partial sums is never another's counter), then holds the partial sums.
constexpr int64_t MAX_SPLIT_TILES = 4096;
constexpr size_t CNT_BYTES = MAX_SPLIT_TILES * 4 * sizeof(uint32_t);

// lanes: weight rows per projection (FWD) or columns K; cols: the other side; red: length of the
// reduction (per source), sources 1 or 2; max_rows: reduction that one accumulator may sum.
inline Plan make_plan(int kind, int64_t lanes, int64_t cols, int64_t red, int sources, int64_t max_rows, int sms) {
    Plan p;
    p.Tw = kind == FWD ? (lanes + 63) / 64 : (lanes + 127) / 128;
    p.Tn = (cols + 255) / 256;
    p.NT = (int)(((cols + p.Tn - 1) / p.Tn + 15) / 16 * 16);
    p.KB0 = (int)((red + BK - 1) / BK);
    p.KB = p.KB0 * sources;
    p.seg = max_rows > 0 && max_rows / BK < p.KB ? (int)(max_rows / BK) : p.KB;
    const uint32_t bb = kind == WGRAD ? (uint32_t)((p.NT + 63) / 64) * 8192u : (uint32_t)p.NT * 128u;
    p.stage_bytes = A_BYTES + bb;
    p.stages = (int)(SMEM_RING / p.stage_bytes);
    if (p.stages > MAX_STAGES) p.stages = MAX_STAGES;
    // Parts of the reduction: the count with the least estimated time. In cycles: a stage takes
    // its MMAs (2 per column) or its expansion (about 300), a unit about 2500 to start and end,
    // and the last part of a tile reads S partial sums at about 60 bytes per cycle.
    const int64_t tiles = p.Tw * p.Tn;
    double best = 0;
    p.S = 1;
    for (int S = 1; S <= 32 && (S == 1 || S * 4 <= p.KB); ++S) {
        if (S > 1 && (tiles * S > 8 * (int64_t)sms || tiles > MAX_SPLIT_TILES)) break;
        const double waves = (double)((tiles * S + sms - 1) / sms);
        const double stage = p.NT * 2 > 300 ? p.NT * 2 : 300;
        const double t = waves * ((double)((p.KB + S - 1) / S) * stage + 2500) + (S > 1 ? 2000 + S * p.NT * 512.0 / 60 : 0);
        if (S == 1 || t < best) {
            best = t;
            p.S = S;
        }
    }
    p.units = tiles * p.S;
    p.bytes = p.S > 1 ? CNT_BYTES + (size_t)p.units * p.NT * 512 : 0;
    return p;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

// 16-bit [rows, width], boxes of 64 columns x box_rows with the 128-byte swizzle; what lies outside
// reads as zero
inline bool make_map(CUtensorMap *tm, const void *p, int64_t rows, int64_t width, int box_rows) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)width * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, es[2] = {1, 1};
    return enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(p), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int KIND, bool GRADS>
w4_status launch(const Plan &p, const CUtensorMap &tm0, const CUtensorMap &tm1, Args a, void *workspace, int sms,
                 cudaStream_t stream) {
    a.units = p.units;
    a.Tw = (int)p.Tw;
    a.S = p.S;
    a.KB = p.KB;
    a.KB0 = p.KB0;
    a.seg = p.seg;
    a.NT = p.NT;
    a.stages = p.stages;
    a.stage_bytes = p.stage_bytes;
    a.cnt = static_cast<uint32_t *>(workspace);
    a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + CNT_BYTES);
    a.status = device_status_ptr();
    if (!a.status) return W4_ERR_CUDA;
    const int smem = (int)(p.stages * p.stage_bytes) + 2048;
    static std::atomic<uint64_t> attr_done{0};  // one bit per device
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = dev >= 0 && dev < 64 ? (uint64_t)1 << dev : 0;
    if (!(attr_done.load(std::memory_order_relaxed) & bit)) {
        if (cudaFuncSetAttribute(expand_gemm_kernel<KIND, GRADS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)SMEM_RING + 2048) != cudaSuccess)
            return W4_ERR_CUDA;
        attr_done.fetch_or(bit, std::memory_order_relaxed);
    }
    const unsigned grid = (unsigned)(p.units < sms ? p.units : sms);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    // FWD and DGRAD follow row_prep_kernel: they may start, and read weights, while it finishes.
    // Whatever came before on the stream was complete when it began.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = KIND == WGRAD ? 0 : 1;
    if (cudaLaunchKernelEx(&cfg, expand_gemm_kernel<KIND, GRADS>, tm0, tm1, a) != cudaSuccess) return W4_ERR_CUDA;
    return launch_status();
}

}  // namespace xg
}  // namespace w4
