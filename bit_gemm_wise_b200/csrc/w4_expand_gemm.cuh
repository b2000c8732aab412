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
// One persistent CTA per SM takes units (tile, part of the reduction), stages of 64 along it. Its warps:
//   0-15 or 0-7  expand A, in four groups that take the stages in turn, so that one group's waits and
//                fences overlap the others' arithmetic. A thread takes two or four chunks of 32
//                consecutive values (half of a row's 64 columns, or a quarter of a row of 128), so that
//                a chunk has a single group scale, which it loads itself a turn ahead;
//   then 4 or 8  read the fp32 accumulators (two buffers in TMEM, so that a tile's results leave while
//                the next one is multiplied) and finish them;
//   one each     loads B by TMA; issues the MMAs (M = 128, N = the token tile, K = 16); loads the codes
//                by TMA, into a ring of their own.
// Lanes are weights and columns are tokens: a small batch takes a small N and the MMAs shrink with
// it, while the expansion is shared by all tokens of a tile. What bounds a stage is the shared memory's
// data path: codes in and out, A in and out and B twice, 128 bytes a cycle, kept it busy for 101% (FWD),
// 98% (DGRAD) and 94% (WGRAD) of a stage's 984, 903 and 836 cycles at N = 256 (192), of which the MMAs
// take 512 (384). So where there are more than 128 columns, two CTAs make a pair: one MMA of both SMs
// (M = 256) on 128 lanes of each, every SM holding half of B, which it writes and reads half as often
// (797, 727 and, at N = 256, 760 cycles a stage). The first CTA of a pair issues the MMAs; the second one
// passes on that its stages are full. Beyond that, instructions count: the codes' pairs (i, i + 4) of
// eight stay in that order, and B's rows (FWD) or the results' lanes (DGRAD, WGRAD) are permuted instead;
// a thread's scale addresses move by one addition. (Not kept: a table of FWD's scales made beforehand,
// side by side for a stage, which loads them in a tenth of the accesses: no faster, and small calls pay
// for it; tiles ordered so that neighbours share their codes in L2: no faster.)
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

constexpr int GROUPS = 4;                     // of expansion warps; stage i is group i % GROUPS's

// How a CTA's warps are divided. Sixteen expansion warps and four for the results leave a thread 80
// registers; where the results take long (two gradients and dH for each pair of accumulators; tiles of
// few stages), eight and eight do better. Us with the two ways in turn, on one GPU:
//                                              one CTA a tile         pairs
//   gated 4096 x 15360 x 3840, silu            944 and 988      848 and 842
//   the same, gelu                             971 and 964      891 and 830
//   gated 512 x 4096 x 4096 in groups of 32   42.7 and 45.1    41.3 and 43.0
//   dgrad 4096 x 4096 x 14336                  446 and 463      383 and 392
//   gradients and dX of 2048 x 14336 x 4096   1128 and 1047    1108 and 869  (both products one way)
//   wgrad 2048 x 4096 x 4096                  88.8 and 87.8    82.0 and 74.3
// So the gradients and WGRAD take eight and eight, and gelu does in pairs, whose stages are shorter.
template <bool LONG_RESULTS> struct Roles {
    static constexpr int EXPAND = LONG_RESULTS ? 8 : 16, OUT = LONG_RESULTS ? 8 : 4;
    static constexpr int WPG = EXPAND / GROUPS;     // expansion warps per group
    static constexpr int TPG = WPG * 32;            // threads per group
    static constexpr int CPT = 256 / TPG;           // chunks of 32 values each, per thread and stage
    static constexpr int W_OUT = EXPAND, W_B = W_OUT + OUT, W_MMA = W_B + 1, W_Q = W_B + 2;
    static constexpr int THREADS = (W_Q + 1) * 32;
    static constexpr int RANKS = W_B / 4, HELPERS = EXPAND / 4;  // warps of a quarter of the lanes; of them, expansion
    static_assert(EXPAND % 4 == 0 && OUT % 4 == 0 && TPG >= 64 && TPG <= 128, "warp roles");
};
template <int KIND, bool GRADS, bool GELU, bool PAIR> using RolesOf = Roles<KIND == 2 || GRADS || (GELU && PAIR)>;

constexpr int BK = 64;                        // reduction per stage
constexpr uint32_t A_BYTES = 128 * BK * 2;    // an expanded stage
constexpr int MAX_STAGES = 8;
constexpr int MIN_STAGES = 4;
constexpr int MAX_RAW = 16;                   // stages of codes
constexpr uint32_t SMEM_MAX = 227 * 1024;     // rings, control and alignment
constexpr long long kWaitCycles = 4000000000ll;

struct Smem {
    uint64_t full[MAX_STAGES];    // B landed (TMA bytes) and A expanded (one arrival per warp)
    uint64_t empty[MAX_STAGES];   // the stage's MMAs completed (commit)
    uint64_t rawf[MAX_RAW];       // codes landed (TMA bytes)
    uint64_t rawe[MAX_RAW];       // the group's warps read them (one arrival per warp)
    uint64_t accf[2];             // an accumulator is complete (commit)
    uint64_t acce[2];             // its columns were read (one arrival per warp)
    uint32_t tmem_base;
    int abort;
    uint32_t arrived[4];  // parts of the tile's lanes that came before
    alignas(16) float row_pow[4][256];  // of the current tile's tokens, a copy for each quarter
};
constexpr uint32_t CONTROL = 5 * 1024;
static_assert(sizeof(Smem) <= CONTROL, "control block");

// one stage of codes (128 x 64 values of 4 or 8 bits)
template <int KIND> struct Raw {
    static constexpr uint32_t BYTES = KIND == WGRAD ? 8192 : 4096;
};
static_assert(MIN_STAGES >= GROUPS, "every group has a stage");
static_assert(MIN_STAGES * (A_BYTES + 256 * 128 + Raw<FWD>::BYTES) <= SMEM_MAX - CONTROL - 1024 &&
                  MIN_STAGES * (A_BYTES + 192 * 128 + Raw<WGRAD>::BYTES) <= SMEM_MAX - CONTROL - 1024,
              "four stages of each ring");

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
    uint16_t *rest;           // FWD with dh: NULL, or [cols, rows]: rest_of dG, and of dU above it
    const float *row_pow;     // FWD, DGRAD: the power of two that each token's row was divided by
    float *part;              // partial sums [tile][part][column / 4][lane][4]; carry: of a CTA's tile, [CTA]
    uint32_t *cnt;            // arrival counters [tile][4], zero between calls
    int *status;
    int64_t rows;             // weight rows (FWD, DGRAD: of one source) or tokens (WGRAD)
    int64_t K;                // columns of the expanded matrix
    int64_t cols;             // tokens, or dY's columns (WGRAD)
    int units;                // Tw * Tn * S
    int Tw, S;                // lane tiles, parts of the reduction
    int KB, KB0;              // stages of the whole reduction, and of the first source
    int part_kb, part_more;   // stages of a part, and how many parts have one more
    int seg;                  // stages that one fp32 accumulator sums at most (KB: a whole unit's)
    int NT;                   // columns per tile, a multiple of 16
    int stages, raws;         // of the expanded operands and of the codes
    uint32_t stage_bytes;
    int gshift, asym, out_fp32;
    int joined;               // results come from `part`: S > 1, or
    int carry;                // S is 1, and a tile's several accumulators are added up there
};

// tensor maps: B (DGRAD: of one or two sources) and the codes of A (FWD: gate, up)
struct Maps {
    CUtensorMap b[2], q[2];
};

template <bool PAIR>
__device__ __forceinline__ void mma(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
    // descriptor high word: 1024 bytes between groups of eight rows, version 1, 128-byte swizzle
    constexpr uint32_t hi = 64u | (1u << 14) | (2u << 29);
    if (PAIR)
        asm volatile(
            "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.b32 p, %4, 0;\n mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
            " tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(d),
            "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(hi));
    else
        asm volatile(
            "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.b32 p, %4, 0;\n mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
            " tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(d),
            "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(hi));
}
// PAIR: arrives at the barrier of either CTA
template <bool PAIR> __device__ __forceinline__ void mma_commit(uint64_t *bar) {
    if (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_addr(bar)),
            "h"((uint16_t)3)
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                     : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// all threads of both CTAs
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Arrives at the first CTA's barrier of that place, and passes on what is ordered before the arrival in
// this CTA's shared memory (its expanded stage, which the first CTA's MMAs read). The release at
// cluster scope is a fence for that memory alone: one for all memory (release.cluster) waits for the
// GPU's and took 900 cycles a stage, 1.9 times the product's time; this one costs nothing.
__device__ __forceinline__ void arrive_first(uint64_t *bar) {
    asm volatile(
        "{\n .reg .b32 r;\n mapa.shared::cluster.u32 r, %0, 0;\n fence.release.sync_restrict::shared::cta.cluster;\n"
        " mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [r];\n}\n" ::"r"(smem_addr(bar))
        : "memory");
}
// A wait for what the other CTA does too: for its arrivals, or for the first CTA's MMAs (their commits).
// It acquires at cluster scope, again by a fence for shared memory alone (with acquire.cluster on the
// wait the gradients and dX of 2048 x 14336 x 4096 took 1066 us, with the fence 1038).
__device__ __forceinline__ bool try_wait_cluster(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n"
        " fence.acquire.sync_restrict::shared::cluster.cluster;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
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
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
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

// A weight is (q - z) s rounded once to fp16: q enters the mantissa of 1024.0 (1024 + q, exact), less
// 1024 + z is q - z (exact for |z| <= 1024), times the fp16 scale as it is. Zero points from 0 to
// 1023 have their two constants formed from bits. Any other (groups of one sign far from zero): beyond
// 1024, ((q - 8) s + c_lo) + c_hi with (8 - z) s = c_hi + c_lo, of which again only the last operation
// rounds at the weight's size.
__device__ __forceinline__ bool is_near(uint32_t sz) { return (sz >> 16) < 1024u; }
__device__ __forceinline__ uint2 near_words(uint32_t sz) {
    return make_uint2(__byte_perm(sz, 0, 0x1010), __byte_perm(sz + 0x64000000u, 0, 0x3232));
}
// Eight codes (nibble i is value i) as fp16 pairs (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ void expand8(uint32_t w, uint32_t s, uint32_t zc, uint32_t (&o)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = hmul(hsub(((w >> (4 * i)) & 0x000F000Fu) | 0x64006400u, zc), s);
}
__device__ __forceinline__ void expand8_any(uint32_t w, uint32_t sz, uint32_t (&o)[4]) {
    const int z = (int)(int16_t)(sz >> 16);
    const uint32_t s = __byte_perm(sz, 0, 0x1010);
    if (z <= 1024 && z >= -1024) {
        expand8(w, s, hpair((float)(1024 + z)), o);
        return;
    }
    const float k = (float)(8 - z) * __half2float(__ushort_as_half((unsigned short)(sz & 0xFFFFu)));
    const uint32_t ch = hpair(k), cl = hpair(k - __half2float(__ushort_as_half((unsigned short)(ch & 0xFFFFu))));
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[i] = hadd(hfma(hsub(((w >> (4 * i)) & 0x000F000Fu) | 0x64006400u, 0x64086408u), s, cl), ch);
}
// Four E4M3 bytes as bf16 pairs (0, 2), (1, 3), times 2^e: the value's seven exponent and mantissa
// bits under bf16's exponent read as the value times 2^-120 (subnormals too), so one multiplication
// by 2^(120 + e) restores it exactly; two where that power is past bf16's range. E4M3's one NaN, 0x7F of
// either sign, reads as 480 there: top, the largest of the magnitudes' bits so far, has 0x07F0 in one of
// its halves then.
__device__ __forceinline__ void expand4(uint32_t w, uint32_t f, uint32_t &o0, uint32_t &o1, uint32_t &top) {
    const uint32_t v0 = (w << 4) & 0x07F007F0u, v1 = (w >> 4) & 0x07F007F0u;
    o0 = bmul(v0 | ((w << 8) & 0x80008000u), f);
    o1 = bmul(v1 | (w & 0x80008000u), f);
    top = __vimax3_u16x2(top, v0, v1);
}
// the top bit of each byte that is E4M3's NaN
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }
// factors of scale byte b = e + 127 (255 is NaN): one up to b = 134, else 2^120 and 2^e
__device__ __forceinline__ uint32_t pow2_one(uint32_t b) { return ((120u + b) << 7) * 0x10001u; }
__device__ __forceinline__ uint32_t pow2_two(uint32_t b) {
    return (b == 255u ? 0x7FC0u : b == 0u ? 0x0040u : b << 7) * 0x10001u;  // 2^-127 is subnormal
}
__device__ __forceinline__ void expand4_any(uint32_t w, uint32_t b, uint32_t &o0, uint32_t &o1) {
    uint32_t top = 0;
    expand4(w, 0x7B807B80u, o0, o1, top);
    o0 = bmul(o0, pow2_two(b));
    o1 = bmul(o1, pow2_two(b));
    const uint32_t n = nan_bytes(w) >> 7;
    o0 |= (n & 0x00010001u) * 0x7FC0u;
    o1 |= ((n >> 8) & 0x00010001u) * 0x7FC0u;
}

// A wait by all lanes of a warp, with one result for all of them (a vote, so that what follows stays
// uniform). A phase that is over costs some 50 cycles this way; a poll by one lane with the rest
// reconverging behind it took over 110. Bounded by the SM's clock (4e9 cycles, about 2 s). PAIR: the phase
// is completed by the other CTA too.
template <bool PAIR>
static __device__ __noinline__ bool slow_wait(uint64_t *bar, uint32_t parity, int *abort, int *status) {
    const long long t0 = clock64();
    bool r;
    while (!(r = __all_sync(FULL, PAIR ? try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)))) {
        if (__any_sync(FULL, *(volatile int *)abort != 0)) break;
        if (__any_sync(FULL, clock64() - t0 > kWaitCycles)) {
            *(volatile int *)abort = 1;
            record_status(status, W4_ERR_TIMEOUT);
            break;
        }
    }
    return r;
}
template <bool PAIR = false>
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, Smem *sm, int *status) {
    if (__all_sync(FULL, PAIR ? try_wait_cluster(bar, parity) : mbar_try_wait_short(bar, parity))) return true;
    return slow_wait<PAIR>(bar, parity, &sm->abort, status);
}
// The same by the one thread that runs a producer's or the MMA issuer's loop.
template <bool PAIR>
static __device__ __noinline__ bool slow_wait1(uint64_t *bar, uint32_t parity, int *abort, int *status) {
    const long long t0 = clock64();
    while (!(PAIR ? try_wait_cluster(bar, parity) : mbar_try_wait_short(bar, parity))) {
        if (*(volatile int *)abort) return false;
        if (clock64() - t0 > kWaitCycles) {
            *(volatile int *)abort = 1;
            record_status(status, W4_ERR_TIMEOUT);
            return false;
        }
    }
    return true;
}
template <bool PAIR = false> __device__ __forceinline__ bool wait1(uint64_t *bar, uint32_t parity, Smem *sm, int *status) {
    return (PAIR ? try_wait_cluster(bar, parity) : mbar_try_wait_short(bar, parity)) ||
           slow_wait1<PAIR>(bar, parity, &sm->abort, status);
}
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}
// Both activations are g times a logistic function: silu of g itself, the tanh form of gelu of
// p(g) = 2 sqrt(2/pi) (g + 0.044715 g^3), since (1 + tanh(y)) / 2 = 1 / (1 + exp(-2 y)).
struct Act {
    float value, slope;
};
__device__ __forceinline__ Act act_of(float g, bool gelu) {
    const float h = fminf(fmaxf(g, -64.0f), 64.0f);              // exp is 0 or inf there; h^3 stays finite
    const float g2 = 0.07135481282f * h * h;                     // 2 sqrt(2/pi) 0.044715 g^2
    const float p = gelu ? h * (1.5957691216f + g2) : g;
    const float dp = gelu ? 1.5957691216f + 3.0f * g2 : 1.0f;     // p'
    const float s = __fdividef(1.0f, 1.0f + __expf(-p));
    Act r;
    r.value = g * s;
    r.slope = s + r.value * (1.0f - s) * dp;
    return r;
}

// A unit: its tile, its part of the reduction (stages [b0, b1)) and its place in the partial sums.
// 32 bits throughout: shape_ok's limits leave fewer than 2^28 units, and a 64-bit division costs hundreds of
// instructions (six of them at a kernel's start took 4 us).
struct Unit {
    uint32_t tile, tw, tn, s;
    int b0, b1;
};
// A pair's tile is two tiles of lanes, one for each CTA; a CTA's place is among the tiles of one.
template <bool PAIR> __device__ __forceinline__ uint32_t first_unit() { return PAIR ? blockIdx.x >> 1 : blockIdx.x; }
template <bool PAIR> __device__ __forceinline__ uint32_t unit_step() { return PAIR ? gridDim.x >> 1 : gridDim.x; }
template <bool PAIR> __device__ __forceinline__ Unit unit_of(const Args &a, uint32_t u) {
    Unit t;
    const uint32_t r = u / (uint32_t)a.Tw;
    t.tw = u - r * (uint32_t)a.Tw;
    if (a.S == 1) {
        t.s = 0;
        t.tn = r;
        t.b0 = 0;
        t.b1 = a.KB;
    } else {
        t.tn = r / (uint32_t)a.S;
        t.s = r - t.tn * (uint32_t)a.S;
        // parts of a.part_kb stages; the first a.part_more of them have one more
        t.b0 = (int)(t.s * (uint32_t)a.part_kb + (t.s < (uint32_t)a.part_more ? t.s : (uint32_t)a.part_more));
        t.b1 = t.b0 + a.part_kb + (t.s < (uint32_t)a.part_more ? 1 : 0);
    }
    t.tile = t.tn * (uint32_t)a.Tw + t.tw;
    if (PAIR) {
        t.tw = 2 * t.tw + cluster_rank();
        t.tile = 2 * t.tile + cluster_rank();
    }
    return t;
}

// The stages of this CTA's units, one after the other.
template <bool PAIR> struct Walk {
    uint32_t u;
    Unit un;
    int kb;
    __device__ __forceinline__ void start(const Args &a) {  // the grid has a unit for every CTA
        u = first_unit<PAIR>();
        un = unit_of<PAIR>(a, u);
        kb = un.b0;
    }
    __device__ __forceinline__ bool skip(const Args &a, int n) {  // false: there are no more
        kb += n;
        while (kb >= un.b1) {
            const int over = kb - un.b1;
            u += unit_step<PAIR>();
            if (u >= (uint32_t)a.units) return false;
            un = unit_of<PAIR>(a, u);
            kb = un.b0 + over;
        }
        return true;
    }
};

// The scales of the chunks that a thread expands in a stage. fetch() only issues loads, from
// addresses that always exist, and nothing waits for them before word(): no branch and no arithmetic
// on a loaded value may stand between the two, or each stage costs a memory latency.
template <int KIND, int TPG> struct Scales {
    static constexpr int CPT = 256 / TPG;
    uint16_t s[CPT], z[CPT];  // fp16 scales and zero points; WGRAD: scale bytes in s
    uint32_t there;           // bit j: chunk j exists
    const uint16_t *ps[2], *pz[2];  // FWD: of the tile's first row (for symmetric weights pz is ps)
    uint32_t tile = ~0u, rows;      // FWD: whose row it is, and which of the thread's rows exist

    template <bool PAIR> __device__ __forceinline__ void fetch(const Args &a, const Walk<PAIR> &w, int tt) {
        const int K = (int)a.K, n = (int)a.rows;  // at most 2^24
        there = 0u;
        if (KIND == WGRAD) {
            const int m = w.kb * BK + (tt >> 2), k = (int)w.un.tw * 128 + 32 * (tt & 3);
            const int64_t at = (int64_t)m * (K >> 5) + (k >> 5);
#pragma unroll
            for (int j = 0; j < CPT; ++j) {
                const bool ok = k < K && m + TPG / 4 * j < n;
                there |= ok ? 1u << j : 0u;
                s[j] = __ldg(a.xs + (ok ? at + (int64_t)(TPG / 4 * j) * (K >> 5) : 0));
            }
            return;
        }
        const int J = K >> a.gshift;
        if (KIND == FWD) {
            // raw rows TPG / 2 apart: those of the gate, then those of up
            if (w.un.tw != tile) {
                tile = w.un.tw;
                const int row = (int)tile * 64 + (tt >> 1);
                rows = 0u;
#pragma unroll
                for (int j = 0; j < CPT; ++j) rows |= row + (TPG / 2 * j & 63) < n ? 1u << j : 0u;
                const int64_t at = row < n ? (int64_t)row * J : 0;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    ps[j] = a.w[j].scales + at;
                    pz[j] = (a.asym ? reinterpret_cast<const uint16_t *>(a.w[j].zeros) : a.w[j].scales) + at;
                }
            }
            const int k = w.kb * BK + 32 * (tt & 1);
            there = k < K ? rows : 0u;
            const int i = k < K ? k >> a.gshift : 0;
#pragma unroll
            for (int j = 0; j < CPT; ++j) {
                const int d = TPG / 2 * j, x = (d & 63) && ((rows >> j) & 1u) ? i + (d & 63) * J : i;
                s[j] = __ldg(ps[d >> 6] + x);
                z[j] = __ldg(pz[d >> 6] + x);
            }
            return;
        }
        const int src = w.kb >= a.KB0 ? 1 : 0;
        const int row = (w.kb - (src ? a.KB0 : 0)) * BK + (tt >> 2), k = (int)w.un.tw * 128 + 32 * (tt & 3);
        const int64_t at = (int64_t)row * J + (k >> a.gshift);
        const Weight &m = a.w[src];
        // symmetric weights: the scale again, for the sake of one instruction stream
        const uint16_t *mz = a.asym ? reinterpret_cast<const uint16_t *>(m.zeros) : m.scales;
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            const bool ok = k < K && row + TPG / 4 * j < n;
            there |= ok ? 1u << j : 0u;
            const int64_t i = ok ? at + (int64_t)(TPG / 4 * j) * J : 0;
            s[j] = __ldg(m.scales + i);
            z[j] = __ldg(mz + i);
        }
    }
    // fp16 scale with the zero point above it, or the scale byte; a chunk that does not exist has
    // scale 0 (its codes read as zero)
    __device__ __forceinline__ uint32_t word(const Args &a, int j) const {
        const bool ok = (there >> j) & 1u;
        if (KIND == WGRAD) return ok ? (uint32_t)s[j] : 127u;
        return ok ? (uint32_t)s[j] | ((a.asym ? (uint32_t)z[j] : 8u) << 16) : 8u << 16;
    }
};

// Chunk c of a stage is 32 values of a row: FWD row c / 2 (64 of the gate, then 64 of up), half
// c % 2; else row c / 4, columns 32 (c % 4). In FWD the rows go to the lanes 16 of the gate, 16 of
// up, 16 of the gate, ..., so that a warp of the results has both of a feature. Its codes are at
// c * 16 (WGRAD: c * 32) of the stage's codes.
// A thread's place in that: chunks tt, tt + TPG, ...
template <int KIND, int TPG> struct Place {
    uint32_t codes;           // of the first chunk, from the start of the stage's codes
    uint32_t swap;            // DGRAD, WGRAD: which half of the codes comes first
    uint32_t out[4];          // of its four 16-byte pieces, from the start of the A tile
    __device__ __forceinline__ explicit Place(int tt) {
        const int r = tt >> 1;
        const int row = KIND == FWD ? 32 * (r >> 4) + (r & 15) : tt >> 2;
        // DGRAD, WGRAD: every other thread (by the parity of three bits of its number) takes its pieces in
        // the order 2, 3, 0, 1: the eight threads of a quarter warp then write eight different 16-byte
        // banks, and threads whose codes are 128 bytes apart read different banks
        const uint32_t flip = KIND != FWD && (((tt >> 1) ^ (tt >> 2) ^ (tt >> 3)) & 1) ? 32u : 0u;
        const uint32_t at = (KIND == FWD ? 0u : (uint32_t)((tt >> 1) & 1) * 8192u) + (uint32_t)row * 128u;
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = at + ((((uint32_t)(tt & 1) << 6) + 16u * i) ^ flip ^ ((uint32_t)(row & 7) << 4));
        codes = (uint32_t)tt * (KIND == WGRAD ? 32u : 16u);
        swap = flip ? (KIND == WGRAD ? 16u : 8u) : 0u;
    }
    // from the first chunk's row of the A tile to chunk j's, in bytes (FWD: the up rows are 16 lanes
    // behind their features' gate rows); whole groups of eight rows
    static __device__ __forceinline__ constexpr uint32_t next(int j) {
        return KIND == FWD ? (TPG / 2 * j & 63) * 2 * 128 + (TPG / 2 * j >> 6) * 16 * 128 : j * (TPG / 4) * 128;
    }
};

template <int KIND> struct Values {
    uint32_t q[KIND == WGRAD ? 8 : 4];
};
// the codes of chunk j of a thread, in the order in which it expands them
template <int KIND, int TPG>
__device__ __forceinline__ void chunk_load(Values<KIND> &c, uint32_t raw, const Place<KIND, TPG> &p, int j) {
    const uint32_t at = raw + p.codes + (uint32_t)(TPG * j) * (KIND == WGRAD ? 32u : 16u);
    if (KIND == FWD) {
        const uint4 v = lds128(at);
        c.q[0] = v.x; c.q[1] = v.y; c.q[2] = v.z; c.q[3] = v.w;
    } else if (KIND == DGRAD) {
        const uint2 v = lds64(at + p.swap), u = lds64(at + (p.swap ^ 8u));
        c.q[0] = v.x; c.q[1] = v.y; c.q[2] = u.x; c.q[3] = u.y;
    } else {
        const uint4 v = lds128(at + p.swap), u = lds128(at + (p.swap ^ 16u));
        c.q[0] = v.x; c.q[1] = v.y; c.q[2] = v.z; c.q[3] = v.w;
        c.q[KIND == WGRAD ? 4 : 0] = u.x; c.q[KIND == WGRAD ? 5 : 1] = u.y;
        c.q[KIND == WGRAD ? 6 : 2] = u.z; c.q[KIND == WGRAD ? 7 : 3] = u.w;
    }
}
// their values into the A tile; ANY: with any scale, zero point and NaN. top: see expand4
template <int KIND, int TPG, bool ANY>
__device__ __forceinline__ void chunk_store(const Values<KIND> &c, uint32_t base, const Place<KIND, TPG> &p, int j, uint32_t sz,
                                            uint32_t &top) {
    const uint2 k = KIND == WGRAD ? make_uint2(pow2_one(sz), 0u) : near_words(sz);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t o[4];
        if (KIND == WGRAD) {
            if (ANY) {
                expand4_any(c.q[KIND == WGRAD ? 2 * i : 0], sz, o[0], o[1]);
                expand4_any(c.q[KIND == WGRAD ? 2 * i + 1 : 0], sz, o[2], o[3]);
            } else {
                expand4(c.q[KIND == WGRAD ? 2 * i : 0], k.x, o[0], o[1], top);
                expand4(c.q[KIND == WGRAD ? 2 * i + 1 : 0], k.x, o[2], o[3], top);
            }
        } else if (ANY) {
            expand8_any(c.q[i], sz, o);
        } else {
            expand8(c.q[i], k.x, k.y, o);
        }
        sts128(base + p.out[i] + Place<KIND, TPG>::next(j), o[0], o[1], o[2], o[3]);
    }
}
template <int KIND, int TPG>
__device__ __forceinline__ void expand_store(uint32_t raw, uint32_t base, const Place<KIND, TPG> &p,
                                             const uint32_t (&sz)[256 / TPG]) {
    constexpr int CPT = 256 / TPG;
    // One branch for the whole warp: scales outside the usual range are rare, and their arithmetic
    // beside the other in one instruction stream cost a third of the expansion's rate.
    bool any = false;
#pragma unroll
    for (int j = 0; j < CPT; ++j) any = any || (KIND == WGRAD ? sz[j] > 134u : !is_near(sz[j]));
    any = __any_sync(FULL, any);
#pragma unroll
    for (int j = 0; j < CPT; j += 2) {
        Values<KIND> c[2];  // two chunks' loads in flight
        chunk_load<KIND, TPG>(c[0], raw, p, j);
        chunk_load<KIND, TPG>(c[1], raw, p, j + 1);
        bool again = any;
        uint32_t top = 0;
        if (!any) {
            chunk_store<KIND, TPG, false>(c[0], base, p, j, sz[j], top);
            chunk_store<KIND, TPG, false>(c[1], base, p, j + 1, sz[j + 1], top);
            // NaN among the values: rare, and found beside the rest in an instruction a word (fp32 wgrad
            // 2048 x 4096 x 4096 80.0 us without, 83.1 with, 85.0 by tests of the bytes)
            if (KIND == WGRAD) again = (top & 0xFFFFu) == 0x07F0u || (top >> 16) == 0x07F0u;
        }
        if (again) {
            chunk_store<KIND, TPG, true>(c[0], base, p, j, sz[j], top);
            chunk_store<KIND, TPG, true>(c[1], base, p, j + 1, sz[j + 1], top);
        }
    }
}
// The place of value i of eight (FWD, DGRAD) or of four (WGRAD) in what expand8 and expand4 write
__host__ __device__ __forceinline__ constexpr int value_at8(int place) { return (place >> 1) | ((place & 1) << 2); }
__host__ __device__ __forceinline__ constexpr int value_at4(int place) { return (place >> 1) | ((place & 1) << 1); }

// What rounding v to the bf16 value b left of it, as a byte: of the 16 bits below b's last place (RN's
// choice makes them signed) the upper eight, rounded. with_rest(b, byte) is v to 16 significant bits.
__device__ __forceinline__ uint32_t rest_of(float v, __nv_bfloat16 b) {
    const int r = (int)(__float_as_uint(v) - ((uint32_t)__bfloat16_as_ushort(b) << 16));
    return (uint32_t)min((r + 128) >> 8, 127) & 0xFFu;
}
// of a pair's word of bf16 values and its word of rests: value e (0 or 1), byte t of its rests
__device__ __forceinline__ float with_rest(uint32_t w, uint32_t rests, int e, int t) {
    const uint32_t r = (uint32_t)((int)(rests << (24 - 8 * (2 * e + t))) >> 16) & 0xFFFFFF00u;
    return __uint_as_float((e ? w & 0xFFFF0000u : w << 16) + r);
}

// dH at the tokens and the feature that this lane finishes of columns [c, c + 16), n of which exist
// (see emit). Only loads: nothing waits for them before emit() uses them.
struct Incoming {
    uint16_t v[8];
    __device__ __forceinline__ void fetch(const Args &a, const Unit &un, int q4, int lane, int c, int n) {
        const int up = lane >> 4;
        const int64_t h = (int64_t)un.tw * 64 + 16 * q4 + (lane & 15);
        const int m = h < a.rows ? n - up : 0;
        const uint16_t *p = reinterpret_cast<const uint16_t *>(a.dh) + ((int64_t)un.tn * a.NT + c + up) * a.rows + h;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 2 * i < m ? __ldg(p + 2 * i * a.rows) : (uint16_t)0;
    }
};

// Results of columns [c, c + 16) of a tile, of which n exist, for this thread's lane.
template <int KIND, bool GRADS, bool GELU>
__device__ __forceinline__ void emit(const Args &a, const float *row_pow, const Unit &un, int q4, int lane, int c, int n,
                                     const float (&v)[16], const Incoming &dh, bool add) {
    const int64_t col = (int64_t)un.tn * a.NT + c;
    float4 pw[KIND == WGRAD ? 1 : 4];
    if (KIND != WGRAD) {
#pragma unroll
        for (int i = 0; i < 4; ++i) pw[KIND == WGRAD ? 0 : i] = reinterpret_cast<const float4 *>(row_pow + c)[i];
    }
    if (KIND == FWD) {
        // lanes 0-15 of a warp hold gate rows, lanes 16-31 the same features' up rows: of each pair
        // of tokens the lower half takes the even one and the upper half the odd one
        const int up = lane >> 4;
        const int64_t h = (int64_t)un.tw * 64 + 16 * q4 + (lane & 15);
        const int64_t at = (col + up) * a.rows + h, step = 2 * a.rows;
        const int m = h < a.rows ? n - up : 0;  // this lane's tokens are those with 2 i < m
        const bool whole = __all_sync(FULL, m >= 15);  // no test a value where all are wanted
        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.out) + at, *o2 = a.out2 + at;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float got = __shfl_xor_sync(FULL, up ? v[2 * i] : v[2 * i + 1], 16);
            const float4 p4 = pw[KIND == WGRAD ? 0 : i >> 1];
            const float f = i & 1 ? (up ? p4.w : p4.z) : (up ? p4.y : p4.x);
            const float g = f * (up ? got : v[2 * i]), u = f * (up ? v[2 * i + 1] : got);
            const Act t = act_of(g, GELU);
            const float d = GRADS ? bf16_lo(dh.v[i]) : 0.0f;
            const float v1 = GRADS ? d * u * t.slope : t.value * u, v2 = d * t.value;
            const __nv_bfloat16 first = __float2bfloat16_rn(v1), second = __float2bfloat16_rn(v2);
            const auto store = [&] {
                o[i * step] = first;
                if (GRADS) o2[i * step] = second;
                if (GRADS && a.rest) a.rest[at + i * step] = (uint16_t)(rest_of(v1, first) | rest_of(v2, second) << 8);
            };
            if (whole)
                store();
            else if (2 * i < m)
                store();
        }
    } else {
        const int pl = KIND == DGRAD ? (lane & ~7) + value_at8(lane & 7) : (lane & ~3) + value_at4(lane & 3);
        const int64_t k = (int64_t)un.tw * 128 + 32 * q4 + pl;
        if (k >= a.K) return;
        const int64_t at = col * a.K + k;
        if (KIND == WGRAD && a.out_fp32) {
            float *o = static_cast<float *>(a.out) + at;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (i < n) o[i * a.K] = add ? o[i * a.K] + v[i] : v[i];
        } else {
            __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.out) + at;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float4 p4 = pw[KIND == WGRAD ? 0 : i >> 2];
                const float f = (i & 3) == 0 ? p4.x : (i & 3) == 1 ? p4.y : (i & 3) == 2 ? p4.z : p4.w;
                if (i < n) o[i * a.K] = __float2bfloat16_rn(KIND == DGRAD ? v[i] * f : v[i]);
            }
        }
    }
}

template <int KIND, bool GRADS, bool GELU, bool PAIR>
__global__ void __launch_bounds__((RolesOf<KIND, GRADS, GELU, PAIR>::THREADS), 1) expand_gemm_kernel(const __grid_constant__ Maps tm,
                                                                                       const __grid_constant__ Args a) {
    using R = RolesOf<KIND, GRADS, GELU, PAIR>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *raw = base + (size_t)a.stages * a.stage_bytes;
    Smem *sm = reinterpret_cast<Smem *>(raw + (size_t)a.raws * Raw<KIND>::BYTES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int NS = a.stages, NR = a.raws;

    // the expansion's first scales, on their way while the CTA sets up
    Walk<PAIR> w;
    bool more = false;
    Scales<KIND, R::TPG> next;
    if (warp < R::EXPAND) {
        w.start(a);
        more = w.skip(a, warp / R::WPG);
        if (more) next.fetch(a, w, threadIdx.x % R::TPG);
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&sm->full[s], 1 + R::WPG + (PAIR && cluster_rank() == 0 ? 1 : 0));
            mbar_init(&sm->empty[s], 1);
        }
        for (int s = 0; s < NR; ++s) {
            mbar_init(&sm->rawf[s], 1);
            mbar_init(&sm->rawe[s], R::WPG);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sm->accf[b], 1);
            mbar_init(&sm->acce[b], PAIR ? 2 * R::OUT : R::OUT);
        }
        sm->abort = 0;
        fence_mbar_init();
    }
    if (warp == R::W_MMA) {
        if (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sm->tmem_base)),
                         "r"(512u)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sm->tmem_base)),
                         "r"(512u)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();  // the other CTA's barriers are ready
    tc_fence_after();
    const uint32_t tmem = sm->tmem_base;

    if (warp < R::EXPAND) {
        // ------------------------------------------------ expansion of A
        const int grp = warp / R::WPG, tt = threadIdx.x % R::TPG;
        const Place<KIND, R::TPG> place(tt);
        int slot = grp, rs = grp;
        uint32_t phase = 0, rphase = 0;
        while (more) {
            uint32_t sz[R::CPT];
#pragma unroll
            for (int j = 0; j < R::CPT; ++j) sz[j] = next.word(a, j);
            more = w.skip(a, GROUPS);
            if (more) next.fetch(a, w, tt);
            if (!warp_wait(&sm->rawf[rs], rphase, sm, a.status)) break;
            if (!warp_wait<PAIR>(&sm->empty[slot], phase ^ 1u, sm, a.status)) break;
            expand_store<KIND, R::TPG>(smem_addr(raw + (size_t)rs * Raw<KIND>::BYTES), smem_addr(base + (size_t)slot * a.stage_bytes),
                               place, sz);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the MMA reads them
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sm->full[slot]);
                mbar_arrive(&sm->rawe[rs]);
            }
            slot += GROUPS;
            if (slot >= NS) { slot -= NS; phase ^= 1u; }
            rs += GROUPS;
            if (rs >= NR) { rs -= NR; rphase ^= 1u; }
        }
    } else if (warp == R::W_B) {
        // ------------------------------------------------ B by TMA
        if (KIND != WGRAD) asm volatile("griddepcontrol.wait;" ::: "memory");  // B is row_prep_kernel's
        if (elect_one()) {
            int slot = 0, issued = 0;
            uint32_t phase = 0;
            bool ok = true;
            const uint32_t bytes = a.stage_bytes - A_BYTES;
            for (uint32_t u = first_unit<PAIR>(); u < (uint32_t)a.units && ok; u += unit_step<PAIR>()) {
                const Unit un = unit_of<PAIR>(a, u);
                const int c0 = (int)(un.tn * a.NT) + (PAIR ? (int)cluster_rank() * (a.NT >> 1) : 0);  // a half each
                for (int kb = un.b0; kb < un.b1; ++kb) {
                    if (!wait1<PAIR>(&sm->empty[slot], phase ^ 1u, sm, a.status)) { ok = false; break; }
                    uint8_t *dst = base + (size_t)slot * a.stage_bytes + A_BYTES;
                    mbar_arrive_expect_tx(&sm->full[slot], bytes);
                    if (KIND == WGRAD) {
                        for (uint32_t o = 0; o < bytes; o += 8192u)  // 64 columns of dY a box
                            tma_load_2d(dst + o, &tm.b[0], c0 + (int)(o >> 7), kb * BK, &sm->full[slot]);
                    } else if (KIND == DGRAD && kb >= a.KB0) {
                        tma_load_2d(dst, &tm.b[1], (kb - a.KB0) * BK, c0, &sm->full[slot]);
                    } else {
                        tma_load_2d(dst, &tm.b[0], kb * BK, c0, &sm->full[slot]);
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
    } else if (warp == R::W_Q) {
        // ------------------------------------------------ codes by TMA
        if (elect_one()) {
            int rs = 0, issued = 0;
            uint32_t rphase = 0;
            bool ok = true;
            for (uint32_t u = first_unit<PAIR>(); u < (uint32_t)a.units && ok; u += unit_step<PAIR>()) {
                const Unit un = unit_of<PAIR>(a, u);
                const int tw = (int)un.tw;
                for (int kb = un.b0; kb < un.b1; ++kb) {
                    if (!wait1(&sm->rawe[rs], rphase ^ 1u, sm, a.status)) { ok = false; break; }
                    uint8_t *dst = raw + (size_t)rs * Raw<KIND>::BYTES;
                    mbar_arrive_expect_tx(&sm->rawf[rs], Raw<KIND>::BYTES);
                    if (KIND == FWD) {
                        tma_load_2d(dst, &tm.q[0], kb * (BK / 2), tw * 64, &sm->rawf[rs]);
                        tma_load_2d(dst + 2048, &tm.q[1], kb * (BK / 2), tw * 64, &sm->rawf[rs]);
                    } else if (KIND == DGRAD && kb >= a.KB0) {
                        tma_load_2d(dst, &tm.q[1], tw * 64, (kb - a.KB0) * BK, &sm->rawf[rs]);
                    } else {
                        tma_load_2d(dst, &tm.q[0], tw * (KIND == DGRAD ? 64 : 128), kb * BK, &sm->rawf[rs]);
                    }
                    ++issued;
                    if (++rs == NR) { rs = 0; rphase ^= 1u; }
                }
            }
            // no copy may land after the CTA exits
            for (int i = issued > NR ? issued - NR : 0; i < issued; ++i)
                (void)mbar_wait_bounded(&sm->rawf[i % NR], (uint32_t)(i / NR) & 1u, a.status);
        }
        __syncwarp();
    } else if (warp == R::W_MMA) {
        // ------------------------------------------------ MMA issue
        // D fp32, A and B fp16 (0) or bf16 (1), M = 128 (a pair: 256), N = NT; A (and B in WGRAD)
        // contiguous along M (N)
        const uint32_t idesc = (1u << 4) | (KIND == WGRAD ? (1u << 7) | (1u << 10) : 0u) | (KIND != FWD ? 1u << 15 : 0u) |
                               (KIND == WGRAD ? 1u << 16 : 0u) | ((uint32_t)(a.NT >> 3) << 17) | ((PAIR ? 16u : 8u) << 24);
        // low word: address / 16 | leading offset / 16 (K-major: unused; MN-major: 8192 bytes
        // between the 64-element atoms); a K step of 16 is 32 bytes, or 16 rows of 128
        constexpr uint32_t alead = KIND == FWD ? 1u << 16 : 512u << 16, astep = KIND == FWD ? 2u : 128u;
        constexpr uint32_t blead = KIND == WGRAD ? 512u << 16 : 1u << 16, bstep = KIND == WGRAD ? 128u : 2u;
        const uint32_t sbase = smem_addr(base);
        if (PAIR && cluster_rank() != 0) {
            // The second CTA of a pair: the first one's MMAs read its stages too, so it passes on that a
            // stage is full.
            if (elect_one()) {
                int slot = 0, done = 0;
                uint32_t phase = 0;
                bool ok = true;
                for (uint32_t u = first_unit<PAIR>(); u < (uint32_t)a.units && ok; u += unit_step<PAIR>()) {
                    const Unit un = unit_of<PAIR>(a, u);
                    for (int kb = un.b0; kb < un.b1; ++kb) {
                        if (!wait1(&sm->full[slot], phase, sm, a.status)) { ok = false; break; }
                        arrive_first(&sm->full[slot]);
                        ++done;
                        if (++slot == NS) { slot = 0; phase ^= 1u; }
                    }
                }
                // no commit may arrive after the CTA exits
                for (int i = done > NS ? done - NS : 0; i < done; ++i)
                    (void)mbar_wait_bounded(&sm->empty[i % NS], (uint32_t)(i / NS) & 1u, a.status);
            }
        } else if (elect_one()) {
            int slot = 0, done = 0, n = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (uint32_t u = first_unit<PAIR>(); u < (uint32_t)a.units && ok; u += unit_step<PAIR>()) {
                const Unit un = unit_of<PAIR>(a, u);
                for (int s0 = un.b0; s0 < un.b1 && ok; s0 += a.seg, ++n) {
                    const int s1 = un.b1 - s0 < a.seg ? un.b1 : s0 + a.seg;
                    const int buf = n & 1;
                    if (!wait1<PAIR>(&sm->acce[buf], ((uint32_t)(n >> 1) & 1u) ^ 1u, sm, a.status)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t d = tmem + (uint32_t)(buf * 256);
                    for (int kb = s0; kb < s1; ++kb) {
                        if (!wait1<PAIR>(&sm->full[slot], phase, sm, a.status)) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t sa = sbase + (uint32_t)slot * a.stage_bytes;
                        const uint32_t alo = (sa >> 4) | alead, blo = ((sa + A_BYTES) >> 4) | blead;
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk)
                            mma<PAIR>(d, alo + kk * astep, blo + kk * bstep, idesc, kb > s0 || kk > 0 ? 1u : 0u);
                        mma_commit<PAIR>(&sm->empty[slot]);
                        if (kb + 1 == s1) mma_commit<PAIR>(&sm->accf[buf]);
                        ++done;
                        if (++slot == NS) { slot = 0; phase ^= 1u; }
                    }
                }
            }
            // no commit may arrive after the CTA exits
            for (int i = done > NS ? done - NS : 0; i < done; ++i)
                (void)mbar_wait_bounded(&sm->empty[i % NS], (uint32_t)(i / NS) & 1u, a.status);
        }
        __syncwarp();
    }

    if (warp < R::W_B) {
        // ------------------------------------------------ results (lane 32 q4 + lane of the tile), 16
        // columns at a time, in turn by the warps of a quarter: the result warps; and, in the CTA's
        // last tile, which has nothing behind it to overlap with, the expansion warps too, whose work is
        // done. Where a unit is summed up in several accumulators, they do not.
        constexpr int RANKS = R::RANKS, HELPERS = R::HELPERS;
        const int q4 = warp & 3, r = q4 * 32 + lane, rank = warp >> 2;
        const uint32_t tl = tmem + ((uint32_t)(q4 * 32) << 16);
        const bool helper = warp < R::EXPAND, shared = a.seg >= a.KB;
        const uint32_t u0 = first_unit<PAIR>(), step = unit_step<PAIR>();
        const uint32_t before = ((uint32_t)a.units - 1u - u0) / step;  // this CTA's units but the last
        float *row_pow = sm->row_pow[q4];
        if (KIND != WGRAD) asm volatile("griddepcontrol.wait;" ::: "memory");  // row_pow too
        uint32_t u = helper ? u0 + before * step : u0;
        if (helper && !shared) u = (uint32_t)a.units;
        int n = helper ? (int)before : 0;
        bool ok = true;
        // A wait that ran out ends this warp's work, but not its way through the tiles: the warps of a
        // quarter meet at barriers that have no time limit of their own.
        for (; u < (uint32_t)a.units; u += step) {
            const bool last = shared && (uint32_t)a.units - u <= step;
            const Unit un = unit_of<PAIR>(a, u);
            const int64_t left = a.cols - (int64_t)un.tn * a.NT;
            const int ncols = left < a.NT ? (int)left : a.NT;
            const int c0 = 16 * (last ? rank : rank - HELPERS), cstep = 16 * (last ? RANKS : RANKS - HELPERS);
            // the warps of this quarter that take part meet at a barrier of their own
            auto meet = [&] { named_bar_sync(last ? 1 + q4 : 5 + q4, 32 * (last ? RANKS : RANKS - HELPERS)); };
            // partial sums: [column / 4][lane][4 columns]
            const uint32_t place = a.carry ? blockIdx.x : un.tile;
            float4 *part = reinterpret_cast<float4 *>(a.part) + ((size_t)place * a.S + un.s) * (a.NT * 32) + r;
            // Also what keeps the helpers from the last tile's accumulator until the result warps have
            // finished the tile before it: a helper sees only the parity of that accumulator's phase, which
            // two tiles back had the same.
            if (KIND != WGRAD || last) meet();  // and the readers of the previous tile's powers
            if (KIND != WGRAD) {
                if (rank == HELPERS)
                    for (int c = lane; c < ncols; c += 32) row_pow[c] = a.row_pow[(int64_t)un.tn * a.NT + c];
                meet();
            }
            Incoming ahead;  // dH of the next columns, on its way while the present ones are finished
            if (GRADS) ahead.fetch(a, un, q4, lane, c0, ncols - c0);
            for (int s0 = un.b0; s0 < un.b1 && ok; s0 += a.seg, ++n) {
                const int buf = n & 1;
                if (!warp_wait<PAIR>(&sm->accf[buf], (uint32_t)(n >> 1) & 1u, sm, a.status)) { ok = false; break; }
                tc_fence_after();
#pragma unroll 1
                for (int c = c0; c < ncols; c += cstep) {
                    uint32_t raw16[16];
                    tmem_ld16(tl + (uint32_t)(buf * 256 + c), raw16);
                    tmem_wait_ld(raw16);
                    float v[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(raw16[i]);
                    if (a.joined) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float4 f = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                            float4 *p = part + (c / 4 + i) * 128;
                            if (s0 > un.b0) {
                                const float4 o = *p;
                                f = make_float4(f.x + o.x, f.y + o.y, f.z + o.z, f.w + o.w);
                            }
                            *p = f;
                        }
                    } else {
                        const Incoming now = ahead;
                        if (GRADS) ahead.fetch(a, un, q4, lane, c + cstep, ncols - c - cstep);
                        emit<KIND, GRADS, GELU>(a, row_pow, un, q4, lane, c, ncols - c, v, now, s0 > un.b0);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && !helper) {
                    if (PAIR)
                        arrive_first(&sm->acce[buf]);
                    else
                        mbar_arrive(&sm->acce[buf]);
                }
            }
            if (!a.joined) continue;
            // the last part of a tile's 32 lanes to arrive adds all parts in order
            uint32_t *cnt = a.cnt + (size_t)place * 4 + q4;
            __threadfence();
            meet();
            if (rank == HELPERS && lane == 0) sm->arrived[q4] = atomicAdd(cnt, 1u);
            meet();
            if (sm->arrived[q4] != (uint32_t)(a.S - 1) || !ok) continue;
            __threadfence();
            const float4 *p0 = reinterpret_cast<const float4 *>(a.part) + (size_t)place * a.S * (a.NT * 32) + r;
#pragma unroll 1
            for (int c = c0; c < ncols; c += cstep) {
                float v[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = 0.0f;
#pragma unroll 1
                for (int s = 0; s < a.S; s += 2) {  // two parts' loads in flight
                    const float4 *p = p0 + (size_t)s * (a.NT * 32) + c / 4 * 128;
                    const bool two = s + 1 < a.S;
                    const float4 *p2 = two ? p + a.NT * 32 : p;
                    float4 x[4], y[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = __ldcg(p + i * 128);
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = __ldcg(p2 + i * 128);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[4 * i] += x[i].x;
                        v[4 * i + 1] += x[i].y;
                        v[4 * i + 2] += x[i].z;
                        v[4 * i + 3] += x[i].w;
                        if (two) {
                            v[4 * i] += y[i].x;
                            v[4 * i + 1] += y[i].y;
                            v[4 * i + 2] += y[i].z;
                            v[4 * i + 3] += y[i].w;
                        }
                    }
                }
                const Incoming now = ahead;
                if (GRADS) ahead.fetch(a, un, q4, lane, c + cstep, ncols - c - cstep);
                emit<KIND, GRADS, GELU>(a, row_pow, un, q4, lane, c, ncols - c, v, now, false);
            }
            if (rank == HELPERS && lane == 0) *cnt = 0u;  // ready for the next call
        }
    }

    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();  // neither CTA leaves while the other may arrive at its barriers or read its stages
    tc_fence_after();
    if (warp == R::W_MMA) {
        if (PAIR)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    }
}

// ------------------------------------------------------------------ activations as fp16 rows

// The fp16 copy of bf16 rows that the products above multiply: row m divided by the power of two
// that brings its largest finite value into [2^14, 2^15). A bf16 value within 2^-31 of the
// largest is exact in it; what is smaller is off by 2^-39 of the largest at most. One or two
// tensors of the same rows (the two gradients, which one accumulator sums) share a power. The
// gradients come with the rests of their rounding, so that dX is formed from them to fp16's 11 bits and
// not bf16's 8 (its error against 64 bits is 0.0017 of it, its own rounding, and was 0.0024). The 8-bit
// checkpoint is restored on the way. One block per row, which it reads twice (the second time from
// L1 or L2); bound by the memory traffic of reading 2 (1) and writing 2 bytes a value.
struct Prep {
    const __nv_bfloat16 *x[2];    // [M, K]: the rows, or dG and dU
    const uint16_t *rest;         // the gradients' [M, K]: byte t of each is x[t]'s rest
    const uint8_t *x8, *xs;       // checkpoint values [M, K] and scale bytes [M, K/32]
    __half *y[2];                 // [M, K] each
    float *row_pow;               // [M]
    int64_t M, K;
    int pairs;                    // ROWS: each eight columns in expand8's order (the reduction of FWD)
};

// a non-finite value takes no part in the maximum
__device__ __forceinline__ float finite_abs(float v) {
    const float f = fabsf(v);
    return f <= 3.4e38f ? f : 0.0f;
}

enum Source { ROWS = 0, CHECKPOINT = 1, GRADIENTS = 2 };

// Eight columns of a row: of x[0], of the checkpoint, or of both gradients (v[1]; `rests` those of their
// rounding, or zeros).
template <int SRC>
__device__ __forceinline__ void prep_read(const Prep &p, int64_t m, int64_t i, const uint4 &rests,
                                          float (&v)[SRC == GRADIENTS ? 2 : 1][8]) {
    if (SRC == CHECKPOINT) {
        const uint2 w = __ldg(reinterpret_cast<const uint2 *>(p.x8 + m * p.K) + i);
        const uint32_t b = __ldg(p.xs + m * (p.K >> 5) + (i >> 2));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t o[2];
            expand4_any(j ? w.y : w.x, b, o[0], o[1]);
            v[0][4 * j] = bf16_lo(o[0]);
            v[0][4 * j + 2] = bf16_hi(o[0]);
            v[0][4 * j + 1] = bf16_lo(o[1]);
            v[0][4 * j + 3] = bf16_hi(o[1]);
        }
    } else {
        const uint32_t l[4] = {rests.x, rests.y, rests.z, rests.w};
#pragma unroll
        for (int t = 0; t < (SRC == GRADIENTS ? 2 : 1); ++t) {
            const uint4 w = __ldcg(reinterpret_cast<const uint4 *>(p.x[t] + m * p.K) + i);
            const uint32_t o[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[t][2 * j] = with_rest(o[j], l[j], 0, t);
                v[t][2 * j + 1] = with_rest(o[j], l[j], 1, t);
            }
        }
    }
}

template <int SRC> __global__ void __launch_bounds__(256) row_prep_kernel(const Prep p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");  // for the product before, where this one is launched behind it
    __shared__ float top[8];
    constexpr int TENSORS = SRC == GRADIENTS ? 2 : 1;
    const int64_t chunks = p.K >> 3;
    const uint4 none = make_uint4(0, 0, 0, 0);
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
        float mx = 0.0f;
        for (int64_t i = threadIdx.x; i < chunks; i += 256) {
            float v[TENSORS][8];
            prep_read<SRC>(p, m, i, none, v);
#pragma unroll
            for (int j = 0; j < 8 * TENSORS; ++j) mx = fmaxf(mx, finite_abs(v[j >> 3][j & 7]));
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
        for (int64_t i = threadIdx.x; i < chunks; i += 256) {
            float v[TENSORS][8];
            prep_read<SRC>(p, m, i, SRC == GRADIENTS ? __ldcg(reinterpret_cast<const uint4 *>(p.rest + m * p.K) + i) : none, v);
#pragma unroll
            for (int t = 0; t < TENSORS; ++t) {
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool pairs = SRC == CHECKPOINT || (SRC == ROWS && p.pairs);
                    const float lo = pairs ? v[t][j] : v[t][2 * j], hi = pairs ? v[t][j + 4] : v[t][2 * j + 1];
                    const __half2 h = __floats2half2_rn(lo * f, hi * f);
                    o[j] = *reinterpret_cast<const uint32_t *>(&h);
                }
                reinterpret_cast<uint4 *>(p.y[t] + m * p.K)[i] = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
    }
}

// The workspace starts with the arrival counters, in a region of one size for all shapes (what
// one call leaves as partial sums or rows is never another's counter), then holds the partial sums.
constexpr int64_t MAX_SPLIT_TILES = 4096;
constexpr size_t CNT_BYTES = MAX_SPLIT_TILES * 4 * sizeof(uint32_t);

// Place of the fp16 copy (of `values` in all) and of its powers (M of them) behind the counters and
// the partial sums, of `sums` bytes together, or 0 where the call has neither.
struct PrepPlace {
    size_t y, row_pow, end;
};
inline PrepPlace place_prep(size_t sums, int64_t values, int64_t M) {
    PrepPlace q;
    q.y = ((sums > CNT_BYTES ? sums : CNT_BYTES) + 255) / 256 * 256;
    q.row_pow = (q.y + (size_t)values * 2 + 255) / 256 * 256;
    q.end = (q.row_pow + (size_t)M * sizeof(float) + 255) / 256 * 256;
    return q;
}

// ------------------------------------------------------------------ host side

// Limits of M tokens, N rows and K columns of a weight: each dimension fits the kernels' 32-bit
// arithmetic, and any two of them (an operand's or a result's size) their count of tiles.
inline bool shape_ok(int64_t M, int64_t N, int64_t K) {
    constexpr int64_t most = (int64_t)1 << 24, area = (int64_t)1 << 40;
    return M >= 1 && M <= most && N >= 1 && N <= most && K >= 32 && K <= most && K % 32 == 0 && M * N <= area &&
           M * K <= area && N * K <= area;
}

struct Plan {
    int64_t Tw, Tn, units;          // pair: Tw counts pairs of tiles
    bool pair;                      // two CTAs share a tile of columns
    int NT, box, S, KB, KB0, seg, stages, raws;  // box: columns of B that a CTA holds
    bool carry;                     // see Args
    uint32_t stage_bytes;
    size_t bytes;                   // of the workspace, 0 where there are no partial sums
};

// lanes: weight rows per projection (FWD) or columns K; cols: the other side; red: length of the
// reduction (per source), sources 1 or 2; grads: FWD with the gradients; fp32: WGRAD with results in
// 32 bits.
//
// The tensor cores truncate: each product, towards zero, to a quarter of the last place of the sum that
// it joins (2^-25 of the sum's power of two), and the sum after each step. So R terms in one
// accumulator lose up to R * 1.25 * 2^-25 of its largest partial sum, half of that where it grows
// steadily (2^20 terms of one sign: up to 2e-2, measured 5.5e-3). An accumulator therefore sums 2^15
// terms at most (6e-4, a sixth of bf16's rounding, measured 1e-4), and for fp32 results 2048 (random
// signs against a 64-bit product: 3e-7 over 1000 rows, 6e-7 from 2048 to 8192). Longer units are added
// up outside, in fp32: in the partial sums of a split reduction, in fp32 results themselves, else in one
// tile's worth of sums for each CTA.
inline Plan make_plan(int kind, int64_t lanes, int64_t cols, int64_t red, int sources, int sms, bool grads = false,
                      bool fp32 = false) {
    const int most = (fp32 ? 2048 : 1 << 15) / BK;
    const int64_t Tw = kind == FWD ? (lanes + 63) / 64 : (lanes + 127) / 128;
    Plan best = {};
    double least = 0;
    for (int pair = 0; pair < 2; ++pair) {
        if (pair && (Tw < 2 || cols <= 128 || sms < 2)) continue;
        Plan p;
        p.pair = pair != 0;
        p.Tw = pair ? (Tw + 1) / 2 : Tw;
        // a CTA of WGRAD holds 192 columns at most, so that four stages of operands and four of codes fit
        const int64_t widest = kind == WGRAD && !pair ? 192 : 256, unit = pair ? 32 : 16;
        p.Tn = (cols + widest - 1) / widest;
        p.NT = (int)(((cols + p.Tn - 1) / p.Tn + unit - 1) / unit * unit);
        p.KB0 = (int)((red + BK - 1) / BK);
        p.KB = p.KB0 * sources;
        p.box = pair ? p.NT / 2 : p.NT;
        const uint32_t bb = kind == WGRAD ? (uint32_t)((p.box + 63) / 64) * 8192u : (uint32_t)p.box * 128u;
        p.stage_bytes = A_BYTES + bb;
        // A wait tells only neighbouring laps of a ring apart, so each slot's previous lap must be known
        // to be over when a warp waits for the next one. The codes' ring has a multiple of GROUPS
        // slots: a slot then belongs to one group, which sees its laps in order. The
        // operands' ring has GROUPS slots at least: a group that filled stage i - GROUPS waited for
        // the MMAs of the lap before it, which complete in order.
        const uint32_t rb = kind == WGRAD ? Raw<WGRAD>::BYTES : Raw<FWD>::BYTES, room = SMEM_MAX - CONTROL - 1024;
        p.stages = MIN_STAGES;
        p.raws = GROUPS;
        const auto grow = [&](int stages, int raws) {  // as far as both fit
            while (p.raws + GROUPS <= raws && p.stages * p.stage_bytes + (p.raws + GROUPS) * rb <= room) p.raws += GROUPS;
            while (p.stages < stages && (p.stages + 1) * p.stage_bytes + p.raws * rb <= room) ++p.stages;
        };
        // Codes come from HBM or a far L2 slice, and a group has one slot in four. Y's, in rows of 32 bytes,
        // take longest (us with 16 slots and 4 stages, and with 12 and 5: 1024 x 14336 x 4096 230 and 240;
        // the gradients of 2048 x 14336 x 4096 with their dX, whose expansion is slower, 980 and 956).
        if (kind == FWD && !grads) grow(MIN_STAGES, MAX_RAW);
        grow(MIN_STAGES + 1, GROUPS);
        grow(MIN_STAGES + 1, 2 * GROUPS);
        grow(MAX_STAGES, MAX_RAW);
        // One CTA or two (more than 128 columns: 77 x 5632 x 2048 takes 16.6 us in pairs, 16.0 without), and
        // parts of the reduction: what has the least estimated time, in cycles. One estimate serves all
        // products. A stage takes the shared memory's traffic (the codes, A and the scales, and two passes
        // of B, which a pair divides) or its MMAs: 916 at 256 columns, measured 984 (FWD) and 903 (DGRAD);
        // in a pair 673, measured 797, 727 and 760 (WGRAD). A unit takes 7000 to start and end, 8500 in a
        // pair; the last part of a tile reads two partial sums of 16 columns in 1300 cycles, five groups of
        // columns at a time, after 1500 for the count.
        const int64_t tiles = p.Tw * p.Tn, workers = pair ? sms / 2 : sms;
        const double mem = 430 + 1.9 * p.box, mma = 2.1 * p.NT, stage = mem > mma ? mem : mma;
        for (int S = 1; S <= 32 && (S == 1 || S * 4 <= p.KB); ++S) {
            if (S > 1 && (tiles * S > 8 * workers || tiles * (pair + 1) > MAX_SPLIT_TILES)) break;
            const int64_t waves = (tiles * S + workers - 1) / workers;
            const double join = S > 1 ? 1500.0 + 1300.0 * ((p.NT + 79) / 80) * ((S + 1) / 2) : 0.0;
            const double t = (double)waves * ((double)((p.KB + S - 1) / S) * stage + (pair ? 8500 : 7000)) + join;
            if (least == 0 || t < least) {
                least = t;
                p.S = S;
                p.units = tiles * S;
                p.seg = (p.KB + S - 1) / S > most ? most : p.KB;
                p.carry = S == 1 && p.seg < p.KB && !fp32;
                const int64_t ctas = (p.units < workers ? p.units : workers) * (pair + 1);
                p.bytes = S > 1 || p.carry ? CNT_BYTES + (size_t)(p.carry ? ctas : p.units * (pair + 1)) * p.NT * 512 : 0;
                best = p;
            }
        }
    }
    return best;
}

// A plan as the schedule queries report it (w4.h).
inline void describe(const Plan &p, int sms, int64_t *out) {
    const int pair = p.pair ? 2 : 1;
    const int64_t workers = sms / pair;
    out[0] = pair;
    out[1] = p.units;
    out[2] = p.S;
    out[3] = p.NT;
    out[4] = p.KB;
    out[5] = p.seg;
    out[6] = (p.units < workers ? p.units : workers) * pair;
    out[7] = (int64_t)p.bytes;
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

// 8-bit [rows, width], plain boxes; what lies outside reads as zero
inline bool make_raw_map(CUtensorMap *tm, const void *p, int64_t rows, int64_t width, int box_width, int box_rows) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)width};
    const cuuint32_t box[2] = {(cuuint32_t)box_width, (cuuint32_t)box_rows}, es[2] = {1, 1};
    return enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(p), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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

// Allows a kernel its dynamic shared memory, once per device (`done` has a bit for each).
template <typename F> bool allow_smem(F *kernel, int bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = dev >= 0 && dev < 64 ? (uint64_t)1 << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

// Launch by programmatic dependent launch where `behind` is 1: the kernel starts, up to its
// griddepcontrol.wait, once every CTA of the one before it on the stream has issued launch_dependents
// (the preparation kernels do at once) or has exited (the products' CTAs).
template <typename... P, typename... A>
w4_status launch_behind(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem, cudaStream_t stream, int behind,
                        int cluster, A &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = behind;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kernel, P(args)...) != cudaSuccess) return W4_ERR_CUDA;
    return launch_status();
}

// Rows or a checkpoint: whatever came before on the stream is complete when this kernel starts, and with
// that the weights that the product behind it reads before it has waited for this kernel. Gradients come
// from this call's own product, so their kernel is launched behind it: its blocks start when the
// product's last CTA exits, which hides the launch and nothing else.
inline w4_status launch_prep(const Prep &p, cudaStream_t stream) {
    const unsigned grid = (unsigned)(p.M < (1 << 20) ? p.M : (1 << 20));
    if (p.rest) return launch_behind(row_prep_kernel<GRADIENTS>, grid, 256, 0, stream, 1, 1, p);
    if (p.x8)
        row_prep_kernel<CHECKPOINT><<<grid, 256, 0, stream>>>(p);
    else
        row_prep_kernel<ROWS><<<grid, 256, 0, stream>>>(p);
    return launch_status();
}

template <int KIND, bool GRADS, bool GELU>
w4_status launch(const Plan &p, Maps &tm, Args a, void *workspace, int sms, cudaStream_t stream) {
    bool maps = true;
    if (KIND == WGRAD) {
        maps = make_raw_map(&tm.q[0], a.x8, a.rows, a.K, 128, BK);
        tm.q[1] = tm.q[0];
    } else {
        for (int i = 0; i < 2; ++i)
            maps = maps && make_raw_map(&tm.q[i], a.w[i].codes, a.rows, a.K / 2, KIND == FWD ? BK / 2 : 64, BK);
    }
    if (!maps) return W4_ERR_CUDA;
    a.units = (int)p.units;
    a.part_kb = p.KB / p.S;
    a.part_more = p.KB % p.S;
    a.Tw = (int)p.Tw;
    a.S = p.S;
    a.KB = p.KB;
    a.KB0 = p.KB0;
    a.seg = p.seg;
    a.carry = p.carry ? 1 : 0;
    a.joined = p.S > 1 || p.carry ? 1 : 0;
    a.NT = p.NT;
    a.asym = a.w[0].zeros != nullptr ? 1 : 0;
    a.stages = p.stages;
    a.raws = p.raws;
    a.stage_bytes = p.stage_bytes;
    a.cnt = static_cast<uint32_t *>(workspace);
    a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + CNT_BYTES);
    a.status = device_status_ptr();
    if (!a.status) return W4_ERR_CUDA;
    const int smem = (int)(p.stages * p.stage_bytes + p.raws * Raw<KIND>::BYTES + CONTROL) + 1024;
    static std::atomic<uint64_t> attr_done{0}, pair_done{0};
    const int cluster = p.pair ? 2 : 1;
    const int64_t most = sms / cluster;
    const unsigned grid = (unsigned)((p.units < most ? p.units : most) * cluster);
    // FWD and DGRAD follow row_prep_kernel: they may start, and read weights, while it finishes.
    // Whatever came before on the stream was complete when it began.
    const int behind = KIND != WGRAD;
    if (p.pair) {
        if (!allow_smem(expand_gemm_kernel<KIND, GRADS, GELU, true>, (int)SMEM_MAX, pair_done)) return W4_ERR_CUDA;
        return launch_behind(expand_gemm_kernel<KIND, GRADS, GELU, true>, grid, RolesOf<KIND, GRADS, GELU, true>::THREADS, (size_t)smem, stream, behind, 2, tm, a);
    }
    if (!allow_smem(expand_gemm_kernel<KIND, GRADS, GELU, false>, (int)SMEM_MAX, attr_done)) return W4_ERR_CUDA;
    return launch_behind(expand_gemm_kernel<KIND, GRADS, GELU, false>, grid, RolesOf<KIND, GRADS, GELU, false>::THREADS, (size_t)smem, stream, behind, 1, tm, a);
}

}  // namespace xg
}  // namespace w4
