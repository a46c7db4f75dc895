// opq_fp8_linear.cuh — y = act(x W^T + bias) for x [M, K] and W [N, K] in the 8-bit block format:
//
//   y[m, n] = act(sum_b sx[b, m] sw[b, n / 128] (sum_{k in block b} xc[m, k] wc[n, k]) + bias[n])
//
// The inner sums run on the tensor cores (tcgen05 kind::f8f6f4, e4m3 operands from shared memory,
// fp32 accumulators in TMEM). The scales are any fp32 numbers, so each 128-column block's sums
// leave TMEM and are added, times their scale, into fp32 registers.
//
// Scales and bias are read by plain loads: the kernel may run beside the previous one of its stream,
// which may be writing them until pdl_wait, and ld.global.nc is only for memory that stays constant.
#pragma once
#include "opq_device.cuh"
#include "opq_fp8_format.cuh"

namespace opqfp8 {

using namespace opqdev;

enum { ACT_NONE = 0, ACT_SILU = 1, ACT_GELU_TANH = 2 };

struct LinearArgs {
    const float *xs;        // [kblocks][ld_xs]
    const float *ws;        // [kblocks][ld_ws]
    const uint16_t *bias;   // 16-bit [N], or null
    uint16_t *y;            // 16-bit [M, ldy]
    const uint8_t *x, *w;   // codes, for redo_tile alone (the others come through tensor maps)
    int64_t ldx, ldw;
    int64_t ld_xs, ld_ws, ldy;
    int M, N, K, kblocks;
    int m_tiles, n_tiles;
    int act;
};

// Instruction descriptor, kind::f8f6f4: fp32 accumulator (bits 4..5 = 1), A and B e4m3 (0 in bits
// 7..9 and 10..12), both K-major, N >> 3 in bits 17..22, M >> 4 in bits 24..28.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(uint32_t M, uint32_t N) {
    return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// D[tmem] (+)= A[smem] * B[smem]^T, 32 columns of K, one CTA.
__device__ __forceinline__ void umma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// tcgen05.ld: 32 lanes x 16 consecutive 32-bit columns
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
          "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(taddr));
}

// tcgen05.ld: 32 lanes x 32 consecutive 32-bit columns
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
          "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]),
          "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
          "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(taddr));
}

// The activations, to fp32's accuracy: y = v / (1 + e^-z), z = v for SiLU and
// 2 sqrt(2 / pi) (v + 0.044715 v^3) for GELU's tanh form, which is the same function. With t = e^-|z|,
//   y = v / (1 + t) for v >= 0, v t / (1 + t) below: no difference of near-equal numbers
// (h + h tanh(h) with one hardware tanh is 2.5e-4 |v| off: at -8 as much as SiLU itself).
// t is the square of 2^-h, h = |z| log2(e) / 2 at most 126, which spans every fp32 exponent with the
// flushing ex2. It is never a NaN, so values may share a reciprocal: 1 + t lies in [1, 2], four of them
// multiply to at most 16, and the reciprocals of two such products are one packed Newton iteration.
// That leaves the special-function unit one ex2 per value, as the tanh did. On one box: 4096 x 10240 x
// 3840 with GELU 159.3 us (tanh 157.0; a hardware reciprocal for two values 163, for each one 165; none
// of it 140.7), 333 x 10240 x 3840 with SiLU 21.4 (tanh 20.6).
__device__ __forceinline__ float ex2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 1 / x for x in [1, 16]. Subtracting the bits from a constant negates the exponent and turns the
// mantissa's line around: 5.1 % off at most with this constant, the best of a scan. Each Newton step
// r += r (1 - x r) squares that: 2.6e-3, 6.5e-6, then fp32's last bit.
__device__ __forceinline__ float2 reciprocal2(float2 x) {
    float2 r = make_float2(__uint_as_float(0x7EF311C0u - __float_as_uint(x.x)),
                           __uint_as_float(0x7EF311C0u - __float_as_uint(x.y)));
    const float2 nx = make_float2(-x.x, -x.y), one = make_float2(1.0f, 1.0f);
#pragma unroll
    for (int i = 0; i < 3; ++i) r = fma2(r, fma2(nx, r, one), r);
    return r;
}
template <int ACT>
__device__ __forceinline__ float2 act_exponent(float2 v) {      // z log2(e) / 2
    if (ACT == ACT_SILU) {
        constexpr float k = (float)(0.5 * 1.4426950408889634);
        return mul2(v, make_float2(k, k));
    }
    constexpr float k = (float)(0.7978845608028654 * 1.4426950408889634);
    constexpr float k3 = (float)(0.044715 * 0.7978845608028654 * 1.4426950408889634);
    return mul2(v, fma2(mul2(v, v), make_float2(k3, k3), make_float2(k, k)));
}
template <int ACT>
__device__ __forceinline__ float2 act_exp(float2 v) {           // t
    const float2 h = act_exponent<ACT>(v);
    const float2 e = make_float2(ex2_fast(fmaxf(-fabsf(h.x), -126.0f)), ex2_fast(fmaxf(-fabsf(h.y), -126.0f)));
    return mul2(e, e);
}
// v, or v t where v is negative: a multiplication under a predicate each (as a selection between v
// and v t, 1 to 2% slower over the whole product)
__device__ __forceinline__ float2 act_numerator(float2 v, float2 t) {
    asm("{\n\t.reg .pred p, q;\n\t"
        "setp.lt.f32 p, %0, 0f00000000;\n\tsetp.lt.f32 q, %1, 0f00000000;\n\t"
        "@p mul.f32 %0, %0, %2;\n\t@q mul.f32 %1, %1, %3;\n\t}"
        : "+f"(v.x), "+f"(v.y) : "f"(t.x), "f"(t.y));
    return v;
}
template <int ACT>
__device__ __forceinline__ void activate8(float2 &v0, float2 &v1, float2 &v2, float2 &v3) {
    const float2 one = make_float2(1.0f, 1.0f);
    const float2 t0 = act_exp<ACT>(v0), t1 = act_exp<ACT>(v1), t2 = act_exp<ACT>(v2), t3 = act_exp<ACT>(v3);
    const float2 d0 = fma2(t0, one, one), d1 = fma2(t1, one, one), d2 = fma2(t2, one, one), d3 = fma2(t3, one, one);
    const float2 a = mul2(d0, d1), b = mul2(d2, d3), q = reciprocal2(mul2(a, b));
    const float2 qa = mul2(q, b), qb = mul2(q, a);              // 1 / a, 1 / b
    v0 = mul2(act_numerator(v0, t0), mul2(qa, d1));
    v1 = mul2(act_numerator(v1, t1), mul2(qa, d0));
    v2 = mul2(act_numerator(v2, t2), mul2(qb, d3));
    v3 = mul2(act_numerator(v3, t3), mul2(qb, d2));
}
template <int ACT>
__device__ __forceinline__ float activate1(float v) {
    const float2 v2 = make_float2(v, v), t = act_exp<ACT>(v2);
    return mul2(act_numerator(v2, t), reciprocal2(make_float2(1.0f + t.x, 1.0f + t.y))).x;
}
__device__ __forceinline__ float activate(float v, int act) {
    if (act == ACT_SILU) return activate1<ACT_SILU>(v);
    if (act == ACT_GELU_TANH) return activate1<ACT_GELU_TANH>(v);
    return v;
}
// a thread's outputs, straight through under one branch
template <int N>
__device__ __forceinline__ void activate_all(float2 (&v)[N], int act) {
    static_assert(N % 4 == 0, "eight values at a time");
    if (act == ACT_SILU) {
#pragma unroll
        for (int j = 0; j < N; j += 4) activate8<ACT_SILU>(v[j], v[j + 1], v[j + 2], v[j + 3]);
    } else if (act == ACT_GELU_TANH) {
#pragma unroll
        for (int j = 0; j < N; j += 4) activate8<ACT_GELU_TANH>(v[j], v[j + 1], v[j + 2], v[j + 3]);
    }
}

// A block's sums are scaled by one number, s = sx sw, in the fused multiply-add that adds them up. The
// scales are any fp32 numbers, so s may overflow (and make a sum of zero a NaN) or fall below the
// normal range (and lose bits) where the scaled sums do neither. Such sums (0, or 2^-18 to 2^25) are
// multiplied by one scale, then added times the other: the smaller first where the product is large,
// the larger first where it is small, so that the normal range is left only if the result leaves it.
//
// The loops that add the blocks up cannot ask for it: a choice inside them, or a second such loop beside
// them, cost 4 to 20% of the product (registers). They keep the smallest and the largest product they
// met. A CTA whose sums can have lost by them (lost_by_scales) does the rows in question again on
// mma.sync, straight from global memory and many times slower. No scales of real data come to that, and the
// asking costs them 1% (4096 x 10240 x 3840 138.0 -> 139.6 us, 256 x 3840 x 3840 12.95 -> 13.35; with every
// row done again 9 and 0.7 ms).
constexpr float kNormal = 1.1754943508222875e-38f, kLargest = 3.4028234663852886e38f;
__device__ __forceinline__ bool two_factors(float sx, float sw) {
    const float s = fabsf(sx * sw);
    return !(s >= kNormal && s <= kLargest) && sx != 0.0f && sw != 0.0f && fabsf(sx) <= kLargest && fabsf(sw) <= kLargest;
}
// Products below the normal range are off by up to 2^-150, so each block's part of a sum by up to
// 2^-125: that shows in sums below 2^-100. Sums of zero stay (zero rows against zero blocks of W).
template <int N>
__device__ __forceinline__ bool small_sums(const float2 (&v)[N]) {
    bool any = false;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const float x = fabsf(v[j].x), y = fabsf(v[j].y);
        any = any || (x < 7.888609052210118e-31f && x > 0.0f) || (y < 7.888609052210118e-31f && y > 0.0f);
    }
    return any;
}
template <int N>
__device__ __forceinline__ bool lost_by_scales(float smallest, float largest, const float2 (&v)[N]) {
    if (smallest >= kNormal && largest <= kLargest) return false;
    return smallest == 0.0f || largest > kLargest || small_sums(v);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ uint32_t decode_f16x2(uint32_t codes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    return h;
}

// Rows m0 .. m0 + 16 MT - 1, features n0 .. n0 + cols - 1 (past the ends too) once more by `warps` warps (a
// multiple of MT), this one the `warp`-th: the rows with a scale in two factors. The k order inside a
// 128-column block is free as long as both operands have it: a lane takes eight codes of each row at a
// time, two MMAs' worth. e4m3 is exact in fp16, and the products in fp32.
template <int DT, int MT>
__device__ __forceinline__ void redo_tile(const LinearArgs &A, int m0, int n0, int cols, int warp, int warps) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int mb = m0 + warp % MT * 16;
    if (mb >= A.M) return;
    bool two = false;
    const float *sx = A.xs + (mb + (lane & 15) < A.M ? mb + (lane & 15) : mb);
    for (int nb = n0; nb < n0 + cols && nb < A.N; nb += kBlock) {
        const float *sw = A.ws + nb / kBlock;
#pragma unroll 8
        for (int b = lane >> 4; b < A.kblocks; b += 2) two |= two_factors(sx[(int64_t)b * A.ld_xs], sw[(int64_t)b * A.ld_ws]);
    }
    uint32_t rows = __ballot_sync(0xFFFFFFFFu, two);
    rows = (rows | rows >> 16) & 0xFFFFu;        // the others' bits stay as they are
    if (rows == 0) return;
    const int r0 = mb + g < A.M ? mb + g : A.M - 1, r1 = mb + g + 8 < A.M ? mb + g + 8 : A.M - 1;
    const float *sx0 = A.xs + r0, *sx1 = A.xs + r1;
#pragma unroll 1
    for (int nb = n0 + warp / MT * 8; nb < n0 + cols && nb < A.N; nb += warps / MT * 8) {
        const int n = nb + g < A.N ? nb + g : A.N - 1;
        const float *sw = A.ws + nb / kBlock;
        const uint8_t *x0 = A.x + (int64_t)r0 * A.ldx + t * 8, *x1 = A.x + (int64_t)r1 * A.ldx + t * 8;
        const uint8_t *w0 = A.w + (int64_t)n * A.ldw + t * 8;
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
        for (int b = 0; b < A.kblocks; ++b) {
            float p[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            const int end = (b + 1) * kBlock < A.K ? (b + 1) * kBlock : A.K;
#pragma unroll 4
            for (int k = b * kBlock; k < end; k += 32) {
                const uint2 xa = *reinterpret_cast<const uint2 *>(x0 + k), xb = *reinterpret_cast<const uint2 *>(x1 + k);
                const uint2 wv = *reinterpret_cast<const uint2 *>(w0 + k);
                const uint32_t a0[4] = {decode_f16x2(xa.x), decode_f16x2(xb.x), decode_f16x2(xa.x >> 16), decode_f16x2(xb.x >> 16)};
                const uint32_t b0[2] = {decode_f16x2(wv.x), decode_f16x2(wv.x >> 16)};
                mma_f16(p, a0, b0);
                const uint32_t a1[4] = {decode_f16x2(xa.y), decode_f16x2(xb.y), decode_f16x2(xa.y >> 16), decode_f16x2(xb.y >> 16)};
                const uint32_t b1[2] = {decode_f16x2(wv.y), decode_f16x2(wv.y >> 16)};
                mma_f16(p, a1, b1);
            }
            const float w = sw[(int64_t)b * A.ld_ws];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float x = (i ? sx1 : sx0)[(int64_t)b * A.ld_xs];
                float first = 1.0f, second = x * w;
                if (two_factors(x, w)) {
                    const bool x_first = (fabsf(x) > fabsf(w)) != (fabsf(second) > 1.0f);
                    first = x_first ? x : w;
                    second = x_first ? w : x;
                }
                sum[2 * i] = fmaf(p[2 * i] * first, second, sum[2 * i]);
                sum[2 * i + 1] = fmaf(p[2 * i + 1] * first, second, sum[2 * i + 1]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = mb + g + (i / 2) * 8, c = nb + 2 * t + (i & 1);
            if (m < A.M && c < A.N && (rows >> (g + (i / 2) * 8) & 1)) {
                const float bv = A.bias != nullptr ? unpack16_1<DT>(A.bias[c]) : 0.0f;
                A.y[(int64_t)m * A.ldy + c] = pack16_1<DT>(activate(sum[i] + bv, A.act));
            }
        }
    }
}

// mbar_wait with the clock left alone at first: reading the time and the limit costs several
// hundred cycles, as much as a block's MMAs, and a wait here rarely succeeds at its first try but
// nearly always within a few. Only a wait that outlasts kSpins tries comes to the time limit.
constexpr int kSpins = 4096;
__device__ __forceinline__ bool wait8(uint64_t *bar, uint32_t parity) {
    const uint32_t a = smem_u32(bar);
#pragma unroll 1
    for (int i = 0; i < kSpins; ++i)
        if (mbar_try_wait(a, parity)) return true;
    return mbar_wait(bar, parity);
}
// one look, without waiting
__device__ __forceinline__ bool mbar_test_wait(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// A wait whose verdict is the whole warp's, so that a time-out seen by one lane never leaves the
// others behind. Every lane polls: one lane polling for the others, with the branch and the
// shuffle that takes, measured 40% slower over the whole wide kernel.
__device__ __forceinline__ bool warp_wait8(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xFFFFFFFFu, wait8(bar, parity)) != 0;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// the address in CTA `rank`'s shared memory that corresponds to this CTA's `addr`
__device__ __forceinline__ uint32_t mapa(uint32_t addr, uint32_t rank) {
    uint32_t d;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(addr), "r"(rank));
    return d;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// true in one lane of a converged warp. Around the MMA issue it keeps the loop itself uniform, so
// that descriptors live in uniform registers; a lane-0 branch around the whole loop moves each
// operand over from the vector side, 70-90 cycles per MMA against the 64-128 that one runs.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// one arrival, by the lanes with `on` (a predicate, no branch)
__device__ __forceinline__ void mbar_arrive_if(uint64_t *bar, bool on) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}"
        ::"r"(smem_u32(bar)), "r"((int)on) : "memory");
}

__device__ __forceinline__ void tma_prefetch_2d(const void *tmap, int32_t c0, int32_t c1) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(tmap), "r"(c0), "r"(c1)
                 : "memory");
}

__device__ __forceinline__ void named_bar(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// the same, and whether any of the threads came with `on`
__device__ __forceinline__ bool named_bar_any(int id, int threads, bool on) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %3, 0;\n\t"
        "bar.red.or.pred q, %1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any) : "r"(id), "r"(threads), "r"((int)on) : "memory");
    return any != 0;
}

// ---------------------------------------------------------------------------------------------
// Narrow tiles: 128 rows of W (the MMA's M, so that a TMEM lane is an output feature) x BX rows
// of x. For few rows of x the product is bound by streaming W once; a cluster of S CTAs cuts the
// tile's blocks into S ranges so that the stream reaches every SM, and the ranges' fp32 sums meet
// through the cluster's shared memory in rank order (no workspace, the same bits every run).
// Measured: 1 x 11520 x 3840 9.9 us (44 MB, 0.68 of the copy bandwidth), 32 x 11520 x 3840 12.0,
// 37 x 3840 x 10240 12.8 (its 64-row kernel keeps to 80 registers for two CTAs per SM and spills 44
// bytes); one launch costs about 3 us before and after its stream (barriers, the first
// copies' latency, the cluster's exchange), and a block is a chain of hand-overs (copy, MMA, sums) of
// about 0.4 us per CTA, which two CTAs per SM and two issuing warps overlap. Reading W straight into
// mma.sync operands instead started faster (2.1 us for 512 x 1024 against 2.9) but was bound by its
// conversions on real layers (13.5 us).
//   warp 0       TMA producer: one 128-column block of W and of x per stage, 128-byte swizzle
//   warps 1, 2   TMEM allocation (warp 1), the MMA issue (4 per block), one block each in turn
//   warps 4..    per block: sums out of TMEM, times the scales, into fp32 registers; the output
// ---------------------------------------------------------------------------------------------
template <int BX>
struct NarrowCfg {
    static constexpr int W_BYTES = 128 * 128;
    static constexpr int X_BYTES = BX * 128;
    static constexpr int STAGE = W_BYTES + X_BYTES;
    static constexpr int STAGES = 4;                                   // two CTAs per SM (79 to 104 KB each)
    // blocks of W asked for ahead of the previous kernel's end: as many as the first copies take
    // (1 x 3840 x 3840 5.98 -> 5.75 us, 64 x 3840 x 3840 9.67 -> 9.35; ten blocks gain nothing more and
    // cost 37 x 3840 x 10240 1.5 us)
    static constexpr int AHEAD = STAGES;
    static constexpr int NACC = 4;                                     // blocks of sums in TMEM
    static constexpr uint32_t TMEM_COLS = NACC * BX;
    // scales of a chunk of blocks, 512 values (4 per epilogue thread), two chunks
    static constexpr int CHUNK = 512 / BX;
    static constexpr int OFF_SCALE = STAGES * STAGE;
    static constexpr int OFF_BAR = OFF_SCALE + 2 * 512 * 4;
    static constexpr int NUM_BARS = 2 * STAGES + NACC + 1;
    static constexpr int OFF_TMEM = OFF_BAR + NUM_BARS * 8;
    static constexpr int SMEM = OFF_TMEM + 16 + 1024;      // 1 KiB to align the stages
    // EP warps per TMEM lane quarter, CW rows of x (columns of sums) each, so that a block is one TMEM
    // load per warp (37 x 3840 x 10240: 12.9 us; one warp for all 64 columns 13.7)
    static constexpr int EP = BX >= 32 ? 2 : 1, CW = BX / EP;
    static constexpr int THREADS = 128 + 128 * EP;
    static_assert(BX * 128 * 4 <= STAGES * STAGE, "the partial sums reuse the stages");
    static_assert(STAGE % 1024 == 0, "swizzle atoms");
    // one commit per block serves the producer (block i's stage) and the epilogue (block i's sums):
    // a stage's barrier completes again for block i + STAGES, whose MMAs wait for the epilogue to
    // have emptied the accumulator of block i + STAGES - NACC, so no completion is missed
    static_assert(STAGES >= NACC && NACC % 2 == 0, "done ring; an accumulator belongs to one issuer");
    static_assert((TMEM_COLS & (TMEM_COLS - 1)) == 0 && 2 * TMEM_COLS <= 512, "two CTAs' TMEM per SM");
};

template <int BX, int DT>
__global__ void __launch_bounds__(NarrowCfg<BX>::THREADS, 2)
    fp8_narrow_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                      const __grid_constant__ LinearArgs A) {
    using C = NarrowCfg<BX>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t pad = ((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw);
    uint8_t *smem = smem_raw + pad;
    const uint32_t sbase = smem_u32(smem);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *done = full + C::STAGES;         // a stage's MMAs are done: its copies may go, its sums are there
    uint64_t *acc_empty = done + C::STAGES;
    uint64_t *drain = acc_empty + C::NACC;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_TMEM);
    volatile uint32_t *low_slot = tmem_slot + 1;     // a scale product lies outside the normal range
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        *low_slot = 0;
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&done[s], 1);
        }
        for (int s = 0; s < C::NACC; ++s) {
            mbar_init(&acc_empty[s], 4 * C::EP);
        }
        mbar_init(drain, 2);
        fence_mbar_init();
        tma_prefetch_desc(&tmap_w);
        tma_prefetch_desc(&tmap_x);
    }
    // Two kernels' CTAs can share an SM here, so that tensor memory must not close a circle of waits:
    // the next kernel may start only when this CTA has its own, and this CTA gives it back before it
    // waits for its cluster.
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
        if (lane == 0) pdl_launch_dependents();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const int S = (int)cluster_size(), rank = (int)cluster_rank();
    const int tile = (int)(blockIdx.x / (unsigned)S);
    bool redo = false;      // this thread saw sums that lost by their scales
    const int n_blk = tile / A.m_tiles, m_blk = tile - n_blk * A.m_tiles;
    const int b0 = (int)((int64_t)A.kblocks * rank / S), b1 = (int)((int64_t)A.kblocks * (rank + 1) / S);

    if (warp == 0) {
        if (lane == 0) {
            // The range's first blocks of W start for L2 before the previous kernel of the stream has
            // ended. A prefetch returns nothing, so it cannot return what that kernel still changes:
            // its writes and the copies below meet in L2.
            for (int b = b0; b < b1 && b < b0 + C::AHEAD; ++b) tma_prefetch_2d(&tmap_w, b * kBlock, n_blk * 128);
            pdl_wait();
            bool ok = true;
            int issued = 0;
            for (int b = b0; b < b1; ++b) {
                const int s = issued % C::STAGES;
                if (!(ok = wait8(&done[s], (uint32_t)(issued / C::STAGES & 1) ^ 1u))) break;
                uint8_t *st = smem + s * C::STAGE;
                mbar_arrive_expect_tx(&full[s], C::STAGE);
                tma_load_2d(st, &tmap_w, b * kBlock, n_blk * 128, &full[s]);
                tma_load_2d(st + C::W_BYTES, &tmap_x, b * kBlock, m_blk * BX, &full[s]);
                ++issued;
            }
            if (!ok)   // a wait gave up: the copies in flight land before the CTA leaves
                for (int i = issued > C::STAGES ? issued - C::STAGES : 0; i < issued; ++i)
                    wait8(&full[i % C::STAGES], (uint32_t)(i / C::STAGES & 1));
        }
    }

    if (warp == 1 || warp == 2) {
        // two warps issue in turn: a block's two waits, four MMAs and commit take one of them longer
        // than its bytes take to arrive
        constexpr uint32_t idesc = idesc_e4m3_f32(128, BX);
        for (int i = warp - 1; i < b1 - b0; i += 2) {
            const int s = i % C::STAGES, a = i % C::NACC;
            if (!warp_wait8(&acc_empty[a], (uint32_t)(i / C::NACC & 1) ^ 1u)) break;
            if (!warp_wait8(&full[s], (uint32_t)(i / C::STAGES & 1))) break;
            tc_fence_after();
            const uint64_t wd = smem_desc_sw128(sbase + s * C::STAGE);
            const uint64_t xd = smem_desc_sw128(sbase + s * C::STAGE + C::W_BYTES);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 4; ++k)     // 32 columns (32 bytes, 2 descriptor units) each
                    umma_f8_ss(tmem + a * BX, wd + 2 * k, xd + 2 * k, idesc, k > 0);
                umma_commit(&done[s]);
            }
            __syncwarp();
        }
        if (elect_one()) umma_commit(drain);
        __syncwarp();
        warp_wait8(drain, 0);
    } else if (warp >= 4) {
        const int q = warp & 3;                      // TMEM lanes 32 q .. 32 q + 31
        const int e = q * 32 + lane;                 // this thread's output feature in the tile
        const int x0 = ((warp - 4) >> 2) * C::CW;    // and its first row of x
        const int m0 = m_blk * BX, n = n_blk * 128 + e;
        const int et = threadIdx.x - 128;
        float *sc = reinterpret_cast<float *>(smem + C::OFF_SCALE);
        float2 acc[C::CW / 2];
#pragma unroll
        for (int j = 0; j < C::CW / 2; ++j) acc[j] = make_float2(0.0f, 0.0f);
        pdl_wait();
        // the scale of (block, row of x), times the block's scale of W: PER per thread and chunk
        constexpr int PER = 4 / C::EP, EPT = 128 * C::EP;
        float pre[PER];
        auto fetch = [&](int c) {
#pragma unroll
            for (int u = 0; u < PER; ++u) {
                const int idx = u * EPT + et, b = c + idx / BX, m = m0 + idx % BX;
                pre[u] = 0.0f;
                if (b < b1 && m < A.M) {
                    const float sx = A.xs[(int64_t)b * A.ld_xs + m], sw = A.ws[(int64_t)b * A.ld_ws + n_blk];
                    pre[u] = sx * sw;
                    if (two_factors(sx, sw)) {
                        *low_slot = 1;
                        redo = redo || pre[u] == 0.0f || fabsf(pre[u]) > 1.0f;
                    }
                }
            }
        };
        fetch(b0);
        bool ok = true;
        for (int c = b0, ci = 0; c < b1; c += C::CHUNK, ++ci) {
            float *buf = sc + (ci & 1) * 512;
#pragma unroll
            for (int u = 0; u < PER; ++u) buf[u * EPT + et] = pre[u];
            named_bar(1, EPT);
            if (c + C::CHUNK < b1) fetch(c + C::CHUNK);
            const int cend = c + C::CHUNK < b1 ? c + C::CHUNK : b1;
#pragma unroll 1
            for (int b = c; b < cend; ++b) {
                const int i = b - b0, a = i % C::NACC;
                // a warp whose wait gave up skips the blocks that are left but still comes to every
                // chunk's barrier: the other warps may not have seen the time-out
                if (ok) ok = warp_wait8(&done[i % C::STAGES], (uint32_t)(i / C::STAGES & 1));
                if (!ok) continue;
                tc_fence_after();
                const float4 *sb = reinterpret_cast<const float4 *>(buf + (b - c) * BX + x0);
                const uint32_t ta = tmem + ((uint32_t)(q * 32) << 16) + a * BX + x0;
                float t[C::CW];
                if (C::CW == 16)
                    tmem_ld16(ta, *reinterpret_cast<float (*)[16]>(t));
                else
                    tmem_ld32(ta, t);
                tmem_ld_wait();
                tc_fence_before();
                mbar_arrive_if(&acc_empty[a], lane == 0);
#pragma unroll
                for (int j = 0; j < C::CW / 4; ++j) {
                    const float4 s4 = sb[j];
                    acc[2 * j] = fma2(make_float2(t[4 * j], t[4 * j + 1]), make_float2(s4.x, s4.y), acc[2 * j]);
                    acc[2 * j + 1] = fma2(make_float2(t[4 * j + 2], t[4 * j + 3]), make_float2(s4.z, s4.w), acc[2 * j + 1]);
                }
            }
        }
        if (*low_slot != 0) redo = redo || small_sums(acc);     // (set before the last chunk's barrier)
        const int rows = A.M - m0 < BX ? A.M - m0 : BX;
        if (S == 1) {
            const float bv = (A.bias != nullptr && n < A.N) ? unpack16_1<DT>(A.bias[n]) : 0.0f;
            if (ok && n < A.N) {
#pragma unroll
                for (int j = 0; j < C::CW / 2; ++j) acc[j] = fma2(acc[j], make_float2(1.0f, 1.0f), make_float2(bv, bv));
                activate_all(acc, A.act);
#pragma unroll
                for (int j = 0; j < C::CW; ++j)
                    if (x0 + j < rows)
                        A.y[(int64_t)(m0 + x0 + j) * A.ldy + n] = pack16_1<DT>(j & 1 ? acc[j / 2].y : acc[j / 2].x);
            }
        } else {
            // this range's sums into the stages (every copy has landed and every MMA has read them
            // once the last block's sums are complete), [row of x][feature]
            float *part = reinterpret_cast<float *>(smem);
#pragma unroll
            for (int j = 0; j < C::CW; ++j)
                if (x0 + j < rows) part[(x0 + j) * 128 + e] = j & 1 ? acc[j / 2].y : acc[j / 2].x;
        }
    }

    __syncwarp();
    tc_fence_before();
    redo = __syncthreads_or(redo) != 0;
    if (warp == 1) tmem_dealloc(tmem, C::TMEM_COLS);
    if (S > 1) {
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        {
            // every warp takes part: a row of x per 128 threads
            const int e = threadIdx.x & 127;
            const int m0 = m_blk * BX, n = n_blk * 128 + e;
            const int rows = A.M - m0 < BX ? A.M - m0 : BX;
            const float bv = (A.bias != nullptr && n < A.N) ? unpack16_1<DT>(A.bias[n]) : 0.0f;
            for (int j = rank + S * (threadIdx.x >> 7); j < rows; j += S * (C::THREADS / 128)) {
                // all ranges' sums asked for at once, added in rank order
                const uint32_t at = sbase + (uint32_t)(j * 128 + e) * 4u;
                float p[8], v = 0.0f;
#pragma unroll
                for (int r = 0; r < 8; ++r) p[r] = r < S ? ld_cluster_f32(mapa(at, (uint32_t)r)) : 0.0f;
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r < S) v += p[r];
                if (n < A.N) A.y[(int64_t)(m0 + j) * A.ldy + n] = pack16_1<DT>(activate(v + bv, A.act));
            }
        }
        __syncwarp();
        cluster_arrive();   // no CTA leaves while another still reads its sums
        cluster_wait();
    }
    // (behind the cluster's stores of the same rows)
    if (redo) redo_tile<DT, BX / 16>(A, m_blk * BX, n_blk * 128, 128, warp, C::THREADS / 32);
}

// ---------------------------------------------------------------------------------------------
// Wide tiles: 128 CG rows of x x BN rows of W, for products bound by the tensor cores. CG = 2
// joins two SMs in one MMA (cta_group::2): each CTA loads its own 128 rows of x and half of the
// tile's rows of W, so a tile costs each SM half of the weight traffic; CG = 1 tiles fill the chip
// when there are few. One persistent CTA (pair) per SM (pair) walks the tiles.
//   warp 0       TMA producer (both CTAs of a pair; all bytes count on the leader's barrier)
//   warps 1, 2   TMEM allocation (warp 1); in the leader, the MMA issue, one block each in turn
//   warp 3       the blocks' scales, by asynchronous copies
//   warps 4..11  TMEM lane = row of x; warps 4..7 take the tile's left columns, 8..11 the right.
//                Each block's sums leave TMEM (two accumulators in turn, so the tensor pipe runs
//                on) and are added times sx[row] sw[block of W]: one scalar per thread and block.
//                The finished rows go through shared memory and leave by TMA.
// Measured: 4096 x 10240 x 3840 140 us (2300 TFLOP/s, 0.70 of twice the bf16 rate; 137 to 146 by box, whose
// power cap sets the clock), with GELU 160; 1089 x 3840 x 3840 18.3 us on single CTAs. Spills, outside
// the block loop as far as times show: pairs 12 bytes stored and 32 loaded, 128 x 128 28 and 120,
// 128 x 256 none. A block is 512 cycles of MMA and takes about 850: the
// sums of two blocks fill TMEM, so block i + 2 waits for block i's trip through the epilogue (commit to
// wait 200 cycles, loads 250, hand-back 250), and the epilogue's own work per block is about 560.
// Leaving out any one of copies, TMEM loads, additions or scales gains 4 to 15%: nothing alone
// bounds it. Halving the tile's MMAs (N = 128, a barrier per half) was 9% slower on pairs.
// ---------------------------------------------------------------------------------------------
template <int CG, int BN>
struct WideCfg {
    static constexpr int X_BYTES = 128 * 128;
    static constexpr int W_ROWS = BN / CG;                 // rows of W in this CTA's shared memory
    static constexpr int W_BYTES = W_ROWS * 128;
    static constexpr int STAGE = X_BYTES + W_BYTES;
    static constexpr int STAGES = CG == 2 ? 163840 / STAGE : 196608 / STAGE;
    static constexpr int NACC = 2;
    static constexpr uint32_t TMEM_COLS = NACC * BN;
    static constexpr int HALF = BN / 2;                    // columns per epilogue warp
    static constexpr int ROUNDS = HALF / 32;               // 32 columns (64 bytes) staged at a time
    static constexpr int OUT_BYTES = 32 * 64;              // one warp's rows
    // pairs run many tiles each: their stores overlap the next tile's MMAs, from three buffers
    static constexpr int OUT_BUFS = CG == 2 ? 3 : 1;
    // Scales of the blocks under way: 128 rows' and two of W per slot. Block i's copies start when
    // the MMAs of block i - STAGES are done, which says that the epilogue is past block
    // i - STAGES - NACC, so STAGES + NACC slots are enough.
    static constexpr int RING = STAGES + 2 <= 8 ? 8 : 16;
    static constexpr int LAG = STAGES >= 6 ? 2 : 1;        // blocks whose scales may still be in flight
    static constexpr int SCALE_WORDS = 128 + 2;
    static constexpr int OFF_OUT = STAGES * STAGE;
    static constexpr int OFF_SCALE = OFF_OUT + 8 * OUT_BUFS * OUT_BYTES;
    static constexpr int OFF_BIAS = OFF_SCALE + RING * SCALE_WORDS * 4;   // 8 warps x HALF 16-bit values
    static constexpr int OFF_BAR = OFF_BIAS + 8 * HALF * 2;
    static constexpr int NUM_BARS = 2 * STAGES + NACC + 1;
    static constexpr int OFF_TMEM = OFF_BAR + NUM_BARS * 8;
    static constexpr int SMEM = OFF_TMEM + 16;             // the kernel checks the 1 KiB alignment
    static constexpr int THREADS = 384;
    // The epilogue's two warpgroups hold a row's sums (HALF) and 64 columns in flight; the first
    // warpgroup gives up what they take. The launch checks that the kernel was built for REG_LAUNCH.
    static constexpr int REG_LAUNCH = 168, REG_EPI = 224, REG_PROD = 3 * REG_LAUNCH - 2 * REG_EPI;
    static_assert(THREADS * REG_LAUNCH <= 65536 && REG_PROD % 8 == 0 && REG_PROD >= 40, "register split");
    static_assert(SMEM <= 232448 && SMEM > 200 * 1024, "shared memory: one CTA per SM");
    static_assert(STAGES >= NACC && RING >= STAGES + NACC && LAG < STAGES, "done ring (as for the narrow tiles)");
    static_assert(STAGE % 1024 == 0 && HALF % 64 == 0 && TMEM_COLS <= 512, "layout");
};

struct WideArgs {
    LinearArgs l;
    int tma_store;      // y rows start and end on 16-byte boundaries
};

template <int CG>
__device__ __forceinline__ void umma_f8_cg(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
    if (CG == 1) {
        umma_f8_ss(d_tmem, a_desc, b_desc, idesc, accumulate);
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
    }
}
// arrive on `bar` (in every CTA of the pair) when the MMAs issued so far are done
template <int CG>
__device__ __forceinline__ void umma_commit_cg(uint64_t *bar) {
    if (CG == 1) {
        umma_commit(bar);
    } else {
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
            ::"r"(smem_u32(bar)), "h"((uint16_t)3) : "memory");
    }
}
// the same, in this CTA only
template <int CG>
__device__ __forceinline__ void umma_commit_own(uint64_t *bar) {
    if (CG == 1)
        umma_commit(bar);
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                     ::"r"(smem_u32(bar)) : "memory");
}
// a tile copy into this CTA, counted on the barrier at `bar` (the leader's, for a pair)
template <int CG>
__device__ __forceinline__ void tma_load_cg(uint32_t dst, const void *tmap, int32_t c0, int32_t c1, uint32_t bar) {
    if (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
            ::"r"(dst), "l"(tmap), "r"(c0), "r"(c1), "r"(bar) : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3}], [%4];"
            ::"r"(dst), "l"(tmap), "r"(c0), "r"(c1), "r"(bar) : "memory");
}
template <int CG>
__device__ __forceinline__ void tmem_alloc_cg(uint32_t *slot, uint32_t cols) {
    if (CG == 1) {
        tmem_alloc(slot, cols);
        tmem_relinquish();
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(slot)), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}
template <int CG>
__device__ __forceinline__ void tmem_dealloc_cg(uint32_t addr, uint32_t cols) {
    if (CG == 1)
        tmem_dealloc(addr, cols);
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
// One arrival on a barrier of any CTA of the cluster, by the lanes with `on` (a predicate, no branch).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr, bool on) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "@p mbarrier.arrive.shared::cluster.b64 _, [%0];\n\t}"
        ::"r"(addr), "r"((int)on) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ float lds_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// byte offset of 16-byte chunk `chunk` (0..3) of row `row` in a 64-byte-swizzled tile
__device__ __forceinline__ uint32_t sw64_offset(uint32_t row, uint32_t chunk) {
    return row * 64u + ((chunk ^ ((row >> 1) & 3u)) << 4);
}
// a thread's bulk stores: groups, and waits for all but N of them (to be read; to be done)
__device__ __forceinline__ void tma_store_2d(const void *tmap, uint32_t src, int32_t c0, int32_t c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];"
                 ::"l"(tmap), "r"(c0), "r"(c1), "r"(src) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

template <int CG, int BN, int DT>
__global__ void __launch_bounds__(WideCfg<CG, BN>::THREADS, 1)
    fp8_wide_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w,
                    const __grid_constant__ CUtensorMap tmap_y, const __grid_constant__ WideArgs W) {
    using C = WideCfg<CG, BN>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const LinearArgs &A = W.l;
    const uint32_t sbase = smem_u32(smem);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *done = full + C::STAGES;         // a stage's MMAs are done: its copies may go, its sums are there
    uint64_t *acc_empty = done + C::STAGES;
    uint64_t *drain = acc_empty + C::NACC;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_TMEM);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
    // the swizzled stages need 1 KiB boundaries; the same for every CTA of the launch
    if ((sbase & 1023u) != 0) {
        if (threadIdx.x == 0) atomicOr(&g_error, kErrSmemAlign);
        return;
    }

    // (the next kernel may start at once: with this CTA's shared memory in use, no other CTA that
    // takes tensor memory fits on the SM, so none can hold it while this one still asks)
    if (threadIdx.x == 0) {
        pdl_launch_dependents();
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full[s], 1 + CG);   // the leader's producer and each CTA's scale warp
            mbar_init(&done[s], 1);
        }
        for (int s = 0; s < C::NACC; ++s) {
            mbar_init(&acc_empty[s], 8 * CG);
        }
        mbar_init(drain, 2);
        fence_mbar_init();
        tma_prefetch_desc(&tmap_x);
        tma_prefetch_desc(&tmap_w);
        if (W.tma_store) tma_prefetch_desc(&tmap_y);
    }
    if (warp == 1) tmem_alloc_cg<CG>(tmem_slot, C::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    if (CG == 2) {
        cluster_arrive();   // the peer's barriers are ready before anything arrives on them
        cluster_wait();
    }
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const int tiles = A.m_tiles * A.n_tiles;
    const int first = (int)blockIdx.x / CG, step = (int)gridDim.x / CG;

    if (warp < 4) {
        setmaxnreg_dec<C::REG_PROD>();
        if (warp == 0 && lane == 0) {
            pdl_wait();
            bool ok = true;
            int64_t issued = 0;
            int s = 0;
            uint32_t ph = 0;
            for (int t = first; t < tiles && ok; t += step) {
                const int n_blk = t / A.m_tiles, m_blk = t - n_blk * A.m_tiles;
                const int m0 = m_blk * 128 * CG + (int)rank * 128, n0 = n_blk * BN + (int)rank * C::W_ROWS;
                for (int b = 0; b < A.kblocks; ++b) {
                    if (!(ok = wait8(&done[s], ph ^ 1u))) break;
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], CG * C::STAGE);
                    const uint32_t st = sbase + s * C::STAGE;
                    const uint32_t bar = CG == 2 ? mapa(smem_u32(&full[s]), 0) : smem_u32(&full[s]);
                    tma_load_cg<CG>(st, &tmap_x, b * kBlock, m0, bar);
                    tma_load_cg<CG>(st + C::X_BYTES, &tmap_w, b * kBlock, n0, bar);
                    ++issued;
                    if (++s == C::STAGES) { s = 0; ph ^= 1u; }
                }
            }
            const int64_t tail0 = issued > C::STAGES ? issued - C::STAGES : 0;
            for (int64_t i = tail0; i < issued; ++i) {
                const int ts = (int)(i % C::STAGES);
                const uint32_t tp = (uint32_t)(i / C::STAGES & 1);
                if (ok)
                    ok = wait8(&done[ts], tp);    // no commit arrives after this CTA has left
                else if (rank == 0)
                    wait8(&full[ts], tp);          // a wait gave up: the copies in flight land first
            }
        }
        if ((warp == 1 || warp == 2) && rank == 0) {
            // Two warps issue in turn, one per accumulator: a block's two waits, four MMAs and commit
            // take one warp longer than the MMAs run.
            constexpr uint32_t idesc = idesc_e4m3_f32(128 * CG, BN);
            const uint64_t xd0 = smem_desc_sw128(sbase), wd0 = smem_desc_sw128(sbase + C::X_BYTES);
            const int a = warp - 1;
            const uint32_t d = tmem + (uint32_t)a * BN;
            const int64_t blocks = first < tiles ? (int64_t)((tiles - 1 - first) / step + 1) * A.kblocks : 0;
            int s = a;
            uint32_t ph = 0, aph = 0;
            for (int64_t i = a; i < blocks; i += 2) {
                // the operands first: they are there long before the accumulator comes back
                if (!warp_wait8(&full[s], ph)) break;
                if (!warp_wait8(&acc_empty[a], aph ^ 1u)) break;
                tc_fence_after();
                const uint64_t xd = xd0 + (uint32_t)(s * (C::STAGE >> 4)), wd = wd0 + (uint32_t)(s * (C::STAGE >> 4));
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) umma_f8_cg<CG>(d, xd + 2 * k, wd + 2 * k, idesc, k > 0);
                    umma_commit_cg<CG>(&done[s]);
                }
                __syncwarp();
                s += 2;
                if (s >= C::STAGES) { s -= C::STAGES; ph ^= 1u; }
                aph ^= 1u;
            }
            if (elect_one()) umma_commit_own<CG>(drain);
            __syncwarp();
            warp_wait8(drain, 0);
        }
        if (warp == 3) {
            // Scales: asynchronous copies into the ring; a block's arrival counts on the barrier that
            // its MMAs wait for, so that whoever sees its sums sees its scales too.
            pdl_wait();
            const uint32_t ring = smem_u32(smem + C::OFF_SCALE);
            const uint32_t bar0 = CG == 2 ? mapa(smem_u32(full), 0) : smem_u32(full);   // the leader's
            bool ok = true;
            int s = 0, sl = 0, behind = 0;
            uint32_t ph = 0, slot = 0;
            auto announce = [&]() {
                __syncwarp();
                mbar_arrive_cluster(bar0 + sl * 8, lane == 0);
                if (++sl == C::STAGES) sl = 0;
            };
            for (int t = first; t < tiles && ok; t += step) {
                const int n_blk = t / A.m_tiles, m_blk = t - n_blk * A.m_tiles;
                const int m = m_blk * 128 * CG + (int)rank * 128 + lane;
                const float *gx = A.xs;
                const float *gw = A.ws;
                const int nh = n_blk * BN + (lane & 1) * C::HALF;
                if (nh < A.N) gw += nh / kBlock;
                for (int b = 0; b < A.kblocks; ++b) {
                    if (!(ok = warp_wait8(&done[s], ph ^ 1u))) break;
                    const uint32_t dst = ring + slot;
#pragma unroll
                    for (int u = 0; u < 4; ++u) cp_async4(dst + (u * 32 + lane) * 4, gx + (m + u * 32 < A.M ? m + u * 32 : 0));
                    if (lane < 2) cp_async4(dst + (128 + lane) * 4, gw);
                    cp_async_commit();
                    gx += A.ld_xs;
                    gw += A.ld_ws;
                    cp_async_wait<C::LAG>();
                    if (behind == C::LAG) announce(); else ++behind;
                    slot = slot == (C::RING - 1) * C::SCALE_WORDS * 4 ? 0 : slot + C::SCALE_WORDS * 4;
                    if (++s == C::STAGES) { s = 0; ph ^= 1u; }
                }
            }
            cp_async_wait<0>();
            if (ok)
                for (; behind > 0; --behind) announce();
        }
    } else {
        setmaxnreg_inc<C::REG_EPI>();
        const int q = warp & 3, half = (warp - 4) >> 2;
        const uint32_t lane_base = tmem + ((uint32_t)(q * 32) << 16) + half * C::HALF;
        uint8_t *stage = smem + C::OFF_OUT + (warp - 4) * C::OUT_BUFS * C::OUT_BYTES;
        uint16_t *bias_s = reinterpret_cast<uint16_t *>(smem + C::OFF_BIAS) + (warp - 4) * C::HALF;
        bool ok = true;
        int a = 0, sd = 0;
        uint32_t sph = 0;
        const uint32_t acc_bar = CG == 2 ? mapa(smem_u32(acc_empty), 0) : smem_u32(acc_empty);   // the leader's
        const uint32_t my_scale = smem_u32(smem + C::OFF_SCALE) + (q * 32 + lane) * 4;
        const uint32_t w_scale = smem_u32(smem + C::OFF_SCALE) + (128 + half) * 4;
        uint32_t slot = 0;
        int ob = 0;
        bool ready = false;      // the next block's sums are known to be complete, and `s` is its scale
        float s = 0.0f;
        float smallest = 1.0f, largest = 1.0f;     // scale products
        bool redo = false;
        pdl_wait();
        for (int t = first; t < tiles && ok; t += step) {
            const int n_blk = t / A.m_tiles, m_blk = t - n_blk * A.m_tiles;
            const int mw = m_blk * 128 * CG + (int)rank * 128 + q * 32;     // the warp's first row
            const int n0 = n_blk * BN + half * C::HALF;                     // and column
            if (A.bias != nullptr) {
                __syncwarp();
                for (int j = lane; j < C::HALF; j += 32) bias_s[j] = n0 + j < A.N ? A.bias[n0 + j] : (uint16_t)0;
                __syncwarp();      // every lane reads what all lanes stored
            }
            float2 acc[C::HALF / 2];
#pragma unroll
            for (int j = 0; j < C::HALF / 2; ++j) acc[j] = make_float2(0.0f, 0.0f);
#pragma unroll 1
            for (int b = 0; b < A.kblocks; ++b) {
                if (!ready) {
                    if (!(ok = warp_wait8(&done[sd], sph))) break;
                    s = lds_f32(my_scale + slot) * lds_f32(w_scale + slot);
                }
                smallest = fminf(smallest, fabsf(s));
                largest = fmaxf(largest, fabsf(s));
                tc_fence_after();
                if (++sd == C::STAGES) { sd = 0; sph ^= 1u; }
                slot = slot == (C::RING - 1) * C::SCALE_WORDS * 4 ? 0 : slot + C::SCALE_WORDS * 4;
                const float2 s2 = make_float2(s, s);
                const uint32_t ta = lane_base + a * BN;
                // 64 columns at a time; the next 32 are asked for as soon as their registers are free, and
                // the accumulator is handed back before the last sums are added
                float r[64];
                tmem_ld32(ta, r);
                tmem_ld32(ta + 32, r + 32);
                // is the next block there already? Asked now, answered for free when this one is added
                const bool peek = mbar_test_wait(&done[sd], sph);
                tmem_ld_wait();
                auto add32 = [&](int c0, const float *v) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        acc[c0 / 2 + j] = fma2(make_float2(v[2 * j], v[2 * j + 1]), s2, acc[c0 / 2 + j]);
                };
                if (C::HALF == 128) {
                    add32(0, r);
                    tmem_ld32(ta + 64, r);
                    add32(32, r + 32);
                    tmem_ld32(ta + 96, r + 32);
                    tmem_ld_wait();
                }
                // (the wait above is the whole warp's: one lane may speak for it)
                tc_fence_before();
                mbar_arrive_cluster(acc_bar + a * 8, lane == 0);
                ready = __all_sync(0xFFFFFFFFu, peek) != 0;
                if (ready) s = lds_f32(my_scale + slot) * lds_f32(w_scale + slot);
                add32(C::HALF - 64, r);
                add32(C::HALF - 32, r + 32);
                if (++a == C::NACC) a = 0;
            }
            if (!ok) break;
            redo = redo || lost_by_scales(smallest, largest, acc);
            // The rows' outputs, 32 columns at a time: each lane leaves its row's 64 bytes in shared
            // memory in the TMA store's swizzle. The store is asynchronous because all CTAs finish
            // their tiles together: 10 MB at once, 2 us of L2 writes (stored by the warps
            // themselves that was 4300 cycles a tile).
            // Bias and activation first, each straight through under one branch: with the choices
            // inside the loops a tile's outputs took 8000 cycles instead of 2000.
            if (A.bias != nullptr) {
#pragma unroll
                for (int j = 0; j < C::HALF / 8; ++j) {
                    const uint4 w = reinterpret_cast<const uint4 *>(bias_s)[j];
                    const uint32_t w4[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[4 * j + i] = fma2(acc[4 * j + i], make_float2(1.0f, 1.0f), unpack16<DT>(w4[i]));
                }
            }
            activate_all(acc, A.act);
#pragma unroll
            for (int rd = 0; rd < C::ROUNDS; ++rd) {
                uint8_t *buf = stage + ob * C::OUT_BYTES;
                uint32_t o[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = pack16<DT>(acc[rd * 16 + j]);
                bulk_wait_read<C::OUT_BUFS - 1>();     // the store that last used this buffer has read it
                __syncwarp();
#pragma unroll
                for (int ch = 0; ch < 4; ++ch)
                    *reinterpret_cast<uint4 *>(buf + sw64_offset((uint32_t)lane, (uint32_t)ch)) =
                        make_uint4(o[4 * ch], o[4 * ch + 1], o[4 * ch + 2], o[4 * ch + 3]);
                const int nr = n0 + rd * 32;
                if (W.tma_store) {
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {
                        if (nr < A.N && mw < A.M) tma_store_2d(&tmap_y, smem_u32(buf), nr, mw);
                        bulk_commit();
                    }
                } else {
                    // rows that TMA cannot store (ldy or N % 8 != 0): lanes along the columns, one element
                    // each, no branch per row (4096 x 11521 x 128 44 us against 24 with N = 11520; in
                    // words, with the odd rows' edges apart, 148)
                    __syncwarp();
                    const int rows = A.M - mw < 32 ? A.M - mw : 32;
                    if (nr + lane < A.N) {
                        uint16_t *yr = A.y + (int64_t)mw * A.ldy + nr + lane;
#pragma unroll 4
                        for (int r = 0; r < rows; ++r, yr += A.ldy)
                            *yr = *reinterpret_cast<const uint16_t *>(
                                buf + sw64_offset((uint32_t)r, (uint32_t)(lane >> 3)) + (lane & 7) * 2);
                    }
                }
                if (++ob == C::OUT_BUFS) ob = 0;
            }
        }
        bulk_wait_all();
        __syncwarp();
        if (named_bar_any(1, 256, redo))      // (the rows are stored: all warps come here behind their stores)
            for (int t = first; t < tiles && ok; t += step) {
                const int n_blk = t / A.m_tiles, m_blk = t - n_blk * A.m_tiles;
                redo_tile<DT, 8>(A, m_blk * 128 * CG + (int)rank * 128, n_blk * BN, BN, warp - 4, 8);
            }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (CG == 2) {
        cluster_arrive();   // the pair leaves together: neither's barriers or TMEM are in use
        cluster_wait();
    }
    if (warp == 1) tmem_dealloc_cg<CG>(tmem, C::TMEM_COLS);
}

}  // namespace opqfp8
