// opq_fp8_linear.cuh — y = act(x W^T + bias) for x [M, K] and W [N, K] in the 8-bit block format:
//
//   y[m, n] = act(sum_b sx[b, m] sw[b, n / 128] (sum_{k in block b} xc[m, k] wc[n, k]) + bias[n])
//
// The inner sums run on the tensor cores (tcgen05 kind::f8f6f4, e4m3 operands from shared memory,
// fp32 accumulators in TMEM). The scales are any fp32 numbers, so each 128-column block's sums
// leave TMEM and are added, times their scale, into fp32 registers.
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
    int64_t ld_xs, ld_ws, ldy;
    int M, N, kblocks;
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

// tanh by the hardware approximation, one MUFU op
__device__ __forceinline__ float tanh_fast(float x) {
    float y;
    asm("tanh.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The activation of one output in fp32, as the packed-weight linears have it: one hardware tanh
// per output (extra error at most about 2.5e-4 |v|).
__device__ __forceinline__ float activate(float v, int act) {
    if (act == ACT_SILU) return v * fmaf(0.5f, tanh_fast(0.5f * v), 0.5f);
    if (act == ACT_GELU_TANH) {
        const float u = 0.7978845608028654f * fmaf(0.044715f * v, v * v, v);
        return 0.5f * v * (1.0f + tanh_fast(u));
    }
    return v;
}

// A wait whose verdict is the whole warp's, so that a time-out seen by one lane never leaves the
// others behind.
__device__ __forceinline__ bool warp_wait8(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity)) != 0;
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

__device__ __forceinline__ void named_bar(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// ---------------------------------------------------------------------------------------------
// Narrow tiles: 128 rows of W (the MMA's M, so that a TMEM lane is an output feature) x BX rows
// of x. For few rows of x the product is bound by streaming W once; a cluster of S CTAs cuts the
// tile's blocks into S ranges so that the stream reaches every SM, and the ranges' fp32 sums meet
// through the cluster's shared memory in rank order (no workspace, the same bits every run).
//   warp 0       TMA producer: one 128-column block of W and of x per stage, 128-byte swizzle
//   warp 1       TMEM allocation, the MMA issue (4 per block)
//   warps 2..5   per block: sums out of TMEM, times the scales, into fp32 registers; the output
// ---------------------------------------------------------------------------------------------
template <int BX>
struct NarrowCfg {
    static constexpr int W_BYTES = 128 * 128;
    static constexpr int X_BYTES = BX * 128;
    static constexpr int STAGE = W_BYTES + X_BYTES;
    static constexpr int STAGES = BX <= 32 ? 5 : (BX <= 64 ? 4 : 3);   // about 100 KiB: two CTAs per SM
    static constexpr int NACC = BX <= 32 ? 4 : (BX <= 64 ? 4 : 2);     // blocks of sums in TMEM
    static constexpr uint32_t TMEM_COLS = NACC * BX < 32 ? 32 : NACC * BX;
    // scales of a chunk of blocks, 512 values (4 per epilogue thread), two chunks
    static constexpr int CHUNK = 512 / BX;
    static constexpr int OFF_SCALE = STAGES * STAGE;
    static constexpr int OFF_BAR = OFF_SCALE + 2 * 512 * 4;
    static constexpr int NUM_BARS = 2 * STAGES + 2 * NACC + 1;
    static constexpr int OFF_TMEM = OFF_BAR + NUM_BARS * 8;
    static constexpr int SMEM = OFF_TMEM + 16 + 1024;      // 1 KiB to align the stages
    static constexpr int THREADS = 192;
    static_assert(BX * 128 * 4 <= STAGES * STAGE, "the partial sums reuse the stages");
    static_assert(STAGE % 1024 == 0, "swizzle atoms");
    static_assert((TMEM_COLS & (TMEM_COLS - 1)) == 0 && 2 * TMEM_COLS <= 512, "two CTAs' TMEM per SM");
};

template <int BX, int DT>
__global__ void __launch_bounds__(NarrowCfg<BX>::THREADS)
    fp8_narrow_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                      const __grid_constant__ LinearArgs A) {
    using C = NarrowCfg<BX>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t pad = ((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw);
    uint8_t *smem = smem_raw + pad;
    const uint32_t sbase = smem_u32(smem);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *empty = full + C::STAGES;
    uint64_t *acc_full = empty + C::STAGES;
    uint64_t *acc_empty = acc_full + C::NACC;
    uint64_t *drain = acc_empty + C::NACC;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_TMEM);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        pdl_launch_dependents();
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < C::NACC; ++s) {
            mbar_init(&acc_full[s], 1);
            mbar_init(&acc_empty[s], 4);
        }
        mbar_init(drain, 1);
        fence_mbar_init();
        tma_prefetch_desc(&tmap_w);
        tma_prefetch_desc(&tmap_x);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const int S = (int)cluster_size(), rank = (int)cluster_rank();
    const int tile = (int)(blockIdx.x / (unsigned)S);
    const int n_blk = tile / A.m_tiles, m_blk = tile - n_blk * A.m_tiles;
    const int b0 = (int)((int64_t)A.kblocks * rank / S), b1 = (int)((int64_t)A.kblocks * (rank + 1) / S);

    if (warp == 0) {
        if (lane == 0) {
            pdl_wait();
            bool ok = true;
            int issued = 0;
            for (int b = b0; b < b1; ++b) {
                const int s = issued % C::STAGES;
                if (!(ok = mbar_wait(&empty[s], (uint32_t)(issued / C::STAGES & 1) ^ 1u))) break;
                uint8_t *st = smem + s * C::STAGE;
                mbar_arrive_expect_tx(&full[s], C::STAGE);
                tma_load_2d(st, &tmap_w, b * kBlock, n_blk * 128, &full[s]);
                tma_load_2d(st + C::W_BYTES, &tmap_x, b * kBlock, m_blk * BX, &full[s]);
                ++issued;
            }
            if (!ok)   // a wait gave up: the copies in flight land before the CTA leaves
                for (int i = issued > C::STAGES ? issued - C::STAGES : 0; i < issued; ++i)
                    mbar_wait(&full[i % C::STAGES], (uint32_t)(i / C::STAGES & 1));
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_e4m3_f32(128, BX);
            for (int b = b0, i = 0; b < b1; ++b, ++i) {
                const int s = i % C::STAGES, a = i % C::NACC;
                if (!mbar_wait(&acc_empty[a], (uint32_t)(i / C::NACC & 1) ^ 1u)) break;
                if (!mbar_wait(&full[s], (uint32_t)(i / C::STAGES & 1))) break;
                tc_fence_after();
                const uint64_t wd = smem_desc_sw128(sbase + s * C::STAGE);
                const uint64_t xd = smem_desc_sw128(sbase + s * C::STAGE + C::W_BYTES);
#pragma unroll
                for (int k = 0; k < 4; ++k)     // 32 columns (32 bytes, 2 descriptor units) each
                    umma_f8_ss(tmem + a * BX, wd + 2 * k, xd + 2 * k, idesc, k > 0);
                umma_commit(&empty[s]);
                umma_commit(&acc_full[a]);
            }
            umma_commit(drain);
            mbar_wait(drain, 0);
        }
    } else {
        const int q = warp & 3;                      // TMEM lanes 32 q .. 32 q + 31
        const int e = q * 32 + lane;                 // this thread's output feature in the tile
        const int m0 = m_blk * BX, n = n_blk * 128 + e;
        float *sc = reinterpret_cast<float *>(smem + C::OFF_SCALE);
        float acc[BX];
#pragma unroll
        for (int j = 0; j < BX; ++j) acc[j] = 0.0f;
        pdl_wait();
        // the scale of (block, row of x), times the block's scale of W: four per thread and chunk
        float pre[4];
        auto fetch = [&](int c) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int idx = u * 128 + e, b = c + idx / BX, m = m0 + idx % BX;
                pre[u] = 0.0f;
                if (b < b1 && m < A.M)
                    pre[u] = __ldg(A.xs + (int64_t)b * A.ld_xs + m) * __ldg(A.ws + (int64_t)b * A.ld_ws + n_blk);
            }
        };
        fetch(b0);
        bool ok = true;
        for (int c = b0, ci = 0; c < b1; c += C::CHUNK, ++ci) {
            float *buf = sc + (ci & 1) * 512;
#pragma unroll
            for (int u = 0; u < 4; ++u) buf[u * 128 + e] = pre[u];
            named_bar(1, 128);
            if (c + C::CHUNK < b1) fetch(c + C::CHUNK);
            const int cend = c + C::CHUNK < b1 ? c + C::CHUNK : b1;
            for (int b = c; b < cend; ++b) {
                const int i = b - b0, a = i % C::NACC;
                // a warp whose wait gave up skips the blocks that are left but still comes to every
                // chunk's barrier: the other warps may not have seen the time-out
                if (ok) ok = warp_wait8(&acc_full[a], (uint32_t)(i / C::NACC & 1));
                if (!ok) continue;
                tc_fence_after();
                const float *sb = buf + (b - c) * BX;
#pragma unroll
                for (int j0 = 0; j0 < BX; j0 += 16) {
                    float t[16];
                    tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + a * BX + j0, t);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const float2 s2 = *reinterpret_cast<const float2 *>(sb + j0 + j);
                        const float2 r = fma2(make_float2(t[j], t[j + 1]), s2, make_float2(acc[j0 + j], acc[j0 + j + 1]));
                        acc[j0 + j] = r.x;
                        acc[j0 + j + 1] = r.y;
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[a]);
            }
        }
        const int rows = A.M - m0 < BX ? A.M - m0 : BX;
        const float bv = (A.bias != nullptr && n < A.N) ? unpack16_1<DT>(__ldg(A.bias + n)) : 0.0f;
        if (S == 1) {
            if (ok && n < A.N) {
#pragma unroll
                for (int j = 0; j < BX; ++j)
                    if (j < rows)
                        A.y[(int64_t)(m0 + j) * A.ldy + n] = pack16_1<DT>(activate(acc[j] + bv, A.act));
            }
        } else {
            // this range's sums into the stages (every copy has landed and every MMA has read them
            // once the last block's sums are complete), [row of x][feature]
            float *part = reinterpret_cast<float *>(smem);
#pragma unroll
            for (int j = 0; j < BX; ++j)
                if (j < rows) part[j * 128 + e] = acc[j];
        }
    }

    if (S > 1) {
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        if (warp >= 2) {
            const int e = (warp & 3) * 32 + lane;
            const int m0 = m_blk * BX, n = n_blk * 128 + e;
            const int rows = A.M - m0 < BX ? A.M - m0 : BX;
            const float bv = (A.bias != nullptr && n < A.N) ? unpack16_1<DT>(__ldg(A.bias + n)) : 0.0f;
            for (int j = rank; j < rows; j += S) {
                float v = 0.0f;
                for (int r = 0; r < S; ++r) v += ld_cluster_f32(mapa(sbase + (uint32_t)(j * 128 + e) * 4u, (uint32_t)r));
                if (n < A.N) A.y[(int64_t)(m0 + j) * A.ldy + n] = pack16_1<DT>(activate(v + bv, A.act));
            }
        }
        __syncwarp();
        cluster_arrive();   // no CTA leaves while another still reads its sums
        cluster_wait();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, C::TMEM_COLS);
}

}  // namespace opqfp8
