// opq_fp8_quantize.cuh — bf16 or fp16 [R, K] to the 8-bit block format (opq_fp8_format.cuh): one
// scale per 128 values of a row (activations), or per 128 x 128 block (weights).
//
// Every value is read once (2 bytes) and written once (1 byte): the bound is HBM. A CTA's loads
// are all issued before the first maximum is formed, so that each SM keeps its share of the
// memory pipe full without a staging buffer; the values wait in registers for their scale.
// Scales are laid out [128-column block][row]: the product reads a block's scales of
// neighbouring rows together.
#pragma once
#include "opq_device.cuh"
#include "opq_fp8_format.cuh"

namespace opqfp8 {

struct QuantArgs {
    const uint8_t *x;   // 16-bit [R, ldx]
    uint8_t *codes;     // [R, ldc]
    float *scales;      // [ceil(K / 128), lds]
    int64_t ldx, ldc, lds;
    int64_t R;
    int K;
    int kgroups;        // CTAs along K
};

constexpr int kQuantThreads = 256;
constexpr int kQuantLoads = 8;     // 16-byte loads per thread in flight

// Scale per row: a CTA takes 32 rows x 4 blocks, sixteen lanes (eight values each) per block.
template <int DT>
__global__ void __launch_bounds__(kQuantThreads) fp8_quantize_rows_kernel(const __grid_constant__ QuantArgs A) {
    __shared__ float s_scale[4][32];
    opqdev::pdl_launch_dependents();
    const int g = threadIdx.x >> 4, l = threadIdx.x & 15;
    const int64_t rt = blockIdx.x / A.kgroups;
    const int kb = (int)(blockIdx.x - rt * A.kgroups) * 4 + (g & 3);
    const int64_t r0 = rt * 32;
    const int col = kb * kBlock + l * 8;
    const bool in_k = col < A.K;       // K % 32 == 0: a lane's eight columns are in or out together
    opqdev::pdl_wait();
    const int left = in_k ? (int)(A.R - r0 < 32 ? A.R - r0 : 32) - (g >> 2) : 0;   // rows from this lane's first
    uint4 v[kQuantLoads];
    const uint8_t *src = A.x + ((r0 + (g >> 2)) * A.ldx + col) * 2;
    const int64_t sstep = 8 * A.ldx, dstep = 4 * A.ldc;
#pragma unroll
    for (int i = 0; i < kQuantLoads; ++i, src += sstep) {
        v[i] = make_uint4(0, 0, 0, 0);
        if (4 * i < left) v[i] = *reinterpret_cast<const uint4 *>(src);
    }
    uint32_t mx[kQuantLoads];
    block_maxima<DT, 16, kQuantLoads>(v, mx);
    // lane l & 7 of a group forms the constants of the group's block l & 7
    uint32_t own = mx[0];
#pragma unroll
    for (int i = 1; i < kQuantLoads; ++i) own = (l & 7) == i ? mx[i] : own;
    const float om = floored(bits_to_float<DT>(own)), omul = block_mul(om);
    if (l < 8) s_scale[g & 3][(g >> 2) + 4 * l] = block_scale(om);
    uint8_t *dst = A.codes + (r0 + (g >> 2)) * A.ldc + col;
#pragma unroll
    for (int i = 0; i < kQuantLoads; ++i, dst += dstep) {
        const uint2 c = encode8<DT>(v[i], __shfl_sync(0xFFFFFFFFu, omul, i, 8));
        if (4 * i < left) *reinterpret_cast<uint2 *>(dst) = c;
    }
    __syncthreads();
    if (threadIdx.x < 128) {
        const int b = threadIdx.x >> 5;
        const int64_t r = r0 + (threadIdx.x & 31);
        const int64_t kbs = (int64_t)(blockIdx.x - rt * A.kgroups) * 4 + b;
        if (r < A.R && kbs * kBlock < A.K) A.scales[kbs * A.lds + r] = s_scale[b][threadIdx.x & 31];
    }
}

// Scale per 128 x 128 block: one CTA per block.
template <int DT>
__global__ void __launch_bounds__(kQuantThreads) fp8_quantize_blocks_kernel(const __grid_constant__ QuantArgs A) {
    __shared__ uint32_t s_max[kQuantThreads / 32];
    opqdev::pdl_launch_dependents();
    const int g = threadIdx.x >> 4, l = threadIdx.x & 15;
    const int64_t rt = blockIdx.x / A.kgroups;
    const int kb = (int)(blockIdx.x - rt * A.kgroups);
    const int64_t r0 = rt * kBlock;
    const int col = kb * kBlock + l * 8;
    const bool in_k = col < A.K;
    opqdev::pdl_wait();
    const int left = in_k ? (int)(A.R - r0 < kBlock ? A.R - r0 : kBlock) - g : 0;   // rows from this lane's first
    uint4 v[kQuantLoads];
    const uint8_t *src = A.x + ((r0 + g) * A.ldx + col) * 2;
    const int64_t sstep = 32 * A.ldx, dstep = 16 * A.ldc;
#pragma unroll
    for (int i = 0; i < kQuantLoads; ++i, src += sstep) {
        v[i] = make_uint4(0, 0, 0, 0);
        if (16 * i < left) v[i] = *reinterpret_cast<const uint4 *>(src);
    }
    auto block_max = [&](uint32_t mx) {
        mx = __reduce_max_sync(0xFFFFFFFFu, mx);
        if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = mx;
        __syncthreads();
        uint32_t best = s_max[0];
#pragma unroll
        for (int w = 1; w < kQuantThreads / 32; ++w) best = max(best, s_max[w]);
        return best;
    };
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < kQuantLoads; ++i) mx = absmax2<DT>(mx, absmax8<DT>(v[i]));
    mx = block_max(absmax_bits<DT>(mx));
    if (mx >= kInfBits<DT>) {      // the same for every thread of the CTA
        uint32_t fin = 0;
#pragma unroll
        for (int i = 0; i < kQuantLoads; ++i) fin = max(fin, absmax8_finite<DT>(v[i]));
        __syncthreads();
        mx = block_max(fin);
    }
    const float m = floored(bits_to_float<DT>(mx)), mul = block_mul(m);
    if (threadIdx.x == 0) A.scales[(int64_t)kb * A.lds + rt] = block_scale(m);
    uint8_t *dst = A.codes + (r0 + g) * A.ldc + col;
#pragma unroll
    for (int i = 0; i < kQuantLoads; ++i, dst += dstep)
        if (16 * i < left) *reinterpret_cast<uint2 *>(dst) = encode8<DT>(v[i], mul);
}

}  // namespace opqfp8
