// opq_fp8_quantize.cuh — bf16 or fp16 [R, K] to the 8-bit block format (opq_fp8_format.cuh): one
// scale per 128 values of a row (activations), or per 128 x 128 block (weights).
//
// Every value is read once (2 bytes) and written once (1 byte): the bound is HBM. Loads are issued
// ahead of the arithmetic, so that each SM keeps its share of the memory pipe full without a
// staging buffer; the values wait in registers for their scale.
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
    int kgroups;        // tiles along K
    int64_t tiles;
};

constexpr int kQuantThreads = 256;
constexpr int kQuantLoads = 8;     // 16-byte loads per thread in flight

// Scale per row: tiles of 16 rows x 4 blocks, sixteen lanes (eight values each) per block and four
// blocks per lane. The CTAs of one wave (four per SM) walk the tiles, and a tile's loads leave before
// the last tile's codes are stored: 23.4 us for 4096 x 10240 (5.4 TB/s; one tile per CTA 24.9, a
// second, partial wave of CTAs 26.7), 2.1 us for one row of 3840 (tiles of 32 rows: 2.6).
constexpr int kRowTile = 16;
constexpr int kRowLoads = kRowTile / 4;

template <int DT>
__global__ void __launch_bounds__(kQuantThreads) fp8_quantize_rows_kernel(const __grid_constant__ QuantArgs A) {
    __shared__ float s_scale[2][4][kRowTile];
    opqdev::pdl_launch_dependents();
    const int g = threadIdx.x >> 4, l = threadIdx.x & 15;
    const int64_t sstep = 8 * A.ldx, dstep = 4 * A.ldc;
    uint4 v[kRowLoads];
    int64_t r0 = 0;
    int kg = 0, left = 0;      // the loaded tile's rows and columns; rows from this lane's first (0: no columns)
    auto load = [&](int64_t tile) {
        const int64_t rt = tile / A.kgroups;
        kg = (int)(tile - rt * A.kgroups);
        r0 = rt * kRowTile;
        const int col = (kg * 4 + (g & 3)) * kBlock + l * 8;
        // K % 32 == 0: a lane's eight columns are in or out together
        left = col < A.K ? (int)(A.R - r0 < kRowTile ? A.R - r0 : kRowTile) - (g >> 2) : 0;
        const uint8_t *src = A.x + ((r0 + (g >> 2)) * A.ldx + col) * 2;
#pragma unroll
        for (int i = 0; i < kRowLoads; ++i, src += sstep) {
            v[i] = make_uint4(0, 0, 0, 0);
            if (4 * i < left) v[i] = *reinterpret_cast<const uint4 *>(src);
        }
    };
    opqdev::pdl_wait();
    load(blockIdx.x);
    int side = 0;
    for (int64_t tile = blockIdx.x; tile < A.tiles; tile += gridDim.x, side ^= 1) {
        uint32_t mx[kRowLoads];
        block_maxima<DT, 16, kRowLoads>(v, mx);
        // lane l & 3 of a group forms the constants of the group's block l & 3
        uint32_t own = mx[0];
#pragma unroll
        for (int i = 1; i < kRowLoads; ++i) own = (l & 3) == i ? mx[i] : own;
        const float om = floored(bits_to_float<DT>(own)), omul = block_mul(om);
        if (l < kRowLoads) s_scale[side][g & 3][(g >> 2) + 4 * l] = block_scale(om);
        uint2 o[kRowLoads];
#pragma unroll
        for (int i = 0; i < kRowLoads; ++i) o[i] = encode8<DT>(v[i], __shfl_sync(0xFFFFFFFFu, omul, i, kRowLoads));
        const int64_t tr = r0;
        const int tkg = kg, tleft = left;
        if (tile + gridDim.x < A.tiles) load(tile + gridDim.x);
        uint8_t *dst = A.codes + (tr + (g >> 2)) * A.ldc + (tkg * 4 + (g & 3)) * kBlock + l * 8;
#pragma unroll
        for (int i = 0; i < kRowLoads; ++i, dst += dstep)
            if (4 * i < tleft) *reinterpret_cast<uint2 *>(dst) = o[i];
        __syncthreads();       // (the other side's readers are past this tile's predecessor)
        if (threadIdx.x < 4 * kRowTile) {
            const int b = threadIdx.x / kRowTile, r = threadIdx.x % kRowTile;
            const int64_t kbs = (int64_t)tkg * 4 + b;
            if (tr + r < A.R && kbs * kBlock < A.K) A.scales[kbs * A.lds + tr + r] = s_scale[side][b][r];
        }
    }
}

// Scale per 128 x 128 block: one CTA per block, which holds it in registers between the maximum and
// the codes: 20.2 us for 10240 x 3840 (5.8 TB/s).
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
