// opq_fp8_cache.cuh — keys and values quantized into a paged cache as they are written, and
// decoded back for a batch of sequences (format: opq_fp8_format.cuh, blocks along the head's
// channels, the last block of a head shorter where head_dim % 128 != 0).
//
// Both move each value once (2 bytes in, 1 out; 1 in, 2 out) and a scale per block: the bound is
// HBM for long prompts and launch latency for single steps. Every slot and page number comes
// from device memory and is checked against the cache before it is used; one that is out of
// range is skipped and recorded in the device error word (kErrIndex).
#pragma once
#include "opq_device.cuh"
#include "opq_fp8_format.cuh"

namespace opqfp8 {

constexpr uint32_t kErrIndex = 4u;

// One tensor (keys or values) of a cache and the rows written to it or read from it.
struct CacheSide {
    uint8_t *codes;
    float *scales;
    int64_t page_stride, token_stride, head_stride;            // of codes, bytes
    int64_t scale_page_stride, scale_token_stride, scale_head_stride;   // floats
    uint8_t *rows;                                             // 16-bit [tokens][heads][dim]
    int64_t row_stride, row_head_stride;                       // elements
    int dim, blocks;                                           // channels per head, blocks of them
};

// position / page_size; positions past 31 bits (a cache of more than 2^31 slots) take the division
__device__ __forceinline__ int64_t page_of(int64_t pos, const FastDiv &d, int64_t page_size) {
    return pos < ((int64_t)1 << 31) ? (int64_t)d.div((uint32_t)pos) : pos / page_size;
}

struct WriteArgs {
    CacheSide side[2];
    const int64_t *slots;
    int64_t slot_count;      // pages * page_size
    int64_t page_size;
    int64_t tokens;
    uint32_t items;          // tokens x per_token
    uint32_t first_v;        // items of side 0 per token
    FastDiv per_token, blocks[2], page_div;
};

constexpr int kWriteThreads = 256;

// LANES lanes (eight channels each) per (token, head, block) item; U items per lane group, all
// loads ahead of the first maximum.
template <int DT, int LANES, int U>
__global__ void __launch_bounds__(kWriteThreads) fp8_cache_write_kernel(const __grid_constant__ WriteArgs A) {
    constexpr int GROUPS = kWriteThreads / LANES;
    opqdev::pdl_launch_dependents();
    const int g = threadIdx.x / LANES, l = threadIdx.x % LANES;
    opqdev::pdl_wait();
    uint4 v[U];
    uint8_t *dst[U];
    float *sdst[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const uint32_t item = (uint32_t)blockIdx.x * (GROUPS * U) + i * GROUPS + g;
        v[i] = make_uint4(0, 0, 0, 0);
        dst[i] = nullptr;
        sdst[i] = nullptr;
        if (item < A.items) {
            const uint32_t t = A.per_token.div(item);
            uint32_t rest = item - t * A.per_token.d;
            const int which = rest >= A.first_v ? 1 : 0;
            rest -= which ? A.first_v : 0u;
            const CacheSide &S = A.side[which];
            const uint32_t head = A.blocks[which].div(rest);
            const uint32_t blk = rest - head * A.blocks[which].d;
            const int c = (int)blk * kBlock + l * 8;
            const int64_t slot = A.slots[t];
            if (slot >= A.slot_count) {
                if (l == 0) atomicOr(&opqdev::g_error, kErrIndex);
            } else if (slot >= 0) {
                const int64_t page = page_of(slot, A.page_div, A.page_size), off = slot - page * A.page_size;
                if (c < S.dim) {
                    v[i] = *reinterpret_cast<const uint4 *>(
                        S.rows + 2 * ((int64_t)t * S.row_stride + (int64_t)head * S.row_head_stride + c));
                    dst[i] = S.codes + page * S.page_stride + off * S.token_stride + (int64_t)head * S.head_stride + c;
                }
                if (l == 0)
                    sdst[i] = S.scales + page * S.scale_page_stride + off * S.scale_token_stride +
                              (int64_t)head * S.scale_head_stride + blk;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        uint32_t mx = absmax8(v[i]);
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
        const bool wild = mx >= kInfBits<DT>;
        if (__any_sync(0xFFFFFFFFu, wild)) {
            mx = absmax8_finite<DT>(v[i]);
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
        }
        const BlockScale s(bits_to_float<DT>(mx));
        const uint2 c = encode8<DT>(v[i], s, wild);
        if (dst[i]) *reinterpret_cast<uint2 *>(dst[i]) = c;
        if (sdst[i]) *sdst[i] = s.scale;
    }
}

struct ReadArgs {
    CacheSide side[2];
    const int32_t *cu_rows;      // [seqs + 1]: output rows of sequence b are cu_rows[b] .. cu_rows[b + 1] - 1
    const int32_t *page_table;   // [seqs, ld_table]
    const int32_t *starts;       // [seqs]: position in the sequence of its first row, or null for 0
    int64_t ld_table;
    int64_t table_width;         // pages listed per sequence
    int64_t pages, page_size;
    int64_t rows;
    int seqs;
    int tensors;
    int row_block;               // rows per CTA
    uint32_t chunks[2];          // 16-code chunks per row of a side: heads x dim / 16
    FastDiv head_chunks[2];      // dim / 16
    FastDiv per_row;             // chunks of both sides
    FastDiv page_div;            // page_size
};

constexpr int kReadThreads = 256;
constexpr int kReadRows = 16;    // most rows per CTA

// A CTA takes row_block consecutive output rows: one thread per row finds the sequence (binary
// search in cu_rows), the page and the slot; then every lane decodes 16-code chunks (16 bytes
// in, 32 out).
template <int DT, int U>
__global__ void __launch_bounds__(kReadThreads) fp8_cache_read_kernel(const __grid_constant__ ReadArgs A) {
    __shared__ int64_t s_page[kReadRows];   // -1: a row that is not read
    __shared__ int32_t s_off[kReadRows];
    opqdev::pdl_launch_dependents();
    const int64_t r0 = (int64_t)blockIdx.x * A.row_block;
    opqdev::pdl_wait();
    if (threadIdx.x < (unsigned)A.row_block) {
        const int64_t r = r0 + threadIdx.x;
        int64_t page = -1, off = 0;
        if (r < A.rows && r >= A.cu_rows[0] && r < A.cu_rows[A.seqs]) {
            int lo = 0, hi = A.seqs;            // cu_rows[lo] <= r < cu_rows[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (A.cu_rows[mid] <= r) lo = mid; else hi = mid;
            }
            const int64_t pos = r - A.cu_rows[lo] + (A.starts ? (int64_t)A.starts[lo] : 0);
            const int64_t pi = pos >= 0 ? page_of(pos, A.page_div, A.page_size) : 0;
            bool ok = pos >= 0 && pi < A.table_width;
            if (ok) {
                page = A.page_table[(int64_t)lo * A.ld_table + pi];
                off = pos - pi * A.page_size;
                ok = page >= 0 && page < A.pages;
            }
            if (!ok) {
                page = -1;
                atomicOr(&opqdev::g_error, kErrIndex);
            }
        }
        s_page[threadIdx.x] = page;
        s_off[threadIdx.x] = (int32_t)off;
    }
    __syncthreads();
    const uint32_t n = (uint32_t)A.row_block * A.per_row.d;
    for (uint32_t i0 = threadIdx.x; i0 < n; i0 += kReadThreads * U) {
        uint4 v[U];
        float sc[U];
        uint8_t *dst[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t i = i0 + u * kReadThreads;
            dst[u] = nullptr;
            if (i < n) {
                const uint32_t rl = A.per_row.div(i);
                uint32_t rest = i - rl * A.per_row.d;
                const int64_t page = s_page[rl];
                if (page >= 0) {
                    const int which = rest >= A.chunks[0] ? 1 : 0;
                    rest -= which ? A.chunks[0] : 0u;
                    const CacheSide &S = A.side[which];
                    const uint32_t head = A.head_chunks[which].div(rest);
                    const uint32_t ch = rest - head * A.head_chunks[which].d;
                    const int64_t off = s_off[rl];
                    v[u] = *reinterpret_cast<const uint4 *>(S.codes + page * S.page_stride + off * S.token_stride +
                                                            (int64_t)head * S.head_stride + ch * 16);
                    sc[u] = S.scales[page * S.scale_page_stride + off * S.scale_token_stride +
                                     (int64_t)head * S.scale_head_stride + ch / 8];
                    dst[u] = S.rows + 2 * ((r0 + rl) * S.row_stride + (int64_t)head * S.row_head_stride + ch * 16);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!dst[u]) continue;
            const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
            uint32_t o[8];
            const float2 s2 = make_float2(sc[u], sc[u]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                o[2 * j] = pack16<DT>(mul2(decode_e4m3x2((uint16_t)(w[j] & 0xFFFFu)), s2));
                o[2 * j + 1] = pack16<DT>(mul2(decode_e4m3x2((uint16_t)(w[j] >> 16)), s2));
            }
            uint4 *d = reinterpret_cast<uint4 *>(dst[u]);
            d[0] = make_uint4(o[0], o[1], o[2], o[3]);
            d[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
}

}  // namespace opqfp8
