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
    int token_block;         // tokens per CTA
    int cols, cols0;         // (head, block) columns of both sides, of side 0
    int pass;                // columns that the CTA's lane groups take at a time
    FastDiv blocks[2], page_div, pass_div;
};

constexpr int kWriteThreads = 256;
constexpr int kWriteTokens = 64;     // most tokens per CTA

// The offsets of a token's slot in one side's codes and scales.
struct SlotAt {
    int64_t codes, scales;
};
__device__ __forceinline__ SlotAt slot_at(const CacheSide &S, int64_t page, int64_t off) {
    return {page * S.page_stride + off * S.token_stride, page * S.scale_page_stride + off * S.scale_token_stride};
}

// A CTA takes token_block tokens. One thread per token looks its slot up; then each group of LANES
// lanes (eight channels a lane) keeps one (head, block) column and walks the tokens, U at a time with
// their loads ahead of the first maximum: what depends on the column is worked out once.
template <int DT, int LANES, int U>
__global__ void __launch_bounds__(kWriteThreads) fp8_cache_write_kernel(const __grid_constant__ WriteArgs A) {
    __shared__ SlotAt s_at[2][kWriteTokens];    // codes -1: a token that is not written
    opqdev::pdl_launch_dependents();
    const int g = threadIdx.x / LANES, l = threadIdx.x % LANES;
    const int64_t t0 = (int64_t)blockIdx.x * A.token_block;
    const int n = (int)(A.tokens - t0 < A.token_block ? A.tokens - t0 : A.token_block);
    opqdev::pdl_wait();
    auto find_slot = [&](int i) {
        const int64_t slot = A.slots[t0 + i];
        SlotAt k{-1, 0}, w{-1, 0};
        if (slot >= A.slot_count) {
            atomicOr(&opqdev::g_error, kErrIndex);
        } else if (slot >= 0) {
            const int64_t page = page_of(slot, A.page_div, A.page_size), off = slot - page * A.page_size;
            k = slot_at(A.side[0], page, off);
            w = slot_at(A.side[1], page, off);
        }
        s_at[0][i] = k;
        s_at[1][i] = w;
    };
    const int row = (int)A.pass_div.div((uint32_t)g), lane_col = g - row * A.pass, step = (int)A.pass_div.div(kWriteThreads / LANES);
    for (int strip = 0; strip < A.cols; strip += A.pass) {
        const int col = strip + lane_col;
        const bool on = row < step && col < A.cols;
        const int which = col >= A.cols0 ? 1 : 0;
        const CacheSide &S = A.side[which];
        const uint32_t rest = on ? (uint32_t)(col - (which ? A.cols0 : 0)) : 0u;
        const uint32_t head = A.blocks[which].div(rest), blk = rest - head * A.blocks[which].d;
        const int c = (int)blk * kBlock + l * 8;
        const bool live = on && c < S.dim;
        const uint8_t *src = S.rows + 2 * ((int64_t)head * S.row_head_stride + c + t0 * S.row_stride);
        uint8_t *codes = S.codes + (int64_t)head * S.head_stride + c;
        float *scales = S.scales + (int64_t)head * S.scale_head_stride + blk;
        // every lane walks the same number of rounds: the maxima are shuffled over the whole warp.
        // The rows are there whatever their slots say, so the first round's loads leave before the
        // slots are known.
        uint4 v[U];
        auto load = [&](int i0) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * step + row;
                v[u] = make_uint4(0, 0, 0, 0);
                if (live && i < n) v[u] = *reinterpret_cast<const uint4 *>(src + 2 * i * S.row_stride);
            }
        };
        load(0);
        if (strip == 0) {
            if (threadIdx.x < (unsigned)n) find_slot(threadIdx.x);
            __syncthreads();
        }
        for (int i0 = 0; i0 < n; i0 += step * U) {
            uint32_t mx[U];
            block_maxima<DT, LANES, U>(v, mx);
            uint32_t own = mx[0];
#pragma unroll
            for (int u = 1; u < U; ++u) own = l % U == u ? mx[u] : own;
            const float om = floored(bits_to_float<DT>(own)), omul = block_mul(om);
            if (on && l < U) {
                const int i = i0 + l * step + row;
                if (i < n && s_at[which][i].codes >= 0) scales[s_at[which][i].scales] = block_scale(om);
            }
            uint2 o[U];
#pragma unroll
            for (int u = 0; u < U; ++u) o[u] = encode8<DT>(v[u], __shfl_sync(0xFFFFFFFFu, omul, u, U));
            load(i0 + step * U);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * step + row;
                if (live && i < n) {
                    const int64_t at = s_at[which][i].codes;
                    if (at >= 0) *reinterpret_cast<uint2 *>(codes + at) = o[u];
                }
            }
        }
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
    int row_block;               // rows per CTA
    int cols, cols0;             // 8-code chunks per row of both sides, of side 0 (heads x dim / 8)
    int pass;                    // chunks that the CTA's threads take at a time
    FastDiv head_chunks[2];      // dim / 8
    FastDiv page_div, pass_div;
};

constexpr int kReadThreads = 256;
constexpr int kReadRows = 64;    // most rows per CTA
constexpr int kReadSeqs = 511;   // most sequences whose cu_rows are staged

// A CTA takes row_block consecutive output rows: one thread per row finds the sequence (binary
// search in cu_rows, staged in shared memory for up to kReadSeqs sequences: one trip to memory
// instead of one per step), the page and the slot; then every thread keeps one 8-code chunk of the
// row (8 bytes in, 16 out: a warp's stores are contiguous) and walks the rows, U loads ahead: what depends on the chunk is worked out
// once.
template <int DT, int U>
__global__ void __launch_bounds__(kReadThreads) fp8_cache_read_kernel(const __grid_constant__ ReadArgs A) {
    __shared__ SlotAt s_at[2][kReadRows];    // codes -1: a row that is not read
    __shared__ int32_t s_cu[kReadSeqs + 1];
    opqdev::pdl_launch_dependents();
    const int64_t r0 = (int64_t)blockIdx.x * A.row_block;
    const int n = (int)(A.rows - r0 < A.row_block ? A.rows - r0 : A.row_block);
    opqdev::pdl_wait();
    const int32_t *cu = A.cu_rows;
    if (A.seqs <= kReadSeqs) {
        for (int i = threadIdx.x; i <= A.seqs; i += kReadThreads) s_cu[i] = A.cu_rows[i];
        __syncthreads();
        cu = s_cu;
    }
    if (threadIdx.x < (unsigned)n) {
        const int64_t r = r0 + threadIdx.x;
        SlotAt k{-1, 0}, w{-1, 0};
        if (r >= cu[0] && r < cu[A.seqs]) {
            int lo = 0, hi = A.seqs;            // cu[lo] <= r < cu[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cu[mid] <= r) lo = mid; else hi = mid;
            }
            const int64_t pos = r - cu[lo] + (A.starts ? (int64_t)A.starts[lo] : 0);
            const int64_t pi = pos >= 0 ? page_of(pos, A.page_div, A.page_size) : A.table_width;
            const int64_t page = pi < A.table_width ? (int64_t)A.page_table[(int64_t)lo * A.ld_table + pi] : -1;
            if (page >= 0 && page < A.pages) {
                k = slot_at(A.side[0], page, pos - pi * A.page_size);
                w = slot_at(A.side[1], page, pos - pi * A.page_size);
            } else {
                atomicOr(&opqdev::g_error, kErrIndex);
            }
        }
        s_at[0][threadIdx.x] = k;
        s_at[1][threadIdx.x] = w;
    }
    __syncthreads();
    const int row = (int)A.pass_div.div(threadIdx.x), lane_col = (int)threadIdx.x - row * A.pass;
    const int step = (int)A.pass_div.div(kReadThreads);
    if (row >= step) return;
    for (int col = lane_col; col < A.cols; col += A.pass) {
        const int which = col >= A.cols0 ? 1 : 0;
        const CacheSide &S = A.side[which];
        const uint32_t rest = (uint32_t)(col - (which ? A.cols0 : 0));
        const uint32_t head = A.head_chunks[which].div(rest), ch = rest - head * A.head_chunks[which].d;
        const uint8_t *codes = S.codes + (int64_t)head * S.head_stride + ch * 8;
        const float *scales = S.scales + (int64_t)head * S.scale_head_stride + ch / 16;
        uint8_t *dst = S.rows + 2 * (r0 * S.row_stride + (int64_t)head * S.row_head_stride + ch * 8);
        for (int i0 = row; i0 < n; i0 += step * U) {
            uint2 v[U];
            float sc[U];
            bool on[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * step;
                on[u] = false;
                if (i < n) {
                    const SlotAt at = s_at[which][i];
                    if (at.codes >= 0) {
                        on[u] = true;
                        v[u] = *reinterpret_cast<const uint2 *>(codes + at.codes);
                        sc[u] = scales[at.scales];
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!on[u]) continue;
                const uint32_t w[2] = {v[u].x, v[u].y};
                uint32_t o[4];
                const float2 s2 = make_float2(sc[u], sc[u]);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    o[2 * j] = pack16<DT>(mul2(decode_e4m3x2((uint16_t)(w[j] & 0xFFFFu)), s2));
                    o[2 * j + 1] = pack16<DT>(mul2(decode_e4m3x2((uint16_t)(w[j] >> 16)), s2));
                }
                *reinterpret_cast<uint4 *>(dst + 2 * (i0 + u * step) * S.row_stride) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
    }
}

}  // namespace opqfp8
