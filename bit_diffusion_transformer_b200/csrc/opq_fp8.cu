// opq_fp8.cu — the C ABI of the 8-bit block format (opq_fp8_* in include/opq.h): argument
// validation, TMA descriptors, kernel selection and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>
#include <mutex>
#include <utility>

#include "opq.h"
#include "opq_fp8_cache.cuh"
#include "opq_fp8_linear.cuh"
#include "opq_fp8_quantize.cuh"
#include "opq_host.h"

namespace opqhost {
cudaError_t fp8_device_error(uint32_t *err) {
    uint32_t zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(err, opqdev::g_error, sizeof *err);
    if (e == cudaSuccess && *err != 0) e = cudaMemcpyToSymbol(opqdev::g_error, &zero, sizeof zero);
    return e;
}
cudaError_t fp8_set_wait_limit(uint64_t ns) { return cudaMemcpyToSymbol(opqdev::g_wait_limit_ns, &ns, sizeof ns); }
cudaError_t fp8_get_wait_limit(uint64_t *ns) { return cudaMemcpyFromSymbol(ns, opqdev::g_wait_limit_ns, sizeof *ns); }
}  // namespace opqhost

namespace {

using namespace opqfp8;
using opqhost::check_device;
using opqhost::check_ptrs;
using opqhost::cuda_fail;

constexpr int kSMs = 148;   // B200; schedules depend on the shape alone

bool dtype_ok(int d) { return d == OPQ_DTYPE_BF16 || d == OPQ_DTYPE_FP16; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// every launch may start while the stream's previous kernel finishes (opq_device.cuh)
template <class Kern, class... Args>
opq_status launch(Kern kernel, int64_t grid, int threads, size_t smem, int cluster, void *stream, const Args &...args) {
    if (grid > INT32_MAX) return OPQ_ERR_UNSUPPORTED_SHAPE;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? OPQ_OK : cuda_fail(e);
}

// dynamic shared memory of a kernel, raised once per device. `regs`: the registers per thread that a
// kernel which moves registers between warpgroups (setmaxnreg) was written for; one that was
// built with any other number is refused, not run.
template <class Kern>
opq_status raise_smem(Kern kernel, int bytes, bool (&done)[64], int regs = 0) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    if (dev < 0 || dev >= 64) return OPQ_ERR_CUDA;
    static std::mutex mu;
    std::lock_guard<std::mutex> lk(mu);
    if (!done[dev]) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return cuda_fail(e);
        if (regs > 0) {
            cudaFuncAttributes fa{};
            if ((e = cudaFuncGetAttributes(&fa, kernel)) != cudaSuccess) return cuda_fail(e);
            if (fa.numRegs != regs) return cuda_fail(cudaErrorInvalidConfiguration);
        }
        done[dev] = true;
    }
    return OPQ_OK;
}

// codes [rows, K] with row stride ld, box {128 columns, box_rows}, 128-byte swizzle, zero fill
opq_status make_code_map(CUtensorMap *map, const void *p, int64_t rows, int64_t K, int64_t ld, uint32_t box_rows) {
    opqhost::EncodeTiledFn fn = opqhost::encode_fn();
    if (!fn) return OPQ_ERR_CUDA;
    cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ld};
    cuuint32_t box[2] = {(cuuint32_t)kBlock, box_rows};
    cuuint32_t estr[2] = {1u, 1u};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(p), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? OPQ_OK : cuda_fail((int)r);
}

template <int BX, int DT>
opq_status launch_narrow(const LinearArgs &a, int split, const void *x, int64_t ldx, const void *w, int64_t ldw,
                         int64_t K, void *stream) {
    using C = NarrowCfg<BX>;
    static bool done[64] = {};
    opq_status s = raise_smem(fp8_narrow_kernel<BX, DT>, C::SMEM, done);
    if (s != OPQ_OK) return s;
    CUtensorMap wmap, xmap;
    if ((s = make_code_map(&wmap, w, a.N, K, ldw, 128)) != OPQ_OK) return s;
    if ((s = make_code_map(&xmap, x, a.M, K, ldx, BX)) != OPQ_OK) return s;
    return launch(fp8_narrow_kernel<BX, DT>, (int64_t)a.m_tiles * a.n_tiles * split, C::THREADS, C::SMEM, split, stream,
                  wmap, xmap, a);
}

// y [M, N] with row stride ldy, box {32 columns, 32 rows}, 64-byte swizzle (the epilogue's staging)
opq_status make_y_map(CUtensorMap *map, const LinearArgs &a) {
    opqhost::EncodeTiledFn fn = opqhost::encode_fn();
    if (!fn) return OPQ_ERR_CUDA;
    cuuint64_t dims[2] = {(cuuint64_t)a.N, (cuuint64_t)a.M};
    cuuint64_t strides[1] = {(cuuint64_t)a.ldy * 2};
    cuuint32_t box[2] = {32u, 32u};
    cuuint32_t estr[2] = {1u, 1u};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, a.y, dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? OPQ_OK : cuda_fail((int)r);
}

template <int CG, int BN, int DT>
opq_status launch_wide(const LinearArgs &a, const void *x, int64_t ldx, const void *w, int64_t ldw, int64_t K,
                       void *stream) {
    using C = WideCfg<CG, BN>;
    static bool done[64] = {};
    opq_status s = raise_smem(fp8_wide_kernel<CG, BN, DT>, C::SMEM, done, C::REG_LAUNCH);
    if (s != OPQ_OK) return s;
    WideArgs wa{};
    wa.l = a;
    // A TMA store writes whole 16-byte pieces: where the last column ends inside one, zeros up to its end,
    // beside the output. (Such rows in part by TMA, in part by the warps: 8% slower for every other shape.)
    wa.tma_store = a.ldy % 8 == 0 && a.N % 8 == 0 ? 1 : 0;
    CUtensorMap xmap, wmap, ymap;
    if ((s = make_code_map(&xmap, x, a.M, K, ldx, 128)) != OPQ_OK) return s;
    if ((s = make_code_map(&wmap, w, a.N, K, ldw, C::W_ROWS)) != OPQ_OK) return s;
    if (wa.tma_store) {
        if ((s = make_y_map(&ymap, a)) != OPQ_OK) return s;
    } else {
        ymap = xmap;   // not read by the kernel
    }
    const int64_t tiles = (int64_t)a.m_tiles * a.n_tiles;
    const int64_t groups = tiles < kSMs / CG ? tiles : kSMs / CG;
    return launch(fp8_wide_kernel<CG, BN, DT>, groups * CG, C::THREADS, C::SMEM, CG, stream, xmap, wmap, ymap, wa);
}

struct Fp8Plan {
    int cg, bn;  // wide tiles: 128 cg rows of x x bn rows of W (bn 0: narrow tiles)
    int bx;      // narrow tiles: rows of x
    int split;   // narrow tiles: CTAs (a cluster) that share a tile's blocks
};

// The schedule, from the shape alone. Narrow tiles (64 rows of x or fewer, a tile's blocks shared by
// a cluster) fit when the product is a stream of W or has few tiles; wide ones when it is bound by
// the tensor cores. Above 32 rows of x, or where narrow tiles take several rounds, the choice is by
// the time each would take, from these rates (ns, measured at 3840 to 10240 columns with every SM busy):
//   narrow             per round of 296 CTAs 6000 + 760 per block of the longest range (440 for 16
//                      rows, 680 for 32)
//   128 x 128, 1 CTA   2500 + per round of 148 tiles ( 500 + 345 per block)
//   128 x 256, 1 CTA   2500 + per round of 148 tiles (1500 + 500 per block)
//   256 x 256, a pair  2500 + per round of  74 tiles (1300 + 490 per block)
// They give, in us (measured, for the tiles taken): 256 x 1024 x 3840 narrow 9.0 (9.2), 128 x 128 13.4;
// 256 x 3840 x 3840 narrow 17.4, 128 x 128 13.4 (13.3); 1089 x 3840 x 3840 128 x 256 19.0 (18.3), 128 x 128
// 24.2, pairs 34.5; 4096 x 10240 x 3840 pairs 146.5 (137 to 146), 128 x 256 151.
Fp8Plan make_fp8_plan(int64_t M, int64_t N, int64_t K) {
    const int64_t kblocks = (K + kBlock - 1) / kBlock;
    auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    Fp8Plan p{};
    p.bx = M <= 16 ? 16 : M <= 32 ? 32 : 64;
    // two CTAs per SM: as many ranges as fill them, of two blocks or more
    const int64_t tiles = up(N, 128) * up(M, p.bx);
    int64_t s = 2 * kSMs / tiles;
    if (s > 8) s = 8;
    if (s > kblocks / 2) s = kblocks / 2;
    if (s < 1) s = 1;
    p.split = (int)s;
    const int64_t rounds = up(tiles * s, 2 * kSMs);
    if (M <= 32 && rounds == 1) return p;
    int64_t best = rounds * (6000 + (p.bx == 16 ? 440 : p.bx == 32 ? 680 : 760) * up(kblocks, s));
    auto offer = [&](int cg, int bn, int64_t tile_ns, int64_t block_ns) {
        const int64_t rounds = up(up(M, 128 * cg) * up(N, bn), kSMs / cg);
        const int64_t ns = 2500 + rounds * (tile_ns + block_ns * kblocks);
        if (ns < best) {
            best = ns;
            p.cg = cg;
            p.bn = bn;
        }
    };
    offer(1, 128, 500, 345);
    offer(1, 256, 1500, 500);
    offer(2, 256, 1300, 490);
    return p;
}

bool product_sizes_ok(int64_t M, int64_t N, int64_t K) {
    return K % 32 == 0 && K <= INT32_MAX - 128 && M <= INT32_MAX - 256 && N <= INT32_MAX - 256;
}

template <int DT>
opq_status run_linear(LinearArgs a, const void *x, int64_t ldx, const void *w, int64_t ldw, int64_t K, void *stream) {
    const Fp8Plan p = make_fp8_plan(a.M, a.N, K);
    if (p.bn) {
        a.n_tiles = (a.N + p.bn - 1) / p.bn;
        a.m_tiles = (a.M + 128 * p.cg - 1) / (128 * p.cg);
        if ((int64_t)a.m_tiles * a.n_tiles > INT32_MAX - 256) return OPQ_ERR_UNSUPPORTED_SHAPE;
        if (p.bn == 256)
            return p.cg == 2 ? launch_wide<2, 256, DT>(a, x, ldx, w, ldw, K, stream)
                             : launch_wide<1, 256, DT>(a, x, ldx, w, ldw, K, stream);
        return launch_wide<1, 128, DT>(a, x, ldx, w, ldw, K, stream);
    }
    a.n_tiles = (a.N + 127) / 128;
    a.m_tiles = (a.M + p.bx - 1) / p.bx;
    switch (p.bx) {
        case 16: return launch_narrow<16, DT>(a, p.split, x, ldx, w, ldw, K, stream);
        case 32: return launch_narrow<32, DT>(a, p.split, x, ldx, w, ldw, K, stream);
        default: return launch_narrow<64, DT>(a, p.split, x, ldx, w, ldw, K, stream);
    }
}

// one side of a cache and its rows
opq_status check_side(const opq_fp8_cache &c, const opq_rows &r, int64_t heads) {
    if (c.head_dim < 1) return OPQ_ERR_INVALID_ARG;
    if (c.head_dim % 16 != 0 || c.head_dim > 65536 || heads * c.head_dim > INT32_MAX) return OPQ_ERR_UNSUPPORTED_SHAPE;
    if (c.page_stride < 0 || c.token_stride < 0 || c.head_stride < 0 || c.scale_page_stride < 0 ||
        c.scale_token_stride < 0 || c.scale_head_stride < 0 || r.token_stride < 0 || r.head_stride < 0)
        return OPQ_ERR_INVALID_ARG;
    if (c.page_stride % 16 != 0 || c.token_stride % 16 != 0 || c.head_stride % 16 != 0 || r.token_stride % 8 != 0 ||
        r.head_stride % 8 != 0)
        return OPQ_ERR_MISALIGNED;
    return OPQ_OK;
}

// Whether elements written through these strides can share memory: `inner` contiguous ones at every
// combination of the dimensions' offsets. Each dimension, in the order of their strides, must step
// past all that the smaller ones span (a layout that interleaves them otherwise is refused too).
bool overlapping(int64_t inner, std::initializer_list<std::pair<int64_t, int64_t>> size_stride) {
    std::pair<int64_t, int64_t> d[3];
    int n = 0;
    for (const auto &s : size_stride)
        if (s.first > 1) d[n++] = {s.second, s.first - 1};
    std::sort(d, d + n);
    __int128 span = inner;      // elements from the first to behind the last
    for (int i = 0; i < n; ++i) {
        if (d[i].first < span) return true;
        span += (__int128)d[i].first * d[i].second;
    }
    return false;
}
bool overlapping(const opq_fp8_cache &c, int64_t pages, int64_t page_size, int64_t heads) {
    return overlapping(c.head_dim, {{pages, c.page_stride}, {page_size, c.token_stride}, {heads, c.head_stride}}) ||
           overlapping((c.head_dim + kBlock - 1) / kBlock,
                       {{pages, c.scale_page_stride}, {page_size, c.scale_token_stride}, {heads, c.scale_head_stride}});
}

CacheSide make_side(const opq_fp8_cache &c, const opq_rows &r) {
    CacheSide s{};
    s.codes = c.codes;
    s.scales = c.scales;
    s.page_stride = c.page_stride;
    s.token_stride = c.token_stride;
    s.head_stride = c.head_stride;
    s.scale_page_stride = c.scale_page_stride;
    s.scale_token_stride = c.scale_token_stride;
    s.scale_head_stride = c.scale_head_stride;
    s.rows = static_cast<uint8_t *>(r.data);
    s.row_stride = r.token_stride;
    s.row_head_stride = r.head_stride;
    s.dim = (int)c.head_dim;
    s.blocks = (int)((c.head_dim + kBlock - 1) / kBlock);
    return s;
}

// What the two cache calls check alike, before any pointer is looked at by the driver. out_rows: the
// rows that a read writes; below zero, the cache itself is written.
opq_status check_cache(const opq_fp8_cache *cache, const opq_rows *rows, int32_t tensors, int64_t pages,
                       int64_t page_size, int64_t heads, int32_t dtype, int64_t out_rows) {
    if (!cache || !rows || tensors < 1 || tensors > 2 || pages < 1 || page_size < 1 || heads < 1 || !dtype_ok(dtype))
        return OPQ_ERR_INVALID_ARG;
    if (pages > INT32_MAX || page_size > INT32_MAX || heads > INT32_MAX) return OPQ_ERR_UNSUPPORTED_SHAPE;
    for (int i = 0; i < tensors; ++i) {
        opq_status s = check_side(cache[i], rows[i], heads);
        if (s != OPQ_OK) return s;
    }
    for (int i = 0; i < tensors; ++i)
        if (!cache[i].scales || !cache[i].codes || !rows[i].data) return OPQ_ERR_INVALID_ARG;
    for (int i = 0; i < tensors; ++i)
        if (out_rows < 0 ? overlapping(cache[i], pages, page_size, heads)
                         : overlapping(cache[i].head_dim, {{out_rows, rows[i].token_stride}, {heads, rows[i].head_stride}}))
            return OPQ_ERR_INVALID_ARG;
    for (int i = 0; i < tensors; ++i)
        if (!aligned4(cache[i].scales)) return OPQ_ERR_MISALIGNED;
    for (int i = 0; i < tensors; ++i) {
        opq_status s = check_ptrs({cache[i].codes, rows[i].data});
        if (s == OPQ_OK) s = check_device({cache[i].scales});
        if (s != OPQ_OK) return s;
    }
    return OPQ_OK;
}

template <int DT, int LANES>
opq_status run_write(WriteArgs a, void *stream) {
    // The CTA's lane groups take `pass` columns of as many tokens as fit at a time. Short calls take
    // one such round per CTA (latency: the work spreads over more SMs). Long ones keep four loads in
    // flight per thread and walk enough rounds that one wave of CTAs, four per SM, does it all: a
    // round's loads leave before the last one's codes are stored, which only works within a CTA
    // (16383 tokens of 8 x 128: 20.4 us; one round per CTA 25.1).
    const int groups = kWriteThreads / LANES;
    a.pass = a.cols < groups ? a.cols : groups;
    a.pass_div = FastDiv::make((uint32_t)a.pass);
    const int step = groups / a.pass;
    const bool longer = a.tokens > (int64_t)step * 2 * kSMs;
    int64_t tb = step;
    if (longer) tb = ((a.tokens + 4 * kSMs - 1) / (4 * kSMs) + 4 * step - 1) / (4 * step) * (4 * step);
    a.token_block = (int)(tb < kWriteTokens ? tb : kWriteTokens);
    const int64_t grid = (a.tokens + a.token_block - 1) / a.token_block;
    return longer ? launch(fp8_cache_write_kernel<DT, LANES, 4>, grid, kWriteThreads, 0, 1, stream, a)
                  : launch(fp8_cache_write_kernel<DT, LANES, 1>, grid, kWriteThreads, 0, 1, stream, a);
}

}  // namespace

extern "C" {

opq_status opq_fp8_quantize(const void *x, int32_t dtype, int64_t R, int64_t K, int64_t ldx, int64_t block_rows,
                            uint8_t *codes, int64_t ldc, float *scales, int64_t lds, void *stream) {
    if (R < 1 || K < 1 || !dtype_ok(dtype) || (block_rows != 1 && block_rows != 128)) return OPQ_ERR_INVALID_ARG;
    if (K % 32 != 0 || K > INT32_MAX || R > INT32_MAX) return OPQ_ERR_UNSUPPORTED_SHAPE;
    const int64_t srows = (R + block_rows - 1) / block_rows;
    if (ldx < K || ldx % 8 != 0 || ldc < K || ldc % 16 != 0 || lds < srows) return OPQ_ERR_INVALID_ARG;
    if (!scales) return OPQ_ERR_INVALID_ARG;
    if (!aligned4(scales)) return OPQ_ERR_MISALIGNED;
    opq_status s = check_ptrs({x, codes});
    if (s == OPQ_OK) s = check_device({scales});
    if (s != OPQ_OK) return s;
    QuantArgs a{};
    a.x = static_cast<const uint8_t *>(x);
    a.codes = codes;
    a.scales = scales;
    a.ldx = ldx;
    a.ldc = ldc;
    a.lds = lds;
    a.R = R;
    a.K = (int)K;
    const int64_t kb = (K + kBlock - 1) / kBlock;
    if (block_rows == 1) {
        a.kgroups = (int)((kb + 3) / 4);
        a.tiles = (R + kRowTile - 1) / kRowTile * a.kgroups;
        const int64_t grid = a.tiles < 4 * kSMs ? a.tiles : 4 * kSMs;
        return dtype == OPQ_DTYPE_BF16
                   ? launch(fp8_quantize_rows_kernel<DT_BF16>, grid, kQuantThreads, 0, 1, stream, a)
                   : launch(fp8_quantize_rows_kernel<DT_FP16>, grid, kQuantThreads, 0, 1, stream, a);
    }
    a.kgroups = (int)kb;
    const int64_t grid = srows * kb;
    return dtype == OPQ_DTYPE_BF16 ? launch(fp8_quantize_blocks_kernel<DT_BF16>, grid, kQuantThreads, 0, 1, stream, a)
                                   : launch(fp8_quantize_blocks_kernel<DT_FP16>, grid, kQuantThreads, 0, 1, stream, a);
}

opq_status opq_fp8_linear(const uint8_t *x, int64_t ldx, const float *x_scales, int64_t ld_xs, int64_t M, int64_t K,
                          const uint8_t *w, int64_t ldw, const float *w_scales, int64_t ld_ws, int64_t N,
                          const void *bias, int32_t activation, void *y, int32_t dtype, int64_t ldy, void *stream) {
    if (M < 1 || N < 1 || K < 1 || !dtype_ok(dtype)) return OPQ_ERR_INVALID_ARG;
    if (activation != OPQ_ACT_NONE && activation != OPQ_ACT_SILU && activation != OPQ_ACT_GELU_TANH)
        return OPQ_ERR_INVALID_ARG;
    if (!product_sizes_ok(M, N, K)) return OPQ_ERR_UNSUPPORTED_SHAPE;
    if (ldx < K || ldx % 16 != 0 || ldw < K || ldw % 16 != 0 || ldy < N || ld_xs < M || ld_ws < (N + 127) / 128)
        return OPQ_ERR_INVALID_ARG;
    if (!x_scales || !w_scales) return OPQ_ERR_INVALID_ARG;
    if (!aligned4(x_scales) || !aligned4(w_scales)) return OPQ_ERR_MISALIGNED;
    opq_status s = check_ptrs({x, w, y});
    if (s == OPQ_OK) s = check_device({x_scales, w_scales});
    if (s == OPQ_OK && bias) s = check_ptrs({bias});
    if (s != OPQ_OK) return s;
    LinearArgs a{};
    a.xs = x_scales;
    a.ws = w_scales;
    a.bias = static_cast<const uint16_t *>(bias);
    a.y = static_cast<uint16_t *>(y);
    a.x = x;
    a.w = w;
    a.ldx = ldx;
    a.ldw = ldw;
    a.ld_xs = ld_xs;
    a.ld_ws = ld_ws;
    a.ldy = ldy;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.kblocks = (int)((K + kBlock - 1) / kBlock);
    a.act = activation;
    return dtype == OPQ_DTYPE_BF16 ? run_linear<DT_BF16>(a, x, ldx, w, ldw, K, stream)
                                   : run_linear<DT_FP16>(a, x, ldx, w, ldw, K, stream);
}

opq_status opq_fp8_linear_plan(int64_t M, int64_t N, int64_t K, int *rows, int *cols, int *ctas) {
    if (M < 1 || N < 1 || K < 1) return OPQ_ERR_INVALID_ARG;
    if (!product_sizes_ok(M, N, K)) return OPQ_ERR_UNSUPPORTED_SHAPE;
    const Fp8Plan p = make_fp8_plan(M, N, K);
    if (rows) *rows = p.bn ? 128 * p.cg : p.bx;
    if (cols) *cols = p.bn ? p.bn : 128;
    if (ctas) *ctas = p.bn ? p.cg : p.split;
    return OPQ_OK;
}

opq_status opq_fp8_cache_write(const opq_fp8_cache *cache, const opq_rows *rows, int32_t tensors, int64_t pages,
                               int64_t page_size, int64_t heads, int32_t dtype, int64_t tokens, const int64_t *slots,
                               void *stream) {
    if (tokens < 0) return OPQ_ERR_INVALID_ARG;
    if (tokens == 0) return OPQ_OK;
    if (!slots) return OPQ_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(slots) & 7u) != 0) return OPQ_ERR_MISALIGNED;
    opq_status s = check_cache(cache, rows, tensors, pages, page_size, heads, dtype, -1);
    if (s == OPQ_OK) s = check_device({slots});
    if (s != OPQ_OK) return s;
    WriteArgs a{};
    int64_t cols[2] = {0, 0};
    bool narrow = true;   // eight lanes hold a whole block of up to 64 channels
    for (int i = 0; i < tensors; ++i) {
        a.side[i] = make_side(cache[i], rows[i]);
        cols[i] = heads * a.side[i].blocks;
        a.blocks[i] = FastDiv::make((uint32_t)a.side[i].blocks);
        if (a.side[i].dim > 64) narrow = false;
    }
    if (tensors == 1) a.blocks[1] = a.blocks[0];
    if (cols[0] + cols[1] > INT32_MAX - 4096 || tokens > INT32_MAX) return OPQ_ERR_UNSUPPORTED_SHAPE;
    a.slots = slots;
    a.slot_count = pages * page_size;
    a.page_size = page_size;
    a.tokens = tokens;
    a.cols0 = (int)cols[0];
    a.cols = (int)(cols[0] + cols[1]);
    a.page_div = FastDiv::make((uint32_t)page_size);
    if (dtype == OPQ_DTYPE_BF16)
        return narrow ? run_write<DT_BF16, 8>(a, stream) : run_write<DT_BF16, 16>(a, stream);
    return narrow ? run_write<DT_FP16, 8>(a, stream) : run_write<DT_FP16, 16>(a, stream);
}

opq_status opq_fp8_cache_read(const opq_fp8_cache *cache, const opq_rows *rows, int32_t tensors, int64_t pages,
                              int64_t page_size, int64_t heads, int32_t dtype, int64_t row_count,
                              const int32_t *cu_rows, int64_t seqs, const int32_t *page_table, int64_t ld_table,
                              int64_t table_width, const int32_t *starts, void *stream) {
    if (row_count < 0 || seqs < 0) return OPQ_ERR_INVALID_ARG;
    if (row_count == 0 || seqs == 0) return OPQ_OK;
    if (seqs > INT32_MAX - 1 || row_count > INT32_MAX) return OPQ_ERR_UNSUPPORTED_SHAPE;
    if (!cu_rows || !page_table || table_width < 1 || ld_table < table_width) return OPQ_ERR_INVALID_ARG;
    if (!aligned4(cu_rows) || !aligned4(page_table) || !aligned4(starts)) return OPQ_ERR_MISALIGNED;
    opq_status s = check_cache(cache, rows, tensors, pages, page_size, heads, dtype, row_count);
    if (s == OPQ_OK) s = check_device({cu_rows, page_table});
    if (s == OPQ_OK && starts) s = check_device({starts});
    if (s != OPQ_OK) return s;
    ReadArgs a{};
    int64_t cols[2] = {0, 0};
    for (int i = 0; i < tensors; ++i) {
        a.side[i] = make_side(cache[i], rows[i]);
        cols[i] = heads * (cache[i].head_dim / 8);
        a.head_chunks[i] = FastDiv::make((uint32_t)(cache[i].head_dim / 8));
    }
    if (tensors == 1) a.head_chunks[1] = a.head_chunks[0];
    if (cols[0] + cols[1] > INT32_MAX / 64) return OPQ_ERR_UNSUPPORTED_SHAPE;
    a.cols0 = (int)cols[0];
    a.cols = (int)(cols[0] + cols[1]);
    a.pass = a.cols < kReadThreads ? a.cols : kReadThreads;
    a.pass_div = FastDiv::make((uint32_t)a.pass);
    a.page_div = FastDiv::make((uint32_t)page_size);
    a.cu_rows = cu_rows;
    a.page_table = page_table;
    a.starts = starts;
    a.ld_table = ld_table;
    a.table_width = table_width;
    a.pages = pages;
    a.page_size = page_size;
    a.rows = row_count;
    a.seqs = (int)seqs;
    // a CTA that finds its rows' slots waits for memory twice before its first load, so it takes
    // several rows; four waves of CTAs cover one another's waits better than one long one (25537
    // rows of 2 x 8 x 128: 30.5 us against 32.3)
    const int64_t rb = (row_count + 16 * kSMs - 1) / (16 * kSMs);
    a.row_block = (int)(rb < 1 ? 1 : rb > kReadRows ? kReadRows : rb);
    const int64_t grid = (row_count + a.row_block - 1) / a.row_block;
    return dtype == OPQ_DTYPE_BF16 ? launch(fp8_cache_read_kernel<DT_BF16, 8>, grid, kReadThreads, 0, 1, stream, a)
                                   : launch(fp8_cache_read_kernel<DT_FP16, 8>, grid, kReadThreads, 0, 1, stream, a);
}

}  // extern "C"
