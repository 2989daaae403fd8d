// C ABI of libbq.so: argument checks (all before any CUDA call) and kernel dispatch.
// The operations and conventions are specified in include/bq.h.
#include <atomic>
#include <cstdint>
#include <mutex>

#include "bq.h"
#include "bq_launch.h"
#include "bq_launch_cache.h"

#ifndef BQ_DEBUG
#define BQ_DEBUG 0
#endif

static_assert(BQ_BF16 == bqk::kBf16 && BQ_F16 == bqk::kF16 && BQ_F32 == bqk::kF32, "row types");
static_assert(BQ_MAX_EXPERTS == bqk::kMaxExperts && BQ_SORT_PARTS == bqk::kSortParts, "expert limits");

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};

Range span(const void *p, int64_t bytes)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{lo, lo + static_cast<uintptr_t>(bytes)};
}

// Bounding interval of a row-major strided region: rows of `row_bytes`, `ld_bytes` apart.
Range span2d(const void *p, int64_t rows, int64_t row_bytes, int64_t ld_bytes)
{
    return span(p, (rows - 1) * ld_bytes + row_bytes);
}

bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

// Outputs must be disjoint from each other and from every input.
bool any_alias(const Range *outs, int n_out, const Range *ins, int n_in)
{
    for (int i = 0; i < n_out; i++) {
        for (int j = i + 1; j < n_out; j++)
            if (overlap(outs[i], outs[j])) return true;
        for (int j = 0; j < n_in; j++)
            if (overlap(outs[i], ins[j])) return true;
    }
    return false;
}

bq_status from_cuda(cudaError_t e) { return e == cudaSuccess ? BQ_OK : BQ_ERR_CUDA; }

}  // namespace

// ------------------------------------------------------------------ launch sizing
namespace bqk {

namespace {
constexpr int kMaxDevices = 64;
std::atomic<int> g_sms[kMaxDevices];

struct Runtime {
    cudaError_t limit(const void *kernel, size_t *bytes)
    {
        cudaFuncAttributes attr;
        if (cudaError_t e = cudaFuncGetAttributes(&attr, kernel)) return e;
        *bytes = static_cast<size_t>(attr.maxDynamicSharedSizeBytes);
        return cudaSuccess;
    }
    cudaError_t raise_limit(const void *kernel, size_t bytes)
    {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    }
    cudaError_t ctas_per_sm(const void *kernel, int block, size_t smem, int *ctas)
    {
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(ctas, kernel, block, smem);
    }
};
LaunchCache<Runtime> g_launches;
}  // namespace

namespace {
cudaError_t sm_count_of(int dev, int *sms)
{
    *sms = (dev >= 0 && dev < kMaxDevices) ? g_sms[dev].load(std::memory_order_relaxed) : 0;
    if (*sms == 0) {
        if (cudaError_t e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev)) return e;
        if (dev >= 0 && dev < kMaxDevices) g_sms[dev].store(*sms, std::memory_order_relaxed);
    }
    return cudaSuccess;
}
}  // namespace

cudaError_t sm_count(int *sms)
{
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    return sm_count_of(dev, sms);
}

cudaError_t grid_for(const void *kernel, int64_t nchunk, int *grid, size_t smem, int block)
{
    int dev = 0, sms = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    if (cudaError_t e = sm_count_of(dev, &sms)) return e;
    int occ = 0;
    Runtime rt;
    if (int e = g_launches.ctas_per_sm(rt, kernel, smem, block, dev, &occ)) return static_cast<cudaError_t>(e);
    const int64_t warps_per_cta = block / 32;
    const int64_t need = (nchunk + warps_per_cta - 1) / warps_per_cta;
    const int64_t full = static_cast<int64_t>(sms) * occ;
    *grid = static_cast<int>(need < full ? (need > 0 ? need : 1) : full);
    return cudaSuccess;
}

}  // namespace bqk

// ------------------------------------------------------------------ C ABI
extern "C" {

int bq_abi_version(void) { return BQ_ABI_VERSION; }

const char *bq_status_string(int status)
{
    switch (status) {
    case BQ_OK: return "ok";
    case BQ_ERR_NULL: return "a required pointer is NULL";
    case BQ_ERR_SHAPE: return "size not a multiple of 128, negative, W out of range, or leading dimension too small";
    case BQ_ERR_ALIGN: return "pointer or leading dimension breaks the alignment rules";
    case BQ_ERR_ALIAS: return "an output overlaps an input or another output";
    case BQ_ERR_CUDA: return "the CUDA runtime reported an error for the launch";
    case BQ_ERR_UNSUPPORTED: return "the call needs the debug build (BQ_DEBUG=1)";
    default: return "unknown status";
    }
}

int64_t bq_wire_bytes(int64_t n)
{
    if (n < 0 || n % BQ_BLOCK_I8) return -1;
    return n + 4 * (n / BQ_BLOCK_I8);
}

bq_status bq_quant_i8(const void *x_bf16, int64_t n, int8_t *q, float *scales, cudaStream_t stream)
{
    if (n < 0 || n % BQ_BLOCK_I8) return BQ_ERR_SHAPE;
    if (n == 0) return BQ_OK;
    if (!x_bf16 || !q || !scales) return BQ_ERR_NULL;
    if (!aligned(x_bf16, 16) || !aligned(q, 16) || !aligned(scales, 4)) return BQ_ERR_ALIGN;
    const int64_t nblk = n / BQ_BLOCK_I8;
    const Range ins[] = {span(x_bf16, 2 * n)};
    const Range outs[] = {span(q, n), span(scales, 4 * nblk)};
    if (any_alias(outs, 2, ins, 1)) return BQ_ERR_ALIAS;
    return from_cuda(bqk::launch_quant_i8(static_cast<const uint16_t *>(x_bf16), nblk, q, scales, stream));
}

bq_status bq_dequant_i8(const int8_t *q, const float *scales, int64_t n, void *out_bf16, cudaStream_t stream)
{
    if (n < 0 || n % BQ_BLOCK_I8) return BQ_ERR_SHAPE;
    if (n == 0) return BQ_OK;
    if (!q || !scales || !out_bf16) return BQ_ERR_NULL;
    if (!aligned(q, 16) || !aligned(scales, 4) || !aligned(out_bf16, 16)) return BQ_ERR_ALIGN;
    const int64_t nblk = n / BQ_BLOCK_I8;
    const Range ins[] = {span(q, n), span(scales, 4 * nblk)};
    const Range outs[] = {span(out_bf16, 2 * n)};
    if (any_alias(outs, 1, ins, 2)) return BQ_ERR_ALIAS;
    return from_cuda(bqk::launch_dequant_i8(q, scales, nblk, static_cast<uint16_t *>(out_bf16), stream));
}

bq_status bq_dequant_accum_i8(const int8_t *const *q_srcs, const float *const *scale_srcs, int W, int64_t n,
                              int8_t *q_out, float *scales_out, void *out_bf16, cudaStream_t stream)
{
    if (W < 1 || W > BQ_MAX_W) return BQ_ERR_SHAPE;
    if (n < 0 || n % BQ_BLOCK_I8) return BQ_ERR_SHAPE;
    if (n == 0) return BQ_OK;
    if (!q_srcs || !scale_srcs || !q_out || !scales_out) return BQ_ERR_NULL;
    const int64_t nblk = n / BQ_BLOCK_I8;
    bqk::SourceList src = {};
    Range ins[2 * BQ_MAX_W];
    for (int w = 0; w < W; w++) {
        if (!q_srcs[w] || !scale_srcs[w]) return BQ_ERR_NULL;
        if (!aligned(q_srcs[w], 16) || !aligned(scale_srcs[w], 4)) return BQ_ERR_ALIGN;
        src.q[w] = q_srcs[w];
        src.s[w] = scale_srcs[w];
        ins[2 * w] = span(q_srcs[w], n);
        ins[2 * w + 1] = span(scale_srcs[w], 4 * nblk);
    }
    if (!aligned(q_out, 16) || !aligned(scales_out, 4) || (out_bf16 && !aligned(out_bf16, 16))) return BQ_ERR_ALIGN;
    Range outs[3] = {span(q_out, n), span(scales_out, 4 * nblk), {}};
    int n_out = 2;
    if (out_bf16) outs[n_out++] = span(out_bf16, 2 * n);
    if (any_alias(outs, n_out, ins, 2 * W)) return BQ_ERR_ALIAS;
    return from_cuda(
        bqk::launch_accum_i8(src, W, nblk, q_out, scales_out, static_cast<uint16_t *>(out_bf16), stream));
}

bq_status bq_ring_hop_i8(const int8_t *q_in, const float *s_in, const void *x_local_bf16, int64_t n, int8_t *q_out,
                         float *s_out, void *out_bf16, cudaStream_t stream)
{
    if (n < 0 || n % BQ_BLOCK_I8) return BQ_ERR_SHAPE;
    if (n == 0) return BQ_OK;
    if (!q_in || !s_in || !x_local_bf16 || !q_out || !s_out) return BQ_ERR_NULL;
    if (!aligned(q_in, 16) || !aligned(s_in, 4) || !aligned(x_local_bf16, 16) || !aligned(q_out, 16) ||
        !aligned(s_out, 4) || (out_bf16 && !aligned(out_bf16, 16)))
        return BQ_ERR_ALIGN;
    const int64_t nblk = n / BQ_BLOCK_I8;
    const Range ins[] = {span(q_in, n), span(s_in, 4 * nblk), span(x_local_bf16, 2 * n)};
    Range outs[3] = {span(q_out, n), span(s_out, 4 * nblk), {}};
    int n_out = 2;
    if (out_bf16) outs[n_out++] = span(out_bf16, 2 * n);
    if (any_alias(outs, n_out, ins, 3)) return BQ_ERR_ALIAS;
    return from_cuda(bqk::launch_ring_hop_i8(q_in, s_in, static_cast<const uint16_t *>(x_local_bf16), nblk, q_out,
                                             s_out, static_cast<uint16_t *>(out_bf16), stream));
}

bq_status bq_quant_mx(const void *x_bf16, int64_t rows, int64_t cols, int64_t ld_x, uint8_t *q_e4m3, int64_t ld_q,
                      uint8_t *s_e8m0, int64_t ld_s, cudaStream_t stream)
{
    if (rows < 0 || cols < 0 || cols % 128) return BQ_ERR_SHAPE;
    if (rows == 0 || cols == 0) return BQ_OK;
    if (ld_x < cols || ld_q < cols || ld_s < cols / BQ_GROUP_MX) return BQ_ERR_SHAPE;
    if (!x_bf16 || !q_e4m3 || !s_e8m0) return BQ_ERR_NULL;
    if (!aligned(x_bf16, 16) || ld_x % 8 || !aligned(q_e4m3, 16) || ld_q % 16 || !aligned(s_e8m0, 4) || ld_s % 4)
        return BQ_ERR_ALIGN;
    const Range ins[] = {span2d(x_bf16, rows, 2 * cols, 2 * ld_x)};
    const Range outs[] = {span2d(q_e4m3, rows, cols, ld_q), span2d(s_e8m0, rows, cols / BQ_GROUP_MX, ld_s)};
    if (any_alias(outs, 2, ins, 1)) return BQ_ERR_ALIAS;
    return from_cuda(bqk::launch_quant_mx(static_cast<const uint16_t *>(x_bf16), ld_x, rows, cols, q_e4m3, ld_q,
                                          s_e8m0, ld_s, stream));
}

bq_status bq_dequant_mx(const uint8_t *q_e4m3, int64_t ld_q, const uint8_t *s_e8m0, int64_t ld_s, int64_t rows,
                        int64_t cols, void *out_bf16, int64_t ld_out, cudaStream_t stream)
{
    if (rows < 0 || cols < 0 || cols % 128) return BQ_ERR_SHAPE;
    if (rows == 0 || cols == 0) return BQ_OK;
    if (ld_q < cols || ld_s < cols / BQ_GROUP_MX || ld_out < cols) return BQ_ERR_SHAPE;
    if (!q_e4m3 || !s_e8m0 || !out_bf16) return BQ_ERR_NULL;
    if (!aligned(q_e4m3, 16) || ld_q % 16 || !aligned(s_e8m0, 4) || ld_s % 4 || !aligned(out_bf16, 16) || ld_out % 8)
        return BQ_ERR_ALIGN;
    const Range ins[] = {span2d(q_e4m3, rows, cols, ld_q), span2d(s_e8m0, rows, cols / BQ_GROUP_MX, ld_s)};
    const Range outs[] = {span2d(out_bf16, rows, 2 * cols, 2 * ld_out)};
    if (any_alias(outs, 1, ins, 2)) return BQ_ERR_ALIAS;
    return from_cuda(bqk::launch_dequant_mx(q_e4m3, ld_q, s_e8m0, ld_s, rows, cols, static_cast<uint16_t *>(out_bf16),
                                            ld_out, stream));
}

bq_status bq_dequant_accum_mx(const uint8_t *const *q_srcs, const uint8_t *const *s_srcs, int W, int64_t n,
                              uint8_t *q_out, uint8_t *s_out, void *out_bf16, cudaStream_t stream)
{
    if (W < 1 || W > BQ_MAX_W) return BQ_ERR_SHAPE;
    if (n < 0 || n % BQ_BLOCK_I8) return BQ_ERR_SHAPE;
    if (n == 0) return BQ_OK;
    if (!q_srcs || !s_srcs || !q_out || !s_out) return BQ_ERR_NULL;
    const int64_t nblk = n / BQ_BLOCK_I8;
    bqk::MxSourceList src = {};
    Range ins[2 * BQ_MAX_W];
    for (int w = 0; w < W; w++) {
        if (!q_srcs[w] || !s_srcs[w]) return BQ_ERR_NULL;
        if (!aligned(q_srcs[w], 16) || !aligned(s_srcs[w], 4)) return BQ_ERR_ALIGN;
        src.q[w] = q_srcs[w];
        src.s[w] = reinterpret_cast<const uint32_t *>(s_srcs[w]);
        ins[2 * w] = span(q_srcs[w], n);
        ins[2 * w + 1] = span(s_srcs[w], 4 * nblk);
    }
    if (!aligned(q_out, 16) || !aligned(s_out, 4) || (out_bf16 && !aligned(out_bf16, 16))) return BQ_ERR_ALIGN;
    Range outs[3] = {span(q_out, n), span(s_out, 4 * nblk), {}};
    int n_out = 2;
    if (out_bf16) outs[n_out++] = span(out_bf16, 2 * n);
    if (any_alias(outs, n_out, ins, 2 * W)) return BQ_ERR_ALIAS;
    return from_cuda(bqk::launch_accum_mx(src, W, nblk, q_out, reinterpret_cast<uint32_t *>(s_out),
                                          static_cast<uint16_t *>(out_bf16), stream));
}

bq_status bq_ring_hop_mx(const uint8_t *q_in, const uint8_t *s_in, const void *x_local_bf16, int64_t n,
                         uint8_t *q_out, uint8_t *s_out, void *out_bf16, cudaStream_t stream)
{
    if (n < 0 || n % BQ_BLOCK_I8) return BQ_ERR_SHAPE;
    if (n == 0) return BQ_OK;
    if (!q_in || !s_in || !x_local_bf16 || !q_out || !s_out) return BQ_ERR_NULL;
    if (!aligned(q_in, 16) || !aligned(s_in, 4) || !aligned(x_local_bf16, 16) || !aligned(q_out, 16) ||
        !aligned(s_out, 4) || (out_bf16 && !aligned(out_bf16, 16)))
        return BQ_ERR_ALIGN;
    const int64_t nblk = n / BQ_BLOCK_I8;
    const Range ins[] = {span(q_in, n), span(s_in, 4 * nblk), span(x_local_bf16, 2 * n)};
    Range outs[3] = {span(q_out, n), span(s_out, 4 * nblk), {}};
    int n_out = 2;
    if (out_bf16) outs[n_out++] = span(out_bf16, 2 * n);
    if (any_alias(outs, n_out, ins, 3)) return BQ_ERR_ALIAS;
    return from_cuda(bqk::launch_ring_hop_mx(q_in, reinterpret_cast<const uint32_t *>(s_in),
                                             static_cast<const uint16_t *>(x_local_bf16), nblk, q_out,
                                             reinterpret_cast<uint32_t *>(s_out), static_cast<uint16_t *>(out_bf16),
                                             stream));
}

bq_status bq_quant_mx_f16(const void *x_f16, int64_t rows, int64_t cols, int64_t ld_x, uint8_t *q_e4m3, int64_t ld_q,
                          uint8_t *s_e8m0, int64_t ld_s, cudaStream_t stream)
{
    if (rows < 0 || cols < 0 || cols % 128) return BQ_ERR_SHAPE;
    if (rows == 0 || cols == 0) return BQ_OK;
    if (ld_x < cols || ld_q < cols || ld_s < cols / BQ_GROUP_MX) return BQ_ERR_SHAPE;
    if (!x_f16 || !q_e4m3 || !s_e8m0) return BQ_ERR_NULL;
    if (!aligned(x_f16, 16) || ld_x % 8 || !aligned(q_e4m3, 16) || ld_q % 16 || !aligned(s_e8m0, 4) || ld_s % 4)
        return BQ_ERR_ALIGN;
    const Range ins[] = {span2d(x_f16, rows, 2 * cols, 2 * ld_x)};
    const Range outs[] = {span2d(q_e4m3, rows, cols, ld_q), span2d(s_e8m0, rows, cols / BQ_GROUP_MX, ld_s)};
    if (any_alias(outs, 2, ins, 1)) return BQ_ERR_ALIAS;
    return from_cuda(bqk::launch_quant_mx_f16(static_cast<const uint16_t *>(x_f16), ld_x, rows, cols, q_e4m3, ld_q,
                                              s_e8m0, ld_s, stream));
}

bq_status bq_quant_mx_tiled(const void *x, int x_is_f16, int64_t rows, int64_t cols, int64_t ld_x, uint8_t *q_e4m3,
                            int64_t ld_q, uint8_t *s_tiled, int64_t g_total, int64_t g0, cudaStream_t stream)
{
    if (rows < 0 || cols < 0 || cols % 128) return BQ_ERR_SHAPE;
    if (g_total < 0 || g_total % 4 || g0 < 0 || g0 % 4 || g0 + cols / BQ_GROUP_MX > g_total) return BQ_ERR_SHAPE;
    if (rows == 0 || cols == 0) return BQ_OK;
    if (ld_x < cols || ld_q < cols) return BQ_ERR_SHAPE;
    if (!x || !q_e4m3 || !s_tiled) return BQ_ERR_NULL;
    if (!aligned(x, 16) || ld_x % 8 || !aligned(q_e4m3, 16) || ld_q % 16 || !aligned(s_tiled, 4)) return BQ_ERR_ALIGN;
    const int64_t tiled_bytes = ((rows + 127) / 128) * (g_total / 4) * 512;
    const Range ins[] = {span2d(x, rows, 2 * cols, 2 * ld_x)};
    const Range outs[] = {span2d(q_e4m3, rows, cols, ld_q), span(s_tiled, tiled_bytes)};
    if (any_alias(outs, 2, ins, 1)) return BQ_ERR_ALIAS;
    return from_cuda(bqk::launch_quant_mx_tiled(static_cast<const uint16_t *>(x), x_is_f16 != 0, ld_x, rows, cols,
                                                q_e4m3, ld_q, s_tiled, g_total / 4, g0 / 4, stream));
}

bq_status bq_quant_mx_slices(const bq_mx_slice *slices, int nslices, int x_is_f16, int64_t rows, uint8_t *q_e4m3,
                             int64_t ld_q, uint8_t *s_e8m0, int64_t ld_s, cudaStream_t stream)
{
    if (nslices < 1 || nslices > BQ_MAX_SLICES || rows < 0) return BQ_ERR_SHAPE;
    if (!slices) return BQ_ERR_NULL;
    int64_t total = 0;
    for (int i = 0; i < nslices; i++) {
        const int64_t c = slices[i].cols;
        if (c < 0 || c % 128 || slices[i].ld_x < c) return BQ_ERR_SHAPE;
        total += c;
    }
    if (rows == 0 || total == 0) return BQ_OK;
    if (ld_q < total || ld_s < total / BQ_GROUP_MX) return BQ_ERR_SHAPE;
    if (!q_e4m3 || !s_e8m0) return BQ_ERR_NULL;
    if (!aligned(q_e4m3, 16) || ld_q % 16 || !aligned(s_e8m0, 4) || ld_s % 4) return BQ_ERR_ALIGN;
    Range ins[BQ_MAX_SLICES];
    bqk::MxSliceList sl = {};
    int64_t col = 0;
    for (int i = 0; i < nslices; i++) {
        const int64_t c = slices[i].cols;
        if (c == 0) continue;
        if (!slices[i].x) return BQ_ERR_NULL;
        if (!aligned(slices[i].x, 16) || slices[i].ld_x % 8) return BQ_ERR_ALIGN;
        ins[sl.n] = span2d(slices[i].x, rows, 2 * c, 2 * slices[i].ld_x);
        sl.x[sl.n] = static_cast<const uint16_t *>(slices[i].x);
        sl.ld_x[sl.n] = slices[i].ld_x;
        sl.bpr[sl.n] = c / 128;
        sl.cb0[sl.n] = col / 128;
        sl.n++;
        col += c;
    }
    const Range outs[] = {span2d(q_e4m3, rows, total, ld_q), span2d(s_e8m0, rows, total / BQ_GROUP_MX, ld_s)};
    if (any_alias(outs, 2, ins, sl.n)) return BQ_ERR_ALIAS;
    return from_cuda(bqk::launch_quant_mx_slices(sl, x_is_f16 != 0, rows, q_e4m3, ld_q, s_e8m0, ld_s, stream));
}

int64_t bq_mx_tiled_scale_bytes(int64_t rows, int64_t g_total)
{
    if (rows < 0 || g_total < 0 || g_total % 4) return -1;
    return ((rows + 127) / 128) * (g_total / 4) * 512;
}

namespace {
// Shared checks of the reduce + quantize calls: W BF16 sources -> payload [n] (1 byte
// per value, 16-byte aligned), FP32 scales [n/128] (4-byte aligned), optional BF16.
bq_status check_reduce(const void *const *x_srcs, int W, int64_t n, const void *q, const void *scales,
                       const void *out_bf16, bqk::Bf16List *src)
{
    if (W < 1 || W > BQ_MAX_W) return BQ_ERR_SHAPE;
    if (n < 0 || n % BQ_BLOCK_I8) return BQ_ERR_SHAPE;
    if (n == 0) return BQ_OK;
    if (!x_srcs || !q || !scales) return BQ_ERR_NULL;
    Range ins[BQ_MAX_W];
    for (int w = 0; w < W; w++) {
        if (!x_srcs[w]) return BQ_ERR_NULL;
        if (!aligned(x_srcs[w], 16)) return BQ_ERR_ALIGN;
        src->x[w] = static_cast<const uint16_t *>(x_srcs[w]);
        ins[w] = span(x_srcs[w], 2 * n);
    }
    if (!aligned(q, 16) || !aligned(scales, 4) || (out_bf16 && !aligned(out_bf16, 16))) return BQ_ERR_ALIGN;
    Range outs[3] = {span(q, n), span(scales, 4 * (n / BQ_BLOCK_I8)), {}};
    int n_out = 2;
    if (out_bf16) outs[n_out++] = span(out_bf16, 2 * n);
    if (any_alias(outs, n_out, ins, W)) return BQ_ERR_ALIAS;
    return BQ_OK;
}
}  // namespace

bq_status bq_reduce_quant_i8(const void *const *x_srcs, int W, int64_t n, int8_t *q, float *scales, void *out_bf16,
                             cudaStream_t stream)
{
    bqk::Bf16List src = {};
    if (bq_status e = check_reduce(x_srcs, W, n, q, scales, out_bf16, &src)) return e;
    if (n == 0) return BQ_OK;
    return from_cuda(bqk::launch_reduce_quant_i8(src, W, n / BQ_BLOCK_I8, q, scales,
                                                 static_cast<uint16_t *>(out_bf16), stream));
}

bq_status bq_quant_e4m3(const void *x_bf16, int64_t n, uint8_t *q, float *scales, cudaStream_t stream)
{
    if (n < 0 || n % BQ_BLOCK_I8) return BQ_ERR_SHAPE;
    if (n == 0) return BQ_OK;
    if (!x_bf16 || !q || !scales) return BQ_ERR_NULL;
    if (!aligned(x_bf16, 16) || !aligned(q, 16) || !aligned(scales, 4)) return BQ_ERR_ALIGN;
    const int64_t nblk = n / BQ_BLOCK_I8;
    const Range ins[] = {span(x_bf16, 2 * n)};
    const Range outs[] = {span(q, n), span(scales, 4 * nblk)};
    if (any_alias(outs, 2, ins, 1)) return BQ_ERR_ALIAS;
    return from_cuda(bqk::launch_quant_e4m3(static_cast<const uint16_t *>(x_bf16), nblk, q, scales, stream));
}

bq_status bq_dequant_e4m3(const uint8_t *q, const float *scales, int64_t n, void *out_bf16, cudaStream_t stream)
{
    if (n < 0 || n % BQ_BLOCK_I8) return BQ_ERR_SHAPE;
    if (n == 0) return BQ_OK;
    if (!q || !scales || !out_bf16) return BQ_ERR_NULL;
    if (!aligned(q, 16) || !aligned(scales, 4) || !aligned(out_bf16, 16)) return BQ_ERR_ALIGN;
    const int64_t nblk = n / BQ_BLOCK_I8;
    const Range ins[] = {span(q, n), span(scales, 4 * nblk)};
    const Range outs[] = {span(out_bf16, 2 * n)};
    if (any_alias(outs, 1, ins, 2)) return BQ_ERR_ALIAS;
    return from_cuda(bqk::launch_dequant_e4m3(q, scales, nblk, static_cast<uint16_t *>(out_bf16), stream));
}

bq_status bq_reduce_quant_e4m3(const void *const *x_srcs, int W, int64_t n, uint8_t *q, float *scales,
                               void *out_bf16, cudaStream_t stream)
{
    bqk::Bf16List src = {};
    if (bq_status e = check_reduce(x_srcs, W, n, q, scales, out_bf16, &src)) return e;
    if (n == 0) return BQ_OK;
    return from_cuda(bqk::launch_reduce_quant_e4m3(src, W, n / BQ_BLOCK_I8, q, scales,
                                                   static_cast<uint16_t *>(out_bf16), stream));
}

}  // extern "C"

// ------------------------------------------------------------------ expert layer
namespace {
// The row ranges and shape rules that the expert-layer calls share.
bool row_type(int type) { return type == BQ_BF16 || type == BQ_F16 || type == BQ_F32; }

bool plan_shape(int64_t tokens, int top_k)
{
    return tokens >= 0 && top_k >= 1 && top_k <= BQ_MAX_TOP_K && tokens <= INT32_MAX / top_k;
}

// rows x cols values of a row type, ld values apart: shape and alignment
bq_status check_rows(const void *p, int type, int64_t rows, int64_t cols, int64_t ld)
{
    if (rows > 0 && ld < cols) return BQ_ERR_SHAPE;
    if (!p) return BQ_ERR_NULL;
    return aligned(p, bqk::row_type_bytes(type)) ? BQ_OK : BQ_ERR_ALIGN;
}

Range rows_span(const void *p, int type, int64_t rows, int64_t cols, int64_t ld)
{
    const int size = bqk::row_type_bytes(type);
    return span2d(p, rows, size * cols, size * ld);
}
}  // namespace

extern "C" {

bq_status bq_expert_sort(const void *ids, int ids_are_i64, int64_t tokens, int top_k, int n_experts, int32_t *offsets,
                         int32_t *order, int32_t *inverse, int32_t *workspace, cudaStream_t stream)
{
    if (!plan_shape(tokens, top_k) || n_experts < 1 || n_experts > BQ_MAX_EXPERTS) return BQ_ERR_SHAPE;
    const int64_t slots = tokens * top_k, id_bytes = ids_are_i64 ? 8 : 4;
    if (!offsets || !workspace || (slots > 0 && (!ids || !order || !inverse))) return BQ_ERR_NULL;
    if (!aligned(ids, id_bytes) || !aligned(offsets, 4) || !aligned(order, 4) || !aligned(inverse, 4) ||
        !aligned(workspace, 4))
        return BQ_ERR_ALIGN;
    const Range ins[] = {span(ids, id_bytes * slots)};
    const Range outs[] = {span(offsets, 4 * (n_experts + 1)), span(order, 4 * slots), span(inverse, 4 * slots),
                          span(workspace, 4ll * BQ_SORT_PARTS * n_experts)};
    if (any_alias(outs, 4, ins, 1)) return BQ_ERR_ALIAS;
    return from_cuda(
        bqk::launch_expert_sort(ids, ids_are_i64 != 0, slots, n_experts, offsets, order, inverse, workspace, stream));
}

bq_status bq_expert_gather(const void *x, int type, int64_t tokens, int64_t hidden, int64_t ld_x,
                           const int32_t *inverse, int top_k, const int32_t *offsets, int n_experts, void *out,
                           int64_t ld_out, cudaStream_t stream)
{
    if (!row_type(type) || !plan_shape(tokens, top_k) || hidden < 0 || n_experts < 1 || n_experts > BQ_MAX_EXPERTS)
        return BQ_ERR_SHAPE;
    if (tokens == 0 || hidden == 0) return BQ_OK;
    const int64_t slots = tokens * top_k;
    if (bq_status e = check_rows(x, type, tokens, hidden, ld_x)) return e;
    if (bq_status e = check_rows(out, type, slots, hidden, ld_out)) return e;
    if (!inverse || !offsets) return BQ_ERR_NULL;
    if (!aligned(inverse, 4) || !aligned(offsets, 4)) return BQ_ERR_ALIGN;
    const Range ins[] = {rows_span(x, type, tokens, hidden, ld_x), span(inverse, 4 * slots),
                         span(offsets, 4 * (n_experts + 1))};
    const Range outs[] = {rows_span(out, type, slots, hidden, ld_out)};
    if (any_alias(outs, 1, ins, 3)) return BQ_ERR_ALIAS;
    const bqk::RowArgs a = {tokens, hidden, inverse, top_k};
    return from_cuda(bqk::launch_expert_gather(type, a, x, ld_x, offsets, n_experts, out, ld_out, stream));
}

bq_status bq_expert_combine(const void *y, int type, int64_t ld_y, const float *weights, const int32_t *inverse,
                            int64_t tokens, int top_k, int64_t hidden, void *out, int64_t ld_out, cudaStream_t stream)
{
    if (!row_type(type) || !plan_shape(tokens, top_k) || hidden < 0) return BQ_ERR_SHAPE;
    if (tokens == 0 || hidden == 0) return BQ_OK;
    const int64_t slots = tokens * top_k;
    if (bq_status e = check_rows(y, type, slots, hidden, ld_y)) return e;
    if (bq_status e = check_rows(out, type, tokens, hidden, ld_out)) return e;
    if (!inverse) return BQ_ERR_NULL;
    if (!aligned(inverse, 4) || !aligned(weights, 4)) return BQ_ERR_ALIGN;
    const Range ins[] = {rows_span(y, type, slots, hidden, ld_y), span(inverse, 4 * slots),
                         span(weights, weights ? 4 * slots : 0)};
    const Range outs[] = {rows_span(out, type, tokens, hidden, ld_out)};
    if (any_alias(outs, 1, ins, 3)) return BQ_ERR_ALIAS;
    const bqk::RowArgs a = {tokens, hidden, inverse, top_k};
    return from_cuda(bqk::launch_expert_combine(type, a, y, ld_y, weights, out, ld_out, stream));
}

bq_status bq_expert_combine_grad(const void *dout, int type, int64_t ld_dout, const void *y, int64_t ld_y,
                                 const float *weights, const int32_t *inverse, const int32_t *offsets, int n_experts,
                                 int64_t tokens, int top_k, int64_t hidden, void *dy, int64_t ld_dy, float *dweights,
                                 cudaStream_t stream)
{
    if (!row_type(type) || !plan_shape(tokens, top_k) || hidden < 0 || n_experts < 1 || n_experts > BQ_MAX_EXPERTS)
        return BQ_ERR_SHAPE;
    if (tokens == 0) return BQ_OK;
    const int64_t slots = tokens * top_k;
    if (hidden > 0) {  // without columns only dweights is written
        if (bq_status e = check_rows(dout, type, tokens, hidden, ld_dout)) return e;
        if (bq_status e = check_rows(y, type, slots, hidden, ld_y)) return e;
        if (bq_status e = check_rows(dy, type, slots, hidden, ld_dy)) return e;
    }
    if (!weights || !inverse || !offsets || !dweights) return BQ_ERR_NULL;
    if (!aligned(weights, 4) || !aligned(inverse, 4) || !aligned(offsets, 4) || !aligned(dweights, 4))
        return BQ_ERR_ALIGN;
    const bool rows = hidden > 0;
    const Range none = span(dweights, 0);
    const Range ins[] = {rows ? rows_span(dout, type, tokens, hidden, ld_dout) : none,
                         rows ? rows_span(y, type, slots, hidden, ld_y) : none, span(weights, 4 * slots),
                         span(inverse, 4 * slots), span(offsets, 4 * (n_experts + 1))};
    const Range outs[] = {rows ? rows_span(dy, type, slots, hidden, ld_dy) : none, span(dweights, 4 * slots)};
    if (any_alias(outs, 2, ins, 5)) return BQ_ERR_ALIAS;
    const bqk::RowArgs a = {tokens, hidden, inverse, top_k};
    return from_cuda(bqk::launch_expert_combine_grad(type, a, dout, ld_dout, y, ld_y, weights, offsets, n_experts, dy,
                                                     ld_dy, dweights, stream));
}
}  // extern "C"

namespace {
// Shared checks of the 4-bit products, and the launch. x_rows rows of x, slots rows of out.
bq_status matvec_w4(int type, int scale_type, int group, bqk::W4Args &a, cudaStream_t stream)
{
    if ((type != BQ_BF16 && type != BQ_F16) || (scale_type != type && scale_type != BQ_F32)) return BQ_ERR_SHAPE;
    if (group != 32 && group != 64 && group != 128) return BQ_ERR_SHAPE;
    if (a.x_rows < 0 || a.x_rows > INT32_MAX || a.slots < 0 || a.slots > INT32_MAX) return BQ_ERR_SHAPE;
    if (a.n < 0 || a.n > BQ_MAX_W4_DIM || a.k < 0 || a.k > BQ_MAX_W4_DIM || a.k % group) return BQ_ERR_SHAPE;
    if (a.slots == 0 || a.n == 0) return BQ_OK;
    if (a.ld_x < a.k || a.ld_q < a.k / 2 || a.ld_s < a.k / group || a.ld_out < a.n) return BQ_ERR_SHAPE;
    const int64_t q_bytes = (a.n - 1) * a.ld_q + a.k / 2, s_values = (a.n - 1) * a.ld_s + a.k / group;
    if (a.n_experts > 1 && (a.expert_q < q_bytes || a.expert_s < s_values)) return BQ_ERR_SHAPE;
    if (!a.out || (a.k > 0 && (!a.q || !a.s || (a.x_rows > 0 && !a.x)))) return BQ_ERR_NULL;
    if (!aligned(a.out, 2) || !aligned(a.offsets, 4) || !aligned(a.order, 4)) return BQ_ERR_ALIGN;
    if (a.k > 0 && (!aligned(a.x, 16) || a.ld_x % 8 || !aligned(a.q, 16) || a.ld_q % 16 || !aligned(a.s, 4) ||
                    (a.n_experts > 1 && a.expert_q % 16)))
        return BQ_ERR_ALIGN;
    const int s_size = bqk::row_type_bytes(scale_type);
    const Range none = span(a.out, 0);
    const Range ins[] = {
        a.k > 0 && a.x_rows > 0 ? rows_span(a.x, type, a.x_rows, a.k, a.ld_x) : none,
        a.k > 0 ? span(a.q, (a.n_experts - 1) * a.expert_q + q_bytes) : none,
        a.k > 0 ? span(a.s, s_size * ((a.n_experts - 1) * a.expert_s + s_values)) : none,
        a.offsets ? span(a.offsets, 4 * (a.n_experts + 1)) : none, a.order ? span(a.order, 4 * a.slots) : none};
    const Range outs[] = {rows_span(a.out, type, a.slots, a.n, a.ld_out)};
    if (any_alias(outs, 1, ins, 5)) return BQ_ERR_ALIAS;
    return from_cuda(bqk::launch_matvec_w4(type, scale_type, group, a, stream));
}
}  // namespace

extern "C" {

bq_status bq_quant_w4(const void *x, int type, int64_t n, int64_t k, int64_t ld_x, int group, uint8_t *q, int64_t ld_q,
                      void *scales, int scale_type, int64_t ld_s, cudaStream_t stream)
{
    if (!row_type(type) || !row_type(scale_type) || (group != 32 && group != 64 && group != 128)) return BQ_ERR_SHAPE;
    if (n < 0 || n > BQ_MAX_W4_DIM || k < 0 || k > BQ_MAX_W4_DIM || k % group) return BQ_ERR_SHAPE;
    if (n == 0 || k == 0) return BQ_OK;
    if (ld_x < k || ld_q < k / 2 || ld_s < k / group) return BQ_ERR_SHAPE;
    if (!x || !q || !scales) return BQ_ERR_NULL;
    const int size = bqk::row_type_bytes(type), s_size = bqk::row_type_bytes(scale_type);
    if (!aligned(x, 16) || ld_x * size % 16 || !aligned(q, 16) || ld_q % 16 || !aligned(scales, 4)) return BQ_ERR_ALIGN;
    const Range ins[] = {rows_span(x, type, n, k, ld_x)};
    const Range outs[] = {span2d(q, n, k / 2, ld_q), span2d(scales, n, s_size * (k / group), s_size * ld_s)};
    if (any_alias(outs, 2, ins, 1)) return BQ_ERR_ALIAS;
    return from_cuda(bqk::launch_quant_w4(type, scale_type, group, x, n, k, ld_x, q, ld_q, scales, ld_s, stream));
}

bq_status bq_matvec_w4(const void *x, int type, int64_t rows, int64_t k, int64_t ld_x, const uint8_t *q, int64_t n,
                       int64_t ld_q, const void *scales, int scale_type, int group, int64_t ld_s, void *out,
                       int64_t ld_out, cudaStream_t stream)
{
    bqk::W4Args a = {};
    a.x = x, a.ld_x = ld_x, a.x_rows = rows, a.slots = rows;
    a.q = q, a.ld_q = ld_q, a.s = scales, a.ld_s = ld_s;
    a.out = out, a.ld_out = ld_out, a.n = n, a.k = k;
    a.n_experts = 1, a.top_k = 1;
    return matvec_w4(type, scale_type, group, a, stream);
}

bq_status bq_matvec_w4_experts(const void *x, int type, int64_t x_rows, int64_t k, int64_t ld_x, const uint8_t *q,
                               int64_t n, int64_t ld_q, int64_t expert_q, const void *scales, int scale_type, int group,
                               int64_t ld_s, int64_t expert_s, const int32_t *offsets, int n_experts,
                               const int32_t *order, int top_k, int64_t slots, void *out, int64_t ld_out,
                               cudaStream_t stream)
{
    if (n_experts < 1 || n_experts > BQ_MAX_EXPERTS || top_k < 1 || top_k > BQ_MAX_TOP_K) return BQ_ERR_SHAPE;
    if (slots > 0 && !offsets) return BQ_ERR_NULL;
    // every place's row exists: a place p takes row order[p] / top_k, or row p
    if (slots > 0 && x_rows < (order ? (slots + top_k - 1) / top_k : slots)) return BQ_ERR_SHAPE;
    bqk::W4Args a = {};
    a.x = x, a.ld_x = ld_x, a.x_rows = x_rows, a.slots = slots;
    a.q = q, a.ld_q = ld_q, a.expert_q = expert_q, a.s = scales, a.ld_s = ld_s, a.expert_s = expert_s;
    a.out = out, a.ld_out = ld_out, a.n = n, a.k = k;
    a.offsets = offsets, a.n_experts = n_experts, a.order = order, a.top_k = top_k;
    return matvec_w4(type, scale_type, group, a, stream);
}

}  // extern "C"

// ------------------------------------------------------------------ key-value cache in 4 bits
namespace {
// Dimensions of rows that lie `stride` bytes apart. True if no two rows of `row` bytes overlap;
// `span` is then the bytes from the first row's start to the last one's end.
struct Dim {
    int64_t n, stride;
};
bool rows_apart(Dim (&d)[3], int64_t row, int64_t *span)
{
    for (int i = 0; i < 2; i++)
        for (int j = 0; j < 2 - i; j++)
            if (d[j].n <= 1 || (d[j + 1].n > 1 && d[j + 1].stride < d[j].stride)) {
                const Dim t = d[j];
                d[j] = d[j + 1];
                d[j + 1] = t;
            }
    *span = row;
    for (const Dim &x : d) {
        if (x.n <= 1) continue;
        if (x.stride < *span || x.stride > INT64_MAX / 4 / x.n) return false;
        *span += (x.n - 1) * x.stride;
        if (*span > INT64_MAX / 4) return false;
    }
    return true;
}

// One of a cache's arrays: where it starts, its bytes, and those of one page.
struct Paged {
    uintptr_t lo;
    int64_t bytes, page_bytes, page_stride;
};

bool disjoint(const Paged &a, const Paged &b)
{
    if (!overlap(Range{a.lo, a.lo + (uintptr_t)a.bytes}, Range{b.lo, b.lo + (uintptr_t)b.bytes})) return true;
    if (a.page_stride != b.page_stride || a.page_stride < a.page_bytes || a.page_stride < b.page_bytes) return false;
    const Paged &first = a.lo < b.lo ? a : b, &second = a.lo < b.lo ? b : a;
    const int64_t at = (int64_t)((second.lo - first.lo) % (uintptr_t)a.page_stride);
    return at >= first.page_bytes && at + second.page_bytes <= a.page_stride;
}

// The checks that every call on a cache shares. Fills c, the spans of the four arrays and whether
// there is a page at all.
bq_status check_cache(const bq_kv4_cache *cache, bqk::Kv4Cache &c, Range (&spans)[4])
{
    if (!cache) return BQ_ERR_NULL;
    const bq_kv4_cache &x = *cache;
    if (x.type != BQ_BF16 && x.type != BQ_F16) return BQ_ERR_SHAPE;
    if (x.head_dim < 64 || x.head_dim > 256 || x.head_dim % 64) return BQ_ERR_SHAPE;
    if ((x.group != 32 && x.group != 64 && x.group != 128) || x.head_dim % x.group) return BQ_ERR_SHAPE;
    if (x.pages < 0 || x.pages > INT32_MAX || x.heads < 1 || x.heads > BQ_KV4_MAX_HEADS) return BQ_ERR_SHAPE;
    if (x.page < 1 || x.page > BQ_KV4_MAX_PAGE) return BQ_ERR_SHAPE;
    const int64_t row = x.head_dim / 2, row_s = 4 * (x.head_dim / x.group);
    const int64_t in_page = x.page > 1 ? (x.page - 1) : 0;
    if (x.page > 1 && (x.token_stride < 0 || x.token_stride > (INT32_MAX - row) / in_page || x.token_stride_s < 0 ||
                       x.token_stride_s > (INT32_MAX - row_s) / in_page))
        return BQ_ERR_SHAPE;
    Paged arrays[4];
    for (int i = 0; i < 2; i++) {  // codes, pairs
        const int64_t ps = i ? x.page_stride_s : x.page_stride, hs = i ? x.head_stride_s : x.head_stride;
        const int64_t ts = i ? x.token_stride_s : x.token_stride;
        const int64_t align = !i ? 16 : row_s % 16 == 0 ? 16 : row_s & -row_s;
        Dim all[3] = {{x.page, ts}, {x.heads, hs}, {x.pages, ps}}, one[3] = {{x.page, ts}, {x.heads, hs}, {1, 0}};
        int64_t bytes = 0, page_bytes = 0;
        if (!rows_apart(one, i ? row_s : row, &page_bytes) || !rows_apart(all, i ? row_s : row, &bytes))
            return BQ_ERR_SHAPE;
        if ((x.page > 1 && ts % align) || (x.heads > 1 && hs % align) || (x.pages > 1 && ps % align)) return BQ_ERR_ALIGN;
        const void *const of[2] = {i ? x.k_scales : x.k, i ? x.v_scales : x.v};
        for (int j = 0; j < 2; j++) {
            if (x.pages > 0 && !of[j]) return BQ_ERR_NULL;
            if (!aligned(of[j], align)) return BQ_ERR_ALIGN;
            arrays[2 * i + j] = Paged{reinterpret_cast<uintptr_t>(of[j]), bytes, page_bytes, x.pages > 1 ? ps : INT64_MAX};
            spans[2 * i + j] = span(of[j], x.pages > 0 ? bytes : 0);
        }
    }
    for (int i = 0; i < 4 && x.pages > 0; i++)
        for (int j = i + 1; j < 4; j++)
            if (!disjoint(arrays[i], arrays[j])) return BQ_ERR_ALIAS;
    c.k = x.k, c.v = x.v;
    c.k_scales = static_cast<unsigned char *>(x.k_scales), c.v_scales = static_cast<unsigned char *>(x.v_scales);
    c.pages = x.pages, c.heads = x.heads, c.page = x.page, c.head_dim = x.head_dim, c.group = x.group;
    c.page_stride = x.pages > 1 ? x.page_stride : 0, c.page_stride_s = x.pages > 1 ? x.page_stride_s : 0;
    c.head_stride = x.heads > 1 ? x.head_stride : 0, c.head_stride_s = x.heads > 1 ? x.head_stride_s : 0;
    c.token_stride = x.page > 1 ? (int32_t)x.token_stride : 0;
    c.token_stride_s = x.page > 1 ? (int32_t)x.token_stride_s : 0;
    return BQ_OK;
}

// [tokens][heads][head_dim] rows of 16-bit values. rows_apart is asked of rows that are written.
bq_status check_kv_rows(const void *p, int64_t tokens, int heads, int dim, int64_t ld_token, int64_t ld_head, bool written,
                        Range *range)
{
    if ((tokens > 1 && ld_token < 0) || (heads > 1 && ld_head < 0)) return BQ_ERR_SHAPE;
    if ((tokens > 1 && ld_token > INT64_MAX / 16 / tokens) || (heads > 1 && ld_head > INT64_MAX / 16 / heads))
        return BQ_ERR_SHAPE;
    Dim d[3] = {{tokens, 2 * ld_token}, {heads, 2 * ld_head}, {1, 0}};
    int64_t bytes = 0;
    if (written && !rows_apart(d, 2 * dim, &bytes)) return BQ_ERR_SHAPE;
    bytes = 2 * ((tokens > 1 ? (tokens - 1) * ld_token : 0) + (heads > 1 ? (heads - 1) * ld_head : 0) + dim);
    if (!p) return BQ_ERR_NULL;
    if (!aligned(p, 16) || (tokens > 1 && ld_token % 8) || (heads > 1 && ld_head % 8)) return BQ_ERR_ALIGN;
    *range = span(p, bytes);
    return BQ_OK;
}

bq_status kv4_rows(const bq_kv4_cache *cache, const void *k, int64_t k_ld_token, int64_t k_ld_head, const void *v,
                   int64_t v_ld_token, int64_t v_ld_head, int64_t tokens, const void *slots, int slots_are_i64,
                   bool write, cudaStream_t stream)
{
    bqk::Kv4Cache c;
    Range held[4], k_rows, v_rows;
    if (bq_status e = check_cache(cache, c, held)) return e;
    if (tokens < 0 || tokens >= (1ll << 34) / c.heads / c.head_dim) return BQ_ERR_SHAPE;
    if (tokens == 0) return BQ_OK;
    if (bq_status e = check_kv_rows(k, tokens, c.heads, c.head_dim, k_ld_token, k_ld_head, !write, &k_rows)) return e;
    if (bq_status e = check_kv_rows(v, tokens, c.heads, c.head_dim, v_ld_token, v_ld_head, !write, &v_rows)) return e;
    if (!slots) return BQ_ERR_NULL;
    const int size = slots_are_i64 ? 8 : 4;
    if (!aligned(slots, size)) return BQ_ERR_ALIGN;
    const Range in_slots = span(slots, size * tokens);
    // the cache's own arrays are apart from each other already
    for (const Range &h : held)
        if (overlap(h, k_rows) || overlap(h, v_rows) || (write && overlap(h, in_slots))) return BQ_ERR_ALIAS;
    if (!write && (overlap(k_rows, v_rows) || overlap(k_rows, in_slots) || overlap(v_rows, in_slots)))
        return BQ_ERR_ALIAS;
    const bqk::Kv4Rows kr = {const_cast<void *>(k), tokens > 1 ? k_ld_token : 0, c.heads > 1 ? k_ld_head : 0};
    const bqk::Kv4Rows vr = {const_cast<void *>(v), tokens > 1 ? v_ld_token : 0, c.heads > 1 ? v_ld_head : 0};
    const bqk::Kv4Slots at = {slots, slots_are_i64 != 0};
    return from_cuda(write ? bqk::launch_kv4_write(cache->type, c, kr, vr, tokens, at, stream)
                           : bqk::launch_kv4_read(cache->type, c, kr, vr, tokens, at, stream));
}
}  // namespace

extern "C" {

bq_status bq_kv4_write(const bq_kv4_cache *cache, const void *k, int64_t k_ld_token, int64_t k_ld_head, const void *v,
                       int64_t v_ld_token, int64_t v_ld_head, int64_t tokens, const void *slots, int slots_are_i64,
                       cudaStream_t stream)
{
    return kv4_rows(cache, k, k_ld_token, k_ld_head, v, v_ld_token, v_ld_head, tokens, slots, slots_are_i64, true, stream);
}

bq_status bq_kv4_read(const bq_kv4_cache *cache, const void *slots, int slots_are_i64, int64_t tokens, void *k,
                      int64_t k_ld_token, int64_t k_ld_head, void *v, int64_t v_ld_token, int64_t v_ld_head,
                      cudaStream_t stream)
{
    return kv4_rows(cache, k, k_ld_token, k_ld_head, v, v_ld_token, v_ld_head, tokens, slots, slots_are_i64, false, stream);
}

int64_t bq_kv4_workspace_bytes(int heads, int head_dim, int n_q, int q_heads)
{
    if (heads < 1 || heads > BQ_KV4_MAX_HEADS || head_dim < 64 || head_dim > 256 || head_dim % 64 || n_q < 1 ||
        q_heads < 1 || q_heads > 65536 || q_heads % heads || n_q > (1 << 20) / q_heads)
        return -1;
    return bqk::kv4_workspace_bytes(heads, head_dim, n_q, q_heads);
}

bq_status bq_kv4_attend(const bq_kv4_cache *cache, const void *q, int64_t q_ld_batch, int64_t q_ld_query,
                        int64_t q_ld_head, int64_t batch, int n_q, int q_heads, const int32_t *table, int64_t ld_table,
                        int64_t width, const int32_t *lengths, float scale, int64_t window, void *out,
                        int64_t out_ld_batch, int64_t out_ld_query, int64_t out_ld_head, float *lse, void *workspace,
                        int64_t workspace_bytes, cudaStream_t stream)
{
    bqk::Kv4Cache c;
    Range held[4];
    if (bq_status e = check_cache(cache, c, held)) return e;
    if (batch < 0 || batch > INT32_MAX || n_q < 0 || q_heads < 0 || q_heads > 65536 || q_heads % c.heads)
        return BQ_ERR_SHAPE;
    if (width < 0 || width > (INT32_MAX - (1 << 20)) / c.page || window < 0 || window > (1 << 30)) return BQ_ERR_SHAPE;
    if (!(scale >= -3.4e38f && scale <= 3.4e38f)) return BQ_ERR_SHAPE;
    if (batch == 0 || n_q == 0 || q_heads == 0) return BQ_OK;
    if (n_q > (1 << 20) / q_heads || (batch > 1 && ld_table < width)) return BQ_ERR_SHAPE;
    // rows of q and out: [batch * n_q][q_heads] where batches and queries are dimensions of their own
    const int64_t row = c.head_dim, lds[2][3] = {{q_ld_batch, q_ld_query, q_ld_head},
                                                 {out_ld_batch, out_ld_query, out_ld_head}};
    const int64_t ns[3] = {batch, n_q, q_heads};
    int64_t bytes[2];
    for (int i = 0; i < 2; i++) {
        bytes[i] = 2 * row;
        Dim d[3];
        for (int j = 0; j < 3; j++) {
            d[j] = Dim{ns[j], 2 * lds[i][j]};
            if (ns[j] == 1) continue;
            if (lds[i][j] < 0 || lds[i][j] > INT64_MAX / 64 / ns[j]) return BQ_ERR_SHAPE;
            bytes[i] += 2 * (ns[j] - 1) * lds[i][j];
        }
        int64_t apart = 0;
        if (i == 1 && !rows_apart(d, 2 * row, &apart)) return BQ_ERR_SHAPE;
        const void *p = i ? out : q;
        if (!p) return BQ_ERR_NULL;
        if (!aligned(p, 16)) return BQ_ERR_ALIGN;
        for (int j = 0; j < 3; j++)
            if (ns[j] > 1 && lds[i][j] % 8) return BQ_ERR_ALIGN;
    }
    const int64_t need = bq_kv4_workspace_bytes(c.heads, c.head_dim, n_q, q_heads);
    if (need < 0 || workspace_bytes < need) return BQ_ERR_SHAPE;
    if (!lengths || !workspace || (width > 0 && !table)) return BQ_ERR_NULL;
    if (!aligned(lengths, 4) || !aligned(table, 4) || !aligned(lse, 4) || !aligned(workspace, 16)) return BQ_ERR_ALIGN;
    const Range none = span(lengths, 0);
    const Range ins[] = {span(q, bytes[0]), width > 0 ? span(table, 4 * ((batch - 1) * ld_table + width)) : none,
                         span(lengths, 4 * batch), held[0], held[1], held[2], held[3]};
    const Range outs[] = {span(out, bytes[1]), span(workspace, need), lse ? span(lse, 4 * batch * n_q * q_heads) : none};
    if (any_alias(outs, 3, ins, 7)) return BQ_ERR_ALIAS;
    bqk::Kv4Attend a = {};
    a.q = q, a.q_batch = batch > 1 ? q_ld_batch : 0, a.q_query = n_q > 1 ? q_ld_query : 0;
    a.q_head = q_heads > 1 ? q_ld_head : 0;
    a.out = out, a.out_batch = batch > 1 ? out_ld_batch : 0, a.out_query = n_q > 1 ? out_ld_query : 0;
    a.out_head = q_heads > 1 ? out_ld_head : 0;
    a.lse = lse, a.table = table, a.lengths = lengths, a.ld_table = batch > 1 ? ld_table : 0;
    a.width = (int)width, a.batch = (int)batch, a.n_q = n_q, a.q_heads = q_heads, a.window = (int)window;
    a.scale = scale, a.workspace = static_cast<float *>(workspace);
    return from_cuda(bqk::launch_kv4_attend(cache->type, c, a, stream));
}

}  // extern "C"

namespace {
// Growth of the current device's counter `which` (0: abandoned waits, 1: copies that
// did not land after one, 2: accesses a debug build declined) since the previous call
// for it. The device counters only grow; the last totals seen are kept per device here,
// and they are advanced only after every translation unit's counters were read.
constexpr int kMaxDevices = 64;
std::mutex g_seen_mu;
unsigned long long g_seen[kMaxDevices][3];

bq_status take_wait_counter(int which, int64_t *count)
{
    if (!count) return BQ_ERR_NULL;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return BQ_ERR_CUDA;
    unsigned long long total = 0;
    for (auto read : {bqk::read_wait_counters_i8, bqk::read_wait_counters_mx_wire, bqk::read_wait_counters_mx,
                      bqk::read_wait_counters_e4m3, bqk::read_wait_counters_experts, bqk::read_wait_counters_w4,
                      bqk::read_wait_counters_kv4, bqk::read_wait_counters_attend,
                      bqk::read_wait_counters_attend_bf16, bqk::read_wait_counters_attend_f16}) {
        unsigned long long v[3] = {0, 0, 0};
        if (read(v) != cudaSuccess) return BQ_ERR_CUDA;
        total += v[which];
    }
    std::lock_guard<std::mutex> lock(g_seen_mu);
    *count = static_cast<int64_t>(total - g_seen[dev][which]);
    g_seen[dev][which] = total;
    return BQ_OK;
}
}  // namespace

extern "C" {

bq_status bq_take_wait_timeouts(int64_t *count) { return take_wait_counter(0, count); }

bq_status bq_take_wait_unlanded(int64_t *count) { return take_wait_counter(1, count); }

bq_status bq_take_index_errors(int64_t *count) { return take_wait_counter(2, count); }

int bq_debug_build(void) { return BQ_DEBUG; }

bq_status bq_selftest_index_check(void *buf, int64_t bytes, cudaStream_t stream)
{
    if (!BQ_DEBUG) return BQ_ERR_UNSUPPORTED;
    if (!buf) return BQ_ERR_NULL;
    if (bytes < 1024) return BQ_ERR_SHAPE;
    if (!aligned(buf, 16)) return BQ_ERR_ALIGN;
    return from_cuda(bqk::launch_index_selftest(buf, stream));
}

bq_status bq_selftest_wait_timeout(cudaStream_t stream) { return from_cuda(bqk::launch_wait_selftest(stream)); }

}  // extern "C"
