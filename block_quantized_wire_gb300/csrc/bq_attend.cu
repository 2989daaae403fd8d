// Attention over a key-value cache in 4 bits: a query row a CTA, its warps taking positions in turn
// with a running maximum and sum each, joined at the end.
#include <cmath>

#include "bq_kv4.cuh"

namespace bqk {
namespace {

constexpr int kRowWarps = kThreads / 32;

template <class T, int kDim>
__global__ void __launch_bounds__(kThreads) attend_row_kernel(const __grid_constant__ Kv4Cache c,
                                                             const __grid_constant__ Kv4Attend a)
{
    constexpr int kPer = kDim / 32;  // columns of a lane
    __shared__ float sums[kRowWarps][kDim], tops[kRowWarps], totals[kRowWarps];
    pdl_begin();
    dbg_begin();
    dbg_cache(c, false);
    dbg_allow(a.q, 2 * ((a.batch - 1) * a.q_batch + (a.n_q - 1) * a.q_query + (a.q_heads - 1) * a.q_head + kDim), false);
    dbg_allow(a.out, 2 * ((a.batch - 1) * a.out_batch + (a.n_q - 1) * a.out_query + (a.q_heads - 1) * a.out_head + kDim),
              true);
    dbg_allow(a.table, 4 * ((a.batch - 1) * a.ld_table + a.width), false);
    dbg_allow(a.lengths, 4ll * a.batch, false);
    dbg_allow(a.lse, a.lse ? 4ll * a.batch * a.n_q * a.q_heads : 0, true);
    dbg_ready();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t rows = (int64_t)a.batch * a.n_q * a.q_heads;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const int h = (int)(row % a.q_heads), i = (int)(row / a.q_heads % a.n_q), b = (int)(row / a.q_heads / a.n_q);
        const int head = h / (a.q_heads / c.heads);
        const int cap = a.width * c.page;
        int length = dbg_ok(a.lengths + b, 4, false) ? a.lengths[b] : 0;
        length = length < 0 ? 0 : length < cap ? length : cap;
        const int end = length - a.n_q + i + 1, begin = a.window > 0 && end > a.window ? end - a.window : 0;
        const T *q = static_cast<const T *>(a.q) + b * a.q_batch + i * a.q_query + h * a.q_head + lane * kPer;
        float x[kPer], o[kPer] = {}, top = -3.0e38f, total = 0.0f;
#pragma unroll
        for (int d = 0; d < kPer; d++)
            x[d] = dbg_ok(q + d, 2, false) ? Value<T>::widen(*reinterpret_cast<const uint16_t *>(q + d)) : 0.0f;
        for (int j = begin + warp; j < end; j += kRowWarps) {
            const int32_t *entry = a.table + b * a.ld_table + j / c.page;
            const int page = dbg_ok(entry, 4, false) ? *entry : -1;
            if (page < 0 || page >= c.pages) continue;
            const int64_t at = page * c.page_stride + head * c.head_stride + (int64_t)(j % c.page) * c.token_stride;
            const int64_t at_s = page * c.page_stride_s + head * c.head_stride_s + (int64_t)(j % c.page) * c.token_stride_s;
            float value[2][kPer];
#pragma unroll
            for (int w = 0; w < 2; w++) {
                const uint8_t *codes = (w ? c.v : c.k) + at + lane * kPer / 2;
                const uint32_t *pairs = reinterpret_cast<const uint32_t *>((w ? c.v_scales : c.k_scales) + at_s);
#pragma unroll
                for (int d = 0; d < kPer; d++) {
                    const uint32_t *pair = pairs + (lane * kPer + d) / c.group;
                    const float2 p = pair_values<T>(dbg_ok(pair, 4, false) ? *pair : 0u);
                    const int two = dbg_ok(codes + d / 2, 1, false) ? codes[d / 2] : 0;
                    const int code = ((d & 1 ? two >> 4 : two & 15) ^ 8) - 8;
                    value[w][d] = __fmaf_rn((float)code, p.x, p.y);
                }
            }
            float score = 0.0f;
#pragma unroll
            for (int d = 0; d < kPer; d++) score = __fmaf_rn(x[d], value[0][d], score);
#pragma unroll
            for (int d = 16; d; d >>= 1) score = __fadd_rn(score, __shfl_xor_sync(kFull, score, d));
            score = __fmul_rn(score, a.scale);
            const float now = fmaxf(top, score), keep = expf(__fsub_rn(top, now)), p = expf(__fsub_rn(score, now));
            top = now;
            total = __fmaf_rn(total, keep, p);
#pragma unroll
            for (int d = 0; d < kPer; d++) o[d] = __fmaf_rn(o[d], keep, __fmul_rn(p, value[1][d]));
        }
        __syncthreads();  // the readers of the row before
#pragma unroll
        for (int d = 0; d < kPer; d++) sums[warp][lane * kPer + d] = o[d];
        if (lane == 0) tops[warp] = top, totals[warp] = total;
        __syncthreads();
        float all = -3.0e38f, sum = 0.0f;
        for (int w = 0; w < kRowWarps; w++) all = fmaxf(all, tops[w]);
        for (int w = 0; w < kRowWarps; w++) sum = __fmaf_rn(totals[w], expf(__fsub_rn(tops[w], all)), sum);
        for (int d = threadIdx.x; d < kDim; d += kThreads) {
            float v = 0.0f;
            for (int w = 0; w < kRowWarps; w++) v = __fmaf_rn(sums[w][d], expf(__fsub_rn(tops[w], all)), v);
            T *dst = static_cast<T *>(a.out) + b * a.out_batch + i * a.out_query + h * a.out_head + d;
            if (dbg_ok(dst, 2, true)) *reinterpret_cast<uint16_t *>(dst) = Value<T>::round(sum == 0.0f ? 0.0f : __fdiv_rn(v, sum));
        }
        if (a.lse && threadIdx.x == 0 && dbg_ok(a.lse + row, 4, true))
            a.lse[row] = sum == 0.0f ? -INFINITY : __fadd_rn(all, logf(sum));
    }
}

template <class T>
cudaError_t launch(const Kv4Cache &c, const Kv4Attend &a, cudaStream_t st)
{
    void (*kernel)(Kv4Cache, Kv4Attend) = c.head_dim == 64    ? attend_row_kernel<T, 64>
                                          : c.head_dim == 128 ? attend_row_kernel<T, 128>
                                          : c.head_dim == 192 ? attend_row_kernel<T, 192>
                                                              : attend_row_kernel<T, 256>;
    int grid = 0;
    const int64_t rows = (int64_t)a.batch * a.n_q * a.q_heads;
    if (cudaError_t e = grid_for((const void *)kernel, rows * kRowWarps, &grid)) return e;
    return launch_kernel(kernel, grid, st, c, a);
}

}  // namespace

int64_t kv4_workspace_bytes(int, int, int, int) { return 0; }

cudaError_t launch_kv4_attend(int type, const Kv4Cache &c, const Kv4Attend &a, cudaStream_t st)
{
    return type == kBf16 ? launch<__nv_bfloat16>(c, a, st) : launch<__half>(c, a, st);
}

cudaError_t read_wait_counters_attend(unsigned long long (&v)[3]) { return read_wait_counters(v); }

}  // namespace bqk
