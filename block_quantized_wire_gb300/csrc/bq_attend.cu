// Attention over a key-value cache in 4 bits: the call's two launches. bq_attend.cuh has the kernel that streams the
// cache; here the pieces that several of its CTAs worked on are put together.
#include "bq_attend.cuh"

namespace bqk {
namespace {

// A warp a row: CTA c of a group of four rows joins the item that goes on from share c to the next, if it began there.
template <class T, int kDim>
__global__ void __launch_bounds__(kAttendThreads) attend_join_kernel(const __grid_constant__ Kv4Cache c,
                                                                    const __grid_constant__ Kv4Attend a,
                                                                    const __grid_constant__ AttendPlan plan, int form, int groups)
{
    constexpr int kPer = kDim / 32;  // columns of a lane
    const int64_t partial = partial_floats(form, kDim);
    pdl_begin();
    dbg_attend(c, a, plan, partial);
    const int cta = blockIdx.x / groups, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Share share;
    Spot at;
    find_share(c, a, plan, cta + 1, share, at);
    if (cta + 1 >= share.ctas || at.tile == 0) return;
    const int64_t begin = share.first(cta + 1) - at.tile, end = begin + at.tiles;
    if (begin < share.first(cta)) return;
    const int head = (int)divide_by(at.item, plan.by_chunks), row = (blockIdx.x - cta * groups) * kAttendWarps + warp;
    const int item_row = (at.item - head * plan.chunks) * form + row;
    if (row >= form || item_row >= plan.rows) return;
    int last = cta + 1;  // past the last share with a part of the item
    while (last < share.ctas && share.first(last) < end) last++;
    // share `cta` left it as what goes on after it, the others as what began before them
    const auto part = [&](int i) { return a.workspace + (2 * (int64_t)i + (i == cta)) * partial; };
    const auto load = [&](const float *p) { return dbg_ok(p, 4, false) ? *p : 0.0f; };
    float ref = kNothing;
    for (int i = cta + lane; i < last; i += 32) ref = fmaxf(ref, load(part(i) + row));
#pragma unroll
    for (int d = 16; d; d >>= 1) ref = fmaxf(ref, __shfl_xor_sync(kFull, ref, d));
    float total = 0.0f, sum[kPer] = {};
#pragma unroll 4
    for (int i = cta; i < last; i++) {
        const float *p = part(i);
        const float by = exp2_fast(__fsub_rn(load(p + row), ref));
        total = __fmaf_rn(load(p + form + row), by, total);
#pragma unroll
        for (int k = 0; k < kPer; k++) sum[k] = __fmaf_rn(load(p + 2 * form + row * kDim + 32 * k + lane), by, sum[k]);
    }
    int64_t at_lse;
    T *to = static_cast<T *>(a.out) + out_row(a, plan, at.b, head, item_row, &at_lse);
    const float inv = total == 0.0f ? 0.0f : __fdiv_rn(1.0f, total);
#pragma unroll
    for (int k = 0; k < kPer; k++)
        if (dbg_ok(to + 32 * k + lane, 2, true))
            *reinterpret_cast<uint16_t *>(to + 32 * k + lane) = Value<T>::round(__fmul_rn(sum[k], inv));
    if (a.lse && lane == 0 && dbg_ok(a.lse + at_lse, 4, true)) a.lse[at_lse] = lse_of(ref, total);
}

template <class T>
cudaError_t launch_join(const Kv4Cache &c, const Kv4Attend &a, const AttendPlan &plan, cudaStream_t st)
{
    void (*kernel)(Kv4Cache, Kv4Attend, AttendPlan, int, int) = c.head_dim == 64    ? attend_join_kernel<T, 64>
                                                                : c.head_dim == 128 ? attend_join_kernel<T, 128>
                                                                : c.head_dim == 192 ? attend_join_kernel<T, 192>
                                                                                    : attend_join_kernel<T, 256>;
    const int form = form_rows(plan.rows, c.head_dim);
    const int groups = ((plan.rows < form ? plan.rows : form) + kAttendWarps - 1) / kAttendWarps;
    return launch_kernel_block(kernel, (plan.ctas - 1) * groups, kAttendThreads, 0, st, c, a, plan, form, groups);
}

}  // namespace

int64_t kv4_workspace_bytes(int heads, int head_dim, int n_q, int q_heads)
{
    return 4 * 2 * kMaxAttendCtas * partial_floats(form_rows(n_q * (q_heads / heads), head_dim), head_dim);
}

cudaError_t launch_kv4_attend(int type, const Kv4Cache &c, const Kv4Attend &a, cudaStream_t st)
{
    AttendPlan plan = {};
    plan.share = a.q_heads / c.heads, plan.rows = a.n_q * plan.share;
    plan.by_share = divisor((uint32_t)plan.share), plan.by_page = divisor((uint32_t)c.page);
    const bool bf16 = type == kBf16;
    if (cudaError_t e = bf16 ? launch_attend_bf16(c, a, plan, st) : launch_attend_f16(c, a, plan, st)) return e;
    if (plan.ctas == 1) return cudaSuccess;  // nothing is shared
    return bf16 ? launch_join<__nv_bfloat16>(c, a, plan, st) : launch_join<__half>(c, a, plan, st);
}

cudaError_t read_wait_counters_attend(unsigned long long (&v)[3]) { return read_wait_counters(v); }

}  // namespace bqk
