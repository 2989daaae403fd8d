// Attention over a key-value cache in 4 bits: the call's two launches. bq_attend.cuh has the kernel that streams the
// cache; here the pieces that several of its CTAs worked on are put together.
#include "bq_attend.cuh"

namespace bqk {
namespace {

__device__ __forceinline__ uint4 ld_plain_v4(const float *p)
{
    if (!dbg_ok(p, 16, false)) return make_uint4(0, 0, 0, 0);
    return *reinterpret_cast<const uint4 *>(p);
}

// CTA i takes rows of the item that word i / splits names, if more than one share worked on it: all of them, or where there
// are few items (a long sequence or two, with many parts each) a few, down to one. A thread takes four columns of one row, of
// every groups-th part.
constexpr int kJoinThreads = 512;

template <class T, int kDim>
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(const __grid_constant__ Kv4Cache c,
                                                                  const __grid_constant__ Kv4Attend a,
                                                                  const __grid_constant__ AttendPlan plan, int form, int per, int splits)
{
    constexpr int kAhead = 4;  // parts that a thread loads before the weights are known
    __shared__ float refs[16], totals[16];
    __shared__ float4 sums[kJoinThreads];
    const int64_t floats = partial_floats(form, kDim);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_begin();
    dbg_attend(c, a, plan, floats);
    const uint4 word = ld_plain_v4(a.workspace + 4 * (blockIdx.x / splits));
    const int parts = (int)word.z;
    if (parts < 2) return;
    const int width = per * (kDim / 4), groups = kJoinThreads / width;
    const int group = threadIdx.x / width, in = threadIdx.x - group * width, row = in / (kDim / 4), col = 4 * (in - row * (kDim / 4));
    const auto load = [&](const float *p) { return dbg_ok(p, 4, false) ? *p : 0.0f; };
    const int b = (int)word.x, item = (int)word.y, cta = (int)word.w, row0 = blockIdx.x % splits * per;
    const int head = (int)divide_by(item, plan.by_chunks), first = (item - head * plan.chunks) * form + row0;
    const int rows = min(min(plan.rows - first, form - row0), per);
    if (rows <= 0) return;
    // the share left it as what goes on after it, the others as what began before them
    const auto part = [&](int i) { return partial_of(a.workspace, cta + i, i == 0, floats); };
    const bool busy = group < groups && row < rows;
    const auto piece = [&](int i) { return ld_plain_v4(part(i) + 2 * form + (row0 + row) * kDim + col); };
    uint4 v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; k++)
        if (busy && group + k * groups < parts) v[k] = piece(group + k * groups);
    if (warp < rows) {
        float ref = kNothing, total = 0.0f;
#pragma unroll 4
        for (int i = lane; i < parts; i += 32) {
            const float r = load(part(i) + row0 + warp), t = load(part(i) + form + row0 + warp), next = fmaxf(ref, r);
            total = __fmaf_rn(t, exp2_fast(__fsub_rn(r, next)), __fmul_rn(total, exp2_fast(__fsub_rn(ref, next))));
            ref = next;
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            const float r = __shfl_xor_sync(kFull, ref, d), t = __shfl_xor_sync(kFull, total, d), next = fmaxf(ref, r);
            total = __fadd_rn(__fmul_rn(t, exp2_fast(__fsub_rn(r, next))), __fmul_rn(total, exp2_fast(__fsub_rn(ref, next))));
            ref = next;
        }
        if (lane == 0) refs[warp] = ref, totals[warp] = total;
    }
    __syncthreads();
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (busy) {
        const float ref = refs[row];
        const auto add = [&](int i, uint4 v) {
            const float by = exp2_fast(__fsub_rn(load(part(i) + row0 + row), ref));
            sum = make_float4(__fmaf_rn(__uint_as_float(v.x), by, sum.x), __fmaf_rn(__uint_as_float(v.y), by, sum.y),
                              __fmaf_rn(__uint_as_float(v.z), by, sum.z), __fmaf_rn(__uint_as_float(v.w), by, sum.w));
        };
#pragma unroll
        for (int k = 0; k < kAhead; k++)
            if (group + k * groups < parts) add(group + k * groups, v[k]);
#pragma unroll 4
        for (int i = group + kAhead * groups; i < parts; i += groups) add(i, piece(i));
    }
    sums[threadIdx.x] = sum;
    __syncthreads();
    if (group == 0 && row < rows) {
        for (int i = 1; i < groups; i++) {
            const float4 v = sums[i * width + in];
            sum = make_float4(__fadd_rn(sum.x, v.x), __fadd_rn(sum.y, v.y), __fadd_rn(sum.z, v.z), __fadd_rn(sum.w, v.w));
        }
        int64_t at_lse;
        T *to = static_cast<T *>(a.out) + out_row(a, plan, b, head, first + row, &at_lse);
        const float total = totals[row], inv = total == 0.0f ? 0.0f : __fdiv_rn(1.0f, total);
        st_v2(to + col, make_uint2(Value<T>::round2(__fmul_rn(sum.x, inv), __fmul_rn(sum.y, inv)),
                                   Value<T>::round2(__fmul_rn(sum.z, inv), __fmul_rn(sum.w, inv))));
        if (a.lse && col == 0 && dbg_ok(a.lse + at_lse, 4, true)) a.lse[at_lse] = lse_of(refs[row], total);
    }
}

template <class T>
cudaError_t launch_join(const Kv4Cache &c, const Kv4Attend &a, const AttendPlan &plan, cudaStream_t st)
{
    void (*kernel)(Kv4Cache, Kv4Attend, AttendPlan, int, int, int) = c.head_dim == 64    ? attend_join_kernel<T, 64>
                                                                : c.head_dim == 128 ? attend_join_kernel<T, 128>
                                                                : c.head_dim == 192 ? attend_join_kernel<T, 192>
                                                                                    : attend_join_kernel<T, 256>;
    const int form = form_rows(plan.rows, c.head_dim);
    int sms = 0;
    if (cudaError_t e = sm_count(&sms)) return e;
    const int rows = plan.rows < form ? plan.rows : form;
    int splits = 1;  // as many as run at once
    while (splits < rows && 2 * splits * plan.words <= 4 * sms) splits *= 2;
    const int per = (rows + splits - 1) / splits;
    splits = (rows + per - 1) / per;
    return launch_kernel_block(kernel, plan.words * splits, kJoinThreads, 0, st, c, a, plan, form, per, splits);
}

}  // namespace

int64_t kv4_workspace_bytes(int heads, int head_dim, int n_q, int q_heads)
{
    return 4 * kMaxAttendCtas * (4 + 2 * partial_floats(form_rows(n_q * (q_heads / heads), head_dim), head_dim));
}

cudaError_t launch_kv4_attend(int type, const Kv4Cache &c, const Kv4Attend &a, cudaStream_t st)
{
    AttendPlan plan = {};
    plan.share = a.q_heads / c.heads, plan.rows = a.n_q * plan.share;
    plan.by_share = divisor((uint32_t)plan.share), plan.page_tiles = c.page % kTokens ? 0 : c.page / kTokens;
    plan.by_page = divisor((uint32_t)(plan.page_tiles ? plan.page_tiles : c.page));
    const bool bf16 = type == kBf16;
    if (cudaError_t e = bf16 ? launch_attend_bf16(c, a, plan, st) : launch_attend_f16(c, a, plan, st)) return e;
    if (plan.ctas == 1) return cudaSuccess;  // nothing is shared
    return bf16 ? launch_join<__nv_bfloat16>(c, a, plan, st) : launch_join<__half>(c, a, plan, st);
}

cudaError_t read_wait_counters_attend(unsigned long long (&v)[3]) { return read_wait_counters(v); }

}  // namespace bqk
