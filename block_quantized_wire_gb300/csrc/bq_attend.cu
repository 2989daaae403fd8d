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

// A CTA four rows of an item that goes on after share blockIdx.x / groups, if there is one. A thread takes four columns of one
// row, of every kGroups-th part.
constexpr int kJoinRows = 4, kJoinThreads = 512;

template <class T, int kDim>
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(const __grid_constant__ Kv4Cache c,
                                                                  const __grid_constant__ Kv4Attend a,
                                                                  const __grid_constant__ AttendPlan plan, int form, int groups)
{
    constexpr int kGroups = kJoinThreads / kDim;
    __shared__ float weight[kJoinRows][kMaxAttendCtas + 1], refs[kJoinRows], totals[kJoinRows];
    __shared__ float4 sums[kGroups][kDim];
    const int64_t floats = partial_floats(form, kDim);
    pdl_begin();
    dbg_attend(c, a, plan, floats);
    const int cta = blockIdx.x / groups, row0 = (blockIdx.x - cta * groups) * kJoinRows;
    const uint4 word = ld_plain_v4(a.workspace + 4 * cta);
    const Split at = {(int)word.x, (int)word.y, (int)word.z, 0};
    const int head = (int)divide_by(at.item, plan.by_chunks), first = (at.item - head * plan.chunks) * form + row0;
    const int rows = min(min(form - row0, plan.rows - first), kJoinRows);
    if (at.parts == 0 || rows <= 0) return;
    // share `cta` left it as what goes on after it, the others as what began before them
    const auto part = [&](int i) { return partial_of(a.workspace, cta + i, i == 0, floats); };
    const auto load = [&](const float *p) { return dbg_ok(p, 4, false) ? *p : 0.0f; };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp < rows) {
        float ref = kNothing, total = 0.0f;
        for (int i = lane; i < at.parts; i += 32) {
            const float r = load(part(i) + row0 + warp);
            weight[warp][i] = r;
            ref = fmaxf(ref, r);
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) ref = fmaxf(ref, __shfl_xor_sync(kFull, ref, d));
        for (int i = lane; i < at.parts; i += 32) {
            const float by = exp2_fast(__fsub_rn(weight[warp][i], ref));
            weight[warp][i] = by;
            total = __fmaf_rn(load(part(i) + form + row0 + warp), by, total);
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) total = __fadd_rn(total, __shfl_xor_sync(kFull, total, d));
        if (lane == 0) refs[warp] = ref, totals[warp] = total;
    }
    __syncthreads();
    const int group = threadIdx.x / kDim, in = threadIdx.x - group * kDim, row = in / (kDim / 4), col = 4 * (in - row * (kDim / 4));
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (group < kGroups && row < rows) {
#pragma unroll 8
        for (int i = group; i < at.parts; i += kGroups) {
            const uint4 v = ld_plain_v4(part(i) + 2 * form + (row0 + row) * kDim + col);
            const float by = weight[row][i];
            sum = make_float4(__fmaf_rn(__uint_as_float(v.x), by, sum.x), __fmaf_rn(__uint_as_float(v.y), by, sum.y),
                              __fmaf_rn(__uint_as_float(v.z), by, sum.z), __fmaf_rn(__uint_as_float(v.w), by, sum.w));
        }
        sums[group][in] = sum;
    }
    __syncthreads();
    if (group != 0 || row >= rows) return;
#pragma unroll
    for (int i = 1; i < kGroups; i++) {
        const float4 v = sums[i][in];
        sum = make_float4(__fadd_rn(sum.x, v.x), __fadd_rn(sum.y, v.y), __fadd_rn(sum.z, v.z), __fadd_rn(sum.w, v.w));
    }
    int64_t at_lse;
    T *to = static_cast<T *>(a.out) + out_row(a, plan, at.b, head, first + row, &at_lse);
    const float total = totals[row], inv = total == 0.0f ? 0.0f : __fdiv_rn(1.0f, total);
    st_v2(to + col, make_uint2(Value<T>::round2(__fmul_rn(sum.x, inv), __fmul_rn(sum.y, inv)),
                               Value<T>::round2(__fmul_rn(sum.z, inv), __fmul_rn(sum.w, inv))));
    if (a.lse && col == 0 && dbg_ok(a.lse + at_lse, 4, true)) a.lse[at_lse] = lse_of(refs[row], total);
}

template <class T>
cudaError_t launch_join(const Kv4Cache &c, const Kv4Attend &a, const AttendPlan &plan, cudaStream_t st)
{
    void (*kernel)(Kv4Cache, Kv4Attend, AttendPlan, int, int) = c.head_dim == 64    ? attend_join_kernel<T, 64>
                                                                : c.head_dim == 128 ? attend_join_kernel<T, 128>
                                                                : c.head_dim == 192 ? attend_join_kernel<T, 192>
                                                                                    : attend_join_kernel<T, 256>;
    const int form = form_rows(plan.rows, c.head_dim);
    const int groups = ((plan.rows < form ? plan.rows : form) + kJoinRows - 1) / kJoinRows;
    return launch_kernel_block(kernel, (plan.ctas - 1) * groups, kJoinThreads, 0, st, c, a, plan, form, groups);
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
    plan.by_share = divisor((uint32_t)plan.share), plan.by_page = divisor((uint32_t)c.page);
    const bool bf16 = type == kBf16;
    if (cudaError_t e = bf16 ? launch_attend_bf16(c, a, plan, st) : launch_attend_f16(c, a, plan, st)) return e;
    if (plan.ctas == 1) return cudaSuccess;  // nothing is shared
    return bf16 ? launch_join<__nv_bfloat16>(c, a, plan, st) : launch_join<__half>(c, a, plan, st);
}

cudaError_t read_wait_counters_attend(unsigned long long (&v)[3]) { return read_wait_counters(v); }

}  // namespace bqk
