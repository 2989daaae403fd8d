// Attention over a 4-bit cache whose pairs and queries are BF16.
#include "bq_attend.cuh"

namespace bqk {

cudaError_t launch_attend_bf16(const Kv4Cache &c, const Kv4Attend &a, AttendPlan &plan, cudaStream_t st)
{
    return launch_attend<__nv_bfloat16>(c, a, plan, st);
}

cudaError_t read_wait_counters_attend_bf16(unsigned long long (&v)[3]) { return read_wait_counters(v); }

}  // namespace bqk
