// Attention over a 4-bit cache whose pairs and queries are FP16.
#include "bq_attend.cuh"

namespace bqk {

cudaError_t launch_attend_f16(const Kv4Cache &c, const Kv4Attend &a, AttendPlan &plan, cudaStream_t st)
{
    return launch_attend<__half>(c, a, plan, st);
}

cudaError_t read_wait_counters_attend_f16(unsigned long long (&v)[3]) { return read_wait_counters(v); }

}  // namespace bqk
