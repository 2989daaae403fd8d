// A key-value cache in 4 bits as its kernels see it: where rows lie, and the numbers that codes
// stand for.
#pragma once

#include "bq_rows.cuh"

namespace bqk {

// n < 2^31
__device__ __forceinline__ uint32_t divide_by(uint32_t n, const Divisor &d) { return (__umulhi(n, d.mul) + n) >> d.shift; }

// The two floats of a (scale, offset) pair.
template <class T>
__device__ __forceinline__ float2 pair_values(uint32_t w)
{
    return make_float2(Value<T>::widen((uint16_t)(w & 0xffffu)), Value<T>::widen((uint16_t)(w >> 16)));
}

// A cache's arrays for the debug build.
__device__ __forceinline__ void dbg_cache(const Kv4Cache &c, bool writable)
{
#if BQ_DEBUG
    const int64_t codes = (c.pages - 1) * c.page_stride + (int64_t)(c.heads - 1) * c.head_stride +
                          (int64_t)(c.page - 1) * c.token_stride + c.head_dim / 2;
    const int64_t pairs = (c.pages - 1) * c.page_stride_s + (int64_t)(c.heads - 1) * c.head_stride_s +
                          (int64_t)(c.page - 1) * c.token_stride_s + 4 * (c.head_dim / c.group);
    dbg_allow(c.k, c.pages ? codes : 0, writable);
    dbg_allow(c.v, c.pages ? codes : 0, writable);
    dbg_allow(c.k_scales, c.pages ? pairs : 0, writable);
    dbg_allow(c.v_scales, c.pages ? pairs : 0, writable);
#else
    (void)c, (void)writable;
#endif
}

}  // namespace bqk
