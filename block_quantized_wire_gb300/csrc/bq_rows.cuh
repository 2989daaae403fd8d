// Rows of BF16, FP16 or FP32 values, as the expert-layer kernels move them.
#pragma once

#include "bq_device.cuh"

namespace bqk {

// Rows are moved in pieces of kWide values per lane where every row starts on a 16-byte
// boundary and holds whole pieces, else value by value.
template <class T>
struct Value;
template <>
struct Value<__nv_bfloat16> {
    static __device__ __forceinline__ float widen(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
    static __device__ __forceinline__ uint16_t round(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
    using Bits = uint16_t;
};
template <>
struct Value<__half> {
    static __device__ __forceinline__ float widen(uint16_t b) { return __half2float(__ushort_as_half(b)); }
    static __device__ __forceinline__ uint16_t round(float v) { return __half_as_ushort(__float2half_rn(v)); }
    using Bits = uint16_t;
};
template <>
struct Value<float> {
    static __device__ __forceinline__ float widen(uint32_t b) { return __uint_as_float(b); }
    static __device__ __forceinline__ uint32_t round(float v) { return __float_as_uint(v); }
    using Bits = uint32_t;
};

// A lane's piece of a row: N values of type T, as raw bits.
template <class T, bool kWide>
struct Piece {
    using Bits = typename Value<T>::Bits;
    static constexpr int N = kWide ? 16 / (int)sizeof(T) : 1;
    Bits b[N];

    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < N; i++) b[i] = 0;
    }
    __device__ __forceinline__ void load(const T *p)
    {
        if constexpr (kWide) {
            *reinterpret_cast<uint4 *>(b) = ld_stream_v4(p);
        } else {
            b[0] = dbg_ok(p, sizeof(T), false) ? __ldg(reinterpret_cast<const Bits *>(p)) : Bits(0);
        }
    }
    __device__ __forceinline__ void store(T *p) const
    {
        if constexpr (kWide) {
            st_v4(p, *reinterpret_cast<const uint4 *>(b));
        } else {
            if (dbg_ok(p, sizeof(T), true)) *reinterpret_cast<Bits *>(p) = b[0];
        }
    }
    __device__ __forceinline__ float at(int i) const { return Value<T>::widen(b[i]); }
    __device__ __forceinline__ void set(int i, float v) { b[i] = Value<T>::round(v); }
};

// True if every row of `hidden` values of `size` bytes, `ld` values apart, starts on a
// 16-byte boundary and is a whole number of 16-byte pieces.
static inline bool wide_rows(const void *p, int64_t hidden, int64_t ld, int size)
{
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && hidden * size % 16 == 0 && ld * size % 16 == 0;
}

}  // namespace bqk
