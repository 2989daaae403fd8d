// Rows of BF16, FP16 or FP32 values, as the expert-layer kernels move them.
#pragma once

#include "bq_device.cuh"

namespace bqk {

template <class T>
struct Value;
template <>
struct Value<__nv_bfloat16> {
    static __device__ __forceinline__ float widen(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
    static __device__ __forceinline__ uint16_t round(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
    static __device__ __forceinline__ uint32_t round2(float lo, float hi)
    {
        return f32x2_to_bf16x2(make_float2(lo, hi));
    }
    using Bits = uint16_t;
};
template <>
struct Value<__half> {
    static __device__ __forceinline__ float widen(uint16_t b) { return __half2float(__ushort_as_half(b)); }
    static __device__ __forceinline__ uint16_t round(float v) { return __half_as_ushort(__float2half_rn(v)); }
    static __device__ __forceinline__ uint32_t round2(float lo, float hi)
    {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    using Bits = uint16_t;
};
template <>
struct Value<float> {
    static __device__ __forceinline__ float widen(uint32_t b) { return __uint_as_float(b); }
    static __device__ __forceinline__ uint32_t round(float v) { return __float_as_uint(v); }
    using Bits = uint32_t;
};

// 16 bytes that other lanes or warps will read too: through L1.
__device__ __forceinline__ uint4 ld_keep_v4(const void *p)
{
    if (!dbg_ok(p, 16, false)) return make_uint4(0, 0, 0, 0);
    return __ldg(static_cast<const uint4 *>(p));
}

// A lane's piece of a row: 16 bytes of values of type T, as raw bits.
template <class T>
struct Piece {
    using Bits = typename Value<T>::Bits;
    static constexpr int N = 16 / (int)sizeof(T);
    uint32_t w[4];

    __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0; }
    __device__ __forceinline__ Bits bits(int i) const
    {
        if constexpr (sizeof(T) == 4) return w[i];
        return (Bits)(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu);
    }
    __device__ __forceinline__ void set_bits(int i, Bits b)
    {
        if constexpr (sizeof(T) == 4)
            w[i] = b;
        else
            w[i / 2] = i & 1 ? (w[i / 2] & 0xffffu) | ((uint32_t)b << 16) : (w[i / 2] & 0xffff0000u) | b;
    }
    __device__ __forceinline__ float at(int i) const { return Value<T>::widen(bits(i)); }
    __device__ __forceinline__ void round(const float (&v)[N])
    {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < N; i++) w[i] = __float_as_uint(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < N / 2; i++) w[i] = Value<T>::round2(v[2 * i], v[2 * i + 1]);
        }
    }
    __device__ __forceinline__ void put(const uint4 v) { w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w; }
};

// How rows are cut into pieces. Where every row starts on a 16-byte boundary and is whole
// pieces (kWide), piece i is the columns [N i, N i + N). Else the pieces are the 16-byte
// words of the row that is written: its first and last may stick out of the row, and a row
// that is read lies at some other alignment to them, so a piece of it is put together from
// the two aligned words that hold it. Only the ends of the buffer are read value by value:
// 10551 tokens' gather gradient of 919 BF16 columns took 24.0 us with whole rows so, 15.1 us
// in words.
template <class T, bool kWide>
struct Cut {
    using P = Piece<T>;
    static constexpr int N = P::N;

    static __host__ __device__ __forceinline__ int64_t pieces(int64_t hidden)
    {
        if (hidden == 0) return 0;  // a row without columns has no words, wherever it starts
        return kWide ? hidden / N : (hidden + 2 * N - 2) / N;
    }
    // first column of piece i of the row written at `row`; it may be negative
    static __host__ __device__ __forceinline__ int64_t column(const T *row, int64_t i)
    {
        return kWide ? N * i : N * i - (int64_t)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    }
    static __host__ __device__ __forceinline__ bool inside(int64_t c, int64_t hidden)
    {
        return c < hidden && (kWide || c > -N);
    }

    // Columns [c, c + N) of a row of the buffer [lo, hi), in two steps: fetch() starts the
    // loads, of several pieces one after the other, and take() puts the piece together. Where
    // a piece sticks out of its row the values there are whatever the buffer holds; keep()
    // clears them.
    struct Raw {
        uint4 x, y;
    };
    static __host__ __device__ __forceinline__ bool windowed(const T *p, const void *lo, const void *hi)
    {
        const uintptr_t a = reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)15;
        const uintptr_t end = reinterpret_cast<uintptr_t>(hi);
        return a >= reinterpret_cast<uintptr_t>(lo) && end >= 32 && a <= end - 32;  // a + 32 could wrap
    }
    static __device__ __forceinline__ void fetch(Raw &raw, const T *row, int64_t c, const void *lo, const void *hi)
    {
        if constexpr (kWide) {
            raw.x = ld_stream_v4(row + c);
        } else if (windowed(row + c, lo, hi)) {
            const char *a = reinterpret_cast<const char *>(reinterpret_cast<uintptr_t>(row + c) & ~(uintptr_t)15);
            raw.x = ld_keep_v4(a);
            raw.y = ld_keep_v4(a + 16);
        }
    }
    static __device__ __forceinline__ void take(P &v, const Raw &raw, const T *row, int64_t c, int64_t hidden,
                                                const void *lo, const void *hi)
    {
        if constexpr (kWide) {
            v.put(raw.x);
        } else if (windowed(row + c, lo, hi)) {
            const int skew = (int)(reinterpret_cast<uintptr_t>(row + c) & 15);
            const uint32_t u[8] = {raw.x.x, raw.x.y, raw.x.z, raw.x.w, raw.y.x, raw.y.y, raw.y.z, raw.y.w};
            uint32_t s[6], r[5];
#pragma unroll
            for (int i = 0; i < 6; i++) s[i] = skew & 8 ? u[i + 2] : u[i];
#pragma unroll
            for (int i = 0; i < 5; i++) r[i] = skew & 4 ? s[i + 1] : s[i];
#pragma unroll
            for (int i = 0; i < 4; i++) v.w[i] = __funnelshift_r(r[i], r[i + 1], 8 * (skew & 2));
        } else {
            v.put(at_end(row + c, -c, hidden - c));
        }
    }
    // a piece at the buffer's ends, value by value: those with lo <= i < hi
    static __device__ __noinline__ uint4 at_end(const T *p, int64_t lo, int64_t hi)
    {
        P v;
        v.zero();
#pragma unroll
        for (int i = 0; i < N; i++)
            if (i >= lo && i < hi && dbg_ok(p + i, sizeof(T), false))
                v.set_bits(i, __ldg(reinterpret_cast<const typename P::Bits *>(p + i)));
        return make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
    }
    static __device__ __forceinline__ void keep(P &v, int64_t c, int64_t hidden)
    {
        if constexpr (!kWide) {
            if (c >= 0 && c + N <= hidden) return;
#pragma unroll
            for (int i = 0; i < N; i++)
                if (c + i < 0 || c + i >= hidden) v.set_bits(i, 0);
        }
    }
    static __device__ __forceinline__ void store(const P &v, T *row, int64_t c, int64_t hidden)
    {
        if (kWide || (c >= 0 && c + N <= hidden)) {
            st_v4(row + c, make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]));
        } else {
#pragma unroll
            for (int i = 0; i < N; i++)
                if (c + i >= 0 && c + i < hidden && dbg_ok(row + c + i, sizeof(T), true))
                    *reinterpret_cast<typename P::Bits *>(row + c + i) = v.bits(i);
        }
    }
};

// Passes of up to `cap` rows over [lo, hi), hi at most 2^31 - 1: how many there are over `rows`
// rows, and the first row after the pass that starts at p0 (hi after the last).
__host__ __device__ __forceinline__ int pass_count(int rows, int cap) { return rows > 0 ? (rows - 1) / cap + 1 : 0; }
__host__ __device__ __forceinline__ int next_pass(int p0, int hi, int cap) { return hi - p0 > cap ? p0 + cap : hi; }

// True if every row of `hidden` values of `size` bytes, `ld` values apart, starts on a
// 16-byte boundary and is a whole number of 16-byte pieces.
static inline bool wide_rows(const void *p, int64_t hidden, int64_t ld, int size)
{
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && hidden * size % 16 == 0 && ld * size % 16 == 0;
}

}  // namespace bqk
