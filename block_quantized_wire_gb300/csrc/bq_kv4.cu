// Rows of keys and values into a cache's 4-bit pages, and back.
//
// Both kernels are one pass: a lane takes 16 columns of a key and of its value (32 bytes each, one 256-bit access
// where the rows allow it) and their 8 bytes of codes; a group's 2, 4 or 8 lanes share its pair. Key and value lie at the same
// offsets of the cache, so that one slot is looked up and one place computed for both.
// Reading 65536 tokens of 8 heads of 128 columns takes 54 us, 6.3 TB/s; writing 32768 of them 34 us, 5.2 TB/s (BF16 and FP16 within
// 3 %). The write fills nothing: its schedulers issue in 61 % of their cycles, the integer pipe is busy in 52 %, and the first
// stall of its 29 warps an SM is for their loads.
#include <type_traits>

#include "bq_codes.cuh"
#include "bq_kv4.cuh"

namespace bqk {
namespace {

struct RowUnits {
    Kv4Cache c;
    Kv4Rows k, v;
    Kv4Slots slots;
    int64_t tokens, n_slots;
    uint32_t units;         // tokens * heads * per_row
    Divisor per_row, heads, page;
    int group_log2;
};

// Where unit u lies: its row beside the cache, and in the cache.
template <class T>
struct Place {
    T *row[2];           // of keys, of values
    uint8_t *codes[2];
    unsigned char *pair[2];
    bool held;

    __device__ __forceinline__ Place(const RowUnits &a, uint32_t u)
    {
        const uint32_t r = divide_by(u, a.per_row), piece = u - r * a.per_row.d;
        const uint32_t token = divide_by(r, a.heads), head = r - token * a.heads.d;
        row[0] = static_cast<T *>(a.k.p) + token * a.k.ld_token + head * a.k.ld_head + 16 * piece;
        row[1] = static_cast<T *>(a.v.p) + token * a.v.ld_token + head * a.v.ld_head + 16 * piece;
        int64_t slot = -1;
        if (a.slots.wide) {
            const int64_t *p = static_cast<const int64_t *>(a.slots.p) + token;
            if (dbg_ok(p, 8, false)) slot = __ldg(reinterpret_cast<const long long *>(p));
        } else {
            const int32_t *p = static_cast<const int32_t *>(a.slots.p) + token;
            if (dbg_ok(p, 4, false)) slot = __ldg(p);
        }
        held = slot >= 0 && slot < a.n_slots;
        if (!held) slot = 0;
        int64_t page;
        uint32_t in_page;
        if (a.n_slots < (1ll << 31)) {
            page = divide_by((uint32_t)slot, a.page);
            in_page = (uint32_t)slot - (uint32_t)page * a.page.d;
        } else {
            page = slot / a.c.page;
            in_page = (uint32_t)(slot - page * a.c.page);
        }
        const int64_t at = page * a.c.page_stride + head * a.c.head_stride + (int64_t)in_page * a.c.token_stride + 8 * piece;
        const int64_t at_s = page * a.c.page_stride_s + head * a.c.head_stride_s + (int64_t)in_page * a.c.token_stride_s +
                             4 * (16 * piece >> a.group_log2);
        codes[0] = a.c.k + at, codes[1] = a.c.v + at;
        pair[0] = a.c.k_scales + at_s, pair[1] = a.c.v_scales + at_s;
    }
};

// ---------------------------------------------------------------- smallest and largest
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b, __nv_bfloat16)
{
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, __nv_bfloat16)
{
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b, __half)
{
    uint32_t r;
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, __half)
{
    uint32_t r;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// ---------------------------------------------------------------- write
// The code of x is the integer nearest to fl(d / s), d = fl(x - offset). With r the reciprocal rounded to nearest and t = fl(d r),
// fl(t + r (d - t s)) is the correctly rounded quotient (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990: t is off by one unit in the last place at most, and d - t s is exact): two paired
// fused multiply-adds. BF16 rows have exact ties in half of all warps, so no shortcut around them pays: with a division
// for values near a tie 32768 tokens of 8 heads took 73 us, where this takes 37 (both a single cold launch under ncu).
// Below 2^-90 remainders could lose bits: every value divides there.
constexpr float kRound = 12582912.0f;  // 1.5 * 2^23: adding it rounds to the nearest integer

__device__ __forceinline__ float exact_code(float d, float s)  // kRound + code
{
    return __fadd_rn(fminf(fmaxf(rintf(__fdiv_rn(d, s)), -8.0f), 7.0f), kRound);
}

// fl(x / 15), likewise.
__device__ __forceinline__ float fifteenth(float x)
{
    constexpr float r = 1.0f / 15.0f;
    const float t = __fmul_rn(x, r);
    return x < 0x1p-90f ? __fdiv_rn(x, 15.0f) : __fmaf_rn(__fmaf_rn(t, -15.0f, x), r, t);
}

// A lane's 16 values, `lo4` the first 8, to codes; the group's pair.
template <class T, int kGroup>
__device__ __forceinline__ void quantize(const uint4 &lo4, const uint4 &hi4, uint2 &codes, uint32_t &pair)
{
    const uint32_t x[8] = {lo4.x, lo4.y, lo4.z, lo4.w, hi4.x, hi4.y, hi4.z, hi4.w};
    uint32_t lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < 8; i++) {
        lo = min2(lo, x[i], T());
        hi = max2(hi, x[i], T());
    }
#pragma unroll
    for (int d = 1; d < kGroup / 16; d <<= 1) {
        lo = min2(lo, __shfl_xor_sync(kFull, lo, d), T());
        hi = max2(hi, __shfl_xor_sync(kFull, hi, d), T());
    }
    lo = min2(lo, lo >> 16, T());
    hi = max2(hi, hi >> 16, T());
    const float low = Value<T>::widen((uint16_t)(lo & 0xffffu)), high = Value<T>::widen((uint16_t)(hi & 0xffffu));
    auto s_bits = Value<T>::round(fifteenth(__fsub_rn(high, low)));
    float s = Value<T>::widen(s_bits);
    auto z_bits = Value<T>::round(__fadd_rn(__fadd_rn(low, 4.0f * s), 4.0f * s));
    const float z = Value<T>::widen(z_bits);
    if (!(s <= 3.0e38f)) s_bits = z_bits = 0x7fffu, s = 0.0f;  // infinity or NaN: a NaN of both types
    uint32_t w[16];
    // Quotients run from -8 to 7 but for the roundings of s and of the offset. Where the offset is at most 32 s it is off by
    // s / 8 at most (BF16: 2^-8 of it), and a normal s by 2^-8 of itself: quotients stay between -8.13 and 7.19, and
    // their nearest integers in the range. Only warps with another group hold them to it.
    constexpr float kNormal = std::is_same<T, __half>::value ? 0x1p-14f : 0x1p-126f;
    const bool far = __any_sync(kFull, fabsf(z) > 32.0f * s || s < kNormal);
    const auto quotients = [&](auto held) {
        const float2 neg_z = splat(-z), r = splat(__frcp_rn(s)), neg_s = splat(-s), up = splat(kRound);
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float2 v = make_float2(Value<T>::widen((uint16_t)(x[i] & 0xffffu)), Value<T>::widen((uint16_t)(x[i] >> 16)));
            const float2 d = add2(v, neg_z), t = mul2(d, r);
            float2 q = fma2(fma2(t, neg_s, d), r, t);
            if constexpr (decltype(held)::value)
                q = make_float2(fminf(fmaxf(q.x, -8.0f), 7.0f), fminf(fmaxf(q.y, -8.0f), 7.0f));
            const float2 n = add2(q, up);
            w[2 * i] = __float_as_uint(n.x);
            w[2 * i + 1] = __float_as_uint(n.y);
        }
    };
    if (s >= 0x1p-90f) {
        if (far)
            quotients(std::true_type());
        else
            quotients(std::false_type());
    } else if (s > 0.0f) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const uint32_t two = x[i];
            w[2 * i] = __float_as_uint(exact_code(__fsub_rn(Value<T>::widen((uint16_t)(two & 0xffffu)), z), s));
            w[2 * i + 1] = __float_as_uint(exact_code(__fsub_rn(Value<T>::widen((uint16_t)(two >> 16)), z), s));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; i++) w[i] = 0;
    }
    uint32_t c[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const uint32_t even = pack_low_bytes(w[8 * i], w[8 * i + 2], w[8 * i + 4], w[8 * i + 6]);
        const uint32_t odd = pack_low_bytes(w[8 * i + 1], w[8 * i + 3], w[8 * i + 5], w[8 * i + 7]);
        c[i] = (even & 0x0f0f0f0fu) | ((odd << 4) & 0xf0f0f0f0u);
    }
    codes = make_uint2(c[0], c[1]);
    pair = (uint32_t)s_bits | ((uint32_t)z_bits << 16);
}

template <class T, int kGroup, bool kV8>
__global__ void __launch_bounds__(kThreads) kv4_write_kernel(const __grid_constant__ RowUnits a)
{
    pdl_begin();
    dbg_begin();
    dbg_cache(a.c, true);
    dbg_allow(a.k.p, 2 * ((a.tokens - 1) * a.k.ld_token + (a.c.heads - 1) * a.k.ld_head + a.c.head_dim), false);
    dbg_allow(a.v.p, 2 * ((a.tokens - 1) * a.v.ld_token + (a.c.heads - 1) * a.v.ld_head + a.c.head_dim), false);
    dbg_allow(a.slots.p, (a.slots.wide ? 8 : 4) * a.tokens, false);
    dbg_ready();
    const uint32_t first = blockIdx.x * kThreads + (threadIdx.x & ~31u), lane = threadIdx.x & 31;
    for (uint32_t u0 = first; u0 < a.units; u0 += gridDim.x * kThreads) {
        // lanes past the end repeat the last unit: a group's lanes are all there
        const bool in = u0 + lane < a.units;
        const Place<T> at(a, in ? u0 + lane : a.units - 1);
        uint4 lo[2], hi[2];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            if constexpr (kV8) {
                ld_stream_v8(at.row[i], lo[i], hi[i]);
            } else {
                lo[i] = ld_stream_v4(at.row[i]);
                hi[i] = ld_stream_v4(at.row[i] + 8);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; i++) {
            uint2 codes;
            uint32_t pair;
            quantize<T, kGroup>(lo[i], hi[i], codes, pair);
            if (in && at.held) {
                st_v2(at.codes[i], codes);
                if (((u0 + lane) & (kGroup / 16 - 1)) == 0) st_u32(at.pair[i], pair);
            }
        }
    }
}

// ---------------------------------------------------------------- read
// The 8 values of a word. Five codes lie within a binary32's mantissa as they are: with the exponent of 2^23 put above it, the
// four bits at place p are 2^23 + 16^p u, u = code + 8, and one exact addition leaves 16^p code, whose product with
// s / 16^p is code s, exact too (s of 16 bits is at least 2^-133). The last three come down by 20 places.
template <class T>
__device__ __forceinline__ void values_of(uint32_t word, const float2 (&s)[4], float2 z, uint32_t *out)
{
    constexpr float b0 = 8388608.0f + 8.0f, b1 = 8388608.0f + 128.0f, b2 = 8388608.0f + 2048.0f, b3 = 8388608.0f + 32768.0f,
                    b4 = 8388608.0f + 524288.0f;
    const uint32_t up = word >> 20;
    const auto at = [](uint32_t w, int p) { return __uint_as_float(and_xor(w, 0xfu << (4 * p), 0x4b000000u | 8u << (4 * p))); };
    const float2 c[4] = {add2(make_float2(at(word, 0), at(word, 1)), make_float2(-b0, -b1)),
                         add2(make_float2(at(word, 2), at(word, 3)), make_float2(-b2, -b3)),
                         add2(make_float2(at(word, 4), at(up, 0)), make_float2(-b4, -b0)),
                         add2(make_float2(at(up, 1), at(up, 2)), make_float2(-b1, -b2))};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 v = fma2(c[i], s[i], z);
        out[i] = Value<T>::round2(v.x, v.y);
    }
}

template <class T, bool kV8>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const __grid_constant__ RowUnits a)
{
    pdl_begin();
    dbg_begin();
    dbg_cache(a.c, false);
    dbg_allow(a.k.p, 2 * ((a.tokens - 1) * a.k.ld_token + (a.c.heads - 1) * a.k.ld_head + a.c.head_dim), true);
    dbg_allow(a.v.p, 2 * ((a.tokens - 1) * a.v.ld_token + (a.c.heads - 1) * a.v.ld_head + a.c.head_dim), true);
    dbg_allow(a.slots.p, (a.slots.wide ? 8 : 4) * a.tokens, false);
    dbg_ready();
    for (uint32_t u = blockIdx.x * kThreads + threadIdx.x; u < a.units; u += gridDim.x * kThreads) {
        const Place<T> at(a, u);
        uint2 codes[2] = {};
        uint32_t pairs[2] = {};
        if (at.held) {
#pragma unroll
            for (int i = 0; i < 2; i++) {
                codes[i] = ld_stream_v2(at.codes[i]);
                pairs[i] = dbg_ok(at.pair[i], 4, false) ? __ldg(reinterpret_cast<const uint32_t *>(at.pair[i])) : 0u;
            }
        }
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const float2 pair = pair_values<T>(pairs[i]), z = splat(pair.y), s0 = make_float2(pair.x, 0.0625f * pair.x);
            const float2 s[4] = {s0, mul2(s0, splat(0x1p-8f)), make_float2(0x1p-16f * pair.x, pair.x),
                                 make_float2(s0.y, 0x1p-8f * pair.x)};
            uint32_t out[8];  // pairs of zeros give zeros
            values_of<T>(codes[i].x, s, z, out);
            values_of<T>(codes[i].y, s, z, out + 4);
            if constexpr (kV8) {
                st_v8(at.row[i], make_uint4(out[0], out[1], out[2], out[3]), make_uint4(out[4], out[5], out[6], out[7]));
            } else {
                st_v4(at.row[i], make_uint4(out[0], out[1], out[2], out[3]));
                st_v4(at.row[i] + 8, make_uint4(out[4], out[5], out[6], out[7]));
            }
        }
    }
}

RowUnits units_of(const Kv4Cache &c, const Kv4Rows &k, const Kv4Rows &v, int64_t tokens, const Kv4Slots &slots)
{
    RowUnits a = {};
    a.c = c, a.k = k, a.v = v, a.slots = slots, a.tokens = tokens, a.n_slots = c.pages * c.page;
    a.units = (uint32_t)(tokens * c.heads * (c.head_dim / 16));
    a.per_row = divisor((uint32_t)(c.head_dim / 16)), a.heads = divisor((uint32_t)c.heads);
    a.page = divisor((uint32_t)c.page), a.group_log2 = c.group == 32 ? 5 : c.group == 64 ? 6 : 7;
    return a;
}

bool v8_rows(const Kv4Rows &r)
{
    return reinterpret_cast<uintptr_t>(r.p) % 32 == 0 && r.ld_token % 16 == 0 && r.ld_head % 16 == 0;
}

cudaError_t launch_rows(void (*kernel)(RowUnits), const RowUnits &a, cudaStream_t st)
{
    int grid = 0;
    if (cudaError_t e = grid_for((const void *)kernel, ((int64_t)a.units + 31) / 32, &grid)) return e;
    return launch_kernel(kernel, grid, st, a);
}

template <class T, bool kV8>
cudaError_t launch_write(const RowUnits &a, cudaStream_t st)
{
    return launch_rows(a.c.group == 32   ? kv4_write_kernel<T, 32, kV8>
                       : a.c.group == 64 ? kv4_write_kernel<T, 64, kV8>
                                         : kv4_write_kernel<T, 128, kV8>, a, st);
}

}  // namespace

cudaError_t launch_kv4_write(int type, const Kv4Cache &c, const Kv4Rows &k, const Kv4Rows &v, int64_t tokens,
                             const Kv4Slots &slots, cudaStream_t st)
{
    const RowUnits a = units_of(c, k, v, tokens, slots);
    const bool v8 = v8_rows(k) && v8_rows(v);
    if (type == kBf16) return v8 ? launch_write<__nv_bfloat16, true>(a, st) : launch_write<__nv_bfloat16, false>(a, st);
    return v8 ? launch_write<__half, true>(a, st) : launch_write<__half, false>(a, st);
}

cudaError_t launch_kv4_read(int type, const Kv4Cache &c, const Kv4Rows &k, const Kv4Rows &v, int64_t tokens,
                            const Kv4Slots &slots, cudaStream_t st)
{
    const RowUnits a = units_of(c, k, v, tokens, slots);
    const bool v8 = v8_rows(k) && v8_rows(v);
    if (type == kBf16)
        return launch_rows(v8 ? kv4_read_kernel<__nv_bfloat16, true> : kv4_read_kernel<__nv_bfloat16, false>, a, st);
    return launch_rows(v8 ? kv4_read_kernel<__half, true> : kv4_read_kernel<__half, false>, a, st);
}

cudaError_t read_wait_counters_kv4(unsigned long long (&v)[3]) { return read_wait_counters(v); }

}  // namespace bqk
