// Rows of keys and values into a cache's 4-bit pages, and back.
//
// Both kernels are one pass: a lane takes 16 values of a row (32 bytes, one 256-bit access where
// the rows allow it) and their 8 bytes of codes; a group's 2, 4 or 8 lanes share its pair. K and V of
// all tokens are one run of such units, so that a decode step's few tokens still spread over lanes
// and SMs and need one launch.
#include "bq_kv4.cuh"

namespace bqk {
namespace {

__device__ __forceinline__ uint32_t divide(uint32_t n, const Divisor &d) { return (__umulhi(n, d.mul) + n) >> d.shift; }

struct RowUnits {
    Kv4Cache c;
    Kv4Rows k, v;
    Kv4Slots slots;
    int64_t tokens, n_slots;
    uint32_t units;         // of K and V together: tokens * 2 * heads * per_row
    Divisor per_row, heads, page;
};

// Where unit u lies: its row beside the cache, and in the cache.
template <class T>
struct Place {
    T *row;
    uint8_t *codes;
    unsigned char *pair;
    bool held;

    __device__ __forceinline__ Place(const RowUnits &a, uint32_t u)
    {
        const uint32_t r = divide(u, a.per_row), piece = u - r * a.per_row.d;
        const uint32_t both = divide(r, a.heads), head = r - both * a.heads.d;
        const uint32_t token = both >> 1;
        const bool values = both & 1;
        const Kv4Rows &rows = values ? a.v : a.k;
        row = static_cast<T *>(rows.p) + token * rows.ld_token + head * rows.ld_head + 16 * piece;
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
            page = divide((uint32_t)slot, a.page);
            in_page = (uint32_t)slot - (uint32_t)page * a.page.d;
        } else {
            page = slot / a.c.page;
            in_page = (uint32_t)(slot - page * a.c.page);
        }
        const int64_t at = page * a.c.page_stride + head * a.c.head_stride + (int64_t)in_page * a.c.token_stride;
        const int64_t at_s = page * a.c.page_stride_s + head * a.c.head_stride_s + (int64_t)in_page * a.c.token_stride_s;
        codes = (values ? a.c.v : a.c.k) + at + 8 * piece;
        pair = (values ? a.c.v_scales : a.c.k_scales) + at_s + 4 * (16 * piece / a.c.group);
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
// The code of x is the integer nearest to fl(d / s), d = fl(x - offset). d * fl(1 / s) is within 2^-21
// of that quotient (|quotient| < 32, or it is clamped), so wherever it lies more than 1e-4 from a tie
// both round alike; only nearer values take the division. Below 2^-100 the reciprocal or its product
// could leave the normal range: every value divides there.
constexpr float kRound = 12582912.0f;  // 1.5 * 2^23: adding it rounds to the nearest integer
constexpr float kNearTie = 0.4999f;

__device__ __forceinline__ float exact_code(float d, float s)  // kRound + code
{
    return __fadd_rn(fminf(fmaxf(rintf(__fdiv_rn(d, s)), -8.0f), 7.0f), kRound);
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
        uint4 lo4, hi4;
        if constexpr (kV8) {
            ld_stream_v8(at.row, lo4, hi4);
        } else {
            lo4 = ld_stream_v4(at.row);
            hi4 = ld_stream_v4(at.row + 8);
        }
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
        auto s_bits = Value<T>::round(__fdiv_rn(__fsub_rn(high, low), 15.0f));
        float s = Value<T>::widen(s_bits);
        auto z_bits = Value<T>::round(__fadd_rn(__fadd_rn(low, 4.0f * s), 4.0f * s));
        const float z = Value<T>::widen(z_bits);
        if (!(s <= 3.0e38f)) s_bits = z_bits = 0x7fffu, s = 0.0f;  // infinity or NaN: a NaN of both types
        uint32_t w[16];
        if (s > 0.0f) {
            const float inv = __frcp_rn(s);
            const float2 neg_z = splat(-z), r = splat(inv), up = splat(kRound), down = splat(-kRound);
            float far = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float2 v = make_float2(Value<T>::widen((uint16_t)(x[i] & 0xffffu)), Value<T>::widen((uint16_t)(x[i] >> 16)));
                float2 t = mul2(add2(v, neg_z), r);
                t = make_float2(fminf(fmaxf(t.x, -8.0f), 7.0f), fminf(fmaxf(t.y, -8.0f), 7.0f));
                const float2 n = add2(t, up), back = add2(n, down);
                const float2 off = add2(t, make_float2(-back.x, -back.y));
                far = max3f(far, fabsf(off.x), fabsf(off.y));
                w[2 * i] = __float_as_uint(n.x);
                w[2 * i + 1] = __float_as_uint(n.y);
            }
            if (far > kNearTie || s < 0x1p-100f) {
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    const float v = Value<T>::widen((uint16_t)(i & 1 ? x[i / 2] >> 16 : x[i / 2] & 0xffffu));
                    w[i] = __float_as_uint(exact_code(__fsub_rn(v, z), s));
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; i++) w[i] = 0;
        }
        uint32_t codes[2];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const uint32_t even = pack_low_bytes(w[8 * i], w[8 * i + 2], w[8 * i + 4], w[8 * i + 6]);
            const uint32_t odd = pack_low_bytes(w[8 * i + 1], w[8 * i + 3], w[8 * i + 5], w[8 * i + 7]);
            codes[i] = (even & 0x0f0f0f0fu) | ((odd << 4) & 0xf0f0f0f0u);
        }
        if (in && at.held) {
            st_v2(at.codes, make_uint2(codes[0], codes[1]));
            if (((u0 + lane) & (kGroup / 16 - 1)) == 0) st_u32(at.pair, (uint32_t)s_bits | ((uint32_t)z_bits << 16));
        }
    }
}

// ---------------------------------------------------------------- read
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
        uint32_t out[8] = {};
        if (at.held) {
            const uint2 codes = ld_stream_v2(at.codes);
            const float2 pair = pair_values<T>(dbg_ok(at.pair, 4, false) ? __ldg(reinterpret_cast<const uint32_t *>(at.pair)) : 0u);
            const float2 s = splat(pair.x), z = splat(pair.y), bias = splat(-8388616.0f);  // -(2^23 + 8)
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const uint32_t two = (i < 4 ? codes.x : codes.y) >> (8 * (i & 3));
                // 2^23 + 8 + code from the code's four bits, the sign bit flipped
                float2 c = make_float2(__uint_as_float((two & 0xfu) ^ 0x4b000008u),
                                       __uint_as_float(((two >> 4) & 0xfu) ^ 0x4b000008u));
                c = fma2(add2(c, bias), s, z);
                out[i] = Value<T>::round2(c.x, c.y);
            }
        }
        if constexpr (kV8) {
            st_v8(at.row, make_uint4(out[0], out[1], out[2], out[3]), make_uint4(out[4], out[5], out[6], out[7]));
        } else {
            st_v4(at.row, make_uint4(out[0], out[1], out[2], out[3]));
            st_v4(at.row + 8, make_uint4(out[4], out[5], out[6], out[7]));
        }
    }
}

RowUnits units_of(const Kv4Cache &c, const Kv4Rows &k, const Kv4Rows &v, int64_t tokens, const Kv4Slots &slots)
{
    RowUnits a = {};
    a.c = c, a.k = k, a.v = v, a.slots = slots, a.tokens = tokens, a.n_slots = c.pages * c.page;
    a.units = (uint32_t)(tokens * 2 * c.heads * (c.head_dim / 16));
    a.per_row = divisor((uint32_t)(c.head_dim / 16)), a.heads = divisor((uint32_t)c.heads);
    a.page = divisor((uint32_t)c.page);
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
