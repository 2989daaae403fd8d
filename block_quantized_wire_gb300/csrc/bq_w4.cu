// Products of a few rows with 4-bit weights: out[m, n] = sum over k of x[m, k] * c[n, k] *
// s[n, k / group], c a signed 4-bit code (two's complement, column 2i in the low half of
// byte i) and s one scale per `group` columns of a weight row.
//
// With few rows the weights are read once and used for little: at M rows 4 M operations
// per byte, so the bound is the memory's rate up to about 16 rows. What has to be kept
// off the critical path is turning codes into numbers. One warp instruction per code
// would already be more than an SM issues at that rate, so the products run on the
// tensor cores: a code becomes an exact BF16 (FP16) integer in half an instruction, the
// 16 x 16 tiles of weights are the A operand of mma.m16n8k16, up to 8 rows of x are B,
// and the binary32 sums of a group are multiplied by its scale outside the mma. Sums are
// binary32 throughout; the output is rounded once.
#include "bq_rows.cuh"

namespace bqk {
namespace {

constexpr int kW4Warps = kThreads / 32;
constexpr int kRowTiles = 2;                 // 16-row tiles per warp
constexpr int kWarpRows = 16 * kRowTiles;    // weight rows per warp
constexpr int kStepCols = 128;               // columns per warp and step
constexpr int kW4Stages = 4;                 // steps in flight per warp
constexpr int kCodeBytes = kWarpRows * kStepCols / 2;
constexpr int kScaleSlot = 16;               // bytes per weight row and step: at most 4 FP32 scales
constexpr int kStageBytes = kCodeBytes + kWarpRows * kScaleSlot;

// ---------------------------------------------------------------- codes to numbers
// Eight codes of a word -> four pairs of exact integers, pair i = codes (i, i + 4). The
// four bits, their sign bit flipped (which adds 8), become the low mantissa bits of a
// power of two whose ulp is 1, and one exact subtraction removes the power and the 8.
template <class T>
struct Codes;

template <>
struct Codes<__nv_bfloat16> {
    static __device__ __forceinline__ void widen(uint32_t w, uint32_t (&v)[4])
    {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t h = ((w >> (4 * i)) & 0x000f000fu) ^ 0x43084308u;  // 128 + 8 + c
            asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(v[i]) : "r"(h), "r"(0x43084308u));
        }
    }
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
    {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

template <>
struct Codes<__half> {
    static __device__ __forceinline__ void widen(uint32_t w, uint32_t (&v)[4])
    {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t h = ((w >> (4 * i)) & 0x000f000fu) ^ 0x64086408u;  // 1024 + 8 + c
            asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(v[i]) : "r"(h), "r"(0x64086408u));
        }
    }
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
    {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

// ---------------------------------------------------------------- shared memory
__device__ __forceinline__ uint32_t lds_u32(uint32_t a)
{
    uint32_t r;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a) : "memory");
    return r;
}

__device__ __forceinline__ uint4 lds_v4(uint32_t a)
{
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
    return r;
}

// Copies `bytes` of kSize bytes and fills the rest with zeros.
template <int kSize>
__device__ __forceinline__ void lane_copy_part(uint32_t dst, const void *src, int bytes)
{
    if (bytes > 0 && !dbg_ok(src, bytes, false)) bytes = 0;
    if constexpr (kSize == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kSize), "r"(bytes) : "memory");
}

// Bytes into a warp's stage at which the 16 bytes (32 codes) c of weight row r lie. Two
// 64-byte rows share a 128-byte line, and the four pieces of a row are permuted by the
// line's number, so that the eight rows that a mma fragment reads at once lie in
// different banks.
__device__ __forceinline__ uint32_t code_at(int r, int c)
{
    return (uint32_t)((r >> 1) * 128 + (((r & 1) * 4 + (c ^ ((r >> 1) & 3))) * 16));
}

// ---------------------------------------------------------------- scales
// A row's scales of one step: 128 / group values, copied as the 4-byte words that hold
// them. `skew` is 1 where 16-bit scales start in the upper half of their first word.
template <class S, int kGroup>
struct Scales {
    static constexpr int kCount = kStepCols / kGroup;
    static constexpr int kSize = sizeof(S);

    // p: the row's first scale of the step; valid: how many of kCount lie in the row
    static __device__ __forceinline__ void fetch(uint32_t dst, const S *p, int valid)
    {
        const uintptr_t a = reinterpret_cast<uintptr_t>(p), base = a & ~(uintptr_t)3;
        const int end = valid > 0 ? (int)(a - base) + valid * kSize : 0;  // valid bytes from base
        constexpr int kWords = (kCount * kSize + 3) / 4;
        if constexpr (kWords == 4) {
            if ((a & 15) == 0) return lane_copy_part<16>(dst, p, end);
        }
        if constexpr (kWords == 2) {
            if ((a & 7) == 0) return lane_copy_part<8>(dst, p, end);
        }
        constexpr int kMost = kWords + (kSize == 2 && kCount > 1 ? 1 : 0);
#pragma unroll
        for (int i = 0; i < kMost; i++) {
            const int left = end - 4 * i;
            lane_copy_part<4>(dst + 4 * i, reinterpret_cast<const char *>(base) + (left > 0 ? 4 * i : 0),
                              left < 0 ? 0 : left < 4 ? left : 4);
        }
    }

    static __device__ __forceinline__ float widen16(uint32_t h) { return Value<S>::widen((uint16_t)h); }

    static __device__ __forceinline__ void read(uint32_t src, int skew, float (&v)[kCount])
    {
        const uint4 w4 = lds_v4(src);
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
        if constexpr (kSize == 4) {
#pragma unroll
            for (int i = 0; i < kCount; i++) v[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < kCount; i += 2) {
                const uint32_t pair = skew ? __funnelshift_r(w[i / 2], w[i / 2 + 1], 16) : w[i / 2];
                v[i] = widen16(pair & 0xffffu);
                if (i + 1 < kCount) v[i + 1] = widen16(pair >> 16);
            }
        }
    }
};

// ---------------------------------------------------------------- kernel
// A CTA takes items of kWarpRows * kRowWarps weight rows of one expert, over all columns
// and for every row of x that the expert has, kTiles * 8 rows at a time. Its warps are
// kRowWarps in the rows times kColWarps in the columns: a warp walks every kColWarps-th
// step of 128 columns on its own, through its own ring of asynchronous copies, and the
// column warps' sums are added in order at the end of an item. The ring runs on over the
// ends of items, so the memory is never idle in between.
struct ExpertRows {
    int expert, lo, hi;
};

template <class T, class S, int kGroup, int kTiles, int kRowWarps, bool kExperts>
__global__ void __launch_bounds__(kThreads, 2) matvec_w4_kernel(const __grid_constant__ W4Args a)
{
    constexpr int kColWarps = kW4Warps / kRowWarps;
    constexpr int kItemRows = kWarpRows * kRowWarps;
    constexpr int kPassRows = 8 * kTiles;
    constexpr int kSumStride = kItemRows + 4;
    constexpr int kPerScale = kGroup / 32;
    using Sc = Scales<S, kGroup>;
    using Bits = typename Value<T>::Bits;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ ExpertRows active[kExperts ? kMaxExperts : 1];
    __shared__ int warp_active[kW4Warps + 1];

    pdl_begin();
    dbg_begin();
    dbg_allow_2d(a.x, a.x_rows, 2 * a.k, 2 * a.ld_x, false);
    dbg_allow(a.q, (a.n_experts - 1) * a.expert_q + (a.n - 1) * a.ld_q + a.k / 2, false);
    dbg_allow(a.s, sizeof(S) * ((a.n_experts - 1) * a.expert_s + (a.n - 1) * a.ld_s + a.k / kGroup), false);
    dbg_allow_2d(a.out, a.slots, 2 * a.n, 2 * a.ld_out, true);
    dbg_allow(a.offsets, kExperts ? 4ll * (a.n_experts + 1) : 0, false);
    dbg_allow(a.order, a.order ? 4 * a.slots : 0, false);
    dbg_ready();

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row_warp = warp / kColWarps, col_warp = warp % kColWarps;
    const int g = lane >> 2, t = lane & 3;  // mma fragment row (or column of C) and quad lane

    // The experts that have rows, in order. Offsets of a wrong plan are clamped.
    int n_active = 1;
    int kept = (int)a.slots;
    if constexpr (kExperts) {
        n_active = 0;
        const int slots = (int)a.slots;
        auto offset = [&](int e) {
            const int v = dbg_ok(a.offsets + e, 4, false) ? __ldg(a.offsets + e) : 0;
            return v < 0 ? 0 : v < slots ? v : slots;
        };
        kept = offset(a.n_experts);
        for (int base = 0; base < a.n_experts; base += kThreads) {
            const int e = base + threadIdx.x;
            const int lo = e < a.n_experts ? offset(e) : 0, hi = e < a.n_experts ? offset(e + 1) : 0;
            const unsigned has = __ballot_sync(kFull, hi > lo);
            if (lane == 0) warp_active[warp] = __popc(has);
            __syncthreads();
            int at = n_active;
            for (int w = 0; w < kW4Warps; w++) {
                at += w < warp ? warp_active[w] : 0;
                n_active += warp_active[w];
            }
            if (hi > lo) active[at + __popc(has & ((1u << lane) - 1u))] = ExpertRows{e, lo, hi};
            __syncthreads();
        }
    } else {
        if (threadIdx.x == 0) active[0] = ExpertRows{0, 0, (int)a.slots};
        __syncthreads();
    }

    const int row_blocks = (int)((a.n + kItemRows - 1) / kItemRows);
    const int64_t items = (int64_t)n_active * row_blocks;
    const int steps = (int)((a.k + kStepCols - 1) / kStepCols);
    const uint32_t ring = smem_u32(smem) + warp * (kW4Stages * kStageBytes);
    float *sums = reinterpret_cast<float *>(smem + kW4Warps * kW4Stages * kStageBytes);
    const S *const scales = static_cast<const S *>(a.s);

    // The copying side of the ring: the next step to fetch.
    int64_t f_item = blockIdx.x;
    int f_step = col_warp, f_pass = 0, f_passes = 0, f_slot = 0;
    const uint8_t *f_q = nullptr;
    const S *f_s = nullptr;
    int f_rows = 0;  // weight rows of this warp in the item
    auto open_item = [&]() {
        if (f_item < items) {
            const ExpertRows er = active[f_item / row_blocks];
            const int64_t r0 = (f_item % row_blocks) * kItemRows + row_warp * kWarpRows;
            f_q = a.q + er.expert * a.expert_q + r0 * a.ld_q;
            f_s = scales + er.expert * a.expert_s + r0 * a.ld_s;
            f_rows = a.n - r0 < kWarpRows ? (int)(a.n - r0) : kWarpRows;
            f_passes = (er.hi - er.lo + kPassRows - 1) / kPassRows;
        }
    };
    auto fetch = [&]() {
        if (f_item < items && f_step < steps) {
            const uint32_t dst = ring + f_slot * kStageBytes;
#pragma unroll
            for (int i = 0; i < kWarpRows * 4 / 32; i++) {
                const int r = (i * 32 + lane) >> 2, c = lane & 3;
                const int64_t byte = (int64_t)f_step * (kStepCols / 2) + 16 * c;
                const bool in = r < f_rows && byte < a.k / 2;
                lane_copy_part<16>(dst + code_at(r, c), in ? f_q + r * a.ld_q + byte : a.q, in ? 16 : 0);
            }
            const int g0 = f_step * Sc::kCount, left = (int)(a.k / kGroup) - g0;
            const bool in = lane < f_rows;
            Sc::fetch(dst + kCodeBytes + lane * kScaleSlot, in ? f_s + lane * a.ld_s + g0 : scales,
                      in ? (left < Sc::kCount ? left : Sc::kCount) : 0);
            f_step += kColWarps;
            if (f_step >= steps) {
                f_step = col_warp;
                if (++f_pass >= f_passes) {
                    f_pass = 0;
                    f_item += gridDim.x;
                    open_item();
                }
            }
        }
        lane_copy_commit();
        f_slot = f_slot + 1 == kW4Stages ? 0 : f_slot + 1;
    };
    open_item();
#pragma unroll
    for (int i = 0; i < kW4Stages - 1; i++) fetch();

    int slot = 0;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const ExpertRows er = active[item / row_blocks];
        const int64_t r0 = (item % row_blocks) * kItemRows;
        const int64_t warp_r0 = r0 + row_warp * kWarpRows;
        // which rows' 16-bit scales start in the upper half of a word
        int skew[2 * kRowTiles];
#pragma unroll
        for (int i = 0; i < 2 * kRowTiles; i++)
            skew[i] = sizeof(S) == 2 ? (int)((reinterpret_cast<uintptr_t>(scales + er.expert * a.expert_s +
                                                                          (warp_r0 + g + 8 * i) * a.ld_s) >> 1) & 1) : 0;
        for (int p0 = er.lo; p0 < er.hi; p0 += kPassRows) {
            const int pass_rows = er.hi - p0 < kPassRows ? er.hi - p0 : kPassRows;
            // this lane's rows of x: row g of each tile
            const T *x[kTiles];
#pragma unroll
            for (int m = 0; m < kTiles; m++) {
                const int p = p0 + 8 * m + g;
                int64_t row = -1;
                if (p < er.hi) {
                    row = p;
                    if (kExperts && a.order) row = dbg_ok(a.order + p, 4, false) ? __ldg(a.order + p) / a.top_k : -1;
                }
                x[m] = row >= 0 && row < a.x_rows ? static_cast<const T *>(a.x) + row * a.ld_x : nullptr;
            }
            float acc[kRowTiles][kTiles][4] = {};
            for (int step = col_warp; step < steps; step += kColWarps) {
                // x of the step: with one or two tiles fetched before the wait for the codes,
                // with more where it is used, because the registers do not hold it
                constexpr bool kEarly = kTiles <= 2;
                uint4 xv[kEarly ? 4 : 1][kTiles];
                auto fetch_x = [&](int j) {
                    const int64_t col = (int64_t)step * kStepCols + 32 * j + 8 * t;
#pragma unroll
                    for (int m = 0; m < kTiles; m++) {
                        uint4 &v = xv[kEarly ? j : 0][m];
                        v = make_uint4(0, 0, 0, 0);
                        if (x[m] && col < a.k && dbg_ok(x[m] + col, 16, false))
                            v = __ldg(reinterpret_cast<const uint4 *>(x[m] + col));
                    }
                };
                if constexpr (kEarly) {
#pragma unroll
                    for (int j = 0; j < 4; j++) fetch_x(j);
                }
                lane_copy_wait<kW4Stages - 2>();
                __syncwarp();
                fetch();
                const uint32_t src = ring + slot * kStageBytes;
                slot = slot + 1 == kW4Stages ? 0 : slot + 1;
                float s[2 * kRowTiles][Sc::kCount];
#pragma unroll
                for (int i = 0; i < 2 * kRowTiles; i++) {
                    // one 16-bit scale a step: its word's half changes from step to step
                    const int k = sizeof(S) == 2 && Sc::kCount == 1 ? skew[i] ^ (step & 1) : skew[i];
                    Sc::read(src + kCodeBytes + (g + 8 * i) * kScaleSlot, k, s[i]);
                }
                float c[kRowTiles][kTiles][4];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    // codes i and i + 4 share a register, so x is paired the same way
                    if constexpr (!kEarly) fetch_x(j);
                    uint32_t b[kTiles][4];
#pragma unroll
                    for (int m = 0; m < kTiles; m++) {
                        const uint4 v = xv[kEarly ? j : 0][m];
                        b[m][0] = __byte_perm(v.x, v.z, 0x5410);
                        b[m][1] = __byte_perm(v.x, v.z, 0x7632);
                        b[m][2] = __byte_perm(v.y, v.w, 0x5410);
                        b[m][3] = __byte_perm(v.y, v.w, 0x7632);
                    }
#pragma unroll
                    for (int r = 0; r < kRowTiles; r++) {
                        uint32_t lo[4], hi[4];
                        Codes<T>::widen(lds_u32(src + code_at(16 * r + g, j) + 4 * t), lo);
                        Codes<T>::widen(lds_u32(src + code_at(16 * r + g + 8, j) + 4 * t), hi);
                        const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
                        for (int m = 0; m < kTiles; m++) {
                            if (m > 0 && 8 * m >= pass_rows) continue;
                            if (j % kPerScale == 0) c[r][m][0] = c[r][m][1] = c[r][m][2] = c[r][m][3] = 0.0f;
                            Codes<T>::mma(c[r][m], a0, b[m][0], b[m][1]);
                            Codes<T>::mma(c[r][m], a1, b[m][2], b[m][3]);
                            if (j % kPerScale == kPerScale - 1) {
                                const float s0 = s[2 * r][j / kPerScale], s1 = s[2 * r + 1][j / kPerScale];
                                acc[r][m][0] = __fmaf_rn(s0, c[r][m][0], acc[r][m][0]);
                                acc[r][m][1] = __fmaf_rn(s0, c[r][m][1], acc[r][m][1]);
                                acc[r][m][2] = __fmaf_rn(s1, c[r][m][2], acc[r][m][2]);
                                acc[r][m][3] = __fmaf_rn(s1, c[r][m][3], acc[r][m][3]);
                            }
                        }
                    }
                }
            }
            // column warps' sums: [col warp][row of x][weight row]
            __syncthreads();
            float *mine = sums + col_warp * kPassRows * kSumStride + row_warp * kWarpRows;
#pragma unroll
            for (int r = 0; r < kRowTiles; r++)
#pragma unroll
                for (int m = 0; m < kTiles; m++)
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        mine[(8 * m + 2 * t + (i & 1)) * kSumStride + 16 * r + g + 8 * (i >> 1)] = acc[r][m][i];
            __syncthreads();
            for (int i = threadIdx.x; i < pass_rows * kItemRows; i += kThreads) {
                const int m = i / kItemRows, r = i % kItemRows;
                float v = sums[m * kSumStride + r];
#pragma unroll
                for (int w = 1; w < kColWarps; w++) v = __fadd_rn(v, sums[(w * kPassRows + m) * kSumStride + r]);
                T *dst = static_cast<T *>(a.out) + (p0 + m) * a.ld_out + r0 + r;
                if (r0 + r < a.n && dbg_ok(dst, sizeof(T), true)) *reinterpret_cast<Bits *>(dst) = Value<T>::round(v);
            }
        }
    }
    lane_copy_wait<0>();
    if constexpr (kExperts) {
        for (int64_t p = kept + blockIdx.x; p < a.slots; p += gridDim.x)
            for (int64_t c = threadIdx.x; c < a.n; c += kThreads) {
                T *dst = static_cast<T *>(a.out) + p * a.ld_out + c;
                if (dbg_ok(dst, sizeof(T), true)) *reinterpret_cast<Bits *>(dst) = 0;
            }
    }
}

template <class T, class S, int kGroup, int kTiles, int kRowWarps, bool kExperts>
cudaError_t launch_w4(const W4Args &a, cudaStream_t st)
{
    constexpr int kColWarps = kW4Warps / kRowWarps;
    constexpr size_t smem = kW4Warps * kW4Stages * kStageBytes +
                            sizeof(float) * kColWarps * 8 * kTiles * (kWarpRows * kRowWarps + 4);
    auto kernel = matvec_w4_kernel<T, S, kGroup, kTiles, kRowWarps, kExperts>;
    const int64_t blocks = (a.n + kWarpRows * kRowWarps - 1) / (kWarpRows * kRowWarps);
    const int64_t with_rows = !kExperts ? 1 : a.slots < a.n_experts ? a.slots : a.n_experts;
    int grid = 0;
    if (cudaError_t e = grid_for((const void *)kernel, blocks * with_rows * kW4Warps, &grid, smem)) return e;
    return launch_kernel_smem(kernel, grid, smem, st, a);
}

template <class T, class S, int kGroup>
cudaError_t launch_w4_rows(const W4Args &a, cudaStream_t st)
{
    if (a.offsets) {
        return a.slots <= 4 * (int64_t)a.n_experts ? launch_w4<T, S, kGroup, 1, 1, true>(a, st)
                                                   : launch_w4<T, S, kGroup, 4, 2, true>(a, st);
    }
    return a.slots <= 8 ? launch_w4<T, S, kGroup, 1, 1, false>(a, st) : launch_w4<T, S, kGroup, 4, 2, false>(a, st);
}

template <class T, class S>
cudaError_t launch_w4_group(int group, const W4Args &a, cudaStream_t st)
{
    switch (group) {
    case 32: return launch_w4_rows<T, S, 32>(a, st);
    case 64: return launch_w4_rows<T, S, 64>(a, st);
    default: return launch_w4_rows<T, S, 128>(a, st);
    }
}

}  // namespace

cudaError_t launch_matvec_w4(int x_type, int scale_type, int group, const W4Args &a, cudaStream_t st)
{
    if (x_type == kBf16)
        return scale_type == kF32 ? launch_w4_group<__nv_bfloat16, float>(group, a, st)
                                  : launch_w4_group<__nv_bfloat16, __nv_bfloat16>(group, a, st);
    return scale_type == kF32 ? launch_w4_group<__half, float>(group, a, st)
                              : launch_w4_group<__half, __half>(group, a, st);
}

cudaError_t read_wait_counters_w4(unsigned long long (&v)[3]) { return read_wait_counters(v); }

}  // namespace bqk
