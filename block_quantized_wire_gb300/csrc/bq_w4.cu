// Products of a few rows with 4-bit weights: out[m, n] = sum over k of x[m, k] * c[n, k] *
// s[n, k / group], c a signed 4-bit code (two's complement, column 2i in the low half of
// byte i) and s one scale per `group` columns of a weight row.
//
// With few rows the weights are read once and used for little: at M rows 4 M operations
// per byte, so the memory would be the bound up to about 16 rows. What keeps the kernel from
// it is turning codes into numbers. One warp instruction per code would already be more than
// an SM issues at that rate, so the products run on the tensor cores: a code becomes an
// exact BF16 (FP16) integer in less than half an instruction, the 16 x 16 tiles of weights
// are the A operand of mma.m16n8k16, up to 8 rows of x are B, and the binary32 sums of a
// group are multiplied by its scale outside the mma. Sums are binary32 throughout (the mma may
// truncate where a binary32 addition would round); the output is rounded once. (The tcgen05
// products take no A operand of 4-bit integers and add all of a tile's groups into one
// accumulator; here each group needs its own sum.)
//
// What it measures: of one token's eight experts of 4096 x 7168 with groups of 32 (132 MB,
// 19.5 us at the copy rate) the copies alone take 25.8 us, the arithmetic alone 25.8 us, both
// together 32.1 us. 2 KB of codes cost a warp 385 (one row, group 128) to 475 instructions (16
// rows, group 32); the integer units, which run one warp instruction in two cycles, are busy 36
// to 53 % of the time, and a mma m16n8k16 takes eight cycles.
// Tried without gain: three CTAs an SM at 80 registers, rings of 2 to 4 steps, codes loaded a
// part ahead, a group's scaling one group late, the mma of one part between the widening of
// the next, shifts as high products (slower: four cycles each), x shared by a ring of its own.
#include <climits>

#include "bq_rows.cuh"

namespace bqk {
namespace {

// A warp's step is 2 KB of codes: kRowTiles tiles of 16 weight rows by 256 / kRowTiles
// columns. One tile makes items small and leaves registers for more warps; two tiles share
// each fragment of x between them.
constexpr int kStepCodeBytes = 2048;
constexpr int kW4Warps = kThreads / 32;
constexpr int kW4Stages = 3;  // steps of a warp's ring

// ---------------------------------------------------------------- codes to numbers
// Eight codes of a word -> four pairs of exact integers, pair i = codes (i, i + 4). The
// four bits, their sign bit flipped (which adds 8), become the low mantissa bits of a
// power of two whose ulp is 1, and one exact operation removes the power and the 8. (Numbers
// from the mantissa bits of a power of two: Y. J. Kim, R. Henry, R. Fahim, H. H. Awadalla, "Who
// Says Elephants Can't Run: Bringing Large Scale MoE Models into Cloud Scale Production", 2022.)
template <class T>
struct Codes;

// (w & mask) ^ x in one instruction
__device__ __forceinline__ uint32_t and_xor(uint32_t w, uint32_t mask, uint32_t x)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(r) : "r"(w), "r"(mask), "r"(x));
    return r;
}

// BF16 codes come out times 2^-12, so that no group's binary32 sum overflows where its
// product with the scale would not (128 codes of 8 times the largest BF16 value are 2^138);
// the sums of all groups are brought up again at the end. Both are exact; the smallest step of
// an output's sum is then 2^-137, a sixteenth of BF16's smallest value.
template <>
struct Codes<__nv_bfloat16> {
    static constexpr float kUp = 4096.0f;
    static __device__ __forceinline__ void widen(uint32_t w, uint32_t (&v)[4])
    {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t h = and_xor(w >> (4 * i), 0x000f000fu, 0x43084308u);  // 128 + 8 + c
            asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(v[i]) : "r"(h), "r"(0x39803980u), "r"(0xbd08bd08u));
        }
    }
    // c = a * b, or c += a * b
    template <bool kFirst>
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t *a, uint32_t b0, uint32_t b1)
    {
        if constexpr (kFirst)
            asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                "{%8, %9}, {%10, %10, %10, %10};"
                : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
        else
            asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                "{%8, %9}, {%0, %1, %2, %3};"
                : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

template <>
struct Codes<__half> {
    static constexpr float kUp = 1.0f;
    static __device__ __forceinline__ void widen(uint32_t w, uint32_t (&v)[4])
    {
        // The mantissa holds both codes of a byte: 1024 + 8 + c from the low one, 1024 + 16 (8 +
        // c) from the high one, whose sixteenth the fused multiply-add takes on its way.
        const uint32_t w8 = w >> 8;
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(v[0]) : "r"(and_xor(w, 0x000f000fu, 0x64086408u)), "r"(0x64086408u));
        asm("fma.rn.f16x2 %0, %1, %2, %3;"
            : "=r"(v[1]) : "r"(and_xor(w, 0x00f000f0u, 0x64806480u)), "r"(0x2c002c00u), "r"(0xd480d480u));
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(v[2]) : "r"(and_xor(w8, 0x000f000fu, 0x64086408u)), "r"(0x64086408u));
        asm("fma.rn.f16x2 %0, %1, %2, %3;"
            : "=r"(v[3]) : "r"(and_xor(w8, 0x00f000f0u, 0x64806480u)), "r"(0x2c002c00u), "r"(0xd480d480u));
    }
    // c = a * b, or c += a * b
    template <bool kFirst>
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t *a, uint32_t b0, uint32_t b1)
    {
        if constexpr (kFirst)
            asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                "{%8, %9}, {%10, %10, %10, %10};"
                : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
        else
            asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                "{%8, %9}, {%0, %1, %2, %3};"
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
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "r"(a)
                 : "memory");
    return r;
}

__device__ __forceinline__ void lds_v2(uint32_t a, uint32_t &x, uint32_t &y)
{
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(a) : "memory");
}

// Copies `bytes` of kSize bytes and fills the rest with zeros.
template <int kSize>
__device__ __forceinline__ void lane_copy_part(uint32_t dst, const void *src, int bytes)
{
    if (bytes > 0 && !dbg_ok(src, bytes, false)) bytes = 0;
    if constexpr (kSize == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kSize), "r"(bytes)
                     : "memory");
}

// Bytes into a warp's stage at which the 16 bytes (32 codes) c of weight row r lie. The
// 16-byte pieces of a 128-byte line (one row of 256 columns or two of 128) are permuted by
// the line's number, so that the eight rows that a mma fragment reads at once lie in
// different banks.
template <int kRowTiles>
__device__ __forceinline__ uint32_t code_at(int r, int c)
{
    if (kRowTiles == 1) return (uint32_t)(r * 128 + ((c ^ (r & 7)) * 16));
    return (uint32_t)((r >> 1) * 128 + (((r & 1) * 4 + (c ^ ((r >> 1) & 3))) * 16));
}

// code_at(r + i * (4 or 8 rows), c) from code_at(r, c), for the rows r < 4 (one tile) or
// r < 8 (two) that a warp's copy covers.
template <int kRowTiles>
__device__ __forceinline__ uint32_t code_row(uint32_t at, int i)
{
    return (kRowTiles == 1 ? at ^ (64 * (i & 1)) : at) + 512 * i;
}

// ---------------------------------------------------------------- scales
// A row's kCount scales of one step, copied as the 4-byte words that hold them: 16-bit
// scales of rows with odd strides may start in the upper half of their first word.
template <class S, int kCount>
struct Scales {
    static constexpr int kSize = sizeof(S);
    static constexpr int kBytes = kCount * kSize;  // 2 to 32
    static constexpr int kWords = (kBytes + 3) / 4;

    // p: the row's first scale of the step; valid: how many of kCount lie in the row
    static __device__ __forceinline__ void fetch(uint32_t dst, const S *p, int valid)
    {
        const uintptr_t a = reinterpret_cast<uintptr_t>(p), base = a & ~(uintptr_t)3;
        const int end = valid > 0 ? (int)(a - base) + valid * kSize : 0;  // valid bytes from base
#pragma unroll
        for (int i = 0; i < kWords + (kSize == 2 && kCount > 1 ? 1 : 0); i++) {
            const int left = end - 4 * i;
            lane_copy_part<4>(dst + 4 * i, reinterpret_cast<const char *>(base) + (left > 0 ? 4 * i : 0),
                              left < 0 ? 0 : left < 4 ? left : 4);
        }
    }

    // A whole step's scales without checks. align is that of pointers and strides, at most 16
    // bytes, 0 where words do not line up: a step is plain where it allows the largest copies.
    // (Choosing the copies by it in every step cost 3 %.) A single 16-bit scale comes with the
    // one it shares a word with, which must exist: rows of an even number of scales.
    static constexpr int kAlign = kBytes < 4 ? 4 : kBytes < 16 ? kBytes : 16;
    static __device__ __forceinline__ int align_of(const S *s, int64_t groups, int64_t ld, int64_t expert_ld)
    {
        const uint64_t strides = (uint64_t)(ld * kSize) | (uint64_t)(expert_ld * kSize);
        const uint64_t bits = reinterpret_cast<uintptr_t>(s) | strides | 16;
        const int align = (int)(bits & (0 - bits));
        return align < 4 || (kBytes < 4 && groups % 2 != 0) ? 0 : align;
    }
    template <int kCopy>
    static __device__ __forceinline__ void copies(uint32_t dst, const S *p)
    {
#pragma unroll
        for (int i = 0; i < kBytes / kCopy; i++) {
            if constexpr (kCopy == 16)
                lane_copy16(dst + 16 * i, reinterpret_cast<const char *>(p) + 16 * i);
            else
                lane_copy_part<kCopy>(dst + kCopy * i, reinterpret_cast<const char *>(p) + kCopy * i, kCopy);
        }
    }
    static __device__ __forceinline__ void fetch_plain(uint32_t dst, const S *p)
    {
        if constexpr (kBytes < 4)
            lane_copy_part<4>(dst, reinterpret_cast<const void *>(reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)3), 4);
        else
            copies<kAlign>(dst, p);
    }
    static __device__ __forceinline__ void fetch_words(uint32_t dst, const S *p, int align)
    {
        if (kBytes >= 8 && align == 8)
            copies<(kBytes < 8 ? 4 : 8)>(dst, p);
        else
            copies<4>(dst, p);
    }

    // a row's scales as copied, shifted into place where skewed
    static __device__ __forceinline__ void read(uint32_t src, uint32_t (&w)[kWords])
    {
        if constexpr (kWords >= 4) {
#pragma unroll
            for (int i = 0; i < kWords / 4; i++) {
                const uint4 v = lds_v4(src + 16 * i);
                w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
            }
        } else if constexpr (kWords == 2) {
            lds_v2(src, w[0], w[1]);
        } else {
            w[0] = lds_u32(src);
        }
    }
    static __device__ __forceinline__ void read_skewed(uint32_t src, int skew, uint32_t (&w)[kWords])
    {
        uint32_t low = lds_u32(src);
#pragma unroll
        for (int i = 0; i < kWords; i++) {
            const uint32_t high = lds_u32(src + 4 * i + 4);
            w[i] = __funnelshift_r(low, high, 16 * skew);
            low = high;
        }
    }
    static __device__ __forceinline__ float at(const uint32_t (&w)[kWords], int i)
    {
        if constexpr (kSize == 4)
            return __uint_as_float(w[i]);
        else
            return Value<S>::widen((uint16_t)(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu));
    }
};

// ---------------------------------------------------------------- kernel
// A CTA takes items of 16 * kRowTiles weight rows of one expert, over all columns and for
// every row of x that the expert has, kPassRows at a time. A warp walks every eighth step on
// its own, through its own ring of asynchronous copies, and the warps' sums are added in
// order at the end of an item. The ring runs on over the ends of items, so the memory is
// never idle in between.
//
// kPassRows is 8 per column tile of the mma, or 4: the rows then take the even columns of
// one tile, and half of the sums (the odd columns) need no scaling and no registers.
struct ExpertRows {
    int expert, lo, hi;
    int before;  // passes over a row block of the experts before this one
};

// Shared memory of a CTA where two stay resident on an SM (228 KB, of which each takes 1 KB
// more than it asks for, less the static part); staged rows of x fill what the rest leaves. A
// row is padded to whole steps.
constexpr int64_t kCtaBytes = 112 * 1024;
inline int64_t staged_row_bytes(int64_t k) { return (k + 255) / 256 * 512; }

template <class T_, class S_, int kGroup_, int kPassRows_, int kRowTiles_, bool kStaged_, bool kExperts_>
struct W4Shape {
    using T = T_;
    using S = S_;
    static constexpr int kGroup = kGroup_, kPassRows = kPassRows_, kRowTiles = kRowTiles_;
    static constexpr bool kStaged = kStaged_, kExperts = kExperts_;
    static constexpr bool kEven = kPassRows == 4;
    static constexpr int kTiles = kEven ? 1 : kPassRows / 8;
    static constexpr int kItemRows = 16 * kRowTiles;
    static constexpr int kStepCols = 256 / kRowTiles;
    static constexpr int kScaleSlot = kStepCols / kGroup * (int)sizeof(S) <= 8 ? 16 : kRowTiles == 1 ? 32 : 16;
    static constexpr int kStageBytes = kStepCodeBytes + kItemRows * kScaleSlot;
    static constexpr int kSumStride = kItemRows + 4;  // rows of x land in different banks
    static constexpr size_t kRingBytes = (size_t)kW4Warps * kW4Stages * kStageBytes;
    static constexpr size_t kSumBytes = sizeof(float) * kW4Warps * kPassRows * kSumStride;
};

template <class Shape>
__global__ void __launch_bounds__(kThreads, 2) matvec_w4_kernel(const __grid_constant__ W4Args a)
{
    using T = typename Shape::T;
    using S = typename Shape::S;
    using Bits = typename Value<T>::Bits;
    constexpr int kGroup = Shape::kGroup, kPassRows = Shape::kPassRows, kTiles = Shape::kTiles;
    constexpr int kRowTiles = Shape::kRowTiles, kStages = kW4Stages, kStageBytes = Shape::kStageBytes;
    constexpr int kItemRows = Shape::kItemRows, kSumStride = Shape::kSumStride;
    constexpr int kStepCols = Shape::kStepCols, kStepBytes = kStepCols / 2, kParts = kStepCols / 32;
    constexpr int kScaleCount = kStepCols / kGroup, kScaleSlot = Shape::kScaleSlot, kPerScale = kGroup / 32;
    constexpr bool kStaged = Shape::kStaged, kExperts = Shape::kExperts, kEven = Shape::kEven;
    using Sc = Scales<S, kScaleCount>;
    extern __shared__ __align__(128) unsigned char smem[];
    ExpertRows *const active = reinterpret_cast<ExpertRows *>(smem + Shape::kRingBytes + Shape::kSumBytes);
    unsigned char *const x_smem = smem + Shape::kRingBytes + Shape::kSumBytes +
                                  ((sizeof(ExpertRows) * a.n_experts + 15) & ~(size_t)15);
    __shared__ int warp_active[kW4Warps], warp_passes[kW4Warps];

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
    const int g = lane >> 2, t = lane & 3;  // mma fragment row (or column of C) and quad lane

    // rows of x a pass takes; staged rows are a whole number of passes, or less than one
    const int pass_cap = kStaged && a.staged_rows < kPassRows ? a.staged_rows : kPassRows;
    const int chunk_cap = kStaged ? a.staged_rows : INT_MAX;

    // The experts that have rows, in order, and the passes that a row block of each takes.
    // Offsets of a wrong plan are clamped.
    int n_active = 1, passes = 1;
    int kept = (int)a.slots;
    if constexpr (kExperts) {
        n_active = passes = 0;
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
            const int mine = pass_count(hi - lo, pass_cap);
            int upto = mine;  // passes of this warp's experts up to this one
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int up = __shfl_up_sync(kFull, upto, d);
                if (lane >= d) upto += up;
            }
            if (lane == 31) {
                warp_active[warp] = __popc(has);
                warp_passes[warp] = upto;
            }
            __syncthreads();
            int at = n_active, before = passes + upto - mine;
            for (int w = 0; w < kW4Warps; w++) {
                at += w < warp ? warp_active[w] : 0;
                before += w < warp ? warp_passes[w] : 0;
                n_active += warp_active[w];
                passes += warp_passes[w];
            }
            if (hi > lo) active[at + __popc(has & ((1u << lane) - 1u))] = ExpertRows{e, lo, hi, before};
            __syncthreads();
        }
    } else {
        if (threadIdx.x == 0) active[0] = ExpertRows{0, 0, (int)a.slots, 0};
        __syncthreads();
    }

    const int row_blocks = (int)((a.n + kItemRows - 1) / kItemRows);
    const int steps = (int)((a.k + kStepCols - 1) / kStepCols);
    const int whole_steps = (int)(a.k / kStepCols);
    const uint32_t ring = smem_u32(smem) + warp * (kStages * kStageBytes);
    float *sums = reinterpret_cast<float *>(smem + Shape::kRingBytes);
    // This CTA's run of items, of equal passes over row blocks for every CTA: an item belongs
    // to the run that its first pass falls in. CTAs are placed on the SMs in turn, so the runs
    // of one SM's CTAs follow one another and every SM's share is the same but for one item.
    const int sms = (int)gridDim.x / a.ctas_per_sm;
    const int64_t rank = (int64_t)(blockIdx.x % sms) * a.ctas_per_sm + blockIdx.x / sms;
    auto item_at = [&](int64_t cost) {  // the first item that starts at or past this many passes
        int lo = 0, hi = n_active;      // the last expert that starts before it
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if ((int64_t)active[mid].before * row_blocks <= cost)
                lo = mid;
            else
                hi = mid;
        }
        const int each = kExperts ? pass_count(active[lo].hi - active[lo].lo, pass_cap) : 1;
        const int64_t block = (cost - (int64_t)active[lo].before * row_blocks + each - 1) / each;
        return lo * row_blocks + (int)(block < row_blocks ? block : row_blocks);
    };
    const S *const scales = static_cast<const S *>(a.s);
    const int64_t costs = n_active > 0 ? (int64_t)passes * row_blocks : 0;
    const int item_lo = costs > 0 ? item_at(costs * rank / gridDim.x) : 0;
    const int item_hi = costs > 0 ? item_at(costs * (rank + 1) / gridDim.x) : 0;
    // 16-bit scales may start in mid-word: in some rows where strides are odd, in every second
    // step where a step has one
    const bool skewed = sizeof(S) == 2 && (kScaleCount == 1 || ((a.ld_s | a.expert_s) & 1));

    // The copying side of the ring: the next step to fetch. A lane copies the 16 bytes
    // f_col of the rows f_row + kLaneRows i, and row `lane`'s scales.
    constexpr int kPieces = kStepBytes / 16, kLaneRows = 32 / kPieces, kCopies = kItemRows / kLaneRows;
    const int f_row = lane / kPieces, f_col = lane % kPieces;
    int f_left = item_hi - item_lo;  // items to go, from this run's on
    int f_active = item_lo / row_blocks, f_first = item_lo - f_active * row_blocks;  // the run's expert, first block
    int f_end = 0, f_block = 0, f_rest = 0;    // the run's last block + 1; the block; rows of x from this chunk on
    int f_passes = 0, f_rows = 0, f_step = warp;
    int f_plain = 0;  // steps ahead that need no checks: whole steps of an item of whole rows
    uint32_t f_slot = ring;
    const uint8_t *f_q = nullptr;  // this lane's 16 bytes of the step
    const S *f_s = nullptr;        // this lane's first scale of the step
    const int64_t ld_rows = kLaneRows * a.ld_q;
    const uint32_t dst_code = code_at<kRowTiles>(f_row, f_col), dst_scale = kStepCodeBytes + lane * kScaleSlot;
    const int my_steps = steps > warp ? (steps - warp - 1) / kW4Warps + 1 : 0;
    const int align_s = Sc::align_of(scales, a.k / kGroup, a.ld_s, a.expert_s);
    const int my_plain = align_s >= Sc::kAlign && whole_steps > warp
                             ? (whole_steps - warp - 1) / kW4Warps + 1 : 0;
    auto chunk_passes = [&](int rest) { return pass_count(rest < chunk_cap ? rest : chunk_cap, pass_cap); };
    auto open_chunk = [&]() {  // the run's first block again
        const int64_t r0 = (int64_t)f_first * kItemRows, e = active[f_active].expert;
        f_block = f_first;
        f_passes = chunk_passes(f_rest);
        f_q = a.q + e * a.expert_q + (r0 + f_row) * a.ld_q + 16 * f_col + warp * kStepBytes;
        f_s = scales + e * a.expert_s + (r0 + lane) * a.ld_s + warp * kScaleCount;
    };
    auto open_run = [&]() {
        f_end = row_blocks - f_first < f_left ? row_blocks : f_first + f_left;
        f_rest = active[f_active].hi - active[f_active].lo;
        open_chunk();
    };
    auto open_rows = [&]() {  // and the pass over them
        const int r0 = f_block * kItemRows;
        f_rows = a.n - r0 < kItemRows ? (int)(a.n - r0) : kItemRows;
        f_step = warp;
        f_plain = f_rows == kItemRows ? my_plain : 0;
    };
    const int64_t back_q = (int64_t)my_steps * kW4Warps * kStepBytes;
    const int64_t back_s = (int64_t)my_steps * kW4Warps * kScaleCount;
    auto advance = [&]() {  // past a pass's last step
        f_q -= back_q;
        f_s -= back_s;
        if (--f_passes == 0) {
            f_q += kItemRows * a.ld_q;
            f_s += kItemRows * a.ld_s;
            f_passes = chunk_passes(f_rest);
            if (++f_block == f_end) {
                f_rest -= chunk_cap;
                if (f_rest > 0) {
                    open_chunk();
                } else {
                    f_left -= f_end - f_first;
                    if (f_left == 0) return;
                    f_first = 0;
                    f_active++;
                    open_run();
                }
            }
        }
        open_rows();
    };
    auto fetch = [&]() {
        if (f_step >= steps && f_left > 0) advance();
        if (f_plain > 0) {
            const uint8_t *q = f_q;
#pragma unroll
            for (int i = 0; i < kCopies; i++, q += ld_rows) lane_copy16(f_slot + code_row<kRowTiles>(dst_code, i), q);
            if (kItemRows == 32 || lane < kItemRows) Sc::fetch_plain(f_slot + dst_scale, f_s);
            f_plain--;
            f_step += kW4Warps;
            f_q += kW4Warps * kStepBytes;
            f_s += kW4Warps * kScaleCount;
        } else if (f_left > 0 && f_step < steps) {
            const bool in_cols = f_step * kStepBytes + 16 * f_col < a.k / 2;
#pragma unroll
            for (int i = 0; i < kCopies; i++) {
                const bool in = in_cols && f_row + kLaneRows * i < f_rows;
                lane_copy_part<16>(f_slot + code_row<kRowTiles>(dst_code, i), in ? f_q + i * ld_rows : a.q,
                                   in ? 16 : 0);
            }
            const int left = (int)(a.k / kGroup) - f_step * kScaleCount;
            const bool in = lane < f_rows;
            if (kItemRows == 32 || lane < kItemRows) {
                if (align_s > 0 && in && left >= kScaleCount && Sc::kBytes >= 4)
                    Sc::fetch_words(f_slot + dst_scale, f_s, align_s);
                else
                    Sc::fetch(f_slot + dst_scale, in ? f_s : scales, !in ? 0 : left < kScaleCount ? left : kScaleCount);
            }
            f_step += kW4Warps;
            f_q += kW4Warps * kStepBytes;
            f_s += kW4Warps * kScaleCount;
        }
        lane_copy_commit();
        f_slot = f_slot == ring + (kStages - 1) * kStageBytes ? ring : f_slot + kStageBytes;
    };
    if (f_left > 0) {
        open_run();
        open_rows();
    }
#pragma unroll 1
    for (int i = 0; i < kStages - 1; i++) fetch();

    // Staged x: rows p0.. of one expert, in the pairs that the codes come in, zeros up to a
    // whole step. A single row is shared out over the CTA, more are taken by a warp each.
    auto stage_x = [&](int p0, int rows) {
        const int padded = steps * kStepCols;
        const bool split = rows == 1;
        const int first = 8 * (split ? (int)threadIdx.x : lane), stride = 8 * (split ? kThreads : 32);
        for (int r = split ? 0 : warp; r < rows; r += split ? 1 : kW4Warps) {
            int row = p0 + r;
            if (kExperts && a.order) row = dbg_ok(a.order + row, 4, false) ? __ldg(a.order + row) / a.top_k : 0;
            if (row < 0 || row >= a.x_rows) row = 0;  // a wrong plan
            const T *src = static_cast<const T *>(a.x) + row * a.ld_x;
#pragma unroll 4
            for (int c = first; c < padded; c += stride) {
                const uint4 v = c < a.k ? ld_keep_v4(src + c) : make_uint4(0, 0, 0, 0);
                const uint4 paired = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                                                __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
                *reinterpret_cast<uint4 *>(x_smem + (((c >> 5) * chunk_cap + r) * 4 + ((c >> 3) & 3)) * 16) = paired;
            }
        }
        __syncthreads();
    };
    uint32_t slot = ring;
    int left = item_hi - item_lo;
    int at = item_lo / row_blocks, first_block = item_lo - at * row_blocks;
    for (; left > 0; at++, first_block = 0) {
        const ExpertRows er = active[at];
        const int end_block = row_blocks - first_block < left ? row_blocks : first_block + left;
        left -= end_block - first_block;
        int next_chunk = er.lo;
        while (next_chunk < er.hi) {
            const int chunk = next_chunk;
            next_chunk = next_pass(chunk, er.hi, chunk_cap);
            if constexpr (kStaged) {
                __syncthreads();  // the readers of the rows before
                stage_x(chunk, next_chunk - chunk);
            }
            for (int block = first_block; block < end_block; block++) {
                const int r0 = block * kItemRows;
                // rows g + 8 i all start in the same half of a word
                const int row_skew = (int)(er.expert * a.expert_s + (r0 + g) * a.ld_s) & 1;
                for (int p0 = chunk, pass_rows; p0 < next_chunk; p0 += pass_rows) {
                    pass_rows = next_chunk - p0 < pass_cap ? next_chunk - p0 : pass_cap;
                    const int in_chunk = kStaged ? p0 - chunk : 0;
                    // This lane's rows of x, column g of each tile. Columns past the last row repeat
                    // it: their products are not stored.
                    const T *x[kTiles];
                    uint4 xv[kStaged ? 1 : kParts][kTiles];
                    uint32_t x_src = 0;
                    if constexpr (kStaged) {
                        const int r = kEven ? g / 2 : g;
                        const int last = pass_rows - 1;
                        const int row = in_chunk + (r < last ? r : last);
                        x_src = smem_u32(x_smem) + ((warp * kParts * chunk_cap + row) * 4 + t) * 16;
                    }
#pragma unroll
                    for (int m = 0; m < (kStaged ? 0 : kTiles); m++) {
                        const int want = 8 * m + (kEven ? g / 2 : g), p = p0 + (want < pass_rows ? want : pass_rows - 1);
                        int row = p;
                        if (kExperts && a.order) row = dbg_ok(a.order + p, 4, false) ? __ldg(a.order + p) / a.top_k : 0;
                        if (row < 0 || row >= a.x_rows) row = 0;  // a wrong plan
                        x[m] = static_cast<const T *>(a.x) + row * a.ld_x + 8 * t + warp * kStepCols;
                    }
                    // x of a step is loaded at the end of the step before it
                    auto load_x = [&](int step) {
                        if constexpr (kStaged) return;
                        if (step < whole_steps) {
#pragma unroll
                            for (int j = 0; j < kParts; j++)
#pragma unroll
                                for (int m = 0; m < kTiles; m++) xv[kStaged ? 0 : j][m] = ld_keep_v4(x[m] + 32 * j);
                        } else if (step < steps) {
#pragma unroll
                            for (int j = 0; j < kParts; j++)
#pragma unroll
                                for (int m = 0; m < kTiles; m++)
                                    xv[kStaged ? 0 : j][m] = step * kStepCols + 32 * j < a.k
                                                                 ? ld_keep_v4(x[m] + 32 * j) : make_uint4(0, 0, 0, 0);
                        }
#pragma unroll
                        for (int m = 0; m < kTiles; m++) x[m] += kW4Warps * kStepCols;
                    };
                    load_x(warp);
                    float acc[kRowTiles][kTiles][4] = {};  // with even columns only, [0] and [2] are used
                    float c[kRowTiles][kTiles][4];
                    for (int step = warp; step < steps; step += kW4Warps) {
                        lane_copy_wait<kStages - 2>();
                        __syncwarp();
                        fetch();
                        // piece j of the rows g + 8 r: their lines are all permuted alike
                        const uint32_t src = slot + code_at<kRowTiles>(g, 0) + 4 * t;
                        const uint32_t src_s = slot + kStepCodeBytes + g * kScaleSlot;
                        uint32_t s[2 * kRowTiles][Sc::kWords];
                        if (skewed) {
                            const int skew = (row_skew + step * kScaleCount) & 1;
#pragma unroll
                            for (int i = 0; i < 2 * kRowTiles; i++)
                                Sc::read_skewed(src_s + 8 * kScaleSlot * i, skew, s[i]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 2 * kRowTiles; i++) Sc::read(src_s + 8 * kScaleSlot * i, s[i]);
                        }
#pragma unroll
                        for (int j = 0; j < kParts; j++) {
                            // the A fragments of two mma: rows g and g + 8 alternate
                            uint32_t codes[kRowTiles][8];
#pragma unroll
                            for (int r = 0; r < kRowTiles; r++) {
                                constexpr int kEightRows = 8 * kStepBytes;
                                uint32_t lo[4], hi[4];
                                Codes<T>::widen(lds_u32((src ^ (16 * j)) + 2 * kEightRows * r), lo);
                                Codes<T>::widen(lds_u32((src ^ (16 * j)) + 2 * kEightRows * r + kEightRows), hi);
#pragma unroll
                                for (int i = 0; i < 4; i++) {
                                    codes[r][2 * i] = lo[i];
                                    codes[r][2 * i + 1] = hi[i];
                                }
                            }
                            // codes i and i + 4 share a register, so x is paired the same way
                            uint32_t b[kTiles][4];
#pragma unroll
                            for (int m = 0; m < kTiles; m++) {
                                if constexpr (kStaged) {
                                    const uint4 v = lds_v4(x_src + j * 64 * chunk_cap);
                                    b[m][0] = v.x, b[m][1] = v.y, b[m][2] = v.z, b[m][3] = v.w;
                                } else {
                                    const uint4 v = xv[j][m];
                                    b[m][0] = __byte_perm(v.x, v.z, 0x5410), b[m][1] = __byte_perm(v.x, v.z, 0x7632);
                                    b[m][2] = __byte_perm(v.y, v.w, 0x5410), b[m][3] = __byte_perm(v.y, v.w, 0x7632);
                                }
                            }
#pragma unroll
                            for (int m = 0; m < kTiles; m++)
#pragma unroll
                                for (int r = 0; r < kRowTiles; r++)
                                    if (j % kPerScale == 0)
                                        Codes<T>::template mma<true>(c[r][m], codes[r], b[m][0], b[m][1]);
                                    else
                                        Codes<T>::template mma<false>(c[r][m], codes[r], b[m][0], b[m][1]);
#pragma unroll
                            for (int m = 0; m < kTiles; m++)
#pragma unroll
                                for (int r = 0; r < kRowTiles; r++)
                                    Codes<T>::template mma<false>(c[r][m], codes[r] + 4, b[m][2], b[m][3]);
                            if (j % kPerScale == kPerScale - 1) {
#pragma unroll
                                for (int r = 0; r < kRowTiles; r++) {
                                    const float s0 = Sc::at(s[2 * r], j / kPerScale);
                                    const float s1 = Sc::at(s[2 * r + 1], j / kPerScale);
#pragma unroll
                                    for (int m = 0; m < kTiles; m++)
#pragma unroll
                                        for (int i = 0; i < 4; i += kEven ? 2 : 1)
                                            acc[r][m][i] = __fmaf_rn(i < 2 ? s0 : s1, c[r][m][i], acc[r][m][i]);
                                }
                            }
                        }
                        if constexpr (kStaged)
                            x_src += kW4Warps * kParts * 64 * chunk_cap;
                        else
                            load_x(step + kW4Warps);
                        slot = slot == ring + (kStages - 1) * kStageBytes ? ring : slot + kStageBytes;
                    }
                    // the warps' sums: [warp][row of x][weight row]
                    __syncthreads();  // the readers of the item before
                    float *mine = sums + warp * kPassRows * kSumStride;
#pragma unroll
                    for (int r = 0; r < kRowTiles; r++)
#pragma unroll
                        for (int m = 0; m < kTiles; m++)
#pragma unroll
                            for (int i = 0; i < 4; i += kEven ? 2 : 1)
                                mine[(kEven ? t : 8 * m + 2 * t + (i & 1)) * kSumStride + 16 * r + g + 8 * (i >> 1)] =
                                    acc[r][m][i];
                    __syncthreads();
                    for (int i = threadIdx.x; i < pass_rows * kItemRows; i += kThreads) {
                        const int m = i / kItemRows, r = i % kItemRows;
                        if (r0 + r >= a.n) continue;
                        const float *of = sums + m * kSumStride + r;
                        float v = of[0];
#pragma unroll
                        for (int w = 1; w < kW4Warps; w++) v = __fadd_rn(v, of[w * kPassRows * kSumStride]);
                        if (Codes<T>::kUp != 1.0f) v = __fmul_rn(v, Codes<T>::kUp);
                        T *dst = static_cast<T *>(a.out) + (p0 + m) * a.ld_out + r0 + r;
                        if (dbg_ok(dst, sizeof(T), true)) *reinterpret_cast<Bits *>(dst) = Value<T>::round(v);
                    }
                }
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

template <class Shape>
cudaError_t launch_w4(W4Args a, cudaStream_t st)
{
    auto kernel = matvec_w4_kernel<Shape>;
    const int64_t blocks = (a.n + Shape::kItemRows - 1) / Shape::kItemRows;
    const int64_t with_rows = !Shape::kExperts ? 1 : a.slots < a.n_experts ? a.slots : a.n_experts;
    size_t smem = Shape::kRingBytes + Shape::kSumBytes + sizeof(ExpertRows) * a.n_experts;
    if (Shape::kStaged) smem = (smem + 15) / 16 * 16 + staged_row_bytes(a.k) * a.staged_rows;
    int grid = 0;
    if (cudaError_t e = grid_for((const void *)kernel, blocks * with_rows * kW4Warps, &grid, smem, kThreads))
        return e;
    int sms = 1;
    if (cudaError_t e = sm_count(&sms)) return e;
    a.ctas_per_sm = grid % sms == 0 ? grid / sms : 1;
    return launch_kernel_block(kernel, grid, kThreads, smem, st, a);
}

template <class T, class S, int kGroup, bool kExperts>
cudaError_t launch_w4_rows(W4Args a, int64_t rows, cudaStream_t st)
{
    // One 16-row tile a warp makes twice the items of half the steps: finer, each step dearer.
    // Rows of x staged in shared memory make the finer one's steps cheaper, for a round's worth of
    // setting up. The least of rounds (of two CTAs an SM) times steps (of a warp, and half a one
    // for an item's end) times what a step takes, by a fit to 409 shapes of 1 to 8 rows. In us, one
    // tile, two, staged:
    //   one row x 9728 x 7168, group 32: 12.1, 11.4, 12.0;  x 14592: 16.4, 18.9, 15.9
    //   one row x 36864 x 2048, group 128: 14.6, 12.4, 14.0;  x 1500 x 7168: 4.8, 6.4, 5.5
    //   one token's eight experts of 4096 x 7168, group 32: 36.3, 36.5, 32.1; 7168 x 2048: 25.4, 21.2, 21.5
    //   eight rows x 14592 x 7168, group 32: 17.8, 20.1;  x 9728 x 11264: 18.1, 16.6
    int sms = 1;
    if (cudaError_t e = sm_count(&sms)) return e;
    const int64_t used = !kExperts ? 1 : a.slots < a.n_experts ? a.slots : a.n_experts;
    auto half_steps = [&](int tiles) {
        const int64_t items = used * ((a.n + 16 * tiles - 1) / (16 * tiles)), ctas = 2 * sms;
        return ((items - 1) / ctas + 1) * (2 * ((a.k * tiles + 2047) / 2048) + 1);
    };
    const int64_t one_cost = 21 * half_steps(1), two_cost = 20 * half_steps(2), staged_cost = 18 * half_steps(1) + 40;
    using Staged = W4Shape<T, S, kGroup, 4, 1, true, kExperts>;
    const int64_t room = kCtaBytes - (int64_t)(Staged::kRingBytes + Staged::kSumBytes + sizeof(ExpertRows) * a.n_experts + 15);
    const int64_t cap = a.k > 0 && room > 0 ? room / staged_row_bytes(a.k) : 0;
    if (rows == 1 && cap >= 1 && staged_cost < one_cost && staged_cost < two_cost) {
        a.staged_rows = (int)(!kExperts ? 1 : cap < 4 ? cap : cap / 4 * 4);
        return launch_w4<Staged>(a, st);
    }
    const bool one = one_cost < two_cost;
    if (rows <= 4)
        return one ? launch_w4<W4Shape<T, S, kGroup, 4, 1, false, kExperts>>(a, st)
                   : launch_w4<W4Shape<T, S, kGroup, 4, 2, false, kExperts>>(a, st);
    if (rows <= 8)
        return one ? launch_w4<W4Shape<T, S, kGroup, 8, 1, false, kExperts>>(a, st)
                   : launch_w4<W4Shape<T, S, kGroup, 8, 2, false, kExperts>>(a, st);
    return launch_w4<W4Shape<T, S, kGroup, 16, 2, false, kExperts>>(a, st);
}

template <class T, class S, bool kExperts>
cudaError_t launch_w4_group(int group, const W4Args &a, cudaStream_t st)
{
    // the rows that a matrix is used for; with experts twice the average, for their spread
    const int64_t rows = kExperts ? (2 * a.slots + a.n_experts - 1) / a.n_experts : a.slots;
    switch (group) {
    case 32: return launch_w4_rows<T, S, 32, kExperts>(a, rows, st);
    case 64: return launch_w4_rows<T, S, 64, kExperts>(a, rows, st);
    default: return launch_w4_rows<T, S, 128, kExperts>(a, rows, st);
    }
}

template <class T, class S>
cudaError_t launch_w4_kind(int group, const W4Args &a, cudaStream_t st)
{
    return a.offsets ? launch_w4_group<T, S, true>(group, a, st) : launch_w4_group<T, S, false>(group, a, st);
}

// ---------------------------------------------------------------- quantize
// Per group: s = amax / 7 in binary32, rounded to the scale's type; code = the integer
// nearest to x / s (ties to even), within [-7, 7]; a group whose scale is 0 has codes 0.
// Weights are quantized once when a model is loaded: a lane takes eight columns, a group's
// lanes find its amax by shuffles. Bound by an IEEE division for each value: 16384 x 8192 BF16
// values take 174 us, 0.29 of the copy rate.
template <class T, class S, int kGroup>
__global__ void __launch_bounds__(kThreads)
quant_w4_kernel(const T *__restrict__ x, int64_t n, int64_t k, int64_t ld_x, uint8_t *__restrict__ q, int64_t ld_q,
                S *__restrict__ scales, int64_t ld_s)
{
    pdl_begin();
    dbg_begin();
    dbg_allow_2d(x, n, k * sizeof(T), ld_x * sizeof(T), false);
    dbg_allow_2d(q, n, k / 2, ld_q, true);
    dbg_allow_2d(scales, n, k / kGroup * sizeof(S), ld_s * sizeof(S), true);
    dbg_ready();
    using P = Piece<T>;
    const int64_t per_row = k / 8, units = n * per_row;
    const int64_t first = (int64_t)blockIdx.x * kThreads + (threadIdx.x & ~31u);
    for (int64_t w0 = first; w0 < units; w0 += (int64_t)gridDim.x * kThreads) {
        const int64_t u = w0 + (threadIdx.x & 31);
        const bool in = u < units;
        const int64_t row = in ? u / per_row : 0, c = in ? (u - row * per_row) * 8 : 0;
        float v[8] = {};
        if (in) {
#pragma unroll
            for (int i = 0; i < 8; i += P::N) {
                P piece;
                piece.put(ld_stream_v4(x + row * ld_x + c + i));
#pragma unroll
                for (int j = 0; j < P::N; j++) v[i + j] = piece.at(j);
            }
        }
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; i++) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
        for (int d = 1; d < kGroup / 8; d <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, d));
        const auto bits = Value<S>::round(__fdiv_rn(amax, 7.0f));
        const float s = Value<S>::widen(bits);
        uint32_t word = 0;
        if (s > 0.0f) {
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float code = fminf(fmaxf(rintf(__fdiv_rn(v[i], s)), -7.0f), 7.0f);
                word |= ((uint32_t)(int)code & 15u) << (4 * i);
            }
        }
        if (in) {
            st_u32(q + row * ld_q + c / 2, word);
            S *dst = scales + row * ld_s + c / kGroup;
            if (c % kGroup == 0 && dbg_ok(dst, sizeof(S), true))
                *reinterpret_cast<typename Value<S>::Bits *>(dst) = bits;
        }
    }
}

template <class T, class S, int kGroup>
cudaError_t launch_quant(const void *x, int64_t n, int64_t k, int64_t ld_x, uint8_t *q, int64_t ld_q, void *scales,
                         int64_t ld_s, cudaStream_t st)
{
    auto kernel = quant_w4_kernel<T, S, kGroup>;
    int grid = 0;
    if (cudaError_t e = grid_for((const void *)kernel, (n * (k / 8) + 31) / 32, &grid)) return e;
    return launch_kernel(kernel, grid, st, static_cast<const T *>(x), n, k, ld_x, q, ld_q, static_cast<S *>(scales),
                         ld_s);
}

template <class T, class S, typename... Args>
cudaError_t launch_quant_group(int group, Args... args)
{
    return group == 32 ? launch_quant<T, S, 32>(args...) : group == 64 ? launch_quant<T, S, 64>(args...)
                                                                       : launch_quant<T, S, 128>(args...);
}

template <class T, typename... Args>
cudaError_t launch_quant_scale(int scale_type, Args... args)
{
    return scale_type == kBf16  ? launch_quant_group<T, __nv_bfloat16>(args...)
           : scale_type == kF16 ? launch_quant_group<T, __half>(args...)
                                : launch_quant_group<T, float>(args...);
}

}  // namespace

cudaError_t launch_quant_w4(int type, int scale_type, int group, const void *x, int64_t n, int64_t k, int64_t ld_x,
                            uint8_t *q, int64_t ld_q, void *scales, int64_t ld_s, cudaStream_t st)
{
    switch (type) {
    case kBf16: return launch_quant_scale<__nv_bfloat16>(scale_type, group, x, n, k, ld_x, q, ld_q, scales, ld_s, st);
    case kF16: return launch_quant_scale<__half>(scale_type, group, x, n, k, ld_x, q, ld_q, scales, ld_s, st);
    default: return launch_quant_scale<float>(scale_type, group, x, n, k, ld_x, q, ld_q, scales, ld_s, st);
    }
}

cudaError_t launch_matvec_w4(int x_type, int scale_type, int group, const W4Args &a, cudaStream_t st)
{
    if (x_type == kBf16)
        return scale_type == kF32 ? launch_w4_kind<__nv_bfloat16, float>(group, a, st)
                                  : launch_w4_kind<__nv_bfloat16, __nv_bfloat16>(group, a, st);
    return scale_type == kF32 ? launch_w4_kind<__half, float>(group, a, st)
                              : launch_w4_kind<__half, __half>(group, a, st);
}

cudaError_t read_wait_counters_w4(unsigned long long (&v)[3]) { return read_wait_counters(v); }

}  // namespace bqk
