// Attention over a key-value cache in 4 bits: the kernel that streams the cache.
//
// Work. The positions of every (sequence, key-value head, chunk of up to kRows query rows) are cut
// into tiles of 32; all tiles of a call are one run that the CTAs take in equal shares, whatever the
// sequences' lengths, and a CTA's warps take its tiles in turn, each with a ring of stages of its
// own that cp.async fills across the borders of the pieces of work. A warp keeps a softmax reference and sums of
// its own; the warps are joined in shared memory, pieces that several CTAs share through the
// workspace by the kernel in bq_attend.cu.
//
// Products. With u = code + 8 (0 to 15) a key is s u + (z - 8 s), so a score is, per group of columns,
//     s <q, u> + (z - 8 s) sum q,
// and an output is  sum_t (p_t s_t) u_t - 8 sum_t (p_t s_t) + sum_t p_t z_t.  Both products run on
// m16n8k16 mma with FP16 operands and binary32 sums. u needs no conversion: four bits in the low mantissa bits of
// an FP16 are the subnormal u 2^-24 (u 2^-20 four bits higher), which the tensor cores take exactly, so that a word of
// eight codes costs five logic instructions. q is scaled by a power of two per row that brings its
// largest value to 2^14 .. 2^15, which FP16 then holds exactly down to 2^-28 of that. Only p s is rounded, to FP16
// (2^-11): it is used rounded in the sum over u and in the -8 correction (a mma with a constant matrix), so that
// u's offset does not enlarge that error. p's reference A takes in the size of s, p = 2^(y - A), A = max(y + log2 s) - 9
// or less over what the row sees, so that p s stays within 2^14, is exact to 2^-11 down to 2^-22 of the row's largest, and
// to 2^-33 of that below.
//
// Fragments. Codes are the m side of both products: tokens of the keys, columns of the values, which ldmatrix and its
// transposing form deliver as they lie. Scores come with tokens as rows and queries as columns; p s, rounded, is
// turned over by movmatrix into the n side of the second product. So up to 8 query rows cost half the mma that 16 do, and all
// that belongs to a query row (reference, sums, weights) lies in the lanes that hold its columns.
//
// What bounds it: the cache's bytes are the floor (144 a token and head at head_dim 128 and groups of 64), and a warp's chain of
// instructions that turn codes into operands comes next: 5 logic instructions for 8 codes, two cycles of a scheduler each, and an
// mma of eight cycles for 256 codes (twice that for more than 8 rows). No pipe is full: for 64 sequences of up to 8192 tokens a
// scheduler issues in 45 % of its cycles, the integer pipe is busy in 43 %, the tensor cores in 26 %, DRAM runs at 54 % of its
// nominal rate. With 216 registers a scheduler has two warps, and the first stall is an instruction's own latency. With the
// arithmetic taken out the copies ran at 6.9 TB/s, with the copies taken out the arithmetic at 5.9 TB/s of cache (each measured on a
// changed copy of the kernel), both together at 5.5; a call's ends (lengths, first tiles, joins) take about 11 us more. One
// sequence of 131072 tokens: 38 us; 64 of up to 8192: 74 us.
#pragma once

#include <cmath>
#include <type_traits>

#include "bq_codes.cuh"
#include "bq_kv4.cuh"

namespace bqk {

constexpr int kAttendWarps = 4, kAttendThreads = 32 * kAttendWarps;
constexpr int kTokens = 32;                       // of a tile
constexpr float kNothing = -3.0e38f;              // the reference of a row that has seen nothing
constexpr float kUnit = 0x1p-24f;                 // of a code held as an FP16's lowest mantissa bits
constexpr float kLift = 13.0f;                    // log2 that p s may have beside a fresh reference; one more before there is another
// The levels that references take in. Beyond them scales come up or down by a power of two that the sums of p s get back at the end,
// in every tile. References of one score then lie within 2^100 of each other, so that no factor between them is zero; a row's
// largest weight is 2^-71 or more, and what ex2.approx.ftz makes zero (below 2^-126) 2^-55 of it; 2^31 weights of 2^(14 - level) are
// 2^65. FP16's levels, -14 to 16, need none of that.
constexpr int kLowest = -20, kHighest = 80;
// A fresh reference leaves a row's largest p s so many places below kLift. A tile is looked at more closely where a p could pass the
// level, whatever its own s, and with less room that is more often: 64 sequences of up to 8192 BF16 tokens took 78.9 us with 0, 76.1
// with 1, 74.4 with 2, 72.5 with 4, 72.1 with 6 (before rows could be far, which costs about 1 us). But sums that a tile's products
// stand far above lose more where the tensor cores truncate: FP16 outputs (32 sequences of up to 4001, groups of 32), of whose
// relative error 2.07e-4 is their own rounding, were 2.15e-4 off with 0, 2.18e-4 with 2 (32.2 us) and 2.22e-4 with 4 (31.9 us).
// BF16's rounding, 1.66e-3, leaves no difference.
template <class T>
constexpr float kSlack = std::is_same<T, __half>::value ? 2.0f : 4.0f;
// A warp one of whose references reaches this size is far from there on: a reference could not hold what the size of s adds to a
// score. References are the largest scores themselves then, and scales come to within 2^kLift, up or down.
constexpr float kFar = 0x1p21f;
constexpr int kMaxAttendCtas = 456;               // three on each of 152 SMs

// What a call's kernels share beside its arguments.
struct AttendPlan {
    int rows, share, chunks, items;  // query rows and query heads of a key-value head; items = heads * chunks
    int ctas;                        // of the launch
    int words;                       // of the workspace that say which items are joined: one an item, or else one a CTA
    bool by_item;
    int page_tiles;                  // of a page, 0 where pages are no whole number of tiles
    Divisor by_share, by_page, by_chunks;  // by_page: tokens, or tiles where page_tiles > 0
};

// ---------------------------------------------------------------- the run of tiles
// First position that any query of sequence b looks at, and the end of the sequence.
__device__ __forceinline__ void sequence_range(const Kv4Cache &c, const Kv4Attend &a, int b, int &begin, int &end)
{
    const int cap = a.width * c.page;
    int length = dbg_ok(a.lengths + b, 4, false) ? __ldg(a.lengths + b) : 0;
    length = length < 0 ? 0 : length < cap ? length : cap;
    const int first = length - a.n_q + 1;  // end of the first query
    begin = a.window > 0 && first > a.window ? first - a.window : 0;
    end = length;
}
// Tiles begin at multiples of 32, so that a window's tiles lie in pages as all others do. A sequence without positions is one
// tile too: its rows are written.
__device__ __forceinline__ int first_of(int begin) { return begin & -kTokens; }
__device__ __forceinline__ int tiles_of(int begin, int end)
{
    return end > begin ? (end - first_of(begin) - 1) / kTokens + 1 : 1;
}

// What an item costs beside its tiles (its queries, the join of its warps), in tiles: chosen where 8 rows of 128 columns share a key
// head, and kept for all forms (64 sequences of up to 8192 tokens, when it was chosen: 78.7 us with 8, 76.0 with 12, 77.7 with 18).
constexpr int kSetup = 12;

// CTA i takes the run from i * per on. An item is kSetup places without a tile, then its tiles.
struct Share {
    int64_t total, per;
    int ctas;  // that take any
    __device__ __forceinline__ int64_t first(int cta) const { return cta < ctas ? cta * per : total; }
};
// Where a tile of the run lies.
struct Spot {
    int b, begin, end, tiles;  // sequence, its range and tiles
    int item;                  // head * chunks + chunk
    int tile;
    int64_t base;              // place of the item's tile 0, counted from the CTA's first
};

// Every CTA finds its share by itself, from the lengths: `spot` is where its first tile lies. All threads call it.
__device__ __forceinline__ void find_share(const Kv4Cache &c, const Kv4Attend &a, const AttendPlan &plan, Share &share, Spot &spot)
{
    __shared__ int64_t warp_sum[kAttendWarps];
    __shared__ Spot found;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int per = (a.batch - 1) / kAttendThreads + 1, b0 = a.batch / per < t ? a.batch : t * per;
    const int b1 = a.batch - b0 < per ? a.batch : b0 + per;
    int64_t mine = 0;
    int begin = 0, end = 0;
    for (int b = b0; b < b1; b++) {
        sequence_range(c, a, b, begin, end);
        mine += tiles_of(begin, end) + kSetup;
    }
    int64_t upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t other = __shfl_up_sync(kFull, upto, d);
        if (lane >= d) upto += other;
    }
    if (lane == 31) warp_sum[warp] = upto;
    __syncthreads();
    int64_t all = 0;
#pragma unroll
    for (int w = 0; w < kAttendWarps; w++) {
        if (w < warp) upto += warp_sum[w];
        all += warp_sum[w];
    }
    share.total = all * plan.items;
    if (share.total < 0x7fffffff) {  // divisions of 64 bits take long
        share.per = max(((uint32_t)share.total - 1) / (uint32_t)plan.ctas + 1, (uint32_t)kAttendWarps);
        share.ctas = (int)(((uint32_t)share.total - 1) / (uint32_t)share.per + 1);
    } else {
        share.per = (share.total - 1) / plan.ctas + 1;
        share.ctas = (int)((share.total - 1) / share.per + 1);
    }
    const int64_t target = share.first(min((int)blockIdx.x, share.ctas - 1));
    int64_t at = upto - mine;  // of one item before sequence b0
    if (target >= at * plan.items && target < upto * plan.items) {
        int b = b0;
        for (;; b++) {
            sequence_range(c, a, b, begin, end);
            const int n = tiles_of(begin, end);
            if (target < (at + n + kSetup) * plan.items) {
                const int64_t in = target - at * plan.items;
                const int cost = n + kSetup;
                const int item = in < 0x7fffffff ? (int)((uint32_t)in / (uint32_t)cost) : (int)(in / cost);
                const int off = (int)(in - (int64_t)item * cost);
                found = Spot{b, begin, end, n, item, off > kSetup ? off - kSetup : 0, kSetup - off};
                break;
            }
            at += n + kSetup;
        }
    }
    __syncthreads();
    spot = found;
}

// The workspace: words, then two partial sums a CTA (an item that began before its share, one that goes on after it):
// [kRows] references, [kRows] totals, [kRows][kDim] sums. Word i is item i's, written by the CTA that begins it, where
// a call has at most kMaxAttendCtas items; else CTA i's, for the item that goes on after its share. It says whose item, on how
// many shares, from which one.
__host__ __device__ __forceinline__ int64_t partial_floats(int rows, int dim) { return (int64_t)rows * (dim + 2); }
__host__ __device__ __forceinline__ float *partial_of(float *workspace, int cta, bool goes_on, int64_t floats)
{
    return workspace + 4 * kMaxAttendCtas + (2 * (int64_t)cta + goes_on) * floats;
}

// ---------------------------------------------------------------- constants of a form
template <int kDim_, int kGroup_, int kRows_>
struct Form {
    static constexpr int kDim = kDim_, kGroup = kGroup_, kRows = kRows_, kHalves = kRows / 8;
    static constexpr int kGroups = kDim / kGroup, kWords = kGroup / 32;  // code words of a lane in a group of keys
    static constexpr int kChunks = kDim / 32;                            // 16-byte pieces of a row of codes
    static constexpr int kCodeBytes = kDim == 192 ? 16 * (kTokens * 6 + kTokens / 4) : 16 * kTokens * kChunks;
    static constexpr int kPairBytes = kTokens * 4 * kGroups;
    static constexpr int kValid = 2 * (kCodeBytes + kPairBytes);  // a bit a token that is there
    static constexpr int kStage = kValid + 16;
    static constexpr int kJoin = 3 * 4 * kRows * (kDim + 2);
    // CTAs of an SM by their registers: 8 rows of 64 columns fit 168 a thread, all else up to 255, of which a few forms spill
    // (at most 208 bytes of stores and 276 of loads a thread: 16 rows of 128 columns with groups of 32 and 64, 8 rows of 192 and
    // 256 columns with groups of 32 and, of 256, 64). 8 rows of 128 columns with three CTAs (168, some spilled) took 77.3 us for 64
    // sequences of up to 8192 tokens where two took 74.6, with four (128) 85.7; the other forms were not tried with more.
    static constexpr int kCtas = kRows == 8 && kDim == 64 ? 3 : 2;
    static constexpr int kRoom = (227 * 1024 / kCtas - 1024 - 512 - kJoin) / (kAttendWarps * kStage);
    static constexpr int kStages = kRoom > 4 ? 4 : kRoom;
    static constexpr int kSmem = kJoin + kAttendWarps * kStages * kStage;
    static_assert(kStages >= 2, "a ring has two stages at least");
};

// 16-byte piece c of token t's row, in a stage: permuted so that a piece of eight tokens in a row lies in
// eight different groups of banks.
template <int kDim>
__host__ __device__ __forceinline__ int chunk_at(int t, int c)
{
    if (kDim == 192) return t * 6 + c + (t >> 2);
    const int key = kDim == 64 ? (t >> 2) & 1 : kDim == 128 ? (t >> 1) & 3 : t & 7;
    return t * (kDim / 32) + (c ^ key);
}

// ---------------------------------------------------------------- small steps
__device__ __forceinline__ float exp2_fast(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float power_of_2(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

// N pairs at a shared address, in the widest loads that its alignment (the largest power of two in 4 N bytes) allows.
template <int N>
__device__ __forceinline__ void lds_words(uint32_t at, uint32_t (&w)[N])
{
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 v = lds_v4(at + 4 * i);
            w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
        }
    } else if constexpr (N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 2) lds_v2(at + 4 * i, w[i], w[i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < N; i++) w[i] = lds_u32(at + 4 * i);
    }
}

__device__ __forceinline__ void sts_u16(uint32_t at, uint16_t v)
{
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(v) : "memory");
}

// 8x8 matrices of 16-bit elements, the row of lane 8 m + i row i of matrix m.
__device__ __forceinline__ void load_matrices(uint32_t at, uint32_t *v)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(at)
                 : "memory");
}
// An 8x8 matrix of 16-bit elements turned over its diagonal.
__device__ __forceinline__ uint32_t transposed(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ void load_transposed(uint32_t at, uint32_t (&v)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(at)
                 : "memory");
}

// Four 16-bit halves of codes -> four pairs of u in an FP16's lowest bits, the second and fourth 16 times as large.
__device__ __forceinline__ void low_bits(uint32_t w, uint32_t (&v)[4])
{
    const uint32_t w8 = w >> 8;
    v[0] = and_xor(w, 0x000f000fu, 0x00080008u);
    v[1] = and_xor(w, 0x00f000f0u, 0x00800080u);
    v[2] = and_xor(w8, 0x000f000fu, 0x00080008u);
    v[3] = and_xor(w8, 0x00f000f0u, 0x00800080u);
}

// Sums of a group's queries, times (scale, offset) pairs as they lie in memory: T operands, binary32 sums. A sum is cut
// into kParts values of T that hold 24 or 22 bits of it.
template <class T>
struct PairSum;
template <>
struct PairSum<__nv_bfloat16> {
    static constexpr int kParts = 3;
    static constexpr float kScale = 1.0f;  // of the sums
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return Value<__nv_bfloat16>::round2(lo, hi); }
    template <bool kFirst>
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
    {
        if constexpr (kFirst)
            c[0] = c[1] = c[2] = c[3] = 0.0f;
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
            "{%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};
template <>
struct PairSum<__half> {
    static constexpr int kParts = 2;
    static constexpr float kScale = 0x1p14f;  // 8 times a sum of 128 values of 2^15 is 2^25 kUnit kScale = 2^15
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_f16(lo, hi); }
    template <bool kFirst>
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
    {
        mma_f16<kFirst>(c, a[0], a[1], a[2], a[3], b0, b1);
    }
};

// log2 bound of a 16-bit magnitude; not finite counts as nothing.
template <class T>
__device__ __forceinline__ int exponent_of(uint32_t bits)
{
    return std::is_same<T, __half>::value ? (int)(bits >> 10) - 15 : (int)(bits >> 7) - 127;
}
template <class T>
__device__ __forceinline__ bool finite_bits(uint32_t bits)
{
    return bits < (std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u);
}

// The level of (scale, offset) bits without signs.
template <class T>
__device__ __forceinline__ int level_of_bits(uint32_t most)
{
    return max(exponent_of<T>(most & 0xffffu) + 1, exponent_of<T>(most >> 16) - 23);
}
__device__ __forceinline__ float power_or_0(int e) { return e < -126 ? 0.0f : power_of_2(e); }  // e <= 127

// The level of a token's (scale, offset) pairs.
template <class T, int N>
__device__ __forceinline__ int level_of(const uint32_t (&pairs)[N])
{
    uint32_t most = 0;
#pragma unroll
    for (int g = 0; g < N; g++) most = __vmaxu2(most, pairs[g] & 0x7fff7fffu);
    if (!finite_bits<T>(most & 0xffffu) || !finite_bits<T>(most >> 16)) {
        most = 0;
#pragma unroll
        for (int g = 0; g < N; g++) {
            const uint32_t scale = pairs[g] & 0x7fffu, offset = (pairs[g] >> 16) & 0x7fffu;
            most = __vmaxu2(most, (finite_bits<T>(scale) ? scale : 0u) | (finite_bits<T>(offset) ? offset << 16 : 0u));
        }
    }
    return level_of_bits<T>(most);
}

// The largest (scale, offset) bits without signs whose scale is below 2^level and offset below 2^(level + 24).
template <class T>
__device__ __forceinline__ uint32_t limit_of(int level)
{
    constexpr int kBits = std::is_same<T, __half>::value ? 10 : 7, kBias = std::is_same<T, __half>::value ? 15 : 127;
    constexpr int kLargest = std::is_same<T, __half>::value ? 0x7bff : 0x7f7f;
    const auto below = [](int e) { return e + kBias <= 0 ? 0 : min(((e + kBias) << kBits) - 1, kLargest); };
    return (uint32_t)below(level) | (uint32_t)below(level + 24) << 16;
}

// ---------------------------------------------------------------- the warps' walk over tiles
struct Walk {
    Spot at;
    int64_t n;  // places of the CTA's share
    int stop;   // the item's tiles in this share end here; none left if at.tile is not below

    __device__ __forceinline__ bool more() const { return at.tile < stop; }
    __device__ __forceinline__ void enter()
    {
        const int64_t left = n - at.base;
        stop = left >= at.tiles ? at.tiles : left > 0 ? (int)left : 0;
    }
    __device__ __forceinline__ void step(const Kv4Cache &c, const Kv4Attend &a, const AttendPlan &plan, int count)
    {
        at.tile += count;
        while (at.tile >= stop && stop == at.tiles) {
            at.tile -= at.tiles;
            at.base += at.tiles + kSetup;
            if (at.base < n && ++at.item == plan.items) {
                at.item = 0;
                at.b++;
                sequence_range(c, a, at.b, at.begin, at.end);
                at.tiles = tiles_of(at.begin, at.end);
            }
            enter();
        }
    }
};

// A warp's copies: the tile after next is looked up in the table while the tile before it is
// still on its way, so that no copy waits for its page number.
template <class T, class F>
struct Feed {
    Walk walk;
    int entry, place;             // the tile's page and first place in it, or each lane's token's
    const int32_t *row;           // of the table
    int64_t at_head, at_head_s;

    __device__ __forceinline__ void new_item(const Kv4Cache &c, const Kv4Attend &a, const AttendPlan &plan)
    {
        const int head = (int)divide_by(walk.at.item, plan.by_chunks);
        at_head = head * c.head_stride;
        at_head_s = head * c.head_stride_s;
        row = a.table + walk.at.b * a.ld_table;
    }
    __device__ __forceinline__ int first_position() const { return first_of(walk.at.begin) + walk.at.tile * kTokens; }

    __device__ __forceinline__ void look_up(const Kv4Cache &c, const AttendPlan &plan, int lane)
    {
        entry = -1;
        if (!walk.more()) return;
        const int at = first_position();
        if (plan.page_tiles) {
            const int tile = at / kTokens, column = (int)divide_by(tile, plan.by_page);
            place = (tile - column * plan.page_tiles) * kTokens;
            if (at < walk.at.end && dbg_ok(row + column, 4, false)) entry = __ldg(row + column);
        } else {
            const int j = at + lane, column = (int)divide_by(j, plan.by_page);
            place = j - column * c.page;
            if (j >= walk.at.begin && j < walk.at.end && dbg_ok(row + column, 4, false)) entry = __ldg(row + column);
        }
    }

    __device__ __forceinline__ void issue(const Kv4Cache &c, const Kv4Attend &a, const AttendPlan &plan, int lane, uint32_t stage)
    {
        if (walk.more()) {
            bool ok = entry >= 0 && entry < c.pages;
            const int from = first_position();
            bool one_page = true;  // whole tiles of one page: tokens at equal steps
            int page = entry, first = place;
            uint32_t there = kFull;
            if (!(plan.page_tiles && ok && from >= walk.at.begin && from + kTokens <= walk.at.end)) {
                if (plan.page_tiles) {
                    ok = ok && from + lane >= walk.at.begin && from + lane < walk.at.end;
                    place += lane;
                }
                there = __ballot_sync(kFull, ok);
                first = __shfl_sync(kFull, place, 0), page = __shfl_sync(kFull, entry, 0);
                one_page = there == kFull && first + kTokens <= c.page;
            }
            if (lane == 0) asm volatile("st.shared.u32 [%0], %1;" ::"r"(stage + F::kValid), "r"(there) : "memory");
            constexpr int kSize = F::kGroups % 4 == 0 ? 16 : F::kGroups % 2 == 0 ? 8 : 4;
            const uint32_t to_s = stage + 2 * F::kCodeBytes + 4 * F::kGroups * lane;
            if (one_page) {
                const int64_t at = page * c.page_stride + at_head + first * (int64_t)c.token_stride;
                const int64_t at_s = page * c.page_stride_s + at_head_s + (first + lane) * (int64_t)c.token_stride_s;
                const uint8_t *const k = c.k + at, *const v = c.v + at;
                if (c.token_stride == F::kDim / 2) {  // one run of bytes
#pragma unroll
                    for (int i = 0; i < F::kChunks; i++) {
                        const int piece = 32 * i + lane;
                        const uint32_t to = stage + 16 * chunk_at<F::kDim>(piece / F::kChunks, piece % F::kChunks);
                        lane_copy16(to, k + 16 * lane + 512 * i);
                        lane_copy16(to + F::kCodeBytes, v + 16 * lane + 512 * i);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < F::kChunks; i++) {
                        const int piece = 32 * i + lane, t = piece / F::kChunks, ch = piece % F::kChunks;
                        const int64_t from = t * (int64_t)c.token_stride + 16 * ch;
                        const uint32_t to = stage + 16 * chunk_at<F::kDim>(t, ch);
                        lane_copy16(to, k + from);
                        lane_copy16(to + F::kCodeBytes, v + from);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4 * F::kGroups; i += kSize) {
                    lane_copy_part<kSize>(to_s + i, c.k_scales + at_s + i, kSize);
                    lane_copy_part<kSize>(to_s + F::kPairBytes + i, c.v_scales + at_s + i, kSize);
                }
            } else {
                const int64_t page = ok ? entry : 0;  // each lane its own token
                const int64_t at = ok ? page * c.page_stride + at_head + place * (int64_t)c.token_stride : 0;
                const int64_t at_s = ok ? page * c.page_stride_s + at_head_s + place * (int64_t)c.token_stride_s : 0;
#pragma unroll
                for (int i = 0; i < F::kChunks; i++) {
                    const int piece = 32 * i + lane, t = piece / F::kChunks, ch = piece % F::kChunks;
                    const int64_t from = __shfl_sync(kFull, at, t) + 16 * ch;
                    const int bytes = (there >> t) & 1 ? 16 : 0;
                    const uint32_t to = stage + 16 * chunk_at<F::kDim>(t, ch);
                    lane_copy_part<16>(to, c.k + from, bytes);
                    lane_copy_part<16>(to + F::kCodeBytes, c.v + from, bytes);
                }
#pragma unroll
                for (int i = 0; i < 4 * F::kGroups; i += kSize) {
                    lane_copy_part<kSize>(to_s + i, c.k_scales + at_s + i, ok ? kSize : 0);
                    lane_copy_part<kSize>(to_s + F::kPairBytes + i, c.v_scales + at_s + i, ok ? kSize : 0);
                }
            }
            const int item = walk.at.item;
            const int b = walk.at.b;
            walk.step(c, a, plan, kAttendWarps);
            if (item != walk.at.item || b != walk.at.b) new_item(c, a, plan);
            look_up(c, plan, lane);
        }
        lane_copy_commit();
    }
};

// ---------------------------------------------------------------- one piece of work of a warp
// Lane 4 r + q. Scores of 16 tokens: tokens r and r + 8, query rows 2 q and 2 q + 1 of each half. Sums of the output:
// columns 4 r .. 4 r + 3 of every 32, the same rows. All that belongs to a row lies in its lanes, eight times over.
template <class T, class F>
struct Rows {
    // mma that multiply the groups' sums of queries: eight pairs of a token each
    static constexpr int kSums = (PairSum<T>::kParts * F::kGroups + 7) / 8;
    uint32_t qf[F::kGroups][F::kWords][2][2][F::kHalves];   // queries as mma fragments
    uint32_t qsum[kSums][2][F::kHalves];                    // fragments of a group's sum of scaled queries, times kUnit
    float2 f[F::kHalves];                                   // from a score in units to its log2
    float2 ref[F::kHalves];                                 // A
    int level;                                              // log2 of the largest scale so far, and the largest (scale, offset)
    uint32_t limit;                                         // bits that do not pass it: offsets count 2^-24
    float bound;                                            // log2 of p that may not be passed; all pass it where scales come down
    bool far;                                               // the warp's rows, see kFar
    float2 total[F::kHalves], off[F::kHalves][F::kGroups];  // sums of p, and of p z
    float sum[F::kDim / 16][F::kHalves][4];                 // of p s u, in units
    float eights[F::kGroups][F::kHalves][4];                // of 8 p s, in units, c0 c1 as c2 c3: groups apart, for their NaNs

    // The lane's queries of an item.
    using Queries = uint4[F::kHalves][F::kChunks];
    static __device__ __forceinline__ void fetch(const Kv4Attend &a, const AttendPlan &plan, int b, int head, int row0, int lane,
                                                 Queries &raw)
    {
        const int r = lane >> 2, q = lane & 3;
#pragma unroll
        for (int h = 0; h < F::kHalves; h++) {
            const int row = row0 + r + 8 * h;
            const int i = (int)divide_by(row < plan.rows ? row : 0, plan.by_share), in = (row < plan.rows ? row : 0) - i * plan.share;
            const T *from = static_cast<const T *>(a.q) + b * a.q_batch + i * a.q_query +
                            (int64_t)(head * plan.share + in) * a.q_head + 8 * q;
#pragma unroll
            for (int w = 0; w < F::kChunks; w++) raw[h][w] = row < plan.rows ? ld_keep_v4(from + 32 * w) : make_uint4(0, 0, 0, 0);
        }
    }

    __device__ __forceinline__ void start(const Kv4Attend &a, int lane, const Queries &raw)
    {
        far = false;
        set_level(level_of_bits<T>(0));
        const int q = lane & 3;
#pragma unroll
        for (int h = 0; h < F::kHalves; h++) {
            uint32_t top = 0;
#pragma unroll
            for (int w = 0; w < F::kChunks; w++) {
                const uint4 &x = raw[h][w];
                top = __vmaxu2(top, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                             __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
            }
            top = max(top & 0xffffu, top >> 16);
            top = max(top, __shfl_xor_sync(kFull, top, 1));
            top = max(top, __shfl_xor_sync(kFull, top, 2));
            const int e = max(exponent_of<T>(top), -100);  // the largest value is below 2^(e + 1)
            const float by = copysignf(power_of_2(14 - e), a.scale), by16 = 0.0625f * by;
            float all[F::kGroups];
            const int half = (e + 10) / 2;
            const float to_log2 = fminf(__fmul_rn(__fmul_rn(__fmul_rn(fabsf(a.scale), 1.4426950408889634f), power_of_2(half)),
                                   power_of_2(e + 10 - half)), 3.0e38f);
            f[h] = make_float2(__shfl_sync(kFull, to_log2, 8 * q), __shfl_sync(kFull, to_log2, 8 * q + 4));
#pragma unroll
            for (int g = 0; g < F::kGroups; g++) {
                float total_q = 0.0f;
#pragma unroll
                for (int w = 0; w < F::kWords; w++) {
                    const uint4 &x = raw[h][g * F::kWords + w];
                    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
                    float v[8];
#pragma unroll
                    for (int k = 0; k < 8; k++) {
                        v[k] = Value<T>::widen((uint16_t)(k & 1 ? u[k / 2] >> 16 : u[k / 2] & 0xffffu));
                        total_q = __fmaf_rn(v[k], by * kUnit, total_q);
                    }
#pragma unroll
                    for (int m = 0; m < 2; m++) {
                        qf[g][w][m][0][h] = pack_f16(__fmul_rn(v[2 * m], by), __fmul_rn(v[2 * m + 4], by));
                        qf[g][w][m][1][h] = pack_f16(__fmul_rn(v[2 * m + 1], by16), __fmul_rn(v[2 * m + 5], by16));
                    }
                }
                total_q = __fadd_rn(total_q, __shfl_xor_sync(kFull, total_q, 1));
                all[g] = __fmul_rn(__fadd_rn(total_q, __shfl_xor_sync(kFull, total_q, 2)), PairSum<T>::kScale);
                off[h][g] = splat(0.0f);
            }
#pragma unroll
            for (int m = 0; m < kSums; m++)
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    // slot: part slot / kGroups of group slot % kGroups
                    const int slot = 8 * m + 4 * j + q, part = slot / F::kGroups;
                    float rest = 0.0f, value = 0.0f;
#pragma unroll
                    for (int g = 0; g < F::kGroups; g++)
                        if (g == slot % F::kGroups) rest = all[g];
#pragma unroll
                    for (int i = 0; i < PairSum<T>::kParts; i++) {
                        const float v = Value<T>::widen(Value<T>::round(rest));
                        if (i == part) value = v;
                        rest = __fsub_rn(rest, v);
                    }
                    qsum[m][j][h] = PairSum<T>::pack(-8.0f * value, value);
                }
            ref[h] = splat(kNothing);
            total[h] = splat(0.0f);
#pragma unroll
            for (int m = 0; m < F::kDim / 16; m++)
#pragma unroll
                for (int k = 0; k < 4; k++) sum[m][h][k] = 0.0f;
#pragma unroll
            for (int g = 0; g < F::kGroups; g++)
#pragma unroll
                for (int k = 0; k < 4; k++) eights[g][h][k] = 0.0f;
        }
    }

    // Binary places that scales come down by.
    __device__ __forceinline__ int places() const
    {
        if (far) return max(level, -100) - (int)kLift;
        return std::is_same<T, __half>::value ? 0 : max(level - kHighest, 0) + min(level - kLowest, 0);
    }
    __device__ __forceinline__ void set_level(int to)
    {
        level = to;
        limit = limit_of<T>(to);
        bound = far || places() != 0 ? -INFINITY : kLift + 1.0f - (float)to;
    }
    // A row's sums after its reference has gone up: times keep, those of p s times less too.
    __device__ __forceinline__ void move(int h, float2 keep, float less)
    {
        total[h] = mul2(total[h], keep);
#pragma unroll
        for (int g = 0; g < F::kGroups; g++) off[h][g] = mul2(off[h][g], keep);
        const float2 keep_ps = mul2(keep, splat(less));
#pragma unroll
        for (int m = 0; m < F::kDim / 16; m++)
#pragma unroll
            for (int i = 0; i < 4; i++) sum[m][h][i] = __fmul_rn(sum[m][h][i], i & 1 ? keep_ps.y : keep_ps.x);
#pragma unroll
        for (int g = 0; g < F::kGroups; g++)
#pragma unroll
            for (int i = 0; i < 4; i++) eights[g][h][i] = __fmul_rn(eights[g][h][i], i & 1 ? keep_ps.y : keep_ps.x);
    }
    // A tile's scales come down, each lane its token's, whose pairs are `mine` as they were copied.
    __device__ __forceinline__ void bring_down(uint32_t pairs, int lane, const uint32_t (&mine)[F::kGroups])
    {
        const float down = power_of_2(-places());
#pragma unroll
        for (int g = 0; g < F::kGroups; g++)
            sts_u16(pairs + 4 * (F::kGroups * lane + g), Value<T>::round(__fmul_rn(pair_values<T>(mine[g]).x, down)));
        __syncwarp();
    }

    // x[n][t]: in units, of token 16 n + 8 t + r
    __device__ __forceinline__ void scores(uint32_t stage, int lane, float2 (&x)[2][2][F::kHalves])
    {
        const int r = lane >> 2, q = lane & 3;
        const uint32_t pairs = stage + 2 * F::kCodeBytes + 4 * F::kGroups * r;
#pragma unroll
        for (int n = 0; n < 2; n++) {
            // word q of every piece of tokens r and r + 8: w[2 piece], w[2 piece + 1]
            uint32_t w[2 * F::kChunks];
            const int row = 16 * n + (lane & 15);
#pragma unroll
            for (int i = 0; i < F::kChunks; i += 2)
                load_matrices(stage + 16 * chunk_at<F::kDim>(row, i + (lane >> 4)), w + 2 * i);
            uint32_t pw[2][F::kGroups];
#pragma unroll
            for (int t = 0; t < 2; t++) lds_words<F::kGroups>(pairs + 4 * F::kGroups * (16 * n + 8 * t), pw[t]);
            float c[F::kHalves][4];
            {
                constexpr bool kOne = 4 % F::kGroups == 0, kTwo = F::kGroups == 8;  // words that all slots share
                const uint32_t at = pairs + 4 * F::kGroups * 16 * n;
                uint32_t a[4];
#pragma unroll
                for (int m = 0; m < kSums; m++) {
#pragma unroll
                    for (int i = 0; i < 4; i++) {  // tokens r, r + 8, then their later slots
                        const int slot = 8 * m + 4 * (i >> 1) + q;
                        if (m == 0 || !(kOne || kTwo))
                            a[i] = i >= 2 && kOne ? a[i - 2] : lds_u32(at + 4 * (F::kGroups * 8 * (i & 1) + slot % F::kGroups));
                    }
#pragma unroll
                    for (int h = 0; h < F::kHalves; h++) {
                        if (m == 0)
                            PairSum<T>::template mma<true>(c[h], a, qsum[m][0][h], qsum[m][1][h]);
                        else
                            PairSum<T>::template mma<false>(c[h], a, qsum[m][0][h], qsum[m][1][h]);
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < F::kHalves; h++)
#pragma unroll
                for (int t = 0; t < 2; t++) {
                    x[n][t][h] = make_float2(c[h][2 * t], c[h][2 * t + 1]);
                    if (PairSum<T>::kScale != 1.0f) x[n][t][h] = mul2(x[n][t][h], splat(1.0f / PairSum<T>::kScale));
                }
#pragma unroll
            for (int g = 0; g < F::kGroups; g++) {
                float d[F::kHalves][4];
#pragma unroll
                for (int i = 0; i < F::kWords; i++) {
                    uint32_t u[4], v[4];
                    low_bits(w[2 * (g * F::kWords + i)], u);
                    low_bits(w[2 * (g * F::kWords + i) + 1], v);
#pragma unroll
                    for (int m = 0; m < 2; m++)
#pragma unroll
                        for (int h = 0; h < F::kHalves; h++) {
                            const uint32_t b0 = qf[g][i][m][0][h], b1 = qf[g][i][m][1][h];
                            if (i == 0 && m == 0)
                                mma_f16<true>(d[h], u[0], v[0], u[1], v[1], b0, b1);
                            else
                                mma_f16<false>(d[h], u[2 * m], v[2 * m], u[2 * m + 1], v[2 * m + 1], b0, b1);
                        }
                }
#pragma unroll
                for (int t = 0; t < 2; t++) {
                    const float2 s = splat(pair_values<T>(pw[t][g]).x);
#pragma unroll
                    for (int h = 0; h < F::kHalves; h++) x[n][t][h] = fma2(s, make_float2(d[h][2 * t], d[h][2 * t + 1]), x[n][t][h]);
                }
            }
        }
    }

    // A tile of a far warp, or of one that may become so: references, sums and exponents. Products are rounded as references are, so
    // that the largest score gives 0.
    template <bool kMasked>
    __device__ __forceinline__ void go_far(uint32_t pairs, int lane, const uint32_t (&mine)[F::kGroups], int k,
                                           const float2 (&x)[2][2][F::kHalves], const uint32_t (&seen)[F::kHalves][2],
                                           float2 (&y)[2][2][F::kHalves])
    {
        const int r = lane >> 2;
        const auto sees = [&](int h, int odd, int n, int t) { return !kMasked || ((seen[h][odd] >> (16 * n + 8 * t + r)) & 1); };
        const auto is_far = [](float ref) { return fabsf(ref) >= kFar && ref != kNothing; };
        bool any = far;
#pragma unroll
        for (int h = 0; h < F::kHalves; h++) any = any || is_far(ref[h].x) || is_far(ref[h].y);
        any = __any_sync(kFull, any);
        const bool was = far;
        const float less_by = (float)(level - places()) + kSlack<T> - kLift;  // what a reference that is not far holds beside a score
        if (any) {
            const int places_was = places();
            far = true;
            set_level(k);
            bring_down(pairs, lane, mine);
            const float less = power_or_0(places_was - places());
#pragma unroll
            for (int h = 0; h < F::kHalves; h++) {
                float2 best = splat(-INFINITY);
#pragma unroll
                for (int n = 0; n < 2; n++)
#pragma unroll
                    for (int t = 0; t < 2; t++) {
                        const float2 v = mul2_unfused(x[n][t][h], f[h]);
                        if (sees(h, 0, n, t)) best.x = fmaxf(best.x, v.x);
                        if (sees(h, 1, n, t)) best.y = fmaxf(best.y, v.y);
                    }
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    best.x = fmaxf(best.x, __shfl_xor_sync(kFull, best.x, d));
                    best.y = fmaxf(best.y, __shfl_xor_sync(kFull, best.y, d));
                }
                // a row whose reference has become so large has nothing yet, or scores far below this tile's
                const auto next_of = [&](float ref, float best) {
                    if (was || ref == kNothing) return fmaxf(ref, best);
                    return is_far(ref) ? best : fmaxf(best, ref - less_by);
                };
                const float2 next = make_float2(next_of(ref[h].x, best.x), next_of(ref[h].y, best.y));
                const float2 keep = make_float2(exp2_fast(fminf(__fsub_rn(ref[h].x, next.x), 100.0f)),
                                                exp2_fast(fminf(__fsub_rn(ref[h].y, next.y), 100.0f)));
                ref[h] = next;
                move(h, keep, less);
            }
        }
#pragma unroll
        for (int n = 0; n < 2; n++)
#pragma unroll
            for (int t = 0; t < 2; t++)
#pragma unroll
                for (int h = 0; h < F::kHalves; h++) {
                    float2 &v = y[n][t][h];
                    const float2 a = make_float2(-ref[h].x, -ref[h].y);
                    v = any ? add2(mul2_unfused(x[n][t][h], f[h]), a) : fma2(x[n][t][h], f[h], a);
                    if (!sees(h, 0, n, t)) v.x = -INFINITY;
                    if (!sees(h, 1, n, t)) v.y = -INFINITY;
                }
    }

    // A tile's values join the sums. seen: a bit a token for the rows 2 q and 2 q + 1 of each half; kMasked is false where
    // all are set.
    template <bool kMasked>
    __device__ __forceinline__ void take(uint32_t stage, int lane, float2 (&x)[2][2][F::kHalves], const uint32_t (&seen)[F::kHalves][2])
    {
        const int r = lane >> 2;
        const uint32_t pairs = stage + 2 * F::kCodeBytes + F::kPairBytes;
        // Do the lane's token's scales, and its offsets times 2^-24 (so that sums of p z stay in range), stay below the level?
        uint32_t mine[F::kGroups], above = limit;
        lds_words<F::kGroups>(pairs + 4 * F::kGroups * lane, mine);
#pragma unroll
        for (int g = 0; g < F::kGroups; g++) above = __vmaxu2(above, mine[g] & 0x7fff7fffu);
        const auto sees = [&](int h, int odd, int n, int t) { return !kMasked || ((seen[h][odd] >> (16 * n + 8 * t + r)) & 1); };
        float2 y[2][2][F::kHalves];
        float most = -INFINITY;
        const auto exponents = [&] {
#pragma unroll
            for (int n = 0; n < 2; n++)
#pragma unroll
                for (int t = 0; t < 2; t++)
#pragma unroll
                    for (int h = 0; h < F::kHalves; h++) {
                        float2 &v = y[n][t][h];
                        v = fma2(x[n][t][h], f[h], make_float2(-ref[h].x, -ref[h].y));
                        if (!sees(h, 0, n, t)) v.x = -INFINITY;
                        if (!sees(h, 1, n, t)) v.y = -INFINITY;
                        most = max3f(most, v.x, v.y);
                    }
        };
        exponents();
        // p s, s come down, stays within 2^14 as long as no scale passes the level and no p 2^(14 - level): every lane looks at its own
        // tokens, and the rows' largest p s are looked for where one does
        if (__any_sync(kFull, most > bound || above != limit)) {
            const int token = level_of<T>(mine);  // the lane's token's level
            const int k = __reduce_max_sync(kFull, max(token, level));
            float reach = INFINITY;
            if (!far) {
                reach = 0.0f;
                const int places_was = places();
                set_level(k);
                // in the tile itself, all such tiles come here: a product for each scale where it is used cost 64 sequences of up
                // to 8192 tokens 1 %
                if (places() != 0) bring_down(pairs, lane, mine);
                const float less = power_or_0(places_was - places());
                // log2 of what a token's p is multiplied by, at most
                const float its = (float)max(token - places(), kLowest);
                float add[2][2];
#pragma unroll
                for (int n = 0; n < 2; n++)
#pragma unroll
                    for (int t = 0; t < 2; t++) add[n][t] = __shfl_sync(kFull, its, 16 * n + 8 * t + r);
#pragma unroll
                for (int h = 0; h < F::kHalves; h++) {
                    float2 top = splat(-INFINITY);
#pragma unroll
                    for (int n = 0; n < 2; n++)
#pragma unroll
                        for (int t = 0; t < 2; t++) {
                            const float2 v = fma2(x[n][t][h], f[h], splat(add[n][t]));
                            if (sees(h, 0, n, t)) top.x = fmaxf(top.x, v.x);
                            if (sees(h, 1, n, t)) top.y = fmaxf(top.y, v.y);
                        }
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) {
                        top.x = fmaxf(top.x, __shfl_xor_sync(kFull, top.x, d));
                        top.y = fmaxf(top.y, __shfl_xor_sync(kFull, top.y, d));
                    }
                    top = add2(top, splat(kSlack<T> - kLift));
                    const float2 next = make_float2(fmaxf(ref[h].x, top.x), fmaxf(ref[h].y, top.y));
                    const float2 keep = make_float2(exp2_fast(__fsub_rn(ref[h].x, next.x)), exp2_fast(__fsub_rn(ref[h].y, next.y)));
                    ref[h] = next;
                    reach = fmaxf(reach, fmaxf(fabsf(next.x), fabsf(next.y)));
                    move(h, keep, less);
                }
            }
            if (__any_sync(kFull, reach >= kFar))
                go_far<kMasked>(pairs, lane, mine, k, x, seen, y);
            else
                exponents();
        }
#pragma unroll
        for (int n = 0; n < 2; n++)
#pragma unroll
            for (int t = 0; t < 2; t++)
#pragma unroll
                for (int h = 0; h < F::kHalves; h++) {
                    x[n][t][h] = make_float2(exp2_fast(y[n][t][h].x), exp2_fast(y[n][t][h].y));  // p from here on
                    total[h] = add2(total[h], x[n][t][h]);
                }
#pragma unroll
        for (int n = 0; n < 2; n++) {
            uint32_t pw[2][F::kGroups], codes[4];
#pragma unroll
            for (int t = 0; t < 2; t++) lds_words<F::kGroups>(pairs + 4 * F::kGroups * (16 * n + 8 * t + r), pw[t]);
#pragma unroll
            for (int g = 0; g < F::kGroups; g++) {
                uint32_t b[F::kHalves][2];
#pragma unroll
                for (int t = 0; t < 2; t++) {
                    const float2 pair = pair_values<T>(pw[t][g]);
#pragma unroll
                    for (int h = 0; h < F::kHalves; h++) {
                        const float2 p = x[n][t][h];
                        float2 s = splat(pair.x), z = splat(pair.y);
                        if (kMasked) {  // a row that does not see a token takes nothing of it, a NaN neither
                            if (!sees(h, 0, n, t)) s.x = z.x = 0.0f;
                            if (!sees(h, 1, n, t)) s.y = z.y = 0.0f;
                        }
                        const float2 ps = mul2(p, s);
                        b[h][t] = transposed(pack_f16(ps.x, ps.y));
                        off[h][g] = fma2(p, z, off[h][g]);
                    }
                }
#pragma unroll
                for (int h = 0; h < F::kHalves; h++) {
                    constexpr uint32_t kEight = 0x00080008u;
                    mma_f16<false>(eights[g][h], kEight, kEight, kEight, kEight, b[h][0], b[h][1]);
                }
                values(stage + F::kCodeBytes, lane, n, g, b, codes);
            }
        }
    }

    // The codes of 16 tokens in group g against b. A transposed matrix of eight tokens and one piece gives a lane four
    // columns' codes of two tokens, side by side as a fragment of the values takes them.
    __device__ __forceinline__ void values(uint32_t codes, int lane, int i, int g, const uint32_t (&b)[F::kHalves][2],
                                           uint32_t (&pieces)[4])
    {
#pragma unroll
        for (int k = 0; k < F::kWords; k++) {
            const int piece = g * F::kWords + k;
            if (piece % 2 == 0) load_transposed(codes + 16 * chunk_at<F::kDim>(16 * i + (lane & 15), piece + (lane >> 4)), pieces);
            uint32_t lo[4], hi[4];
            low_bits(pieces[2 * (piece % 2)], lo);
            low_bits(pieces[2 * (piece % 2) + 1], hi);
#pragma unroll
            for (int odd = 0; odd < 2; odd++)
#pragma unroll
                for (int h = 0; h < F::kHalves; h++)
                    mma_f16<false>(sum[2 * piece + odd][h], lo[odd], lo[2 + odd], hi[odd], hi[2 + odd], b[h][0], b[h][1]);
        }
    }

    // The lanes' parts brought together: total in every lane of a row, sum the true sums of p v.
    __device__ __forceinline__ void finish()
    {
        const float up = power_of_2(min(24 + places(), 126));  // 1 / kUnit and what scales came down by
        if (24 + places() > 126) {
#pragma unroll
            for (int h = 0; h < F::kHalves; h++) move(h, splat(1.0f), power_of_2(24 + places() - 126));
        }
        const auto all = [](float2 v) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1)
                v = add2(v, make_float2(__shfl_xor_sync(kFull, v.x, d), __shfl_xor_sync(kFull, v.y, d)));
            return v;
        };
#pragma unroll
        for (int h = 0; h < F::kHalves; h++) {
            total[h] = all(total[h]);
#pragma unroll
            for (int g = 0; g < F::kGroups; g++) {
                const float2 z = all(off[h][g]);
#pragma unroll
                for (int k = 0; k < F::kGroup / 16; k++) {
                    float(&v)[4] = sum[g * (F::kGroup / 16) + k][h];
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const float u = k & 1 ? __fmul_rn(v[i], 0.0625f) : v[i];
                        const float c = eights[g][h][i];
                        v[i] = __fmaf_rn(__fsub_rn(u, c), up, i & 1 ? z.y : z.x);
                    }
                }
            }
        }
    }
};

// ---------------------------------------------------------------- the kernel
// Where an item's row goes.
__device__ __forceinline__ int64_t out_row(const Kv4Attend &a, const AttendPlan &plan, int b, int head, int row, int64_t *lse)
{
    const int i = (int)divide_by(row, plan.by_share), h = head * plan.share + row - i * plan.share;
    *lse = ((int64_t)b * a.n_q + i) * a.q_heads + h;
    return b * a.out_batch + i * a.out_query + h * a.out_head;
}

__device__ __forceinline__ float lse_of(float ref, float total)
{
    return total == 0.0f ? -INFINITY : __fmul_rn(__fadd_rn(ref, log2f(total)), 0.6931471805599453f);
}

__device__ __forceinline__ void dbg_attend(const Kv4Cache &c, const Kv4Attend &a, const AttendPlan &plan, int64_t floats)
{
    dbg_begin();
    dbg_cache(c, false);
    dbg_allow(a.q, 2 * ((a.batch - 1) * a.q_batch + (a.n_q - 1) * a.q_query + (a.q_heads - 1) * a.q_head + c.head_dim), false);
    dbg_allow(a.out, 2 * ((a.batch - 1) * a.out_batch + (a.n_q - 1) * a.out_query + (a.q_heads - 1) * a.out_head + c.head_dim),
              true);
    dbg_allow(a.table, a.width ? 4 * ((a.batch - 1) * a.ld_table + a.width) : 0, false);
    dbg_allow(a.lengths, 4ll * a.batch, false);
    dbg_allow(a.lse, a.lse ? 4ll * a.batch * a.n_q * a.q_heads : 0, true);
    dbg_allow(a.workspace, 4 * (4 * kMaxAttendCtas + 2 * plan.ctas * floats), true);
    dbg_ready();
}

// A warp's sums beside those of another warp in shared memory: [kRows] references, [kRows] totals, [kRows][kDim].
template <class T, class F>
struct Join {
    static constexpr int kRuns = F::kDim / 32;  // of four columns of a lane
    static __device__ __forceinline__ int column(int r, int k) { return 32 * k + 4 * r; }
    // run k's values of row 2 q + odd of half h, in order: rows r and r + 8 of the even columns' tile and the odd ones'
    static __device__ __forceinline__ float4 run_of(const Rows<T, F> &x, int k, int h, int odd)
    {
        return make_float4(x.sum[2 * k][h][odd], x.sum[2 * k + 1][h][odd], x.sum[2 * k][h][2 + odd], x.sum[2 * k + 1][h][2 + odd]);
    }
    static __device__ __forceinline__ void put(const Rows<T, F> &x, float *to, int lane)
    {
        const int r = lane >> 2, q = lane & 3;
#pragma unroll
        for (int h = 0; h < F::kHalves; h++) {
            if (r == 0) {
                *reinterpret_cast<float2 *>(to + 8 * h + 2 * q) = x.ref[h];
                *reinterpret_cast<float2 *>(to + F::kRows + 8 * h + 2 * q) = x.total[h];
            }
#pragma unroll
            for (int odd = 0; odd < 2; odd++)
#pragma unroll
                for (int k = 0; k < kRuns; k++)
                    *reinterpret_cast<float4 *>(to + 2 * F::kRows + (8 * h + 2 * q + odd) * F::kDim + column(r, k)) =
                        run_of(x, k, h, odd);
        }
    }
    static __device__ __forceinline__ void add(Rows<T, F> &x, const float *from, int lane)
    {
        const int r = lane >> 2, q = lane & 3;
#pragma unroll
        for (int h = 0; h < F::kHalves; h++) {
            const float2 other = *reinterpret_cast<const float2 *>(from + 8 * h + 2 * q), ref = x.ref[h];
            const float2 next = make_float2(fmaxf(ref.x, other.x), fmaxf(ref.y, other.y));
            const float2 mine = make_float2(exp2_fast(__fsub_rn(ref.x, next.x)), exp2_fast(__fsub_rn(ref.y, next.y)));
            const float2 theirs = make_float2(exp2_fast(__fsub_rn(other.x, next.x)), exp2_fast(__fsub_rn(other.y, next.y)));
            x.ref[h] = next;
            x.total[h] = fma2(*reinterpret_cast<const float2 *>(from + F::kRows + 8 * h + 2 * q), theirs, mul2(x.total[h], mine));
#pragma unroll
            for (int odd = 0; odd < 2; odd++) {
                const float m = odd ? mine.y : mine.x, t = odd ? theirs.y : theirs.x;
#pragma unroll
                for (int k = 0; k < kRuns; k++) {
                    const float4 v = *reinterpret_cast<const float4 *>(from + 2 * F::kRows + (8 * h + 2 * q + odd) * F::kDim +
                                                                       column(r, k));
                    const float w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        float &s = x.sum[2 * k + (j & 1)][h][2 * (j >> 1) + odd];
                        s = __fmaf_rn(w[j], t, __fmul_rn(s, m));
                    }
                }
            }
        }
    }
};

template <class T, class F>
__global__ void __launch_bounds__(kAttendThreads, F::kCtas)
    attend_kernel(const __grid_constant__ Kv4Cache c, const __grid_constant__ Kv4Attend a, const __grid_constant__ AttendPlan plan)
{
    extern __shared__ __align__(16) unsigned char smem[];
    using J = Join<T, F>;
    constexpr int64_t kPartial = (int64_t)F::kRows * (F::kDim + 2);
    pdl_begin();
    dbg_attend(c, a, plan, kPartial);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Share share;
    Spot now;
    if (threadIdx.x == 0 && !plan.by_item) st_v4(a.workspace + 4 * blockIdx.x, make_uint4(0, 0, 0, 0));
    find_share(c, a, plan, share, now);  // its barriers order that before other threads' word
    if ((int)blockIdx.x >= share.ctas) return;
    const int64_t places = share.first(blockIdx.x + 1) - share.first(blockIdx.x);

    float *const joins = reinterpret_cast<float *>(smem);
    const uint32_t ring = smem_u32(smem) + F::kJoin + warp * F::kStages * F::kStage;
    Feed<T, F> feed;
    feed.walk = Walk{now, places, 0};
    feed.walk.enter();
    feed.walk.step(c, a, plan, warp);
    feed.new_item(c, a, plan);
    feed.look_up(c, plan, lane);
#pragma unroll
    for (int s = 0; s < F::kStages - 1; s++) feed.issue(c, a, plan, lane, ring + s * F::kStage);

    Rows<T, F> x;
    uint32_t stage = ring, fill = ring + (F::kStages - 1) * F::kStage;  // the tile's, and the one that is free
    for (int turn = 0; now.base + now.tile < places;) {
        const int64_t left = places - now.base;
        const int last = left < now.tiles ? (int)left : now.tiles;  // of the item in this share
        const int head = (int)divide_by(now.item, plan.by_chunks), row0 = (now.item - head * plan.chunks) * F::kRows;
        // One tile is one warp's item, without a join: the others are at the next one meanwhile.
        const bool alone = last - now.tile == 1;
        const int writer = alone ? turn & (kAttendWarps - 1) : 0;
        const bool mine = !alone || warp == writer;
        if (mine) {
            typename Rows<T, F>::Queries queries;
            x.fetch(a, plan, now.b, head, row0, lane, queries);
            x.start(a, lane, queries);
            // the positions that the lane's rows see, and that all rows of the item do
            int lo[F::kHalves][2], hi[F::kHalves][2];
#pragma unroll
            for (int i = 0; i < 2 * F::kHalves; i++) {
                const int row = min(row0 + 8 * (i >> 1) + 2 * (lane & 3) + (i & 1), plan.rows - 1);
                int &end = hi[i >> 1][i & 1];
                end = now.end - a.n_q + 1 + (int)divide_by(row, plan.by_share);
                lo[i >> 1][i & 1] = a.window > 0 && end > a.window ? end - a.window : 0;
            }
            const int all_hi = now.end - a.n_q + 1 + (int)divide_by(row0, plan.by_share);
            const int last_hi = now.end - a.n_q + 1 + (int)divide_by(min(row0 + F::kRows, plan.rows) - 1, plan.by_share);
            const int all_lo = a.window > 0 && last_hi > a.window ? last_hi - a.window : 0;
            for (int t = now.tile + ((warp - turn) & (kAttendWarps - 1)); t < last; t += kAttendWarps) {
                lane_copy_wait<F::kStages - 2>();
                __syncwarp();
                feed.issue(c, a, plan, lane, fill);
                const uint32_t there = lds_u32(stage + F::kValid);
                const int at = first_of(now.begin) + t * kTokens;
                float2 s[2][2][F::kHalves];
                x.scores(stage, lane, s);
                uint32_t seen[F::kHalves][2];
                if (there == kFull && at >= all_lo && at + kTokens <= all_hi) {
                    x.template take<false>(stage, lane, s, seen);
                } else {
#pragma unroll
                    for (int i = 0; i < 2 * F::kHalves; i++) {
                        const int from = max(lo[i >> 1][i & 1] - at, 0), to = min(hi[i >> 1][i & 1] - at, kTokens);
                        const uint32_t above = from < kTokens ? kFull << from : 0u, below = to <= 0 ? 0u : kFull >> (kTokens - to);
                        seen[i >> 1][i & 1] = there & above & below;
                    }
                    x.template take<true>(stage, lane, s, seen);
                }
                fill = stage;
                stage = stage == ring + (F::kStages - 1) * F::kStage ? ring : stage + F::kStage;
            }
        }
        const int b = now.b, item = now.item, rest = now.tiles - last;
        const bool from_start = now.tile == 0;
        turn += last - now.tile;
        now.base = rest ? places : now.base + now.tiles + kSetup;
        now.tile = 0;
        if (now.base < places) {
            if (++now.item == plan.items) {
                now.item = 0;
                now.b++;
                sequence_range(c, a, now.b, now.begin, now.end);
                now.tiles = tiles_of(now.begin, now.end);
            }
        }
        if (!mine) continue;
        x.finish();
        // warps 2 and 3 to 0 and 1, then 1 to 0; the last step's place is read by warp 0 before the next item's first
        // barrier, and the first step's before this item's second
        if (!alone) {
            if (warp >= 2) J::put(x, joins + (warp - 2) * kPartial, lane);
            __syncthreads();
            if (warp < 2) J::add(x, joins + warp * kPartial, lane);
            if (warp == 1) J::put(x, joins + 2 * kPartial, lane);
            __syncthreads();
            if (warp == 0) J::add(x, joins + 2 * kPartial, lane);
        }
        if (warp == writer) {
            const int r = lane >> 2, q = lane & 3;
            if (from_start && lane == 0 && (rest || plan.by_item)) {
                const int64_t after = rest + share.per - 1;
                const int more = after < 0x7fffffff ? (int)((uint32_t)after / (uint32_t)share.per) : (int)(after / share.per);
                st_v4(a.workspace + 4 * (plan.by_item ? (int64_t)b * plan.items + item : blockIdx.x),
                      make_uint4(b, item, 1 + more, blockIdx.x));
            }
            if (from_start && rest == 0) {
#pragma unroll
                for (int h = 0; h < F::kHalves; h++) {
#pragma unroll
                    for (int odd = 0; odd < 2; odd++) {
                        const int row = row0 + 8 * h + 2 * q + odd;
                        const float total = odd ? x.total[h].y : x.total[h].x, by = total == 0.0f ? 0.0f : __fdiv_rn(1.0f, total);
                        if (row < plan.rows) {
                            int64_t at;
                            T *to = static_cast<T *>(a.out) + out_row(a, plan, b, head, row, &at);
                            if (r == 0 && a.lse && dbg_ok(a.lse + at, 4, true))
                                a.lse[at] = lse_of(odd ? x.ref[h].y : x.ref[h].x, total);
#pragma unroll
                            for (int k = 0; k < J::kRuns; k++) {
                                const float4 v = J::run_of(x, k, h, odd);
                                st_v2(to + J::column(r, k), make_uint2(Value<T>::round2(__fmul_rn(v.x, by), __fmul_rn(v.y, by)),
                                                                       Value<T>::round2(__fmul_rn(v.z, by), __fmul_rn(v.w, by))));
                            }
                        }
                    }
                }
            } else {
                float *const to = partial_of(a.workspace, blockIdx.x, from_start, kPartial);
#pragma unroll
                for (int h = 0; h < F::kHalves; h++) {
                    if (r == 0) {
                        st_v2(to + 8 * h + 2 * q, make_uint2(__float_as_uint(x.ref[h].x), __float_as_uint(x.ref[h].y)));
                        st_v2(to + F::kRows + 8 * h + 2 * q, make_uint2(__float_as_uint(x.total[h].x), __float_as_uint(x.total[h].y)));
                    }
#pragma unroll
                    for (int odd = 0; odd < 2; odd++)
#pragma unroll
                        for (int k = 0; k < J::kRuns; k++) {
                            const float4 v = J::run_of(x, k, h, odd);
                            st_v4(to + 2 * F::kRows + (8 * h + 2 * q + odd) * F::kDim + J::column(r, k),
                                  make_uint4(__float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z), __float_as_uint(v.w)));
                        }
                }
            }
        }
    }
    lane_copy_wait<0>();
}

// ---------------------------------------------------------------- launch
template <class T, class F>
cudaError_t launch_form(const Kv4Cache &c, const Kv4Attend &a, AttendPlan &plan, cudaStream_t st)
{
    void (*kernel)(Kv4Cache, Kv4Attend, AttendPlan) = attend_kernel<T, F>;
    plan.chunks = (plan.rows + F::kRows - 1) / F::kRows;
    plan.items = c.heads * plan.chunks;
    plan.by_chunks = divisor((uint32_t)plan.chunks);
    // enough CTAs for any lengths: a share of one tile a warp at least
    const int64_t longest = ((int64_t)a.width * c.page + kTokens) / kTokens;
    const int64_t tiles = (int64_t)(a.batch < 4096 ? a.batch : 4096) * plan.items * longest;
    if (cudaError_t e = grid_for((const void *)kernel, tiles, &plan.ctas, F::kSmem, kAttendThreads)) return e;
    if (plan.ctas > kMaxAttendCtas) plan.ctas = kMaxAttendCtas;
    plan.by_item = a.batch <= kMaxAttendCtas / plan.items;
    plan.words = plan.by_item ? a.batch * plan.items : plan.ctas;
    return launch_kernel_block(kernel, plan.ctas, kAttendThreads, F::kSmem, st, c, a, plan);
}

// Rows of a form: 16 where their sums, fragments of queries and corrections leave at most the spills named above. 16 rows of 192
// columns would hold 96 sums and 48 fragments of queries, where 8 rows of 256, 64 and 32 of them, spill already.
__host__ __device__ inline int form_rows(int rows, int dim) { return rows > 8 && dim <= 128 ? 16 : 8; }

template <class T>
cudaError_t launch_attend(const Kv4Cache &c, const Kv4Attend &a, AttendPlan &plan, cudaStream_t st)
{
    const bool wide = form_rows(plan.rows, c.head_dim) == 16;
#define BQ_FORM(D, G) \
    if (c.head_dim == D && c.group == G) return launch_form<T, Form<D, G, 8>>(c, a, plan, st);
#define BQ_FORMS(D, G)                                                                       \
    if (c.head_dim == D && c.group == G)                                                     \
        return wide ? launch_form<T, Form<D, G, 16>>(c, a, plan, st) : launch_form<T, Form<D, G, 8>>(c, a, plan, st);
    BQ_FORMS(64, 32)
    BQ_FORMS(64, 64)
    BQ_FORMS(128, 32)
    BQ_FORMS(128, 64)
    BQ_FORMS(128, 128)
    BQ_FORM(192, 32)
    BQ_FORM(192, 64)
    BQ_FORM(256, 32)
    BQ_FORM(256, 64)
    BQ_FORM(256, 128)
#undef BQ_FORM
#undef BQ_FORMS
    return cudaErrorInvalidValue;
}

cudaError_t launch_attend_bf16(const Kv4Cache &c, const Kv4Attend &a, AttendPlan &plan, cudaStream_t st);
cudaError_t launch_attend_f16(const Kv4Cache &c, const Kv4Attend &a, AttendPlan &plan, cudaStream_t st);

}  // namespace bqk
