// The token side of a mixture-of-experts layer: slots sorted by expert, token rows
// gathered into that order, and expert rows combined back with their weights, with the
// gradients of both.
//
// A slot is one choice of the router: slot i = t * top_k + j is token t's j-th expert.
// The sort gives every kept slot a place, the places of one expert consecutive and in
// slot order; `inverse` maps slots to places and `order` places to slots. An id outside
// [0, n_experts) is an expert held elsewhere: its slot is dropped (inverse -1) and takes
// no part in anything below.
#include "bq_rows.cuh"

namespace bqk {
namespace {

// ---------------------------------------------------------------- sort
// A stable counting sort. Every warp owns a run of consecutive slots and a row of
// counters in shared memory, one per expert. It counts its slots with shared-memory
// additions, whose order does not matter. The counters are then turned into the first place
// of each (warp, expert), and a second walk over the same slots, 32 at a time, hands the
// places out in lane order: match_any gives each lane the lanes with the same id. Nothing
// depends on the order in which warps run. match_any is the slow part, an SM finishes one
// every 49 cycles: with it in the counting too, 524288 slots of 64 experts took 11.4 us, and
// with a ballot per bit of the id in its place 13.1 us.
//
// Lane w of a warp holds warp w's counter when the counters are summed or scanned over the
// warps; a row of counters has an odd stride, so that these 32 lie in different banks.
//
// Up to kSortOneCta slots one CTA does all of it in one launch. More slots are cut into
// `parts` runs, one CTA each: a first launch writes each run's counts to the workspace, the
// second adds up the runs before its own and all runs, and places. An SM stores at most one
// of the scattered places per cycle: 12728 slots took 22.4 us in one CTA, 7.8 us in two
// launches of 13.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int64_t kSortOneCta = 4096;
constexpr int kFewWarps = 8;  // counters of so few warps are scanned by a thread per expert
static_assert(kSortWarps == 32, "a lane per warp");
__host__ __device__ constexpr int count_stride(int n_experts) { return n_experts | 1; }

// The id of slot i, or -1 where the slot is dropped.
__device__ __forceinline__ int slot_expert(const int32_t *ids, int64_t i, int n_experts)
{
    if (!dbg_ok(ids + i, 4, false)) return -1;
    const int32_t e = ids[i];
    return e >= 0 && e < n_experts ? e : -1;
}

__device__ __forceinline__ int slot_expert(const int64_t *ids, int64_t i, int n_experts)
{
    if (!dbg_ok(ids + i, 8, false)) return -1;
    const int64_t e = ids[i];
    return e >= 0 && e < n_experts ? static_cast<int>(e) : -1;
}

__device__ __forceinline__ void st_i32(int32_t *p, int32_t v)
{
    if (dbg_ok(p, 4, true)) *p = v;
}

// Slots [lo, hi) of warp w of run `part`: runs and warps take multiples of 32 slots.
struct SlotRun {
    int64_t lo, hi;
};
__device__ __forceinline__ SlotRun warp_run(int64_t slots, int parts, int part, int warp)
{
    const int64_t batches = (slots + 31) / 32;
    const int64_t per_warp = (batches + (int64_t)parts * kSortWarps - 1) / ((int64_t)parts * kSortWarps) * 32;
    const int64_t lo = ((int64_t)part * kSortWarps + warp) * per_warp;
    const int64_t hi = lo + per_warp;
    return SlotRun{lo < slots ? lo : slots, hi < slots ? hi : slots};
}

// The experts of a warp's next kAhead batches of 32 slots, this lane's slot of each: loaded
// together, so that their latencies overlap.
constexpr int kAhead = 4;
template <class Id>
__device__ __forceinline__ void load_experts(const Id *ids, int64_t i0, int64_t hi, int n_experts, int lane,
                                             int (&e)[kAhead])
{
#pragma unroll
    for (int k = 0; k < kAhead; k++) {
        const int64_t i = i0 + 32 * k + lane;
        e[k] = i < hi ? slot_expert(ids, i, n_experts) : -1;
    }
}

// count[w][e] over this CTA's run, e0 its first batches; the caller synchronizes.
template <class Id>
__device__ __forceinline__ void count_run(const Id *ids, SlotRun run, int n_experts, const int (&e0)[kAhead], int *mine,
                                          int lane)
{
    int e[kAhead];
    for (int64_t i0 = run.lo; i0 < run.hi; i0 += 32 * kAhead) {
        if (i0 == run.lo) {
#pragma unroll
            for (int k = 0; k < kAhead; k++) e[k] = e0[k];
        } else {
            load_experts(ids, i0, run.hi, n_experts, lane, e);
        }
#pragma unroll
        for (int k = 0; k < kAhead; k++) {
            if (i0 + 32 * k >= run.hi) break;
            if (e[k] >= 0) atomicAdd(&mine[e[k]], 1);
        }
    }
}

template <class Id>
__global__ void __launch_bounds__(kSortThreads)
sort_count_kernel(const Id *__restrict__ ids, int64_t slots, int n_experts, int parts, int32_t *__restrict__ ws)
{
    extern __shared__ int count[];  // [kSortWarps][count_stride(n_experts)]
    pdl_begin();
    dbg_begin();
    dbg_allow(ids, slots * (int64_t)sizeof(Id), false);
    dbg_allow(ws, 4ll * parts * n_experts, true);
    dbg_ready();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int stride = count_stride(n_experts);
    const SlotRun run = warp_run(slots, parts, blockIdx.x, warp);
    int e0[kAhead];
    load_experts(ids, run.lo, run.hi, n_experts, lane, e0);
    for (int i = threadIdx.x; i < kSortWarps * stride; i += kSortThreads) count[i] = 0;
    __syncthreads();
    count_run(ids, run, n_experts, e0, count + warp * stride, lane);
    __syncthreads();
    for (int e = warp; e < n_experts; e += kSortWarps) {
        const int sum = __reduce_add_sync(kFull, count[lane * stride + e]);
        if (lane == 0) st_i32(ws + (int64_t)blockIdx.x * n_experts + e, sum);
    }
}

template <class Id>
__global__ void __launch_bounds__(kSortThreads)
sort_place_kernel(const Id *__restrict__ ids, int64_t slots, int n_experts, int parts, const int32_t *__restrict__ ws,
                  int32_t *__restrict__ offsets, int32_t *__restrict__ order, int32_t *__restrict__ inverse)
{
    extern __shared__ int count[];  // [kSortWarps][count_stride(n_experts)], then total and before [n_experts]
    __shared__ int warp_sum[32];
    pdl_begin();
    dbg_begin();
    dbg_allow(ids, slots * (int64_t)sizeof(Id), false);
    dbg_allow(ws, parts > 1 ? 4ll * parts * n_experts : 0, false);
    dbg_allow(offsets, 4ll * (n_experts + 1), true);
    dbg_allow(order, 4 * slots, true);
    dbg_allow(inverse, 4 * slots, true);
    dbg_ready();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = blockIdx.x;
    const int stride = count_stride(n_experts);
    int *total = count + kSortWarps * stride, *before = total + n_experts;
    const SlotRun run = warp_run(slots, parts, part, warp);
    int e0[kAhead];
    load_experts(ids, run.lo, run.hi, n_experts, lane, e0);
    // warps past the last slot have nothing to count, and their counters are not used
    const int64_t batches = (slots + 31) / 32;
    const int busy = parts == 1 && batches < kSortWarps ? (int)batches : kSortWarps;
    for (int i = threadIdx.x; i < busy * stride; i += kSortThreads) count[i] = 0;
    for (int i = threadIdx.x; i < 2 * n_experts; i += kSortThreads) total[i] = 0;
    __syncthreads();
    int *mine = count + warp * stride;
    count_run(ids, run, n_experts, e0, mine, lane);
    // Sums over the runs: thread group g of the expert takes every groups-th run. Integer
    // additions, so their order does not matter.
    if (parts > 1) {
        const int groups = kSortThreads / n_experts;  // n_experts <= kSortThreads
        const int e = threadIdx.x % n_experts, g = threadIdx.x / n_experts;
        if (g < groups) {
            int all = 0, below = 0;
            for (int p = g; p < parts; p += groups) {
                const int32_t *src = ws + (int64_t)p * n_experts + e;
                const int v = dbg_ok(src, 4, false) ? *src : 0;
                all += v;
                below += p < part ? v : 0;
            }
            atomicAdd(&total[e], all);
            atomicAdd(&before[e], below);
        }
    }
    __syncthreads();
    // An expert's counts over the warps become first places within the run.
    for (int e = threadIdx.x; busy <= kFewWarps && e < n_experts; e += kSortThreads) {
        int upto = 0;
        for (int w = 0; w < busy; w++) {
            const int v = count[w * stride + e];
            count[w * stride + e] = upto;
            upto += v;
        }
        total[e] = upto;
    }
    for (int e = warp; busy > kFewWarps && e < n_experts; e += kSortWarps) {
        const int v = lane < busy ? count[lane * stride + e] : 0;
        int upto = v;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int up = __shfl_up_sync(kFull, upto, d);
            if (lane >= d) upto += up;
        }
        if (lane < busy) count[lane * stride + e] = upto - v;
        if (parts == 1 && lane == 31) total[e] = upto;
    }
    __syncthreads();
    // Thread e: a scan over the experts gives the expert's first place among all.
    const int e = threadIdx.x;
    const int all = e < n_experts ? total[e] : 0;
    int scan = all;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(kFull, scan, d);
        if (lane >= d) scan += up;
    }
    if (lane == 31) warp_sum[warp] = scan;
    __syncthreads();
    if (warp == 0) {
        int s = warp_sum[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int up = __shfl_up_sync(kFull, s, d);
            if (lane >= d) s += up;
        }
        warp_sum[lane] = s;
    }
    __syncthreads();
    const int first = scan - all + (warp > 0 ? warp_sum[warp - 1] : 0);
    const int kept = warp_sum[31];
    if (e < n_experts) {
        before[e] += first;
        if (part == 0) {
            st_i32(offsets + e, first);
            if (e == n_experts - 1) st_i32(offsets + n_experts, kept);
        }
    }
    __syncthreads();
    for (int64_t i0 = run.lo; i0 < run.hi; i0 += 32 * kAhead) {
        if (i0 != run.lo) load_experts(ids, i0, run.hi, n_experts, lane, e0);
#pragma unroll
        for (int k = 0; k < kAhead; k++) {
            const int64_t i = i0 + 32 * k + lane;
            if (i0 + 32 * k >= run.hi) break;
            const int id = e0[k];
            const unsigned same = __match_any_sync(kFull, id);
            int place = -1;
            if (id >= 0) {
                place = before[id] + mine[id] + __popc(same & ((1u << lane) - 1u));
                st_i32(order + place, static_cast<int32_t>(i));
            }
            if (i < run.hi) st_i32(inverse + i, place);
            __syncwarp();
            if (id >= 0 && lane == __ffs(same) - 1) mine[id] += __popc(same);
            __syncwarp();
        }
    }
    // places that no slot takes
    for (int64_t p = kept + (int64_t)part * kSortThreads + threadIdx.x; p < slots; p += (int64_t)parts * kSortThreads)
        st_i32(order + p, -1);
}

template <class Id>
cudaError_t launch_sort(const Id *ids, int64_t slots, int n_experts, int32_t *offsets, int32_t *order,
                        int32_t *inverse, int32_t *ws, cudaStream_t st)
{
    int parts = 1;
    if (slots > kSortOneCta) {
        const int64_t need = (slots + kSortThreads - 1) / kSortThreads;
        parts = static_cast<int>(need < kSortParts ? need : kSortParts);
    }
    const size_t smem_count = sizeof(int) * kSortWarps * count_stride(n_experts);
    const size_t smem = smem_count + sizeof(int) * 2 * n_experts;
    const size_t smem_max = sizeof(int) * (kSortWarps * count_stride(kMaxExperts) + 2 * kMaxExperts);
    int grid = 0;  // not used: grid_for raises the kernels' shared memory limit
    auto place = sort_place_kernel<Id>;
    if (cudaError_t e = grid_for((const void *)place, 1, &grid, smem_max, kSortThreads)) return e;
    if (parts > 1) {
        auto count = sort_count_kernel<Id>;
        if (cudaError_t e = grid_for((const void *)count, 1, &grid, smem_max, kSortThreads)) return e;
        if (cudaError_t e =
                launch_kernel_block(count, parts, kSortThreads, smem_count, st, ids, slots, n_experts, parts, ws))
            return e;
    }
    return launch_kernel_block(place, parts, kSortThreads, smem, st, ids, slots, n_experts, parts, ws, offsets, order,
                               inverse);
}

// ---------------------------------------------------------------- places
// The place of a slot, or -1: a place outside [0, slots) counts as dropped, so that no
// index of a wrong plan leaves the buffers.
__device__ __forceinline__ int slot_place(const int32_t *inverse, int64_t slot, int64_t slots)
{
    if (!dbg_ok(inverse + slot, 4, false)) return -1;
    const int p = __ldg(inverse + slot);
    return p >= 0 && p < slots ? p : -1;
}

__device__ __forceinline__ int64_t kept_places(const int32_t *offsets, int n_experts, int64_t slots)
{
    if (!dbg_ok(offsets + n_experts, 4, false)) return slots;
    const int64_t kept = __ldg(offsets + n_experts);
    return kept < 0 ? 0 : kept < slots ? kept : slots;
}

// The warp units of a row kernel: unit u = t * per_token + v is segment v of token t's row. A
// walker steps from one of a warp's units to its next without a division.
struct Units {
    int64_t t, tokens, dt;
    int v, per_token, dv;
    __device__ __forceinline__ Units(int64_t tokens_, int per_token_) : tokens(tokens_), per_token(per_token_)
    {
        const int64_t block_warps = blockDim.x >> 5, warps = gridDim.x * block_warps;
        const int64_t u = blockIdx.x * block_warps + (threadIdx.x >> 5);
        t = u / per_token, v = (int)(u - t * per_token);
        dt = warps / per_token, dv = (int)(warps - dt * per_token);
    }
    __device__ __forceinline__ bool more() const { return t < tokens; }
    __device__ __forceinline__ void step()
    {
        t += dt, v += dv;
        if (v >= per_token) v -= per_token, t++;
    }
};

// ---------------------------------------------------------------- gather
// out[inverse[t, j]] = x[t]: a warp holds a segment of one token's row in registers and
// stores it to each of the token's places, so every row of x is read once. Rows past the
// kept places are zeros. Bound by the stores: 16384 rows of 7168 BF16 values to 131072 places
// (2.1 GB, 8 of 9 parts written) take 348 us, 6.08 TB/s, where the GPU writes at 6.55 TB/s
// without reading. Rows of odd widths: 16384 x 1001 FP16, top-6, 78 us, 2.9 TB/s.
constexpr int kGatherPieces = 4;
constexpr int kGatherRows = 4;

template <class T, bool kWide>
__global__ void __launch_bounds__(kThreads)
gather_kernel(const T *__restrict__ x, int64_t tokens, int64_t hidden, int64_t ld_x,
              const int32_t *__restrict__ inverse, int top_k, const int32_t *__restrict__ offsets, int n_experts,
              T *__restrict__ out, int64_t ld_out)
{
    using P = Piece<T>;
    using C = Cut<T, kWide>;
    pdl_begin();
    const int64_t slots = tokens * top_k;
    dbg_begin();
    dbg_allow_2d(x, tokens, hidden * sizeof(T), ld_x * sizeof(T), false);
    dbg_allow(inverse, 4 * slots, false);
    dbg_allow(offsets, 4ll * (n_experts + 1), false);
    dbg_allow_2d(out, slots, hidden * sizeof(T), ld_out * sizeof(T), true);
    dbg_ready();
    const int lane = threadIdx.x & 31;
    constexpr int kSegment = 32 * kGatherPieces;
    const int64_t pieces = C::pieces(hidden), segments = (pieces + kSegment - 1) / kSegment;
    const void *x_end = x + (tokens - 1) * ld_x + hidden;
    auto places = [&](int64_t t, int j0) {  // lane j: the place of slot j0 + j
        return j0 + lane < top_k ? slot_place(inverse, t * top_k + j0 + lane, slots) : -1;
    };
    for (Units u(tokens, (int)segments); u.more(); u.step()) {
        const int64_t t = u.t;
        const T *row = x + t * ld_x;
        const int64_t i0 = (int64_t)u.v * kSegment + lane;
        typename C::Raw raw[kGatherPieces];
        if constexpr (kWide) {
#pragma unroll
            for (int i = 0; i < kGatherPieces; i++)
                if (i0 + 32 * i < pieces) C::fetch(raw[i], row, C::column(row, i0 + 32 * i), x, x_end);
        }
        for (int j0 = 0; j0 < top_k; j0 += 32) {
            const int place = places(t, j0);
            for (unsigned rest = __ballot_sync(kFull, place >= 0); rest != 0;) {
                T *dst[kGatherRows];
                bool has[kGatherRows];
#pragma unroll
                for (int r = 0; r < kGatherRows; r++) {
                    has[r] = rest != 0;
                    dst[r] = out + __shfl_sync(kFull, place, has[r] ? __ffs(rest) - 1 : 0) * ld_out;
                    rest &= rest - 1;  // 0 stays 0
                }
#pragma unroll
                for (int r = 0; r < kGatherRows; r++) {
                    if (!has[r]) break;
                    if constexpr (!kWide) {  // every place has its own alignment; after the first from L1
#pragma unroll
                        for (int i = 0; i < kGatherPieces; i++) {
                            const int64_t c = C::column(dst[r], i0 + 32 * i);
                            if (i0 + 32 * i < pieces && C::inside(c, hidden)) C::fetch(raw[i], row, c, x, x_end);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kGatherPieces; i++) {
                        const int64_t c = C::column(dst[r], i0 + 32 * i);
                        if (i0 + 32 * i >= pieces || !C::inside(c, hidden)) continue;
                        P v;
                        C::take(v, raw[i], row, c, hidden, x, x_end);
                        C::store(v, dst[r], c, hidden);
                    }
                }
            }
        }
    }
    const int64_t kept = kept_places(offsets, n_experts, slots);
    P z;
    z.zero();
    for (Units w(slots - kept, (int)segments); w.more(); w.step()) {
        T *dst = out + (kept + w.t) * ld_out;
#pragma unroll
        for (int i = 0; i < kGatherPieces; i++) {
            const int64_t at = (int64_t)w.v * kSegment + lane + 32 * i, c = C::column(dst, at);
            if (at < pieces && C::inside(c, hidden)) C::store(z, dst, c, hidden);
        }
    }
}

// ---------------------------------------------------------------- combine
// out[t] = sum over j of w[t, j] * y[inverse[t, j]] in binary32, j ascending, dropped
// slots left out (their weights too), one rounding to T. Without weights it is the plain
// sum, which is the gather's gradient. A warp takes a segment of one token's row. Its lanes
// fetch the token's places and weights together, one each, and the rows of kCombineRows
// kept slots are loaded before any is added, so that enough loads are in flight. Bound by the
// memory: 65536 rows of 7168 BF16 values summed into 16384 take 176 to 181 us, 6.5 to 6.7 TB/s
// (254 us with one row loaded after the other). Rows of odd widths are bound by the instructions
// that put their pieces together: 16384 x 1001 FP16, top-6, 50.3 us, 3.3 TB/s, the integer units
// busy half of the time.
template <bool kWide>
constexpr int kCombinePieces = kWide ? 2 : 1;  // a piece put together holds twice the registers
constexpr int kCombineRows = 4;

template <class T, bool kWide, bool kWeights>
__global__ void __launch_bounds__(kThreads)
combine_kernel(const T *__restrict__ y, int64_t ld_y, const float *__restrict__ weights,
               const int32_t *__restrict__ inverse, int64_t tokens, int top_k, int64_t hidden, T *__restrict__ out,
               int64_t ld_out)
{
    using P = Piece<T>;
    using C = Cut<T, kWide>;
    pdl_begin();
    const int64_t slots = tokens * top_k;
    dbg_begin();
    dbg_allow_2d(y, slots, hidden * sizeof(T), ld_y * sizeof(T), false);
    dbg_allow(weights, kWeights ? 4 * slots : 0, false);
    dbg_allow(inverse, 4 * slots, false);
    dbg_allow_2d(out, tokens, hidden * sizeof(T), ld_out * sizeof(T), true);
    dbg_ready();
    const int lane = threadIdx.x & 31;
    constexpr int kPieces = kCombinePieces<kWide>, kSegment = 32 * kPieces;
    const int64_t pieces = C::pieces(hidden), segments = (pieces + kSegment - 1) / kSegment;
    const void *y_end = y + (slots - 1) * ld_y + hidden;
    for (Units u(tokens, (int)segments); u.more(); u.step()) {
        const int64_t t = u.t, i0 = (int64_t)u.v * kSegment + lane;
        T *dst = out + t * ld_out;
        int64_t c[kPieces];
        bool in[kPieces];
#pragma unroll
        for (int k = 0; k < kPieces; k++) {
            c[k] = C::column(dst, i0 + 32 * k);
            in[k] = i0 + 32 * k < pieces && C::inside(c[k], hidden);
        }
        float acc[kPieces][P::N] = {};
        for (int j0 = 0; j0 < top_k; j0 += 32) {
            const int64_t slot = t * top_k + j0 + lane;
            const int place = j0 + lane < top_k ? slot_place(inverse, slot, slots) : -1;
            float weight = 1.0f;
            if (kWeights && place >= 0 && dbg_ok(weights + slot, 4, false)) weight = __ldg(weights + slot);
            unsigned rest = __ballot_sync(kFull, place >= 0);
            while (rest != 0) {
                typename C::Raw raw[kCombineRows][kPieces];
                const T *rows[kCombineRows];
                float w[kCombineRows];
                bool has[kCombineRows];
#pragma unroll
                for (int i = 0; i < kCombineRows; i++) {
                    has[i] = rest != 0;
                    const int j = has[i] ? __ffs(rest) - 1 : 0;
                    rest &= rest - 1;  // 0 stays 0
                    w[i] = __shfl_sync(kFull, weight, j);
                    rows[i] = y + __shfl_sync(kFull, place, j) * ld_y;
#pragma unroll
                    for (int k = 0; k < kPieces; k++)
                        if (has[i] && in[k]) C::fetch(raw[i][k], rows[i], c[k], y, y_end);
                }
#pragma unroll
                for (int i = 0; i < kCombineRows; i++) {
                    if (!has[i]) break;
#pragma unroll
                    for (int k = 0; k < kPieces; k++) {
                        if (!in[k]) continue;
                        P v;
                        C::take(v, raw[i][k], rows[i], c[k], hidden, y, y_end);
#pragma unroll
                        for (int n = 0; n < P::N; n++)
                            acc[k][n] = kWeights ? __fmaf_rn(w[i], v.at(n), acc[k][n]) : __fadd_rn(acc[k][n], v.at(n));
                    }
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kPieces; k++) {
            if (!in[k]) continue;
            P v;
            v.round(acc[k]);
            C::store(v, dst, c[k], hidden);
        }
    }
}

// ---------------------------------------------------------------- combine's gradient
// dy[inverse[t, j]] = w[t, j] * dout[t] and dw[t, j] = <dout[t], y[inverse[t, j]]>, in
// one pass over dout and y. A CTA takes up to kGradSlots slots of one token; its threads
// walk the row together, each keeping one partial dot product per slot, and the partial
// products are added up in a fixed tree at the end. dw of a dropped slot is 0. Bound by the
// memory: 65536 rows of 4096 BF16 values (1.14 GB) take 176 us, 6.5 TB/s. Rows of odd widths, for
// which dout is put together anew for every slot: 16384 x 1001 FP16, top-6, 202 us, 1.8 TB/s.
constexpr int kGradSlots = 4;
constexpr int kGradMaxThreads = 256;

template <class T, bool kWide>
__global__ void __launch_bounds__(kGradMaxThreads)
combine_grad_kernel(const T *__restrict__ dout, int64_t ld_dout, const T *__restrict__ y, int64_t ld_y,
                    const float *__restrict__ weights, const int32_t *__restrict__ inverse,
                    const int32_t *__restrict__ offsets, int n_experts, int64_t tokens, int top_k, int64_t hidden,
                    T *__restrict__ dy, int64_t ld_dy, float *__restrict__ dweights)
{
    using P = Piece<T>;
    using C = Cut<T, kWide>;
    __shared__ float partial[kGradMaxThreads / 32][kGradSlots];
    pdl_begin();
    const int64_t slots = tokens * top_k;
    dbg_begin();
    dbg_allow_2d(dout, tokens, hidden * sizeof(T), ld_dout * sizeof(T), false);
    dbg_allow_2d(y, slots, hidden * sizeof(T), ld_y * sizeof(T), false);
    dbg_allow(weights, 4 * slots, false);
    dbg_allow(inverse, 4 * slots, false);
    dbg_allow(offsets, 4ll * (n_experts + 1), false);
    dbg_allow_2d(dy, slots, hidden * sizeof(T), ld_dy * sizeof(T), true);
    dbg_allow(dweights, 4 * slots, true);
    dbg_ready();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int groups = (top_k + kGradSlots - 1) / kGradSlots;
    const int64_t pieces = C::pieces(hidden);
    const void *d_end = dout + (tokens - 1) * ld_dout + hidden, *y_end = y + (slots - 1) * ld_y + hidden;
    for (int64_t u = blockIdx.x; u < tokens * groups; u += gridDim.x) {
        const int64_t t = u / groups;
        const int j0 = static_cast<int>(u - t * groups) * kGradSlots;
        int64_t place[kGradSlots];
        float w[kGradSlots], dot[kGradSlots] = {};
#pragma unroll
        for (int s = 0; s < kGradSlots; s++) {
            const int64_t slot = t * top_k + j0 + s;
            place[s] = j0 + s < top_k ? slot_place(inverse, slot, slots) : -1;
            w[s] = j0 + s < top_k && dbg_ok(weights + slot, 4, false) ? __ldg(weights + slot) : 0.0f;
        }
        const T *d_row = dout + t * ld_dout;
        for (int64_t i = threadIdx.x; i < pieces; i += blockDim.x) {
            typename C::Raw d_raw[kWide ? 1 : kGradSlots], y_raw[kGradSlots];
            if constexpr (kWide) C::fetch(d_raw[0], d_row, C::column(d_row, i), dout, d_end);
#pragma unroll
            for (int s = 0; s < kGradSlots; s++) {
                const int64_t c = place[s] >= 0 ? C::column(dy + place[s] * ld_dy, i) : hidden;
                if (!C::inside(c, hidden)) continue;
                if constexpr (!kWide) C::fetch(d_raw[s], d_row, c, dout, d_end);
                C::fetch(y_raw[s], y + place[s] * ld_y, c, y, y_end);
            }
#pragma unroll
            for (int s = 0; s < kGradSlots; s++) {
                T *dst = dy + place[s] * ld_dy;
                const int64_t c = place[s] >= 0 ? C::column(dst, i) : hidden;
                if (!C::inside(c, hidden)) continue;
                P d, v, g;
                C::take(d, d_raw[kWide ? 0 : s], d_row, c, hidden, dout, d_end);
                C::take(v, y_raw[s], y + place[s] * ld_y, c, hidden, y, y_end);
                C::keep(d, c, hidden);
                C::keep(v, c, hidden);
                float scaled[P::N];
#pragma unroll
                for (int n = 0; n < P::N; n++) {
                    dot[s] = __fmaf_rn(d.at(n), v.at(n), dot[s]);
                    scaled[n] = __fmul_rn(w[s], d.at(n));
                }
                g.round(scaled);
                C::store(g, dst, c, hidden);
            }
        }
#pragma unroll
        for (int s = 0; s < kGradSlots; s++) {
#pragma unroll
            for (int b = 16; b > 0; b >>= 1) dot[s] = __fadd_rn(dot[s], __shfl_xor_sync(kFull, dot[s], b));
            if (lane == 0) partial[warp][s] = dot[s];
        }
        __syncthreads();
        if (threadIdx.x < kGradSlots && j0 + (int)threadIdx.x < top_k) {
            float sum = 0.0f;
            for (int i = 0; i < warps; i++) sum = __fadd_rn(sum, partial[i][threadIdx.x]);
            float *dst = dweights + t * top_k + j0 + threadIdx.x;
            if (dbg_ok(dst, 4, true)) *dst = sum;
        }
        __syncthreads();
    }
    const int64_t kept = kept_places(offsets, n_experts, slots);
    P z;
    z.zero();
    for (int64_t p = kept + blockIdx.x; p < slots; p += gridDim.x)
        for (int64_t i = threadIdx.x; i < pieces; i += blockDim.x) {
            T *dst = dy + p * ld_dy;
            const int64_t c = C::column(dst, i);
            if (C::inside(c, hidden)) C::store(z, dst, c, hidden);
        }
}

// Launches a kernel of warp units. Few units go out in small CTAs, so that they spread over
// all SMs: 16 tokens' combine of 7168 columns in 28 CTAs of 8 warps took 5.0 us.
template <typename... KArgs, typename... Args>
cudaError_t launch_units(void (*kernel)(KArgs...), int64_t units, cudaStream_t st, Args... args)
{
    int sms = 1, grid = 0;
    if (cudaError_t e = sm_count(&sms)) return e;
    const int64_t per_sm = (units + sms - 1) / sms;
    const int block = per_sm >= 8 ? 256 : per_sm >= 4 ? 128 : per_sm >= 2 ? 64 : 32;
    if (cudaError_t e = grid_for((const void *)kernel, units, &grid, 0, block)) return e;
    return launch_kernel_block(kernel, grid, block, 0, st, args...);
}

int64_t row_units(int64_t rows, int64_t pieces, int per_segment)
{
    return rows * ((pieces + per_segment - 1) / per_segment);
}

template <class T, bool kWide>
cudaError_t launch_gather_t(const RowArgs &a, const void *x, int64_t ld_x, const int32_t *offsets, int n_experts,
                            void *out, int64_t ld_out, cudaStream_t st)
{
    const int64_t units = row_units(a.tokens, Cut<T, kWide>::pieces(a.hidden), 32 * kGatherPieces);
    return launch_units(gather_kernel<T, kWide>, units, st, static_cast<const T *>(x), a.tokens, a.hidden, ld_x,
                        a.inverse, a.top_k, offsets, n_experts, static_cast<T *>(out), ld_out);
}

template <class T, bool kWide>
cudaError_t launch_combine_t(const RowArgs &a, const void *y, int64_t ld_y, const float *weights, void *out,
                             int64_t ld_out, cudaStream_t st)
{
    auto kernel = weights ? combine_kernel<T, kWide, true> : combine_kernel<T, kWide, false>;
    const int64_t units = row_units(a.tokens, Cut<T, kWide>::pieces(a.hidden), 32 * kCombinePieces<kWide>);
    return launch_units(kernel, units, st, static_cast<const T *>(y), ld_y, weights, a.inverse, a.tokens, a.top_k,
                        a.hidden, static_cast<T *>(out), ld_out);
}

template <class T, bool kWide>
cudaError_t launch_combine_grad_t(const RowArgs &a, const void *dout, int64_t ld_dout, const void *y, int64_t ld_y,
                                  const float *weights, const int32_t *offsets, int n_experts, void *dy, int64_t ld_dy,
                                  float *dweights, cudaStream_t st)
{
    auto kernel = combine_grad_kernel<T, kWide>;
    const int64_t pieces = Cut<T, kWide>::pieces(a.hidden);
    const int64_t units = a.tokens * ((a.top_k + kGradSlots - 1) / kGradSlots);
    int sms = 1, grid = 0;
    if (cudaError_t e = sm_count(&sms)) return e;
    // Few units go out in few rounds over the row, else the CTA is the largest whose rounds (four,
    // or as many as it takes) are fullest: 257 pieces take 3 rounds of 96 threads (12.6 us for
    // 3000 tokens of 1028 FP32 columns; 14.5 us with 160 threads, 16.0 us with 256).
    const int64_t least = (pieces + kGradMaxThreads - 1) / kGradMaxThreads;
    const int64_t most = units < (int64_t)16 * sms || least > 4 ? least : 4;
    int block = 32;  // without columns one warp writes the zeros of dw
    double fullest = 0.0;
    for (int threads = kGradMaxThreads; threads >= 32; threads -= 32) {
        const int64_t rounds = (pieces + threads - 1) / threads;
        const double full = (double)pieces / (double)(rounds * threads);
        if (rounds <= most && full > fullest) {
            fullest = full;
            block = threads;
        }
    }
    if (cudaError_t e = grid_for((const void *)kernel, units * (block / 32), &grid, 0, block)) return e;
    return launch_kernel_block(kernel, grid, block, 0, st, static_cast<const T *>(dout), ld_dout,
                               static_cast<const T *>(y), ld_y, weights, a.inverse, offsets, n_experts, a.tokens,
                               a.top_k, a.hidden, static_cast<T *>(dy), ld_dy, dweights);
}

// Calls F<T, wide>(args...) for the row type.
#define BQK_ROWS(type, wide, F, ...)                                                                        \
    switch (type) {                                                                                         \
    case kBf16: return wide ? F<__nv_bfloat16, true>(__VA_ARGS__) : F<__nv_bfloat16, false>(__VA_ARGS__);   \
    case kF16: return wide ? F<__half, true>(__VA_ARGS__) : F<__half, false>(__VA_ARGS__);                  \
    default: return wide ? F<float, true>(__VA_ARGS__) : F<float, false>(__VA_ARGS__);                      \
    }

}  // namespace

cudaError_t launch_expert_sort(const void *ids, bool ids_are_i64, int64_t slots, int n_experts, int32_t *offsets,
                               int32_t *order, int32_t *inverse, int32_t *ws, cudaStream_t st)
{
    if (ids_are_i64)
        return launch_sort(static_cast<const int64_t *>(ids), slots, n_experts, offsets, order, inverse, ws, st);
    return launch_sort(static_cast<const int32_t *>(ids), slots, n_experts, offsets, order, inverse, ws, st);
}

cudaError_t launch_expert_gather(int type, const RowArgs &a, const void *x, int64_t ld_x, const int32_t *offsets,
                                 int n_experts, void *out, int64_t ld_out, cudaStream_t st)
{
    const int size = row_type_bytes(type);
    const bool wide = wide_rows(x, a.hidden, ld_x, size) && wide_rows(out, a.hidden, ld_out, size);
    BQK_ROWS(type, wide, launch_gather_t, a, x, ld_x, offsets, n_experts, out, ld_out, st)
}

cudaError_t launch_expert_combine(int type, const RowArgs &a, const void *y, int64_t ld_y, const float *weights,
                                  void *out, int64_t ld_out, cudaStream_t st)
{
    const int size = row_type_bytes(type);
    const bool wide = wide_rows(y, a.hidden, ld_y, size) && wide_rows(out, a.hidden, ld_out, size);
    BQK_ROWS(type, wide, launch_combine_t, a, y, ld_y, weights, out, ld_out, st)
}

cudaError_t launch_expert_combine_grad(int type, const RowArgs &a, const void *dout, int64_t ld_dout, const void *y,
                                       int64_t ld_y, const float *weights, const int32_t *offsets, int n_experts,
                                       void *dy, int64_t ld_dy, float *dweights, cudaStream_t st)
{
    const int size = row_type_bytes(type);
    const bool wide = wide_rows(dout, a.hidden, ld_dout, size) && wide_rows(y, a.hidden, ld_y, size) &&
                      wide_rows(dy, a.hidden, ld_dy, size);
    BQK_ROWS(type, wide, launch_combine_grad_t, a, dout, ld_dout, y, ld_y, weights, offsets, n_experts, dy, ld_dy,
             dweights, st)
}

cudaError_t read_wait_counters_experts(unsigned long long (&v)[3]) { return read_wait_counters(v); }

}  // namespace bqk
