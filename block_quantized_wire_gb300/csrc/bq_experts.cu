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
// counters in shared memory, one per expert. It counts its slots 32 at a time:
// match_any gives each lane the lanes with the same id, and the lowest of them adds
// their number, so no counter is ever contended. The counters are then turned into the
// first place of each (warp, expert), and a second walk over the same slots hands the
// places out in lane order. Nothing depends on the order in which warps run.
//
// Up to kSortOneCta slots one CTA does all of it in one launch. More slots are cut into
// `parts` runs, one CTA each: a first launch writes each run's counts to the workspace,
// the second adds up the runs before its own and all runs, and places.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int64_t kSortOneCta = 4096;

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

// count[w][e] over this CTA's run; the caller synchronizes.
template <class Id>
__device__ __forceinline__ void count_run(const Id *ids, SlotRun run, int n_experts, int *mine, int lane)
{
    for (int64_t i0 = run.lo; i0 < run.hi; i0 += 32) {
        const int64_t i = i0 + lane;
        const int e = i < run.hi ? slot_expert(ids, i, n_experts) : -1;
        const unsigned same = __match_any_sync(kFull, e);
        if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
        __syncwarp();
    }
}

template <class Id>
__global__ void __launch_bounds__(kSortThreads)
sort_count_kernel(const Id *__restrict__ ids, int64_t slots, int n_experts, int parts, int32_t *__restrict__ ws)
{
    extern __shared__ int count[];  // [kSortWarps][n_experts]
    pdl_begin();
    dbg_begin();
    dbg_allow(ids, slots * (int64_t)sizeof(Id), false);
    dbg_allow(ws, 4ll * parts * n_experts, true);
    dbg_ready();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < kSortWarps * n_experts; i += kSortThreads) count[i] = 0;
    __syncthreads();
    count_run(ids, warp_run(slots, parts, blockIdx.x, warp), n_experts, count + warp * n_experts, lane);
    __syncthreads();
    for (int e = threadIdx.x; e < n_experts; e += kSortThreads) {
        int sum = 0;
        for (int w = 0; w < kSortWarps; w++) sum += count[w * n_experts + e];
        st_i32(ws + (int64_t)blockIdx.x * n_experts + e, sum);
    }
}

template <class Id>
__global__ void __launch_bounds__(kSortThreads)
sort_place_kernel(const Id *__restrict__ ids, int64_t slots, int n_experts, int parts, const int32_t *__restrict__ ws,
                  int32_t *__restrict__ offsets, int32_t *__restrict__ order, int32_t *__restrict__ inverse)
{
    extern __shared__ int count[];  // [kSortWarps][n_experts], then total and before [n_experts] each
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
    int *total = count + kSortWarps * n_experts, *before = total + n_experts;
    for (int i = threadIdx.x; i < (kSortWarps + 2) * n_experts; i += kSortThreads) count[i] = 0;
    __syncthreads();
    const SlotRun run = warp_run(slots, parts, part, warp);
    int *mine = count + warp * n_experts;
    count_run(ids, run, n_experts, mine, lane);
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
    // Thread e: the expert's counts over the warps become first places within the run, and
    // a scan over the experts gives its first place among all.
    const int e = threadIdx.x;
    int run_total = 0;
    if (e < n_experts) {
        for (int w = 0; w < kSortWarps; w++) {
            const int v = count[w * n_experts + e];
            count[w * n_experts + e] = run_total;
            run_total += v;
        }
    }
    const int all = e < n_experts ? (parts > 1 ? total[e] : run_total) : 0;
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
        for (int w = 0; w < kSortWarps; w++) count[w * n_experts + e] += first + before[e];
        if (part == 0) {
            st_i32(offsets + e, first);
            if (e == n_experts - 1) st_i32(offsets + n_experts, kept);
        }
    }
    __syncthreads();
    for (int64_t i0 = run.lo; i0 < run.hi; i0 += 32) {
        const int64_t i = i0 + lane;
        const int id = i < run.hi ? slot_expert(ids, i, n_experts) : -1;
        const unsigned same = __match_any_sync(kFull, id);
        int place = -1;
        if (id >= 0) {
            place = mine[id] + __popc(same & ((1u << lane) - 1u));
            st_i32(order + place, static_cast<int32_t>(i));
        }
        if (i < run.hi) st_i32(inverse + i, place);
        __syncwarp();
        if (id >= 0 && lane == __ffs(same) - 1) mine[id] += __popc(same);
        __syncwarp();
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
    const size_t smem_count = sizeof(int) * kSortWarps * n_experts, smem = smem_count + sizeof(int) * 2 * n_experts;
    const size_t smem_max = sizeof(int) * (kSortWarps + 2) * kMaxExperts;
    int grid = 0;  // not used: grid_for raises the kernels' shared memory limit
    auto place = sort_place_kernel<Id>;
    if (cudaError_t e = grid_for((const void *)place, 1, &grid, smem_max, kSortThreads)) return e;
    if (parts > 1) {
        auto count = sort_count_kernel<Id>;
        if (cudaError_t e = grid_for((const void *)count, 1, &grid, smem_max, kSortThreads)) return e;
        if (cudaError_t e = launch_kernel_block(count, parts, kSortThreads, smem_count, st, ids, slots, n_experts, parts, ws))
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

// ---------------------------------------------------------------- gather
// out[inverse[t, j]] = x[t]: a warp holds a segment of one token's row in registers and
// stores it to each of the token's places, so every row of x is read once. Rows past the
// kept places are zeros.
constexpr int kGatherPieces = 4;

template <class T, bool kWide>
__global__ void __launch_bounds__(kThreads)
gather_kernel(const T *__restrict__ x, int64_t tokens, int64_t hidden, int64_t ld_x, const int32_t *__restrict__ inverse,
              int top_k, const int32_t *__restrict__ offsets, int n_experts, T *__restrict__ out, int64_t ld_out)
{
    using P = Piece<T, kWide>;
    pdl_begin();
    const int64_t slots = tokens * top_k;
    dbg_begin();
    dbg_allow_2d(x, tokens, hidden * sizeof(T), ld_x * sizeof(T), false);
    dbg_allow(inverse, 4 * slots, false);
    dbg_allow(offsets, 4ll * (n_experts + 1), false);
    dbg_allow_2d(out, slots, hidden * sizeof(T), ld_out * sizeof(T), true);
    dbg_ready();
    const int lane = threadIdx.x & 31;
    const int64_t warp = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
    constexpr int kSegment = 32 * P::N * kGatherPieces;
    const int64_t segments = (hidden + kSegment - 1) / kSegment;
    for (int64_t u = warp; u < tokens * segments; u += warps) {
        const int64_t t = u / segments, c0 = (u - t * segments) * kSegment + lane * P::N;
        P v[kGatherPieces];
#pragma unroll
        for (int i = 0; i < kGatherPieces; i++)
            if (c0 + i * 32 * P::N < hidden) v[i].load(x + t * ld_x + c0 + i * 32 * P::N);
        for (int j = 0; j < top_k; j++) {
            const int p = slot_place(inverse, t * top_k + j, slots);
            if (p < 0) continue;
            T *row = out + p * ld_out + c0;
#pragma unroll
            for (int i = 0; i < kGatherPieces; i++)
                if (c0 + i * 32 * P::N < hidden) v[i].store(row + i * 32 * P::N);
        }
    }
    const int64_t kept = kept_places(offsets, n_experts, slots);
    P z;
    z.zero();
    for (int64_t u = warp; u < (slots - kept) * segments; u += warps) {
        const int64_t r = u / segments, c0 = (u - r * segments) * kSegment + lane * P::N;
        T *row = out + (kept + r) * ld_out + c0;
#pragma unroll
        for (int i = 0; i < kGatherPieces; i++)
            if (c0 + i * 32 * P::N < hidden) z.store(row + i * 32 * P::N);
    }
}

// ---------------------------------------------------------------- combine
// out[t] = sum over j of w[t, j] * y[inverse[t, j]] in binary32, j ascending, dropped
// slots left out (their weights too), one rounding to T. Without weights it is the plain
// sum, which is the gather's gradient.
constexpr int kCombinePieces = 2;

template <class T, bool kWide, bool kWeights>
__global__ void __launch_bounds__(kThreads)
combine_kernel(const T *__restrict__ y, int64_t ld_y, const float *__restrict__ weights,
               const int32_t *__restrict__ inverse, int64_t tokens, int top_k, int64_t hidden, T *__restrict__ out,
               int64_t ld_out)
{
    using P = Piece<T, kWide>;
    pdl_begin();
    const int64_t slots = tokens * top_k;
    dbg_begin();
    dbg_allow_2d(y, slots, hidden * sizeof(T), ld_y * sizeof(T), false);
    dbg_allow(weights, kWeights ? 4 * slots : 0, false);
    dbg_allow(inverse, 4 * slots, false);
    dbg_allow_2d(out, tokens, hidden * sizeof(T), ld_out * sizeof(T), true);
    dbg_ready();
    const int lane = threadIdx.x & 31;
    const int64_t warp = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
    constexpr int kSegment = 32 * P::N * kCombinePieces;
    const int64_t segments = (hidden + kSegment - 1) / kSegment;
    for (int64_t u = warp; u < tokens * segments; u += warps) {
        const int64_t t = u / segments, c0 = (u - t * segments) * kSegment + lane * P::N;
        float acc[kCombinePieces][P::N] = {};
#pragma unroll 4
        for (int j = 0; j < top_k; j++) {
            const int p = slot_place(inverse, t * top_k + j, slots);
            if (p < 0) continue;
            const float w = kWeights && dbg_ok(weights + t * top_k + j, 4, false) ? __ldg(weights + t * top_k + j) : 1.0f;
            const T *row = y + p * ld_y + c0;
#pragma unroll
            for (int i = 0; i < kCombinePieces; i++) {
                if (c0 + i * 32 * P::N < hidden) {
                    P v;
                    v.load(row + i * 32 * P::N);
#pragma unroll
                    for (int n = 0; n < P::N; n++)
                        acc[i][n] = kWeights ? __fmaf_rn(w, v.at(n), acc[i][n]) : __fadd_rn(acc[i][n], v.at(n));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kCombinePieces; i++) {
            if (c0 + i * 32 * P::N < hidden) {
                P v;
#pragma unroll
                for (int n = 0; n < P::N; n++) v.set(n, acc[i][n]);
                v.store(out + t * ld_out + c0 + i * 32 * P::N);
            }
        }
    }
}

// ---------------------------------------------------------------- combine's gradient
// dy[inverse[t, j]] = w[t, j] * dout[t] and dw[t, j] = <dout[t], y[inverse[t, j]]>, in
// one pass over dout and y. A CTA takes up to kGradSlots slots of one token; its threads
// walk the row together, each keeping one partial dot product per slot, and the partial
// products are added up in a fixed tree at the end. dw of a dropped slot is 0.
constexpr int kGradSlots = 4;
constexpr int kGradMaxThreads = 256;

template <class T, bool kWide>
__global__ void __launch_bounds__(kGradMaxThreads)
combine_grad_kernel(const T *__restrict__ dout, int64_t ld_dout, const T *__restrict__ y, int64_t ld_y,
                    const float *__restrict__ weights, const int32_t *__restrict__ inverse,
                    const int32_t *__restrict__ offsets, int n_experts, int64_t tokens, int top_k, int64_t hidden,
                    T *__restrict__ dy, int64_t ld_dy, float *__restrict__ dweights)
{
    using P = Piece<T, kWide>;
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
    const int64_t step = (int64_t)blockDim.x * P::N;
    for (int64_t u = blockIdx.x; u < tokens * groups; u += gridDim.x) {
        const int64_t t = u / groups;
        const int j0 = static_cast<int>(u - t * groups) * kGradSlots;
        int64_t place[kGradSlots];
        float w[kGradSlots], dot[kGradSlots] = {};
#pragma unroll
        for (int s = 0; s < kGradSlots; s++) {
            const int64_t slot = t * top_k + j0 + s;
            place[s] = j0 + s < top_k ? slot_place(inverse, slot, slots) : -1;
            w[s] = place[s] >= 0 && dbg_ok(weights + slot, 4, false) ? __ldg(weights + slot) : 0.0f;
        }
        for (int64_t c = threadIdx.x * P::N; c < hidden; c += step) {
            P d, v[kGradSlots];
            d.load(dout + t * ld_dout + c);
#pragma unroll
            for (int s = 0; s < kGradSlots; s++)
                if (place[s] >= 0) v[s].load(y + place[s] * ld_y + c);
#pragma unroll
            for (int s = 0; s < kGradSlots; s++) {
                if (place[s] < 0) continue;
                P g;
#pragma unroll
                for (int n = 0; n < P::N; n++) {
                    dot[s] = __fmaf_rn(d.at(n), v[s].at(n), dot[s]);
                    g.set(n, __fmul_rn(w[s], d.at(n)));
                }
                g.store(dy + place[s] * ld_dy + c);
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
        for (int64_t c = threadIdx.x * P::N; c < hidden; c += step) z.store(dy + p * ld_dy + c);
}

// Warps that the grid of a row kernel needs, for grid_for.
int64_t row_units(int64_t rows, int64_t hidden, int per_segment) { return rows * ((hidden + per_segment - 1) / per_segment); }

template <class T, bool kWide>
cudaError_t launch_gather_t(const RowArgs &a, const void *x, int64_t ld_x, const int32_t *offsets, int n_experts,
                            void *out, int64_t ld_out, cudaStream_t st)
{
    auto kernel = gather_kernel<T, kWide>;
    int grid = 0;
    const int64_t units = row_units(a.tokens * a.top_k, a.hidden, 32 * Piece<T, kWide>::N * kGatherPieces);
    if (cudaError_t e = grid_for((const void *)kernel, units, &grid)) return e;
    return launch_kernel(kernel, grid, st, static_cast<const T *>(x), a.tokens, a.hidden, ld_x, a.inverse, a.top_k,
                         offsets, n_experts, static_cast<T *>(out), ld_out);
}

template <class T, bool kWide>
cudaError_t launch_combine_t(const RowArgs &a, const void *y, int64_t ld_y, const float *weights, void *out,
                             int64_t ld_out, cudaStream_t st)
{
    auto kernel = weights ? combine_kernel<T, kWide, true> : combine_kernel<T, kWide, false>;
    int grid = 0;
    const int64_t units = row_units(a.tokens, a.hidden, 32 * Piece<T, kWide>::N * kCombinePieces);
    if (cudaError_t e = grid_for((const void *)kernel, units, &grid)) return e;
    return launch_kernel(kernel, grid, st, static_cast<const T *>(y), ld_y, weights, a.inverse, a.tokens, a.top_k,
                         a.hidden, static_cast<T *>(out), ld_out);
}

template <class T, bool kWide>
cudaError_t launch_combine_grad_t(const RowArgs &a, const void *dout, int64_t ld_dout, const void *y, int64_t ld_y,
                                  const float *weights, const int32_t *offsets, int n_experts, void *dy, int64_t ld_dy,
                                  float *dweights, cudaStream_t st)
{
    auto kernel = combine_grad_kernel<T, kWide>;
    const int64_t pieces = (a.hidden + Piece<T, kWide>::N - 1) / Piece<T, kWide>::N;
    const int64_t want = (pieces + 31) / 32 * 32;  // without columns one warp writes the zeros of dw
    const int block = static_cast<int>(want < 32 ? 32 : want < kGradMaxThreads ? want : kGradMaxThreads);
    const int64_t units = a.tokens * ((a.top_k + kGradSlots - 1) / kGradSlots);
    int grid = 0;
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
    return ids_are_i64 ? launch_sort(static_cast<const int64_t *>(ids), slots, n_experts, offsets, order, inverse, ws, st)
                       : launch_sort(static_cast<const int32_t *>(ids), slots, n_experts, offsets, order, inverse, ws, st);
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
