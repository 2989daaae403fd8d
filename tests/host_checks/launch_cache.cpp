// The launch cache (bq_launch_cache.h) over a fake runtime: a kernel's shared memory limit
// never falls below what a call was granted, whatever was asked for before and since.
#include <cstdio>
#include <map>
#include <utility>

#include "bq_launch_cache.h"

namespace {
struct Fake {
    int device = 0, queries = 0, fail = 0;
    std::map<std::pair<const void *, int>, size_t> limits;
    size_t &limit_of(const void *k) { return limits.emplace(std::make_pair(k, device), 48 * 1024).first->second; }
    int limit(const void *k, size_t *bytes) { return *bytes = limit_of(k), fail; }
    int raise_limit(const void *k, size_t bytes) { return limit_of(k) = bytes, 0; }
    int ctas_per_sm(const void *k, int block, size_t smem, int *ctas)
    {
        queries++;
        if (smem > limit_of(k)) return 1;  // as the runtime answers
        *ctas = smem > 200 * 1024 ? 0 : (int)(2048 / block) + (int)(smem % 7);
        return 0;
    }
};

int failures = 0;
void expect(bool ok, const char *what)
{
    if (!ok && failures++ < 10) std::printf("%s\n", what);
}
const void *kernel(int i) { return reinterpret_cast<const void *>((uintptr_t)0x7f0000100000 + 64 * (uintptr_t)i); }
}  // namespace

int main()
{
    Fake rt;
    int ctas = 0;
    static bqk::LaunchCache<Fake> cache;
    std::map<std::pair<const void *, int>, size_t> granted;
    auto call = [&](const void *k, size_t smem, int block) {
        ctas = -1;
        expect(cache.ctas_per_sm(rt, k, smem, block, rt.device, &ctas) == 0, "a call failed");
        const int want = smem > 200 * 1024 ? 1 : 2048 / block + (int)(smem % 7);
        expect(ctas == want, "a wrong number of CTAs");
        size_t &most = granted[{k, rt.device}];
        if (smem > most) most = smem;
        for (const auto &g : granted) expect(rt.limits[g.first] >= g.second, "a limit fell below a granted size");
    };

    // one kernel is granted much; then more keys than any table holds; then it asks for less
    call(kernel(0), 180 * 1024, 256);
    for (int i = 0; i < 5000; i++) call(kernel(1 + i % 40), 16 * (size_t)(i / 40), 32 << (i % 4));
    for (size_t smem : {60 * 1024, 50 * 1024, 0, 220 * 1024, 100 * 1024}) call(kernel(0), smem, 256);
    rt.device = 1;
    call(kernel(0), 70 * 1024, 256);
    rt.device = 0;
    call(kernel(0), 180 * 1024, 256);

    // some hundred keys in use are found again without a query
    static bqk::LaunchCache<Fake> fresh;
    for (int round = 0; round < 2; round++) {
        const int before = rt.queries;
        for (int i = 0; i < 120; i++)
            expect(fresh.ctas_per_sm(rt, kernel(i / 4), 1024 * (i % 4), 256, 0, &ctas) == 0, "a call failed");
        expect(rt.queries - before == (round == 0 ? 120 : 0), "a key was queried twice, or not at all");
    }

    // an error is the caller's, and is not remembered as an answer
    rt.fail = 7;
    expect(cache.ctas_per_sm(rt, kernel(60), 64, 256, 0, &ctas) == 7, "an error was lost");
    rt.fail = 0;
    call(kernel(60), 64, 256);
    return failures != 0;
}
