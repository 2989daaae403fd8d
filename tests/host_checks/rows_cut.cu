// The cutting of rows into pieces (bq_rows.cuh), evaluated on the host: which 16-byte windows
// the expert-layer kernels would load. Prints a line for each check that fails.
#include <cstdio>

#include "bq_rows.cuh"

namespace {
int failures = 0;
void expect(bool ok, const char *what, const char *type, long long at)
{
    if (!ok && failures++ < 20) std::printf("%s: %s (%lld)\n", type, what, at);
}

const void *address(uintptr_t a) { return reinterpret_cast<const void *>(a); }

template <class T>
void check(const char *type)
{
    using Narrow = bqk::Cut<T, false>;
    using Wide = bqk::Cut<T, true>;
    constexpr int kSize = sizeof(T);

    // Rows without columns have no pieces. Their tensors have a null pointer and rows one
    // value apart: no piece of any row may be loaded.
    expect(Narrow::pieces(0) == 0 && Wide::pieces(0) == 0, "pieces of no columns", type, Narrow::pieces(0));
    for (int rows : {1, 2, 17, 32, 64, 2000}) {
        const T *null = nullptr;
        const uintptr_t end = (uintptr_t)(rows - 1) * kSize;
        for (int row = 0; row < rows; row++) {
            const T *at = reinterpret_cast<const T *>((uintptr_t)row * kSize);
            for (int64_t i = 0; i < Narrow::pieces(0); i++) {
                const int64_t c = Narrow::column(at, i);
                const T *p = reinterpret_cast<const T *>((uintptr_t)at + (uintptr_t)(c * kSize));
                expect(!Narrow::inside(c, 0) || !Narrow::windowed(p, null, address(end)), "a row without columns is read",
                       type, row);
            }
        }
    }

    // A window is the 32 bytes from the 16-byte word that holds p, all inside [lo, hi).
    for (uintptr_t lo : {(uintptr_t)0, (uintptr_t)kSize, (uintptr_t)4096, (uintptr_t)4096 + kSize})
        for (uintptr_t bytes = 0; bytes <= 96; bytes += kSize)
            for (intptr_t d = -64; d <= 160; d += kSize) {
                const uintptr_t p = lo + (uintptr_t)d, hi = lo + bytes;  // below 0 it wraps, as a pointer does
                bool want = false;
                if (d >= 0) {
                    const uintptr_t a = p / 16 * 16;
                    want = a >= lo && hi >= a && hi - a >= 32;
                }
                expect(Narrow::windowed(reinterpret_cast<const T *>(p), address(lo), address(hi)) == want, "window", type,
                       (long long)d);
            }

    // The pieces of a row cover each column once, at every alignment of the row.
    for (int64_t hidden : {1, 2, 7, 8, 9, 31, 100})
        for (int skew = 0; skew < 16 / kSize; skew++) {
            const T *row = reinterpret_cast<const T *>((uintptr_t)4096 + skew * kSize);
            int64_t next = 0;
            for (int64_t i = 0; i < Narrow::pieces(hidden); i++) {
                const int64_t c = Narrow::column(row, i);
                if (!Narrow::inside(c, hidden)) continue;
                expect((c < 0 ? 0 : c) == next, "a gap between pieces", type, c);
                next = c + Narrow::N < hidden ? c + Narrow::N : hidden;
            }
            expect(next == hidden, "columns left over", type, next);
        }
}
}  // namespace

int main()
{
    check<__nv_bfloat16>("bf16");
    check<__half>("f16");
    check<float>("f32");
    std::printf("%d failures\n", failures);
    return failures != 0;
}
