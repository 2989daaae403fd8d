// Passes over rows (bq_rows.cuh), evaluated on the host up to the largest number of rows.
#include <climits>
#include <cstdio>

#include "bq_rows.cuh"

int main()
{
    int failures = 0;
    for (int cap : {1, 3, 4, 8, 16, INT_MAX})
        for (int rows : {0, 1, 2, 3, 4, 5, 15, 16, 17, 33, 100})
            for (int hi : {rows, rows + 7, INT_MAX}) {
                const int lo = hi - rows, want = rows / cap + (rows % cap != 0);
                int passes = 0, covered = 0;
                for (int p0 = lo; p0 < hi && passes <= rows; p0 = bqk::next_pass(p0, hi, cap)) {
                    const int next = bqk::next_pass(p0, hi, cap);
                    if (next <= p0 || next - p0 > cap) failures++;
                    covered += next - p0;
                    passes++;
                }
                if (passes != want || covered != rows || bqk::pass_count(rows, cap) != want) {
                    std::printf("cap %d, rows [%d, %d): %d passes over %d rows\n", cap, lo, hi, passes, covered);
                    failures++;
                }
            }
    for (int cap : {1, 4, 16, INT_MAX})
        if (bqk::pass_count(INT_MAX, cap) != INT_MAX / cap + (INT_MAX % cap != 0)) {
            std::printf("cap %d: %d passes over all rows\n", cap, bqk::pass_count(INT_MAX, cap));
            failures++;
        }
    return failures != 0;
}
