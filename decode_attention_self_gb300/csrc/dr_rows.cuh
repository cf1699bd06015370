// Ragged token batches: row b holds tokens [row_start[b], row_start[b+1]).
#pragma once

#include "dr_device.cuh"

namespace dr {

// The row of token t, by the whole warp (each lane gets it), with the row's token range [s0, s1); -1 when t is in no
// row.  row_start is expected to rise from 0 to at most T; whatever it holds, the result is a row whose range, cut to
// [0, T), holds t, or -1.  The first guess is the row of an even batch, which is exact for one token per row; then a
// 32-way search (two dependent loads for up to 1024 rows).  With err, `warps` warps, of which this
// is number `warp`, look over all rows between them, one per lane at a time (the first is loaded while the row is found).
__device__ __forceinline__ int find_row(const int32_t *row_start, int B, int T, int t, int lane, int &s0, int &s1,
                                        int32_t *err, long long warp, long long warps) {
    const long long x = 32 * warp + lane;   // the first row that this lane looks over
    const bool looks = err && x < B;
    int from = 0, to = 0;
    if (looks) {
        from = __ldg(row_start + x);
        to = __ldg(row_start + x + 1);
    }
    int b = (int)((long long)t * B / T);
    s0 = __ldg(row_start + b);
    s1 = __ldg(row_start + b + 1);
    if (!(s0 <= t && t < s1)) {
        int lo = 0, n = B;   // the last b in [lo, lo + n) with row_start[b] <= t
        while (n > 1) {
            const int step = (n + 31) / 32;
            const int probe = lane * step;
            const bool le = probe < n && __ldg(row_start + lo + probe) <= t;
            const unsigned m = __ballot_sync(0xFFFFFFFFu, le);
            const int last = m ? 31 - __clz(m) : 0;
            lo += last * step;
            n = min(step, n - last * step);
        }
        b = lo;
        s0 = __ldg(row_start + b);
        s1 = __ldg(row_start + b + 1);
    }
    if (looks) {
        bool bad = from < 0 || to < from || to > T || (x == 0 && from != 0);
#pragma unroll 4
        for (long long y = x + 32 * warps; y < B; y += 32 * warps) {
            const int a = __ldg(row_start + y), e = __ldg(row_start + y + 1);
            bad |= a < 0 || e < a || e > T;
        }
        if (bad) flag_error(err, DR_ERRF_ROW_START);
    }
    if (!(s0 >= 0 && s0 <= t && t < s1)) return -1;
    s1 = min(s1, T);
    return b;
}

}  // namespace dr
