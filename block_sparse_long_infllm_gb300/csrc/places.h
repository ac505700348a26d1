// places.h -- index arithmetic of the kernels that a host compiler builds too, so that it can be checked
// for every small size without a GPU.
#pragma once

#include <limits.h>

#ifdef __CUDACC__
#define INFLLMV2_HD __host__ __device__ __forceinline__
#else
#define INFLLMV2_HD inline
#endif

namespace infllmv2 {

// Token t of sequence b, of len tokens; len 0: the row belongs to no sequence that can be taken.
struct PackedRow {
    int b, t, len;
};

// Where row r of a packed call is, cu[0 .. B] the sequences' offsets, by binary search for the last one at
// or below r.  A sequence is taken whole or not at all, whatever the offsets hold: it has to lie within
// [0, rows) and be at most Tq long, and every offset that the search compared r with has to leave all of
// its rows on one side, so each of them takes the same way through the search and ends here too.  (Offsets
// that ascend from 0 to at most `rows` always do.)
INFLLMV2_HD PackedRow packed_row(const int* cu, int B, int r, int rows, int Tq) {
    int lo = 0, hi = B, below = INT_MIN, above = INT_MAX;
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2, x = cu[mid];
        if (x <= r) {
            lo = mid;
            below = x > below ? x : below;
        } else {
            hi = mid;
            above = x < above ? x : above;
        }
    }
    const int first = cu[lo], end = cu[lo + 1];
    const bool whole = first >= 0 && end <= rows && first <= r && r < end && end - first <= Tq && below <= first &&
                       above >= end;
    return PackedRow{lo, r - first, whole ? end - first : 0};
}

// A row of V elements in memory's chunks of N, chunk k the row's elements k*N - skew and on, `skew` the
// row's distance from a chunk's boundary.  The first and the last chunk may hold elements of the rows beside
// it, and the last one may reach past the tensor; then it is not loaded whole (open_end false).
template <int N>
struct RowChunks {
    int skew, V;
    bool open_end;
    INFLLMV2_HD int chunks() const { return (skew + V + N - 1) / N; }
    INFLLMV2_HD int whole() const { return (skew + V) / N; }  // chunks [skew != 0, whole) are uncut
    INFLLMV2_HD int end() const { return open_end ? chunks() : whole(); }  // chunks [0, end) lie in the tensor
    INFLLMV2_HD bool cut(int k) const { return k >= whole() || (k == 0 && skew != 0); }
};
// Row `row` of a tensor of `rows` rows that starts on a chunk's boundary.
template <int N>
INFLLMV2_HD RowChunks<N> row_chunks(unsigned long long row, unsigned long long rows, int V) {
    const unsigned long long first = row * V;
    RowChunks<N> c{static_cast<int>(first % N), V, true};
    c.open_end = first - c.skew + static_cast<unsigned long long>(c.chunks()) * N <= rows * V;
    return c;
}

}  // namespace infllmv2
