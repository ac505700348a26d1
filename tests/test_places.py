"""The kernels' index arithmetic (csrc/places.h), built by the host compiler and checked for every small
size, without a GPU."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <algorithm>
#include <cstddef>
#include <vector>
#include "places.h"
using namespace infllmv2;

// Every array of B + 1 offsets in [lo, hi], every number of rows and every longest length: the number of
// cases in which a sequence is taken in part, a row is taken that the offsets give to no or another place, a
// good sequence is skipped, or something is skipped though the offsets are in order.
extern "C" long long packed(int B, int lo, int hi, int most_rows) {
    long long wrong = 0;
    std::vector<int> cu(B + 1, lo);
    for (;;) {
        for (int rows = 1; rows <= most_rows; ++rows)
            for (int Tq = 1; Tq <= 3; ++Tq) {
                std::vector<int> taken(B, 0);
                for (int r = 0; r < rows; ++r) {
                    const PackedRow p = packed_row(cu.data(), B, r, rows, Tq);
                    if (p.len == 0) continue;
                    wrong += p.b < 0 || p.b >= B || cu[p.b] + p.t != r || p.t < 0 || p.t >= p.len ||
                             p.len != cu[p.b + 1] - cu[p.b] || p.len > Tq;
                    ++taken[p.b];
                }
                bool order = cu[0] == 0 && cu[B] <= rows;
                for (int b = 0; b < B; ++b) order = order && cu[b + 1] >= cu[b] && cu[b + 1] - cu[b] <= Tq;
                for (int b = 0; b < B; ++b) {
                    const int len = cu[b + 1] - cu[b];
                    wrong += taken[b] != 0 && taken[b] != len;  // (a row is taken once, so those taken share none)
                    if (order) wrong += taken[b] != len;
                    // no other offset crosses it: it has to be taken
                    const bool apart = *std::max_element(cu.begin(), cu.begin() + b + 1) <= cu[b] &&
                                       *std::min_element(cu.begin() + b + 1, cu.end()) >= cu[b + 1];
                    if (apart && len > 0 && len <= Tq && cu[b] >= 0 && cu[b + 1] <= rows) wrong += taken[b] != len;
                }
            }
        int i = 0;
        while (i <= B && cu[i] == hi) cu[i++] = lo;
        if (i > B) return wrong;
        ++cu[i];
    }
}

// Every row of a tensor of `rows` rows of V elements, in chunks of N: the number of loads that reach outside
// the tensor, of elements of the row that no load takes or two take, and of chunks wrongly called uncut.
template <int N>
static long long chunks_wrong(int rows, int V) {
    long long wrong = 0;
    for (int row = 0; row < rows; ++row) {
        const RowChunks<N> c = row_chunks<N>(row, rows, V);
        std::vector<int> taken(V, 0);
        wrong += c.chunks() - c.end() > 1 || c.end() > c.chunks();
        for (int k = 0; k < c.chunks(); ++k)
            for (int e = 0; e < N; ++e) {
                const long long x = static_cast<long long>(k) * N - c.skew + e, at = static_cast<long long>(row) * V + x;
                if (e == 0) wrong += at % N != 0;
                if (k < c.end()) wrong += at < 0 || at >= static_cast<long long>(rows) * V;
                if (x >= 0 && x < V) ++taken[x];
                else wrong += !c.cut(k);
            }
        for (int x = 0; x < V; ++x) wrong += taken[x] != 1;
    }
    return wrong;
}
extern "C" long long chunks(int n, int rows, int V) { return n == 4 ? chunks_wrong<4>(rows, V) : chunks_wrong<8>(rows, V); }

extern "C" int packed_len(const int* cu, int B, int r, int rows, int Tq) { return packed_row(cu, B, r, rows, Tq).len; }
"""


@pytest.fixture(scope="module")
def places(tmp_path_factory):
    path = tmp_path_factory.mktemp("places")
    src, so = path / "places.cpp", path / "places.so"
    src.write_text(PROGRAM)
    inc = os.path.join(ROOT, "block_sparse_long_infllm_gb300", "csrc")
    subprocess.run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I", inc,
                    str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    lib.packed.restype = lib.chunks.restype = ctypes.c_longlong
    return lib


@pytest.mark.parametrize("B,lo,hi,rows", [(1, -2, 6, 6), (2, -2, 6, 6), (3, -1, 5, 5), (4, 0, 5, 5), (5, 0, 4, 4)])
def test_packed_sequences_are_taken_whole_or_not_at_all(places, B, lo, hi, rows):
    assert places.packed(B, lo, hi, rows) == 0


def test_packed_offsets_at_the_ends_of_int32(places):
    big, small = 2 ** 31 - 1, -2 ** 31
    for cu in ([0, small], [small, big], [small, 5], [0, big], [big, small], [small, small, 5], [0, big, 5]):
        for r in range(4):
            assert places.packed_len((ctypes.c_int * len(cu))(*cu), len(cu) - 1, r, 4, 4) == 0


@pytest.mark.parametrize("n", [4, 8])
def test_chunks_of_rows_lie_in_the_tensor(places, n):
    """16-byte chunks of fp32 and bf16 rows: rows of few elements, where more than the last one's chunks
    reach past the tensor, and longer ones."""
    for V in list(range(1, 40)) + [77, 100, 257, 1001]:
        for rows in range(1, 24):
            assert places.chunks(n, rows, V) == 0, (V, rows)
