// pool.cuh -- exact mean of c bf16 rows rounded once to bf16 (semantic-kernel pooling, "MiniCPM4:
// 如何在手机电脑上高效运行大语言模型", section 1.1), in integer arithmetic: per column the lanes
// agree on the largest bf16 exponent, every value becomes an integer multiple of 2^-40 of that
// magnitude (exact for every value within 2^40 of the largest -- the condition under which an
// fp64 sum of bf16 values is exact as well), the integers are added, and the quotient by c, with
// its remainder as a sticky bit, is rounded once, nearest with ties to even.  (This GPU's fp64
// rate is a few operations per clock per SM, so no fp64 is used.)  Exponent 255 is no number of that
// scale: a column with infinities of one sign has that mean, one with both or with a NaN is NaN.
#pragma once

#include "common.cuh"

namespace infllmv2 {

constexpr int kMeanLanes = 16;                    // lanes per (kernel, 8-element slice)
constexpr int kMeanRows = 128 / kMeanLanes;       // rows per lane: kernel_size <= block_size <= 128

// bf16 bits of (A / c) * 2^E0 (negated when neg), rounded once, nearest with ties to even; A < 2^62.
__device__ __forceinline__ uint32_t bf16_of_ratio(unsigned long long A, int c, int E0, bool neg) {
    if (A == 0ull) return 0u;  // +0, as an fp64 sum that starts from +0 gives
    const uint32_t sign = neg ? 0x8000u : 0u;
    const int t = __clzll(static_cast<long long>(A)) - 2;   // N = A << t in [2^61, 2^62)
    const unsigned long long N = A << t;
    unsigned long long Q;
    bool sticky;
    if ((c & (c - 1)) == 0) {  // a power of two (the pages' 32): a shift
        const int lc = __ffs(c) - 1;
        Q = N >> lc;
        sticky = (N & static_cast<unsigned long long>(c - 1)) != 0ull;
    } else {
        Q = N / static_cast<unsigned long long>(c);
        sticky = N - Q * static_cast<unsigned long long>(c) != 0ull;
    }
    const int nb = 64 - __clzll(static_cast<long long>(Q));  // >= 55: Q >= 2^61 / 128
    int X = nb - 1 + E0 - t;                                // exponent of the leading bit
    const int sh = X >= -126 ? nb - 8 : nb - 8 + (-126 - X); // bits below the kept ones (subnormal: fewer kept)
    if (sh >= 63) return sign;                              // below half the smallest subnormal
    unsigned long long top = Q >> sh;
    const unsigned long long rem = Q & ((1ull << sh) - 1ull), half = 1ull << (sh - 1);
    if (rem > half || (rem == half && (sticky || (top & 1ull)))) ++top;
    if (X < -126) return sign | static_cast<uint32_t>(top);  // subnormal (128: the smallest normal)
    if (top == 256ull) {
        top = 128ull;
        ++X;
    }
    const int ef = X + 127;
    if (ef >= 255) return sign | 0x7F80u;
    return sign | (static_cast<uint32_t>(ef) << 7) | static_cast<uint32_t>(top & 127ull);
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t max_s16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.s16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// bf16 bits of the mean of column ln % 8 of a slice where it holds an infinity or a NaN, else 0.  Without
// their sign the largest bits are a NaN's or an infinity's; where they are an infinity's, +inf is the
// largest signed and -inf the largest unsigned pattern.
template <int kRows>
__device__ __forceinline__ uint32_t special_mean(const uint32_t (&w)[kRows][4], int ln) {
    uint32_t out = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t mag = 0u, pos = 0x80008000u, neg = 0u;
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            mag = max_u16x2(mag, w[u][i] & 0x7FFF7FFFu);
            pos = max_s16x2(pos, w[u][i]);
            neg = max_u16x2(neg, w[u][i]);
        }
#pragma unroll
        for (int off = 1; off < kMeanLanes; off <<= 1) {
            mag = max_u16x2(mag, __shfl_xor_sync(0xffffffffu, mag, off));
            pos = max_s16x2(pos, __shfl_xor_sync(0xffffffffu, pos, off));
            neg = max_u16x2(neg, __shfl_xor_sync(0xffffffffu, neg, off));
        }
        const int sh = 16 * (ln & 1);
        const uint32_t m = (mag >> sh) & 0xFFFFu, p = (pos >> sh) & 0xFFFFu, n = (neg >> sh) & 0xFFFFu;
        if (i == (ln & 7) >> 1 && m >= 0x7F80u)
            out = m > 0x7F80u || (p == 0x7F80u && n == 0xFF80u) ? 0x7FFFu : p == 0x7F80u ? p : n;
    }
    return out;
}

// Exact mean of the c rows of one 8-element slice; lane ln (of the 16 aligned lanes sharing the
// slice) takes rows ln, ln + 16, ... (at most kRows of them) from row(i).  Every lane of the group
// returns the 8 bf16 results, packed.
template <int kRows = kMeanRows, typename RowOf>
__device__ __forceinline__ uint4 exact_mean_rows(int c, int ln, RowOf row) {
    uint32_t w[kRows][4];
    const int n_u = (c + kMeanLanes - 1) / kMeanLanes;  // row rounds any lane of the group has
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        const int i = ln + kMeanLanes * u;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (u < n_u && i < c) x = row(i);
        w[u][0] = x.x;
        w[u][1] = x.y;
        w[u][2] = x.z;
        w[u][3] = x.w;
    }
    // largest biased exponent per column (1 for zeros and subnormals), two columns to a word in place
    uint32_t xm2[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) xm2[i] = 0x00800080u;
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        if (u >= n_u) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) xm2[i] = max_u16x2(xm2[i], w[u][i] & 0x7F807F80u);
    }
#pragma unroll
    for (int off = 1; off < kMeanLanes; off <<= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) xm2[i] = max_u16x2(xm2[i], __shfl_xor_sync(0xffffffffu, xm2[i], off));
    const uint32_t top = max_u16x2(max_u16x2(xm2[0], xm2[1]), max_u16x2(xm2[2], xm2[3]));
    uint32_t special = 0u;
    if (__any_sync(0xffffffffu, (top >> 16) == 0x7F80u || (top & 0xFFFFu) == 0x7F80u)) special = special_mean<kRows>(w, ln);
    int emax[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) emax[e] = static_cast<int>((xm2[e >> 1] >> (16 * (e & 1) + 7)) & 0xFFu);
    long long S[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) S[e] = 0;
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        if (u >= n_u) break;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t h = (w[u][e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
            const int ef = static_cast<int>((h >> 7) & 0xFFu);
            const uint32_t mant = (h & 127u) | (ef != 0 ? 128u : 0u);
            const int sh = max(ef, 1) - (emax[e] - 40);  // value = mant * 2^(max(ef,1) - 134); sh <= 40
            // +-(mant << sh), bits below 1 dropped, added by one multiply-add: the mantissa is shifted right
            // (from 10 places up) or multiplied by a power of two up to 2^30
            const int mag = static_cast<int>((mant << 10) >> min(max(10 - sh, 0), 31));
            S[e] += static_cast<long long>((h & 0x8000u) ? -mag : mag) * (1 << max(sh - 10, 0));
        }
    }
    // Sums over the lanes, halving the columns as they go: a lane keeps those that agree with its number in
    // one bit after another and hands the rest to its neighbour, so lane ln ends with column ln % 8 (16
    // shuffles of a word instead of 64), which it rounds; the 8 results are then gathered.
    long long S4[4], S2[2], Sm;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const long long keep = (ln & 1) ? S[2 * i + 1] : S[2 * i], give = (ln & 1) ? S[2 * i] : S[2 * i + 1];
        S4[i] = keep + __shfl_xor_sync(0xffffffffu, give, 1);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const long long keep = (ln & 2) ? S4[2 * i + 1] : S4[2 * i], give = (ln & 2) ? S4[2 * i] : S4[2 * i + 1];
        S2[i] = keep + __shfl_xor_sync(0xffffffffu, give, 2);
    }
    Sm = ((ln & 4) ? S2[1] : S2[0]) + __shfl_xor_sync(0xffffffffu, (ln & 4) ? S2[0] : S2[1], 4);
    Sm += __shfl_xor_sync(0xffffffffu, Sm, 8);
    const uint32_t xw = (ln & 4) ? ((ln & 2) ? xm2[3] : xm2[2]) : ((ln & 2) ? xm2[1] : xm2[0]);
    const int xm = static_cast<int>((xw >> (16 * (ln & 1) + 7)) & 0xFFu);
    uint32_t bits = bf16_of_ratio(static_cast<unsigned long long>(Sm < 0 ? -Sm : Sm), c, xm - 40 - 134, Sm < 0);
    if (special != 0u) bits = special;
    const int g0 = (threadIdx.x & 31) & ~(kMeanLanes - 1);  // first lane of this group in the warp
    uint32_t out[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        out[e] = __shfl_sync(0xffffffffu, bits, g0 + 2 * e) | (__shfl_sync(0xffffffffu, bits, g0 + 2 * e + 1) << 16);
    return make_uint4(out[0], out[1], out[2], out[3]);
}

// The same with the rows in memory, row_stride apart, but row `sub_row` taken from `sub_val`.
__device__ __forceinline__ uint4 exact_mean_slice(const uint4* src, size_t row_stride, int c, int ln, int sub_row,
                                                  uint4 sub_val) {
    return exact_mean_rows(c, ln, [&](int i) {
        return i == sub_row ? sub_val : ldg_v4(src + static_cast<size_t>(i) * row_stride);
    });
}

}  // namespace infllmv2
