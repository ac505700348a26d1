// verify.cu -- verification of a draft tree against the target's probabilities ("MiniCPM4: 如何在手机电
// 脑上高效运行大语言模型", section 1.1, tree-speculative decoding), from given random numbers.
//
// At node c with target row p and draft row q its children are tried in turn (recursive rejection
// sampling).  After some of them were rejected the target's remaining weight of token x is
//   w(x) = max(p(x) - c q(x), 0):  one rejection takes w/Z to max(w/Z - q/R, 0), which is
//   max(p - (c + Z/R) q, 0) / Z,   Z = sum of w (1 at first),  R = 1 (drafts drawn with replacement)
//   or 1 - the rejected drafts' q (without),
// so c, Z and R are all that a node has to remember, and child x stands iff u Z q(x) < w(x) R.  With
// no draft probabilities (drafts chosen, not drawn) q is 1 at the child alone: it stands iff
// u Z < w(x), and a rejected token leaves w.  The last token is the first whose running sum of w
// passes u_0 times the whole.
//
// Sums over the vocabulary are 64-bit integers in units of 2^-62: fp32 (and bf16) probabilities
// become integers by a shift, differences and sums of integers are exact and independent of their
// order, so every cluster size samples the same token (fp32 sums would move the border between two
// tokens by more than a rare token's probability, and this GPU's fp64 rate is a few operations per
// clock and SM).  After one rejection c is 1 and w exact; from the second on c is a sum of quotients, each
// rounded up by less than 2^-58 of itself, and c q is cut to whole units: where the rejections leave the
// target nothing (one token with all of w, and with all that is left of the drafts), nothing is left here
// too, since c' q = (c + Z/R) q is at least what c q was cut to and Z = w, together p.
//
// What bounds it is memory: the last node's target row (and draft row, once a child was rejected).
// One thread-block cluster per sequence; a row is cut into one contiguous piece per warp.  In each
// sweep the warps send their pieces' sums to every CTA (asynchronous stores counted on the receiver's
// barrier: a cluster barrier that also orders plain stores took about 0.9 us instead of 0.25), warp 0
// of every CTA takes the same decisions from them, and at the end the warp whose piece holds the
// sampled token finds it from the running sums that its lanes left in shared memory.  Decisions are
// integer too: 128-bit products compare u Z q with w R exactly, and warp 0 finds how far the drafts that
// stand at their first trial lead by comparing masks.
//
// Measured on a GB300 (programmatic launches back to back): one tree of 16 drafts over 32001 tokens,
// two to three sweeps, 10.7 us, and 6.7 us where one sweep does; 64 chains of 8 over 131072 tokens 21.7
// us, of which about 12 move the 67 MB (10.0 us at the copy rate), 3.5 pass before the last node is known
// (tokens, then their probabilities: two loads that miss every cache) and 2.5 after the sums.  CTAs per SM:
// 4 (64 registers) 21.5, 3 27.6, 2 25.6; cluster sizes are with launch() below.  For one tree 16 instead of
// 8 CTAs: 11.7 instead of 12.6.  Rows kept in registers from sweep to sweep spilled and were slower (15.6).
#include "internal.h"
#include "places.h"
#include "tma.cuh"

namespace infllmv2 {

namespace {

using u64 = unsigned long long;

constexpr int kVerifyThreads = 256;
constexpr int kWarpsLog = 3, kVerifyWarps = 1 << kWarpsLog;
static_assert(kVerifyWarps * 32 == kVerifyThreads, "");
constexpr int kResident = 4;  // CTAs per SM
constexpr int kMaxCluster = 16;
constexpr int kMaxPieces = kMaxCluster * kVerifyWarps;  // pieces of a row: one per warp of the cluster
constexpr int kLanePieces = kMaxPieces / 32;
constexpr int kBatch = 4;     // chunks of each row that a lane loads together
constexpr int kSegments = 16; // running sums of a piece that its lanes leave for the search
constexpr u64 kOne = 1ull << 62;  // probability 1 in the units of the sums
constexpr float kMostSum = 2.f;   // a row whose sum is above this holds no probabilities

// ---- 64-bit numbers

// Shift right by any amount (PTX clamps it: 64 and more leave 0).
__device__ __forceinline__ u64 shr(u64 x, int n) {
    u64 y;
    asm("shr.u64 %0, %1, %2;" : "=l"(y) : "l"(x), "r"(n));
    return y;
}

// max(a - b, 0).
__device__ __forceinline__ u64 less(u64 a, u64 b) { return a > b ? a - b : 0ull; }

// A probability as read: NaN and negative values are 0, values past 1 are 1.
__device__ __forceinline__ float prob(float x) { return __saturatef(x); }

// acc + p in units of 2^-62, p in [0, 1], bits below that dropped: the mantissa (leading bit at 31)
// times 2^(exponent - 96), or shifted right where that is negative -- one 64-bit multiply-add.
__device__ __forceinline__ u64 add_fixed(u64 acc, float p) {
    const uint32_t b = __float_as_uint(p), m = (b << 8) | 0x80000000u;
    const int e = static_cast<int>(b >> 23) - 96;
    return acc + static_cast<u64>(__funnelshift_rc(m, 0u, max(-e, 0))) * (1u << max(e, 0));
}

// A positive number m 2^(e - 63), the leading bit of m set.
struct Num {
    u64 m;
    int e;
};
// x in units of 2^-62 (x != 0).
__device__ __forceinline__ Num num(u64 x) {
    const int z = __clzll(static_cast<long long>(x));
    return Num{x << z, 1 - z};
}
// a + b, rounded up.
__device__ __forceinline__ Num add(Num a, Num b) {
    if (a.e < b.e) {
        const Num t = a;
        a = b;
        b = t;
    }
    const int d = a.e - b.e;
    const u64 s = shr(b.m, d);
    Num r{a.m + s + (d < 64 && (s << d) == b.m ? 0ull : 1ull), a.e};
    if (r.m < a.m) {
        r.m = (r.m >> 1) + (r.m & 1ull) + (1ull << 63);
        ++r.e;
    }
    return r;
}
// a / b, rounded up by less than 2^-58 of it: two Newton steps from an fp32 reciprocal, y -> y + y (1 - b y),
// y 2^-62 the reciprocal of b's mantissa in [1, 2): 2^-23, 2^-46, then less than 2^-59 below the quotient (a
// unit of y, at least 2^61, and one of q, at least 2^60), which the 32 of at most 2^64 make up for.
__device__ __forceinline__ Num divide(Num a, Num b) {
    u64 y = static_cast<u64>(__fdiv_rn(0x1p62f, __ull2float_rn(b.m) * 0x1p-63f));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const long long err = static_cast<long long>((1ull << 61) - __umul64hi(b.m, y));  // (1 - b y) 2^61, below 2^40
        y += static_cast<u64>(__mul64hi(static_cast<long long>(y), err * 8));
    }
    const u64 q = __umul64hi(a.m, y);  // quotient of the mantissas in (1/2, 2), times 2^61
    const int z = __clzll(static_cast<long long>(q));
    Num r{(q << z) + 32ull, a.e - b.e + 2 - z};
    if (r.m < 32ull) {
        r.m = (1ull << 63) + 16ull;
        ++r.e;
    }
    return r;
}

// c, the factor of the draft's row in w.
struct Coef {
    Num v;
    int kind;  // 0: c = 0, 1: c = 1, 2: any other
};

// c q in units of 2^-62; all ones where it is 2 or more (past any p).
__device__ __forceinline__ u64 scaled(float q, const Num& c) {
    const uint32_t b = __float_as_uint(q);
    const int e = c.e + static_cast<int>(b >> 23) - 127;
    // both mantissas have their leading bit at 63: the product's high word is c q 2^(62 - e)
    const u64 h = __umul64hi(c.m, static_cast<u64>((b << 8) | 0x80000000u) << 32);
    return b == 0u ? 0ull : e > 0 ? ~0ull : shr(h, -e);
}

// w = max(p - c q, 0) in units of 2^-62.
__device__ __forceinline__ u64 weight(float p, float q, const Coef& c) {
    const u64 P = add_fixed(0ull, p);
    const u64 Q = c.kind == 0 ? 0ull : c.kind == 1 ? add_fixed(0ull, q) : scaled(q, c.v);
    return less(P, Q);
}

// u Z q < w R, exactly: u, q in [0, 1]; Z, w, R in units of 2^-62.  The 128-bit products are compared
// after the left one is cut to whole units of the right one (x < n iff floor(x) < n).
__device__ __forceinline__ bool stands(float u, u64 Z, float q, u64 w, u64 R) {
    const uint32_t ub = __float_as_uint(u), qb = __float_as_uint(q);
    const u64 uq = static_cast<u64>((ub << 8) | 0x80000000u) * ((qb << 8) | 0x80000000u);
    const int s = 254 - static_cast<int>(ub >> 23) - static_cast<int>(qb >> 23);  // u q = uq 2^(-62 - s)
    u64 lo = uq * Z, hi = __umul64hi(uq, Z);
    if (s >= 64) {
        lo = shr(hi, s - 64);
        hi = 0ull;
    } else if (s > 0) {
        lo = (lo >> s) | (hi << (64 - s));
        hi >>= s;
    }
    const u64 rh = __umul64hi(w, R), rl = w * R;
    return hi < rh || (hi == rh && lo < rl);
}

// ---- rows

// A row in 16-byte chunks of memory.
template <typename T>
struct RowView : RowChunks<16 / sizeof(T)> {
    static constexpr int N = 16 / sizeof(T);
    const T* p;
    using RowChunks<N>::skew;
    using RowChunks<N>::V;
    using RowChunks<N>::whole;
    __device__ __forceinline__ RowView(const T* row, const RowChunks<N>& c) : RowChunks<N>(c), p(row) {}
    // Chunk k if `want`, else 0.  One predicated load, so that several in a row are in flight together
    // (a branch around each load would make them wait for one another).
    __device__ __forceinline__ uint4 load(int k, bool want) const {
        uint4 r = make_uint4(0u, 0u, 0u, 0u);
        asm("{\n"
            " .reg .pred p;\n"
            " setp.ne.s32 p, %5, 0;\n"
            " @p ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n"
            "}\n"
            : "+r"(r.x), "+r"(r.y), "+r"(r.z), "+r"(r.w)
            : "l"(p - skew + static_cast<long long>(k) * N), "r"(want ? 1 : 0));
        return r;
    }
    // What a cut chunk holds of other rows becomes 0.
    __device__ __forceinline__ void trim(uint4& x, int k) const {
        const int a = k * N - skew;
        if constexpr (sizeof(T) == 4) {
            x.x = a >= 0 && a < V ? x.x : 0u;
            x.y = a + 1 >= 0 && a + 1 < V ? x.y : 0u;
            x.z = a + 2 >= 0 && a + 2 < V ? x.z : 0u;
            x.w = a + 3 >= 0 && a + 3 < V ? x.w : 0u;
        } else {
            const auto pair = [&](uint32_t w, int i) {
                return (i >= 0 && i < V ? w & 0xFFFFu : 0u) | (i + 1 >= 0 && i + 1 < V ? w & 0xFFFF0000u : 0u);
            };
            x.x = pair(x.x, a);
            x.y = pair(x.y, a + 2);
            x.z = pair(x.z, a + 4);
            x.w = pair(x.w, a + 6);
        }
    }
    // The cut chunk that reaches past the tensor, element by element.
    __device__ __noinline__ uint4 tail() const {
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        const int a = whole() * N - skew;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            if (a + e < 0 || a + e >= V) continue;
            if constexpr (sizeof(T) == 4)
                w[e] = __float_as_uint(p[a + e]);
            else
                w[e >> 1] |= static_cast<uint32_t>(__bfloat16_as_ushort(p[a + e])) << (16 * (e & 1));
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Element e of a chunk as a probability.
template <typename T>
__device__ __forceinline__ float element(const uint4& x, int e) {
    if constexpr (sizeof(T) == 4) {
        return prob(__uint_as_float(e == 0 ? x.x : e == 1 ? x.y : e == 2 ? x.z : x.w));
    } else {
        const uint32_t w = (e >> 1) == 0 ? x.x : (e >> 1) == 1 ? x.y : (e >> 1) == 2 ? x.z : x.w;
        return prob((e & 1) ? bf16_hi(w) : bf16_lo(w));
    }
}

__device__ __forceinline__ float load1(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// A lane's sums over its chunks: of p, and of what w loses against it.
struct Sums {
    u64 p = 0ull, q = 0ull;
    uint32_t top = 0u;  // bit 31: the sum of p reached 2 (before it could wrap)

    // w = max(p - c q, 0) = p - min(p, c q)
    template <typename T, int KIND>
    __device__ __forceinline__ void take(const uint4& P, const uint4& Q, const Num& c) {
#pragma unroll
        for (int e = 0; e < 16 / static_cast<int>(sizeof(T)); ++e) {
            const float x = element<T>(P, e);
            if constexpr (KIND == 2) {
                const u64 px = add_fixed(0ull, x), y = scaled(element<T>(Q, e), c);
                p += px;
                q += px < y ? px : y;
            } else {
                p = add_fixed(p, x);
                if constexpr (KIND == 1) q = add_fixed(q, fminf(x, element<T>(Q, e)));
            }
            if (e & 1) top |= static_cast<uint32_t>(p >> 32);
        }
    }
    __device__ __forceinline__ float about() const {  // the sum of p
        return (top >> 31) != 0u ? 4.f : __uint2float_rn(static_cast<uint32_t>(p >> 32)) * 0x1p-30f;
    }
};

struct Part {  // one piece's sums
    u64 w;
    float p;
    float pad;
};

struct Shared {
    alignas(16) Part part[2][kMaxPieces];
    alignas(8) uint64_t bar[2];  // bytes of part[.] that came from the cluster's warps
    int tok[64];
    u64 mask[64];
    float u[64];
    float p[64], q[64];  // of each node's token in its parent's rows
    u64 kids[64];
    u64 stands;          // nodes that stand if they are tried first
    u64 cum[kSegments][kVerifyThreads];  // each lane's sum of w up to the end of a segment of its piece
    // what warp 0 tells the others: the next sweep, then where the last token is
    Coef c;
    u64 gone;            // children of `node` whose tokens weigh nothing (drafts without probabilities)
    u64 on;              // the path
    u64 rem;             // what is left of the target in piece `own`
    int node, own, state;
};
enum : int { kSweep = 0, kDraw = 1, kBad = 2, kLost = 3 };  // kLost: a wait ran out

__device__ __forceinline__ u64 warp_sum(u64 x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}
__device__ __forceinline__ u64 warp_scan(u64 x) {  // inclusive
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    return x;
}

__device__ __forceinline__ uint32_t peer_addr(uint32_t local, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}
// 16 bytes into a peer's shared memory, counted on the peer's barrier.
__device__ __forceinline__ void send16(uint32_t dst, u64 a, u64 b, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b64 [%0], {%1, %2}, [%3];" ::"r"(dst), "l"(a),
                 "l"(b), "r"(bar)
                 : "memory");
}
// Whether a phase completed within the limit, the same for every lane: a warp that shuffles behind the wait
// must not part over it.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity)) != 0;
}
// A CTA whose wait ran out in `round`: its peers may still send to it.  Each of them ends (their waits are
// bounded too, and this CTA sends no more), and it stays until all have, then until what they sent is here.
__device__ __noinline__ void outstay(uint64_t* bars, int round) {
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
    if (threadIdx.x < 32)
        for (int r = round; r < round + 2; ++r) (void)warp_wait(&bars[r & 1], (r >> 1) & 1);
}
__device__ __forceinline__ int lowest(u64 x) { return __ffsll(static_cast<long long>(x)) - 1; }

// One row's weights, as a search reads them.
template <typename T>
struct Weights {
    static constexpr int N = RowView<T>::N;
    RowView<T> P, Q;
    Coef c;
    u64 out;         // children whose tokens weigh nothing (drafts without probabilities)
    const int* tok;

    __device__ __forceinline__ void chunk(int k, int k1, u64 (&w)[N]) const {
#pragma unroll
        for (int e = 0; e < N; ++e) w[e] = 0ull;
        const bool in = k < min(k1, P.end());
        uint4 x = P.load(k, in), y = Q.load(k, in && c.kind != 0);
        if (k < k1 && !in) {
            x = P.tail();
            if (c.kind != 0) y = Q.tail();
        } else if (P.cut(k)) {
            P.trim(x, k);
            Q.trim(y, k);
        }
#pragma unroll
        for (int e = 0; e < N; ++e) w[e] = weight(element<T>(x, e), element<T>(y, e), c);
        for (u64 g = out; g != 0ull; g &= g - 1) {
            const int at = tok[lowest(g)] - (k * N - P.skew);
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (e == at) w[e] = 0ull;
        }
    }

    // The first element of chunks [k0, k1) whose running sum passes `target` (below their sum), by one
    // warp; every lane returns it.
    __device__ __noinline__ int search(int k0, int k1, u64 target) const {
        const int lane = threadIdx.x & 31;
        u64 base = 0ull;
        for (int kb = k0; kb < k1; kb += 32) {
            u64 w[N], sum = 0ull;
            chunk(kb + lane, k1, w);
#pragma unroll
            for (int e = 0; e < N; ++e) sum += w[e];
            const u64 incl = base + warp_scan(sum);
            const uint32_t hit = __ballot_sync(0xffffffffu, incl > target);
            if (hit != 0u) {
                int found = -1;
                u64 run = incl - sum;
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    run += w[e];
                    if (found < 0 && run > target) found = (kb + lane) * N - P.skew + e;
                }
                return __shfl_sync(0xffffffffu, found, __ffs(hit) - 1);
            }
            base = __shfl_sync(0xffffffffu, incl, 31);
        }
        return -1;
    }
};

// A warp's sums over its piece, chunks [k0, k1) in `its` rounds of 32; each lane leaves its running sum
// behind every `seg` rounds.
template <typename T, int KIND>
__device__ __forceinline__ Sums sweep(const RowView<T>& P, const RowView<T>& Q, const Num& c, int k0, int k1, int its,
                                      int seg, u64 (*cum)[kVerifyThreads]) {
    const int lane = threadIdx.x & 31, hi = min(P.end(), k1);
    Sums s;
    u64* out = &cum[0][threadIdx.x];
    int left = seg;  // rounds of the segment
    for (int it = 0; it < its; it += kBatch) {
        uint4 x[kBatch], y[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int k = k0 + 32 * (it + i) + lane;
            x[i] = P.load(k, k < hi);
            if (KIND != 0) y[i] = Q.load(k, k < hi);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (it + i >= its) break;
            const int k = k0 + 32 * (it + i) + lane;
            if (P.cut(k)) {
                P.trim(x[i], k);
                if (KIND != 0) Q.trim(y[i], k);
            }
            s.template take<T, KIND>(x[i], KIND != 0 ? y[i] : x[i], c);
            if (--left == 0 || it + i + 1 == its) {
                *out = s.p - s.q;
                out += kVerifyThreads;
                left = seg;
            }
        }
    }
    const int last = P.chunks() - 1;
    if (last >= P.end() && last >= k0 && last < k1 && (last - k0) % 32 == lane) {  // the end of the tensor
        const u64 before = s.p - s.q;
        const uint4 x = P.tail();
        s.template take<T, KIND>(x, KIND != 0 ? Q.tail() : x, c);
        for (int i = (last - k0) / 32 / seg; i <= (its - 1) / seg; ++i) cum[i][threadIdx.x] += s.p - s.q - before;
    }
    return s;
}

template <typename T>
__global__ void __launch_bounds__(kVerifyThreads, kResident) verify_kernel(VerifyArgs a, int cl_log) {
    constexpr int N = RowView<T>::N;
    __shared__ Shared sh;
    const int CL = 1 << cl_log, rank = blockIdx.x & (CL - 1), b = blockIdx.x >> cl_log;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int pieces = CL * kVerifyWarps, piece = rank * kVerifyWarps + warp;
    const size_t at = static_cast<size_t>(b) * a.n;
    const T* target = static_cast<const T*>(a.target) + at * a.V;
    const T* draft = a.draft != nullptr ? static_cast<const T*>(a.draft) + at * a.V : nullptr;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.bar[i], 1);
            mbar_arrive_expect_tx(&sh.bar[i], pieces * sizeof(Part));
        }
        fence_mbar_init();
        sh.stands = 0ull;
    }
    if (tid < 64) sh.kids[tid] = 0ull;
    pdl_wait();
    pdl_trigger();
    const int n = a.n_nodes != nullptr ? a.n_nodes[b] : a.n;
    bool bad = n < 0 || n > a.n;
    if (tid < a.n) {
        sh.tok[tid] = a.tokens[at + tid];
        sh.u[tid] = __saturatef(a.u[at + tid]);
        const u64 own = 1ull << tid;
        sh.mask[tid] = a.tree_mask != nullptr ? a.tree_mask[at + tid] : own | (own - 1);
    }
    __syncthreads();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // this CTA's barriers are there
    if (!bad && tid < n) {
        const u64 own = 1ull << tid, up = sh.mask[tid] ^ own;
        if (tid == 0) {
            bad = up != 0ull;
        } else {
            const int parent = 63 - __clzll(static_cast<long long>(up));
            const int x = sh.tok[tid];
            bad = up == 0ull || up >= own || sh.mask[max(parent, 0)] != up || x < 0 || x >= a.V;
            if (!bad) {
                atomicOr(&sh.kids[parent], own);
                const size_t i = static_cast<size_t>(parent) * a.V + x;
                const float p = prob(load1(target + i)), q = draft != nullptr ? prob(load1(draft + i)) : 1.f;
                sh.p[tid] = p;
                sh.q[tid] = q;
                if (stands(sh.u[tid], kOne, q, add_fixed(0ull, p), kOne)) atomicOr(&sh.stands, own);
            }
        }
    }
    bad = __syncthreads_or(bad) != 0;
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    const bool idle = n <= 0 || bad;
    int drawn = -1;
    if (!idle) {
        // the walk (warp 0)
        u64 on = 1ull, rest = 0ull, gone = 0ull, Z = kOne, easy = 0ull;
        u64 R = kOne;  // what is left of the drafts' weight; 0 stays 0, however many siblings follow
        Coef c{{0ull, 0}, 0};
        int cur = 0;
        bool fresh = true, z_known = true;  // no child of cur was tried yet; Z belongs to c
        if (warp == 0) {
            // nodes that are tried first and stand: a way of nothing but these needs no arithmetic
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = 32 * h + lane;
                bool yes = i > 0 && i < n && ((sh.stands >> i) & 1ull) != 0ull;
                if (yes) yes = lowest(sh.kids[63 - __clzll(static_cast<long long>(sh.mask[i] ^ (1ull << i)))]) == i;
                easy |= static_cast<u64>(__ballot_sync(0xffffffffu, yes)) << (32 * h);
            }
        }
        for (int round = 0;; ++round) {
            if (warp == 0) {
                while (z_known) {
                    if (fresh) {
                        // the last node below cur that the easy ones lead to; its first child, if it has one, falls
                        u64 reach = 0ull;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int i = 32 * h + lane;
                            const bool yes = i < n && (sh.mask[i] & on) == on && (sh.mask[i] & ~on & ~easy) == 0ull;
                            reach |= static_cast<u64>(__ballot_sync(0xffffffffu, yes)) << (32 * h);
                        }
                        cur = 63 - __clzll(static_cast<long long>(reach));
                        on = sh.mask[cur];
                        rest = sh.kids[cur];
                        if (rest == 0ull) break;
                        const int i = lowest(rest);
                        rest &= rest - 1;
                        fresh = false;
                        if (draft == nullptr) {
                            const u64 w = add_fixed(0ull, sh.p[i]);
                            gone = 1ull << i;
                            Z = less(Z, w);
                        } else {
                            c = Coef{{1ull << 63, 0}, 1};
                            z_known = false;
                            if (!a.replace) R = less(R, add_fixed(0ull, sh.q[i]));
                        }
                        continue;
                    }
                    if (rest == 0ull) break;
                    const int i = lowest(rest);
                    const float q = sh.q[i];
                    u64 w = weight(sh.p[i], q, c);  // c = 0 without draft probabilities
                    for (u64 g = gone; g != 0ull; g &= g - 1)
                        if (sh.tok[lowest(g)] == sh.tok[i]) w = 0ull;
                    if (R != 0ull && stands(sh.u[i], Z, q, w, R)) {
                        on |= 1ull << i;
                        gone = 0ull;
                        c.kind = 0;
                        Z = kOne;
                        R = kOne;
                        fresh = true;
                        continue;
                    }
                    rest &= rest - 1;
                    if (draft == nullptr) {
                        gone |= 1ull << i;
                        Z = less(Z, w);
                    } else {
                        if (R != 0ull && Z != 0ull) {
                            Num z = num(Z);
                            if (R != kOne) z = divide(z, num(R));
                            c.v = add(c.v, z);
                            c.kind = 2;  // past 1
                            z_known = false;
                        }
                        if (!a.replace) R = less(R, add_fixed(0ull, q));
                    }
                }
                if (lane == 0) {
                    sh.c = c;
                    sh.gone = gone;
                    sh.on = on;
                    sh.node = cur;
                }
            }
            __syncthreads();
            const Coef cf = sh.c;
            const u64 out = sh.gone;
            const int node = sh.node;
            const RowChunks<N> cut = row_chunks<N>(at + node, static_cast<size_t>(a.B) * a.n, a.V);
            const int skew = cut.skew;
            const RowView<T> P(target + static_cast<size_t>(node) * a.V, cut);
            const RowView<T> Q(draft + (draft != nullptr ? static_cast<size_t>(node) * a.V : 0), cut);
            const int per_piece = (P.chunks() + pieces - 1) >> (cl_log + kWarpsLog), its = (per_piece + 31) >> 5;
            const int seg = (its + kSegments - 1) / kSegments;
            const int k0 = min(piece * per_piece, P.chunks()), k1 = min(k0 + per_piece, P.chunks());
            const Sums s = cf.kind == 0   ? sweep<T, 0>(P, Q, cf.v, k0, k1, its, seg, sh.cum)
                           : cf.kind == 1 ? sweep<T, 1>(P, Q, cf.v, k0, k1, its, seg, sh.cum)
                                          : sweep<T, 2>(P, Q, cf.v, k0, k1, its, seg, sh.cum);
            u64 sw = warp_sum(s.p - s.q);
            const float sp = warp_sum(s.about());
            for (u64 g = out; g != 0ull; g &= g - 1) {  // rejected tokens leave their piece's sum, once each
                const int i = lowest(g), x = sh.tok[i];
                bool first = true;
                for (u64 f = out & ((1ull << i) - 1); f != 0ull; f &= f - 1) first = first && sh.tok[lowest(f)] != x;
                const int k = (x + skew) / N;
                if (first && k >= k0 && k < k1) sw -= add_fixed(0ull, sh.p[i]);
            }
            const int buf = round & 1;
            if (lane < CL)
                send16(peer_addr(smem_u32(&sh.part[buf][piece]), lane), sw, __float_as_uint(sp),
                       peer_addr(smem_u32(&sh.bar[buf]), lane));
            if (warp == 0) {
                int state = kSweep, own = -1;
                u64 rem = 0ull;
                if (!warp_wait(&sh.bar[buf], (round >> 1) & 1)) {
                    if (lane == 0) raise_error(a.err, kDevErrTimeout);
                    state = kLost;
                    own = round;
                } else {
                    if (lane == 0) mbar_arrive_expect_tx(&sh.bar[buf], pieces * sizeof(Part));  // the round after the next
                    // a lane sums its pieces; a scan over the lanes orders them
                    u64 wl[kLanePieces], sum = 0ull;
                    float all = 0.f;
#pragma unroll
                    for (int i = 0; i < kLanePieces; ++i) {
                        const int e = lane * kLanePieces + i;
                        wl[i] = e < pieces ? sh.part[buf][e].w : 0ull;
                        all += e < pieces ? sh.part[buf][e].p : 0.f;
                        sum += wl[i];
                    }
                    all = warp_sum(all);
                    const u64 incl = warp_scan(sum), whole = __shfl_sync(0xffffffffu, incl, 31);
                    if (!(all <= kMostSum)) {
                        state = kBad;
                    } else if (rest != 0ull) {
                        Z = whole;
                        z_known = true;
                    } else if (whole == 0ull) {  // nothing of p is left: draw from p itself
                        if (c.kind == 0 && gone == 0ull) state = kBad;
                        c.kind = 0;
                        gone = 0ull;
                    } else {
                        state = kDraw;
                        // floor(u whole): u = m 2^(exponent - 126) / 2^32, m with its leading bit at 31
                        const uint32_t ub = __float_as_uint(sh.u[0]);
                        u64 T0 = shr(__umul64hi(whole, static_cast<u64>((ub << 8) | 0x80000000u) << 32),
                                     126 - static_cast<int>(ub >> 23));
                        if (ub >= 0x3F800000u) T0 = whole - 1;  // u = 1: the last token with any weight
                        // the piece that holds it, and how far into it
                        const int hit = __ffs(__ballot_sync(0xffffffffu, incl > T0)) - 1;
                        rem = T0 - (incl - sum);
#pragma unroll
                        for (int i = 0; i < kLanePieces; ++i) {
                            if (own < 0 && rem < wl[i]) own = lane * kLanePieces + i;
                            if (own < 0) rem -= wl[i];
                        }
                        own = __shfl_sync(0xffffffffu, own, hit);
                        rem = __shfl_sync(0xffffffffu, rem, hit);
                    }
                }
                if (lane == 0) {
                    sh.state = state;
                    sh.own = own;
                    sh.rem = rem;
                }
            }
            __syncthreads();
            const int state = sh.state;
            if (state == kSweep) continue;
            bad = state != kDraw;
            if (!bad && sh.own == piece) {
                // the segment (lane i sums the piece's i-th), then the token in it
                u64 rem = sh.rem, tot = 0ull;
                const int segs = (its - 1) / seg + 1;
                if (lane < segs)
                    for (int i = 0; i < 32; ++i) tot += sh.cum[lane][warp * 32 + ((i + lane) & 31)];
                for (u64 g = out; g != 0ull; g &= g - 1) {
                    const int i = lowest(g), x = sh.tok[i];
                    bool first = true;
                    for (u64 f = out & ((1ull << i) - 1); f != 0ull; f &= f - 1) first = first && sh.tok[lowest(f)] != x;
                    const int k = (x + skew) / N;
                    if (first && k >= k0 && k < k1 && lane >= (k - k0) / 32 / seg) tot -= add_fixed(0ull, sh.p[i]);
                }
                const int which = __ffs(__ballot_sync(0xffffffffu, lane < segs && tot > rem)) - 1;
                const u64 prev = __shfl_sync(0xffffffffu, tot, max(which - 1, 0));
                if (which > 0) rem -= prev;
                const int s0 = k0 + 32 * seg * which;
                drawn = Weights<T>{P, Q, cf, out, sh.tok}.search(s0, min(s0 + 32 * seg, k1), rem);
            }
            break;
        }
    }
    const u64 path = idle || bad ? 0ull : sh.on;
    const int count = __popcll(path);
    if (rank == 0 && tid < a.n) {
        if (tid == 0 && bad && (idle || sh.state != kLost)) raise_error(a.err, kDevErrIndex);
        if (((path >> tid) & 1ull) != 0ull) {
            const int t = __popcll(path & ((1ull << tid) - 1));
            a.path[at + t] = tid;
            if (t > 0) a.out_tokens[at + t - 1] = sh.tok[tid];
        }
        if (tid >= count) a.path[at + tid] = a.out_tokens[at + tid] = -1;
        if (tid == 0) {
            a.n_path[b] = count;
            if (a.kv_len_out != nullptr) a.kv_len_out[b] = a.kv_len[b] + count;
        }
    }
    if (drawn >= 0 && lane == 0) a.out_tokens[at + count - 1] = drawn;
    if (!idle && sh.state == kLost) outstay(sh.bar, sh.own);
}

// The row of each of B sequences goes to the largest cluster (a power of two) whose CTAs are all resident at
// once and whose warps each have at least 32 chunks; to more than 8 CTAs only for up to 16 sequences.  us
// for B chains of 8 over 131072 fp32 tokens by CTAs per cluster, the rule's choice in brackets:
//     B      8     16     17     32     38     48     64     77    100    152    200    304    608
//    16 [10.2] [12.6]  14.5   18.0   20.3   23.2   27.9   32.2
//     8  11.7   13.4  [13.9] [15.0] [21.0] [21.2] [21.8]  26.5   32.8   42.1
//     4         17.9   18.1   18.5   22.0   22.8   23.5  [34.7] [34.9] [40.4]  50.8   66.3
//     2                       29.5   30.6   30.8   30.9   35.6   38.6   40.3  [61.8] [63.0] 112.7
//     1                                            54.2   55.0   55.4   56.2   70.2   72.6 [118.0]
// Up to 64 sequences it is within 4 % of the best power of two.  Just past the sizes that fit at once (64, 152, 304)
// twice as many CTAs in two waves would still be faster, by up to a quarter.
template <typename T>
cudaError_t launch(const VerifyArgs& a) {
    int cl_log = a.B <= 16 ? 4 : 3;
    while (cl_log > 0 && ((static_cast<long long>(a.B) << cl_log) > kResident * 152 ||
                          a.V < (kVerifyThreads * RowView<T>::N) << cl_log))
        --cl_log;
    if (cl_log > 3 &&  // past the portable size
        cudaFuncSetAttribute(verify_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
        (void)cudaGetLastError();
        cl_log = 3;
    }
    const int CL = 1 << cl_log;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.B) * CL);
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CL;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, verify_kernel<T>, a, cl_log);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a) {
    return a.bf16 ? launch<__nv_bfloat16>(a) : launch<float>(a);
}

}  // namespace infllmv2
