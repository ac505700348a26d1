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
// clock and SM).
//
// What bounds it is memory: the last node's target row (and draft row, once a child was rejected).
// One thread-block cluster per sequence, the row split over its CTAs and warps in contiguous
// pieces; the CTAs exchange their sums in distributed shared memory, and the warp that holds the
// sampled token reads its piece again.
#include <cooperative_groups.h>

#include "internal.h"

namespace infllmv2 {

namespace {

namespace cg = cooperative_groups;
using u64 = unsigned long long;

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxCluster = 8;
constexpr float kMostSum = 2.f;  // a row whose sum is above this holds no probabilities

// Shift right by any amount (63 and more leave 0; PTX clamps the amount).
__device__ __forceinline__ u64 shr(u64 x, int n) {
    u64 y;
    asm("shr.u64 %0, %1, %2;" : "=l"(y) : "l"(x), "r"(n));
    return y;
}

// A probability as read: NaN and negative values are 0, values past 1 are 1.
__device__ __forceinline__ float prob(float x) { return __saturatef(x); }

// p in [0, 1] in units of 2^-62, bits below that dropped.
__device__ __forceinline__ u64 fixed(float p) {
    const uint32_t b = __float_as_uint(p);
    return shr(static_cast<u64>(((b & 0x7FFFFFu) | 0x800000u) << 7) << 32, 127 - static_cast<int>(b >> 23));
}

// c as a 64-bit mantissa with its leading bit set and an exponent: c = m 2^(e - 63).
struct Coef {
    u64 m;
    int e;
    int kind;  // 0: c = 0, 1: c = 1, 2: any other
};
__device__ __forceinline__ Coef coef(double c) {
    const u64 b = static_cast<u64>(__double_as_longlong(c));
    Coef r;
    r.m = ((b & 0xFFFFFFFFFFFFFull) | 0x10000000000000ull) << 11;
    r.e = static_cast<int>(b >> 52) - 1023;
    r.kind = c == 0.0 ? 0 : c == 1.0 ? 1 : 2;
    return r;
}

// w = max(p - c q, 0) in units of 2^-62.
template <int KIND>
__device__ __forceinline__ u64 weight(float p, float q, const Coef& c) {
    const u64 P = fixed(p);
    if constexpr (KIND == 0) return P;
    u64 Q;
    if constexpr (KIND == 1) {
        Q = fixed(q);
    } else {
        const uint32_t b = __float_as_uint(q);
        const int e = c.e + static_cast<int>(b >> 23) - 127;
        // both mantissas have their leading bit at 63: the product's high word is c q 2^(62 - e)
        const u64 h = __umul64hi(c.m, static_cast<u64>((b << 8) | 0x80000000u) << 32);
        Q = e > 0 ? ~0ull : shr(h, -e);  // e > 0: c q is at least 2, past any p
        if (b == 0u) Q = 0ull;
    }
    return P > Q ? P - Q : 0ull;
}

template <typename T>
struct Chunk {  // 16 bytes of a row
    static constexpr int N = 16 / sizeof(T);
    float x[N];
};

__device__ __forceinline__ float load1(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// Elements k*N - a .. of the row (a: the row's distance from a 16-byte boundary), 0 outside it.
template <typename T>
__device__ __forceinline__ Chunk<T> load_chunk(const T* row, int k, int a, int V) {
    constexpr int N = Chunk<T>::N;
    Chunk<T> r;
    const int i0 = k * N - a;
    if (i0 >= 0 && i0 + N <= V) {
        const uint4 w = ldg_v4_stream(row + i0);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < N; ++e) {
            if constexpr (sizeof(T) == 4) {
                r.x[e] = prob(__uint_as_float(ws[e]));
            } else {
                r.x[e] = prob((e & 1) ? bf16_hi(ws[e >> 1]) : bf16_lo(ws[e >> 1]));
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) r.x[e] = i0 + e >= 0 && i0 + e < V ? prob(load1(row + i0 + e)) : 0.f;
    }
    return r;
}

struct Sums {
    u64 w;
    float p;
};

// Sum of w and of p over chunks [k0, k1), for this lane.
template <typename T, int KIND>
__device__ __forceinline__ Sums sweep(const T* p, const T* q, int k0, int k1, int a, int V, const Coef& c) {
    constexpr int N = Chunk<T>::N;
    Sums s{0ull, 0.f};
#pragma unroll 4
    for (int k = k0 + (threadIdx.x & 31); k < k1; k += 32) {
        const Chunk<T> P = load_chunk(p, k, a, V);
        Chunk<T> Q = P;
        if constexpr (KIND != 0) Q = load_chunk(q, k, a, V);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            s.w += weight<KIND>(P.x[e], Q.x[e], c);
            s.p += P.x[e];
        }
    }
    return s;
}

struct Shared {
    int tok[64];
    u64 mask[64];
    float u[64];
    float p[64], q[64];  // of each node's token in its parent's rows
    u64 kids[64];
    u64 warp_w[kVerifyWarps];
    float warp_p[kVerifyWarps];
    u64 part_w[2][kMaxCluster];
    float part_p[2][kMaxCluster];
    // the next sweep
    double c;
    int node;
    int last;   // it draws the final token
    u64 gone;   // children of `node` whose tokens are out (drafts without probabilities)
    u64 on;     // the path so far
};

// The first element of chunks [k0, k1) whose running sum of w passes T (T below their sum), by one warp.
template <typename T, int KIND>
__device__ int search(const T* p, const T* q, int k0, int k1, int a, int V, const Coef& c, u64 target, u64 gone,
                      const int* tok) {
    constexpr int N = Chunk<T>::N;
    const int lane = threadIdx.x & 31;
    u64 base = 0ull;
    for (int kb = k0; kb < k1; kb += 32) {
        const int k = kb + lane;
        u64 w[N], sum = 0ull;
        if (k < k1) {
            const Chunk<T> P = load_chunk(p, k, a, V);
            Chunk<T> Q = P;
            if constexpr (KIND != 0) Q = load_chunk(q, k, a, V);
#pragma unroll
            for (int e = 0; e < N; ++e) w[e] = weight<KIND>(P.x[e], Q.x[e], c);
            for (u64 g = gone; g != 0ull; g &= g - 1) {
                const int at = tok[__ffsll(static_cast<long long>(g)) - 1] - (k * N - a);
#pragma unroll
                for (int e = 0; e < N; ++e)
                    if (e == at) w[e] = 0ull;
            }
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) w[e] = 0ull;
        }
#pragma unroll
        for (int e = 0; e < N; ++e) sum += w[e];
        u64 incl = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const u64 y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += y;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, base + incl > target);
        if (hit != 0u) {
            int found = -1;
            if (lane == __ffs(hit) - 1) {
                u64 run = base + incl - sum;
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    run += w[e];
                    if (found < 0 && run > target) found = k * N - a + e;
                }
            }
            return __shfl_sync(0xffffffffu, found, __ffs(hit) - 1);
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    return -1;
}

template <typename T>
__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(VerifyArgs a) {
    constexpr int N = Chunk<T>::N;
    __shared__ Shared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int CL = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int b = blockIdx.x / CL, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const size_t at = static_cast<size_t>(b) * a.n;
    const T* target = static_cast<const T*>(a.target) + at * a.V;
    const T* draft = a.draft != nullptr ? static_cast<const T*>(a.draft) + at * a.V : nullptr;
    const int n = a.n_nodes != nullptr ? a.n_nodes[b] : a.n;
    bool bad = n < 0 || n > a.n;
    if (tid < 64) sh.kids[tid] = 0ull;
    if (!bad && tid < n) {
        sh.tok[tid] = a.tokens[at + tid];
        sh.u[tid] = __saturatef(a.u[at + tid]);
        const u64 own = 1ull << tid;
        sh.mask[tid] = a.tree_mask != nullptr ? a.tree_mask[at + tid] : own | (own - 1);
    }
    __syncthreads();
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
                sh.p[tid] = prob(load1(target + i));
                sh.q[tid] = draft != nullptr ? prob(load1(draft + i)) : 1.f;
            }
        }
    }
    bad = __syncthreads_or(bad) != 0;
    if (n <= 0) bad = true;
    // thread 0's walk
    int cur = 0, drawn = -1;
    u64 rest = bad ? 0ull : sh.kids[0];
    u64 gone = 0ull, on = 1ull;
    double c = 0.0, Z = 1.0, R = 1.0;
    bool z_known = true;
    if (!bad) {
        cluster.sync();  // every CTA of the cluster runs before any writes into another
        for (int round = 0;; ++round) {
            if (tid == 0) {
                while (rest != 0ull) {
                    const int i = __ffsll(static_cast<long long>(rest)) - 1;
                    const double p = sh.p[i], q = sh.q[i], u = sh.u[i];
                    double w;
                    if (draft != nullptr) {
                        if (!z_known) break;
                        w = fmax(p - c * q, 0.0);
                    } else {
                        w = p;
                        for (u64 g = gone; g != 0ull; g &= g - 1)
                            if (sh.tok[__ffsll(static_cast<long long>(g)) - 1] == sh.tok[i]) w = 0.0;
                    }
                    if (u * Z * q < w * R) {
                        cur = i;
                        on |= 1ull << i;
                        rest = sh.kids[i];
                        gone = 0ull;
                        c = 0.0;
                        Z = R = 1.0;
                        z_known = true;
                        continue;
                    }
                    rest &= rest - 1;
                    if (draft == nullptr) {
                        gone |= 1ull << i;
                        Z = fmax(Z - w, 0.0);
                    } else {
                        if (R > 0.0) {
                            c += Z / R;
                            z_known = false;
                        }
                        if (!a.replace) R -= q;
                    }
                }
                sh.c = c;
                sh.node = cur;
                sh.last = rest == 0ull;
                sh.gone = gone;
                sh.on = on;
            }
            __syncthreads();
            const int node = sh.node, fin = sh.last;
            Coef cf = coef(sh.c);
            u64 out = sh.gone;
            const T* p = target + static_cast<size_t>(node) * a.V;
            const T* q = draft + (draft != nullptr ? static_cast<size_t>(node) * a.V : 0);
            // the row in 16-byte chunks of memory, contiguous ones for each warp of the cluster
            const int skew = static_cast<int>(((at + node) * a.V) % N);
            const int chunks = (skew + a.V + N - 1) / N;
            const int per_warp = (chunks + CL * kVerifyWarps - 1) / (CL * kVerifyWarps);
            const int k0 = min((rank * kVerifyWarps + warp) * per_warp, chunks), k1 = min(k0 + per_warp, chunks);
            u64 whole = 0ull, mine = 0ull, before = 0ull;
            float sum_p = 0.f;
            for (int again = 0;; ++again) {  // once, and once more where nothing is left to draw from
                Sums s = cf.kind == 0   ? sweep<T, 0>(p, q, k0, k1, skew, a.V, cf)
                         : cf.kind == 1 ? sweep<T, 1>(p, q, k0, k1, skew, a.V, cf)
                                        : sweep<T, 2>(p, q, k0, k1, skew, a.V, cf);
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) {
                    s.w += __shfl_xor_sync(0xffffffffu, s.w, off);
                    s.p += __shfl_xor_sync(0xffffffffu, s.p, off);
                }
                if (lane == 0) {
                    sh.warp_w[warp] = s.w;
                    sh.warp_p[warp] = s.p;
                }
                __syncthreads();
                if (tid < 64 && ((out >> tid) & 1ull) != 0ull) {  // rejected tokens leave their warp's sum, once each
                    bool first = true;
                    for (u64 g = out & ((1ull << tid) - 1); g != 0ull; g &= g - 1)
                        if (sh.tok[__ffsll(static_cast<long long>(g)) - 1] == sh.tok[tid]) first = false;
                    const int owner = (sh.tok[tid] + skew) / N / per_warp;
                    if (first && owner / kVerifyWarps == rank)
                        atomicAdd(&sh.warp_w[owner % kVerifyWarps], 0ull - fixed(sh.p[tid]));
                }
                __syncthreads();
                const int buf = (round + again) & 1;
                if (tid < CL) {
                    u64 w = 0ull;
                    float pp = 0.f;
                    for (int i = 0; i < kVerifyWarps; ++i) {
                        w += sh.warp_w[i];
                        pp += sh.warp_p[i];
                    }
                    Shared* peer = cluster.map_shared_rank(&sh, tid);
                    peer->part_w[buf][rank] = w;
                    peer->part_p[buf][rank] = pp;
                }
                cluster.sync();
                whole = before = 0ull;
                sum_p = 0.f;
                for (int i = 0; i < CL; ++i) {
                    if (i < rank) before += sh.part_w[buf][i];
                    whole += sh.part_w[buf][i];
                    sum_p += sh.part_p[buf][i];
                }
                mine = sh.part_w[buf][rank];
                if (!fin || whole != 0ull || (cf.kind == 0 && out == 0ull)) {
                    round += again;
                    break;
                }
                cf = coef(0.0);  // nothing of p is left: draw from p itself
                out = 0ull;
            }
            if (!(sum_p <= kMostSum) || (fin && whole == 0ull)) {
                bad = true;
                break;
            }
            if (fin) {
                // floor(u whole): u = m 2^-(150 - exponent), m of 24 bits
                const uint32_t ub = __float_as_uint(sh.u[0]);
                u64 T0 = shr(__umul64hi(whole, static_cast<u64>((ub << 8) | 0x80000000u) << 32),
                             126 - static_cast<int>(ub >> 23));
                if (ub >= 0x3F800000u) T0 = whole - 1;  // u = 1: the last token with any weight
                if (T0 >= before && T0 - before < mine) {
                    u64 rem = T0 - before;
                    int w = 0;
                    while (w < kVerifyWarps - 1 && rem >= sh.warp_w[w]) rem -= sh.warp_w[w++];
                    if (warp == w) {
                        drawn = cf.kind == 0   ? search<T, 0>(p, q, k0, k1, skew, a.V, cf, rem, out, sh.tok)
                                : cf.kind == 1 ? search<T, 1>(p, q, k0, k1, skew, a.V, cf, rem, out, sh.tok)
                                               : search<T, 2>(p, q, k0, k1, skew, a.V, cf, rem, out, sh.tok);
                    }
                }
                break;
            }
            Z = static_cast<double>(whole) * 0x1p-62;
            z_known = true;
        }
    }
    const u64 path = bad ? 0ull : sh.on;
    const int count = __popcll(path);
    if (rank == 0) {
        if (bad && n != 0 && tid == 0) raise_error(a.err, kDevErrIndex);
        if (tid < a.n) {
            a.path[at + tid] = -1;
            if (tid != count - 1) a.out_tokens[at + tid] = -1;
        }
        if (tid == 0) {
            a.n_path[b] = count;
            if (a.kv_len_out != nullptr) a.kv_len_out[b] = a.kv_len[b] + count;
        }
        __syncthreads();
        if (tid < 64 && ((path >> tid) & 1ull) != 0ull) {
            const int t = __popcll(path & ((1ull << tid) - 1));
            a.path[at + t] = tid;
            if (t > 0) a.out_tokens[at + t - 1] = sh.tok[tid];
        }
    }
    if (drawn >= 0 && lane == 0) a.out_tokens[at + count - 1] = drawn;
}

template <typename T>
cudaError_t launch(const VerifyArgs& a) {
    int CL = 1;
    while (CL < kMaxCluster && a.V >= CL * 2 * kVerifyThreads * Chunk<T>::N) CL *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.B) * CL);
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CL;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, verify_kernel<T>, a);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a) {
    return a.bf16 ? launch<__nv_bfloat16>(a) : launch<float>(a);
}

}  // namespace infllmv2
