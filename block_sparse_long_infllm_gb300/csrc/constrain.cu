// constrain.cu -- penalties for repeated tokens, biases and grammar masks on logits, and the distributions
// they leave (what verify.cu reads); and the token counts that the penalties read.
//
// Row i of a sequence's draft tree is its logits after node i.  With c(t) how often token t was generated (in
// the history, and among the drafts on node i's way) and seen(t) whether c(t) > 0 or t is in the prompt:
//   l1 = seen ? (l > 0 ? l / repetition : l repetition) : l
//   l2 = l1 - frequency c - presence [c > 0],  l3 = l2 + bias,  -inf where the mask has no bit
// and the row becomes l3, or softmax(l3 / temperature), or at temperature 0 a one at its first largest element.
// All of it is fp32, and the same for equal logits, so what was equal stays equal.
//
// What bounds it is memory: logits read once, the result written once.  A row goes to one thread-block cluster, a
// contiguous piece of it to each warp.  Bulk copies bring the pieces, a warp walks over its own once, with running
// sums of exponentials, and leaves the adjusted logits in shared memory; the warps' sums are exchanged by
// asynchronous stores counted on the receiver's barrier, every warp joins them by itself, and the elements become
// probabilities on their way out.  Clusters are persistent (as many as fit at once) and take several rows, so a
// row's load overlaps the last one's way out.
//
// Measured on a GB300: 64 chains of 8 over 131072 fp32 logits with counts and a bias 150 us (3.7 TB/s; 108 us, 5.0
// TB/s, without either: the counts cost about 12 of 39 instructions an element), one step of it (64 rows) 24.7; bf16
// logits 159, to bf16 135; adjusted logits alone 103; 2 trees of 16 over 32001 bf16 logits with masks 7.0; one row of 131072 5.7.  By CTA and
// CTAs per SM, the 64 chains: 256 threads, 2 CTAs 150; 192, 3: 160; 512, 2: 195.  With the cluster barrier instead
// of counted stores 5 % more; values in registers instead of shared memory spilled; elements adjusted one unit at a
// time, with the checks of what there is in the innermost loop, took 55 instructions an element and 200 us.  The kept
// form's kernels by whole units spill a little at 128 registers: 40 bytes stored a thread for fp32, 24 for bf16.
#include <float.h>
#include <string.h>

#include <type_traits>

#include "internal.h"
#include "places.h"
#include "tma.cuh"

namespace infllmv2 {

namespace {

using u64 = unsigned long long;

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kResident = 2;   // CTAs per SM
constexpr int kResidentLogits = 3;  // the same of CTAs that keep nothing
constexpr int kMaxCluster = 16;
// Elements of a row that a warp keeps where a cluster's CTAs suffice, and at most (a CTA has 227 KB of shared memory).
// Clusters are powers of two, so 8 CTAs keep rows of 65537 to 131072 and 16, of which fewer fit at once, longer ones:
// 64 chains of 8 over 73448, 128256, 131072, 151936, 200064 take 112, 153, 150, 266, 320 us, their 64 rows alone 16,
// 25, 25, 40, 47.
constexpr int kPiece = 2048;
constexpr int kMostPiece = 6912;
constexpr int kSlice = kWarps * kPiece;
constexpr int kStepValues = 8;        // elements that a lane takes in one step
constexpr int kStepValuesStaged = 16; // the same out of shared memory, by whole units
constexpr float kInf = __builtin_huge_valf();

struct Controls {
    float repetition, frequency, presence, temperature;
};

__device__ __forceinline__ bool valid(const Controls& c) {
    return c.repetition > 0.f && c.repetition <= FLT_MAX && fabsf(c.frequency) <= FLT_MAX && fabsf(c.presence) <= FLT_MAX &&
           c.temperature >= 0.f && c.temperature <= FLT_MAX;
}

// A token's logit under the penalties: h its history, extra its occurrences among the drafts on the way (below
// 64); shrink is 1 / repetition.
__device__ __forceinline__ float penalised(float l, unsigned h, unsigned extra, const Controls& c, float shrink) {
    const unsigned count = (h & 0x7fffu) + extra;
    // (a count becomes fp32 by its bits: below 2^23 they are those of 2^23 + count)
    const float n = __uint_as_float(count | 0x4b000000u) - 8388608.f;
    const float less = count != 0u ? fmaf(c.frequency, n, c.presence) : 0.f;
    const float times = l > 0.f ? shrink : c.repetition;
    return fmaf(l, (h | extra) != 0u ? times : 1.f, -less);
}
// NaN weighs nothing.
__device__ __forceinline__ float number(float x) { return fmaxf(x, -kInf); }

template <typename T>
__device__ __forceinline__ float as_float(T x) {
    if constexpr (sizeof(T) == 4)
        return x;
    else
        return __bfloat162float(x);
}
template <typename T>
__device__ __forceinline__ float load1(const T* p) {
    return as_float(*p);
}
template <typename T>
__device__ __forceinline__ void store1(T* p, float x) {
    if constexpr (sizeof(T) == 4)
        *p = x;
    else
        *p = __float2bfloat16_rn(x);
}

// U consecutive elements, as they lie in memory.
template <typename T, int U>
struct alignas(sizeof(T) * U > 16 ? 16 : sizeof(T) * U) Unit {
    T v[U];
};
template <typename T, int U>
__device__ __forceinline__ Unit<T, U> load_unit(const T* p) {
    constexpr int kBytes = sizeof(T) * U;
    Unit<T, U> r;
    if constexpr (kBytes >= 16) {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i) reinterpret_cast<uint4*>(&r)[i] = reinterpret_cast<const uint4*>(p)[i];
    } else if constexpr (kBytes == 8) {
        *reinterpret_cast<uint2*>(&r) = *reinterpret_cast<const uint2*>(p);
    } else {
        r.v[0] = *p;
    }
    return r;
}
template <typename T, int U>
__device__ __forceinline__ void store_unit(T* p, const float (&x)[U]) {
    if constexpr (U == 1) {
        store1(p, x[0]);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < U; e += 4)
            *reinterpret_cast<float4*>(p + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
    } else {
        uint32_t w[U / 2];
#pragma unroll
        for (int e = 0; e < U; e += 2) w[e / 2] = pack_bf16x2(x[e], x[e + 1]);
        if constexpr (U == 8)
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    }
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kAll, x, o));
    return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kAll, x, o);
    return x;
}
__device__ __forceinline__ u64 warp_max(u64 x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = max(x, __shfl_xor_sync(kAll, x, o));
    return x;
}

// What a warp knows of its elements: their maximum (or its exponent of 2) and their sum in its units, or (in `key`)
// the largest element and, inverted, its place.
union Pair {
    struct {
        float top, sum;
    };
    u64 key;
};

// exp((x - top) / temperature), k = log2(e) / temperature; x <= top, and 1 where x is top (both may be infinite).
__device__ __forceinline__ float weight(float x, float top, float k) { return x == top ? 1.f : fast_exp2((x - top) * k); }

// A warp's piece of a row, and what becomes of its logits.
template <typename Tin>
struct Piece {
    const Tin* logits;
    uint32_t stage;             // where in shared memory bulk copies brought them
    int staged;                 // and how many of them
    const unsigned short* history;
    const unsigned* allowed;    // of the whole row
    const float* bias;
    const int2* fixes;          // places of tokens of the drafts on the way, and the bits of their logits
    int begin, count, n_fixes;  // its first token, how many (whole units)
    unsigned mine;              // this lane's steps with some of those places (modulo 32)
    Controls c;
    float shrink;
};
// What a step looks at: nothing; the history and the bias, where there is one; everything.
enum : int { kPlain = 0, kHistory = 1, kAny = 2 };

// What a step reads beside the logits, of the units that are there.  (The bias of staged single elements is loaded in
// the step itself, in fewer registers: 64 chains of 8 over 131071 249 -> 201 us; not of others, whose logits alone over
// 32001 it slows from 55 to 71.)
template <bool kStaged, int U>
constexpr bool kBiasAhead = !kStaged || U > 1;
template <int U, int S>
struct Beside {
    static constexpr int N = S / U, kWords = (U + 1) / 2;
    unsigned h[N][kWords];  // counts, two to a word
    Unit<float, U> w[N];
    unsigned ok[N];
    __device__ __forceinline__ unsigned count(int i, int e) const { return U == 1 ? h[i][0] : (e & 1) ? h[i][e / 2] >> 16 : h[i][e / 2] & 0xffffu; }
};
template <int kLook, bool kStaged, typename Tin, int U, int S>
__device__ __forceinline__ void look(const Piece<Tin>& p, int at, Beside<U, S>& s) {
#pragma unroll
    for (int i = 0; i < Beside<U, S>::N; ++i) {
        const int x = at + i * 32 * U;
        const bool there = x < p.count;
        if (there && (kLook == kHistory || (kLook == kAny && p.history != nullptr))) {
            if constexpr (U == 8) {
                const uint4 h = *reinterpret_cast<const uint4*>(p.history + x);
                s.h[i][0] = h.x;
                s.h[i][1] = h.y;
                s.h[i][2] = h.z;
                s.h[i][3] = h.w;
            } else if constexpr (U == 4) {
                const uint2 h = *reinterpret_cast<const uint2*>(p.history + x);
                s.h[i][0] = h.x;
                s.h[i][1] = h.y;
            } else {
                s.h[i][0] = p.history[x];
            }
        }
        if constexpr (kBiasAhead<kStaged, U>)
            if (there && kLook != kPlain && p.bias != nullptr) s.w[i] = load_unit<float, U>(p.bias + x);
        if (kLook == kAny) s.ok[i] = !there ? 0u : p.allowed != nullptr ? p.allowed[(p.begin + x) >> 5] >> ((p.begin + x) & 31) : ~0u;
    }
}

// One step: the values of unit i from at + 32 U i on; units that are not there are -inf.
template <int kLook, bool kStaged, typename Tin, int U, int S>
__device__ __forceinline__ void take(const Piece<Tin>& p, int at, const Beside<U, S>& s, float (&v)[S / U][U]) {
    constexpr int N = S / U;
    constexpr bool kAhead = kBiasAhead<kStaged, U>;
    float bias[kAhead ? 1 : N];
    if constexpr (!kAhead)
        if (kLook != kPlain && p.bias != nullptr) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (at + i * 32 < p.count) bias[i] = p.bias[at + i * 32];
        }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int x = at + i * 32 * U;
        Unit<Tin, U> raw;
#pragma unroll
        for (int e = 0; e < U; ++e) raw.v[e] = static_cast<Tin>(-kInf);
        const uint32_t in_stage = p.stage + x * static_cast<uint32_t>(sizeof(Tin));
        if constexpr (kStaged && U > 1) {
            if (x < p.count) {
                const uint4 w = lds_v4(in_stage);
                memcpy(&raw, &w, sizeof(raw));
            }
        } else if (kStaged && x < p.staged) {
            if constexpr (sizeof(Tin) == 4)
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(raw.v[0]) : "r"(in_stage));
            else
                asm volatile("ld.shared.b16 %0, [%1];" : "=h"(*reinterpret_cast<unsigned short*>(&raw.v[0])) : "r"(in_stage));
        } else if (x < p.count) {
            raw = load_unit<Tin, U>(p.logits + x);
        }
#pragma unroll
        for (int e = 0; e < U; ++e) v[i][e] = as_float(raw.v[e]);
    }
    if (kLook == kHistory || (kLook == kAny && p.history != nullptr)) {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int e = 0; e < U; ++e)
                if (kLook == kHistory || at + i * 32 * U < p.count) v[i][e] = penalised(v[i][e], s.count(i, e), 0u, p.c, p.shrink);
    }
    if (kLook == kAny && ((p.mine >> (at / (32 * S) % 32)) & 1u) != 0u) {
#pragma unroll 1
        for (int k = 0; k < p.n_fixes; ++k) {
            const int2 fix = p.fixes[k];
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int e = 0; e < U; ++e)
                    if (at + i * 32 * U + e == fix.x) v[i][e] = __int_as_float(fix.y);
        }
    }
    if (kLook != kPlain && p.bias != nullptr) {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int e = 0; e < U; ++e)
                if (at + i * 32 * U < p.count) {
                    if constexpr (kAhead)
                        v[i][e] += s.w[i].v[e];
                    else
                        v[i][e] += bias[i];
                }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int e = 0; e < U; ++e) {
            v[i][e] = number(v[i][e]);
            if (kLook == kAny && (s.ok[i] & (1u << e)) == 0u) v[i][e] = -kInf;
            if (kLook == kHistory && at + i * 32 * U >= p.count) v[i][e] = -kInf;
        }
    if (kStaged && (sizeof(Tin) < 4 || U == 1)) __syncwarp();  // what is kept goes over logits that were read
}

// A row goes to a cluster of `parts` CTAs (without kProbs they are independent), one contiguous piece of it to each
// warp, and a cluster takes its share of the rows (`share` of them, one more for the first `more` clusters).  A
// warp's lanes walk over its piece by units of U elements.  kStaged: a bulk copy brings a warp's piece of the next
// row to shared memory as soon as the last one is written, and the piece stays there, as fp32 over its own logits,
// until the row's sum is known.  Without (pieces past kMostPiece) it is read again.
template <typename Tin, typename Tout, int U, bool kProbs, bool kStaged>
__global__ void __launch_bounds__(kThreads, kProbs ? kResident : kResidentLogits)
    constrain_kernel(ConstrainArgs a, int parts, int piece, int share, int more) {
    constexpr int S = kStaged && U > 1 ? kStepValuesStaged : kStepValues;
    constexpr int N = S / U, kStep = 32 * S;  // units of a lane, elements of a warp in a step
    extern __shared__ float4 keep4[];  // kStaged: [warp][piece + 4] floats
    __shared__ int way_s[kWarps][64];  // tokens of the drafts on the way, by node (-1: not on it); one copy per warp
    __shared__ int2 fixes_s[kWarps][64];
    __shared__ Pair pairs[2][kMaxCluster * kWarps];
    __shared__ alignas(8) uint64_t full[kWarps], sent[2];  // sent: bytes of pairs[.] that came from the cluster's warps
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int part = blockIdx.x, cluster = blockIdx.y;
    const int from = cluster * share + min(cluster, more), to = from + share + (cluster < more ? 1 : 0);  // its rows
    // the warp's piece
    const int begin = (part * kWarps + warp) * piece;
    const int count = max(min(piece, a.V - begin), 0);  // a multiple of U
    const int steps = (count + kStep - 1) / kStep;
    // (what is kept from the memory's start on, and the 16-bit logits in its second half: a step's elements are kept
    // over logits of this step and of those before it)
    float* const keep = reinterpret_cast<float*>(keep4) + warp * (piece + 4);
    unsigned char* const stage = reinterpret_cast<unsigned char*>(keep) + (sizeof(Tin) < 4 ? piece * 2 : 0);
    const int all = parts * kWarps;
    if (kStaged && lane == 0) mbar_init(&full[warp], 1);
    if (kProbs && tid == 0) {
        mbar_init(&sent[0], 1);
        mbar_init(&sent[1], 1);
    }
    fence_mbar_init();
    __syncwarp();
    if constexpr (kProbs) {
        if (tid == 0) {
            mbar_arrive_expect_tx(&sent[0], all * sizeof(Pair));
            mbar_arrive_expect_tx(&sent[1], all * sizeof(Pair));
        }
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // this CTA's barriers are there
    }
    pdl_wait();
    pdl_trigger();

    int row = from, b = from / a.n, node = from % a.n;
    const auto step = [&] {
        ++row;
        if (++node == a.n) {
            node = 0;
            ++b;
        }
    };
    const auto unused = [&] {  // rows behind their sequence's last node are left as they are
        if (a.n_nodes == nullptr || row >= to) return false;
        const int nodes = a.n_nodes[b];
        return nodes >= 0 && nodes <= node;
    };
    while (unused()) step();
    // The whole 16 bytes that hold the row's piece: they start `skew` elements before it, and hold `staged` of it.
    int skew = 0, staged = 0;
    const auto fetch = [&] {
        const Tin* const first = static_cast<const Tin*>(a.logits) + row * a.ld + begin;
        const Tin* const tensor_end = static_cast<const Tin*>(a.logits) + (a.B * a.n - 1) * a.ld + a.V;
        const unsigned char* const src = reinterpret_cast<const unsigned char*>(reinterpret_cast<uintptr_t>(first) & ~uintptr_t{15});
        skew = static_cast<int>(first - reinterpret_cast<const Tin*>(src));
        uint32_t bytes = (static_cast<uint32_t>(skew + count) * static_cast<uint32_t>(sizeof(Tin)) + 15u) & ~15u;
        if (src + bytes > reinterpret_cast<const unsigned char*>(tensor_end)) bytes -= 16u;
        if (count == 0) bytes = 0u;
        staged = min(static_cast<int>(bytes / sizeof(Tin)) - skew, count);
        if (lane != 0) return;
        fence_proxy_async_shared();  // what is overwritten was read before
        mbar_arrive_expect_tx(&full[warp], bytes);
        if (bytes != 0u) bulk_load(stage, src, bytes, &full[warp]);
    };
    if (kStaged && row < to) fetch();
    // A wait ran out: this warp goes through its rows without waiting, loading or sending, and writes none but bad ones.
    // (It has not seen the others' pairs, so it does not know how many turns of a row they take: a pair too many would
    // reach a CTA that has ended.  Those who miss its pairs are lost as well.)
    bool lost = false;
    uint32_t loads = 0u;
    int turn = 0;
    const auto wait = [&](uint64_t* bar, uint32_t parity) {
        lost = !__all_sync(kAll, mbar_wait(bar, parity));
        if (lost && lane == 0) raise_error(a.err, kDevErrTimeout);
    };

    // every warp's pair to every CTA of the cluster, counted on the receiver's barrier; returns those of all
    const auto exchange = [&](Pair p) -> const Pair* {
        if (turn == 0) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        Pair* const buf = pairs[turn & 1];
        uint64_t* const bar = &sent[turn & 1];
        if (lane < parts && !lost) {
            uint32_t dst, dst_bar;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(dst) : "r"(smem_u32(&buf[part * kWarps + warp])), "r"(lane));
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(dst_bar) : "r"(smem_u32(bar)), "r"(lane));
            asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(dst), "l"(p.key),
                         "r"(dst_bar)
                         : "memory");
        }
        if (!lost) wait(bar, (turn >> 1) & 1);
        // (this buffer's next pairs come after every warp has read these: they are sent with the next turn's known)
        if (tid == 0 && !lost) mbar_arrive_expect_tx(bar, all * sizeof(Pair));
        ++turn;
        return buf;
    };

#pragma unroll 1
    while (row < to) {
        Tout* const out = static_cast<Tout*>(a.out) + row * a.ld_out + begin;
        Controls c{1.f, 0.f, 0.f, 1.f};
        if (a.controls != nullptr) {
            const float* const p = a.controls + 4ll * b;
            c = Controls{p[0], p[1], p[2], p[3]};
        }
        const int nodes = a.n_nodes != nullptr ? a.n_nodes[b] : a.n;
        bool bad = nodes < 0 || nodes > a.n || !valid(c);
        const Tin* const logits = static_cast<const Tin*>(a.logits) + row * a.ld + begin;
        const unsigned short* const history = a.history != nullptr ? a.history + b * a.ld_history + begin : nullptr;
        const float shrink = 1.f / c.repetition;

        // the drafts on the way (a root has none, but its mask is checked like the others'): each warp looks for those
        // in its piece and makes their logits
        unsigned mine = 0u;
        int n_fixes = 0;
        const u64 way = a.tree_mask != nullptr ? a.tree_mask[row] : ~0ull >> (63 - node);
        if (a.n < 64) bad = bad || (way >> a.n) != 0ull;
        if (a.tokens != nullptr && node > 0) {
            __syncwarp();  // the last row's were read
#pragma unroll 1
            for (int k = lane; k < (a.n + 31) / 32 * 32; k += 32) {
                int t = -1;
                if (k > 0 && k < a.n && ((way >> k) & 1ull) != 0ull) {
                    t = a.tokens[b * a.n + k];
                    if (t < 0 || t >= a.V) {
                        bad = true;
                        t = -1;
                    }
                }
                way_s[warp][k] = t;
            }
            bad = __any_sync(kAll, bad) != 0;  // alike in all warps
            __syncwarp();
#pragma unroll 1
            for (int k0 = 0; k0 < a.n && !bad; k0 += 32) {
                const int t = k0 + lane < a.n ? way_s[warp][k0 + lane] : -1, in = t - begin;
                const bool here = t >= begin && in < count;
                const unsigned found = __ballot_sync(kAll, here);
                if (found == 0u) continue;
                if (here) {
                    unsigned extra = 0u;
#pragma unroll 4
                    for (int m = 1; m < a.n; ++m) extra += way_s[warp][m] == t;
                    const float l = penalised(load1(logits + in), history != nullptr ? history[in] : 0u, extra, c, shrink);
                    fixes_s[warp][n_fixes + __popc(found & ((1u << lane) - 1u))] = make_int2(in, __float_as_int(l));
                }
                n_fixes += __popc(found);
            }
            __syncwarp();
#pragma unroll 1
            for (int k = 0; k < n_fixes; ++k) {
                const int in = fixes_s[warp][k].x;
                if (in / U % 32 == lane) mine |= 1u << (in / kStep % 32);
            }
        }
        const Piece<Tin> p{logits, smem_u32(stage) + skew * static_cast<uint32_t>(sizeof(Tin)), staged, history,
                           a.allowed != nullptr ? a.allowed + row * a.ld_allowed : nullptr,
                           a.bias != nullptr ? a.bias + b * a.ld_bias + begin : nullptr, fixes_s[warp], begin, count, n_fixes,
                           mine, c, shrink};
        const int how = p.allowed != nullptr || n_fixes > 0 || (p.bias != nullptr && p.history == nullptr)
                            ? kAny
                        : p.history != nullptr ? kHistory : kPlain;
        const auto arrived = [&] {
            if constexpr (kStaged) {
                if (!lost) wait(&full[warp], loads++ & 1u);
            }
        };
        // f(first place, values) for each step
        const auto sweep = [&](auto f) {
            float v[N][U];
            Beside<U, S> one, two;
            int at = lane * U;
            if (kStaged && how != kHistory) arrived();
            if (how == kPlain) {
#pragma unroll 1
                for (int s = 0; s < steps; ++s, at += kStep) {
                    take<kPlain, kStaged, Tin, U, S>(p, at, one, v);
                    f(at, v);
                }
            } else if (how == kHistory) {  // loaded a step ahead
                look<kHistory, kStaged, Tin, U, S>(p, at, one);
                if (kStaged) arrived();
#pragma unroll 1
                for (int s = 0; s < steps; s += 2, at += 2 * kStep) {
                    look<kHistory, kStaged, Tin, U, S>(p, at + kStep, two);
                    take<kHistory, kStaged, Tin, U, S>(p, at, one, v);
                    f(at, v);
                    if (s + 1 == steps) break;
                    look<kHistory, kStaged, Tin, U, S>(p, at + 2 * kStep, one);
                    take<kHistory, kStaged, Tin, U, S>(p, at + kStep, two, v);
                    f(at + kStep, v);
                }
            } else {
#pragma unroll 1
                for (int s = 0; s < steps; ++s, at += kStep) {
                    look<kAny, kStaged, Tin, U, S>(p, at, one);
                    take<kAny, kStaged, Tin, U, S>(p, at, one, v);
                    f(at, v);
                }
            }
        };
        const auto put = [&](int at, const float (&v)[N][U]) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (at + i * 32 * U < count) store_unit<Tout, U>(out + at + i * 32 * U, v[i]);
        };
        // every step as f(first place, values) makes it
        const auto fill = [&](auto f) {
            float v[N][U];
#pragma unroll 1
            for (int at = lane * U; at < steps * kStep; at += kStep) {
                f(at, v);
                put(at, v);
            }
        };
        // ... from what was kept (-inf where nothing is), or read again
        const auto again = [&](auto f) {
            float v[N][U];
#pragma unroll 1
            for (int at = lane * U; at < steps * kStep; at += kStep) {
                if constexpr (kStaged) {
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const int x = at + i * 32 * U;
#pragma unroll
                        for (int e = 0; e < U; ++e) v[i][e] = -kInf;
                        if (x >= count) continue;
                        if constexpr (U == 1) {
                            v[i][0] = keep[x];
                        } else {
#pragma unroll
                            for (int e = 0; e < U; e += 4) {
                                const float4 w = *reinterpret_cast<const float4*>(keep + x + e);
                                v[i][e] = w.x;
                                v[i][e + 1] = w.y;
                                v[i][e + 2] = w.z;
                                v[i][e + 3] = w.w;
                            }
                        }
                    }
                } else {
                    Beside<U, S> s;
                    look<kAny, false, Tin, U, S>(p, at, s);
                    take<kAny, false, Tin, U, S>(p, at, s, v);
                }
                f(at, v);
            }
        };
        // this warp is through with the row
        const auto done = [&] {
            do step();
            while (unused());
            if constexpr (kStaged) {
                __syncwarp();
                if (row < to && !lost) fetch();
            }
        };
        if (bad) {  // alike in all CTAs of the row
            arrived();
            if (part == 0 && tid == 0) raise_error(a.err, kDevErrIndex);
            fill([&](int, float (&v)[N][U]) {
#pragma unroll
                for (int i = 0; i < S; ++i) v[i / U][i % U] = kProbs ? 0.f : -kInf;
            });
            done();
            continue;
        }
        if constexpr (!kProbs) {
            sweep(put);
            done();
        } else {
            // exp(l / temperature) is 2^(l k); sums are in units of 2^ref, ref the rounded product of k and a logit that
            // is not 32 / k below the largest so far (at first that of a number below every usual logit)
            const bool greedy = c.temperature == 0.f;
            const float k = fminf(1.44269504088896341f / c.temperature, FLT_MAX);
            const float least = -0x1p90f, ref0 = least * k;
            float top = greedy ? -kInf : least, ref = ref0, sum = 0.f;
            int place = 0;
            sweep([&](int at, const float (&v)[N][U]) {
                if (lost) return;
                if (greedy) {
#pragma unroll
                    for (int i = 0; i < S; ++i)
                        if (v[i / U][i % U] > top) {
                            top = v[i / U][i % U];
                            place = begin + at + i / U * 32 * U + i % U;
                        }
                    return;
                }
                float most = v[0][0];
#pragma unroll
                for (int i = 1; i < S; ++i) most = fmaxf(most, v[i / U][i % U]);
                if (fmaf(most, k, -ref) > 32.f) {  // (rarely: fp32's range is wide)
                    const float to = most * k;
                    sum *= fast_exp2(ref - to);
                    ref = to;
                }
                float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < S; ++i) s[i % 4] += fast_exp2(fmaf(v[i / U][i % U], k, -ref));
                sum += (s[0] + s[1]) + (s[2] + s[3]);
                if constexpr (kStaged) {
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const int x = at + i * 32 * U;
                        if (x >= count) continue;
                        if constexpr (U == 1) {
                            keep[x] = v[i][0];
                        } else {
#pragma unroll
                            for (int e = 0; e < U; e += 4)
                                *reinterpret_cast<float4*>(keep + x + e) = make_float4(v[i][e], v[i][e + 1], v[i][e + 2], v[i][e + 3]);
                        }
                    }
                }
            });
            Pair own;
            if (greedy) {
                own.key = warp_max((static_cast<u64>(ordered_key(top)) << 32) | ~static_cast<unsigned>(place));
                const Pair* const theirs = exchange(own);
                u64 best = 0ull;
#pragma unroll 1
                for (int i = lane; i < all; i += 32) best = max(best, theirs[i].key);
                best = warp_max(best);
                const bool some = static_cast<unsigned>(best >> 32) != ordered_key(-kInf);
                const int first = some ? static_cast<int>(~static_cast<unsigned>(best)) - begin : -1;
                if (!lost)
                    fill([&](int at, float (&v)[N][U]) {
#pragma unroll
                        for (int i = 0; i < S; ++i) v[i / U][i % U] = at + i / U * 32 * U + i % U == first ? 1.f : 0.f;
                    });
                done();
                continue;
            }
            own.top = warp_max(ref);
            own.sum = warp_sum(sum * fast_exp2(ref - own.top));
            const Pair* theirs = exchange(own);
            float most = ref0, total = 0.f;
#pragma unroll 1
            for (int i = lane; i < all; i += 32) {
                const Pair q = theirs[i];
                const float to = fmaxf(most, q.top);
                total = total * fast_exp2(most - to) + q.sum * fast_exp2(q.top - to);
                most = to;
            }
            top = warp_max(most);
            total = warp_sum(total * fast_exp2(most - top));
            most = top;
            // rows of nothing, of infinities, of numbers or temperatures at fp32's ends: the maximum, then the sum
            const bool usual = k <= 0x1p30f && most > ref0 && most < kInf;
            float inv = 1.f / total;
            if (usual && !lost)
                again([&](int at, float (&v)[N][U]) {
#pragma unroll
                    for (int i = 0; i < S; ++i) v[i / U][i % U] = fast_exp2(fmaf(v[i / U][i % U], k, -most)) * inv;
                    put(at, v);
                });
#pragma unroll 1
            for (int phase = 0; phase < 3 && !usual; ++phase) {
                top = -kInf;
                sum = 0.f;
                if (!lost)
                    again([&](int at, float (&v)[N][U]) {
#pragma unroll
                        for (int i = 0; i < S; ++i) {
                            float& x = v[i / U][i % U];
                            top = fmaxf(top, x);
                            x = most > -kInf ? weight(x, most, k) : 0.f;
                            sum += x;
                            x *= inv;
                        }
                        if (phase == 2) put(at, v);
                    });
                if (phase == 2) break;
                own.top = warp_max(top);
                own.sum = warp_sum(sum);
                theirs = exchange(own);
                if (phase == 0) {
                    most = -kInf;
#pragma unroll 1
                    for (int i = lane; i < all; i += 32) most = fmaxf(most, theirs[i].top);
                    most = warp_max(most);
                } else {
                    total = 0.f;
#pragma unroll 1
                    for (int i = lane; i < all; i += 32) total += theirs[i].sum;
                    total = warp_sum(total);
                    inv = total > 0.f ? 1.f / total : 0.f;
                }
            }
            done();
        }
    }
    if constexpr (kProbs) {
        if (turn == 0) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (lost) {
            // its peers may still send to this CTA: it stays until all of them have ended or are lost, then for the length
            // of a wait (what they sent last is on its way, and nobody counts it), and until its own copy is here
            asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
            for (const long long t0 = clock64(); clock64() - t0 < kWaitBudgetCycles;) __nanosleep(1000);
            __syncwarp();
            if (kStaged) (void)__all_sync(kAll, mbar_wait(&full[warp], (loads - 1u) & 1u));
        }
    }
}

template <typename Tin, typename Tout, int U, bool kProbs, bool kStaged>
cudaError_t launch_kind(const ConstrainArgs& a, int parts, int piece, int clusters) {
    const auto kern = constrain_kernel<Tin, Tout, U, kProbs, kStaged>;
    if (kProbs && parts > 8) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    const auto bytes = [](int n) { return (n + 4) * kWarps * static_cast<int>(sizeof(float)); };
    const int smem = kStaged ? bytes(piece) : 0;
    if (kStaged) {
        // (the limit belongs to the function and all host threads share it: each call sets the same one, the largest)
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes(kMostPiece));
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    const int rows = a.B * a.n;
    if (clusters > 65535) clusters = 65535;  // (the grid's limit)
    cfg.gridDim = dim3(parts, clusters);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = parts;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kProbs ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a, parts, piece, rows / clusters, rows % clusters);
}

template <typename Tin, typename Tout, int U>
cudaError_t launch_units(const ConstrainArgs& a) {
    const int rows = a.B * a.n;
    const auto pieces = [&](int n) { return ((a.V + n * kWarps - 1) / (n * kWarps) + 31) / 32 * 32; };
    if (!a.probs) {
        const int parts = (a.V + kSlice - 1) / kSlice;
        return launch_kind<Tin, Tout, U, false, false>(a, parts, pieces(parts), rows);
    }
    // as many CTAs as keep a row, more where that leaves SMs without work
    int parts = 1;
    while (parts < kMaxCluster && (parts * kSlice < a.V || (rows * parts * 2 <= kResident * 152 && parts * kThreads * U < a.V)))
        parts *= 2;
    const int piece = pieces(parts);
    if (piece > kMostPiece) return launch_kind<Tin, Tout, 1, true, false>(a, parts, piece, rows);
    // clusters that are resident at once (fewer for pieces past kPiece): the SMs of a part of the GPU do not always divide by their size
    const int fit = parts <= 2 ? kResident * 152 / parts : parts == 4 ? 36 * kResident : parts == 8 ? 17 * kResident : 7 * kResident;
    return launch_kind<Tin, Tout, U, true, true>(a, parts, piece, rows < fit ? rows : fit);
}

// Units of 16 bytes of the logits where the rows of every tensor start on one of theirs and end with a whole one,
// else single elements.
template <typename Tin, typename Tout>
cudaError_t launch(const ConstrainArgs& a) {
    constexpr int U = 16 / sizeof(Tin);
    const bool aligned = (a.V | a.ld | a.ld_out | a.ld_history | a.ld_bias) % U == 0;
    return aligned ? launch_units<Tin, Tout, U>(a) : launch_units<Tin, Tout, 1>(a);
}

// ---- token counts
//
// Measured: a prompt chunk's 4 x 4096 tokens marked 3.2 us (a launch), a step's 64 x 8 tokens 2.3; 64 sequences that start anew with prompts of up
// to 32768 tokens and 4096 generated ones, two launches, 15.6 us (17 MB of rows written: 2.5 at the copy rate; most of
// the rest is the longest sequences' reading, 2.4 us a round of 8192 tokens, and two starts).  By compare-and-swap
// on global memory it took 112 us (frequent tokens wait for one another), with tokens sent to their slices' CTAs
// through distributed shared memory 28, with 512 threads 18.8.

constexpr int kFewThreads = 256;
constexpr int kHistThreads = 1024;
constexpr int kHistSlice = 16384;  // tokens of the vocabulary that a CTA counts
constexpr int kMarkSlice = 32768;  // the same of a prompt's tokens
constexpr int kHistUnroll = 2;     // loads of four tokens under way
constexpr int kFewTokens = 128;    // generated tokens of a sequence, on average, that one CTA counts alone
constexpr int kFewLongest = 1024;  // the same of packed ones, of which one may have nearly all
constexpr int kFewMarks = 32768;   // tokens of prompts, of all sequences, that are marked one by one

// How a 16-bit count takes n more of its token.
__device__ __forceinline__ unsigned counted(unsigned h, int n) {
    return (h & 0x8000u) | min((h & 0x7fffu) + static_cast<unsigned>(n), 0x7fffu);
}

// A sequence's tokens: tokens[first .. first + n); n < 0 where they are not to be read.
struct Text {
    long long first;
    int n;
};
__device__ __forceinline__ Text text_of(const CountArgs& a, int b) {
    if (a.cu == nullptr) {
        const int n = a.n_tokens != nullptr ? a.n_tokens[b] : a.T;
        return Text{static_cast<long long>(b) * a.T, n < 0 || n > a.T ? -1 : n};
    }
    const int lo = a.cu[b], hi = a.cu[b + 1];
    const bool bad = lo < 0 || hi < lo || hi > a.total || (b == 0 && lo != 0);
    return Text{lo, bad ? -1 : hi - lo};
}

// The sequence of the which-th list (from 0) of more than kFewLongest tokens, or -1, found by the whole CTA.
__device__ int long_list(const CountArgs& a, int which) {
    __shared__ int in_warp[kHistThreads / 32], found;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    for (int first = 0; first < a.B; first += kHistThreads) {
        const bool is = first + tid < a.B && text_of(a, first + tid).n > kFewLongest;
        const unsigned ones = __ballot_sync(kAll, is);
        if (lane == 0) in_warp[warp] = __popc(ones);
        const int here = __syncthreads_count(is);
        if (which < here) {
            int rank = __popc(ones & ((1u << lane) - 1u));
            for (int w = 0; w < warp; ++w) rank += in_warp[w];
            if (is && rank == which) found = first + tid;
            __syncthreads();
            return found;
        }
        which -= here;
        __syncthreads();
    }
    return -1;
}

// One CTA counts a slice of the vocabulary over all of a sequence's tokens, in shared memory, and then owns the
// slice of the row: no atomics on global memory, however often a token comes.  A prompt's tokens are marked in
// bytes (of 0x80, the sign of a 16-bit word), so a slice can be longer.  kLong: of long lists alone.
template <bool kPrompt, bool kLong>
__global__ void __launch_bounds__(kHistThreads) count_slice_kernel(CountArgs a, bool vectors) {
    using Cell = std::conditional_t<kPrompt, unsigned char, int>;
    constexpr int kSlice = kPrompt ? kMarkSlice : kHistSlice;
    extern __shared__ int4 cells4[];
    Cell* const cells = reinterpret_cast<Cell*>(cells4);
    const int tid = threadIdx.x;
    int b = blockIdx.y;
    if constexpr (kLong) {
        pdl_wait();
        b = long_list(a, b);
        if (b < 0) return;
    }
    const int begin = blockIdx.x * kSlice, width = min(kSlice, a.V - begin);
    for (int i = tid; i < kSlice * static_cast<int>(sizeof(Cell)) / 16; i += kHistThreads) cells4[i] = make_int4(0, 0, 0, 0);
    pdl_wait();
    pdl_trigger();
    const Text text = text_of(a, b);
    bool bad = text.n < 0;
    const int* const t = a.tokens + text.first;
    __syncthreads();
    const auto add = [&](int x) {
        if (blockIdx.x == 0) bad = bad || static_cast<unsigned>(x) >= static_cast<unsigned>(a.V);
        const unsigned at = static_cast<unsigned>(x) - static_cast<unsigned>(begin);
        if (at >= static_cast<unsigned>(width)) return;
        if constexpr (kPrompt)
            cells[at] = 0x80;
        else
            atomicAdd(&cells[at], 1);
    };
    if (text.n > 0) {
        const int head = min(static_cast<int>((16 - (reinterpret_cast<uintptr_t>(t) & 15u)) / 4 % 4), text.n);
        const int quads = (text.n - head) / 4;
        const int4* const t4 = reinterpret_cast<const int4*>(t + head);
        for (int i = tid; i < quads; i += kHistThreads * kHistUnroll) {
            int4 x[kHistUnroll];
#pragma unroll
            for (int u = 0; u < kHistUnroll; ++u)
                if (i + u * kHistThreads < quads) x[u] = t4[i + u * kHistThreads];
#pragma unroll
            for (int u = 0; u < kHistUnroll; ++u)
                if (i + u * kHistThreads < quads) {
                    add(x[u].x);
                    add(x[u].y);
                    add(x[u].z);
                    add(x[u].w);
                }
        }
        const int rest = head + quads * 4 + tid;
        if (tid < head) add(t[tid]);
        if (rest < text.n) add(t[rest]);
    }
    if (bad) raise_error(a.err, kDevErrIndex);
    __syncthreads();
    unsigned short* const row = a.history + b * a.ld_history + begin;
    const auto joined = [&](unsigned was, Cell n) {
        return kPrompt ? was | static_cast<unsigned>(n) << 8 : n != 0 ? counted(was, static_cast<int>(n)) : was;
    };
    const int whole = vectors ? width / 8 * 8 : 0;
    for (int i = tid * 8; i < whole; i += kHistThreads * 8) {
        alignas(16) Cell n[8];
        if constexpr (kPrompt) {
            *reinterpret_cast<uint2*>(n) = *reinterpret_cast<const uint2*>(&cells[i]);
        } else {
            reinterpret_cast<int4*>(n)[0] = *reinterpret_cast<const int4*>(&cells[i]);
            reinterpret_cast<int4*>(n)[1] = *reinterpret_cast<const int4*>(&cells[i + 4]);
        }
        bool any = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) any = any || n[e] != 0;
        if (!any && !a.reset) continue;
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (!a.reset) w = *reinterpret_cast<const uint4*>(row + i);
        unsigned h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = joined(h[e] & 0xffffu, n[2 * e]) | joined(h[e] >> 16, n[2 * e + 1]) << 16;
        *reinterpret_cast<uint4*>(row + i) = make_uint4(h[0], h[1], h[2], h[3]);
    }
    const auto one = [&](int x) {
        const Cell n = cells[x];
        if (n != 0 || a.reset) row[x] = static_cast<unsigned short>(joined(a.reset ? 0u : row[x], n));
    };
    int rest = whole;
    if (!vectors) {  // rows off a vector's boundary go by words
        const int odd = (reinterpret_cast<uintptr_t>(row) & 2u) != 0u ? 1 : 0, words = (width - odd) / 2;
        unsigned* const w = reinterpret_cast<unsigned*>(row + odd);
        if (tid < min(odd, width)) one(tid);
#pragma unroll 4
        for (int i = tid; i < words; i += kHistThreads) {
            const Cell lo = cells[odd + 2 * i], hi = cells[odd + 2 * i + 1];
            if (lo == 0 && hi == 0 && !a.reset) continue;
            const unsigned was = a.reset ? 0u : w[i];
            w[i] = joined(was & 0xffffu, lo) | joined(was >> 16, hi) << 16;
        }
        rest = odd + max(words, 0) * 2;
    }
    if (rest + tid < width) one(rest + tid);
}

// Few generated tokens: one CTA per sequence.  The first of each kFewThreads tokens' equals adds all of them, so
// nothing is added to twice at once.  Packed lists of more than kFewLongest are left to the other kernel: 4 us for each
// kFewThreads tokens, one list of 8192 would take 128 (5.7 there; the other launch costs the rest of such calls 2.1).
__global__ void __launch_bounds__(kFewThreads) count_few_kernel(CountArgs a) {
    __shared__ alignas(16) int near[kFewThreads];
    const int b = blockIdx.x, tid = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    const Text text = text_of(a, b);
    bool bad = text.n < 0;
    unsigned short* const row = a.history + b * a.ld_history;
    const int tokens = a.cu != nullptr && text.n > kFewLongest ? 0 : text.n;
    for (int at = 0; at < tokens; at += kFewThreads) {
        const int n = min(kFewThreads, tokens - at);
        int t = -1;
        if (tid < n) {
            t = a.tokens[text.first + at + tid];
            if (static_cast<unsigned>(t) >= static_cast<unsigned>(a.V)) {
                bad = true;
                t = -1;
            }
        }
        __syncthreads();  // the last tokens were read, and counted
        near[tid] = t;
        __syncthreads();
        if (t < 0) continue;
        int same = 0, before = 0;
        for (int i = 0; i < n; i += 4) {
            const int4 x = *reinterpret_cast<const int4*>(&near[i]);
            const int y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                same += y[e] == t;
                before += y[e] == t && i + e < tid;
            }
        }
        if (before == 0) row[t] = static_cast<unsigned short>(counted(row[t], same));
    }
    if (bad) raise_error(a.err, kDevErrIndex);
}

// Few tokens of prompts: one per thread (a word that several mark gets the same from each).
__global__ void __launch_bounds__(kFewThreads) count_mark_kernel(CountArgs a) {
    pdl_wait();
    pdl_trigger();
    const long long r = static_cast<long long>(blockIdx.x) * kFewThreads + threadIdx.x;
    int b = -1;
    bool bad = false;
    if (r < a.total) {
        if (a.cu == nullptr) {
            b = static_cast<int>(r / a.T);
            const int n = a.n_tokens != nullptr ? a.n_tokens[b] : a.T;
            bad = n < 0 || n > a.T;
            if (bad || r % a.T >= n) b = -1;
        } else {
            const PackedRow p = packed_row(a.cu, a.B, static_cast<int>(r), static_cast<int>(a.total), static_cast<int>(a.total));
            if (p.len > 0) b = p.b;
        }
    }
    if (a.cu != nullptr && blockIdx.x == 0)
        for (int i = threadIdx.x; i < a.B; i += kFewThreads) bad = bad || text_of(a, i).n < 0;
    if (b >= 0) {
        const int t = a.tokens[r];
        if (static_cast<unsigned>(t) >= static_cast<unsigned>(a.V)) {
            bad = true;
        } else {
            unsigned short* const h = a.history + b * a.ld_history + t;
            *h = static_cast<unsigned short>(*h | 0x8000u);
        }
    }
    if (bad) raise_error(a.err, kDevErrIndex);
}

}  // namespace

cudaError_t launch_constrain(const ConstrainArgs& a) {
    using bf16 = __nv_bfloat16;
    if (a.in_bf16) return a.out_bf16 ? launch<bf16, bf16>(a) : launch<bf16, float>(a);
    return a.out_bf16 ? launch<float, bf16>(a) : launch<float, float>(a);
}

template <bool kPrompt, bool kLong>
static cudaError_t launch_slices(const CountArgs& a, long long lists) {
    constexpr int slice = kPrompt ? kMarkSlice : kHistSlice;
    constexpr int smem = kPrompt ? kMarkSlice : kHistSlice * static_cast<int>(sizeof(int));
    const auto kern = count_slice_kernel<kPrompt, kLong>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, dim3((a.V + slice - 1) / slice, static_cast<unsigned>(lists)), dim3(kHistThreads), smem, a.stream,
                         true, a, a.ld_history % 8 == 0);
}

cudaError_t launch_count(const CountArgs& a) {
    if (a.reset || a.total > (a.prompt ? kFewMarks : static_cast<long long>(a.B) * kFewTokens))
        return a.prompt ? launch_slices<true, false>(a, a.B) : launch_slices<false, false>(a, a.B);
    if (!a.prompt) {
        const cudaError_t e = launch_kernel(count_few_kernel, dim3(a.B), dim3(kFewThreads), 0, a.stream, true, a);
        // (offsets in order leave room for no more long lists)
        const long long lists = a.cu != nullptr ? a.total / (kFewLongest + 1) : 0;
        return e != cudaSuccess || lists == 0 ? e : launch_slices<false, true>(a, lists);
    }
    return launch_kernel(count_mark_kernel, dim3(static_cast<unsigned>((a.total + kFewThreads - 1) / kFewThreads)),
                         dim3(kFewThreads), 0, a.stream, true, a);
}

}  // namespace infllmv2
