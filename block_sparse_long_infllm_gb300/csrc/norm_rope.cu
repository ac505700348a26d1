// norm_rope.cu -- norms of q and K rows for each head, with the rotary positions in the same pass: alone,
// into the caches, of draft trees, and the gradients of the first two.
//
// A head x of d elements becomes R(x r w): r = 1 / sqrt(mean(x^2) + eps), w the weight of q or of K (plus an
// offset, for weights stored as their distance from 1), R the rotation of rope.cu; V rows are copied.  With
// g = R^T dy, the gradient of the rotated head turned back,
//   dx = r (g w - x r mean(g w x r)),   dw = sum over rows and heads of g x r.
//
// What bounds them is memory, as in rope.cu: each element is read once and written once (a gradient reads x
// as well), and a head's sum of squares is joined by shuffles while it lies in registers.  All sums are fp32;
// a head whose squares pass fp32's range is summed again scaled by 2^-70.
//
// Measured on a GB300: 4 prompts of 16384 tokens of 32 + 2 + 2 heads of 128, bf16, 204 us (5.9 TB/s; the rotation
// alone 176); packed prompts of 8 sequences 48; 4096 rows of fp32 27.5; a decode step of 4 rows 3.4 (a launch, host
// included).  Gradients: 4096 rows of fp32 42.5 us (5.0 TB/s), 16384 145 (5.9), 4096 of bf16 31; a chunk of 4096
// tokens from fp32 gradients to bf16 36.9 (4.0 TB/s, of which 2.5 join the weights' sums).
#include <float.h>

#include "rope.cuh"

namespace infllmv2 {

namespace {

constexpr unsigned kAll = 0xffffffffu;

// 1 / sqrt(ss / d + eps): the hardware's approximation and one Newton step (r -> r + r/2 (1 - m r^2)).
__device__ __forceinline__ float inverse_root(float ss, float inv_d, float eps) {
    const float m = fmaf(ss, inv_d, eps), r = rsqrtf(m);
    return m > FLT_MAX ? 0.f : fmaf(0.5f * r, fmaf(-m * r, r, 1.f), r);
}

// Sum over the J (a power of two) neighbouring lanes of a head.
template <int J>
__device__ __forceinline__ float head_sum(float x) {
#pragma unroll
    for (int o = J >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(kAll, x, o);
    return x;
}

// What a head of E elements per lane, x, is multiplied by.  Where its squares passed fp32's range its elements are
// scaled by 2^-70 first, and the factor is that of the scaled head, 1 / sqrt(2^-140 (mean + eps)); scale says so.
template <int J, int E>
__device__ __forceinline__ float head_factor(float (&x)[E], float inv_d, float eps, float& scale) {
    scale = 1.f;
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) ss = fmaf(x[e], x[e], ss);
    ss = head_sum<J>(ss);
    if (__any_sync(kAll, !(ss <= FLT_MAX))) {
        scale = ss <= FLT_MAX ? 1.f : 0x1p-70f;
        float s2 = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            x[e] *= scale;
            s2 = fmaf(x[e], x[e], s2);
        }
        ss = head_sum<J>(s2);
        eps *= scale * scale;
    }
    return inverse_root(ss, inv_d, eps);
}

__device__ __forceinline__ float weight(const void* w, int f32, int i) {
    return f32 ? static_cast<const float*>(w)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
}
// w_s[0]: q's factors, w_s[1]: K's.
__device__ __forceinline__ void fill_weights(const NormArgs& n, int d, float (*w_s)[128]) {
    for (int i = threadIdx.x; i < 2 * d; i += kRopeThreads) {
        const int which = i >= d, e = which ? i - d : i;
        const void* w = which ? n.k_weight : n.q_weight;
        w_s[which][e] = w == nullptr ? 1.f : weight(w, n.w_f32, e) + n.offset;
    }
}

// The first elements of place j's two vectors of VEC elements: its pairs, or what does not turn.
struct Place {
    bool turns;
    int ea, eb;
};
template <int VEC>
__device__ __forceinline__ Place place_of(const RopeArgs& a, int j) {
    const int rt = a.rot / (2 * VEC);
    if (j >= rt) return Place{false, a.rot + 2 * (j - rt) * VEC, a.rot + (2 * (j - rt) + 1) * VEC};
    return a.interleaved ? Place{true, 2 * j * VEC, (2 * j + 1) * VEC} : Place{true, j * VEC, a.rot / 2 + j * VEC};
}

// ---- forward

// As in rope.cu: heads that a thread loads together, rows that a CTA takes at most, CTAs per SM.  us for the prompts
// and the packed ones (bf16) by heads, rows, CTAs: 2, 16, 3 205, 49; 2, 32, 3 212, 47; 1, 16, 4 230, 61; 2, 16, 4
// (spills) 245, 69; 3, 16, 3 222, 57; 3, 8, 3 247, 63; the next heads' loads under way while these are at work
// (spills) 222 to 244.  (The kept form's bf16 kernels of many rows store 16 to 24 bytes a thread, too.)  16384 rows of fp32: 2, 8, 4 89.6; 2, 16, 3 102; 3, 4, 3 100.
template <typename T>
struct Plan;
template <>
struct Plan<__nv_bfloat16> {
    static constexpr int kHeads = 2, kRows = 16, kResident = 3;
};
template <>
struct Plan<float> {
    static constexpr int kHeads = 2, kRows = 8, kResident = 4;
};

// VEC floats of shared memory, from a multiple of 4 on.
template <int VEC>
__device__ __forceinline__ void load_floats(const float* p, float (&x)[VEC]) {
#pragma unroll
    for (int e = 0; e < VEC; e += 4) {
        const float4 w = *reinterpret_cast<const float4*>(p + e);
        x[e] = w.x;
        x[e + 1] = w.y;
        x[e + 2] = w.z;
        x[e + 3] = w.w;
    }
}

// Pair e of a thread's place: (first, second) -> (first fc - second ss, first fs + second sc), times the head's
// factor (the weights are in them).
template <int VEC>
struct Factors {
    float fc[VEC], fs[VEC], ss[VEC], sc[VEC];
};

// One CTA takes `rows` rows.  A thread keeps one row and one place j of the heads (two vectors of VEC elements) and
// walks over the heads; the J lanes of a head are neighbours in a warp.  kSmall (calls of few CTAs): the heads of q,
// K and V are one list, and the first of them are loaded while the row is located and its angles are computed.
// Else those of q come first, then those of K and V, so that one set of factors is held at a time.
template <int FORM, typename T, int D, bool kInterleaved, bool kSmall>
__global__ void __launch_bounds__(kRopeThreads, kSmall ? 2 : Plan<T>::kResident)
    norm_rope_kernel(RopeArgs a, NormArgs n, int rows) {
    constexpr int VEC = 16 / sizeof(T), kHeads = Plan<T>::kHeads, J = D / (2 * VEC), kSlots = kRopeThreads / J;
    constexpr bool kToCache = FORM == kRopeChunk || FORM == kRopeDrafts;
    using V = Vec<T, VEC>;
    extern __shared__ float2 table[];  // [rows][rot / 2] (cos, sin)
    __shared__ Row rows_s[kRopeThreads];
    __shared__ alignas(16) float w_s[2][128];
    const int tid = threadIdx.x, r0 = blockIdx.x * rows, half = a.rot / 2;
    const int per_row = kSlots / rows;
    const int j = tid % J, slot = tid / J, t = slot / per_row, first = slot % per_row;
    const long long r = r0 + t, per_head = static_cast<long long>(a.L_max) * D;
    const Place at = place_of<VEC>(a, j);
    const int Hqk = a.Hq + a.Hk, heads = Hqk + a.Hv;
    const T* const q = static_cast<const T*>(a.q) + r * a.ld_q;
    const T* const k = static_cast<const T*>(a.k) + r * a.ld_k;
    const T* const v = static_cast<const T*>(a.v) + r * a.ld_v;
    V A[kHeads] = {}, B[kHeads] = {};
    // heads h0, h0 + per_row, ... below `end`
    const auto load = [&](int h0, int end) {
#pragma unroll
        for (int u = 0; u < kHeads; ++u) {
            const int h = h0 + u * per_row;
            if (h >= end) continue;
            const T* const src = h < a.Hq ? q + h * D : h < Hqk ? k + (h - a.Hq) * D : v + (h - Hqk) * D;
            A[u].load(src + at.ea);
            B[u].load(src + at.eb);
        }
    };
    pdl_wait();
    pdl_trigger();
    if (kSmall && r < a.rows) load(first, heads);
    if (tid < rows) rows_s[tid] = locate<FORM>(a, r0 + tid);
    if constexpr (FORM == kRopeChunk)
        if (blockIdx.x == 0 && a.cu_q != nullptr) check_offsets(a);
    fill_weights(n, D, w_s);
    __syncthreads();
    fill_table(a, rows, rows_s, table);
    __syncthreads();
    const Row row = rows_s[t];
    const float inv_d = 1.f / D;
    const auto factors = [&](const float* w, Factors<VEC>& f) {
        float wa[VEC], wb[VEC];
        load_floats(w + at.ea, wa);
        load_floats(w + at.eb, wb);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int m = 2 * e, o = 2 * e + 1;
            const float w1 = kInterleaved && at.turns ? (m < VEC ? wa[m % VEC] : wb[m % VEC]) : wa[e];
            const float w2 = kInterleaved && at.turns ? (o < VEC ? wa[o % VEC] : wb[o % VEC]) : wb[e];
            const float2 x = at.turns && row.ok ? table[t * half + j * VEC + e] : make_float2(1.f, 0.f);
            f.fc[e] = w1 * x.x;
            f.fs[e] = w1 * x.y;
            f.ss[e] = w2 * x.y;
            f.sc[e] = w2 * x.x;
        }
    };
    const auto turn = [&](int u, const Factors<VEC>& f) {  // (all lanes of a warp)
        float x[2 * VEC], scale;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            x[e] = A[u].get(e);
            x[VEC + e] = B[u].get(e);
        }
        const float inv = head_factor<J>(x, inv_d, n.eps, scale);
        float y[VEC], z[VEC];
        if (!at.turns) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                y[e] = x[e] * f.fc[e] * inv;
                z[e] = x[VEC + e] * f.sc[e] * inv;
            }
        } else if (kInterleaved) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float m = x[2 * e], o = x[2 * e + 1];
                const float p = (m * f.fc[e] - o * f.ss[e]) * inv, s = (m * f.fs[e] + o * f.sc[e]) * inv;
                (2 * e < VEC ? y : z)[2 * e % VEC] = p;
                (2 * e < VEC ? y : z)[2 * e % VEC + 1] = s;
            }
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float m = x[e], o = x[VEC + e];
                y[e] = (m * f.fc[e] - o * f.ss[e]) * inv;
                z[e] = (m * f.fs[e] + o * f.sc[e]) * inv;
            }
        }
        A[u].set(y);
        B[u].set(z);
    };
    T* const qo = static_cast<T*>(a.q_out) + r * a.ld_qo;
    T* const ko = static_cast<T*>(a.k_out) + (kToCache ? row.cache : r * a.ld_ko);
    T* const vo = static_cast<T*>(a.v_out) + (kToCache ? row.cache : 0);
    const auto store = [&](int u, int h) {
        const long long apart = kToCache ? per_head : D;
        T* const dst = h < a.Hq ? qo + h * D : h < Hqk ? ko + (h - a.Hq) * apart : vo + (h - Hqk) * apart;
        A[u].store(dst + at.ea);
        B[u].store(dst + at.eb);
    };
    // heads [begin, end) with one set of factors; those from Hqk on (V's) are copied bit for bit
    const auto walk = [&](int begin, int end, const Factors<VEC>& f) {
#pragma unroll 1
        for (int base = begin; base < end; base += kHeads * per_row) {  // alike for every lane of a warp
            const int h0 = base + first;
            if (row.ok) load(h0, end);
#pragma unroll
            for (int u = 0; u < kHeads; ++u) {
                const int h = h0 + u * per_row;
                const V a0 = A[u], b0 = B[u];
                turn(u, f);
                if (begin > 0 && h >= Hqk) {
                    A[u] = a0;
                    B[u] = b0;
                }
                if (row.ok && h < end) store(u, h);
            }
        }
    };
    Factors<VEC> fq;
    factors(w_s[0], fq);
    if constexpr (kSmall) {
        Factors<VEC> fk;
        factors(w_s[1], fk);
#pragma unroll 1
        for (int base = 0; base < heads; base += kHeads * per_row) {
            const int h0 = base + first;
            if (row.ok && base != 0) load(h0, heads);
#pragma unroll
            for (int u = 0; u < kHeads; ++u) {
                const int h = h0 + u * per_row;
                const V a0 = A[u], b0 = B[u];
                Factors<VEC> f;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    f.fc[e] = h < a.Hq ? fq.fc[e] : fk.fc[e];
                    f.fs[e] = h < a.Hq ? fq.fs[e] : fk.fs[e];
                    f.ss[e] = h < a.Hq ? fq.ss[e] : fk.ss[e];
                    f.sc[e] = h < a.Hq ? fq.sc[e] : fk.sc[e];
                }
                turn(u, f);
                if (h >= Hqk) {
                    A[u] = a0;
                    B[u] = b0;
                }
                if (row.ok && h < heads) store(u, h);
            }
        }
    } else {
        walk(0, a.Hq, fq);
        if (a.Hk == 0) return;
        factors(w_s[1], fq);
        walk(a.Hq, heads, fq);
    }
}

// VEC consecutive elements that start on a vector's boundary or anywhere.
template <bool kAligned, typename T, int VEC>
__device__ __forceinline__ void load_elements(const T* p, float (&x)[VEC]) {
    if constexpr (kAligned) {
        Vec<T, VEC> v;
        v.load(p);
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[e] = v.get(e);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            Vec<T, 1> v;
            v.load(p + e);
            x[e] = v.get(0);
        }
    }
}
template <bool kAligned, typename T, int VEC>
__device__ __forceinline__ void store_elements(T* p, const float (&x)[VEC]) {
    if constexpr (kAligned) {
        Vec<T, VEC> v;
        v.set(x);
        v.store(p);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            Vec<T, 1> v;
            const float one[1] = {x[e]};
            v.set(one);
            v.store(p + e);
        }
    }
}

// The partner of each of a lane's VEC elements (by its place in the head; itself where it does not turn), and
// its factors: y = x cos + partner sin.
template <int VEC>
struct Partners {
    int partner[VEC];
    float cs[VEC], sn[VEC];
    __device__ __forceinline__ void find(const RopeArgs& a, int at, const float2* row) {
        const int half = a.rot / 2;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int x = at + e;
            const bool upper = a.interleaved ? (x & 1) != 0 : x >= half;
            const int pair = a.interleaved ? x >> 1 : upper ? x - half : x;
            partner[e] = x >= a.rot ? x : a.interleaved ? x ^ 1 : upper ? x - half : x + half;
            const float2 w = x < a.rot ? row[pair] : make_float2(1.f, 0.f);
            cs[e] = w.x;
            sn[e] = upper ? w.y : -w.y;
        }
    }
};

// The same for rotated parts whose halves do not start on a vector's boundary, and (kAligned false) rows that
// do not: a thread takes one vector of a head, and each element finds its partner in the warp's shared memory.
template <int FORM, typename T, int D, bool kAligned>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_any_kernel(RopeArgs a, NormArgs n, int rows) {
    constexpr int VEC = 16 / sizeof(T), kHeads = 2, J = D / VEC;  // J vectors of a head: 8, 16 or 32 lanes of a warp
    constexpr bool kToCache = FORM == kRopeChunk || FORM == kRopeDrafts;
    extern __shared__ float2 table[];  // [rows][rot / 2] (cos, sin)
    __shared__ Row rows_s[kRopeThreads];
    __shared__ alignas(16) float w_s[2][128];
    __shared__ float side[kHeads][kRopeThreads * VEC];
    const int tid = threadIdx.x, r0 = blockIdx.x * rows, half = a.rot / 2;
    pdl_wait();
    pdl_trigger();
    if (tid < rows) rows_s[tid] = locate<FORM>(a, r0 + tid);
    if constexpr (FORM == kRopeChunk)
        if (blockIdx.x == 0 && a.cu_q != nullptr) check_offsets(a);
    fill_weights(n, a.d, w_s);
    __syncthreads();
    fill_table(a, rows, rows_s, table);
    __syncthreads();
    const int per_row = kRopeThreads / J / rows;  // heads of a row in flight
    const int j = tid % J, slot = tid / J, t = slot / per_row, first = slot % per_row;
    const Row row = rows_s[t];
    const int at = j * VEC;  // the vector's first element
    Partners<VEC> pt;
    pt.find(a, at, table + t * half);
    const long long r = r0 + t, per_head = static_cast<long long>(a.L_max) * a.d;
    const int Hqk = a.Hq + a.Hk, heads = Hqk + a.Hv;
    const float inv_d = 1.f / a.d;
    const T* const q = static_cast<const T*>(a.q) + r * a.ld_q;
    const T* const k = static_cast<const T*>(a.k) + r * a.ld_k;
    const T* const v = static_cast<const T*>(a.v) + r * a.ld_v;
    T* const qo = static_cast<T*>(a.q_out) + r * a.ld_qo;
    T* const ko = static_cast<T*>(a.k_out) + (kToCache ? row.cache : r * a.ld_ko);
    T* const vo = static_cast<T*>(a.v_out) + (kToCache ? row.cache : 0);
    for (int base = 0; base < heads; base += kHeads * per_row) {  // alike for every lane of a warp
        float x[kHeads][VEC];
#pragma unroll
        for (int u = 0; u < kHeads; ++u) {
            const int h = base + first + u * per_row;
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[u][e] = 0.f;
            if (!row.ok || h >= Hqk) continue;
            const bool is_q = h < a.Hq;
            load_elements<kAligned, T, VEC>((is_q ? q : k) + (is_q ? h : h - a.Hq) * D + at, x[u]);
        }
#pragma unroll
        for (int u = 0; u < kHeads; ++u) {
            float w[VEC], scale;
            const float inv = head_factor<J>(x[u], inv_d, n.eps, scale);
            load_floats(w_s[base + first + u * per_row < a.Hq ? 0 : 1] + at, w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[u][e] = x[u][e] * inv * w[e];
        }
        __syncwarp();  // the last heads' partners were read
#pragma unroll
        for (int u = 0; u < kHeads; ++u)
#pragma unroll
            for (int e = 0; e < VEC; ++e) side[u][tid * VEC + e] = x[u][e];
        __syncwarp();
#pragma unroll
        for (int u = 0; u < kHeads; ++u) {
            const int h = base + first + u * per_row;
            if (!row.ok || h >= heads) continue;
            const bool is_q = h < a.Hq, is_k = h < Hqk;
            T* dst = is_q ? qo : is_k ? ko : vo;
            dst += (is_q ? h : is_k ? h - a.Hq : h - Hqk) * (kToCache && !is_q ? per_head : a.d);
            if (!is_k) {  // bit for bit
                const T* const src = v + (h - Hqk) * a.d + at;
                if constexpr (kAligned) {
                    Vec<T, VEC> m;
                    m.load(src);
                    m.store(dst + at);
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        Vec<T, 1> m;
                        m.load(src + e);
                        m.store(dst + at + e);
                    }
                }
                continue;
            }
            const float* const head = &side[u][(tid - j) * VEC];
            float y[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) y[e] = x[u][e] * pt.cs[e] + head[pt.partner[e]] * pt.sn[e];
            store_elements<kAligned, T, VEC>(dst + at, y);
        }
    }
}

template <int FORM, typename T, int D>
cudaError_t launch_sized(const RopeArgs& a, const NormArgs& n) {
    constexpr int VEC = 16 / sizeof(T);
    const bool aligned = (a.ld_q | a.ld_k | a.ld_v | a.ld_qo | a.ld_ko | a.ld_vo) % VEC == 0;
    if (!aligned || a.rot % (2 * VEC) != 0) {
        const int rows = rows_per_cta(a, kRopeThreads / (D / VEC), 4, 2);
        return launch_kernel(aligned ? norm_rope_any_kernel<FORM, T, D, true> : norm_rope_any_kernel<FORM, T, D, false>,
                             dim3((a.rows - 1) / rows + 1), dim3(kRopeThreads),
                             static_cast<size_t>(rows) * (a.rot / 2) * sizeof(float2), a.stream, true, a, n, rows);
    }
    const int slots = kRopeThreads / (D / (2 * VEC));
    const int rows = rows_per_cta(a, slots, Plan<T>::kRows, Plan<T>::kHeads);
    const int grid = (a.rows - 1) / rows + 1;
    const bool small = grid <= 2 * kSms;
    const auto kern = a.interleaved ? (small ? norm_rope_kernel<FORM, T, D, true, true> : norm_rope_kernel<FORM, T, D, true, false>)
                                    : (small ? norm_rope_kernel<FORM, T, D, false, true> : norm_rope_kernel<FORM, T, D, false, false>);
    return launch_kernel(kern, dim3(grid), dim3(kRopeThreads), static_cast<size_t>(rows) * (a.rot / 2) * sizeof(float2),
                         a.stream, true, a, n, rows);
}
template <int FORM, typename T>
cudaError_t launch(const RopeArgs& a, const NormArgs& n) {
    return a.d == 64 ? launch_sized<FORM, T, 64>(a, n) : launch_sized<FORM, T, 128>(a, n);
}

// ---- backward

constexpr int kBackVec = 4;    // elements of a vector
constexpr int kBackRows = 32;  // rows whose angles are held at once
constexpr int kBackItems = 2;  // heads of a group of lanes, at least
constexpr int kBackBatch = 16;  // rows of a batch, at most
static_assert(kBackBatch <= kBackRows, "");
// Heads that a thread loads together and CTAs per SM, by the rows' type.  (4096 rows and 16384 of fp32: 42.8 and 145
// us; one head and 3 CTAs 45.5 and 160.  4096 of bf16: 31.3; two heads and 2 CTAs 33.9.  Chunks, of bf16 rows, spill
// at 80 registers: 56 to 96 bytes stored a thread; rows alone do not.)
template <typename T>
constexpr int kBackHeadsOf = sizeof(T) == 4 ? 2 : 1;
template <typename T>
constexpr int kBackResidentOf = sizeof(T) == 4 ? 2 : 3;
static_assert(kBackResidentOf<__nv_bfloat16> * kSms <= kNormBackCtas, "");

// CTA c takes an even share of the rows, whose angles lie in shared memory, kBackRows at a time, in batches.  A
// thread keeps one row of a batch and one place of the heads and walks over the heads of q, of K, then of V.  With kPairs a lane has two
// vectors of a head that hold whole pairs (as in the forward kernel); without, one vector, and partners meet in
// shared memory.  A lane sums its part of the weights' gradients over all of its heads; the CTA's sums go to
// n.parts, which norm_rope_weights joins.
template <int FORM, typename Tx, typename Tg, typename To, int D, bool kPairs, bool kAligned, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, kBackResidentOf<Tx>)
    norm_rope_back_kernel(RopeArgs a, NormArgs n, int batch) {
    constexpr bool kFromCache = FORM == kRopeChunkBack;
    constexpr int VEC = kBackVec, E = kPairs ? 2 * VEC : VEC;  // elements of a lane
    constexpr int kBackHeads = kBackHeadsOf<Tx>;
    constexpr int J = D / E, kSlots = kRopeThreads / J;
    extern __shared__ float4 table4[];
    float2* const table = reinterpret_cast<float2*>(table4);  // [kBackRows][rot / 2] (cos, sin)
    __shared__ Row rows_s[kBackRows];
    __shared__ alignas(16) float w_s[2][128];
    __shared__ float side[kPairs ? 1 : kBackHeads][kPairs ? 1 : kRopeThreads * VEC];
    __shared__ float sums[kRopeThreads / 32][2][128];
    const int tid = threadIdx.x, half = a.rot / 2, j = tid % J, slot = tid / J;
    const long long per_head = static_cast<long long>(a.L_max) * D;
    const float inv_d = 1.f / D;
    const Place at = kPairs ? place_of<VEC>(a, j) : Place{true, j * VEC, 0};
    // each row of a batch has a group of lanes at least: without whole pairs a head of 128 leaves 8 groups
    if constexpr (kSlots < kBackBatch) batch = min(batch, kSlots);
    float dw[2][E];
#pragma unroll
    for (int e = 0; e < E; ++e) dw[0][e] = dw[1][e] = 0.f;
    const int begin = static_cast<int>(static_cast<long long>(a.rows) * blockIdx.x / gridDim.x);
    const int end = static_cast<int>(static_cast<long long>(a.rows) * (blockIdx.x + 1) / gridDim.x);
    pdl_wait();
    pdl_trigger();
    if constexpr (kFromCache)
        if (blockIdx.x == 0 && a.cu_q != nullptr) check_offsets(a);
    fill_weights(n, D, w_s);
#pragma unroll 1
    for (int r0 = begin; r0 < end; r0 += batch) {
        const int held = (r0 - begin) % (kBackRows / batch * batch);  // rows of the table before this batch's
        if (held == 0) {
            const int rows = min(kBackRows / batch * batch, end - r0);
            __syncthreads();  // the last table was read
            if (tid < rows) rows_s[tid] = locate<FORM>(a, r0 + tid);
            __syncthreads();
            fill_table(a, rows, rows_s, table);
            __syncthreads();
        }
        const int rows = min(batch, end - r0), per_row = kSlots / rows;
        const int in = slot / per_row, t = held + min(in, rows - 1), first = slot % per_row;
        const Row row = rows_s[t];
        const bool ok = in < rows && row.ok;
        const long long r = r0 + in;
        // (the table holds the opposite angles)
        float cs[2 * VEC];  // (cos, sin) of the lane's pairs
        Partners<VEC> pt;
        if constexpr (kPairs) {
            if (at.turns && ok) load_floats(reinterpret_cast<const float*>(table + t * half + j * VEC), cs);
        } else if (ok) {
            pt.find(a, at.ea, table + t * half);
        }
        // `heads` heads: their gradients and rows from gs and xs on, the results to dst
        const auto walk = [&](int heads, const Tg* gs, long long g_apart, const Tx* xs, To* dst, const float* ws, float (&sum)[E]) {
            float w[E];
            {
                float x[VEC];
                load_floats(ws + at.ea, x);
#pragma unroll
                for (int e = 0; e < VEC; ++e) w[e] = x[e];
                if constexpr (kPairs) {
                    load_floats(ws + at.eb, x);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) w[VEC + e] = x[e];
                }
            }
            // (the next heads' vectors are loaded while these are at work)
            Vec<Tg, VEC> ga[kBackHeads] = {}, gb[kBackHeads] = {};
            Vec<Tx, VEC> xa[kBackHeads] = {}, xb[kBackHeads] = {};
            const auto fetch = [&](int base) {
#pragma unroll
                for (int u = 0; u < kBackHeads; ++u) {
                    const int h = base + u * per_row;
                    if (!kPairs || !ok || h >= heads) continue;
                    ga[u].load(gs + h * g_apart + at.ea);
                    gb[u].load(gs + h * g_apart + at.eb);
                    xa[u].load(xs + h * D + at.ea);
                    xb[u].load(xs + h * D + at.eb);
                }
            };
            fetch(first);
#pragma unroll 1
            for (int base = first; base - first < heads; base += kBackHeads * per_row) {  // alike for every lane
                float g[kBackHeads][E], x[kBackHeads][E];
#pragma unroll
                for (int u = 0; u < kBackHeads; ++u) {
                    const int h = base + u * per_row;
                    const bool there = ok && h < heads;
                    if constexpr (kPairs) {
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            g[u][e] = there ? ga[u].get(e) : 0.f;
                            g[u][VEC + e] = there ? gb[u].get(e) : 0.f;
                            x[u][e] = xa[u].get(e);
                            x[u][VEC + e] = xb[u].get(e);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < E; ++e) g[u][e] = x[u][e] = 0.f;
                        if (!there) continue;
                        load_elements<kAligned, Tg, VEC>(gs + h * g_apart + at.ea, g[u]);
                        load_elements<kAligned, Tx, VEC>(xs + h * D + at.ea, x[u]);
                    }
                }
                fetch(base + kBackHeads * per_row);
                if constexpr (!kPairs) {
                    __syncwarp();  // the last heads' partners were read
#pragma unroll
                    for (int u = 0; u < kBackHeads; ++u)
#pragma unroll
                        for (int e = 0; e < E; ++e) side[u][tid * VEC + e] = g[u][e];
                    __syncwarp();
                }
#pragma unroll
                for (int u = 0; u < kBackHeads; ++u) {
                    const int h = base + u * per_row;
                    // the gradient of the head before it was turned
                    if constexpr (kPairs) {
                        if (at.turns && ok) {
#pragma unroll
                            for (int e = 0; e < VEC; ++e) {
                                float& m = g[u][kInterleaved ? 2 * e : e];
                                float& o = g[u][kInterleaved ? 2 * e + 1 : VEC + e];
                                const float p = m * cs[2 * e] - o * cs[2 * e + 1];
                                o = m * cs[2 * e + 1] + o * cs[2 * e];
                                m = p;
                            }
                        }
                    } else if (ok) {
                        const float* const head = &side[u][(tid - j) * VEC];
#pragma unroll
                        for (int e = 0; e < VEC; ++e) g[u][e] = g[u][e] * pt.cs[e] + head[pt.partner[e]] * pt.sn[e];
                    }
                    float scale, dot = 0.f;
                    const float inv = head_factor<J>(x[u], inv_d, n.eps, scale);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        x[u][e] *= inv;
                        sum[e] = fmaf(g[u][e], x[u][e], sum[e]);  // (0 where there is no head)
                        g[u][e] *= w[e];
                        dot = fmaf(g[u][e], x[u][e], dot);
                    }
                    const float mean = head_sum<J>(dot) * inv_d, r = inv * scale;
                    if (!ok || h >= heads) continue;
#pragma unroll
                    for (int e = 0; e < E; ++e) g[u][e] = r * (g[u][e] - x[u][e] * mean);
                    To* const to = dst + h * D;
                    if constexpr (kPairs) {
                        float p[VEC], s[VEC];
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            p[e] = g[u][e];
                            s[e] = g[u][VEC + e];
                        }
                        store_elements<true, To, VEC>(to + at.ea, p);
                        store_elements<true, To, VEC>(to + at.eb, s);
                    } else {
                        store_elements<kAligned, To, VEC>(to + at.ea, g[u]);
                    }
                }
            }
        };
        walk(a.Hq, static_cast<const Tg*>(a.q) + r * a.ld_q, D, static_cast<const Tx*>(n.xq) + r * n.ld_xq,
             static_cast<To*>(a.q_out) + r * a.ld_qo, w_s[0], dw[0]);
        if (a.Hk > 0)
            walk(a.Hk, static_cast<const Tg*>(a.k) + (kFromCache ? row.cache : r * a.ld_k), kFromCache ? per_head : D,
                 static_cast<const Tx*>(n.xk) + r * n.ld_xk, static_cast<To*>(a.k_out) + r * a.ld_ko, w_s[1], dw[1]);
        if (kFromCache && ok) {
            const Tg* const gs = static_cast<const Tg*>(a.v) + row.cache;
            To* const dst = static_cast<To*>(a.v_out) + r * a.ld_vo;
            for (int h = first; h < a.Hv; h += per_row) {
#pragma unroll
                for (int e0 = 0; e0 < E; e0 += VEC) {
                    const int x = e0 == 0 ? at.ea : at.eb;
                    float g[VEC];
                    load_elements<kAligned, Tg, VEC>(gs + h * per_head + x, g);
                    store_elements<kAligned, To, VEC>(dst + h * D + x, g);
                }
            }
        }
    }
    if (n.parts == nullptr) return;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            float s = dw[which][e];
            for (int o = J; o < 32; o <<= 1) s += __shfl_xor_sync(kAll, s, o);
            if (tid % 32 == j) sums[tid / 32][which][(kPairs && e >= VEC ? at.eb - VEC : at.ea) + e] = s;
        }
    }
    __syncthreads();
    for (int i = tid; i < 2 * a.d; i += kRopeThreads) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kRopeThreads / 32; ++w) s += sums[w][i / a.d][i % a.d];
        n.parts[static_cast<size_t>(blockIdx.x) * 2 * a.d + i] = s;
    }
}

// dq_weight, dk_weight = the CTAs' sums, joined.  A warp's lanes are 32 neighbouring elements.
__global__ void __launch_bounds__(1024) norm_rope_weights(const float* parts, int ctas, int d, float* dq_weight,
                                                          float* dk_weight) {
    __shared__ float s[32][33];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, i = blockIdx.x * 32 + lane;  // d is a multiple of 32
    pdl_wait();
    pdl_trigger();
    float x = 0.f;
#pragma unroll 8
    for (int c = warp; c < ctas; c += 32) x += parts[static_cast<size_t>(c) * 2 * d + i];
    s[warp][lane] = x;
    __syncthreads();
    if (warp != 0) return;
    x = 0.f;
#pragma unroll
    for (int w = 0; w < 32; ++w) x += s[w][lane];
    float* const out = i < d ? dq_weight : dk_weight;
    if (out != nullptr) out[i < d ? i : i - d] = x;
}

template <int FORM, typename Tx, typename Tg, typename To, int D>
cudaError_t launch_back_sized(const RopeArgs& a, const NormArgs& n) {
    // rows of a batch, fewer where a row has many heads.  With whole pairs there are 16 groups of lanes (32 for heads of
    // 64): 5 rows have 3 each.  Without there are 8 (16): 5 rows have 1 each and 3 groups no row, and nothing is
    // loaded ahead there (the chunk of 4096 tokens to bf16 with 18 to 126 rotated elements 65 us, with 128 37).
    const int heads = a.Hq + a.Hk + a.Hv, batch = heads <= 4 ? kBackBatch : heads <= 12 ? 8 : 5;
    // CTAs: all that fit at once, fewer where they would have less than kBackItems heads for each group of lanes
    const long long items = static_cast<long long>(a.rows) * heads, per_cta = kBackItems * kRopeThreads * 2 * kBackVec / D;
    constexpr int kMost = kBackResidentOf<Tx> * kSms;
    const int most = a.rows < kMost ? a.rows : kMost;
    const int grid = items >= most * per_cta ? most : static_cast<int>((items + per_cta - 1) / per_cta);
    const bool aligned = (a.ld_q | a.ld_k | a.ld_v | a.ld_qo | a.ld_ko | a.ld_vo | n.ld_xq | n.ld_xk) % kBackVec == 0;
    const auto kern = !aligned ? norm_rope_back_kernel<FORM, Tx, Tg, To, D, false, false, false>
                      : a.rot % (2 * kBackVec) != 0 ? norm_rope_back_kernel<FORM, Tx, Tg, To, D, false, true, false>
                      : a.interleaved ? norm_rope_back_kernel<FORM, Tx, Tg, To, D, true, true, true>
                                      : norm_rope_back_kernel<FORM, Tx, Tg, To, D, true, true, false>;
    const int per_cta_rows = (a.rows + grid - 1) / grid;
    const size_t smem = static_cast<size_t>(per_cta_rows < kBackRows ? per_cta_rows : kBackRows) * (a.rot / 2) * sizeof(float2);
    cudaError_t e = launch_kernel(kern, dim3(grid), dim3(kRopeThreads), smem, a.stream, true, a, n, batch);
    if (e == cudaSuccess && n.parts != nullptr)
        e = launch_kernel(norm_rope_weights, dim3(2 * D / 32), dim3(1024), 0, a.stream, true, n.parts, grid, D, n.dq_weight,
                          n.dk_weight);
    return e;
}
template <int FORM, typename Tx, typename Tg, typename To>
cudaError_t launch_back(const RopeArgs& a, const NormArgs& n) {
    return a.d == 64 ? launch_back_sized<FORM, Tx, Tg, To, 64>(a, n) : launch_back_sized<FORM, Tx, Tg, To, 128>(a, n);
}

}  // namespace

cudaError_t launch_norm_rope(const RopeArgs& a, const NormArgs& n) {
    using bf16 = __nv_bfloat16;
    switch (a.form) {
        case kRopeRows: return a.in_f32 ? launch<kRopeRows, float>(a, n) : launch<kRopeRows, bf16>(a, n);
        case kRopeChunk: return launch<kRopeChunk, bf16>(a, n);
        default: return launch<kRopeDrafts, bf16>(a, n);
    }
}

cudaError_t launch_norm_rope_back(const RopeArgs& a, const NormArgs& n) {
    using bf16 = __nv_bfloat16;
    if (a.form == kRopeRows)
        return a.in_f32 ? launch_back<kRopeRows, float, float, float>(a, n) : launch_back<kRopeRows, bf16, bf16, bf16>(a, n);
    return a.out_f32 ? launch_back<kRopeChunkBack, bf16, float, float>(a, n)
                     : launch_back<kRopeChunkBack, bf16, float, bf16>(a, n);
}

}  // namespace infllmv2
