// rope.cu -- rotary positions of q and K rows: alone, into the caches (and back for the gradient),
// and of draft trees.
//
// Pair i of a head (elements i and rot/2 + i, or 2i and 2i + 1) of the row at position x turns by
// the angle x * theta_i:
//   y_a = s (a cos - b sin),  y_b = s (a sin + b cos)
// and its transpose (the gradient) by the opposite angle; elements past rot are copied.  theta_i
// comes as turns per position in units of 2^-64 (theta_i / 2 pi, fraction only): x times it, modulo
// 2^64, is that many turns' fraction without a rounding for any 32-bit position, so an angle is as good as
// the table, which is made in fp64 (in fp32 the angle of position 10^6 would be off by up to 0.03
// radians).  angle.h takes cosine and sine of it.
//
// What bounds it is memory: every element is read once and written once.  4 prompts of 16384 tokens of
// 32 + 2 + 2 heads of 128, bf16: 176 us, 6.85 TB/s; a decode step of 4 rows: 2.0 us, a launch's latency.
// The launches carry programmatic stream serialisation, so a call's start-up overlaps the tail of the one
// before (0.3 to 0.5 us of a small call).
#include "angle.h"
#include "internal.h"
#include "places.h"

namespace infllmv2 {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kSms = 152;


// W consecutive 4-byte words, moved as one access.
template <int W>
struct alignas(W * 4) Words {
    uint32_t w[W];
};
// VEC consecutive elements of a type, as they lie in memory and as fp32.  Vectors of 16 bytes (8 bytes for
// the bf16 results of fp32 inputs), or single elements.
template <typename T, int VEC>
struct Vec {
    Words<VEC * static_cast<int>(sizeof(T)) / 4> m;
    __device__ __forceinline__ void load(const T* p) { m = *reinterpret_cast<const decltype(m)*>(p); }
    __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<decltype(m)*>(p) = m; }
    __device__ __forceinline__ float get(int e) const {
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(m.w[e]);
        else
            return (e & 1) ? bf16_hi(m.w[e >> 1]) : bf16_lo(m.w[e >> 1]);
    }
    __device__ __forceinline__ void set(const float (&x)[VEC]) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) m.w[e] = __float_as_uint(x[e]);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; e += 2) m.w[e >> 1] = pack_bf16x2(x[e], x[e + 1]);
        }
    }
};
template <>
struct Vec<__nv_bfloat16, 1> {
    uint16_t m;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { m = *reinterpret_cast<const uint16_t*>(p); }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint16_t*>(p) = m; }
    __device__ __forceinline__ float get(int) const { return bf16_lo(m); }
    __device__ __forceinline__ void set(const float (&x)[1]) { m = __bfloat16_as_ushort(__float2bfloat16_rn(x[0])); }
};

template <typename Tin, typename Tout, int VEC>
__device__ __forceinline__ Vec<Tout, VEC> convert(const Vec<Tin, VEC>& x) {
    Vec<Tout, VEC> y;
    if constexpr (sizeof(Tin) == sizeof(Tout)) {
        y.m = x.m;  // a copy keeps every bit
    } else {
        float f[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = x.get(e);
        y.set(f);
    }
    return y;
}

struct Row {
    long long cache;  // element offset of the row's first head in a [B, Hkv, L, d] tensor
    int pos;
    int ok;
};

// Where row r sits: its position, and its row of the caches (or of the draft buffers).
template <int FORM>
__device__ __forceinline__ Row locate(const RopeArgs& a, int r) {
    Row w{0, 0, 0};
    if (r >= a.rows) return w;
    if constexpr (FORM == kRopeRows) {
        w.pos = a.pos[r];
        w.ok = 1;
    } else if constexpr (FORM == kRopeDrafts) {
        const int b = r / a.Tq, i = r % a.Tq, L = a.kv_len[b];
        if (L < 0 || L > (1 << 28)) {  // the committed tokens a cache can hold
            raise_error(a.err, kDevErrIndex);
            return w;
        }
        const int depth = __popcll(a.tree_mask[r]);
        w.pos = L + max(depth, 1) - 1;
        w.cache = (static_cast<long long>(b) * a.Hkv * a.Tq + i) * a.d;
        w.ok = 1;
    } else {
        int b, t, len;
        if (a.cu_q == nullptr) {
            b = r / a.Tq;
            t = r % a.Tq;
            len = a.Tq;
        } else {
            // bad offsets are reported by check_offsets; rows behind the last sequence are left as they are
            const PackedRow p = packed_row(a.cu_q, a.B, r, a.rows, a.Tq);
            if (p.len == 0) return w;
            b = p.b;
            t = p.t;
            len = p.len;
        }
        const int L = a.kv_len[b];
        if (L < len || L > a.L_max) {
            raise_error(a.err, kDevErrIndex);
            return w;
        }
        w.pos = L - len + t;
        w.cache = (static_cast<long long>(b) * a.Hkv * a.L_max + w.pos) * a.d;
        w.ok = 1;
    }
    return w;
}

// Packed offsets that are not ascending from 0 within total_q in steps of at most Tq (one CTA looks).
__device__ __forceinline__ void check_offsets(const RopeArgs& a) {
    bool bad = false;
    for (int b = threadIdx.x; b < a.B; b += kRopeThreads) {
        const long long len = static_cast<long long>(a.cu_q[b + 1]) - a.cu_q[b];
        bad = bad || len < 0 || len > a.Tq;
    }
    if (threadIdx.x == 0) bad = bad || a.cu_q[0] != 0 || a.cu_q[a.B] > a.rows;
    if (bad) raise_error(a.err, kDevErrIndex);
}

// (cos, sin) of every pair of the CTA's T rows, times the scale.
__device__ __forceinline__ void fill_table(const RopeArgs& a, int T, const Row* rows, float2* table) {
    const int half = a.rot / 2, width = 32 - __clz(half - 1);  // 2^width places for the pairs of a row
    for (int i = threadIdx.x; i < T << width; i += kRopeThreads) {
        const int t = i >> width, pair = i & ((1 << width) - 1);
        if (pair >= half) continue;
        const unsigned long long turn =
            a.freqs[pair] * static_cast<unsigned long long>(static_cast<long long>(rows[t].pos));
        float cs, sn;
        cos_sin_of_turn(turn, a.scale, &cs, &sn);
        table[t * half + pair] = make_float2(cs, a.transposed ? -sn : sn);
    }
}

// How a type's rows are spread: heads that a thread loads together, rows that a CTA takes at most, CTAs
// per SM that the registers have to allow.  Measured on 4 x 16384 tokens of 32 + 2 + 2 heads of 128
// (1.21 GB, 180 us at the copy rate) for bf16, us: heads 3, rows 8, 3 CTAs 175; 1, 4, 5: 190; 2, 8, 4:
// 184; 3, 8, 4 (spills): 198; 5, 8, 2: 190.  On the gradient of a 4096-token chunk (113 MB, 16.9 us) for
// fp32: heads 3, rows 4, 4 CTAs 20.3; 1, 4, 5: 23.6; 4, 4, 4: 24.8; 3, 4, 5 (spills): 29.5.
template <typename T>
struct Plan;
template <>
struct Plan<__nv_bfloat16> {
    static constexpr int kHeads = 3, kRows = 8, kResident = 3;
};
template <>
struct Plan<float> {
    static constexpr int kHeads = 3, kRows = 4, kResident = 4;
};

// One CTA takes T rows.  A thread keeps one row and one place j of the heads (two vectors of VEC
// elements) and walks over the heads, so its sines and cosines are loaded once.  kEarly: the first
// heads' loads are under way while the row is located and its angles are computed.
template <int FORM, typename Tin, typename Tout, int VEC, bool kEarly>
__global__ void __launch_bounds__(kRopeThreads, Plan<Tin>::kResident) rope_kernel(RopeArgs a, int T) {
    constexpr int kHeads = Plan<Tin>::kHeads;
    constexpr bool kFromCache = FORM == kRopeChunkBack, kToCache = FORM == kRopeChunk || FORM == kRopeDrafts;
    using VI = Vec<Tin, VEC>;
    using VO = Vec<Tout, VEC>;
    extern __shared__ float2 table[];  // [T][rot / 2] (cos, sin)
    __shared__ Row rows_s[kRopeThreads];
    const int tid = threadIdx.x;
    const int r0 = blockIdx.x * T;
    const int half = a.rot / 2;
    const int J = a.d / (2 * VEC);             // places of a head
    const int per_row = kRopeThreads / J / T;  // heads of a row in flight
    const int j = tid % J, slot = tid / J;
    const int t = slot / per_row;  // < T: T divides the slots
    const long long r = r0 + t, per_head = static_cast<long long>(a.L_max) * a.d;
    const int rt = a.rot / (2 * VEC);
    const bool turns = j < rt;
    int ea, eb;
    if (!turns) {
        ea = a.rot + 2 * (j - rt) * VEC;
        eb = ea + VEC;
    } else if (a.interleaved) {
        ea = 2 * j * VEC;
        eb = ea + VEC;
    } else {
        ea = j * VEC;
        eb = half + ea;
    }
    const int Hqk = a.Hq + a.Hk, heads = Hqk + a.Hv, first = slot % per_row;
    const Tin* const q = static_cast<const Tin*>(a.q) + r * a.ld_q;
    const Tin* k = static_cast<const Tin*>(a.k) + (kFromCache ? 0 : r * a.ld_k);
    const Tin* v = static_cast<const Tin*>(a.v) + (kFromCache ? 0 : r * a.ld_v);
    VI A[kHeads], B[kHeads];
    // heads h0, h0 + per_row, ... below `end`, from `begin` on
    const auto load = [&](int h0, int begin, int end) {
#pragma unroll
        for (int u = 0; u < kHeads; ++u) {
            const int h = h0 + u * per_row;
            if (h < begin || h >= end) continue;
            const bool is_q = h < a.Hq, is_k = h < Hqk;
            const Tin* src = is_q ? q : is_k ? k : v;
            src += (is_q ? h : is_k ? h - a.Hq : h - Hqk) * (kFromCache && !is_q ? per_head : a.d);
            A[u].load(src + ea);
            B[u].load(src + eb);
        }
    };
    pdl_wait();
    pdl_trigger();
    // (a row past the last one has nothing to load; one that turns out bad is only read)
    if (kEarly && r < a.rows) load(first, 0, kFromCache ? a.Hq : heads);
    if (tid < T) rows_s[tid] = locate<FORM>(a, r0 + tid);
    if constexpr (FORM == kRopeChunk || FORM == kRopeChunkBack)
        if (blockIdx.x == 0 && a.cu_q != nullptr) check_offsets(a);
    __syncthreads();
    fill_table(a, T, rows_s, table);
    __syncthreads();
    const Row row = rows_s[t];
    if (!row.ok) return;
    float cs[VEC], sn[VEC];
    if (turns) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float2 w = table[t * half + j * VEC + e];
            cs[e] = w.x;
            sn[e] = w.y;
        }
    }
    if constexpr (kFromCache) {
        k += row.cache;
        v += row.cache;
    }
    Tout* const qo = static_cast<Tout*>(a.q_out) + r * a.ld_qo;
    Tout* const ko = static_cast<Tout*>(a.k_out) + (kToCache ? row.cache : r * a.ld_ko);
    Tout* const vo = static_cast<Tout*>(a.v_out) + (kToCache ? row.cache : r * a.ld_vo);
    for (int h0 = first; h0 < heads; h0 += kHeads * per_row) {
        if (!kEarly || h0 != first) load(h0, 0, heads);
        if (kEarly && kFromCache && h0 == first) load(h0, a.Hq, heads);
#pragma unroll
        for (int u = 0; u < kHeads; ++u) {
            const int h = h0 + u * per_row;
            if (h >= heads) continue;
            const bool is_q = h < a.Hq, is_k = h < Hqk;
            Tout* dst = is_q ? qo : is_k ? ko : vo;
            dst += (is_q ? h : is_k ? h - a.Hq : h - Hqk) * (kToCache && !is_q ? per_head : a.d);
            VO X, Y;
            if (!turns || !is_k) {
                X = convert<Tin, Tout, VEC>(A[u]);
                Y = convert<Tin, Tout, VEC>(B[u]);
            } else {
                float x[VEC], y[VEC];
                if (a.interleaved) {  // pair e is elements 2e, 2e + 1 of A followed by B
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const int i = 2 * e, j2 = 2 * e + 1;
                        const float m = i < VEC ? A[u].get(i % VEC) : B[u].get(i % VEC);
                        const float n = j2 < VEC ? A[u].get(j2 % VEC) : B[u].get(j2 % VEC);
                        const float fm = m * cs[e] - n * sn[e], fn = m * sn[e] + n * cs[e];
                        if (i < VEC) x[i % VEC] = fm; else y[i % VEC] = fm;
                        if (j2 < VEC) x[j2 % VEC] = fn; else y[j2 % VEC] = fn;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float m = A[u].get(e), n = B[u].get(e);
                        x[e] = m * cs[e] - n * sn[e];
                        y[e] = m * sn[e] + n * cs[e];
                    }
                }
                X.set(x);
                Y.set(y);
            }
            X.store(dst + ea);
            Y.store(dst + eb);
        }
    }
}

// The same for rotated parts whose halves do not start on a vector's boundary (and neighbouring pairs
// that end inside one): a thread takes one vector of a head, the heads' vectors are laid side by side in
// the warp's shared memory, and each element finds its partner there.  (All lanes have read a head before
// any writes it, so outputs may be inputs here too.)
template <int FORM, typename Tin, typename Tout>
__global__ void __launch_bounds__(kRopeThreads) rope_any_kernel(RopeArgs a, int T) {
    constexpr int VEC = 16 / sizeof(Tin), kHeads = 2;
    constexpr bool kFromCache = FORM == kRopeChunkBack, kToCache = FORM == kRopeChunk || FORM == kRopeDrafts;
    using VI = Vec<Tin, VEC>;
    using VO = Vec<Tout, VEC>;
    extern __shared__ float2 table[];  // [T][rot / 2] (cos, sin)
    __shared__ Row rows_s[kRopeThreads];
    __shared__ alignas(16) Tin side[kHeads][kRopeThreads * VEC];
    const int tid = threadIdx.x, r0 = blockIdx.x * T, half = a.rot / 2;
    pdl_wait();
    pdl_trigger();
    if (tid < T) rows_s[tid] = locate<FORM>(a, r0 + tid);
    if constexpr (FORM == kRopeChunk || FORM == kRopeChunkBack)
        if (blockIdx.x == 0 && a.cu_q != nullptr) check_offsets(a);
    __syncthreads();
    fill_table(a, T, rows_s, table);
    __syncthreads();
    const int J = a.d / VEC;                   // vectors of a head: 8, 16 or 32 lanes of a warp
    const int per_row = kRopeThreads / J / T;  // heads of a row in flight
    const int j = tid % J, slot = tid / J, t = slot / per_row;
    const Row row = rows_s[t];
    const int at = j * VEC;  // the vector's first element
    // each element's partner (by its place in the head) and factors: y = x cos + partner sin
    int partner[VEC];
    float cs[VEC], sn[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const int x = at + e;
        const bool upper = a.interleaved ? (x & 1) != 0 : x >= half;
        const int pair = a.interleaved ? x >> 1 : upper ? x - half : x;
        partner[e] = x >= a.rot ? x : a.interleaved ? x ^ 1 : upper ? x - half : x + half;
        const float2 w = x < a.rot && row.ok ? table[t * half + pair] : make_float2(1.f, 0.f);
        cs[e] = w.x;
        sn[e] = upper ? w.y : -w.y;
    }
    const long long r = r0 + t, per_head = static_cast<long long>(a.L_max) * a.d;
    const int Hqk = a.Hq + a.Hk, heads = Hqk + a.Hv, first = slot % per_row;
    const Tin* const q = static_cast<const Tin*>(a.q) + r * a.ld_q;
    const Tin* const k = static_cast<const Tin*>(a.k) + (kFromCache ? row.cache : r * a.ld_k);
    const Tin* const v = static_cast<const Tin*>(a.v) + (kFromCache ? row.cache : r * a.ld_v);
    Tout* const qo = static_cast<Tout*>(a.q_out) + r * a.ld_qo;
    Tout* const ko = static_cast<Tout*>(a.k_out) + (kToCache ? row.cache : r * a.ld_ko);
    Tout* const vo = static_cast<Tout*>(a.v_out) + (kToCache ? row.cache : r * a.ld_vo);
    for (int base = 0; base < heads; base += kHeads * per_row) {  // alike for every lane of a warp
        VI A[kHeads];
#pragma unroll
        for (int u = 0; u < kHeads; ++u) {
            const int h = base + first + u * per_row;
            if (!row.ok || h >= heads) continue;
            const bool is_q = h < a.Hq, is_k = h < Hqk;
            const Tin* src = is_q ? q : is_k ? k : v;
            src += (is_q ? h : is_k ? h - a.Hq : h - Hqk) * (kFromCache && !is_q ? per_head : a.d);
            A[u].load(src + at);
        }
        __syncwarp();  // the last heads' partners were read
#pragma unroll
        for (int u = 0; u < kHeads; ++u) A[u].store(&side[u][tid * VEC]);
        __syncwarp();
#pragma unroll
        for (int u = 0; u < kHeads; ++u) {
            const int h = base + first + u * per_row;
            if (!row.ok || h >= heads) continue;
            const bool is_q = h < a.Hq, is_k = h < Hqk;
            Tout* dst = is_q ? qo : is_k ? ko : vo;
            dst += (is_q ? h : is_k ? h - a.Hq : h - Hqk) * (kToCache && !is_q ? per_head : a.d);
            VO Y = convert<Tin, Tout, VEC>(A[u]);
            if (is_k && at < a.rot) {
                const Tin* const head = &side[u][(tid - j) * VEC];
                float y[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    Vec<Tin, 1> o;
                    o.load(head + partner[e]);
                    y[e] = A[u].get(e) * cs[e] + o.get(0) * sn[e];
                }
                VO turned;
                turned.set(y);
                // what lies behind the rotated part stays bit for bit (rot is even: whole words of bf16)
                constexpr int kPerWord = sizeof(Tout) == 4 ? 1 : 2;
#pragma unroll
                for (int w = 0; w < VEC / kPerWord; ++w)
                    if (at + w * kPerWord < a.rot) Y.m.w[w] = turned.m.w[w];
            }
            Y.store(dst + at);
        }
    }
}

// Rows that a CTA takes: up to `most`, more where a row has too few heads to occupy its threads (64K rows
// of 3 heads: 32 rows 28 us, 8 rows 57), fewer where that leaves SMs without work.
int rows_per_cta(const RopeArgs& a, int slots, int most, int heads_at_once) {
    const int heads = a.Hq + a.Hk + a.Hv;
    int T = slots < most ? slots : most;
    while (T < slots && slots / T * heads_at_once > heads) T *= 2;
    while (T > 1 && a.rows < T * 2 * kSms) T /= 2;
    return T;
}

template <int FORM, typename Tin, typename Tout, int VEC>
cudaError_t launch(const RopeArgs& a) {
    const int T = rows_per_cta(a, kRopeThreads / (a.d / (2 * VEC)), Plan<Tin>::kRows, Plan<Tin>::kHeads);
    const int grid = (a.rows - 1) / T + 1;
    const size_t smem = static_cast<size_t>(T) * (a.rot / 2) * sizeof(float2);
    // Loading before the row is located shortens a call of few CTAs (4 rows 2.34 -> 2.03 us, 16 drafts 2.8
    // -> 2.5), and one whose threads load no further heads (64K rows of 3 heads 28.1 -> 26.8), but costs the
    // larger ones, where other CTAs fill the wait (16384-token prompts 175 -> 198 us).
    const int per_row = kRopeThreads / (a.d / (2 * VEC)) / T;
    const bool early = grid <= 2 * kSms || a.Hq + a.Hk + a.Hv <= Plan<Tin>::kHeads * per_row;
    return launch_kernel(early ? rope_kernel<FORM, Tin, Tout, VEC, true> : rope_kernel<FORM, Tin, Tout, VEC, false>,
                         dim3(grid), dim3(kRopeThreads), smem, a.stream, true, a, T);
}

template <int FORM, typename Tin, typename Tout>
cudaError_t launch_any(const RopeArgs& a) {
    constexpr int VEC = 16 / sizeof(Tin);
    const int T = rows_per_cta(a, kRopeThreads / (a.d / VEC), 4, 2);
    return launch_kernel(rope_any_kernel<FORM, Tin, Tout>, dim3((a.rows - 1) / T + 1), dim3(kRopeThreads),
                         static_cast<size_t>(T) * (a.rot / 2) * sizeof(float2), a.stream, true, a, T);
}

// Vectors of 16 bytes where every row starts on a vector's boundary, else single elements; the pairs
// within two vectors of a thread where both halves of the rotated part start on one as well (packed
// prompts of 36 heads, us: 64 of 128 elements turned 41, 50 of them by rope_any_kernel 53 and by single
// elements 85).
template <int FORM, typename Tin, typename Tout>
cudaError_t launch_vec(const RopeArgs& a) {
    constexpr int VEC = 16 / sizeof(Tin);
    const long long ld = a.ld_q | a.ld_k | a.ld_v | a.ld_qo | a.ld_ko | a.ld_vo;
    if (ld % VEC != 0) return launch<FORM, Tin, Tout, 1>(a);
    return a.rot % (2 * VEC) == 0 ? launch<FORM, Tin, Tout, VEC>(a) : launch_any<FORM, Tin, Tout>(a);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a) {
    using bf16 = __nv_bfloat16;
    switch (a.form) {
        case kRopeRows:
            return a.in_f32 ? launch_vec<kRopeRows, float, float>(a) : launch_vec<kRopeRows, bf16, bf16>(a);
        case kRopeChunk: return launch_vec<kRopeChunk, bf16, bf16>(a);
        case kRopeDrafts: return launch_vec<kRopeDrafts, bf16, bf16>(a);
        default:
            return a.out_f32 ? launch_vec<kRopeChunkBack, float, float>(a) : launch_vec<kRopeChunkBack, float, bf16>(a);
    }
}

}  // namespace infllmv2
