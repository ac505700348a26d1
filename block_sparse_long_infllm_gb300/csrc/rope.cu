// rope.cu -- rotary positions of q and K rows: alone, into the caches (and back for the gradient),
// and of draft trees.
//
// Pair i of a head (elements i and rot/2 + i, or 2i and 2i + 1) of the row at position x turns by
// the angle x * theta_i:
//   y_a = s (a cos - b sin),  y_b = s (a sin + b cos)
// and its transpose (the gradient) by the opposite angle; elements past rot are copied.  theta_i
// comes as turns per position in units of 2^-64 (theta_i / 2 pi, fraction only): x times it, modulo
// 2^64, is the exact fraction of a turn for any 32-bit position, so a far position loses nothing
// (in fp32 the angle of position 10^6 would be off by up to 0.03 radians).
//
// What bounds it is memory: every element is read once and written once.
#include "internal.h"

namespace infllmv2 {

namespace {

constexpr int kRopeThreads = 256;

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// VEC consecutive elements, moved as one access.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Vec {
    T v[VEC];
};

template <typename Tin, typename Tout, int VEC>
__device__ __forceinline__ Vec<Tout, VEC> convert(const Vec<Tin, VEC>& x) {
    if constexpr (sizeof(Tin) == sizeof(Tout)) {
        return x;  // a copy keeps every bit
    } else {
        Vec<Tout, VEC> y;
#pragma unroll
        for (int e = 0; e < VEC; ++e) y.v[e] = from_f32<Tout>(to_f32(x.v[e]));
        return y;
    }
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
            int lo = 0, hi = a.B;  // the last b with cu[b] <= r
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (a.cu_q[mid] <= r) lo = mid; else hi = mid;
            }
            b = lo;
            t = r - a.cu_q[b];
            len = a.cu_q[b + 1] - a.cu_q[b];
            // a bad length is reported by check_offsets; rows behind the last sequence are left as they are
            if (t < 0 || t >= len || len > a.Tq) return w;
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
        const int len = a.cu_q[b + 1] - a.cu_q[b];
        bad = bad || len < 0 || len > a.Tq;
    }
    if (threadIdx.x == 0) bad = bad || a.cu_q[0] != 0 || a.cu_q[a.B] > a.rows;
    if (bad) raise_error(a.err, kDevErrIndex);
}

// One CTA takes T rows.  A thread keeps one row and one place j of the heads (two vectors of VEC
// elements) and walks over the heads, so its sines and cosines are loaded once.
template <int FORM, typename Tin, typename Tout, int VEC>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs a, int T) {
    extern __shared__ float2 table[];  // [T][rot / 2] (cos, sin)
    __shared__ Row rows_s[kRopeThreads];
    const int tid = threadIdx.x;
    const int r0 = blockIdx.x * T;
    const int half = a.rot / 2;
    if (tid < T) rows_s[tid] = locate<FORM>(a, r0 + tid);
    if constexpr (FORM == kRopeChunk || FORM == kRopeChunkBack)
        if (blockIdx.x == 0 && a.cu_q != nullptr) check_offsets(a);
    __syncthreads();
    for (int i = tid; i < T * half; i += kRopeThreads) {
        const int t = i / half, pair = i % half;
        const unsigned long long turn =
            a.freqs[pair] * static_cast<unsigned long long>(static_cast<long long>(rows_s[t].pos));
        float sn, cs;
        // the top 32 bits as a signed fraction of half a turn
        sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f, &sn, &cs);
        table[i] = make_float2(cs * a.scale, (a.transposed ? -sn : sn) * a.scale);
    }
    __syncthreads();
    const int J = a.d / (2 * VEC);             // places of a head
    const int per_row = kRopeThreads / J / T;  // heads of a row in flight
    const int j = tid % J, slot = tid / J;
    const int t = slot / per_row;
    if (t >= T) return;
    const Row row = rows_s[t];
    if (!row.ok) return;
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
    float cs[VEC], sn[VEC];
    if (turns) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float2 w = table[t * half + j * VEC + e];
            cs[e] = w.x;
            sn[e] = w.y;
        }
    }
    using VI = Vec<Tin, VEC>;
    using VO = Vec<Tout, VEC>;
    const long long r = r0 + t;
    const int heads = a.Hq + a.Hk + a.Hv;
    for (int h = slot % per_row; h < heads; h += per_row) {
        const Tin* src;
        Tout* dst;
        if (h < a.Hq) {
            src = static_cast<const Tin*>(a.q) + r * a.ld_q + h * a.d;
            dst = static_cast<Tout*>(a.q_out) + r * a.ld_qo + h * a.d;
        } else {
            const bool is_k = h < a.Hq + a.Hk;
            const int g = is_k ? h - a.Hq : h - a.Hq - a.Hk;
            const Tin* s = static_cast<const Tin*>(is_k ? a.k : a.v);
            Tout* o = static_cast<Tout*>(is_k ? a.k_out : a.v_out);
            if constexpr (FORM == kRopeChunkBack) {
                src = s + row.cache + static_cast<long long>(g) * a.L_max * a.d;
            } else {
                src = s + r * (is_k ? a.ld_k : a.ld_v) + g * a.d;
            }
            if constexpr (FORM == kRopeChunk || FORM == kRopeDrafts) {
                dst = o + row.cache + static_cast<long long>(g) * a.L_max * a.d;
            } else {
                dst = o + r * (is_k ? a.ld_ko : a.ld_vo) + g * a.d;
            }
        }
        const VI A = *reinterpret_cast<const VI*>(src + ea), B = *reinterpret_cast<const VI*>(src + eb);
        VO X, Y;
        if (!turns || h >= a.Hq + a.Hk) {
            X = convert<Tin, Tout, VEC>(A);
            Y = convert<Tin, Tout, VEC>(B);
        } else if (a.interleaved) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {  // pair e is elements 2e, 2e + 1 of A followed by B
                const int i0 = 2 * e, i1 = 2 * e + 1;
                const float x = to_f32(i0 < VEC ? A.v[i0 % VEC] : B.v[i0 % VEC]);
                const float y = to_f32(i1 < VEC ? A.v[i1 % VEC] : B.v[i1 % VEC]);
                const Tout fx = from_f32<Tout>(x * cs[e] - y * sn[e]), fy = from_f32<Tout>(x * sn[e] + y * cs[e]);
                if (i0 < VEC) X.v[i0 % VEC] = fx; else Y.v[i0 % VEC] = fx;
                if (i1 < VEC) X.v[i1 % VEC] = fy; else Y.v[i1 % VEC] = fy;
            }
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float x = to_f32(A.v[e]), y = to_f32(B.v[e]);
                X.v[e] = from_f32<Tout>(x * cs[e] - y * sn[e]);
                Y.v[e] = from_f32<Tout>(x * sn[e] + y * cs[e]);
            }
        }
        *reinterpret_cast<VO*>(dst + ea) = X;
        *reinterpret_cast<VO*>(dst + eb) = Y;
    }
}

template <int FORM, typename Tin, typename Tout, int VEC>
cudaError_t launch(const RopeArgs& a) {
    const int slots = kRopeThreads / (a.d / (2 * VEC));
    int T = slots < 4 ? slots : 4;  // rows a CTA takes
    if (a.rows < 4 * 152) T = 1;
    const int grid = (a.rows + T - 1) / T;
    rope_kernel<FORM, Tin, Tout, VEC>
        <<<grid, kRopeThreads, static_cast<size_t>(T) * (a.rot / 2) * sizeof(float2), a.stream>>>(a, T);
    return cudaGetLastError();
}

// Vectors of 16 bytes where both halves of the rotated part and every row start on a vector's
// boundary, else single elements.
template <int FORM, typename Tin, typename Tout>
cudaError_t launch_vec(const RopeArgs& a) {
    constexpr int VEC = 16 / sizeof(Tin);
    const long long ld = a.ld_q | a.ld_k | a.ld_v | a.ld_qo | a.ld_ko | a.ld_vo;
    if (a.rot % (2 * VEC) == 0 && ld % VEC == 0) return launch<FORM, Tin, Tout, VEC>(a);
    return launch<FORM, Tin, Tout, 1>(a);
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
