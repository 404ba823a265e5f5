// sel_distill.cu -- the divergence of logits rows from a teacher's top logits, and
// its gradient.
//
//   y = x / T, q = softmax(y); p_i = exp(v_i / T - L) on the list's ids,
//   L the list's own ln sum exp or the teacher's given one
//   loss = sum_i p_i (ln p_i - ln q_i) [+ r ln(r / s)], r = 1 - sum p the teacher's
//   mass outside the list, s = sum of the unlisted q
//   d loss / d x_j = (m q_j - p_j) / T listed, (m - r / s) q_j / T unlisted,
//   m = sum p + r
//
// One cluster of C CTAs per row, each with a share of its vectors. A CTA marks the
// list's ids that fall in its share in a bitmap (an id marked twice is a repeated
// one), so that the unlisted sum leaves them out instead of subtracting them:
// lists hold nearly all of a peaked row, and 1 - sum q_i would be rounding. The
// shares' sums meet through distributed shared memory, joined in the shares'
// order; then the gradient is written from a second read of the share, which L2
// still holds, and the listed ids' entries after it.
#include <algorithm>
#include <type_traits>

#include <cuda_runtime.h>

#include "sel_common.cuh"
#include "sel_dtype.cuh"
#include "sel_plan.h"
#include "sel_units.cuh"

using namespace sel;

namespace sel {
namespace {

constexpr uint32_t kNT = 256, kWarps = kNT / 32, kMaxC = 8;
constexpr uint32_t kEntries = SEL_MAX_K / kNT;  // of a list, a thread
constexpr uint32_t kBatch = 4;                  // vectors a thread takes at a time
constexpr float kLog2E = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct DistillArgs {
    const void* x;
    const float* vals;
    const uint32_t* ids;
    const float* teacher_lse;
    const float* grad;
    float* loss;
    void* out;
    uint64_t ld, ld_out;
    uint32_t V, k, C, share;  // share: vectors a CTA
    float kf, kl;             // log2(e) / T as a sum of two floats
    float inv_t;
};

// Sums of 2^(x kf - m), m a whole number of at least -kHuge, so that sums meet by
// exact shifts; apart for unlisted and listed ids. (x kf is not rounded before m
// is subtracted.)
struct Sums {
    float m, rest, list;
};

// 2^n for a whole n <= 0; 0 below the normal numbers (and for NaN).
__device__ __forceinline__ float pow2(float n) {
    return n >= -126.0f ? __uint_as_float(static_cast<uint32_t>(static_cast<int>(n) + 127) << 23) : 0.0f;
}

// References from here to kHuge: beyond, the rounding of x kf is no longer small
// next to 1, and a row goes by x - its largest logit instead (slow_sums). Smaller
// ones count as -kHuge: what lies that far below a row's largest weighs nothing.
constexpr float kHuge = 1048576.0f;

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (uint32_t m = 1; m < 32; m <<= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, m));
    return v;
}
// The sum over the warp, the same in every lane.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (uint32_t m = 1; m < 32; m <<= 1) v += __shfl_xor_sync(kFull, v, m);
    return v;
}
__device__ __forceinline__ Sums warp_join(const Sums& s) {
    const float m = warp_max(s.m), f = pow2(s.m - m);
    return {m, warp_sum(s.rest * f), warp_sum(s.list * f)};
}

// Two floats side by side, for the instructions that take pairs.
struct Pair {
    unsigned long long v;
    __device__ __forceinline__ Pair() {}
    __device__ __forceinline__ Pair(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ __forceinline__ void get(float& a, float& b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
};
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

// 16 bytes of a row: kN logits, taken as four pairs of two (f32: two pairs).
template <typename T>
struct Vec {
    static constexpr uint32_t kN = 16 / sizeof(T), kPairs = kN / 2;
    uint32_t w[4];
    __device__ __forceinline__ Pair pair(uint32_t j) const;
    __device__ __forceinline__ void set(uint32_t j, Pair p);
    __device__ __forceinline__ void mask(uint32_t bits);  // -Inf where a bit is set
};
template <typename T>
struct NegInf;
template <>
struct NegInf<float> { static constexpr uint32_t kWord = 0xFF800000u; };
template <>
struct NegInf<__half> { static constexpr uint32_t kWord = 0xFC00FC00u; };
template <>
struct NegInf<__nv_bfloat16> { static constexpr uint32_t kWord = 0xFF80FF80u; };

template <typename T>
__device__ __forceinline__ Pair Vec<T>::pair(uint32_t j) const {
    if constexpr (kN == 4) return Pair(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
    else return Pair(bits_f32<T>(static_cast<uint16_t>(w[j])), bits_f32<T>(static_cast<uint16_t>(w[j] >> 16)));
}
template <>
__device__ __forceinline__ Pair Vec<__nv_bfloat16>::pair(uint32_t j) const {
    return Pair(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
}
template <typename T>
__device__ __forceinline__ void Vec<T>::set(uint32_t j, Pair p) {
    float a, b;
    p.get(a, b);
    if constexpr (kN == 4) {
        w[2 * j] = __float_as_uint(a);
        w[2 * j + 1] = __float_as_uint(b);
    } else if constexpr (std::is_same_v<T, __half>) {
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(b), "f"(a));
    } else {
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(b), "f"(a));
    }
}
template <typename T>
__device__ __forceinline__ void Vec<T>::mask(uint32_t bits) {
#pragma unroll
    for (uint32_t j = 0; j < kN; ++j) {
        if (bits >> j & 1) {
            if constexpr (kN == 4) w[j] = NegInf<T>::kWord;
            else w[j / 2] = j % 2 ? (w[j / 2] & 0xFFFFu) | (NegInf<T>::kWord & 0xFFFF0000u) : (w[j / 2] & 0xFFFF0000u) | (NegInf<T>::kWord & 0xFFFFu);
        }
    }
}
// The largest entry of some vectors (a NaN shows in the sums, not here).
template <typename T, uint32_t kB>
__device__ __forceinline__ float batch_top(const Vec<T> (&q)[kB]) {
    if constexpr (sizeof(T) == 4) {
        float t = -INFINITY;
#pragma unroll
        for (uint32_t u = 0; u < kB; ++u) {
            t = max3f(t, __uint_as_float(q[u].w[0]), __uint_as_float(q[u].w[1]));
            t = max3f(t, __uint_as_float(q[u].w[2]), __uint_as_float(q[u].w[3]));
        }
        return t;
    } else {
        uint32_t t = q[0].w[0];
#pragma unroll
        for (uint32_t i = 1; i < 4 * kB; ++i) {
            if constexpr (std::is_same_v<T, __half>) asm("max.f16x2 %0, %0, %1;" : "+r"(t) : "r"(q[i / 4].w[i % 4]));
            else asm("max.bf16x2 %0, %0, %1;" : "+r"(t) : "r"(q[i / 4].w[i % 4]));
        }
        return fmaxf(bits_f32<T>(static_cast<uint16_t>(t)), bits_f32<T>(static_cast<uint16_t>(t >> 16)));
    }
}

// A CTA's share of a row: vectors that lie whole in the row, aligned, and the
// entries before and after them one by one, at most one a thread.
template <typename T>
struct Share {
    static constexpr uint32_t kN = Vec<T>::kN;
    const T* row;
    const Vec<T>* vec;  // vector 0 holds the ids from `base`
    int64_t base;
    uint32_t span;      // ids from `base` on that the share may hold
    uint32_t w0, w1;    // its whole vectors
    int64_t head, tail; // first ids of the entries beside them
    uint32_t heads, tails;

    __device__ __forceinline__ Share(const void* x, uint64_t at, uint32_t V, uint32_t rank, uint32_t share) {
        row = static_cast<const T*>(x) + at;
        const uint32_t skew = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(T));
        const uint32_t vecs = (V + skew + kN - 1) / kN, v0 = min(vecs, rank * share), v1 = min(vecs, v0 + share);
        base = static_cast<int64_t>(v0) * kN - skew;
        span = (v1 - v0) * kN;
        vec = reinterpret_cast<const Vec<T>*>(row + base);
        const int64_t lo = max(base, static_cast<int64_t>(0)), hi = min(base + span, static_cast<int64_t>(V));
        w0 = base < 0 ? 1 : 0;
        w1 = static_cast<uint32_t>((hi - base) / kN);
        head = lo;
        if (hi <= lo) {
            w0 = w1 = heads = tails = 0;
            tail = lo;
        } else if (w1 <= w0) {
            w0 = w1 = 0;
            heads = static_cast<uint32_t>(hi - lo);
            tail = hi;
            tails = 0;
        } else {
            heads = base < 0 ? static_cast<uint32_t>(base + kN) : 0;
            tail = base + static_cast<int64_t>(w1) * kN;
            tails = static_cast<uint32_t>(hi - tail);
        }
    }
    // The entry beside the vectors that is this thread's, or -1.
    __device__ __forceinline__ int64_t single() const {
        if (threadIdx.x < heads) return head + threadIdx.x;
        return threadIdx.x < heads + tails ? tail + (threadIdx.x - heads) : -1;
    }
    template <uint32_t kB>
    __device__ __forceinline__ void load(uint32_t i0, Vec<T> (&q)[kB]) const {
#pragma unroll
        for (uint32_t u = 0; u < kB; ++u) {
            const uint4 t = *reinterpret_cast<const uint4*>(vec + i0 + u * kNT);
            q[u].w[0] = t.x, q[u].w[1] = t.y, q[u].w[2] = t.z, q[u].w[3] = t.w;
        }
    }
};

struct Shared {
    Sums warps[kWarps];
    float losses[kWarps];
    float teacher[3];        // the list's largest value, log2 of its normaliser, sum p
    Sums table[kMaxC];       // every CTA's sums
    float row_losses[kMaxC];
    uint32_t twice;
};

__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_peer(uint32_t a, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_sync(uint32_t C) {
    if (C > 1) asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    else __syncthreads();
}

// log2 of a listed value's probability. `lh`: log2 of the list's normaliser over its
// largest value `top`; or with the teacher's own lse, log2(e) of it as lh + ll.
struct LogP {
    float kf, kl, top, lh, ll;
    bool given;
    __device__ __forceinline__ float operator()(float v) const {
        if (v == -INFINITY) return v;
        return given ? fmaf(v, kf, -lh) + fmaf(v, kl, -ll) : (v - top) * kf - lh;
    }
};

// This thread's sums over whole vectors and over single entries. Vector i's bits
// of the list are byte i (f32: half a byte).
template <typename T>
struct Summer {
    const uint32_t* bits;
    float kf, m, sum;

    template <uint32_t kB>
    __device__ __forceinline__ void add(uint32_t i0, Vec<T> (&q)[kB]) {
        const auto* marks = reinterpret_cast<const uint8_t*>(bits);
        uint32_t listed[kB], any = 0;
#pragma unroll
        for (uint32_t u = 0; u < kB; ++u) {
            const uint32_t i = i0 + u * kNT;
            listed[u] = Vec<T>::kN == 8 ? marks[i] : marks[i / 2] >> (i % 2 * 4) & 15;
            any |= listed[u];
        }
        if (any) {
#pragma unroll
            for (uint32_t u = 0; u < kB; ++u) q[u].mask(listed[u]);
        }
        const float n = fmaxf(m, ceilf(batch_top(q) * kf));
        sum *= pow2(m - n);
        m = n;
        const Pair k(kf, kf), r(-m, -m);
        Pair s0(0.0f, 0.0f), s1(0.0f, 0.0f);
#pragma unroll
        for (uint32_t u = 0; u < kB; ++u) {
#pragma unroll
            for (uint32_t j = 0; j < Vec<T>::kPairs; ++j) {
                float e0, e1;
                fma2(q[u].pair(j), k, r).get(e0, e1);
                Pair& s = j % 2 ? s1 : s0;
                s = add2(s, Pair(ex2_approx(e0), ex2_approx(e1)));
            }
        }
        float e0, e1;
        add2(s0, s1).get(e0, e1);
        sum += e0 + e1;
    }
    __device__ __forceinline__ void add_one(float v) {
        const float n = fmaxf(m, ceilf(v * kf));
        sum = sum * pow2(m - n) + ex2_approx(fmaf(v, kf, -n));
        m = n;
    }
};

// One number of every CTA of the row, in every CTA. (Its first barrier: the table
// is no longer read.)
__device__ __forceinline__ void exchange(Shared& s, uint32_t rank, uint32_t C, Sums v) {
    cluster_sync(C);
    if (threadIdx.x < C) {
        const uint32_t p = peer_addr(&s.table[rank], threadIdx.x);
        st_peer(p, __float_as_uint(v.m));
        st_peer(p + 4, __float_as_uint(v.rest));
        st_peer(p + 8, __float_as_uint(v.list));
    }
    __syncwarp();
    cluster_sync(C);
}

// The row's largest logit and the sums of 2^((x - it) kf), for rows whose logits are
// too large, or all too small, for whole-number references.
template <typename T>
__device__ __noinline__ Sums slow_sums(Shared& s, const uint32_t* bits, const Share<T>& x, uint32_t V, uint32_t rank,
                                       uint32_t C, float kf) {
    const uint32_t warp = threadIdx.x / 32;
    const int64_t lo = max(x.base, static_cast<int64_t>(0)), hi = min(x.base + x.span, static_cast<int64_t>(V));
    float m = -INFINITY;
    for (int64_t i = lo + threadIdx.x; i < hi; i += kNT) m = fmaxf(m, to_f32(x.row[i]));
    m = warp_max(m);
    __syncthreads();
    if (threadIdx.x % 32 == 0) s.warps[warp].m = m;
    __syncthreads();
    for (uint32_t i = 0; i < kWarps; ++i) m = fmaxf(m, s.warps[i].m);
    exchange(s, rank, C, Sums{m, 0.0f, 0.0f});
    for (uint32_t i = 0; i < C; ++i) m = fmaxf(m, s.table[i].m);
    float rest = 0.0f, list = 0.0f;
    for (int64_t i = lo + threadIdx.x; i < hi; i += kNT) {
        const uint32_t off = static_cast<uint32_t>(i - x.base);
        const float e = ex2_approx((to_f32(x.row[i]) - m) * kf);  // (NaN where the row's largest is infinite)
        if (bits[off >> 5] >> (off & 31) & 1) list += e;
        else rest += e;
    }
    rest = warp_sum(rest);
    list = warp_sum(list);
    if (threadIdx.x % 32 == 0) s.warps[warp] = {m, rest, list};
    __syncthreads();
    rest = list = 0.0f;
    for (uint32_t i = 0; i < kWarps; ++i) rest += s.warps[i].rest, list += s.warps[i].list;
    if (s.twice) rest = NAN;
    exchange(s, rank, C, Sums{m, rest, list});
    rest = list = 0.0f;
    for (uint32_t i = 0; i < C; ++i) rest += s.table[i].rest, list += s.table[i].list;
    return {m, rest, list};
}

template <typename T, bool kAligned>
__device__ __forceinline__ void store_vec(T* to, const Vec<T>& q) {
    if constexpr (kAligned) {
        *reinterpret_cast<uint4*>(to) = make_uint4(q.w[0], q.w[1], q.w[2], q.w[3]);
    } else {
        T t[Vec<T>::kN];
        memcpy(t, q.w, 16);
#pragma unroll
        for (uint32_t j = 0; j < Vec<T>::kN; ++j) to[j] = t[j];
    }
}

// The share's gradient but for the listed ids: factor * 2^(x kf - m), over the loads
// that a first batch already has.
template <typename T, bool kAligned>
__device__ __forceinline__ void write_share(const Share<T>& x, T* out, float kf, float m, float factor) {
    constexpr uint32_t kN = Vec<T>::kN;
    const Pair k(kf, kf), r(-m, -m), f(factor, factor);
    T* to = out + x.base;
    auto write = [&](uint32_t i0, auto& q) {
#pragma unroll
        for (uint32_t u = 0; u < sizeof(q) / 16; ++u) {
#pragma unroll
            for (uint32_t j = 0; j < Vec<T>::kPairs; ++j) {
                float e0, e1;
                fma2(q[u].pair(j), k, r).get(e0, e1);
                q[u].set(j, mul2(Pair(ex2_approx(e0), ex2_approx(e1)), f));
            }
            store_vec<T, kAligned>(to + static_cast<uint64_t>(i0 + u * kNT) * kN, q[u]);
        }
    };
    uint32_t i = x.w0 + threadIdx.x;
    for (; i + (kBatch - 1) * kNT < x.w1; i += kBatch * kNT) {
        Vec<T> q[kBatch];
        x.load(i, q);
        write(i, q);
    }
    for (; i < x.w1; i += kNT) {
        Vec<T> q[1];
        x.load(i, q);
        write(i, q);
    }
}

template <typename T, bool kGrad>
__global__ void __launch_bounds__(kNT, 4) distill_kernel(DistillArgs a) {
    constexpr uint32_t kN = Vec<T>::kN;
    extern __shared__ uint32_t bits[];
    __shared__ Shared s;
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, C = a.C;
    const uint32_t row = blockIdx.x / C, rank = blockIdx.x - row * C;
    const uint32_t words = (a.share * kN + 31) / 32;
    for (uint32_t i = tid; i < words; i += kNT) bits[i] = 0;
    if (tid == 0) s.twice = 0;
    // (a peer's memory is written only once the peer runs)
    if (C > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    pdl_wait();
    pdl_trigger();
    const Share<T> x(a.x, row * a.ld, a.V, rank, a.share);
    const float* vals = a.vals + static_cast<uint64_t>(row) * a.k;
    const uint32_t* ids = a.ids + static_cast<uint64_t>(row) * a.k;
    T* out = kGrad ? static_cast<T*>(a.out) + row * a.ld_out : nullptr;
    auto zeros = [&] {
        const int64_t lo = max(x.base, static_cast<int64_t>(0)), hi = min(x.base + x.span, static_cast<int64_t>(a.V));
        for (int64_t i = lo + tid; i < hi; i += kNT) out[i] = from_f32<T>(0.0f);
    };
    uint32_t i0 = x.w0 + tid;
    const bool ahead = i0 + (kBatch - 1) * kNT < x.w1;
    Vec<T> q[kBatch];
    if (ahead) x.load(i0, q);  // on their way while the list is read
    const int64_t single = x.single();
    const float alone = single >= 0 ? to_f32(x.row[single]) : -INFINITY;
    if (C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    else __syncthreads();

    // The list: entries of this thread that this share holds, marked in the bitmap.
    uint32_t id[kEntries];
    float val[kEntries], at[kEntries];
    bool some = false;
#pragma unroll
    for (uint32_t e = 0; e < kEntries; ++e) {
        const uint32_t i = tid + e * kNT;
        id[e] = SEL_INVALID_ID;
        val[e] = -INFINITY;
        at[e] = -INFINITY;
        if (i >= a.k) continue;
        const uint32_t n = ids[i];
        if (n >= a.V) continue;
        val[e] = vals[i];
        some |= !(val[e] == -INFINITY);
        const int64_t off = static_cast<int64_t>(n) - x.base;
        if (off < 0 || off >= x.span) continue;
        id[e] = n;
        at[e] = to_f32(x.row[n]);
        const uint32_t bit = 1u << (off & 31);
        if (atomicOr(&bits[off >> 5], bit) & bit) s.twice = 1;
    }
    // (the same in every CTA of the row)
    if (!__syncthreads_or(some)) {
        if (rank == 0 && tid == 0 && a.loss) a.loss[row] = 0.0f;
        if constexpr (kGrad) zeros();
        return;
    }

    // The teacher's normaliser and mass, by one warp that has time for it.
    const bool given = a.teacher_lse != nullptr;
    LogP log_p{a.kf, a.kl, 0.0f, 0.0f, 0.0f, given};
    if (given) {
        const float l = a.teacher_lse[row];
        log_p.lh = l * kLog2E;
        log_p.ll = fmaf(l, kLog2E, -log_p.lh) + l * 1.9259629911e-8f;  // (log2(e) less its float)
        if (!(fabsf(l) < INFINITY)) log_p.lh = NAN;
    }
    if (warp == kWarps - 1) {
        float top = -INFINITY;
        uint32_t named = 0;
        bool nan = false;
        for (uint32_t i = lane; i < a.k; i += 32) {
            if (ids[i] >= a.V) continue;
            ++named;
            nan |= !(vals[i] < INFINITY);
            top = fmaxf(top, vals[i]);
        }
        top = warp_max(top);
        named = __reduce_add_sync(kFull, named);
        nan = __any_sync(kFull, nan);
        FF w{0.0f, 0.0f};
        for (uint32_t i = lane; i < a.k; i += 32)
            if (ids[i] < a.V) w = ff_add(w, FF{exp2f(given ? log_p(vals[i]) : (vals[i] - top) * a.kf), 0.0f});
        w = ff_warp_sum(w);
        float left = 0.0f, mass = 1.0f;  // r, and the sum of p and r
        if (given) {
            left = named == a.V ? 0.0f : fmaxf(0.0f, (1.0f - w.hi) - w.lo);
            if (left == 0.0f) mass = w.hi + w.lo;
        }
        if (nan || isnan(w.hi)) mass = NAN;
        if (lane == 0) {
            s.teacher[0] = top;
            s.teacher[1] = given ? left : log2f(w.hi + w.lo);
            s.teacher[2] = mass;
        }
    }

    // This share's sums.
    Summer<T> mine{bits, a.kf, -kHuge, 0.0f};
    if (ahead) {
        while (true) {
            mine.add(i0, q);
            i0 += kBatch * kNT;
            if (i0 + (kBatch - 1) * kNT >= x.w1) break;
            x.load(i0, q);
        }
    }
    for (; i0 < x.w1; i0 += kNT) {
        Vec<T> one[1];
        x.load(i0, one);
        mine.add(i0, one);
    }
    if (single >= 0) {
        const uint32_t off = static_cast<uint32_t>(single - x.base);
        if (!(bits[off >> 5] >> (off & 31) & 1)) mine.add_one(alone);
    }
    Sums z{mine.m, mine.sum, 0.0f};
#pragma unroll
    for (uint32_t e = 0; e < kEntries; ++e) {
        if (id[e] == SEL_INVALID_ID) continue;
        const float n = fmaxf(z.m, ceilf(at[e] * a.kf)), f = pow2(z.m - n);
        z = {n, z.rest * f, z.list * f + ex2_approx(fmaf(at[e], a.kf, -n))};
    }
    z = warp_join(z);
    if (lane == 0) s.warps[warp] = z;
    __syncthreads();
    if (warp == 0) {
        z = warp_join(lane < kWarps ? s.warps[lane] : Sums{-kHuge, 0.0f, 0.0f});
        if (s.twice) z.rest = NAN;
        if (lane < C) {
            const uint32_t p = peer_addr(&s.table[rank], lane);
            st_peer(p, __float_as_uint(z.m));
            st_peer(p + 4, __float_as_uint(z.rest));
            st_peer(p + 8, __float_as_uint(z.list));
        }
    }
    __syncwarp();
    cluster_sync(C);
    z = {-kHuge, 0.0f, 0.0f};
    for (uint32_t i = 0; i < C; ++i) z.m = fmaxf(z.m, s.table[i].m);
    for (uint32_t i = 0; i < C; ++i) {
        const float f = pow2(s.table[i].m - z.m);
        z.rest += s.table[i].rest * f;
        z.list += s.table[i].list * f;
    }
    // (the same in every CTA of the row)
    const bool slow = !(fabsf(z.m) < kHuge);
    if (slow) z = slow_sums(s, bits, x, a.V, rank, C, a.kf);
    const float total = z.rest + z.list, log_z = log2f(total);
    auto exponent = [&](float v) { return slow ? (v - z.m) * a.kf : fmaf(v, a.kf, -z.m); };
    float left = 0.0f;
    const float mass = s.teacher[2];
    log_p.top = s.teacher[0];
    if (given) left = s.teacher[1];
    else log_p.lh = s.teacher[1];

    const float grad = kGrad ? a.grad[row] : 0.0f, g = grad * a.inv_t;
    float part = 0.0f;
#pragma unroll
    for (uint32_t e = 0; e < kEntries; ++e) {
        if (id[e] == SEL_INVALID_ID) continue;
        const float lp = log_p(val[e]), y = exponent(at[e]), p = exp2f(lp);
        if (p != 0.0f) part += p * (lp - (y - log_z));
        if (kGrad) at[e] = g * (mass * (ex2_approx(y) / total) - p);
    }
    part = warp_sum(part);
    if (lane == 0) s.losses[warp] = part;
    __syncthreads();
    if (a.loss && tid == 0) {
        part = 0.0f;
#pragma unroll
        for (uint32_t i = 0; i < kWarps; ++i) part += s.losses[i];
        st_peer(peer_addr(&s.row_losses[rank], 0), __float_as_uint(part));
    }
    if constexpr (kGrad) {
        if (grad == 0.0f) {
            zeros();
        } else {
            const float f = g / total * (left != 0.0f && z.rest != 0.0f ? mass - left * total / z.rest : mass);
            if (slow) {
                const int64_t lo = max(x.base, static_cast<int64_t>(0)), hi = min(x.base + x.span, static_cast<int64_t>(a.V));
                for (int64_t i = lo + tid; i < hi; i += kNT) out[i] = from_f32<T>(ex2_approx(exponent(to_f32(x.row[i]))) * f);
            } else {
                if ((reinterpret_cast<uintptr_t>(out) - reinterpret_cast<uintptr_t>(x.row)) % 16 == 0)
                    write_share<T, true>(x, out, a.kf, z.m, f);
                else write_share<T, false>(x, out, a.kf, z.m, f);
                if (single >= 0) out[single] = from_f32<T>(ex2_approx(exponent(alone)) * f);
            }
            __syncthreads();
#pragma unroll
            for (uint32_t e = 0; e < kEntries; ++e)
                if (id[e] != SEL_INVALID_ID) out[id[e]] = from_f32<T>(at[e]);
        }
    }
    if (!a.loss) return;
    __syncwarp();
    cluster_sync(C);
    if (rank == 0 && tid == 0) {
        float loss = 0.0f;
        for (uint32_t i = 0; i < C; ++i) loss += s.row_losses[i];
        if (left != 0.0f) loss += left * (log2f(left) - (log2f(z.rest) - log_z));
        a.loss[row] = mass == mass ? loss * kLn2 : NAN;
    }
}

// CTAs a row: enough that the device is full with few rows, and that the rows that
// are on the device at a time stay in L2 until their second read.
template <typename T>
uint32_t ctas_for(uint32_t rows, uint32_t V, int sms) {
    const uint64_t row_bytes = static_cast<uint64_t>(V) * sizeof(T), at_a_time = 3ull * sms;
    uint32_t C = 1;
    while (C < kMaxC && V / C > 4096 && (rows * static_cast<uint64_t>(C) < at_a_time || at_a_time / C * row_bytes > (48ull << 20)))
        C *= 2;
    return C;
}

template <typename T, bool kGrad>
sel_status launch(const DistillArgs& in, uint32_t rows, cudaStream_t stream) {
    const int sms = device_sms();
    if (sms <= 0) return SEL_ECUDA;
    DistillArgs a = in;
    a.C = ctas_for<T>(rows, a.V, sms);
    a.share = ceil_div(ceil_div(static_cast<uint64_t>(a.V) + Vec<T>::kN - 1, Vec<T>::kN), a.C);
    // a CTA's bitmap starts on a whole word of its own
    const size_t smem = align_up(static_cast<size_t>(a.share) * Vec<T>::kN / 8 + 4, 16);
    if (static_cast<uint64_t>(rows) * a.C > 0x7fffffffull) return SEL_EUNSUPPORTED;
    if (smem > 160 * 1024) return SEL_EUNSUPPORTED;
    if (smem > 32 * 1024 && !dynamic_smem_once<distill_kernel<T, kGrad>>(160 * 1024)) return SEL_ECUDA;
    return launch_pdl_cluster(distill_kernel<T, kGrad>, dim3(rows * a.C), dim3(kNT), a.C, smem, stream, a) == cudaSuccess
               ? SEL_OK
               : SEL_ECUDA;
}

sel_status check(const void* x, int dtype, uint32_t rows, uint32_t V, uint64_t ld, const float* vals, const uint32_t* ids,
                 uint32_t k, const float* teacher_lse, float T) {
    const uint32_t size = dtype_bytes(dtype);
    if (size == 0 || V == 0 || V > SEL_MAX_V || ld < V || ld > SEL_MAX_LD) return SEL_EINVAL;
    if (!(T > 0.0f) || !(T < INFINITY) || k == 0 || k > V) return SEL_EINVAL;
    if (k > SEL_MAX_K || V > SEL_DISTILL_MAX_V) return SEL_EUNSUPPORTED;
    if (rows == 0) return SEL_OK;
    if (!x || !vals || !ids) return SEL_EINVAL;
    if (misaligned(x, size) || misaligned(vals, 4) || misaligned(ids, 4) || misaligned(teacher_lse, 4)) return SEL_EINVAL;
    return SEL_OK;
}

DistillArgs arguments(const void* x, uint32_t V, uint64_t ld, const float* vals, const uint32_t* ids, uint32_t k,
                      const float* teacher_lse, float T) {
    DistillArgs a{};
    a.x = x;
    a.V = V;
    a.ld = ld;
    a.vals = vals;
    a.ids = ids;
    a.k = k;
    a.teacher_lse = teacher_lse;
    const double kf = 1.4426950408889634074 / static_cast<double>(T);
    a.kf = static_cast<float>(kf);
    a.kl = static_cast<float>(kf - static_cast<double>(a.kf));
    a.inv_t = 1.0f / T;
    return a;
}

template <bool kGrad>
sel_status launch_any(int dtype, const DistillArgs& a, uint32_t rows, cudaStream_t stream) {
    if (dtype == SEL_F32) return launch<float, kGrad>(a, rows, stream);
    if (dtype == SEL_F16) return launch<__half, kGrad>(a, rows, stream);
    return launch<__nv_bfloat16, kGrad>(a, rows, stream);
}

}  // namespace
}  // namespace sel

extern "C" sel_status sel_distill(const void* d_logits, int dtype, uint32_t rows, uint32_t V, uint64_t ld,
                                  const float* d_vals, const uint32_t* d_ids, uint32_t k, const float* d_teacher_lse,
                                  float temperature, float* d_loss, cudaStream_t stream) {
    if (const sel_status s = check(d_logits, dtype, rows, V, ld, d_vals, d_ids, k, d_teacher_lse, temperature); s != SEL_OK)
        return s;
    if (rows == 0) return SEL_OK;
    if (!d_loss || misaligned(d_loss, 4)) return SEL_EINVAL;
    DistillArgs a = arguments(d_logits, V, ld, d_vals, d_ids, k, d_teacher_lse, temperature);
    a.loss = d_loss;
    return launch_any<false>(dtype, a, rows, stream);
}

extern "C" sel_status sel_distill_grad(const void* d_logits, int dtype, uint32_t rows, uint32_t V, uint64_t ld,
                                       const float* d_vals, const uint32_t* d_ids, uint32_t k, const float* d_teacher_lse,
                                       float temperature, const float* d_grad, float* d_loss, void* d_logits_grad,
                                       uint64_t ld_grad, cudaStream_t stream) {
    if (const sel_status s = check(d_logits, dtype, rows, V, ld, d_vals, d_ids, k, d_teacher_lse, temperature); s != SEL_OK)
        return s;
    if (ld_grad < V || ld_grad > SEL_MAX_LD) return SEL_EINVAL;
    if (rows == 0) return SEL_OK;
    if (!d_grad || !d_logits_grad || misaligned(d_grad, 4) || misaligned(d_loss, 4)) return SEL_EINVAL;
    if (misaligned(d_logits_grad, dtype_bytes(dtype))) return SEL_EINVAL;
    if (d_logits_grad == d_logits && ld_grad != ld) return SEL_EINVAL;
    DistillArgs a = arguments(d_logits, V, ld, d_vals, d_ids, k, d_teacher_lse, temperature);
    a.grad = d_grad;
    a.loss = d_loss;
    a.out = d_logits_grad;
    a.ld_out = ld_grad;
    return launch_any<true>(dtype, a, rows, stream);
}
