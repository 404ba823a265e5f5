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
// Clusters of C CTAs walk the rows, each CTA with a share of a row's vectors. Warp
// roles:
//   warp 8     copies the share into a ring of shared-memory chunks; it runs ahead,
//              into the next row as its chunks become free
//   warp 9     reads the lists for the teacher's normaliser and mass, up to two rows
//              ahead (by the copying warp, lists of 200 held up its copies: 777 rows
//              of 93,001 in 77 us)
//   warps 0-7  mark the list's ids that fall in the share in a bitmap (an id marked
//              twice is a repeated one), sum the share's weights, exchange the sums
//              with the row's other CTAs, and write the gradient from the same
//              chunks, then the listed ids' entries
// The bitmap leaves listed ids out of the unlisted sum instead of subtracting them:
// lists hold nearly all of a peaked row, and 1 - sum q_i would be rounding. The two
// sums have a reference each: under one for both, s was 0 where the unlisted ids lie
// 87 nats below the listed ones, though ln s and their shares of s are ordinary
// numbers. Sums meet as messages between the warps of the cluster (st.async), joined
// in one order; no barrier of the cluster stands between a row and the next. Every
// wait is bounded. One that runs out ends its CTA's roles before the next row but
// one (the others' waits then run out too), and whatever was written till then, the
// cluster's CTAs make all of its rows NaN at the end.
//
// What bounds it: large batches the row's bytes, and the second copy through L2 (4,096
// x 151,936 bf16, lists of 64: 435 us, 5.7 TB/s, 51 percent of the issue slots); a few
// hundred rows the last round of clusters (512 x 202,048 bf16, loss alone: 42; 777 x
// 93,001 f16, lists of 200: 72); few rows the chain from the list to the last store (49 x
// 248,320 f32: 23; 7 x 151,936, loss alone: 6.4 on the GPU, 12 with the host's call).
#include <algorithm>
#include <type_traits>

#include <cuda_runtime.h>

#include "sel_common.cuh"
#include "sel_dtype.cuh"
#include "sel_per_device.h"
#include "sel_plan.h"
#include "sel_tma.cuh"
#include "sel_units.cuh"

using namespace sel;

namespace sel {
namespace {

constexpr uint32_t kNT = 256, kWarps = kNT / 32, kThreads = kNT + 64, kMaxC = 8;
constexpr uint32_t kEntries = SEL_MAX_K / kNT;  // of a list, a thread
constexpr uint32_t kBatch = 4;                  // vectors a thread takes at a time
constexpr uint32_t kChunkVecs = kBatch * kNT, kChunkBytes = 16 * kChunkVecs, kMaxSlots = 6;
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
    uint32_t rows, V, k;
    uint32_t C, share, slots;  // CTAs a row, vectors and chunks a CTA
    bool resident;             // a share's chunks stay until its gradient is written
    float kf, kl;             // log2(e) / T as a sum of two floats
    float inv_t;
};

// Sums of 2^(x kf - m) for unlisted and for listed ids, each under an m of its own, a
// whole number of at least -kHuge, so that sums meet by exact shifts. (x kf is not
// rounded before m is subtracted.)
struct Sums {
    float rest_m, rest, list_m, list;
};

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
    const float m = warp_max(s.rest_m), n = warp_max(s.list_m);
    return {m, warp_sum(s.rest * pow2(s.rest_m - m)), n, warp_sum(s.list * pow2(s.list_m - n))};
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

// What logits are taken relative to, under a largest of `m`: 0 where all are -Inf.
__device__ __forceinline__ float reference(float m) { return m == -INFINITY ? 0.0f : m; }

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
    for (uint32_t j = 0; j < 4; ++j) {
        if constexpr (kN == 4) {
            if (bits >> j & 1) w[j] = NegInf<T>::kWord;
        } else {
            // bits 2 j and 2 j + 1 to the halves of a mask
            const uint32_t m = (bits >> (2 * j) & 1) * 0xFFFFu | (bits >> (2 * j + 1) & 1) * 0xFFFF0000u;
            w[j] = (w[j] & ~m) | (NegInf<T>::kWord & m);
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
};

// log2 of a sum as a whole number, which goes with others, and the logarithm of what
// is between 0.7 and 1.5: that one is rounded to 2^-25, log2(sum) of a flat row would
// be to 2^-20, for every entry alike.
struct Log2 {
    float whole, part;
    Log2() = default;
    __device__ __forceinline__ explicit Log2(float v) {
        int e = static_cast<int>(__float_as_uint(v) >> 23) - 127;
        const bool normal = v >= 1.17549435e-38f && v < INFINITY;
        e = normal ? e : 0;
        const float f = normal ? __uint_as_float((__float_as_uint(v) & 0x007FFFFFu) | 0x3F800000u) : v;  // [1, 2)
        const bool high = f >= 1.41421356f;
        whole = static_cast<float>(e + (normal && high));
        part = log2f(normal && high ? 0.5f * f : f);
    }
};

// What the teacher's list comes to. norm: log2 of its normaliser over its largest
// value `top`; left: r, and `log_left` its logarithm; sum: of p; mass: of p and r (NaN fails
// the row). noise: r is no more than the rounding of the given lse, and is nothing
// where s is too.
struct Teacher {
    float top;
    Log2 norm;
    float left, log_left, sum, mass;
    uint32_t noise, live;
};

// A given lse from here on is a NaN: its own rounding is far more than 1, and the pair
// lh, ll holds log2(e) times it no better.
constexpr float kMaxLse = 1.09951163e12f;  // 2^40
// What is taken for nothing, of p as of s; and what an fp32 lse may be off, itself and
// in the sums that gave it, in units of max(1, |lse|): a list that names every id with
// a probability leaves an r of that size, half of the time above 0.
constexpr float kNothing = 1.17549435e-38f, kNothingLog2 = -126.0f, kLseNoise = 4.76837158e-7f;

// ln of 1 - p, p and 1 - p both at hand.
__device__ __forceinline__ float log_rest(float p, float rest) { return rest > 0.5f ? log1pf(-p) : logf(rest); }

// A build of the tests names a row and a CTA of its cluster whose list's result is not
// handed on, so that waits run out.
#ifdef SEL_TEST_DROP_ROW
__device__ __forceinline__ bool dropped(uint32_t row, uint32_t rank) {
    return row == SEL_TEST_DROP_ROW && rank == SEL_TEST_DROP_RANK;
}
#else
__device__ __forceinline__ bool dropped(uint32_t, uint32_t) { return false; }
#endif

struct Shared {
    alignas(16) float4 table[2][kMaxC * kWarps];  // sums of every warp of the cluster
    float losses[2][kMaxC * kWarps];
    Teacher teacher[2];
    uint64_t full[kMaxSlots], empty[kMaxSlots];
    uint64_t t_full[2], t_empty[2], sums[2], loss[2];
    uint32_t err;      // a wait ran out
    uint32_t stop[2];  // that as one thread saw it before a row's barrier: the same for all
    __device__ __forceinline__ bool failed() const { return *static_cast<const volatile uint32_t*>(&err) != 0; }
};

__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
// Stores into a CTA of the cluster, counted on a barrier there.
__device__ __forceinline__ void send(uint32_t to, uint32_t bar, const Sums& s) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
                 "r"(__float_as_uint(s.rest_m)), "r"(__float_as_uint(s.rest)), "r"(__float_as_uint(s.list_m)),
                 "r"(__float_as_uint(s.list)), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void send(uint32_t to, uint32_t bar, float a) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(to),
                 "r"(__float_as_uint(a)), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(kSuspendNs)
        : "memory");
    return ok != 0;
}
// Waits of which this thread keeps whether it saw the phase end.
__device__ __forceinline__ void wait_cluster(uint64_t* bar, uint32_t parity, volatile uint32_t* err, bool& missed) {
    if (!try_wait_cluster(bar, parity)) {
        bool ok = false;
        for (uint32_t i = 0; !ok && i < kWaitPolls && !*err; ++i) ok = try_wait_cluster(bar, parity);
        if (!ok) {
            *err = 1;
            missed = true;
        }
    }
    __syncwarp();
}
__device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity, volatile uint32_t* err, bool& missed) {
    if (!mbar_try_wait(bar, parity)) {
        bool ok = false;
        for (uint32_t i = 0; !ok && i < kWaitPolls && !*err; ++i) ok = mbar_try_wait(bar, parity);
        if (!ok) {
            *err = 1;
            missed = true;
        }
    }
    __syncwarp();
}
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kNT) : "memory"); }
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// log2 of a listed value's probability; with the teacher's own lse, log2(e) of that
// is lh + ll.
struct LogP {
    float kf, kl, top, lh, ll;
    bool given;
    __device__ __forceinline__ float operator()(float v) const {
        if (v == -INFINITY) return v;
        return given ? fmaf(v, kf, -lh) + fmaf(v, kl, -ll) : fmaf(v - top, kf, -lh) - ll;
    }
    __device__ __forceinline__ LogP(const DistillArgs& a, uint32_t row) {
        kf = a.kf;
        kl = a.kl;
        top = lh = ll = 0.0f;
        given = a.teacher_lse != nullptr;
        if (given) {
            const float l = a.teacher_lse[row];
            lh = l * kLog2E;
            ll = fmaf(l, kLog2E, -lh) + l * 1.9259629911e-8f;  // (log2(e) less its float)
            if (!(fabsf(l) < kMaxLse)) lh = NAN;
        }
    }
};

// By one warp.
__device__ __forceinline__ Teacher read_teacher(const DistillArgs& a, uint32_t row) {
    const uint32_t lane = threadIdx.x & 31;
    const float* vals = a.vals + static_cast<uint64_t>(row) * a.k;
    const uint32_t* ids = a.ids + static_cast<uint64_t>(row) * a.k;
    const LogP log_p(a, row);
    float top = -INFINITY;
    uint32_t named = 0;
    bool nan = false;
#pragma unroll 4
    for (uint32_t i = lane; i < a.k; i += 32) {
        const uint32_t id = ids[i];
        const float v = vals[i];
        if (id >= a.V) continue;
        ++named;
        nan |= !(v < INFINITY);
        top = fmaxf(top, v);
    }
    top = warp_max(top);
    named = __reduce_add_sync(kFull, named);
    nan = __any_sync(kFull, nan);
    FF w{0.0f, 0.0f};
    bool end = false;  // (of a top-k list: nothing follows)
#pragma unroll 4
    for (uint32_t i = lane; i < a.k; i += 32) {
        const uint32_t id = ids[i];
        const float v = vals[i];
        if (id >= a.V) continue;
        const float lp = log_p.given ? log_p(v) : (v - top) * a.kf;
        end |= lp < kNothingLog2;
        w = ff_add(w, FF{exp2f(lp), 0.0f});
    }
    w = ff_warp_sum(w);
    end = __any_sync(kFull, end);
    Teacher t{top, Log2{}, 0.0f, 0.0f, w.hi + w.lo, 1.0f, 0, nan || top > -INFINITY};
    if (log_p.given) {
        t.left = named == a.V ? 0.0f : fmaxf(0.0f, (1.0f - w.hi) - w.lo);
        t.noise = t.left <= kLseNoise * fmaxf(1.0f, fabsf(a.teacher_lse[row]));
        if (t.noise && end) t.left = 0.0f;
        t.log_left = log_rest(t.sum, t.left);
        if (t.left == 0.0f) t.mass = t.sum;
    } else {
        t.norm = Log2(w.hi + w.lo);
    }
    if (nan || isnan(w.hi)) t.mass = NAN;
    return t;
}

// This thread's sums. Vector i's bits of the list are byte i (f32: half a byte).
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
            for (uint32_t u = 0; u < kB; ++u)
                if (listed[u]) q[u].mask(listed[u]);
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

// factor * 2^(x kf - m) for some vectors, to where they go.
template <typename T, bool kAligned, uint32_t kB>
__device__ __forceinline__ void write_vecs(T* to, Vec<T> (&q)[kB], Pair k, Pair r, Pair f) {
#pragma unroll
    for (uint32_t u = 0; u < kB; ++u) {
#pragma unroll
        for (uint32_t j = 0; j < Vec<T>::kPairs; ++j) {
            float e0, e1;
            fma2(q[u].pair(j), k, r).get(e0, e1);
            q[u].set(j, mul2(Pair(ex2_approx(e0), ex2_approx(e1)), f));
        }
        store_vec<T, kAligned>(to + u * kNT * Vec<T>::kN, q[u]);
    }
}

// A place in the ring of chunks.
struct Place {
    uint32_t slot = 0, phase = 0;
    __device__ __forceinline__ void next(uint32_t slots) {
        if (++slot == slots) {
            slot = 0;
            phase ^= 1;
        }
    }
};

// The eight warps that work on the rows.
template <typename T, bool kGrad>
struct Worker {
    const DistillArgs& a;
    Shared& s;
    const unsigned char* ring;
    uint32_t* bitmaps;  // two, of `words` each
    uint32_t words, rank, tid, lane, warp;
    Place at;
    uint32_t messages = 0;  // exchanges so far
    bool missed = false;    // a wait of this thread's ran out: it arms no barrier and hands nothing on

    // The sums of all of the row's warps.
    __device__ __forceinline__ Sums exchange(Sums z) {
        const uint32_t p = messages & 1;
        if (tid == 0 && !missed) expect_tx(&s.sums[p], a.C * kWarps * 16);  // (never twice in a phase)
        z = warp_join(z);
        if (lane < a.C) send(peer_addr(&s.table[p][rank * kWarps + warp], lane), peer_addr(&s.sums[p], lane), z);
        wait_cluster(&s.sums[p], messages >> 1 & 1, &s.err, missed);
        ++messages;
        z = {-INFINITY, 0.0f, -INFINITY, 0.0f};
        for (uint32_t i = lane; i < a.C * kWarps; i += 32) {
            const float4 o = s.table[p][i];
            const float m = fmaxf(z.rest_m, o.x), n = fmaxf(z.list_m, o.z);
            z = {m, z.rest * pow2(z.rest_m - m) + o.y * pow2(o.x - m), n, z.list * pow2(z.list_m - n) + o.w * pow2(o.z - n)};
        }
        return warp_join(z);
    }
    template <uint32_t kB>
    __device__ __forceinline__ void read(uint32_t j, Vec<T> (&q)[kB]) const {
        const auto* src = reinterpret_cast<const uint4*>(ring + at.slot * kChunkBytes) + j;
#pragma unroll
        for (uint32_t u = 0; u < kB; ++u) {
            const uint4 t = src[u * kNT];
            q[u].w[0] = t.x, q[u].w[1] = t.y, q[u].w[2] = t.z, q[u].w[3] = t.w;
        }
    }
    __device__ __forceinline__ void release() {
        __syncwarp();
        if (lane == 0 && !missed) arrive(&s.empty[at.slot]);
        at.next(a.slots);
    }
    __device__ __forceinline__ void await_chunk() { wait(&s.full[at.slot], at.phase, &s.err, missed); }
    // Chunks that nobody reads.
    __device__ __forceinline__ void skip(uint32_t chunks) {
        for (uint32_t c = 0; c < chunks; ++c) {
            await_chunk();
            release();
        }
    }
    // f(j, q): vectors j + 256 u of the share's whole ones, all of a chunk's four or
    // one at a time.
    template <typename F>
    __device__ __forceinline__ void chunk(uint32_t first, uint32_t vecs, F f) const {
        if (first + kChunkVecs <= vecs) {
            Vec<T> q[kBatch];
            read(tid, q);
            f(first + tid, q);
        } else {
            for (uint32_t j = tid; first + j < vecs; j += kNT) {
                Vec<T> q[1];
                read(j, q);
                f(first + j, q);
            }
        }
    }
    __device__ __forceinline__ void zeros(const Share<T>& x, T* out) const {
        const int64_t lo = max(x.base, static_cast<int64_t>(0)), hi = min(x.base + x.span, static_cast<int64_t>(a.V));
        for (int64_t i = lo + tid; i < hi; i += kNT) out[i] = from_f32<T>(0.0f);
    }
    template <bool kAligned>
    __device__ __forceinline__ void write_share(const Share<T>& x, T* out, float m, float factor, uint32_t vecs) {
        const Pair k(a.kf, a.kf), r(-m, -m), f(factor, factor);
        T* to = out + (x.base + static_cast<int64_t>(x.w0) * Vec<T>::kN);
        for (uint32_t first = 0; first < vecs; first += kChunkVecs) {
            if (!a.resident) await_chunk();
            chunk(first, vecs, [&](uint32_t j, auto& q) { write_vecs<T, kAligned>(to + static_cast<uint64_t>(j) * Vec<T>::kN, q, k, r, f); });
            release();
        }
    }
    // The largest unlisted and listed logits and the sums of 2^((x - it) kf), for rows
    // whose logits are too large, or too small, for whole-number references.
    __device__ __forceinline__ Sums slow_sums(const Share<T>& x, const uint32_t* bits, bool twice) {
        const int64_t lo = max(x.base, static_cast<int64_t>(0)), hi = min(x.base + x.span, static_cast<int64_t>(a.V));
        auto listed = [&](int64_t i) {
            const uint32_t off = static_cast<uint32_t>(i - x.base);
            return (bits[off >> 5] >> (off & 31) & 1) != 0;
        };
        Sums z{-INFINITY, 0.0f, -INFINITY, 0.0f};
        for (int64_t i = lo + tid; i < hi; i += kNT) {
            float& m = listed(i) ? z.list_m : z.rest_m;
            m = fmaxf(m, to_f32(x.row[i]));
        }
        z = exchange(z);
        const float rest_ref = reference(z.rest_m), list_ref = reference(z.list_m);
        z.rest = twice ? NAN : 0.0f;
        z.list = 0.0f;
        for (int64_t i = lo + tid; i < hi; i += kNT) {
            const bool of = listed(i);
            const float e = ex2_approx((to_f32(x.row[i]) - (of ? list_ref : rest_ref)) * a.kf);  // (NaN where a largest is +Inf)
            (of ? z.list : z.rest) += e;
        }
        return exchange(z);
    }

    __device__ __forceinline__ void run(uint32_t first_row, uint32_t step) {
        // of the row before: what its loss still needs, and listed entries to write
        uint32_t pending = 0, pending_row = 0, lives = 0;
        float p_rest = 0.0f, p_mass = 0.0f;
        T* p_out = nullptr;
        uint32_t id[kEntries];
        float grads[kEntries];
#pragma unroll
        for (uint32_t e = 0; e < kEntries; ++e) id[e] = SEL_INVALID_ID;
        auto finish = [&] {  // by the first warp of the row's first CTA
            const uint32_t p = (pending - 1) & 1;
            wait_cluster(&s.loss[p], (pending - 1) >> 1 & 1, &s.err, missed);
            float loss = 0.0f;
            for (uint32_t i = lane; i < a.C * kWarps; i += 32) loss += s.losses[p][i];
            loss = warp_sum(loss);
            loss += p_rest;
            if (loss < 0.0f) loss = 0.0f;  // (ln p and ln q are rounded apart; a NaN stays)
            if (lane == 0) a.loss[pending_row] = p_mass == p_mass ? loss : NAN;
        };
        auto scatter = [&] {
            if constexpr (kGrad) {
#pragma unroll
                for (uint32_t e = 0; e < kEntries; ++e) {
                    if (id[e] != SEL_INVALID_ID) p_out[id[e]] = from_f32<T>(grads[e]);
                    id[e] = SEL_INVALID_ID;
                }
            }
        };
        uint32_t n = 0;
        bool stop = false;
        uint32_t list[kEntries];  // the row's ids, on their way since the row before
        auto read_list = [&](uint32_t row) {
#pragma unroll
            for (uint32_t e = 0; e < kEntries; ++e) {
                list[e] = SEL_INVALID_ID;
                if (e * kNT < a.k && tid + e * kNT < a.k && row < a.rows)
                    list[e] = a.ids[static_cast<uint64_t>(row) * a.k + tid + e * kNT];
            }
        };
        read_list(first_row);
        for (uint32_t row = first_row; row < a.rows; row += step, ++n) {
            const Share<T> x(a.x, row * a.ld, a.V, rank, a.share);
            const uint32_t vecs = x.w1 - x.w0, chunks = (vecs + kChunkVecs - 1) / kChunkVecs;
            T* out = kGrad ? static_cast<T*>(a.out) + row * a.ld_out : nullptr;
            const float* vals = a.vals + static_cast<uint64_t>(row) * a.k;
            uint32_t* bits = bitmaps + (n & 1) * words;
            const float grad = kGrad ? a.grad[row] : 0.0f, g = grad * a.inv_t;
            LogP log_p(a, row);
            const int64_t single = x.single();
            const float alone = single >= 0 ? to_f32(x.row[single]) : -INFINITY;

            // The list: this thread's entries that the share holds, marked.
            uint32_t new_id[kEntries];
            float val[kEntries], logit[kEntries];
            bool twice = false;
#pragma unroll
            for (uint32_t e = 0; e < kEntries; ++e) {
                new_id[e] = SEL_INVALID_ID;
                val[e] = logit[e] = -INFINITY;
                if (e * kNT >= a.k) continue;
                const uint32_t at_id = list[e];
                const int64_t off = static_cast<int64_t>(at_id) - x.base;
                if (at_id >= a.V || off < 0 || off >= x.span) continue;
                new_id[e] = at_id;
                val[e] = vals[tid + e * kNT];
                logit[e] = to_f32(x.row[at_id]);
                const uint32_t bit = 1u << (off & 31);
                twice |= (atomicOr(&bits[off >> 5], bit) & bit) != 0;
            }
            read_list(row + step);
            if (stop) return;
            if (tid == 0) *static_cast<volatile uint32_t*>(&s.stop[n & 1]) = s.failed();
            consumers_sync();
            stop = *static_cast<volatile uint32_t*>(&s.stop[n & 1]);  // (looked at before the next barrier)
            // (all of the row before is written, and this row's bitmap is whole)
            scatter();
            wait(&s.t_full[n & 1], n >> 1 & 1, &s.err, missed);
            Teacher t = s.teacher[n & 1];
            __syncwarp();
            if (lane == 0 && !missed) arrive(&s.t_empty[n & 1]);
            if (!t.live) {
                if (n == 0) skip(min(chunks, a.slots));  // (copied before the list was read)
                if (rank == 0 && tid == 0 && a.loss) a.loss[row] = 0.0f;
                if constexpr (kGrad) zeros(x, out);
#pragma unroll
                for (uint32_t e = 0; e < kEntries; ++e)
                    if (new_id[e] != SEL_INVALID_ID) bits[(new_id[e] - x.base) >> 5] = 0;
                continue;
            }

            Summer<T> mine{bits, a.kf, -kHuge, 0.0f};
            const Place begin = at;
            for (uint32_t first = 0; first < vecs; first += kChunkVecs) {
                await_chunk();
                chunk(first, vecs, [&](uint32_t j, auto& q) { mine.add(x.w0 + j, q); });
                if (a.resident) at.next(a.slots);
                else release();
            }
            if (single >= 0) {
                const uint32_t off = static_cast<uint32_t>(single - x.base);
                if (!(bits[off >> 5] >> (off & 31) & 1)) mine.add_one(alone);
            }
            Sums z{mine.m, mine.sum, -kHuge, 0.0f};
#pragma unroll
            for (uint32_t e = 0; e < kEntries; ++e) {
                if (new_id[e] == SEL_INVALID_ID) continue;
                const float m = fmaxf(z.list_m, ceilf(logit[e] * a.kf));
                z.list = z.list * pow2(z.list_m - m) + ex2_approx(fmaf(logit[e], a.kf, -m));
                z.list_m = m;
            }
            if (twice) z.rest = NAN;
            z = exchange(z);
            // (the same in every warp of the cluster)
            // (slow too where r > 0 is shared out among unlisted ids that lie below -kHuge)
            const bool slow = !(fabsf(fmaxf(z.rest_m, z.list_m)) < kHuge) || (t.left != 0.0f && z.rest == 0.0f);
            if (slow) z = slow_sums(x, bits, twice);
            const float top = fmaxf(z.rest_m, z.list_m), rest_ref = reference(z.rest_m);
            auto under = [&](float m) { return slow ? ex2_approx((m - top) * a.kf) : pow2(m - top); };
            const float rest_up = under(z.rest_m);  // a unit of the unlisted sum in the row's
            float total = z.rest * rest_up + z.list * under(z.list_m);
            if (!(total > 0.0f)) total = NAN;  // (every id at -Inf)
            if (t.noise && z.rest * rest_up < kNothing * total) {
                t.left = 0.0f;
                t.mass = t.sum;
            }
            const Log2 log_z(total);
            auto exponent = [&](float v, float ref) { return slow ? (v - ref) * a.kf : fmaf(v, a.kf, -ref); };
            auto log_q = [&](float v) {
                return (slow ? fmaf(v - top, a.kf, -log_z.whole) : fmaf(v, a.kf, -(top + log_z.whole))) - log_z.part;
            };
            log_p.top = t.top;
            if (!log_p.given) {
                log_p.lh = t.norm.whole;
                log_p.ll = t.norm.part;
            }

            // (every warp has read this bitmap; it is marked again two rows on)
#pragma unroll
            for (uint32_t e = 0; e < kEntries; ++e)
                if (new_id[e] != SEL_INVALID_ID) bits[(new_id[e] - x.base) >> 5] = 0;
            float part = 0.0f, far = 0.0f;  // far: of logits that log2(e) / T takes past fp32 (a mask's lowest value)
#pragma unroll
            for (uint32_t e = 0; e < kEntries; ++e) {
                id[e] = new_id[e];
                if (id[e] == SEL_INVALID_ID) continue;
                const float lp = log_p(val[e]), p = exp2f(lp);
                const float lq = log_q(logit[e]);
                if (p != 0.0f) {  // (halves: their difference stays in fp32)
                    if (lq == -INFINITY && logit[e] > -INFINITY) far += (2.0f * (p * a.inv_t)) * ((slow ? 0.5f * top : 0.0f) - 0.5f * logit[e]);
                    else part += p * (lp - lq);
                }
                grads[e] = g * (t.mass * (ex2_approx(exponent(logit[e], top)) / total) - p);
                if (kGrad && grad == 0.0f) id[e] = SEL_INVALID_ID;
            }
            if (a.loss) {
                if (rank == 0 && tid == 0 && !missed) expect_tx(&s.loss[lives & 1], a.C * kWarps * 4);
                if (rank == 0 && warp == 0 && pending) finish();
                part = warp_sum(fmaf(part, kLn2, far));
                if (lane == 0) send(peer_addr(&s.losses[lives & 1][rank * kWarps + warp], 0), peer_addr(&s.loss[lives & 1], 0), part);
            }
            if constexpr (kGrad) {
                p_out = out;
                if (a.resident) at = begin;
                // Unlisted ids: m q_j - r q_j / s is their weight in the unlisted sum times this
                // (left without r, q_j's own factor, one rounding less)
                float f = g * t.mass * (rest_up / total);
                if (t.left != 0.0f) f = z.rest != 0.0f ? g * (t.mass * (z.rest * rest_up / total) - t.left) / z.rest : 0.0f * total;
                if (grad == 0.0f || slow) {
                    skip(chunks);
                    if (slow && grad != 0.0f) {
                        const int64_t lo = max(x.base, static_cast<int64_t>(0)), hi = min(x.base + x.span, static_cast<int64_t>(a.V));
                        for (int64_t i = lo + tid; i < hi; i += kNT) out[i] = from_f32<T>(ex2_approx(exponent(to_f32(x.row[i]), rest_ref)) * f);
                    } else {
                        zeros(x, out);
                    }
                } else {
                    if ((reinterpret_cast<uintptr_t>(out) - reinterpret_cast<uintptr_t>(x.row)) % 16 == 0)
                        write_share<true>(x, out, z.rest_m, f, vecs);
                    else write_share<false>(x, out, z.rest_m, f, vecs);
                    if (single >= 0) out[single] = from_f32<T>(ex2_approx(exponent(alone, z.rest_m)) * f);
                }
            }
            // r (ln r - ln s); ln s where it is small: the references' distance, and the sums
            p_rest = 0.0f;
            if (t.left != 0.0f) {
                const float share = z.rest * rest_up / total;
                const bool most = share > 0.5f;
                const float ln_s = most ? log1pf(-(z.list * under(z.list_m)) / total)
                                        : ((log2f(z.rest) - log_z.part) - log_z.whole) * kLn2;
                p_rest = t.left * (t.log_left - ln_s);
                if (!most) p_rest = fmaf(-(t.left * (slow ? a.inv_t : kLn2)), z.rest_m - top, p_rest);
            }
            p_mass = t.mass;
            pending_row = row;
            ++lives;
            pending = lives;
        }
        if (stop) return;
        consumers_sync();
        scatter();
        if (a.loss && rank == 0 && warp == 0 && pending) finish();
    }
};

template <typename T, bool kGrad>
__global__ void __launch_bounds__(kThreads, 2) distill_kernel(DistillArgs a) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Shared s;
    const uint32_t tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), C = a.C;
    const uint32_t cluster = blockIdx.x / C, rank = blockIdx.x - cluster * C, clusters = gridDim.x / C;
    unsigned char* ring = smem;
    auto* bitmaps = reinterpret_cast<uint32_t*>(smem + a.slots * kChunkBytes);
    const uint32_t words = (a.share * Vec<T>::kN + 31) / 32;
    for (uint32_t i = tid; i < 2 * words; i += kThreads) bitmaps[i] = 0;
    if (tid == 0) {
        for (uint32_t i = 0; i < a.slots; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], kWarps);
        }
        for (uint32_t i = 0; i < 2; ++i) {
            mbar_init(&s.t_full[i], 1);
            mbar_init(&s.t_empty[i], kWarps + 1);
            mbar_init(&s.sums[i], 1);
            mbar_init(&s.loss[i], 1);
        }
        s.err = 0;
    }
    cluster_sync_all();
    pdl_wait();
    pdl_trigger();
    if (warp == kWarps) {
        // what launches before wrote with ordinary stores, the copies read
        asm volatile("fence.proxy.async.global;" ::: "memory");
        Place at;
        uint32_t issued = 0, n = 0;
        bool missed = false;
        for (uint32_t row = cluster; row < a.rows && !missed; row += clusters, ++n) {
            const Share<T> x(a.x, row * a.ld, a.V, rank, a.share);
            const uint32_t vecs = x.w1 - x.w0;
            const auto* src = reinterpret_cast<const unsigned char*>(x.vec + x.w0);
            const uint32_t early = min(vecs, a.slots * kChunkVecs);
            auto copy = [&](uint32_t from, uint32_t to) {
                for (uint32_t first = from; first < to && !missed; first += kChunkVecs) {
                    wait(&s.empty[at.slot], at.phase ^ 1, &s.err, missed);
                    missed = __any_sync(kFull, missed);
                    if (missed) break;
                    if ((tid & 31) == 0)
                        bulk_load(ring + at.slot * kChunkBytes, src + static_cast<uint64_t>(first) * 16,
                                  min(kChunkVecs, vecs - first) * 16, &s.full[at.slot]);
                    ++issued;
                    at.next(a.slots);
                }
            };
            if (n == 0) copy(0, early);  // (before it is known whether the row counts)
            wait(&s.t_full[n & 1], n >> 1 & 1, &s.err, missed);
            missed = __any_sync(kFull, missed);
            if (missed) break;
            const bool live = s.teacher[n & 1].live;
            __syncwarp();
            if ((tid & 31) == 0) arrive(&s.t_empty[n & 1]);
            if (live) copy(n == 0 ? early : 0, vecs);
            if (kGrad && !a.resident && live) copy(0, vecs);  // for the gradient
        }
        // every copy has landed before the CTA may end
        Place last = at;
        for (uint32_t i = 0; i < min(issued, a.slots); ++i) {
            last.phase ^= last.slot == 0;
            last.slot = (last.slot == 0 ? a.slots : last.slot) - 1;
            if (!mbar_wait(&s.full[last.slot], last.phase)) s.err = 1;
        }
        __syncwarp();
    } else if (warp == kWarps + 1) {
        uint32_t n = 0;
        bool missed = false;
        for (uint32_t row = cluster; row < a.rows; row += clusters, ++n) {
            if (n >= 2) wait(&s.t_empty[n & 1], (n >> 1) + 1 & 1, &s.err, missed);
            if (__any_sync(kFull, missed)) break;
            const Teacher t = read_teacher(a, row);
            if ((tid & 31) == 0 && !dropped(row, rank)) {
                s.teacher[n & 1] = t;
                arrive(&s.t_full[n & 1]);
            }
            __syncwarp();
        }
    } else {
        Worker<T, kGrad> w{a, s, ring, bitmaps, words, rank, tid, tid & 31, warp};
        w.run(cluster, clusters);
    }
    __syncwarp();
    if (s.failed() && (tid & 31) < C)
        asm volatile("st.shared::cluster.u32 [%0], 1;" ::"r"(peer_addr(&s.err, tid & 31)) : "memory");
    __syncwarp();
    // (nothing is on its way to this CTA, or from it to one that has ended)
    cluster_sync_all();
    if (s.failed()) {
        for (uint32_t row = cluster; row < a.rows; row += clusters) {
            if (a.loss && rank == 0 && tid == 0) a.loss[row] = NAN;
            if constexpr (kGrad) {
                const Share<T> x(a.x, row * a.ld, a.V, rank, a.share);
                T* out = static_cast<T*>(a.out) + row * a.ld_out;
                const int64_t lo = max(x.base, static_cast<int64_t>(0)), hi = min(x.base + x.span, static_cast<int64_t>(a.V));
                for (int64_t i = lo + tid; i < hi; i += kThreads) out[i] = from_f32<T>(NAN);
            }
        }
    }
}

constexpr size_t kSmem = 110 * 1024;  // a CTA's ring and bitmaps: two CTAs an SM
constexpr uint32_t kMinSlots = 3;
constexpr size_t bitmap_bytes(uint64_t ids) { return 2 * ((ids + 31) / 32 * 4); }
static_assert(bitmap_bytes(SEL_DISTILL_MAX_V / kMaxC + 16) + kMinSlots * kChunkBytes <= kSmem);

struct Layout {
    uint32_t C, share, slots, clusters;
    bool resident;
};

// CTAs a row: what takes least by a model of the rounds of resident clusters. A CTA
// takes 4 us a row and 1 us for 28 KB; shares that do not fit the ring cross it
// twice, the second time out of L2 (as 0.2 of a read from memory), unless the rows
// on the device at a time are too many for it; over several rounds clusters of odd sizes
// take about 1.3 times as long. Measured, 1 / 2 / 3 / 4 / 5 / 6 CTAs a row: 4,096 rows of
// 151,936 bf16 (with 4 a share fits) 541 / 434 / 608 / 502 / 730 / 631 us; 777 of 93,001
// f16 72 / 80 / 104 / 99 / 150 / 120; 49 of 248,320 f32 52 / 34 / 29 / 25 / 23 / 30.
template <typename T, bool kGrad>
bool layout_for(uint32_t rows, uint32_t V, Layout& best) {
    struct Table {
        int clusters[kMaxC + 1];  // resident at a time
    };
    static PerDevice<Table> tables;
    Table t{};
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const bool known = tables.get(dev, t, [](Table& r) {
        for (uint32_t c = 1; c <= kMaxC; ++c) {
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(c);
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = kSmem;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = c;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&r.clusters[c], distill_kernel<T, kGrad>, &cfg) != cudaSuccess) {
                (void)cudaGetLastError();
                return false;
            }
        }
        return true;
    });
    if (!known) return false;
    double least = 1e30;
    for (uint32_t c = 1; c <= kMaxC; ++c) {
        if (t.clusters[c] <= 0) continue;
        const uint32_t share = ceil_div(ceil_div(static_cast<uint64_t>(V) + Vec<T>::kN - 1, Vec<T>::kN), c);
        const size_t bits = bitmap_bytes(static_cast<uint64_t>(share) * Vec<T>::kN);
        if (bits + kMinSlots * kChunkBytes > kSmem) continue;
        const uint32_t slots = std::min(kMaxSlots, static_cast<uint32_t>((kSmem - bits) / kChunkBytes));
        const bool resident = kGrad && ceil_div(share, kChunkVecs) <= slots;
        const bool in_l2 = static_cast<double>(t.clusters[c]) * V * sizeof(T) <= 64e6;
        const double moved = share * 16.0 * (!kGrad ? 1.0 : resident ? 2.0 : in_l2 ? 2.2 : 3.0);
        const uint32_t rounds = ceil_div(rows, static_cast<uint64_t>(t.clusters[c]));
        const double us = rounds * (4.0 + moved / 28e3) * (rounds > 1 && c > 1 && c % 2 == 1 ? 1.3 : 1.0);
        if (us < least) {
            least = us;
            best = {c, share, slots, static_cast<uint32_t>(t.clusters[c]), resident};
        }
    }
    return least < 1e30;
}

template <typename T, bool kGrad>
sel_status launch(const DistillArgs& in, uint32_t rows, cudaStream_t stream) {
    DistillArgs a = in;
    if (!dynamic_smem_once<distill_kernel<T, kGrad>>(kSmem)) return SEL_ECUDA;
    Layout l{};
    if (!layout_for<T, kGrad>(rows, a.V, l)) return SEL_ECUDA;
    a.rows = rows;
    a.C = l.C;
    a.share = l.share;
    a.slots = l.slots;
    a.resident = l.resident;
    const size_t smem = a.slots * static_cast<size_t>(kChunkBytes) + bitmap_bytes(static_cast<uint64_t>(a.share) * Vec<T>::kN);
    return launch_pdl_cluster(distill_kernel<T, kGrad>, dim3(std::min(rows, l.clusters) * a.C), dim3(kThreads), a.C, smem,
                              stream, a) == cudaSuccess
               ? SEL_OK
               : SEL_ECUDA;
}

sel_status check(const void* x, int dtype, uint32_t rows, uint32_t V, uint64_t ld, const float* vals, const uint32_t* ids,
                 uint32_t k, const float* teacher_lse, float T) {
    const uint32_t size = dtype_bytes(dtype);
    if (size == 0 || V == 0 || V > SEL_MAX_V || ld < V || ld > SEL_MAX_LD) return SEL_EINVAL;
    // (below the normal numbers log2(e) / T would be infinite)
    if (!(T >= 1.17549435e-38f) || !(T < INFINITY) || k == 0 || k > V) return SEL_EINVAL;
    if (k > SEL_MAX_K || V > SEL_DISTILL_MAX_V || rows > 0x7fffffffu) return SEL_EUNSUPPORTED;
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
