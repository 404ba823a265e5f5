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

#include <cuda_runtime.h>

#include "sel_common.cuh"
#include "sel_dtype.cuh"
#include "sel_plan.h"
#include "sel_units.cuh"

using namespace sel;

namespace sel {
namespace {

constexpr uint32_t kNT = 512, kMaxC = 8;
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

// Sums of 2^(y - m) in base-2 logits, m a whole number, apart for unlisted and
// listed ids.
struct Sums {
    float m;
    FF rest, list;
};

__device__ __forceinline__ float pow2(float n) {
    return n >= -126.0f ? __uint_as_float(static_cast<uint32_t>(static_cast<int>(n) + 127) << 23) : 0.0f;
}
__device__ __forceinline__ FF ff_scale(FF a, float f) { return FF{a.hi * f, a.lo * f}; }  // (f a power of two)
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b) {
    const float m = fmaxf(a.m, b.m), ref = m == -INFINITY ? 0.0f : m;
    const float fa = pow2(a.m - ref), fb = pow2(b.m - ref);
    return {m, ff_add(ff_scale(a.rest, fa), ff_scale(b.rest, fb)), ff_add(ff_scale(a.list, fa), ff_scale(b.list, fb))};
}
__device__ __forceinline__ Sums shfl_xor(const Sums& a, uint32_t m) {
    return {__shfl_xor_sync(kFull, a.m, m), ff_shfl_xor(a.rest, m), ff_shfl_xor(a.list, m)};
}
__device__ __forceinline__ Sums warp_join(Sums s) {
#pragma unroll
    for (uint32_t m = 1; m < 32; m <<= 1) {
        const Sums o = shfl_xor(s, m);
        s = (threadIdx.x & m) == 0 ? join(s, o) : join(o, s);  // in lane order on both sides
    }
    return s;
}

template <typename T>
struct Vec {
    static constexpr uint32_t kN = 16 / sizeof(T);
};

// Entries of a row as aligned 16-byte vectors: vector i holds ids i kN - skew ..
// (those outside the row read as -Inf, without a load).
template <typename T>
struct Row {
    static constexpr uint32_t kN = Vec<T>::kN;
    const T* p;
    uint32_t V, skew, vecs;
    __device__ __forceinline__ Row(const void* base, uint64_t at, uint32_t v) {
        p = static_cast<const T*>(base) + at;
        V = v;
        skew = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) % 16 / sizeof(T));
        vecs = (V + skew + kN - 1) / kN;
    }
    __device__ __forceinline__ uint4 load(uint32_t i) const {
        const int64_t e = static_cast<int64_t>(i) * kN - skew;
        if (e >= 0 && e + kN <= V) return *reinterpret_cast<const uint4*>(p + e);
        T t[kN];
#pragma unroll
        for (uint32_t j = 0; j < kN; ++j) t[j] = e + j >= 0 && e + j < V ? p[e + j] : from_f32<T>(-INFINITY);
        uint4 q;
        memcpy(&q, t, 16);
        return q;
    }
    // f(i, x) for this thread's vectors of [v0, v1), kBatch loads at a time.
    template <uint32_t kBatch, typename F>
    __device__ __forceinline__ void each(uint32_t v0, uint32_t v1, F f) const {
        for (uint32_t i0 = v0 + threadIdx.x; i0 < v1; i0 += kBatch * kNT) {
            uint4 q[kBatch];
#pragma unroll
            for (uint32_t u = 0; u < kBatch; ++u)
                if (i0 + u * kNT < v1) q[u] = load(i0 + u * kNT);
#pragma unroll
            for (uint32_t u = 0; u < kBatch; ++u) {
                if (i0 + u * kNT < v1) {
                    float x[kN];
                    unpack(q[u], x);
                    f(i0 + u * kNT, x);
                }
            }
        }
    }
    static __device__ __forceinline__ void unpack(const uint4& q, float (&x)[kN]) {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) {
            if constexpr (kN == 4) {
                x[j] = __uint_as_float(w[j]);
            } else {
                x[2 * j] = bits_f32<T>(static_cast<uint16_t>(w[j]));
                x[2 * j + 1] = bits_f32<T>(static_cast<uint16_t>(w[j] >> 16));
            }
        }
    }
};

struct Shared {
    float m[kNT / 32];
    FF a[kNT / 32], b[kNT / 32];
    Sums table[kMaxC];  // every CTA's sums
    FF losses[kMaxC];
    uint32_t twice;
};

__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_peer(uint32_t a, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ void cluster_sync(uint32_t C) {
    if (C > 1) asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    else __syncthreads();
}

// Sum over the block, the same in every thread: warps in order.
__device__ __forceinline__ FF block_sum(FF v, FF* sh) {
    v = ff_warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    FF s = sh[0];
#pragma unroll
    for (uint32_t i = 1; i < kNT / 32; ++i) s = ff_add(s, sh[i]);
    return s;
}

template <typename T, bool kGrad>
__global__ void __launch_bounds__(kNT, 2) distill_kernel(DistillArgs a) {
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
    const Row<T> x(a.x, row * a.ld, a.V);
    const uint32_t v0 = min(x.vecs, rank * a.share), v1 = min(x.vecs, v0 + a.share);
    const int64_t base = static_cast<int64_t>(v0) * kN - x.skew;  // the share's first id
    const uint32_t span = (v1 - v0) * kN;
    const float* vals = a.vals + static_cast<uint64_t>(row) * a.k;
    const uint32_t* ids = a.ids + static_cast<uint64_t>(row) * a.k;
    __syncthreads();

    // The list: its ids in this share, and its largest value.
    float top = -INFINITY;
    uint32_t named = 0;
    bool nan = false;
    for (uint32_t i = tid; i < a.k; i += kNT) {
        const uint32_t id = ids[i];
        if (id >= a.V) continue;
        ++named;
        const float v = vals[i];
        nan |= !(v < INFINITY);
        top = fmaxf(top, v);
        const int64_t at = static_cast<int64_t>(id) - base;
        if (at >= 0 && at < span) {
            const uint32_t bit = 1u << (at & 31);
            if (atomicOr(&bits[at >> 5], bit) & bit) s.twice = 1;
        }
    }
    named = __reduce_add_sync(kFull, named);
    nan = __any_sync(kFull, nan);
#pragma unroll
    for (uint32_t m = 16; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, m));
    if (lane == 0) s.m[warp] = nan ? NAN : top, s.a[warp].hi = static_cast<float>(named);
    __syncthreads();
    top = -INFINITY;
    float count = 0.0f;
#pragma unroll
    for (uint32_t i = 0; i < kNT / 32; ++i) {
        nan |= isnan(s.m[i]);
        top = fmaxf(top, s.m[i]);
        count += s.a[i].hi;
    }
    const bool live = nan || top > -INFINITY;
    if (C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    // (the same in every CTA of the row)
    if (!live) {
        if (rank == 0 && tid == 0 && a.loss) a.loss[row] = 0.0f;
        if (kGrad) {
            T* o = static_cast<T*>(a.out) + row * a.ld_out;
            for (int64_t i = base + tid; i < base + span; i += kNT)
                if (i >= 0 && i < a.V) o[i] = from_f32<T>(0.0f);
        }
        return;
    }

    // This share's sums. A thread keeps its own reference.
    float m = -INFINITY, sum = 0.0f;
    x.template each<4>(v0, v1, [&](uint32_t i, float(&v)[kN]) {
        const uint32_t bit = (i - v0) * kN;
        const uint32_t mine = bits[bit >> 5] >> (bit & 31);
        if (mine & ((1u << kN) - 1)) {
#pragma unroll
            for (uint32_t j = 0; j < kN; ++j)
                if (mine >> j & 1) v[j] = -INFINITY;
        }
        float t = v[0];
#pragma unroll
        for (uint32_t j = 1; j < kN; ++j) t = fmaxf(t, v[j]);
        t = ceilf(t * a.kf);
        if (t > m) {
            sum *= pow2(m - t);
            m = t;
        }
        const float ref = m == -INFINITY ? 0.0f : m;
        float e = 0.0f;
#pragma unroll
        for (uint32_t j = 0; j < kN; ++j) e += ex2_approx(fmaf(v[j], a.kf, -ref));
        sum += e;
    });
    Sums z{m, FF{sum, 0.0f}, FF{0.0f, 0.0f}};
    for (uint32_t i = tid; i < a.k; i += kNT) {
        const uint32_t id = ids[i];
        const int64_t at = static_cast<int64_t>(id) - base;
        if (id >= a.V || at < 0 || at >= span) continue;
        const float v = to_f32(x.p[id]), t = ceilf(v * a.kf), ref = t == -INFINITY ? 0.0f : t;
        z = join(z, Sums{t, FF{0.0f, 0.0f}, FF{ex2_approx(fmaf(v, a.kf, -ref)), 0.0f}});
    }
    z = warp_join(z);
    if (lane == 0) s.m[warp] = z.m, s.a[warp] = z.rest, s.b[warp] = z.list;
    __syncthreads();
    z = {s.m[0], s.a[0], s.b[0]};
#pragma unroll
    for (uint32_t i = 1; i < kNT / 32; ++i) z = join(z, Sums{s.m[i], s.a[i], s.b[i]});
    if (s.twice) z.rest.hi = NAN;
    if (C > 1) {
        if (tid < C) {
            const uint32_t p = peer_addr(&s.table[rank], tid);
            st_peer(p, z.m);
            st_peer(p + 4, z.rest.hi);
            st_peer(p + 8, z.rest.lo);
            st_peer(p + 12, z.list.hi);
            st_peer(p + 16, z.list.lo);
        }
        cluster_sync(C);
        z = s.table[0];
        for (uint32_t i = 1; i < C; ++i) z = join(z, s.table[i]);
    }
    const FF Z = ff_add(z.rest, z.list);
    const float log_z = log2f(Z.hi + Z.lo), ref = z.m == -INFINITY ? 0.0f : z.m;

    // The teacher's: a_i = log2 p_i, and their sum.
    float lh, ll;  // log2 of its normaliser
    if (a.teacher_lse) {
        const float l = a.teacher_lse[row];
        lh = l * kLog2E;
        ll = fmaf(l, kLog2E, -lh) + l * 1.9259629911e-8f;  // (log2(e) less its float)
        if (!(fabsf(l) < INFINITY)) lh = NAN;
    } else {
        FF w{0.0f, 0.0f};
        for (uint32_t i = tid; i < a.k; i += kNT)
            if (ids[i] < a.V) w = ff_add(w, FF{exp2f((vals[i] - top) * a.kf), 0.0f});
        w = block_sum(w, s.a);
        lh = log2f(w.hi + w.lo);
        ll = 0.0f;
    }
    auto log_p = [&](float v) {
        if (v == -INFINITY) return v;
        return a.teacher_lse ? fmaf(v, a.kf, -lh) + fmaf(v, a.kl, -ll) : (v - top) * a.kf - lh;
    };
    FF mass{0.0f, 0.0f}, part{0.0f, 0.0f};
    for (uint32_t i = tid; i < a.k; i += kNT) {
        const uint32_t id = ids[i];
        if (id >= a.V) continue;
        const float lp = log_p(vals[i]), p = exp2f(lp);
        mass = ff_add(mass, FF{p, 0.0f});
        const int64_t at = static_cast<int64_t>(id) - base;
        if (at < 0 || at >= span || p == 0.0f) continue;
        const float lq = (fmaf(to_f32(x.p[id]), a.kf, -ref)) - log_z;
        part = ff_add(part, FF{p * (lp - lq), 0.0f});
    }
    mass = block_sum(mass, s.a);
    part = block_sum(part, s.b);
    if (C > 1) {
        if (tid == 0) {
            const uint32_t p = peer_addr(&s.losses[rank], 0);
            st_peer(p, part.hi);
            st_peer(p + 4, part.lo);
        }
        cluster_sync(C);
        if (rank == 0)
            for (uint32_t i = 0; i < C; ++i) part = i == 0 ? s.losses[0] : ff_add(part, s.losses[i]);
    }
    float r = 0.0f, whole = nan ? NAN : 1.0f;
    if (a.teacher_lse) {
        r = count == static_cast<float>(a.V) ? 0.0f : fmaxf(0.0f, (1.0f - mass.hi) - mass.lo);
        if (isnan(mass.hi)) r = NAN;
        if (r == 0.0f) whole = mass.hi + mass.lo;
    }
    const float rest = z.rest.hi + z.rest.lo, total = Z.hi + Z.lo;
    if (rank == 0 && tid == 0 && a.loss) {
        float loss = part.hi + part.lo;
        if (r != 0.0f) loss += r * (log2f(r) - (log2f(rest) - log_z));
        a.loss[row] = loss * kLn2 * whole / whole;  // (NaN for a list with one)
    }
    if constexpr (kGrad) {
        const float g = a.grad[row] * a.inv_t;
        const bool zero = a.grad[row] == 0.0f;
        const float f = zero ? 0.0f : g / total * (r != 0.0f && rest != 0.0f ? whole - r * total / rest : whole);
        T* o = static_cast<T*>(a.out) + row * a.ld_out;
        const bool vec = (reinterpret_cast<uintptr_t>(o) - reinterpret_cast<uintptr_t>(x.p)) % 16 == 0;
        // listed ids' entries are computed before any is written: out may be x
        float mine = 0.0f;
        uint32_t my_id = SEL_INVALID_ID;
        auto listed = [&](uint32_t i, uint32_t& id) {
            id = ids[i];
            const int64_t at = static_cast<int64_t>(id) - base;
            if (id >= a.V || at < 0 || at >= span) {
                id = SEL_INVALID_ID;
                return 0.0f;
            }
            const float q = ex2_approx(fmaf(to_f32(x.p[id]), a.kf, -ref)) / total;
            return zero ? 0.0f : g * (whole * q - exp2f(log_p(vals[i])));
        };
        float more = 0.0f;
        uint32_t more_id = SEL_INVALID_ID;
        if (tid < a.k) mine = listed(tid, my_id);
        if (tid + kNT < a.k) more = listed(tid + kNT, more_id);
        __syncthreads();
        x.template each<4>(v0, v1, [&](uint32_t i, float(&v)[kN]) {
#pragma unroll
            for (uint32_t j = 0; j < kN; ++j) v[j] = zero ? 0.0f : ex2_approx(fmaf(v[j], a.kf, -ref)) * f;
            const int64_t e = static_cast<int64_t>(i) * kN - x.skew;
            if (vec && e >= 0 && e + kN <= a.V) {
                uint4 q;
                uint32_t* w = &q.x;
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j) {
                    if constexpr (kN == 4) {
                        w[j] = __float_as_uint(v[j]);
                    } else {
                        T two[2] = {from_f32<T>(v[2 * j]), from_f32<T>(v[2 * j + 1])};
                        memcpy(&w[j], two, 4);
                    }
                }
                *reinterpret_cast<uint4*>(o + e) = q;
            } else {
#pragma unroll
                for (uint32_t j = 0; j < kN; ++j)
                    if (e + j >= 0 && e + j < a.V) o[e + j] = from_f32<T>(v[j]);
            }
        });
        __syncthreads();
        if (my_id != SEL_INVALID_ID) o[my_id] = from_f32<T>(mine);
        if (more_id != SEL_INVALID_ID) o[more_id] = from_f32<T>(more);
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
