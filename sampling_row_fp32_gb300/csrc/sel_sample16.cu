// sel_sample16.cu -- sampling of 16-bit logits rows with a policy per row.
//
// Order a row's ids by (logit descending, id ascending). Every filter of the
// chain keeps a prefix of that order: top-k the first k ids, top-p the
// shortest prefix whose mass reaches top_p, min-p the ids whose weight
// w = exp((x - max) / T) is at least min_p. The draw is the first id of the
// surviving prefix whose cumulative mass exceeds u times the prefix's mass.
// A 16-bit row holds at most 65,536 distinct logits, so a histogram of the
// 16-bit patterns holds all of it: ranks are integer sums of counts, masses
// are sums of count * w in 64 bits, and the drawn id is the r-th id of one
// pattern.
//
// One cluster of C CTAs per row. Each CTA reads its share of the row once,
// into registers, and counts it into a histogram of 65,536 16-bit counters in
// its shared memory (a share holds fewer than 65,536 ids, so no counter
// overflows). After one cluster barrier every CTA walks the row's non-empty
// bins through distributed shared memory, decides the cut and the draw (all
// CTAs decide the same), and the CTA that holds the drawn rank finds its id
// in its registers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cooperative_groups.h>

#include "sel.h"
#include "sel_common.cuh"
#include "sel_dtype.cuh"
#include "sel_plan.h"
#include "sel_units.cuh"

namespace cg = cooperative_groups;

namespace sel {
namespace {

constexpr int kNT = 1024;
constexpr int kWarps = kNT / 32;
constexpr int kVPT = 8;                     // 16-byte vectors a thread holds
constexpr uint32_t kShareVecs = 8191;       // vectors a CTA takes at most: 65,528 ids
constexpr uint32_t kMaxCluster = 8;
constexpr uint32_t kBins = 65536;
constexpr uint32_t kUnitBins = 8;           // a 16-byte unit of the histogram
constexpr uint32_t kUnits = kBins / kUnitBins;
constexpr uint32_t kWords = kUnits / 32;    // occupancy bitmap
constexpr uint32_t kZeroBin = 0x7FFF;       // +0
constexpr uint32_t kMinusZeroBin = 0x8000;  // -0, counted as +0
static_assert(kShareVecs * 8 < 65536 && kShareVecs <= kNT * kVPT);
static_assert(static_cast<uint64_t>(kMaxCluster) * kShareVecs * 8 >= SEL_SAMPLE16_MAX_V + 7ull);

// Bin of a bit pattern: descending by value, so bin 0 side is the largest.
// (For two patterns packed in a word.)
__device__ __forceinline__ uint32_t bins_of(uint32_t w) {
    const uint32_t pos = (~w >> 15) & 0x00010001u;  // 1 where the sign bit is clear
    return w ^ (pos * 0x7FFFu);
}

template <typename T>
struct Kind;
template <>
struct Kind<__nv_bfloat16> {
    static constexpr uint32_t kInf = 0x7F80;
};
template <>
struct Kind<__half> {
    static constexpr uint32_t kInf = 0x7C00;
};

template <typename T>
__device__ __forceinline__ double bin_value(uint32_t bin) {
    const uint32_t u = bin < 0x8000u ? 0x7FFFu - bin : bin;
    if constexpr (sizeof(T) == 2 && Kind<T>::kInf == 0x7F80) return static_cast<double>(__uint_as_float(u << 16));
    return static_cast<double>(__half2float(__ushort_as_half(static_cast<unsigned short>(u))));
}

struct SampleArgs {
    const void* logits;
    uint64_t ld;
    const float* temperature;
    const uint32_t* top_k;
    const float* top_p;
    const float* min_p;
    const float* uniforms;
    uint32_t* out_ids;
    float* out_probs;
    uint32_t V;
    uint32_t share;  // vectors a CTA takes
};

struct Shared {
    uint32_t hist[kBins / 2];
    uint16_t units[kUnits];  // the row's non-empty units, in bin order
    double incl_m[kNT];
    uint32_t incl_c[kNT];
    uint32_t bits[kWords];
    uint32_t off[kWords];
    double warp_m[kWarps];
    uint32_t warp_c[kWarps];
    uint32_t seg[kVPT * kWarps];
    double d[4];     // broadcast results of the walks
    uint32_t u[8];
};

template <typename T>
__global__ void __launch_bounds__(kNT, 1) sample16_kernel(SampleArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Shared& s = *reinterpret_cast<Shared*>(smem_raw);
    cg::cluster_group cl = cg::this_cluster();
    const uint32_t C = cl.num_blocks(), rank = cl.block_rank();
    const uint32_t row = blockIdx.x / C;
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr uint32_t kPosInf = 0x7FFFu - Kind<T>::kInf;     // this bin and lower: +Inf, NaN
    constexpr uint32_t kNegInf = 0x8000u | Kind<T>::kInf;     // masked; higher bins: NaN
    constexpr uint32_t kFill = kNegInf | (kNegInf << 16);

    uint4* h4 = reinterpret_cast<uint4*>(s.hist);
#pragma unroll
    for (int i = 0; i < static_cast<int>(kUnits / kNT); ++i) h4[i * kNT + tid] = make_uint4(0, 0, 0, 0);
    pdl_wait();

    // The row as 16-byte vectors from the aligned address at or below its
    // start; `skew` ids of the first vector are not the row's. Vectors that
    // reach over either end of the row are read by element.
    const uint16_t* x = static_cast<const uint16_t*>(a.logits) + static_cast<uint64_t>(row) * a.ld;
    const uint32_t skew = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(x) & 15u) / 2u;
    const uint32_t vecs = (a.V + skew + 7u) / 8u;
    const uint32_t lo = rank * a.share, hi = min(vecs, lo + a.share);
    uint4 q[kVPT];
#pragma unroll
    for (int j = 0; j < kVPT; ++j) {
        const uint32_t v = lo + j * kNT + tid;
        q[j] = make_uint4(kFill, kFill, kFill, kFill);
        if (v < hi) {
            const int64_t e0 = static_cast<int64_t>(v) * 8 - skew;
            if (e0 >= 0 && e0 + 8 <= a.V) {
                q[j] = ldg_stream16(x + e0);
            } else {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t e = e0 + 2 * i;
                    const uint32_t b0 = e >= 0 && e < a.V ? x[e] : kNegInf;
                    const uint32_t b1 = e + 1 >= 0 && e + 1 < a.V ? x[e + 1] : kNegInf;
                    w[i] = b0 | (b1 << 16);
                }
                q[j] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
    const float Tf = a.temperature ? a.temperature[row] : 1.0f;
    const uint32_t kk = a.top_k ? a.top_k[row] : 0u;
    const float pf = a.top_p ? a.top_p[row] : 1.0f;
    const float mf = a.min_p ? a.min_p[row] : 0.0f;
    const float uf = a.uniforms[row];
    pdl_trigger();
    __syncthreads();  // the histogram is clear

#pragma unroll
    for (int j = 0; j < kVPT; ++j) {
        uint32_t w[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t d = bins_of(w[i]);
            const uint32_t d0 = d & 0xFFFFu, d1 = d >> 16;
            if (d0 != kNegInf) atomicAdd(&s.hist[d0 >> 1], 1u << (16 * (d0 & 1)));
            if (d1 != kNegInf) atomicAdd(&s.hist[d1 >> 1], 1u << (16 * (d1 & 1)));
            w[i] = d;
        }
        q[j] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncthreads();
    if (tid == 0) {
        // -0 ties with +0: one bin (bins 0x7FFF and 0x8000)
        const uint32_t neg = s.hist[kMinusZeroBin / 2] & 0xFFFFu;
        s.hist[kMinusZeroBin / 2] -= neg;
        s.hist[kZeroBin / 2] += neg << 16;
    }
    __syncthreads();
    // occupancy: bit l of word w is unit 32 w + l
#pragma unroll
    for (int i = 0; i < static_cast<int>(kUnits / kNT); ++i) {
        const uint32_t unit = (warp * (kUnits / kNT) + i) * 32 + lane;
        const uint4 v = h4[unit];
        const uint32_t b = __ballot_sync(kFull, (v.x | v.y | v.z | v.w) != 0);
        if (lane == 0) s.bits[warp * (kUnits / kNT) + i] = b;
    }
    cl.sync();

    // The row's non-empty units, in order.
    uint32_t word = 0, pc = 0;
    if (tid < kWords) {
        for (uint32_t c = 0; c < C; ++c) word |= cl.map_shared_rank(s.bits, c)[tid];
        pc = __popc(word);
        uint32_t in = pc;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t t = __shfl_up_sync(kFull, in, o);
            if (lane >= static_cast<uint32_t>(o)) in += t;
        }
        s.off[tid] = in;
    }
    __syncthreads();
    uint32_t nu = 0;
#pragma unroll
    for (uint32_t w = 0; w < kWords / 32; ++w) nu += s.off[w * 32 + 31];
    if (tid < kWords) {
        uint32_t at = s.off[tid] - pc;
        for (uint32_t w = 0; w < warp; ++w) at += s.off[w * 32 + 31];
        while (word) {
            const int b = __ffs(word) - 1;
            word &= word - 1;
            s.units[at++] = static_cast<uint16_t>(tid * 32 + b);
        }
    }
    __syncthreads();

    // counts of one unit's bins over the cluster
    auto counts = [&](uint32_t unit, uint32_t (&c)[kUnitBins]) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(kUnitBins); ++i) c[i] = 0;
        for (uint32_t r = 0; r < C; ++r) {
            const uint4 v = reinterpret_cast<const uint4*>(cl.map_shared_rank(s.hist, r))[unit];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c[2 * i] += w[i] & 0xFFFFu;
                c[2 * i + 1] += w[i] >> 16;
            }
        }
    };

    // The policy, and the row's validity: a NaN or +Inf logit, nothing
    // unmasked, a uniform or a parameter out of its range.
    bool bad = !(Tf >= 0.0f) || isinf(Tf) || !(pf > 0.0f && pf <= 1.0f) || !(mf >= 0.0f && mf < 1.0f) ||
               !(uf >= 0.0f && uf < 1.0f) || nu == 0;
    double xmax = 0.0;
    if (!bad) {
        uint32_t c[kUnitBins];
        const uint32_t first = s.units[0], last = s.units[nu - 1];
        counts(first, c);
        int f = 0;
        while (c[f] == 0) ++f;  // a listed unit has a count
        xmax = bin_value<T>(first * kUnitBins + f);
        bad = first * kUnitBins + f <= kPosInf;
        counts(last, c);
        int l = kUnitBins - 1;
        while (l > 0 && c[l] == 0) --l;
        bad = bad || last * kUnitBins + l > kNegInf;
    }
    if (bad) {  // the same in every CTA of the cluster
        if (rank == 0 && tid == 0) {
            a.out_ids[row] = SEL_INVALID_ID;
            a.out_probs[row] = __uint_as_float(0x7FC00000u);
        }
        cl.sync();  // no CTA leaves while another reads its histogram
        return;
    }
    const bool greedy = Tf == 0.0f;
    const double Td = greedy ? 1.0 : static_cast<double>(Tf);
    const double minp = mf;
    auto weight = [&](uint32_t bin) { return exp((bin_value<T>(bin) - xmax) / Td); };

    // Counts and masses up to each thread's units, in order.
    const uint32_t per = (nu + kNT - 1) / kNT;
    const uint32_t i0 = min(nu, tid * per), i1 = min(nu, i0 + per);
    uint32_t c_in = 0, n_min = 0;
    double m_in = 0.0;
    for (uint32_t i = i0; i < i1; ++i) {
        uint32_t c[kUnitBins];
        const uint32_t unit = s.units[i];
        counts(unit, c);
#pragma unroll
        for (uint32_t b = 0; b < kUnitBins; ++b) {
            if (c[b]) {
                const double w = weight(unit * kUnitBins + b);
                c_in += c[b];
                m_in += c[b] * w;
                if (w >= minp) n_min += c[b];
            }
        }
    }
    n_min = __reduce_add_sync(kFull, n_min);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t tc = __shfl_up_sync(kFull, c_in, o);
        const double tm = __shfl_up_sync(kFull, m_in, o);
        if (lane >= static_cast<uint32_t>(o)) {
            c_in += tc;
            m_in += tm;
        }
    }
    if (lane == 31) {
        s.warp_c[warp] = c_in;
        s.warp_m[warp] = m_in;
    }
    if (lane == 0) s.seg[warp] = n_min;
    __syncthreads();
    if (warp == 0) {
        uint32_t wc = s.warp_c[lane];
        double wm = s.warp_m[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t tc = __shfl_up_sync(kFull, wc, o);
            const double tm = __shfl_up_sync(kFull, wm, o);
            if (lane >= static_cast<uint32_t>(o)) {
                wc += tc;
                wm += tm;
            }
        }
        s.warp_c[lane] = wc;
        s.warp_m[lane] = wm;
        n_min = __reduce_add_sync(kFull, s.seg[lane]);
        if (lane == 0) s.u[0] = n_min;
    }
    __syncthreads();
    if (warp > 0) {
        c_in += s.warp_c[warp - 1];
        m_in += s.warp_m[warp - 1];
    }
    s.incl_c[tid] = c_in;
    s.incl_m[tid] = m_in;
    __syncthreads();
    n_min = s.u[0];
    const uint32_t c_before = tid ? s.incl_c[tid - 1] : 0u;
    const double m_before = tid ? s.incl_m[tid - 1] : 0.0;
    const uint32_t n_all = s.incl_c[kNT - 1];

    // Mass of the first n ids of the order.
    auto prefix_mass = [&](uint32_t n, int slot) {
        const int t = __syncthreads_count(c_in < n);
        if (static_cast<int>(tid) == t) {
            uint32_t left = n - c_before;
            double mass = m_before;
            for (uint32_t i = i0; i < i1 && left; ++i) {
                uint32_t c[kUnitBins];
                const uint32_t unit = s.units[i];
                counts(unit, c);
                for (uint32_t b = 0; b < kUnitBins && left; ++b) {
                    const uint32_t take = min(left, c[b]);
                    if (take) mass += take * weight(unit * kUnitBins + b);
                    left -= take;
                }
            }
            s.d[slot] = mass;
        }
        __syncthreads();
        return s.d[slot];
    };
    // 0-based rank of the first id whose cumulative mass is at least `goal`
    // (kOver: exceeds it); n_all when rounding leaves none.
    auto rank_of = [&](double goal, bool over, int slot) {
        const int t = min(__syncthreads_count(over ? m_in <= goal : m_in < goal), kNT - 1);
        if (static_cast<int>(tid) == t) {
            uint32_t at = c_in;  // not found inside: the next thread's first id
            uint32_t seen = c_before;
            double mass = m_before;
            bool found = false;
            for (uint32_t i = i0; i < i1 && !found; ++i) {
                uint32_t c[kUnitBins];
                const uint32_t unit = s.units[i];
                counts(unit, c);
                for (uint32_t b = 0; b < kUnitBins && !found; ++b) {
                    if (c[b] == 0) continue;
                    const double w = weight(unit * kUnitBins + b);
                    const double end = mass + c[b] * w;
                    if (over ? end > goal : end >= goal) {
                        // w > 0 here; the r-th id (from 0) ends at mass + (r + 1) w
                        const double r = over ? floor((goal - mass) / w) : ceil((goal - mass) / w) - 1.0;
                        at = seen + static_cast<uint32_t>(fmin(fmax(r, 0.0), c[b] - 1.0));
                        found = true;
                    }
                    mass = end;
                    seen += c[b];
                }
            }
            s.u[slot] = at;
        }
        __syncthreads();
        return s.u[slot];
    };

    uint32_t at = 0;
    double Zs = 1.0;
    if (!greedy) {
        const uint32_t n_k = kk == 0 ? n_all : min(kk, n_all);
        const double Z = prefix_mass(n_k, 0);
        uint32_t n = min(n_k, n_min);
        if (pf < 1.0f) n = min(n, rank_of(static_cast<double>(pf) * Z, false, 1) + 1u);
        Zs = n == n_k ? Z : prefix_mass(n, 1);
        at = min(rank_of(static_cast<double>(uf) * Zs, true, 2), n - 1u);
    }
    {
        // the drawn rank's bin, and its place among the bin's ids
        const int t = __syncthreads_count(c_in <= at);
        if (static_cast<int>(tid) == t) {
            uint32_t r = at - c_before;
            bool found = false;
            for (uint32_t i = i0; i < i1 && !found; ++i) {
                uint32_t c[kUnitBins];
                const uint32_t unit = s.units[i];
                counts(unit, c);
                for (uint32_t b = 0; b < kUnitBins && !found; ++b) {
                    if (r < c[b]) {
                        const uint32_t bin = unit * kUnitBins + b;
                        s.u[3] = bin;
                        s.u[4] = r;
                        s.d[2] = greedy ? 1.0 : weight(bin) / Zs;
                        found = true;
                    }
                    r -= c[b];
                }
            }
        }
        __syncthreads();
    }
    const uint32_t bin = s.u[3];
    uint32_t r = s.u[4];
    uint32_t owner = C;
    for (uint32_t c = 0; c < C && owner == C; ++c) {
        const uint32_t n = (cl.map_shared_rank(s.hist, c)[bin >> 1] >> (16 * (bin & 1))) & 0xFFFFu;
        if (r < n) owner = c;
        else r -= n;
    }
    if (owner == rank) {
        auto hit = [&](uint32_t w, int half) {
            const uint32_t b = half ? w >> 16 : w & 0xFFFFu;
            return b == bin || (bin == kZeroBin && b == kMinusZeroBin);
        };
        auto hits = [&](const uint4& v) {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint32_t n = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) n += hit(w[i >> 1], i & 1);
            return n;
        };
        // ids rise with j, then the warp, the lane and the element
#pragma unroll
        for (int j = 0; j < kVPT; ++j) {
            const uint32_t n = __reduce_add_sync(kFull, hits(q[j]));
            if (lane == 0) s.seg[j * kWarps + warp] = n;
        }
        __syncthreads();
        if (warp == 0) {
            uint32_t sum = 0;
#pragma unroll
            for (int i = 0; i < kVPT; ++i) sum += s.seg[lane * kVPT + i];
            uint32_t in = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t t = __shfl_up_sync(kFull, in, o);
                if (lane >= static_cast<uint32_t>(o)) in += t;
            }
            uint32_t before = in - sum;
            if (before <= r && r < in) {
                uint32_t i = lane * kVPT;
                while (r - before >= s.seg[i]) before += s.seg[i++];
                s.u[5] = i;
                s.u[6] = r - before;
            }
        }
        __syncthreads();
        const uint32_t seg = s.u[5];
        r = s.u[6];
        if (warp == seg % kWarps) {
#pragma unroll
            for (int j = 0; j < kVPT; ++j) {
                if (static_cast<uint32_t>(j) != seg / kWarps) continue;
                const uint32_t n = hits(q[j]);
                uint32_t in = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t t = __shfl_up_sync(kFull, in, o);
                    if (lane >= static_cast<uint32_t>(o)) in += t;
                }
                uint32_t left = r - (in - n);
                if (in - n <= r && r < in) {
                    const uint32_t w[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (hit(w[i >> 1], i & 1)) {
                            if (left == 0) {
                                a.out_ids[row] = (lo + j * kNT + tid) * 8u + i - skew;
                                a.out_probs[row] = static_cast<float>(s.d[2]);
                            }
                            --left;
                        }
                    }
                }
            }
        }
    }
    cl.sync();  // no CTA leaves while another reads its histogram
}

template <typename T>
sel_status launch(const SampleArgs& in, uint32_t rows, cudaStream_t stream) {
    const int sms = device_sms();
    if (sms <= 0) return SEL_ECUDA;
    // the fewest CTAs whose shares hold the row; more while every CTA of the
    // batch still has an SM of its own
    const uint32_t vecs = ceil_div(static_cast<uint64_t>(in.V) + 7, 8);
    uint32_t C = 1;
    while (ceil_div(vecs, C) > kShareVecs) C *= 2;
    while (C < kMaxCluster && vecs > C * static_cast<uint32_t>(kNT) &&
           static_cast<uint64_t>(rows) * C * 2 <= static_cast<uint64_t>(sms))
        C *= 2;
    if (static_cast<uint64_t>(rows) * C > 0x7fffffffull) return SEL_EUNSUPPORTED;
    SampleArgs a = in;
    a.share = ceil_div(vecs, C);
    if (!set_dynamic_smem(sample16_kernel<T>, sizeof(Shared))) return SEL_ECUDA;
    const cudaError_t e = launch_pdl_cluster(sample16_kernel<T>, dim3(rows * C), dim3(kNT), C, sizeof(Shared), stream, a);
    return e == cudaSuccess ? SEL_OK : SEL_ECUDA;
}

}  // namespace
}  // namespace sel

using namespace sel;

extern "C" sel_status sel_sample16(const void* d_logits, int dtype, uint32_t rows, uint32_t V, uint64_t ld,
                                   const float* d_temperature, const uint32_t* d_top_k, const float* d_top_p,
                                   const float* d_min_p, const float* d_uniforms, uint32_t* d_out_ids,
                                   float* d_out_probs, cudaStream_t stream) {
    if (V == 0 || V > SEL_MAX_V || ld < V || ld > SEL_MAX_LD) return SEL_EINVAL;
    if (dtype == SEL_F32) return SEL_EUNSUPPORTED;  // sel_sample's type
    if (dtype_bytes(dtype) != 2) return SEL_EINVAL;
    if (V > SEL_SAMPLE16_MAX_V) return SEL_EUNSUPPORTED;
    if (rows == 0) return SEL_OK;
    if (!d_logits || !d_uniforms || !d_out_ids || !d_out_probs) return SEL_EINVAL;
    if (misaligned(d_logits, 2) || misaligned(d_temperature, 4) || misaligned(d_top_k, 4) || misaligned(d_top_p, 4) ||
        misaligned(d_min_p, 4) || misaligned(d_uniforms, 4) || misaligned(d_out_ids, 4) || misaligned(d_out_probs, 4))
        return SEL_EINVAL;
    SampleArgs a{};
    a.logits = d_logits;
    a.ld = ld;
    a.temperature = d_temperature;
    a.top_k = d_top_k;
    a.top_p = d_top_p;
    a.min_p = d_min_p;
    a.uniforms = d_uniforms;
    a.out_ids = d_out_ids;
    a.out_probs = d_out_probs;
    a.V = V;
    return dtype == SEL_F16 ? launch<__half>(a, rows, stream) : launch<__nv_bfloat16>(a, rows, stream);
}
