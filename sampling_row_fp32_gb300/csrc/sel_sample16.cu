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
// overflows). After a cluster barrier the CTAs share the row's non-empty bins
// between them, sum their counts through distributed shared memory, and
// exchange the totals; each border (of top-k, top-p, the draw) is then found
// by the CTA whose bins hold it. The CTA whose share holds the drawn id finds it
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
__device__ __forceinline__ float bin_value(uint32_t bin) {
    const uint32_t u = bin < 0x8000u ? 0x7FFFu - bin : bin;
    return bits_f32<T>(static_cast<uint16_t>(u));
}

// ---------------------------------------------------------------------------
// weights: exp((x - max) / T) to about 45 bits without FP64, whose units would
// take 25 us over the distinct values of one f16 row
// ---------------------------------------------------------------------------
// With r = log2(e) / T as a sum of two floats, 2^y for y = (x - max) r, also
// kept as two floats: y = k / 256 + g with |g| <= 1/512, and
// 2^g = 1 + z + z^2/2 + z^3/6 + z^4/24 with z = g ln 2 <= 0.0014, whose next
// term is below 2^-56. Only z itself needs its second float; the higher terms
// are below 2^-20 and good to 2^-44 in one. 2^(j/256) comes from a table of
// float pairs, summed from its series at compile time.

constexpr int kTable = 256;
struct ExpTable {
    float2 v[kTable];
    constexpr ExpTable() : v{} {
        for (int j = 0; j < kTable; ++j) {
            const double z = j * 0.693147180559945309417232121458 / kTable;
            double term = 1.0, sum = 1.0;
            for (int k = 1; k < 24; ++k) {
                term *= z / k;
                sum += term;
            }
            const float hi = static_cast<float>(sum);
            v[j].x = hi;
            v[j].y = static_cast<float>(sum - static_cast<double>(hi));
        }
    }
};
__constant__ const ExpTable kExpTable;

struct Weights {
    float top;            // the row's largest logit, times `pre`
    float pre, post;      // powers of two, their product about 1 / T: r stays near 1
    FF r;                 // log2(e) / (T pre post)
    const float2* table;  // in shared memory

    __device__ __forceinline__ Weights(float row_max, float T, const float2* tab) : table(tab) {
        const int e = min(max(static_cast<int>(__float_as_uint(T) >> 23) - 127, -126), 126);  // T is about 2^e
        pre = exp2i(e > 0 ? -e : 0);
        post = exp2i(e > 0 ? 0 : -e);
        top = row_max * pre;
        r = ff_from_double(1.4426950408889634 / (static_cast<double>(T) * pre * post));
    }
    static __device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }

    // 0 below 2^-100, the whole tail of a row weighing less than 2^-80 then
    __device__ __forceinline__ FF operator()(float logit) const {
        constexpr float kLn2 = 0.693147182464599609375f, kLn2Lo = -1.904654299957767e-9f;
        const float x = logit * pre;
        const float ds = x - top;  // and the subtraction's rounding error
        const float v = ds - x;
        const float dl = ((x - (ds - v)) - (top + v)) * post;
        const float dh = ds * post;
        const float yh = dh * r.hi;
        if (!(yh > -100.0f)) return FF{0.0f, 0.0f};
        const float yl = __fmaf_rn(dh, r.hi, -yh) + __fmaf_rn(dl, r.hi, dh * r.lo);
        const float magic = __fmaf_rn(yh, static_cast<float>(kTable), 12582912.0f);  // 1.5 * 2^23: rounds to a whole number
        const int k = __float_as_int(magic) - 0x4B400000;
        const float g = __fmaf_rn(magic - 12582912.0f, -1.0f / kTable, yh);  // exact
        const float zh = g * kLn2;
        const float zl = __fmaf_rn(g, kLn2, -zh) + __fmaf_rn(g, kLn2Lo, yl * kLn2);
        const float q = __fmaf_rn(zh, __fmaf_rn(zh, 1.0f / 24, 1.0f / 6), 0.5f);
        const float el = zl + __fmaf_rn(zh * zh, q, zh * zl);  // 2^(g + yl) = 1 + zh + el
        const float2 t = table[k & (kTable - 1)];
        const float ph = t.x * zh, pl = __fmaf_rn(t.x, zh, -ph);
        const float s = t.x + ph;
        const float lo = (ph - (s - t.x)) + (pl + (t.y + __fmaf_rn(t.x, el, t.y * zh)));
        const float scale = __int_as_float(((k >> 8) + 127) << 23);
        return FF{s * scale, lo * scale};
    }
};
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

// What the CTAs of a row tell each other: each writes its line of every CTA's
// table, and the CTA that decides a step its results.
struct Totals {
    double mass;
    uint32_t count, min_count;
};
enum { kMassK, kMassN, kProb, kDoubles };
enum { kRankP, kBin, kPlace, kRank, kInts };

struct Shared {
    uint32_t hist[kBins / 2];
    uint16_t units[kUnits];  // the row's non-empty units, in bin order
    float2 table[kTable];
    double incl_m[kNT];
    uint32_t incl_c[kNT];
    uint32_t bits[kWords];
    uint32_t off[kWords];
    double warp_m[kWarps];
    uint32_t warp_c[kWarps];
    uint32_t seg[kVPT * kWarps];
    Totals totals[kMaxCluster];
    double d[kDoubles];
    uint32_t u[kInts];
    uint32_t find[2];
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
    if (tid < kTable) s.table[tid] = kExpTable.v[tid];
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
    float xmax = 0.0f;
    uint32_t first_bin = 0;
    if (!bad) {
        uint32_t c[kUnitBins];
        const uint32_t first = s.units[0], last = s.units[nu - 1];
        counts(first, c);
        uint32_t f = kUnitBins, l = 0;
#pragma unroll
        for (uint32_t b = kUnitBins; b-- > 0;)
            if (c[b]) f = b;
        counts(last, c);
#pragma unroll
        for (uint32_t b = 0; b < kUnitBins; ++b)
            if (c[b]) l = b;
        first_bin = first * kUnitBins + f;
        xmax = bin_value<T>(first_bin);
        bad = first_bin <= kPosInf || last * kUnitBins + l > kNegInf;
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
    const Weights weight(xmax, greedy ? 1.0f : Tf, s.table);

    // This CTA's part of the list, and each thread's.
    const uint32_t first = static_cast<uint32_t>(static_cast<uint64_t>(nu) * rank / C);
    const uint32_t last = static_cast<uint32_t>(static_cast<uint64_t>(nu) * (rank + 1) / C);
    const uint32_t per = (last - first + kNT - 1) / kNT;
    const uint32_t i0 = min(last, first + tid * per), i1 = min(last, i0 + per);

    // Counts and masses up to each thread's units, in order.
    uint32_t c_in = 0, n_min = 0;
    FF mass{0.0f, 0.0f};
    for (uint32_t i = i0; i < i1; ++i) {
        uint32_t c[kUnitBins];
        const uint32_t unit = s.units[i];
        counts(unit, c);
#pragma unroll
        for (uint32_t b = 0; b < kUnitBins; ++b) {
            const FF w = weight(bin_value<T>(unit * kUnitBins + b));
            if (c[b]) {
                c_in += c[b];
                mass = ff_add(mass, ff_mul_f(w, static_cast<float>(c[b])));
                if (w.hi > mf || (w.hi == mf && w.lo >= 0.0f)) n_min += c[b];
            }
        }
    }
    double m_in = ff_to_double(mass);
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
        wc = __shfl_sync(kFull, wc, 31);
        wm = __shfl_sync(kFull, wm, 31);
        if (lane < C) cl.map_shared_rank(s.totals, lane)[rank] = Totals{wm, wc, n_min};
    }
    cl.sync();
    // sums before this CTA's units and over the row, in the same order everywhere
    uint32_t c_base = 0, n_all = 0;
    double m_base = 0.0, m_all = 0.0;
    n_min = 0;
    for (uint32_t r = 0; r < C; ++r) {
        if (r == rank) {
            c_base = n_all;
            m_base = m_all;
        }
        n_all += s.totals[r].count;
        m_all += s.totals[r].mass;
        n_min += s.totals[r].min_count;
    }
    if (warp > 0) {
        c_in += s.warp_c[warp - 1];
        m_in += s.warp_m[warp - 1];
    }
    c_in += c_base;
    m_in += m_base;
    s.incl_c[tid] = c_in;
    s.incl_m[tid] = m_in;
    __syncthreads();
    const uint32_t c_before = tid ? s.incl_c[tid - 1] : c_base, c_end = s.incl_c[kNT - 1];
    const double m_before = tid ? s.incl_m[tid - 1] : m_base;

    // A thread's bins in order: f(bin, count, weight, ids before, mass before)
    // until it returns true.
    auto walk = [&](auto f) {
        uint32_t seen = c_before;
        double m = m_before;
        for (uint32_t i = i0; i < i1; ++i) {
            uint32_t c[kUnitBins];
            const uint32_t unit = s.units[i];
            counts(unit, c);
#pragma unroll
            for (uint32_t b = 0; b < kUnitBins; ++b) {
                if (c[b] == 0) continue;
                const uint32_t bin = unit * kUnitBins + b;
                const double w = ff_to_double(weight(bin_value<T>(bin)));
                if (f(bin, c[b], w, seen, m)) return;
                seen += c[b];
                m += c[b] * w;
            }
        }
    };
    auto tell = [&](auto&& field, auto value) {  // the same word of every CTA
        for (uint32_t r = 0; r < C; ++r) *cl.map_shared_rank(&field, r) = value;
    };
    // Mass of the first n ids of the order.
    auto prefix_mass = [&](uint32_t n, int slot) {
        if (n == n_all) return m_all;
        if (c_base < n && n <= c_end) {
            if (static_cast<int>(tid) == __syncthreads_count(c_in < n)) {
                double mass = 0.0;
                walk([&](uint32_t, uint32_t c, double w, uint32_t seen, double m) {
                    mass = m + min(n - seen, c) * w;
                    return seen + c >= n;
                });
                tell(s.d[slot], mass);
            }
        }
        cl.sync();
        return s.d[slot];
    };
    // Whether the first id whose cumulative mass reaches `goal` (over: exceeds
    // it) is among this CTA's, its last one's when rounding leaves none.
    auto reached = [&](double m, double goal, bool over) { return over ? m > goal : m >= goal; };
    auto holds = [&](double goal, bool over) {
        double m = 0.0;
        uint32_t r = 0;
        for (; r + 1 < C; ++r) {
            m += s.totals[r].mass;
            if (reached(m, goal, over)) break;
        }
        return r == rank;
    };
    // The thread that has it, and that id: its bin, its place among the bin's
    // ids, its rank in the row.
    auto find_mass = [&](double goal, bool over, auto f) {
        if (!holds(goal, over)) return;
        if (static_cast<int>(tid) != min(__syncthreads_count(!reached(m_in, goal, over)), kNT - 1)) return;
        uint32_t bin = 0, place = 0, at = c_in;  // not found inside: the next thread's first id
        double weight_of = 1.0;
        walk([&](uint32_t b, uint32_t c, double w, uint32_t seen, double m) {
            bin = b;
            weight_of = w;
            if (!reached(m + c * w, goal, over)) {
                place = c - 1;
                return false;
            }
            // w > 0 here; the r-th id (from 0) ends at m + (r + 1) w
            const double r = over ? floor((goal - m) / w) : ceil((goal - m) / w) - 1.0;
            place = static_cast<uint32_t>(fmin(fmax(r, 0.0), c - 1.0));
            at = seen + place;
            return true;
        });
        f(bin, place, at, weight_of);
    };

    if (greedy) {
        if (tid == 0) {
            s.u[kBin] = first_bin;
            s.u[kPlace] = 0;
            s.d[kProb] = 1.0;
        }
        __syncthreads();
    } else {
        const uint32_t n_k = kk == 0 ? n_all : min(kk, n_all);
        const double Z = prefix_mass(n_k, kMassK);
        uint32_t n = min(n_k, n_min);
        if (pf < 1.0f) {
            find_mass(static_cast<double>(pf) * Z, false,
                      [&](uint32_t, uint32_t, uint32_t at, double) { tell(s.u[kRankP], at); });
            cl.sync();
            n = min(n, s.u[kRankP] + 1u);
        }
        const double Zs = n == n_k ? Z : prefix_mass(n, kMassN);
        auto drawn = [&](uint32_t bin, uint32_t place, uint32_t at, double w) {
            tell(s.u[kBin], bin);
            tell(s.u[kPlace], place);
            tell(s.u[kRank], at);
            tell(s.d[kProb], w / Zs);
        };
        find_mass(static_cast<double>(uf) * Zs, true, drawn);
        cl.sync();
        if (s.u[kRank] >= n) {  // rounding left none: the last survivor
            cl.sync();          // every CTA has read the rank
            if (c_base < n && n <= c_end && static_cast<int>(tid) == __syncthreads_count(c_in < n)) {
                walk([&](uint32_t b, uint32_t c, double w, uint32_t seen, double) {
                    if (seen + c < n) return false;
                    drawn(b, n - 1 - seen, n - 1, w);
                    return true;
                });
            }
            cl.sync();
        }
    }
    const uint32_t bin = s.u[kBin];
    uint32_t r = s.u[kPlace];
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
                s.find[0] = i;
                s.find[1] = r - before;
            }
        }
        __syncthreads();
        const uint32_t seg = s.find[0];
        r = s.find[1];
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
                                a.out_probs[row] = static_cast<float>(s.d[kProb]);
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
