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
// between them, a lane a bin, and sum counts (through distributed shared
// memory) and masses of up to 2,048 entries in the first CTA. There one warp
// finds every border (of top-k, top-p, the draw): ballots over the entries'
// prefix sums, then the 32 bins of the entry. The CTA whose share holds the
// drawn id finds it in its registers.
//
// FP64 runs at two results a clock and SM here, so only that one warp uses it:
// a single FP64 addition by all 32 warps costs 460 clocks.
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

    // (by one thread, while the row is counted; `top` follows)
    __device__ __forceinline__ void temperature(float T) {
        const int e = min(max(static_cast<int>(__float_as_uint(T) >> 23) - 127, -126), 126);  // T is about 2^e
        pre = exp2i(e > 0 ? -e : 0);
        post = exp2i(e > 0 ? 0 : -e);
        r = ff_from_double(1.4426950408889634 / (static_cast<double>(T) * pre * post));
    }
    static __device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }

    // 0 below 2^-100, the whole tail of a row weighing less than 2^-80 then
    __device__ __forceinline__ FF operator()(float logit, const float2* table) const {
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

constexpr uint32_t kEntries = 2048;             // at most; of up to four units, a lane a bin
constexpr uint32_t kCoarse = kEntries / 32;     // entries a lane of the deciding warp looks at first
static_assert(kUnits <= kEntries * 4 && kEntries == 2 * kNT);

struct Shared {
    uint32_t hist[kBins / 2];
    uint16_t units[kUnits];   // the row's non-empty units, in bin order
    float2 table[kTable];
    uint32_t entry_c[kEntries];  // in the row's first CTA: counts and masses of the entries,
    FF entry_m[kEntries];        // then up to and with each entry
    uint32_t bits[kWords];    // occupancy: bit l of word w is unit 32 w + l
    uint32_t off[kWords];
    FF warp_m[kWarps];
    uint32_t warp_c[kWarps];
    uint32_t seg[kVPT * kWarps];
    Weights weights;
    uint32_t n_min;           // ids that min-p leaves
    uint32_t first_bin;       // the largest logit's
    uint32_t bad;
    uint32_t bin, owner, place;  // the drawn bin, the CTA of the drawn id, its place among that CTA's ids of the bin
    float prob;
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
    if (tid == 0) s.n_min = 0;
    pdl_wait();

    // The row as 16-byte vectors from the aligned address at or below its
    // start; `skew` ids of the first vector are not the row's. Vectors that
    // reach over either end of the row are read by element.
    const uint16_t* x = static_cast<const uint16_t*>(a.logits) + static_cast<uint64_t>(row) * a.ld;
    const uint32_t skew = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(x) & 15u) / 2u;
    const uint32_t vecs = (a.V + skew + 7u) / 8u;
    const uint32_t lo = rank * a.share, hi = min(vecs, lo + a.share);
    const uint32_t full_lo = max(lo, skew ? 1u : 0u), full_hi = min(hi, (a.V + skew) / 8u);
    uint4 q[kVPT];
#pragma unroll
    for (int j = 0; j < kVPT; ++j) {
        const uint32_t v = lo + j * kNT + tid;
        q[j] = make_uint4(kFill, kFill, kFill, kFill);
        if (v >= full_lo && v < full_hi) q[j] = ldg_stream16(x - skew + static_cast<uint64_t>(v) * 8u);
    }
    const float Tf = a.temperature ? a.temperature[row] : 1.0f;
    const uint32_t kk = a.top_k ? a.top_k[row] : 0u;
    const float pf = a.top_p ? a.top_p[row] : 1.0f;
    const float mf = a.min_p ? a.min_p[row] : 0.0f;
    const float uf = a.uniforms[row];
    auto edge = [&](uint32_t v) {  // the vector v, if it is this thread's
        if (v < lo || v >= hi || (v - lo) % kNT != tid) return;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t e = static_cast<int64_t>(v) * 8 - skew + 2 * i + h;
                w[i] |= (e >= 0 && e < a.V ? x[e] : kNegInf) << (16 * h);
            }
        }
#pragma unroll
        for (int j = 0; j < kVPT; ++j)
            if ((v - lo) / kNT == static_cast<uint32_t>(j)) q[j] = make_uint4(w[0], w[1], w[2], w[3]);
    };
    if (skew) edge(0);
    if ((a.V + skew) % 8u && (vecs > 1 || !skew)) edge(vecs - 1);
    pdl_trigger();
    if (tid == 32) s.weights.temperature(Tf > 0.0f ? Tf : 1.0f);
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
#pragma unroll
    for (int i = 0; i < static_cast<int>(kUnits / kNT); ++i) {
        const uint32_t word = i * kWarps + warp;
        const uint4 v = h4[word * 32 + lane];
        const uint32_t b = __ballot_sync(kFull, (v.x | v.y | v.z | v.w) != 0);
        if (lane == 0) s.bits[word] = b;
    }
    cl.sync();

    // The row's non-empty units, in order.
    uint32_t word = 0;
    if (tid < kWords) {
        for (uint32_t r = 0; r < C; ++r) word |= cl.map_shared_rank(s.bits, r)[tid];
        uint32_t in = __popc(word);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t n = __shfl_up_sync(kFull, in, o);
            if (lane >= static_cast<uint32_t>(o)) in += n;
        }
        s.off[tid] = in;  // up to and with this word, in its 32
        s.seg[tid] = word;
    }
    __syncthreads();
    uint32_t nu = 0;
#pragma unroll
    for (int i = 0; i < static_cast<int>(kUnits / kNT); ++i) {
        const uint32_t w = i * kWarps + warp, m = s.seg[w], before = s.off[w] - __popc(m);
        if (m >> lane & 1) s.units[nu + before + __popc(m & ((1u << lane) - 1u))] = static_cast<uint16_t>(w * 32 + lane);
        nu += s.off[i * kWarps + 31];
    }
    __syncthreads();

    auto count = [&](uint32_t bin) {  // over the row
        uint32_t n = 0;
        for (uint32_t r = 0; r < C; ++r) n += reinterpret_cast<const uint16_t*>(cl.map_shared_rank(s.hist, r))[bin];
        return n;
    };
    if (warp == 0) {
        // The policy, and the row's validity: a NaN or +Inf logit, nothing
        // unmasked, a uniform or a parameter out of its range.
        bool bad = !(Tf >= 0.0f) || isinf(Tf) || !(pf > 0.0f && pf <= 1.0f) || !(mf >= 0.0f && mf < 1.0f) ||
                   !(uf >= 0.0f && uf < 1.0f) || nu == 0;
        if (!bad) {
            const uint32_t unit = lane < 8 ? s.units[0] : s.units[nu - 1];
            const uint32_t used = __ballot_sync(kFull, lane < 16 && count(unit * kUnitBins + lane % 8) > 0);
            const uint32_t first = s.units[0] * kUnitBins + __ffs(used & 0xFFu) - 1;
            const uint32_t last = s.units[nu - 1] * kUnitBins + (31 - __clz(used >> 8));
            bad = first <= kPosInf || last > kNegInf;
            if (lane == 0) {
                s.first_bin = first;
                s.weights.top = bin_value<T>(first) * s.weights.pre;
            }
        }
        if (lane == 0) s.bad = bad;
    }
    __syncthreads();
    if (s.bad) {  // the same in every CTA of the cluster
        if (rank == 0 && tid == 0) {
            a.out_ids[row] = SEL_INVALID_ID;
            a.out_probs[row] = __uint_as_float(0x7FC00000u);
        }
        cl.sync();  // no CTA leaves while another reads its histogram
        return;
    }
    const bool greedy = Tf == 0.0f;
    const Weights weights = s.weights;

    // Entries of up to four units, shared between the CTAs; a lane a bin.
    const uint32_t per = (nu + kEntries - 1) / kEntries, entries = (nu + per - 1) / per;
    if (!greedy) {
        const uint32_t e0 = entries * rank / C, e1 = entries * (rank + 1) / C;
        uint32_t n_min = 0;
        for (uint32_t base = e0 + warp * 4; base < e1; base += kWarps * 4) {
            const uint32_t e = base + lane / 8;
            uint32_t c = 0;
            FF m{0.0f, 0.0f};
            for (uint32_t g = 0; g < per; ++g) {
                const uint32_t i = e * per + g;
                if (e < e1 && i < nu) {
                    const uint32_t bin = s.units[i] * kUnitBins + lane % 8, n = count(bin);
                    const FF w = weights(bin_value<T>(bin), s.table);
                    if (n) {
                        c += n;
                        m = ff_add(m, ff_mul_f(w, static_cast<float>(n)));
                        if (w.hi > mf || (w.hi == mf && w.lo >= 0.0f)) n_min += n;
                    }
                }
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                c += __shfl_xor_sync(kFull, c, o);
                const FF other = ff_shfl_xor(m, o);
                m = lane & o ? ff_add(other, m) : ff_add(m, other);
            }
            if (lane % 8 == 0 && e < e1) {
                cl.map_shared_rank(s.entry_c, 0)[e] = c;
                cl.map_shared_rank(s.entry_m, 0)[e] = m;
            }
        }
        n_min = __reduce_add_sync(kFull, n_min);
        if (lane == 0 && n_min) atomicAdd(cl.map_shared_rank(&s.n_min, 0), n_min);
    }
    cl.sync();

    if (rank == 0) {
        if (!greedy) {
            // the entries' prefix sums, two a thread
            uint32_t c[2];
            FF m[2];
#pragma unroll
            for (uint32_t i = 0; i < 2; ++i) {
                const uint32_t e = 2 * tid + i;
                c[i] = e < entries ? s.entry_c[e] : 0u;
                m[i] = e < entries ? s.entry_m[e] : FF{0.0f, 0.0f};
            }
            uint32_t wc = c[0] + c[1];
            const FF both = ff_add(m[0], m[1]);
            FF wm = ff_warp_scan(both);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t n = __shfl_up_sync(kFull, wc, o);
                if (lane >= static_cast<uint32_t>(o)) wc += n;
            }
            if (lane == 31) {
                s.warp_c[warp] = wc;
                s.warp_m[warp] = wm;
            }
            __syncthreads();
            if (warp == 0) {
                uint32_t tc = s.warp_c[lane];
                const FF tm = ff_warp_scan(s.warp_m[lane]);
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t n = __shfl_up_sync(kFull, tc, o);
                    if (lane >= static_cast<uint32_t>(o)) tc += n;
                }
                s.warp_c[lane] = tc;
                s.warp_m[lane] = tm;
            }
            __syncthreads();
            // up to the first and the second entry: what lies before the pair, and on
            uint32_t before_c = wc - (c[0] + c[1]);
            FF before_m = ff_shfl_up(wm, 1);
            if (lane == 0) before_m = FF{0.0f, 0.0f};
            if (warp > 0) {
                before_c += s.warp_c[warp - 1];
                before_m = ff_add(s.warp_m[warp - 1], before_m);
            }
            s.entry_c[2 * tid] = before_c + c[0];
            s.entry_c[2 * tid + 1] = before_c + c[0] + c[1];
            s.entry_m[2 * tid] = ff_add(before_m, m[0]);
            s.entry_m[2 * tid + 1] = ff_add(before_m, both);
            __syncthreads();
        }
        if (warp == 0) {
            // Lane l holds bin l of an entry's up to 32; sums up to and with it.
            struct Bins {
                uint32_t bin, c;      // the lane's bin and its count
                uint32_t c_before, c_in;
                double w, m_before, m_in;
            };
            auto open = [&](uint32_t e) {
                Bins b{};
                const uint32_t i = e * per + lane / 8;
                FF m{0.0f, 0.0f};
                if (lane / 8 < per && i < nu) {
                    b.bin = s.units[i] * kUnitBins + lane % 8;
                    b.c = count(b.bin);
                    const FF w = weights(bin_value<T>(b.bin), s.table);
                    b.w = ff_to_double(w);
                    if (b.c) m = ff_mul_f(w, static_cast<float>(b.c));
                }
                b.c_in = b.c;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t n = __shfl_up_sync(kFull, b.c_in, o);
                    if (lane >= static_cast<uint32_t>(o)) b.c_in += n;
                }
                const FF scan = ff_warp_scan(m);
                if (e) b.c_in += s.entry_c[e - 1];
                b.m_in = ff_to_double(e ? ff_add(s.entry_m[e - 1], scan) : scan);
                b.c_before = b.c_in - b.c;
                b.m_before = __shfl_up_sync(kFull, b.m_in, 1);
                if (lane == 0) b.m_before = e ? ff_to_double(s.entry_m[e - 1]) : 0.0;
                return b;
            };
            // The first entry for which `past` holds, the last one when none does.
            auto first_entry = [&](auto past) {
                const uint32_t coarse = __ballot_sync(kFull, past(lane * kCoarse + kCoarse - 1));
                const uint32_t at = (coarse ? __ffs(coarse) - 1 : 31) * kCoarse;
                uint32_t e = at + kCoarse - 1;
#pragma unroll
                for (uint32_t i = kCoarse / 32; i-- > 0;) {
                    const uint32_t fine = __ballot_sync(kFull, past(at + i * 32 + lane));
                    if (fine) e = at + i * 32 + __ffs(fine) - 1;
                }
                return min(e, entries - 1);
            };
            const uint32_t n_all = s.entry_c[kEntries - 1];
            const double m_all = ff_to_double(s.entry_m[kEntries - 1]);
            auto prefix_mass = [&](uint32_t n) {  // of the first n ids of the order
                if (n == n_all) return m_all;
                const Bins b = open(first_entry([&](uint32_t e) { return s.entry_c[e] >= n; }));
                const int l = __ffs(__ballot_sync(kFull, b.c_in >= n)) - 1;
                return __shfl_sync(kFull, b.m_before + (n - b.c_before) * b.w, l);
            };
            // The first id whose cumulative mass reaches `goal` (over: exceeds
            // it): its lane, its place among the bin's ids; and its rank.
            auto by_mass = [&](double goal, bool over, Bins& b, uint32_t& place, int& l) {
                auto past = [&](double m) { return over ? m > goal : m >= goal; };
                b = open(first_entry([&](uint32_t e) { return past(ff_to_double(s.entry_m[e])); }));
                const uint32_t hit = __ballot_sync(kFull, b.c > 0 && past(b.m_in));
                // (rounding may leave none: the entry's last id)
                l = hit ? __ffs(hit) - 1 : 31 - __clz(__ballot_sync(kFull, b.c > 0));
                // the r-th id of the bin (from 0) ends at m_before + (r + 1) w
                const double r = over ? floor((goal - b.m_before) / b.w) : ceil((goal - b.m_before) / b.w) - 1.0;
                place = hit ? static_cast<uint32_t>(fmin(fmax(r, 0.0), b.c - 1.0)) : b.c - 1u;
                place = __shfl_sync(kFull, place, l);
                return __shfl_sync(kFull, b.c_before, l) + place;
            };

            uint32_t bin = s.first_bin, place = 0;
            double prob = 1.0;
            if (!greedy) {
                const uint32_t n_k = kk == 0 ? n_all : min(kk, n_all);
                const double Z = prefix_mass(n_k);
                uint32_t n = min(n_k, s.n_min);
                Bins b;
                int l;
                if (pf < 1.0f) n = min(n, by_mass(static_cast<double>(pf) * Z, false, b, place, l) + 1u);
                const double Zs = n == n_k ? Z : prefix_mass(n);
                if (by_mass(static_cast<double>(uf) * Zs, true, b, place, l) >= n) {
                    // rounding: the last survivor
                    b = open(first_entry([&](uint32_t e) { return s.entry_c[e] >= n; }));
                    l = __ffs(__ballot_sync(kFull, b.c_in >= n)) - 1;
                    place = __shfl_sync(kFull, n - 1u - b.c_before, l);
                }
                bin = __shfl_sync(kFull, b.bin, l);
                prob = __shfl_sync(kFull, b.w, l) / Zs;
            }
            // the CTA that holds it: ids rise with the CTAs
            const uint32_t c = lane < C ? reinterpret_cast<const uint16_t*>(cl.map_shared_rank(s.hist, lane))[bin] : 0u;
            uint32_t in = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t n = __shfl_up_sync(kFull, in, o);
                if (lane >= static_cast<uint32_t>(o)) in += n;
            }
            const int owner = __ffs(__ballot_sync(kFull, place < in)) - 1;
            place = __shfl_sync(kFull, place - (in - c), owner);
            if (lane < C) {
                Shared& o = *cl.map_shared_rank(&s, lane);
                o.bin = bin;
                o.owner = owner;
                o.place = place;
                o.prob = static_cast<float>(prob);
            }
        }
    }
    cl.sync();
    if (rank != s.owner) return;

    // The place-th id of the bin in this CTA's registers: ids rise with j, then
    // the warp, the lane and the element.
    const uint32_t bin = s.bin, pattern = bin * 0x00010001u;
    uint32_t r = s.place;
    auto flags = [&](uint32_t w) {  // bits 0 and 16: the halves that match
        uint32_t f = __vcmpeq2(w, pattern);
        if (bin == kZeroBin) f |= __vcmpeq2(w, kMinusZeroBin * 0x00010001u);
        return f & 0x00010001u;
    };
    auto hits = [&](const uint4& v) {
        const uint32_t f = flags(v.x) + flags(v.y) + flags(v.z) + flags(v.w);
        return (f & 0xFFFFu) + (f >> 16);
    };
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
            const uint32_t n = __shfl_up_sync(kFull, in, o);
            if (lane >= static_cast<uint32_t>(o)) in += n;
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
    if (warp != seg % kWarps) return;
#pragma unroll
    for (int j = 0; j < kVPT; ++j) {
        if (static_cast<uint32_t>(j) != seg / kWarps) continue;
        const uint32_t n = hits(q[j]);
        uint32_t in = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t m = __shfl_up_sync(kFull, in, o);
            if (lane >= static_cast<uint32_t>(o)) in += m;
        }
        uint32_t left = r - (in - n);
        if (in - n <= r && r < in) {
            const uint32_t w[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (flags(w[i >> 1]) >> (16 * (i & 1)) & 1) {
                    if (left == 0) {
                        a.out_ids[row] = (lo + j * kNT + tid) * 8u + i - skew;
                        a.out_probs[row] = s.prob;
                    }
                    --left;
                }
            }
        }
    }
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
