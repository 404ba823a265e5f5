// sel_sample16.cu -- sampling of 16-bit logits rows with a policy per row.
//
// Order a row's ids by (logit descending, id ascending). Every filter of the
// chain keeps a prefix of that order: top-k the first k ids, top-p the
// shortest prefix whose mass reaches top_p, min-p the ids whose weight
// w = exp((x - max) / T) is at least min_p. The draw is the first id of the
// surviving prefix whose cumulative mass exceeds u times the prefix's mass.
// A 16-bit row holds at most 65,536 distinct logits, so a histogram of the
// 16-bit patterns holds all of it: ranks are integer sums of counts, masses
// are sums of count * w to about 45 bits, and the drawn id is the r-th id of
// one pattern.
//
// One cluster of C CTAs per row. Each CTA counts its share of the row into a
// histogram of 65,536 16-bit counters in its shared memory. After a cluster
// barrier the CTAs share the row's non-empty bins between them, a lane a bin,
// and sum counts (through distributed shared memory) and masses of up to
// 2,048 entries in the first CTA. There one warp finds every border (of top-k,
// top-p, the draw): ballots over the entries' prefix sums, then the 32 bins of
// the entry. The CTA whose share holds the drawn id reads its share again.
//
// Where top-k is on, the first batch of a share gives a bound that the top k
// of the row are not under, and the rest of the share is only counted down to
// it: what bounds counting every id is the atomics, at about five a clock and SM.
// Ids past the first batch that are not under the bound are listed as well, where
// they are few, and the drawn id is looked for there.
//
// A counter that overflows (a value that more than 65,535 ids of a share have)
// makes the counters' sum differ from the ids counted; the share is then
// counted again in batches, and counters past half are taken down in between.
//
// Masses are pairs of floats: FP64 runs at two results a clock and SM here.
//
// One row of 151,936 takes 14-18 us, 9 when it is greedy, a chain of about a dozen
// dependent steps; 49 rows of 248,320 32 us and 256 of 202,048 72-74 us (the rows'
// bytes alone would take 3.6 and 15). Of the 40 us of 152 rows of 202,048 without
// top-k, counting takes
// 15, the second look at the share 10 and the chain most of the rest; with a small
// top-k counting runs at 5.9 TB/s.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cooperative_groups.h>

#include "sel.h"
#include "sel_common.cuh"
#include "sel_dtype.cuh"
#include "sel_per_device.h"
#include "sel_plan.h"
#include "sel_units.cuh"

namespace cg = cooperative_groups;

namespace sel {
namespace {

constexpr int kNT = 1024;
constexpr int kWarps = kNT / 32;
// 16-byte vectors a thread loads ahead. Two: every further one lengthens the code
// of a pass, which a small batch fetches for its first and only use (16.9 us a
// row of 151,936 with two, 18.9 with four), and large ones gain nothing. Four where
// most vectors need a comparison only.
constexpr uint32_t kAhead = 2, kAheadFrom = 4;
constexpr uint32_t kMaxCluster = 8;
constexpr uint32_t kBatchVecs = 4095;       // vectors whose ids overflow no counter below half
constexpr uint32_t kHalf = 32768;
constexpr uint32_t kMaxHeavy = SEL_SAMPLE16_MAX_V / kHalf + 1;
constexpr uint32_t kBins = 65536;
constexpr uint32_t kUnitBins = 8;           // a 16-byte unit of the histogram
constexpr uint32_t kUnits = kBins / kUnitBins;
constexpr uint32_t kWords = kUnits / 32;    // occupancy bitmap
static_assert(kBatchVecs * 8 + kHalf <= 65536);

// Counters are indexed by the logits' bit patterns. Bins number the patterns by
// value, descending: bin 0 is the largest. (Its own inverse.)
__device__ __forceinline__ uint32_t pattern_of(uint32_t bin) { return bin < 0x8000u ? 0x7FFFu - bin : bin; }
// The unit of eight counters that holds the bins of unit u.
__device__ __forceinline__ uint32_t stored_unit(uint32_t u) { return u < kUnits / 2 ? kUnits / 2 - 1 - u : u; }

// Per type: the pattern of +Inf, and comparisons of two packed logits, done by
// the half-precision pipe; the integer pipe is what bounds the passes over a row.
template <typename T>
struct Kind;
template <>
struct Kind<__nv_bfloat16> {
    static constexpr uint32_t kInf = 0x7F80;
    using Pair = __nv_bfloat162;
};
template <>
struct Kind<__half> {
    static constexpr uint32_t kInf = 0x7C00;
    using Pair = __half2;
};
template <typename T>
__device__ __forceinline__ typename Kind<T>::Pair as_pair(uint32_t w) {
    typename Kind<T>::Pair p;
    memcpy(&p, &w, 4);
    return p;
}
// All ones in each half that equals (-0 equals +0); that differs, that is not
// below, NaNs included.
template <typename T>
__device__ __forceinline__ uint32_t equal2(uint32_t a, uint32_t b) { return __heq2_mask(as_pair<T>(a), as_pair<T>(b)); }
template <typename T>
__device__ __forceinline__ uint32_t differ2(uint32_t a, uint32_t b) { return __hneu2_mask(as_pair<T>(a), as_pair<T>(b)); }
template <typename T>
__device__ __forceinline__ uint32_t not_below2(typename Kind<T>::Pair a, typename Kind<T>::Pair b) { return __hgeu2_mask(a, b); }

template <typename T>
__device__ __forceinline__ float bin_value(uint32_t bin) {
    return bits_f32<T>(static_cast<uint16_t>(pattern_of(bin)));
}

template <typename T>
__device__ __forceinline__ uint32_t bin_of(float x) {  // of a logit (an f16 or bf16 value; +0 for -0)
    const T h = from_f32<T>(x + 0.0f);
    uint16_t u;
    memcpy(&u, &h, 2);
    return pattern_of(u);
}

// ---------------------------------------------------------------------------
// weights: exp((x - max) / T) to about 45 bits without FP64, with which the
// distinct values of an f16 row took longer than all else (158 us against 45)
// ---------------------------------------------------------------------------
// With r = log2(e) / T as a sum of two floats, 2^y for y = (x - max) r, also
// kept as two floats: y = k / 256 + g with |g| <= 1/512, and
// 2^g = 1 + z + z^2/2 + z^3/6 + z^4/24 with z = g ln 2 <= 0.0014, whose next
// term is below 2^-54. z and its square need a second float each; the terms
// beyond are below 2^-31 and good to 2^-54 in one. y's second float, up to
// 2^-18 at y = -100, joins g before the series, so that it counts in every term.
// 2^(j/256) comes from a table of float pairs, summed from its series at
// compile time. A weight's relative error, measured: at most 2^-46 near the
// largest logit, 2^-44 down to weights of 2^-16, 2^-42 down to 2^-30, and 2^-41
// at the end, where it is y's, good to about 2^-48 of itself.

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
// (in global memory: constant memory serves one address a request)
__device__ const ExpTable kExpTable;

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
        // (every step rounded by itself, as for float pairs at large)
        const float x = __fmul_rn(logit, pre);
        const float ds = __fsub_rn(x, top);  // and the subtraction's rounding error
        const float v = __fsub_rn(ds, x);
        const float dl = __fmul_rn(__fsub_rn(__fsub_rn(x, __fsub_rn(ds, v)), __fadd_rn(top, v)), post);
        const float dh = __fmul_rn(ds, post);
        const float yh = __fmul_rn(dh, r.hi);
        if (!(yh > -100.0f)) return FF{0.0f, 0.0f};
        const float yl = __fadd_rn(__fmaf_rn(dh, r.hi, -yh), __fmaf_rn(dl, r.hi, __fmul_rn(dh, r.lo)));
        const float magic = __fmaf_rn(yh, static_cast<float>(kTable), 12582912.0f);  // 1.5 * 2^23: rounds to a whole number
        const int k = __float_as_int(magic) - 0x4B400000;
        const float g0 = __fmaf_rn(__fsub_rn(magic, 12582912.0f), -1.0f / kTable, yh);  // exact
        const float g = __fadd_rn(g0, yl), gl = __fsub_rn(yl, __fsub_rn(g, g0));
        const float zh = __fmul_rn(g, kLn2);
        const float zl = __fadd_rn(__fmaf_rn(g, kLn2, -zh), __fmaf_rn(g, kLn2Lo, __fmul_rn(gl, kLn2)));
        const float sq = __fmul_rn(zh, zh), half = __fmul_rn(0.5f, sq), sql = __fmaf_rn(zh, zh, -sq);
        const float rest = sq * zh * __fmaf_rn(zh, 1.0f / 24, 1.0f / 6);  // of the series, beyond the square
        const float u = __fadd_rn(zh, half);  // 2^(g + gl) = 1 + u + ul
        const float ul = __fsub_rn(half, __fsub_rn(u, zh)) + (rest + (zl + __fmaf_rn(zh, zl, 0.5f * sql)));
        const float2 t = table[k & (kTable - 1)];
        const float ph = __fmul_rn(t.x, u), pl = __fmaf_rn(t.x, u, -ph);
        const float s = __fadd_rn(t.x, ph);
        const float lo = __fsub_rn(ph, __fsub_rn(s, t.x)) + (pl + (t.y + __fmaf_rn(t.x, ul, t.y * u)));
        const float scale = __int_as_float(((k >> 8) + 127) << 23);
        const float hi = __fadd_rn(s, lo);  // normalised, as comparisons with it need
        return FF{__fmul_rn(hi, scale), __fmul_rn(__fsub_rn(lo, __fsub_rn(hi, s)), scale)};
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
    uint32_t ctas;   // of a row's cluster
    uint32_t share;  // vectors a CTA takes
};

constexpr uint32_t kEntries = 2048;             // at most; of up to four units, a lane a bin
constexpr uint32_t kCoarse = kEntries / kWarps;  // entries of a warp's prefix sums
// Entries of a share's list. Twice as many cost the L1 cache 12 KB more, and rows
// that list nothing 7 % (152 of 202,048 without top-k: 41.5 -> 44.7 us).
constexpr uint32_t kList = 2048;
static_assert(kUnits <= kEntries * 4 && kCoarse == 64);

struct Shared {
    uint32_t hist[kBins / 2];
    uint16_t units[kUnits];   // the row's non-empty units, in bin order
    float2 table[kTable];
    uint32_t entry_c[kEntries];  // in the row's first CTA: counts and masses of the entries,
    FF entry_m[kEntries];        // then up to and with each entry within its 64
    uint32_t bits[kWords];    // occupancy: bit l of word w is unit 32 w + l
    uint32_t off[kWords];
    uint32_t row_bits[kWords];
    FF warp_m[kWarps];        // of 64 entries
    uint32_t warp_c[kWarps];
    uint32_t seg[kWarps];
    uint32_t heavy[kMaxHeavy];  // bins with 32,768 ids more than their counter says, once for each
    uint32_t heavies, counted, n_bits, any_heavy;
    uint32_t list_at[kList];  // ids past the first batch that the bound lets through: 8 times the vector and the place,
    uint16_t list_pattern[kList];  // and logits (0 for -0)
    Weights weights;
    uint32_t n_min;           // ids that min-p leaves
    uint32_t listed, matches;  // (listed: kList and more when some found no place)
    uint32_t top, row_top;    // the share's and the row's largest logit, by f2key; all ones for a NaN
    uint32_t bin, owner, place;  // the drawn bin, the CTA of the drawn id, its place among that CTA's ids of the bin
    float prob;
};

// A vector of 16 bytes where `on` holds, else four times `fill`: without a
// branch, so that a thread's loads are all on their way together.
__device__ __forceinline__ uint4 load_or(const void* p, bool on, uint32_t fill) {
    uint4 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %5, 0;\n\t"
        "mov.b32 %0, %6;\n\tmov.b32 %1, %6;\n\tmov.b32 %2, %6;\n\tmov.b32 %3, %6;\n\t"
        "@p ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"(static_cast<uint32_t>(on)), "r"(fill));
    return v;
}

// A CTA's share of a row, as 16-byte vectors from the aligned address at or
// below the row's start; `skew` ids of the first vector are not the row's.
template <typename T>
struct Share {
    const uint16_t* x;
    uint32_t V, skew, lo, hi;  // vectors [lo, hi)

    // Vector v where it reaches over an end of the row: by element, -Inf (a masked
    // id) outside.
    __device__ __forceinline__ uint4 edge(uint32_t v) const {
        constexpr uint32_t kNegInf = 0x8000u | Kind<T>::kInf;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t e = static_cast<int64_t>(v) * 8 - skew + 2 * i + h;
                w[i] |= (e >= 0 && e < V ? x[e] : kNegInf) << (16 * h);
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // f(v, logits) for vectors base + me, + kStride, ... below end, kAhead at a time
    // with the next ones on their way. Every thread calls it for all kAhead, past
    // the end with masked ids.
    template <uint32_t kStride, typename F>
    __device__ __forceinline__ void each(uint32_t base, uint32_t end, uint32_t me, F f) const {
        constexpr uint32_t kNegInf = 0x8000u | Kind<T>::kInf, kFill = kNegInf | (kNegInf << 16);
        const uint32_t full_lo = skew ? 1u : 0u, full_hi = (V + skew) / 8u;
        const uint16_t* origin = x - skew;
        uint4 next[kAhead];
        auto load = [&](uint32_t v) {
            return load_or(origin + static_cast<uint64_t>(v) * 8u, v >= full_lo && v < full_hi && v < end, kFill);
        };
#pragma unroll
        for (int j = 0; j < kAhead; ++j) next[j] = load(base + j * kStride + me);
        for (uint32_t at = base + me; at - me < end; at += kAhead * kStride) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const uint32_t v = at + j * kStride;
                uint4 q = next[j];
                next[j] = load(v + kAhead * kStride);
                if (v < end && (v < full_lo || v >= full_hi)) q = edge(v);
                f(v, q);
            }
        }
    }
    // f(v, logits) for the vectors of [base, end) in any order, thread `me` of
    // kStride taking every kStride-th, kDepth ahead. f gets vectors of masked ids
    // too; a row's end vectors, which reach over it, come in a step of their own.
    template <uint32_t kStride, uint32_t kDepth, typename F>
    __device__ __forceinline__ void sweep(uint32_t base, uint32_t end, uint32_t me, F f) const {
        constexpr uint32_t kNegInf = 0x8000u | Kind<T>::kInf, kFill = kNegInf | (kNegInf << 16);
        const uint32_t full_lo = skew ? 1u : 0u, full_hi = (V + skew) / 8u;
        const uint32_t lo = max(base, full_lo), hi = max(lo, min(end, full_hi));
        const bool edges = base < full_lo || end > full_hi;
        int left = static_cast<int>(hi - lo) - static_cast<int>(me) + (edges ? static_cast<int>(kStride) : 0);
        const char* p = reinterpret_cast<const char*>(x - skew) + (static_cast<int64_t>(lo) + me) * 16 -
                        (edges ? static_cast<int64_t>(kStride) * 16 : 0);
        uint4 next[kDepth];
#pragma unroll
        for (uint32_t j = 0; j < kDepth; ++j)
            next[j] = load_or(p + j * kStride * 16u, left > static_cast<int>(j * kStride) && !(edges && j == 0), kFill);
        if (edges && me < 2) {
            const uint32_t v = me ? full_hi : 0u;
            if (v >= base && v < end && (me ? full_hi >= full_lo : skew != 0)) next[0] = edge(v);
        }
        while (left > 0) {
#pragma unroll
            for (uint32_t j = 0; j < kDepth; ++j) {
                const uint4 q = next[j];
                next[j] = load_or(p + (kDepth + j) * kStride * 16u, left > static_cast<int>((kDepth + j) * kStride), kFill);
                const int v = static_cast<int>(hi) - left + static_cast<int>(j * kStride);
                f(v >= static_cast<int>(lo) ? static_cast<uint32_t>(v) : me ? full_hi : 0u, q);
            }
            p += kDepth * kStride * 16u;
            left -= static_cast<int>(kDepth * kStride);
        }
    }
};

// Ids of a unit's eight counters.
__device__ __forceinline__ uint32_t unit_sum(const uint4& v) {
    return (v.x & 0xFFFFu) + (v.x >> 16) + (v.y & 0xFFFFu) + (v.y >> 16) + (v.z & 0xFFFFu) + (v.z >> 16) + (v.w & 0xFFFFu) +
           (v.w >> 16);
}
// Inclusive sums over the warp's lanes.
__device__ __forceinline__ uint32_t warp_scan(uint32_t v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t n = __shfl_up_sync(kFull, v, o);
        if ((threadIdx.x & 31) >= static_cast<uint32_t>(o)) v += n;
    }
    return v;
}
__device__ __forceinline__ uint32_t ceil_div32(uint32_t a, uint32_t b) { return (a + b - 1) / b; }

template <typename T>
__global__ void __launch_bounds__(kNT, 1) sample16_kernel(SampleArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Shared& s = *reinterpret_cast<Shared*>(smem_raw);
    cg::cluster_group cl = cg::this_cluster();
    const uint32_t C = a.ctas, rank = C > 1 ? cl.block_rank() : 0u;
    const uint32_t row = blockIdx.x / C;
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr uint32_t kPosInf = 0x7FFFu - Kind<T>::kInf;     // lower bins: NaN
    constexpr uint32_t kNegInf = 0x8000u | Kind<T>::kInf;     // masked; higher bins: NaN
    auto cluster_sync = [&] {
        if (C > 1) cl.sync();
        else __syncthreads();
    };
    auto peer = [&](auto* p, uint32_t r) { return C > 1 ? cl.map_shared_rank(p, r) : p; };

    uint4* h4 = reinterpret_cast<uint4*>(s.hist);
    auto clear = [&] {
#pragma unroll
        for (int i = 0; i < static_cast<int>(kUnits / kNT); ++i) h4[i * kNT + tid] = make_uint4(0, 0, 0, 0);
    };
    clear();
    if (tid < kTable) s.table[tid] = kExpTable.v[tid];
    if (tid == 0) s.n_min = s.heavies = s.counted = s.n_bits = s.any_heavy = s.top = s.row_top = s.listed = s.matches = 0;
    pdl_wait();

    Share<T> share;
    share.x = static_cast<const uint16_t*>(a.logits) + static_cast<uint64_t>(row) * a.ld;
    share.V = a.V;
    share.skew = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(share.x) & 15u) / 2u;
    share.lo = rank * a.share;
    share.hi = max(share.lo, min((a.V + share.skew + 7u) / 8u, share.lo + a.share));
    const float Tf = a.temperature ? a.temperature[row] : 1.0f;
    const uint32_t kk = a.top_k ? a.top_k[row] : 0u;
    const float pf = a.top_p ? a.top_p[row] : 1.0f;
    const float mf = a.min_p ? a.min_p[row] : 0.0f;
    const float uf = a.uniforms[row];
    pdl_trigger();
    __syncthreads();  // the histogram is clear

    // The thread's largest logits, NaN once it has seen one: all that a row's
    // validity needs. (Masked ids and those outside the row are -Inf.)
    typename Kind<T>::Pair top = as_pair<T>(kNegInf * 0x00010001u);
    // Counting. The counter of pattern u is half u & 1 of word u >> 1. Ids are added
    // under a predicate: branches took twice the instructions of all the rest.
    const uint32_t hist = smem_u32(s.hist);
    auto add = [&](uint32_t w, uint32_t in) {  // the halves of w whose half of `in` is all ones
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t.reg .b32 t;\n\t"
            "and.b32 t, %4, 1;\n\tsetp.ne.u32 p, t, 0;\n\tsetp.lt.s32 q, %4, 0;\n\t"
            "@p red.shared.add.u32 [%0], %1;\n\t"
            "@q red.shared.add.u32 [%2], %3;\n\t}" ::"r"(hist + ((w & 0xFFFEu) << 1)),
            "r"(1u + (w & 1u) * 0xFFFFu), "r"(hist + ((w >> 17) << 2)), "r"(max(w & 0x10000u, 1u)), "r"(in)
            : "memory");
    };
    // Halves that are all ones in the masks that `sum` adds up (fewer than 65,536 each).
    auto halves = [](uint32_t sum) {
        const uint32_t low = -sum & 0xFFFFu;  // sum = 65535 low - 65536 high
        return low + ((65535u * low - sum) >> 16);
    };
    auto largest = [&](const uint4& q) {
        return __hmax2_nan(__hmax2_nan(as_pair<T>(q.x), as_pair<T>(q.y)), __hmax2_nan(as_pair<T>(q.z), as_pair<T>(q.w)));
    };
    // Counts the unmasked ids; returns how many the thread counted.
    auto count_all = [&](uint32_t base, uint32_t end) {
        uint32_t sum = 0;
        share.template sweep<kNT, kAhead>(base, end, tid, [&](uint32_t, const uint4& q) {
            top = __hmax2_nan(top, largest(q));
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t in = differ2<T>(w[i], kNegInf * 0x00010001u);
                sum += in;
                add(w[i], in);
            }
        });
        return halves(sum);
    };
    // The same of ids that are not below `bound` (a pair of the same pattern).
    // note: they go into the list.
    auto count_from = [&](uint32_t base, uint32_t end, uint32_t bound, bool note) {
        uint32_t sum = 0;
        const auto low = as_pair<T>(bound);
        share.template sweep<kNT, kAheadFrom>(base, end, tid, [&](uint32_t v, const uint4& q) {
            const auto most = largest(q);
            top = __hmax2_nan(top, most);
            if (!not_below2<T>(most, low)) return;
            uint32_t which = 0;
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t in = not_below2<T>(as_pair<T>(w[i]), low);
                sum += in;
                add(w[i], in);
            }
            if (!note) return;
#pragma unroll
            for (int i = 0; i < 4; ++i) which |= (not_below2<T>(as_pair<T>(w[i]), low) & 0x10001u) << i;
            while (which && *const_cast<volatile uint32_t*>(&s.listed) < kList) {  // bit i + 16 h: half h of word i
                const uint32_t b = __ffs(which) - 1, k = b & 3;
                which &= which - 1;
                const uint32_t u = (k & 2 ? (k & 1 ? q.w : q.z) : (k & 1 ? q.y : q.x)) >> (b & 16) & 0xFFFFu;
                const uint32_t i = atomicAdd(&s.listed, 1u);
                if (i < kList) {
                    s.list_at[i] = v * 8 + 2 * k + (b >> 4);
                    s.list_pattern[i] = static_cast<uint16_t>(u == 0x8000u ? 0u : u);
                }
            }
        });
        return halves(sum);
    };
    // fewer than 65,536 ids: no counter can overflow
    const bool small = share.hi - share.lo <= kBatchVecs * 2;
    // ids of the row that can matter, from the largest
    const uint32_t want = Tf == 0.0f ? 1u : kk && kk < kBatchVecs * 8 ? kk : a.V;
    uint32_t bound = (kNegInf - 1) * 0x00010001u;  // a pair of the least pattern that counts: the least finite one
    uint32_t last_unit = kUnits - 1;  // that holds one: later units' masses are not needed
    if (tid == 32) s.weights.temperature(Tf > 0.0f ? Tf : 1.0f);
    // The top `want` ids of a first batch bound those of the row from below: the
    // rest of the share only counts what is not under them. (A 64th of the batch,
    // where it can be: the bound then lets about that much through.)
    uint32_t at = share.hi;  // the first batch's end
    if (!small && want < kBatchVecs * 8) at = share.lo + min(kBatchVecs, max(2 * static_cast<uint32_t>(kNT), want * 8u));
    // Where the bound lets few through, they are listed, so that the drawn id need
    // not be looked for in the rest of the share (152 rows of 202,048, top 40: 36.7
    // -> 32.5 us, greedy 29 -> 19).
    const bool listing = at < share.hi && want * static_cast<uint64_t>(share.hi - at) <= kList / 2 * (at - share.lo);
    uint32_t n = count_all(share.lo, at);
    if (at < share.hi) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < static_cast<int>(kUnits / kNT); ++i) {
            const uint32_t word = warp * (kUnits / kNT) + i;
            const uint32_t sum = __reduce_add_sync(kFull, unit_sum(h4[stored_unit(word * 32 + lane)]));
            if (lane == 0) s.off[word] = sum;
        }
        __syncthreads();
        // every warp finds the same: the 256 bins where the count gets there, then their unit
        uint32_t sum = 0;
#pragma unroll
        for (uint32_t i = 0; i < kWords / 32; ++i) sum += s.off[lane * (kWords / 32) + i];
        const uint32_t in = warp_scan(sum), hit = __ballot_sync(kFull, in >= want);
        if (hit) {
            const int l = __ffs(hit) - 1;
            uint32_t before = __shfl_sync(kFull, in - sum, l), word = l * (kWords / 32);
            while (before + s.off[word] < want) before += s.off[word++];
            const uint32_t units = warp_scan(unit_sum(h4[stored_unit(word * 32 + lane)]));
            const uint32_t unit = word * 32 + __ffs(__ballot_sync(kFull, before + units >= want)) - 1;
            last_unit = unit;
            // (the unit's least value, from +Inf to the least finite one: no NaN, with
            // which every comparison would let -Inf through)
            bound = pattern_of(max(kPosInf, min(unit * kUnitBins + kUnitBins - 1, kNegInf - 1))) * 0x00010001u;
        }
        __syncthreads();
        n += count_from(at, share.hi, bound, listing);
    }
    if (!small) {
        n = __reduce_add_sync(kFull, n);
        if (lane == 0) atomicAdd(&s.counted, n);
    }
    {
        // as a whole number in the order of the values, NaN above all
        const float x0 = to_f32(top.x), x1 = to_f32(top.y);
        const uint32_t key = isnan(x0) || isnan(x1) ? 0xFFFFFFFFu : f2key(fmaxf(x0, x1));
        const uint32_t most = __reduce_max_sync(kFull, key);
        if (lane == 0) atomicMax(&s.top, most);
    }
    __syncthreads();
    auto merge_zeros = [&] {  // -0 ties with +0: its pattern, 0x8000, is counted with 0
        const uint32_t neg = s.hist[0x8000 / 2] & 0xFFFFu;
        if ((s.hist[0] & 0xFFFFu) + neg < 65536u) {
            s.hist[0x8000 / 2] -= neg;
            s.hist[0] += neg;
        } else {
            s.counted = 0;  // counted again below
        }
    };
    if (tid == 0) merge_zeros();
    __syncthreads();
    auto occupancy = [&] {
        uint32_t sum = 0;
#pragma unroll
        for (int i = 0; i < static_cast<int>(kUnits / kNT); ++i) {
            const uint32_t word = i * kWarps + warp;
            const uint4 v = h4[stored_unit(word * 32 + lane)];
            const uint32_t b = __ballot_sync(kFull, (v.x | v.y | v.z | v.w) != 0 && word * 32 + lane <= last_unit);
            if (lane == 0) s.bits[word] = b;
            sum += unit_sum(v);
        }
        return __reduce_add_sync(kFull, sum);
    };
    if (small) {
        (void)occupancy();
        __syncthreads();
    } else {
        const uint32_t sum = occupancy();
        if (lane == 0) atomicAdd(&s.n_bits, sum);
        __syncthreads();
        if (s.n_bits != s.counted) {
            // Some counter overflowed (each overflow takes 65,535 or 65,536 from the
            // sum): again in batches, none of which overflows a counter below half.
            __syncthreads();
            clear();
            __syncthreads();
            for (uint32_t b = share.lo; b < share.hi; b += kBatchVecs) {
                count_from(b, min(share.hi, b + kBatchVecs), bound, false);
                __syncthreads();
                if (tid == 0) merge_zeros();
                __syncthreads();
                for (uint32_t i = tid; i < kBins / 2; i += kNT) {
                    const uint32_t w = s.hist[i], over = w & 0x80008000u;
                    if (over) {
                        s.hist[i] = w - over;
                        if (over & 0x8000u) s.heavy[atomicAdd(&s.heavies, 1u)] = pattern_of(2 * i);
                        if (over >> 31) s.heavy[atomicAdd(&s.heavies, 1u)] = pattern_of(2 * i + 1);
                    }
                }
                __syncthreads();
            }
            (void)occupancy();
            __syncthreads();
            if (tid < s.heavies) atomicOr(&s.bits[s.heavy[tid] / (kUnitBins * 32)], 1u << (s.heavy[tid] / kUnitBins % 32));
        }
    }
    cluster_sync();

    // The row's non-empty units, in order.
    if (tid < kWords) {
        uint32_t word = 0;
        for (uint32_t r = 0; r < C; ++r) word |= peer(s.bits, r)[tid];
        const uint32_t in = warp_scan(__popc(word));
        s.off[tid] = in;  // up to and with this word, in its 32
        s.row_bits[tid] = word;
    } else if (tid < kWords + C) {
        if (*peer(&s.heavies, tid - kWords)) s.any_heavy = 1;
        atomicMax(&s.row_top, *peer(&s.top, tid - kWords));
    }
    __syncthreads();
    uint32_t nu = 0;
#pragma unroll
    for (int i = 0; i < static_cast<int>(kUnits / kNT); ++i) {
        const uint32_t w = i * kWarps + warp, m = s.row_bits[w], before = s.off[w] - __popc(m);
        if (m >> lane & 1) s.units[nu + before + __popc(m & ((1u << lane) - 1u))] = static_cast<uint16_t>(w * 32 + lane);
        nu += s.off[i * kWarps + 31];
    }
    __syncthreads();

    const bool any_heavy = s.any_heavy != 0;
    auto heavy_of = [&](uint32_t bin, uint32_t r) {  // ids of CTA r that its counter leaves out
        uint32_t n = 0;
        const uint32_t* heavy = peer(s.heavy, r);
        for (uint32_t i = 0; i < *peer(&s.heavies, r); ++i) n += heavy[i] == bin ? kHalf : 0u;
        return n;
    };
    auto count_of = [&](uint32_t bin, uint32_t r) {  // in CTA r
        const uint32_t n = reinterpret_cast<const uint16_t*>(peer(s.hist, r))[pattern_of(bin)];
        return any_heavy ? n + heavy_of(bin, r) : n;
    };
    auto count = [&](uint32_t bin) {  // over the row; the loads of all CTAs on their way together
        if (C == 1) return count_of(bin, 0);
        uint32_t v[kMaxCluster], n = 0;
#pragma unroll
        for (uint32_t r = 0; r < kMaxCluster; ++r)
            v[r] = r < C ? reinterpret_cast<const uint16_t*>(cl.map_shared_rank(s.hist, r))[pattern_of(bin)] : 0u;
#pragma unroll
        for (uint32_t r = 0; r < kMaxCluster; ++r) n += v[r];
        if (any_heavy)
            for (uint32_t r = 0; r < C; ++r) n += heavy_of(bin, r);
        return n;
    };
    // The policy, and the row's validity: a NaN or +Inf logit, nothing unmasked, a
    // uniform or a parameter out of its range; the same in every CTA of the cluster.
    const bool bad = !(Tf >= 0.0f) || isinf(Tf) || !(pf > 0.0f && pf <= 1.0f) || !(mf >= 0.0f && mf < 1.0f) ||
                     !(uf >= 0.0f && uf < 1.0f) || nu == 0 || s.row_top > kKeyMaxFinite;
    if (bad) {
        if (rank == 0 && tid == 0) {
            a.out_ids[row] = SEL_INVALID_ID;
            a.out_probs[row] = __uint_as_float(0x7FC00000u);
        }
        cluster_sync();  // no CTA leaves while another reads its tables
        return;
    }
    const float row_top = key2f(s.row_top);
    const bool greedy = Tf == 0.0f;
    Weights weights = s.weights;
    weights.top = row_top * weights.pre;

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
                peer(s.entry_c, 0)[e] = c;
                peer(s.entry_m, 0)[e] = m;
            }
        }
        n_min = __reduce_add_sync(kFull, n_min);
        if (lane == 0 && n_min) atomicAdd(peer(&s.n_min, 0), n_min);
    }
    cluster_sync();

    if (rank == 0) {
        if (!greedy) {
            // prefix sums of each 64 entries, two a lane
            const uint32_t e = 2 * tid;
            const uint32_t c0 = e < entries ? s.entry_c[e] : 0u, c1 = e + 1 < entries ? s.entry_c[e + 1] : 0u;
            const FF m0 = e < entries ? s.entry_m[e] : FF{0.0f, 0.0f};
            const FF m1 = e + 1 < entries ? s.entry_m[e + 1] : FF{0.0f, 0.0f};
            const uint32_t wc = warp_scan(c0 + c1);
            const FF both = ff_add(m0, m1);
            const FF wm = ff_warp_scan(both);
            FF before = ff_shfl_up(wm, 1);
            if (lane == 0) before = FF{0.0f, 0.0f};
            s.entry_c[e] = wc - c1;
            s.entry_c[e + 1] = wc;
            s.entry_m[e] = ff_add(before, m0);
            s.entry_m[e + 1] = wm;
            if (lane == 31) {
                s.warp_c[warp] = wc;
                s.warp_m[warp] = wm;
            }
            __syncthreads();
        }
        if (warp == 0) {
            // sums up to and with the lane's 64 entries, and before them
            uint32_t seg_c = 0, seg_c0 = 0;
            FF seg_m{0.0f, 0.0f}, seg_m0{0.0f, 0.0f};
            if (!greedy) {
                seg_c = warp_scan(s.warp_c[lane]);
                seg_m = ff_warp_scan(s.warp_m[lane]);
                seg_c0 = __shfl_up_sync(kFull, seg_c, 1);
                seg_m0 = ff_shfl_up(seg_m, 1);
                if (lane == 0) {
                    seg_c0 = 0;
                    seg_m0 = FF{0.0f, 0.0f};
                }
            }
            const uint32_t n_all = __shfl_sync(kFull, seg_c, 31);
            const FF m_all = ff_shfl(seg_m, 31);
            // Lane l holds bin l of an entry's up to 32; sums before and with it.
            struct Bins {
                uint32_t bin, c, c_before, c_in;
                FF w, m_before, m_in;
            };
            // The bins of the first entry for which past(count, mass up to and with
            // it) holds, of the last one when none does.
            auto open = [&](auto past) {
                const uint32_t coarse = __ballot_sync(kFull, past(seg_c, seg_m));
                const int sg = coarse ? __ffs(coarse) - 1 : 31;
                const uint32_t c0 = __shfl_sync(kFull, seg_c0, sg);
                const FF m0 = ff_shfl(seg_m0, sg);
                uint32_t e = sg * kCoarse + kCoarse - 1;
#pragma unroll
                for (int i = static_cast<int>(kCoarse / 32) - 1; i >= 0; --i) {
                    const uint32_t at = sg * kCoarse + i * 32 + lane;
                    const uint32_t fine = __ballot_sync(kFull, past(c0 + s.entry_c[at], ff_add(m0, s.entry_m[at])));
                    if (fine) e = sg * kCoarse + i * 32 + __ffs(fine) - 1;
                }
                e = min(e, entries - 1);
                const uint32_t first = e / kCoarse * kCoarse;  // (e may lie before the segment by that)
                uint32_t c_base = __shfl_sync(kFull, seg_c0, e / kCoarse);
                FF m_base = ff_shfl(seg_m0, e / kCoarse);
                if (e > first) {
                    c_base += s.entry_c[e - 1];
                    m_base = ff_add(m_base, s.entry_m[e - 1]);
                }
                Bins b{};
                const uint32_t i = e * per + lane / 8;
                FF m{0.0f, 0.0f};
                if (lane / 8 < per && i < nu) {
                    b.bin = s.units[i] * kUnitBins + lane % 8;
                    b.c = count(b.bin);
                    b.w = weights(bin_value<T>(b.bin), s.table);
                    if (b.c) m = ff_mul_f(b.w, static_cast<float>(b.c));
                }
                b.c_in = c_base + warp_scan(b.c);
                b.c_before = b.c_in - b.c;
                b.m_in = ff_add(m_base, ff_warp_scan(m));
                b.m_before = ff_shfl_up(b.m_in, 1);
                if (lane == 0) b.m_before = m_base;
                return b;
            };
            auto prefix_mass = [&](uint32_t n) {  // of the first n ids of the order
                if (n == n_all) return m_all;
                const Bins b = open([&](uint32_t c, FF) { return c >= n; });
                const int l = __ffs(__ballot_sync(kFull, b.c_in >= n)) - 1;
                return ff_shfl(ff_add(b.m_before, ff_mul_f(b.w, static_cast<float>(n - b.c_before))), l);
            };
            // The first id whose cumulative mass reaches `goal` (over: exceeds
            // it): its lane, its place among the bin's ids; and its rank.
            auto by_mass = [&](FF goal, bool over, Bins& b, uint32_t& place, int& l) {
                auto past = [&](FF m) { return over ? ff_lt(goal, m) : !ff_lt(m, goal); };
                b = open([&](uint32_t, FF m) { return past(m); });
                const uint32_t hit = __ballot_sync(kFull, b.c > 0 && past(b.m_in));
                // (rounding may leave none: the entry's last id)
                l = hit ? __ffs(hit) - 1 : 31 - __clz(__ballot_sync(kFull, b.c > 0));
                // The r-th id of the bin (from 0) ends at m_before + (r + 1) w: r to
                // within one from the quotient of the leading floats, then the first
                // of its neighbourhood that is past.
                const FF gap = ff_add(goal, FF{-b.m_before.hi, -b.m_before.lo});
                float r = fminf(fmaxf(floorf(gap.hi / b.w.hi) - 2.0f, 0.0f), static_cast<float>(b.c) - 1.0f);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (r + 1.0f < static_cast<float>(b.c) && !past(ff_add(b.m_before, ff_mul_f(b.w, r + 1.0f)))) r += 1.0f;
                place = __shfl_sync(kFull, hit ? static_cast<uint32_t>(fmaxf(r, 0.0f)) : b.c - 1u, l);
                return __shfl_sync(kFull, b.c_before, l) + place;
            };

            uint32_t bin = bin_of<T>(row_top), place = 0;  // greedy: the largest logit's first id
            float prob = 1.0f;
            if (!greedy) {
                const uint32_t n_k = kk == 0 ? n_all : min(kk, n_all);
                const FF Z = prefix_mass(n_k);
                uint32_t n = min(n_k, s.n_min);
                Bins b;
                int l;
                if (pf < 1.0f) n = min(n, by_mass(ff_mul_f(Z, pf), false, b, place, l) + 1u);
                const FF Zs = n == n_k ? Z : prefix_mass(n);
                if (by_mass(ff_mul_f(Zs, uf), true, b, place, l) >= n) {
                    // rounding: the last survivor
                    b = open([&](uint32_t c, FF) { return c >= n; });
                    l = __ffs(__ballot_sync(kFull, b.c_in >= n)) - 1;
                    place = __shfl_sync(kFull, n - 1u - b.c_before, l);
                }
                bin = __shfl_sync(kFull, b.bin, l);
                const FF w = ff_shfl(b.w, l);
                // w / Zs, rounded once: the quotient of the leading floats and its remainder
                const float q0 = w.hi / Zs.hi;
                prob = q0 + (__fmaf_rn(-q0, Zs.hi, w.hi) + __fmaf_rn(-q0, Zs.lo, w.lo)) / Zs.hi;
            }
            // the CTA that holds it: ids rise with the CTAs
            const uint32_t c = lane < C ? count_of(bin, lane) : 0u;
            const uint32_t in = warp_scan(c);
            const int owner = __ffs(__ballot_sync(kFull, place < in)) - 1;
            place = __shfl_sync(kFull, place - (in - c), owner);
            if (lane < C) {
                Shared& o = *peer(&s, lane);
                o.bin = bin;
                o.owner = owner;
                o.place = place;
                o.prob = prob;
            }
        }
    }
    cluster_sync();
    if (rank != s.owner) return;

    // The place-th id of the bin in this CTA's share: each warp counts the bin's
    // ids in a run of vectors of its own, then the warp that has the id goes
    // through its run again. Where the ids past the first batch are listed, in that
    // batch only, and then in the list.
    const bool in_list = listing && s.listed < kList;
    const uint32_t find_hi = in_list ? at : share.hi;
    const uint32_t pattern = pattern_of(s.bin) * 0x00010001u;
    const uint32_t run = ceil_div32(find_hi - share.lo, kWarps);
    const uint32_t run_lo = min(find_hi, share.lo + warp * run), run_hi = min(find_hi, run_lo + run);
    uint32_t mine;
    {
        // A lane sees up to 64 whole vectors and an end of the row: 260 ids a half, of
        // which each sum takes 130. Either type holds whole numbers up to 256. (Masks
        // added up in the integer pipe instead: 1 % slower at 256 rows of 202,048.)
        static_assert((SEL_SAMPLE16_MAX_V / (8 * 32 * kWarps) + 2) * 2 <= 256);
        auto sum_xy = as_pair<T>(0), sum_zw = as_pair<T>(0);
        const auto drawn = as_pair<T>(pattern);
        share.template sweep<32, kAheadFrom>(run_lo, run_hi, lane, [&](uint32_t, const uint4& q) {
            sum_xy = __hadd2(sum_xy, __hadd2(__heq2(as_pair<T>(q.x), drawn), __heq2(as_pair<T>(q.y), drawn)));
            sum_zw = __hadd2(sum_zw, __hadd2(__heq2(as_pair<T>(q.z), drawn), __heq2(as_pair<T>(q.w), drawn)));
        });
        mine = __reduce_add_sync(kFull, static_cast<uint32_t>(to_f32(sum_xy.x) + to_f32(sum_xy.y) + to_f32(sum_zw.x) +
                                                              to_f32(sum_zw.y)));
    }
    if (lane == 0) s.seg[warp] = mine;
    __syncthreads();
    const uint32_t in = warp_scan(s.seg[lane]);
    const uint32_t place = s.place;
    const uint32_t has = __ballot_sync(kFull, place < in);
    if (!has) {  // (the same in every warp; with a list only)
        uint32_t* match = s.hist;  // which nothing reads any more
        const uint32_t rank_in_list = place - __shfl_sync(kFull, in, 31);
        const uint32_t wanted = pattern & 0xFFFFu;
        for (uint32_t i = tid; i < s.listed; i += kNT)
            if (s.list_pattern[i] == wanted) match[atomicAdd(&s.matches, 1u)] = s.list_at[i];
        __syncthreads();
        const uint32_t n = s.matches;
        for (uint32_t i = tid; i < n; i += kNT) {
            uint32_t before = 0;
            for (uint32_t j = 0; j < n; ++j) before += match[j] < match[i];
            if (before == rank_in_list) {
                a.out_ids[row] = match[i] - share.skew;
                a.out_probs[row] = s.prob;
            }
        }
        return;
    }
    if (static_cast<int>(warp) != __ffs(has) - 1) return;
    uint32_t left = place - (__shfl_sync(kFull, in, warp) - mine);  // ids of the bin before it in the run
    bool found = false;
    share.template each<32>(run_lo, run_hi, lane, [&](uint32_t v, const uint4& q) {
        if (found) return;
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        uint32_t which = 0;  // bit i: id i of the vector
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t f = equal2<T>(w[i], pattern);
            which |= (f & 1u) << (2 * i) | f >> 31 << (2 * i + 1);
        }
        const uint32_t n = __popc(which);
        const uint32_t upto = warp_scan(n);
        const uint32_t all = __shfl_sync(kFull, upto, 31);
        if (left >= all) {
            left -= all;
            return;
        }
        found = true;
        uint32_t skip = left - (upto - n);
        if (upto - n <= left && left < upto) {
            for (; skip > 0; --skip) which &= which - 1;
            a.out_ids[row] = v * 8u + __ffs(which) - 1 - share.skew;
            a.out_probs[row] = s.prob;
        }
    });
}

// CTAs a row for a batch: the cluster size whose rounds of resident clusters
// take least. A CTA takes 14.5 us beside its share, and 1 us for 10,000 ids (8,000
// without top-k, 12,000 where the rows' top-k is small).
template <typename T>
uint32_t ctas_for(uint32_t rows, uint32_t V) {
    struct Table {
        int resident[kMaxCluster + 1];  // clusters of that size on the device at a time
    };
    static PerDevice<Table> tables;
    Table t{};
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = -1;
    // (where a query fails, this call goes by the ones that did not)
    (void)tables.get(dev, t, [](Table& r) {
        bool ok = true;
        for (uint32_t c = 1; c <= kMaxCluster; ++c) {
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(c, 1, 1);
            cfg.blockDim = dim3(kNT, 1, 1);
            cfg.dynamicSmemBytes = sizeof(Shared);
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = c;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, sample16_kernel<T>, &cfg) != cudaSuccess || n < 0) {
                (void)cudaGetLastError();
                ok = false;
                n = 0;
            }
            r.resident[c] = n;
        }
        return ok;
    });
    uint32_t best = 1;
    double least = 1e30;
    for (uint32_t c = 1; c <= kMaxCluster; ++c) {
        if (t.resident[c] == 0) continue;
        const double rounds = ceil_div(rows, static_cast<uint64_t>(t.resident[c]));
        const double us = rounds * (14.5 + static_cast<double>(V) / c / 10000.0);
        if (us < least) {
            least = us;
            best = c;
        }
    }
    return best;
}

static_assert(sizeof(Shared) <= 227 * 1024);

template <typename T>
sel_status launch(const SampleArgs& in, uint32_t rows, cudaStream_t stream) {
    if (!dynamic_smem_once<sample16_kernel<T>>(sizeof(Shared))) return SEL_ECUDA;
    const uint32_t vecs = ceil_div(static_cast<uint64_t>(in.V) + 7, 8), C = ctas_for<T>(rows, in.V);
    if (static_cast<uint64_t>(rows) * C > 0x7fffffffull) return SEL_EUNSUPPORTED;
    SampleArgs a = in;
    a.ctas = C;
    a.share = ceil_div(vecs, C);
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
