// sel_head_loss.cu -- cross entropy through a 16-bit output head without its
// logits rows, and the gradient of that.
//
//   z = X W^T;  lse_r = ln sum_v exp z_rv;  loss_r = lse_r - z_r,t
//   P_rv = exp(z_rv - lse_r) - [v == t_r]
//   dX_r = g_r sum_v P_rv W_v;  dW_v = sum_r g_r P_rv X_r
//
// The loss is one product (sel_gemm.cuh) whose epilogue keeps two numbers of each row
// and 128 ids, or of each row and all ids of a worker: a reference exponent and the
// sum of the others' weights over it. A small launch joins them. The target's logit is
// kept apart, so that loss = ln(1 + sum_others / e^z_t) holds its bits near zero.
//
// The gradient goes over the vocabulary in pieces. For each, one launch computes
// z again and leaves P in the workspace, rounded to the operands' type; a second
// one computes the piece's rows of dW (K = rows) and adds the piece's share of
// dX (K = the piece) to fp32 sums.
//
// What bounds them: the matrix's bytes for few rows (49 of 4,096 x 248,320: 307 us,
// 6.6 TB/s; one of 1,024 x 151,936: 51.5), the tensor cores for many (4,096 rows: 98.5,
// 96.4 and 96.6 percent of their cycles in the three products; 4,096 x 151,936 in 2.70 ms
// in a short run and 2.79 in a long one, where the card's power limits it; the gradient of
// 2,048 x 151,936 in 4.34 and 4.49). Between them padding counts: 777 rows of 2,880 x
// 93,001 take 269 us and 313 (1.55 and 1.33 PFLOP/s), their gradient 899 and 951. The
// gradient of 64 rows of 1,024 x 151,936 takes 205, 55 for P and 130 for the rest: the
// matrix is read twice. Small calls are their chain of launches (256 rows of 128 x 8,000:
// 10 us on the GPU for two, the gradient 24 for three; the host needs 10 and 13).
#include <algorithm>

#include <cuda_runtime.h>

#include "sel_gemm.cuh"

using namespace sel;

namespace sel {
namespace {

constexpr float kLog2E = 1.4426950408889634f;

// Row tiles run fastest over up to 32 of them, then columns: the rows' operand
// stays in L2 while the matrix passes once.
struct Raster {
    uint32_t mt, nt;
    __device__ __forceinline__ void at(uint32_t i, uint32_t& m, uint32_t& n) const {
        constexpr uint32_t kGroup = 32;
        const uint32_t g = i / (kGroup * nt), r = i - g * kGroup * nt, gm = min(kGroup, mt - g * kGroup);
        n = r / gm;
        m = g * kGroup + r - n * gm;
    }
    __device__ __forceinline__ uint32_t share(uint32_t worker, uint32_t workers) const {
        const uint32_t n = mt * nt;
        return worker < n ? (n - worker - 1) / workers + 1 : 0;
    }
};

// Every workers-th tile of a raster.
template <typename P>
struct RasterCursor {
    const P& p;
    uint32_t worker, workers, count;
    __device__ __forceinline__ RasterCursor(const P& of, uint32_t w, uint32_t n)
        : p(of), worker(w), workers(n), count(of.raster.share(w, n)) {}
    __device__ __forceinline__ GemmTile tile(uint32_t j) const {
        uint32_t m, n;
        p.raster.at(worker + j * workers, m, n);
        return p.tile(m, n);
    }
};

// v 2^e for any e that floats and P's shift give.
struct Shift {
    float a, b;
    __device__ __forceinline__ explicit Shift(int e) {
        a = __int_as_float((e / 2 + 127) << 23);
        b = __int_as_float((e - e / 2 + 127) << 23);
    }
    __device__ __forceinline__ float operator()(float v) const { return v * a * b; }
};

__device__ __forceinline__ bool any_target(uint32_t t, uint32_t col) { return t - col < 32u; }

// A row of z in logarithms to base 2: sum over its ids but the target of 2^(y - m),
// m a whole number, so that sums of different tiles meet by exact shifts.
struct Part {
    float m, s;
};

// The reference for a largest logit `top`, and the weights under it.
struct Weights {
    float ref, k0, k1;
    __device__ __forceinline__ explicit Weights(float m) {
        ref = m == -INFINITY ? 0.0f : m;
        // The product z log2(e) is not rounded before the subtraction, but where
        // its rounding is no longer small next to 1 it has to be: then the largest
        // is m itself.
        const bool big = fabsf(ref) >= 1048576.0f;
        k0 = big ? kLog2E : 1.0f;
        k1 = big ? 1.0f : kLog2E;
    }
    __device__ __forceinline__ float operator()(float z) const { return ex2_approx(fmaf(z * k0, k1, -ref)); }
};

// The tensor cores round their sums towards zero, 16 products at a time: a logit of
// 4,096 products comes out 1.6e-6 too small, which a loss shows. So a logit is summed in
// parts of 1,024, joined in the epilogue's registers. (P and the gradients are rounded
// to 16 bits and take it as it comes: dX's sums over a piece's ids leave f16 gradients
// 2.2e-4 from the definition, where a product summed in fp32 leaves 2.1e-4.)
constexpr uint32_t kLossPart = 1024 / kStepK;

// Hidden rows on the product's rows: a lane has one of them, and half a tile's
// columns of z, so that its sum crosses no lanes. For rows that fill their tiles.
template <typename T>
struct LossProblem {
    using Type = T;
    static constexpr uint32_t kPart = kLossPart;
    CUtensorMap x, w;
    const uint32_t* targets;
    Part* parts;  // [2 column tiles][rows]
    float* at;    // [rows]: the target's logit
    uint32_t* error;
    uint32_t rows, V, steps;
    Raster raster;

    using Cursor = RasterCursor<LossProblem>;
    __device__ __forceinline__ void aside(uint32_t, uint32_t) const {}
    __device__ __forceinline__ GemmTile tile(uint32_t m, uint32_t n) const {
        return {&x, &w, m * kTileM, n * kTileN, 0, 0, steps, kTileN, false, false};
    }
    template <typename Arrive, typename Load>
    __device__ __forceinline__ void epilogue(const Cursor& cursor, const GemmTile& t, EpiWarp& w, Arrive arrived, Load load) const {
        const uint32_t row = t.am + w.row, col = t.bn + w.col;
        const uint32_t target = row < rows ? targets[row] : SEL_INVALID_ID;
        Part p{-INFINITY, 0.0f};
        arrived();
#pragma unroll
        for (uint32_t c = 0; c < 4; ++c) {
            if (c >= w.chunks) break;
            float v[32];
            load(c, v);
            const uint32_t c0 = col + 32 * c;
            if (any_target(target, c0)) {
#pragma unroll
                for (uint32_t i = 0; i < 32; ++i) {
                    if (target == c0 + i) {
                        if (target < V) at[row] = v[i];
                        v[i] = -INFINITY;
                    }
                }
            }
            if (c0 + 32 > V) {
#pragma unroll
                for (uint32_t i = 0; i < 32; ++i)
                    if (c0 + i >= V) v[i] = -INFINITY;
            }
            float top = v[0];
#pragma unroll
            for (uint32_t i = 1; i < 31; i += 2) top = max3f(top, v[i], v[i + 1]);
            top = fmaxf(top, v[31]);
            const float m = fmaxf(p.m, ceilf(top * kLog2E));
            const Weights e(m);
            float s[4] = {p.s * pow2(p.m - e.ref), 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (uint32_t i = 0; i < 32; ++i) s[i % 4] += e(v[i]);
            p.m = m;
            p.s = (s[0] + s[1]) + (s[2] + s[3]);
        }
        if (row < rows) parts[static_cast<uint64_t>(col / 128) * rows + row] = p;
    }
};

// Hidden rows on the product's columns, so that a tile has as few as 16 of them (one row
// of 1,024 x 151,936: 71 us on rows, 50 here; 777: 335 and 264): a lane has one id, and
// the logits of half a tile's rows for it. About 4 more instructions a logit for the
// sums across the lanes, which the product of one more row tile outweighs.

// Of 32 rows' values in each lane, the sums over the lanes: lane i gets row i's.
__device__ __forceinline__ float sum_across(float (&v)[32]) {
    const uint32_t lane = threadIdx.x & 31;
#pragma unroll
    for (uint32_t n = 16; n > 0; n >>= 1) {
        const bool up = lane & n;
#pragma unroll
        for (uint32_t i = 0; i < n; ++i) {
            const float keep = up ? v[i + n] : v[i], give = up ? v[i] : v[i + n];
            v[i] = keep + __shfl_xor_sync(kFull, give, n);
        }
    }
    return v[0];
}
__device__ __forceinline__ float max_across(float v) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(r) : "f"(v));  // (a NaN shows in the sums, not here)
    return r;
}

template <typename T>
struct LossColumnsProblem {
    using Type = T;
    static constexpr uint32_t kPart = kLossPart;
    CUtensorMap x, w;
    const uint32_t* targets;
    Part* parts;  // [8 workers of a row tile][rows]
    float* at;
    uint32_t* error;
    uint32_t rows, V, steps, n, row_tiles, v_tiles;

    __device__ __forceinline__ void aside(uint32_t, uint32_t) const {}
    // A worker stays with its row tile and keeps that one's sums from tile to tile;
    // neighbours take the same ids with the other row tiles.
    struct Cursor {
        const LossColumnsProblem& p;
        uint32_t row, v, step, count;
        __device__ __forceinline__ Cursor(const LossColumnsProblem& of, uint32_t worker, uint32_t workers) : p(of) {
            v = worker / p.row_tiles;
            row = worker - v * p.row_tiles;
            step = workers / p.row_tiles;
            count = v < p.v_tiles ? (p.v_tiles - v - 1) / step + 1 : 0;
        }
        __device__ __forceinline__ GemmTile tile(uint32_t j) const {
            return {&p.w, &p.x, (v + j * step) * kTileM, row * p.n, 0, 0, p.steps, p.n, false, false};
        }
    };
    template <typename Arrive, typename Load>
    __device__ __forceinline__ void epilogue(const Cursor& cursor, const GemmTile& t, EpiWarp& w, Arrive arrived, Load load) const {
        const uint32_t id = t.am + w.row, first = t.bn + w.col;
        auto* sums = reinterpret_cast<Part*>(w.smem) + w.lane;
        auto* wanted = reinterpret_cast<uint32_t*>(w.smem + 1024) + w.lane;  // targets of the rows, which stay
        if (w.j == 0) {
            for (uint32_t c = 0; c < w.chunks; ++c) {
                const uint32_t row = first + 32 * c + w.lane;
                wanted[32 * c] = 32 * c + w.lane < w.cols && row < rows ? targets[row] : SEL_INVALID_ID;
            }
        }
        arrived();
#pragma unroll
        for (uint32_t c = 0; c < 4; ++c) {
            if (c >= w.chunks) break;
            const uint32_t row = first + 32 * c + w.lane;  // whose result this lane will have
            const bool mine = 32 * c + w.lane < w.cols && row < rows;
            const uint32_t target = wanted[32 * c];
            float v[32];
            load(c, v);
            if (32 * c + 32 > w.cols) {  // (what lies beyond the tile)
#pragma unroll
                for (uint32_t i = 1; i < 32; ++i)
                    if (32 * c + i >= w.cols) v[i] = v[0];
            }
            if (id >= V) {
#pragma unroll
                for (uint32_t i = 0; i < 32; ++i) v[i] = -INFINITY;
            }
            // targets among this warp's 32 ids
            uint32_t hits = __ballot_sync(kFull, target < V && target - (id - w.lane) < 32u);
            while (hits) {
                const uint32_t i = __ffs(hits) - 1;
                hits &= hits - 1;
                const uint32_t its = __shfl_sync(kFull, target, i);
                if (its == id) {
#pragma unroll
                    for (uint32_t k = 0; k < 32; ++k) {
                        if (k == i) {
                            at[first + 32 * c + i] = v[k];
                            v[k] = -INFINITY;
                        }
                    }
                }
            }
            // One reference for all 32 rows, if no row's largest can lie far below it: the
            // smallest of a lane's logits bounds every row's largest from below, and the
            // largest such bound of all lanes is near where the rows are alike. Else a
            // reference a row (777 rows: 282 us, 265 with one for all).
            float m = v[0], least = v[0];
#pragma unroll
            for (uint32_t i = 1; i < 31; i += 2) {
                m = max3f(m, v[i], v[i + 1]);
                least = fminf(least, fminf(v[i], v[i + 1]));
            }
            m = ceilf(max_across(fmaxf(m, v[31])) * kLog2E);
            least = max_across(fminf(least, v[31])) * kLog2E;
            if (m - least < 60.0f) {
                const Weights e(m);
#pragma unroll
                for (uint32_t i = 0; i < 32; ++i) v[i] = e(v[i]);
            } else {
#pragma unroll
                for (uint32_t i = 0; i < 32; ++i) {
                    const float top = ceilf(max_across(v[i]) * kLog2E);
                    v[i] = Weights(top)(v[i]);
                    if (w.lane == i) m = top;
                }
            }
            Part p{m, sum_across(v)};
            if (w.j > 0) {
                const Part before = sums[32 * c];
                const float top = fmaxf(p.m, before.m), ref = top == -INFINITY ? 0.0f : top;
                p = {top, p.s * pow2(p.m - ref) + before.s * pow2(before.m - ref)};
            }
            sums[32 * c] = p;
            if (w.j == cursor.count - 1 && mine)
                parts[static_cast<uint64_t>(cursor.v * 8 + w.row / 32) * rows + row] = p;
        }
    }
};

struct Joined {
    float m;
    FF s;
};
__device__ __forceinline__ Joined join(const Joined& a, const Joined& b) {
    const float m = fmaxf(a.m, b.m), ref = m == -INFINITY ? 0.0f : m;
    const float fa = pow2(a.m - ref), fb = pow2(b.m - ref);
    return {m, ff_add(FF{a.s.hi * fa, a.s.lo * fa}, FF{b.s.hi * fb, b.s.lo * fb})};
}

struct LossFinishArgs {
    const Part* parts;
    const float* at;
    const uint32_t* targets;
    const uint32_t* error;
    float* loss;
    float* lse;
    uint32_t rows, V, slots;
};

// The loss and lse of a row from the joined weights of its other ids. The difference
// of ln sum others and the target's logit is a float pair, so that a loss near zero,
// its exponential, keeps its bits. (In 64 bits these few steps took 5 us more, of a
// row's 54.)
__device__ __forceinline__ void finish_row(const LossFinishArgs& a, uint32_t row, const Joined& j) {
    const uint32_t t = a.targets[row];
    // ln of the sum: its power of two over log2(e) as the weights have it, and the rest
    constexpr double kOver = 1.0 / static_cast<double>(kLog2E);
    constexpr float kHi = static_cast<float>(kOver), kLo = static_cast<float>(kOver - static_cast<double>(kHi));
    const float sum = j.s.hi + j.s.lo;
    const bool some = sum > 0.0f && sum < INFINITY;
    int e = 0;
    const float f = some ? frexpf(sum, &e) : sum;  // in [1/2, 1); the sum is at least 2^-61 or nothing
    const float n = j.m + static_cast<float>(e);
    const float p = __fmul_rn(n, kHi);
    FF others{p, __fmaf_rn(n, kLo, __fmaf_rn(n, kHi, -p))};
    others = ff_add(others, FF{logf(f), 0.0f});
    if (!some) others = FF{sum == 0.0f ? -INFINITY : NAN, 0.0f};
    float loss = 0.0f, lse = others.hi;
    if (t < a.V) {
        const float z = a.at[row];
        FF d = ff_add(others, FF{-z, 0.0f});
        if (!(fabsf(d.hi) < INFINITY)) d = FF{others.hi - z, 0.0f};
        loss = d.hi > 20.0f ? d.hi + (d.lo + expf(-d.hi)) : log1pf(expf(d.hi) * (1.0f + d.lo));
        lse = z == -INFINITY ? others.hi : z + loss;
        if (z == INFINITY) loss = lse = NAN;
    }
    if (*a.error) loss = lse = NAN;
    a.loss[row] = loss;
    if (a.lse) a.lse[row] = lse;
}

constexpr uint32_t kFinishThreads = 1024, kFinishWarps = kFinishThreads / 32;

// kWide: 32 rows a block, a lane each, the slots spread over the warps; else a
// row a block.
template <bool kWide>
__global__ void __launch_bounds__(kFinishThreads) loss_finish_kernel(LossFinishArgs a) {
    __shared__ Joined sh[kFinishWarps][32];
    pdl_wait();
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t row = kWide ? blockIdx.x * 32 + lane : blockIdx.x;
    Joined j{-INFINITY, FF{0.0f, 0.0f}};
    if (row < a.rows) {
        const uint32_t step = kWide ? kFinishWarps : kFinishThreads;
#pragma unroll 8
        for (uint32_t i = kWide ? warp : threadIdx.x; i < a.slots; i += step) {
            const Part p = a.parts[static_cast<uint64_t>(i) * a.rows + row];
            j = join(j, Joined{p.m, FF{p.s, 0.0f}});
        }
    }
    auto across = [](Joined v) {
#pragma unroll
        for (uint32_t m = 16; m > 0; m >>= 1) v = join(v, Joined{__shfl_xor_sync(kFull, v.m, m), ff_shfl_xor(v.s, m)});
        return v;
    };
    if (!kWide) j = across(j);
    sh[warp][lane] = j;
    __syncthreads();
    if (kWide) {
        // a warp takes a row, a lane another warp's share of it; the last steps by the
        // lanes of one warp
        j = across(sh[lane][warp]);
        __syncthreads();
        if (lane == 0) sh[0][warp] = j;
        __syncthreads();
        if (warp == 0 && row < a.rows) finish_row(a, row, sh[0][lane]);
    } else if (warp == 0) {
        j = across(sh[lane][0]);
        if (lane == 0) finish_row(a, row, j);
    }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------

// A row's gradient g = m 2^e, m in (1/2, 1): m goes into P before P is rounded, 2^e into
// the hidden rows for dW (unrounded within their type's exponents, see Prep) and into
// dX's sums. So P's rounding and the results' are all there is.
struct GradParts {
    float m;
    int e;
    __device__ __forceinline__ explicit GradParts(float g) {
        m = frexpf(g, &e);
        if (!(fabsf(g) < INFINITY)) {
            m = NAN;
            e = 0;
        }
    }
};

// The target's entry, e^(z - lse) - 1, carries most of a row's gradient, so that its
// rounding would show in all of it. What it lost is kept, one number a row, and added
// back in fp32: to dX by the last launch, to dW's rows in the epilogue, for the first
// few hidden rows with a target among a warp's ids (of many the roundings average).
constexpr uint32_t kKeptRows = 8;
constexpr uint32_t kHitWords = 1 + 2 * kKeptRows;  // of 32 ids: how many rows, the rows, their targets

// f16 holds P times 2^14: entries down to 2^-28 stay normal numbers, and the
// target's, no smaller than -1, does not overflow.
template <typename T>
constexpr float kProbShift = 0.0f;
template <>
constexpr float kProbShift<__half> = 14.0f;

// The row of the i-th vector of all rows.
__device__ __forceinline__ uint32_t row_of(uint64_t i, const Div& by) {
    return i < (1ull << 31) ? by(static_cast<uint32_t>(i)) : static_cast<uint32_t>(i / by.d);
}

template <typename T>
__device__ __forceinline__ void unpack2(uint32_t w, float& lo, float& hi) {
    lo = bits_f32<T>(static_cast<uint16_t>(w));
    hi = bits_f32<T>(static_cast<uint16_t>(w >> 16));
}

// Hidden rows enter dW times the power of two of their gradient, over one for all rows.
// bf16 has the exponents for that: over the largest gradient's. f16 has 30, of
// which the hidden rows take some: over that of the largest product of an entry and its
// row's gradient, which then lies at 2^14 or above, so that a row keeps its bits down to
// 2^-28 of it. (Over the largest gradient's, rows 2^14 below it were 2.6e-4 off, 2^20
// below 2 percent, 2^25 below nothing.) That largest product takes a launch of its own
// ahead of P's (777 rows of 2,880 x 93,001: 952 -> 957 us).
template <typename T>
constexpr int kTopExponent = 0;  // of the largest scaled entry
template <>
constexpr int kTopExponent<__half> = 15;
constexpr int kNoTop = -1000;
constexpr uint32_t kTopBlocks = 256, kTopThreads = 256;

struct TopArgs {
    const uint4* x;
    const uint32_t* targets;
    const float* grad;
    int* tops;  // [kTopBlocks]
    uint32_t rows, V;
    Div by_vecs;
};

// The exponent e, entries below 2^e, of f16 hidden rows times their gradients, of each
// block's share of them.
__global__ void __launch_bounds__(kTopThreads) row_tops_kernel(TopArgs a) {
    __shared__ int sh[kTopThreads / 32];
    pdl_wait();
    pdl_trigger();
    int top = kNoTop;
    const uint64_t n = static_cast<uint64_t>(a.rows) * a.by_vecs.d, step = static_cast<uint64_t>(gridDim.x) * kTopThreads;
#pragma unroll 4
    for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * kTopThreads + threadIdx.x; i < n; i += step) {
        const uint32_t r = row_of(i, a.by_vecs);
        const uint4 q = a.x[i];
        const float g = a.grad[r];
        if (!(a.targets[r] < a.V && g != 0.0f)) continue;
        uint32_t bits = 0;
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) bits = max(bits, max(w[k] & 0x7FFFu, w[k] >> 16 & 0x7FFFu));
        if (bits == 0) continue;
        int e;
        frexpf(bits_f32<__half>(static_cast<uint16_t>(min(bits, 0x7BFFu))), &e);  // (what is not finite fails its row anyway)
        top = max(top, e + GradParts(g).e);
    }
    top = __reduce_max_sync(kFull, top);
    if (threadIdx.x % 32 == 0) sh[threadIdx.x / 32] = top;
    __syncthreads();
    if (threadIdx.x < 32) {
        top = __reduce_max_sync(kFull, threadIdx.x < kTopThreads / 32 ? sh[threadIdx.x] : kNoTop);
        if (threadIdx.x == 0) a.tops[blockIdx.x] = top;
    }
}

// What dW needs beside P, done by warps that the launch of P has to spare: hidden rows
// times their powers of two (exact, but for entries that become subnormal; rows that
// do not count are zeros, whatever they hold), the exponent of its sums, and of each
// 32 ids the first rows that have one of them for a target. (As a launch of its own:
// 4 us for 64 rows, 36 for 4,096.)
template <typename T>
struct Prep {
    const uint4* x;  // NULL: nothing to do
    uint4* scaled;
    const uint32_t* targets;
    const float* grad;
    const int* tops;  // f16: from the launch before
    uint32_t top_blocks;
    int* exponent;
    uint32_t* hits;
    uint32_t rows, V;
    Div by_vecs;  // vectors of 8 entries a row
    int shift;    // P's

    __device__ __forceinline__ void run(uint32_t warp, uint32_t warps) const {
        const uint32_t lane = threadIdx.x & 31;
        int top = kNoTop;
        if constexpr (kTopExponent<T> != 0) {
            for (uint32_t i = lane; i < top_blocks; i += 32) top = max(top, tops[i]);
        } else {
#pragma unroll 4
            for (uint32_t r = lane; r < rows; r += 32)
                if (targets[r] < V && grad[r] != 0.0f) top = max(top, GradParts(grad[r]).e);
        }
        top = max(__reduce_max_sync(kFull, top), -200) - kTopExponent<T>;
        if (warp == 0 && lane == 0) *exponent = top - shift;
        const uint64_t n = static_cast<uint64_t>(rows) * by_vecs.d;
        for (uint64_t i = static_cast<uint64_t>(warp) * 32 + lane; i < n; i += static_cast<uint64_t>(warps) * 32) {
            const uint32_t r = row_of(i, by_vecs);
            const float g = grad[r];
            uint4 q = make_uint4(0, 0, 0, 0);
            if (targets[r] < V && g != 0.0f) {
                q = x[i];
                // (an f16 entry may be 2^-24, so 2^38 at most; more where no row has an entry but 0)
                const float f = pow2(static_cast<float>(min(GradParts(g).e - top, 38)));
                uint32_t* p = &q.x;
#pragma unroll
                for (uint32_t k = 0; k < 4; ++k) {
                    float lo, hi;
                    unpack2<T>(p[k], lo, hi);
                    p[k] = pack2<T>(lo * f, hi * f);
                }
            }
            scaled[i] = q;
        }
        // a run of groups of 32 ids a warp, one pass over the rows
        const uint32_t groups = (V + 31) / 32, per = (groups + warps - 1) / warps;
        const uint32_t v0 = min(groups, warp * per), v1 = min(groups, v0 + per);
        for (uint32_t v = v0 + lane; v < v1; v += 32) hits[static_cast<uint64_t>(v) * kHitWords] = 0;
        __syncwarp();
#pragma unroll 4
        for (uint32_t r0 = 0; r0 < rows && v0 < v1; r0 += 32) {
            const uint32_t r = r0 + lane, t = r < rows ? targets[r] : SEL_INVALID_ID;
            uint32_t mine = __ballot_sync(kFull, t < V && t / 32 >= v0 && t / 32 < v1 && grad[r] != 0.0f);
            for (; mine; mine &= mine - 1) {  // (few)
                const uint32_t i = __ffs(mine) - 1, its = __shfl_sync(kFull, t, i);
                if (lane == 0) {
                    uint32_t* to = hits + static_cast<uint64_t>(its / 32) * kHitWords;
                    const uint32_t at = to[0];
                    if (at < kKeptRows) {
                        to[0] = at + 1;
                        to[1 + at] = r0 + i;
                        to[1 + kKeptRows + at] = its;
                    }
                }
            }
        }
    }
};

// 16 entries, rounded to T, as one 32-byte store: a whole sector a lane.
template <typename T>
__device__ __forceinline__ void store16(T* to, const float (&v)[32], uint32_t i) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(pack2<T>(v[i], v[i + 1])),
                 "r"(pack2<T>(v[i + 2], v[i + 3])), "r"(pack2<T>(v[i + 4], v[i + 5])), "r"(pack2<T>(v[i + 6], v[i + 7])),
                 "r"(pack2<T>(v[i + 8], v[i + 9])), "r"(pack2<T>(v[i + 10], v[i + 11])),
                 "r"(pack2<T>(v[i + 12], v[i + 13])), "r"(pack2<T>(v[i + 14], v[i + 15]))
                 : "memory");
}

// P of a piece: [its ids][hidden rows]. Hidden rows lie on the product's columns, so
// that a tile has no more of them than it needs. (Stores of 16 bytes: 474 us instead of
// 430 for a piece of 4,096 rows.)
template <typename T>
struct ProbProblem {
    using Type = T;
    static constexpr uint32_t kPart = 0;
    CUtensorMap x, w;
    Prep<T> prep;
    T* p;
    float* lost;  // [rows]: of the targets' entries, by their rounding
    const uint32_t* targets;
    const float* lse;
    const float* grad;
    uint32_t* error;
    uint32_t rows, V, v0, width, steps, n, pitch;
    Raster raster;

    using Cursor = RasterCursor<ProbProblem>;
    __device__ __forceinline__ void aside(uint32_t warp, uint32_t warps) const {
        if (prep.x) prep.run(warp, warps);
    }
    __device__ __forceinline__ GemmTile tile(uint32_t r, uint32_t v) const {
        return {&w, &x, v0 + v * kTileM, r * n, 0, 0, steps, n, false, false};
    }
    template <typename Arrive, typename Load>
    __device__ __forceinline__ void epilogue(const Cursor& cursor, const GemmTile& t, EpiWarp& w, Arrive arrived, Load load) const {
        const uint32_t id = t.am + w.row, first = t.bn + w.col;
        // the warp's rows: lse less ln |m|, and of 32 a bit for those that do not count,
        // one for a negative m, one for a target among the warp's ids
        auto* refs = reinterpret_cast<float*>(w.smem);
        auto* bits = reinterpret_cast<uint4*>(w.smem + 512);
        auto* ids = reinterpret_cast<uint32_t*>(w.smem + 576);
        // (All loads at once. One after the other, a group of rows at a time, a narrow
        // hidden state's product waited for them: 250 x 512 x 100,000 122.8 us in all, now
        // 118.5; the same at 1,000 and above.)
        uint32_t wanted[4];
        float gs[4], ls[4];
#pragma unroll
        for (uint32_t c = 0; c < 4; ++c) {
            const uint32_t i = 32 * c + w.lane, row = first + i;
            const bool in = i < w.cols && row < rows;
            wanted[c] = in ? targets[row] : SEL_INVALID_ID;
            gs[c] = in ? grad[row] : 0.0f;
            ls[c] = in ? lse[row] : 0.0f;
        }
        __syncwarp();
#pragma unroll
        for (uint32_t c = 0; c < 4; ++c) {
            if (c >= w.chunks) break;
            const uint32_t i = 32 * c + w.lane, target = wanted[c];
            const float m = target < V ? GradParts(gs[c]).m : 0.0f;
            const bool live = m != 0.0f;
            // (an lse of +Inf would make every probability 0, and the row's gradient a finite one)
            refs[i] = !live ? 0.0f : fabsf(ls[c]) < INFINITY ? ls[c] - logf(fabsf(m)) : NAN;
            ids[i] = target;
            const uint32_t dead = __ballot_sync(kFull, !live), negative = __ballot_sync(kFull, m < 0.0f);
            const uint32_t hits = __ballot_sync(kFull, live && target - (id - w.lane) < 32u);
            if (w.lane == 0) bits[c] = make_uint4(dead, hits, negative, 0);
        }
        arrived();  // (and the warp's lanes are together again)
        const float up = kProbShift<T>;
        T* out = p + static_cast<uint64_t>(id - v0) * pitch + first;
        const uint32_t cols = min(w.cols, first < pitch ? pitch - first : 0);
#pragma unroll 1
        for (uint32_t c = 0; c < w.chunks; ++c) {
            float v[32];
            load(c, v);
            const uint4 of = bits[c];
            // targets' entries, rare, through shared memory: a lane may have several
            auto* kept = reinterpret_cast<float*>(w.smem + 1088);
            if (of.y) {
#pragma unroll
                for (uint32_t i = 0; i < 32; ++i) {
                    if ((of.y >> i & 1) && ids[32 * c + i] == id) {
                        const uint32_t row = first + 32 * c + i;
                        const float m = GradParts(grad[row]).m;
                        const float e = expm1f(v[i] - lse[row]) * fabsf(m) * static_cast<float>(1 << static_cast<int>(kProbShift<T>));
                        const float less = e - to_f32(from_f32<T>(e));
                        kept[i] = isnan(refs[32 * c + i]) ? NAN : e;
                        lost[row] = m < 0.0f ? -less : less;
                    }
                }
            }
#pragma unroll
            for (uint32_t i = 0; i < 32; i += 4) {
                const float4 r = *reinterpret_cast<const float4*>(refs + 32 * c + i);
                v[i] = ex2_approx(fmaf(v[i] - r.x, kLog2E, up));
                v[i + 1] = ex2_approx(fmaf(v[i + 1] - r.y, kLog2E, up));
                v[i + 2] = ex2_approx(fmaf(v[i + 2] - r.z, kLog2E, up));
                v[i + 3] = ex2_approx(fmaf(v[i + 3] - r.w, kLog2E, up));
            }
            if (of.y) {
#pragma unroll
                for (uint32_t i = 0; i < 32; ++i)
                    if ((of.y >> i & 1) && ids[32 * c + i] == id) v[i] = kept[i];
            }
            if (of.z) {
#pragma unroll
                for (uint32_t i = 0; i < 32; ++i)
                    if (of.z >> i & 1) v[i] = -v[i];
            }
            if (of.x) {
#pragma unroll
                for (uint32_t i = 0; i < 32; ++i)
                    if (of.x >> i & 1) v[i] = 0.0f;
            }
            if (id - v0 < width) {
#pragma unroll
                for (uint32_t i = 0; i < 32; i += 16)
                    if (32 * c + i < cols) store16<T>(out + 32 * c + i, v, i);
            }
        }
    }
};

// Items of a worker: its tiles of dX first, each a long sum, then its tiles of dW, one
// launch for both so that those even out what these leave.
template <typename T>
struct GradsProblem {
    using Type = T;
    static constexpr uint32_t kPart = 0;
    CUtensorMap p_k, x_mn, dw, p_mn, w_mn;
    const int* exponent;  // of dW's sums
    const T* scaled;      // [rows][H]: the hidden rows of dW
    const float* lost;
    const uint32_t* hits;  // [V / 32][kHitWords]
    float* acc;            // [slices][rows][H]
    uint32_t* error;
    uint32_t rows, V, H, v0, width;
    uint32_t n_rows;                            // dX: columns a tile
    Div by_row_tiles, by_dx_tiles, by_h_tiles;  // (dW's last column tile: 128 where that is enough)
    uint32_t dx_items, k_slice;                 // k_slice: ids of the piece a slice sums
    uint32_t dw_items, dw_steps, extra;         // extra: dW tiles ahead for workers with one dX tile less
    bool add;

    __device__ __forceinline__ void aside(uint32_t, uint32_t) const {}
    struct Cursor {
        const GradsProblem& p;
        uint32_t worker, workers, dx, more, light, ahead, count;
        __device__ __forceinline__ Cursor(const GradsProblem& of, uint32_t w, uint32_t n) : p(of), worker(w), workers(n) {
            dx = w < p.dx_items ? (p.dx_items - w - 1) / n + 1 : 0;
            more = p.dx_items % n;
            light = n - more;
            ahead = w >= more ? p.extra : 0;
            const uint32_t rest = p.dw_items - p.extra * light;
            count = dx + ahead + (w < rest ? (rest - w - 1) / n + 1 : 0);
        }
        __device__ __forceinline__ GemmTile tile(uint32_t j) const {
            if (j < dx) {
                const uint32_t i = worker + j * workers, slice = p.by_dx_tiles(i), at = i - slice * p.by_dx_tiles.d;
                const uint32_t h = p.by_row_tiles(at), r = at - h * p.by_row_tiles.d;
                const uint32_t k0 = slice * p.k_slice, k1 = min(p.width, k0 + p.k_slice);
                // (an empty slice sums one step of zeros past the piece's end)
                const uint32_t steps = k1 > k0 ? (k1 - k0 + kStepK - 1) / kStepK : 1;
                return {&p.w_mn, &p.p_mn, h * kTileM, r * p.n_rows, p.v0 + k0, k0, steps, p.n_rows, true, true};
            }
            j -= dx;
            const uint32_t i = j < ahead ? worker - more + j * light : p.extra * light + worker + (j - ahead) * workers;
            const uint32_t v = p.by_h_tiles(i), h = (i - v * p.by_h_tiles.d) * kTileN;
            return {&p.p_k, &p.x_mn, v * kTileM, h, 0, 0, p.dw_steps, p.H - h <= kTileN / 2 ? kTileN / 2 : kTileN, false, true};
        }
    };
    template <typename Arrive, typename Load>
    __device__ __forceinline__ void epilogue(const Cursor& cursor, const GemmTile& t, EpiWarp& w, Arrive arrived, Load load) const {
        if (!t.a_mn) {
            const Shift shift(*exponent);
            const uint32_t id = v0 + t.am + w.row - w.lane;
            // (lane k has word k of the ids' hits; the next tile's are asked for a tile ahead)
            auto entry = [&](uint32_t of) {
                return of < V && w.lane < kHitWords ? hits[static_cast<uint64_t>(of / 32) * kHitWords + w.lane] : 0u;
            };
            const uint32_t kept = w.j > cursor.dx ? w.kept : entry(id);
            if (w.j + 1 < cursor.count) w.kept = entry(id - t.am + cursor.tile(w.j + 1).am);
            const uint32_t n = __shfl_sync(kFull, kept, 0);
            // lane k: what the k-th row's entry lost; x0: the first row's columns of all
            // pieces, so that nothing is waited for below
            float less = 0.0f;
            T x0[4] = {};
            const uint32_t col = t.bn + w.col + w.lane;
            auto hidden = [&](uint32_t r, uint32_t x) { return x < H ? scaled[static_cast<uint64_t>(r) * H + x] : T{}; };
            if (n > 0) {
                const uint32_t r = __shfl_sync(kFull, kept, 1), mine = __shfl_sync(kFull, kept, 1 + w.lane);
                if (w.lane < n) less = lost[mine];
#pragma unroll
                for (uint32_t c = 0; c < 4; ++c) x0[c] = hidden(r, col + 32 * c);
            }
            arrived();
#pragma unroll 1
            for (uint32_t c = 0; c < w.chunks; ++c) {
                float v[32];
                load(c, v);
                for (uint32_t k = 0; k < n; ++k) {
                    const float f = __shfl_sync(kFull, less, k);
                    const bool mine = __shfl_sync(kFull, kept, 1 + kKeptRows + k) == id + w.lane;
                    const uint32_t r = __shfl_sync(kFull, kept, 1 + k);
                    const T x = k > 0 ? hidden(r, col + 32 * c) : c == 0 ? x0[0] : c == 1 ? x0[1] : c == 2 ? x0[2] : x0[3];
                    const float xf = to_f32(x);
#pragma unroll
                    for (uint32_t i = 0; i < 32; ++i) {
                        const float xi = __shfl_sync(kFull, xf, i);
                        if (mine) v[i] = fmaf(f, xi, v[i]);
                    }
                }
#pragma unroll
                for (uint32_t i = 0; i < 32; ++i) v[i] = shift(v[i]);
                const uint32_t x = t.bn + w.col + c / 2 * 64;
                store_chunk<T>(w, &dw, x, id, c, x < H && id < V, v);
            }
        } else {
            const uint32_t h = t.am + w.row, slice = by_dx_tiles(cursor.worker + w.j * cursor.workers), first = t.bn + w.col;
            float* o = acc + (static_cast<uint64_t>(slice) * rows + first) * H + h;
            arrived();
#pragma unroll 1
            for (uint32_t c = 0; c < w.chunks; ++c) {
                float v[32];
                load(c, v);
                const uint32_t n = min(w.cols, first < rows ? rows - first : 0);
                if (h < H) {
#pragma unroll
                    for (uint32_t i = 0; i < 32; ++i) {
                        if (32 * c + i < n) {
                            float* q = o + static_cast<uint64_t>(32 * c + i) * H;
                            *q = add ? *q + v[i] : v[i];
                        }
                    }
                }
            }
        }
    }
};

constexpr uint32_t kGradThreads = 128;

struct GradFinishArgs {
    const float* acc;
    const float* lost;
    const uint4* w;
    const uint32_t* targets;
    const float* grad;
    const uint32_t* error;
    uint4* dx;  // NULL: not wanted
    uint4* dw;
    uint32_t rows, V, slices;
    Div by_vecs;
    int shift;  // P's
};

// dX from its sums, rounded once. With the error word raised both gradients
// become NaN. kSplit: a block takes 32 vectors, each of its warps every fourth of their
// slices (one thread for all 19 slices of 64 rows took 9 us, of 206).
template <typename T, bool kSplit>
__global__ void __launch_bounds__(kGradThreads) grad_finish_kernel(GradFinishArgs a) {
    constexpr uint32_t kParts = kSplit ? kGradThreads / 32 : 1, kVecs = kGradThreads / kParts;
    __shared__ float4 sh[kSplit ? kGradThreads : 1][2];
    pdl_wait();
    pdl_trigger();
    const uint64_t n = static_cast<uint64_t>(a.rows) * a.by_vecs.d;
    const uint32_t part = threadIdx.x / kVecs, at = threadIdx.x % kVecs;
    const bool bad = *a.error != 0;
    const uint32_t nan2 = pack2<T>(NAN, NAN);
    for (uint64_t i0 = static_cast<uint64_t>(blockIdx.x) * kVecs; a.dx && i0 < n; i0 += static_cast<uint64_t>(gridDim.x) * kVecs) {
        const uint64_t i = i0 + at;
        const uint32_t r = i < n ? row_of(i, a.by_vecs) : 0;
        const float g = i < n ? a.grad[r] : 0.0f;
        const bool live = i < n && a.targets[r] < a.V && g != 0.0f;
        float s[8] = {};
        if (live) {
#pragma unroll 5
            for (uint32_t k = part; k < a.slices; k += kParts) {
                const float4* p = reinterpret_cast<const float4*>(a.acc) + 2 * (k * n + i);
                const float4 u = p[0], v = p[1];
                s[0] += u.x, s[1] += u.y, s[2] += u.z, s[3] += u.w;
                s[4] += v.x, s[5] += v.y, s[6] += v.z, s[7] += v.w;
            }
        }
        if constexpr (kSplit) {
            sh[threadIdx.x][0] = make_float4(s[0], s[1], s[2], s[3]);
            sh[threadIdx.x][1] = make_float4(s[4], s[5], s[6], s[7]);
            __syncthreads();
            if (part == 0) {
#pragma unroll
                for (uint32_t k = 1; k < kParts; ++k) {
                    const float4 u = sh[k * kVecs + at][0], v = sh[k * kVecs + at][1];
                    s[0] += u.x, s[1] += u.y, s[2] += u.z, s[3] += u.w;
                    s[4] += v.x, s[5] += v.y, s[6] += v.z, s[7] += v.w;
                }
            }
            __syncthreads();
        }
        if (part > 0 || i >= n) continue;
        uint4 q = make_uint4(0, 0, 0, 0);
        if (live) {
            const float f = a.lost[r];
            const uint4 of = a.w[static_cast<uint64_t>(a.targets[r]) * a.by_vecs.d + (i - static_cast<uint64_t>(r) * a.by_vecs.d)];
            const uint32_t u[4] = {of.x, of.y, of.z, of.w};
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k) {
                float lo, hi;
                unpack2<T>(u[k], lo, hi);
                s[2 * k] = fmaf(f, lo, s[2 * k]);
                s[2 * k + 1] = fmaf(f, hi, s[2 * k + 1]);
            }
            const Shift shift(GradParts(g).e - a.shift);
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) s[k] = shift(s[k]);
            q = make_uint4(pack2<T>(s[0], s[1]), pack2<T>(s[2], s[3]), pack2<T>(s[4], s[5]), pack2<T>(s[6], s[7]));
        }
        if (bad) q = make_uint4(nan2, nan2, nan2, nan2);
        a.dx[i] = q;
    }
    if (bad && a.dw) {
        for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * kGradThreads + threadIdx.x;
             i < static_cast<uint64_t>(a.V) * a.by_vecs.d; i += static_cast<uint64_t>(gridDim.x) * kGradThreads)
            a.dw[i] = make_uint4(nan2, nan2, nan2, nan2);
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// Hidden rows on a product's columns: tiles of up to 256, all alike, a multiple of 16.
struct Columns {
    uint32_t n, tiles;
    explicit Columns(uint32_t rows) {
        n = ceil_div(ceil_div(rows, ceil_div(rows, kTileN)), 16) * 16;
        tiles = ceil_div(rows, n);
    }
    uint32_t padded() const { return n * tiles; }
};

inline bool sizes_fit(uint32_t rows, uint32_t V, uint32_t H) {
    const uint64_t m = ceil_div(rows, 128), n = ceil_div(V, 128), h = ceil_div(H, 128);
    return rows <= 0x7fffffffu && m * n < (1ull << 31) && n * h < (1ull << 31) && m * h * 64 < (1ull << 31);
}

constexpr uint32_t kMaxWorkers = 96;  // (the workspace's size goes by no device)

struct LossPlan {
    bool columns;  // hidden rows on the products' columns
    uint32_t slots;
    size_t at, parts, bytes;
};
// Rows on the columns pad less, but their workers are a multiple of the row tiles
// (of some 76).
inline LossPlan loss_plan(uint32_t rows, uint32_t V) {
    LossPlan p;
    const Columns c(rows);
    p.columns = c.tiles <= 76 && static_cast<uint64_t>(ceil_div(rows, kTileM)) * kTileM * (76 / c.tiles * c.tiles) >
                                     static_cast<uint64_t>(c.padded()) * 76;
    p.slots = std::max(2 * ceil_div(V, kTileN), 8 * kMaxWorkers);  // (of either form, so that more rows take no less)
    p.at = kWsHeaderBytes;
    p.parts = p.at + align_up(static_cast<size_t>(rows) * sizeof(float), 256);
    p.bytes = p.parts + align_up(static_cast<size_t>(p.slots) * rows * sizeof(Part), 256);
    return p;
}

// The vocabulary in pieces: as few as keep P within 2^28 entries, but none below
// 16,384 ids, and all alike.
struct GradPlan {
    uint32_t piece, pieces, slices, pitch, dx_n;
    size_t lost, tops, hits, scaled, acc, p, bytes;
};
inline GradPlan grad_plan(uint32_t rows, uint32_t V, uint32_t H) {
    GradPlan g;
    g.pitch = ceil_div(rows, 16) * 16;
    const uint64_t cap = std::max<uint64_t>(16384, (1ull << 28) / g.pitch);
    g.piece = ceil_div(ceil_div(V, ceil_div(V, cap)), kTileM) * kTileM;
    g.pieces = ceil_div(V, g.piece);
    // dX's columns a tile: equal tiles pad less, but their halves begin anywhere in a
    // sector of P and are copied 64 rows at a time, so they have to pad a good deal less
    // (equal / whole tiles, 2,048 x 60,000, the whole call: 777 rows, 1.23 times as many
    // columns, 408-421 / 384-404 us; 400, 1.23 times, 247 / 245; 550, 1.33 times, 308 / 314;
    // 290, 1.6 times, 223 / 227)
    const Columns c(rows);
    g.dx_n = rows <= kTileN || c.padded() * 1.28 < static_cast<double>(ceil_div(rows, kTileN)) * kTileN ? c.n : kTileN;
    // few tiles of dX: the sum over the piece is split
    const uint64_t tiles = static_cast<uint64_t>(ceil_div(H, kTileM)) * ceil_div(rows, g.dx_n);
    g.slices = std::min(std::max(1u, g.piece / 1024), tiles >= 76 ? 1u : ceil_div(76, tiles));
    g.lost = kWsHeaderBytes;
    g.tops = g.lost + align_up(static_cast<size_t>(rows) * sizeof(float), 256);
    g.hits = g.tops + kTopBlocks * sizeof(int);
    g.scaled = g.hits + align_up(static_cast<size_t>(ceil_div(V, 32)) * kHitWords * sizeof(uint32_t), 256);
    g.acc = g.scaled + align_up(static_cast<size_t>(rows) * H * 2, 256);
    // What the sums and P take at most: slices * tiles < 76 + tiles, and P as above;
    // these bounds grow with each size, so that a workspace serves smaller calls too.
    const size_t sums = static_cast<size_t>(std::min(rows, kTileN)) * std::min(H, kTileM) * 76 + static_cast<size_t>(rows) * H;
    const size_t whole = static_cast<size_t>(g.pitch) * (ceil_div(V, kTileM) * static_cast<size_t>(kTileM));
    const size_t most = std::max<size_t>(g.pitch * 16384ull, 1ull << 28) + g.pitch * static_cast<size_t>(kTileM);
    g.p = g.acc + align_up(sums * sizeof(float), 256);
    g.bytes = g.p + std::min(whole, most) * 2;
    return g;
}

inline bool map16(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint32_t box_cols, uint32_t box_rows,
                  uint64_t pitch = 0) {
    return make_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, base, cols, rows, box_cols, box_rows, CU_TENSOR_MAP_SWIZZLE_128B,
                    pitch);
}

struct HeadLossCall {
    const void *x, *w;
    const uint32_t* targets;
    uint32_t rows, V, H;
    unsigned char* ws;
    cudaStream_t stream;
};

template <typename T>
sel_status run_loss(const HeadLossCall& c, float* loss, float* lse) {
    const int sms = device_sms();
    if (sms < 2) return SEL_ECUDA;
    const LossPlan plan = loss_plan(c.rows, c.V);
    auto* at = reinterpret_cast<float*>(c.ws + plan.at);
    auto* parts = reinterpret_cast<Part*>(c.ws + plan.parts);
    auto* error = reinterpret_cast<uint32_t*>(c.ws);
    const uint32_t v_tiles = ceil_div(c.V, kTileM);
    uint32_t workers = std::min<uint32_t>(sms / 2, kMaxWorkers), slots;
    auto launch = [&](auto& p, uint32_t x_box) {
        if (!map16(&p.x, c.x, c.H, c.rows, kStepK, x_box) || !map16(&p.w, c.w, c.H, c.V, kStepK, kCtaM)) return SEL_ECUDA;
        p.targets = c.targets;
        p.at = at;
        p.parts = parts;
        p.error = error;
        p.rows = c.rows;
        p.V = c.V;
        p.steps = ceil_div(c.H, kStepK);
        return launch_gemm(p, workers, c.stream);
    };
    sel_status st;
    const Columns cols(c.rows);
    if (plan.columns && cols.tiles <= workers) {
        const uint32_t each = std::min(workers / cols.tiles, v_tiles);  // workers of a row tile
        workers = each * cols.tiles;
        slots = 8 * each;
        LossColumnsProblem<T> p{};
        p.n = cols.n;
        p.row_tiles = cols.tiles;
        p.v_tiles = v_tiles;
        st = launch(p, cols.n / 2);
    } else {
        LossProblem<T> p{};
        p.raster = {ceil_div(c.rows, kTileM), v_tiles};
        slots = 2 * v_tiles;
        workers = std::min(workers, p.raster.mt * p.raster.nt);
        st = launch(p, kCtaM);
    }
    if (st != SEL_OK) return st;
    const LossFinishArgs f{parts, at, c.targets, error, loss, lse, c.rows, c.V, slots};
    // A block a row until those outnumber what runs at a time (the whole call, a row a
    // block / 32 rows a block, 1,024 x 151,936: 64 rows 54 / 62 us, 256 61 / 74, 512 102 /
    // 108, 777 180 / 177, 1,024 198 / 190, 4,096 733 / 682)
    const cudaError_t e = c.rows >= 640
                              ? launch_pdl(loss_finish_kernel<true>, dim3(ceil_div(c.rows, 32)), dim3(kFinishThreads), 0, c.stream, f)
                              : launch_pdl(loss_finish_kernel<false>, dim3(c.rows), dim3(kFinishThreads), 0, c.stream, f);
    return e == cudaSuccess ? SEL_OK : SEL_ECUDA;
}

template <typename T>
sel_status run_grad(const HeadLossCall& c, const float* lse, const float* grad, void* dx, void* dw) {
    const int sms = device_sms();
    if (sms < 2) return SEL_ECUDA;
    const GradPlan plan = grad_plan(c.rows, c.V, c.H);
    const Columns rows(c.rows);
    auto* error = reinterpret_cast<uint32_t*>(c.ws);
    auto* exponent = reinterpret_cast<int*>(c.ws + 16);
    auto* acc = reinterpret_cast<float*>(c.ws + plan.acc);
    void* prob = c.ws + plan.p;
    void* scaled = c.ws + plan.scaled;
    auto* lost = reinterpret_cast<float*>(c.ws + plan.lost);
    auto* hits = reinterpret_cast<uint32_t*>(c.ws + plan.hits);
    const int shift = static_cast<int>(kProbShift<T>);
    const uint32_t vecs = c.H / 8, all = sms / 2;
    const TopArgs tops{static_cast<const uint4*>(c.x), c.targets, grad, reinterpret_cast<int*>(c.ws + plan.tops), c.rows, c.V, Div(vecs)};
    const uint32_t top_blocks = std::min<uint64_t>(kTopBlocks, ceil_div(static_cast<uint64_t>(c.rows) * vecs, kTopThreads));
    if (dw && kTopExponent<T> != 0 &&
        launch_pdl(row_tops_kernel, dim3(top_blocks), dim3(kTopThreads), 0, c.stream, tops) != cudaSuccess)
        return SEL_ECUDA;
    for (uint32_t i = 0; i < plan.pieces; ++i) {
        const uint32_t v0 = i * plan.piece, width = std::min(plan.piece, c.V - v0);
        const uint64_t pitch = static_cast<uint64_t>(plan.pitch) * 2;
        ProbProblem<T> p{};
        if (!map16(&p.x, c.x, c.H, c.rows, kStepK, rows.n / 2) || !map16(&p.w, c.w, c.H, c.V, kStepK, kCtaM)) return SEL_ECUDA;
        if (dw && i == 0)
            p.prep = {static_cast<const uint4*>(c.x), static_cast<uint4*>(scaled), c.targets, grad, tops.tops, top_blocks,
                      exponent, hits, c.rows, c.V, Div(vecs), shift};
        p.p = static_cast<T*>(prob);
        p.lost = lost;
        p.targets = c.targets;
        p.lse = lse;
        p.grad = grad;
        p.error = error;
        p.rows = c.rows;
        p.V = c.V;
        p.v0 = v0;
        p.width = width;
        p.steps = ceil_div(c.H, kStepK);
        p.n = rows.n;
        p.pitch = plan.pitch;
        p.raster = {rows.tiles, ceil_div(width, kTileM)};
        if (const sel_status s = launch_gemm(p, std::min(all, p.raster.mt * p.raster.nt), c.stream); s != SEL_OK) return s;
        GradsProblem<T> g{};
        if (!map16(&g.p_k, prob, c.rows, width, kStepK, kCtaM, pitch) || !map16(&g.x_mn, scaled, c.H, c.rows, 64, kStepK) ||
            (dw && !map16(&g.dw, dw, c.H, c.V, 64, 32)) || !map16(&g.p_mn, prob, c.rows, width, 64, kStepK, pitch) ||
            !map16(&g.w_mn, c.w, c.H, c.V, 64, kStepK))
            return SEL_ECUDA;
        g.exponent = exponent;
        g.scaled = static_cast<const T*>(scaled);
        g.lost = lost;
        g.hits = hits;
        g.acc = acc;
        g.error = error;
        g.rows = c.rows;
        g.V = c.V;
        g.H = c.H;
        g.v0 = v0;
        g.width = width;
        g.n_rows = plan.dx_n;
        g.by_row_tiles = Div(ceil_div(c.rows, plan.dx_n));
        g.by_dx_tiles = Div(ceil_div(c.H, kTileM) * g.by_row_tiles.d);
        g.dx_items = dx ? g.by_dx_tiles.d * plan.slices : 0;
        g.k_slice = ceil_div(ceil_div(plan.piece, plan.slices), kStepK) * kStepK;
        g.by_h_tiles = Div(ceil_div(c.H, kTileN));
        g.dw_items = dw ? ceil_div(width, kTileM) * g.by_h_tiles.d : 0;
        g.dw_steps = ceil_div(c.rows, kStepK);
        g.add = i > 0;
        const uint32_t workers = std::min(all, g.dx_items + g.dw_items);
        const uint32_t light = workers - g.dx_items % workers;
        g.extra = light == workers ? 0 : std::min(g.dw_items / light, (g.k_slice / kStepK) / (g.dw_steps + 2));
        if (const sel_status s = launch_gemm(g, workers, c.stream); s != SEL_OK) return s;
    }
    const GradFinishArgs f{acc, lost, static_cast<const uint4*>(c.w), c.targets, grad, error, static_cast<uint4*>(dx), static_cast<uint4*>(dw), c.rows, c.V, plan.slices, Div(vecs), shift};
    // (one thread for all slices / a warp for every fourth, the whole call: 1,024 rows of
    // 2,560 x 30,000, 2 slices, 282 / 290 us; of 1,280, 4 slices, 171 / 175; of 768, 7
    // slices, 125 / 124; 64 rows of 1,024 x 151,936, 19 slices, 207 / 205)
    const bool split = plan.slices >= 6;
    const uint64_t vectors = static_cast<uint64_t>(c.rows) * vecs;
    const dim3 blocks(static_cast<uint32_t>(std::min<uint64_t>(8 * sms, ceil_div(vectors, split ? 32 : kGradThreads))));
    const cudaError_t e = split ? launch_pdl(grad_finish_kernel<T, true>, blocks, dim3(kGradThreads), 0, c.stream, f)
                                : launch_pdl(grad_finish_kernel<T, false>, blocks, dim3(kGradThreads), 0, c.stream, f);
    return e == cudaSuccess ? SEL_OK : SEL_ECUDA;
}

sel_status check_head(const void* x, const void* w, const uint32_t* targets, int dtype, uint32_t rows, uint32_t V, uint32_t H) {
    if (dtype != SEL_F16 && dtype != SEL_BF16) return SEL_EINVAL;
    if (V == 0 || V > SEL_MAX_V || H == 0 || H > SEL_MAX_H) return SEL_EINVAL;
    if (H % 8 != 0) return SEL_EUNSUPPORTED;
    if (rows == 0) return SEL_OK;
    if (!x || !w || !targets) return SEL_EINVAL;
    if (misaligned(x, 16) || misaligned(w, 16) || misaligned(targets, 4)) return SEL_EINVAL;
    return sizes_fit(rows, V, H) ? SEL_OK : SEL_EUNSUPPORTED;
}

}  // namespace

size_t head_loss_ws_bytes(uint32_t rows, uint32_t V, uint32_t H) {
    if (rows == 0 || H == 0 || H > SEL_MAX_H || H % 8 != 0 || !sizes_fit(rows, V, H)) return 0;
    return loss_plan(rows, V).bytes;
}
size_t head_loss_grad_ws_bytes(uint32_t rows, uint32_t V, uint32_t H) {
    if (rows == 0 || H == 0 || H > SEL_MAX_H || H % 8 != 0 || !sizes_fit(rows, V, H)) return 0;
    return grad_plan(rows, V, H).bytes;
}

}  // namespace sel

extern "C" sel_status sel_head_loss(const void* d_hidden, uint32_t rows, const void* d_weight, int dtype, uint32_t V,
                                    uint32_t H, const uint32_t* d_targets, float* d_loss, float* d_lse, void* d_ws,
                                    size_t ws_bytes, cudaStream_t stream) {
    if (const sel_status s = check_head(d_hidden, d_weight, d_targets, dtype, rows, V, H); s != SEL_OK) return s;
    if (rows == 0) return SEL_OK;
    if (!d_loss || misaligned(d_loss, 4) || misaligned(d_lse, 4)) return SEL_EINVAL;
    if (!d_ws || misaligned(d_ws, SEL_WS_ALIGN)) return SEL_EINVAL;
    if (ws_bytes < head_loss_ws_bytes(rows, V, H)) return SEL_EWORKSPACE;
    const HeadLossCall c{d_hidden, d_weight, d_targets, rows, V, H, static_cast<unsigned char*>(d_ws), stream};
    return dtype == SEL_F16 ? run_loss<__half>(c, d_loss, d_lse) : run_loss<__nv_bfloat16>(c, d_loss, d_lse);
}

extern "C" sel_status sel_head_loss_grad(const void* d_hidden, uint32_t rows, const void* d_weight, int dtype, uint32_t V,
                                         uint32_t H, const uint32_t* d_targets, const float* d_lse, const float* d_grad,
                                         void* d_hidden_grad, void* d_weight_grad, void* d_ws, size_t ws_bytes,
                                         cudaStream_t stream) {
    if (const sel_status s = check_head(d_hidden, d_weight, d_targets, dtype, rows, V, H); s != SEL_OK) return s;
    if (misaligned(d_hidden_grad, 16) || misaligned(d_weight_grad, 16)) return SEL_EINVAL;
    if (rows > 0 && !d_hidden_grad && !d_weight_grad) return SEL_EINVAL;
    if (rows == 0) {  // (an empty hidden_grad may have no address)
        if (!d_weight_grad) return SEL_OK;
        return cudaMemsetAsync(d_weight_grad, 0, static_cast<size_t>(V) * H * 2, stream) == cudaSuccess ? SEL_OK : SEL_ECUDA;
    }
    if (!d_lse || !d_grad || misaligned(d_lse, 4) || misaligned(d_grad, 4)) return SEL_EINVAL;
    if (!d_ws || misaligned(d_ws, SEL_WS_ALIGN)) return SEL_EINVAL;
    if (ws_bytes < head_loss_grad_ws_bytes(rows, V, H)) return SEL_EWORKSPACE;
    const HeadLossCall c{d_hidden, d_weight, d_targets, rows, V, H, static_cast<unsigned char*>(d_ws), stream};
    return dtype == SEL_F16 ? run_grad<__half>(c, d_lse, d_grad, d_hidden_grad, d_weight_grad)
                            : run_grad<__nv_bfloat16>(c, d_lse, d_grad, d_hidden_grad, d_weight_grad);
}
