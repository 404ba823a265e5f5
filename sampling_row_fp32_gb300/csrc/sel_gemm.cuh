// sel_gemm.cuh -- matrix products of 16-bit operands on the tensor cores, their
// results handed to an epilogue in fp32 while the next tile is computed.
//
//   D[m][n] = sum_k A[m][k] * B[n][k]
//
// Each operand may lie with k or with its own index (m or n) in the rows of its
// matrix: the tensor cores take both, so nothing is transposed. A worker, a
// pair of CTAs whose products run as one, walks a list of tiles that the problem P
// gives it: 256 rows (128 a CTA) and up to 256 columns. Warp roles:
//   warp 0      copies both operands, 64 k a stage, into a ring (TMA, swizzled)
//   warp 1      issues the products (the pair's first CTA for both)
//   warps 2, 3  what else P has to do
//   warps 4-11  read a tile's D from tensor memory, 32 rows and about half of the
//               columns a warp, and run P's epilogue; D is double-buffered, so that the
//               products of the next tile run meanwhile
// Each CTA of a pair holds half of the tile's columns of B and both halves feed
// both, which halves what a product reads through L2 and shared memory: 32 KB a CTA
// and stage for 256 x 256, where a CTA on its own takes 48 for its 128 x 256.
// Every wait is bounded; one that runs out raises the workspace's error word.
//
// Products of 4,096 x 4,096 x 151,936 and the like keep the tensor pipe 96 to 99 percent
// active; few columns are bound by A's bytes (6.7 TB/s at n = 64). Six stages: five
// took 4 percent longer there; more and smaller ones where n is small gained nothing.
#pragma once

#include <cstdint>
#include <type_traits>

#include "sel_dtype.cuh"
#include "sel_plan.h"
#include "sel_tc.cuh"
#include "sel_tma.cuh"
#include "sel_units.cuh"

namespace sel {

constexpr uint32_t kTileM = 256, kTileN = 256, kCtaM = 128, kStepK = 64;
constexpr int kGemmThreads = 384;
constexpr uint32_t kEpiWarps = 8, kGemmStages = 6;
constexpr uint32_t kStageABytes = kCtaM * kStepK * 2, kStageBytes = kStageABytes + kTileN / 2 * kStepK * 2;
constexpr uint32_t kWarpBytes = 32 * 128;  // shared memory of an epilogue warp: 32 rows x 64 columns on their way out
constexpr uint32_t kGemmSmem = 1024 + kGemmStages * kStageBytes + kEpiWarps * kWarpBytes;
static_assert(kGemmSmem + 1024 <= 227 * 1024);

// A tile of a product: its columns n (a multiple of 16, at most 256), its steps of
// 64 k, and the operands' maps; *_mn: the operand's own index lies in the rows of its
// matrix. Maps of operands with k in the rows have boxes of 64 k x the rows a CTA
// holds (128 of A, n / 2 of B), the others boxes of 64 x 64 k.
struct GemmTile {
    const CUtensorMap *a, *b;
    uint32_t am, bn;  // where the operands' own indices begin
    uint32_t ak, bk;  // where their k begin
    uint32_t steps, n;
    bool a_mn, b_mn;
};

struct GemmShared {
    uint64_t full[kGemmStages], empty[kGemmStages], d_full[2], d_empty[2], drain;
    uint32_t tmem, err;
};

// Division by a number that the host knows, of numbers below 2^31.
struct Div {
    uint32_t d, mul, shift;
    Div() = default;
    explicit Div(uint32_t by) : d(by), shift(0) {
        while ((1ull << shift) < by) ++shift;
        mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << shift) - by)) / by + 1);
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
};

// A warp's place in a tile: this lane's row, the warp's first column and how many it
// has, in pieces of 32 (the last may be short: what it reads beyond is meaningless).
struct EpiWarp {
    uint32_t row, col, cols, chunks, lane;
    uint32_t j;           // the tile's number among the worker's
    uint32_t kept;        // P's, from a tile to the next
    unsigned char* smem;  // kWarpBytes of its own
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of a barrier of the pair's first CTA.
__device__ __forceinline__ uint32_t first_cta(uint64_t* bar) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(bar)));
    return r;
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A copy into this CTA's memory, counted on a barrier of the pair's first CTA.
__device__ __forceinline__ void tma_2d_pair(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int x, int y, const void* src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x), "r"(y),
                 "r"(smem_u32(src))
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void store_read_wait() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void gemm_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
        : "memory");
}
// The barrier, of both CTAs, completes once every product issued before by this
// thread has.
__device__ __forceinline__ void gemm_commit(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}
// The same for a barrier of this CTA alone.
__device__ __forceinline__ void gemm_commit_here(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

// Descriptor of an operand tile whose own index lies in its 128-byte rows (64
// entries of one k): 8 k are 1,024 bytes, 64 entries 8,192 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t addr) {
    return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(8192 >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Columns 32 c .. of a warp's rows, rounded to T, on their way to a matrix: 64 at
// a time leave as one box of 32 rows, whose first column and row are x and y,
// unless they lie outside.
// (Swizzled like the map's box: 16-byte piece ch of row r at ch ^ (r & 7).)
template <typename T>
__device__ __forceinline__ void store_chunk(const EpiWarp& w, const CUtensorMap* map, uint32_t x, uint32_t y, uint32_t c,
                                            bool inside, const float (&v)[32]) {
    if (c % 2 == 0) {
        if (w.lane == 0) store_read_wait();
        __syncwarp();
    }
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) {
        uint4 q;
        q.x = pack2<T>(v[8 * j], v[8 * j + 1]);
        q.y = pack2<T>(v[8 * j + 2], v[8 * j + 3]);
        q.z = pack2<T>(v[8 * j + 4], v[8 * j + 5]);
        q.w = pack2<T>(v[8 * j + 6], v[8 * j + 7]);
        const uint32_t ch = (c % 2) * 4 + j;
        *reinterpret_cast<uint4*>(w.smem + w.lane * 128 + ((ch ^ (w.lane & 7)) << 4)) = q;
    }
    if (c % 2 == 1) {
        proxy_fence();
        __syncwarp();
        if (w.lane == 0 && inside) tma_store_2d(map, x, y, w.smem);
    }
}

// P: a trivially copyable problem with its maps, and
//   using Type                         the operands' type
//   kPart                              steps that are summed in tensor memory: the sums
//                                      of a tile's parts meet in the epilogue's
//                                      registers (0: all of them in tensor memory)
//   uint32_t* error                    the workspace's error word
//   Cursor(p, worker, workers)         a worker's tiles: `count` of them, tile(j)
//   aside(warp, warps)                 what two warps a CTA do meanwhile
//   epilogue(cursor, tile, w, arrive, load)  arrive(): waits for the sums; then load(c, v): the
//                                      warp's columns 32 c .., for c = 0 .. chunks - 1 in
//                                      order, each once
template <typename P>
__global__ void __launch_bounds__(kGemmThreads, 1) gemm_kernel(const __grid_constant__ P p) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ GemmShared c;
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(kFull, tid >> 5, 0);
    const uint32_t rank = cluster_rank(), worker = blockIdx.x / 2, workers = gridDim.x / 2;

    if (tid == 0) {
        for (uint32_t i = 0; i < kGemmStages; ++i) {
            mbar_init(&c.full[i], 1);
            mbar_init(&c.empty[i], 1);
        }
        for (uint32_t i = 0; i < 2; ++i) {
            mbar_init(&c.d_full[i], 1);
            mbar_init(&c.d_empty[i], 2 * kEpiWarps);
        }
        mbar_init(&c.drain, 1);
        c.err = 0;
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&c.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(kFull, c.tmem, 0);
    pdl_wait();
    pdl_trigger();
    const typename P::Cursor cursor(p, worker, workers);
    const uint32_t count = cursor.count;

    if (warp == 0) {
        // what launches before wrote with ordinary stores, the copies read
        asm volatile("fence.proxy.async.global;" ::: "memory");
        const bool leader = elect_one();
        Ring<kGemmStages> st;
        uint32_t issued = 0;
        bool ok = true;
        for (uint32_t j = 0; j < count && ok; ++j) {
            const GemmTile t = cursor.tile(j);
            const uint32_t am = t.am + rank * kCtaM, bn = t.bn + rank * (t.n / 2);
            const uint32_t b_boxes = (t.n + 127) / 128;  // of 64
            const uint32_t bytes = 2 * (kStageABytes + (t.b_mn ? b_boxes * 8192 : t.n * 64));
            for (uint32_t s = 0; s < t.steps; ++s) {
                ok = __all_sync(kFull, mbar_wait(&c.empty[st.i], st.phase ^ 1));
                if (!ok) break;
                if (leader) {
                    unsigned char* da = ring + st.i * kStageBytes;
                    unsigned char* db = da + kStageABytes;
                    const uint32_t ak = t.ak + s * kStepK, bk = t.bk + s * kStepK;
                    if (rank == 0) expect_tx(&c.full[st.i], bytes);
                    const uint32_t bar = first_cta(&c.full[st.i]);
                    if (t.a_mn) {
                        for (uint32_t i = 0; i < kCtaM / 64; ++i) tma_2d_pair(da + i * 8192, t.a, am + i * 64, ak, bar);
                    } else {
                        tma_2d_pair(da, t.a, ak, am, bar);
                    }
                    if (t.b_mn) {
                        for (uint32_t i = 0; i < b_boxes; ++i) tma_2d_pair(db + i * 8192, t.b, bn + i * 64, bk, bar);
                    } else {
                        tma_2d_pair(db, t.b, bk, bn, bar);
                    }
                }
                ++issued;
                st.next();
            }
        }
        // every copy has landed before the CTAs may end
        if (leader && rank == 0) {
            for (uint32_t i = issued > kGemmStages ? issued - kGemmStages : 0; i < issued; ++i)
                if (!mbar_wait(&c.full[i % kGemmStages], (i / kGemmStages) & 1)) ok = false;
        }
        if (!ok) c.err = 1;
        __syncwarp();
    } else if (warp == 1 && rank == 0) {
        const bool leader = elect_one();
        constexpr uint32_t kType = std::is_same_v<typename P::Type, __nv_bfloat16> ? 1 : 0;
        constexpr uint32_t kIdesc = (1u << 4) | (kType << 7) | (kType << 10) | ((kTileM >> 4) << 24);
        Ring<kGemmStages> st;
        Ring<2> dr;
        for (uint32_t j = 0; j < count; ++j) {
            const GemmTile t = cursor.tile(j);
            const uint32_t idesc = kIdesc | (t.a_mn ? 1u << 15 : 0) | (t.b_mn ? 1u << 16 : 0) | ((t.n >> 3) << 17);
            const uint32_t step_a = t.a_mn ? 2048 >> 4 : 32 >> 4, step_b = t.b_mn ? 2048 >> 4 : 32 >> 4;
            wait(&c.d_empty[dr.i], dr.phase ^ 1, &c.err);
            tc_fence_after();
            uint32_t d = tmem + dr.i * kTileN;
            uint32_t left = P::kPart;  // of a part
            for (uint32_t s = 0; s < t.steps; ++s) {
                if (P::kPart != 0 && left == 0) {
                    if (leader) gemm_commit(&c.d_full[dr.i]);
                    __syncwarp();
                    dr.next();
                    wait(&c.d_empty[dr.i], dr.phase ^ 1, &c.err);
                    tc_fence_after();
                    d = tmem + dr.i * kTileN;
                    left = P::kPart;
                }
                const bool fresh = P::kPart != 0 ? left == P::kPart : s == 0;
                --left;
                wait(&c.full[st.i], st.phase, &c.err);
                tc_fence_after();
                if (leader) {
                    const uint32_t sa = smem_u32(ring + st.i * kStageBytes), sb = sa + kStageABytes;
                    const uint64_t a = t.a_mn ? smem_desc_mn(sa) : smem_desc(sa);
                    const uint64_t b = t.b_mn ? smem_desc_mn(sb) : smem_desc(sb);
#pragma unroll
                    for (uint32_t k = 0; k < kStepK / 16; ++k)
                        gemm_mma(d, a + k * step_a, b + k * step_b, idesc, !fresh || k > 0);
                    gemm_commit(&c.empty[st.i]);
                }
                __syncwarp();
                st.next();
            }
            if (leader) gemm_commit(&c.d_full[dr.i]);
            __syncwarp();
            dr.next();
        }
        // no product is in flight when the tensor memory is given back
        if (leader) gemm_commit_here(&c.drain);
        if (!mbar_wait(&c.drain, 0)) c.err = 1;
        __syncwarp();
    } else if (warp == 2 || warp == 3) {
        p.aside(2 * blockIdx.x + warp - 2, 2 * gridDim.x);
        __syncwarp();
    } else if (warp >= 4) {
        const uint32_t quarter = warp & 3, half = (warp - 4) >> 2;
        EpiWarp w;
        w.row = rank * kCtaM + quarter * 32 + lane;
        w.lane = lane;
        w.kept = 0;
        w.smem = ring + kGemmStages * kStageBytes + (warp - 4) * kWarpBytes;
        Ring<2> dr;
        for (uint32_t j = 0; j < count; ++j) {
            const GemmTile t = cursor.tile(j);
            const uint32_t low = (t.n / 2 + 15) / 16 * 16;  // (whole 32 bytes of 16-bit results)
            w.cols = half ? t.n - low : low;
            w.col = half * low;
            w.chunks = (w.cols + 31) / 32;
            w.j = j;
            // (a short last piece reads on, at most to the end of the tensor memory)
            const uint32_t d = tmem + (quarter << 21) + w.col;
            auto piece = [&](uint32_t i, uint32_t (&r)[32]) {
                __syncwarp();
                tmem_ld(d + dr.i * kTileN + i * 32, r);
            };
            auto release = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_cluster(first_cta(&c.d_empty[dr.i]));
            };
            float sums[P::kPart != 0 ? 128 : 1];  // of the parts before the last
            if constexpr (P::kPart != 0) {
#pragma unroll
                for (uint32_t i = 0; i < 128; ++i) sums[i] = 0.0f;
                for (uint32_t s = P::kPart; s < t.steps; s += P::kPart) {
                    wait(&c.d_full[dr.i], dr.phase, &c.err);
                    tc_fence_after();
#pragma unroll
                    for (uint32_t i = 0; i < 4; ++i) {
                        if (i >= w.chunks) break;
                        uint32_t r[32];
                        piece(i, r);
#pragma unroll
                        for (uint32_t k = 0; k < 32; ++k) sums[32 * i + k] += __uint_as_float(r[k]);
                    }
                    release();
                    dr.next();
                }
            }
            auto arrived = [&] {
                wait(&c.d_full[dr.i], dr.phase, &c.err);
                tc_fence_after();
                if (w.chunks == 0) release();  // (16 columns: all of them the other half's)
            };
            p.epilogue(cursor, t, w, arrived, [&](uint32_t i, float(&v)[32]) {
                uint32_t r[32];
                piece(i, r);
                if (i == w.chunks - 1) release();  // the buffer is read
#pragma unroll
                for (uint32_t k = 0; k < 32; ++k) {
                    v[k] = __uint_as_float(r[k]);
                    if constexpr (P::kPart != 0) v[k] += sums[32 * i + k];
                }
            });
            dr.next();
        }
        if (lane == 0) store_wait();
        __syncwarp();
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    if (tid == 0 && c.err) atomicOr(p.error, kErrTimeout);
}

template <typename P>
inline sel_status launch_gemm(const P& p, uint32_t workers, cudaStream_t stream) {
    if (!dynamic_smem_once<gemm_kernel<P>>(kGemmSmem)) return SEL_ECUDA;
    const cudaError_t e =
        launch_pdl_cluster(gemm_kernel<P>, dim3(2 * workers), dim3(kGemmThreads), 2, kGemmSmem, stream, p);
    return e == cudaSuccess ? SEL_OK : SEL_ECUDA;
}

}  // namespace sel
