// sel_gemm.cuh -- matrix products of 16-bit operands on the tensor cores, their
// results handed to an epilogue in fp32 while the next tile is computed.
//
//   D[m][n] = sum_k A[m][k] * B[n][k]
//
// Each operand may lie with k or with its own index (m or n) in the rows of its
// matrix: tensor memory's products take both, so nothing is transposed. A
// worker (a CTA, or a pair of CTAs whose products run as one) walks a list of
// tiles that the problem P gives it: 256 columns, 128 rows a CTA. Warp roles:
//   warp 0      copies both operands, 64 k a stage, into a ring (TMA, swizzled)
//   warp 1      issues the products (the pair's first CTA for both)
//   warps 4-11  read a tile's D from tensor memory, 32 rows x 128 columns a
//               warp, and run P's epilogue; D is double-buffered, so that
//               the products of the next tile run meanwhile
// A pair shares the tile's 256 columns of B: each CTA holds half of them and both
// halves feed both, which halves what a product reads through L2 and shared
// memory: 32 KB a CTA and stage instead of 48.
// Every wait is bounded; one that runs out raises the workspace's error word.
#pragma once

#include <cstdint>
#include <type_traits>

#include "sel_dtype.cuh"
#include "sel_plan.h"
#include "sel_tc.cuh"
#include "sel_tma.cuh"
#include "sel_units.cuh"

namespace sel {

constexpr uint32_t kTileN = 256, kCtaM = 128, kStepK = 64;
constexpr int kGemmThreads = 384;
constexpr uint32_t kEpiWarps = 8;
constexpr uint32_t kStageABytes = kCtaM * kStepK * 2;
constexpr uint32_t kStoreBytes = 32 * 128;  // a warp's 32 rows x 64 columns on their way out

template <bool kPair>
struct GemmConfig {
    static constexpr uint32_t kTileM = kPair ? 2 * kCtaM : kCtaM;
    static constexpr uint32_t kCtaN = kPair ? kTileN / 2 : kTileN;  // rows of B a CTA holds
    static constexpr uint32_t kStageBytes = kStageABytes + kCtaN * kStepK * 2;
    static constexpr uint32_t kStages = kPair ? 6 : 4;
    static constexpr uint32_t kSmem = 1024 + kStages * kStageBytes + kEpiWarps * kStoreBytes;
    static_assert(kSmem + 1024 <= 227 * 1024);
};

// A tile of a product: its first row, column and k, its steps of 64 k, and the
// operands' maps; *_mn: the operand's own index lies in the rows of its matrix.
// Maps of operands with k in the rows have boxes of 64 k x the rows a CTA holds,
// the others boxes of 64 x 64 k.
struct GemmTile {
    const CUtensorMap *a, *b;
    uint32_t am, bn;  // where the operands' own indices begin
    uint32_t ak, bk;  // where their k begin
    uint32_t steps;
    bool a_mn, b_mn;
};

struct GemmShared {
    uint64_t full[6], empty[6], d_full[2], d_empty[2], drain;
    uint32_t tmem, err;
};

// A warp's place in a tile, and what it writes through.
struct EpiWarp {
    uint32_t row, col;  // of the tile's first row and column: this lane's row, the warp's first of 128 columns
    uint32_t lane;
    unsigned char* store;  // kStoreBytes of shared memory
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

template <bool kPair>
__device__ __forceinline__ void gemm_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    if constexpr (kPair)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
            : "memory");
}
// The barrier, of both CTAs of a pair, completes once every product issued before
// by this thread has.
template <bool kPair>
__device__ __forceinline__ void gemm_commit(uint64_t* bar) {
    if constexpr (kPair)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_u32(bar)),
            "h"(static_cast<uint16_t>(3))
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                     : "memory");
}

// The same for a barrier of this CTA alone.
template <bool kPair>
__device__ __forceinline__ void gemm_commit_here(uint64_t* bar) {
    if constexpr (kPair)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                     : "memory");
    else gemm_commit<false>(bar);
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
        *reinterpret_cast<uint4*>(w.store + w.lane * 128 + ((ch ^ (w.lane & 7)) << 4)) = q;
    }
    if (c % 2 == 1) {
        proxy_fence();
        __syncwarp();
        if (w.lane == 0 && inside) tma_store_2d(map, x, y, w.store);
    }
}

// P: a trivially copyable problem with its maps, and
//   using Type                         the operands' type
//   uint32_t* error                    the workspace's error word
//   count(worker, workers)             how many tiles a worker has
//   tile(worker, workers, j)           the j-th of them
//   epilogue(tile, w, load)            load(c, v): columns 32 c .. of the warp's rows,
//                                      c = 0, 1, 2, 3 in order, each once
template <typename P, bool kPair>
__global__ void __launch_bounds__(kGemmThreads, 1) gemm_kernel(const __grid_constant__ P p) {
    using C = GemmConfig<kPair>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char* store = ring + C::kStages * C::kStageBytes;
    __shared__ GemmShared c;
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(kFull, tid >> 5, 0);
    const uint32_t rank = kPair ? cluster_rank() : 0;
    const uint32_t worker = kPair ? blockIdx.x / 2 : blockIdx.x, workers = kPair ? gridDim.x / 2 : gridDim.x;

    if (tid == 0) {
        for (uint32_t i = 0; i < C::kStages; ++i) {
            mbar_init(&c.full[i], 1);
            mbar_init(&c.empty[i], 1);
        }
        for (uint32_t i = 0; i < 2; ++i) {
            mbar_init(&c.d_full[i], 1);
            mbar_init(&c.d_empty[i], kPair ? 2 * kEpiWarps : kEpiWarps);
        }
        mbar_init(&c.drain, 1);
        c.err = 0;
    }
    if (warp == 2) {
        if constexpr (kPair) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&c.tmem))
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&c.tmem))
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        }
    }
    tc_fence_before();
    if constexpr (kPair) cluster_sync_all();
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(kFull, c.tmem, 0);
    pdl_wait();
    pdl_trigger();
    const uint32_t count = p.count(worker, workers);

    if (warp == 0) {
        const bool leader = elect_one();
        Ring<C::kStages> st;
        uint32_t issued = 0;
        bool ok = true;
        for (uint32_t j = 0; j < count && ok; ++j) {
            const GemmTile t = p.tile(worker, workers, j);
            const uint32_t am = t.am + rank * kCtaM, bn = t.bn + rank * C::kCtaN;
            for (uint32_t s = 0; s < t.steps; ++s) {
                ok = __all_sync(kFull, mbar_wait(&c.empty[st.i], st.phase ^ 1));
                if (!ok) break;
                if (leader) {
                    unsigned char* da = ring + st.i * C::kStageBytes;
                    unsigned char* db = da + kStageABytes;
                    const uint32_t ak = t.ak + s * kStepK, bk = t.bk + s * kStepK;
                    if (rank == 0) expect_tx(&c.full[st.i], (kPair ? 2 : 1) * C::kStageBytes);
                    const uint32_t bar = kPair ? first_cta(&c.full[st.i]) : 0;
                    auto copy = [&](unsigned char* dst, const CUtensorMap* map, uint32_t x, uint32_t y) {
                        if constexpr (kPair) tma_2d_pair(dst, map, x, y, bar);
                        else tma_2d(dst, map, x, y, &c.full[st.i]);
                    };
                    if (t.a_mn) {
                        for (uint32_t i = 0; i < kCtaM / 64; ++i) copy(da + i * 8192, t.a, am + i * 64, ak);
                    } else {
                        copy(da, t.a, ak, am);
                    }
                    if (t.b_mn) {
                        for (uint32_t i = 0; i < C::kCtaN / 64; ++i) copy(db + i * 8192, t.b, bn + i * 64, bk);
                    } else {
                        copy(db, t.b, bk, bn);
                    }
                }
                ++issued;
                st.next();
            }
        }
        // every copy has landed before the CTAs may end
        if (leader && rank == 0) {
            for (uint32_t i = issued > C::kStages ? issued - C::kStages : 0; i < issued; ++i)
                if (!mbar_wait(&c.full[i % C::kStages], (i / C::kStages) & 1)) ok = false;
        }
        if (!ok) c.err = 1;
        __syncwarp();
    } else if (warp == 1 && rank == 0) {
        const bool leader = elect_one();
        constexpr uint32_t kType = std::is_same_v<typename P::Type, __nv_bfloat16> ? 1 : 0;
        constexpr uint32_t kIdesc = (1u << 4) | (kType << 7) | (kType << 10) | ((kTileN >> 3) << 17) | ((C::kTileM >> 4) << 24);
        Ring<C::kStages> st;
        Ring<2> dr;
        for (uint32_t j = 0; j < count; ++j) {
            const GemmTile t = p.tile(worker, workers, j);
            const uint32_t idesc = kIdesc | (t.a_mn ? 1u << 15 : 0) | (t.b_mn ? 1u << 16 : 0);
            const uint32_t step_a = t.a_mn ? 2048 >> 4 : 32 >> 4, step_b = t.b_mn ? 2048 >> 4 : 32 >> 4;
            wait(&c.d_empty[dr.i], dr.phase ^ 1, &c.err);
            tc_fence_after();
            const uint32_t d = tmem + dr.i * kTileN;
            for (uint32_t s = 0; s < t.steps; ++s) {
                wait(&c.full[st.i], st.phase, &c.err);
                tc_fence_after();
                if (leader) {
                    const uint32_t sa = smem_u32(ring + st.i * C::kStageBytes), sb = sa + kStageABytes;
                    const uint64_t a = t.a_mn ? smem_desc_mn(sa) : smem_desc(sa);
                    const uint64_t b = t.b_mn ? smem_desc_mn(sb) : smem_desc(sb);
#pragma unroll
                    for (uint32_t k = 0; k < kStepK / 16; ++k)
                        gemm_mma<kPair>(d, a + k * step_a, b + k * step_b, idesc, s > 0 || k > 0);
                    gemm_commit<kPair>(&c.empty[st.i]);
                }
                __syncwarp();
                st.next();
            }
            if (leader) gemm_commit<kPair>(&c.d_full[dr.i]);
            __syncwarp();
            dr.next();
        }
        // no product is in flight when the tensor memory is given back
        if (leader) gemm_commit_here<kPair>(&c.drain);
        if (!mbar_wait(&c.drain, 0)) c.err = 1;
        __syncwarp();
    } else if (warp >= 4) {
        const uint32_t quarter = warp & 3, half = (warp - 4) >> 2;
        EpiWarp w;
        w.row = rank * kCtaM + quarter * 32 + lane;
        w.col = half * 128;
        w.lane = lane;
        w.store = store + (warp - 4) * kStoreBytes;
        Ring<2> dr;
        for (uint32_t j = 0; j < count; ++j) {
            const GemmTile t = p.tile(worker, workers, j);
            wait(&c.d_full[dr.i], dr.phase, &c.err);
            tc_fence_after();
            const uint32_t d = tmem + (quarter << 21) + dr.i * kTileN + half * 128;
            p.epilogue(t, w, [&](uint32_t i, float(&v)[32]) {
                uint32_t r[32];
                __syncwarp();
                tmem_ld(d + i * 32, r);
                if (i == 3) {  // the buffer is read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (kPair) arrive_cluster(first_cta(&c.d_empty[dr.i]));
                        else arrive(&c.d_empty[dr.i]);
                    }
                }
#pragma unroll
                for (uint32_t k = 0; k < 32; ++k) v[k] = __uint_as_float(r[k]);
            });
            dr.next();
        }
        if (lane == 0) store_wait();
        __syncwarp();
    }
    tc_fence_before();
    if constexpr (kPair) cluster_sync_all();
    else __syncthreads();
    tc_fence_after();
    if (warp == 2) {
        if constexpr (kPair) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
        else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
    if (tid == 0 && c.err) atomicOr(p.error, kErrTimeout);
}

template <typename P, bool kPair>
inline sel_status launch_gemm(const P& p, uint32_t workers, cudaStream_t stream) {
    using C = GemmConfig<kPair>;
    if (!dynamic_smem_once<gemm_kernel<P, kPair>>(C::kSmem)) return SEL_ECUDA;
    cudaError_t e;
    if constexpr (kPair)
        e = launch_pdl_cluster(gemm_kernel<P, kPair>, dim3(2 * workers), dim3(kGemmThreads), 2, C::kSmem, stream, p);
    else
        e = launch_pdl(gemm_kernel<P, kPair>, dim3(workers), dim3(kGemmThreads), C::kSmem, stream, p);
    return e == cudaSuccess ? SEL_OK : SEL_ECUDA;
}

}  // namespace sel
