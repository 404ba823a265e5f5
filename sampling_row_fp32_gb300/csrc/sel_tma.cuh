// sel_tma.cuh -- tensor copies into a ring of shared-memory stages: the copies,
// the ring's barriers with bounded waits, and the tensor maps.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "sel_common.cuh"
#include "sel_units.cuh"

namespace sel {

__device__ __forceinline__ void tma_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}
// Brings the box into L2. Allowed before this launch's predecessor is done: what
// that one still writes, L2 has too. A CTA's first stages asked for so, launch
// after launch: 5 rows of 2,880 x 93,001 49.0 -> 47.6 us, 49 of 4,096 x 248,320
// 197.8 -> 192.0.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void expect_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// A slot of a ring of barriers and the parity of the round it is in.
template <uint32_t kN>
struct Ring {
    uint32_t i = 0, phase = 0;
    __device__ __forceinline__ void next() {
        if (++i == kN) {
            i = 0;
            phase ^= 1;
        }
    }
};

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// Waits for a barrier's phase. A wait that runs out raises `err`, and with
// `err` raised every other one returns at once: the roles then run to their
// ends on whatever the buffers hold (in bounds as ever) and the CTA's logits
// become NaN.
__device__ __forceinline__ void wait_slow(uint64_t* bar, uint32_t phase, volatile uint32_t* err) {
    for (uint32_t i = 0; i < kWaitPolls; ++i) {
        if (mbar_try_wait(bar, phase) || *err) return;
    }
    *err = 1;
}
__device__ __forceinline__ void wait(uint64_t* bar, uint32_t phase, uint32_t* err) {
    if (!mbar_try_wait(bar, phase)) wait_slow(bar, phase, err);
    __syncwarp();
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_tiled() {
    static const EncodeTiled f = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult r{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return f;
}

// A row-major matrix [rows][cols], its rows `pitch` bytes apart (0: without
// gaps), read in boxes of box_cols x box_rows.
inline bool make_map(CUtensorMap* map, CUtensorMapDataType type, uint32_t elem, const void* base, uint64_t cols, uint64_t rows,
              uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swizzle, uint64_t pitch = 0) {
    const EncodeTiled f = encode_tiled();
    if (!f) return false;
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {pitch ? pitch : cols * elem};
    const cuuint32_t box[2] = {box_cols, box_rows}, step[2] = {1, 1};
    auto encode = [&] {
        return f(map, type, 2, const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                 CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    if (encode()) return true;
    // A host thread whose first CUDA call this is has no context yet, which the
    // driver's function, unlike the runtime's, does not see to.
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && encode();
}

}  // namespace sel
