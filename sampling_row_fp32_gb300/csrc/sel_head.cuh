// sel_head.cuh -- what the kernels of the 4-bit output head share: the ring of
// weight stages, nibbles to operands, group entries, and the weights' maps.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "sel.h"
#include "sel_common.cuh"
#include "sel_dtype.cuh"
#include "sel_plan.h"
#include "sel_tma.cuh"
#include "sel_units.cuh"

namespace sel {

// A stage holds 256 columns (128 bytes) of up to 256 matrix rows, with the
// 128-byte swizzle: 16-byte chunk ch of row r lies at ch ^ (r & 7).
constexpr uint32_t kTileV = 256;   // matrix rows a tile
constexpr uint32_t kBoxV = 32;     // rows a copy of a partial tile
constexpr uint32_t kStageK = 256;  // columns a stage
constexpr uint32_t kUnitK = 128;   // columns whose group entries are read together
constexpr uint32_t kWBytes = kTileV * kStageK / 2;

struct HeadArgs {
    const void* scales;
    const uint8_t* zeros;
    void* out;
    uint64_t ld;
    int out_dtype;
    uint32_t rows, V, H, group_log2;
    uint32_t range;  // matrix rows a CTA
};

struct HeadIn {
    const void* x;
    const void* q;
};

// At most 8 hidden rows (the columns of one warp-level product) that fit shared
// memory next to a ring of at least three stages. Times of 1 / 2 / 4 / 8 rows in
// us, head_few against the tcgen05 kernel:
//   4,096 x 248,320, groups of 64     99 / 107 / 110 / 114    115 / 116 / 116 / 116
//   4,096 x 248,320, groups of 128    94 / 95 / 98 / 104      110 / 110 / 110 / 111
//   8,192 x 202,048, 128, zeros      168 / 173 / 180 / 199    199 / 199 / 199 / 199
//   2,880 x 93,001, 32, zeros (f16)   47 / 48 / 48 / 52       128 / 128 / 128 / 128
//   1,024 x 151,936, groups of 64     20 / 20 / 20 / 22        22 / 22 / 22 / 23
// 16 rows, two products a pair of words, took head_few 155 at the first size
// against 117.
inline bool head_few_fits(uint32_t rows, uint32_t H) {
    return rows <= 8 && static_cast<uint64_t>(rows) * ceil_div(H, kStageK) * kStageK * 2 <= 128u * 1024u;
}
sel_status head_few(int dtype, const HeadIn& in, const HeadArgs& a, cudaStream_t stream);

// Any number of hidden rows; the matrix is read once for every 64.
template <typename T>
sel_status head_many(const HeadIn& in, const HeadArgs& a, cudaStream_t stream);

template <typename T>
struct Unpack;
template <>
struct Unpack<__nv_bfloat16> {
    static constexpr uint32_t kMagic = 0x43004300u;  // 128: the mantissa's last bit is 1
    static constexpr uint32_t kType = 1;
    static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
};
template <>
struct Unpack<__half> {
    static constexpr uint32_t kMagic = 0x64006400u;  // 1024
    static constexpr uint32_t kType = 0;
    static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
};

// Group entries (scales or zero points) travel with their stage: helper warps
// load the rows' entries of the stage and leave them in shared memory. Read by
// their users straight from global memory they stalled them for up to a third
// of a call, prefetched a stage ahead or not: a row's entries of a stage are a
// piece far smaller than a line.

template <uint32_t kBytes>
struct Word;
template <>
struct Word<16> { using Type = uint4; };
template <>
struct Word<8> { using Type = uint2; };
template <>
struct Word<4> { using Type = uint32_t; };
template <>
struct Word<2> { using Type = uint16_t; };
template <>
struct Word<1> { using Type = uint8_t; };

// A warp copies kBytes bytes at byte `at` of each of `rows` rows of row_bytes
// bytes, zeros past a row's end, as words of kW bytes (which divide the rows'
// addresses and length, so that a word is all in a row or all past its end).
// Neighbouring lanes take neighbouring words; u0 is the lane's first.
template <uint32_t kBytes, uint32_t kW, uint32_t kBatch>
__device__ __forceinline__ void load_words(typename Word<kW>::Type (&v)[kBatch], const unsigned char* src, uint32_t at,
                                           uint32_t row_bytes, uint32_t rows, uint32_t u0) {
    using W = typename Word<kW>::Type;
    constexpr uint32_t kPerRow = kBytes / kW;
#pragma unroll
    for (uint32_t j = 0; j < kBatch; ++j) {
        const uint32_t u = u0 + 32 * j, off = at + u % kPerRow * kW;
        v[j] = W{};
        if (u < rows * kPerRow && off < row_bytes)
            v[j] = *reinterpret_cast<const W*>(src + static_cast<uint64_t>(u / kPerRow) * row_bytes + off);
    }
}
template <uint32_t kBytes, uint32_t kW, uint32_t kBatch>
__device__ __forceinline__ void store_words(unsigned char* dst, const typename Word<kW>::Type (&v)[kBatch], uint32_t rows,
                                            uint32_t u0) {
#pragma unroll
    for (uint32_t j = 0; j < kBatch; ++j) {
        const uint32_t u = u0 + 32 * j;
        if (u < rows * (kBytes / kW)) *reinterpret_cast<typename Word<kW>::Type*>(dst + u * kW) = v[j];
    }
}
template <uint32_t kBytes, uint32_t kW, uint32_t kBatch>
__device__ __forceinline__ void copy_words(unsigned char* dst, const unsigned char* src, uint32_t at, uint32_t row_bytes,
                                           uint32_t rows) {
    for (uint32_t u0 = threadIdx.x & 31; u0 < rows * (kBytes / kW); u0 += 32 * kBatch) {
        typename Word<kW>::Type v[kBatch];
        load_words<kBytes, kW, kBatch>(v, src, at, row_bytes, rows, u0);
        store_words<kBytes, kW, kBatch>(dst, v, rows, u0);
    }
}
template <uint32_t kBytes, uint32_t kBatch>
__device__ __forceinline__ void copy_rows(unsigned char* dst, const unsigned char* src, uint32_t at, uint32_t row_bytes,
                                          uint32_t rows, uint32_t width) {
    // (narrow words: twice as many on their way, 49 us against 54 for 5 rows of
    // 2,880 x 93,001 with groups of 32, whose rows of scales are 180 bytes)
    if (width >= kBytes) copy_words<kBytes, kBytes, kBatch>(dst, src, at, row_bytes, rows);
    else if (kBytes > 4 && width >= 4) copy_words<kBytes, kBytes < 4 ? kBytes : 4, 2 * kBatch>(dst, src, at, row_bytes, rows);
    else if (kBytes > 2 && width >= 2) copy_words<kBytes, 2, 2 * kBatch>(dst, src, at, row_bytes, rows);
    else copy_words<kBytes, 1, 2 * kBatch>(dst, src, at, row_bytes, rows);
}
template <uint32_t kBytes>
__device__ __forceinline__ void read_entries(uint32_t src, uint32_t (&v)[(kBytes + 3) / 4]) {
    if constexpr (kBytes == 16)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(src));
    else if constexpr (kBytes == 8) asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(src));
    else if constexpr (kBytes == 4) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v[0]) : "r"(src));
    else {
        uint16_t u;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(u) : "r"(src));
        v[0] = u;
    }
}
// Entry e (a constant after unrolling) of the words that read_entries gave.
__device__ __forceinline__ uint16_t entry16(const uint32_t* v, uint32_t e) {
    return static_cast<uint16_t>(v[e / 2] >> (16 * (e % 2)));
}
__device__ __forceinline__ uint32_t zero_point(const uint32_t* v, uint32_t e) { return (v[e / 4] >> (8 * (e % 4))) & 15; }

// Largest power of two up to 16 that divides an address and a row's length.
__device__ __forceinline__ uint32_t entry_width(const void* p, uint32_t row_bytes) {
    const uint32_t bits = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) | row_bytes | 16u;
    return bits & (~bits + 1);
}

// Bytes of a stage's entries for one matrix row.
template <int kGroupLog2>
struct EntryBytes {
    static constexpr uint32_t kGroups = kStageK >> kGroupLog2;
    static constexpr uint32_t kScales = 2 * kGroups, kZeros = kGroups;
};
inline uint32_t entry_row_bytes(uint32_t group_log2, bool zeros) { return (kStageK >> group_log2) * (zeros ? 3 : 2); }

// A helper warp's share of a CTA's stages: number first, first + step, ...
// `wait_empty(slot, phase)` waits for a slot, `done(slot)` reports it filled.
template <int kGroupLog2, bool kZeros, uint32_t kBatch, typename Wait, typename Done>
__device__ __forceinline__ void copy_entries(const HeadArgs& a, unsigned char* entries, uint32_t slot_bytes, uint32_t tile,
                                             uint32_t slots, uint32_t first, uint32_t step,
                                             uint32_t v_begin, uint32_t v_end, Wait wait_empty, Done done) {
    using B = EntryBytes<kGroupLog2>;
    const uint32_t groups = a.H >> kGroupLog2, stages = (a.H + kStageK - 1) / kStageK;
    const auto* scales = static_cast<const unsigned char*>(a.scales);
    const uint32_t ws = entry_width(scales, 2 * groups), wz = kZeros ? entry_width(a.zeros, groups) : 0;
    uint32_t slot = 0, phase = 0, turn = first;  // stages until this warp's next one
    for (uint32_t vt = v_begin; vt < v_end; vt += tile) {
        const uint32_t rows = min(tile, v_end - vt);
        for (uint32_t i = 0; i < stages; ++i) {
            if (turn == 0) {
                turn = step;
                wait_empty(slot, phase);
                unsigned char* dst = entries + slot * slot_bytes;
                const uint64_t row = static_cast<uint64_t>(vt) * groups;
                copy_rows<B::kScales, kBatch>(dst, scales + 2 * row, i * B::kScales, 2 * groups, rows, ws);
                if (kZeros)
                    copy_rows<B::kZeros, kBatch>(dst + tile * B::kScales, a.zeros + row, i * B::kZeros, groups, rows, wz);
                __syncwarp();
                done(slot);
            }
            --turn;
            if (++slot == slots) {
                slot = 0;
                phase ^= 1;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// Packed weights in copies of box_rows rows of a stage.
inline bool make_weight_map(CUtensorMap* map, const void* q, uint32_t V, uint32_t H, uint32_t box_rows) {
    return make_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, q, H / 2, V, kStageK / 2, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Rows a CTA takes: all SMs, as even as whole copies allow.
inline uint32_t head_range(uint32_t V, int sms) {
    return ceil_div(ceil_div(V, static_cast<uint64_t>(sms)), kBoxV) * kBoxV;
}

}  // namespace sel
