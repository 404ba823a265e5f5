// sel_embed.cu -- the input vectors of drawn ids: rows of a table, or of the
// 4-bit matrix that also serves as the output head, times a scale.
//
// Each output element is one rounding of scale * E[id][h], formed in fp32:
// for 4-bit rows s * (q - z) is exact there (at most 11 + 8 significant bits).
// An id >= V (SEL_INVALID_ID among them: a failed row, or the places behind a
// sequence's last emitted token) gives zeros, and reads nothing of the table.
//
// Bound by memory: each table row is read once and each output row written
// once. A thread owns one 16-byte output vector, so loads and stores of a
// warp are contiguous; the vectors of all rows form one index space, so that
// a single long row spreads over several blocks and many short rows fill one.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "sel.h"
#include "sel_common.cuh"
#include "sel_dtype.cuh"
#include "sel_plan.h"
#include "sel_units.cuh"

namespace sel {
namespace {

constexpr int kNT = 256;

struct EmbedArgs {
    const uint32_t* ids;
    const void* table;  // [V][H], or the packed rows [V][H / 2]
    const void* scales;  // 4-bit: [V][H / group]
    const uint8_t* zeros;  // 4-bit: [V][H / group] or null (8)
    void* out;           // [n][H]
    uint64_t total;      // output vectors (or elements): n * per_row
    uint32_t per_row;    // vectors (or elements) a row
    uint32_t V, H, group;
    float scale;
};

// One 16-byte vector (kVec) or one element of a table row.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kNT) embed_kernel(EmbedArgs a) {
    pdl_wait();
    pdl_trigger();
    const uint64_t i = static_cast<uint64_t>(blockIdx.x) * kNT + threadIdx.x;
    if (i >= a.total) return;
    const uint64_t row = i / a.per_row;
    const uint32_t c = static_cast<uint32_t>(i - row * a.per_row);
    const uint32_t id = a.ids[row];
    constexpr int kPer = 16 / sizeof(T);
    if (kVec) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (id < a.V) {
            v = ldg_stream16(static_cast<const T*>(a.table) + static_cast<size_t>(id) * a.H + static_cast<size_t>(c) * kPer);
            T* e = reinterpret_cast<T*>(&v);
#pragma unroll
            for (int j = 0; j < kPer; ++j) e[j] = from_f32<T>(to_f32(e[j]) * a.scale);
        }
        reinterpret_cast<uint4*>(a.out)[i] = v;
    } else {
        float x = 0.0f;
        if (id < a.V) x = to_f32(static_cast<const T*>(a.table)[static_cast<size_t>(id) * a.H + c]) * a.scale;
        static_cast<T*>(a.out)[i] = from_f32<T>(x);
    }
}

// Eight columns (one 32-bit word of nibbles, one 16-byte output vector).
template <typename T>
__global__ void __launch_bounds__(kNT) embed_w4_kernel(EmbedArgs a) {
    pdl_wait();
    pdl_trigger();
    const uint64_t i = static_cast<uint64_t>(blockIdx.x) * kNT + threadIdx.x;
    if (i >= a.total) return;
    const uint64_t row = i / a.per_row;
    const uint32_t c = static_cast<uint32_t>(i - row * a.per_row);
    const uint32_t id = a.ids[row];
    uint4 v = make_uint4(0, 0, 0, 0);
    if (id < a.V) {
        const uint32_t w = static_cast<const uint32_t*>(a.table)[static_cast<size_t>(id) * a.per_row + c];
        const size_t g = static_cast<size_t>(id) * (a.H / a.group) + (c * 8u) / a.group;
        const float s = to_f32(static_cast<const T*>(a.scales)[g]);
        const int z = a.zeros ? a.zeros[g] & 15 : 8;
        T* e = reinterpret_cast<T*>(&v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            e[j] = from_f32<T>(s * static_cast<float>(static_cast<int>((w >> (4 * j)) & 15u) - z) * a.scale);
    }
    reinterpret_cast<uint4*>(a.out)[i] = v;
}

template <typename K>
sel_status launch(K kernel, const EmbedArgs& a, cudaStream_t stream) {
    const uint64_t blocks = (a.total + kNT - 1) / kNT;
    if (blocks > 0x7fffffffull) return SEL_EUNSUPPORTED;
    const cudaError_t e = launch_pdl(kernel, dim3(static_cast<uint32_t>(blocks)), dim3(kNT), 0, stream, a);
    return e == cudaSuccess ? SEL_OK : SEL_ECUDA;
}

template <typename T>
sel_status embed(EmbedArgs a, uint32_t n, cudaStream_t stream) {
    const bool vec = reinterpret_cast<uintptr_t>(a.table) % 16 == 0 && reinterpret_cast<uintptr_t>(a.out) % 16 == 0 &&
                     (static_cast<uint64_t>(a.H) * sizeof(T)) % 16 == 0;
    a.per_row = vec ? static_cast<uint32_t>(a.H * sizeof(T) / 16) : a.H;
    a.total = static_cast<uint64_t>(n) * a.per_row;
    return vec ? launch(embed_kernel<T, true>, a, stream) : launch(embed_kernel<T, false>, a, stream);
}

}  // namespace
}  // namespace sel

using namespace sel;

extern "C" sel_status sel_embed(const uint32_t* d_ids, uint32_t n, const void* d_table, int dtype, uint32_t V,
                                uint32_t H, float scale, void* d_out, cudaStream_t stream) {
    const uint32_t size = dtype_bytes(dtype);
    if (size == 0 || V == 0 || V > SEL_MAX_V || H == 0 || H > SEL_MAX_H) return SEL_EINVAL;
    if (n == 0) return SEL_OK;
    if (!d_ids || !d_table || !d_out) return SEL_EINVAL;
    if (misaligned(d_ids, 4) || misaligned(d_table, size) || misaligned(d_out, size)) return SEL_EINVAL;
    EmbedArgs a{};
    a.ids = d_ids;
    a.table = d_table;
    a.out = d_out;
    a.V = V;
    a.H = H;
    a.scale = scale;
    switch (dtype) {
        case SEL_F32: return embed<float>(a, n, stream);
        case SEL_F16: return embed<__half>(a, n, stream);
        default: return embed<__nv_bfloat16>(a, n, stream);
    }
}

extern "C" sel_status sel_embed_w4(const uint32_t* d_ids, uint32_t n, const uint8_t* d_q, const void* d_scales,
                                   const uint8_t* d_zeros, uint32_t group, int dtype, uint32_t V, uint32_t H,
                                   float scale, void* d_out, cudaStream_t stream) {
    if (const sel_status s = check_w4(dtype, V, H, group); s != SEL_OK) return s;
    if (n == 0) return SEL_OK;
    if (!d_ids || !d_q || !d_scales || !d_out) return SEL_EINVAL;
    if (misaligned(d_ids, 4) || misaligned(d_q, 16) || misaligned(d_scales, 2) || misaligned(d_out, 16)) return SEL_EINVAL;
    EmbedArgs a{};
    a.ids = d_ids;
    a.table = d_q;
    a.scales = d_scales;
    a.zeros = d_zeros;
    a.out = d_out;
    a.V = V;
    a.H = H;
    a.group = group;
    a.scale = scale;
    a.per_row = H / 8;
    a.total = static_cast<uint64_t>(n) * a.per_row;
    return dtype == SEL_F16 ? launch(embed_w4_kernel<__half>, a, stream)
                            : launch(embed_w4_kernel<__nv_bfloat16>, a, stream);
}
