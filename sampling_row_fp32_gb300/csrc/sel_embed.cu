// sel_embed.cu -- the input vectors of drawn ids: rows of a table, or of the
// 4-bit matrix that also serves as the output head, times a scale.
//
// Each output element is one rounding of scale * E[id][h], formed in fp32:
// for 4-bit rows s * (q - z) is exact there (at most 11 + 8 significant bits).
// An id >= V (SEL_INVALID_ID among them: a failed row, or the places behind a
// sequence's last emitted token) gives zeros, and reads nothing of the table.
//
// Bound by memory: each table row is read once and each output row written
// once. A block takes up to 512 of a row's 16-byte output vectors, four a
// thread whose loads are on their way together (a row alone is then spread
// over several blocks); loads and stores of a warp are contiguous. 16,384 rows
// of 5,120 bf16: 49 us, 6.8 TB/s.
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

constexpr int kPer = 4;        // vectors (or elements) a thread
constexpr uint32_t kMaxNT = 128;

struct EmbedArgs {
    const uint32_t* ids;
    const void* table;  // [V][H], or the packed rows [V][H / 2]
    const void* scales;  // 4-bit: [V][H / group]
    const uint8_t* zeros;  // 4-bit: [V][H / group] or null (8)
    void* out;           // [n][H]
    uint32_t per_row;    // vectors (or elements) a row
    uint32_t chunks, chunk;  // blocks a row, vectors a block
    uint32_t V, H, group_log2;
    float scale;
};

// The block's row, its id, and the vectors [c0, c1) of the row.
struct Piece {
    uint64_t row;
    uint32_t id, c0, c1;
};
__device__ __forceinline__ Piece piece(const EmbedArgs& a) {
    Piece p;
    p.row = blockIdx.x / a.chunks;
    p.c0 = (blockIdx.x % a.chunks) * a.chunk;
    p.c1 = min(a.per_row, p.c0 + a.chunk);
    p.id = a.ids[p.row];
    return p;
}

// 16-byte vectors (kVec) or elements of a table row.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kMaxNT) embed_kernel(EmbedArgs a) {
    pdl_wait();
    pdl_trigger();
    const Piece p = piece(a);
    if constexpr (kVec) {
        const uint4* src = static_cast<const uint4*>(a.table) + static_cast<uint64_t>(p.id) * a.per_row;
        uint4* dst = static_cast<uint4*>(a.out) + p.row * a.per_row;
        uint4 v[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const uint32_t c = p.c0 + j * blockDim.x + threadIdx.x;
            v[j] = make_uint4(0, 0, 0, 0);
            if (c < p.c1 && p.id < a.V) v[j] = ldg_stream16(src + c);
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const uint32_t c = p.c0 + j * blockDim.x + threadIdx.x;
            T* e = reinterpret_cast<T*>(&v[j]);
#pragma unroll
            for (int k = 0; k < static_cast<int>(16 / sizeof(T)); ++k) e[k] = from_f32<T>(to_f32(e[k]) * a.scale);
            if (p.id >= a.V) v[j] = make_uint4(0, 0, 0, 0);  // (0 * scale may be NaN)
            if (c < p.c1) dst[c] = v[j];
        }
    } else {
        const T* src = static_cast<const T*>(a.table) + static_cast<uint64_t>(p.id) * a.H;
        T* dst = static_cast<T*>(a.out) + p.row * a.H;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const uint32_t c = p.c0 + j * blockDim.x + threadIdx.x;
            if (c < p.c1) dst[c] = p.id < a.V ? from_f32<T>(to_f32(src[c]) * a.scale) : from_f32<T>(0.0f);
        }
    }
}

// Vectors of eight columns: one 32-bit word of nibbles each.
template <typename T>
__global__ void __launch_bounds__(kMaxNT) embed_w4_kernel(EmbedArgs a) {
    pdl_wait();
    pdl_trigger();
    const Piece p = piece(a);
    const uint32_t* src = static_cast<const uint32_t*>(a.table) + static_cast<uint64_t>(p.id) * a.per_row;
    const uint64_t g0 = static_cast<uint64_t>(p.id) * (a.H >> a.group_log2);
    uint4* dst = static_cast<uint4*>(a.out) + p.row * a.per_row;
    uint32_t w[kPer];
    float s[kPer];
    int z[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const uint32_t c = p.c0 + j * blockDim.x + threadIdx.x;
        w[j] = 0;
        s[j] = 0.0f;
        z[j] = 8;
        if (c < p.c1 && p.id < a.V) {
            const uint64_t g = g0 + (c * 8u >> a.group_log2);
            w[j] = src[c];
            s[j] = to_f32(static_cast<const T*>(a.scales)[g]);
            if (a.zeros) z[j] = a.zeros[g] & 15;
        }
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const uint32_t c = p.c0 + j * blockDim.x + threadIdx.x;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (p.id < a.V) {
            T* e = reinterpret_cast<T*>(&v);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                e[k] = from_f32<T>(s[j] * static_cast<float>(static_cast<int>((w[j] >> (4 * k)) & 15u) - z[j]) * a.scale);
        }
        if (c < p.c1) dst[c] = v;
    }
}

// per_row vectors a row, in equal pieces of at most kPer a thread.
template <typename K>
sel_status launch(K kernel, EmbedArgs a, uint32_t n, cudaStream_t stream) {
    a.chunks = ceil_div(a.per_row, kPer * kMaxNT);
    a.chunk = ceil_div(a.per_row, a.chunks);
    const uint64_t blocks = static_cast<uint64_t>(n) * a.chunks;
    if (blocks > 0x7fffffffull) return SEL_EUNSUPPORTED;
    const uint32_t nt = ceil_div(ceil_div(a.chunk, kPer), 32) * 32;
    const cudaError_t e = launch_pdl(kernel, dim3(static_cast<uint32_t>(blocks)), dim3(nt), 0, stream, a);
    return e == cudaSuccess ? SEL_OK : SEL_ECUDA;
}

template <typename T>
sel_status embed(EmbedArgs a, uint32_t n, cudaStream_t stream) {
    const bool vec = reinterpret_cast<uintptr_t>(a.table) % 16 == 0 && reinterpret_cast<uintptr_t>(a.out) % 16 == 0 &&
                     (static_cast<uint64_t>(a.H) * sizeof(T)) % 16 == 0;
    a.per_row = vec ? static_cast<uint32_t>(a.H * sizeof(T) / 16) : a.H;
    return vec ? launch(embed_kernel<T, true>, a, n, stream) : launch(embed_kernel<T, false>, a, n, stream);
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
    a.group_log2 = group == 32 ? 5 : group == 64 ? 6 : 7;
    a.scale = scale;
    a.per_row = H / 8;
    return dtype == SEL_F16 ? launch(embed_w4_kernel<__half>, a, n, stream)
                            : launch(embed_w4_kernel<__nv_bfloat16>, a, n, stream);
}
