// sel_head.cu -- logits rows of hidden states through a 4-bit output head.
//
//   L[r][v] = sum_g s[v][g] * sum_{k in g} x[r][k] * (q[v][k] - z[v][g])
//
// x is a 16-bit float and q - z a small integer, so every product is exact in
// fp32; a group's products are summed in fp32 before its scale is applied.
//
// One warp per matrix row and eight hidden rows: a lane takes a 32-bit word
// (eight columns, which never straddle a group) at a time.
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
constexpr int kRows = 8;  // hidden rows a warp carries at once

struct HeadArgs {
    const void* x;
    const uint32_t* q;
    const void* scales;
    const uint8_t* zeros;
    void* out;
    uint64_t ld;
    uint32_t rows, V, H, group;
};

template <typename T, typename O>
__global__ void __launch_bounds__(kNT) head_kernel(HeadArgs a) {
    pdl_wait();
    pdl_trigger();
    const uint32_t lane = threadIdx.x & 31;
    const uint64_t v = static_cast<uint64_t>(blockIdx.x) * (kNT / 32) + (threadIdx.x >> 5);
    if (v >= a.V) return;
    const uint32_t r0 = blockIdx.y * kRows;
    const uint32_t words = a.H / 8, groups = a.H / a.group;
    float acc[kRows] = {};
    for (uint32_t w = lane; w < words; w += 32) {
        const uint32_t nib = a.q[v * words + w];
        const uint64_t g = v * groups + w * 8 / a.group;
        const float s = to_f32(static_cast<const T*>(a.scales)[g]);
        const int z = a.zeros ? a.zeros[g] : 8;
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = static_cast<float>(static_cast<int>((nib >> (4 * j)) & 15u) - z);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (r0 + r < a.rows) {
                const uint4 xv = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) +
                                                                 static_cast<uint64_t>(r0 + r) * a.H + w * 8u);
                const T* e = reinterpret_cast<const T*>(&xv);
                float p = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) p = fmaf(to_f32(e[j]), f[j], p);
                acc[r] = fmaf(s, p, acc[r]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        float t = acc[r];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(kFull, t, o);
        if (lane == 0 && r0 + r < a.rows) static_cast<O*>(a.out)[(r0 + r) * a.ld + v] = from_f32<O>(t);
    }
}

template <typename T, typename O>
sel_status launch(const HeadArgs& a, cudaStream_t stream) {
    const uint32_t gy = ceil_div(a.rows, kRows);
    if (gy > 65535u) return SEL_EUNSUPPORTED;
    const cudaError_t e = launch_pdl(head_kernel<T, O>, dim3(ceil_div(a.V, kNT / 32), gy), dim3(kNT), 0, stream, a);
    return e == cudaSuccess ? SEL_OK : SEL_ECUDA;
}

template <typename T>
sel_status launch_out(int out_dtype, const HeadArgs& a, cudaStream_t stream) {
    switch (out_dtype) {
        case SEL_F32: return launch<T, float>(a, stream);
        case SEL_F16: return launch<T, __half>(a, stream);
        default: return launch<T, __nv_bfloat16>(a, stream);
    }
}

}  // namespace
}  // namespace sel

using namespace sel;

extern "C" sel_status sel_head_w4(const void* d_hidden, uint32_t rows, const uint8_t* d_q, const void* d_scales,
                                  const uint8_t* d_zeros, uint32_t group, int dtype, uint32_t V, uint32_t H,
                                  void* d_logits, int logits_dtype, uint64_t ld, cudaStream_t stream) {
    if (const sel_status s = check_w4(dtype, V, H, group); s != SEL_OK) return s;
    const uint32_t out_size = dtype_bytes(logits_dtype);
    if (out_size == 0 || ld < V || ld > SEL_MAX_LD) return SEL_EINVAL;
    if (rows == 0) return SEL_OK;
    if (!d_hidden || !d_q || !d_scales || !d_logits) return SEL_EINVAL;
    if (misaligned(d_hidden, 16) || misaligned(d_q, 16) || misaligned(d_scales, 2) || misaligned(d_logits, out_size))
        return SEL_EINVAL;
    HeadArgs a{};
    a.x = d_hidden;
    a.q = reinterpret_cast<const uint32_t*>(d_q);
    a.scales = d_scales;
    a.zeros = d_zeros;
    a.out = d_logits;
    a.ld = ld;
    a.rows = rows;
    a.V = V;
    a.H = H;
    a.group = group;
    return dtype == SEL_F16 ? launch_out<__half>(logits_dtype, a, stream)
                            : launch_out<__nv_bfloat16>(logits_dtype, a, stream);
}
