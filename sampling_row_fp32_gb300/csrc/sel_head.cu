// sel_head.cu -- logits rows of hidden states through a 4-bit output head: the
// entry point's checks, and which kernel takes a call.
#include "sel_head.cuh"

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
    if (rows > 0x7fffffffu) return SEL_EUNSUPPORTED;
    HeadArgs a{};
    a.scales = d_scales;
    a.zeros = d_zeros;
    a.out = d_logits;
    a.ld = ld;
    a.out_dtype = logits_dtype;
    a.rows = rows;
    a.V = V;
    a.H = H;
    a.group_log2 = group == 32 ? 5 : group == 64 ? 6 : 7;
    const HeadIn in{d_hidden, d_q};
    if (head_few_fits(rows, H)) return head_few(dtype, in, a, stream);
    return dtype == SEL_F16 ? head_many<__half>(in, a, stream) : head_many<__nv_bfloat16>(in, a, stream);
}
