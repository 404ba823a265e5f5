// sel_head_many_bf16.cu -- sel_head_many.cuh for bf16 hidden states (the operand
// types compile side by side).
#include "sel_head_many.cuh"

namespace sel {

template sel_status head_many<__nv_bfloat16>(const HeadIn&, const HeadArgs&, cudaStream_t);

}  // namespace sel
