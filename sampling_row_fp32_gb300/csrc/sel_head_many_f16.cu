// sel_head_many_f16.cu -- sel_head_many.cuh for f16 hidden states (the operand
// types compile side by side).
#include "sel_head_many.cuh"

namespace sel {

template sel_status head_many<__half>(const HeadIn&, const HeadArgs&, cudaStream_t);

}  // namespace sel
