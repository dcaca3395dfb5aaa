// Products in INT8 with a scale per row and per output column, dense and by expert group, and the gate/up
// half of the SwiGLU FFN: sums in 32-bit integers (exact), scaled once in the epilogue.
#include "grouped_gemm.h"

namespace moe {

moe_status_t launch_matmul_int8(const GgArgs& a, moe_dtype_t out, hipStream_t s) {
  if (out == MOE_F32) return launch_gg_any<ElI8, true, true, true>(a, s);
  return launch_gg_any<ElI8, true, true, false>(a, s);
}

moe_status_t launch_gate_up_int8(const GgArgs& a, hipStream_t s) {
  return launch_gg_any<ElI8, true, true, false, true>(a, s);
}

}  // namespace moe
