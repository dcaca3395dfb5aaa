// Products of ragged expert groups in bf16 and fp32, and the gradient of their weights ("Distributed
// expert parallelism", "Grouped expert computation": one launch for every expert's variable-size group;
// MoonEP "Integration": stacked weights, cu_seqlens selecting each expert's rows).
#include "grouped_gemm.h"

namespace moe {

moe_status_t launch_grouped_matmul(const GgArgs& a, moe_dtype_t dt, bool transposed, moe_dtype_t out, hipStream_t s) {
  if (dt == MOE_F32) return transposed ? launch_gg_any<ElF32, true, true, true>(a, s) : launch_gg_any<ElF32, true, false, true>(a, s);
  if (out == MOE_F32)
    return transposed ? launch_gg_any<ElBf16, true, true, true>(a, s) : launch_gg_any<ElBf16, true, false, true>(a, s);
  return transposed ? launch_gg_any<ElBf16, true, true, false>(a, s) : launch_gg_any<ElBf16, true, false, false>(a, s);
}

moe_status_t launch_grouped_wgrad(const GgArgs& a, moe_dtype_t dt, moe_dtype_t out, hipStream_t s) {
  if (dt == MOE_F32) return launch_gg_any<ElF32, false, false, true>(a, s);
  if (out == MOE_F32) return launch_gg_any<ElBf16, false, false, true>(a, s);
  return launch_gg_any<ElBf16, false, false, false>(a, s);
}

}  // namespace moe
