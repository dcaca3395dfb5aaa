// Products in INT8 with a scale per row and per output column, dense and by expert group, and the gate/up
// half of the SwiGLU FFN: sums in 32-bit integers (exact), scaled once in the epilogue.
#include "grouped_tiles.h"

namespace moe {

namespace {

using Large = GtCfg<ElI8, 4, 2, 2, 4>;
using Small = GtCfg<ElI8, 2, 2, 2, 2>;

template <bool OUT_F32, bool GATED>
moe_status_t launch(const GgArgs& a, hipStream_t s) {
  if (few_large_tiles(a, false, GATED ? 2 * a.N : a.N)) return launch_gg_tiles<ElI8, true, true, OUT_F32, GATED, Small>(a, s);
  return launch_gg_tiles<ElI8, true, true, OUT_F32, GATED, Large>(a, s);
}

}  // namespace

moe_status_t launch_matmul_int8(const GgArgs& a, moe_dtype_t out, hipStream_t s) {
  return out == MOE_F32 ? launch<true, false>(a, s) : launch<false, false>(a, s);
}

moe_status_t launch_gate_up_int8(const GgArgs& a, hipStream_t s) { return launch<false, true>(a, s); }

}  // namespace moe
