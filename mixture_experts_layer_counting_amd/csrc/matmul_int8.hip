// Products in INT8 with a scale per row and per output column, dense and by expert group, and the gate/up
// half of the SwiGLU FFN: sums in 32-bit integers (exact), scaled once in the epilogue.
#include "grouped_stream.h"
#include "grouped_tiles.h"

namespace moe {

namespace {

template <bool OUT_F32, bool GATED>
moe_status_t launch(const GgArgs& a, hipStream_t s) {
  switch (gg_form(a, false, true, false, GATED ? 2 * a.N : a.N)) {
    case GG_STREAM:  // (not where rows are gathered from no token at all)
      if (!a.row_src || a.a_rows > 0) return launch_gg_stream<ElI8, true, OUT_F32, GATED>(a, s);
      [[fallthrough]];
    case GG_THIN: return launch_gg_tiles<ElI8, true, true, OUT_F32, GATED, GtThin<ElI8>>(a, s);
    case GG_SMALL: return launch_gg_tiles<ElI8, true, true, OUT_F32, GATED, GtSmall<ElI8>>(a, s);
    default: return launch_gg_tiles<ElI8, true, true, OUT_F32, GATED, GtLarge<ElI8>>(a, s);
  }
}

}  // namespace

moe_status_t launch_matmul_int8(const GgArgs& a, moe_dtype_t out, hipStream_t s) {
  return out == MOE_F32 ? launch<true, false>(a, s) : launch<false, false>(a, s);
}

moe_status_t launch_gate_up_int8(const GgArgs& a, hipStream_t s) { return launch<false, true>(a, s); }

}  // namespace moe
