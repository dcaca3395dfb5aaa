// Products of ragged expert groups in bf16 and fp32, and the gradient of their weights ("Distributed
// expert parallelism", "Grouped expert computation": one launch for every expert's variable-size group;
// MoonEP "Integration": stacked weights, cu_seqlens selecting each expert's rows).
#include "grouped_stream.h"
#include "grouped_tiles.h"

namespace moe {

namespace {

template <class EL, bool AKC, bool BKC, bool OUT_F32>
moe_status_t launch(const GgArgs& a, hipStream_t s) {
  constexpr int ES = EL::BYTES;
  // whole 16-byte words along every axis that a load runs along
  const bool words = (size_t)a.Kd * ES % 16 == 0 && (BKC || (size_t)a.N * ES % 16 == 0) && (uintptr_t)a.A % 16 == 0 &&
                     (uintptr_t)a.B0 % 16 == 0;
  const GgForm form = gg_form(a, !AKC, BKC, ES == 4, a.N);
  if (!words) {
    if constexpr (ES == 2) return launch_gg_any<AKC, BKC, OUT_F32>(a, s);
    else if (form <= GG_THIN) return launch_gg_tiles<EL, AKC, BKC, OUT_F32, false, GtThinDw>(a, s);
    else return launch_gg_tiles<EL, AKC, BKC, OUT_F32, false, GtSmallDw>(a, s);
  }
  switch (form) {
    case GG_STREAM:  // (not where rows are gathered from no token at all)
      if constexpr (AKC)
        if (!a.row_src || a.a_rows > 0) return launch_gg_stream<EL, BKC, OUT_F32, false>(a, s);
      [[fallthrough]];
    case GG_THIN: return launch_gg_tiles<EL, AKC, BKC, OUT_F32, false, GtThin<EL>>(a, s);
    case GG_SMALL: return launch_gg_tiles<EL, AKC, BKC, OUT_F32, false, GtSmall<EL>>(a, s);
    default: return launch_gg_tiles<EL, AKC, BKC, OUT_F32, false, GtLarge<EL>>(a, s);
  }
}

}  // namespace

moe_status_t launch_grouped_matmul(const GgArgs& a, moe_dtype_t dt, bool transposed, moe_dtype_t out, hipStream_t s) {
  if (dt == MOE_F32) return transposed ? launch<ElF32, true, true, true>(a, s) : launch<ElF32, true, false, true>(a, s);
  if (out == MOE_F32) return transposed ? launch<ElBf16, true, true, true>(a, s) : launch<ElBf16, true, false, true>(a, s);
  return transposed ? launch<ElBf16, true, true, false>(a, s) : launch<ElBf16, true, false, false>(a, s);
}

moe_status_t launch_grouped_wgrad(const GgArgs& a, moe_dtype_t dt, moe_dtype_t out, hipStream_t s) {
  if (dt == MOE_F32) return launch<ElF32, false, false, true>(a, s);
  if (out == MOE_F32) return launch<ElBf16, false, false, true>(a, s);
  return launch<ElBf16, false, false, false>(a, s);
}

}  // namespace moe
