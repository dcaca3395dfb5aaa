// Routing by scores: sigmoid or softmax scores, an optional per-expert bias that takes part in
// the choice only, optional group limits, top-k, optional renormalisation, and its gradient.
//
// For a token with logits l:
//   s_e = 1 / (1 + exp(-l_e))  or  exp(l_e) / sum exp(l)        (masked experts: none)
//   c_e = s_e + bias_e with a bias, else l_e (the same order as s_e)
//   groups: the topk_groups groups of E/groups neighbouring experts whose group_top largest
//           choices have the largest sum stay; the others' experts drop out
//   picks:  the K largest c (equal: lower id);  w_k = scale * s_k [/ sum over the picks]
// The choices are compared as if in binary64. One wave takes one token with its logits in
// registers. It computes the choices in fp32, whose error the bounds below limit; only where two
// neighbouring picks (or two group scores) lie within their own bound does the wave redo
// the choice in fp64. Everything else needs no 64-bit arithmetic, and the result is the fp64 one
// in every case. Reading the logits once is the whole memory traffic.
//
// Lanes hold experts group by group: p = 64 / (groups rounded up to a power of two) lanes per
// group, so a group's reduction is a butterfly over neighbouring lanes. Without group limits
// that is lane + 64 i.
#include "route_common.h"

namespace moe {

namespace {

constexpr float NEG_INF = -__builtin_inff();
constexpr int RS_WAVES = 4;
constexpr int RS_MAX_E = 1024;
constexpr float HUGE_CHOICE = 1e30f;  // past this a sum of choices or a bound may overflow in fp32
// Eight waves a SIMD where the logits leave the registers for it.
#define RS_OCCUPANCY(items) __attribute__((amdgpu_waves_per_eu((items) <= 8 ? 8 : 1)))

struct ScoredArgs {
  const void* logits;
  const float* bias;
  int T, E, K;
  int bf16, sigmoid, renorm;
  int G, S, lp;  // groups that limit the choice (1: none), experts per group, log2(lanes per group)
  int topk_groups, group_top;
  float scale;
};

// A float as a signed integer of the same order (-0 just below +0; no NaN), and back. Integer
// maxima need no quieting of their operands and take the lane moves as operand modifiers.
__device__ __forceinline__ int order_key(float x) {
  const int b = __float_as_int(x);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float key_value(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7fffffff)); }

// The largest x over the 64 lanes, uniform: within the rows of 16 by lane moves, over the rows in
// scalar registers.
__device__ __forceinline__ int wave_max_key(int x) {
  x = max(x, __builtin_amdgcn_update_dpp(0, x, DPP_XOR1, 0xF, 0xF, true));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, DPP_XOR2, 0xF, 0xF, true));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, DPP_HALF_MIRROR, 0xF, 0xF, true));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, DPP_MIRROR, 0xF, 0xF, true));
  return max(max(__builtin_amdgcn_readlane(x, 0), __builtin_amdgcn_readlane(x, 16)),
             max(__builtin_amdgcn_readlane(x, 32), __builtin_amdgcn_readlane(x, 48)));
}
__device__ __forceinline__ float wave_max(float x) { return key_value(wave_max_key(order_key(x))); }

// LDS written by some lanes of this wave is read by others after this.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A logit, masked (NaN, -inf, the type's lowest value) as -inf, +inf as the largest fp32.
__device__ __forceinline__ float unmask(float x, int bf16) {
  const float lowest = bf16 ? -3.38953139e38f : -3.40282347e38f;
  return x > lowest ? __builtin_amdgcn_fmed3f(x, -3.40282347e38f, 3.40282347e38f) : NEG_INF;
}

__device__ __forceinline__ float read_logit(const void* row, int e, int bf16) {
  return unmask(bf16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(row)[e]) : static_cast<const float*>(row)[e], bf16);
}

__device__ __forceinline__ const void* logit_row(const ScoredArgs& a, int t) {
  return static_cast<const char*>(a.logits) + (size_t)t * a.E * (a.bf16 ? 2 : 4);
}

// The fp32 choices of one lane's experts, -inf where masked, by the logit or by a bias of -inf or NaN (a NaN
// must not go on: fmed3 may return it, and as an integer key it would be the largest). top, total: the softmax's
// largest logit and sum. (The branches are uniform and outside the loops: each loop is straight code.)
template <int ITEMS>
__device__ __forceinline__ void choices(const ScoredArgs& a, bool scores, const float (&l)[ITEMS],
                                        const float (&bias)[ITEMS], float top, float total, float (&s)[ITEMS],
                                        float (&c)[ITEMS]) {
  if (!scores) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) s[i] = 0.f;
  } else if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) s[i] = __builtin_amdgcn_rcpf(1.0f + __expf(-l[i]));
  } else {
    const float inv = 1.0f / total;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) s[i] = __expf(l[i] - top) * inv;
  }
  const bool with_bias = a.bias != nullptr;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    c[i] = with_bias ? s[i] + bias[i] : l[i];
    if (!(l[i] > NEG_INF && c[i] > NEG_INF)) c[i] = NEG_INF;
  }
}

// The fp64 score of a logit.
__device__ __forceinline__ double exact_score(const ScoredArgs& a, float l, float top, double total) {
  return a.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)top) / total;
}

// The softmax's sum in fp64.
template <int ITEMS>
__device__ __forceinline__ double exact_total(const float (&l)[ITEMS], float top) {
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) sum += exp((double)l[i] - (double)top);
  for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d, 64);
  return sum;
}

// A step of a butterfly over neighbouring lanes: xor with D for D < 4, else with the mirror image within 2 D
// lanes, which pairs the same groups once the smaller steps are done.
template <int D, typename F>
__device__ __forceinline__ F pair_lane(F v) {
  constexpr int C = D == 1 ? DPP_XOR1 : D == 2 ? DPP_XOR2 : D == 4 ? DPP_HALF_MIRROR : DPP_MIRROR;
  if constexpr (D >= 16) {
    return __shfl_xor(v, D, 64);
  } else if constexpr (sizeof(F) == 4) {
    return __int_as_float(dpp_mov<C>(__float_as_int(v)));
  } else {
    const int lo = dpp_mov<C>(__double2loint(v)), hi = dpp_mov<C>(__double2hiint(v));
    return __hiloint2double(hi, lo);
  }
}

__device__ __forceinline__ float lane_value(float v, int j) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), j));
}
__device__ __forceinline__ double lane_value(double v, int j) {
  return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), j), __builtin_amdgcn_readlane(__double2loint(v), j));
}

// The two largest choices of a lane's experts, m1 >= m2.
template <typename F>
__device__ __forceinline__ void top_two(F u, F& m1, F& m2) {
  m2 = u > m1 ? m1 : (u > m2 ? u : m2);
  m1 = u > m1 ? u : m1;
}

// How far a choice of value v has to lie from another for their order in fp32 to be the exact one.
struct Bound {
  float base, slope;
  __device__ __forceinline__ float at(float v) const { return base + slope * __builtin_fabsf(v); }
};

// Whether this lane's group stays, from its lanes' two largest choices. In fp32, with a bound > 0, `close` is set
// (for the whole wave) where a kept and a dropped group's scores may be ordered the other way.
template <typename F>
__device__ __forceinline__ bool group_kept(const ScoredArgs& a, int lane, Bound bound, F m1, F m2, bool& close) {
  const F ninf = (F)NEG_INF;
  const int g = lane >> a.lp;
  auto merge = [&](F o1, F o2) {
    const F lo = o1 > m1 ? m1 : o1;
    const F hi = o2 > m2 ? o2 : m2;
    m2 = lo > hi ? lo : hi;
    m1 = o1 > m1 ? o1 : m1;
  };
  if (a.lp >= 1) merge(pair_lane<1>(m1), pair_lane<1>(m2));
  if (a.lp >= 2) merge(pair_lane<2>(m1), pair_lane<2>(m2));
  if (a.lp >= 3) merge(pair_lane<4>(m1), pair_lane<4>(m2));
  if (a.lp >= 4) merge(pair_lane<8>(m1), pair_lane<8>(m2));
  if (a.lp >= 5) merge(pair_lane<16>(m1), pair_lane<16>(m2));
  const bool both = a.group_top == 2 && m2 > ninf;
  F score = both ? m1 + m2 : m1;
  // a sum of huge negative choices stays above a group that has none
  if constexpr (sizeof(F) == 4) score = both ? fmaxf(score, -3.40282347e38f) : score;
  int rank = 0;
  for (int j = 0; j < a.G; ++j) {
    const F o = lane_value(score, j << a.lp);
    const bool before = j < g ? o >= score : o > score;
    rank += before ? 1 : 0;
  }
  const bool kept = g < a.G && rank < a.topk_groups;
  if constexpr (sizeof(F) == 4) {
    if (bound.base > 0.f) {
      // Each of the two largest choices errs by at most a quarter of its bound, their sum by 2^-24 of it: the
      // score stays within `wide` of the exact one, with room for the roundings here. (Two sums of huge negative
      // choices that would overflow lie within `wide` of each other. Huge positive ones go the plain way.)
      const bool live = g < a.G && m1 > ninf;
      const float wide = 0.5f * (bound.at(m1) + bound.at(both ? m2 : m1));
      const float dropped = wave_max(live && !kept ? score + wide : NEG_INF);
      const float least = -wave_max(live && kept ? wide - score : NEG_INF);
      close = dropped >= least;
    }
  }
  return kept;
}

// The plain way, in fp64: K rounds of a wave-wide arg-max over the logits in row (LDS). Lane k < K
// gets pick k, or -1. Few tokens come here: it is kept small, with rolled loops
// that compute a choice anew each time, so that its registers do not cost the common path waves.
__device__ __forceinline__ int choose_exact(ScoredArgs a, const float* row, float top) {
  const int lane = threadIdx.x & 63;
  const int g = lane >> a.lp, p = 1 << a.lp, sub = lane & (p - 1);
  const double ninf = (double)NEG_INF;
  const int items = g < a.G ? (a.S - sub + p - 1) >> a.lp : 0;
  double total = 0.0;
  if (!a.sigmoid) {
#pragma unroll 1
    for (int i = 0; i < items; ++i) total += exp((double)row[g * a.S + (i << a.lp) + sub] - (double)top);
    for (int d = 1; d < 64; d <<= 1) total += __shfl_xor(total, d, 64);
  }
  // want_s: the score where a choice is a bare logit
  auto choice = [&](int i, bool want_s) {
    const int e = g * a.S + (i << a.lp) + sub;
    const float l = row[e];
    const float b = a.bias ? a.bias[e] : 0.f;
    if (!(l > NEG_INF && b > NEG_INF)) return ninf;
    if (a.bias || want_s) return exact_score(a, l, top, total) + (double)b;
    return (double)l;
  };
  bool kept = true;
  if (a.G > 1) {
    double m1 = ninf, m2 = ninf;
#pragma unroll 1
    for (int i = 0; i < items; ++i) top_two(choice(i, a.group_top == 2), m1, m2);
    bool close = false;
    kept = group_kept<double>(a, lane, Bound{0.f, 0.f}, m1, m2, close);
  }
  uint32_t taken = 0;
  int my_e = -1;
#pragma unroll 1
  for (int k = 0; k < a.K; ++k) {
    double bv = ninf;
    int bi = -1;
    if (kept) {
#pragma unroll 1
      for (int i = 0; i < items; ++i) {
        if ((taken >> i) & 1) continue;
        const double c = choice(i, false);
        if (c > bv) {  // a lane's experts rise with i: ties keep the lower
          bv = c;
          bi = i;
        }
      }
    }
    const int mine = bi < 0 ? 0x7fffffff : g * a.S + (bi << a.lp) + sub;
    int be = mine;
#pragma unroll 1
    for (int d = 1; d < 64; d <<= 1) {
      const double ov = __shfl_xor(bv, d, 64);
      const int oe = __shfl_xor(be, d, 64);
      if (ov > bv || (ov == bv && oe < be)) {
        bv = ov;
        be = oe;
      }
    }
    if (be == 0x7fffffff) break;  // no expert left (the same in every lane)
    if (mine == be) taken |= 1u << bi;
    if (lane == k) my_e = be;
  }
  return my_e;
}

// For the scores that are returned: expf is good to about an ulp at any x, the hardware's reciprocal too.
__device__ __forceinline__ float sigmoid_f32(float l) { return __builtin_amdgcn_rcpf(1.0f + expf(-l)); }

// The pick's score as a share of the picks' sum (lanes without a pick: on = false). Where every
// sigmoid is so small that their sum may underflow, sigma(l) = exp(l) to the last bit and the
// share is a softmax.
__device__ __forceinline__ float pick_share(float l, bool on, bool sigmoid) {
  const float top = wave_max(on ? l : NEG_INF);
  const bool ratio = sigmoid && top > -60.0f;
  const float s = on ? (ratio ? sigmoid_f32(l) : expf(l - top)) : 0.f;
  const float sum = wave_sum(s);
  return on ? s * __builtin_amdgcn_rcpf(sum) : 0.f;
}

// One wave per token:
//  1. the choices in fp32, group limits;
//  2. a threshold: the K-th largest of the lanes' two largest, at most the K-th largest choice,
//     found by K rounds of a wave maximum of one value per lane (with one value a lane, a few kept
//     groups leave hardly more lanes than picks, and the bar falls too low for 64 candidates);
//  3. the few choices from the threshold up (less the error bound) go to LDS and come back one per lane: the
//     candidates, usually K to 2 K of them;
//  4. a candidate's rank is the number of candidates before it. Where two of them lie within the error bound,
//     each lane computes its own candidate's choice in fp64 and the ranks are taken from those.
// Where the scores of a kept and a dropped group lie within the bound, the group scores are taken in fp64
// too. A rank below K is a pick, written by the lane that holds it. Tokens with more than 64
// candidates (many equal choices) take the plain way in fp64.
template <int ITEMS>
__global__ __launch_bounds__(64 * RS_WAVES) RS_OCCUPANCY(ITEMS) void route_scored_kernel(ScoredArgs a, int* __restrict__ topk_idx,
                                                                     float* __restrict__ topk_w) {
  __shared__ float rows[RS_WAVES][RS_MAX_E];
  __shared__ float2 cand[RS_WAVES][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = blockIdx.x * RS_WAVES + wave;
  if (t >= a.T) return;
  const void* row = logit_row(a, t);
  const int g = lane >> a.lp, sub = lane & ((1 << a.lp) - 1);
  float* mine = rows[wave];
  float l[ITEMS], bias[ITEMS];
  int at[ITEMS];
  bool in[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int r = (i << a.lp) + sub;
    in[i] = g < a.G && r < a.S;
    at[i] = in[i] ? g * a.S + r : 0;  // lanes without an expert read expert 0: all loads go out together
  }
  if (a.bf16) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) l[i] = bf16_bits_to_f32(static_cast<const uint16_t*>(row)[at[i]]);
  } else {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) l[i] = static_cast<const float*>(row)[at[i]];
  }
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) bias[i] = a.bias[at[i]];
  } else {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) bias[i] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    l[i] = in[i] ? unmask(l[i], a.bf16) : NEG_INF;
    if (in[i]) mine[at[i]] = l[i];
  }
  float top = 0.f, total = 1.f;
  if (!a.sigmoid && (a.bias || a.G > 1 || !a.renorm)) {
    float m = NEG_INF;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) m = fmaxf(m, l[i]);
    m = wave_max(m);
    top = m > NEG_INF ? m : 0.f;
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) z += __expf(l[i] - top);
    z = wave_sum(z);
    total = z > 0.f ? z : 1.f;  // (nothing left to pick from)
  }
  const bool scores = a.bias || (a.G > 1 && a.group_top == 2);
  float s[ITEMS], c[ITEMS];
  choices<ITEMS>(a, scores, l, bias, top, total, s, c);
  // How far apart two choices are surely ordered alike in fp32 and exactly. exp errs by
  // (2 |x| + 2) 2^-24 of its value. Sigmoid: s (1 - s) |x| <= 0.23, so s errs by less than 1.5 *
  // 2^-22, and rounding c by 2^-24 |c|: below 2^-21 (1 + |c|). Softmax: the sum over up to 1024
  // experts adds at most 2^-18.2, relative to the largest score, 1 / total. The bound is four times
  // a choice's error e(c). Two choices c > d may be ordered the other way only if c - d <= e(c) + e(d), and e grows
  // with |c| so slowly that e(d) <= e(c) + 2^-19 (c - d): then c - d is below the bound at c (and at d). So each
  // choice counts with its own size: an expert switched off by a bias of -1e9 does not widen the others' bound.
  // Without scores the choices are the logits: exact.
  Bound bound{0.f, 0.f};
  if (scores) bound = a.sigmoid ? Bound{0x1p-19f, 0x1p-19f} : Bound{0x1p-16f / total, 0x1p-20f};
  bool plain = false;  // an infinite or huge choice
  if (a.G > 1) {
    const bool use_s = a.group_top == 2 && !a.bias;
    float m1 = NEG_INF, m2 = NEG_INF;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const float u = c[i] > NEG_INF ? (use_s ? s[i] : c[i]) : NEG_INF;
      m2 = __builtin_amdgcn_fmed3f(u, m1, m2);  // the second of the three, m1 >= m2
      m1 = u > m1 ? u : m1;
    }
    plain = a.bias && __ballot(m1 > HUGE_CHOICE) != 0;
    bool close = false;
    bool kept = group_kept<float>(a, lane, bound, m1, m2, close);
    if (close) {
      const double sum = a.sigmoid ? 1.0 : exact_total<ITEMS>(l, top);
      double d1 = (double)NEG_INF, d2 = d1;
      // a lane's two largest in fp64 are among those within the bound of its second in fp32
      const float low = m2 - 2.0f * bound.at(m2);
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const bool in = c[i] > NEG_INF && (use_s ? s[i] : c[i]) >= low;
        if (__ballot(in)) {
          const double d = exact_score(a, l[i], top, sum) + (double)bias[i];
          if (in) top_two(d, d1, d2);
        }
      }
      kept = group_kept<double>(a, lane, bound, d1, d2, close);
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
      if (!kept) c[i] = NEG_INF;
  }

  float best = NEG_INF, second = NEG_INF;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    second = __builtin_amdgcn_fmed3f(c[i], best, second);
    best = c[i] > best ? c[i] : best;
  }
  if (a.bias && a.G == 1) plain = __ballot(best > HUGE_CHOICE) != 0;
  const int none = order_key(NEG_INF);
  int own = order_key(best), next = order_key(second), key = none;
  for (int k = 0; k < a.K; ++k) {
    key = wave_max_key(own);
    const bool taken = own == key;
    own = taken ? next : own;
    next = taken ? none : next;
  }
  const float last = key_value(key);
  const float bar = a.bias ? last - bound.at(last) : last;
  int n = 0;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const bool is = c[i] >= bar && c[i] > NEG_INF;
    const uint64_t m = __ballot(is);
    if (m) {
      const int place = n + popc_below(m);
      if (is && place < 64) cand[wave][place] = make_float2(c[i], __int_as_float(at[i]));
      n += __popcll(m);
    }
  }
  plain = plain || n > 64;
  wave_sync();
  int my_e = -1, rank = 64;
  if (!plain) {
    float v = NEG_INF;
    int e = 0x7fffffff;
    if (lane < n) {
      const float2 x = cand[wave][lane];
      v = x.x;
      e = __float_as_int(x.y);
    }
    // the candidates before this one: larger choices, equal ones with a lower id
    // (+0 makes -0 and 0 equal)
    const uint64_t mine64 = (uint64_t)(uint32_t)(order_key(v + 0.0f) ^ 0x80000000) << 32 | (uint32_t)~e;
    const int hi = (int)(mine64 >> 32), lo = (int)mine64;
    rank = 0;
    for (int j = 0; j < n; ++j) {
      const uint64_t o =
          (uint64_t)(uint32_t)__builtin_amdgcn_readlane(hi, j) << 32 | (uint32_t)__builtin_amdgcn_readlane(lo, j);
      rank += o > mine64 ? 1 : 0;
    }
    if (a.bias) {
      // the neighbours in rank, through LDS
      if (lane < n) cand[wave][rank].x = v;
      wave_sync();
      const float here = lane < n ? cand[wave][lane].x : NEG_INF;
      const float after = lane + 1 < n ? cand[wave][lane + 1].x : NEG_INF;
      if (__ballot(lane + 1 < n && here - after <= bound.at(here))) {
        const float lv = lane < n ? mine[e] : 0.f;
        const double sum = a.sigmoid ? 1.0 : exact_total<ITEMS>(l, top);
        const double x = lane < n ? exact_score(a, lv, top, sum) + (double)a.bias[e] : (double)NEG_INF;
        rank = 0;
        for (int j = 0; j < n; ++j) {
          const double o = lane_value(x, j);
          const int oe = __builtin_amdgcn_readlane(e, j);
          rank += (o > x || (o == x && oe < e)) ? 1 : 0;
        }
      }
    }
    const bool on = lane < n && rank < a.K;
    my_e = on ? e : -1;
    // positions that no candidate takes: -1 from the lanes above the candidates
    if (!on) rank = lane >= n && lane < a.K ? lane : 64;
  } else {
    my_e = choose_exact(a, mine, top);
    rank = lane;
  }
  const bool on = my_e >= 0;
  const float lv = on ? mine[my_e] : NEG_INF;
  float w;
  if (a.renorm)
    w = pick_share(lv, on, a.sigmoid);
  else
    w = !on ? 0.f : a.sigmoid ? sigmoid_f32(lv) : expf(lv - top) / total;
  if (rank < a.K) {
    topk_idx[(size_t)t * a.K + rank] = my_e;
    topk_w[(size_t)t * a.K + rank] = w * a.scale;
  }
}

// The gradient of the logits for fixed picks, d = dL/dw:
//   renormalised, r = the pick's share: scale r (d - <d, r>), times (1 - s) for sigmoid scores;
//   sigmoid: scale d s (1 - s);   softmax: scale p ([picked] d - <d, p>) for every expert.
// One wave per token; the row is put together in LDS (picks added in their order, so the same
// expert twice gets the sum) and written once with wide stores. Only the dense softmax form
// reads all logits of the row, the others those of the picks.
template <int VEC>
__global__ __launch_bounds__(64 * RS_WAVES) void route_scored_bwd_kernel(ScoredArgs a,
                                                                         const int* __restrict__ topk_idx,
                                                                         const float* __restrict__ d_topk_w,
                                                                         void* __restrict__ d_logits) {
  __shared__ __attribute__((aligned(16))) float rows[RS_WAVES][RS_MAX_E];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = blockIdx.x * RS_WAVES + wave;
  if (t >= a.T) return;
  const void* row = logit_row(a, t);
  float* g = rows[wave];
  const int e = lane < a.K ? topk_idx[(size_t)t * a.K + lane] : -1;
  bool on = (unsigned)e < (unsigned)a.E;
  const float l = on ? read_logit(row, e, a.bf16) : NEG_INF;
  on = on && l > NEG_INF;
  const float d = on ? d_topk_w[(size_t)t * a.K + lane] : 0.f;
  const bool dense = !a.sigmoid && !a.renorm;
  float v = 0.f, dot = 0.f, top = 0.f, inv = 0.f;
  if (dense) {
    float m = NEG_INF;
    for (int i = lane; i < a.E; i += 64) {
      const float x = read_logit(row, i, a.bf16);
      g[i] = x;
      m = fmaxf(m, x);
    }
    m = wave_max(m);
    top = m > NEG_INF ? m : 0.f;
    float z = 0.f;
    for (int i = lane; i < a.E; i += 64) {
      const float x = expf(g[i] - top);
      g[i] = x;
      z += x;
    }
    z = wave_sum(z);
    inv = z > 0.f ? 1.0f / z : 0.f;
    const float ps = on ? expf(l - top) * inv : 0.f;
    v = d * ps * a.scale;
    dot = wave_sum(v);
    for (int i = lane; i < a.E; i += 64) g[i] = -dot * (g[i] * inv);
  } else {
    if (a.renorm) {
      const float r = pick_share(l, on, a.sigmoid);
      dot = wave_sum(d * r);
      v = a.scale * r * (d - dot);
      if (a.sigmoid && on) v *= sigmoid_f32(-l);
    } else if (on) {
      v = a.scale * d * sigmoid_f32(l) * sigmoid_f32(-l);
    }
    for (int i = lane; i < a.E; i += 64) g[i] = 0.f;
  }
  // an expert's picks add up in their order, in each lane that holds one of them
  float sum = 0.f;
  const int mine = on ? e : -1;
  for (int k = 0; k < a.K; ++k) {
    const float o = lane_value(v, k);
    sum += __builtin_amdgcn_readlane(mine, k) == e ? o : 0.f;
  }
  wave_sync();
  const float at = on ? g[e] : 0.f;
  wave_sync();
  if (on) g[e] = at + sum;
  wave_sync();
  if (a.bf16) {
    uint16_t* out = static_cast<uint16_t*>(d_logits) + (size_t)t * a.E;
    if constexpr (VEC == 4) {
      for (int i = lane * 4; i < a.E; i += 256) {
        const float4 x = *reinterpret_cast<const float4*>(g + i);
        *reinterpret_cast<uint2*>(out + i) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
      }
    } else {
      for (int i = lane; i < a.E; i += 64) out[i] = f32_to_bf16_bits(g[i]);
    }
  } else {
    float* out = static_cast<float*>(d_logits) + (size_t)t * a.E;
    if constexpr (VEC == 4) {
      for (int i = lane * 4; i < a.E; i += 256)
        *reinterpret_cast<float4*>(out + i) = *reinterpret_cast<const float4*>(g + i);
    } else {
      for (int i = lane; i < a.E; i += 64) out[i] = g[i];
    }
  }
}

ScoredArgs scored_args(const moe_route_desc_t& d, const void* logits, moe_dtype_t lt, const float* bias) {
  ScoredArgs a{};
  a.logits = logits;
  a.bias = bias;
  a.T = d.T;
  a.E = d.E;
  a.K = d.K;
  a.bf16 = lt == MOE_BF16;
  a.sigmoid = d.score == MOE_SCORE_SIGMOID;
  a.renorm = d.renorm != 0;
  a.G = d.topk_groups < d.groups ? d.groups : 1;
  a.S = d.E / a.G;
  int slots = 1;
  while (slots < a.G) slots <<= 1;
  a.lp = 0;
  while ((slots << (a.lp + 1)) <= 64) ++a.lp;
  a.topk_groups = d.topk_groups;
  a.group_top = d.group_top;
  a.scale = d.scale;
  return a;
}

}  // namespace

moe_status_t launch_route_scored(const moe_route_desc_t& d, const void* logits, moe_dtype_t lt, const float* bias,
                                 int* topk_idx, float* topk_w, hipStream_t s) {
  if (d.T == 0) return MOE_OK;
  const ScoredArgs a = scored_args(d, logits, lt, bias);
  // A lane holds `items` experts; the kernel is built for the powers of two and for 6, and an empty slot costs what
  // a full one does. 8192 tokens, 8 picks, bias, sigmoid, us, a form against the next larger one (without groups; 8 groups):
  //   64 experts   1 /  2:  6.3 /  6.7;   8.4 /  9.0      384 experts   6 /  8:  8.6 /  9.5;  11.4 / 12.6
  //   128          2 /  4:  7.1 /  7.9;   9.1 / 10.2      512           8 / 16:  9.6 / 14.2;  12.6 / 18.0
  //   256          4 /  6:  8.0 /  8.6;  11.0 / 11.9      1024         16 / 32: 14.4 / 30.4;  21.6 / 41.0
  // From 16 on the logits no longer leave the registers for eight waves a SIMD. 32 serves groups that fill their
  // lanes badly (33 groups of 31: one lane each).
  const int items = (a.S + (1 << a.lp) - 1) >> a.lp;
  const dim3 grid((a.T + RS_WAVES - 1) / RS_WAVES), block(64 * RS_WAVES);
  if (items <= 1)
    route_scored_kernel<1><<<grid, block, 0, s>>>(a, topk_idx, topk_w);
  else if (items <= 2)
    route_scored_kernel<2><<<grid, block, 0, s>>>(a, topk_idx, topk_w);
  else if (items <= 4)
    route_scored_kernel<4><<<grid, block, 0, s>>>(a, topk_idx, topk_w);
  else if (items <= 6)
    route_scored_kernel<6><<<grid, block, 0, s>>>(a, topk_idx, topk_w);
  else if (items <= 8)
    route_scored_kernel<8><<<grid, block, 0, s>>>(a, topk_idx, topk_w);
  else if (items <= 16)
    route_scored_kernel<16><<<grid, block, 0, s>>>(a, topk_idx, topk_w);
  else
    route_scored_kernel<32><<<grid, block, 0, s>>>(a, topk_idx, topk_w);
  return launch_status();
}

moe_status_t launch_route_scored_bwd(const moe_route_desc_t& d, const void* logits, moe_dtype_t lt,
                                     const int* topk_idx, const float* d_topk_w, void* d_logits, hipStream_t s) {
  if (d.T == 0) return MOE_OK;
  const ScoredArgs a = scored_args(d, logits, lt, nullptr);
  const dim3 grid((a.T + RS_WAVES - 1) / RS_WAVES), block(64 * RS_WAVES);
  const size_t vec_bytes = lt == MOE_BF16 ? 8 : 16;
  if (a.E % 4 == 0 && reinterpret_cast<uintptr_t>(d_logits) % vec_bytes == 0)
    route_scored_bwd_kernel<4><<<grid, block, 0, s>>>(a, topk_idx, d_topk_w, d_logits);
  else
    route_scored_bwd_kernel<1><<<grid, block, 0, s>>>(a, topk_idx, d_topk_w, d_logits);
  return launch_status();
}

}  // namespace moe
