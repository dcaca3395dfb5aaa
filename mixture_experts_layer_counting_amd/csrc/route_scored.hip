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
// neighbouring picks (or two group scores) lie closer than twice that error does the wave redo
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

struct ScoredArgs {
  const void* logits;
  const float* bias;
  int T, E, K;
  int bf16, sigmoid, renorm;
  int G, S, lp;  // groups that limit the choice (1: none), experts per group, log2(lanes per group)
  int topk_groups, group_top;
  float scale;
};

// The largest x over the 64 lanes, in every lane.
__device__ __forceinline__ float wave_max(float x) {
  x = fmaxf(x, __int_as_float(dpp_mov<DPP_XOR1>(__float_as_int(x))));
  x = fmaxf(x, __int_as_float(dpp_mov<DPP_XOR2>(__float_as_int(x))));
  x = fmaxf(x, __int_as_float(dpp_mov<DPP_HALF_MIRROR>(__float_as_int(x))));
  x = fmaxf(x, __int_as_float(dpp_mov<DPP_MIRROR>(__float_as_int(x))));
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// LDS written by some lanes of this wave is read by others after this.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Logit `e` of a row, masked (NaN, -inf, the type's lowest value) as -inf, +inf as the largest
// fp32.
__device__ __forceinline__ float read_logit(const void* row, int e, int bf16) {
  const float x = bf16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(row)[e]) : static_cast<const float*>(row)[e];
  const float lowest = bf16 ? -3.38953139e38f : -3.40282347e38f;
  return x > lowest ? fminf(x, 3.40282347e38f) : NEG_INF;
}

__device__ __forceinline__ const void* logit_row(const ScoredArgs& a, int t) {
  return static_cast<const char*>(a.logits) + (size_t)t * a.E * (a.bf16 ? 2 : 4);
}

__device__ __forceinline__ double exp_f(double x) { return exp(x); }
__device__ __forceinline__ float exp_f(float x) { return __expf(x); }

// The picks of one token in arithmetic F (float: with `close` set where the order of two
// choices is within their error; double: final). Lane k < K gets the expert of pick k, -1 where
// no expert was left. l: this lane's logits.
template <typename F, int ITEMS>
__device__ __forceinline__ int choose(const ScoredArgs& a, const float (&l)[ITEMS], const float (&bias)[ITEMS],
                                      float top, F total, int lane, bool& close) {
  constexpr bool FAST = sizeof(F) == 4;
  const F ninf = (F)NEG_INF;
  const int g = lane >> a.lp, p = 1 << a.lp, sub = lane & (p - 1);
  const bool sums = a.G > 1 && a.group_top == 2;
  const bool scores = a.bias || sums;
  F s[ITEMS], c[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    s[i] = (F)0;
    if (scores) {
      if (a.sigmoid)
        s[i] = (F)1 / ((F)1 + exp_f(-(F)l[i]));
      else
        s[i] = exp_f((F)l[i] - (F)top) / total;
    }
    c[i] = a.bias ? s[i] + (F)bias[i] : (F)l[i];
    if (!(l[i] > NEG_INF && bias[i] > NEG_INF)) c[i] = ninf;
  }
  // How far apart two choices are surely ordered alike in fp32 and exactly. exp errs by
  // (2 |x| + 2) 2^-24 of its value. Sigmoid: s (1 - s) |x| <= 0.23, so s errs by less than 1.5 *
  // 2^-22, and rounding c by 2^-24 |c|; twice that is below 2^-20 (1 + |c|). Softmax: the sum
  // over up to 1024 experts adds at most 2^-18.2, relative to the largest score. Both get a
  // factor of two on top.
  F tol = 0;
  if (FAST && scores) {
    float big = 0.f;
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
        if (c[i] > ninf) big = fmaxf(big, __builtin_fabsf((float)c[i]));
      big = wave_max(big);
    }
    tol = a.sigmoid ? (F)0x1p-19 * ((F)1 + big) : (F)0x1p-16 / total + (F)0x1p-20 * big;
  }
  bool out = false;  // this lane's group is limited away
  if (a.G > 1) {
    F m1 = ninf, m2 = ninf;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const F u = c[i] > ninf ? (sums && !a.bias ? s[i] : c[i]) : ninf;
      m2 = u > m1 ? m1 : (u > m2 ? u : m2);
      m1 = u > m1 ? u : m1;
    }
    for (int d = 1; d < p; d <<= 1) {
      const F o1 = __shfl_xor(m1, d, 64), o2 = __shfl_xor(m2, d, 64);
      const F lo = o1 > m1 ? m1 : o1;
      const F hi2 = o2 > m2 ? o2 : m2;
      m2 = lo > hi2 ? lo : hi2;
      m1 = o1 > m1 ? o1 : m1;
    }
    F score = m1;
    if (sums && m2 > ninf) score = m1 + m2;
    int rank = 0;
    for (int j = 0; j < a.G; ++j) {
      const F o = __shfl(score, j << a.lp, 64);
      rank += (o > score || (o == score && j < g)) ? 1 : 0;
      if (FAST && scores && j != g && o > ninf && score > ninf && o - score <= 2 * tol && score - o <= 2 * tol)
        close = true;
    }
    out = g >= a.G || rank >= a.topk_groups;
  }
  uint32_t taken = 0;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i)
    if (out || !(c[i] > ninf)) taken |= 1u << i;
  int my_e = -1;
  F last = ninf;
  // with a bias, in fp32 one round more: the best expert not picked, against the last pick
  const bool near = FAST && a.bias;
  const int rounds = near ? a.K + 1 : a.K;
  for (int k = 0; k < rounds; ++k) {
    F bv = ninf;
    int bi = -1;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
      if (!((taken >> i) & 1) && c[i] > bv) {  // a lane's experts rise with i: ties keep the lower
        bv = c[i];
        bi = i;
      }
    const int mine = bi < 0 ? 0x7fffffff : g * a.S + (bi << a.lp) + sub;
    int be = mine;
    if constexpr (FAST) {
      wave_best(bv, be);
    } else {
      for (int d = 1; d < 64; d <<= 1) {
        const F ov = __shfl_xor(bv, d, 64);
        const int oe = __shfl_xor(be, d, 64);
        if (ov > bv || (ov == bv && oe < be)) {
          bv = ov;
          be = oe;
        }
      }
    }
    if (be == 0x7fffffff) break;  // no expert left (the same in every lane)
    if (mine == be) taken |= 1u << bi;
    if (near && k > 0 && last - bv <= tol) close = true;
    last = bv;
    if (lane == k && k < a.K) my_e = be;
  }
  return my_e;
}

// For the scores that are returned: expf is good to about an ulp at any x.
__device__ __forceinline__ float sigmoid_f32(float l) { return 1.0f / (1.0f + expf(-l)); }

// The pick's score as a share of the picks' sum (lanes without a pick: on = false). Where every
// sigmoid is so small that their sum may underflow, sigma(l) = exp(l) to the last bit and the
// share is a softmax.
__device__ __forceinline__ float pick_share(float l, bool on, bool sigmoid) {
  const float top = wave_max(on ? l : NEG_INF);
  const bool ratio = sigmoid && top > -60.0f;
  const float s = on ? (ratio ? sigmoid_f32(l) : expf(l - top)) : 0.f;
  const float sum = wave_sum(s);
  return on ? s / sum : 0.f;
}

template <int ITEMS>
__global__ __launch_bounds__(64 * RS_WAVES) void route_scored_kernel(ScoredArgs a, int* __restrict__ topk_idx,
                                                                     float* __restrict__ topk_w) {
  __shared__ float rows[RS_WAVES][RS_MAX_E];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = blockIdx.x * RS_WAVES + wave;
  if (t >= a.T) return;
  const void* row = logit_row(a, t);
  const int g = lane >> a.lp, p = 1 << a.lp, sub = lane & (p - 1);
  float* mine = rows[wave];
  float l[ITEMS], bias[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int r = (i << a.lp) + sub;
    const bool in = g < a.G && r < a.S;
    const int e = in ? g * a.S + r : 0;
    bias[i] = a.bias ? a.bias[e] : 0.f;
    l[i] = in ? read_logit(row, e, a.bf16) : NEG_INF;
    if (in) mine[e] = l[i];
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
    total = wave_sum(z);
  }
  bool close = false;
  int my_e = choose<float, ITEMS>(a, l, bias, top, total, lane, close);
  if (__ballot(close)) {
    double sum = 1.0;
    if (!a.sigmoid) {
      sum = 0.0;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) sum += exp((double)l[i] - (double)top);
      for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d, 64);
    }
    my_e = choose<double, ITEMS>(a, l, bias, top, sum, lane, close);
  }
  wave_sync();
  const bool on = my_e >= 0;
  const float lp = on ? mine[my_e] : NEG_INF;
  float w;
  if (a.renorm) {
    w = pick_share(lp, on, a.sigmoid);
  } else {
    w = !on ? 0.f : a.sigmoid ? sigmoid_f32(lp) : expf(lp - top) / total;
  }
  if (lane < a.K) {
    topk_idx[(size_t)t * a.K + lane] = my_e;
    topk_w[(size_t)t * a.K + lane] = w * a.scale;
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
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
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
  // picks in their order: the same expert twice adds up
  for (int k = 0; k < a.K; ++k) {
    wave_sync();
    if (lane == k && on) g[e] += v;
  }
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
