// MXFP4 quantisation of activations and of stacked weights, and the way back ("Mixture of
// Kittens", Step 8: weights pre-quantised once, activations quantised on the way into the
// GEMMs; the format's arithmetic is in mxfp4.h).
//
//  rows:     x [R, C] -> q [R, C/2], sf [R, C/32]. A block of 32 elements is four lanes of eight
//            (one 16-byte load of bf16, two of fp32); its largest magnitude goes round the quad by two
//            DPP steps.
//  weights:  w [E, K, N] (reduction first) -> q [E, N, K/2] (or the paired layout), sf [E, K/32,
//            N]. The codes of a column run along k, its source values across rows, so the
//            kernel transposes. A lane takes COLS neighbouring columns (16 bytes) of the 32 rows
//            of one block: the block's maximum and codes need no other lane. A wave is 8 column
//            groups x 8 k-blocks: each load instruction reads eight whole 128-byte lines, each
//            store writes eight 128-byte runs of codes, without a pass through LDS.
// All four are bound by HBM (a large copy reaches 4.9 TB/s here): rows 8192 x 7168 bf16 29 us, 5.1 TB/s, and
// back 23 us; weights 52 x 7168 x 2048 bf16 385 us, 5.0 TB/s, and back 335 us; 64 x 2048 x 1024 fp32 136 us, 4.5
// TB/s, and back to bf16 66 us. Rows that do not end on whole lines: see the kernels.
#include "mxfp4.h"
#include "tile_sched.h"

namespace moe {

namespace {

// Unaligned 16- and 8-byte accesses: rows of odd length start at any element.
struct raw16 {
  uint32_t u[4];
};
__device__ __forceinline__ raw16 load16(const void* p) {
  raw16 r;
  __builtin_memcpy(&r, p, 16);
  return r;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

template <int CTRL>
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp((int)m, (int)m, CTRL, 0xF, 0xF, false);
  return o > m ? o : m;
}

template <typename XT>
__device__ __forceinline__ void load8(const XT* p, float (&v)[8]) {
  if constexpr (sizeof(XT) == 2) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  } else {
    const float4 a = reinterpret_cast<const float4*>(p)[0];
    const float4 b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

// n8 = R * C / 8 groups of eight elements. Whole quads are live or not: n8 is a multiple of 4.
template <typename XT>
__global__ __launch_bounds__(256) void quant_rows_kernel(const XT* __restrict__ x, size_t n8,
                                                         uint8_t* __restrict__ q, uint8_t* __restrict__ sf) {
  const size_t g = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (g >= n8) return;
  float v[8];
  load8(x + g * 8, v);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
  m = quad_max<0xB1>(m);  // lane ^ 1
  m = quad_max<0x4E>(m);  // lane ^ 2
  const uint32_t b = mx_scale_byte(m);
  reinterpret_cast<uint32_t*>(q)[g] = mx_pack8(v, b);
  if ((threadIdx.x & 3) == 0) sf[g >> 2] = (uint8_t)b;
}

__device__ __forceinline__ void unpack8(uint32_t w, float x, float (&v)[8]) {
  mx_unpack2<0>(w, x, v[0], v[1]);
  mx_unpack2<1>(w, x, v[2], v[3]);
  mx_unpack2<2>(w, x, v[4], v[5]);
  mx_unpack2<3>(w, x, v[6], v[7]);
}

template <typename XT>
__global__ __launch_bounds__(256) void dequant_rows_kernel(const uint8_t* __restrict__ q,
                                                           const uint8_t* __restrict__ sf, size_t n8,
                                                           XT* __restrict__ out) {
  const size_t g = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (g >= n8) return;
  float v[8];
  unpack8(reinterpret_cast<const uint32_t*>(q)[g], mx_scale_f32(sf[g >> 2]), v);
  if constexpr (sizeof(XT) == 2) {
    *reinterpret_cast<uint4*>(out + g * 8) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                        pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  } else {
    reinterpret_cast<float4*>(out + g * 8)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(out + g * 8)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// Byte offset of code byte `kb` (k / 2) of column n inside one expert's codes.
template <bool PAIRED>
__device__ __forceinline__ size_t code_at(int n, int kb, int K) {
  if constexpr (PAIRED)  // [N/2][K/128][2][64]
    return (size_t)(n >> 1) * K + (size_t)(kb >> 6) * 128 + (n & 1) * 64 + (kb & 63);
  return (size_t)n * (K / 2) + kb;
}

// Block x of a matrix's nx * ny blocks -> column block bx and k block by, in row order of the k blocks. With
// `near`, column neighbours run on one XCD: where rows do not end on whole lines, two blocks share the
// line at their border, and its parts meet in one L2.
__device__ __forceinline__ void weight_block(int x, int blocks, int nx, bool near, int& bx, int& by) {
  const int even = blocks & ~7;
  const int at = near && x < even ? xcd_slot(x, even) : x;
  by = at / nx;
  bx = at - by * nx;
}

template <typename XT>
__host__ __device__ __forceinline__ bool whole_lines(int N) {
  return (size_t)N * sizeof(XT) % 128 == 0;
}

// Column groups of a matrix whose last group overlaps the one before where COLS does not divide N (the shared
// columns are computed and written twice, alike). COLS = 1: fewer columns than a group.
template <typename XT, int COLS, bool PAIRED>
__global__ __launch_bounds__(256) void quant_weights_kernel(const XT* __restrict__ w, int K, int N, int nx,
                                                            uint8_t* __restrict__ q, uint8_t* __restrict__ sf) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int bx, by;  // in dispatch order whole lines are 2 % faster: 26 x 7168 x 2048 bf16 175 us, near 178
  weight_block(blockIdx.x, gridDim.x, nx, !whole_lines<XT>(N), bx, by);
  const int cg = (bx * 4 + wave) * 8 + (lane & 7);
  const int kb = by * 8 + (lane >> 3);
  const int e = blockIdx.z;
  if (cg * COLS >= N || kb * 32 >= K) return;
  const int n0 = min(cg * COLS, N - COLS);
  const XT* src = w + ((size_t)e * K + (size_t)kb * 32) * N + n0;
  uint8_t* qe = q + (size_t)e * N * (K / 2);
  uint32_t byte[COLS];
  if constexpr (COLS == 1) {
    float v[32];
    uint32_t m = 0;
#pragma unroll
    for (int r = 0; r < 32; ++r) {
      if constexpr (sizeof(XT) == 2)
        v[r] = bf16_bits_to_f32(src[(size_t)r * N]);
      else
        v[r] = src[(size_t)r * N];
      m = max(m, abs_bits(v[r]));
    }
    byte[0] = mx_scale_byte(m);
    *reinterpret_cast<uint4*>(qe + code_at<PAIRED>(n0, kb * 16, K)) =
        make_uint4(mx_pack8(v, byte[0]), mx_pack8(v + 8, byte[0]), mx_pack8(v + 16, byte[0]), mx_pack8(v + 24, byte[0]));
  } else {
    raw16 d[32];
#pragma unroll
    for (int r = 0; r < 32; ++r) d[r] = load16(src + (size_t)r * N);
    auto at = [&](int r, int c) {
      if constexpr (sizeof(XT) == 2)
        return __uint_as_float((c & 1) ? d[r].u[c >> 1] & 0xffff0000u : d[r].u[c >> 1] << 16);
      else
        return __uint_as_float(d[r].u[c]);
    };
#pragma unroll
    for (int c = 0; c < COLS; ++c) {
      uint32_t m = 0;
#pragma unroll
      for (int r = 0; r < 32; ++r) m = max(m, abs_bits(at(r, c)));
      byte[c] = mx_scale_byte(m);
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = at(8 * j + i, c);
        o[j] = mx_pack8(v, byte[c]);
      }
      *reinterpret_cast<uint4*>(qe + code_at<PAIRED>(n0 + c, kb * 16, K)) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
  uint8_t pack[COLS];
#pragma unroll
  for (int c = 0; c < COLS; ++c) pack[c] = (uint8_t)byte[c];
  __builtin_memcpy(sf + ((size_t)e * (K / 32) + kb) * N + n0, pack, COLS);
}

// The way back: codes read in 16-byte runs per column, rows written in runs of COLS values. A wave is CW column
// groups x 64 / CW k-blocks: the wider, the fewer lines of the output it shares with a neighbour.
// 26 x 7168 x N, us, CW 8 in dispatch order / 8, 16, 32 with near blocks:
//   bf16  N 2048: 196 / 193, 185, 192   N 2046: 295 / 269, 230, 220   N 1001: 142 / 126, 112, 110
//   fp32  N 2048: 321 / 328, 332, 333   N 2046: 589 / 519, 429, 387   N 1001: 282 / 250, 211, 190
template <typename XT, int COLS, bool PAIRED, int CW>
__global__ __launch_bounds__(256) void dequant_weights_kernel(const uint8_t* __restrict__ q,
                                                              const uint8_t* __restrict__ sf, int K, int N, int nx,
                                                              XT* __restrict__ out) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int bx, by;
  weight_block(blockIdx.x, gridDim.x, nx, true, bx, by);
  const int cg = (bx * 4 + wave) * CW + lane % CW;
  const int kb = by * (64 / CW) + lane / CW;
  const int e = blockIdx.z;
  if (cg * COLS >= N || kb * 32 >= K) return;
  const int n0 = min(cg * COLS, N - COLS);
  const uint8_t* qe = q + (size_t)e * N * (K / 2);
  uint8_t byte[COLS];
  __builtin_memcpy(byte, sf + ((size_t)e * (K / 32) + kb) * N + n0, COLS);
  uint4 c4[COLS];
#pragma unroll
  for (int c = 0; c < COLS; ++c) c4[c] = *reinterpret_cast<const uint4*>(qe + code_at<PAIRED>(n0 + c, kb * 16, K));
  XT* dst = out + ((size_t)e * K + (size_t)kb * 32) * N + n0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float v[COLS][8];
#pragma unroll
    for (int c = 0; c < COLS; ++c) {
      const uint32_t word = j == 0 ? c4[c].x : j == 1 ? c4[c].y : j == 2 ? c4[c].z : c4[c].w;
      unpack8(word, mx_scale_f32(byte[c]), v[c]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      XT* row = dst + (size_t)(8 * j + i) * N;
      if constexpr (COLS == 1) {
        if constexpr (sizeof(XT) == 2)
          *row = f32_to_bf16_bits(v[0][i]);
        else
          *row = v[0][i];
      } else {
        uint32_t o[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if constexpr (sizeof(XT) == 2)
            o[c] = pack_bf16x2(v[2 * c][i], v[2 * c + 1][i]);
          else
            o[c] = __float_as_uint(v[c][i]);
        }
        __builtin_memcpy(row, o, 16);
      }
    }
  }
}

// Blocks of CW column groups per wave x 64 / CW k-blocks: nx of them along the columns, the matrix's in x.
template <int COLS, int CW>
dim3 weight_grid(int E, int K, int N, int& nx) {
  const int groups = (N + COLS - 1) / COLS;
  nx = (groups + 4 * CW - 1) / (4 * CW);
  const unsigned ny = (K / 32 + 64 / CW - 1) / (64 / CW);
  return dim3((unsigned)nx * ny, 1, E);
}

template <typename XT, bool PAIRED, int COLS>
void quant_weights_cols(const XT* w, int E, int K, int N, uint8_t* q, uint8_t* sf, hipStream_t s) {
  int nx;
  const dim3 grid = weight_grid<COLS, 8>(E, K, N, nx);
  quant_weights_kernel<XT, COLS, PAIRED><<<grid, 256, 0, s>>>(w, K, N, nx, q, sf);
}

template <typename XT, bool PAIRED>
void quant_weights(const void* w, int E, int K, int N, uint8_t* q, uint8_t* sf, hipStream_t s) {
  constexpr int COLS = 16 / sizeof(XT);
  const XT* src = static_cast<const XT*>(w);
  if (N >= COLS)
    quant_weights_cols<XT, PAIRED, COLS>(src, E, K, N, q, sf, s);
  else
    quant_weights_cols<XT, PAIRED, 1>(src, E, K, N, q, sf, s);
}

template <typename XT, bool PAIRED, int COLS, int CW>
void dequant_weights_cols(const uint8_t* q, const uint8_t* sf, int E, int K, int N, XT* out, hipStream_t s) {
  int nx;
  const dim3 grid = weight_grid<COLS, CW>(E, K, N, nx);
  dequant_weights_kernel<XT, COLS, PAIRED, CW><<<grid, 256, 0, s>>>(q, sf, K, N, nx, out);
}

template <typename XT, bool PAIRED>
void dequant_weights(const uint8_t* q, const uint8_t* sf, int E, int K, int N, void* out, hipStream_t s) {
  constexpr int COLS = 16 / sizeof(XT);
  XT* dst = static_cast<XT*>(out);
  if (N < COLS)
    dequant_weights_cols<XT, PAIRED, 1, 8>(q, sf, E, K, N, dst, s);
  else if (whole_lines<XT>(N))
    dequant_weights_cols<XT, PAIRED, COLS, 16>(q, sf, E, K, N, dst, s);
  else
    dequant_weights_cols<XT, PAIRED, COLS, 32>(q, sf, E, K, N, dst, s);
}

}  // namespace

moe_status_t launch_quantize_mxfp4(const void* x, moe_dtype_t xt, int R, int C, uint8_t* q, uint8_t* sf,
                                   hipStream_t s) {
  const size_t n8 = (size_t)R * C / 8;
  if (n8 == 0) return MOE_OK;
  const unsigned grid = (unsigned)((n8 + 255) / 256);
  if (xt == MOE_BF16)
    quant_rows_kernel<uint16_t><<<grid, 256, 0, s>>>(static_cast<const uint16_t*>(x), n8, q, sf);
  else
    quant_rows_kernel<float><<<grid, 256, 0, s>>>(static_cast<const float*>(x), n8, q, sf);
  return launch_status();
}

moe_status_t launch_dequantize_mxfp4(const uint8_t* q, const uint8_t* sf, int R, int C, void* out,
                                     moe_dtype_t ot, hipStream_t s) {
  const size_t n8 = (size_t)R * C / 8;
  if (n8 == 0) return MOE_OK;
  const unsigned grid = (unsigned)((n8 + 255) / 256);
  if (ot == MOE_BF16)
    dequant_rows_kernel<uint16_t><<<grid, 256, 0, s>>>(q, sf, n8, static_cast<uint16_t*>(out));
  else
    dequant_rows_kernel<float><<<grid, 256, 0, s>>>(q, sf, n8, static_cast<float*>(out));
  return launch_status();
}

moe_status_t launch_quantize_mxfp4_weights(const void* w, moe_dtype_t wt, int E, int K, int N, bool paired,
                                           uint8_t* q, uint8_t* sf, hipStream_t s) {
  if ((size_t)E * K * N == 0) return MOE_OK;
  if (wt == MOE_BF16)
    paired ? quant_weights<uint16_t, true>(w, E, K, N, q, sf, s) : quant_weights<uint16_t, false>(w, E, K, N, q, sf, s);
  else
    paired ? quant_weights<float, true>(w, E, K, N, q, sf, s) : quant_weights<float, false>(w, E, K, N, q, sf, s);
  return launch_status();
}

moe_status_t launch_dequantize_mxfp4_weights(const uint8_t* q, const uint8_t* sf, bool paired, int E, int K, int N,
                                             void* out, moe_dtype_t ot, hipStream_t s) {
  if ((size_t)E * K * N == 0) return MOE_OK;
  if (ot == MOE_BF16)
    paired ? dequant_weights<uint16_t, true>(q, sf, E, K, N, out, s) : dequant_weights<uint16_t, false>(q, sf, E, K, N, out, s);
  else
    paired ? dequant_weights<float, true>(q, sf, E, K, N, out, s) : dequant_weights<float, false>(q, sf, E, K, N, out, s);
  return launch_status();
}

}  // namespace moe
