// INT8 quantisation of activations (a scale per row) and of stacked weights (a scale per output
// column), and the way back. The arithmetic is in int8.h.
//
//  rows:     x [R, C] -> q [R, C], sf [R]. A row belongs to 64 or 256 threads; each holds its
//            values in registers between the maximum and the codes, so that x is read once (rows of
//            more than 8192 values are read again, from the cache).
//  weights:  w [E, K, N] (reduction first) -> q [E, N, K], sf [E, N]. The maximum of a column needs
//            all of K before the first code: one kernel finds the scales, a second one reads the
//            values again, turns 64 x 64 tiles through LDS and writes runs of codes along k.
// All are bound by HBM. Any C, K and N: rows may start at any element, whole 16-byte words are
// loaded where they lie inside the row and single elements at its end.
#include "int8.h"
#include "tile_sched.h"

namespace moe {

namespace {

// Eight values at p, of which the first n are inside the row (the others read as zero).
template <typename XT>
__device__ __forceinline__ void load8(const XT* p, int n, float (&v)[8]) {
  if (n >= 8) {
    if constexpr (sizeof(XT) == 2) {
      uint32_t u[4];
      __builtin_memcpy(u, p, 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
    } else {
      __builtin_memcpy(v, p, 16);
      __builtin_memcpy(v + 4, p + 4, 16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = 0.f;
      if (i < n) {
        if constexpr (sizeof(XT) == 2) v[i] = bf16_bits_to_f32(p[i]);
        else v[i] = p[i];
      }
    }
  }
}

template <typename XT>
__device__ __forceinline__ void store8(XT* p, int n, const float (&v)[8]) {
  if (n >= 8) {
    if constexpr (sizeof(XT) == 2) {
      const uint32_t u[4] = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                             pack_bf16x2(v[6], v[7])};
      __builtin_memcpy(p, u, 16);
    } else {
      __builtin_memcpy(p, v, 16);
      __builtin_memcpy(p + 4, v + 4, 16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) {
        if constexpr (sizeof(XT) == 2) p[i] = f32_to_bf16_bits(v[i]);
        else p[i] = v[i];
      }
  }
}

__device__ __forceinline__ void store_codes(int8_t* q, int n, const float (&v)[8], float s, float inv) {
  float c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = int8_code(v[i], s, inv);
  const uint32_t u[2] = {pack_i8x4(c[0], c[1], c[2], c[3]), pack_i8x4(c[4], c[5], c[6], c[7])};
  if (n >= 8) {
    __builtin_memcpy(q, u, 8);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) q[i] = (int8_t)(u[i >> 2] >> (8 * (i & 3)));
  }
}

// TPR threads per row, a block of 256; CH: groups of eight values that a thread keeps.
template <typename XT, int TPR, int CH>
__global__ __launch_bounds__(256) void quant_rows_i8_kernel(const XT* __restrict__ x, int R, int C,
                                                            int8_t* __restrict__ q, float* __restrict__ sf) {
  __shared__ uint32_t part[2][4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = threadIdx.x % TPR;
  constexpr int RPB = 256 / TPR;
  int turn = 0;
  for (int64_t r = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; r < R; r += (int64_t)gridDim.x * RPB, turn ^= 1) {
    const XT* xr = x + (size_t)r * C;
    float v[CH][8];
    uint32_t m = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int at = (c * TPR + t) * 8;
      load8(xr + (at < C ? at : 0), C - at, v[c]);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[c][i]));
    for (int64_t at = (int64_t)(CH * TPR + t) * 8; at < C; at += TPR * 8) {  // rows longer than the registers
      float u[8];
      load8(xr + at, (int)min((int64_t)8, C - at), u);
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, abs_bits(u[i]));
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 64));
    if constexpr (TPR == 256) {
      if (lane == 0) part[turn][wave] = m;
      __syncthreads();  // the other half is written next: its readers all passed this barrier
      m = max(max(part[turn][0], part[turn][1]), max(part[turn][2], part[turn][3]));
    }
    float s = int8_scale(m);
    if (t == 0) sf[r] = s;
    int8_t* qr = q + (size_t)r * C;
    const bool bad = m >= 0x7f800000u;
    const float inv = bad ? 0.f : __fdiv_rn(1.0f, s);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int at = (c * TPR + t) * 8;
      if (bad) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] = 0.f;
      }
      if (at < C) store_codes(qr + at, C - at, v[c], s, inv);
    }
    for (int64_t at = (int64_t)(CH * TPR + t) * 8; at < C; at += TPR * 8) {
      const int n = (int)min((int64_t)8, C - at);
      float u[8];
      load8(xr + at, n, u);
      if (bad) {
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = 0.f;
      }
      store_codes(qr + at, n, u, s, inv);
    }
  }
}

template <typename XT, int TPR>
__global__ __launch_bounds__(256) void dequant_rows_i8_kernel(const int8_t* __restrict__ q,
                                                              const float* __restrict__ sf, int R, int C,
                                                              XT* __restrict__ out) {
  constexpr int RPB = 256 / TPR;
  for (int64_t r = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; r < R; r += (int64_t)gridDim.x * RPB) {
    const float s = sf[r];
    const int8_t* qr = q + (size_t)r * C;
    for (int64_t at = (threadIdx.x % TPR) * 8; at < C; at += TPR * 8) {
      const int n = (int)min((int64_t)8, C - at);
      uint32_t u[2] = {0, 0};
      if (n >= 8) {
        __builtin_memcpy(u, qr + at, 8);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < n) u[i >> 2] |= (uint32_t)(uint8_t)qr[at + i] << (8 * (i & 3));
      }
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i8_at(u[i >> 2], i & 3) * s;
      store8(out + (size_t)r * C + at, n, v);
    }
  }
}

// Scales of CW = 8 LW neighbouring columns: LW lanes of eight columns side by side, 1024 / LW rows at a time.
template <typename XT, int LW>
__global__ __launch_bounds__(1024) void weight_scales_i8_kernel(const XT* __restrict__ w, int K, int N, int ncb,
                                                                int64_t blocks, float* __restrict__ sf) {
  constexpr int CW = 8 * LW, ROWS = 1024 / LW;
  __shared__ uint32_t best[16][CW];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lc = threadIdx.x % LW, lr = threadIdx.x / LW;
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
    const int64_t e = b / ncb;
    const int n0 = (int)(b - e * ncb) * CW;
    const int n = N - n0 - lc * 8;
    const XT* p = w + (size_t)e * K * N + n0 + (n > 0 ? lc * 8 : 0);
    uint32_t m[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (n > 0) {
#pragma unroll 4
      for (int k = lr; k < K; k += ROWS) {
        float v[8];
        load8(p + (size_t)k * N, n, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] = max(m[i], abs_bits(v[i]));
      }
    }
#pragma unroll
    for (int o = 32; o >= LW; o >>= 1)
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] = max(m[i], (uint32_t)__shfl_xor((int)m[i], o, 64));
    if (lane < LW) {
#pragma unroll
      for (int i = 0; i < 8; ++i) best[wave][lane * 8 + i] = m[i];
    }
    __syncthreads();
    if (threadIdx.x < CW && n0 + threadIdx.x < N) {
      uint32_t a = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) a = max(a, best[i][threadIdx.x]);
      sf[(size_t)e * N + n0 + threadIdx.x] = int8_scale(a);
    }
    __syncthreads();
  }
}

constexpr int QT = 64;  // columns and reduction elements of a turned tile

// Tile x of nx column tiles by ny reduction tiles of matrix e; a thread loads 8 columns of 2 rows.
template <typename XT>
__global__ __launch_bounds__(256) void quant_weights_i8_kernel(const XT* __restrict__ w, int K, int N, int nx, int ny,
                                                               int64_t tiles, const float* __restrict__ sf,
                                                               int8_t* __restrict__ q) {
  __shared__ int8_t tile[QT][QT + 4];  // [column][k]
  const int lc = threadIdx.x & 7, lr = threadIdx.x >> 3;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t e = t / ((int64_t)nx * ny);
    const int rem = (int)(t - e * nx * ny);
    const int by = rem / nx, n0 = (rem - by * nx) * QT, k0 = by * QT;
    const int n = N - n0 - lc * 8;
    float s[8], inv[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s[i] = i < n ? sf[(size_t)e * N + n0 + lc * 8 + i] : 1.0f;
      inv[i] = s[i] == s[i] ? __fdiv_rn(1.0f, s[i]) : 0.f;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = lr + 32 * h;
      if (n > 0 && k0 + k < K) {
        float v[8];
        load8(w + ((size_t)e * K + k0 + k) * N + n0 + lc * 8, n, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = inv[i] == 0.f ? 0.f : v[i];  // a column with a NaN or an infinity: codes 0
          tile[lc * 8 + i][k] = (int8_t)(int)int8_code(x, s[i], inv[i]);
        }
      }
    }
    __syncthreads();
    // four threads of sixteen codes per column
    const int col = threadIdx.x >> 2, kq = (threadIdx.x & 3) * 16;
    const int left = K - k0 - kq;
    if (n0 + col < N && left > 0) {
      int8_t* dst = q + ((size_t)e * N + n0 + col) * K + k0 + kq;
      if (left >= 16) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = *reinterpret_cast<const uint32_t*>(&tile[col][kq + 4 * i]);
        __builtin_memcpy(dst, u, 16);
      } else {
        for (int i = 0; i < left; ++i) dst[i] = tile[col][kq + i];
      }
    }
    __syncthreads();
  }
}

template <typename XT>
__global__ __launch_bounds__(256) void dequant_weights_i8_kernel(const int8_t* __restrict__ q,
                                                                 const float* __restrict__ sf, int K, int N, int nx,
                                                                 int ny, int64_t tiles, XT* __restrict__ out) {
  __shared__ int8_t tile[QT][QT + 4];  // [column][k]
  const int lc = threadIdx.x & 7, lr = threadIdx.x >> 3;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t e = t / ((int64_t)nx * ny);
    const int rem = (int)(t - e * nx * ny);
    const int by = rem / nx, n0 = (rem - by * nx) * QT, k0 = by * QT;
    const int col = threadIdx.x >> 2, kq = (threadIdx.x & 3) * 16;
    const int left = K - k0 - kq;
    if (n0 + col < N && left > 0) {
      const int8_t* src = q + ((size_t)e * N + n0 + col) * K + k0 + kq;
      if (left >= 16) {
        uint32_t u[4];
        __builtin_memcpy(u, src, 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint32_t*>(&tile[col][kq + 4 * i]) = u[i];
      } else {
        for (int i = 0; i < left; ++i) tile[col][kq + i] = src[i];
      }
    }
    __syncthreads();
    const int n = N - n0 - lc * 8;
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = i < n ? sf[(size_t)e * N + n0 + lc * 8 + i] : 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = lr + 32 * h;
      if (n > 0 && k0 + k < K) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? (float)tile[lc * 8 + i][k] * s[i] : 0.f;
        store8(out + ((size_t)e * K + k0 + k) * N + n0 + lc * 8, n, v);
      }
    }
    __syncthreads();
  }
}

constexpr int64_t MAX_GRID = 1 << 22;  // blocks of 256 threads: a launch counts its threads in 32 bits

unsigned grid_of(int64_t blocks) { return (unsigned)(blocks < MAX_GRID ? blocks : MAX_GRID); }

template <typename XT>
moe_status_t quantize_rows(const XT* x, int R, int C, int8_t* q, float* sf, hipStream_t s) {
  // a wave per row holds up to 1024 values, a block up to 8192
  if (C <= 512)
    quant_rows_i8_kernel<XT, 64, 1><<<grid_of(((int64_t)R + 3) / 4), 256, 0, s>>>(x, R, C, q, sf);
  else if (C <= 1024)
    quant_rows_i8_kernel<XT, 64, 2><<<grid_of(((int64_t)R + 3) / 4), 256, 0, s>>>(x, R, C, q, sf);
  else if (C <= 2048)
    quant_rows_i8_kernel<XT, 256, 1><<<grid_of(R), 256, 0, s>>>(x, R, C, q, sf);
  else if (C <= 4096)
    quant_rows_i8_kernel<XT, 256, 2><<<grid_of(R), 256, 0, s>>>(x, R, C, q, sf);
  else
    quant_rows_i8_kernel<XT, 256, 4><<<grid_of(R), 256, 0, s>>>(x, R, C, q, sf);
  return launch_status();
}

template <typename XT>
moe_status_t dequantize_rows(const int8_t* q, const float* sf, int R, int C, XT* out, hipStream_t s) {
  if (C <= 1024)
    dequant_rows_i8_kernel<XT, 64><<<grid_of(((int64_t)R + 3) / 4), 256, 0, s>>>(q, sf, R, C, out);
  else
    dequant_rows_i8_kernel<XT, 256><<<grid_of(R), 256, 0, s>>>(q, sf, R, C, out);
  return launch_status();
}

template <typename XT>
moe_status_t quantize_weights(const XT* w, int E, int K, int N, int8_t* q, float* sf, hipStream_t s) {
  const int ncb = (N + 63) / 64;
  const int64_t blocks = (int64_t)E * ncb;
  weight_scales_i8_kernel<XT, 8><<<(unsigned)(blocks < 1 << 20 ? blocks : 1 << 20), 1024, 0, s>>>(w, K, N, ncb, blocks, sf);
  const moe_status_t st = launch_status();
  if (st != MOE_OK) return st;
  const int nx = (N + QT - 1) / QT, ny = (K + QT - 1) / QT;
  const int64_t tiles = (int64_t)E * nx * ny;
  quant_weights_i8_kernel<XT><<<grid_of(tiles), 256, 0, s>>>(w, K, N, nx, ny, tiles, sf, q);
  return launch_status();
}

template <typename XT>
moe_status_t dequantize_weights(const int8_t* q, const float* sf, int E, int K, int N, XT* out, hipStream_t s) {
  const int nx = (N + QT - 1) / QT, ny = (K + QT - 1) / QT;
  const int64_t tiles = (int64_t)E * nx * ny;
  dequant_weights_i8_kernel<XT><<<grid_of(tiles), 256, 0, s>>>(q, sf, K, N, nx, ny, tiles, out);
  return launch_status();
}

}  // namespace

moe_status_t launch_quantize_int8(const void* x, moe_dtype_t xt, int R, int C, int8_t* q, float* sf, hipStream_t s) {
  if (xt == MOE_BF16) return quantize_rows(static_cast<const uint16_t*>(x), R, C, q, sf, s);
  return quantize_rows(static_cast<const float*>(x), R, C, q, sf, s);
}

moe_status_t launch_dequantize_int8(const int8_t* q, const float* sf, int R, int C, void* out, moe_dtype_t ot,
                                    hipStream_t s) {
  if (ot == MOE_BF16) return dequantize_rows(q, sf, R, C, static_cast<uint16_t*>(out), s);
  return dequantize_rows(q, sf, R, C, static_cast<float*>(out), s);
}

moe_status_t launch_quantize_int8_weights(const void* w, moe_dtype_t wt, int E, int K, int N, int8_t* q, float* sf,
                                          hipStream_t s) {
  if (wt == MOE_BF16) return quantize_weights(static_cast<const uint16_t*>(w), E, K, N, q, sf, s);
  return quantize_weights(static_cast<const float*>(w), E, K, N, q, sf, s);
}

moe_status_t launch_dequantize_int8_weights(const int8_t* q, const float* sf, int E, int K, int N, void* out,
                                            moe_dtype_t ot, hipStream_t s) {
  if (ot == MOE_BF16) return dequantize_weights(q, sf, E, K, N, static_cast<uint16_t*>(out), s);
  return dequantize_weights(q, sf, E, K, N, static_cast<float*>(out), s);
}

}  // namespace moe
