// INT8 quantisation of activations (a scale per row) and of stacked weights (a scale per output
// column), and the way back. The arithmetic is in int8.h.
//
//  rows:     x [R, C] -> q [R, C], sf [R]. A row belongs to 64 or 256 threads; each holds its
//            values in registers between the maximum and the codes, so that x is read once (rows of
//            more than 8192 values are read again, from the cache).
//  weights:  w [E, K, N] (reduction first) -> q [E, N, K], sf [E, N]. The maximum of a column needs all
//            of K before the first code, so the values are read twice; codes are turned through LDS
//            and written in runs along k.
// All are bound by HBM (a large copy reaches 4.8 TB/s here): rows 8191 x 7168 bf16, operands not cached 41 us
// (4.25 TB/s), read and written again 35, and back 33 and 27; 65536 x 2048 70 either way (5.75 TB/s);
// operands read and written again: weights 64 x 2048 x 1024 fp32 212-220 us, 5.6 TB/s over both reads, and
// back to bf16 90; 52 x 7168 x 2048 bf16 790-805, and back 447-467. The second read of the weights costs a
// third to a half of a call that is made once per weight: values that stay in registers between the passes
// need a column's whole reduction in one block, which holds for K up to some 2048 in fp32 (32 columns: 256 KB
// of a CU's 512) and was not tried.
// Any C, K and N: rows may start at any element, whole 16-byte words are loaded where they lie inside the row
// and single elements at its end.
#include "int8.h"
#include "tile_sched.h"

namespace moe {

namespace {

// Eight values at p, at any element.
template <typename XT>
__device__ __forceinline__ void load8(const XT* p, float (&v)[8]) {
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
}

// The first n (at most eight, or none) of them; the others zero. A loop over several takes the whole ones
// without a branch in between, or each would wait for the one before.
template <typename XT>
__device__ __forceinline__ void load8(const XT* p, int n, float (&v)[8]) {
  if (n >= 8) {
    load8(p, v);
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
  const float s1[1] = {s}, inv1[1] = {inv};
  uint32_t c[8];
  int8_codes<8, 1>(v, s1, inv1, inv == 0.f, c);
  const uint32_t u[2] = {low_bytes(c[0], c[1], c[2], c[3]), low_bytes(c[4], c[5], c[6], c[7])};
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
    if (((CH - 1) * TPR + t) * 8 + 8 <= C) {
#pragma unroll
      for (int c = 0; c < CH; ++c) load8(xr + (c * TPR + t) * 8, v[c]);
    } else {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int at = (c * TPR + t) * 8;
        load8(xr + (at < C ? at : 0), C - at, v[c]);
      }
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
    const float s = int8_scale(m);
    if (t == 0) sf[r] = s;
    int8_t* qr = q + (size_t)r * C;
    const float inv = m >= 0x7f800000u ? 0.f : __fdiv_rn(1.0f, s);  // 0: zero codes
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int at = (c * TPR + t) * 8;
      if (at < C) store_codes(qr + at, C - at, v[c], s, inv);
    }
    for (int64_t at = (int64_t)(CH * TPR + t) * 8; at < C; at += TPR * 8) {
      const int n = (int)min((int64_t)8, C - at);
      float u[8];
      load8(xr + at, n, u);
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

// ---- weights -----------------------------------------------------------------------------
// Slabs of 64 columns: eight lanes side by side take eight columns each. The threads of a block along k take
// four neighbouring rows each, so that four codes of a column make one dword of the turned tile [column][k]
// in LDS. Its rows are 65 dwords long: the dwords that a wave writes (eight columns apart, eight along k)
// fall on different banks. (Slabs of 128 columns of bf16, 256 bytes of a row, took longer: 52 x 7168 x 2048
// 930 us against 809, and back 582 against 446.)
constexpr int QW_THREADS = 512;
constexpr int QW_COLS = 64, QW_K = 256;
constexpr int QW_LD = QW_K / 4 + 1;

// First of the eight columns of a lane whose own begin at n: the last eight where fewer are left (shared with
// its neighbour, computed twice, alike).
__device__ __forceinline__ int first_column(int n, int N) { return N >= 8 ? min(n, N - 8) : n; }

// Block b of G: neighbours on one XCD, so that the lines that two tiles or slabs share (rows that do not end
// on whole lines) meet in one L2.
__device__ __forceinline__ int64_t near_block(int b, int G) {
  const int even = G & ~7;
  return b < even ? xcd_slot(b, even) : b;
}

typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));

// Largest magnitudes of the n columns from p on (at most eight count; none: n = 0) over the K rows of w,
// joined over the block: best[..][first + i].
// Eight rows are loaded before the first is looked at: the bytes in flight bound this pass.
template <int WAVES, typename XT>
__device__ __forceinline__ void column_max(const XT* p, int n, int first, int K, int N, uint32_t (&best)[WAVES][QW_COLS]) {
  constexpr int STEP = 8 * WAVES, U = sizeof(XT) == 2 ? 8 : 4, WORDS = 8 * sizeof(XT) / 4;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, lr = threadIdx.x >> 3;
  uint32_t m[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  int k = lr;
  if (n >= 8) {
    uint32_t top[WORDS] = {};  // bf16: two columns a word
    for (; k + (U - 1) * STEP < K; k += U * STEP) {
      uint32_t raw[U][WORDS];
#pragma unroll
      for (int u = 0; u < U; ++u) __builtin_memcpy(raw[u], p + (size_t)(k + u * STEP) * N, WORDS * 4);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
          if constexpr (sizeof(XT) == 2)
            top[i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, top[i]),
                                                                           __builtin_bit_cast(u16x2_t, raw[u][i] & 0x7fff7fffu)));
          else
            top[i] = max(top[i], raw[u][i] & 0x7fffffffu);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(XT) == 2) m[i] = i & 1 ? top[i / 2] & 0xffff0000u : top[i / 2] << 16;
      else m[i] = top[i];
    }
  }
  if (n > 0) {
    for (; k < K; k += STEP) {
      float v[8];
      load8(p + (size_t)k * N, n, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] = max(m[i], abs_bits(v[i]));
    }
  }
#pragma unroll
  for (int o = 32; o >= 8; o >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = max(m[i], (uint32_t)__shfl_xor((int)m[i], o, 64));
  if (lane < 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (first + i >= 0 && i < n) best[wave][first + i] = m[i];
  }
  __syncthreads();
}

template <typename XT>
__global__ __launch_bounds__(1024) void weight_scales_i8_kernel(const XT* __restrict__ w, int K, int N, int ncb,
                                                                int64_t blocks, float* __restrict__ sf) {
  __shared__ uint32_t best[16][QW_COLS];
  for (int64_t b = near_block(blockIdx.x, gridDim.x); b < blocks; b += gridDim.x) {
    const int64_t e = b / ncb;
    const int n0 = (int)(b - e * ncb) * QW_COLS;
    const int lc = threadIdx.x & 7;
    const bool live = n0 + lc * 8 < N;
    const int c0 = live ? first_column(n0 + lc * 8, N) : 0;
    column_max<16>(w + (size_t)e * K * N + c0, live ? N - c0 : 0, c0 - n0, K, N, best);
    if (threadIdx.x < QW_COLS && n0 + threadIdx.x < N) {
      uint32_t a = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) a = max(a, best[i][threadIdx.x]);
      sf[(size_t)e * N + n0 + threadIdx.x] = int8_scale(a);
    }
    __syncthreads();
  }
}

// Codes, a turned tile at a time, last tiles first: what the scales' pass read last is still in the
// last-level cache.
template <typename XT>
__global__ __launch_bounds__(QW_THREADS) void quant_weights_i8_kernel(const XT* __restrict__ w, int K, int N, int ncb,
                                                                      int ny, int64_t tiles,
                                                                      const float* __restrict__ sf,
                                                                      int8_t* __restrict__ q) {
  __shared__ uint32_t tile[QW_COLS][QW_LD];
  const int lc = threadIdx.x & 7, lr = threadIdx.x >> 3;
  for (int64_t t = tiles - 1 - near_block(blockIdx.x, gridDim.x); t >= 0; t -= gridDim.x) {
    const int64_t slab = t / ny;
    const int64_t e = slab / ncb;
    const int n0 = (int)(slab - e * ncb) * QW_COLS, k0 = (int)(t - slab * ny) * QW_K;
    const bool live = n0 + lc * 8 < N;
    const int c0 = live ? first_column(n0 + lc * 8, N) : 0, n = live ? N - c0 : 0;
    const XT* p = w + ((size_t)e * K + k0 + 4 * lr) * N + c0;
    float v[4][8], s[8], inv[8];
    if (n >= 8 && k0 + 4 * lr + 4 <= K) {
#pragma unroll
      for (int j = 0; j < 4; ++j) load8(p + (size_t)j * N, v[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = n > 0 && k0 + 4 * lr + j < K;
        load8(in ? p + (size_t)j * N : w, in ? n : 0, v[j]);
      }
    }
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s[i] = i < n ? sf[(size_t)e * N + c0 + i] : 1.0f;
      inv[i] = s[i] == s[i] ? __fdiv_rn(1.0f, s[i]) : 0.f;
      bad |= inv[i] == 0.f;
    }
    uint32_t r[4][8];
#pragma unroll
    for (int j = 0; j < 4; ++j) int8_codes<8, 8>(v[j], s, inv, bad, r[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n && c0 + i >= n0) tile[c0 + i - n0][lr] = low_bytes(r[0][i], r[1][i], r[2][i], r[3][i]);
    __syncthreads();
    const int col = threadIdx.x >> 3;
    if (n0 + col < N) {
      int8_t* dst = q + ((size_t)e * N + n0 + col) * K + k0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = (threadIdx.x & 7) * 16 + 128 * h, left = K - k0 - at;
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = tile[col][at / 4 + i];
        if (left >= 16) {
          __builtin_memcpy(dst + at, u, 16);
        } else {
          for (int i = 0; i < left; ++i) dst[at + i] = (int8_t)(u[i >> 2] >> (8 * (i & 3)));
        }
      }
    }
    __syncthreads();
  }
}

// The way back, by the same turned tiles.
template <typename XT>
__global__ __launch_bounds__(QW_THREADS) void dequant_weights_i8_kernel(const int8_t* __restrict__ q,
                                                                        const float* __restrict__ sf, int K, int N,
                                                                        int ncb, int ny, int64_t tiles,
                                                                        XT* __restrict__ out) {
  __shared__ uint32_t tile[QW_COLS][QW_LD];
  const int lc = threadIdx.x & 7, lr = threadIdx.x >> 3;
  for (int64_t t = near_block(blockIdx.x, gridDim.x); t < tiles; t += gridDim.x) {
    const int64_t slab = t / ny;
    const int64_t e = slab / ncb;
    const int n0 = (int)(slab - e * ncb) * QW_COLS, k0 = (int)(t - slab * ny) * QW_K;
    const int col = threadIdx.x >> 3;
    if (n0 + col < N) {
      const int8_t* src = q + ((size_t)e * N + n0 + col) * K + k0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = (threadIdx.x & 7) * 16 + 128 * h, left = K - k0 - at;
        uint32_t u[4] = {0, 0, 0, 0};
        if (left >= 16) {
          __builtin_memcpy(u, src + at, 16);
        } else {
          for (int i = 0; i < left; ++i) u[i >> 2] |= (uint32_t)(uint8_t)src[at + i] << (8 * (i & 3));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) tile[col][at / 4 + i] = u[i];
      }
    }
    __syncthreads();
    const int n = N - n0 - lc * 8;
    if (n > 0) {
      float s[8];
      uint32_t c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[i] = i < n ? sf[(size_t)e * N + n0 + lc * 8 + i] : 0.f;
        c[i] = i < n ? tile[lc * 8 + i][lr] : 0;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = k0 + 4 * lr + j;
        if (k >= K) break;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i8_at(c[i], j) * s[i];
        store8(out + ((size_t)e * K + k) * N + n0 + lc * 8, n, v);
      }
    }
    __syncthreads();
  }
}

constexpr int64_t MAX_GRID = 1 << 21;  // blocks of up to 1024 threads: a launch counts its threads in 32 bits

unsigned grid_of(int64_t blocks) { return (unsigned)(blocks < MAX_GRID ? blocks : MAX_GRID); }

template <typename XT>
moe_status_t quantize_rows(const XT* x, int R, int C, int8_t* q, float* sf, hipStream_t s) {
  // a wave per row holds up to 2048 values (65536 rows of 2048: 118 us with a block each), a block 8192
  if (C <= 512)
    quant_rows_i8_kernel<XT, 64, 1><<<grid_of(((int64_t)R + 3) / 4), 256, 0, s>>>(x, R, C, q, sf);
  else if (C <= 1024)
    quant_rows_i8_kernel<XT, 64, 2><<<grid_of(((int64_t)R + 3) / 4), 256, 0, s>>>(x, R, C, q, sf);
  else if (C <= 2048)
    quant_rows_i8_kernel<XT, 64, 4><<<grid_of(((int64_t)R + 3) / 4), 256, 0, s>>>(x, R, C, q, sf);
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
  const int ncb = (N + QW_COLS - 1) / QW_COLS;
  const int64_t slabs = (int64_t)E * ncb;
  weight_scales_i8_kernel<XT><<<grid_of(slabs), 1024, 0, s>>>(w, K, N, ncb, slabs, sf);
  const moe_status_t st = launch_status();
  if (st != MOE_OK || K == 0) return st;
  const int ny = (K + QW_K - 1) / QW_K;
  quant_weights_i8_kernel<XT><<<grid_of(slabs * ny), QW_THREADS, 0, s>>>(w, K, N, ncb, ny, slabs * ny, sf, q);
  return launch_status();
}

template <typename XT>
moe_status_t dequantize_weights(const int8_t* q, const float* sf, int E, int K, int N, XT* out, hipStream_t s) {
  const int ncb = (N + QW_COLS - 1) / QW_COLS, ny = (K + QW_K - 1) / QW_K;
  const int64_t tiles = (int64_t)E * ncb * ny;
  dequant_weights_i8_kernel<XT><<<grid_of(tiles), QW_THREADS, 0, s>>>(q, sf, K, N, ncb, ny, tiles, out);
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
