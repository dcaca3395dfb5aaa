// Grouped products with few rows and few columns: the weights are read once and hardly reused, so what counts
// is to have many of their bytes in flight. A wave takes a few columns and a slice of the reduction and
// streams the weights past up to 16 rows straight into registers, with the weights as the first operand of
// the 16 x 16 matrix instructions (lane l: column l % 16, quarter G = l / 16 of the instruction's k) and the
// rows as the second.
//   weights [N][K]  16 columns a wave. In a step a lane takes the 64 bytes at 64 G of its column's next 256: two whole
//                   lines per column and step. Which k an instruction multiplies is free as long as the rows agree.
//   weights [K][N]  64 columns a wave, 32 k a step. A lane takes four neighbouring columns of the eight k rows
//                   8 G + j; instruction i multiplies the columns 4 (l % 16) + i. bf16 pairs of rows are brought
//                   together by byte permutes, fp32 needs none.
// What bounds it is the weights' HBM stream: one token of 8 experts, 7168 x 2048, weights not cached: bf16 44
// us (235 MB, 5.3 TB/s; a plain read of 4 GiB reaches 5.95), INT8 gate/up 50 (235 MB, 4.7 TB/s); one row of a
// dense INT8 7168 x 2048, 14.7 MB, 6-7 us: the launch and one trip to memory.
// The next step's loads are out before this one's products. A block of eight waves splits the reduction `ks`
// ways and adds the slices in their order through LDS, so the result does not depend on timing. An expert
// with more rows gets a block per 16 of them.
#pragma once

#include "grouped_gemm.h"

namespace moe {

constexpr int GS_THREADS = 512;

template <class EL, bool BKC>
struct GsStep {
  static constexpr int WV = BKC || EL::BYTES == 2 ? 4 : 8;     // 16-byte words of weights a lane holds
  static constexpr int XV = BKC ? 4 : EL::BYTES == 2 ? 1 : 2;  // and of its row
  i32x4_t w[WV], x[XV];
};

template <class EL, typename ACC>
__device__ __forceinline__ void gs_mma(ACC& acc, i32x4_t w, i32x4_t x) {
  if constexpr (EL::BYTES == 1) {
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x, acc, 0, 0, 0);
  } else if constexpr (EL::BYTES == 2) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w), __builtin_bit_cast(bf16x8_t, x), acc, 0, 0,
                                                  0);
  } else {
    const f32x4_t wf = __builtin_bit_cast(f32x4_t, w), xf = __builtin_bit_cast(f32x4_t, x);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(wf[j], xf[j], acc, 0, 0, 0);
  }
}

template <class EL, bool BKC, bool OUT_F32, bool GATED>
__global__ __launch_bounds__(GS_THREADS) void gg_stream_kernel(GgArgs a, int ks) {
  using acc_t = typename std::conditional<std::is_same<EL, ElI8>::value, i32x4_t, f32x4_t>::type;
  using out_t = typename std::conditional<std::is_same<EL, ElI8>::value, int, float>::type;
  using Step = GsStep<EL, BKC>;
  constexpr bool SCALED = std::is_same<EL, ElI8>::value;
  constexpr int ES = EL::BYTES, ROWS = 16;
  constexpr int WC = BKC ? 16 : 64;             // columns of a wave
  constexpr int NA = BKC ? 1 : 4;               // its 16 x 16 accumulators
  constexpr int WM = GATED ? 4 : 8;             // waves per matrix
  constexpr int KB = BKC ? 256 : 32 * ES;       // bytes of a row of x that a step takes
  constexpr int LD = WC + 4;
  __shared__ __attribute__((aligned(16))) out_t part[8][16][LD];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int N = a.N, Kd = a.Kd;
  const int groups = WM / ks;                   // column groups of a block
  const int BN = groups * WC;
  const int ncb = (N + BN - 1) / BN;
  // Eight neighbours on one XCD (they share lines at their borders, and a heavy expert's panels), the eights
  // round-robin.
  const int whole = gridDim.x & ~63;
  const int b = blockIdx.x;
  const int idx = b < whole ? (b & ~63) + (b & 7) * 8 + ((b >> 3) & 7) : b;
  const int left = idx / ncb;  // this block's chunk among the experts' chunks of ROWS rows, in expert order
  int e = -1, before = 0, chunks = 0;
  for (int base = 0; base < a.E; base += 64) {
    const int i = min(base + lane, a.E - 1);
    const int beg = group_begin(a.cu, i, a.M);
    const int n = base + lane < a.E ? (group_rows(a.cu, i, a.M, beg) + ROWS - 1) / ROWS : 0;
    const int upto = sched_wave_incl_scan(n);
    const uint64_t hit = __ballot(before + upto > left);
    if (hit) {
      const int j = __builtin_ctzll(hit);
      e = base + j;
      chunks = __builtin_amdgcn_readlane(n, j);
      before += __builtin_amdgcn_readlane(upto, j) - chunks;
      break;
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  if (e < 0) return;
  const int local = idx - before * ncb;
  const int cb = local / chunks, r0 = (local - cb * chunks) * ROWS;
  const int gbeg = __builtin_amdgcn_readfirstlane(group_begin(a.cu, e, a.M));
  const int rows = __builtin_amdgcn_readfirstlane(group_rows(a.cu, e, a.M, gbeg));

  const int c16 = lane & 15, G = lane >> 4;
  const int wl = wave % WM;
  const int slice = wl % ks;
  const int n0 = cb * BN + wl / ks * WC;        // the wave's first column
  const size_t pitch = (size_t)Kd * ES, npitch = (size_t)N * ES;
  const int steps = (int)((pitch + KB - 1) / KB);
  const unsigned char* B = static_cast<const unsigned char*>(GATED && wave >= WM ? a.B1 : a.B0);
  // columns past the last read another one's values; their results are not stored
  const unsigned char* wp;
  if constexpr (BKC) wp = B + ((size_t)e * N + min(n0 + c16, N - 1)) * pitch + G * 64;
  else wp = B + ((size_t)e * Kd + 8 * G) * npitch + (size_t)min(n0 + 4 * c16, N - 4) * ES;

  // rows past the last read it again; their results are not stored
  int xr = gbeg + min(r0 + c16, rows - 1);
  bool dead = false;  // a row that reads zeros
  if (a.row_src) {
    const int src = a.row_src[xr];
    xr = src / a.a_k;
    dead = src < 0 || xr >= a.a_rows;
    if (dead) xr = 0;
  }
  const unsigned char* xp = static_cast<const unsigned char*>(a.A) + (size_t)xr * pitch + G * (BKC ? 64 : 8 * ES);
  const bool any_dead = __ballot(dead) != 0;

  acc_t acc[NA];
#pragma unroll
  for (int i = 0; i < NA; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[i][c] = 0;

  const i32x4_t z = {0, 0, 0, 0};
  // Step `it` of this lane; what lies past the end of the reduction reads as zeros.
  auto load = [&](Step& d, int it) __attribute__((always_inline)) {
    const bool tail = (size_t)(it + 1) * KB > pitch;
    if constexpr (BKC) {
      const int left_b = (int)(pitch - (size_t)it * KB) - G * 64;  // bytes of the row from this lane's word on
      const size_t o = (size_t)it * KB;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const bool in = !tail || 16 * q < left_b;
        const ptrdiff_t at = in ? (ptrdiff_t)(o + 16 * q) : -G * 64;
        d.w[q] = *reinterpret_cast<const i32x4_t*>(wp + at);
        d.x[q] = *reinterpret_cast<const i32x4_t*>(xp + at);
        if (!in) d.w[q] = d.x[q] = z;
      }
    } else {
      const int left_k = Kd - it * 32 - 8 * G;                  // k rows from this lane's first on
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool in = !tail || j < left_k;
        const unsigned char* p = wp + (in ? (ptrdiff_t)((size_t)(it * 32 + j) * npitch) : -(ptrdiff_t)(8 * G * npitch));
        if constexpr (ES == 4) {
          d.w[j] = *reinterpret_cast<const i32x4_t*>(p);
          if (!in) d.w[j] = z;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(p);
          d.w[j / 2][2 * (j & 1)] = in ? (int)v.x : 0;
          d.w[j / 2][2 * (j & 1) + 1] = in ? (int)v.y : 0;
        }
      }
#pragma unroll
      for (int q = 0; q < Step::XV; ++q) {
        const bool in = !tail || q * (16 / ES) < left_k;
        d.x[q] = *reinterpret_cast<const i32x4_t*>(xp + (in ? (ptrdiff_t)((size_t)it * KB + 16 * q) : -G * 8 * ES));
        if (!in) d.x[q] = z;
      }
    }
    if (any_dead) {
#pragma unroll
      for (int q = 0; q < Step::XV; ++q)
        if (dead) d.x[q] = z;
    }
  };
  auto mul = [&](const Step& d) __attribute__((always_inline)) {
    if constexpr (BKC) {
#pragma unroll
      for (int q = 0; q < 4; ++q) gs_mma<EL>(acc[0], d.w[q], d.x[q]);
    } else if constexpr (ES == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // column i of the lane's four: its values of k rows 2 p and 2 p + 1 side by side
        i32x4_t w;
#pragma unroll
        for (int p = 0; p < 4; ++p)
          w[p] = (int)__builtin_amdgcn_perm((uint32_t)d.w[p][2 + i / 2], (uint32_t)d.w[p][i / 2], i & 1 ? 0x07060302u : 0x05040100u);
        gs_mma<EL>(acc[i], w, d.x[0]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const f32x4_t w = __builtin_bit_cast(f32x4_t, d.w[j]);
        const float x = __builtin_bit_cast(f32x4_t, d.x[j / 4])[j & 3];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(w[i], x, acc[i], 0, 0, 0);
      }
    }
  };
  Step s0, s1;
  // slice s takes every ks-th step: the waves of a block read neighbouring lines
  if (slice < steps) load(s0, slice);
  for (int it = slice; it < steps; it += 2 * ks) {
    if (it + ks < steps) load(s1, it + ks);
    mul(s0);
    if (it + 2 * ks < steps) load(s0, it + 2 * ks);
    if (it + ks < steps) mul(s1);
  }

  // lane l holds row l % 16 and the columns 4 G + c (weights [N][K]) or 16 G + 4 c + i ([K][N]) of the wave's
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int i = 0; i < NA; ++i) part[wave][c16][BKC ? 4 * G + c : 16 * G + 4 * c + i] = acc[i][c];
  __syncthreads();
  for (int q = tid; q < 16 * BN; q += GS_THREADS) {
    const int r = q / BN, cl = q - r * BN;
    const int col = cb * BN + cl;
    if (r0 + r >= rows || col >= N) continue;
    const int w0 = cl / WC * ks, cc = cl % WC;
    out_t s = 0, s1v = 0;
    for (int k = 0; k < ks; ++k) {
      s += part[w0 + k][r][cc];
      if constexpr (GATED) s1v += part[WM + w0 + k][r][cc];
    }
    float v = (float)s;
    const size_t row = (size_t)gbeg + r0 + r;
    if constexpr (SCALED) {
      size_t src_row = row;
      bool live = true;
      if (a.row_src) {
        const int src = a.row_src[row];
        live = src >= 0 && src / a.a_k < a.a_rows;
        src_row = live ? src / a.a_k : 0;
      }
      const float sa = live ? a.a_sf[src_row] : 0.f;
      v = v * sa * a.b_sf0[(size_t)e * N + col];
      if constexpr (GATED) v = silu_f32(v) * ((float)s1v * sa * a.b_sf1[(size_t)e * N + col]);
      if (sa == 0.f) v = 0.f;  // a padding row is zeros whatever the weights' scales hold
    }
    if constexpr (OUT_F32) static_cast<float*>(a.C)[row * N + col] = v;
    else static_cast<uint16_t*>(a.C)[row * N + col] = f32_to_bf16_bits(v);
  }
}

template <class EL, bool BKC, bool OUT_F32, bool GATED>
moe_status_t launch_gg_stream(const GgArgs& a, hipStream_t s) {
  constexpr int WC = BKC ? 16 : 64, WM = GATED ? 4 : 8;
  const int64_t slots = a.M < a.E ? a.M : a.E;  // at most so many experts have rows
  // n experts with R rows make at most n + (R - n) / 16 chunks; blocks past the last one have none
  const int64_t chunks = slots + (a.M - slots) / 16;
  // Slices of the reduction: as many as leave 8 waves a CU (fp32, whose products take longer: 16). Measured,
  // us, by 8 / 4 / 2 / 1 slices, weights not in a cache (gated: 4 / 2 / 1): INT8 1 x 7168 x 2048 (128 waves
  // unsplit) 7 / 11 / 18 / 33; gate/up, 8 experts 7168 x 2048 (2048) 57 / 58 / 50; bf16 [K][N], 8 experts
  // 7168 x 2048 (256) 44 / 68 / 125 / 243. In a cache: INT8, 8 experts 7168 x 2048 (1024) 24.5 / 24.2 / 23.9
  // / 39, 2048 x 7168 (3584) 37 / 31 / 26 / 25; fp32, 64 experts 2048 x 1024 (1024) 101 / 98 / - / 153.
  // (counted for evenly filled groups)
  const int64_t waves = slots * (((a.M + slots - 1) / slots + 15) / 16) * ((a.N + WC - 1) / WC) * (GATED ? 2 : 1);
  int ks = WM;
  while (ks > 1 && waves * ks > (EL::BYTES == 4 ? 16 : 8) * (int64_t)device_cu_count()) ks /= 2;
  const int BN = WM / ks * WC;
  const unsigned blocks = (unsigned)(chunks * ((a.N + BN - 1) / BN));
  gg_stream_kernel<EL, BKC, OUT_F32, GATED><<<blocks, GS_THREADS, 0, s>>>(a, ks);
  return launch_status();
}

}  // namespace moe
