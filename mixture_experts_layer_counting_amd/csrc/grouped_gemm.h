// Products of ragged expert groups on gfx950's matrix cores: what the kernels of bf16, fp32 and INT8
// share.
//
// Three products, C = A B per expert, all accumulated in 32 bits:
//   rows x weights [K][N]     y[r, n]  = sum_k x[r, k] W[k, n]
//   rows x weights [N][K]     y[r, n]  = sum_k x[r, k] W[n, k]
//   rows^T x rows             dW[m, n] = sum_r x[r, m] dy[r, n]
// An operand whose reduction runs along memory (KC) is staged as [rows][128 bytes], the other kind (MC) as
// [k][columns]. One stage is 128 bytes of reduction per row of a KC operand: 64 bf16, 32 fp32 or 128 INT8
// elements. In a step kk = 0..3 of a stage, lane l (half g = l / 32) feeds the matrix cores the 16 bytes of
// chunk 2 kk + g of its row or column l % 32:
//   bf16  v_mfma_f32_32x32x16_bf16, eight elements a lane: one instruction
//   INT8  v_mfma_i32_32x32x32_i8, sixteen: one instruction
//   fp32  v_mfma_f32_32x32x2_f32, one element a lane: four instructions, element j of each chunk
// Which k a lane takes is free as long as both operands agree. The weights (B) are the first operand, so
// a lane holds output row l % 32 and, in acc[4 j + c], column 8 j + 4 g + c.
#pragma once

#include "grouped_args.h"
#include "lds_dma.h"
#include "moe_common.h"
#include "tile_sched.h"

#include <type_traits>
#include <utility>

typedef int i32x16_t __attribute__((ext_vector_type(16)));

namespace moe {

constexpr int GG_MAX_E = 1024;

// First row of group e, kept inside [0, M] whatever cu holds.
__device__ __forceinline__ int group_begin(const int* cu, int e, int M) { return cu ? min(max(cu[e], 0), M) : e * M; }
__device__ __forceinline__ int group_rows(const int* cu, int e, int M, int begin) {
  return max(group_begin(cu, e + 1, M) - begin, 0);
}

// Writes tstart[0..E], the exclusive prefix of tiles(rows of e), and returns the total.
template <int THREADS, typename F>
__device__ int group_prefix(const int* cu, int M, int E, F tiles, int* tstart, int* wsum) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int total = 0;
  for (int base = 0; base < E; base += THREADS) {
    const int e = base + tid;
    int c = 0;
    if (e < E) c = tiles(group_rows(cu, e, M, group_begin(cu, e, M)));
    const int incl = sched_wave_incl_scan(c);
    if (lane == 63) wsum[wave] = incl;
    __syncthreads();
    int before = total;
    for (int w = 0; w < THREADS / 64; ++w) {
      if (w < wave) before += wsum[w];
      total += wsum[w];
    }
    if (e < E) tstart[e] = before + incl - c;
    __syncthreads();
  }
  if (tid == 0) tstart[E] = total;
  __syncthreads();
  return total;
}

// f(0), f(1), .. f(N - 1) with compile-time numbers.
template <typename F, int... I>
__device__ __forceinline__ void gg_for_impl(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void gg_for(F&& f) {
  gg_for_impl(f, std::make_integer_sequence<int, N>{});
}

// ---- element types ---------------------------------------------------------------------

struct ElBf16 {
  using acc_t = f32x16_t;
  static constexpr int BYTES = 2;
  static __device__ __forceinline__ void mma(acc_t& acc, i32x4_t b, i32x4_t a) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, b), __builtin_bit_cast(bf16x8_t, a), acc,
                                                  0, 0, 0);
  }
};

struct ElI8 {
  using acc_t = i32x16_t;
  static constexpr int BYTES = 1;
  static __device__ __forceinline__ void mma(acc_t& acc, i32x4_t b, i32x4_t a) {
    acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(b, a, acc, 0, 0, 0);
  }
};

struct ElF32 {
  using acc_t = f32x16_t;
  static constexpr int BYTES = 4;
  static __device__ __forceinline__ void mma(acc_t& acc, i32x4_t b, i32x4_t a) {
    const f32x4_t bf = __builtin_bit_cast(f32x4_t, b), af = __builtin_bit_cast(f32x4_t, a);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(bf[j], af[j], acc, 0, 0, 0);
  }
};

// ---- staged operands -------------------------------------------------------------------
// An operand of R rows (KC) or columns (MC) takes R * 128 bytes of LDS per stage, R * 8 chunks of 16.
// Chunk c lies at byte 16 c and holds:
//   KC  row c / 8, k chunk (c % 8) ^ (row / 2 % 8): sixteen lanes that read one chunk of sixteen rows
//       hit all banks once
//   MC  bf16: k row c / (R / 8), 32-byte segments swizzled by k, for the transposing reads;
//       fp32: k row c / (R / 4), in order
template <class EL, bool KC, int R>
struct Staged {
  static constexpr int EPC = 16 / EL::BYTES;       // elements of a chunk
  static constexpr int BK = 128 / EL::BYTES;       // reduction of a stage
  static constexpr int CPK = R / EPC;              // MC: chunks of a k row
  static __device__ __forceinline__ int row(int c) { return KC ? c >> 3 : c / CPK; }  // KC: operand row; MC: k
  static __device__ __forceinline__ int chunk(int c) {                               // along the other axis
    if constexpr (KC) {
      return (c & 7) ^ ((c >> 4) & 7);
    } else if constexpr (EL::BYTES == 2) {
      const int q = c % CPK;
      return ((((q >> 1) ^ swizzle(c / CPK)) << 1) | (q & 1));
    } else {
      return c % CPK;
    }
  }

  // MC bf16: a transposing read takes 64 bytes of four k rows, which have to fall on different banks; rows of
  // 64 columns are half of them long
  static __device__ __forceinline__ int swizzle(int k) { return R >= 128 ? (k & 3) << 1 : k & 2; }

  // Where this lane's fragments of the 32 rows or columns from `block` on (a multiple of 32) begin. Blocks
  // that differ by the bits of `flip` in at() share it.
  static __device__ __forceinline__ int base(int block, int lane) {
    const int l32 = lane & 31, g2 = lane >> 5;
    if constexpr (KC) {
      return (block + l32) * 128;
    } else if constexpr (EL::BYTES == 2) {
      const int g = lane >> 4, jj = lane & 15;  // the transposing read works on groups of sixteen lanes
      return (8 * (g >> 1) + (jj >> 2)) * (R * 2) + 8 * (jj & 3) + (((block / 16 + (g & 1)) ^ swizzle(jj >> 2)) << 5);
    } else {
      return 4 * g2 * (R * 4) + (block + l32) * 4;
    }
  }
  // The fragment of step kk from a base; `nt`: blocks of 32 further on (MC bf16: base's block has zeros in
  // the bits of nt)
  static __device__ __forceinline__ i32x4_t frag(const unsigned char* st, int base, int nt, int kk, int lane) {
    if constexpr (KC) {
      const int at = base + nt * 32 * 128 + (((2 * kk + (lane >> 5)) ^ ((lane >> 1) & 7)) << 4);
      return *reinterpret_cast<const i32x4_t*>(st + at);
    } else if constexpr (EL::BYTES == 2) {
      const unsigned char* p = st + (base ^ (nt << 6)) + kk * 16 * (R * 2);
      const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS i16x4_t*)(p));
      const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS i16x4_t*)(p + 4 * (R * 2)));
      return __builtin_bit_cast(i32x4_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      const unsigned char* p = st + base + nt * 128 + kk * 8 * (R * 4);
      i32x4_t v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const int*>(p + j * (R * 4));
      return v;
    }
  }
};

// Eight bf16 at p, at any alignment. What lies past `end`, the operand's last element, reads as zeros.
__device__ __forceinline__ i32x4_t load_chunk(const uint16_t* p, const uint16_t* end) {
  i32x4_t v = {0, 0, 0, 0};
  if (p + 8 <= end) {
    __builtin_memcpy(&v, p, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (p + i < end) v[i / 2] |= (int)p[i] << (16 * (i & 1));
  }
  return v;
}

// The first n elements of a chunk; the others zero.
__device__ __forceinline__ i32x4_t first_of_chunk(i32x4_t v, int n) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (2 * i >= n) v[i] = 0;
    else if (2 * i + 1 >= n) v[i] &= 0xffff;
  }
  return v;
}

// ---- epilogue --------------------------------------------------------------------------

// Eight values of a row: v[0..3] at columns c .. c + 3 and v[4..7] at c + 8 .. c + 11, c = c0 + 4 (lane / 32);
// the wave's row block covers columns c0 .. c0 + 15. `vec`: rows are whole 16-byte words of the output.
template <bool OUT_F32>
__device__ __forceinline__ void store_run(void* C, size_t row, int N, int c0, int lane, bool ok, bool vec,
                                          const float (&v)[8]) {
  const int g2 = lane >> 5;
  if constexpr (OUT_F32) {
    float* p = static_cast<float*>(C) + row * N;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = c0 + 8 * h + 4 * g2;
      if (vec) {
        if (ok && c < N) *reinterpret_cast<float4*>(p + c) = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (ok && c + i < N) p[c + i] = v[4 * h + i];
      }
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(C) + row * N;
    if (vec) {
      const uint4 q = pack_row16(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]);
      const int c = c0 + 8 * g2;
      if (ok && c < N) *reinterpret_cast<uint4*>(p + c) = q;
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = c0 + 8 * h + 4 * g2 + i;
          if (ok && c < N) p[c] = f32_to_bf16_bits(v[4 * h + i]);
        }
    }
  }
}

// Whether rows of N output values start and end on 16-byte words.
template <bool OUT_F32>
__device__ __forceinline__ bool whole_words(const void* C, int N) {
  return N % (OUT_F32 ? 4 : 8) == 0 && (uintptr_t)C % 16 == 0;
}

// ---- bf16 rows that are not whole 16-byte words --------------------------------------------
//
// Tiles of T x T by four waves; a thread loads its chunks of a stage into registers PD stages ahead and
// writes them to one of two LDS buffers. A chunk that reaches past its row reads the next row's elements,
// which count for columns that are not stored or are cut off in the last stage of the reduction.
// TN: rows^T x rows.
constexpr int GA_THREADS = 256;

template <bool AKC, bool BKC, bool OUT_F32, int T, int PD>
__global__ __launch_bounds__(GA_THREADS, 2) void gg_any_kernel(GgArgs a) {
  constexpr bool TN = !AKC;
  using EL = ElBf16;
  using SA = Staged<EL, AKC, T>;
  using SB = Staged<EL, BKC, T>;
  using mem_t = uint16_t;
  constexpr int BK = SA::BK, EPC = SA::EPC;
  constexpr int CH = T * 8 / GA_THREADS;  // chunks of an operand that a thread loads per stage
  constexpr int W = T / 64;               // blocks of 32 x 32 of a wave along each axis
  constexpr int STAGE = 2 * T * 128;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  int* tstart = reinterpret_cast<int*>(smem + 2 * STAGE);
  int* wsum = tstart + GG_MAX_E + 1;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int ntn = (a.N + T - 1) / T;
  const int mtn = (a.Kd + T - 1) / T;  // TN: row tiles of dW
  int total;
  if constexpr (TN) total = a.E * mtn * ntn;
  else total = group_prefix<GA_THREADS>(a.cu, a.M, a.E, [&](int rows) { return (rows + T - 1) / T * ntn; }, tstart, wsum);
  const mem_t* A = static_cast<const mem_t*>(a.A);
  const mem_t* B = static_cast<const mem_t*>(a.B0);
  const mem_t* a_end = A + (size_t)(a.row_src ? a.a_rows : a.M) * a.Kd;
  const mem_t* b_end = B + (TN ? (size_t)a.M * a.N : (size_t)a.E * a.Kd * a.N);
  const bool vec = whole_words<OUT_F32>(a.C, a.N);
  const int a_base = SA::base(wm * 32 * W, lane), b_base = SB::base(wn * 32 * W, lane);

  for (int t = xcd_slot(blockIdx.x, gridDim.x); t < total; t += gridDim.x) {
    int e, mtile, ntile;
    if constexpr (TN) {
      e = t / (mtn * ntn);
      const int rem = t - e * mtn * ntn;
      mtile = rem / ntn;
      ntile = rem - mtile * ntn;
    } else {
      e = find_expert(tstart, a.E, t);
    }
    const int gbeg = group_begin(a.cu, e, a.M);
    const int rows_e = group_rows(a.cu, e, a.M, gbeg);
    if constexpr (!TN) {
      const int mte = (rows_e + T - 1) / T;
      const int lt = t - tstart[e];
      ntile = lt / mte;
      mtile = lt - ntile * mte;
    }
    const int m0 = mtile * T, n0 = ntile * T;
    const int mvalid = min(T, (TN ? a.Kd : rows_e) - m0);
    const int red = TN ? rows_e : a.Kd;        // length of the reduction
    const int nk = (red + BK - 1) / BK;
    // first element of this thread's chunks in stage 0; NULL where the row or column does not exist
    const mem_t *ap[CH], *bp[CH];
    int ak[CH], bk[CH];                        // their k in stage 0
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = tid + i * GA_THREADS;
      if constexpr (TN) {
        ak[i] = SA::row(c);
        const int col = m0 + SA::chunk(c) * EPC;
        ap[i] = col < a.Kd ? A + (size_t)(gbeg + ak[i]) * a.Kd + col : nullptr;
      } else {
        ak[i] = SA::chunk(c) * EPC;
        const int r = SA::row(c);
        int64_t row = r < mvalid ? gbeg + m0 + r : -1;
        if (a.row_src && row >= 0) {
          const int src = a.row_src[row];
          row = src < 0 || src / a.a_k >= a.a_rows ? -1 : src / a.a_k;
        }
        ap[i] = row >= 0 ? A + (size_t)row * a.Kd + ak[i] : nullptr;
      }
      if constexpr (BKC) {
        const int n = n0 + SB::row(c);
        bk[i] = SB::chunk(c) * EPC;
        bp[i] = n < a.N ? B + ((size_t)e * a.N + n) * a.Kd + bk[i] : nullptr;
      } else {
        bk[i] = SB::row(c);
        const int col = n0 + SB::chunk(c) * EPC;
        bp[i] = col < a.N ? B + ((TN ? (size_t)gbeg : (size_t)e * a.Kd) + bk[i]) * a.N + col : nullptr;
      }
    }
    struct Regs {
      i32x4_t a[CH], b[CH];
    };
    auto load = [&](Regs& r, int kt) __attribute__((always_inline)) {
      const size_t a_step = (size_t)kt * BK * (AKC ? 1 : a.Kd), b_step = (size_t)kt * BK * (BKC ? 1 : a.N);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const i32x4_t z = {0, 0, 0, 0};
        r.a[i] = r.b[i] = z;
        if (ap[i] && kt * BK + ak[i] < red) r.a[i] = load_chunk(ap[i] + a_step, a_end);
        if (bp[i] && kt * BK + bk[i] < red) r.b[i] = load_chunk(bp[i] + b_step, b_end);
      }
      if (kt == nk - 1) {  // chunks along the reduction end with it
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          if constexpr (AKC) r.a[i] = first_of_chunk(r.a[i], red - kt * BK - ak[i]);
          if constexpr (BKC) r.b[i] = first_of_chunk(r.b[i], red - kt * BK - bk[i]);
        }
      }
    };
    typename EL::acc_t acc[W][W];
#pragma unroll
    for (int mt = 0; mt < W; ++mt)
#pragma unroll
      for (int nt = 0; nt < W; ++nt)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[mt][nt][i] = 0;
    Regs regs[PD];
#pragma unroll
    for (int p = 0; p < PD; ++p)
      if (p < nk) load(regs[p], p);
    __syncthreads();  // the last tile's reads are done
    for (int k0 = 0; k0 < nk; k0 += PD) {
#pragma unroll
      for (int p = 0; p < PD; ++p) {
        const int kt = k0 + p;
        if (kt >= nk) break;
        unsigned char* st = smem + (kt & 1) * STAGE;  // its readers of stage kt - 2 all passed the barrier of kt - 1
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          *reinterpret_cast<i32x4_t*>(st + (tid + i * GA_THREADS) * 16) = regs[p].a[i];
          *reinterpret_cast<i32x4_t*>(st + T * 128 + (tid + i * GA_THREADS) * 16) = regs[p].b[i];
        }
        __syncthreads();
        if (kt + PD < nk) load(regs[p], kt + PD);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          i32x4_t fa[W], fb[W];
#pragma unroll
          for (int mt = 0; mt < W; ++mt) fa[mt] = SA::frag(st, a_base, mt, kk, lane);
#pragma unroll
          for (int nt = 0; nt < W; ++nt) fb[nt] = SB::frag(st + T * 128, b_base, nt, kk, lane);
#pragma unroll
          for (int mt = 0; mt < W; ++mt)
#pragma unroll
            for (int nt = 0; nt < W; ++nt) EL::mma(acc[mt][nt], fb[nt], fa[mt]);
        }
      }
    }
#pragma unroll
    for (int mt = 0; mt < W; ++mt) {
      const int r = wm * 32 * W + mt * 32 + (lane & 31);
      const bool ok = r < mvalid;
      const size_t row = TN ? (size_t)e * a.Kd + m0 + (ok ? r : 0) : (size_t)(gbeg + m0 + (ok ? r : 0));
#pragma unroll
      for (int nt = 0; nt < W; ++nt)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int c0 = n0 + wn * 32 * W + nt * 32 + 16 * p;
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int c = c0 + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3);
            v[i] = acc[mt][nt][8 * p + i];
            if (TN && OUT_F32 && a.accumulate && ok && c < a.N) v[i] += static_cast<const float*>(a.C)[row * a.N + c];
          }
          store_run<OUT_F32>(a.C, row, a.N, c0, lane, ok, vec, v);
        }
    }
  }
}

template <bool AKC, bool BKC, bool OUT_F32, int T, int PD>
moe_status_t launch_gg_any_t(const GgArgs& a, hipStream_t s) {
  constexpr int LDS = 4 * T * 128 + (GG_MAX_E + 1 + GA_THREADS / 64) * 4;
  static std::atomic<unsigned char> lds_set[MOE_MAX_DEVICES];
  const auto kernel = &gg_any_kernel<AKC, BKC, OUT_F32, T, PD>;
  if (ensure_lds_limit(reinterpret_cast<const void*>(kernel), LDS, lds_set) != MOE_OK) return MOE_EHIP;
  constexpr int PER_CU = 160 * 1024 / LDS;
  gg_any_kernel<AKC, BKC, OUT_F32, T, PD><<<PER_CU * device_cu_count(), GA_THREADS, LDS, s>>>(a);
  return launch_status();
}

// Tiles of 128 x 128 where there are two for each CU, else of 64 x 64, us beside each other (64 / 128):
//   8 experts 2047 x 1023, 100 rows each (64 tiles of 128) 58 / 63; 64 experts, 384 rows each (1792) 447 / 284, dW 776 / 605;
//   8192 rows, 7167 x 2047 (1024) 760 / 386
template <bool AKC, bool BKC, bool OUT_F32>
moe_status_t launch_gg_any(const GgArgs& a, hipStream_t s) {
  const int64_t groups = !AKC || a.E < a.M ? a.E : a.M;
  const int64_t down = !AKC ? groups * ((a.Kd + 127) / 128) : groups + (a.M - groups) / 128;
  if (down * ((a.N + 127) / 128) < 2 * (int64_t)device_cu_count()) return launch_gg_any_t<AKC, BKC, OUT_F32, 64, 3>(a, s);
  return launch_gg_any_t<AKC, BKC, OUT_F32, 128, AKC ? 2 : 1>(a, s);
}

}  // namespace moe
