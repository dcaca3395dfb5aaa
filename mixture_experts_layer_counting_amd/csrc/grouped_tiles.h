// Tiles of the grouped products for rows of whole 16-byte words: both operands go from memory to LDS directly, two stages in
// turn, and within a wave the loads of the next stage and the fragment reads of the next step are spread between
// the products of this one, across the stage barrier too.
//
// A block of WM x WN waves, each with MT x NT blocks of 32 x 32. A wave's row blocks lie WM * 32 rows apart, so that
// the padded rows of a group's last tile fall on all waves alike; a wave skips the blocks that lie wholly past the rows.
// The persistent loop never waits for its stores: the next tile's first stage is loaded under the last stage of
// this one and waited for before the stores go out, so its first products need the barrier only.
#pragma once

#include "grouped_gemm.h"

namespace moe {

constexpr int GT_OUT = (int)0x80000000u;  // an offset past every range: loads zeros

template <class EL, int WM_, int WN_, int MT_, int NT_>
struct GtCfg {
  static constexpr int WM = WM_, WN = WN_, MT = MT_, NT = NT_;
  static constexpr int W = WM * WN, THREADS = 64 * W;
  static constexpr int BM = WM * MT * 32, BN = WN * NT * 32;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128, STAGE = A_BYTES + B_BYTES;
  static constexpr int LDA = BM / (8 * W), LDB = BN / (8 * W);  // wave loads per stage
  static constexpr bool SCALED = std::is_same<EL, ElI8>::value;
  static constexpr int SC_BYTES = SCALED ? (BM + BN) * 4 : 0;   // scales of a tile's rows and columns, twice
  static constexpr int SC_LD = SCALED ? (BM + BN) / 64 / W : 0;
  static constexpr int SCHED = 2 * STAGE + 2 * SC_BYTES;
  static constexpr int LDS = SCHED + (GG_MAX_E + 1 + W) * 4;
  static_assert(BM % (8 * W) == 0 && BN % (8 * W) == 0 && (4 * W) % 8 == 0, "whole wave loads, one swizzle per lane");
  static_assert(!SCALED || ((BM + BN) / 64 % W == 0 && BM % (64 * 1) == 0), "whole wave loads of scales");
  static_assert(LDS <= 160 * 1024, "LDS budget");
};

template <class EL, bool AKC, bool BKC, bool OUT_F32, bool GATED, class CF>
__global__ __launch_bounds__(CF::THREADS, 2) void gg_tile_kernel(GgArgs a) {
  constexpr bool TN = !AKC;
  constexpr int W = CF::W, BM = CF::BM, MT = CF::MT, NT = CF::NT;
  constexpr int BN = GATED ? CF::BN / 2 : CF::BN;  // columns per matrix
  using SA = Staged<EL, AKC, BM>;
  using SB = Staged<EL, BKC, CF::BN>;
  constexpr int BK = SA::BK, ES = EL::BYTES;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  int* tstart = reinterpret_cast<int*>(smem + CF::SCHED);
  int* wsum = tstart + GG_MAX_E + 1;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / CF::WN, wn = wave % CF::WN;
  const int N = a.N, Kd = a.Kd;
  const int ntn = (N + BN - 1) / BN;
  const int mtn = (Kd + BM - 1) / BM;  // TN: row tiles of dW
  int total;
  if constexpr (TN) total = a.E * mtn * ntn;
  else total = group_prefix<CF::THREADS>(a.cu, a.M, a.E, [&](int rows) { return (rows + BM - 1) / BM * ntn; }, tstart, wsum);
  const int G = gridDim.x;
  const int slot = xcd_slot(blockIdx.x, G);
  const uint32_t lds0 = lds_addr(smem);
  const int pitch = Kd * ES, npitch = N * ES;  // bytes of a KC row, of an MC row of B (and pitch: of A, TN)

  // Wave load j = wave + W i fills chunks 64 j .. 64 j + 63 of an operand's stage.
  int a_row[CF::LDA], b_off[CF::LDB];
#pragma unroll
  for (int i = 0; i < CF::LDA; ++i) a_row[i] = SA::row((wave + W * i) * 64 + lane);
  const int a_chunk = SA::chunk(wave * 64 + lane);  // KC: the same for every i
#pragma unroll
  for (int i = 0; i < CF::LDB; ++i) {
    const int c = (wave + W * i) * 64 + lane;
    const int r = SB::row(c);
    if constexpr (BKC) b_off[i] = (GATED ? r % BN : r) * pitch + SB::chunk(c) * 16;
    else b_off[i] = r * npitch + SB::chunk(c) * 16;
  }
  const int b_chunk = SB::chunk(wave * 64 + lane);

  struct Tile {
    int e, gbeg, row0, rows_valid, n0, nmt, nk, red;
    i32x4_t rA, rB0, rB1;        // KC operands
    int a_off[CF::LDA];
    const unsigned char *pA, *pB;  // MC operands: the first stage's first byte
    int sc_off[CF::SC_LD ? CF::SC_LD : 1];
  };
  auto uniform = [](int v) __attribute__((always_inline)) { return __builtin_amdgcn_readfirstlane(v); };
  auto decode = [&](int t) __attribute__((always_inline)) {
    Tile d;
    int mtile, ntile;
    if constexpr (TN) {
      const int per_e = mtn * ntn;
      d.e = uniform(t / per_e);
      const int rem = t - d.e * per_e;
      mtile = rem / ntn;
      ntile = rem - mtile * ntn;
    } else {
      d.e = uniform(find_expert(tstart, a.E, t));
    }
    d.gbeg = uniform(group_begin(a.cu, d.e, a.M));
    const int rows_e = uniform(group_rows(a.cu, d.e, a.M, d.gbeg));
    if constexpr (TN) {
      d.row0 = uniform(mtile * BM);                  // first row of dW
      d.rows_valid = uniform(min(BM, Kd - d.row0));
      d.red = rows_e;
    } else {
      const int lt = t - tstart[d.e];
      const int mte = (rows_e + BM - 1) / BM;
      ntile = lt / mte;
      mtile = lt - ntile * mte;
      const int chunk = even_chunk(rows_e, mte);
      d.row0 = uniform(d.gbeg + mtile * chunk);
      d.rows_valid = uniform(min(chunk, rows_e - mtile * chunk));
      d.red = Kd;
    }
    d.n0 = uniform(ntile * BN);
    d.nk = uniform((d.red + BK - 1) / BK);
    d.nmt = 0;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) d.nmt += mt * CF::WM * 32 + wm * 32 < d.rows_valid;
    d.nmt = uniform(d.nmt);
    const unsigned char* A = static_cast<const unsigned char*>(a.A);
    if constexpr (TN) {
      d.pA = A + ((size_t)d.gbeg * Kd + d.row0) * ES;
      d.pB = static_cast<const unsigned char*>(a.B0) + ((size_t)d.gbeg * N + d.n0) * ES;
#pragma unroll
      for (int i = 0; i < CF::LDA; ++i) d.a_off[i] = a_row[i] * pitch + SA::chunk((wave + W * i) * 64 + lane) * 16;
    } else {
      if (a.row_src) {
        d.rA = make_rsrc(A, (uint32_t)a.a_rows * (uint32_t)pitch);
        int src[CF::LDA], ssrc[CF::SC_LD ? CF::SC_LD : 1];
#pragma unroll
        for (int i = 0; i < CF::LDA; ++i) src[i] = a.row_src[d.row0 + min(a_row[i], d.rows_valid - 1)];
#pragma unroll
        for (int i = 0; i < CF::SC_LD; ++i) ssrc[i] = a.row_src[d.row0 + min((wave + W * i) * 64 % BM + lane, d.rows_valid - 1)];
#pragma unroll
        for (int i = 0; i < CF::LDA; ++i) {
          const int at = src[i] / a.a_k;
          d.a_off[i] = a_row[i] < d.rows_valid && src[i] >= 0 && at < a.a_rows ? at * pitch + a_chunk * 16 : GT_OUT;
        }
#pragma unroll
        for (int i = 0; i < CF::SC_LD; ++i) {
          const int r = (wave + W * i) * 64 + lane, at = ssrc[i] / a.a_k;
          d.sc_off[i] = r < d.rows_valid && ssrc[i] >= 0 && at < a.a_rows ? at * 4 : GT_OUT;
        }
      } else {
        d.rA = make_rsrc(A + (size_t)d.row0 * pitch, (uint32_t)d.rows_valid * (uint32_t)pitch);
#pragma unroll
        for (int i = 0; i < CF::LDA; ++i) d.a_off[i] = a_row[i] < d.rows_valid ? a_row[i] * pitch + a_chunk * 16 : GT_OUT;
#pragma unroll
        for (int i = 0; i < CF::SC_LD; ++i) {
          const int r = (wave + W * i) * 64 + lane;
          d.sc_off[i] = r < d.rows_valid ? r * 4 : GT_OUT;
        }
      }
      if constexpr (BKC) {
        const size_t wbase = ((size_t)d.e * N + d.n0) * pitch;
        const uint32_t range = (uint32_t)min(N - d.n0, BN) * (uint32_t)pitch;
        d.rB0 = make_rsrc(static_cast<const unsigned char*>(a.B0) + wbase, range);
        if constexpr (GATED) d.rB1 = make_rsrc(static_cast<const unsigned char*>(a.B1) + wbase, range);
      } else {
        d.pB = static_cast<const unsigned char*>(a.B0) + ((size_t)d.e * Kd * N + d.n0) * ES;
      }
      // scales: rows then columns; a column's offset goes from the tile's first one
#pragma unroll
      for (int i = 0; i < CF::SC_LD; ++i) {
        const int c = (wave + W * i) * 64 - BM + lane;
        if ((wave + W * i) * 64 >= BM) d.sc_off[i] = d.n0 + (GATED ? c % BN : c) < N ? (GATED ? c % BN : c) * 4 : GT_OUT;
      }
    }
    return d;
  };
  // Piece j of this wave's loads of stage kt into buffer buf: A, then B.
  constexpr int PIECES = CF::LDA + CF::LDB;
  auto piece = [&](const Tile& d, int kt, int buf, auto j_) __attribute__((always_inline)) {
    constexpr int j = decltype(j_)::value;
    const uint32_t so = lds0 + (uint32_t)buf * CF::STAGE;
    if constexpr (j < CF::LDA) {
      const uint32_t to = so + (wave + W * j) * 1024;
      if constexpr (AKC) {
        const bool cut = kt * 128 + a_chunk * 16 >= pitch;  // the row ends inside this stage
        lds_dma16(d.rA, to, cut ? GT_OUT : d.a_off[j], kt * 128);
      } else {
        // the descriptor begins at this stage's first row and ends with the group: rows past it read as zeros
        const uint32_t rows = (uint32_t)min(BK, d.red - kt * BK);
        lds_dma16(make_rsrc(d.pA + (size_t)kt * BK * pitch, rows * (uint32_t)pitch - (uint32_t)d.row0 * ES), to, d.a_off[j], 0);
      }
    } else if constexpr (j < PIECES) {
      constexpr int i = j - CF::LDA;
      const uint32_t to = so + CF::A_BYTES + (wave + W * i) * 1024;
      if constexpr (BKC) {
        constexpr bool second = GATED && i >= CF::LDB / 2;
        const bool cut = kt * 128 + b_chunk * 16 >= pitch;
        lds_dma16(second ? d.rB1 : d.rB0, to, cut ? GT_OUT : b_off[i], kt * 128);
      } else {
        const uint32_t rows = (uint32_t)min(BK, d.red - kt * BK);
        lds_dma16(make_rsrc(d.pB + (size_t)kt * BK * npitch, rows * (uint32_t)npitch - (uint32_t)d.n0 * ES), to, b_off[i], 0);
      }
    }
  };
  auto issue_scales = [&](const Tile& d, int par) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < CF::SC_LD; ++i) {
      const int at = (wave + W * i) * 64;
      const uint32_t to = lds0 + 2 * CF::STAGE + par * CF::SC_BYTES + at * 4;
      if (at < BM) {
        if (a.row_src) lds_dma4(make_rsrc(a.a_sf, (uint32_t)a.a_rows * 4u), to, d.sc_off[i], 0);
        else lds_dma4(make_rsrc(a.a_sf + d.row0, (uint32_t)d.rows_valid * 4u), to, d.sc_off[i], 0);
      } else {
        const float* sf = GATED && at - BM >= BN ? a.b_sf1 : a.b_sf0;
        lds_dma4(make_rsrc(sf + (size_t)d.e * N + d.n0, (uint32_t)(N - d.n0) * 4u), to, d.sc_off[i], 0);
      }
    }
  };

  auto load_all = [&](const Tile& d, int kt, int to) __attribute__((always_inline)) {
    gg_for<PIECES>([&](auto j_) __attribute__((always_inline)) { piece(d, kt, to, j_); });
  };

  const int a_base = SA::base(wm * 32, lane);
  const int b_base = SB::base(wn * (GATED ? NT / 2 : NT) * 32, lane);
  const bool vec = whole_words<OUT_F32>(a.C, N);

  int buf = 0, par = 0;
  Tile cur, nxt;
  if (slot < total) {
    cur = decode(slot);
    if (CF::SCALED) issue_scales(cur, par);
    if (cur.nk > 0) load_all(cur, 0, buf);
    wait_vm<0>();
  }
  for (int t = slot; t < total; t += G) {
    const bool more = t + G < total;
    bool nxt_load = false;
    typename EL::acc_t acc[MT][NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[mt][nt][i] = 0;

    // The K loop over the first MTV row blocks of this wave.
    auto k_loop = [&](auto mtv) {
      constexpr int MTV = decltype(mtv)::value;
      constexpr int MR = MTV ? MTV : 1;
      struct Frag {
        i32x4_t a[MR], b[NT];
      };
      Frag f0, f1;
      constexpr int READS = MTV + NT;
      auto read_one = [&](Frag& f, const unsigned char* st, auto kk_, auto i_) __attribute__((always_inline)) {
        constexpr int i = decltype(i_)::value, kk = decltype(kk_)::value;
        if constexpr (i < MTV) {
          f.a[i] = SA::frag(st, a_base, i * CF::WM, kk, lane);
        } else if constexpr (i < READS) {
          constexpr int nt = i - MTV;
          constexpr int at = GATED ? nt % (NT / 2) + nt / (NT / 2) * (BN / 32) : nt;
          f.b[nt] = SB::frag(st + CF::A_BYTES, b_base, at, kk, lane);
        }
      };
      // The products of step kk, with the reads of the next spread between them and, with LOAD, the loads of
      // stage kt of tile d where `load`: a wave that issued them in a row would hold up its matrix core.
      auto step = [&](const Frag& f, Frag& next, const unsigned char* st, auto next_, auto load_, const Tile& d, int kt,
                      bool load) __attribute__((always_inline)) {
        constexpr int kk_next = decltype(next_)::value;  // < 0: none
        constexpr bool LOAD = decltype(load_)::value;
        constexpr int PRODUCTS = NT * MR;
        gg_for<PRODUCTS>([&](auto m_) __attribute__((always_inline)) {
          constexpr int m = decltype(m_)::value;
          constexpr int mt = m % MR, nt = m / MR;
          EL::mma(acc[mt][nt], f.b[nt], f.a[mt]);
          __builtin_amdgcn_sched_barrier(0);
          if constexpr (kk_next >= 0) {
            constexpr int per = (READS + PRODUCTS - 1) / PRODUCTS;
            gg_for<per>([&](auto i_) __attribute__((always_inline)) {
              read_one(next, st, std::integral_constant<int, kk_next>{}, std::integral_constant<int, per * m + decltype(i_)::value>{});
            });
          }
          if constexpr (LOAD) {
            constexpr int per = (PIECES + PRODUCTS - 1) / PRODUCTS;
            if (load)
              gg_for<per>([&](auto i_) __attribute__((always_inline)) {
                piece(d, kt, buf ^ 1, std::integral_constant<int, per * m + decltype(i_)::value>{});
              });
          }
          __builtin_amdgcn_sched_barrier(0);
        });
      };
      using std::integral_constant;
      auto rest = [&](const unsigned char* st) __attribute__((always_inline)) {
        step(f0, f1, st, integral_constant<int, 1>{}, std::false_type{}, cur, 0, false);
        step(f1, f0, st, integral_constant<int, 2>{}, std::false_type{}, cur, 0, false);
        step(f0, f1, st, integral_constant<int, 3>{}, std::false_type{}, cur, 0, false);
      };
      // Stage kt: it has landed for every wave, and every wave has read all it needs of the other buffer, into which stage
      // `kl` of tile d goes.
      auto stage = [&](const Tile& d, int kl, bool load) __attribute__((always_inline)) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        wait_barrier<0>();
        if constexpr (MTV > 0) {
          const unsigned char* st = smem + buf * CF::STAGE;
          step(f1, f0, st, integral_constant<int, 0>{}, std::true_type{}, d, kl, load);
          rest(st);
        } else if (load) {
          load_all(d, kl, buf ^ 1);
        }
        buf ^= 1;
      };
      if constexpr (MTV > 0) {
        const unsigned char* st = smem + buf * CF::STAGE;
        gg_for<READS>([&](auto i_) __attribute__((always_inline)) { read_one(f0, st, integral_constant<int, 0>{}, i_); });
        rest(st);
      }
      buf ^= 1;
      const int nk = cur.nk;
      for (int kt = 1; kt + 1 < nk; ++kt) stage(cur, kt + 1, true);
      if (nk > 1) stage(nxt, 0, nxt_load);
      if constexpr (MTV > 0) step(f1, f0, smem, integral_constant<int, -1>{}, std::false_type{}, cur, 0, false);
    };
    // every wave waited for its loads of this tile's first stage; the reads of the last tile's are done
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (cur.nk > 1) load_all(cur, 1, buf ^ 1);
    if (more) {
      nxt = decode(t + G);
      nxt_load = nxt.nk > 0;
      if (CF::SCALED) issue_scales(nxt, par ^ 1);
      if (nxt_load && cur.nk < 2) load_all(nxt, 0, cur.nk ? buf ^ 1 : buf);  // a longer tile: under its last stage
    }
    if constexpr (TN) {
      if (cur.nk > 0) k_loop(std::integral_constant<int, MT>{});
    } else {
      static_assert(MT <= 2, "the cases below");
      if (MT == 2 && cur.nmt == 2) k_loop(std::integral_constant<int, MT>{});
      else if (cur.nmt == 1) k_loop(std::integral_constant<int, 1>{});
      else k_loop(std::integral_constant<int, 0>{});
    }
    wait_vm<0>();

    const float* sc = reinterpret_cast<const float*>(smem + 2 * CF::STAGE + par * CF::SC_BYTES);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (!TN && mt >= cur.nmt) break;
      const int r = mt * CF::WM * 32 + wm * 32 + (lane & 31);
      const bool ok = r < cur.rows_valid;
      const size_t row = (TN ? (size_t)cur.e * Kd : 0) + cur.row0 + (ok ? r : 0);
      float sa = 1.f;
      if constexpr (CF::SCALED) sa = sc[r];
#pragma unroll
      for (int nt = 0; nt < (GATED ? NT / 2 : NT); ++nt) {
        const int cw = wn * (GATED ? NT / 2 : NT) * 32 + nt * 32;  // inside the tile
        if (cur.n0 + cw >= N) break;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          float v[8];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            f32x4_t s0, s1;
            const int cl = cw + 16 * p + 8 * h + 4 * (lane >> 5);
            if constexpr (CF::SCALED) {
              s0 = *reinterpret_cast<const f32x4_t*>(sc + BM + cl);
              if constexpr (GATED) s1 = *reinterpret_cast<const f32x4_t*>(sc + BM + BN + cl);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int i = 4 * h + c;
              if constexpr (CF::SCALED) {
                float y = (float)acc[mt][nt][8 * p + i] * sa * s0[c];
                if constexpr (GATED) y = silu_f32(y) * ((float)acc[mt][nt + NT / 2][8 * p + i] * sa * s1[c]);
                v[i] = sa == 0.f ? 0.f : y;  // a padding row is zeros whatever the weights' scales hold
              } else {
                v[i] = acc[mt][nt][8 * p + i];
                if constexpr (TN && OUT_F32) {
                  const int col = cur.n0 + cl + c;
                  if (a.accumulate && ok && col < N) v[i] += static_cast<const float*>(a.C)[row * N + col];
                }
              }
            }
          }
          store_run<OUT_F32>(a.C, row, N, cur.n0 + cw + 16 * p, lane, ok, vec, v);
        }
      }
    }
    cur = nxt;
    par ^= 1;
  }
}

// Whether tiles of 256 x 256 leave CUs without one: as many groups as can have rows, evenly filled.
inline bool few_large_tiles(const GgArgs& a, bool tn, int columns) {
  const int64_t across = (columns + 255) / 256;
  const int64_t groups = a.M < a.E ? a.M : a.E;
  const int64_t tiles = tn ? (int64_t)a.E * ((a.Kd + 255) / 256) * across : (groups + (a.M - groups) / 256) * across;
  return tiles < device_cu_count();
}

template <class EL, bool AKC, bool BKC, bool OUT_F32, bool GATED, class CF>
moe_status_t launch_gg_tiles(const GgArgs& a, hipStream_t s) {
  static std::atomic<unsigned char> lds_set[MOE_MAX_DEVICES];
  const auto kernel = &gg_tile_kernel<EL, AKC, BKC, OUT_F32, GATED, CF>;
  if (ensure_lds_limit(reinterpret_cast<const void*>(kernel), CF::LDS, lds_set) != MOE_OK) return MOE_EHIP;
  constexpr int PER_CU = 160 * 1024 / CF::LDS < 1024 / CF::THREADS ? 160 * 1024 / CF::LDS : 1024 / CF::THREADS;
  gg_tile_kernel<EL, AKC, BKC, OUT_F32, GATED, CF><<<PER_CU * device_cu_count(), CF::THREADS, CF::LDS, s>>>(a);
  return launch_status();
}

}  // namespace moe
