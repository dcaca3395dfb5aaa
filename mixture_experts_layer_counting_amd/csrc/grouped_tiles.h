// Tiles of the grouped products for rows of whole 16-byte words, or in fp32 of any length: both operands go
// from memory to LDS directly, two stages in turn, and within a wave the loads of the next stage and the
// fragment reads of the next step are spread between the products of this one, across the stage barrier too.
//
// A block of WM x WN waves, each with MT x NT blocks of 32 x 32. A wave's row blocks lie WM * 32 rows apart,
// so that the padded rows of a group's last tile fall on all waves alike; a wave skips the blocks that lie
// wholly past the rows.
// The next tile's first stage is loaded under the last stage of this one and waited for before the stores go
// out, so that its first products need a barrier only; the stores have until its second stage.
//
// What bounds it, 256 x 256 tiles. 8192^3: INT8 2.46 POP/s (a library's product 2.02), bf16 1.33-1.34 PFLOP/s
// in both weight orders (a library's 1.19 with the weights [K][N], 1.52 with [N][K]): the matrix cores are
// busy for 68 and 72 % of the cycles, at 1.75 GHz: the power limit. 65536 rows over 52 experts, us:
// 7168 x 2048 INT8 867 (2.2 POP/s), bf16 1650-1680 (1.16 PFLOP/s); 2048 x 7168 INT8 1030 (1.9), bf16 1730;
// gate/up INT8 1700.
// 384 rows per expert (64 experts, 2048 x 1024, operands read again): bf16 122 us (419 MB, 3.4 TB/s), INT8 62.
// They make two tiles of 192 rows, of whose four row-waves two have one block instead of two: a quarter of
// the matrix cores' time is empty.
// dW: 65536 rows over 52 experts, 2048 x 7168 2.0 ms; without its 3 GB of stores 1.55: the tile's 256 KB
// leave its CU at the rate at which all CUs together fill the memory (5.5 TB/s), and its waves' loads wait
// behind them (one counter counts both, in order). Two blocks of 256 x 128 with half the stage, one computing
// while the other stores: 2.27; blocks started out of phase: no change.
#pragma once

#include "grouped_gemm.h"

namespace moe {

constexpr int GT_PANEL = 8;
constexpr int GT_OUT = (int)0x80000000u;  // an offset past every range: loads zeros

// A 32 x 32 block of fp32 whose lane l holds row l % 32 and, in v[4 j + c], column 8 j + 4 (l / 32) + c, to
// rows of whole 16-byte words, turned through 4.5 KB of LDS that no other wave uses: eight lanes then hold
// the 128 bytes of a row. `rows`: how many of the 32 there are; p: the first one's first column; `left`:
// columns from there on. All lanes must be active.
// A store then writes whole lines, 1 KB in all: dW, 64 experts of 384 rows, 2048 x 1024 188 -> 179 us beside
// a column per lane and 4 bytes (64 rows over 64 experts, nothing but stores, 97 -> 102).
// PAST: the stores ask the caches not to keep them. For weight gradients, which outgrow the caches and are
// read much later, where rows are whole lines (us, kept / past, operands read again): 64 experts 2048 x 1024
// 179 / 152, 8 of 4096 x 4096 307 / 275, 52 of 2048 x 7168 2059 / 2019; rows that share lines the other way,
// 2048 x 1000 231 / 257.
constexpr int GT_TURN = 32 * 144;  // rows of 128 bytes, 16 apart: neighbours begin on other banks
template <bool PAST>
__device__ __forceinline__ void store_turned(unsigned char* turn, float* p, int N, int rows, int left, int lane, bool add,
                                             const float (&v)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<f32x4_t*>(turn + (lane & 31) * 144 + 32 * j + 16 * (lane >> 5)) =
        f32x4_t{v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]};
  const int c = 4 * (lane & 7);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + (lane >> 3);
    f32x4_t u = *reinterpret_cast<const f32x4_t*>(turn + r * 144 + 4 * c);
    if (r < rows && c < left) {
      f32x4_t* to = reinterpret_cast<f32x4_t*>(p + (size_t)r * N + c);
      if (add) u += *to;
      if constexpr (PAST) __builtin_nontemporal_store(u, to);
      else *to = u;
    }
  }
}

// DW: rows of any length, loaded by the dword (a quarter of the bytes per wave load).
template <class EL, int WM_, int WN_, int MT_, int NT_, int NS_ = 2, bool DW_ = false>
struct GtCfg {
  static constexpr int WM = WM_, WN = WN_, MT = MT_, NT = NT_;
  static constexpr int NS = NS_;  // stages in LDS
  static constexpr bool DW = DW_;
  static constexpr int W = WM * WN, THREADS = 64 * W;
  static constexpr int BM = WM * MT * 32, BN = WN * NT * 32;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128, STAGE = A_BYTES + B_BYTES;
  static constexpr int LOAD = DW ? 256 : 1024;                     // bytes of a wave load
  static constexpr int LDA = A_BYTES / (LOAD * W), LDB = B_BYTES / (LOAD * W);
  static constexpr bool SCALED = std::is_same<EL, ElI8>::value;
  // scales of a tile's rows and columns, twice (gated: both matrices' columns, in runs of 64 at least)
  static constexpr int SC_WAVES = SCALED ? (BM + (BN > 128 ? BN : 128)) / 64 : 0;
  static constexpr int SC_BYTES = SC_WAVES * 256;
  static constexpr int SC_LD = (SC_WAVES + W - 1) / W;
  static constexpr int SCHED = NS * STAGE + 2 * SC_BYTES;
  static constexpr int LDS = SCHED + (GG_MAX_E + 1 + W) * 4;
  static_assert(BM % (8 * W) == 0 && BN % (8 * W) == 0 && (4 * W) % 8 == 0, "whole wave loads, one swizzle per lane");
  static_assert(BM % 64 == 0 && (NS - 2) * (LDA + LDB) <= 63, "whole wave loads of scales; waits count to 63");
  static_assert(!DW || EL::BYTES == 4, "a dword is an element");
  static_assert(LDS <= 160 * 1024, "LDS budget");
};

template <class EL, bool AKC, bool BKC, bool OUT_F32, bool GATED, class CF, bool PAST = false>
__global__ __launch_bounds__(CF::THREADS, 2) void gg_tile_kernel(GgArgs a) {
  constexpr bool TN = !AKC;
  constexpr int W = CF::W, BM = CF::BM, MT = CF::MT, NT = CF::NT;
  constexpr int BN = GATED ? CF::BN / 2 : CF::BN;  // columns per matrix
  constexpr int SCN = BN < 64 ? 64 : BN;           // and their places among the scales
  constexpr int NS = CF::NS;
  // fp32 gradients whose rows are not whole words leave with a column per lane, 128 neighbouring bytes of two
  // rows a store
  constexpr bool COL_LANES = TN && CF::DW;
  static_assert(W * GT_TURN <= CF::STAGE, "a wave's share of a stage");
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
  // Round by round, the blocks of an XCD take neighbouring tiles. The last round, which may have fewer tiles
  // than blocks, gives each XCD an eighth of them; where at most one whole round went before and tiles are
  // left for half of the blocks or fewer, they are cut along the rows into two or four parts, one a block.
  // Dense INT8, 7168 reduction, us: 6000 x 2048 (192 tiles of 256 x 256) 99 -> 84, 8000 x 2304 (288) 162 ->
  // 142; bf16, 8 experts of 512 rows, 2048 x 1024 35 -> 27. Cut after more rounds it costs more than it
  // gives, as the clock rises while few CUs work: 65536 rows over 52 experts (2080) 867 -> 886.
  const int slot = xcd_slot(blockIdx.x, G);
  const int whole = total / G * G, rest_tiles = total - whole;
  constexpr int MOST = TN ? 1 : BM / 64;
  const int cut = whole > G ? 1 : rest_tiles * 4 <= G && MOST >= 4 ? 4 : rest_tiles * 2 <= G && MOST >= 2 ? 2 : 1;
  const int end = whole + rest_tiles * cut;
  // the tile of the last round: each XCD an eighth of them, neighbours again
  const int per = (rest_tiles * cut + 7) / 8;
  const int last = whole + (G % 8 ? (int)blockIdx.x : (int)blockIdx.x / 8 < per ? (int)(blockIdx.x % 8) * per + (int)blockIdx.x / 8 : G);
  const int first_tile = slot < whole ? slot : last;
  auto next_tile = [&](int t) __attribute__((always_inline)) { return t >= whole ? end : t + G < whole ? t + G : last; };
  const uint32_t lds0 = lds_addr(smem);
  const int pitch = Kd * ES, npitch = N * ES;  // bytes of a KC row, of an MC row of B (and pitch: of A, TN)

  // Wave load j = wave + W i fills chunks 64 j to 64 j + 63 of an operand's stage (DW: those dwords).
  auto chunk_of = [&](int i) __attribute__((always_inline)) {
    return CF::DW ? (wave + W * i) * 16 + (lane >> 2) : (wave + W * i) * 64 + lane;
  };
  const int sub = CF::DW ? (lane & 3) * 4 : 0;
  // byte along the row; whole words of a KC operand: the same for every i
  auto a_byte = [&](int i) __attribute__((always_inline)) { return SA::chunk(chunk_of(AKC && !CF::DW ? 0 : i)) * 16 + sub; };
  auto b_byte = [&](int i) __attribute__((always_inline)) { return SB::chunk(chunk_of(BKC && !CF::DW ? 0 : i)) * 16 + sub; };
  int a_row[CF::LDA], b_off[CF::LDB];
#pragma unroll
  for (int i = 0; i < CF::LDA; ++i) a_row[i] = SA::row(chunk_of(i));
#pragma unroll
  for (int i = 0; i < CF::LDB; ++i) {
    const int r = SB::row(chunk_of(i));
    b_off[i] = BKC ? (GATED ? r % BN : r) * pitch + b_byte(i) : r * npitch + b_byte(i);
  }
  auto lds_dma = [&](i32x4_t rsrc, uint32_t to, int voff, int soff) __attribute__((always_inline)) {
    if constexpr (CF::DW) lds_dma4(rsrc, to, voff, soff);
    else lds_dma16(rsrc, to, voff, soff);
  };

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
    int mtile, ntile, part = 0, parts = 1;
    if (t >= whole && cut > 1) {
      parts = cut;
      part = (t - whole) % cut;
      t = whole + (t - whole) / cut;
    }
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
      // eight row tiles under one column tile, then the next column tile: the blocks of an XCD share rows and
      // columns
      const int panel = lt / (GT_PANEL * ntn), in_panel = lt - panel * GT_PANEL * ntn;
      const int deep = min(GT_PANEL, mte - panel * GT_PANEL);
      ntile = in_panel / deep;
      mtile = panel * GT_PANEL + in_panel - ntile * deep;
      const int chunk = even_chunk(rows_e, mte);
      const int tile_rows = min(chunk, rows_e - mtile * chunk);
      const int part_rows = ((tile_rows + parts - 1) / parts + 31) & ~31;
      d.rows_valid = uniform(max(0, min(part_rows, tile_rows - part * part_rows)));  // a part may have none
      d.row0 = uniform(d.gbeg + mtile * chunk + (d.rows_valid ? part * part_rows : 0));
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
      for (int i = 0; i < CF::LDA; ++i) d.a_off[i] = a_row[i] * pitch + a_byte(i);
    } else {
      if (a.row_src) {
        d.rA = make_rsrc(A, (uint32_t)a.a_rows * (uint32_t)pitch);
        int src[CF::LDA], ssrc[CF::SC_LD ? CF::SC_LD : 1];
#pragma unroll
        for (int i = 0; i < CF::LDA; ++i) src[i] = a.row_src[d.row0 + max(0, min(a_row[i], d.rows_valid - 1))];
#pragma unroll
        for (int i = 0; i < CF::SC_LD; ++i) ssrc[i] = a.row_src[d.row0 + max(0, min((wave + W * i) * 64 % BM + lane, d.rows_valid - 1))];
#pragma unroll
        for (int i = 0; i < CF::LDA; ++i) {
          const int at = src[i] / a.a_k;
          d.a_off[i] = a_row[i] < d.rows_valid && src[i] >= 0 && at < a.a_rows ? at * pitch + a_byte(i) : GT_OUT;
        }
#pragma unroll
        for (int i = 0; i < CF::SC_LD; ++i) {
          const int r = (wave + W * i) * 64 + lane, at = ssrc[i] / a.a_k;
          d.sc_off[i] = r < d.rows_valid && ssrc[i] >= 0 && at < a.a_rows ? at * 4 : GT_OUT;
        }
      } else {
        d.rA = make_rsrc(A + (size_t)d.row0 * pitch, (uint32_t)d.rows_valid * (uint32_t)pitch);
#pragma unroll
        for (int i = 0; i < CF::LDA; ++i) d.a_off[i] = a_row[i] < d.rows_valid ? a_row[i] * pitch + a_byte(i) : GT_OUT;
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
        const int c = ((wave + W * i) * 64 - BM + lane) % SCN;
        if ((wave + W * i) * 64 >= BM) d.sc_off[i] = c < BN && d.n0 + c < N ? c * 4 : GT_OUT;
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
      const uint32_t to = so + (wave + W * j) * CF::LOAD;
      if constexpr (AKC) {
        const bool cut = kt * 128 + a_byte(j) >= pitch;  // the row ends inside this stage
        lds_dma(d.rA, to, cut ? GT_OUT : d.a_off[j], kt * 128);
      } else {
        // the descriptor begins at this stage's first row and ends with the group: rows past it read as zeros
        const uint32_t rows = (uint32_t)min(BK, d.red - kt * BK);
        lds_dma(make_rsrc(d.pA + (size_t)kt * BK * pitch, rows * (uint32_t)pitch - (uint32_t)d.row0 * ES), to, d.a_off[j], 0);
      }
    } else if constexpr (j < PIECES) {
      constexpr int i = j - CF::LDA;
      const uint32_t to = so + CF::A_BYTES + (wave + W * i) * CF::LOAD;
      if constexpr (BKC) {
        constexpr bool second = GATED && i >= CF::LDB / 2;
        const bool cut = kt * 128 + b_byte(i) >= pitch;
        lds_dma(second ? d.rB1 : d.rB0, to, cut ? GT_OUT : b_off[i], kt * 128);
      } else {
        const uint32_t rows = (uint32_t)min(BK, d.red - kt * BK);
        lds_dma(make_rsrc(d.pB + (size_t)kt * BK * npitch, rows * (uint32_t)npitch - (uint32_t)d.n0 * ES), to, b_off[i], 0);
      }
    }
  };
  auto issue_scales = [&](const Tile& d, int par) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < CF::SC_LD; ++i) {
      const int at = (wave + W * i) * 64;
      const uint32_t to = lds0 + NS * CF::STAGE + par * CF::SC_BYTES + at * 4;
      if (at >= BM + (GATED ? 2 : 1) * SCN) break;
      if (at < BM) {
        if (a.row_src) lds_dma4(make_rsrc(a.a_sf, (uint32_t)a.a_rows * 4u), to, d.sc_off[i], 0);
        else lds_dma4(make_rsrc(a.a_sf + d.row0, (uint32_t)d.rows_valid * 4u), to, d.sc_off[i], 0);
      } else {
        const float* sf = GATED && at - BM >= SCN ? a.b_sf1 : a.b_sf0;
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

  auto after = [](int b) __attribute__((always_inline)) { return b + 1 == NS ? 0 : b + 1; };
  auto before = [](int b) __attribute__((always_inline)) { return b == 0 ? NS - 1 : b - 1; };
  int buf = 0, ahead = 1, par = 0;
  Tile cur, nxt;
  if (NS == 2 && first_tile < end) {
    cur = decode(first_tile);
    if (CF::SCALED) issue_scales(cur, par);
    if (cur.nk > 0) load_all(cur, 0, buf);
    wait_vm<0>();
  }
  for (int t = first_tile; t < end; t = next_tile(t)) {
    const bool more = next_tile(t) < end;
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
          if constexpr (COL_LANES) EL::mma(acc[mt][nt], f.a[mt], f.b[nt]);
          else EL::mma(acc[mt][nt], f.b[nt], f.a[mt]);
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
                piece(d, kt, ahead, std::integral_constant<int, per * m + decltype(i_)::value>{});
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
      // A stage: it has landed for every wave (at most `younger` loads are outstanding), and every wave has
      // read all it needs of the buffer before it, into which stage `kl` of tile d goes.
      auto stage = [&](const Tile& d, int kl, bool load, int younger) __attribute__((always_inline)) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        wait_vm_dyn<(NS - 2) * PIECES>(younger);
        asm volatile("s_barrier" ::: "memory");
        ahead = before(buf);
        if constexpr (MTV > 0) {
          const unsigned char* st = smem + buf * CF::STAGE;
          step(f1, f0, st, integral_constant<int, 0>{}, std::true_type{}, d, kl, load);
          rest(st);
        } else if (load) {
          load_all(d, kl, ahead);
        }
        buf = after(buf);
      };
      if constexpr (MTV > 0) {
        const unsigned char* st = smem + buf * CF::STAGE;
        gg_for<READS>([&](auto i_) __attribute__((always_inline)) { read_one(f0, st, integral_constant<int, 0>{}, i_); });
        rest(st);
      }
      buf = after(buf);
      const int nk = cur.nk;
      if constexpr (NS == 2) {
        for (int kt = 1; kt + 1 < nk; ++kt) stage(cur, kt + 1, true, 0);
        if (nk > 1) stage(nxt, 0, nxt_load, 0);
      } else {
        for (int kt = 1; kt < nk; ++kt) stage(cur, kt + NS - 1, kt + NS - 1 < nk, min(NS - 2, nk - 1 - kt) * PIECES);
      }
      if constexpr (MTV > 0) step(f1, f0, smem, integral_constant<int, -1>{}, std::false_type{}, cur, 0, false);
    };
    // (NS = 2: every wave waited for its loads of this tile's first stage); the last tile's reads are done
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if constexpr (NS == 2) {
      if (cur.nk > 1) load_all(cur, 1, buf ^ 1);
      if (more) {
        nxt = decode(next_tile(t));
        nxt_load = nxt.nk > 0;
        if (CF::SCALED) issue_scales(nxt, par ^ 1);
        if (nxt_load && cur.nk < 2) load_all(nxt, 0, cur.nk ? buf ^ 1 : buf);  // a longer tile: under its last stage
      }
    } else {
      // all stages that fit, and a wait for the first (the last tile's stores and the scales are older)
      cur = decode(t);
      if (CF::SCALED) issue_scales(cur, par);
      buf = 0;
      const int first = min(NS, cur.nk);
      for (int st = 0; st < first; ++st) load_all(cur, st, st);
      constexpr int MOST = (NS - 1) * PIECES < 63 ? (NS - 1) * PIECES : 63;
      wait_vm_dyn<MOST>(min((first - 1) * PIECES, MOST));
      asm volatile("s_barrier" ::: "memory");
    }
    if constexpr (TN) {
      if (cur.nk > 0) k_loop(std::integral_constant<int, MT>{});
    } else {
      static_assert(MT <= 2, "the cases below");
      if (cur.nmt == MT) k_loop(std::integral_constant<int, MT>{});
      else if (MT > 1 && cur.nmt == 1) k_loop(std::integral_constant<int, 1>{});
      else k_loop(std::integral_constant<int, 0>{});
    }
    wait_vm<0>();

    if constexpr (COL_LANES) {
      // lane l holds column l % 32 and, in acc[4 j + c], row 8 j + 4 (l / 32) + c
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int col = cur.n0 + wn * NT * 32 + nt * 32 + (lane & 31);
          const int r0 = mt * CF::WM * 32 + wm * 32 + 4 * (lane >> 5);
          float* p = static_cast<float*>(a.C) + ((size_t)cur.e * Kd + cur.row0 + r0) * N + col;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int dr = 8 * (i >> 2) + (i & 3);
            if (col < N && r0 + dr < cur.rows_valid) {
              float v = acc[mt][nt][i];
              if (a.accumulate) v += p[(size_t)dr * N];
              p[(size_t)dr * N] = v;
            }
          }
        }
      if (NS == 2) cur = nxt;
      par ^= 1;
      continue;
    }
    const float* sc = reinterpret_cast<const float*>(smem + NS * CF::STAGE + par * CF::SC_BYTES);
    // the stage that is not the next tile's first, once every wave has read it
    unsigned char* turn = smem + (NS == 2 ? buf ^ 1 : 0) * CF::STAGE + wave * GT_TURN;
    if (OUT_F32 && vec) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
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
        if constexpr (OUT_F32) {
          if (vec) {
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              v[i] = (float)acc[mt][nt][i];
              if constexpr (CF::SCALED) {  // a padding row is zeros whatever the weights' scales hold
                v[i] = v[i] * sa * sc[BM + cw + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3)];
                if (sa == 0.f) v[i] = 0.f;
              }
            }
            const size_t row0 = (TN ? (size_t)cur.e * Kd : 0) + cur.row0 + (r - (lane & 31));
            store_turned<PAST>(turn, static_cast<float*>(a.C) + row0 * N + cur.n0 + cw, N, cur.rows_valid - (r - (lane & 31)),
                         N - cur.n0 - cw, lane, TN && a.accumulate, v);
            continue;
          }
        }
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          float v[8];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            f32x4_t s0, s1;
            const int cl = cw + 16 * p + 8 * h + 4 * (lane >> 5);
            if constexpr (CF::SCALED) {
              s0 = *reinterpret_cast<const f32x4_t*>(sc + BM + cl);
              if constexpr (GATED) s1 = *reinterpret_cast<const f32x4_t*>(sc + BM + SCN + cl);
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
    if (NS == 2) cur = nxt;
    par ^= 1;
  }
}

// The forms of the kernel: 256 x 256 by eight waves; 128 x 128 by four, two blocks a CU; 128 x 64 by four
// with four stages in LDS, for products whose tiles are so few that the loads' latency counts.
// (Large with two waves down and four across, which halves the rows a wave may skip, took 1.5-2.5 % longer on
// every shape: INT8, 65536 rows over 52 experts, 7168 x 2048 883 us beside 863.)
template <class EL>
using GtLarge = GtCfg<EL, 4, 2, 2, 4>;
template <class EL>
using GtSmall = GtCfg<EL, 2, 2, 2, 2>;
template <class EL>
using GtThin = GtCfg<EL, 4, 1, 1, 2, 4>;
// fp32 rows of any length. (Large has no registers left for four times the offsets.)
using GtSmallDw = GtCfg<ElF32, 2, 2, 2, 2, 2, true>;
using GtThinDw = GtCfg<ElF32, 4, 1, 1, 2, 4, true>;

enum GgForm { GG_STREAM, GG_THIN, GG_SMALL, GG_LARGE };

// Which kernel takes a product whose rows are whole 16-byte words, from the number of 128 x 64 tiles (`thin`;
// of both matrices where gated) and the rows per group. Measured on 256 CUs, us, stream / thin / small /
// large, rows per group in brackets:
//   INT8, dense 7168 x 2048 (32 thin tiles): [1] 7.5 / 23 / 35 / 50  [16] 10 / 23 / 36 / 50  [64] 16 / 23 / 38 / 54
//     [128] 30 / 25 / 43 / 54  [2048, 512 tiles] - / 50 / 58 / 99  [4096] - / 130 / 62 / 103
//   INT8, 8 experts 7168 x 2048 (256): [1] 22 / 24 / 49 / 57  [8] 25 / 24 / 49 / 57  [16] 32 / 25 / 50 / 57
//     [128] 200 / 27 / 62 / 67
//   bf16 [N][K], the same: [1] 39 / 42 / 92 / 104  [8] 44 / 42 / 92 / 105  [16] 58 / 43 / 92 / 105
//   bf16 [N][K], 16 experts 1024 x 512 (128): [16] 7 / 9 / 17 / 19
//   INT8 gate/up, the same (512): [1] 40 / 49 / 63 / 67  [8] 47 / 49 / 63 / 67  [16] 57 / 49 / 64 / 67
//   INT8, 8 experts 2048 x 7168 (896): [1] 25 / 34 / 22 / 24  [16] 35 / 33 / 23 / 25
//   bf16 [K][N], 8 experts 7168 x 2048 (256): [1] 37 / 44 / 93 / 103  [16] 39 / 44 / 94 / 102  [128] 158 / 48 / 110 / 115
//   bf16 [K][N], 16 experts 1024 x 512 (128): [1] 6.8 / 9.6 / 17 / 18  [16] 7.3 / 9.8 / 18 / 19  [64] 11 / 10 / 20 / 21
//   bf16 [K][N], 64 experts 2048 x 1024 (1024): [32] 66 / 56 / 44 / 47  [128] 220 / 80 / 58 / 60  [384] - / - / 148 / 122
//   fp32 [K][N], 8 experts 7168 x 2048 (256): [16] 89 / 260 / 425 / 458  [32] 141 / 260 / 429 / 463  [64] 251 / 262 / 433 / 467
//   fp32 [K][N], 64 experts 2048 x 1024 (1024): [1] 98 / 303 / 128 / 139  [16] 102 / 303 / 129 / 140
//   dW, 64 experts 2048 x 24 (384 rows; 1024): - / 22 / 22 / 28, 24 x 2048 (2048): - / 38 / 23 / 34
//   dW in fp32, 64 experts 2047 x 23 (by the dword): - / 79 / 112
//   dW, one expert 1024 x 1024 (8192 rows; 128): - / 50 / 87 / 150, 7168 x 2048 (1792): - / 352 / 243 / 204
// (weights [N][K], whose rows x come with every 16 columns, stop streaming earlier: `kc`)
inline GgForm gg_form(const GgArgs& a, bool tn, bool kc, bool f32, int columns) {
  const int64_t cus = device_cu_count();
  const int64_t slots = tn || a.E < a.M ? a.E : a.M;  // at most so many groups have rows
  auto tiles = [&](int bm, int bn) -> int64_t {
    const int64_t down = tn ? slots * ((a.Kd + bm - 1) / bm) : slots + (a.M - slots) / bm;
    return down * ((columns + bn - 1) / bn);
  };
  const int64_t thin = tiles(128, 64);
  if (!tn) {
    if (a.M <= 16 * slots && (f32 ? thin <= 4 * cus : (kc ? 2 : 1) * thin <= cus)) return GG_STREAM;
    if (a.M <= 8 * slots && thin <= 2 * cus) return GG_STREAM;
    if (a.M <= 32 * slots && (f32 ? 1 : 4) * thin <= cus) return GG_STREAM;
    if (a.M <= 64 * slots && 8 * thin <= cus) return GG_STREAM;
  }
  if (thin <= 2 * cus || columns <= 64) return GG_THIN;
  return !(tn && a.Kd <= 64) && (tn || a.M > 128 * slots) && 4 * tiles(256, 256) >= 3 * cus ? GG_LARGE : GG_SMALL;
}

template <class EL, bool AKC, bool BKC, bool OUT_F32, bool GATED, class CF, bool PAST = false>
moe_status_t launch_gg_tiles(const GgArgs& a, hipStream_t s) {
  if constexpr (!AKC && OUT_F32 && !CF::DW && !PAST) {
    // weight gradients whose rows are whole lines
    if (a.N % 32 == 0 && reinterpret_cast<uintptr_t>(a.C) % 128 == 0)
      return launch_gg_tiles<EL, AKC, BKC, OUT_F32, GATED, CF, true>(a, s);
  }
  static std::atomic<unsigned char> lds_set[MOE_MAX_DEVICES];
  const auto kernel = &gg_tile_kernel<EL, AKC, BKC, OUT_F32, GATED, CF, PAST>;
  if (ensure_lds_limit(reinterpret_cast<const void*>(kernel), CF::LDS, lds_set) != MOE_OK) return MOE_EHIP;
  constexpr int PER_CU = 160 * 1024 / CF::LDS < 1024 / CF::THREADS ? 160 * 1024 / CF::LDS : 1024 / CF::THREADS;
  gg_tile_kernel<EL, AKC, BKC, OUT_F32, GATED, CF, PAST><<<PER_CU * device_cu_count(), CF::THREADS, CF::LDS, s>>>(a);
  return launch_status();
}

}  // namespace moe
