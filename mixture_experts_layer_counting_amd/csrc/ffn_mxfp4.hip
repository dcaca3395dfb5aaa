// Grouped expert FFN with both operands in MXFP4, on gfx950's block-scaled matrix cores.
//
//   gate/up:  h = silu(x.Wg) * (x.Wu), fp32, rounded in the epilogue to MXFP4 (mxfp4.h)
//   down:     y = h.Wd, bf16
//
// MFMA v_mfma_scale_f32_32x32x64_f8f6f4 with two fp4 operands. A lane in group G = lane / 32
// holds 16 bytes, 32 consecutive k of its row (or column), and the scale byte of that block.
// Which 32 k of a stage a group takes is free as long as both operands agree: MFMA step kk of a
// 256-wide stage takes block 4G + kk, so a lane's four steps read 64 neighbouring bytes and
// their four scale bytes are one dword of the row's scales, picked by the instruction's byte
// select.
//
// Tiles: 256 rows x 256 weight columns (128 of gate and the same 128 of up), 8 waves of 64 rows
// x 128 columns, K stages of 256 (128 bytes of codes per row and per column: whole cache lines in
// the stored layout), two stages in LDS filled by direct global->LDS loads, one in flight while
// the other is consumed. Persistent grid, XCD-contiguous tile order and row blocks as in the fp8
// kernel. Both operands are staged [256][128 B], 16-byte chunks swizzled by row. A last half stage
// (K % 256 == 128) loads zeros for its absent blocks, codes and scales both.
// Within a wave the loads of the next stage and the fragment reads of the next step are spread between the
// products of this one, across the stage barrier too.
//
// What bounds it. With random codes the matrix cores alone, operands in registers, reach 6.5 PFLOP/s
// here (zeros: 9.7): the power limit. Gate/up of 65536 rows, 52 experts, H 7168, Hp 2048 takes 944-979
// us (medians by events on three cards; 3.9-4.1 PFLOP/s) and 1022-1086 in profiler traces (3.5-3.8), down with its
// 0.94 GB of output 626 (3.1) and 646-663. The
// same gate/up work takes 780 us when all codes are zero, and without its epilogue then exactly as long as its
// loads alone (731; the LDS reads alone 323): the load path is the second bound. With random codes products
// and LDS reads without the loads take 740. With 384 experts (170 rows each) the weights' HBM stream bounds
// it: gate/up 1.53-1.55 ms (3.9 TB/s; traces 1.60), down 0.88-0.89 (4.4 TB/s; traces 0.94).
// Tried and not kept (gate/up, 52 experts, beside 968): stages of 128 with four in LDS, 64-byte requests
// (1039 us); four waves of 128 x 128, a third less LDS traffic but one wave a SIMD and all 512
// registers (1109); the next tile's first two stages before the stores (973). Touching the lines two or
// three stages ahead, by one block per shared row or column panel and outside the stage's wait: no
// change (down 620 -> 605, but 384 experts 1550 -> 1670 and 888 -> 922). No difference: wave priorities,
// CUs started half a tile apart.
#include "lds_dma.h"
#include "mxfp4.h"
#include "tile_sched.h"

#include <type_traits>
#include <utility>

namespace moe {

namespace {

constexpr int M4_BM = 256;
constexpr int M4_BN = 256;      // weight columns per tile over both matrices
constexpr int M4_BK = 256;
constexpr int M4_NS = 2;
constexpr int M4_THREADS = 512;
constexpr int M4_MAX_E = 1024;
constexpr int M4_OUT = (int)0x80000000u;  // an offset past every range: loads zeros

constexpr int M4_A_BYTES = M4_BM * M4_BK / 2;
constexpr int M4_B_BYTES = M4_BN * M4_BK / 2;
constexpr int M4_LD = M4_A_BYTES / (1024 * 8);    // wave loads per stage, each operand
constexpr int M4_VM = 2 * M4_LD + 1;              // loads of a wave per stage, with the column scales
constexpr int M4_SF_B = M4_A_BYTES + M4_B_BYTES;  // weight scales [8][BN per matrix] per matrix
constexpr int M4_STAGE = M4_SF_B + M4_BN * 8;
constexpr int M4_SF_A = M4_BM * 32;               // activation scales of four stages [256][32]
constexpr int M4_SCHED = M4_NS * (M4_STAGE + M4_SF_A);
constexpr int M4_LDS = M4_SCHED + (M4_MAX_E + 1 + 16) * 4;
static_assert(M4_LDS <= 160 * 1024, "LDS budget");

// f(0), f(1), .. f(N - 1) with compile-time numbers.
template <int N, typename F, int... I>
__device__ __forceinline__ void static_for_impl(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_impl<N>(f, std::make_integer_sequence<int, N>{});
}

struct Mx4Args {
  const uint8_t *A, *A_sf;
  const int* row_src;  // gate/up only: rows gathered from A [a_rows]
  int a_k, a_rows;
  const int* cu;
  int E, Kd, N;
  const uint8_t *B0, *B0_sf, *B1, *B1_sf;
  uint8_t *h_q, *h_sf;
  uint16_t* y;
};

template <bool GATED>
__global__ __launch_bounds__(M4_THREADS, 1) void ffn_mxfp4_kernel(Mx4Args a) {
  constexpr int NB = GATED ? 2 : 1;
  constexpr int BN = M4_BN / NB;   // columns per matrix
  constexpr int NT = BN / 64;      // 32-column blocks of a wave per matrix
  constexpr int MT = 2;            // 32-row blocks of a wave
  constexpr int STORES = GATED ? 2 : 16;  // 8-byte stores of a row block (down: a whole one), at least
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  unsigned char* sf_a = smem + M4_NS * M4_STAGE;
  int* tstart = reinterpret_cast<int*>(smem + M4_SCHED);
  int* wsum = tstart + M4_MAX_E + 1;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int Kd = a.Kd, N = a.N;
  const int ntn = (N + BN - 1) / BN;
  const int total = build_tile_prefix<M4_BM, M4_THREADS>(a.cu, a.E, ntn, tstart, wsum);
  const int kb = Kd / 2, ksf = Kd / 32;
  const int nk = (Kd + M4_BK - 1) / M4_BK;
  const bool half = Kd % M4_BK != 0;
  const int G = gridDim.x;
  const int slot = xcd_slot(blockIdx.x, G);
  const uint32_t lds0 = lds_addr(smem);

  // Loads of a stage: wave load j = wave + 8 i fills LDS rows 8j..8j+7 of 128 bytes, lane -> row 8j + lane/8, slot
  // lane % 8 of which holds chunk slot ^ (row/2 mod 8): sixteen neighbouring lanes of a fragment read, a row
  // each, then hit all 64 banks once. The columns lie in the order in which the fragments take them: LDS row
  // 32 nt + l of a wave's holds its column NT l + nt (in column order the lanes of a read, NT columns apart,
  // met in half of the banks). Chunks 4..7 are absent in a half stage.
  int ld_row[M4_LD];
#pragma unroll
  for (int i = 0; i < M4_LD; ++i) ld_row[i] = (wave + 8 * i) * 8 + (lane >> 3);
  const int ld_chunk = (lane & 7) ^ ((ld_row[0] >> 1) & 7);   // rows 64 apart share it
  const int b_off = (NT * (ld_row[0] & 31) + (ld_row[0] >> 5)) * kb + ld_chunk * 16;
  // Scales of the columns: LDS [NB][8][BN], bytes 256 wave .. of the block. Scales of the rows: half
  // lane % 2 of the 32 bytes of row 32 wave + lane / 2, for four stages at once. They lie row by row, a cache
  // line per row however few bytes are taken, and the lines asked for cost as much as the bytes.
  const int sa_row = wave * 32 + (lane >> 1), sa_half = lane & 1;
  const int sb_byte = wave * 256 + lane * 4;
  const int sb_nb = sb_byte / (8 * BN), sb_kb = (sb_byte / BN) & 7, sb_col = sb_byte % BN;

  struct Tile {
    int e, row0, rows_valid, n0, nmt;
    i32x4_t rA, rS, rB0, rB1;
    int a_off[M4_LD], s_off;
  };
  auto decode = [&](int t) __attribute__((always_inline)) {
    Tile d;
    d.e = __builtin_amdgcn_readfirstlane(find_expert(tstart, a.E, t));
    const int lt = t - tstart[d.e];
    const int gbeg = a.cu[d.e];
    const int rows_e = a.cu[d.e + 1] - gbeg;
    const int mte = (rows_e + M4_BM - 1) / M4_BM;
    const int ntile = lt / mte;
    const int mtile = lt - ntile * mte;
    const int chunk = even_chunk(rows_e, mte);
    d.row0 = __builtin_amdgcn_readfirstlane(gbeg + mtile * chunk);
    d.rows_valid = __builtin_amdgcn_readfirstlane(min(chunk, rows_e - mtile * chunk));
    d.n0 = __builtin_amdgcn_readfirstlane(ntile * BN);
    if (GATED && a.row_src) {
      d.rA = make_rsrc(a.A, (uint32_t)a.a_rows * (uint32_t)kb);
      d.rS = make_rsrc(a.A_sf, (uint32_t)a.a_rows * (uint32_t)ksf);
      int src[M4_LD];
#pragma unroll
      for (int i = 0; i < M4_LD; ++i) src[i] = a.row_src[d.row0 + min(ld_row[i], d.rows_valid - 1)];
      const int ssrc = a.row_src[d.row0 + min(sa_row, d.rows_valid - 1)];
#pragma unroll
      for (int i = 0; i < M4_LD; ++i)
        d.a_off[i] = (ld_row[i] < d.rows_valid && src[i] >= 0) ? (src[i] / a.a_k) * kb + ld_chunk * 16 : M4_OUT;
      d.s_off = (sa_row < d.rows_valid && ssrc >= 0) ? (ssrc / a.a_k) * ksf + sa_half * 16 : M4_OUT;
    } else {
      d.rA = make_rsrc(a.A + (size_t)d.row0 * kb, (uint32_t)d.rows_valid * (uint32_t)kb);
      d.rS = make_rsrc(a.A_sf + (size_t)d.row0 * ksf, (uint32_t)d.rows_valid * (uint32_t)ksf);
#pragma unroll
      for (int i = 0; i < M4_LD; ++i)
        d.a_off[i] = ld_row[i] < d.rows_valid ? ld_row[i] * kb + ld_chunk * 16 : M4_OUT;
      d.s_off = sa_row < d.rows_valid ? sa_row * ksf + sa_half * 16 : M4_OUT;
    }
    d.nmt = __builtin_amdgcn_readfirstlane((wm * 32 < d.rows_valid) + (128 + wm * 32 < d.rows_valid));
    const size_t wbase = ((size_t)d.e * N + d.n0) * kb;
    const uint32_t range = (uint32_t)(N - d.n0) * (uint32_t)kb;
    d.rB0 = make_rsrc(a.B0 + wbase, range);
    d.rB1 = GATED ? make_rsrc(a.B1 + wbase, range) : d.rB0;
    return d;
  };
  // Piece j of this wave's loads of stage kt into buffer buf: row loads, column loads, column scales.
  auto piece = [&](const Tile& d, int kt, int buf, auto j_) __attribute__((always_inline)) {
    constexpr int j = decltype(j_)::value;
    const uint32_t so = lds0 + (uint32_t)buf * M4_STAGE;
    const bool cut = half && kt == nk - 1;
    if constexpr (j < M4_LD) {
      lds_dma16(d.rA, so + (wave + 8 * j) * 1024, cut && ld_chunk >= 4 ? M4_OUT : d.a_off[j], kt * (M4_BK / 2));
    } else if constexpr (j < 2 * M4_LD) {
      constexpr int i = j - M4_LD;
      constexpr bool second = GATED && i >= M4_LD / 2;
      // rows 64 i..64 i + 63: 32-column blocks 2 i and 2 i + 1, NT of them a wave's
      constexpr int blk = 2 * i - (second ? BN / 32 : 0);
      constexpr int c0 = blk / NT * (BN / 2) + blk % NT;
      lds_dma16(second ? d.rB1 : d.rB0, so + M4_A_BYTES + (wave + 8 * i) * 1024,
                (cut && ld_chunk >= 4) || (!GATED && d.n0 + c0 >= N) ? M4_OUT : b_off, kt * (M4_BK / 2) + c0 * kb);
    } else {
      const int planes = min(8, ksf - 8 * kt);
      const uint8_t* sfb = (GATED && sb_nb) ? a.B1_sf : a.B0_sf;
      lds_dma4(make_rsrc(sfb + ((size_t)d.e * ksf + 8 * (size_t)kt) * N, (uint32_t)N * (uint32_t)planes),
               so + M4_SF_B + wave * 256, sb_kb < planes && d.n0 + sb_col < N ? sb_kb * N + d.n0 + sb_col : M4_OUT, 0);
    }
  };
  auto issue = [&](const Tile& d, int kt, int buf) __attribute__((always_inline)) {
    static_for<M4_VM>([&](auto j_) __attribute__((always_inline)) { piece(d, kt, buf, j_); });
  };
  // The row scales of stages 4q..4q+3, into half `ab`; bytes past the last row's read as zero, so the whole
  // offset is in the checked part.
  auto issue_sf = [&](const Tile& d, int q, int ab) __attribute__((always_inline)) {
    lds_dma16(d.rS, lds0 + M4_NS * M4_STAGE + ab * M4_SF_A + wave * 1024, d.s_off + q * 32, 0);
  };

  // Fragments: chunk 4G + kk of row (block) + l, l = lane % 32. Block nt of a wave's columns takes every NT-th
  // column, nt + NT l, so that the scale bytes of a lane's NT columns are neighbours and one LDS
  // read brings them all.
  const int g2 = lane >> 5, l32 = lane & 31;
  const int ar = wm * 32 + l32;
  const int wcol = wn * (BN / 2) + NT * l32;
  int fa_off[4], fb_off[4];
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
    fa_off[kk] = ar * 128 + (((4 * g2 + kk) ^ ((l32 >> 1) & 7)) << 4);  // the same for every 32-row block
    fb_off[kk] = M4_A_BYTES + (wn * (BN / 2) + l32) * 128 + (((4 * g2 + kk) ^ ((l32 >> 1) & 7)) << 4);
  }
  const int sb_off = M4_SF_B + 4 * g2 * BN + wcol;

  int buf = 0, ab = 0, stored = 0;  // stored: row blocks that this wave stored after the prologue's loads
  Tile cur;
  if (slot < total) {
    cur = decode(slot);
    issue_sf(cur, 0, ab);
    issue(cur, 0, buf);
  }
  for (int t = slot; t < total; t += G) {
    f32x16_t acc[NB][MT][NT];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[nb][mt][nt][i] = 0.f;

    // The K loop over the first MTV row blocks of this wave. The fragments of a step are read while
    // the products of the step before run, across the stage barrier too: the last step of a stage
    // is in registers when the stage is given up.
    auto k_loop = [&](auto mtv) {
      constexpr int MTV = decltype(mtv)::value;
      constexpr int MR = MTV ? MTV : 1;
      struct Frag {
        i32x4_t a[MR], b[NB][NT];
        int sb[NB];
      };
      Frag f0, f1;
      int sa[MR];
      // Read `i` of a step's fragments, in the order in which the products take them.
      constexpr int READS = MTV + NB * (1 + NT);
      auto read_one = [&](Frag& f, const unsigned char* st, int kk, auto i_) __attribute__((always_inline)) {
        constexpr int i = decltype(i_)::value;
        if constexpr (i < MTV) {
          f.a[i] = *reinterpret_cast<const i32x4_t*>(st + fa_off[kk] + i * 128 * 128);
        } else if constexpr (i < MTV + NB) {
          const unsigned char* sp = st + sb_off + ((i - MTV) * 8 + kk) * BN;
          f.sb[i - MTV] = NT == 2 ? *reinterpret_cast<const uint16_t*>(sp) : *reinterpret_cast<const int*>(sp);
        } else if constexpr (i < READS) {
          constexpr int nt = (i - MTV - NB) / NB, nb = (i - MTV - NB) % NB;
          f.b[nb][nt] = *reinterpret_cast<const i32x4_t*>(st + fb_off[kk] + (nb * BN + nt * 32) * 128);
        }
      };
      // The products of one step, with the reads of the next spread between them, and with the loads of stage
      // kt + 1 (LOAD): a wave that issued them in a row would hold up its matrix core.
      auto step = [&](const Frag& f, const int* s4, auto kk_, Frag& next, const unsigned char* st, auto next_,
                      auto load_, int kt) __attribute__((always_inline)) {
        constexpr int kk = decltype(kk_)::value, kk_next = decltype(next_)::value;  // kk_next < 0: none
        constexpr bool LOAD = decltype(load_)::value;
        constexpr int PRODUCTS = NB * NT * MR;
        static_for<PRODUCTS>([&](auto m_) __attribute__((always_inline)) {
          constexpr int m = decltype(m_)::value;
          constexpr int mt = m % MR, nb = m / MR % NB, nt = m / MR / NB;
          const i32x4_t z = {0, 0, 0, 0};
          const i32x8_t bf = __builtin_shufflevector(f.b[nb][nt], z, 0, 1, 2, 3, 4, 5, 6, 7);
          const i32x8_t af = __builtin_shufflevector(f.a[mt], z, 0, 1, 2, 3, 4, 5, 6, 7);
          // gate/up: weights first, lane l then holds output row l % 32; down: rows first, a lane holds a column
          if constexpr (GATED)
            acc[nb][mt][nt] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(bf, af, acc[nb][mt][nt], 4, 4, nt, f.sb[nb],
                                                                             kk, s4[mt]);
          else
            acc[nb][mt][nt] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(af, bf, acc[nb][mt][nt], 4, 4, kk, s4[mt],
                                                                             nt, f.sb[nb]);
          __builtin_amdgcn_sched_barrier(0);
          if constexpr (kk_next >= 0) {
            constexpr int per = (READS + PRODUCTS - 1) / PRODUCTS;
            static_for<per>([&](auto i_) __attribute__((always_inline)) {
              read_one(next, st, kk_next, std::integral_constant<int, per * m + decltype(i_)::value>{});
            });
          }
          if constexpr (LOAD) {
            constexpr int per = (M4_VM + PRODUCTS - 1) / PRODUCTS;
            static_for<per>([&](auto i_) __attribute__((always_inline)) {
              constexpr int j = per * m + decltype(i_)::value;
              if constexpr (j < M4_VM) piece(cur, kt + 1, buf ^ 1, std::integral_constant<int, j>{});
            });
          }
          __builtin_amdgcn_sched_barrier(0);
        });
      };
      using std::integral_constant;
      auto scales = [&](int kt) __attribute__((always_inline)) {
#pragma unroll
        for (int mt = 0; mt < MTV; ++mt) {
          sa[mt] = *reinterpret_cast<const int*>(sf_a + ab * M4_SF_A + (mt * 128 + ar) * 32 + (kt & 3) * 8 + 4 * g2);
          if (half && kt == nk - 1 && g2) sa[mt] = 0;  // the absent blocks' bytes are another row's
        }
      };
      auto rest = [&](const unsigned char* st, int kt) __attribute__((always_inline)) {
        step(f0, sa, integral_constant<int, 0>{}, f1, st, integral_constant<int, 1>{}, std::false_type{}, kt);
        step(f1, sa, integral_constant<int, 1>{}, f0, st, integral_constant<int, 2>{}, std::false_type{}, kt);
        step(f0, sa, integral_constant<int, 2>{}, f1, st, integral_constant<int, 3>{}, std::false_type{}, kt);
      };
      // Stage kt has landed for every wave, and every wave has read all it needs of the other buffer.
      auto stage = [&](int kt, auto load_) __attribute__((always_inline)) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        wait_barrier<0>();
        if ((kt & 3) == 0) {
          ab ^= 1;
          if (kt + 4 < nk) issue_sf(cur, kt / 4 + 1, ab ^ 1);
        }
        if constexpr (MTV > 0) {
          const unsigned char* st = smem + buf * M4_STAGE;
          step(f1, sa, integral_constant<int, 3>{}, f0, st, integral_constant<int, 0>{}, load_, kt);
          scales(kt);
          rest(st, kt);
        } else if constexpr (decltype(load_)::value) {
          issue(cur, kt + 1, buf ^ 1);
        }
        buf ^= 1;
      };
      // The first stage: the previous tile's stores, younger than its loads, need not be done (memory operations
      // complete in order). Then the stages that load another one, then the last.
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (stored == 0) wait_barrier<0>();
      else if (stored == 1) wait_barrier<STORES>();
      else wait_barrier<2 * STORES>();
      if (nk > 4) issue_sf(cur, 1, ab ^ 1);
      if (nk > 1) issue(cur, 1, buf ^ 1);
      if constexpr (MTV > 0) {
        const unsigned char* st = smem + buf * M4_STAGE;
        static_for<READS>([&](auto i_) __attribute__((always_inline)) { read_one(f0, st, 0, i_); });
        scales(0);
        rest(st, 0);
      }
      buf ^= 1;
      for (int kt = 1; kt + 1 < nk; ++kt) stage(kt, std::true_type{});
      if (nk > 1) stage(nk - 1, std::false_type{});
      if constexpr (MTV > 0)
        step(f1, sa, integral_constant<int, 3>{}, f0, smem, integral_constant<int, -1>{}, std::false_type{}, 0);
    };
    if (cur.nmt == 2) k_loop(std::integral_constant<int, 2>{});
    else if (cur.nmt == 1) k_loop(std::integral_constant<int, 1>{});
    else k_loop(std::integral_constant<int, 0>{});

    const int row0 = cur.row0, rows_valid = cur.rows_valid, n0 = cur.n0, nmt = cur.nmt;
    // The next tile's first stage goes into the buffer that stage nk - 1 did not use, whose readers all
    // passed the last barrier. So do those of the row scales' other half.
    if (t + G < total) {
      cur = decode(t + G);
      ab ^= 1;
      issue_sf(cur, 0, ab);
      issue(cur, 0, buf);
    }
    const bool wave_in = GATED || n0 + wn * (BN / 2) < N;  // the wave's columns are inside the matrix
    if constexpr (GATED)
      stored = nmt;
    else
      stored = wave_in ? (wm * 32 + 32 <= rows_valid) + (wm * 32 + 160 <= rows_valid) : 0;

    // Gate/up: lane l holds row l % 32 of its block; acc[..][nt][4j + c] is column NT (8j + 4G + c) + nt of the
    // wave's: for each j a run of 4 NT neighbouring columns. Down: lane l holds columns 4 (l % 32) + nt, and
    // acc[..][4j + c] is row 8j + 4G + c: a store writes 256 neighbouring bytes of
    // two rows (65536 rows, 52 experts: 620 us; with a row per lane, 16 bytes in each of 32 rows, 660 us).
    if (wave_in) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        if (mt >= nmt) break;
        const int r = mt * 128 + ar;
        const bool ok = r < rows_valid;
        const size_t row = (size_t)row0 + (ok ? r : 0);
        const int c0 = n0 + wn * (BN / 2);
        if constexpr (GATED) {
          // a block of 32 columns is the runs of j = 2p and 2p + 1 of this lane and of lane ^ 32
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            float v[16];
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int at = 8 * p + i / 2;  // 4j + c, two columns each
              v[i] = silu_f32(acc[0][mt][i & 1][at]) * acc[1][mt][i & 1][at];
              m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
            }
            const auto both = __builtin_amdgcn_permlane32_swap(m, m, false, false);
            uint32_t byte = mx_scale_byte(max((uint32_t)both[0], (uint32_t)both[1]));
            // A padding row is zeros, but its zero codes times a weight block whose scale is NaN are NaN. Looked up
            // only where a NaN came out, so that the tiles without one load nothing for it.
            if (a.row_src && __ballot(byte == MX_NAN_SCALE) != 0) {
              if (ok && byte == MX_NAN_SCALE && a.row_src[row] < 0) {
                byte = 0;
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = 0.f;
              }
            }
            // the halves trade runs: group 0 gets columns 0..15 of the block, group 1 columns 16..31
            const auto tr = __builtin_amdgcn_permlane32_swap(mx_pack8(v, byte), mx_pack8(v + 8, byte), false, false);
            if (ok) {
              const int c = c0 + 32 * p;
              *reinterpret_cast<uint2*>(a.h_q + row * (N / 2) + c / 2 + 8 * g2) = make_uint2(tr[0], tr[1]);
              if (g2 == 0) a.h_sf[row * (N / 32) + c / 32] = (uint8_t)byte;
            }
          }
        } else {
          const int r0 = mt * 128 + wm * 32 + 4 * g2;  // this lane's rows: r0 + 8j + c
          uint16_t* yp = a.y + (size_t)(row0 + r0) * N + c0 + 4 * l32;
          const bool whole = mt * 128 + wm * 32 + 32 <= rows_valid;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int dr = 8 * (i >> 2) + (i & 3);
            if (whole || r0 + dr < rows_valid)
              *reinterpret_cast<uint2*>(yp + (size_t)dr * N) =
                  make_uint2(pack_bf16x2(acc[0][mt][0][i], acc[0][mt][1][i]), pack_bf16x2(acc[0][mt][2][i], acc[0][mt][3][i]));
          }
        }
      }
    }
  }
}

// ---- few rows per expert --------------------------------------------------------------
//
// With a handful of rows per expert the weights are read once and hardly reused: what counts is to
// have many of their bytes in flight. A wave takes 16 columns of one matrix and streams them past up to
// 16 RG rows straight into registers, no LDS, with the weights as the first operand of
// v_mfma_scale_f32_16x16x128_f8f6f4 (lane l: column l % 16, block G = l / 16 of the step's four) and the rows as
// the second. In a step of 512 a lane takes the 64 bytes at 64 G of its column, two whole lines
// per column and step, and the next step's loads are out before this one's products. A block
// of eight waves takes 32 columns of gate and of up, each split in two along the reduction, and adds and rounds
// through LDS (one block of the format is 32 columns), or 128 columns of down. An expert with more
// rows than that gets a block per 16 RG of them: one after the other in one block, an uneven batch
// would wait for its largest expert (gate/up, H 7168, Hp 128, 2048 rows all on one of 64 experts: 1413 us, side
// by side 26, as long as the same rows spread evenly; 128 rows on one of 8, Hp 2048: 184, 26).

constexpr int S4_THREADS = 512;

template <int RG>
struct S4Step {
  i32x4_t w[4], x[RG][4];
  int ws[4], xs[RG];
};

template <bool GATED, int RG>
__global__ __launch_bounds__(S4_THREADS) void ffn_mxfp4_stream_kernel(Mx4Args a) {
  constexpr int BN = GATED ? 32 : 128;  // columns of a block
  constexpr int ROWS = 16 * RG;
  __shared__ float part[GATED ? 8 : 1][GATED ? RG : 1][16][17];  // [wave][row group][row][column]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int N = a.N, kb = a.Kd / 2, ksf = a.Kd / 32;
  const int ncb = N / BN;
  // Eight neighbours on one XCD (they share scale lines, a heavy expert's also panels), the eights round-robin:
  // the blocks without a chunk are the last ones and leave every XCD the same work (8 experts, 16 rows each: 35 us;
  // with the whole range cut into eight, 49).
  const int whole = gridDim.x & ~63;
  const int b = blockIdx.x;
  const int idx = b < whole ? (b & ~63) + (b & 7) * 8 + ((b >> 3) & 7) : b;
  const int left = idx / ncb;  // this block's chunk among the experts' chunks of ROWS rows, in expert order
  int e = -1, before = 0, chunks = 0;
  for (int base = 0; base < a.E; base += 64) {
    const int i = min(base + lane, a.E - 1);
    const int n = base + lane < a.E ? (a.cu[i + 1] - a.cu[i] + ROWS - 1) / ROWS : 0;
    int upto = popc_below(__ballot(n > 0)) + n;
    if (__ballot(n > 1)) upto = sched_wave_incl_scan(n);
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
  const int gbeg = __builtin_amdgcn_readfirstlane(a.cu[e]);
  const int rows = __builtin_amdgcn_readfirstlane(a.cu[e + 1]) - gbeg;

  const int c16 = lane & 15, G = lane >> 4;
  const int nb = GATED ? (wave >> 1) & 1 : 0;
  const int n0 = cb * BN + (GATED ? (wave & 1) * 16 : wave * 16);
  const uint8_t* wp = (nb ? a.B1 : a.B0) + ((size_t)e * N + n0 + c16) * kb + G * 64;
  const uint8_t* wsp = (nb ? a.B1_sf : a.B0_sf) + ((size_t)e * ksf + 4 * G) * N + n0 + c16;
  const int steps = (kb + 255) / 256;
  const int first = GATED && wave >= 4 ? (steps + 1) / 2 : 0;
  const int last = GATED && wave < 4 ? (steps + 1) / 2 : steps;

  const uint8_t *xp[RG], *xsp[RG];
  int nrg = 0;
#pragma unroll
  for (int g = 0; g < RG; ++g) {
    // rows past the last read it again; their results are not stored
    int r = gbeg + min(r0 + 16 * g + c16, rows - 1);
    if (GATED && a.row_src) {
      const int src = a.row_src[r];
      r = src < 0 ? 0 : min(src / a.a_k, a.a_rows - 1);
    }
    xp[g] = a.A + (size_t)r * kb + G * 64;
    xsp[g] = a.A_sf + (size_t)r * ksf + 4 * G;
    nrg += r0 + 16 * g < rows;
  }
  f32x4_t acc[RG];
#pragma unroll
  for (int g = 0; g < RG; ++g) acc[g] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  // Step `it` of this lane; past the end of the reduction (a last step that is not whole) zeros.
  auto load = [&](S4Step<RG>& d, int it) __attribute__((always_inline)) {
    const bool in = it * 256 + G * 64 < kb;
    const int o = in ? it * 256 : 0, os = in ? it * 16 : 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) d.w[q] = *reinterpret_cast<const i32x4_t*>(wp + (in ? o : -G * 64) + 16 * q);
#pragma unroll
    for (int q = 0; q < 4; ++q) d.ws[q] = wsp[(ptrdiff_t)(in ? os + q : -4 * G) * N];
#pragma unroll
    for (int g = 0; g < RG; ++g)
      if (g < nrg) {
#pragma unroll
        for (int q = 0; q < 4; ++q) d.x[g][q] = *reinterpret_cast<const i32x4_t*>(xp[g] + (in ? o : -G * 64) + 16 * q);
        d.xs[g] = *reinterpret_cast<const int*>(xsp[g] + (in ? os : -4 * G));
      }
    if (!in) {
      const i32x4_t z = {0, 0, 0, 0};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        d.w[q] = z;
        d.ws[q] = 0;
      }
#pragma unroll
      for (int g = 0; g < RG; ++g) {
#pragma unroll
        for (int q = 0; q < 4; ++q) d.x[g][q] = z;
        d.xs[g] = 0;
      }
    }
  };
  auto mul = [&](const S4Step<RG>& d) __attribute__((always_inline)) {
    const i32x4_t z = {0, 0, 0, 0};
    auto one = [&](auto q_) __attribute__((always_inline)) {
      constexpr int q = decltype(q_)::value;
      const i32x8_t wf = __builtin_shufflevector(d.w[q], z, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
      for (int g = 0; g < RG; ++g)
        if (g < nrg) {
          const i32x8_t xf = __builtin_shufflevector(d.x[g][q], z, 0, 1, 2, 3, 4, 5, 6, 7);
          acc[g] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf, xf, acc[g], 4, 4, 0, d.ws[q], q, d.xs[g]);
        }
    };
    one(std::integral_constant<int, 0>{});
    one(std::integral_constant<int, 1>{});
    one(std::integral_constant<int, 2>{});
    one(std::integral_constant<int, 3>{});
  };
  S4Step<RG> s0, s1;
  if (first < last) load(s0, first);
  for (int it = first; it < last; it += 2) {
    if (it + 1 < last) load(s1, it + 1);
    mul(s0);
    if (it + 2 < last) load(s0, it + 2);
    if (it + 1 < last) mul(s1);
  }

  // lane l holds row l % 16 of its group, columns 4G..4G+3 of the wave's 16
  if constexpr (GATED) {
#pragma unroll
    for (int g = 0; g < RG; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[wave][g][c16][4 * G + i] = acc[g][i];
    __syncthreads();
    // wave g rounds row group g: lane = 4 row + quarter of the 32 columns
    const int r = lane >> 2, j = lane & 3;
    if (wave < RG && r0 + 16 * wave + r < rows) {
      const int row = gbeg + r0 + 16 * wave + r;
      const bool pad = a.row_src && a.row_src[row] < 0;
      float v[8];
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int hw = j >> 1, c = (j & 1) * 8 + i;
        const float gate = part[hw][wave][r][c] + part[4 + hw][wave][r][c];
        const float up = part[2 + hw][wave][r][c] + part[6 + hw][wave][r][c];
        v[i] = pad ? 0.f : silu_f32(gate) * up;
        m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
      }
      m = max(m, (uint32_t)__builtin_amdgcn_update_dpp((int)m, (int)m, 0xB1, 0xF, 0xF, false));
      m = max(m, (uint32_t)__builtin_amdgcn_update_dpp((int)m, (int)m, 0x4E, 0xF, 0xF, false));
      const uint32_t byte = mx_scale_byte(m);
      *reinterpret_cast<uint32_t*>(a.h_q + (size_t)row * (N / 2) + cb * 16 + 4 * j) = mx_pack8(v, byte);
      if (j == 0) a.h_sf[(size_t)row * (N / 32) + cb] = (uint8_t)byte;
    }
  } else {
#pragma unroll
    for (int g = 0; g < RG; ++g) {
      const int r = r0 + 16 * g + c16;
      if (r < rows)
        *reinterpret_cast<uint2*>(a.y + (size_t)(gbeg + r) * N + n0 + 4 * G) =
            make_uint2(pack_bf16x2(acc[g][0], acc[g][1]), pack_bf16x2(acc[g][2], acc[g][3]));
    }
  }
}

template <bool GATED>
moe_status_t launch_stream(const Mx4Args& a, int M, hipStream_t s) {
  const int slots = M < a.E ? M : a.E;  // at most so many experts have rows
  // (two groups of 16 rows a pass cost more than one where most experts have fewer than eight)
  const int rg = M <= 8 * slots ? 1 : 2;
  // n experts with R rows make at most n + (R - n) / (16 rg) chunks; blocks past the last one have none
  const int64_t chunks = slots + (M - slots) / (16 * rg);
  const unsigned grid = (unsigned)(chunks * (a.N / (GATED ? 32 : 128)));
  if (rg == 1)
    ffn_mxfp4_stream_kernel<GATED, 1><<<grid, S4_THREADS, 0, s>>>(a);
  else
    ffn_mxfp4_stream_kernel<GATED, 2><<<grid, S4_THREADS, 0, s>>>(a);
  return launch_status();
}

// Whether the streaming kernel takes M rows over E experts and N columns. It does where the tiles
// could not fill the chip: up to `slots` experts have rows, each with N / bn tiles. Measured on 256
// CUs, us, streamed against tiles, rows per expert in brackets:
//   gate/up  8 experts, H 7168, Hp 2048 (128 tiles): [4] 25 / 38  [16] 34 / 38  [24] 44 / 38
//            12 experts, the same (192 tiles): [1] 31 / 38  [8] 38 / 38  [16] 50 / 39
//            16 experts, the same (256 tiles): [1] 39 / 39  [4] 43 / 39  [16] 66 / 39
//            24 experts, H 1024, Hp 1024 (192 tiles): [1] 8.6 / 9.8  [8] 9.4 / 9.9  [16] 12.8 / 9.8
//            4 experts, H 2560, Hp 1280 (40 tiles): [16] 8.4 / 15.8  [32] 11.1 / 16.1  [48] 19.7 / 16.6
//            all rows on one of 8 experts (128 tiles): [4] 18 / 29  [16] 27 / 32  [32] 50 / 45
//            1000 rows on one of 256 experts, 12 on the others, Hp 128 (256 tiles): 77 / 75
//   down     8 experts, Hp 2048, H 7168 (224 tiles): [1] 13.3 / 15.9  [4] 14.7 / 15.8  [16] 21 / 16
//            128 experts, Hp 128, H 7168 (3584 tiles): [1] 40 / 35
//            4 experts, Hp 1280, H 2560 (40 tiles): [16] 8.9 / 10.1  [32] 11.5 / 10.9
//            all rows on one of 16 experts, Hp 2048, H 1024 (64 tiles): [8] 11.0 / 11.8  [16] 15.5 / 15.9
// Gate/up streams up to 32, 16 and 8 rows per expert while the tiles are a quarter, a half and three quarters of
// the CUs; down, whose reduction is short, up to 16 and 2 while they are a quarter and all of them.
bool streams(bool gated, int M, int E, int N) {
  const int slots = M < E ? M : E;
  const int bn = gated ? M4_BN / 2 : M4_BN;
  const int64_t tiles = (int64_t)slots * ((N + bn - 1) / bn);
  const int cus = device_cu_count();
  if (gated)
    return (M <= 32 * slots && 4 * tiles <= cus) || (M <= 16 * slots && 2 * tiles <= cus) ||
           (M <= 8 * slots && 4 * tiles <= 3 * cus);
  return (M <= 16 * slots && 4 * tiles <= cus) || (M <= 2 * slots && tiles <= cus);
}

template <bool GATED>
moe_status_t launch_tiles(const Mx4Args& a, hipStream_t s) {
  static std::atomic<unsigned char> lds_set[MOE_MAX_DEVICES];
  if (ensure_lds_limit(reinterpret_cast<const void*>(&ffn_mxfp4_kernel<GATED>), M4_LDS, lds_set) != MOE_OK)
    return MOE_EHIP;
  ffn_mxfp4_kernel<GATED><<<device_cu_count(), M4_THREADS, M4_LDS, s>>>(a);
  return launch_status();
}

}  // namespace

moe_status_t launch_ffn_gate_up_mxfp4(const uint8_t* x_q, const uint8_t* x_sf, const int* row_src, int T, int K,
                                      const int* cu, int M, int E, int H, int Hp, const uint8_t* wg,
                                      const uint8_t* wu, const uint8_t* sg, const uint8_t* su, uint8_t* h_q,
                                      uint8_t* h_sf, hipStream_t s) {
  if (M == 0) return MOE_OK;
  const Mx4Args a{x_q, x_sf, row_src, K, T, cu, E, H, Hp, wg, sg, wu, su, h_q, h_sf, nullptr};
  if (streams(true, M, E, Hp) && (!row_src || T > 0)) return launch_stream<true>(a, M, s);
  return launch_tiles<true>(a, s);
}

moe_status_t launch_ffn_down_mxfp4(const uint8_t* h_q, const uint8_t* h_sf, const int* cu, int M, int E, int H,
                                   int Hp, const uint8_t* wd, const uint8_t* sd, void* y, hipStream_t s) {
  if (M == 0) return MOE_OK;
  const Mx4Args a{h_q, h_sf, nullptr, 1, 0, cu, E, Hp, H, wd, sd, nullptr, nullptr, nullptr, nullptr,
                  static_cast<uint16_t*>(y)};
  if (streams(false, M, E, H)) return launch_stream<false>(a, M, s);
  return launch_tiles<false>(a, s);
}

}  // namespace moe
