// Arguments of the grouped-product launchers (matmul_int8.hip, grouped_matmul.hip).
#pragma once

namespace moe {

struct GgArgs {
  const void* A;          // rows [M, Kd], or the tokens that row_src gathers from
  const int* row_src;     // row r is row row_src[r] / a_k of A [a_rows, Kd]; negative: zeros. NULL: no gather
  int a_k, a_rows;
  const int* cu;          // NULL: one group of all M rows
  int M, E;
  int Kd, N;              // reduction and columns; rows^T x rows: rows and columns of dW
  const void *B0, *B1;    // B1: the second matrix of a gated product
  const float *a_sf, *b_sf0, *b_sf1;  // INT8: scales of A's rows and of the matrices' columns [E, N]
  void* C;
  int accumulate;         // rows^T x rows: add to what C holds
};

}  // namespace moe
