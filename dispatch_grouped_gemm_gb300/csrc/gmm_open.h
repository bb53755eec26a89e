// gmm_open.h -- the products of gmm_open.cu: grouped by expert, and over a stack
// of matrices.
#pragma once

#include <cuda_fp16.h>

#include "hmm_internal.h"

namespace hmm {

constexpr int OPEN_ROWS = 0;
constexpr int OPEN_DEPTH = 1;
constexpr int OPEN_STACK = 2;

// Epilogues of OPEN_STACK on acc(m, n), operands and results in fp16:
//   GRAM    out = alpha acc                                   symmetric
//   POLY    out = alpha acc + beta in_hi + gamma [m = n]      symmetric
//   UPDATE  v = alpha acc + beta in_hi + gamma in_lo; out = fp16(v), out_lo = fp16(v - out)
//   LAST    the same v as the caller's result (bf16 or fp16)
// A symmetric result is computed for tiles on and above the diagonal and written
// twice.
constexpr int OPEN_EPI_GRAM = 0;
constexpr int OPEN_EPI_POLY = 1;
constexpr int OPEN_EPI_UPDATE = 2;
constexpr int OPEN_EPI_LAST = 3;

// [batch][rows][cols], rows ld and matrices stride elements apart (multiples of 8;
// 16-byte aligned)
struct OpenOperand {
  const void* ptr;
  int64_t rows, cols, batch, ld, stride;
};

struct OpenParams {
  int M, N, Z, R;     // extent of m, of n; experts or matrices; rows
  int K, kb;          // depth, in blocks (DEPTH: per expert)
  int mt, nt, tiles;  // 256-tiles of m, of n, per expert or matrix
  int a_mn, b_mn;     // operands with m / n contiguous
  int sym, epi, out_f16, plain_out;
  uint32_t idesc;
  float alpha, beta, gamma;
  const int32_t* offsets;  // [Z + 1] rows of the experts
  const __half *in_hi, *in_lo;
  int64_t ld_in;           // of in_hi, in_lo and of fp16 results
  void *out, *out_lo;
  unsigned* status;
  unsigned long long budget_ns;
};

struct OpenStack {
  OpenOperand a, b;
  bool a_mn, b_mn;
  int64_t M, N, K;
  int epi;
  float alpha, beta, gamma;
  const void *in_hi, *in_lo;
  int64_t ld_in;           // of in_hi, in_lo and the fp16 results (LAST is dense)
  void *out, *out_lo;
  int out_f16;
};

// out[r, :] = x[r, :] . op(w[e]), 0 for rows of no expert.  w: [E][rows][cols] with
// cols = M (w_mn) or cols = K (not w_mn); out dense [R, M]
int launch_open_rows(const GemmEnv& env, bool f16, const OpenOperand& w, bool w_mn, const void* x,
                     int64_t ld_x, int64_t R, int64_t K, int64_t M, int64_t E,
                     const int32_t* offsets, void* out);
// out[e] = a_e^T . b_e, dense [E, M, N]
int launch_open_depth(const GemmEnv& env, bool f16, const void* a, int64_t ld_a, int64_t M,
                      const void* b, int64_t ld_b, int64_t N, int64_t R, int64_t E,
                      const int32_t* offsets, void* out);
int launch_open_stack(const GemmEnv& env, const OpenStack& s);

}  // namespace hmm
