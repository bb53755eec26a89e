// mx4.cu -- values (bf16 or fp32) to microscaled 4-bit operands and back: rows
// with the contraction contiguous, and stacks of expert weights [cols, rows]
// that are transposed on the way.  Bound by memory: a value is read once and
// half a byte plus a 32nd of a byte written (and the other way round).
#include "mx4.cuh"

#include <algorithm>

namespace hmm {

namespace {

constexpr int MX_THREADS = 256;
constexpr int MX_STEPS = 4;  // most steps of a row that a warp loads at once

__device__ __forceinline__ void ld_values8(const void* p, int64_t i, float (&v)[8]) {
  const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
  const float4 a = q[0], b = q[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

__device__ __forceinline__ void st_values8(void* p, int64_t i, const float (&v)[8]) {
  uint4 q;
  uint32_t* u = reinterpret_cast<uint32_t*>(&q);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
    u[j] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = q;
}

}  // namespace

// One warp per row; blockIdx.y and gridDim.y share out the pieces of a row, U
// steps of 256 columns each.  A lane holds 8 elements, four lanes a block, the
// first of which writes the scale.  Rows and columns run over whole scale tiles,
// so that the padding scales are written too.  (Lane
// groups walking (row, scale tile) pairs in one flat order, without idle lanes
// at the end of a row, were slower: their index arithmetic costs more.)
template <bool F32, int U>
__global__ void __launch_bounds__(MX_THREADS)
    mx4_quantize_rows_kernel(const void* __restrict__ src, int64_t rows, int64_t cols, int64_t ld,
                             int64_t kt, uint8_t* __restrict__ codes,
                             uint8_t* __restrict__ scales) {
  const int lane = threadIdx.x & 31;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * (MX_THREADS / 32) + (threadIdx.x >> 5);
  const bool in = r < rows;
  const int64_t kp = (cols + 31) / 32 * 32;
  grid_dep_wait();
  grid_dep_launch();
  for (int64_t p = static_cast<int64_t>(blockIdx.y) * (256 * U); p < kt * 128;
       p += static_cast<int64_t>(gridDim.y) * (256 * U)) {
    const int64_t c0 = p + 8 * lane;
    // (a step of 256 columns: 128 bytes of codes, two scale tiles)
    uint32_t* crow = reinterpret_cast<uint32_t*>(codes + r * (kp / 2) + c0 / 2);
    uint8_t* srow = scales + mx_scale_offset(r, c0 / 32, kt);
    float v[U][F32 ? 8 : 1];
    uint4 b[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t c = c0 + 256 * i;
      const bool on = in && c < cols;
      if constexpr (F32) {
        if (on) {
          ld_values8(src, r * ld + c, v[i]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
        }
      } else {
        b[i] = on ? *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(src) + r * ld + c)
                  : make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t c = c0 + 256 * i;
      uint32_t s, q;
      if constexpr (F32) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        s = mx_scale_byte(m);
        const float inv = mx_inverse_scale(s);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= inv;
        q = mx_codes8(v[i]);
      } else {
        const uint32_t u[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
        s = quad_scale_bf16(u);
        q = codes8_bf16(u, s);
      }
      if (in && c < kp) crow[32 * i] = q;
      if ((lane & 3) == 0 && c < kt * 128)
        srow[2 * MX_TILE_BYTES * i] = static_cast<uint8_t>(s);
    }
  }
}

// The way back: 16-byte stores, so 8 bf16 or 4 fp32 values per lane and step.
template <bool F32, int U>
__global__ void __launch_bounds__(MX_THREADS)
    mx4_dequantize_rows_kernel(const uint8_t* __restrict__ codes,
                               const uint8_t* __restrict__ scales, int64_t rows, int64_t cols,
                               int64_t ld, int64_t kt, void* __restrict__ dst) {
  constexpr int PER = F32 ? 4 : 8, STEP = 32 * PER;
  const int lane = threadIdx.x & 31;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * (MX_THREADS / 32) + (threadIdx.x >> 5);
  const int64_t kp = (cols + 31) / 32 * 32;
  grid_dep_wait();
  grid_dep_launch();
  if (r >= rows) return;
  for (int64_t p = static_cast<int64_t>(blockIdx.y) * (STEP * U); p < cols;
       p += static_cast<int64_t>(gridDim.y) * (STEP * U)) {
    const int64_t c0 = p + PER * lane;
    const uint8_t* crow = codes + r * (kp / 2) + c0 / 2;
    const uint8_t* srow = scales + mx_scale_offset(r, c0 / 32, kt);
    uint32_t q[U], s[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (c0 + STEP * i < cols) {
        const uint8_t* at = crow + STEP / 2 * i;
        q[i] = F32 ? *reinterpret_cast<const uint16_t*>(at) : *reinterpret_cast<const uint32_t*>(at);
        s[i] = srow[STEP / 128 * MX_TILE_BYTES * i];
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t c = c0 + STEP * i;
      if (c < cols) {
        float v[8];
        mx_values8(q[i], mx_scale(s[i]), v);
        if constexpr (F32)
          *reinterpret_cast<float4*>(static_cast<float*>(dst) + r * ld + c) =
              make_float4(v[0], v[1], v[2], v[3]);
        else
          st_values8(dst, r * ld + c, v);
      }
    }
  }
}

namespace {

// Tile of the transposing kernels: 64 stored rows x 128 elements of the
// contraction, one warp per block of 32; lane l handles the rows 2 l, 2 l + 1.
constexpr int TW_ROWS = 64;
constexpr int TW_THREADS = 128;
constexpr int TW_PITCH = 80;  // bytes per row of the tile in shared memory

// Column of the source [cols, n] that stored row d comes from, -1: a zero row.
__device__ __forceinline__ int64_t source_column(int64_t d, int64_t n, bool gate_up) {
  if (!gate_up) return d < n ? d : -1;
  const int64_t half = n / 2;
  const int64_t j = (d >> 6) * 32 + (d & 31);
  if (j >= half) return -1;
  return (d & 32) ? half + j : j;
}

}  // namespace

template <bool F32>
__global__ void __launch_bounds__(TW_THREADS)
    mx4_quantize_columns_kernel(const void* __restrict__ src, int64_t n, int64_t stored,
                                int64_t cols, int64_t kt, bool gate_up,
                                uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  __shared__ __align__(16) uint8_t s_codes[TW_ROWS * TW_PITCH];
  __shared__ __align__(4) uint8_t s_scales[TW_ROWS * 4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t e = blockIdx.z, d0 = static_cast<int64_t>(blockIdx.y) * TW_ROWS;
  const int64_t k0 = static_cast<int64_t>(blockIdx.x) * 128;
  const int64_t kp = (cols + 31) / 32 * 32;
  grid_dep_wait();
  grid_dep_launch();
  const int64_t c = source_column(d0 + 2 * lane, n, gate_up);
  const int64_t kb = k0 + warp * 32;
  const int64_t at = (e * cols + kb) * n + c;
  const int kn = c < 0 ? 0 : static_cast<int>(max(int64_t(0), min(int64_t(32), cols - kb)));
  uint32_t q[2][4], s[2];
  if constexpr (F32) {
    const float* p = static_cast<const float*>(src) + at;
    float2 v[32];
#pragma unroll
    for (int k = 0; k < 32; ++k)
      v[k] = k < kn ? *reinterpret_cast<const float2*>(p + k * n) : make_float2(0.0f, 0.0f);
    uint32_t m0 = 0, m1 = 0;
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      m0 = max(m0, __float_as_uint(v[k].x) & 0x7FFFFFFFu);
      m1 = max(m1, __float_as_uint(v[k].y) & 0x7FFFFFFFu);
    }
    s[0] = mx_scale_byte(m0);
    s[1] = mx_scale_byte(m1);
    const float i0 = mx_inverse_scale(s[0]), i1 = mx_inverse_scale(s[1]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float w0[8], w1[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        w0[k] = v[8 * j + k].x * i0;
        w1[k] = v[8 * j + k].y * i1;
      }
      q[0][j] = mx_codes8(w0);
      q[1][j] = mx_codes8(w1);
    }
  } else {
    // both columns of the lane in one word: maxima and scaling two at a time
    const uint16_t* p = static_cast<const uint16_t*>(src) + at;
    uint32_t v[32];
    if (kn == 32) {
#pragma unroll
      for (int k = 0; k < 32; ++k) v[k] = *reinterpret_cast<const uint32_t*>(p + k * n);
    } else {
#pragma unroll
      for (int k = 0; k < 32; ++k)
        v[k] = k < kn ? *reinterpret_cast<const uint32_t*>(p + k * n) : 0u;
    }
    uint32_t m[4] = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 32; ++k) m[k & 3] = pair_amax(m[k & 3], v[k]);
    const uint32_t mm = pair_amax(pair_amax(m[0], m[1]), pair_amax(m[2], m[3]));
    s[0] = mx_scale_byte(mm << 16);
    s[1] = mx_scale_byte(mm & 0xFFFF0000u);
    // (powers of two up to 2^127: their upper halves are the bf16 values)
    const uint32_t inv = (__float_as_uint(mx_inverse_scale(s[0])) >> 16) |
                         (__float_as_uint(mx_inverse_scale(s[1])) & 0xFFFF0000u);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float w0[8], w1[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t x = pair_mul(v[8 * j + k], inv);
        w0[k] = pair_lo(x);
        w1[k] = pair_hi(x);
      }
      q[0][j] = mx_codes8(w0);
      q[1][j] = mx_codes8(w1);
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = 2 * lane + h;
    *reinterpret_cast<uint4*>(s_codes + row * TW_PITCH + warp * 16) =
        make_uint4(q[h][0], q[h][1], q[h][2], q[h][3]);
    s_scales[row * 4 + warp] = static_cast<uint8_t>(s[h]);
  }
  __syncthreads();
  uint8_t* dst = codes + e * stored * (kp / 2);
  for (int i = threadIdx.x; i < TW_ROWS * 4; i += TW_THREADS) {
    const int row = i >> 2, part = i & 3;
    if (d0 + row < stored && k0 + part * 32 < kp)
      *reinterpret_cast<uint4*>(dst + (d0 + row) * (kp / 2) + k0 / 2 + part * 16) =
          *reinterpret_cast<const uint4*>(s_codes + row * TW_PITCH + part * 16);
  }
  if (threadIdx.x < TW_ROWS) {
    const int64_t rt = (stored + 127) / 128;
    *reinterpret_cast<uint32_t*>(scales + e * rt * kt * MX_TILE_BYTES +
                                 mx_scale_offset(d0 + threadIdx.x, k0 / 32, kt)) =
        *reinterpret_cast<const uint32_t*>(s_scales + threadIdx.x * 4);
  }
}

// The way back, 256 stored rows x 128 elements of the contraction per block:
// a warp takes 64 rows (lane l: rows 2 l, 2 l + 1) and the four blocks one after
// another, so that the warps of a block write neighbouring pieces of the same
// output rows.
template <bool F32>
__global__ void __launch_bounds__(TW_THREADS)
    mx4_dequantize_columns_kernel(const uint8_t* __restrict__ codes,
                                  const uint8_t* __restrict__ scales, int64_t n, int64_t stored,
                                  int64_t cols, int64_t kt, bool gate_up,
                                  void* __restrict__ dst) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t e = blockIdx.z;
  const int64_t d = (static_cast<int64_t>(blockIdx.y) * 4 + warp) * TW_ROWS + 2 * lane;
  const int64_t k0 = static_cast<int64_t>(blockIdx.x) * 128;
  const int64_t kp = (cols + 31) / 32 * 32;
  grid_dep_wait();
  grid_dep_launch();
  if (d >= stored) return;
  const int64_t c = source_column(d, n, gate_up);
  if (c < 0) return;
  const int64_t rt = (stored + 127) / 128;
  const uint8_t* p = codes + (e * stored + d) * (kp / 2) + k0 / 2;
  uint4 q[2][4];
  uint32_t s[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int b = 0; b < 4; ++b)
      q[h][b] = k0 + 32 * b < kp ? *reinterpret_cast<const uint4*>(p + h * (kp / 2) + 16 * b)
                                 : make_uint4(0, 0, 0, 0);
    s[h] = *reinterpret_cast<const uint32_t*>(scales + e * rt * kt * MX_TILE_BYTES +
                                              mx_scale_offset(d + h, k0 / 32, kt));
  }
  const int64_t at = (e * cols + k0) * n + c;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const float s0 = mx_scale((s[0] >> (8 * b)) & 255u), s1 = mx_scale((s[1] >> (8 * b)) & 255u);
    const uint32_t u0[4] = {q[0][b].x, q[0][b].y, q[0][b].z, q[0][b].w};
    const uint32_t u1[4] = {q[1][b].x, q[1][b].y, q[1][b].z, q[1][b].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (k0 + 32 * b + 8 * j >= cols) break;  // (cols is a multiple of 8)
      float v0[8], v1[8];
      mx_values8(u0[j], s0, v0);
      mx_values8(u1[j], s1, v1);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int64_t i = at + (32 * b + 8 * j + k) * n;
        if constexpr (F32) {
          *reinterpret_cast<float2*>(static_cast<float*>(dst) + i) = make_float2(v0[k], v1[k]);
        } else {
          *reinterpret_cast<__nv_bfloat162*>(static_cast<uint16_t*>(dst) + i) =
              __floats2bfloat162_rn(v0[k], v1[k]);
        }
      }
    }
  }
}

// A row of `steps` warp steps goes in pieces of u <= MX_STEPS steps, about the
// same for every piece (9 steps as 3 + 3 + 3, not 4 + 4 + 1).  Few rows: the
// pieces of a row go to several warps.
struct RowsGrid {
  dim3 grid;
  int u;
};
static RowsGrid rows_grid(int64_t rows, int64_t steps) {
  constexpr int64_t WARPS = MX_THREADS / 32;
  const int64_t pieces = (steps + MX_STEPS - 1) / MX_STEPS;
  const int64_t parts = rows >= 16384 ? 1 : std::min<int64_t>(pieces, 64);
  return {dim3(static_cast<unsigned>((rows + WARPS - 1) / WARPS), static_cast<unsigned>(parts)),
          static_cast<int>((steps + pieces - 1) / pieces)};
}

Mx4Plan mx4_plan(const hmm_mx4& d) {
  Mx4Plan p;
  p.gate_up = d.layout == HMM_MX4_GATE_UP;
  p.kp = (d.cols + 31) / 32 * 32;
  p.kt = (d.cols + 127) / 128;
  p.stored = p.gate_up ? (d.rows / 2 + 31) / 32 * 64 : d.rows;
  p.rt = (p.stored + 127) / 128;
  p.codes_bytes = d.batch * p.stored * (p.kp / 2);
  p.scales_bytes = d.batch * p.rt * p.kt * MX_TILE_BYTES;
  return p;
}

int check_mx4(const hmm_mx4* d) {
  if (!d) return HMM_ERR_ARG;
  if (d->dtype != HMM_DTYPE_BF16 && d->dtype != HMM_DTYPE_F32) return HMM_ERR_DTYPE;
  if (d->layout != HMM_MX4_ROWS && d->layout != HMM_MX4_COLUMNS && d->layout != HMM_MX4_GATE_UP)
    return HMM_ERR_ARG;
  if (d->batch < 0 || d->rows < 0 || d->cols <= 0) return HMM_ERR_SHAPE;
  if (d->cols % 8 != 0) return HMM_ERR_LAYOUT;
  if (d->layout == HMM_MX4_ROWS) {
    if (d->batch != 1) return HMM_ERR_SHAPE;  // rows are one operand
    if (d->ld < d->cols) return HMM_ERR_SHAPE;
    if (d->ld % 8 != 0) return HMM_ERR_LAYOUT;
    if (d->cols > (1 << 24) || d->rows > (int64_t(1) << 32)) return HMM_ERR_SHAPE;
  } else {
    if (d->rows % (d->layout == HMM_MX4_GATE_UP ? 16 : 8) != 0) return HMM_ERR_LAYOUT;
    if (d->batch > 65535 || d->rows > (1 << 21) || d->cols > (1 << 24)) return HMM_ERR_SHAPE;
  }
  return HMM_OK;
}

cudaError_t launch_mx4_quantize(const hmm_mx4& d, const void* values, void* codes, void* scales,
                                cudaStream_t st, bool pdl) {
  const Mx4Plan p = mx4_plan(d);
  const bool f32 = d.dtype == HMM_DTYPE_F32;
  uint8_t* c = static_cast<uint8_t*>(codes);
  uint8_t* s = static_cast<uint8_t*>(scales);
  if (d.layout == HMM_MX4_ROWS) {
    const RowsGrid g = rows_grid(p.rt * 128, (p.kt + 1) / 2);
    auto kern = f32 ? (g.u == 1   ? mx4_quantize_rows_kernel<true, 1>
                       : g.u == 2 ? mx4_quantize_rows_kernel<true, 2>
                       : g.u == 3 ? mx4_quantize_rows_kernel<true, 3>
                                  : mx4_quantize_rows_kernel<true, 4>)
                    : (g.u == 1   ? mx4_quantize_rows_kernel<false, 1>
                       : g.u == 2 ? mx4_quantize_rows_kernel<false, 2>
                       : g.u == 3 ? mx4_quantize_rows_kernel<false, 3>
                                  : mx4_quantize_rows_kernel<false, 4>);
    return launch_kernel(kern, g.grid, MX_THREADS, 0, st, pdl, 1, values, d.rows, d.cols, d.ld,
                         p.kt, c, s);
  }
  const dim3 grid(static_cast<unsigned>(p.kt), static_cast<unsigned>(p.rt * 2),
                  static_cast<unsigned>(d.batch));
  auto kern = f32 ? mx4_quantize_columns_kernel<true> : mx4_quantize_columns_kernel<false>;
  return launch_kernel(kern, grid, TW_THREADS, 0, st, pdl, 1, values, d.rows, p.stored, d.cols,
                       p.kt, p.gate_up, c, s);
}

cudaError_t launch_mx4_dequantize(const hmm_mx4& d, const void* codes, const void* scales,
                                  void* values, cudaStream_t st, bool pdl) {
  const Mx4Plan p = mx4_plan(d);
  const bool f32 = d.dtype == HMM_DTYPE_F32;
  const uint8_t* c = static_cast<const uint8_t*>(codes);
  const uint8_t* s = static_cast<const uint8_t*>(scales);
  if (d.layout == HMM_MX4_ROWS) {
    const RowsGrid g = rows_grid(d.rows, (d.cols + (f32 ? 127 : 255)) / (f32 ? 128 : 256));
    auto kern = f32 ? (g.u == 1   ? mx4_dequantize_rows_kernel<true, 1>
                       : g.u == 2 ? mx4_dequantize_rows_kernel<true, 2>
                       : g.u == 3 ? mx4_dequantize_rows_kernel<true, 3>
                                  : mx4_dequantize_rows_kernel<true, 4>)
                    : (g.u == 1   ? mx4_dequantize_rows_kernel<false, 1>
                       : g.u == 2 ? mx4_dequantize_rows_kernel<false, 2>
                       : g.u == 3 ? mx4_dequantize_rows_kernel<false, 3>
                                  : mx4_dequantize_rows_kernel<false, 4>);
    return launch_kernel(kern, g.grid, MX_THREADS, 0, st, pdl, 1, c, s, d.rows, d.cols, d.ld, p.kt,
                         values);
  }
  const dim3 grid(static_cast<unsigned>(p.kt),
                  static_cast<unsigned>((p.stored + 4 * TW_ROWS - 1) / (4 * TW_ROWS)),
                  static_cast<unsigned>(d.batch));
  auto kern = f32 ? mx4_dequantize_columns_kernel<true> : mx4_dequantize_columns_kernel<false>;
  return launch_kernel(kern, grid, TW_THREADS, 0, st, pdl, 1, c, s, d.rows, p.stored, d.cols, p.kt,
                       p.gate_up, values);
}

}  // namespace hmm
