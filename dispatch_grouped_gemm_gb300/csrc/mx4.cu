// mx4.cu -- values (bf16 or fp32) to microscaled 4-bit operands and back: rows
// with the contraction contiguous, and stacks of expert weights [cols, rows]
// that are transposed on the way.  Bound by memory: a value is read once and
// half a byte plus a 32nd of a byte written (and the other way round).
#include "mx4.cuh"

namespace hmm {

namespace {

constexpr int MX_THREADS = 256;

template <bool F32>
__device__ __forceinline__ void ld_values8(const void* p, int64_t i, float (&v)[8]) {
  if constexpr (F32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = q[0], b = q[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(u[j] << 16);
      v[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
    }
  }
}

template <bool F32>
__device__ __forceinline__ void st_values8(void* p, int64_t i, const float (&v)[8]) {
  if constexpr (F32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint4 q;
    uint32_t* u = reinterpret_cast<uint32_t*>(&q);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      u[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = q;
  }
}

// The 8 values of one thread and those of its three neighbours are one block.
__device__ __forceinline__ uint32_t quad_scale(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  return mx_scale_byte(m);
}

}  // namespace

// One thread per 8 elements; rows and columns run over the scale tiles'
// 128 x 128, so that the padding scales are written as zeros too.
template <bool F32>
__global__ void __launch_bounds__(MX_THREADS)
    mx4_quantize_rows_kernel(const void* __restrict__ src, int64_t rows, int64_t cols, int64_t ld,
                             int64_t kt, uint8_t* __restrict__ codes,
                             uint8_t* __restrict__ scales) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * MX_THREADS + threadIdx.x;
  const int64_t g = i % (kt * 16), r = i / (kt * 16);
  grid_dep_wait();
  grid_dep_launch();
  const int64_t c = g * 8;
  float v[8] = {};
  if (r < rows && c < cols) ld_values8<F32>(src, r * ld + c, v);
  const uint32_t s = quad_scale(v);
  const float inv = mx_inverse_scale(s);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] *= inv;
  const int64_t kp = (cols + 31) / 32 * 32;
  if (r < rows && c < kp)
    *reinterpret_cast<uint32_t*>(codes + r * (kp / 2) + c / 2) = mx_codes8(v);
  if ((g & 3) == 0 && r < (rows + 127) / 128 * 128)
    scales[mx_scale_offset(r, g >> 2, kt)] = static_cast<uint8_t>(s);
}

template <bool F32>
__global__ void __launch_bounds__(MX_THREADS)
    mx4_dequantize_rows_kernel(const uint8_t* __restrict__ codes,
                               const uint8_t* __restrict__ scales, int64_t rows, int64_t cols,
                               int64_t ld, int64_t kt, void* __restrict__ dst) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * MX_THREADS + threadIdx.x;
  const int64_t n8 = cols / 8;
  const int64_t g = i % n8, r = i / n8;
  grid_dep_wait();
  grid_dep_launch();
  if (r >= rows) return;
  const int64_t kp = (cols + 31) / 32 * 32;
  float v[8];
  mx_values8(*reinterpret_cast<const uint32_t*>(codes + r * (kp / 2) + g * 4),
             mx_scale(scales[mx_scale_offset(r, g >> 2, kt)]), v);
  st_values8<F32>(dst, r * ld + g * 8, v);
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
  const int64_t base = e * cols * n;
  float v[2][32];
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    v[0][k] = v[1][k] = 0.0f;
    if (c >= 0 && kb + k < cols) {
      const int64_t at = base + (kb + k) * n + c;
      if constexpr (F32) {
        const float2 f = *reinterpret_cast<const float2*>(static_cast<const float*>(src) + at);
        v[0][k] = f.x;
        v[1][k] = f.y;
      } else {
        const uint32_t u =
            *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(src) + at);
        v[0][k] = __uint_as_float(u << 16);
        v[1][k] = __uint_as_float(u & 0xFFFF0000u);
      }
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 32; ++k) m = max(m, __float_as_uint(v[h][k]) & 0x7FFFFFFFu);
    const uint32_t s = mx_scale_byte(m);
    const float inv = mx_inverse_scale(s);
    uint32_t q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = v[h][8 * j + k] * inv;
      q[j] = mx_codes8(w);
    }
    const int row = 2 * lane + h;
    *reinterpret_cast<uint4*>(s_codes + row * TW_PITCH + warp * 16) =
        make_uint4(q[0], q[1], q[2], q[3]);
    s_scales[row * 4 + warp] = static_cast<uint8_t>(s);
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

template <bool F32>
__global__ void __launch_bounds__(TW_THREADS)
    mx4_dequantize_columns_kernel(const uint8_t* __restrict__ codes,
                                  const uint8_t* __restrict__ scales, int64_t n, int64_t stored,
                                  int64_t cols, int64_t kt, bool gate_up,
                                  void* __restrict__ dst) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t e = blockIdx.z, d0 = static_cast<int64_t>(blockIdx.y) * TW_ROWS;
  const int64_t kb = static_cast<int64_t>(blockIdx.x) * 128 + warp * 32;
  const int64_t kp = (cols + 31) / 32 * 32;
  grid_dep_wait();
  grid_dep_launch();
  const int64_t d = d0 + 2 * lane;
  const int64_t c = source_column(d, n, gate_up);
  if (c < 0 || kb >= cols) return;
  const int64_t rt = (stored + 127) / 128;
  float v[2][32];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint4 q =
        *reinterpret_cast<const uint4*>(codes + (e * stored + d + h) * (kp / 2) + kb / 2);
    const float s = mx_scale(
        scales[e * rt * kt * MX_TILE_BYTES + mx_scale_offset(d + h, kb / 32, kt)]);
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float w[8];
      mx_values8(u[j], s, w);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[h][8 * j + k] = w[k];
    }
  }
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    if (kb + k >= cols) break;
    const int64_t at = e * cols * n + (kb + k) * n + c;
    if constexpr (F32) {
      *reinterpret_cast<float2*>(static_cast<float*>(dst) + at) = make_float2(v[0][k], v[1][k]);
    } else {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[0][k], v[1][k]);
      *reinterpret_cast<__nv_bfloat162*>(static_cast<uint16_t*>(dst) + at) = b;
    }
  }
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
    // one thread per 8 elements of whole 128 x 128 tiles
    if (d->cols > (1 << 24) || d->rows > (int64_t(1) << 38) / ((d->cols + 127) / 128 * 128))
      return HMM_ERR_SHAPE;
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
    const int64_t threads = p.rt * 128 * p.kt * 16;
    const unsigned grid = static_cast<unsigned>((threads + MX_THREADS - 1) / MX_THREADS);
    auto kern = f32 ? mx4_quantize_rows_kernel<true> : mx4_quantize_rows_kernel<false>;
    return launch_kernel(kern, grid, MX_THREADS, 0, st, pdl, 1, values, d.rows, d.cols, d.ld, p.kt,
                         c, s);
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
    const int64_t threads = d.rows * (d.cols / 8);
    const unsigned grid = static_cast<unsigned>((threads + MX_THREADS - 1) / MX_THREADS);
    auto kern = f32 ? mx4_dequantize_rows_kernel<true> : mx4_dequantize_rows_kernel<false>;
    return launch_kernel(kern, grid, MX_THREADS, 0, st, pdl, 1, c, s, d.rows, d.cols, d.ld, p.kt,
                         values);
  }
  const dim3 grid(static_cast<unsigned>(p.kt),
                  static_cast<unsigned>((p.stored + TW_ROWS - 1) / TW_ROWS),
                  static_cast<unsigned>(d.batch));
  auto kern = f32 ? mx4_dequantize_columns_kernel<true> : mx4_dequantize_columns_kernel<false>;
  return launch_kernel(kern, grid, TW_THREADS, 0, st, pdl, 1, c, s, d.rows, p.stored, d.cols, p.kt,
                       p.gate_up, values);
}

}  // namespace hmm
