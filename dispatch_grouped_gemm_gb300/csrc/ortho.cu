// ortho.cu -- the orthogonalised update of a stack of weight matrices by
// Newton-Schulz products, as the Muon optimiser takes it.
//
//   X_0 = G / (|G|_F + eps);  A = X X^T, B = b A + c A A, X <- a X + B X   (n steps)
//   result = scale X_n
// on the smaller side: for more rows than columns A = X^T X and X <- a X + X B, the
// same values without a transposed copy (the products read either order).  Each
// step maps every singular value s of X to a s + b s^3 + c s^5 and leaves the
// singular vectors alone.
//
// Precision.  The products run on the tensor cores in fp16 with fp32 sums, three
// per step (gmm_open.cu).  A step multiplies small singular values by a (3.4 with
// the usual coefficients, 485 in five steps), and so what rounding X to 16 bits adds
// in directions that X hardly has: with X in fp16 alone a matrix of rank 64 + noise
// comes out 2 % off, with bf16 18 %.  The rounding of A and B, and of the X inside
// B X, only turns directions that X has, and is not multiplied.  So X is kept as
// hi + lo, two fp16 (22 bits), and the epilogue adds a (hi + lo) in fp32, while the
// products read hi alone: 0.2 % off for every spectrum, most of it the result's own
// rounding to bf16 (0.17 %).  Three bits more than bf16 at the same rate are why it
// is fp16: its range is enough, because every matrix here has a known bound.
//   Bounds.  All singular values of X lie in [0, u] with u = 1 at first and then
// the largest |a s + b s^3 + c s^5| on [0, u]; an element is at most the largest
// singular value.  From that each matrix gets its power-of-two scale on the host,
// at most 2^14 in storage, a quarter of fp16's range.  B is stored as B + d I with d
// = -(b + c): where X is nearly orthogonal its diagonal is near b + c, and without
// it the rounding of the diagonal alone costs as much as all others; the epilogue
// takes d hi off again.
//
// Bounds of time: 3 m^2 n + m^3 operations per step (A and A A are symmetric: one
// triangle of tiles each) at the tensor rate; between them X moves four times
// (hi, lo in and out).  The norm and the first conversion read G twice.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "gmm_open.h"

namespace hmm {

namespace {

constexpr int ORTHO_THREADS = 256;
constexpr int64_t ORTHO_PIECE = 32768;  // elements per block and matrix, at least
constexpr int ORTHO_MAX_PIECES = 256;

// Sums of squares in three ranges, so that neither the squares of large elements
// overflow nor those of small ones vanish.
struct Sums {
  float big, mid, small;
};
constexpr float SUM_BIG = 0x1p60f;  // squares of larger elements scaled by 2^-160
constexpr float SUM_BIG_SCALE = 0x1p-80f;
constexpr float SUM_SMALL = 0x1p-50f;  // squares of smaller ones by 2^160
constexpr float SUM_SMALL_SCALE = 0x1p80f;

__device__ __forceinline__ void sum_add(Sums& s, float v) {
  const float a = fabsf(v);
  if (a > SUM_BIG) {
    const float t = a * SUM_BIG_SCALE;
    s.big = fmaf(t, t, s.big);
  } else if (a < SUM_SMALL) {
    const float t = a * SUM_SMALL_SCALE;
    s.small = fmaf(t, t, s.small);
  } else {
    s.mid = fmaf(v, v, s.mid);  // NaN comes here
  }
}

__device__ __forceinline__ float ortho_get(float v) { return v; }
__device__ __forceinline__ float ortho_get(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float ortho_get(__half v) { return __half2float(v); }

struct OrthoArgs {
  const void* g;
  int64_t M, N, ld, stride;
  int pieces;
  int64_t rows_per_piece;
  Sums* sums;  // [batch][pieces]
  __half *hi, *lo;
  int64_t ld_x;
  float eps;
  float scale;  // 2^e of the stored X
};

// Eight elements of a row at a time (VEC: 16-byte aligned rows), the last ones of a
// row one by one.
template <typename T, bool VEC, typename F>
__device__ __forceinline__ void ortho_walk(const OrthoArgs& a, const F& f) {
  const int64_t r0 = blockIdx.x * a.rows_per_piece, r1 = min(a.M, r0 + a.rows_per_piece);
  const int64_t per = (a.N + 7) / 8;
  const T* g = static_cast<const T*>(a.g) + blockIdx.y * a.stride;
  for (int64_t i = threadIdx.x; i < (r1 - r0) * per; i += ORTHO_THREADS) {
    const int64_t q = i / per, r = r0 + q, c = (i - q * per) * 8;
    const T* src = g + r * a.ld + c;
    float v[8];
    if (VEC && c + 8 <= a.N) {
      alignas(16) T t[8];
#pragma unroll
      for (int j = 0; j < static_cast<int>(8 * sizeof(T) / 16); ++j)
        reinterpret_cast<uint4*>(t)[j] = reinterpret_cast<const uint4*>(src)[j];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = ortho_get(t[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = c + j < a.N ? ortho_get(src[j]) : 0.f;
    }
    f(r, c, v);
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(ORTHO_THREADS) ortho_norm_kernel(const OrthoArgs a) {
  __shared__ Sums part[ORTHO_THREADS / 32];
  grid_dep_wait();
  grid_dep_launch();
  Sums s{0.f, 0.f, 0.f};
  ortho_walk<T, VEC>(a, [&](int64_t, int64_t, const float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) sum_add(s, v[j]);
  });
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    s.big += __shfl_xor_sync(0xffffffffu, s.big, d);
    s.mid += __shfl_xor_sync(0xffffffffu, s.mid, d);
    s.small += __shfl_xor_sync(0xffffffffu, s.small, d);
  }
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < ORTHO_THREADS / 32; ++w) {
      s.big += part[w].big;
      s.mid += part[w].mid;
      s.small += part[w].small;
    }
    a.sums[static_cast<int64_t>(blockIdx.y) * a.pieces + blockIdx.x] = s;
  }
}

// Factor of the stored X_0 of a matrix, as two floats whose product it is (alone it
// may lie outside fp32's range).  Every thread of a block.
__device__ float2 ortho_factor(const OrthoArgs& a) {
  __shared__ double part[3][ORTHO_THREADS / 32];
  double big = 0, mid = 0, small = 0;
  for (int i = threadIdx.x; i < a.pieces; i += ORTHO_THREADS) {
    const Sums s = a.sums[static_cast<int64_t>(blockIdx.y) * a.pieces + i];
    big += s.big;
    mid += s.mid;
    small += s.small;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    big += __shfl_xor_sync(0xffffffffu, big, d);
    mid += __shfl_xor_sync(0xffffffffu, mid, d);
    small += __shfl_xor_sync(0xffffffffu, small, d);
  }
  if ((threadIdx.x & 31) == 0) {
    part[0][threadIdx.x >> 5] = big;
    part[1][threadIdx.x >> 5] = mid;
    part[2][threadIdx.x >> 5] = small;
  }
  __syncthreads();
  big = mid = small = 0;
  for (int w = 0; w < ORTHO_THREADS / 32; ++w) {
    big += part[0][w];
    mid += part[1][w];
    small += part[2][w];
  }
  const double norm = sqrt(big * 0x1p160 + mid + small * 0x1p-160);
  const double f = static_cast<double>(a.scale) / (norm + static_cast<double>(a.eps));
  // a matrix of zeros stays zeros, with eps 0 too
  if (norm == 0.0) return make_float2(0.f, 0.f);
  if (!(f > 0.0) || isinf(f)) return make_float2(static_cast<float>(f), 1.f);  // NaN, 0, inf
  int e = 0;
  const double m = frexp(f, &e);
  const int e1 = e / 2;
  return make_float2(static_cast<float>(ldexp(1.0, e1)), static_cast<float>(ldexp(m, e - e1)));
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(ORTHO_THREADS) ortho_first_kernel(const OrthoArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const float2 f = ortho_factor(a);
  __half* hi = a.hi + blockIdx.y * a.M * a.ld_x;
  __half* lo = a.lo + blockIdx.y * a.M * a.ld_x;
  ortho_walk<T, VEC>(a, [&](int64_t r, int64_t c, const float (&v)[8]) {
    alignas(16) __half h[8], l[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = v[j] * f.x * f.y;
      h[j] = __float2half_rn(x);
      l[j] = __float2half_rn(x - __half2float(h[j]));
    }
    // (rows of X are padded to eight elements)
    *reinterpret_cast<uint4*>(hi + r * a.ld_x + c) = *reinterpret_cast<const uint4*>(h);
    *reinterpret_cast<uint4*>(lo + r * a.ld_x + c) = *reinterpret_cast<const uint4*>(l);
  });
}

template <typename T>
cudaError_t launch_first(const GemmEnv& env, const OrthoArgs& a, int64_t batch) {
  const bool vec = (reinterpret_cast<uintptr_t>(a.g) & 15u) == 0 &&
                   a.ld * sizeof(T) % 16 == 0 && a.stride * sizeof(T) % 16 == 0;
  const dim3 grid(static_cast<unsigned>(a.pieces), static_cast<unsigned>(batch));
  cudaError_t e =
      launch_kernel(vec ? ortho_norm_kernel<T, true> : ortho_norm_kernel<T, false>, grid,
                    ORTHO_THREADS, 0, env.stream, env.pdl, 1, a);
  if (e != cudaSuccess) return e;
  return launch_kernel(vec ? ortho_first_kernel<T, true> : ortho_first_kernel<T, false>, grid,
                       ORTHO_THREADS, 0, env.stream, env.pdl, 1, a);
}

int64_t round8(int64_t v) { return (v + 7) / 8 * 8; }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Largest |f| on [0, u], from a fine grid and with its spacing's margin.
template <typename F>
double largest(double u, const F& f) {
  constexpr int n = 1024;
  double m = 0;
  for (int i = 0; i <= n; ++i) m = std::max(m, std::fabs(f(u * i / n)));
  return m * 1.01;
}

// Exponent e with u 2^e at most 2^14.
int scale_for(double u) { return static_cast<int>(std::floor(14 - std::log2(std::max(u, 1e-3)))); }

struct OrthoStep {
  float alpha_a;                     // A
  float alpha_b, beta_b, gamma_b;    // B + d I
  float alpha_x, beta_x, gamma_x;    // X
};

// The steps' factors; false if the coefficients let X grow past 2^20.
bool ortho_steps(const hmm_ortho& d, OrthoStep* out) {
  constexpr double most = 1048576.0;
  double u = 1.0;
  int ex = scale_for(u);
  for (int i = 0; i < d.steps; ++i) {
    const double a = d.coefficients[3 * i], b = d.coefficients[3 * i + 1],
                 c = d.coefficients[3 * i + 2];
    // (NaN fails the comparison)
    if (!(std::fabs(a) <= most && std::fabs(b) <= most && std::fabs(c) <= most)) return false;
    const double shift = -(b + c);
    const double ub = largest(u, [&](double s) { return b * s * s + c * s * s * s * s + shift; });
    const double un = largest(u, [&](double s) { return s * (a + b * s * s + c * s * s * s * s); });
    if (!(ub <= most && un <= most)) return false;
    const int ea = scale_for(u * u), eb = scale_for(ub), en = scale_for(un);
    OrthoStep& s = out[i];
    s.alpha_a = static_cast<float>(std::ldexp(1.0, ea - 2 * ex));
    s.alpha_b = static_cast<float>(std::ldexp(c, eb - 2 * ea));
    s.beta_b = static_cast<float>(std::ldexp(b, eb - ea));
    s.gamma_b = static_cast<float>(std::ldexp(shift, eb));
    const bool last = i == d.steps - 1;
    const double k = last ? d.scale : 1.0;
    const int e = last ? 0 : en;
    s.alpha_x = static_cast<float>(k * std::ldexp(1.0, e - eb - ex));
    s.beta_x = static_cast<float>(k * std::ldexp(a - shift, e - ex));
    s.gamma_x = static_cast<float>(k * std::ldexp(a, e - ex));
    u = un;
    ex = en;
  }
  return true;
}

}  // namespace

int check_ortho(const hmm_ortho* d) {
  if (!d || !d->coefficients) return HMM_ERR_ARG;
  for (int dt : {d->dtype, d->out_dtype})
    if (dt != HMM_DTYPE_BF16 && dt != HMM_DTYPE_F32 && dt != HMM_DTYPE_F16) return HMM_ERR_DTYPE;
  if (d->out_dtype == HMM_DTYPE_F32) return HMM_ERR_DTYPE;
  if (d->batch < 0 || d->batch > 65535 || d->M <= 0 || d->N <= 0 || d->M > (1 << 17) ||
      d->N > (1 << 17) || d->ld < d->N || d->ld > (1 << 30) || d->stride < 0 ||
      d->stride > (int64_t(1) << 48))
    return HMM_ERR_SHAPE;
  if (d->steps < 1 || d->steps > HMM_ORTHO_MAX_STEPS) return HMM_ERR_ARG;
  if (!(d->eps >= 0.f) || std::isinf(d->eps) || !std::isfinite(d->scale)) return HMM_ERR_ARG;
  OrthoStep s[HMM_ORTHO_MAX_STEPS];
  return ortho_steps(*d, s) ? HMM_OK : HMM_ERR_ARG;
}

OrthoPlan ortho_plan(const hmm_ortho& d) {
  OrthoPlan p;
  p.m = std::min(d.M, d.N);
  p.ld_x = round8(d.N);
  p.ld_a = round8(p.m);
  const int64_t n = d.M * round8(d.N);
  p.pieces = static_cast<int>(
      std::min<int64_t>({(n + ORTHO_PIECE - 1) / ORTHO_PIECE, ORTHO_MAX_PIECES, d.M}));
  p.rows_per_piece = (d.M + p.pieces - 1) / p.pieces;
  const size_t x = up256(static_cast<size_t>(d.batch) * d.M * p.ld_x * 2);
  const size_t a = up256(static_cast<size_t>(d.batch) * p.m * p.ld_a * 2);
  size_t o = up256(static_cast<size_t>(d.batch) * p.pieces * sizeof(Sums));
  for (int i = 0; i < 4; ++i) {  // hi, lo of two X
    p.off_x[i] = o;
    o += x;
  }
  p.off_a = o;
  p.off_b = o + a;
  p.bytes = o + 2 * a;
  return p;
}

int launch_ortho(const GemmEnv& env, const hmm_ortho& d, const OrthoPlan& p, const void* g,
                 void* out, uint8_t* ws) {
  OrthoStep steps[HMM_ORTHO_MAX_STEPS];
  if (!ortho_steps(d, steps)) return HMM_ERR_ARG;
  OrthoArgs a{};
  a.g = g;
  a.M = d.M;
  a.N = d.N;
  a.ld = d.ld;
  a.stride = d.stride;
  a.pieces = p.pieces;
  a.rows_per_piece = p.rows_per_piece;
  a.sums = reinterpret_cast<Sums*>(ws);
  a.hi = reinterpret_cast<__half*>(ws + p.off_x[0]);
  a.lo = reinterpret_cast<__half*>(ws + p.off_x[1]);
  a.ld_x = p.ld_x;
  a.eps = d.eps;
  a.scale = static_cast<float>(std::ldexp(1.0, scale_for(1.0)));
  const cudaError_t e = d.dtype == HMM_DTYPE_F32   ? launch_first<float>(env, a, d.batch)
                        : d.dtype == HMM_DTYPE_F16 ? launch_first<__half>(env, a, d.batch)
                                                   : launch_first<__nv_bfloat16>(env, a, d.batch);
  if (e != cudaSuccess) return HMM_ERR_CUDA;
  const bool wide = d.M <= d.N;
  const int64_t m = p.m, lx = p.ld_x, la = p.ld_a;
  const OpenOperand A{ws + p.off_a, m, m, d.batch, la, m * la};
  const OpenOperand B{ws + p.off_b, m, m, d.batch, la, m * la};
  for (int i = 0; i < d.steps; ++i) {
    const OrthoStep& s = steps[i];
    const int from = (i & 1) * 2, to = 2 - from;
    const OpenOperand X{ws + p.off_x[from], d.M, d.N, d.batch, lx, d.M * lx};
    const bool last = i == d.steps - 1;
    // A: rows (wide) or columns of X against each other
    OpenStack q{};
    q.a = q.b = X;
    q.a_mn = q.b_mn = !wide;
    q.M = q.N = m;
    q.K = wide ? d.N : d.M;
    q.epi = OPEN_EPI_GRAM;
    q.alpha = s.alpha_a;
    q.out = ws + p.off_a;
    q.ld_in = la;
    int rc = launch_open_stack(env, q);
    if (rc != HMM_OK) return rc;
    // B + d I
    q = OpenStack{};
    q.a = q.b = A;
    q.M = q.N = q.K = m;
    q.epi = OPEN_EPI_POLY;
    q.alpha = s.alpha_b;
    q.beta = s.beta_b;
    q.gamma = s.gamma_b;
    q.in_hi = ws + p.off_a;
    q.ld_in = la;
    q.out = ws + p.off_b;
    rc = launch_open_stack(env, q);
    if (rc != HMM_OK) return rc;
    // X: B X (X's rows are the contraction) or X B
    q = OpenStack{};
    q.a = wide ? B : X;
    q.b = wide ? X : B;
    q.b_mn = wide;
    q.M = d.M;
    q.N = d.N;
    q.K = m;
    q.epi = last ? OPEN_EPI_LAST : OPEN_EPI_UPDATE;
    q.alpha = s.alpha_x;
    q.beta = s.beta_x;
    q.gamma = s.gamma_x;
    q.in_hi = ws + p.off_x[from];
    q.in_lo = ws + p.off_x[from + 1];
    q.ld_in = lx;
    q.out = last ? out : ws + p.off_x[to];
    q.out_lo = last ? nullptr : ws + p.off_x[to + 1];
    q.out_f16 = last ? d.out_dtype == HMM_DTYPE_F16 : 1;
    rc = launch_open_stack(env, q);
    if (rc != HMM_OK) return rc;
  }
  return HMM_OK;
}

}  // namespace hmm
