// gate.cu -- the router in front of the experts: scores of E experts per
// token, group-limited top-k selection and the routing weights, forward and
// backward.
//
//   p = softmax(l) or sigmoid(l)                                    [T, E]
//   key = p + bias (softmax without a bias, one group or groups counted by one
//         key: l itself, whose order is that of p)
//   groups > 1: a group of E / groups experts counts by the sum of its
//         group_top best keys; the topk_groups best groups stay open
//   topk_ids = the K best keys of the open groups, best first, ties to the
//         lowest index
//   topk_weights = scale * p[topk_ids], over sum_k p[topk_ids] with renormalize
//
// Renormalised softmax weights are the softmax of the K selected logits: they
// come from these alone, so that scores too small for fp32 (a bias can choose
// them) keep their weights and their gradient.
//
// One warp per token.  Lane i holds the c = ceil(E / 32) consecutive experts
// from c i in registers, so that the lowest of equal keys is in the lowest
// lane, a row of logits is read once with vector loads, and (E a multiple of
// 32, groups a power of two) a group is a run of 32 / groups lanes.
#include <cuda_bf16.h>

#include <algorithm>

#include "hmm_internal.h"

namespace hmm {

namespace {

constexpr int GATE_WARPS = 4;  // tokens per block at a time
constexpr unsigned FULL = 0xffffffffu;

template <bool BF16>
__device__ __forceinline__ float ld_logit(const void* p, int64_t i) {
  if constexpr (BF16)
    return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
  else
    return static_cast<const float*>(p)[i];
}

// The lane's experts base .. base + c - 1 of a row starting at element `row`;
// -inf past E.  VEC: c == C, every chunk whole and 16-byte aligned.
template <int C, bool BF16, bool VEC>
__device__ __forceinline__ void ld_chunk(const void* p, int64_t row, int base, int c, int E,
                                         float (&l)[C]) {
  if constexpr (VEC && !BF16 && C % 4 == 0) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + row + base);
#pragma unroll
    for (int j = 0; j < C / 4; ++j) {
      const float4 v = q[j];
      l[4 * j] = v.x;
      l[4 * j + 1] = v.y;
      l[4 * j + 2] = v.z;
      l[4 * j + 3] = v.w;
    }
  } else if constexpr (VEC && BF16 && C % 8 == 0) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + row + base);
#pragma unroll
    for (int j = 0; j < C / 8; ++j) {
      const uint4 v = q[j];
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        l[8 * j + 2 * k] = __uint_as_float(u[k] << 16);
        l[8 * j + 2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < C; ++j)
      l[j] = j < c && base + j < E ? ld_logit<BF16>(p, row + base + j) : -INFINITY;
  }
}

template <int C, bool BF16, bool VEC>
__device__ __forceinline__ void st_chunk(void* p, int64_t row, int base, int c, int E,
                                         const float (&v)[C]) {
  if constexpr (VEC && !BF16 && C % 4 == 0) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + row + base);
#pragma unroll
    for (int j = 0; j < C / 4; ++j)
      q[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  } else if constexpr (VEC && BF16 && C % 8 == 0) {
    uint4* q = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + row + base);
#pragma unroll
    for (int j = 0; j < C / 8; ++j) {
      uint32_t u[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[8 * j + 2 * k], v[8 * j + 2 * k + 1]);
        u[k] = *reinterpret_cast<const uint32_t*>(&b);
      }
      q[j] = make_uint4(u[0], u[1], u[2], u[3]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < C; ++j)
      if (j < c && base + j < E) {
        if constexpr (BF16)
          static_cast<__nv_bfloat16*>(p)[row + base + j] = __float2bfloat16_rn(v[j]);
        else
          static_cast<float*>(p)[row + base + j] = v[j];
      }
  }
}

__device__ __forceinline__ float ld_w(const void* w, int64_t i, int f32) {
  return f32 ? static_cast<const float*>(w)[i]
             : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
}

// Order-preserving map of a float to an integer above CLOSED: -inf is the
// least, NaN the greatest (the addition returns the one positive NaN, and +0
// for -0); and back.
constexpr int CLOSED = static_cast<int>(0x80000000u);
__device__ __forceinline__ int order_key(float v) {
  const int u = __float_as_int(v + 0.0f);
  return u ^ ((u >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float key_value(int k) {
  return __int_as_float(k ^ ((k >> 31) & 0x7fffffff));
}

template <int L = 32>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) v += __shfl_xor_sync(FULL, v, d);
  return v;
}

template <int L = 32>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, d));
  return v;
}
// The largest of some logits of a row as its exponentials subtract it: 0 where
// they are all -inf, closed experts, whose exponentials are 0.
__device__ __forceinline__ float row_shift(float m) { return m == -INFINITY ? 0.0f : m; }
__device__ __forceinline__ float nonzero(float sum) { return sum == 0.0f ? 1.0f : sum; }

// 1 / (1 + exp(-l)) with the accurate exponential and a correctly rounded
// reciprocal: the selection compares these values, so they are rounded as the
// formula's own fp32 evaluation rounds them.
__device__ __forceinline__ float sigmoid_rn(float l) { return __frcp_rn(1.0f + expf(-l)); }

// Largest logit of a row.  (A NaN turns the row's sum into NaN.)
template <int C>
__device__ __forceinline__ float row_max(const float (&l)[C]) {
  float m = l[0];
#pragma unroll
  for (int j = 1; j < C; ++j) m = fmaxf(m, l[j]);
  return row_shift(lanes_max(m));
}

template <int C>
__device__ __forceinline__ float exp_row(const float (&l)[C], float m, float (&p)[C]) {
  float z = 0.0f;
#pragma unroll
  for (int j = 0; j < C; ++j) {
    p[j] = expf(l[j] - m);
    z += p[j];
  }
  return nonzero(lanes_sum(z));
}

// Lanes per token in the kernels for many tokens (up to 40 experts per lane).
__host__ __device__ constexpr int many_lanes(int E) {
  return E <= 160 ? 4 : (E <= 256 ? 8 : (E <= 512 ? 16 : 32));
}

// Sum over a row's p in the order of gate_forward_many_kernel: lane q of
// many_lanes(E) adds the experts (i LT + q) 4 .. + 3, then the lanes add theirs.
// Keys that hold the sum's rounding are then the same in a long batch and in a
// short one, and with them the selection.  row: 33 c values (a place left free
// after every 32, so that lanes do not meet in a bank).  (Softmax with a bias, us
// with the butterfly of exp_row alone and with this: E = 256, T = 1 2.8 and 3.3, T =
// 2000 4.6 and 5.3; E = 1024, T = 2000 17.7 and 20.8.)
template <int C>
__device__ __forceinline__ float sum_like_many(const float (&p)[C], int base, int c, int E,
                                               int lane, float* row) {
#pragma unroll
  for (int j = 0; j < C; ++j)
    if (j < c && base + j < E) row[base + j + ((base + j) >> 5)] = p[j];
  __syncwarp();
  const int lanes = many_lanes(E);
  float z = 0.0f;
  for (int e = 4 * (lane & (lanes - 1)); e < E; e += 4 * lanes) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (e + r < E) z += row[e + r + (e >> 5)];
  }
  __syncwarp();
  for (int d = lanes / 2; d > 0; d >>= 1) z += __shfl_xor_sync(FULL, z, d);
  return nonzero(z);
}

}  // namespace

struct GateArgs {
  int64_t T, ld;
  int E, K, c, groups, topk_groups, group_top;
  int lane_groups;  // groups are runs of 32 / groups lanes
  int weights_f32, renorm;
  float scale;
};

namespace {

// Worth of group `lane` from the keys of the whole row (any group shape): the
// group_top best keys by repeated selection.
__device__ __noinline__ int group_worth(const int* keys, int n, int top) {
  const int* k = keys + (threadIdx.x & 31) * n;
  float worth = 0.0f;
  int last = 0x7fffffff;
  int last_i = -1;
  for (int r = 0; r < top; ++r) {
    int bk = CLOSED, bi = 0;
    for (int i = 0; i < n; ++i) {
      const bool taken = r > 0 && (k[i] > last || (k[i] == last && i <= last_i));
      if (!taken && k[i] > bk) {
        bk = k[i];
        bi = i;
      }
    }
    last = bk;
    last_i = bi;
    worth = r == 0 ? key_value(bk) : worth + key_value(bk);
  }
  return order_key(worth);
}

// Closes the experts of all but the topk_groups best groups.
template <int C>
__device__ __forceinline__ void keep_groups(const GateArgs& a, int (&key)[C], int lane,
                                            int base, int* smem) {
  if (a.lane_groups) {
    const int L = 32 / a.groups;  // lanes per group
    int k1 = key[0], k2 = CLOSED;
#pragma unroll
    for (int j = 1; j < C; ++j) {
      k2 = max(k2, min(k1, key[j]));
      k1 = max(k1, key[j]);
    }
    for (int d = 1; d < L; d <<= 1) {
      const int o1 = __shfl_xor_sync(FULL, k1, d), o2 = __shfl_xor_sync(FULL, k2, d);
      k2 = max(min(k1, o1), max(k2, o2));
      k1 = max(k1, o1);
    }
    const int worth = a.group_top == 1 ? k1 : order_key(key_value(k1) + key_value(k2));
    const int g = lane / L;
    int better = 0;  // groups that come before this one
    for (int x = 1; x < a.groups; ++x) {
      const int o = __shfl_xor_sync(FULL, worth, x * L);
      better += o > worth || (o == worth && (g ^ x) < g);
    }
    if (better >= a.topk_groups) {
#pragma unroll
      for (int j = 0; j < C; ++j) key[j] = CLOSED;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < C; ++j)
    if (j < a.c && base + j < a.E) smem[base + j] = key[j];
  __syncwarp();
  const int n = a.E / a.groups;
  int worth = lane < a.groups ? group_worth(smem, n, a.group_top) : CLOSED;
  __syncwarp();
  uint32_t open = 0;
  for (int r = 0; r < a.topk_groups; ++r) {
    const int best = __reduce_max_sync(FULL, worth);
    const int g = __ffs(__ballot_sync(FULL, worth == best)) - 1;
    open |= 1u << g;
    if (lane == g) worth = CLOSED;
  }
#pragma unroll
  for (int j = 0; j < C; ++j)
    if (base + j < a.E && !((open >> ((base + j) / n)) & 1u)) key[j] = CLOSED;
}

}  // namespace

template <int C, bool BF16, bool SIG, bool VEC>
__global__ void __launch_bounds__(GATE_WARPS * 32)
    gate_forward_kernel(const GateArgs a, const void* __restrict__ logits,
                        const float* __restrict__ bias, int32_t* __restrict__ ids,
                        void* __restrict__ weights, float* __restrict__ scores) {
  // per warp [33 c] (groups that are no lane runs, softmax keys that are no logits)
  extern __shared__ int gate_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int base = lane * a.c;
  const bool by_logit = !SIG && bias == nullptr && a.group_top == 1;
  grid_dep_wait();
  grid_dep_launch();
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * GATE_WARPS + warp; t < a.T;
       t += static_cast<int64_t>(gridDim.x) * GATE_WARPS) {
    float l[C], p[C];
    int key[C];
    ld_chunk<C, BF16, VEC>(logits, t * a.ld, base, a.c, a.E, l);
    float m = 0.0f, z = 1.0f;
    if constexpr (SIG) {
#pragma unroll
      for (int j = 0; j < C; ++j) p[j] = sigmoid_rn(l[j]);
    } else {
      m = row_max(l);
      // (renormalised weights of the best logits need no sum over the row)
      if (scores || !by_logit || !a.renorm) z = exp_row(l, m, p);
      if (!by_logit)
        z = sum_like_many(p, base, a.c, a.E, lane,
                          reinterpret_cast<float*>(gate_smem) + warp * 33 * a.c);
      if (scores || !by_logit) {
#pragma unroll
        for (int j = 0; j < C; ++j) p[j] = p[j] / z;
      }
    }
    if (scores) st_chunk<C, false, VEC && C % 4 == 0>(scores, t * a.E, base, a.c, a.E, p);
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const bool in = VEC || (j < a.c && base + j < a.E);
      float v = by_logit ? l[j] : p[j];
      if (bias && in) v += __ldg(bias + base + j);
      key[j] = in ? order_key(v) : CLOSED;
    }
    if (a.groups > 1) keep_groups<C>(a, key, lane, base, gate_smem + warp * 33 * a.c);
    // K rounds: the best key of the lanes' best; lane k keeps expert k
    int bk = key[0], bj = 0;
#pragma unroll
    for (int j = 1; j < C; ++j)
      if (key[j] > bk) {
        bk = key[j];
        bj = j;
      }
    int my_id = 0;
    for (int k = 0; k < a.K; ++k) {
      const int best = __reduce_max_sync(FULL, bk);
      const int win = __ffs(__ballot_sync(FULL, bk == best)) - 1;
      const int e = __shfl_sync(FULL, base + bj, win);
      if (lane == k) my_id = e;
      if (lane == win) {
        int nk = CLOSED, nj = 0;
#pragma unroll
        for (int j = 0; j < C; ++j) {
          if (j == bj) key[j] = CLOSED;
          if (key[j] > nk) {
            nk = key[j];
            nj = j;
          }
        }
        bk = nk;
        bj = nj;
      }
    }
    // the selected scores again, from their logits
    const float lk = lane < a.K ? ld_logit<BF16>(logits, t * a.ld + my_id) : -INFINITY;
    float shift = m, div = z;
    if (!SIG && a.renorm) {
      shift = row_shift(lanes_max(lk));
      div = 1.0f;
    }
    float w = SIG ? sigmoid_rn(lk) : expf(lk - shift) / div;
    if (a.renorm) {
      w = w / nonzero(lanes_sum(w));
      if (z != z) w = z;  // a NaN that was not selected shows all the same
    }
    if (lane < a.K) {
      w *= a.scale;
      ids[t * a.K + lane] = my_id;
      if (a.weights_f32)
        static_cast<float*>(weights)[t * a.K + lane] = w;
      else
        static_cast<__nv_bfloat16*>(weights)[t * a.K + lane] = __float2bfloat16_rn(w);
    }
  }
}

namespace {

// Lane q's experts (i LT + q) 4 .. + 3 of a row starting at element `row`, LT
// lanes per token; -inf past E.
template <int N, int LT, bool BF16>
__device__ __forceinline__ void ld_token(const void* p, int64_t row, int q, int E, float (&l)[N]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const int e = (i * LT + q) * 4;
    l[4 * i] = l[4 * i + 1] = l[4 * i + 2] = l[4 * i + 3] = -INFINITY;
    if (e < E) {
      if constexpr (BF16) {
        const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + row + e);
        l[4 * i] = __uint_as_float(v.x << 16);
        l[4 * i + 1] = __uint_as_float(v.x & 0xFFFF0000u);
        l[4 * i + 2] = __uint_as_float(v.y << 16);
        l[4 * i + 3] = __uint_as_float(v.y & 0xFFFF0000u);
      } else {
        const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + row + e);
        l[4 * i] = v.x;
        l[4 * i + 1] = v.y;
        l[4 * i + 2] = v.z;
        l[4 * i + 3] = v.w;
      }
    }
  }
}

}  // namespace

// Many tokens: LT lanes per token, up to N experts per lane, so that a warp
// works on 32 / LT tokens at once.  Lane q of a token holds the experts
// (i LT + q) 4 .. + 3 (16-byte loads); its keys also sit in shared memory,
// where a round of the selection reaches them by a computed index, and the
// maxima of its runs of eight in registers.  A round serves all of the warp's
// tokens with about the instructions that the kernel above spends on one.
// Needs E to be a multiple of 4.
template <int N, int LT, bool BF16, bool SIG>
__global__ void __launch_bounds__(GATE_WARPS * 32, N > 32 ? 6 : 8)
    gate_forward_many_kernel(const GateArgs a, const void* __restrict__ logits,
                             const float* __restrict__ bias, int32_t* __restrict__ ids,
                             void* __restrict__ weights, float* __restrict__ scores) {
  constexpr int TW = 32 / LT;     // tokens per warp
  constexpr int S = N / 8;        // runs of eight per lane
  extern __shared__ int gate_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = lane % LT, tok = lane / LT;
  // per warp: the keys [32 lanes][N], the 16-byte pieces of a lane permuted so
  // that lanes do not meet in a bank; then per token the groups' worths and,
  // after them, the chosen experts
  int* wkeys = gate_smem + warp * (32 * N + TW * 32);
  int* worths = wkeys + 32 * N + tok * 32;
  int* chosen = worths;
  auto piece = [&](int of_lane, int i) {
    return reinterpret_cast<int4*>(wkeys + of_lane * N) +
           (N == 32 ? i ^ (of_lane & 7)
                    : (N == 16 ? i ^ ((of_lane >> 1) & 3) : i ^ ((of_lane >> 2) & 1)));
  };
  const bool by_logit = !SIG && bias == nullptr && a.group_top == 1;
  grid_dep_wait();
  grid_dep_launch();
  const int64_t t_raw = (static_cast<int64_t>(blockIdx.x) * GATE_WARPS + warp) * TW + tok;
  const bool live = t_raw < a.T;
  const int64_t t = live ? t_raw : a.T - 1;  // (every lane takes part in the shuffles)
  float l[N];
  ld_token<N, LT, BF16>(logits, t * a.ld, q, a.E, l);
  float m = 0.0f, z = 1.0f;
  if constexpr (!SIG) {
    m = l[0];
#pragma unroll
    for (int j = 1; j < N; ++j) m = fmaxf(m, l[j]);
#pragma unroll
    for (int d = LT / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, d));
    m = row_shift(m);
    if (scores || !by_logit || !a.renorm) {
      z = 0.0f;
#pragma unroll
      for (int j = 0; j < N; ++j) z += expf(l[j] - m);
      z = nonzero(lanes_sum<LT>(z));
    }
  }
  int seg[S];
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const int e = (i * LT + q) * 4;
    const bool in = e < a.E;
    float v[4];
    int k[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      v[r] = l[4 * i + r];
      if (SIG)
        v[r] = sigmoid_rn(v[r]);
      else if (scores || !by_logit)
        v[r] = expf(v[r] - m) / z;
    }
    if (scores && in && live)
      *reinterpret_cast<float4*>(scores + t * a.E + e) = make_float4(v[0], v[1], v[2], v[3]);
    if (bias && in) {
      const float4 b = __ldg(reinterpret_cast<const float4*>(bias + e));
      v[0] += b.x;
      v[1] += b.y;
      v[2] += b.z;
      v[3] += b.w;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) k[r] = in ? order_key(by_logit ? l[4 * i + r] : v[r]) : CLOSED;
    *piece(lane, i) = make_int4(k[0], k[1], k[2], k[3]);
    const int top = max(max(k[0], k[1]), max(k[2], k[3]));
    seg[i / 2] = i % 2 ? max(seg[i / 2], top) : top;
  }
  __syncwarp();
  if (a.groups > 1) {
    const int n = a.E / a.groups;
    // the worths: a lane per group, or several where there are fewer groups than
    // lanes (E = 300 in 4 groups, T = 65537: 112 us with one lane each, 92 so)
    int parts = 1;
    while (2 * parts * a.groups <= LT) parts *= 2;
    const int part = q % parts;
    for (int g0 = 0; g0 < a.groups; g0 += LT / parts) {
      const int g = g0 + q / parts;
      int k1 = CLOSED, k2 = CLOSED;
      if (g < a.groups) {
        if (n % 4) {  // groups that end inside a vector
          for (int e = g * n + part; e < (g + 1) * n; e += parts) {
            const int k = reinterpret_cast<const int*>(
                piece(tok * LT + (e >> 2) % LT, (e >> 2) / LT))[e & 3];
            k2 = max(k2, min(k1, k));
            k1 = max(k1, k);
          }
        } else {
          for (int e = g * n + 4 * part; e < (g + 1) * n; e += 4 * parts) {
            const int4 k = *piece(tok * LT + (e >> 2) % LT, (e >> 2) / LT);
            const int h1 = max(k.x, k.y), h2 = max(k.z, k.w);
            const int s2 = max(min(h1, h2), max(min(k.x, k.y), min(k.z, k.w)));
            const int s1 = max(h1, h2);
            k2 = max(min(k1, s1), max(k2, s2));
            k1 = max(k1, s1);
          }
        }
      }
      for (int d = parts / 2; d > 0; d >>= 1) {
        const int o1 = __shfl_xor_sync(FULL, k1, d), o2 = __shfl_xor_sync(FULL, k2, d);
        k2 = max(min(k1, o1), max(k2, o2));
        k1 = max(k1, o1);
      }
      if (g < a.groups && part == 0)
        worths[g] = a.group_top == 1 ? k1 : order_key(key_value(k1) + key_value(k2));
    }
    __syncwarp();
    uint32_t open = 0u;
    for (int g = q; g < a.groups; g += LT) {
      const int w = worths[g];
      int better = 0;
      for (int o = 0; o < a.groups; ++o) better += worths[o] > w || (worths[o] == w && o < g);
      if (better < a.topk_groups) open |= 1u << g;
    }
#pragma unroll
    for (int d = LT / 2; d > 0; d >>= 1) open |= __shfl_xor_sync(FULL, open, d);
    __syncwarp();  // (chosen takes the worths' place)
    // close the others; e / n by a reciprocal, exact for e < 1024
    const uint32_t inv = ((1u << 20) + n - 1) / n;
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const int e = (i * LT + q) * 4;
      if (n % 4 == 0) {
        const bool on = (open >> ((e * inv) >> 20)) & 1u;
        if (!on && e < a.E) *piece(lane, i) = make_int4(CLOSED, CLOSED, CLOSED, CLOSED);
      } else if (e < a.E) {
        int* k = reinterpret_cast<int*>(piece(lane, i));
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (!((open >> (((e + r) * inv) >> 20)) & 1u)) k[r] = CLOSED;
      }
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int4 x = *piece(lane, 2 * s), y = *piece(lane, 2 * s + 1);
      seg[s] = max(max(max(x.x, x.y), max(x.z, x.w)), max(max(y.x, y.y), max(y.z, y.w)));
    }
  }
  for (int k = 0; k < a.K; ++k) {
    int mine = seg[0];
#pragma unroll
    for (int s = 1; s < S; ++s) mine = max(mine, seg[s]);
    int best = mine;
#pragma unroll
    for (int d = LT / 2; d > 0; d >>= 1) best = max(best, __shfl_xor_sync(FULL, best, d));
    // the first of this lane's keys that equals its maximum, and the maximum
    // of the rest of its run
    int s0 = S - 1;
#pragma unroll
    for (int s = S - 2; s >= 0; --s)
      if (seg[s] == mine) s0 = s;
    const int4 x = *piece(lane, 2 * s0), y = *piece(lane, 2 * s0 + 1);
    const int run[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    int first = 8, rest = CLOSED;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (first == 8 && run[j] == mine)
        first = j;
      else
        rest = max(rest, run[j]);  // (an equal key behind the first stays)
    }
    const int at = 8 * s0 + first;
    const int e = (((at >> 2) * LT) + q) * 4 + (at & 3);
    int pick = mine == best ? e : 0x7fffffff;
#pragma unroll
    for (int d = LT / 2; d > 0; d >>= 1) pick = min(pick, __shfl_xor_sync(FULL, pick, d));
    if (mine == best && pick == e) {
      reinterpret_cast<int*>(piece(lane, at >> 2))[at & 3] = CLOSED;
      chosen[k] = e;
#pragma unroll
      for (int s = 0; s < S; ++s)
        if (s == s0) seg[s] = rest;
    }
  }
  __syncwarp();
  float w[32 / LT];
  float sum = 0.0f, top = -INFINITY;
#pragma unroll
  for (int x = 0; x < 32 / LT; ++x) {
    const int k = q + x * LT;
    w[x] = k < a.K ? ld_logit<BF16>(logits, t * a.ld + chosen[k]) : -INFINITY;
    top = fmaxf(top, w[x]);
  }
  float shift = m, div = z;
  if (!SIG && a.renorm) {
    shift = row_shift(lanes_max<LT>(top));
    div = 1.0f;
  }
#pragma unroll
  for (int x = 0; x < 32 / LT; ++x) {
    if (x * LT >= a.K) break;
    w[x] = SIG ? sigmoid_rn(w[x]) : expf(w[x] - shift) / div;
    sum += w[x];
  }
  if (a.renorm) sum = nonzero(lanes_sum<LT>(sum));
#pragma unroll
  for (int x = 0; x < 32 / LT; ++x) {
    const int k = q + x * LT;
    if (k < a.K && live) {
      float v = w[x];
      if (a.renorm) v = z == z ? v / sum : z;  // (a NaN that was not selected shows all the same)
      v *= a.scale;
      ids[t * a.K + k] = chosen[k];
      if (a.weights_f32)
        static_cast<float*>(weights)[t * a.K + k] = v;
      else
        static_cast<__nv_bfloat16*>(weights)[t * a.K + k] = __float2bfloat16_rn(v);
    }
  }
}

// With g_k = scale * d_topk_weights[k], n_k = p_k / sum_sel p and D = sum g n:
//   without renormalize   dp[topk_ids[k]] = g_k
//   with it               dp[topk_ids[k]] = (g_k - D) / sum_sel p
//   dp += d_scores
//   sigmoid  dl = dp p (1 - p)
//   softmax  dl = p (dp - sum dp p); the renormalised weights' part of that sum
//            is D - D = 0, so their gradient n_k (g_k - D) stays on the
//            selected experts; n is the softmax of their logits.
// This kernel: every expert has a gradient (d_scores, or softmax weights that
// are not renormalised).  One warp per token, the forward's layout; the
// selected part is scattered through shared memory.
template <int C, bool BF16, bool SIG, bool VEC>
__global__ void __launch_bounds__(GATE_WARPS * 32)
    gate_backward_kernel(const GateArgs a, const void* __restrict__ logits,
                         const int32_t* __restrict__ ids, const void* __restrict__ d_weights,
                         const float* __restrict__ d_scores, void* __restrict__ d_logits) {
  extern __shared__ int gate_smem[];  // per warp: gradients at the selected experts
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int base = lane * a.c;
  float* sd = reinterpret_cast<float*>(gate_smem) + warp * (32 * C);
#pragma unroll
  for (int j = 0; j < C; ++j) sd[lane + 32 * j] = 0.0f;
  __syncwarp();
  grid_dep_wait();
  grid_dep_launch();
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * GATE_WARPS + warp; t < a.T;
       t += static_cast<int64_t>(gridDim.x) * GATE_WARPS) {
    float l[C], p[C];
    ld_chunk<C, BF16, VEC>(logits, t * a.ld, base, a.c, a.E, l);
    int id = -1;
    float g = 0.0f, lk = -INFINITY, m = 0.0f, z = 1.0f;
    if constexpr (SIG) {
#pragma unroll
      for (int j = 0; j < C; ++j) p[j] = sigmoid_rn(l[j]);
    } else {
      m = row_max(l);
      z = 1.0f / exp_row(l, m, p);  // (p: one rounding more than the forward's division)
#pragma unroll
      for (int j = 0; j < C; ++j) p[j] *= z;
    }
    if (lane < a.K && d_weights) {
      id = ids[t * a.K + lane];
      if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.E)) id = -1;
      g = a.scale * ld_w(d_weights, t * a.K + lane, a.weights_f32);
    }
    if (id >= 0) lk = ld_logit<BF16>(logits, t * a.ld + id);
    const bool selected_softmax = !SIG && a.renorm;  // g becomes its part of dl itself
    float sum = 0.0f;  // softmax: sum dp p
    if (selected_softmax) {
      float n = expf(lk - row_shift(lanes_max(lk)));
      n /= nonzero(lanes_sum(n));
      g = n * (g - lanes_sum(g * n));
    } else {
      const float ps = id < 0 ? 0.0f : (SIG ? sigmoid_rn(lk) : expf(lk - m) * z);
      if (a.renorm) {
        const float tot = nonzero(lanes_sum(ps));
        g = (g - lanes_sum(g * (ps / tot))) / tot;
      } else {
        sum = g * ps;
      }
    }
    if (id >= 0) sd[id] = g;
    __syncwarp();
    float dp[C];
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int e = base + j;
      const bool in = VEC || (j < a.c && e < a.E);
      dp[j] = in && d_scores ? d_scores[t * a.E + e] : 0.0f;
      if constexpr (!SIG) sum += dp[j] * p[j];
    }
    if constexpr (!SIG) sum = lanes_sum(sum);
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const bool in = VEC || (j < a.c && base + j < a.E);
      const float s = in ? sd[base + j] : 0.0f;
      dp[j] = SIG ? (s + dp[j]) * p[j] * sigmoid_rn(-l[j])
                  : (selected_softmax ? s + p[j] * (dp[j] - sum) : p[j] * (s + (dp[j] - sum)));
    }
    st_chunk<C, BF16, VEC>(d_logits, t * a.E, base, a.c, a.E, dp);
    __syncwarp();
    if (id >= 0) sd[id] = 0.0f;
    __syncwarp();
  }
}

// The same for many tokens: LT lanes per token, N experts per lane, in the
// layout of gate_forward_many_kernel; bound by memory from there on.
template <int N, int LT, bool BF16, bool SIG>
__global__ void __launch_bounds__(GATE_WARPS * 32, N > 32 ? 4 : 5)
    gate_backward_many_kernel(const GateArgs a, const void* __restrict__ logits,
                              const int32_t* __restrict__ ids,
                              const void* __restrict__ d_weights,
                              const float* __restrict__ d_scores, void* __restrict__ d_logits) {
  constexpr int TW = 32 / LT, KL = 32 / LT;  // tokens per warp; selected experts per lane
  extern __shared__ int gate_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = lane % LT, tok = lane / LT;
  // gradients at the selected experts, in the order of the token's experts
  float* sd = reinterpret_cast<float*>(gate_smem) + (warp * TW + tok) * (N * LT);
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    reinterpret_cast<float4*>(sd)[i * LT + q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  grid_dep_wait();
  grid_dep_launch();
  const int64_t t_raw = (static_cast<int64_t>(blockIdx.x) * GATE_WARPS + warp) * TW + tok;
  const bool live = t_raw < a.T;
  const int64_t t = live ? t_raw : a.T - 1;  // (every lane takes part in the shuffles)
  float p[N];
  ld_token<N, LT, BF16>(logits, t * a.ld, q, a.E, p);
  float m = 0.0f, z = 1.0f;
  if constexpr (!SIG) {
    m = p[0];
#pragma unroll
    for (int j = 1; j < N; ++j) m = fmaxf(m, p[j]);
#pragma unroll
    for (int d = LT / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, d));
    m = row_shift(m);
    z = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      p[j] = expf(p[j] - m);
      z += p[j];
    }
    z = 1.0f / nonzero(lanes_sum<LT>(z));
  }
  // the selected experts, KL per lane
  const bool selected_softmax = !SIG && a.renorm;  // g becomes its part of dl itself
  int id[KL];
  float g[KL], ps[KL], top = -INFINITY, tot = 0.0f, gn = 0.0f;
#pragma unroll
  for (int x = 0; x < KL; ++x) {
    const int k = q + x * LT;
    id[x] = -1;
    g[x] = 0.0f;
    ps[x] = -INFINITY;
    if (k < a.K && d_weights) {
      id[x] = ids[t * a.K + k];
      if (static_cast<unsigned>(id[x]) >= static_cast<unsigned>(a.E)) id[x] = -1;
      g[x] = a.scale * ld_w(d_weights, t * a.K + k, a.weights_f32);
      if (id[x] >= 0) ps[x] = ld_logit<BF16>(logits, t * a.ld + id[x]);
    }
    top = fmaxf(top, ps[x]);
  }
  const float shift = selected_softmax ? row_shift(lanes_max<LT>(top)) : m;
  const float times = selected_softmax ? 1.0f : z;
#pragma unroll
  for (int x = 0; x < KL; ++x) {
    if (x * LT >= a.K) break;
    ps[x] = SIG ? sigmoid_rn(ps[x]) : expf(ps[x] - shift) * times;
    tot += ps[x];
    gn += g[x] * ps[x];
  }
  float sum = gn;  // softmax: sum dp p
  if (a.renorm) {
    tot = nonzero(lanes_sum<LT>(tot));
    gn = lanes_sum<LT>(gn) / tot;
    sum = 0.0f;
  }
  __syncwarp();
#pragma unroll
  for (int x = 0; x < KL; ++x)
    if (id[x] >= 0)
      sd[id[x]] = !a.renorm ? g[x] : (g[x] - gn) * (SIG ? 1.0f : ps[x]) / tot;
  __syncwarp();
  float4 ds[N / 4];
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const int e = (i * LT + q) * 4;
    ds[i] = d_scores && e < a.E ? *reinterpret_cast<const float4*>(d_scores + t * a.E + e)
                                : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if constexpr (!SIG) {
#pragma unroll
      for (int r = 0; r < 4; ++r) p[4 * i + r] *= z;
      sum += ds[i].x * p[4 * i] + ds[i].y * p[4 * i + 1] + ds[i].z * p[4 * i + 2] +
             ds[i].w * p[4 * i + 3];
    }
  }
  if constexpr (!SIG) sum = lanes_sum<LT>(sum);
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const int e = (i * LT + q) * 4;
    if (e >= a.E || !live) continue;
    const float4 s = reinterpret_cast<const float4*>(sd)[i * LT + q];
    const float sv[4] = {s.x, s.y, s.z, s.w};
    const float dv[4] = {ds[i].x, ds[i].y, ds[i].z, ds[i].w};
    float d[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float v = p[4 * i + r];
      d[r] = SIG ? (sv[r] + dv[r]) * sigmoid_rn(v) * sigmoid_rn(-v)
                 : (selected_softmax ? sv[r] + v * (dv[r] - sum) : v * (sv[r] + (dv[r] - sum)));
    }
    if constexpr (BF16) {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(d[0], d[1]);
      const __nv_bfloat162 hi = __floats2bfloat162_rn(d[2], d[3]);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(d_logits) + t * a.E + e) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    } else {
      *reinterpret_cast<float4*>(static_cast<float*>(d_logits) + t * a.E + e) =
          make_float4(d[0], d[1], d[2], d[3]);
    }
  }
}

// Only the selected experts have a gradient (sigmoid or renormalised weights,
// no d_scores): L lanes per token, K <= L, read the K selected logits, write
// the row's zeros and then the K values.  VEC: rows are whole 16-byte vectors.
template <int L, bool BF16, bool SIG, bool VEC>
__global__ void __launch_bounds__(GATE_WARPS * 32)
    gate_backward_selected_kernel(const GateArgs a, const void* __restrict__ logits,
                                  const int32_t* __restrict__ ids,
                                  const void* __restrict__ d_weights,
                                  void* __restrict__ d_logits) {
  constexpr int TOKENS = GATE_WARPS * 32 / L;
  const int lane = threadIdx.x % L;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * TOKENS + threadIdx.x / L;
  const bool live = t0 < a.T;
  const int64_t t = live ? t0 : 0;  // (every lane takes part in the sums)
  grid_dep_wait();
  grid_dep_launch();
  int id = -1;
  float g = 0.0f, lk = -INFINITY;
  if (live && lane < a.K) {
    id = ids[t * a.K + lane];
    if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.E)) id = -1;
    g = a.scale * ld_w(d_weights, t * a.K + lane, a.weights_f32);
    if (id >= 0) lk = ld_logit<BF16>(logits, t * a.ld + id);
  }
  if (live) {
    if constexpr (VEC) {
      const int n = a.E / (BF16 ? 8 : 4);
      uint4* row = static_cast<uint4*>(d_logits) + t * n;
      for (int i = lane; i < n; i += L) row[i] = make_uint4(0, 0, 0, 0);
    } else {
      for (int i = lane; i < a.E; i += L) {
        if constexpr (BF16)
          static_cast<uint16_t*>(d_logits)[t * a.E + i] = 0;
        else
          static_cast<float*>(d_logits)[t * a.E + i] = 0.0f;
      }
    }
  }
  float d;
  if constexpr (SIG) {
    const float p = id >= 0 ? sigmoid_rn(lk) : 0.0f;
    if (a.renorm) {
      const float tot = nonzero(lanes_sum<L>(p));
      g = (g - lanes_sum<L>(g * (p / tot))) / tot;
    }
    d = g * p * sigmoid_rn(-lk);
    if (lk == -INFINITY) d = 0.0f;
  } else {
    // n_k: softmax over the selected logits
    float n = expf(lk - row_shift(lanes_max<L>(lk)));
    n /= nonzero(lanes_sum<L>(n));
    d = n * (g - lanes_sum<L>(g * n));
  }
  __syncwarp();  // the zeros come first
  if (live && id >= 0) {
    if constexpr (BF16)
      static_cast<__nv_bfloat16*>(d_logits)[t * a.E + id] = __float2bfloat16_rn(d);
    else
      static_cast<float*>(d_logits)[t * a.E + id] = d;
  }
}

namespace {

bool aligned_to(const void* p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

GateArgs gate_args(const hmm_gate& g) {
  GateArgs a;
  a.T = g.T;
  a.ld = g.ld_logits;
  a.E = static_cast<int>(g.E);
  a.K = static_cast<int>(g.K);
  a.c = (a.E + 31) / 32;
  a.groups = g.groups;
  a.topk_groups = g.topk_groups;
  a.group_top = g.groups > 1 ? g.group_top : 1;  // (one group needs no worth)
  a.lane_groups = a.E % 32 == 0 && 32 % a.groups == 0 && a.group_top <= 2;
  a.weights_f32 = g.weights_dtype == HMM_DTYPE_F32;
  a.renorm = g.renormalize;
  a.scale = g.scale;
  return a;
}

// Whole chunks of 16-byte vectors: `bytes` per element of the logits (or their
// gradient), row starts ld elements apart.
bool gate_vec(const GateArgs& a, int bytes, int64_t ld, const void* p) {
  const int per = 16 / bytes;
  return a.E % 32 == 0 && a.c % per == 0 && ld % per == 0 && aligned_to(p, 16);
}

// F::run<C, BF16, SIG, VEC>(...): the smallest C >= c that is built; VEC needs
// c == C.
template <class F, int C, typename... Args>
cudaError_t by_type(const hmm_gate& g, bool vec, Args&&... args) {
  const bool bf16 = g.logits_dtype == HMM_DTYPE_BF16, sig = g.score == HMM_SCORE_SIGMOID;
  vec = vec && (g.E + 31) / 32 == C;
  if constexpr (C % 8 == 0) {
    if (vec && bf16) return sig ? F::template run<C, true, true, true>(g, args...)
                                : F::template run<C, true, false, true>(g, args...);
  }
  if constexpr (C % 4 == 0) {
    if (vec && !bf16) return sig ? F::template run<C, false, true, true>(g, args...)
                                 : F::template run<C, false, false, true>(g, args...);
  }
  if (bf16) return sig ? F::template run<C, true, true, false>(g, args...)
                       : F::template run<C, true, false, false>(g, args...);
  return sig ? F::template run<C, false, true, false>(g, args...)
             : F::template run<C, false, false, false>(g, args...);
}
template <class F, typename... Args>
cudaError_t by_length(const hmm_gate& g, bool vec, Args&&... args) {
  const int c = static_cast<int>((g.E + 31) / 32);
  if (c <= 1) return by_type<F, 1>(g, vec, args...);
  if (c <= 2) return by_type<F, 2>(g, vec, args...);
  if (c <= 4) return by_type<F, 4>(g, vec, args...);
  if (c <= 8) return by_type<F, 8>(g, vec, args...);
  if (c <= 16) return by_type<F, 16>(g, vec, args...);
  return by_type<F, 32>(g, vec, args...);
}

// one token per warp, several in turn past 2^20 blocks
unsigned gate_grid(int64_t tokens) {
  return static_cast<unsigned>(
      std::min<int64_t>((tokens + GATE_WARPS - 1) / GATE_WARPS, int64_t(1) << 20));
}

struct RunForward {
  template <int C, bool BF16, bool SIG, bool VEC>
  static cudaError_t run(const hmm_gate& g, const void* logits, const float* bias, int32_t* ids,
                         void* weights, float* scores, cudaStream_t st, bool pdl) {
    const GateArgs a = gate_args(g);
    const bool rounded_sums = !SIG && (bias || a.group_top > 1);
    const size_t smem = rounded_sums || (a.groups > 1 && !a.lane_groups)
                            ? sizeof(float) * GATE_WARPS * 33 * a.c : 0;
    return launch_kernel(gate_forward_kernel<C, BF16, SIG, VEC>, gate_grid(g.T), GATE_WARPS * 32,
                         smem, st, pdl, 1, a, logits, bias, ids, weights, scores);
  }
};

template <int N, int LT>
cudaError_t run_many(const hmm_gate& g, const void* logits, const float* bias, int32_t* ids,
                     void* weights, float* scores, cudaStream_t st, bool pdl) {
  constexpr int TOKENS = GATE_WARPS * 32 / LT;
  const bool sig = g.score == HMM_SCORE_SIGMOID;
  auto kern = g.logits_dtype == HMM_DTYPE_BF16
                  ? (sig ? gate_forward_many_kernel<N, LT, true, true>
                         : gate_forward_many_kernel<N, LT, true, false>)
                  : (sig ? gate_forward_many_kernel<N, LT, false, true>
                         : gate_forward_many_kernel<N, LT, false, false>);
  const size_t smem = sizeof(uint32_t) * GATE_WARPS * (32 * N + 32 / LT * 32);
  return launch_kernel(kern, static_cast<unsigned>((g.T + TOKENS - 1) / TOKENS), GATE_WARPS * 32,
                       smem, st, pdl, 1, gate_args(g), logits, bias, ids, weights, scores);
}

template <int N, int LT>
cudaError_t run_backward_many(const hmm_gate& g, const void* logits, const int32_t* ids,
                              const void* d_weights, const float* d_scores, void* d_logits,
                              cudaStream_t st, bool pdl) {
  constexpr int TOKENS = GATE_WARPS * 32 / LT;
  const bool sig = g.score == HMM_SCORE_SIGMOID;
  auto kern = g.logits_dtype == HMM_DTYPE_BF16
                  ? (sig ? gate_backward_many_kernel<N, LT, true, true>
                         : gate_backward_many_kernel<N, LT, true, false>)
                  : (sig ? gate_backward_many_kernel<N, LT, false, true>
                         : gate_backward_many_kernel<N, LT, false, false>);
  const size_t smem = sizeof(float) * GATE_WARPS * 32 * N;
  return launch_kernel(kern, static_cast<unsigned>((g.T + TOKENS - 1) / TOKENS), GATE_WARPS * 32,
                       smem, st, pdl, 1, gate_args(g), logits, ids, d_weights, d_scores, d_logits);
}

// Tokens from which the kernels for many tokens run.  One limit for every E,
// near where most of them cross (us of a call in a graph of 20, one token per
// warp and many; s: softmax, g: sigmoid in 8 groups, 4 for E = 64; T = 2048,
// 4096, 8192: E = 64 s 2.8 and 3.6, 3.8 and 3.6, 5.7 and 4.0, g 3.4 and 5.5, 5.6
// and 5.5, 6.6 and 6.1; E = 160 s 4.2 and 5.1, 5.7 and 5.1, 9.7 and 5.7, g 5.7 and
// 9.5, 8.8 and 9.6, 12.7 and 10.3; E = 256 s 4.0 and 4.5, 5.5 and 5.0, 9.2 and 6.4,
// g 5.7 and 8.1, 8.8 and 8.7, 12.4 and 10.3; the worst at the limit, E = 128 g, 4.2
// and 8.4, 6.6 and 8.4, 8.7 and 9.2.  From E = 512 on the many win earlier, E = 1024
// g 22.3 and 10.3, 30.9 and 15.7.  Dense backward: E = 64 2.8 and 2.9, 3.4 and 3.0,
// E = 256 3.9 and 3.1, 6.1 and 3.5).
constexpr int64_t GATE_MANY = 4096;

struct RunBackward {
  template <int C, bool BF16, bool SIG, bool VEC>
  static cudaError_t run(const hmm_gate& g, const void* logits, const int32_t* ids,
                         const void* d_weights, const float* d_scores, void* d_logits,
                         cudaStream_t st, bool pdl) {
    const size_t smem = sizeof(float) * GATE_WARPS * 32 * C;
    return launch_kernel(gate_backward_kernel<C, BF16, SIG, VEC>, gate_grid(g.T), GATE_WARPS * 32,
                         smem, st, pdl, 1, gate_args(g), logits, ids, d_weights, d_scores,
                         d_logits);
  }
};

template <int L, bool BF16, bool SIG>
cudaError_t run_selected(const hmm_gate& g, const void* logits, const int32_t* ids,
                         const void* d_weights, void* d_logits, cudaStream_t st, bool pdl) {
  const bool vec = g.E % (BF16 ? 8 : 4) == 0 && aligned_to(d_logits, 16);
  auto kern = vec ? gate_backward_selected_kernel<L, BF16, SIG, true>
                  : gate_backward_selected_kernel<L, BF16, SIG, false>;
  constexpr int TOKENS = GATE_WARPS * 32 / L;
  return launch_kernel(kern, static_cast<unsigned>((g.T + TOKENS - 1) / TOKENS), GATE_WARPS * 32,
                       0, st, pdl, 1, gate_args(g), logits, ids, d_weights, d_logits);
}
template <int L>
cudaError_t run_selected_by_type(const hmm_gate& g, const void* logits, const int32_t* ids,
                                 const void* d_weights, void* d_logits, cudaStream_t st,
                                 bool pdl) {
  const bool bf16 = g.logits_dtype == HMM_DTYPE_BF16, sig = g.score == HMM_SCORE_SIGMOID;
  if (bf16)
    return sig ? run_selected<L, true, true>(g, logits, ids, d_weights, d_logits, st, pdl)
               : run_selected<L, true, false>(g, logits, ids, d_weights, d_logits, st, pdl);
  return sig ? run_selected<L, false, true>(g, logits, ids, d_weights, d_logits, st, pdl)
             : run_selected<L, false, false>(g, logits, ids, d_weights, d_logits, st, pdl);
}

}  // namespace

int check_gate(const hmm_gate* g) {
  if (!g) return HMM_ERR_ARG;
  for (int d : {g->logits_dtype, g->weights_dtype})
    if (d != HMM_DTYPE_BF16 && d != HMM_DTYPE_F32) return HMM_ERR_DTYPE;
  if (g->score != HMM_SCORE_SOFTMAX && g->score != HMM_SCORE_SIGMOID) return HMM_ERR_ARG;
  if (g->renormalize != 0 && g->renormalize != 1) return HMM_ERR_ARG;
  if (!(g->scale > -INFINITY && g->scale < INFINITY)) return HMM_ERR_ARG;
  if (g->T < 0 || g->E <= 0 || g->K <= 0 || g->E > MAX_E || g->K > 32) return HMM_ERR_SHAPE;
  if (g->T > (int64_t(1) << 31) || g->ld_logits < g->E) return HMM_ERR_SHAPE;
  if (g->groups < 1 || g->groups > 32 || g->E % g->groups != 0) return HMM_ERR_SHAPE;
  const int64_t n = g->E / g->groups;
  if (g->topk_groups < 1 || g->topk_groups > g->groups || g->group_top < 1 || g->group_top > n)
    return HMM_ERR_SHAPE;
  if (g->K > n * g->topk_groups) return HMM_ERR_SHAPE;
  return HMM_OK;
}

cudaError_t launch_gate_forward(const hmm_gate& g, const void* logits, const float* bias,
                                int32_t* ids, void* weights, float* scores, cudaStream_t st,
                                bool pdl) {
  const GateArgs a = gate_args(g);
  const bool vec = gate_vec(a, g.logits_dtype == HMM_DTYPE_BF16 ? 2 : 4, g.ld_logits, logits) &&
                   (!scores || aligned_to(scores, 16));
  const int64_t logit_bytes = g.logits_dtype == HMM_DTYPE_BF16 ? 2 : 4;
  if (g.T >= GATE_MANY && g.E % 4 == 0 && (g.groups == 1 || g.group_top <= 2) &&
      g.ld_logits % 4 == 0 && aligned_to(logits, 4 * logit_bytes) && aligned_to(bias, 16) &&
      aligned_to(scores, 16)) {
    // 32 to 40 experts per lane (E = 256, T = 65537: 64 per lane 64 us, few warps
    // fit; 32 51 us; 16 72 us, fewer tokens share a round.  E = 160, T = 131072: 40
    // per lane 59 us, 24 63 us), and 24 where they leave fewer places empty (grouped
    // sigmoid, 32 and 24 per lane: E = 192, T = 65536 55 and 45 us, E = 300 135 and
    // 113, E = 384, T = 32768 57 and 49, E = 768 127 and 107; E = 32 with 16 and 8 per
    // lane 20 and 16).  The second number is many_lanes(E).
    if (g.E <= 32) return run_many<8, 4>(g, logits, bias, ids, weights, scores, st, pdl);
    if (g.E <= 64) return run_many<16, 4>(g, logits, bias, ids, weights, scores, st, pdl);
    if (g.E <= 96) return run_many<24, 4>(g, logits, bias, ids, weights, scores, st, pdl);
    if (g.E <= 128) return run_many<32, 4>(g, logits, bias, ids, weights, scores, st, pdl);
    if (g.E <= 160) return run_many<40, 4>(g, logits, bias, ids, weights, scores, st, pdl);
    if (g.E <= 192) return run_many<24, 8>(g, logits, bias, ids, weights, scores, st, pdl);
    if (g.E <= 256) return run_many<32, 8>(g, logits, bias, ids, weights, scores, st, pdl);
    if (g.E <= 384) return run_many<24, 16>(g, logits, bias, ids, weights, scores, st, pdl);
    if (g.E <= 512) return run_many<32, 16>(g, logits, bias, ids, weights, scores, st, pdl);
    if (g.E <= 768) return run_many<24, 32>(g, logits, bias, ids, weights, scores, st, pdl);
    return run_many<32, 32>(g, logits, bias, ids, weights, scores, st, pdl);
  }
  return by_length<RunForward>(g, vec, logits, bias, ids, weights, scores, st, pdl);
}

cudaError_t launch_gate_backward(const hmm_gate& g, const void* logits, const int32_t* ids,
                                 const void* d_weights, const float* d_scores, void* d_logits,
                                 cudaStream_t st, bool pdl) {
  if (!d_scores && d_weights && (g.renormalize || g.score == HMM_SCORE_SIGMOID)) {
    if (g.K <= 8)
      return run_selected_by_type<8>(g, logits, ids, d_weights, d_logits, st, pdl);
    return run_selected_by_type<32>(g, logits, ids, d_weights, d_logits, st, pdl);
  }
  const GateArgs a = gate_args(g);
  const int bytes = g.logits_dtype == HMM_DTYPE_BF16 ? 2 : 4;
  if (g.T >= GATE_MANY && g.E % 4 == 0 && g.ld_logits % 4 == 0 &&
      aligned_to(logits, 4 * bytes) && aligned_to(d_logits, 4 * bytes) &&
      aligned_to(d_scores, 16)) {
    if (g.E <= 32)
      return run_backward_many<8, 4>(g, logits, ids, d_weights, d_scores, d_logits, st, pdl);
    if (g.E <= 64)
      return run_backward_many<16, 4>(g, logits, ids, d_weights, d_scores, d_logits, st, pdl);
    if (g.E <= 96)
      return run_backward_many<24, 4>(g, logits, ids, d_weights, d_scores, d_logits, st, pdl);
    if (g.E <= 128)
      return run_backward_many<32, 4>(g, logits, ids, d_weights, d_scores, d_logits, st, pdl);
    if (g.E <= 160)
      return run_backward_many<40, 4>(g, logits, ids, d_weights, d_scores, d_logits, st, pdl);
    if (g.E <= 192)
      return run_backward_many<24, 8>(g, logits, ids, d_weights, d_scores, d_logits, st, pdl);
    if (g.E <= 256)
      return run_backward_many<32, 8>(g, logits, ids, d_weights, d_scores, d_logits, st, pdl);
    if (g.E <= 384)
      return run_backward_many<24, 16>(g, logits, ids, d_weights, d_scores, d_logits, st, pdl);
    if (g.E <= 512)
      return run_backward_many<32, 16>(g, logits, ids, d_weights, d_scores, d_logits, st, pdl);
    if (g.E <= 768)
      return run_backward_many<24, 32>(g, logits, ids, d_weights, d_scores, d_logits, st, pdl);
    return run_backward_many<32, 32>(g, logits, ids, d_weights, d_scores, d_logits, st, pdl);
  }
  const bool vec = gate_vec(a, bytes, g.ld_logits, logits) && gate_vec(a, bytes, g.E, d_logits);
  return by_length<RunBackward>(g, vec, logits, ids, d_weights, d_scores, d_logits, st, pdl);
}

}  // namespace hmm
