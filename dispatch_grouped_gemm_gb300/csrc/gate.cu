// gate.cu -- the router in front of the experts: scores of E experts per
// token, group-limited top-k selection and the routing weights, forward and
// backward.
//
//   p = softmax(l) or sigmoid(l)                                    [T, E]
//   key = p + bias (softmax without a bias, groups counted by one key: l
//         itself, whose order is that of p)
//   groups > 1: a group of E / groups experts counts by the sum of its
//         group_top best keys; the topk_groups best groups stay open
//   topk_ids = the K best keys of the open groups, best first, ties to the
//         lowest index
//   topk_weights = scale * p[topk_ids], over sum_k p[topk_ids] with renormalize
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

// Order-preserving map of a float to an unsigned integer above 0: -inf is the
// least, NaN (any) the greatest, -0 equals +0; and back.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0xffffffffu;
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k >> 31) ? k ^ 0x80000000u : ~k);
}

template <int L = 32>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) v += __shfl_xor_sync(FULL, v, d);
  return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, d));
  return v;
}

// 1 / (1 + exp(-l)) with the accurate exponential and a correctly rounded
// reciprocal: the selection compares these values, so they are rounded as the
// formula's own fp32 evaluation rounds them.
__device__ __forceinline__ float sigmoid_rn(float l) { return __frcp_rn(1.0f + expf(-l)); }

// Largest logit of a row, 0 for a row that is all -inf: its experts are all
// closed, their exponentials 0.  (A NaN turns the row's sum into NaN.)
template <int C>
__device__ __forceinline__ float row_max(const float (&l)[C]) {
  float m = l[0];
#pragma unroll
  for (int j = 1; j < C; ++j) m = fmaxf(m, l[j]);
  m = warp_max(m);
  return m == -INFINITY ? 0.0f : m;
}

template <int C>
__device__ __forceinline__ float exp_row(const float (&l)[C], float m, float (&p)[C]) {
  float z = 0.0f;
#pragma unroll
  for (int j = 0; j < C; ++j) {
    p[j] = expf(l[j] - m);
    z += p[j];
  }
  z = lanes_sum(z);
  return z == 0.0f ? 1.0f : z;
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
__device__ __noinline__ uint32_t group_worth(const uint32_t* keys, int n, int top) {
  const uint32_t* k = keys + (threadIdx.x & 31) * n;
  float worth = 0.0f;
  uint32_t last = 0xffffffffu;
  int last_i = -1;
  for (int r = 0; r < top; ++r) {
    uint32_t bk = 0;
    int bi = 0;
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

// Closes (key 0) the experts of all but the topk_groups best groups.
template <int C>
__device__ __forceinline__ void keep_groups(const GateArgs& a, uint32_t (&key)[C], int lane,
                                            int base, uint32_t* smem) {
  if (a.lane_groups) {
    const int L = 32 / a.groups;  // lanes per group
    uint32_t k1 = key[0], k2 = 0u;
#pragma unroll
    for (int j = 1; j < C; ++j) {
      k2 = max(k2, min(k1, key[j]));
      k1 = max(k1, key[j]);
    }
    for (int d = 1; d < L; d <<= 1) {
      const uint32_t o1 = __shfl_xor_sync(FULL, k1, d), o2 = __shfl_xor_sync(FULL, k2, d);
      k2 = max(min(k1, o1), max(k2, o2));
      k1 = max(k1, o1);
    }
    const uint32_t worth = a.group_top == 1 ? k1 : order_key(key_value(k1) + key_value(k2));
    const int g = lane / L;
    int better = 0;  // groups that come before this one
    for (int x = 1; x < a.groups; ++x) {
      const uint32_t o = __shfl_xor_sync(FULL, worth, x * L);
      better += o > worth || (o == worth && (g ^ x) < g);
    }
    if (better >= a.topk_groups) {
#pragma unroll
      for (int j = 0; j < C; ++j) key[j] = 0u;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < C; ++j)
    if (j < a.c && base + j < a.E) smem[base + j] = key[j];
  __syncwarp();
  const int n = a.E / a.groups;
  uint32_t worth = lane < a.groups ? group_worth(smem, n, a.group_top) : 0u;
  __syncwarp();
  uint32_t open = 0;
  for (int r = 0; r < a.topk_groups; ++r) {
    const uint32_t best = __reduce_max_sync(FULL, worth);
    const int g = __ffs(__ballot_sync(FULL, worth == best)) - 1;
    open |= 1u << g;
    if (lane == g) worth = 0u;
  }
#pragma unroll
  for (int j = 0; j < C; ++j)
    if (base + j < a.E && !((open >> ((base + j) / n)) & 1u)) key[j] = 0u;
}

}  // namespace

template <int C, bool BF16, bool SIG, bool VEC>
__global__ void __launch_bounds__(GATE_WARPS * 32)
    gate_forward_kernel(const GateArgs a, const void* __restrict__ logits,
                        const float* __restrict__ bias, int32_t* __restrict__ ids,
                        void* __restrict__ weights, float* __restrict__ scores) {
  extern __shared__ uint32_t gate_smem[];  // per warp [E] (groups that are no lane runs)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int base = lane * a.c;
  const bool by_logit = !SIG && bias == nullptr && a.group_top == 1;
  grid_dep_wait();
  grid_dep_launch();
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * GATE_WARPS + warp; t < a.T;
       t += static_cast<int64_t>(gridDim.x) * GATE_WARPS) {
    float l[C], p[C];
    uint32_t key[C];
    ld_chunk<C, BF16, VEC>(logits, t * a.ld, base, a.c, a.E, l);
    float m = 0.0f, z = 1.0f;
    if constexpr (SIG) {
#pragma unroll
      for (int j = 0; j < C; ++j) p[j] = sigmoid_rn(l[j]);
    } else {
      m = row_max(l);
      // (renormalised weights of the best logits need no sum over the row)
      if (scores || !by_logit || !a.renorm) z = exp_row(l, m, p);
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
      key[j] = in ? order_key(v) : 0u;
    }
    if (a.groups > 1) keep_groups<C>(a, key, lane, base, gate_smem + warp * a.E);
    // K rounds: the best key of the lanes' best; lane k keeps expert k
    uint32_t bk = key[0];
    int bj = 0;
#pragma unroll
    for (int j = 1; j < C; ++j)
      if (key[j] > bk) {
        bk = key[j];
        bj = j;
      }
    int my_id = 0;
    for (int k = 0; k < a.K; ++k) {
      const uint32_t best = __reduce_max_sync(FULL, bk);
      const int win = __ffs(__ballot_sync(FULL, bk == best)) - 1;
      const int e = __shfl_sync(FULL, base + bj, win);
      if (lane == k) my_id = e;
      if (lane == win) {
        uint32_t nk = 0u;
        int nj = 0;
#pragma unroll
        for (int j = 0; j < C; ++j) {
          if (j == bj) key[j] = 0u;
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
    float w = 0.0f;
    if (lane < a.K) {
      const float lk = ld_logit<BF16>(logits, t * a.ld + my_id);
      w = SIG ? sigmoid_rn(lk) : expf(lk - m) / z;
    }
    if (a.renorm) {
      const float sum = lanes_sum(w);
      w = w / (sum == 0.0f ? 1.0f : sum);
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

// With g_k = scale * d_topk_weights[k], n_k = p_k / sum_sel p and D = sum g n:
//   without renormalize   dp[topk_ids[k]] = g_k
//   with it               dp[topk_ids[k]] = (g_k - D) / sum_sel p
//   dp += d_scores
//   sigmoid  dl = dp p (1 - p)
//   softmax  dl = p (dp - sum dp p); the renormalised weights' part of that sum
//            is D - D = 0, so their gradient n_k (g_k - D) stays on the
//            selected experts.
// This kernel: every expert has a gradient (d_scores, or softmax weights that
// are not renormalised).  One warp per token, the forward's layout; the
// selected part is scattered through shared memory.
template <int C, bool BF16, bool SIG, bool VEC>
__global__ void __launch_bounds__(GATE_WARPS * 32)
    gate_backward_kernel(const GateArgs a, const void* __restrict__ logits,
                         const int32_t* __restrict__ ids, const void* __restrict__ d_weights,
                         const float* __restrict__ d_scores, void* __restrict__ d_logits) {
  extern __shared__ uint32_t gate_smem[];  // per warp: gradients at the selected experts
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
    float g = 0.0f, ps = 0.0f, m = 0.0f, z = 1.0f;
    if constexpr (SIG) {
#pragma unroll
      for (int j = 0; j < C; ++j) p[j] = sigmoid_rn(l[j]);
    } else {
      m = row_max(l);
      z = 1.0f / exp_row(l, m, p);
#pragma unroll
      for (int j = 0; j < C; ++j) p[j] *= z;
    }
    if (lane < a.K && d_weights) {
      id = ids[t * a.K + lane];
      if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.E)) id = -1;
      g = a.scale * ld_w(d_weights, t * a.K + lane, a.weights_f32);
    }
    if (id >= 0) {
      const float lk = ld_logit<BF16>(logits, t * a.ld + id);
      ps = SIG ? sigmoid_rn(lk) : expf(lk - m) * z;
    }
    float sum = 0.0f;  // softmax: sum dp p
    if (a.renorm) {
      float tot = lanes_sum(ps);
      if (tot == 0.0f) tot = 1.0f;
      g = (g - lanes_sum(g * (ps / tot))) / tot;
    } else {
      sum = g * ps;
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
      dp[j] = SIG ? (s + dp[j]) * p[j] * sigmoid_rn(-l[j]) : p[j] * (s + (dp[j] - sum));
    }
    st_chunk<C, BF16, VEC>(d_logits, t * a.E, base, a.c, a.E, dp);
    __syncwarp();
    if (id >= 0) sd[id] = 0.0f;
    __syncwarp();
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
      float tot = lanes_sum<L>(p);
      if (tot == 0.0f) tot = 1.0f;
      g = (g - lanes_sum<L>(g * (p / tot))) / tot;
    }
    d = g * p * sigmoid_rn(-lk);
    if (lk == -INFINITY) d = 0.0f;
  } else {
    // n_k: softmax over the selected logits
    float m = lk;
#pragma unroll
    for (int x = L / 2; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, x));
    if (m == -INFINITY) m = 0.0f;
    float n = expf(lk - m);
    const float tot = lanes_sum<L>(n);
    n = n / (tot == 0.0f ? 1.0f : tot);
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
  a.group_top = g.group_top;
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
  if (c <= 6) return by_type<F, 6>(g, vec, args...);
  if (c <= 8) return by_type<F, 8>(g, vec, args...);
  if (c <= 12) return by_type<F, 12>(g, vec, args...);
  if (c <= 16) return by_type<F, 16>(g, vec, args...);
  return by_type<F, 32>(g, vec, args...);
}

// one token per warp up to 64 blocks per SM's worth, then several in turn
unsigned gate_grid(int64_t tokens) {
  return static_cast<unsigned>(
      std::min<int64_t>((tokens + GATE_WARPS - 1) / GATE_WARPS, int64_t(1) << 20));
}

struct RunForward {
  template <int C, bool BF16, bool SIG, bool VEC>
  static cudaError_t run(const hmm_gate& g, const void* logits, const float* bias, int32_t* ids,
                         void* weights, float* scores, cudaStream_t st, bool pdl) {
    const GateArgs a = gate_args(g);
    const size_t smem = a.groups > 1 && !a.lane_groups ? sizeof(float) * GATE_WARPS * a.E : 0;
    return launch_kernel(gate_forward_kernel<C, BF16, SIG, VEC>, gate_grid(g.T), GATE_WARPS * 32,
                         smem, st, pdl, 1, a, logits, bias, ids, weights, scores);
  }
};

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
  const bool vec = gate_vec(a, bytes, g.ld_logits, logits) && gate_vec(a, bytes, g.E, d_logits);
  return by_length<RunBackward>(g, vec, logits, ids, d_weights, d_scores, d_logits, st, pdl);
}

}  // namespace hmm
