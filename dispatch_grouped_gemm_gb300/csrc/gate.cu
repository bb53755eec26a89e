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
// One warp per token: lane i holds experts i, i + 32, ... in registers, every
// reduction is a warp shuffle or redux, and a row of logits is read once.
#include <cuda_bf16.h>

#include "hmm_internal.h"

namespace hmm {

namespace {

constexpr int GATE_WARPS = 4;  // tokens per block
constexpr unsigned FULL = 0xffffffffu;

template <bool BF16>
__device__ __forceinline__ float ld_logit(const void* p, int64_t i) {
  if constexpr (BF16)
    return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
  else
    return static_cast<const float*>(p)[i];
}

// Order-preserving map of a float to an unsigned integer above 0: -inf is the
// least, NaN (any) the greatest, -0 equals +0.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0xffffffffu;
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(FULL, v, d);
  return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, d));
  return v;
}

// 1 / (1 + exp(-l)) with the accurate exponential and an IEEE division: the
// selection compares these values, so they are rounded as the formula's own
// fp32 evaluation rounds them.
__device__ __forceinline__ float sigmoid_rn(float l) { return 1.0f / (1.0f + expf(-l)); }

// Scores of one row in registers (lane i: experts i + 32 j).  A softmax row
// whose logits are all -inf has no open expert: its scores are 0.
template <int NV, bool SIG>
__device__ __forceinline__ void row_scores(const float (&l)[NV], float (&p)[NV]) {
  if constexpr (SIG) {
#pragma unroll
    for (int j = 0; j < NV; ++j) p[j] = sigmoid_rn(l[j]);
  } else {
    float m = l[0];
#pragma unroll
    for (int j = 1; j < NV; ++j) m = fmaxf(m, l[j]);
    m = warp_max(m);  // (a NaN logit turns the whole row to NaN below)
    if (m == -INFINITY) m = 0.0f;
    float z = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      p[j] = expf(l[j] - m);
      z += p[j];
    }
    z = warp_sum(z);
    const float d = z == 0.0f ? 1.0f : z;
#pragma unroll
    for (int j = 0; j < NV; ++j) p[j] = p[j] / d;
  }
}

}  // namespace

struct GateArgs {
  int64_t T, ld;
  int E, K, groups, topk_groups, group_top;
  int weights_f32, renorm;
  float scale;
};

template <int NV, bool BF16, bool SIG>
__global__ void __launch_bounds__(GATE_WARPS * 32)
    gate_forward_kernel(const GateArgs a, const void* __restrict__ logits,
                        const float* __restrict__ bias, int32_t* __restrict__ ids,
                        void* __restrict__ weights, float* __restrict__ scores) {
  extern __shared__ float gate_smem[];  // per warp: the keys [E] (groups only)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * GATE_WARPS + warp;
  grid_dep_wait();
  grid_dep_launch();
  if (t >= a.T) return;
  float l[NV], p[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = lane + 32 * j;
    l[j] = e < a.E ? ld_logit<BF16>(logits, t * a.ld + e) : -INFINITY;
  }
  row_scores<NV, SIG>(l, p);
  if (scores) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = lane + 32 * j;
      if (e < a.E) scores[t * a.E + e] = p[j];
    }
  }
  const bool by_logit = !SIG && bias == nullptr && a.group_top == 1;
  float kf[NV];
  uint32_t key[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = lane + 32 * j;
    kf[j] = by_logit ? l[j] : p[j];
    if (bias && e < a.E) kf[j] += bias[e];
    key[j] = e < a.E ? order_key(kf[j]) : 0u;
  }
  if (a.groups > 1) {
    float* sk = gate_smem + warp * a.E;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = lane + 32 * j;
      if (e < a.E) sk[e] = kf[j];
    }
    __syncwarp();
    const int n = a.E / a.groups;
    uint32_t gk = 0;  // lane g: key of group g's worth
    if (lane < a.groups) {
      // the group_top best keys by order (NaN first), by repeated selection
      float worth = 0.0f;
      uint32_t last = 0xffffffffu;
      int last_i = -1;
      for (int r = 0; r < a.group_top; ++r) {
        uint32_t bk = 0;
        int bi = -1;
        for (int i = 0; i < n; ++i) {
          const uint32_t k = order_key(sk[lane * n + i]);
          const bool taken = r > 0 && (k > last || (k == last && i <= last_i));
          if (!taken && k > bk) {
            bk = k;
            bi = i;
          }
        }
        last = bk;
        last_i = bi;
        worth = r == 0 ? sk[lane * n + bi] : worth + sk[lane * n + bi];
      }
      gk = order_key(worth);
    }
    uint32_t open = 0;
    for (int r = 0; r < a.topk_groups; ++r) {
      const uint32_t best = __reduce_max_sync(FULL, gk);
      const int g = __ffs(__ballot_sync(FULL, gk == best)) - 1;
      open |= 1u << g;
      if (lane == g) gk = 0;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = lane + 32 * j;
      if (e < a.E && !((open >> (e / n)) & 1u)) key[j] = 0u;
    }
  }
  // K best keys: lane k keeps the k-th expert and its score
  int my_id = 0;
  float my_p = 0.0f, sum = 0.0f;
  for (int k = 0; k < a.K; ++k) {
    uint32_t bk = key[0];
    int bj = 0;
    float bp = p[0];
#pragma unroll
    for (int j = 1; j < NV; ++j) {
      if (key[j] > bk) {
        bk = key[j];
        bj = j;
        bp = p[j];
      }
    }
    const uint32_t best = __reduce_max_sync(FULL, bk);
    const unsigned cand = bk == best ? static_cast<unsigned>(lane + 32 * bj) : 0xffffffffu;
    const int e = static_cast<int>(__reduce_min_sync(FULL, cand));
    const float pe = __shfl_sync(FULL, bp, e & 31);
    if (lane == k) {
      my_id = e;
      my_p = pe;
    }
    sum += pe;
    if ((e & 31) == lane) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (j == (e >> 5)) key[j] = 0u;
    }
  }
  if (lane < a.K) {
    float w = my_p;
    if (a.renorm) w = w / (sum == 0.0f ? 1.0f : sum);
    w *= a.scale;
    ids[t * a.K + lane] = my_id;
    if (a.weights_f32)
      static_cast<float*>(weights)[t * a.K + lane] = w;
    else
      static_cast<__nv_bfloat16*>(weights)[t * a.K + lane] = __float2bfloat16_rn(w);
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
template <int NV, bool BF16, bool SIG>
__global__ void __launch_bounds__(GATE_WARPS * 32)
    gate_backward_kernel(const GateArgs a, const void* __restrict__ logits,
                         const int32_t* __restrict__ ids, const void* __restrict__ d_weights,
                         const float* __restrict__ d_scores, void* __restrict__ d_logits) {
  extern __shared__ float gate_smem[];  // per warp: gradients at the selected experts [E]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * GATE_WARPS + warp;
  float* sd = gate_smem + warp * a.E;
  grid_dep_wait();
  grid_dep_launch();
  if (t >= a.T) return;
  float l[NV], p[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = lane + 32 * j;
    l[j] = e < a.E ? ld_logit<BF16>(logits, t * a.ld + e) : -INFINITY;
    if (e < a.E) sd[e] = 0.0f;
  }
  row_scores<NV, SIG>(l, p);
  int id = -1;
  float g = 0.0f;
  if (lane < a.K && d_weights) {
    id = ids[t * a.K + lane];
    if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.E)) id = -1;
    const int64_t i = t * a.K + lane;
    g = a.scale * (a.weights_f32
                       ? static_cast<const float*>(d_weights)[i]
                       : __bfloat162float(static_cast<const __nv_bfloat16*>(d_weights)[i]));
  }
  // score of this lane's expert, from the lane that holds it
  float ps = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const float v = __shfl_sync(FULL, p[j], id & 31);
    if (id >= 0 && (id >> 5) == j) ps = v;
  }
  float dw = g;  // renormalize: n_k (g_k - D) / p_k
  float tot = 1.0f;
  if (a.renorm) {
    tot = warp_sum(ps);
    if (tot == 0.0f) tot = 1.0f;
    dw = g - warp_sum(g * (ps / tot));
  }
  __syncwarp();
  if (id >= 0) sd[id] = dw / tot;
  __syncwarp();
  float dp[NV], ds[NV];
  float sum = 0.0f;
  const bool own_sum = !SIG && !a.renorm;  // the selected part enters the softmax sum
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = lane + 32 * j;
    dp[j] = e < a.E ? sd[e] : 0.0f;
    ds[j] = e < a.E && d_scores ? d_scores[t * a.E + e] : 0.0f;
    sum += (ds[j] + (own_sum ? dp[j] : 0.0f)) * p[j];
  }
  if constexpr (!SIG) sum = warp_sum(sum);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = lane + 32 * j;
    float d;
    if constexpr (SIG) {
      d = (dp[j] + ds[j]) * p[j] * sigmoid_rn(-l[j]);
    } else {
      d = p[j] * (dp[j] + (ds[j] - sum));
    }
    if (e < a.E) {
      if constexpr (BF16)
        static_cast<__nv_bfloat16*>(d_logits)[t * a.E + e] = __float2bfloat16_rn(d);
      else
        static_cast<float*>(d_logits)[t * a.E + e] = d;
    }
  }
}

namespace {

GateArgs gate_args(const hmm_gate& g) {
  GateArgs a;
  a.T = g.T;
  a.ld = g.ld_logits;
  a.E = static_cast<int>(g.E);
  a.K = static_cast<int>(g.K);
  a.groups = g.groups;
  a.topk_groups = g.topk_groups;
  a.group_top = g.group_top;
  a.weights_f32 = g.weights_dtype == HMM_DTYPE_F32;
  a.renorm = g.renormalize;
  a.scale = g.scale;
  return a;
}

// F::run<NV, BF16, SIG>(...) for the row length, type and score of g
template <class F, int NV, typename... Args>
cudaError_t by_type(const hmm_gate& g, Args&&... args) {
  const bool bf16 = g.logits_dtype == HMM_DTYPE_BF16, sig = g.score == HMM_SCORE_SIGMOID;
  if (bf16) return sig ? F::template run<NV, true, true>(g, args...)
                       : F::template run<NV, true, false>(g, args...);
  return sig ? F::template run<NV, false, true>(g, args...)
             : F::template run<NV, false, false>(g, args...);
}
template <class F, typename... Args>
cudaError_t by_length(const hmm_gate& g, Args&&... args) {
  const int nv = static_cast<int>((g.E + 31) / 32);
  if (nv <= 1) return by_type<F, 1>(g, args...);
  if (nv <= 2) return by_type<F, 2>(g, args...);
  if (nv <= 4) return by_type<F, 4>(g, args...);
  if (nv <= 8) return by_type<F, 8>(g, args...);
  if (nv <= 16) return by_type<F, 16>(g, args...);
  return by_type<F, 32>(g, args...);
}

unsigned gate_grid(const hmm_gate& g) {
  return static_cast<unsigned>((g.T + GATE_WARPS - 1) / GATE_WARPS);
}

struct RunForward {
  template <int NV, bool BF16, bool SIG>
  static cudaError_t run(const hmm_gate& g, const void* logits, const float* bias, int32_t* ids,
                         void* weights, float* scores, cudaStream_t st, bool pdl) {
    const size_t smem = g.groups > 1 ? sizeof(float) * GATE_WARPS * g.E : 0;
    return launch_kernel(gate_forward_kernel<NV, BF16, SIG>, gate_grid(g), GATE_WARPS * 32, smem,
                         st, pdl, 1, gate_args(g), logits, bias, ids, weights, scores);
  }
};

struct RunBackward {
  template <int NV, bool BF16, bool SIG>
  static cudaError_t run(const hmm_gate& g, const void* logits, const int32_t* ids,
                         const void* d_weights, const float* d_scores, void* d_logits,
                         cudaStream_t st, bool pdl) {
    const size_t smem = sizeof(float) * GATE_WARPS * g.E;
    return launch_kernel(gate_backward_kernel<NV, BF16, SIG>, gate_grid(g), GATE_WARPS * 32, smem,
                         st, pdl, 1, gate_args(g), logits, ids, d_weights, d_scores, d_logits);
  }
};

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
  return by_length<RunForward>(g, logits, bias, ids, weights, scores, st, pdl);
}

cudaError_t launch_gate_backward(const hmm_gate& g, const void* logits, const int32_t* ids,
                                 const void* d_weights, const float* d_scores, void* d_logits,
                                 cudaStream_t st, bool pdl) {
  return by_length<RunBackward>(g, logits, ids, d_weights, d_scores, d_logits, st, pdl);
}

}  // namespace hmm
