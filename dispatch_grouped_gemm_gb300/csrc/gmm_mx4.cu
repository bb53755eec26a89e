// gmm_mx4.cu -- the experts' products with microscaled 4-bit operands: token
// dispatch with quantisation, and GMM1 (SwiGLU and re-quantisation in its
// epilogue) and GMM2 in one persistent launch.
//
//   a = Q(silu(Q(x) . W1g^T) * (Q(x) . W1u^T)),   o = a . W2^T    per expert
//
// tcgen05.mma kind::mxf4 multiplies e2m1 codes with one power-of-two scale per
// 32 elements of the contraction on either side, accumulating in fp32.  The
// token rows sit on M (128 TMEM lanes), the weight rows on N (256 accumulator
// columns): a thread of the epilogue then holds whole blocks of 32
// consecutive outputs of one token, so a block's maximum, its scale and its
// codes need no exchange between threads.  Both operands are contraction-major
// with 128-byte rows of 256 elements per K block; their scales come as 512-byte
// tiles (128 rows x 4 blocks) that tcgen05.cp spreads over the TMEM lanes.
//
// TMEM: two accumulators of 256 columns and 24 columns of scales do not fit
// into 512 columns side by side, so the accumulators share 32 columns: [0, 256)
// and [224, 480), scales from 480.  A tile that would write shared columns of
// the tile before waits until its epilogue has read those, which it does first;
// that costs about 0.6 us per tile.  (Tiles of 192 weight rows, which share
// nothing, were slower all the same: 106 us for 99 at T = 4096, H = 2048, I =
// 1408.  The loads from L2 bound the loop, and narrower tiles load more.)  Tiles
// of 128 rows wait for the accumulator's previous use only.
//
// The rows of the up-projection are stored as 32 gate rows and the matching 32
// up rows in turn: accumulator columns 64 c .. 64 c + 31 are the gate and the
// next 32 the up values of chunk c.
#include <cuda_bf16.h>

#include <algorithm>

#include "mx4.cuh"
#include "ptx.cuh"

namespace hmm {

namespace {

constexpr int XM = 128;              // token rows per tile
constexpr int XN = 256;              // weight rows per tile
constexpr int XK = 256;              // contraction per stage: 128 bytes of codes
constexpr int XA_BYTES = XM * 128;   // 16 KB
constexpr int XB_BYTES = XN * 128;   // 32 KB
constexpr int XS_BYTES = 2 * MX_TILE_BYTES;  // scales of 128 rows
constexpr int XSTAGE_BYTES = XA_BYTES + XB_BYTES + 3 * XS_BYTES;  // 51 KB
constexpr int XSTAGES = 4;
constexpr int XRING = XSTAGES * XSTAGE_BYTES;
// CTA pairs: each CTA stages its 128 token rows, half of the weight rows, and the
// scales of all of them
constexpr int XP_B_BYTES = XB_BYTES / 2;
constexpr int XP_STAGE_BYTES = XA_BYTES + XP_B_BYTES + 3 * XS_BYTES;  // 35 KB
constexpr int XP_STAGES = XRING / XP_STAGE_BYTES;                     // 5
constexpr int XP_W_BYTES = XP_B_BYTES + 2 * XS_BYTES;  // loads of one CTA and stage
constexpr int XP_T_BYTES = XA_BYTES + XS_BYTES;
static_assert(XP_STAGES >= XSTAGES, "ring");
constexpr int XEPI_WARPS = 8;        // two per TMEM lane quarter
constexpr int XTOKEN_WARP = 3 + XEPI_WARPS;
constexpr int XTHREADS = 32 * (XEPI_WARPS + 4);
constexpr int XBUF = 32 * 64;        // staged output: 32 rows of 32 bf16
constexpr int XTI_DEPTH = 3;
constexpr int XACC1 = XN - 32;       // second accumulator's first column
constexpr int XSF_COL = XACC1 + XN;  // scales of A: 2 x 4 columns, then of B: 2 x 8
constexpr int XBARS = 2 * XP_STAGES + 5 + 2 * XTI_DEPTH + 2;
constexpr int XSMEM = 1024 + XRING + XEPI_WARPS * XBUF + 256 +
                      XTI_DEPTH * 24 + 32 + 4 * (MAX_E + 1);
static_assert(XSMEM <= 232448, "shared memory per CTA");
static_assert(XSF_COL + 24 <= 512, "TMEM columns");
static_assert(XBARS * 8 <= 256, "barriers");

struct XProb {
  int kp;        // contraction, padded to 32
  int n;         // stored weight rows
  int rt;        // scale tiles along them
};

struct XParams {
  XProb p[2];
  const int32_t* poff;
  const int32_t* counts;
  int E;
  int* ticket;      // tiles taken
  int* ready;       // per 128 token rows: epilogue warps of GMM1 that are done
  int signal;       // 0: test-only fault injection, nothing is released
  uint8_t* a_codes;
  uint8_t* a_scales;
  int a_blocks;     // blocks of 32 along I
  int a_pitch;      // bytes of a row of a
  int a_kt;
  __nv_bfloat16* o;
  int H;
  unsigned* status;
  unsigned long long budget_ns;
};

// Weight rows per tile: 256, or 128 where a problem has at most one tile of 128
// per CTA, so that the work spreads over more SMs (a graph of 21 calls, 128 and
// 256 wide in both problems, even and Zipf(1.2) routing: within the limit T = 1, H =
// 1024, I = 512 15.8 and 16.9, 15.5 and 16.8 us; T = 1, H = 2048, I = 1408 20.1 and
// 20.8, 20.1 and 20.8; T = 64, E = 8, H = 1024, I = 512 17.3 and 18.3, 17.2 and
// 18.4; above it T = 47, E = 30, H = 3792, I = 536 35.1 and 32.6, 34.3 and 33.6; T =
// 512, E = 8, H = 4096, I = 1024 33.4 and 31.5, 33.4 and 31.7; T = 700, E = 8, H = I =
// 1024 24.0 and 22.9, 23.3 and 22.9).  The token blocks are known on the device
// only, so every CTA decides there, which costs about a microsecond beside kernels
// built for one width (T = 1, H = 2048 21.4, T = 1, H = 1024 15.6).
__device__ __forceinline__ uint32_t xtiles(const XProb& p, uint32_t tn) {
  return (static_cast<uint32_t>(p.n) + tn - 1) / tn;
}
__device__ __forceinline__ uint32_t xwidth(const XProb& p, uint32_t blocks) {
  return blocks * xtiles(p, XN / 2) <= gridDim.x ? XN / 2 : XN;
}

struct XMaps {
  CUtensorMap a[2][2];  // token rows: boxes of 32 and 128 rows
  CUtensorMap w[2][2];  // weights: boxes of 128 and 256 rows
  CUtensorMap o;        // expert outputs: boxes of 32 rows x 32 columns
  CUtensorMap sa[2];    // scales of the token rows: one scale tile row, 2 tiles
  CUtensorMap sw[2][2]; // scales of the weights: 1 and 2 scale tile rows, 2 tiles each
};

struct XTile {
  int prob;  // -1: no more tiles
  int e;
  int row0;  // first padded token row
  int rows;  // valid rows, 1 .. 128 (pairs: 1 .. 256, the odd CTA has those from 128)
  int n0;    // first weight row
  int tn;    // weight rows: 128 or 256
};

// ---------------------------------------------------------------------- PTX
// The issuing warps run their loops with all lanes and issue under elect_one().
// (With a lane == 0 branch around the loops an MMA took 205 and a scale copy 111
// cycles to issue, 1490 per K block, for 540 cycles of tensor work.)
//
// Store the box at src to the tensor at {c0, c1}; parts outside it are left out.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, const void* src, int c0,
                                             int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(m)),
      "r"(smem_u32(src)), "r"(c0), "r"(c1)
      : "memory");
}
// 512 bytes of scales (32 lanes x 16 bytes) to 4 TMEM columns, the same in
// each of the four lane quarters.
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}
// D[tmem] (+)= A * B, e2m1 codes with a ue8m0 scale per 32 elements.
__device__ __forceinline__ void umma_mx4(uint32_t d, uint64_t adesc, uint64_t bdesc,
                                         uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], "
      "[%6], p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}
// The same for a CTA pair: scales of either CTA from its own shared memory to
// its own TMEM; D of both CTAs, A by CTA, B half from each.
__device__ __forceinline__ void tmem_cp_scales_pair(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}
__device__ __forceinline__ void umma_mx4_pair(uint32_t d, uint64_t adesc, uint64_t bdesc,
                                              uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], "
      "[%6], p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void cp_scales(uint32_t taddr, uint64_t desc) {
  if constexpr (PAIR)
    tmem_cp_scales_pair(taddr, desc);
  else
    tmem_cp_scales(taddr, desc);
}
template <bool PAIR>
__device__ __forceinline__ void umma(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                     uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if constexpr (PAIR)
    umma_mx4_pair(d, adesc, bdesc, idesc, sfa, sfb, accumulate);
  else
    umma_mx4(d, adesc, bdesc, idesc, sfa, sfb, accumulate);
}
// Instruction descriptor of kind::mxf4: e2m1 x e2m1, ue8m0 scales, both
// operands K-major; sf: which half of a 4-byte scale column (0 or 2).
template <bool PAIR>
__device__ __forceinline__ uint32_t idesc_mx4(int n, uint32_t sf) {
  return (sf << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) |
         (static_cast<uint32_t>((PAIR ? 2 * XM : XM) >> 4) << 24) | (sf << 29);
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// ---------------------------------------------------------------- scheduling
// Tickets run over the GMM1 tiles of all experts, then over the GMM2 tiles.
// pref[e]: token blocks of the experts before e, times 128, plus the rows that
// e's last block lacks (0 .. 127); pref[E]: all token blocks, times 128.  (The
// padded row space gives every expert whole blocks, so 128 times its blocks is
// also e's first row.)  Pairs: the same with pairs of blocks, whose first rows come
// from poff.
template <bool PAIR>
__device__ void xschedule(const XParams& P, uint32_t* pref) {
  constexpr int U = 8;  // loads in flight per lane
  const int lane = threadIdx.x & 31;
  uint32_t carry = 0;
  for (int base = 0; base < P.E; base += 32 * U) {
    uint32_t cnt[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = base + 32 * u + lane;
      cnt[u] = e < P.E ? static_cast<uint32_t>(__ldcg(P.counts + e)) : 0u;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = base + 32 * u + lane;
      const uint32_t lack = (XM - cnt[u] % XM) % XM;
      const uint32_t blocks = PAIR ? (cnt[u] + 2 * XM - 1) / (2 * XM) : (cnt[u] + XM - 1) / XM;
      uint32_t inc = blocks;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t n = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += n;
      }
      if (e < P.E) pref[e] = ((carry + inc - blocks) << 7) | lack;
      carry += __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  if (lane == 0) pref[P.E] = carry << 7;
  __syncwarp();
}

template <bool PAIR>
__device__ bool xlocate(const XParams& P, const uint32_t* pref, uint32_t t, XTile& ti) {
  const uint32_t blocks = pref[P.E] >> 7;
  ti.prob = 0;
  ti.tn = PAIR ? XN : xwidth(P.p[0], blocks);
  uint32_t nt = xtiles(P.p[0], ti.tn);
  if (t >= blocks * nt) {
    t -= blocks * nt;
    ti.prob = 1;
    ti.tn = PAIR ? XN : xwidth(P.p[1], blocks);
    nt = xtiles(P.p[1], ti.tn);
  }
  if (t >= blocks * nt) {
    ti.prob = -1;
    return false;
  }
  int lo = 0, hi = P.E - 1;  // largest expert whose first tile is at most t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((pref[mid] >> 7) * nt <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  ti.e = lo;
  const uint32_t b0 = pref[lo] >> 7, nb = (pref[lo + 1] >> 7) - b0;
  const uint32_t r = t - b0 * nt;
  const uint32_t wt = r / nb;  // token blocks innermost: a weight tile is reused from L2
  const uint32_t b = r - wt * nb;
  if constexpr (PAIR) {
    ti.row0 = __ldcg(P.poff + lo) + static_cast<int>(b) * 2 * XM;
    ti.rows = min(2 * XM, __ldcg(P.counts + lo) - static_cast<int>(b) * 2 * XM);
  } else {
    ti.row0 = static_cast<int>((b0 + b) * XM);
    ti.rows = b + 1 == nb ? XM - static_cast<int>(pref[lo] & 127u) : XM;
  }
  ti.n0 = static_cast<int>(wt * ti.tn);
  return true;
}

// ------------------------------------------------------------------ epilogue
// GMM1: one chunk (32 gate and 32 up columns) of this thread's row.  Returns
// the block's scale byte and writes its codes.
__device__ __forceinline__ uint32_t swiglu_block(const uint32_t (&g)[32], const uint32_t (&u)[32],
                                                 uint4* codes, bool valid) {
  float v[32];
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const float x = __uint_as_float(g[j]);
    // silu(g) * u; exp(-g) overflowing to inf gives 0.  (The fast exponential and
    // division: about 1e-6 relative, where the rounding to 4 bits that follows
    // is 1e-1; a value that close to a rounding boundary is one in 10^5, and the
    // order of the sums of g and u moves it as easily.)
    v[j] = __fdividef(x, 1.0f + __expf(-x)) * __uint_as_float(u[j]);
    m = max_nan(m, fabsf(v[j]));
  }
  const uint32_t s = mx_scale_byte(__float_as_uint(m));
  const float inv = mx_inverse_scale(s);
  uint32_t q[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = v[8 * j + k] * inv;
    q[j] = mx_codes8(w);
  }
  if (valid) *codes = make_uint4(q[0], q[1], q[2], q[3]);
  return s;
}

}  // namespace

// PAIR: clusters of two CTAs run 256 token rows x 256 weight rows with 2-SM MMAs:
// each CTA holds its 128 token rows and half of the weight rows, so that a stage
// is 35 KB for the same work per SM, and five fit.  The even CTA schedules, arms
// the stages for both CTAs' loads and issues.  Single CTAs and pairs, us of this
// kernel with evenly spread tokens: H = 7168, I = 2048, E = 32, K = 8: T = 16384
// 1823 and 1638 (skewed 1873 and 1690), T = 4096 523 and 484; H = 2048, I = 1408,
// K = 6: E = 64, T = 16384 371 and 349, T = 8192 203 and 200, T = 6144 (4.5 blocks
// an expert) 162 and 173, T = 4096 121 and 125; E = 6, T = 2048 55.5 and 53.2, T =
// 1024 (too few tiles) 35.6 and 36.4; H = 1024, I = 512, E = 8, K = 2, T = 16384
// (contractions of 4 and 2 stages) 44.8 and 46.5.
template <bool PAIR>
__global__ void __launch_bounds__(XTHREADS, 1)
    gmm_mx4_kernel(const __grid_constant__ XParams P, const __grid_constant__ XMaps maps) {
  constexpr int NST = PAIR ? XP_STAGES : XSTAGES;
  constexpr int SBYTES = PAIR ? XP_STAGE_BYTES : XSTAGE_BYTES;
  constexpr int BBYTES = PAIR ? XP_B_BYTES : XB_BYTES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* bufs = smem + XRING;
  uint64_t* bars = reinterpret_cast<uint64_t*>(bufs + XEPI_WARPS * XBUF);
  uint64_t* full = bars;
  uint64_t* empty = bars + NST;
  uint64_t* tfull = bars + 2 * NST;      // [2]
  uint64_t* tempty = tfull + 2;          // [2] the accumulator has been read
  uint64_t* tfree = tempty + 2;          // one phase per tile: its shared columns have been
                                         // read, and all of the tile before
  uint64_t* ti_full = tfree + 1;
  uint64_t* ti_empty = ti_full + XTI_DEPTH;
  uint64_t* mma_done = ti_empty + XTI_DEPTH;
  uint64_t* want = mma_done + 1;
  XTile* s_ti = reinterpret_cast<XTile*>(bars + 32);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(s_ti + XTI_DEPTH);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  uint32_t* s_issued = s_tmem + 2;  // stages issued by the two producers
  uint32_t* s_peer = s_tmem + 4;    // even CTA of a pair: the odd one's counts and abort flag
  uint32_t* s_pref = s_tmem + 8;    // [E + 1]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  constexpr int EPIS = PAIR ? 2 * XEPI_WARPS : XEPI_WARPS;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&full[s], 2);  // both producers arm it
      mbar_init(&empty[s], 1);
    }
    mbar_init(&tfull[0], 1);
    mbar_init(&tfull[1], 1);
    mbar_init(&tempty[0], EPIS);
    mbar_init(&tempty[1], EPIS);
    mbar_init(tfree, EPIS);
    for (int i = 0; i < XTI_DEPTH; ++i) {
      mbar_init(&ti_full[i], 1);
      // producers, MMA issuer, epilogue warps (+ the odd CTA's producers and epilogue)
      mbar_init(&ti_empty[i], 3 + EPIS + (PAIR ? 2 : 0));
    }
    mbar_init(mma_done, 1);
    mbar_init(want, 1);
    *s_abort = 0;
    fence_mbar_init();
  }
  if constexpr (PAIR) cluster_sync_all();  // barriers initialised before any remote arrive
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(s_tmem, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(s_tmem, 512);
      tmem_relinquish();
    }
  } else if (warp == 0 && lane < 2) {
    for (int i = 0; i < 2; ++i) {
      tma_prefetch_desc(&maps.w[lane][i]);
      tma_prefetch_desc(&maps.sw[lane][i]);
    }
    tma_prefetch_desc(&maps.sa[lane]);
    tma_prefetch_desc(&maps.a[lane][0]);
    tma_prefetch_desc(&maps.a[lane][1]);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *s_tmem, 0);  // uniform
  // The previous kernel (the dispatch of x) lets this one in after its own wait
  // for the routing, so the routing's results are there (read past L1, which
  // could hold older ones) and the weights can start; only the token rows of
  // GMM1 wait for the dispatch itself.
  const WaitCtl wc{s_abort, P.status, P.budget_ns};
  // arrivals on the even CTA's barriers
  auto arrive = [&](uint64_t* bar) {
    if (!PAIR || leader)
      mbar_arrive(bar);
    else
      mbar_arrive_peer(mapa_shared(smem_u32(bar), 0));
  };

  if (warp == 2 + XEPI_WARPS) {
    // --------------------------------------------------------- tile scheduler
    // Every tile comes by ticket, the first one too: a tile belongs to a CTA
    // that runs, however many of the grid's CTAs have an SM (another stream's
    // kernel may hold some), so that GMM2's wait for GMM1 below cannot wait for
    // a CTA that has not started.  The first ticket is drawn beside the prefix
    // scan, the later ones only when the producer is about to need them
    // (`want`): the atomic's latency is hidden, and a CTA does not sit on a
    // second tile while another has none.  (With tickets drawn as soon as a slot
    // was free, half of the CTAs took two of a decode step's 128 GMM1 tiles.)
    uint32_t t = 0;
    if (lane == 0 && leader) t = static_cast<uint32_t>(atomicAdd(P.ticket, 1));
    if (leader) xschedule<PAIR>(P, s_pref);
    if (lane == 0 && leader) {
      int slot = 0;
      uint32_t phase = 0, want_phase = 0;
      for (;;) {
        XTile ti{-1, 0, 0, 0, 0, 0};
        xlocate<PAIR>(P, s_pref, t, ti);
        if (!mbar_wait<PAIR>(&ti_empty[slot], phase ^ 1u, wc)) break;
        s_ti[slot] = ti;
        if constexpr (PAIR) {
          const uint32_t dst = mapa_shared(smem_u32(&s_ti[slot]), 1);
          const int* src = reinterpret_cast<const int*>(&ti);
#pragma unroll
          for (int j = 0; j < static_cast<int>(sizeof(XTile) / 4); ++j)
            st_shared_cluster(dst + 4 * j, src[j]);
          mbar_arrive_cluster(mapa_shared(smem_u32(&ti_full[slot]), 1));
        }
        mbar_arrive(&ti_full[slot]);
        if (++slot == XTI_DEPTH) {
          slot = 0;
          phase ^= 1u;
        }
        if (ti.prob < 0) break;
        if (!mbar_wait(want, want_phase, wc)) break;
        want_phase ^= 1u;
        t = static_cast<uint32_t>(atomicAdd(P.ticket, 1));
      }
    }
  } else if (warp == 0 || warp == XTOKEN_WARP) {
    // --------------------------------------------------------------- producers
    // One warp for the weights and their scales, one for the token rows and
    // theirs: each arms a stage for its own bytes.  Weights wait for nothing:
    // while GMM2's token rows are not there yet, they are streamed into the free
    // stages.
    const bool weights = warp == 0;
    if (!weights) grid_dep_wait();
    uint32_t stage = 0, sphase = 0, issued = 0;
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (;;) {
      ok = warp_all(mbar_wait<PAIR>(&ti_full[slot], phase, wc));
      if (!ok) break;
      const XTile ti = s_ti[slot];
      __syncwarp();
      if (elect_one()) arrive(&ti_empty[slot]);
      if (++slot == XTI_DEPTH) {
        slot = 0;
        phase ^= 1u;
      }
      if (ti.prob < 0) break;
      const XProb& pr = P.p[ti.prob];
      const int nkb = (pr.kp + XK - 1) / XK;
      auto next_stage = [&]() {
        __syncwarp();
        ++issued;
        if (++stage == NST) {
          stage = 0;
          sphase ^= 1u;
        }
      };
      if (weights) {
        // (a pair's tile takes the first half of its weight rows from the even
        // CTA, the second from the odd one)
        const int cols = min(ti.tn, (pr.n - ti.n0 + 31) / 32 * 32);
        const int first = ti.n0 + static_cast<int>(rank) * cols / 2;
        const CUtensorMap* mw = &maps.w[ti.prob][PAIR ? 0 : ti.tn / 128 - 1];
        const CUtensorMap* msw = &maps.sw[ti.prob][ti.tn / 128 - 1];
        const uint32_t bytes = PAIR ? 2 * XP_W_BYTES : ti.tn * 128 + ti.tn / 128 * XS_BYTES;
        const int wrow = ti.e * pr.rt + ti.n0 / 128;
        const int ask = max(0, nkb - 8);  // K block at which the next tile is asked for
        for (int kb = 0; kb < nkb; ++kb) {
          ok = warp_all(mbar_wait(&empty[stage], sphase ^ 1u, wc));
          if (!ok) break;
          if (elect_one()) {
            uint8_t* sB = smem + stage * SBYTES + XA_BYTES;
            if constexpr (PAIR) {
              const uint32_t bar = mapa_shared(smem_u32(&full[stage]), 0);
              if (leader) mbar_arrive_expect_tx(&full[stage], bytes);
              tma_load_3d_pair(sB, mw, bar, kb * (XK / 2), first, ti.e);
              tma_load_2d_pair(sB + BBYTES + XS_BYTES, msw, bar, kb * 256, wrow);
            } else {
              mbar_arrive_expect_tx(&full[stage], bytes);
              tma_load_3d(sB, mw, &full[stage], kb * (XK / 2), ti.n0, ti.e);
              tma_load_2d(sB + BBYTES + XS_BYTES, msw, &full[stage], kb * 256, wrow);
            }
            if (kb == ask && leader) mbar_arrive(want);
          }
          next_stage();
        }
      } else {
        const int row0 = ti.row0 + XM * static_cast<int>(rank);
        const bool few = !PAIR && ti.rows <= 32;
        const CUtensorMap* ma = &maps.a[ti.prob][few ? 0 : 1];
        const CUtensorMap* msa = &maps.sa[ti.prob];
        const uint32_t bytes = PAIR ? 2 * XP_T_BYTES : (few ? 32 : XM) * 128 + XS_BYTES;
        if (ti.prob == 1 && ti.rows > XM * static_cast<int>(rank)) {
          // a comes from this launch's GMM1 tiles; each has a smaller ticket,
          // which a running CTA drew, and GMM1 tiles wait for no other tile.
          // Order the counter's acquire with the asynchronous copies of a.
          // (all of GMM1's tiles of these rows, every epilogue warp once)
          const int done =
              XEPI_WARPS * xtiles(P.p[0], PAIR ? XN : xwidth(P.p[0], s_pref[P.E] >> 7));
          ok = warp_all(lane != 0 || counter_wait(&P.ready[row0 / XM], done, wc));
          if (!ok) break;
          fence_proxy_async_global();
        }
        for (int kb = 0; kb < nkb; ++kb) {
          ok = warp_all(mbar_wait(&empty[stage], sphase ^ 1u, wc));
          if (!ok) break;
          if (elect_one()) {
            uint8_t* sA = smem + stage * SBYTES;
            if constexpr (PAIR) {
              const uint32_t bar = mapa_shared(smem_u32(&full[stage]), 0);
              if (leader) mbar_arrive_expect_tx(&full[stage], bytes);
              tma_load_2d_pair(sA, ma, bar, kb * (XK / 2), row0);
              tma_load_2d_pair(sA + XA_BYTES + BBYTES, msa, bar, kb * 256, row0 / XM);
            } else {
              mbar_arrive_expect_tx(&full[stage], bytes);
              tma_load_2d(sA, ma, &full[stage], kb * (XK / 2), row0);
              tma_load_2d(sA + XA_BYTES + BBYTES, msa, &full[stage], kb * 256, row0 / XM);
            }
          }
          next_stage();
        }
      }
      if (!ok) break;
    }
    if (lane == 0) s_issued[weights ? 0 : 1] = issued;
    if (weights) grid_dep_launch();  // this CTA is in its last tile
  } else if (warp == 1 && (!PAIR || leader)) {
    // -------------------------------------------------------------- MMA issue
    uint32_t stage = 0, sphase = 0;
    int slot = 0;
    uint32_t phase = 0;
    uint32_t n = 0;  // tiles so far
    int last_cols = 0;  // columns of the tile before
    for (;;) {
      if (!warp_all(mbar_wait<PAIR>(&ti_full[slot], phase, wc))) break;
      const int prob = __shfl_sync(0xffffffffu, s_ti[slot].prob, 0);
      const int n0 = __shfl_sync(0xffffffffu, s_ti[slot].n0, 0);
      const int tn = __shfl_sync(0xffffffffu, s_ti[slot].tn, 0);
      if (elect_one()) mbar_arrive(&ti_empty[slot]);
      if (++slot == XTI_DEPTH) {
        slot = 0;
        phase ^= 1u;
      }
      if (prob < 0) break;
      const int kp = prob == 0 ? P.p[0].kp : P.p[1].kp;
      const int rows = prob == 0 ? P.p[0].n : P.p[1].n;
      const uint32_t acc = n & 1u;
      const uint32_t d = tmem + acc * XACC1;
      const int cols = min(tn, (rows - n0 + 31) / 32 * 32);
      // the accumulator-0 one of this tile and the tile before decides whether
      // the two meet
      const bool shared = n > 0 && (acc ? last_cols : cols) > XACC1;
      last_cols = cols;
      // the first operands, then the accumulator: the waits' latencies overlap
      bool ok = warp_all(mbar_wait(&full[stage], sphase, wc));
      if (!ok) break;
      // (always the accumulator's last use: with it tfree has completed the phase
      // of tile n - 2, so that the parity below can only mean tile n - 1's)
      ok = warp_all(mbar_wait<PAIR>(&tempty[acc], ((n >> 1) & 1u) ^ 1u, wc));
      if (ok && shared) ok = warp_all(mbar_wait<PAIR>(tfree, (n - 1) & 1u, wc));
      if (!ok) break;
      const bool wide = cols > 128;  // the second scale tile row is in use
      const uint32_t id0 = idesc_mx4<PAIR>(cols, 0), id1 = idesc_mx4<PAIR>(cols, 2);
      const uint32_t sfa = tmem + XSF_COL, sfb = tmem + XSF_COL + 8;
      for (int k = 0; k < kp; k += XK) {
        if (k > 0) ok = warp_all(mbar_wait(&full[stage], sphase, wc));
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t a = smem_u32(smem) + stage * SBYTES;
          const uint32_t b = a + XA_BYTES, sc = b + BBYTES;
          const uint64_t da = smem_desc(a, 16, 1024, LAYOUT_SW128);
          const uint64_t db = smem_desc(b, 16, 1024, LAYOUT_SW128);
          const uint64_t ds = smem_desc(sc, 0, 128, LAYOUT_NONE);
          const uint64_t dt = smem_desc(sc + XS_BYTES, 0, 128, LAYOUT_NONE);
          const int left = kp - k;
          // scales of 128 elements, the MMAs of 64 elements that use them
          // (descriptor addresses count 16 bytes)
          if (left >= XK && wide) {
            // a whole K block without a branch between the instructions (with
            // the conditions of the other path: 103 us for 99 at T = 4096)
            cp_scales<PAIR>(sfa, ds);
            cp_scales<PAIR>(sfb, dt);
            cp_scales<PAIR>(sfb + 4, dt + 64);
            cp_scales<PAIR>(sfa + 4, ds + 32);
            cp_scales<PAIR>(sfb + 8, dt + 32);
            cp_scales<PAIR>(sfb + 12, dt + 96);
            umma<PAIR>(d, da, db, id0, sfa, sfb, k > 0 ? 1u : 0u);
            umma<PAIR>(d, da + 2, db + 2, id1, sfa, sfb, 1u);
            umma<PAIR>(d, da + 4, db + 4, id0, sfa + 4, sfb + 8, 1u);
            umma<PAIR>(d, da + 6, db + 6, id1, sfa + 4, sfb + 8, 1u);
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (128 * i < left) {
                cp_scales<PAIR>(sfa + 4 * i, ds + i * 32);
                cp_scales<PAIR>(sfb + 8 * i, dt + i * 32);
                if (wide) cp_scales<PAIR>(sfb + 4 + 8 * i, dt + (2 + i) * 32);
              }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (64 * j < left)
                umma<PAIR>(d, da + 2 * j, db + 2 * j, (j & 1) ? id1 : id0, sfa + 4 * (j >> 1),
                         sfb + 8 * (j >> 1), (k > 0 || j > 0) ? 1u : 0u);
          }
          if constexpr (PAIR)
            umma_commit_pair(&empty[stage], 0x3);
          else
            umma_commit(&empty[stage]);
        }
        __syncwarp();
        if (++stage == NST) {
          stage = 0;
          sphase ^= 1u;
        }
      }
      if (!ok) break;
      if (elect_one()) {
        if constexpr (PAIR)
          umma_commit_pair(&tfull[acc], 0x3);
        else
          umma_commit(&tfull[acc]);
      }
      __syncwarp();
      ++n;
    }
    // every MMA issued by this warp's elected lane completes before TMEM is released
    __syncwarp();
    if (elect_one()) {
      if constexpr (PAIR)
        umma_commit_pair(mma_done, 0x1);
      else
        umma_commit(mma_done);
    }
    __syncwarp();
    drain_wait(mma_done, 0, P.budget_ns);
  } else if (warp >= 2 && warp < 2 + XEPI_WARPS) {
    // --------------------------------------------------------------- epilogue
    const int q = warp & 3;          // TMEM lane quarter
    const int h = (warp - 2) >> 2;   // half of the tile's columns
    uint8_t* buf = bufs + (warp - 2) * XBUF;
    int slot = 0;
    uint32_t phase = 0;
    uint32_t n = 0;
    for (;;) {
      bool got = false;
      if (lane == 0) got = mbar_wait<PAIR>(&ti_full[slot], phase, wc);
      got = __shfl_sync(0xffffffffu, got, 0);
      if (!got) break;
      XTile ti = s_ti[slot];
      __syncwarp();
      if (lane == 0) arrive(&ti_empty[slot]);
      if constexpr (PAIR) {  // this CTA's rows (none for the odd CTA of a last block)
        ti.row0 += XM * static_cast<int>(rank);
        ti.rows = min(XM, ti.rows - XM * static_cast<int>(rank));
      }
      if (++slot == XTI_DEPTH) {
        slot = 0;
        phase ^= 1u;
      }
      if (ti.prob < 0) break;
      const uint32_t acc = n & 1u;
      // Accumulator 0 shares its last columns (half 1), accumulator 1 its first
      // (half 0).  The half that does not read them says only that it has left
      // the previous tile, once this tile's accumulator is complete.  (Where
      // neighbouring tiles share no columns nobody waits for the barrier, so a
      // warp may be a tile ahead of another and both count in one phase.  That
      // mixes no phases up: the issuer waits for tempty, every warp's read of tile
      // n - 2, before it starts tile n, so by then the barrier has counted that
      // tile's arrivals in full, and at tfree it can only be short of tile n - 1's.)
      const bool shares = h == (acc ^ 1);
      const bool live = 32 * q < ti.rows;
      uint64_t* drained = &tempty[acc];
      if (lane == 0) got = mbar_wait(&tfull[acc], (n >> 1) & 1u, wc);
      got = __shfl_sync(0xffffffffu, got, 0);
      if (!got) break;
      ++n;
      tc_fence_after();
      if (!(shares && live) && lane == 0) arrive(tfree);
      if (!live && lane == 0) arrive(drained);
      if (live) {
        const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * XACC1;
        const int row = 32 * q + lane;
        const bool valid = row < ti.rows;
        if (ti.prob == 0) {
          // chunks of gate and up columns, the one with the shared columns
          // first: the last of half 1 (accumulator 0), the first of half 0
          const int64_t prow = ti.row0 + row;
          const int nch = ti.tn / 64, mine = nch / 2;
          uint8_t* crow = P.a_codes + prow * P.a_pitch;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (i < mine) {
              const int c = h ? nch - 1 - i : i;
              uint32_t g[32], u[32];
              if (i == 0 && shares) {
                // the 32 shared columns alone: the up half (half 1), the gate half
                if (h)
                  tmem_ld32(taddr + 64 * c + 32, u);
                else
                  tmem_ld32(taddr + 64 * c, g);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive(tfree);
                if (h)
                  tmem_ld32(taddr + 64 * c, g);
                else
                  tmem_ld32(taddr + 64 * c + 32, u);
              } else {
                tmem_ld32(taddr + 64 * c, g);
                tmem_ld32(taddr + 64 * c + 32, u);
              }
              tmem_ld_wait_for(g);
              tmem_ld_wait_for(u);
              if (i + 1 == mine) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive(drained);
              }
              const int blk = ti.n0 / 64 + c;
              if (blk < P.a_blocks) {
                const uint32_t s =
                    swiglu_block(g, u, reinterpret_cast<uint4*>(crow + blk * 16), valid);
                if (valid) {
                  uint8_t* at = P.a_scales + mx_scale_offset(prow, blk, P.a_kt);
                  // (a last block without a partner: the last MMA step of GMM2
                  // covers the missing one with zero codes, its scale is 0)
                  if (blk + 1 == P.a_blocks && !(blk & 1))
                    *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(s);
                  else
                    *at = static_cast<uint8_t>(s);
                }
              }
            }
          }
        } else {
          // 32 columns at a time, the shared ones first, rounded to bf16 as an
          // expert's output row is in hmm_forward (fp32 rows would double what the
          // combine reads back: 3.8 GB for 1.9 at T = 16384, H = 7168, K = 8, where
          // it takes 325 us of 2200; y's error is 2.4e-3 relative for 1.7e-3 of one
          // rounding), through this warp's buffer (16-byte pieces permuted by the row as the store's
          // 64-byte swizzle wants them: no bank conflicts).  Whole quarters of
          // 32 rows leave by one asynchronous tensor store; fewer rows by plain
          // stores of the valid ones, four lanes per row.
          const int nu = ti.tn / 64;  // units of this half
          const bool whole = ti.rows - 32 * q >= 32;
#pragma unroll 1
          for (int i = 0; i < nu; ++i) {
            const int c = h ? 2 * nu - 1 - i : i;
            uint32_t v[32];
            tmem_ld32(taddr + 32 * c, v);
            tmem_ld_wait_for(v);
            if (i == 0 && shares) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) arrive(tfree);
            }
            if (i + 1 == nu) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) arrive(drained);
            }
            const int c0 = ti.n0 + 32 * c;
            if (c0 >= P.H) continue;
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j)
              w[j] = pack_bf16(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
            if (lane == 0) bulk_wait_group_read<0>();  // the buffer's last store has read it
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<uint4*>(buf + lane * 64 + 16 * (j ^ ((lane >> 1) & 3))) =
                  make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
            if (whole) {
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_store_2d(&maps.o, buf, c0, ti.row0 + 32 * q);
                bulk_commit_group();
              }
            } else {
              __syncwarp();
#pragma unroll
              for (int r8 = 0; r8 < 4; ++r8) {
                const int r = 8 * r8 + (lane >> 2);
                const int col = c0 + 8 * (lane & 3);
                if (32 * q + r < ti.rows && col < P.H)
                  *reinterpret_cast<uint4*>(P.o + static_cast<int64_t>(ti.row0 + 32 * q + r) * P.H +
                                            col) =
                      *reinterpret_cast<const uint4*>(buf + r * 64 +
                                                      16 * ((lane & 3) ^ ((r >> 1) & 3)));
              }
            }
          }
        }
      }
      tc_fence_before();
      if (ti.prob == 0 && P.signal && (!PAIR || ti.rows > 0)) {
        fence_proxy_async_global();
        __syncwarp();
        if (lane == 0) red_release_add(&P.ready[ti.row0 / XM], 1);
      }
    }
    if (lane == 0) bulk_wait_group<0>();  // the stores of o are performed
  }
  tc_fence_before();
  __syncthreads();
  // The producers may have left after different numbers of stages: complete what
  // one of them never armed or loaded, and wait (bounded) for the last copies into
  // every slot before the memory goes.
  if constexpr (PAIR) {
    if (!leader && threadIdx.x == 0) {
      const uint32_t dst = mapa_shared(smem_u32(s_peer), 0);
      st_shared_cluster(dst, static_cast<int>(s_issued[0]));
      st_shared_cluster(dst + 4, static_cast<int>(s_issued[1]));
      st_shared_cluster(dst + 8, *s_abort);
    }
    cluster_sync_all();
    if (leader && threadIdx.x == 0 && (*s_abort || s_peer[2])) {
      uint32_t n = 0;
      for (int i = 0; i < 2; ++i) n = max(n, max(s_issued[i], s_peer[i]));
      for (uint32_t k = n > NST ? n - NST : 0u; k < n; ++k) {
        uint64_t* bar = &full[k % NST];
        for (int i = 0; i < 2; ++i) {
          const uint32_t bytes = i == 0 ? XP_W_BYTES : XP_T_BYTES;  // of one CTA
          if (k >= s_issued[i]) {  // never armed: for what the odd CTA loads, if it does
            if (k < s_peer[i])
              mbar_arrive_expect_tx(bar, bytes);
            else
              mbar_arrive(bar);
          } else if (k >= s_peer[i]) {
            mbar_complete_tx(bar, bytes);  // armed for both, loaded by the even CTA only
          }
        }
        drain_wait(bar, (k / NST) & 1u, P.budget_ns);
      }
    }
    cluster_sync_all();
  } else {
    if (*s_abort && threadIdx.x == 0) {
      const uint32_t n0 = s_issued[0], n1 = s_issued[1], n = max(n0, n1);
      for (uint32_t k = n > NST ? n - NST : 0u; k < n; ++k) {
        uint64_t* bar = &full[k % NST];
        if (k >= min(n0, n1)) mbar_arrive(bar);
        drain_wait(bar, (k / NST) & 1u, P.budget_ns);
      }
    }
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR)
      tmem_dealloc_pair(tmem, 512);
    else
      tmem_dealloc(tmem, 512);
  }
}

// Dispatch: token t's row of x in 4-bit form, once, to the padded rows of its
// K slots.  One warp per token and MXD_COLS columns; a lane holds 8 elements,
// four lanes a block, the first of which writes the scale.
namespace {
constexpr int MXD_UNROLL = 4;
constexpr int MXD_COLS = 256 * MXD_UNROLL;
constexpr int MXD_WARPS = 4;
}  // namespace

__global__ void __launch_bounds__(MXD_WARPS * 32)
    dispatch_mx4_kernel(const uint4* __restrict__ x, int64_t T, int K, int64_t H, int64_t kp,
                        int64_t kt, const int32_t* __restrict__ slot2prow,
                        uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, bool early) {
  const int lane = threadIdx.x & 31;
  const int64_t parts = (H + MXD_COLS - 1) / MXD_COLS;
  const int64_t g = static_cast<int64_t>(blockIdx.x) * MXD_WARPS + (threadIdx.x >> 5);
  const int64_t t = g / parts;
  // early (few tokens): x is read (past L1) and quantised before the wait for the
  // routing kernel: that kernel lets this one in after its own wait, so whatever
  // wrote x has completed.  With many tokens the rows' places are better fetched
  // beside x (T = 16384: 142 us, early 155 us).
  if (!early || t >= T) {
    grid_dep_wait();
    grid_dep_launch();
  }
  if (t >= T) return;
  const int64_t c0 = (g - t * parts) * MXD_COLS + 8 * lane;
  int32_t prow_l = -1;
  if (!early && lane < K) prow_l = slot2prow[t * K + lane];
  uint4 v[MXD_UNROLL];
#pragma unroll
  for (int i = 0; i < MXD_UNROLL; ++i) {
    const int64_t c = c0 + 256 * i;
    v[i] = c < H ? __ldcg(x + (t * H + c) / 8) : make_uint4(0, 0, 0, 0);
  }
  uint32_t q[MXD_UNROLL], s[MXD_UNROLL];
#pragma unroll
  for (int i = 0; i < MXD_UNROLL; ++i) {
    const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    const uint32_t b = quad_scale_bf16(u);
    q[i] = codes8_bf16(u, b);
    s[i] = b;
  }
  if (early) {
    grid_dep_wait();
    grid_dep_launch();
    if (lane < K) prow_l = slot2prow[t * K + lane];
  }
  // (a step of 256 columns: 128 bytes of codes, two scale tiles)
  for (int k = 0; k < K; ++k) {
    const int32_t prow = __shfl_sync(0xffffffffu, prow_l, k);
    if (prow < 0) continue;
    uint32_t* crow = reinterpret_cast<uint32_t*>(codes + prow * (kp / 2) + c0 / 2);
    uint8_t* srow = scales + mx_scale_offset(prow, c0 / 32, kt);
#pragma unroll
    for (int i = 0; i < MXD_UNROLL; ++i) {
      const int64_t c = c0 + 256 * i;
      if (c < kp) crow[32 * i] = q[i];
      if ((lane & 3) == 0 && c < kt * 128)
        srow[2 * MX_TILE_BYTES * i] = static_cast<uint8_t>(s[i]);
    }
  }
}

cudaError_t launch_dispatch_mx4(const Plan& p, const FfnMx4Plan& f, const void* x, MetaPtrs m,
                                uint8_t* codes, uint8_t* scales, cudaStream_t st, bool pdl) {
  const int64_t warps = p.T * ((p.H + MXD_COLS - 1) / MXD_COLS);
  return launch_kernel(dispatch_mx4_kernel,
                       static_cast<unsigned>((warps + MXD_WARPS - 1) / MXD_WARPS), MXD_WARPS * 32,
                       0, st, pdl, 1, static_cast<const uint4*>(x), p.T, static_cast<int>(p.K),
                       p.H, f.hp, f.h_kt, static_cast<const int32_t*>(m.slot2prow), codes, scales,
                       p.T < 1024);
}

namespace {

// codes [outer, rows, bytes] as a tensor map with boxes of 128 bytes x box rows
int map_codes(const GemmEnv& env, CUtensorMap* map, const void* base, int64_t bytes, int64_t rows,
              int64_t outer, uint32_t box_rows) {
  const cuuint32_t rank = outer > 0 ? 3 : 2;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(bytes), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(outer)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(bytes),
                                 static_cast<cuuint64_t>(bytes * rows)};
  const cuuint32_t box[3] = {128, box_rows, 1}, es[3] = {1, 1, 1};
  return env.encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(base), dims,
                    strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? HMM_OK
             : HMM_ERR_CUDA;
}

// a scale array (rows of kt tiles) with boxes of 2 tiles x box_rows rows
int map_scales(const GemmEnv& env, CUtensorMap* map, const void* base, int64_t kt, int64_t rows,
               uint32_t box_rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(kt * (MX_TILE_BYTES / 4)),
                              static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(kt * MX_TILE_BYTES)};
  const cuuint32_t box[2] = {2 * MX_TILE_BYTES / 4, box_rows}, es[2] = {1, 1};
  return env.encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, strides,
                    box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? HMM_OK
             : HMM_ERR_CUDA;
}

// expert outputs [rows, cols] bf16 with boxes of 32 x 32
int map_out(const GemmEnv& env, CUtensorMap* map, const void* base, int64_t cols, int64_t rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols * 2)};
  const cuuint32_t box[2] = {32, 32}, es[2] = {1, 1};
  return env.encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
                    strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                    CU_TENSOR_MAP_L2_PROMOTION_NONE,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? HMM_OK
             : HMM_ERR_CUDA;
}

}  // namespace

int launch_forward_mx4(const GemmEnv& env, const Plan& p, const FfnMx4Plan& f, MetaPtrs m,
                       CtrlPtrs c, uint8_t* ws, const void* up_codes, const void* up_scales,
                       const void* down_codes, const void* down_scales, bool skip_ready_release) {
  XMaps maps;
  XParams P{};
  int rc = HMM_OK;
  for (int i = 0; i < 2; ++i) {
    rc |= map_codes(env, &maps.a[0][i], ws + f.off_x, f.hp / 2, p.R, 0, i ? XM : 32);
    rc |= map_codes(env, &maps.a[1][i], ws + f.off_a, f.ip / 2, p.R, 0, i ? XM : 32);
  }
  for (int i = 0; i < 2; ++i) {
    const int tn = 128 * (i + 1);
    rc |= map_codes(env, &maps.w[0][i], up_codes, f.hp / 2, 2 * f.ip, p.E, tn);
    rc |= map_codes(env, &maps.w[1][i], down_codes, f.ip / 2, p.H, p.E, tn);
    rc |= map_scales(env, &maps.sw[0][i], up_scales, f.h_kt, p.E * ((2 * f.ip + 127) / 128),
                     tn / 128);
    rc |= map_scales(env, &maps.sw[1][i], down_scales, f.i_kt, p.E * ((p.H + 127) / 128),
                     tn / 128);
  }
  rc |= map_out(env, &maps.o, ws + f.off_o, p.H, p.R);
  rc |= map_scales(env, &maps.sa[0], ws + f.off_xs, f.h_kt, p.R / XM, 1);
  rc |= map_scales(env, &maps.sa[1], ws + f.off_as, f.i_kt, p.R / XM, 1);
  if (rc != HMM_OK) return HMM_ERR_CUDA;
  auto prob = [](XProb& q, int64_t kp, int64_t n) {
    q.kp = static_cast<int>(kp);
    q.n = static_cast<int>(n);
    q.rt = static_cast<int>((n + 127) / 128);
  };
  prob(P.p[0], f.hp, 2 * f.ip);
  prob(P.p[1], f.ip, p.H);
  P.poff = m.poff;
  P.counts = m.counts;
  P.E = static_cast<int>(p.E);
  P.ticket = c.tickets;
  P.ready = c.ready;
  P.signal = skip_ready_release ? 0 : 1;
  P.a_codes = ws + f.off_a;
  P.a_scales = ws + f.off_as;
  P.a_blocks = static_cast<int>(f.ip / 32);
  P.a_pitch = static_cast<int>(f.ip / 2);
  P.a_kt = static_cast<int>(f.i_kt);
  P.o = reinterpret_cast<__nv_bfloat16*>(ws + f.off_o);
  P.H = static_cast<int>(p.H);
  P.status = env.status;
  P.budget_ns = env.budget_ns;
  if (!*env.mx4_set) {  // once per context
    if (cudaFuncSetAttribute(gmm_mx4_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             XSMEM) != cudaSuccess ||
        cudaFuncSetAttribute(gmm_mx4_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             XSMEM) != cudaSuccess)
      return HMM_ERR_CUDA;
    *env.mx4_set = true;
  }
  const int64_t tiles = (p.R / XM) * ((2 * f.ip + 127) / 128 + (p.H + 127) / 128);
  if (tiles >= (int64_t(1) << 31)) return HMM_ERR_SHAPE;
  // Pairs: six token blocks per expert on average (an odd last one idles a CTA),
  // two GMM1 tiles per CTA, contractions long beside a tile's epilogue; both
  // sides' figures are at the kernel.
  const bool pays =
      p.TK >= int64_t(6) * XM * p.E && p.H >= 2048 &&
      p.TK / (2 * XM) * ((2 * f.ip + XN - 1) / XN) >= int64_t(2) * env.num_sms;
  const bool pair = env.mx4_pairs == 1 || (env.mx4_pairs == 2 && pays);
  if (pair) {
    // as many pairs as can be resident at once: the tiles wait for one another
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(env.num_sms / 2 * 2));
    cfg.blockDim = dim3(XTHREADS);
    cfg.dynamicSmemBytes = XSMEM;
    cfg.stream = env.stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int active = 0;
    if (cudaOccupancyMaxActiveClusters(&active, gmm_mx4_kernel<true>, &cfg) != cudaSuccess ||
        active <= 0)
      return HMM_ERR_CUDA;
    const unsigned clusters = static_cast<unsigned>(std::min(active, env.num_sms / 2));
    return launch_kernel(gmm_mx4_kernel<true>, 2 * clusters, XTHREADS, XSMEM, env.stream, env.pdl,
                         2, P, maps) == cudaSuccess
               ? HMM_OK
               : HMM_ERR_CUDA;
  }
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(env.num_sms, tiles));
  return launch_kernel(gmm_mx4_kernel<false>, grid, XTHREADS, XSMEM, env.stream, env.pdl, 1, P,
                       maps) == cudaSuccess
             ? HMM_OK
             : HMM_ERR_CUDA;
}

}  // namespace hmm
