// gmm_open.cu -- matrix products grouped by expert, and batched products of the
// orthogonalised weight update, on CTA pairs (tcgen05 cta_group::2).
//
// One product is acc(m, n) = sum_k A(m, k) B(n, k) over 16-bit operands with an
// fp32 accumulator in TMEM, for a list of (expert or matrix, tile of m, tile of
// n).  An operand lies in memory with k contiguous (K-major) or with m / n
// contiguous (MN-major); TMA brings either into shared memory as it is and the
// MMA reads it there, so nothing is transposed on the way.
//
//   ROWS    y[r, :] = x[r, :] . w[e] for the rows of expert e (forward and dx).
//           m = columns of y, n = rows of the expert: the MMA's N can be any
//           multiple of 16, so an expert's rows are split into equal blocks of at
//           most 256 and few rows cost few columns of work, while the weights,
//           256 columns per pair, fill the M side.
//   DEPTH   dw[e] = x_e^T . dy_e: the contraction runs over the rows of the expert.
//   STACK   products of a stack of matrices, with the epilogues of the
//           Newton-Schulz step (gmm_open.h).
//
// Rows of one expert start anywhere, and a block of them may end inside a box.
// ROWS loads whole boxes: rows of the next expert fill columns of the accumulator
// that are not stored; a chunk of results that the expert's last row cuts is
// written by ordinary stores, the others by TMA.  In DEPTH the extra rows of an
// expert's last box would be summed: the MMAs of whole 16-row steps behind the end
// are left out, and a warp of each CTA sets the rest of the last step to zero in
// shared memory, in both operands (the rows may hold infinities), before the MMA
// may read it.  Every tensor map describes exactly the caller's array.
//
// Two CTAs of a cluster compute a 256 x (up to 256) tile with 2-SM MMAs: each
// loads its 128 rows of A and half of B's rows and accumulates its 128 rows over
// all columns.  Warp 0 issues TMA (both CTAs, one thread), warp 1 the MMAs (even
// CTA), the others drain TMEM (both CTAs) while the next tile accumulates in the
// other half of it.  Every role walks the same static list of tiles: pair c of C
// takes tiles c, 2C - 1 - c, 2C + c, ... (back and forth, so that a list sorted by
// cost, as DEPTH's experts are by rows, loads the pairs evenly).  Every wait is
// bounded.
#include <cuda_fp16.h>

#include <algorithm>

#include "epilogue.cuh"
#include "gmm_open.h"
#include "ptx.cuh"

namespace hmm {

namespace {

constexpr int OK_ = 64;                  // k per stage: one 128-byte swizzle row of 16-bit elements
constexpr int OA_BYTES = 128 * OK_ * 2;  // this CTA's 128 rows of A
constexpr int OB_BYTES = 128 * OK_ * 2;  // this CTA's half of B's rows, at most 128
constexpr int OSTAGE = OA_BYTES + OB_BYTES;
constexpr int OBUF = 2048;             // staging of one 32 x 32 chunk of 16-bit results
constexpr uint32_t O_TMEM_COLS = 512;  // two accumulators of 256 columns
constexpr int O_SORT_MAX_E = 512;      // experts that DEPTH sorts by rows (E^2 / threads compares)
constexpr int O_LIST_BYTES = 4 * (MAX_E + 4);

template <int KIND>
struct Cfg {
  // ROWS streams weights for few rows: all the stages that fit.  The others have
  // long epilogues (two results, or a mirrored one): eight warps for them.
  static constexpr int STAGES = KIND == OPEN_ROWS ? 6 : 5;
  static constexpr int EPI_WARPS = KIND == OPEN_ROWS ? 4 : 8;
  // DEPTH: one more warp, for the ends of the experts
  static constexpr int THREADS = 32 * (2 + EPI_WARPS + (KIND == OPEN_DEPTH ? 1 : 0));
  static constexpr int SMEM = 1024 + STAGES * OSTAGE + EPI_WARPS * 2 * OBUF + 1024 + O_LIST_BYTES;
  static_assert(SMEM <= 232448, "shared memory per CTA");
};

struct OpenMaps {
  CUtensorMap a, b, out, out2;
  CUtensorMap brows[8];  // ROWS: x in boxes of 16, 32 .. 128 rows
};

struct OpenTile {
  int z;       // expert or matrix
  int m0, n0;  // ROWS: n0 = first row of the block
  int nv, nb;  // ROWS: rows of the block, MMA columns (a multiple of 16); else 256
  int kb;      // K blocks
  int k0, k1;  // DEPTH: the expert's rows
};

// The pair's i-th tile (tiles go back and forth over the pairs).
__device__ __forceinline__ int64_t open_index(int64_t i) {
  const int64_t C = ncluster_x(), c = cluster_id_x();
  return i * C + ((i & 1) ? C - 1 - c : c);
}

// offsets clamped into [0, R]: whatever the caller's offsets hold, every access stays inside.
__device__ __forceinline__ int open_off(const OpenParams& P, int e) {
  return min(max(P.offsets[e], 0), P.R);
}

__device__ __forceinline__ int open_blocks(int rows) { return (rows + 255) >> 8; }

// list: ROWS: blocks of the experts before e (E + 1 entries); DEPTH: experts by
// rows, descending.  All threads of the CTA; ends with a barrier.
template <int KIND>
__device__ void open_list(const OpenParams& P, int* list) {
  if constexpr (KIND == OPEN_ROWS) {
    if (threadIdx.x < 32) {
      const int lane = threadIdx.x;
      int carry = 0;
      if (lane == 0) list[0] = 0;
      for (int base = 0; base < P.Z; base += 32) {
        const int e = base + lane;
        int v = e < P.Z ? open_blocks(max(0, open_off(P, e + 1) - open_off(P, e))) : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int n = __shfl_up_sync(0xffffffffu, v, d);
          if (lane >= d) v += n;
        }
        if (e < P.Z) list[e + 1] = carry + v;
        carry += __shfl_sync(0xffffffffu, v, 31);
      }
    }
  } else if constexpr (KIND == OPEN_DEPTH) {
    if (P.Z > O_SORT_MAX_E) {
      for (int e = threadIdx.x; e < P.Z; e += blockDim.x) list[e] = e;
    } else {
      int* rows = list + O_SORT_MAX_E;
      for (int e = threadIdx.x; e < P.Z; e += blockDim.x)
        rows[e] = max(0, open_off(P, e + 1) - open_off(P, e));
      __syncthreads();
      for (int e = threadIdx.x; e < P.Z; e += blockDim.x) {
        const int re = rows[e];
        int rank = 0;
        for (int f = 0; f < P.Z; ++f) rank += (rows[f] > re || (rows[f] == re && f < e)) ? 1 : 0;
        list[rank] = e;
      }
    }
  }
  __syncthreads();
}

template <int KIND>
__device__ __forceinline__ int64_t open_total(const OpenParams& P, const int* list) {
  if constexpr (KIND == OPEN_ROWS) return static_cast<int64_t>(list[P.Z]) * P.mt;
  return static_cast<int64_t>(P.Z) * P.tiles;
}

template <int KIND>
__device__ __forceinline__ void open_tile(const OpenParams& P, const int* list, int64_t u,
                                          OpenTile& t) {
  if constexpr (KIND == OPEN_ROWS) {
    const int blk = static_cast<int>(u / P.mt);
    t.m0 = static_cast<int>(u - static_cast<int64_t>(blk) * P.mt) * 256;
    int lo = 0, hi = P.Z - 1;  // the largest e with list[e] <= blk
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (list[mid] <= blk)
        lo = mid;
      else
        hi = mid - 1;
    }
    const int o = open_off(P, lo), rows = open_off(P, lo + 1) - o;
    const int nblk = open_blocks(rows), j = blk - list[lo];
    t.z = lo;
    t.nb = ((rows + nblk - 1) / nblk + 15) & ~15;
    t.n0 = o + j * t.nb;
    t.nv = min(t.nb, rows - j * t.nb);
    t.kb = P.kb;
  } else {
    const int i = static_cast<int>(u / P.tiles);
    int r = static_cast<int>(u - static_cast<int64_t>(i) * P.tiles);
    t.nv = t.nb = 256;
    if (P.sym) {  // tiles on and right of the diagonal, row by row
      int mi = 0;
      for (int w = P.mt; r >= w; --w) {
        r -= w;
        ++mi;
      }
      t.m0 = mi * 256;
      t.n0 = (mi + r) * 256;
    } else {
      t.m0 = r / P.nt * 256;
      t.n0 = r % P.nt * 256;
    }
    if constexpr (KIND == OPEN_DEPTH) {
      t.z = list[i];
      t.k0 = open_off(P, t.z);
      t.k1 = max(t.k0, open_off(P, t.z + 1));
      t.kb = (t.k1 - t.k0 + OK_ - 1) / OK_;
    } else {
      t.z = i;
      t.kb = P.kb;
    }
  }
}

// Rows of the tile's last K block (DEPTH) if it ends inside a 16-row step, else 0.
__device__ __forceinline__ int open_tail(const OpenTile& t) {
  const int v = (t.k1 - t.k0) & (OK_ - 1);
  return (v & 15) ? v : 0;
}

__device__ __forceinline__ uint32_t pack16(bool f16, float lo, float hi) {
  if (f16) {
    __half2 p = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&p);
  }
  return pack_bf16(lo, hi);
}

// A warp's 32 x 32 chunk (lane = m, register = n) to staging rows of n, m
// contiguous (64 bytes a row, plain): neighbouring lanes swap halves, so that each
// store is a pair of m and a warp's store covers two whole rows, all banks once.
__device__ __forceinline__ void stage_t(uint8_t* sb, int lane, bool f16, const float (&v)[32]) {
  const bool odd = lane & 1;
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const float send = odd ? v[i] : v[i + 1];
    const float got = __shfl_xor_sync(0xffffffffu, send, 1);
    // even lane: row i, columns (lane, lane + 1); odd: row i + 1, columns (lane - 1, lane)
    const uint32_t p = odd ? pack16(f16, got, v[i + 1]) : pack16(f16, v[i], got);
    *reinterpret_cast<uint32_t*>(sb + (i + (odd ? 1 : 0)) * 64 + (lane >> 1) * 4) = p;
  }
}

// The same chunk as rows of m, n contiguous: lane = row, its 16-byte unit u at
// u ^ ((row >> 1) & 3) (the 64-byte swizzle of the map).
__device__ __forceinline__ void stage_d(uint8_t* sb, int lane, bool f16, const float (&v)[32]) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    uint4 q;
    q.x = pack16(f16, v[8 * u], v[8 * u + 1]);
    q.y = pack16(f16, v[8 * u + 2], v[8 * u + 3]);
    q.z = pack16(f16, v[8 * u + 4], v[8 * u + 5]);
    q.w = pack16(f16, v[8 * u + 6], v[8 * u + 7]);
    *reinterpret_cast<uint4*>(sb + lane * 64 + 16 * (u ^ ((lane >> 1) & 3))) = q;
  }
}

__device__ __forceinline__ float half_round(float v) { return __half2float(__float2half_rn(v)); }

// 32 consecutive fp16 values (16-byte aligned)
__device__ __forceinline__ void load32h(const __half* p, float (&v)[32]) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const uint4 q = *reinterpret_cast<const uint4*>(p + 8 * u);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
      v[8 * u + 2 * j] = f.x;
      v[8 * u + 2 * j + 1] = f.y;
    }
  }
}

template <int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Cfg<KIND>::THREADS, 1)
    open_kernel(const __grid_constant__ OpenParams P, const __grid_constant__ OpenMaps maps) {
  using C = Cfg<KIND>;
  constexpr int ST = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* stages = smem;
  uint8_t* obufs = smem + ST * OSTAGE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(obufs + C::EPI_WARPS * 2 * OBUF);
  uint64_t* full = bars;         // used in the even CTA: bytes of both
  uint64_t* empty = full + ST;   // both CTAs
  uint64_t* tfull = empty + ST;  // both CTAs
  uint64_t* tempty = tfull + 2;  // even CTA: every epilogue warp of both
  uint64_t* mma_done = tempty + 2;
  // DEPTH, per slot: the loads of a block that has to be cut have landed (this CTA's
  // own), and it is cut (even CTA: one arrival per CTA)
  uint64_t* landed = mma_done + 1;
  uint64_t* cut = landed + ST;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(cut + ST);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  uint32_t* s_issued = s_tmem + 2;
  uint32_t* s_sbytes = s_tmem + 3;   // [ST] bytes of this CTA's last load per slot
  uint32_t* s_peer = s_sbytes + ST;  // [2 + ST]
  int* list = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + 1024);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&landed[s], 1);
      mbar_init(&cut[s], 2);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * C::EPI_WARPS);
    }
    mbar_init(mma_done, 1);
    *s_abort = 0;
    *s_issued = 0;
    for (int i = 0; i < ST; ++i) s_sbytes[i] = OSTAGE;
    for (int i = 0; i < 2 + ST; ++i) s_peer[i] = 0;
    fence_mbar_init();
  }
  cluster_sync_all();  // the peer's barriers are initialised before any remote arrive
  if (warp == 1) {
    tmem_alloc_pair(s_tmem, O_TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *s_tmem;
  grid_dep_wait();  // from here on memory that earlier kernels write
  const WaitCtl wc{s_abort, P.status, P.budget_ns};
  open_list<KIND>(P, list);
  const int64_t total = open_total<KIND>(P, list);

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------- TMA producer
      tma_prefetch_desc(&maps.a);
      tma_prefetch_desc(&maps.out);
      uint32_t stage = 0, sphase = 0, issued = 0;
      uint32_t landed_phase = 0, landed_used = 0;  // a bit per slot
      bool ok = true;
      for (int64_t i = 0; ok; ++i) {
        const int64_t u = open_index(i);
        if (u >= total) break;
        OpenTile t;
        open_tile<KIND>(P, list, u, t);
        const int ma = t.m0 + 128 * static_cast<int>(rank);
        // B: this CTA's half of the columns, in boxes of a multiple of 16 rows
        const int half = t.nb >> 1;
        const int nbase = t.n0 + half * static_cast<int>(rank);
        const int box = (half + 15) >> 4;
        const uint32_t b_bytes = KIND == OPEN_ROWS ? box * 16 * OK_ * 2 : OB_BYTES;
        const CUtensorMap* bm = KIND == OPEN_ROWS ? &maps.brows[box - 1] : &maps.b;
        for (int kb = 0; kb < t.kb; ++kb) {
          if (!mbar_wait(&empty[stage], sphase ^ 1u, wc)) {
            ok = false;
            break;
          }
          uint8_t* sA = stages + stage * OSTAGE;
          uint8_t* sB = sA + OA_BYTES;
          const int k = kb * OK_;
          if (KIND == OPEN_DEPTH && kb == t.kb - 1 && open_tail(t) != 0) {
            // counted on this CTA's own barrier; `full` completes at once
            if (leader) mbar_arrive(&full[stage]);
            s_sbytes[stage] = 0;
            mbar_arrive_expect_tx(&landed[stage], OSTAGE);
            landed_used |= 1u << stage;
            landed_phase ^= 1u << stage;
            tma_load_3d(sA, &maps.a, &landed[stage], ma, t.k0 + k, 0);
            tma_load_3d(sA + OA_BYTES / 2, &maps.a, &landed[stage], ma + 64, t.k0 + k, 0);
            tma_load_3d(sB, bm, &landed[stage], nbase, t.k0 + k, 0);
            tma_load_3d(sB + OB_BYTES / 2, bm, &landed[stage], nbase + 64, t.k0 + k, 0);
          } else {
            if (leader) mbar_arrive_expect_tx(&full[stage], 2 * (OA_BYTES + b_bytes));
            s_sbytes[stage] = OA_BYTES + b_bytes;
            const uint32_t bar = mapa_shared(smem_u32(&full[stage]), 0);
            // coordinates of an MN-major box: (m or n, c1, c2)
            const int c1 = KIND == OPEN_DEPTH ? t.k0 + k : k, c2 = KIND == OPEN_DEPTH ? 0 : t.z;
            if (KIND == OPEN_DEPTH || P.a_mn) {
              tma_load_3d_pair(sA, &maps.a, bar, ma, c1, c2);
              tma_load_3d_pair(sA + OA_BYTES / 2, &maps.a, bar, ma + 64, c1, c2);
            } else {
              tma_load_3d_pair(sA, &maps.a, bar, k, ma, t.z);
            }
            if (KIND == OPEN_DEPTH || (KIND == OPEN_STACK && P.b_mn)) {
              tma_load_3d_pair(sB, bm, bar, nbase, c1, c2);
              tma_load_3d_pair(sB + OB_BYTES / 2, bm, bar, nbase + 64, c1, c2);
            } else {
              tma_load_3d_pair(sB, bm, bar, k, nbase, KIND == OPEN_ROWS ? 0 : t.z);
            }
          }
          ++issued;
          if (++stage == ST) {
            stage = 0;
            sphase ^= 1u;
          }
        }
      }
      // after an abort: this CTA's own copies (the others are drained at teardown)
      if (KIND == OPEN_DEPTH && !ok)
        for (int s = 0; s < ST; ++s)
          if (landed_used >> s & 1u)
            drain_wait(&landed[s], (landed_phase >> s & 1u) ^ 1u, P.budget_ns);
      *s_issued = issued;
      grid_dep_launch();  // this CTA is in its last tile
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ------------------------------------------------------------ MMA issue
      // 16 deep per MMA: K-major 32 bytes on inside the swizzled row, MN-major
      // 16 rows of 128 bytes on (two 64-wide chunks half a tile apart)
      const bool a_mn = KIND == OPEN_DEPTH || P.a_mn;
      const bool b_mn = KIND == OPEN_DEPTH || (KIND == OPEN_STACK && P.b_mn);
      const uint32_t a_step = a_mn ? 2048 : 32, b_step = b_mn ? 2048 : 32;
      const uint32_t a_lbo = a_mn ? OA_BYTES / 2 : 16, b_lbo = b_mn ? OB_BYTES / 2 : 16;
      uint32_t stage = 0, sphase = 0, acc = 0, acc_phase = 0, cut_phase = 0;
      bool ok = true;
      for (int64_t i = 0; ok; ++i) {
        const int64_t u = open_index(i);
        if (u >= total) break;
        OpenTile t;
        open_tile<KIND>(P, list, u, t);
        if (t.kb == 0) continue;
        const uint32_t idesc = P.idesc | (static_cast<uint32_t>(t.nb >> 3) << 17);
        if (!mbar_wait(&tempty[acc], acc_phase ^ 1u, wc)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * 256;
        for (int kb = 0; kb < t.kb; ++kb) {
          if (!mbar_wait(&full[stage], sphase, wc)) {
            ok = false;
            break;
          }
          int steps = OK_ / 16;
          if (KIND == OPEN_DEPTH && kb == t.kb - 1) {
            steps = (t.k1 - t.k0 - kb * OK_ + 15) >> 4;
            if (open_tail(t) != 0) {
              if (!mbar_wait<true>(&cut[stage], cut_phase >> stage & 1u, wc)) {
                ok = false;
                break;
              }
              cut_phase ^= 1u << stage;
            }
          }
          tc_fence_after();
          const uint32_t a_base = smem_u32(stages + stage * OSTAGE);
          const uint32_t b_base = a_base + OA_BYTES;
#pragma unroll
          for (int kk = 0; kk < OK_ / 16; ++kk) {
            if (KIND == OPEN_DEPTH && kk >= steps) break;
            const uint64_t ad = smem_desc(a_base + kk * a_step, a_lbo, 1024, LAYOUT_SW128);
            const uint64_t bd = smem_desc(b_base + kk * b_step, b_lbo, 1024, LAYOUT_SW128);
            umma_bf16_pair(d_tmem, ad, bd, idesc, (kb == 0 && kk == 0) ? 0u : 1u);
          }
          umma_commit_pair(&empty[stage], 0x3);
          if (++stage == ST) {
            stage = 0;
            sphase ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit_pair(&tfull[acc], 0x3);
        acc ^= 1u;
        if (acc == 0) acc_phase ^= 1u;
      }
      umma_commit_pair(mma_done, 0x1);
      drain_wait(mma_done, 0, P.budget_ns);
    }
  } else if (KIND == OPEN_DEPTH && warp == 2 + C::EPI_WARPS) {
    // ------------------------------------------------- the ends of the experts
    // Rows v .. of the last step of an expert's last block, of both operands and
    // this CTA: a row is 128 bytes in each of the four 64-wide chunks, swizzled
    // inside itself.
    uint32_t slot = 0, landed_phase = 0;
    for (int64_t i = 0;; ++i) {
      const int64_t u = open_index(i);
      if (u >= total) break;
      OpenTile t;
      open_tile<KIND>(P, list, u, t);
      if (t.kb == 0) continue;
      const uint32_t last = (slot + t.kb - 1) % ST;
      slot = (slot + t.kb) % ST;
      const int v = open_tail(t);
      if (v == 0) continue;
      bool got = false;
      if (lane == 0) got = mbar_wait(&landed[last], landed_phase >> last & 1u, wc);
      __syncwarp();
      if (!__shfl_sync(0xffffffffu, got, 0)) break;
      landed_phase ^= 1u << last;
      const int rows = 16 - (v & 15);
      for (int j = lane; j < 4 * 8 * rows; j += 32) {
        const int chunk = j & 3, unit = j >> 2 & 7, row = v + (j >> 5);
        *reinterpret_cast<uint4*>(stages + last * OSTAGE + chunk * (OA_BYTES / 2) + row * 128 +
                                  unit * 16) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&cut[last]), 0));
    }
  } else {
    // ------------------------------------------------------------- epilogue
    const int q4 = warp & 3;
    // chunks of 32 columns: all of them, or every other one of the warp's lane quarter
    constexpr int SHARE = C::EPI_WARPS / 4;
    const int first = SHARE == 1 ? 0 : (warp - 2) >> 2;
    uint8_t* obuf = obufs + (warp - 2) * 2 * OBUF;
    const bool f16 = P.out_f16 != 0;
    uint32_t ck = 0;  // buffers this warp has stored from
    uint32_t acc = 0, acc_phase = 0;
    const uint32_t tempty_cl[2] = {mapa_shared(smem_u32(&tempty[0]), 0),
                                   mapa_shared(smem_u32(&tempty[1]), 0)};
    // the next staging buffer, its earlier store read out
    const auto take_buf = [&]() {
      if (lane == 0) bulk_wait_group_read<1>();
      __syncwarp();
      return obuf + (ck++ & 1u) * OBUF;
    };
    const auto send = [&](const CUtensorMap* m, const uint8_t* sb, int c0, int c1, int c2) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_3d(m, sb, c0, c1, c2);
        bulk_commit_group();
      }
    };
    if constexpr (KIND == OPEN_ROWS) {
      // rows of no expert (in front of the first, behind the last) are zero
      const int r0 = open_off(P, 0), r1 = max(r0, open_off(P, P.Z));
      const int64_t per = P.M / 8, n = (static_cast<int64_t>(r0) + P.R - r1) * per;
      const int64_t step = static_cast<int64_t>(gridDim.x) * (32 * C::EPI_WARPS);
      for (int64_t i = static_cast<int64_t>(blockIdx.x) * (32 * C::EPI_WARPS) +
                       (threadIdx.x - 64);
           i < n; i += step) {
        int64_t r = i / per;
        const int64_t c = i - r * per;
        if (r >= r0) r += r1 - r0;
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(P.out) + r * P.M + c * 8) =
            make_uint4(0, 0, 0, 0);
      }
    }
    for (int64_t i = 0;; ++i) {
      const int64_t u = open_index(i);
      if (u >= total) break;
      OpenTile t;
      open_tile<KIND>(P, list, u, t);
      const int mw = t.m0 + 128 * static_cast<int>(rank) + q4 * 32;  // this warp's rows of m
      if constexpr (KIND == OPEN_DEPTH) {
        if (t.kb == 0) {  // an expert with no rows: zeros
          float z[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) z[j] = 0.f;
          if (mw < P.M)
            for (int c = first; c < 8 && t.n0 + 32 * c < P.N; c += SHARE) {
              uint8_t* sb = take_buf();
              stage_d(sb, lane, f16, z);
              send(&maps.out, sb, t.n0 + 32 * c, mw, t.z);
            }
          continue;
        }
      }
      bool got = false;
      if (lane == 0) got = mbar_wait(&tfull[acc], acc_phase, wc);
      __syncwarp();
      if (!__shfl_sync(0xffffffffu, got, 0)) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q4 * 32) << 16) + acc * 256;
      // chunks that hold results
      const int nch = mw >= P.M ? 0
                      : KIND == OPEN_ROWS
                          ? (t.nv + 31) >> 5
                          : min(8, (P.N - t.n0 + 31) >> 5);
      for (int c = first; c < nch; c += SHARE) {
        uint32_t r[32];
        tmem_ld32(taddr + c * 32, r);
        tmem_ld_wait_for(r);
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
        if constexpr (KIND == OPEN_ROWS) {
          const int rows = min(32, t.nv - 32 * c);
          uint8_t* sb = take_buf();
          stage_t(sb, lane, f16, v);
          if (rows == 32) {
            send(&maps.out, sb, mw, t.n0 + 32 * c, 0);
          } else {
            // the expert's last rows: eight rows of 64 bytes at a time
            __syncwarp();
            const int col = mw + (lane & 3) * 8;
            for (int j = lane >> 2; j < rows; j += 8)
              if (col < P.M)
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(P.out) +
                                          static_cast<int64_t>(t.n0 + 32 * c + j) * P.M + col) =
                    *reinterpret_cast<const uint4*>(sb + j * 64 + (lane & 3) * 16);
            __syncwarp();
          }
        } else if constexpr (KIND == OPEN_DEPTH) {
          uint8_t* sb = take_buf();
          stage_d(sb, lane, f16, v);
          send(&maps.out, sb, t.n0 + 32 * c, mw, t.z);
        } else {
          const int n = t.n0 + 32 * c, m = mw + lane;
          if (P.epi == OPEN_EPI_GRAM || P.epi == OPEN_EPI_POLY) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] *= P.alpha;
            if (P.epi == OPEN_EPI_POLY) {
              float s[32];
#pragma unroll
              for (int j = 0; j < 32; ++j) s[j] = 0.f;
              if (m < P.M) {
                // (rows are padded to 8 elements: what lies behind N is not stored)
                const __half* src = P.in_hi + (static_cast<int64_t>(t.z) * P.M + m) * P.ld_in + n;
                if (n + 32 <= P.ld_in) {
                  load32h(src, s);
                } else {
#pragma unroll
                  for (int j = 0; j < 32; ++j)
                    if (n + j < P.ld_in) s[j] = __half2float(src[j]);
                }
              }
#pragma unroll
              for (int j = 0; j < 32; ++j)
                v[j] = fmaf(P.beta, s[j], v[j]) + (m == n + j ? P.gamma : 0.f);
            }
            uint8_t* sb = take_buf();
            stage_d(sb, lane, true, v);
            send(&maps.out, sb, n, mw, t.z);
            if (t.n0 > t.m0) {  // the mirrored chunk (the results are symmetric)
              sb = take_buf();
              stage_t(sb, lane, true, v);
              send(&maps.out2, sb, mw, n, t.z);
            }
          } else {
            // X <- alpha acc + beta hi + gamma lo
            float h[32], l[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) h[j] = l[j] = 0.f;
            if (m < P.M) {
              const int64_t at = (static_cast<int64_t>(t.z) * P.M + m) * P.ld_in + n;
              if (n + 32 <= P.ld_in) {
                load32h(P.in_hi + at, h);
                load32h(P.in_lo + at, l);
              } else {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (n + j < P.ld_in) {
                    h[j] = __half2float(P.in_hi[at + j]);
                    l[j] = __half2float(P.in_lo[at + j]);
                  }
              }
            }
#pragma unroll
            for (int j = 0; j < 32; ++j)
              v[j] = fmaf(P.gamma, l[j], fmaf(P.beta, h[j], P.alpha * v[j]));
            if (P.epi == OPEN_EPI_UPDATE) {
#pragma unroll
              for (int j = 0; j < 32; ++j) l[j] = v[j] - half_round(v[j]);
              uint8_t* sb = take_buf();
              stage_d(sb, lane, true, v);
              send(&maps.out, sb, n, mw, t.z);
              sb = take_buf();
              stage_d(sb, lane, true, l);
              send(&maps.out2, sb, n, mw, t.z);
            } else if (!P.plain_out) {
              uint8_t* sb = take_buf();
              stage_d(sb, lane, f16, v);
              send(&maps.out, sb, n, mw, t.z);
            } else if (m < P.M) {
              // rows of the result that no tensor map can describe (N no multiple of 8)
              uint16_t* dst =
                  static_cast<uint16_t*>(P.out) + (static_cast<int64_t>(t.z) * P.M + m) * P.N + n;
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (n + j < P.N) dst[j] = static_cast<uint16_t>(pack16(f16, v[j], 0.f) & 0xFFFFu);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (leader)
          mbar_arrive(&tempty[acc]);
        else
          mbar_arrive_peer(tempty_cl[acc]);
      }
      acc ^= 1u;
      if (acc == 0) acc_phase ^= 1u;
    }
    if (lane == 0) bulk_wait_group<0>();  // every store has landed
  }

  tc_fence_before();
  __syncthreads();
  pair_teardown<ST>(leader, *s_issued, *s_abort, s_peer, s_sbytes, full, P.budget_ns);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, O_TMEM_COLS);
  }
}

// ------------------------------------------------------------------ host side
// A map of rank 3: dimensions d0 (contiguous), d1, d2 with strides in elements.
int encode3(const GemmEnv& env, CUtensorMap* m, bool f16, const void* base, int64_t d0, int64_t d1,
            int64_t d2, int64_t s1, int64_t s2, int b0, int b1, CUtensorMapSwizzle sw) {
  const cuuint64_t gd[3] = {static_cast<cuuint64_t>(d0), static_cast<cuuint64_t>(d1),
                            static_cast<cuuint64_t>(d2)};
  const cuuint64_t gs[2] = {static_cast<cuuint64_t>(s1) * 2, static_cast<cuuint64_t>(s2) * 2};
  const cuuint32_t bx[3] = {static_cast<cuuint32_t>(b0), static_cast<cuuint32_t>(b1), 1};
  const cuuint32_t es[3] = {1, 1, 1};
  const CUresult r = env.encode(
      m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
      const_cast<void*>(base), gd, gs, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
      sw == CU_TENSOR_MAP_SWIZZLE_128B ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                       : CU_TENSOR_MAP_L2_PROMOTION_NONE,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? HMM_OK : HMM_ERR_CUDA;
}

// An operand [batch][rows][cols] as loaded: K-major (cols = k): boxes of 64 x
// `box` rows; MN-major (rows = k): boxes of 64 columns x 64 rows.
int encode_operand(const GemmEnv& env, CUtensorMap* m, bool f16, const OpenOperand& o, int box) {
  return encode3(env, m, f16, o.ptr, o.cols, o.rows, o.batch, o.ld, o.stride, 64, box,
                 CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int KIND>
int launch_open(const GemmEnv& env, const OpenParams& P, const OpenMaps& maps, int64_t tiles) {
  using C = Cfg<KIND>;
  if (tiles <= 0) return HMM_OK;
  if (cudaFuncSetAttribute(open_kernel<KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           C::SMEM) != cudaSuccess)
    return HMM_ERR_CUDA;
  const int clusters = static_cast<int>(std::min<int64_t>(env.num_sms / 2, tiles));
  return launch_kernel(open_kernel<KIND>, 2 * clusters, C::THREADS, C::SMEM, env.stream, env.pdl,
                       1, P, maps) == cudaSuccess
             ? HMM_OK
             : HMM_ERR_CUDA;
}

uint32_t open_idesc(bool f16, bool a_mn, bool b_mn) {
  // (N is added per tile)
  uint32_t d = idesc_bf16_f32(256, 0, a_mn ? 1 : 0, b_mn ? 1 : 0);
  if (f16) d &= ~((1u << 7) | (1u << 10));  // operand formats: fp16
  return d;
}

void open_common(const GemmEnv& env, OpenParams* P) {
  P->status = env.status;
  P->budget_ns = env.budget_ns;
}

}  // namespace

int launch_open_rows(const GemmEnv& env, bool f16, const OpenOperand& w, bool w_mn, const void* x,
                     int64_t ld_x, int64_t R, int64_t K, int64_t M, int64_t E,
                     const int32_t* offsets, void* out) {
  OpenParams P{};
  OpenMaps maps;
  open_common(env, &P);
  P.idesc = open_idesc(f16, w_mn, false);
  P.a_mn = w_mn;
  P.M = static_cast<int>(M);
  P.Z = static_cast<int>(E);
  P.R = static_cast<int>(R);
  P.kb = static_cast<int>((K + OK_ - 1) / OK_);
  P.mt = static_cast<int>((M + 255) / 256);
  P.offsets = offsets;
  P.out = out;
  P.out_f16 = f16;
  int rc = encode_operand(env, &maps.a, f16, w, w_mn ? 64 : 128);
  const OpenOperand xo{x, R, K, 1, ld_x, R * ld_x};
  for (int i = 0; i < 8; ++i) rc |= encode_operand(env, &maps.brows[i], f16, xo, 16 * (i + 1));
  rc |= encode3(env, &maps.out, f16, out, M, R, 1, M, R * M, 32, 32, CU_TENSOR_MAP_SWIZZLE_NONE);
  if (rc != HMM_OK) return HMM_ERR_CUDA;
  // at most a partly filled block per expert beside the full ones
  const int64_t blocks = std::min<int64_t>(R, R / 256 + E);
  return launch_open<OPEN_ROWS>(env, P, maps, blocks * P.mt);
}

int launch_open_depth(const GemmEnv& env, bool f16, const void* a, int64_t ld_a, int64_t M,
                      const void* b, int64_t ld_b, int64_t N, int64_t R, int64_t E,
                      const int32_t* offsets, void* out) {
  OpenParams P{};
  OpenMaps maps;
  open_common(env, &P);
  P.idesc = open_idesc(f16, true, true);
  P.a_mn = P.b_mn = 1;
  P.M = static_cast<int>(M);
  P.N = static_cast<int>(N);
  P.Z = static_cast<int>(E);
  P.R = static_cast<int>(R);
  P.mt = static_cast<int>((M + 255) / 256);
  P.nt = static_cast<int>((N + 255) / 256);
  P.tiles = P.mt * P.nt;
  P.offsets = offsets;
  P.out = out;
  P.out_f16 = f16;
  int rc = encode_operand(env, &maps.a, f16, OpenOperand{a, R, M, 1, ld_a, R * ld_a}, OK_);
  rc |= encode_operand(env, &maps.b, f16, OpenOperand{b, R, N, 1, ld_b, R * ld_b}, OK_);
  rc |= encode3(env, &maps.out, f16, out, N, M, E, N, M * N, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  if (rc != HMM_OK) return HMM_ERR_CUDA;
  return launch_open<OPEN_DEPTH>(env, P, maps, E * static_cast<int64_t>(P.tiles));
}

int launch_open_stack(const GemmEnv& env, const OpenStack& s) {
  OpenParams P{};
  OpenMaps maps;
  open_common(env, &P);
  P.idesc = open_idesc(true, s.a_mn, s.b_mn);
  P.a_mn = s.a_mn;
  P.b_mn = s.b_mn;
  P.M = static_cast<int>(s.M);
  P.N = static_cast<int>(s.N);
  P.Z = static_cast<int>(s.a.batch);
  P.kb = static_cast<int>((s.K + OK_ - 1) / OK_);
  P.mt = static_cast<int>((s.M + 255) / 256);
  P.nt = static_cast<int>((s.N + 255) / 256);
  P.epi = s.epi;
  P.sym = s.epi == OPEN_EPI_GRAM || s.epi == OPEN_EPI_POLY;
  P.tiles = P.sym ? P.mt * (P.mt + 1) / 2 : P.mt * P.nt;
  P.alpha = s.alpha;
  P.beta = s.beta;
  P.gamma = s.gamma;
  P.in_hi = static_cast<const __half*>(s.in_hi);
  P.in_lo = static_cast<const __half*>(s.in_lo);
  P.ld_in = s.ld_in;
  P.out = s.out;
  P.out_f16 = s.out_f16;
  int rc = encode_operand(env, &maps.a, true, s.a, s.a_mn ? 64 : 128);
  rc |= encode_operand(env, &maps.b, true, s.b, s.b_mn ? 64 : 128);
  const int64_t Z = s.a.batch;
  // results: rows of ld_out elements; the mirrored or low ones beside them
  const bool last = s.epi == OPEN_EPI_LAST;
  P.plain_out = last && (s.ld_out % 8 != 0 || (reinterpret_cast<uintptr_t>(s.out) & 15u) != 0);
  const bool f16 = !last || s.out_f16;
  if (P.plain_out)
    maps.out = maps.a;  // (prefetched, not used)
  else
    rc |= encode3(env, &maps.out, f16, s.out, s.N, s.M, Z, s.ld_out, s.M * s.ld_out, 32, 32,
                  CU_TENSOR_MAP_SWIZZLE_64B);
  if (P.sym)
    rc |= encode3(env, &maps.out2, true, s.out, s.M, s.N, Z, s.ld_out, s.M * s.ld_out, 32, 32,
                  CU_TENSOR_MAP_SWIZZLE_NONE);
  else if (s.epi == OPEN_EPI_UPDATE)
    rc |= encode3(env, &maps.out2, true, s.out_lo, s.N, s.M, Z, s.ld_out, s.M * s.ld_out, 32, 32,
                  CU_TENSOR_MAP_SWIZZLE_64B);
  if (rc != HMM_OK) return HMM_ERR_CUDA;
  return launch_open<OPEN_STACK>(env, P, maps, Z * static_cast<int64_t>(P.tiles));
}

}  // namespace hmm
