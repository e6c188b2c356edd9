// The block-wise kernel of scored attention (TMA + tcgen05 + TMEM, sm_103a),
// shared by its two sources of tiles:
//   FormatSource  the listed outer tiles of the query tiles of a mask format
//                 (format_source.cuh, stof_mha_fwd_score);
//   CacheSource   the tiles of the requests' K/V caches (tree_attn.cu,
//                 stof_tree_attn_fwd).
// A segment is a run of K/V tiles of BN keys for one tile of 128 query rows;
// its online softmax gives the rows' O, or a partial O with the rows' max and
// sum where other workers hold the rest.
//
// A CTA runs two workers g = 0, 1 that share nothing but the SM's units: each
// has segments of its own, one after the other, a Q tile and K and V rings
// in shared memory, S, P and O in TMEM, and its own warps:
//   warp g          producer (one thread): takes segments, copies Q, K, V (TMA);
//   warp 2 + g      score MMAs S = Q K^T and PV MMAs O += P V (P read from
//                   TMEM), the scores of the next tile before the PV of this;
//   warps 4 + 4 g ..  softmax, a thread per query row.
// A segment's tiles go from the last to the first: the keys nearest to the
// rows come first, so that with distance the running max is settled by the
// first tile.
// While one worker loads Q, starts or finishes a segment or waits for a tile,
// the other one's tiles go on, so that short segments (a few tiles, as
// packed documents and short caches give) cost little more than their tiles.
// No unit is full (profiles: issue slots 48 to 57%, tensor pipe 25 to 63%): the
// time is that of a tile's chain of steps, and every role's instructions and
// registers count.  Both workers run the same code, since the instruction
// cache's 32 KB hold the softmax's straight-line code for a tile and the other
// warps' loops.  (With K, V, score and PV warps that served both workers in turn the loops
// took 32 KB, and 92% of the instruction fetch bandwidth behind the cache:
// 723 us instead of 485 us for 8192 causal tokens, 32 heads of 128.)  The MMA
// branch has 56 registers: code for tiles with V rows to clear, spilling 16 to
// 90 bytes there, cost 2 to 8% where no tile took it.
// REP > 1 (few query rows): Q's rows are in the tile REP times, 128 / REP rows
// apart, and each copy's softmax threads take one REP-th of the tile's keys,
// their P being 0 in the other columns: a tile then costs a thread BN / REP
// scores instead of BN, in a fraction of the code.  The copies' partial rows are
// merged at the segment's end through shared memory (through a scratch in
// global memory by all threads, a call of 32 rows took 3 us longer, one of a
// few rows 0.2 to 1 us less).  7 rows per K/V head, 32 requests, d = 64: 26
// to 30 us from run to run, with a thread a row 50.
// A softmax warp whose 32 query rows are all past the tile's last one only
// keeps the barriers' step.
// BN is 128 for d = 64 and 64 for d = 128: S, P and O of both workers then fit
// the 512 TMEM columns, and a ring stage is 16 KB.  TMEM columns: S_g [BN g,
// +BN), P_g [2 BN + BN / 2 g, +BN / 2), O_g [512 - 2 d + d g, +d).
// Every wait is bounded; on timeout the CTA raises STOF_DEVERR_PIPE_TIMEOUT
// (in the call's error word, where it has one, and in what the source keeps),
// drains its copies and MMAs, frees TMEM and exits.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <type_traits>

#include "internal.h"
#include "score_tile.cuh"
#include "sm100_ptx.cuh"

namespace stof {
namespace scored {

using namespace ptx;
using namespace bw;

// What becomes of the products: MODE_PLAIN scale > 0 only; MODE_CAP a cap of
// at most kMaxCapOnly only; MODE_DISTANCE anything.
constexpr int MODE_PLAIN = 0, MODE_CAP = 1, MODE_DISTANCE = 2;
// 60 log2 e = 87: sums of 2^31 keys of 2^87 times |V| below 2^8 stay in fp32,
// and with every score at -60 a V above 2^-39 still does.
constexpr float kMaxCapOnly = 60.f;

// Sum of a row's P in a tile up to which its reference may be left as it is:
// P itself stays within the type.
template <bool BF16>
constexpr float kSlack = BF16 ? 0x1p20f : 0x1p15f;

struct CommonParams {
  ScoreConst k;
  const float* slopes;  // [H] or null
  void* o;
  int64_t* err;         // or null
  int H, group;         // query heads; query heads per K/V head
};

// One run of K/V tiles for one tile of query rows; `item` is the source's own.
template <class ITEM>
struct Segment {
  int q_plane, q_row;   // box of the Q map
  int kv_plane;
  int n;                // tiles
  ITEM item;
};

// Tile width and ring depths (per worker): 16 KB a stage.  K tiles leave
// early (their MMA comes first), V tiles a softmax later.
// Copies of Q's rows (REP > 1) are merged through what a third V stage takes.
template <int D, int REP = 1>
struct Shape {
  static constexpr int BN = D == 128 ? 64 : 128;
  static constexpr int K = 3, V = D == 128 || REP > 1 ? 2 : 3;
  static constexpr int STAGE = BN * D * 2;
  static constexpr int ATOM = BN * 128;  // bytes of a 64-column swizzle atom of a K or V tile
};

// A worker's producer takes its segments from the source and hands them to
// the worker's other warps through a ring in shared memory.
constexpr int kRing = 4;     // segments in flight
constexpr int kReaders = 5;  // the MMA warp, four softmax warps
enum class Next { segment, none, lost };  // lost: a wait ran out

// What one worker has in shared memory.
template <class SRC, int D, int REP>
struct Worker {
  uint64_t q_full, q_done;  // Q is in place; the segment's score MMAs are done
  uint64_t k_full[Shape<D, REP>::K], k_free[Shape<D, REP>::K], v_full[Shape<D, REP>::V], v_free[Shape<D, REP>::V];
  uint64_t s_full, s_free, p_full, pv_done, merge, drain;
  uint64_t ring_full[kRing], ring_free[kRing];
  Segment<typename SRC::Item> ring[kRing];  // n < 0: no more segments
  // First keys of the K tiles, for the distance.  The K tile 8 later is copied
  // once the score MMA 5 later is done, and so the softmax 4 later has begun.
  int key[8];
};

template <class SRC, int D, int REP>
struct alignas(1024) Smem {
  using Sh = Shape<D, REP>;
  uint8_t q[2][kBM * D * 2];
  uint8_t k[2][Sh::K][Sh::STAGE];
  uint8_t v[2][Sh::V][Sh::STAGE];
  // REP > 1: 32 columns of O of the copies but the first, and their (max, sum)
  float4 merge[2][REP > 1 ? (REP - 1) * (kBM / REP) * 8 : 1];
  float2 merge_stats[2][REP > 1 ? (REP - 1) * (kBM / REP) : 1];
  Worker<SRC, D, REP> w[2];
  uint32_t tmem_base;
  int abort_flag;
  typename SRC::Shared src;
};

// ---- a split item (SRC::kSplit): its parts' rows are merged through the
// shared memory of the cluster's CTAs.
// Address in CTA `rank` of the cluster of what is at `addr` in this one.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
  uint32_t x;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(x) : "r"(addr), "r"(rank));
  return x;
}
// (LOCAL: of this CTA, `rank` is not read)
template <bool LOCAL>
__device__ __forceinline__ float4 cluster_ld4(uint32_t addr, uint32_t rank) {
  float4 x;
  if constexpr (LOCAL)
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(addr));
  else
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                 : "r"(cluster_addr(addr, rank)));
  return x;
}
template <bool LOCAL>
__device__ __forceinline__ float2 cluster_ld2(uint32_t addr, uint32_t rank) {
  float2 x;
  if constexpr (LOCAL)
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(x.x), "=f"(x.y) : "r"(addr));
  else
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(x.x), "=f"(x.y) : "r"(cluster_addr(addr, rank)));
  return x;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t x;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(x));
  return x;
}
// All threads of the cluster's CTAs; every one of them gets here, its waits being bounded.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Where a worker leaves 4 columns (c4) of row r of its O: chunks of 32 columns
// in its K stages and, at d = 128, its first V stage (all of its MMAs are done).
template <class SMEM>
__device__ __forceinline__ uint32_t split_o(SMEM& s, int g, int r, int c4) {
  const int cc = c4 >> 3;
  return smem_u32(cc < 3 ? s.k[g][cc] : s.v[g][0]) + r * 128 + (((c4 & 7) ^ (r & 7)) << 4);
}

// O = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i over the item's parts.  Each
// worker's softmax threads take an equal share of the rows' columns, four
// columns at a time, kOnce of those at once (a round trip to another CTA is
// some 200 ns).
template <class SRC, int D, bool BF16, bool LOCAL, class SMEM, class PARAMS>
__device__ __forceinline__ void merge_split(const PARAMS& p, SMEM& s, int g) {
  constexpr int kOnce = 4;
  size_t out;
  const int rows = SRC::place(p, out), parts = LOCAL ? 2 : 2 * p.cluster;
  const int part = LOCAL ? g : 2 * static_cast<int>(cluster_rank()) + g;
#pragma unroll 1
  for (int i0 = part * 128 + (threadIdx.x & 127); i0 < rows * (D / 4); i0 += 128 * kOnce * parts) {
    float m[kOnce], sum[kOnce];
    float4 y[kOnce];
#pragma unroll
    for (int u = 0; u < kOnce; ++u) {
      m[u] = -INFINITY;
      sum[u] = 0.f;
      y[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll 2
    for (int k = 0; k < parts; ++k) {
      float2 st[kOnce];
      float4 x[kOnce];
#pragma unroll
      for (int u = 0; u < kOnce; ++u) {
        const int i = min(i0 + 128 * parts * u, 128 * (D / 4) - 1), r = i / (D / 4);
        st[u] = cluster_ld2<LOCAL>(smem_u32(s.q[k & 1]) + r * 8, k >> 1);
        x[u] = cluster_ld4<LOCAL>(split_o(s, k & 1, r, i % (D / 4)), k >> 1);
      }
#pragma unroll
      for (int u = 0; u < kOnce; ++u) {
        const float mn = fmaxf(m[u], st[u].x), ref = mn == -INFINITY ? 0.f : mn, a = ex2(m[u] - ref), b = ex2(st[u].x - ref);
        sum[u] = fmaf(sum[u], a, b * st[u].y);
        y[u] = make_float4(fmaf(y[u].x, a, b * x[u].x), fmaf(y[u].y, a, b * x[u].y), fmaf(y[u].z, a, b * x[u].z),
                           fmaf(y[u].w, a, b * x[u].w));
        m[u] = mn;
      }
    }
#pragma unroll
    for (int u = 0; u < kOnce; ++u) {
      const int i = i0 + 128 * parts * u;
      if (i >= rows * (D / 4)) break;
      const float inv = sum[u] == 0.f ? 0.f : 1.f / sum[u];
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + (out + i / (D / 4)) * D + i % (D / 4) * 4) =
          make_uint2(pack2<BF16>(y[u].x * inv, y[u].y * inv), pack2<BF16>(y[u].z * inv, y[u].w * inv));
    }
  }
}

// A wait that gives the same answer in every lane of the warp.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const volatile int* abort_flag) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, kWaitNs));
}

// O row (d fp32 columns at tOr) *= alpha, in TMEM; a loop, being rare.
template <int D>
__device__ __forceinline__ void rescale_row(uint32_t tOr, float alpha) {
#pragma unroll 1
  for (int cc = 0; cc < D / 32; ++cc) {
    uint32_t o[32];
    tmem_ld32(tOr + cc * 32, o);
    tmem_ld_wait(o);
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
    tmem_st32(tOr + cc * 32, o);
  }
}

template <class SRC, int D, bool BF16, int MODE, int REP>
__global__ void __launch_bounds__(kThreads, 1)
    scored_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const __grid_constant__ typename SRC::Params p) {
  using Sh = Shape<D, REP>;
  constexpr int BN = Sh::BN, REGIONS = D / 64, Q_ATOM = kBM * 128;
  constexpr int KEYS = BN / REP, CHUNKS = KEYS / 32, ROWS = kBM / REP;  // a thread's keys; rows of one copy of Q
  using Shared = Smem<SRC, D, REP>;
  extern __shared__ uint8_t smem_raw[];
  Shared& s = *reinterpret_cast<Shared*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x < 2) {
    Worker<SRC, D, REP>& w = s.w[threadIdx.x];
    mbar_init(&w.q_full, 1);
    mbar_init(&w.q_done, 1);
    for (int i = 0; i < Sh::K; ++i) {
      mbar_init(&w.k_full[i], 1);
      mbar_init(&w.k_free[i], 1);
    }
    for (int i = 0; i < Sh::V; ++i) {
      mbar_init(&w.v_full[i], 1);
      mbar_init(&w.v_free[i], 1);
    }
    mbar_init(&w.s_full, 1);
    mbar_init(&w.s_free, 128);
    mbar_init(&w.p_full, 128);
    mbar_init(&w.pv_done, 1);
    mbar_init(&w.merge, 128);
    mbar_init(&w.drain, 1);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&w.ring_full[i], 1);
      mbar_init(&w.ring_free[i], kReaders);
    }
    if (threadIdx.x == 0) {
      s.abort_flag = 0;
      SRC::init(s.src);
    }
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(&s.tmem_base, 512);
    tmem_relinquish();
  }
  SRC::prologue(p, s.src);  // all threads; may use __syncthreads
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int g = warp < 4 ? warp & 1 : (warp - 4) >> 2;  // the warp's worker
  Worker<SRC, D, REP>& w = s.w[g];
  const uint32_t tS = s.tmem_base + BN * g, tP = s.tmem_base + 2 * BN + BN / 2 * g, tO = s.tmem_base + 512 - 2 * D + D * g;
  volatile int* abort_flag = &s.abort_flag;
  auto fail = [&]() {
    *abort_flag = 1;
    if (p.err) raise_error(p.err, STOF_DEVERR_PIPE_TIMEOUT);
  };
  // the worker's segment number `handed`, out of its ring (a whole warp)
  auto read_ring = [&](int handed, Segment<typename SRC::Item>& seg) {
    const int slot = handed % kRing;
    if (!warp_wait(&w.ring_full[slot], (handed / kRing) & 1, abort_flag)) return Next::lost;
    seg = w.ring[slot];
    __syncwarp();  // every lane has read it
    if (lane == 0) mbar_arrive(&w.ring_free[slot]);
    return seg.n >= 0 ? Next::segment : Next::none;
  };
  Segment<typename SRC::Item> seg{};
  bool ok = true;

  if (warp < 4)
    regs_dec<kProducerRegs>();
  else
    regs_inc<kSoftmaxRegs>();
  if (warp < 2) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tmap(&tmQ);
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
      typename SRC::Lead lead(p, s.src, g);
      int ik = 0, iv = 0, nq = 0;  // K, V and Q tiles so far
      int sk = 0, pk = 0, sv = 0, pv = 0;
      // one K or V tile of the segment; K runs one tile ahead of V
      auto copy = [&](bool is_k, int t) {
        int& i = is_k ? ik : iv;
        int& st = is_k ? sk : sv;
        int& ph = is_k ? pk : pv;
        const int depth = is_k ? Sh::K : Sh::V;
        uint64_t* full = (is_k ? w.k_full : w.v_full) + st;
        const int row = SRC::tile_key(p, seg.item, seg.n - 1 - t);
        if (i >= depth && !mbar_wait((is_k ? w.k_free : w.v_free) + st, ph ^ 1, abort_flag, kWaitNs)) return false;
        uint8_t* to = is_k ? s.k[g][st] : s.v[g][st];
        const CUtensorMap* map = is_k ? &tmK : &tmV;
        if (MODE == MODE_DISTANCE && is_k) w.key[i & 7] = row;
        mbar_arrive_expect_tx(full, Sh::STAGE);
#pragma unroll
        for (int r = 0; r < REGIONS; ++r) tma_load_3d(to + r * Sh::ATOM, map, full, 64 * r, row, seg.kv_plane);
        ++i;
        if (++st == depth) {
          st = 0;
          ph ^= 1;
        }
        return true;
      };
#pragma unroll 1
      for (int handed = 0; ok; ++handed) {
        const Next got = lead.next(p, s.src, abort_flag, seg);
        const int slot = handed % kRing;
        if (got == Next::lost ||
            (handed >= kRing && !mbar_wait(&w.ring_free[slot], (handed / kRing - 1) & 1, abort_flag, kWaitNs))) {
          ok = false;
          break;
        }
        if (got == Next::none) seg.n = -1;
        w.ring[slot] = seg;
        mbar_arrive(&w.ring_full[slot]);
        if (got == Next::none) break;
        if (seg.n == 0) continue;  // a query tile without listed tiles
        // Q is overwritten once the last segment's score MMAs are done
        if (nq > 0 && !mbar_wait(&w.q_done, (nq - 1) & 1, abort_flag, kWaitNs)) {
          ok = false;
          break;
        }
        ++nq;
        mbar_arrive_expect_tx(&w.q_full, kBM * D * 2);
#pragma unroll
        for (int r = 0; r < REGIONS; ++r)
#pragma unroll
          for (int x = 0; x < REP; ++x)
            tma_load_3d(s.q[g] + r * Q_ATOM + x * ROWS * 128, &tmQ, &w.q_full, 64 * r, seg.q_row, seg.q_plane);
        // K_0, K_1, V_0, K_2, V_1, ...
#pragma unroll 1
        for (int x = 0; ok && x < 2 * seg.n; ++x) {
          const bool is_k = x == 0 || (x & 1 && x < 2 * seg.n - 1);
          ok = copy(is_k, is_k ? (x + 1) >> 1 : (x - 1) >> 1);
        }
      }
      if (!ok) fail();
      lead.drain(s.src);
      if (*abort_flag) {  // let every copy this thread started land before exit
        if (nq > 0) mbar_wait_timeout(&w.q_full, (nq - 1) & 1, kWaitNs);
        for (int i = ik - Sh::K < 0 ? 0 : ik - Sh::K; i < ik; ++i) mbar_wait_timeout(&w.k_full[i % Sh::K], (i / Sh::K) & 1, kWaitNs);
        for (int i = iv - Sh::V < 0 ? 0 : iv - Sh::V; i < iv; ++i) mbar_wait_timeout(&w.v_full[i % Sh::V], (i / Sh::V) & 1, kWaitNs);
      }
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------ MMAs
    constexpr uint32_t idesc_qk = idesc_f16(BF16 ? 1 : 0, 0, kBM, BN);
    constexpr uint32_t idesc_pv = idesc_f16(BF16 ? 1 : 0, 1, kBM, D);
    const uint64_t qdesc = smem_desc_sw128(smem_u32(s.q[g]), 16, 1024);
    const uint64_t kdesc0 = smem_desc_sw128(smem_u32(s.k[g][0]), 16, 1024);
    const uint64_t vdesc0 = smem_desc_sw128(smem_u32(s.v[g][0]), Sh::ATOM, 1024);
    int j = 0, i = 0;  // tiles scored, tiles accumulated so far
    int sk = 0, pk = 0, sv = 0, pv = 0, nq = 0;
    // S = Q K_t^T
    auto score = [&](int t) {
      if (!warp_wait(&w.k_full[sk], pk, abort_flag)) return false;
      if (j > 0 && !warp_wait(&w.s_free, (j - 1) & 1, abort_flag)) return false;  // S has been loaded
      tc_fence_after();
      if (elect_one()) {
        const uint64_t kd = kdesc0 + static_cast<uint64_t>(sk) * (Sh::STAGE / 16);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)  // 32 B per K step inside an atom
          mma_f16_ss(tS, qdesc + (kk >> 2) * (Q_ATOM / 16) + (kk & 3) * 2, kd + (kk >> 2) * (Sh::ATOM / 16) + (kk & 3) * 2,
                     idesc_qk, kk > 0 ? 1u : 0u);
        mma_commit(&w.s_full);
        mma_commit(&w.k_free[sk]);
        if (t == seg.n - 1) mma_commit(&w.q_done);
      }
      __syncwarp();
      ++j;
      if (++sk == Sh::K) {
        sk = 0;
        pk ^= 1;
      }
      return true;
    };
    // O += P V_t
    auto accumulate = [&](int t) {
      if (!warp_wait(&w.v_full[sv], pv, abort_flag)) return false;
      if constexpr (SRC::kClearsV) {
        // V rows behind the request's last token may hold anything, and
        // 0 * NaN is NaN: clear them before the MMA reads the tile
        const int end = SRC::tile_end(seg.item, seg.n - 1 - t);
        if (end < BN) {
#pragma unroll 1
          for (int x = lane + end * 8; x < BN * 8; x += 32)
#pragma unroll
            for (int r = 0; r < REGIONS; ++r)
              *reinterpret_cast<uint4*>(s.v[g][sv] + r * Sh::ATOM + x * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
        }
      }
      if (!warp_wait(&w.p_full, i & 1, abort_flag)) return false;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t vd = vdesc0 + static_cast<uint64_t>(sv) * (Sh::STAGE / 16);
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk)  // 16 keys a K step; the segment's first tile overwrites O
          mma_f16_ts(tO, tP + kk * 8, vd + kk * 128, idesc_pv, (t > 0 || kk > 0) ? 1u : 0u);
        mma_commit(&w.pv_done);
        mma_commit(&w.v_free[sv]);
      }
      __syncwarp();
      ++i;
      if (++sv == Sh::V) {
        sv = 0;
        pv ^= 1;
      }
      return true;
    };
#pragma unroll 1
    for (int handed = 0; ok; ++handed) {
      const Next got = read_ring(handed, seg);
      if (got == Next::none) break;
      ok = got == Next::segment;
      if (!ok || seg.n == 0) continue;
      ok = warp_wait(&w.q_full, nq & 1, abort_flag);
      ++nq;
      // S_0, S_1, O_0, S_2, O_1, ...
#pragma unroll 1
      for (int t = -1; ok && t < seg.n; ++t) {
        if (t + 1 < seg.n) ok = score(t + 1);
        if (ok && t >= 0) ok = accumulate(t);
      }
    }
    if (elect_one()) {  // the lane that issued the MMAs
      if (!ok) fail();
      mma_commit(&w.drain);
      mbar_wait_timeout(&w.drain, 0, kWaitNs);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;  // query row in the tile == TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const int part = r / ROWS;  // the copy of Q this thread's row belongs to: its keys of a tile are KEYS part ..
    const uint32_t tSr = tS + lane_off + KEYS * part, tPr = tP + lane_off + KEYS / 2 * part, tOr = tO + lane_off;
    typename SRC::Row row;
    int j = 0, merges = 0;  // tiles so far; segments merged (REP > 1)
    if constexpr (REP > 1) {  // P is 0 outside this copy's keys, from here on
      const uint32_t zero[16] = {};
#pragma unroll
      for (int x = 0; x < BN / 32; ++x) tmem_st16(tP + lane_off + 16 * x, zero);
      tmem_st_wait();
    }
#pragma unroll 1
    for (int handed = 0;; ++handed) {
      const Next got = read_ring(handed, seg);
      if (got != Next::segment) {
        ok = got == Next::none;
        break;
      }
      const bool live = SRC::begin_row(p, row, seg, r % ROWS);   // the row is one of the call's
      const bool alive = __any_sync(0xffffffffu, live);   // the warp has such a row
      float slope = 0.f;
      uint32_t base = 0;  // the row's reference distance
      if (MODE == MODE_DISTANCE && p.slopes && live) {
        slope = __ldg(p.slopes + row.head) * kLog2e;
        base = SRC::reference(p, row, seg.item, slope < 0.f);
      }
      float m_ref = -INFINITY, l = 0.f;
      SRC::template prefetch<BN>(p, row, seg.item, seg.n - 1);
#pragma unroll 1
      for (int t = 0; t < seg.n; ++t, ++j) {
        if (!warp_wait(&w.s_full, j & 1, abort_flag)) { ok = false; break; }
        tc_fence_after();
        if (alive) {
          uint32_t sr[CHUNKS][32];
          load_scores(tSr, sr);
          tc_fence_before();
          mbar_arrive(&w.s_free);  // the scores are in registers: S may be overwritten
          const int tile = seg.n - 1 - t;
          const bool partial = SRC::partial(seg.item, tile);
          uint32_t bits[CHUNKS] = {};
          if (partial) SRC::template bits<BN>(p, row, seg.item, tile, KEYS * part, bits);
          SRC::template prefetch<BN>(p, row, seg.item, tile - 1);
          uint32_t pk[CHUNKS][16];
          float alpha = 1.f;
          // the max mt of the tile's scores (log2 units) becomes the
          // reference when it exceeds it by more than 2^8 (their difference
          // is exact where it counts, while m_ref + 8 is rounded: at -2^27 to
          // m_ref + 16, and 2^16 is past fp16)
          auto raise_ref = [&](float mt) {
            if (mt - m_ref > kRescaleThreshold) {
              alpha = ex2(m_ref - mt);  // 0 when m_ref = -inf
              m_ref = mt;
            }
            l *= alpha;
            return m_ref == -INFINITY ? 0.f : -m_ref;
          };
          // P of final scores (times c) and its sum.  With 64 scores a thread
          // (registers to keep them) the max is not looked for: P is taken with
          // the reference so far, and taken again only if a row's sum says
          // that a score exceeds it by kSlack.  (512 rows per K/V head over 2
          // x 131000 keys: 366 -> 339 us; with 32 scores, 27.7 -> 30.5 for 7
          // rows, 32 requests.)
          auto exp_rows = [&](float c) {
            float sum;
            if constexpr (CHUNKS != 2) {
              sum = exp_row<CHUNKS, BF16>(sr, c, raise_ref(row_max(sr) * c), pk);
            } else {
              bool look = __any_sync(0xffffffffu, live && m_ref == -INFINITY);
#pragma unroll 1
              for (;;) {
                const float nmu = look ? raise_ref(row_max(sr) * c) : -m_ref;
                sum = exp_row<CHUNKS, BF16>(sr, c, nmu, pk);
                if (look || !__any_sync(0xffffffffu, live && sum > kSlack<BF16>)) break;
                look = true;
              }
            }
            return sum;
          };
          if constexpr (MODE == MODE_PLAIN) {
            if (partial) mask_scores(sr, bits);
            l += exp_rows(p.k.c);
          } else if constexpr (MODE == MODE_CAP && BF16) {
            // Capped scores lie within a of 0 (log2 units; the host sends a
            // larger cap to MODE_DISTANCE), and bf16 and fp32 hold 2^-a to
            // 2^a: no running max, the reference is 0 throughout.
            m_ref = 0.f;
            if constexpr (CHUNKS > 2) {
              const bool within = __all_sync(0xffffffffu, row_within(sr, p.k.lim));
              if (!partial && within) {
                l += exp_row_capped<CHUNKS, BF16, false>(sr, p.k, 0.f, pk, bits);
              } else {
                cap_scores(sr, p.k, within);
                if (partial) mask_scores(sr, bits);
                l += exp_row<CHUNKS, BF16>(sr, 1.f, 0.f, pk);
              }
            } else {
              // up to 64 scores: the polynomial for all while its range is
              // being checked (there are registers to keep the scores; with
              // 128 of them this spills 530 bytes a thread)
              float sum = partial ? exp_row_capped<CHUNKS, BF16, true>(sr, p.k, 0.f, pk, bits)
                                  : exp_row_capped<CHUNKS, BF16, false>(sr, p.k, 0.f, pk, bits);
              if (!__all_sync(0xffffffffu, row_within(sr, p.k.lim))) {
                cap_scores(sr, p.k, false);
                if (partial) mask_scores(sr, bits);
                sum = exp_row<CHUNKS, BF16>(sr, 1.f, 0.f, pk);
              }
              l += sum;
            }
          } else if constexpr (MODE == MODE_CAP) {
            const bool within = __all_sync(0xffffffffu, row_within(sr, p.k.lim));
            if (within && !partial && p.k.k1 > 0.f) {
              // the cap is increasing: its max is that of the largest product
              const float nmu = raise_ref(cap_poly(p.k, row_max(sr)));
              l += exp_row_capped<CHUNKS, BF16, false>(sr, p.k, nmu, pk, bits);
            } else {
              cap_scores(sr, p.k, within);
              if (partial) mask_scores(sr, bits);
              l += exp_rows(1.f);
            }
          } else {
            float c = p.k.c;
            if (p.k.cap) {
              cap_scores(sr, p.k, __all_sync(0xffffffffu, row_within(sr, p.k.lim)));
              c = 1.f;
            }
            SRC::template lower<BN>(p, row, seg.item, tile, w.key[j & 7] + KEYS * part, sr, c, slope, base);
            c = 1.f;
            if (partial) mask_scores(sr, bits);
            l += exp_rows(c);
          }
          if (t > 0) {
            // P is rewritten and O rescaled once the PV of the tile before is done
            if (!warp_wait(&w.pv_done, (j - 1) & 1, abort_flag)) { ok = false; break; }
            tc_fence_after();
            if (__any_sync(0xffffffffu, alpha != 1.f)) rescale_row<D>(tOr, alpha);
          }
          store_p(tPr, pk);
        } else {  // no row of the call: keep the barriers' step
          mbar_arrive(&w.s_free);
          if (t > 0 && !warp_wait(&w.pv_done, (j - 1) & 1, abort_flag)) { ok = false; break; }
        }
        tc_fence_before();
        mbar_arrive(&w.p_full);
      }
      // ---- the segment's end
      if (!ok || (seg.n > 0 && !warp_wait(&w.pv_done, (j - 1) & 1, abort_flag))) {
        ok = false;
        break;
      }
      if constexpr (REP > 1) {
        // A warp has rows of one copy: the first copy's warps merge the
        // others' rows with their own, 32 columns at a time through shared
        // memory.  (The next segment's rows come after barriers of its tiles.)
        static_assert(ROWS % 32 == 0, "whole warps per copy");
        const int rr = r % ROWS;
        auto barrier = [&]() {
          mbar_arrive(&w.merge);
          return warp_wait(&w.merge, merges++ & 1, abort_flag);
        };
        const int at = (part - 1) * ROWS + rr;  // part > 0: this thread's place
        float a[REP];
        tc_fence_after();
        if (part > 0) s.merge_stats[g][at] = make_float2(m_ref, l);
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t o[32];
          if (alive) {
            tmem_ld32(tOr + cc * 32, o);
            tmem_ld_wait(o);
            // a copy that has seen no key: its O is a sum of zeros, or unset
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = l == 0.f ? 0u : o[i];
          }
          if (part > 0 && alive) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              s.merge[g][at * 8 + (i ^ (rr & 7))] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                                                  __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
          }
          if (!(ok = barrier())) break;
          if (part == 0 && alive) {
            if (cc == 0) {
              float m = m_ref, sum = 0.f;
              float2 st[REP];
              st[0] = make_float2(m_ref, l);
#pragma unroll
              for (int k = 1; k < REP; ++k) {
                st[k] = s.merge_stats[g][(k - 1) * ROWS + rr];
                m = fmaxf(m, st[k].x);
              }
              const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
              for (int k = 0; k < REP; ++k) {
                a[k] = ex2(st[k].x - ref);
                sum = fmaf(a[k], st[k].y, sum);
              }
              if (SRC::whole(seg.item)) {
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
                for (int k = 0; k < REP; ++k) a[k] *= inv;
              } else if (live) {
                SRC::put_stats(p, seg.item, g, rr, m, sum);
              }
            }
            float y[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = a[0] * __uint_as_float(o[i]);
#pragma unroll
            for (int k = 1; k < REP; ++k)
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 x = s.merge[g][((k - 1) * ROWS + rr) * 8 + (i ^ (rr & 7))];
                y[4 * i] = fmaf(a[k], x.x, y[4 * i]);
                y[4 * i + 1] = fmaf(a[k], x.y, y[4 * i + 1]);
                y[4 * i + 2] = fmaf(a[k], x.z, y[4 * i + 2]);
                y[4 * i + 3] = fmaf(a[k], x.w, y[4 * i + 3]);
              }
            if (live) {
              if (SRC::whole(seg.item)) {
                uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + row.out * D + cc * 32);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  dst[i] = make_uint4(pack2<BF16>(y[8 * i], y[8 * i + 1]), pack2<BF16>(y[8 * i + 2], y[8 * i + 3]),
                                      pack2<BF16>(y[8 * i + 4], y[8 * i + 5]), pack2<BF16>(y[8 * i + 6], y[8 * i + 7]));
              } else {
                float4* dst = reinterpret_cast<float4*>(SRC::partial_o(p, seg.item, g, rr, D) + cc * 32);
#pragma unroll
                for (int i = 0; i < 8; ++i) dst[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
              }
            }
          }
          if (cc + 1 < D / 32 && !(ok = barrier())) break;  // read before the next columns are written
        }
        if (!ok) break;
        tc_fence_before();
        continue;
      }
      if (!alive) continue;
      tc_fence_after();
      if constexpr (SRC::kSplit) {
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t o[32];
          if (seg.n > 0) {
            tmem_ld32(tOr + cc * 32, o);
            tmem_ld_wait(o);
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = l == 0.f ? 0u : o[i];  // no key seen: a sum of zeros, or unset
#pragma unroll
          for (int i = 0; i < 8; ++i)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(split_o(s, g, r, cc * 8 + i)), "r"(o[4 * i]),
                         "r"(o[4 * i + 1]), "r"(o[4 * i + 2]), "r"(o[4 * i + 3])
                         : "memory");
        }
        reinterpret_cast<float2*>(s.q[g])[r] = make_float2(m_ref, l);
        tc_fence_before();
        continue;
      }
      const bool whole = SRC::whole(seg.item);
      const float scale = whole ? 1.f / l : 1.f;
#pragma unroll 1
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t o[32];
        float x[32];
        if (seg.n > 0) {
          tmem_ld32(tOr + cc * 32, o);
          tmem_ld_wait(o);
        }
        // a row that has seen no key gives 0 (its O is a sum of zeros, or unset)
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = l == 0.f ? 0.f : scale * __uint_as_float(o[i]);
        if (live) {
          if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + row.out * D + cc * 32);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              dst[i] = make_uint4(pack2<BF16>(x[8 * i], x[8 * i + 1]), pack2<BF16>(x[8 * i + 2], x[8 * i + 3]),
                                  pack2<BF16>(x[8 * i + 4], x[8 * i + 5]), pack2<BF16>(x[8 * i + 6], x[8 * i + 7]));
          } else {
            float4* dst = reinterpret_cast<float4*>(SRC::partial_o(p, seg.item, g, r, D) + cc * 32);
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
          }
        }
      }
      if (live && !whole) SRC::put_stats(p, seg.item, g, r, m_ref, l);
      tc_fence_before();  // O is read before the next segment's first p_full lets it be overwritten
    }
    if (!ok && lane == 0) fail();
  }
  tc_fence_before();
  if constexpr (SRC::kSplit) {
    __syncwarp();
    if (p.cluster > 1) {
      cluster_sync();
      if (warp >= 4) merge_split<SRC, D, BF16, false>(p, s, g);
      __syncwarp();
      cluster_sync();  // no CTA ends while another one reads its rows
    } else {
      __syncthreads();
      if (warp >= 4) merge_split<SRC, D, BF16, true>(p, s, g);
    }
  } else {
    __syncthreads();
  }
  if (threadIdx.x == 0) SRC::finish(p, s.src, abort_flag);
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(s.tmem_base, 512);
  }
}

// Launches an instance with its shared memory and register split prepared.
template <class SRC, int D, bool BF16, int MODE, int REP = 1>
stof_status launch_scored(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                          const typename SRC::Params& p, unsigned grid, cudaStream_t s) {
  auto* kernel = scored_kernel<SRC, D, BF16, MODE, REP>;
  constexpr size_t smem = sizeof(Smem<SRC, D, REP>) + 1024;
  static_assert(smem <= 232448, "shared memory");
  stof_status prep = STOF_OK;
  auto prepare = [](const void* arg) {
    stof_status* st = static_cast<stof_status*>(const_cast<void*>(arg));
    auto* k = scored_kernel<SRC, D, BF16, MODE, REP>;
    cudaFuncAttributes fa;
    if (record_cuda(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem))) !=
            cudaSuccess ||
        record_cuda(cudaFuncGetAttributes(&fa, k)) != cudaSuccess) {
      *st = STOF_ERR_CUDA;
      return false;
    }
    if (fa.numRegs != kLaunchRegs) {  // the register split needs exactly this
      *st = STOF_ERR_UNSUPPORTED;
      return false;
    }
    return true;
  };
  if (!once_per_device(reinterpret_cast<const void*>(kernel), prepare, &prep)) return prep;
  if constexpr (SRC::kSplit) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {static_cast<unsigned>(p.cluster), 1, 1};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, mq, mk, mv, p), last = cudaGetLastError();
    return record_cuda(e != cudaSuccess ? e : last) == cudaSuccess ? STOF_OK : STOF_ERR_CUDA;
  }
  kernel<<<grid, kThreads, smem, s>>>(mq, mk, mv, p);
  return record_cuda(cudaGetLastError()) == cudaSuccess ? STOF_OK : STOF_ERR_CUDA;
}

// The mode a call's score options need.
inline int mode_of(float scale, float softcap, bool slopes) {
  if (slopes || softcap > kMaxCapOnly || (softcap <= 0.f && !(scale > 0.f))) return MODE_DISTANCE;
  return softcap > 0.f ? MODE_CAP : MODE_PLAIN;
}

}  // namespace scored
}  // namespace stof
