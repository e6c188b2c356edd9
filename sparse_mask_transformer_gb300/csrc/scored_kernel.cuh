// The block-wise kernel of scored attention (TMA + tcgen05 + TMEM, sm_103a),
// shared by its two sources of tiles:
//   FormatSource  the listed outer tiles of the query tiles of a mask format
//                 (blockwise_score.cu, stof_mha_fwd_score);
//   CacheSource   the 128-key tiles of the requests' K/V caches (tree_attn.cu,
//                 stof_tree_attn_fwd).
// A segment is a run of K/V tiles of 128 keys for one tile of 128 query
// rows; its online softmax gives the rows' O, or a partial O with the rows'
// max and sum where other workers hold the rest.
//
// A CTA runs two workers, softmax warpgroups g = 0 and 1, each with segments
// of its own (its Q tile in shared memory, its P and O in TMEM, its running
// max and sum in registers), one after the other.  While one worker loads Q,
// starts or finishes a segment, the tensor cores, the copies and the other
// worker go on, so that short segments (a few tiles, as packed documents and
// short caches give) cost little more than their tiles.  (Both warpgroups on
// the tiles of one segment, merged at its end, took 88 us instead of
// @DOCS@ us on 4096 tokens of five documents, 32 heads of 128, and 6 us for
// every one-tile segment of a cache.)
//   warp 0      K producer (TMA ring);
//   warp 1      V producer (TMA ring) and the workers' Q tiles;
//   warp 2      TMEM, score MMAs S = Q_g K^T;
//   warp 3      PV MMAs O_g += P_g V, P read from TMEM;
//   warps 4-7, 8-11  the workers' softmax, a thread per query row.
// The workers' tiles take turns (g = 0, 1, 0, 1, ...; when one has no more
// segments, the other goes on alone), in the same order in warps 0 to 3, so
// the rings need no labels.  A softmax warp whose 32 query rows are all past
// the tile's last one only keeps the barriers' step: a decode step of four
// query rows runs one warp in four.
// TMEM columns, d = 128: S [0,128), one buffer that a worker hands on as
// soon as its scores are in registers; P_g [128 + 64 g, +64); O_g [256 +
// 128 g, +128).  d = 64: S_g [128 g, +128), P_g [256 + 64 g, +64), O_g [384 +
// 64 g, +64).
// Every wait is bounded; on timeout the CTA raises STOF_DEVERR_PIPE_TIMEOUT
// (where there is an error word), drains its copies and MMAs, frees TMEM and
// exits.
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

// What becomes of the products: MODE_PLAIN scale > 0 only; MODE_CAP a cap
// only; MODE_DISTANCE distance, with or without a cap, and any scale.
constexpr int MODE_PLAIN = 0, MODE_CAP = 1, MODE_DISTANCE = 2;

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

// Ring depths: K tiles leave early (their MMA comes first), V tiles a softmax
// later; 160 KB in both at d = 64 and 128.
template <int D>
struct Depth {
  static constexpr int K = D == 128 ? 3 : 5, V = D == 128 ? 2 : 5;
};

template <class SRC, int D>
struct alignas(1024) Smem {
  uint8_t q[2][kBM * D * 2];  // per worker
  uint8_t k[Depth<D>::K][128 * D * 2];
  uint8_t v[Depth<D>::V][128 * D * 2];
  uint64_t q_full[2], q_done[2];  // per worker: Q is in place; its segment's score MMAs are done
  uint64_t k_full[Depth<D>::K], k_free[Depth<D>::K], v_full[Depth<D>::V], v_free[Depth<D>::V];
  uint64_t s_full[2], s_free[2], p_full[2], pv_done[2];
  uint64_t drain, drain_qk;
  uint32_t tmem_base;
  int abort_flag;
  typename SRC::Shared src;
};

// Who reads a worker's segments: the K producer (which takes them from the
// source), one thread, or a whole warp.
constexpr int FEED_LEAD = 0, FEED_THREAD = 1, FEED_WARP = 2;

// A wait that gives the same answer in every lane of the warp.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const volatile int* abort_flag) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, kWaitNs));
}

template <class SRC, int D, bool BF16, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    scored_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const __grid_constant__ typename SRC::Params p) {
  constexpr int REGIONS = D / 64, ATOM = 128 * 128, KV_BYTES = 128 * D * 2, CHUNKS = 4;
  constexpr int STK = Depth<D>::K, STV = Depth<D>::V;
  using Seg = Segment<typename SRC::Item>;
  extern __shared__ uint8_t smem_raw[];
  using Shared = Smem<SRC, D>;
  Shared& s = *reinterpret_cast<Shared*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < STK; ++i) {
      mbar_init(&s.k_full[i], 1);
      mbar_init(&s.k_free[i], 1);
    }
    for (int i = 0; i < STV; ++i) {
      mbar_init(&s.v_full[i], 1);
      mbar_init(&s.v_free[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.q_full[i], 1);
      mbar_init(&s.q_done[i], 1);
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.s_free[i], 128);
      mbar_init(&s.p_full[i], 128);
      mbar_init(&s.pv_done[i], 1);
    }
    mbar_init(&s.drain, 1);
    mbar_init(&s.drain_qk, 1);
    s.abort_flag = 0;
    SRC::init(s.src);
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
  const uint32_t tbase = s.tmem_base;
  constexpr uint32_t kP = D == 128 ? 128 : 256, kO = D == 128 ? 256 : 384;
  auto s_at = [&](int g) { return D == 128 ? tbase : tbase + 128 * g; };
  volatile int* abort_flag = &s.abort_flag;
  auto fail = [&]() {
    *abort_flag = 1;
    if (p.err) raise_error(p.err, STOF_DEVERR_PIPE_TIMEOUT);
  };
  // The two workers' tiles in turn: begin(g) at each new segment with tiles,
  // tile(g) for every tile (false: give up), until both have no more.
  auto turns = [&](auto& feed0, auto& feed1, Seg (&seg)[2], int (&t)[2], auto&& begin, auto&& tile) {
    bool has[2], ok = true;
    auto advance = [&](auto gc, auto& feed) {
      constexpr int G = decltype(gc)::value;
      do has[G] = feed.next(seg[G]);
      while (has[G] && seg[G].n == 0);
      t[G] = 0;
      if (has[G]) ok = begin(gc) && ok;
    };
    auto step = [&](auto gc, auto& feed) {
      constexpr int G = decltype(gc)::value;
      ok = tile(gc);
      if (ok && ++t[G] == seg[G].n) advance(gc, feed);
    };
    std::integral_constant<int, 0> w0;
    std::integral_constant<int, 1> w1;
    advance(w0, feed0);
    advance(w1, feed1);
    while (ok && (has[0] || has[1])) {
      if (has[0]) step(w0, feed0);
      if (ok && has[1]) step(w1, feed1);
    }
    return ok && feed0.ok && feed1.ok;
  };

  if (warp < 4) {
    regs_dec<kProducerRegs>();
    Seg seg[2];
    int t[2] = {0, 0};
    if (warp == 0) {
      // ------------------------------------------------------------ K producer
      if (lane == 0) {
        prefetch_tmap(&tmK);
        typename SRC::Lead lead(p, s.src, abort_flag);
        typename SRC::template Feed<FEED_LEAD> f0(p, s.src, 0, abort_flag, &lead), f1(p, s.src, 1, abort_flag, &lead);
        int it = 0, st = 0, ph = 0;
        const bool ok = turns(f0, f1, seg, t, [&](auto) { return true; }, [&](auto gc) {
          constexpr int G = decltype(gc)::value;
          if (it >= STK && !mbar_wait(&s.k_free[st], ph ^ 1, abort_flag, kWaitNs)) return false;
          const int row = SRC::tile_key(p, seg[G].item, t[G]);
          mbar_arrive_expect_tx(&s.k_full[st], KV_BYTES);
#pragma unroll
          for (int r = 0; r < REGIONS; ++r)
            tma_load_3d(s.k[st] + r * ATOM, &tmK, &s.k_full[st], 64 * r, row, seg[G].kv_plane);
          ++it;
          if (++st == STK) {
            st = 0;
            ph ^= 1;
          }
          return true;
        });
        if (!ok) fail();
        lead.drain();
        if (*abort_flag) {  // let every copy this thread started land before exit
          for (int i = it - STK < 0 ? 0 : it - STK; i < it; ++i) mbar_wait_timeout(&s.k_full[i % STK], (i / STK) & 1, kWaitNs);
        }
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ Q tiles, V producer
      if (lane == 0) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmV);
        typename SRC::template Feed<FEED_THREAD> f0(p, s.src, 0, abort_flag, nullptr), f1(p, s.src, 1, abort_flag, nullptr);
        int it = 0, st = 0, ph = 0, nq[2] = {0, 0};
        const bool ok = turns(f0, f1, seg, t, [&](auto gc) {
          constexpr int G = decltype(gc)::value;
          // the worker's Q is overwritten once its last segment's score MMAs are done
          if (nq[G] > 0 && !mbar_wait(&s.q_done[G], (nq[G] - 1) & 1, abort_flag, kWaitNs)) return false;
          ++nq[G];
          mbar_arrive_expect_tx(&s.q_full[G], kBM * D * 2);
#pragma unroll
          for (int r = 0; r < REGIONS; ++r)
            tma_load_3d(s.q[G] + r * ATOM, &tmQ, &s.q_full[G], 64 * r, seg[G].q_row, seg[G].q_plane);
          return true;
        }, [&](auto gc) {
          constexpr int G = decltype(gc)::value;
          if (it >= STV && !mbar_wait(&s.v_free[st], ph ^ 1, abort_flag, kWaitNs)) return false;
          const int row = SRC::tile_key(p, seg[G].item, t[G]);
          mbar_arrive_expect_tx(&s.v_full[st], KV_BYTES);
#pragma unroll
          for (int r = 0; r < REGIONS; ++r)
            tma_load_3d(s.v[st] + r * ATOM, &tmV, &s.v_full[st], 64 * r, row, seg[G].kv_plane);
          ++it;
          if (++st == STV) {
            st = 0;
            ph ^= 1;
          }
          return true;
        });
        if (!ok) fail();
        if (*abort_flag) {
          for (int g = 0; g < 2; ++g)
            if (nq[g] > 0) mbar_wait_timeout(&s.q_full[g], (nq[g] - 1) & 1, kWaitNs);
          for (int i = it - STV < 0 ? 0 : it - STV; i < it; ++i) mbar_wait_timeout(&s.v_full[i % STV], (i / STV) & 1, kWaitNs);
        }
      }
    } else if (warp == 2) {
      // ------------------------------------------------------------ score MMAs
      constexpr uint32_t idesc_qk = idesc_f16(BF16 ? 1 : 0, 0, kBM, 128);
      const uint64_t qdesc0 = smem_desc_sw128(smem_u32(s.q[0]), 16, 1024);
      const uint64_t kdesc0 = smem_desc_sw128(smem_u32(s.k[0]), 16, 1024);
      typename SRC::template Feed<FEED_WARP> f0(p, s.src, 0, abort_flag, nullptr), f1(p, s.src, 1, abort_flag, nullptr);
      int st = 0, ph = 0, nq[2] = {0, 0}, j[2] = {0, 0};
      int prev_g = -1, prev_j = 0;  // the tile issued last
      const bool ok = turns(f0, f1, seg, t, [&](auto) { return true; }, [&](auto gc) {
        constexpr int G = decltype(gc)::value;
        if (t[G] == 0) {
          if (!warp_wait(&s.q_full[G], nq[G] & 1, abort_flag)) return false;
          ++nq[G];
        }
        if (!warp_wait(&s.k_full[st], ph, abort_flag)) return false;
        if constexpr (D == 128) {  // one S: the tile before this one has been loaded
          if (prev_g >= 0 && !warp_wait(&s.s_free[prev_g], prev_j & 1, abort_flag)) return false;
          prev_g = G;
          prev_j = j[G];
        } else {
          if (j[G] > 0 && !warp_wait(&s.s_free[G], (j[G] - 1) & 1, abort_flag)) return false;
        }
        tc_fence_after();
        const uint64_t qd = qdesc0 + static_cast<uint64_t>(G) * (kBM * D * 2 / 16);
        const uint64_t kd = kdesc0 + static_cast<uint64_t>(st) * (KV_BYTES / 16);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t off = (kk >> 2) * (ATOM / 16) + (kk & 3) * 2;
            mma_f16_ss(s_at(G), qd + off, kd + off, idesc_qk, kk > 0 ? 1u : 0u);
          }
          mma_commit(&s.s_full[G]);
          mma_commit(&s.k_free[st]);
          if (t[G] == seg[G].n - 1) mma_commit(&s.q_done[G]);
        }
        __syncwarp();
        ++j[G];
        if (++st == STK) {
          st = 0;
          ph ^= 1;
        }
        return true;
      });
      if (elect_one()) {  // the lane that issued the MMAs
        if (!ok) fail();
        mma_commit(&s.drain_qk);
        mbar_wait_timeout(&s.drain_qk, 0, kWaitNs);
      }
    } else {
      // ------------------------------------------------------------ PV MMAs
      constexpr uint32_t idesc_pv = idesc_f16(BF16 ? 1 : 0, 1, kBM, D);
      const uint64_t vdesc0 = smem_desc_sw128(smem_u32(s.v[0]), ATOM, 1024);
      typename SRC::template Feed<FEED_WARP> f0(p, s.src, 0, abort_flag, nullptr), f1(p, s.src, 1, abort_flag, nullptr);
      int st = 0, ph = 0, j[2] = {0, 0};
      const bool ok = turns(f0, f1, seg, t, [&](auto) { return true; }, [&](auto gc) {
        constexpr int G = decltype(gc)::value;
        if (!warp_wait(&s.v_full[st], ph, abort_flag)) return false;
        if constexpr (SRC::kClearsV) {
          // V rows behind the request's last token may hold anything, and
          // 0 * NaN is NaN: clear them before the MMA reads the tile
          const int end = SRC::tile_end(seg[G].item, t[G]);
          if (end < 128) {
            for (int x = lane; x < (128 - end) * 8 * REGIONS; x += 32) {
              const int region = x / ((128 - end) * 8), y = x - region * (128 - end) * 8;
              *reinterpret_cast<uint4*>(s.v[st] + region * ATOM + end * 128 + y * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
        }
        if (!warp_wait(&s.p_full[G], j[G] & 1, abort_flag)) return false;
        tc_fence_after();
        const uint64_t vd = vdesc0 + static_cast<uint64_t>(st) * (KV_BYTES / 16);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)  // the segment's first tile overwrites O_g
            mma_f16_ts(tbase + kO + G * D, tbase + kP + G * 64 + kk * 8, vd + kk * 128, idesc_pv,
                       (t[G] > 0 || kk > 0) ? 1u : 0u);
          mma_commit(&s.pv_done[G]);
          mma_commit(&s.v_free[st]);
        }
        __syncwarp();
        ++j[G];
        if (++st == STV) {
          st = 0;
          ph ^= 1;
        }
        return true;
      });
      if (elect_one()) {
        if (!ok) fail();
        mma_commit(&s.drain);
        mbar_wait_timeout(&s.drain, 0, kWaitNs);
      }
    }
  } else {
    regs_inc<kSoftmaxRegs>();
    // ------------------------------------------------------------ softmax
    const int quarter = warp & 3, g = (warp - 4) >> 2;
    const int r = quarter * 32 + lane;  // query row in the tile == TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tSr = s_at(g) + lane_off, tP = tbase + kP + g * 64 + lane_off, tO = tbase + kO + g * D + lane_off;
    typename SRC::template Feed<FEED_WARP> feed(p, s.src, g, abort_flag, nullptr);
    typename SRC::Row row;
    Seg seg;
    int j = 0;  // this worker's tile count
    bool ok = true;
    while (ok && feed.next(seg)) {
      const bool live = SRC::begin_row(p, row, seg.item, r);  // the row is one of the call's
      const bool alive = __any_sync(0xffffffffu, live);       // the warp has such a row
      float slope = 0.f;
      if (MODE == MODE_DISTANCE && p.slopes && live) slope = __ldg(p.slopes + row.head) * kLog2e;
      float m_ref = -INFINITY, l = 0.f;
      SRC::prefetch(p, row, seg.item, 0, seg.n);
      for (int t = 0; t < seg.n; ++t, ++j) {
        if (!warp_wait(&s.s_full[g], j & 1, abort_flag)) { ok = false; break; }
        tc_fence_after();
        if (alive) {
          uint32_t sr[CHUNKS][32];
          load_scores(tSr, sr);
          tc_fence_before();
          mbar_arrive(&s.s_free[g]);
          const bool partial = SRC::partial(seg.item, t);
          uint32_t bits[CHUNKS] = {};
          if (partial) SRC::bits(p, row, seg.item, t, bits);
          SRC::prefetch(p, row, seg.item, t + 1, seg.n);
          uint32_t pk[CHUNKS][16];
          float alpha = 1.f;
          // the max mt of the tile's scores (log2 units) becomes the
          // reference when it exceeds it by more than 2^8
          auto raise_ref = [&](float mt) {
            if (mt > m_ref + kRescaleThreshold) {
              alpha = ex2(m_ref - mt);  // 0 when m_ref = -inf
              m_ref = mt;
            }
            l *= alpha;
            return m_ref == -INFINITY ? 0.f : -m_ref;
          };
          if constexpr (MODE == MODE_PLAIN) {
            if (partial) mask_scores(sr, bits);
            const float nmu = raise_ref(row_max(sr) * p.k.c);
            l += exp_pack<CHUNKS, BF16>(sr, p.k.c, nmu, pk);
          } else if constexpr (MODE == MODE_CAP) {
            const bool within = __all_sync(0xffffffffu, row_within(sr, p.k.lim));
            if (within && !partial && p.k.k1 > 0.f) {
              // the cap is increasing: its max is that of the largest product
              const float nmu = raise_ref(cap_poly(p.k, row_max(sr)));
              l += exp_pack_capped<CHUNKS, BF16>(sr, p.k, nmu, pk);
            } else {
              cap_scores(sr, p.k, within);
              if (partial) mask_scores(sr, bits);
              const float nmu = raise_ref(row_max(sr));
              l += exp_pack<CHUNKS, BF16>(sr, 1.f, nmu, pk);
            }
          } else {
            float c = p.k.c;
            if (p.k.cap) {
              cap_scores(sr, p.k, __all_sync(0xffffffffu, row_within(sr, p.k.lim)));
              c = 1.f;
            }
            SRC::lower(p, row, seg.item, t, sr, c, slope);
            if (partial) mask_scores(sr, bits);
            const float nmu = raise_ref(row_max(sr));
            l += exp_pack<CHUNKS, BF16>(sr, 1.f, nmu, pk);
          }
          if (t > 0) {
            // P_g is rewritten and O_g rescaled once the PV of the tile before is done
            if (!warp_wait(&s.pv_done[g], (j - 1) & 1, abort_flag)) { ok = false; break; }
            tc_fence_after();
            if (__any_sync(0xffffffffu, alpha != 1.f)) rescale_o<D>(tO, alpha);
          }
          store_p(tP, pk);
        } else {  // no row of the call: keep the barriers' step
          mbar_arrive(&s.s_free[g]);
          if (t > 0 && !warp_wait(&s.pv_done[g], (j - 1) & 1, abort_flag)) { ok = false; break; }
        }
        tc_fence_before();
        mbar_arrive(&s.p_full[g]);
      }
      // ---- the segment's end
      if (!ok || (seg.n > 0 && !warp_wait(&s.pv_done[g], (j - 1) & 1, abort_flag))) {
        ok = false;
        break;
      }
      if (!alive) continue;
      tc_fence_after();
      const bool whole = SRC::whole(seg.item);
      const float w = whole ? 1.f / l : 1.f;
#pragma unroll
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t o[32];
        float x[32];
        if (seg.n > 0) {
          tmem_ld32(tO + cc * 32, o);
          tmem_ld_wait(o);
        }
        // a row that has seen no key gives 0 (its O is a sum of zeros, or unset)
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = l == 0.f ? 0.f : w * __uint_as_float(o[i]);
        if (live) {
          if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + SRC::out_row(p, row, seg.item) * D + cc * 32);
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
      tc_fence_before();  // O_g is read before the next segment's first p_full lets it be overwritten
    }
    if (!(ok && feed.ok) && lane == 0) fail();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// Launches an instance with its shared memory and register split prepared.
template <class SRC, int D, bool BF16, int MODE>
stof_status launch_scored(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                          const typename SRC::Params& p, unsigned grid, cudaStream_t s) {
  auto* kernel = scored_kernel<SRC, D, BF16, MODE>;
  constexpr size_t smem = sizeof(Smem<SRC, D>) + 1024;
  static_assert(smem <= 232448, "shared memory");
  stof_status prep = STOF_OK;
  auto prepare = [](const void* arg) {
    stof_status* st = static_cast<stof_status*>(const_cast<void*>(arg));
    auto* k = scored_kernel<SRC, D, BF16, MODE>;
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
  kernel<<<grid, kThreads, smem, s>>>(mq, mk, mv, p);
  return record_cuda(cudaGetLastError()) == cudaSuccess ? STOF_OK : STOF_ERR_CUDA;
}

// The mode a call's score options need.
inline int mode_of(float scale, float softcap, bool slopes) {
  if (slopes || (softcap <= 0.f && !(scale > 0.f))) return MODE_DISTANCE;
  return softcap > 0.f ? MODE_CAP : MODE_PLAIN;
}

}  // namespace scored
}  // namespace stof
