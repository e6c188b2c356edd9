// The block-wise kernel of scored attention (TMA + tcgen05 + TMEM, sm_103a),
// shared by its two sources of tiles:
//   FormatSource  the listed outer tiles of one query tile of a mask format
//                 (blockwise_score.cu, stof_mha_fwd_score): one CTA a query tile;
//   CacheSource   the 128-row tiles of the requests' K/V caches (tree_attn.cu,
//                 stof_tree_attn_fwd): every CTA an equal share of all tiles
//                 of the call, cut into segments of one query tile each.
// A segment is a run of K/V tiles of 128 keys for one tile of 128 query
// rows; its online softmax gives the rows' O, or a partial O with the rows'
// max and sum where other CTAs hold the rest.  The pipeline is that of the
// library's other block-wise kernels (blockwise.cu), run over segments: the
// rings and barrier phases go on across them.
//   warp 0      K producer (TMA ring);  warp 1  V producer (TMA ring);
//   warp 2      TMEM, the Q tile of each segment, score MMAs S = Q K^T;
//   warp 3      PV MMAs O_g += P_g V, P read from TMEM;
//   warps 4-7, 8-11  softmax warpgroups g = 0, 1: the CTA's tile number
//               parity picks the one that takes a tile; each has its own P
//               and O in TMEM and its own running max and sum, merged at a
//               segment's end.
// A softmax warp whose 32 query rows are all past the tile's last one only
// keeps the barriers' step: a decode step of four query rows runs one warp
// in four.
// TMEM columns: S [0,128) P_0 [128,192) P_1 [192,256) O_g [256 + d g, +d).
// Every wait is bounded; on timeout the CTA raises STOF_DEVERR_PIPE_TIMEOUT
// (where there is an error word), drains its copies and MMAs, frees TMEM and
// exits.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

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

// One run of K/V tiles for one tile of query rows.
struct Segment {
  int q_plane, q_row;   // box of the Q map
  int kv_plane;
  int n;                // tiles
};

template <int D, int ST>
struct alignas(1024) Smem {
  uint8_t q[kBM * D * 2];
  uint8_t k[ST][128 * D * 2];
  uint8_t v[ST][128 * D * 2];
  uint64_t q_full;
  uint64_t q_done;          // the segment's score MMAs are done: Q may be overwritten
  uint64_t k_full[ST], k_free[ST], v_full[ST], v_free[ST];
  uint64_t s_full[2], s_free[2], p_full[2], pv_done[2];
  uint64_t drain, drain_qk;
  uint32_t tmem_base;
  int abort_flag;
  int failed;               // 1 once a softmax thread has failed
};

__device__ __forceinline__ void named_bar_sync(int id, int count) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}

template <class SRC, int D, bool BF16, int MODE, int ST>
__global__ void __launch_bounds__(kThreads, 1)
    scored_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const __grid_constant__ typename SRC::Params p) {
  constexpr int REGIONS = D / 64, ATOM = 128 * 128, KV_BYTES = 128 * D * 2, CHUNKS = 4;
  extern __shared__ uint8_t smem_raw[];
  Smem<D, ST>& s = *reinterpret_cast<Smem<D, ST>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(&s.q_full, 1);
    mbar_init(&s.q_done, 1);
    for (int i = 0; i < ST; ++i) {
      mbar_init(&s.k_full[i], 1);
      mbar_init(&s.k_free[i], 1);
      mbar_init(&s.v_full[i], 1);
      mbar_init(&s.v_free[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.s_free[i], 128);
      mbar_init(&s.p_full[i], 128);
      mbar_init(&s.pv_done[i], 1);
    }
    mbar_init(&s.drain, 1);
    mbar_init(&s.drain_qk, 1);
    s.abort_flag = 0;
    s.failed = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(&s.tmem_base, 512);
    tmem_relinquish();
  }
  SRC src(p);  // may use __syncthreads
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = s.tmem_base, tS = tbase, tP0 = tbase + 128, tO0 = tbase + 256;
  volatile int* abort_flag = &s.abort_flag;
  auto fail = [&]() {
    *abort_flag = 1;
    if (p.err) raise_error(p.err, STOF_DEVERR_PIPE_TIMEOUT);
  };
  auto wwait = [&](uint64_t* bar, uint32_t parity) {  // the same answer in every lane of the warp
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, kWaitNs));
  };
  Segment seg;

  if (warp < 4) {
    regs_dec<kProducerRegs>();
    if (warp < 2) {
      // ------------------------------------------------------------ K and V producers
      if (lane == 0) {
        const CUtensorMap* map = warp == 0 ? &tmK : &tmV;
        uint8_t(*ring)[KV_BYTES] = warp == 0 ? s.k : s.v;
        uint64_t* full = warp == 0 ? s.k_full : s.v_full;
        uint64_t* free_ = warp == 0 ? s.k_free : s.v_free;
        prefetch_tmap(map);
        int it = 0, st = 0, ph = 0;
        bool ok = true;
        while (ok && src.next(seg)) {
          for (int t = 0; t < seg.n; ++t, ++it) {
            if (it >= ST && !mbar_wait(&free_[st], ph ^ 1, abort_flag, kWaitNs)) {
              fail();
              ok = false;
              break;
            }
            const int row = src.tile_key(t);
            mbar_arrive_expect_tx(&full[st], KV_BYTES);
#pragma unroll
            for (int r = 0; r < REGIONS; ++r) tma_load_3d(ring[st] + r * ATOM, map, &full[st], 64 * r, row, seg.kv_plane);
            if (++st == ST) {
              st = 0;
              ph ^= 1;
            }
          }
        }
        if (*abort_flag) {  // let every copy this thread started land before exit
          for (int t = it - ST < 0 ? 0 : it - ST; t < it; ++t) mbar_wait_timeout(&full[t % ST], (t / ST) & 1, kWaitNs);
        }
      }
    } else if (warp == 2) {
      // ------------------------------------------------------------ Q tiles and score MMAs
      constexpr uint32_t idesc_qk = idesc_f16(BF16 ? 1 : 0, 0, kBM, 128);
      const uint64_t qdesc = smem_desc_sw128(smem_u32(s.q), 16, 1024);
      const uint64_t kdesc0 = smem_desc_sw128(smem_u32(s.k[0]), 16, 1024);
      if (lane == 0) prefetch_tmap(&tmQ);
      bool ok = true;
      int it = 0, st = 0, ph = 0, n_seg = 0;
      while (ok && src.next(seg)) {
        if (seg.n == 0) continue;  // a query tile without listed tiles
        // Q is overwritten once the previous segment's score MMAs are done
        if (n_seg > 0 && !wwait(&s.q_done, (n_seg - 1) & 1)) { ok = false; break; }
        if (elect_one()) {
          mbar_arrive_expect_tx(&s.q_full, kBM * D * 2);
#pragma unroll
          for (int r = 0; r < REGIONS; ++r) tma_load_3d(s.q + r * ATOM, &tmQ, &s.q_full, 64 * r, seg.q_row, seg.q_plane);
        }
        __syncwarp();
        ++n_seg;
        if (!wwait(&s.q_full, (n_seg - 1) & 1)) { ok = false; break; }
        for (int t = 0; t < seg.n; ++t, ++it) {
          if (!wwait(&s.k_full[st], ph)) { ok = false; break; }
          if (it >= 1 && !wwait(&s.s_free[(it - 1) & 1], ((it - 1) >> 1) & 1)) { ok = false; break; }
          tc_fence_after();
          const uint64_t kd = kdesc0 + static_cast<uint64_t>(st) * (KV_BYTES / 16);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t off = (kk >> 2) * (ATOM / 16) + (kk & 3) * 2;
              mma_f16_ss(tS, qdesc + off, kd + off, idesc_qk, kk > 0 ? 1u : 0u);
            }
            mma_commit(&s.s_full[it & 1]);
            mma_commit(&s.k_free[st]);
            if (t == seg.n - 1) mma_commit(&s.q_done);
          }
          __syncwarp();
          if (++st == ST) {
            st = 0;
            ph ^= 1;
          }
        }
      }
      if (elect_one()) {  // the lane that issued the copies and MMAs
        if (!ok) fail();
        if (n_seg > 0) mbar_wait_timeout(&s.q_full, (n_seg - 1) & 1, kWaitNs);
        mma_commit(&s.drain_qk);
        mbar_wait_timeout(&s.drain_qk, 0, kWaitNs);
      }
    } else {
      // ------------------------------------------------------------ PV MMAs
      constexpr uint32_t idesc_pv = idesc_f16(BF16 ? 1 : 0, 1, kBM, D);
      const uint64_t vdesc0 = smem_desc_sw128(smem_u32(s.v[0]), ATOM, 1024);
      bool ok = true;
      int it = 0, st = 0, ph = 0;
      while (ok && src.next(seg)) {
        for (int t = 0; t < seg.n; ++t, ++it) {
          const int g = it & 1;
          if (!wwait(&s.v_full[st], ph)) { ok = false; break; }
          if (!wwait(&s.p_full[g], (it >> 1) & 1)) { ok = false; break; }
          tc_fence_after();
          const uint64_t vd = vdesc0 + static_cast<uint64_t>(st) * (KV_BYTES / 16);
          const uint32_t d_tmem = tO0 + g * D, a_tmem = tP0 + g * 64;
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)  // the segment's first tile of a warpgroup overwrites O_g
              mma_f16_ts(d_tmem, a_tmem + kk * 8, vd + kk * 128, idesc_pv, (t >= 2 || kk > 0) ? 1u : 0u);
            mma_commit(&s.pv_done[g]);
            mma_commit(&s.v_free[st]);
          }
          __syncwarp();
          if (++st == ST) {
            st = 0;
            ph ^= 1;
          }
        }
      }
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
    const uint32_t tSr = tS + lane_off, tP = tP0 + g * 64 + lane_off, tO = tO0 + g * D + lane_off;
    typename SRC::Row row;
    int it0 = 0;  // the segment's first tile number
    while (src.next(seg)) {
      const bool live = src.begin_row(row, seg, r);          // the row is one of the call's
      const bool alive = __any_sync(0xffffffffu, live);      // the warp has such a row
      float slope = 0.f;
      if (MODE == MODE_DISTANCE && p.slopes && live) slope = __ldg(p.slopes + row.head) * kLog2e;
      float m_ref = -INFINITY, l = 0.f;
      bool ok = true;
      const int first = (g - it0) & 1;  // this warpgroup's first tile of the segment
      src.prefetch(row, seg, first);
      for (int t = first; ok && t < seg.n; t += 2) {
        const int it = it0 + t, j = it >> 1;  // j: this warpgroup's tile count so far
        if (!wwait(&s.s_full[g], j & 1)) { ok = false; break; }
        tc_fence_after();
        const typename SRC::Tile tile = src.tile(row, seg, t);
        if (alive) {
          uint32_t sr[CHUNKS][32];
          load_scores(tSr, sr);
          tc_fence_before();
          mbar_arrive(&s.s_free[g]);
          uint32_t bits[CHUNKS] = {};
          if (tile.partial) src.bits(row, seg, t, bits);
          src.prefetch(row, seg, t + 2);
          uint32_t pk[CHUNKS][16];
          float alpha = 1.f;
          // the running max mt of the tile's scores (log2 units) becomes the
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
            if (tile.partial) mask_scores(sr, bits);
            const float nmu = raise_ref(row_max(sr) * p.k.c);
            l += exp_pack<CHUNKS, BF16>(sr, p.k.c, nmu, pk);
          } else if constexpr (MODE == MODE_CAP) {
            const bool within = __all_sync(0xffffffffu, row_within(sr, p.k.lim));
            if (within && !tile.partial && p.k.k1 > 0.f) {
              // the cap is increasing: its max is that of the largest product
              const float nmu = raise_ref(cap_poly(p.k, row_max(sr)));
              l += exp_pack_capped<CHUNKS, BF16>(sr, p.k, nmu, pk);
            } else {
              cap_scores(sr, p.k, within);
              if (tile.partial) mask_scores(sr, bits);
              const float nmu = raise_ref(row_max(sr));
              l += exp_pack<CHUNKS, BF16>(sr, 1.f, nmu, pk);
            }
          } else {
            float c = p.k.c;
            if (p.k.cap) {
              cap_scores(sr, p.k, __all_sync(0xffffffffu, row_within(sr, p.k.lim)));
              c = 1.f;
            }
            src.lower(row, tile, sr, c, slope);
            if (tile.partial) mask_scores(sr, bits);
            const float nmu = raise_ref(row_max(sr));
            l += exp_pack<CHUNKS, BF16>(sr, 1.f, nmu, pk);
          }
          if (j > 0) {
            // P_g is rewritten and O_g rescaled once the PV of this
            // warpgroup's previous tile is done
            if (!wwait(&s.pv_done[g], (j - 1) & 1)) { ok = false; break; }
            tc_fence_after();
            if (t > first && __any_sync(0xffffffffu, alpha != 1.f)) rescale_o<D>(tO, alpha);
          }
          store_p(tP, pk);
          tc_fence_before();
        } else {  // no row of the call: keep the barriers' step
          tc_fence_before();
          mbar_arrive(&s.s_free[g]);
          if (j > 0 && !wwait(&s.pv_done[g], (j - 1) & 1)) { ok = false; break; }
        }
        if constexpr (SRC::kClearsV) {
          // V rows behind the request's last token may hold anything, and
          // 0 * NaN is NaN: clear them before the MMA reads the tile
          if (tile.end < 128) {
            const int vst = it % ST;
            if (!wwait(&s.v_full[vst], (it / ST) & 1)) { ok = false; break; }
            if (r >= tile.end) {
#pragma unroll
              for (int x = 0; x < REGIONS * 8; ++x)
                *reinterpret_cast<uint4*>(s.v[vst] + (x >> 3) * ATOM + r * 128 + (x & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
          }
        }
        mbar_arrive(&s.p_full[g]);
      }
      // ---- the segment's end: merge the two warpgroups' partial results;
      // warpgroup g writes columns g d/2 .. g d/2 + d/2 - 1 of each row
      const int mine = seg.n > first ? (seg.n - 1 - first) / 2 + 1 : 0;  // tiles of this warpgroup
      if (ok && mine > 0) ok = wwait(&s.pv_done[g], ((it0 + first + 2 * (mine - 1)) >> 1) & 1);
      if (!ok) s.failed = 1;
      // P_g is free once this warpgroup's last PV is done: its first two
      // columns carry the row's max and sum to the other warpgroup
      if (ok) {
        tmem_st2(tP, __float_as_uint(m_ref), __float_as_uint(l));
        tmem_st_wait();
      }
      tc_fence_before();
      named_bar_sync(1, 256);
      if (s.failed) {
        if (g == 0 && quarter == 0 && lane == 0) fail();
        break;  // all 256 threads
      }
      tc_fence_after();
      if (alive) {
        uint32_t other_m, other_l;
        tmem_ld2(tP0 + (g ^ 1) * 64 + lane_off, other_m, other_l);
        tmem_ld_wait2(other_m, other_l);
        const float m0 = g == 0 ? m_ref : __uint_as_float(other_m), l0 = g == 0 ? l : __uint_as_float(other_l);
        const float m1 = g == 1 ? m_ref : __uint_as_float(other_m), l1 = g == 1 ? l : __uint_as_float(other_l);
        const float m = fmaxf(m0, m1);
        // a warpgroup without a tile of this segment left O_g as it was
        const bool has0 = ((0 - it0) & 1) < seg.n, has1 = ((1 - it0) & 1) < seg.n;
        const float a0 = m0 != -INFINITY ? ex2(m0 - m) : 0.f;
        const float a1 = m1 != -INFINITY ? ex2(m1 - m) : 0.f;
        const float lt = a0 * l0 + a1 * l1;
        const bool whole = src.whole(seg);
        const float inv = whole ? (lt > 0.f ? 1.f / lt : 0.f) : 1.f;
        const float w0 = a0 * inv, w1 = a1 * inv;
#pragma unroll
        for (int cc = 0; cc < D / 64; ++cc) {
          const int col = g * (D / 2) + cc * 32;
          uint32_t o0[32], o1[32];
          float x[32];
          if (has0) {
            tmem_ld32(tO0 + lane_off + col, o0);
            tmem_ld_wait(o0);
          }
          if (has1) {
            tmem_ld32(tO0 + D + lane_off + col, o1);
            tmem_ld_wait(o1);
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            x[i] = has0 ? w0 * __uint_as_float(o0[i]) : 0.f;
            if (has1) x[i] = fmaf(w1, __uint_as_float(o1[i]), x[i]);
          }
          if (live) {
            if (whole) {
              uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + src.out_row(row) * D + col);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                dst[i] = make_uint4(pack2<BF16>(x[8 * i], x[8 * i + 1]), pack2<BF16>(x[8 * i + 2], x[8 * i + 3]),
                                    pack2<BF16>(x[8 * i + 4], x[8 * i + 5]), pack2<BF16>(x[8 * i + 6], x[8 * i + 7]));
            } else {
              float4* dst = reinterpret_cast<float4*>(src.partial_o(seg, r) + col);
#pragma unroll
              for (int i = 0; i < 8; ++i) dst[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
            }
          }
        }
        if (live && !whole && g == 0) src.put_stats(seg, r, m, lt);
        tc_fence_before();
      }
      named_bar_sync(1, 256);  // O_0, O_1 and the statistics are read: the next segment may overwrite them
      it0 += seg.n;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// Launches an instance with its shared memory and register split prepared.
template <class SRC, int D, bool BF16, int MODE, int ST>
stof_status launch_scored(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                          const typename SRC::Params& p, unsigned grid, cudaStream_t s) {
  auto* kernel = scored_kernel<SRC, D, BF16, MODE, ST>;
  constexpr size_t smem = sizeof(Smem<D, ST>) + 1024;
  static_assert(smem <= 232448, "shared memory");
  stof_status prep = STOF_OK;
  auto prepare = [](const void* arg) {
    stof_status* st = static_cast<stof_status*>(const_cast<void*>(arg));
    auto* k = scored_kernel<SRC, D, BF16, MODE, ST>;
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
