// The listed outer tiles of a mask format as a source of scored_kernel.cuh.
//
// An item is a query tile (b, h, OT row I).
//
// FormatSource<false>: the grid has one CTA per item.  The heads go in groups
// whose K and V fit L2 together; inside a group the last, usually longest rows
// of all its heads come first, so that the call ends with short items.  (64 K/V heads of 128, 8192 causal tokens: 949 us;
// all heads in one group 985; head after head, the last head's long rows
// running alone at the end, 1024.)  A running CTA takes the items of CTAs that
// have not started yet (clusterlaunchcontrol.try_cancel: the hardware hands
// out the pending CTA's index instead of launching it) and gives them to its
// two workers, so items are handed out as workers come free, with no counter
// in memory that calls would share.  The first item of worker 0 is the CTA's
// own.
//
// FormatSource<true>, for calls with few items: an item's tiles are cut into
// 2, 4 or 8 equal parts, one for each worker of a cluster of 1, 2 or 4 CTAs;
// every CTA has one part of one item for each of its workers, and the cluster
// merges the parts' rows through its shared memory (no workspace).
#pragma once
#include "scored_kernel.cuh"

namespace stof {
namespace scored {

struct FormatParams : CommonParams {
  int L, n_tr, n_tc, q_start;
  int per_ot;      // tiles per OT: 128 / BN
  int heads;       // B * H
  int head_group;  // heads whose items are interleaved
  int cluster;     // SPLIT: CTAs that share an item
  int64_t stride_b, stride_h;
  const int32_t* full_row_ptr;
  const int32_t* full_col_idx;
  const int32_t* part_row_ptr;
  const int32_t* part_col_idx;
  const uint64_t* bitmaps;
};

template <bool SPLIT>
struct FormatSource {
  using Params = FormatParams;
  static constexpr bool kClearsV = false, kSplit = SPLIT, kTwoPlaces = false;
  struct Item {
    int head;
    int t0;      // SPLIT: the part's first tile
    int f0, nf;  // its first full OT in the list, tiles of its full OTs
    int p0;      // its first partial OT
    int per_ot;  // tiles per OT: 128 / BN
  };
  struct Shared {
    alignas(16) uint4 answer;  // of try_cancel
    uint64_t answered;
    int lock;                  // the producer that handles the answer
    int asked;                 // requests so far; under the lock
    int done;                  // a request was refused: none follows
  };
  struct Loads {};
  template <bool>
  struct Lane {  // what a softmax thread knows of its row in every tile
    int r;
    __device__ Lane(const Params&, const Shared&, int, int row) : r(row) {}
  };
  struct Row {
    int head;
    int pos;                 // the row's position among the keys
    int i;                   // query row of the head
    size_t out;              // row of O
    const uint8_t* bits;     // the row's byte of IT column 0 in a partial tile's bitmaps
    uint32_t nb[16];         // its bytes of the next partial tile, loaded a tile ahead
  };

  static __device__ void init(Shared& s) {
    if (SPLIT) return;
    mbar_init(&s.answered, 1);
    s.lock = s.asked = s.done = 0;
  }
  static __device__ void prologue(const Params&, Shared&) {}
  static __device__ void finish(const Params&, const Shared&, const volatile int*) {}  // the format always has an error word

  // A producer's way to its items.  One request to the hardware is in flight
  // at a time; either producer takes the answer and makes the next request,
  // until one is refused (after which none may follow).
  struct Lead {
    int g;
    bool first = true, ended = false;
    __device__ Lead(const Params&, Shared& s, int worker) : g(worker) {
      if (!SPLIT && g == 0) ask(s);
    }
    static __device__ void ask(Shared& s) {
      mbar_arrive_expect_tx(&s.answered, 16);
      asm volatile(
          "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
              smem_u32(&s.answer)),
          "r"(smem_u32(&s.answered))
          : "memory");
      *static_cast<volatile int*>(&s.asked) = *static_cast<volatile int*>(&s.asked) + 1;
    }
    // Next item, -1: no more, -2: a wait ran out.
    __device__ int take(Shared& s, const volatile int* abort_flag) {
      if (g == 0 && first) {
        first = false;
        return static_cast<int>(blockIdx.x);
      }
      const uint64_t t0 = globaltimer_ns();
      while (atomicCAS_block(&s.lock, 0, 1) != 0)
        if (*abort_flag || globaltimer_ns() - t0 > kWaitNs) return -2;
      __threadfence_block();
      int id = -1;
      if (!*static_cast<volatile int*>(&s.done)) {
        // worker 0 makes the first request as it starts
        while (*static_cast<volatile int*>(&s.asked) == 0)
          if (*abort_flag || globaltimer_ns() - t0 > kWaitNs) return -2;
        if (!mbar_wait(&s.answered, (*static_cast<volatile int*>(&s.asked) - 1) & 1, abort_flag, kWaitNs)) return -2;
        uint32_t got, x;
        asm volatile(
            "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
            "ld.shared.b128 h, [%2];\n\t"
            "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t"
            "mov.u32 %1, 0;\n\t"
            "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
            : "=r"(got), "=r"(x)
            : "r"(smem_u32(&s.answer))
            : "memory");
        if (got) {
          id = static_cast<int>(x);
          fence_proxy_async_smem();  // the answer is read before it is overwritten
          ask(s);
        } else {
          *static_cast<volatile int*>(&s.done) = 1;
        }
      }
      __threadfence_block();
      atomicExch_block(&s.lock, 0);
      return id;
    }
    __device__ Next next(const Params& p, Shared& s, const volatile int* abort_flag, Segment<Item>& seg) {
      int id;
      if constexpr (SPLIT) {
        if (!first) return Next::none;
        first = false;
        id = static_cast<int>(blockIdx.x) / p.cluster;
      } else {
        id = take(s, abort_flag);
        if (id < 0) {
          ended = id == -1;
          return ended ? Next::none : Next::lost;
        }
      }
      int bh, I;
      item(p, id, bh, I);
      const int b = bh / p.H, h = bh - b * p.H;
      const long long mrow = (b * p.stride_b + h * p.stride_h) * p.n_tr + I;
      const int f0 = __ldg(p.full_row_ptr + mrow), f1 = __ldg(p.full_row_ptr + mrow + 1);
      const int p0 = __ldg(p.part_row_ptr + mrow), p1 = __ldg(p.part_row_ptr + mrow + 1);
      seg.q_plane = bh;
      seg.q_row = I * kBM;
      seg.kv_plane = b * (p.H / p.group) + h / p.group;
      seg.n = (f1 - f0 + p1 - p0) * p.per_ot;
      seg.item = Item{h, 0, f0, (f1 - f0) * p.per_ot, p0, p.per_ot};
      if constexpr (SPLIT) {  // part 2 rank + g of the item's tiles
        const int parts = 2 * p.cluster, part = 2 * static_cast<int>(cluster_rank()) + g;
        const int t0 = static_cast<int>(static_cast<long long>(seg.n) * part / parts);
        seg.n = static_cast<int>(static_cast<long long>(seg.n) * (part + 1) / parts) - t0;
        seg.item.t0 = t0;
      }
      return Next::segment;
    }
    // Nothing is written to this CTA's memory after its end: a refusal is the
    // last answer; without one a request may still be in flight.
    __device__ void drain(Shared& s) {
      if (SPLIT) return;
      const int asked = *static_cast<volatile int*>(&s.asked);
      if (!ended && asked > 0) mbar_wait_timeout(&s.answered, (asked - 1) & 1, kWaitNs);
    }
  };

  // Head and query tile of item `id`: the groups' heads interleaved, OT rows from the last.
  static __device__ void item(const Params& p, int id, int& bh, int& I) {
    const int in_group = p.head_group * p.n_tr, head0 = id / in_group * p.head_group, x = id % in_group;
    const int nh = min(p.head_group, p.heads - head0), back = x / nh;
    I = p.n_tr - 1 - back;
    bh = head0 + x - back * nh;
  }
  // SPLIT: first row of O of the CTA's item, and its number of rows.
  static __device__ int place(const Params& p, size_t& out) {
    int bh, I;
    item(p, static_cast<int>(blockIdx.x) / p.cluster, bh, I);
    out = static_cast<size_t>(bh) * p.L + I * kBM;
    return min(kBM, p.L - I * kBM);
  }
  // a tile of the segment among the item's
  static __device__ int at(const Item& x, int t) { return SPLIT ? x.t0 + t : t; }

  // first key of tile t (the OTs' tiles in list order, full ones first)
  static __device__ int tile_key(const Params& p, const Item& x, int t) {
    t = at(x, t);
    const int two = x.per_ot - 1;  // tile t is half t & two of OT t >> two
    int J = t >= x.nf ? p.part_col_idx[x.p0 + ((t - x.nf) >> two)] : p.full_col_idx[x.f0 + (t >> two)];
    if (J < 0 || J >= p.n_tc) {
      raise_error(p.err, STOF_DEVERR_BAD_FORMAT);
      J = 0;
    }
    return J * 128 + 64 * (t & two);
  }
  template <bool KEEP>
  static __device__ bool begin_row(const Params& p, Row& row, const Loads&, const Segment<Item>& seg, const Lane<KEEP>& lane) {
    const int r = lane.r;
    row.head = seg.item.head;
    row.i = seg.q_row + r;
    row.pos = row.i + p.q_start;
    row.out = static_cast<size_t>(seg.q_plane) * p.L + row.i;
    row.bits = reinterpret_cast<const uint8_t*>(p.bitmaps) + (r >> 3) * 128 + (r & 7);
    return row.i < p.L;
  }
  template <int BN>
  static __device__ void prefetch(const Params&, Row& row, const Item& x, int t) {
    if (t < 0) return;
    t = at(x, t);
    if (t >= x.nf) {
      const int u = t - x.nf;
      const uint8_t* src = row.bits + static_cast<long long>(x.p0 + (BN == 64 ? u >> 1 : u)) * 2048 + (BN == 64 ? (u & 1) * 64 : 0);
#pragma unroll
      for (int w = 0; w < BN / 8; ++w) row.nb[w] = __ldg(src + w * 8);
    }
  }
  static __device__ bool partial(const Item& x, int t) { return at(x, t) >= x.nf; }
  template <int BN>
  static __device__ void bits(const Params&, const Row& row, const Item&, int, int, uint32_t (&b)[BN / 32]) {
#pragma unroll
    for (int cc = 0; cc < BN / 32; ++cc)
      b[cc] = row.nb[4 * cc] | (row.nb[4 * cc + 1] << 8) | (row.nb[4 * cc + 2] << 16) | (row.nb[4 * cc + 3] << 24);
  }
  static __device__ float slope(const Params& p, const Row& row) { return __ldg(p.slopes + row.head); }
  // Distance of the nearest (far: farthest) key.
  static __device__ uint32_t reference(const Params& p, const Row& row, const Item&, bool far) {
    return reference_distance(row.pos, p.n_tc * 128 - 1, far);
  }
  template <int BN>
  static __device__ void lower(const Params&, const Row& row, const Item&, int, int key, uint32_t (&sr)[BN / 32][32], float c,
                               float slope, uint32_t base) {
    lower_by_distance(sr, c, slope, row.pos, key, base);
  }
  static __device__ bool whole(const Params&, const Item&) { return true; }
  static __device__ float* partial_o(const Params&, const Item&, const Row&, int, int, int) { return nullptr; }
  static __device__ void put_stats(const Params&, const Item&, const Row&, int, int, float, float) {}
};

// The call's kernel over one of the sources.
template <bool SPLIT, int D, bool BF16>
stof_status launch_format(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const FormatParams& p, int mode,
                          unsigned grid, cudaStream_t s) {
  switch (mode) {
    case MODE_PLAIN: return launch_scored<FormatSource<SPLIT>, D, BF16, MODE_PLAIN>(mq, mk, mv, p, grid, s);
    case MODE_CAP: return launch_scored<FormatSource<SPLIT>, D, BF16, MODE_CAP>(mq, mk, mv, p, grid, s);
    default: return launch_scored<FormatSource<SPLIT>, D, BF16, MODE_DISTANCE>(mq, mk, mv, p, grid, s);
  }
}
// launch_format<true, d, bf16> (blockwise_score_split.cu).
stof_status launch_format_split(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const FormatParams& p,
                                int d, bool bf16, int mode, unsigned grid, cudaStream_t s);

}  // namespace scored
}  // namespace stof
