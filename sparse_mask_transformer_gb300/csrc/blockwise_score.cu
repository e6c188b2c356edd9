// Block-wise kernel of stof_mha_fwd_score: scored_kernel.cuh over the listed
// outer tiles of a mask format ("Accelerating Sparse Transformer Inference on
// GPU", gist.science technical summary, Methodology 1, block-wise kernel and
// two-level storage format: listed tiles only, full ones without a mask test,
// partial ones through their 8x8 inner-tile bitmaps).
//
// An item is a query tile (b, h, OT row I); the grid has one CTA per item.
// The heads go in groups whose K and V fit L2 together; inside a group the
// last, usually longest rows of all its heads come first, so that the call
// ends with short items.  (64 K/V heads of 128, 8192 causal tokens: 949 us;
// all heads in one group 985; head after head, the last head's long rows
// running alone at the end, 1024.)  A running CTA takes the items of CTAs that
// have not started yet (clusterlaunchcontrol.try_cancel: the hardware hands
// out the pending CTA's index instead of launching it) and gives them to its
// two workers, so items are handed out as workers come free, with no counter
// in memory that calls would share.  The first item of worker 0 is the CTA's
// own.
#include "scored_kernel.cuh"

namespace stof {
namespace {

using namespace scored;

struct FormatParams : CommonParams {
  int L, n_tr, n_tc, q_start;
  int per_ot;      // tiles per OT: 128 / BN
  int heads;       // B * H
  int head_group;  // heads whose items are interleaved
  int64_t stride_b, stride_h;
  const int32_t* full_row_ptr;
  const int32_t* full_col_idx;
  const int32_t* part_row_ptr;
  const int32_t* part_col_idx;
  const uint64_t* bitmaps;
};

struct FormatSource {
  using Params = FormatParams;
  static constexpr bool kClearsV = false;
  struct Item {
    int head;
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
  struct Row {
    int head;
    int pos;                 // the row's position among the keys
    int i;                   // query row of the head
    size_t out;              // row of O
    const uint8_t* bits;     // the row's byte of IT column 0 in a partial tile's bitmaps
    uint32_t nb[16];         // its bytes of the next partial tile, loaded a tile ahead
  };

  static __device__ void init(Shared& s) {
    mbar_init(&s.answered, 1);
    s.lock = s.asked = s.done = 0;
  }
  static __device__ void prologue(const Params&, Shared&) {}

  // A producer's way to its items.  One request to the hardware is in flight
  // at a time; either producer takes the answer and makes the next request,
  // until one is refused (after which none may follow).
  struct Lead {
    int g;
    bool first = true, ended = false;
    __device__ Lead(const Params&, Shared& s, int worker) : g(worker) {
      if (g == 0) ask(s);
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
      const int id = take(s, abort_flag);
      if (id < 0) {
        ended = id == -1;
        return ended ? Next::none : Next::lost;
      }
      const int in_group = p.head_group * p.n_tr, first = id / in_group * p.head_group, x = id % in_group;
      const int nh = min(p.head_group, p.heads - first), back = x / nh;  // heads of the group; OT rows from the last
      const int I = p.n_tr - 1 - back, bh = first + x - back * nh, b = bh / p.H, h = bh - b * p.H;
      const long long mrow = (b * p.stride_b + h * p.stride_h) * p.n_tr + I;
      const int f0 = __ldg(p.full_row_ptr + mrow), f1 = __ldg(p.full_row_ptr + mrow + 1);
      const int p0 = __ldg(p.part_row_ptr + mrow), p1 = __ldg(p.part_row_ptr + mrow + 1);
      seg.q_plane = bh;
      seg.q_row = I * kBM;
      seg.kv_plane = b * (p.H / p.group) + h / p.group;
      seg.n = (f1 - f0 + p1 - p0) * p.per_ot;
      seg.item = Item{h, f0, (f1 - f0) * p.per_ot, p0, p.per_ot};
      return Next::segment;
    }
    // Nothing is written to this CTA's memory after its end: a refusal is the
    // last answer; without one a request may still be in flight.
    __device__ void drain(Shared& s) {
      const int asked = *static_cast<volatile int*>(&s.asked);
      if (!ended && asked > 0) mbar_wait_timeout(&s.answered, (asked - 1) & 1, kWaitNs);
    }
  };

  // first key of tile t (the OTs' tiles in list order, full ones first)
  static __device__ int tile_key(const Params& p, const Item& x, int t) {
    const int two = x.per_ot - 1;  // tile t is half t & two of OT t >> two
    int J = t >= x.nf ? p.part_col_idx[x.p0 + ((t - x.nf) >> two)] : p.full_col_idx[x.f0 + (t >> two)];
    if (J < 0 || J >= p.n_tc) {
      raise_error(p.err, STOF_DEVERR_BAD_FORMAT);
      J = 0;
    }
    return J * 128 + 64 * (t & two);
  }
  static __device__ bool begin_row(const Params& p, Row& row, const Segment<Item>& seg, int r) {
    row.head = seg.item.head;
    row.i = seg.q_row + r;
    row.pos = row.i + p.q_start;
    row.out = static_cast<size_t>(seg.q_plane) * p.L + row.i;
    row.bits = reinterpret_cast<const uint8_t*>(p.bitmaps) + (r >> 3) * 128 + (r & 7);
    return row.i < p.L;
  }
  template <int BN>
  static __device__ void prefetch(const Params&, Row& row, const Item& x, int t) {
    if (t >= x.nf) {
      const int u = t - x.nf;
      const uint8_t* src = row.bits + static_cast<long long>(x.p0 + (BN == 64 ? u >> 1 : u)) * 2048 + (BN == 64 ? (u & 1) * 64 : 0);
#pragma unroll
      for (int w = 0; w < BN / 8; ++w) row.nb[w] = __ldg(src + w * 8);
    }
  }
  static __device__ bool partial(const Item& x, int t) { return t >= x.nf; }
  template <int BN>
  static __device__ void bits(const Params&, const Row& row, const Item&, int, int, uint32_t (&b)[BN / 32]) {
#pragma unroll
    for (int cc = 0; cc < BN / 32; ++cc)
      b[cc] = row.nb[4 * cc] | (row.nb[4 * cc + 1] << 8) | (row.nb[4 * cc + 2] << 16) | (row.nb[4 * cc + 3] << 24);
  }
  template <int BN>
  static __device__ void lower(const Params&, const Row& row, const Item&, int, int key, uint32_t (&sr)[BN / 32][32], float c,
                               float slope) {
    const int rel = row.pos - key;
    lower_by_distance(sr, c, slope, static_cast<float>(rel), __all_sync(0xffffffffu, rel >= BN - 1));
  }
  static __device__ bool whole(const Item&) { return true; }
  static __device__ float* partial_o(const Params&, const Item&, int, int, int) { return nullptr; }
  static __device__ void put_stats(const Params&, const Item&, int, int, float, float) {}
};

template <int D, bool BF16>
stof_status launch_d(const ScoredParams& a, cudaStream_t s) {
  CUtensorMap mq, mk, mv;
  const uint64_t heads = static_cast<uint64_t>(a.B) * a.H, kv = heads / a.group;
  if (!make_bw_map(&mq, a.q, heads, a.L, D, kBM, BF16) || !make_bw_map(&mk, a.k, kv, a.Lk, D, Shape<D>::BN, BF16) ||
      !make_bw_map(&mv, a.v, kv, a.Lk, D, Shape<D>::BN, BF16))
    return STOF_ERR_CUDA;
  FormatParams p;
  p.k = make_score_const(a.scale, a.softcap);
  p.slopes = a.slopes;
  p.o = a.o;
  p.err = a.err;
  p.H = a.H;
  p.group = a.group;
  p.L = a.L;
  p.n_tr = a.n_tr;
  p.n_tc = a.n_tc;
  p.q_start = a.q_start;
  p.per_ot = 128 / Shape<D>::BN;
  p.stride_b = a.stride_b;
  p.stride_h = a.stride_h;
  p.full_row_ptr = a.full_row_ptr;
  p.full_col_idx = a.full_col_idx;
  p.part_row_ptr = a.part_row_ptr;
  p.part_col_idx = a.part_col_idx;
  p.bitmaps = a.bitmaps;
  p.heads = static_cast<int>(heads);
  // 64 MB of K and V, half of the L2 cache; whole groups that share K/V heads
  const uint64_t kv_bytes = static_cast<uint64_t>(a.Lk) * D * 4, fit = (64ull << 20) / kv_bytes;
  const uint64_t together = (fit > 0 ? fit : 1) * a.group;
  p.head_group = static_cast<int>(together < heads ? together : heads);
  const unsigned grid = static_cast<unsigned>(heads * a.n_tr);
  switch (mode_of(a.scale, a.softcap, a.slopes != nullptr)) {
    case MODE_PLAIN: return launch_scored<FormatSource, D, BF16, MODE_PLAIN>(mq, mk, mv, p, grid, s);
    case MODE_CAP: return launch_scored<FormatSource, D, BF16, MODE_CAP>(mq, mk, mv, p, grid, s);
    default: return launch_scored<FormatSource, D, BF16, MODE_DISTANCE>(mq, mk, mv, p, grid, s);
  }
}

}  // namespace

stof_status launch_blockwise_scored(const ScoredParams& p, bool bf16, cudaStream_t s) {
  if (p.bm != kBM || p.bn != 128 || (p.d != 64 && p.d != 128)) return STOF_ERR_UNSUPPORTED;
  // items, heads and rows are counted in 32 bits (n_tr <= L)
  if (static_cast<long long>(p.B) * p.H * (p.L > p.Lk ? p.L : p.Lk) >= (1ll << 31)) return STOF_ERR_SHAPE;
  if (p.d == 64) return bf16 ? launch_d<64, true>(p, s) : launch_d<64, false>(p, s);
  return bf16 ? launch_d<128, true>(p, s) : launch_d<128, false>(p, s);
}

}  // namespace stof
