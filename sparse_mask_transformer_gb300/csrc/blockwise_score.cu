// Block-wise kernel of stof_mha_fwd_score: scored_kernel.cuh over the listed
// outer tiles of a mask format ("Accelerating Sparse Transformer Inference on
// GPU", gist.science technical summary, Methodology 1, block-wise kernel and
// two-level storage format: listed tiles only, full ones without a mask test,
// partial ones through their 8x8 inner-tile bitmaps).
//
// An item is a query tile (b, h, OT row I); the grid has one CTA per item in
// the order of the other block-wise kernels (head-major, so that the CTAs
// running together share a K/V head's tiles in L2; a head's last, usually
// longest rows first).  A running CTA takes the items of CTAs that have not
// started yet (clusterlaunchcontrol.try_cancel: the hardware hands out the
// pending CTA's index instead of launching it) and gives them to its two
// workers, so items are handed out as workers come free, with no counter in
// memory that calls would share.  The K producer takes them; an item and its
// list bounds reach the other warps through a ring in shared memory.
#include "scored_kernel.cuh"

namespace stof {
namespace {

using namespace scored;

struct FormatParams : CommonParams {
  int L, n_tr, n_tc, q_start;
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
  static constexpr int kRing = 4;       // items in flight per worker
  static constexpr int kReaders = 7;    // V producer, score and PV issuers, four softmax warps
  struct Item {
    int id;      // query tile, head-major; negative: no more
    int f0, nf;  // its full OTs in the lists
    int p0;      // its first partial OT
  };
  struct Slot {
    Item item;
    int n;
  };
  struct Shared {
    alignas(16) uint4 answer;           // of try_cancel
    uint64_t answered;
    uint64_t full[2][kRing], free_[2][kRing];
    Slot ring[2][kRing];
  };
  struct Row {
    int head;
    int pos;                 // the row's position among the keys
    int i;                   // query row of the head
    const uint8_t* bits;     // the row's byte of IT column 0 in a partial tile's bitmaps
    uint32_t nb[16];         // its bytes of the next partial tile, loaded a tile ahead
  };

  static __device__ void init(Shared& s) {
    mbar_init(&s.answered, 1);
    for (int g = 0; g < 2; ++g)
      for (int i = 0; i < kRing; ++i) {
        mbar_init(&s.full[g][i], 1);
        mbar_init(&s.free_[g][i], kReaders);
      }
  }
  static __device__ void prologue(const Params&, Shared&) {}

  // The K producer's hold on the items: this CTA's own first, then those of
  // CTAs that have not started.  One request is always in flight until one
  // is refused; none follows a refusal.
  struct Lead {
    const Params& p;
    Shared& s;
    const volatile int* abort_flag;
    int asked = 0;
    bool own = true, done = false, waiting = false;
    __device__ Lead(const Params& params, Shared& sh, const volatile int* abort) : p(params), s(sh), abort_flag(abort) { ask(); }
    __device__ void ask() {
      mbar_arrive_expect_tx(&s.answered, 16);
      asm volatile(
          "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
              smem_u32(&s.answer)),
          "r"(smem_u32(&s.answered))
          : "memory");
      waiting = true;
      ++asked;
    }
    // Next item, -1: no more, -2: the wait ran out.
    __device__ int take() {
      if (own) {
        own = false;
        return static_cast<int>(blockIdx.x);
      }
      if (done) return -1;
      if (!mbar_wait(&s.answered, (asked - 1) & 1, abort_flag, kWaitNs)) return -2;
      waiting = false;
      uint32_t got, id;
      asm volatile(
          "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
          "ld.shared.b128 h, [%2];\n\t"
          "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t"
          "mov.u32 %1, 0;\n\t"
          "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
          : "=r"(got), "=r"(id)
          : "r"(smem_u32(&s.answer))
          : "memory");
      if (!got) {
        done = true;
        return -1;
      }
      fence_proxy_async_smem();  // the answer is read before it is overwritten
      ask();
      return static_cast<int>(id);
    }
    __device__ void drain() {  // no copy into this CTA's memory outlives it
      if (waiting) mbar_wait_timeout(&s.answered, (asked - 1) & 1, kWaitNs);
    }
  };

  // A worker's items.
  template <int WHO>
  struct Feed {
    const Params& p;
    Shared& s;
    const volatile int* abort_flag;
    Lead* lead;
    int g, k = 0;
    bool ok = true;
    __device__ Feed(const Params& params, Shared& sh, int worker, const volatile int* abort, Lead* l)
        : p(params), s(sh), abort_flag(abort), lead(l), g(worker) {}
    __device__ bool next(Segment<Item>& seg) {
      if (!ok) return false;
      const int slot = k % kRing, ph = (k / kRing) & 1;
      Slot& x = s.ring[g][slot];
      if constexpr (WHO == FEED_LEAD) {
        const int id = lead->take();
        Item item{id, 0, 0, 0};
        int n = 0;
        if (id >= 0) {
          const int bh = id / p.n_tr, I = p.n_tr - 1 - (id - bh * p.n_tr);
          const long long mrow = ((bh / p.H) * p.stride_b + (bh % p.H) * p.stride_h) * p.n_tr + I;
          item.f0 = __ldg(p.full_row_ptr + mrow);
          item.p0 = __ldg(p.part_row_ptr + mrow);
          item.nf = __ldg(p.full_row_ptr + mrow + 1) - item.f0;
          n = item.nf + __ldg(p.part_row_ptr + mrow + 1) - item.p0;
        }
        if (k >= kRing && !mbar_wait(&s.free_[g][slot], ph ^ 1, abort_flag, kWaitNs)) return ok = false;
        x.item = item;
        x.n = n;
        mbar_arrive(&s.full[g][slot]);
        if (id == -2) return ok = false;
        fill(seg, item, n);
      } else {
        ok = WHO == FEED_WARP ? warp_wait(&s.full[g][slot], ph, abort_flag)
                              : mbar_wait(&s.full[g][slot], ph, abort_flag, kWaitNs);
        if (!ok) return false;
        fill(seg, x.item, x.n);
        if (WHO == FEED_WARP) __syncwarp();  // every lane has read the slot
        if (WHO == FEED_THREAD || (threadIdx.x & 31) == 0) mbar_arrive(&s.free_[g][slot]);
      }
      ++k;
      return seg.item.id >= 0;
    }
    __device__ void fill(Segment<Item>& seg, const Item& item, int n) {
      const int bh = item.id / p.n_tr;
      seg.item = item;
      seg.q_plane = bh;
      seg.q_row = (p.n_tr - 1 - (item.id - bh * p.n_tr)) * kBM;
      seg.kv_plane = (bh / p.H) * (p.H / p.group) + (bh % p.H) / p.group;
      seg.n = n;
    }
  };

  // first key of the t-th listed OT (full ones first)
  static __device__ int tile_key(const Params& p, const Item& x, int t) {
    int J = t >= x.nf ? p.part_col_idx[x.p0 + (t - x.nf)] : p.full_col_idx[x.f0 + t];
    if (J < 0 || J >= p.n_tc) {
      raise_error(p.err, STOF_DEVERR_BAD_FORMAT);
      J = 0;
    }
    return J * 128;
  }
  static __device__ bool begin_row(const Params& p, Row& row, const Item& x, int r) {
    const int bh = x.id / p.n_tr;
    row.head = bh % p.H;
    row.i = (p.n_tr - 1 - (x.id - bh * p.n_tr)) * kBM + r;
    row.pos = row.i + p.q_start;
    row.bits = reinterpret_cast<const uint8_t*>(p.bitmaps) + (r >> 3) * 128 + (r & 7);
    return row.i < p.L;
  }
  static __device__ void prefetch(const Params&, Row& row, const Item& x, int t, int n) {
    if (t < n && t >= x.nf) {
      const uint8_t* src = row.bits + static_cast<long long>(x.p0 + (t - x.nf)) * 2048;
#pragma unroll
      for (int w = 0; w < 16; ++w) row.nb[w] = __ldg(src + w * 8);
    }
  }
  static __device__ bool partial(const Item& x, int t) { return t >= x.nf; }
  static __device__ void bits(const Params&, const Row& row, const Item&, int, uint32_t (&b)[4]) { assemble_bits<4>(row.nb, b); }
  static __device__ void lower(const Params& p, const Row& row, const Item& x, int t, uint32_t (&sr)[4][32], float c,
                               float slope) {
    const int rel = row.pos - tile_key(p, x, t);
    lower_by_distance(sr, c, slope, static_cast<float>(rel), __all_sync(0xffffffffu, rel >= 127));
  }
  static __device__ bool whole(const Item&) { return true; }
  static __device__ size_t out_row(const Params& p, const Row& row, const Item& x) {
    return static_cast<size_t>(x.id / p.n_tr) * p.L + row.i;
  }
  static __device__ float* partial_o(const Params&, const Item&, int, int, int) { return nullptr; }
  static __device__ void put_stats(const Params&, const Item&, int, int, float, float) {}
};

template <int D, bool BF16>
stof_status launch_d(const ScoredParams& a, cudaStream_t s) {
  CUtensorMap mq, mk, mv;
  const uint64_t heads = static_cast<uint64_t>(a.B) * a.H, kv = heads / a.group;
  if (!make_bw_map(&mq, a.q, heads, a.L, D, kBM, BF16) || !make_bw_map(&mk, a.k, kv, a.Lk, D, 128, BF16) ||
      !make_bw_map(&mv, a.v, kv, a.Lk, D, 128, BF16))
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
  p.stride_b = a.stride_b;
  p.stride_h = a.stride_h;
  p.full_row_ptr = a.full_row_ptr;
  p.full_col_idx = a.full_col_idx;
  p.part_row_ptr = a.part_row_ptr;
  p.part_col_idx = a.part_col_idx;
  p.bitmaps = a.bitmaps;
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
  if (static_cast<long long>(p.B) * p.H * (p.L > p.Lk ? p.L : p.Lk) >= (1ll << 31)) return STOF_ERR_SHAPE;
  if (p.d == 64) return bf16 ? launch_d<64, true>(p, s) : launch_d<64, false>(p, s);
  return bf16 ? launch_d<128, true>(p, s) : launch_d<128, false>(p, s);
}

}  // namespace stof
