// Block-wise kernel of stof_mha_fwd_score: scored_kernel.cuh over the listed
// outer tiles of a mask format ("Accelerating Sparse Transformer Inference on
// GPU", gist.science technical summary, Methodology 1, block-wise kernel and
// two-level storage format: listed tiles only, full ones without a mask test,
// partial ones through their 8x8 inner-tile bitmaps); format_source.cuh has
// the order and the split of the work.
#include <climits>

#include "format_source.cuh"

namespace stof {
namespace {

using namespace scored;

// CTAs that share each item (format_source.cuh), 0: items stay whole.  As many
// as are on the SMs at once; 512 keys or more of the longest possible item for
// each of them.  Whole and split, one K/V head: d = 64, 1024
// keys, 8 items 14.1 and 12.5 us, 4096 keys, 32 items 43.2 and 19.1, 128 items
// 43.0 and 33.7; d = 128, 512 keys (one CTA per item) 11.2 and 14.1, 1024 17.4
// and 16.5, 2048 keys, 16 items 30.1 and 18.7, 4096 keys, 32 items 55.7 and
// 23.4.  Eight CTAs an item: 16 clusters of them are not resident at once,
// 46.3 us instead of 18.7; 1024 keys for each CTA 29.6 instead of 23.4.  256
// items in two rounds of one CTA each: 61 us instead of 46.
constexpr uint64_t kSplitCtas = 128;
constexpr int kSplitKeys = 512;
int cluster_of(uint64_t items, int keys) {
  if (keys < 1024) return 0;
  for (int c = 4; c; c /= 2)
    if (items * c <= kSplitCtas && keys >= kSplitKeys * c) return c;
  return 0;
}

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
  const uint64_t items = heads * a.n_tr;
  const int mode = mode_of(a.scale, a.softcap, a.slopes != nullptr);
  p.cluster = cluster_of(items, a.row_ots * 128);
  if (p.cluster)
    return launch_format_split(mq, mk, mv, p, D, BF16, mode, static_cast<unsigned>(items * p.cluster), s);
  return launch_format<false, D, BF16>(mq, mk, mv, p, mode, static_cast<unsigned>(items), s);
}

}  // namespace

bool blockwise_scored_takes(const stof_format& f, int B, int H, int d) {
  // 128 x 128 OTs; items (and with them heads), a head's rows and its keys are counted in 32 bits
  constexpr int kMost = INT_MAX - 128;
  return f.bm == kBM && f.bn == 128 && (d == 64 || d == 128) && static_cast<long long>(B) * H * f.n_tr <= INT_MAX &&
         f.lq <= kMost && f.lk <= kMost;
}

stof_status launch_blockwise_scored(const ScoredParams& p, bool bf16, cudaStream_t s) {
  if (p.d == 64) return bf16 ? launch_d<64, true>(p, s) : launch_d<64, false>(p, s);
  return bf16 ? launch_d<128, true>(p, s) : launch_d<128, false>(p, s);
}

}  // namespace stof
