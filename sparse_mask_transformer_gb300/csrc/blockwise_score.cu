// Block-wise kernel of stof_mha_fwd_score: scored_kernel.cuh over the listed
// outer tiles of a mask format ("Accelerating Sparse Transformer Inference on
// GPU", gist.science technical summary, Methodology 1, block-wise kernel and
// two-level storage format: listed tiles only, full ones without a mask test,
// partial ones through their 8x8 inner-tile bitmaps).
//
// One CTA per query tile (b, h, OT row I), heaviest rows of a head first; the
// K and V of a group's heads are read through the group's plane, whose tiles
// the group's CTAs, adjacent in the grid, find in L2.
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
  struct Row {
    int head;
    int pos;                 // the row's position among the keys
    int i;                   // query row of the head
    const uint8_t* bits;     // the row's byte of IT column 0 in a partial tile's bitmaps
    uint32_t nb[16];         // its bytes of this warpgroup's next partial tile, loaded a tile ahead
  };
  struct Tile {
    bool partial;
    int j0;
  };

  const Params& p;
  int bh, I, f0, nf, p0, n;
  bool done = false;

  __device__ explicit FormatSource(const Params& params) : p(params) {
    bh = static_cast<int>(blockIdx.x / p.n_tr);
    I = p.n_tr - 1 - static_cast<int>(blockIdx.x % p.n_tr);
    const int b = bh / p.H, h = bh % p.H;
    const long long mrow = (b * p.stride_b + h * p.stride_h) * p.n_tr + I;
    f0 = p.full_row_ptr[mrow];
    nf = p.full_row_ptr[mrow + 1] - f0;
    p0 = p.part_row_ptr[mrow];
    n = nf + p.part_row_ptr[mrow + 1] - p0;
  }
  __device__ bool next(Segment& seg) {
    if (done) return false;
    done = true;
    seg.q_plane = bh;
    seg.q_row = I * kBM;
    seg.kv_plane = (bh / p.H) * (p.H / p.group) + (bh % p.H) / p.group;
    seg.n = n;
    return true;
  }
  // first key of the t-th listed OT (full ones first)
  __device__ int tile_key(int t) const {
    int J = t >= nf ? p.part_col_idx[p0 + (t - nf)] : p.full_col_idx[f0 + t];
    if (J < 0 || J >= p.n_tc) {
      raise_error(p.err, STOF_DEVERR_BAD_FORMAT);
      J = 0;
    }
    return J * 128;
  }
  __device__ bool begin_row(Row& row, const Segment&, int r) const {
    row.head = bh % p.H;
    row.i = I * kBM + r;
    row.pos = row.i + p.q_start;
    row.bits = reinterpret_cast<const uint8_t*>(p.bitmaps) + (r >> 3) * 128 + (r & 7);
    return row.i < p.L;
  }
  __device__ void prefetch(Row& row, const Segment& seg, int t) const {
    if (t < seg.n && t >= nf) {
      const uint8_t* src = row.bits + static_cast<long long>(p0 + (t - nf)) * 2048;
#pragma unroll
      for (int w = 0; w < 16; ++w) row.nb[w] = __ldg(src + w * 8);
    }
  }
  __device__ Tile tile(const Row&, const Segment&, int t) const {
    Tile x;
    x.partial = t >= nf;
    x.j0 = p.slopes ? tile_key(t) : 0;  // the keys' place matters to their distance only
    return x;
  }
  __device__ void bits(const Row& row, const Segment&, int, uint32_t (&b)[4]) const { assemble_bits<4>(row.nb, b); }
  __device__ void lower(const Row& row, const Tile& t, uint32_t (&sr)[4][32], float c, float slope) const {
    const int rel = row.pos - t.j0;
    lower_by_distance(sr, c, slope, static_cast<float>(rel), __all_sync(0xffffffffu, rel >= 127));
  }
  __device__ bool whole(const Segment&) const { return true; }
  __device__ size_t out_row(const Row& row) const { return static_cast<size_t>(bh) * p.L + row.i; }
  __device__ float* partial_o(const Segment&, int) const { return nullptr; }
  __device__ void put_stats(const Segment&, int, float, float) const {}
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
  constexpr int ST = D == 128 ? 3 : 4;
  switch (mode_of(a.scale, a.softcap, a.slopes != nullptr)) {
    case MODE_PLAIN: return launch_scored<FormatSource, D, BF16, MODE_PLAIN, ST>(mq, mk, mv, p, grid, s);
    case MODE_CAP: return launch_scored<FormatSource, D, BF16, MODE_CAP, ST>(mq, mk, mv, p, grid, s);
    default: return launch_scored<FormatSource, D, BF16, MODE_DISTANCE, ST>(mq, mk, mv, p, grid, s);
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
