// The tiles of requests' K/V caches as a source of scored_kernel.cuh
// (stof_tree_attn_fwd, and the requests' own rows of stof_prefix_attn_fwd):
// how the work is cut is said in tree_attn.cu.
#pragma once
#include "scored_kernel.cuh"

namespace stof {
namespace scored {

constexpr int kTreeCtas = 152;             // one CTA per SM
constexpr int kWorkers = 2 * kTreeCtas;
constexpr int kItemCost = 2;               // a run's start and end, in tiles
constexpr int kRowGroup = 8;               // row tiles that go along the line together, at most

struct TreeParams : CommonParams {
  int B, Hkv, T, d, cap, words;
  int tile;        // keys per tile: 128 (d = 64) or 64 (d = 128)
  int rows;        // group * T: query rows per K/V head
  int row_tiles;   // ceil(rows / 128)
  int row_group;   // row tiles per share; row_groups = ceil(row_tiles / row_group)
  int row_groups;
  int shares;      // kWorkers / row_group
  int slot_rows;   // rows of a partial result: min(rows, 128)
  const int32_t* lens;
  const int32_t* counts;
  const uint32_t* tree;
  const int32_t* positions;
  int copies;      // copies of Q's rows in a tile
  long long* word;  // the call's error bits, put together by combine_kernel
  int* status;      // [kTreeCtas] the CTAs' error bits
  float* slots;    // [2 kWorkers][slot_rows][d] partial O
  float2* stats;   // [2 kWorkers][slot_rows] (max, sum)
  int32_t* line;   // [B + 1] place of each request on the line, its length
};

// Committed and drafted tokens of request b; false for a request that breaks
// the bounds or has no drafted token.
__device__ __forceinline__ bool request(const TreeParams& p, int b, int& ctx, int& count) {
  ctx = __ldg(p.lens + b);
  count = p.counts ? __ldg(p.counts + b) : p.T;
  return ctx >= 0 && count >= 1 && count <= p.T && ctx <= p.cap - count;
}
__device__ __forceinline__ int tiles_of(const TreeParams& p, int keys) {
  return p.tile == 128 ? (keys + 127) >> 7 : (keys + 63) >> 6;
}
// Length of a request's items on the line (0: none).
__device__ __forceinline__ int item_length(const TreeParams& p, int b) {
  int ctx, count;
  return request(p, b, ctx, count) ? tiles_of(p, ctx + count) + kItemCost : 0;
}

// Exclusive prefix of v over the block's threads and the total (all threads
// call it; `sums` has a word per warp).
__device__ __forceinline__ int block_prefix(int v, int* sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  __syncthreads();  // sums may still be read from the previous call
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  int before = 0;
  total = 0;
  for (int w = 0; w < warps; ++w) {
    if (w < warp) before += sums[w];
    total += sums[w];
  }
  return before + x - v;
}

// Length of a share of a line of this length.
__device__ __forceinline__ int share_of(const TreeParams& p, int all) { return max(1, (all + p.shares - 1) / p.shares); }

struct CacheSource {
  using Params = TreeParams;
  static constexpr bool kClearsV = true, kSplit = false, kTwoPlaces = false;
  struct Item {
    int b, hk;         // request, K/V head
    int ctx, count;    // committed and drafted tokens
    int t0;            // first tile of the segment
    int tile;          // keys per tile
    bool whole;        // the segment is the whole item
  };
  struct Shared {
    int sums[kThreads / 32];
    int begin[2], end[2];  // the workers' shares
    int b[2], base[2];     // request that holds a share's begin, its place on the line
    int bad;               // CTA 0: a request breaks the bounds
  };
  struct Loads {};
  template <bool>
  struct Lane {  // what a softmax thread knows of its row in every tile
    int r;
    __device__ Lane(const Params&, const Shared&, int, int row) : r(row) {}
  };
  struct Row {
    int head, t, pos;
    size_t out;
    const uint32_t* tree;  // the row's bits, or null
  };

  static __device__ void init(Shared& s) { s.bad = 0; }
  // Finds the requests at the workers' begins; CTA 0 reports bad requests and
  // leaves the line for combine_kernel.
  static __device__ void prologue(const Params& p, Shared& s) {
    dependents_launch();  // combine_kernel may be set up
    const int per = p.Hkv * p.row_groups;
    int all = 0, v = 0, at = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
      const int b = b0 + threadIdx.x;
      int total;
      v = b < p.B ? item_length(p, b) * per : 0;
      at = all + block_prefix(v, s.sums, total);
      if (blockIdx.x == 0 && b < p.B) {
        p.line[b] = at;
        int c, n;
        if (v == 0 && !request(p, b, c, n) && !(n == 0 && c >= 0 && c <= p.cap)) {
          s.bad = 1;
          if (p.err) raise_error(p.err, STOF_DEVERR_BAD_LENGTH);
        }
      }
      all += total;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) p.line[p.B] = all;
    const int share = share_of(p, all);
    int begin[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int x = (2 * static_cast<int>(blockIdx.x) + g) / p.row_group;  // the worker's share
      begin[g] = x < p.shares ? min(x * share, all) : all;
      if (threadIdx.x == 0) {
        s.begin[g] = begin[g];
        s.end[g] = begin[g] + min(share, all - begin[g]);
      }
    }
    int base = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
      if (p.B > kThreads) {  // else v and at are those of the one round above
        int total;
        v = b0 + static_cast<int>(threadIdx.x) < p.B ? item_length(p, b0 + threadIdx.x) * per : 0;
        at = base + block_prefix(v, s.sums, total);
        base += total;
      }
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (at <= begin[g] && begin[g] < at + v) {
          s.b[g] = b0 + threadIdx.x;
          s.base[g] = at;
        }
      }
    }
  }
  // The CTA's error bits, at its end (one thread).  A word per CTA and no
  // atomic: none has to be cleared before the call.
  static __device__ void finish(const Params& p, const Shared& s, const volatile int* abort_flag) {
    p.status[blockIdx.x] = (*abort_flag ? STOF_DEVERR_PIPE_TIMEOUT : 0) | (s.bad ? STOF_DEVERR_BAD_LENGTH : 0);
  }
  // A worker's place on the line.
  struct Lead {
    int w, end;                      // place, end of the share
    int row;                         // the worker's row tile within a group
    int b = 0, base = 0, len = 0;    // request, its place, length of its items
    int ctx = 0, count = 0;
    __device__ Lead(const Params& p, Shared& s, int g) {
      w = s.begin[g];
      end = s.end[g];
      row = (2 * static_cast<int>(blockIdx.x) + g) % p.row_group;
      if (w < end) {
        b = s.b[g];
        base = s.base[g];
        load(p);
      }
    }
    __device__ void load(const Params& p) { len = request(p, b, ctx, count) ? tiles_of(p, ctx + count) + kItemCost : 0; }
    __device__ Next next(const Params& p, Shared&, const volatile int*, Segment<Item>& seg) {
      const int per = p.Hkv * p.row_groups;
#pragma unroll 1
      while (w < end) {
#pragma unroll 1
        while (w >= base + len * per) {  // on to the next request on the line
          base += len * per;
          ++b;
          load(p);
        }
        const int off = w - base, item = off / len, at = off - item * len;
        const int to = min(end - base - item * len, len);  // the share's part of the item: [at, to)
        w += to - at;
        const int t0 = max(0, at - kItemCost), t1 = max(0, to - kItemCost);
        const int hk = item / p.row_groups, rt = (item - hk * p.row_groups) * p.row_group + row;
        // the share ends before the run's first tile, or the last group has no such row tile
        if (t1 <= t0 || rt >= p.row_tiles) continue;
        seg.q_plane = seg.kv_plane = b * p.Hkv + hk;
        seg.q_row = rt * 128;
        seg.n = t1 - t0;
        seg.item = Item{b, hk, ctx, count, t0, p.tile, t1 - t0 == len - kItemCost};
        return Next::segment;
      }
      return Next::none;
    }
    __device__ void drain(Shared&) {}
  };

  static __device__ int tile_key(const Params&, const Item& x, int t) { return (x.t0 + t) * x.tile; }
  static __device__ int tile_end(const Item& x, int t) { return min(x.tile, x.ctx + x.count - (x.t0 + t) * x.tile); }
  template <bool KEEP>
  static __device__ bool begin_row(const Params& p, Row& row, const Loads&, const Segment<Item>& seg, const Lane<KEEP>& lane) {
    const int r = lane.r;
    const Item& x = seg.item;
    const int rr = seg.q_row + r, gq = rr / p.T;
    row.t = rr - gq * p.T;
    row.head = x.hk * p.group + gq;
    const bool live = rr < p.rows && row.t < x.count;
    const size_t token = static_cast<size_t>(x.b) * p.T + row.t;
    row.pos = live && p.positions ? __ldg(p.positions + token) : x.ctx + row.t;
    row.out = (static_cast<size_t>(x.b) * p.H + row.head) * p.T + row.t;
    row.tree = live && p.tree ? p.tree + token * p.words : nullptr;
    return live;
  }
  template <int BN>
  static __device__ void prefetch(const Params&, Row&, const Item&, int) {}
  static __device__ bool partial(const Item& x, int t) { return (x.t0 + t + 1) * x.tile > x.ctx; }  // it has drafted keys
  // Bits of drafted tokens 32 x .. 32 x + 31 that the row sees.
  static __device__ uint32_t seen(const Params& p, const Row& row, const Item& x, int word) {
    if (32 * word >= x.count) return 0u;
    uint32_t bits;
    if (p.tree)
      bits = row.tree ? __ldg(row.tree + word) : 0u;
    else
      bits = row.t >= 32 * word + 31 ? ~0u : (row.t < 32 * word ? 0u : (2u << (row.t - 32 * word)) - 1u);
    const int left = x.count - 32 * word;
    return left >= 32 ? bits : bits & ((1u << left) - 1u);
  }
  template <int BN, int CHUNKS>
  static __device__ void bits(const Params& p, const Row& row, const Item& x, int t, int first, uint32_t (&out)[CHUNKS]) {
#pragma unroll
    for (int cc = 0; cc < CHUNKS; ++cc) {
      const int u0 = (x.t0 + t) * BN + first + 32 * cc - x.ctx;  // drafted token of the chunk's first key
      if (u0 <= -32)
        out[cc] = ~0u;
      else if (u0 < 0)
        out[cc] = ((1u << -u0) - 1u) | (seen(p, row, x, 0) << -u0);
      else
        out[cc] = __funnelshift_r(seen(p, row, x, u0 >> 5), seen(p, row, x, (u0 >> 5) + 1), u0 & 31);
    }
  }
  static __device__ float slope(const Params& p, const Row& row) { return __ldg(p.slopes + row.head); }
  // Distance of the row's nearest (far: farthest) visible key.  Without
  // positions a bound on it does as well: it is 1024 away from it at most.
  static __device__ uint32_t reference(const Params& p, const Row& row, const Item& x, bool far) {
    if (!p.positions) return far ? max(row.pos, x.count) : 0;
    if (!far && seen(p, row, x, row.t >> 5) >> (row.t & 31) & 1u) return 0u;  // it sees itself
    uint32_t best = far ? 0u : ~0u;
    if (x.ctx > 0) best = reference_distance(row.pos, x.ctx - 1, far);
#pragma unroll 1
    for (int word = 0; 32 * word < x.count; ++word) {
#pragma unroll 1
      for (uint32_t bits = seen(p, row, x, word); bits; bits &= bits - 1) {
        const int u = 32 * word + __ffs(bits) - 1;
        const uint32_t d = __sad(row.pos, __ldg(p.positions + static_cast<size_t>(x.b) * p.T + u), 0u);
        best = far ? max(best, d) : min(best, d);
      }
    }
    return best;
  }
  template <int BN, int CHUNKS>
  static __device__ void lower(const Params& p, const Row& row, const Item& x, int t, int j0, uint32_t (&sr)[CHUNKS][32],
                               float c, float slope, uint32_t base) {
    if (p.positions && partial(x, t)) {
      int at[CHUNKS];  // position of key 32 i + lane of the tile
#pragma unroll
      for (int i = 0; i < CHUNKS; ++i) {
        const int key = j0 + 32 * i + static_cast<int>(threadIdx.x & 31), u = key - x.ctx;
        at[i] = u < 0 ? key : (u < x.count ? __ldg(p.positions + static_cast<size_t>(x.b) * p.T + u) : 0);
      }
      lower_by_positions(sr, c, slope, row.pos, base, at);
    } else {
      lower_by_distance(sr, c, slope, row.pos, j0, base);
    }
  }
  static __device__ bool whole(const Params&, const Item& x) { return x.whole; }
  // A segment that begins its item goes on in a later share: slot 2 w + 1 of
  // worker w; one that does not: slot 2 w.
  static __device__ size_t slot_row(const Params& p, const Item& x, int g, int r) {
    return static_cast<size_t>(2 * (2 * blockIdx.x + g) + (x.t0 == 0 ? 1 : 0)) * p.slot_rows + r;
  }
  static __device__ float* partial_o(const Params& p, const Item& x, const Row&, int g, int r, int d) {
    return p.slots + slot_row(p, x, g, r) * d;
  }
  static __device__ void put_stats(const Params& p, const Item& x, const Row&, int g, int r, float m, float l) {
    p.stats[slot_row(p, x, g, r)] = make_float2(m, l);
  }
};

// Copies of Q's rows in a tile, each with a part of its keys: four or two at
// d = 64 where the rows leave room for them.  7 rows per K/V head, 32 requests:
// 26 to 30 us with four copies, 50 with one; two and one: 64 rows, 32 requests of
// 1500, cap and slopes 51.2 and 74.8, cap 44.5 and 57.4, plain 43.9 and 44.6, 56
// rows, 2 requests of 2200, plain 11.9 and 11.5.  At d = 128 a tile is 64 keys
// and one copy's code fits the instruction cache; two (with two K stages) and
// one, 64 rows, 8 requests of 4000: plain 36.3 and 34.6, cap and slopes 36.3
// and 37.5; 4 rows, one request 14.5 and 13.5.
inline int copies_of(int d, long long rows) { return d != 64 || 2 * rows > kBM ? 1 : (4 * rows > kBM ? 2 : 4); }

constexpr size_t kErrorBytes = 256 + (kTreeCtas * sizeof(int) + 255) / 256 * 256;  // the error bits: the call's, the CTAs'
inline size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace scored
}  // namespace stof
