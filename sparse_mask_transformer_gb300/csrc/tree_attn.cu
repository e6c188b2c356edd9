// Attention of drafted tokens over a K/V cache (stof_tree_attn_fwd).
//
// A request's rows for one K/V head are its group's heads times its drafted
// tokens, contiguous in Q: row r = head-in-group * T + t, in tiles of 128.
// Bound by memory while a K/V head has up to a few hundred rows: every K and V
// row has to be read once (4 d bytes), and 128 rows cost the tensor cores
// half of the time that 128 keys take to arrive.  So the work is cut by keys:
// all (request, K/V head) runs of key tiles in order, each with kItemCost
// more for its start and end, are one long line, cut into equal shares (the
// lengths are read on the device, so the shares follow them).  The row tiles
// of a K/V head, up to kRowGroup of them, go along a share together, each
// with a worker of its own (two workers per SM, scored_kernel.cuh): their
// neighbours' requests for the same K/V tiles are then L2 hits.  (One row tile
// after the other read the cache once per row tile: 524 us instead of 337
// for 512 rows per K/V head over 2 x 131000 keys.)  A head whose tiles lie in
// one share is finished there; the others leave partial rows (O relative to
// the rows' max, max and sum) in the workspace, which combine_kernel merges in
// the order of the keys: the result does not depend on timing.  A worker has at most one item that began before its
// share and one that goes on after it: two slots.
#include <cmath>

#include "scored_kernel.cuh"

namespace stof {
namespace {

using namespace scored;

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
  static constexpr bool kClearsV = true, kSplit = false;
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
  static __device__ bool begin_row(const Params& p, Row& row, const Segment<Item>& seg, int r) {
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
  static __device__ bool whole(const Item& x) { return x.whole; }
  // A segment that begins its item goes on in a later share: slot 2 w + 1 of
  // worker w; one that does not: slot 2 w.
  static __device__ size_t slot_row(const Params& p, const Item& x, int g, int r) {
    return static_cast<size_t>(2 * (2 * blockIdx.x + g) + (x.t0 == 0 ? 1 : 0)) * p.slot_rows + r;
  }
  static __device__ float* partial_o(const Params& p, const Item& x, int g, int r, int d) {
    return p.slots + slot_row(p, x, g, r) * d;
  }
  static __device__ void put_stats(const Params& p, const Item& x, int g, int r, float m, float l) {
    p.stats[slot_row(p, x, g, r)] = make_float2(m, l);
  }
};

// A row is merged by four warps while the call has fewer rows than 128 times
// the shares that a run lies in, else by one: many parts take one warp long,
// many rows keep the SMs busy without more warps.  d = 128, one warp and four:
// 32 rows of 38 shares each 40.0 and 31.8 us (the whole call), 1024 rows of 38
// shares 46.9 and 40.7, 640 of 7.6 36.6 and 35.3; 1024 of 4.8 30.6 and 31.3,
// 4096 of 9.5 73.5 and 78.0, 16384 of 1.2 61.5 and 84.6.
constexpr int kRowsPerShare = 128;

// Merges the partial rows of the runs that lie in several shares:
// O = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i.  WPR warps per query row,
// warp x of a row the parts x, x + WPR, ..., eight of them in flight; four
// rows of one warp, or one row of four, a block.  (Launched while the main
// kernel still runs, it begins when that has ended.)
template <int D, bool BF16, int WPR>
__global__ void __launch_bounds__(128) combine_kernel(const __grid_constant__ TreeParams p) {
  constexpr int E = D / 32, kBatch = 8;
  __shared__ float s_o[4][D], s_m[4], s_l[4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % WPR;
  const int per = p.Hkv * p.row_tiles;
  const int b = static_cast<int>(blockIdx.x) / per, item = static_cast<int>(blockIdx.x) - b * per;
  const int hk = item / p.row_tiles, rt = item - hk * p.row_tiles, group = rt / p.row_group;
  if (b == p.B) {  // the last blocks: the call's error bits
    if (blockIdx.y) return;
    dependents_wait();
    int bits = 0;
    for (int c = threadIdx.x; c < kTreeCtas; c += blockDim.x) bits |= __ldcg(p.status + c);
    const int late = __syncthreads_or(bits & STOF_DEVERR_PIPE_TIMEOUT), bad = __syncthreads_or(bits & STOF_DEVERR_BAD_LENGTH);
    if (threadIdx.x == 0) *p.word = (late ? STOF_DEVERR_PIPE_TIMEOUT : 0) | (bad ? STOF_DEVERR_BAD_LENGTH : 0);
    return;
  }
  const int r = static_cast<int>(blockIdx.y) * (4 / WPR) + warp / WPR, rr = rt * 128 + r, gq = rr / p.T, t = rr - gq * p.T;
  dependents_wait();
  int ctx, count;
  if (!request(p, b, ctx, count)) return;
  const int all = __ldcg(p.line + p.B), line = __ldcg(p.line + b);
  const int len = tiles_of(p, ctx + count) + kItemCost, share = share_of(p, all);
  const int at = line + (hk * p.row_groups + group) * len;
  const int w0 = (at + kItemCost) / share, w1 = (at + len - 1) / share;  // shares of its first and last tile
  if (w0 == w1) return;                                                  // finished by its one worker
  if (r >= p.slot_rows || rr >= p.rows || t >= count) return;            // (one row: the whole block)
  // the first share's part is its worker's last segment, the others' their first
  auto slot = [&](int w) {
    const int worker = w * p.row_group + rt - group * p.row_group;
    return static_cast<size_t>(2 * worker + (w == w0 ? 1 : 0)) * p.slot_rows + r;
  };
  float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 1
  for (int i0 = w0 + part; i0 <= w1; i0 += WPR * kBatch) {
    float2 st[kBatch];
    float x[kBatch][E];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int w = i0 + i * WPR;
      st[i] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < E; ++e) x[i][e] = 0.f;
      if (w <= w1) {
        st[i] = __ldcg(p.stats + slot(w));
        const float* src = p.slots + slot(w) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 y = __ldcg(reinterpret_cast<const float2*>(src + e));
          x[i][e] = y.x;
          x[i][e + 1] = y.y;
        }
      }
    }
    float mn = m;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) mn = fmaxf(mn, st[i].x);
    const float ref = mn == -INFINITY ? 0.f : mn, a = ex2(m - ref);
    l *= a;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= a;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float w = ex2(st[i].x - ref);
      l = fmaf(w, st[i].y, l);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(w, x[i][e], o[e]);
    }
    m = mn;
  }
  uint32_t* out = static_cast<uint32_t*>(p.o) +
                  ((((static_cast<size_t>(b) * p.H + hk * p.group + gq) * p.T + t) * D) >> 1);
  if constexpr (WPR == 1) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < E; e += 2) out[(lane * E + e) >> 1] = pack2<BF16>(o[e] * inv, o[e + 1] * inv);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
    if (lane == 0) {
      s_m[warp] = m;
      s_l[warp] = l;
    }
    __syncthreads();
    float mm = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) mm = fmaxf(mm, s_m[w]);
    if (mm == -INFINITY) mm = 0.f;
    const int c = 2 * threadIdx.x;  // two columns a thread
    if (c >= D) return;
    float y0 = 0.f, y1 = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float a = ex2(s_m[w] - mm);
      sum = fmaf(a, s_l[w], sum);
      y0 = fmaf(a, s_o[w][c], y0);
      y1 = fmaf(a, s_o[w][c + 1], y1);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    out[c >> 1] = pack2<BF16>(y0 * inv, y1 * inv);
  }
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
constexpr size_t kErrorBytes = 256 + (kTreeCtas * sizeof(int) + 255) / 256 * 256;  // the error bits: the call's, the CTAs'

// Copies of Q's rows in a tile, each with a part of its keys: four or two at
// d = 64 where the rows leave room for them.  7 rows per K/V head, 32 requests:
// 26 to 30 us with four copies, 50 with one; two and one: 64 rows, 32 requests of
// 1500, cap and slopes 51.2 and 74.8, cap 44.5 and 57.4, plain 43.9 and 44.6, 56
// rows, 2 requests of 2200, plain 11.9 and 11.5.  At d = 128 a tile is 64 keys
// and one copy's code fits the instruction cache; two (with two K stages) and
// one, 64 rows, 8 requests of 4000: plain 36.3 and 34.6, cap and slopes 36.3
// and 37.5; 4 rows, one request 14.5 and 13.5.
inline int copies_of(int d, long long rows) { return d != 64 || 2 * rows > kBM ? 1 : (4 * rows > kBM ? 2 : 4); }

template <int D, bool BF16, int MODE>
stof_status launch_mode(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const TreeParams& p,
                        cudaStream_t s) {
  if constexpr (D == 64) {
    if (p.copies == 4) return launch_scored<CacheSource, D, BF16, MODE, 4>(mq, mk, mv, p, kTreeCtas, s);
    if (p.copies == 2) return launch_scored<CacheSource, D, BF16, MODE, 2>(mq, mk, mv, p, kTreeCtas, s);
  }
  return launch_scored<CacheSource, D, BF16, MODE, 1>(mq, mk, mv, p, kTreeCtas, s);
}

template <int D, bool BF16>
stof_status launch_tree(const void* q, const void* k, const void* v, const TreeParams& p, int mode, cudaStream_t s) {
  CUtensorMap mq, mk, mv;
  const uint64_t planes = static_cast<uint64_t>(p.B) * p.Hkv;
  if (!make_bw_map(&mq, q, planes, p.rows, D, kBM / p.copies, BF16) ||
      !make_bw_map(&mk, k, planes, p.cap, D, Shape<D>::BN, BF16) || !make_bw_map(&mv, v, planes, p.cap, D, Shape<D>::BN, BF16))
    return STOF_ERR_CUDA;
  stof_status st;
  switch (mode) {
    case MODE_PLAIN: st = launch_mode<D, BF16, MODE_PLAIN>(mq, mk, mv, p, s); break;
    case MODE_CAP: st = launch_mode<D, BF16, MODE_CAP>(mq, mk, mv, p, s); break;
    default: st = launch_mode<D, BF16, MODE_DISTANCE>(mq, mk, mv, p, s); break;
  }
  if (st != STOF_OK) return st;
  const bool one = planes * p.rows * planes * p.row_groups >= static_cast<uint64_t>(kRowsPerShare) * p.shares;
  const dim3 grid(static_cast<unsigned>(planes * p.row_tiles + 1), static_cast<unsigned>(one ? (p.slot_rows + 3) / 4 : p.slot_rows));
  const cudaError_t e = launch_early(one ? combine_kernel<D, BF16, 1> : combine_kernel<D, BF16, 4>, grid, 128, 0, s, p);
  return record_cuda(e) == cudaSuccess ? STOF_OK : STOF_ERR_CUDA;
}

}  // namespace
}  // namespace stof

using namespace stof;

extern "C" size_t stof_tree_attn_workspace_bytes(int B, int H, int Hkv, int T, int d) {
  if (B < 1 || H < 1 || Hkv < 1 || H % Hkv || T < 1 || T > STOF_TREE_MAX_TOKENS || (d != 64 && d != 128)) return 0;
  const long long rows = static_cast<long long>(H / Hkv) * T;
  const size_t slots = static_cast<size_t>(2 * kWorkers) * (rows < 128 ? rows : 128);
  return kErrorBytes + up256(slots * d * sizeof(float)) + up256(slots * sizeof(float2)) + (static_cast<size_t>(B) + 1) * sizeof(int32_t);
}

extern "C" stof_status stof_tree_attn_fwd(const void* q, const void* k, const void* v, stof_dtype dt, int B, int H,
                                          int Hkv, int T, int d, int cap, const int32_t* lens, const int32_t* counts,
                                          const uint32_t* tree, const int32_t* positions, float scale,
                                          const stof_score* score, void* o, void* workspace, size_t ws_bytes,
                                          int64_t* device_error, void* stream) {
  if (!q || !k || !v || !o || !lens || !workspace) return STOF_ERR_INVALID_ARG;
  if (dt != STOF_F16 && dt != STOF_BF16) return STOF_ERR_DTYPE;
  if (B < 1 || H < 1 || Hkv < 1 || T < 1 || d < 1 || cap < 1 || !std::isfinite(scale)) return STOF_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return STOF_ERR_UNSUPPORTED;
  if (H % Hkv || T > STOF_TREE_MAX_TOKENS) return STOF_ERR_SHAPE;
  const long long rows = static_cast<long long>(H / Hkv) * T, row_tiles = (rows + 127) / 128;
  // the line of the call's tiles and its query rows are counted in 32 bits
  if (static_cast<long long>(B) * H * T >= (1ll << 31) || static_cast<long long>(B) * Hkv >= (1ll << 31) ||
      static_cast<long double>(B) * Hkv * row_tiles * ((static_cast<long long>(cap) + 63) / 64 + kItemCost) >= 2147480000.0L)
    return STOF_ERR_SHAPE;
  if (score) {
    stof_score s = *score;
    s.q_start = 0;  // not read by this call
    const stof_status st = check_score(s, scale);
    if (st != STOF_OK) return st;
  }
  const uintptr_t wide = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
                         reinterpret_cast<uintptr_t>(o) | reinterpret_cast<uintptr_t>(workspace);
  const uintptr_t words = reinterpret_cast<uintptr_t>(lens) | reinterpret_cast<uintptr_t>(counts) |
                          reinterpret_cast<uintptr_t>(tree) | reinterpret_cast<uintptr_t>(positions);
  if (wide % 16 || words % 4 || reinterpret_cast<uintptr_t>(device_error) % 8) return STOF_ERR_ALIGNMENT;
  if (ws_bytes < stof_tree_attn_workspace_bytes(B, H, Hkv, T, d)) return STOF_ERR_WORKSPACE;
  const float softcap = score ? score->softcap : 0.f;
  TreeParams p;
  p.k = make_score_const(scale, softcap);
  p.slopes = score ? score->slopes : nullptr;
  p.o = o;
  p.err = device_error;
  p.H = H;
  p.group = H / Hkv;
  p.B = B;
  p.Hkv = Hkv;
  p.T = T;
  p.d = d;
  p.cap = cap;
  p.tile = d == 64 ? Shape<64>::BN : Shape<128>::BN;
  p.words = (T + 31) / 32;
  p.rows = static_cast<int>(rows);
  p.row_tiles = static_cast<int>(row_tiles);
  p.row_groups = static_cast<int>((row_tiles + kRowGroup - 1) / kRowGroup);
  p.row_group = (p.row_tiles + p.row_groups - 1) / p.row_groups;
  p.shares = kWorkers / p.row_group;
  p.slot_rows = static_cast<int>(rows < 128 ? rows : 128);
  p.lens = lens;
  p.counts = counts;
  p.tree = tree;
  p.positions = p.slopes ? positions : nullptr;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.word = reinterpret_cast<long long*>(ws);
  p.status = reinterpret_cast<int*>(ws + 256);
  ws += kErrorBytes;
  p.slots = reinterpret_cast<float*>(ws);
  const size_t slots = static_cast<size_t>(2 * kWorkers) * p.slot_rows;
  ws += up256(slots * d * sizeof(float));
  p.stats = reinterpret_cast<float2*>(ws);
  ws += up256(slots * sizeof(float2));
  p.line = reinterpret_cast<int32_t*>(ws);
  const int mode = mode_of(scale, softcap, p.slopes != nullptr);
  p.copies = copies_of(d, rows);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d == 64)
    return dt == STOF_BF16 ? launch_tree<64, true>(q, k, v, p, mode, s) : launch_tree<64, false>(q, k, v, p, mode, s);
  return dt == STOF_BF16 ? launch_tree<128, true>(q, k, v, p, mode, s) : launch_tree<128, false>(q, k, v, p, mode, s);
}
