// Attention over a prefix that groups of requests share and over the requests'
// own caches (stof_prefix_attn_fwd).
//
// A softmax over two sets of keys is that of each set, merged: with (m, l, O)
// the max, the sum and the unnormalised output of a set,
//   O = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i,  m = max m_i.
// So the prefix is read for all requests of its group at once: their query rows
// for one K/V head (requests times heads of a group times tokens) are the rows
// of its tiles, as many requests to a tile of 128 rows as fit, and a K or V row
// of the prefix is read once per tile instead of once per request.  A
// request's own rows are those of stof_tree_attn_fwd().
//
// Bound by memory while a prefix's K/V head has up to some 128 rows (a K and a V
// row, 4 d bytes, are then read once), by the tensor cores' and the softmax's
// work above that; calls of a few tiles by launch, start and merge.
//
// Both are cut by keys (tree_attn.cu): the (prefix, K/V head) runs of key
// tiles, row tiles side by side, are one line, the (request, K/V head) runs
// another, and the workers are divided between the two lines so that both end
// at the same time; each line is cut into equal shares.  What a worker finds
// of a row is a part: in the worker's own two slots if the run goes on in
// another share, in a buffer of the rows if it does not; merge_kernel puts a
// row's parts together in a fixed order.  (Runs that are all a row sees, without
// own rows, could be finished by their worker: the code for it, in the kernel of
// every call, cost 7 to 10% where runs are short, d = 128, and gained nothing.)
// With few rows at d = 64 the copies of the tile's rows (scored_kernel.cuh) are
// parts too: merging them inside the kernel cost 1 us at every run's end (8
// prefixes of 16 requests, caps and slopes: 61.6 us instead of 50.2 without).
// An SM's two workers are numbered far apart, so that one of them reads
// prefixes and the other own rows where both lines are long: 64 requests of a
// 16384-row prefix 81.6 -> 74.8 us.
//
// Measured (a call among others; of the memory's copy rate, of the bf16 rate):
// 64 requests with 100 to 1500 rows of their own behind one prefix of 16384, 32
// heads of 128 on 8: 59.9 us, 70%, the main kernel 53 of them, the first tile's
// arrival 4.2; 8 prefixes of 16 requests with cap and slopes, 12 heads of 64, 50.8
// us, 56%; 16 requests of up to 16 tokens behind 131072 rows 433 to 442 us, 57%; 4
// beams of 24 sources, 16 heads of 64, 24.7 us, 50%.
#include <cmath>

#include "cache_source.cuh"

namespace stof {
namespace {

using namespace scored;

struct PrefixParams : TreeParams {
  CUtensorMap own_q, own_k, own_v;  // boxes of one request's rows; the requests' own caches
  int NP, n, pcap;                  // prefixes, requests of each, rows of a prefix cache
  int nb;                           // requests in a row tile of a prefix
  int per_request;                  // row tiles of a request there (nb = 1)
  int fill, own_fill;               // rows of a tile: of a prefix's, of a request's
  int prow_tiles, prow_group, prow_groups;  // as row_tiles, ..., of a prefix
  float per_row_group, per_prow_group;      // 1 / row_group, 1 / prow_group
  const int32_t* plens;
  int32_t* pline;                   // [NP], as line [B]: places of the items on their lines
  // [kTreeCtas] first worker of the requests' line; share lengths of the prefixes' line, of the requests'; -.  Every
  // CTA leaves them: the warps of merge_kernel, each of which reads them first, would wait 1 to 3 us for one place
  int4* meta;
  // behind the workers' slots: [2][copies][B H T] parts of runs that lie in one share, of prefixes and of requests
  int64_t parts;                    // their first row
  int64_t out_rows;                 // B H T
};

// Whether a prefix's rows, a request's committed and drafted tokens, are what
// the call takes.
__device__ __forceinline__ bool prefix_ok(const PrefixParams& p, int plen) { return plen >= 0 && plen <= p.pcap; }
__device__ __forceinline__ bool request_ok(const PrefixParams& p, int ctx, int count) {
  return ctx >= 0 && count >= 1 && count <= p.T && (!p.lens || ctx <= p.cap - count);
}
struct Lengths {
  int plen, ctx, count;
};
// Of request b, three loads at once.
__device__ __forceinline__ Lengths lengths_of(const PrefixParams& p, int b) {
  Lengths x;
  x.plen = __ldg(p.plens + static_cast<unsigned>(b) / static_cast<unsigned>(p.n));
  x.ctx = p.lens ? __ldg(p.lens + b) : 0;
  x.count = p.counts ? __ldg(p.counts + b) : p.T;
  return x;
}
// Length of a run of key tiles on its line (0: none).
__device__ __forceinline__ int prefix_run(const PrefixParams& p, int plen) {
  return prefix_ok(p, plen) && plen > 0 ? tiles_of(p, plen) + kItemCost : 0;
}
__device__ __forceinline__ int request_run(const PrefixParams& p, const Lengths& x) {
  return p.lens && prefix_ok(p, x.plen) && request_ok(p, x.ctx, x.count) ? tiles_of(p, x.ctx + x.count) + kItemCost : 0;
}
// a / b of small numbers (a < 2^15), per_b = 1 / b
__device__ __forceinline__ int small_div(int a, float per_b) { return __float2int_rd((a + 0.5f) * per_b); }
__device__ __forceinline__ int share_length(int all, int shares) { return max(1, (all + shares - 1) / max(1, shares)); }

// Shares of the two lines, of lengths lp and lo: as many workers for each as
// bring the later end forward.
__device__ __forceinline__ void divide(const PrefixParams& p, int lp, int lo, int& sp, int& so) {
  sp = lp > 0 ? small_div(kWorkers, p.per_prow_group) : 0;
  if (lp > 0 && lo > 0) {
    const float wp = static_cast<float>(lp) * p.prow_group, wo = static_cast<float>(lo) * p.row_group;
    const int most = small_div(kWorkers - p.row_group, p.per_prow_group);
    sp = max(1, min(most, small_div(static_cast<int>(kWorkers * __fdividef(wp, wp + wo)), p.per_prow_group)));
    // one share more?
    const int y = small_div(kWorkers - sp * p.prow_group, p.per_row_group);
    const int y1 = small_div(kWorkers - (sp + 1) * p.prow_group, p.per_row_group);
    if (sp < most && fmaxf(__fdividef(lp, sp + 1), __fdividef(lo, y1)) < fmaxf(__fdividef(lp, sp), __fdividef(lo, y))) ++sp;
  }
  so = small_div(kWorkers - sp * p.prow_group, p.per_row_group);
}

struct PrefixSource : CacheSource {
  using Params = PrefixParams;
  static constexpr bool kTwoPlaces = true;
  struct Item : CacheSource::Item {  // of a prefix: ctx its rows, count 0, b its number
    bool prefix;
    int base;  // position of the item's first key: 0, or the prefix's rows
  };
  struct Shared {
    int2 sums[kThreads / 32];
    bool prefix[2];        // the workers' lines
    int row[2];            // their row tiles within a group
    int begin[2], end[2];  // and shares
    int i[2], base[2];     // the prefix or request that holds a share's begin, its place on the line
    Lengths lengths[2];    // its rows (of a prefix: plen)
    int bad;               // CTA 0: a length breaks the bounds
  };
  struct Loads {
    int ctx, count, position;
    uint32_t self;
    float slope;
  };
  struct Row : CacheSource::Row {
    int b, plen, ctx, count;  // the row's request
    uint32_t self;            // the word of its tree row that has its own bit
    float given_slope;
    bool listed;              // drafted keys' positions are read from the list (one value per warp)
  };

  static __device__ void init(Shared& s) { s.bad = 0; }

  // What a thread has of both lines: prefix i's rows, request i's lengths.
  struct Mine {
    int plen;
    Lengths x;
  };
  static __device__ Mine load_items(const Params& p, int i) {
    Mine m{0, Lengths{0, 0, 0}};
    if (i < p.NP) m.plen = __ldg(p.plens + i);
    if (i < p.B) m.x = lengths_of(p, i);
    return m;
  }
  // Lengths of their runs on the lines.
  static __device__ int2 item_lengths(const Params& p, const Mine& m, int i) {
    return make_int2(i < p.NP ? prefix_run(p, m.plen) * p.Hkv * p.prow_groups : 0,
                     i < p.B ? request_run(p, m.x) * p.Hkv * p.row_groups : 0);
  }
  // Reports lengths out of range.
  static __device__ void report(const Params& p, Shared& s, const Mine& m, int i) {
    const bool none = m.x.count == 0 && m.x.ctx >= 0 && (!p.lens || m.x.ctx <= p.cap);  // a request without tokens
    if (!prefix_ok(p, m.plen) || (i < p.B && !request_ok(p, m.x.ctx, m.x.count) && !none)) {
      s.bad = 1;
      if (p.err) raise_error(p.err, STOF_DEVERR_BAD_LENGTH);
    }
  }
  // Exclusive prefixes of v over the block's threads, and the totals.
  static __device__ int2 both_prefixes(int2 v, int2* sums, int2& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int2 x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x.x, off), z = __shfl_up_sync(0xffffffffu, x.y, off);
      if (lane >= off) {
        x.x += y;
        x.y += z;
      }
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int2 before = make_int2(0, 0);
    total = make_int2(0, 0);
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      const int2 y = sums[w];
      if (w < warp) before = make_int2(before.x + y.x, before.y + y.y);
      total = make_int2(total.x + y.x, total.y + y.y);
    }
    return make_int2(before.x + x.x - v.x, before.y + x.y - v.y);
  }
  // Both lines at once: a thread has prefix i and request i.
  template <class MEANWHILE>
  static __device__ void prologue(const Params& p, Shared& s, MEANWHILE meanwhile) {
    dependents_launch();  // merge_kernel may be set up
    const int items = max(p.NP, p.B);
    Mine m = load_items(p, threadIdx.x);
    meanwhile();
    int2 v, at, all = make_int2(0, 0);
#pragma unroll 1
    for (int i0 = 0; i0 < items; i0 += kThreads) {
      const int i = i0 + static_cast<int>(threadIdx.x);
      if (i0) {
        m = load_items(p, i);
        __syncthreads();  // the sums have been read
      }
      v = item_lengths(p, m, i);
      int2 total;
      at = both_prefixes(v, s.sums, total);
      at = make_int2(all.x + at.x, all.y + at.y);
      if (blockIdx.x == 0) {  // for merge_kernel
        if (i < p.NP) p.pline[i] = at.x;
        if (i < p.B) p.line[i] = at.y;
        report(p, s, m, i);  // behind a barrier: `bad` has been cleared by another warp
      }
      all = make_int2(all.x + total.x, all.y + total.y);
    }
    int shares[2];
    divide(p, all.x, all.y, shares[0], shares[1]);
    const int first_own = shares[0] * p.prow_group;  // workers before it are the prefixes'
    const int length[2] = {share_length(all.x, shares[0]), share_length(all.y, shares[1])};
    if (threadIdx.x == 0) p.meta[blockIdx.x] = make_int4(first_own, length[0], length[1], 0);
    bool mine[2];
    int begin[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int w = worker(g);
      mine[g] = w < first_own;
      const int in = mine[g] ? w : w - first_own, group = mine[g] ? p.prow_group : p.row_group;
      const int nth = small_div(in, mine[g] ? p.per_prow_group : p.per_row_group);
      const int line = mine[g] ? all.x : all.y, len = mine[g] ? length[0] : length[1];
      begin[g] = nth < (mine[g] ? shares[0] : shares[1]) ? min(nth * len, line) : line;
      if (threadIdx.x == 0) {
        s.prefix[g] = mine[g];
        s.row[g] = in - nth * group;
        s.begin[g] = begin[g];
        s.end[g] = begin[g] + min(len, line - begin[g]);
      }
    }
    int2 base = make_int2(0, 0);
#pragma unroll 1
    for (int i0 = 0; i0 < items; i0 += kThreads) {
      if (items > kThreads) {  // else v and at are those of the one round above
        m = load_items(p, i0 + threadIdx.x);
        v = item_lengths(p, m, i0 + threadIdx.x);
        __syncthreads();
        int2 total;
        at = both_prefixes(v, s.sums, total);
        at = make_int2(base.x + at.x, base.y + at.y);
        base = make_int2(base.x + total.x, base.y + total.y);
      }
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int from = mine[g] ? at.x : at.y, to = from + (mine[g] ? v.x : v.y);
        if (from <= begin[g] && begin[g] < to) {
          s.i[g] = i0 + threadIdx.x;
          s.base[g] = from;
          s.lengths[g] = mine[g] ? Lengths{m.plen, 0, 0} : m.x;
        }
      }
    }
  }
  static __device__ void finish(const Params& p, const Shared& s, const volatile int* abort_flag) {
    p.status[blockIdx.x] = (*abort_flag ? STOF_DEVERR_PIPE_TIMEOUT : 0) | (s.bad ? STOF_DEVERR_BAD_LENGTH : 0);
  }
  // A worker's number: an SM's two workers are far apart, so that where both
  // lines are long one of them reads a prefix, for many rows, and the other a
  // request's own rows, for few.
  static __device__ int worker(int g) { return g * kTreeCtas + static_cast<int>(blockIdx.x); }

  // A worker's place on its line.
  struct Lead {
    bool prefix;
    int w, end, row;
    int i = 0, base = 0, len = 0;  // prefix or request, its place, length of its runs
    int plen = 0, ctx = 0, count = 0;
    __device__ Lead(const Params& p, Shared& s, int g) : prefix(s.prefix[g]), w(s.begin[g]), end(s.end[g]), row(s.row[g]) {
      if (w < end) {
        i = s.i[g];
        base = s.base[g];
        take(p, s.lengths[g]);
      }
    }
    __device__ void take(const Params& p, const Lengths& x) {
      plen = prefix ? 0 : x.plen;
      ctx = prefix ? x.plen : x.ctx;
      count = x.count;
      len = prefix ? prefix_run(p, x.plen) : request_run(p, x);
    }
    __device__ Next next(const Params& p, Shared&, const volatile int*, Segment<Item>& seg) {
      const int row_tiles = prefix ? p.prow_tiles : p.row_tiles, row_group = prefix ? p.prow_group : p.row_group;
      const int row_groups = prefix ? p.prow_groups : p.row_groups, per = p.Hkv * row_groups;
#pragma unroll 1
      while (w < end) {
#pragma unroll 1
        while (w >= base + len * per) {  // on to the next item on the line
          base += len * per;
          ++i;
          take(p, prefix ? Lengths{__ldg(p.plens + i), 0, 0} : lengths_of(p, i));
        }
        const int off = w - base, item = off / len, at = off - item * len;
        const int to = min(end - base - item * len, len);  // the share's part of the run: [at, to)
        w += to - at;
        const int t0 = max(0, at - kItemCost), t1 = max(0, to - kItemCost);
        const int hk = row_groups == 1 ? item : item / row_groups, rt = (item - hk * row_groups) * row_group + row;
        if (t1 <= t0 || rt >= row_tiles) continue;
        if (prefix) {
          const int x = p.per_request == 1 ? rt : rt / p.per_request;
          seg.q_plane = i * p.n + (p.nb > 1 ? rt * p.nb : x);
          seg.q_row = p.nb > 1 ? 0 : (rt - x * p.per_request) * 128;
        } else {
          seg.q_plane = i;
          seg.q_row = rt * 128;
        }
        seg.kv_plane = i * p.Hkv + hk;
        seg.n = t1 - t0;
        seg.item.b = i;
        seg.item.hk = hk;
        seg.item.ctx = ctx;
        seg.item.count = count;
        seg.item.t0 = t0;
        seg.item.tile = p.tile;
        seg.item.whole = t1 - t0 == len - kItemCost;
        seg.item.prefix = prefix;
        seg.item.base = plen;
        return Next::segment;
      }
      return Next::none;
    }
    __device__ void drain(Shared&) {}
  };

  // A row's request and head in a tile that begins with a request's first row,
  // and its token.
  struct Place {
    int in, head, t;
    bool is;  // there is one
  };
  static __device__ Place place_in_tile(const Params& p, bool prefix, int r) {
    const int in = prefix && p.nb > 1 ? r / p.rows : 0, rr = r - in * p.rows, head = rr / p.T;
    return Place{in, head, rr - head * p.T, rr < p.rows && in < p.nb};
  }
  // What a softmax thread knows of its row r in every tile.  A worker has tiles
  // of one line only, so where runs are short (KEEP: with copies) the place is
  // found once: 8 prefixes of 16 requests, d = 64, 50.6 -> 48.9 us.  Kept where
  // runs are long (d = 128, 131072 rows) it costs registers: 403 -> 428 us.
  template <bool KEEP>
  struct Lane {
    int r;
    Place place;
    __device__ Lane(const Params& p, const Shared& s, int g, int row) : r(row), place{} {
      if (KEEP) place = place_in_tile(p, s.prefix[g], r);
    }
  };
  // Request, head and token of a segment's row; whether the call has such a
  // row, its lengths aside.
  template <bool KEEP>
  static __device__ bool place_row(const Params& p, const Segment<Item>& seg, const Lane<KEEP>& lane, int& b, int& head, int& t) {
    const Item& x = seg.item;
    Place y;
    if (seg.q_row > 0) {  // a later tile of a request's rows
      const int rr = seg.q_row + lane.r;
      y.in = 0;
      y.head = rr / p.T;
      y.t = rr - y.head * p.T;
      y.is = rr < p.rows;
    } else {
      y = KEEP ? lane.place : place_in_tile(p, x.prefix, lane.r);
    }
    b = seg.q_plane + y.in;
    head = x.hk * p.group + y.head;
    t = y.t;
    return y.is && (!x.prefix || b < (x.b + 1) * p.n);
  }
  // What is loaded for a row, all of it at once.
  template <bool KEEP>
  static __device__ void load_row(const Params& p, Loads& y, const Segment<Item>& seg, const Lane<KEEP>& lane) {
    const Item& x = seg.item;
    int b, head, t;
    place_row(p, seg, lane, b, head, t);
    b = min(b, p.B - 1);
    const size_t token = static_cast<size_t>(b) * p.T + t;
    y.ctx = x.ctx;
    y.count = x.count;
    if (x.prefix) {
      y.ctx = p.lens ? __ldg(p.lens + b) : 0;
      y.count = p.counts ? __ldg(p.counts + b) : p.T;
    }
    if (p.positions) {
      y.position = __ldg(p.positions + token);
      if (p.tree) y.self = __ldg(p.tree + token * p.words + (t >> 5));
    }
    if (p.slopes) y.slope = __ldg(p.slopes + min(head, p.H - 1));
  }
  template <bool KEEP>
  static __device__ bool begin_row(const Params& p, Row& row, const Loads& y, const Segment<Item>& seg, const Lane<KEEP>& lane) {
    const Item& x = seg.item;
    const bool live = place_row(p, seg, lane, row.b, row.head, row.t) && request_ok(p, y.ctx, y.count) && row.t < y.count;
    row.plen = live ? (x.prefix ? x.ctx : x.base) : 0;
    row.ctx = live ? y.ctx : 0;
    row.count = live ? y.count : 0;
    row.self = p.positions && p.tree ? y.self : ~0u;
    row.given_slope = y.slope;
    // one token at the place behind its request's rows needs no list
    row.listed = p.positions && __any_sync(0xffffffffu, live && !(y.count == 1 && y.position == row.plen + row.ctx));
    row.pos = p.positions ? y.position : row.plen + row.ctx + row.t;
    row.out = (static_cast<size_t>(row.b) * p.H + row.head) * p.T + row.t;
    row.tree = live && p.tree ? p.tree + (static_cast<size_t>(row.b) * p.T + row.t) * p.words : nullptr;
    return live;
  }
  static __device__ float slope(const Params&, const Row& row) { return row.given_slope; }
  // Distance of the nearest (far: farthest) key that the row sees, in the
  // prefix or of the request's own: the parts of a row have one reference.
  static __device__ uint32_t reference(const Params& p, const Row& row, const Item&, bool far) {
    if (!far && row.self >> (row.t & 31) & 1u) return 0u;  // it sees itself
    CacheSource::Item own;
    own.b = row.b;
    own.count = row.count;
    own.ctx = row.plen + row.ctx;  // rows 0 .. of the prefix and the request are positions 0 ..
    return CacheSource::reference(p, row, own, far);
  }
  template <int BN, int CHUNKS>
  static __device__ void lower(const Params& p, const Row& row, const Item& x, int t, int j0, uint32_t (&sr)[CHUNKS][32],
                               float c, float slope, uint32_t base) {
    if (row.listed && !x.prefix && partial(x, t)) {
      int at[CHUNKS];  // position of key 32 i + lane of the tile
#pragma unroll
      for (int i = 0; i < CHUNKS; ++i) {
        const int key = j0 + 32 * i + static_cast<int>(threadIdx.x & 31), u = key - x.ctx;
        at[i] = u < 0 ? x.base + key : (u < x.count ? __ldg(p.positions + static_cast<size_t>(x.b) * p.T + u) : 0);
      }
      lower_by_positions(sr, c, slope, row.pos, base, at);
    } else {
      lower_by_distance(sr, c, slope, row.pos, x.base + j0, base);
    }
  }
  // Parts of whole runs by the row of O; of others by the worker, as
  // CacheSource; those of the copies (r: the row of the tile) one after the other.
  static __device__ size_t slot_row(const Params& p, const Item& x, int g, int r) {
    return static_cast<size_t>(2 * worker(g) + (x.t0 == 0 ? 1 : 0)) * p.slot_rows + r;
  }
  static __device__ float* partial_o(const Params& p, const Item& x, const Row& row, int g, int r, int d) {
    return p.slots + part_row(p, x, row, g, r) * d;
  }
  static __device__ void put_stats(const Params& p, const Item& x, const Row& row, int g, int r, float m, float l) {
    p.stats[part_row(p, x, row, g, r)] = make_float2(m, l);
  }
  static __device__ size_t part_row(const Params& p, const Item& x, const Row& row, int g, int r) {
    return x.whole ? p.parts + ((x.prefix ? 0 : p.copies) + r * p.copies / kBM) * p.out_rows + row.out : slot_row(p, x, g, r);
  }
};

// Merges the parts of the rows, those of the prefix first.  WPR warps per row;
// a part takes D / 4 lanes, four columns each, so that a warp takes one (d =
// 128) or two (d = 64) parts at a time, kBatch times that in flight.  Four rows
// of one warp, or one row of four, a block.  (Launched while the main kernel
// still runs, it begins when that has ended.)
template <int D, bool BF16, int WPR>
__global__ void __launch_bounds__(128) merge_kernel(const __grid_constant__ PrefixParams p) {
  constexpr int kLanes = D / 4, kAtOnce = 32 / kLanes, kBatch = 8;
  __shared__ float4 s_o[4][kLanes];
  __shared__ float s_m[4], s_l[4];
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), part = warp % WPR;
  if (blockIdx.x == gridDim.x - 1) {  // the last block: the call's error bits
    dependents_wait();
    int bits = 0;
    for (int c = threadIdx.x; c < kTreeCtas; c += blockDim.x) bits |= __ldcg(p.status + c);
    const int late = __syncthreads_or(bits & STOF_DEVERR_PIPE_TIMEOUT), bad = __syncthreads_or(bits & STOF_DEVERR_BAD_LENGTH);
    if (threadIdx.x == 0) *p.word = (late ? STOF_DEVERR_PIPE_TIMEOUT : 0) | (bad ? STOF_DEVERR_BAD_LENGTH : 0);
    return;
  }
  const unsigned out = blockIdx.x * (4 / WPR) + warp / WPR;
  if (out >= p.out_rows) return;  // (one row: the whole block)
  const unsigned bh = out / p.T, b = bh / p.H, h = bh - b * p.H, hk = h / p.group;
  const int t = static_cast<int>(out - bh * p.T), rr = static_cast<int>(h - hk * p.group) * p.T + t;
  const Lengths x = lengths_of(p, b);
  if (!prefix_ok(p, x.plen) || !request_ok(p, x.ctx, x.count) || t >= x.count) return;
  // the row's tile of its prefix's run and place in it
  const unsigned np = b / p.n, in = b - np * p.n;
  int prt = p.nb > 1 ? in / p.nb : in * p.per_request + rr / 128;
  const int pr = p.nb > 1 ? (in - prt * p.nb) * p.rows + rr : rr % 128;
  const int lens[2] = {prefix_run(p, x.plen), request_run(p, x)};
  dependents_wait();
  // (through the L1 cache, which nothing has filled with these: an SM's warps read few different ones)
  const int4 meta = p.meta[blockIdx.x % kTreeCtas];
  const int first_own = meta.x, share[2] = {meta.y, meta.z};
  const int place0[2] = {np ? p.pline[np] : 0, b ? p.line[b] : 0};  // the first items' places are 0
  // A run's parts, and where they are: the first, the others, from one to the
  // next, from copy to copy.  A whole run's is by the row; else the first
  // share's part is its worker's last segment, the others' their first.
  const int copies = p.copies, shift = copies >> 1;  // 1, 2, 4: shifts of 0, 1, 2
  struct Run {
    int n, step;
    int64_t first, rest, copy;
  };
  auto run_of = [&](int y, int rt, int r, int row_group, int row_groups, int worker0) {
    const int len = lens[y];
    if (len == 0) return Run{0, 0, 0, 0, 0};
    const int group = rt / row_group, at = place0[y] + (static_cast<int>(hk) * row_groups + group) * len;
    const int w0 = (at + kItemCost) / share[y], n = (at + len - 1) / share[y] - w0 + 1;
    if (n == 1) return Run{1, 0, p.parts + y * copies * p.out_rows + static_cast<int64_t>(out), 0, p.out_rows};
    const int rest = 2 * (worker0 + w0 * row_group + rt - group * row_group) * p.slot_rows + r;
    return Run{n, 2 * row_group * p.slot_rows, rest + p.slot_rows, rest, kBM / copies};
  };
  const Run pre = run_of(0, prt, pr, p.prow_group, p.prow_groups, 0);
  const Run own = run_of(1, rr / 128, rr % 128, p.row_group, p.row_groups, first_own);
  const int parts = (pre.n + own.n) * copies;
  auto place = [&](int i) {
    const int copy = i & (copies - 1);
    i >>= shift;
    if (i < pre.n) return (i ? pre.rest + i * pre.step : pre.first) + copy * pre.copy;
    i -= pre.n;
    return (i ? own.rest + i * own.step : own.first) + copy * own.copy;
  };
  // A round takes up to 32 parts of the warp: lane i has the place, the weight
  // and the sum of part i, and all lanes add the parts' columns.
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int k0 = part; k0 < parts; k0 += 32 * WPR) {
    const int k = k0 + lane * WPR, n = min(32, (parts - k0 + WPR - 1) / WPR);
    int64_t at = 0;
    float2 st = make_float2(-INFINITY, 0.f);
    if (k < parts) {
      at = place(k);
      st = __ldcg(p.stats + at);
    }
    float w = 0.f;
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += kBatch * kAtOnce) {
      float4 y[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int j = i0 + i * kAtOnce + lane / kLanes;
        const int64_t row = __shfl_sync(0xffffffffu, at, j & 31);
        y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j < n) y[i] = __ldcg(reinterpret_cast<const float4*>(p.slots) + row * kLanes + lane % kLanes);
      }
      if (i0 == 0) {  // the first columns are on their way
        float mn = fmaxf(m, st.x);
#pragma unroll
        for (int off = 16; off; off >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
        const float ref = mn == -INFINITY ? 0.f : mn, a = ex2(m - ref);
        w = ex2(st.x - ref);
        l = fmaf(w, st.y, l * a);
        o = make_float4(o.x * a, o.y * a, o.z * a, o.w * a);
        m = mn;
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const float x = __shfl_sync(0xffffffffu, w, (i0 + i * kAtOnce + lane / kLanes) & 31);
        o = make_float4(fmaf(x, y[i].x, o.x), fmaf(x, y[i].y, o.y), fmaf(x, y[i].z, o.z), fmaf(x, y[i].w, o.w));
      }
    }
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
  if constexpr (kAtOnce == 2) {  // the two halves of the warp
    o.x += __shfl_xor_sync(0xffffffffu, o.x, 16);
    o.y += __shfl_xor_sync(0xffffffffu, o.y, 16);
    o.z += __shfl_xor_sync(0xffffffffu, o.z, 16);
    o.w += __shfl_xor_sync(0xffffffffu, o.w, 16);
  }
  if constexpr (WPR > 1) {
    if (lane < kLanes) s_o[warp][lane] = o;
    if (lane == 0) {
      s_m[warp] = m;
      s_l[warp] = l;
    }
    __syncthreads();
    if (warp) return;
    float ref = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
    if (ref == -INFINITY) ref = 0.f;
    l = 0.f;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float a = ex2(s_m[w] - ref);
      const float4 y = s_o[w][lane % kLanes];
      l = fmaf(a, s_l[w], l);
      o = make_float4(fmaf(a, y.x, o.x), fmaf(a, y.y, o.y), fmaf(a, y.z, o.z), fmaf(a, y.w, o.w));
    }
  }
  if (lane >= kLanes) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  static_cast<uint2*>(p.o)[static_cast<size_t>(out) * kLanes + lane] =
      make_uint2(pack2<BF16>(o.x * inv, o.y * inv), pack2<BF16>(o.z * inv, o.w * inv));
}

template <int D, bool BF16, int MODE>
stof_status launch_mode(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const PrefixParams& p,
                        cudaStream_t s) {
  if constexpr (D == 64) {
    if (p.copies == 4) return launch_scored<PrefixSource, D, BF16, MODE, 4>(mq, mk, mv, p, kTreeCtas, s);
    if (p.copies == 2) return launch_scored<PrefixSource, D, BF16, MODE, 2>(mq, mk, mv, p, kTreeCtas, s);
  }
  return launch_scored<PrefixSource, D, BF16, MODE, 1>(mq, mk, mv, p, kTreeCtas, s);
}

template <int D, bool BF16>
stof_status launch_prefix(const void* q, const void* kp, const void* vp, const void* k, const void* v, PrefixParams& p,
                          int mode, cudaStream_t s) {
  CUtensorMap mq, mk, mv;
  const uint64_t pplanes = static_cast<uint64_t>(p.NP) * p.Hkv, planes = static_cast<uint64_t>(p.B) * p.Hkv;
  if (!make_requests_map(&mq, q, p.B, p.Hkv, p.rows, D, p.own_fill, p.nb, BF16) ||
      !make_bw_map(&mk, kp, pplanes, p.pcap, D, Shape<D>::BN, BF16) || !make_bw_map(&mv, vp, pplanes, p.pcap, D, Shape<D>::BN, BF16))
    return STOF_ERR_CUDA;
  p.own_q = mq;
  p.own_k = mk;
  p.own_v = mv;
  if (p.lens && (!make_requests_map(&p.own_q, q, p.B, p.Hkv, p.rows, D, p.own_fill, 1, BF16) ||
                 !make_bw_map(&p.own_k, k, planes, p.cap, D, Shape<D>::BN, BF16) ||
                 !make_bw_map(&p.own_v, v, planes, p.cap, D, Shape<D>::BN, BF16)))
    return STOF_ERR_CUDA;
  stof_status st;
  switch (mode) {
    case MODE_PLAIN: st = launch_mode<D, BF16, MODE_PLAIN>(mq, mk, mv, p, s); break;
    case MODE_CAP: st = launch_mode<D, BF16, MODE_CAP>(mq, mk, mv, p, s); break;
    default: st = launch_mode<D, BF16, MODE_DISTANCE>(mq, mk, mv, p, s); break;
  }
  if (st != STOF_OK) return st;
  // A row is merged by one warp where the rows are many for their parts (of
  // which the host knows the most that a prefix's run may have), else by four.
  // One and four, the whole call: d = 128, 64 rows 26.9 and 22.6 us, 512 rows of
  // 39 parts 28.9 and 24.6, 1024 35.1 and 31.3, 1536 of 20 40.5 and 41.0, 4096 of
  // 5 49.3 and 66.7; d = 64, 256 rows of 39 20.4 and 16.5, 512 16.5 and 16.6, 1024
  // 18.6 and 19.5.
  const int64_t runs = static_cast<int64_t>(p.NP) * p.Hkv * p.prow_tiles, parts = 1 + kWorkers / (runs < kWorkers ? runs : kWorkers);
  const bool one = p.out_rows >= (D == 128 ? 64 : 24) * parts;
  const unsigned grid = static_cast<unsigned>(one ? (p.out_rows + 3) / 4 : p.out_rows) + 1;
  const cudaError_t e = launch_early(one ? merge_kernel<D, BF16, 1> : merge_kernel<D, BF16, 4>, dim3(grid), 128, 0, s, p);
  return record_cuda(e) == cudaSuccess ? STOF_OK : STOF_ERR_CUDA;
}

// The sizes that follow from a call's.
struct Sizes {
  int64_t rows, slot_rows, out_rows;
  int nb, per_request, fill, copies;
};
// False for sizes that the call does not take.
bool sizes_of(int B, int n_prefixes, int H, int Hkv, int T, int d, Sizes* z) {
  if (B < 1 || n_prefixes < 1 || B % n_prefixes || H < 1 || Hkv < 1 || H % Hkv || T < 1 || T > STOF_TREE_MAX_TOKENS ||
      (d != 64 && d != 128))
    return false;
  z->rows = static_cast<int64_t>(H / Hkv) * T;
  const int64_t n = B / n_prefixes, fit = z->rows < 128 ? 128 / z->rows : 1;
  z->nb = static_cast<int>(n < fit ? n : fit);
  z->per_request = static_cast<int>((z->rows + 127) / 128);
  z->fill = static_cast<int>(z->rows < 128 ? z->rows * z->nb : 128);
  z->copies = copies_of(d, z->fill);
  z->slot_rows = z->copies > 1 ? kBM : z->fill;
  z->out_rows = static_cast<int64_t>(B) * H * T;
  return true;
}

}  // namespace
}  // namespace stof

using namespace stof;

extern "C" size_t stof_prefix_attn_workspace_bytes(int B, int n_prefixes, int H, int Hkv, int T, int d) {
  Sizes z;
  if (!sizes_of(B, n_prefixes, H, Hkv, T, d, &z) || z.out_rows >= (1ll << 31)) return 0;
  const size_t rows = static_cast<size_t>(2 * kWorkers) * z.slot_rows + 2 * static_cast<size_t>(z.copies) * z.out_rows;
  return kErrorBytes + up256(rows * d * sizeof(float)) + up256(rows * sizeof(float2)) +
         kTreeCtas * sizeof(int4) + (static_cast<size_t>(B) + n_prefixes) * sizeof(int32_t);
}

extern "C" stof_status stof_prefix_attn_fwd(const void* q, const void* k_prefix, const void* v_prefix, const void* k,
                                            const void* v, stof_dtype dt, int B, int n_prefixes, int H, int Hkv, int T,
                                            int d, int prefix_cap, int cap, const int32_t* prefix_lens,
                                            const int32_t* lens, const int32_t* counts, const uint32_t* tree,
                                            const int32_t* positions, float scale, const stof_score* score, void* o,
                                            void* workspace, size_t ws_bytes, int64_t* device_error, void* stream) {
  const bool own = k || v || lens;
  if (!q || !k_prefix || !v_prefix || !o || !prefix_lens || !workspace || (own && (!k || !v || !lens))) return STOF_ERR_INVALID_ARG;
  if (dt != STOF_F16 && dt != STOF_BF16) return STOF_ERR_DTYPE;
  if (B < 1 || n_prefixes < 1 || H < 1 || Hkv < 1 || T < 1 || d < 1 || prefix_cap < 1 || (own && cap < 1) ||
      !std::isfinite(scale))
    return STOF_ERR_INVALID_ARG;
  if (!own && (tree || positions)) return STOF_ERR_INVALID_ARG;  // of drafted rows that are not there
  if (d != 64 && d != 128) return STOF_ERR_UNSUPPORTED;
  if (!own && score && score->slopes) return STOF_ERR_UNSUPPORTED;  // the queries have no place among the keys
  Sizes z;
  if (!sizes_of(B, n_prefixes, H, Hkv, T, d, &z)) return STOF_ERR_SHAPE;
  if (!own) cap = 1;
  const int64_t n = B / n_prefixes, row_tiles = (z.rows + 127) / 128;
  const int64_t prow_tiles = z.nb > 1 ? (n + z.nb - 1) / z.nb : n * z.per_request;
  // the lines of the call's tiles, its query rows and the keys' positions are counted in 32 bits
  const auto line = [&](int64_t items, int64_t tiles, int64_t keys) {
    return static_cast<long double>(items) * Hkv * tiles * ((keys + 63) / 64 + kItemCost);
  };
  if (z.out_rows >= (1ll << 31) || static_cast<int64_t>(B) * Hkv >= (1ll << 31) ||
      static_cast<int64_t>(prefix_cap) + cap >= 2147480000ll || line(B, row_tiles, cap) >= 2147480000.0L ||
      line(n_prefixes, prow_tiles, prefix_cap) >= 2147480000.0L)
    return STOF_ERR_SHAPE;
  if (score) {
    stof_score s = *score;
    s.q_start = 0;  // not read by this call
    const stof_status st = check_score(s, scale);
    if (st != STOF_OK) return st;
  }
  const uintptr_t wide = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_prefix) |
                         reinterpret_cast<uintptr_t>(v_prefix) | reinterpret_cast<uintptr_t>(k) |
                         reinterpret_cast<uintptr_t>(v) | reinterpret_cast<uintptr_t>(o) |
                         reinterpret_cast<uintptr_t>(workspace);
  const uintptr_t words = reinterpret_cast<uintptr_t>(prefix_lens) | reinterpret_cast<uintptr_t>(lens) |
                          reinterpret_cast<uintptr_t>(counts) | reinterpret_cast<uintptr_t>(tree) |
                          reinterpret_cast<uintptr_t>(positions);
  if (wide % 16 || words % 4 || reinterpret_cast<uintptr_t>(device_error) % 8) return STOF_ERR_ALIGNMENT;
  if (ws_bytes < stof_prefix_attn_workspace_bytes(B, n_prefixes, H, Hkv, T, d)) return STOF_ERR_WORKSPACE;
  const float softcap = score ? score->softcap : 0.f;
  PrefixParams p = {};
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
  p.words = (T + 31) / 32;
  p.tile = d == 64 ? Shape<64>::BN : Shape<128>::BN;
  p.rows = static_cast<int>(z.rows);
  p.row_tiles = static_cast<int>(row_tiles);
  p.row_groups = static_cast<int>((row_tiles + kRowGroup - 1) / kRowGroup);
  p.row_group = (p.row_tiles + p.row_groups - 1) / p.row_groups;
  p.prow_tiles = static_cast<int>(prow_tiles);
  p.prow_groups = static_cast<int>((prow_tiles + kRowGroup - 1) / kRowGroup);
  p.prow_group = (p.prow_tiles + p.prow_groups - 1) / p.prow_groups;
  p.per_row_group = 1.f / static_cast<float>(p.row_group);
  p.per_prow_group = 1.f / static_cast<float>(p.prow_group);
  p.slot_rows = static_cast<int>(z.slot_rows);
  p.lens = lens;
  p.counts = counts;
  p.tree = tree;
  p.positions = p.slopes ? positions : nullptr;
  p.NP = n_prefixes;
  p.n = static_cast<int>(n);
  p.pcap = prefix_cap;
  p.nb = z.nb;
  p.per_request = z.per_request;
  p.own_fill = static_cast<int>(z.rows < 128 ? z.rows : 128);
  p.fill = z.fill;
  p.plens = prefix_lens;
  p.out_rows = z.out_rows;
  p.copies = z.copies;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.parts = static_cast<int64_t>(2 * kWorkers) * p.slot_rows;
  const size_t rows = p.parts + 2 * static_cast<size_t>(z.copies) * z.out_rows;
  p.word = reinterpret_cast<long long*>(ws);
  p.status = reinterpret_cast<int*>(ws + 256);
  ws += kErrorBytes;
  p.slots = reinterpret_cast<float*>(ws);
  ws += up256(rows * d * sizeof(float));
  p.stats = reinterpret_cast<float2*>(ws);
  ws += up256(rows * sizeof(float2));
  p.meta = reinterpret_cast<int4*>(ws);
  p.line = reinterpret_cast<int32_t*>(p.meta + kTreeCtas);
  p.pline = p.line + B;
  const int mode = mode_of(scale, softcap, p.slopes != nullptr);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf16 = dt == STOF_BF16;
  if (d == 64)
    return bf16 ? launch_prefix<64, true>(q, k_prefix, v_prefix, k, v, p, mode, s)
                : launch_prefix<64, false>(q, k_prefix, v_prefix, k, v, p, mode, s);
  return bf16 ? launch_prefix<128, true>(q, k_prefix, v_prefix, k, v, p, mode, s)
              : launch_prefix<128, false>(q, k_prefix, v_prefix, k, v, p, mode, s);
}
