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
// Both are cut by keys (tree_attn.cu): the (prefix, K/V head) runs of key
// tiles, row tiles side by side, are one line, the (request, K/V head) runs
// another, and the workers are divided between the two lines so that both end
// at the same time; each line is cut into equal shares.  What a worker finds
// of a row is a part: in the worker's own two slots if the run goes on in
// another share, in a buffer of the rows if it does not; merge_kernel puts a
// row's parts together in a fixed order.  A run that is all a row sees (no own
// rows, or an empty prefix) and lies in one share is finished there.
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
  const int32_t* plens;
  int32_t* pline;                   // [NP + 1], as line
  int32_t* meta;                    // [2] shares of the prefixes' line, of the requests'
  float* part_o;                    // [2][B H T][d]: parts of runs that lie in one share, of prefixes and requests
  float2* part_stats;               // [2][B H T]
  int64_t out_rows;                 // B H T
};

// Rows of prefix np; -1: out of range.
__device__ __forceinline__ int prefix_rows(const PrefixParams& p, int np) {
  const int x = __ldg(p.plens + np);
  return x >= 0 && x <= p.pcap ? x : -1;
}
// Prefix rows, committed and drafted tokens of request b; false for one that
// breaks the bounds or has no token.
__device__ __forceinline__ bool request_of(const PrefixParams& p, int b, int& plen, int& ctx, int& count) {
  plen = prefix_rows(p, b / p.n);
  ctx = p.lens ? __ldg(p.lens + b) : 0;
  count = p.counts ? __ldg(p.counts + b) : p.T;
  return plen >= 0 && ctx >= 0 && count >= 1 && count <= p.T && (!p.lens || ctx <= p.cap - count);
}

// One of the two lines: runs of key tiles of its items.
struct Line {
  int row_tiles, row_group, row_groups;
};
__device__ __forceinline__ Line line_of(const PrefixParams& p, bool prefix) {
  return prefix ? Line{p.prow_tiles, p.prow_group, p.prow_groups} : Line{p.row_tiles, p.row_group, p.row_groups};
}
// Length of a run of prefix i or request i (0: none).
__device__ __forceinline__ int run_length(const PrefixParams& p, bool prefix, int i) {
  if (prefix) {
    const int rows = prefix_rows(p, i);
    return rows > 0 ? tiles_of(p, rows) + kItemCost : 0;
  }
  int plen, ctx, count;
  return p.lens && request_of(p, i, plen, ctx, count) ? tiles_of(p, ctx + count) + kItemCost : 0;
}
__device__ __forceinline__ int share_length(int all, int shares) { return max(1, (all + shares - 1) / max(1, shares)); }

// Shares of the two lines, of lengths lp and lo: as many workers for each as
// bring the later end forward.
__device__ __forceinline__ void divide(const PrefixParams& p, int lp, int lo, int& sp, int& so) {
  sp = lp > 0 ? kWorkers / p.prow_group : 0;
  so = lo > 0 ? kWorkers / p.row_group : 0;
  if (lp == 0 || lo == 0) return;
  const float wp = static_cast<float>(lp) * p.prow_group, wo = static_cast<float>(lo) * p.row_group;
  const int most = (kWorkers - p.row_group) / p.prow_group;
  int best = 0x7fffffff;
  const int x0 = max(1, min(most, static_cast<int>(kWorkers * (wp / (wp + wo)) / p.prow_group)));
  for (int x = x0; x <= min(most, x0 + 1); ++x) {
    const int y = (kWorkers - x * p.prow_group) / p.row_group;
    const int end = max(share_length(lp, x), share_length(lo, y));
    if (end < best) {
      best = end;
      sp = x;
      so = y;
    }
  }
}

struct PrefixSource : CacheSource {
  using Params = PrefixParams;
  static constexpr bool kTwoPlaces = true;
  struct Item : CacheSource::Item {  // of a prefix: ctx its rows, count 0, b its number
    bool prefix;
    int base;  // position of the item's first key: 0, or the prefix's rows
  };
  struct Shared {
    int sums[kThreads / 32];
    bool prefix[2];        // the workers' lines
    int row[2];            // their row tiles within a group
    int begin[2], end[2];  // and shares
    int i[2], base[2];     // the prefix or request that holds a share's begin, its place on the line
    int bad;               // CTA 0: a length breaks the bounds
  };
  struct Row : CacheSource::Row {
    int b, plen, ctx, count;  // the row's request
  };

  static __device__ void init(Shared& s) { s.bad = 0; }

  // Place of thread's item in the round that begins with item i0 (all threads).
  static __device__ int place(const Params& p, Shared& s, bool prefix, int i0, int before, int& v, int& total) {
    const Line l = line_of(p, prefix);
    const int i = i0 + static_cast<int>(threadIdx.x);
    v = i < (prefix ? p.NP : p.B) ? run_length(p, prefix, i) * p.Hkv * l.row_groups : 0;
    return before + block_prefix(v, s.sums, total);
  }
  // Length of a line; CTA 0 leaves the items' places for merge_kernel and
  // reports bad lengths.
  static __device__ int measure(const Params& p, Shared& s, bool prefix, int& v, int& at) {
    const int items = prefix ? p.NP : p.B;
    int32_t* line = prefix ? p.pline : p.line;
    int all = 0;
    v = at = 0;
    for (int i0 = 0; i0 < items; i0 += kThreads) {
      int total;
      at = place(p, s, prefix, i0, all, v, total);
      const int i = i0 + static_cast<int>(threadIdx.x);
      if (blockIdx.x == 0 && i < items) {
        line[i] = at;
        bool bad;
        if (prefix) {
          bad = prefix_rows(p, i) < 0;
        } else {
          int plen, ctx, count;
          bad = !request_of(p, i, plen, ctx, count) && plen >= 0 &&
                !(count == 0 && ctx >= 0 && (!p.lens || ctx <= p.cap));
        }
        if (bad) {
          s.bad = 1;
          if (p.err) raise_error(p.err, STOF_DEVERR_BAD_LENGTH);
        }
      }
      all += total;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) line[items] = all;
    return all;
  }
  static __device__ void prologue(const Params& p, Shared& s) {
    dependents_launch();  // merge_kernel may be set up
    int v[2], at[2], all[2], shares[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) all[x] = measure(p, s, x == 0, v[x], at[x]);
    divide(p, all[0], all[1], shares[0], shares[1]);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      p.meta[0] = shares[0];
      p.meta[1] = shares[1];
    }
    const int first_own = shares[0] * p.prow_group;  // workers before it are the prefixes'
    bool mine[2];
    int begin[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int w = worker(g), x = w < first_own ? 0 : 1;
      const int in = w - x * first_own, group = x ? p.row_group : p.prow_group;
      const int length = share_length(all[x], shares[x]), nth = in / group;
      mine[g] = x == 0;
      begin[g] = nth < shares[x] ? min(nth * length, all[x]) : all[x];
      if (threadIdx.x == 0) {
        s.prefix[g] = mine[g];
        s.row[g] = in - nth * group;
        s.begin[g] = begin[g];
        s.end[g] = begin[g] + min(length, all[x] - begin[g]);
      }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int items = x == 0 ? p.NP : p.B;
      int base = 0;
      for (int i0 = 0; i0 < items; i0 += kThreads) {
        if (items > kThreads) {  // else v and at are those of the one round above
          int total;
          at[x] = place(p, s, x == 0, i0, base, v[x], total);
          base += total;
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          if (mine[g] == (x == 0) && at[x] <= begin[g] && begin[g] < at[x] + v[x]) {
            s.i[g] = i0 + threadIdx.x;
            s.base[g] = at[x];
          }
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
        load(p);
      }
    }
    __device__ void load(const Params& p) {
      len = run_length(p, prefix, i);
      if (prefix) {
        ctx = prefix_rows(p, i);
        count = 0;
        plen = 0;
      } else {
        request_of(p, i, plen, ctx, count);
      }
    }
    __device__ Next next(const Params& p, Shared&, const volatile int*, Segment<Item>& seg) {
      const Line l = line_of(p, prefix);
      const int per = p.Hkv * l.row_groups;
#pragma unroll 1
      while (w < end) {
#pragma unroll 1
        while (w >= base + len * per) {  // on to the next item on the line
          base += len * per;
          ++i;
          load(p);
        }
        const int off = w - base, item = off / len, at = off - item * len;
        const int to = min(end - base - item * len, len);  // the share's part of the run: [at, to)
        w += to - at;
        const int t0 = max(0, at - kItemCost), t1 = max(0, to - kItemCost);
        const int hk = item / l.row_groups, rt = (item - hk * l.row_groups) * l.row_group + row;
        if (t1 <= t0 || rt >= l.row_tiles) continue;
        if (prefix) {
          const int x = rt / p.per_request;
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

  static __device__ bool begin_row(const Params& p, Row& row, const Segment<Item>& seg, int r) {
    const Item& x = seg.item;
    int rr = seg.q_row + r;
    row.b = seg.q_plane;
    bool live = true;
    if (x.prefix && p.nb > 1) {
      const int in = r / p.rows;
      rr = r - in * p.rows;
      row.b += in;
      live = in < p.nb && row.b < (x.b + 1) * p.n;
    }
    const int gq = rr / p.T;
    row.t = rr - gq * p.T;
    row.head = x.hk * p.group + gq;
    live = live && rr < p.rows && request_of(p, row.b, row.plen, row.ctx, row.count) && row.t < row.count;
    const size_t token = static_cast<size_t>(row.b) * p.T + row.t;
    row.pos = live && p.positions ? __ldg(p.positions + token) : (live ? row.plen + row.ctx + row.t : 0);
    row.out = (static_cast<size_t>(row.b) * p.H + row.head) * p.T + row.t;
    row.tree = live && p.tree ? p.tree + token * p.words : nullptr;
    return live;
  }
  // Distance of the nearest (far: farthest) key that the row sees, in the
  // prefix or of the request's own: the parts of a row have one reference.
  static __device__ uint32_t reference(const Params& p, const Row& row, const Item&, bool far) {
    CacheSource::Item own;
    own.b = row.b;
    own.count = row.count;
    own.ctx = row.plen + row.ctx;  // rows 0 .. of the prefix and the request are positions 0 ..
    return CacheSource::reference(p, row, own, far);
  }
  template <int BN, int CHUNKS>
  static __device__ void lower(const Params& p, const Row& row, const Item& x, int t, int j0, uint32_t (&sr)[CHUNKS][32],
                               float c, float slope, uint32_t base) {
    if (p.positions && !x.prefix && partial(x, t)) {
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
  // The run is all that its rows see, and lies in one share.
  static __device__ bool whole(const Params& p, const Item& x) { return x.whole && (x.prefix ? !p.lens : x.base == 0); }
  // Parts of whole runs by the row of O; of others by the worker, as CacheSource.
  static __device__ size_t slot_row(const Params& p, const Item& x, int g, int r) {
    return static_cast<size_t>(2 * worker(g) + (x.t0 == 0 ? 1 : 0)) * p.slot_rows + r;
  }
  static __device__ float* partial_o(const Params& p, const Item& x, const Row& row, int g, int r, int d) {
    return x.whole ? p.part_o + ((x.prefix ? 0 : p.out_rows) + row.out) * d : p.slots + slot_row(p, x, g, r) * d;
  }
  static __device__ void put_stats(const Params& p, const Item& x, const Row& row, int g, int r, float m, float l) {
    (x.whole ? p.part_stats[(x.prefix ? 0 : p.out_rows) + row.out] : p.stats[slot_row(p, x, g, r)]) = make_float2(m, l);
  }
};

// Merges the parts of the rows, those of the prefix first.  WPR warps per row,
// warp x of a row the parts x, x + WPR, ..., kBatch of them in flight; four
// rows of one warp, or one row of four, a block.  (Launched while the main
// kernel still runs, it begins when that has ended.)
template <int D, bool BF16, int WPR>
__global__ void __launch_bounds__(128) merge_kernel(const __grid_constant__ PrefixParams p) {
  constexpr int E = D / 32, kBatch = 8;
  __shared__ float s_o[4][D], s_m[4], s_l[4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % WPR;
  if (blockIdx.x == gridDim.x - 1) {  // the last block: the call's error bits
    dependents_wait();
    int bits = 0;
    for (int c = threadIdx.x; c < kTreeCtas; c += blockDim.x) bits |= __ldcg(p.status + c);
    const int late = __syncthreads_or(bits & STOF_DEVERR_PIPE_TIMEOUT), bad = __syncthreads_or(bits & STOF_DEVERR_BAD_LENGTH);
    if (threadIdx.x == 0) *p.word = (late ? STOF_DEVERR_PIPE_TIMEOUT : 0) | (bad ? STOF_DEVERR_BAD_LENGTH : 0);
    return;
  }
  const int64_t out = static_cast<int64_t>(blockIdx.x) * (4 / WPR) + warp / WPR;
  if (out >= p.out_rows) return;  // (one row: the whole block)
  const int x = static_cast<int>(out / p.T), t = static_cast<int>(out - static_cast<int64_t>(x) * p.T);
  const int b = x / p.H, h = x - b * p.H, hk = h / p.group, rr = (h - hk * p.group) * p.T + t;
  int plen, ctx, count;
  if (!request_of(p, b, plen, ctx, count) || t >= count) return;
  dependents_wait();
  const int sp = __ldcg(p.meta), so = __ldcg(p.meta + 1);
  // a run's parts; the slot of its row in the share of the first of them, slots from share to share
  struct Run {
    int n;
    int64_t slot, step;
  };
  auto run_of = [&](bool prefix) {
    const int item = prefix ? b / p.n : b, len = run_length(p, prefix, item);
    if (len == 0) return Run{0, 0, 0};
    const Line l = line_of(p, prefix);
    int rt = rr / 128, r = rr - rt * 128;  // the row's tile of the run and place in it
    if (prefix) {
      const int in = b - item * p.n;
      rt = p.nb > 1 ? in / p.nb : in * p.per_request + rt;
      if (p.nb > 1) r = (in - rt * p.nb) * p.rows + rr;
    }
    const int32_t* line = prefix ? p.pline : p.line;
    const int share = share_length(__ldcg(line + (prefix ? p.NP : p.B)), prefix ? sp : so), group = rt / l.row_group;
    const int at = __ldcg(line + item) + (hk * l.row_groups + group) * len, w0 = (at + kItemCost) / share;
    const int64_t worker = (prefix ? 0 : sp * p.prow_group) + w0 * l.row_group + rt - group * l.row_group;
    return Run{(at + len - 1) / share - w0 + 1, 2 * worker * p.slot_rows + r, 2 * static_cast<int64_t>(l.row_group) * p.slot_rows};
  };
  const Run pre = run_of(true), own = run_of(false);
  const int parts = pre.n + own.n;
  if (parts == 1) return;  // finished by its one worker (none: a row that sees nothing, 0)
  auto place = [&](int i, const float*& o, const float2*& st) {
    const bool prefix = i < pre.n;
    const Run u = prefix ? pre : own;
    if (!prefix) i -= pre.n;
    // a whole run: by the row; else the first share's part is its worker's last segment, the others' their first
    const int64_t at = u.n == 1 ? (prefix ? 0 : p.out_rows) + out : u.slot + i * u.step + (i == 0 ? p.slot_rows : 0);
    o = (u.n == 1 ? p.part_o : p.slots) + at * D;
    st = (u.n == 1 ? p.part_stats : p.stats) + at;
  };
  float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 1
  for (int i0 = part; i0 < parts; i0 += WPR * kBatch) {
    float2 st[kBatch];
    float y[kBatch][E];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int k = i0 + i * WPR;
      st[i] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < E; ++e) y[i][e] = 0.f;
      if (k < parts) {
        const float* src;
        const float2* stats;
        place(k, src, stats);
        st[i] = __ldcg(stats);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 z = __ldcg(reinterpret_cast<const float2*>(src + lane * E + e));
          y[i][e] = z.x;
          y[i][e + 1] = z.y;
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
      for (int e = 0; e < E; ++e) o[e] = fmaf(w, y[i][e], o[e]);
    }
    m = mn;
  }
  uint32_t* to = static_cast<uint32_t*>(p.o) + ((static_cast<size_t>(out) * D) >> 1);
  if constexpr (WPR == 1) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < E; e += 2) to[(lane * E + e) >> 1] = pack2<BF16>(o[e] * inv, o[e + 1] * inv);
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
    to[c >> 1] = pack2<BF16>(y0 * inv, y1 * inv);
  }
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
  // one warp a row where the rows are many for their parts, as in tree_attn.cu
  const int64_t runs = static_cast<int64_t>(p.NP) * p.Hkv * p.prow_tiles;
  const bool one = p.out_rows >= 128 * (1 + kWorkers / (runs < kWorkers ? runs : kWorkers));
  const unsigned grid = static_cast<unsigned>(one ? (p.out_rows + 3) / 4 : p.out_rows) + 1;
  const cudaError_t e = launch_early(one ? merge_kernel<D, BF16, 1> : merge_kernel<D, BF16, 4>, dim3(grid), 128, 0, s, p);
  return record_cuda(e) == cudaSuccess ? STOF_OK : STOF_ERR_CUDA;
}

// The sizes that follow from a call's.
struct Sizes {
  int64_t rows, slot_rows, out_rows;
  int nb, per_request;
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
  z->slot_rows = z->rows < 128 ? z->rows * z->nb : 128;
  z->out_rows = static_cast<int64_t>(B) * H * T;
  return true;
}

}  // namespace
}  // namespace stof

using namespace stof;

extern "C" size_t stof_prefix_attn_workspace_bytes(int B, int n_prefixes, int H, int Hkv, int T, int d) {
  Sizes z;
  if (!sizes_of(B, n_prefixes, H, Hkv, T, d, &z) || z.out_rows >= (1ll << 31)) return 0;
  const size_t slots = static_cast<size_t>(2 * kWorkers) * z.slot_rows, parts = 2 * static_cast<size_t>(z.out_rows);
  return kErrorBytes + up256(slots * d * sizeof(float)) + up256(slots * sizeof(float2)) + up256(parts * d * sizeof(float)) +
         up256(parts * sizeof(float2)) + (static_cast<size_t>(B) + n_prefixes + 4) * sizeof(int32_t);
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
  p.fill = p.own_fill * p.nb;
  p.plens = prefix_lens;
  p.out_rows = z.out_rows;
  p.copies = copies_of(d, p.fill);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const size_t slots = static_cast<size_t>(2 * kWorkers) * p.slot_rows, parts = 2 * static_cast<size_t>(z.out_rows);
  p.word = reinterpret_cast<long long*>(ws);
  p.status = reinterpret_cast<int*>(ws + 256);
  ws += kErrorBytes;
  p.slots = reinterpret_cast<float*>(ws);
  ws += up256(slots * d * sizeof(float));
  p.stats = reinterpret_cast<float2*>(ws);
  ws += up256(slots * sizeof(float2));
  p.part_o = reinterpret_cast<float*>(ws);
  ws += up256(parts * d * sizeof(float));
  p.part_stats = reinterpret_cast<float2*>(ws);
  ws += up256(parts * sizeof(float2));
  p.line = reinterpret_cast<int32_t*>(ws);
  p.pline = p.line + B + 1;
  p.meta = p.pline + n_prefixes + 1;
  const int mode = mode_of(scale, softcap, p.slopes != nullptr);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf16 = dt == STOF_BF16;
  if (d == 64)
    return bf16 ? launch_prefix<64, true>(q, k_prefix, v_prefix, k, v, p, mode, s)
                : launch_prefix<64, false>(q, k_prefix, v_prefix, k, v, p, mode, s);
  return bf16 ? launch_prefix<128, true>(q, k_prefix, v_prefix, k, v, p, mode, s)
              : launch_prefix<128, false>(q, k_prefix, v_prefix, k, v, p, mode, s);
}
