// Attention of drafted tokens over a K/V cache (stof_tree_attn_fwd).
//
// A request's rows for one K/V head are its group's heads times its drafted
// tokens, contiguous in Q: row r = head-in-group * T + t, in tiles of 128.
// Bound by memory while a K/V head has up to a few hundred rows: every K and V
// row has to be read once (4 d bytes), and 128 rows cost the tensor cores
// half of the time that 128 keys take to arrive.  So the work is cut by keys:
// all (request, K/V head, row tile) items in order, each a run of 128-key
// tiles, are one long sequence of tiles, of which each of kTreeCtas CTAs
// takes an equal share (the lengths are read on the device, so the shares
// follow them).  A CTA streams its share through scored_kernel.cuh, a
// segment per item it touches; an item that lies in one share is finished
// there, the others leave partial rows (O relative to the rows' max, max and
// sum) in the workspace, which combine_kernel merges in the order of the
// keys: the result does not depend on timing.  A CTA has at most one item
// that began before its share and one that goes on after it: two slots.
#include <cmath>

#include "scored_kernel.cuh"

namespace stof {
namespace {

using namespace scored;

constexpr int kTreeCtas = 152;  // one CTA per SM

struct TreeParams : CommonParams {
  int B, Hkv, T, d, cap, words;
  int rows;        // group * T: query rows per K/V head
  int row_tiles;   // ceil(rows / 128)
  int slot_rows;   // rows of a partial result: min(rows, 128)
  const int32_t* lens;
  const int32_t* counts;
  const uint32_t* tree;
  const int32_t* positions;
  float* slots;    // [2 kTreeCtas][slot_rows][d] partial O
  float2* stats;   // [2 kTreeCtas][slot_rows] (max, sum)
};

// Committed and drafted tokens of request b; false for a request that breaks
// the bounds or has no drafted token.
__device__ __forceinline__ bool request(const TreeParams& p, int b, int& ctx, int& count) {
  ctx = __ldg(p.lens + b);
  count = p.counts ? __ldg(p.counts + b) : p.T;
  return ctx >= 0 && count >= 1 && count <= p.T && ctx <= p.cap - count;
}
__device__ __forceinline__ int tiles_of(const TreeParams& p, int b) {
  int ctx, count;
  return request(p, b, ctx, count) ? (ctx + count + 127) >> 7 : 0;
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

// All tiles of the call.
__device__ __forceinline__ int total_tiles(const TreeParams& p, int* sums) {
  int all = 0;
  for (int b0 = 0; b0 < p.B; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    int total;
    block_prefix(b < p.B ? tiles_of(p, b) * p.Hkv * p.row_tiles : 0, sums, total);
    all += total;
  }
  return all;
}

// Tiles per CTA.
__device__ __forceinline__ int share_of(int all) { return max(1, (all + kTreeCtas - 1) / kTreeCtas); }

struct CacheSource {
  using Params = TreeParams;
  static constexpr bool kClearsV = true;
  struct Row {
    int head, t, pos;
    size_t out;
    const uint32_t* tree;  // the row's bits, or null
  };
  struct Tile {
    bool partial;   // not every key is visible to every row
    bool drafted;   // it has drafted keys
    int j0;
    int end;        // keys of the tile that the request has
  };

  const Params& p;
  int w, w_end;            // next tile of the share, its end
  int b, base, nt;         // request, the number of its first tile, tiles per item
  int ctx, count;
  int t0, hk, rt;          // the segment: first tile of the item, K/V head, row tile
  bool whole_;

  __device__ explicit CacheSource(const Params& params) : p(params) {
    __shared__ int sums[kThreads / 32];
    __shared__ int s_b, s_base;
    const int all = total_tiles(p, sums), share = share_of(all);
    w = min(static_cast<int>(blockIdx.x) * share, all);
    w_end = min(w + share, all);
    if (threadIdx.x == 0) s_b = p.B;
    int base0 = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {  // the request that holds tile w
      const int bb = b0 + threadIdx.x;
      const int v = bb < p.B ? tiles_of(p, bb) * p.Hkv * p.row_tiles : 0;
      if (blockIdx.x == 0 && p.err && bb < p.B && v == 0) {
        int c, n;
        if (!request(p, bb, c, n) && !(n == 0 && c >= 0 && c <= p.cap))
          raise_error(p.err, STOF_DEVERR_BAD_LENGTH);
      }
      int total;
      const int first = base0 + block_prefix(v, sums, total);
      if (v > 0 && first <= w && w < first + v) {
        s_b = bb;
        s_base = first;
      }
      base0 += total;
    }
    __syncthreads();
    b = s_b;
    base = s_base;
    if (w < w_end) load_request();
  }
  __device__ void load_request() {
    nt = request(p, b, ctx, count) ? (ctx + count + 127) >> 7 : 0;
  }
  __device__ bool next(Segment& seg) {
    if (w >= w_end) return false;
    while (w >= base + nt * p.Hkv * p.row_tiles) {  // on to the next request with tiles
      base += nt * p.Hkv * p.row_tiles;
      ++b;
      load_request();
    }
    const int off = w - base, item = off / nt;
    t0 = off - item * nt;
    hk = item / p.row_tiles;
    rt = item - hk * p.row_tiles;
    seg.q_plane = seg.kv_plane = b * p.Hkv + hk;
    seg.q_row = rt * 128;
    seg.n = min(nt - t0, w_end - w);
    whole_ = seg.n == nt;
    w += seg.n;
    return true;
  }
  __device__ int tile_key(int t) const { return (t0 + t) * 128; }
  __device__ bool begin_row(Row& row, const Segment&, int r) const {
    const int rr = rt * 128 + r;
    const int gq = rr / p.T;
    row.t = rr - gq * p.T;
    row.head = hk * p.group + gq;
    const bool live = rr < p.rows && row.t < count;
    const size_t token = static_cast<size_t>(b) * p.T + row.t;
    row.pos = live && p.positions ? __ldg(p.positions + token) : ctx + row.t;
    row.out = (static_cast<size_t>(b) * p.H + row.head) * p.T + row.t;
    row.tree = live && p.tree ? p.tree + token * p.words : nullptr;
    return live;
  }
  __device__ void prefetch(Row&, const Segment&, int) const {}
  __device__ Tile tile(const Row&, const Segment&, int t) const {
    Tile x;
    x.j0 = (t0 + t) * 128;
    x.end = min(128, ctx + count - x.j0);
    x.drafted = x.j0 + 128 > ctx;
    x.partial = x.drafted;
    return x;
  }
  // Bits of drafted tokens 32 x .. 32 x + 31 that the row sees.
  __device__ uint32_t seen(const Row& row, int x) const {
    if (x < 0 || 32 * x >= count) return 0u;
    uint32_t word;
    if (p.tree)
      word = row.tree ? __ldg(row.tree + x) : 0u;
    else
      word = row.t >= 32 * x + 31 ? ~0u : (row.t < 32 * x ? 0u : (2u << (row.t - 32 * x)) - 1u);
    const int left = count - 32 * x;
    return left >= 32 ? word : word & ((1u << left) - 1u);
  }
  __device__ void bits(const Row& row, const Segment&, int t, uint32_t (&out)[4]) const {
#pragma unroll
    for (int cc = 0; cc < 4; ++cc) {
      const int u0 = (t0 + t) * 128 + 32 * cc - ctx;  // drafted token of the chunk's first key
      if (u0 <= -32) {
        out[cc] = ~0u;
      } else if (u0 < 0) {
        out[cc] = ((1u << -u0) - 1u) | (seen(row, 0) << -u0);
      } else {
        const int x = u0 >> 5, sh = u0 & 31;
        out[cc] = __funnelshift_r(seen(row, x), seen(row, x + 1), sh);
      }
    }
  }
  __device__ void lower(const Row& row, const Tile& t, uint32_t (&sr)[4][32], float c, float slope) const {
    const long long rel = static_cast<long long>(row.pos) - t.j0;
    if (t.drafted && p.positions) {
      float at[4];  // position of key 32 i + lane of the tile
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = 32 * i + static_cast<int>(threadIdx.x & 31), u = t.j0 + key - ctx;
        long long x = key;
        if (u >= 0) x = u < count ? static_cast<long long>(__ldg(p.positions + static_cast<size_t>(b) * p.T + u)) - t.j0 : 0;
        at[i] = static_cast<float>(x);
      }
      lower_by_positions(sr, c, slope, static_cast<float>(rel), at);
    } else {
      lower_by_distance(sr, c, slope, static_cast<float>(rel), __all_sync(0xffffffffu, rel >= 127));
    }
  }
  __device__ bool whole(const Segment&) const { return whole_; }
  __device__ size_t out_row(const Row& row) const { return row.out; }
  // A segment that begins its item goes on in the next CTA's share: slot 2 c + 1; else slot 2 c.
  __device__ size_t slot_row(int r) const {
    return static_cast<size_t>(2 * blockIdx.x + (t0 == 0 ? 1 : 0)) * p.slot_rows + r;
  }
  __device__ float* partial_o(const Segment&, int r) const { return p.slots + slot_row(r) * p.d; }
  __device__ void put_stats(const Segment&, int r, float m, float l) const { p.stats[slot_row(r)] = make_float2(m, l); }
};

// Merges the partial rows of the items that lie in several CTAs' shares, a
// warp per query row: O = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ TreeParams p) {
  constexpr int E = D / 32;
  __shared__ int sums[8];
  __shared__ int s_base;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = p.Hkv * p.row_tiles;
  const int b = static_cast<int>(blockIdx.x) / per, item = static_cast<int>(blockIdx.x) - b * per;
  int all = 0;
  for (int b0 = 0; b0 < p.B; b0 += 256) {
    const int bb = b0 + threadIdx.x;
    int total;
    const int first = all + block_prefix(bb < p.B ? tiles_of(p, bb) * per : 0, sums, total);
    if (bb == b) s_base = first;
    all += total;
  }
  __syncthreads();
  int ctx, count;
  if (!request(p, b, ctx, count)) return;
  const int nt = (ctx + count + 127) >> 7, share = share_of(all), w0 = s_base + item * nt;
  const int c0 = w0 / share, c1 = (w0 + nt - 1) / share;
  if (c0 == c1) return;  // finished by its one CTA
  const int hk = item / p.row_tiles, rt = item - hk * p.row_tiles;
  const int r = static_cast<int>(blockIdx.y) * 8 + warp, rr = rt * 128 + r, gq = rr / p.T, t = rr - gq * p.T;
  if (r >= p.slot_rows || rr >= p.rows || t >= count) return;
  // the first CTA's part is its last segment, the others' their first
  auto slot = [&](int c) { return static_cast<size_t>(2 * c + (c == c0 ? 1 : 0)) * p.slot_rows + r; };
  float m = -INFINITY;
  for (int c = c0 + lane; c <= c1; c += 32) m = fmaxf(m, p.stats[slot(c)].x);
#pragma unroll
  for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  float l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int i0 = c0; i0 <= c1; i0 += 32) {
    float w = 0.f;
    if (i0 + lane <= c1) {
      const float2 st = p.stats[slot(i0 + lane)];
      w = st.x == -INFINITY ? 0.f : ex2(st.x - m);
      l = fmaf(w, st.y, l);
    }
    const int n = min(32, c1 - i0 + 1);
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      const float* src = p.slots + slot(i0 + i) * D + lane * E;
      if constexpr (E == 4) {
        const float4 x = *reinterpret_cast<const float4*>(src);
        o[0] = fmaf(wi, x.x, o[0]);
        o[1] = fmaf(wi, x.y, o[1]);
        o[2] = fmaf(wi, x.z, o[2]);
        o[3] = fmaf(wi, x.w, o[3]);
      } else {
        const float2 x = *reinterpret_cast<const float2*>(src);
        o[0] = fmaf(wi, x.x, o[0]);
        o[1] = fmaf(wi, x.y, o[1]);
      }
    }
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint32_t* out = static_cast<uint32_t*>(p.o) +
                  ((((static_cast<size_t>(b) * p.H + hk * p.group + gq) * p.T + t) * D + lane * E) >> 1);
#pragma unroll
  for (int e = 0; e < E; e += 2) out[e / 2] = pack2<BF16>(o[e] * inv, o[e + 1] * inv);
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

template <int D, bool BF16>
stof_status launch_tree(const void* q, const void* k, const void* v, const TreeParams& p, int mode, cudaStream_t s) {
  CUtensorMap mq, mk, mv;
  const uint64_t planes = static_cast<uint64_t>(p.B) * p.Hkv;
  if (!make_bw_map(&mq, q, planes, p.rows, D, kBM, BF16) || !make_bw_map(&mk, k, planes, p.cap, D, 128, BF16) ||
      !make_bw_map(&mv, v, planes, p.cap, D, 128, BF16))
    return STOF_ERR_CUDA;
  constexpr int ST = D == 128 ? 3 : 6;  // 32 or 16 KB a stage: about 200 KB of K and V in flight or in use
  stof_status st;
  switch (mode) {
    case MODE_PLAIN: st = launch_scored<CacheSource, D, BF16, MODE_PLAIN, ST>(mq, mk, mv, p, kTreeCtas, s); break;
    case MODE_CAP: st = launch_scored<CacheSource, D, BF16, MODE_CAP, ST>(mq, mk, mv, p, kTreeCtas, s); break;
    default: st = launch_scored<CacheSource, D, BF16, MODE_DISTANCE, ST>(mq, mk, mv, p, kTreeCtas, s); break;
  }
  if (st != STOF_OK) return st;
  const dim3 grid(static_cast<unsigned>(planes * p.row_tiles), static_cast<unsigned>((p.slot_rows + 7) / 8));
  combine_kernel<D, BF16><<<grid, 256, 0, s>>>(p);
  return record_cuda(cudaGetLastError()) == cudaSuccess ? STOF_OK : STOF_ERR_CUDA;
}

}  // namespace
}  // namespace stof

using namespace stof;

extern "C" size_t stof_tree_attn_workspace_bytes(int B, int H, int Hkv, int T, int d) {
  if (B < 1 || H < 1 || Hkv < 1 || H % Hkv || T < 1 || T > STOF_TREE_MAX_TOKENS || (d != 64 && d != 128)) return 0;
  const long long rows = static_cast<long long>(H / Hkv) * T;
  const size_t slots = static_cast<size_t>(2 * kTreeCtas) * (rows < 128 ? rows : 128);
  return up256(slots * d * sizeof(float)) + slots * sizeof(float2);
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
  // tiles of the call and query rows are counted in 32 bits
  if (static_cast<long long>(B) * H * T >= (1ll << 31) || static_cast<long long>(B) * Hkv >= (1ll << 31) ||
      static_cast<long double>(B) * Hkv * row_tiles * ((static_cast<long long>(cap) + 127) / 128) >= 2147483000.0L)
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
  p.words = (T + 31) / 32;
  p.rows = static_cast<int>(rows);
  p.row_tiles = static_cast<int>(row_tiles);
  p.slot_rows = static_cast<int>(rows < 128 ? rows : 128);
  p.lens = lens;
  p.counts = counts;
  p.tree = tree;
  p.positions = p.slopes ? positions : nullptr;
  p.slots = static_cast<float*>(workspace);
  const size_t slots = static_cast<size_t>(2 * kTreeCtas) * p.slot_rows;
  p.stats = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + up256(slots * d * sizeof(float)));
  const int mode = mode_of(scale, softcap, p.slopes != nullptr);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d == 64)
    return dt == STOF_BF16 ? launch_tree<64, true>(q, k, v, p, mode, s) : launch_tree<64, false>(q, k, v, p, mode, s);
  return dt == STOF_BF16 ? launch_tree<128, true>(q, k, v, p, mode, s) : launch_tree<128, false>(q, k, v, p, mode, s);
}
