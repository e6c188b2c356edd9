// Moves of rows of K/V caches (stof_cache_keep, stof_cache_fork).  No
// arithmetic: every moved row is read and written once, so both are bound by
// memory, and a call of one layer by the latency of its two or three dependent
// loads.  One launch takes the caches of many layers.
//
// Keep moves drafted rows in place, row n + path[i] to row n + i with path
// ascending, so path[i] >= i and what row i is moved over is a row that no
// later move reads.  A thread owns 16 bytes of the rows of one head and takes
// the path in order, kRowsKeep rows read before any of them is written: no
// thread waits for another, and nothing is staged.
//
// Fork copies runs of rows between slots.  A run (one head's rows of one
// cache and slot) is contiguous, and is cut into pieces of kPiece units, which
// its blocks take in turn.  Runs that read the same rows follow one another
// (slots go fastest), so that all but the first read the L2 cache.
//
// Measured: 12 requests' rows of 24 caches (12 heads of 64, 400 to 1111 rows)
// into a second set 70 us, 6.3 TB/s of rows read once and written, 92% of the
// copy rate; kept rows of 48 caches (16 requests, 8 heads of 128, 16 MB) 6.4 us,
// of 2 caches 4.3: launch and latency.
#include <cuda_runtime.h>

#include <algorithm>

#include "internal.h"

namespace stof {
namespace {

constexpr int kThreadsRows = 128;
constexpr int kRowsKeep = 8;  // rows in flight per thread

struct KeepParams {
  int T, heads, rows, units, n;  // units: 16-byte columns of a row
  const int32_t* lens;
  const int32_t* path;
  const int32_t* kept;
  int32_t* new_lens;
  int64_t* err;
  uint4* data[STOF_CACHES_MAX];
};

__device__ __forceinline__ void bad_length(int64_t* err) {
  if (err) atomicOr(reinterpret_cast<unsigned long long*>(err), static_cast<unsigned long long>(STOF_DEVERR_BAD_LENGTH));
}

// Block (x, b): some of the 16-byte columns of request b's heads in all caches.
__global__ void __launch_bounds__(kThreadsRows) keep_kernel(const __grid_constant__ KeepParams p) {
  __shared__ int32_t s_path[STOF_TREE_MAX_TOKENS];
  const int b = blockIdx.y;
  const int32_t* path = p.path + static_cast<int64_t>(b) * p.T;
  const int len = __ldg(p.lens + b), kept = __ldg(p.kept + b);
  for (int i = threadIdx.x; i < p.T; i += kThreadsRows) s_path[i] = __ldg(path + i);
  __syncthreads();
  // ascending from 0, inside the cache; the first rows may already be in place
  bool bad = len < 0 || len > p.rows || kept < 0 || kept > p.T;
  int same = 0;
  for (int i = threadIdx.x; !bad && i < kept; i += kThreadsRows) {
    const int u = s_path[i];
    bad = u < (i ? s_path[i - 1] + 1 : 0) || u >= p.T || len > p.rows - 1 - u;
    same += u == i;
  }
  bad = __syncthreads_or(bad);
  if (bad) {
    if (blockIdx.x == 0 && threadIdx.x == 0) bad_length(p.err);
    return;
  }
  if (p.new_lens && blockIdx.x == 0 && threadIdx.x == 0) p.new_lens[b] = len + kept;
  // path[i] = i holds up to some i and for none after it
  __shared__ int s_same[kThreadsRows / 32];
  same = __reduce_add_sync(0xffffffffu, same);
  if ((threadIdx.x & 31) == 0) s_same[threadIdx.x >> 5] = same;
  __syncthreads();
  int first = 0;
#pragma unroll
  for (int w = 0; w < kThreadsRows / 32; ++w) first += s_same[w];
  const int per = p.heads * p.units;  // columns of a cache's slot
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kThreadsRows + threadIdx.x;
  if (c >= static_cast<int64_t>(p.n) * per) return;
  const int cache = static_cast<int>(c / per), in = static_cast<int>(c - static_cast<int64_t>(cache) * per);
  const int head = in / p.units, unit = in - head * p.units;
  uint4* row0 = p.data[cache] + ((static_cast<int64_t>(b) * p.heads + head) * p.rows + len) * p.units + unit;
#pragma unroll 1
  for (int i0 = first; i0 < kept; i0 += kRowsKeep) {
    uint4 x[kRowsKeep];
#pragma unroll
    for (int i = 0; i < kRowsKeep; ++i)
      if (i0 + i < kept) x[i] = row0[static_cast<int64_t>(s_path[i0 + i]) * p.units];
#pragma unroll
    for (int i = 0; i < kRowsKeep; ++i)
      if (i0 + i < kept) row0[static_cast<int64_t>(i0 + i) * p.units] = x[i];
  }
}

struct ForkParams {
  int slots, from_slots, heads, rows, from_rows, units, blocks;  // blocks: of each run
  int same;                                                      // `to` is `from`
  const int32_t* src;
  const int32_t* lens;
  int32_t* new_lens;
  int64_t* err;
  const uint4* from[STOF_CACHES_MAX];
  uint4* to[STOF_CACHES_MAX];
};

constexpr int kThreadsFork = 256, kLoads = 4;              // 16-byte loads in flight per thread
constexpr int kPiece = kThreadsFork * kLoads;              // 16-byte units of a piece

__global__ void __launch_bounds__(kThreadsFork) fork_kernel(const __grid_constant__ ForkParams p) {
  const int b = static_cast<int>(blockIdx.x % p.slots);
  const int64_t rest = blockIdx.x / p.slots;  // (cache, head, block of the run)
  const int part = static_cast<int>(rest % p.blocks);
  const int plane = static_cast<int>(rest / p.blocks), cache = plane / p.heads, head = plane - cache * p.heads;
  const int s = __ldg(p.src + b);
  const bool first = rest == 0;  // the slot's first block
  if (s < 0) return;
  const bool stays = p.same && s == b;
  bool bad = s >= p.from_slots;
  if (p.same && !stays) {  // is the slot one that others are copied from?
    bool read = false;
    for (int i = threadIdx.x; i < p.slots; i += kThreadsFork) read |= i != b && __ldg(p.src + i) == b;
    bad = __syncthreads_or(bad || read);
  }
  const int len = bad ? 0 : p.lens[s];
  if (bad || len < 0 || len > p.rows || len > p.from_rows) {
    if (first && threadIdx.x == 0) bad_length(p.err);
    return;
  }
  if (first && threadIdx.x == 0 && p.new_lens) p.new_lens[b] = len;
  if (stays) return;
  const uint4* from = p.from[cache] + (static_cast<int64_t>(s) * p.heads + head) * p.from_rows * p.units;
  uint4* to = p.to[cache] + (static_cast<int64_t>(b) * p.heads + head) * p.rows * p.units;
  const int64_t n = static_cast<int64_t>(len) * p.units;
#pragma unroll 1
  for (int64_t x0 = static_cast<int64_t>(part) * kPiece + threadIdx.x; x0 < n; x0 += static_cast<int64_t>(p.blocks) * kPiece) {
    uint4 x[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      if (x0 + i * kThreadsFork < n) x[i] = from[x0 + i * kThreadsFork];
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      if (x0 + i * kThreadsFork < n) to[x0 + i * kThreadsFork] = x[i];
  }
}

// What is wrong with a set of caches.
stof_status check_caches(const stof_caches* c) {
  if (!c || !c->data || c->n < 1 || c->slots < 1 || c->heads < 1 || c->rows < 1 || c->d < 1) return STOF_ERR_INVALID_ARG;
  if (c->n > STOF_CACHES_MAX || c->d % 8 || c->d > 1024) return STOF_ERR_UNSUPPORTED;
  // a slot's columns of all caches, and a cache's heads, are counted in 32 bits
  if (static_cast<int64_t>(c->n) * c->heads * (c->d / 8) >= (1ll << 31)) return STOF_ERR_SHAPE;
  for (int i = 0; i < c->n; ++i) {
    if (!c->data[i]) return STOF_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(c->data[i]) % 16) return STOF_ERR_ALIGNMENT;
  }
  return STOF_OK;
}

// A set's addresses in ascending order (a program's caches mostly are).
struct Sorted {
  uintptr_t at[STOF_CACHES_MAX];
  int n;
  unsigned __int128 bytes;  // of a cache
  explicit Sorted(const stof_caches* c) : n(c->n) {
    bytes = static_cast<unsigned __int128>(c->slots) * c->heads * c->d * 2 * static_cast<unsigned>(c->rows);
    for (int i = 0; i < n; ++i) at[i] = reinterpret_cast<uintptr_t>(c->data[i]);
    if (!std::is_sorted(at, at + n)) std::sort(at, at + n);
  }
  // Whether two of the set share bytes: their rows would be moved by several threads in no order.
  bool overlapping() const {
    for (int i = 1; i < n; ++i)
      if (at[i] - at[i - 1] < bytes) return true;
    return false;
  }
};

// Whether a cache of one set shares bytes with one of the other.  The one that
// begins first either reaches into the other's first or ends before all of them.
// (All pairs took 20.6 us for two sets of 160 caches.)
bool overlap(const Sorted& a, const Sorted& b) {
  for (int i = 0, j = 0; i < a.n && j < b.n;) {
    const uintptr_t x = a.at[i], y = b.at[j];
    if (x < y ? y - x < a.bytes : x - y < b.bytes) return true;
    x < y ? ++i : ++j;
  }
  return false;
}

}  // namespace
}  // namespace stof

using namespace stof;

extern "C" stof_status stof_cache_keep(const stof_caches* caches, int T, const int32_t* lens, const int32_t* path,
                                       const int32_t* kept, int32_t* new_lens, int64_t* device_error, void* stream) {
  const stof_status st = check_caches(caches);
  if (st != STOF_OK) return st;
  if (!lens || !path || !kept || T < 1 || new_lens == lens || (new_lens && new_lens == kept)) return STOF_ERR_INVALID_ARG;
  if (T > STOF_TREE_MAX_TOKENS || caches->slots > 65535) return STOF_ERR_SHAPE;
  if (Sorted(caches).overlapping()) return STOF_ERR_INVALID_ARG;
  const uintptr_t words = reinterpret_cast<uintptr_t>(lens) | reinterpret_cast<uintptr_t>(path) |
                          reinterpret_cast<uintptr_t>(kept) | reinterpret_cast<uintptr_t>(new_lens);
  if (words % 4 || reinterpret_cast<uintptr_t>(device_error) % 8) return STOF_ERR_ALIGNMENT;
  KeepParams p;
  p.T = T;
  p.heads = caches->heads;
  p.rows = caches->rows;
  p.units = caches->d / 8;
  p.n = caches->n;
  p.lens = lens;
  p.path = path;
  p.kept = kept;
  p.new_lens = new_lens;
  p.err = device_error;
  for (int i = 0; i < caches->n; ++i) p.data[i] = static_cast<uint4*>(caches->data[i]);
  const int64_t columns = static_cast<int64_t>(p.n) * p.heads * p.units;
  const dim3 grid(static_cast<unsigned>((columns + kThreadsRows - 1) / kThreadsRows), static_cast<unsigned>(caches->slots));
  keep_kernel<<<grid, kThreadsRows, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return record_cuda(cudaGetLastError()) == cudaSuccess ? STOF_OK : STOF_ERR_CUDA;
}

extern "C" stof_status stof_cache_fork(const stof_caches* from, const stof_caches* to, const int32_t* src,
                                       const int32_t* lens, int32_t* new_lens, int64_t* device_error, void* stream) {
  stof_status st = check_caches(from);
  if (st == STOF_OK) st = check_caches(to);
  if (st != STOF_OK) return st;
  if (!src || !lens || new_lens == src) return STOF_ERR_INVALID_ARG;
  if (from->n != to->n || from->heads != to->heads || from->d != to->d) return STOF_ERR_SHAPE;
  int equal = 0;
  for (int i = 0; i < from->n; ++i) equal += from->data[i] == to->data[i];
  if (equal && (equal != from->n || from->slots != to->slots || from->rows != to->rows)) return STOF_ERR_INVALID_ARG;
  const Sorted sources(from);
  if (sources.overlapping()) return STOF_ERR_INVALID_ARG;
  if (!equal) {
    const Sorted places(to);
    if (new_lens == lens || places.overlapping() || overlap(sources, places)) return STOF_ERR_INVALID_ARG;
  }
  const uintptr_t words = reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(lens) |
                          reinterpret_cast<uintptr_t>(new_lens);
  if (words % 4 || reinterpret_cast<uintptr_t>(device_error) % 8) return STOF_ERR_ALIGNMENT;
  ForkParams p;
  p.slots = to->slots;
  p.from_slots = from->slots;
  p.heads = to->heads;
  p.rows = to->rows;
  p.from_rows = from->rows;
  p.units = to->d / 8;
  p.same = equal != 0;
  p.src = src;
  p.lens = lens;
  p.new_lens = new_lens;
  p.err = device_error;
  for (int i = 0; i < from->n; ++i) {
    p.from[i] = static_cast<const uint4*>(from->data[i]);
    p.to[i] = static_cast<uint4*>(to->data[i]);
  }
  // Blocks of a run: as many as its longest has pieces, but no more than give
  // the SMs 64 blocks each in all (the lengths are on the device, and blocks
  // past a run's end only read its length).
  const int64_t runs = static_cast<int64_t>(p.slots) * p.heads * from->n;
  const int longest = p.rows < p.from_rows ? p.rows : p.from_rows;
  const int64_t pieces = (static_cast<int64_t>(longest) * p.units + kPiece - 1) / kPiece;
  const int64_t want = (64ll * device_sm_count() + runs - 1) / runs;
  const int64_t blocks = pieces < want ? pieces : want;
  if (runs * blocks >= (1ll << 31)) return STOF_ERR_SHAPE;
  p.blocks = static_cast<int>(blocks);
  fork_kernel<<<static_cast<unsigned>(runs * blocks), kThreadsFork, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return record_cuda(cudaGetLastError()) == cudaSuccess ? STOF_OK : STOF_ERR_CUDA;
}
