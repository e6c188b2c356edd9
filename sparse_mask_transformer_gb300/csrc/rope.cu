// Rotary positions on Q and K, with the move between the projection's layout
// and the attention's (or a K/V cache), forward and gradient.
//
// Every pair (x_a, x_c) of a head's first rot_dim elements is turned by
// phi = position * w_p:
//   y_a = A (x_a cos phi - x_c sin phi),  y_c = A (x_c cos phi + x_a sin phi),
// and the gradient is the turn by -phi.  A turn is a fraction of 2^64
// (plan.step), so position * step wraps modulo 2^64 exactly as the angle
// wraps modulo a turn: the reduced angle carries no rounding at any position,
// where an fp32 product of position and frequency has lost 2^-24 of it (half a
// radian at position 10^7).  Its top 32 bits, as a signed fraction of a half turn, go
// through sincospif.
//
// Bound by memory: 4 bytes per element and 3 operations per turned one.  A
// thread owns 8 pairs of one token (16 bytes of each half; 4 pairs, 16 bytes,
// if interleaved), computes their angles once and turns
// those elements of every `slots`-th head, kBatch heads in flight at a time.
// V rows and elements past rot_dim are copied by the same threads.
//
// With several axes (stof_rope_axes_fwd, stof_rope_axes_bwd) each pair has the
// position of its own axis; a thread reads the position of each of its pairs,
// most of them in the L1 cache already.  16384 tokens, 48 heads of 128: 69.7 us,
// 5.8 TB/s, 85% of the copy rate, as with one axis.  Angles computed once per
// block into shared memory, for all heads of one to eight tokens: 74.0 us (a
// gradient of 32 heads of 64, 29.0 instead of 25.1): short blocks wait for
// their angles.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "internal.h"

namespace stof {
namespace {

constexpr int kThreadsRope = 256;
// Heads in flight per thread and blocks per SM: the product of loads in flight
// is what counts.  16384 tokens: 4 heads x 2 blocks 73.2 us, 2 x 4 67.6, 2 x 5
// (spills) 91.6, 1 x 6 80.0.
constexpr int kBatch = 2, kBlocksRope = 4;
constexpr int kCopies = 4;  // copies in flight per thread

struct Rows {
  uint16_t* data;
  int64_t sb, sh, st;
};

struct RopeParams {
  Rows q, k, v, qo, ko, vo;
  int H, Hkv, T, d, rot;   // H = 0: no q; Hkv = 0: no k
  int has_v;
  int slots;               // head slots per token
  uint32_t n_threads;
  const int32_t* positions;
  const int32_t* counts;
  const int32_t* rows;
  int kv_rows;
  int64_t* err;
  float amplitude, sin_amplitude;  // A and +-A
  uint64_t step[STOF_ROPE_MAX_PAIRS];
};

// Positions with several axes: positions is [n_axes][tokens].
struct AxesParams : RopeParams {
  int64_t tokens;
  uint8_t axis[STOF_ROPE_MAX_PAIRS];  // of each pair
};

template <bool BF16>
__device__ __forceinline__ float widen(uint32_t bits) {
  if constexpr (BF16)
    return __uint_as_float(bits << 16);
  else
    return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
}
template <bool BF16>
__device__ __forceinline__ float2 widen2(uint32_t u) {
  if constexpr (BF16)
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
template <bool BF16>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
  if constexpr (BF16) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  } else {
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  }
}

// Cosine and sine (times the amplitude) of pair p at position pos.
__device__ __forceinline__ void angle(const RopeParams& p, int pair, int64_t pos, float& c, float& s) {
  const uint64_t turn = static_cast<uint64_t>(pos) * p.step[pair];
  const float half_turns = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
  sincospif(half_turns, &s, &c);
  c *= p.amplitude;
  s *= p.sin_amplitude;
}

// Accesses of E elements: of 8 (16 bytes) a unit is 8 pairs (one access in
// each of the two halves) or, interleaved, 4 pairs (one access); of 4 half as
// many pairs; of one (E = 1) one pair.
template <int E, bool INTER>
constexpr int kPairs = E == 1 ? 1 : (INTER ? E / 2 : E);
template <int E>
using Access = std::conditional_t<E == 8, uint4, std::conditional_t<E == 4, uint2, uint16_t>>;

template <bool BF16, bool INTER, int E, class PARAMS>
__global__ void __launch_bounds__(kThreadsRope, kBlocksRope) rope_kernel(const __grid_constant__ PARAMS p) {
  constexpr bool AXES = std::is_same<PARAMS, AxesParams>::value;
  constexpr int PAIRS = kPairs<E, INTER>;  // pairs per unit
  using Unit = Access<E>;
  const uint32_t tid = blockIdx.x * kThreadsRope + threadIdx.x;
  if (tid >= p.n_threads) return;
  const uint32_t units = static_cast<uint32_t>(p.rot / 2) / PAIRS;
  const uint32_t per_token = units * p.slots;
  const uint32_t token = tid / per_token, in_token = tid - token * per_token;
  const int slot = static_cast<int>(in_token / units), unit = static_cast<int>(in_token - slot * units);
  const int b = static_cast<int>(token / p.T), t = static_cast<int>(token - static_cast<uint32_t>(b) * p.T);
  if (p.counts && t >= __ldg(p.counts + b)) return;
  const int64_t row0 = p.rows ? __ldg(p.rows + b) : 0;
  const int64_t row = row0 + t;  // row of this token in k_out and v_out
  const int64_t pos = !AXES && p.positions ? static_cast<int64_t>(__ldg(p.positions + token)) : row;
  int heads = p.H + p.Hkv;
  bool kv = p.Hkv > 0;
  if (kv && (row < 0 || row >= p.kv_rows)) {  // the request's K and V are not written
    if (in_token == 0 && p.err)
      atomicOr(reinterpret_cast<unsigned long long*>(p.err), static_cast<unsigned long long>(STOF_DEVERR_BAD_LENGTH));
    kv = false;
    heads = p.H;
  }
  const uint16_t* q = p.q.data + b * p.q.sb + t * p.q.st;
  uint16_t* qo = p.qo.data + b * p.qo.sb + t * p.qo.st;
  const uint16_t* k = p.k.data + b * p.k.sb + t * p.k.st;
  uint16_t* ko = p.ko.data + b * p.ko.sb + row * p.ko.st;
  // row of head h: the first H heads are Q's, the others K's
  auto src = [&](int h) { return h < p.H ? q + h * p.q.sh : k + (h - p.H) * p.k.sh; };
  auto dst = [&](int h) { return h < p.H ? qo + h * p.qo.sh : ko + (h - p.H) * p.ko.sh; };

  float c[PAIRS], s[PAIRS];
#pragma unroll
  for (int i = 0; i < PAIRS; ++i) {
    const int pair = unit * PAIRS + i;
    if constexpr (AXES)
      angle(p, pair, __ldg(p.positions + p.axis[pair] * p.tokens + token), c[i], s[i]);
    else
      angle(p, pair, pos, c[i], s[i]);
  }

  if constexpr (E > 1) {
    // first element of the unit's first access, and of its second (halves)
    const int e0 = unit * E, e1 = p.rot / 2 + e0;
    for (int h0 = slot; h0 < heads; h0 += p.slots * kBatch) {
      Unit x[kBatch], y[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int h = h0 + i * p.slots;
        if (h < heads) {
          x[i] = *reinterpret_cast<const Unit*>(src(h) + e0);
          if constexpr (!INTER) y[i] = *reinterpret_cast<const Unit*>(src(h) + e1);
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int h = h0 + i * p.slots;
        if (h >= heads) break;
        uint32_t* xw = reinterpret_cast<uint32_t*>(&x[i]);  // two elements a word
        if constexpr (INTER) {
#pragma unroll
          for (int w = 0; w < E / 2; ++w) {
            const float2 a = widen2<BF16>(xw[w]);
            xw[w] = narrow2<BF16>(a.x * c[w] - a.y * s[w], a.y * c[w] + a.x * s[w]);
          }
          *reinterpret_cast<Unit*>(dst(h) + e0) = x[i];
        } else {
          uint32_t* yw = reinterpret_cast<uint32_t*>(&y[i]);
#pragma unroll
          for (int w = 0; w < E / 2; ++w) {
            const float2 a = widen2<BF16>(xw[w]), g = widen2<BF16>(yw[w]);
            xw[w] = narrow2<BF16>(a.x * c[2 * w] - g.x * s[2 * w], a.y * c[2 * w + 1] - g.y * s[2 * w + 1]);
            yw[w] = narrow2<BF16>(g.x * c[2 * w] + a.x * s[2 * w], g.y * c[2 * w + 1] + a.y * s[2 * w + 1]);
          }
          *reinterpret_cast<Unit*>(dst(h) + e0) = x[i];
          *reinterpret_cast<Unit*>(dst(h) + e1) = y[i];
        }
      }
    }
  } else {
    const int e0 = INTER ? 2 * unit : unit, e1 = INTER ? e0 + 1 : p.rot / 2 + unit;
    for (int h = slot; h < heads; h += p.slots) {
      const float a = widen<BF16>(src(h)[e0]), g = widen<BF16>(src(h)[e1]);
      const uint32_t w = narrow2<BF16>(a * c[0] - g * s[0], g * c[0] + a * s[0]);
      dst(h)[e0] = static_cast<uint16_t>(w & 0xFFFFu);
      dst(h)[e1] = static_cast<uint16_t>(w >> 16);
    }
  }

  // what is only copied: the elements past rot of Q's and K's heads, and V
  // n copies of E elements, `from` and `to` giving the places of copy x
  auto copy_all = [&](uint32_t n, auto&& from, auto&& to) {
    for (uint32_t x0 = in_token; x0 < n; x0 += per_token * kCopies) {
      Unit u[kCopies];
#pragma unroll
      for (int i = 0; i < kCopies; ++i)
        if (x0 + i * per_token < n) u[i] = *reinterpret_cast<const Unit*>(from(x0 + i * per_token));
#pragma unroll
      for (int i = 0; i < kCopies; ++i)
        if (x0 + i * per_token < n) *reinterpret_cast<Unit*>(to(x0 + i * per_token)) = u[i];
    }
  };
  const uint32_t rest = static_cast<uint32_t>(p.d - p.rot) / E;
  if (rest) {
    copy_all(
        rest * heads,
        [&](uint32_t x) { return src(static_cast<int>(x / rest)) + p.rot + x % rest * E; },
        [&](uint32_t x) { return dst(static_cast<int>(x / rest)) + p.rot + x % rest * E; });
  }
  if (p.has_v && kv) {
    const uint16_t* v = p.v.data + b * p.v.sb + t * p.v.st;
    uint16_t* vo = p.vo.data + b * p.vo.sb + row * p.vo.st;
    const uint32_t per_head = static_cast<uint32_t>(p.d) / E;
    copy_all(
        per_head * p.Hkv, [&](uint32_t x) { return v + static_cast<int64_t>(x / per_head) * p.v.sh + x % per_head * E; },
        [&](uint32_t x) { return vo + static_cast<int64_t>(x / per_head) * p.vo.sh + x % per_head * E; });
  }
}

// Whether a row's elements can be taken e at a time.
bool rows_of(const Rows& r, int e) {
  return reinterpret_cast<uintptr_t>(r.data) % (2 * e) == 0 && r.sb % e == 0 && r.sh % e == 0 && r.st % e == 0;
}

// Head slots per token, one axis: as few as come near the 1024 threads per SM
// that are resident (an angle is then computed for as many heads as can be), up
// to a thread per head when there are few tokens.  16384 tokens, 40 heads of
// 128: 1 slot 71.6 us, 2 slots 67.5, 4 slots 69.8, 8 slots 73.8.
long long slots_of(const RopeParams& p, long long tokens, long long units, int) {
  const long long want = 870ll * device_sm_count(), heads = p.H + p.Hkv;
  long long slots = (want + tokens * units - 1) / (tokens * units);
  if (slots > heads) slots = heads;
  // as many heads for every slot where a number up to twice as large divides them (3 slots for 32 heads: 41.5 us, 4: 36.2)
  for (long long more = slots; more <= 2 * slots; ++more) {
    if (heads % more == 0) {
      slots = more;
      break;
    }
  }
  return slots;
}

// Several axes.  The most slots that the resident threads hold are best, and a
// little more than that is a second round of a few blocks, the worst.  Over 161
// calls of 16 to 65536 tokens, all access widths and parts of heads turned, each
// timed with 1 to 32 slots, the rule is 4% over the best number of slots in the
// mean and 30% at most (6000 tokens of 40 heads of 128, half turned: 7 slots 42.5
// us, 6 32.7).
// - One wave of the resident threads where it holds two slots or more: 9805
//   tokens of 32 heads of 64, 3 slots (0.76 waves) 24.1 us, 4 (1.01) 27.3; 10500:
//   25.1, (1.08) 28.2; 12500: 28.5, (1.28) 31.3; 4096 of 72, 4 (0.95) 15.2, 5
//   (1.18) 19.6, 16 (3.8) 21.6; 14000 of 64, 2 (0.72) 31.3, 4 (1.44) 32.8.
// - Else a wave and a half or more: 24000 of 64, 1 slot (0.62) 52.0, 2 (1.23)
//   55.1, 3 (1.85) 50.5; 16384 of 128, 1 (0.84) 75.3, 2 (1.68) 68.3, 4 68.7; 16384
//   of 72, 1 (0.95) 47.4, 2 47.4, 4 50.2.
// - At most kCopiesMost copies a thread of what is not turned, 16: 24000 tokens
//   of 40 heads of 128, half of each turned, 2 slots (56 copies) 139, 4 119, 8 109;
//   16384 of 32 heads of 80, half turned, 4 (32) 67.9, 8 59.0, 16 62.3; V alone, 16384
//   of 72, 1 slot (32) 47.4, 2 47.4, 3 50.5.
// - No more slots than give a thread that many heads: 1000 tokens of 32 heads of
//   72, 24 slots 9.9 us, 16 7.5.
constexpr long long kCopiesMost = 16;
long long slots_of(const AxesParams& p, long long tokens, long long units, int e) {
  const long long wave = static_cast<long long>(kThreadsRope) * kBlocksRope * device_sm_count(), n = tokens * units;
  const long long heads = p.H + p.Hkv;
  const long long copies = (p.d - p.rot) / e * heads + (p.has_v ? p.d / e * static_cast<long long>(p.Hkv) : 0);
  long long slots = wave / n;
  if (slots < 2) slots = (3 * wave + 2 * n - 1) / (2 * n);
  slots = std::max(slots, (copies + kCopiesMost * units - 1) / (kCopiesMost * units));
  slots = std::max(1ll, std::min({slots, heads, ((1ll << 31) - 1) / n}));  // threads are counted in 32 bits
  const long long each = (heads + slots - 1) / slots;
  return (heads + each - 1) / each;
}

template <bool BF16, bool INTER, int E, class PARAMS>
cudaError_t launch(PARAMS& p, long long tokens, cudaStream_t s) {
  const long long units = p.rot / 2 / kPairs<E, INTER>, slots = slots_of(p, tokens, units, E);
  p.slots = static_cast<int>(slots);
  p.n_threads = static_cast<uint32_t>(tokens * units * slots);
  const unsigned grid = static_cast<unsigned>((tokens * units * slots + kThreadsRope - 1) / kThreadsRope);
  rope_kernel<BF16, INTER, E><<<grid, kThreadsRope, 0, s>>>(p);
  return cudaGetLastError();
}

template <bool BF16, bool INTER, class PARAMS>
cudaError_t launch_e(PARAMS& p, int e, long long tokens, cudaStream_t s) {
  if (e == 8) return launch<BF16, INTER, 8>(p, tokens, s);
  if constexpr (std::is_same<PARAMS, AxesParams>::value)
    if (e == 4) return launch<BF16, INTER, 4>(p, tokens, s);
  return launch<BF16, INTER, 1>(p, tokens, s);
}
template <class PARAMS>
cudaError_t launch_t(PARAMS& p, bool bf16, bool inter, int e, long long tokens, cudaStream_t s) {
  if (bf16) return inter ? launch_e<true, true>(p, e, tokens, s) : launch_e<true, false>(p, e, tokens, s);
  return inter ? launch_e<false, true>(p, e, tokens, s) : launch_e<false, false>(p, e, tokens, s);
}

bool plan_ok(const stof_rope_plan* plan) {
  return plan && plan->made == 1 && plan->rot_dim >= 2 && plan->rot_dim <= 2 * STOF_ROPE_MAX_PAIRS &&
         plan->rot_dim % 2 == 0 && (plan->interleaved == 0 || plan->interleaved == 1) && std::isfinite(plan->amplitude);
}

// axes: null for positions with one axis.
stof_status rope_call(const stof_rope_plan* plan, const stof_rope_axes* axes, const stof_rope_rows* x, stof_dtype dt, int B,
                      int H, int Hkv, int T, int d, const int32_t* positions, const int32_t* counts, const int32_t* rows,
                      int kv_rows, bool backward, int64_t* err, void* stream) {
  if (!plan_ok(plan) || !x) return STOF_ERR_INVALID_ARG;
  if (dt != STOF_F16 && dt != STOF_BF16) return STOF_ERR_DTYPE;
  if (B < 0 || T < 0 || H < 0 || Hkv < 0 || d < 1 || kv_rows < 0) return STOF_ERR_INVALID_ARG;
  const long long tokens = static_cast<long long>(B) * T;
  // (without tokens the inputs have no memory, and may be null beside the caches they would go to)
  if (tokens && (!x->q.data != !x->q_out.data || !x->k.data != !x->k_out.data || !x->v.data != !x->v_out.data))
    return STOF_ERR_INVALID_ARG;
  if (tokens && x->v.data && !x->k.data) return STOF_ERR_INVALID_ARG;  // V is moved beside K
  if (d > 256 || d % 2) return STOF_ERR_UNSUPPORTED;
  if (plan->rot_dim > d) return STOF_ERR_SHAPE;
  AxesParams p;
  std::memset(&p, 0, sizeof(p));
  const stof_rows* in[6] = {&x->q, &x->k, &x->v, &x->q_out, &x->k_out, &x->v_out};
  Rows* to[6] = {&p.q, &p.k, &p.v, &p.qo, &p.ko, &p.vo};
  for (int i = 0; i < 6; ++i) {
    if (!in[i]->data) continue;
    if (reinterpret_cast<uintptr_t>(in[i]->data) % 2) return STOF_ERR_ALIGNMENT;
    *to[i] = Rows{static_cast<uint16_t*>(in[i]->data), in[i]->stride_b, in[i]->stride_h, in[i]->stride_t};
  }
  const uintptr_t words = reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(counts) |
                          reinterpret_cast<uintptr_t>(rows);
  if (words % 4 || reinterpret_cast<uintptr_t>(err) % 8) return STOF_ERR_ALIGNMENT;
  if (tokens && axes && !positions) return STOF_ERR_INVALID_ARG;
  // elements an access takes: 8, one, or between them (several axes) 4
  auto takes = [&](int e) {
    if (d % e || plan->rot_dim % (plan->interleaved ? e : 2 * e)) return false;
    for (int i = 0; i < 6; ++i)
      if (in[i]->data && !rows_of(*to[i], e)) return false;
    return true;
  };
  const int e = takes(8) ? 8 : (axes && takes(4) ? 4 : 1);
  if (H > (1 << 20) || Hkv > (1 << 20) || tokens * (plan->rot_dim / 2) >= (1ll << 31)) return STOF_ERR_SHAPE;
  p.H = x->q.data ? H : 0;
  p.Hkv = x->k.data ? Hkv : 0;
  p.has_v = x->v.data ? 1 : 0;
  if (tokens == 0 || p.H + p.Hkv == 0) return STOF_OK;  // nothing to turn
  p.T = T;
  p.d = d;
  p.rot = plan->rot_dim;
  p.positions = positions;
  p.counts = counts;
  p.rows = rows;
  p.kv_rows = kv_rows;
  p.err = err;
  p.amplitude = plan->amplitude;
  p.sin_amplitude = backward ? -plan->amplitude : plan->amplitude;
  std::memcpy(p.step, plan->step, sizeof(p.step));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool inter = plan->interleaved != 0, bf16 = dt == STOF_BF16;
  if (!axes)
    return record_cuda(launch_t<RopeParams>(p, bf16, inter, e, tokens, s)) == cudaSuccess ? STOF_OK : STOF_ERR_CUDA;
  p.tokens = tokens;
  std::memcpy(p.axis, axes->axis, sizeof(p.axis));
  return record_cuda(launch_t<AxesParams>(p, bf16, inter, e, tokens, s)) == cudaSuccess ? STOF_OK : STOF_ERR_CUDA;
}

constexpr double kTwoPi = 6.283185307179586476925286766559;

// An angle per position (radians) in units of 2^-64 turns.  A product with a
// whole position only needs the turn modulo 1.
uint64_t step_of(double radians) {
  const double turns = radians / kTwoPi;
  const double f = turns - std::floor(turns);
  return f >= 1.0 ? 0 : static_cast<uint64_t>(std::ldexp(f, 64));
}

bool axes_ok(const stof_rope_axes* a) {
  if (!a || a->made != 1 || !plan_ok(&a->turn) || a->n_axes < 1 || a->n_axes > STOF_ROPE_MAX_AXES) return false;
  for (int i = 0; i < a->turn.rot_dim / 2; ++i)
    if (a->axis[i] >= a->n_axes) return false;
  return true;
}

stof_status plan_start(stof_rope_plan* plan, int rot_dim, int interleaved, double amplitude) {
  if (!plan) return STOF_ERR_INVALID_ARG;
  std::memset(plan, 0, sizeof(*plan));
  if (rot_dim < 2 || rot_dim % 2 || (interleaved != 0 && interleaved != 1)) return STOF_ERR_INVALID_ARG;
  if (rot_dim > 2 * STOF_ROPE_MAX_PAIRS) return STOF_ERR_UNSUPPORTED;
  if (!std::isfinite(static_cast<float>(amplitude))) return STOF_ERR_INVALID_ARG;
  plan->rot_dim = rot_dim;
  plan->interleaved = interleaved;
  plan->amplitude = static_cast<float>(amplitude);
  return STOF_OK;
}

}  // namespace
}  // namespace stof

using namespace stof;

extern "C" stof_status stof_rope_plan_init(stof_rope_plan* plan, int rot_dim, int interleaved, double theta,
                                           stof_rope_scaling scaling, double factor, int64_t original_length,
                                           double turns_lo, double turns_hi, double amplitude) {
  const stof_status st = plan_start(plan, rot_dim, interleaved, amplitude);
  if (st != STOF_OK) return st;
  if (!(theta > 1.0) || !std::isfinite(theta)) return STOF_ERR_INVALID_ARG;
  if (scaling != STOF_ROPE_PLAIN && scaling != STOF_ROPE_LINEAR && scaling != STOF_ROPE_BY_INDEX &&
      scaling != STOF_ROPE_BY_TURNS)
    return STOF_ERR_INVALID_ARG;
  if (scaling != STOF_ROPE_PLAIN && (!(factor > 0.0) || !std::isfinite(factor))) return STOF_ERR_INVALID_ARG;
  const bool ramp = scaling == STOF_ROPE_BY_INDEX || scaling == STOF_ROPE_BY_TURNS;
  if (ramp && (original_length < 1 || !(turns_lo > 0.0) || !(turns_hi > turns_lo) || !std::isfinite(turns_hi)))
    return STOF_ERR_INVALID_ARG;
  double low = 0.0, high = 0.0;  // the pairs between which STOF_ROPE_BY_INDEX ramps
  if (scaling == STOF_ROPE_BY_INDEX) {
    auto pair_of = [&](double turns) {
      return rot_dim * std::log(static_cast<double>(original_length) / (kTwoPi * turns)) / (2.0 * std::log(theta));
    };
    low = std::fmax(std::floor(pair_of(turns_hi)), 0.0);
    high = std::fmin(std::ceil(pair_of(turns_lo)), rot_dim - 1.0);
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double w = std::pow(theta, -2.0 * i / rot_dim);
    double keep = 1.0;  // share of the unscaled frequency
    if (scaling == STOF_ROPE_LINEAR)
      keep = 0.0;
    else if (scaling == STOF_ROPE_BY_INDEX)
      keep = 1.0 - std::fmin(std::fmax((i - low) / std::fmax(high - low, 0.001), 0.0), 1.0);
    else if (scaling == STOF_ROPE_BY_TURNS)
      keep = std::fmin(std::fmax((original_length * w / kTwoPi - turns_lo) / (turns_hi - turns_lo), 0.0), 1.0);
    plan->step[i] = step_of(keep * w + (keep < 1.0 ? (1.0 - keep) * w / factor : 0.0));
  }
  plan->made = 1;
  return STOF_OK;
}

extern "C" stof_status stof_rope_plan_custom(stof_rope_plan* plan, int rot_dim, int interleaved,
                                             const double* frequencies, double amplitude) {
  const stof_status st = plan_start(plan, rot_dim, interleaved, amplitude);
  if (st != STOF_OK) return st;
  if (!frequencies) return STOF_ERR_INVALID_ARG;
  for (int i = 0; i < rot_dim / 2; ++i)
    if (!std::isfinite(frequencies[i])) return STOF_ERR_INVALID_ARG;
  for (int i = 0; i < rot_dim / 2; ++i) plan->step[i] = step_of(frequencies[i]);
  plan->made = 1;
  return STOF_OK;
}

extern "C" stof_status stof_rope_fwd(const stof_rope_plan* plan, const stof_rope_rows* x, stof_dtype dt, int B, int H,
                                     int Hkv, int T, int d, const int32_t* positions, const int32_t* counts,
                                     const int32_t* rows, int kv_rows, int64_t* device_error, void* stream) {
  return rope_call(plan, nullptr, x, dt, B, H, Hkv, T, d, positions, counts, rows, kv_rows, false, device_error, stream);
}

extern "C" stof_status stof_rope_bwd(const stof_rope_plan* plan, const stof_rope_rows* x, stof_dtype dt, int B, int H,
                                     int Hkv, int T, int d, const int32_t* positions, const int32_t* counts, void* stream) {
  return rope_call(plan, nullptr, x, dt, B, H, Hkv, T, d, positions, counts, nullptr, T, true, nullptr, stream);
}

extern "C" stof_status stof_rope_axes_init(stof_rope_axes* axes, const stof_rope_plan* plan, int n_axes,
                                           const int32_t* axis_of_pair) {
  if (!axes) return STOF_ERR_INVALID_ARG;
  stof_rope_plan turn = {};  // the plan may be *axes' own
  if (plan) turn = *plan;
  std::memset(axes, 0, sizeof(*axes));
  if (!plan || !plan_ok(&turn) || !axis_of_pair || n_axes < 1) return STOF_ERR_INVALID_ARG;
  if (n_axes > STOF_ROPE_MAX_AXES) return STOF_ERR_UNSUPPORTED;
  for (int i = 0; i < turn.rot_dim / 2; ++i)
    if (axis_of_pair[i] < 0 || axis_of_pair[i] >= n_axes) return STOF_ERR_INVALID_ARG;
  axes->turn = turn;
  axes->n_axes = n_axes;
  for (int i = 0; i < turn.rot_dim / 2; ++i) axes->axis[i] = static_cast<uint8_t>(axis_of_pair[i]);
  axes->made = 1;
  return STOF_OK;
}

extern "C" stof_status stof_rope_axes_fwd(const stof_rope_axes* axes, const stof_rope_rows* x, stof_dtype dt, int B, int H,
                                          int Hkv, int T, int d, const int32_t* positions, const int32_t* counts,
                                          const int32_t* rows, int kv_rows, int64_t* device_error, void* stream) {
  if (!axes_ok(axes)) return STOF_ERR_INVALID_ARG;
  return rope_call(&axes->turn, axes, x, dt, B, H, Hkv, T, d, positions, counts, rows, kv_rows, false, device_error, stream);
}

extern "C" stof_status stof_rope_axes_bwd(const stof_rope_axes* axes, const stof_rope_rows* x, stof_dtype dt, int B, int H,
                                          int Hkv, int T, int d, const int32_t* positions, const int32_t* counts,
                                          void* stream) {
  if (!axes_ok(axes)) return STOF_ERR_INVALID_ARG;
  return rope_call(&axes->turn, axes, x, dt, B, H, Hkv, T, d, positions, counts, nullptr, T, true, nullptr, stream);
}
