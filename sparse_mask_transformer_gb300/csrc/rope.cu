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
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

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

// WIDE: a unit is 8 pairs (2 x 16 bytes of the two halves) or, interleaved, 4
// pairs (16 bytes), moved by 16-byte accesses; else one pair by 2-byte ones.
template <bool BF16, bool INTER, bool WIDE>
__global__ void __launch_bounds__(kThreadsRope, kBlocksRope) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int PAIRS = WIDE ? (INTER ? 4 : 8) : 1;  // pairs per unit
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
  const int64_t pos = p.positions ? static_cast<int64_t>(__ldg(p.positions + token)) : row;
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
  for (int i = 0; i < PAIRS; ++i) angle(p, unit * PAIRS + i, pos, c[i], s[i]);

  if constexpr (WIDE) {
    // first element of the unit's first 16 bytes, and of its second (halves)
    const int e0 = unit * 8, e1 = p.rot / 2 + e0;
    for (int h0 = slot; h0 < heads; h0 += p.slots * kBatch) {
      uint4 x[kBatch], y[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int h = h0 + i * p.slots;
        if (h < heads) {
          x[i] = *reinterpret_cast<const uint4*>(src(h) + e0);
          if constexpr (!INTER) y[i] = *reinterpret_cast<const uint4*>(src(h) + e1);
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int h = h0 + i * p.slots;
        if (h >= heads) break;
        uint32_t xw[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        if constexpr (INTER) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float2 a = widen2<BF16>(xw[w]);
            xw[w] = narrow2<BF16>(a.x * c[w] - a.y * s[w], a.y * c[w] + a.x * s[w]);
          }
          *reinterpret_cast<uint4*>(dst(h) + e0) = make_uint4(xw[0], xw[1], xw[2], xw[3]);
        } else {
          uint32_t yw[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float2 a = widen2<BF16>(xw[w]), g = widen2<BF16>(yw[w]);
            xw[w] = narrow2<BF16>(a.x * c[2 * w] - g.x * s[2 * w], a.y * c[2 * w + 1] - g.y * s[2 * w + 1]);
            yw[w] = narrow2<BF16>(g.x * c[2 * w] + a.x * s[2 * w], g.y * c[2 * w + 1] + a.y * s[2 * w + 1]);
          }
          *reinterpret_cast<uint4*>(dst(h) + e0) = make_uint4(xw[0], xw[1], xw[2], xw[3]);
          *reinterpret_cast<uint4*>(dst(h) + e1) = make_uint4(yw[0], yw[1], yw[2], yw[3]);
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
  constexpr int E = WIDE ? 8 : 1;  // elements per copy
  using Unit = std::conditional_t<WIDE, uint4, uint16_t>;
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

bool wide_rows(const Rows& r) {
  return reinterpret_cast<uintptr_t>(r.data) % 16 == 0 && r.sb % 8 == 0 && r.sh % 8 == 0 && r.st % 8 == 0;
}

template <bool BF16, bool INTER, bool WIDE>
cudaError_t launch(RopeParams& p, long long tokens, cudaStream_t s) {
  constexpr int PAIRS = WIDE ? (INTER ? 4 : 8) : 1;
  const long long units = p.rot / 2 / PAIRS, heads = p.H + p.Hkv;
  // Head slots per token: as few as come near the 1024 threads per SM that
  // are resident (an angle is then computed for as many heads as can be), up
  // to a thread per head when there are few tokens.  16384 tokens, 40 heads of
  // 128: 1 slot 71.6 us, 2 slots 67.5, 4 slots 69.8, 8 slots 73.8.
  const long long want = 870ll * device_sm_count();
  long long slots = (want + tokens * units - 1) / (tokens * units);
  if (slots > heads) slots = heads;
  // as many heads for every slot where a number up to twice as large divides them (3 slots for 32 heads: 41.5 us, 4: 36.2)
  for (long long more = slots; more <= 2 * slots; ++more) {
    if (heads % more == 0) {
      slots = more;
      break;
    }
  }
  p.slots = static_cast<int>(slots);
  p.n_threads = static_cast<uint32_t>(tokens * units * slots);
  const unsigned grid = static_cast<unsigned>((tokens * units * slots + kThreadsRope - 1) / kThreadsRope);
  rope_kernel<BF16, INTER, WIDE><<<grid, kThreadsRope, 0, s>>>(p);
  return cudaGetLastError();
}

template <bool BF16>
cudaError_t launch_t(RopeParams& p, bool inter, bool wide, long long tokens, cudaStream_t s) {
  if (inter) return wide ? launch<BF16, true, true>(p, tokens, s) : launch<BF16, true, false>(p, tokens, s);
  return wide ? launch<BF16, false, true>(p, tokens, s) : launch<BF16, false, false>(p, tokens, s);
}

bool plan_ok(const stof_rope_plan* plan) {
  return plan && plan->made == 1 && plan->rot_dim >= 2 && plan->rot_dim <= 2 * STOF_ROPE_MAX_PAIRS &&
         plan->rot_dim % 2 == 0 && (plan->interleaved == 0 || plan->interleaved == 1) && std::isfinite(plan->amplitude);
}

stof_status rope_call(const stof_rope_plan* plan, const stof_rope_rows* x, stof_dtype dt, int B, int H, int Hkv, int T, int d,
                      const int32_t* positions, const int32_t* counts, const int32_t* rows, int kv_rows, bool backward,
                      int64_t* err, void* stream) {
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
  RopeParams p;
  std::memset(&p, 0, sizeof(p));
  bool wide = d % 8 == 0 && plan->rot_dim % (plan->interleaved ? 8 : 16) == 0;
  const stof_rows* in[6] = {&x->q, &x->k, &x->v, &x->q_out, &x->k_out, &x->v_out};
  Rows* to[6] = {&p.q, &p.k, &p.v, &p.qo, &p.ko, &p.vo};
  for (int i = 0; i < 6; ++i) {
    if (!in[i]->data) continue;
    if (reinterpret_cast<uintptr_t>(in[i]->data) % 2) return STOF_ERR_ALIGNMENT;
    *to[i] = Rows{static_cast<uint16_t*>(in[i]->data), in[i]->stride_b, in[i]->stride_h, in[i]->stride_t};
    wide = wide && wide_rows(*to[i]);
  }
  const uintptr_t words = reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(counts) |
                          reinterpret_cast<uintptr_t>(rows);
  if (words % 4 || reinterpret_cast<uintptr_t>(err) % 8) return STOF_ERR_ALIGNMENT;
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
  const bool inter = plan->interleaved != 0;
  const cudaError_t e = dt == STOF_BF16 ? launch_t<true>(p, inter, wide, tokens, s) : launch_t<false>(p, inter, wide, tokens, s);
  return record_cuda(e) == cudaSuccess ? STOF_OK : STOF_ERR_CUDA;
}

constexpr double kTwoPi = 6.283185307179586476925286766559;

// An angle per position (radians) in units of 2^-64 turns.  A product with a
// whole position only needs the turn modulo 1.
uint64_t step_of(double radians) {
  const double turns = radians / kTwoPi;
  const double f = turns - std::floor(turns);
  return f >= 1.0 ? 0 : static_cast<uint64_t>(std::ldexp(f, 64));
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
  return rope_call(plan, x, dt, B, H, Hkv, T, d, positions, counts, rows, kv_rows, false, device_error, stream);
}

extern "C" stof_status stof_rope_bwd(const stof_rope_plan* plan, const stof_rope_rows* x, stof_dtype dt, int B, int H,
                                     int Hkv, int T, int d, const int32_t* positions, const int32_t* counts, void* stream) {
  return rope_call(plan, x, dt, B, H, Hkv, T, d, positions, counts, nullptr, T, true, nullptr, stream);
}
