// Capped and distance-lowered scores of a block-wise tile, on the scores of
// one query row that a softmax thread holds in registers: 128 (d = 64) or 64
// (d = 128), or a copy's share of them (see score.cuh for the formulas).
//
// The cap.  A tile whose products all stay within half the cap (scaled), as
// they do in trained models (caps of 30 to 50, scores of a few units), takes
//   log2 e cap tanh(scale s / cap) = s (k1 + t (k3 + t (k5 + t k7))),  t = s^2,
// the odd polynomial of csrc/tanh_poly.py (within 1.3e-7 of the tanh), on the
// FMA pipe in packed pairs: four instructions a pair, the last product folded
// into the subtraction of the running max.  Any other tile takes the exact
// formula with an exponential and a reciprocal of the special-function unit
// for every score, which beside the softmax's own exponential would be the
// kernel's bound for every tile.
// The distance.  Row at position pos, keys of the tile at j0 + i: where no
// warp's row lies among the tile's keys, -slope |pos - j| is linear in i for
// each row and takes a packed addition a pair; else a subtraction and two
// multiply-adds per score.
#pragma once
#include "blockwise_common.cuh"
#include "score.cuh"

namespace stof {
namespace bw {

constexpr float kTanhLimit = 0.5f;  // |scale s / cap| the polynomial is made for
constexpr float kTanh1 = 0x1.ffffb2p-1f, kTanh3 = -0x1.55341ap-2f, kTanh5 = 0x1.0d366cp-3f, kTanh7 = -0x1.634eb0p-5f;

// The call's score constants, in log2 units.
struct ScoreConst {
  float c;               // scale log2 e (no cap)
  float k1, k3, k5, k7;  // the polynomial in s
  float lim;             // |s| up to which it holds; negative: never
  float a, two_a, b;     // the exact form: a + two_a u, u = -1 / (1 + 2^(b s))
  int cap;
};

inline ScoreConst make_score_const(float scale, float softcap) {
  ScoreConst r{};
  const double log2e = 1.4426950408889634;
  r.c = static_cast<float>(scale * log2e);
  r.cap = softcap > 0.f;
  r.lim = -1.f;
  if (r.cap) {
    const double x = static_cast<double>(scale) / softcap, a = softcap * log2e;  // y = x s
    r.a = static_cast<float>(a);
    r.two_a = static_cast<float>(2.0 * a);
    r.b = static_cast<float>(2.0 * log2e * x);
    const double m = x < 0 ? -x : x;
    if (m > 1e-4 && m < 1e4 && a < 1e5) {  // the powers of x stay well inside fp32
      r.k1 = static_cast<float>(a * kTanh1 * x);
      r.k3 = static_cast<float>(a * kTanh3 * x * x * x);
      r.k5 = static_cast<float>(a * kTanh5 * x * x * x * x * x);
      r.k7 = static_cast<float>(a * kTanh7 * x * x * x * x * x * x * x);
      r.lim = static_cast<float>(kTanhLimit / m);
    }
  }
  return r;
}

__device__ __forceinline__ void fmul2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mul.rn.ftz.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// The polynomial's bracket for two products: P(s^2), to be multiplied by s.
__device__ __forceinline__ void cap_bracket(const ScoreConst& k, float s0, float s1, float& p0, float& p1) {
  float t0, t1;
  fmul2(t0, t1, s0, s1, s0, s1);
  ffma2(p0, p1, t0, t1, k.k7, k.k7, k.k5, k.k5);
  ffma2(p0, p1, p0, p1, t0, t1, k.k3, k.k3);
  ffma2(p0, p1, p0, p1, t0, t1, k.k1, k.k1);
}
__device__ __forceinline__ float cap_poly(const ScoreConst& k, float s) {
  const float t = s * s;
  return s * fmaf(fmaf(fmaf(k.k7, t, k.k5), t, k.k3), t, k.k1);
}
__device__ __forceinline__ float cap_exact(const ScoreConst& k, float s) {
  return fmaf(k.two_a, score_rcp(-1.f - score_ex2(k.b * s)), k.a);
}

// Whether every product of the row is within the polynomial's range.  (A NaN
// does not count: it stays NaN either way, until a mask drops it.)
template <int CHUNKS>
__device__ __forceinline__ bool row_within(const uint32_t (&sr)[CHUNKS][32], float lim) {
  float m[CHUNKS];
#pragma unroll
  for (int cc = 0; cc < CHUNKS; ++cc) {
    m[cc] = 0.f;
#pragma unroll
    for (int i = 0; i < 32; i += 2)
      m[cc] = max3(m[cc], fabsf(__uint_as_float(sr[cc][i])), fabsf(__uint_as_float(sr[cc][i + 1])));
  }
  float x = m[0];
#pragma unroll
  for (int cc = 1; cc < CHUNKS; ++cc) x = fmaxf(x, m[cc]);
  return x <= lim;
}

// Capped scores (log2 units) in place.
template <int CHUNKS>
__device__ __forceinline__ void cap_scores(uint32_t (&sr)[CHUNKS][32], const ScoreConst& k, bool within) {
  if (within) {
#pragma unroll
    for (int cc = 0; cc < CHUNKS; ++cc)
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const float s0 = __uint_as_float(sr[cc][i]), s1 = __uint_as_float(sr[cc][i + 1]);
        float p0, p1;
        cap_bracket(k, s0, s1, p0, p1);
        fmul2(p0, p1, p0, p1, s0, s1);
        sr[cc][i] = __float_as_uint(p0);
        sr[cc][i + 1] = __float_as_uint(p1);
      }
  } else {
#pragma unroll
    for (int cc = 0; cc < CHUNKS; ++cc)
#pragma unroll
      for (int i = 0; i < 32; ++i) sr[cc][i] = __float_as_uint(cap_exact(k, __uint_as_float(sr[cc][i])));
  }
}

// sr <- c sr - slope (|pos - (j0 + i)| - base); `base` is the row's reference
// distance (the sources' reference()), no more than any visible key's (slope <
// 0: no less).  A row's softmax does not change when all its scores move by
// slope base, and with it the differences are small where the weights are not.
// They are taken as integers, so that keys 2^30 away differ as near ones do:
// with r the tile's key nearest to the row and e that key's distance,
// |pos - (j0 + i)| - base = |i - r| + (e - base).  A warp-wide call.
template <int CHUNKS>
__device__ __forceinline__ void lower_by_distance(uint32_t (&sr)[CHUNKS][32], float c, float slope, int pos, int j0, uint32_t base) {
  constexpr int N = CHUNKS * 32;
  const bool before = pos >= j0 + N - 1, after = pos <= j0;  // the tile's keys are all before the row, all after it
  const uint32_t rel = static_cast<uint32_t>(pos) - static_cast<uint32_t>(j0);
  const uint32_t e = before ? rel - (N - 1) : (after ? 0u - rel : 0u);
  // e - base, which is more than -N (slope < 0: less than N)
  const float k = slope < 0.f ? N - static_cast<float>(base - e + N) : static_cast<float>(e - base + N) - N;
  if (__all_sync(0xffffffffu, before || after)) {  // |i - r| is linear in i
    const float step = before ? slope : -slope;
    const float at0 = -slope * (before ? k + (N - 1) : k);
#pragma unroll
    for (int cc = 0; cc < CHUNKS; ++cc)
#pragma unroll
      for (int i0 = 0; i0 < 32; i0 += 8) {
        float b0 = fmaf(step, static_cast<float>(cc * 32 + i0), at0), b1 = b0 + step;
        const float two = 2.f * step;
#pragma unroll
        for (int i = i0; i < i0 + 8; i += 2) {
          float x0, x1;
          ffma2(x0, x1, __uint_as_float(sr[cc][i]), __uint_as_float(sr[cc][i + 1]), c, c, b0, b1);
          sr[cc][i] = __float_as_uint(x0);
          sr[cc][i + 1] = __float_as_uint(x1);
          fadd2(b0, b1, two, two);
        }
      }
  } else {
    const float r = before ? N - 1.f : (after ? 0.f : static_cast<float>(static_cast<int>(rel))), at0 = -slope * k;
#pragma unroll
    for (int cc = 0; cc < CHUNKS; ++cc)
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float x = fmaf(__uint_as_float(sr[cc][i]), c, at0);
        sr[cc][i] = __float_as_uint(fmaf(-slope, fabsf(r - static_cast<float>(cc * 32 + i)), x));
      }
  }
}

// The same with the keys' own positions: lane x holds at[i] = position of key
// 32 i + x.  The positions are any and `base` is the least distance of the
// row's visible keys (slope < 0: the greatest), so that what is left, modulo
// 2^32, is the visible keys' difference.  A warp-wide call.
template <int CHUNKS>
__device__ __forceinline__ void lower_by_positions(uint32_t (&sr)[CHUNKS][32], float c, float slope, int pos, uint32_t base,
                                                   const int (&at)[CHUNKS]) {
  const uint32_t flip = slope < 0.f ? ~0u : 0u, less = slope < 0.f ? ~base : 0u - base;  // ~(x + ~base) = base - x
  const float down = -fabsf(slope);
#pragma unroll
  for (int cc = 0; cc < CHUNKS; ++cc)
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const uint32_t x = __sad(pos, __shfl_sync(0xffffffffu, at[cc], i), less);  // |pos - at| + less, 32 bits unsigned
      sr[cc][i] = __float_as_uint(fmaf(__uint_as_float(sr[cc][i]), c, down * static_cast<float>(x ^ flip)));
    }
}

// The sum of P that O is divided by is that of the rounded values which the
// tensor cores multiply: a rounding d of p_j then moves O by d (V_j - O), not
// d V_j, so a key that has nearly all the weight is not rounded at all.
// (Adds both halves of a pair, exactly widened, to s0 and s1.)
template <bool BF16>
__device__ __forceinline__ void add_pair(float& s0, float& s1, uint32_t pair) {
  if constexpr (BF16)
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tadd.f32.bf16 %0, l, %0;\n\tadd.f32.bf16 %1, h, %1;\n\t}"
        : "+f"(s0), "+f"(s1)
        : "r"(pair));
  else
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tadd.f32.f16 %0, l, %0;\n\tadd.f32.f16 %1, h, %1;\n\t}"
        : "+f"(s0), "+f"(s1)
        : "r"(pair));
}

// P = 2^(c s + nmu) of the row's scores, rounded and packed; the sum of the rounded values.
template <int CHUNKS, bool BF16>
__device__ __forceinline__ float exp_row(const uint32_t (&sr)[CHUNKS][32], float c, float nmu, uint32_t (&pk)[CHUNKS][16]) {
  float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int cc = 0; cc < CHUNKS; ++cc)
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      float x0, x1;
      ffma2(x0, x1, __uint_as_float(sr[cc][i]), __uint_as_float(sr[cc][i + 1]), c, c, nmu, nmu);
      pk[cc][i / 2] = pack2<BF16>(ex2(x0), ex2(x1));
      add_pair<BF16>(ls[((i >> 1) & 1) * 2], ls[((i >> 1) & 1) * 2 + 1], pk[cc][i / 2]);
    }
  return (ls[0] + ls[1]) + (ls[2] + ls[3]);
}

// exp_row of capped scores straight from the products: P = 2^(s P(s^2) + nmu),
// MASKED: 0 for keys whose bit is not set.
template <int CHUNKS, bool BF16, bool MASKED>
__device__ __forceinline__ float exp_row_capped(const uint32_t (&sr)[CHUNKS][32], const ScoreConst& k, float nmu,
                                                 uint32_t (&pk)[CHUNKS][16], const uint32_t (&bits)[CHUNKS]) {
  float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int cc = 0; cc < CHUNKS; ++cc)
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const float s0 = __uint_as_float(sr[cc][i]), s1 = __uint_as_float(sr[cc][i + 1]);
      float x0, x1;
      cap_bracket(k, s0, s1, x0, x1);
      ffma2(x0, x1, x0, x1, s0, s1, nmu, nmu);
      if (MASKED) {
        uint32_t m0 = __float_as_uint(x0), m1 = __float_as_uint(x1);
        keep_if_set(m0, bits[cc], 1u << i);
        keep_if_set(m1, bits[cc], 2u << i);
        x0 = __uint_as_float(m0);
        x1 = __uint_as_float(m1);
      }
      pk[cc][i / 2] = pack2<BF16>(ex2(x0), ex2(x1));
      add_pair<BF16>(ls[((i >> 1) & 1) * 2], ls[((i >> 1) & 1) * 2 + 1], pk[cc][i / 2]);
    }
  return (ls[0] + ls[1]) + (ls[2] + ls[3]);
}

}  // namespace bw
}  // namespace stof
