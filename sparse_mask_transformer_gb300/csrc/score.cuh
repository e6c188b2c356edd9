// Scores of an attention row that are capped and / or lowered with distance,
// in the log2 domain (score times log2 e) that the kernels' exponentials use:
//   x = scale q.k;   x <- cap tanh(x / cap) if cap > 0;   x <- x - slope |pos - key|.
// With A = cap log2 e and tanh y = 1 - 2 / (1 + e^(2 y)),
//   log2 e cap tanh(x / cap) = A + 2 A u,   u = -1 / (1 + 2^(B q.k)),   B = 2 scale log2 e / cap:
// one exponential, one reciprocal and two additions or multiplications; u is
// in [-1, 0], so the cap's error is a few 2^-24 of cap, whatever the score
// (tanh.approx would be 2^-11 of the score).  2^(B q.k) may overflow: u is
// then -0, the cap's upper end.
#pragma once
#include <cuda_runtime.h>

namespace stof {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float score_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float score_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Distance from `pos` to the nearest (far: the farthest) of the keys 0 .. last.
__device__ __forceinline__ uint32_t reference_distance(int pos, int last, bool far) {
  const uint32_t a = __sad(pos, 0, 0u), b = __sad(pos, last, 0u);  // |pos|, |pos - last|
  return far ? max(a, b) : (pos >= 0 && pos <= last ? 0u : min(a, b));
}

// What one query row needs: with a cap, the score is a + two_a u(b q.k);
// without, two_a q.k.  slope is in log2 units per position, and the distances
// are counted from `base`, the head's nearest key's (slope < 0: the farthest's):
// a row's softmax does not change when all its scores move by slope base, and
// keys 2^30 away differ as near ones do.
struct ScoreRow {
  float a, two_a, b, slope;
  int pos;
  uint32_t base;
  bool cap;
};

__device__ __forceinline__ ScoreRow make_score_row(float scale, float cap, float slope, int pos) {
  ScoreRow r;
  r.cap = cap > 0.f;
  r.a = r.cap ? cap * kLog2e : 0.f;
  r.two_a = r.cap ? 2.f * r.a : scale * kLog2e;
  r.b = r.cap ? 2.f * kLog2e * (scale / cap) : 0.f;
  r.slope = slope * kLog2e;
  r.pos = pos;
  r.base = 0;
  return r;
}

// The log2-domain score of the row's product `dot` with key `key`.
__device__ __forceinline__ float score_of(const ScoreRow& r, float dot, int key) {
  const float u = r.cap ? score_rcp(-1.f - score_ex2(r.b * dot)) : dot;
  const float distance = static_cast<float>(static_cast<int>(__sad(r.pos, key, 0u - r.base)));  // |pos - key| - base
  return fmaf(-r.slope, distance, fmaf(r.two_a, u, r.a));
}

}  // namespace stof
