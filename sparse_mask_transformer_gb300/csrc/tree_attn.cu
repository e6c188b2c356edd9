// Attention of drafted tokens over a K/V cache (stof_tree_attn_fwd).
//
// One warp per query row: the row's visible keys one after the other, a lane
// holding d / 32 dimensions, with an online softmax.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "internal.h"
#include "score.cuh"

namespace stof {
namespace {

struct TreeParams {
  const void* q;
  const void* k;
  const void* v;
  void* o;
  int B, H, Hkv, group, T, d, cap, words;
  const int32_t* lens;
  const int32_t* counts;
  const uint32_t* tree;
  const int32_t* positions;
  float scale, softcap;
  const float* slopes;
  int64_t* err;
};

template <bool BF16>
__device__ __forceinline__ float widen(const uint16_t* p) {
  if constexpr (BF16)
    return __bfloat162float(__ushort_as_bfloat16(*p));
  else
    return __half2float(__ushort_as_half(*p));
}

template <int D, bool BF16>
__global__ void __launch_bounds__(128) tree_kernel(const TreeParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= static_cast<long long>(p.B) * p.H * p.T) return;
  const int t = static_cast<int>(row % p.T);
  const long long bh = row / p.T;
  const int b = static_cast<int>(bh / p.H), h = static_cast<int>(bh % p.H);
  const int ctx = p.lens[b], count = p.counts ? p.counts[b] : p.T;
  if (ctx < 0 || count < 0 || count > p.T || static_cast<long long>(ctx) + count > p.cap) {
    if (lane == 0 && p.err)
      atomicOr(reinterpret_cast<unsigned long long*>(p.err), static_cast<unsigned long long>(STOF_DEVERR_BAD_LENGTH));
    return;
  }
  if (t >= count) return;
  const long long plane = static_cast<long long>(b) * p.Hkv + h / p.group;
  const uint16_t* q = static_cast<const uint16_t*>(p.q) + row * D;
  const uint16_t* k = static_cast<const uint16_t*>(p.k) + plane * p.cap * D;
  const uint16_t* v = static_cast<const uint16_t*>(p.v) + plane * p.cap * D;
  const int32_t* positions = p.positions ? p.positions + static_cast<long long>(b) * p.T : nullptr;
  const ScoreRow score = make_score_row(p.scale, p.softcap, p.slopes ? p.slopes[h] : 0.f, positions ? positions[t] : ctx + t);
  float qf[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) qf[e] = widen<BF16>(q + lane + 32 * e), o[e] = 0.f;
  for (int j = 0; j < ctx + count; ++j) {
    const int u = j - ctx;
    if (u >= 0) {
      const bool sees = p.tree ? (p.tree[(static_cast<long long>(b) * p.T + t) * p.words + u / 32] >> (u % 32)) & 1 : u <= t;
      if (!sees) continue;
    }
    float dot = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) dot = fmaf(qf[e], widen<BF16>(k + static_cast<long long>(j) * D + lane + 32 * e), dot);
#pragma unroll
    for (int off = 16; off; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
    const float s = score_of(score, dot, u >= 0 && positions ? positions[u] : j);
    const float mn = fmaxf(m, s), alpha = score_ex2(m - mn), w = score_ex2(s - mn);
    m = mn;
    l = l * alpha + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * alpha + w * widen<BF16>(v + static_cast<long long>(j) * D + lane + 32 * e);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint16_t* out = static_cast<uint16_t*>(p.o) + row * D;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if constexpr (BF16)
      out[lane + 32 * e] = __bfloat16_as_ushort(__float2bfloat16(o[e] * inv));
    else
      out[lane + 32 * e] = __half_as_ushort(__float2half(o[e] * inv));
  }
}

}  // namespace
}  // namespace stof

using namespace stof;

extern "C" size_t stof_tree_attn_workspace_bytes(int B, int H, int Hkv, int T, int d) {
  if (B < 1 || H < 1 || Hkv < 1 || H % Hkv || T < 1 || T > STOF_TREE_MAX_TOKENS || (d != 64 && d != 128)) return 0;
  return 16;
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
  if (static_cast<long long>(B) * H * T >= (1ll << 31) || static_cast<long long>(B) * Hkv * ((cap + 127) / 128) >= (1ll << 31))
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
  TreeParams p;
  p.q = q;
  p.k = k;
  p.v = v;
  p.o = o;
  p.B = B;
  p.H = H;
  p.Hkv = Hkv;
  p.group = H / Hkv;
  p.T = T;
  p.d = d;
  p.cap = cap;
  p.words = (T + 31) / 32;
  p.lens = lens;
  p.counts = counts;
  p.tree = tree;
  p.positions = positions;
  p.scale = scale;
  p.softcap = score ? score->softcap : 0.f;
  p.slopes = score ? score->slopes : nullptr;
  p.err = device_error;
  const long long rows = static_cast<long long>(B) * H * T;
  const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d == 64)
    dt == STOF_BF16 ? tree_kernel<64, true><<<grid, 128, 0, s>>>(p) : tree_kernel<64, false><<<grid, 128, 0, s>>>(p);
  else
    dt == STOF_BF16 ? tree_kernel<128, true><<<grid, 128, 0, s>>>(p) : tree_kernel<128, false><<<grid, 128, 0, s>>>(p);
  return record_cuda(cudaGetLastError()) == cudaSuccess ? STOF_OK : STOF_ERR_CUDA;
}
