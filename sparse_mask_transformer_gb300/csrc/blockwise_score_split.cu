// The split instances of the block-wise kernel of stof_mha_fwd_score
// (format_source.cuh).
#include "format_source.cuh"

namespace stof {
namespace scored {

stof_status launch_format_split(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const FormatParams& p,
                                int d, bool bf16, int mode, unsigned grid, cudaStream_t s) {
  if (d == 64)
    return bf16 ? launch_format<true, 64, true>(mq, mk, mv, p, mode, grid, s)
                : launch_format<true, 64, false>(mq, mk, mv, p, mode, grid, s);
  return bf16 ? launch_format<true, 128, true>(mq, mk, mv, p, mode, grid, s)
              : launch_format<true, 128, false>(mq, mk, mv, p, mode, grid, s);
}

}  // namespace scored
}  // namespace stof
