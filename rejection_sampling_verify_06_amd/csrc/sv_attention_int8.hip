// Attention over a paged cache of int8 codes, for gfx950 (the kernel and its
// reasons are in sv_attention_kernel.h).

#include "sv_attention_kernel.h"

namespace sv {

hipError_t launch_attention_int8(const AttnParams& p, int row_tiles, int blocks, hipStream_t st) {
  return p.bf16 ? launch_type<true, codes::kInt8, false>(p, row_tiles, blocks, st)
                : launch_type<false, codes::kInt8, false>(p, row_tiles, blocks, st);
}

}  // namespace sv
