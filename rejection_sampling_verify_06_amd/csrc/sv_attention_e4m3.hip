// Attention over a paged cache of e4m3 codes, for gfx950 (the kernel and its
// reasons are in sv_attention_kernel.h).

#include "sv_attention_kernel.h"

namespace sv {

hipError_t launch_attention_e4m3(const AttnParams& p, int row_tiles, int blocks, hipStream_t st) {
  return p.bf16 ? launch_type<true, codes::kE4m3, false>(p, row_tiles, blocks, st)
                : launch_type<false, codes::kE4m3, false>(p, row_tiles, blocks, st);
}

}  // namespace sv
