// Attention with shared prefixes over a paged cache of e4m3 codes,
// for gfx950 (the kernels are in sv_attention_kernel.h and sv_prefix.h, the
// plan and the merge in sv_attention_shared.hip).

#include "sv_prefix.h"

namespace sv {

hipError_t launch_attention_shared_e4m3(const AttnParams& p, int row_tiles, int blocks, hipStream_t st) {
  return p.bf16 ? launch_type<true, codes::kE4m3, true>(p, row_tiles, blocks, st) : launch_type<false, codes::kE4m3, true>(p, row_tiles, blocks, st);
}

hipError_t launch_attention_prefix_e4m3(const AttnParams& p, hipStream_t st) { return launch_prefix_rows<codes::kE4m3>(p, st); }

}  // namespace sv
