// The stages of attention with shared prefixes over a paged cache of e4m3 codes,
// for gfx950 (their kernel is in sv_attention_kernel.h, the plan in
// sv_attention_shared.hip).

#include "sv_prefix.h"

namespace sv {

hipError_t launch_attention_shared_e4m3(const AttnParams& p, int stage, int row_tiles, int blocks, hipStream_t st) {
  if (stage == kPrefix && row_tiles == kAttnManyRows) return launch_prefix_rows<codes::kE4m3>(p, blocks, st);
  return launch_shared<codes::kE4m3>(p, stage, row_tiles, blocks, st);
}

}  // namespace sv
