// Host side of the serving operators declared in include/spec_verify.h (token
// log probabilities): argument validation and workspace layout.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "spec_verify.h"
#include "sv_internal.h"

using sv::hip_fail;
using sv::set_err;

namespace {

constexpr int64_t kMaxVocab = (int64_t)sv::kMaxTiles * sv::kTileElems;

// Chunks of a row: its elements behind at most the 16-byte boundary in front of them.
int64_t logprob_chunks(int64_t vocab, int es) { return (vocab * es + (16 - es) + sv::kChunkBytes - 1) / sv::kChunkBytes; }

bool logprob_sizes_ok(const char* who, int64_t rows, int64_t vocab, int32_t dtype, int32_t top) {
  if (dtype != SV_F32 && dtype != SV_BF16) {
    set_err("%s: unknown logits dtype %d", who, dtype);
    return false;
  }
  if (vocab < 1 || vocab > kMaxVocab) {
    set_err("%s: vocab %lld outside 1..%lld", who, (long long)vocab, (long long)kMaxVocab);
    return false;
  }
  if (rows < 0 || rows > INT32_MAX / logprob_chunks(vocab, dtype == SV_BF16 ? 2 : 4)) {
    set_err("%s: rows %lld outside 0..2^31 / (32 KB chunks of a row)", who, (long long)rows);
    return false;
  }
  if (top < 0 || top > SV_LOGPROBS_MAX_TOP || top > vocab) {
    set_err("%s: top %d outside 0..min(%d, vocab)", who, top, SV_LOGPROBS_MAX_TOP);
    return false;
  }
  return true;
}

}  // namespace

extern "C" {

int64_t spec_verify_logprobs_args_size(void) { return (int64_t)sizeof(spec_verify_logprobs_args); }

int64_t spec_verify_logprobs_workspace(int64_t rows, int64_t vocab, int32_t dtype, int32_t top) {
  if (!logprob_sizes_ok("spec_verify_logprobs_workspace", rows, vocab, dtype, top)) return SV_ERR_INVALID;
  const int64_t chunks = rows * logprob_chunks(vocab, dtype == SV_BF16 ? 2 : 4);
  return chunks * (16 + (top > 0 ? 4 * 64 : 0));
}

int spec_verify_token_logprobs(const spec_verify_logprobs_args* a, void* hip_stream) {
  const char* who = "spec_verify_token_logprobs";
  if (!a) {
    set_err("%s: args is NULL", who);
    return SV_ERR_INVALID;
  }
  if (!logprob_sizes_ok(who, a->rows, a->vocab, a->dtype, a->top)) return SV_ERR_INVALID;
  if (a->rows == 0) return SV_OK;
  const int es = a->dtype == SV_BF16 ? 2 : 4;
  if (!a->logits || ((uintptr_t)a->logits & (es - 1)) || a->ld < a->vocab || a->ld > INT64_MAX / 8 / a->rows) {
    set_err("%s: logits (aligned to %d bytes) with ld (%lld) >= vocab are required", who, es, (long long)a->ld);
    return SV_ERR_INVALID;
  }
  if (!a->tokens && (a->logprob || a->rank)) {
    set_err("%s: logprob and rank need tokens", who);
    return SV_ERR_INVALID;
  }
  if ((a->top > 0) != (a->top_tokens != nullptr) || (a->top_logprobs && !a->top_tokens)) {
    set_err("%s: top_tokens goes with top > 0 (%d), top_logprobs with top_tokens", who, a->top);
    return SV_ERR_INVALID;
  }
  const int64_t need = spec_verify_logprobs_workspace(a->rows, a->vocab, a->dtype, a->top);
  if (!a->workspace || ((uintptr_t)a->workspace & 15) || a->workspace_bytes < need) {
    set_err("%s: a 16-byte aligned workspace of %lld bytes is required, got %lld", who, (long long)need,
            (long long)a->workspace_bytes);
    return SV_ERR_INVALID;
  }
  sv::LogprobParams p{};
  p.rows = a->rows;
  p.V = a->vocab;
  p.ld = a->ld;
  p.logits = a->logits;
  p.bf16 = a->dtype == SV_BF16;
  p.top = a->top;
  p.nch = logprob_chunks(a->vocab, es);
  p.tokens = a->tokens;
  p.temperature = a->temperature;
  p.logprob = a->logprob;
  p.entropy = a->entropy;
  p.rank = a->rank;
  p.top_tokens = a->top_tokens;
  p.top_logprobs = a->top_logprobs;
  p.status = a->status;
  p.partials = static_cast<float*>(a->workspace);
  p.segmax = a->top > 0 ? p.partials + a->rows * p.nch * 4 : nullptr;
  hipError_t e = sv::launch_logprobs(p, (hipStream_t)hip_stream);
  if (e != hipSuccess) return hip_fail(who, e);
  return SV_OK;
}

}  // extern "C"
