// Host side of the serving operators declared in include/spec_verify.h (token
// log probabilities, attention over a paged cache, the cache itself): argument validation and workspace layout.

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "spec_verify.h"
#include "sv_internal.h"

using sv::hip_fail;
using sv::set_err;

namespace {

constexpr int64_t kMaxVocab = (int64_t)sv::kMaxTiles * sv::kTileElems;

// Chunks of a row: its elements behind at most the 16-byte boundary in front of them.
int64_t logprob_chunks(int64_t vocab, int es) { return (vocab * es + (16 - es) + sv::kLpChunkBytes - 1) / sv::kLpChunkBytes; }

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
    set_err("%s: rows %lld outside 0..2^31 / (16 KB chunks of a row)", who, (long long)rows);
    return false;
  }
  if (top < 0 || top > SV_LOGPROBS_MAX_TOP || top > vocab) {
    set_err("%s: top %d outside 0..min(%d, vocab)", who, top, SV_LOGPROBS_MAX_TOP);
    return false;
  }
  return true;
}

// How a call's work is laid out: 16-row tiles per block, and blocks.
struct AttnShape {
  int row_tiles;
  int blocks;
  int64_t part_bytes;   // of one block's two parts
};

bool is_pow2(int32_t x) { return x > 0 && (x & (x - 1)) == 0; }

bool attention_sizes_ok(const char* who, const spec_verify_attention_args* a, AttnShape* s) {
  if (!a) {
    set_err("%s: args is NULL", who);
    return false;
  }
  if (a->dtype != SV_BF16 && a->dtype != SV_F16) {
    set_err("%s: dtype %d is neither SV_BF16 nor SV_F16", who, a->dtype);
    return false;
  }
  if (a->head_dim != 64 && a->head_dim != 128 && a->head_dim != 256) {
    set_err("%s: head_dim %d is not 64, 128 or 256", who, a->head_dim);
    return false;
  }
  if (!is_pow2(a->page_size) || a->page_size < 16 || a->page_size > 1024) {
    set_err("%s: page_size %d is not a power of two from 16 to 1024", who, a->page_size);
    return false;
  }
  if (a->heads < 1 || a->kv_heads < 1 || a->heads % a->kv_heads || a->heads / a->kv_heads > 256 || a->heads > 65536) {
    set_err("%s: heads %d must be a multiple, up to 256 times, of kv_heads %d", who, a->heads, a->kv_heads);
    return false;
  }
  if (a->batch < 0 || a->batch > 4096 || a->total_rows < a->batch || a->total_rows > 524288) {
    set_err("%s: batch %d outside 0..4096, or total_rows %d outside batch..524288", who, a->batch, a->total_rows);
    return false;
  }
  if (a->batch == 0 && a->total_rows != 0) {
    set_err("%s: total_rows %d belong to no sequence", who, a->total_rows);
    return false;
  }
  if (a->window < 0 || a->num_pages < 1 || a->num_pages > INT32_MAX || a->slots < 1 || a->max_pages < 1 ||
      (int64_t)a->max_pages * a->page_size > INT32_MAX - 4096) {
    set_err("%s: window %d < 0, or num_pages %lld, slots %d, max_pages %d outside their range", who, a->window,
            (long long)a->num_pages, a->slots, a->max_pages);
    return false;
  }
  if (a->batch == 0) {
    *s = AttnShape{1, 1, 0};
    return true;
  }
  // A (sequence, key head)'s rows should fit one block's row tiles: every
  // further block of tiles reads the keys again, at the same rate.  Tiles that
  // a short sequence leaves empty cost registers and code, not products.  Only
  // the sum of the rows is known here, so room is made for half again the
  // average, or for all that one sequence can have.  32 sequences of 4096, 8
  // key heads of 128: 4 rows with room for 16, 32, 48 95, 96, 97 us; 24 rows
  // with 32, 48 97, 99 (ragged, 8 to 24 rows and 1024 to 8192 tokens: 127 and
  // 134); 36 rows with 32, 48 114, 101.  One token of one sequence, 16 and 48 7
  // and 10 us.  More than 48 rows of 128 do not fit the registers (64 rows: 2
  // tiles twice 113 us, 3 tiles twice 182, 4 spilled 187), nor more than 16 of
  // 256 (16 to 40 rows in a window of 4096: 39 us, 2 tiles spilled 63); 64 sequences
  // of 4096 with 8 heads of 64: 8 rows with room for 16, 32, 64 94, 96, 96 us,
  // 64 rows with 64, 32 104, 153.
  const int64_t group = a->heads / a->kv_heads;
  const int64_t avg = (a->total_rows * group + a->batch - 1) / a->batch;
  const int64_t room = std::min(avg + avg / 2, (int64_t)(a->total_rows - a->batch + 1) * group);
  if (a->head_dim == 256 || room <= 16) s->row_tiles = 1;
  else if (room <= 32 || (a->head_dim == 128 && avg > 48)) s->row_tiles = 2;
  else s->row_tiles = a->head_dim == 128 ? 3 : 4;
  const int64_t tm = 16 * s->row_tiles;
  const int64_t keys = (int64_t)a->max_pages * a->page_size;
  const int64_t units = (a->total_rows * group / tm + a->batch) * a->kv_heads *
                        ((keys + sv::kAttnUnitKeys - 1) / sv::kAttnUnitKeys);
  if (units > INT32_MAX) {
    set_err("%s: %lld units of work: batch, heads and max_pages are too large together", who, (long long)units);
    return false;
  }
  // One block per CU keeps enough reads in flight for heads of 128 and 256 and
  // leaves the fewest parts to join (32 sequences of 4096 with 24 rows of 128:
  // 97 + 4 us, with two 101 + 9; ragged 126 + 6 and 128 + 8, with four 132 +
  // 10); heads of 64, and tiles that read the keys again, want two (64
  // sequences of 4096 with 8 heads of 64: 96 and 94 us; 64 rows of 128: 156 and
  // 113).  One row tile of 64 leaves room for four, which hide each other's
  // changes from tile to tile (256 ragged sequences of 125 to 1000 tokens, 16
  // heads: 140 + 6 us with two, 126 + 7 with four, 124 + 9 with eight in turn).
  int per_cu = 1;
  if (a->head_dim == 64) per_cu = s->row_tiles == 1 ? 4 : 2;
  else if (a->head_dim == 128 && avg > 48) per_cu = 2;
  s->blocks = (int)std::min<int64_t>(units, 256 * per_cu);
  s->part_bytes = 2 * tm * (a->head_dim + 2) * 4;
  return true;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// strides of a tensor of 16-bit elements: multiples of 16 bytes, small enough for the kernels' offsets
bool strides_ok(int64_t a, int64_t b, int64_t c) {
  for (int64_t x : {a, b, c})
    if (x < 0 || x % 8 || x > (int64_t)1 << 40) return false;
  return true;
}

// workspace of a cache: the list's length, the ids, the list
struct CacheLayout {
  int64_t ids, pairs, bytes;
};

bool cache_sizes_ok(const char* who, const spec_verify_cache* c, CacheLayout* l) {
  if (!c) {
    set_err("%s: cache is NULL", who);
    return false;
  }
  if (c->slots < 1 || c->slots > SV_CACHE_MAX_SLOTS || c->max_pages < 1 || c->max_pages > 131072 || c->num_pages < 1 ||
      c->num_pages >= 1 << 30 || c->layers < 1 || c->layers > 4096) {
    set_err("%s: slots %d, max_pages %d, num_pages %d or layers %d outside their range", who, c->slots, c->max_pages,
            c->num_pages, c->layers);
    return false;
  }
  if (!is_pow2(c->page_size) || c->page_size < 16 || c->page_size > 1024) {
    set_err("%s: page_size %d is not a power of two from 16 to 1024", who, c->page_size);
    return false;
  }
  if (c->kv_heads < 1 || c->head_dim < 8 || c->head_dim % 8 || (int64_t)c->kv_heads * c->head_dim > 65536) {
    set_err("%s: head_dim %d is not a multiple of 8, or kv_heads %d * head_dim outside 1..65536", who, c->head_dim,
            c->kv_heads);
    return false;
  }
  static_assert(SV_CACHE_MAX_SLOTS == sv::kCacheMaxSlots, "slots");
  l->ids = 256;
  l->pairs = l->ids + (int64_t)sv::align_up((size_t)c->num_pages * 4, 256);
  l->bytes = l->pairs + (int64_t)std::max(c->num_pages, c->slots) * 8;
  return true;
}

// The checks every call on a cache shares, and its parameters.
bool cache_params(const char* who, const spec_verify_cache* c, int32_t batch, sv::CacheParams* p) {
  CacheLayout l;
  if (!cache_sizes_ok(who, c, &l)) return false;
  if (!c->page_table || !c->seq_len || !c->refcount || !c->k || !c->v || !c->workspace || !aligned16(c->refcount) ||
      !aligned16(c->k) || !aligned16(c->v) || !aligned16(c->workspace) || c->workspace_bytes < l.bytes) {
    set_err("%s: page_table, seq_len, refcount, k, v (the last three 16-byte aligned) and a workspace of %lld bytes "
            "are required", who, (long long)l.bytes);
    return false;
  }
  if (batch < 0 || batch > c->slots) {
    set_err("%s: batch %d outside 0..%d slots", who, batch, c->slots);
    return false;
  }
  *p = sv::CacheParams{};
  p->B = batch;
  p->slots = c->slots;
  p->max_pages = c->max_pages;
  p->page_size = c->page_size;
  p->page_log2 = __builtin_ctz((unsigned)c->page_size);
  p->num_pages = c->num_pages;
  p->max_len = c->max_pages * c->page_size;
  p->layers = c->layers;
  p->table = c->page_table;
  p->seq_len = c->seq_len;
  p->refcount = c->refcount;
  p->k = c->k;
  p->v = c->v;
  p->page_bytes = (int64_t)c->kv_heads * c->head_dim * c->page_size * 2;
  p->layer_bytes = p->page_bytes * c->num_pages;
  char* ws = static_cast<char*>(c->workspace);
  p->count = reinterpret_cast<int32_t*>(ws);
  p->ids = reinterpret_cast<int32_t*>(ws + l.ids);
  p->pairs = reinterpret_cast<int2*>(ws + l.pairs);
  return true;
}

}  // namespace

extern "C" {

int64_t spec_verify_logprobs_args_size(void) { return (int64_t)sizeof(spec_verify_logprobs_args); }

int64_t spec_verify_logprobs_workspace(int64_t rows, int64_t vocab, int32_t dtype, int32_t top) {
  if (!logprob_sizes_ok("spec_verify_logprobs_workspace", rows, vocab, dtype, top)) return SV_ERR_INVALID;
  const int64_t chunks = rows * logprob_chunks(vocab, dtype == SV_BF16 ? 2 : 4);
  return chunks * (16 + (top > 0 ? 4 * sv::kLpSegs : 0));
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

int64_t spec_verify_attention_args_size(void) { return (int64_t)sizeof(spec_verify_attention_args); }

int64_t spec_verify_attention_workspace(const spec_verify_attention_args* a) {
  AttnShape s;
  if (!attention_sizes_ok("spec_verify_attention_workspace", a, &s)) return SV_ERR_INVALID;
  return s.blocks * s.part_bytes + (int64_t)s.blocks * sv::kAttnPartBytes;
}

int spec_verify_paged_attention(const spec_verify_attention_args* a, void* hip_stream) {
  const char* who = "spec_verify_paged_attention";
  AttnShape s;
  if (!attention_sizes_ok(who, a, &s)) return SV_ERR_INVALID;
  if (a->batch == 0) return SV_OK;
  if (!a->q || !a->k || !a->v || !a->page_table || !a->seq_len || !a->num_draft || !a->out) {
    set_err("%s: q, k, v, page_table, seq_len, num_draft and out are required", who);
    return SV_ERR_INVALID;
  }
  if (!aligned16(a->q) || !aligned16(a->k) || !aligned16(a->v) || !aligned16(a->out) ||
      !strides_ok(a->q_row_stride, a->q_head_stride, 0) ||
      !strides_ok(a->k_page_stride, a->k_head_stride, a->k_token_stride) ||
      !strides_ok(a->v_page_stride, a->v_head_stride, a->v_token_stride) || a->k_token_stride > 1 << 24 ||
      a->v_token_stride > 1 << 24) {
    set_err("%s: q, k, v and out need 16-byte alignment, and strides that are multiples of 8 elements "
            "(a token's at most 2^24)", who);
    return SV_ERR_INVALID;
  }
  if (a->page_table_stride < a->max_pages || a->page_table_stride > INT32_MAX) {
    set_err("%s: page_table_stride %lld < max_pages %d", who, (long long)a->page_table_stride, a->max_pages);
    return SV_ERR_INVALID;
  }
  const float scale_log2 = (float)(a->scale * 1.4426950408889634);
  if (!isfinite(scale_log2)) {
    set_err("%s: scale %g (times log2 e) is not finite in 32 bits", who, a->scale);
    return SV_ERR_INVALID;
  }
  const int64_t need = spec_verify_attention_workspace(a);
  if (!a->workspace || !aligned16(a->workspace) || a->workspace_bytes < need) {
    set_err("%s: a 16-byte aligned workspace of %lld bytes is required, got %lld", who, (long long)need,
            (long long)a->workspace_bytes);
    return SV_ERR_INVALID;
  }
  sv::AttnParams p{};
  p.B = a->batch;
  p.total_rows = a->total_rows;
  p.heads = a->heads;
  p.kv_heads = a->kv_heads;
  p.group = a->heads / a->kv_heads;
  p.head_dim = a->head_dim;
  p.bf16 = a->dtype == SV_BF16;
  p.window = std::min(a->window, 1 << 30);   // beyond every length; keeps the differences of positions in 32 bits
  p.page_log2 = __builtin_ctz((unsigned)a->page_size);
  p.slots = a->slots;
  p.max_len = a->max_pages * a->page_size;
  p.num_pages = a->num_pages;
  p.scale_log2 = scale_log2;
  p.q = a->q;
  p.q_row = a->q_row_stride;
  p.q_head = a->q_head_stride;
  p.k = a->k;
  p.k_page = a->k_page_stride;
  p.k_head = a->k_head_stride;
  p.k_tok = a->k_token_stride;
  p.v = a->v;
  p.v_page = a->v_page_stride;
  p.v_head = a->v_head_stride;
  p.v_tok = a->v_token_stride;
  p.table = a->page_table;
  p.table_stride = a->page_table_stride;
  p.seq_len = a->seq_len;
  p.num_draft = a->num_draft;
  p.seqs = a->seqs;
  p.start = a->start;
  p.out = a->out;
  p.lse = a->lse;
  p.status = a->status;
  p.parts = static_cast<float*>(a->workspace);
  p.desc = static_cast<char*>(a->workspace) + s.blocks * s.part_bytes;
  hipError_t e = sv::launch_attention(p, s.row_tiles, s.blocks, (hipStream_t)hip_stream);
  if (e != hipSuccess) return hip_fail(who, e);
  return SV_OK;
}

int64_t spec_verify_cache_size(void) { return (int64_t)sizeof(spec_verify_cache); }

int64_t spec_verify_cache_workspace(const spec_verify_cache* c) {
  CacheLayout l;
  return cache_sizes_ok("spec_verify_cache_workspace", c, &l) ? l.bytes : SV_ERR_INVALID;
}

int spec_verify_cache_reserve(const spec_verify_cache* c, int32_t batch, const int32_t* seqs, const int32_t* num_new,
                              int64_t total_new, int32_t* start, int64_t* slots, int32_t* status, void* hip_stream) {
  const char* who = "spec_verify_cache_reserve";
  sv::CacheParams p;
  if (!cache_params(who, c, batch, &p)) return SV_ERR_INVALID;
  if (batch == 0) return SV_OK;
  if (!num_new || !start || total_new < 0 || total_new > sv::kCacheMaxRows || (total_new > 0 && !slots)) {
    set_err("%s: num_new, start and slots are required, total_new %lld in 0..%d", who, (long long)total_new,
            sv::kCacheMaxRows);
    return SV_ERR_INVALID;
  }
  p.seqs = seqs;
  p.num_new = num_new;
  p.total_new = total_new;
  p.start = start;
  p.new_slots = slots;
  p.status = status;
  hipError_t e = sv::launch_cache_reserve(p, (hipStream_t)hip_stream);
  return e == hipSuccess ? SV_OK : hip_fail(who, e);
}

int spec_verify_cache_truncate(const spec_verify_cache* c, int32_t batch, const int32_t* seqs, const int32_t* drop,
                               int32_t* status, void* hip_stream) {
  const char* who = "spec_verify_cache_truncate";
  sv::CacheParams p;
  if (!cache_params(who, c, batch, &p)) return SV_ERR_INVALID;
  if (batch == 0) return SV_OK;
  p.seqs = seqs;
  p.drop = drop;
  p.status = status;
  hipError_t e = sv::launch_cache_truncate(p, (hipStream_t)hip_stream);
  return e == hipSuccess ? SV_OK : hip_fail(who, e);
}

static int cache_commit(const char* who, const spec_verify_cache* c, int32_t batch, const int32_t* seqs, const int32_t* num_draft,
                        const int32_t* accepted_len, const int32_t* start, int32_t* status, void* hip_stream) {
  sv::CacheParams p;
  if (!cache_params(who, c, batch, &p)) return SV_ERR_INVALID;
  if (batch == 0) return SV_OK;
  if (!num_draft || !accepted_len) {
    set_err("%s: num_draft and accepted_len are required", who);
    return SV_ERR_INVALID;
  }
  p.seqs = seqs;
  p.num_draft = num_draft;
  p.accepted = accepted_len;
  p.reserved = start;
  p.status = status;
  hipError_t e = sv::launch_cache_truncate(p, (hipStream_t)hip_stream);
  return e == hipSuccess ? SV_OK : hip_fail(who, e);
}

int spec_verify_cache_commit(const spec_verify_cache* c, int32_t batch, const int32_t* seqs, const int32_t* num_draft,
                             const int32_t* accepted_len, int32_t* status, void* hip_stream) {
  return cache_commit("spec_verify_cache_commit", c, batch, seqs, num_draft, accepted_len, nullptr, status, hip_stream);
}

int spec_verify_cache_commit_reserved(const spec_verify_cache* c, int32_t batch, const int32_t* seqs, const int32_t* num_draft,
                                      const int32_t* accepted_len, const int32_t* start, int32_t* status, void* hip_stream) {
  const char* who = "spec_verify_cache_commit_reserved";
  if (batch != 0 && !start) {
    set_err("%s: start is required", who);
    return SV_ERR_INVALID;
  }
  return cache_commit(who, c, batch, seqs, num_draft, accepted_len, start, status, hip_stream);
}

int spec_verify_cache_fork(const spec_verify_cache* c, int32_t batch, const int32_t* parents, const int32_t* children,
                           int32_t* status, void* hip_stream) {
  const char* who = "spec_verify_cache_fork";
  sv::CacheParams p;
  if (!cache_params(who, c, batch, &p)) return SV_ERR_INVALID;
  if (batch == 0) return SV_OK;
  if (!parents || !children) {
    set_err("%s: parents and children are required", who);
    return SV_ERR_INVALID;
  }
  p.seqs = parents;
  p.children = children;
  p.status = status;
  hipError_t e = sv::launch_cache_fork(p, (hipStream_t)hip_stream);
  return e == hipSuccess ? SV_OK : hip_fail(who, e);
}

int spec_verify_cache_compact(const spec_verify_cache* c, int32_t* live, void* hip_stream) {
  const char* who = "spec_verify_cache_compact";
  sv::CacheParams p;
  if (!cache_params(who, c, 0, &p)) return SV_ERR_INVALID;
  p.live = live;
  hipError_t e = sv::launch_cache_compact(p, (hipStream_t)hip_stream);
  return e == hipSuccess ? SV_OK : hip_fail(who, e);
}

int spec_verify_cache_write(const spec_verify_cache* c, int32_t layer, int64_t rows, const void* k_new,
                            int64_t k_row_stride, int64_t k_head_stride, const void* v_new, int64_t v_row_stride,
                            int64_t v_head_stride, const int64_t* slots, void* hip_stream) {
  const char* who = "spec_verify_cache_write";
  sv::CacheParams p;
  if (!cache_params(who, c, 0, &p)) return SV_ERR_INVALID;
  if (layer < 0 || layer >= c->layers || rows < 0 || rows > sv::kCacheMaxRows) {
    set_err("%s: layer %d outside 0..%d, or rows %lld outside 0..%d", who, layer, c->layers - 1, (long long)rows,
            sv::kCacheMaxRows);
    return SV_ERR_INVALID;
  }
  if (rows == 0) return SV_OK;
  if (!k_new || !v_new || !slots || !aligned16(k_new) || !aligned16(v_new) ||
      !strides_ok(k_row_stride, k_head_stride, 0) || !strides_ok(v_row_stride, v_head_stride, 0)) {
    set_err("%s: k_new and v_new (16-byte aligned, strides in multiples of 8 elements) and slots are required", who);
    return SV_ERR_INVALID;
  }
  sv::CacheWriteParams w{};
  w.rows = rows;
  w.places = (int64_t)c->num_pages * c->page_size;
  w.kv_heads = c->kv_heads;
  w.head_dim = c->head_dim;
  w.head_vecs = c->head_dim / 8;
  w.vecs = c->kv_heads * w.head_vecs;
  w.page_log2 = p.page_log2;
  w.k = static_cast<char*>(c->k) + layer * p.layer_bytes;
  w.v = static_cast<char*>(c->v) + layer * p.layer_bytes;
  w.k_new = k_new;
  w.v_new = v_new;
  w.k_row = k_row_stride;
  w.k_head = k_head_stride;
  w.v_row = v_row_stride;
  w.v_head = v_head_stride;
  w.new_slots = slots;
  hipError_t e = sv::launch_cache_write(w, (hipStream_t)hip_stream);
  return e == hipSuccess ? SV_OK : hip_fail(who, e);
}

}  // extern "C"
