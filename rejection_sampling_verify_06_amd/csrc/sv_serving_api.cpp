// Host side of the serving operators declared in include/spec_verify.h (token
// log probabilities, attention over a paged cache, the cache itself in 16 or 8
// bits, norms and rotation): argument validation and workspace layout.

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

// The layout of `rows` rows of `batch` sequences (or groups) each with up to all the keys that a page table holds.
bool attention_shape(const char* who, const spec_verify_attention_args* a, int32_t codes, int32_t rows, int32_t batch, AttnShape* s) {
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
  // 256 over 16-bit pages (16 to 40 rows in a window of 4096: 39 us, 2 tiles spilled
  // 63; over codes, whose one tile has 226 of 256 registers, not tried); 64 sequences
  // of 4096 with 8 heads of 64: 8 rows with room for 16, 32, 64 94, 96, 96 us,
  // 64 rows with 64, 32 104, 153.
  const int64_t group = a->heads / a->kv_heads;
  const int64_t avg = ((int64_t)rows * group + batch - 1) / batch;
  const int64_t room = std::min(avg + avg / 2, (int64_t)(rows - batch + 1) * group);
  if (a->head_dim == 256 || room <= 16) s->row_tiles = 1;
  else if (room <= 32 || (a->head_dim == 128 && avg > 48)) s->row_tiles = 2;
  else s->row_tiles = a->head_dim == 128 ? 3 : 4;
  const int64_t tm = 16 * s->row_tiles;
  const int64_t keys = (int64_t)a->max_pages * a->page_size;
  const int64_t units = ((int64_t)rows * group / tm + batch) * a->kv_heads *
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
  // 113), and so do codes, whose unpacking one wave a SIMD does not hide (16
  // sequences of up to 20000 with heads of 256, one and two: 55 and 52 us, 40
  // sequences 88 and 82; 33 units a sequence 34.2 and 34.6).  One row tile of 64 leaves room for four, which hide each other's
  // changes from tile to tile (256 ragged sequences of 125 to 1000 tokens, 16
  // heads: 140 + 6 us with two, 126 + 7 with four, 124 + 9 with eight in turn).
  int per_cu = 1;
  if (a->head_dim == 64) per_cu = s->row_tiles == 1 ? 4 : 2;
  else if (codes != SV_CODES_NONE || (a->head_dim == 128 && avg > 48)) per_cu = 2;
  s->blocks = (int)std::min<int64_t>(units, 256 * per_cu);
  s->part_bytes = 2 * tm * (a->head_dim + 2) * 4;
  return true;
}

// The layout of a call.  With shared prefixes `tiles` is that of the sequences'
// own parts where the kernel for many rows takes the groups' (of prefix_blocks
// blocks), otherwise of groups and sequences together.
struct AttnLayout {
  AttnShape tiles;
  int32_t groups;
  bool many;
  int prefix_blocks;
  AttnShape together;   // should `many` not do after all
};

bool shared_shape(const char* who, const spec_verify_attention_args* a, int32_t codes, AttnLayout* s) {
  AttnShape own, prefix;
  if (!attention_shape(who, a, codes, a->total_rows, a->batch, &own) ||
      !attention_shape(who, a, codes, a->total_rows, s->groups, &prefix))
    return false;
  const int64_t group = a->heads / a->kv_heads;
  const int64_t blocks = ((int64_t)a->max_pages * a->page_size + sv::kAttnUnitKeys - 1) / sv::kAttnUnitKeys;
  if (((int64_t)a->total_rows * group / 16 + a->batch + s->groups) * a->kv_heads * blocks > INT32_MAX) {
    set_err("%s: batch, heads and max_pages are too large together", who);
    return false;
  }
  // a tile's start is most of a short part's time: two blocks a CU overlap
  own.blocks = std::max(own.blocks, a->head_dim == 256 ? 256 : 512);
  s->together = own;
  s->together.row_tiles = std::max(own.row_tiles, prefix.row_tiles);
  s->together.part_bytes = std::max(own.part_bytes, prefix.part_bytes);
  const int64_t avg = ((int64_t)a->total_rows * group + s->groups - 1) / s->groups;
  const int64_t units = ((int64_t)a->total_rows * group / sv::kAttnPrefixRows + s->groups) * a->kv_heads * blocks;
  // The kernel for many rows (tiles of 128) has its own launch and adds its parts
  // to the merge's; k_attention reads the keys once for each 16 to 48 rows, and
  // spills nothing of codes.  8 groups behind 8000 tokens, 8 key heads of 128, whole
  // call, k_attention and this one: 14 rows of a group and key head 55 and 60 us, 24
  // 94 and 77, 28 84 and 65, 56 106 and 77; heads of 256 28 118 and 93; but heads
  // of 64 28 47 and 51, 42 46 and 56, 56 60 and 58, e4m3 42 64 and 72, 56 88 and 79,
  // int8 of 256 42 115 and 138, 52 189 and 180, 60 172 and 177, 72 269 and 233, 84 283
  // and 229 (52 rows on: with longer own parts).  Short prefixes pay for the launch
  // whatever their rows, which the rule does not look at: 8 groups behind 500 or 2000
  // tokens, 52 to 256 rows, 58 to 258 us and 62 to 279 (behind 130 69 to 318 and 63
  // to 248); one group behind 130 to 2000 is latency alone, 52 rows 23 to 26 and 27 to
  // 31, 256 29 to 38 and 30 to 42; behind 8000 52 rows 41 and 49, 128 53 and 53, 256 82
  // and 53; behind 30000 32 rows 62 and 62.
  s->many = avg > 48 || (codes == SV_CODES_NONE && a->head_dim >= 128 && avg > 16 && units >= 2048);
  s->tiles = s->many ? own : s->together;
  s->prefix_blocks = s->many ? (int)std::min<int64_t>(units, a->head_dim == 256 ? 256 : 512) : 0;
  return true;
}

bool attention_sizes_ok(const char* who, const spec_verify_attention_args* a, const spec_verify_attention_options* o, AttnLayout* s) {
  if (!a) {
    set_err("%s: args is NULL", who);
    return false;
  }
  if (a->dtype != SV_BF16 && a->dtype != SV_F16) {
    set_err("%s: dtype %d is neither SV_BF16 nor SV_F16", who, a->dtype);
    return false;
  }
  const int32_t codes = o ? o->codes : SV_CODES_NONE;
  if (codes != SV_CODES_NONE && codes != SV_CODES_E4M3 && codes != SV_CODES_INT8) {
    set_err("%s: codes %d is none of SV_CODES_*", who, codes);
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
  const int32_t groups = o ? o->num_groups : 0;
  if (groups < 0 || groups > a->batch) {
    set_err("%s: num_groups %d outside 0..batch", who, groups);
    return false;
  }
  if (groups > 0 && a->window > 0) {
    set_err("%s: a window (%d) hides the prefix that groups share; call without groups", who, a->window);
    return false;
  }
  *s = AttnLayout{};
  s->groups = groups;
  if (a->batch == 0) {
    s->tiles = AttnShape{1, 1, 0};
    return true;
  }
  return groups > 0 ? shared_shape(who, a, codes, s) : attention_shape(who, a, codes, a->total_rows, a->batch, &s->tiles);
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// strides of a tensor of 16-bit elements: multiples of 16 bytes, small enough for the kernels' offsets
bool strides_ok(int64_t a, int64_t b, int64_t c) {
  for (int64_t x : {a, b, c})
    if (x < 0 || x % 8 || x > (int64_t)1 << 40) return false;
  return true;
}

// Where a call's parts, records and (with groups) its plan and states lie in its
// workspace; returns the bytes.
int64_t attention_workspace(const spec_verify_attention_args* a, const AttnLayout& l, char* base, sv::AttnParams* p) {
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    char* x = base + at;
    at += (int64_t)sv::align_up((size_t)bytes, 16);
    return x;
  };
  if (l.groups == 0) {
    p->parts = reinterpret_cast<float*>(take(l.tiles.blocks * l.tiles.part_bytes));
    p->desc = take((int64_t)l.tiles.blocks * sv::kAttnPartBytes);
    return at;
  }
  p->parts = reinterpret_cast<float*>(take(l.together.blocks * l.together.part_bytes));
  const int64_t B = a->batch, G = l.groups, rows = (int64_t)a->total_rows * a->heads;
  p->prefix_parts = l.many ? reinterpret_cast<float*>(take(2 * (int64_t)l.prefix_blocks * sv::kAttnPrefixRows * (a->head_dim + 2) * 4)) : p->parts;
  auto ints = [&](int64_t n) { return reinterpret_cast<int32_t*>(take(n * 4)); };
  sv::AttnPlan& n = p->plan;
  n.bad = ints(1);
  n.units = ints(G + B + 1);
  n.group_units = ints(G + 1);
  n.group = reinterpret_cast<sv::AttnRecord*>(take((G + B) * (int64_t)sizeof(sv::AttnRecord)));
  n.seq = n.group + G;
  n.flags = ints(B);
  n.row_seq = ints(a->total_rows);
  // tiles have 16 rows at least; the last of a group's, or of a sequence's, may be cut
  n.tile = reinterpret_cast<int2*>(take((2 * (rows / a->kv_heads / 16) + G + B) * a->kv_heads * (int64_t)sizeof(int2)));
  p->state_m = reinterpret_cast<float*>(take(2 * rows * 4));
  p->state_o = reinterpret_cast<float*>(take(2 * rows * a->head_dim * 4));
  return at;
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

bool codes_ok(const char* who, const spec_verify_codes* q, int32_t head_dim) {
  if (q->codes != SV_CODES_E4M3 && q->codes != SV_CODES_INT8) {
    set_err("%s: codes %d is neither SV_CODES_E4M3 nor SV_CODES_INT8", who, q->codes);
    return false;
  }
  if (q->dtype != SV_BF16 && q->dtype != SV_F16) {
    set_err("%s: dtype %d is neither SV_BF16 nor SV_F16", who, q->dtype);
    return false;
  }
  if (head_dim % 16 || head_dim > 512) {
    set_err("%s: a head_dim of %d in 8 bits is not a multiple of 16, at most 512", who, head_dim);
    return false;
  }
  if (!q->k_scale || !q->v_scale || !aligned16(q->k_scale) || !aligned16(q->v_scale)) {
    set_err("%s: k_scale and v_scale (16-byte aligned) are required", who);
    return false;
  }
  return true;
}

// The checks every call on a cache shares, and its parameters.
bool cache_params(const char* who, const spec_verify_cache* c, int32_t batch, sv::CacheParams* p,
                  const spec_verify_codes* q = nullptr) {
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
  if (q && !codes_ok(who, q, c->head_dim)) return false;
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
  p->page_bytes = (int64_t)c->kv_heads * c->head_dim * c->page_size * (q ? 1 : 2);
  if (q) {
    p->ks = q->k_scale;
    p->vs = q->v_scale;
    p->scale_bytes = (int64_t)c->kv_heads * c->page_size * 4;
  }
  p->layer_bytes = p->page_bytes * c->num_pages;
  char* ws = static_cast<char*>(c->workspace);
  p->count = reinterpret_cast<int32_t*>(ws);
  p->ids = reinterpret_cast<int32_t*>(ws + l.ids);
  p->pairs = reinterpret_cast<int2*>(ws + l.pairs);
  return true;
}

// Where a layer of the cache takes rows, for the kernel that norms, rotates and codes.
void rope_cache(const spec_verify_cache* c, const spec_verify_codes* q, int32_t layer, const int64_t* slots,
                const sv::CacheParams& p, sv::RopeParams* r) {
  r->NV = c->kv_heads;
  r->slots = slots;
  r->places = (int64_t)c->num_pages * c->page_size;
  r->page_log2 = p.page_log2;
  r->codes = q ? q->codes : SV_CODES_NONE;
  r->ck = static_cast<char*>(c->k) + layer * p.layer_bytes;
  r->cv = static_cast<char*>(c->v) + layer * p.layer_bytes;
  if (q) {
    r->ks = q->k_scale + layer * (p.scale_bytes / 4) * c->num_pages;
    r->vs = q->v_scale + layer * (p.scale_bytes / 4) * c->num_pages;
  }
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

int64_t spec_verify_attention_options_size(void) { return (int64_t)sizeof(spec_verify_attention_options); }

int64_t spec_verify_attention_options_workspace(const spec_verify_attention_args* a, const spec_verify_attention_options* o) {
  AttnLayout l;
  if (!attention_sizes_ok("spec_verify_attention_workspace", a, o, &l)) return SV_ERR_INVALID;
  sv::AttnParams p{};
  return attention_workspace(a, l, nullptr, &p);
}

int64_t spec_verify_attention_workspace(const spec_verify_attention_args* a) {
  return spec_verify_attention_options_workspace(a, nullptr);
}

int spec_verify_paged_attention(const spec_verify_attention_args* a, void* hip_stream) {
  return spec_verify_paged_attention_options(a, nullptr, hip_stream);
}

int spec_verify_paged_attention_options(const spec_verify_attention_args* a, const spec_verify_attention_options* o,
                                        void* hip_stream) {
  const char* who = "spec_verify_paged_attention";
  AttnLayout l;
  if (!attention_sizes_ok(who, a, o, &l)) return SV_ERR_INVALID;
  if (a->batch == 0) return SV_OK;
  const int32_t codes = o ? o->codes : SV_CODES_NONE;
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
  if (l.groups > 0 && (!o->groups || !o->prefix_len)) {
    set_err("%s: groups and prefix_len are required for num_groups %d", who, l.groups);
    return SV_ERR_INVALID;
  }
  if (codes != SV_CODES_NONE) {
    for (int64_t x : {a->k_page_stride, a->k_head_stride, a->k_token_stride, a->v_page_stride, a->v_head_stride, a->v_token_stride})
      if (x % 16) {
        set_err("%s: strides of codes need to be multiples of 16", who);
        return SV_ERR_INVALID;
      }
    if (!o->k_scale || !o->v_scale || !aligned16(o->k_scale) || !aligned16(o->v_scale)) {
      set_err("%s: k_scale and v_scale (16-byte aligned) are required", who);
      return SV_ERR_INVALID;
    }
    for (int64_t x : {o->k_scale_page_stride, o->k_scale_head_stride, o->v_scale_page_stride, o->v_scale_head_stride})
      if (x < 0 || x % 4 || x > (int64_t)1 << 40) {
        set_err("%s: strides of scales need to be multiples of 4", who);
        return SV_ERR_INVALID;
      }
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
  const int64_t need = spec_verify_attention_options_workspace(a, o);
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
  attention_workspace(a, l, static_cast<char*>(a->workspace), &p);
  if (codes != SV_CODES_NONE) {
    p.ks = o->k_scale;
    p.ks_page = o->k_scale_page_stride;
    p.ks_head = o->k_scale_head_stride;
    p.vs = o->v_scale;
    p.vs_page = o->v_scale_page_stride;
    p.vs_head = o->v_scale_head_stride;
  }
  const hipStream_t st = (hipStream_t)hip_stream;
  hipError_t e;
  if (l.groups == 0) {
    e = (codes == SV_CODES_E4M3   ? sv::launch_attention_e4m3
         : codes == SV_CODES_INT8 ? sv::launch_attention_int8
                                  : sv::launch_attention)(p, l.tiles.row_tiles, l.tiles.blocks, st);
  } else {
    p.G = l.groups;
    p.groups = o->groups;
    p.prefix_len = o->prefix_len;
    // The kernel for many rows takes strides in bytes in 32 bits; and its scores take
    // the scale on behind the mask, where a scale of 0 makes 0 * -inf.  (Scores scaled
    // in front of it cost 0.7 to 1 % of a long prefix's time: its registers are all in use.)
    const int64_t es = codes == SV_CODES_NONE ? 2 : 1;
    const int64_t most = std::max(std::max(a->k_page_stride, a->v_page_stride), a->page_size * std::max(a->k_token_stride, a->v_token_stride));
    if (l.many && (most * es > UINT32_MAX || p.scale_log2 == 0.f)) {
      l.many = false;
      l.tiles = l.together;
      p.prefix_parts = p.parts;
    }
    p.own_rows = 16 * l.tiles.row_tiles;
    p.prefix_rows = l.many ? sv::kAttnPrefixRows : p.own_rows;
    p.prefix_blocks = l.prefix_blocks;
    p.group_entries = l.many ? 0 : l.groups;
    p.entries = p.group_entries + a->batch;
    p.plan.entry = l.many ? p.plan.seq : p.plan.group;
    e = sv::launch_attention_plan(p, st);
    if (e == hipSuccess && l.many)
      e = (codes == SV_CODES_E4M3   ? sv::launch_attention_prefix_e4m3
           : codes == SV_CODES_INT8 ? sv::launch_attention_prefix_int8
                                    : sv::launch_attention_prefix)(p, st);
    if (e == hipSuccess)
      e = (codes == SV_CODES_E4M3   ? sv::launch_attention_shared_e4m3
           : codes == SV_CODES_INT8 ? sv::launch_attention_shared_int8
                                    : sv::launch_attention_shared)(p, l.tiles.row_tiles, l.tiles.blocks, st);
    if (e == hipSuccess) e = sv::launch_attention_merge(p, st);
  }
  if (e != hipSuccess) return hip_fail(who, e);
  return SV_OK;
}

int64_t spec_verify_cache_size(void) { return (int64_t)sizeof(spec_verify_cache); }

int64_t spec_verify_cache_workspace(const spec_verify_cache* c) {
  CacheLayout l;
  return cache_sizes_ok("spec_verify_cache_workspace", c, &l) ? l.bytes : SV_ERR_INVALID;
}

static int cache_reserve(const char* who, const spec_verify_cache* c, const spec_verify_codes* q, int32_t batch,
                         const int32_t* seqs, const int32_t* num_new, int64_t total_new, int32_t* start, int64_t* slots,
                         int32_t* positions, int32_t* status, void* hip_stream) {
  sv::CacheParams p;
  if (!cache_params(who, c, batch, &p, q)) return SV_ERR_INVALID;
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
  p.positions = positions;
  p.status = status;
  hipError_t e = sv::launch_cache_reserve(p, (hipStream_t)hip_stream);
  return e == hipSuccess ? SV_OK : hip_fail(who, e);
}

int spec_verify_cache_reserve(const spec_verify_cache* c, int32_t batch, const int32_t* seqs, const int32_t* num_new,
                              int64_t total_new, int32_t* start, int64_t* slots, int32_t* status, void* hip_stream) {
  return cache_reserve("spec_verify_cache_reserve", c, nullptr, batch, seqs, num_new, total_new, start, slots, nullptr, status,
                       hip_stream);
}

int spec_verify_coded_cache_reserve(const spec_verify_cache* c, const spec_verify_codes* q, int32_t batch, const int32_t* seqs,
                                    const int32_t* num_new, int64_t total_new, int32_t* start, int64_t* slots,
                                    int32_t* positions, int32_t* status, void* hip_stream) {
  return cache_reserve("spec_verify_coded_cache_reserve", c, q, batch, seqs, num_new, total_new, start, slots, positions, status,
                       hip_stream);
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

static int cache_compact(const char* who, const spec_verify_cache* c, const spec_verify_codes* q, int32_t* live, void* hip_stream) {
  sv::CacheParams p;
  if (!cache_params(who, c, 0, &p, q)) return SV_ERR_INVALID;
  p.live = live;
  hipError_t e = sv::launch_cache_compact(p, (hipStream_t)hip_stream);
  return e == hipSuccess ? SV_OK : hip_fail(who, e);
}

int spec_verify_cache_compact(const spec_verify_cache* c, int32_t* live, void* hip_stream) {
  return cache_compact("spec_verify_cache_compact", c, nullptr, live, hip_stream);
}

int spec_verify_coded_cache_compact(const spec_verify_cache* c, const spec_verify_codes* q, int32_t* live, void* hip_stream) {
  return cache_compact("spec_verify_coded_cache_compact", c, q, live, hip_stream);
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

int64_t spec_verify_codes_size(void) { return (int64_t)sizeof(spec_verify_codes); }

int spec_verify_coded_cache_write(const spec_verify_cache* c, const spec_verify_codes* q, int32_t layer, int64_t rows,
                                  const void* k_new, int64_t k_row_stride, int64_t k_head_stride, const void* v_new,
                                  int64_t v_row_stride, int64_t v_head_stride, const int64_t* slots, void* hip_stream) {
  const char* who = "spec_verify_coded_cache_write";
  if (!q) {
    set_err("%s: codes is NULL", who);
    return SV_ERR_INVALID;
  }
  sv::CacheParams p;
  if (!cache_params(who, c, 0, &p, q)) return SV_ERR_INVALID;
  if (layer < 0 || layer >= c->layers || rows < 0 || rows > sv::kCacheMaxRows || c->kv_heads > 2048) {
    set_err("%s: layer %d outside 0..%d, rows %lld outside 0..%d, or kv_heads %d above 2048", who, layer, c->layers - 1,
            (long long)rows, sv::kCacheMaxRows, c->kv_heads);
    return SV_ERR_INVALID;
  }
  if (rows == 0) return SV_OK;
  if (!k_new || !v_new || !slots || !aligned16(k_new) || !aligned16(v_new) ||
      !strides_ok(k_row_stride, k_head_stride, 0) || !strides_ok(v_row_stride, v_head_stride, 0)) {
    set_err("%s: k_new and v_new (16-byte aligned, strides in multiples of 8 elements) and slots are required", who);
    return SV_ERR_INVALID;
  }
  sv::RopeParams r{};
  r.rows = rows;
  r.KV = c->kv_heads;
  r.D = c->head_dim;
  r.bf16 = q->dtype == SV_BF16;
  r.k = k_new;
  r.k_row = k_row_stride;
  r.k_head = k_head_stride;
  r.v = v_new;
  r.v_row = v_row_stride;
  r.v_head = v_head_stride;
  rope_cache(c, q, layer, slots, p, &r);
  hipError_t e = sv::launch_rope(r, (hipStream_t)hip_stream);
  return e == hipSuccess ? SV_OK : hip_fail(who, e);
}

int spec_verify_cache_read(const spec_verify_cache* c, const spec_verify_codes* q, int32_t dtype, int32_t layer, int32_t batch,
                           const int32_t* seqs, const int32_t* first, const int32_t* count, int64_t total, void* k_out,
                           void* v_out, int32_t* status, void* hip_stream) {
  const char* who = "spec_verify_cache_read";
  sv::CacheParams p;
  if (!cache_params(who, c, 0, &p, q)) return SV_ERR_INVALID;
  if (batch < 0 || batch > SV_CACHE_MAX_SLOTS) {
    set_err("%s: batch %d outside 0..%d", who, batch, SV_CACHE_MAX_SLOTS);
    return SV_ERR_INVALID;
  }
  if ((dtype != SV_BF16 && dtype != SV_F16) || (q && q->dtype != dtype)) {
    set_err("%s: dtype %d is neither SV_BF16 nor SV_F16, or not what the codes were written from", who, dtype);
    return SV_ERR_INVALID;
  }
  if (layer < 0 || layer >= c->layers || total < 0 || total > sv::kCacheMaxRows) {
    set_err("%s: layer %d outside 0..%d, or total %lld outside 0..%d", who, layer, c->layers - 1, (long long)total,
            sv::kCacheMaxRows);
    return SV_ERR_INVALID;
  }
  if (batch == 0 && total != 0) {
    set_err("%s: total %lld belongs to no sequence", who, (long long)total);
    return SV_ERR_INVALID;
  }
  if (batch == 0) return SV_OK;
  if (!first || !count || (total > 0 && (!k_out || !v_out)) || !aligned16(k_out) || !aligned16(v_out)) {
    set_err("%s: first, count, k_out and v_out (16-byte aligned) are required", who);
    return SV_ERR_INVALID;
  }
  sv::CacheReadParams r{};
  r.B = batch;
  r.slots = c->slots;
  r.max_pages = c->max_pages;
  r.page_size = c->page_size;
  r.page_log2 = p.page_log2;
  r.num_pages = c->num_pages;
  r.max_len = p.max_len;
  r.kv_heads = c->kv_heads;
  r.D = c->head_dim;
  r.head_vecs = c->head_dim / 8;
  r.bf16 = dtype == SV_BF16;
  r.codes = q ? q->codes : SV_CODES_NONE;
  r.total = (int32_t)total;
  r.table = c->page_table;
  r.seq_len = c->seq_len;
  r.seqs = seqs;
  r.first = first;
  r.count = count;
  r.k = static_cast<char*>(c->k) + layer * p.layer_bytes;
  r.v = static_cast<char*>(c->v) + layer * p.layer_bytes;
  if (q) {
    r.ks = q->k_scale + layer * (p.scale_bytes / 4) * c->num_pages;
    r.vs = q->v_scale + layer * (p.scale_bytes / 4) * c->num_pages;
  }
  r.k_out = k_out;
  r.v_out = v_out;
  r.status = status;
  hipError_t e = sv::launch_cache_read(r, (hipStream_t)hip_stream);
  return e == hipSuccess ? SV_OK : hip_fail(who, e);
}

int64_t spec_verify_rope_args_size(void) { return (int64_t)sizeof(spec_verify_rope_args); }

int spec_verify_qk_norm_rope(const spec_verify_rope_args* a, const spec_verify_cache* c, const spec_verify_codes* q,
                             void* hip_stream) {
  const char* who = "spec_verify_qk_norm_rope";
  if (!a) {
    set_err("%s: args is NULL", who);
    return SV_ERR_INVALID;
  }
  if (a->dtype != SV_BF16 && a->dtype != SV_F16) {
    set_err("%s: dtype %d is neither SV_BF16 nor SV_F16", who, a->dtype);
    return SV_ERR_INVALID;
  }
  if (a->head_dim < 16 || a->head_dim > 512 || a->head_dim % 16 || a->rotary < 0 || a->rotary > a->head_dim || a->rotary % 16) {
    set_err("%s: head_dim %d or rotary %d is not a multiple of 16, up to 512 and head_dim", who, a->head_dim, a->rotary);
    return SV_ERR_INVALID;
  }
  if (a->heads < 1 || a->kv_heads < 1 || (int64_t)a->heads + a->kv_heads > 4096 || a->rows < 0 || a->rows > sv::kCacheMaxRows) {
    set_err("%s: heads %d and kv_heads %d outside 1..4096 together, or rows %lld outside 0..%d", who, a->heads, a->kv_heads,
            (long long)a->rows, sv::kCacheMaxRows);
    return SV_ERR_INVALID;
  }
  if ((a->q_weight || a->k_weight) && a->weight_dtype != SV_F32 && a->weight_dtype != a->dtype) {
    set_err("%s: weight_dtype %d is neither SV_F32 nor the dtype", who, a->weight_dtype);
    return SV_ERR_INVALID;
  }
  if (!(a->eps >= 0) || !isfinite((float)a->eps)) {
    set_err("%s: eps %g is negative or not finite", who, a->eps);
    return SV_ERR_INVALID;
  }
  sv::CacheParams p;
  if (c) {
    if (!cache_params(who, c, 0, &p, q)) return SV_ERR_INVALID;
    if (c->kv_heads != a->kv_heads || c->head_dim != a->head_dim || (q && q->dtype != a->dtype)) {
      set_err("%s: the cache has %d heads of %d, the keys %d of %d (or another type)", who, c->kv_heads, c->head_dim, a->kv_heads,
              a->head_dim);
      return SV_ERR_INVALID;
    }
    if (a->layer < 0 || a->layer >= c->layers) {
      set_err("%s: layer %d outside 0..%d", who, a->layer, c->layers - 1);
      return SV_ERR_INVALID;
    }
  } else if (q) {
    set_err("%s: codes without a cache", who);
    return SV_ERR_INVALID;
  }
  if (a->rows == 0) return SV_OK;
  if (!a->q || !a->k || !a->positions || !a->q_out || (a->rotary > 0 && !a->inv_freq) || (c != nullptr) != (a->v != nullptr) ||
      (c != nullptr) != (a->slots != nullptr) || (c != nullptr) != (a->k_out == nullptr)) {
    set_err("%s: q, k, positions, inv_freq and q_out are required, and k_out, or with a cache v and slots", who);
    return SV_ERR_INVALID;
  }
  for (const void* x : {a->q, a->k, a->v, a->q_weight, a->k_weight, (const void*)a->q_out, (const void*)a->k_out})
    if (!aligned16(x)) {
      set_err("%s: q, k, v, weights and outputs need 16-byte alignment", who);
      return SV_ERR_INVALID;
    }
  if (!strides_ok(a->q_row_stride, a->q_head_stride, 0) || !strides_ok(a->k_row_stride, a->k_head_stride, 0) ||
      (c && !strides_ok(a->v_row_stride, a->v_head_stride, 0))) {
    set_err("%s: strides need to be multiples of 8 elements", who);
    return SV_ERR_INVALID;
  }
  sv::RopeParams r{};
  r.rows = a->rows;
  r.H = a->heads;
  r.KV = a->kv_heads;
  r.D = a->head_dim;
  r.R = a->rotary;
  r.bf16 = a->dtype == SV_BF16;
  r.neighbours = a->interleaved != 0;
  r.weight_f32 = a->weight_dtype == SV_F32;
  r.eps = (float)a->eps;
  r.inv_dim = 1.f / (float)a->head_dim;
  r.q = a->q;
  r.q_row = a->q_row_stride;
  r.q_head = a->q_head_stride;
  r.k = a->k;
  r.k_row = a->k_row_stride;
  r.k_head = a->k_head_stride;
  r.v = a->v;
  r.v_row = a->v_row_stride;
  r.v_head = a->v_head_stride;
  r.positions = a->positions;
  r.inv_freq = a->inv_freq;
  r.q_weight = a->q_weight;
  r.k_weight = a->k_weight;
  r.q_out = a->q_out;
  r.k_out = a->k_out;
  if (c) rope_cache(c, q, a->layer, a->slots, p, &r);
  hipError_t e = sv::launch_rope(r, (hipStream_t)hip_stream);
  return e == hipSuccess ? SV_OK : hip_fail(who, e);
}

}  // extern "C"
