// Attention of a batch whose sequences share prefixes, for gfx950: the plan of
// a call, and its stages over the 16-bit cache (their kernel is in
// sv_attention_kernel.h).
//
// Softmax over a row's keys splits into parts (m, l, O) that join exactly, so
// a prefix that a group of sequences shares is read once for the rows of all
// of them instead of once for each.  A call is five launches:
//   plan     rows and units of both stages, every refusal
//   prefix   the groups' rows over the prefixes: k_attention's stage 1, or
//            k_prefix (sv_prefix.h) where a group has many rows; the parts' join
//   own      each sequence's tokens behind the prefix, starting from what the
//            prefix left for its rows; the parts' join

#include "sv_prefix.h"

namespace sv {

namespace {

// Rows or groups that do not add up, found by every block for itself.
__device__ __forceinline__ bool layout_bad(const AttnParams& P) {
  __shared__ unsigned long long sum;
  __shared__ int bad;
  const int t = threadIdx.x;
  if (t == 0) {
    sum = 0;
    bad = 0;
  }
  __syncthreads();
  unsigned long long r = 0;
  bool b = false;
  for (int i = t; i < P.B; i += kAtThreads) {
    const int K = P.num_draft[i];
    b |= K < 0 || K >= P.total_rows;
    r += (unsigned)max(K, 0) + 1u;
  }
  for (int g = t; g < P.G; g += kAtThreads) {
    const int a = P.groups[g], e = P.groups[g + 1];
    b |= a < 0 || e < a || e > P.B || (g == 0 && a != 0) || (g == P.G - 1 && e != P.B);
  }
  if (b) bad = 1;
  atomicAdd(&sum, r);
  __syncthreads();
  return bad || sum != (unsigned long long)P.total_rows;
}

// What can be said of sequence b without its pages: its slot and length, 0 or SV_ST_*.
struct Seq {
  int slot, len, status;
};
__device__ __forceinline__ Seq seq_check(const AttnParams& P, int b, int prefix, bool leads) {
  Seq s;
  s.slot = P.seqs ? P.seqs[b] : b;
  s.len = 0;
  s.status = 0;
  if ((unsigned)s.slot >= (unsigned)P.slots) {
    s.status = SV_ST_BAD_SEQ;
    return s;
  }
  s.len = P.seq_len[s.slot];
  if (s.len < 0 || s.len > P.max_len) {
    s.status = SV_ST_BAD_LENGTH;
  } else {
    // a leader that sits the round out still has the prefix
    const int n = leads ? 0 : P.num_draft[b] + 1;
    if (prefix < 0 || prefix > max(s.len - n, 0) || (!leads && !in_place(P, b, n, s.len))) s.status = SV_ST_BAD_LENGTH;
  }
  return s;
}

}  // namespace

// Block 0 makes the plan; block 1 + b looks at the pages of sequence b: those
// of the prefix have to be its leader's (the first sequence of its group), but
// for a partly filled last one, which may be a copy.
__global__ void __launch_bounds__(kAtThreads) k_attention_plan(AttnParams P, int own_rows, int group_rows) {
  extern __shared__ uint32_t dyn[];
  __shared__ uint32_t tr[kAtWaves], tu[kAtWaves];
  __shared__ int shared_g, shared_st;
  const int t = threadIdx.x, lane = t & (kWave - 1), wv = t / kWave;
  const bool bad = layout_bad(P);
  if (blockIdx.x > 0) {
    const int b = (int)blockIdx.x - 1;
    if (bad) {
      if (t == 0 && P.status) P.status[b] = SV_ST_BAD_LAYOUT;
      return;
    }
    if (t == 0) shared_st = 0;
    for (int g = t; g < P.G; g += kAtThreads)
      if (P.groups[g] <= b && b < P.groups[g + 1]) shared_g = g;
    __syncthreads();
    const int prefix = P.prefix_len[shared_g], lead = P.groups[shared_g];
    const Seq l = seq_check(P, lead, prefix, true), s = seq_check(P, b, prefix, false);
    int st = s.status | l.status;
    if (!st) {
      const int32_t* mine = P.table + (int64_t)s.slot * P.table_stride;
      const int32_t* theirs = P.table + (int64_t)l.slot * P.table_stride;
      const int mask = (1 << P.page_log2) - 1, whole = prefix >> P.page_log2;
      int f = 0;
      for (int i = t; i < whole; i += kAtThreads) {
        const int id = theirs[i];
        if (id != mine[i] || (unsigned)id >= (unsigned)P.num_pages) f = SV_ST_BAD_PAGE;
      }
      if (t == 0 && (prefix & mask) && (unsigned)theirs[whole] >= (unsigned)P.num_pages) f = SV_ST_BAD_PAGE;
      const int end = (s.len + mask) >> P.page_log2;
      for (int i = whole + t; i < end; i += kAtThreads)
        if ((unsigned)mine[i] >= (unsigned)P.num_pages) f = SV_ST_BAD_PAGE;
      if (f) atomicOr(&shared_st, f);
    }
    __syncthreads();
    if (t == 0) {
      st |= shared_st;
      P.plan.flags[b] = st;
      if (P.status) P.status[b] = st;
    }
    return;
  }
  if (t == 0) *P.plan.bad = bad ? 1 : 0;
  if (bad) {                                     // no stage has any work; the last one clears the outputs
    if (t == 0) P.plan.units[P.B] = P.plan.group_units[P.G] = 0;
    return;
  }
  uint32_t* rows = dyn;                          // [B + 1]
  uint32_t* first = dyn + P.B + 1;               // [G + 1]
  for (int g = t; g <= P.G; g += kAtThreads) first[g] = (uint32_t)P.groups[g];
  // exclusive prefix over the block of a thread's value, and the block's total
  auto scan = [&](uint32_t v, uint32_t* total, uint32_t* waves) {
    const uint32_t in = wave_incl_scan_u32(v);
    __syncthreads();
    if (lane == kWave - 1) waves[wv] = in;
    __syncthreads();
    uint32_t before = in - v;
    *total = 0;
    for (int i = 0; i < kAtWaves; ++i) {
      if (i < wv) before += waves[i];
      *total += waves[i];
    }
    return before;
  };
  uint32_t total;
  {
    const int per = (P.B + kAtThreads - 1) / kAtThreads;
    const int b0 = min(t * per, P.B), b1 = min(b0 + per, P.B);
    uint32_t r = 0;
    for (int b = b0; b < b1; ++b) r += (uint32_t)P.num_draft[b] + 1u;
    uint32_t at = scan(r, &total, tr);
    for (int b = b0; b < b1; ++b) {
      rows[b] = at;
      P.plan.rows[b] = (int)at;
      at += (uint32_t)P.num_draft[b] + 1u;
    }
    if (t == 0) P.plan.rows[P.B] = rows[P.B] = total;
    __syncthreads();
    auto own = [&](int b, bool write) -> uint32_t {
      int lo = 0, hi = P.G - 1;                  // the last group that begins at or before b and is not empty
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= (uint32_t)b) lo = mid;
        else hi = mid - 1;
      }
      const int prefix = P.prefix_len[lo];
      Seq s = seq_check(P, b, prefix, false);
      s.status |= seq_check(P, (int)first[lo], prefix, true).status;
      const int len = s.status ? 0 : s.len, f = s.status ? 0 : prefix;
      if (write) {
        P.plan.slot[b] = s.status ? -1 : s.slot;
        P.plan.len[b] = len;
        P.plan.first[b] = f;
      }
      const uint32_t n = rows[b + 1] - rows[b];
      const int blocks = max(1, (len + kUnitKeys - 1) / kUnitKeys - f / kUnitKeys);
      return (n * P.group + own_rows - 1) / own_rows * P.kv_heads * (uint32_t)blocks;
    };
    uint32_t u = 0;
    for (int b = b0; b < b1; ++b) u += own(b, true);
    uint32_t ua = scan(u, &total, tu);
    for (int b = b0; b < b1; ++b) {
      P.plan.units[b] = (int)ua;
      ua += own(b, false);
    }
    if (t == 0) P.plan.units[P.B] = (int)total;
  }
  {
    const int per = (P.G + kAtThreads - 1) / kAtThreads;
    const int g0 = min(t * per, P.G), g1 = min(g0 + per, P.G);
    auto units = [&](int g, bool write) -> uint32_t {
      const uint32_t n = rows[first[g + 1]] - rows[first[g]];
      int len = 0, slot = -1;
      if (n > 0) {
        const Seq l = seq_check(P, (int)first[g], P.prefix_len[g], true);
        if (!l.status) {
          len = P.prefix_len[g];
          slot = l.slot;
        }
      }
      if (write) {
        P.plan.group_rows[g] = (int)rows[first[g]];
        P.plan.group_slot[g] = slot;
        P.plan.group_len[g] = len;
      }
      return (n * P.group + group_rows - 1) / group_rows * P.kv_heads * (uint32_t)((len + kUnitKeys - 1) / kUnitKeys);
    };
    uint32_t u = 0;
    for (int g = g0; g < g1; ++g) u += units(g, true);
    uint32_t ua = scan(u, &total, tu);
    for (int g = g0; g < g1; ++g) {
      P.plan.group_units[g] = (int)ua;
      ua += units(g, false);
    }
    if (t == 0) {
      P.plan.group_units[P.G] = (int)total;
      P.plan.group_rows[P.G] = (int)rows[P.B];
    }
  }
}

hipError_t launch_attention_plan(const AttnParams& p, int own_rows, int group_rows, hipStream_t st) {
  const size_t lds = ((size_t)p.B + p.G + 2) * 4;
  hipLaunchKernelGGL(k_attention_plan, dim3((unsigned)p.B + 1), dim3(kAtThreads), lds, st, p, own_rows, group_rows);
  return hipGetLastError();
}

hipError_t launch_attention_shared(const AttnParams& p, int stage, int row_tiles, int blocks, hipStream_t st) {
  if (stage == kPrefix && row_tiles == kAttnManyRows) return launch_prefix_rows<codes::kNone>(p, blocks, st);
  return launch_shared<codes::kNone>(p, stage, row_tiles, blocks, st);
}

}  // namespace sv
