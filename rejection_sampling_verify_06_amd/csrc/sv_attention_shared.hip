// Attention of a batch whose sequences share prefixes, for gfx950: the plan of
// a call, and its stages over the 16-bit cache (their kernel is in
// sv_attention_kernel.h).
//
// Softmax over a row's keys splits into parts (m, l, O) that join exactly, so
// a prefix that a group of sequences shares is read once for the rows of all
// of them instead of once for each.  A call is three or four launches:
//   plan     rows and units of groups and sequences, every refusal
//   prefix   the groups' rows over the prefixes, where they are many (k_prefix,
//            sv_prefix.h)
//   tiles    each sequence's tokens behind its prefix, and groups of few rows over
//            theirs (k_attention)
//   merge    of all that belongs to a row
//
// Measured on one MI355X (rocprofv3, plan + prefix + tiles + merge): 4 branches of
// 2000 tokens 5 + 8 + 9 us; 64 sequences behind 32768 tokens 9 + 186 + 25 + 11 us
// (one by one, without groups, 64 times the prefix's bytes: 1.7 ms at 5 TB/s); 8 groups
// of 8 behind 8000 over e4m3 8 + 46 + 30 + 12 us.  Plan and merge are chains of loads: the
// merge's 17 parts a row took 14 us with one load after the other, 8.5 with eight parts'
// under way; 11 us of 64 sequences' merge are its 50 MB of parts.

#include "sv_prefix.h"

namespace sv {

namespace {

// Rows or groups that do not add up, found by every block for itself; and, on
// the way, the rows in front of sequence b and its group.
struct Layout {
  bool bad;
  int row0, group;
};
__device__ __forceinline__ Layout layout(const AttnParams& P, int b) {
  __shared__ unsigned long long sum;
  __shared__ int bad, row0, group;
  const int t = threadIdx.x;
  if (t == 0) {
    sum = 0;
    bad = row0 = group = 0;
  }
  __syncthreads();
  unsigned long long r = 0;
  uint32_t before = 0;
  bool f = false;
  for (int i = t; i < P.B; i += kAtThreads) {
    const int K = P.num_draft[i];
    f |= K < 0 || K >= P.total_rows;
    const uint32_t n = (uint32_t)max(K, 0) + 1u;
    r += n;
    if (i < b) before += n;
  }
  for (int g = t; g < P.G; g += kAtThreads) {
    const int a = P.groups[g], e = P.groups[g + 1];
    f |= a < 0 || e < a || e > P.B || (g == 0 && a != 0) || (g == P.G - 1 && e != P.B);
    if (a <= b && b < e) group = g;              // one thread's, where the groups are in order
  }
  if (f) bad = 1;
  if (r) atomicAdd(&sum, r);
  if (before) atomicAdd(&row0, (int)before);
  __syncthreads();
  return Layout{bad || sum != (unsigned long long)P.total_rows, row0, group};
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
__global__ void __launch_bounds__(kAtThreads) k_attention_plan(AttnParams P) {
  extern __shared__ uint32_t dyn[];
  __shared__ uint32_t tw[kAtWaves];
  __shared__ int shared_st;
  const int t = threadIdx.x, lane = t & (kWave - 1), wv = t / kWave;
  const int b = (int)blockIdx.x - 1;
  if (t == 0) shared_st = 0;
  const Layout at = layout(P, b);
  const bool bad = at.bad;
  if (b >= 0) {
    if (bad) {
      if (t == 0 && P.status) P.status[b] = SV_ST_BAD_LAYOUT;
      return;
    }
    const int n = P.num_draft[b] + 1;
    for (int i = t; i < n; i += kAtThreads) P.plan.row_seq[at.row0 + i] = b;
    const int prefix = P.prefix_len[at.group], lead = P.groups[at.group];
    const Seq l = seq_check(P, lead, prefix, true), s = seq_check(P, b, prefix, false);
    int st = s.status | l.status;
    if (!st) {
      const int32_t* mine = P.table + (int64_t)s.slot * P.table_stride;
      const int32_t* theirs = P.table + (int64_t)l.slot * P.table_stride;
      const int mask = (1 << P.page_log2) - 1, whole = prefix >> P.page_log2;
      int f = 0;
      // loads of eight pages of both at once: one at a time 2048 pages took 11.5 us
      for (int i = t; i < whole; i += 8 * kAtThreads) {
        int a[8], e[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int at = min(i + k * kAtThreads, whole - 1);
          a[k] = theirs[at];
          e[k] = mine[at];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (a[k] != e[k] || (unsigned)a[k] >= (unsigned)P.num_pages) f = SV_ST_BAD_PAGE;
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
  if (bad) {                                     // no tile has any work; the merge clears the outputs
    if (t == 0) P.plan.units[P.entries] = P.plan.group_units[P.G] = 0;
    return;
  }
  uint32_t* rows = dyn;                          // [B + 1]
  uint32_t* first = dyn + P.B + 1;               // [G + 1] first sequences
  uint32_t* mine = first + P.G + 1;              // [B] units of a sequence, or of a group
  // exclusive prefix over the block of a thread's value, and the block's total
  auto scan = [&](uint32_t v, uint32_t* total) {
    const uint32_t in = wave_incl_scan_u32(v);
    __syncthreads();
    if (lane == kWave - 1) tw[wv] = in;
    __syncthreads();
    uint32_t before = in - v;
    *total = 0;
    for (int i = 0; i < kAtWaves; ++i) {
      if (i < wv) before += tw[i];
      *total += tw[i];
    }
    return before;
  };
  for (int g = t; g <= P.G; g += kAtThreads) first[g] = (uint32_t)P.groups[g];
  const int per = (P.B + kAtThreads - 1) / kAtThreads, b0 = min(t * per, P.B), b1 = min(b0 + per, P.B);
  const int gper = (P.G + kAtThreads - 1) / kAtThreads, g0 = min(t * gper, P.G), g1 = min(g0 + gper, P.G);
  uint32_t total, tiles, units;
  {
    uint32_t r = 0;
    for (int b = b0; b < b1; ++b) r += (uint32_t)P.num_draft[b] + 1u;
    uint32_t at = scan(r, &total);
    for (int b = b0; b < b1; ++b) {
      rows[b] = at;
      at += (uint32_t)P.num_draft[b] + 1u;
    }
    if (t == 0) rows[P.B] = total;
    __syncthreads();
  }
  auto ceil_div = [](uint32_t a, uint32_t b) { return (a + b - 1) / b; };
  {
    // the groups: their tiles, and units where the kernel for many rows takes them
    auto count = [&](int g) { return ceil_div((rows[first[g + 1]] - rows[first[g]]) * (uint32_t)P.group, (uint32_t)P.prefix_rows) * (uint32_t)P.kv_heads; };
    uint32_t c = 0, u = 0;
    for (int g = g0; g < g1; ++g) c += count(g);
    uint32_t at = scan(c, &tiles);
    for (int g = g0; g < g1; ++g) {
      AttnRecord rec{};
      rec.row0 = (int)rows[first[g]];
      rec.n = (int)rows[first[g + 1]] - rec.row0;
      rec.slot = -1;
      if (rec.n > 0) {
        const Seq l = seq_check(P, (int)first[g], P.prefix_len[g], true);
        if (!l.status) {
          rec.len = P.prefix_len[g];
          rec.slot = l.slot;
        }
      }
      rec.tile0 = (int)at;
      P.plan.group[g] = rec;
      const uint32_t n = count(g);
      at += n;
      u += mine[g] = n * (uint32_t)((rec.len + kUnitKeys - 1) / kUnitKeys);
    }
    uint32_t ua = scan(u, &units);
    int32_t* to = P.group_entries ? P.plan.units : P.plan.group_units;
    for (int g = g0; g < g1; ++g) {
      to[g] = (int)ua;
      ua += mine[g];
    }
    if (t == 0) {
      P.plan.group_units[P.G] = P.group_entries ? 0 : (int)units;
      if (!P.group_entries) units = 0;
    }
    if (!P.group_entries) units = 0;
    __syncthreads();                             // `mine` is used again
  }
  {
    uint32_t c = 0, u = 0;
    auto count = [&](int b) { return ceil_div((rows[b + 1] - rows[b]) * (uint32_t)P.group, (uint32_t)P.own_rows) * (uint32_t)P.kv_heads; };
    for (int b = b0; b < b1; ++b) c += count(b);
    uint32_t at = tiles + scan(c, &total);
    for (int b = b0; b < b1; ++b) {
      int lo = 0, hi = P.G - 1;                  // the last group that begins at or before b: not empty
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= (uint32_t)b) lo = mid;
        else hi = mid - 1;
      }
      const int prefix = P.prefix_len[lo];
      Seq s = seq_check(P, b, prefix, false);
      s.status |= seq_check(P, (int)first[lo], prefix, true).status;
      AttnRecord rec{};
      rec.slot = s.status ? -1 : s.slot;
      rec.len = s.status ? 0 : s.len;
      rec.first = s.status ? 0 : prefix;
      rec.row0 = (int)rows[b];
      rec.n = (int)(rows[b + 1] - rows[b]);
      rec.tile0 = (int)at;
      rec.group_row = (int)(rows[b] - rows[first[lo]]);
      rec.group_tile0 = P.plan.group[lo].tile0;
      P.plan.seq[b] = rec;
      const uint32_t n = count(b);
      at += n;
      u += mine[b] = n * (uint32_t)max(1, (rec.len + kUnitKeys - 1) / kUnitKeys - rec.first / kUnitKeys);
    }
    uint32_t ua = units + scan(u, &total);
    for (int b = b0; b < b1; ++b) {
      P.plan.units[P.group_entries + b] = (int)ua;
      ua += mine[b];
    }
    if (t == 0) P.plan.units[P.entries] = (int)(units + total);
  }
}

// Adds up, for 16 rows of a key head in packed order, what the tiles of their
// groups and sequences came to: states of tiles that one block had whole, parts
// of others.  A lane has a row and D / 64 fours of the head dimension, the waves
// a quarter of it each; kBatch tiles' worth of loads are under way at a time.
template <bool BF, int D>
__global__ void __launch_bounds__(kAtThreads) k_attention_merge(AttnParams P) {
  constexpr int GN = D / 64;                     // a lane's fours
  constexpr int kBatch = D == 256 ? 4 : 8;
  const int t = threadIdx.x, lane = t & (kWave - 1), wv = t / kWave, g = lane >> 4;
  const int head = (int)blockIdx.y, four0 = wv * (D / 16) + g * GN;
  const int rows = P.total_rows * P.group;       // of a key head
  const int X = (int)blockIdx.x * 16 + (lane & 15);
  const bool in = X < rows;
  const int row = (in ? X : 0) / P.group, hh = (in ? X : 0) - row * P.group;
  const int64_t at = (int64_t)row * P.heads + head * P.group + hh;
  const bool bad = *P.plan.bad != 0;
  // loaded beside `bad`: where the layout is, it may be anything
  const int b = min((unsigned)P.plan.row_seq[row], (unsigned)P.B - 1u);
  const AttnRecord rec = P.plan.seq[b];
  const int flags = P.plan.flags[b];
  f32x4 acc[GN];
  float M = -INFINITY, L = 0.f;
#pragma unroll
  for (int j = 0; j < GN; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (bad) {
    L = __builtin_nanf("");
  } else {
    const int R = (row - rec.row0) * P.group + hh, mb = R / P.own_rows;
    const int pR = R + rec.group_row * P.group, pmb = pR / P.prefix_rows;
    const int2 mine = P.plan.tile[rec.tile0 + mb * P.kv_heads + head];
    const int2 theirs = rec.first > 0 ? P.plan.tile[rec.group_tile0 + pmb * P.kv_heads + head] : make_int2(0, 0);
    const int parts = flags ? 0 : mine.y + theirs.y;
    if (flags) L = __builtin_nanf("");
    const int64_t total = (int64_t)P.total_rows * P.heads, sr = state_row(P, row, head, hh);
    const int most = wave_max_i(parts);
    for (int k0 = 0; k0 < most; k0 += kBatch) {
      float m[kBatch], l[kBatch];
      f32x4 v[kBatch][GN];
      uint32_t wholes = 0;                       // looked at behind all loads: here it would wait for each
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (k0 + i >= most) break;
        // No branch here depends on the lane: a register written on one side and
        // loaded on the other is waited for.  Lanes out of parts load again.
        const int kk = min(k0 + i, max(parts - 1, 0));
        const bool own = kk < mine.y;
        const int k = own ? kk : kk - mine.y;
        const int2 tile = own ? mine : theirs;
        const int tm = own ? P.own_rows : P.prefix_rows, r = own ? R - mb * P.own_rows : pR - pmb * P.prefix_rows;
        const bool whole = tile.y == 1;
        const float* part = part_at(own ? P.parts : P.prefix_parts, tile.x + k, k == 0 ? 1 : 0, tm, D);
        const float* pm = whole ? P.state_m + (own ? total : 0) + sr : part + tm * D + r;
        const float* po = whole ? P.state_o + ((own ? total * (D / 4) : 0) + sr) * 4 : part + r * 4;
        const int64_t four = 4 * (whole ? total : (int64_t)tm);
        m[i] = *pm;
        l[i] = pm[whole ? 0 : tm];
        wholes |= (uint32_t)whole << i;
#pragma unroll
        for (int j = 0; j < GN; ++j) v[i][j] = *(const f32x4*)(po + (four0 + j) * four);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (k0 + i >= parts) continue;
        // Nothing else is left out: where the row's weights are 0 (m = -inf) its O is 0,
        // unless it saw a value that is not finite, and where its scores are all NaN l is.
        const float li = !(wholes >> i & 1) ? l[i] : m[i] == -INFINITY ? 0.f : 1.f;
        const float nm = fmaxf(M, m[i]);
        const float f0 = M == nm ? 1.f : at_exp2(M - nm), f1 = m[i] == nm ? 1.f : at_exp2(m[i] - nm);
        M = nm;
        L = L * f0 + li * f1;
#pragma unroll
        for (int j = 0; j < GN; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[j][c] = fmaf(v[i][j][c], f1, acc[j][c] * f0);
      }
    }
  }
  if (!in) return;
  const float inv = L == 0.f ? 0.f : 1.f / L;    // NaN stays
#pragma unroll
  for (int j = 0; j < GN; ++j) {
    float x[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = L != L ? L : acc[j][c] * inv;
    *(u32x2*)((uint16_t*)P.out + at * D + (four0 + j) * 4) = u32x2{pack16<BF>(x[0], x[1]), pack16<BF>(x[2], x[3])};
  }
  if (P.lse && wv == 0 && g == 0) P.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

hipError_t launch_attention_plan(const AttnParams& p, hipStream_t st) {
  const size_t lds = (2 * (size_t)p.B + p.G + 2) * 4;
  hipLaunchKernelGGL(k_attention_plan, dim3((unsigned)p.B + 1), dim3(kAtThreads), lds, st, p);
  return hipGetLastError();
}

hipError_t launch_attention_merge(const AttnParams& p, hipStream_t st) {
  const dim3 grid((unsigned)(((int64_t)p.total_rows * p.group + 15) / 16), (unsigned)p.kv_heads), block(kAtThreads);
  switch (p.head_dim * 2 + (p.bf16 ? 1 : 0)) {
    case 64 * 2: hipLaunchKernelGGL((k_attention_merge<false, 64>), grid, block, 0, st, p); break;
    case 64 * 2 + 1: hipLaunchKernelGGL((k_attention_merge<true, 64>), grid, block, 0, st, p); break;
    case 128 * 2: hipLaunchKernelGGL((k_attention_merge<false, 128>), grid, block, 0, st, p); break;
    case 128 * 2 + 1: hipLaunchKernelGGL((k_attention_merge<true, 128>), grid, block, 0, st, p); break;
    case 256 * 2: hipLaunchKernelGGL((k_attention_merge<false, 256>), grid, block, 0, st, p); break;
    case 256 * 2 + 1: hipLaunchKernelGGL((k_attention_merge<true, 256>), grid, block, 0, st, p); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

hipError_t launch_attention_shared(const AttnParams& p, int row_tiles, int blocks, hipStream_t st) {
  return p.bf16 ? launch_type<true, codes::kNone, true>(p, row_tiles, blocks, st) : launch_type<false, codes::kNone, true>(p, row_tiles, blocks, st);
}

hipError_t launch_attention_prefix(const AttnParams& p, hipStream_t st) { return launch_prefix_rows<codes::kNone>(p, st); }

}  // namespace sv
