// The kernels of attention over a paged key-value cache, for gfx950 (internal;
// instantiated by sv_attention*.hip).
//
// Sequence b brings n = num_draft[b] + 1 query rows (packed like a verify
// call's target rows; n = 1 is plain decoding) and holds L = seq_len[b]
// tokens in its pages, the new ones among them.  Row i sees positions
// j <= L - n + i, with a window only the last `window` of them:
//   o_i = sum_j softmax_j(scale q_i . k_j) v_j
// in one pass over the cache, with a running maximum m, sum l and
// unnormalised O:  O += 2^(s_j - m) v_j,  l += 2^(s_j - m),  s in log2 units.
//
// Bound by the cache's bytes.  The rows of all query heads that share a key
// head form one tile (16 MT rows), so that each key and value is read once:
//   S^T = K Q^T   (keys x rows)     O^T += V^T P^T   (head dim x rows)
// with 16x16x32 MFMAs.  In this orientation a lane holds the scores of one
// row (column lane & 15) for keys 4g..4g+3 of two 16-key tiles (g = lane >>
// 4), and that is the layout of P^T as the second product's right operand if
// the reduction's slots are numbered so: slot (g, e) is key 4g + e of the
// first tile for e < 4, key 4g + e - 4 of the second above.  V^T is taken
// under the same numbering: a lane loads D/16 adjacent elements of the 8 rows
// of its slots and pairs them with byte permutes.  Neither scores nor values
// pass through shared memory; K and V come straight from the pages into
// registers, K of the next 32 keys while the softmax runs, V of them while
// the next scores are formed.
//
// P is split into two halves of the 16-bit type, p = hi + lo, each its own
// product: rounding p once would put an error of the output's own rounding
// on top of it, and the second product hides behind the cache's reads.  A
// bfloat16 pair holds a weight to 2^-16, a float16 pair to 2^-22 and no finer
// than its smallest step of 2^-24: there m is the maximum less 14, so that the
// weights reach up to 2^14 and the step is 2^-38 of the largest.  (Three
// bfloat16 hold all 24 bits, for the last bit of 1 in 1000 outputs: 8 to 24 rows
// of 128 133.5 -> 134.5 us, 16 and 36 rows of two long sequences 87 -> 89.5, 64
// rows of 64 106 -> 111.)
//
// Work is cut into units of 128 keys of one (sequence, row tile, key head)
// and dealt out in equal contiguous ranges, one per block, so that neither a
// few long sequences nor a ragged batch leaves blocks idle.  The lengths are
// only known on the device: every block forms the prefix of the units for
// itself.  A range may end inside a tile; such parts (at most two per block)
// go to the workspace as (O, m, l), and k_attention_join adds them up in
// order.
//
// Measured on one MI355X (rocprofv3, both kernels): 32 sequences of 4096
// tokens, 8 key heads of 128, 24 rows a tile, 97 + 5 us (5.5 TB/s of keys and
// values), of 16384 tokens 368 + 11 us (5.8 TB/s); one row, 99 + 5 us; 64
// sequences of 4096, 8 heads of 64, 95 + 4 us (5.7 TB/s); one token of one
// sequence of 777, 7 + 4 us.  A large device copy moves 5.1 TB/s here.

// Over codes (C, see sv_codes.h) the same, from half the bytes: scores are
// products of the queries with the codes, times the key's scale; the values'
// scales go into the weights in front of their split, and codes are bfloat16
// numbers exactly, also where the queries are float16 (whose range a weight
// times a scale would leave).  Half the bytes leave less time to hide the
// unpacking in, so two waves share a SIMD everywhere, and three row tiles go
// without branches between their products: 36 rows over int8 226 us with one
// wave a SIMD, 134 with two; 24 and 36 rows over e4m3 85 and 124 us with branches
// where codes without a number are looked for, which spilled, 81 and 100 without.
// Measured: 32 sequences of 1024 to 8192, up to 24 rows, e4m3 68 + 7 us (300 MB,
// 4.4 TB/s), of which a tile's start and end take some 10; 98925 and 116850
// tokens with 16 and 36 rows, int8 under float16 116 + 8 us (456 MB, 3.9 TB/s:
// products, unpacking and softmax of 36 rows take as long as the reads); 16 sequences in a
// window of 4096, heads of 256, 28 + 5 us; one token of 777, 8 + 4 us.
//
// With shared prefixes (S) the kernel's entries are groups, whose rows are those
// of all members and whose keys are the prefix, and sequences, whose keys begin
// behind it.  What a tile of either comes to goes to the workspace, and
// k_attention_merge (sv_attention_shared.hip) adds up what belongs to a row.

#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "sv_codes.h"
#include "sv_internal.h"
#include "sv_wave.h"

namespace sv {

namespace {

using namespace wave;

using codes::u32x2;
using codes::u32x4;
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kAtThreads = 256;
constexpr int kAtWaves = kAtThreads / kWave;
constexpr int kTileKeys = 32;                    // keys a wave takes at a time
constexpr int kUnitKeys = kTileKeys * kAtWaves;  // keys of a unit of work
static_assert(kUnitKeys == kAttnUnitKeys, "unit of work");
constexpr float kLn2 = 0.693147180559945309417f;

// a value every lane holds, as a scalar
__device__ __forceinline__ int uni(int x) { return __builtin_amdgcn_readfirstlane(x); }

__device__ __forceinline__ float at_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

template <bool BF>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// shared memory between the lanes of one wave
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// two floats rounded to the 16-bit type (to nearest even), a in the low half
template <bool BF>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if constexpr (BF) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    const b2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
  } else {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    const h2 v = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, v);
  }
}
template <bool BF>
__device__ __forceinline__ float lo16(uint32_t w) {
  if constexpr (BF) return __uint_as_float(w << 16);
  else return (float)__builtin_bit_cast(_Float16, (uint16_t)w);
}
template <bool BF>
__device__ __forceinline__ float hi16(uint32_t w) {
  if constexpr (BF) return __uint_as_float(w & 0xFFFF0000u);
  else return (float)__builtin_bit_cast(_Float16, (uint16_t)(w >> 16));
}

// What the weights of a row with maximum m are taken against.  Lowered by 14
// for float16; above 2^24, where 14 less may not be a float32, scores are known
// to no better than 1, and the weights stay at or below 1.
template <bool BF>
__device__ __forceinline__ float reference(float m) {
  return !BF && fabsf(m) < 0x1p24f ? m - 14.f : m;
}

// the low half is an infinity or NaN
template <bool BF>
__device__ __forceinline__ bool not_finite(uint32_t w) {
  constexpr uint32_t EX = BF ? 0x7F80u : 0x7C00u;
  return (w & EX) == EX;
}
template <bool BF>
constexpr uint32_t kOne = BF ? 0x3F80u : 0x3C00u;

// maximum over the four lanes that share a column (lanes l, l ^ 16, l ^ 32, l ^ 48)
__device__ __forceinline__ float column_max(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float column_sum(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// A sequence of the round, as every block works it out for itself.
struct Extent {
  int slot;       // row of page_table and seq_len; -1: refused
  int len;        // cached tokens (0 for a refused sequence)
  int first;      // first position any row sees
  int blk0;       // first 128-key block any row sees
  int nblk;       // blocks, at least 1 (an empty sequence still writes its rows)
};

// the n new tokens lie where they were reserved
__device__ __forceinline__ bool in_place(const AttnParams& P, int b, int n, int len) {
  return !P.start || (P.start[b] >= 0 && P.start[b] == len - n);
}

__device__ __forceinline__ Extent seq_extent(const AttnParams& P, int b, int n) {
  Extent x;
  x.slot = P.seqs ? P.seqs[b] : b;
  const int len = P.seq_len[(unsigned)x.slot < (unsigned)P.slots ? x.slot : 0];
  const bool ok = (unsigned)x.slot < (unsigned)P.slots && len >= 0 && len <= P.max_len && in_place(P, b, n, len);
  x.slot = ok ? x.slot : -1;
  x.len = ok ? len : 0;
  x.first = P.window > 0 ? max(0, x.len - n + 1 - P.window) : 0;
  x.blk0 = x.first / kUnitKeys;
  x.nblk = max(1, (x.len + kUnitKeys - 1) / kUnitKeys - x.blk0);
  return x;
}

// Prefix sums of the sequences' rows and units of work, B + 1 entries each in
// shared memory, for tiles of TM rows.
__device__ __forceinline__ bool plan(const AttnParams& P, int TM, uint32_t* rows, uint32_t* units) {
  __shared__ uint32_t tr[kAtWaves], tu[kAtWaves];
  __shared__ int bad;
  const int t = threadIdx.x, lane = t & (kWave - 1), w = t / kWave;
  if (t == 0) bad = 0;
  __syncthreads();
  const int per = (P.B + kAtThreads - 1) / kAtThreads;
  const int b0 = min(t * per, P.B), b1 = min(b0 + per, P.B);
  uint32_t r = 0, u = 0;
  for (int b = b0; b < b1; ++b) {
    const int K = P.num_draft[b], n = min(max(K, 0), P.total_rows - 1) + 1;
    const Extent x = seq_extent(P, b, n);
    if (n != K + 1) bad = 1;
    rows[b] = r;                                 // within this thread's sequences for now
    units[b] = u;
    r += (uint32_t)n;
    u += (uint32_t)((n * P.group + TM - 1) / TM * P.kv_heads) * (uint32_t)x.nblk;
  }
  const uint32_t ir = wave_incl_scan_u32(r), iu = wave_incl_scan_u32(u);
  if (lane == kWave - 1) {
    tr[w] = ir;
    tu[w] = iu;
  }
  __syncthreads();
  uint32_t ar = ir - r, au = iu - u;
  for (int i = 0; i < w; ++i) {
    ar += tr[i];
    au += tu[i];
  }
  for (int b = b0; b < b1; ++b) {
    rows[b] += ar;
    units[b] += au;
  }
  if (t == kAtThreads - 1) {
    rows[P.B] = ar + r;
    units[P.B] = au + u;
    if (ar + r != (uint32_t)P.total_rows) bad = 1;
  }
  __syncthreads();
  return bad == 0;
}

// eight codes as 16-bit numbers, in order
template <bool BF, int C>
__device__ __forceinline__ u32x4 widen8(uint32_t a, uint32_t b) {
  u32x4 x;
  if constexpr (C == codes::kE4m3) {
    if constexpr (BF) {
      x[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, false));
      x[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, true));
      x[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, false));
      x[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, true));
    } else {
      x[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.f, false));
      x[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.f, true));
      x[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.f, false));
      x[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.f, true));
    }
  } else if constexpr (BF) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = i < 2 ? a : b;
      x[i] = pack16<true>((float)(int8_t)(w >> (16 * (i & 1))), (float)(int8_t)(w >> (16 * (i & 1) + 8)));
    }
  } else {
    // 1024 + (c + 128) by its bits, less 1152: exact
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = (i < 2 ? a : b) ^ 0x80808080u;
      const uint32_t y = __builtin_amdgcn_perm(0x64646464u, w, (i & 1) ? 0x04030402u : 0x04010400u);
      x[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(h2, y) - h2{(_Float16)1152.f, (_Float16)1152.f});
    }
  }
  return x;
}

// bit 7 of each byte that is a code without a number (e4m3 has two)
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// The right order of bytes for the second product: of four elements (a byte
// each) of eight keys, element i's eight codes as 16-bit numbers.
template <int C>
__device__ __forceinline__ void turn_codes(const uint32_t* k, u32x4 (&out)[4]) {
  if constexpr (C == codes::kInt8) {             // each code is a number of its own on the way: nothing to turn
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) out[i][j] = pack16<true>((float)(int8_t)(k[2 * j] >> (8 * i)), (float)(int8_t)(k[2 * j + 1] >> (8 * i)));
    return;
  }
  uint32_t t[2][4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t a = __builtin_amdgcn_perm(k[4 * h + 1], k[4 * h], 0x05010400u), b = __builtin_amdgcn_perm(k[4 * h + 3], k[4 * h + 2], 0x05010400u);
    const uint32_t c = __builtin_amdgcn_perm(k[4 * h + 1], k[4 * h], 0x07030602u), d = __builtin_amdgcn_perm(k[4 * h + 3], k[4 * h + 2], 0x07030602u);
    t[h][0] = __builtin_amdgcn_perm(b, a, 0x05040100u);
    t[h][1] = __builtin_amdgcn_perm(b, a, 0x07060302u);
    t[h][2] = __builtin_amdgcn_perm(d, c, 0x05040100u);
    t[h][3] = __builtin_amdgcn_perm(d, c, 0x07060302u);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = widen8<true, C>(t[0][i], t[1][i]);
}

// What a block that starts inside a tile leaves for the join.
struct Part {
  int first_unit, end_unit;   // the tile's units; first_unit -1: the block starts at a tile's beginning
  int row0, n;                // the sequence's packed rows
  int head, mb;
  uint32_t U, W;              // all units, and the blocks they are dealt out to
};
static_assert(sizeof(Part) == kAttnPartBytes, "part record");

// block w of W takes units [w U / W, (w + 1) U / W); the block that holds unit u
__device__ __forceinline__ uint32_t range_start(uint32_t w, uint32_t W, uint32_t U) { return (uint32_t)((uint64_t)w * U / W); }
__device__ __forceinline__ uint32_t range_of(uint32_t u, uint32_t W, uint32_t U) {
  return (uint32_t)((((uint64_t)u + 1) * W - 1) / U);
}

// a part in the workspace: TM rows of O, then what their weights were taken against, then TM sums
__device__ __forceinline__ float* part_at(float* parts, int w, int slot, int TM, int D) {
  return parts + ((int64_t)w * 2 + slot) * TM * (D + 2);
}

// Shared prefixes: row X of a key head (its rows in packed order) in what whole tiles leave.
__device__ __forceinline__ int64_t state_row(const AttnParams& P, int row0, int head, int R) {
  return ((int64_t)head * P.total_rows + row0) * P.group + R;
}

}  // namespace

// S: with shared prefixes, whose plan is in the workspace
template <bool BF, int D, int MT, int C, bool S>
__global__ void __launch_bounds__(kAtThreads, D * MT <= 64 ? 4 : C != codes::kNone || (D * MT <= 256 && D < 256) ? 2 : 1) k_attention(AttnParams P) {
  constexpr bool PB = BF || C != codes::kNone;   // the second product's type
  constexpr int ES = C != codes::kNone ? 1 : 2;  // bytes of a cached number
  constexpr int TM = 16 * MT;                    // rows of a tile
  constexpr int NS = D / 32;                     // 32-element slices of the head dimension (scores)
  constexpr int NJ = D / 16;                     // 16-row tiles of O^T; also a lane's elements of a V row
  constexpr int VW = NJ * ES / 4;                // dwords of those
  constexpr int NL = D * ES / 64;                // 16-byte loads of a lane's part of a key
  constexpr bool kTight = C != codes::kNone && D * MT > 256;   // registers are short: the order of stages is kept
  extern __shared__ uint32_t dyn[];
  const int nseq = S ? P.entries : P.B;
  uint32_t* rows = dyn;                          // not with S
  uint32_t* units = S ? dyn : dyn + P.B + 1;
  constexpr int RS = 256 / D;                    // of a lane's 4 rows of each O^T tile, those that are joined at a time
  __shared__ u32x4 qs[MT][NS][kWave];        // the tile's queries as the first product's right operands
  __shared__ float ml[kAtWaves][2][TM];
  __shared__ float ob[kAtWaves][16][64 + 4];     // 64 of the D values of 16 rows, rows 4 banks apart
  const int t = threadIdx.x, lane = t & (kWave - 1), wv = uni(t / kWave);
  const int g = lane >> 4, col = lane & 15;
  bool ok = true;
  if constexpr (S) {
    for (int i = t; i <= nseq; i += kAtThreads) units[i] = (uint32_t)P.plan.units[i];   // none where the layout is bad
    __syncthreads();
  } else {
    ok = plan(P, TM, rows, units);
  }
  Part* desc = reinterpret_cast<Part*>(P.desc);
  const uint32_t U = (uint32_t)uni((int)units[nseq]), W = min((uint32_t)gridDim.x, U);
  const uint32_t w = blockIdx.x;
  if (!ok) {                                     // the rows do not add up: every output is cleared
    if (t == 0) desc[w].first_unit = -1;
    const int64_t total = (int64_t)P.total_rows * P.heads * D;
    for (int64_t i = (int64_t)w * kAtThreads + t; i < total; i += (int64_t)gridDim.x * kAtThreads)
      ((uint16_t*)P.out)[i] = BF ? 0x7FC0 : 0x7E00;
    if (P.lse)
      for (int64_t i = (int64_t)w * kAtThreads + t; i < (int64_t)P.total_rows * P.heads; i += (int64_t)gridDim.x * kAtThreads)
        P.lse[i] = __builtin_nanf("");
    return;
  }
  if (w >= W) {
    if (!S && t == 0) desc[w].first_unit = -1;
    return;
  }
  uint32_t u = range_start(w, W, U);
  const uint32_t u_end = range_start(w + 1, W, U);
  // the sequence that holds unit u
  int b = 0;
  for (int step = S ? 8192 : 4096; step > 0; step >>= 1)
    if (b + step < nseq && (uint32_t)uni((int)units[b + step]) <= u) b += step;
  bool first_part = true;
  while (u < u_end) {
    while ((uint32_t)uni((int)units[b + 1]) <= u) ++b;
    int row0, n, tile0 = 0;
    bool group = false;                          // S: a group and its prefix
    Extent x;
    if constexpr (S) {
      const AttnRecord rec = P.plan.entry[b];
      group = b < P.group_entries;
      const int flags = group ? 0 : P.plan.flags[b - P.group_entries];
      row0 = uni(rec.row0);
      n = uni(rec.n);
      tile0 = uni(rec.tile0);
      x.slot = uni(flags ? -1 : rec.slot);
      x.len = uni(rec.len);
      x.first = uni(rec.first);
      x.blk0 = x.first / kUnitKeys;
      x.nblk = max(1, (x.len + kUnitKeys - 1) / kUnitKeys - x.blk0);
    } else {
      row0 = uni((int)rows[b]);
      n = uni((int)rows[b + 1]) - row0;
      x = seq_extent(P, b, n);
      x = Extent{uni(x.slot), uni(x.len), uni(x.first), uni(x.blk0), uni(x.nblk)};
    }
    const uint32_t rel = u - (uint32_t)uni((int)units[b]);
    const int seg = (int)(rel / (uint32_t)x.nblk), b0 = (int)(rel - (uint32_t)seg * x.nblk);
    const int b1 = (int)min((uint32_t)x.nblk, b0 + (u_end - u));
    const int mb = seg / P.kv_heads, head = seg - mb * P.kv_heads;
    if constexpr (S) {
      if (b0 == 0 && t == 0) P.plan.tile[tile0 + seg] = make_int2((int)w, (int)(range_of(u + (uint32_t)x.nblk - 1, W, U) - w) + 1);
    } else if (first_part && t == 0) {
      Part d;
      d.first_unit = b0 > 0 ? (int)(u - b0) : -1;
      d.end_unit = (int)(u - b0) + x.nblk;
      d.row0 = row0;
      d.n = n;
      d.head = head;
      d.mb = mb;
      d.U = U;
      d.W = W;
      desc[w] = d;
    }
    const int nrow = min(TM, n * P.group - mb * TM);   // rows of this tile
    // the rows of this lane's columns: their query, and the positions they see
    int last[MT], from[MT];
    int min_last = 0x7FFFFFFF, max_from = 0;
    {
      const int i0 = mb * TM / P.group, i1 = (mb * TM + nrow - 1) / P.group;
      min_last = S && group ? x.len - 1 : x.len - n + i0;
      max_from = S ? x.first : P.window > 0 ? max(0, x.len - n + i1 + 1 - P.window) : 0;
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int r = m * 16 + col;
      const bool in = r < nrow;
      const int rr = mb * TM + (in ? r : 0);
      const int i = rr / P.group, h = head * P.group + rr - i * P.group;
      last[m] = !in ? -1 : S && group ? x.len - 1 : x.len - n + i;
      from[m] = S ? x.first : P.window > 0 ? max(0, last[m] + 1 - P.window) : 0;
      // 16 bytes of a key are 8 numbers of one slice, or codes of two: 64 s' + 16 g .. + 15
      const uint16_t* qp = (const uint16_t*)P.q + (int64_t)(row0 + i) * P.q_row + (int64_t)h * P.q_head;
#pragma unroll
      for (int s = 0; s < NS; ++s)
        if ((m * NS + s) % kAtWaves == wv) qs[m][s][lane] = *(const u32x4*)(qp + (ES == 2 ? 32 * s + 8 * g : 64 * (s >> 1) + 8 * (s & 1) + 16 * g));
    }
    f32x4 o[MT][NJ];
    float mx[MT], ls[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      mx[m] = -INFINITY;
      ls[m] = 0.f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) o[m][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    bool bad = x.slot < 0;
    // read with scalar loads, whose counter is not the one the keys and values in flight are waited for with
    typedef const __attribute__((address_space(4))) int32_t* Names;
    const Names table = (Names)(uintptr_t)(P.table + (int64_t)max(x.slot, 0) * P.table_stride);
    const int pmask = (1 << P.page_log2) - 1;
    u32x4 kr[2][NL];
    uint32_t vr[8][VW];
    f32x4 ksc[2], vsc[2];                        // scales of the keys 4 g .. 4 g + 3 of both tiles
    const char *kb[2], *vb[2];
    const float *ksb[2], *vsb[2];
    // first key of block blk for this wave
    auto key0 = [&](int blk) { return (x.blk0 + blk) * kUnitKeys + wv * kTileKeys; };
    // The pages of the wave's two 16-key tiles (a tile lies in one page);
    // behind the last token the first tile's is used again, so that its reads
    // stay in bounds: they are masked.
    int id0 = 0, id1 = 0;
    auto names = [&](int pos) {
      id0 = table[pos >> P.page_log2];
      id1 = table[min(pos + 16, x.len - 1) >> P.page_log2];
    };
    // Base addresses; a page outside the pool is replaced by page 0, and noted
    // unless a window hides all of the tile (its pages may be gone by then).
    auto locate = [&](int pos) {
      const bool bad0 = (unsigned)id0 >= (unsigned)P.num_pages, bad1 = (unsigned)id1 >= (unsigned)P.num_pages;
      bad |= (bad0 && pos + 16 > x.first) || (bad1 && pos + 32 > x.first);
      id0 = bad0 ? 0 : id0;
      id1 = bad1 ? 0 : id1;
      const int off0 = pos & pmask, off1 = (pos + 16) & pmask;
      kb[0] = (const char*)P.k + ES * ((int64_t)id0 * P.k_page + (int64_t)head * P.k_head + (int64_t)off0 * P.k_tok);
      kb[1] = (const char*)P.k + ES * ((int64_t)id1 * P.k_page + (int64_t)head * P.k_head + (int64_t)off1 * P.k_tok);
      vb[0] = (const char*)P.v + ES * ((int64_t)id0 * P.v_page + (int64_t)head * P.v_head + (int64_t)off0 * P.v_tok);
      vb[1] = (const char*)P.v + ES * ((int64_t)id1 * P.v_page + (int64_t)head * P.v_head + (int64_t)off1 * P.v_tok);
      if constexpr (C != codes::kNone) {
        ksb[0] = P.ks + (int64_t)id0 * P.ks_page + (int64_t)head * P.ks_head + off0;
        ksb[1] = P.ks + (int64_t)id1 * P.ks_page + (int64_t)head * P.ks_head + off1;
        vsb[0] = P.vs + (int64_t)id0 * P.vs_page + (int64_t)head * P.vs_head + off0;
        vsb[1] = P.vs + (int64_t)id1 * P.vs_page + (int64_t)head * P.vs_head + off1;
      }
    };
    const uint32_t ko = ES == 2 ? 2u * ((uint32_t)col * (uint32_t)P.k_tok + 8u * g) : (uint32_t)col * (uint32_t)P.k_tok + 16u * g;
    auto load_k = [&]() {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int s = 0; s < NL; ++s) kr[h][s] = *(const u32x4*)(kb[h] + ko + 64 * s);
      if constexpr (C != codes::kNone) {
        ksc[0] = *(const f32x4*)(ksb[0] + 4 * g);
        ksc[1] = *(const f32x4*)(ksb[1] + 4 * g);
      }
    };
    auto load_v = [&]() {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const char* p = !kTight ? vb[e >> 2] + (uint32_t)ES * ((uint32_t)(4 * g + (e & 3)) * (uint32_t)P.v_tok + (uint32_t)NJ * col)
                                          : vb[e >> 2] + (e & 3) * (int64_t)P.v_tok + (4u * g * (uint32_t)P.v_tok + (uint32_t)NJ * col);
        if constexpr (VW == 1) {
          vr[e][0] = *(const uint32_t*)p;
        } else if constexpr (VW == 2) {
          const u32x2 a = *(const u32x2*)p;
          vr[e][0] = a[0];
          vr[e][1] = a[1];
        } else {
#pragma unroll
          for (int c = 0; c < VW / 4; ++c) {
            const u32x4 a = *(const u32x4*)(p + 16 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i) vr[e][4 * c + i] = a[i];
          }
        }
      }
      if constexpr (C != codes::kNone) {
        vsc[0] = *(const f32x4*)(vsb[0] + 4 * g);
        vsc[1] = *(const f32x4*)(vsb[1] + 4 * g);
      }
    };
    int pos = key0(b0);
    const int pos_end = min(x.len, key0(b1));
    if (pos < pos_end) {
      names(pos);
      locate(pos);
      load_k();
      load_v();
    }
    __syncthreads();                             // the queries are in place
    for (; pos < pos_end; pos += kUnitKeys) {
      const bool more = pos + kUnitKeys < pos_end;
      if (more) names(pos + kUnitKeys);
      f32x4 sc[MT][2];
      f32x4 kf[2];                               // what a score is multiplied by
      if constexpr (C == codes::kNone) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
          if (m == 0 || m * 16 < nrow) {         // a short sequence leaves the higher tiles out
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              sc[m][h] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int s = 0; s < NS; ++s) sc[m][h] = mfma<BF>(kr[h][s], qs[m][s][lane], sc[m][h]);
            }
          }
      } else {
        // Else the codes are unpacked where they were loaded, which waits for them there.
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int s = 0; s < NL; ++s) asm volatile("" : "+v"(kr[h][s]));
#pragma unroll
        for (int m = 0; m < MT; ++m) sc[m][0] = sc[m][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            const u32x4 a = widen8<BF, C>(kr[h][s >> 1][2 * (s & 1)], kr[h][s >> 1][2 * (s & 1) + 1]);
#pragma unroll
            for (int m = 0; m < MT; ++m) sc[m][h] = mfma<BF>(a, qs[m][s][lane], sc[m][h]);
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) kf[h][r] = ksc[h][r] * P.scale_log2;
          if (kTight) __builtin_amdgcn_sched_barrier(0);
        }
      }
      if (more) {
        locate(pos + kUnitKeys);
        load_k();
      }
      const bool masked = pos + kTileKeys - 1 > min_last || pos < max_from;   // some row does not see some key
      // what the mask hides of V must not be multiplied: 0 * NaN is NaN
      bool strange = false;
      // ones where a row of tile m sees the key, as the second product's right operand
      auto seen = [&](int m) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int kp = pos + 16 * (i >> 1) + 4 * g + 2 * (i & 1);
          w[i] = (kp <= last[m] && kp >= from[m] ? kOne<true> : 0u) | (kp < last[m] && kp + 1 >= from[m] ? kOne<true> << 16 : 0u);
        }
        return w;
      };
      if (masked) {
        float all = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int kp = pos + 16 * (e >> 2) + 4 * g + (e & 3);
          const bool gone = kp >= x.len;
#pragma unroll
          for (int i = 0; i < VW; ++i) {
            vr[e][i] = gone ? 0u : vr[e][i];
            if constexpr (C == codes::kNone) strange |= not_finite<BF>(vr[e][i]) || not_finite<BF>(vr[e][i] >> 16);
            else if constexpr (C == codes::kE4m3) strange |= nan_codes(vr[e][i]) != 0;
          }
          if constexpr (C != codes::kNone) all = fmaf(vsc[e >> 2][e & 3], 0.f, all);
        }
        strange = __ballot(strange) != 0;
        if (C != codes::kNone && __ballot(all != 0.f)) {
          // A value's scale that is not finite: a product of ones there with ones where a
          // row sees the key finds the rows that do, which become NaN; the value becomes 0.
          u32x4 marks = {0u, 0u, 0u, 0u};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int kp = pos + 16 * (e >> 2) + 4 * g + (e & 3);
            const bool odd = (__float_as_uint(vsc[e >> 2][e & 3]) & 0x7F800000u) == 0x7F800000u;
            vsc[e >> 2][e & 3] = odd ? 0.f : vsc[e >> 2][e & 3];
            marks[e >> 1] |= odd && kp < x.len ? kOne<true> << (16 * (e & 1)) : 0u;
          }
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const f32x4 d = mfma<true>(marks, seen(m), f32x4{0.f, 0.f, 0.f, 0.f});
            const float add = d[0] != 0.f ? __builtin_nanf("") : 0.f;     // the same in all of d
#pragma unroll
            for (int j = 0; j < NJ; ++j) o[m][j] += add;
          }
        }
      }
      u32x4 ph[MT], pl[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (m > 0 && m * 16 >= nrow) {
          if constexpr (C != codes::kNone) ph[m] = pl[m] = u32x4{0u, 0u, 0u, 0u};
          continue;
        }
        float s[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = sc[m][e >> 2][e & 3] * (C == codes::kNone ? P.scale_log2 : kf[e >> 2][e & 3]);
        if (masked) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int kp = pos + 16 * (e >> 2) + 4 * g + (e & 3);
            s[e] = kp <= last[m] && kp >= from[m] ? s[e] : -INFINITY;
          }
        }
        float top = s[0];
#pragma unroll
        for (int e = 1; e < 8; ++e) top = fmaxf(top, s[e]);
        if (__ballot(top > mx[m])) {             // a new maximum in some row: rescale
          const float nm = fmaxf(mx[m], column_max(top));
          const float f = mx[m] == nm ? 1.f : at_exp2(reference<PB>(mx[m]) - reference<PB>(nm));
          mx[m] = nm;
          ls[m] *= f;
#pragma unroll
          for (int j = 0; j < NJ; ++j) o[m][j] *= f;
        }
        const float ref = mx[m] == -INFINITY ? 0.f : reference<PB>(mx[m]);
        float p[8], eight;                       // summed up first: next to ls the weights of a long tail are below half a step
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          p[e] = at_exp2(s[e] - ref);
          eight = e ? eight + p[e] : p[e];
        }
        ls[m] += eight;
        if constexpr (C != codes::kNone) {
#pragma unroll
          for (int e = 0; e < 8; ++e) p[e] *= vsc[e >> 2][e & 3];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ph[m][i] = pack16<PB>(p[2 * i], p[2 * i + 1]);
          pl[m][i] = pack16<PB>(p[2 * i] - lo16<PB>(ph[m][i]), p[2 * i + 1] - hi16<PB>(ph[m][i]));
        }
        if (kTight) __builtin_amdgcn_sched_barrier(0);
      }
      // The schedule that the compiler takes without this holds up to 16
      // registers more: two float16 tiles of 128 spilled two (134 us, 133 with it).
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (C == codes::kNone) {
        if (strange) {
          // A value that is not finite next to a key that some row does not
          // see.  Where it stands, a third product with ones in such places
          // finds the rows that do see one; they become NaN, and the value 0.
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            u32x4 a;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t w = __builtin_amdgcn_perm(vr[2 * i + 1][j >> 1], vr[2 * i][j >> 1], (j & 1) ? 0x07060302u : 0x05040100u);
              a[i] = (not_finite<BF>(w) ? kOne<BF> : 0u) | (not_finite<BF>(w >> 16) ? kOne<BF> << 16 : 0u);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              if (m > 0 && m * 16 >= nrow) continue;
              f32x4 d = mfma<BF>(a, ph[m], f32x4{0.f, 0.f, 0.f, 0.f});
              d = mfma<BF>(a, pl[m], d);
#pragma unroll
              for (int r = 0; r < 4; ++r) o[m][j][r] += d[r] > 0.f ? __builtin_nanf("") : 0.f;
            }
          }
#pragma unroll
          for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int i = 0; i < VW; ++i)
              vr[e][i] &= (not_finite<BF>(vr[e][i]) ? 0u : 0xFFFFu) | (not_finite<BF>(vr[e][i] >> 16) ? 0u : 0xFFFF0000u);
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          u32x4 a;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            a[i] = __builtin_amdgcn_perm(vr[2 * i + 1][j >> 1], vr[2 * i][j >> 1], (j & 1) ? 0x07060302u : 0x05040100u);
#pragma unroll
          for (int m = 0; m < MT; ++m)
            if (m == 0 || m * 16 < nrow) {
              o[m][j] = mfma<BF>(a, ph[m], o[m][j]);
              o[m][j] = mfma<BF>(a, pl[m], o[m][j]);
            }
        }
      } else {
        if (C == codes::kE4m3 && strange) {
          // As above, with codes that are no numbers, and all rows that see them, whatever the weight.
          u32x4 sees[MT];
#pragma unroll
          for (int m = 0; m < MT; ++m) sees[m] = seen(m);
#pragma unroll
          for (int c = 0; c < VW; ++c) {
            uint32_t w[8];
            u32x4 a[4];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              w[e] = nan_codes(vr[e][c]) >> 7;
              vr[e][c] &= ~(w[e] * 0xFFu);
              w[e] *= 0x38u;                     // 1 in such places
            }
            turn_codes<C>(w, a);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int m = 0; m < MT; ++m) {
                const f32x4 d = mfma<true>(a[i], sees[m], f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                for (int r = 0; r < 4; ++r) o[m][4 * c + i][r] += d[r] != 0.f ? __builtin_nanf("") : 0.f;
              }
          }
        }
#pragma unroll
        for (int c = 0; c < VW; ++c) {
          uint32_t w[8];
          u32x4 a[4];
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = vr[e][c];
          turn_codes<C>(w, a);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              o[m][4 * c + i] = mfma<true>(a[i], ph[m], o[m][4 * c + i]);
              o[m][4 * c + i] = mfma<true>(a[i], pl[m], o[m][4 * c + i]);
            }
        }
      }
      if (more) load_v();
    }
    // The waves' parts of the tile become one: a lane brings its O to the
    // rows' common maximum (and divides by the sum, where this block has the
    // whole tile), 64 values of 16 rows at a time go through shared memory,
    // and a thread adds up 4 neighbours of a row.
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      mx[m] = reference<PB>(mx[m]);              // from here on all parts are compared by what they were taken against
      ls[m] = column_sum(ls[m]);
      if (bad) ls[m] = __builtin_nanf("");
      if (g == 0) {
        ml[wv][0][m * 16 + col] = mx[m];
        ml[wv][1][m * 16 + col] = ls[m];
      }
    }
    __syncthreads();
    const bool whole = b0 == 0 && b1 == x.nblk;
    float* part = part_at(P.parts, (int)w, b0 > 0 ? 0 : 1, TM, D);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (m * 16 >= nrow) break;
      const int r = m * 16 + col;
      float M = ml[0][0][r], L = 0.f;
#pragma unroll
      for (int i = 1; i < kAtWaves; ++i) M = fmaxf(M, ml[i][0][r]);
#pragma unroll
      for (int i = 0; i < kAtWaves; ++i) L += ml[i][1][r] * (ml[i][0][r] == M ? 1.f : at_exp2(ml[i][0][r] - M));
      float f = mx[m] == M ? 1.f : at_exp2(mx[m] - M);
      if (whole) f = L == 0.f ? 0.f : f / L;
      if (wv == 0 && g == 0 && r < nrow) {
        if (!whole) {
          part[TM * D + r] = M;
          part[TM * D + TM + r] = L;
        } else if (S) {
          P.state_m[(group ? 0 : (int64_t)P.total_rows * P.heads) + state_row(P, row0, head, mb * TM + r)] = L == 0.f ? -INFINITY : M + log2f(L);
        } else if (P.lse) {
          const int R = mb * TM + r, ri = R / P.group;
          P.lse[(int64_t)(row0 + ri) * P.heads + head * P.group + R - ri * P.group] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
        }
      }
#pragma unroll
      for (int r0 = 0; r0 < 4; r0 += RS) {
#pragma unroll
        for (int rr = 0; rr < RS; ++rr)
#pragma unroll
          for (int j = 0; j < NJ; j += 4) {
            f32x4 v;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = o[m][j + i][r0 + rr] * f;
            *(f32x4*)&ob[wv][col][(g * RS + rr) * NJ + j] = v;
          }
        __syncthreads();
        {
          const int qr = t >> 4, c = (t & 15) * 4;
          const int row = m * 16 + qr;
          f32x4 v = *(const f32x4*)&ob[0][qr][c];
#pragma unroll
          for (int i = 1; i < kAtWaves; ++i) {
            const f32x4 y = *(const f32x4*)&ob[i][qr][c];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] += y[k];
          }
          if (row < nrow) {
            const int gr = c / NJ;               // g RS + rr
            const int d = NJ * (4 * (gr / RS) + r0 + gr % RS) + c % NJ;
            if constexpr (S) {
              // by fours of the head dimension, then rows: k_attention_merge takes neighbouring rows side by side
              const int64_t total = (int64_t)P.total_rows * P.heads;
              float* to = whole ? P.state_o + ((group ? 0 : total * (D / 4)) + state_row(P, row0, head, mb * TM + row)) * 4 : part + row * 4;
              *(f32x4*)(to + (int64_t)(d / 4) * 4 * (whole ? total : TM)) = v;
            } else if (whole) {
              const int R = mb * TM + row, ri = R / P.group;
              const int64_t at = (int64_t)(row0 + ri) * P.heads + head * P.group + R - ri * P.group;
              *(u32x2*)((uint16_t*)P.out + at * D + d) = u32x2{pack16<BF>(v[0], v[1]), pack16<BF>(v[2], v[3])};
            } else {
              *(f32x4*)(part + row * D + d) = v;
            }
          }
        }
        __syncthreads();
      }
    }
    first_part = false;
    u += (uint32_t)(b1 - b0);
  }
}

namespace {

template <bool BF, int D, int MT, int C, bool S>
hipError_t launch_one(const AttnParams& p, int W, hipStream_t st) {
  const size_t lds = S ? (size_t)(p.entries + 1) * 4 : (size_t)(p.B + 1) * 8;
  hipLaunchKernelGGL((k_attention<BF, D, MT, C, S>), dim3((unsigned)W), dim3(kAtThreads), lds, st, p);
  hipError_t e = hipGetLastError();
  if (S || e != hipSuccess) return e;
  return launch_attention_join(p, 16 * MT, W, st);
}

template <bool BF, int C, bool S>
hipError_t launch_type(const AttnParams& p, int mt, int W, hipStream_t st) {
  switch (p.head_dim * 8 + mt) {
    case 64 * 8 + 1: return launch_one<BF, 64, 1, C, S>(p, W, st);
    case 64 * 8 + 2: return launch_one<BF, 64, 2, C, S>(p, W, st);
    case 64 * 8 + 4: return launch_one<BF, 64, 4, C, S>(p, W, st);
    case 128 * 8 + 1: return launch_one<BF, 128, 1, C, S>(p, W, st);
    case 128 * 8 + 2: return launch_one<BF, 128, 2, C, S>(p, W, st);
    case 128 * 8 + 3: return launch_one<BF, 128, 3, C, S>(p, W, st);
    case 256 * 8 + 1: return launch_one<BF, 256, 1, C, S>(p, W, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace

}  // namespace sv
