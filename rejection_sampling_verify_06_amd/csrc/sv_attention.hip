// Attention of a round's new tokens over a paged key-value cache, for gfx950.
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

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "sv_internal.h"
#include "sv_wave.h"

namespace sv {

namespace {

using namespace wave;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
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
__device__ __forceinline__ float* part_at(const AttnParams& P, int w, int slot, int TM, int D) {
  return P.parts + ((int64_t)w * 2 + slot) * TM * (D + 2);
}

}  // namespace

template <bool BF, int D, int MT>
__global__ void __launch_bounds__(kAtThreads, D * MT <= 64 ? 4 : D * MT <= 256 && D < 256 ? 2 : 1) k_attention(AttnParams P) {
  constexpr int TM = 16 * MT;                    // rows of a tile
  constexpr int NS = D / 32;                     // 32-element slices of the head dimension (scores)
  constexpr int NJ = D / 16;                     // 16-row tiles of O^T; also a lane's elements of a V row
  constexpr int VW = NJ / 2;                     // dwords of those
  extern __shared__ uint32_t dyn[];
  uint32_t* rows = dyn;
  uint32_t* units = dyn + P.B + 1;
  constexpr int RS = 256 / D;                    // of a lane's 4 rows of each O^T tile, those that are joined at a time
  __shared__ u32x4 qs[MT][NS][kWave];        // the tile's queries as the first product's right operands
  __shared__ float ml[kAtWaves][2][TM];
  __shared__ float ob[kAtWaves][16][64 + 4];     // 64 of the D values of 16 rows, rows 4 banks apart
  const int t = threadIdx.x, lane = t & (kWave - 1), wv = uni(t / kWave);
  const int g = lane >> 4, col = lane & 15;
  const bool ok = plan(P, TM, rows, units);
  Part* desc = reinterpret_cast<Part*>(P.desc);
  const uint32_t U = (uint32_t)uni((int)units[P.B]), W = min((uint32_t)gridDim.x, U);
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
    if (t == 0) desc[w].first_unit = -1;
    return;
  }
  uint32_t u = range_start(w, W, U);
  const uint32_t u_end = range_start(w + 1, W, U);
  // the sequence that holds unit u
  int b = 0;
  for (int step = 4096; step > 0; step >>= 1)
    if (b + step < P.B && (uint32_t)uni((int)units[b + step]) <= u) b += step;
  bool first_part = true;
  while (u < u_end) {
    while ((uint32_t)uni((int)units[b + 1]) <= u) ++b;
    const int row0 = uni((int)rows[b]), n = uni((int)rows[b + 1]) - row0;
    Extent x = seq_extent(P, b, n);
    x = Extent{uni(x.slot), uni(x.len), uni(x.first), uni(x.blk0), uni(x.nblk)};
    const uint32_t rel = u - (uint32_t)uni((int)units[b]);
    const int seg = (int)(rel / (uint32_t)x.nblk), b0 = (int)(rel - (uint32_t)seg * x.nblk);
    const int b1 = (int)min((uint32_t)x.nblk, b0 + (u_end - u));
    const int mb = seg / P.kv_heads, head = seg - mb * P.kv_heads;
    if (first_part && t == 0) {
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
      min_last = x.len - n + i0;
      max_from = P.window > 0 ? max(0, x.len - n + i1 + 1 - P.window) : 0;
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int r = m * 16 + col;
      const bool in = r < nrow;
      const int rr = mb * TM + (in ? r : 0);
      const int i = rr / P.group, h = head * P.group + rr - i * P.group;
      last[m] = in ? x.len - n + i : -1;
      from[m] = P.window > 0 ? max(0, last[m] + 1 - P.window) : 0;
      const uint16_t* qp = (const uint16_t*)P.q + (int64_t)(row0 + i) * P.q_row + (int64_t)h * P.q_head + 8 * g;
#pragma unroll
      for (int s = 0; s < NS; ++s)
        if ((m * NS + s) % kAtWaves == wv) qs[m][s][lane] = *(const u32x4*)(qp + 32 * s);
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
    u32x4 kr[2][NS];
    uint32_t vr[8][VW];
    const char *kb[2], *vb[2];
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
      kb[0] = (const char*)P.k + 2 * ((int64_t)id0 * P.k_page + (int64_t)head * P.k_head + (int64_t)off0 * P.k_tok);
      kb[1] = (const char*)P.k + 2 * ((int64_t)id1 * P.k_page + (int64_t)head * P.k_head + (int64_t)off1 * P.k_tok);
      vb[0] = (const char*)P.v + 2 * ((int64_t)id0 * P.v_page + (int64_t)head * P.v_head + (int64_t)off0 * P.v_tok);
      vb[1] = (const char*)P.v + 2 * ((int64_t)id1 * P.v_page + (int64_t)head * P.v_head + (int64_t)off1 * P.v_tok);
    };
    const uint32_t ko = 2u * ((uint32_t)col * (uint32_t)P.k_tok + 8u * g);
    auto load_k = [&]() {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int s = 0; s < NS; ++s) kr[h][s] = *(const u32x4*)(kb[h] + ko + 64 * s);
    };
    auto load_v = [&]() {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const char* p = vb[e >> 2] + 2u * ((uint32_t)(4 * g + (e & 3)) * (uint32_t)P.v_tok + (uint32_t)NJ * col);
        if constexpr (VW == 2) {
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
#pragma unroll
      for (int m = 0; m < MT; ++m)
        if (m == 0 || m * 16 < nrow) {           // a short sequence leaves the higher tiles out
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            sc[m][h] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < NS; ++s) sc[m][h] = mfma<BF>(kr[h][s], qs[m][s][lane], sc[m][h]);
          }
        }
      if (more) {
        locate(pos + kUnitKeys);
        load_k();
      }
      const bool masked = pos + kTileKeys - 1 > min_last || pos < max_from;   // some row does not see some key
      // what the mask hides of V must not be multiplied: 0 * NaN is NaN
      bool strange = false;
      if (masked) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int kp = pos + 16 * (e >> 2) + 4 * g + (e & 3);
          const bool gone = kp >= x.len;
#pragma unroll
          for (int i = 0; i < VW; ++i) {
            vr[e][i] = gone ? 0u : vr[e][i];
            strange |= not_finite<BF>(vr[e][i]) || not_finite<BF>(vr[e][i] >> 16);
          }
        }
        strange = __ballot(strange) != 0;
      }
      u32x4 ph[MT], pl[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (m > 0 && m * 16 >= nrow) continue;
        float s[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = sc[m][e >> 2][e & 3] * P.scale_log2;
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
          const float f = mx[m] == nm ? 1.f : at_exp2(reference<BF>(mx[m]) - reference<BF>(nm));
          mx[m] = nm;
          ls[m] *= f;
#pragma unroll
          for (int j = 0; j < NJ; ++j) o[m][j] *= f;
        }
        const float ref = mx[m] == -INFINITY ? 0.f : reference<BF>(mx[m]);
        float p[8], eight;                       // summed up first: next to ls the weights of a long tail are below half a step
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          p[e] = at_exp2(s[e] - ref);
          eight = e ? eight + p[e] : p[e];
        }
        ls[m] += eight;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ph[m][i] = pack16<BF>(p[2 * i], p[2 * i + 1]);
          pl[m][i] = pack16<BF>(p[2 * i] - lo16<BF>(ph[m][i]), p[2 * i + 1] - hi16<BF>(ph[m][i]));
        }
      }
      // The schedule that the compiler takes without this holds up to 16
      // registers more: two float16 tiles of 128 spilled two (134 us, 133 with it).
      __builtin_amdgcn_sched_barrier(0);
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
      if (more) load_v();
    }
    // The waves' parts of the tile become one: a lane brings its O to the
    // rows' common maximum (and divides by the sum, where this block has the
    // whole tile), 64 values of 16 rows at a time go through shared memory,
    // and a thread adds up 4 neighbours of a row.
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      mx[m] = reference<BF>(mx[m]);              // from here on all parts are compared by what they were taken against
      ls[m] = column_sum(ls[m]);
      if (bad) ls[m] = __builtin_nanf("");
      if (g == 0) {
        ml[wv][0][m * 16 + col] = mx[m];
        ml[wv][1][m * 16 + col] = ls[m];
      }
    }
    __syncthreads();
    const bool whole = b0 == 0 && b1 == x.nblk;
    float* part = part_at(P, (int)w, b0 > 0 ? 0 : 1, TM, D);
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
            if (whole) {
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

// Adds up the parts of each tile that was cut: block (w, y) serves the tile
// that block w of k_attention entered in its middle, if no earlier block did,
// and rows 4 y .. 4 y + 3 of it, a row to a wave.  Bound by latency: the
// record, then maxima, sums and the first parts' O at once, 8 parts of a
// lane's 16 bytes in flight.  Further blocks check the sequences' pages for
// `status`.
template <bool BF, int D>
__global__ void __launch_bounds__(kAtThreads) k_attention_join(AttnParams P, int TM, int W0) {
  __shared__ float wt[kAtWaves][kWave];
  const int t = threadIdx.x, lane = t & (kWave - 1), wv = t / kWave;
  if ((int)blockIdx.x >= W0) {
    if (blockIdx.y) return;
    // status of sequence b; block W0 checks the layout for all
    const int b = (int)blockIdx.x - W0;
    __shared__ int st;
    __shared__ unsigned long long sum;
    if (t == 0) {
      st = 0;
      sum = 0;
    }
    __syncthreads();
    unsigned long long r = 0;
    int f = 0;
    for (int i = t; i < P.B; i += kAtThreads) {
      const int K = P.num_draft[i];
      if (K < 0 || K >= P.total_rows) f = SV_ST_BAD_LAYOUT;
      else r += (unsigned)K + 1u;
    }
    if (f) atomicOr(&st, f);
    atomicAdd(&sum, r);
    __syncthreads();
    if (t == 0 && sum != (unsigned long long)P.total_rows) atomicOr(&st, SV_ST_BAD_LAYOUT);
    __syncthreads();
    if (st == 0) {
      const int n = P.num_draft[b] + 1;
      const int slot = P.seqs ? P.seqs[b] : b;
      int s = 0;
      if ((unsigned)slot >= (unsigned)P.slots) {
        s = SV_ST_BAD_SEQ;
      } else {
        const int len = P.seq_len[slot];
        if (len < 0 || len > P.max_len || !in_place(P, b, n, len)) {
          s = SV_ST_BAD_LENGTH;
        } else {
          const Extent x = seq_extent(P, b, n);
          const int p0 = x.first >> P.page_log2;
          const int p1 = (len + (1 << P.page_log2) - 1) >> P.page_log2;
          for (int i = p0 + t; i < p1; i += kAtThreads)
            if ((unsigned)P.table[(int64_t)slot * P.table_stride + i] >= (unsigned)P.num_pages) s = SV_ST_BAD_PAGE;
        }
      }
      __syncthreads();
      if (s) atomicOr(&st, s);
    }
    __syncthreads();
    if (t == 0) P.status[b] = st;
    return;
  }
  const Part d = reinterpret_cast<const Part*>(P.desc)[blockIdx.x];
  if (d.first_unit < 0) return;
  const uint32_t w = blockIdx.x;
  if (range_start(w - 1, d.W, d.U) > (uint32_t)d.first_unit) return;   // an earlier block joins this tile
  const int row = (int)blockIdx.y * kAtWaves + wv;
  const int nrow = min(TM, d.n * P.group - d.mb * TM);
  if (row >= nrow) return;                       // whole waves; no block barrier below
  const int parts = (int)(range_of((uint32_t)d.end_unit - 1, d.W, d.U) - w) + 2;
  // part 0: slot 1 of block w - 1; part i: slot 0 of block w - 1 + i
  auto part = [&](int i) { return (const float*)part_at(P, (int)w - 1 + i, i == 0 ? 1 : 0, TM, D); };
  constexpr int Q = D / 4;                       // lanes that cover a row with 4 floats each
  constexpr int GR = kWave / Q;                  // parts side by side: 4, 2 or 1
  const int pg = lane / Q, dq = (lane - pg * Q) * 4;
  f32x4 v[8];
  auto load_o = [&](int i) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = *(const f32x4*)(part(min(i + k * GR, parts - 1)) + row * D + dq);
  };
  const float* mine = part(min(lane, parts - 1)) + TM * D + row;
  const float m0 = mine[0], l0 = mine[TM];
  load_o(pg);
  float M = lane < parts ? m0 : -INFINITY;
  for (int i = lane + kWave; i < parts; i += kWave) M = fmaxf(M, part(i)[TM * D + row]);
  M = wave_max(M);
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  float L = 0.f;
  for (int i0 = 0; i0 < parts; i0 += kWave) {
    float f = 0.f;
    if (i0 + lane < parts) {
      const float* pp = part(i0 + lane) + TM * D + row;
      const float m = i0 ? pp[0] : m0, l = i0 ? pp[TM] : l0;
      f = m == M ? 1.f : at_exp2(m - M);
      L += l * f;
    }
    wt[wv][lane] = f;
    wave_sync();
    const int e = min(kWave, parts - i0);
    for (int i = pg; i < e; i += 8 * GR) {
      if (i0 + i != pg) load_o(i0 + i);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (i + k * GR < e) {
          const float f2 = wt[wv][i + k * GR];
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[c] = fmaf(v[k][c], f2, acc[c]);
        }
    }
    wave_sync();
  }
  L = wave_sum(L);
#pragma unroll
  for (int off = Q; off < kWave; off <<= 1)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c] += __shfl_xor(acc[c], off);
  const int R = d.mb * TM + row, ri = R / P.group, h = d.head * P.group + R - ri * P.group;
  const int64_t at = (int64_t)(d.row0 + ri) * P.heads + h;
  if (pg == 0) {
    uint16_t* op = (uint16_t*)P.out + at * D + dq;
    u32x2 z;
    z[0] = L == 0.f ? 0u : pack16<BF>(acc[0] / L, acc[1] / L);
    z[1] = L == 0.f ? 0u : pack16<BF>(acc[2] / L, acc[3] / L);
    *(u32x2*)op = z;
  }
  if (P.lse && lane == 0) P.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

namespace {

template <bool BF, int D, int MT>
hipError_t launch_one(const AttnParams& p, int W, hipStream_t st) {
  const size_t lds = (size_t)(p.B + 1) * 8;
  hipLaunchKernelGGL((k_attention<BF, D, MT>), dim3((unsigned)W), dim3(kAtThreads), lds, st, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_attention_join<BF, D>), dim3((unsigned)(W + (p.status ? p.B : 0)), 16 * MT / kAtWaves),
                     dim3(kAtThreads), 0, st, p, 16 * MT, W);
  return hipGetLastError();
}

template <bool BF>
hipError_t launch_type(const AttnParams& p, int mt, int W, hipStream_t st) {
  switch (p.head_dim * 8 + mt) {
    case 64 * 8 + 1: return launch_one<BF, 64, 1>(p, W, st);
    case 64 * 8 + 2: return launch_one<BF, 64, 2>(p, W, st);
    case 64 * 8 + 4: return launch_one<BF, 64, 4>(p, W, st);
    case 128 * 8 + 1: return launch_one<BF, 128, 1>(p, W, st);
    case 128 * 8 + 2: return launch_one<BF, 128, 2>(p, W, st);
    case 128 * 8 + 3: return launch_one<BF, 128, 3>(p, W, st);
    case 256 * 8 + 1: return launch_one<BF, 256, 1>(p, W, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_attention(const AttnParams& p, int row_tiles, int blocks, hipStream_t st) {
  return p.bf16 ? launch_type<true>(p, row_tiles, blocks, st) : launch_type<false>(p, row_tiles, blocks, st);
}

}  // namespace sv
