// Norms of queries and keys for each head with the position rotation in the
// same pass, writing the cache (16-bit values or 8-bit codes) as it goes, and
// reading the cache back, for gfx950.
//
// For a head's vector x of a token at position p:
//   y = x / sqrt(mean(x^2) + eps) * w            (or y = x)
//   pair i < rotary / 2:  (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = p f_i
// where pair i is (y_i, y_{i + rotary/2}), or (y_2i, y_2i+1).  Sums and products
// in float32, rounded once.  The angle is taken in turns, p (f_i / 2 pi), in
// float64: at position 10^6 a float32 product would be off by 0.06 radians.  Its
// fraction goes to the hardware's sine and cosine, which take turns (1.3e-7 off
// at most over [0, 1), measured at 2^20 points).
//
// Bound by the rows' bytes, or by latency for a round's few rows.  A lane holds 8
// numbers and their 8 partners (16 neighbours where pairs are neighbours), so
// that a pair never crosses lanes and loads are 16 bytes; a head is 4 to 32
// lanes, whose sum or maximum is a few lane moves.  A wave takes one token's
// heads, so that a lane's 8 angles serve all of them.
//
// Measured on one MI355X (rocprofv3): 9101 prompt rows of 32 + 8 + 8 heads of 128
// into a 16-bit cache 43 us (224 MB, 5.2 TB/s); a round's 138 rows 5 us, a chain of
// loads, sines and stores.  As int8 codes a layer's 6905 rows are written in 12.5 us
// and read back in 13 (43 MB each, 3.3 TB/s; more blocks, or 32-bit divisions, changed
// nothing); a round's in 3.7 and 5.

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

constexpr int kRoThreads = 256;
constexpr int kRoWaves = kRoThreads / kWave;

// sum and maximum over the LPH neighbouring lanes of a head, in each of them
template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
  v += dpp_f<kDppQuadXor1>(0.f, v);
  v += dpp_f<kDppQuadXor2>(0.f, v);
  if constexpr (LPH >= 8) v += dpp_f<kDppRowHalfMirror>(0.f, v);
  if constexpr (LPH >= 16) v += dpp_f<kDppRowMirror>(0.f, v);
  if constexpr (LPH >= 32) v += __shfl_xor(v, 16);
  return v;
}
template <int LPH>
__device__ __forceinline__ uint32_t head_max(uint32_t v) {
  v = max(v, (uint32_t)dpp_i<kDppQuadXor1>(0, (int)v));
  v = max(v, (uint32_t)dpp_i<kDppQuadXor2>(0, (int)v));
  if constexpr (LPH >= 8) v = max(v, (uint32_t)dpp_i<kDppRowHalfMirror>(0, (int)v));
  if constexpr (LPH >= 16) v = max(v, (uint32_t)dpp_i<kDppRowMirror>(0, (int)v));
  if constexpr (LPH >= 32) v = max(v, (uint32_t)__shfl_xor((int)v, 16));
  return v;
}

template <bool BF>
__device__ __forceinline__ void unpack8(u32x4 w, float* x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      x[2 * i] = (float)__builtin_bit_cast(_Float16, (uint16_t)w[i]);
      x[2 * i + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i] >> 16));
    }
  }
}
template <bool BF>
__device__ __forceinline__ u32x4 pack8(const float* x) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF) {
      typedef __bf16 b2 __attribute__((ext_vector_type(2)));
      const b2 v = {(__bf16)x[2 * i], (__bf16)x[2 * i + 1]};
      w[i] = __builtin_bit_cast(uint32_t, v);
    } else {
      typedef _Float16 h2 __attribute__((ext_vector_type(2)));
      const h2 v = {(_Float16)x[2 * i], (_Float16)x[2 * i + 1]};
      w[i] = __builtin_bit_cast(uint32_t, v);
    }
  }
  return w;
}

template <bool BF>
__device__ __forceinline__ void load_weight(const void* w, int f32, int at, float* x) {
  if (f32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = ((const float*)w)[at + i];
  } else {
    unpack8<BF>(*(const u32x4*)((const uint16_t*)w + at), x);
  }
}

}  // namespace

// Wave (row, part): heads part * per * (64 / LPH) .. of the row's queries, keys and values.
template <bool BF, int LPH, int C>
__global__ void __launch_bounds__(kRoThreads) k_rope(RopeParams P) {
  constexpr int HPW = kWave / LPH;               // heads side by side
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t wid = (int64_t)blockIdx.x * kRoWaves + threadIdx.x / kWave;
  const int64_t row = wid / P.parts;
  if (row >= P.rows) return;
  const int part = (int)(wid - row * P.parts);
  const int c = lane % LPH;
  const bool in = c * 16 < P.D;
  const int half = P.R >> 1;
  const bool turn = c * 16 < P.R;                // this lane's numbers are rotated
  int at0, at1;                                  // where they begin
  if (P.neighbours || !turn) {
    at0 = 16 * c;
    at1 = at0 + 8;
  } else {
    at0 = 8 * c;
    at1 = at0 + half;
  }
  const int pos = P.positions ? P.positions[row] : 0;
  const int64_t place = P.slots ? P.slots[row] : -1;
  const bool stored = place >= 0 && place < P.places && pos >= 0;
  float cs[8], sn[8];
  if (turn && in) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double t = (double)pos * (P.inv_freq[8 * c + i] * 0.15915494309189533577);
      const float f = (float)(t - floor(t));
      cs[i] = __builtin_amdgcn_cosf(f);
      sn[i] = __builtin_amdgcn_sinf(f);
    }
  }
  const int heads = P.H + P.KV + P.NV;
  const int h_end = min(heads, (part + 1) * P.per * HPW);
  for (int h0 = part * P.per * HPW; h0 < h_end; h0 += HPW) {
    const int hh = h0 + lane / LPH;
    if (hh >= heads) continue;                   // whole heads: the lane moves below stay inside one
    const int kind = hh < P.H ? 0 : hh < P.H + P.KV ? 1 : 2;
    const int h = kind == 0 ? hh : kind == 1 ? hh - P.H : hh - P.H - P.KV;
    const uint16_t* src = (const uint16_t*)(kind == 0 ? P.q : kind == 1 ? P.k : P.v) +
                          row * (kind == 0 ? P.q_row : kind == 1 ? P.k_row : P.v_row) +
                          h * (kind == 0 ? P.q_head : kind == 1 ? P.k_head : P.v_head);
    float x[16];
    if (in) {
      unpack8<BF>(*(const u32x4*)(src + at0), x);
      unpack8<BF>(*(const u32x4*)(src + at1), x + 8);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = 0.f;
    }
    if (kind < 2) {
      const void* w = kind == 0 ? P.q_weight : P.k_weight;
      if (w) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
        const float r = 1.f / sqrtf(head_sum<LPH>(ss) * P.inv_dim + P.eps);
        float g[16];
        if (in) {
          load_weight<BF>(w, P.weight_f32, at0, g);
          load_weight<BF>(w, P.weight_f32, at1, g + 8);
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = x[i] * r * g[i];
        }
      }
      if (turn && in) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int ia = P.neighbours ? 2 * i : i, ib = P.neighbours ? 2 * i + 1 : i + 8;
          const float a = x[ia], b = x[ib];
          x[ia] = a * cs[i] - b * sn[i];
          x[ib] = b * cs[i] + a * sn[i];
        }
      }
    }
    if (kind == 0 || (kind == 1 && P.k_out)) {
      if (pos < 0) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = __builtin_nanf("");
      }
      if (in) {
        uint16_t* dst = (uint16_t*)(kind == 0 ? P.q_out : P.k_out) + (row * (kind == 0 ? P.H : P.KV) + h) * P.D;
        *(u32x4*)(dst + at0) = pack8<BF>(x);
        *(u32x4*)(dst + at1) = pack8<BF>(x + 8);
      }
      continue;
    }
    // into the cache
    uint32_t top = 0;
    if constexpr (C != codes::kNone) {
#pragma unroll
      for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
      top = head_max<LPH>(top);
    }
    if (!stored || !in) continue;
    const int64_t page = place >> P.page_log2;
    const int off = (int)(place & ((1 << P.page_log2) - 1));
    const int64_t vec = ((page * P.KV + h) << P.page_log2) + off;      // the vector's number in the layer
    if constexpr (C == codes::kNone) {
      uint16_t* dst = (uint16_t*)(kind == 1 ? P.ck : P.cv) + vec * P.D;
      *(u32x4*)(dst + at0) = pack8<BF>(x);
      *(u32x4*)(dst + at1) = pack8<BF>(x + 8);
    } else {
      float scale, inv;
      codes::scale_of<C>(top, &scale, &inv);
      uint8_t* dst = (uint8_t*)(kind == 1 ? P.ck : P.cv) + vec * P.D;
      *(u32x2*)(dst + at0) = u32x2{codes::pack4<C>(x[0], x[1], x[2], x[3], inv), codes::pack4<C>(x[4], x[5], x[6], x[7], inv)};
      *(u32x2*)(dst + at1) = u32x2{codes::pack4<C>(x[8], x[9], x[10], x[11], inv), codes::pack4<C>(x[12], x[13], x[14], x[15], inv)};
      if (c == 0) (kind == 1 ? P.ks : P.vs)[vec] = scale;
    }
  }
}

namespace {

// What entry b of a read asks for: its slot and first position, or why it is refused.
struct ReadEntry {
  int slot, first, status;
};
__device__ __forceinline__ ReadEntry read_entry(const CacheReadParams& P, int b) {
  ReadEntry e;
  e.slot = P.seqs ? P.seqs[b] : b;
  e.first = P.first[b];
  e.status = 0;
  const int n = P.count[b];
  if ((unsigned)e.slot >= (unsigned)P.slots) {
    e.status = SV_ST_BAD_SEQ;
  } else {
    const int len = P.seq_len[e.slot];
    if (len < 0 || len > P.max_len || e.first < 0 || n < 0 || (int64_t)e.first + n > len) e.status = SV_ST_BAD_LENGTH;
  }
  return e;
}

}  // namespace

// Rows of a layer's keys and values, out of the pages and back in 16 bits.
// Block i < work serves rows i, i + work, ... (kRoThreads / lanes of a row at a
// time); the others check an entry's pages for its status.
template <bool BF, int C>
__global__ void __launch_bounds__(kRoThreads) k_cache_read(CacheReadParams P) {
  extern __shared__ uint32_t ends[];             // inclusive prefix of the counts
  __shared__ uint32_t wave_total[kRoWaves];
  __shared__ int bad;
  const int t = threadIdx.x, lane = t & (kWave - 1), wv = t / kWave;
  if (t == 0) bad = 0;
  __syncthreads();
  {
    const int per = (P.B + kRoThreads - 1) / kRoThreads;
    const int b0 = min(t * per, P.B), b1 = min(b0 + per, P.B);
    uint32_t r = 0;
    for (int b = b0; b < b1; ++b) {
      const int n = P.count[b];
      if (n < 0 || n > P.total) bad = 1;
      else r += (uint32_t)n;
      ends[b] = r;
    }
    const uint32_t incl = wave_incl_scan_u32(r);
    if (lane == kWave - 1) wave_total[wv] = incl;
    __syncthreads();
    uint32_t before = incl - r;
    for (int i = 0; i < wv; ++i) before += wave_total[i];
    for (int b = b0; b < b1; ++b) ends[b] += before;
    if (t == kRoThreads - 1 && before + r != (uint32_t)P.total) bad = 1;
    __syncthreads();
  }
  const int layout = bad ? SV_ST_BAD_LAYOUT : 0;
  if ((int)blockIdx.x >= P.work) {
    const int b = (int)blockIdx.x - P.work;
    const ReadEntry e = read_entry(P, b);
    int s = layout ? layout : e.status;
    if (!s) {
      const int p1 = (int)(((int64_t)e.first + P.count[b] + P.page_size - 1) >> P.page_log2);
      for (int i = (e.first >> P.page_log2) + t; i < p1 && P.count[b] > 0; i += kRoThreads)
        if ((unsigned)P.table[(int64_t)e.slot * P.max_pages + i] >= (unsigned)P.num_pages) s = SV_ST_BAD_PAGE;
    }
    __syncthreads();
    if (s) atomicOr(&bad, s << 1);
    __syncthreads();
    if (t == 0) P.status[b] = bad >> 1;
    return;
  }
  const int64_t vecs = (int64_t)P.kv_heads * P.head_vecs;              // 8 numbers each
  const int64_t total = (int64_t)P.total * vecs;
  for (int64_t i = (int64_t)blockIdx.x * kRoThreads + t; i < total; i += (int64_t)P.work * kRoThreads) {
    const int64_t row = i / vecs;
    const int v = (int)(i - row * vecs), h = v / P.head_vecs, d = (v - h * P.head_vecs) * 8;
    bool ok = !layout;
    int64_t vec = 0;
    if (ok) {
      int lo = 0, hi = P.B - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (ends[mid] > (uint32_t)row) hi = mid;
        else lo = mid + 1;
      }
      const ReadEntry e = read_entry(P, lo);
      ok = e.status == 0;
      if (ok) {
        const int pos = e.first + (int)((uint32_t)row - (lo ? ends[lo - 1] : 0u));
        const int page = P.table[(int64_t)e.slot * P.max_pages + (pos >> P.page_log2)];
        ok = (unsigned)page < (unsigned)P.num_pages;
        vec = (((int64_t)page * P.kv_heads + h) << P.page_log2) + (pos & (P.page_size - 1));
      }
    }
    const int64_t to = (row * P.kv_heads + h) * P.D + d;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      u32x4 out = {BF ? 0x7FC07FC0u : 0x7E007E00u, BF ? 0x7FC07FC0u : 0x7E007E00u, BF ? 0x7FC07FC0u : 0x7E007E00u,
                   BF ? 0x7FC07FC0u : 0x7E007E00u};
      if (ok) {
        if constexpr (C == codes::kNone) {
          out = *(const u32x4*)((const uint16_t*)(w ? P.v : P.k) + vec * P.D + d);
        } else {
          const u32x2 a = *(const u32x2*)((const uint8_t*)(w ? P.v : P.k) + vec * P.D + d);
          const float s = (w ? P.vs : P.ks)[vec];
          float x[8];
          codes::unpack4<C>(a[0], x);
          codes::unpack4<C>(a[1], x + 4);
          constexpr float top = BF ? 0x1.FEp127f : 65504.f;            // a code may stand for more than the type's largest
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            x[k] *= s;
            x[k] = x[k] > top ? top : x[k] < -top ? -top : x[k];
          }
          out = pack8<BF>(x);
        }
      }
      *(u32x4*)((uint16_t*)(w ? P.v_out : P.k_out) + to) = out;
    }
  }
}

namespace {

template <bool BF, int LPH>
hipError_t launch_rope_lph(const RopeParams& p, int blocks, hipStream_t st) {
  switch (p.codes) {
    case codes::kNone: hipLaunchKernelGGL((k_rope<BF, LPH, codes::kNone>), dim3((unsigned)blocks), dim3(kRoThreads), 0, st, p); break;
    case codes::kE4m3: hipLaunchKernelGGL((k_rope<BF, LPH, codes::kE4m3>), dim3((unsigned)blocks), dim3(kRoThreads), 0, st, p); break;
    case codes::kInt8: hipLaunchKernelGGL((k_rope<BF, LPH, codes::kInt8>), dim3((unsigned)blocks), dim3(kRoThreads), 0, st, p); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

template <bool BF>
hipError_t launch_rope_type(const RopeParams& p, int lph, int blocks, hipStream_t st) {
  switch (lph) {
    case 4: return launch_rope_lph<BF, 4>(p, blocks, st);
    case 8: return launch_rope_lph<BF, 8>(p, blocks, st);
    case 16: return launch_rope_lph<BF, 16>(p, blocks, st);
    case 32: return launch_rope_lph<BF, 32>(p, blocks, st);
  }
  return hipErrorInvalidValue;
}

template <bool BF>
hipError_t launch_read_type(const CacheReadParams& p, hipStream_t st) {
  const dim3 grid((unsigned)(p.work + (p.status ? p.B : 0))), block(kRoThreads);
  const size_t lds = (size_t)p.B * 4;
  switch (p.codes) {
    case codes::kNone: hipLaunchKernelGGL((k_cache_read<BF, codes::kNone>), grid, block, lds, st, p); break;
    case codes::kE4m3: hipLaunchKernelGGL((k_cache_read<BF, codes::kE4m3>), grid, block, lds, st, p); break;
    case codes::kInt8: hipLaunchKernelGGL((k_cache_read<BF, codes::kInt8>), grid, block, lds, st, p); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(RopeParams p, hipStream_t st) {
  const int lph = p.D <= 64 ? 4 : p.D <= 128 ? 8 : p.D <= 256 ? 16 : 32, hpw = kWave / lph;
  const int head_blocks = (p.H + p.KV + p.NV + hpw - 1) / hpw;
  // Where there are more waves than the chip holds (8 on each of 1024 SIMDs), a
  // wave takes up to three blocks of heads, for which a lane's angles are the same;
  // fewer rows want the waves.  One, two, three, six blocks a wave, 48 heads of 128:
  // 9101 rows 48.8, 44.0, 43.4, 42.6 us, some 2400 17.8, 16.7, 16.4, 19.0, 300 8.0, 8.9,
  // 9.6, 12.4, 138 6.6, 7.7, 9.1, 12.0 (48 heads of 256 110.7, 100.8, 100.5, 102.5).
  p.parts = p.rows * head_blocks >= 8192 ? (head_blocks + 2) / 3 : head_blocks;
  p.per = (head_blocks + p.parts - 1) / p.parts;
  const int64_t blocks = (p.rows * p.parts + kRoWaves - 1) / kRoWaves;
  return p.bf16 ? launch_rope_type<true>(p, lph, (int)blocks, st) : launch_rope_type<false>(p, lph, (int)blocks, st);
}

hipError_t launch_cache_read(CacheReadParams p, hipStream_t st) {
  const int64_t blocks = ((int64_t)p.total * p.kv_heads * p.head_vecs + kRoThreads - 1) / kRoThreads;
  p.work = (int)(blocks < 2048 ? blocks : 2048);
  if (p.work + (p.status ? p.B : 0) == 0) return hipSuccess;
  return p.bf16 ? launch_read_type<true>(p, st) : launch_read_type<false>(p, st);
}

}  // namespace sv
