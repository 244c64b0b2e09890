// Attention of many rows over a shared prefix, for gfx950 (internal;
// instantiated by sv_attention_shared*.hip).
//
// A group's rows (those of all its sequences, for one key head) all see the
// whole prefix.  From about 50 rows on the products bound, not the bytes: a
// block takes 32 rows a wave, stages 64 keys at a time in shared memory for all
// of its waves (codes widened on the way, once for all rows) and forms
//   S^T = K Q^T   (keys x rows)     O^T += V^T P^T   (head dim x rows)
// with 32x32x16 MFMAs.  As in k_attention a lane holds the scores of one row
// (column lane & 31): keys 8 q + 4 h + r, h = lane >> 5, in register 4 q + r,
// and these are the second product's right operand if slot (h, e) of 16 keys is
// key 8 (e >> 2) + 4 h + (e & 3).  V^T under that numbering is two transposing
// reads of four keys each; softmax needs one exchange between lanes.
//
// Keys lie in shared memory as in the pages, 16-byte pieces permuted within a
// row so that the reads of 16 neighbouring keys (K), and of 64 bytes of four
// keys (V, transposed), fall on different banks.  The next 64 keys are in
// flight while these are worked on, 16-bit ones straight to the other half of
// shared memory, codes to registers.  Reads, products and the arithmetic of the
// weights are in a fixed order (257 us with registers and the compiler's own, 206).
//
// Weights are split in two 16-bit halves and units dealt out in equal ranges,
// for the same reasons as in k_attention; k_attention_merge adds the parts up.
//
// Bound by the matrix pipes and, beside them, the issue of 308 vector instructions
// a step.  Measured on one MI355X (rocprofv3): 64 sequences of up to 6 rows behind 32768
// tokens, 8 key heads of 128, 186 us after a hundred calls, 212 among the first twenty: 0.7
// PFLOP/s of the formula's products, 1.05 with the split's second one (a library product
// of 8192^3 reaches 1.2); among the first twenty one 16-bit weight instead of two took
// 178, a ring of four tiles of 32 keys 218.  8 groups of 8 behind 8000 tokens over e4m3
// 46 us.  Over codes heads of 256 have 22 registers too many (44 bytes a lane in
// scratch), heads of 128 two (12 bytes).

#pragma once

#include "sv_attention_kernel.h"

namespace sv {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* TrPtr;

template <bool BF>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// maximum and sum over the two lanes that share a column (l, l ^ 32)
__device__ __forceinline__ float pair_max(float v) {
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float pair_sum(float v) {
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Piece c of key r lies at c ^ k_turn(r) among the row's 16-byte pieces, and of a value at c ^ v_turn(r).
template <int D>
__device__ __forceinline__ int k_turn(int r) {
  return D == 64 ? (r >> 1) & 7 : r & 15;
}
template <int D>
__device__ __forceinline__ int v_turn(int r) {
  return D == 64 ? ((r >> 1) & 1) << 2 : (r & 3) << 2;
}

// 16 bytes a lane from memory to the wave's 1 KB of shared memory at `to`; there behind the next barrier
__device__ __forceinline__ void load_lds(const char* base, uint32_t offset, u32x4* to) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(base + offset), (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}

// two floats as the sum of two pairs of 16-bit numbers
template <bool BF>
__device__ __forceinline__ void split16(float a, float b, uint32_t* hi, uint32_t* lo) {
  uint32_t x = pack16<BF>(a, b);
  asm("" : "+v"(x));                             // or the compiler rounds a once more for its own half
  *hi = x;
  *lo = pack16<BF>(a - lo16<BF>(x), b - hi16<BF>(x));
}

}  // namespace

constexpr int kPfWaves = 4;
constexpr int kPfThreads = kPfWaves * 64;
constexpr int kPfRows = 32 * kPfWaves;
static_assert(kPfRows == kAttnPrefixRows, "rows of a tile");

template <int D>
constexpr int kPfKeys = D == 256 ? 32 : 64;      // keys staged at a time

template <bool BF, int D, int C>
__global__ void __launch_bounds__(kPfThreads, D == 256 ? 1 : 2) k_prefix(AttnParams P) {
  constexpr bool PB = BF || C != codes::kNone;   // the second product's type
  // Weights need not stay below 1: two bfloat16 hold 2^8 as well as 1, float16
  // (weights against the maximum less 14) ends at 2^16.  Without it 32 rows find a
  // new maximum in some two of three steps.
  constexpr float kSlack = PB ? 8.f : 1.f;
  constexpr int ES = C != codes::kNone ? 1 : 2;
  constexpr int KT = kPfKeys<D>;
  constexpr int TM = kPfRows;
  constexpr int NS = D / 16;                     // 16-number slices of the head dimension (scores)
  constexpr int NJ = D / 32;                     // 32-row tiles of O^T
  constexpr int NT = KT / 32;                    // 32-key tiles
  constexpr int CPR = D * ES / 16;               // 16-byte pieces of a cached key
  constexpr int NI = KT * CPR / kPfThreads;      // pieces of K (and of V) that a thread brings
  static_assert(KT * CPR % kPfThreads == 0 && kUnitKeys % KT == 0, "pieces");
  extern __shared__ uint32_t dyn[];
  uint32_t* units = dyn;
  __shared__ u32x4 ksh[2][KT * D / 8], vsh[2][KT * D / 8];
  __shared__ float kscale[2][KT], vscale[2][KT];
  const int t = threadIdx.x, lane = t & (kWave - 1), wv = uni(t / kWave);
  const int h = lane >> 5, col = lane & 31;
  // Where a lane reads: piece 2 i + h of key col, at 32 i ^ this; and of four
  // values the 16 numbers around its own, 4 (lane & 3) .. + 3 of 16 ((lane >> 4)
  // & 1) .. + 15 of key 4 h + ((lane >> 2) & 3), at 64 j ^ this for number 32 j on.
  const int vkey = 4 * h + ((lane >> 2) & 3), vd = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
  const char* kbase = (const char*)&ksh[0][0] + col * (2 * D);
  char* vbase = (char*)&vsh[0][0] + vkey * (2 * D);
  const int koff = 16 * (h ^ k_turn<D>(col)), voff = (16 * ((vd >> 3) ^ v_turn<D>(vkey))) | (2 * (vd & 7));
  // A wave brings (part of) 16 keys, which lie in one page: what a lane's pieces
  // add to the place of the first, and where they begin among the staged ones.
  constexpr int GW = kPfWaves / (KT / 16);       // waves that share 16 keys
  const int grp = wv / GW, piece0 = grp * (16 * CPR) + (wv % GW) * (NI * kWave);
  uint32_t klane[NI], vlane[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int key = (piece0 + i * kWave + lane) / CPR, c = lane % CPR;
    klane[i] = ES * (uint32_t)(key & 15) * (uint32_t)P.k_tok + 16 * (C == codes::kNone ? c ^ k_turn<D>(key) : c);
    vlane[i] = ES * (uint32_t)(key & 15) * (uint32_t)P.v_tok + 16 * (C == codes::kNone ? c ^ v_turn<D>(key) : c);
  }
  // scalar instructions are a quarter of the loop's: 32-bit strides (the host has seen to it), and one place for K and V alike
  const uint32_t k_page = (uint32_t)(ES * P.k_page), k_tok = (uint32_t)(ES * P.k_tok);
  const uint32_t v_page = (uint32_t)(ES * P.v_page), v_tok = (uint32_t)(ES * P.v_tok);
  const bool alike = k_page == v_page && k_tok == v_tok;
  for (int i = t; i <= P.G; i += kPfThreads) units[i] = (uint32_t)P.plan.group_units[i];   // none where the layout is bad
  __syncthreads();
  const uint32_t U = (uint32_t)uni((int)units[P.G]), W = min((uint32_t)gridDim.x, U);
  // Neighbouring ranges on one die: blocks go to the eight dies in turn
  const uint32_t per_die = gridDim.x / 8;
  const uint32_t w = U >= gridDim.x && gridDim.x % 8 == 0 ? blockIdx.x % 8 * per_die + blockIdx.x / 8 : blockIdx.x;
  if (w >= W) return;
  uint32_t u = range_start(w, W, U);
  const uint32_t u_end = range_start(w + 1, W, U);
  int gi = 0;
  for (int step = 4096; step > 0; step >>= 1)
    if (gi + step < P.G && (uint32_t)uni((int)units[gi + step]) <= u) gi += step;
  const float sl = fabsf(P.scale_log2);                              // not 0 (the host has seen to it): scores behind the prefix are -inf
  const uint32_t flip = P.scale_log2 < 0.f ? 0x80008000u : 0u;       // the sign of the scale goes to the queries
  while (u < u_end) {
    while ((uint32_t)uni((int)units[gi + 1]) <= u) ++gi;
    const AttnRecord rec = P.plan.group[gi];
    const int row0 = uni(rec.row0), n = uni(rec.n), slot = uni(rec.slot), len = uni(rec.len), tile0 = uni(rec.tile0);
    const int nblk = (len + kUnitKeys - 1) / kUnitKeys;
    const uint32_t rel = u - (uint32_t)uni((int)units[gi]);
    const int seg = (int)(rel / (uint32_t)nblk), b0 = (int)(rel - (uint32_t)seg * nblk);
    const int b1 = (int)min((uint32_t)nblk, b0 + (u_end - u));
    const int tiles = (n * P.group + TM - 1) / TM;
    const int head = seg / tiles, mb = seg - head * tiles;
    if (b0 == 0 && t == 0) P.plan.tile[tile0 + mb * P.kv_heads + head] = make_int2((int)w, (int)(range_of(u + (uint32_t)nblk - 1, W, U) - w) + 1);
    const int nrow = min(TM, n * P.group - mb * TM);
    const bool busy = wv * 32 < nrow;            // this wave has rows
    const int r = wv * 32 + col;
    const int rr = mb * TM + (r < nrow ? r : 0), ri = rr / P.group;
    u32x4 q[NS];
    {
      const uint16_t* qp = (const uint16_t*)P.q + (int64_t)(row0 + ri) * P.q_row + (int64_t)(head * P.group + rr - ri * P.group) * P.q_head + 8 * h;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        q[s] = *(const u32x4*)(qp + 16 * s);
#pragma unroll
        for (int i = 0; i < 4; ++i) q[s][i] ^= flip;
      }
    }
    f32x16 o[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[j][i] = 0.f;
    float mx = -INFINITY, ls = 0.f;
    bool bad = slot < 0;
    const int32_t* table = P.table + (int64_t)max(slot, 0) * P.table_stride;
    const int pmask = (1 << P.page_log2) - 1;
    const char* khead = (const char*)P.k + ES * (int64_t)head * P.k_head;
    const char* vhead = (const char*)P.v + ES * (int64_t)head * P.v_head;
    u32x4 kr[NI], vr[NI];                        // codes on their way
    float scr = 0.f;                             // and a scale: of key lane & 15 of the wave's, values' from lane 16 on
    int id = 0;
    // by a vector load: with a scalar one under way each wait for shared memory is one for everything
    auto names = [&](int pos) {
      int i = min(pos + 16 * grp, len - 1) >> P.page_log2;
      asm("" : "+v"(i));
      id = table[i];
    };
    // 16-bit keys go straight to shared memory, 1 KB a wave at a time: the lane
    // whose place is piece c of a row brings the piece that belongs there
    auto load = [&](int buf, int pos) {
      const int name = uni(id);
      const bool out = (unsigned)name >= (unsigned)P.num_pages;
      bad |= out;
      const uint32_t page = out ? 0u : (uint32_t)name, tok = (uint32_t)((pos + 16 * grp) & pmask);
      const char* kp = khead + ((uint64_t)page * k_page + tok * k_tok);
      const char* vp = alike ? vhead + (kp - khead) : vhead + ((uint64_t)page * v_page + tok * v_tok);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        if constexpr (C == codes::kNone) {
          load_lds(kp, klane[i], &ksh[buf][piece0 + i * kWave]);
          load_lds(vp, vlane[i], &vsh[buf][piece0 + i * kWave]);
        } else {
          kr[i] = *(const u32x4*)(kp + klane[i]);
          vr[i] = *(const u32x4*)(vp + vlane[i]);
        }
      }
      if constexpr (C != codes::kNone) {
        if (wv % GW == 0) {
          const float* kq = P.ks + ((int64_t)page * P.ks_page + (int64_t)head * P.ks_head + tok);
          const float* vq = P.vs + ((int64_t)page * P.vs_page + (int64_t)head * P.vs_head + tok);
          scr = (lane < 16 ? kq : vq)[lane & 15];
        }
      }
    };
    // Codes into shared memory.  Values behind the prefix become 0 (0 * NaN is
    // NaN; their scores are replaced).
    auto stage = [&](int buf, int pos) {
      if constexpr (C == codes::kNone) {
        if (pos + KT > len) {
          __syncthreads();                       // the values have come
          for (int i = (len - pos) * (D / 8) + t; i < KT * (D / 8); i += kPfThreads) vsh[buf][i] = u32x4{0u, 0u, 0u, 0u};
        }
      } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int key = (piece0 + i * kWave + lane) / CPR, c0 = lane % CPR;
          if (pos + key >= len) vr[i] = u32x4{0u, 0u, 0u, 0u};
          u32x4* kd = &ksh[buf][key * (D / 8)];
          u32x4* vd = &vsh[buf][key * (D / 8)];
          kd[(2 * c0) ^ k_turn<D>(key)] = widen8<BF, C>(kr[i][0], kr[i][1]);
          kd[(2 * c0 + 1) ^ k_turn<D>(key)] = widen8<BF, C>(kr[i][2], kr[i][3]);
          vd[(2 * c0) ^ v_turn<D>(key)] = widen8<true, C>(vr[i][0], vr[i][1]);
          vd[(2 * c0 + 1) ^ v_turn<D>(key)] = widen8<true, C>(vr[i][2], vr[i][3]);
        }
        if (wv % GW == 0) {
          const int key = 16 * grp + (lane & 15);
          const float s = pos + key < len ? scr : 0.f;
          if (lane < 16) kscale[buf][key] = s * sl;
          else if (lane < 32) vscale[buf][key] = s;
        }
      }
    };
    const int pos0 = b0 * kUnitKeys, pos_end = min(len, b1 * kUnitKeys);
    names(pos0);
    load(0, pos0);                               // the last tile's keys have been read
    if (pos0 + KT < pos_end) names(pos0 + KT);
    stage(0, pos0);
    __syncthreads();
    int buf = 0;
    for (int pos = pos0; pos < pos_end; pos += KT, buf ^= 1) {
      const bool more = pos + KT < pos_end;
      // The compiler would wait for each read right in front of its product: the
      // order is fixed here, with kAhead reads under way, the first of them while
      // the next keys are sent for.
      const char* kb = kbase + buf * (KT * D * 2);
      char* vb = vbase + buf * (KT * D * 2);
      constexpr int N = NT * NS, kAhead = C == codes::kNone ? 8 : 5;
      u32x4 k[kAhead];
      auto read = [&](int i) { k[i % kAhead] = *(const u32x4*)(kb + (i % NT) * (64 * D) + (koff ^ (32 * (i / NT)))); };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) read(i);
      __builtin_amdgcn_sched_barrier(0);
      if (more) {
        load(buf ^ 1, pos + KT);
        if (pos + 2 * KT < pos_end) names(pos + 2 * KT);
      }
      if (busy) {
        f32x16 s[NT];
        {
#pragma unroll
          for (int a = 0; a < NT; ++a)
#pragma unroll
            for (int i = 0; i < 16; ++i) s[a][i] = 0.f;
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            s[i % NT] = mfma32<BF>(k[i % kAhead], q[i / NT], s[i % NT]);
            if (i + kAhead < N) read(i + kAhead);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
        u32x4 v[2][NJ];                          // the values of 16 keys, and of the next
        auto read_v = [&](int c, int k) {        // half k & 1 of tile k >> 1's operand, keys 16 c ..
          const u32x2 y = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (TrPtr)(vb + (16 * c + 8 * (k & 1)) * (2 * D) + (voff ^ (64 * (k >> 1))))));
          v[c & 1][k >> 1][2 * (k & 1)] = y[0];
          v[c & 1][k >> 1][2 * (k & 1) + 1] = y[1];
        };
#pragma unroll
        for (int k = 0; k < 2 * NJ; ++k) read_v(0, k);
        if constexpr (C != codes::kNone) {
#pragma unroll
          for (int a = 0; a < NT; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const f32x4 f = *(const f32x4*)&kscale[buf][32 * a + 8 * i + 4 * h];
#pragma unroll
              for (int k = 0; k < 4; ++k) s[a][4 * i + k] *= f[k];
            }
        }
        if (pos + KT > len) {
#pragma unroll
          for (int a = 0; a < NT; ++a)
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (pos + 32 * a + 8 * (i >> 2) + 4 * h + (i & 3) >= len) s[a][i] = -INFINITY;
        }
        float top = s[0][0];
#pragma unroll
        for (int a = 0; a < NT; ++a)
#pragma unroll
          for (int i = 0; i < 16; ++i) top = fmaxf(top, s[a][i]);
        if constexpr (C == codes::kNone) top *= sl;
        if (__ballot(top > mx + kSlack)) {       // far above what some row's weights are taken against: rescale
          const float nm = fmaxf(mx, pair_max(top));
          const float f = mx == nm ? 1.f : at_exp2(reference<PB>(mx) - reference<PB>(nm));
          mx = nm;
          ls *= f;
#pragma unroll
          for (int j = 0; j < NJ; ++j) o[j] *= f;
        }
        const float ref = mx == -INFINITY ? 0.f : reference<PB>(mx);
        // 16 keys at a time, the slots of one product.  A wave's products and the next
        // 16 keys' weights are interleaved by hand, since each takes about as long as
        // the other: 2 NJ products of 32 cycles, 8 weights of about 40.
        u32x4 ph[2], pl[2];
        float p[8], eight = 0.f;
        f32x4 vf[2];
        auto weight = [&](int c, int e) {
          if constexpr (C != codes::kNone)
            if (e == 0) {
              vf[0] = *(const f32x4*)&vscale[buf][16 * c + 4 * h];
              vf[1] = *(const f32x4*)&vscale[buf][16 * c + 8 + 4 * h];
            }
          const float x = s[c >> 1][8 * (c & 1) + e];
          p[e] = at_exp2(C == codes::kNone ? fmaf(x, sl, -ref) : x - ref);
          eight = e ? eight + p[e] : p[e];
          if (e == 7) ls += eight;               // summed up first, as in k_attention
          if constexpr (C != codes::kNone) p[e] *= vf[e >> 2][e & 3];
          if (e & 1) {
            uint32_t hi, lo;
            split16<PB>(p[e - 1], p[e], &hi, &lo);
            ph[c & 1][e >> 1] = hi;
            pl[c & 1][e >> 1] = lo;
          }
        };
#pragma unroll
        for (int e = 0; e < 8; ++e) weight(0, e);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int c = 0; c < 2 * NT; ++c) {
#pragma unroll
          for (int k = 0; k < 2 * NJ; ++k) {
            const int j = k % NJ;
            o[j] = mfma32<PB>(v[c & 1][j], k < NJ ? ph[c & 1] : pl[c & 1], o[j]);
            if (c + 1 < 2 * NT) {
              read_v(c + 1, k);
#pragma unroll
              for (int e = k * 8 / (2 * NJ); e < (k + 1) * 8 / (2 * NJ); ++e) weight(c + 1, e);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
      if (more) stage(buf ^ 1, pos + KT);
      __syncthreads();
    }
    // a lane's row: numbers 32 j + 8 i + 4 h .. + 3
    const float M = reference<PB>(mx);
    float L = pair_sum(ls);
    if (__syncthreads_or(bad)) L = __builtin_nanf("");
    if (r < nrow) {
      const bool whole = b0 == 0 && b1 == nblk;
      float* part = part_at(P.prefix_parts, (int)w, b0 > 0 ? 0 : 1, TM, D);
      const int64_t at = state_row(P, row0, head, mb * TM + r);
      float* to = whole ? P.state_o + at * 4 : part + r * 4;
      const int64_t four = 4 * (whole ? (int64_t)P.total_rows * P.heads : TM);
      const float f = whole ? (L == 0.f ? 0.f : 1.f / L) : 1.f;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f32x4 v;
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = o[j][4 * i + k] * f;
          *(f32x4*)(to + (8 * j + 2 * i + h) * four) = v;
        }
      if (h == 0) {
        if (whole) {
          P.state_m[at] = L == 0.f ? -INFINITY : M + log2f(L);
        } else {
          part[TM * D + r] = M;
          part[TM * D + TM + r] = L;
        }
      }
    }
    u += (uint32_t)(b1 - b0);
  }
}

namespace {

template <bool BF, int D, int C>
hipError_t launch_prefix_one(const AttnParams& p, hipStream_t st) {
  hipLaunchKernelGGL((k_prefix<BF, D, C>), dim3((unsigned)p.prefix_blocks), dim3(kPfThreads), (size_t)(p.G + 1) * 4, st, p);
  return hipGetLastError();
}

template <int C>
hipError_t launch_prefix_rows(const AttnParams& p, hipStream_t st) {
  switch (p.head_dim) {
    case 64: return p.bf16 ? launch_prefix_one<true, 64, C>(p, st) : launch_prefix_one<false, 64, C>(p, st);
    case 128: return p.bf16 ? launch_prefix_one<true, 128, C>(p, st) : launch_prefix_one<false, 128, C>(p, st);
    case 256: return p.bf16 ? launch_prefix_one<true, 256, C>(p, st) : launch_prefix_one<false, 256, C>(p, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace

}  // namespace sv
