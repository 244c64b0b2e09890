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
// flight to registers while these are worked on.
//
// Weights are split in two 16-bit halves and units dealt out in equal
// ranges, for the same reasons as in k_attention, whose join adds the parts up.

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

// Where 16-byte piece c of key r lies among the pieces of the staged keys.
template <int D>
__device__ __forceinline__ int k_piece(int r, int c) {
  return r * (D / 8) + (c ^ (D == 64 ? (r >> 1) & 7 : r & 15));
}
template <int D>
__device__ __forceinline__ int v_piece(int r, int c) {
  return r * (D / 8) + (c ^ (D == 64 ? ((r >> 1) & 1) << 2 : (r & 3) << 2));
}

}  // namespace

constexpr int kPfWaves = 4;
constexpr int kPfThreads = kPfWaves * 64;
constexpr int kPfRows = 32 * kPfWaves;
static_assert(kPfRows == kAttnPrefixRows, "rows of a tile");

template <int D>
constexpr int kPfKeys = D == 256 ? 32 : 64;      // keys staged at a time

template <bool BF, int D, int C>
__global__ void __launch_bounds__(kPfThreads, D == 256 ? 1 : D == 128 ? 2 : 3) k_prefix(AttnParams P) {
  constexpr bool PB = BF || C != codes::kNone;   // the second product's type
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
  uint32_t* rows = dyn;
  uint32_t* units = dyn + P.G + 1;
  __shared__ u32x4 ksh[2][KT * D / 8], vsh[2][KT * D / 8];
  __shared__ float kscale[2][KT], vscale[2][KT];
  const int t = threadIdx.x, lane = t & (kWave - 1), wv = uni(t / kWave);
  const int h = lane >> 5, col = lane & 31;
  load_plan(P, kPrefix, rows, units);
  Part* desc = reinterpret_cast<Part*>(P.desc);
  const uint32_t U = (uint32_t)uni((int)units[P.G]), W = min((uint32_t)gridDim.x, U);
  const uint32_t w = blockIdx.x;
  if (w >= W) {
    if (t == 0) desc[w].first_unit = -1;
    return;
  }
  uint32_t u = range_start(w, W, U);
  const uint32_t u_end = range_start(w + 1, W, U);
  int gi = 0;
  for (int step = 4096; step > 0; step >>= 1)
    if (gi + step < P.G && (uint32_t)uni((int)units[gi + step]) <= u) gi += step;
  bool first_part = true;
  const float sl = fabsf(P.scale_log2);
  const uint32_t flip = P.scale_log2 < 0.f ? 0x80008000u : 0u;       // the sign of the scale goes to the queries
  while (u < u_end) {
    while ((uint32_t)uni((int)units[gi + 1]) <= u) ++gi;
    const int row0 = uni((int)rows[gi]), n = uni((int)rows[gi + 1]) - row0;
    const int slot = uni(P.plan.group_slot[gi]), len = uni(P.plan.group_len[gi]);
    const int nblk = (len + kUnitKeys - 1) / kUnitKeys;
    const uint32_t rel = u - (uint32_t)uni((int)units[gi]);
    const int seg = (int)(rel / (uint32_t)nblk), b0 = (int)(rel - (uint32_t)seg * nblk);
    const int b1 = (int)min((uint32_t)nblk, b0 + (u_end - u));
    const int mb = seg / P.kv_heads, head = seg - mb * P.kv_heads;
    if (first_part && t == 0) {
      Part d;
      d.first_unit = b0 > 0 ? (int)(u - b0) : -1;
      d.end_unit = (int)(u - b0) + nblk;
      d.row0 = row0;
      d.n = n;
      d.head = head;
      d.mb = mb;
      d.U = U;
      d.W = W;
      desc[w] = d;
    }
    const int nrow = min(TM, n * P.group - mb * TM);
    const bool busy = wv * 32 < nrow;            // this wave has rows
    const int r = wv * 32 + col;
    const int rr = mb * TM + (r < nrow ? r : 0), ri = rr / P.group;
    const int64_t at = (int64_t)(row0 + ri) * P.heads + head * P.group + rr - ri * P.group;   // the row's place in the outputs
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
    typedef const __attribute__((address_space(4))) int32_t* Names;
    const Names table = (Names)(uintptr_t)(P.table + (int64_t)max(slot, 0) * P.table_stride);
    const int pmask = (1 << P.page_log2) - 1;
    const int c0 = t % CPR;
    u32x4 kr[NI], vr[NI];
    float scr = 0.f;                             // a scale: thread k brings that of key k, KT + k of value k
    int id[NI];
    // piece i of this thread is one of 16 keys of one page: those from 16 group(i) on
    auto group = [&](int i) { return (i * kPfThreads + wv * kWave) / (16 * CPR); };
    auto names = [&](int pos) {
#pragma unroll
      for (int i = 0; i < NI; ++i) id[i] = table[min(pos + 16 * group(i), len - 1) >> P.page_log2];
    };
    auto load = [&](int pos) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const bool out = (unsigned)id[i] >= (unsigned)P.num_pages;
        bad |= out;
        const int64_t page = out ? 0 : id[i];
        const int tok = ((pos + 16 * group(i)) & pmask) + (((i * kPfThreads + t) / CPR) & 15);
        kr[i] = *(const u32x4*)((const char*)P.k + ES * (page * P.k_page + (int64_t)head * P.k_head + (int64_t)tok * P.k_tok) + 16 * c0);
        vr[i] = *(const u32x4*)((const char*)P.v + ES * (page * P.v_page + (int64_t)head * P.v_head + (int64_t)tok * P.v_tok) + 16 * c0);
      }
      if constexpr (C != codes::kNone) {
        if (t < 2 * KT) {
          const int key = t % KT, kp = min(pos + key, len - 1);
          int pg = table[kp >> P.page_log2];
          pg = (unsigned)pg >= (unsigned)P.num_pages ? 0 : pg;
          scr = t < KT ? P.ks[(int64_t)pg * P.ks_page + (int64_t)head * P.ks_head + (kp & pmask)]
                       : P.vs[(int64_t)pg * P.vs_page + (int64_t)head * P.vs_head + (kp & pmask)];
        }
      }
    };
    // into shared memory; what is behind the prefix becomes 0 (0 * NaN is NaN)
    auto stage = [&](int buf, int pos) {
      const bool tail = pos + KT > len;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int key = (i * kPfThreads + t) / CPR;
        if (tail && pos + key >= len) {
          kr[i] = u32x4{0u, 0u, 0u, 0u};
          vr[i] = u32x4{0u, 0u, 0u, 0u};
        }
        if constexpr (C == codes::kNone) {
          ksh[buf][k_piece<D>(key, c0)] = kr[i];
          vsh[buf][v_piece<D>(key, c0)] = vr[i];
        } else {
          ksh[buf][k_piece<D>(key, 2 * c0)] = widen8<BF, C>(kr[i][0], kr[i][1]);
          ksh[buf][k_piece<D>(key, 2 * c0 + 1)] = widen8<BF, C>(kr[i][2], kr[i][3]);
          vsh[buf][v_piece<D>(key, 2 * c0)] = widen8<true, C>(vr[i][0], vr[i][1]);
          vsh[buf][v_piece<D>(key, 2 * c0 + 1)] = widen8<true, C>(vr[i][2], vr[i][3]);
        }
      }
      if constexpr (C != codes::kNone) {
        if (t < 2 * KT) {
          const int key = t % KT;
          const float s = pos + key < len ? scr : 0.f;
          if (t < KT) kscale[buf][key] = s * sl;
          else vscale[buf][key] = s;
        }
      }
    };
    const int pos0 = b0 * kUnitKeys, pos_end = min(len, b1 * kUnitKeys);
    names(pos0);
    load(pos0);
    if (pos0 + KT < pos_end) names(pos0 + KT);
    __syncthreads();                             // the last tile's keys have been read
    stage(0, pos0);
    __syncthreads();
    int buf = 0;
    for (int pos = pos0; pos < pos_end; pos += KT, buf ^= 1) {
      const bool more = pos + KT < pos_end;
      if (more) {
        load(pos + KT);
        if (pos + 2 * KT < pos_end) names(pos + 2 * KT);
      }
      if (busy) {
        f32x16 s[NT];
#pragma unroll
        for (int a = 0; a < NT; ++a) {
#pragma unroll
          for (int i = 0; i < 16; ++i) s[a][i] = 0.f;
#pragma unroll
          for (int i = 0; i < NS; ++i) s[a] = mfma32<BF>(ksh[buf][k_piece<D>(32 * a + col, 2 * i + h)], q[i], s[a]);
        }
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
        if (__ballot(top > mx)) {                // a new maximum in some row: rescale
          const float nm = fmaxf(mx, pair_max(top));
          const float f = mx == nm ? 1.f : at_exp2(reference<PB>(mx) - reference<PB>(nm));
          mx = nm;
          ls *= f;
#pragma unroll
          for (int j = 0; j < NJ; ++j) o[j] *= f;
        }
        const float ref = mx == -INFINITY ? 0.f : reference<PB>(mx);
#pragma unroll
        for (int a = 0; a < NT; ++a) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {          // 16 keys: the slots of one product
            float p[8], eight;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float x = s[a][8 * b + e];
              p[e] = at_exp2(C == codes::kNone ? fmaf(x, sl, -ref) : x - ref);
              eight = e ? eight + p[e] : p[e];
            }
            ls += eight;
            if constexpr (C != codes::kNone) {
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const f32x4 f = *(const f32x4*)&vscale[buf][32 * a + 16 * b + 8 * i + 4 * h];
#pragma unroll
                for (int k = 0; k < 4; ++k) p[4 * i + k] *= f[k];
              }
            }
            u32x4 ph, pl;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              ph[i] = pack16<PB>(p[2 * i], p[2 * i + 1]);
              pl[i] = pack16<PB>(p[2 * i] - lo16<PB>(ph[i]), p[2 * i + 1] - hi16<PB>(ph[i]));
            }
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
              u32x4 v;
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                // of four keys the 16 numbers around this lane's: 4 (lane & 3) .. + 3 of key (lane >> 2) & 3
                const int key = 32 * a + 16 * b + 8 * i + 4 * h + ((lane >> 2) & 3);
                const int d = 32 * j + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
                const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TrPtr)((char*)&vsh[buf][v_piece<D>(key, d >> 3)] + 2 * (d & 7)));
                const u32x2 y = __builtin_bit_cast(u32x2, x);
                v[2 * i] = y[0];
                v[2 * i + 1] = y[1];
              }
              o[j] = mfma32<PB>(v, ph, o[j]);
              o[j] = mfma32<PB>(v, pl, o[j]);
            }
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
      float* part = part_at(P, (int)w, b0 > 0 ? 0 : 1, TM, D);
      float* to = whole ? P.state_o + at * D : part + r * D;
      const float f = whole ? (L == 0.f ? 0.f : 1.f / L) : 1.f;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f32x4 v;
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = o[j][4 * i + k] * f;
          *(f32x4*)(to + 32 * j + 8 * i + 4 * h) = v;
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
    first_part = false;
    u += (uint32_t)(b1 - b0);
  }
}

namespace {

template <bool BF, int D, int C>
hipError_t launch_prefix_one(const AttnParams& p, int W, hipStream_t st) {
  hipLaunchKernelGGL((k_prefix<BF, D, C>), dim3((unsigned)W), dim3(kPfThreads), (size_t)(p.G + 1) * 8, st, p);
  hipError_t e = hipGetLastError();
  return e == hipSuccess ? launch_attention_join(p, kPrefix, kPfRows, W, st) : e;
}

template <int C>
hipError_t launch_prefix_rows(const AttnParams& p, int W, hipStream_t st) {
  switch (p.head_dim) {
    case 64: return p.bf16 ? launch_prefix_one<true, 64, C>(p, W, st) : launch_prefix_one<false, 64, C>(p, W, st);
    case 128: return p.bf16 ? launch_prefix_one<true, 128, C>(p, W, st) : launch_prefix_one<false, 128, C>(p, W, st);
    case 256: return p.bf16 ? launch_prefix_one<true, 256, C>(p, W, st) : launch_prefix_one<false, 256, C>(p, W, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace

}  // namespace sv
