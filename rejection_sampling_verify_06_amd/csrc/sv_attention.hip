// Attention of a round's new tokens over a paged key-value cache, for gfx950:
// the 16-bit cache, and the parts' join of every kind of cache (the kernel and
// its reasons are in sv_attention_kernel.h).

#include "sv_attention_kernel.h"

namespace sv {

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
  auto part = [&](int i) { return (const float*)part_at(P.parts, (int)w - 1 + i, i == 0 ? 1 : 0, TM, D); };
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

hipError_t launch_attention_join(const AttnParams& p, int tm, int W, hipStream_t st) {
  const dim3 grid((unsigned)(W + (p.status ? p.B : 0)), (unsigned)(tm / kAtWaves)), block(kAtThreads);
  switch (p.head_dim * 2 + (p.bf16 ? 1 : 0)) {
    case 64 * 2: hipLaunchKernelGGL((k_attention_join<false, 64>), grid, block, 0, st, p, tm, W); break;
    case 64 * 2 + 1: hipLaunchKernelGGL((k_attention_join<true, 64>), grid, block, 0, st, p, tm, W); break;
    case 128 * 2: hipLaunchKernelGGL((k_attention_join<false, 128>), grid, block, 0, st, p, tm, W); break;
    case 128 * 2 + 1: hipLaunchKernelGGL((k_attention_join<true, 128>), grid, block, 0, st, p, tm, W); break;
    case 256 * 2: hipLaunchKernelGGL((k_attention_join<false, 256>), grid, block, 0, st, p, tm, W); break;
    case 256 * 2 + 1: hipLaunchKernelGGL((k_attention_join<true, 256>), grid, block, 0, st, p, tm, W); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

hipError_t launch_attention(const AttnParams& p, int row_tiles, int blocks, hipStream_t st) {
  return p.bf16 ? launch_type<true, codes::kNone, false>(p, row_tiles, blocks, st)
                : launch_type<false, codes::kNone, false>(p, row_tiles, blocks, st);
}

}  // namespace sv
