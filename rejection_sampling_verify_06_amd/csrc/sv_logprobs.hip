// Log probabilities of given tokens, with entropy, rank and top alternatives,
// for gfx950.
//
// For a row of logits x over V tokens and a temperature T (c = log2(e) / T):
//   M = max x,  y_j = x_j c - round(M c),  S = sum 2^y_j,  W = sum 2^y_j (-y_j)
//   log p(t)  = (y_t - log2 S) ln 2
//   entropy   = (log2 S + W / S) ln 2            (both terms are >= 0 up to rounding)
//   rank(t)   = 1 + the number of logits > x_t
//   top n     = the n largest logits, the lower index first on ties
// One read of the logits carries all of it: k_logprob_chunks reduces 32 KB of
// a row to (M, S, W, count) and the maximum of each 512-byte segment, and
// k_logprob_rows merges a row's chunks and finds its top n.  A token of the
// top n lies in one of the n first segments ordered by (maximum, index): a
// segment behind n others has n tokens in front of each of its own.  So the
// second kernel reads n segments again, 20 of 594 for 152064 bf16 logits,
// whatever the values.
//
// Sums are kept in 32 bits, in a fixed order; y is rounded once (fma).

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "sv_internal.h"
#include "sv_wave.h"

namespace sv {

namespace {

using namespace wave;

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int kLpThreads = 256;
constexpr int kLpWaves = kLpThreads / kWave;
constexpr int kSegBytes = 512;                              // a segment: 8 lanes, 4 vectors of 16 bytes each
constexpr int kSegs = kChunkBytes / kSegBytes;              // 64 segments to a chunk
constexpr int kPasses = kSegs / (kLpThreads / 8);           // 2: segments per group of 8 lanes
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;
constexpr float kSafe = 0x1p120f;                           // |M c| below this: fma(x, c, -M c) cannot overflow upwards
constexpr float kMinTemp = SV_MIN_TEMPERATURE;

__device__ __forceinline__ float lp_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// Where a row starts: its first 16-byte boundary lies `shift` elements before
// element 0, so that the vectors of every row are aligned.
template <bool BF>
struct Row {
  static constexpr int ES = BF ? 2 : 4;
  static constexpr int VEC = 16 / ES;
  static constexpr int SEG = kSegBytes / ES;
  static constexpr int CHUNK = kChunkBytes / ES;
  const char* base;
  int shift;
  __device__ __forceinline__ Row(const LogprobParams& P, int64_t row) {
    base = (const char*)P.logits + row * P.ld * ES;
    shift = (int)((uintptr_t)base & 15) / ES;
  }
  __device__ __forceinline__ float at(int e) const {
    return BF ? __uint_as_float((uint32_t)((const uint16_t*)base)[e] << 16) : ((const float*)base)[e];
  }
  // raw element, or -inf outside [0, V)
  __device__ __forceinline__ uint32_t raw(int e, int V) const {
    if (e < 0 || e >= V) return BF ? 0xFF80u : 0xFF800000u;
    return BF ? (uint32_t)((const uint16_t*)base)[e] : ((const uint32_t*)base)[e];
  }
  // elements e .. e + VEC - 1 (e + shift is a multiple of VEC); only elements of the row are read
  __device__ __forceinline__ u32x4 vec(int e, int V) const {
    if (e >= 0 && e + VEC <= V) return __builtin_nontemporal_load((const u32x4*)(base + (int64_t)e * ES));
    u32x4 v;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      v[q] = BF ? raw(e + 2 * q, V) | (raw(e + 2 * q + 1, V) << 16) : raw(e + q, V);
    return v;
  }
  static __device__ __forceinline__ void unpack(const u32x4& v, float (&x)[VEC]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if constexpr (BF) {
        x[2 * q] = __uint_as_float(v[q] << 16);
        x[2 * q + 1] = __uint_as_float(v[q] & 0xFFFF0000u);
      } else {
        x[q] = __uint_as_float(v[q]);
      }
    }
  }
};

// c = log2(e) / T, or NaN for a temperature that is refused
__device__ __forceinline__ float lp_scale(const LogprobParams& P, int64_t row) {
  if (!P.temperature) return kLog2e;
  const float T = P.temperature[row];
  return (isfinite(T) && T >= kMinTemp) ? kLog2e / T : __builtin_nanf("");
}

// log p(x) of a row with maximum M and log2 S = logS.  A logit near the
// type's lowest value (a mask) would overflow in log2 units before its natural
// logarithm does: log2 S is lost in its rounding anyway.
__device__ __forceinline__ float lp_value(const LogprobParams& P, int64_t row, float x, float M, float c, float logS) {
  if (x - M < -0x1p100f) return P.temperature ? (x - M) / P.temperature[row] : x - M;
  const float K = M * c;
  const float y = fabsf(K) < kSafe ? fmaf(x, c, -K) : (x - M) * c;
  return fminf((y - logS) * kLn2, 0.f);
}

// (S, W) of maximum m brought to maximum M >= m.  The shift is the difference
// of the two rounded references; where one of them would overflow the sums
// were taken against (x - m) c instead.
__device__ __forceinline__ void rebase(float m, float M, float c, float& S, float& W) {
  if (m == M || m == -INFINITY) return;                     // an empty part has S = W = 0 (or NaN, which stays)
  const bool safe = fabsf(m * c) < kSafe && fabsf(M * c) < kSafe;
  const float d = safe ? M * c - m * c : (M - m) * c;
  const float r = lp_exp2(-d);
  W = r > 0.f ? (W + d * S) * r : (S == S ? 0.f : S);
  S = r > 0.f ? S * r : (S == S ? 0.f : S);
}

struct ChunkStats {
  float M, S, W;
  int n;
};

}  // namespace

// One block per (row, 32 KB chunk).  Bound by HBM: the 8 vectors of a thread
// are in flight together, and the waves reduce against their own maximum, so
// one barrier is left.
template <bool BF, bool ENT, bool RANK>
__global__ void __launch_bounds__(kLpThreads) k_logprob_chunks(LogprobParams P) {
  using R = Row<BF>;
  constexpr int VEC = R::VEC;
  __shared__ ChunkStats part[kLpWaves];
  const int64_t lin = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (lin >= P.rows * P.nch) return;
  const int64_t row = lin / P.nch;
  const int chunk = (int)(lin - row * P.nch);
  int tok = 0;
  if (P.tokens) {
    tok = P.tokens[row];
    if (tok < 0) return;                                    // a row without a token is not read
  }
  const float c = lp_scale(P, row);
  if (!(c > 0.f)) return;
  const R r(P, row);
  const int V = (int)P.V;
  const int t = threadIdx.x, lane = t & (kWave - 1), w = t / kWave;
  // group of 8 lanes g takes segments g and g + 32 of the chunk, 128 contiguous bytes at a time
  const int e0 = chunk * R::CHUNK + (t >> 3) * R::SEG + (t & 7) * VEC - r.shift;
  u32x4 v[kPasses][4];
  const int c0 = chunk * R::CHUNK - r.shift;
  if (c0 >= 0 && c0 + R::CHUNK <= V) {
#pragma unroll
    for (int p = 0; p < kPasses; ++p)
#pragma unroll
      for (int u = 0; u < 4; ++u)
        v[p][u] = __builtin_nontemporal_load(
            (const u32x4*)(r.base + ((int64_t)e0 + p * (kLpThreads / 8) * R::SEG + u * 8 * VEC) * R::ES));
  } else {
#pragma unroll
    for (int p = 0; p < kPasses; ++p)
#pragma unroll
      for (int u = 0; u < 4; ++u) v[p][u] = r.vec(e0 + p * (kLpThreads / 8) * R::SEG + u * 8 * VEC, V);
  }
  const float xt = (RANK && tok < V) ? r.at(tok) : INFINITY;
  float m = -INFINITY;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    float sm = -INFINITY;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float x[VEC];
      R::unpack(v[p][u], x);
#pragma unroll
      for (int q = 0; q < VEC; ++q) sm = fmaxf(sm, x[q]);
    }
    sm = row8_max(sm);
    if (P.segmax && (t & 7) == 0) P.segmax[lin * kSegs + p * (kLpThreads / 8) + (t >> 3)] = sm;
    m = fmaxf(m, sm);
  }
  const float M = wave_max(m);
  float S = 0.f, W = 0.f;
  int n = 0;
  const float K = M * c;
  const bool safe = fabsf(K) < kSafe;                       // false for M = -inf or inf as well
  const float Mr = M == -INFINITY ? 0.f : M;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float x[VEC];
      R::unpack(v[p][u], x);
#pragma unroll
      for (int q = 0; q < VEC; ++q) {
        if (RANK) n += __popcll(__ballot(x[q] > xt));
        x[q] = safe ? fmaf(x[q], c, -K) : (x[q] - Mr) * c;
      }
#pragma unroll
      for (int q = 0; q < VEC; ++q) {
        const float e = lp_exp2(x[q]);                      // NaN stays NaN
        S += e;
        if (ENT) W = fmaf(-fmaxf(x[q], -1e30f), e, W);      // 0 * (-inf) is 0 here
      }
    }
  }
  S = wave_sum(S);
  if (ENT) W = wave_sum(W);
  if (lane == 0) part[w] = ChunkStats{M, S, W, n};
  __syncthreads();
  if (t == 0) {
    ChunkStats a = part[0];
#pragma unroll
    for (int i = 1; i < kLpWaves; ++i) a.M = fmaxf(a.M, part[i].M);
    rebase(part[0].M, a.M, c, a.S, a.W);
#pragma unroll
    for (int i = 1; i < kLpWaves; ++i) {
      ChunkStats b = part[i];
      rebase(b.M, a.M, c, b.S, b.W);
      a.S += b.S;
      a.W += b.W;
      a.n += b.n;
    }
    reinterpret_cast<float4*>(P.partials)[lin] = make_float4(a.M, a.S, a.W, __int_as_float(a.n));
  }
}

namespace {

// floats as unsigned integers of the same order (-0 and 0 alike)
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

constexpr int kSegRegs = 20;                                // segment maxima a lane keeps: rows of up to 1280 segments

// Calls f(r, key) for the segments r * 64 + lane of a row; keys of absent segments are 0 (below every float's).
template <bool REG, typename F>
__device__ __forceinline__ void each_segment(const uint32_t (&key)[kSegRegs], const float* sm, int nseg, int lane, F f) {
  if constexpr (REG) {
#pragma unroll
    for (int r = 0; r < kSegRegs; ++r)
      if (r * kWave < nseg) f(r, key[r]);
  } else {
    for (int r = 0; r * kWave < nseg; ++r) {
      const int i = r * kWave + lane;
      f(r, i < nseg ? ordered(sm[i]) : 0u);
    }
  }
}

// The n first segments by (maximum, index), n < nseg, into list[]: the n-th
// largest maximum is found bit by bit with ballots over all maxima (a wave
// holds them in registers up to 1280 segments), then the segments above it
// and, in index order, as many that equal it as are missing.
template <bool REG, bool BF>
__device__ __forceinline__ void first_segments(const float* sm, int nseg, int n, int lane, int* list) {
  uint32_t key[kSegRegs];
  if constexpr (REG) {
#pragma unroll
    for (int r = 0; r < kSegRegs; ++r) {
      const int i = r * kWave + lane;
      key[r] = i < nseg ? ordered(sm[i]) : 0u;
    }
  }
  // bf16 keys end in 16 equal bits: all 0 above zero, all 1 below it
  uint32_t thr = 0;
  for (int bit = 31; bit >= (BF ? 16 : 0); --bit) {
    const uint32_t cand = thr | (1u << bit);
    int cnt = 0;
    each_segment<REG>(key, sm, nseg, lane, [&](int, uint32_t k) { cnt += __popcll(__ballot(k >= cand)); });
    if (cnt >= n) thr = cand;
  }
  const uint32_t last = BF ? thr | 0xFFFFu : thr;           // keys in [thr, last] are the n-th maximum's
  int above = 0;
  each_segment<REG>(key, sm, nseg, lane, [&](int, uint32_t k) { above += __popcll(__ballot(k > last)); });
  int want = n - above, at = 0;
  const uint64_t lower = (1ull << lane) - 1;
  each_segment<REG>(key, sm, nseg, lane, [&](int r, uint32_t k) {
    const uint64_t eq = __ballot(k >= thr && k <= last);
    const bool take = k > last || (k >= thr && __popcll(eq & lower) < want);
    const uint64_t all = __ballot(take);
    if (take) list[at + __popcll(all & lower)] = r * kWave + lane;
    want -= min(want, (int)__popcll(eq));
    at += __popcll(all);
  });
}

}  // namespace

// One wave per row: merges the chunks, writes the row's values, finds its top
// n.  Bound by latency (four dependent loads: token, partials and maxima,
// segments, and the search between them).
template <bool BF>
__global__ void __launch_bounds__(kWave) k_logprob_rows(LogprobParams P) {
  using R = Row<BF>;
  __shared__ int list[SV_LOGPROBS_MAX_TOP];
  const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= P.rows) return;
  const int lane = threadIdx.x;
  const int top = P.top, V = (int)P.V;
  const int tok = P.tokens ? P.tokens[row] : -1;
  const float c = lp_scale(P, row);
  const bool skip = P.tokens && tok < 0;
  int st = skip ? 0 : (!(c > 0.f) ? SV_ST_BAD_TEMPERATURE : 0) | (P.tokens && tok >= V ? SV_ST_BAD_TOKEN : 0);
  float lp = 0.f, ent = 0.f, M = -INFINITY, S = 0.f, W = 0.f;
  int n = 0;
  const R r(P, row);
  if (!skip && !st) {
    const float xt = P.tokens ? r.at(tok) : 0.f;
    const float4* pp = reinterpret_cast<const float4*>(P.partials) + row * P.nch;
    for (int k = lane; k < P.nch; k += kWave) {
      const float4 q = pp[k];
      const float m = fmaxf(M, q.x);
      float s = q.y, wq = q.z;
      rebase(M, m, c, S, W);
      rebase(q.x, m, c, s, wq);
      M = m;
      S += s;
      W += wq;
      n += __float_as_int(q.w);
    }
    const float m = wave_max(M);
    rebase(M, m, c, S, W);
    M = m;
    S = wave_sum(S);
    W = wave_sum(W);
    n = (int)wave_sum_u32((uint32_t)n);
    if (!(S > 0.f) || !(fabsf(M) < INFINITY)) {             // NaN, +inf, or nothing but -inf
      st |= SV_ST_NONFINITE;
    } else {
      const float logS = log2f(S);
      lp = lp_value(P, row, xt, M, c, logS);
      ent = fmaxf((logS + W / S) * kLn2, 0.f);
    }
  }
  const bool bad = st != 0;
  if (lane == 0) {
    const float nan = __builtin_nanf("");
    if (P.logprob) P.logprob[row] = bad ? nan : lp;
    if (P.entropy) P.entropy[row] = bad ? nan : ent;
    if (P.rank) P.rank[row] = (bad || skip) ? 0 : n + 1;
    if (P.status) P.status[row] = st;
  }
  if (top == 0) return;
  float bv = -INFINITY;                                     // the top list: lane i holds the i-th, best first
  int bi = 0x7FFFFFFF;
  if (!skip && !bad) {
    const int nseg = (V + r.shift + R::SEG - 1) / R::SEG;
    const int ns = min(top, nseg);
    if (nseg > top) {
      const float* sm = P.segmax + row * P.nch * kSegs;
      if (nseg <= kSegRegs * kWave) first_segments<true, BF>(sm, nseg, top, lane, list);
      else first_segments<false, BF>(sm, nseg, top, lane, list);
    } else if (lane < ns) {
      list[lane] = lane;
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    constexpr int PER = R::SEG / kWave;                     // a lane's elements of a segment: 4 bf16 or 2 floats
    constexpr int NB = 8;                                   // segments in flight
    for (int s0 = 0; s0 < ns; s0 += NB) {
      uint32_t raw[NB][PER];
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int e = (s0 + j < ns ? list[s0 + j] : list[0]) * R::SEG - r.shift + lane * PER;
#pragma unroll
        for (int q = 0; q < PER; ++q) raw[j][q] = r.raw(e + q, V);
      }
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        if (s0 + j >= ns) break;
        const int e = list[s0 + j] * R::SEG - r.shift + lane * PER;
#pragma unroll
        for (int q = 0; q < PER; ++q) {
          const float x = __uint_as_float(BF ? raw[j][q] << 16 : raw[j][q]);
          const int id = e + q;
          const float wv = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(bv), top - 1));
          const int wi = __builtin_amdgcn_readlane(bi, top - 1);
          uint64_t better = __ballot(id >= 0 && id < V && (x > wv || (x == wv && id < wi)));
          while (better) {
            const int src = __builtin_ctzll(better);
            better &= better - 1;
            const float nv = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), src));
            const int ni = __builtin_amdgcn_readlane(id, src);
            // the entries in front of the new one stay, the others move one lane up
            const int pos = __popcll(__ballot(bv > nv || (bv == nv && bi < ni)));
            const float pv = __shfl_up(bv, 1);
            const int pi = __shfl_up(bi, 1);
            bv = lane < pos ? bv : (lane == pos ? nv : pv);
            bi = lane < pos ? bi : (lane == pos ? ni : pi);
          }
        }
      }
    }
  }
  if (lane < top) {
    float out = skip ? -INFINITY : __builtin_nanf("");
    if (!skip && !bad) out = lp_value(P, row, bv, M, c, log2f(S));
    P.top_tokens[row * top + lane] = (skip || bad) ? -1 : bi;
    if (P.top_logprobs) P.top_logprobs[row * top + lane] = out;
  }
}

hipError_t launch_logprobs(const LogprobParams& p, hipStream_t st) {
  const int64_t blocks = p.rows * p.nch;
  const int64_t gy = (blocks + kMaxGrid - 1) / kMaxGrid, gx = (blocks + gy - 1) / gy;
  const dim3 g((unsigned)gx, (unsigned)gy), b(kLpThreads);
  const bool ent = p.entropy != nullptr, rank = p.rank != nullptr;
  auto go = [&](auto k) { hipLaunchKernelGGL(k, g, b, 0, st, p); };
  if (p.bf16) {
    if (ent) rank ? go(k_logprob_chunks<true, true, true>) : go(k_logprob_chunks<true, true, false>);
    else rank ? go(k_logprob_chunks<true, false, true>) : go(k_logprob_chunks<true, false, false>);
  } else {
    if (ent) rank ? go(k_logprob_chunks<false, true, true>) : go(k_logprob_chunks<false, true, false>);
    else rank ? go(k_logprob_chunks<false, false, true>) : go(k_logprob_chunks<false, false, false>);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t ry = (p.rows + kMaxGrid - 1) / kMaxGrid, rx = (p.rows + ry - 1) / ry;
  const dim3 gr((unsigned)rx, (unsigned)ry);
  if (p.bf16) hipLaunchKernelGGL(k_logprob_rows<true>, gr, dim3(kWave), 0, st, p);
  else hipLaunchKernelGGL(k_logprob_rows<false>, gr, dim3(kWave), 0, st, p);
  return hipGetLastError();
}

}  // namespace sv
