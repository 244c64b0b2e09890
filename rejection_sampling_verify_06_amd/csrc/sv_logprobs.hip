// Log probabilities of given tokens, with entropy, rank and top alternatives,
// for gfx950.
//
// For a row of logits x over V tokens and a temperature T (c = log2(e) / T):
//   M = max x,  y_j = x_j c - round(M c),  S = sum 2^y_j,  W = sum 2^y_j (-y_j)
//   log p(t)  = (y_t - log2 S) ln 2
//   entropy   = (log2 S + W / S) ln 2            (both terms are >= 0 up to rounding)
//   rank(t)   = 1 + the number of logits > x_t
//   top n     = the n largest logits, the lower index first on ties
// One read of the logits carries all of it: k_logprob_chunks reduces 16 KB of
// a row to (M, S, W, count) and the maximum of each 512-byte segment, and
// k_logprob_rows merges a row's chunks and finds its top n.  It takes the
// largest segment maximum of each lane (64 interleaved sets of segments); the
// n-th largest of those is a floor that n tokens reach, so only the segments
// that reach it are read again, about 24 of 594 for n = 20 and 152064 bf16
// logits (all of them where a row ties).
//
// Sums are kept in 32 bits, in a fixed order; y is rounded once (fma).
//
// Measured on one MI355X (rocprofv3): 865 rows of 152064 bf16 logits among
// 1410 (263 MB) with 20 alternatives, chunks 52 us (5.1 TB/s), rows 18 us; every
// one of the 1410 rows, without alternatives, 69 us (6.2 TB/s); 119 rows of
// 128255 floats (61 MB) 15 + 4 us (4.0 TB/s: 3808 blocks, a short launch); 6
// rows of 32000 bf16 with 5 alternatives 5.3 + 8.4.

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "sv_internal.h"
#include "sv_wave.h"

namespace sv {

namespace {

using namespace wave;

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int kLpThreads = 256;
constexpr int kLpWaves = kLpThreads / kWave;
constexpr int kSegBytes = kLpSegBytes;
constexpr int kSegs = kLpSegs;
constexpr int kPasses = kSegs / (kLpThreads / 8);           // segments per group of 8 lanes
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;
constexpr float kSafe = 0x1p20f;                            // |M c| below this: 2^(M c - round(M c)) is near 1
constexpr float kMinTemp = SV_MIN_TEMPERATURE;

__device__ __forceinline__ float lp_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// Where a row starts: its first 16-byte boundary lies `shift` elements before
// element 0, so that the vectors of every row are aligned.
template <bool BF>
struct Row {
  static constexpr int ES = BF ? 2 : 4;
  static constexpr int VEC = 16 / ES;
  static constexpr int SEG = kSegBytes / ES;
  static constexpr int CHUNK = kLpChunkBytes / ES;
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
    const int i = min(max(e, 0), V - 1);
    const uint32_t x = BF ? (uint32_t)((const uint16_t*)base)[i] : ((const uint32_t*)base)[i];
    return e == i ? x : (BF ? 0xFF80u : 0xFF800000u);
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

// (S, W) of maximum m brought to maximum M >= m.  Sums are taken against
// round(m c) where that is below kSafe (one rounding per term, and the same
// reference for all), against m c itself, as (x - m) c, above; the shift is the
// difference of the two references.
__device__ __forceinline__ void rebase(float m, float M, float c, float& S, float& W) {
  if (m == M || m == -INFINITY) return;                     // an empty part has S = W = 0 (or NaN, which stays)
  const float k = m * c, K = M * c;
  const bool sm = fabsf(k) < kSafe, sM = fabsf(K) < kSafe;
  const float d = sm && sM ? K - k : (M - m) * c + (sm ? fmaf(m, c, -k) : 0.f) - (sM ? fmaf(M, c, -K) : 0.f);
  const float r = lp_exp2(-d);
  W = r > 0.f ? (W + d * S) * r : (S == S ? 0.f : S);
  S = r > 0.f ? S * r : (S == S ? 0.f : S);
}

// Each pass over the vectors unpacks them again: held unpacked from one pass
// to the next they would take twice the registers, and half of the waves that
// hide the reads.
__device__ __forceinline__ void forget_unpacked(u32x4 (&v)[kPasses][4]) {
#pragma unroll
  for (int p = 0; p < kPasses; ++p)
#pragma unroll
    for (int u = 0; u < 4; ++u) asm volatile("" : "+v"(v[p][u]));
}

// S = sum 2^y and W = sum 2^y (-y) over a thread's vectors, y = f(x), and n,
// the wave's elements above xt.  A masked token (y = -inf) adds 0 to W; NaN
// stays NaN in S.  The sums of a vector end with it: left for later by the
// compiler they would keep every exponential in registers.
template <typename R, bool ENT, bool COUNT, typename F>
__device__ __forceinline__ void chunk_sums(u32x4 (&v)[kPasses][4], F f, float xt, float& S, float& W, int& n) {
  forget_unpacked(v);
  S = W = 0.f;
  float S1 = 0.f, W1 = 0.f;
#pragma unroll
  for (int p = 0; p < kPasses; ++p)
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float x[R::VEC];
      R::unpack(v[p][u], x);
#pragma unroll
      for (int q = 0; q < R::VEC; q += 2) {
        if (COUNT) n += __popcll(__ballot(x[q] > xt)) + __popcll(__ballot(x[q + 1] > xt));
        const float y0 = f(x[q]), y1 = f(x[q + 1]);
        const float e0 = lp_exp2(y0), e1 = lp_exp2(y1);
        S += e0;
        S1 += e1;
        if (ENT) {
          W = fmaf(-fmaxf(y0, -1e30f), e0, W);
          W1 = fmaf(-fmaxf(y1, -1e30f), e1, W1);
        }
      }
      asm volatile("" : "+v"(S), "+v"(W), "+v"(S1), "+v"(W1));
      if (COUNT) asm volatile("" : "+s"(n));
    }
  S += S1;
  W += W1;
}

struct ChunkStats {
  float M, S, W;
  int n;
};

}  // namespace

// One block per (row, 16 KB chunk).  Bound by HBM and by its own ramp (about
// 10 us of a launch do not scale with the bytes): the 4 vectors of a thread are
// in flight together, and the waves reduce against their own maximum, so one
// barrier is left.  Chunks of 32 KB (8 vectors, 79 registers, 6 waves to a SIMD)
// took 58 us where these (47 registers) take 52.
template <bool BF, bool ENT, bool RANK>
__global__ void __launch_bounds__(kLpThreads, 8) k_logprob_chunks(LogprobParams P) {
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
      for (int u = 0; u < 4; ++u) {
        v[p][u] = r.vec(e0 + p * (kLpThreads / 8) * R::SEG + u * 8 * VEC, V);
        __builtin_amdgcn_sched_barrier(0);                  // the few edge chunks do not set the register count
      }
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
  forget_unpacked(v);
  const float M = wave_max(m);
  float S, W;
  int n = 0;
  const float K = M * c;
  if (fabsf(K) < kSafe) {
    chunk_sums<R, ENT, RANK>(v, [&](float x) { return fmaf(x, c, -K); }, xt, S, W, n);
  } else {                                                  // no finite maximum, or a small temperature
    const float Mr = M == -INFINITY ? 0.f : M;
    chunk_sums<R, ENT, RANK>(v, [&](float x) { return (x - Mr) * c; }, xt, S, W, n);
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

// The value of a key whose last 16 bits, for a bf16, were not looked at: they
// are equal bits, all 0 above zero and all 1 below it.
template <bool BF>
__device__ __forceinline__ float from_ordered(uint32_t k) {
  if (BF && !(k & 0x80000000u)) k |= 0xFFFFu;
  return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

// shared memory between the lanes of one wave
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A token of the top list: larger values first, then lower indices; 0 is below every token.
__device__ __forceinline__ uint64_t top_key(float x, int id) { return (uint64_t)ordered(x) << 32 | (uint32_t)~id; }
__device__ __forceinline__ float key_value(uint64_t k) {
  return k ? from_ordered<false>((uint32_t)(k >> 32)) : -INFINITY;
}
__device__ __forceinline__ uint64_t lane_key(uint64_t k, int l) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(k >> 32), l) << 32 |
         (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)k, l);
}

// the value of lane (lane ^ MASK): row moves inside 16 lanes where there is
// one, the row swaps of this ISA family across them
template <int MASK>
__device__ __forceinline__ uint32_t from_xor(uint32_t v, int lane) {
  if constexpr (MASK == 1) {
    return (uint32_t)dpp_i<kDppQuadXor1>(0, (int)v);
  } else if constexpr (MASK == 2) {
    return (uint32_t)dpp_i<kDppQuadXor2>(0, (int)v);
  } else if constexpr (MASK == 16) {
    const auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return lane & 16 ? s[0] : s[1];
  } else if constexpr (MASK == 32) {
    const auto s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return lane & 32 ? s[0] : s[1];
  } else {
    return (uint32_t)__builtin_amdgcn_ds_swizzle((int)v, 0x1F | MASK << 10);   // xor inside 32 lanes
  }
}
// one step of a bitonic network: the larger key to the lanes where `larger`
template <int MASK>
__device__ __forceinline__ void exchange(uint64_t& k, bool larger, int lane) {
  const uint64_t o = (uint64_t)from_xor<MASK>((uint32_t)(k >> 32), lane) << 32 | from_xor<MASK>((uint32_t)k, lane);
  k = (k > o) == larger ? k : o;
}
// The steps MASK, MASK / 2, .. 1 of a network whose lanes with `up` false sort the other way round.
template <int MASK>
__device__ __forceinline__ void bitonic(uint64_t& k, bool up, int lane) {
  exchange<MASK>(k, ((lane & MASK) == 0) == up, lane);
  if constexpr (MASK > 1) bitonic<MASK / 2>(k, up, lane);
}
// the wave's keys, largest first
__device__ __forceinline__ void sort_keys(uint64_t& k, int lane) {
  bitonic<1>(k, (lane & 2) == 0, lane);
  bitonic<2>(k, (lane & 4) == 0, lane);
  bitonic<4>(k, (lane & 8) == 0, lane);
  bitonic<8>(k, (lane & 16) == 0, lane);
  bitonic<16>(k, (lane & 32) == 0, lane);
  bitonic<32>(k, true, lane);
}
// the 64 largest of two sorted lists of 64, sorted: one list against the other's reverse, then one merge
__device__ __forceinline__ void merge_keys(uint64_t& a, uint64_t b, int lane) {
  const int back = (kWave - 1 - lane) * 4;
  const uint64_t r = (uint64_t)(uint32_t)__builtin_amdgcn_ds_bpermute(back, (int)(b >> 32)) << 32 |
                     (uint32_t)__builtin_amdgcn_ds_bpermute(back, (int)(uint32_t)b);
  a = a > r ? a : r;
  bitonic<32>(a, true, lane);
}

constexpr int kHeldMore = 512;                              // gathered tokens that may wait for more
constexpr int kListed = 16 * kWave;                         // segments listed before they are read
constexpr int kStage = 32;                                  // of those, read together

// The n-th largest of the wave's values (n <= 64), found bit by bit.
template <bool BF>
__device__ __forceinline__ float nth_of_wave(float x, int n) {
  const uint32_t key = ordered(x);
  uint32_t thr = 0;
  for (int bit = 31; bit >= (BF ? 16 : 0); --bit) {
    const uint32_t cand = thr | (1u << bit);
    if (__popcll(__ballot(key >= cand)) >= n) thr = cand;
  }
  return from_ordered<BF>(thr);
}

// The same over N values of every lane (NaN: none).
template <bool BF, int N>
__device__ __forceinline__ float nth_of_all(const float (&x)[N], int n) {
  uint32_t thr = 0;
  for (int bit = 31; bit >= (BF ? 16 : 0); --bit) {
    const uint32_t cand = thr | (1u << bit);
    int cnt = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) cnt += __popcll(__ballot(x[j] == x[j] && ordered(x[j]) >= cand));
    if (cnt >= n) thr = cand;
  }
  return from_ordered<BF>(thr);
}

}  // namespace

// One wave per row: merges the chunks, writes the row's values, finds its top
// n.  Bound by latency: the token, the partials and maxima, the segments, the
// search and sorts between them, and the fetch of code that runs once (8 us
// for one alternative, 14 us for 20, 35 us for 64; gathering the tokens of up
// to 32 segments and sorting them 64 at a time took 18 us where inserting them
// one by one took 61).
template <bool BF>
__global__ void __launch_bounds__(kWave) k_logprob_rows(LogprobParams P) {
  using R = Row<BF>;
  static_assert(R::SEG % kWave == 0, "a lane's share of a segment");
  __shared__ int list[kListed];
  __shared__ uint64_t cand[4 * R::SEG + kHeldMore];         // at least the two partial segments, or four whole ones more
  __shared__ u32x2 stage[kStage][kWave];
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
  uint64_t best = 0;                                        // the top list: lane i holds the i-th, best first
  if (!skip && !bad) {
    const int nseg = (V + r.shift + R::SEG - 1) / R::SEG;
    constexpr int PER = R::SEG / kWave;                     // a lane's tokens of a segment: 4 bf16 or 2 floats
    constexpr int NM = 16;                                  // maxima of a lane in flight: 1024 segments at a time
    const float* sm = P.segmax + row * P.nch * kSegs;
    const uint64_t lower = (1ull << lane) - 1;
    // `floor`: at least `top` segments (as many lanes' maxima), hence tokens, reach it
    float x[NM], lm = -INFINITY;
    auto load_maxima = [&](int i0) {
#pragma unroll
      for (int j = 0; j < NM; ++j) x[j] = sm[min(i0 + j * kWave + lane, nseg - 1)];
#pragma unroll
      for (int j = 0; j < NM; ++j) x[j] = i0 + j * kWave + lane < nseg ? x[j] : __builtin_nanf("");
    };
    for (int i0 = 0; i0 < nseg; i0 += NM * kWave) {
      load_maxima(i0);
#pragma unroll
      for (int j = 0; j < NM; ++j) lm = fmaxf(lm, x[j]);
    }
    float floor = nth_of_wave<BF>(lm, top);
    // Near 64 the n-th of 64 lane maxima is loose (64 of 594 segments are
    // wanted and about 300 reach it), and the n-th of all maxima pays: top 64
    // of 256 rows 35 us against 134; up to 32 both list about as many.
    if (top > 32 && nseg > top && nseg <= NM * kWave) floor = fmaxf(floor, nth_of_all<BF, NM>(x, top));
    int held = 0;
    // tokens of a segment that reach `floor`, gathered to be sorted 64 at a time and merged into the top list
    auto gather = [&](const uint32_t (&raw)[PER], int e) {
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        const float v = __uint_as_float(BF ? raw[q] << 16 : raw[q]);
        const bool in = (unsigned)(e + q) < (unsigned)V && v >= floor;
        const uint64_t mask = __ballot(in);
        if (mask) {
          if (in) cand[held + __popcll(mask & lower)] = top_key(v, e + q);
          held += __popcll(mask);
        }
      }
    };
    // the segments that lie only partly inside the row (the first and the last may), token by token
    const int inner0 = r.shift ? 1 : 0, inner1 = (V + r.shift) / R::SEG;   // whole segments: inner0 .. inner1 - 1
    for (int k = 0; k < 2; ++k) {
      const int sg = k ? nseg - 1 : 0;
      if ((sg >= inner0 && sg < inner1) || (k && nseg == 1)) continue;
      const int e = sg * R::SEG - r.shift + lane * PER;
      uint32_t raw[PER];
#pragma unroll
      for (int q = 0; q < PER; ++q) raw[q] = r.raw(e + q, V);
      gather(raw, e);
    }
    // A list of the whole segments that reach the floor, batches of it read
    // into shared memory, their tokens gathered until there are enough to
    // sort: one loop, so that its code, most of which runs once, is there once.
    int r0 = 0, listed = 0, s0 = 0, j0 = 0, here = 0, names = 0;
    bool done = false;
    while (true) {
      while (!done && held <= kHeldMore) {
        if (j0 < here) {                                    // four segments of the batch
          u32x2 v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = stage[j0 + j][lane];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (j0 + j >= here) break;
            uint32_t raw[PER];
#pragma unroll
            for (int q = 0; q < PER; ++q) raw[q] = BF ? (v[j][q / 2] >> (q & 1) * 16) & 0xFFFFu : v[j][q & 1];
            gather(raw, __builtin_amdgcn_readlane(names, j0 + j) * R::SEG - r.shift + lane * PER);
          }
          j0 += 4;
        } else if (s0 < listed) {                           // the next batch: 8 bytes a lane, all in flight
          wave_sync();
          u32x2 w[kStage];
          here = min(kStage, listed - s0);
          names = list[min(s0 + lane, listed - 1)];
#pragma unroll
          for (int j = 0; j < kStage; ++j)
            w[j] = *(const u32x2*)(r.base + (int64_t)(__builtin_amdgcn_readlane(names, j) * R::SEG - r.shift + lane * PER) * R::ES);
          float m = -INFINITY;                              // the lanes' largest tokens may raise the floor
#pragma unroll
          for (int j = 0; j < kStage; ++j) {
            stage[j][lane] = w[j];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              m = fmaxf(m, __uint_as_float(BF ? w[j][q] & 0xFFFF0000u : w[j][q]));
              if (BF) m = fmaxf(m, __uint_as_float(w[j][q] << 16));
            }
          }
          // a batch that is not full repeats its last segment in every lane alike: lane maxima stay what they are
          floor = fmaxf(floor, nth_of_wave<BF>(m, top));
          wave_sync();
          s0 += kStage;
          j0 = 0;
        } else if (r0 < nseg) {                             // the next 1024 segments
          if (nseg > NM * kWave) load_maxima(r0);
          wave_sync();
          listed = s0 = 0;
#pragma unroll
          for (int j = 0; j < NM; ++j) {
            const int i = r0 + j * kWave + lane;
            const bool reach = x[j] >= floor && i >= inner0 && i < inner1;
            const uint64_t all = __ballot(reach);
            if (all) {
              if (reach) list[listed + __popcll(all & lower)] = i;
              listed += __popcll(all);
            }
          }
          wave_sync();
          r0 += NM * kWave;
        } else {
          done = true;
        }
      }
      wave_sync();
      for (int k0 = 0; k0 < held; k0 += kWave) {
        uint64_t k = k0 + lane < held ? cand[k0 + lane] : 0;
        if (__ballot(k > lane_key(best, top - 1))) {
          sort_keys(k, lane);
          merge_keys(best, k, lane);
        }
      }
      if (done) break;
      held = 0;
      floor = fmaxf(floor, key_value(lane_key(best, top - 1)));
      wave_sync();
    }
  }
  if (lane < top) {
    float out = skip ? -INFINITY : __builtin_nanf("");
    if (!skip && !bad) out = lp_value(P, row, key_value(best), M, c, log2f(S));
    P.top_tokens[row * top + lane] = (skip || bad) ? -1 : (int)~(uint32_t)best;
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
