// The paged key-value cache's own operations, for gfx950: pages for a round's
// new tokens (reserve, with copy on write), rolling a round back to what the
// verify call accepted (commit, truncate, release), sharing a prefix between
// sequences (fork), moving the live pages to the front of the pool (compact),
// and writing new keys and values into their places (write).
//
// A page is free where its count of users is 0, and the lowest free pages are
// taken first, in the order of the entries: what a call does is a pure
// function of the state, whatever the blocks' timing.
//
// The bookkeeping is integers on small arrays, bound by the latency of
// dependent steps, so each operation is one block of 1024 threads that keeps
// the entries' prefix sums in shared memory; work on pages or rows is spread
// over its threads by position, the owning entry found by a binary search of
// those sums.  (Four positions of a thread at a time, so that their loads
// overlap, measured slower: reserve 7.5 -> 10.3 us, truncate 3.2 -> 4.5; the
// longer code costs more than the overlap saves.)  Copies of pages and rows are
// bound by HBM and run on the whole chip, from a list that stays on the device.
//
// Measured on one MI355X (rocprofv3): 32 sequences growing by up to 6 tokens,
// reserve 7.1 us and its empty copy 1.9 us, commit 3.2 us, write 2.9 us a layer;
// 6905 prompt tokens, reserve 13 us, write 14 us a layer (57 MB, 4.0 TB/s); 180
// pages of 32 KB in 16 pools copied on write, 36 us (189 MB, 5.2 TB/s; where
// three branches copy the same page it is read behind the L2 about twice, 166
// MB in all by the counters).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sv_internal.h"
#include "sv_wave.h"

namespace sv {

namespace {

using namespace wave;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kCaThreads = 1024;
constexpr int kCaWaves = kCaThreads / kWave;
constexpr int kScanPer = 16;                     // counts of users a thread takes at a time
constexpr int kCopyThreads = 256;
constexpr int kCopyBytes = kCopyThreads * 64;    // bytes a block copies at a time: four 16-byte vectors a thread
constexpr uint32_t kCow = 0x80000000u;           // entry flags above a prefix sum of pages
constexpr uint32_t kRefused = 0x40000000u;
constexpr uint32_t kSum = 0x3FFFFFFFu;

struct CacheShared {
  uint32_t wave[kCaWaves];
  int flag;
  uint32_t count;
};

// exclusive prefix of v over the block, and the block's total
__device__ __forceinline__ uint32_t block_scan(uint32_t v, CacheShared& sh, uint32_t* total) {
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
  const uint32_t in = wave_incl_scan_u32(v);
  __syncthreads();                               // the last scan's totals have been read
  if (lane == kWave - 1) sh.wave[w] = in;
  __syncthreads();
  uint32_t before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kCaWaves; ++i) {
    const uint32_t x = sh.wave[i];
    before += i < w ? x : 0u;
    all += x;
  }
  *total = all;
  return before + in - v;
}

// The first entry whose inclusive prefix sum is above j.
__device__ __forceinline__ int owner(const uint32_t* end, int n, uint32_t j) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if ((end[mid] & kSum) > j) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}
__device__ __forceinline__ uint32_t before(const uint32_t* end, int b) { return b ? end[b - 1] & kSum : 0u; }

__device__ __forceinline__ int slot_of(const CacheParams& P, const int32_t* seqs, int b) { return seqs ? seqs[b] : b; }

// Each slot's first entry: an entry whose slot is out of range or belongs to an earlier one is refused.
__device__ __forceinline__ void claim_slots(const CacheParams& P, const int32_t* seqs, int* claim) {
  for (int i = threadIdx.x; i < P.slots; i += kCaThreads) claim[i] = 0x7FFFFFFF;
  __syncthreads();
  for (int b = threadIdx.x; b < P.B; b += kCaThreads) {
    const int s = slot_of(P, seqs, b);
    if ((unsigned)s < (unsigned)P.slots) atomicMin(&claim[s], b);
  }
  __syncthreads();
}
__device__ __forceinline__ bool claimed(const CacheParams& P, const int* claim, int s, int b) {
  return (unsigned)s < (unsigned)P.slots && claim[s] == b;
}

__device__ __forceinline__ int pages_of(const CacheParams& P, int len) { return (int)(((int64_t)len + P.page_size - 1) >> P.page_log2); }

// 16 counts of users from page p on; pages outside the pool read as used
__device__ __forceinline__ void load_counts(const CacheParams& P, int p, int (&c)[kScanPer]) {
  if (p + kScanPer <= P.num_pages) {
#pragma unroll
    for (int i = 0; i < kScanPer / 4; ++i) {
      const int4 v = reinterpret_cast<const int4*>(P.refcount + p)[i];
      c[4 * i] = v.x;
      c[4 * i + 1] = v.y;
      c[4 * i + 2] = v.z;
      c[4 * i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kScanPer; ++i) c[i] = p + i < P.num_pages ? P.refcount[p + i] : 1;
  }
}

}  // namespace

__global__ void __launch_bounds__(kCaThreads) k_cache_reserve(CacheParams P) {
  extern __shared__ uint32_t dyn[];
  __shared__ CacheShared sh;
  uint32_t* pend = dyn;                          // inclusive prefix of the pages asked for, with flags
  uint32_t* rend = dyn + P.B;                    // inclusive prefix of the new tokens
  int* claim = reinterpret_cast<int*>(dyn + 2 * P.B);
  const int t = threadIdx.x;
  const int mask = P.page_size - 1;
  if (t == 0) {
    sh.flag = 0;
    sh.count = 0;
  }
  claim_slots(P, P.seqs, claim);
  uint32_t pages = 0, rows = 0;
  for (int b0 = 0; b0 < P.B; b0 += kCaThreads) {
    const int b = b0 + t;
    uint32_t need = 0, n = 0, flags = 0;
    if (b < P.B) {
      const int nn = P.num_new[b], s = slot_of(P, P.seqs, b);
      int st = 0;
      if (nn < 0 || nn > P.total_new) sh.flag = 1;
      else n = (uint32_t)nn;
      if (!claimed(P, claim, s, b)) {
        st = SV_ST_BAD_SEQ;
      } else {
        const int L = P.seq_len[s];
        if (L < 0 || (int64_t)L + n > P.max_len) {
          st = SV_ST_BAD_LENGTH;
        } else if (n > 0) {
          const int had = pages_of(P, L);
          if (L & mask) {
            const int tail = P.table[(int64_t)s * P.max_pages + had - 1];
            if ((unsigned)tail >= (unsigned)P.num_pages) st = SV_ST_BAD_PAGE;
            else if (P.refcount[tail] > 1) flags = kCow;
          }
          if (!st) need = (uint32_t)(pages_of(P, L + (int)n) - had) + (flags ? 1u : 0u);
        }
      }
      if (st) flags = kRefused;
      if (P.status) P.status[b] = st;
    }
    uint32_t tp, tr;
    const uint32_t ap = block_scan(need, sh, &tp), ar = block_scan(n, sh, &tr);
    if (b < P.B) {
      pend[b] = (pages + ap + need) | flags;
      rend[b] = rows + ar + n;
    }
    pages += tp;
    rows += tr;
  }
  __syncthreads();
  if (sh.flag || rows != (uint32_t)P.total_new) {   // the rows do not add up: nothing changes
    for (int b = t; b < P.B; b += kCaThreads) {
      P.start[b] = -1;
      if (P.status) P.status[b] = SV_ST_BAD_LAYOUT;
    }
    for (int64_t r = t; r < P.total_new; r += kCaThreads) P.new_slots[r] = -1;
    if (t == 0) *P.count = 0;
    return;
  }
  // the lowest free pages, as many as were asked for
  uint32_t found = 0;
  for (int p0 = 0; p0 < P.num_pages && found < pages; p0 += kCaThreads * kScanPer) {
    int c[kScanPer];
    const int p = p0 + t * kScanPer;
    load_counts(P, p, c);
    uint32_t mine = 0, total;
#pragma unroll
    for (int i = 0; i < kScanPer; ++i) mine += c[i] == 0;
    uint32_t at = found + block_scan(mine, sh, &total);
#pragma unroll
    for (int i = 0; i < kScanPer; ++i)
      if (c[i] == 0) {
        if (at < pages) P.ids[at] = p + i;
        ++at;
      }
    found += total;
  }
  const uint32_t have = min(found, pages);
  __syncthreads();
  // the entries: lengths, and the copies of shared last pages
  for (int b = t; b < P.B; b += kCaThreads) {
    const uint32_t e = pend[b], end = e & kSum, beg = before(pend, b);
    const int s = slot_of(P, P.seqs, b);
    int start = -1;
    if (!(e & kRefused)) {
      if (end != beg && end > have) {
        if (P.status) P.status[b] = SV_ST_CACHE_FULL;
      } else {
        start = P.seq_len[s];
        P.seq_len[s] = start + P.num_new[b];
        if (e & kCow) {
          int32_t* tail = P.table + (int64_t)s * P.max_pages + pages_of(P, start) - 1;
          const int src = *tail, dst = P.ids[beg];
          *tail = dst;
          P.refcount[dst] = 1;
          atomicSub(&P.refcount[src], 1);
          P.pairs[atomicAdd(&sh.count, 1u)] = make_int2(src, dst);
        }
      }
    }
    P.start[b] = start;
  }
  __syncthreads();
  // the other new pages
  for (uint32_t j = t; j < have; j += kCaThreads) {
    const int b = owner(pend, P.B, j);
    const int start = P.start[b];
    const int k = (int)(j - before(pend, b)), cow = pend[b] & kCow ? 1 : 0;
    if (start < 0 || k < cow) continue;
    const int id = P.ids[j];
    P.table[(int64_t)slot_of(P, P.seqs, b) * P.max_pages + pages_of(P, start) + k - cow] = id;
    P.refcount[id] = 1;
  }
  __syncthreads();
  // where each new token goes
  for (int64_t r = t; r < P.total_new; r += kCaThreads) {
    int lo = 0, hi = P.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (rend[mid] > (uint32_t)r) hi = mid;
      else lo = mid + 1;
    }
    const int start = P.start[lo];
    int64_t at = -1;
    if (start >= 0) {
      const int pos = start + (int)((uint32_t)r - (lo ? rend[lo - 1] : 0u));
      at = (int64_t)P.table[(int64_t)slot_of(P, P.seqs, lo) * P.max_pages + (pos >> P.page_log2)] * P.page_size + (pos & mask);
    }
    P.new_slots[r] = at;
  }
  if (t == 0) *P.count = (int)sh.count;
}

// Takes the last tokens off each entry's sequence: drop[b] of them, or with
// num_draft / accepted what a verify call did not accept, or all.  Pages that
// no longer hold a token of the sequence lose it as a user.
__global__ void __launch_bounds__(kCaThreads) k_cache_truncate(CacheParams P) {
  extern __shared__ uint32_t dyn[];
  __shared__ CacheShared sh;
  uint32_t* pend = dyn;                          // inclusive prefix of the pages given up
  uint32_t* left = dyn + P.B;                    // pages each entry keeps
  int* claim = reinterpret_cast<int*>(dyn + 2 * P.B);
  const int t = threadIdx.x;
  claim_slots(P, P.seqs, claim);
  uint32_t pages = 0;
  for (int b0 = 0; b0 < P.B; b0 += kCaThreads) {
    const int b = b0 + t;
    uint32_t gone = 0, keep = 0;
    if (b < P.B) {
      const int s = slot_of(P, P.seqs, b);
      int st = 0;
      if (!claimed(P, claim, s, b)) {
        st = SV_ST_BAD_SEQ;
      } else {
        const int L = P.seq_len[s];
        int64_t d = L;
        bool ok = L >= 0 && L <= P.max_len;
        if (P.drop) {
          d = P.drop[b];
        } else if (P.num_draft) {
          const int K = P.num_draft[b], A = P.accepted[b];
          ok = ok && K >= 0 && A >= -1 && A <= K;
          // what a refused reserve did not add is not there to be dropped
          if (P.reserved) ok = ok && P.reserved[b] >= 0 && (int64_t)P.reserved[b] + K + 1 == L;
          d = (int64_t)K - A;                    // A = -1, not verified: all K + 1 new tokens
        }
        ok = ok && d >= 0 && d <= L;
        if (!ok) {
          st = SV_ST_BAD_LENGTH;
        } else {
          keep = (uint32_t)pages_of(P, L - (int)d);
          gone = (uint32_t)pages_of(P, L) - keep;
          P.seq_len[s] = L - (int)d;
        }
      }
      if (P.status) P.status[b] = st;
    }
    uint32_t total;
    const uint32_t at = block_scan(gone, sh, &total);
    if (b < P.B) {
      pend[b] = pages + at + gone;
      left[b] = keep;
    }
    pages += total;
  }
  __syncthreads();
  for (uint32_t j = t; j < pages; j += kCaThreads) {
    const int b = owner(pend, P.B, j);
    int32_t* e = P.table + (int64_t)slot_of(P, P.seqs, b) * P.max_pages + left[b] + (j - before(pend, b));
    const int id = *e;
    *e = -1;
    if ((unsigned)id < (unsigned)P.num_pages) atomicSub(&P.refcount[id], 1);
  }
}

// children[b] becomes a second user of everything parents[b] holds.  A child
// has to be empty; parents are taken as they were before the call.
__global__ void __launch_bounds__(kCaThreads) k_cache_fork(CacheParams P) {
  extern __shared__ uint32_t dyn[];
  __shared__ CacheShared sh;
  uint32_t* pend = dyn;
  int* plen = reinterpret_cast<int*>(dyn + P.B);
  int* claim = reinterpret_cast<int*>(dyn + 2 * P.B);
  const int t = threadIdx.x;
  claim_slots(P, P.children, claim);
  uint32_t pages = 0;
  for (int b0 = 0; b0 < P.B; b0 += kCaThreads) {
    const int b = b0 + t;
    uint32_t n = 0;
    if (b < P.B) {
      const int s = P.seqs[b], c = P.children[b];
      int st = 0, L = -1;
      if (!claimed(P, claim, c, b) || (unsigned)s >= (unsigned)P.slots) {
        st = SV_ST_BAD_SEQ;
      } else {
        L = P.seq_len[s];
        if (L < 0 || L > P.max_len || P.seq_len[c] != 0) {
          st = SV_ST_BAD_LENGTH;
          L = -1;
        } else {
          n = (uint32_t)pages_of(P, L);
        }
      }
      plen[b] = L;
      if (P.status) P.status[b] = st;
    }
    uint32_t total;
    const uint32_t at = block_scan(n, sh, &total);
    if (b < P.B) pend[b] = pages + at + n;
    pages += total;
  }
  __syncthreads();
  for (int b = t; b < P.B; b += kCaThreads)
    if (plen[b] >= 0) P.seq_len[P.children[b]] = plen[b];
  for (uint32_t j = t; j < pages; j += kCaThreads) {
    const int b = owner(pend, P.B, j);
    const int64_t k = j - before(pend, b);
    const int id = P.table[(int64_t)P.seqs[b] * P.max_pages + k];
    P.table[(int64_t)P.children[b] * P.max_pages + k] = id;
    if ((unsigned)id < (unsigned)P.num_pages) atomicAdd(&P.refcount[id], 1);
  }
}

// The live pages behind the first `live` places, in order, against the free
// places among those, in order: pairs (from, to), and the new names in ids.
__global__ void __launch_bounds__(kCaThreads) k_cache_compact(CacheParams P) {
  __shared__ CacheShared sh;
  const int t = threadIdx.x;
  uint32_t live = 0;
  for (int p0 = 0; p0 < P.num_pages; p0 += kCaThreads * kScanPer) {
    int c[kScanPer];
    const int p = p0 + t * kScanPer;
    load_counts(P, p, c);
    uint32_t mine = 0, total;
#pragma unroll
    for (int i = 0; i < kScanPer; ++i) mine += c[i] != 0 && p + i < P.num_pages;
    block_scan(mine, sh, &total);
    live += total;
  }
  uint32_t holes = 0, moves = 0;
  for (int p0 = 0; p0 < P.num_pages; p0 += kCaThreads * kScanPer) {
    int c[kScanPer];
    const int p = p0 + t * kScanPer;
    load_counts(P, p, c);
    uint32_t h = 0, m = 0, th, tm;
#pragma unroll
    for (int i = 0; i < kScanPer; ++i) {
      h += c[i] == 0 && p + i < (int)live;
      m += c[i] != 0 && p + i >= (int)live && p + i < P.num_pages;
    }
    uint32_t ah = holes + block_scan(h, sh, &th), am = moves + block_scan(m, sh, &tm);
#pragma unroll
    for (int i = 0; i < kScanPer; ++i) {
      if (p + i >= P.num_pages) break;
      if (c[i] == 0 && p + i < (int)live) P.pairs[ah++].y = p + i;
      if (c[i] != 0 && p + i >= (int)live) P.pairs[am++].x = p + i;
      P.ids[p + i] = p + i;
    }
    holes += th;
    moves += tm;
  }
  __syncthreads();
  for (uint32_t k = t; k < moves; k += kCaThreads) {
    const int2 m = P.pairs[k];
    P.ids[m.x] = m.y;
    P.refcount[m.y] = P.refcount[m.x];
    P.refcount[m.x] = 0;
  }
  if (t == 0) {
    *P.count = (int)moves;
    if (P.live) P.live[0] = (int)live;
  }
}

// The pages of the list, in every layer, K and V; with `remap` the first
// blocks give the page tables their new names (which the copies do not read).
__global__ void __launch_bounds__(kCopyThreads) k_cache_copy(CacheParams P, int remap) {
  const int t = threadIdx.x;
  if ((int)blockIdx.x < remap) {
    for (int s = blockIdx.x; s < P.slots; s += remap) {
      const int n = pages_of(P, min(max(P.seq_len[s], 0), P.max_len));
      int32_t* row = P.table + (int64_t)s * P.max_pages;
      for (int i = t; i < n; i += kCopyThreads) {
        const int id = row[i];
        if ((unsigned)id < (unsigned)P.num_pages) row[i] = P.ids[id];
      }
    }
    return;
  }
  const int count = *P.count;
  const int64_t chunks = (P.page_bytes + kCopyBytes - 1) / kCopyBytes;
  const int64_t total = (int64_t)count * P.layers * 2 * chunks;
  for (int64_t i = blockIdx.x - remap; i < total; i += gridDim.x - remap) {
    const int64_t c = i % chunks, r = i / chunks;
    const int which = (int)(r & 1);
    const int64_t r2 = r >> 1, layer = r2 / count, k = r2 - layer * count;
    const int2 m = P.pairs[k];
    char* pool = (char*)(which ? P.v : P.k) + layer * P.layer_bytes;
    const char* src = pool + (int64_t)m.x * P.page_bytes + c * kCopyBytes;
    char* dst = pool + (int64_t)m.y * P.page_bytes + c * kCopyBytes;
    const int64_t n = min((int64_t)kCopyBytes, P.page_bytes - c * kCopyBytes);
    u32x4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int at = (u * kCopyThreads + t) * 16;
      if (at < n) v[u] = __builtin_nontemporal_load((const u32x4*)(src + at));
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int at = (u * kCopyThreads + t) * 16;
      if (at < n) __builtin_nontemporal_store(v[u], (u32x4*)(dst + at));
    }
  }
}

// New keys and values into their places: one 16-byte vector to a thread, a
// row's K and V together.  A place outside the pool (-1: refused) is left out.
__global__ void __launch_bounds__(kCopyThreads) k_cache_write(CacheWriteParams P) {
  const int64_t i = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x;
  const int64_t row = i / P.vecs;
  if (row >= P.rows) return;
  const int c = (int)(i - row * P.vecs);
  const int64_t at = P.new_slots[row];
  if (at < 0 || at >= P.places) return;
  const int64_t page = at >> P.page_log2;
  const int off = (int)(at & ((1 << P.page_log2) - 1));
  const int h = c / P.head_vecs, d = (c - h * P.head_vecs) * 8;
  const int64_t dst = (((page * P.kv_heads + h) << P.page_log2) + off) * P.head_dim + d;
  const u32x4 k = *(const u32x4*)((const uint16_t*)P.k_new + row * P.k_row + h * P.k_head + d);
  const u32x4 v = *(const u32x4*)((const uint16_t*)P.v_new + row * P.v_row + h * P.v_head + d);
  *(u32x4*)((uint16_t*)P.k + dst) = k;
  *(u32x4*)((uint16_t*)P.v + dst) = v;
}

namespace {

size_t lds_bytes(const CacheParams& p) { return 4 * (2 * (size_t)p.B + (size_t)p.slots); }

// Blocks of a copy whose length only the device knows: enough to fill the
// chip when there is work, few enough to cost little when there is none.
int copy_blocks(const CacheParams& p, int64_t most) {
  const int64_t chunks = (p.page_bytes + kCopyBytes - 1) / kCopyBytes;
  const int64_t n = most * p.layers * 2 * chunks;
  return (int)(n < 2048 ? n : 2048);
}

}  // namespace

hipError_t launch_cache_reserve(const CacheParams& p, hipStream_t st) {
  hipLaunchKernelGGL(k_cache_reserve, dim3(1), dim3(kCaThreads), lds_bytes(p), st, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_cache_copy, dim3((unsigned)copy_blocks(p, p.B)), dim3(kCopyThreads), 0, st, p, 0);
  return hipGetLastError();
}

hipError_t launch_cache_truncate(const CacheParams& p, hipStream_t st) {
  hipLaunchKernelGGL(k_cache_truncate, dim3(1), dim3(kCaThreads), lds_bytes(p), st, p);
  return hipGetLastError();
}

hipError_t launch_cache_fork(const CacheParams& p, hipStream_t st) {
  hipLaunchKernelGGL(k_cache_fork, dim3(1), dim3(kCaThreads), lds_bytes(p), st, p);
  return hipGetLastError();
}

hipError_t launch_cache_compact(const CacheParams& p, hipStream_t st) {
  hipLaunchKernelGGL(k_cache_compact, dim3(1), dim3(kCaThreads), 0, st, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int remap = p.slots < 256 ? p.slots : 256;
  hipLaunchKernelGGL(k_cache_copy, dim3((unsigned)(remap + copy_blocks(p, (p.num_pages + 1) / 2))), dim3(kCopyThreads), 0, st, p, remap);
  return hipGetLastError();
}

hipError_t launch_cache_write(const CacheWriteParams& p, hipStream_t st) {
  const int64_t n = p.rows * p.vecs;
  hipLaunchKernelGGL(k_cache_write, dim3((unsigned)((n + kCopyThreads - 1) / kCopyThreads)), dim3(kCopyThreads), 0, st, p);
  return hipGetLastError();
}

}  // namespace sv
