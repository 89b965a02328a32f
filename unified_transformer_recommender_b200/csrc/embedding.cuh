// Embedding table: lookup of rows by id with scaling, and its gradient by
// sorted ids.
//
//   lookup    out[r] = scale * table[ids[r]]
//   gradient  dT[v]  = scale * sum over r with ids[r] = v of dout[r]
//
// Id -1 is padding: a zero row, no gradient.  Any other id outside
// 0 .. n_rows-1 is taken as padding too and sets the device status word.
//
// The gradient groups equal ids by a stable radix sort of (id, position), so
// each row's terms are added in one fixed order whatever the launch timing
// (atomic adds on the table would not give that), and a row that occurs many
// thousand times is summed by many warps at once.  All sums are float32.
#pragma once
#include "tc_ptx.cuh"

namespace ot {

// --------------------------------------------------------------- elements --
// N consecutive elements as float32 by vector accesses (the address aligned
// to N elements, 16 bytes at most).
template <int N> __device__ inline void emb_ld(const float* p, float* v) {
  if constexpr (N >= 4) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 q = *(const float4*)(p + i);
      v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
    }
  } else if constexpr (N == 2) {
    const float2 q = *(const float2*)p;
    v[0] = q.x; v[1] = q.y;
  } else {
    v[0] = *p;
  }
}
template <int N> __device__ inline void emb_ld(const __nv_bfloat16* p, float* v) {
  if constexpr (N == 1) {
    v[0] = __bfloat162float(*p);
  } else {
    uint32_t w[N / 2];
    if constexpr (N == 8) { const uint4 q = *(const uint4*)p; w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w; }
    else if constexpr (N == 4) { const uint2 q = *(const uint2*)p; w[0] = q.x; w[1] = q.y; }
    else { w[0] = *(const uint32_t*)p; }
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float2 f = __bfloat1622float2(*(const __nv_bfloat162*)&w[i]);
      v[2 * i] = f.x; v[2 * i + 1] = f.y;
    }
  }
}
template <int N> __device__ inline void emb_st(float* p, const float* v) {
  if constexpr (N >= 4) {
#pragma unroll
    for (int i = 0; i < N; i += 4) *(float4*)(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else if constexpr (N == 2) {
    *(float2*)p = make_float2(v[0], v[1]);
  } else {
    *p = v[0];
  }
}
template <int N> __device__ inline void emb_st(__nv_bfloat16* p, const float* v) {
  if constexpr (N == 1) {
    *p = __float2bfloat16_rn(v[0]);
  } else {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    if constexpr (N == 8) *(uint4*)p = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (N == 4) *(uint2*)p = make_uint2(w[0], w[1]);
    else *(uint32_t*)p = w[0];
  }
}

// The sort key of an id: itself, or n_rows (behind every row) for padding.
template <typename Id>
__device__ inline uint32_t emb_key(Id id, uint32_t n_rows) {
  if (id >= 0 && (unsigned long long)id < n_rows) return (uint32_t)id;
  if (id != (Id)-1) flag_error(3);
  return n_rows;
}

// ----------------------------------------------------------------- lookup --
constexpr int kLookThreads = 256, kLookUnroll = 4;

// Each CTA takes `rows` output rows, each thread kLookUnroll groups of VE
// columns per round: the ids of all groups are loaded before the first row
// access, so that kLookUnroll row reads are in flight per thread.
template <typename Tt, typename To, typename Id, int VE>
__global__ void __launch_bounds__(kLookThreads) emb_lookup_kernel(const Tt* __restrict__ table, uint32_t n_rows,
                                                                  int width, const Id* __restrict__ ids, long long R,
                                                                  int rows, float scale, To* __restrict__ out,
                                                                  long long out_ld) {
  const int cpr = width / VE;
  const long long r0 = (long long)blockIdx.x * rows;
  const int items = (int)min((long long)rows, R - r0) * cpr;
  grid_dep_wait();
  grid_dep_launch();
  for (int i0 = threadIdx.x; i0 < items; i0 += kLookThreads * kLookUnroll) {
    uint32_t key[kLookUnroll];
    int row[kLookUnroll], col[kLookUnroll];
#pragma unroll
    for (int u = 0; u < kLookUnroll; ++u) {
      const int i = i0 + u * kLookThreads;
      row[u] = i / cpr;
      col[u] = (i - row[u] * cpr) * VE;
      key[u] = i < items ? emb_key(ids[r0 + row[u]], n_rows) : n_rows;
    }
    float v[kLookUnroll][VE];
#pragma unroll
    for (int u = 0; u < kLookUnroll; ++u) {
      if (key[u] < n_rows) {
        emb_ld<VE>(table + (long long)key[u] * width + col[u], v[u]);
#pragma unroll
        for (int e = 0; e < VE; ++e) v[u][e] *= scale;
      } else {
#pragma unroll
        for (int e = 0; e < VE; ++e) v[u][e] = 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < kLookUnroll; ++u)
      if (i0 + u * kLookThreads < items) emb_st<VE>(out + (r0 + row[u]) * out_ld + col[u], v[u]);
  }
}

// ------------------------------------------------------------------- sort --
// Stable least-significant-digit radix sort of (key, position).  A tile of
// kSortTile items per CTA; a pass ranks the items of its tile per digit (per
// warp by matching lanes, then across warps) and scatters them behind the
// same digits of the tiles before.  The counts of every (tile, digit) of a
// pass are ready when it starts: the first pass's come from sort_hist_kernel,
// a later pass's are added up, as integers, by the pass before it while it
// scatters (a destination's tile is known there).
constexpr int kSortThreads = 1024, kSortItems = 4, kSortTile = kSortThreads * kSortItems;
constexpr int kSortWarps = kSortThreads / 32, kSortMaxBits = 11;

struct SortArgs {
  uint32_t n_rows;       // keys 0 .. n_rows
  long long R;
  int tiles, bits, shift;   // digit = (key >> shift) & (2^bits - 1)
  int scanned;           // hist already holds the tile prefixes, tot the digit totals
  int* hist;             // this pass: [tiles][2^bits]
  int* tot;              // [2^bits]
  int* hist_next;        // the next pass's counts, or null
};

// Exclusive prefix of v over the CTA's threads; every thread calls it.
__device__ inline int block_exclusive(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();   // warp_sums free again
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int s = lane < nw ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(~0u, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  total = warp_sums[31];
  return x - v + (warp ? warp_sums[warp - 1] : 0);
}

template <typename Id>
__global__ void __launch_bounds__(kSortThreads) sort_hist_kernel(const Id* __restrict__ ids, SortArgs a,
                                                                 long long zero_ints) {
  __shared__ int h[1 << kSortMaxBits];
  const int bins = 1 << a.bits;
  for (int b = threadIdx.x; b < bins; b += kSortThreads) h[b] = 0;
  grid_dep_wait();
  grid_dep_launch();
  __syncthreads();
  const long long i0 = (long long)blockIdx.x * kSortTile;
#pragma unroll
  for (int u = 0; u < kSortItems; ++u) {
    const long long i = i0 + u * kSortThreads + threadIdx.x;
    if (i < a.R) atomicAdd(&h[(emb_key(ids[i], a.n_rows) >> a.shift) & (bins - 1)], 1);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kSortThreads) a.hist[(long long)blockIdx.x * bins + b] = h[b];
  // the later passes' counts start from zero
  for (long long i = (long long)blockIdx.x * kSortThreads + threadIdx.x; i < zero_ints;
       i += (long long)gridDim.x * kSortThreads)
    a.hist_next[i] = 0;
}

// hist[tile][digit] -> the digit's count in the tiles before, tot[digit] its
// total.  One CTA per 32 digits, the tiles split among the warps.
__global__ void __launch_bounds__(kSortThreads) sort_scan_kernel(SortArgs a) {
  __shared__ int part[kSortWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, bins = 1 << a.bits;
  const int b = blockIdx.x * 32 + lane;
  const int per = (a.tiles + kSortWarps - 1) / kSortWarps;
  const int t0 = min(a.tiles, warp * per), t1 = min(a.tiles, t0 + per);
  const bool on = b < bins;
  grid_dep_wait();
  grid_dep_launch();
  int s = 0;
  if (on)
    for (int t = t0; t < t1; ++t) s += a.hist[(long long)t * bins + b];
  part[warp][lane] = s;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kSortWarps; ++w) {
    const int p = part[w][lane];
    if (w < warp) before += p;
    all += p;
  }
  if (!on) return;
  if (warp == 0) a.tot[b] = all;
  for (int t = t0; t < t1; ++t) {
    int* p = a.hist + (long long)t * bins + b;
    const int c = *p;
    *p = before;
    before += c;
  }
}

// Ranks the CTA's items by digit, stably.  wh: [kSortWarps][bins] counts,
// zeroed by the caller; on return wh[w][b] is the count of digit b in the
// warps before w.  rank[u]: the item's rank among its warp's items of that
// digit.  Warp w's items are contiguous, item u of lane l at
// (w * kSortItems + u) * 32 + l.
__device__ inline void sort_rank(const uint32_t* digit, const bool* on, uint16_t* wh, int bins, int* rank) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint16_t* mine = wh + (long long)warp * bins;
#pragma unroll
  for (int u = 0; u < kSortItems; ++u) {
    const uint32_t same = __match_any_sync(~0u, on[u] ? digit[u] : 0xffffffffu);
    const int below = __popc(same & ((1u << lane) - 1));
    int base = 0;
    if (on[u]) base = mine[digit[u]];
    __syncwarp();
    if (on[u] && below == 0) mine[digit[u]] = (uint16_t)(base + __popc(same));
    __syncwarp();
    rank[u] = base + below;
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kSortThreads) {
    int s = 0;
#pragma unroll 8
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = wh[w * bins + b];
      wh[w * bins + b] = (uint16_t)s;
      s += c;
    }
  }
  __syncthreads();
}

// One pass.  FIRST: items are (id, position) from the caller's ids.
template <typename Id, bool FIRST>
__global__ void __launch_bounds__(kSortThreads) sort_pass_kernel(const Id* __restrict__ ids,
                                                                 const uint32_t* __restrict__ keys_in,
                                                                 const uint32_t* __restrict__ vals_in,
                                                                 uint32_t* __restrict__ keys, uint32_t* __restrict__ vals,
                                                                 SortArgs a, int next_bits, int next_shift) {
  extern __shared__ uint16_t sort_sm[];   // [kSortWarps][bins] u16, then [bins] int digit bases
  __shared__ int warp_sums[32];
  const int bins = 1 << a.bits, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int* base = (int*)(sort_sm + kSortWarps * bins);
  for (int i = threadIdx.x; i < kSortWarps * bins / 2; i += kSortThreads) ((uint32_t*)sort_sm)[i] = 0;
  grid_dep_wait();
  grid_dep_launch();
  uint32_t key[kSortItems], val[kSortItems], digit[kSortItems];
  bool on[kSortItems];
#pragma unroll
  for (int u = 0; u < kSortItems; ++u) {
    const long long i = (long long)blockIdx.x * kSortTile + (warp * kSortItems + u) * 32 + lane;
    on[u] = i < a.R;
    key[u] = !on[u] ? 0u : FIRST ? emb_key(ids[i], a.n_rows) : keys_in[i];
    val[u] = !on[u] ? 0u : FIRST ? (uint32_t)i : vals_in[i];
    digit[u] = (key[u] >> a.shift) & (bins - 1);
  }
  // where the tile's items of each digit begin
  int tot[2] = {0, 0}, mine[2] = {0, 0};
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int b = threadIdx.x * 2 + q;   // two neighbouring digits a thread (kSortMaxBits = 11)
    if (b < bins) {
      if (a.scanned) {
        tot[q] = a.tot[b];
        mine[q] = a.hist[(long long)blockIdx.x * bins + b];
      } else {
#pragma unroll 8
        for (int t = 0; t < a.tiles; ++t) {
          const int c = a.hist[(long long)t * bins + b];
          tot[q] += c;
          if (t < (int)blockIdx.x) mine[q] += c;
        }
      }
    }
  }
  int all;
  const int ex = block_exclusive(tot[0] + tot[1], warp_sums, all);
  if (threadIdx.x * 2 < bins) base[threadIdx.x * 2] = ex + mine[0];
  if (threadIdx.x * 2 + 1 < bins) base[threadIdx.x * 2 + 1] = ex + tot[0] + mine[1];
  int rank[kSortItems];
  sort_rank(digit, on, sort_sm, bins, rank);
#pragma unroll
  for (int u = 0; u < kSortItems; ++u) {
    if (!on[u]) continue;
    const int to = base[digit[u]] + sort_sm[warp * bins + digit[u]] + rank[u];
    keys[to] = key[u];
    vals[to] = val[u];
    if (a.hist_next)
      atomicAdd(&a.hist_next[((long long)(to / kSortTile) << next_bits) + ((key[u] >> next_shift) & ((1 << next_bits) - 1))], 1);
  }
}

// Up to kSortTile ids in one CTA: every pass through shared memory.
template <typename Id>
__global__ void __launch_bounds__(kSortThreads) sort_small_kernel(const Id* __restrict__ ids, uint32_t n_rows, int R,
                                                                  int passes, int bits, uint32_t* __restrict__ keys,
                                                                  uint32_t* __restrict__ vals, int* __restrict__ heads,
                                                                  int chunk) {
  extern __shared__ uint16_t sort_sm[];
  __shared__ int warp_sums[32];
  const int bins = 1 << bits, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int* base = (int*)(sort_sm + kSortWarps * bins);
  uint32_t* sk = (uint32_t*)(base + max(bins, 32));   // [kSortTile] keys, then positions
  uint32_t* sv = sk + kSortTile;
  grid_dep_wait();
  grid_dep_launch();
  uint32_t key[kSortItems], val[kSortItems], digit[kSortItems];
  bool on[kSortItems];
#pragma unroll
  for (int u = 0; u < kSortItems; ++u) {
    const int i = (warp * kSortItems + u) * 32 + lane;
    on[u] = i < R;
    key[u] = on[u] ? emb_key(ids[i], n_rows) : 0u;
    val[u] = (uint32_t)i;
  }
  for (int p = 0; p < passes; ++p) {
    for (int i = threadIdx.x; i < kSortWarps * bins / 2; i += kSortThreads) ((uint32_t*)sort_sm)[i] = 0;
    for (int i = threadIdx.x; i < bins; i += kSortThreads) base[i] = 0;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kSortItems; ++u) {
      digit[u] = (key[u] >> (p * bits)) & (bins - 1);
      if (on[u]) atomicAdd(&base[digit[u]], 1);
    }
    int rank[kSortItems];
    sort_rank(digit, on, sort_sm, bins, rank);   // its barriers also close the counts
    const int b0 = threadIdx.x * 2;
    const int c0 = b0 < bins ? base[b0] : 0, c1 = b0 + 1 < bins ? base[b0 + 1] : 0;
    int all;
    const int ex = block_exclusive(c0 + c1, warp_sums, all);
    if (b0 < bins) base[b0] = ex;
    if (b0 + 1 < bins) base[b0 + 1] = ex + c0;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kSortItems; ++u)
      if (on[u]) {
        const int to = base[digit[u]] + sort_sm[warp * bins + digit[u]] + rank[u];
        sk[to] = key[u];
        sv[to] = val[u];
      }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kSortItems; ++u) {
      const int i = (warp * kSortItems + u) * 32 + lane;
      if (on[u]) {
        key[u] = sk[i];
        val[u] = sv[i];
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kSortItems; ++u) {
    const int i = (warp * kSortItems + u) * 32 + lane;
    if (on[u]) {
      keys[i] = key[u];
      vals[i] = val[u];
    }
  }
  if (!heads) return;
  // heads[c]: rows that begin in chunk c (chunk is a multiple of 32, and 32
  // consecutive items are one warp's round)
  __syncthreads();   // sk read by every warp
  for (int i = threadIdx.x; i < (R + chunk - 1) / chunk; i += kSortThreads) base[i] = 0;
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kSortItems; ++u) {
    const int i = (warp * kSortItems + u) * 32 + lane;
    const bool head = on[u] && key[u] < n_rows && (i == 0 || sk[i - 1] != key[u]);
    const int n = __popc(__ballot_sync(~0u, head));
    if (lane == 0 && n) atomicAdd(&base[i / chunk], n);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < (R + chunk - 1) / chunk; i += kSortThreads) heads[i] = base[i];
}

// ----------------------------------------------------------------- reduce --
// heads[c]: distinct rows that begin in chunk c of the sorted order.
__global__ void __launch_bounds__(256) emb_heads_kernel(const uint32_t* __restrict__ keys, long long R, uint32_t n_rows,
                                                        int chunk, int* __restrict__ heads) {
  __shared__ int sum;
  if (threadIdx.x == 0) sum = 0;
  grid_dep_wait();
  grid_dep_launch();
  __syncthreads();
  const long long p0 = (long long)blockIdx.x * chunk, p1 = min(R, p0 + chunk);
  int n = 0;
  for (long long p = p0 + threadIdx.x; p < p1; p += 256) {
    const uint32_t k = keys[p];
    n += k < n_rows && (p == 0 || keys[p - 1] != k);
  }
  n = __reduce_add_sync(~0u, n);
  if ((threadIdx.x & 31) == 0 && n) atomicAdd(&sum, n);
  __syncthreads();
  if (threadIdx.x == 0) heads[blockIdx.x] = sum;
}

constexpr int kRedWarps = 8, kRedBatch = 8;

struct ReduceArgs {
  const uint32_t *keys, *vals;   // sorted
  uint32_t n_rows;
  long long R, dout_ld;
  int width, chunk, chunks;      // chunk: sorted positions a CTA, a multiple of 32 * kRedWarps
  float scale;
  float* out;                    // dense: [n_rows][width]; sparse: [..][width]
  void* uniq;                    // sparse: row ids in ascending order
  int* n_uniq;
  const int* heads;              // sparse: heads per chunk
  // runs that cross a chunk's ends, joined by emb_join_kernel
  float *first, *tail;           // [chunks][width]
  int* state;                    // bit 0: a run goes on past the chunk, bit 1: the chunk is all one older run
  long long* tail_row;           // output row of the run that goes on
};
enum { kRunGoesOn = 1, kRunThrough = 2 };

// Sums the sorted rows of one chunk, run by run.  Warp w walks the positions
// [w, w + 1) * chunk / 8 of the chunk, kRedBatch gathered rows in flight, a
// lane holding CPL columns (blockIdx.y picks 32 * CPL of them).  A run inside
// a warp's positions is written at once; parts of runs that cross the warps'
// borders are joined in shared memory, in position order, and parts that
// cross the chunk's borders go to first / tail.  Dense: CTAs past the chunks
// write zeros to the table rows that no id names, found by binary search in
// the sorted ids, so every element of the table is written exactly once.
template <typename T, typename Id, int CPL, bool DENSE>
__global__ void __launch_bounds__(32 * kRedWarps) emb_reduce_kernel(const T* __restrict__ dout, ReduceArgs a) {
  __shared__ float s_first[kRedWarps][32 * CPL], s_last[kRedWarps][32 * CPL];
  __shared__ int s_flags[kRedWarps], s_heads[kRedWarps], s_before;
  __shared__ long long s_row[kRedWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.y * 32 * CPL + lane * CPL;
  grid_dep_wait();
  grid_dep_launch();

  if (DENSE && (int)blockIdx.x >= a.chunks) {
    // 256 table rows a CTA: a row is absent when the first sorted key >= it is another
    __shared__ unsigned s_absent[kRedWarps];
    const long long v0 = (long long)(blockIdx.x - a.chunks) * 256;
    const long long v = v0 + threadIdx.x;
    bool absent = false;
    if (v < a.n_rows) {
      long long lo = 0, hi = a.R;
      while (lo < hi) {
        const long long mid = (lo + hi) >> 1;
        if (a.keys[mid] < (uint32_t)v) lo = mid + 1; else hi = mid;
      }
      absent = lo == a.R || a.keys[lo] != (uint32_t)v;
    }
    const unsigned m = __ballot_sync(~0u, absent);
    if (lane == 0) s_absent[warp] = m;
    __syncthreads();
    if (col >= a.width) return;
    float z[CPL];
#pragma unroll
    for (int e = 0; e < CPL; ++e) z[e] = 0.f;
    for (int i = warp; i < 256; i += kRedWarps)
      if (s_absent[i >> 5] >> (i & 31) & 1) emb_st<CPL>(a.out + (v0 + i) * a.width + col, z);
    return;
  }

  const int wrows = a.chunk / kRedWarps;   // a multiple of 32
  const long long c0 = (long long)blockIdx.x * a.chunk;
  const long long p0 = c0 + (long long)warp * wrows, p1 = min(a.R, p0 + wrows);

  long long urow = 0;   // sparse: output row of the next run that begins here
  if (!DENSE) {
    int n = 0;
    for (long long p = p0 + lane; p < p1; p += 32) {
      const uint32_t k = a.keys[p];
      n += k < a.n_rows && (p == 0 || a.keys[p - 1] != k);
    }
    n = __reduce_add_sync(~0u, n);
    int before = 0, all = 0;
    const bool count_all = blockIdx.x == 0 && blockIdx.y == 0;
    for (int i = threadIdx.x; i < (count_all ? a.chunks : (int)blockIdx.x); i += 32 * kRedWarps) {
      const int h = a.heads[i];
      all += h;
      if (i < (int)blockIdx.x) before += h;
    }
    before = __reduce_add_sync(~0u, count_all ? all : before);
    if (threadIdx.x == 0) s_before = 0;
    __syncthreads();
    if (lane == 0) {
      s_heads[warp] = n;
      if (before) atomicAdd(&s_before, before);   // integers: any order
    }
    __syncthreads();
    if (count_all) {
      if (threadIdx.x == 0) *a.n_uniq = s_before;
    } else {
      urow = s_before;
    }
    for (int w = 0; w < warp; ++w) urow += s_heads[w];
  }

  float acc[CPL];
#pragma unroll
  for (int e = 0; e < CPL; ++e) acc[e] = 0.f;
  uint32_t cur = a.n_rows;          // key of the open run, n_rows: none
  long long cur_row = 0;
  bool older = false;               // the open run began before this warp's positions
  int flags = 0;                    // bit 0: an older run's part in s_first, bit 1: a run goes on after (s_last), bit 2: all one older run
  const bool on = col < a.width;

  auto flush = [&]() {              // the open run ends inside the warp's positions
    if (cur >= a.n_rows) return;
    if (older) {
#pragma unroll
      for (int e = 0; e < CPL; ++e) s_first[warp][lane * CPL + e] = acc[e];
      flags |= 1;
    } else if (on) {
#pragma unroll
      for (int e = 0; e < CPL; ++e) acc[e] *= a.scale;
      emb_st<CPL>(a.out + cur_row * a.width + col, acc);
    }
  };

  for (long long p = p0; p < p1; p += 32) {
    const int n = (int)min(32LL, p1 - p);
    const uint32_t k = lane < n ? a.keys[p + lane] : a.n_rows;
    const uint32_t r = lane < n ? a.vals[p + lane] : 0;
    if (__shfl_sync(~0u, k, 0) >= a.n_rows) break;   // padding only from here on
    if (p == p0 && p0 > 0) {
      const uint32_t prev = a.keys[p0 - 1];
      if (prev == __shfl_sync(~0u, k, 0)) {
        cur = prev;
        older = true;
      }
    }
    for (int i0 = 0; i0 < n; i0 += kRedBatch) {
      float v[kRedBatch][CPL];
#pragma unroll
      for (int i = 0; i < kRedBatch; ++i) {
        const uint32_t ki = __shfl_sync(~0u, k, i0 + i), ri = __shfl_sync(~0u, r, i0 + i);
        if (ki < a.n_rows && on) {
          emb_ld<CPL>(dout + (long long)ri * a.dout_ld + col, v[i]);
        } else {
#pragma unroll
          for (int e = 0; e < CPL; ++e) v[i][e] = 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < kRedBatch; ++i) {
        const uint32_t ki = __shfl_sync(~0u, k, i0 + i);
        if (i0 + i < n && ki != cur) {    // the same for the whole warp
          flush();
          cur = ki;
          older = false;
#pragma unroll
          for (int e = 0; e < CPL; ++e) acc[e] = 0.f;
          if (ki < a.n_rows) {
            cur_row = DENSE ? (long long)ki : urow++;
            if (!DENSE && blockIdx.y == 0 && lane == 0) ((Id*)a.uniq)[cur_row] = (Id)ki;
          }
        }
        if (i0 + i < n) {
#pragma unroll
          for (int e = 0; e < CPL; ++e) acc[e] += v[i][e];
        }
      }
    }
  }
  const bool goes_on = cur < a.n_rows && p1 < a.R && p0 < p1 && a.keys[p1] == cur;
  if (goes_on) {
    if (older) {
#pragma unroll
      for (int e = 0; e < CPL; ++e) s_first[warp][lane * CPL + e] = acc[e];
      flags |= 1 | 4;
    } else {
#pragma unroll
      for (int e = 0; e < CPL; ++e) s_last[warp][lane * CPL + e] = acc[e];
      flags |= 2;
    }
  } else {
    flush();
  }
  if (lane == 0) {
    s_flags[warp] = flags;
    s_row[warp] = cur_row;
  }
  __syncthreads();
  if (warp) return;

  // warp 0 joins the warps' parts in order
  float head[CPL], carry[CPL];
#pragma unroll
  for (int e = 0; e < CPL; ++e) head[e] = carry[e] = 0.f;
  bool open = false, through = true;   // an open run that began in this chunk; the chunk so far is one older run
  long long row = 0;
  for (int w = 0; w < kRedWarps; ++w) {
    const int f = s_flags[w];
    if (f & 1) {
#pragma unroll
      for (int e = 0; e < CPL; ++e) {
        const float x = s_first[w][lane * CPL + e];
        if (open) carry[e] += x; else head[e] += x;
      }
      if (!(f & 4) && open) {
        if (on) {
#pragma unroll
          for (int e = 0; e < CPL; ++e) carry[e] *= a.scale;
          emb_st<CPL>(a.out + row * a.width + col, carry);
        }
        open = false;
      }
    }
    if (!(f & 4)) through = false;
    if (f & 2) {
#pragma unroll
      for (int e = 0; e < CPL; ++e) carry[e] = s_last[w][lane * CPL + e];
      open = true;
      row = s_row[w];
    }
  }
  if (a.chunks > 1) {
    if (on) {
      emb_st<CPL>(a.first + (long long)blockIdx.x * a.width + col, head);
      if (open) emb_st<CPL>(a.tail + (long long)blockIdx.x * a.width + col, carry);
    }
    if (lane == 0 && blockIdx.y == 0) {
      a.state[blockIdx.x] = (open ? kRunGoesOn : 0) | (through ? kRunThrough : 0);
      a.tail_row[blockIdx.x] = row;
    }
  }
}

// A run that goes on past chunk c: its part there, the whole chunks it fills
// and its part of the chunk it ends in, added by warps over strided chunks
// and then in warp order (a fixed order).
template <int CPL>
__global__ void __launch_bounds__(1024) emb_join_kernel(ReduceArgs a) {
  __shared__ float part[32][32 * CPL];
  __shared__ int s_end;
  grid_dep_wait();
  grid_dep_launch();
  const int c = blockIdx.x;
  if (!(a.state[c] & kRunGoesOn)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // the chunk the run ends in: the first one after c that is not all one older run
  int end = c + 1;
  for (;;) {
    if (threadIdx.x == 0) s_end = 0x7fffffff;
    __syncthreads();
    const int i = end + threadIdx.x;
    if (i >= a.chunks - 1 || !(a.state[i] & kRunThrough)) atomicMin(&s_end, min(i, a.chunks - 1));
    __syncthreads();
    const int e = s_end;
    __syncthreads();
    if (e != 0x7fffffff) {
      end = e;
      break;
    }
    end += blockDim.x;
  }
  const int col = blockIdx.y * 32 * CPL + lane * CPL;
  const bool on = col < a.width;
  float acc[CPL];
#pragma unroll
  for (int e = 0; e < CPL; ++e) acc[e] = 0.f;
  if (on) {
#pragma unroll 4
    for (int i = c + 1 + warp; i <= end; i += 32) {
      float v[CPL];
      emb_ld<CPL>(a.first + (long long)i * a.width + col, v);
#pragma unroll
      for (int e = 0; e < CPL; ++e) acc[e] += v[e];
    }
  }
#pragma unroll
  for (int e = 0; e < CPL; ++e) part[warp][lane * CPL + e] = acc[e];
  __syncthreads();
  if (warp || !on) return;
  float s[CPL];
  emb_ld<CPL>(a.tail + (long long)c * a.width + col, s);
  for (int w = 0; w < min(32, end - c); ++w)
#pragma unroll
    for (int e = 0; e < CPL; ++e) s[e] += part[w][lane * CPL + e];
#pragma unroll
  for (int e = 0; e < CPL; ++e) s[e] *= a.scale;
  emb_st<CPL>(a.out + a.tail_row[c] * a.width + col, s);
}

}  // namespace ot
