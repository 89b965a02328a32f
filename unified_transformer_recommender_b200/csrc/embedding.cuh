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
constexpr int kLookThreads = 256;

// N consecutive elements as they are in memory, 16 bytes at most per access.
template <typename T, int N> struct EmbRaw {
  static constexpr int W = N * (int)sizeof(T) / 4;      // words (a lone bf16: half of one)
  uint32_t w[W ? W : 1];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (W == 0) w[0] = *(const unsigned short*)p;
    else if constexpr (W == 1) w[0] = *(const uint32_t*)p;
    else if constexpr (W == 2) { const uint2 q = *(const uint2*)p; w[0] = q.x; w[1] = q.y; }
    else
#pragma unroll
      for (int i = 0; i < W; i += 4) {
        const uint4 q = *(const uint4*)(p + i * 4 / (int)sizeof(T));
        w[i] = q.x; w[i + 1] = q.y; w[i + 2] = q.z; w[i + 3] = q.w;
      }
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
    else return __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
  }
};

// A thread keeps its group of VE columns (cpr of them a row, at most
// kLookThreads; wider rows go over in blocks, blockIdx.y) and walks rows, U at
// a time: U row reads are in flight, as read, and with them the ids of the
// next U rows, so that only the first ids are waited for.  Bound by the reads of
// scattered 128-byte rows: 524288 rows of 64 bf16 in 21 us, 6.4 TB/s of ids,
// rows and output, with every distinct row counted once 4.2 TB/s (one CTA per
// U rows, which waits for ids and rows in turn: 29-34 us).  How U is chosen
// stands at the launch.
template <typename Tt, typename To, typename Id, int VE, int U>
__global__ void __launch_bounds__(kLookThreads) emb_lookup_kernel(const Tt* __restrict__ table, uint32_t n_rows,
                                                                  int width, const Id* __restrict__ ids, long long R,
                                                                  int cpr, float scale, To* __restrict__ out,
                                                                  long long out_ld) {
  const int rpb = kLookThreads / cpr, r = threadIdx.x / cpr;   // rows a CTA looks at together
  const int col = (blockIdx.y * kLookThreads + threadIdx.x - r * cpr) * VE;
  const long long step = (long long)gridDim.x * rpb * U;
  grid_dep_wait();
  grid_dep_launch();
  if (r >= rpb || col >= width) return;
  long long r0 = (long long)blockIdx.x * rpb * U + r;
  Id id[U];
#pragma unroll
  for (int u = 0; u < U; ++u) id[u] = r0 + u * rpb < R ? ids[r0 + u * rpb] : (Id)-1;
  for (; r0 < R; r0 += step) {
    EmbRaw<Tt, VE> v[U];
    unsigned on = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t key = emb_key(id[u], n_rows);
      if (key < n_rows) {
        v[u].load(table + (long long)key * width + col);
        on |= 1u << u;
      }
    }
    const long long next = r0 + step;
#pragma unroll
    for (int u = 0; u < U; ++u) id[u] = next + u * rpb < R ? ids[next + u * rpb] : (Id)-1;
    To* o = out + r0 * out_ld + col;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (r0 + u * rpb < R) {
        float x[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) x[e] = on >> u & 1 ? v[u].get(e) * scale : 0.f;
        emb_st<VE>(o + (long long)u * rpb * out_ld, x);
      }
    }
  }
}

// ------------------------------------------------------------------- sort --
// Stable least-significant-digit radix sort of (key, position).  A CTA takes a
// tile of 512 x ITEMS items; a pass ranks the items of its tile per digit (per
// warp by ballots, then across warps), puts the tile in order in shared memory
// and writes it out behind the same digits of the tiles before, so that
// neighbouring threads mostly write neighbouring places.  The counts of every
// (tile, digit) of a pass are ready when it starts: the first pass's come from
// sort_hist_kernel, a later pass's are added up, as integers, by the pass
// before it while it writes (a destination's tile is known there).
//
// A pass is a chain of latencies (load, ballots, two barriers, scattered
// store) more than work: three passes over 75392 ids of 20 bits (7 bits each,
// 74 tiles) take about 7 us each, 1.2 MB of keys and positions at 0.2 TB/s.
// Every launch of the chain starts under the one before it (programmatic
// dependent launch).  How many items a tile has, and whether its CTA adds up
// the tiles' counts itself, is chosen by the host from R; both sides' times
// are there.
constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32, kSortMinBits = 4, kSortMaxBits = 8;

struct SortArgs {
  uint32_t n_rows;       // keys 0 .. n_rows
  long long R;
  int tile, tiles, bits, shift;   // items a tile; digit = (key >> shift) & (2^bits - 1)
  int scanned;           // hist already holds the tile prefixes, tot the digit totals
  int* hist;             // this pass: [tiles][2^bits]
  int* tot;              // [2^bits]
  int* hist_next;        // the next pass's counts, or null
};

// Exclusive prefix of v over the CTA's threads; every thread calls it.
__device__ inline unsigned long long block_exclusive(unsigned long long v, unsigned long long* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  unsigned long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    unsigned long long s = lane < nw ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(~0u, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
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
  const long long i0 = (long long)blockIdx.x * a.tile;
  for (int u = 0; u < a.tile; u += kSortThreads) {
    const long long i = i0 + u + threadIdx.x;
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
__global__ void __launch_bounds__(1024) sort_scan_kernel(SortArgs a) {
  __shared__ int part[32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, bins = 1 << a.bits;
  const int b = blockIdx.x * 32 + lane;
  const int per = (a.tiles + 31) / 32;
  const int t0 = min(a.tiles, warp * per), t1 = min(a.tiles, t0 + per);
  const bool on = b < bins;
  grid_dep_wait();
  grid_dep_launch();
  int s = 0;
  if (on) {
#pragma unroll 4
    for (int t = t0; t < t1; ++t) s += a.hist[(long long)t * bins + b];
  }
  part[warp][lane] = s;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < 32; ++w) {
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
// (w * ITEMS + u) * 32 + l.
template <int ITEMS>
__device__ inline void sort_rank(const uint32_t* digit, const bool* on, uint16_t* wh, int bits, int* rank) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, bins = 1 << bits;
  uint16_t* mine = wh + warp * bins;
  unsigned same[ITEMS];
#pragma unroll
  for (int u = 0; u < ITEMS; ++u) {   // the lanes with this digit: one ballot per bit
    same[u] = __ballot_sync(~0u, on[u]);
#pragma unroll
    for (int i = 0; i < kSortMaxBits; ++i)
      if (i < bits) {
        const bool one = digit[u] >> i & 1;
        const unsigned v = __ballot_sync(~0u, one);
        same[u] &= one ? v : ~v;
      }
  }
#pragma unroll
  for (int u = 0; u < ITEMS; ++u) {
    const int below = __popc(same[u] & ((1u << lane) - 1));
    int base = 0;
    if (on[u]) base = mine[digit[u]];
    __syncwarp();
    if (on[u] && below == 0) mine[digit[u]] = (uint16_t)(base + __popc(same[u]));
    __syncwarp();
    rank[u] = base + below;
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kSortThreads) {
    int c[kSortWarps], s = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) c[w] = wh[w * bins + b];
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      wh[w * bins + b] = (uint16_t)s;
      s += c[w];
    }
  }
  __syncthreads();
}

// One pass.  FIRST: items are (id, position) from the caller's ids.
template <typename Id, bool FIRST, int ITEMS>
__global__ void __launch_bounds__(kSortThreads) sort_pass_kernel(const Id* __restrict__ ids,
                                                                 const uint32_t* __restrict__ keys_in,
                                                                 const uint32_t* __restrict__ vals_in,
                                                                 uint32_t* __restrict__ keys, uint32_t* __restrict__ vals,
                                                                 SortArgs a, int next_bits, int next_shift) {
  constexpr int TILE = kSortThreads * ITEMS;
  extern __shared__ __align__(16) uint8_t sort_sm[];
  __shared__ unsigned long long warp_sums[32];
  const int bins = 1 << a.bits, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint2* pairs = (uint2*)sort_sm;                       // [TILE] the tile in digit order
  int2* base = (int2*)(pairs + TILE);              // [bins] x: place of the digit's first item minus y, y: its first slot in the tile
  uint16_t* wh = (uint16_t*)(base + bins);              // [kSortWarps][bins]
  for (int i = threadIdx.x; i < kSortWarps * bins / 2; i += kSortThreads) ((uint32_t*)wh)[i] = 0;
  grid_dep_wait();
  grid_dep_launch();
  const long long i0 = (long long)blockIdx.x * TILE;
  const int n = (int)min((long long)TILE, a.R - i0);
  uint32_t key[ITEMS], val[ITEMS], digit[ITEMS];
  bool on[ITEMS];
#pragma unroll
  for (int u = 0; u < ITEMS; ++u) {
    const int j = (warp * ITEMS + u) * 32 + lane;
    on[u] = j < n;
    key[u] = !on[u] ? 0u : FIRST ? emb_key(ids[i0 + j], a.n_rows) : keys_in[i0 + j];
    val[u] = !on[u] ? 0u : FIRST ? (uint32_t)(i0 + j) : vals_in[i0 + j];
  }
  // where the tile's items of each digit begin, in the whole and in the tile:
  // neighbouring threads share a digit and its tiles' counts, 16 in flight each
  static_assert(kSortThreads >= 2 << kSortMaxBits && kSortThreads >> kSortMinBits <= 32, "2 to 32 threads per digit");
  const int tpd = kSortThreads >> a.bits, b = threadIdx.x / tpd, sub = threadIdx.x & (tpd - 1);
  int tot = 0, before = 0, own = 0;
  if (a.scanned) {
    if (sub == 0) {
      tot = a.tot[b];
      before = a.hist[(long long)blockIdx.x * bins + b];
      own = (blockIdx.x + 1 < gridDim.x ? a.hist[(long long)(blockIdx.x + 1) * bins + b] : tot) - before;
    }
  } else {
    for (int t0 = sub; t0 < a.tiles; t0 += 16 * tpd) {
      int c[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) c[i] = t0 + tpd * i < a.tiles ? a.hist[(long long)(t0 + tpd * i) * bins + b] : 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        tot += c[i];
        if (t0 + tpd * i < (int)blockIdx.x) before += c[i];
        if (t0 + tpd * i == (int)blockIdx.x) own += c[i];
      }
    }
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_xor_sync(~0u, before, o);
    if (o < tpd) before += x;
  }
#pragma unroll
  for (int u = 0; u < ITEMS; ++u) digit[u] = (key[u] >> a.shift) & (bins - 1);
  const unsigned long long ex = block_exclusive((unsigned long long)(unsigned)tot | (unsigned long long)own << 32, warp_sums);
  if (sub == 0) {
    const int slot = (int)(ex >> 32);
    base[b] = make_int2((int)(unsigned)ex + before - slot, slot);
  }
  int rank[ITEMS];
  sort_rank<ITEMS>(digit, on, wh, a.bits, rank);
#pragma unroll
  for (int u = 0; u < ITEMS; ++u)
    if (on[u]) pairs[base[digit[u]].y + wh[warp * bins + digit[u]] + rank[u]] = make_uint2(key[u], val[u]);
  __syncthreads();
#pragma unroll
  for (int u = 0; u < ITEMS; ++u) {
    const int j = u * kSortThreads + threadIdx.x;
    int counter = -1;
    if (j < n) {
      const uint2 q = pairs[j];
      const int to = base[(q.x >> a.shift) & (bins - 1)].x + j;
      keys[to] = q.x;
      vals[to] = q.y;
      counter = ((to / TILE) << next_bits) + ((q.x >> next_shift) & ((1 << next_bits) - 1));
    }
    // a popular id sends many lanes to one counter: one add for all of them
    // (adds to the same address queue up)
    if (a.hist_next) {
      const unsigned same = __match_any_sync(~0u, counter);
      if (counter >= 0 && (same & ((1u << lane) - 1)) == 0) atomicAdd(&a.hist_next[counter], __popc(same));
    }
  }
}

// Up to kRankMax ids: every id's place is the number of ids before it (smaller,
// or equal and earlier), counted against all of them in shared memory, four
// ids per warp.  One launch and one barrier where the radix sort takes a chain
// of them; the R^2 comparisons are spread over the GPU.  Whole sparse gradient
// of rows of 64, counted / radix sort: 512 ids 6.9 / 18.5 us, 2048 ids 12-13 /
// 22.1, 4096 ids 18.5 / 21.9; at 5000 the radix sort's 22.3 are ahead.
constexpr int kRankMax = 4096, kRankThreads = 256, kRankIds = 4;
template <typename Id>
__global__ void __launch_bounds__(kRankThreads) sort_rank_kernel(const Id* __restrict__ ids, uint32_t n_rows, int R,
                                                                 uint32_t* __restrict__ keys,
                                                                 uint32_t* __restrict__ vals) {
  __shared__ __align__(16) uint32_t sk[kRankMax];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dep_wait();
  grid_dep_launch();
  const int n4 = (R + 127) & ~127;     // whole rounds of 32 lanes x 4 keys
  for (int i = threadIdx.x; i < n4; i += kRankThreads) sk[i] = i < R ? emb_key(ids[i], n_rows) : 0xffffffffu;
  __syncthreads();
  const int i0 = (blockIdx.x * (kRankThreads / 32) + warp) * kRankIds;
  if (i0 >= R) return;
  uint32_t k[kRankIds];
  int n[kRankIds];
#pragma unroll
  for (int u = 0; u < kRankIds; ++u) {
    k[u] = sk[min(i0 + u, R - 1)];
    n[u] = 0;
  }
  for (int j0 = lane * 4; j0 < n4; j0 += 128) {
    const uint4 q = *(const uint4*)&sk[j0];
#pragma unroll
    for (int u = 0; u < kRankIds; ++u) {   // id j is before id i when key j < key i + (j < i)
      const int i = i0 + u;
      n[u] += (q.x < k[u] + (j0 < i)) + (q.y < k[u] + (j0 + 1 < i)) + (q.z < k[u] + (j0 + 2 < i)) +
              (q.w < k[u] + (j0 + 3 < i));
    }
  }
#pragma unroll
  for (int u = 0; u < kRankIds; ++u) {
    const int to = __reduce_add_sync(~0u, n[u]);
    if (lane == u && i0 + u < R) {
      keys[to] = k[u];
      vals[to] = (uint32_t)(i0 + u);
    }
  }
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

constexpr int kRedWarps = 8, kJoinWarps = 8;

struct ReduceArgs {
  const uint32_t *keys, *vals;   // sorted
  uint32_t n_rows;
  long long R, dout_ld;
  int width, chunk, chunks;      // chunk: sorted positions a CTA, a multiple of kRedWarps
  int fill;                      // dense: CTAs that write the rows no id names
  float scale;
  float* out;                    // dense: [n_rows][width]; sparse: [..][width]
  void* uniq;                    // sparse: row ids in ascending order
  int* n_uniq;
  const int* heads;              // sparse: heads per chunk (null: counted from the keys)
  // runs that cross a chunk's ends, joined by emb_join_kernel
  float *first, *tail;           // [chunks][width]
  int* state;                    // bit 0: a run goes on past the chunk, bit 1: the chunk is all one older run
  long long* tail_row;           // output row of the run that goes on
};
enum { kRunGoesOn = 1, kRunThrough = 2 };

// The first position in the sorted keys with a key >= v, by a warp: 32 probes a
// round.
__device__ inline long long emb_lower_bound(const uint32_t* __restrict__ keys, long long R, uint32_t v) {
  const int lane = threadIdx.x & 31;
  long long lo = 0, hi = R;              // keys[lo - 1] < v <= keys[hi]
  while (hi - lo > 0) {
    const long long step = (hi - lo + 31) >> 5;
    const long long at = min(hi - 1, lo + step * (lane + 1) - 1);
    const unsigned less = __ballot_sync(~0u, keys[at] < v);   // a prefix of the lanes
    const int n = __popc(less);
    if (n == 32) return hi;
    hi = min(hi - 1, lo + step * (n + 1) - 1);
    lo = min(hi, lo + step * n);
  }
  return lo;
}

// Zeros for the 256 table rows from v0 that no id names.  Which ones the sorted
// ids between the rows' bounds say: a short span is walked, each position that
// begins a run marking its row; in a long one (small tables, popular ids) each
// thread searches for its own row, about 20 dependent loads whatever R.  Whole
// dense gradient of 262144 ids, rows of 64, walk / search, us: 1024 ids a span
// 59 / 66, 4096 53 / 57, 8192 57 / 57, 16384 63 / 56, 65536 103 / 55; of 2^22
// ids of 256 rows of 16 (one span) 7600 / 480, the sums alone 450.
constexpr int kFillWalk = 8192;    // ids of a span that is walked
template <int CPL>
__device__ inline void emb_fill_absent(const ReduceArgs& a, long long v0, int col) {
  static_assert(32 * kRedWarps == 256, "a thread per row");
  __shared__ unsigned s_there[kRedWarps];
  __shared__ long long s_span[2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x < kRedWarps) s_there[threadIdx.x] = 0;
  if (warp < 2) {
    const long long p = emb_lower_bound(a.keys, a.R, (uint32_t)min((long long)a.n_rows, v0 + warp * 256));
    if (lane == 0) s_span[warp] = p;
  }
  __syncthreads();
  const long long s0 = s_span[0], s1 = s_span[1];
  if (s1 - s0 <= kFillWalk) {
    for (long long p = s0 + threadIdx.x; p < s1; p += 32 * kRedWarps) {
      const uint32_t k = a.keys[p];
      if (p == s0 || a.keys[p - 1] != k) atomicOr(&s_there[(k - v0) >> 5], 1u << ((k - v0) & 31));
    }
  } else {
    const uint32_t v = (uint32_t)(v0 + threadIdx.x);
    long long lo = s0, hi = s1;          // keys before lo are < v, keys from hi on are not
    while (lo < hi) {
      const long long mid = (lo + hi) >> 1;
      if (a.keys[mid] < v) lo = mid + 1; else hi = mid;
    }
    const unsigned there = __ballot_sync(~0u, lo < s1 && a.keys[lo] == v);
    if (lane == 0) s_there[warp] = there;
  }
  __syncthreads();
  if (col >= a.width) return;
  float z[CPL];
#pragma unroll
  for (int e = 0; e < CPL; ++e) z[e] = 0.f;
  const int n = (int)min(256LL, (long long)a.n_rows - v0);
  for (int i = warp; i < n; i += kRedWarps)
    if (!(s_there[i >> 5] >> (i & 31) & 1)) emb_st<CPL>(a.out + (v0 + i) * a.width + col, z);
}

// Sums the sorted rows of one chunk, run by run.  Warp w walks the positions
// [w, w + 1) * chunk / 8 of the chunk, a batch of gathered rows in flight, a
// lane holding CPL columns (blockIdx.y picks 32 * CPL of them).  A run inside
// a warp's positions is written at once; parts of runs that cross the warps'
// borders are joined in shared memory, in position order, and parts that
// cross the chunk's borders go to first / tail.  Dense: fill CTAs, spread
// between the chunks' so that their searches overlap the sums, write zeros to
// the table rows that no id names, so that every element of the table is
// written exactly once.
// Bound by the scattered reads of dout's rows and, dense, by the table's writes:
// 262147 float32 rows of 128 into a table of 200003 take 51 us (239 MB, 4.7
// TB/s).  Eight to sixteen gathered rows in flight per warp, four CTAs an SM.
template <typename T, typename Id, int CPL, bool DENSE>
__global__ void __launch_bounds__(32 * kRedWarps, CPL <= 2 ? 4 : CPL == 4 ? 3 : 2) emb_reduce_kernel(const T* __restrict__ dout, ReduceArgs a) {
  constexpr int BATCH = CPL == 1 ? 16 : 8;    // gathered rows in flight per warp
  __shared__ __align__(16) float s_first[kRedWarps][32 * CPL], s_last[kRedWarps][32 * CPL];
  __shared__ int s_flags[kRedWarps], s_heads[kRedWarps], s_part[kRedWarps];
  __shared__ long long s_row[kRedWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.y * 32 * CPL + lane * CPL;
  grid_dep_wait();
  grid_dep_launch();
  int cta = blockIdx.x;
  if (DENSE && a.fill) {
    const long long all = (long long)a.chunks + a.fill;
    const int f0 = (int)(cta * (long long)a.fill / all), f1 = (int)((cta + 1LL) * a.fill / all);
    if (f1 > f0) {
      emb_fill_absent<CPL>(a, f0 * 256LL, col);
      return;
    }
    cta -= f0;
  }

  const int wrows = a.chunk / kRedWarps;
  const long long c0 = (long long)cta * a.chunk;
  const long long p0 = c0 + (long long)warp * wrows, p1 = min(a.R, p0 + wrows);
  const bool on = col < a.width, some = p0 < p1;

  // the first 32 positions and the keys on either side of the warp's
  uint32_t k = a.n_rows, r = 0;
  if (p0 + lane < p1) {
    k = a.keys[p0 + lane];
    r = a.vals[p0 + lane];
  }
  const uint32_t prev = some && p0 > 0 ? a.keys[p0 - 1] : a.n_rows;
  const uint32_t next = some && p1 < a.R ? a.keys[p1] : a.n_rows;
  const uint32_t last = some ? a.keys[p1 - 1] : a.n_rows;

  // sparse: heads in the chunks before (all of them at CTA 0, for the count)
  int part = 0;
  const bool count_all = !DENSE && cta == 0 && blockIdx.y == 0;
  if (!DENSE) {
    if (a.heads) {
      for (int i = threadIdx.x; i < (count_all ? a.chunks : cta); i += 32 * kRedWarps) part += a.heads[i];
    } else {
      for (long long p = threadIdx.x; p < (count_all ? a.R : c0); p += 32 * kRedWarps) {
        const uint32_t q = a.keys[p];
        part += q < a.n_rows && (p == 0 || a.keys[p - 1] != q);
      }
    }
  }

  // which of the 32 positions begin a run, and how many are no padding
  auto heads_of = [&](uint32_t before) {
    uint32_t q = __shfl_up_sync(~0u, k, 1);
    if (lane == 0) q = before;
    return __ballot_sync(~0u, k < a.n_rows && k != q);
  };
  unsigned heads = heads_of(prev);
  int n = __popc(__ballot_sync(~0u, k < a.n_rows));
  float v[BATCH][CPL];
  auto load = [&](int i0) {
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const uint32_t ri = __shfl_sync(~0u, r, (i0 + i) & 31);
      if (i0 + i < n && on) emb_ld<CPL>(dout + (long long)ri * a.dout_ld + col, v[i]);
    }
  };
  load(0);     // in flight over the count

  const bool older = some && prev < a.n_rows && !(heads & 1) && n > 0;   // the first run began before
  const bool goes_on = some && last < a.n_rows && next == last;          // the last one goes on after
  Id* uniq = (Id*)a.uniq;
  float* o = a.out + col;        // sparse: where the next run that begins here goes
  long long urow = 0;
  if (!DENSE) {
    int mine = __popc(heads);
    for (long long p = p0 + 32; p < p1; p += 32) {     // only with more than 32 positions a warp
      const uint32_t q = p + lane < p1 ? a.keys[p + lane] : a.n_rows;
      mine += __popc(__ballot_sync(~0u, q < a.n_rows && q != a.keys[p + lane - 1]));
    }
    part = __reduce_add_sync(~0u, part);
    if (lane == 0) {
      s_part[warp] = part;
      s_heads[warp] = mine;
    }
    __syncthreads();
    int before = lane < kRedWarps ? (count_all ? 0 : s_part[lane]) + (lane < warp ? s_heads[lane] : 0) : 0;
    urow = __reduce_add_sync(~0u, before);
    if (count_all && warp == 0) {
      const int all = __reduce_add_sync(~0u, lane < kRedWarps ? s_part[lane] : 0);
      if (lane == 0) *a.n_uniq = all;
    }
    o += urow * a.width;
  }

  float acc[CPL];
#pragma unroll
  for (int e = 0; e < CPL; ++e) acc[e] = 0.f;
  // the open run's sum goes to dst: its output row, times the scale, or (part_of)
  // shared memory, for a piece of a run that crosses the warp's border
  float* dst = older ? &s_first[warp][lane * CPL] : nullptr;
  bool part_of = older;
  bool open = older, begun = false;      // begun: a run began here
  long long row = 0;                     // output row of the run that began here last
  auto flush = [&]() {
    if (open && (on || part_of)) {       // lanes past the width own no output
      float w[CPL];
#pragma unroll
      for (int e = 0; e < CPL; ++e) w[e] = part_of ? acc[e] : acc[e] * a.scale;
#pragma unroll
      for (int e = 0; e < CPL; ++e) acc[e] = 0.f;
      emb_st<CPL>(dst, w);
    }
  };

  for (long long p = p0; n > 0; ) {
    if (!DENSE) {
      if (blockIdx.y == 0 && (heads >> lane & 1)) uniq[urow + __popc(heads & ((1u << lane) - 1))] = (Id)k;
    }
    for (int i0 = 0; i0 < n; i0 += BATCH) {
      if (i0 > 0 || p > p0) load(i0);
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        if (i0 + i < n) {                       // the same for the whole warp, as every branch here
          if (heads >> (i0 + i) & 1) {
            flush();
            if (DENSE) {
              row = __shfl_sync(~0u, k, i0 + i);
              dst = a.out + row * a.width + col;
            } else {
              dst = o;
              o += a.width;
              row = urow++;
            }
            part_of = false;
            open = begun = true;
          }
          if (on) {
#pragma unroll
            for (int e = 0; e < CPL; ++e) acc[e] += v[i][e];
          }
        }
      }
    }
    p += 32;
    if (p >= p1 || n < 32) break;
    const uint32_t before = __shfl_sync(~0u, k, 31);
    k = p + lane < p1 ? a.keys[p + lane] : a.n_rows;
    r = p + lane < p1 ? a.vals[p + lane] : 0;
    heads = heads_of(before);
    n = __popc(__ballot_sync(~0u, k < a.n_rows));
  }
  if (goes_on) {
    dst = begun ? &s_last[warp][lane * CPL] : &s_first[warp][lane * CPL];
    part_of = true;
  }
  flush();
  if (lane == 0) {
    // bit 0: an older run's part in s_first, bit 1: a run goes on after
    // (s_last), bit 2: all one older run
    s_flags[warp] = (older ? 1 : 0) | (goes_on && begun ? 2 : 0) | (goes_on && !begun ? 4 : 0);
    s_row[warp] = row;
  }
  __syncthreads();
  if (warp) return;

  // warp 0 joins the warps' parts in order
  const int flags = lane < kRedWarps ? s_flags[lane] : 0;
  if (!__any_sync(~0u, flags)) {         // no run crosses a border
    if (a.chunks > 1 && lane == 0 && blockIdx.y == 0) a.state[cta] = 0;
    return;
  }
  float head[CPL], carry[CPL];
#pragma unroll
  for (int e = 0; e < CPL; ++e) head[e] = carry[e] = 0.f;
  bool open_run = false, through = true;   // an open run that began in this chunk; the chunk so far is one older run
  long long at = 0;
  for (int w = 0; w < kRedWarps; ++w) {
    const int f = __shfl_sync(~0u, flags, w);
    if (f & 1) {
#pragma unroll
      for (int e = 0; e < CPL; ++e) {
        const float x = s_first[w][lane * CPL + e];
        if (open_run) carry[e] += x; else head[e] += x;
      }
      if (!(f & 4) && open_run) {
        if (on) {
#pragma unroll
          for (int e = 0; e < CPL; ++e) carry[e] *= a.scale;
          emb_st<CPL>(a.out + at * a.width + col, carry);
        }
        open_run = false;
      }
    }
    if (!(f & 4)) through = false;
    if (f & 2) {
#pragma unroll
      for (int e = 0; e < CPL; ++e) carry[e] = s_last[w][lane * CPL + e];
      open_run = true;
      at = s_row[w];
    }
  }
  if (a.chunks > 1) {
    if (on) {
      emb_st<CPL>(a.first + (long long)cta * a.width + col, head);
      if (open_run) emb_st<CPL>(a.tail + (long long)cta * a.width + col, carry);
    }
    if (lane == 0 && blockIdx.y == 0) {
      a.state[cta] = (open_run ? kRunGoesOn : 0) | (through ? kRunThrough : 0);
      a.tail_row[cta] = at;
    }
  }
}

// A run that goes on past chunk c: its part there, the whole chunks it fills
// and its part of the chunk it ends in, added by warps over strided chunks
// and then in warp order (a fixed order).  Most CTAs find no such run and end:
// 6 us for 2049 chunks, launch and one dependent load.
template <int CPL>
__global__ void __launch_bounds__(32 * kJoinWarps) emb_join_kernel(ReduceArgs a) {
  __shared__ float part[kJoinWarps][32 * CPL];
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
    for (int i = c + 1 + warp; i <= end; i += kJoinWarps) {
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
  for (int w = 0; w < min(kJoinWarps, end - c); ++w)
#pragma unroll
    for (int e = 0; e < CPL; ++e) s[e] += part[w][lane * CPL + e];
#pragma unroll
  for (int e = 0; e < CPL; ++e) s[e] *= a.scale;
  emb_st<CPL>(a.out + a.tail_row[c] * a.width + col, s);
}

}  // namespace ot
