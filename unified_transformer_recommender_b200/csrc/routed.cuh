// Routed event tokenizer: events sorted by behaviour, each through its
// behaviour's MLP, weighted and put back, with its gradient.  Event r has k
// choices (t, w) = (types[r][j], weights[r][j]):
//
//   u = W1_t e + b1_t,  z = GELU(u),  y = W2_t z + b2_t + emb_t
//   token[r] = sum_j w y                              (t = -1: no term)
//
//   dz = W2_t^T dtoken[r],  dw = <dz, z> + <dtoken[r], b2_t + emb_t>
//   du = w dz GELU'(u),     de[r] = sum_j W1_t^T du
//   dW2_t = sum w dtoken z^T, db2_t = demb_t = sum w dtoken,
//   dW1_t = sum du e^T,       db1_t = sum du
//
// The plan sorts the R * k choices by behaviour, stably, into slots; each
// behaviour's slots start at a multiple of 128, so that a 128-row tile belongs
// to one behaviour.  Slots between a behaviour's last choice and the next
// multiple of 128 are padding (order = -1).
//
// This file: the plan, the CUDA-core kernels (float32 mode, and shapes the
// tensor-core kernels do not take) and the passes both sets share.
#pragma once
#include "embedding.cuh"

namespace ot {

constexpr int kMaxTypes = 8, kMaxChoices = 8;
constexpr int kPlanMagic = 0x6f74726e, kPlanHeader = 64;   // ints

// Plan: int32 header (magic, R, k, T, cnt[8] from 8, first slot[9] from 16),
// order[n_cap] (choice index r * k + j of each slot, -1 padding) and pos[R*k]
// (slot of each choice, -1: none).
struct PlanView {
  const int* head;
  const int* order;
  const int* pos;
  int R, k, T;
};
__device__ inline int plan_count(const PlanView& p, int t) { return p.head[8 + t]; }
__device__ inline int plan_first(const PlanView& p, int t) { return p.head[16 + t]; }

// A plan made for other sizes (or never made) is refused, with the device
// status word set, before anything is read through it.
__device__ inline bool plan_ok(const PlanView& p) {
  const bool ok = p.head[0] == kPlanMagic && p.head[1] == p.R && p.head[2] == p.k && p.head[3] == p.T;
  if (!ok && threadIdx.x == 0) flag_error(3);
  return ok;
}
// Behaviour of a slot below plan_first(T).
__device__ inline int plan_type(const PlanView& p, int slot) {
  int t = 0;
  while (t + 1 < p.T && slot >= plan_first(p, t + 1)) ++t;
  return t;
}

struct RoutedMLP {
  const void *W1[kMaxTypes], *b1[kMaxTypes], *W2[kMaxTypes], *b2[kMaxTypes];
  const void* emb;
};

// Token rows: row r at (r / per) * sample_ld + (r % per) * d (elements).
struct TokenRows {
  int per;
  long long sample_ld;
};
__device__ inline long long token_off(const TokenRows& t, int r, int d) {
  const int b = r / t.per;
  return (long long)b * t.sample_ld + (long long)(r - b * t.per) * d;
}

// ------------------------------------------------------------------- plan --
constexpr int kRouteThreads = 256, kRouteItems = 4, kRouteTile = kRouteThreads * kRouteItems;

__device__ inline int route_type(const int* types, int i, int n, int T) {
  if (i >= n) return -1;
  const int t = types[i];
  if (t >= 0 && t < T) return t;
  if (t != -1) flag_error(3);
  return -1;
}

// counts[tile][8]: choices of each behaviour in the tile.  Both plan kernels
// are a launch and a few dependent loads: 75392 choices in 5.7 us together.
__global__ void __launch_bounds__(kRouteThreads) route_count_kernel(const int* __restrict__ types, int n, int T,
                                                                    int* __restrict__ counts) {
  __shared__ int c[kMaxTypes];
  if (threadIdx.x < kMaxTypes) c[threadIdx.x] = 0;
  grid_dep_wait();
  grid_dep_launch();
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kRouteItems; ++u) {
    const int i = blockIdx.x * kRouteTile + u * kRouteThreads + threadIdx.x;
    const int t = route_type(types, i, n, T);
    const unsigned same = __match_any_sync(~0u, t);
    if (t >= 0 && (same & ((1u << (threadIdx.x & 31)) - 1)) == 0) atomicAdd(&c[t], __popc(same));
  }
  __syncthreads();
  if (threadIdx.x < kMaxTypes) counts[blockIdx.x * kMaxTypes + threadIdx.x] = c[threadIdx.x];
}

// Places the tile's choices behind those of the same behaviour in the tiles
// before.  With one tile it counts by itself (counts is not read); with many
// (tot not null) counts holds the prefixes over the tiles already and tot the
// behaviours' totals, else each CTA adds up all tiles' counts.
__global__ void __launch_bounds__(kRouteThreads) route_place_kernel(const int* __restrict__ types, int n, int R, int k,
                                                                    int T, const int* __restrict__ counts,
                                                                    const int* __restrict__ tot,
                                                                    int* __restrict__ plan, int* __restrict__ order,
                                                                    int* __restrict__ pos) {
  constexpr int NW = kRouteThreads / 32;
  __shared__ int s_all[kMaxTypes], s_before[kMaxTypes], s_first[kMaxTypes + 1];
  __shared__ int s_warp[NW][kMaxTypes];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned lower = (1u << lane) - 1;
  if (threadIdx.x < kMaxTypes) s_all[threadIdx.x] = s_before[threadIdx.x] = 0;
  if (threadIdx.x < NW * kMaxTypes) ((int*)s_warp)[threadIdx.x] = 0;
  grid_dep_wait();
  grid_dep_launch();
  __syncthreads();
  // warp w takes kRouteItems * 32 consecutive choices
  int ty[kRouteItems], rank[kRouteItems];
  const int i0 = blockIdx.x * kRouteTile + warp * kRouteItems * 32 + lane;
#pragma unroll
  for (int u = 0; u < kRouteItems; ++u) ty[u] = route_type(types, i0 + u * 32, n, T);
  if (tot) {
    if (threadIdx.x < kMaxTypes) {
      s_all[threadIdx.x] = tot[threadIdx.x];
      s_before[threadIdx.x] = counts[blockIdx.x * kMaxTypes + threadIdx.x];
    }
  } else if (gridDim.x > 1) {
    int all = 0, before = 0;   // thread i always meets behaviour i % 8
#pragma unroll 4
    for (int i = threadIdx.x; i < (int)gridDim.x * kMaxTypes; i += kRouteThreads) {
      const int c = counts[i];
      all += c;
      if (i / kMaxTypes < (int)blockIdx.x) before += c;
    }
    static_assert(kRouteThreads % kMaxTypes == 0, "a thread's counts are all of one behaviour");
    if (all) atomicAdd(&s_all[threadIdx.x % kMaxTypes], all);
    if (before) atomicAdd(&s_before[threadIdx.x % kMaxTypes], before);
  }
#pragma unroll
  for (int u = 0; u < kRouteItems; ++u) {
    const unsigned same = __match_any_sync(~0u, ty[u]);
    rank[u] = ty[u] >= 0 ? s_warp[warp][ty[u]] + __popc(same & lower) : 0;
    __syncwarp();
    if (ty[u] >= 0 && (same & lower) == 0) s_warp[warp][ty[u]] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  if (threadIdx.x < kMaxTypes) {
    int s = 0;
    for (int w = 0; w < NW; ++w) {
      const int c = s_warp[w][threadIdx.x];
      s_warp[w][threadIdx.x] = s;
      s += c;
    }
    if (gridDim.x == 1) s_all[threadIdx.x] = s;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int at = 0;
    for (int t = 0; t < T; ++t) {
      s_first[t] = at;
      at += (s_all[t] + 127) & ~127;
    }
    for (int t = T; t <= kMaxTypes; ++t) s_first[t] = at;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kRouteItems; ++u) {
    const int i = i0 + u * 32;
    if (i >= n) continue;
    int slot = -1;
    if (ty[u] >= 0) {
      slot = s_first[ty[u]] + s_before[ty[u]] + s_warp[warp][ty[u]] + rank[u];
      order[slot] = i;
    }
    pos[i] = slot;
  }
  if (blockIdx.x == 0) {
    for (int t = 0; t < T; ++t)   // the padding behind each behaviour's choices
      for (int s = s_first[t] + s_all[t] + threadIdx.x; s < s_first[t + 1]; s += kRouteThreads) order[s] = -1;
    if (threadIdx.x < kMaxTypes) plan[8 + threadIdx.x] = s_all[threadIdx.x];
    if (threadIdx.x <= kMaxTypes) plan[16 + threadIdx.x] = s_first[threadIdx.x];
    if (threadIdx.x == 0) {
      plan[0] = kPlanMagic;
      plan[1] = R;
      plan[2] = k;
      plan[3] = T;
    }
  }
}

// ----------------------------------------------------- CUDA-core products --
// GELU-tanh and its slope in float32 (accurate tanh).  u^2 is bounded in the
// slope: past |u| = 16 its factor 1 - th^2 is 0, and inf * 0 would follow.
__device__ inline void gelu_and_slope(float u, float& z, float& g) {
  const float c = 0.7978845608028654f, a = 0.044715f;
  const float th = tanhf(c * (u + a * u * u * u));
  z = 0.5f * u * (1.f + th);
  g = 0.5f * (1.f + th) + 0.5f * u * (1.f - th * th) * c * (1.f + 3.f * a * fminf(u * u, 256.f));
}

// An upstream gradient as a matrix operand: of the mode's type, also where the
// caller's is float32 (the same value on the tensor cores and here).
template <typename T, typename Td> __device__ inline float operand(Td v) { return to_f(from_f<T>(to_f(v))); }

// What one product of the CUDA-core path contracts and does with its result.
enum RoutedStep : int {
  RS_HIDDEN,      // u = e W1^T + b1: z -> buf0
  RS_TOKEN,       // y = z W2^T + b2 + emb, times w -> token rows (k = 1) or part[choice]
  RS_DU,          // u = e W1^T + b1 and dz = dtoken W2: w z -> buf0, w dz GELU'(u) -> buf1, <dz, z> over 64 columns -> dot
  RS_DEVENT       // de = du W1 -> event rows (k = 1) or part[choice]
};

struct RoutedArgs {
  PlanView plan;
  RoutedMLP mlp;
  int e, d;
  const void* events;
  const float* weights;        // [R*k] or null
  void* tokens;                // RS_TOKEN, k = 1
  const void* dtokens;         // RS_DU
  TokenRows rows;
  void* devents;               // RS_DEVENT, k = 1
  float *buf0, *buf1;          // [slots][d]
  float* part;                 // [R*k][d or e], k > 1
  float* dot;                  // [slots][d / 64 rounded up]
};

// 64 slots x 64 columns per CTA, 4 x 4 results per thread of a group of 256;
// the contraction goes in blocks of 32, the next block loaded into registers
// during this one's sums.  RS_DU runs two products one after the other.  T: the
// mode's type, Td: the type of dtokens.
// Float32 sums on the CUDA cores bound it at many events.  With fewer than two
// CTAs an SM a block of the contraction is a chain of latencies (load, store,
// barrier, sums); two groups (GROUPS) then take the blocks in turn and add up
// at the end, each for half of the rows.  Whole gradient (d 256, e 64), one /
// two groups: 1178 events 85 / 69 us, 10000 events 218 / 232, 75392 events
// 1217 / 1416.
constexpr int kSimtK = 32;
typedef float SimtTile[kSimtK][68];

// Four neighbouring elements p[0 .. 3], those past n zero; vec: 4-element
// accesses are aligned (and n a multiple of 4).
template <typename T>
__device__ inline void load_four(const T* p, int n, bool vec, float* v) {
  if (vec) {
    if (n > 0) {
      if constexpr (sizeof(T) == 4) {
        const float4 q = *(const float4*)p;
        v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
      } else {
        const uint2 q = *(const uint2*)p;
        v[0] = __uint_as_float(q.x << 16); v[1] = __uint_as_float(q.x & 0xffff0000u);
        v[2] = __uint_as_float(q.y << 16); v[3] = __uint_as_float(q.y & 0xffff0000u);
      }
    } else {
      v[0] = v[1] = v[2] = v[3] = 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < n ? to_f(p[i]) : 0.f;
  }
}

// acc += A B over the contraction K: A rows arow (null: zero), B K-major
// (b + n * K) or not (b + k * N).
template <int GROUPS, typename Ta, typename Tb, bool B_KMAJOR, typename Round>
__device__ inline void simt_product(SimtTile* tiles, float (*acc)[4], const Ta* arow, const Tb* b, int K, int N, int n0,
                                    bool vec, Round round) {
  const int tid = threadIdx.x & 255, group = GROUPS == 2 ? threadIdx.x >> 8 : 0;
  const int ar = tid >> 2, ak = (tid & 3) * 4;
  const int ty = tid >> 4, tx = tid & 15;
  SimtTile &As = tiles[group * 2], &Bs = tiles[group * 2 + 1];
  auto group_sync = [&]() { asm volatile("bar.sync %0, 256;" ::"r"(group + 1) : "memory"); };
  float av[2][4], bv[2][4];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int kk = k0 + h * 16 + ak;
      load_four(arow + kk, arow ? K - kk : 0, vec, av[h]);
      if constexpr (B_KMAJOR) {           // n = ar, contraction = kk
        load_four(b + (long long)(n0 + ar) * K + kk, n0 + ar < N ? K - kk : 0, vec, bv[h]);
      } else {                            // contraction = ty, n = tx * 4
        const int kb = k0 + h * 16 + ty, n = n0 + tx * 4;
        load_four(b + (long long)kb * N + n, kb < K ? N - n : 0, vec, bv[h]);
      }
    }
  };
  fetch(group * kSimtK);
  for (int k0 = group * kSimtK; k0 < K; k0 += GROUPS * kSimtK) {
    group_sync();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 4; ++i) As[h * 16 + ak + i][ar] = round(av[h][i]);
      if constexpr (B_KMAJOR) {
#pragma unroll
        for (int i = 0; i < 4; ++i) Bs[h * 16 + ak + i][ar] = bv[h][i];
      } else {
        *(float4*)&Bs[h * 16 + ty][tx * 4] = make_float4(bv[h][0], bv[h][1], bv[h][2], bv[h][3]);
      }
    }
    group_sync();
    fetch(k0 + GROUPS * kSimtK);          // past K: zeros, no access
#pragma unroll 8
    for (int kk = 0; kk < kSimtK; ++kk) {
      const float4 x = *(const float4*)&As[kk][ty * 4], w = *(const float4*)&Bs[kk][tx * 4];
      const float xs[4] = {x.x, x.y, x.z, x.w}, wsv[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xs[i], wsv[j], acc[i][j]);
    }
  }
}

// The two groups' sums of the thread's results, in acc[0] and acc[1]: rows 0
// and 1 of them in group 0, rows 2 and 3 in group 1.  `to`: 2 x 8 x 256 floats
// of shared memory.
__device__ inline void simt_join(float* to, float (*acc)[4]) {
  const int tid = threadIdx.x & 255, group = threadIdx.x >> 8;
  float* mine = to + group * 2048 + tid;
  const float* other = to + (group ^ 1) * 2048 + tid;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) mine[(i * 4 + j) * 256] = group ? acc[i][j] : acc[2 + i][j];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = (group ? acc[2 + i][j] : acc[i][j]) + other[(i * 4 + j) * 256];
}

template <typename T, typename Td, int STEP, int GROUPS>
__global__ void __launch_bounds__(256 * GROUPS) routed_simt_kernel(RoutedArgs a) {
  __shared__ __align__(16) SimtTile tiles[2 * GROUPS];
  __shared__ int s_flat[64];
  grid_dep_wait();
  grid_dep_launch();
  if (!plan_ok(a.plan)) return;
  // column blocks of a slot tile are neighbours (they share its rows)
  const int N = STEP == RS_DEVENT ? a.e : a.d, blocks = (N + 63) / 64;
  const int s0 = blockIdx.x / blocks * 64, block = blockIdx.x % blocks, n0 = block * 64;
  if (s0 >= plan_first(a.plan, a.plan.T)) return;
  const int t = plan_type(a.plan, s0);
  // a tile of padding only has nothing to store but the zeros of the backward's buffers
  if (STEP != RS_DU && s0 >= plan_first(a.plan, t) + plan_count(a.plan, t)) return;
  if (threadIdx.x < 64) s_flat[threadIdx.x] = a.plan.order[s0 + threadIdx.x];
  __syncthreads();
  const int k = a.plan.k;
  constexpr int ROWS = 4 / GROUPS;               // result rows a thread finishes
  const int tid = threadIdx.x & 255, group = GROUPS == 2 ? threadIdx.x >> 8 : 0;
  const int ar = tid >> 2, aflat = s_flat[ar];
  const T* W1 = (const T*)a.mlp.W1[t];
  const T* W2 = (const T*)a.mlp.W2[t];
  const int ty = tid >> 4, tx = tid & 15;
  const bool vec = a.e % 4 == 0 && a.d % 4 == 0 && a.rows.sample_ld % 4 == 0;
  auto same = [](float x) { return x; };
  float acc[4][4] = {}, u[STEP == RS_DU ? 4 : 1][4] = {};
  const T* erow = aflat >= 0 ? (const T*)a.events + (long long)(aflat / k) * a.e : nullptr;
  const float* r0 = a.buf0 + (long long)(s0 + ar) * a.d;
  const float* r1 = a.buf1 + (long long)(s0 + ar) * a.d;
  if constexpr (STEP == RS_HIDDEN) {
    simt_product<GROUPS, T, T, true>(tiles, acc, erow, W1, a.e, N, n0, vec, same);
  } else if constexpr (STEP == RS_TOKEN) {
    simt_product<GROUPS, float, T, true>(tiles, acc, aflat >= 0 ? r0 : nullptr, W2, a.d, N, n0, vec, same);
  } else if constexpr (STEP == RS_DEVENT) {
    simt_product<GROUPS, float, T, false>(tiles, acc, aflat >= 0 ? r1 : nullptr, W1, a.d, N, n0, vec, same);
  } else {
    const Td* yrow = aflat >= 0 ? (const Td*)a.dtokens + token_off(a.rows, aflat / k, a.d) : nullptr;
    simt_product<GROUPS, T, T, true>(tiles, u, erow, W1, a.e, N, n0, vec, same);
    simt_product<GROUPS, Td, T, false>(tiles, acc, yrow, W2, a.d, N, n0, vec, [](float x) { return to_f(from_f<T>(x)); });
  }
  if constexpr (GROUPS == 2) {
    static_assert(sizeof(tiles) >= 2 * 4096 * sizeof(float), "room for both products' sums");
    __syncthreads();
    simt_join((float*)tiles, acc);
    if constexpr (STEP == RS_DU) simt_join((float*)tiles + 4096, u);
  }
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int row = ty * 4 + group * ROWS + i, flat = s_flat[row];
    const long long slot = s0 + row;
    const float w = flat < 0 ? 0.f : a.weights ? a.weights[flat] : 1.f;
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx * 4 + j;
      if (n >= N) continue;
      const float v = acc[i][j];
      if constexpr (STEP == RS_HIDDEN) {
        float z, g;
        gelu_and_slope(v + to_f(((const T*)a.mlp.b1[t])[n]), z, g);
        a.buf0[slot * a.d + n] = flat < 0 ? 0.f : z;
      } else if constexpr (STEP == RS_DU) {
        float z = 0.f, g = 0.f;
        if (flat >= 0) gelu_and_slope(u[i][j] + to_f(((const T*)a.mlp.b1[t])[n]), z, g);
        dot = fmaf(v, z, dot);
        a.buf0[slot * a.d + n] = flat < 0 ? 0.f : w * z;
        a.buf1[slot * a.d + n] = flat < 0 ? 0.f : w * v * g;
      } else if (flat >= 0) {
        if constexpr (STEP == RS_TOKEN) {
          const float y = v + (to_f(((const T*)a.mlp.b2[t])[n]) + to_f(((const T*)a.mlp.emb)[(long long)t * a.d + n]));
          if (k == 1) ((T*)a.tokens)[token_off(a.rows, flat, a.d) + n] = from_f<T>(w * y);
          else a.part[(long long)flat * a.d + n] = w * y;
        } else {
          if (k == 1) ((T*)a.devents)[(long long)flat * a.e + n] = from_f<T>(v);
          else a.part[(long long)flat * a.e + n] = v;
        }
      }
    }
    if constexpr (STEP == RS_DU) {
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) dot += __shfl_xor_sync(~0u, dot, o);   // the row's 16 lanes
      if (tx == 0) a.dot[slot * blocks + block] = dot;
    }
  }
}

// ---------------------------------------------------------- shared passes --
// out[r] = sum over the choices of part[r * k + j] (choices that are none
// left out), rounded once.  k = 1: the products wrote the rows themselves,
// and only rows without a behaviour are zeroed here.  A thread takes V
// neighbouring columns of a row, four choices in flight.  Bound by reading
// part: 20011 x 2 choices of 384 columns 14.5 us, 77 MB at 5.3 TB/s.
template <typename T, int V>
__global__ void __launch_bounds__(256) routed_combine_kernel(PlanView plan, const float* __restrict__ part, int width,
                                                             T* __restrict__ out, TokenRows rows) {
  grid_dep_wait();
  grid_dep_launch();
  if (!plan_ok(plan)) return;
  const int per = width / V;
  const long long items = (long long)plan.R * per;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < items; i += (long long)gridDim.x * 256) {
    const int r = i <= 0x7fffffff ? (int)i / per : (int)(i / per), c = (int)(i - (long long)r * per) * V;
    T* o = out + token_off(rows, r, width) + c;
    float s[V];
#pragma unroll
    for (int e = 0; e < V; ++e) s[e] = 0.f;
    if (plan.k == 1) {
      if (plan.pos[r] >= 0) continue;
    } else {
      for (int j0 = 0; j0 < plan.k; j0 += 4) {      // four choices in flight
        float v[4][V];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const long long f = (long long)r * plan.k + j0 + j;
          if (j0 + j < plan.k && plan.pos[f] >= 0) {
            const float* p = part + f * width + c;
            if constexpr (V == 1) v[j][0] = *p;
            else
#pragma unroll
              for (int e = 0; e < V; e += 4) {
                const float4 q = *(const float4*)(p + e);
                v[j][e] = q.x; v[j][e + 1] = q.y; v[j][e + 2] = q.z; v[j][e + 3] = q.w;
              }
          } else {
#pragma unroll
            for (int e = 0; e < V; ++e) v[j][e] = 0.f;
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < V; ++e) s[e] += v[j][e];
      }
    }
    if constexpr (V == 8 && sizeof(T) == 2) {
      *(uint4*)o = make_uint4(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]), pack_bf16x2(s[4], s[5]),
                              pack_bf16x2(s[6], s[7]));
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = from_f<T>(s[e]);
    }
  }
}

// dweights[choice] = <dz, z> (in `parts` partial dots) + <dtoken, b2 + emb>;
// 0 for a choice that is none.  One warp per choice: a chain of latencies
// (place, behaviour, row), so the row is read eight columns a lane.
template <typename T, typename Td>
__global__ void __launch_bounds__(256) routed_dweight_kernel(PlanView plan, RoutedMLP mlp, int d,
                                                             const Td* __restrict__ dtokens, TokenRows rows,
                                                             const float* __restrict__ dot, int parts,
                                                             float* __restrict__ dweights) {
  grid_dep_wait();
  grid_dep_launch();
  if (!plan_ok(plan)) return;
  const int lane = threadIdx.x & 31, n = plan.R * plan.k;
  const bool vec = d % 8 == 0 && rows.sample_ld % 8 == 0;
  int first[kMaxTypes - 1];      // where behaviours 1, 2, .. begin (all slots before those past the last)
#pragma unroll
  for (int i = 0; i < kMaxTypes - 1; ++i) first[i] = plan_first(plan, i + 1);
  for (long long c = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); c < n; c += (long long)gridDim.x * 8) {
    const int slot = plan.pos[c];
    float s = 0.f;
    if (slot >= 0) {
      int t = 0;
#pragma unroll
      for (int i = 0; i < kMaxTypes - 1; ++i) t += slot >= first[i];
      const Td* dy = dtokens + token_off(rows, (int)c / plan.k, d);
      const T *b2 = (const T*)mlp.b2[t], *emb = (const T*)mlp.emb + (long long)t * d;
      if (vec) {
#pragma unroll 2
        for (int i = lane * 8; i < d; i += 256) {
          float y[8], b[8], m[8];
          emb_ld<8>(dy + i, y);
          emb_ld<8>(b2 + i, b);
          emb_ld<8>(emb + i, m);
#pragma unroll
          for (int n = 0; n < 8; ++n) s = fmaf(y[n], b[n] + m[n], s);
        }
      } else {
        for (int i = lane; i < d; i += 32) s = fmaf(to_f(dy[i]), to_f(b2[i]) + to_f(emb[i]), s);
      }
      for (int i = lane; i < parts; i += 32) s += dot[(long long)slot * parts + i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    if (lane == 0) dweights[c] = s;
  }
}

// ------------------------------------------------------- weight gradients --
// The 128-row tiles are cut into slices of `per` tiles; the part of a
// behaviour t in slice s is piece s + t (two pieces never share a number:
// along the tiles, s or t grows).  Each piece holds its own partial
// gradients; the sum over a behaviour's pieces follows in slice order.
struct WeightPieces {
  int per, slices;
  float* part;           // [slices + T - 1][stride]
  long long stride;      // floats of one piece: a weight gradient, then its bias's
};
__device__ inline float* piece_at(const WeightPieces& w, int s, int t) { return w.part + (long long)(s + t) * w.stride; }

// CUDA-core partial gradients: 64 x 64 of dW2 (blockIdx.x below n2) or dW1,
// one slice, behaviour after behaviour.  The CTAs of the first column block
// also add up db2 (dW2) or db1 (dW1) of their 64 rows.  16 slots a step, the
// next step's rows and the choices of the one after in flight: 1178 events (d
// 256, e 64) 19 us, a chain of eight such steps.
template <typename T, typename Td>
__global__ void __launch_bounds__(256) routed_wgrad_simt_kernel(RoutedArgs a, WeightPieces w1, WeightPieces w2,
                                                                int n2) {
  __shared__ __align__(16) float As[16][68], Bs[16][68];
  grid_dep_wait();
  grid_dep_launch();
  if (!plan_ok(a.plan)) return;
  const bool second = (int)blockIdx.x < n2;      // dW2
  const int blk = second ? blockIdx.x : blockIdx.x - n2;
  const int cols = second ? a.d : a.e, ncol = (cols + 63) / 64;
  const int m0 = (blk / ncol) * 64, c0 = (blk % ncol) * 64;
  const int k = a.plan.k;
  const int lr = threadIdx.x >> 4, lc = (threadIdx.x & 15) * 4;   // slot, 4 columns
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const WeightPieces& w = second ? w2 : w1;
  const int tile0 = blockIdx.y * w.per, tile1 = min(tile0 + w.per, plan_first(a.plan, a.plan.T) / 128);
  for (int t = 0; t < a.plan.T; ++t) {
    const int first = plan_first(a.plan, t);
    const int lo = max(tile0 * 128, first), hi = min(tile1 * 128, first + plan_count(a.plan, t));
    const int end = min(tile1 * 128, plan_first(a.plan, t + 1));
    if (lo >= end) continue;
    float acc[4][4] = {}, colsum = 0.f, av[4], bv[4], wt;
    int ahead = lo + lr < hi ? a.plan.order[lo + lr] : -1;   // of the step fetched next
    auto fetch = [&](int s) {
      const int slot = s + lr, flat = ahead;
      ahead = slot + 16 < hi ? a.plan.order[slot + 16] : -1;
      wt = flat < 0 ? 0.f : a.weights ? a.weights[flat] : 1.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) av[i] = bv[i] = 0.f;
      if (flat < 0) return;
      const long long row = second ? token_off(a.rows, flat / k, a.d) : (long long)(flat / k) * a.e;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = m0 + lc + i, c = c0 + lc + i;
        if (second) {
          if (m < a.d) av[i] = operand<T>(((const Td*)a.dtokens)[row + m]);
          if (c < a.d) bv[i] = a.buf0[(long long)slot * a.d + c];
        } else {
          if (m < a.d) av[i] = a.buf1[(long long)slot * a.d + m];
          if (c < a.e) bv[i] = to_f(((const T*)a.events)[row + c]);
        }
      }
    };
    fetch(lo);
    for (int s = lo; s < hi; s += 16) {
      __syncthreads();
      *(float4*)&As[lr][lc] = make_float4(av[0], av[1], av[2], av[3]);
      *(float4*)&Bs[lr][lc] = make_float4(bv[0], bv[1], bv[2], bv[3]);
      if (lc == 0) Bs[lr][64] = second ? wt : 1.f;
      __syncthreads();
      fetch(s + 16);              // in flight over this step's sums
#pragma unroll
      for (int kk = 0; kk < 16; ++kk) {
        const float4 x = *(const float4*)&As[kk][ty * 4], y = *(const float4*)&Bs[kk][tx * 4];
        const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xs[i], ys[j], acc[i][j]);
      }
      if (c0 == 0 && threadIdx.x < 64)
        for (int kk = 0; kk < 16; ++kk) colsum = fmaf(As[kk][threadIdx.x], Bs[kk][64], colsum);
    }
    float* mat = piece_at(w, blockIdx.y, t);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int m = m0 + ty * 4 + i, c = c0 + tx * 4 + j;
        if (m < a.d && c < cols) mat[(long long)m * cols + c] = acc[i][j];
      }
    if (c0 == 0 && threadIdx.x < 64 && m0 + threadIdx.x < a.d) mat[(long long)a.d * cols + m0 + threadIdx.x] = colsum;
  }
}

struct RoutedGrads {
  float *W1[kMaxTypes], *b1[kMaxTypes], *W2[kMaxTypes], *b2[kMaxTypes];
  float* emb;
};

// Each behaviour's pieces added in slice order (zeros where it has none);
// blockIdx.y = behaviour, V neighbouring values a thread, eight pieces in
// flight.  p1: dW1 and db1, p2: dW2 and db2.  The pieces are mostly still in
// L2: 39 pieces of d 256, e 64 in 3.9 us.
template <int V>
__global__ void __launch_bounds__(256) routed_wsum_kernel(PlanView plan, WeightPieces p1, WeightPieces p2, int d, int e,
                                                          RoutedGrads g) {
  grid_dep_wait();
  grid_dep_launch();
  if (!plan_ok(plan)) return;
  const int t = blockIdx.y;
  const int tile0 = plan_first(plan, t) / 128, tile1 = plan_first(plan, t + 1) / 128;
  const long long n1 = (long long)d * e, n2 = (long long)d * d;
  for (long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * V; i < p1.stride + p2.stride;
       i += (long long)gridDim.x * 256 * V) {
    const bool one = i < p1.stride;
    const WeightPieces& w = one ? p1 : p2;
    const long long j = one ? i : i - p1.stride;
    const int s0 = tile0 / w.per, s1 = tile1 > tile0 ? (tile1 - 1) / w.per + 1 : s0;
    float s[V];
#pragma unroll
    for (int k = 0; k < V; ++k) s[k] = 0.f;
    for (int q0 = s0; q0 < s1; q0 += 8) {
      float v[8][V];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float* p = piece_at(w, q0 + q, t) + j;
        if (q0 + q >= s1) {
#pragma unroll
          for (int k = 0; k < V; ++k) v[q][k] = 0.f;
        } else if constexpr (V == 4) {
          const float4 x = *(const float4*)p;
          v[q][0] = x.x; v[q][1] = x.y; v[q][2] = x.z; v[q][3] = x.w;
        } else {
          v[q][0] = *p;
        }
      }
#pragma unroll
      for (int q = 0; q < 8; ++q)
#pragma unroll
        for (int k = 0; k < V; ++k) s[k] += v[q][k];
    }
    auto put = [&](float* o) {
      if constexpr (V == 4) *(float4*)o = make_float4(s[0], s[1], s[2], s[3]);
      else *o = s[0];
    };
    if (one) {
      put(j < n1 ? g.W1[t] + j : g.b1[t] + (j - n1));
    } else if (j < n2) {
      put(g.W2[t] + j);
    } else {
      put(g.b2[t] + (j - n2));
      put(g.emb + (long long)t * d + (j - n2));
    }
  }
}

}  // namespace ot
