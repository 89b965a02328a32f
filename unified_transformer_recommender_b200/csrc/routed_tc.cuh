// Tensor-core kernels of the routed event tokenizer (bf16 mode, d a multiple
// of 64 up to 384, event_dim a multiple of 16 up to 128).  NC = d / 64.
#pragma once
#include "routed.cuh"

namespace ot {

// W1 [d][e] and W2 [d][d] of each behaviour as boxes of 64 rows x 64 columns.
struct RoutedMaps {
  CUtensorMap w1[kMaxTypes], w2[kMaxTypes];
};

struct RoutedTcArgs {
  PlanView plan;
  RoutedMLP mlp;
  int e;
  const __nv_bfloat16* events;
  const float* weights;          // [R*k] or null
  TokenRows rows;                // of tokens or dtokens
  // tokens
  __nv_bfloat16* tokens;         // k = 1
  // gradient
  const __nv_bfloat16* dtokens;
  __nv_bfloat16* devents;        // k = 1
  float* part;                   // k > 1: [R*k][d] of the tokens, [R*k][e] of the event gradient
};

constexpr int kSmemMax = 232448;

__device__ inline void cp_async16(void* dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
// Arrives on `bar` when every cp.async that this thread has issued is done (the
// barrier counts one such arrival per thread).
__device__ inline void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Shared memory written by threads (cp.async among them) before, seen by
// tensor-core products and TMA after.
__device__ inline void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// The product warps run their loops with all 32 lanes and let one elected lane
// issue: control flow and descriptors then stay warp-uniform, and the
// descriptors in uniform registers, where the tensor-core instructions want
// them (a branch on the lane number costs a register move per operand).
// elect.sync picks the same lane every time, so a commit covers the products
// that lane issued.  It names all 32 lanes: these warps wait with
// mbar_wait_warp, so that no lane leaves a loop alone.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}

// A slot of a ring and the parity of its current round.  Kept as a counter
// pair: the product thread issues alone, and a division per step would cost
// it as much as the products.
struct RingPos {
  int s = 0;
  uint32_t ph = 0;
  __device__ inline void next(int n) {
    if (++s == n) {
      s = 0;
      ph ^= 1;
    }
  }
};
// One arrival per warp: 32 would serialise on the barrier's word.
__device__ inline void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// Where each behaviour's slots begin and how many it has, from the plan into
// shared memory (nothing, and the status word set, if the plan is not this
// call's); every thread calls it, between grid_dep_wait and the roles.
struct PlanSpans {
  int first[kMaxTypes + 1], cnt[kMaxTypes];
};
__device__ inline bool load_spans(const PlanView& p, PlanSpans* s) {
  const bool ok = plan_ok(p);
  const int i = threadIdx.x;
  if (i <= kMaxTypes) s->first[i] = ok ? plan_first(p, i) : 0;
  if (i < kMaxTypes) s->cnt[i] = ok ? plan_count(p, i) : 0;
  __syncthreads();
  return ok;
}
__device__ inline int span_type(const PlanSpans* s, int T, int slot) {
  int t = 0;
  while (t + 1 < T && slot >= s->first[t + 1]) ++t;
  return t;
}

// Four warps copy gathered rows into boxes of [rows x 64 columns] with the
// 128-byte swizzle by cp.async, 16 rows at a time: a thread keeps one 16-byte
// column of rows r8, r8 + 16, ..., so that the pointers of a tile's rows are
// set up once for all its boxes and a box is one instruction per row (the
// gathering warps are otherwise what a step waits for).  No thread waits for
// its copies: they arrive on the box's barrier by themselves, and the products'
// warp fences before it reads.
struct GatherLane {
  int r8, c, at;                 // first row, 16-byte column, byte offset of it in a box
  __device__ inline explicit GatherLane(int tid)
      : r8(tid >> 3), c(tid & 7), at((tid >> 3) * 128 + (((tid & 7) ^ ((tid >> 3) & 7)) << 4)) {}
};
// ROWS / 16 rows of a box, p[j] + `shift` elements (rows without a source zero).
template <int ROWS>
__device__ __forceinline__ void gather_box(const GatherLane& g, uint8_t* box, const __nv_bfloat16* const* p, unsigned on,
                                           int shift) {
#pragma unroll
  for (int j = 0; j < ROWS / 16; ++j) cp_async16(box + g.at + j * 2048, p[j] + (on >> j & 1 ? shift : 0), on >> j & 1);
}
// An event tile of 128 rows (row[] in shared memory, -1: none) by NT threads:
// one or two boxes, columns past the width zero.
template <int NT>
__device__ __forceinline__ void gather_events(const GatherLane& g, uint8_t* tile, const __nv_bfloat16* events,
                                              const int* row, int width) {
  constexpr int RS = NT / 8;     // rows at a time: a multiple of 8, so the swizzle is the same for all of a thread's
#pragma unroll
  for (int j = 0; j < 128 / RS; ++j) {
    const int r = row[g.r8 + RS * j];
    const __nv_bfloat16* p = events + (long long)max(r, 0) * width;
    const bool on = r >= 0 && g.c * 8 < width;
    cp_async16(tile + g.at + j * RS * 128, p + (on ? g.c * 8 : 0), on);
    if (width > 64) {
      const bool on2 = r >= 0 && 64 + g.c * 8 < width;
      cp_async16(tile + 16384 + g.at + j * RS * 128, p + (on2 ? 64 + g.c * 8 : 0), on2);
    }
  }
}

// Zero rows for the events without any behaviour (k = 1): a warp looks at 32
// events at a time.
__device__ inline void zero_unrouted(const PlanView& plan, __nv_bfloat16* out, const TokenRows& rows, int width,
                                     int warp, int n_warps) {
  const int lane = threadIdx.x & 31;
  for (long long r0 = (long long)warp * 32; r0 < plan.R; r0 += (long long)n_warps * 32) {
    const int r = (int)r0 + lane;
    unsigned none = __ballot_sync(~0u, r < plan.R && plan.pos[r] < 0);
    while (none) {
      const int i = __ffs(none) - 1;
      none &= none - 1;
      uint4* o = (uint4*)(out + token_off(rows, (int)r0 + i, width));
      for (int c = lane; c < width / 8; c += 32) o[c] = make_uint4(0, 0, 0, 0);
    }
  }
}

// A behaviour's biases as float32: b1, and b2 + emb behind it at stride d.
__device__ inline void load_biases(float* to, const RoutedMLP& mlp, int t, int d, int tid, int nt) {
  const __nv_bfloat16 *b1 = (const __nv_bfloat16*)mlp.b1[t], *b2 = (const __nv_bfloat16*)mlp.b2[t];
  const __nv_bfloat16* emb = (const __nv_bfloat16*)mlp.emb + (long long)t * d;
  for (int c = tid * 2; c < d; c += nt * 2) {
    const float2 x = __bfloat1622float2(*(const __nv_bfloat162*)(b1 + c));
    const float2 y = __bfloat1622float2(*(const __nv_bfloat162*)(b2 + c));
    const float2 z = __bfloat1622float2(*(const __nv_bfloat162*)(emb + c));
    *(float2*)(to + c) = x;
    *(float2*)(to + d + c) = make_float2(y.x + z.x, y.y + z.y);
  }
}

// ----------------------------------------------------------------- tokens --
// One CTA per SM walks 128-slot tiles.  Per 64 hidden units: U = E W1c^T
// (tcgen05, M = 128, N = 64), bias and GELU by eight warps, z packed to bf16
// over U's own TMEM columns, D += z W2c^T with z read from TMEM (N = d).  The
// hidden row therefore never leaves the SM.  A chunk's weights and its U
// columns form one slot of a ring: both are free when its second product is
// done, so the chain product - GELU - product of up to four chunks overlaps
// (one chunk's chain takes about 1600 cycles, its products 640).  The weights
// stream through that ring from L2 (the tiles of one behaviour read the same
// 2 d (e + d) bytes).  The gathered event rows come through cp.async into the
// swizzled operand layout; four warps of their own take D out, weighted, as
// 128-byte pieces of the destination rows, while the next tile's first
// hidden units are computed.
// Warps 0-7 GELU, 8-11 output, 12-15 gather, 16 weights, 17 first products,
// 18 second products (one issuing warp would be the bottleneck).
// 75392 events (d 256, e 64) take 25 us, 500 TFLOP/s, four tiles a CTA (the
// products alone would be 5.5 us).  By the roles' clocks a tile takes 8.1 K
// cycles: for 4.9 K the output warps hold D, the one there is, while they read,
// weight and store it; for 3.1 K the next tile's second products follow, whose
// hidden units have been ready (0.9 K cycles of GELU a chunk).  10.7 K cycles
// before the first D and 4 K after the last are uncovered.  On CUDA cores the
// same call takes 605 us.
// z is rounded to bf16 as an operand, which decides the tokens' error: relative
// to 64 bits 2.31e-3, where the token's own rounding alone makes 1.65e-3.  GELU
// goes by the hardware's tanh, as in the block stack: off by up to 2^-12 |u|,
// less than z's rounding down to u of about -1.2, more in the tail (1e-3 at
// most, where z itself is small).  A GELU that is exact there too, by an
// exponential and a reciprocal, leaves the tokens' error at 2.31e-3 and took
// 28.4 us against 27.2 (256 events 12.6 / 11.6).
constexpr int kTokThreads = 608, kTokGelu = 8, kTokOut = 4;

struct TokCfg {
  int ebuf, slots;                // event tiles in flight, ring slots
  int e_bytes, w1_bytes, stage_bytes, smem;
};
__host__ __device__ inline TokCfg tok_cfg(int e, int d) {
  TokCfg c;
  const int eb = (e + 63) / 64;   // 64-column boxes of an event row
  c.e_bytes = eb * 16384;
  c.w1_bytes = eb * 8192;
  c.stage_bytes = c.w1_bytes + d * 128;
  // output staging, biases of two tiles, row indices, barriers and spans
  const int fixed = kTokOut * 32 * 144 + 4 * d * 4 + 256 * 4 + 512;
  const int room = kSmemMax - fixed;
  c.ebuf = eb == 1 ? 2 : 1;
  c.slots = (room - c.ebuf * c.e_bytes) / c.stage_bytes;
  const int cols = (512 - d) / 64;                // U buffers beside D in TMEM
  if (c.slots > cols) c.slots = cols;
  if (c.slots > 4) c.slots = 4;
  c.smem = fixed + c.ebuf * c.e_bytes + c.slots * c.stage_bytes;
  return c;
}

template <int NC, bool COMBINE>
__global__ void __launch_bounds__(kTokThreads, 1)
    routed_tokens_kernel(const __grid_constant__ RoutedMaps maps, const RoutedTcArgs a) {
  constexpr int d = NC * 64;
  extern __shared__ __align__(1024) uint8_t smem[];
  const TokCfg cfg = tok_cfg(a.e, d);
  uint8_t* sE = smem;
  uint8_t* sW = sE + cfg.ebuf * cfg.e_bytes;
  uint8_t* sOut = sW + cfg.slots * cfg.stage_bytes;
  float* sBias = (float*)(sOut + kTokOut * 32 * 144);       // [2][2 d]
  int* sRow = (int*)(sBias + 4 * d);                        // [2][128]
  uint64_t* bars = (uint64_t*)(sRow + 256);
  uint64_t* e_full = bars;          // [2]
  uint64_t* e_empty = bars + 2;     // [2]
  uint64_t* w_full = bars + 4;      // [4] a slot's weights
  uint64_t* u_full = bars + 8;      // [4]
  uint64_t* z_ready = bars + 12;    // [4]
  uint64_t* slot_free = bars + 16;  // [4]
  uint64_t* b_full = bars + 20;     // [2] a tile's biases
  uint64_t* b_free = bars + 22;     // [2]
  uint64_t* d_full = bars + 24;
  uint64_t* d_empty = bars + 25;
  uint32_t* tmem_slot = (uint32_t*)(bars + 26);
  PlanSpans* spans = (PlanSpans*)(bars + 28);

  if (smem_u32(smem) & 1023) {
    if (threadIdx.x == 0) flag_error(kErrSmemAlign);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&e_full[i], 128);
      mbar_init(&e_empty[i], 1);
      mbar_init(&b_full[i], 4);
      mbar_init(&b_free[i], kTokGelu + kTokOut);
    }
    for (int i = 0; i < cfg.slots; ++i) {
      mbar_init(&w_full[i], 1);
      mbar_init(&u_full[i], 1);
      mbar_init(&z_ready[i], kTokGelu);
      mbar_init(&slot_free[i], 1);
    }
    mbar_init(d_full, 1);
    mbar_init(d_empty, kTokOut);
    fence_barrier_init();
  }
  if (warp == 17) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tD = tmem, tU = tmem + d;   // U of slot s at tU + 64 s
  grid_dep_wait();
  grid_dep_launch();
  const bool fine = load_spans(a.plan, spans);
  const int T = a.plan.T, n_tiles = spans->first[T] / 128;
  const int step = gridDim.x;

  if (warp == 16) {
    // ------------------------------------------------------ weight producer
    if (lane == 0) {
      const uint64_t keep = l2_evict_last();
      RingPos w;
      bool wrapped = false, ok = true;
      for (int tile = blockIdx.x; tile < n_tiles && ok; tile += step) {
        const int t = span_type(spans, T, tile * 128);
        for (int c = 0; c < NC; ++c) {
          ok = !wrapped || mbar_wait(&slot_free[w.s], w.ph ^ 1);
          if (!ok) break;
          uint8_t* w1 = sW + w.s * cfg.stage_bytes;
          mbar_expect_tx(&w_full[w.s], cfg.stage_bytes);
          tma_load_3d_hint(&maps.w1[t], &w_full[w.s], w1, 0, c * 64, 0, keep);
          if (cfg.w1_bytes > 8192) tma_load_3d_hint(&maps.w1[t], &w_full[w.s], w1 + 8192, 64, c * 64, 0, keep);
#pragma unroll
          for (int b = 0; b < NC; ++b)
            tma_load_3d_hint(&maps.w2[t], &w_full[w.s], w1 + cfg.w1_bytes + b * 8192, c * 64, b * 64, 0, keep);
          w.next(cfg.slots);
          wrapped = wrapped || w.s == 0;
        }
      }
    }
  } else if (warp == 17) {
    // ------------------------------------------------------- first products
    const uint64_t dE = sdesc_k128(smem_u32(sE)), dW = sdesc_k128(smem_u32(sW));
    constexpr uint32_t id_u = idesc_bf16(128, 64);
    const int ksteps = a.e / 16;
    bool ok = true;
    RingPos r, er;
    for (int tile = blockIdx.x; tile < n_tiles && ok; tile += step) {
      for (int c = 0; c < NC; ++c) {
        ok = mbar_wait_warp(&w_full[r.s], r.ph);      // refilled, so the slot's U is free too
        if (c == 0) {
          ok = ok && mbar_wait_warp(&e_full[er.s], er.ph);
          fence_async_smem();
        }
        if (!ok) break;
        tc_fence_after();
        const uint64_t de = desc_add(dE, er.s * cfg.e_bytes), dw = desc_add(dW, r.s * cfg.stage_bytes);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < ksteps)
            mma_ss(tU + r.s * 64, desc_add(de, (k >> 2) * 16384 + (k & 3) * 32),
                   desc_add(dw, (k >> 2) * 8192 + (k & 3) * 32), id_u, k ? 1u : 0u);
        mma_commit(&u_full[r.s]);
        r.next(cfg.slots);
      }
      mma_commit(&e_empty[er.s]);
      er.next(cfg.ebuf);
    }
  } else if (warp == 18) {
    // ------------------------------------------------------ second products
    const uint64_t dW = sdesc_k128(smem_u32(sW) + cfg.w1_bytes);
    constexpr int n0 = d > 256 ? 256 : d, n1 = d - n0;
    constexpr uint32_t id_0 = idesc_bf16(128, n0), id_1 = idesc_bf16(128, n1 ? n1 : 16);
    bool ok = true;
    RingPos r;
    int i = 0;
    for (int tile = blockIdx.x; tile < n_tiles && ok; tile += step, ++i) {
      for (int c = 0; c < NC; ++c) {
        ok = mbar_wait_warp(&z_ready[r.s], r.ph);
        if (c == 0 && i > 0) ok = ok && mbar_wait_warp(d_empty, (i - 1) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint64_t w2 = desc_add(dW, r.s * cfg.stage_bytes);
#pragma unroll
        for (int k = 0; k < 4; ++k) {   // units 16k .. 16k+15 packed over U columns 16k .. 16k+7
          const uint32_t z = tU + r.s * 64 + k * 16;
          mma_ts(tD, z, desc_add(w2, k * 32), id_0, (c | k) ? 1u : 0u);
          if (n1) mma_ts(tD + n0, z, desc_add(w2, n0 * 128 + k * 32), id_1, (c | k) ? 1u : 0u);
        }
        mma_commit(&slot_free[r.s]);
        r.next(cfg.slots);
      }
      mma_commit(d_full);
    }
  } else if (warp >= 12) {
    // --------------------------------------------------------------- gather
    const int tid = threadIdx.x - 12 * 32;
    const GatherLane lane_of(tid);
    bool ok = true;
    RingPos e;
    int i = 0;
    int flat = (int)blockIdx.x < n_tiles ? a.plan.order[(long long)blockIdx.x * 128 + tid] : -1;
    for (int tile = blockIdx.x; tile < n_tiles; tile += step, ++i) {
      int* rows = sRow + (i & 1) * 128;
      rows[tid] = flat < 0 ? -1 : flat / a.plan.k;
      if (tile + step < n_tiles) flat = a.plan.order[(long long)(tile + step) * 128 + tid];
      asm volatile("bar.sync 1, 128;" ::: "memory");
      if (i >= cfg.ebuf) ok = ok && mbar_wait(&e_empty[e.s], e.ph ^ 1);
      if (ok) gather_events<128>(lane_of, sE + e.s * cfg.e_bytes, a.events, rows, a.e);
      cp_async_arrive(&e_full[e.s]);
      e.next(cfg.ebuf);
      if (i >= 2) ok = ok && mbar_wait(&b_free[i & 1], ((i >> 1) & 1) ^ 1);
      load_biases(sBias + (i & 1) * 2 * d, a.mlp, span_type(spans, T, tile * 128), d, tid, 128);
      warp_arrive(&b_full[i & 1]);
    }
    if (!COMBINE && fine) zero_unrouted(a.plan, a.tokens, a.rows, d, blockIdx.x * 4 + warp - 12, gridDim.x * 4);
  } else if (warp >= 8) {
    // --------------------------------------------------------------- output
    const int q4 = warp & 3;                    // row quarter
    const uint32_t lb = (uint32_t)(q4 * 32) << 16;
    uint8_t* stage = sOut + q4 * 32 * 144;
    bool ok = true;
    int i = 0;
    for (int tile = blockIdx.x; tile < n_tiles; tile += step, ++i) {
      const int flat = a.plan.order[(long long)tile * 128 + q4 * 32 + lane];
      const float w = flat >= 0 && a.weights ? a.weights[flat] : 1.f;
      const long long off = flat < 0 ? -1LL : COMBINE ? (long long)flat * d : token_off(a.rows, flat, d);
      const float* s = sBias + (i & 1) * 2 * d + d;
      ok = ok && mbar_wait(&b_full[i & 1], (i >> 1) & 1);
      ok = ok && mbar_wait(d_full, i & 1);
      tc_fence_after();
      constexpr int PW = COMBINE ? 32 : 64;     // columns of a 128-byte piece
#pragma unroll 1
      for (int c0 = 0; c0 < d; c0 += PW) {
#pragma unroll
        for (int h = 0; h < PW; h += 32) {
          float v[32];
          tmem_ld32(tD + lb + c0 + h, v);
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 b = *(const float4*)(s + c0 + h + j);
            v[j] = w * (v[j] + b.x); v[j + 1] = w * (v[j + 1] + b.y);
            v[j + 2] = w * (v[j + 2] + b.z); v[j + 3] = w * (v[j + 3] + b.w);
          }
          if (COMBINE) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *(float4*)(stage + lane * 144 + j * 16) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          } else {
            store_bf16x32((__nv_bfloat16*)(stage + lane * 144 + h * 2), v);
          }
        }
        if (c0 + PW == d) {               // D read: the next tile may overwrite it
          tc_fence_before();
          warp_arrive(d_empty);
          warp_arrive(&b_free[i & 1]);
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int r = j * 4 + (lane >> 3), ch = lane & 7;
          const long long o = __shfl_sync(~0u, off, r);
          if (o >= 0 && ok) {
            const uint4 x = *(const uint4*)(stage + r * 144 + ch * 16);
            if (COMBINE) *(uint4*)(a.part + o + c0 + ch * 4) = x;
            else *(uint4*)(a.tokens + o + c0 + ch * 8) = x;
          }
        }
        __syncwarp();
      }
    }
  } else {
    // ----------------------------------------------------------------- GELU
    const int q4 = warp & 3, wq = warp >> 2;    // row quarter, half of the chunk's columns
    const uint32_t mine = tU + ((uint32_t)(q4 * 32) << 16) + wq * 32;
    bool ok = true;
    RingPos r;
    int i = 0;
    for (int tile = blockIdx.x; tile < n_tiles; tile += step, ++i) {
      const float* b1 = sBias + (i & 1) * 2 * d + wq * 32;
      ok = ok && mbar_wait(&b_full[i & 1], (i >> 1) & 1);
#pragma unroll 1
      for (int c = 0; c < NC; ++c) {
        ok = ok && mbar_wait(&u_full[r.s], r.ph);
        tc_fence_after();
        const uint32_t col = mine + r.s * 64;
        float v[32];
        tmem_ld32(col, v);
        uint32_t pk[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 b = *(const float4*)(b1 + c * 64 + j * 4);
          pk[2 * j] = gelu_bias_bf16x2(v[4 * j], v[4 * j + 1], b.x, b.y);
          pk[2 * j + 1] = gelu_bias_bf16x2(v[4 * j + 2], v[4 * j + 3], b.z, b.w);
        }
        tmem_st8(col, pk);
        tmem_st8(col + 16, pk + 8);
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&z_ready[r.s]);
        r.next(cfg.slots);
      }
      warp_arrive(&b_free[i & 1]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 17) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------- shared, backward --
__device__ inline float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ inline float rcp_ftz(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// GELU-tanh and its slope of a pair, to float32 accuracy: with
// s = 1 / (1 + exp(-2v)), v = c (u + a u^3), GELU(u) = u s and
// d/du = s + u s (1 - s) (2c + 6 c a u^2)  (0.5 (1 + tanh v) = s).  Two
// special-function results a value (16 a clock an SM), the rest on packed
// float32 pairs; one reciprocal for the two values of a pair (1/p = q / (p q))
// saved special-function time but cost more in moves and bounds.  |u| large
// gives s = 0 or 1 exactly; u^2 is bounded in the slope, where inf * 0 would
// follow.
struct GeluPair {
  uint64_t u2, s, z;
};
__device__ __forceinline__ GeluPair gelu_pair(uint64_t u) {
  const float c = 0.7978845608028654f, a = 0.044715f, m2l = -2.8853900817779268f;   // -2 log2(e)
  GeluPair r;
  r.u2 = f2_mul(u, u);
  const uint64_t v = f2_mul(u, f2_fma(r.u2, f2_pack(m2l * c * a, m2l * c * a), f2_pack(m2l * c, m2l * c)));
  float x, y;
  f2_unpack(v, x, y);
  const uint64_t d = f2_add(f2_pack(ex2_ftz(x), ex2_ftz(y)), f2_pack(1.f, 1.f));
  f2_unpack(d, x, y);
  r.s = f2_pack(rcp_ftz(x), rcp_ftz(y));
  r.z = f2_mul(u, r.s);
  return r;
}
__device__ __forceinline__ uint64_t gelu_slope(const GeluPair& r) {
  const float c = 0.7978845608028654f, a = 0.044715f;
  float x, y;
  f2_unpack(r.u2, x, y);
  const uint64_t q = f2_fma(f2_pack(fminf(x, 256.f), fminf(y, 256.f)), f2_pack(6.f * c * a, 6.f * c * a), f2_pack(2.f * c, 2.f * c));
  return f2_fma(f2_mul(r.z, f2_fma(r.s, f2_pack(-1.f, -1.f), f2_pack(1.f, 1.f))), q, r.s);
}
// A pair as bf16 hi + lo: 16 bits of significand in two operands.
__device__ __forceinline__ void split_pair(uint64_t x, uint32_t& hi, uint32_t& lo) {
  float x0, x1;
  f2_unpack(x, x0, x1);
  hi = pack_bf16x2(x0, x1);
  const uint64_t h = f2_pack(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u));
  f2_unpack(f2_fma(h, f2_pack(-1.f, -1.f), x), x0, x1);
  lo = pack_bf16x2(x0, x1);
}

// float32 dtokens rounded to bf16 rows [R][d], the operand type of the
// products (a pass of its own: the gathers copy rows asynchronously, which
// leaves no room for a conversion).
__global__ void __launch_bounds__(256) routed_round_rows_kernel(const float* __restrict__ src, TokenRows rows, int R,
                                                                int d, __nv_bfloat16* __restrict__ dst) {
  grid_dep_wait();
  grid_dep_launch();
  const int per = d / 8;
  const long long n = (long long)R * per;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    const int r = (int)(i / per), c = (int)(i - (long long)r * per) * 8;
    const float4* p = (const float4*)(src + token_off(rows, r, d) + c);
    const float4 x = p[0], y = p[1];
    *(uint4*)(dst + (long long)r * d + c) = make_uint4(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w),
                                                       pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
  }
}

// ----------------------------------------------------------- weight gradients --
// A CTA holds 128 hidden units of one behaviour at a time and walks its slice
// of the slots, 128 (one tile) a step, transposed so that hidden units are
// TMEM lanes:
//   U^T = W1c E^T (M = 128 units, N = 128 slots, K = e),
//   DZ^T = W2c^T DY^T (K = d); then, from z and du in TMEM as A operands,
//   dW2c^T [128][d] += z DY and dW1c [128][e] += du E (K = 128 slots).
// z = w GELU(u) and du = w dz GELU'(u) overwrite the columns they come from
// as two bf16 terms each, so the hidden rows are recomputed but never stored,
// db1 is a sum inside a thread, and the gathered rows serve as both K-major
// and MN-major operands.  Both gradients need U but nothing else of one
// another, and together more TMEM than there is; so half of the CTAs (role 1)
// compute U, DZ, du, dW1 and db1, the other half (role 2) U, z, dW2 and db2,
// about 2400 tensor-core cycles a step (d = 256, e = 64) each.
// Role 1 also writes du, rounded once to bf16, as rows for the event gradient
// and, where asked, each slot's <dz, z> over its units.
// The compute warps bound it.  By their clocks a step takes 5.4 K cycles, one
// phase after the other (the warps are mostly in the same one): in role 1 2.6 K
// for GELU and its slope (the two special-function results a value alone would
// be 2.0 K), 0.4 K waiting for dz, 0.9 K multiplying and splitting, 0.7 K
// storing du, 0.6 K waiting for the next U; in role 2 3.1 K for GELU and the
// split, 1.7 K for db2, 0.7 K waiting.  The first step takes 12 K, the end of a
// piece 4-7 K.  768 threads leave 80 registers each, and every instantiation
// spills (d 256: 80 bytes stored and 116 loaded, with choice weights' gradients
// 216 and 264; d 384 with them 348 and 348).
// Warps 0-15 compute, 16-19 gather DY, 20-21 events (on their own, so that
// the next step's do not queue behind this step's DY), 22 weights and first
// products, 23 second products.
// 75392 events (d 256, e 64): 71 us in a list of launches, 16 steps a CTA, of
// the call's 110; on CUDA cores the call takes 1217 (float32).  Three event tiles in
// flight against two: 109 / 113.5 us (e <= 64; wider rows leave room for two).
// The sums' error: the second term's rounding (2^-17 of a value) and the tensor
// cores' float32 sums, which truncate; 5.5e-6 of dW1 over 75392 events
// together, where float32 sums in another order differ by 3.1e-6 (9973 events
// of two of eight behaviours: 3.2e-6 and 1.0e-6).  One term would leave 2^-9 of
// each value; a third costs half the products again.
constexpr int kWgThreads = 768, kWgCompute = 16;

struct WgCfg {
  int eb, chunks;                  // event boxes, hidden chunks of 128
  int w1_bytes, e_bytes;
  int ebuf;                        // event tiles in flight
  int units1, units2;              // DY ring: role 1 [128 slots x 64], role 2 [64 slots x d]
  int ring;                        // bytes behind the event tiles
  int smem;
};
__host__ __device__ inline WgCfg wg_cfg(int e, int d) {
  WgCfg c;
  c.eb = (e + 63) / 64;
  c.chunks = (d + 127) / 128;
  c.w1_bytes = c.eb * 16384;
  c.e_bytes = c.eb * 16384;
  c.ebuf = c.eb == 1 ? 3 : 2;
  // barriers and spans; dtoken row offsets of two steps, event rows and weights
  // of ebuf
  const int fixed = 512 + 2 * 128 * 8 + 3 * 128 * 8;
  const int room = kSmemMax - fixed - c.w1_bytes - c.ebuf * c.e_bytes;
  c.units1 = (room - d * 256) / 16384;
  if (c.units1 > 8) c.units1 = 8;
  c.units2 = room / (d * 128);
  if (c.units2 > 8) c.units2 = 8;
  const int s1 = d * 256 + c.units1 * 16384, s2 = c.units2 * d * 128;
  c.ring = s1 > s2 ? s1 : s2;
  c.smem = fixed + c.w1_bytes + c.ebuf * c.e_bytes + c.ring;
  return c;
}

struct WgArgs {
  WeightPieces p1, p2;           // dW1 [d][e] and db1 [d]; dW2 [d][d] and db2 [d]
  __nv_bfloat16* du;             // [slots][d], or null
  float* dot;                    // [slots][4 chunks], or null
};

struct WgShared {                // one CTA's shared memory
  uint8_t *w1, *e, *w2, *y;      // w2: role 1; y: the DY ring
  long long* off;                // [2][128] dtoken rows
  int* row;                      // [ebuf][128] event rows
  float* wt;                     // [ebuf][128] choice weights
  uint64_t* bars;
  PlanSpans* spans;
};
enum : int {   // barriers; pairs and rings by index
  WB_EFULL = 0, WB_EEMPTY = 3, WB_YFULL = 6, WB_YEMPTY = 14, WB_UFULL = 22, WB_UFREE = 24, WB_ZFULL = 26, WB_READY = 28,
  WB_USED = 30, WB_W = 32, WB_ACCFULL = 33, WB_ACCFREE = 34, WB_TMEM = 35, WB_SPANS = 36
};

// The slots of behaviour t in tiles [tile0, tile1): [lo, hi), hi before the padding.
__device__ inline bool wg_piece(const PlanSpans* s, int tile0, int tile1, int t, int& lo, int& hi) {
  lo = max(tile0 * 128, s->first[t]);
  hi = min(tile1 * 128, s->first[t] + s->cnt[t]);
  return lo < hi;
}

// Gathers the steps' event tiles and choice weights (two warps).
__device__ inline void wg_gather_events(const RoutedTcArgs& a, const WgCfg& cfg, const WgShared& m, int tile0, int tile1) {
  const int tid = threadIdx.x - (kWgCompute + 4) * 32;
  const GatherLane g(tid);
  bool ok = true, wrapped = false;
  RingPos er;
  for (int t = 0; t < a.plan.T; ++t) {
    int lo, hi;
    if (!wg_piece(m.spans, tile0, tile1, t, lo, hi)) continue;
    for (int at = lo; at < hi; at += 128) {
      const int b = er.s;
      int flat[2];
      float wt[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) flat[j] = at + j * 64 + tid < hi ? a.plan.order[at + j * 64 + tid] : -1;
#pragma unroll
      for (int j = 0; j < 2; ++j) wt[j] = flat[j] < 0 ? 0.f : a.weights ? a.weights[flat[j]] : 1.f;
      if (wrapped) ok = ok && mbar_wait(&m.bars[WB_EEMPTY + b], er.ph ^ 1);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m.row[b * 128 + j * 64 + tid] = flat[j] < 0 ? -1 : flat[j] / a.plan.k;
        m.wt[b * 128 + j * 64 + tid] = wt[j];
      }
      asm volatile("bar.sync 3, 64;" ::: "memory");
      if (ok) gather_events<64>(g, m.e + b * cfg.e_bytes, a.events, m.row + b * 128, a.e);
      cp_async_arrive(&m.bars[WB_EFULL + b]);
      warp_arrive(&m.bars[WB_EFULL + b]);         // releases the weights: the arrival above covers the copies alone
      er.next(cfg.ebuf);
      wrapped = wrapped || er.s == 0;
    }
  }
}

// Gathers the steps' DY units (four warps).
template <int NC, bool ROLE1>
__device__ inline void wg_gather(const RoutedTcArgs& a, const WgCfg& cfg, const WgShared& m, int tile0, int tile1) {
  constexpr int d = NC * 64;
  const int tid = threadIdx.x - kWgCompute * 32, units = ROLE1 ? cfg.units1 : cfg.units2;
  const GatherLane g(tid);
  bool ok = true, wrapped = false;
  int i = 0;
  RingPos y;
  for (int t = 0; t < a.plan.T; ++t) {
    int lo, hi;
    if (!wg_piece(m.spans, tile0, tile1, t, lo, hi)) continue;
    int flat = lo + tid < hi ? a.plan.order[lo + tid] : -1;
    for (int at = lo; at < hi; at += 128, ++i) {
      const int b = i & 1;
      m.off[b * 128 + tid] = flat < 0 ? -1LL : token_off(a.rows, flat / a.plan.k, d);
      flat = at + 128 + tid < hi ? a.plan.order[at + 128 + tid] : -1;   // of the next step
      asm volatile("bar.sync 1, 128;" ::: "memory");
      const __nv_bfloat16* p[8];
      unsigned on = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const long long o = m.off[b * 128 + g.r8 + 16 * j];
        on |= (o >= 0 ? 1u : 0u) << j;
        p[j] = o >= 0 ? a.dtokens + o + g.c * 8 : a.dtokens;
      }
#pragma unroll 1
      for (int u = 0; u < (ROLE1 ? NC : 2); ++u) {
        if (wrapped) ok = ok && mbar_wait(&m.bars[WB_YEMPTY + y.s], y.ph ^ 1);
        if (ok && ROLE1) gather_box<128>(g, m.y + y.s * 16384, p, on, u * 64);
        if (ok && !ROLE1) {
          uint8_t* to = m.y + y.s * (d * 128);
#pragma unroll
          for (int c = 0; c < NC; ++c) {           // the unit's 64 slots: rows j = 4 u .. 4 u + 3
            if (u == 0) gather_box<64>(g, to + c * 8192, p, on, c * 64);
            else gather_box<64>(g, to + c * 8192, p + 4, on >> 4, c * 64);
          }
        }
        cp_async_arrive(&m.bars[WB_YFULL + y.s]);
        y.next(units);
        wrapped = wrapped || y.s == 0;
      }
    }
  }
}

// The hidden chunk's weights of behaviour t, when the last piece's sums have
// been taken out (its products are then done).
template <int NC, bool ROLE1>
__device__ inline bool wg_weights(const RoutedMaps& maps, const WgCfg& cfg, const WgShared& m, int t, int chunk, int p) {
  constexpr int d = NC * 64;
  if (p > 0 && !mbar_wait_warp(&m.bars[WB_ACCFREE], (p - 1) & 1)) return false;
  if ((threadIdx.x & 31) == 0) {
    const uint64_t keep = l2_evict_last();
    uint64_t* full = &m.bars[WB_W];
    mbar_expect_tx(full, cfg.w1_bytes + (ROLE1 ? d * 256 : 0));
    for (int b = 0; b < cfg.eb; ++b)
      for (int j = 0; j < 2; ++j)
        tma_load_3d_hint(&maps.w1[t], full, m.w1 + b * 16384 + j * 8192, b * 64, chunk * 128 + j * 64, 0, keep);
    for (int j = 0; ROLE1 && j < 2; ++j)
      for (int b = 0; b < NC; ++b)
        tma_load_3d_hint(&maps.w2[t], full, m.w2 + j * d * 128 + b * 8192, chunk * 128 + j * 64, b * 64, 0, keep);
  }
  __syncwarp();
  return mbar_wait_warp(&m.bars[WB_W], p & 1);
}

// Role 1's products.
template <int NC>
__device__ inline void wg_products1(const RoutedMaps& maps, int chunk, const RoutedTcArgs& a, const WgCfg& cfg, const WgShared& m, uint32_t tmem, int tile0,
                                    int tile1, bool first) {
  constexpr int d = NC * 64;
  const uint32_t tU = tmem, tZ = tmem + 128, tW1 = tmem + 384;   // U, two DZ buffers, dW1
  const int ksteps = a.e / 16;
  bool ok = true;
  int i = 0, p = 0;
  RingPos er;
  if (first) {
    const uint64_t dW1 = sdesc_k128(smem_u32(m.w1)), dW2 = sdesc_mn128(smem_u32(m.w2), d * 128);
    const uint64_t dE = sdesc_k128(smem_u32(m.e)), dY = sdesc_k128(smem_u32(m.y));
    constexpr uint32_t id_u = idesc_bf16(128, 128), id_z = idesc_bf16(128, 128, true, false);
    RingPos y;
    for (int t = 0; t < a.plan.T && ok; ++t) {
      int lo, hi;
      if (!wg_piece(m.spans, tile0, tile1, t, lo, hi)) continue;
      ok = wg_weights<NC, true>(maps, cfg, m, t, chunk, p);
      ++p;
      for (int at = lo; at < hi; at += 128, ++i) {
        const int b = i & 1;
        ok = ok && mbar_wait_warp(&m.bars[WB_EFULL + er.s], er.ph);
        if (i > 0) ok = ok && mbar_wait_warp(&m.bars[WB_UFREE], (i - 1) & 1);   // U read into registers
        if (!ok) break;
        fence_async_smem();
        tc_fence_after();
        const uint64_t de = desc_add(dE, er.s * cfg.e_bytes);
        er.next(cfg.ebuf);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < ksteps)
            mma_ss(tU, desc_add(dW1, (k >> 2) * 16384 + (k & 3) * 32), desc_add(de, (k >> 2) * 16384 + (k & 3) * 32), id_u,
                   k ? 1u : 0u);
        mma_commit(&m.bars[WB_UFULL]);
        if (i >= 2) ok = mbar_wait_warp(&m.bars[WB_USED + b], ((i >> 1) & 1) ^ 1);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          ok = ok && mbar_wait_warp(&m.bars[WB_YFULL + y.s], y.ph);
          if (!ok) break;
          fence_async_smem();
          tc_fence_after();
          const uint64_t dy = desc_add(dY, y.s * 16384);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ss(tZ + b * 128, desc_add(dW2, c * 8192 + k * 2048), desc_add(dy, k * 32), id_z, (c | k) ? 1u : 0u);
          mma_commit(&m.bars[WB_YEMPTY + y.s]);
          y.next(cfg.units1);
        }
        if (!ok) break;
        mma_commit(&m.bars[WB_ZFULL + b]);
      }
    }
    return;
  }
  const uint64_t dEm = sdesc_mn128(smem_u32(m.e), 16384);
  const uint32_t id_1 = idesc_bf16(128, a.e, false, true);
  for (int t = 0; t < a.plan.T && ok; ++t) {
    int lo, hi;
    if (!wg_piece(m.spans, tile0, tile1, t, lo, hi)) continue;
    if (p > 0) ok = mbar_wait_warp(&m.bars[WB_ACCFREE], (p - 1) & 1);
    ++p;
    for (int at = lo; at < hi; at += 128, ++i) {
      const int b = i & 1;
      ok = ok && mbar_wait_warp(&m.bars[WB_READY + b], (i >> 1) & 1);
      if (!ok) break;
      fence_async_smem();
      tc_fence_after();
      const uint64_t de = desc_add(dEm, er.s * cfg.e_bytes);
#pragma unroll
      for (int k = 0; k < 8; ++k) {      // 16 slots: hi in 8 columns, lo in the next 8
        const uint32_t du = tZ + b * 128 + k * 16;
        mma_ts(tW1, du, desc_add(de, k * 2048), id_1, at > lo || k ? 1u : 0u);
        mma_ts(tW1, du + 8, desc_add(de, k * 2048), id_1, 1u);
      }
      mma_commit(&m.bars[WB_USED + b]);
      mma_commit(&m.bars[WB_EEMPTY + er.s]);
      er.next(cfg.ebuf);
    }
    mma_commit(&m.bars[WB_ACCFULL]);
  }
}

// Role 2's products; U buffers beside dW2: two up to d = 256, else one.
template <int NC>
__device__ inline void wg_products2(const RoutedMaps& maps, int chunk, const RoutedTcArgs& a, const WgCfg& cfg, const WgShared& m, uint32_t tmem, int tile0,
                                    int tile1, bool first) {
  constexpr int d = NC * 64, NBU = d <= 256 ? 2 : 1;
  const uint32_t tW2 = tmem, tU = tmem + (NBU == 2 ? 256 : 384);
  const int ksteps = a.e / 16;
  bool ok = true;
  int i = 0, p = 0;
  RingPos u, er;                   // U buffer and event tile of the step
  if (first) {
    const uint64_t dW1 = sdesc_k128(smem_u32(m.w1)), dE = sdesc_k128(smem_u32(m.e));
    constexpr uint32_t id_u = idesc_bf16(128, 128);
    for (int t = 0; t < a.plan.T && ok; ++t) {
      int lo, hi;
      if (!wg_piece(m.spans, tile0, tile1, t, lo, hi)) continue;
      ok = wg_weights<NC, false>(maps, cfg, m, t, chunk, p);
      ++p;
      for (int at = lo; at < hi; at += 128, ++i) {
        ok = ok && mbar_wait_warp(&m.bars[WB_EFULL + er.s], er.ph);
        if (i >= NBU) ok = ok && mbar_wait_warp(&m.bars[WB_USED + u.s], u.ph ^ 1);
        if (!ok) break;
        fence_async_smem();
        tc_fence_after();
        const uint64_t de = desc_add(dE, er.s * cfg.e_bytes);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < ksteps)
            mma_ss(tU + u.s * 128, desc_add(dW1, (k >> 2) * 16384 + (k & 3) * 32),
                   desc_add(de, (k >> 2) * 16384 + (k & 3) * 32), id_u, k ? 1u : 0u);
        mma_commit(&m.bars[WB_UFULL + u.s]);
        mma_commit(&m.bars[WB_EEMPTY + er.s]);
        er.next(cfg.ebuf);
        u.next(NBU);
      }
    }
    return;
  }
  const uint64_t dY = sdesc_mn128(smem_u32(m.y), 8192);
  constexpr int n0 = d > 256 ? 256 : d, n1 = d - n0;
  constexpr uint32_t id_2 = idesc_bf16(128, n0, false, true), id_2b = idesc_bf16(128, n1 ? n1 : 16, false, true);
  RingPos y;
  for (int t = 0; t < a.plan.T && ok; ++t) {
    int lo, hi;
    if (!wg_piece(m.spans, tile0, tile1, t, lo, hi)) continue;
    if (p > 0) ok = mbar_wait_warp(&m.bars[WB_ACCFREE], (p - 1) & 1);
    ++p;
    for (int at = lo; at < hi; at += 128, ++i) {
      ok = ok && mbar_wait_warp(&m.bars[WB_READY + u.s], u.ph);
      if (!ok) break;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        ok = ok && mbar_wait_warp(&m.bars[WB_YFULL + y.s], y.ph);
        if (!ok) break;
        fence_async_smem();
        tc_fence_after();
        const uint64_t dy = desc_add(dY, y.s * (d * 128));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t z = tU + u.s * 128 + h * 64 + k * 16;
          mma_ts(tW2, z, desc_add(dy, k * 2048), id_2, at > lo || h || k ? 1u : 0u);
          mma_ts(tW2, z + 8, desc_add(dy, k * 2048), id_2, 1u);
          if (n1) {
            mma_ts(tW2 + n0, z, desc_add(dy, n0 * 128 + k * 2048), id_2b, at > lo || h || k ? 1u : 0u);
            mma_ts(tW2 + n0, z + 8, desc_add(dy, n0 * 128 + k * 2048), id_2b, 1u);
          }
        }
        mma_commit(&m.bars[WB_YEMPTY + y.s]);
        y.next(cfg.units2);
      }
      mma_commit(&m.bars[WB_USED + u.s]);
      u.next(NBU);
    }
    mma_commit(&m.bars[WB_ACCFULL]);
  }
}

// The lane's partial sums of 32 slots added over the warp's 32 lanes: lane l
// returns slot l's total (halving exchanges, 31 shuffles).
__device__ inline float reduce_slots(float* v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int j = 0; j < o; ++j) {
      const float give = up ? v[j] : v[j + o], keep = up ? v[j + o] : v[j];
      v[j] = keep + __shfl_xor_sync(~0u, give, o);
    }
  }
  return v[0];
}

template <int NC, bool DOT>
__device__ inline void wg_compute1(const RoutedTcArgs& a, const WgCfg& cfg, const WgShared& m, const WgArgs& w,
                                   uint32_t tmem, int tile0, int tile1, int chunk, int slice) {
  constexpr int d = NC * 64;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q4 = warp & 3, sg = warp >> 2;         // hidden quarter, 32 of the step's slots
  const int h = chunk * 128 + q4 * 32 + lane;
  const bool real = chunk * 128 + q4 * 32 < d;     // the same for the warp: d is a multiple of 64
  const uint32_t lb = ((uint32_t)(q4 * 32) << 16) + sg * 32;
  const uint32_t tU = tmem + lb, tZ = tmem + 128 + lb, tW1 = tmem + 384 + ((uint32_t)(q4 * 32) << 16);
  bool ok = true;
  int i = 0, p = 0;
  RingPos er;
  for (int t = 0; t < a.plan.T; ++t) {
    int lo, hi;
    if (!wg_piece(m.spans, tile0, tile1, t, lo, hi)) continue;
    const float b1s = real ? __bfloat162float(((const __nv_bfloat16*)a.mlp.b1[t])[h]) : 0.f;
    const uint64_t b1 = f2_pack(b1s, b1s);
    uint64_t db1 = f2_pack(0.f, 0.f);
#pragma unroll 1
    for (int at = lo; at < hi; at += 128, ++i) {
      const int b = i & 1;
      ok = ok && mbar_wait(&m.bars[WB_EFULL + er.s], er.ph);   // the choice weights
      ok = ok && mbar_wait(&m.bars[WB_UFULL], i & 1);
      tc_fence_after();
      const float* wt = m.wt + er.s * 128 + sg * 32;
      er.next(cfg.ebuf);
      uint64_t g[16], z[DOT ? 16 : 1];             // w GELU'(u), GELU(u)
      {
        float v[32];
        tmem_ld32(tU, v);
        tc_fence_before();
        warp_arrive(&m.bars[WB_UFREE]);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const GeluPair r = gelu_pair(f2_add(f2_pack(v[2 * j], v[2 * j + 1]), b1));
          const float2 wj = *(const float2*)(wt + 2 * j);
          g[j] = f2_mul(gelu_slope(r), f2_pack(wj.x, wj.y));
          if (DOT) z[j] = r.z;
        }
      }
      ok = ok && mbar_wait(&m.bars[WB_ZFULL + b], (i >> 1) & 1);
      tc_fence_after();
      uint32_t rows[16];                           // du of slots 2j, 2j + 1, rounded
      float dot[DOT ? 32 : 1];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float y[16];
        tmem_ld16(tZ + b * 128 + hf * 16, y);
        uint32_t pk[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint64_t dz = f2_pack(y[2 * j], y[2 * j + 1]);
          if (DOT) f2_unpack(f2_mul(dz, z[hf * 8 + j]), dot[hf * 16 + 2 * j], dot[hf * 16 + 2 * j + 1]);
          const uint64_t du = f2_mul(dz, g[hf * 8 + j]);
          db1 = f2_add(db1, du);
          split_pair(du, pk[j], pk[8 + j]);
          rows[hf * 8 + j] = pk[j];
        }
        tmem_st16(tZ + b * 128 + hf * 16, pk);
      }
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(&m.bars[WB_READY + b]);
      if (w.du && real) {
        // two lanes exchange halves, so that each stores two neighbouring
        // units of one slot: the even lane slot 2j, the odd one slot 2j + 1
        // (unit by unit, 16 bytes a lane, took twice as long: a line a lane)
        __nv_bfloat16* o = w.du + (long long)(at + sg * 32 + (lane & 1)) * d + (h & ~1);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const uint32_t other = __shfl_xor_sync(~0u, rows[j], 1);
          *(uint32_t*)(o + (long long)j * 2 * d) =
              lane & 1 ? __byte_perm(other, rows[j], 0x7632) : __byte_perm(rows[j], other, 0x5410);
        }
      }
      if (DOT) {
        const float s = reduce_slots(dot);
        w.dot[(long long)(at + sg * 32 + lane) * (cfg.chunks * 4) + chunk * 4 + q4] = s;
      }
    }
    ok = ok && mbar_wait(&m.bars[WB_ACCFULL], p & 1);
    tc_fence_after();
    float* out = piece_at(w.p1, slice, t);
    for (int c0 = sg * 16; c0 < a.e; c0 += 64) {
      float v[16];
      tmem_ld16(tW1 + c0, v);
      if (real && ok) {
        float4* o = (float4*)(out + (long long)h * a.e + c0);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      }
    }
    tc_fence_before();
    // db1: the four slot groups, through W1's tile (its products are done, and
    // the next weights wait for the accumulators to be free)
    float* red = (float*)m.w1;
    float x, y;
    f2_unpack(db1, x, y);
    red[sg * 128 + q4 * 32 + lane] = x + y;
    asm volatile("bar.sync 2, 512;" ::: "memory");
    if (sg == 0 && real && ok) {
      const float* r = red + q4 * 32 + lane;
      out[(long long)d * a.e + h] = (r[0] + r[128]) + (r[256] + r[384]);
    }
    asm volatile("bar.sync 2, 512;" ::: "memory");
    fence_async_smem();            // the weights that follow are written by TMA
    warp_arrive(&m.bars[WB_ACCFREE]);
    ++p;
  }
}

template <int NC>
__device__ inline void wg_compute2(const RoutedTcArgs& a, const WgCfg& cfg, const WgShared& m, const WgArgs& w,
                                   uint32_t tmem, int tile0, int tile1, int chunk, int slice) {
  constexpr int d = NC * 64, NBU = d <= 256 ? 2 : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q4 = warp & 3, sg = warp >> 2;
  const int h = chunk * 128 + q4 * 32 + lane;
  const bool real = chunk * 128 + q4 * 32 < d;
  const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
  const uint32_t tW2 = tmem + lane_base, tU = tmem + (NBU == 2 ? 256 : 384) + lane_base + sg * 32;
  bool ok = true;
  int i = 0, p = 0;
  const int oc = chunk * 16 + (threadIdx.x & 15), og = threadIdx.x >> 4;   // db2: 8 output columns, 2 slots of a unit
  RingPos u, er, yr;
  for (int t = 0; t < a.plan.T; ++t) {
    int lo, hi;
    if (!wg_piece(m.spans, tile0, tile1, t, lo, hi)) continue;
    const float b1s = real ? __bfloat162float(((const __nv_bfloat16*)a.mlp.b1[t])[h]) : 0.f;
    const uint64_t b1 = f2_pack(b1s, b1s);
    float db2[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int at = lo; at < hi; at += 128, ++i) {
      ok = ok && mbar_wait(&m.bars[WB_EFULL + er.s], er.ph);   // the choice weights
      ok = ok && mbar_wait(&m.bars[WB_UFULL + u.s], u.ph);
      tc_fence_after();
      const float* wt = m.wt + er.s * 128;
      const uint32_t from = tU + u.s * 128;
      {
        float v[32];
        tmem_ld32(from, v);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int n = hf * 16 + 2 * j;
            const GeluPair r = gelu_pair(f2_add(f2_pack(v[n], v[n + 1]), b1));
            const float2 wj = *(const float2*)(wt + sg * 32 + n);
            split_pair(f2_mul(r.z, f2_pack(wj.x, wj.y)), pk[j], pk[8 + j]);
          }
          tmem_st16(from + hf * 16, pk);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(&m.bars[WB_READY + u.s]);
      u.next(NBU);
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {             // db2 from the DY units, before they are freed
        ok = ok && mbar_wait(&m.bars[WB_YFULL + yr.s], yr.ph);
        if (oc * 8 < d) {
          const uint8_t* box = m.y + yr.s * (d * 128) + (oc >> 3) * 8192;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int r = og * 2 + j;
            const uint4 x = *(const uint4*)(box + r * 128 + (((oc & 7) ^ (r & 7)) << 4));
            const __nv_bfloat162* xh = (const __nv_bfloat162*)&x;
            const float wr = wt[hf * 64 + r];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              const float2 f = __bfloat1622float2(xh[n]);
              db2[2 * n] = fmaf(wr, f.x, db2[2 * n]);
              db2[2 * n + 1] = fmaf(wr, f.y, db2[2 * n + 1]);
            }
          }
        }
        warp_arrive(&m.bars[WB_YEMPTY + yr.s]);
        yr.next(cfg.units2);
      }
      warp_arrive(&m.bars[WB_EEMPTY + er.s]);      // the choice weights have been used
      er.next(cfg.ebuf);
    }
    // the piece's sums: dW2 [o][h] with neighbouring lanes on neighbouring h
    ok = ok && mbar_wait(&m.bars[WB_ACCFULL], p & 1);
    tc_fence_after();
    float* out = piece_at(w.p2, slice, t);
    for (int c0 = sg * 32; c0 < d; c0 += 128) {
      float v[32];
      tmem_ld32(tW2 + c0, v);
      if (real && ok)
#pragma unroll
        for (int j = 0; j < 32; ++j) out[(long long)(c0 + j) * d + h] = v[j];
    }
    tc_fence_before();
    float* red = (float*)m.w1;     // [32][128]; W1's products are done, the next weights wait for ACCFREE
#pragma unroll
    for (int n = 0; n < 8; ++n) red[og * 128 + (threadIdx.x & 15) * 8 + n] = db2[n];
    asm volatile("bar.sync 2, 512;" ::: "memory");
    if (threadIdx.x < 128 && chunk * 128 + threadIdx.x < d && ok) {
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < 32; ++n) sum += red[n * 128 + threadIdx.x];
      out[(long long)d * d + chunk * 128 + threadIdx.x] = sum;
    }
    asm volatile("bar.sync 2, 512;" ::: "memory");
    fence_async_smem();
    warp_arrive(&m.bars[WB_ACCFREE]);
    ++p;
  }
}

template <int NC, bool DOT>
__global__ void __launch_bounds__(kWgThreads, 1)
    routed_wgrad_kernel(const __grid_constant__ RoutedMaps maps, const RoutedTcArgs a, const WgArgs w) {
  constexpr int d = NC * 64;
  extern __shared__ __align__(1024) uint8_t smem[];
  const WgCfg cfg = wg_cfg(a.e, d);
  WgShared m;
  m.w1 = smem;
  m.e = m.w1 + cfg.w1_bytes;
  m.w2 = m.e + cfg.ebuf * cfg.e_bytes;
  m.off = (long long*)(m.w2 + cfg.ring);
  m.row = (int*)(m.off + 256);
  m.wt = (float*)(m.row + 3 * 128);
  m.bars = (uint64_t*)(m.wt + 3 * 128);
  m.spans = (PlanSpans*)(m.bars + WB_SPANS);
  if (smem_u32(smem) & 1023) {
    if (threadIdx.x == 0) flag_error(kErrSmemAlign);
    return;
  }
  const int warp = threadIdx.x >> 5;
  // role 1 takes the first CTAs: chunk after chunk of every slice
  const int n1 = cfg.chunks * w.p1.slices;
  const bool role1 = (int)blockIdx.x < n1;
  const int id = role1 ? blockIdx.x : blockIdx.x - n1;
  const int chunk = id % cfg.chunks, slice = id / cfg.chunks;
  m.y = role1 ? m.w2 + d * 256 : m.w2;
  uint32_t* tmem_slot = (uint32_t*)(m.bars + WB_TMEM);
  if (threadIdx.x == 0) {
    auto init = [&](int bar, int n, int count) {
      for (int i = 0; i < n; ++i) mbar_init(&m.bars[bar + i], count);
    };
    init(WB_EFULL, 3, 64 + 2);     // every gather thread's copies, every gather warp's stores of the weights
    init(WB_EEMPTY, 3, role1 ? 1 : 1 + kWgCompute);
    init(WB_YFULL, 8, 128);
    init(WB_YEMPTY, 8, role1 ? 1 : 1 + kWgCompute);
    init(WB_UFULL, 2, 1);
    init(WB_UFREE, 2, kWgCompute);
    init(WB_ZFULL, 2, 1);
    init(WB_READY, 2, kWgCompute);
    init(WB_USED, 2, 1);
    init(WB_W, 1, 1);
    init(WB_ACCFULL, 1, 1);
    init(WB_ACCFREE, 1, kWgCompute);
    fence_barrier_init();
  }
  if (warp == 22) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dep_wait();
  grid_dep_launch();
  load_spans(a.plan, m.spans);
  const WeightPieces& wp = role1 ? w.p1 : w.p2;
  const int tile0 = slice * wp.per, tile1 = min(tile0 + wp.per, m.spans->first[a.plan.T] / 128);

  if (warp >= 22) {
    if (role1) wg_products1<NC>(maps, chunk, a, cfg, m, tmem, tile0, tile1, warp == 22);
    else wg_products2<NC>(maps, chunk, a, cfg, m, tmem, tile0, tile1, warp == 22);
  } else if (warp >= kWgCompute + 4) {
    wg_gather_events(a, cfg, m, tile0, tile1);
  } else if (warp >= kWgCompute) {
    if (role1) wg_gather<NC, true>(a, cfg, m, tile0, tile1);
    else wg_gather<NC, false>(a, cfg, m, tile0, tile1);
  } else {
    if (role1) wg_compute1<NC, DOT>(a, cfg, m, w, tmem, tile0, tile1, chunk, slice);
    else wg_compute2<NC>(a, cfg, m, w, tmem, tile0, tile1, chunk, slice);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 22) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------ event gradient --
// DE = du W1 (M = 128 slots, N = e, K = d) from the rows of du that the
// weight-gradient kernel left, tile by tile; out to the events' rows (k = 1)
// or to part.  Bound by reading du (2 d bytes a slot, most of it still in L2):
// 75392 slots (d 256, e 64) 12.5 us, 3.9 TB/s.
// Warps 0-3 output, 4-7 load du, 8 loads weights, 9 products.
constexpr int kDevThreads = 320;

struct DevCfg {
  int w_bytes, units, smem;                      // W1 of one behaviour, ring of [128 slots x 64] boxes
};
__host__ __device__ inline DevCfg dev_cfg(int e, int d) {
  DevCfg c;
  c.w_bytes = (e + 63) / 64 * d * 128;
  c.units = (kSmemMax - 1024 - c.w_bytes) / 16384;
  if (c.units > 8) c.units = 8;
  c.smem = 1024 + c.w_bytes + c.units * 16384;
  return c;
}

template <int NC>
__global__ void __launch_bounds__(kDevThreads, 1)
    routed_devents_kernel(const __grid_constant__ RoutedMaps maps, const RoutedTcArgs a, const __nv_bfloat16* __restrict__ du) {
  constexpr int d = NC * 64;
  extern __shared__ __align__(1024) uint8_t smem[];
  const DevCfg cfg = dev_cfg(a.e, d);
  uint8_t* sW = smem;
  uint8_t* sA = sW + cfg.w_bytes;
  uint64_t* bars = (uint64_t*)(sA + cfg.units * 16384);
  uint64_t* a_full = bars;           // [8]
  uint64_t* a_empty = bars + 8;      // [8]
  uint64_t* e_full = bars + 16;      // [2]
  uint64_t* e_empty = bars + 18;     // [2]
  uint64_t* w_full = bars + 20;
  uint64_t* w_empty = bars + 21;
  uint32_t* tmem_slot = (uint32_t*)(bars + 22);
  PlanSpans* spans = (PlanSpans*)(bars + 24);
  if (smem_u32(smem) & 1023) {
    if (threadIdx.x == 0) flag_error(kErrSmemAlign);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < cfg.units; ++i) {
      mbar_init(&a_full[i], 128);
      mbar_init(&a_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&e_full[i], 1);
      mbar_init(&e_empty[i], 4);
    }
    mbar_init(w_full, 1);
    mbar_init(w_empty, 1);
    fence_barrier_init();
  }
  if (warp == 9) tmem_alloc(tmem_slot, 256);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dep_wait();
  grid_dep_launch();
  const bool fine = load_spans(a.plan, spans);
  const int T = a.plan.T, n_tiles = spans->first[T] / 128;
  // neighbouring tiles to one CTA: its weights change only between behaviours
  const int per = (n_tiles + gridDim.x - 1) / gridDim.x;
  const int t0 = blockIdx.x * per, t1 = min(t0 + per, n_tiles);

  if (warp == 8) {
    if (lane == 0) {
      const uint64_t keep = l2_evict_last();
      int prev = -1, p = 0;
      for (int tile = t0; tile < t1; ++tile) {
        const int t = span_type(spans, T, tile * 128);
        if (t == prev) continue;
        if (p > 0 && !mbar_wait(w_empty, (p - 1) & 1)) break;
        prev = t;
        ++p;
        mbar_expect_tx(w_full, cfg.w_bytes);
        for (int b = 0; b * 64 < a.e; ++b)
          for (int c = 0; c < NC; ++c)
            tma_load_3d_hint(&maps.w1[t], w_full, sW + b * (d * 128) + c * 8192, b * 64, c * 64, 0, keep);
      }
    }
  } else if (warp == 9) {
    const uint64_t dA = sdesc_k128(smem_u32(sA)), dW = sdesc_mn128(smem_u32(sW), d * 128);
    const uint32_t id_e = idesc_bf16(128, a.e, false, true);
    bool ok = true;
    RingPos r;
    int prev = -1, p = 0, i = 0;
    for (int tile = t0; tile < t1 && ok; ++tile, ++i) {
      const int t = span_type(spans, T, tile * 128);
      if (t != prev) {
        if (p > 0) mma_commit(w_empty);      // the last behaviour's products
        ok = mbar_wait_warp(w_full, p & 1);
        prev = t;
        ++p;
      }
      if (i >= 2) ok = ok && mbar_wait_warp(&e_empty[i & 1], ((i >> 1) & 1) ^ 1);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        ok = ok && mbar_wait_warp(&a_full[r.s], r.ph);
        if (!ok) break;
        fence_async_smem();
        tc_fence_after();
        const uint64_t da = desc_add(dA, r.s * 16384);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_ss(tmem + (i & 1) * 128, desc_add(da, k * 32), desc_add(dW, c * 8192 + k * 2048), id_e, (c | k) ? 1u : 0u);
        mma_commit(&a_empty[r.s]);
        r.next(cfg.units);
      }
      mma_commit(&e_full[i & 1]);
    }
  } else if (warp >= 4) {
    const GatherLane g(threadIdx.x - 128);
    bool ok = true, wrapped = false;
    RingPos r;
    for (int tile = t0; tile < t1; ++tile) {
      const __nv_bfloat16* p[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] = du + ((long long)tile * 128 + g.r8 + 16 * j) * d + g.c * 8;
#pragma unroll 1
      for (int c = 0; c < NC; ++c) {
        if (wrapped) ok = ok && mbar_wait(&a_empty[r.s], r.ph ^ 1);
        if (ok) gather_box<128>(g, sA + r.s * 16384, p, 0xffu, c * 64);
        cp_async_arrive(&a_full[r.s]);
        r.next(cfg.units);
        wrapped = wrapped || r.s == 0;
      }
    }
    if (fine && a.devents)
      zero_unrouted(a.plan, a.devents, TokenRows{0x7fffffff, 0}, a.e, blockIdx.x * 4 + warp - 4, gridDim.x * 4);
  } else {
    const uint32_t lb = (uint32_t)(warp * 32) << 16;
    bool ok = true;
    int i = 0;
    for (int tile = t0; tile < t1; ++tile, ++i) {
      const int flat = a.plan.order[(long long)tile * 128 + warp * 32 + lane];
      ok = ok && mbar_wait(&e_full[i & 1], (i >> 1) & 1);
      tc_fence_after();
      const uint32_t from = tmem + (i & 1) * 128 + lb;
      for (int c0 = 0; c0 < a.e; c0 += 16) {
        float v[16];
        tmem_ld16(from + c0, v);
        if (flat < 0 || !ok) continue;
        if (a.part) {
          float4* o = (float4*)(a.part + (long long)flat * a.e + c0);
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        } else {
          uint4* o = (uint4*)(a.devents + (long long)flat * a.e + c0);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            o[j] = make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                              pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
        }
      }
      tc_fence_before();
      warp_arrive(&e_empty[i & 1]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) tmem_dealloc(tmem, 256);
}

}  // namespace ot
