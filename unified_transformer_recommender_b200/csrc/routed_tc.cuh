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
  __nv_bfloat16* devents;        // k = 1, or null
  float* dweights;               // [R*k] or null
  float* part;                   // k > 1: [R*k][d] of the tokens, [R*k][e] of the event gradient (or null)
};

constexpr int kSmemMax = 232448;

__device__ inline void cp_async16(void* dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
__device__ inline void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ inline void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ inline void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// The product warps run their loops with all 32 lanes and let one elected lane
// issue: control flow and descriptors then stay warp-uniform, and the
// descriptors in uniform registers, where the tensor-core instructions want
// them (a branch on the lane number costs a register move per operand).
// elect.sync picks the same lane every time, so a commit covers the products
// that lane issued.
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

// Rows of `width` bf16 elements (a multiple of 8, up to 64 NB) into NB boxes
// of [rows x 64 columns] with the 128-byte swizzle; columns past the width and
// rows with a negative offset become zero.  off(r): element offset of row r.
// NT threads; the copies stay in flight.
template <int NT, int NB, typename Off>
__device__ inline void gather_boxes(uint8_t* tile, Off off, int rows, int width, const __nv_bfloat16* src, int tid) {
  for (int i = tid; i < rows * NB * 8; i += NT) {
    const int r = i / (NB * 8), c = i - r * (NB * 8);   // row, 16-byte chunk
    const long long o = off(r);
    const bool on = o >= 0 && c * 8 < width;
    cp_async16(tile + (c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4), src + (on ? o + c * 8 : 0), on);
  }
}
// Event rows by index (shared memory, -1: none).
template <int NT>
__device__ inline void gather_events(uint8_t* tile, const int* row, int rows, int width, const __nv_bfloat16* src,
                                     int tid) {
  auto off = [&](int r) { return (long long)row[r] * width; };
  if (width <= 64) gather_boxes<NT, 1>(tile, off, rows, width, src, tid);
  else gather_boxes<NT, 2>(tile, off, rows, width, src, tid);
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
// hidden row therefore never leaves the SM.  Two U buffers let the next
// chunk's first product run during this one's GELU; the weights stream
// through a ring (the tiles of one behaviour read the same 2 d (e + d) bytes,
// which stay in L2).  The gathered event rows come through cp.async into the
// swizzled operand layout; four warps of their own take D out, weighted, as
// 128-byte pieces of the destination rows, while the next tile's first
// hidden units are computed.
// Warps 0-7 GELU, 8-11 output, 12-15 gather, 16 weights, 17 products.
constexpr int kTokThreads = 576, kTokGelu = 8, kTokOut = 4;

struct TokCfg {
  int ebuf, stages;               // event tiles and weight stages in flight
  int e_bytes, w1_bytes, stage_bytes, smem;
};
__host__ __device__ inline TokCfg tok_cfg(int e, int d) {
  TokCfg c;
  const int eb = (e + 63) / 64;   // 64-column boxes of an event row
  c.e_bytes = eb * 16384;
  c.w1_bytes = eb * 8192;
  c.stage_bytes = c.w1_bytes + d * 128;
  // output staging, biases of two tiles, row indices, barriers and spans
  const int fixed = kTokOut * 32 * 144 + 4 * d * 4 + 128 * 4 + 512;
  const int room = kSmemMax - fixed;
  c.ebuf = eb == 1 ? 2 : 1;
  c.stages = (room - c.ebuf * c.e_bytes) / c.stage_bytes;
  if (c.stages > 4) c.stages = 4;
  c.smem = fixed + c.ebuf * c.e_bytes + c.stages * c.stage_bytes;
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
  uint8_t* sOut = sW + cfg.stages * cfg.stage_bytes;
  float* sBias = (float*)(sOut + kTokOut * 32 * 144);       // [2][2 d]
  int* sRow = (int*)(sBias + 4 * d);                        // [128]
  uint64_t* bars = (uint64_t*)(sRow + 128);
  uint64_t* e_full = bars;          // [2]
  uint64_t* e_empty = bars + 2;     // [2]
  uint64_t* w_full = bars + 4;      // [4]
  uint64_t* w_empty = bars + 8;     // [4]
  uint64_t* u_full = bars + 12;     // [2]
  uint64_t* z_ready = bars + 14;    // [2]
  uint64_t* dn_done = bars + 16;    // [2]
  uint64_t* b_free = bars + 18;     // [2]: a tile's biases have been used
  uint64_t* d_full = bars + 20;
  uint64_t* d_empty = bars + 21;
  uint64_t* b_full = bars + 22;     // [2]
  uint32_t* tmem_slot = (uint32_t*)(bars + 24);
  PlanSpans* spans = (PlanSpans*)(bars + 26);

  if (smem_u32(smem) & 1023) {
    if (threadIdx.x == 0) flag_error(kErrSmemAlign);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&e_full[i], 4);
      mbar_init(&e_empty[i], 1);
      mbar_init(&u_full[i], 1);
      mbar_init(&z_ready[i], kTokGelu);
      mbar_init(&dn_done[i], 1);
      mbar_init(&b_full[i], 4);
      mbar_init(&b_free[i], kTokGelu + kTokOut);
    }
    for (int i = 0; i < cfg.stages; ++i) {
      mbar_init(&w_full[i], 1);
      mbar_init(&w_empty[i], 1);
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
  const uint32_t tD = tmem, tU = tmem + 384;   // U buffers at 384 and 448
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
          ok = !wrapped || mbar_wait(&w_empty[w.s], w.ph ^ 1);
          if (!ok) break;
          uint8_t* w1 = sW + w.s * cfg.stage_bytes;
          mbar_expect_tx(&w_full[w.s], cfg.stage_bytes);
          tma_load_3d_hint(&maps.w1[t], &w_full[w.s], w1, 0, c * 64, 0, keep);
          if (cfg.w1_bytes > 8192) tma_load_3d_hint(&maps.w1[t], &w_full[w.s], w1 + 8192, 64, c * 64, 0, keep);
#pragma unroll
          for (int b = 0; b < NC; ++b)
            tma_load_3d_hint(&maps.w2[t], &w_full[w.s], w1 + cfg.w1_bytes + b * 8192, c * 64, b * 64, 0, keep);
          w.next(cfg.stages);
          wrapped = wrapped || w.s == 0;
        }
      }
    }
  } else if (warp == 17) {
    // ------------------------------------------------------------- products
    {
      const uint64_t dE = sdesc_k128(smem_u32(sE)), dW = sdesc_k128(smem_u32(sW));
      constexpr uint32_t id_u = idesc_bf16(128, 64);
      constexpr int n0 = d > 256 ? 256 : d, n1 = d - n0;
      constexpr uint32_t id_0 = idesc_bf16(128, n0), id_1 = idesc_bf16(128, n1 ? n1 : 16);
      const int ksteps = a.e / 16;
      const int mine = n_tiles > (int)blockIdx.x ? (n_tiles - 1 - (int)blockIdx.x) / step + 1 : 0;
      const int total = mine * NC;
      bool ok = true;
      RingPos wu, wd, eu;           // weight stage of the next up / down product, event tile of the next up
      int gu = 0, cu = 0, cd = 0, tiles_done = 0;
      auto up = [&]() {
        ok = ok && mbar_wait(&w_full[wu.s], wu.ph);
        if (cu == 0) ok = ok && mbar_wait(&e_full[eu.s], eu.ph);
        if (gu >= 2) ok = ok && mbar_wait(&dn_done[gu & 1], ((gu >> 1) & 1) ^ 1);   // z of two chunks before consumed
        if (!ok) return;
        tc_fence_after();
        const uint64_t de = desc_add(dE, eu.s * cfg.e_bytes), dw = desc_add(dW, wu.s * cfg.stage_bytes);
        const uint32_t to = tU + (gu & 1) * 64;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < ksteps)
            mma_ss(to, desc_add(de, (k >> 2) * 16384 + (k & 3) * 32), desc_add(dw, (k >> 2) * 8192 + (k & 3) * 32), id_u,
                      k ? 1u : 0u);
        mma_commit(&u_full[gu & 1]);
        if (++cu == NC) {
          cu = 0;
          mma_commit(&e_empty[eu.s]);
          eu.next(cfg.ebuf);
        }
        wu.next(cfg.stages);
        ++gu;
      };
      if (total > 0) up();
      for (int g = 0; g < total && ok; ++g) {
        if (g + 1 < total) up();
        ok = ok && mbar_wait(&z_ready[g & 1], (g >> 1) & 1);
        if (cd == 0 && tiles_done > 0) ok = ok && mbar_wait(d_empty, (tiles_done - 1) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint64_t w2 = desc_add(dW, wd.s * cfg.stage_bytes + cfg.w1_bytes);
#pragma unroll
        for (int k = 0; k < 4; ++k) {   // units 16k .. 16k+15 packed over U columns 16k .. 16k+7
          const uint32_t z = tU + (g & 1) * 64 + k * 16;
          mma_ts(tD, z, desc_add(w2, k * 32), id_0, (cd | k) ? 1u : 0u);
          if (n1) mma_ts(tD + n0, z, desc_add(w2, n0 * 128 + k * 32), id_1, (cd | k) ? 1u : 0u);
        }
        mma_commit(&w_empty[wd.s]);
        mma_commit(&dn_done[g & 1]);
        if (++cd == NC) {
          cd = 0;
          ++tiles_done;
          mma_commit(d_full);
        }
        wd.next(cfg.stages);
      }
    }
  } else if (warp >= 12) {
    // --------------------------------------------------------------- gather
    const int tid = threadIdx.x - 12 * 32;
    bool ok = true;
    RingPos e;
    int i = 0;
    int flat = (int)blockIdx.x < n_tiles ? a.plan.order[(long long)blockIdx.x * 128 + tid] : -1;
    for (int tile = blockIdx.x; tile < n_tiles; tile += step, ++i) {
      if (i >= cfg.ebuf) ok = ok && mbar_wait(&e_empty[e.s], e.ph ^ 1);
      sRow[tid] = flat < 0 ? -1 : flat / a.plan.k;
      asm volatile("bar.sync 1, 128;" ::: "memory");
      if (ok) gather_events<128>(sE + e.s * cfg.e_bytes, sRow, 128, a.e, a.events, tid);
      if (tile + step < n_tiles) flat = a.plan.order[(long long)(tile + step) * 128 + tid];
      if (i >= 2) ok = ok && mbar_wait(&b_free[i & 1], ((i >> 1) & 1) ^ 1);
      load_biases(sBias + (i & 1) * 2 * d, a.mlp, span_type(spans, T, tile * 128), d, tid, 128);
      warp_arrive(&b_full[i & 1]);
      cp_async_commit();
      cp_async_wait<0>();
      fence_async_smem();
      asm volatile("bar.sync 1, 128;" ::: "memory");   // sRow free again
      warp_arrive(&e_full[e.s]);
      e.next(cfg.ebuf);
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
    const uint32_t col = tU + ((uint32_t)(q4 * 32) << 16) + wq * 32;
    bool ok = true;
    int i = 0, g = 0;
    for (int tile = blockIdx.x; tile < n_tiles; tile += step, ++i) {
      const float* b1 = sBias + (i & 1) * 2 * d + wq * 32;
      ok = ok && mbar_wait(&b_full[i & 1], (i >> 1) & 1);
#pragma unroll 1
      for (int c = 0; c < NC; ++c, ++g) {
        ok = ok && mbar_wait(&u_full[g & 1], (g >> 1) & 1);
        tc_fence_after();
        float v[32];
        tmem_ld32(col + (g & 1) * 64, v);
        uint32_t pk[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 b = *(const float4*)(b1 + c * 64 + j * 4);
          pk[2 * j] = gelu_bias_bf16x2(v[4 * j], v[4 * j + 1], b.x, b.y);
          pk[2 * j + 1] = gelu_bias_bf16x2(v[4 * j + 2], v[4 * j + 3], b.z, b.w);
        }
        tmem_st8(col + (g & 1) * 64, pk);
        tmem_st8(col + (g & 1) * 64 + 16, pk + 8);
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&z_ready[g & 1]);
      }
      warp_arrive(&b_free[i & 1]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 17) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------- shared, backward --
// GELU-tanh and its slope to float32 accuracy: with s = 1 / (1 + exp(-2v)),
// v = c (u + a u^3), GELU(u) = u s and d/du = s + 2 u s (1 - s) c (1 + 3 a u^2)
// (0.5 (1 + tanh v) = s).  Two special-function results per value (exp, the
// reciprocal); |v| large gives s = 0 or 1 exactly.
__device__ inline void gelu_and_slope_fast(float u, float& z, float& g) {
  const float c = 0.7978845608028654f, a = 0.044715f;
  const float u2 = u * u;
  const float v = u * fmaf(c * a, u2, c);
  const float s = __fdividef(1.f, 1.f + __expf(-2.f * v));
  z = u * s;
  // at |u| past 10 the second term is zero, but u2 * (1 - s) could be inf * 0
  const float q = fmaf(6.f * c * a, u2, 2.f * c);
  g = fabsf(u) < 16.f ? fmaf(z * (1.f - s), q, s) : s;
}
// x0, x1 as bf16 pairs hi + lo: 16 bits of significand in two operands.
__device__ inline void split_bf16x2(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(x0, x1);
  lo = pack_bf16x2(x0 - __uint_as_float(hi << 16), x1 - __uint_as_float(hi & 0xffff0000u));
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

// ------------------------------------------------------------ event gradient --
// de = W1^T du and dw, tile by tile like the forward: per 64 hidden units
// U = E W1c^T (K = e) and DZ = DY W2c (K = d) into TMEM, du = w dz GELU'(u) by
// eight warps, split into two bf16 terms over U's columns, DE += du W1c.
// W1's chunk serves both of its products from one shared-memory tile (K-major
// for U, MN-major for DE), as W2's does in the forward.  dw's row sums stay
// with the threads that own the row.
// Warps 0-7 GELU, 8-11 output, 12-15 gather, 16 weights, 17 products.
struct DevCfg {
  int abuf, units;                // row tiles in flight, W2 units of 64 rows
  int a_bytes, w1_bytes, smem;
};
constexpr int kDevW1 = 2;         // W1 stages
__host__ __device__ inline DevCfg dev_cfg(int e, int d) {
  DevCfg c;
  const int eb = (e + 63) / 64;
  c.a_bytes = d * 256 + eb * 16384;              // dtoken rows, then event rows
  c.w1_bytes = eb * 8192;
  const int fixed = 512 + 512 + 1024 + 512;      // barriers and spans, dw partials, row offsets and indices
  const int bias = 4 * d * 4;
  const int room = kSmemMax - fixed - bias - kDevW1 * c.w1_bytes;
  c.abuf = room >= 2 * c.a_bytes + 4 * 8192 ? 2 : 1;
  c.units = (room - c.abuf * c.a_bytes) / 8192;
  if (c.units > 12) c.units = 12;
  c.smem = fixed + bias + c.abuf * c.a_bytes + kDevW1 * c.w1_bytes + c.units * 8192;
  return c;
}

template <int NC>
__global__ void __launch_bounds__(kTokThreads, 1)
    routed_devents_kernel(const __grid_constant__ RoutedMaps maps, const RoutedTcArgs a) {
  constexpr int d = NC * 64;
  extern __shared__ __align__(1024) uint8_t smem[];
  const DevCfg cfg = dev_cfg(a.e, d);
  uint8_t* sA = smem;
  uint8_t* sW1 = sA + cfg.abuf * cfg.a_bytes;
  uint8_t* sW2 = sW1 + kDevW1 * cfg.w1_bytes;
  float* sBias = (float*)(sW2 + cfg.units * 8192);   // [2][2 d]
  long long* sOff = (long long*)(sBias + 4 * d);     // [128]
  int* sRow = (int*)(sOff + 128);                    // [128]
  float* sDot = (float*)(sRow + 128);                // [128]
  uint64_t* bars = (uint64_t*)(sDot + 128);
  uint64_t* a_full = bars;           // [2]
  uint64_t* a_empty = bars + 2;      // [2]
  uint64_t* w1_full = bars + 4;      // [2]
  uint64_t* w1_empty = bars + 6;     // [2]
  uint64_t* w2_full = bars + 8;      // [12]
  uint64_t* w2_empty = bars + 20;    // [12]
  uint64_t* u_full = bars + 32;      // [2]
  uint64_t* du_ready = bars + 34;    // [2]
  uint64_t* du_done = bars + 36;     // [2]
  uint64_t* de_full = bars + 38;     // [2]
  uint64_t* de_empty = bars + 40;    // [2]
  uint64_t* b_free = bars + 42;      // [2]
  uint64_t* b_full = bars + 44;      // [2]
  uint32_t* tmem_slot = (uint32_t*)(bars + 46);
  PlanSpans* spans = (PlanSpans*)(bars + 48);

  if (smem_u32(smem) & 1023) {
    if (threadIdx.x == 0) flag_error(kErrSmemAlign);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&a_full[i], 4);
      mbar_init(&a_empty[i], 1 + kTokGelu);
      mbar_init(&w1_full[i], 1);
      mbar_init(&w1_empty[i], 1);
      mbar_init(&u_full[i], 1);
      mbar_init(&du_ready[i], kTokGelu);
      mbar_init(&du_done[i], 1);
      mbar_init(&de_full[i], 1);
      mbar_init(&de_empty[i], kTokOut);
      mbar_init(&b_full[i], 4);
      mbar_init(&b_free[i], kTokGelu);
    }
    for (int i = 0; i < cfg.units; ++i) {
      mbar_init(&w2_full[i], 1);
      mbar_init(&w2_empty[i], 1);
    }
    fence_barrier_init();
  }
  if (warp == 17) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tE = tmem, tU = tmem + 256, tZ = tmem + 384;   // two buffers each of DE (128), U, DZ (64 columns)
  grid_dep_wait();
  grid_dep_launch();
  const bool fine = load_spans(a.plan, spans);
  const int T = a.plan.T, n_tiles = spans->first[T] / 128;
  const int step = gridDim.x;

  if (warp == 16) {
    // ------------------------------------------------------ weight producer
    if (lane == 0) {
      const uint64_t keep = l2_evict_last();
      RingPos w1, w2;
      bool wrap1 = false, wrap2 = false, ok = true;
      for (int tile = blockIdx.x; tile < n_tiles && ok; tile += step) {
        const int t = span_type(spans, T, tile * 128);
        for (int c = 0; c < NC && ok; ++c) {
          ok = !wrap1 || mbar_wait(&w1_empty[w1.s], w1.ph ^ 1);
          if (!ok) break;
          uint8_t* to = sW1 + w1.s * cfg.w1_bytes;
          mbar_expect_tx(&w1_full[w1.s], cfg.w1_bytes);
          tma_load_3d_hint(&maps.w1[t], &w1_full[w1.s], to, 0, c * 64, 0, keep);
          if (cfg.w1_bytes > 8192) tma_load_3d_hint(&maps.w1[t], &w1_full[w1.s], to + 8192, 64, c * 64, 0, keep);
          w1.next(kDevW1);
          wrap1 = wrap1 || w1.s == 0;
          for (int b = 0; b < NC; ++b) {
            ok = !wrap2 || mbar_wait(&w2_empty[w2.s], w2.ph ^ 1);
            if (!ok) break;
            mbar_expect_tx(&w2_full[w2.s], 8192);
            tma_load_3d_hint(&maps.w2[t], &w2_full[w2.s], sW2 + w2.s * 8192, c * 64, b * 64, 0, keep);
            w2.next(cfg.units);
            wrap2 = wrap2 || w2.s == 0;
          }
        }
      }
    }
  } else if (warp == 17) {
    // ------------------------------------------------------------- products
    {
      const uint64_t dA = sdesc_k128(smem_u32(sA)), dW1 = sdesc_k128(smem_u32(sW1));
      const uint64_t dW1t = sdesc_mn128(smem_u32(sW1), 8192), dW2t = sdesc_mn128(smem_u32(sW2), 8192);
      constexpr uint32_t id_u = idesc_bf16(128, 64), id_z = idesc_bf16(128, 64, false, true);
      const uint32_t id_e = idesc_bf16(128, a.e, false, true);
      const int ksteps = a.e / 16;
      const int mine = n_tiles > (int)blockIdx.x ? (n_tiles - 1 - (int)blockIdx.x) / step + 1 : 0;
      const int total = mine * NC;
      bool ok = true;
      RingPos ar, w1u, w1d, w2;
      int gu = 0, cu = 0, cd = 0, i = 0;
      auto up = [&]() {
        ok = ok && mbar_wait(&w1_full[w1u.s], w1u.ph);
        if (cu == 0) ok = ok && mbar_wait(&a_full[ar.s], ar.ph);
        if (gu >= 2) ok = ok && mbar_wait(&du_done[gu & 1], ((gu >> 1) & 1) ^ 1);
        if (!ok) return;
        tc_fence_after();
        const uint64_t da = desc_add(dA, ar.s * cfg.a_bytes), dw = desc_add(dW1, w1u.s * cfg.w1_bytes);
        const uint32_t u = tU + (gu & 1) * 64, z = tZ + (gu & 1) * 64;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < ksteps)
            mma_ss(u, desc_add(da, d * 256 + (k >> 2) * 16384 + (k & 3) * 32),
                      desc_add(dw, (k >> 2) * 8192 + (k & 3) * 32), id_u, k ? 1u : 0u);
#pragma unroll
        for (int b = 0; b < NC; ++b) {       // 64 of the contraction per W2 unit
          ok = mbar_wait(&w2_full[w2.s], w2.ph);
          if (!ok) return;
          tc_fence_after();
          const uint64_t dz = desc_add(dW2t, w2.s * 8192);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ss(z, desc_add(da, b * 16384 + k * 32), desc_add(dz, k * 2048), id_z, (b | k) ? 1u : 0u);
          mma_commit(&w2_empty[w2.s]);
          w2.next(cfg.units);
        }
        mma_commit(&u_full[gu & 1]);
        if (++cu == NC) {
          cu = 0;
          mma_commit(&a_empty[ar.s]);
          ar.next(cfg.abuf);
        }
        w1u.next(kDevW1);
        ++gu;
      };
      if (total > 0) up();
      for (int g = 0; g < total && ok; ++g) {
        // the next chunk's products run during this chunk's GELU; a new
        // tile's only after this one's last, since its rows may still be coming
        const bool same = cd + 1 < NC;
        if (same) up();
        ok = ok && mbar_wait(&du_ready[g & 1], (g >> 1) & 1);
        if (cd == 0 && i >= 2) ok = ok && mbar_wait(&de_empty[i & 1], ((i >> 1) & 1) ^ 1);
        if (!ok) break;
        tc_fence_after();
        const uint64_t w1 = desc_add(dW1t, w1d.s * cfg.w1_bytes);
        const uint32_t to = tE + (i & 1) * 128;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t du = tU + (g & 1) * 64 + k * 16;   // hi in 8 columns, lo in the next 8
          mma_ts(to, du, desc_add(w1, k * 2048), id_e, (cd | k) ? 1u : 0u);
          mma_ts(to, du + 8, desc_add(w1, k * 2048), id_e, 1u);
        }
        mma_commit(&w1_empty[w1d.s]);
        mma_commit(&du_done[g & 1]);
        w1d.next(kDevW1);
        if (++cd == NC) {
          cd = 0;
          mma_commit(&de_full[i & 1]);
          ++i;
        }
        if (!same && g + 1 < total) up();
      }
    }
  } else if (warp >= 12) {
    // --------------------------------------------------------------- gather
    const int tid = threadIdx.x - 12 * 32;
    bool ok = true;
    RingPos ar;
    int i = 0;
    int flat = (int)blockIdx.x < n_tiles ? a.plan.order[(long long)blockIdx.x * 128 + tid] : -1;
    for (int tile = blockIdx.x; tile < n_tiles; tile += step, ++i) {
      const int row = flat < 0 ? -1 : flat / a.plan.k;
      if (tile + step < n_tiles) flat = a.plan.order[(long long)(tile + step) * 128 + tid];
      if (i >= cfg.abuf) ok = ok && mbar_wait(&a_empty[ar.s], ar.ph ^ 1);
      uint8_t* at = sA + ar.s * cfg.a_bytes;
      sOff[tid] = row < 0 ? -1LL : token_off(a.rows, row, d);
      sRow[tid] = row;
      asm volatile("bar.sync 1, 128;" ::: "memory");
      if (ok) {
        gather_boxes<128, NC>(at, [&](int r) { return sOff[r]; }, 128, d, a.dtokens, tid);
        gather_events<128>(at + d * 256, sRow, 128, a.e, a.events, tid);
      }
      if (i >= 2) ok = ok && mbar_wait(&b_free[i & 1], ((i >> 1) & 1) ^ 1);
      load_biases(sBias + (i & 1) * 2 * d, a.mlp, span_type(spans, T, tile * 128), d, tid, 128);
      warp_arrive(&b_full[i & 1]);
      cp_async_commit();
      cp_async_wait<0>();
      fence_async_smem();
      asm volatile("bar.sync 1, 128;" ::: "memory");
      warp_arrive(&a_full[ar.s]);
      ar.next(cfg.abuf);
    }
    if (fine && a.devents)
      zero_unrouted(a.plan, a.devents, TokenRows{0x7fffffff, 0}, a.e, blockIdx.x * 4 + warp - 12, gridDim.x * 4);
    if (fine && a.dweights) {
      const long long n = (long long)a.plan.R * a.plan.k;
      for (long long c = (long long)blockIdx.x * 128 + tid; c < n; c += (long long)gridDim.x * 128)
        if (a.plan.pos[c] < 0) a.dweights[c] = 0.f;
    }
  } else if (warp >= 8) {
    // --------------------------------------------------------------- output
    const int q4 = warp & 3;
    const uint32_t lb = (uint32_t)(q4 * 32) << 16;
    bool ok = true;
    int i = 0;
    for (int tile = blockIdx.x; tile < n_tiles; tile += step, ++i) {
      const int flat = a.plan.order[(long long)tile * 128 + q4 * 32 + lane];
      ok = ok && mbar_wait(&de_full[i & 1], (i >> 1) & 1);
      tc_fence_after();
      const uint32_t from = tE + (i & 1) * 128 + lb;
      for (int c0 = 0; c0 < a.e; c0 += 16) {
        float v[16];
        tmem_ld16(from + c0, v);
        if (flat < 0 || !ok) continue;
        if (a.part) {
          float4* o = (float4*)(a.part + (long long)flat * a.e + c0);
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        } else if (a.devents) {
          uint4* o = (uint4*)(a.devents + (long long)flat * a.e + c0);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            o[j] = make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                              pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
        }
      }
      tc_fence_before();
      warp_arrive(&de_empty[i & 1]);
    }
  } else {
    // ----------------------------------------------------------------- GELU
    const int q4 = warp & 3, wq = warp >> 2;
    const uint32_t lb = ((uint32_t)(q4 * 32) << 16) + wq * 32;
    const int row = q4 * 32 + lane;
    bool ok = true;
    RingPos ar;
    int i = 0, g = 0;
    for (int tile = blockIdx.x; tile < n_tiles; tile += step, ++i) {
      const int flat = a.plan.order[(long long)tile * 128 + row];
      const float w = flat < 0 ? 0.f : a.weights ? a.weights[flat] : 1.f;
      const float* bias = sBias + (i & 1) * 2 * d;
      ok = ok && mbar_wait(&b_full[i & 1], (i >> 1) & 1);
      float dot = 0.f;
      if (a.dweights) {       // <dtoken, b2 + emb> over this half of the row's columns
        ok = ok && mbar_wait(&a_full[ar.s], ar.ph);
        const uint8_t* at = sA + ar.s * cfg.a_bytes + row * 128;
#pragma unroll 4
        for (int c = wq * NC * 4; c < (wq + 1) * NC * 4; ++c) {
          const uint4 x = *(const uint4*)(at + (c >> 3) * 16384 + (((c & 7) ^ (row & 7)) << 4));
          const float4 s0 = *(const float4*)(bias + d + c * 8), s1 = *(const float4*)(bias + d + c * 8 + 4);
          const __nv_bfloat162* xh = (const __nv_bfloat162*)&x;
          const float2 p0 = __bfloat1622float2(xh[0]), p1 = __bfloat1622float2(xh[1]);
          const float2 p2 = __bfloat1622float2(xh[2]), p3 = __bfloat1622float2(xh[3]);
          dot = fmaf(p0.x, s0.x, fmaf(p0.y, s0.y, fmaf(p1.x, s0.z, fmaf(p1.y, s0.w, dot))));
          dot = fmaf(p2.x, s1.x, fmaf(p2.y, s1.y, fmaf(p3.x, s1.z, fmaf(p3.y, s1.w, dot))));
        }
      }
      warp_arrive(&a_empty[ar.s]);
      ar.next(cfg.abuf);
#pragma unroll 1
      for (int c = 0; c < NC; ++c, ++g) {
        ok = ok && mbar_wait(&u_full[g & 1], (g >> 1) & 1);
        tc_fence_after();
        const uint32_t u = tU + (g & 1) * 64 + lb, z = tZ + (g & 1) * 64 + lb;
        const float* b1 = bias + c * 64 + wq * 32;
#pragma unroll
        for (int h = 0; h < 2; ++h) {       // 16 units: 8 columns of hi, 8 of lo
          float v[16], y[16];
          tmem_ld16(u + h * 16, v);
          tmem_ld16(z + h * 16, y);
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 b = *(const float2*)(b1 + h * 16 + 2 * j);
            float z0, g0, z1, g1;
            gelu_and_slope_fast(v[2 * j] + b.x, z0, g0);
            gelu_and_slope_fast(v[2 * j + 1] + b.y, z1, g1);
            dot = fmaf(y[2 * j], z0, dot);
            dot = fmaf(y[2 * j + 1], z1, dot);
            split_bf16x2(w * y[2 * j] * g0, w * y[2 * j + 1] * g1, pk[j], pk[8 + j]);
          }
          tmem_st16(u + h * 16, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&du_ready[g & 1]);
      }
      warp_arrive(&b_free[i & 1]);
      if (a.dweights) {
        if (wq == 1) sDot[row] = dot;
        asm volatile("bar.sync 2, 256;" ::: "memory");
        if (wq == 0 && flat >= 0 && ok) a.dweights[flat] = dot + sDot[row];
        asm volatile("bar.sync 2, 256;" ::: "memory");
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 17) tmem_dealloc(tmem, 512);
}

// ----------------------------------------------------------- weight gradients --
// A CTA holds 128 hidden units of one behaviour at a time and walks its slice
// of the slots, 64 per step, transposed so that hidden units are TMEM lanes:
//   U^T = W1c E^T (M = 128, N = 64, K = e), DZ^T = W2c^T DY^T (K = d);
//   z, du by eight warps, each split into two bf16 terms over the columns it
//   came from, which makes them A operands where they are:
//   dW2c^T [128][d] += z DY, dW1c [128][e] += du E (K = 64 slots).
// So the hidden rows are recomputed but never stored, db1 is a sum inside a
// thread, and the gathered rows serve as both K-major and MN-major operands.
// With d > 256 dW2c^T takes 384 TMEM columns and leaves no room for the rest:
// two CTAs share a hidden chunk, one with U, DZ and dW1c, one with U and dW2c
// (about the same number of tensor-core cycles each).
// u(i + 1) is issued once dW2(i) has read z, and GELU(i + 1) then runs during
// dW1(i) and dz(i + 1).
// Warps 0-7 compute, 8-11 gather, 12 loads weights, 13 issues the products.
constexpr int kWgThreads = 448, kWgCompute = 8;

struct WgCfg {
  int eb, chunks, roles, stages;   // hidden chunks of 128, CTAs per slice, row stages
  int w1_bytes, w2_bytes, stage_bytes, smem;
};
__host__ __device__ inline WgCfg wg_cfg(int e, int d) {
  WgCfg c;
  c.eb = (e + 63) / 64;
  c.chunks = (d + 127) / 128;
  c.roles = d > 256 ? 2 * c.chunks : c.chunks;
  c.w1_bytes = c.eb * 16384;
  c.w2_bytes = 2 * d * 128;
  c.stage_bytes = d * 128 + c.eb * 8192;
  // barriers and spans, row offsets and indices of two steps; a stage also
  // holds its 64 choice weights
  const int fixed = 512 + 2 * 64 * 12;
  c.stages = (kSmemMax - fixed - c.w1_bytes - c.w2_bytes) / (c.stage_bytes + 256);
  if (c.stages > 4) c.stages = 4;
  c.smem = fixed + c.w1_bytes + c.w2_bytes + c.stages * (c.stage_bytes + 256);
  return c;
}

template <int NC>
__global__ void __launch_bounds__(kWgThreads, 1)
    routed_wgrad_kernel(const __grid_constant__ RoutedMaps maps, const RoutedTcArgs a, const WeightPieces w) {
  constexpr int d = NC * 64;
  extern __shared__ __align__(1024) uint8_t smem[];
  const WgCfg cfg = wg_cfg(a.e, d);
  uint8_t* sW1 = smem;
  uint8_t* sW2 = sW1 + cfg.w1_bytes;
  uint8_t* sS = sW2 + cfg.w2_bytes;
  float* sWt = (float*)(sS + cfg.stages * cfg.stage_bytes);    // [stages][64] choice weights
  long long* sOff = (long long*)(sWt + cfg.stages * 64);       // [2][64] dtoken rows of two steps
  int* sRow = (int*)(sOff + 128);                              // [2][64] event rows
  uint64_t* bars = (uint64_t*)(sRow + 128);
  uint64_t* s_full = bars;           // [4]
  uint64_t* s_empty = bars + 4;      // [4]
  uint64_t* w_full = bars + 8;
  uint64_t* u_full = bars + 9;
  uint64_t* z_ready = bars + 10;
  uint64_t* z_free = bars + 11;
  uint64_t* dz_full = bars + 12;
  uint64_t* du_ready = bars + 13;
  uint64_t* du_free = bars + 14;
  uint64_t* acc_full = bars + 15;
  uint64_t* acc_empty = bars + 16;
  uint32_t* tmem_slot = (uint32_t*)(bars + 17);
  PlanSpans* spans = (PlanSpans*)(bars + 18);

  if (smem_u32(smem) & 1023) {
    if (threadIdx.x == 0) flag_error(kErrSmemAlign);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int role = blockIdx.x % cfg.roles, slice = blockIdx.x / cfg.roles;
  const int chunk = role % cfg.chunks, h0 = chunk * 128;
  const bool do1 = role < cfg.chunks;                // DZ, dW1, db1 and db2
  const bool do2 = d <= 256 || !do1;                 // dW2
  if (threadIdx.x == 0) {
    for (int i = 0; i < cfg.stages; ++i) {
      mbar_init(&s_full[i], 4);
      mbar_init(&s_empty[i], 1 + kWgCompute);
    }
    mbar_init(w_full, 1);
    mbar_init(u_full, 1);
    mbar_init(z_ready, kWgCompute);
    mbar_init(z_free, 1);
    mbar_init(dz_full, 1);
    mbar_init(du_ready, kWgCompute);
    mbar_init(du_free, 1);
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, kWgCompute);
    fence_barrier_init();
  }
  if (warp == 13) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tW2 = tmem, tW1 = tmem + 256, tU = tmem + 384, tZ = tmem + 448;
  grid_dep_wait();
  grid_dep_launch();
  load_spans(a.plan, spans);
  const int T = a.plan.T;
  const int tile0 = slice * w.per, tile1 = min(tile0 + w.per, spans->first[T] / 128);
  // the slots of behaviour t in this slice: [lo, hi), hi before the padding
  auto piece = [&](int t, int& lo, int& hi) {
    lo = max(tile0 * 128, spans->first[t]);
    hi = min(tile1 * 128, spans->first[t] + spans->cnt[t]);
    return lo < hi;
  };

  if (warp == 12) {
    // ------------------------------------------------------ weight producer
    if (lane == 0) {
      const uint64_t keep = l2_evict_last();
      int p = 0;
      for (int t = 0; t < T; ++t) {
        int lo, hi;
        if (!piece(t, lo, hi)) continue;
        // the last piece's products are done when its sums have been taken out
        if (p > 0 && !mbar_wait(acc_empty, (p - 1) & 1)) break;
        ++p;
        mbar_expect_tx(w_full, cfg.w1_bytes + (do1 ? cfg.w2_bytes : 0));
        for (int b = 0; b < cfg.eb; ++b)
          for (int j = 0; j < 2; ++j)
            tma_load_3d_hint(&maps.w1[t], w_full, sW1 + b * 16384 + j * 8192, b * 64, h0 + j * 64, 0, keep);
        for (int j = 0; do1 && j < 2; ++j)
          for (int b = 0; b < NC; ++b)
            tma_load_3d_hint(&maps.w2[t], w_full, sW2 + j * d * 128 + b * 8192, h0 + j * 64, b * 64, 0, keep);
      }
    }
  } else if (warp == 13) {
    // ------------------------------------------------------------- products
    {
      const uint64_t dW1 = sdesc_k128(smem_u32(sW1)), dW2 = sdesc_mn128(smem_u32(sW2), d * 128);
      const uint64_t dSk = sdesc_k128(smem_u32(sS)), dSm = sdesc_mn128(smem_u32(sS), 8192);
      constexpr uint32_t id_u = idesc_bf16(128, 64), id_z = idesc_bf16(128, 64, true, false);
      constexpr int n0 = d > 256 ? 256 : d, n1 = d - n0;
      constexpr uint32_t id_2 = idesc_bf16(128, n0, false, true), id_2b = idesc_bf16(128, n1 ? n1 : 16, false, true);
      const uint32_t id_1 = idesc_bf16(128, a.e, false, true);
      const int ksteps = a.e / 16;
      const bool early = cfg.stages == 1;    // the only row stage is free after dW1 of the step before
      bool ok = true;
      int i = 0, p = 0;                      // steps and pieces so far
      RingPos sn, sg;                        // row stage of the next step, and of the next dW1
      auto grad1 = [&](int j, bool fresh) {  // dW1 of step j, then its rows are free
        if (do1) {
          ok = ok && mbar_wait(du_ready, j & 1);
          if (!ok) return;
          tc_fence_after();
          const uint64_t rows = desc_add(dSm, sg.s * cfg.stage_bytes + d * 128);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            mma_ts(tW1, tZ + k * 16, desc_add(rows, k * 2048), id_1, fresh && !k ? 0u : 1u);
            mma_ts(tW1, tZ + k * 16 + 8, desc_add(rows, k * 2048), id_1, 1u);
          }
        }
        mma_commit(du_free);
        mma_commit(&s_empty[sg.s]);
        sg.next(cfg.stages);
      };
      for (int t = 0; t < T && ok; ++t) {
        int lo, hi;
        if (!piece(t, lo, hi)) continue;
        ok = ok && mbar_wait(w_full, p & 1);
        if (p > 0) ok = ok && mbar_wait(acc_empty, (p - 1) & 1);
        const int n = (hi - lo + 63) / 64;
        for (int q = 0; q < n && ok; ++q, ++i) {
          if (early && q > 0) grad1(i - 1, q == 1);
          ok = ok && mbar_wait(&s_full[sn.s], sn.ph);
          if (i > 0) ok = ok && mbar_wait(z_free, (i - 1) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t rk = desc_add(dSk, sn.s * cfg.stage_bytes), rm = desc_add(dSm, sn.s * cfg.stage_bytes);
          sn.next(cfg.stages);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < ksteps)
              mma_ss(tU, desc_add(dW1, (k >> 2) * 16384 + (k & 3) * 32),
                        desc_add(rk, d * 128 + (k >> 2) * 8192 + (k & 3) * 32), id_u, k ? 1u : 0u);
          mma_commit(u_full);
          if (q > 0) {
            if (!early) grad1(i - 1, q == 1);
            ok = ok && mbar_wait(du_free, (i - 1) & 1);
          }
          if (!ok) break;
          tc_fence_after();
          if (do1) {
#pragma unroll
            for (int k = 0; k < NC * 4; ++k)
              mma_ss(tZ, desc_add(dW2, k * 2048), desc_add(rk, (k >> 2) * 8192 + (k & 3) * 32), id_z, k ? 1u : 0u);
            mma_commit(dz_full);
          }
          ok = mbar_wait(z_ready, i & 1);
          if (!ok) break;
          tc_fence_after();
          if (do2) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t z = tU + k * 16;
              mma_ts(tW2, z, desc_add(rm, k * 2048), id_2, q || k ? 1u : 0u);
              mma_ts(tW2, z + 8, desc_add(rm, k * 2048), id_2, 1u);
              if (n1) {
                mma_ts(tW2 + n0, z, desc_add(rm, n0 * 128 + k * 2048), id_2b, q || k ? 1u : 0u);
                mma_ts(tW2 + n0, z + 8, desc_add(rm, n0 * 128 + k * 2048), id_2b, 1u);
              }
            }
          }
          mma_commit(z_free);
        }
        if (!ok) break;
        grad1(i - 1, n == 1);
        ok = ok && mbar_wait(du_free, (i - 1) & 1);
        mma_commit(acc_full);
        ++p;
      }
    }
  } else if (warp >= 8) {
    // --------------------------------------------------------------- gather
    // With three stages or more a step's copies are in flight while the next
    // step's are issued, and its arrival follows then.  (With two, the next
    // step's stage is free only after the products that wait for this arrival.)
    const bool defer = cfg.stages > 2;
    const int tid = threadIdx.x - 8 * 32;
    bool ok = true;
    int i = 0;
    RingPos sn, sa;
    auto arrive = [&]() {
      fence_async_smem();
      asm volatile("bar.sync 1, 128;" ::: "memory");
      warp_arrive(&s_full[sa.s]);
      sa.next(cfg.stages);
    };
    for (int t = 0; t < T; ++t) {
      int lo, hi;
      if (!piece(t, lo, hi)) continue;
      int flat = tid < 64 && lo + tid < hi ? a.plan.order[lo + tid] : -1;
      for (int at = lo; at < hi; at += 64, ++i) {
        const int row = flat < 0 ? -1 : flat / a.plan.k;
        long long* off = sOff + (i & 1) * 64;
        int* rows = sRow + (i & 1) * 64;
        float wt = 0.f;
        if (tid < 64) {
          off[tid] = row < 0 ? -1LL : token_off(a.rows, row, d);
          rows[tid] = row;
          wt = flat < 0 ? 0.f : a.weights ? a.weights[flat] : 1.f;
          flat = at + 64 + tid < hi ? a.plan.order[at + 64 + tid] : -1;   // of the next step
        }
        if (i >= cfg.stages) ok = ok && mbar_wait(&s_empty[sn.s], sn.ph ^ 1);
        if (tid < 64) sWt[sn.s * 64 + tid] = wt;
        asm volatile("bar.sync 1, 128;" ::: "memory");
        uint8_t* to = sS + sn.s * cfg.stage_bytes;
        if (ok) {
          gather_events<128>(to + d * 128, rows, 64, a.e, a.events, tid);
          gather_boxes<128, NC>(to, [&](int r) { return off[r]; }, 64, d, a.dtokens, tid);
        }
        cp_async_commit();
        sn.next(cfg.stages);
        if (!defer) {
          cp_async_wait<0>();
          arrive();
        } else if (i > 0) {
          cp_async_wait<1>();
          arrive();
        }
      }
    }
    if (defer && i > 0) {
      cp_async_wait<0>();
      arrive();
    }
  } else {
    // -------------------------------------------------------------- compute
    const int q4 = warp & 3, wq = warp >> 2;       // hidden quarter, half of the step's slots
    const uint32_t lb = (uint32_t)(q4 * 32) << 16;
    const int h = h0 + q4 * 32 + lane;
    const int oc = threadIdx.x & 15, og = threadIdx.x >> 4;   // db2: 8 columns, 4 slots a step
    bool ok = true;
    int i = 0, p = 0;
    RingPos sn;
    for (int t = 0; t < T; ++t) {
      int lo, hi;
      if (!piece(t, lo, hi)) continue;
      const float b1 = h < d ? __bfloat162float(((const __nv_bfloat16*)a.mlp.b1[t])[h]) : 0.f;
      float db1 = 0.f, db2[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int at = lo; at < hi; at += 64, ++i) {
        ok = ok && mbar_wait(&s_full[sn.s], sn.ph);   // the choice weights
        const float* wt = sWt + sn.s * 64 + wq * 32;
        ok = ok && mbar_wait(u_full, i & 1);
        tc_fence_after();
        const uint32_t col = lb + wq * 32;
        float v[32];
        tmem_ld32(tU + col, v);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int n = hf * 16 + 2 * j;
            const float2 wj = *(const float2*)(wt + n);
            float z0, z1, g0, g1;
            gelu_and_slope_fast(v[n] + b1, z0, g0);
            gelu_and_slope_fast(v[n + 1] + b1, z1, g1);
            v[n] = wj.x * g0;
            v[n + 1] = wj.y * g1;
            split_bf16x2(wj.x * z0, wj.y * z1, pk[j], pk[8 + j]);
          }
          tmem_st16(tU + col + hf * 16, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(z_ready);
        if (do1) {
          ok = ok && mbar_wait(dz_full, i & 1);
          tc_fence_after();
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            float y[16];
            tmem_ld16(tZ + col + hf * 16, y);
            uint32_t pk[16];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int n = hf * 16 + 2 * j;
              const float x0 = y[2 * j] * v[n], x1 = y[2 * j + 1] * v[n + 1];
              db1 += x0 + x1;
              split_bf16x2(x0, x1, pk[j], pk[8 + j]);
            }
            tmem_st16(tZ + col + hf * 16, pk);
          }
          tmem_st_wait();
          tc_fence_before();
          warp_arrive(du_ready);
          const int c = h0 / 8 + oc;   // db2 of output columns h0 + 8 oc .. + 7
          if (c * 8 < d) {
            const uint8_t* box = sS + sn.s * cfg.stage_bytes + (c >> 3) * 8192;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int r = og * 4 + j;
              const uint4 x = *(const uint4*)(box + r * 128 + (((c & 7) ^ (r & 7)) << 4));
              const __nv_bfloat162* xh = (const __nv_bfloat162*)&x;
              const float wr = sWt[sn.s * 64 + r];
#pragma unroll
              for (int n = 0; n < 4; ++n) {
                const float2 f = __bfloat1622float2(xh[n]);
                db2[2 * n] = fmaf(wr, f.x, db2[2 * n]);
                db2[2 * n + 1] = fmaf(wr, f.y, db2[2 * n + 1]);
              }
            }
          }
        }
        warp_arrive(&s_empty[sn.s]);
        sn.next(cfg.stages);
      }
      // the piece's sums: dW2 [o][h] with neighbouring lanes on neighbouring h
      ok = ok && mbar_wait(acc_full, p & 1);
      tc_fence_after();
      float* out = piece_at(w, slice, t);
      for (int c0 = wq * 32; do2 && c0 < d; c0 += 64) {
        float v[32];
        tmem_ld32(tW2 + lb + c0, v);
        if (h < d && ok)
#pragma unroll
          for (int j = 0; j < 32; ++j) out[(long long)(c0 + j) * d + h] = v[j];
      }
      if (do1) {
        for (int c0 = wq * 16; c0 < a.e; c0 += 32) {
          float v[16];
          tmem_ld16(tW1 + lb + c0, v);
          if (h < d && ok) {
            float4* o = (float4*)(out + (long long)d * d + (long long)h * a.e + c0);
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          }
        }
      }
      tc_fence_before();
      if (do1) {
        // db1: the two halves; db2: the 16 slot groups, through W1's tile (its
        // products are done, and the next weights wait for acc_empty)
        float* red = (float*)sW1;    // 128 + 16 x 128 floats
        asm volatile("bar.sync 2, 256;" ::: "memory");
        if (wq) red[q4 * 32 + lane] = db1;
#pragma unroll
        for (int n = 0; n < 8; ++n) red[128 + og * 128 + oc * 8 + n] = db2[n];
        asm volatile("bar.sync 2, 256;" ::: "memory");
        float* bias = out + (long long)d * (d + a.e);
        if (!wq && h < d && ok) bias[h] = db1 + red[q4 * 32 + lane];
        if (wq && ok) {
          const int c = threadIdx.x - 128;
          float sum = 0.f;
          for (int n = 0; n < 16; ++n) sum += red[128 + n * 128 + c];
          if (h0 + c < d) bias[d + h0 + c] = sum;
        }
        asm volatile("bar.sync 2, 256;" ::: "memory");
        fence_async_smem();          // the weights that follow are written by TMA
      }
      warp_arrive(acc_empty);
      ++p;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 13) tmem_dealloc(tmem, 512);
}

}  // namespace ot
