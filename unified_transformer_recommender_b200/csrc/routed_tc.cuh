// Tensor-core kernels of the routed event tokenizer (bf16 mode, d a multiple
// of 64 up to 384, event_dim a multiple of 16 up to 128).
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
  int e, d;
  const __nv_bfloat16* events;
  const float* weights;          // [R*k] or null
  __nv_bfloat16* tokens;         // k = 1
  TokenRows rows;
  float* part;                   // [R*k][d], k > 1
};

__device__ inline void cp_async16(void* dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
__device__ inline void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ inline void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Rows of `width` bf16 elements (a multiple of 8) into boxes of [rows x 64
// columns] with the 128-byte swizzle, columns past the width and rows with a
// negative offset zero.  `off` (shared memory): element offset of each row.
// NT threads; the copies are in flight until cp_async_wait.
template <int NT>
__device__ inline void gather_boxes(uint8_t* tile, const long long* off, int rows, int width, const __nv_bfloat16* src,
                                    int tid) {
  const int per_row = ((width + 63) >> 6) << 3;   // 16-byte chunks
  for (int i = tid; i < rows * per_row; i += NT) {
    const int r = i / per_row, c = i - r * per_row;
    const long long o = off[r];
    const bool on = o >= 0 && c * 8 < width;
    cp_async16(tile + (c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4), src + (on ? o + c * 8 : 0), on);
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

// ----------------------------------------------------------------- tokens --
// One CTA per SM walks 128-slot tiles.  Per 64 hidden units: U = E W1c^T
// (tcgen05, M = 128, N = 64), bias and GELU by eight warps, z packed to bf16
// over U's own TMEM columns, D += z W2c^T with z read from TMEM (N = d).  The
// hidden row therefore never leaves the SM.  Two U buffers let the next
// chunk's first product run during this one's GELU; the weights stream
// through a ring (the tiles of one behaviour read the same 2 d (e + d) bytes,
// which stay in L2).  The gathered event rows come through cp.async into the
// swizzled operand layout, the weighted token rows leave through a transposing
// staging area as 128-byte pieces of their destination rows.
// Warps 0-7 compute, 8-11 gather, 12 loads weights, 13 issues the products.
constexpr int kTokThreads = 448, kTokCompute = 256;

struct TokCfg {
  int eb;        // 64-column boxes of an event row
  int ebuf;      // event tiles in flight
  int stages;    // weight stages
  int w1_bytes, stage_bytes, e_bytes;
  int smem;
};
__host__ __device__ inline TokCfg tok_cfg(int e, int d) {
  TokCfg c;
  c.eb = (e + 63) / 64;
  c.e_bytes = c.eb * 16384;
  c.w1_bytes = c.eb * 8192;
  c.stage_bytes = c.w1_bytes + d * 128;
  const int fixed = 1024 + 1024 + 128 * 8 + 8 * 32 * 144;   // alignment, barriers, row offsets, staging
  const int room = 232448 - fixed;
  c.ebuf = c.eb == 1 ? 2 : 1;
  c.stages = (room - c.ebuf * c.e_bytes) / c.stage_bytes;
  if (c.stages > 4) c.stages = 4;
  c.smem = fixed + c.ebuf * c.e_bytes + c.stages * c.stage_bytes;
  return c;
}

template <bool COMBINE>
__global__ void __launch_bounds__(kTokThreads, 1)
    routed_tokens_kernel(const __grid_constant__ RoutedMaps maps, const RoutedTcArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const TokCfg cfg = tok_cfg(a.e, a.d);
  uint8_t* sE = smem;
  uint8_t* sW = sE + cfg.ebuf * cfg.e_bytes;
  uint8_t* sOut = sW + cfg.stages * cfg.stage_bytes;       // 8 warps x 32 rows x 144 B
  long long* sOff = (long long*)(sOut + 8 * 32 * 144);     // row offsets of the tile being gathered
  uint64_t* bars = (uint64_t*)(sOff + 128);
  uint64_t* e_full = bars;          // [2]
  uint64_t* e_empty = bars + 2;     // [2]
  uint64_t* w_full = bars + 4;      // [4]
  uint64_t* w_empty = bars + 8;     // [4]
  uint64_t* u_full = bars + 12;     // [2]
  uint64_t* z_ready = bars + 14;    // [2]
  uint64_t* dn_done = bars + 16;    // [2]
  uint64_t* d_full = bars + 18;
  uint64_t* d_empty = bars + 19;
  uint32_t* tmem_slot = (uint32_t*)(bars + 20);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int d = a.d, NC = d / 64;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&e_full[i], 128);
      mbar_init(&e_empty[i], 1);
      mbar_init(&u_full[i], 1);
      mbar_init(&z_ready[i], kTokCompute);
      mbar_init(&dn_done[i], 1);
    }
    for (int i = 0; i < cfg.stages; ++i) {
      mbar_init(&w_full[i], 1);
      mbar_init(&w_empty[i], 1);
    }
    mbar_init(d_full, 1);
    mbar_init(d_empty, kTokCompute);
    fence_barrier_init();
  }
  if (warp == 13) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tD = tmem, tU = tmem + 384;   // U buffers at 384 and 448
  grid_dep_wait();
  grid_dep_launch();

  const bool fine = plan_ok(a.plan);
  const int n_tiles = fine ? plan_first(a.plan, a.plan.T) / 128 : 0;
  const int mine = n_tiles > (int)blockIdx.x ? (n_tiles - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
  auto tile_at = [&](int i) { return (int)blockIdx.x + i * (int)gridDim.x; };

  if (warp == 12) {
    // ------------------------------------------------------ weight producer
    if (lane == 0) {
      const uint64_t keep = l2_evict_last();
      for (int g = 0; g < mine * NC; ++g) {
        const int s = g % cfg.stages;
        if (g >= cfg.stages && !mbar_wait(&w_empty[s], ((g / cfg.stages) - 1) & 1)) break;
        const int t = plan_type(a.plan, tile_at(g / NC) * 128), h0 = (g % NC) * 64;
        uint8_t* w1 = sW + s * cfg.stage_bytes;
        mbar_expect_tx(&w_full[s], cfg.stage_bytes);
        for (int b = 0; b < cfg.eb; ++b) tma_load_3d_hint(&maps.w1[t], &w_full[s], w1 + b * 8192, b * 64, h0, 0, keep);
        for (int b = 0; b < NC; ++b)
          tma_load_3d_hint(&maps.w2[t], &w_full[s], w1 + cfg.w1_bytes + b * 8192, h0, b * 64, 0, keep);
      }
    }
  } else if (warp == 13) {
    // ------------------------------------------------------------- products
    if (lane == 0) {
      const uint64_t dE = sdesc_k128(smem_u32(sE)), dW = sdesc_k128(smem_u32(sW));
      const uint32_t id_u = idesc_bf16(128, 64);
      const int n0 = d > 256 ? 256 : d, n1 = d - n0;
      const uint32_t id_0 = idesc_bf16(128, n0), id_1 = idesc_bf16(128, n1 ? n1 : 16);
      const int ksteps = a.e / 16, total = mine * NC;
      bool ok = true;
      auto up = [&](int g) {
        const int s = g % cfg.stages, i = g / NC, c = g - i * NC, eb = i % cfg.ebuf;
        ok = ok && mbar_wait(&w_full[s], (g / cfg.stages) & 1);
        if (c == 0) ok = ok && mbar_wait(&e_full[eb], (i / cfg.ebuf) & 1);
        if (g >= 2) ok = ok && mbar_wait(&dn_done[g & 1], ((g >> 1) - 1) & 1);   // z of chunk g - 2 consumed
        if (!ok) return;
        tc_fence_after();
        for (int k = 0; k < ksteps; ++k)
          umma_bf16(tU + (g & 1) * 64, desc_add(dE, eb * cfg.e_bytes + (k >> 2) * 16384 + (k & 3) * 32),
                    desc_add(dW, s * cfg.stage_bytes + (k >> 2) * 8192 + (k & 3) * 32), id_u, k ? 1u : 0u);
        umma_commit(&u_full[g & 1]);
        if (c == NC - 1) umma_commit(&e_empty[eb]);
      };
      if (total > 0) up(0);
      for (int g = 0; g < total && ok; ++g) {
        if (g + 1 < total) up(g + 1);
        const int s = g % cfg.stages, i = g / NC, c = g - i * NC;
        ok = ok && mbar_wait(&z_ready[g & 1], (g >> 1) & 1);
        if (c == 0 && i > 0) ok = ok && mbar_wait(d_empty, (i - 1) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint64_t w2 = desc_add(dW, s * cfg.stage_bytes + cfg.w1_bytes);
#pragma unroll
        for (int k = 0; k < 4; ++k) {   // units 16k .. 16k+15 packed over U columns 16k .. 16k+7
          const uint32_t z = tU + (g & 1) * 64 + k * 16;
          umma_bf16_ts(tD, z, desc_add(w2, k * 32), id_0, (c | k) ? 1u : 0u);
          if (n1) umma_bf16_ts(tD + n0, z, desc_add(w2, n0 * 128 + k * 32), id_1, (c | k) ? 1u : 0u);
        }
        umma_commit(&w_empty[s]);
        umma_commit(&dn_done[g & 1]);
        if (c == NC - 1) umma_commit(d_full);
      }
    }
  } else if (warp >= 8) {
    // --------------------------------------------------------------- gather
    const int tid = threadIdx.x - kTokCompute;
    bool ok = true;
    for (int i = 0; i < mine; ++i) {
      const int eb = i % cfg.ebuf;
      const int flat = a.plan.order[(long long)tile_at(i) * 128 + tid];
      if (i >= cfg.ebuf) ok = ok && mbar_wait(&e_empty[eb], ((i / cfg.ebuf) - 1) & 1);
      sOff[tid] = flat < 0 ? -1LL : (long long)(flat / a.plan.k) * a.e;
      asm volatile("bar.sync 1, 128;" ::: "memory");
      if (ok) gather_boxes<128>(sE + eb * cfg.e_bytes, sOff, 128, a.e, a.events, tid);
      cp_async_wait();
      fence_async_smem();
      asm volatile("bar.sync 1, 128;" ::: "memory");   // sOff free again
      mbar_arrive(&e_full[eb]);
    }
    if (!COMBINE && fine) zero_unrouted(a.plan, a.tokens, a.rows, d, blockIdx.x * 4 + warp - 8, gridDim.x * 4);
  } else {
    // -------------------------------------------------------------- compute
    const int q4 = warp & 3, wq = warp >> 2;    // row quarter, column half
    const uint32_t lb = (uint32_t)(q4 * 32) << 16;
    uint8_t* stage = sOut + warp * 32 * 144;
    bool ok = true;
    for (int i = 0; i < mine; ++i) {
      const int slot = tile_at(i) * 128 + q4 * 32 + lane;
      const int t = plan_type(a.plan, tile_at(i) * 128);
      const int flat = a.plan.order[slot];
      const float w = flat >= 0 && a.weights ? a.weights[flat] : 1.f;
      long long off = -1;
      if (flat >= 0) off = COMBINE ? (long long)flat * d : token_off(a.rows, flat, d);
      const __nv_bfloat16* b1 = (const __nv_bfloat16*)a.mlp.b1[t];
      for (int c = 0; c < NC; ++c) {
        const int g = i * NC + c;
        uint4 bq[4];     // this chunk's b1, ahead of the wait
#pragma unroll
        for (int j = 0; j < 4; ++j) bq[j] = ((const uint4*)(b1 + c * 64 + wq * 32))[j];
        ok = ok && mbar_wait(&u_full[g & 1], (g >> 1) & 1);
        tc_fence_after();
        const uint32_t col = tU + (g & 1) * 64 + lb + wq * 32;
        float v[32];
        tmem_ld32(col, v);
        const uint32_t* bu = (const uint32_t*)bq;
        uint32_t pk[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float2 bf = __bfloat1622float2(*(const __nv_bfloat162*)&bu[j]);
          pk[j] = gelu_bias_bf16x2(v[2 * j], v[2 * j + 1], bf.x, bf.y);
        }
        tmem_st8(col, pk);
        tmem_st8(col + 16, pk + 8);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&z_ready[g & 1]);
      }
      // the weighted tokens: row by row in TMEM, out in 128-byte pieces
      const __nv_bfloat16* b2 = (const __nv_bfloat16*)a.mlp.b2[t];
      const __nv_bfloat16* emb = (const __nv_bfloat16*)a.mlp.emb + (long long)t * d;
      ok = ok && mbar_wait(d_full, i & 1);
      tc_fence_after();
      const int half = d / 2;
      for (int c0 = wq * half; c0 < (wq + 1) * half; c0 += 32) {
        float v[32], s0[32], s1[32];
        tmem_ld32(tD + lb + c0, v);
        load_bf16x32(b2 + c0, s0);
        load_bf16x32(emb + c0, s1);
        if (c0 + 32 == (wq + 1) * half) {   // D read: the next tile may overwrite it
          tc_fence_before();
          mbar_arrive(d_empty);
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = w * (v[j] + (s0[j] + s1[j]));
        const bool last = c0 + 32 == (wq + 1) * half;
        if (COMBINE) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *(float4*)(stage + lane * 144 + j * 16) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        } else {
          // two 32-column steps fill a piece of 64 columns
          const int h = ((c0 - wq * half) >> 5) & 1;
          store_bf16x32((__nv_bfloat16*)(stage + lane * 144 + h * 64), v);
          if (!h && !last) continue;
        }
        __syncwarp();
        const int first = COMBINE ? c0 : c0 - (((c0 - wq * half) >> 5) & 1) * 32;
        const int chunks = COMBINE ? 8 : (c0 + 32 - first) / 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int r = j * 4 + (lane >> 3), ch = lane & 7;
          const long long o = __shfl_sync(~0u, off, r);
          if (o >= 0 && ch < chunks && ok) {
            const uint4 x = *(const uint4*)(stage + r * 144 + ch * 16);
            if (COMBINE) *(uint4*)(a.part + o + first + ch * 4) = x;
            else *(uint4*)(a.tokens + o + first + ch * 8) = x;
          }
        }
        __syncwarp();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 13) tmem_dealloc(tmem, 512);
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

// gather_boxes from float32 rows, rounded to bf16 (through registers: the
// conversion keeps them from being copied asynchronously).
template <int NT>
__device__ inline void gather_boxes(uint8_t* tile, const long long* off, int rows, int width, const float* src,
                                    int tid) {
  const int per_row = ((width + 63) >> 6) << 3, n = rows * per_row;
  for (int i0 = tid; i0 < n; i0 += NT * 4) {
    float4 v[4][2];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * NT, r = i / per_row, c = i - r * per_row;
      v[u][0] = v[u][1] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n && off[r] >= 0 && c * 8 < width) {
        const float4* p = (const float4*)(src + off[r] + c * 8);
        v[u][0] = p[0];
        v[u][1] = p[1];
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * NT, r = i / per_row, c = i - r * per_row;
      if (i < n)
        *(uint4*)(tile + (c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
            make_uint4(pack_bf16x2(v[u][0].x, v[u][0].y), pack_bf16x2(v[u][0].z, v[u][0].w),
                       pack_bf16x2(v[u][1].x, v[u][1].y), pack_bf16x2(v[u][1].z, v[u][1].w));
    }
  }
}

struct RoutedBwdArgs {
  PlanView plan;
  RoutedMLP mlp;
  int e, d;
  const __nv_bfloat16* events;
  const float* weights;          // [R*k] or null
  const void* dtokens;
  TokenRows rows;
  __nv_bfloat16* devents;        // k = 1, or null
  float* part;                   // [R*k][e], k > 1, or null
  float* dweights;               // [R*k] or null
};

// ------------------------------------------------------------ event gradient --
// de = W1^T du and dw, tile by tile like the forward: per 64 hidden units
// U = E W1c^T (K = e) and DZ = DY W2c (K = d) into TMEM, du = w dz GELU'(u) by
// eight warps, split into two bf16 terms over U's columns, DE += du W1c.
// W1's chunk serves both of its products from one shared-memory tile (K-major
// for U, MN-major for DE), as W2's does in the forward.  dw's row sums stay
// with the thread that owns the row.
// Warps 0-7 compute, 8-11 gather, 12 loads weights, 13 issues the products.
struct DevCfg {
  int eb, abuf, units, w1st;      // event boxes, row tiles in flight, W2 units of 64 rows, W1 stages
  int a_bytes, w1_bytes, smem;
};
__host__ __device__ inline DevCfg dev_cfg(int e, int d) {
  DevCfg c;
  c.eb = (e + 63) / 64;
  c.a_bytes = d * 256 + c.eb * 16384;            // dtoken rows, then event rows
  c.w1_bytes = c.eb * 8192;
  c.w1st = 2;
  const int fixed = 1024 + 1024 + 1024;          // alignment, barriers and dw partials, row offsets
  const int room = 232448 - fixed - c.w1st * c.w1_bytes;
  c.abuf = room >= 2 * c.a_bytes + 4 * 8192 ? 2 : 1;
  c.units = (room - c.abuf * c.a_bytes) / 8192;
  if (c.units > 12) c.units = 12;
  c.smem = fixed + c.abuf * c.a_bytes + c.w1st * c.w1_bytes + c.units * 8192;
  return c;
}

template <typename Td>
__global__ void __launch_bounds__(kTokThreads, 1)
    routed_devents_kernel(const __grid_constant__ RoutedMaps maps, const RoutedBwdArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const DevCfg cfg = dev_cfg(a.e, a.d);
  const int d = a.d, NC = d / 64;
  uint8_t* sA = smem;
  uint8_t* sW1 = sA + cfg.abuf * cfg.a_bytes;
  uint8_t* sW2 = sW1 + cfg.w1st * cfg.w1_bytes;
  long long* sOff = (long long*)(sW2 + cfg.units * 8192);
  uint64_t* bars = (uint64_t*)(sOff + 128);
  uint64_t* a_full = bars;           // [2]
  uint64_t* a_empty = bars + 2;      // [2]
  uint64_t* w1_full = bars + 4;      // [2]
  uint64_t* w1_empty = bars + 6;     // [2]
  uint64_t* w2_full = bars + 8;      // [12]
  uint64_t* w2_empty = bars + 20;    // [12]
  uint64_t* u_full = bars + 32;      // [2]
  uint64_t* du_ready = bars + 34;    // [2]
  uint64_t* du_done = bars + 36;     // [2]
  uint64_t* de_full = bars + 38;
  uint64_t* de_empty = bars + 39;
  uint32_t* tmem_slot = (uint32_t*)(bars + 40);
  float* sDot = (float*)(bars + 64);  // [128]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&a_full[i], 128);
      mbar_init(&a_empty[i], 1 + kTokCompute);
      mbar_init(&w1_full[i], 1);
      mbar_init(&w1_empty[i], 1);
      mbar_init(&u_full[i], 1);
      mbar_init(&du_ready[i], kTokCompute);
      mbar_init(&du_done[i], 1);
    }
    for (int i = 0; i < cfg.units; ++i) {
      mbar_init(&w2_full[i], 1);
      mbar_init(&w2_empty[i], 1);
    }
    mbar_init(de_full, 1);
    mbar_init(de_empty, kTokCompute);
    fence_barrier_init();
  }
  if (warp == 13) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tE = tmem, tU = tmem + 128, tZ = tmem + 256;   // DE, two U, two DZ buffers
  grid_dep_wait();
  grid_dep_launch();

  const bool fine = plan_ok(a.plan);
  const int n_tiles = fine ? plan_first(a.plan, a.plan.T) / 128 : 0;
  const int mine = n_tiles > (int)blockIdx.x ? (n_tiles - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
  auto tile_at = [&](int i) { return (int)blockIdx.x + i * (int)gridDim.x; };

  if (warp == 12) {
    // ------------------------------------------------------ weight producer
    if (lane == 0) {
      const uint64_t keep = l2_evict_last();
      bool ok = true;
      for (int g = 0, q = 0; g < mine * NC && ok; ++g) {
        const int s = g % cfg.w1st;
        ok = g < cfg.w1st || mbar_wait(&w1_empty[s], ((g / cfg.w1st) - 1) & 1);
        if (!ok) break;
        const int t = plan_type(a.plan, tile_at(g / NC) * 128), h0 = (g % NC) * 64;
        mbar_expect_tx(&w1_full[s], cfg.w1_bytes);
        for (int b = 0; b < cfg.eb; ++b)
          tma_load_3d_hint(&maps.w1[t], &w1_full[s], sW1 + s * cfg.w1_bytes + b * 8192, b * 64, h0, 0, keep);
        for (int b = 0; b < NC && ok; ++b, ++q) {
          const int w = q % cfg.units;
          ok = q < cfg.units || mbar_wait(&w2_empty[w], ((q / cfg.units) - 1) & 1);
          if (!ok) break;
          mbar_expect_tx(&w2_full[w], 8192);
          tma_load_3d_hint(&maps.w2[t], &w2_full[w], sW2 + w * 8192, h0, b * 64, 0, keep);
        }
      }
    }
  } else if (warp == 13) {
    // ------------------------------------------------------------- products
    if (lane == 0) {
      const uint64_t dA = sdesc_k128(smem_u32(sA)), dW1 = sdesc_k128(smem_u32(sW1));
      const uint64_t dW1t = sdesc_mn128(smem_u32(sW1), 8192), dW2t = sdesc_mn128(smem_u32(sW2), 8192);
      const uint32_t id_u = idesc_bf16(128, 64), id_z = idesc_bf16(128, 64, false, true);
      const uint32_t id_e = idesc_bf16(128, a.e, false, true);
      const int ksteps = a.e / 16, total = mine * NC;
      bool ok = true;
      int q = 0;
      auto up = [&](int g) {
        const int s = g % cfg.w1st, i = g / NC, c = g - i * NC, ab = i % cfg.abuf;
        ok = ok && mbar_wait(&w1_full[s], (g / cfg.w1st) & 1);
        if (c == 0) ok = ok && mbar_wait(&a_full[ab], (i / cfg.abuf) & 1);
        if (g >= 2) ok = ok && mbar_wait(&du_done[g & 1], ((g >> 1) - 1) & 1);
        if (!ok) return;
        tc_fence_after();
        const uint64_t da = desc_add(dA, ab * cfg.a_bytes);
        for (int k = 0; k < ksteps; ++k)
          umma_bf16(tU + (g & 1) * 64, desc_add(da, d * 256 + (k >> 2) * 16384 + (k & 3) * 32),
                    desc_add(dW1, s * cfg.w1_bytes + (k >> 2) * 8192 + (k & 3) * 32), id_u, k ? 1u : 0u);
        for (int b = 0; b < NC; ++b, ++q) {       // 64 of the contraction per W2 unit
          const int w = q % cfg.units;
          ok = mbar_wait(&w2_full[w], (q / cfg.units) & 1);
          if (!ok) return;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_bf16(tZ + (g & 1) * 64, desc_add(da, b * 16384 + k * 32), desc_add(dW2t, w * 8192 + k * 2048), id_z,
                      (b | k) ? 1u : 0u);
          umma_commit(&w2_empty[w]);
        }
        umma_commit(&u_full[g & 1]);
        if (c == NC - 1) umma_commit(&a_empty[ab]);
      };
      auto down = [&](int g) {
        const int s = g % cfg.w1st, i = g / NC, c = g - i * NC;
        ok = ok && mbar_wait(&du_ready[g & 1], (g >> 1) & 1);
        if (c == 0 && i > 0) ok = ok && mbar_wait(de_empty, (i - 1) & 1);
        if (!ok) return;
        tc_fence_after();
        const uint64_t w1 = desc_add(dW1t, s * cfg.w1_bytes);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t du = tU + (g & 1) * 64 + k * 16;   // hi in 8 columns, lo in the next 8
          umma_bf16_ts(tE, du, desc_add(w1, k * 2048), id_e, (c | k) ? 1u : 0u);
          umma_bf16_ts(tE, du + 8, desc_add(w1, k * 2048), id_e, 1u);
        }
        umma_commit(&w1_empty[s]);
        umma_commit(&du_done[g & 1]);
        if (c == NC - 1) umma_commit(de_full);
      };
      if (total > 0) up(0);
      for (int g = 0; g < total && ok; ++g) {
        const bool same = g + 1 < total && (g + 1) % NC != 0;
        if (same) up(g + 1);          // runs during this chunk's GELU
        down(g);
        if (!same && g + 1 < total) up(g + 1);   // a new tile: its rows may still be on their way
      }
    }
  } else if (warp >= 8) {
    // --------------------------------------------------------------- gather
    const int tid = threadIdx.x - kTokCompute;
    bool ok = true;
    for (int i = 0; i < mine; ++i) {
      const int ab = i % cfg.abuf;
      const int flat = a.plan.order[(long long)tile_at(i) * 128 + tid];
      const int row = flat < 0 ? -1 : flat / a.plan.k;
      if (i >= cfg.abuf) ok = ok && mbar_wait(&a_empty[ab], ((i / cfg.abuf) - 1) & 1);
      uint8_t* at = sA + ab * cfg.a_bytes;
      sOff[tid] = row < 0 ? -1LL : (long long)row * a.e;
      asm volatile("bar.sync 1, 128;" ::: "memory");
      if (ok) gather_boxes<128>(at + d * 256, sOff, 128, a.e, a.events, tid);
      asm volatile("bar.sync 1, 128;" ::: "memory");
      sOff[tid] = row < 0 ? -1LL : token_off(a.rows, row, d);
      asm volatile("bar.sync 1, 128;" ::: "memory");
      if (ok) gather_boxes<128>(at, sOff, 128, d, (const Td*)a.dtokens, tid);
      cp_async_wait();
      fence_async_smem();
      asm volatile("bar.sync 1, 128;" ::: "memory");
      mbar_arrive(&a_full[ab]);
    }
    if (fine && a.devents && a.plan.k == 1)
      zero_unrouted(a.plan, a.devents, TokenRows{0x7fffffff, 0}, a.e, blockIdx.x * 4 + warp - 8, gridDim.x * 4);
    if (fine && a.dweights) {
      const long long n = (long long)a.plan.R * a.plan.k;
      for (long long c = (long long)blockIdx.x * 128 + tid; c < n; c += (long long)gridDim.x * 128)
        if (a.plan.pos[c] < 0) a.dweights[c] = 0.f;
    }
  } else {
    // -------------------------------------------------------------- compute
    const int q4 = warp & 3, wq = warp >> 2;
    const uint32_t lb = (uint32_t)(q4 * 32) << 16;
    const int row = q4 * 32 + lane;
    bool ok = true;
    for (int i = 0; i < mine; ++i) {
      const int t = plan_type(a.plan, tile_at(i) * 128);
      const int flat = a.plan.order[tile_at(i) * 128 + row];
      const float w = flat < 0 ? 0.f : a.weights ? a.weights[flat] : 1.f;
      const __nv_bfloat16* b1 = (const __nv_bfloat16*)a.mlp.b1[t];
      const int ab = i % cfg.abuf;
      float dot = 0.f;
      if (a.dweights) {       // <dtoken, b2 + emb> over this half of the row's columns
        const __nv_bfloat16* b2 = (const __nv_bfloat16*)a.mlp.b2[t];
        const __nv_bfloat16* emb = (const __nv_bfloat16*)a.mlp.emb + (long long)t * d;
        ok = ok && mbar_wait(&a_full[ab], (i / cfg.abuf) & 1);
        const uint8_t* at = sA + ab * cfg.a_bytes + row * 128;
        for (int c = wq * (d / 16); c < (wq + 1) * (d / 16); ++c) {
          const uint4 x = *(const uint4*)(at + (c >> 3) * 16384 + (((c & 7) ^ (row & 7)) << 4));
          const uint4 y = ((const uint4*)b2)[c], z = ((const uint4*)emb)[c];
          const __nv_bfloat162 *xh = (const __nv_bfloat162*)&x, *yh = (const __nv_bfloat162*)&y, *zh = (const __nv_bfloat162*)&z;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 p = __bfloat1622float2(xh[j]), s0 = __bfloat1622float2(yh[j]), s1 = __bfloat1622float2(zh[j]);
            dot = fmaf(p.x, s0.x + s1.x, dot);
            dot = fmaf(p.y, s0.y + s1.y, dot);
          }
        }
      }
      mbar_arrive(&a_empty[ab]);
      for (int c = 0; c < NC; ++c) {
        const int g = i * NC + c;
        uint4 bq[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) bq[j] = ((const uint4*)(b1 + c * 64 + wq * 32))[j];
        ok = ok && mbar_wait(&u_full[g & 1], (g >> 1) & 1);
        tc_fence_after();
        const uint32_t col = (g & 1) * 64 + lb + wq * 32;
        float v[32], y[32];
        tmem_ld32(tU + col, v);
        tmem_ld32(tZ + col, y);
        const uint32_t* bu = (const uint32_t*)bq;
#pragma unroll
        for (int h = 0; h < 2; ++h) {       // 16 units: 8 columns of hi, 8 of lo
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 bf = __bfloat1622float2(*(const __nv_bfloat162*)&bu[h * 8 + j]);
            const int n = h * 16 + 2 * j;
            float z0, g0, z1, g1;
            gelu_and_slope_fast(v[n] + bf.x, z0, g0);
            gelu_and_slope_fast(v[n + 1] + bf.y, z1, g1);
            dot = fmaf(y[n], z0, dot);
            dot = fmaf(y[n + 1], z1, dot);
            split_bf16x2(w * y[n] * g0, w * y[n + 1] * g1, pk[j], pk[8 + j]);
          }
          tmem_st16(tU + col + h * 16, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&du_ready[g & 1]);
      }
      if (a.dweights) {
        if (wq == 1) sDot[row] = dot;
        asm volatile("bar.sync 2, 256;" ::: "memory");
        if (wq == 0 && flat >= 0 && ok) a.dweights[flat] = dot + sDot[row];
        asm volatile("bar.sync 2, 256;" ::: "memory");
      }
      ok = ok && mbar_wait(de_full, i & 1);
      tc_fence_after();
      // 16 columns at a time, alternately by the two warps of a row quarter
      for (int c0 = wq * 16; c0 < a.e; c0 += 32) {
        float v[16];
        tmem_ld16(tE + lb + c0, v);
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
      mbar_arrive(de_empty);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 13) tmem_dealloc(tmem, 512);
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
  const int fixed = 1024 + 512 + 512 + 4 * 256;   // alignment, barriers, row offsets, choice weights
  c.stages = (232448 - fixed - c.w1_bytes - c.w2_bytes) / c.stage_bytes;
  if (c.stages > 4) c.stages = 4;
  c.smem = fixed + c.w1_bytes + c.w2_bytes + c.stages * c.stage_bytes;
  return c;
}

template <typename Td>
__global__ void __launch_bounds__(kTokThreads, 1)
    routed_wgrad_kernel(const __grid_constant__ RoutedMaps maps, const RoutedBwdArgs a, const WeightPieces w) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const WgCfg cfg = wg_cfg(a.e, a.d);
  const int d = a.d, DB = d / 64;
  uint8_t* sW1 = smem;
  uint8_t* sW2 = sW1 + cfg.w1_bytes;
  uint8_t* sS = sW2 + cfg.w2_bytes;
  float* sWt = (float*)(sS + cfg.stages * cfg.stage_bytes);    // [4][64] choice weights of the stages
  long long* sOff = (long long*)(sWt + 256);                   // [64]
  uint64_t* bars = (uint64_t*)(sOff + 64);
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

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int role = blockIdx.x % cfg.roles, slice = blockIdx.x / cfg.roles;
  const int chunk = role % cfg.chunks, h0 = chunk * 128;
  const bool do1 = role < cfg.chunks;                // DZ, dW1, db1 and db2
  const bool do2 = d <= 256 || !do1;                 // dW2
  if (threadIdx.x == 0) {
    for (int i = 0; i < cfg.stages; ++i) {
      mbar_init(&s_full[i], 128);
      mbar_init(&s_empty[i], 1 + kTokCompute);
    }
    mbar_init(w_full, 1);
    mbar_init(u_full, 1);
    mbar_init(z_ready, kTokCompute);
    mbar_init(z_free, 1);
    mbar_init(dz_full, 1);
    mbar_init(du_ready, kTokCompute);
    mbar_init(du_free, 1);
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, kTokCompute);
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

  const bool fine = plan_ok(a.plan);
  const int T = fine ? a.plan.T : 0;
  const int tile0 = slice * w.per, tile1 = fine ? min(tile0 + w.per, plan_first(a.plan, a.plan.T) / 128) : 0;
  // the slots of behaviour t in this slice: [lo, hi), hi before the padding
  auto piece = [&](int t, int& lo, int& hi) {
    const int first = plan_first(a.plan, t);
    lo = max(tile0 * 128, first);
    hi = min(tile1 * 128, first + plan_count(a.plan, t));
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
        mbar_expect_tx(w_full, cfg.w1_bytes + cfg.w2_bytes);
        for (int b = 0; b < cfg.eb; ++b)
          for (int j = 0; j < 2; ++j)
            tma_load_3d_hint(&maps.w1[t], w_full, sW1 + b * 16384 + j * 8192, b * 64, h0 + j * 64, 0, keep);
        for (int j = 0; j < 2; ++j)
          for (int b = 0; b < DB; ++b)
            tma_load_3d_hint(&maps.w2[t], w_full, sW2 + j * d * 128 + b * 8192, h0 + j * 64, b * 64, 0, keep);
      }
    }
  } else if (warp == 13) {
    // ------------------------------------------------------------- products
    if (lane == 0) {
      const uint64_t dW1 = sdesc_k128(smem_u32(sW1)), dW2 = sdesc_mn128(smem_u32(sW2), d * 128);
      const uint64_t dSk = sdesc_k128(smem_u32(sS)), dSm = sdesc_mn128(smem_u32(sS), 8192);
      const uint32_t id_u = idesc_bf16(128, 64), id_z = idesc_bf16(128, 64, true, false);
      const int n0 = min(d, 256), n1 = d - n0;
      const uint32_t id_2 = idesc_bf16(128, n0, false, true), id_2b = idesc_bf16(128, n1 ? n1 : 16, false, true);
      const uint32_t id_1 = idesc_bf16(128, a.e, false, true);
      const int ksteps = a.e / 16;
      bool ok = true;
      int i = 0, p = 0;              // steps and pieces so far
      auto grad1 = [&](int j, bool fresh) {   // dW1 of step j, then its rows are free
        const int s = j % cfg.stages;
        if (do1) {
          ok = ok && mbar_wait(du_ready, j & 1);
          if (!ok) return;
          tc_fence_after();
          const uint64_t rows = desc_add(dSm, s * cfg.stage_bytes + d * 128);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            umma_bf16_ts(tW1, tZ + k * 16, desc_add(rows, k * 2048), id_1, fresh && !k ? 0u : 1u);
            umma_bf16_ts(tW1, tZ + k * 16 + 8, desc_add(rows, k * 2048), id_1, 1u);
          }
        }
        umma_commit(du_free);
        umma_commit(&s_empty[s]);
      };
      for (int t = 0; t < T && ok; ++t) {
        int lo, hi;
        if (!piece(t, lo, hi)) continue;
        ok = ok && mbar_wait(w_full, p & 1);
        if (p > 0) ok = ok && mbar_wait(acc_empty, (p - 1) & 1);
        const int n = (hi - lo + 63) / 64;
        for (int q = 0; q < n && ok; ++q, ++i) {
          const int s = i % cfg.stages;
          const bool early = cfg.stages == 1;    // the only row stage is free after dW1 of the step before
          if (early && q > 0) grad1(i - 1, q == 1);
          ok = ok && mbar_wait(&s_full[s], (i / cfg.stages) & 1);
          if (i > 0) ok = ok && mbar_wait(z_free, (i - 1) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t rk = desc_add(dSk, s * cfg.stage_bytes), rm = desc_add(dSm, s * cfg.stage_bytes);
          for (int k = 0; k < ksteps; ++k)
            umma_bf16(tU, desc_add(dW1, (k >> 2) * 16384 + (k & 3) * 32),
                      desc_add(rk, d * 128 + (k >> 2) * 8192 + (k & 3) * 32), id_u, k ? 1u : 0u);
          umma_commit(u_full);
          if (q > 0) {
            if (!early) grad1(i - 1, q == 1);
            ok = ok && mbar_wait(du_free, (i - 1) & 1);
          }
          if (!ok) break;
          tc_fence_after();
          if (do1) {
            for (int k = 0; k < DB * 4; ++k)
              umma_bf16(tZ, desc_add(dW2, k * 2048), desc_add(rk, (k >> 2) * 8192 + (k & 3) * 32), id_z, k ? 1u : 0u);
            umma_commit(dz_full);
          }
          ok = mbar_wait(z_ready, i & 1);
          if (!ok) break;
          tc_fence_after();
          if (do2) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t z = tU + k * 16;
              umma_bf16_ts(tW2, z, desc_add(rm, k * 2048), id_2, q || k ? 1u : 0u);
              umma_bf16_ts(tW2, z + 8, desc_add(rm, k * 2048), id_2, 1u);
              if (n1) {
                umma_bf16_ts(tW2 + n0, z, desc_add(rm, n0 * 128 + k * 2048), id_2b, q || k ? 1u : 0u);
                umma_bf16_ts(tW2 + n0, z + 8, desc_add(rm, n0 * 128 + k * 2048), id_2b, 1u);
              }
            }
          }
          umma_commit(z_free);
        }
        if (!ok) break;
        grad1(i - 1, n == 1);
        ok = ok && mbar_wait(du_free, (i - 1) & 1);
        umma_commit(acc_full);
        ++p;
      }
    }
  } else if (warp >= 8) {
    // --------------------------------------------------------------- gather
    const int tid = threadIdx.x - kTokCompute;
    bool ok = true;
    int i = 0;
    for (int t = 0; t < T; ++t) {
      int lo, hi;
      if (!piece(t, lo, hi)) continue;
      for (int at = lo; at < hi; at += 64, ++i) {
        const int s = i % cfg.stages;
        int flat = -1, row = -1;
        if (tid < 64 && at + tid < hi) {
          flat = a.plan.order[at + tid];
          row = flat / a.plan.k;
        }
        if (i >= cfg.stages) ok = ok && mbar_wait(&s_empty[s], ((i / cfg.stages) - 1) & 1);
        uint8_t* to = sS + s * cfg.stage_bytes;
        if (tid < 64) {
          sOff[tid] = row < 0 ? -1LL : (long long)row * a.e;
          sWt[s * 64 + tid] = flat < 0 ? 0.f : a.weights ? a.weights[flat] : 1.f;
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (ok) gather_boxes<128>(to + d * 128, sOff, 64, a.e, a.events, tid);
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (tid < 64) sOff[tid] = row < 0 ? -1LL : token_off(a.rows, row, d);
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (ok) gather_boxes<128>(to, sOff, 64, d, (const Td*)a.dtokens, tid);
        cp_async_wait();
        fence_async_smem();
        asm volatile("bar.sync 1, 128;" ::: "memory");
        mbar_arrive(&s_full[s]);
      }
    }
  } else {
    // -------------------------------------------------------------- compute
    const int q4 = warp & 3, wq = warp >> 2;       // hidden quarter, half of the step's slots
    const uint32_t lb = (uint32_t)(q4 * 32) << 16;
    const int h = h0 + q4 * 32 + lane;
    const int oc = threadIdx.x & 15, og = threadIdx.x >> 4;   // db2: 8 columns, 4 slots a step
    bool ok = true;
    int i = 0, p = 0;
    for (int t = 0; t < T; ++t) {
      int lo, hi;
      if (!piece(t, lo, hi)) continue;
      const float b1 = h < d ? __bfloat162float(((const __nv_bfloat16*)a.mlp.b1[t])[h]) : 0.f;
      float db1 = 0.f, db2[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int at = lo; at < hi; at += 64, ++i) {
        const int s = i % cfg.stages;
        ok = ok && mbar_wait(&s_full[s], (i / cfg.stages) & 1);   // the choice weights
        const float* wt = sWt + s * 64 + wq * 32;
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
        mbar_arrive(z_ready);
        if (do1) {
          ok = ok && mbar_wait(dz_full, i & 1);
          tc_fence_after();
          float y[32];
          tmem_ld32(tZ + col, y);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t pk[16];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int n = hf * 16 + 2 * j;
              const float x0 = y[n] * v[n], x1 = y[n + 1] * v[n + 1];
              db1 += x0 + x1;
              split_bf16x2(x0, x1, pk[j], pk[8 + j]);
            }
            tmem_st16(tZ + col + hf * 16, pk);
          }
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(du_ready);
          const int c = h0 / 8 + oc;   // db2 of output columns h0 + 8 oc .. + 7
          if (c * 8 < d) {
            const uint8_t* box = sS + s * cfg.stage_bytes + (c >> 3) * 8192;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int r = og * 4 + j;
              const uint4 x = *(const uint4*)(box + r * 128 + (((c & 7) ^ (r & 7)) << 4));
              const __nv_bfloat162* xh = (const __nv_bfloat162*)&x;
              const float wr = sWt[s * 64 + r];
#pragma unroll
              for (int n = 0; n < 4; ++n) {
                const float2 f = __bfloat1622float2(xh[n]);
                db2[2 * n] = fmaf(wr, f.x, db2[2 * n]);
                db2[2 * n + 1] = fmaf(wr, f.y, db2[2 * n + 1]);
              }
            }
          }
        }
        mbar_arrive(&s_empty[s]);
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
      mbar_arrive(acc_empty);
      ++p;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 13) tmem_dealloc(tmem, 512);
}

}  // namespace ot
