// Tensor-core kernels of the routed event tokenizer (bf16 mode, d a multiple
// of 64 up to 384, event_dim a multiple of 16 up to 128).
#pragma once
#include "routed.cuh"

namespace ot {

// W1 [d][e] as boxes of 64 event columns x `w1_rows` hidden rows, W2 [d][d]
// as boxes of 64 hidden columns x `w2_rows` output rows, per behaviour.
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
      const int boxes = d > 256 ? 2 : 1, rows = d / boxes;
      for (int g = 0; g < mine * NC; ++g) {
        const int s = g % cfg.stages;
        if (g >= cfg.stages && !mbar_wait(&w_empty[s], ((g / cfg.stages) - 1) & 1)) break;
        const int t = plan_type(a.plan, tile_at(g / NC) * 128), h0 = (g % NC) * 64;
        uint8_t* w1 = sW + s * cfg.stage_bytes;
        mbar_expect_tx(&w_full[s], cfg.stage_bytes);
        for (int b = 0; b < cfg.eb; ++b) tma_load_3d_hint(&maps.w1[t], &w_full[s], w1 + b * 8192, b * 64, h0, 0, keep);
        for (int b = 0; b < boxes; ++b)
          tma_load_3d_hint(&maps.w2[t], &w_full[s], w1 + cfg.w1_bytes + b * rows * 128, h0, b * rows, 0, keep);
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

}  // namespace ot
