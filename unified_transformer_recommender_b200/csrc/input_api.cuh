// Host side of the input layer's C ABI (onetrans_input.h): checks, workspace
// carving and launches of the embedding and routed-tokenizer kernels.
// Included by onetrans.cu after the model, workspace and profiling helpers.
#pragma once

// Raises a kernel's dynamic shared memory limit on the current device (the
// attribute is per device and cheap to set again).
template <typename K>
static bool allow_smem(K kernel, size_t bytes) {
  return bytes <= 48 * 1024 ||
         cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess;
}

// 148 in the rules below: the SMs of a B200, as a constant, since workspace
// sizes are asked for without a device and the order of sums is not to depend
// on one.
static const long long kMaxTableRows = 0x7fffffff, kMaxGradIds = 1LL << 26;
static const int kMaxWidth = 65536;

// Whether groups of n elements that start at p and at multiples of n elements
// after it can be accessed as vectors of 16 bytes at most.
static bool vec_at(const void* p, int n, size_t elem) { return aligned(p, std::min<size_t>(n * elem, 16)); }

static bool mode_ok(int32_t mode) { return mode == ONETRANS_BF16 || mode == ONETRANS_FP32; }

// ----------------------------------------------------------------- lookup --
template <typename Tt, typename To, typename Id>
static onetrans_status lookup_impl(const void* table, long long n_rows, int width, const void* ids, long long R,
                                   float scale, void* out, long long out_ld, cudaStream_t st) {
  // 16 bytes of the narrower type's row per access where the rows keep that
  // alignment (a field inside a wider row may start at any 4 bytes)
  int ve = sizeof(Tt) == 4 && sizeof(To) == 4 ? 4 : 8;
  while (width % ve || out_ld % ve || !vec_at(out, ve, sizeof(To))) ve >>= 1;
  const int groups = width / ve, cpr = std::min(groups, kLookThreads), rpb = kLookThreads / cpr;
  // four rows in flight per thread once that still gives every SM two CTAs
  // (rows of 64 bf16, one row against four: 8192 2.1 / 2.3 us, 65536 4.3 / 4.0,
  // 131072 6.8 / 5.1, 2^20 63 / 49)
  const bool many = R >= 148LL * 2 * 4 * rpb;
  const dim3 grid((unsigned)(many ? std::min(148LL * 6, cdiv(R, 4 * rpb)) : cdiv(R, rpb)), (unsigned)cdiv(groups, cpr));
  ProfScope prof(PK_EMBEDDING, 0.0, (double)R * (sizeof(Id) + width * (double)(sizeof(Tt) + sizeof(To))), st);
  auto go = [&](auto one, auto four) {
    launch_dependent(many ? four : one, grid, dim3(kLookThreads), 0, st, (const Tt*)table, (uint32_t)n_rows, width,
                     (const Id*)ids, R, cpr, scale, (To*)out, out_ld);
  };
  switch (ve) {
    case 8: go(emb_lookup_kernel<Tt, To, Id, 8, 1>, emb_lookup_kernel<Tt, To, Id, 8, 4>); break;
    case 4: go(emb_lookup_kernel<Tt, To, Id, 4, 1>, emb_lookup_kernel<Tt, To, Id, 4, 4>); break;
    case 2: go(emb_lookup_kernel<Tt, To, Id, 2, 1>, emb_lookup_kernel<Tt, To, Id, 2, 4>); break;
    default: go(emb_lookup_kernel<Tt, To, Id, 1, 1>, emb_lookup_kernel<Tt, To, Id, 1, 4>); break;
  }
  return last_launch();
}

// ---------------------------------------------------------------- gradient --
struct EmbGrad {
  const void* dout;
  int dout_mode;
  long long dout_ld;
  const void* ids;
  int ids_bits;
  long long R, n_rows;
  int width;
  float scale;
  float* out;       // dense: the table gradient; sparse: the touched rows
  void* uniq;       // null: dense
  int32_t* n_uniq;
};

// Sort items a thread: the fewer a CTA ranks the sooner a pass is done, until
// the tiles' counts cost more.  Whole sparse gradient of rows of 64, us:
// 37000 ids 2 / 4 items 25.7 / 28.9, 75392 ids 31.6 / 32.0, 150000 ids 53.7 /
// 42.9; 4 / 8 items: 327680 ids 89 / 98, 800000 ids 165 / 168, 2^20 ids 195 /
// 191, 3 million 488 / 468.
static int sort_items(long long R) { return R <= 80 * 1024 ? 2 : R < 1 << 20 ? 4 : 8; }

// Sorted positions a warp: 8 while that leaves all CTAs resident at once (4 an
// SM), then more as the joins of the chunks would cost (whole gradient, rows
// of 64: 1024 ids 8 / 32 positions 9.8 / 13.8 us, 75392 ids 8 / 16 33.8 / 31.4,
// 524288 ids 16 / 32 132 / 120); at most 4096 chunks
static int warp_rows(long long R) {
  return R <= 148 * 4 * 8 * kRedWarps ? 8 : R <= 320 * 1024 ? 16 : 32 * (int)cdiv(R, 1 << 20);
}

// The last R, in no order, before one of the two rules above steps up.  With
// the step come fewer tiles or chunks and so a smaller workspace: a buffer that
// has to serve every call of up to n ids is sized for n and for each of these
// below n.
static const int kGradRuleEnds = 3 + (int)(kMaxGradIds >> 20);
static long long grad_rule_end(int i) {
  switch (i) {
    case 0: return 148 * 4 * 8 * kRedWarps;
    case 1: return 80 * 1024;
    case 2: return 320 * 1024;
    case 3: return (1 << 20) - 1;
    default: return (long long)(i - 3) << 20;
  }
}

static int key_bits(long long n_rows) {
  int b = 1;
  while ((n_rows >> b) != 0) ++b;
  return b;
}

// Tiles whose counts every CTA of a pass adds up itself (it reads tiles x
// digits of them); with more, a scan kernel turns them into prefixes first, a
// launch more a pass.  Whole sparse gradient, rows of 64, popular ids of a
// million, direct / scanned, us: 48 tiles (49152 ids) 29 / 43, 74 (75392 ids)
// 34 / 38, 74 (150000 ids) 43 / 48, 80 (81920 ids) 44 / 42, 96 (196608 ids)
// 57 / 53, 147 (300000 ids) 75 / 70.
static const int kSortDirectTiles = 76;

template <typename T, typename Id, bool DENSE>
static onetrans_status emb_reduce_launch(const EmbGrad& g, ReduceArgs a, cudaStream_t st) {
  int cpl = 1;
  while (cpl < 8 && 32 * cpl < g.width) cpl *= 2;
  while (g.width % cpl || g.dout_ld % cpl || !vec_at(g.dout, cpl, sizeof(T))) cpl >>= 1;
  a.fill = DENSE ? (int)cdiv(g.n_rows, 256) : 0;
  const dim3 grid((unsigned)(a.chunks + a.fill), (unsigned)cdiv(g.width, 32 * cpl));
  const dim3 jgrid((unsigned)a.chunks, grid.y);
  auto go = [&](auto reduce, auto join) {
    launch_dependent(reduce, grid, dim3(32 * kRedWarps), 0, st, (const T*)g.dout, a);
    if (a.chunks > 1) launch_dependent(join, jgrid, dim3(32 * kJoinWarps), 0, st, a);
  };
  switch (cpl) {
    case 8: go(emb_reduce_kernel<T, Id, 8, DENSE>, emb_join_kernel<8>); break;
    case 4: go(emb_reduce_kernel<T, Id, 4, DENSE>, emb_join_kernel<4>); break;
    case 2: go(emb_reduce_kernel<T, Id, 2, DENSE>, emb_join_kernel<2>); break;
    default: go(emb_reduce_kernel<T, Id, 1, DENSE>, emb_join_kernel<1>); break;
  }
  return last_launch();
}

template <typename Id>
static onetrans_status emb_grad_impl(const EmbGrad& g, void* ws, size_t ws_bytes, cudaStream_t st, size_t* need) {
  const long long R = g.R;
  const int items = sort_items(R), tile = kSortThreads * items;
  const int tiles = (int)cdiv(R, tile);
  const int chunk = kRedWarps * warp_rows(R);
  const int chunks = (int)cdiv(R, chunk);
  Carve cv(ws, ws_bytes);
  uint32_t* keys[2];
  uint32_t* vals[2];
  for (int i = 0; i < 2; ++i) {
    keys[i] = (uint32_t*)cv.take(R * 4);
    vals[i] = (uint32_t*)cv.take(R * 4);
  }
  const int max_passes = (31 + kSortMaxBits - 1) / kSortMaxBits;
  int* hist = (int*)cv.take(((size_t)tiles * max_passes + 1) * (sizeof(int) << kSortMaxBits));
  int* heads = (int*)cv.take((size_t)chunks * 4);
  float* first = (float*)cv.take((size_t)chunks * g.width * 4);
  float* tail = (float*)cv.take((size_t)chunks * g.width * 4);
  int* state = (int*)cv.take((size_t)chunks * 4);
  long long* tail_row = (long long*)cv.take((size_t)chunks * 8);
  if (need) {
    *need = cv.used;
    return ONETRANS_OK;
  }
  if (cv.overflow) return ONETRANS_ERR_CAPACITY;

  const bool dense = !g.uniq;
  const uint32_t n_rows = (uint32_t)g.n_rows;
  const int bits = key_bits(g.n_rows);
  const int passes = (int)cdiv(bits, kSortMaxBits), per = std::max((int)cdiv(bits, passes), kSortMinBits), bins = 1 << per;
  const double row_bytes = (double)R * g.width * (g.dout_mode == ONETRANS_BF16 ? 2 : 4);
  ProfScope prof(PK_EMBEDDING_GRAD, (double)R * g.width,
                 row_bytes + (double)R * sizeof(Id) +
                     (double)(dense ? g.n_rows : std::min(R, g.n_rows)) * g.width * 4, st);
  int at = 0;   // the sorted pairs are in keys[at], vals[at]
  const bool ranked = R <= kRankMax;
  if (R > 0 && ranked) {
    launch_dependent(sort_rank_kernel<Id>, dim3((unsigned)cdiv(R, kRankThreads / 32 * kRankIds)), dim3(kRankThreads), 0,
                     st, (const Id*)g.ids, n_rows, (int)R, keys[0], vals[0]);
  } else if (R > 0) {
    const long long per_pass = (long long)tiles * bins;
    SortArgs a;
    std::memset(&a, 0, sizeof(a));
    a.n_rows = n_rows;
    a.R = R;
    a.tile = tile;
    a.tiles = tiles;
    a.bits = per;
    a.tot = hist + per_pass * passes;
    a.hist = hist;
    a.hist_next = hist + per_pass;
    a.scanned = tiles > kSortDirectTiles;
    launch_dependent(sort_hist_kernel<Id>, dim3(tiles), dim3(kSortThreads), 0, st, (const Id*)g.ids, a,
                     per_pass * (passes - 1));
    const size_t smem = (size_t)tile * 8 + (size_t)bins * 8 + (size_t)kSortWarps * bins * 2;
    auto pass = [&](auto first, auto later) {
      if (!allow_smem(first, smem) || !allow_smem(later, smem)) return ONETRANS_ERR_CUDA;
      for (int p = 0; p < passes; ++p) {
        a.shift = p * per;
        a.hist = hist + per_pass * p;
        a.hist_next = p + 1 < passes ? a.hist + per_pass : nullptr;
        if (a.scanned) launch_dependent(sort_scan_kernel, dim3((unsigned)cdiv(bins, 32)), dim3(1024), 0, st, a);
        const uint32_t *ki = keys[at], *vi = vals[at];
        if (p > 0) at ^= 1;
        launch_dependent(p == 0 ? first : later, dim3(tiles), dim3(kSortThreads), smem, st,
                         p == 0 ? (const Id*)g.ids : nullptr, ki, vi, keys[at], vals[at], a, per, a.shift + per);
      }
      return ONETRANS_OK;
    };
    OT_TRY(items == 2   ? pass(sort_pass_kernel<Id, true, 2>, sort_pass_kernel<Id, false, 2>)
           : items == 4 ? pass(sort_pass_kernel<Id, true, 4>, sort_pass_kernel<Id, false, 4>)
                        : pass(sort_pass_kernel<Id, true, 8>, sort_pass_kernel<Id, false, 8>));
    if (!dense)
      launch_dependent(emb_heads_kernel, dim3(chunks), dim3(256), 0, st, (const uint32_t*)keys[at], R, n_rows, chunk,
                       heads);
  }
  OT_TRY(last_launch());
  ReduceArgs r;
  std::memset(&r, 0, sizeof(r));
  r.keys = keys[at]; r.vals = vals[at];
  r.n_rows = n_rows;
  r.R = R; r.dout_ld = g.dout_ld;
  r.width = g.width; r.chunk = chunk; r.chunks = chunks;
  r.scale = g.scale;
  r.out = g.out; r.uniq = g.uniq; r.n_uniq = g.n_uniq;
  r.heads = ranked ? nullptr : heads; r.first = first; r.tail = tail; r.state = state; r.tail_row = tail_row;
  if (g.dout_mode == ONETRANS_BF16)
    return dense ? emb_reduce_launch<__nv_bfloat16, int32_t, true>(g, r, st)
                 : emb_reduce_launch<__nv_bfloat16, Id, false>(g, r, st);
  return dense ? emb_reduce_launch<float, int32_t, true>(g, r, st) : emb_reduce_launch<float, Id, false>(g, r, st);
}

static onetrans_status emb_grad_check(const onetrans_model* m, const EmbGrad& g) {
  if (!m || !mode_ok(g.dout_mode) || (g.ids_bits != 32 && g.ids_bits != 64)) return ONETRANS_ERR_INVALID_ARG;
  if (g.R < 0 || g.R > kMaxGradIds || g.n_rows < 1 || g.n_rows > kMaxTableRows || g.width < 1 ||
      g.width > kMaxWidth || g.dout_ld < g.width)
    return ONETRANS_ERR_SHAPE;
  return ONETRANS_OK;
}

static onetrans_status emb_grad_run(const EmbGrad& g, void* ws, size_t ws_bytes, cudaStream_t st) {
  if (g.R > 0 && (!g.dout || !g.ids || !ws || !aligned(g.dout, 4) || !aligned(g.ids, 16) || !aligned(ws, 256)))
    return ONETRANS_ERR_INVALID_ARG;
  return g.ids_bits == 32 ? emb_grad_impl<int32_t>(g, ws, ws_bytes, st, nullptr)
                          : emb_grad_impl<int64_t>(g, ws, ws_bytes, st, nullptr);
}

// ------------------------------------------------------- routed tokenizer --
static const long long kMaxChoicesTotal = 1LL << 26;   // R * k

// The plan in the caller's buffer.
struct PlanBuf {
  int* head;
  int* order;
  int* pos;
  int* counts;       // per tile, while the plan is made
  long long cap;     // slots: every choice, each behaviour filled up to 128
  int tiles;
  size_t bytes;
};
static PlanBuf plan_buf(const onetrans_model* m, void* base, long long R, int k) {
  PlanBuf p;
  const long long n = R * k;
  Carve cv(base, 0);
  p.cap = cdiv(n, 128) * 128 + 128LL * m->cfg.n_behaviors;
  p.tiles = (int)cdiv(n, kRouteTile);
  p.head = (int*)cv.take(kPlanHeader * sizeof(int));
  p.order = (int*)cv.take((size_t)p.cap * sizeof(int));
  p.pos = (int*)cv.take((size_t)n * sizeof(int));
  p.counts = (int*)cv.take((size_t)(p.tiles + 1) * kMaxTypes * sizeof(int));   // and the totals
  p.bytes = cv.used;
  return p;
}
static PlanView plan_view(const onetrans_model* m, const PlanBuf& p, long long R, int k) {
  return PlanView{p.head, p.order, p.pos, (int)R, k, m->cfg.n_behaviors};
}

static bool has_behavior_mlps(const onetrans_model* m) {
  if (m->cfg.n_behaviors < 1 || m->cfg.event_dim < 1 || m->Wb1.empty() || !m->type_emb) return false;
  return true;
}

// What every call on routed events checks: the model, the sizes, and the
// behaviour weights' pointers (model_create leaves those unchecked).
static onetrans_status routed_check(const onetrans_model* m, long long R, int k) {
  if (!m) return ONETRANS_ERR_INVALID_ARG;
  if (!has_behavior_mlps(m)) return ONETRANS_ERR_UNSUPPORTED;
  if (R < 0 || k < 1 || k > kMaxChoices || R > kMaxChoicesTotal / k) return ONETRANS_ERR_SHAPE;
  for (int t = 0; t < m->cfg.n_behaviors; ++t)
    for (const void* p : {m->Wb1[t], m->bb1[t], m->Wb2[t], m->bb2[t]})
      if (!p || !aligned(p, 16)) return ONETRANS_ERR_INVALID_ARG;
  if (!aligned(m->type_emb, 16)) return ONETRANS_ERR_INVALID_ARG;
  return ONETRANS_OK;
}
// With R <= per (any per) there is one sample and its stride is not looked at.
static onetrans_status token_rows_check(const onetrans_model* m, long long R, long long per, long long sample_ld) {
  if (per < 1 || (R > per && sample_ld < per * m->d)) return ONETRANS_ERR_SHAPE;
  return ONETRANS_OK;
}
// The stride of a lone sample is 0 from here on, so that no choice of kernels
// or accesses depends on it.
static TokenRows token_rows(long long R, long long per, long long sample_ld) {
  return R <= per ? TokenRows{0x7fffffff, 0} : TokenRows{(int)per, sample_ld};
}

static RoutedMLP routed_mlp_of(const onetrans_model* m) {
  RoutedMLP w;
  std::memset(&w, 0, sizeof(w));
  for (int t = 0; t < m->cfg.n_behaviors; ++t) {
    w.W1[t] = m->Wb1[t]; w.b1[t] = m->bb1[t]; w.W2[t] = m->Wb2[t]; w.b2[t] = m->bb2[t];
  }
  w.emb = m->type_emb;
  return w;
}

static onetrans_status route_impl(const onetrans_model* m, const int32_t* types, long long R, int k, const PlanBuf& p,
                                  cudaStream_t st) {
  const int n = (int)(R * k), T = m->cfg.n_behaviors;
  ProfScope prof(PK_ROUTE, 0.0, (double)n * 12, st);
  if (p.tiles > 1)
    launch_dependent(route_count_kernel, dim3(p.tiles), dim3(kRouteThreads), 0, st, types, n, T, p.counts);
  // every CTA adding up all tiles' counts costs tiles^2 reads; past 2.6 million
  // choices a scan does it once (direct / scan: 1.5 million 16.3 / 19.8 us, 3
  // million 33.2 / 31.8, 10 million 259 / 110)
  int* tot = nullptr;
  if (p.tiles > 2560) {
    SortArgs a;
    std::memset(&a, 0, sizeof(a));
    a.tiles = p.tiles;
    a.bits = 3;
    a.hist = p.counts;
    a.tot = tot = p.counts + (size_t)p.tiles * kMaxTypes;
    static_assert(kMaxTypes == 8, "three bits of behaviour");
    launch_dependent(sort_scan_kernel, dim3(1), dim3(1024), 0, st, a);
  }
  launch_dependent(route_place_kernel, dim3(p.tiles), dim3(kRouteThreads), 0, st, types, n, (int)R, k, T,
                   (const int*)p.counts, (const int*)tot, p.head, p.order, p.pos);
  return last_launch();
}

template <typename T>
static onetrans_status combine_launch(const PlanView& plan, const float* part, int width, void* out,
                                      const TokenRows& rows, cudaStream_t st) {
  const bool wide = width % 8 == 0 && rows.sample_ld % 8 == 0;
  const long long items = (long long)plan.R * (width / (wide ? 8 : 1));
  const dim3 grid((unsigned)std::min<long long>(cdiv(items, 256), 148 * 8));
  if (wide) launch_dependent(routed_combine_kernel<T, 8>, grid, dim3(256), 0, st, plan, part, width, (T*)out, rows);
  else launch_dependent(routed_combine_kernel<T, 1>, grid, dim3(256), 0, st, plan, part, width, (T*)out, rows);
  return last_launch();
}

// Shapes the tensor-core kernels take (d 256, e 64, tensor cores / CUDA cores:
// tokens of 16 events 16.5 / 26.6 us, of 75392 29 / 453; gradient 39 / 47 and
// 109 / 1272).  TMEM holds 512 columns: D of d and at least one U of 64 beside
// it, or dW2 of d and one U of 128; the event rows are one or two boxes of 64.
static bool routed_tc(const onetrans_model* m) {
  const int d = m->d, e = m->cfg.event_dim;
  return m->bf16 && d % 64 == 0 && d <= 384 && e % 16 == 0 && e <= 128;
}
// f(integral constant of d / 64)
template <typename F>
static onetrans_status by_chunks(int d, F f) {
  switch (d / 64) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 3: return f(std::integral_constant<int, 3>());
    case 4: return f(std::integral_constant<int, 4>());
    case 5: return f(std::integral_constant<int, 5>());
    case 6: return f(std::integral_constant<int, 6>());
    default: return ONETRANS_ERR_UNSUPPORTED;
  }
}
static onetrans_status routed_maps(const onetrans_model* m, const RoutedMaps** out) {
  std::lock_guard<std::mutex> lk(m->maps_mu);
  if (!m->maps_made) {
    const int d = m->d, e = m->cfg.event_dim;
    for (int t = 0; t < kMaxTypes; ++t) {
      const int u = std::min(t, m->cfg.n_behaviors - 1);
      if (!make_tmap_3d(&m->maps.w1[t], m->Wb1[u], e, d, 1, e, (uint64_t)e * d, 64, 64, 1) ||
          !make_tmap_3d(&m->maps.w2[t], m->Wb2[u], d, d, 1, d, (uint64_t)d * d, 64, 64, 1))
        return ONETRANS_ERR_CUDA;
    }
    m->maps_made = true;
  }
  *out = &m->maps;
  return ONETRANS_OK;
}

struct RoutedCall {
  const void* events;
  const float* weights;
  long long R;
  int k;
  const PlanBuf* plan;
  void* tokens;           // forward
  const void* dtokens;    // backward
  int dtokens_mode;
  TokenRows rows;
  void* devents;
  float* dweights;
  RoutedGrads grads;
};

// One product of the CUDA-core path over `columns` output columns; see the
// kernel for when two groups of threads share a CTA.
template <typename T, typename Td, int STEP>
static onetrans_status simt_launch(const RoutedArgs& a, int columns, long long cap, cudaStream_t st) {
  const long long ctas = cdiv(columns, 64) * (cap / 64);
  if (ctas <= 148 * 2)
    launch_dependent(routed_simt_kernel<T, Td, STEP, 2>, dim3((unsigned)ctas), dim3(512), 0, st, a);
  else
    launch_dependent(routed_simt_kernel<T, Td, STEP, 1>, dim3((unsigned)ctas), dim3(256), 0, st, a);
  return last_launch();
}

template <typename T>
static onetrans_status tokenize_routed_impl(const onetrans_model* m, const RoutedCall* c, long long R, int k, void* ws,
                                            size_t ws_bytes, cudaStream_t st, size_t* need) {
  const int d = m->d, e = m->cfg.event_dim;
  const long long cap = plan_buf(m, nullptr, R, k).cap;
  const bool tc = routed_tc(m) && g_policy == 0 && (!c || c->rows.sample_ld % 8 == 0);
  Carve cv(ws, ws_bytes);
  float* part = k > 1 ? (float*)cv.take((size_t)R * k * d * 4) : nullptr;
  // the hidden rows of the CUDA-core kernels (sized for them whatever runs)
  float* hidden = (float*)cv.take((size_t)cap * d * 4);
  if (need) {
    *need = cv.used;
    return ONETRANS_OK;
  }
  if (cv.overflow) return ONETRANS_ERR_CAPACITY;
  RoutedArgs a;
  std::memset(&a, 0, sizeof(a));
  a.plan = plan_view(m, *c->plan, R, k);
  a.mlp = routed_mlp_of(m);
  a.e = e; a.d = d;
  a.events = c->events; a.weights = c->weights; a.tokens = c->tokens; a.rows = c->rows;
  a.buf0 = hidden; a.part = part;
  ProfScope prof(PK_ROUTED, 2.0 * R * k * ((double)e * d + (double)d * d), (double)R * (e + d) * m->es, st);
  if (tc) {
    const RoutedMaps* maps;
    OT_TRY(routed_maps(m, &maps));
    RoutedTcArgs ta;
    std::memset(&ta, 0, sizeof(ta));
    ta.plan = a.plan; ta.mlp = a.mlp; ta.e = e;
    ta.events = (const __nv_bfloat16*)c->events; ta.weights = c->weights;
    ta.tokens = (__nv_bfloat16*)c->tokens; ta.rows = c->rows; ta.part = part;
    const int smem = tok_cfg(e, d).smem;
    const unsigned grid = (unsigned)std::min<long long>(cap / 128, device_sm_count());
    OT_TRY(by_chunks(d, [&](auto nc) {
      constexpr int NC = decltype(nc)::value;
      auto go = [&](auto kernel) {
        if (!allow_smem(kernel, smem)) return ONETRANS_ERR_CUDA;
        launch_dependent(kernel, dim3(grid), dim3(kTokThreads), smem, st, *maps, ta);
        return last_launch();
      };
      return k > 1 ? go(routed_tokens_kernel<NC, true>) : go(routed_tokens_kernel<NC, false>);
    }));
    return k > 1 ? combine_launch<T>(a.plan, part, d, c->tokens, c->rows, st) : ONETRANS_OK;
  }
  OT_TRY((simt_launch<T, T, RS_HIDDEN>(a, d, cap, st)));
  OT_TRY((simt_launch<T, T, RS_TOKEN>(a, d, cap, st)));
  return combine_launch<T>(a.plan, part, d, c->tokens, c->rows, st);
}

// Slices of the weight gradients: `ctas` of them where that is no more than
// one a tile, and as many more as keep a slice within kPieceTiles tiles.  A
// piece is summed in float32 by one CTA, on tensor cores by additions that
// truncate, 16 a tile: about 3e-7 of the piece is lost a tile (75392 events, 16
// tiles a piece, 5.5e-6; 151552 events, 32 tiles, 1.0e-5).  Without the second
// rule 10^6 events were off by 6.4e-5, 4 million by 2.5e-4, and so on; with it
// none is by more than about 2e-5.
static const int kPieceTiles = 64;
static int weight_slices(long long tiles, long long ctas) {
  return (int)std::max<long long>({1, std::min<long long>(tiles, ctas), cdiv(tiles, kPieceTiles)});
}

static onetrans_status wsum_launch(const PlanView& plan, const WeightPieces& w1, const WeightPieces& w2, int d, int e,
                                   int T, const RoutedGrads& g, cudaStream_t st) {
  const int v = d % 4 == 0 && e % 4 == 0 ? 4 : 1;
  const dim3 grid((unsigned)std::min<long long>(cdiv(w1.stride + w2.stride, 256 * v), 1024), T);
  if (v == 4) launch_dependent(routed_wsum_kernel<4>, grid, dim3(256), 0, st, plan, w1, w2, d, e, g);
  else launch_dependent(routed_wsum_kernel<1>, grid, dim3(256), 0, st, plan, w1, w2, d, e, g);
  return last_launch();
}

template <typename T, typename Td>
static onetrans_status dweight_launch(const PlanView& plan, const RoutedMLP& mlp, int d, const void* dtokens,
                                      const TokenRows& rows, const float* dot, int parts, float* dweights,
                                      cudaStream_t st) {
  const long long n = (long long)plan.R * plan.k;
  launch_dependent(routed_dweight_kernel<T, Td>, dim3((unsigned)std::min<long long>(cdiv(n, 8), 148 * 8)), dim3(256), 0,
                   st, plan, mlp, d, (const Td*)dtokens, rows, dot, parts, dweights);
  return last_launch();
}

template <typename T, typename Td>
static onetrans_status routed_backward_simt(const onetrans_model* m, const RoutedCall* c, long long R, int k, void* ws,
                                            size_t ws_bytes, cudaStream_t st, size_t* need) {
  const int d = m->d, e = m->cfg.event_dim, T_n = m->cfg.n_behaviors;
  const long long cap = plan_buf(m, nullptr, R, k).cap, tiles = cap / 128;
  const int nb = (int)cdiv(d, 64), eb = (int)cdiv(e, 64);
  const int n2 = nb * nb, n1 = nb * eb;
  WeightPieces w1, w2;
  w1.slices = weight_slices(tiles, cdiv(148 * 4, n2 + n1));   // four CTAs an SM
  w1.per = (int)cdiv(tiles, w1.slices);
  w2 = w1;
  w1.stride = (long long)d * e + d;
  w2.stride = (long long)d * d + d;
  Carve cv(ws, ws_bytes);
  RoutedArgs a;
  std::memset(&a, 0, sizeof(a));
  a.part = k > 1 ? (float*)cv.take((size_t)R * k * e * 4) : nullptr;
  a.buf0 = (float*)cv.take((size_t)cap * d * 4);
  a.buf1 = (float*)cv.take((size_t)cap * d * 4);
  a.dot = (float*)cv.take((size_t)cap * nb * 4);
  w1.part = (float*)cv.take((size_t)(w1.slices + T_n) * w1.stride * 4);
  w2.part = (float*)cv.take((size_t)(w2.slices + T_n) * w2.stride * 4);
  if (need) {
    *need = cv.used;
    return ONETRANS_OK;
  }
  if (cv.overflow) return ONETRANS_ERR_CAPACITY;
  a.plan = plan_view(m, *c->plan, R, k);
  a.mlp = routed_mlp_of(m);
  a.e = e; a.d = d;
  a.events = c->events; a.weights = c->weights; a.dtokens = c->dtokens; a.rows = c->rows; a.devents = c->devents;
  ProfScope prof(PK_ROUTED_GRAD, 2.0 * R * k * (3.0 * e * d + 2.0 * d * d), (double)R * (2 * e + d) * m->es, st);
  OT_TRY((simt_launch<T, Td, RS_DU>(a, d, cap, st)));
  launch_dependent(routed_wgrad_simt_kernel<T, Td>, dim3(n2 + n1, w1.slices), dim3(256), 0, st, a, w1, w2, n2);
  OT_TRY(last_launch());
  OT_TRY(wsum_launch(a.plan, w1, w2, d, e, T_n, c->grads, st));
  if (c->devents) {
    OT_TRY((simt_launch<T, Td, RS_DEVENT>(a, e, cap, st)));
    OT_TRY(combine_launch<T>(a.plan, a.part, e, c->devents, TokenRows{0x7fffffff, 0}, st));
  }
  if (c->dweights)
    return dweight_launch<T, Td>(a.plan, a.mlp, d, c->dtokens, c->rows, a.dot, nb, c->dweights, st);
  return ONETRANS_OK;
}

static onetrans_status routed_backward_tc(const onetrans_model* m, const RoutedCall* c, long long R, int k, void* ws,
                                          size_t ws_bytes, cudaStream_t st, size_t* need) {
  const int d = m->d, e = m->cfg.event_dim, T = m->cfg.n_behaviors;
  const long long cap = plan_buf(m, nullptr, R, k).cap, tiles = cap / 128;
  const WgCfg wc = wg_cfg(e, d);
  WgArgs w;
  std::memset(&w, 0, sizeof(w));
  w.p1.slices = weight_slices(tiles, 74 / wc.chunks);   // both roles of every hidden chunk on the 148 SMs at once
  w.p1.per = (int)cdiv(tiles, w.p1.slices);
  w.p2 = w.p1;
  w.p1.stride = (long long)d * e + d;
  w.p2.stride = (long long)d * d + d;
  Carve cv(ws, ws_bytes);
  w.p1.part = (float*)cv.take((size_t)(w.p1.slices + T) * w.p1.stride * 4);
  w.p2.part = (float*)cv.take((size_t)(w.p2.slices + T) * w.p2.stride * 4);
  w.du = (__nv_bfloat16*)cv.take((size_t)cap * d * 2);
  w.dot = (float*)cv.take((size_t)cap * wc.chunks * 4 * 4);
  float* part = k > 1 ? (float*)cv.take((size_t)R * k * e * 4) : nullptr;
  __nv_bfloat16* rounded = (__nv_bfloat16*)cv.take((size_t)R * d * 2);   // of float32 dtokens
  if (need) {
    *need = cv.used;
    return ONETRANS_OK;
  }
  if (cv.overflow) return ONETRANS_ERR_CAPACITY;
  const RoutedMaps* maps;
  OT_TRY(routed_maps(m, &maps));
  RoutedTcArgs a;
  std::memset(&a, 0, sizeof(a));
  a.plan = plan_view(m, *c->plan, R, k);
  a.mlp = routed_mlp_of(m);
  a.e = e;
  a.events = (const __nv_bfloat16*)c->events; a.weights = c->weights;
  a.dtokens = (const __nv_bfloat16*)c->dtokens; a.rows = c->rows;
  a.devents = k == 1 ? (__nv_bfloat16*)c->devents : nullptr;
  a.part = k > 1 ? part : nullptr;
  ProfScope prof(PK_ROUTED_GRAD, 2.0 * R * k * (3.0 * e * d + 2.0 * d * d), (double)R * (2 * e + d) * m->es, st);
  const bool f32 = c->dtokens_mode == ONETRANS_FP32;
  if (f32) {
    launch_dependent(routed_round_rows_kernel, dim3((unsigned)std::min<long long>(cdiv(R * (d / 8), 256), 148 * 8)),
                     dim3(256), 0, st, (const float*)c->dtokens, c->rows, (int)R, d, rounded);
    OT_TRY(last_launch());
    a.dtokens = rounded;
    a.rows = TokenRows{0x7fffffff, 0};
  }
  if (!c->devents) w.du = nullptr;
  if (!c->dweights) w.dot = nullptr;
  const dim3 grid(wc.chunks * (w.p1.slices + w.p2.slices));
  OT_TRY(by_chunks(d, [&](auto nc) {
    constexpr int NC = decltype(nc)::value;
    auto go = [&](auto kernel) {
      if (!allow_smem(kernel, wc.smem)) return ONETRANS_ERR_CUDA;
      launch_dependent(kernel, grid, dim3(kWgThreads), wc.smem, st, *maps, a, w);
      return last_launch();
    };
    return w.dot ? go(routed_wgrad_kernel<NC, true>) : go(routed_wgrad_kernel<NC, false>);
  }));
  OT_TRY(wsum_launch(a.plan, w.p1, w.p2, d, e, T, c->grads, st));
  if (c->devents) {
    const int smem = dev_cfg(e, d).smem;
    OT_TRY(by_chunks(d, [&](auto nc) {
      constexpr int NC = decltype(nc)::value;
      if (!allow_smem(routed_devents_kernel<NC>, smem)) return ONETRANS_ERR_CUDA;
      launch_dependent(routed_devents_kernel<NC>, dim3((unsigned)std::min<long long>(tiles, device_sm_count())),
                       dim3(kDevThreads), smem, st, *maps, a, (const __nv_bfloat16*)w.du);
      return last_launch();
    }));
    if (part) OT_TRY(combine_launch<__nv_bfloat16>(a.plan, part, e, c->devents, TokenRows{0x7fffffff, 0}, st));
  }
  if (!c->dweights) return ONETRANS_OK;
  return f32 ? dweight_launch<__nv_bfloat16, float>(a.plan, a.mlp, d, c->dtokens, c->rows, w.dot, wc.chunks * 4, c->dweights, st)
             : dweight_launch<__nv_bfloat16, __nv_bfloat16>(a.plan, a.mlp, d, c->dtokens, c->rows, w.dot, wc.chunks * 4,
                                                            c->dweights, st);
}

static onetrans_status tokenize_routed_any(const onetrans_model* m, const RoutedCall* c, long long R, int k, void* ws,
                                           size_t ws_bytes, cudaStream_t st, size_t* need) {
  return m->bf16 ? tokenize_routed_impl<__nv_bfloat16>(m, c, R, k, ws, ws_bytes, st, need)
                 : tokenize_routed_impl<float>(m, c, R, k, ws, ws_bytes, st, need);
}
static onetrans_status routed_backward_any(const onetrans_model* m, const RoutedCall* c, long long R, int k, void* ws,
                                           size_t ws_bytes, cudaStream_t st, size_t* need) {
  const bool f32 = c && c->dtokens_mode == ONETRANS_FP32;
  if (!m->bf16) return routed_backward_simt<float, float>(m, c, R, k, ws, ws_bytes, st, need);
  if (routed_tc(m) && need) {   // whichever kernels the policy picks later
    size_t tc = 0;
    OT_TRY(routed_backward_tc(m, nullptr, R, k, nullptr, 0, nullptr, &tc));
    OT_TRY((routed_backward_simt<__nv_bfloat16, float>(m, nullptr, R, k, nullptr, 0, nullptr, need)));
    *need = std::max(*need, tc);
    return ONETRANS_OK;
  }
  if (routed_tc(m) && g_policy == 0 && c->rows.sample_ld % 8 == 0)
    return routed_backward_tc(m, c, R, k, ws, ws_bytes, st, need);
  return f32 ? routed_backward_simt<__nv_bfloat16, float>(m, c, R, k, ws, ws_bytes, st, need)
             : routed_backward_simt<__nv_bfloat16, __nv_bfloat16>(m, c, R, k, ws, ws_bytes, st, need);
}

// ============================================================== C ABI ====
extern "C" {

onetrans_status onetrans_input_workspace_size(const onetrans_model* m, int32_t op, int64_t n, int32_t L,
                                              size_t* bytes) {
  if (!m || !bytes) return ONETRANS_ERR_INVALID_ARG;
  *bytes = 0;
  if (n < 0 || L < 1) return ONETRANS_ERR_SHAPE;
  switch (op) {
    case ONETRANS_OP_EMBEDDING_BACKWARD: {
      if (n > kMaxGradIds || L > kMaxWidth) return ONETRANS_ERR_SHAPE;
      EmbGrad g;
      std::memset(&g, 0, sizeof(g));
      g.R = n;
      g.width = L;
      OT_TRY(emb_grad_impl<int32_t>(g, nullptr, 0, nullptr, bytes));
      for (int i = 0; i < kGradRuleEnds; ++i) {   // and whatever a call of fewer ids takes
        size_t need = 0;
        g.R = grad_rule_end(i);
        if (g.R >= n) continue;
        OT_TRY(emb_grad_impl<int32_t>(g, nullptr, 0, nullptr, &need));
        *bytes = std::max(*bytes, need);
      }
      return ONETRANS_OK;
    }
    case ONETRANS_OP_ROUTE:
      OT_TRY(routed_check(m, n, L));
      *bytes = plan_buf(m, nullptr, n, L).bytes;
      return ONETRANS_OK;
    case ONETRANS_OP_ROUTED:
      OT_TRY(routed_check(m, n, L));
      return tokenize_routed_any(m, nullptr, n, L, nullptr, 0, nullptr, bytes);
    case ONETRANS_OP_ROUTED_BACKWARD:
      OT_TRY(routed_check(m, n, L));
      return routed_backward_any(m, nullptr, n, L, nullptr, 0, nullptr, bytes);
    default:
      return ONETRANS_ERR_INVALID_ARG;
  }
}

onetrans_status onetrans_embedding_lookup(const onetrans_model* m, const void* table, int32_t table_mode,
                                          int64_t n_rows, int32_t width, const void* ids, int32_t ids_bits, int64_t R,
                                          float scale, void* out, int64_t out_ld, void* stream) {
  if (!m || !mode_ok(table_mode) || (ids_bits != 32 && ids_bits != 64)) return ONETRANS_ERR_INVALID_ARG;
  if (R < 0 || R > kMaxTableRows || n_rows < 1 || n_rows > kMaxTableRows || width < 1 || width > kMaxWidth ||
      out_ld < width)
    return ONETRANS_ERR_SHAPE;
  if (R == 0) return ONETRANS_OK;
  if (!table || !ids || !out || !aligned(table, 16) || !aligned(ids, 16) || !aligned(out, 4))
    return ONETRANS_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  const bool tb = table_mode == ONETRANS_BF16, w = ids_bits == 64;
  auto go = [&](auto t, auto o) {
    using Tt = decltype(t);
    using To = decltype(o);
    return w ? lookup_impl<Tt, To, int64_t>(table, n_rows, width, ids, R, scale, out, out_ld, st)
             : lookup_impl<Tt, To, int32_t>(table, n_rows, width, ids, R, scale, out, out_ld, st);
  };
  if (tb) return m->bf16 ? go(__nv_bfloat16(), __nv_bfloat16()) : go(__nv_bfloat16(), float());
  return m->bf16 ? go(float(), __nv_bfloat16()) : go(float(), float());
}

onetrans_status onetrans_embedding_backward(const onetrans_model* m, const void* dout, int32_t dout_mode,
                                            int64_t dout_ld, const void* ids, int32_t ids_bits, int64_t R,
                                            int64_t n_rows, int32_t width, float scale, float* dtable, void* ws,
                                            size_t ws_bytes, void* stream) {
  const EmbGrad g{dout, dout_mode, dout_ld, ids, ids_bits, R, n_rows, width, scale, dtable, nullptr, nullptr};
  OT_TRY(emb_grad_check(m, g));
  if (!dtable || !aligned(dtable, 16)) return ONETRANS_ERR_INVALID_ARG;
  return emb_grad_run(g, ws, ws_bytes, (cudaStream_t)stream);
}

onetrans_status onetrans_embedding_backward_sparse(const onetrans_model* m, const void* dout, int32_t dout_mode,
                                                   int64_t dout_ld, const void* ids, int32_t ids_bits, int64_t R,
                                                   int64_t n_rows, int32_t width, float scale, void* uniq,
                                                   float* rows, int32_t* n_uniq, void* ws, size_t ws_bytes,
                                                   void* stream) {
  const EmbGrad g{dout, dout_mode, dout_ld, ids, ids_bits, R, n_rows, width, scale, rows, uniq, n_uniq};
  OT_TRY(emb_grad_check(m, g));
  if (!n_uniq || !aligned(n_uniq, 16)) return ONETRANS_ERR_INVALID_ARG;
  if (R == 0) return cuda_ok(cudaMemsetAsync(n_uniq, 0, sizeof(int32_t), (cudaStream_t)stream));
  if (!uniq || !rows || !aligned(uniq, 16) || !aligned(rows, 16)) return ONETRANS_ERR_INVALID_ARG;
  return emb_grad_run(g, ws, ws_bytes, (cudaStream_t)stream);
}

onetrans_status onetrans_route_events(const onetrans_model* m, const int32_t* types, int64_t R, int32_t k, void* plan,
                                      size_t plan_bytes, void* stream) {
  OT_TRY(routed_check(m, R, k));
  if (R == 0) return ONETRANS_OK;
  if (!types || !plan || !aligned(types, 16) || !aligned(plan, 256)) return ONETRANS_ERR_INVALID_ARG;
  const PlanBuf p = plan_buf(m, plan, R, k);
  if (p.bytes > plan_bytes) return ONETRANS_ERR_CAPACITY;
  return route_impl(m, types, R, k, p, (cudaStream_t)stream);
}

onetrans_status onetrans_tokenize_routed(const onetrans_model* m, const void* events, const float* weights, int64_t R,
                                         int32_t k, const void* plan, size_t plan_bytes, void* tokens,
                                         int64_t rows_per_sample, int64_t sample_ld, void* ws, size_t ws_bytes,
                                         void* stream) {
  OT_TRY(routed_check(m, R, k));
  OT_TRY(token_rows_check(m, R, rows_per_sample, sample_ld));
  if (R == 0) return ONETRANS_OK;
  if (!events || !plan || !tokens || !ws || !aligned(events, 16) || !aligned(weights, 16) || !aligned(plan, 256) ||
      !aligned(tokens, 16) || !aligned(ws, 256))
    return ONETRANS_ERR_INVALID_ARG;
  const PlanBuf p = plan_buf(m, const_cast<void*>(plan), R, k);
  if (p.bytes > plan_bytes) return ONETRANS_ERR_CAPACITY;
  size_t need = 0;
  OT_TRY(tokenize_routed_any(m, nullptr, R, k, nullptr, 0, nullptr, &need));
  if (ws_bytes < need) return ONETRANS_ERR_CAPACITY;
  RoutedCall c;
  std::memset(&c, 0, sizeof(c));
  c.events = events; c.weights = weights; c.R = R; c.k = k; c.plan = &p;
  c.tokens = tokens;
  c.rows = token_rows(R, rows_per_sample, sample_ld);
  return tokenize_routed_any(m, &c, R, k, ws, ws_bytes, (cudaStream_t)stream, nullptr);
}

onetrans_status onetrans_tokenize_routed_backward(const onetrans_model* m, const void* events, const float* weights,
                                                  int64_t R, int32_t k, const void* plan, size_t plan_bytes,
                                                  const void* dtokens, int32_t dtokens_mode, int64_t rows_per_sample,
                                                  int64_t sample_ld, void* devents, float* dweights,
                                                  const onetrans_event_grads* grads, void* ws, size_t ws_bytes,
                                                  void* stream) {
  OT_TRY(routed_check(m, R, k));
  if (!mode_ok(dtokens_mode)) return ONETRANS_ERR_INVALID_ARG;
  if (!m->bf16 && dtokens_mode == ONETRANS_BF16) return ONETRANS_ERR_UNSUPPORTED;
  OT_TRY(token_rows_check(m, R, rows_per_sample, sample_ld));
  if (!grads || !grads->Wb1 || !grads->bb1 || !grads->Wb2 || !grads->bb2 || !grads->type_emb ||
      !aligned(grads->type_emb, 16))
    return ONETRANS_ERR_INVALID_ARG;
  RoutedCall c;
  std::memset(&c, 0, sizeof(c));
  const int T = m->cfg.n_behaviors, d = m->d, e = m->cfg.event_dim;
  for (int t = 0; t < T; ++t) {
    c.grads.W1[t] = grads->Wb1[t]; c.grads.b1[t] = grads->bb1[t];
    c.grads.W2[t] = grads->Wb2[t]; c.grads.b2[t] = grads->bb2[t];
    for (const void* p : {(void*)c.grads.W1[t], (void*)c.grads.b1[t], (void*)c.grads.W2[t], (void*)c.grads.b2[t]})
      if (!p || !aligned(p, 16)) return ONETRANS_ERR_INVALID_ARG;
  }
  c.grads.emb = grads->type_emb;
  cudaStream_t st = (cudaStream_t)stream;
  if (R == 0) {   // no events: every gradient is zero
    for (int t = 0; t < T; ++t) {
      OT_TRY(cuda_ok(cudaMemsetAsync(c.grads.W1[t], 0, (size_t)d * e * 4, st)));
      OT_TRY(cuda_ok(cudaMemsetAsync(c.grads.b1[t], 0, (size_t)d * 4, st)));
      OT_TRY(cuda_ok(cudaMemsetAsync(c.grads.W2[t], 0, (size_t)d * d * 4, st)));
      OT_TRY(cuda_ok(cudaMemsetAsync(c.grads.b2[t], 0, (size_t)d * 4, st)));
    }
    return cuda_ok(cudaMemsetAsync(c.grads.emb, 0, (size_t)T * d * 4, st));
  }
  if (!events || !plan || !dtokens || !ws || !aligned(events, 16) || !aligned(weights, 16) || !aligned(plan, 256) ||
      !aligned(dtokens, 16) || !aligned(devents, 16) || !aligned(dweights, 16) || !aligned(ws, 256))
    return ONETRANS_ERR_INVALID_ARG;
  const PlanBuf p = plan_buf(m, const_cast<void*>(plan), R, k);
  if (p.bytes > plan_bytes) return ONETRANS_ERR_CAPACITY;
  size_t need = 0;
  OT_TRY(routed_backward_any(m, nullptr, R, k, nullptr, 0, nullptr, &need));
  if (ws_bytes < need) return ONETRANS_ERR_CAPACITY;
  c.events = events; c.weights = weights; c.R = R; c.k = k; c.plan = &p;
  c.dtokens = dtokens; c.dtokens_mode = dtokens_mode;
  c.rows = token_rows(R, rows_per_sample, sample_ld);
  c.devents = devents; c.dweights = dweights;
  return routed_backward_any(m, &c, R, k, ws, ws_bytes, st, nullptr);
}

}  // extern "C"
