// tern_host_decoder.h -- host side of the decoder operators of include/tern.h
// (norm, cache, attention): checks of the arguments and launch plans. Part of
// tern_host.cpp, inside its extern "C" block.

namespace {

tern_status no_unit() { return fail(TERN_ERR_HIP, "this build of the library has no kernels for the decoder operators"); }

int type_bytes(int type) { return type == TERN_F32 ? 4 : 2; }
bool known_type(int type) { return type == TERN_F32 || type == TERN_BF16; }
bool rows_aligned(int64_t stride, int type, int bytes) { return stride * type_bytes(type) % bytes == 0; }
bool aligned(const void* p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

// Cache and batch of a call over `rows` rows, as the kernels take them.
tern_status check_kv(const tern_kv_cache* c, const tern_kv_batch* b, int rows, tern::KvCache* co, tern::KvBatch* bo) {
  if (!c || !b) return fail(TERN_ERR_NULL, "cache or batch is NULL");
  if (!c->k || !c->v || !c->k_scale || !c->v_scale) return fail(TERN_ERR_NULL, "a pointer of the cache is NULL");
  if (!b->q_begin || !b->kv_len || !b->page_table) return fail(TERN_ERR_NULL, "a pointer of the batch is NULL");
  if (c->dim != 64 && c->dim != 128 && c->dim != 256)
    return fail(TERN_ERR_SHAPE, "dim=%d must be 64, 128 or 256", c->dim);
  if (c->heads < 1 || c->heads > 1024) return fail(TERN_ERR_SHAPE, "heads=%d out of range [1, 1024]", c->heads);
  if (c->pages < 1) return fail(TERN_ERR_SHAPE, "pages=%d must be positive", c->pages);
  if (b->seqs < 1 || b->seqs > 65535) return fail(TERN_ERR_SHAPE, "seqs=%d out of range [1, 65535]", b->seqs);
  if (rows < 1 || rows > kMaxTokens) return fail(TERN_ERR_SHAPE, "rows=%d out of range [1, %d]", rows, kMaxTokens);
  if (b->max_q < 1 || b->max_q > kMaxTokens)
    return fail(TERN_ERR_SHAPE, "max_q=%d out of range [1, %d]", b->max_q, kMaxTokens);
  if (b->table_width < 1 || b->table_width > (1 << 24))
    return fail(TERN_ERR_SHAPE, "table_width=%d out of range [1, 2^24]", b->table_width);
  if (b->max_kv < 1 || b->max_kv > (int64_t)b->table_width * TERN_KV_PAGE)
    return fail(TERN_ERR_SHAPE, "max_kv=%d must be in [1, 64 table_width=%lld]", b->max_kv,
                (long long)b->table_width * TERN_KV_PAGE);
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) ||
      !aligned(b->q_begin, 4) || !aligned(b->kv_len, 4) || !aligned(b->page_table, 4))
    return fail(TERN_ERR_ALIGN, "k and v must be 16-byte aligned, scales and batch arrays 4-byte");
  *co = tern::KvCache{c->k, c->v, c->k_scale, c->v_scale, c->pages, c->heads, c->dim};
  *bo = tern::KvBatch{b->q_begin, b->kv_len, b->page_table, b->seqs, b->max_q, b->max_kv, b->table_width};
  return TERN_OK;
}

// Workgroups of a launch, all of 256 threads: the runtime counts a grid's
// threads in 32 bits, and of a grid past that it launches the remainder only.
constexpr int64_t kMaxGrid = 0xffffffffu / 256;

}  // namespace

tern_status tern_rmsnorm(const void* x, tern_dtype x_type, int64_t x_stride, const void* residual,
                         int64_t residual_stride, void* residual_out, int64_t residual_out_stride,
                         tern_dtype residual_type, const void* weight, tern_dtype weight_type, float eps,
                         int T, int k, int8_t* q, float* act_scale, tern_q_layout layout, void* y_bf16,
                         int64_t y_stride, void* stream) {
  call_begin();
  if (!x || !weight) return fail(TERN_ERR_NULL, "tern_rmsnorm: x or weight is NULL");
  if (!q && !y_bf16) return fail(TERN_ERR_NULL, "tern_rmsnorm: neither q nor y asked for");
  if (!q != !act_scale) return fail(TERN_ERR_NULL, "tern_rmsnorm: q and act_scale go together");
  if (!residual != !residual_out) return fail(TERN_ERR_NULL, "tern_rmsnorm: residual and residual_out go together");
  if (!known_type(x_type) || !known_type(weight_type) || (residual && !known_type(residual_type)))
    return fail(TERN_ERR_VALUE, "tern_rmsnorm: unknown type");
  if (layout != TERN_Q_ROW_MAJOR && layout != TERN_Q_OPERAND_ORDER)
    return fail(TERN_ERR_VALUE, "unknown q layout %d", (int)layout);
  if (!(eps >= 0.f) || std::isinf(eps)) return fail(TERN_ERR_VALUE, "eps=%g must be finite and not negative", (double)eps);
  if (T < 1 || T > kMaxTokens) return fail(TERN_ERR_SHAPE, "T=%d out of range [1, %d]", T, kMaxTokens);
  const int mult = layout == TERN_Q_OPERAND_ORDER ? 64 : 16;
  if (k < mult || k % mult != 0 || k > tern::kNormMaxK)
    return fail(TERN_ERR_SHAPE, "K=%d must be a positive multiple of %d, at most %d", k, mult, tern::kNormMaxK);
  if (x_stride < k || (residual && (residual_stride < k || residual_out_stride < k)) || (y_bf16 && y_stride < k))
    return fail(TERN_ERR_SHAPE, "a row stride is smaller than K=%d", k);
  if (!aligned16(x) || !aligned16(weight) || !aligned16(q) || !aligned16(y_bf16) || !aligned16(residual) ||
      !aligned16(residual_out) || !aligned(act_scale, 4) || !rows_aligned(x_stride, x_type, 16) ||
      (residual && (!rows_aligned(residual_stride, residual_type, 16) ||
                    !rows_aligned(residual_out_stride, residual_type, 16))) ||
      (y_bf16 && !rows_aligned(y_stride, TERN_BF16, 16)))
    return fail(TERN_ERR_ALIGN, "tern_rmsnorm: pointers and rows must be 16-byte aligned");
  if (!tern::launch_rmsnorm) return no_unit();
  tern::NormArgs a{};
  a.x = x, a.r = residual, a.r_out = residual_out, a.w = weight;
  a.q = q, a.act_scale = act_scale, a.y = (uint16_t*)y_bf16;
  a.x_stride = x_stride, a.r_stride = residual_stride, a.r_out_stride = residual_out_stride, a.y_stride = y_stride;
  a.x_type = x_type, a.r_type = residual ? (int)residual_type : -1, a.w_type = weight_type;
  a.T = T, a.K = k, a.eps = eps, a.operand_order = layout == TERN_Q_OPERAND_ORDER;
  const int err = tern::launch_rmsnorm(a, stream);
  if (err) return hip_fail(err, "rmsnorm launch");
  return call_ok();
}

tern_status tern_kv_append(const tern_kv_cache* cache, const tern_kv_batch* batch, int tokens,
                           const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                           const void* q, int64_t q_stride, int q_heads, void* q_out_bf16,
                           tern_dtype type, const tern_rope* rope, const int32_t* positions, void* stream) {
  call_begin();
  tern::KvAppendArgs a{};
  if (tern_status st = check_kv(cache, batch, tokens, &a.cache, &a.batch)) return st;
  if (!k || !v) return fail(TERN_ERR_NULL, "tern_kv_append: k or v is NULL");
  if (!q != !q_out_bf16) return fail(TERN_ERR_NULL, "tern_kv_append: q and q_out go together");
  if (!known_type(type)) return fail(TERN_ERR_VALUE, "tern_kv_append: unknown type %d", (int)type);
  if (q && (q_heads < 1 || q_heads > 65536)) return fail(TERN_ERR_SHAPE, "q_heads=%d out of range [1, 65536]", q_heads);
  const int64_t kv_row = (int64_t)cache->heads * cache->dim;
  if (k_stride < kv_row || v_stride < kv_row || (q && q_stride < (int64_t)q_heads * cache->dim))
    return fail(TERN_ERR_SHAPE, "tern_kv_append: a row stride is smaller than the row");
  const int bytes = 4 * type_bytes(type);
  if (!aligned(k, bytes) || !aligned(v, bytes) || !aligned(q, bytes) || !aligned16(q_out_bf16) ||
      !rows_aligned(k_stride, type, bytes) || !rows_aligned(v_stride, type, bytes) ||
      (q && !rows_aligned(q_stride, type, bytes)))
    return fail(TERN_ERR_ALIGN, "tern_kv_append: inputs and their rows must be %d-byte aligned, q_out 16-byte", bytes);
  if (rope) {
    if (!rope->table || !rope->axis || !positions)
      return fail(TERN_ERR_NULL, "tern_kv_append: rope without table, axis map or positions");
    if (rope->pairs < 4 || rope->pairs % 4 != 0 || rope->pairs > cache->dim / 2)
      return fail(TERN_ERR_SHAPE, "rope pairs=%d must be a multiple of 4 in [4, dim/2=%d]", rope->pairs, cache->dim / 2);
    if (rope->max_pos < 1 || rope->axes < 1 || rope->axes > 255)
      return fail(TERN_ERR_SHAPE, "rope max_pos=%d, axes=%d out of range", rope->max_pos, rope->axes);
    if (!aligned(rope->table, 8) || !aligned(positions, 4))
      return fail(TERN_ERR_ALIGN, "rope table must be 8-byte aligned, positions 4-byte");
    a.rope = tern::RopeArgs{rope->table, rope->axis, positions, rope->pairs, rope->max_pos, rope->axes};
  }
  if (!tern::launch_kv_append) return no_unit();
  a.k = k, a.v = v, a.q = q, a.q_out = (uint16_t*)q_out_bf16;
  a.k_stride = k_stride, a.v_stride = v_stride, a.q_stride = q_stride;
  a.tokens = tokens, a.q_heads = q ? q_heads : 0, a.type = type;
  int64_t kv_blocks;
  if (tern::kv_append_blocks(a, &kv_blocks) > kMaxGrid)
    return fail(TERN_ERR_SHAPE, "tern_kv_append: seqs * max_q * heads too large for one launch");
  const int err = tern::launch_kv_append(a, stream);
  if (err) return hip_fail(err, "kv_append launch");
  return call_ok();
}

tern_status tern_kv_read(const tern_kv_cache* cache, const tern_kv_batch* batch, int rows, void* k_out_bf16,
                         void* v_out_bf16, void* stream) {
  call_begin();
  tern::KvReadArgs a{};
  if (tern_status st = check_kv(cache, batch, rows, &a.cache, &a.batch)) return st;
  if (!k_out_bf16 && !v_out_bf16) return fail(TERN_ERR_NULL, "tern_kv_read: neither k_out nor v_out asked for");
  if (!aligned16(k_out_bf16) || !aligned16(v_out_bf16))
    return fail(TERN_ERR_ALIGN, "tern_kv_read: outputs must be 16-byte aligned");
  if (!tern::launch_kv_read) return no_unit();
  a.k_out = (uint16_t*)k_out_bf16, a.v_out = (uint16_t*)v_out_bf16, a.rows = rows;
  if (tern::kv_read_blocks(a) > kMaxGrid)
    return fail(TERN_ERR_SHAPE, "tern_kv_read: seqs * max_q * heads too large for one launch");
  const int err = tern::launch_kv_read(a, stream);
  if (err) return hip_fail(err, "kv_read launch");
  return call_ok();
}

namespace {

tern_status check_attn(const tern_kv_cache* cache, const tern_kv_batch* batch, int tokens, int q_heads, int window,
                       int sinks, tern::KvAttnArgs* a) {
  if (tern_status st = check_kv(cache, batch, tokens, &a->cache, &a->batch)) return st;
  if (q_heads < cache->heads || q_heads % cache->heads != 0 || q_heads > 65535)
    return fail(TERN_ERR_SHAPE, "q_heads=%d must be a multiple of the cache's heads=%d, at most 65535", q_heads,
                cache->heads);
  if ((int64_t)(q_heads / cache->heads) * batch->max_q > (1 << 30))
    return fail(TERN_ERR_SHAPE, "max_q=%d times %d query heads a kv head is too large", batch->max_q,
                q_heads / cache->heads);
  if (window < 0 || sinks < 0) return fail(TERN_ERR_VALUE, "window=%d and sinks=%d must not be negative", window, sinks);
  a->tokens = tokens, a->q_heads = q_heads;
  a->window = window >= batch->max_kv ? 0 : window;  // one that no sequence reaches hides nothing
  a->sinks = a->window ? std::min(sinks, batch->max_kv) : 0;
  return TERN_OK;
}

// Pages a block of query rows may have to visit.
int64_t attn_pages(const tern::KvAttnArgs& a, int tokens_of_block) {
  const int64_t all = ((int64_t)a.batch.max_kv + TERN_KV_PAGE - 1) / TERN_KV_PAGE;
  if (!a.window) return all;
  const int64_t seen = ((int64_t)a.window + tokens_of_block + TERN_KV_PAGE - 2) / TERN_KV_PAGE + 1 +
                       ((int64_t)a.sinks + TERN_KV_PAGE - 1) / TERN_KV_PAGE;
  return std::min(all, seen);
}

constexpr int kComputeUnits = 256;  // of the part that this library is built for

tern::KvAttnPlan plan_attn(const tern::KvAttnArgs& a) {
  tern::KvAttnPlan p{};
  const int64_t group = a.q_heads / a.cache.heads, rows = group * a.batch.max_q;
  // Up to 32 rows a kv head the kernel for few rows reads every code once. With
  // 33 to 64 it reads them twice, which only pays while few (sequence, head)
  // pairs share the machine (35 rows: 32 us against 39 on one sequence of 32768
  // tokens and 8 heads, 24 against 27 on 4 of 1500, but 50 against 44 on 16 of
  // 4096); from 65 on the kernel for many rows wins (65 rows: 47 against 42, 66
  // against 48).
  const bool few = rows <= 32 || (rows <= 64 && (int64_t)a.batch.seqs * a.cache.heads <= 64);
  p.rows = rows <= 16 ? 16 : few ? 32 : 128;
  p.row_blocks = (int)((rows + p.rows - 1) / p.rows);
  const int64_t pages = attn_pages(a, std::min<int64_t>(a.batch.max_q, (p.rows + group - 2) / group + 1));
  const int64_t units = (int64_t)p.row_blocks * a.batch.seqs;
  // Equal runs, one workgroup each, or a workgroup a unit. With fewer than two
  // units a compute unit the longest of them decides, and runs share their
  // pages evenly, for the price of partial results and of the join. `saved` is
  // the pages by which that shortens the wait, at most: `lone` units follow each
  // other on a compute unit without runs, `shared` with them.
  p.least = 8;
  const double each = (double)(units * a.cache.heads) / kComputeUnits;  // units a compute unit
  int held = kComputeUnits;
  bool pays;
  if (p.rows <= 32) {
    // Bound by memory, where one workgroup a compute unit fills its share (256 /
    // 320 / 512 / 768 runs: 64 / 83 / 68 / 72 us for 32 sequences of 1024 to 8192
    // tokens). A page costs about (d + 64) / 192 of one at 128; lengths are
    // taken as three quarters of the bound. Measured, without and with runs: 8
    // units of 16, 32 and 63 pages 11.0 and 12.5, 15.5 and 12.5, 25.7 and 14.3 us;
    // 128 units of 16, 32 and 63 pages 11.8 and 20.6, 19.1 and 19.3, 33.1 and
    // 26.2 us; 64 units of two row tiles and 32 pages, which it cuts, 22.4 and 24.4 us;
    // 256 units of 128 pages 71 and 60 us; of 63 pages 64 wide 18.9 and
    // 26.1 us; 512 of 65 pages 46 and 54 us.
    const double saved = pages * (1 - 0.75 * each) * (a.cache.dim + 64) / 192;
    pays = saved > 25;
  } else {
    // Bound by instruction issue, where two workgroups share a compute unit at up
    // to 128 (219 us with 512 runs, 290 with 256, 237 with 768 for 320 units of 128
    // pages) and one fits at 256. Two that share take 1.25 to 1.5 times as long as
    // one. Measured, without and with runs: 64 units of 62 pages 109 and 47 us, 160
    // of 8, 31 and 62 pages 21 and 21, 62 and 52, 112 and 76 us; 320 of 16, 32, 64 and
    // 128 pages 39 and 60, 67 and 72, 139 and 119, 282 and 219 us; 640 of 32 pages 71
    // and 113 us; at 256: 128 units of 16 and 64 pages 54 and 79, 169 and 110 us, 384
    // of 31 pages 105 and 163 us, 288 of 20 window pages 135 and 106 us.
    const bool wide = a.cache.dim == 256;
    const double mean = a.window ? pages : std::max(0.0, pages - a.batch.max_q / (2.0 * TERN_KV_PAGE));
    const double lone = wide ? std::ceil(each) : each <= 1 ? 1 : 1.25;
    const double saved = mean * (lone - each * (wide ? 1 : 0.75));
    if (!wide) held = 2 * kComputeUnits;
    pays = each < 2 && saved > 12;
  }
  if (pays && pages > p.least && units <= tern::kKvMaxUnits && units * pages <= (1 << 30))
    p.runs = (int)std::max<int64_t>(
        1, std::min<int64_t>({held / a.cache.heads, units * pages / p.least, tern::kKvMaxRuns}));
  return p;
}

// fp32 words: run length and prefix sums, then two slots a run of partial sums, maximum and sum of each row.
size_t attn_ws(const tern::KvAttnArgs& a, const tern::KvAttnPlan& p) {
  if (!p.runs) return 0;
  const size_t head = ((size_t)a.batch.seqs * p.row_blocks + 2 + 63) / 64 * 64;
  return (head + (size_t)a.cache.heads * p.runs * 2 * p.rows * (a.cache.dim + 2)) * sizeof(float);
}

}  // namespace

size_t tern_kv_attn_workspace_bytes(const tern_kv_cache* cache, const tern_kv_batch* batch, int tokens, int q_heads,
                                    int window, int sinks) {
  tern::KvAttnArgs a{};
  if (check_attn(cache, batch, tokens, q_heads, window, sinks, &a)) return (size_t)-1;
  g_last_error.clear();
  return attn_ws(a, plan_attn(a));
}

tern_status tern_kv_attn(const tern_kv_cache* cache, const tern_kv_batch* batch, int tokens, const void* q_bf16,
                         int64_t q_stride, int q_heads, float scale, int window, int sinks, void* out_bf16, void* ws,
                         size_t ws_bytes, void* stream) {
  call_begin();
  tern::KvAttnArgs a{};
  if (tern_status st = check_attn(cache, batch, tokens, q_heads, window, sinks, &a)) return st;
  if (!q_bf16 || !out_bf16) return fail(TERN_ERR_NULL, "tern_kv_attn: q or out is NULL");
  if (!(scale > 0.f) || std::isinf(scale))
    return fail(TERN_ERR_VALUE, "scale=%g must be finite and positive", (double)scale);
  if (q_stride < (int64_t)q_heads * cache->dim) return fail(TERN_ERR_SHAPE, "q_stride is smaller than a row");
  if (!aligned16(q_bf16) || !aligned16(out_bf16) || q_stride % 8 != 0)
    return fail(TERN_ERR_ALIGN, "tern_kv_attn: q, its rows and out must be 16-byte aligned");
  const tern::KvAttnPlan p = plan_attn(a);
  const size_t need = attn_ws(a, p);
  if (need && (!ws || ws_bytes < need))
    return fail(TERN_ERR_WORKSPACE, "tern_kv_attn needs %zu bytes of workspace, got %zu", need, ws ? ws_bytes : (size_t)0);
  if (need && !aligned16(ws)) return fail(TERN_ERR_ALIGN, "the workspace must be 16-byte aligned");
  if ((int64_t)p.row_blocks * a.cache.heads * a.batch.seqs > kMaxGrid)
    return fail(TERN_ERR_SHAPE, "tern_kv_attn: too many rows or pages for one launch");
  if (!tern::launch_kv_attn) return no_unit();
  a.q = (const uint16_t*)q_bf16, a.out = (uint16_t*)out_bf16, a.q_stride = q_stride, a.scale = scale;
  const int err = tern::launch_kv_attn(a, p, ws, stream);
  if (err) return hip_fail(err, "kv_attn launch");
  return call_ok();
}
