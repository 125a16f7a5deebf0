// tern_host_recurrent.h -- host side of the recurrent block's operators of
// include/tern.h (convolution, scan, gated norm, norm behind a block): checks
// of the arguments and launch plans. Part of tern_host.cpp, inside its extern
// "C" block, after tern_host_decoder.h.

namespace {

tern_status check_states(const tern_state_batch* b, int rows, int slots, tern::StateBatch* o) {
  if (!b) return fail(TERN_ERR_NULL, "batch is NULL");
  if (!b->begin || !b->src || !b->dst) return fail(TERN_ERR_NULL, "a pointer of the batch is NULL");
  if (b->seqs < 1 || b->seqs > 65535) return fail(TERN_ERR_SHAPE, "seqs=%d out of range [1, 65535]", b->seqs);
  if (rows < 1 || rows > kMaxTokens) return fail(TERN_ERR_SHAPE, "rows=%d out of range [1, %d]", rows, kMaxTokens);
  if (b->max_q < 1 || b->max_q > kMaxTokens)
    return fail(TERN_ERR_SHAPE, "max_q=%d out of range [1, %d]", b->max_q, kMaxTokens);
  if (slots < 1) return fail(TERN_ERR_SHAPE, "slots=%d must be positive", slots);
  if (!aligned(b->begin, 4) || !aligned(b->src, 4) || !aligned(b->dst, 4))
    return fail(TERN_ERR_ALIGN, "the batch arrays must be 4-byte aligned");
  *o = tern::StateBatch{b->begin, b->src, b->dst, b->seqs, b->max_q, rows};
  return TERN_OK;
}

}  // namespace

tern_status tern_causal_conv(const tern_state_batch* batch, int rows, const void* x, tern_dtype type,
                             int64_t x_stride, int channels, int width, const void* weight, const void* bias,
                             tern_dtype weight_type, int silu, void* state, int slots, void* y_bf16,
                             int64_t y_stride, void* stream) {
  call_begin();
  tern::ConvArgs a{};
  if (tern_status st = check_states(batch, rows, slots, &a.batch)) return st;
  if (!x || !weight || !state || !y_bf16) return fail(TERN_ERR_NULL, "tern_causal_conv: x, weight, state or y is NULL");
  if (!known_type(type) || !known_type(weight_type)) return fail(TERN_ERR_VALUE, "tern_causal_conv: unknown type");
  if (x == y_bf16) return fail(TERN_ERR_VALUE, "tern_causal_conv: y must not be x");
  if (channels < 8 || channels % 8 != 0 || channels > (1 << 20))
    return fail(TERN_ERR_SHAPE, "channels=%d must be a positive multiple of 8, at most 2^20", channels);
  if (width < 2 || width > 4) return fail(TERN_ERR_SHAPE, "width=%d must be 2, 3 or 4", width);
  if (x_stride < channels || y_stride < channels)
    return fail(TERN_ERR_SHAPE, "a row stride is smaller than channels=%d", channels);
  if (!aligned16(x) || !aligned16(weight) || !aligned16(bias) || !aligned16(state) || !aligned16(y_bf16) ||
      !rows_aligned(x_stride, type, 16) || !rows_aligned(y_stride, TERN_BF16, 16))
    return fail(TERN_ERR_ALIGN, "tern_causal_conv: pointers and rows must be 16-byte aligned");
  if (!tern::launch_conv) return no_unit();
  a.x = x, a.w = weight, a.bias = bias, a.state = state, a.y = (uint16_t*)y_bf16;
  a.x_stride = x_stride, a.y_stride = y_stride;
  a.type = type, a.w_type = weight_type, a.channels = channels, a.width = width, a.slots = slots, a.silu = silu != 0;
  // a thread's number within its sequence is an int in the kernel: 2^31 threads of 256 a workgroup
  if (tern::conv_blocks(a) > kMaxGrid || tern::conv_blocks(a) / batch->seqs > (INT64_C(1) << 31) / 256)
    return fail(TERN_ERR_SHAPE, "tern_causal_conv: seqs * max_q * channels too large for one launch");
  const int err = tern::launch_conv(a, stream);
  if (err) return hip_fail(err, "causal_conv launch");
  return call_ok();
}

namespace {

// Up to so many rows a sequence go token by token. Measured, token by token and in
// blocks: 16 sequences of 160 heads of 64 x 128 with 8 rows 46 and 56 us, with 12 rows 52 and 57,
// with 16 59 and 57; 64 sequences 137 and 180, 166 and 181, 196 and 183; 2 of 40 heads of 128 x 256 22
// and 25, 25 and 24, 30 and 24.
constexpr int kScanStepRows = 8;

tern_status check_scan(const tern_state_batch* batch, int rows, int heads, int dim, int groups, int state_dim,
                       int slots, tern::ScanArgs* a) {
  if (tern_status st = check_states(batch, rows, slots, &a->batch)) return st;
  if (dim != 32 && dim != 64 && dim != 128) return fail(TERN_ERR_SHAPE, "dim=%d must be 32, 64 or 128", dim);
  if (state_dim != 64 && state_dim != 128 && state_dim != 256)
    return fail(TERN_ERR_SHAPE, "state_dim=%d must be 64, 128 or 256", state_dim);
  if (heads < 1 || heads > 65535) return fail(TERN_ERR_SHAPE, "heads=%d out of range [1, 65535]", heads);
  if (groups < 1 || heads % groups != 0)
    return fail(TERN_ERR_SHAPE, "groups=%d must divide heads=%d", groups, heads);
  a->heads = heads, a->dim = dim, a->groups = groups, a->state_dim = state_dim, a->slots = slots;
  // Token by token, workgroups of 256 threads, one a head; in blocks, of 512, one for
  // every 64 columns of a group's heads (segments are cut only where those are few),
  // behind a launch of 256. A grid's threads are counted in 32 bits.
  const bool blocks = batch->max_q > kScanStepRows;
  if (blocks ? 2 * tern::scan_units(*a) > kMaxGrid || tern::scan_prepare_blocks(*a) > kMaxGrid
             : (int64_t)batch->seqs * heads > kMaxGrid)
    return fail(TERN_ERR_SHAPE, "tern_scan: seqs * heads or seqs * max_q * groups too large for one launch");
  return TERN_OK;
}

constexpr int64_t kScanMaxStride = 1 << 22;  // elements: 64 rows stay below 2^30 bytes

// Segments of a prompt: as many as make the launches shortest, in microseconds as measured.
// A block of 32 tokens takes a workgroup alone on its compute unit `last` in the last
// launch and `before` in the one before it, which only several segments need; k
// workgroups on a unit take about 0.85 k times as long (two 1.55 to 1.9, three 2.5); two
// launches more cost 16, and the segments' states cross the memory four times, 256
// bytes a row of state each. Measured with so many segments, those taken here in brackets:
//   64 blocks of 160 units of 64 x 128: [1] 95, 2 121, 3 103, 4 109 us;
//   256 blocks of 20 units of 64 x 128: 1 299, 4 131, 8 79, 11 67, [12] 63, 16 70, 24 61, 32 67;
//   of 64 x 64: 1 225, 8 62, 11 54, 12 51, 16 57, [24] 49; of 64 x 256: 1 440, 8 109, 11 94, [12] 88, 16 110, 24 97;
//   64 blocks of 40 units of 64 x 128: 1 84, 3 59, 4 50, [6] 44, 8 48, 16 51;
//   128 blocks of 80 units of 64 x 128: 1 165, 3 117, 4 122, [6] 104, 8 118, 16 126.
tern::ScanPlan plan_scan(const tern::ScanArgs& a) {
  const int64_t blocks = (a.batch.max_q + tern::kScanBlock - 1) / tern::kScanBlock, units = tern::scan_units(a);
  const double last = a.state_dim == 64 ? 0.85 : a.state_dim == 128 ? 1.13 : 1.68;
  const double before = a.state_dim == 64 ? 0.51 : a.state_dim == 128 ? 0.67 : 0.82;
  const auto shared = [](int64_t workgroups) {
    const int64_t k = (workgroups + kComputeUnits - 1) / kComputeUnits;
    return k <= 1 ? 1.0 : 0.85 * (double)k;
  };
  tern::ScanPlan p{1, (int)blocks * tern::kScanBlock};
  double least = 0;
  for (int64_t s = 1; s <= std::min<int64_t>(64, blocks / 4 + 1) && (s == 1 || units < kComputeUnits); ++s) {
    const int64_t length = (blocks + s - 1) / s, used = (blocks + length - 1) / length;
    double us = length * last * shared(units * used);
    if (used > 1) us += length * before * shared(units * (used - 1)) + 16 + 2e-4 * (double)(units * used * a.state_dim);
    if (s == 1 || us < least) {
      least = us;
      p.length = (int)length * tern::kScanBlock, p.segments = (int)used;
    }
  }
  return p;
}

size_t scan_ws(const tern::ScanArgs& a) {
  return a.batch.max_q <= kScanStepRows ? 0 : (size_t)tern::scan_ws_bytes(a, plan_scan(a));
}

}  // namespace

size_t tern_scan_workspace_bytes(const tern_state_batch* batch, int rows, int heads, int dim, int groups,
                                 int state_dim) {
  tern::ScanArgs a{};
  if (check_scan(batch, rows, heads, dim, groups, state_dim, 1, &a)) return (size_t)-1;
  g_last_error.clear();
  return scan_ws(a);
}

tern_status tern_scan(const tern_state_batch* batch, int rows, int heads, int dim, int groups, int state_dim,
                      const void* x_bf16, int64_t x_stride, const void* b_bf16, int64_t b_stride,
                      const void* c_bf16, int64_t c_stride, const void* dt, tern_dtype dt_type, int64_t dt_stride,
                      const float* dt_bias, int softplus, const float* a_decay, const float* d, float* state, int slots,
                      void* y_bf16, void* ws, size_t ws_bytes, void* stream) {
  call_begin();
  tern::ScanArgs a{};
  if (tern_status st = check_scan(batch, rows, heads, dim, groups, state_dim, slots, &a)) return st;
  if (!x_bf16 || !b_bf16 || !c_bf16 || !dt || !a_decay || !state || !y_bf16)
    return fail(TERN_ERR_NULL, "tern_scan: x, b, c, dt, a, state or y is NULL");
  if (!known_type(dt_type)) return fail(TERN_ERR_VALUE, "tern_scan: unknown type of dt");
  if (y_bf16 == x_bf16) return fail(TERN_ERR_VALUE, "tern_scan: y must not be x");
  const int64_t shared = (int64_t)groups * state_dim;
  if (x_stride < (int64_t)heads * dim || b_stride < shared || c_stride < shared || dt_stride < heads)
    return fail(TERN_ERR_SHAPE, "tern_scan: a row stride is smaller than the row");
  if (x_stride > kScanMaxStride || b_stride > kScanMaxStride || c_stride > kScanMaxStride)
    return fail(TERN_ERR_SHAPE, "tern_scan: a row stride of x, b or c is larger than 2^22");
  if (!aligned16(x_bf16) || !aligned16(b_bf16) || !aligned16(c_bf16) || !aligned16(state) || !aligned16(y_bf16) ||
      x_stride % 8 != 0 || b_stride % 8 != 0 || c_stride % 8 != 0)
    return fail(TERN_ERR_ALIGN, "tern_scan: x, b, c, their rows, state and y must be 16-byte aligned");
  if (!aligned(dt, type_bytes(dt_type)) || !aligned(dt_bias, 4) || !aligned(a_decay, 4) || !aligned(d, 4))
    return fail(TERN_ERR_ALIGN, "tern_scan: dt, dt_bias, a and d must be aligned to their elements");
  const size_t need = scan_ws(a);
  if (need && (!ws || ws_bytes < need))
    return fail(TERN_ERR_WORKSPACE, "tern_scan needs %zu bytes of workspace, got %zu", need, ws ? ws_bytes : (size_t)0);
  if (need && !aligned16(ws)) return fail(TERN_ERR_ALIGN, "the workspace must be 16-byte aligned");
  if (!tern::launch_scan_step || !tern::launch_scan_blocks) return no_unit();
  a.x = (const uint16_t*)x_bf16, a.b = (const uint16_t*)b_bf16, a.c = (const uint16_t*)c_bf16, a.dt = dt;
  a.dt_bias = dt_bias, a.a = a_decay, a.d = d, a.state = state, a.y = (uint16_t*)y_bf16;
  a.x_stride = x_stride, a.b_stride = b_stride, a.c_stride = c_stride, a.dt_stride = dt_stride;
  a.dt_type = dt_type, a.softplus = softplus != 0;
  const int err = a.batch.max_q <= kScanStepRows ? tern::launch_scan_step(a, stream)
                                                 : tern::launch_scan_blocks(a, plan_scan(a), ws, stream);
  if (err) return hip_fail(err, "scan launch");
  return call_ok();
}

namespace {

// The outputs that the norms share.
tern_status check_norm_out(const char* call, int T, int k, int mult, int8_t* q, float* act_scale, tern_q_layout layout,
                           void* y, int64_t y_stride, float eps) {
  if (!q != !act_scale) return fail(TERN_ERR_NULL, "%s: q and act_scale go together", call);
  if (layout != TERN_Q_ROW_MAJOR && layout != TERN_Q_OPERAND_ORDER)
    return fail(TERN_ERR_VALUE, "unknown q layout %d", (int)layout);
  if (!(eps >= 0.f) || std::isinf(eps)) return fail(TERN_ERR_VALUE, "eps=%g must be finite and not negative", (double)eps);
  if (T < 1 || T > kMaxTokens) return fail(TERN_ERR_SHAPE, "T=%d out of range [1, %d]", T, kMaxTokens);
  if (k < mult || k % mult != 0 || k > tern::kNormMaxK)
    return fail(TERN_ERR_SHAPE, "K=%d must be a positive multiple of %d, at most %d", k, mult, tern::kNormMaxK);
  if (y && y_stride < k) return fail(TERN_ERR_SHAPE, "a row stride is smaller than K=%d", k);
  if (!aligned16(q) || !aligned16(y) || !aligned(act_scale, 4) || (y && !rows_aligned(y_stride, TERN_BF16, 16)))
    return fail(TERN_ERR_ALIGN, "%s: pointers and rows must be 16-byte aligned", call);
  return TERN_OK;
}

}  // namespace

tern_status tern_rmsnorm_gated(const void* x, tern_dtype x_type, int64_t x_stride, const void* z,
                               tern_dtype z_type, int64_t z_stride, const void* weight, tern_dtype weight_type,
                               int group, int gate_first, float eps, int T, int k, int8_t* q, float* act_scale,
                               tern_q_layout layout, void* y_bf16, int64_t y_stride, void* stream) {
  call_begin();
  if (!x || !z || !weight) return fail(TERN_ERR_NULL, "tern_rmsnorm_gated: x, z or weight is NULL");
  if (!q && !y_bf16) return fail(TERN_ERR_NULL, "tern_rmsnorm_gated: neither q nor y asked for");
  if (!known_type(x_type) || !known_type(z_type) || !known_type(weight_type))
    return fail(TERN_ERR_VALUE, "tern_rmsnorm_gated: unknown type");
  const int mult = layout == TERN_Q_OPERAND_ORDER ? 64 : 16;
  if (tern_status st = check_norm_out("tern_rmsnorm_gated", T, k, mult, q, act_scale, layout, y_bf16, y_stride, eps))
    return st;
  if (group < mult || group % mult != 0 || k % group != 0)
    return fail(TERN_ERR_SHAPE, "group=%d must divide K=%d and be a multiple of %d", group, k, mult);
  if (x_stride < k || z_stride < k) return fail(TERN_ERR_SHAPE, "a row stride is smaller than K=%d", k);
  if (!aligned16(x) || !aligned16(z) || !aligned16(weight) || !rows_aligned(x_stride, x_type, 16) ||
      !rows_aligned(z_stride, z_type, 16))
    return fail(TERN_ERR_ALIGN, "tern_rmsnorm_gated: pointers and rows must be 16-byte aligned");
  if (!tern::launch_rmsnorm_gated) return no_unit();
  tern::GatedNormArgs a{};
  a.x = x, a.z = z, a.w = weight, a.q = q, a.act_scale = act_scale, a.y = (uint16_t*)y_bf16;
  a.x_stride = x_stride, a.z_stride = z_stride, a.y_stride = y_stride;
  a.x_type = x_type, a.z_type = z_type, a.w_type = weight_type, a.T = T, a.K = k, a.group = group, a.eps = eps;
  a.gate_first = gate_first != 0, a.operand_order = layout == TERN_Q_OPERAND_ORDER;
  const int err = tern::launch_rmsnorm_gated(a, stream);
  if (err) return hip_fail(err, "rmsnorm_gated launch");
  return call_ok();
}

tern_status tern_rmsnorm_post(const void* x, tern_dtype x_type, int64_t x_stride, const void* post_weight,
                              const void* gate, tern_dtype gate_type, int64_t gate_stride, float scale,
                              const void* residual, int64_t residual_stride, void* residual_out,
                              int64_t residual_out_stride, tern_dtype residual_type, const void* weight,
                              tern_dtype weight_type, float eps, int T, int k, int8_t* q, float* act_scale,
                              tern_q_layout layout, void* y_bf16, int64_t y_stride, void* stream) {
  call_begin();
  if (!x || !post_weight || !residual || !residual_out)
    return fail(TERN_ERR_NULL, "tern_rmsnorm_post: x, post_weight, residual or residual_out is NULL");
  if (weight ? !q && !y_bf16 : q || act_scale || y_bf16)
    return fail(TERN_ERR_NULL, "tern_rmsnorm_post: a weight and q or y go together");
  if (!known_type(x_type) || !known_type(weight_type) || !known_type(residual_type) || (gate && !known_type(gate_type)))
    return fail(TERN_ERR_VALUE, "tern_rmsnorm_post: unknown type");
  if (!std::isfinite(scale)) return fail(TERN_ERR_VALUE, "scale=%g must be finite", (double)scale);
  const int mult = layout == TERN_Q_OPERAND_ORDER ? 64 : 16;
  if (tern_status st = check_norm_out("tern_rmsnorm_post", T, k, mult, q, act_scale, layout, y_bf16, y_stride, eps))
    return st;
  if (x_stride < k || residual_stride < k || residual_out_stride < k || (gate && gate_stride != 0 && gate_stride < k))
    return fail(TERN_ERR_SHAPE, "a row stride is smaller than K=%d", k);
  if (!aligned16(x) || !aligned16(post_weight) || !aligned16(gate) || !aligned16(residual) || !aligned16(residual_out) ||
      !aligned16(weight) || !rows_aligned(x_stride, x_type, 16) || !rows_aligned(residual_stride, residual_type, 16) ||
      !rows_aligned(residual_out_stride, residual_type, 16) || (gate && !rows_aligned(gate_stride, gate_type, 16)))
    return fail(TERN_ERR_ALIGN, "tern_rmsnorm_post: pointers and rows must be 16-byte aligned");
  if (!tern::launch_rmsnorm_post) return no_unit();
  tern::PostNormArgs a{};
  a.x = x, a.post_w = post_weight, a.gate = gate, a.r = residual, a.w = weight, a.r_out = residual_out;
  a.q = q, a.act_scale = act_scale, a.y = (uint16_t*)y_bf16;
  a.x_stride = x_stride, a.gate_stride = gate ? gate_stride : 0, a.r_stride = residual_stride;
  a.r_out_stride = residual_out_stride, a.y_stride = y_stride;
  a.x_type = x_type, a.gate_type = gate_type, a.r_type = residual_type, a.w_type = weight_type;
  a.T = T, a.K = k, a.scale = scale, a.eps = eps, a.operand_order = layout == TERN_Q_OPERAND_ORDER;
  const int err = tern::launch_rmsnorm_post(a, stream);
  if (err) return hip_fail(err, "rmsnorm_post launch");
  return call_ok();
}
