// C ABI: AdamW over a list of tensors, and microscaled 4-bit matrices.
#include <algorithm>
#include <new>

#include "adamw.h"
#include "ctx.h"
#include "mx.h"

struct psgd_adamw_plan {
  psgd_ctx* ctx = nullptr;
  char* memory = nullptr;               // chunk table, then the norm's partial sums
  psgd::AdamwChunk* chunks = nullptr;
  double* partial = nullptr;
  int64_t n_chunks = 0;
  int pt = 0, gt = 0;
  bool low = false;
  ~psgd_adamw_plan() { (void)hipFree(memory); }
};

namespace {

constexpr int64_t kMaxBlocks = int64_t(1) << 24;      // of 256 threads: a launch holds fewer than 2^32
constexpr int64_t kMaxMxDim = int64_t(1) << 25;       // rows of a panel are addressed by 32-bit byte offsets

psgd_status check_rounding(psgd_ctx* ctx, psgd_rounding r) {
  if (r != PSGD_NEAREST && r != PSGD_STOCHASTIC) return fail(ctx, PSGD_EINVAL, "unknown rounding %d", (int)r);
  return PSGD_OK;
}
psgd_status check_adamw(psgd_ctx* ctx, const psgd_adamw_plan* plan) {
  ctx->err.clear();
  if (!plan || plan->ctx != ctx) return fail(ctx, PSGD_EINVAL, "plan does not belong to this context");
  return PSGD_OK;
}
bool mx_size_ok(int64_t rows, int64_t k) { return rows >= 0 && k >= 0 && rows <= kMaxMxDim && k <= kMaxMxDim; }

// t: an operand of rows x k (-1: any) called `name`
psgd_status check_mx(psgd_ctx* ctx, const psgd_mx_tensor* t, int64_t rows, int64_t k, const char* name) {
  if (!t) return fail(ctx, PSGD_EINVAL, "%s is required", name);
  if (!mx_size_ok(t->rows, t->k))
    return fail(ctx, PSGD_EINVAL, "%s: bad shape %lld x %lld", name, (long long)t->rows, (long long)t->k);
  if ((rows >= 0 && t->rows != rows) || (k >= 0 && t->k != k))
    return fail(ctx, PSGD_EINVAL, "%s is %lld x %lld, expected %lld x %lld", name, (long long)t->rows, (long long)t->k,
                (long long)(rows < 0 ? t->rows : rows), (long long)(k < 0 ? t->k : k));
  if (t->rows > 0 && t->k > 0 && (!t->data || !aligned16(t->data)))
    return fail(ctx, PSGD_EINVAL, "%s: data must be a 16-byte aligned pointer", name);
  return PSGD_OK;
}

// Whether a byte range that is written lies in another one of the list, or in a gradient.
struct Range { uintptr_t first, end; };
bool any_overlap(std::vector<Range>& written, const std::vector<Range>& read) {
  std::sort(written.begin(), written.end(), [](const Range& a, const Range& b) { return a.first < b.first; });
  for (size_t i = 1; i < written.size(); ++i)
    if (written[i].first < written[i - 1].end) return true;
  for (const Range& r : read) {
    const auto next = std::lower_bound(written.begin(), written.end(), r.end, [](const Range& w, uintptr_t e) { return w.first < e; });
    if (next != written.begin() && std::prev(next)->end > r.first) return true;
  }
  return false;
}

struct Bytes { const void* data; int64_t size; };
Bytes strided(const void* p, int64_t rows, int64_t cols, int64_t ld, int size) { return {p, ((rows - 1) * ld + cols) * size}; }
Bytes bytes_of(const psgd_mx_tensor* t) { return t ? Bytes{t->data, psgd::mx_bytes(t->rows, t->k)} : Bytes{nullptr, 0}; }
bool meet(Bytes a, Bytes b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.data), y = reinterpret_cast<uintptr_t>(b.data);
  return a.data && b.data && x < y + b.size && y < x + a.size;
}

}  // namespace

extern "C" {

psgd_status psgd_adamw_plan_create(psgd_ctx* ctx, const psgd_adamw_tensor* tensors, int n, psgd_dtype param_dtype,
                                   psgd_dtype grad_dtype, psgd_state state, psgd_adamw_plan** plan_out) try {
  if (!ctx) return PSGD_EINVAL;
  ctx->err.clear();
  if (!plan_out) return fail(ctx, PSGD_EINVAL, "plan pointer is NULL");
  *plan_out = nullptr;
  if (!tensors || n < 1) return fail(ctx, PSGD_EINVAL, "need at least one tensor");
  const int pt = grad_type(param_dtype), gt = grad_type(grad_dtype);
  if (!pt) return fail(ctx, PSGD_EDTYPE, "unknown parameter dtype %d", (int)param_dtype);
  if (!gt) return fail(ctx, PSGD_EDTYPE, "unknown gradient dtype %d", (int)grad_dtype);
  if (state != PSGD_STATE_F32 && state != PSGD_STATE_BYTE) return fail(ctx, PSGD_EINVAL, "unknown state %d", (int)state);
  const bool low = state == PSGD_STATE_BYTE;
  int64_t count = 0;
  for (int i = 0; i < n; ++i) {
    const psgd_adamw_tensor& t = tensors[i];
    if (t.numel < 0) return fail(ctx, PSGD_EINVAL, "tensor %d: negative size", i);
    if (t.numel == 0) continue;
    if (!t.param || !t.grad || !t.m1 || !t.m2 || (low && (!t.e1 || !t.e2)))
      return fail(ctx, PSGD_EINVAL, "tensor %d: NULL pointer", i);
    if (!aligned_to(t.param, type_size(pt)) || !aligned_to(t.grad, type_size(gt)))
      return fail(ctx, PSGD_EINVAL, "tensor %d: param and grad must be aligned to their element type", i);
    if (!aligned16(t.m1) || !aligned16(t.m2)) return fail(ctx, PSGD_EINVAL, "tensor %d: m1 and m2 must be 16-byte aligned", i);
    const int64_t chunks = t.numel / psgd::kAdamwChunk + (t.numel % psgd::kAdamwChunk != 0);
    if (chunks >= kMaxBlocks - count) return fail(ctx, PSGD_EUNSUPPORTED, "more than 2^36 elements in a list");
    count += chunks;
  }
  std::vector<psgd::AdamwChunk> table;
  table.reserve(count);
  const int ps = type_size(pt), gs = type_size(gt), ms = low ? 1 : 4;
  std::vector<Range> written, read;
  for (int i = 0; i < n; ++i) {
    const psgd_adamw_tensor& t = tensors[i];
    if (t.numel == 0) continue;
    const int64_t room = rup(t.numel, psgd::kAdamwGroup);
    auto add = [](std::vector<Range>& v, const void* p, int64_t bytes) {
      v.push_back({reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + bytes});
    };
    add(written, t.param, t.numel * ps);
    add(written, t.m1, room * ms);
    add(written, t.m2, room * ms);
    if (low) {
      add(written, t.e1, room / psgd::kAdamwGroup);
      add(written, t.e2, room / psgd::kAdamwGroup);
    }
    add(read, t.grad, t.numel * gs);
  }
  if (any_overlap(written, read)) return fail(ctx, PSGD_EINVAL, "buffers of the list overlap");
  for (int i = 0; i < n; ++i) {
    const psgd_adamw_tensor& t = tensors[i];
    for (int64_t o = 0; o < t.numel; o += psgd::kAdamwChunk)
      table.push_back({static_cast<char*>(t.param) + o * ps, static_cast<const char*>(t.grad) + o * gs,
                       static_cast<char*>(t.m1) + o * ms, static_cast<char*>(t.m2) + o * ms,
                       low ? t.e1 + o / psgd::kAdamwGroup : nullptr, low ? t.e2 + o / psgd::kAdamwGroup : nullptr, o,
                       (int32_t)std::min<int64_t>(psgd::kAdamwChunk, t.numel - o), i});
  }
  DeviceGuard dev(ctx->device);
  HIPCHK(ctx, dev.err, "hipSetDevice");
  std::unique_ptr<psgd_adamw_plan> p(new psgd_adamw_plan);
  p->ctx = ctx;
  p->pt = pt; p->gt = gt; p->low = low;
  p->n_chunks = count;
  const size_t list = count * sizeof(psgd::AdamwChunk), sums = psgd::kAdamwNormGrid * sizeof(double);
  void* mem = nullptr;
  if (psgd::device_alloc(&mem, list + sums) != hipSuccess) return fail(ctx, PSGD_ENOMEM, "list table of %zu bytes", list + sums);
  p->memory = static_cast<char*>(mem);
  p->chunks = reinterpret_cast<psgd::AdamwChunk*>(p->memory);
  p->partial = reinterpret_cast<double*>(p->memory + list);
  if (count > 0) HIPCHK(ctx, hipMemcpy(p->chunks, table.data(), list, hipMemcpyHostToDevice), "list table upload");
  *plan_out = p.release();
  return PSGD_OK;
} catch (const std::exception&) {
  return fail(ctx, PSGD_ENOMEM, "out of host memory");
}

psgd_status psgd_adamw_plan_destroy(psgd_adamw_plan* plan) {
  if (!plan) return PSGD_OK;
  DeviceGuard dev(plan->ctx->device);
  (void)hipDeviceSynchronize();
  delete plan;
  return PSGD_OK;
}

psgd_status psgd_adamw_prepare(psgd_ctx* ctx, psgd_adamw_plan* plan, float max_norm, const int32_t* skip_in, int32_t* skip_dev,
                               int32_t* step_dev, float* norm_dev, hipStream_t stream) {
  if (!ctx) return PSGD_EINVAL;
  if (psgd_status st = check_adamw(ctx, plan); st != PSGD_OK) return st;
  if (!skip_dev || !step_dev || !norm_dev) return fail(ctx, PSGD_EINVAL, "skip_dev, step_dev and norm_dev are required");
  if (std::isnan(max_norm)) return fail(ctx, PSGD_EINVAL, "max_norm is NaN");
  DeviceGuard dev(ctx->device);
  HIPCHK(ctx, dev.err, "hipSetDevice");
  const psgd::AdamwNorm a{plan->partial, max_norm, skip_in, skip_dev, step_dev, norm_dev};
  HIPCHK(ctx, psgd::launch_adamw_norm(plan->chunks, plan->n_chunks, plan->gt, a, stream), "gradient norm");
  return PSGD_OK;
}

psgd_status psgd_adamw_update(psgd_ctx* ctx, psgd_adamw_plan* plan, const int32_t* skip_dev, const int32_t* step_dev,
                              const float* norm_dev, const psgd_adam_hparams* hp, psgd_rounding rounding, uint64_t seed,
                              hipStream_t stream) {
  if (!ctx) return PSGD_EINVAL;
  if (psgd_status st = check_adamw(ctx, plan); st != PSGD_OK) return st;
  if (!skip_dev || !step_dev) return fail(ctx, PSGD_EINVAL, "skip_dev and step_dev are required");
  if (psgd_status st = check_hparams(ctx, hp); st != PSGD_OK) return st;
  if (psgd_status st = check_rounding(ctx, rounding); st != PSGD_OK) return st;
  DeviceGuard dev(ctx->device);
  HIPCHK(ctx, dev.err, "hipSetDevice");
  const psgd::AdamwArgs a{hp->lr, hp->beta1, hp->beta2, hp->eps, hp->weight_decay, std::log((double)hp->beta1),
                          std::log((double)hp->beta2), skip_dev, step_dev, norm_dev, seed};
  HIPCHK(ctx, psgd::launch_adamw(plan->chunks, plan->n_chunks, plan->pt, plan->gt, plan->low, rounding == PSGD_STOCHASTIC, a, stream),
         "AdamW update");
  return PSGD_OK;
}

psgd_status psgd_adamw_moments(psgd_ctx* ctx, const uint8_t* m1, const uint8_t* e1, const uint8_t* m2, const uint8_t* e2, int64_t n,
                               void* out1, void* out2, psgd_dtype out_dtype, hipStream_t stream) {
  if (!ctx) return PSGD_EINVAL;
  ctx->err.clear();
  if (out_dtype != PSGD_F32 && out_dtype != PSGD_BF16) return fail(ctx, PSGD_EDTYPE, "moments come as fp32 or bf16, not dtype %d", (int)out_dtype);
  const int ot = grad_type(out_dtype);
  if (n < 0) return fail(ctx, PSGD_EINVAL, "negative size");
  if (n > int64_t(1) << 35) return fail(ctx, PSGD_EUNSUPPORTED, "more than 2^35 values in a call");
  if (n == 0) return PSGD_OK;
  if (!m1 || !e1 || !m2 || !e2 || !out1 || !out2) return fail(ctx, PSGD_EINVAL, "NULL pointer");
  if (!aligned16(m1) || !aligned16(m2) || !aligned_to(out1, type_size(ot)) || !aligned_to(out2, type_size(ot)))
    return fail(ctx, PSGD_EINVAL, "m1 and m2 must be 16-byte aligned, the outputs aligned to their element type");
  const int64_t groups = rup(n, psgd::kAdamwGroup) / psgd::kAdamwGroup;
  const Bytes o1{out1, n * type_size(ot)}, o2{out2, n * type_size(ot)};
  for (const Bytes& in : {Bytes{m1, groups * psgd::kAdamwGroup}, Bytes{e1, groups}, Bytes{m2, groups * psgd::kAdamwGroup}, Bytes{e2, groups}})
    if (meet(o1, in) || meet(o2, in)) return fail(ctx, PSGD_EINVAL, "the outputs must not overlap the moments");
  if (meet(o1, o2)) return fail(ctx, PSGD_EINVAL, "the outputs must not overlap");
  DeviceGuard dev(ctx->device);
  HIPCHK(ctx, dev.err, "hipSetDevice");
  HIPCHK(ctx, psgd::launch_adamw_moments(m1, e1, m2, e2, n, out1, out2, ot, stream), "moments");
  return PSGD_OK;
}

psgd_status psgd_mx_bytes(int64_t rows, int64_t k, int64_t* bytes) {
  if (!bytes || !mx_size_ok(rows, k)) return PSGD_EINVAL;
  *bytes = psgd::mx_bytes(rows, k);
  return PSGD_OK;
}

psgd_status psgd_mx_quantize(psgd_ctx* ctx, const void* x, int64_t ld_x, int64_t m, int64_t n, psgd_dtype x_dtype,
                             const psgd_mx_tensor* row, const psgd_mx_tensor* col, psgd_rounding rounding, uint64_t seed,
                             const int32_t* step_dev, hipStream_t stream) {
  if (!ctx) return PSGD_EINVAL;
  ctx->err.clear();
  const int it = grad_type(x_dtype);
  if (!it) return fail(ctx, PSGD_EDTYPE, "unknown input dtype %d", (int)x_dtype);
  if (psgd_status st = check_rounding(ctx, rounding); st != PSGD_OK) return st;
  if (!mx_size_ok(m, n)) return fail(ctx, PSGD_EINVAL, "bad shape %lld x %lld", (long long)m, (long long)n);
  if (!row && !col) return fail(ctx, PSGD_EINVAL, "row or col is required");
  if (row)
    if (psgd_status st = check_mx(ctx, row, m, n, "row"); st != PSGD_OK) return st;
  if (col)
    if (psgd_status st = check_mx(ctx, col, n, m, "col"); st != PSGD_OK) return st;
  if (m > 1 && ld_x < n) return fail(ctx, PSGD_EINVAL, "the leading dimension must be >= n");
  if (m == 0 || n == 0) return PSGD_OK;
  if (!x || !aligned_to(x, type_size(it))) return fail(ctx, PSGD_EINVAL, "x must be a pointer aligned to its element type");
  if ((n + psgd::kMxPanel - 1) / psgd::kMxPanel * ((m + psgd::kMxGroup - 1) / psgd::kMxGroup) >= kMaxBlocks)
    return fail(ctx, PSGD_EUNSUPPORTED, "%lld x %lld is past what one launch takes", (long long)m, (long long)n);
  const Bytes in = strided(x, m, n, ld_x, type_size(it)), r = bytes_of(row), c = bytes_of(col);
  if (meet(in, r) || meet(in, c) || meet(r, c)) return fail(ctx, PSGD_EINVAL, "x, row and col must not overlap");
  DeviceGuard dev(ctx->device);
  HIPCHK(ctx, dev.err, "hipSetDevice");
  psgd::MxQuantize a{};
  a.x = x; a.ld = ld_x; a.m = m; a.n = n;
  if (row) a.row = psgd::mx_view(row->data, m, n);
  if (col) a.col = psgd::mx_view(col->data, n, m);
  a.seed = seed; a.step = step_dev;
  HIPCHK(ctx, psgd::launch_mx_quantize(a, it, rounding == PSGD_STOCHASTIC, stream), "4-bit quantisation");
  return PSGD_OK;
}

psgd_status psgd_mx_dequantize(psgd_ctx* ctx, const psgd_mx_tensor* t, void* out, int64_t ld_out, psgd_dtype out_dtype,
                               hipStream_t stream) {
  if (!ctx) return PSGD_EINVAL;
  ctx->err.clear();
  const int ot = grad_type(out_dtype);
  if (!ot) return fail(ctx, PSGD_EDTYPE, "unknown output dtype %d", (int)out_dtype);
  if (psgd_status st = check_mx(ctx, t, -1, -1, "the matrix"); st != PSGD_OK) return st;
  if (t->rows > 1 && ld_out < t->k) return fail(ctx, PSGD_EINVAL, "the leading dimension must be >= k");
  if (t->rows == 0 || t->k == 0) return PSGD_OK;
  if (!out || !aligned_to(out, type_size(ot))) return fail(ctx, PSGD_EINVAL, "out must be a pointer aligned to its element type");
  const psgd::MxView v = psgd::mx_view(t->data, t->rows, t->k);
  if (v.panels * v.groups >= kMaxBlocks)
    return fail(ctx, PSGD_EUNSUPPORTED, "%lld x %lld is past what one launch takes", (long long)t->rows, (long long)t->k);
  if (meet(strided(out, t->rows, t->k, ld_out, type_size(ot)), bytes_of(t)))
    return fail(ctx, PSGD_EINVAL, "out must not overlap the matrix");
  DeviceGuard dev(ctx->device);
  HIPCHK(ctx, dev.err, "hipSetDevice");
  HIPCHK(ctx, psgd::launch_mx_dequantize(v, out, ld_out, ot, stream), "4-bit values");
  return PSGD_OK;
}

psgd_status psgd_mx_product_workspace(int64_t m, int64_t n, int64_t k, int64_t* bytes) {
  if (!bytes || !mx_size_ok(m, k) || !mx_size_ok(n, k)) return PSGD_EINVAL;
  const psgd::MxPlan p = psgd::mx_plan(m, n, (k + psgd::kMxPanel - 1) / psgd::kMxPanel);
  *bytes = p.splits > 1 ? p.splits * m * n * 4 : 0;
  return PSGD_OK;
}

psgd_status psgd_mx_product(psgd_ctx* ctx, const psgd_mx_tensor* a, const psgd_mx_tensor* b, const float* scale, void* c, int64_t ld_c,
                            psgd_dtype c_dtype, int accumulate, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  if (!ctx) return PSGD_EINVAL;
  ctx->err.clear();
  const int ot = grad_type(c_dtype);
  if (!ot) return fail(ctx, PSGD_EDTYPE, "unknown output dtype %d", (int)c_dtype);
  if (accumulate && ot != psgd::G_F32) return fail(ctx, PSGD_EDTYPE, "products are added to fp32 only");
  if (psgd_status st = check_mx(ctx, a, -1, -1, "a"); st != PSGD_OK) return st;
  if (psgd_status st = check_mx(ctx, b, -1, a->k, "b"); st != PSGD_OK) return st;
  const int64_t m = a->rows, n = b->rows;
  if (m > 1 && ld_c < n) return fail(ctx, PSGD_EINVAL, "the leading dimension must be >= the rows of b");
  if (m == 0 || n == 0) return PSGD_OK;
  if (!c || !aligned_to(c, type_size(ot))) return fail(ctx, PSGD_EINVAL, "c must be a pointer aligned to its element type");
  if (scale && !aligned_to(scale, 4)) return fail(ctx, PSGD_EINVAL, "scale must be aligned to its element type");
  psgd::MxProduct p{};
  p.p = psgd::mx_view(b->data, n, b->k);
  p.q = psgd::mx_view(a->data, m, a->k);
  const psgd::MxPlan plan = psgd::mx_plan(m, n, p.p.panels);
  const int64_t need = plan.splits > 1 ? plan.splits * m * n * 4 : 0;
  if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need))
    return fail(ctx, PSGD_EINVAL, "the workspace needs %lld bytes at a 16-byte aligned address, got %lld", (long long)need,
                (long long)workspace_bytes);
  const Bytes out = strided(c, m, n, ld_c, type_size(ot)), ws{workspace, need}, s{scale, 4};
  for (const Bytes& in : {bytes_of(a), bytes_of(b), s})
    if (meet(out, in) || meet(ws, in)) return fail(ctx, PSGD_EINVAL, "c and the workspace must not overlap a, b or scale");
  if (meet(out, ws)) return fail(ctx, PSGD_EINVAL, "c must not overlap the workspace");
  p.m = m; p.n = n;
  p.c = c; p.ldc = ld_c;
  p.scale = scale; p.accumulate = accumulate != 0;
  p.per = (int32_t)((p.p.panels + plan.splits - 1) / plan.splits);
  p.splits = p.per > 0 ? (int32_t)((p.p.panels + p.per - 1) / p.per) : 1;      // no part is empty
  p.partial = static_cast<float*>(workspace);
  DeviceGuard dev(ctx->device);
  HIPCHK(ctx, dev.err, "hipSetDevice");
  HIPCHK(ctx, psgd::launch_mx_product(p, plan.tile, ot, stream), "4-bit product");
  return PSGD_OK;
}

}  // extern "C"
