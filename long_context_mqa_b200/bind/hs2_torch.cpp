// Argument marshalling for the per-step calls of the C ABI (include/hs2.h) from torch tensors: the
// dtype, device, rank, contiguity and shape checks of the Python binding, done in C++ so that a
// decode step's calls cost the host a few microseconds. No arithmetic: every entry checks its
// tensors and calls the C function whose address the Python binding passes in once (the functions
// live in libhs2.so, loaded by the binding). Argument errors raise ValueError.
#include <c10/core/DeviceGuard.h>
#include <torch/extension.h>

#include <cstdint>

namespace {

using hs2_status = int;
using FullFn = hs2_status (*)(const void*, const void*, const void*, int, int, int, int, int, float, int, int, void*,
                              float*, int32_t*, void*, size_t, void*);
using SparseFn = hs2_status (*)(const void*, const void*, const void*, const int32_t*, int, int, int, int, int, int,
                                float, void*, float*, void*, size_t, void*);

FullFn g_full = nullptr;
SparseFn g_sparse = nullptr;

void set_entries(int64_t full, int64_t sparse) {
  g_full = reinterpret_cast<FullFn>(full);
  g_sparse = reinterpret_cast<SparseFn>(sparse);
}

// argument errors surface in Python as ValueError, as in the binding's other entries
#define HS2_ARG_CHECK(cond, ...) \
  do {                              \
    if (!(cond)) throw pybind11::value_error(c10::str(__VA_ARGS__)); \
  } while (0)

inline void need(const at::Tensor& t, const char* name, at::ScalarType dt, int64_t dim) {
  HS2_ARG_CHECK(t.is_cuda(), name, " must be a CUDA tensor");
  HS2_ARG_CHECK(t.scalar_type() == dt, name, " must be ", c10::toString(dt), ", got ", c10::toString(t.scalar_type()));
  HS2_ARG_CHECK(t.dim() == dim, name, " must have ", dim, " dims, got ", t.sizes());
  HS2_ARG_CHECK(t.is_contiguous(), name, " must be contiguous");
}

// hs2_full_attn_select: q [B,Lq,H,d] bf16; k, v [B,Lk,d] bf16; out [B,Lq,H,d] bf16; lse [B,Lq,H]
// fp32; idx [B,Lq,window+topk] int32; ws uint8. Returns the C status.
int64_t full_attn_select(const at::Tensor& q, const at::Tensor& k, const at::Tensor& v, double scale, int64_t window,
                         int64_t topk, const at::Tensor& out, const at::Tensor& lse, const at::Tensor& idx,
                         const at::Tensor& ws, int64_t stream) {
  HS2_ARG_CHECK(g_full != nullptr, "entry points not set");
  need(q, "q", at::kBFloat16, 4);
  need(k, "k", at::kBFloat16, 3);
  need(v, "v", at::kBFloat16, 3);
  const int64_t B = q.size(0), Lq = q.size(1), H = q.size(2), d = q.size(3), Lk = k.size(1);
  HS2_ARG_CHECK(k.size(0) == B && k.size(2) == d && v.sizes() == k.sizes(), "k and v must be [B, Lk, d] matching q");
  need(out, "out", at::kBFloat16, 4);
  need(lse, "lse", at::kFloat, 3);
  need(idx, "idx", at::kInt, 3);
  HS2_ARG_CHECK(out.sizes() == q.sizes(), "out must be shaped like q");
  HS2_ARG_CHECK(lse.size(0) == B && lse.size(1) == Lq && lse.size(2) == H, "lse must be [B, Lq, H]");
  HS2_ARG_CHECK(idx.size(0) == B && idx.size(1) == Lq && idx.size(2) == window + topk, "idx must be [B, Lq, window + topk]");
  HS2_ARG_CHECK(ws.is_cuda() && ws.is_contiguous(), "workspace must be a contiguous CUDA tensor");
  return g_full(q.data_ptr(), k.data_ptr(), v.data_ptr(), (int)B, (int)Lq, (int)Lk, (int)H, (int)d, (float)scale,
                (int)window, (int)topk, out.data_ptr(), lse.data_ptr<float>(), idx.data_ptr<int32_t>(), ws.data_ptr(),
                (size_t)ws.nbytes(), reinterpret_cast<void*>(stream));
}

// hs2_sparse_attn: q [B,Lq,H,d] bf16; k, v [B,Lk,d] bf16; idx [B,Lq,S] int32; out like q; lse
// [B,Lq,H] fp32 or None; ws uint8. Returns the C status.
int64_t sparse_attn(const at::Tensor& q, const at::Tensor& k, const at::Tensor& v, const at::Tensor& idx, double scale,
                    const at::Tensor& out, const c10::optional<at::Tensor>& lse, const at::Tensor& ws, int64_t stream) {
  HS2_ARG_CHECK(g_sparse != nullptr, "entry points not set");
  need(q, "q", at::kBFloat16, 4);
  need(k, "k", at::kBFloat16, 3);
  need(v, "v", at::kBFloat16, 3);
  need(idx, "idx", at::kInt, 3);
  const int64_t B = q.size(0), Lq = q.size(1), H = q.size(2), d = q.size(3), Lk = k.size(1), S = idx.size(2);
  HS2_ARG_CHECK(k.size(0) == B && k.size(2) == d && v.sizes() == k.sizes(), "k and v must be [B, Lk, d] matching q");
  HS2_ARG_CHECK(idx.size(0) == B && idx.size(1) == Lq, "idx must be [B, Lq, S]");
  need(out, "out", at::kBFloat16, 4);
  HS2_ARG_CHECK(out.sizes() == q.sizes(), "out must be shaped like q");
  float* lse_p = nullptr;
  if (lse.has_value()) {
    need(*lse, "lse", at::kFloat, 3);
    HS2_ARG_CHECK(lse->size(0) == B && lse->size(1) == Lq && lse->size(2) == H, "lse must be [B, Lq, H]");
    lse_p = lse->data_ptr<float>();
  }
  HS2_ARG_CHECK(ws.is_cuda() && ws.is_contiguous(), "workspace must be a contiguous CUDA tensor");
  return g_sparse(q.data_ptr(), k.data_ptr(), v.data_ptr(), idx.data_ptr<int32_t>(), (int)B, (int)Lq, (int)Lk, (int)H,
                  (int)d, (int)S, (float)scale, out.data_ptr(), lse_p, ws.data_ptr(), (size_t)ws.nbytes(),
                  reinterpret_cast<void*>(stream));
}

// ---------------------------------------------------------------------------------------------
// norm and rotation of query and key heads, page tables, decode attention over pages
// ---------------------------------------------------------------------------------------------
using ll = long long;
using OptT = c10::optional<at::Tensor>;
using RopeFn = hs2_status (*)(const void*, const void*, ll, ll, ll, ll, const int32_t*, const double*, int, int, int, int,
                              int, int, float, float, const void*, const void*, int, void*, void*, void*);
using RopeBwdFn = hs2_status (*)(const void*, const void*, ll, ll, ll, ll, const int32_t*, const double*, int, int, int,
                                 int, int, int, float, float, const void*, const void*, int, const void*, const void*,
                                 int, void*, void*, float*, float*, void*, size_t, void*);
using RopePagedFn = hs2_status (*)(const void*, const void*, const void*, ll, ll, ll, ll, ll, ll, const int32_t*,
                                   const int32_t*, const double*, int, int, int, int, int, int, float, float, const void*,
                                   const void*, int, void*, void*, void*, const ll*, const ll*, int, int, int, float,
                                   float, void*, size_t, void*);
using TableFn = hs2_status (*)(int32_t*, int, int, const int32_t*, const int32_t*, int32_t*, int, const int32_t*, int,
                               int, int32_t*, int32_t*, int32_t*, int32_t*, int32_t*, void*, size_t, void*);
using PagedFn = hs2_status (*)(const void*, const void*, const void*, const ll*, const ll*, int, int, const int32_t*, int,
                               const int32_t*, int, int, int, int, int, float, float, float, int, void*, float*, void*,
                               size_t, void*);
RopeFn g_rope = nullptr;
RopeBwdFn g_rope_bwd = nullptr;
RopePagedFn g_rope_paged = nullptr;
TableFn g_table = nullptr;
PagedFn g_paged = nullptr;

using CapturingFn = int (*)(void*);
CapturingFn g_capturing = nullptr;

void set_cache_entries(int64_t rope, int64_t rope_bwd, int64_t rope_paged, int64_t table, int64_t paged,
                       int64_t stream_capturing) {
  g_rope = reinterpret_cast<RopeFn>(rope);
  g_rope_bwd = reinterpret_cast<RopeBwdFn>(rope_bwd);
  g_rope_paged = reinterpret_cast<RopePagedFn>(rope_paged);
  g_table = reinterpret_cast<TableFn>(table);
  g_paged = reinterpret_cast<PagedFn>(paged);
  g_capturing = reinterpret_cast<CapturingFn>(stream_capturing);
}

inline void need_on(const at::Tensor& t, const char* name, at::ScalarType dt, int64_t dim, const at::Tensor& like) {
  need(t, name, dt, dim);
  HS2_ARG_CHECK(t.device() == like.device(), name, " is on ", t.device(), ", not on ", like.device());
}
inline int fits(int64_t n, const char* what) {
  HS2_ARG_CHECK(n >= 0 && n <= 0x7FFFFFFF, what, " is out of range");
  return (int)n;
}

// Rows of heads: x [T, H, d] or [B, L, H, d] (no head dimension: one head) as `lead` leading dims of
// evenly spaced tokens, heads and elements; any strides but the last.
struct Rows {
  const void* p = nullptr;
  int64_t T = 0, H = 0, d = 0;
  ll ts = 0, hs = 0;
};
Rows rows_of(const at::Tensor& x, const char* name, int64_t lead, const at::Tensor& like) {
  HS2_ARG_CHECK(x.is_cuda(), name, " must be a CUDA tensor");
  HS2_ARG_CHECK(x.scalar_type() == at::kBFloat16, name, " must be BFloat16, got ", c10::toString(x.scalar_type()));
  HS2_ARG_CHECK(x.device() == like.device(), name, " is on ", x.device(), ", not on ", like.device());
  HS2_ARG_CHECK(x.dim() == lead + 2 || x.dim() == lead + 1, name, " must have ", lead + 2, " dims, got ", x.sizes());
  Rows r;
  const bool heads = x.dim() == lead + 2;
  r.p = x.data_ptr();
  r.d = x.size(-1);
  r.H = heads ? x.size(-2) : 1;
  HS2_ARG_CHECK(x.stride(-1) == 1 || r.d <= 1, name, "'s last dimension must be contiguous");
  r.T = lead == 1 ? x.size(0) : x.size(0) * x.size(1);
  if (lead == 1 || x.size(1) == 1) {
    r.ts = x.stride(0);
  } else {
    HS2_ARG_CHECK(x.size(0) <= 1 || x.stride(0) == x.size(1) * x.stride(1), name, "'s tokens must be evenly spaced");
    r.ts = x.stride(1);
  }
  r.hs = heads ? x.stride(-2) : 0;
  if (r.T <= 1) r.ts = 0;
  if (r.H <= 1) r.hs = 0;
  for (int64_t i = 0; i < lead; ++i) HS2_ARG_CHECK(x.size(i) == like.size(i), name, " must have q's leading dims");
  HS2_ARG_CHECK(r.ts % 8 == 0 && r.hs % 8 == 0 && reinterpret_cast<uintptr_t>(r.p) % 16 == 0, name,
                "'s heads must start on 16-byte boundaries");
  return r;
}
const void* weight_of(const OptT& w, const char* name, int64_t d, const at::Tensor& like, int* f32) {
  if (!w.has_value()) return nullptr;
  *f32 = w->scalar_type() == at::kFloat;
  need_on(*w, name, *f32 ? at::kFloat : at::kBFloat16, 1, like);
  HS2_ARG_CHECK(w->size(0) == d, name, " must have ", d, " elements");
  return w->data_ptr();
}
struct RopeArgs {
  Rows q, k;
  const int32_t* pos;
  const double* freq;
  const void *qw, *kw;
  int T, Hq, Hk, d, rot, f32;
};
RopeArgs rope_args(const at::Tensor& q, const OptT& k, const at::Tensor& positions, const at::Tensor& inv_freq,
                   const OptT& qw, const OptT& kw) {
  RopeArgs a{};
  HS2_ARG_CHECK(q.dim() == 3 || q.dim() == 4, "q must be [T, Hq, d] or [B, L, Hq, d], got ", q.sizes());
  const int64_t lead = q.dim() - 2;
  a.q = rows_of(q, "q", lead, q);
  if (k.has_value()) {
    a.k = rows_of(*k, "k", lead, q);
    HS2_ARG_CHECK(a.k.d == a.q.d, "k must have q's head dimension");
  }
  need_on(positions, "positions", at::kInt, lead, q);
  for (int64_t i = 0; i < lead; ++i) HS2_ARG_CHECK(positions.size(i) == q.size(i), "positions must have q's leading dims");
  need_on(inv_freq, "inv_freq", at::kDouble, 1, q);
  a.T = fits(a.q.T, "the number of tokens");
  a.Hq = fits(a.q.H, "Hq");
  a.Hk = fits(a.k.H, "Hk");
  a.d = fits(a.q.d, "d");
  a.rot = fits(2 * inv_freq.size(0), "the rotated part");
  a.pos = positions.data_ptr<int32_t>();
  a.freq = inv_freq.data_ptr<double>();
  int f2 = 0;
  a.qw = weight_of(qw, "q_weight", a.d, q, &a.f32);
  a.kw = weight_of(kw, "k_weight", a.d, q, &f2);
  HS2_ARG_CHECK(a.Hk == 0 || (a.qw == nullptr) == (a.kw == nullptr), "give both norm weights or neither");
  HS2_ARG_CHECK(a.Hk > 0 || a.kw == nullptr, "k_weight without k");
  HS2_ARG_CHECK(a.kw == nullptr || f2 == a.f32, "q_weight and k_weight must have one dtype");
  return a;
}
void* out_of(const at::Tensor& o, const char* name, at::ScalarType dt, const at::Tensor& shape) {
  need_on(o, name, dt, shape.dim(), shape);
  HS2_ARG_CHECK(o.sizes() == shape.sizes(), name, " must be shaped ", shape.sizes(), ", got ", o.sizes());
  return o.data_ptr();
}
// kept: the binding's own workspace of the stream. A captured graph would outlive the binding's choice of a
// buffer, and two graphs would share it.
void need_ws(const at::Tensor& ws, const at::Tensor& like, bool kept, int64_t stream) {
  HS2_ARG_CHECK(!kept || g_capturing(reinterpret_cast<void*>(stream)) == 0,
                "give a workspace of your own while capturing a graph");
  HS2_ARG_CHECK(ws.is_cuda() && ws.is_contiguous(), "workspace must be a contiguous CUDA tensor");
  HS2_ARG_CHECK(ws.device() == like.device(), "workspace is on ", ws.device(), ", not on ", like.device());
}

// hs2_qk_norm_rope
int64_t qk_norm_rope(const at::Tensor& q, const OptT& k, const at::Tensor& positions, const at::Tensor& inv_freq,
                     const OptT& qw, const OptT& kw, double eps, bool interleaved, double mscale, const at::Tensor& q_out,
                     const OptT& k_out, int64_t stream) {
  const RopeArgs a = rope_args(q, k, positions, inv_freq, qw, kw);
  void* qo = out_of(q_out, "q_out", at::kBFloat16, q);
  HS2_ARG_CHECK(k.has_value() == k_out.has_value(), "k_out goes with k");
  void* ko = k.has_value() ? out_of(*k_out, "k_out", at::kBFloat16, *k) : nullptr;
  c10::DeviceGuard guard(q.device());
  return g_rope(a.q.p, a.k.p, a.q.ts, a.q.hs, a.k.ts, a.k.hs, a.pos, a.freq, a.T, a.Hq, a.Hk, a.d, a.rot, interleaved,
                (float)mscale, (float)eps, a.qw, a.kw, a.f32, qo, ko, reinterpret_cast<void*>(stream));
}

// hs2_qk_norm_rope_bwd
int64_t qk_norm_rope_bwd(const at::Tensor& q, const OptT& k, const at::Tensor& positions, const at::Tensor& inv_freq,
                         const at::Tensor& dq_out, const OptT& dk_out, const OptT& qw, const OptT& kw, double eps,
                         bool interleaved, double mscale, const at::Tensor& dq, const OptT& dk, const OptT& dqw,
                         const OptT& dkw, const OptT& ws, bool kept, int64_t stream) {
  const RopeArgs a = rope_args(q, k, positions, inv_freq, qw, kw);
  const void* gq = out_of(dq_out, "dq_out", at::kBFloat16, q);
  void* xq = out_of(dq, "dq", at::kBFloat16, q);
  HS2_ARG_CHECK(k.has_value() == dk_out.has_value() && k.has_value() == dk.has_value(), "dk_out and dk go with k");
  const void* gk = nullptr;
  void* xk = nullptr;
  bool g32 = false;
  if (k.has_value()) {
    g32 = dk_out->scalar_type() == at::kFloat;
    gk = out_of(*dk_out, "dk_out", g32 ? at::kFloat : at::kBFloat16, *k);
    xk = out_of(*dk, "dk", at::kBFloat16, *k);
  }
  HS2_ARG_CHECK((a.qw != nullptr) == dqw.has_value() && (a.kw != nullptr) == dkw.has_value(),
                "dq_weight and dk_weight go with the weights");
  if (dqw.has_value()) {
    need_on(*dqw, "dq_weight", at::kFloat, 1, q);
    HS2_ARG_CHECK(dqw->size(0) == a.d, "dq_weight must have ", a.d, " elements");
  }
  if (dkw.has_value()) {
    need_on(*dkw, "dk_weight", at::kFloat, 1, q);
    HS2_ARG_CHECK(dkw->size(0) == a.d, "dk_weight must have ", a.d, " elements");
  }
  if (ws.has_value()) need_ws(*ws, q, kept, stream);
  c10::DeviceGuard guard(q.device());
  return g_rope_bwd(a.q.p, a.k.p, a.q.ts, a.q.hs, a.k.ts, a.k.hs, a.pos, a.freq, a.T, a.Hq, a.Hk, a.d, a.rot, interleaved,
                    (float)mscale, (float)eps, a.qw, a.kw, a.f32, gq, gk, g32, xq, xk,
                    dqw.has_value() ? dqw->data_ptr<float>() : nullptr, dkw.has_value() ? dkw->data_ptr<float>() : nullptr,
                    ws.has_value() ? ws->data_ptr() : nullptr, ws.has_value() ? (size_t)ws->nbytes() : 0,
                    reinterpret_cast<void*>(stream));
}

// A page pool [n_pages, page, Hk, d] (or [n_pages, page, d]: one head), any strides but the last
struct Pool {
  void* p;
  int64_t n, page, H, d;
  ll strides[3];
};
Pool pool_of(const at::Tensor& t, const char* name, bool f8, const at::Tensor& like) {
  HS2_ARG_CHECK(t.is_cuda(), name, " must be a CUDA tensor");
  HS2_ARG_CHECK(t.device() == like.device(), name, " is on ", t.device(), ", not on ", like.device());
  HS2_ARG_CHECK(t.scalar_type() == (f8 ? at::kByte : at::kBFloat16), name, " must be ",
                f8 ? "uint8 e4m3 codes (scales were given)" : "BFloat16 (or uint8 with k_scale and v_scale)", ", got ",
                c10::toString(t.scalar_type()));
  HS2_ARG_CHECK(t.dim() == 3 || t.dim() == 4, name, " must be [n_pages, page, Hk, d] or [n_pages, page, d], got ", t.sizes());
  const bool heads = t.dim() == 4;
  Pool r{t.data_ptr(), t.size(0), t.size(1), heads ? t.size(2) : 1, t.size(-1), {}};
  HS2_ARG_CHECK(t.stride(-1) == 1, name, "'s last dimension must be contiguous");
  // (the stride of a dimension of one element says nothing)
  r.strides[1] = r.page > 1 ? t.stride(1) : r.d;
  r.strides[2] = heads && r.H > 1 ? t.stride(2) : r.d;
  r.strides[0] = r.n > 1 ? t.stride(0) : r.d;
  const ll unit = f8 ? 16 : 8;
  for (ll s : r.strides) HS2_ARG_CHECK(s > 0 && s % unit == 0, name, "'s rows must be 16-byte aligned and apart");
  HS2_ARG_CHECK(reinterpret_cast<uintptr_t>(r.p) % 16 == 0, name, " must start on a 16-byte boundary");
  return r;
}
bool same_shape(const Pool& a, const Pool& b) { return a.n == b.n && a.page == b.page && a.H == b.H && a.d == b.d; }

// hs2_qk_norm_rope_paged
int64_t qk_norm_rope_paged(const at::Tensor& q, const at::Tensor& k, const at::Tensor& v, const at::Tensor& positions,
                           const at::Tensor& slots, const at::Tensor& k_pages, const at::Tensor& v_pages,
                           const at::Tensor& inv_freq, const OptT& qw, const OptT& kw, double eps, bool interleaved,
                           double mscale, bool f8, double k_scale, double v_scale, const at::Tensor& q_out,
                           const at::Tensor& ws, bool kept, int64_t stream) {
  const RopeArgs a = rope_args(q, k, positions, inv_freq, qw, kw);
  const Rows vr = rows_of(v, "v", q.dim() - 2, q);
  HS2_ARG_CHECK(vr.H == a.Hk && vr.d == a.d, "v must be shaped like k");
  need_on(slots, "slots", at::kInt, positions.dim(), q);
  HS2_ARG_CHECK(slots.sizes() == positions.sizes(), "slots must be shaped like positions");
  void* qo = out_of(q_out, "q_out", at::kBFloat16, q);
  const Pool kp = pool_of(k_pages, "k_pages", f8, q), vp = pool_of(v_pages, "v_pages", f8, q);
  HS2_ARG_CHECK(same_shape(kp, vp) && kp.H == a.Hk && kp.d == a.d, "k_pages and v_pages must be [n_pages, page, Hk, d]");
  need_ws(ws, q, kept, stream);
  c10::DeviceGuard guard(q.device());
  return g_rope_paged(a.q.p, a.k.p, vr.p, a.q.ts, a.q.hs, a.k.ts, a.k.hs, vr.ts, vr.hs, a.pos, slots.data_ptr<int32_t>(),
                      a.freq, a.T, a.Hq, a.Hk, a.d, a.rot, interleaved, (float)mscale, (float)eps, a.qw, a.kw, a.f32, qo,
                      kp.p, vp.p, kp.strides, vp.strides, fits(kp.n, "n_pages"), fits(kp.page, "page size"), f8,
                      (float)k_scale, (float)v_scale, ws.data_ptr(), (size_t)ws.nbytes(), reinterpret_cast<void*>(stream));
}

// hs2_page_table_update
int64_t page_table_update(const at::Tensor& table, const at::Tensor& lens, const at::Tensor& delta,
                          const at::Tensor& ring, const at::Tensor& state, int64_t page, int64_t max_tokens,
                          const at::Tensor& lens_out, const at::Tensor& state_out, const at::Tensor& cu,
                          const at::Tensor& positions, const at::Tensor& slots, const at::Tensor& ws, bool kept, int64_t stream) {
  need(table, "page_table", at::kInt, 2);
  const int64_t B = table.size(0);
  need_on(lens, "lens", at::kInt, 1, table);
  need_on(delta, "delta", at::kInt, 1, table);
  need_on(ring, "free_ring", at::kInt, 1, table);
  need_on(state, "free_state", at::kInt, 1, table);
  need_on(lens_out, "lens_out", at::kInt, 1, table);
  need_on(state_out, "free_state_out", at::kInt, 1, table);
  need_on(cu, "cu_tokens", at::kInt, 1, table);
  need_on(positions, "positions", at::kInt, 1, table);
  need_on(slots, "slots", at::kInt, 1, table);
  HS2_ARG_CHECK(lens.size(0) == B && delta.size(0) == B && lens_out.size(0) == B, "lens, delta and lens_out must be [B]");
  HS2_ARG_CHECK(state.size(0) == 2 && state_out.size(0) == 2, "free_state must hold the ring's head and count");
  HS2_ARG_CHECK(cu.size(0) == B + 1, "cu_tokens must be [B + 1]");
  HS2_ARG_CHECK(positions.size(0) == max_tokens && slots.size(0) == max_tokens, "positions and slots must be [max_tokens]");
  need_ws(ws, table, kept, stream);
  c10::DeviceGuard guard(table.device());
  return g_table(table.data_ptr<int32_t>(), fits(B, "B"), fits(table.size(1), "max_pages"), lens.data_ptr<int32_t>(),
                 delta.data_ptr<int32_t>(), ring.data_ptr<int32_t>(), fits(ring.size(0), "the ring's size"),
                 state.data_ptr<int32_t>(), fits(page, "page_size"), fits(max_tokens, "max_tokens"),
                 lens_out.data_ptr<int32_t>(), state_out.data_ptr<int32_t>(), cu.data_ptr<int32_t>(),
                 positions.data_ptr<int32_t>(), slots.data_ptr<int32_t>(), ws.data_ptr(), (size_t)ws.nbytes(),
                 reinterpret_cast<void*>(stream));
}

// hs2_paged_attn
int64_t paged_attn(const at::Tensor& q, const at::Tensor& k_pages, const at::Tensor& v_pages, const at::Tensor& table,
                   const at::Tensor& lens, bool f8, double k_scale, double v_scale, double scale, int64_t window,
                   const at::Tensor& out, const OptT& lse, const at::Tensor& ws, bool kept, int64_t stream) {
  need(q, "q", at::kBFloat16, 4);
  const int64_t B = q.size(0), Hq = q.size(2), d = q.size(3);
  HS2_ARG_CHECK(q.size(1) == 1, "q must be [B, 1, Hq, d], got ", q.sizes());
  const Pool kp = pool_of(k_pages, "k_pages", f8, q), vp = pool_of(v_pages, "v_pages", f8, q);
  HS2_ARG_CHECK(same_shape(kp, vp) && kp.d == d, "k_pages and v_pages must be [n_pages, page, Hk, d] with q's d");
  HS2_ARG_CHECK(kp.H > 0 && Hq % kp.H == 0, "Hq must be a multiple of the key heads");
  need_on(table, "page_table", at::kInt, 2, q);
  need_on(lens, "lens", at::kInt, 1, q);
  HS2_ARG_CHECK(table.size(0) == B && lens.size(0) == B, "page_table must be [B, max_pages] and lens [B]");
  void* o = out_of(out, "out", at::kBFloat16, q);
  float* l = nullptr;
  if (lse.has_value()) {
    need_on(*lse, "lse", at::kFloat, 3, q);
    HS2_ARG_CHECK(lse->size(0) == B && lse->size(1) == 1 && lse->size(2) == Hq, "lse must be [B, 1, Hq]");
    l = lse->data_ptr<float>();
  }
  need_ws(ws, q, kept, stream);
  c10::DeviceGuard guard(q.device());
  return g_paged(q.data_ptr(), kp.p, vp.p, kp.strides, vp.strides, fits(kp.n, "n_pages"), fits(kp.page, "page size"),
                 table.data_ptr<int32_t>(), fits(table.size(1), "max_pages"), lens.data_ptr<int32_t>(), fits(B, "B"),
                 fits(Hq, "Hq"), fits(kp.H, "Hk"), fits(d, "d"), f8, (float)k_scale, (float)v_scale, (float)scale,
                 fits(window, "window"), o, l, ws.data_ptr(), (size_t)ws.nbytes(), reinterpret_cast<void*>(stream));
}

}  // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m) {
  m.def("set_entries", &set_entries);
  m.def("set_cache_entries", &set_cache_entries);
  m.def("qk_norm_rope", &qk_norm_rope);
  m.def("qk_norm_rope_bwd", &qk_norm_rope_bwd);
  m.def("qk_norm_rope_paged", &qk_norm_rope_paged);
  m.def("page_table_update", &page_table_update);
  m.def("paged_attn", &paged_attn);
  m.def("full_attn_select", &full_attn_select);
  m.def("sparse_attn", &sparse_attn);
}
