// C ABI of a decoder block's operators around its deployed products
// (lcp_rms_norm*, lcp_sparse_pack_e4m3*, lcp_sparse_linear*): argument
// validation. Every check runs before the first launch, so an error return means
// nothing was enqueued.
#include <math.h>

#include "../../include/lcp.h"
#include "block.h"

using namespace lcp;

namespace {

inline bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
inline hipStream_t S(void* s) { return reinterpret_cast<hipStream_t>(s); }
inline uintptr_t esize(int t) { return t == LCP_F32 ? 4 : t == LCP_BF16 ? 2 : 1; }
inline bool float_type(int t) { return t == LCP_F32 || t == LCP_BF16; }
constexpr int64_t kMaxStride = (int64_t)1 << 40;
// Bytes from a matrix's first row to its last: offsets then stay far inside 64 bits.
constexpr int64_t kMaxSpan = (int64_t)1 << 58;

bool good_in(const void* p, int64_t row, int T, uintptr_t unit) {
  return p && row >= 0 && row <= kMaxStride && row <= kMaxSpan / T && aligned(p, unit);
}
bool good_out(const void* p, int64_t row, int T, int C, uintptr_t unit) {
  return good_in(p, row, T, unit) && (T == 1 || row >= C);
}
// An output at an input's own address has to have its rows.
bool same_rows(const void* out, int64_t out_row, const void* in, int64_t in_row, int T) {
  return out != in || out_row == in_row || T == 1;
}

constexpr int kMaxC = 32768;

int check_pack(int cout, int cin) {
  if (cout <= 0 || cin <= 0 || cout % 32 || cin % 32 || (int64_t)cout * cin >= ((int64_t)1 << 31)) return LCP_E_INVAL;
  return LCP_OK;
}

int check_packed(const lcp_packed* w, PackedArgs* out) {
  if (!w) return LCP_E_INVAL;
  if (w->dt != LCP_BF16 && w->dt != LCP_E4M3) return LCP_E_UNSUPPORTED;
  const int rc = check_pack(w->cout, w->cin);
  if (rc != LCP_OK) return rc;
  if (!w->vals || !w->meta || !aligned(w->vals, 16) || !aligned(w->meta, 4)) return LCP_E_INVAL;
  const bool fp8 = w->dt == LCP_E4M3;
  if (w->fast != 0 && (w->fast != 1 || !fp8)) return LCP_E_INVAL;
  if (fp8 && (!w->wscale || !aligned(w->wscale, 16))) return LCP_E_INVAL;
  // the weights are read through 32-bit byte offsets
  if ((int64_t)w->cout * w->cin >= ((int64_t)1 << (fp8 ? 31 : 30))) return LCP_E_INVAL;
  *out = PackedArgs{(const u32x4*)w->vals, w->meta, fp8 ? w->wscale : nullptr, fp8, w->cout, w->cin, w->fast};
  return LCP_OK;
}

#define LCP_RUN(expr)                                                                             \
  do {                                                                                            \
    const hipError_t err = (expr);                                                                \
    if (err != hipSuccess) return err == hipErrorInvalidConfiguration ? LCP_E_INVAL : LCP_E_HIP; \
  } while (0)

}  // namespace

extern "C" {

int lcp_rms_norm(const lcp_norm* n, void* stream) {
  if (!n || n->T <= 0 || n->C <= 0) return LCP_E_INVAL;
  if (!float_type(n->dt) || !float_type(n->weight_dt) || (!float_type(n->y_dt) && n->y_dt != LCP_E4M3))
    return LCP_E_UNSUPPORTED;
  if (n->C > kMaxC) return LCP_E_UNSUPPORTED;
  if (!isfinite(n->eps) || !(n->eps > 0.f)) return LCP_E_INVAL;
  const uintptr_t es = esize(n->dt);
  if (!good_in(n->x, n->x_row, n->T, es) || !n->weight || !aligned(n->weight, esize(n->weight_dt))) return LCP_E_INVAL;
  if (n->residual && !good_in(n->residual, n->residual_row, n->T, es)) return LCP_E_INVAL;
  if (!good_out(n->y, n->y_row, n->T, n->C, esize(n->y_dt))) return LCP_E_INVAL;
  if (n->y == n->x || n->y == n->residual || n->y == n->sum || n->y == n->weight) return LCP_E_INVAL;
  if (n->sum) {
    if (!good_out(n->sum, n->sum_row, n->T, n->C, es)) return LCP_E_INVAL;
    if (!same_rows(n->sum, n->sum_row, n->x, n->x_row, n->T) ||
        !same_rows(n->sum, n->sum_row, n->residual, n->residual_row, n->T))
      return LCP_E_INVAL;
  }
  if (n->y_dt == LCP_E4M3 && (!n->scale || !aligned(n->scale, 4))) return LCP_E_INVAL;
  if (n->perm) {
    if (!aligned(n->perm, 4)) return LCP_E_INVAL;
    if (n->B != 32 && n->B != 64 && n->B != 128) return LCP_E_UNSUPPORTED;
    if (n->C % n->B != 0) return LCP_E_INVAL;
  }
  NormArgs a{};
  a.x = Mat{n->x, n->x_row};
  a.res = Mat{n->residual, n->residual_row};
  a.sum = MatOut{n->sum, n->sum_row};
  a.y = MatOut{n->y, n->y_row};
  a.w = n->weight;
  a.scale = n->scale;
  a.perm = n->perm;
  a.wt = n->weight_dt;
  a.yt = n->y_dt;
  a.T = n->T;
  a.C = n->C;
  a.B = n->perm ? n->B : 0;
  a.eps = n->eps;
  LCP_RUN(launch_rms_norm(a, n->dt, S(stream)));
  return LCP_OK;
}

int lcp_rms_norm_bwd_workspace_bytes(int T, int C, size_t* bytes) {
  if (!bytes || T <= 0 || C <= 0) return LCP_E_INVAL;
  if (C > kMaxC) return LCP_E_UNSUPPORTED;
  *bytes = norm_grad_workspace_bytes(T, C);
  return LCP_OK;
}

int lcp_rms_norm_bwd(const void* h, int64_t h_row, const void* dy, int64_t dy_row, const void* dsum, int64_t dsum_row,
                     const void* weight, lcp_dtype dt, lcp_dtype weight_dt, int T, int C, float eps, void* dx,
                     int64_t dx_row, void* dweight, void* ws, size_t ws_bytes, void* stream) {
  if (T <= 0 || C <= 0) return LCP_E_INVAL;
  if (!float_type(dt) || !float_type(weight_dt) || C > kMaxC) return LCP_E_UNSUPPORTED;
  if (!isfinite(eps) || !(eps > 0.f)) return LCP_E_INVAL;
  const uintptr_t es = esize(dt), wes = esize(weight_dt);
  if (!good_in(h, h_row, T, es) || !good_in(dy, dy_row, T, es) || !weight || !aligned(weight, wes)) return LCP_E_INVAL;
  if (dsum && !good_in(dsum, dsum_row, T, es)) return LCP_E_INVAL;
  if (!good_out(dx, dx_row, T, C, es) || !dweight || !aligned(dweight, wes)) return LCP_E_INVAL;
  if (dx == h || dx == dy || dx == weight || dx == dweight || dweight == weight || dweight == h || dweight == dy ||
      dweight == dsum || !same_rows(dx, dx_row, dsum, dsum_row, T))
    return LCP_E_INVAL;
  const size_t need = norm_grad_workspace_bytes(T, C);
  if (!ws) return LCP_E_INVAL;
  if (!aligned(ws, 256) || ws_bytes < need) return LCP_E_WORKSPACE;
  NormGradArgs a{};
  a.h = Mat{h, h_row};
  a.dy = Mat{dy, dy_row};
  a.dsum = Mat{dsum, dsum_row};
  a.dx = MatOut{dx, dx_row};
  a.w = weight;
  a.dw = dweight;
  a.ws = (float*)ws;
  a.wt = weight_dt;
  a.T = T;
  a.C = C;
  a.eps = eps;
  LCP_RUN(launch_rms_norm_bwd(a, dt, S(stream)));
  return LCP_OK;
}

int lcp_sparse_pack_e4m3_bytes(int cout, int cin, size_t* vals_bytes, size_t* meta_bytes) {
  if (!vals_bytes || !meta_bytes) return LCP_E_INVAL;
  const int rc = check_pack(cout, cin);
  if (rc != LCP_OK) return rc;
  *vals_bytes = sparse_vals_bytes_e4m3(cout, cin);
  *meta_bytes = sparse_meta_bytes_e4m3(cout, cin);
  return LCP_OK;
}

int lcp_sparse_pack_e4m3(const void* W, int cout, int cin, int B, const int32_t* perm, const uint32_t* bits, void* vals,
                         uint32_t* meta, float* wscale, void* stream) {
  if (!W || !perm || !bits || !vals || !meta || !wscale) return LCP_E_INVAL;
  const int rc = check_pack(cout, cin);
  if (rc != LCP_OK) return rc;
  if (B != 32 && B != 64 && B != 128) return LCP_E_UNSUPPORTED;
  if (cin % B) return LCP_E_INVAL;
  if (!aligned(W, 2) || !aligned(perm, 4) || !aligned(bits, 4) || !aligned(vals, 16) || !aligned(meta, 4) ||
      !aligned(wscale, 16))
    return LCP_E_INVAL;
  LCP_RUN(launch_sparse_pack_e4m3((const uint16_t*)W, cout, cin, B, perm, bits, (u32x4*)vals, meta, wscale, S(stream)));
  return LCP_OK;
}

int lcp_sparse_linear_workspace_bytes(const lcp_packed* w, int T, size_t* bytes) {
  PackedArgs p;
  const int rc = check_packed(w, &p);
  if (rc != LCP_OK) return rc;
  if (!bytes || T <= 0) return LCP_E_INVAL;
  *bytes = sparse_linear_workspace_bytes(p, T);
  return LCP_OK;
}

int lcp_sparse_linear_cut(const lcp_packed* w, int T, lcp_dtype y_dt, int32_t* cut) {
  PackedArgs p;
  const int rc = check_packed(w, &p);
  if (rc != LCP_OK) return rc;
  if (!cut || T <= 0) return LCP_E_INVAL;
  if (!float_type(y_dt)) return LCP_E_UNSUPPORTED;
  sparse_linear_cut(p, T, y_dt == LCP_F32, cut);
  return LCP_OK;
}

int lcp_sparse_linear(const lcp_packed* w, const void* x, int64_t x_row, const float* x_scale, int T,
                      const lcp_epilogue* e, void* y, int64_t y_row, lcp_dtype y_dt, void* ws, size_t ws_bytes,
                      void* stream) {
  LinearArgs a{};
  const int rc = check_packed(w, &a.w);
  if (rc != LCP_OK) return rc;
  if (T <= 0) return LCP_E_INVAL;
  if (!float_type(y_dt)) return LCP_E_UNSUPPORTED;
  const int64_t xe = a.w.fp8 ? 1 : 2, ye = (int64_t)esize(y_dt);
  if (!good_in(x, x_row, T, 16) || (T > 1 && x_row * xe % 16 != 0) || y == x) return LCP_E_INVAL;
  if (((int64_t)(T - 1) * x_row + w->cin) * xe >= ((int64_t)1 << 31)) return LCP_E_INVAL;
  if (a.w.fp8 && (!x_scale || !aligned(x_scale, 4))) return LCP_E_INVAL;
  if (!good_out(y, y_row, T, w->cout, 16) || (T > 1 && y_row * ye % 16 != 0)) return LCP_E_INVAL;
  Epilogue& p = a.e;
  if (e) {
    if (e->act < LCP_ACT_NONE || e->act > LCP_ACT_GELU_TANH) return LCP_E_UNSUPPORTED;
    p.act = e->act;
    if (e->bias && !aligned(e->bias, 16)) return LCP_E_INVAL;
    if (e->gate && (!good_in(e->gate, e->gate_row, T, 16) || (T > 1 && e->gate_row % 8 != 0) || e->gate == y))
      return LCP_E_INVAL;
    if (e->residual) {
      if (!float_type(e->residual_dt)) return LCP_E_UNSUPPORTED;
      const int64_t re = (int64_t)esize(e->residual_dt);
      if (!good_in(e->residual, e->residual_row, T, 16) || (T > 1 && e->residual_row * re % 16 != 0)) return LCP_E_INVAL;
      if (e->residual == y && (e->residual_dt != y_dt || !same_rows(y, y_row, e->residual, e->residual_row, T)))
        return LCP_E_INVAL;
      p.res = e->residual;
      p.res_row = e->residual_row;
      p.res_f32 = e->residual_dt == LCP_F32;
    }
    p.bias = (const uint16_t*)e->bias;
    p.gate = (const uint16_t*)e->gate;
    p.gate_row = e->gate_row;
  }
  const size_t need = sparse_linear_workspace_bytes(a.w, T);
  if (need > 0 && !ws) return LCP_E_INVAL;
  if (need > 0 && (!aligned(ws, 256) || ws_bytes < need)) return LCP_E_WORKSPACE;
  p.xscale = a.w.fp8 ? x_scale : nullptr;
  p.wscale = a.w.wscale;
  p.y = y;
  p.y_row = y_row;
  p.y_f32 = y_dt == LCP_F32;
  a.x = Mat{x, x_row};
  a.T = T;
  a.ws = (float*)ws;
  LCP_RUN(launch_sparse_linear(a, S(stream)));
  return LCP_OK;
}

}  // extern "C"
