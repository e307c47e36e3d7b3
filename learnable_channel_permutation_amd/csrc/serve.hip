// C ABI of the serving operators (lcp_rope*, lcp_kv_*, lcp_attn_decode*):
// argument validation. Every check runs before the first launch, so an error
// return means nothing was enqueued.
#include <math.h>

#include "../../include/lcp.h"
#include "serve.h"

using namespace lcp;

namespace {

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
inline bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }      // index arrays
inline hipStream_t S(void* s) { return reinterpret_cast<hipStream_t>(s); }
constexpr int64_t kMaxStride = (int64_t)1 << 40;
// Elements from one side of a tensor to the other along an axis: every offset and sum of offsets then stays inside 64 bits.
constexpr int64_t kMaxSpan = (int64_t)1 << 60;

// Input rows: pointer, head count and strides. Rows may share memory (a
// broadcast input has stride 0).
bool good_rows_in(const lcp_heads* h, int T) {
  return h->x && h->heads >= 1 && h->heads <= 65536 && h->x_token >= 0 && h->x_head >= 0 && h->x_token <= kMaxStride &&
         h->x_head <= kMaxStride && h->x_token <= kMaxSpan / T;
}
// Output rows must not overlap each other: either nesting of the two strides.
bool good_rows_out(const lcp_heads* h, int T, int D) {
  if (!h->y || h->y_token < 0 || h->y_head < 0 || h->y_token > kMaxStride || h->y_head > kMaxStride ||
      h->y_token > kMaxSpan / T)
    return false;
  const int64_t H = h->heads;
  if (h->y == h->x && (h->x_token != h->y_token || h->x_head != h->y_head) && !(T == 1 && h->x_head == h->y_head) &&
      !(H == 1 && h->x_token == h->y_token) && !(T == 1 && H == 1))
    return false;
  const bool token_major = (H == 1 || h->y_head >= D) && (T == 1 || h->y_token >= (H - 1) * h->y_head + D);
  const bool head_major = (T == 1 || h->y_token >= D) && (H == 1 || h->y_head >= (int64_t)(T - 1) * h->y_token + D);
  return token_major || head_major;
}
Rows rows_of(const lcp_heads* h) {
  return Rows{h->x, h->y, h->heads, h->x_token, h->x_head, h->y_token, h->y_head};
}

int check_cache(const lcp_kv_cache* c, KvCache* out) {
  if (!c || !c->k || !c->v || c->pages <= 0 || c->page_size <= 0 || c->heads <= 0 || c->D <= 0) return LCP_E_INVAL;
  if (c->format != LCP_KV_BF16 && c->format != LCP_KV_E4M3 && c->format != LCP_KV_INT8) return LCP_E_UNSUPPORTED;
  if (c->D != 64 && c->D != 128 && c->D != 256) return LCP_E_UNSUPPORTED;
  if (c->page_size % 16 != 0 || c->page_size > 4096 || c->heads > 65536) return LCP_E_UNSUPPORTED;
  if ((int64_t)c->pages * c->page_size >= ((int64_t)1 << 31)) return LCP_E_INVAL;
  if (!aligned16(c->k) || !aligned16(c->v) || c->k == c->v) return LCP_E_INVAL;
  const bool scaled = c->format != LCP_KV_BF16;
  if (scaled && (!c->k_scale || !c->v_scale || !aligned16(c->k_scale) || !aligned16(c->v_scale))) return LCP_E_INVAL;
  *out = KvCache{c->k, c->v, c->k_scale, c->v_scale, c->format, c->pages, c->page_size, c->heads, c->D};
  return LCP_OK;
}

int check_attn_sizes(const lcp_kv_cache* c, int B, int hq, int max_len, int window) {
  if (B <= 0 || hq <= 0 || max_len < 0 || window < 0) return LCP_E_INVAL;
  if (hq % c->heads != 0) return LCP_E_INVAL;
  if ((int64_t)B * hq * c->D >= ((int64_t)1 << 31) || max_len >= (1 << 28)) return LCP_E_INVAL;
  // steps of 32 tokens over all sequences and head tiles in 32 bits
  const int64_t units = (int64_t)B * c->heads * ((hq / c->heads + 15) / 16);
  if (units * ((int64_t)max_len / 32 + 10) >= ((int64_t)1 << 31)) return LCP_E_INVAL;
  if (units * 256 > kMaxThreads) return LCP_E_INVAL;           // a workgroup a unit
  return LCP_OK;
}

#define LCP_RUN(expr)                                                                             \
  do {                                                                                            \
    const hipError_t err = (expr);                                                                \
    if (err != hipSuccess) return err == hipErrorInvalidConfiguration ? LCP_E_INVAL : LCP_E_HIP; \
  } while (0)

}  // namespace

extern "C" {

int lcp_rope_table(const lcp_rope_cfg* rc, int max_pos, float* table, void* stream) {
  if (!rc || !table || max_pos <= 0 || !aligned16(table)) return LCP_E_INVAL;
  if (rc->rot_dim < 2 || rc->rot_dim % 2 != 0) return LCP_E_INVAL;
  if (rc->rot_dim > 1024) return LCP_E_UNSUPPORTED;
  if (!isfinite(rc->base) || !(rc->base > 1.0) || !isfinite(rc->magnitude) || !(rc->magnitude > 0.0)) return LCP_E_INVAL;
  switch (rc->scaling) {
    case LCP_ROPE_NONE: break;
    case LCP_ROPE_BY_PARTS:
      if (!isfinite(rc->orig_len) || !(rc->orig_len > 0.0) || !isfinite(rc->low_turns) || !isfinite(rc->high_turns) ||
          !(rc->low_turns < rc->high_turns))
        return LCP_E_INVAL;
      [[fallthrough]];
    case LCP_ROPE_BASE:
      if (rc->scaling == LCP_ROPE_BASE && rc->rot_dim <= 2) return LCP_E_INVAL;
      [[fallthrough]];
    case LCP_ROPE_LINEAR:
      if (!isfinite(rc->factor) || !(rc->factor >= 1.0)) return LCP_E_INVAL;
      break;
    default: return LCP_E_UNSUPPORTED;
  }
  if ((int64_t)max_pos * (rc->rot_dim / 2) >= ((int64_t)1 << 31)) return LCP_E_INVAL;
  const RopeFreq f{rc->rot_dim, rc->scaling, rc->base, rc->factor, rc->orig_len, rc->low_turns, rc->high_turns,
                   rc->magnitude};
  LCP_RUN(launch_rope_table(f, max_pos, (float2*)table, S(stream)));
  return LCP_OK;
}

int lcp_rope(const lcp_heads* q, const lcp_heads* k, lcp_dtype dt, int T, int D, const float* table, int max_pos,
             const int32_t* pos, int rot_dim, int interleaved, int inverse, void* stream) {
  if (!q || !table || !pos || T <= 0 || max_pos <= 0) return LCP_E_INVAL;
  if (dt != LCP_F32 && dt != LCP_BF16) return LCP_E_UNSUPPORTED;
  if (D < 2 || rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > D) return LCP_E_INVAL;
  if (D > 1024) return LCP_E_UNSUPPORTED;
  if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1) || !aligned16(table)) return LCP_E_INVAL;
  const uintptr_t es = dt == LCP_BF16 ? 1 : 3;
  for (const lcp_heads* h : {q, k}) {
    if (!h) continue;
    if (!good_rows_in(h, T) || !good_rows_out(h, T, D)) return LCP_E_INVAL;
    if (((uintptr_t)h->x & es) != 0 || ((uintptr_t)h->y & es) != 0) return LCP_E_INVAL;
  }
  const int64_t rows = (int64_t)T * (q->heads + (k ? k->heads : 0));
  if (rows >= ((int64_t)1 << 31)) return LCP_E_INVAL;
  if (!aligned4(pos)) return LCP_E_INVAL;
  RopeArgs a{};
  a.q = rows_of(q);
  if (k) a.k = rows_of(k);
  a.T = T; a.D = D; a.rot = rot_dim; a.max_pos = max_pos;
  a.interleaved = interleaved; a.inverse = inverse;
  a.table = (const float2*)table;
  a.pos = pos;
  LCP_RUN(launch_rope(a, dt == LCP_BF16, S(stream)));
  return LCP_OK;
}

int lcp_kv_append(const lcp_kv_cache* c, const lcp_heads* q, const lcp_heads* k, const lcp_heads* v, int T,
                  const int32_t* slots, const float* table, int max_pos, const int32_t* pos, int rot_dim,
                  int interleaved, void* stream) {
  KvAppendArgs a{};
  int rc = check_cache(c, &a.c);
  if (rc != LCP_OK) return rc;
  if (!k || !v || !slots || T <= 0 || !aligned4(slots)) return LCP_E_INVAL;
  if (!good_rows_in(k, T) || !good_rows_in(v, T) || k->heads != c->heads || v->heads != c->heads) return LCP_E_INVAL;
  if (((uintptr_t)k->x & 1) != 0 || ((uintptr_t)v->x & 1) != 0) return LCP_E_INVAL;
  if (q) {
    if (!table || !good_rows_in(q, T) || !good_rows_out(q, T, c->D)) return LCP_E_INVAL;
    if (((uintptr_t)q->x & 1) != 0 || ((uintptr_t)q->y & 1) != 0) return LCP_E_INVAL;
  }
  if (table) {
    if (!pos || max_pos <= 0 || !aligned4(pos) || !aligned16(table) || rot_dim <= 0 || rot_dim > c->D) return LCP_E_INVAL;
    if (interleaved != 0 && interleaved != 1) return LCP_E_INVAL;
    if (rot_dim % 16 != 0) return LCP_E_UNSUPPORTED;
  }
  if ((int64_t)T * ((q ? q->heads : 0) + 2 * (int64_t)c->heads) >= ((int64_t)1 << 31)) return LCP_E_INVAL;
  if (q) a.q = rows_of(q);
  a.k = Rows{k->x, nullptr, k->heads, k->x_token, k->x_head, 0, 0};       // their y is not used
  a.v = Rows{v->x, nullptr, v->heads, v->x_token, v->x_head, 0, 0};
  a.T = T;
  a.rot = table ? rot_dim : 0;
  a.max_pos = max_pos;
  a.interleaved = interleaved;
  a.slots = slots;
  a.table = (const float2*)table;
  a.pos = pos;
  LCP_RUN(launch_kv_append(a, S(stream)));
  return LCP_OK;
}

int lcp_kv_read(const lcp_kv_cache* c, const int32_t* slots, int T, void* k_out, void* v_out, lcp_dtype odt,
                void* stream) {
  KvCache kc;
  int rc = check_cache(c, &kc);
  if (rc != LCP_OK) return rc;
  if (!slots || T <= 0 || !aligned4(slots) || !k_out || !v_out || k_out == v_out) return LCP_E_INVAL;
  if (odt != LCP_F32 && odt != LCP_BF16) return LCP_E_UNSUPPORTED;
  if (!aligned16(k_out) || !aligned16(v_out)) return LCP_E_INVAL;
  LCP_RUN(launch_kv_read(kc, slots, T, k_out, v_out, odt == LCP_BF16, S(stream)));
  return LCP_OK;
}

int lcp_attn_decode_workspace_bytes(const lcp_kv_cache* c, int B, int hq, int max_len, int window, size_t* bytes) {
  KvCache kc;
  int rc = check_cache(c, &kc);
  if (rc != LCP_OK) return rc;
  if (!bytes) return LCP_E_INVAL;
  rc = check_attn_sizes(c, B, hq, max_len, window);
  if (rc != LCP_OK) return rc;
  *bytes = attn_workspace_bytes(kc, B, hq, max_len, window);
  return LCP_OK;
}

int lcp_attn_decode(const lcp_kv_cache* c, const void* q, int64_t q_row, int B, int hq, const int32_t* pages,
                    int max_pages, const int32_t* lens, int max_len, float scale, int window, void* out, lcp_dtype odt,
                    float* lse, void* ws, size_t ws_bytes, void* stream) {
  AttnArgs a{};
  int rc = check_cache(c, &a.c);
  if (rc != LCP_OK) return rc;
  if (!q || !pages || !lens || !out || max_pages <= 0 || !aligned4(pages) || !aligned4(lens)) return LCP_E_INVAL;
  rc = check_attn_sizes(c, B, hq, max_len, window);
  if (rc != LCP_OK) return rc;
  if (odt != LCP_F32 && odt != LCP_BF16) return LCP_E_UNSUPPORTED;
  if (!isfinite(scale) || (int64_t)max_len > (int64_t)max_pages * c->page_size) return LCP_E_INVAL;
  if ((int64_t)B * max_pages >= ((int64_t)1 << 31)) return LCP_E_INVAL;
  if (q_row < (int64_t)hq * c->D || q_row > kMaxStride || q_row % 8 != 0) return LCP_E_INVAL;
  if (!aligned16(q) || !aligned16(out) || ((uintptr_t)lse & 3) != 0) return LCP_E_INVAL;
  const size_t need = attn_workspace_bytes(a.c, B, hq, max_len, window);
  if (need > 0 && !ws) return LCP_E_INVAL;
  if (need > 0 && (((uintptr_t)ws & 255) != 0 || ws_bytes < need)) return LCP_E_WORKSPACE;
  a.q = (const uint16_t*)q;
  a.qrow = q_row;
  a.B = B;
  a.hq = hq;
  a.max_pages = max_pages;
  a.max_len = max_len;
  a.window = window;
  a.pages = pages;
  a.lens = lens;
  a.scale2 = (float)((double)scale * 1.4426950408889634);
  a.out = out;
  a.out_bf16 = odt == LCP_BF16;
  a.lse = lse;
  a.ws = (float*)ws;
  LCP_RUN(launch_attn_decode(a, S(stream)));
  return LCP_OK;
}

}  // extern "C"
