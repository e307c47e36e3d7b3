// Paged key/value cache: rotation, quantisation and writing of new tokens, and
// reading slots back.
#include "serve.h"

namespace lcp {
namespace {

// fp32 -> one e4m3 code (nearest even); |v| <= 448 or NaN
__device__ __forceinline__ uint32_t to_e4m3(float v) { return __builtin_amdgcn_cvt_pk_fp8_f32(v, v, 0, false) & 0xff; }
__device__ __forceinline__ float from_e4m3(uint32_t c) { return __builtin_amdgcn_cvt_f32_fp8((int)c, 0); }

// The rotation with two rounded products and one rounded sum, never a fused
// multiply-add: the 8-bit codes then follow from the definition in fp32 to the
// last bit, however this is compiled.
__device__ __forceinline__ float rot_first(float a, float b, float c, float s) {
#pragma clang fp contract(off)
  return a * c - b * s;
}
__device__ __forceinline__ float rot_second(float a, float b, float c, float s) {
#pragma clang fp contract(off)
  return b * c + a * s;
}

// Scale of a row with maximum magnitude bits `a` (the bits of max |x|; a NaN
// has the largest). Not finite: NaN.
__device__ __forceinline__ float row_scale(uint32_t a, int format) {
  if (a >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  if (format == KV_INT8) return fmaxf(__uint_as_float(a) / 127.f, 0x1p-126f);
  // a = m 2^k: 2^(k-8) while m <= 1.75, else 2^(k-7)
  int e = (int)(a >> 23) - 127 - 8 + ((a & 0x7fffffu) > 0x600000u);
  e = e < -126 ? -126 : e;
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// One wave per (token, head row): lane l holds channels l, l + 64, ..
__global__ __launch_bounds__(64) void kv_append_rows_kernel(KvAppendArgs a) {
  const int lane = threadIdx.x, rows = a.q.heads + 2 * a.c.heads;
  const int64_t id = blockIdx.x;
  const int t = (int)(id / rows);
  int h = (int)(id % rows);
  const int which = h < a.q.heads ? 0 : h < a.q.heads + a.c.heads ? 1 : 2;   // q, k, v
  const Rows& r = which == 0 ? a.q : which == 1 ? a.k : a.v;
  h -= which == 0 ? 0 : which == 1 ? a.q.heads : a.q.heads + a.c.heads;
  const uint16_t* x = (const uint16_t*)r.x + t * r.xt + h * r.xh;
  const int n = a.c.D / 64, half = a.rot / 2;
  const int p = a.rot ? min(max(a.pos[t], 0), a.max_pos - 1) : 0;
  float y[4];
  uint32_t top = 0;
  for (int i = 0; i < 4; ++i) {
    if (i >= n) break;
    const int d = lane + 64 * i;
    float v = bf2f(x[d]);
    if (which != 2 && d < a.rot) {
      const int pair = a.interleaved ? d / 2 : d % half;
      const bool second = a.interleaved ? d & 1 : d >= half;
      const int other = a.interleaved ? d ^ 1 : second ? d - half : d + half;
      const float2 cs = a.table[(int64_t)p * half + pair];
      const float w = bf2f(x[other]);
      v = second ? rot_second(w, v, cs.x, cs.y) : rot_first(v, w, cs.x, cs.y);
    }
    y[i] = v;
    top = max(top, __float_as_uint(v) & 0x7fffffffu);
  }
  if (which == 0) {
    uint16_t* out = (uint16_t*)r.y + t * r.yt + h * r.yh;
    for (int i = 0; i < 4; ++i)
      if (i < n) out[lane + 64 * i] = (uint16_t)f2bf(y[i]);
    return;
  }
  const int slot = a.slots[t];
  if (slot < 0 || slot >= a.c.pages * a.c.ps) return;
  const int64_t row = ((int64_t)(slot / a.c.ps) * a.c.heads + h) * a.c.ps + slot % a.c.ps;
  void* dst = which == 1 ? a.c.k : a.c.v;
  if (a.c.format == KV_BF16) {
    for (int i = 0; i < 4; ++i)
      if (i < n) ((uint16_t*)dst)[row * a.c.D + lane + 64 * i] = (uint16_t)f2bf(y[i]);
    return;
  }
  for (int m = 1; m < 64; m <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m, 64));
  const float s = row_scale(top, a.c.format);
  const bool ok = top < 0x7f800000u;
  for (int i = 0; i < 4; ++i) {
    if (i >= n) break;
    const float v = ok ? y[i] / s : 0.f;
    const uint32_t code = a.c.format == KV_E4M3 ? to_e4m3(v) : (uint32_t)(int)fminf(fmaxf(rintf(v), -127.f), 127.f);
    ((uint8_t*)dst)[row * a.c.D + lane + 64 * i] = (uint8_t)code;
  }
  if (lane == 0) (which == 1 ? a.c.ks : a.c.vs)[row] = s;
}

// One thread per element.
__global__ void kv_read_kernel(KvCache c, const int* slots, int64_t n, void* k, void* v, int bf16) {
  const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (id >= 2 * n) return;
  const bool isv = id >= n;
  const int64_t i = isv ? id - n : id;
  const int d = (int)(i % c.D);
  const int64_t th = i / c.D;
  const int h = (int)(th % c.heads), slot = slots[th / c.heads];
  float x = 0.f;
  if (slot >= 0 && slot < c.pages * c.ps) {
    const int64_t row = ((int64_t)(slot / c.ps) * c.heads + h) * c.ps + slot % c.ps;
    const void* src = isv ? c.v : c.k;
    if (c.format == KV_BF16) {
      x = bf2f(((const uint16_t*)src)[row * c.D + d]);
    } else {
      const uint8_t code = ((const uint8_t*)src)[row * c.D + d];
      x = c.format == KV_E4M3 ? from_e4m3(code) : (float)(int8_t)code;
      x *= (isv ? c.vs : c.ks)[row];
    }
  }
  void* dst = isv ? v : k;
  if (bf16) ((uint16_t*)dst)[i] = (uint16_t)f2bf(x);
  else ((float*)dst)[i] = x;
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t s) {
  const int64_t rows = (int64_t)a.T * (a.q.heads + 2 * a.c.heads);
  kv_append_rows_kernel<<<(unsigned)rows, 64, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvCache& c, const int* slots, int T, void* k, void* v, int bf16, hipStream_t s) {
  const int64_t n = (int64_t)T * c.heads * c.D;
  kv_read_kernel<<<(unsigned)((2 * n + 255) / 256), 256, 0, s>>>(c, slots, n, k, v, bf16);
  return hipGetLastError();
}

}  // namespace lcp
