// Rotary positions: the table of cosines and sines, and the rotation of query
// and key rows (forward and transposed).
#include "../../include/lcp.h"
#include "serve.h"

namespace lcp {
namespace {

__global__ void rope_table_kernel(RopeFreq f, int n, float2* table) {
  const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int half = f.rot / 2;
  if (id >= (int64_t)n * half) return;
  const int p = (int)(id / half), i = (int)(id % half);
  const double base = f.scaling == LCP_ROPE_BASE ? f.base * pow(f.factor, (double)f.rot / (f.rot - 2)) : f.base;
  double theta = pow(base, -2.0 * i / f.rot);
  if (f.scaling == LCP_ROPE_LINEAR) theta /= f.factor;
  if (f.scaling == LCP_ROPE_BY_PARTS) {
    const double turns = f.orig_len * theta / 6.283185307179586476925;
    const double g = fmin(fmax((turns - f.low) / (f.high - f.low), 0.0), 1.0);
    theta *= g + (1.0 - g) / f.factor;
  }
  double s, c;
  sincos(p * theta, &s, &c);
  table[id] = make_float2((float)(f.mag * c), (float)(f.mag * s));
}

template <typename E>
__device__ __forceinline__ float load(const void* p, int64_t i);
template <>
__device__ __forceinline__ float load<float>(const void* p, int64_t i) { return ((const float*)p)[i]; }
template <>
__device__ __forceinline__ float load<uint16_t>(const void* p, int64_t i) { return bf2f(((const uint16_t*)p)[i]); }
__device__ __forceinline__ void store(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void store(uint16_t* p, int64_t i, float v) { p[i] = (uint16_t)f2bf(v); }

// One thread per pair (or unrotated channel) of one head row; any size, stride
// and alignment. In place: a thread reads its pair before it writes it.
template <typename E>
__global__ void rope_pairs_kernel(RopeArgs a, int64_t n) {
  const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (id >= n) return;
  const int half = a.rot / 2, per = half + a.D - a.rot;
  const int i = (int)(id % per);
  const int64_t row = id / per;
  const int heads = a.q.heads + a.k.heads;
  const int t = (int)(row / heads);
  int h = (int)(row % heads);
  const bool isk = h >= a.q.heads;
  const Rows& r = isk ? a.k : a.q;
  if (isk) h -= a.q.heads;
  const int64_t x = t * r.xt + h * r.xh, y = t * r.yt + h * r.yh;
  E* out = (E*)r.y;
  if (i >= half) {
    const int d = i + half;
    out[y + d] = ((const E*)r.x)[x + d];
    return;
  }
  const int p = min(max(a.pos[t], 0), a.max_pos - 1);
  const float2 cs = a.table[(int64_t)p * half + i];
  const float s = a.inverse ? -cs.y : cs.y;
  const int d0 = a.interleaved ? 2 * i : i, d1 = a.interleaved ? 2 * i + 1 : i + half;
  const float u = load<E>(r.x, x + d0), v = load<E>(r.x, x + d1);
  store(out, y + d0, u * cs.x - v * s);
  store(out, y + d1, v * cs.x + u * s);
}

}  // namespace

hipError_t launch_rope_table(const RopeFreq& f, int max_pos, float2* table, hipStream_t s) {
  const int64_t n = (int64_t)max_pos * (f.rot / 2);
  rope_table_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(f, max_pos, table);
  return hipGetLastError();
}

hipError_t launch_rope(const RopeArgs& a, int bf16, hipStream_t s) {
  const int64_t n = (int64_t)a.T * (a.q.heads + a.k.heads) * (a.rot / 2 + a.D - a.rot);
  const int64_t grid = (n + 255) / 256;
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  if (bf16) rope_pairs_kernel<uint16_t><<<(unsigned)grid, 256, 0, s>>>(a, n);
  else rope_pairs_kernel<float><<<(unsigned)grid, 256, 0, s>>>(a, n);
  return hipGetLastError();
}

}  // namespace lcp
