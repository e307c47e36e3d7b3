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

// Items of the vector kernel: (token, group of heads, unit). A unit is 2 V
// channels of a head row, V pairs: the chunks [V u, +V) and [V u + rot / 2, +V)
// (half layout) or two adjacent chunks (interleaved and unrotated channels).
// A thread keeps its pairs' cosines and sines and applies them to the same
// unit of N heads, whose loads it issues together. It reads both chunks of a
// pair before it writes them, so in place needs nothing more.
// The bytes of the rows bound it. At 16384 tokens x 80 heads of 128 bf16
// (680 MB): one thread a pair 452 us (1.5 TB/s), see launch_rope for this one.
struct RopeItems {
  int gq, gk;            // groups of N heads of q and of k
  int units, rotated;    // units of a row, and those that are rotated
  int64_t n;             // items
};

template <typename E, int V, int N>
__global__ __launch_bounds__(256) void rope_units_kernel(RopeArgs a, RopeItems it) {
  typedef RopeChunk<E, V> C;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= it.n) return;
  const uint32_t per = (uint32_t)((it.gq + it.gk) * it.units);
  const int t = (int)(id / per);
  const uint32_t in = (uint32_t)(id - (int64_t)t * per);
  const int u = (int)(in % it.units);
  int h = (int)(in / it.units);
  const bool isk = h >= it.gq;
  if (isk) h -= it.gq;
  const Rows r = isk ? a.k : a.q;
  const int step = isk ? it.gk : it.gq;        // heads h, h + step, .. : neighbours in a wave are neighbours in memory
  const bool turn = u < it.rotated, split = turn && !a.interleaved;
  const int d0 = split ? V * u : 2 * V * u, d1 = split ? d0 + a.rot / 2 : d0 + V;
  const E* x = (const E*)r.x + t * r.xt;
  E* y = (E*)r.y + t * r.yt;
  typename C::T w0[N], w1[N];
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (h + i * step < r.heads) {
      const E* xi = x + (h + i * step) * r.xh;
      w0[i] = *(const typename C::T*)(xi + d0);
      w1[i] = *(const typename C::T*)(xi + d1);
    }
  float c[V], s[V];
  if (turn) {
    const int p = min(max(a.pos[t], 0), a.max_pos - 1);
    const floatx4* tab = (const floatx4*)(a.table + (int64_t)p * (a.rot / 2) + V * u);
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      const floatx4 q = tab[j];
      c[2 * j] = q[0]; c[2 * j + 1] = q[2];
      s[2 * j] = a.inverse ? -q[1] : q[1]; s[2 * j + 1] = a.inverse ? -q[3] : q[3];
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (h + i * step >= r.heads) break;
    if (turn) {
      float f[2 * V];
      C::unpack(w0[i], f);
      C::unpack(w1[i], f + V);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float& u0 = f[a.interleaved ? 2 * j : j];
        float& u1 = f[a.interleaved ? 2 * j + 1 : j + V];
        const float p = u0, q = u1;
        u0 = p * c[j] - q * s[j];
        u1 = q * c[j] + p * s[j];
      }
      w0[i] = C::pack(f);
      w1[i] = C::pack(f + V);
    }
    E* yi = y + (h + i * step) * r.yh;
    *(typename C::T*)(yi + d0) = w0[i];
    *(typename C::T*)(yi + d1) = w1[i];
  }
}

template <typename E, int V, int N>
hipError_t run_units(const RopeArgs& a, hipStream_t s) {
  RopeItems it{};
  it.gq = (a.q.heads + N - 1) / N;
  it.gk = (a.k.heads + N - 1) / N;
  it.units = a.D / (2 * V);
  it.rotated = a.rot / (2 * V);
  it.n = (int64_t)a.T * (it.gq + it.gk) * it.units;
  const int64_t grid = (it.n + 255) / 256;
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  rope_units_kernel<E, V, N><<<(unsigned)grid, 256, 0, s>>>(a, it);
  return hipGetLastError();
}

// Whether rows can be read and written in chunks of V elements of size e.
bool chunked(const Rows& r, int V, int e) {
  if (r.heads == 0) return true;
  const uintptr_t m = (uintptr_t)V * e - 1;
  return (((uintptr_t)r.x | (uintptr_t)r.y) & m) == 0 && (r.xt | r.xh | r.yt | r.yh) % V == 0;
}

}  // namespace

hipError_t launch_rope_table(const RopeFreq& f, int max_pos, float2* table, hipStream_t s) {
  const int64_t n = (int64_t)max_pos * (f.rot / 2);
  rope_table_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(f, max_pos, table);
  return hipGetLastError();
}

// Heads of a thread: 4 share one read of the table once that still leaves
// every CU work for several waves, else 1 (a decode step's rows are spread as
// wide as they go).
template <typename E, int V>
hipError_t run_vector(const RopeArgs& a, hipStream_t s) {
  const int64_t items = (int64_t)a.T * (a.q.heads + a.k.heads) * (a.D / (2 * V));
  return items >= (int64_t)4 * 256 * 1024 ? run_units<E, V, 4>(a, s) : run_units<E, V, 1>(a, s);
}

hipError_t launch_rope(const RopeArgs& a, int bf16, hipStream_t s) {
  const auto fits = [&](int V, int e) {
    return a.D % (2 * V) == 0 && a.rot % (2 * V) == 0 && chunked(a.q, V, e) && chunked(a.k, V, e);
  };
  if (bf16 && fits(8, 2)) return run_vector<uint16_t, 8>(a, s);
  if (bf16 && fits(4, 2)) return run_vector<uint16_t, 4>(a, s);
  if (!bf16 && fits(4, 4)) return run_vector<float, 4>(a, s);
  const int64_t n = (int64_t)a.T * (a.q.heads + a.k.heads) * (a.rot / 2 + a.D - a.rot);
  const int64_t grid = (n + 255) / 256;
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  if (bf16) rope_pairs_kernel<uint16_t><<<(unsigned)grid, 256, 0, s>>>(a, n);
  else rope_pairs_kernel<float><<<(unsigned)grid, 256, 0, s>>>(a, n);
  return hipGetLastError();
}

}  // namespace lcp
