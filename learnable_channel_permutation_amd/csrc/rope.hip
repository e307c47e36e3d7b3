// Rotary positions: the table of cosines and sines, and the rotation of query
// and key rows (forward and transposed).
#include "../../include/lcp.h"
#include "serve.h"

namespace lcp {
namespace {

// One thread an entry, in 64 bits: an angle of p theta radians has no accurate
// fp32 form at large p. Written once and kept; the 64-bit functions bound it
// (131072 positions x 64 pairs, 67 MB: 95 us).
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
// and alignment. In place: a thread reads its pair before it writes it. Two-byte
// accesses bound it: 16384 tokens x 80 heads of 128 bf16 from an odd address 415
// us, where chunks of 8 bytes take 160 and of 16 bytes 119 (calls in a row).
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
  store(out, y + d0, rot_first(u, v, cs.x, s));
  store(out, y + d1, rot_second(u, v, cs.x, s));
}

// One thread per (token, head, unit). A unit is 2 V channels of a head row, V
// pairs: the chunks [V u, +V) and [V u + rot / 2, +V), in the half layout a
// pair's two channels; the unrotated channels are split alike. Adjacent lanes
// take adjacent chunks, so that every load and store of a wave covers whole
// lines (two adjacent chunks a lane measured 4 % slower, and 30 % with streaming
// stores). A thread reads both chunks before it writes them: in place needs
// nothing more. The bytes of the rows bound it; the table's rows, which all
// heads of a token share, come from the caches (a thread that kept its table
// entries for 2 or 4 heads was 0 - 8 % slower: fewer loads in flight).
// 16384 tokens x 80 heads of 128 bf16 (680 MB): one thread a pair 452 us, this
// 114 us = 6.0 TB/s; 8191 x 72, 306 MB: 184 -> 54 us = 5.7 TB/s.
template <typename E, int V, bool STREAM>
__global__ __launch_bounds__(256) void rope_units_kernel(RopeArgs a, int64_t n) {
  typedef RopeChunk<E, V> C;
  typedef typename C::T W;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= n) return;
  const int units = a.D / (2 * V), rotated = a.rot / (2 * V);
  const uint32_t per = (uint32_t)((a.q.heads + a.k.heads) * units);
  const int t = (int)(id / per);
  const uint32_t in = (uint32_t)(id - (int64_t)t * per);
  const int u = (int)(in % units);
  int h = (int)(in / units);
  const bool isk = h >= a.q.heads;
  if (isk) h -= a.q.heads;
  const Rows& r = isk ? a.k : a.q;
  const bool turn = u < rotated;
  const int d0 = turn ? V * u : a.rot + V * (u - rotated), d1 = d0 + (turn ? a.rot : a.D - a.rot) / 2;
  const E* x = (const E*)r.x + t * r.xt + h * r.xh;
  E* y = (E*)r.y + t * r.yt + h * r.yh;
  W w0 = load_as<STREAM, W>(x + d0), w1 = load_as<STREAM, W>(x + d1);
  if (turn) {
    const int p = min(max(a.pos[t], 0), a.max_pos - 1);
    // V pairs from d0 on, or half of them from each chunk
    const float2* tab = a.table + (int64_t)p * (a.rot / 2) + (a.interleaved ? d0 / 2 : d0);
    const int skip = a.interleaved ? (a.rot / 2 - V) / 2 : 0;
    float f[2 * V];
    C::unpack(w0, f);
    C::unpack(w1, f + V);
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      const floatx4 cs = *(const floatx4*)(tab + j + (j >= V / 2 ? skip : 0));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float& u0 = f[a.interleaved ? 2 * (j + i) : j + i];
        float& u1 = f[a.interleaved ? 2 * (j + i) + 1 : j + i + V];
        const float c = cs[2 * i], s = a.inverse ? -cs[2 * i + 1] : cs[2 * i + 1], p0 = u0, p1 = u1;
        u0 = rot_first(p0, p1, c, s);
        u1 = rot_second(p0, p1, c, s);
      }
    }
    w0 = C::pack(f);
    w1 = C::pack(f + V);
  }
  store_as<STREAM, W>(y + d0, w0);
  store_as<STREAM, W>(y + d1, w1);
}

template <typename E, int V>
hipError_t run_units(const RopeArgs& a, hipStream_t s) {
  const int64_t rows = (int64_t)a.T * (a.q.heads + a.k.heads), n = rows * (a.D / (2 * V)), grid = (n + 255) / 256;
  if (n > kMaxThreads) return hipErrorInvalidConfiguration;
  if (rows * a.D * 2 * (int64_t)sizeof(E) > kStreamBytes)
    rope_units_kernel<E, V, true><<<(unsigned)grid, 256, 0, s>>>(a, n);
  else
    rope_units_kernel<E, V, false><<<(unsigned)grid, 256, 0, s>>>(a, n);
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

hipError_t launch_rope(const RopeArgs& a, int bf16, hipStream_t s) {
  const auto fits = [&](int V, int e) {
    return a.D % (2 * V) == 0 && a.rot % (2 * V) == 0 && chunked(a.q, V, e) && chunked(a.k, V, e);
  };
  if (bf16 && fits(8, 2)) return run_units<uint16_t, 8>(a, s);
  if (bf16 && fits(4, 2)) return run_units<uint16_t, 4>(a, s);
  if (!bf16 && fits(4, 4)) return run_units<float, 4>(a, s);
  const int64_t n = (int64_t)a.T * (a.q.heads + a.k.heads) * (a.rot / 2 + a.D - a.rot);
  const int64_t grid = (n + 255) / 256;
  if (n > kMaxThreads) return hipErrorInvalidConfiguration;
  if (bf16) rope_pairs_kernel<uint16_t><<<(unsigned)grid, 256, 0, s>>>(a, n);
  else rope_pairs_kernel<float><<<(unsigned)grid, 256, 0, s>>>(a, n);
  return hipGetLastError();
}

}  // namespace lcp
