// Paged key/value cache: rotation, quantisation and writing of new tokens, and
// reading slots back.
#include "serve.h"

namespace lcp {
namespace {

// fp32 -> one e4m3 code (nearest even); |v| <= 448 or NaN
__device__ __forceinline__ uint32_t to_e4m3(float v) { return __builtin_amdgcn_cvt_pk_fp8_f32(v, v, 0, false) & 0xff; }

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

// Rows that are not 16-byte aligned: one wave per (token, head row), lane l
// holds channels l, l + 64, .. and loads element by element, which bounds it
// (16001 tokens x 96 rows of 128: 660 us, aligned ones below 130).
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

// x / s rounded to the nearest fp32, with inv the rounded 1 / s: a product, its
// exact remainder and one correction (Markstein), while s is large enough for
// the remainder to be exact.
__device__ __forceinline__ float divided(float x, float s, float inv) {
  const float q = x * inv;
  return fmaf(fmaf(-q, s, x), inv, q);
}

// Largest magnitude (as bits) over the L adjacent lanes that hold a row.
template <int L>
__device__ __forceinline__ uint32_t row_top(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, false));
  if (L >= 8) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, false));
  if (L >= 16) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, false));
  return v;
}

// Eight fp32 numbers -> eight codes.
template <int FMT>
__device__ __forceinline__ uint2 encode8(const float* f, float s, float inv) {
  uint2 w;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (FMT == KV_E4M3) y[i] = f[4 * j + i] * inv;           // a power of two: exact
      else y[i] = s < 0x1p-100f ? f[4 * j + i] / s : divided(f[4 * j + i], s, inv);
    }
    if (FMT == KV_E4M3) {
      uint32_t r = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
      r = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], (int)r, true);
      (j ? w.y : w.x) = r;
    } else {
      uint32_t r = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        r |= ((uint32_t)(int)fminf(fmaxf(rintf(y[i]), -127.f), 127.f) & 0xffu) << (8 * i);
      (j ? w.y : w.x) = r;
    }
  }
  return w;
}

// One thread per (token, head row of q, k or v, unit). A unit is 16 channels of a
// row, two chunks of 8 chosen as in the rotary kernel; the D / 16 units of a row
// are adjacent lanes, which find its maximum among themselves, so that K is read,
// rotated, quantised and written in one pass. The bytes bound it: a row is read
// once and its codes written once. 16001 tokens x (32 + 32 + 32) heads of 128,
// fp8 (655 MB), with the read back of 20097 slots (494 MB): one wave a row and one
// thread an element 1320 us, these two kernels 207 us = 5.6 TB/s.
template <int FMT, int D, bool STREAM>
__global__ __launch_bounds__(256) void kv_append_kernel(KvAppendArgs a, int64_t n) {
  typedef RopeChunk<uint16_t, 8> C;
  constexpr int U = D / 16;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= n) return;                         // n is a multiple of U: rows leave whole
  const uint32_t per = (uint32_t)((a.q.heads + 2 * a.c.heads) * U);
  const int t = (int)(id / per);
  const uint32_t in = (uint32_t)(id - (int64_t)t * per);
  const int u = (int)(in % U);
  int h = (int)(in / U);
  const int which = h < a.q.heads ? 0 : h < a.q.heads + a.c.heads ? 1 : 2;   // q, k, v
  h -= which == 0 ? 0 : which == 1 ? a.q.heads : a.q.heads + a.c.heads;
  const Rows& r = which == 0 ? a.q : which == 1 ? a.k : a.v;
  // V, and rows that are not rotated, have no pairs and split at D / 2
  const int rot = which == 2 ? 0 : a.rot;
  const bool turn = 16 * u < rot;
  const int d0 = turn ? 8 * u : rot + 8 * (u - rot / 16), d1 = d0 + (turn ? rot : D - rot) / 2;
  const uint16_t* x = (const uint16_t*)r.x + t * r.xt + h * r.xh;
  const u32x4 w0 = load_as<STREAM, u32x4>(x + d0), w1 = load_as<STREAM, u32x4>(x + d1);
  float f[16];
  C::unpack(w0, f);
  C::unpack(w1, f + 8);
  if (turn) {
    const int p = min(max(a.pos[t], 0), a.max_pos - 1);
    const float2* tab = a.table + (int64_t)p * (rot / 2) + (a.interleaved ? d0 / 2 : d0);
    const int skip = a.interleaved ? (rot / 2 - 8) / 2 : 0;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const floatx4 cs = *(const floatx4*)(tab + j + (j >= 4 ? skip : 0));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float& y0 = f[a.interleaved ? 2 * (j + i) : j + i];
        float& y1 = f[a.interleaved ? 2 * (j + i) + 1 : j + i + 8];
        const float p0 = y0, p1 = y1;
        y0 = rot_first(p0, p1, cs[2 * i], cs[2 * i + 1]);
        y1 = rot_second(p0, p1, cs[2 * i], cs[2 * i + 1]);
      }
    }
  }
  if (which == 0) {
    uint16_t* y = (uint16_t*)r.y + t * r.yt + h * r.yh;
    store_as<STREAM, u32x4>(y + d0, C::pack(f));
    store_as<STREAM, u32x4>(y + d1, C::pack(f + 8));
    return;
  }
  const int slot = a.slots[t];
  if (slot < 0 || slot >= a.c.pages * a.c.ps) return;          // a row's lanes together
  const int page = slot / a.c.ps;
  const int64_t row = ((int64_t)page * a.c.heads + h) * a.c.ps + (slot - page * a.c.ps);
  char* dst = (char*)(which == 1 ? a.c.k : a.c.v);
  if (FMT == KV_BF16) {
    *(u32x4*)(dst + (row * D + d0) * 2) = C::pack(f);
    *(u32x4*)(dst + (row * D + d1) * 2) = C::pack(f + 8);
    return;
  }
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) top = max(top, __float_as_uint(f[j]) & 0x7fffffffu);
  top = row_top<U>(top);
  const float sc = row_scale(top, FMT), inv = 1.f / sc;
  uint2 c0 = encode8<FMT>(f, sc, inv), c1 = encode8<FMT>(f + 8, sc, inv);
  if (top >= 0x7f800000u) c0 = c1 = make_uint2(0u, 0u);
  *(uint2*)(dst + row * D + d0) = c0;          // the halves of a line come by different stores: not streamed
  *(uint2*)(dst + row * D + d1) = c1;
  if (u == 0) (which == 1 ? a.c.ks : a.c.vs)[row] = sc;
}

// One thread per eight channels of a slot and head, K and V: one 16-byte store of
// each (bf16), whole lines of both sides by adjacent lanes. The bytes bound it:
// 20097 slots x 32 heads of 128, fp8 to bf16 (499 MB), 91 us = 5.5 TB/s; to fp32, in two
// 16-byte stores a lane (828 MB), 169 us = 4.9 TB/s.
template <int FMT, bool BF, bool STREAM>
__global__ __launch_bounds__(256) void kv_read_kernel(KvCache c, const int* slots, int64_t n, char* ko, char* vo) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= n) return;
  const uint32_t U = c.D / 8, per = U * c.heads;
  const int t = (int)(id / per);
  const uint32_t in = (uint32_t)(id - (int64_t)t * per);
  const int d = (int)(in % U) * 8, h = (int)(in / U), slot = slots[t];
  float f[2][8] = {};
  if (slot >= 0 && slot < c.pages * c.ps) {
    const int page = slot / c.ps;
    const int64_t row = ((int64_t)page * c.heads + h) * c.ps + (slot - page * c.ps);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const char* src = (const char*)(i ? c.v : c.k);
      if (FMT == KV_BF16) {
        RopeChunk<uint16_t, 8>::unpack(load_as<STREAM, u32x4>(src + (row * c.D + d) * 2), f[i]);
      } else {
        const u32x2 w = load_as<STREAM, u32x2>(src + row * c.D + d);
        const float s = (i ? c.vs : c.ks)[row];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int word = (int)w[j >> 2];
          if (FMT == KV_INT8) f[i][j] = (float)(int8_t)(word >> (8 * (j & 3)));
        }
        if (FMT == KV_E4M3) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int word = (int)w[j];
            const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(word, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(word, true);
            f[i][4 * j] = a[0]; f[i][4 * j + 1] = a[1]; f[i][4 * j + 2] = b[0]; f[i][4 * j + 3] = b[1];
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) f[i][j] *= s;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    char* dst = i ? vo : ko;
    if (BF) {
      store_as<STREAM, u32x4>(dst + id * 16, RopeChunk<uint16_t, 8>::pack(f[i]));
    } else {
      store_as<STREAM, floatx4>(dst + id * 32, floatx4{f[i][0], f[i][1], f[i][2], f[i][3]});
      store_as<STREAM, floatx4>(dst + id * 32 + 16, floatx4{f[i][4], f[i][5], f[i][6], f[i][7]});
    }
  }
}

template <int FMT, int D>
hipError_t run_append(const KvAppendArgs& a, hipStream_t s) {
  const int64_t rows = (int64_t)a.T * (a.q.heads + 2 * a.c.heads), n = rows * (D / 16), grid = (n + 255) / 256;
  if (n > kMaxThreads) return hipErrorInvalidConfiguration;
  const int64_t q = (int64_t)a.T * a.q.heads * D * 4, kv = (int64_t)a.T * a.c.heads * 2 * D * (FMT == KV_BF16 ? 4 : 3);
  if (q + kv > kStreamBytes) kv_append_kernel<FMT, D, true><<<(unsigned)grid, 256, 0, s>>>(a, n);
  else kv_append_kernel<FMT, D, false><<<(unsigned)grid, 256, 0, s>>>(a, n);
  return hipGetLastError();
}

template <int FMT>
hipError_t run_append_d(const KvAppendArgs& a, hipStream_t s) {
  if (a.c.D == 64) return run_append<FMT, 64>(a, s);
  if (a.c.D == 128) return run_append<FMT, 128>(a, s);
  return run_append<FMT, 256>(a, s);
}

template <int FMT, bool BF>
hipError_t run_read(const KvCache& c, const int* slots, int T, void* k, void* v, hipStream_t s) {
  const int64_t n = (int64_t)T * c.heads * (c.D / 8), grid = (n + 255) / 256;
  if (n > kMaxThreads) return hipErrorInvalidConfiguration;
  const bool stream = n * 16 * ((FMT == KV_BF16 ? 2 : 1) + (BF ? 2 : 4)) > kStreamBytes;
  if (stream) kv_read_kernel<FMT, BF, true><<<(unsigned)grid, 256, 0, s>>>(c, slots, n, (char*)k, (char*)v);
  else kv_read_kernel<FMT, BF, false><<<(unsigned)grid, 256, 0, s>>>(c, slots, n, (char*)k, (char*)v);
  return hipGetLastError();
}

template <int FMT>
hipError_t run_read_bf(const KvCache& c, const int* slots, int T, void* k, void* v, int bf16, hipStream_t s) {
  return bf16 ? run_read<FMT, true>(c, slots, T, k, v, s) : run_read<FMT, false>(c, slots, T, k, v, s);
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t s) {
  const auto aligned = [](const Rows& r) {
    return r.heads == 0 || ((((uintptr_t)r.x | (uintptr_t)r.y) & 15) == 0 && (r.xt | r.xh | r.yt | r.yh) % 8 == 0);
  };
  if (!aligned(a.q) || !aligned(a.k) || !aligned(a.v)) {
    const int64_t rows = (int64_t)a.T * (a.q.heads + 2 * a.c.heads);
    if (rows * 64 > kMaxThreads) return hipErrorInvalidConfiguration;
    kv_append_rows_kernel<<<(unsigned)rows, 64, 0, s>>>(a);
    return hipGetLastError();
  }
  if (a.c.format == KV_BF16) return run_append_d<KV_BF16>(a, s);
  if (a.c.format == KV_E4M3) return run_append_d<KV_E4M3>(a, s);
  return run_append_d<KV_INT8>(a, s);
}

hipError_t launch_kv_read(const KvCache& c, const int* slots, int T, void* k, void* v, int bf16, hipStream_t s) {
  if (c.format == KV_BF16) return run_read_bf<KV_BF16>(c, slots, T, k, v, bf16, s);
  if (c.format == KV_E4M3) return run_read_bf<KV_E4M3>(c, slots, T, k, v, bf16, s);
  return run_read_bf<KV_INT8>(c, slots, T, k, v, bf16, s);
}

}  // namespace lcp
