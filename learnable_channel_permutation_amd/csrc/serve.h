// Serving operators of an attention block (rotary positions, paged key/value
// cache, one-token attention): arguments of their launchers. Validation is done
// by serve.hip before any launcher runs; every launcher enqueues on `s` and
// returns hipGetLastError().
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.h"

namespace lcp {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// V adjacent elements of a row: the word that is loaded and stored, and its fp32 values.
template <typename E, int V>
struct RopeChunk;
template <>
struct RopeChunk<uint16_t, 8> {
  typedef u32x4 T;
  static __device__ __forceinline__ void unpack(T w, float* f) {
#pragma unroll
    for (int j = 0; j < 4; ++j) { f[2 * j] = lo_bf(w[j]); f[2 * j + 1] = hi_bf(w[j]); }
  }
  static __device__ __forceinline__ T pack(const float* f) {
    return T{pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7])};
  }
};
template <>
struct RopeChunk<uint16_t, 4> {
  typedef u32x2 T;
  static __device__ __forceinline__ void unpack(T w, float* f) {
    f[0] = lo_bf(w[0]); f[1] = hi_bf(w[0]); f[2] = lo_bf(w[1]); f[3] = hi_bf(w[1]);
  }
  static __device__ __forceinline__ T pack(const float* f) { return T{pack2(f[0], f[1]), pack2(f[2], f[3])}; }
};
template <>
struct RopeChunk<float, 4> {
  typedef floatx4 T;
  static __device__ __forceinline__ void unpack(T w, float* f) {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = w[j];
  }
  static __device__ __forceinline__ T pack(const float* f) { return T{f[0], f[1], f[2], f[3]}; }
};

// The rotation of a pair (a, b) with two rounded products and one rounded sum, never
// a fused multiply-add: every kernel that rotates gives the same bits, and the 8-bit
// codes of keys follow from the definition in fp32, however this is compiled.
__device__ __forceinline__ float rot_first(float a, float b, float c, float s) {
#pragma clang fp contract(off)
  return a * c - b * s;
}
__device__ __forceinline__ float rot_second(float a, float b, float c, float s) {
#pragma clang fp contract(off)
  return b * c + a * s;
}

// Loads and stores of data that nobody finds in the caches again: a call that
// moves more than the 256 MB of the last-level cache hints them as streaming.
// Measured on the rotary kernel (72 heads of 128 bf16) with a kernel that reads
// its result, plain against hinted (us): 75 MB 30.2 / 30.2, 150 MB 53.5 / 54.8,
// 226 MB 79.6 / 77.5, 301 MB 106.7 / 99.8, 603 MB 197.7 / 191.9. Writing tokens into
// an fp8 cache and reading them back, with nobody to read the result: 2000 (82 +
// 49 MB) 32.4 / 29.0, 6000 82.3 / 74.0, 8000 (328 + 197 MB) 112 / 97, 16001 209 / 187.
constexpr int64_t kStreamBytes = (int64_t)256 << 20;
template <bool STREAM, typename T>
__device__ __forceinline__ T load_as(const void* p) {
  if (STREAM) return __builtin_nontemporal_load((const T*)p);
  return *(const T*)p;
}
template <bool STREAM, typename T>
__device__ __forceinline__ void store_as(void* p, T v) {
  if (STREAM) __builtin_nontemporal_store(v, (T*)p);
  else *(T*)p = v;
}

// A grid's threads are counted in 32 bits. A launcher whose call needs more returns
// hipErrorInvalidConfiguration and launches nothing.
constexpr int64_t kMaxThreads = ((int64_t)1 << 32) - 256;

// Head rows [T][heads][D] with strides in elements, input and output.
struct Rows {
  const void* x;
  void* y;
  int heads;
  int64_t xt, xh, yt, yh;
};

struct RopeArgs {
  Rows q, k;             // k.heads == 0: queries only
  int T, D, rot, max_pos;
  int interleaved, inverse;
  const float2* table;   // [max_pos][rot / 2] (cos, sin)
  const int* pos;
};
hipError_t launch_rope(const RopeArgs& a, int bf16, hipStream_t s);

struct RopeFreq {        // theta_i of the table, see lcp_rope_cfg
  int rot, scaling;
  double base, factor, orig_len, low, high, mag;
};
hipError_t launch_rope_table(const RopeFreq& f, int max_pos, float2* table, hipStream_t s);

enum KvFormat { KV_BF16 = 0, KV_E4M3 = 1, KV_INT8 = 2 };
struct KvCache {
  void *k, *v;           // [pages][heads][page_size][D]
  float *ks, *vs;        // [pages][heads][page_size]
  int format, pages, ps, heads, D;
};

struct KvAppendArgs {
  KvCache c;
  Rows q, k, v;          // bf16; q.heads == 0: no queries
  int T, rot, max_pos, interleaved;   // rot == 0: K stored as it is
  const int* slots;
  const float2* table;
  const int* pos;
};
hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t s);
hipError_t launch_kv_read(const KvCache& c, const int* slots, int T, void* k, void* v, int bf16, hipStream_t s);

struct AttnArgs {
  KvCache c;
  const uint16_t* q;     // [B][hq][D], qrow elements between sequences
  int64_t qrow;
  int B, hq, max_pages, max_len, window;
  const int* pages;
  const int* lens;
  float scale2;          // softmax scale x log2 e
  void* out;             // [B][hq][D]
  int out_bf16;
  float* lse;            // nullable
  float* ws;
};
size_t attn_workspace_bytes(const KvCache& c, int B, int hq, int max_len, int window);
hipError_t launch_attn_decode(const AttnArgs& a, hipStream_t s);

}  // namespace lcp
