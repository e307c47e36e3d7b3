// Root-mean-square norm with the residual's addition, a layer's channel order and
// an 8-bit output, and its gradient.
//
//   h = x + residual,  y = h s weight,  s = (mean h^2 + eps)^(-1/2)
//   n = h s,  g = dy weight,  dx = s (g - n mean(g n)) + dsum,  dweight = sum dy n
//
// A few flops an element: the bytes bound both. A workgroup takes a row at a time,
// NT threads with NV chunks of 16 bytes each, in registers from the loads to the
// stores, so that every input is read once; the next row's loads fly during this
// one's sums. The weight (and the gather's places) are loaded once a workgroup.
#include "block.h"

namespace lcp {
namespace {

// Rows begin anywhere that their element type may: the hardware takes wide loads and
// stores at any address, and only lines that a piece straddles are touched twice.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32_any __attribute__((aligned(1)));
typedef floatx4 f32x4_any __attribute__((aligned(4)));

template <typename XT>
constexpr int kChunk = 16 / sizeof(XT);        // elements of a chunk

template <typename XT>
__device__ __forceinline__ float element(const void* p, int64_t i) {
  if constexpr (sizeof(XT) == 2) return bf2f(((const uint16_t*)p)[i]);
  else return ((const float*)p)[i];
}

// Rows are the same for a whole workgroup and places in them unsigned, so that an
// address is a scalar base and a 32-bit offset.
template <typename XT>
__device__ __forceinline__ const void* row_at(const Mat& m, int64_t t) {
  return (const XT*)m.p + t * m.row;
}
__device__ __forceinline__ void* row_at(const MatOut& m, int64_t t, int size) {
  return (char*)m.p + t * m.row * size;
}

// Calls that move more than the last-level cache's 256 MB hint what they touch as
// streaming: 16384 x 5120 bf16 with residual and e4m3 output, 587 MB, 106 -> 100 us.
template <bool STREAM, typename T>
__device__ __forceinline__ T load_hint(const T* p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(p);
  else return *p;
}
template <bool STREAM, typename T, typename U>
__device__ __forceinline__ void store_hint(U* p, T v) {
  if constexpr (STREAM) __builtin_nontemporal_store((U)v, p);
  else *p = v;
}

// Elements c .. of a row; those from C on are 0.
template <typename XT, bool STREAM>
__device__ __forceinline__ u32x4 load_chunk(const void* row, uint32_t c, uint32_t C) {
  const XT* q = (const XT*)row + c;
  if (c + kChunk<XT> <= C) return load_hint<STREAM>((const u32x4_any*)q);
  u32x4 w = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < kChunk<XT>; ++i)
    if (c + i < C) {
      if constexpr (sizeof(XT) == 2) w[i / 2] |= (uint32_t)q[i] << (16 * (i & 1));
      else w[i] = __float_as_uint(q[i]);
    }
  return w;
}
template <typename XT>
__device__ __forceinline__ void unpack(u32x4 w, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(XT) == 2) { f[2 * i] = lo_bf(w[i]); f[2 * i + 1] = hi_bf(w[i]); }
    else f[i] = __uint_as_float(w[i]);
  }
}
// V numbers to elements c .. of a row of bf16 (two a word) or fp32.
template <int V, bool STREAM>
__device__ __forceinline__ void store_bf16(void* row, uint32_t c, uint32_t C, const uint32_t* w) {
  uint16_t* q = (uint16_t*)row + c;
  if (c + V <= C) {
    if constexpr (V == 8) store_hint<STREAM>((u32x4_any*)q, u32x4{w[0], w[1], w[2], w[3]});
    else store_hint<STREAM>((u32x2_any*)q, u32x2_any{w[0], w[1]});
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (c + i < C) q[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
}
template <int V, bool STREAM>
__device__ __forceinline__ void store_bf16(void* row, uint32_t c, uint32_t C, const float* f) {
  uint32_t w[V / 2];
#pragma unroll
  for (int i = 0; i < V / 2; ++i) w[i] = pack2(f[2 * i], f[2 * i + 1]);
  store_bf16<V, STREAM>(row, c, C, w);
}
template <int V, bool STREAM>
__device__ __forceinline__ void store_f32(void* row, uint32_t c, uint32_t C, const float* f) {
  float* q = (float*)row + c;
  if (c + V <= C) {
#pragma unroll
    for (int i = 0; i < V; i += 4) store_hint<STREAM>((f32x4_any*)(q + i), floatx4{f[i], f[i + 1], f[i + 2], f[i + 3]});
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (c + i < C) q[i] = f[i];
}
template <typename XT, bool STREAM>
__device__ __forceinline__ void store_as(void* row, uint32_t c, uint32_t C, const float* f) {
  if constexpr (sizeof(XT) == 2) store_bf16<kChunk<XT>, STREAM>(row, c, C, f);
  else store_f32<kChunk<XT>, STREAM>(row, c, C, f);
}
// e4m3 codes of V numbers of at most 448, four a word.
template <int V>
__device__ __forceinline__ void e4m3_codes(const float* f, uint32_t* w) {
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i], f[4 * i + 1], 0, false);
    w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i + 2], f[4 * i + 3], (int)w[i], true);
  }
}
template <int V, bool STREAM>
__device__ __forceinline__ void store_e4m3(void* row, uint32_t c, uint32_t C, const uint32_t* w) {
  uint8_t* q = (uint8_t*)row + c;
  if (c + V <= C) {
    if constexpr (V == 8) store_hint<STREAM>((u32x2_any*)q, u32x2_any{w[0], w[1]});
    else store_hint<STREAM>((u32_any*)q, w[0]);
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (c + i < C) q[i] = (uint8_t)(w[i / 4] >> (8 * (i & 3)));
}

// A layer's channel order, on elements as they are stored (rounding and permuting may be
// swapped): V of E in the words w to LDS at their own places, and back from the places `from`, two
// a register. A block of at most 128 channels lies within the 64 V elements of a wave's
// chunk, so that nothing waits for another wave. A lane's reads are random places of its
// block: the smaller the elements, the more of them share a bank's word (16384 x 5120 to e4m3 in fp32
// 110 us, in codes 100; without an order 98. 33 x 8192 5.8 and 4.7).
template <typename E, int V>
__device__ __forceinline__ void to_order(unsigned char* lds, uint32_t c, const uint32_t* w) {
  constexpr int N = V * sizeof(E) / 4;
  typedef uint32_t Words __attribute__((ext_vector_type(N > 4 ? 4 : N), may_alias));
  if constexpr (N == 1) {
    *(Words*)(lds + c * sizeof(E)) = w[0];
  } else {
#pragma unroll
    for (int i = 0; i < N; i += (N > 4 ? 4 : N)) {
      Words v;
#pragma unroll
      for (int j = 0; j < (N > 4 ? 4 : N); ++j) v[j] = w[i + j];
      *(Words*)(lds + c * sizeof(E) + 4 * i) = v;
    }
  }
}
template <typename E, int V>
__device__ __forceinline__ void in_order(const unsigned char* lds, const uint32_t* from, uint32_t* w) {
  constexpr int K = 4 / sizeof(E);             // elements a word
  typedef E E_ __attribute__((may_alias));
#pragma unroll
  for (int i = 0; i < V / K; ++i) w[i] = 0;
#pragma unroll
  for (int j = 0; j < V; j += 2) {
    uint32_t two = from[j / 2];
    asm volatile("" : "+v"(two));              // the addresses of all rows are the same, but not worth the registers
    w[j / K] |= (uint32_t)((const E_*)lds)[two & 0xffffu] << (8 * sizeof(E) * (j % K));
    w[(j + 1) / K] |= (uint32_t)((const E_*)lds)[two >> 16] << (8 * sizeof(E) * ((j + 1) % K));
  }
}

// V weights from c on as fp32.
template <int V>
__device__ __forceinline__ void load_weights(const void* p, int type, uint32_t c, uint32_t C, float* w) {
  if (c + V <= C) {
    if (type == T_BF16) {
      if constexpr (V == 8) {
        unpack<uint16_t>(*(const u32x4_any*)((const uint16_t*)p + c), w);
      } else {
        const u32x2_any b = *(const u32x2_any*)((const uint16_t*)p + c);
        w[0] = lo_bf(b[0]); w[1] = hi_bf(b[0]); w[2] = lo_bf(b[1]); w[3] = hi_bf(b[1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const floatx4 f = *(const f32x4_any*)((const float*)p + c + i);
        w[i] = f[0]; w[i + 1] = f[1]; w[i + 2] = f[2]; w[i + 3] = f[3];
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    w[i] = 0.f;
    if (c + i < C) w[i] = type == T_BF16 ? element<uint16_t>(p, c + i) : element<float>(p, c + i);
  }
}

__device__ __forceinline__ float wave_sum(float v) { return xor32_sum(xor16_sum(row16_sum(v))); }
// Largest of a wave's magnitudes as unsigned numbers, a NaN above all, without a trip
// through LDS (six of those, one after the other, took as long as the row's loads).
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  const auto step = [](uint32_t v, uint32_t o) { return v > o ? v : o; };
  v = step(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, false));
  v = step(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, false));
  v = step(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, false));
  v = step(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, false));
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = step(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return step(b[0], b[1]);
}
// The waves' parts in LDS, added in order.
template <int W>
__device__ __forceinline__ float sum_of(const float* p) {
  float v = p[0];
#pragma unroll
  for (int i = 1; i < W; ++i) v += p[i];
  return v;
}

// The factor s from a row's sum of squares. Where that passed fp32's range, h is scaled by
// 2^-96 for it: the sum then has a square of 1e17 2^-96 or more, of 2^64 at most, and
// eps is nothing beside it. Where eps is subnormal and the sum small enough for the squares'
// lost bits to count beside it, h is scaled by 2^64: eps is then 2^-21 or more. The factor
// that meets the row is the unscaled one: it is subnormal, and keeps 21 bits of 24, only
// where the mean square passes 2^252.
__device__ __forceinline__ float factor(float ss, int C, float eps) { return 1.f / sqrtf(ss / (float)C + eps); }
// The root of the scaling for a row whose plain sum of squares is ss: 1 for none.
__device__ __forceinline__ float scaling_root(float ss, float eps) {
  if (!(ss < __builtin_inff())) return 0x1p-48f;
  return eps < 0x1p-126f && ss < 0x1p-80f ? 0x1p32f : 1.f;
}
// The factor of a row scaled by root^2 (its sum of squares ss), over root.
__device__ __forceinline__ float scaled_factor(float ss, int C, float eps, float root) {
  return factor(ss, C, root > 1.f ? eps * root * root * root * root : 0.f) * root;
}

// What the registers hold besides a thread's elements (1024 threads leave 128 of them):
// HELD, the weights, which rows of more than 16384 elements read again; AHEAD, the next
// row.
template <typename XT, int NT, int NV, bool STREAM>
__global__ __launch_bounds__(NT) void norm_kernel(NormArgs a) {
  constexpr int V = kChunk<XT>, W = NT / 64;
  constexpr bool HELD = NV * V <= 16, AHEAD = HELD;
  extern __shared__ __attribute__((aligned(16))) unsigned char row_[];       // a row to be permuted, as it is stored
  __shared__ float part[2][W];                 // two rows in turn: a row's parts are read while the next one's come
  __shared__ uint32_t tops[W];
  const uint32_t tid = threadIdx.x, wave = tid >> 6, C = a.C;
  const bool more = a.res.p != nullptr, e4m3 = a.yt == T_E4M3;
  float w[HELD ? NV : 1][V];
  uint32_t from[NV][V / 2];                    // places that the outputs come from, two a register
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t c = (i * NT + tid) * V;
    if (HELD) load_weights<V>(a.w, a.wt, c, C, w[i]);
    if (a.B && c < C) {
      const uint32_t b = (uint32_t)(c & -a.B) * 0x10001u, m = (uint32_t)(a.B - 1);
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        const u32x4_any p = *(const u32x4_any*)(a.perm + c + j);
        from[i][j / 2] = b + ((p[0] & m) | (p[1] & m) << 16);
        from[i][j / 2 + 1] = b + ((p[2] & m) | (p[3] & m) << 16);
      }
    }
  }
  u32x4 nx[NV], nr[NV];
  auto load = [&](int64_t t) {
    const void *x = row_at<XT>(a.x, t), *r = more ? row_at<XT>(a.res, t) : nullptr;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t c = (i * NT + tid) * V;
      if (c < C) nx[i] = load_chunk<XT, STREAM>(x, c, C);
    }
    if (more) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const uint32_t c = (i * NT + tid) * V;
        if (c < C) nr[i] = load_chunk<XT, STREAM>(r, c, C);
      }
    }
  };
  if (AHEAD) load(blockIdx.x);
  int turn = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
    if (!AHEAD) load(t);
    float h[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t c = (i * NT + tid) * V;
      if (c < C) {
        unpack<XT>(nx[i], h[i]);
        if (more) {
          float r[V];
          unpack<XT>(nr[i], r);
#pragma unroll
          for (int j = 0; j < V; ++j) h[i][j] += r[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) h[i][j] = 0.f;
      }
    }
    if (AHEAD && t + gridDim.x < a.T) load(t + gridDim.x);
    auto squares = [&](float by) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) { const float v = h[i][j] * by; ss = fmaf(v, v, ss); }
      ss = wave_sum(ss);
      if ((tid & 63) == 0) part[turn][wave] = ss;
      __syncthreads();
      return sum_of<W>(part[turn]);
    };
    float ss = squares(1.f), s = factor(ss, a.C, a.eps);
    if (a.sum.p) {
      void* sum = row_at(a.sum, t, sizeof(XT));
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const uint32_t c = (i * NT + tid) * V;
        if (c < C) store_as<XT, STREAM>(sum, c, C, h[i]);
      }
    }
    const float root = scaling_root(ss, a.eps);
    if (root != 1.f) {                         // the same for the whole workgroup
      __syncthreads();
      s = scaled_factor(squares(root * root), a.C, a.eps, root) * root;
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!HELD) {
        __builtin_amdgcn_sched_barrier(0);     // a chunk's weights at a time
        load_weights<V>(a.w, a.wt, (i * NT + tid) * V, C, w[0]);
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        h[i][j] = h[i][j] * s * w[HELD ? i : 0][j];
        top = max(top, __float_as_uint(h[i][j]) & 0x7fffffffu);
      }
    }
    void* y = row_at(a.y, t, a.yt == T_E4M3 ? 1 : a.yt == T_BF16 ? 2 : 4);
    // the outputs' words w(i) of E, permuted if the layer asks for it; rows of a layer end with whole chunks
    auto finish = [&](auto element, auto words, auto store) {
      typedef decltype(element) E;
      constexpr int N = V * sizeof(E) / 4;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const uint32_t c = (i * NT + tid) * V;
        if (c >= C) continue;
        uint32_t w[N];
        words(h[i], w);
        if (a.B) to_order<E, V>(row_, c, w);
        else store(c, w);
      }
      if (!a.B) return;
      wave_fence();
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const uint32_t c = (i * NT + tid) * V;
        if (c >= C) continue;
        uint32_t w[N];
        in_order<E, V>(row_, from[i], w);
        store(c, w);
      }
      wave_fence();
    };
    if (e4m3) {
      top = wave_max(top);
      if ((tid & 63) == 0) tops[wave] = top;
      __syncthreads();
      top = tops[0];
#pragma unroll
      for (int i = 1; i < W; ++i) top = max(top, tops[i]);
      const float sc = e4m3_scale(top), inv = 1.f / sc;        // a power of two: the products below are exact
      if (tid == 0) a.scale[t] = sc;
      finish(
          uint8_t{},
          [&](float* f, uint32_t* w) {
#pragma unroll
            for (int j = 0; j < V; ++j) f[j] = top < 0x7f800000u ? f[j] * inv : 0.f;
            e4m3_codes<V>(f, w);
          },
          [&](uint32_t c, const uint32_t* w) { store_e4m3<V, STREAM>(y, c, C, w); });
    } else if (a.yt == T_BF16) {
      finish(
          uint16_t{},
          [&](const float* f, uint32_t* w) {
#pragma unroll
            for (int j = 0; j < V / 2; ++j) w[j] = pack2(f[2 * j], f[2 * j + 1]);
          },
          [&](uint32_t c, const uint32_t* w) { store_bf16<V, STREAM>(y, c, C, w); });
    } else {
      finish(
          uint32_t{},
          [&](const float* f, uint32_t* w) {
#pragma unroll
            for (int j = 0; j < V; ++j) w[j] = __float_as_uint(f[j]);
          },
          [&](uint32_t c, const uint32_t* w) {
            float f[V];
#pragma unroll
            for (int j = 0; j < V; ++j) f[j] = __uint_as_float(w[j]);
            store_f32<V, STREAM>(y, c, C, f);
          });
    }
  }
}

// The gradient: dx row by row as above, with the weight's gradient of the
// workgroup's rows in registers; it leaves them as a row of the workspace.
template <typename XT, int NT, int NV, bool STREAM>
__global__ __launch_bounds__(NT) void norm_grad_kernel(NormGradArgs a) {
  constexpr int V = kChunk<XT>, W = NT / 64;
  constexpr bool HELD = NV * V <= 16, AHEAD = HELD && NT < 1024, LATE = !HELD;
  __shared__ float part[2][2][W];
  const uint32_t tid = threadIdx.x, wave = tid >> 6, C = a.C;
  const bool more = a.dsum.p != nullptr;
  float w[HELD ? NV : 1][V], dw[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (HELD) load_weights<V>(a.w, a.wt, (i * NT + tid) * V, C, w[i]);
#pragma unroll
    for (int j = 0; j < V; ++j) dw[i][j] = 0.f;
  }
  u32x4 nh[NV], ny[NV], ns[NV];
  auto load = [&](int64_t t) {
    const void *h = row_at<XT>(a.h, t), *dy = row_at<XT>(a.dy, t), *ds = more ? row_at<XT>(a.dsum, t) : nullptr;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t c = (i * NT + tid) * V;
      nh[i] = ny[i] = u32x4{0, 0, 0, 0};
      if (c < C) {
        nh[i] = load_chunk<XT, STREAM>(h, c, C);
        ny[i] = load_chunk<XT, STREAM>(dy, c, C);
      }
    }
    if (!LATE && more) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const uint32_t c = (i * NT + tid) * V;
        if (c < C) ns[i] = load_chunk<XT, STREAM>(ds, c, C);
      }
    }
  };
  if (AHEAD) load(blockIdx.x);
  int turn = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
    if (!AHEAD) load(t);
    u32x4 ch[NV], cy[NV], cs[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) { ch[i] = nh[i]; cy[i] = ny[i]; cs[i] = ns[i]; }
    if (AHEAD && t + gridDim.x < a.T) load(t + gridDim.x);
    // the waves' shares of both sums, joined
    auto joined = [&](float& ss, float& gh) {
      ss = wave_sum(ss);
      gh = wave_sum(gh);
      if ((tid & 63) == 0) { part[turn][0][wave] = ss; part[turn][1][wave] = gh; }
      __syncthreads();
      ss = sum_of<W>(part[turn][0]);
      gh = sum_of<W>(part[turn][1]);
    };
    float ss = 0.f, gh = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float h[V], dy[V];
      unpack<XT>(ch[i], h);
      unpack<XT>(cy[i], dy);
      if (!HELD) {
        __builtin_amdgcn_sched_barrier(0);
        load_weights<V>(a.w, a.wt, (i * NT + tid) * V, C, w[0]);
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        ss = fmaf(h[j], h[j], ss);
        gh = fmaf(dy[j] * w[HELD ? i : 0][j], h[j], gh);
      }
    }
    joined(ss, gh);
    float s = factor(ss, a.C, a.eps), gn = gh * s / (float)a.C;            // gn: mean(g n)
    const float root = scaling_root(ss, a.eps);
    if (root != 1.f || !(fabsf(gh) < __builtin_inff())) {                  // the same for the whole workgroup
      // Once more with h scaled; and once more with g cut where their products' sum passes fp32's range, which their
      // mean over n does not: (g cut) (h root) is at most 2^32 2^80 then. From memory, a chunk at a time: such rows
      // are few, and what they hold in registers all rows would.
      const void *h_ = row_at<XT>(a.h, t), *dy_ = row_at<XT>(a.dy, t);
      float cut = root != 1.f ? 1.f : 0x1p-96f;
      for (;;) {
        __syncthreads();
        ss = gh = 0.f;
#pragma nounroll
        for (uint32_t c = tid * V; c < C; c += NT * V) {
          float h[V], dy[V], w[V];
          unpack<XT>(load_chunk<XT, false>(h_, c, C), h);
          unpack<XT>(load_chunk<XT, false>(dy_, c, C), dy);
          load_weights<V>(a.w, a.wt, c, C, w);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float v = h[j] * root, u = v * root;
            ss = fmaf(u, u, ss);
            gh = fmaf(dy[j] * cut * w[j], v, gh);
          }
        }
        joined(ss, gh);
        if (fabsf(gh) < __builtin_inff() || cut != 1.f) break;
        cut = 0x1p-96f;
      }
      if (root != 1.f) s = scaled_factor(ss, a.C, a.eps, root);
      gn = gh * s / (float)a.C / cut;
      s *= root;
    }
    // Elements are unpacked again below: kept as fp32 since the sums they would take the registers of 1024 threads
    // (with and without, us: 2000 x 28672 bf16 135 / 191, 700 x 11008 fp32 34 / 44; of 64 threads 16384 x 512 23.8 / 22.9).
    if constexpr (NT == 1024) {
#pragma unroll
      for (int i = 0; i < NV; ++i) asm volatile("" : "+v"(ch[i]), "+v"(cy[i]));
    }
    const void* ds_ = more && LATE ? row_at<XT>(a.dsum, t) : nullptr;
    void* dx = row_at(a.dx, t, sizeof(XT));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t c = (i * NT + tid) * V;
      if (c >= C) continue;
      if (!HELD) __builtin_amdgcn_sched_barrier(0);
      float h[V], dy[V], ds[V];
      unpack<XT>(ch[i], h);
      unpack<XT>(cy[i], dy);
      if (more) unpack<XT>(!LATE ? cs[i] : load_chunk<XT, STREAM>(ds_, c, C), ds);
      if (!HELD) load_weights<V>(a.w, a.wt, c, C, w[0]);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float n = h[j] * s;
        dw[i][j] = fmaf(dy[j], n, dw[i][j]);
        h[j] = (dy[j] * w[HELD ? i : 0][j] - n * gn) * s;
        if (more) h[j] += ds[j];
      }
      store_as<XT, STREAM>(dx, c, C, h);
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t c = (i * NT + tid) * V;
    if (c < C) store_f32<V, false>(a.ws + (int64_t)blockIdx.x * C, c, C, dw[i]);
  }
}

// dweight from the workgroups' rows: 8 threads of 4 channels each, 32 shares of the
// rows, joined in order.
__global__ __launch_bounds__(256) void norm_dw_kernel(const float* part, int rows, int C, void* dw, int wt) {
  __shared__ floatx4 lds[32][8];
  const int l = threadIdx.x & 7, share = threadIdx.x >> 3, c = (blockIdx.x * 8 + l) * 4;
  floatx4 v = {0.f, 0.f, 0.f, 0.f};
  if (c + 4 <= C) {
#pragma unroll 8
    for (int r = share; r < rows; r += 32) v += *(const f32x4_any*)(part + (int64_t)r * C + c);
  } else {
    for (int r = share; r < rows; r += 32)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < C) v[i] += part[(int64_t)r * C + c + i];
  }
  lds[share][l] = v;
  __syncthreads();
  if (share != 0 || c >= C) return;
  for (int i = 1; i < 32; ++i) v += lds[i][l];
  const float f[4] = {v[0], v[1], v[2], v[3]};
  if (wt == T_BF16) store_bf16<4, false>(dw, c, C, f);
  else store_f32<4, false>(dw, c, C, f);
}

// Threads and chunks for rows of C elements: up to 16 elements a thread, more past
// 16384 only.
// Measured (us): bf16 with residual, 512 workgroups, 16384 x 5120 to e4m3 in a layer's order
// 256 x 4 134, 512 x 2 98, 1024 x 1 147; 8192 x 8192 256 x 4 94, 512 x 2 89, 1024 x 1 89; 5000
// x 13824 512 x 4 112, 1024 x 2 93. fp32 2049 x 4097 256 x 8 17.1, 512 x 4 13.0, 1024 x 2 15.7.
// 512 x 1 and 256 x 2 (768 workgroups): 1 x 4096 3.0 and 3.4; 200 x 4096 3.5 and 4.0; 2000 x 4096
// 11.5 and 12.4; 10000 x 4096 59.6 and 60.1, x 2560 39.6 and 40.6. Gradient with dsum, 256 workgroups (us):
// 8191 x 8192 256 x 4 193, 512 x 2 91; 5000 x 13824 512 x 4 148, 1024 x 2 106; 16384 x 4096 256 x 2 99, 512 x 1
// 88; fp32 16384 x 2048 256 x 2 88, 512 x 1 91, 2049 x 4097 512 x 4 37, 1024 x 2 34, 5000 x 8192 512 x 4
// 113.6, 1024 x 2 114.0: one rule for both serves them within 10 %.
struct Shape {
  int nt, nv;
};
template <typename XT>
Shape shape_of(int C) {
  const int chunks = (C + kChunk<XT> - 1) / kChunk<XT>;
  if (chunks <= 64) return {64, 1};
  if (chunks <= 256) return {256, 1};
  if (chunks <= 512) return {512, 1};
  if (chunks <= 1024) return {512, 2};
  if (chunks <= 2048) return sizeof(XT) == 4 ? Shape{512, 4} : Shape{1024, 2};
  if (chunks <= 4096) return {1024, 4};
  return {1024, 8};
}
constexpr int64_t kStreamBytes = (int64_t)256 << 20;

// Workgroups of the gradient, each of which leaves a row in the workspace: 256 / 512
// / 1024 / 2048, us, with dsum: 8191 x 8192 91 / 94, 16384 x 4096 89 / 93, 16384 x 2048 70 / 49 / 54, 16384 x
// 512 - / 35 / 22.9 / 20.3 (the last for a workspace of twice the size).
int grad_rows(int T, int C) {
  const int most = C <= 512 ? 1024 : C <= 2048 ? 512 : 256;
  return T < most ? T : most;
}

template <typename XT, int NT, int NV>
hipError_t run_norm(const NormArgs& a, hipStream_t s) {
  // workgroups, us: 16384 x 5120 to e4m3 with 256 / 512 / 768 / 1024 146 / 98 / 123 / 103, 16384 x 4096
  // 512 / 1024 89 / 104, 10000 x 4096 512 / 768 58.6 / 59.6, x 2560 45.6 / 39.6, 16384 x 2048 512 / 1024 / 2048
  // 66 / 47 / 60, 16384 x 512 with 512 / 1024 / 2048 / 4096 31 / 18 / 13 / 12
  const int most = NT == 64 ? 4096 : NT * NV == 256 ? 1024 : NT * NV == 512 ? 768 : 512;
  const int64_t y = a.yt == T_E4M3 ? 1 : a.yt == T_BF16 ? 2 : 4;
  const int64_t bytes = (int64_t)a.T * a.C * (sizeof(XT) * (1 + (a.res.p != nullptr) + (a.sum.p != nullptr)) + y);
  const unsigned grid = a.T < most ? a.T : most;
  const size_t lds = a.B ? (size_t)a.C * y : 0;
  if (bytes > kStreamBytes) norm_kernel<XT, NT, NV, true><<<grid, NT, lds, s>>>(a);
  else norm_kernel<XT, NT, NV, false><<<grid, NT, lds, s>>>(a);
  return hipGetLastError();
}
template <typename XT, int NT, int NV>
hipError_t run_grad(const NormGradArgs& a, hipStream_t s) {
  const int rows = grad_rows(a.T, a.C);
  const int64_t bytes = (int64_t)a.T * a.C * sizeof(XT) * (3 + (a.dsum.p != nullptr));
  if (bytes > kStreamBytes) norm_grad_kernel<XT, NT, NV, true><<<(unsigned)rows, NT, 0, s>>>(a);
  else norm_grad_kernel<XT, NT, NV, false><<<(unsigned)rows, NT, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  norm_dw_kernel<<<(unsigned)((a.C + 31) / 32), 256, 0, s>>>(a.ws, rows, a.C, a.dw, a.wt);
  return hipGetLastError();
}

#define LCP_SHAPES(XT, RUN)                                                    \
  do {                                                                         \
    const Shape f = shape_of<XT>(a.C);                                         \
    if (f.nt == 64) return RUN<XT, 64, 1>(a, s);                               \
    if (f.nt == 256) return RUN<XT, 256, 1>(a, s);                             \
    if (f.nt == 512 && f.nv == 1) return RUN<XT, 512, 1>(a, s);                \
    if (f.nt == 512 && f.nv == 2) return RUN<XT, 512, 2>(a, s);                \
    if constexpr (sizeof(XT) == 4) {                                           \
      if (f.nt == 512) return RUN<XT, 512, 4>(a, s);                           \
      if (f.nv == 8) return RUN<XT, 1024, 8>(a, s);                            \
    } else {                                                                   \
      if (f.nv == 2) return RUN<XT, 1024, 2>(a, s);                            \
    }                                                                          \
    return RUN<XT, 1024, 4>(a, s);                                             \
  } while (0)

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, int xt, hipStream_t s) {
  if (xt == T_BF16) LCP_SHAPES(uint16_t, run_norm);
  LCP_SHAPES(float, run_norm);
}

size_t norm_grad_workspace_bytes(int T, int C) { return ((size_t)grad_rows(T, C) * C * 4 + 255) / 256 * 256; }

hipError_t launch_rms_norm_bwd(const NormGradArgs& a, int xt, hipStream_t s) {
  if (xt == T_BF16) LCP_SHAPES(uint16_t, run_grad);
  LCP_SHAPES(float, run_grad);
}

}  // namespace lcp
