// The deployed 2:4 product with an epilogue, in bf16 and in 8 bits (e4m3).
//
//   y[t][o] = act(sx_t sw_o sum_k Ws[o][k] x[t][k] + bias_o) gate[t][o] + residual[t][o]
//
// Packed weights: fragments of 32 rows x 32 (bf16) or 64 (e4m3) positions, 64 lanes
// of 16 bytes of kept values each; lane (h, n) holds row remap_row(n) and half h of
// the positions. In bytes both types are alike: what follows counts K in steps of
// two fragments, whose activations are 128 bytes of a row.
#include <algorithm>

#include "block.h"
#include "spgemm.h"

namespace lcp {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Exponentials and reciprocals are the hardware's, each good to one unit in the last place (the library's take
// ten times as long, as long as a tile's whole product: 256 x 128 values in 12 us). Where bf16 comes out an
// exponent is rounded as it is formed: off by 2^-15 at most. Where fp32 comes out what it loses is a second
// number, and all of an activation is good to 12 roundings, relative to its value.
// 2^(hi + lo), lo small beside 1.
__device__ __forceinline__ float exp2_sum(float hi, float lo) {
  const float e = exp2_(hi);
  return fmaf(0.693147181f * e, lo, e);
}
// log2 e and what fp32 drops of it.
constexpr float kLog2e = 1.4426950216293335f, kLog2eLow = 1.925963033500011e-08f;
// 1 / (1 + exp(-v)).
__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.f + exp2_(-kLog2e * v));
}
// The same from e = exp(-|v|).
__device__ __forceinline__ float sigmoid_of(float v, float e) {
  return (v < 0.f ? e : 1.f) * __builtin_amdgcn_rcpf(1.f + e);
}
template <bool FP32>
__device__ __forceinline__ float silu(float v) {
  if constexpr (!FP32) return v * sigmoid(v);
  const float x = fminf(fabsf(v), 128.f), hi = -kLog2e * x;             // exp(-128) is 0
  return v * sigmoid_of(v, exp2_sum(hi, fmaf(-kLog2eLow, x, fmaf(-kLog2e, x, -hi))));
}
// v (1 + erf(v / sqrt 2)) / 2 = v erfc(z) / 2 for v < 0 and v (1 - erfc(z) / 2) else, z = |v| / sqrt 2. erfc(z) / 2 is
// t P(t) exp(-z^2) with t = 1 / (1 + q z): P of degree 8 (fp32) or 5 (bf16) fitted to the smallest relative error on
// z <= 11 (beyond, exp(-z^2) is 0), 2^-25.7 and 2^-17.7 (degree 8 for both: 1000 tokens of 11008 <- 4096 79.4 against
// 78.6 us). An erfc that is good to 1.5e-7 absolute alone leaves 2 % of the values between v = -10 and -4.
template <bool FP32>
__device__ __forceinline__ float gelu(float v) {
  const float x = fminf(fabsf(v), 16.f), a = x * x, hi = -0.5f * kLog2e * a;
  float e;
  if constexpr (FP32) {
    const float low = fmaf(x, x, -a);
    e = exp2_sum(hi, fmaf(-0.5f * kLog2e, low, fmaf(-0.5f * kLog2eLow, a, fmaf(-0.5f * kLog2e, a, -hi))));
  } else {
    e = exp2_(hi);
  }
  constexpr float Q = FP32 ? 0.2651650309562683f : 0.30935922265052795f;               // 3 / 8 and 7 / 16, over sqrt 2
  const float t = __builtin_amdgcn_rcpf(fmaf(Q, x, 1.f));
  float p;
  if constexpr (FP32) {
    p = fmaf(0.03024500422179699f, t, -0.14119213819503784f);
    p = fmaf(p, t, 0.21124452352523804f);
    p = fmaf(p, t, -0.10921130329370499f);
    p = fmaf(p, t, 0.1331809163093567f);
    p = fmaf(p, t, 0.062274374067783356f);
    p = fmaf(p, t, 0.10227838158607483f);
    p = fmaf(p, t, 0.1053764596581459f);
    p = fmaf(p, t, 0.10580378025770187f);
  } else {
    p = fmaf(-0.07429610192775726f, t, 0.1830364316701889f);
    p = fmaf(p, t, 0.013430431485176086f);
    p = fmaf(p, t, 0.1342155933380127f);
    p = fmaf(p, t, 0.11999236047267914f);
    p = fmaf(p, t, 0.12361963838338852f);
  }
  const float tail = p * t * e;
  return v * (v < 0.f ? tail : 1.f - tail);
}
// 1 + tanh(u) = 2 / (1 + exp(-2u)), 2 u = 2 sqrt(2 / pi) v (1 + 0.044715 v^2).
template <bool FP32>
__device__ __forceinline__ float gelu_tanh(float v) {
  if constexpr (!FP32) return v * sigmoid(1.5957691216057308f * fmaf(0.044715f * v * v, v, v));
  constexpr float K = 0.044714998453855515f, KLOW = 1.5461444347053543e-09f;
  constexpr float C = 2.302208185195923f, CLOW = 1.2948402350332344e-08f;      // 2 sqrt(2 / pi) log2 e
  const float x = fminf(fabsf(v), 16.f), a = x * x;                            // exp(-2u) is 0 from there on
  const float q = fmaf(K, a, 1.f), qlow = fmaf(K, fmaf(x, x, -a), fmaf(KLOW, a, fmaf(K, a, 1.f - q)));
  const float m = x * q, mlow = fmaf(x, qlow, fmaf(x, q, -m)), hi = -C * m;
  return v * sigmoid_of(v, exp2_sum(hi, fmaf(-C, mlow, fmaf(-CLOW, m, fmaf(-C, m, -hi)))));
}
// The activation of N values; the branch on which one is taken once for all of them.
template <int N, bool FP32>
__device__ __forceinline__ void activate(f32x4* v, int act) {
  const auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i / 4][i % 4] = f(v[i / 4][i % 4]);
  };
  switch (act) {
    case 1: each([](float v) { return v < 0.f ? 0.f : v; }); break;
    case 2: each([](float v) { return silu<FP32>(v); }); break;
    case 3: each([](float v) { return gelu<FP32>(v); }); break;
    case 4: each([](float v) { return gelu_tanh<FP32>(v); }); break;
    default: break;
  }
}

__device__ __forceinline__ f32x4 pairs(u32x2 w) { return f32x4{lo_bf(w[0]), hi_bf(w[0]), lo_bf(w[1]), hi_bf(w[1])}; }

// The epilogue for R rows of a token (4, or 8 with a wave on whole lines): what it reads
// by row alone, what it reads by token, and the rest. A row's and a token's scale may each be
// 2^120 or 2^-126, and their product past fp32's normal numbers where the scaled sum is not:
// their fractions are then multiplied and their exponents added (always so, 17 tokens of
// 11008 <- 4096 take 9.7 instead of 9.25 us).
template <int R>
struct Finish {
  static constexpr int kRows = R, Q = R / 4;
  static constexpr bool kSplit = false;
  typedef uint32_t Words __attribute__((ext_vector_type(R / 2)));      // R bf16 numbers
  Epilogue e;
  struct Fixed {
    f32x4 scale[Q];
    Words bias;
  };
  struct Loaded {
    Words gate;
    f32x4 res[Q];                              // fp32, or bf16 in the first words
    float xscale;
  };
  __device__ __forceinline__ Fixed fixed(int o) const {
    Fixed f;
    if (e.wscale) {
#pragma unroll
      for (int i = 0; i < Q; ++i) f.scale[i] = *(const f32x4*)(e.wscale + o + 4 * i);
    }
    if (e.bias) f.bias = *(const Words*)(e.bias + o);
    return f;
  }
  __device__ __forceinline__ Loaded load(int64_t t, int o) const {
    Loaded l;
    if (e.wscale) l.xscale = e.xscale[t];
    if (e.gate) l.gate = *(const Words*)(e.gate + t * e.gate_row + o);
    if (e.res) {
      if (e.res_f32) {
#pragma unroll
        for (int i = 0; i < Q; ++i) l.res[i] = *(const f32x4*)((const float*)e.res + t * e.res_row + o + 4 * i);
      } else {
        const Words w = *(const Words*)((const uint16_t*)e.res + t * e.res_row + o);
#pragma unroll
        for (int i = 0; i < R / 2; ++i) l.res[0][i] = __uint_as_float(w[i]);
      }
    }
    return l;
  }
  __device__ __forceinline__ void finish(int64_t t, int o, f32x4* v, const Fixed& f, const Loaded& l) const {
    if (e.wscale) {
      f32x4 s[Q];
      float most = 0.f, least = __builtin_inff();
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        s[i] = f.scale[i] * l.xscale;
#pragma unroll
        for (int j = 0; j < 4; ++j) { most = fmaxf(most, fabsf(s[i][j])); least = fminf(least, fabsf(s[i][j])); }
      }
      if (__builtin_expect(most < __builtin_inff() && least >= 0x1p-126f, 1)) {
#pragma unroll
        for (int i = 0; i < Q; ++i) v[i] *= s[i];
      } else {
#pragma unroll
        for (int i = 0; i < Q; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            v[i][j] = __builtin_ldexpf(
                v[i][j] * (__builtin_amdgcn_frexp_mantf(f.scale[i][j]) * __builtin_amdgcn_frexp_mantf(l.xscale)),
                __builtin_amdgcn_frexp_expf(f.scale[i][j]) + __builtin_amdgcn_frexp_expf(l.xscale));
      }
    }
    if (e.bias) {
#pragma unroll
      for (int i = 0; i < Q; ++i) v[i] += pairs(u32x2{f.bias[2 * i], f.bias[2 * i + 1]});
    }
    if (e.y_f32) activate<R, true>(v, e.act);
    else activate<R, false>(v, e.act);
    if (e.gate) {
#pragma unroll
      for (int i = 0; i < Q; ++i) v[i] *= pairs(u32x2{l.gate[2 * i], l.gate[2 * i + 1]});
    }
    if (e.res) {
#pragma unroll
      for (int i = 0; i < Q; ++i)
        v[i] += e.res_f32 ? l.res[i] : pairs(u32x2{__float_as_uint(l.res[0][2 * i]), __float_as_uint(l.res[0][2 * i + 1])});
    }
    if (e.y_f32) {
#pragma unroll
      for (int i = 0; i < Q; ++i) *(f32x4*)((float*)e.y + t * e.y_row + o + 4 * i) = v[i];
    } else {
      Words w;
#pragma unroll
      for (int i = 0; i < R; i += 2) w[i / 2] = pack2(v[i / 4][i % 4], v[i / 4][i % 4 + 1]);
      *(Words*)((uint16_t*)e.y + t * e.y_row + o) = w;
    }
  }
  __device__ __forceinline__ void store(int64_t t, int o, f32x4 a, f32x4 b, const Fixed& f, const Loaded& l) const {
    f32x4 v[2] = {a, b};
    finish(t, o, v, f, l);
  }
};
// A part's sums as they are, fp32, for linear_join_kernel.
struct Part {
  static constexpr int kRows = 8;
  static constexpr bool kSplit = true;
  float* ws;                                   // [parts][T][cout]
  int T, cout, part;
  struct Fixed {};
  struct Loaded {};
  __device__ __forceinline__ Fixed fixed(int) const { return {}; }
  __device__ __forceinline__ Loaded load(int64_t, int) const { return {}; }
  __device__ __forceinline__ void store(int64_t t, int o, f32x4 a, f32x4 b, const Fixed&, const Loaded&) const {
    f32x4* y = (f32x4*)(ws + ((int64_t)part * T + t) * cout + o);
    y[0] = a;
    y[1] = b;
  }
};

__device__ __forceinline__ void finish4(const Epilogue& e, int64_t t, int o, f32x4 v) {
  const Finish<4> f{e};
  f.finish(t, o, &v, f.fixed(o), f.load(t, o));
}

// 16 rows x 16 tokens over two fragments' positions: w = lane (g, r)'s 16 bytes of
// kept values, b0 and b1 = bytes 16 g and 64 + 16 g of token r's 128.
template <int MODE>
struct Act16 {                                 // a lane's activations of a step, as the instructions take them
  u32x8 b[MODE == M_E4M3 ? 2 : 1];
  __device__ __forceinline__ Act16(u32x4 b0, u32x4 b1) {
    b[0] = cat(b0, b1);
    if constexpr (MODE == M_E4M3) {
      b[1] = half_acts(b[0], 1);
      b[0] = half_acts(b[0], 0);
    }
  }
};
template <int MODE>
struct Wgt16 {
  u32x4 a[MODE == M_E4M3 ? 2 : 1];
  uint32_t idx[MODE == M_E4M3 ? 2 : 1];
  __device__ __forceinline__ Wgt16(u32x4 w, uint32_t i) {
    a[0] = w;
    idx[0] = i;
    if constexpr (MODE == M_E4M3) {
#pragma unroll
      for (int j = 1; j >= 0; --j) { a[j] = half_vals(w, j); idx[j] = half_idx(i, j); }
    }
  }
};
template <int MODE>
__device__ __forceinline__ f32x4 smfma16(const Wgt16<MODE>& w, const Act16<MODE>& x, f32x4 c) {
  if constexpr (MODE == M_E4M3_FAST) {
    return __builtin_amdgcn_smfmac_f32_16x16x128_fp8_fp8(__builtin_bit_cast(i32x4, w.a[0]), __builtin_bit_cast(i32x8, x.b[0]),
                                                         c, (int)w.idx[0], 0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < (MODE == M_E4M3 ? 2 : 1); ++j)
      c = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(as_bf16x8(w.a[j]), __builtin_bit_cast(bf16x16, x.b[j]), c,
                                                    (int)w.idx[j], 0, 0);
    return c;
  }
}

// Few tokens: the bytes of the weights bound it. A workgroup takes RT tiles of 16
// packed rows and NT tiles of 16 tokens over all of K; its W waves take the steps of K in
// turn and join their sums in LDS, in order. Nothing is shared on the way there: a step's
// weights are read once by one wave, straight into the operands. Its activations are 128
// bytes of every token: read in whole lines and turned through the wave's own LDS (each
// lane's two halves of a line straight from memory took twice as long from 32 tokens on:
// 64 tokens of 4096 <- 4096 17.2 against 9.4 us). The next step's loads fly during a step.
// `tokens`: workgroups over the tokens; those of the same rows come one after the other on
// one XCD (id mod 8), whose L2 then serves the rows' weights again.
template <int MODE, int RT, int NT, int W>
__global__ __launch_bounds__(64 * W) void linear_thin_kernel(LinearArgs a, uint32_t tokens) {
  constexpr int E = MODE == M_BF16 ? 2 : 1, X = 2 * NT;                     // X: loads of a lane for a step's tokens
  constexpr int TILES = RT * NT, ROUND = X < TILES ? X : TILES;             // tiles joined at a time
  __shared__ __attribute__((aligned(16))) u32x4 lds[W * 64 * X];
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int KF = E == 1 ? (a.w.cin + 63) / 64 : a.w.cin / 32, KS = (KF + 1) / 2, KW = E == 1 ? KF : KS;
  const uint32_t id = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
  const int row0 = (int)(id / tokens) * (16 * RT);             // in packed rows: fragment rows in lane order
  const int64_t t0 = (int64_t)(id % tokens) * (16 * NT);
  if (row0 >= a.w.cout) return;                // the grid is a multiple of 8
  const uint32_t bytes = (uint32_t)a.w.cin * E;
  const char* vals[RT];
  const char* meta[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int row = min(row0 + 16 * i, a.w.cout - 16), l = 32 * (g & 1) + (row & 16) + r;
    vals[i] = (const char*)(a.w.vals + ((int64_t)(row >> 5) * KF + (g >> 1)) * 64 + l);
    meta[i] = (const char*)(a.w.meta + ((int64_t)(row >> 5) * KW + (E == 1 ? g >> 1 : 0)) * 64 + l);
  }
  // columns past T are not stored: their tokens are the last one again
  const char* x[X];
#pragma unroll
  for (int j = 0; j < X; ++j) {
    const int64_t t = t0 + 8 * j + (lane >> 3);
    x[j] = (const char*)a.x.p + (t < a.T ? t : a.T - 1) * a.x.row * E + 16 * (lane & 7);
  }
  u32x4* const mine = lds + wave * (64 * X);
  // places in a stage of 16 NT tokens x 8 pieces of 16 bytes: piece p of token n at p ^ (n / 2 % 8), so that neither
  // the writes (eight tokens whole) nor the reads (a piece of 16 tokens) meet in a bank
  const int put = (lane >> 3) * 8 + ((lane & 7) ^ ((lane >> 4) & 3));
  f32x4 acc[RT][NT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  u32x4 w[RT], v[X];
  uint32_t idx[RT];
  const int whole = bytes / 128u;              // steps before K's end
  auto load = [&](int s) {
    if (s < whole) {
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        w[i] = *(const u32x4*)(vals[i] + (uint32_t)s * 2048u);
        idx[i] = *(const uint32_t*)(meta[i] + (uint32_t)s * (E == 1 ? 512u : 256u));
      }
#pragma unroll
      for (int j = 0; j < X; ++j) v[j] = *(const u32x4*)(x[j] + (uint32_t)s * 128u);
    } else {
      // K ends inside the step: positions past the end are empty on both sides
      const bool in = 2 * s + (g >> 1) < KF;
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        w[i] = u32x4{0, 0, 0, 0};
        idx[i] = 0x44444444u;
        if (in) w[i] = *(const u32x4*)(vals[i] + (uint32_t)s * 2048u);
        if (E == 2 || in) idx[i] = *(const uint32_t*)(meta[i] + (uint32_t)s * (E == 1 ? 512u : 256u));
      }
#pragma unroll
      for (int j = 0; j < X; ++j) {
        v[j] = u32x4{0, 0, 0, 0};
        if ((uint32_t)s * 128u + 16u * (lane & 7) < bytes) v[j] = *(const u32x4*)(x[j] + (uint32_t)s * 128u);
      }
    }
  };
  int s = wave;
  if (s < KS) load(s);
  while (s < KS) {
    u32x4 cw[RT];
    uint32_t ci[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) { cw[i] = w[i]; ci[i] = E == 1 ? idx[i] : idx[i] >> (16 * (g >> 1)); }
#pragma unroll
    for (int j = 0; j < X; ++j) mine[64 * j + (put ^ (4 * (j & 1)))] = v[j];
    wave_fence();
    s += W;
    if (s < KS) load(s);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int n = (16 * j + r) * 8, k = (r >> 1) & 7;
      const Act16<MODE> b(mine[n + (g ^ k)], mine[n + ((4 + g) ^ k)]);
#pragma unroll
      for (int i = 0; i < RT; ++i) acc[i][j] = smfma16<MODE>(Wgt16<MODE>(cw[i], ci[i]), b, acc[i][j]);
    }
    wave_fence();
  }
  // a round of tiles: every wave's sums to LDS, then added in the waves' order
  f32x4* const sums = (f32x4*)lds;
#pragma unroll
  for (int r0 = 0; r0 < TILES; r0 += ROUND) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < ROUND; ++k)
      if (r0 + k < TILES) sums[(wave * ROUND + k) * 64 + lane] = acc[(r0 + k) / NT][(r0 + k) % NT];
    __syncthreads();
    for (int k = wave; k < ROUND && r0 + k < TILES; k += W) {
      f32x4 y = sums[k * 64 + lane];
#pragma unroll
      for (int u = 1; u < W; ++u) y += sums[(u * ROUND + k) * 64 + lane];
      // lane (g, r): token r of the tile, packed rows 4 g .. 4 g + 3
      const int row = row0 + 16 * ((r0 + k) / NT) + 4 * g;
      const int64_t t = t0 + 16 * ((r0 + k) % NT) + r;
      if (t >= a.T || row >= a.w.cout) continue;
      finish4(a.e, t, (row & ~31) + remap_row(row & 31), y);
    }
  }
}

// The parts of K, added in order, all of them loaded first (the last one again past the
// end, without a branch between the loads).
constexpr int kMostParts = 8;
__global__ __launch_bounds__(256) void linear_join_kernel(LinearArgs a, int parts) {
  const uint32_t id = blockIdx.x * 256 + threadIdx.x, quads = a.w.cout / 4, n = a.T * quads;      // within kMostPartBytes
  if (id >= n) return;
  const Finish<4> f{a.e};
  const uint32_t t = id / quads, o = (id - t * quads) * 4;
  f32x4 p[kMostParts];
#pragma unroll
  for (int z = 0; z < kMostParts; ++z) p[z] = ((const f32x4*)a.ws)[(uint32_t)min(z, parts - 1) * n + id];
  const auto fixed = f.fixed(o);
  const auto loaded = f.load(t, o);
  f32x4 v = p[0];
#pragma unroll
  for (int z = 1; z < kMostParts; ++z) v = z < parts ? v + p[z] : v;
  f.finish(t, o, &v, fixed, loaded);
}

// The first two kept positions of a group of four, completed by the lowest free ones
// with value 0, ascending: bit mask of the positions whose values count in `real`.
__device__ __forceinline__ void two_of(uint32_t kept, int* pos, bool* real) {
  int n = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (((kept >> q) & 1u) && n < 2) pos[n++] = q;
  real[0] = n > 0;
  real[1] = n > 1;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (!((kept >> q) & 1u) && n < 2) pos[n++] = q;
  if (pos[0] > pos[1]) {
    const int p = pos[0]; pos[0] = pos[1]; pos[1] = p;
    const bool b = real[0]; real[0] = real[1]; real[1] = b;
  }
}

// The scale of a row's kept values, one workgroup a row.
__global__ __launch_bounds__(256) void pack_scale_kernel(const uint16_t* W, int cin, int B, const int* perm,
                                                         const uint32_t* bits, float* wscale) {
  __shared__ uint32_t lds[4];
  const int o = blockIdx.x;
  uint32_t top = 0;
  for (int g = threadIdx.x; g < cin / 4; g += 256) {
    int pos[2];
    bool real[2];
    two_of((bits[(int64_t)o * (cin / 32) + g / 8] >> (4 * (g & 7))) & 0xFu, pos, real);
    for (int i = 0; i < 2; ++i) {
      const int k = 4 * g + pos[i], src = k / B * B + (perm[k] & (B - 1));
      if (real[i]) top = max(top, (uint32_t)(W[(int64_t)o * cin + src] & 0x7fffu) << 16);
    }
  }
  for (int m = 1; m < 64; m <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m, 64));
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = top;
  __syncthreads();
  if (threadIdx.x == 0) wscale[o] = e4m3_scale(max(max(lds[0], lds[1]), max(lds[2], lds[3])));
}

// One thread per fragment and lane: 32 positions of a row.
__global__ __launch_bounds__(256) void pack_e4m3_kernel(const uint16_t* W, int cout, int cin, int B, const int* perm,
                                                        const uint32_t* bits, u32x4* vals, uint32_t* meta,
                                                        const float* wscale) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int KF = (cin + 63) / 64;
  if (id >= (int64_t)(cout / 32) * KF * 64) return;
  const int l = (int)(id & 63), kf = (int)((id >> 6) % KF), rg = (int)((id >> 6) / KF);
  const int o = 32 * rg + remap_row(l & 31), k0 = 64 * kf + 32 * (l >> 5);
  const bool in = k0 < cin;                              // cin is a multiple of 32
  const uint32_t word = in ? bits[(int64_t)o * (cin / 32) + k0 / 32] : 0u;
  const float s = wscale[o], inv = 1.f / s;              // a power of two, or NaN
  u32x4 v = {0, 0, 0, 0};
  uint32_t m = 0;
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    int pos[2];
    bool real[2];
    two_of((word >> (4 * g)) & 0xFu, pos, real);
    m |= (uint32_t)(pos[0] | (pos[1] << 2)) << (4 * g);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float y = 0.f;
      if (real[i] && s == s) {
        const int k = k0 + 4 * g + pos[i];
        y = bf2f(W[(int64_t)o * cin + k / B * B + (perm[k] & (B - 1))]) * inv;
      }
      const uint32_t c = __builtin_amdgcn_cvt_pk_fp8_f32(y, y, 0, false) & 0xff;
      v[g / 2] |= c << (16 * (g & 1) + 8 * i);
    }
  }
  vals[id] = v;
  meta[id] = m;
}

}  // namespace

constexpr int64_t kMaxThreads = ((int64_t)1 << 32) - 256;

size_t sparse_vals_bytes_e4m3(int cout, int cin) { return (size_t)(cout / 32) * ((cin + 63) / 64) * 1024; }
size_t sparse_meta_bytes_e4m3(int cout, int cin) { return (size_t)(cout / 32) * ((cin + 63) / 64) * 256; }

hipError_t launch_sparse_pack_e4m3(const uint16_t* W, int cout, int cin, int B, const int* perm, const uint32_t* bits,
                                   u32x4* vals, uint32_t* meta, float* wscale, hipStream_t s) {
  if ((int64_t)cout * 256 > kMaxThreads) return hipErrorInvalidConfiguration;
  pack_scale_kernel<<<(unsigned)cout, 256, 0, s>>>(W, cin, B, perm, bits, wscale);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t n = (int64_t)(cout / 32) * ((cin + 63) / 64) * 64;
  pack_e4m3_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(W, cout, cin, B, perm, bits, vals, meta, wscale);
  return hipGetLastError();
}

namespace {

// How a product is cut: RT x NT tiles of 16 rows x 16 tokens and W waves a workgroup, or
// (RT 0) 256 x 128 tiles with K in `parts`, each of which has steps.
struct Cut {
  int rt, nt, w, parts;
};

// Parts' sums are kept up to this size. One workspace then serves every smaller call.
constexpr int64_t kMostPartBytes = (int64_t)48 << 20;
// Tokens from which the tiles are looked at, and a workspace is asked for. Up to 64 they would gain at
// the longest K alone: bf16, 64 tokens on the thin kernel against 80 on tiles, us: 8192 <- 28672 74.1 / 66.5,
// 28672 <- 8192 57.6 / 68.7, 5120 <- 13824 23.4 / 29.3.
constexpr int kTilesFrom = 65;

// The estimates that choose, in us, fitted to 351 calls (4096 <- 4096, 11008 <- 4096, 4096 <- 11008,
// 5120 <- 13824, 13824 <- 5120, 28672 <- 8192, 8192 <- 28672, 6400 <- 2720, 2080 <- 9600; 24 to 1000
// tokens; each mode): the chosen cut is 1.2 % slower than the best measured one in the mean, over
// 10 % at 16 calls, 23 % at one. No call was held out of the fit, and past 1000 tokens it is
// carried on. A workgroup of the thin kernel takes in 80 KB a us, a tile's
// step takes 0.46 us (e4m3 0.53, converted 0.82), and what a call takes follows from the rounds
// of 256 workgroups. Measured, us: 128 tokens of 4096 <- 4096 bf16 2 x 4 x 8 11.0, 4 x 4 x 8 13.1, tiles
// in four parts 18.2; 200 4 x 4 x 8 13.4, 2 x 4 x 8 18.7; 100 of 11008 <- 4096 6 x 4 x 4 18.6, 4 x 4 x 4 21.3,
// tiles in two parts 23.4; 333 31.0 on tiles, 4 x 4 x 4 49.8; 100 of 5120 <- 13824 e4m3 converted 3 x 4 x 8
// 20.4, 4 x 4 x 8 22.1, tiles in seven parts 27.1; 200 tokens of it in e4m3 5 x 4 x 8 21.7, tiles in
// four parts 26.9, 4 x 4 x 4 29.
double tiles_cost(int tiles) { return tiles >= 32 ? 1.43 : tiles >= 24 ? 1.31 : tiles >= 20 ? 1.2 : 1.0; }      // a step's, of more
double thin_us(const LinearArgs& a, int mode, const Cut& c) {
  // KB a row tile and a token tile bring a step; converted operands cost their conversion, too
  const double w = mode == M_BF16 ? 1.15 : mode == M_E4M3 ? 2.0 : 1.45, x = mode == M_E4M3 ? 2.1 : 2.05;
  const int64_t steps = ((int64_t)a.w.cin * (mode == M_BF16 ? 2 : 1) + 127) / 128;
  const int64_t n = (int64_t)((a.w.cout + 16 * c.rt - 1) / (16 * c.rt)) * (((int64_t)a.T + 16 * c.nt - 1) / (16 * c.nt));
  const double each = (double)steps * (c.rt * w + c.nt * x) / 80.0;
  return 2.9 + (double)((n + 255) / 256) * each * tiles_cost(c.rt * c.nt);
}
double tiles_us(const LinearArgs& a, int mode, int64_t steps, int parts) {
  const int64_t n = (int64_t)((a.w.cout + SP_BM - 1) / SP_BM) * (((int64_t)a.T + SP_BN - 1) / SP_BN) * parts;
  const double step = mode == M_BF16 ? 0.46 : mode == M_E4M3 ? 0.82 : 0.53;
  const double join = parts > 1 ? 2.8 + (2.0 * parts + 1) * a.T * a.w.cout * 4.0 / 4.1e6 : 0.0;
  return 3.3 + (double)((n + 255) / 256) * ((double)((steps + parts - 1) / parts) * step + 1.25) + join;
}

Cut cut_for(const LinearArgs& a, int mode) {
  const int groups = a.w.cout / 32;
  // Up to 16 tokens the weights' bytes alone count: the waves in flight for them. 1 x 16, 2 x 16, 2 x 8,
  // 4 x 8 (row tiles x waves), us, 16 tokens, bf16: 2080 <- 9600 8.0 / 9.9 / 11.1 / 13.5, 4096 <- 4096 6.1 / 6.5 / 6.8 /
  // 8.1, 4096 <- 11008 10.1 / 11.5 / 13.1 / 15.7, 5120 <- 13824 19.3 / 14.7 / 16.1 / 19.0, 13824 <- 5120 18.1 / 15.4 /
  // 14.1 / 14.3, 28672 <- 8192 66 / 56 / 53 / 49; e4m3 in the same order 5.6 / 6.7 / 7.4 / 9.4, 4.2 / 4.6 / 4.7 / 6.2,
  // 7.0 / 7.9 / 8.5 / 10.5, 12.3 / 9.7 / 10.1 / 12.3, 12.6 / 10.6 / 9.7 / 10.1, 41 / 36 / 33 / 30.
  if (a.T <= 16) {
    if (groups <= 128) return {1, 1, 16, 1};
    if (groups <= 256) return {2, 1, 16, 1};
    return groups <= 512 ? Cut{2, 1, 8, 1} : Cut{4, 1, 8, 1};
  }
  // 4 x 4: more waves while every workgroup has its compute unit
  const int wide = (a.w.cout + 63) / 64 * (((int64_t)a.T + 63) / 64) <= 256 ? 8 : 4;
  const Cut all[] = {{2, 2, 8, 1}, {4, 2, 8, 1}, {2, 4, 8, 1},    {3, 4, 8, 1},
                     {5, 4, 8, 1}, {6, 4, 4, 1}, {4, 4, wide, 1}, {8, 4, 4, 1}};
  Cut best{};
  double least = 1e30;
  for (const Cut& c : all) {
    if (c.nt == 2 ? a.T > 64 : a.T <= 32) continue;
    if (c.rt == 8 && mode != M_BF16) continue;           // in 8 bits never the least
    if (c.rt == 5 && mode == M_E4M3) continue;           // the conversions would spill registers
    const double us = thin_us(a, mode, c);
    if (us < least) { least = us; best = c; }
  }
  if (a.T < kTilesFrom) return best;
  const int64_t steps = ((int64_t)a.w.cin * (mode == M_BF16 ? 2 : 1) + 127) / 128;
  for (int most = 1; most <= kMostParts; ++most) {
    const int64_t each = (steps + most - 1) / most;
    const int parts = (int)((steps + each - 1) / each);
    if (most > steps || (parts > 1 && (int64_t)parts * a.T * a.w.cout * 4 > kMostPartBytes)) break;
    const double us = tiles_us(a, mode, steps, parts);
    if (us < least) { least = us; best = {0, 0, 0, parts}; }
  }
  return best;
}

template <int MODE, int RT, int NT, int W>
hipError_t run_thin(const LinearArgs& a, hipStream_t s) {
  const int64_t tokens = (a.T + (int64_t)16 * NT - 1) / (16 * NT);
  const int64_t n = ((int64_t)((a.w.cout + 16 * RT - 1) / (16 * RT)) * tokens + 7) / 8 * 8;
  if (n * 64 * W > kMaxThreads) return hipErrorInvalidConfiguration;
  linear_thin_kernel<MODE, RT, NT, W><<<(unsigned)n, 64 * W, 0, s>>>(a, (uint32_t)tokens);
  return hipGetLastError();
}

template <int MODE>
hipError_t run_tiles(const LinearArgs& a, int parts, hipStream_t s) {
  constexpr int NPRE = MODE == M_E4M3 ? 8 : SP_NPRE;
  const int64_t G = (int64_t)((a.w.cout + SP_BM - 1) / SP_BM) * ((a.T + (int64_t)SP_BN - 1) / SP_BN);
  const auto grid = [](int64_t n) { return (unsigned)((n + 7) / 8 * 8); };          // the same for every XCD
  if ((G * parts + 7) * SP_NT > kMaxThreads) return hipErrorInvalidConfiguration;
  const int all = (int)(((int64_t)a.w.cin * (MODE == M_BF16 ? 2 : 1) + 127) / 128);
  if (parts == 1) {
    spgemm_kernel<MODE, SP_RS, NPRE, SP_LSPAN><<<grid(G), SP_NT, SP_LDS<MODE>, s>>>(
        a.w.vals, a.w.meta, a.x.p, a.x.row, a.T, a.w.cout, a.w.cin, all, Finish<8>{a.e});
    return hipGetLastError();
  }
  const int steps = (all + parts - 1) / parts;
  spgemm_kernel<MODE, SP_RS, NPRE, SP_LSPAN><<<grid(G * parts), SP_NT, SP_LDS<MODE>, s>>>(
      a.w.vals, a.w.meta, a.x.p, a.x.row, a.T, a.w.cout, a.w.cin, steps, Part{a.ws, a.T, a.w.cout, 0});
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  linear_join_kernel<<<(unsigned)(((int64_t)a.T * a.w.cout / 4 + 255) / 256), 256, 0, s>>>(a, parts);
  return hipGetLastError();
}

template <int MODE>
hipError_t run_linear(const LinearArgs& a, hipStream_t s) {
  const Cut c = cut_for(a, MODE);
  if (c.rt == 0) return run_tiles<MODE>(a, c.parts, s);
  if (c.nt == 4) {
    if (c.rt == 2) return run_thin<MODE, 2, 4, 8>(a, s);
    if (c.rt == 3) return run_thin<MODE, 3, 4, 8>(a, s);
    if constexpr (MODE != M_E4M3) {
      if (c.rt == 5) return run_thin<MODE, 5, 4, 8>(a, s);
    }
    if (c.rt == 6) return run_thin<MODE, 6, 4, 4>(a, s);
    if constexpr (MODE == M_BF16) {
      if (c.rt == 8) return run_thin<MODE, 8, 4, 4>(a, s);
    }
    return c.w == 8 ? run_thin<MODE, 4, 4, 8>(a, s) : run_thin<MODE, 4, 4, 4>(a, s);
  }
  if constexpr (MODE != M_E4M3_FAST) {         // more than 64 tokens, with four token tiles
    if (c.nt == 2) return c.rt == 2 ? run_thin<MODE, 2, 2, 8>(a, s) : run_thin<MODE, 4, 2, 8>(a, s);
    if (c.rt == 2) return c.w == 8 ? run_thin<MODE, 2, 1, 8>(a, s) : run_thin<MODE, 2, 1, 16>(a, s);
    return c.rt == 1 ? run_thin<MODE, 1, 1, 16>(a, s) : run_thin<MODE, 4, 1, 8>(a, s);
  }
  return hipErrorInvalidConfiguration;
}

// e4m3: exact products, but where the layer's user asked for the e4m3 instructions, whose dropped bits are the whole
// result where sums cancel; not for fp32 outputs, nor for few tokens, where exact products cost nothing (us,
// converted against e4m3 instructions: 64 tokens of 4096 <- 4096 5.8 / 5.5, 128 8.6 / 7.6; random operands, 1000
// tokens of 11008 <- 4096 85 / 67, 4096 of 28672 <- 8192 965 / 640).
int mode_for(const PackedArgs& w, int T, int y_f32) {
  if (!w.fp8) return M_BF16;
  return !w.fast || y_f32 || T < kTilesFrom ? M_E4M3 : M_E4M3_FAST;
}
}  // namespace

size_t sparse_linear_workspace_bytes(const PackedArgs& w, int T) {
  if (T < kTilesFrom) return 0;
  const int64_t most = std::min((int64_t)kMostParts * T * w.cout * 4, kMostPartBytes);
  return (size_t)((most + 255) / 256 * 256);
}

void sparse_linear_cut(const PackedArgs& w, int T, int y_f32, int* out) {
  LinearArgs a{};
  a.w = w;
  a.T = T;
  out[0] = mode_for(w, T, y_f32);
  const Cut c = cut_for(a, out[0]);
  out[1] = c.rt;
  out[2] = c.nt;
  out[3] = c.w;
  out[4] = c.parts;
}

hipError_t launch_sparse_linear(const LinearArgs& a, hipStream_t s) {
  const int mode = mode_for(a.w, a.T, a.e.y_f32);
  if (mode == M_BF16) return run_linear<M_BF16>(a, s);
  return mode == M_E4M3 ? run_linear<M_E4M3>(a, s) : run_linear<M_E4M3_FAST>(a, s);
}

}  // namespace lcp
