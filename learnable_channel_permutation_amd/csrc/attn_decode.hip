// Attention of one new token of each sequence over the paged cache.
//
//   z_t = scale q.k_t,  out = sum_t exp(z_t - m) v_t / sum_t exp(z_t - m)
//
// Every cached element is used by the G query heads of its group only (2 G
// flops a byte with 8-bit codes), so the bytes of K and V bound the operator.
// One pass over them with the running maximum and sum of the softmax; a
// workgroup takes a chunk of one sequence's tokens for one key/value head and
// (up to 16 of) its query heads, and chunks are joined by a second kernel.
//
// A wave takes 32 tokens at a time and keeps everything in registers, from the
// loads to the matrix instructions (16x16x32 bf16, fp32 sums):
//   S[token][head] = K Q^T   A = K rows as loaded, B = Q. Lane (r, g) = (lane %
//     16, lane / 16) loads 16-byte pieces g, g + 4, .. of token r's row; which
//     channels meet in one product does not matter as long as Q's fragment
//     holds the same ones.
//   The result leaves lane (h, g) with tokens 4g .. 4g+3 of each half of the 32
//   for head h: a softmax over registers, no exchange between lanes except for
//   a new maximum.
//   O^T[channel][head] += V^T P^T   B = P as it stands in the registers: lane
//     (h, g) supplies K slots 8g .. 8g+7, which are the tokens named above. So
//     lane (c, g) loads those eight tokens' channels c D/16 .. of V, and the
//     transposition is a byte permutation within the lane.
#include "serve.h"

namespace lcp {
namespace {

constexpr int kWaves = 4;
constexpr int kStep = 32;                    // tokens of a wave's step
constexpr int kRound = kWaves * kStep;       // tokens of a workgroup's round
constexpr float kLowest = -3.402823466e38f;  // running maximum before any token: below every finite score but
                                             // itself, and finite, so that masked scores (-inf) give exp2 = 0
constexpr float kLazy = 8.f;                 // the maximum follows once a score passes it by this (in log2)

typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
}

// Two 8-bit codes (bytes 2 * HI and 2 * HI + 1 of w) -> a bf16 pair, exactly:
// e4m3 has 4 significant bits, an int8 at most 8.
template <int FMT, bool HI>
__device__ __forceinline__ uint32_t codes2(uint32_t w) {
  if (FMT == KV_E4M3) return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
  const int8_t c0 = (int8_t)(w >> (HI ? 16 : 0)), c1 = (int8_t)(w >> (HI ? 24 : 8));
  return pack2_exact((float)c0, (float)c1);
}

struct Plan {            // the same for every workgroup
  int chunk, nch;        // tokens of a chunk (a multiple of kRound), chunks a sequence can have
  int G, ht;             // query heads of a group, head tiles of 16 in it
  uint32_t tpm;          // ceil(2^32 / (page_size / 16)): page of a 16-token tile by a high product
  float* part;           // partial sums [B * hq][nch][D], then maxima and sums [B * hq][nch][2]
  float2* ml;
};

// A half step: 16 tokens, all of one page.
struct Half {
  int64_t row;           // first cache row
  int ok;                // whether the page exists and the half begins before the end
};

template <int FMT, int D>
__global__ __launch_bounds__(256) void attn_chunk_kernel(AttnArgs a, Plan p) {
  constexpr int E = FMT == KV_BF16 ? 2 : 1;
  constexpr int KL = D * E / 64;               // 16-byte K loads of a lane for 16 tokens
  constexpr int VC = D / 16;                   // channels of V a lane holds of each of its 8 tokens
  constexpr int VW = VC * E / 4;               // their 32-bit words
  constexpr int QF = D / 32;                   // products over the channels
  constexpr int OS = D + 4;                    // row stride of the waves' sums in LDS
  __shared__ float so[kWaves][16][OS];
  __shared__ float sm[kWaves][16], sl[kWaves][16];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, g = lane >> 4;
  const int units = a.c.heads * p.ht;
  const int chunk_id = blockIdx.x / (a.B * units);
  const int rest = blockIdx.x % (a.B * units);
  const int b = rest / units, hk = rest % units / p.ht, h0 = rest % p.ht * 16;
  const int len = min(max(a.lens[b], 0), a.max_len);
  const int lo = a.window && len > a.window ? len - a.window : 0;
  const int begin = (lo & ~(kStep - 1)) + chunk_id * p.chunk;
  const int end = min(len, begin + p.chunk);
  if (begin >= end && chunk_id > 0) return;    // chunk 0 of an empty sequence writes its zeros
  const int nh = min(16, p.G - h0);
  const int head0 = hk * p.G + h0;

  // Q fragments: head c16, the channels that the K loads bring
  u32x4 qf[QF];
#pragma unroll
  for (int m = 0; m < QF; ++m) {
    const int d = E == 2 ? 32 * m + 8 * g : 64 * (m >> 1) + 16 * g + 8 * (m & 1);
    qf[m] = u32x4{0, 0, 0, 0};
    if (c16 < nh) qf[m] = *(const u32x4*)(a.q + b * a.qrow + (int64_t)(head0 + c16) * D + d);
  }

  const int* pages = a.pages + (int64_t)b * a.max_pages;
  const int tp = a.c.ps >> 4;
  auto half_at = [&](int t) {                  // t: first token, a multiple of 16
    Half r;
    r.row = 0;
    r.ok = 0;
    if (t < end) {
      const uint32_t tile = (uint32_t)t >> 4, pg = __umulhi(tile, p.tpm);
      const uint32_t pgi = p.tpm == 0 ? tile : pg;      // one tile a page
      const int id = __builtin_amdgcn_readfirstlane(pages[pgi]);
      if (id >= 0 && id < a.c.pages) {
        r.row = ((int64_t)id * a.c.heads + hk) * a.c.ps + (int)(tile - pgi * tp) * 16;
        r.ok = 1;
      }
    }
    return r;
  };

  u32x4 kf[2][KL];
  uint32_t vw[8][VW];
  f32x4 ks[2], vs[2];
  const uint32_t koff = c16 * (D * E) + 16 * g, voff = 4 * g * (D * E) + c16 * (VC * E);
  auto load_k = [&](const Half* hf) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const char* base = (const char*)a.c.k + hf[i].row * (D * E);
#pragma unroll
      for (int j = 0; j < KL; ++j) kf[i][j] = *(const u32x4*)(base + (koff + 64 * j));
      if (E == 1) ks[i] = *(const f32x4*)(a.c.ks + hf[i].row + 4 * g);
    }
  };
  auto load_v = [&](const Half* hf) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const char* base = (const char*)a.c.v + hf[i].row * (D * E);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const char* src = base + (voff + e * (D * E));
        uint32_t* dst = vw[4 * i + e];
        if constexpr (VW == 1) dst[0] = *(const uint32_t*)src;
        if constexpr (VW == 2) {
          const uint2 w = *(const uint2*)src;
          dst[0] = w.x; dst[1] = w.y;
        }
        if constexpr (VW >= 4) {
#pragma unroll
          for (int j = 0; j < VW / 4; ++j) {
            const u32x4 w = *(const u32x4*)(src + 16 * j);
            dst[4 * j] = w[0]; dst[4 * j + 1] = w[1]; dst[4 * j + 2] = w[2]; dst[4 * j + 3] = w[3];
          }
        }
      }
      if (E == 1) vs[i] = *(const f32x4*)(a.c.vs + hf[i].row + 4 * g);
    }
  };

  f32x4 o[VC];
#pragma unroll
  for (int j = 0; j < VC; ++j) o[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = kLowest, l = 0.f;

  int t = begin + wave * kStep;
  Half cur[2], nxt[2];
  if (t < end) {
    cur[0] = half_at(t);
    cur[1] = half_at(t + 16);
    load_k(cur);
    load_v(cur);
  }
  for (; t < end; t += kRound) {
    const bool more = t + kRound < end;
    if (more) {
      nxt[0] = half_at(t + kRound);
      nxt[1] = half_at(t + kRound + 16);
    }
    // scores of tokens 16 i + 4 g + e for head c16
    f32x4 s[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      s[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int mm = 0; mm < QF; ++mm) {
        u32x4 kk;
        if constexpr (E == 2) {
          kk = kf[i][mm];
        } else {
          const uint32_t w0 = kf[i][mm >> 1][2 * (mm & 1)], w1 = kf[i][mm >> 1][2 * (mm & 1) + 1];
          kk = u32x4{codes2<FMT, false>(w0), codes2<FMT, true>(w0), codes2<FMT, false>(w1), codes2<FMT, true>(w1)};
        }
        s[i] = mfma16(kk, qf[mm], s[i]);
      }
      if (E == 1) s[i] *= ks[i] * a.scale2;
      else s[i] *= a.scale2;
    }
    f32x4 vsc[2];
    if (E == 1) { vsc[0] = vs[0]; vsc[1] = vs[1]; }
    const bool full = cur[0].ok && cur[1].ok && t >= lo && t + kStep <= end;
    if (!full) {
      // what lies outside the counted tokens has no effect whatever its bits:
      // scores -inf, V and its scale 0
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tt = t + 16 * i + 4 * g + e;
          const bool in = cur[i].ok && tt >= lo && tt < end;
          s[i][e] = in ? s[i][e] : -__builtin_inff();
          if (E == 1) vsc[i][e] = in ? vsc[i][e] : 0.f;
#pragma unroll
          for (int w = 0; w < VW; ++w) vw[4 * i + e][w] = in ? vw[4 * i + e][w] : 0u;
        }
    }
    if (more) load_k(nxt);
    float top = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                      fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
    if (__any(top > m + kLazy)) {
      top = xor32_max(xor16_max(top));         // the head's four lanes agree on the maximum
      const float mn = fmaxf(m, top), r = exp2_(m - mn);
      m = mn;
      l *= r;
#pragma unroll
      for (int j = 0; j < VC; ++j) o[j] *= r;
    }
    // p in two bfloat16 parts (their sum is p to 2^-16): the weights reach the
    // sums with what fp32 arithmetic on them would keep
    u32x4 ph, pl;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        float p0 = exp2_(s[i][e] - m), p1 = exp2_(s[i][e + 1] - m);
        l += p0 + p1;
        if (E == 1) { p0 *= vsc[i][e]; p1 *= vsc[i][e + 1]; }
        const uint32_t hi = pack2(p0, p1);
        ph[2 * i + e / 2] = hi;
        pl[2 * i + e / 2] = pack2(p0 - lo_bf(hi), p1 - hi_bf(hi));
      }
#pragma unroll
    for (int j = 0; j < VC; ++j) {
      u32x4 vv;
      if constexpr (E == 2) {
#pragma unroll
        for (int w = 0; w < 4; ++w)
          vv[w] = __builtin_amdgcn_perm(vw[2 * w + 1][j >> 1], vw[2 * w][j >> 1], j & 1 ? 0x07060302u : 0x05040100u);
      } else {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          // bytes j and j + 1 of both tokens; the odd channel uses the upper half
          const uint32_t pr = __builtin_amdgcn_perm(vw[2 * w + 1][j >> 2], vw[2 * w][j >> 2],
                                                    (j & 2) ? 0x07030602u : 0x05010400u);
          vv[w] = j & 1 ? codes2<FMT, true>(pr) : codes2<FMT, false>(pr);
        }
      }
      o[j] = mfma16(vv, ph, o[j]);
      o[j] = mfma16(vv, pl, o[j]);
    }
    if (more) {
      load_v(nxt);
      cur[0] = nxt[0];
      cur[1] = nxt[1];
    }
  }

  // join the waves: O^T tile j, register i of lane (h, g) is channel
  // VC (4 g + i) + j of head h
  l = xor32_sum(xor16_sum(l));
  if (g == 0) { sm[wave][c16] = m; sl[wave][c16] = l; }
  if (c16 < nh) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < VC; ++j) so[wave][c16][VC * (4 * g + i) + j] = o[j][i];
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < nh * D; idx += 256) {
    const int h = idx / D, d = idx % D;
    float M = sm[0][h];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) M = fmaxf(M, sm[w][h]);
    float L = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float r = exp2_(sm[w][h] - M);
      L += sl[w][h] * r;
      y += so[w][h][d] * r;
    }
    const int64_t row = (int64_t)b * a.hq + head0 + h;
    if (p.nch > 1) {
      p.part[(row * p.nch + chunk_id) * D + d] = y;
      if (d == 0) p.ml[row * p.nch + chunk_id] = make_float2(M, L);
      continue;
    }
    y = L == 0.f ? 0.f : y / L;
    if (a.out_bf16) ((uint16_t*)a.out)[row * D + d] = (uint16_t)f2bf(y);
    else ((float*)a.out)[row * D + d] = y;
    if (d == 0 && a.lse) a.lse[row] = L == 0.f ? -__builtin_inff() : (M + log2_(L)) * 0.6931471805599453f;
  }
}

// Joins the chunks of one query head: a workgroup per row, wave w takes chunks
// w, w + 4, .. in order, then the waves in order.
template <int D>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, Plan p) {
  constexpr int N = D / 64;
  __shared__ float so[kWaves][D], sl[kWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = blockIdx.x;
  const int b = (int)(row / a.hq);
  const int len = min(max(a.lens[b], 0), a.max_len);
  const int lo = a.window && len > a.window ? len - a.window : 0;
  const int n = max(1, (len - (lo & ~(kStep - 1)) + p.chunk - 1) / p.chunk);
  const float2* ml = p.ml + row * p.nch;
  const float* part = p.part + row * p.nch * D;
  float M = kLowest;
  for (int c = lane; c < n; c += 64) M = fmaxf(M, ml[c].x);
  M = row16_max(M);
  M = xor32_max(xor16_max(M));
  float L = 0.f, y[N];
#pragma unroll
  for (int i = 0; i < N; ++i) y[i] = 0.f;
  for (int c = wave; c < n; c += kWaves) {
    const float2 v = ml[c];
    const float r = exp2_(v.x - M);
    L += v.y * r;
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] += part[(int64_t)c * D + lane + 64 * i] * r;
  }
  if (lane == 0) sl[wave] = L;
#pragma unroll
  for (int i = 0; i < N; ++i) so[wave][lane + 64 * i] = y[i];
  __syncthreads();
  const int d = threadIdx.x;
  if (d >= D) return;
  float Z = 0.f, o = 0.f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) { Z += sl[w]; o += so[w][d]; }
  o = Z == 0.f ? 0.f : o / Z;
  if (a.out_bf16) ((uint16_t*)a.out)[row * D + d] = (uint16_t)f2bf(o);
  else ((float*)a.out)[row * D + d] = o;
  if (d == 0 && a.lse) a.lse[row] = Z == 0.f ? -__builtin_inff() : (M + log2_(Z)) * 0.6931471805599453f;
}

inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }

Plan make_plan(const KvCache& c, int B, int hq, int max_len, int window) {
  Plan p{};
  p.G = hq / c.heads;
  p.ht = (p.G + 15) / 16;
  const int tp = c.ps / 16;
  p.tpm = tp == 1 ? 0u : (uint32_t)(((1ull << 32) + tp - 1) / tp);
  // the tokens a sequence can span: a window begins anywhere in a step
  int64_t span = max_len;
  if (window && window + (int64_t)kStep - 1 < span) span = window + (int64_t)kStep - 1;
  const int64_t units = (int64_t)B * c.heads * p.ht;
  const int64_t want = 2048;
  int64_t chunk = (span * units / want + kRound - 1) / kRound * kRound;
  if (chunk < 2 * kRound) chunk = 2 * kRound;
  p.chunk = (int)chunk;
  p.nch = (int)((span + chunk - 1) / chunk);
  if (p.nch < 1) p.nch = 1;
  return p;
}

template <int FMT, int D>
hipError_t run(const AttnArgs& a, const Plan& p, hipStream_t s) {
  const int64_t grid = (int64_t)a.B * a.c.heads * p.ht * p.nch;
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  attn_chunk_kernel<FMT, D><<<(unsigned)grid, 256, 0, s>>>(a, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.nch == 1) return e;
  attn_join_kernel<D><<<(unsigned)(a.B * a.hq), 256, 0, s>>>(a, p);
  return hipGetLastError();
}

template <int FMT>
hipError_t run_d(const AttnArgs& a, const Plan& p, hipStream_t s) {
  if (a.c.D == 64) return run<FMT, 64>(a, p, s);
  if (a.c.D == 128) return run<FMT, 128>(a, p, s);
  return run<FMT, 256>(a, p, s);
}

}  // namespace

size_t attn_workspace_bytes(const KvCache& c, int B, int hq, int max_len, int window) {
  const Plan p = make_plan(c, B, hq, max_len, window);
  if (p.nch == 1) return 0;
  const size_t n = (size_t)B * hq * p.nch;
  return align256(n * c.D * 4) + align256(n * 8);
}

hipError_t launch_attn_decode(const AttnArgs& a, hipStream_t s) {
  Plan p = make_plan(a.c, a.B, a.hq, a.max_len, a.window);
  p.part = a.ws;
  p.ml = (float2*)((char*)a.ws + align256((size_t)a.B * a.hq * p.nch * a.c.D * 4));
  if (a.c.format == KV_BF16) return run_d<KV_BF16>(a, p, s);
  if (a.c.format == KV_E4M3) return run_d<KV_E4M3>(a, p, s);
  return run_d<KV_INT8>(a, p, s);
}

}  // namespace lcp
