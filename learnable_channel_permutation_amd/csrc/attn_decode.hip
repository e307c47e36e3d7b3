// Attention of one new token of each sequence over the paged cache.
//
//   z_t = scale q.k_t,  out = sum_t exp(z_t - m) v_t / sum_t exp(z_t - m)
//
// Every cached element is used by the G query heads of its group only (2 G
// flops a byte with 8-bit codes), so the bytes of K and V bound the operator.
// They are read once, with the running maximum and sum of the softmax; many
// workgroups share a long sequence and a second kernel joins their sums.
//
// A wave takes 32 tokens at a time and keeps everything in registers, from the
// loads to the matrix instructions (16x16x32 bf16, fp32 sums):
//   S[token][head] = K Q^T   A = K rows as loaded, B = Q. Lane (r, g) = (lane %
//     16, lane / 16) loads 16-byte pieces g, g + 4, .. of token r's row; which
//     channels meet in one product does not matter as long as Q's fragment
//     holds the same ones.
//   The result leaves lane (h, g) with tokens 4g .. 4g+3 of each half of the 32
//     for head h: a softmax over registers, no exchange between lanes except
//     for a new maximum.
//   O^T[channel][head] += V^T P^T   B = P as it stands in the registers: lane
//     (h, g) supplies K slots 8g .. 8g+7, which are the tokens named above. So
//     lane (c, g) loads those eight tokens' channels VP c .. of V, and the
//     transposition is a byte permutation within the lane.
// 8-bit codes become bf16 exactly; their scales multiply the scores and the
// weights. Groups of fewer than 16 heads leave columns of the products empty,
// which costs nothing while the bytes bound it. In larger groups two tiles of 16
// heads share a wave's loads; beyond that K and V are read again, from the L2 when
// the workgroups meet there.
//
// Measured (us; bytes of K, V and scales over time), 64 heads in 8 groups of 128
// channels unless said: 128 sequences up to 8192, bf16, 2.15 GB 323 (6.6 TB/s);
// 2 x 131071 int8, 32 heads, 448 MB 76 (5.9); 48 up to 4096 fp8, 203 MB 43 (4.8);
// 24 windows of 4096, 16 heads of 256, bf16, 345 MB 63 (5.5); 1 x 333 bf16, 32
// heads of their own, 7.0 (latency). One workgroup a query head, a
// wave a token, took 11830, 58755, 2861, 4036 and 92.
#include <algorithm>

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

// How the work is dealt. A unit is one sequence, one key/value head and up to
// 16 HT of its query heads (HT tiles of 16, which share the loads of K and V); its
// work is counted in steps.
//   direct (wgs == 0): a workgroup a unit, no second kernel. Where no unit can
//     have more than kDirect bytes of K (kDirectMany with many units).
//   else: the steps of all units in a row, each unit led by kExtra steps that
//     stand for what beginning and ending it costs, cut into parts that differ
//     by one step at most, whatever the sequences' lengths are. A workgroup finds
//     its part from the lengths and writes a unit that it holds whole to the
//     output, a unit's piece to the workspace: at most two, in its places 0 (its
//     first unit) and 1 (its last). Whoever has a unit's first step notes where
//     the first piece is and how many there are, and the second kernel joins the
//     pieces of each unit in order.
struct Plan {
  int wgs;               // workgroups launched: parts at most
  int G, tile, gu;       // query heads of a group, of a unit at most (16 HT), and units of a group
  int units;             // units of a sequence: heads * gu
  int nh;                // query heads of a unit (a group's last one may have fewer)
  uint32_t tpm;          // ceil(2^32 / (page_size / 16)): page of a 16-token tile by a high product
  bool space;            // whether calls of this length can be dealt: need the workspace
  float* part;           // [2 wgs][nh][D]
  float2* ml;            // [2 wgs][nh] maximum and sum
  int2* cuts;            // [B][units] place of the first piece, number of pieces
};
// Direct against dealt with its second kernel, us a pass, fp8, 8 / 32 / 128 / 264 / 512
// / 1024 units with K of half to all of: 96 KB 8.5 9.7 10.2 17.6 19.1 36.7 against 10.4
// 11.0 13.4 17.6 25.2 41.1; 128 KB 10.1 11.2 12.1 21.7 23.8 44.8 against 10.1 10.9 13.8
// 18.9 28.9 48.4; 160 KB 11.5 13.4 14.0 25.1 27.4 54.2 against 10.5 11.0 15.3 21.0 32.8
// 56.8; 192 KB 13.0 15.1 16.1 29.2 32.1 63.3 against 10.9 11.2 16.0 23.0 36.9 65.2; 256
// KB 16.9 18.8 20.1 37.5 41.3 81.7 against 11.0 11.4 17.8 27.9 45.0 81.7 (bf16 alike).
// So direct up to 128 KB, and up to 192 where every compute unit has a unit, which loses
// where a few units more than compute units make a second turn (264). A compute unit
// takes in about 50 KB a us, so that a direct workgroup of eight waves instead of four
// was slower (1 x 1000: 10.9 us).
constexpr int kDirect = 128 << 10, kDirectMany = 192 << 10;
// Cost of beginning and ending a unit, in steps: 4, 8, 12, 18 gave 47.4, 45.4, 45.8,
// 47.2 us at 48 sequences of 1 to 4096, fp8; 56.9, 56.1, 58.1, 59.7 at 128 up to 1000,
// bf16; 18.4, 16.6, 17.6, 17.4 at 12 up to 3000 of 256 int8 channels. Sequences of like
// lengths (half of the largest at least) differ by 3 % between 8 and 12.
constexpr int kExtra = 8;

// How many parts the work is cut into, by its cost and the bytes of a step: parts of
// 64 KB at least, and one a compute unit. A workgroup's four waves keep enough loads
// in flight for it, and fewer streams reach more of the bandwidth; two workgroups a
// unit pay only where conversions and unit ends, not the bytes, take the time: 8-bit
// codes with 64 channels, or with 128 where the units are many and short.
// 256 / 512 / 768 parts, us: bf16 128 x 8192 323 / 334 / 341, 24 windows of 4096 (256
// channels) 63.3 / 66.6 / -, 1 x 131071 87.2 / 90.9 / 93.9, 64 x 8000 (64 channels)
// 85.7 / 88.7 / 90.2; int8 2 x 131071 75.3 / 78.1 / 80.0. Smaller work, with 768 parts
// of 96 KB at least against this: 1 x 131071 of one head 24.4 / 19.3, 8 x 3000 22.2 /
// 16.8, 1 x 40000 18.8 / 15.8.
// 256 / 512 parts of 8-bit codes, us (fp8; int8 is 2 % higher). 64 channels: 11 x 3000
// 15.7 / 15.1, 30 x 3000 28.4 / 24.0, 5 x 8000 17.4 / 16.2, 64 x 8000 118 / 93, 4 x 30000
// 32.4 / 27.9. 128 channels, 64 heads in 8 groups, lengths from 1 on, by the cost of the
// work in thousands of steps: 8 (30 x 1600) 19.2 / 20.0, 9 (16 x 4096) 21.2 / 21.9, 14 (24
// x 4096) 27.5 / 27.9, 14 (32 x 3000) 27.3 / 27.8, 16 (60 x 1600) 31.5 / 29.1, 21 (36 x
// 4096) 37.0 / 36.3, 28 (64 x 3000) 47.3 / 44.7, 28 (48 x 4096) 46.1 / 43.9: from 12 on;
// and by the mean cost of a unit: 39 (64 x 2000) 37.5 / 35.3, 55 (64 x 3000) 47.3 / 44.7,
// 72 (96 x 4096) 80.0 / 79.6, 102 (32 x 6000) 42.9 / 43.4, 102 (64 x 6000) 78.1 / 76.8,
// 133 (24 x 8000) 42.6 / 43.4, 258 (16 x 16000) 52.0 / 53.0: below 96. Sequences of like
// lengths (half to one and a half of the mean) gain nothing: 36 x 1700 29.9 / 31.1, 50 x
// 1700 39.6 / 40.0, 45 x 2000 39.8 / 40.6, 100 x 2500 94.5 / 96.0; the cut does not look
// at how they differ.
constexpr int most_parts(int E, int D) { return E == 1 && D <= 128 ? 512 : 256; }
template <int E, int D>
__device__ __forceinline__ uint32_t parts_of(uint32_t all, uint32_t units) {
  constexpr uint32_t least = (64 << 10) / (2 * kStep * D * E);
  const bool two = most_parts(E, D) == 512 && all >= (D == 64 ? 1 : 3) * 512 * least && (D == 64 || all / 96 < units);
  return two ? 512u : min(256u, max(1u, all / least));
}

// The cut of `all` steps.
struct Cut {
  uint32_t parts, q, r;        // the first r parts have q + 1 steps, the others q
  __device__ __forceinline__ Cut(uint32_t all, uint32_t n) : parts(n) {
    q = all / parts;
    r = all - q * parts;
  }
  __device__ __forceinline__ uint32_t start(uint32_t i) const { return i * q + min(i, r); }
  __device__ __forceinline__ uint32_t part_of(uint32_t x) const {
    const uint32_t big = r * (q + 1);
    return x < big ? x / (q + 1) : r + (x - big) / q;
  }
};

// An index array entry at an address that is the same for the whole wave, read
// through the scalar cache (the kernel that reads it does not write it): it does
// not queue behind the loads of K and V, which return in order.
__device__ __forceinline__ int uniform(const int* p, int64_t i) {
  typedef const int __attribute__((address_space(4))) * ConstPtr;
  return ((ConstPtr)(uintptr_t)p)[i];
}

// A store that the compiler knows to be to global memory. Through a pointer it
// cannot place it makes flat stores, whose completion is out of order with the
// loads: every wait in the kernel then becomes one for all of them.
template <typename T>
__device__ __forceinline__ void put(void* p, int64_t i, T v) {
  typedef T __attribute__((address_space(1))) * GlobalPtr;
  ((GlobalPtr)(uintptr_t)p)[i] = v;
}
// Channels 4 td .. of a finished row from its unscaled sums, and (td 0) its
// log-sum-exp, from its maximum and sum in base 2.
template <int D>
__device__ __forceinline__ void put_row(const AttnArgs& a, int64_t row, int td, f32x4 y, float m, float l) {
  if (l == 0.f) y = f32x4{0.f, 0.f, 0.f, 0.f};
  else y /= l;
  const int64_t i = row * (D / 4) + td;
  if (a.out_bf16) put<u32x2>(a.out, i, u32x2{pack2(y[0], y[1]), pack2(y[2], y[3])});
  else put<f32x4>(a.out, i, y);
  if (td == 0 && a.lse) put<float>(a.lse, row, l == 0.f ? -__builtin_inff() : (m + log2_(l)) * 0.6931471805599453f);
}

// Tokens of a sequence: the first counted one, the end, and the steps between.
struct Span {
  int lo, end, steps;
  __device__ __forceinline__ uint32_t cost() const { return steps ? steps + kExtra : 0; }
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, int len) {
  Span s;
  s.end = min(max(len, 0), a.max_len);
  s.lo = a.window && s.end > a.window ? s.end - a.window : 0;
  s.steps = (s.end - (s.lo & ~(kStep - 1)) + kStep - 1) / kStep;
  return s;
}

// Cost (of one unit) of the sequences before each thread's first, threadIdx.x *
// per, and of all, by the 256 threads of a workgroup.
__device__ __forceinline__ uint32_t cost_before(const AttnArgs& a, int per, uint32_t* total, uint32_t* lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t mine = 0;
  for (int i = 0; i < per; ++i) {
    const int b = threadIdx.x * per + i;
    if (b < a.B) mine += span_of(a, a.lens[b]).cost();
  }
  uint32_t sum = mine;
  for (int k = 1; k < 64; k <<= 1) {
    const uint32_t v = __shfl_up(sum, k, 64);
    if (lane >= k) sum += v;
  }
  if (lane == 63) lds[wave] = sum;
  __syncthreads();
  *total = __builtin_amdgcn_readfirstlane(lds[0] + lds[1] + lds[2] + lds[3]);
  for (int w = 0; w < wave; ++w) sum += lds[w];
  return sum - mine;
}

// A half step: 16 tokens, all of one page.
struct Half {
  int64_t row;           // first cache row
  int ok;                // whether the page exists and the half begins before the end
};

template <typename T>
__device__ __forceinline__ T once(const void* p) { return __builtin_nontemporal_load((const T*)p); }

// Waves per SIMD that the registers leave (checked by the compiler).
constexpr int waves_for(int D, int HT) { return (D == 64 ? 4 : D == 128 ? 3 : 2) - (HT - 1); }

template <int FMT, int D, int HT, bool DEALT>
__global__ __launch_bounds__(256, waves_for(D, HT)) void attn_units_kernel(AttnArgs a, Plan p) {
  constexpr int E = FMT == KV_BF16 ? 2 : 1;
  constexpr int KL = D * E / 64;               // 16-byte K loads of a lane for 16 tokens
  constexpr int VC = D / 16;                   // channels of V a lane holds of each of its 8 tokens
  constexpr int VW = VC * E / 4;               // their 32-bit words
  constexpr int VP = VC * E > 16 ? 16 / E : VC;        // those that are adjacent: 16 bytes at most, so that the 16
                                               // lanes of a token cover whole lines with every load
  constexpr int QF = D / 32;                   // products over the channels
  constexpr int OS = D + 4;                    // row stride of the waves' sums in LDS
  // Where Q's fragments are: in registers, or (256 bf16 channels, whose K, V and
  // sums leave no room for them) in LDS, a quarter written by each wave
  constexpr bool QL = D == 256 && E == 2;
  constexpr int QR = QL ? QF / kWaves : QF;    // fragments that a wave loads
  __shared__ float so[kWaves][16 * HT][OS];
  __shared__ float sm[kWaves][16 * HT], sl[kWaves][16 * HT];
  __shared__ u32x4 sq[QL ? QF : 1][QL ? 64 : 1];
  __shared__ uint32_t scan[kWaves + 2];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, g = lane >> 4;

  // this workgroup's part: sequence b, unit u of it, from v of its cost on, `left`
  // in all. What steers the loops has to be uniform for the compiler too: as lane
  // values they cost 40 spilled registers (2 x 131071 int8: 150 us)
  int b, u, v = 0, left = 1, place = 0;
  uint32_t start = 0;                          // where the unit begins in the row of all
  Cut cut(1, 1);
  if (DEALT) {
    const int per = (a.B + 255) / 256;
    uint32_t all;
    uint32_t at = cost_before(a, per, &all, scan);
    all *= p.units;
    cut = Cut(all, parts_of<E, D>(all, (uint32_t)a.B * p.units));
    // neighbouring parts on one XCD (workgroups go to the eight in turn): head
    // tiles of one key/value head then meet in its L2
    const uint32_t run = (cut.parts + 7) >> 3, rank = (blockIdx.x & 7) * run + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= run || rank >= cut.parts || all == 0) return;
    const uint32_t x = cut.start(rank);
    left = cut.start(rank + 1) - x;
    place = 2 * rank;
    for (int i = 0; i < per; ++i) {
      const int bb = threadIdx.x * per + i;
      if (bb >= a.B) break;
      const uint32_t n = span_of(a, a.lens[bb]).cost();
      if (at * p.units <= x && x < (at + n) * p.units) {
        scan[kWaves] = bb;
        scan[kWaves + 1] = x - at * p.units;
      }
      at += n;
    }
    __syncthreads();
    b = __builtin_amdgcn_readfirstlane(scan[kWaves]);
    const int in = __builtin_amdgcn_readfirstlane(scan[kWaves + 1]);
    const int n = span_of(a, uniform(a.lens, b)).cost();
    u = in / n;
    v = in - u * n;
    start = x - v;
  } else {
    b = blockIdx.x / p.units;
    u = blockIdx.x % p.units;
  }

  // the unit (or the piece of it) at work: its tokens from lo to end, this wave's
  // next step t, its heads, and whether it is whole
  int lo, end, t, hk, nh, head0, last;
  bool whole;
  const int* pages;
  u32x4 qf[HT][QR];
  const int tp = a.c.ps >> 4;
  // the page of the 16 tokens from t on (past the end: of the last ones), its
  // number, and the cache row; row 0 stands in where there is nothing to read
  auto page_at = [&](int t) {
    const int tile = min(t >> 4, last);
    return p.tpm == 0 ? tile : (int)__umulhi((uint32_t)tile, p.tpm);      // 0: one tile a page
  };
  auto half_at = [&](int t, int id) {
    Half r;
    r.ok = t < end && id >= 0 && id < a.c.pages;
    const int64_t row = ((int64_t)id * a.c.heads + hk) * a.c.ps + (min(t >> 4, last) - page_at(t) * tp) * 16;
    r.row = r.ok ? row : 0;
    return r;
  };

  u32x4 kf[2][KL];
  uint32_t vw[8][VW];
  f32x4 ks[2], vs[2];
  const uint32_t koff = c16 * (D * E) + 16 * g, voff = 4 * g * (D * E) + c16 * (VP * E);
  auto load_k = [&](const Half* hf) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const char* base = (const char*)a.c.k + hf[i].row * (D * E);
#pragma unroll
      for (int j = 0; j < KL; ++j) kf[i][j] = once<u32x4>(base + (koff + 64 * j));
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
        if constexpr (VW == 1) dst[0] = once<uint32_t>(src);
        if constexpr (VW == 2) {
          const u32x2 w = once<u32x2>(src);
          dst[0] = w[0]; dst[1] = w[1];
        }
        if constexpr (VW >= 4) {
#pragma unroll
          for (int j = 0; j < VW / 4; ++j) {
            const u32x4 w = once<u32x4>(src + 256 * j);
            dst[4 * j] = w[0]; dst[4 * j + 1] = w[1]; dst[4 * j + 2] = w[2]; dst[4 * j + 3] = w[3];
          }
        }
      }
      if (E == 1) vs[i] = *(const f32x4*)(a.c.vs + hf[i].row + 4 * g);
    }
  };

  // loads run a step ahead, page numbers two
  Half cur[2], nxt[2];
  int id0, id1;
  // takes the unit at (b, u, v) up and issues its first loads; false if the part
  // ends before its first step
  auto begin_unit = [&]() {
    if (left <= 0 || b >= a.B) return false;
    const Span sp = span_of(a, uniform(a.lens, b));
    int r0 = 0, r1 = sp.steps;
    if (DEALT) {
      r0 = max(0, v - kExtra);
      r1 = min(r1, v + left - kExtra);
      left -= sp.steps + kExtra - v;
      v = 0;
      if (r1 <= r0) return false;
      start += sp.steps + kExtra;
    } else {
      left = 0;
    }
    whole = r0 == 0 && r1 == sp.steps;
    hk = u / p.gu;
    const int h0 = u % p.gu * (16 * HT);
    nh = min(16 * HT, p.G - h0);
    head0 = hk * p.G + h0;
    lo = sp.lo;
    const int begin = lo & ~(kStep - 1);
    end = min(sp.end, begin + r1 * kStep);
    last = max(end - 1, 0) >> 4;
    t = begin + r0 * kStep + wave * kStep;
    pages = a.pages + (int64_t)b * a.max_pages;
    // Q fragments: head c16 of each tile, the channels that the K loads bring
#pragma unroll
    for (int h = 0; h < HT; ++h)
#pragma unroll
      for (int m = 0; m < QR; ++m) {
        const int f = QL ? QR * wave + m : m;
        const int d = E == 2 ? 32 * f + 8 * g : 64 * (f >> 1) + 16 * g + 8 * (f & 1);
        qf[h][m] = u32x4{0, 0, 0, 0};
        if (16 * h + c16 < nh) qf[h][m] = *(const u32x4*)(a.q + b * a.qrow + (int64_t)(head0 + 16 * h + c16) * D + d);
      }
    cur[0] = half_at(t, uniform(pages, page_at(t)));
    cur[1] = half_at(t + 16, uniform(pages, page_at(t + 16)));
    id0 = uniform(pages, page_at(t + kRound));
    id1 = uniform(pages, page_at(t + kRound + 16));
    // Q has come by the time the page numbers have; with this wait for it (vmcnt 0
    // alone) the first product waits for K's loads only, not for V's behind them
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0x0f70);
    load_k(cur);
    __builtin_amdgcn_sched_barrier(0);         // K before V, for the same reason
    load_v(cur);
    __builtin_amdgcn_sched_barrier(0);
    if (DEALT && r0 == 0 && threadIdx.x == 0) {
      const uint32_t pieces = whole ? 1 : cut.part_of(start - 1) - (place >> 1) + 1;
      put<u32x2>(p.cuts, (int64_t)b * p.units + u, u32x2{(uint32_t)place, pieces});
    }
    return true;
  };

  f32x4 o[HT][VC];
  float m[HT], l[HT];
  bool done = false;                           // whether o, m and l hold a finished unit: the last one
  int nh_ = 0, place_ = 0;
  bool whole_ = false;
  int64_t row0 = 0;
  for (;;) {
    // the next unit's first loads fly while the last one is joined and written
    const bool more = begin_unit();
    if (done) {
      // join the waves: O^T tile j, register i of lane (h, g) is channel
      // 16 VP (j / VP) + VP (4 g + i) + j % VP of head h
#pragma unroll
      for (int t = 0; t < HT; ++t) {
        const int h = 16 * t + c16;
        l[t] = xor32_sum(xor16_sum(l[t]));
        if (g == 0) { sm[wave][h] = m[t]; sl[wave][h] = l[t]; }
        if (h < nh_) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < VC; j += 4)
              *(f32x4*)&so[wave][h][16 * VP * (j / VP) + VP * (4 * g + i) + j % VP] =
                  f32x4{o[t][j][i], o[t][j + 1][i], o[t][j + 2][i], o[t][j + 3][i]};
        }
      }
      __syncthreads();
      for (int idx = threadIdx.x; idx < nh_ * (D / 4); idx += 256) {
        const int h = idx / (D / 4), td = idx % (D / 4);
        float M = sm[0][h];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) M = fmaxf(M, sm[w][h]);
        float L = 0.f;
        f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          const float r = exp2_(sm[w][h] - M);
          L += sl[w][h] * r;
          y += *(const f32x4*)&so[w][h][4 * td] * r;
        }
        if (whole_) {
          put_row<D>(a, row0 + h, td, y, M, L);
        } else {
          const int at = place_ * p.nh + h;
          put<f32x4>(p.part, (int64_t)at * (D / 4) + td, y);
          if (td == 0) put<u32x2>(p.ml, at, u32x2{__float_as_uint(M), __float_as_uint(L)});
        }
      }
      if (!more) return;
      __syncthreads();                         // the sums in LDS have been read
    }
    if (!more) return;
    if (QL) {
#pragma unroll
      for (int f = 0; f < QR; ++f) sq[QR * wave + f][lane] = qf[0][f];       // HT is 1
      __syncthreads();
    }
#pragma unroll
    for (int h = 0; h < HT; ++h) {
#pragma unroll
      for (int j = 0; j < VC; ++j) o[h][j] = f32x4{0.f, 0.f, 0.f, 0.f};
      m[h] = kLowest;
      l[h] = 0.f;
    }
    for (; t < end; t += kRound) {
      nxt[0] = half_at(t + kRound, id0);
      nxt[1] = half_at(t + kRound + 16, id1);
      id0 = uniform(pages, page_at(t + 2 * kRound));
      id1 = uniform(pages, page_at(t + 2 * kRound + 16));
      // scores of tokens 16 i + 4 g + e for head c16 of each tile
      f32x4 s[HT][2];
#pragma unroll
      for (int h = 0; h < HT; ++h) s[h][0] = s[h][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int mm = 0; mm < QF; ++mm) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          u32x4 kk;
          if constexpr (E == 2) {
            kk = kf[i][mm];
          } else {
            const uint32_t w0 = kf[i][mm >> 1][2 * (mm & 1)], w1 = kf[i][mm >> 1][2 * (mm & 1) + 1];
            kk = u32x4{codes2<FMT, false>(w0), codes2<FMT, true>(w0), codes2<FMT, false>(w1), codes2<FMT, true>(w1)};
          }
#pragma unroll
          for (int h = 0; h < HT; ++h)
            s[h][i] = mfma16(kk, QL ? sq[QL ? mm : 0][QL ? lane : 0] : qf[h][QL ? 0 : mm], s[h][i]);
        }
      }
#pragma unroll
      for (int h = 0; h < HT; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (E == 1) s[h][i] *= ks[i] * a.scale2;
          else s[h][i] *= a.scale2;
        }
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
#pragma unroll
            for (int h = 0; h < HT; ++h) s[h][i][e] = in ? s[h][i][e] : -__builtin_inff();
            if (E == 1) vs[i][e] = in ? vs[i][e] : 0.f;
#pragma unroll
            for (int w = 0; w < VW; ++w) vw[4 * i + e][w] = in ? vw[4 * i + e][w] : 0u;
          }
      }
      // the next step's K flies during the softmax and the products with V, its V
      // during the next scores. Unconditional (past the end: row 0 of the cache),
      // so that the waits can count on the loads in between
      load_k(nxt);
      __builtin_amdgcn_sched_barrier(0);
      // p in two bfloat16 parts (their sum is p to 2^-16): the weights reach the
      // sums with what fp32 arithmetic on them would keep
      u32x4 ph[HT], pl[HT];
#pragma unroll
      for (int h = 0; h < HT; ++h) {
        float top = fmaxf(fmaxf(fmaxf(s[h][0][0], s[h][0][1]), fmaxf(s[h][0][2], s[h][0][3])),
                          fmaxf(fmaxf(s[h][1][0], s[h][1][1]), fmaxf(s[h][1][2], s[h][1][3])));
        if (__any(top > m[h] + kLazy)) {
          top = xor32_max(xor16_max(top));       // the head's four lanes agree on the maximum
          const float mn = fmaxf(m[h], top), r = exp2_(m[h] - mn);
          m[h] = mn;
          l[h] *= r;
#pragma unroll
          for (int j = 0; j < VC; ++j) o[h][j] *= r;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            float p0 = exp2_(s[h][i][e] - m[h]), p1 = exp2_(s[h][i][e + 1] - m[h]);
            l[h] += p0 + p1;
            if (E == 1) { p0 *= vs[i][e]; p1 *= vs[i][e + 1]; }
            const uint32_t hi = pack2(p0, p1);
            ph[h][2 * i + e / 2] = hi;
            pl[h][2 * i + e / 2] = pack2(p0 - lo_bf(hi), p1 - hi_bf(hi));
          }
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
#pragma unroll
        for (int h = 0; h < HT; ++h) {
          o[h][j] = mfma16(vv, ph[h], o[h][j]);
          o[h][j] = mfma16(vv, pl[h], o[h][j]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      load_v(nxt);
      cur[0] = nxt[0];
      cur[1] = nxt[1];
    }

    done = true;
    nh_ = nh;
    place_ = place;
    whole_ = whole;
    row0 = (int64_t)b * a.hq + head0;
    place |= 1;
    if (DEALT && left > 0 && ++u == p.units) {
      u = 0;
      do ++b; while (b < a.B && span_of(a, uniform(a.lens, b)).steps == 0);
    }
  }
}

// Joins the pieces of the units that were cut, and answers for sequences
// without tokens. D / 4 threads hold a head's channels, four each. ROWS: a
// workgroup per query head, its thread groups share the pieces (few units of
// many pieces); else a sequence's units go over `groups` workgroups, a thread
// group takes a head at a time. Its three reads in a row (lengths, cuts, pieces)
// bound it: 4.5 us with 1 to 3 MB of pieces.
template <int D, bool ROWS>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, Plan p, int groups) {
  constexpr int TG = 256 / (D / 4);            // thread groups
  constexpr int STEP = ROWS ? TG : 1;          // from a thread group's piece to its next
  __shared__ f32x4 so[TG][D / 4];
  __shared__ float sm[TG], sl[TG];
  const int b = (int)(blockIdx.x / groups), group = (int)(blockIdx.x % groups);
  const bool some = span_of(a, uniform(a.lens, b)).steps > 0;
  const int tg = threadIdx.x / (D / 4), td = threadIdx.x % (D / 4);
  const auto add = [](float& M, float& L, f32x4& y, float m, float l, f32x4 v) {
    const float mn = fmaxf(M, m), r0 = exp2_(M - mn), r1 = exp2_(m - mn);
    L = L * r0 + l * r1;
    y = y * r0 + v * r1;
    M = mn;
  };
  for (int u = ROWS ? group / p.nh : group; u < p.units; u += ROWS ? p.units : groups) {
    const int64_t unit = (int64_t)b * p.units + u;
    const int place0 = uniform((const int*)p.cuts, 2 * unit);
    const int pieces = some ? uniform((const int*)p.cuts, 2 * unit + 1) : 0;
    if (pieces == 1) continue;                 // written whole by its workgroup
    const int h0 = u % p.gu * p.tile, nh = min(p.tile, p.G - h0);
    for (int h = ROWS ? group % p.nh : tg; h < nh; h += ROWS ? p.nh : TG) {        // one writer a row
      float M = kLowest, L = 0.f;
      f32x4 y = {0.f, 0.f, 0.f, 0.f};
      for (int i = ROWS ? tg : 0; i < pieces; i += 4 * STEP) {
        // four pieces' loads together, then one after the other
        f32x4 v[4];
        float2 ml[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int j = i + k * STEP;
          if (j < pieces) {
            // the first piece ends its workgroup's part, the others begin theirs
            const int q = (j == 0 ? place0 : 2 * ((place0 >> 1) + j)) * p.nh + h;
            ml[k] = p.ml[q];
            v[k] = *(const f32x4*)(p.part + (int64_t)q * D + 4 * td);
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (i + k * STEP < pieces) add(M, L, y, ml[k].x, ml[k].y, v[k]);
      }
      if (ROWS) {
        so[tg][td] = y;
        if (td == 0) { sm[tg] = M; sl[tg] = L; }
        __syncthreads();
        if (tg != 0) return;
        for (int w = 1; w < TG; ++w) add(M, L, y, sm[w], sl[w], so[w][td]);
      }
      put_row<D>(a, (int64_t)b * a.hq + u / p.gu * p.G + h0 + h, td, y, M, L);
    }
  }
}

inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }

Plan make_plan(const KvCache& c, int B, int hq, int max_len, int window) {
  Plan p{};
  p.G = hq / c.heads;
  const int tp = c.ps / 16;
  p.tpm = tp == 1 ? 0u : (uint32_t)(((1ull << 32) + tp - 1) / tp);
  // the tokens a sequence can span: a window begins anywhere in a step
  int64_t span = max_len;
  if (window && window + (int64_t)kStep - 1 < span) span = window + (int64_t)kStep - 1;
  const int64_t units1 = (int64_t)B * c.heads * ((p.G + 15) / 16), row = c.D * (c.format == KV_BF16 ? 2 : 1);
  p.space = span * row > kDirect;
  const bool dealt = span * row > (units1 > 256 ? kDirectMany : kDirect);
  // Two head tiles a unit where a group has them, the registers hold them and one
  // tile would read more than 48 MB, or (direct) leave more than a unit for each
  // compute unit: below, half as many units cost more than the bytes. One tile
  // against two, us (32 heads a group, 2 groups): dealt, 4 / 8 / 16 x 4000 bf16, 33 to
  // 131 MB, 12.9 / 13.4, 14.6 / 14.7, 19.0 / 16.2; fp8, 16 to 66 MB, 11.4 / 12.9, 12.3 /
  // 13.7, 14.6 / 14.7; 16 x 4000 of 64 int8 channels, 33 MB, 12.9 / 14.5; direct, 64 /
  // 128 x 500 bf16 12.1 / 12.7, 19.4 / 13.5. One group of 32, 64 x 8192 bf16 48.6 / 33.5.
  const bool enough = dealt ? units1 * span * 2 * row > ((int64_t)48 << 20) : units1 > 256;
  const int HT = p.G > 16 && c.D <= 128 && enough ? 2 : 1;
  p.tile = 16 * HT;
  p.gu = (p.G + p.tile - 1) / p.tile;
  p.units = c.heads * p.gu;
  p.nh = std::min(p.G, p.tile);
  if (dealt) p.wgs = most_parts(c.format == KV_BF16 ? 2 : 1, c.D);
  return p;
}

// The workspace's parts, of either number of tiles: a workspace for the largest
// call serves the smaller ones.
struct Space {
  size_t part, ml, cuts;       // bytes
};
Space space_for(const KvCache& c, int B, const Plan& p) {
  const size_t rows = (size_t)most_parts(c.format == KV_BF16 ? 2 : 1, c.D) * std::min(p.G, c.D <= 128 ? 32 : 16);
  return {align256(2 * rows * c.D * 4), align256(2 * rows * 8),
          align256((size_t)B * c.heads * ((p.G + 15) / 16) * 8)};
}

template <int FMT, int D, int HT>
hipError_t run(const AttnArgs& a, const Plan& p, hipStream_t s) {
  const int64_t units = (int64_t)a.B * p.units;
  if (p.wgs == 0) {
    attn_units_kernel<FMT, D, HT, false><<<(unsigned)units, 256, 0, s>>>(a, p);
    return hipGetLastError();
  }
  attn_units_kernel<FMT, D, HT, true><<<(unsigned)p.wgs, 256, 0, s>>>(a, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // units against rows, us (bf16): 1 unit 58.5 / 24.4 (1 x 131071, 8 heads), 24 units 31.1 /
  // 20.6 (24 x 8192, 32 heads), 64 units 37.3 / 35.9 (64 x 8192, 32 heads), 96 units 40.8 /
  // 40.6 (96 x 8192, 16 heads), 128 units 30.3 / 31.1 (128 x 4000), 256 units 50.2 / 53.8
  if (units <= 64) {
    const int groups = p.units * p.nh;         // four pieces a unit and more, where the sequences are alike
    attn_join_kernel<D, true><<<(unsigned)(a.B * groups), 256, 0, s>>>(a, p, groups);
  } else {
    const int groups = std::min(p.units, std::max(1, 4096 / a.B));
    attn_join_kernel<D, false><<<(unsigned)(a.B * groups), 256, 0, s>>>(a, p, groups);
  }
  return hipGetLastError();
}

template <int FMT>
hipError_t run_d(const AttnArgs& a, const Plan& p, hipStream_t s) {
  if (a.c.D == 256) return run<FMT, 256, 1>(a, p, s);
  if (p.tile == 16) return a.c.D == 64 ? run<FMT, 64, 1>(a, p, s) : run<FMT, 128, 1>(a, p, s);
  return a.c.D == 64 ? run<FMT, 64, 2>(a, p, s) : run<FMT, 128, 2>(a, p, s);
}

}  // namespace

size_t attn_workspace_bytes(const KvCache& c, int B, int hq, int max_len, int window) {
  const Plan p = make_plan(c, B, hq, max_len, window);
  const Space n = space_for(c, B, p);
  return p.space ? n.part + n.ml + n.cuts : 0;
}

hipError_t launch_attn_decode(const AttnArgs& a, hipStream_t s) {
  Plan p = make_plan(a.c, a.B, a.hq, a.max_len, a.window);
  const Space n = space_for(a.c, a.B, p);
  p.part = a.ws;
  p.ml = (float2*)((char*)a.ws + n.part);
  p.cuts = (int2*)((char*)p.ml + n.ml);
  if (a.c.format == KV_BF16) return run_d<KV_BF16>(a, p, s);
  if (a.c.format == KV_E4M3) return run_d<KV_E4M3>(a, p, s);
  return run_d<KV_INT8>(a, p, s);
}

}  // namespace lcp
