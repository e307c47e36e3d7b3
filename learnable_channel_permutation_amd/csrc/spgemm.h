// The 2:4 sparse product on tiles, in bf16 and in 8 bits: one kernel for the deployed
// layer (deploy.hip) and for the one with an epilogue (linear.hip).
#pragma once

#include <type_traits>

#include "common.h"

namespace lcp {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x16 __attribute__((ext_vector_type(16)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void* dep_lds_t;

// How a product's operands are multiplied. The e4m3 instructions add the products of
// one lane (sixteen) with bits below 2^-13 of the largest dropped, 1.5e-5 of a sum's
// size (measured; the dense and the scaled ones alike): less than a bf16 output's 2^-9 of
// a sum as large as its terms, but all of one whose terms cancel (224 terms of size 1 beside
// 16 pairs of +-2^14: 0 for 224). M_E4M3 turns the codes into bf16 instead, exactly.
enum SparseMode { M_BF16 = 0, M_E4M3 = 1, M_E4M3_FAST = 2 };

__device__ __forceinline__ u32x8 cat(u32x4 a, u32x4 b) {
  return u32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}
// Two e4m3 codes (bytes 2 HI and 2 HI + 1 of w) -> a bf16 pair, exactly.
template <bool HI>
__device__ __forceinline__ uint32_t bf16_pair(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
}
__device__ __forceinline__ u32x4 bf16_eight(uint32_t a, uint32_t b) {
  return u32x4{bf16_pair<false>(a), bf16_pair<true>(a), bf16_pair<false>(b), bf16_pair<true>(b)};
}
// A lane's e4m3 operands as those of two bf16 instructions: instruction j takes every
// lane's groups 2j, 2j + 1, 2j + 4 and 2j + 5 of four positions, which are bytes 8j ..
// 8j + 7 of both 16-byte pieces of all lanes' activations.
__device__ __forceinline__ u32x8 half_acts(u32x8 b, int j) {
  return cat(bf16_eight(b[2 * j], b[2 * j + 1]), bf16_eight(b[4 + 2 * j], b[5 + 2 * j]));
}
__device__ __forceinline__ u32x4 half_vals(u32x4 a, int j) { return bf16_eight(a[j], a[2 + j]); }
__device__ __forceinline__ uint32_t half_idx(uint32_t i, int j) {
  return ((i >> (8 * j)) & 0xffu) | ((i >> (8 + 8 * j)) & 0xff00u);
}

// 32 rows x 32 tokens over one fragment's positions (not M_E4M3).
template <int MODE>
__device__ __forceinline__ floatx16 smfma32(u32x4 a, u32x8 b, floatx16 c, uint32_t idx) {
  if constexpr (MODE == M_BF16)
    return __builtin_amdgcn_smfmac_f32_32x32x32_bf16(as_bf16x8(a), __builtin_bit_cast(bf16x16, b), c, (int)idx, 0, 0);
  if constexpr (MODE == M_E4M3_FAST)
    return __builtin_amdgcn_smfmac_f32_32x32x64_fp8_fp8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x8, b), c,
                                                        (int)idx, 0, 0);
}

// Y[t][o] = epilogue of sum_k Ws[o][k] Xp[t][k]. 256 (rows o) x 128 (tokens t) tiles (a
// 4096 x 2048 output is one round of 256 workgroups), 8 waves, K steps of 64
// positions. The two 32-position halves of every K step go to two groups of
// four waves (the K sum is split inside the workgroup): wave v of group g
// computes rows 128 (v / 2) + [0, 128) and tokens 64 (v % 2) + [0, 64) of the
// tile (4 x 2 sparse MFMA blocks) over half g of every step, and at the end
// the groups exchange half of their accumulators through LDS, each adding
// and storing one half. A 128 x 64 wave tile reads 9 KB of fragments for its
// 8 MFMAs of a step; 64 x 64 tiles over both halves would read 13 KB.
// A ring stage holds the 16 weight fragments of one step (16 KB, lane order,
// linear LDS reads), their position words (2 KB) and the 128 x 64 activation
// tile (16 KB, rows swizzled as in the dense GEMM), all moved with
// direct-to-LDS loads; four stages (136 KB of LDS) keep three tiles in flight
// per CU. Pipeline of step kt: the wave's first two MFMAs, the barrier, then
// the next stage's fragments are read into the second register set while the
// last six MFMAs run from the first; the five loads of tile kt + RS - 1 go
// out one at a time between the eight MFMAs (a burst right after the barrier
// stalls every wave on the vector-memory queue).
// SP_NPRE: MFMAs of a step before its barrier; SP_LSPAN: MFMAs the five
// loads are spread over
// e4m3: a fragment holds 64 positions in the same 16 bytes a lane, and two fragments
// of every row group take a step of 128 positions in the same bytes, but for twice the
// position words. Those come in 16-byte loads by the first four waves; the others
// issue one that reads nothing, so that every wave counts the same loads.
constexpr int SP_BM = 256, SP_BN = 128, SP_NT = 512, SP_RS = 4, SP_NL = 5, SP_NPRE = 2, SP_LSPAN = 8;
constexpr int SP_A1 = (SP_BM / 32) * 2 * 1024, SP_B1 = SP_BN * 64 * 2;
template <int MODE>
constexpr int SP_M1 = (SP_BM / 32) * (MODE == M_BF16 ? 256 : 512);
template <int MODE>
constexpr int SP_STAGE = SP_A1 + SP_M1<MODE> + SP_B1;
// the ring, and where the loads that read nothing write
template <int MODE>
constexpr int SP_LDS = SP_RS * SP_STAGE<MODE> + (MODE == M_BF16 ? 0 : 4096);

// Workgroup g of P to a tile, or to a part of K and a tile (SPLIT: `parts` of K); false past
// the last one. Consecutive workgroups of one XCD (id mod 8; P is a multiple of 8 where a
// launch pads it) take a compact group of 4 row panels x all token panels, or, in parts, one
// part's tiles, token panels first: an XCD's L2 then holds a few panels' piece of K, and the weights
// come from memory about once.
template <bool SPLIT>
__device__ __forceinline__ bool sp_tile_coords(int g, int P, int tiles_m, int tiles_n, int parts, int& tm, int& tn,
                                               int& part) {
  int logical = g;
  if ((P & 7) == 0) logical = (g & 7) * (P >> 3) + (g >> 3);
  if constexpr (SPLIT) {
    part = logical / (tiles_m * tiles_n);
    const int rem = logical - part * (tiles_m * tiles_n);
    tm = rem / tiles_n;
    tn = rem - tm * tiles_n;
    return part < parts;
  } else {
    if (logical >= tiles_m * tiles_n) return false;
    const int in_group = 4 * tiles_n;
    const int gid = logical / in_group;
    const int first_m = gid * 4;
    const int gsm = min(tiles_m - first_m, 4);
    const int rem = logical - gid * in_group;
    tm = first_m + rem % gsm;
    tn = rem / gsm;
    part = 0;
    return true;
  }
}

__device__ __forceinline__ int sp_swz(int row, int ch) { return row * 64 + ((ch ^ ((row >> 1) & 7)) << 3); }

// s_waitcnt vmcnt(N) (expcnt and lgkmcnt not waited on)
template <int N>
__device__ __forceinline__ void sp_wait_vmcnt() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// x_row: elements between tokens; steps: K steps of a part (all of them for one part;
// Epi::kSplit: one of several, which the epilogue is told). Epi ends the sums: kRows = 16, store(token, first of 16
// rows, their sums); or kRows = 8, for epilogues that read: a thread then holds eight
// rows of one token after the other, a wave whole lines of two tokens, with fixed(first
// row) read once and load(token, first row) ahead of store(.., two quarters of the rows'
// sums, fixed, loaded).
template <int MODE, int RS, int NPRE, int LSPAN, typename Epi>
__global__ __launch_bounds__(SP_NT, 1) void spgemm_kernel(const u32x4* __restrict__ vals,
                                                          const uint32_t* __restrict__ meta,
                                                          const void* __restrict__ Xp, int64_t x_row, int T, int cout,
                                                          int cin, int steps, Epi epi) {
  constexpr int E = MODE == M_BF16 ? 2 : 1, STAGE = SP_STAGE<MODE>, MOFF = SP_A1, BOFF = SP_A1 + SP_M1<MODE>;
  constexpr int FM = 4, FN = 2, NM = FM * FN, WM = 128, WN = 64, NL = SP_NL;
  static_assert(RS >= 3 && RS % 2 == 0 && (RS - 2) * NL < 64, "ring depth");
  static_assert(8 * FM * 4 * 64 * 16 <= RS * STAGE && SP_BM * SP_BN * 4 <= RS * STAGE, "the accumulator exchange fits in the ring");
  extern __shared__ __attribute__((aligned(16))) unsigned char sp_lds[];
  const int tiles_m = (cout + SP_BM - 1) / SP_BM, tiles_n = (T + SP_BN - 1) / SP_BN;
  const int KF = E == 2 ? cin / 32 : (cin + 63) / 64, KA = (KF + 1) / 2, RG = cout / 32;
  int tm, tn, part;
  if (!sp_tile_coords<Epi::kSplit>(blockIdx.x, gridDim.x, tiles_m, tiles_n, (KA + steps - 1) / steps, tm, tn, part)) return;
  if constexpr (Epi::kSplit) epi.part = part;
  const int m0 = tm * SP_BM, n0 = tn * SP_BN;
  const int t = threadIdx.x, l = t & 63, w = t >> 6;
  const int g = __builtin_amdgcn_readfirstlane(w >> 2), v = w & 3, wm = v >> 1, wn = v & 1;
  const int h = l >> 5, ln = l & 31;
  const int k0 = part * steps, NK = min(KA - k0, steps);          // of KA steps, this part's

  // load o of this thread for K step ks into ring stage `stage`: o < 2 the
  // weight fragment f = 8 o + w (row group f / 2, 32-position half f % 2),
  // o = 2 the position words of row group w, o > 2 activation chunks. The
  // loads go through buffer resources: each lane's byte offset is fixed per
  // tile and a K step moves only the scalar offset; row groups and tokens
  // past the matrices, and (in a step that may be the last, TAIL) K chunks
  // past cin or whole steps past the end, read zeros from an offset past the
  // resource.
  constexpr uint32_t OOB = 0x80000000u;
  const __amdgpu_buffer_rsrc_t rV = __builtin_amdgcn_make_buffer_rsrc(const_cast<u32x4*>(vals), (short)0,
                                                                    (int)(uint32_t)((size_t)RG * KF * 1024), 0x00020000);
  const __amdgpu_buffer_rsrc_t rMt = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint32_t*>(meta), (short)0,
                                                                     (int)(uint32_t)((size_t)RG * (E == 2 ? KA : KF) * 256), 0x00020000);
  const __amdgpu_buffer_rsrc_t rX = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(Xp), (short)0,
                                                                    (int)(uint32_t)(((size_t)(T - 1) * x_row + cin) * E),
                                                                    0x00020000);
  const int wu = __builtin_amdgcn_readfirstlane(w);
  uint32_t voffV[2], voffX[2], voffM;
  int kchX[2];
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    const int f = 8 * o + w, rg = m0 / 32 + (f >> 1);
    voffV[o] = (rg < RG) ? (uint32_t)((((size_t)rg * KF + (f & 1)) * 64 + l) * 16) : OOB;
    const int c = (o * 8 + w) * 64 + l, row = c >> 3, ch = (c & 7) ^ ((row >> 1) & 7);
    kchX[o] = ch * 16;
    voffX[o] = (n0 + row < T) ? (uint32_t)((size_t)(n0 + row) * x_row * E + ch * 16) : OOB;
  }
  if (E == 2) {
    voffM = (m0 / 32 + w < RG) ? (uint32_t)(((size_t)(m0 / 32 + w) * KA * 64 + l) * 4) : OOB;
  } else {                                                 // two row groups a wave, 512 bytes each
    const int rg = m0 / 32 + 2 * w + h;
    voffM = (w < 4 && rg < RG) ? (uint32_t)((size_t)rg * KF * 256 + ln * 16) : OOB;
  }
  auto issue_one = [&](int stage, int k, int o, auto TAIL) {
    const int ks = k0 + k;
    unsigned char* sb = sp_lds + stage * STAGE;
    constexpr bool TL = decltype(TAIL)::value;
    if (o < 2) {
      uint32_t vo = voffV[o];
      if (TL && 2 * ks + (wu & 1) >= KF) vo = OOB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rV, (dep_lds_t)(sb + (8 * o + wu) * 1024), 16, (int)vo,
                                               (int)((uint32_t)ks * 2048u), 0, 0);
    } else if (o == 2) {
      uint32_t vo = voffM;
      if (E == 2) {
        if (TL && ks >= KA) vo = OOB;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rMt, (dep_lds_t)(sb + MOFF + wu * 256), 4, (int)vo,
                                                 (int)((uint32_t)ks * 256u), 0, 0);
      } else {
        if (TL && 2 * ks + (ln >> 4) >= KF) vo = OOB;      // 16 lanes a fragment
        unsigned char* to = wu < 4 ? sb + MOFF + wu * 1024 : sp_lds + RS * STAGE + (wu - 4) * 1024;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rMt, (dep_lds_t)to, 16, (int)vo, (int)((uint32_t)ks * 512u), 0, 0);
      }
    } else {
      uint32_t vo = voffX[o - 3];
      if (TL && ks * 128 + kchX[o - 3] >= cin * E) vo = OOB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rX, (dep_lds_t)(sb + BOFF + ((o - 3) * 8 + wu) * 1024), 16, (int)vo,
                                               (int)((uint32_t)ks * 128u), 0, 0);
    }
  };

  floatx16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = floatx16{};

  // fragments of half g of a stage, two register sets (the next stage is read
  // while the current one still feeds MFMAs); the position word of a row
  // group is read as the 16-bit half g
  constexpr int SETS = MODE == M_E4M3 ? 1 : 2;             // the conversions leave registers for one: read when all
  static_assert(SETS == 2 || NPRE == NM, "one set is read when its MFMAs are done");    // of a step's MFMAs are done
  u32x4 fa[SETS][FM];
  u32x8 fb[SETS][FN];
  uint32_t fm[SETS][FM];
  u32x8 cb[MODE == M_E4M3 ? 2 : 1];
  int boff[FN][2];
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int row = wn * WN + 32 * j + ln;
    boff[j][0] = sp_swz(row, 4 * g + h);
    boff[j][1] = sp_swz(row, 4 * g + 2 + h);
  }
  auto rd = [&](int stage, auto SET) {
    constexpr int S = decltype(SET)::value;
    const unsigned char* sb = sp_lds + stage * STAGE;
    const u32x4* LA = reinterpret_cast<const u32x4*>(sb);
    const uint16_t* LM = reinterpret_cast<const uint16_t*>(sb + MOFF);
    const uint32_t* LM4 = reinterpret_cast<const uint32_t*>(sb + MOFF);
    const uint16_t* LB = reinterpret_cast<const uint16_t*>(sb + BOFF);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      fa[S][i] = LA[((wm * FM + i) * 2 + g) * 64 + l];
      if (E == 2) fm[S][i] = LM[((wm * FM + i) * 64 + l) * 2 + g];
      else fm[S][i] = LM4[((wm * FM + i) * 2 + g) * 64 + l];
    }
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const u32x4 b0 = *reinterpret_cast<const u32x4*>(&LB[boff[j][0]]);
      const u32x4 b1 = *reinterpret_cast<const u32x4*>(&LB[boff[j][1]]);
      fb[S][j] = cat(b0, b1);
    }
  };
  // MFMA m of a step: block (m % FM, m / FM); the index-set field stays 0
  // since the position word already holds half g in its low bits
  auto mma = [&](auto SET, int m) {
    constexpr int S = SETS == 2 ? decltype(SET)::value : 0;
    const int i = m % FM, j = m / FM;
    if constexpr (MODE == M_E4M3) {
      // one token block's activations are converted for the FM row groups that follow
      __builtin_amdgcn_sched_barrier(0);
      if (i == 0) { cb[0] = half_acts(fb[S][j], 0); cb[1] = half_acts(fb[S][j], 1); }
#pragma unroll
      for (int k = 0; k < 2; ++k)
        acc[i][j] = smfma32<M_BF16>(half_vals(fa[S][i], k), cb[k], acc[i][j], half_idx(fm[S][i], k));
      __builtin_amdgcn_sched_barrier(0);
    } else {
      acc[i][j] = smfma32<MODE>(fa[S][i], fb[S][j], acc[i][j], fm[S][i]);
    }
  };
  // step on stage `stage`, its fragments in set SET: with `load` the tile of K
  // step ks goes to stage `lstage` (its slot was last read before the previous
  // barrier); with `next` the fragments of stage `nstage` are read into the
  // other set after the barrier. WAIT (steady state): before the barrier the
  // wave's loads of the next tile must be done, those of the RS - 3 tiles
  // after it and the PRE loads of this step's tile issued so far may stay in
  // flight (vmcnt counts in issue order).
  constexpr int PRE = [] {                                 // loads issued before the barrier
    int n = 0;
    for (int o = 0; o < NL; ++o) n += (o * LSPAN / NL < NPRE);
    return n;
  }();
  auto step = [&](auto SET, int stage, int lstage, int ks, int nstage, bool load, bool next, auto WAIT, auto TAIL) {
    constexpr int S = decltype(SET)::value;
    auto mfma_loads = [&](int m) {
#pragma unroll
      for (int o = 0; o < NL; ++o)
        if (load && o * LSPAN / NL == m) {
          __builtin_amdgcn_sched_barrier(0);
          issue_one(lstage, ks, o, TAIL);
          __builtin_amdgcn_sched_barrier(0);
        }
      mma(SET, m);
    };
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int m = 0; m < NPRE; ++m) mfma_loads(m);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (decltype(WAIT)::value) sp_wait_vmcnt<(RS - 3) * NL + PRE>();
    else sp_wait_vmcnt<0>();
    __builtin_amdgcn_s_waitcnt(0xC07F);                    // lgkmcnt(0): this stage's reads are done
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    if (next) rd(nstage, std::integral_constant<int, SETS == 2 ? 1 - S : 0>{});
    __builtin_amdgcn_sched_barrier(0);                     // nothing here waits for those reads
#pragma unroll
    for (int m = NPRE; m < NM; ++m) mfma_loads(m);
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr std::integral_constant<int, 0> S0{};
  constexpr std::integral_constant<int, 1> S1{};

  // prologue: tiles 0 .. RS - 2 (a tile past K reads zeros and is never multiplied)
#pragma unroll
  for (int s = 0; s < RS - 1; ++s)
#pragma unroll
    for (int o = 0; o < NL; ++o) issue_one(s, s, o, std::true_type{});
  sp_wait_vmcnt<(RS - 2) * NL>();
  __builtin_amdgcn_s_barrier();
  rd(0, S0);
  int kt = 0;
  // RS steady-state steps (RS is even: step kt uses set kt % 2); they load K
  // steps up to kt + 2 RS - 2 < NK - 1, never the last one
  for (; kt + 2 * RS - 1 < NK; kt += RS) {
#pragma unroll
    for (int s = 0; s < RS; s += 2) {
      step(S0, s, (s + RS - 1) % RS, kt + s + RS - 1, s + 1, true, true, std::true_type{}, std::false_type{});
      step(S1, s + 1, s, kt + s + RS, (s + 2) % RS, true, true, std::true_type{}, std::false_type{});
    }
  }
  for (; kt < NK; kt += 2) {                               // the last steps, all loads retired at each barrier
    step(S0, kt % RS, (kt + RS - 1) % RS, kt + RS - 1, (kt + 1) % RS, kt + RS - 1 < NK, kt + 1 < NK,
         std::false_type{}, std::true_type{});
    if (kt + 1 < NK)
      step(S1, (kt + 1) % RS, kt % RS, kt + RS, (kt + 2) % RS, kt + RS < NK, kt + 2 < NK, std::false_type{},
           std::true_type{});
  }
  sp_wait_vmcnt<0>();                                      // the zero tiles of a short K
  __syncthreads();                                         // every wave is done with the ring

  if constexpr (Epi::kRows == 8) {
    // group 1's sums, group 0's on top, to LDS by token: quarter rows c of token t at c ^ (t % 16), conflict-free by
    // token and by row
    floatx4* sums = reinterpret_cast<floatx4*>(sp_lds);
    const auto place = [](int token, int c) { return token * (SP_BM / 4) + (c ^ (token & 15)); };
    const int c8 = t & 31, o = m0 + 8 * c8, first = t >> 5;    // this thread's rows and tokens first + 16 n
    constexpr int NP = SP_BN / 16, HALF = NP / 2;
    const bool mine = o < cout;
    typename Epi::Fixed fx;
    typename Epi::Loaded ex[NP];
    if (mine) fx = epi.fixed(o);
#pragma unroll
    for (int n = 0; n < HALF; ++n)
      if (mine && n0 + first + 16 * n < T) ex[n] = epi.load(n0 + first + 16 * n, o);
    auto each = [&](auto F) {
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            floatx4& at = sums[place(wn * WN + 32 * j + ln, wm * 32 + 8 * i + 4 * h + q)];
            const floatx4 a = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
            if constexpr (decltype(F)::value) at = a;
            else at = at + a;
          }
    };
    if (g == 1) each(std::true_type{});
    __syncthreads();
    if (g == 0) each(std::false_type{});
    __syncthreads();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (half == 0) {
#pragma unroll
        for (int n = HALF; n < NP; ++n)
          if (mine && n0 + first + 16 * n < T) ex[n] = epi.load(n0 + first + 16 * n, o);
      }
#pragma unroll
      for (int n = half * HALF; n < (half + 1) * HALF; ++n) {
        const int token = first + 16 * n;
        const floatx4 a = sums[place(token, 2 * c8)], b = sums[place(token, 2 * c8 + 1)];
        if (mine && n0 + token < T) epi.store(n0 + token, o, a, b, fx, ex[n]);
      }
    }
    return;
  } else {
  // exchange: group g hands its blocks of column 1 - g to the other group and
  // adds the other group's blocks of column g to its own (x + y = y + x, so
  // both halves get the same sum as any fixed order)
  floatx4* xl = reinterpret_cast<floatx4*>(sp_lds);
  auto put = [&](auto J) {
    constexpr int j = decltype(J)::value;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        xl[(((g * 4 + v) * FM + i) * 4 + q) * 64 + l] =
            floatx4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
  };
  auto take_store = [&](auto J) {
    constexpr int j = decltype(J)::value;
    const int tk = n0 + wn * WN + 32 * j + ln;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      floatx16 a = acc[i][j];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const floatx4 x = xl[((((1 - g) * 4 + v) * FM + i) * 4 + q) * 64 + l];
        a[4 * q] += x[0];
        a[4 * q + 1] += x[1];
        a[4 * q + 2] += x[2];
        a[4 * q + 3] += x[3];
      }
      // lane (h, ln): token tk, rows m0 + wm*128 + 32i + 16h + r (r < 16)
      const int o = m0 + wm * WM + 32 * i + 16 * h;
      if (o >= cout || tk >= T) continue;
      epi.store(tk, o, a);
    }
  };
  if (g == 0) put(S1);
  else put(S0);
  __syncthreads();
  if (g == 0) take_store(S0);
  else take_store(S1);
  }
}

}  // namespace lcp
