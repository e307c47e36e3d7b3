// Operators of a decoder block around its deployed products (root-mean-square
// norm, its gradient, the 2:4 product with an epilogue): arguments of their
// launchers. Validation is done by block.hip before any launcher runs; every
// launcher enqueues on `s` and returns hipGetLastError().
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.h"

namespace lcp {

// A matrix's rows: pointer and stride in elements.
struct Mat {
  const void* p;
  int64_t row;
};
struct MatOut {
  void* p;
  int64_t row;
};

enum ElemType { T_F32 = 0, T_BF16 = 1, T_E4M3 = 2 };

struct NormArgs {
  Mat x, res;            // res.p nullable
  MatOut sum, y;         // sum.p nullable
  const void* w;
  float* scale;
  const int* perm;       // nullable
  int wt, yt;            // ElemType
  int T, C, B;
  float eps;
};
hipError_t launch_rms_norm(const NormArgs& a, int xt, hipStream_t s);

struct NormGradArgs {
  Mat h, dy, dsum;       // dsum.p nullable
  MatOut dx;
  const void* w;
  void* dw;
  float* ws;
  int wt;
  int T, C;
  float eps;
};
size_t norm_grad_workspace_bytes(int T, int C);
hipError_t launch_rms_norm_bwd(const NormGradArgs& a, int xt, hipStream_t s);

struct PackedArgs {
  const u32x4* vals;
  const uint32_t* meta;
  const float* wscale;
  int fp8, cout, cin, fast;
};
size_t sparse_vals_bytes_e4m3(int cout, int cin);
size_t sparse_meta_bytes_e4m3(int cout, int cin);
hipError_t launch_sparse_pack_e4m3(const uint16_t* W, int cout, int cin, int B, const int* perm, const uint32_t* bits,
                                   u32x4* vals, uint32_t* meta, float* wscale, hipStream_t s);

struct Epilogue {
  const uint16_t *bias, *gate;
  const void* res;
  const float *xscale, *wscale;      // E4M3
  void* y;
  int64_t gate_row, res_row, y_row;
  int res_f32, y_f32, act;
};

struct LinearArgs {
  PackedArgs w;
  Mat x;
  int T;
  Epilogue e;
  float* ws;
};
size_t sparse_linear_workspace_bytes(const PackedArgs& w, int T);
// SparseMode, row tiles, token tiles, waves, parts (as lcp_sparse_linear_cut)
void sparse_linear_cut(const PackedArgs& w, int T, int y_f32, int* out);
hipError_t launch_sparse_linear(const LinearArgs& a, hipStream_t s);

}  // namespace lcp
