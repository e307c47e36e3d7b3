// Attention of one new token of each sequence over the paged cache.
#include "serve.h"

namespace lcp {
namespace {

__device__ __forceinline__ float kv_value(const KvCache& c, const void* p, const float* scale, int64_t row, int d) {
  if (c.format == KV_BF16) return bf2f(((const uint16_t*)p)[row * c.D + d]);
  const uint8_t code = ((const uint8_t*)p)[row * c.D + d];
  const float x = c.format == KV_E4M3 ? __builtin_amdgcn_cvt_f32_fp8((int)code, 0) : (float)(int8_t)code;
  return x * scale[row];
}

// One workgroup per (sequence, query head); wave w takes every fourth token,
// lane l holds channels l, l + 64, ..; one pass with the running maximum and sum
// of the softmax, the four waves joined through LDS.
__global__ __launch_bounds__(256) void attn_rows_kernel(AttnArgs a) {
  __shared__ float sm[4], sl[4], so[4][256];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int b = blockIdx.x / a.hq, h = blockIdx.x % a.hq, hk = h / (a.hq / a.c.heads);
  const int n = a.c.D / 64;
  const int len = min(max(a.lens[b], 0), a.max_len);
  const int lo = a.window && len > a.window ? len - a.window : 0;
  float q[4] = {0.f, 0.f, 0.f, 0.f}, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < 4; ++i)
    if (i < n) q[i] = bf2f(a.q[b * a.qrow + (int64_t)h * a.c.D + lane + 64 * i]);
  float m = -__builtin_inff(), l = 0.f;
  for (int t = lo + wave; t < len; t += 4) {
    const int page = a.pages[(int64_t)b * a.max_pages + t / a.c.ps];
    if (page < 0 || page >= a.c.pages) continue;
    const int64_t row = ((int64_t)page * a.c.heads + hk) * a.c.ps + t % a.c.ps;
    float z = 0.f;
    for (int i = 0; i < 4; ++i)
      if (i < n) z += q[i] * kv_value(a.c, a.c.k, a.c.ks, row, lane + 64 * i);
    for (int k = 1; k < 64; k <<= 1) z += shfl_xor(z, k);
    z *= a.scale2;
    const float mn = fmaxf(m, z), base = mn == -__builtin_inff() ? 0.f : mn;
    const float r = exp2_(m - base), p = exp2_(z - base);
    l = l * r + p;
    for (int i = 0; i < 4; ++i)
      if (i < n) o[i] = o[i] * r + p * kv_value(a.c, a.c.v, a.c.vs, row, lane + 64 * i);
    m = mn;
  }
  if (lane == 0) { sm[wave] = m; sl[wave] = l; }
  for (int i = 0; i < 4; ++i) so[wave][lane + 64 * i] = o[i];
  __syncthreads();
  float M = sm[0];
  for (int w = 1; w < 4; ++w) M = fmaxf(M, sm[w]);
  const float base = M == -__builtin_inff() ? 0.f : M;
  float L = 0.f, y = 0.f;
  for (int w = 0; w < 4; ++w) {
    const float r = exp2_(sm[w] - base);
    L += sl[w] * r;
    y += so[w][threadIdx.x] * r;
  }
  if ((int)threadIdx.x < a.c.D) {
    y = L == 0.f ? 0.f : y / L;
    const int64_t i = ((int64_t)b * a.hq + h) * a.c.D + threadIdx.x;
    if (a.out_bf16) ((uint16_t*)a.out)[i] = (uint16_t)f2bf(y);
    else ((float*)a.out)[i] = y;
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[(int64_t)b * a.hq + h] = L == 0.f ? -__builtin_inff() : (M + log2_(L)) * 0.6931471805599453f;
}

}  // namespace

size_t attn_workspace_bytes(const KvCache&, int, int, int, int) { return 256; }

hipError_t launch_attn_decode(const AttnArgs& a, hipStream_t s) {
  attn_rows_kernel<<<(unsigned)(a.B * a.hq), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace lcp
