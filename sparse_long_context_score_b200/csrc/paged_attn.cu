// paged_attn.cu -- MLA attention of a chunk of new tokens over a paged compressed cache.
//
//   out[t, h] = sum_s softmax_s(scale q[t, h] . c[s]) c[s][0:512],  s <= position of t,
// c[s] the 576-wide row of position s, in page table[b][s / page_size] at s % page_size.
// lse[t, h] = ln sum_s exp(scale q[t, h] . c[s]).
#include <cuda_bf16.h>

#include "dsa_common.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int kWarps = 8;

// One block per (token, head); a warp takes every eighth visible row with an online
// softmax of its own, and the eight are merged in shared memory.
__global__ void __launch_bounds__(32 * kWarps) paged_attn_kernel(const uint16_t* __restrict__ q,
                                                                 const uint16_t* __restrict__ cache, PagedBatch pb, int H,
                                                                 float scale, uint16_t* __restrict__ out,
                                                                 float* __restrict__ lse) {
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][kDv];
  const int token = blockIdx.x, head = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int b = -1;
  for (int i = 0; i < pb.B; ++i)
    if (pb.cu_q[i] <= token && token < pb.cu_q[i + 1]) b = i;
  if (b < 0) return;
  const size_t unit = (size_t)token * H + head;
  const __nv_bfloat162* qr = reinterpret_cast<const __nv_bfloat162*>(q) + unit * (kDqk / 2);
  float2 qv[9], acc[8];
  for (int i = 0; i < 9; ++i) qv[i] = __bfloat1622float2(qr[32 * i + lane]);
  for (int i = 0; i < 8; ++i) acc[i] = make_float2(0.f, 0.f);
  float m = -INFINITY, l = 0.f;
  const long long last = (long long)pb.ctx_len[b] - pb.cu_q[b + 1] + token;
  for (long long s = warp; s <= last; s += kWarps) {
    const long long row = paged_row(pb, b, s);
    if (row < 0) continue;
    const __nv_bfloat162* c = reinterpret_cast<const __nv_bfloat162*>(cache) + row * (kDqk / 2);
    float2 cv[9];
    float z = 0.f;
    for (int i = 0; i < 9; ++i) {
      cv[i] = __bfloat1622float2(c[32 * i + lane]);
      z += qv[i].x * cv[i].x + qv[i].y * cv[i].y;
    }
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
    z *= scale;
    const float mn = fmaxf(m, z), a = expf(m - mn), p = expf(z - mn);
    for (int i = 0; i < 8; ++i) {
      acc[i].x = acc[i].x * a + p * cv[i].x;
      acc[i].y = acc[i].y * a + p * cv[i].y;
    }
    l = l * a + p;
    m = mn;
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  for (int i = 0; i < 8; ++i) {
    s_o[warp][64 * i + 2 * lane] = acc[i].x;
    s_o[warp][64 * i + 2 * lane + 1] = acc[i].y;
  }
  __syncthreads();
  float M = -INFINITY, L = 0.f, coef[kWarps];
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w]);
  for (int w = 0; w < kWarps; ++w) {
    coef[w] = s_l[w] > 0.f ? expf(s_m[w] - M) : 0.f;
    L += coef[w] * s_l[w];
  }
  for (int d = threadIdx.x; d < kDv; d += 32 * kWarps) {
    float o = 0.f;
    for (int w = 0; w < kWarps; ++w) o += coef[w] * s_o[w][d];
    reinterpret_cast<__nv_bfloat16*>(out)[unit * kDv + d] = __float2bfloat16_rn(L > 0.f ? o / L : 0.f);
  }
  if (threadIdx.x == 0 && lse) lse[unit] = L > 0.f ? M + logf(L) : -INFINITY;
}

}  // namespace

size_t paged_attn_workspace_bytes(long long, int, int) { return 256; }

cudaError_t launch_paged_attn(const uint16_t* q, const uint16_t* cache, const PagedBatch& pb, int H, float scale,
                              uint16_t* out, float* lse, void*, cudaStream_t stream) {
  paged_attn_kernel<<<dim3((unsigned)pb.n, (unsigned)H), 32 * kWarps, 0, stream>>>(q, cache, pb, H, scale, out, lse);
  return cudaGetLastError();
}

}  // namespace dsa
