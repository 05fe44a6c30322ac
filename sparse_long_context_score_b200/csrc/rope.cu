// rope.cu -- rotary positions, and the rows of a paged compressed cache.
//
// A rotary pair (a, b) of a token at position p turns by the angle p f_i:
//   (a cos - b sin, a sin + b cos),  i the pair's index, f_i radians per position.
// The plan holds f_i in revolutions per position (f_i / 2 pi, 64 bits).  p times that is
// taken in 64 bits and reduced to a fraction of a revolution in [-1/2, 1/2] before it is
// rounded to 32 bits, so the angle is good to 2^-24 of half a revolution at any position up
// to 2^31 (32-bit products would be off by whole degrees at a million tokens).
//
// The row appended for a token is [x[0:512] rsqrt(mean x[0:512]^2 + eps) gamma, rope(x[512:576])],
// sums and products in 32 bits, rounded once to bf16 as the cache holds it.
#include <cuda_bf16.h>

#include "dsa_common.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

// cosine and sine of position * turns revolutions, times mscale
__device__ __forceinline__ float2 rope_angle(long long position, double turns, float mscale) {
  const double t = (double)position * turns;
  float s, c;
  sincospif(2.f * (float)(t - rint(t)), &s, &c);
  return make_float2(c * mscale, s * mscale);
}

__device__ __forceinline__ float load_f32(const float* p) { return *p; }
__device__ __forceinline__ float load_f32(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_f32(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_f32(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

struct RopeArgs {
  const void* x;
  void* out;
  const long long* positions;
  long long n;
  int heads, dim, rot_offset;
  long long x_token, x_head, out_token, out_head;  // strides in elements
};

// One thread per rotary pair or passed-through element.
template <class T>
__global__ void __launch_bounds__(256) rope_kernel(RopeArgs a, const __grid_constant__ dsa_rope_plan plan, int per_head) {
  const long long g = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long cell = g / per_head;
  const int u = (int)(g - cell * per_head);
  const long long token = cell / a.heads;
  if (token >= a.n) return;
  const int head = (int)(cell - token * a.heads), half = plan.rot_dim / 2;
  const T* x = static_cast<const T*>(a.x) + token * a.x_token + head * a.x_head;
  T* out = static_cast<T*>(a.out) + token * a.out_token + head * a.out_head;
  if (u >= half) {  // an element outside the rotated part
    int e = u - half;
    if (e >= a.rot_offset) e += plan.rot_dim;
    out[e] = x[e];
    return;
  }
  const float2 r = rope_angle(a.positions[token], plan.turns[u], plan.mscale);
  const int i0 = a.rot_offset + (plan.layout == DSA_ROPE_HALF ? u : 2 * u);
  const int i1 = a.rot_offset + (plan.layout == DSA_ROPE_HALF ? u + half : 2 * u + 1);
  const float x0 = load_f32(x + i0), x1 = load_f32(x + i1);
  store_f32(out + i0, x0 * r.x - x1 * r.y);
  store_f32(out + i1, x0 * r.y + x1 * r.x);
}

// The scale that sums of squares outside [2^-100, 2^120] are taken again under, so that rows
// of any bf16 magnitude keep their norm (1 otherwise).  Small sums matter only beside a
// smaller eps.
__device__ __forceinline__ float norm_rescale(float sum, float eps) {
  if (sum > 0x1p120f) return 0x1p-70f;
  return sum < 0x1p-100f && eps < 0x1p-90f ? 0x1p70f : 1.f;
}

// One block of 64 threads per token: thread c holds the eight latent entries 8c .. 8c + 7;
// the first 32 threads then rotate one pair each.
__global__ void __launch_bounds__(64) append_kernel(const uint16_t* __restrict__ x, long long x_stride,
                                                    const uint16_t* __restrict__ gamma, float eps,
                                                    const __grid_constant__ dsa_rope_plan plan, PagedBatch pb,
                                                    uint16_t* __restrict__ cache) {
  const int token = blockIdx.x;
  int b = -1;
  for (int i = 0; i < pb.B; ++i)
    if (pb.cu_q[i] <= token && token < pb.cu_q[i + 1]) b = i;
  if (b < 0) return;
  const long long position = (long long)pb.ctx_len[b] - pb.cu_q[b + 1] + token;
  const long long row = paged_row(pb, b, position);
  if (row < 0) return;
  const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(x) + token * x_stride;
  const __nv_bfloat16* gm = reinterpret_cast<const __nv_bfloat16*>(gamma);
  __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(cache) + row * kDqk;
  __shared__ float part[2];
  float v[8];
  for (int i = 0; i < 8; ++i) v[i] = __bfloat162float(src[threadIdx.x * 8 + i]);
  auto squares = [&](float s) {
    float sum = 0.f;
    for (int i = 0; i < 8; ++i) sum += (v[i] * s) * (v[i] * s);
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    __syncthreads();
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = sum;
    __syncthreads();
    return part[0] + part[1];
  };
  float sum = squares(1.f);
  const float s = norm_rescale(sum, eps);
  if (s != 1.f) sum = squares(s);
  const float inv = rsqrtf(sum / kDv + eps * s * s) * s;
  for (int i = 0; i < 8; ++i) {
    const int e = threadIdx.x * 8 + i;
    dst[e] = __float2bfloat16_rn(v[i] * inv * __bfloat162float(gm[e]));
  }
  if (threadIdx.x < 32) {
    const float2 r = rope_angle(position, plan.turns[threadIdx.x], plan.mscale);
    const int i0 = kDv + (plan.layout == DSA_ROPE_HALF ? (int)threadIdx.x : 2 * (int)threadIdx.x);
    const int i1 = plan.layout == DSA_ROPE_HALF ? i0 + 32 : i0 + 1;
    const float x0 = __bfloat162float(src[i0]), x1 = __bfloat162float(src[i1]);
    dst[i0] = __float2bfloat16_rn(x0 * r.x - x1 * r.y);
    dst[i1] = __float2bfloat16_rn(x0 * r.y + x1 * r.x);
  }
}

}  // namespace

cudaError_t launch_rope(const void* x, const long long* positions, long long n, int heads, int dim, int rot_offset,
                        const dsa_rope_plan& plan, int dtype, long long x_token, long long x_head, void* out,
                        long long out_token, long long out_head, cudaStream_t stream) {
  const RopeArgs a{x, out, positions, n, heads, dim, rot_offset, x_token, x_head, out_token, out_head};
  const int per_head = plan.rot_dim / 2 + (out == x ? 0 : dim - plan.rot_dim);
  const long long blocks = (n * heads * per_head + 255) / 256;
  if (dtype == DSA_F32)
    rope_kernel<float><<<(unsigned)blocks, 256, 0, stream>>>(a, plan, per_head);
  else
    rope_kernel<__nv_bfloat16><<<(unsigned)blocks, 256, 0, stream>>>(a, plan, per_head);
  return cudaGetLastError();
}

cudaError_t launch_cache_append(const uint16_t* x, long long x_stride, const uint16_t* gamma, float eps,
                                const dsa_rope_plan& plan, const PagedBatch& pb, uint16_t* cache, cudaStream_t stream) {
  append_kernel<<<(unsigned)pb.n, 64, 0, stream>>>(x, x_stride, gamma, eps, plan, pb, cache);
  return cudaGetLastError();
}

}  // namespace dsa
