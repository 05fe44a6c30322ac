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
//
// Both are bound by memory where they are large and by launch latency where they are small:
// one pass, 16-byte accesses, and no shared memory or second launch.
#include <cuda_bf16.h>

#include <type_traits>

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
__device__ __forceinline__ float2 turn(float a, float b, float2 r) { return make_float2(a * r.x - b * r.y, a * r.y + b * r.x); }

__device__ __forceinline__ float load_f32(const float* p) { return *p; }
__device__ __forceinline__ float load_f32(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_f32(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_f32(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// 16 bytes as floats
template <class T>
struct Chunk;
template <>
struct Chunk<float> {
  static constexpr int n = 4;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x), f[1] = __uint_as_float(u.y), f[2] = __uint_as_float(u.z), f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
template <>
struct Chunk<__nv_bfloat16> {
  static constexpr int n = 8;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
};

struct RopeArgs {
  const void* x;
  void* out;
  const long long* positions;
  long long n;
  int heads, dim, rot_offset;
  long long x_token, x_head, out_token, out_head;  // strides in elements
};

// Wide accesses.  A thread keeps one place of the head -- a chunk of an interleaved part, the
// two chunks of a half layout that hold the same pairs' ends, or a passed-through chunk -- and
// walks kHeads heads of its token.  Threads: x the place, y the head, z the token; a block
// covers tokens z, heads y + blockDim.y i.  Its tokens' angles are computed once for all of
// them, while the loads are in flight, and shared.
// 4096 tokens, 67 MB read and written: 64 heads x 64 interleaved in views of wider rows, and
// 32 heads x 128 of which 64 rotate in the half layout; a plain copy of the latter takes
// 14.5 us.  16.4 and 14.4 us; in 32 bits 25.0 and 23.5 us (134 MB; the copy 24.7).  (With every thread
// computing its own angles the second took 3.3 us more, the first as long.)
template <class T, int kHeads, bool kHalf>
__global__ void __launch_bounds__(256) rope_wide_kernel(RopeArgs a, const __grid_constant__ dsa_rope_plan plan, int places,
                                                        int turned) {
  extern __shared__ float2 s_angle[];  // [blockDim.z][rot_dim / 2]
  constexpr int V = Chunk<T>::n;
  const int u = blockIdx.z * blockDim.x + threadIdx.x, half = plan.rot_dim / 2;
  const long long token0 = (long long)blockIdx.x * blockDim.z, token = token0 + threadIdx.z;
  const bool there = token < a.n && u < places;
  const int head0 = blockIdx.y * blockDim.y * kHeads + threadIdx.y;
  const bool pass = u >= turned;
  int e0 = pass ? V * (u - turned) : a.rot_offset + V * u;  // first element of the chunk
  if (pass && e0 >= a.rot_offset) e0 += plan.rot_dim;
  const int e1 = half;                                       // ... and how far behind it the second one is
  const T* x = static_cast<const T*>(a.x) + token * a.x_token + e0;
  T* out = static_cast<T*>(a.out) + token * a.out_token + e0;
  uint4 v0[kHeads], v1[kHalf ? kHeads : 1];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = head0 + i * (int)blockDim.y;
    if (there && h < a.heads) {
      v0[i] = *reinterpret_cast<const uint4*>(x + h * a.x_head);
      if constexpr (kHalf) {
        if (!pass) v1[i] = *reinterpret_cast<const uint4*>(x + h * a.x_head + e1);
      }
    }
  }
  const int threads = blockDim.x * blockDim.y * blockDim.z;
  for (int i = (threadIdx.z * blockDim.y + threadIdx.y) * blockDim.x + threadIdx.x; i < half * (int)blockDim.z; i += threads) {
    const int z = i / half;
    if (token0 + z < a.n) s_angle[i] = rope_angle(a.positions[token0 + z], plan.turns[i - z * half], plan.mscale);
  }
  __syncthreads();
  if (!there) return;
  constexpr int A = kHalf ? V : V / 2;  // angles of a chunk
  float2 r[A];
  if (!pass) {
#pragma unroll
    for (int j = 0; j < A; ++j) r[j] = s_angle[threadIdx.z * half + A * u + j];
  }
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = head0 + i * (int)blockDim.y;
    if (h >= a.heads) break;
    if (!pass) {
      float f0[V];
      Chunk<T>::unpack(v0[i], f0);
      if constexpr (kHalf) {
        float f1[V];
        Chunk<T>::unpack(v1[i], f1);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float2 y = turn(f0[j], f1[j], r[j]);
          f0[j] = y.x;
          f1[j] = y.y;
        }
        *reinterpret_cast<uint4*>(out + h * a.out_head + e1) = Chunk<T>::pack(f1);
      } else {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
          const float2 y = turn(f0[2 * j], f0[2 * j + 1], r[j]);
          f0[2 * j] = y.x;
          f0[2 * j + 1] = y.y;
        }
      }
      v0[i] = Chunk<T>::pack(f0);
    }
    *reinterpret_cast<uint4*>(out + h * a.out_head) = v0[i];
  }
}

// Any alignment and any even rot_dim: one thread per rotary pair or passed-through element.
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
  const int i1 = plan.layout == DSA_ROPE_HALF ? i0 + half : i0 + 1;
  const float2 y = turn(load_f32(x + i0), load_f32(x + i1), r);
  store_f32(out + i0, y.x);
  store_f32(out + i1, y.y);
}

// The scale that sums of squares outside [2^-100, 2^120] are taken again under, so that rows
// of any bf16 magnitude keep their norm (1 otherwise): entries up to 2^-50 times 2^90 have squares
// between 2^-86 and 2^80.  Small sums matter only beside a smaller eps.
__device__ __forceinline__ float norm_rescale(float sum, float eps) {
  if (sum > 0x1p120f) return 0x1p-70f;
  return sum < 0x1p-100f && eps < 0x1p-90f ? 0x1p90f : 1.f;
}

// The sequence b with cu_q[b] <= token < cu_q[b + 1], for the lanes of a warp alike; -1 if
// there is none.  32 entries are read at a time.
__device__ __forceinline__ int find_sequence(const PagedBatch& p, int token, int lane) {
  int lo = 0, size = p.B + 1;  // the last entry <= token is one of [lo, lo + size)
  while (true) {
    const int step = (size + 31) / 32, i = lo + lane * step;
    const bool below = lane * step < size && p.cu_q[i] <= token;
    const int count = __popc(__ballot_sync(0xFFFFFFFFu, below));
    if (count == 0) return -1;
    lo += (count - 1) * step;
    size = min(step, size - (count - 1) * step);
    if (step == 1) return lo < p.B ? lo : -1;
  }
}

// One warp per token: lane l holds latent entries 8 l .. 8 l + 7 and 256 + 8 l .. 256 + 8 l + 7
// and the angle of rotary pair l; lanes 0 .. 7 hold the rotary part's eight chunks and take the
// angles (in the half layout also the other ends) from the lanes that have them.  The row is
// loaded before its place is looked up.  16 chunks of up to 8 tokens take 2.6 us, 10.9K tokens 7.9 us
// (3.2 TB/s): the chain of loads from the lengths over the table to the row's place.
constexpr int kAppendWarps = 4;
__global__ void __launch_bounds__(32 * kAppendWarps) append_kernel(const uint16_t* __restrict__ x, long long x_stride,
                                                                   const uint16_t* __restrict__ gamma, float eps,
                                                                   const __grid_constant__ dsa_rope_plan plan,
                                                                   PagedBatch pb, uint16_t* __restrict__ cache) {
  using B16 = Chunk<__nv_bfloat16>;
  const long long at = (long long)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  if (at >= pb.n) return;
  const int token = (int)at, lane = threadIdx.x & 31;
  const uint4* src = reinterpret_cast<const uint4*>(x + token * x_stride);
  const uint4* gm = reinterpret_cast<const uint4*>(gamma);
  const uint4 c0 = src[lane], c1 = src[32 + lane], g0 = gm[lane], g1 = gm[32 + lane];
  const uint4 cr = lane < 8 ? src[64 + lane] : make_uint4(0, 0, 0, 0);
  const int b = find_sequence(pb, token, lane);
  if (b < 0) return;
  const long long position = (long long)pb.ctx_len[b] - pb.cu_q[b + 1] + token;
  const long long row = paged_row(pb, b, position);
  if (row < 0) return;
  float v0[8], v1[8], w[8];
  B16::unpack(c0, v0);
  B16::unpack(c1, v1);
  auto squares = [&](float s) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += (v0[i] * s) * (v0[i] * s) + (v1[i] * s) * (v1[i] * s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    return sum;
  };
  float sum = squares(1.f);
  const float s = norm_rescale(sum, eps);
  if (s != 1.f) sum = squares(s);
  // y = x s rsqrt(mean (x s)^2 + eps s^2).  A large s stays with x: times the root, some 2^133 for
  // entries of 2^-133, it would pass 32 bits.  A small one stays with the root: x s would lose bits.
  const float up = fmaxf(s, 1.f), inv = rsqrtf(sum / kDv + eps * s * s) * fminf(s, 1.f);
  uint4* dst = reinterpret_cast<uint4*>(cache + row * kDqk);
  B16::unpack(g0, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) v0[i] = v0[i] * up * inv * w[i];
  dst[lane] = B16::pack(v0);
  B16::unpack(g1, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) v1[i] = v1[i] * up * inv * w[i];
  dst[32 + lane] = B16::pack(v1);
  const float2 r = rope_angle(position, plan.turns[lane], plan.mscale);
  B16::unpack(cr, v0);
  if (plan.layout == DSA_ROPE_HALF) {
    // chunk c < 4 holds the first ends of pairs 8 c .. 8 c + 7, chunk c + 4 the second
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = __shfl_sync(0xFFFFFFFFu, r.x, 8 * (lane & 3) + i), si = __shfl_sync(0xFFFFFFFFu, r.y, 8 * (lane & 3) + i);
      const float other = __shfl_xor_sync(0xFFFFFFFFu, v0[i], 4);
      v1[i] = lane & 4 ? other * si + v0[i] * c : v0[i] * c - other * si;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int pair = 4 * (lane & 7) + i;
      const float2 y = turn(v0[2 * i], v0[2 * i + 1],
                            make_float2(__shfl_sync(0xFFFFFFFFu, r.x, pair), __shfl_sync(0xFFFFFFFFu, r.y, pair)));
      v1[2 * i] = y.x;
      v1[2 * i + 1] = y.y;
    }
  }
  if (lane < 8) dst[64 + lane] = B16::pack(v1);
}

constexpr int kManyHeads = 4;

template <class T>
cudaError_t rope_launch(const RopeArgs& a, const dsa_rope_plan& plan, bool in_place, cudaStream_t stream) {
  constexpr int V = Chunk<T>::n;
  const int rest = in_place ? 0 : a.dim - plan.rot_dim;
  auto even = [](long long v) { return v % V == 0; };
  auto base = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  // wide: every chunk of 16 bytes lies within the rotated part (of the half layout: within one
  // half of it) or outside, and is aligned
  const bool wide = base(a.x) && base(a.out) && even(a.x_token) && even(a.x_head) && even(a.out_token) && even(a.out_head) &&
                    even(a.rot_offset) && even(a.dim) && even(plan.layout == DSA_ROPE_HALF ? plan.rot_dim / 2 : plan.rot_dim);
  if (!wide) {
    const int per_head = plan.rot_dim / 2 + rest;
    const long long blocks = (a.n * a.heads * per_head + 255) / 256;
    if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
    rope_kernel<T><<<(unsigned)blocks, 256, 0, stream>>>(a, plan, per_head);
    return cudaGetLastError();
  }
  const int turned = (plan.layout == DSA_ROPE_HALF ? plan.rot_dim / 2 : plan.rot_dim) / V, places = turned + rest / V;
  auto launch = [&](auto heads, auto half) {
    constexpr int kHeads = decltype(heads)::value;
    const int group = (a.heads + kHeads - 1) / kHeads;
    dim3 block(places < 256 ? places : 256);
    block.y = group < 256 / (int)block.x ? group : 256 / block.x;
    block.z = 256 / (block.x * block.y) < 64 ? 256 / (block.x * block.y) : 64;
    const long long tokens = (a.n + block.z - 1) / block.z;
    const dim3 grid((unsigned)tokens, (group + block.y - 1) / block.y, (places + block.x - 1) / block.x);
    if (tokens > 0x7FFFFFFFLL || grid.y > 65535 || grid.z > 65535) return cudaErrorInvalidConfiguration;
    rope_wide_kernel<T, kHeads, decltype(half)::value>
        <<<grid, block, (size_t)block.z * (plan.rot_dim / 2) * sizeof(float2), stream>>>(a, plan, places, turned);
    return cudaGetLastError();
  };
  // few tokens: a thread a chunk, so that the call is one wave of short threads
  const bool few = a.n * a.heads * places < 4LL * 2048 * device_sm_count();
  const std::integral_constant<int, 1> one;
  const std::integral_constant<int, kManyHeads> many;
  if (plan.layout == DSA_ROPE_HALF) return few ? launch(one, std::true_type()) : launch(many, std::true_type());
  return few ? launch(one, std::false_type()) : launch(many, std::false_type());
}

}  // namespace

cudaError_t launch_rope(const void* x, const long long* positions, long long n, int heads, int dim, int rot_offset,
                        const dsa_rope_plan& plan, int dtype, long long x_token, long long x_head, void* out,
                        long long out_token, long long out_head, cudaStream_t stream) {
  const RopeArgs a{x, out, positions, n, heads, dim, rot_offset, x_token, x_head, out_token, out_head};
  return dtype == DSA_F32 ? rope_launch<float>(a, plan, out == x, stream)
                          : rope_launch<__nv_bfloat16>(a, plan, out == x, stream);
}

cudaError_t launch_cache_append(const uint16_t* x, long long x_stride, const uint16_t* gamma, float eps,
                                const dsa_rope_plan& plan, const PagedBatch& pb, uint16_t* cache, cudaStream_t stream) {
  append_kernel<<<(unsigned)((pb.n + kAppendWarps - 1LL) / kAppendWarps), 32 * kAppendWarps, 0, stream>>>(x, x_stride, gamma,
                                                                                                       eps, plan, pb, cache);
  return cudaGetLastError();
}

}  // namespace dsa
