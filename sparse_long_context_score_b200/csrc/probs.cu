// probs.cu -- logits of draft positions to the probabilities that dsa_verify takes.
//
// Per row (sequence b, position j), for every entry v of the vocabulary, in this order:
//   z = logit
//   z = z > 0 ? z / rep : z * rep       v among the history or the drafts before j
//   z = z - freq count - pres [count > 0]   count: how often v was generated
//   z = z + sum of v's biases
//   z = -inf                              v's mask bit is 0, or z is NaN
//   p = exp((z - max z) / T) / sum        T > 0; else 1 at the lowest index of the maximum
// A row that its mask leaves empty gets zeros.
#include <cuda_bf16.h>

#include "dsa_common.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

// What is known of an entry before its logit is read, one word an entry: how often it was
// generated, whether it was seen at all, and whether a bias names it.
constexpr uint32_t kSeen = 0x80000000u, kBiased = 0x40000000u, kCount = 0x3FFFFFFFu;

__device__ __forceinline__ float adjust(float z, uint32_t word, const ProbsArgs& a, int b, int v, float rep, float freq,
                                        float pres) {
  if (word & kSeen) z = z > 0.f ? z / rep : z * rep;
  const uint32_t count = word & kCount;
  if (count) z = z - freq * (float)count - pres;
  if (word & kBiased) {
    float s = 0.f;
    for (int i = 0; i < a.nbias; ++i)
      if (a.bias_ids[(size_t)b * a.nbias + i] == v) s += a.bias_values[(size_t)b * a.nbias + i];
    z += s;
  }
  return z != z ? -INFINITY : z;
}

__device__ __forceinline__ float load_logit(const void* p, size_t i, int dtype) {
  return dtype == DSA_F32 ? static_cast<const float*>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

constexpr int kThreads = 1024;

template <class F>
__device__ __forceinline__ float block_reduce(float v, float* s, F f) {
  for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  __syncthreads();
  if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = v;
  __syncthreads();
  v = s[threadIdx.x % 32];
  for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// One block per row.  The row of p holds, in turn, the words of the entries, their
// adjusted logits and their probabilities.
__global__ void __launch_bounds__(kThreads) probs_kernel(const __grid_constant__ ProbsArgs a) {
  __shared__ float s_red[32];
  const int row = blockIdx.x, b = row / a.S, j = row - b * a.S, V = a.V;
  float* p = a.p + (size_t)row * V;
  uint32_t* words = reinterpret_cast<uint32_t*>(p);
  for (int v = threadIdx.x; v < V; v += kThreads) words[v] = 0u;
  __syncthreads();
  if (a.history) {
    const int len = a.history_len ? min(a.history_len[b], a.history_cap) : a.history_cap;
    const int prompt = a.prompt_len ? a.prompt_len[b] : 0;
    for (int i = threadIdx.x; i < len; i += kThreads) {
      const int v = a.history[(size_t)b * a.history_cap + i];
      if (v < 0 || v >= V) continue;
      atomicOr(&words[v], kSeen);
      if (i >= prompt) atomicAdd(&words[v], 1u);
    }
  }
  if (a.draft)
    for (int i = threadIdx.x; i < j; i += kThreads) {
      const int v = a.draft[(size_t)b * a.S + i];
      if (v < 0 || v >= V) continue;
      atomicOr(&words[v], kSeen);
      atomicAdd(&words[v], 1u);
    }
  for (int i = threadIdx.x; i < a.nbias; i += kThreads) {
    const int v = a.bias_ids[(size_t)b * a.nbias + i];
    if (v >= 0 && v < V) atomicOr(&words[v], kBiased);
  }
  __syncthreads();
  const float rep = a.repetition ? a.repetition[b] : 1.f, freq = a.frequency ? a.frequency[b] : 0.f;
  const float pres = a.presence ? a.presence[b] : 0.f, T = a.temperature ? a.temperature[b] : 1.f;
  const uint32_t* mask = a.mask ? a.mask + (size_t)row * ((V + 31) / 32) : nullptr;
  float m = -INFINITY;
  for (int v = threadIdx.x; v < V; v += kThreads) {
    float z = adjust(load_logit(a.logits, (size_t)row * V + v, a.dtype), words[v], a, b, v, rep, freq, pres);
    if (mask && !((mask[v >> 5] >> (v & 31)) & 1u)) z = -INFINITY;
    p[v] = z;
    m = fmaxf(m, z);
  }
  m = block_reduce(m, s_red, [](float x, float y) { return fmaxf(x, y); });
  if (m == -INFINITY) {
    for (int v = threadIdx.x; v < V; v += kThreads) p[v] = 0.f;
    return;
  }
  const bool greedy = !(T > 0.f);
  const float c = 1.4426950408889634f / T;
  // (entries at the maximum count as 1 whatever the temperature; -inf never counts)
  auto weight = [&](float z) { return z == m ? 1.f : z == -INFINITY ? 0.f : exp2f((z - m) * c); };
  float sum = 0.f, first = (float)V;
  for (int v = threadIdx.x; v < V; v += kThreads) {
    if (greedy) {
      if (p[v] == m) first = fminf(first, (float)v);
    } else {
      sum += weight(p[v]);
    }
  }
  sum = block_reduce(sum, s_red, [](float x, float y) { return x + y; });
  first = block_reduce(first, s_red, [](float x, float y) { return fminf(x, y); });
  for (int v = threadIdx.x; v < V; v += kThreads)
    p[v] = greedy ? ((float)v == first ? 1.f : 0.f) : weight(p[v]) / sum;
}

}  // namespace

cudaError_t launch_probs(const ProbsArgs& a, cudaStream_t stream) {
  probs_kernel<<<(unsigned)(a.B * a.S), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace dsa
