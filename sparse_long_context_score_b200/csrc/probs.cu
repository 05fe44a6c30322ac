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
//
// Two passes over chunks of 4096 entries: the first forms each chunk's maximum and sum (or the
// place of its maximum), the second joins the row's chunks and writes p.  The second reads the
// logits from L2: sequences are taken in groups whose logits fit there.  A CTA takes its chunk
// for several rows of a sequence, with the next row's logits in flight.
// The entries that the history, the drafts and the biases name are few and lie anywhere, and what
// they cost must not be paid by all: the first pass gathers them and takes them out of the dense
// stream by a bit each; a kernel behind it adds their share to the row's sums, and one behind the
// second pass puts their probabilities over what that wrote there, a thread an entry.
// 16 x 7 rows of 151552 (68 MB of logits, 68 MB of p), us, without lists / with 4096 tokens of
// history, 32 biases and a mask: 34 / 56.  Tried: a row held in the registers of a cluster of
// eight CTAs, one pass (83 / 133: one such CTA fills an SM, and its loads, lists, exchanges and
// stores follow one another); lists as a number and a bit for every entry (34 / 82: a warp does
// the repetition's arithmetic wherever one of its lanes needs it); the listed entries treated by
// their chunk's CTA, row by row (34 / 144) or behind all rows (34 / 114): most of a history lies
// in one chunk.
#include <cuda_bf16.h>

#include "dsa_common.cuh"
#include "dsa_internal.h"
#include "sm100.cuh"

namespace dsa {
namespace {

// What is known of an entry while the lists are gathered: how often it was generated (drafts
// aside), whether it was seen at all, and whether a bias or a draft names it.
constexpr uint32_t kSeen = 0x80000000u, kBiased = 0x40000000u, kDrafted = 0x20000000u, kCount = 0x1FFFFFFFu;

constexpr double kL2Bytes = 72e6;  // of 126 MB, beside the probabilities that leave through it

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// One pair of a chunk or a row: the largest logit and the sum of exp((z - m) / T) -- where the
// temperature asks for the maximum alone, the lowest index at it.
struct Partial {
  float m, s;
};
constexpr float kNoPlace = 1e9f;  // behind every entry (places are below 2^24: exact in f32)

// Weights are 2^((z - m) c), c = log2(e) / T, wherever m is finite and c is neither zero nor
// infinite.  Other rows (an infinite maximum, temperatures outside the normal range): entries at
// the maximum count as 1 and the others not at all -- but for T = inf, where all above -inf count
// as 1.
__device__ __forceinline__ bool ordinary(float m, float c) { return fabsf(m) < INFINITY && c > 0.f && c < INFINITY; }
__device__ __forceinline__ bool counts_as_one(float z, float m, float c) {
  return c == 0.f && m != INFINITY ? z != -INFINITY : z == m;
}

// The partials of a warp's lanes as one, in every lane.
__device__ __forceinline__ Partial warp_join(Partial x, float c, bool greedy) {
  const float m = warp_max(x.m);
  if (greedy) {
    float first = x.m == m ? x.s : kNoPlace;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) first = fminf(first, __shfl_xor_sync(0xFFFFFFFFu, first, o));
    return {m, first};
  }
  float s = 0.f;
  if (x.m != -INFINITY) s = ordinary(m, c) ? x.s * exp2_approx((x.m - m) * c) : counts_as_one(x.m, m, c) ? x.s : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  return {m, s};
}

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kItems = 16;                  // entries of a thread
constexpr int kChunk = kThreads * kItems;   // 4096
constexpr int kBlocks = 4;                  // CTAs of an SM
constexpr int kRowBlock = 64;               // rows whose partials are joined at once

// The chunk's entry that item i of this thread is: four in a row where rows start on a vector
// (16 bytes of f32, 8 of bf16), else neighbours in neighbouring threads.
template <bool kVector>
__device__ __forceinline__ int place(int i) {
  return kVector ? 4 * (kThreads * (i / 4) + (int)threadIdx.x) + i % 4 : kThreads * i + (int)threadIdx.x;
}
__device__ __forceinline__ float load_f32(const float* p) { return *p; }
__device__ __forceinline__ float load_f32(const __nv_bfloat16* p) { return __bfloat162float(*p); }

template <class T, bool kVector, bool kOnce>
__device__ __forceinline__ void load_row(const T* row, int v0, int v1, float (&z)[kItems]) {
  if constexpr (kVector) {
#pragma unroll
    for (int i = 0; i < kItems; i += 4) {
      const int v = v0 + place<true>(i);
      if (v < v1) {  // (V is a multiple of four)
        if constexpr (sizeof(T) == 4) {
          const float4* p = reinterpret_cast<const float4*>(row + v);
          const float4 x = kOnce ? __ldcs(p) : *p;
          z[i] = x.x, z[i + 1] = x.y, z[i + 2] = x.z, z[i + 3] = x.w;
        } else {
          const uint2* p = reinterpret_cast<const uint2*>(row + v);
          const uint2 x = kOnce ? __ldcs(p) : *p;
          z[i] = __uint_as_float(x.x << 16), z[i + 1] = __uint_as_float(x.x & 0xFFFF0000u);
          z[i + 2] = __uint_as_float(x.y << 16), z[i + 3] = __uint_as_float(x.y & 0xFFFF0000u);
        }
      } else {
        z[i] = z[i + 1] = z[i + 2] = z[i + 3] = -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int v = v0 + place<false>(i);
      z[i] = v < v1 ? load_f32(row + v) : -INFINITY;
    }
  }
}

// A listed entry of a sequence.
struct Listed {
  uint32_t v;      // the entry; kSeen, kBiased; kNobody: a gap
  uint32_t count;  // how often it was generated, drafts aside
  float bias;      // sum of its biases
};
constexpr uint32_t kNobody = 0xFFFFFFFFu, kEntry = 0xFFFFFFu;
// What the first pass leaves for the others: a sequence's listed entries chunk after chunk, with
// gaps -- a chunk's start where they do if every name in the lists were another entry.
struct Lists {
  Listed* entries;  // [B][room]
  int room;         // names in the lists of a sequence at most, rounded up to whole CTAs
};

struct RowSettings {
  float rep, freq, pres, c;
  bool greedy;
};
__device__ __forceinline__ RowSettings row_settings(const ProbsArgs& a, int b) {
  const float temperature = a.temperature ? a.temperature[b] : 1.f;
  return {a.repetition ? a.repetition[b] : 1.f, a.frequency ? a.frequency[b] : 0.f, a.presence ? a.presence[b] : 0.f,
          1.4426950408889634f / temperature, !(temperature > 0.f)};
}

// Two partials as one.
__device__ __forceinline__ Partial lane_join(Partial x, Partial y, float c, bool greedy) {
  const float m = fmaxf(x.m, y.m);
  if (greedy) return {m, fminf(x.m == m ? x.s : kNoPlace, y.m == m ? y.s : kNoPlace)};
  const bool usual = ordinary(m, c);
  auto share = [&](const Partial& p) {
    if (p.m == -INFINITY) return 0.f;
    return usual ? p.s * exp2_approx((p.m - m) * c) : counts_as_one(p.m, m, c) ? p.s : 0.f;
  };
  return {m, share(x) + share(y)};
}
// A row's partials as one, in every lane of the warp.
__device__ __forceinline__ Partial join_row(const Partial* partials, int parts, float c, bool greedy) {
  Partial x{-INFINITY, greedy ? kNoPlace : 0.f};
#pragma unroll 4
  for (int i = threadIdx.x & 31; i < parts; i += 32) {
    const float2 y = __ldcg(reinterpret_cast<const float2*>(partials) + i);
    x = lane_join(x, {y.x, y.y}, c, greedy);
  }
  return warp_join(x, c, greedy);
}

// Notes in words, by entry, what the history and the drafts before row `said` say of the entries
// [v0, v1) of sequence b, and which of them the other drafts name; also counts the names there
// and those before.  words are zero, and the CTA synchronises behind it.
__device__ __forceinline__ void note_tokens(const ProbsArgs& a, int b, int v0, int v1, int said, uint32_t* words, int& names,
                                            int& below) {
  auto note = [&](int v, bool generated, uint32_t mark) {
    below += v >= 0 && v < v0;
    if (v < v0 || v >= v1) return;
    ++names;
    atomicOr(&words[v - v0], mark);
    if (generated) atomicAdd(&words[v - v0], 1u);
  };
  if (a.history) {
    const int32_t* list = a.history + (size_t)b * a.history_cap;
    constexpr int kBatch = 8;
    int v[kBatch];
    auto load = [&](int i0) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = i0 + u * (int)blockDim.x + (int)threadIdx.x;
        v[u] = i < a.history_cap ? list[i] : -1;
      }
    };
    load(0);  // (whatever the length is: that would come first)
    const int len = a.history_len ? min(a.history_len[b], a.history_cap) : a.history_cap;
    const int prompt = a.prompt_len ? a.prompt_len[b] : 0;
    for (int i0 = 0; i0 < len;) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = i0 + u * (int)blockDim.x + (int)threadIdx.x;
        if (i < len) note(v[u], i >= prompt, kSeen);
      }
      i0 += kBatch * (int)blockDim.x;
      if (i0 < len) load(i0);
    }
  }
  if (a.draft)
    for (int i = threadIdx.x; i < a.S - 1; i += blockDim.x)
      note(a.draft[(size_t)b * a.S + i], i < said, i < said ? kSeen : kDrafted);
}

// The shared memory that gathers a chunk's listed entries.
struct Gathered {
  uint32_t words[kChunk];  // by entry
  int number[kWarps];      // listed entries of the warps' threads
  int names, below;        // names in the chunk, and in those before
};
// s_bias: by entry, where biases are given
__device__ __forceinline__ void gather(const ProbsArgs& a, int b, int v0, int v1, Gathered& g, float* s_bias) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i < kChunk / 4; i += kThreads) reinterpret_cast<uint4*>(g.words)[i] = make_uint4(0, 0, 0, 0);
  if (tid == 0) g.names = g.below = 0;
  __syncthreads();
  int below = 0, names = 0;
  note_tokens(a, b, v0, v1, 0, g.words, names, below);
  // a warp sums an entry's biases in the list's order, so that equal ids always sum alike
  const int32_t* ids = a.bias_ids + (size_t)b * a.nbias;
  const float* values = a.bias_values + (size_t)b * a.nbias;
  for (int i0 = 32 * warp; i0 < a.nbias; i0 += kThreads) {
    const int own = i0 + lane < a.nbias ? ids[i0 + lane] : -1;
    below += own >= 0 && own < v0;
    names += own >= v0 && own < v1;
    for (uint32_t todo = __ballot_sync(0xFFFFFFFFu, own >= v0 && own < v1); todo; todo &= todo - 1) {
      const int v = __shfl_sync(0xFFFFFFFFu, own, __ffs(todo) - 1);
      float sum = 0.f;
      for (int k0 = 0; k0 < a.nbias; k0 += 32) {
        const bool same = k0 + lane < a.nbias && ids[k0 + lane] == v;
        const float value = same ? values[k0 + lane] : 0.f;
        for (uint32_t hits = __ballot_sync(0xFFFFFFFFu, same); hits; hits &= hits - 1)
          sum += __shfl_sync(0xFFFFFFFFu, value, __ffs(hits) - 1);
      }
      if (lane == 0) {
        s_bias[v - v0] = sum;
        atomicOr(&g.words[v - v0], kBiased);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    below += __shfl_xor_sync(0xFFFFFFFFu, below, o);
    names += __shfl_xor_sync(0xFFFFFFFFu, names, o);
  }
  if (lane == 0 && below) atomicAdd(&g.below, below);
  if (lane == 0 && names) atomicAdd(&g.names, names);
  __syncthreads();
}

// The listed entries: their partials (kWrite false), or their probabilities, over those that the
// second pass wrote there.  CTA (256 of a sequence's entries, sequence b0 + blockIdx.y, row
// blockIdx.z).  (A CTA for four rows, which finds an entry's count once: 58.6 us the whole call at
// 16 x 7 rows against 55.9; for two 56.4.)
template <class T, bool kWrite>
__global__ void __launch_bounds__(kThreads) probs_listed_kernel(const __grid_constant__ ProbsArgs a, int b0, int chunks,
                                                                Lists lists, Partial* partials) {
  __shared__ Partial s_part[kWarps];
  const int e = blockIdx.x, parts = chunks + gridDim.x, b = b0 + blockIdx.y, j = blockIdx.z, V = a.V;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t row = (size_t)b * a.S + j;
  // Nothing that a kernel before wrote is read ahead of the wait.  (The second of these kernels
  // starts when all CTAs of the second pass are past theirs, which the lists and the partials are
  // complete behind; but only its own wait makes them visible to it.)
  sm100::grid_dep_wait();
  if constexpr (!kWrite) {
    sm100::grid_dep_launch();
  }
  const Listed* entry = lists.entries + (size_t)b * lists.room + kThreads * e + threadIdx.x;
  const uint32_t word = __ldcg(&entry->v), generated = __ldcg(&entry->count);
  const float given = __ldcg(&entry->bias);
  const bool there = word != kNobody;
  const int v = there ? (int)(word & kEntry) : 0;
  const RowSettings set = row_settings(a, b);
  const Partial none{-INFINITY, set.greedy ? kNoPlace : 0.f};
  if (!__syncthreads_or(there)) {  // nothing but gaps
    if constexpr (!kWrite) {
      if (threadIdx.x == 0) partials[row * parts + chunks + e] = none;
    }
    return;
  }
  float z = there ? load_f32(static_cast<const T*>(a.logits) + row * V + v) : -INFINITY;
  const bool allowed = there && (!a.mask || (a.mask[row * ((V + 31) / 32) + (v >> 5)] >> (v & 31)) & 1u);
  uint32_t count = there ? generated : 0u;
  if (a.draft)
    for (int k = 0; k < j; ++k) count += a.draft[(size_t)b * a.S + k] == v;
  if ((word & kSeen) || count) z = z > 0.f ? z / set.rep : z * set.rep;
  if (count) z = z - set.freq * (float)count - set.pres;
  if (there && (word & kBiased)) z += given;
  z = allowed ? fmaxf(z, -INFINITY) : -INFINITY;  // NaN becomes -inf
  if constexpr (!kWrite) {
    Partial x = warp_join({z, set.greedy ? (there ? (float)v : kNoPlace) : z == -INFINITY ? 0.f : 1.f}, set.c, set.greedy);
    if (lane == 0) s_part[warp] = x;
    __syncthreads();
    if (warp == 0) {
      x = warp_join(lane < kWarps ? s_part[lane] : none, set.c, set.greedy);
      if (lane == 0) partials[row * parts + chunks + e] = x;
    }
  } else {
    if (warp == 0) {
      const Partial x = join_row(partials + row * parts, parts, set.c, set.greedy);
      if (lane == 0) s_part[0] = x;
    }
    __syncthreads();
    const Partial x = s_part[0];
    float share = 0.f;
    if (x.m != -INFINITY) {
      if (set.greedy) share = (float)v == x.s ? 1.f : 0.f;
      else share = (ordinary(x.m, set.c) ? exp2_approx((z - x.m) * set.c) : counts_as_one(z, x.m, set.c) ? 1.f : 0.f) / x.s;
    }
    if (there) a.p[row * V + v] = share;
  }
}

// Pass 1 (kWrite false): partials[row][parts], those of the chunks, without the listed entries
// (kLists).  Pass 2: p of all entries, from the row's partials; the listed ones' is put right
// behind it.  CTA (chunk, sequence b0 + blockIdx.y, rows rows_each blockIdx.z ...).
template <class T, bool kVector, bool kLists, bool kWrite>
__global__ void __launch_bounds__(kThreads, kBlocks) probs_kernel(const __grid_constant__ ProbsArgs a, int b0, int rows_each,
                                                                  int parts, Lists lists, Partial* partials) {
  __shared__ __align__(16) unsigned char s_gathered[kLists && !kWrite ? sizeof(Gathered) : 16];
  __shared__ Partial s_part[kWrite ? kRowBlock : kRowBlock * kWarps];
  extern __shared__ float s_bias[];
  Gathered& g = *reinterpret_cast<Gathered*>(s_gathered);
  const int chunk = blockIdx.x, b = b0 + blockIdx.y, V = a.V, S = a.S;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j0 = blockIdx.z * rows_each, j1 = min(S, j0 + rows_each);
  const size_t row0 = (size_t)b * S;
  const int v0 = chunk * kChunk, v1 = min(V, v0 + kChunk);
  const T* logits = static_cast<const T*>(a.logits) + row0 * V;
  float next[kItems];
  load_row<T, kVector, kWrite>(logits + (size_t)j0 * V, v0, v1, next);
  if (kWrite) sm100::grid_dep_wait();  // the partials
  sm100::grid_dep_launch();
  const RowSettings set = row_settings(a, b);
  const float c = set.c;
  const bool greedy = set.greedy;
  uint32_t listed = 0;  // which of this thread's entries are
  if constexpr (kLists && !kWrite) {
    gather(a, b, v0, v1, g, s_bias);
#pragma unroll
    for (int i = 0; i < kItems; ++i) listed |= (g.words[place<kVector>(i)] != 0u ? 1u : 0u) << i;
    if (blockIdx.z == 0) {
      Listed* out = lists.entries + (size_t)b * lists.room + g.below;
      // by thread, not as they come: the order decides how the row's sum is rounded
      const int own = __popc(listed);
      int at = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, at, o);
        if (lane >= o) at += u;
      }
      if (lane == 31) g.number[warp] = at;
      at -= own;
      __syncthreads();
      int number = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) at += g.number[w];
        number += g.number[w];
      }
      for (uint32_t todo = listed; todo; todo &= todo - 1) {
        const uint32_t e = place<kVector>(__ffs(todo) - 1), word = g.words[e];
        out[at++] = {(v0 + e) | (word & (kSeen | kBiased)), word & kCount, word & kBiased ? s_bias[e] : 0.f};
      }
      // gaps: behind this chunk's entries, and behind the last chunk's
      const int end = chunk == (int)gridDim.x - 1 ? lists.room - g.below : g.names;
      for (int i = number + threadIdx.x; i < end; i += kThreads) out[i].v = kNobody;
    }
  }
  // the mask's bits of a row, by entry, without the listed entries; loaded a row ahead
  auto load_bits = [&](int j) {
    uint32_t bits = ~listed;
    if (a.mask) {
      const uint32_t* mask = a.mask + (row0 + j) * ((V + 31) / 32);
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kItems; i += kVector ? 4 : 1) {  // (four in a row lie in one word)
        const int v = v0 + place<kVector>(i);
        m |= ((v < v1 ? mask[v >> 5] >> (v & 31) : 0u) & (kVector ? 15u : 1u)) << i;
      }
      bits &= m;
    }
    return bits;
  };
  uint32_t next_bits = load_bits(j0);
  for (int j = j0; j < j1; ++j) {
    const size_t row = row0 + j;
    if constexpr (kWrite) {
      if ((j - j0) % kRowBlock == 0) {
        __syncthreads();
        for (int r = j + warp; r < min(j1, j + kRowBlock); r += kWarps) {
          const Partial x = join_row(partials + (row0 + r) * parts, parts, c, greedy);
          if (lane == 0) s_part[r - j] = x;
        }
        __syncthreads();
      }
    }
    float z[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) z[i] = next[i];
    const uint32_t bits = next_bits;
    if (j + 1 < j1) {
      load_row<T, kVector, kWrite>(logits + (size_t)(j + 1) * V, v0, v1, next);
      next_bits = load_bits(j + 1);
    }
    if (a.mask || (kLists && !kWrite)) {  // the dense stream goes on without the masked and the listed entries
#pragma unroll
      for (int i = 0; i < kItems; ++i)
        if (!((bits >> i) & 1u)) z[i] = -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) z[i] = fmaxf(z[i], -INFINITY);  // NaN becomes -inf
    if constexpr (!kWrite) {
      Partial x{-INFINITY, greedy ? kNoPlace : 0.f};
#pragma unroll
      for (int i = 0; i < kItems; ++i) x.m = fmaxf(x.m, z[i]);
      // (a warp's maximum, so that its lanes' sums add up without weights)
      x.m = warp_max(x.m);
      if (greedy) {
#pragma unroll
        for (int i = 0; i < kItems; ++i)
          if (z[i] == x.m) x.s = fminf(x.s, (float)(v0 + place<kVector>(i)));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x.s = fminf(x.s, __shfl_xor_sync(0xFFFFFFFFu, x.s, o));
      } else if (x.m != -INFINITY) {
        float m = x.m, scale = c;
        if (!ordinary(m, c)) {
#pragma unroll
          for (int i = 0; i < kItems; ++i) z[i] = counts_as_one(z[i], x.m, c) ? 0.f : -INFINITY;
          m = 0.f;
          scale = 1.f;
        }
#pragma unroll
        for (int i = 0; i < kItems; ++i) x.s += exp2_approx((z[i] - m) * scale);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x.s += __shfl_xor_sync(0xFFFFFFFFu, x.s, o);
      }
      // (the CTA's warps meet once for many rows)
      const int at = (j - j0) % kRowBlock;
      if (lane == 0) s_part[at * kWarps + warp] = x;
      if (at + 1 == kRowBlock || j + 1 == j1) {
        __syncthreads();
        for (int r = warp; r <= at; r += kWarps) {
          const Partial y =
              warp_join(lane < kWarps ? s_part[r * kWarps + lane] : Partial{-INFINITY, greedy ? kNoPlace : 0.f}, c, greedy);
          if (lane == 0) partials[(row - at + r) * parts + chunk] = y;
        }
        if (j + 1 < j1) __syncthreads();
      }
    } else {
      const Partial x = s_part[(j - j0) % kRowBlock];
      const bool usual = ordinary(x.m, c);
      const float m = usual ? x.m : 0.f, scale = usual ? c : 1.f, share = 1.f / x.s;
      if (x.m == -INFINITY) {
#pragma unroll
        for (int i = 0; i < kItems; ++i) z[i] = 0.f;
      } else if (greedy) {
#pragma unroll
        for (int i = 0; i < kItems; ++i) z[i] = (float)(v0 + place<kVector>(i)) == x.s ? 1.f : 0.f;
      } else {
        if (!usual) {
#pragma unroll
          for (int i = 0; i < kItems; ++i) z[i] = counts_as_one(z[i], x.m, c) ? 0.f : -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < kItems; ++i) z[i] = exp2_approx((z[i] - m) * scale) * share;
      }
      float* p = a.p + row * V;
#pragma unroll
      for (int i = 0; i < kItems; i += kVector ? 4 : 1) {
        const int v = v0 + place<kVector>(i);
        if (v >= v1) continue;
        if constexpr (kVector) {
          __stcs(reinterpret_cast<float4*>(p + v), make_float4(z[i], z[i + 1], z[i + 2], z[i + 3]));
        } else {
          __stcs(p + v, z[i]);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- few rows
// One launch: a cluster of up to eight CTAs per row holds it in registers while its maximum and
// sum are formed.  Each warp weighs its entries from its own maximum, and one exchange through
// distributed shared memory joins the warps' pairs (the maximum first, then the sum: 6.1 us
// instead of 5.3 for one row of 50257, replayed).  Few rows are bound by latency and, called one by
// one, by launches: 8 rows of 151552 with 1000 tokens of history take 12.4 us against 21 in two
// passes, replayed 10.1 against 11.3; one row of 50257 8.9 against 14, replayed 5.3 against 4.4.
constexpr int kRowThreads = 512, kMaxRowItems = 40, kMaxCluster = 8;

// A CTA holds kHeld x 512 consecutive entries, a thread four at a time.  kVector as above.
template <class T, int kHeld, bool kVector>
__global__ void __launch_bounds__(kRowThreads) probs_row_kernel(const __grid_constant__ ProbsArgs a, bool lists) {
  using namespace sm100;
  extern __shared__ __align__(16) uint32_t row_words[];  // by entry, when there are lists; behind them logits
  __shared__ Partial s_part[kRowThreads / 32], s_peer[kMaxCluster];
  constexpr int kSlice = kHeld * kRowThreads;
  const int C = gridDim.x, rank = blockIdx.x, row = blockIdx.y, b = row / a.S, j = row - b * a.S, V = a.V;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int v0 = rank * kSlice, v1 = min(V, v0 + kSlice);
  const T* logits = static_cast<const T*>(a.logits) + (size_t)row * V;
  cluster_arrive();  // (a CTA's shared memory is written by its peers once it has started)
  float z[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; i += 4) {
    const int v = v0 + kRowThreads * i + 4 * tid;
    if (kVector && v < v1) {
      if constexpr (sizeof(T) == 4) {
        const float4 x = *reinterpret_cast<const float4*>(logits + v);
        z[i] = x.x, z[i + 1] = x.y, z[i + 2] = x.z, z[i + 3] = x.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(logits + v);
        z[i] = __uint_as_float(x.x << 16), z[i + 1] = __uint_as_float(x.x & 0xFFFF0000u);
        z[i + 2] = __uint_as_float(x.y << 16), z[i + 3] = __uint_as_float(x.y & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) z[i + e] = v + e < v1 ? load_f32(logits + v + e) : -INFINITY;
    }
  }
  const RowSettings set = row_settings(a, b);
  if (lists) {
    for (int i = tid; i < kSlice / 4; i += kRowThreads) reinterpret_cast<uint4*>(row_words)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    int names = 0, below = 0;
    note_tokens(a, b, v0, v1, j, row_words, names, below);
    for (int i = tid; i < a.nbias; i += kRowThreads) {
      const int v = a.bias_ids[(size_t)b * a.nbias + i];
      if (v >= v0 && v < v1) atomicOr(&row_words[v - v0], kBiased);
    }
    __syncthreads();
  }
  auto adjust = [&](float x, uint32_t word, int v) {
    if (word & kSeen) x = x > 0.f ? x / set.rep : x * set.rep;
    if (word & kCount) x = x - set.freq * (float)(word & kCount) - set.pres;
    if (word & kBiased) {  // in the list's order, so that equal ids always sum alike
      float sum = 0.f;
      for (int i = 0; i < a.nbias; ++i)
        if (a.bias_ids[(size_t)b * a.nbias + i] == v) sum += a.bias_values[(size_t)b * a.nbias + i];
      x += sum;
    }
    return x;
  };
  // A thread's listed entries one after another, by way of shared memory: the arithmetic on them is
  // long, and a warp goes through it as often as its lane of most such entries has them, not for
  // every entry that one of its lanes has listed (8 rows of 151552 with 1000 tokens of history:
  // 13.2 us that way).
  unsigned long long listed = 0;
  if (lists) {
    float* s_z = reinterpret_cast<float*>(row_words + kSlice);
#pragma unroll
    for (int i = 0; i < kHeld; i += 4) {
      const int at = kRowThreads * i + 4 * tid;
      const uint4 w = *reinterpret_cast<const uint4*>(row_words + at);
      if (w.x | w.y | w.z | w.w) {
        listed |= (unsigned long long)((w.x ? 1 : 0) | (w.y ? 2 : 0) | (w.z ? 4 : 0) | (w.w ? 8 : 0)) << i;
        *reinterpret_cast<float4*>(s_z + at) = make_float4(z[i], z[i + 1], z[i + 2], z[i + 3]);
      }
    }
    for (unsigned long long todo = listed; todo; todo &= todo - 1) {
      const int i = __ffsll(todo) - 1, at = kRowThreads * (i & ~3) + 4 * tid + (i & 3);
      s_z[at] = adjust(s_z[at], row_words[at], v0 + at);
    }
#pragma unroll
    for (int i = 0; i < kHeld; i += 4) {
      if ((listed >> i) & 15u) {
        const float4 x = *reinterpret_cast<const float4*>(s_z + kRowThreads * i + 4 * tid);
        z[i] = x.x, z[i + 1] = x.y, z[i + 2] = x.z, z[i + 3] = x.w;
      }
    }
  }
  const uint32_t* mask = a.mask ? a.mask + (size_t)row * ((V + 31) / 32) : nullptr;
  Partial x{-INFINITY, set.greedy ? kNoPlace : 0.f};  // the warp's, then the CTA's, then the row's
#pragma unroll
  for (int i = 0; i < kHeld; i += 4) {
    const int v = v0 + kRowThreads * i + 4 * tid;
    const uint32_t bits = mask && v < v1 ? mask[v >> 5] >> (v & 31) : 0xFu;  // (four in a row lie in one word)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      z[i + e] = (bits >> e) & 1u ? fmaxf(z[i + e], -INFINITY) : -INFINITY;  // NaN becomes -inf
      x.m = fmaxf(x.m, z[i + e]);
    }
  }
  x.m = warp_max(x.m);
  const float own = x.m;
  if (set.greedy) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (z[i] == own) x.s = fminf(x.s, (float)(v0 + kRowThreads * (i / 4 * 4) + 4 * tid + i % 4));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x.s = fminf(x.s, __shfl_xor_sync(0xFFFFFFFFu, x.s, o));
  } else {  // weights from the warp's maximum
    const bool usual = ordinary(own, set.c);
    if (!usual) {
#pragma unroll
      for (int i = 0; i < kHeld; ++i) z[i] = own != -INFINITY && counts_as_one(z[i], own, set.c) ? 0.f : -INFINITY;
    }
    const float from = usual ? own : 0.f, scale = usual ? set.c : 1.f;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      z[i] = exp2_approx((z[i] - from) * scale);
      x.s += z[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x.s += __shfl_xor_sync(0xFFFFFFFFu, x.s, o);
  }
  const Partial none{-INFINITY, set.greedy ? kNoPlace : 0.f};
  if (lane == 0) s_part[warp] = x;
  __syncthreads();
  cluster_wait();
  if (warp == 0) {
    x = warp_join(lane < kRowThreads / 32 ? s_part[lane] : none, set.c, set.greedy);
    if (lane < C) {
      const uint32_t to = cluster_map(smem_u32(&s_peer[rank]), lane);
      st_cluster_u32(to, __float_as_uint(x.m));
      st_cluster_u32(to + 4, __float_as_uint(x.s));
    }
  }
  cluster_sync();
  x = warp_join(lane < C ? s_peer[lane] : none, set.c, set.greedy);
  // what a weight from the warp's maximum is of the row's sum
  float share = 0.f;
  if (set.greedy) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) z[i] = (float)(v0 + kRowThreads * (i / 4 * 4) + 4 * tid + i % 4) == x.s ? 1.f : 0.f;
    share = x.m == -INFINITY ? 0.f : 1.f;
  } else if (own != -INFINITY) {
    share = (ordinary(x.m, set.c) ? exp2_approx((own - x.m) * set.c) : counts_as_one(own, x.m, set.c) ? 1.f : 0.f) / x.s;
  }
  float* p = a.p + (size_t)row * V;
#pragma unroll
  for (int i = 0; i < kHeld; i += 4) {
    const int v = v0 + kRowThreads * i + 4 * tid;
    if (kVector && v < v1) {
      *reinterpret_cast<float4*>(p + v) = make_float4(z[i] * share, z[i + 1] * share, z[i + 2] * share, z[i + 3] * share);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (v + e < v1) p[v + e] = z[i + e] * share;
    }
  }
}

template <class T, int kHeld, bool kVector>
cudaError_t launch_rows(const ProbsArgs& a, int C, cudaStream_t stream) {
  auto kernel = probs_row_kernel<T, kHeld, kVector>;
  const bool lists = a.history || (a.draft && a.S > 1) || a.nbias > 0;
  static DeviceOnce once;
  cudaError_t e = once.run([&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * kHeld * kRowThreads * (int)sizeof(uint32_t));
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C, a.B * a.S);
  cfg.blockDim = dim3(kRowThreads);
  cfg.dynamicSmemBytes = lists ? 2 * kHeld * kRowThreads * sizeof(uint32_t) : 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, lists);
}

// ---------------------------------------------------------------- launches
struct ProbsLayout {
  size_t partials, entries, total;
  int chunks, room;
};
ProbsLayout probs_layout(int B, int S, int V, int history_cap, int nbias) {
  ProbsLayout l;
  l.chunks = (V + kChunk - 1) / kChunk;
  l.room = (history_cap + S + nbias + kThreads - 1) / kThreads * kThreads;
  l.partials = 0;
  l.entries = ((size_t)B * S * (l.chunks + l.room / kThreads) * sizeof(Partial) + 255) & ~(size_t)255;
  l.total = l.entries + (size_t)B * l.room * sizeof(Listed);
  return l;
}

template <class T, bool kVector, bool kLists>
cudaError_t launch_passes(const ProbsArgs& a, unsigned char* ws, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const ProbsLayout l = probs_layout(a.B, a.S, a.V, a.history ? a.history_cap : 0, a.nbias);
  const int entry_parts = kLists ? l.room / kThreads : 0, parts = l.chunks + entry_parts;
  Partial* partials = reinterpret_cast<Partial*>(ws + l.partials);
  const Lists lists{reinterpret_cast<Listed*>(ws + l.entries), l.room};
  // sequences whose logits stay in L2 between the passes, and that the grid can number
  const double each = (double)a.S * a.V * sizeof(T);
  int group = each >= kL2Bytes ? 1 : (int)(kL2Bytes / each);
  if (group > 65535) group = 65535;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // waits in-kernel
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  for (int b0 = 0; b0 < a.B; b0 += group) {
    const int n = a.B - b0 < group ? a.B - b0 : group;
    // rows of a CTA: as many as leave a CTA for each place on the GPU
    long long rows_each = (long long)l.chunks * n * a.S / ((long long)kBlocks * sms);
    rows_each = rows_each < 1 ? 1 : rows_each > a.S ? a.S : rows_each;
    const dim3 grid(l.chunks, n, (unsigned)((a.S + rows_each - 1) / rows_each));
    const dim3 entry_grid(entry_parts, n, a.S);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.dynamicSmemBytes = kLists && a.nbias > 0 ? kChunk * sizeof(float) : 0;
    cudaError_t e = cudaLaunchKernelEx(&cfg, probs_kernel<T, kVector, kLists, false>, a, b0, (int)rows_each, parts, lists, partials);
    if (e != cudaSuccess) return e;
    cfg.dynamicSmemBytes = 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (kLists) {
      cfg.gridDim = entry_grid;
      if ((e = cudaLaunchKernelEx(&cfg, probs_listed_kernel<T, false>, a, b0, l.chunks, lists, partials)) != cudaSuccess)
        return e;
      cfg.gridDim = grid;
    }
    if ((e = cudaLaunchKernelEx(&cfg, probs_kernel<T, kVector, false, true>, a, b0, (int)rows_each, parts, lists, partials)) !=
        cudaSuccess)
      return e;
    if (kLists) {
      cfg.gridDim = entry_grid;
      if ((e = cudaLaunchKernelEx(&cfg, probs_listed_kernel<T, true>, a, b0, l.chunks, lists, partials)) != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

// CTAs of a cluster for each row, or 0: two passes.  Rows that clusters hold all at once take as
// many CTAs as keep a thread at eight entries or more.  Two CTAs of up to 24 entries a thread share
// an SM (32 rows of 50257 take 17 us either way); of 40, one, and clusters leave some SMs out
// (151552, with 1000 tokens of history: 12 rows 12.5 us against 21, 16 rows 20.8 either way and
// 18.6 against 14.3 replayed).
int row_cluster(int B, int S, int V, int& held) {
  const int per_cta = 8 * kRowThreads, sms = device_sm_count();
  const int C = (V + per_cta - 1) / per_cta < kMaxCluster ? (V + per_cta - 1) / per_cta : kMaxCluster;
  held = (V + C * kRowThreads - 1) / (C * kRowThreads);
  return held <= kMaxRowItems && (long long)B * S * C <= (held <= 24 ? 2 * sms : sms * 3 / 4) ? C : 0;
}

template <class T, bool kVector>
cudaError_t launch(const ProbsArgs& a, unsigned char* ws, cudaStream_t stream) {
  int held;
  if (const int C = row_cluster(a.B, a.S, a.V, held)) {  // the fewest entries a thread that hold a row
    if (held <= 8) return launch_rows<T, 8, kVector>(a, C, stream);
    if (held <= 16) return launch_rows<T, 16, kVector>(a, C, stream);
    if (held <= 24) return launch_rows<T, 24, kVector>(a, C, stream);
    return launch_rows<T, 40, kVector>(a, C, stream);
  }
  // (one row's drafts have none before it)
  return a.history || (a.draft && a.S > 1) || a.nbias > 0 ? launch_passes<T, kVector, true>(a, ws, stream)
                                                          : launch_passes<T, kVector, false>(a, ws, stream);
}

}  // namespace

size_t probs_workspace_bytes(int B, int S, int V, int history_cap, int nbias) {
  int held;
  return row_cluster(B, S, V, held) ? 0 : probs_layout(B, S, V, history_cap, nbias).total;
}

cudaError_t launch_probs(const ProbsArgs& a, void* workspace, cudaStream_t stream) {
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  const uintptr_t align = a.dtype == DSA_F32 ? 16 : 8;
  const bool vector = a.V % 4 == 0 && reinterpret_cast<uintptr_t>(a.logits) % align == 0 &&
                      reinterpret_cast<uintptr_t>(a.p) % 16 == 0;
  if (a.dtype == DSA_F32) return vector ? launch<float, true>(a, ws, stream) : launch<float, false>(a, ws, stream);
  return vector ? launch<__nv_bfloat16, true>(a, ws, stream) : launch<__nv_bfloat16, false>(a, ws, stream);
}

}  // namespace dsa
