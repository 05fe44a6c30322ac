// paged_attn.cu -- MLA attention of a chunk of new tokens over a paged compressed cache.
//
//   out[t, h] = sum_s softmax_s(scale q[t, h] . c[s]) c[s][0:512],  s <= position of t,
// c[s] the 576-wide row of position s, in page table[b][s / page_size] at s % page_size.
// lse[t, h] = ln sum_s exp(scale q[t, h] . c[s]).
//
// A sequence's query rows (token, head) are one matrix [n_b H, 576], cut into tiles of 64
// rows whatever H is; a tile visits the 128-row key tiles that its last token sees.  The
// (query tile, key tile) pairs of the whole batch, in order, are dealt out in equal
// contiguous shares, one a CTA and one CTA an SM: a long context is split over CTAs when
// there are few query rows, and a CTA works through many query tiles when there are many.
// paged_plan_kernel finds where each share starts (lengths are read on the device);
// a query tile that one CTA covers is written directly, the parts of one that crosses a
// share's border go to the workspace in 32 bits and paged_combine_kernel joins them in the
// CTAs' order (no atomics: the result does not depend on timing).
//
// One key tile of a CTA, everything in shared memory beside the 64 query rows (73.7 KB):
//   S   = Q K^T    M = 64 rows, N = 128 keys, K = 576   (36 MMAs; TMEM lane = query row)
//   O^T += V^T P^T M = 4 x 128 value dims, N = 64 rows, K = 128 keys (32 MMAs)
// The tile (147.5 KB) fills the rest of shared memory as nine blocks of 64 columns, and
// there is no second one: S takes the blocks as they arrive, and each quarter of PV gives
// two of them back, so the next tile's loads run behind PV and the next S behind the
// loads.  (Two half tiles of 64 keys in turn would hide the softmax, but an MMA with M = 64
// costs nearly as much at N = 64 as at N = 128: S would take 1.7 times as long.)
#include <cudaTypedefs.h>

#include "dsa_common.cuh"
#include "dsa_internal.h"
#include "sm100.cuh"

namespace dsa {
namespace {

using namespace sm100;

__device__ int g_paged_error;

constexpr int kRows = 64;                        // query rows of a tile
constexpr int kKeys = 128;                       // cached rows of a key tile
constexpr int kBlocks = kDqk / 64;               // nine 64-wide column blocks of a row
constexpr int kQBlockBytes = kRows * 128;
constexpr int kQBytes = kBlocks * kQBlockBytes;  // 73728
constexpr int kBlockBytes = kKeys * 128;         // 16384
constexpr int kStageBytes = kBlocks * kBlockBytes;  // 147456
// P of a tile (64 rows x 128 keys bf16, two 8 KB halves of 64 keys) is written over the
// tile's rotary block, which only S reads
constexpr int kPBlock = kDv / 64;
constexpr int kSegs = 4;                         // query tile segments in flight

constexpr int kLoadWarp = 0, kMmaWarp = 1, kQueryWarp = 2, kWalkWarp = 3, kSoftmaxWarp0 = 4;
constexpr int kSoftmaxThreads = 256;             // eight warps: two per TMEM lane quarter
constexpr int kThreadsP = kSoftmaxWarp0 * 32 + kSoftmaxThreads;  // 384
constexpr float kRescaleLog2 = 8.f;

// One CTA's part of a query tile.
struct Segment {
  int b;         // sequence; -1: no more
  int row0;      // first query row (token * H + head) in q
  int nrows;     // rows of the tile that exist
  int tile_row;  // the same row, counted from the sequence's first
  int k0, k1;    // key tiles
  int seen0;     // cached rows that the sequence's first new token sees
  int limit;     // cached rows of the sequence
  int part;      // workspace slot of this part of the tile; -1: the tile is whole
};

// Where a CTA's share starts: key tile k0 of query tile `tile` of sequence b.
struct Share {
  int b, tile, k0;
};
struct Plan {
  int per_cta;  // key tiles of a share
  int pad[3];
};

constexpr int kOffQ = 0;
constexpr int kOffStage = kOffQ + kQBytes;
constexpr int kOffMax = kOffStage + kStageBytes;     // [2][64] f32: a tile's maxima, per half of the keys
constexpr int kOffAlpha = kOffMax + 2 * 64 * 4;      // [64] f32
constexpr int kOffL = kOffAlpha + 64 * 4;            // [2][64] f32
constexpr int kOffM = kOffL + 2 * 64 * 4;            // [64] f32
constexpr int kOffVote = kOffM + 64 * 4;             // [8] u32, one per softmax warp
constexpr int kOffBad = kOffVote + 8 * 4;            // u32: 16-row groups of the tile that are not there
constexpr int kOffSeg = kOffBad + 32;
constexpr int kOffBar = kOffSeg + kSegs * (int)sizeof(Segment) + 16;
constexpr int kNumBars = kBlocks + 5 + 2 * kSegs + 8;
constexpr int kOffTmem = kOffBar + kNumBars * 8;
constexpr int kSmemP = kOffTmem + 16 + 1024;         // + alignment slack
static_assert(kOffBar % 8 == 0, "barrier alignment");
static_assert(kSmemP <= 232448, "shared memory budget");

constexpr int kTmemO = 0;      // O^T: 4 blocks x 64 columns, all 128 lanes
constexpr int kTmemS = 256;    // S: 128 columns, lanes 0..15 of each quarter
constexpr int kTmemCols = 512;

constexpr int kPartFloats = kRows * kDv;             // one part's [64][512] sums

// The plan and the parts are read behind griddepcontrol.wait by volatile loads: a load that
// the compiler may take for one of constant data could move above the wait.
__device__ __forceinline__ Share load_share(const Share* p) {
  const volatile int* v = reinterpret_cast<const volatile int*>(p);
  return Share{v[0], v[1], v[2]};
}

// rows of a sequence's query tile, and the key tiles that it visits (at least one, so that
// rows which see nothing are written too)
struct SequenceWork {
  int tiles, rows, seen0, limit;
};
__device__ __forceinline__ SequenceWork sequence_work(const PagedBatch& p, int b, int H) {
  const int q0 = p.cu_q[b], nb = max(min(p.cu_q[b + 1], p.n) - q0, 0);
  const int full = p.cu_q[b + 1] - q0;
  SequenceWork w;
  w.rows = q0 < 0 ? 0 : nb * H;
  w.tiles = (w.rows + kRows - 1) / kRows;
  const long long most = (long long)p.max_pages * p.page_size;
  w.limit = (int)max(0LL, min((long long)p.ctx_len[b], most));
  w.seen0 = p.ctx_len[b] - full + 1;
  return w;
}
__device__ __forceinline__ int tile_keys(const SequenceWork& w, int tile, int H) {
  const int last = min(kRows * (tile + 1), w.rows) - 1;
  const int seen = min(w.seen0 + last / H, w.limit);
  return max(1, (seen + kKeys - 1) / kKeys);
}

// Deals the (query tile, key tile) pairs out: one warp sums a sequence's pairs, a scan over
// the sequences gives the total, and a second pass over the tiles notes where each share
// starts.
__global__ void __launch_bounds__(1024) paged_plan_kernel(PagedBatch p, int H, int ctas, long long* __restrict__ before,
                                                          Plan* __restrict__ plan, Share* __restrict__ shares) {
  __shared__ long long s_warp[32];
  __shared__ long long s_total;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_launch();
  for (int g = threadIdx.x; g < ctas; g += 1024) shares[g].b = -1;
  for (int b = warp; b < p.B; b += 32) {
    const SequenceWork w = sequence_work(p, b, H);
    long long sum = 0;
    for (int i = lane; i < w.tiles; i += 32) sum += tile_keys(w, i, H);
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) before[b] = sum;
  }
  if (threadIdx.x == 0) s_total = 0;
  __syncthreads();
  for (int b0 = 0; b0 < p.B; b0 += 1024) {  // exclusive sums over the sequences
    const int b = b0 + threadIdx.x;
    const long long own = b < p.B ? before[b] : 0;
    long long v = own;
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) s_warp[warp] = v;
    __syncthreads();
    if (warp == 0) {
      long long t = s_warp[lane];
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xFFFFFFFFu, t, o);
        if (lane >= o) t += u;
      }
      s_warp[lane] = t;
    }
    __syncthreads();
    const long long base = s_total;
    if (b < p.B) before[b] = base + (warp ? s_warp[warp - 1] : 0) + v - own;
    __syncthreads();
    if (threadIdx.x == 0) s_total = base + s_warp[31];
    __syncthreads();
  }
  const long long total = s_total;
  const int per = (int)max(1LL, (total + ctas - 1) / ctas);
  if (threadIdx.x == 0) plan->per_cta = per;
  for (int b = warp; b < p.B; b += 32) {
    const SequenceWork w = sequence_work(p, b, H);
    long long at = before[b];
    for (int i0 = 0; i0 < w.tiles; i0 += 32) {
      const int i = i0 + lane, k = i < w.tiles ? tile_keys(w, i, H) : 0;
      int v = k;
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += u;
      }
      const long long first = at + v - k;  // the tile's pairs are [first, first + k)
      for (long long g = (first + per - 1) / per; g * per < first + k; ++g) {
        Share s{b, i, (int)(g * per - first)};
        shares[g] = s;
      }
      at += __shfl_sync(0xFFFFFFFFu, v, 31);
    }
  }
}

__global__ void __launch_bounds__(kThreadsP, 1)
paged_attn_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap cmap, PagedBatch p, int H,
                  int box, float scale_log2, const Plan* plan, const Share* shares, uint16_t* out, float* lse, float* parts,
                  float2* part_ml, int* err) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sQ = sbase + kOffQ, sStage = sbase + kOffStage;
  float* s_max = reinterpret_cast<float*>(smem + kOffMax);
  float* s_alpha = reinterpret_cast<float*>(smem + kOffAlpha);
  float* s_l = reinterpret_cast<float*>(smem + kOffL);
  float* s_m = reinterpret_cast<float*>(smem + kOffM);
  volatile uint32_t* s_vote = reinterpret_cast<volatile uint32_t*>(smem + kOffVote);
  volatile uint32_t* s_bad = reinterpret_cast<volatile uint32_t*>(smem + kOffBad);
  Segment* s_seg = reinterpret_cast<Segment*>(smem + kOffSeg);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kOffTmem);
  const uint32_t bar0 = sbase + kOffBar;
  auto full_bar = [&](int i) { return bar0 + 8u * i; };                          // block i has landed
  auto free_bar = [&](int i) { return bar0 + 8u * (kBlocks + i); };              // blocks 2i, 2i + 1 (i < 4), block 8
  auto segfull_bar = [&](int i) { return bar0 + 8u * (kBlocks + 5 + i); };
  auto segfree_bar = [&](int i) { return bar0 + 8u * (kBlocks + 5 + kSegs + i); };
  const uint32_t bars = bar0 + 8u * (kBlocks + 5 + 2 * kSegs);
  const uint32_t qfull_bar = bars, qfree_bar = bars + 8, sfull_bar = bars + 16, pfull_bar = bars + 24;
  const uint32_t ofull_bar = bars + 32, ofree_bar = bars + 40, grp_bar = bars + 48, done_bar = bars + 56;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;
  grid_dep_launch();  // the combine may be scheduled; it waits on the device for this grid
  if (threadIdx.x == 0) {
    for (int i = 0; i < kBlocks; ++i) mbar_init(full_bar(i), 1);
    for (int i = 0; i < 5; ++i) mbar_init(free_bar(i), 1);
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(segfull_bar(i), 1);
      mbar_init(segfree_bar(i), 3 + kSoftmaxThreads / 32);  // load, MMA, query and softmax warps
    }
    mbar_init(qfull_bar, 1);
    mbar_init(qfree_bar, 1);
    mbar_init(sfull_bar, 1);
    mbar_init(pfull_bar, kSoftmaxThreads);
    mbar_init(ofull_bar, 1);
    mbar_init(ofree_bar, kSoftmaxThreads);
    mbar_init(grp_bar, kSoftmaxThreads);
    mbar_init(done_bar, 1);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(s_tmem), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  // A bounded wait of a whole warp, which goes on or gives up together.
  auto warp_wait = [&](uint32_t bar, uint32_t parity, int code) {
    return (bool)__all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, err, code));
  };
  // The next segment of this CTA's share, for the warp's lanes alike; false at the end.
  int seg_i = 0;
  auto next_segment = [&](Segment& s) {
    const int at = seg_i % kSegs;
    if (!warp_wait(segfull_bar(at), (seg_i / kSegs) & 1, 41)) return false;
    s = s_seg[at];
    __syncwarp();
    if (lane == 0) mbar_arrive(segfree_bar(at));
    ++seg_i;
    return s.b >= 0;
  };

  if (warp == kWalkWarp) {
    // ------------------------------------------------------------------ segments
    if (lane == 0) {
      tma_prefetch(&qmap);
      tma_prefetch(&cmap);
      grid_dep_wait();  // the plan (and with it all that was written before it)
      const Share first = load_share(shares + cta);
      int left = *reinterpret_cast<const volatile int*>(&plan->per_cta), b = first.b, tile = first.tile, k0 = first.k0;
      SequenceWork w{0, 0, 0, 0};
      if (b >= 0) w = sequence_work(p, b, H);
      for (int i = 0;; ++i) {
        const int at = i % kSegs;
        Segment s;
        s.b = -1;
        while (b >= 0 && b < p.B && tile >= w.tiles) {  // the next sequence that has rows
          tile = 0;
          if (++b < p.B) w = sequence_work(p, b, H);
        }
        if (b >= 0 && b < p.B && left > 0) {
          const int keys = tile_keys(w, tile, H);
          s.b = b;
          s.tile_row = kRows * tile;
          s.row0 = p.cu_q[b] * H + s.tile_row;
          s.nrows = min(kRows, w.rows - s.tile_row);
          s.k0 = k0;
          s.k1 = min(keys, k0 + left);
          s.seen0 = w.seen0;
          s.limit = w.limit;
          s.part = k0 > 0 ? 2 * cta : s.k1 < keys ? 2 * cta + 1 : -1;
          left -= s.k1 - k0;
          k0 = 0;
          ++tile;
        }
        if (!mbar_wait(segfree_bar(at), ((i / kSegs) & 1) ^ 1, err, 42)) break;
        s_seg[at] = s;
        mbar_arrive(segfull_bar(at));
        if (s.b < 0) break;
      }
    }
    __syncwarp();
  } else if (warp == kQueryWarp) {
    // ------------------------------------------------------------------ queries
    Segment s;
    int issued = 0;
    for (int i = 0; next_segment(s); ++i) {
      if (!warp_wait(qfree_bar, (i & 1) ^ 1, 43)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(qfull_bar, kQBytes);
        for (int kb = 0; kb < kBlocks; ++kb) tma_load_2d(sQ + kb * kQBlockBytes, &qmap, qfull_bar, 64 * kb, s.row0);
      }
      issued = i + 1;
    }
    if (lane == 0 && issued) mbar_wait_drain(qfull_bar, (issued - 1) & 1);  // none in flight on the way out
    __syncwarp();
  } else if (warp == kLoadWarp) {
    // ------------------------------------------------------------------ key tiles
    // lane l brings rows [box l, box (l + 1)) of a tile, which lie in one page
    const int boxes = kKeys / box;
    Segment s;
    int it = 0, posted = 0;  // key tiles, and blocks asked for
    bool ok = true;
    while (ok && next_segment(s)) {
      const int32_t* table = p.table + (size_t)s.b * p.max_pages;
      auto page_row = [&](int k) {  // pool row of this lane's box in key tile k, -1 where there is none
        if (lane >= boxes || k >= s.k1) return -1;
        const long long pos = (long long)kKeys * k + box * lane;
        const long long i = pos / p.page_size;
        if (i >= p.max_pages) return -1;
        const int page = table[i];
        return page >= 0 && page < p.num_pages ? page * p.page_size + (int)(pos - i * p.page_size) : -1;
      };
      int row = page_row(s.k0);
      for (int k = s.k0; k < s.k1; ++k, ++it) {
        const int ahead = page_row(k + 1);  // in flight while this tile is waited for
        const uint32_t there = __ballot_sync(0xFFFFFFFFu, row >= 0);
        uint32_t bad = 0;  // per 16 rows
        for (int i = 0; i < kKeys / 16; ++i) bad |= ((there >> (i * 16 / box)) & 1u ? 0u : 1u) << i;
#pragma unroll 1
        for (int kb = 0; kb < kBlocks; ++kb) {
          if ((kb & 1) == 0) {
            ok = warp_wait(free_bar(kb >> 1), (it & 1) ^ 1, 44);
            if (!ok) break;
          }
          if (lane == 0) {
            if (kb == 0) *s_bad = bad;
            mbar_arrive_expect_tx(full_bar(kb), kBlockBytes);
          }
          __syncwarp();
          if (lane < boxes)
            tma_load_2d(sStage + kb * kBlockBytes + lane * box * 128, &cmap, full_bar(kb), 64 * kb, row >= 0 ? row : 0);
          ++posted;
        }
        if (!ok) break;
        row = ahead;
      }
    }
    // nothing in flight on the way out: every block that was asked for has landed
    if (lane == 0)
      for (int kb = 0; kb < kBlocks && kb < posted; ++kb) mbar_wait_drain(full_bar(kb), ((posted - 1 - kb) / kBlocks) & 1);
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------ tensor core
    const bool leader = elect_one();
    constexpr uint32_t idS = idesc_bf16_f32(kRows, kKeys);          // Q (K-major) x K (K-major)
    constexpr uint32_t idPV = idesc_bf16_f32(128, kRows, true, false);  // V^T (M-major) x P (K-major)
    const uint64_t dq = sdesc_kmajor_sw128(sQ), dk = sdesc_kmajor_sw128(sStage);
    const uint64_t dv = sdesc_mnmajor_sw128(sStage, kBlockBytes, 1024);
    const uint64_t dp = sdesc_kmajor_sw128(sStage + kPBlock * kBlockBytes);
    Segment s;
    int it = 0;
    bool ok = true;
    for (int i = 0; ok && next_segment(s); ++i) {
      ok = warp_wait(qfull_bar, i & 1, 45);
      for (int k = s.k0; ok && k < s.k1; ++k, ++it) {
#pragma unroll 1
        for (int kb = 0; ok && kb < kBlocks; ++kb) {
          ok = warp_wait(full_bar(kb), it & 1, 46);
          if (!ok) break;
          if (kb == 0) tc_fence_after();
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16(tmem + kTmemS, dq + (uint64_t)((kb * kQBlockBytes + kk * 32) >> 4),
                       dk + (uint64_t)((kb * kBlockBytes + kk * 32) >> 4), idS, kb + kk > 0);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (leader) {
          mma_commit(sfull_bar);
          if (k + 1 == s.k1) mma_commit(qfree_bar);
        }
        __syncwarp();
        // the epilogue of the segment before has read O
        if (k == s.k0) ok = warp_wait(ofree_bar, (i & 1) ^ 1, 47);
        ok = ok && warp_wait(pfull_bar, it & 1, 48);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
#pragma unroll 1
          for (int mb = 0; mb < 4; ++mb) {
#pragma unroll
            for (int ks = 0; ks < kKeys / 16; ++ks)
              mma_bf16(tmem + kTmemO + 64 * mb, dv + (uint64_t)((2 * mb * kBlockBytes + ks * 16 * 128) >> 4),
                       dp + (uint64_t)(((ks >> 2) * (kBlockBytes / 2) + (ks & 3) * 32) >> 4), idPV,
                       k > s.k0 || ks > 0 ? 1u : 0u);
            mma_commit(free_bar(mb));
          }
          mma_commit(free_bar(4));
          if (k + 1 == s.k1) mma_commit(ofull_bar);
        }
        __syncwarp();
      }
    }
    if (leader) {
      mma_commit(done_bar);
      if (!mbar_wait_drain(done_bar, 0)) atomicCAS(err, 0, 49);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ softmax and epilogue
    // Warp w reads TMEM lane quarter w % 4 and keys [64 half, 64 half + 64) of a tile: a
    // thread gets rows rA = 16 quarter + lane / 4 and rB = rA + 8, keys 8 j + 2 (lane % 4) +
    // {0, 1} of the half (j < 8).
    const int quarter = warp & 3, half = (warp - kSoftmaxWarp0) >> 2, c4 = lane & 3;
    const int rA = 16 * quarter + (lane >> 2), rB = rA + 8;
    const uint32_t lane_addr = (uint32_t)(32 * quarter) << 16;
    const int st = threadIdx.x - 32 * kSoftmaxWarp0;  // 0 .. 255
    unsigned char* pbase = smem + kOffStage + kPBlock * kBlockBytes + half * (kBlockBytes / 2);
    unsigned char* prowA = pbase + rA * 128 + 4 * c4;
    unsigned char* prowB = pbase + rB * 128 + 4 * c4;
    uint32_t grp_phase = 0;
    auto group_sync = [&](int code) {
      mbar_arrive(grp_bar);
      const bool ok = mbar_wait(grp_bar, grp_phase, err, code);
      grp_phase ^= 1;
      return ok;
    };
    Segment s;
    int it = 0;
    bool ok = true;
    for (int i = 0; ok && next_segment(s); ++i) {
      // cached rows that this thread's query rows see
      const int seenA = rA < s.nrows ? max(0, min(s.seen0 + (s.tile_row + rA) / H, s.limit)) : 0;
      const int seenB = rB < s.nrows ? max(0, min(s.seen0 + (s.tile_row + rB) / H, s.limit)) : 0;
      float mA = -INFINITY, mB = -INFINITY, lA = 0.f, lB = 0.f;
      for (int k = s.k0; k < s.k1; ++k, ++it) {
        ok = warp_wait(full_bar(0), it & 1, 50) && warp_wait(sfull_bar, it & 1, 51);
        if (!ok) break;
        tc_fence_after();
        const uint32_t bad = *s_bad;
        uint32_t r[32];
        tmem_ld16x256b_x8(tmem + lane_addr + kTmemS + 64 * half, r);
        tmem_ld_wait();
        const int key0 = kKeys * k + 64 * half + 2 * c4;
        float tA = -INFINITY, tB = -INFINITY;
        if (bad == 0 && __all_sync(0xFFFFFFFFu, kKeys * (k + 1) <= min(seenA, seenB))) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              r[4 * j + e] = __float_as_uint(__uint_as_float(r[4 * j + e]) * scale_log2);
              r[4 * j + 2 + e] = __float_as_uint(__uint_as_float(r[4 * j + 2 + e]) * scale_log2);
              tA = fmaxf(tA, __uint_as_float(r[4 * j + e]));
              tB = fmaxf(tB, __uint_as_float(r[4 * j + 2 + e]));
            }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int key = key0 + 8 * j + e;
              const bool there = !((bad >> (4 * half + (j >> 1))) & 1u);
              const float zA = there && key < seenA ? __uint_as_float(r[4 * j + e]) * scale_log2 : -INFINITY;
              const float zB = there && key < seenB ? __uint_as_float(r[4 * j + 2 + e]) * scale_log2 : -INFINITY;
              r[4 * j + e] = __float_as_uint(zA);
              r[4 * j + 2 + e] = __float_as_uint(zB);
              tA = fmaxf(tA, zA);
              tB = fmaxf(tB, zB);
            }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          tA = fmaxf(tA, __shfl_xor_sync(0xFFFFFFFFu, tA, o));
          tB = fmaxf(tB, __shfl_xor_sync(0xFFFFFFFFu, tB, o));
        }
        // The running maximum moves only when a row sees its first key (its O and l are still
        // zero) or when a tile exceeds it by more than 2^8: O is rescaled rarely, and weights
        // up to 2^8 lose nothing in f32 or bf16.
        const bool over = (mA != -INFINITY && tA > mA + kRescaleLog2) || (mB != -INFINITY && tB > mB + kRescaleLog2);
        const bool vote = __any_sync(0xFFFFFFFFu, over);
        if (c4 == 0) {
          s_max[64 * half + rA] = tA;
          s_max[64 * half + rB] = tB;
        }
        if (lane == 0) s_vote[warp - kSoftmaxWarp0] = vote ? 1u : 0u;
        ok = group_sync(52);
        if (!ok) break;
        tA = fmaxf(tA, s_max[64 * (half ^ 1) + rA]);
        tB = fmaxf(tB, s_max[64 * (half ^ 1) + rB]);
        uint32_t any = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) any |= s_vote[w];
        auto update = [](float& m, float& l, float t) {
          float a = 1.f;
          if (m == -INFINITY) {
            m = t;
          } else if (t > m + kRescaleLog2) {
            a = exp2f(m - t);
            m = t;
            l *= a;
          }
          return a;
        };
        const float aA = update(mA, lA, tA), aB = update(mB, lB, tB);
        if (any) {
          // O^T: a thread's lane is a value dim, its columns the rows; each half takes two of
          // the four blocks.  (S was issued behind the PV of the tile before, so that is done.)
          if (half == 0 && c4 == 0) {
            s_alpha[rA] = aA;
            s_alpha[rB] = aB;
          }
          ok = group_sync(53);
          if (!ok) break;
#pragma unroll 1
          for (int mb = 2 * half; mb < 2 * half + 2; ++mb)
#pragma unroll 1
            for (int c0 = 0; c0 < 64; c0 += 32) {
              uint32_t o[32];
              const uint32_t ta = tmem + lane_addr + kTmemO + 64 * mb + c0;
              tmem_ld32(ta, o);
              tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * s_alpha[c0 + c]);
              tmem_st32(ta, o);
            }
          tmem_st_wait();
        }
        const float muA = mA == -INFINITY ? 0.f : mA, muB = mB == -INFINITY ? 0.f : mB;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float pA0 = exp2f(__uint_as_float(r[4 * j]) - muA), pA1 = exp2f(__uint_as_float(r[4 * j + 1]) - muA);
          const float pB0 = exp2f(__uint_as_float(r[4 * j + 2]) - muB), pB1 = exp2f(__uint_as_float(r[4 * j + 3]) - muB);
          lA += pA0 + pA1;
          lB += pB0 + pB1;
          // 16-byte chunk j of row r sits at chunk j ^ (r % 8) (128-byte swizzle)
          *reinterpret_cast<uint32_t*>(prowA + ((j ^ (rA & 7)) << 4)) = pack_bf16x2(pA0, pA1);
          *reinterpret_cast<uint32_t*>(prowB + ((j ^ (rB & 7)) << 4)) = pack_bf16x2(pB0, pB1);
        }
        if (bad != 0 || kKeys * (k + 1) > s.limit) {
          // rows that are no cached rows may hold anything, NaN included: as values they are zero
          for (int x = st; x < kKeys * 64; x += kSoftmaxThreads) {  // (row, 16-byte chunk of 8 blocks)
            const int row = x >> 6, blk = (x >> 3) & 7, ch = x & 7;
            if (kKeys * k + row >= s.limit || ((bad >> (row >> 4)) & 1u))
              *reinterpret_cast<uint4*>(smem + kOffStage + blk * kBlockBytes + row * 128 + ch * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async();  // P (and the zeros) are visible to the tensor core
        tc_fence_before();
        mbar_arrive(pfull_bar);
      }
      if (!ok) break;
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        lA += __shfl_xor_sync(0xFFFFFFFFu, lA, o);
        lB += __shfl_xor_sync(0xFFFFFFFFu, lB, o);
      }
      if (c4 == 0) {
        s_l[64 * half + rA] = lA;
        s_l[64 * half + rB] = lB;
        if (half == 0) {
          s_m[rA] = mA;
          s_m[rB] = mB;
        }
      }
      ok = group_sync(54) && warp_wait(ofull_bar, i & 1, 55);
      if (!ok) break;
      tc_fence_after();
      if (st < s.nrows) {
        const float m = s_m[st], l = s_l[st] + s_l[64 + st];
        if (s.part >= 0)
          part_ml[(size_t)s.part * kRows + st] = make_float2(m, l);
        else if (lse)
          lse[(size_t)s.row0 + st] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
      }
#pragma unroll 1
      for (int mb = 2 * half; mb < 2 * half + 2; ++mb)
#pragma unroll 1
        for (int c0 = 0; c0 < 64; c0 += 32) {
          uint32_t o[32];
          tmem_ld32(tmem + lane_addr + kTmemO + 64 * mb + c0, o);
          tmem_ld_wait();
          const int d = 128 * mb + 32 * quarter + lane, rows = s.nrows - c0;
          if (s.part >= 0) {
            float* dst = parts + (size_t)s.part * kPartFloats + c0 * kDv + d;
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (c < rows) dst[c * kDv] = __uint_as_float(o[c]);
          } else {
            uint16_t* dst = out + ((size_t)s.row0 + c0) * kDv + d;
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (c < rows) {
                const float l = s_l[c0 + c] + s_l[64 + c0 + c];
                dst[(size_t)c * kDv] = (uint16_t)pack_bf16x2(l > 0.f ? __uint_as_float(o[c]) / l : 0.f, 0.f);
              }
          }
        }
      tc_fence_before();
      mbar_arrive(ofree_bar);
      ok = group_sync(56);  // s_l and s_m are free again
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the parts of the query tiles that cross a border between shares:
//   out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i,  M = max m_i.
// Block (x, g): rows 8x .. 8x + 7 (one a warp) of the tile that CTA g is the first to
// continue.  Its parts are CTA g - 1's last and the first of CTAs g, g + 1, ...
__global__ void __launch_bounds__(256) paged_combine_kernel(PagedBatch p, int H, int ctas, const Share* shares,
                                                            const float* parts, const float2* part_ml, uint16_t* out,
                                                            float* lse) {
  grid_dep_wait();
  const int g = blockIdx.y + 1;
  const Share s = load_share(shares + g);
  if (s.b < 0 || s.k0 == 0) return;
  const Share last = load_share(shares + g - 1);
  if (last.b == s.b && last.tile == s.tile && last.k0 > 0) return;  // an earlier block's tile
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = 8 * blockIdx.x + warp;
  const SequenceWork w = sequence_work(p, s.b, H);
  if (kRows * s.tile + row >= w.rows) return;
  int end = g + 1;  // CTAs g .. end - 1 continue the tile
  for (; end < ctas; ++end) {
    const Share t = load_share(shares + end);
    if (t.b != s.b || t.tile != s.tile || t.k0 == 0) break;
  }
  auto slot = [&](int i) { return i == g - 1 ? 2 * i + 1 : 2 * i; };
  float M = -INFINITY;
  for (int i = g - 1 + lane; i < end; i += 32) M = fmaxf(M, __ldcg(part_ml + (size_t)slot(i) * kRows + row).x);
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
  float den = 0.f;
  float4 acc[4];
  for (int j = 0; j < 4; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = g - 1; i < end; ++i) {
    const float2 ml = __ldcg(part_ml + (size_t)slot(i) * kRows + row);
    const float c = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
    den += c * ml.y;
    const float4* src = reinterpret_cast<const float4*>(parts + (size_t)slot(i) * kPartFloats + row * kDv) + lane;
    for (int j = 0; j < 4; ++j) {
      const float4 v = __ldcg(src + 32 * j);
      acc[j].x += c * v.x;
      acc[j].y += c * v.y;
      acc[j].z += c * v.z;
      acc[j].w += c * v.w;
    }
  }
  const float inv = den > 0.f ? 1.f / den : 0.f;
  const size_t unit = (size_t)p.cu_q[s.b] * H + kRows * s.tile + row;
  uint2* dst = reinterpret_cast<uint2*>(out + unit * kDv) + lane;
  for (int j = 0; j < 4; ++j)
    dst[32 * j] = make_uint2(pack_bf16x2(acc[j].x * inv, acc[j].y * inv), pack_bf16x2(acc[j].z * inv, acc[j].w * inv));
  if (lane == 0 && lse) lse[unit] = den > 0.f ? (M + log2f(den)) * 0.69314718055994531f : -INFINITY;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p) : nullptr;
  }();
  return fn;
}

// 2-D bf16 map over [rows][576] with a 64-column x box_rows box and 128-byte swizzle
bool make_map_576(CUtensorMap* map, const void* base, long long rows, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)kDqk, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)kDqk * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

SymbolAddress g_err_addr;

struct PagedLayout {
  size_t before, plan, shares, part_ml, parts, total;
};
size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }
PagedLayout paged_layout(int B, int ctas) {
  PagedLayout l;
  l.before = 0;
  l.plan = round256((size_t)B * sizeof(long long));
  l.shares = l.plan + 256;
  l.part_ml = l.shares + round256((size_t)ctas * sizeof(Share));
  l.parts = l.part_ml + round256((size_t)ctas * 2 * kRows * sizeof(float2));
  l.total = l.parts + (size_t)ctas * 2 * kPartFloats * sizeof(float);
  return l;
}

}  // namespace

size_t paged_attn_workspace_bytes(long long, int B, int) {
  const int sms = device_sm_count();
  return sms > 0 ? paged_layout(B, sms).total : 0;
}

cudaError_t launch_paged_attn(const uint16_t* q, const uint16_t* cache, const PagedBatch& p, int H, float scale,
                              uint16_t* out, float* lse, void* workspace, cudaStream_t stream) {
  const int ctas = device_sm_count();
  if (ctas <= 0) return cudaErrorInvalidDevice;
  static DeviceOnce once;
  cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(paged_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemP);
  });
  if (e != cudaSuccess) return e;
  int* err = nullptr;
  if ((e = g_err_addr.get(g_paged_error, &err)) != cudaSuccess) return e;
  int box = 16;  // rows of one copy: the largest power of two up to a tile that divides a page
  while (box < kKeys && p.page_size % (2 * box) == 0) box *= 2;
  CUtensorMap qmap, cmap;
  if (!make_map_576(&qmap, q, (long long)p.n * H, kRows) ||
      !make_map_576(&cmap, cache, (long long)p.num_pages * p.page_size, box))
    return cudaErrorInvalidValue;
  const PagedLayout l = paged_layout(p.B, ctas);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  Plan* plan = reinterpret_cast<Plan*>(ws + l.plan);
  Share* shares = reinterpret_cast<Share*>(ws + l.shares);
  float2* part_ml = reinterpret_cast<float2*>(ws + l.part_ml);
  float* parts = reinterpret_cast<float*>(ws + l.parts);
  paged_plan_kernel<<<1, 1024, 0, stream>>>(p, H, ctas, reinterpret_cast<long long*>(ws + l.before), plan, shares);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // waits in-kernel
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreadsP);
  cfg.dynamicSmemBytes = kSmemP;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, paged_attn_kernel, qmap, cmap, p, H, box, scale * 1.4426950408889634f,
                         static_cast<const Plan*>(plan), static_cast<const Share*>(shares), out, lse, parts, part_ml, err);
  if (e != cudaSuccess || ctas == 1) return e;
  cudaLaunchConfig_t ccfg = {};
  ccfg.gridDim = dim3(kRows / 8, ctas - 1);
  ccfg.blockDim = dim3(256);
  ccfg.stream = stream;
  ccfg.attrs = attr;
  ccfg.numAttrs = 1;
  return cudaLaunchKernelEx(&ccfg, paged_combine_kernel, p, H, ctas, static_cast<const Share*>(shares),
                            static_cast<const float*>(parts), static_cast<const float2*>(part_ml), out, lse);
}

cudaError_t paged_error_word(int** p) { return g_err_addr.get(g_paged_error, p); }

}  // namespace dsa
