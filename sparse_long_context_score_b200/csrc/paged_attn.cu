// paged_attn.cu -- MLA attention of a chunk of new tokens over a paged compressed cache.
//
//   out[t, h] = sum_s softmax_s(scale q[t, h] . c[s]) c[s][0:512],  s <= position of t,
// c[s] the 576-wide row of position s, in page table[b][s / page_size] at s % page_size.
// lse[t, h] = ln sum_s exp(scale q[t, h] . c[s]).
//
// A sequence's query rows (token, head) are one matrix [n_b H, 576], cut into tiles of 64
// rows whatever H is; a tile visits the 128-row key tiles that its last token sees.  The
// (query tile, key tile) pairs of the whole batch, in order, are dealt out in contiguous
// shares of equal work, one a CTA and one CTA an SM: a long context is split over CTAs when
// there are few query rows, and a CTA works through many query tiles when there are many.
// The lengths are read on the device, and every CTA finds its own share.  A query tile that one
// CTA covers is written directly; the parts of one that crosses a share's border go to the
// workspace in 32 bits, and paged_combine_kernel joins them in the CTAs' order (no atomics: the
// result does not depend on timing).
// Query tiles of one sequence meet its rows in L2 only where their CTAs read the same ones at
// about the same time, and the shares' borders shift from tile to tile.  So every CTA starts where
// its key tile's number is a multiple of the share's length, and takes the ones before that
// last: at any time the CTAs of a sequence are at the same few places (16 sequences of 2 to 8 new
// tokens x 64 heads over 4K to 32K: 1.29 -> 0.72 GB from HBM, 371 -> 351 us).  (Prefetching two
// key tiles ahead into L2 on top of that gained 3 to 6% in short bursts of such calls, and lost 2 to
// 4% of decode and of many sequences once the power limit is met.)
//
// One key tile of a CTA, everything in shared memory beside the 64 query rows (73.7 KB):
//   S^T = K Q^T     M = 128 keys, N = 64 rows, K = 576        (36 MMAs; TMEM lane = key)
//   O^T += V^T P^T  M = 4 x 128 value dims, N = 64 rows, K = 128 keys (32 MMAs)
// The tile (147.5 KB) fills the rest of shared memory as nine blocks of 64 columns, and
// there is no second one: S takes the blocks as they arrive, and each quarter of PV gives
// two of them back, so the next tile's loads run behind PV and the next S behind the loads.
// What bounds it: 512 query tokens x 64 heads x 2 over 16K take 5.37K cycles a key tile, 27.5
// bytes a cycle into each SM of the 29.5 that all SMs at once get out of L2 (S 1.73K and PV 1.54K
// cycles of MMAs, the softmax 1.32K).  8 tokens over 128K each: 7.0K cycles a key tile, HBM.
// Keys on the M side: an MMA of M = 128, N = 64, K = 16 takes 48 cycles (its operands'
// 6 KB at 128 bytes a cycle); with the rows there, M = 64, N = 128 takes 64.
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
constexpr int kMaxCtas = 256;                    // shares at most (one an SM)
constexpr int kSegs = 4;                         // query tile segments in flight

constexpr int kLoadWarp = 0, kMmaWarp = 1, kQueryWarp = 2, kWalkWarp = 3, kSoftmaxWarp0 = 4;
constexpr int kSoftmaxThreads = 256;             // eight warps: two per TMEM lane quarter
constexpr int kThreadsP = kSoftmaxWarp0 * 32 + kSoftmaxThreads;  // 384
constexpr float kRescaleLog2 = 8.f;
// Beginning a query tile costs a CTA as much as so many key tiles: the end of the one before
// (maxima, sums, 131 KB of values) and a first key tile that nothing runs ahead of take 10K cycles
// more than the 5.4K of a key tile.  Shares of equal key tiles: 16 verify chunks 360 us instead of
// 351, 8 x 128K 266 instead of 265 (a prefill chunk 2754 instead of 2757).
constexpr int kTileCost = 2;

// One CTA's part of a query tile.
struct Segment {
  int b;         // sequence; -1: no more
  int row0;      // first query row (token * H + head) in q
  int nrows;     // rows of the tile that exist
  int tile_row;  // the same row, counted from the sequence's first
  int k0, k1;    // key tiles, visited from `turn` on: k0 + turn .. k1 - 1, then k0 ..
  int turn;
  int seen0;     // cached rows that the sequence's first new token sees
  int limit;     // cached rows of the sequence
  int part;      // workspace slot of this part of the tile; -1: the tile is whole
};

// The i-th key tile that a segment visits.
__device__ __forceinline__ int tile_at(const Segment& s, int i) {
  const int k = s.k0 + s.turn + i;
  return k < s.k1 ? k : k - (s.k1 - s.k0);
}

// Query rows of a sequence and the cached rows that they see.
struct SequenceWork {
  int tiles, rows, row0, seen0, limit;
};
// A CTA's share: it starts `at` into query tile `tile` of sequence b (-1: nowhere).
struct Share {
  int b, tile, at, length;
  SequenceWork work;  // of that sequence
};
// A query tile that CTA g begins and later CTAs go on with, for the combine.
struct Join {
  int row0, nrows;  // as in Segment
  int parts;        // CTAs g .. g + parts - 1 hold one each; 0: none
  int pad;
};

constexpr int kOffQ = 0;
constexpr int kOffStage = kOffQ + kQBytes;
constexpr int kOffMax = kOffStage + kStageBytes;     // [4][64] f32: a tile's maxima, per quarter of the keys
constexpr int kOffAlpha = kOffMax + 4 * 64 * 4;      // [64] f32
constexpr int kOffL = kOffAlpha + 64 * 4;            // [4][64] f32: a segment's sums, likewise
constexpr int kOffM = kOffL + 4 * 64 * 4;            // [64] f32
constexpr int kOffVote = kOffM + 64 * 4;             // [2] u32: a half of the rows has one to rescale
constexpr int kOffOver = kOffVote + 16;              // u32: number of the last guessed tile that exceeded the maximum
constexpr int kOffBad = kOffOver + 16;               // u32: 16-row groups of the tile that are not there
constexpr int kOffShare = kOffBad + 16;
constexpr int kOffSum = kOffShare + 48;              // [12] i64: per warp
constexpr int kOffSeg = kOffSum + kThreadsP / 32 * 8;
constexpr int kOffBar = kOffSeg + kSegs * (int)sizeof(Segment) + 16;
constexpr int kNumBars = 10 + 2 * kSegs + 8;
constexpr int kOffTmem = kOffBar + kNumBars * 8;
constexpr int kSmemP = kOffTmem + 16 + 1024;         // + alignment slack
static_assert(kOffBar % 8 == 0, "barrier alignment");
static_assert(sizeof(Share) <= 48, "a share's place");
static_assert(kSmemP <= 232448, "shared memory budget");

constexpr int kTmemO = 0;      // O^T: 4 blocks x 64 columns, all 128 lanes
constexpr int kTmemS = 256;    // S^T: 64 columns, all 128 lanes
constexpr int kTmemCols = 512;

constexpr int kPartFloats = kRows * kDv;             // one part's [64][512] sums

constexpr float kRescaleFactor = 256.f;  // 2^kRescaleLog2
// The maximum that weights are taken from before a row has one: a logit of minus infinity weighs
// nothing (from -inf it would be NaN), any other one too much, so that a guess is taken back.  (What
// lies below it, -2.08e38 in base e, counts as minus infinity.)
constexpr float kNoMax = -3e38f;
// A weight is 2^(scale z - m), m the rounded scale z of the row's maximum, and one fused operation
// does not round scale z: what the two differ by, up to 2^-24 |m|, is common to the row and cancels,
// but from some 2^31 on it takes the largest weight itself out of range.  From this size of a tile's
// maximum on, every product is rounded on its own, as m was.
constexpr float kLargeMax = 65536.f;

// 2^x; results below the normal range become zero
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float min_nan(float x, float y) {  // NaN if x is
  float z;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}
// natural logarithm of 2^m sum; -inf for an empty sum
__device__ __forceinline__ float log_sum(float m, float sum) {
  return sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.69314718055994531f;
}
// eight bf16 values, NaN and infinity made zero
__device__ __forceinline__ uint4 finite_bf16(uint4 x) {
  auto two = [](uint32_t w) {
    if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
    return (w & 0x7F800000u) == 0x7F800000u ? w & 0xFFFFu : w;
  };
  return make_uint4(two(x.x), two(x.y), two(x.z), two(x.w));
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ SequenceWork sequence_work(const PagedBatch& p, int b, int H) {
  const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1];
  SequenceWork w;
  w.rows = q0 < 0 ? 0 : max(min(q1, p.n) - q0, 0) * H;
  w.row0 = q0 * H;
  w.tiles = (w.rows + kRows - 1) / kRows;
  // (below 2^31 by two key tiles, so that a tile's end stays an int)
  w.limit = (int)max(0LL, min(min((long long)p.ctx_len[b], 0x7FFFFF00LL), (long long)p.max_pages * p.page_size));
  w.seen0 = p.ctx_len[b] - (q1 - q0) + 1;
  return w;
}
// Key tiles that a query tile visits: those its last row sees, and at least one, so that
// rows which see nothing are written too.
__device__ __forceinline__ int tile_keys(const SequenceWork& w, int tile, int H) {
  const int last = min(kRows * (tile + 1), w.rows) - 1;
  const int seen = min(w.seen0 + last / H, w.limit);
  return max(1, (seen + kKeys - 1) / kKeys);
}
// Key tiles that the query tiles before `tile` visit, and what beginning them costs.  Tiles see ever more rows, so each key
// tile m is visited from one query tile on: the first whose last row, of token
// (64 (i + 1) - 1) / H, sees more than 128 m rows.
__device__ __forceinline__ long long work_before(const SequenceWork& w, int tile, int H) {
  if (tile <= 0) return 0;
  long long sum = (long long)kTileCost * tile;
  const int whole = min(tile, w.tiles - 1);  // all but the last tile have 64 rows
  if (whole > 0) {
    const int first = tile_keys(w, 0, H), last = tile_keys(w, whole - 1, H);
    sum += (long long)whole * first;
    for (int m = first; m < last; ++m) {
      const long long token = (long long)kKeys * m + 1 - w.seen0;  // the first that sees key tile m
      const long long i = max(0LL, (token * H + kRows) / kRows - 1);  // (64 (i + 1) - 1) / H >= token
      if (i < whole) sum += whole - i;
    }
  }
  return tile == w.tiles ? sum + tile_keys(w, w.tiles - 1, H) : sum;
}

__global__ void __launch_bounds__(kThreadsP, 1)
paged_attn_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap cmap,
                  const __grid_constant__ CUtensorMap rmap, PagedBatch p, int H, int box, float scale_log2, uint32_t negate, uint16_t* out, float* lse, Join* joins, float* parts, float2* part_ml, int* err) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sQ = sbase + kOffQ, sStage = sbase + kOffStage;
  float* s_max = reinterpret_cast<float*>(smem + kOffMax);
  float* s_alpha = reinterpret_cast<float*>(smem + kOffAlpha);
  float* s_l = reinterpret_cast<float*>(smem + kOffL);
  float* s_m = reinterpret_cast<float*>(smem + kOffM);
  volatile uint32_t* s_vote = reinterpret_cast<volatile uint32_t*>(smem + kOffVote);
  volatile uint32_t* s_over = reinterpret_cast<volatile uint32_t*>(smem + kOffOver);
  volatile uint32_t* s_bad = reinterpret_cast<volatile uint32_t*>(smem + kOffBad);
  Share* s_share = reinterpret_cast<Share*>(smem + kOffShare);
  Segment* s_seg = reinterpret_cast<Segment*>(smem + kOffSeg);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kOffTmem);
  const uint32_t bar0 = sbase + kOffBar;
  auto full_bar = [&](int i) { return bar0 + 8u * i; };                 // blocks 2i, 2i + 1 (i < 4), block 8 landed
  auto free_bar = [&](int i) { return bar0 + 8u * (5 + i); };           // ... are free
  auto segfull_bar = [&](int i) { return bar0 + 8u * (10 + i); };
  auto segfree_bar = [&](int i) { return bar0 + 8u * (10 + kSegs + i); };
  const uint32_t bars = bar0 + 8u * (10 + 2 * kSegs);
  const uint32_t qfull_bar = bars, qfree_bar = bars + 8, sfull_bar = bars + 16, pfull_bar = bars + 24;
  const uint32_t ofull_bar = bars + 32, ofree_bar = bars + 40, grp_bar = bars + 48, done_bar = bars + 56;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;
  grid_dep_launch();  // the combine may be scheduled; it waits on the device for this grid
  if (threadIdx.x == 0) {
    for (int i = 0; i < 5; ++i) {
      mbar_init(full_bar(i), 1);
      mbar_init(free_bar(i), 1);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(segfull_bar(i), 1);
      mbar_init(segfree_bar(i), 3 + kSoftmaxThreads / 32);  // load, MMA, query and softmax warps
    }
    mbar_init(qfull_bar, 1);
    mbar_init(qfree_bar, 1);
    mbar_init(sfull_bar, 1);
    mbar_init(pfull_bar, kSoftmaxThreads / 32);
    mbar_init(ofull_bar, 1);
    mbar_init(ofree_bar, kSoftmaxThreads / 32);
    mbar_init(grp_bar, kSoftmaxThreads / 32);
    mbar_init(done_bar, 1);
    *s_over = 0u;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(s_tmem), kTmemCols);
    tmem_relinquish();
  }
  // Where this CTA's share starts: every CTA sums the batch's work, a thread a sequence.
  // (A launch of its own for that, read by all CTAs, took 6 us more at 8 sequences.)
  {
    long long* s_sum = reinterpret_cast<long long*>(smem + kOffSum);
    long long total = 0, own = 0, before = 0;
    SequenceWork w{0, 0, 0, 0, 0};
    auto scan = [&](int b0) {  // work of sequence b0 + threadIdx.x, the sum before it, the sum of all 384
      const int b = b0 + threadIdx.x;
      own = 0;
      if (b < p.B) {
        w = sequence_work(p, b, H);
        own = work_before(w, w.tiles, H);
      }
      long long v = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += u;
      }
      __syncthreads();
      if (lane == 31) s_sum[warp] = v;
      __syncthreads();
      long long all = 0, mine = 0;
#pragma unroll
      for (int i = 0; i < kThreadsP / 32; ++i) {
        if (i == warp) mine = all;
        all += s_sum[i];
      }
      before = mine + v - own;
      return all;
    };
    for (int b0 = 0; b0 < p.B; b0 += kThreadsP) total += scan(b0);
    const long long per = max(1LL, (total + gridDim.x - 1) / gridDim.x), start = per * cta;
    if (threadIdx.x == 0) s_share->b = -1;
    long long base = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreadsP) {
      long long all = total;
      if (p.B > kThreadsP) all = scan(b0);
      else __syncthreads();
      const long long at = start - base - before;
      if (at >= 0 && at < own) {
        int lo = 0, hi = w.tiles - 1;  // the last tile that starts at or before it
        while (lo < hi) {
          const int mid = (lo + hi + 1) / 2;
          if (work_before(w, mid, H) <= at) lo = mid;
          else hi = mid - 1;
        }
        *s_share = Share{b0 + (int)threadIdx.x, lo, (int)(at - work_before(w, lo, H)), (int)min(per, 0x7FFFFFFFLL), w};
      }
      base += all;
    }
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
      tma_prefetch(&rmap);
      const Share first = *s_share;
      int b = first.b, tile = first.tile, k0 = max(0, first.at - kTileCost);
      int left = first.length - max(0, kTileCost - first.at);
      Join join{0, 0, 0, 0};
      SequenceWork w = first.work;
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
          s.row0 = w.row0 + s.tile_row;
          s.nrows = min(kRows, w.rows - s.tile_row);
          s.k0 = k0;
          s.k1 = min(keys, k0 + left);
          s.seen0 = w.seen0;
          s.limit = w.limit;
          s.part = k0 > 0 ? 2 * cta : s.k1 < keys ? 2 * cta + 1 : -1;
          if (k0 == 0 && s.k1 < keys) join = Join{s.row0, s.nrows, 1 + (keys - s.k1 + first.length - 1) / first.length, 0};
          const int next_phase = (k0 + first.length - 1) / first.length * first.length;  // a multiple of the share
          s.turn = next_phase < s.k1 ? next_phase - k0 : 0;
          left -= s.k1 - k0 + kTileCost;
          k0 = 0;
          ++tile;
        }
        if (!mbar_wait(segfree_bar(at), ((i / kSegs) & 1) ^ 1, err, 42)) break;
        s_seg[at] = s;
        mbar_arrive(segfull_bar(at));
        if (s.b < 0) break;
      }
      joins[cta] = join;
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
        tma_load_3d(sQ, &qmap, qfull_bar, 0, s.row0, 0);
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
    int it = 0;
    bool ok = true;
    while (ok && next_segment(s)) {
      const int32_t* table = p.table + (size_t)s.b * p.max_pages;
      const int count = s.k1 - s.k0;
      auto page_row = [&](int n) {  // pool row of this lane's box in the n-th key tile, -1 where there is none
        if (lane >= boxes || n >= count) return -1;
        const long long pos = (long long)kKeys * tile_at(s, n) + box * lane;
        if (pos >= s.limit) return -1;
        const long long i = pos / p.page_size;
        if (i >= p.max_pages) return -1;
        const int page = table[i];
        return page >= 0 && page < p.num_pages ? page * p.page_size + (int)(pos - i * p.page_size) : -1;
      };
      int row = page_row(0), next = page_row(1);
      for (int n = 0; n < count; ++n, ++it) {
        const int ahead = page_row(n + 2);
        const uint32_t there = __ballot_sync(0xFFFFFFFFu, row >= 0);
        uint32_t bad = 0;  // per 16 rows
        for (int i = 0; i < kKeys / 16; ++i) bad |= ((there >> (i * 16 / box)) & 1u ? 0u : 1u) << i;
        const int y = row >= 0 ? row : p.num_pages * p.page_size;  // behind the pool: zeros
#pragma unroll
        for (int i = 0; i < 5; ++i) {  // blocks 2i, 2i + 1; the rotary block alone
          ok &= mbar_wait(free_bar(i), (it & 1) ^ 1, err, 44);
          if (i == 0) {  // the tile before is read up to its last block by then
            if (lane == 0) *s_bad = bad;
            if (lane < 5) mbar_arrive_expect_tx(full_bar(lane), lane < 4 ? 2 * kBlockBytes : kBlockBytes);
            __syncwarp();
          }
          const uint32_t dst = sStage + 2 * i * kBlockBytes + lane * box * 128;
          if (i == 4) {
            if (lane < boxes) tma_load_3d(dst, &rmap, full_bar(4), 0, y, 8);
          } else if (box == kKeys) {
            if (lane == 0) tma_load_3d(dst, &cmap, full_bar(i), 0, y, 2 * i);
          } else if (lane < boxes) {
            // (a box of two blocks would put the second one right behind the box's rows)
            tma_load_3d(dst, &rmap, full_bar(i), 0, y, 2 * i);
            tma_load_3d(dst + kBlockBytes, &rmap, full_bar(i), 0, y, 2 * i + 1);
          }
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        row = next;
        next = ahead;
      }
    }
    // nothing in flight on the way out: every block that was asked for has landed
    if (lane == 0 && it + !ok > 0)
      for (int i = 0; i < 5; ++i) mbar_wait_drain(full_bar(i), (it + !ok - 1) & 1);
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------ tensor core
    const bool leader = elect_one();
    // K (K-major) x Q (K-major); a negative scale negates K, so that the largest S is the
    // largest logit
    const uint32_t idS = idesc_bf16_f32(kKeys, kRows) | negate;
    constexpr uint32_t idPV = idesc_bf16_f32(128, kRows, true, true);  // V^T (M-major) x P (N-major)
    const uint64_t dq = sdesc_kmajor_sw128(sQ), dk = sdesc_kmajor_sw128(sStage);
    const uint64_t dv = sdesc_mnmajor_sw128(sStage, kBlockBytes, 1024);
    const uint64_t dp = sdesc_mnmajor_sw128(sStage + kPBlock * kBlockBytes, 1024, 1024);
    Segment s;
    int it = 0;
    uint32_t pp = 0;  // phases of pfull seen
    bool ok = true;
    for (int i = 0; ok && next_segment(s); ++i) {
      ok = warp_wait(qfull_bar, i & 1, 45);
      const int count = s.k1 - s.k0;
      for (int n = 0; ok && n < count; ++n, ++it) {
        // (unrolled, so that descriptors are a base and a constant: an issue loop that adds
        // them up at run time is slower than the tensor core)
#pragma unroll
        for (int kb = 0; kb < kBlocks; ++kb) {
          if (kb % 2 == 0) ok &= mbar_wait(full_bar(kb / 2), it & 1, err, 46);
          if (kb == 0) tc_fence_after();
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16(tmem + kTmemS, dk + (uint64_t)((kb * kBlockBytes + kk * 32) >> 4),
                       dq + (uint64_t)((kb * kQBlockBytes + kk * 32) >> 4), idS, kb + kk > 0);
          }
          __syncwarp();
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        if (leader) {
          mma_commit(sfull_bar);
          if (n + 1 == count) mma_commit(qfree_bar);
        }
        __syncwarp();
        // the epilogue of the segment before has read O
        if (n == 0) ok = warp_wait(ofree_bar, (i & 1) ^ 1, 47);
        ok = ok && warp_wait(pfull_bar, pp++ & 1, 48);
        if (!ok) break;
        if (n > 0 && n + 1 < count && *s_over == (uint32_t)it + 1u) {  // a wrong guess: the tile's weights again
          __syncwarp();
          if (lane == 0) mbar_arrive(sfull_bar);
          ok = warp_wait(pfull_bar, pp++ & 1, 57);
          if (!ok) break;
        }
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int mb = 0; mb < 4; ++mb) {
#pragma unroll
            for (int ks = 0; ks < kKeys / 16; ++ks)
              mma_bf16(tmem + kTmemO + 64 * mb, dv + (uint64_t)((2 * mb * kBlockBytes + ks * 16 * 128) >> 4),
                       dp + (uint64_t)(ks * 16 * 128 >> 4), idPV,
                       n > 0 || ks > 0 ? 1u : 0u);
            mma_commit(free_bar(mb));
          }
          mma_commit(free_bar(4));
          if (n + 1 == count) mma_commit(ofull_bar);
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
    // Warp w reads TMEM lane quarter w % 4, i.e. keys 32 quarter .. 32 quarter + 31 of a tile,
    // a lane a key, and 32 of the 64 rows.  A row's running maximum is the same in all of its
    // threads, and each keeps its own key's share of the row's sum to the end of a segment:
    // no tile needs a reduction over keys.
    const int quarter = warp & 3, half = (warp - kSoftmaxWarp0) >> 2;
    const uint32_t lane_addr = (uint32_t)(32 * quarter) << 16;
    const int st = threadIdx.x - 32 * kSoftmaxWarp0;  // 0 .. 255
    // P: a row of 128 bytes a key, 64 query rows; 16-byte chunk c of key x at chunk c ^ (x % 8)
    const uint32_t prow = sStage + kPBlock * kBlockBytes + (32 * quarter + lane) * 128;
    uint32_t grp_phase = 0;
    auto group_sync = [&](int code) {
      __syncwarp();
      if (lane == 0) mbar_arrive(grp_bar);
      const bool ok = warp_wait(grp_bar, grp_phase, code);
      grp_phase ^= 1;
      return ok;
    };
    Segment s;
    uint32_t sp = 0;     // phases of sfull seen
    uint32_t tiles = 0;  // key tiles weighted, this CTA's first being number 1
    bool ok = true;
    for (int i = 0; ok && next_segment(s); ++i) {
      // cached rows that all of the tile's query rows see, and those that some do
      const int seen_first = min(s.seen0 + s.tile_row / H, s.limit);
      const int seen_last = min(s.seen0 + (s.tile_row + s.nrows - 1) / H, s.limit);
      float m[32], l[32];
      float mrow = 32 * half + lane < s.nrows ? -INFINITY : INFINITY;  // row 32 half + lane's maximum
#pragma unroll
      for (int r = 0; r < 32; ++r) {
        l[r] = 0.f;
      }
      bool guessed = false, large = false;
      const int count = s.k1 - s.k0;
      for (int next = 0; next < count;) {
        ok = warp_wait(sfull_bar, sp & 1, 51);
        if (!ok) break;
        ++sp;
        tc_fence_after();
        // Tiles in the middle of a segment are weighted with the running maximum as it
        // stands; where one turns out to exceed it by more than 2^8 the MMA warp asks for the
        // tile again (S is still there), which then goes through the exchange of maxima as a
        // segment's first and last tiles do.
        const bool redo = guessed && *s_over == tiles;
        const int n = redo ? next - 1 : next, k = tile_at(s, n);
        const bool exchange = redo || n == 0 || n + 1 == count || large;
        if (!redo) ++tiles;
        const uint32_t bad = *s_bad;
        uint32_t z[32];
        tmem_ld32(tmem + lane_addr + kTmemS + 32 * half, z);
        // rows from `from` on (of this warp's 32) see this thread's key
        const int key = kKeys * k + 32 * quarter + lane;
        const bool whole = bad == 0 && kKeys * (k + 1) <= seen_first;
        int from = 0;
        if (!whole) {
          const bool there = key < s.limit && !((bad >> (2 * quarter + (lane >> 4))) & 1u);
          const long long first = (long long)(key + 1 - s.seen0) * H - s.tile_row - 32 * half;
          from = there ? (int)max(0LL, min(32LL, first)) : 32;
        }
        tmem_ld_wait();
        // this thread's key for row r
        auto weight = [&](int r) {
          const float p = min_nan(exp2_approx(fmaf(__uint_as_float(z[r]), scale_log2, -m[r])), 2.f * kRescaleFactor);
          return !whole && r < from ? 0.f : p;  // (a masked key weighs nothing whatever its logit and the scale)
        };
        // A guess is taken back by subtracting what it added: that costs the row's sum one
        // rounding, since weights are capped (above the cap the guess is wrong anyway).
        if (redo) {
#pragma unroll
          for (int r = 0; r < 32; ++r) l[r] -= weight(r);
        }
        // The running maximum moves only when a row sees its first key or when a tile exceeds
        // it by more than 2^8: O is rescaled rarely, and weights up to 2^8 lose nothing in f32
        // or bf16.
        if (exchange) {
          float mine = -INFINITY;  // of row 32 half + lane over the warp's keys
#pragma unroll
          for (int r = 0; r < 32; ++r) {
            const float t = warp_max(r >= from ? __fmul_rn(__uint_as_float(z[r]), scale_log2) : -INFINITY);
            if (lane == r) mine = t;
          }
          s_max[64 * quarter + 32 * half + lane] = mine;
          ok = group_sync(52);
          if (!ok) break;
          float t = -INFINITY, other = -INFINITY;  // of the other half's rows, so that all warps agree on `large`
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            t = fmaxf(t, s_max[64 * q + 32 * half + lane]);
            other = fmaxf(other, s_max[64 * q + 32 * (half ^ 1) + lane]);
          }
          auto far = [](float x) { return fabsf(x) > kLargeMax && fabsf(x) < INFINITY; };
          large = large || __any_sync(0xFFFFFFFFu, far(t) || far(other));
          float alpha = 1.f;
          if (mrow == -INFINITY) {
            mrow = t;
          } else if (t > mrow + kRescaleLog2) {
            alpha = exp2_approx(mrow - t);
            mrow = t;
          }
          const bool scaled = __any_sync(0xFFFFFFFFu, alpha != 1.f);
#pragma unroll
          for (int r = 0; r < 32; ++r) {
            m[r] = fmaxf(__shfl_sync(0xFFFFFFFFu, mrow, r), kNoMax);
          }
          if (scaled) {
#pragma unroll
            for (int r = 0; r < 32; ++r) l[r] *= __shfl_sync(0xFFFFFFFFu, alpha, r);
          }
          if (large) {  // `weight` takes what is left of each exponent (all tiles of the segment come here from now on)
            const float back = 1.f / scale_log2;
#pragma unroll
            for (int r = 0; r < 32; ++r) {
              z[r] = __float_as_uint((__fmul_rn(__uint_as_float(z[r]), scale_log2) - m[r]) * back);
              m[r] = 0.f;
            }
          }
          if (n > 0) {
            if (quarter == 0) {
              s_alpha[32 * half + lane] = alpha;
              if (lane == 0) s_vote[half] = scaled ? 1u : 0u;
            }
            ok = group_sync(53);
            if (!ok) break;
            if (s_vote[0] | s_vote[1]) {
              // O^T: a thread's lane is a value dim, its columns the rows; each half takes two
              // of the four blocks.  (S was issued behind the PV of the tile before, which is
              // done.)
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
          }
        }
        float most = 0.f;
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += 8) {
          float p[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            p[j] = weight(r0 + j);
            l[r0 + j] += p[j];
            most = fmaxf(most, p[j]);
          }
          st_shared_v4(prow + (((4 * half + r0 / 8) ^ (lane & 7)) << 4), pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]),
                       pack_bf16x2(p[4], p[5]), pack_bf16x2(p[6], p[7]));
        }
        // One vote for what is rare: a weight above the cap, and a key whose values may be NaN or
        // infinite (no product with such a value is finite, so that any one row's logit tells).
        const bool odd = !(fabsf(__uint_as_float(z[0])) < INFINITY);
        if (__any_sync(0xFFFFFFFFu, most > kRescaleFactor || odd)) {
          if (!exchange && __any_sync(0xFFFFFFFFu, most > kRescaleFactor) && lane == 0) *s_over = tiles;
          // A weight of zero does not silence such a value.  A row that all query rows of the tile see
          // has a weight of zero where its logit is -inf (NaN and +inf make the weight NaN, which stays
          // so whatever the values are): its values that are not finite become zero.
          for (uint32_t todo = __ballot_sync(0xFFFFFFFFu, odd && key < seen_first && half == 0); todo; todo &= todo - 1) {
            const int row = 32 * quarter + __ffs(todo) - 1;
            for (int c = lane; c < kDv / 8; c += 32) {
              uint4* at = reinterpret_cast<uint4*>(smem + kOffStage + (c >> 3) * kBlockBytes + (c & 7) * 16 + row * 128);
              *at = finite_bf16(*at);
            }
          }
        }
        if (!whole) {
          // Rows that no query row of the tile sees may hold anything: as values they are zero.  Of a
          // row that some see, only such entries become zero: S has them, so where the row is seen
          // they count.  (Boxes without a page or behind the context were loaded as zeros.)
          const int past = s.limit - kKeys * k, end = min(kKeys, (past + box - 1) & -box);
          const int chunk = (st >> 3 & 7) * kBlockBytes + (st & 7) * 16;  // a thread's 16 bytes of a row
#pragma unroll 4
          for (int row = max(0, seen_first - kKeys * k) + (st >> 6); row < end; row += kSoftmaxThreads / 64) {
            uint4* at = reinterpret_cast<uint4*>(smem + kOffStage + chunk + row * 128);
            *at = kKeys * k + row >= seen_last ? make_uint4(0, 0, 0, 0) : finite_bf16(*at);
          }
        }
        fence_proxy_async();  // P (and the zeros) are visible to the tensor core
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull_bar);
        guessed = !exchange;
        next = n + 1;
      }
      if (!ok) break;
      // sums over the warp's keys, row 32 half + lane to each lane: at step o the rows whose
      // index has bit o go to the lanes that have it
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int r = 0; r < o; ++r) {
          const float keep = lane & o ? l[r + o] : l[r], give = lane & o ? l[r] : l[r + o];
          l[r] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
        }
      s_l[64 * quarter + 32 * half + lane] = l[0];
      if (quarter == 0) s_m[32 * half + lane] = mrow;
      ok = group_sync(54) && warp_wait(ofull_bar, i & 1, 55);
      if (!ok) break;
      tc_fence_after();
      if (st < 64) {
        const float sum = (s_l[st] + s_l[64 + st]) + (s_l[128 + st] + s_l[192 + st]);
        if (st < s.nrows) {
          if (s.part >= 0)
            part_ml[(size_t)s.part * kRows + st] = make_float2(s_m[st], sum);
          else if (lse)
            lse[(size_t)s.row0 + st] = log_sum(s_m[st], sum);
        }
        s_alpha[st] = sum == 0.f ? 0.f : 1.f / sum;
      }
      ok = group_sync(57);
      if (!ok) break;
#pragma unroll 1
      for (int mb = 2 * half; mb < 2 * half + 2; ++mb)
#pragma unroll 1
        for (int c0 = 0; c0 < s.nrows; c0 += 32) {
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
              if (c < rows) dst[(size_t)c * kDv] = (uint16_t)pack_bf16x2(__uint_as_float(o[c]) * s_alpha[c0 + c], 0.f);
          }
        }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ofree_bar);
      ok = group_sync(56);  // s_l, s_m and s_alpha are free again
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the parts of a query tile that crosses borders between shares:
//   out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i,  M = max m_i.
// The parts are CTA g's last and the first of the CTAs behind it.  Four warps take a row, 128
// value dims each, with eight parts' loads in flight beside those of their (m, l); the (tile,
// row) pairs of all joins are spread over the whole grid, since a few long contexts leave few
// tiles of many parts, and many short ones the other way round.  (16 verify chunks: some 220
// parts, 29 MB; 14 us with cold caches.)
constexpr int kJoinThreads = 256, kJoinRows = kJoinThreads / 128, kJoinBlocks = 3;  // blocks per SM
__global__ void __launch_bounds__(kJoinThreads, kJoinBlocks)
paged_combine_kernel(int ctas, const Join* joins, const float* parts, const float2* part_ml, uint16_t* out, float* lse) {
  __shared__ int s_warp[kJoinThreads / 32];
  __shared__ int4 s_join[kMaxCtas];  // CTAs that leave a tile to the next ones: (row0, nrows, parts, g)
  static_assert(kMaxCtas <= kJoinThreads, "a thread a CTA");
  grid_dep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int4 jv = make_int4(0, 0, 0, 0);
  if ((int)threadIdx.x < ctas) jv = __ldcg(reinterpret_cast<const int4*>(joins + threadIdx.x));
  const uint32_t votes = __ballot_sync(0xFFFFFFFFu, jv.z > 0);
  if (lane == 0) s_warp[warp] = __popc(votes);
  __syncthreads();
  int count = 0, place = __popc(votes & ((1u << lane) - 1));
  for (int i = 0; i < kJoinThreads / 32; ++i) {
    place += i < warp ? s_warp[i] : 0;
    count += s_warp[i];
  }
  if (jv.z > 0) s_join[place] = make_int4(jv.x, jv.y, jv.z, threadIdx.x);
  __syncthreads();
  const int d = 128 * (warp & 3) + 4 * lane;
  for (int unit = kJoinRows * blockIdx.x + warp / 4; unit < count * kRows; unit += kJoinRows * gridDim.x) {
    const int4 join = s_join[unit / kRows];
    const int row = unit % kRows, n = join.z;
    if (row >= join.y) continue;
    auto slot = [&](int i) { return (size_t)(i == 0 ? 2 * join.w + 1 : 2 * (join.w + i)); };
    float M = -INFINITY, den = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int m = min(32, n - i0);
      float2 ml = make_float2(-INFINITY, 0.f);  // lane i holds part i0 + i's
      if (lane < m) ml = __ldcg(part_ml + slot(i0 + lane) * kRows + row);
      float c = 0.f;
      for (int i = 0; i < m; i += 8) {
        float4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (i + j < m) v[j] = __ldcg(reinterpret_cast<const float4*>(parts + slot(i0 + i + j) * kPartFloats + row * kDv + d));
        if (i == 0) {  // the maximum so far, and the factors of these 32
          float t = ml.x;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, o));
          const float big = fmaxf(M, t), old = M == -INFINITY ? 0.f : exp2_approx(M - big);
          M = big;
          c = ml.y == 0.f ? 0.f : ml.x == -INFINITY ? ml.y : exp2_approx(ml.x - M);  // (a NaN sum stays one)
          den = den * old + c * ml.y;
          acc = make_float4(acc.x * old, acc.y * old, acc.z * old, acc.w * old);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float cj = __shfl_sync(0xFFFFFFFFu, c, (i + j) & 31);
          if (i + j < m) {
            acc.x += cj * v[j].x;
            acc.y += cj * v[j].y;
            acc.z += cj * v[j].z;
            acc.w += cj * v[j].w;
          }
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xFFFFFFFFu, den, o);
    const float inv = den == 0.f ? 0.f : 1.f / den;
    const size_t at = (size_t)join.x + row;
    *reinterpret_cast<uint2*>(out + at * kDv + d) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if ((warp & 3) == 0 && lane == 0 && lse) lse[at] = log_sum(M, den);
  }
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

// bf16 map over [rows][576] as [blocks of 64 columns][rows][64]: a box of box_rows rows and
// box_blocks column blocks lands block after block, with the 128-byte swizzle
bool make_map_576(CUtensorMap* map, const void* base, long long rows, int box_rows, int box_blocks) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)kBlocks};
  cuuint64_t strides[2] = {(cuuint64_t)kDqk * 2, 128};
  cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_blocks};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

SymbolAddress g_err_addr;

struct PagedLayout {
  size_t joins, part_ml, parts, total;
};
PagedLayout paged_layout(int ctas) {
  auto round256 = [](size_t b) { return (b + 255) & ~(size_t)255; };
  PagedLayout l;
  l.joins = 0;
  l.part_ml = round256((size_t)ctas * sizeof(Join));
  l.parts = l.part_ml + round256((size_t)ctas * 2 * kRows * sizeof(float2));
  l.total = l.parts + (size_t)ctas * 2 * kPartFloats * sizeof(float);
  return l;
}

}  // namespace

size_t paged_attn_workspace_bytes() {
  const int ctas = min(device_sm_count(), kMaxCtas);
  return ctas > 0 ? paged_layout(ctas).total : 0;
}

cudaError_t launch_paged_attn(const uint16_t* q, const uint16_t* cache, const PagedBatch& p, int H, float scale,
                              uint16_t* out, float* lse, void* workspace, cudaStream_t stream) {
  const int ctas = min(device_sm_count(), kMaxCtas);
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
  CUtensorMap qmap, cmap, rmap;
  const long long pool = (long long)p.num_pages * p.page_size;
  if (!make_map_576(&qmap, q, (long long)p.n * H, kRows, kBlocks) || !make_map_576(&rmap, cache, pool, box, 1))
    return cudaErrorInvalidValue;
  cmap = rmap;  // (only whole tiles are copied two blocks at a time)
  if (box == kKeys && !make_map_576(&cmap, cache, pool, box, 2)) return cudaErrorInvalidValue;
  const PagedLayout l = paged_layout(ctas);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  Join* joins = reinterpret_cast<Join*>(ws + l.joins);
  float2* part_ml = reinterpret_cast<float2*>(ws + l.part_ml);
  float* parts = reinterpret_cast<float*>(ws + l.parts);
  paged_attn_kernel<<<ctas, kThreadsP, kSmemP, stream>>>(qmap, cmap, rmap, p, H, box, fabsf(scale) * 1.4426950408889634f,
                                                         scale < 0.f ? 1u << 13 : 0u, out, lse, joins, parts, part_ml, err);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // waits in-kernel
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kJoinBlocks * ctas);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_combine_kernel, ctas, static_cast<const Join*>(joins),
                            static_cast<const float*>(parts), static_cast<const float2*>(part_ml), out, lse);
}

cudaError_t paged_error_word(int** p) { return g_err_addr.get(g_paged_error, p); }

}  // namespace dsa
