// Attention of many query rows over the paged 4-bit history: tcgen05 tiles.
//
// The arithmetic of the kernel of few rows (history_attn.cu) with 128 rows,
// (token, query head) pairs of one key head, against tiles of two pages (128
// keys), but with the scales inside the products, so that the softmax has
// nothing to do for them:
//   K  s (c - 8) over a power of two of the tile: a significand of 8 bits times
//      a number of -8 ... 7 has 11 bits, so it is exact in fp16 (but for what lies
//      2^-25 below the tile's largest key).  What is left, h sum(q), is one more
//      step of the product: h and sum(q) are split into three fp16 parts each, and
//      six of the 16 columns of that step hold the pairs that matter (the rest is
//      below 2^-32 of it).
//   V  s' (c' - 8) + h' in fp16 (2^-11, eight times finer than the bf16 it was
//      made from) over a power of two that no value of the item so far exceeds.
//      Where a causal item's last tiles hold values that some rows do not see and
//      that are far from the others, V and P are bf16 from there on, over a power of
//      two that leaves room for every bf16 value: rounded to 2^-8 each, but no row's
//      values depend on another's keys.
// P is fp16.
//
// One block of threads an SM takes two row tiles (256 rows) against the same
// keys, so that a page is unpacked once for both.  Six warps unpack the codes
// and write the two operands in the 128-byte swizzled form of the descriptors,
// K and V apart and both twice buffered: a V buffer is in use from one row
// tile's product to the other's, half a step later, so that a single one leaves
// no time to write it (with it, and with the codes staged in shared memory by
// bulk copies, the call below took 2.06 ms).  The codes are
// read 16 bytes at a time into the registers that the tile before just left.
// Channels keep the unpacked order (0 4 1 5 2 6 3 7 of each 8), and of the
// second 64 the groups of 16 are exchanged in pairs of groups, which spreads the
// 16-byte writes of 8 threads over all banks; Q is written in the same order, O
// put back at the end.
//   warps 0-3, 4-7  softmax of row tile 0 and 1, a thread a row; they also write
//                   Q and store O
//   warp  8         TMEM owner, MMA issuer (one thread): while one tile is
//                   exponentiated, the other's products run
//   warp  9         writes the tiles' records
//   warps 10-12     K producers
//   warps 13-15     V producers
// TMEM: S0 [0, 128), S1 [128, 256), O0 [256, 384), O1 [384, 512); the fp16 P
// overwrites the first 64 columns of its S.  Each block takes an equal share of
// the line of work.
//
// 3600 queries over 25200 tokens, 24 heads of 96: 1.21 ms, 690 TFLOP/s (42% of the
// measured bf16 rate); the tensor pipe is busy 36% of the time, the exponentials'
// unit 45%, the issue slots 46%.  4000 causal queries over their own tokens, 40 query
// and 8 key heads of 128: 0.70 ms (tiles that no row of an item sees are computed like
// the others, half of all here).  The step of a row tile is a chain, Q K^T (1/5 of
// it), softmax (3/5) and P V (1/5), of which the two row tiles hide only each
// other's products.  Scores in halves of 64 keys, so that one half's product runs
// under the other's softmax, took away most of the wait for S but make Q K^T twice
// as dear (64 columns do not fill the tensor pipe) and crowd the exponentials:
// 1.32 ms.

#include <cuda_fp16.h>

#include "history_attn.cuh"

namespace ditango {
namespace hchunk {

using hattn::Params;

constexpr int BM = 128;              // rows of a tile
constexpr int TR = 2 * BM;           // rows of an item
constexpr int BN = 2 * kPage;        // keys of a tile
constexpr int kThreads = 512;
constexpr int kLaunchRegs = 128;     // 65536 / 512
// of the splits that were tried at 3600 queries of 24 heads of 96 channels after 25200
// tokens, 1.19 ms with this one then: 176/80 1.30 ms, where the producers spill, 160/96 1.37
constexpr int kSoftmaxRegs = 168, kControlRegs = 88;
static_assert(2 * 128 * kSoftmaxRegs + 2 * 128 * kControlRegs == kThreads * kLaunchRegs, "register split");
constexpr int kProducers = 96;       // threads that unpack K, and as many for V
constexpr int kTmemCols = 512;
constexpr int kMaxBlocks = 160;      // most blocks of a launch (the workspace has room for them)
// A block's share is at least this many tiles: below, joining the parts of an
// item costs more than the shorter share saves.
constexpr int kMinUnits = 4;
constexpr int kSetup = 2;            // tiles that beginning and finishing an item counts for

// P in fp16: a row exponentiates against its maximum less 7, so that p is 2^7
// where it was 1, and 2^15 where a maximum grew by the 2^8 that it may before
// the row is rescaled (fp16 ends at 65504).  Smaller ones are then kept to 2^-32
// of the largest, half a step of fp16's least numbers: 300000 keys of 2^-27 each
// beside one of 1 are a thousandth of the sum, and were lost whole with p at 1.
// Sums, maximum and lse go by the same shift.  Past kHuge neither the shift nor the
// growth is small against the rounding of the maximum, and both are left out.
constexpr float kSpareLog2 = 7.0f;
__device__ __forceinline__ float reference_of(float mx) { return fabsf(mx) > kHuge ? mx : mx - kSpareLog2; }
__device__ __forceinline__ bool outgrown(float mx, float m) {
  return mx > (fabsf(m) > kHuge ? m : m + (kSpareLog2 + kRescaleLog2));
}

// A causal item's last tiles hold keys that not all of its rows see, and those may
// be of any size beside the others.  (Keys that a row sees need no such care: what
// the largest takes from the others is below the rounding of its own score, and
// 2^-25 of the largest value.)  A call that is causal is launched twice: kAsIs looks,
// before it begins, whether any of these keys are 2^6, or their values 2^10, from
// one another, and kFarApart, which does nothing else, does the work once more where
// they are; with lists, where a row may see none of its neighbours, it does the work
// alone.  Tests for it in the loops of one kernel cost them 3% (K) to 25% (K and V):
// their registers are full.  The look costs 1%, the empty launch 3 us.
enum Sizes { kAsIs, kFarApart };

// What is known of a tile before its codes are unpacked.
//
// kFarApart: where the sizes of the keys of a tile that not all rows see differ by
// more than 2^4, K is held key by key: each over a power of two of its own, which
// the softmax puts back into the scores.  Where the values differ by more than 2^10,
// from one another or from those before, this tile and those after it hold V in
// bf16, and the softmax P.
constexpr int kRing = 4;
constexpr uint32_t kEven = 4, kEvenV = 10;
constexpr uint32_t kOwnK = 1, kWideV = 2;
// V and O in bf16's range: values of 2^128 give sums of 2^(15 + 128 - 40) a key,
// and those below 2^-86 are lost.
constexpr uint32_t kWideRef = (127u + 40u) << 23;
constexpr float kWideDown = 0x1p-40f;
struct alignas(16) Tile {
  uint2 v[BN];                  // V's s and h over vref, as fp16 pairs
  uint32_t ks[BN];              // K's s over kref, as an fp16 pair
  float kh[BN];                 // K's h over kref
  float2 vw[BN];                // kWideV: V's s and h over vref, and v is (1, 0)
  float kf[BN];                 // kOwnK: the keys' own powers of two, over kref
  float kref, vref;             // the powers of two over which K and V are held
  uint32_t flags;               // kOwnK, kWideV
  int pos[2];                   // first token of each page, past every length where there is none
  uint32_t bad[4];              // keys whose V is not finite (written as 0: the softmax marks who sees it)
};

// Tiles of a segment with keys that some rows of a causal item see and others do
// not: [first, last).  (Lists hold blocks in any order.)
struct Edge {
  int first, last;
  __device__ __forceinline__ Edge(const Params &p, const hattn::Segment &sg) {
    const int row0 = sg.tile * TR, row1 = (int)min((long long)row0 + TR, (long long)sg.rq.n_q * p.G) - 1;
    const int seen = sg.rq.kv - (sg.rq.n_q - 1);       // of the request's first token, which sees this many
    first = p.sel ? 0 : max(0, seen + row0 / p.G) / BN - sg.u0;
    last = p.sel ? 0x7fffffff : (max(0, seen + row1 / p.G) + BN - 1) / BN - sg.u0;
  }
};

template <int D>
struct Cfg {
  static constexpr int NCH = (D + 63) / 64;
  static constexpr int CHUNK = 128 * 128;            // 128 rows of 128 bytes
  static constexpr int TILE = NCH * CHUNK;
  static constexpr int OFF_Q = 0, OFF_K = 2 * TILE, OFF_V = 4 * TILE;   // each twice
  // the additional step of Q K^T: 128 rows of 16 columns, unswizzled (8 rows of
  // 16 bytes are 128 bytes together, the two column halves next to each other)
  static constexpr int AUG = 128 * 32, OFF_QA = 6 * TILE, OFF_KA = OFF_QA + 2 * AUG;
  static constexpr int OFF_TILE = OFF_KA + 2 * AUG;
  static_assert(OFF_TILE % 16 == 0, "records are aligned");
  static constexpr int OFF_BAR = OFF_TILE + kRing * (int)sizeof(Tile);
  static constexpr int USED = OFF_BAR + 240;
  // more than half of the SM's, since a block allocates all TMEM columns
  static constexpr int SMEM = (USED + 1024 > 120 * 1024) ? USED + 1024 : 120 * 1024;
  static constexpr int PARTS = D / 32;               // 16-byte pieces of a key's codes
  // a producer takes piece pt % PARTS of every STEP-th key from pt / PARTS on
  static constexpr int STEP = kProducers / PARTS;
  static constexpr int LOADS = (BN + STEP - 1) / STEP;
  static_assert(kProducers % PARTS == 0 && STEP % 8 == 0, "the swizzle is the same for all keys of a thread");
  static constexpr int SLOT = TR * (D + 2);          // floats of a part of an item
  static_assert(SMEM <= 227 * 1024, "shared memory of an SM");
};

// 32 lanes x 8 consecutive columns.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// 16-byte piece of row r of the additional step's operands, columns 0 to 7
// (columns 8 to 15 are 8 pieces on).
__device__ __forceinline__ int aug_at(int r) { return (r >> 3) * 16 + (r & 7); }

// x as the sum of three fp16 numbers.
__device__ __forceinline__ void split3(float x, float &a, float &b, float &c) {
  a = __half2float(__float2half_rn(x));
  b = __half2float(__float2half_rn(x - a));
  c = x - a - b;
}

// Shared-memory matrix descriptor of an unswizzled operand: lbo between the two
// 16-byte columns, sbo between groups of 8 rows.
__device__ __forceinline__ uint64_t smem_desc_plain(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)((sbo >> 4) & 0x3FFFu) << 32;
  d |= (uint64_t)1 << 46;
  return d;
}

// Instruction descriptor of kind::f16 with fp16 A/B and fp32 accumulation.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, int b_mn_major) {
  return (1u << 4) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

constexpr uint32_t kBothBf16 = (1u << 7) | (1u << 10);

// The sizes of a causal item's keys and values that not all of its rows see, and of
// its first row's own, are near enough to one another for kAsIs.  All threads.
// near[4]: largest and least K, V.
constexpr uint32_t kNearK = 6, kNearV = 10;
__device__ __forceinline__ float bound_of(uint32_t meta) {     // of |x| of a row: |least| or |least + 15 s|, or not finite
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(bf_hi(meta))), "f"(fabsf(fmaf(15.f, bf_lo(meta), bf_hi(meta)))));
  return r;
}
template <int D>
__device__ __forceinline__ bool far_apart(const Params &p, const hattn::Segment &sg, uint32_t *near) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int from = max(0, sg.rq.kv - (sg.rq.n_q - 1) + sg.tile * TR / p.G - 1);
  __syncthreads();
  if (threadIdx.x < 4) near[threadIdx.x] = (threadIdx.x & 1) ? ~0u : 0u;
  __syncthreads();
  const int *table = p.block_table + (size_t)sg.r * p.max_blocks;
  uint32_t lim[4] = {0u, ~0u, 0u, ~0u};
  const int last = (sg.rq.kv + kPage - 1) / kPage;
  constexpr int U = 4, WARPS = kThreads / 32;
  for (int b0 = from / kPage + warp; b0 < last; b0 += WARPS * U) {
    int page[U];
#pragma unroll
    for (int e = 0; e < U; ++e) page[e] = b0 + e * WARPS < last ? __ldg(table + b0 + e * WARPS) : -1;
#pragma unroll
    for (int e = 0; e < U; ++e) {
      if (page[e] < 0 || page[e] >= p.n_pages) continue;
      const uint32_t *src = reinterpret_cast<const uint32_t *>(
          p.data + ((size_t)page[e] * p.Hkv + sg.h) * page_bytes(D) + kPage * D);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int pos = (b0 + e * WARPS) * kPage + (k & 1) * 32 + lane;
        const float x = bound_of(__ldg(src + k * 32 + lane));
        if (pos >= from && pos < sg.rq.kv && x > 0.f && x < INFINITY) {
          lim[(k >> 1) * 2] = max(lim[(k >> 1) * 2], __float_as_uint(x));
          lim[(k >> 1) * 2 + 1] = min(lim[(k >> 1) * 2 + 1], __float_as_uint(x));
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    lim[k] = (k & 1) ? __reduce_min_sync(0xffffffffu, lim[k]) : __reduce_max_sync(0xffffffffu, lim[k]);
    if (lane == 0) {
      if (k & 1) atomicMin(near + k, lim[k]);
      else atomicMax(near + k, lim[k]);
    }
  }
  __syncthreads();
  return (near[0] >> 23) > (near[1] >> 23) + kNearK || (near[2] >> 23) > (near[3] >> 23) + kNearV;
}

template <int D, Sizes SIZES>
__global__ void __launch_bounds__(kThreads, 1) kv4_chunk_kernel(const __grid_constant__ Params p) {
  using C = Cfg<D>;
  constexpr bool FAR = SIZES == kFarApart;
  if constexpr (FAR) {
    // the words of every block of the launch before, if there was one
    if (p.words && !__syncthreads_or(threadIdx.x < gridDim.x && p.words[threadIdx.x] != 0)) return;
  }
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ long long s_scan[kThreads / 32 + 1];
  __shared__ int s_request, s_last[2];
  // each warp's place on the line; in shared memory, since the registers hold
  // scores and codes
  using WalkT = hattn::Walk<TR, 2, kSetup>;
  __shared__ hattn::Range s_range;
  __shared__ WalkT s_walk[kThreads / 32];
  __shared__ hattn::Segment s_seg[kThreads / 32];
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar = sbase + C::OFF_BAR;
  auto q_full = [&](int k) { return bar + 8 * k; };
  auto k_full = [&](uint32_t n) { return bar + 16 + 8 * (n & 1); };
  auto k_empty = [&](uint32_t n) { return bar + 32 + 8 * (n & 1); };
  auto v_full = [&](uint32_t n) { return bar + 48 + 8 * (n & 1); };
  auto v_empty = [&](uint32_t n) { return bar + 64 + 8 * (n & 1); };
  auto s_full = [&](int k) { return bar + 80 + 8 * k; };
  auto p_full = [&](int k) { return bar + 96 + 8 * k; };
  auto o_full = [&](int k) { return bar + 112 + 8 * k; };
  auto tile_full = [&](uint32_t n) { return bar + 128 + 8 * (n % kRing); };
  auto tile_empty = [&](uint32_t n) { return bar + 160 + 8 * (n % kRing); };
  // the softmax warps of a row tile meet here when a part of an item is written
  // (barriers with a limit, since any of them may have given up)
  auto part_bar = [&](int k) { return bar + 192 + 8 * k; };
  auto join_bar = [&](int k) { return bar + 208 + 8 * k; };
  const uint32_t drain_bar = bar + 224;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_BAR + 232);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_BAR + 236);
  Tile *tiles = reinterpret_cast<Tile *>(smem + C::OFF_TILE);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  WaitCtl ctl{abort_flag, p.dev_status, p.wait_limit_ns};

  {
    hattn::Range g;
    if (!hattn::find_range<TR, 2, kSetup, kThreads, true>(p, kMinUnits, g, s_scan, &s_request)) {
      if (!FAR && p.causal && threadIdx.x == 0) p.words[blockIdx.x] = 0;
      return;
    }
    if (!FAR && p.causal) {
      __shared__ uint32_t s_near[4];
      WalkT look;
      hattn::Segment part;
      look.start(p, g);
      bool far = false;
      while (look.next(p, part)) far = far_apart<D>(p, part, s_near) || far;
      if (threadIdx.x == 0) p.words[blockIdx.x] = far;
    }
    if (p.sel && blockIdx.x == 0)                 // counts out of range
      for (int i = threadIdx.x; i < p.R * p.Hkv; i += kThreads) {
        const int count = __ldg(p.sel_count + i);
        if (count < 0 || count > p.max_sel) set_status(p.dev_status, DITANGO_ERR_BOUNDS);
      }
    if (lane == 0) s_walk[warp].start(p, g);
    if (threadIdx.x == 0) s_range = g;
  }
  const hattn::Segment &sg = s_seg[warp];
  auto next_segment = [&]() -> bool {
    bool more = false;
    __syncwarp();
    if (lane == 0) more = s_walk[warp].next(p, s_seg[warp]);
    __syncwarp();
    return __shfl_sync(0xffffffffu, (int)more, 0) != 0;
  };

  if (threadIdx.x == 0) {
    for (int k = 0; k < 2; ++k) {
      mbar_init(q_full(k), 4);        // one arrival per softmax warp
      mbar_init(k_full(k), 3);        // one per producer warp
      mbar_init(k_empty(k), 1);
      mbar_init(s_full(k), 1);
      mbar_init(p_full(k), 4);
      mbar_init(o_full(k), 1);
      mbar_init(v_full(k), 3);
      mbar_init(v_empty(k), 1);
      mbar_init(part_bar(k), 4);
      mbar_init(join_bar(k), 1);
    }
    mbar_init(drain_bar, 1);
    for (int k = 0; k < kRing; ++k) {
      mbar_init(tile_full(k), 1);
      mbar_init(tile_empty(k), 1);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  // columns 8 to 15 of the additional step stay zero
  for (int k = threadIdx.x; k < 4 * 128; k += kThreads)
    reinterpret_cast<uint4 *>(smem + C::OFF_QA + (k >> 7) * C::AUG)[aug_at(k & 127) + 8] = make_uint4(0, 0, 0, 0);
  fence_proxy_async();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kControlRegs));
    bool ok = true;
    uint32_t n0 = 0;             // tiles of the segments before
    if (warp == 9) {
      // ---------------------------------------------------------- records
      // bound of |x|: |least| or |least + 15 s|; not finite: the row stands for NaN
      auto bound = [](uint32_t m) { return bound_of(m); };
      auto reference = [](uint32_t top) { return min(max((top >> 23) + 1u, 64u), 253u) << 23; };
      while (ok && next_segment()) {
        const hattn::Pages pages(p, sg, false);
        const int T = sg.u1 - sg.u0, first = 2 * sg.u0, head = sg.h;
        uint32_t vref_bits = 64u << 23;        // 2^-63: a power of two that no V of the segment exceeds
        bool wide = false;
        const Edge edge(p, sg);
        // page numbers are read two tiles ahead, scales one
        int page[2], ppos[2], pos[2], at[2];   // the next tile's pages and places, this one's
        uint32_t mk[4], mv[4];
        auto look = [&](int j) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            int blk = -1;
            page[e] = j < T ? pages.page(first + 2 * j + e, blk, lane == 0) : -1;
            ppos[e] = page[e] >= 0 ? blk * kPage : 0x7fffffff;
          }
        };
        auto fetch = [&]() {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int e = k >> 1, key = (k & 1) * 32 + lane;
            mk[k] = mv[k] = 0u;                // tokens past the end: scale and h 0
            if (page[e] >= 0 && key < pages.kv - ppos[e]) {
              const uint32_t *src = reinterpret_cast<const uint32_t *>(
                  p.data + ((size_t)page[e] * p.Hkv + head) * page_bytes(D) + kPage * D) + key;
              mk[k] = __ldg(src);
              mv[k] = __ldg(src + kPage);
            }
          }
          pos[0] = ppos[0];
          pos[1] = ppos[1];
          at[0] = max(page[0], 0);             // (no page: pos is past every length)
          at[1] = max(page[1], 0);
        };
        look(0);
        fetch();
        look(1);
        for (int j = 0; j < T; ++j) {
          const uint32_t n = n0 + j;
          if (!(ok = wait_warp(tile_empty(n), ((n / kRing) & 1) ^ 1, ctl))) break;
          Tile &tile = tiles[n % kRing];
          uint32_t ktop = 0, vtop = 0;
          if (FAR && j >= edge.last) {      // seen by no row
#pragma unroll
            for (int k = 0; k < 4; ++k) mv[k] = 0u;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float kb = bound(mk[k]), vb = bound(mv[k]);
            if (kb < INFINITY) ktop = max(ktop, __float_as_uint(kb));
            const bool bad = !(vb < INFINITY);
            if (bad) mv[k] = 0u; else vtop = max(vtop, __float_as_uint(vb));
            const uint32_t word = __ballot_sync(0xffffffffu, bad);
            if (lane == 0) tile.bad[k] = word;
          }
          const uint32_t kref_bits = reference(__reduce_max_sync(0xffffffffu, ktop));
          const uint32_t vnew = reference(__reduce_max_sync(0xffffffffu, vtop));
          if (FAR && j >= edge.first && j < edge.last && !wide) {
            uint32_t low = ~0u;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float vb = bound(mv[k]);
              if (vb > 0.f) low = min(low, __float_as_uint(vb));
            }
            low = __reduce_min_sync(0xffffffffu, low);
            wide = (max(vnew, vref_bits) >> 23) > (low >> 23) + 1u + kEvenV ||
                   (vref_bits > 64u << 23 && vnew > vref_bits + (kEvenV << 23));
          }
          vref_bits = FAR && wide ? kWideRef : max(vref_bits, vnew);
          const float kdown = __uint_as_float((254u << 23) - kref_bits), vdown = __uint_as_float((254u << 23) - vref_bits);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int key = k * 32 + lane;
            const float ks = bf_lo(mk[k]), vs = bf_lo(mv[k]);
            tile.ks[key] = hattn::pack_f16x2(ks * kdown, ks * kdown);
            tile.kh[key] = fmaf(8.f, ks, bf_hi(mk[k])) * kdown;
            const float vh = fmaf(8.f, vs, bf_hi(mv[k])) * vdown;
            tile.v[key] = make_uint2(hattn::pack_f16x2(vs * vdown, vs * vdown), hattn::pack_f16x2(vh, vh));
            if (FAR && wide) {
              tile.v[key] = make_uint2(0x3c003c00u, 0u);
              tile.vw[key] = make_float2(vs * vdown, vh);
            }
          }
          if (lane == 0) {
            tile.kref = __uint_as_float(kref_bits);
            tile.vref = __uint_as_float(vref_bits);
            if (FAR) tile.flags = wide ? kWideV : 0u;
            tile.pos[0] = pos[0];
            tile.pos[1] = pos[1];
          }
          if (FAR && j >= edge.first && j < edge.last) {
            // K once more, key by key, if the sizes are far apart (the scales are read
            // again: this is rare, and the code around it stays as fast as it is)
            auto meta = [&](int k) {
              const uint8_t *src = p.data + ((size_t)(k < 2 ? at[0] : at[1]) * p.Hkv + head) * page_bytes(D) + kPage * D;
              const int key = (k & 1) * 32 + lane, from = k < 2 ? pos[0] : pos[1];
              return key < pages.kv - from ? __ldg(reinterpret_cast<const uint32_t *>(src) + key) : 0u;
            };
            uint32_t low = ~0u;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float kb = bound(mk[k]);
              if (kb > 0.f && kb < INFINITY) low = min(low, __float_as_uint(kb));
            }
            low = __reduce_min_sync(0xffffffffu, low);
            if ((kref_bits >> 23) > (low >> 23) + 1u + kEven) {
#pragma unroll 1
              for (int k = 0; k < 4; ++k) {
                const uint32_t m = meta(k);
                const float kb = bound(m), s = bf_lo(m);
                const uint32_t own = kb < INFINITY ? reference(__float_as_uint(kb)) : 127u << 23;
                const float down = __uint_as_float((254u << 23) - own);
                const int key = k * 32 + lane;
                tile.ks[key] = hattn::pack_f16x2(s * down, s * down);
                tile.kh[key] = fmaf(8.f, s, bf_hi(m)) * down;
                tile.kf[key] = __uint_as_float(own - (20u << 23));
              }
              if (lane == 0) {
                // a power of two in the middle, so that no score with its key's own
                // factor leaves fp32
                tile.kref = 0x1p20f;
                tile.flags = kOwnK | (wide ? kWideV : 0u);
              }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(tile_full(n));
          fetch();
          look(j + 2);
        }
        n0 += T;
      }
    } else if (warp >= 10) {
      // ---------------------------------------------------------- producers
      const bool is_v = warp >= 13;
      const int pt = threadIdx.x - (is_v ? 416 : 320);
      const int row0 = pt / C::PARTS, part = pt % C::PARTS;
      // 8 channels (word w of the piece) of key row0, 128-byte swizzled
      auto place = [&](int w) {
        const int atom = (part & 1) * 4 + (part >= 2 ? w ^ 2 : w);
        return (part >> 1) * C::CHUNK + row0 * 128 + ((atom ^ (row0 & 7)) << 4);
      };
      const hattn::Unpack unpack8;
      const int at[4] = {place(0), place(1), place(2), place(3)};
      const int from = (is_v ? kPage * D / 2 : 0) + row0 * (D / 2) + part * 16;
      while (ok && next_segment()) {
        const hattn::Pages pages(p, sg, false);
        const int T = sg.u1 - sg.u0, first = 2 * sg.u0, head = sg.h;
        // page numbers are read two tiles ahead, codes one
        int page[2];
        auto look = [&](int j) {
          int blk;
#pragma unroll
          for (int e = 0; e < 2; ++e) page[e] = j < T ? pages.page(first + 2 * j + e, blk, false) : -1;
        };
        uint4 c[C::LOADS];
        auto fetch = [&](int k) {
          const int row = row0 + k * C::STEP, e = row >= kPage;
          const int pg = e ? page[1] : page[0];
          c[k] = make_uint4(0, 0, 0, 0);
          if (row < BN && pg >= 0)
            c[k] = __ldg(reinterpret_cast<const uint4 *>(p.data + ((size_t)pg * p.Hkv + head) * page_bytes(D) + from +
                                                         k * C::STEP * (D / 2) - (e ? kPage * D / 2 : 0)));
        };
        look(0);
#pragma unroll
        for (int k = 0; k < C::LOADS; ++k) fetch(k);
        look(1);
        for (int j = 0; j < T; ++j) {
          const uint32_t n = n0 + j;
          if (!(ok = wait_warp(tile_full(n), (n / kRing) & 1, ctl))) break;
          if (!(ok = wait_warp(is_v ? v_empty(n) : k_empty(n), ((n >> 1) & 1) ^ 1, ctl))) break;
          const Tile &tile = tiles[n % kRing];
          uint8_t *dst = smem + (is_v ? C::OFF_V : C::OFF_K) + (n & 1) * C::TILE;
#pragma unroll
          for (int k = 0; k < C::LOADS; ++k) {
            const int row = row0 + k * C::STEP;
            if (row < BN) {
              // K: s (c - 8), exactly; V: s (c - 8) + h
              const uint2 sh = is_v ? tile.v[row] : make_uint2(tile.ks[row], 0x80008000u);
              const uint32_t w[4] = {c[k].x, c[k].y, c[k].z, c[k].w};
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                uint32_t x[4];
                unpack8(w[q], x);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = hattn::hfma2(x[e], sh.x, sh.y);
                *reinterpret_cast<uint4 *>(dst + at[q] + k * C::STEP * 128) = make_uint4(x[0], x[1], x[2], x[3]);
              }
            }
            fetch(k);                  // the next tile's
          }
          if (!is_v) {
            // h against sum(q) = (1 1 2 1 3 2): 1 2 1 3 1 2
            for (int row = pt; row < BN; row += kProducers) {
              float h1, h2, h3;
              split3(tile.kh[row], h1, h2, h3);
              const uint32_t h12 = hattn::pack_f16x2(h1, h2), h13 = hattn::pack_f16x2(h1, h3);
              reinterpret_cast<uint4 *>(smem + C::OFF_KA + (n & 1) * C::AUG)[aug_at(row)] = make_uint4(h12, h13, h12, 0);
            }
          }
          if (FAR && is_v && (tile.flags & kWideV)) {
            // c - 8 stands there: s (c - 8) + h as bf16 in its place
#pragma unroll 1
            for (int row = row0; row < BN; row += C::STEP) {
              const float2 sh = tile.vw[row];
              auto wide = [&](uint32_t x) {
                return pack_bf16x2(fmaf(__half2float(__ushort_as_half((unsigned short)(x & 0xffffu))), sh.x, sh.y),
                                   fmaf(__half2float(__ushort_as_half((unsigned short)(x >> 16))), sh.x, sh.y));
              };
#pragma unroll 1
              for (int q = 0; q < 4; ++q) {
                uint4 *to = reinterpret_cast<uint4 *>(dst + place(q) + (row - row0) * 128);
                const uint4 x = *to;
                *to = make_uint4(wide(x.x), wide(x.y), wide(x.z), wide(x.w));
              }
            }
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(is_v ? v_full(n) : k_full(n));
          look(j + 2);
        }
        n0 += T;
      }
    } else {
      // ---------------------------------------------------------- MMA issuer
      // The whole warp runs the loop; one elected lane issues and commits, what it
      // names being pinned before its branch.
      const bool leader = elect_one();
      constexpr uint32_t idesc_qk = idesc_f16_f32(BM, BN, 0);
      constexpr uint32_t idesc_pv = idesc_f16_f32(BM, D, 1);
      auto commit = [&](uint32_t at) {
        at = pinned(at);
        if (leader) tc_commit(at);
      };
      auto qk = [&](int k, uint32_t n) {
        const uint64_t a = pinned(smem_desc_sw128(sbase + C::OFF_Q + k * C::TILE, 16, 1024));
        const uint64_t b = pinned(smem_desc_sw128(sbase + C::OFF_K + (n & 1) * C::TILE, 16, 1024));
        const uint64_t qa = pinned(smem_desc_plain(sbase + C::OFF_QA + k * C::AUG, 128, 256));
        const uint64_t ka = pinned(smem_desc_plain(sbase + C::OFF_KA + (n & 1) * C::AUG, 128, 256));
        const uint32_t full = pinned(s_full(k));
        // S_k = Q_k K^T.  P of the tile before lives in S_k: its product was
        // issued before, and one thread's products run in order.
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t off = (uint64_t)(((kk >> 2) * C::CHUNK + (kk & 3) * 32) >> 4);
            mma_ss(tmem + 128 * k, a + off, b + off, idesc_qk, kk > 0);
          }
          mma_ss(tmem + 128 * k, qa, ka, idesc_qk, 1);
          tc_commit(full);
        }
      };
      auto pv = [&](int k, uint32_t n, bool acc, uint32_t idesc) {
        const uint64_t b = pinned(smem_desc_sw128(sbase + C::OFF_V + (n & 1) * C::TILE, C::CHUNK, 1024));
        const uint32_t accumulate = pinned(acc ? 1u : 0u);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            mma_ts(tmem + 256 + 128 * k, tmem + 128 * k + kk * 8, b + (uint64_t)((kk * 2048) >> 4), idesc,
                   kk > 0 ? 1u : accumulate);
        }
      };
      uint32_t segs = 0, segs1 = 0, pc1 = 0;
      while (ok && next_segment()) {
        const int T = sg.u1 - sg.u0;
        const bool has1 = (long long)sg.rq.n_q * p.G - (long long)sg.tile * TR > BM;
        if (!(ok = wait_warp(q_full(0), segs & 1, ctl))) break;
        ++segs;
        if (has1) {
          if (!(ok = wait_warp(q_full(1), segs1 & 1, ctl))) break;
          ++segs1;
        }
        if (!(ok = wait_warp(k_full(n0), (n0 >> 1) & 1, ctl))) break;
        tc_fence_after();
        qk(0, n0);
        if (has1) qk(1, n0);
        commit(k_empty(n0));
        for (int t = 0; t < T; ++t) {
          const uint32_t n = n0 + t;
          const bool more = t + 1 < T;
          if (!(ok = wait_warp(v_full(n), (n >> 1) & 1, ctl))) break;
          uint32_t kind = idesc_pv;
          if (FAR && (tiles[n % kRing].flags & kWideV)) kind |= kBothBf16;
          kind = pinned(kind);
          if (!(ok = wait_warp(p_full(0), n & 1, ctl))) break;
          tc_fence_after();
          pv(0, n, t > 0, kind);
          if (more) {
            if (!(ok = wait_warp(k_full(n + 1), ((n + 1) >> 1) & 1, ctl))) break;
            tc_fence_after();
            qk(0, n + 1);
          } else {
            commit(o_full(0));
          }
          if (has1) {
            if (!(ok = wait_warp(p_full(1), pc1 & 1, ctl))) break;
            ++pc1;
            tc_fence_after();
            pv(1, n, t > 0, kind);
            if (more) qk(1, n + 1);
            else commit(o_full(1));
          }
          if (more) commit(k_empty(n + 1));
          commit(v_empty(n));
          commit(tile_empty(n));
        }
        n0 += T;
      }
      // what was issued ends before TMEM is released, on both paths
      volatile int never = 0;
      WaitCtl drain{&never, nullptr, 100000000LL};
      commit(drain_bar);
      wait_bounded(drain_bar, 0, drain);
      __syncwarp();
    }
    if (warp == 8) {
      named_bar_sync(1, kThreads);
      tc_fence_after();
      tmem_dealloc(tmem, kTmemCols);
    } else {
      tc_fence_before();
      named_bar_arrive(1, kThreads);
    }
    return;
  }

  // -------------------------------------------------------------- softmax
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
  const int kt = warp >> 2;                     // row tile
  const int r = threadIdx.x & 127;              // row of the tile = TMEM lane
  const uint32_t tS = tmem + 128 * kt + ((uint32_t)((warp & 3) * 32) << 16);
  const uint32_t tO = tS + 256;
  bool ok = true;
  uint32_t n = 0;                               // tiles of all segments
  uint32_t sc = 0, segs = 0, parts = 0;         // of those with rows of this tile
  while (ok && next_segment()) {
    const int row0 = sg.tile * TR + kt * BM;
    const int rows = (int)min((long long)BM, (long long)sg.rq.n_q * p.G - row0);
    const int units = sg.u1 - sg.u0;
    if (rows <= 0) {                            // a tile of rows that are not there
      n += units;
      continue;
    }
    // ---- Q of this row: fp16 below 2, channels in the codes' order
    float qsum = 0.f, mul;
    int vis = sg.rq.kv;                         // keys that the row sees
    {
      const bool live = r < rows;
      const int tok = live ? (row0 + r) / p.G : 0, head = live ? (row0 + r) % p.G : 0;
      if (p.causal && live) vis -= sg.rq.n_q - 1 - tok;
      const uint4 *src = reinterpret_cast<const uint4 *>(p.Q + (sg.rq.q0 + tok) * p.qt + (sg.h * p.G + head) * p.qh);
      uint4 u[D / 8];
      float big = 0.f;
#pragma unroll
      for (int k = 0; k < D / 8; ++k) {
        u[k] = live ? __ldg(src + k) : make_uint4(0, 0, 0, 0);
        big = fmaxf(big, hattn::max_abs8(u[k]));
      }
      const uint32_t ex = min(max(__float_as_uint(big) >> 23, 1u), 253u);
      const float down = __uint_as_float((254u - ex) << 23);
#pragma unroll
      for (int k = 0; k < D / 8; ++k) {
        uint32_t x[4];
        hattn::q_pairs(u[k], down, x, qsum);
        *reinterpret_cast<uint4 *>(smem + C::OFF_Q + kt * C::TILE + (k >> 3) * C::CHUNK + r * 128 +
                                  ((((k & 7) ^ (k >= 8 ? 2 : 0)) ^ (r & 7)) << 4)) =
            make_uint4(x[0], x[1], x[2], x[3]);
      }
      mul = p.scale_log2 * __uint_as_float(ex << 23);
      float q1, q2, q3;
      split3(qsum, q1, q2, q3);
      reinterpret_cast<uint4 *>(smem + C::OFF_QA + kt * C::AUG)[aug_at(r)] =
          make_uint4(hattn::pack_f16x2(q1, q1), hattn::pack_f16x2(q2, q1), hattn::pack_f16x2(q3, q2), 0);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full(kt));
    }
    vis = max(vis, 0);
    float m_used = -INFINITY, l = 0.f, vref = 1.f;
    bool poison = false;            // the row sees a key whose V is not finite
    for (int u = 0; u < units; ++u, ++n, ++sc) {
      // S first: then the record of tile n is there and the ring not yet round
      // (warps that passed over segments may come early)
      if (!(ok = wait_bounded(s_full(kt), sc & 1, ctl))) break;
      if (!(ok = wait_bounded(tile_full(n), (n / kRing) & 1, ctl))) break;
      const Tile &tile = tiles[n % kRing];
      const int n0 = max(0, min(kPage, vis - tile.pos[0])), n1 = max(0, min(kPage, vis - tile.pos[1]));
      __syncwarp();
      tc_fence_after();
      if constexpr (FAR) {
        if (__any_sync(0xffffffffu, (tile.flags & kOwnK) != 0u)) {
          // the keys' own factors, in place, before the scores take the registers
          // (this test alone costs the loop 3%: calls that are not causal have none)
#pragma unroll 1
          for (int c = 0; c < BN; c += 8) {
            uint32_t v[8];
            tmem_ld8(tS + c, v);
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * tile.kf[c + e]);
            tmem_st8(tS + c, v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]);
          }
          tc_wait_st();
        }
      }
      uint32_t sv[BN];
#pragma unroll
      for (int c = 0; c < BN / 16; ++c) tmem_ld16p(tS + c * 16, &sv[c * 16]);
      tc_wait_ld();
      const float v_now = tile.vref, mulk = hattn::score_factor(mul * tile.kref);
      // rows of a warp may see different keys: the branch is the warp's, so that it
      // stays together for the tensor memory instructions
      if (__any_sync(0xffffffffu, n0 + n1 < BN)) {
#pragma unroll
        for (int c = 0; c < BN; ++c)
          if (c < kPage ? c >= n0 : c - kPage >= n1) sv[c] = __float_as_uint(-INFINITY);
      }
      if (tile.bad[0] | tile.bad[1] | tile.bad[2] | tile.bad[3]) {
        auto low = [](int k) { return k <= 0 ? 0u : (k >= 32 ? ~0u : (1u << k) - 1u); };
        poison = poison || ((tile.bad[0] & low(n0)) | (tile.bad[1] & low(n0 - 32)) | (tile.bad[2] & low(n1)) |
                            (tile.bad[3] & low(n1 - 32))) != 0u;
      }
      float m8[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        m8[q] = max3(__uint_as_float(sv[q]), __uint_as_float(sv[q + 8]), __uint_as_float(sv[q + 16]));
#pragma unroll
      for (int c = 24; c + 16 <= BN; c += 16)
#pragma unroll
        for (int q = 0; q < 8; ++q)
          m8[q] = max3(m8[q], __uint_as_float(sv[c + q]), __uint_as_float(sv[c + q + 8]));
#pragma unroll
      for (int q = 0; q < 8; ++q) m8[q] = fmaxf(m8[q], __uint_as_float(sv[BN - 8 + q]));
      const float mx2 =
          max3(max3(m8[0], m8[1], m8[2]), max3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7])) * mulk;
      if (u == 0) {
        m_used = reference_of(mx2);
      } else {
        // S of this tile is complete, and with it every product issued before:
        // O may be rescaled, when a maximum grew by more than 2^8 or V's reference did
        const bool need = outgrown(mx2, m_used);
        if (__any_sync(0xffffffffu, need || v_now != vref)) {
          const float m_new = need ? reference_of(mx2) : m_used;
          const float alpha = need ? fast_ex2(m_used - m_new) : 1.f;
          l *= alpha;
          m_used = m_new;
          const float ao = alpha * (vref / v_now);
          // 16 columns at a time, one piece after the other: the scores hold the registers
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t v[16];
            tmem_ld16p(tO + c, v);
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * ao);
            tmem_st8(tO + c, v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]);
            tmem_st8(tO + c + 8, v[8], v[9], v[10], v[11], v[12], v[13], v[14], v[15]);
          }
        }
      }
      vref = v_now;
      const float neg = m_used > -INFINITY ? -m_used : 0.f;   // no key so far: exponentiate against 0
      const uint64_t neg2 = f2(neg, neg);
      uint64_t factor = f2(mulk, mulk);
      if (__any_sync(0xffffffffu, fabsf(neg) > kHuge)) {
#pragma unroll
        for (int c = 0; c < BN; ++c) sv[c] = __float_as_uint(__fmul_rn(__uint_as_float(sv[c]), mulk));
        factor = f2(1.f, 1.f);
      }
      uint64_t lsum[4] = {0, 0, 0, 0};
#pragma unroll
      for (int g8 = 0; g8 < BN / 16; ++g8) {
        uint32_t pk[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = g8 * 16 + 2 * e;
          float xa, xb;
          unf2(fma2(f2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), factor, neg2), xa, xb);
          const float a = fast_ex2(xa), b = fast_ex2(xb);
          lsum[e & 3] = add2(lsum[e & 3], f2(a, b));
          pk[e] = hattn::pack_f16x2(a, b);
        }
        tmem_st8(tS + g8 * 8, pk[0], pk[1], pk[2], pk[3], pk[4], pk[5], pk[6], pk[7]);
      }
      {
        float s0, s1, s2, s3;
        unf2(add2(lsum[0], lsum[2]), s0, s1);
        unf2(add2(lsum[1], lsum[3]), s2, s3);
        l += (s0 + s1) + (s2 + s3);
      }
      if constexpr (FAR) {
        if (__any_sync(0xffffffffu, (tile.flags & kWideV) != 0u)) {     // P in bf16, as V
          tc_wait_st();
#pragma unroll 1
          for (int c = 0; c < BN / 2; c += 8) {
            uint32_t v[8];
            tmem_ld8(tS + c, v);
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e)
              v[e] = pack_bf16x2(__half2float(__ushort_as_half((unsigned short)(v[e] & 0xffffu))),
                                 __half2float(__ushort_as_half((unsigned short)(v[e] >> 16))));
            tmem_st8(tS + c, v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]);
          }
        }
      }
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full(kt));
    }
    if (!ok) break;
    if (!(ok = wait_bounded(o_full(kt), segs & 1, ctl))) break;
    ++segs;
    tc_fence_after();
    // ---- O: every product of the segment is done, so this warp's rows of the
    // Q tile are free to stage 32 columns at a time
    const bool whole = sg.whole();
    float *part = p.partial + ((size_t)blockIdx.x * 2 + (sg.u0 == 0 ? 1 : 0)) * C::SLOT + kt * BM * (D + 2);
    const bool none = !(l > 0.f) && l == l;
    // (parts are over 2^40: a sum of the largest values that is not yet divided stays finite)
    float fac = whole ? (l > 0.f ? vref / l : 0.f) : vref * kWideDown;
    if (!(l == l) || poison) fac = __uint_as_float(0x7fc00000u);
    float4 *epi = reinterpret_cast<float4 *>(smem + C::OFF_Q + kt * C::TILE + (warp & 3) * 4096);
    auto out_row = [&](int row) -> long long {      // element offset of a row of the tile in out
      const int at = row0 + row;
      return (sg.rq.q0 + at / p.G) * p.ot + (sg.h * p.G + at % p.G) * p.oh;
    };
    const int wrow = r & ~31;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      uint32_t ov[32];
      tmem_ld32(tO + c * 32, ov);
      tc_wait_ld();
      if (none) {
#pragma unroll
        for (int e = 0; e < 32; ++e) ov[e] = 0u;
      }
      // columns 8 g + 2 i and 8 g + 2 i + 1 are channels 8 g + i and 8 g + 4 + i,
      // of the second 64 those of group g ^ 2
      auto val = [&](int ch) {
        return __uint_as_float(ov[((ch & ~7) ^ (c >= 2 ? 16 : 0)) + ((ch & 3) << 1) + ((ch >> 2) & 1)]) * fac;
      };
      if (!whole || p.out_fp32) {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          epi[lane * 8 + (q ^ (lane & 7))] = make_float4(val(4 * q), val(4 * q + 1), val(4 * q + 2), val(4 * q + 3));
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int row = (lane >> 3) + 4 * q, seg = lane & 7;
          if (wrow + row < rows) {
            float *dst = whole ? static_cast<float *>(p.out) + out_row(wrow + row) : part + (wrow + row) * D;
            reinterpret_cast<float4 *>(dst + c * 32)[seg] = epi[row * 8 + (seg ^ (row & 7))];
          }
        }
      } else {
        uint2 *ep = reinterpret_cast<uint2 *>(epi);
#pragma unroll
        for (int q = 0; q < 8; ++q)
          ep[lane * 8 + (q ^ (lane & 7))] = make_uint2(pack_bf16x2(val(4 * q), val(4 * q + 1)),
                                                       pack_bf16x2(val(4 * q + 2), val(4 * q + 3)));
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int row = (lane >> 3) + 4 * q, seg = lane & 7;
          if (wrow + row < rows)
            reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + out_row(wrow + row) + c * 32)[seg] =
                ep[row * 8 + (seg ^ (row & 7))];
        }
      }
      __syncwarp();
    }
    auto store_lse = [&](int row, float m_, float l_) {
      const int at = row0 + row;
      if (p.out_lse)
        p.out_lse[(sg.rq.q0 + at / p.G) * p.lt + (sg.h * p.G + at % p.G) * p.lh] =
            l_ > 0.f ? (m_ + log2f(l_)) * 0.69314718055994531f : (l_ == l_ ? -INFINITY : l_);
    };
    if (whole) {
      if (r < rows) store_lse(r, m_used, l);
      continue;
    }
    // ---- a part of an item: the block that finishes it last joins the parts
    if (r < rows) {
      part[BM * D + 2 * r] = m_used;
      part[BM * D + 2 * r + 1] = l;
    }
    long long first, last;
    hattn::sharers<kSetup>(s_range, sg, first, last);
    __threadfence();
    __syncwarp();
    if (lane == 0) mbar_arrive(part_bar(kt));
    if ((warp & 3) == 0) {
      if (!(ok = wait_warp(part_bar(kt), parts & 1, ctl))) break;
      if (lane == 0) {
        int *counter = p.counters + 2 * first + kt;
        const int before = atomicAdd(counter, 1);
        s_last[kt] = before == (int)(last - first + 1);
        if (s_last[kt]) *counter = 0;         // left at zero for the next launch
        mbar_arrive(join_bar(kt));
      }
    }
    if (!(ok = wait_warp(join_bar(kt), parts & 1, ctl))) break;
    ++parts;
    const bool join = *static_cast<volatile int *>(&s_last[kt]) != 0;   // written again only after all four warps came back
    if (!join) continue;
    __threadfence();
    // Eight lanes take a row, D / 8 channels each, so that its m and l are read
    // once; two rows and PB parts of each are in flight together: with one group of
    // four channels a thread at a time the join of ten parts took 40 us.
    constexpr int NV = D / 32, UR = 2, PB = D == 64 ? 4 : (D == 96 ? 3 : 2);
    const int sub = lane & 7, row_in = (warp & 3) * 4 + (lane >> 3);
    for (int base = 0; base < rows; base += 16 * UR) {
      float mt[UR], lt[UR];
      float4 v[UR][NV];
#pragma unroll
      for (int w = 0; w < UR; ++w) {
        mt[w] = -INFINITY;
        lt[w] = 0.f;
#pragma unroll
        for (int q = 0; q < NV; ++q) v[w][q] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      for (long long c0 = first - 1; c0 <= last; c0 += PB) {
        float2 ml[UR][PB];
        float4 x[UR][PB][NV];
#pragma unroll
        for (int w = 0; w < UR; ++w)
#pragma unroll
          for (int e = 0; e < PB; ++e) {
            const long long c = c0 + e;
            const int row = base + 16 * w + row_in;
            ml[w][e] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int q = 0; q < NV; ++q) x[w][e][q] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c <= last && row < rows) {
              const float *src = p.partial + (c * 2 + (c == first - 1 ? 1 : 0)) * C::SLOT + kt * BM * (D + 2);
              ml[w][e] = __ldcg(reinterpret_cast<const float2 *>(src + BM * D + 2 * row));
#pragma unroll
              for (int q = 0; q < NV; ++q)
                x[w][e][q] = __ldcg(reinterpret_cast<const float4 *>(src + row * D) + sub + 8 * q);
            }
          }
#pragma unroll
        for (int w = 0; w < UR; ++w)
#pragma unroll
          for (int e = 0; e < PB; ++e) {
            const float mn = fmaxf(mt[w], ml[w][e].x), less = mn > -INFINITY ? mn : 0.f;
            const float f0 = fast_ex2(mt[w] - less), f1 = fast_ex2(ml[w][e].x - less);
            lt[w] = lt[w] * f0 + ml[w][e].y * f1;
#pragma unroll
            for (int q = 0; q < NV; ++q) {
              const float4 y = x[w][e][q];
              float4 &z = v[w][q];
              z = make_float4(z.x * f0 + y.x * f1, z.y * f0 + y.y * f1, z.z * f0 + y.z * f1, z.w * f0 + y.w * f1);
            }
            mt[w] = mn;
          }
      }
#pragma unroll
      for (int w = 0; w < UR; ++w) {
        const int row = base + 16 * w + row_in;
        if (row >= rows) continue;
        const float inv = lt[w] > 0.f ? 1.f / kWideDown / lt[w] : (lt[w] == lt[w] ? 0.f : lt[w]);
#pragma unroll
        for (int q = 0; q < NV; ++q) {
          const float4 z = make_float4(v[w][q].x * inv, v[w][q].y * inv, v[w][q].z * inv, v[w][q].w * inv);
          const int ch = (sub + 8 * q) * 4;
          if (p.out_fp32)
            *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + out_row(row) + ch) = z;
          else
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + out_row(row) + ch) =
                make_uint2(pack_bf16x2(z.x, z.y), pack_bf16x2(z.z, z.w));
        }
        if (sub == 0) store_lse(row, mt[w], lt[w]);
      }
    }
  }
  tc_fence_before();
  named_bar_arrive(1, kThreads);
}

template <int D, Sizes SIZES>
cudaError_t launch(const Params &p, int num_sms, cudaStream_t stream) {
  auto kfn = kv4_chunk_kernel<D, SIZES>;
  static OnDevices ready;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!ready.has(dev)) {
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kfn);
    if (e != cudaSuccess) return e;
    // another count would leave setmaxnreg waiting for registers that do not come
    if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::SMEM);
    if (e != cudaSuccess) return e;
    ready.add(dev);
  }
  const int blocks = num_sms < kMaxBlocks ? num_sms : kMaxBlocks;
  kfn<<<blocks, kThreads, Cfg<D>::SMEM, stream>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch(const Params &p, int num_sms, cudaStream_t stream) {
  if (p.causal && p.sel) {          // what a row sees of a list may be of any size beside the new tokens
    Params always = p;
    always.words = nullptr;
    return launch<D, kFarApart>(always, num_sms, stream);
  }
  const cudaError_t e = launch<D, kAsIs>(p, num_sms, stream);
  return e != cudaSuccess || !p.causal ? e : launch<D, kFarApart>(p, num_sms, stream);
}

}  // namespace hchunk

int kv4_chunk_words() { return hchunk::kMaxBlocks; }
size_t kv4_chunk_partial_floats(int d) { return (size_t)hchunk::kMaxBlocks * 2 * hchunk::TR * (d + 2); }
int kv4_chunk_counters() { return 2 * hchunk::kMaxBlocks; }

cudaError_t launch_kv4_chunk(const hattn::Params &p, int d, int num_sms, cudaStream_t stream) {
  switch (d) {
    case 64: return hchunk::launch<64>(p, num_sms, stream);
    case 96: return hchunk::launch<96>(p, num_sms, stream);
    case 128: return hchunk::launch<128>(p, num_sms, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace ditango
