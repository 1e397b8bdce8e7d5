// What the two kernels of attention over the 4-bit history share: their
// parameters and the line of work.
//
// The units (runs of pages) of all (request, row tile, key head) items are one
// line of work that is cut into equal ranges, one a block, so that a single
// long request and a ragged batch fill the GPU alike.  Each item stands on the
// line with SETUP units more, what it costs to begin and to finish one (without
// them a block that got many short requests worked 1.3 times as long as the
// others); a boundary that falls among those moves to the item's start.  An item
// cut by a boundary is joined by the block that finishes it last, from the
// partial states in block order (a fixed order: the result does not depend on
// which block is last).
#pragma once

#include "blocks.cuh"

namespace ditango {
namespace hattn {

struct Params {
  int R, H, Hkv, G, T, max_blocks, n_pages, max_sel, causal;
  const uint16_t *Q;
  long long qt, qh;                  // token and head strides
  const int *q_off, *kv_len, *block_table, *sel, *sel_count;
  const uint8_t *data;
  float scale_log2;
  void *out;
  int out_fp32;
  long long ot, oh;
  float *out_lse;
  long long lt, lh;
  float *partial;                    // two parts of items a block
  int *counters;                     // one a block, all zero between launches
  int *words;                        // many rows, causal: one a block, see Sizes
  int side;                          // which requests are this launch's, see Side
  int *dev_status;
  long long wait_limit_ns;
};

// A launch takes all requests, or the ones that are the few-row kernel's or the
// many-row kernel's of a batch that is launched on both.
enum Side : int { kAllRequests = 0, kFewSide = 1, kManySide = 2 };

// The requests that a launch takes, once the device has looked: the others are
// left to the other kernel.
enum Rows : int { kAllRows, kFewRows, kManyRows, kNoRows };
constexpr int kRows = 16;            // rows of a key head that the kernel of few rows takes in one tile

struct Request {
  int n_q, kv, q0, tiles, units;   // units: work of one item, at least 1
};

// Request r in row tiles of TR rows and units of UNIT pages.  Offsets and lengths
// that cannot be are recorded and clipped.
template <int TR, int UNIT>
__device__ __forceinline__ Request request_of(const Params &p, int r, Rows mine) {
  Request q;
  q.q0 = __ldg(p.q_off + r);
  const int q1 = __ldg(p.q_off + r + 1);
  q.kv = __ldg(p.kv_len + r);
  const long long most = (long long)p.max_blocks * kPage;
  q.n_q = q1 - q.q0;
  if (q.q0 < 0 || q1 < q.q0 || q1 > p.T || q.kv < 0 || q.kv > most) {
    set_status(p.dev_status, DITANGO_ERR_BOUNDS);
    q.kv = (int)max(0LL, min((long long)q.kv, most));
    if (q.q0 < 0 || q1 < q.q0 || q1 > p.T) q.n_q = 0;
  }
  const long long rows = (long long)q.n_q * p.G;
  const bool take = mine == kAllRows || (mine == kFewRows ? rows <= kRows : mine == kManyRows && rows > kRows);
  q.tiles = take ? (int)((rows + TR - 1) / TR) : 0;
  q.units = p.sel ? p.max_sel : (q.kv + kPage - 1) / kPage;
  q.units = q.units < 1 ? 1 : (q.units + UNIT - 1) / UNIT;
  return q;
}

template <int SETUP>
__device__ __forceinline__ long long work_of(const Params &p, const Request &q) {
  return (long long)q.tiles * p.Hkv * (q.units + SETUP);
}

// Sum and exclusive prefix over the block.
template <int WARPS>
__device__ __forceinline__ long long block_scan(long long v, long long &total, long long *sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) sm[warp] = x;
  __syncthreads();
  total = 0;
  long long before = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += sm[w];
    total += sm[w];
  }
  return before + x - v;
}

// The requests with more than 16 rows of a key head go to the kernel of tiles of
// 128 rows where their work, in tiles of 16 rows by a page and 8 pages an item, is
// more than this: the kernel of few rows does 500 a us after 13 us, the other 2 to
// 4 times as many after 30 to 45 us.  (Few against many rows' kernel, 25000 tokens,
// 8 key heads of 128: 12768, 64 rows, 49 against 67 us, 51072, 256 rows, 134 against
// 94 us.  24 key heads of 96, 4000 tokens: 13632, 128 rows, 43 against 45 us, 27264,
// 256 rows, 69 against 53 us.)
constexpr long long kFewWork = 14000;

// All THREADS threads take part; both kernels come to the same answer.
template <int THREADS>
__device__ __forceinline__ Rows rows_of_launch(const Params &p, long long *sm) {
  if (p.side == kAllRequests) return kAllRows;
  long long work = 0;
  for (int base = 0; base < p.R; base += THREADS) {
    const int r = base + (int)threadIdx.x;
    long long v = 0, sum;
    if (r < p.R) v = work_of<8>(p, request_of<kRows, 1>(p, r, kManyRows));
    block_scan<THREADS / 32>(v, sum, sm);
    work += sum;
  }
  const bool many = work > kFewWork;
  if (p.side == kFewSide) return many ? kFewRows : kAllRows;
  return many ? kManyRows : kNoRows;
}

// This block's range [w0, w1) of the line and the request in which it begins.
struct Range {
  Rows rows;
  long long total, n_blk, w0, w1, r_start;
  int r;
};

// All THREADS threads take part; sm: WARPS + 1 long longs and an int.  WHOLE: a
// number of blocks that is a multiple of the items' is preferred where it costs
// less than one block in 16: items of one length are then cut into equal parts
// and no block begins two, and an item of n units is cut into sqrt(2 n) parts at
// most, since one block joins them all, 1.3 us a part (500 queries over 5000 tokens, 10 and 2 heads: 57 us
// without it, 50 us with it.  Few rows: the same, less the time to count the items).
template <int TR, int UNIT, int SETUP, int THREADS, bool WHOLE = false>
__device__ __forceinline__ bool find_range(const Params &p, long long min_units, Range &g, long long *sm, int *sm_r) {
  constexpr int WARPS = THREADS / 32;
  const int tid = threadIdx.x;
  g.rows = rows_of_launch<THREADS>(p, sm);
  g.total = 0;
  long long items = 0;
  long long v = 0, at = 0;           // of request tid: its work and place; all there is up to THREADS requests
  for (int base = 0; base < p.R; base += THREADS) {
    const int r = base + tid;
    long long sum;
    Request q;
    q.tiles = q.units = 0;
    if (r < p.R) q = request_of<TR, UNIT>(p, r, g.rows);
    v = work_of<SETUP>(p, q);
    at = block_scan<WARPS>(v, sum, sm);
    g.total += sum;
    if constexpr (WHOLE) {
      block_scan<WARPS>((long long)q.tiles * p.Hkv, sum, sm);
      items += sum;
    }
  }
  const long long most = (g.total + min_units - 1) / min_units;
  g.n_blk = most < (long long)gridDim.x ? most : (long long)gridDim.x;
  if (WHOLE && items > 0) {
    const long long parts = (long long)ceilf(sqrtf(2.f * ((float)g.total / (float)items)));
    if (items * parts < g.n_blk) g.n_blk = items * parts;
  }
  if (items > 0 && items < g.n_blk && (g.n_blk % items) * 16 <= g.n_blk) g.n_blk -= g.n_blk % items;
  if ((long long)blockIdx.x >= g.n_blk) return false;
  g.w0 = g.total * blockIdx.x / g.n_blk;
  g.w1 = g.total * (blockIdx.x + 1) / g.n_blk;
  long long before = 0;
  for (int base = 0; base < p.R; base += THREADS) {
    const int r = base + tid;
    long long sum = g.total;
    if (p.R > THREADS) {
      v = r < p.R ? work_of<SETUP>(p, request_of<TR, UNIT>(p, r, g.rows)) : 0;
      at = before + block_scan<WARPS>(v, sum, sm);
    }
    if (v > 0 && at <= g.w0 && g.w0 < at + v) {
      *sm_r = r;
      sm[WARPS] = at;
    }
    before += sum;
    if (before > g.w0) break;       // uniform: every thread has the same sum
  }
  __syncthreads();
  g.r = *sm_r;
  g.r_start = sm[WARPS];
  return true;
}

// The part of one item that lies in a block's range.
struct Segment {
  Request rq;
  int r, h, tile, u0, u1;           // units [u0, u1) of the item
  long long start, end;             // of the item, on the line
  __device__ __forceinline__ bool whole() const { return u0 == 0 && u1 == rq.units; }
};

template <int TR, int UNIT, int SETUP>
struct Walk {
  Rows rows;
  long long pos, w1, r_start;
  int r;
  Request rq;
  __device__ __forceinline__ void start(const Params &p, const Range &g) {
    rows = g.rows;
    pos = g.w0;
    w1 = g.w1;
    r_start = g.r_start;
    r = g.r;
    rq = request_of<TR, UNIT>(p, r, rows);
  }
  __device__ __forceinline__ bool next(const Params &p, Segment &s) {
    if (pos >= w1) return false;
    while (pos >= r_start + work_of<SETUP>(p, rq)) {
      r_start += work_of<SETUP>(p, rq);
      ++r;
      rq = request_of<TR, UNIT>(p, r, rows);
    }
    const int cost = rq.units + SETUP;
    const long long item = (pos - r_start) / cost;
    s.rq = rq;
    s.r = r;
    s.start = r_start + item * cost;
    s.end = s.start + cost;
    s.tile = (int)(item / p.Hkv);
    s.h = (int)(item % p.Hkv);
    const int from = (int)(pos - s.start), to = (int)(w1 < s.end ? w1 - s.start : cost);
    if (to <= SETUP) return false;              // the boundary moves to the item's start
    s.u0 = from < SETUP ? 0 : from - SETUP;
    s.u1 = to - SETUP;
    pos = s.start + to;
    return true;
  }
};

// The blocks that share a cut item: the first boundary inside it belongs to
// block `first`, so the parts are those of first - 1 (its second slot) and of
// first ... last (their first slots).
template <int SETUP>
__device__ __forceinline__ void sharers(const Range &g, const Segment &s, long long &first, long long &last) {
  first = ((s.start + SETUP + 1) * g.n_blk + g.total - 1) / g.total;
  last = (s.end * g.n_blk + g.total - 1) / g.total - 1;
}

// Pages of a request (or of its list): block e, its page or -1.  Blocks without
// tokens have none; block and page numbers out of range are recorded.
struct Pages {
  const int *table, *sel;
  int n, kv, max_blocks, n_pages;
  int *dev_status;
  // record: whether this thread records a count out of range (which counts as the
  // nearest that is in range)
  __device__ __forceinline__ Pages(const Params &p, const Segment &s, bool record) {
    table = p.block_table + (size_t)s.r * p.max_blocks;
    kv = s.rq.kv;
    max_blocks = p.max_blocks;
    n_pages = p.n_pages;
    dev_status = p.dev_status;
    sel = nullptr;
    n = (kv + kPage - 1) / kPage;
    if (p.sel) {
      const size_t at = (size_t)s.r * p.Hkv + s.h;
      sel = p.sel + at * p.max_sel;
      const int count = __ldg(p.sel_count + at);
      n = max(0, min(p.max_sel, count));
      if (record && count != n) set_status(dev_status, DITANGO_ERR_BOUNDS);
    }
  }
  __device__ __forceinline__ int page(int e, int &block, bool record) const {
    block = -1;
    if (e >= n) return -1;
    block = sel ? __ldg(sel + e) : e;
    bool bad = block < 0 || block >= max_blocks;
    if (!bad) {
      if (block * kPage >= kv) return -1;
      const int q = __ldg(table + block);
      if (q >= 0 && q < n_pages) return q;
      bad = true;
    }
    if (record) set_status(dev_status, DITANGO_ERR_BOUNDS);
    return -1;
  }
};

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Two codes a register: codes i and i + 4 of a word, i = 0..3, less 8, as fp16.
// Codes in bits 0-3 of a half go into the significand of 1024 (1024 + c), those
// in bits 4-7 into that of 64 (64 + c): one shift serves four codes, one LOP3
// and one addition two.  The masks and exponents are kept in registers that the
// compiler cannot form again at each use: as literals they cost one more
// instruction a pair, a third of the loop.
struct Unpack {
  uint32_t mask0, mask1, exp0, exp1;
  __device__ __forceinline__ Unpack() {
    asm volatile("mov.b32 %0, 0x000f000f;" : "=r"(mask0));
    asm volatile("mov.b32 %0, 0x00f000f0;" : "=r"(mask1));
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(exp0));
    asm volatile("mov.b32 %0, 0x54005400;" : "=r"(exp1));
  }
  __device__ __forceinline__ void operator()(uint32_t w, uint32_t (&pair)[4]) const {
    const uint32_t k1032 = 0xe408e408u, k72 = 0xd480d480u;   // -1032, -72
    const uint32_t v = w >> 8;
    pair[0] = hadd2(pick(w, mask0, exp0), k1032);
    pair[1] = hadd2(pick(w, mask1, exp1), k72);
    pair[2] = hadd2(pick(v, mask0, exp0), k1032);
    pair[3] = hadd2(pick(v, mask1, exp1), k72);
  }
  static __device__ __forceinline__ uint32_t pick(uint32_t w, uint32_t mask, uint32_t exp) {   // (w & mask) | exp
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(w), "r"(mask), "r"(exp));
    return r;
  }
};

// The factor of a row's scores.  A row of zeros (or a tiny scale) takes it below
// the least fp32 number, and 0 times the -inf of a masked score would be NaN: it
// stays positive.  What it multiplies is then below 2^136, so that a score that
// should be 0 comes out below 2^-12.  A factor past fp32 stays finite likewise.
__device__ __forceinline__ float score_factor(float x) {
  return fminf(fmaxf(x, __uint_as_float(1u)), __uint_as_float(0x7f7fffffu));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Eight values of a row of Q (16 bytes) times `down`, paired as Unpack pairs codes.
__device__ __forceinline__ void q_pairs(const uint4 &u, float down, uint32_t (&pair)[4], float &sum) {
  const float f0 = bf_lo(u.x) * down, f1 = bf_hi(u.x) * down, f2 = bf_lo(u.y) * down, f3 = bf_hi(u.y) * down;
  const float f4 = bf_lo(u.z) * down, f5 = bf_hi(u.z) * down, f6 = bf_lo(u.w) * down, f7 = bf_hi(u.w) * down;
  sum += ((f0 + f1) + (f2 + f3)) + ((f4 + f5) + (f6 + f7));
  pair[0] = pack_f16x2(f0, f4);
  pair[1] = pack_f16x2(f1, f5);
  pair[2] = pack_f16x2(f2, f6);
  pair[3] = pack_f16x2(f3, f7);
}

__device__ __forceinline__ float max_abs8(const uint4 &u) {
  const uint32_t v[4] = {u.x, u.y, u.z, u.w};
  float big = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) big = fmaxf(big, fmaxf(fabsf(bf_lo(v[e])), fabsf(bf_hi(v[e]))));
  return big;
}

}  // namespace hattn

cudaError_t launch_kv4_chunk(const hattn::Params &p, int d, int num_sms, cudaStream_t stream);
size_t kv4_chunk_partial_floats(int d);
int kv4_chunk_counters();
int kv4_chunk_words();

}  // namespace ditango
