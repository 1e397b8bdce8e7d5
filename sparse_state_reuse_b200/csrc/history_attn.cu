// Attention of few query rows over the paged 4-bit history.
//
// For request r, key head h and row (token, query head of the group):
//   k_j = s_j c_j + m_j  =>  q.k_j = s_j (q.c_j) + m_j sum(q)
//   O = sum_j p_j v_j    =   sum_j (p_j s'_j) c'_j + sum_j p_j m'_j
// so that the 4-bit codes enter the tensor core as they are: a code c is put
// into the significand of a bf16 number, 1 + c/16, by a shift and one LOP3 for
// two codes (exact), and scale and least value are applied to whole rows of
// scores and to the probabilities in fp32.  Of the values that are rounded
// only the probabilities times the V scale are (to bf16, as everywhere in the
// library); the part that the added 1 contributes is taken out again with the
// same rounded values, so that it cancels.
//
// It is bound by the history's bytes: d + 8 a key and key head.  Each warp is
// by itself: it takes every fourth page of its block's range, fetches a page
// of one head (one contiguous run) with one bulk copy into a ring of its own
// and runs m16n8k16 products over it, 16 rows a tile; no block-wide barrier
// until the end of a range.  The tile has 16 rows because a few rows are all
// there is; with so few the legacy tensor instructions already outrun the
// memory, and a tcgen05 tile of 128 rows would be mostly padding.
//
// Work split: the pages of all (request, key head, row tile) items are one
// line of work that is cut into equal ranges, one a block, so that a single
// long request and a ragged batch fill the GPU alike.  An item cut by a
// boundary is joined by the block that finishes it last, from the partial
// states in block order (a fixed order: the result does not depend on which
// block is last).
#include <mutex>
#include <set>
#include <utility>

#include "blocks.cuh"

namespace ditango {
namespace hattn {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;            // rows of a tile, at most
constexpr int kMaxBlocks = 512;      // most blocks of a launch (the workspace has room for them)
constexpr float kRescaleLog2 = 8.0f;

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
  float *partial;                    // [2 * kMaxBlocks][kRows * (d + 2)]
  int *counters;                     // [kMaxBlocks]
  int max_rows;                      // requests of more rows are left to the other kernel
  int *dev_status;
  long long wait_limit_ns;
};

// Key of column n of an 8-key tile.  The order within a tile is free (scores
// and values use the same); this one spreads the rows that a warp reads at
// once over the shared-memory banks.
__device__ __forceinline__ int key_of(int n) { return n ^ ((n >> 1) & 1); }

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Codes i and i + 4 of a word (i = 0..3) as the bf16 pair 1 + c/16.
template <int I>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
  const uint32_t x = (I == 0) ? (w << 3) : (w >> (4 * I - 3));
  return (x & 0x00780078u) | 0x3f803f80u;
}

struct Request {
  int n_q, kv, q0, tiles, pages;   // pages: work units of one item, at least 1
};

template <int TR>
__device__ __forceinline__ Request request_of(const Params &p, int r) {
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
  q.tiles = rows > p.max_rows ? 0 : (int)((rows + TR - 1) / TR);
  q.pages = p.sel ? p.max_sel : (q.kv + kPage - 1) / kPage;
  if (q.pages < 1) q.pages = 1;
  return q;
}

__device__ __forceinline__ long long work_of(const Params &p, const Request &q) {
  return (long long)q.tiles * p.Hkv * q.pages;
}

// Sum and exclusive prefix over the block.
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
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sm[w];
    total += sm[w];
  }
  return before + x - v;
}

template <int D, int NS>
struct Smem {
  static constexpr int kStage = page_bytes(D);
  static constexpr int kWarpBytes = NS * kStage;
  static constexpr int kMergeStride = D + 4;     // floats of a merged row: O, then m and l
  static constexpr int kBytes = kWarps * kWarpBytes;
  static_assert(kRows * kMergeStride * 4 <= kWarpBytes, "the join reuses the ring");
  static_assert(kStage % 16 == 0, "bulk copies");
};

// LOW: tiles of 8 rows (the upper half of each product is padding).
template <int D, bool LOW, int NS>
__global__ void __launch_bounds__(kThreads) kv4_attn_kernel(const __grid_constant__ Params p) {
  using S = Smem<D, NS>;
  constexpr int W = D / 32;          // words of K codes of a lane and key
  constexpr int NT = D / 8;          // channel tiles of O
  constexpr int NR = LOW ? 1 : 2;    // rows of a lane
  constexpr int TR = 8 * NR;         // rows of a tile
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) unsigned long long bars[kWarps][NS];
  __shared__ long long s_scan[kWarps], s_before;
  __shared__ int s_request, s_abort, s_last;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t = lane & 3, n8 = lane >> 2;
  WaitCtl ctl{&s_abort, p.dev_status, p.wait_limit_ns};

  if (tid < kWarps * NS) mbar_init(smem_u32(&bars[0][0]) + 8 * tid, 1);
  if (tid == 0) {
    s_abort = 0;
    s_request = -1;
    fence_barrier_init();
  }

  // this block's range [w0, w1) of the line of work
  long long total = 0;
  for (int base = 0; base < p.R; base += kThreads) {
    const int r = base + tid;
    long long sum;
    block_scan(r < p.R ? work_of(p, request_of<TR>(p, r)) : 0, sum, s_scan);
    total += sum;
  }
  const long long n_blk = total < (long long)gridDim.x ? total : (long long)gridDim.x;
  if ((long long)blockIdx.x >= n_blk) return;
  const long long w0 = total * blockIdx.x / n_blk, w1 = total * (blockIdx.x + 1) / n_blk;
  {
    long long before = 0;
    for (int base = 0; base < p.R; base += kThreads) {
      const int r = base + tid;
      const long long v = r < p.R ? work_of(p, request_of<TR>(p, r)) : 0;
      long long sum;
      const long long at = before + block_scan(v, sum, s_scan);
      if (v > 0 && at <= w0 && w0 < at + v) {
        s_request = r;
        s_before = at;
      }
      before += sum;
      if (before > w0) break;       // uniform: every thread has the same sum
    }
    __syncthreads();
  }
  int r = s_request;
  long long r_start = s_before;
  if (r < 0) return;                // cannot happen: w0 < total
  Request rq = request_of<TR>(p, r);

  uint8_t *ring = smem + warp * S::kWarpBytes;
  const uint32_t ring_s = smem_u32(ring);
  const uint32_t bar0 = smem_u32(&bars[warp][0]);
  uint32_t it = 0;                  // pages this warp has consumed (ring position and phase)
  bool ok = true;

  for (long long pos = w0; pos < w1;) {
    while (pos >= r_start + work_of(p, rq)) {
      r_start += work_of(p, rq);
      ++r;
      rq = request_of<TR>(p, r);
    }
    // the segment: pages [p0, p1) of one item
    const long long item = (pos - r_start) / rq.pages;
    const long long item_start = r_start + item * rq.pages;
    const int p0 = (int)(pos - item_start);
    const int p1 = (int)(w1 - item_start < rq.pages ? w1 - item_start : rq.pages);
    const int tile = (int)(item / p.Hkv), h = (int)(item % p.Hkv);
    const int row0 = tile * TR;
    const int rows = min(TR, rq.n_q * p.G - row0);
    const int *table = p.block_table + (size_t)r * p.max_blocks;
    const int *sel = p.sel ? p.sel + ((size_t)r * p.Hkv + h) * p.max_sel : nullptr;
    const int n_list = sel ? max(0, min(p.max_sel, __ldg(p.sel_count + (size_t)r * p.Hkv + h)))
                           : (rq.kv + kPage - 1) / kPage;
    const int end = min(p1, n_list);

    // Q of the lane's rows, in the order in which code_pair gives the codes
    uint32_t qa[2 * W][4];
    float qsum[NR];
    int vis[NR];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int row = n8 + 8 * x;
      float sum = 0.f;
      const bool live = (x < NR) && row < rows;
      const int tok = live ? (row0 + row) / p.G : 0, head = live ? (row0 + row) % p.G : 0;
      const uint16_t *src = p.Q + (rq.q0 + tok) * p.qt + (h * p.G + head) * p.qh + t * (D / 4);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (live) u = __ldg(reinterpret_cast<const uint4 *>(src) + w);
        qa[2 * w][x] = __byte_perm(u.x, u.z, 0x5410);
        qa[2 * w][2 + x] = __byte_perm(u.x, u.z, 0x7632);
        qa[2 * w + 1][x] = __byte_perm(u.y, u.w, 0x5410);
        qa[2 * w + 1][2 + x] = __byte_perm(u.y, u.w, 0x7632);
        sum += ((bf_lo(u.x) + bf_hi(u.x)) + (bf_lo(u.y) + bf_hi(u.y))) +
               ((bf_lo(u.z) + bf_hi(u.z)) + (bf_lo(u.w) + bf_hi(u.w)));
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      if (x < NR) {
        qsum[x] = sum;
        vis[x] = p.causal && live ? rq.kv - (rq.n_q - 1 - tok) : rq.kv;
      }
    }
    // keys that every row of the tile sees
    const int vis_all = p.causal ? rq.kv - (rq.n_q - 1 - row0 / p.G) : rq.kv;

    float o[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    float m[NR], l[NR], z[NR];      // running maximum; lane's sums of p, and of p least - p'
#pragma unroll
    for (int x = 0; x < NR; ++x) {
      m[x] = -INFINITY;
      l[x] = z[x] = 0.f;
    }

    auto issue = [&](uint32_t at, int page) {
      if (lane == 0 && page >= 0) {
        const uint32_t bar = bar0 + 8 * (at % NS);
        mbar_arrive_expect_tx(bar, S::kStage);
        bulk_load(ring_s + (at % NS) * S::kStage, p.data + ((size_t)page * p.Hkv + h) * S::kStage,
                  S::kStage, bar);
      }
    };
    // The next page of this warp and its block, -1 at the end.  Blocks without
    // tokens are passed over, block and page numbers out of range recorded.
    auto next_page = [&](int &i, int &blk) -> int {
      while (i < end) {
        blk = sel ? __ldg(sel + i) : i;
        i += kWarps;
        bool bad = blk < 0 || blk >= p.max_blocks;
        if (!bad && blk * kPage < rq.kv) {
          const int page = __ldg(table + blk);
          if (page >= 0 && page < p.n_pages) return page;
          bad = true;
        }
        if (bad && lane == 0) set_status(p.dev_status, DITANGO_ERR_BOUNDS);
      }
      return -1;
    };
    int li = p0 + warp;
    int blk[NS];                    // blocks in flight, oldest first; -1: none
    uint32_t issued = it;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      blk[s] = -1;
      int b = -1;
      const int page = next_page(li, b);
      if (page >= 0) {
        blk[s] = b;
        issue(issued++, page);
      }
    }
    while (blk[0] >= 0) {
      // the next page's number is read under this page's work
      int nb = -1;
      const int npage = next_page(li, nb);
      if (!(ok = wait_warp(bar0 + 8 * (it % NS), (it / NS) & 1, ctl))) break;
      const uint8_t *st = ring + (it % NS) * S::kStage;
      const int k_base = blk[0] * kPage;
      const bool masked = k_base + kPage > vis_all;

      // scores of 64 keys: x = log2(e) scale (s 16 acc + (m - 16 s) sum q)
      float sc[8][2 * NR];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        const uint8_t *kr = st + (8 * u + key_of(n8)) * (D / 2) + t * (D / 8);
        uint32_t kw[W];
        if constexpr (W == 4) {
          const uint4 v = *reinterpret_cast<const uint4 *>(kr);
          kw[0] = v.x; kw[1] = v.y; kw[2] = v.z; kw[3] = v.w;
        } else if constexpr (W == 2) {
          const uint2 v = *reinterpret_cast<const uint2 *>(kr);
          kw[0] = v.x; kw[1] = v.y;
        } else {
#pragma unroll
          for (int w = 0; w < W; ++w) kw[w] = *reinterpret_cast<const uint32_t *>(kr + 4 * w);
        }
#pragma unroll
        for (int w = 0; w < W; ++w) {
          mma16816(acc, qa[2 * w], code_pair<0>(kw[w]), code_pair<1>(kw[w]));
          mma16816(acc, qa[2 * w + 1], code_pair<2>(kw[w]), code_pair<3>(kw[w]));
        }
        // columns 2t and 2t + 1 are keys 2t and 2t + 1, exchanged where t is odd
        const uint2 mt = *reinterpret_cast<const uint2 *>(st + kPage * D + (8 * u + 2 * t) * 4);
        const uint32_t m0 = (t & 1) ? mt.y : mt.x, m1 = (t & 1) ? mt.x : mt.y;
        const float a0 = bf_lo(m0) * (16.f * p.scale_log2), a1 = bf_lo(m1) * (16.f * p.scale_log2);
        const float b0 = fmaf(bf_hi(m0), p.scale_log2, -a0), b1 = fmaf(bf_hi(m1), p.scale_log2, -a1);
#pragma unroll
        for (int x = 0; x < NR; ++x) {
          sc[u][2 * x] = fmaf(acc[2 * x], a0, b0 * qsum[x]);
          sc[u][2 * x + 1] = fmaf(acc[2 * x + 1], a1, b1 * qsum[x]);
        }
      }
      if (masked) {
#pragma unroll
        for (int u = 0; u < 8; ++u)
#pragma unroll
          for (int e = 0; e < 2 * NR; ++e) {
            const int key = k_base + 8 * u + key_of(2 * t + (e & 1));
            if (key >= vis[e >> 1]) sc[u][e] = -INFINITY;
          }
      }
      // running maximum; O is rescaled only when it grew by more than 2^8
      bool need = false;
      float mx[NR];
#pragma unroll
      for (int x = 0; x < NR; ++x) {
        float v = -INFINITY;
#pragma unroll
        for (int u = 0; u < 8; ++u) v = fmaxf(v, fmaxf(sc[u][2 * x], sc[u][2 * x + 1]));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
        mx[x] = v;
        need = need || v > m[x] + kRescaleLog2;
      }
      if (__any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int x = 0; x < NR; ++x) {
          const float mn = fmaxf(m[x], mx[x]);
          const float al = m[x] == mn ? 1.f : fast_ex2(m[x] - mn);
          m[x] = mn;
          l[x] *= al;
          z[x] *= al;
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            o[j][2 * x] *= al;
            o[j][2 * x + 1] *= al;
          }
        }
      }
      // 16 keys at a time: p, then p times the V scale, rounded, and the products
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        uint32_t pa[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int u = 2 * v + g;
          const uint2 mt = *reinterpret_cast<const uint2 *>(st + kPage * D + kPage * 4 + (8 * u + 2 * t) * 4);
          const uint32_t m0 = (t & 1) ? mt.y : mt.x, m1 = (t & 1) ? mt.x : mt.y;
          const float s0 = 16.f * bf_lo(m0), s1 = 16.f * bf_lo(m1), h0 = bf_hi(m0), h1 = bf_hi(m1);
#pragma unroll
          for (int x = 0; x < NR; ++x) {
            const float neg = m[x] > -INFINITY ? -m[x] : 0.f;
            const float e0 = fast_ex2(sc[u][2 * x] + neg), e1 = fast_ex2(sc[u][2 * x + 1] + neg);
            l[x] += e0 + e1;
            float w0_ = e0 * s0, w1_ = e1 * s1, c0 = e0 * h0, c1 = e1 * h1;
            if (masked) {           // a masked token's scale may be anything
              const int kb = k_base + 8 * u;
              if (kb + key_of(2 * t) >= vis[x]) w0_ = c0 = 0.f;
              if (kb + key_of(2 * t + 1) >= vis[x]) w1_ = c1 = 0.f;
            }
            const uint32_t pk = pack_bf16x2(w0_, w1_);
            pa[2 * g + x] = pk;
            z[x] += (c0 - bf_lo(pk)) + (c1 - bf_hi(pk));
          }
        }
        const uint8_t *vr = st + kPage * (D / 2);
        const uint8_t *r0p = vr + (16 * v + key_of(2 * t)) * (D / 2);
        const uint8_t *r1p = vr + (16 * v + key_of(2 * t + 1)) * (D / 2);
#pragma unroll
        for (int w = 0; w < D / 64; ++w) {
          const int at = 32 * w + 4 * n8;
          const uint32_t ka = *reinterpret_cast<const uint32_t *>(r0p + at);
          const uint32_t kb = *reinterpret_cast<const uint32_t *>(r1p + at);
          const uint32_t kc = *reinterpret_cast<const uint32_t *>(r0p + 8 * (D / 2) + at);
          const uint32_t kd = *reinterpret_cast<const uint32_t *>(r1p + 8 * (D / 2) + at);
          const uint32_t xl = __byte_perm(ka, kb, 0x5410), xh = __byte_perm(ka, kb, 0x7632);
          const uint32_t yl = __byte_perm(kc, kd, 0x5410), yh = __byte_perm(kc, kd, 0x7632);
          mma16816(o[8 * w + 0], pa, code_pair<0>(xl), code_pair<0>(yl));
          mma16816(o[8 * w + 1], pa, code_pair<1>(xl), code_pair<1>(yl));
          mma16816(o[8 * w + 2], pa, code_pair<2>(xl), code_pair<2>(yl));
          mma16816(o[8 * w + 3], pa, code_pair<3>(xl), code_pair<3>(yl));
          mma16816(o[8 * w + 4], pa, code_pair<0>(xh), code_pair<0>(yh));
          mma16816(o[8 * w + 5], pa, code_pair<1>(xh), code_pair<1>(yh));
          mma16816(o[8 * w + 6], pa, code_pair<2>(xh), code_pair<2>(yh));
          mma16816(o[8 * w + 7], pa, code_pair<3>(xh), code_pair<3>(yh));
        }
        if constexpr (D % 64 != 0) {   // d = 96: the last 32 channels, four a lane
          const int at = 32 * (D / 64) + 2 * n8;
          const uint32_t ka = *reinterpret_cast<const uint16_t *>(r0p + at);
          const uint32_t kb = *reinterpret_cast<const uint16_t *>(r1p + at);
          const uint32_t kc = *reinterpret_cast<const uint16_t *>(r0p + 8 * (D / 2) + at);
          const uint32_t kd = *reinterpret_cast<const uint16_t *>(r1p + 8 * (D / 2) + at);
          const uint32_t xl = __byte_perm(ka, kb, 0x5410), yl = __byte_perm(kc, kd, 0x5410);
          mma16816(o[NT - 4], pa, code_pair<0>(xl), code_pair<0>(yl));
          mma16816(o[NT - 3], pa, code_pair<1>(xl), code_pair<1>(yl));
          mma16816(o[NT - 2], pa, code_pair<2>(xl), code_pair<2>(yl));
          mma16816(o[NT - 1], pa, code_pair<3>(xl), code_pair<3>(yl));
        }
      }
      ++it;
      __syncwarp();                 // every lane has read the page
#pragma unroll
      for (int s = 0; s + 1 < NS; ++s) blk[s] = blk[s + 1];
      blk[NS - 1] = -1;
      if (npage >= 0) {
        // the free places are taken in order: the oldest -1
        bool put = false;
#pragma unroll
        for (int s = 0; s < NS; ++s)
          if (!put && blk[s] < 0) {
            blk[s] = nb;
            put = true;
          }
        issue(issued++, npage);
      }
    }
    if (!ok) {
      // gave up: wait, with a limit, for the copies in flight before leaving
      volatile int never = 0;
      WaitCtl drain{&never, nullptr, 100000000LL};
      for (uint32_t q = it; q < issued; ++q) wait_bounded(bar0 + 8 * (q % NS), (q / NS) & 1, drain);
    }
    // ---- join the four warps: O + z, m, l of each row into the ring
    __syncthreads();
    if (s_abort) return;            // uniform after the barrier: a wait gave up
    float *mg = reinterpret_cast<float *>(ring);
#pragma unroll
    for (int x = 0; x < NR; ++x) {
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
      z[x] += __shfl_xor_sync(0xffffffffu, z[x], 1);
      z[x] += __shfl_xor_sync(0xffffffffu, z[x], 2);
      float *row = mg + (n8 + 8 * x) * S::kMergeStride;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int n = 2 * t + e;
#pragma unroll
        for (int w = 0; w < D / 64; ++w)
#pragma unroll
          for (int j = 0; j < 8; j += 4)
            *reinterpret_cast<float4 *>(row + 64 * w + 8 * n + j) =
                make_float4(o[8 * w + j][2 * x + e] + z[x], o[8 * w + j + 1][2 * x + e] + z[x],
                            o[8 * w + j + 2][2 * x + e] + z[x], o[8 * w + j + 3][2 * x + e] + z[x]);
        if constexpr (D % 64 != 0)
          *reinterpret_cast<float4 *>(row + 64 * (D / 64) + 4 * n) =
              make_float4(o[NT - 4][2 * x + e] + z[x], o[NT - 3][2 * x + e] + z[x],
                          o[NT - 2][2 * x + e] + z[x], o[NT - 1][2 * x + e] + z[x]);
      }
      if (t == 0) {
        row[D] = m[x];
        row[D + 1] = l[x];
      }
    }
    __syncthreads();

    auto store = [&](int row, int ch, float4 v, float mt_, float lt_) {
      const int tok = rq.q0 + (row0 + row) / p.G, head = h * p.G + (row0 + row) % p.G;
      const float inv = lt_ > 0.f ? 1.f / lt_ : 0.f;
      if (!(lt_ > 0.f) && lt_ == lt_) v = make_float4(0.f, 0.f, 0.f, 0.f);   // a row that sees no key
      else v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
      if (lt_ != lt_) v = make_float4(lt_, lt_, lt_, lt_);
      if (p.out_fp32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + tok * p.ot + head * p.oh + ch) = v;
      } else {
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + tok * p.ot + head * p.oh + ch) =
            make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
      }
      if (ch == 0 && p.out_lse)
        p.out_lse[tok * p.lt + head * p.lh] =
            lt_ > 0.f ? (mt_ + log2f(lt_)) * 0.69314718055994531f : (lt_ == lt_ ? -INFINITY : lt_);
    };
    // O, m and l of a row and four channels from the four warps
    auto joined = [&](int row, int ch, float &mt_, float &lt_) -> float4 {
      float mm[kWarps];
      mt_ = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        mm[w] = (reinterpret_cast<const float *>(smem + w * S::kWarpBytes) + row * S::kMergeStride)[D];
        mt_ = fmaxf(mt_, mm[w]);
      }
      const float sub = mt_ > -INFINITY ? mt_ : 0.f;
      lt_ = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float *src = reinterpret_cast<const float *>(smem + w * S::kWarpBytes) + row * S::kMergeStride;
        const float f = fast_ex2(mm[w] - sub);
        const float4 a = *reinterpret_cast<const float4 *>(src + ch);
        lt_ = fmaf(src[D + 1], f, lt_);
        v.x = fmaf(a.x, f, v.x);
        v.y = fmaf(a.y, f, v.y);
        v.z = fmaf(a.z, f, v.z);
        v.w = fmaf(a.w, f, v.w);
      }
      return v;
    };
    const bool whole = p0 == 0 && p1 == rq.pages;
    constexpr int kVec = D / 4;
    if (whole) {
      for (int i = tid; i < rows * kVec; i += kThreads) {
        float mt_, lt_;
        const float4 v = joined(i / kVec, (i % kVec) * 4, mt_, lt_);
        store(i / kVec, (i % kVec) * 4, v, mt_, lt_);
      }
    } else {
      // a part: the block whose range begins inside the item uses its first
      // slot, the one in whose range the item begins its second
      constexpr int kSlot = kRows * (D + 2);
      float *mine = p.partial + ((size_t)blockIdx.x * 2 + (p0 == 0 ? 1 : 0)) * kSlot;
      for (int i = tid; i < rows * kVec; i += kThreads) {
        const int row = i / kVec, ch = (i % kVec) * 4;
        float mt_, lt_;
        const float4 v = joined(row, ch, mt_, lt_);
        float *dst = mine + row * (D + 2) + ch;
        *reinterpret_cast<float2 *>(dst) = make_float2(v.x, v.y);
        *reinterpret_cast<float2 *>(dst + 2) = make_float2(v.z, v.w);
        if (ch == 0) {
          mine[row * (D + 2) + D] = mt_;
          mine[row * (D + 2) + D + 1] = lt_;
        }
      }
      // first block boundary inside the item, and the last block that shares it
      const long long iend = item_start + rq.pages;
      const long long c1 = ((item_start + 1) * n_blk + total - 1) / total;
      const long long cl = (iend * n_blk + total - 1) / total - 1;
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const int before = atomicAdd(p.counters + c1, 1);
        s_last = before == (int)(cl - c1 + 1);
        if (s_last) p.counters[c1] = 0;     // left at zero for the next launch
      }
      __syncthreads();
      if (s_last) {
        __threadfence();
        for (int i = tid; i < rows * kVec; i += kThreads) {
          const int row = i / kVec, ch = (i % kVec) * 4;
          float mt_ = -INFINITY, lt_ = 0.f;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          for (long long c = c1 - 1; c <= cl; ++c) {
            const float *src = p.partial + (c * 2 + (c == c1 - 1 ? 1 : 0)) * kSlot + row * (D + 2);
            const float pm = __ldcg(src + D), pl = __ldcg(src + D + 1);
            const float2 a = __ldcg(reinterpret_cast<const float2 *>(src + ch));
            const float2 b = __ldcg(reinterpret_cast<const float2 *>(src + ch + 2));
            const float mn = fmaxf(mt_, pm);
            const float sub = mn > -INFINITY ? mn : 0.f;
            const float f0 = fast_ex2(mt_ - sub), f1 = fast_ex2(pm - sub);
            lt_ = lt_ * f0 + pl * f1;
            v = make_float4(v.x * f0 + a.x * f1, v.y * f0 + a.y * f1, v.z * f0 + b.x * f1, v.w * f0 + b.y * f1);
            mt_ = mn;
          }
          store(row, ch, v, mt_, lt_);
        }
      }
    }
    fence_proxy_async();            // the ring was written by stores; copies follow
    __syncthreads();
    pos = item_start + p1;
  }
}

template <int D, bool LOW>
cudaError_t launch(const Params &p, int num_sms, cudaStream_t stream) {
  constexpr int NS = 2;
  auto kfn = kv4_attn_kernel<D, LOW, NS>;
  constexpr int bytes = Smem<D, NS>::kBytes;
  static std::mutex mu;
  static std::set<int> ready;
  static int per_sm = 1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int blocks;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!ready.count(dev)) {
      e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
      if (e != cudaSuccess) return e;
      int n = 1;
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kfn, kThreads, bytes);
      if (e != cudaSuccess) return e;
      per_sm = n < 1 ? 1 : n;
      ready.insert(dev);
    }
    blocks = per_sm * num_sms;
  }
  if (blocks > kMaxBlocks) blocks = kMaxBlocks;
  kfn<<<blocks, kThreads, bytes, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace hattn

size_t kv4_attn_workspace_bytes(int d) {
  return (size_t)hattn::kMaxBlocks * (2 * hattn::kRows * (size_t)(d + 2) * sizeof(float) + sizeof(int));
}

cudaError_t launch_kv4_attn(int R, int H, int Hkv, int d, int T, int max_q, int max_blocks, int n_pages,
                            const uint16_t *Q, const int64_t *q_strides, const int *q_off, const int *kv_len,
                            const int *block_table, const uint8_t *data, const int *sel, const int *sel_count,
                            int max_sel, float scale, int causal, void *out, int out_fp32,
                            const int64_t *out_strides, float *out_lse, const int64_t *lse_strides,
                            void *workspace, int *dev_status, long long wait_limit_ns, int num_sms,
                            cudaStream_t stream) {
  hattn::Params p;
  p.R = R;
  p.H = H;
  p.Hkv = Hkv;
  p.G = H / Hkv;
  p.T = T;
  p.max_blocks = max_blocks;
  p.n_pages = n_pages;
  p.max_sel = max_sel;
  p.causal = causal;
  p.Q = Q;
  p.qt = q_strides[0];
  p.qh = q_strides[1];
  p.q_off = q_off;
  p.kv_len = kv_len;
  p.block_table = block_table;
  p.sel = sel;
  p.sel_count = sel_count;
  p.data = data;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.out = out;
  p.out_fp32 = out_fp32;
  p.ot = out_strides[0];
  p.oh = out_strides[1];
  p.out_lse = out_lse;
  p.lt = lse_strides[0];
  p.lh = lse_strides[1];
  p.partial = static_cast<float *>(workspace);
  p.counters = reinterpret_cast<int *>(p.partial + (size_t)hattn::kMaxBlocks * 2 * hattn::kRows * (d + 2));
  p.max_rows = 0x7fffffff;
  p.dev_status = dev_status;
  p.wait_limit_ns = wait_limit_ns;
  const bool low = (long long)max_q * p.G <= 8;
  switch (d) {
#define DITANGO_KV4(D)                                                                     \
  case D:                                                                                  \
    return low ? hattn::launch<D, true>(p, num_sms, stream) : hattn::launch<D, false>(p, num_sms, stream)
    DITANGO_KV4(64);
    DITANGO_KV4(96);
    DITANGO_KV4(128);
#undef DITANGO_KV4
    default:
      return cudaErrorInvalidValue;
  }
}

}  // namespace ditango
