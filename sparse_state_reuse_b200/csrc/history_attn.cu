// Attention of few query rows over the paged 4-bit history.
//
// For request r, key head h and row (token, query head of the group), with the
// codes taken around the middle, k_j = s_j (c_j - 8) + h_j, h_j = m_j + 8 s_j:
//   q.k_j = s_j (q.(c_j - 8)) + h_j sum(q)
//   O     = sum_j (p_j s'_j) (c'_j - 8) + sum_j p_j h'_j
// so that the 4-bit codes enter the tensor core as they are.  Two codes become
// a pair of fp16 numbers by one LOP3 and one packed addition that leaves c - 8,
// exactly; scales and h are applied to scores and probabilities in fp32.  fp16 and not
// bf16: its longer significand takes two codes in place, and it rounds p s' to
// 2^-11.  Q is scaled by a power of two a row to lie below 2 (an exact step for
// all but values 2^-24 of the row's largest), p s' by one of the row's own: 2^6
// over the largest V scale met so far, as long as the scales that the warp meets
// are of one size.  Where they are not (those of a page are 2^8 and more apart, or
// its largest is above what the row is held to, or 2^6 below it), the row is held to
// the weights that it has itself, so that neither a key that it does not see nor one
// whose probability is nothing pushes the others out of fp16.
//
// Keys and channels are the rows of the products (m16n8k16, S^T = K Q^T and
// O^T = V^T P^T) and query rows their 8 columns: 8 rows at a time, of which a
// decode step has few.  A lane holds two neighbouring columns; up to four rows
// take every other column, so that a lane exponentiates one.  P^T goes from the first product's layout to the
// second's by a transpose of 8x8 tiles in registers.
//
// It is bound by the history's bytes, d + 8 a key and key head, as long as the
// instructions that unpack them keep up.  Each warp is by itself: it takes
// every fourth page of its block's range and fetches each page of one head (one
// contiguous run) with one bulk copy into one of two places of its own; no
// block-wide barrier until the end of a range.  (K and V fetched apart, with
// their scales, are four copies a page: 10% slower.)  With so few rows the
// legacy tensor instructions are not what bounds it (30% of their rate), and a
// tcgen05 tile of 128 rows would be mostly padding.
//
// One token over 86400 of 24 heads of 96: 58 us, 3.7 TB/s (57% of the copy rate);
// the copies alone, without arithmetic, 44 us.  48 requests of 1 to 16000 tokens, 8
// key heads of 128: 108 us (the copies alone 76 us).  The first page lands 7.7 us
// after the start (lengths, page numbers and the copy follow one another), and the
// join of the parts takes the last 4 us.  Reading Q before the pages, which shortens
// its own wait, delays the copies as much (59 us).

#include "history_attn.cuh"

namespace ditango {
namespace hattn {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxBlocks = 768;      // most blocks of a launch (the workspace has room for them)
constexpr int kSetup = 8;            // pages that beginning and finishing an item counts for
// p s' in fp16: p is at most 2^8 (the lazy rescaling), s' at most the reference;
// 2^6 more uses the range that is left but for one power of two, in which the next
// pages' scales may be larger.
constexpr float kWeightScale = 64.f, kMostScale = 128.f;
constexpr float kFirstScale = 0x1p69f;   // before the first weight: 2^6 over 2^-63

// Key of row n of an 8-key tile.  The order within a tile is free (scores and
// values use the same); this one spreads the rows that a warp reads at once
// over the shared-memory banks.
__device__ __forceinline__ int key_of(int n) { return n ^ ((n >> 1) & 1); }

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8x8 tile of 16-bit values held by the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// The least power of two above x >= 0, from 2^-63 to 2^127.
__device__ __forceinline__ float power_above(float x) {
  return __uint_as_float(min(max((__float_as_uint(x) >> 23) + 1u, 64u), 254u) << 23);
}
// Of powers of two a and b: a / b, as long as that is one of 2^-126 ... 2^127 (0 below),
// without a division's code.
__device__ __forceinline__ float power_ratio(float a, float b) {
  const int bits = (int)(__float_as_uint(a) - __float_as_uint(b)) + (127 << 23);
  return __uint_as_float((uint32_t)max(bits, 0));
}

template <int D>
struct Smem {
  static constexpr int kStage = page_bytes(D);
  static constexpr int kV = kPage * D / 2;       // in a page: V's codes,
  static constexpr int kKMeta = kPage * D, kVMeta = kKMeta + kPage * 4;   // K's and V's (scale, least) pairs
  static constexpr int kMergeStride = D + 4;     // floats of a merged row: O, then m and l
  static constexpr int kMerge = kRows * kMergeStride * 4;
  static constexpr int kWarpBytes = 2 * kStage;  // two places; the join reuses them
  static constexpr int kBytes = kWarps * kWarpBytes;
  static_assert(kWarpBytes >= kMerge, "the join reuses the places");
  static_assert(kStage % 16 == 0, "bulk copies");
};

// What a warp holds of a row tile: Q as the second operand of K Q^T, O^T, and of
// its columns 2t, 2t + 1 (+ 8) the softmax state.  NR: groups of 8 columns; E:
// columns of a lane and group that hold rows (1: the even columns only).
template <int D, int NR>
struct WarpTile {
  static constexpr int W = D / 32;   // words of K codes of a lane and key
  static constexpr int MT = D / 16;  // 16-channel tiles of O^T
  uint32_t q[NR][2 * W][2];
  float o[NR][MT][4];
  float qsum[2 * NR], mul[2 * NR];   // sum of the scaled q; log2(e) scale 2^exponent
  float m[2 * NR], l[2 * NR], z[2 * NR];   // running maximum (log2), lane's sums of p and of p h'
  int vis[2 * NR];                   // keys that the row sees
  float vs[2 * NR];                  // power of two by which the row's weights p s' are multiplied
};

// Scores of the 64 keys of a page (at st) for the lane's columns, before
// the column's factor: keys 16 u + {key_of(n8), 8 + key_of(n8)}.
template <int D, int NR, int E, bool MASKED>
__device__ __forceinline__ void page_scores(const WarpTile<D, NR> &w, const Unpack &unpack8, const uint8_t *st, int k_base,
                                            float (&sc)[4][NR][4]) {
  using T = WarpTile<D, NR>;
  const int lane = threadIdx.x & 31, t = lane & 3, n8 = lane >> 2;
  const int kn = key_of(n8);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
#pragma unroll
    for (int x = 0; x < NR; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[u][x][e] = 0.f;
    const uint8_t *ra = st + (16 * u + kn) * (D / 2) + t * (D / 8), *rb = ra + 8 * (D / 2);
    uint32_t ka[T::W], kb[T::W];
    if constexpr (T::W == 4) {
      const uint4 a = *reinterpret_cast<const uint4 *>(ra), b = *reinterpret_cast<const uint4 *>(rb);
      ka[0] = a.x; ka[1] = a.y; ka[2] = a.z; ka[3] = a.w;
      kb[0] = b.x; kb[1] = b.y; kb[2] = b.z; kb[3] = b.w;
    } else if constexpr (T::W == 2) {
      const uint2 a = *reinterpret_cast<const uint2 *>(ra), b = *reinterpret_cast<const uint2 *>(rb);
      ka[0] = a.x; ka[1] = a.y;
      kb[0] = b.x; kb[1] = b.y;
    } else {
#pragma unroll
      for (int i = 0; i < T::W; ++i) {
        ka[i] = *reinterpret_cast<const uint32_t *>(ra + 4 * i);
        kb[i] = *reinterpret_cast<const uint32_t *>(rb + 4 * i);
      }
    }
#pragma unroll
    for (int i = 0; i < T::W; ++i) {
      uint32_t pa[4], pb[4];
      unpack8(ka[i], pa);
      unpack8(kb[i], pb);
#pragma unroll
      for (int x = 0; x < NR; ++x) {
        mma16816(sc[u][x], pa[0], pb[0], pa[1], pb[1], w.q[x][2 * i][0], w.q[x][2 * i][1]);
        mma16816(sc[u][x], pa[2], pb[2], pa[3], pb[3], w.q[x][2 * i + 1][0], w.q[x][2 * i + 1][1]);
      }
    }
    const uint8_t *meta = st + Smem<D>::kKMeta + (16 * u + kn) * 4;
    const uint32_t ma = *reinterpret_cast<const uint32_t *>(meta), mb = *reinterpret_cast<const uint32_t *>(meta + 32);
    const float sa = bf_lo(ma), sb = bf_lo(mb);
    const float ha = fmaf(8.f, sa, bf_hi(ma)), hb = fmaf(8.f, sb, bf_hi(mb));
#pragma unroll
    for (int x = 0; x < NR; ++x)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        sc[u][x][e] = fmaf(sc[u][x][e], sa, ha * w.qsum[2 * x + e]);
        sc[u][x][2 + e] = fmaf(sc[u][x][2 + e], sb, hb * w.qsum[2 * x + e]);
        if constexpr (MASKED) {
          const int key = k_base + 16 * u + kn;
          if (key >= w.vis[2 * x + e]) sc[u][x][e] = -INFINITY;
          if (key + 8 >= w.vis[2 * x + e]) sc[u][x][2 + e] = -INFINITY;
        }
      }
  }
}

// The softmax step and the second product of a page (at st).
template <int D, int NR, int E, bool MASKED>
__device__ __forceinline__ void page_values(WarpTile<D, NR> &w, const Unpack &unpack8, const uint8_t *st, int k_base, int kv, int vis_all,
                                            float (&sc)[4][NR][4]) {
  using T = WarpTile<D, NR>;
  const int lane = threadIdx.x & 31, t = lane & 3, n8 = lane >> 2;
  const int kn = key_of(n8);
  // running maximum; O is rescaled only when it grew by more than 2^8
  bool need = false;
  float mx[2 * NR];
#pragma unroll
  for (int x = 0; x < NR; ++x)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int y = 2 * x + e;
      float v = -INFINITY;
#pragma unroll
      for (int u = 0; u < 4; ++u) v = fmaxf(v, fmaxf(sc[u][x][e], sc[u][x][2 + e]));
      v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
      v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
      v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
      mx[y] = v * w.mul[y];
      need = need || mx[y] > w.m[y] + kRescaleLog2;
    }
  // the largest V scale of the page (rows that stand for NaN have none)
  const uint32_t *vm = reinterpret_cast<const uint32_t *>(st + Smem<D>::kVMeta);
  uint32_t sa16 = vm[lane] & 0xffffu, sb16 = vm[lane + 32] & 0xffffu;
  if constexpr (MASKED) {
    if (k_base + lane >= kv) sa16 = 0u;
    if (k_base + lane + 32 >= kv) sb16 = 0u;
  }
  if (sa16 >= 0x7f80u) sa16 = 0u;
  if (sb16 >= 0x7f80u) sb16 = 0u;
  const uint32_t top = __reduce_max_sync(0xffffffffu, max(sa16, sb16));
  const uint32_t low = __reduce_min_sync(0xffffffffu, min(sa16 ? sa16 : 0xffffu, sb16 ? sb16 : 0xffffu));
  const float top_s = __uint_as_float(top << 16);
  const bool spread = top > low + (8u << 7);        // by more than 2^8 (0 is no scale)
  bool misfit = spread, refit = false;
#pragma unroll
  for (int x = 0; x < NR; ++x)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float fit = top_s * w.vs[2 * x + e];
      misfit = misfit || fit > kMostScale || (fit < 1.f && top != 0u);
    }
  if (__any_sync(0xffffffffu, need || misfit)) {
    float vmul[2 * NR];
#pragma unroll
    for (int y = 0; y < 2 * NR; ++y) vmul[y] = 1.f;
    if (__any_sync(0xffffffffu, misfit)) {
      // scales of one size that every row sees, and within 2^6 of those before: the
      // largest holds for all rows
      const float vnew = power_ratio(kWeightScale, power_above(top_s));
      bool alike = !spread && (!MASKED || vis_all >= kv);
#pragma unroll
      for (int x = 0; x < NR; ++x)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float vs = w.vs[2 * x + e], fit = top_s * vs;
          alike = alike && fit >= 1.f && (fit <= 64.f * kWeightScale || vs == kFirstScale);
        }
      refit = __any_sync(0xffffffffu, !alike);
      if (!refit) {
#pragma unroll
        for (int x = 0; x < NR; ++x)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int y = 2 * x + e;
            if (top_s * w.vs[y] > kWeightScale) {
              vmul[y] = power_ratio(vnew, w.vs[y]);
              w.vs[y] = vnew;
            }
          }
      }
    }
#pragma unroll
    for (int x = 0; x < NR; ++x)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int y = 2 * x + e;
        const float mn = fmaxf(w.m[y], mx[y]);
        const float al = w.m[y] == mn ? 1.f : fast_ex2(w.m[y] - mn);
        w.m[y] = mn;
        w.l[y] *= al;
        w.z[y] *= al;
        const float ao = al * vmul[y];
#pragma unroll
        for (int j = 0; j < T::MT; ++j) {
          w.o[x][j][e] *= ao;
          w.o[x][j][2 + e] *= ao;
        }
      }
  }
  float neg[2 * NR], mul[2 * NR];
  bool huge = false;
#pragma unroll
  for (int x = 0; x < NR; ++x)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int y = 2 * x + e;
      neg[y] = w.m[y] > -INFINITY ? -w.m[y] : 0.f;   // no key so far: against 0
      mul[y] = w.mul[y];
      huge = huge || fabsf(neg[y]) > kHuge;
    }
  if (__any_sync(0xffffffffu, huge)) {
#pragma unroll
    for (int x = 0; x < NR; ++x)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int y = 2 * x + e;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          sc[u][x][e] = __fmul_rn(sc[u][x][e], mul[y]);
          sc[u][x][2 + e] = __fmul_rn(sc[u][x][2 + e], mul[y]);
        }
        mul[y] = 1.f;
      }
  }
  if (refit) {
    // each row by itself: the largest weight p s' that it has in this page.  2^-8
    // keeps that product finite.
#pragma unroll
    for (int x = 0; x < NR; ++x)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int y = 2 * x + e;
        float most = 0.f, big = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int key = 16 * u + kn + 8 * half;
            const float sv = bf_lo(vm[key]) * 0x1p-8f;
            const float ex = fast_ex2(fmaf(sc[u][x][2 * half + e], mul[y], neg[y]));
            if ((!MASKED || k_base + key < w.vis[y]) && sv < INFINITY) most = fmaxf(most, ex * sv);
          }
#pragma unroll
        for (int j = 0; j < T::MT; ++j) big = fmaxf(big, fmaxf(fabsf(w.o[x][j][e]), fabsf(w.o[x][j][2 + e])));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
        }
        const float old = w.vs[y];
        float vs = old, ao = 1.f;
        if (most > 0.f) {
          // that weight becomes 1/2 to 2^13, where the page's largest scale asks for
          // neither more nor less
          const float unit = 0x1p-8f / power_above(most), want = top_s > 0.f ? kWeightScale / power_above(top_s) : unit;
          vs = fminf(fminf(fmaxf(want, unit), unit * 0x1p13f), kFirstScale);
        }
        vs = fminf(vs, 0x1p126f / power_above(top_s));       // s' vs is finite where p is 0
        if (big > 0.f) {                                     // and what there is of O
          vs = fminf(vs, old * fminf(0x1p100f / power_above(big), 0x1p90f));
          ao = vs / old;
        }
        w.vs[y] = vs;
#pragma unroll
        for (int j = 0; j < T::MT; ++j) {
          w.o[x][j][e] *= ao;
          w.o[x][j][2 + e] *= ao;
        }
      }
  }
  // 16 keys at a time: p, the weights p s', and the product
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const uint8_t *meta = st + Smem<D>::kVMeta + (16 * u + kn) * 4;
    const uint32_t ma = *reinterpret_cast<const uint32_t *>(meta), mb = *reinterpret_cast<const uint32_t *>(meta + 32);
    const float sa = bf_lo(ma), sb = bf_lo(mb);
    const float ha = fmaf(8.f, sa, bf_hi(ma)), hb = fmaf(8.f, sb, bf_hi(mb));
    uint32_t pb[NR][2];
#pragma unroll
    for (int x = 0; x < NR; ++x) {
      float g[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int y = 2 * x + e, q = 2 * half + e;
          const float ex = fast_ex2(fmaf(sc[u][x][q], mul[y], neg[y]));
          g[q] = ex * ((half ? sb : sa) * w.vs[y]);
          w.l[y] += ex;
          if constexpr (MASKED) {       // a masked token's scale may be anything
            if (k_base + 16 * u + kn + 8 * half >= w.vis[y]) g[q] = 0.f;
            else w.z[y] = fmaf(ex, half ? hb : ha, w.z[y]);
          } else {
            w.z[y] = fmaf(ex, half ? hb : ha, w.z[y]);
          }
        }
      pb[x][0] = transpose8x8(pack_f16x2(g[0], g[1]));
      pb[x][1] = transpose8x8(pack_f16x2(g[2], g[3]));
    }
    // keys 2t, 2t + 1 (+ 8) of the 16, channels by lane: 8 n8 + i of each 64
    const uint8_t *r0 = st + Smem<D>::kV + (16 * u + key_of(2 * t)) * (D / 2);
    const uint8_t *r1 = st + Smem<D>::kV + (16 * u + key_of(2 * t + 1)) * (D / 2);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const int at = 32 * i + 4 * n8;
      const uint32_t a = *reinterpret_cast<const uint32_t *>(r0 + at);
      const uint32_t b = *reinterpret_cast<const uint32_t *>(r1 + at);
      const uint32_t c = *reinterpret_cast<const uint32_t *>(r0 + 8 * (D / 2) + at);
      const uint32_t d = *reinterpret_cast<const uint32_t *>(r1 + 8 * (D / 2) + at);
      uint32_t xl[4], xh[4], yl[4], yh[4];
      unpack8(__byte_perm(a, b, 0x5410), xl);
      unpack8(__byte_perm(a, b, 0x7632), xh);
      unpack8(__byte_perm(c, d, 0x5410), yl);
      unpack8(__byte_perm(c, d, 0x7632), yh);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int x = 0; x < NR; ++x)
          mma16816(w.o[x][4 * i + j], xl[j], xh[j], yl[j], yh[j], pb[x][0], pb[x][1]);
    }
    if constexpr (D % 64 != 0) {     // d = 96: the last 32 channels, 4 n8 + i
      const int at = 32 * (D / 64) + 2 * n8;
      const uint32_t a = *reinterpret_cast<const uint16_t *>(r0 + at);
      const uint32_t b = *reinterpret_cast<const uint16_t *>(r1 + at);
      const uint32_t c = *reinterpret_cast<const uint16_t *>(r0 + 8 * (D / 2) + at);
      const uint32_t d = *reinterpret_cast<const uint16_t *>(r1 + 8 * (D / 2) + at);
      uint32_t xl[4], yl[4];
      unpack8(__byte_perm(a, b, 0x5410), xl);
      unpack8(__byte_perm(c, d, 0x5410), yl);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int x = 0; x < NR; ++x)
          mma16816(w.o[x][T::MT - 2 + j], xl[2 * j], xl[2 * j + 1], yl[2 * j], yl[2 * j + 1], pb[x][0], pb[x][1]);
    }
  }
}

// NR, E: as in WarpTile.
template <int D, int NR, int E>
__global__ void __launch_bounds__(kThreads, NR == 2 ? 2 : (D == 128 ? 3 : 4)) kv4_attn_kernel(const __grid_constant__ Params p) {
  using S = Smem<D>;
  using WT = WarpTile<D, NR>;
  constexpr int W = WT::W, MT = WT::MT;
  constexpr int TR = 4 * E * NR;     // rows of a tile
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) unsigned long long bars[kWarps][2];
  __shared__ long long s_scan[kWarps + 1];
  __shared__ int s_request, s_abort, s_last;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t = lane & 3, n8 = lane >> 2;
  WaitCtl ctl{&s_abort, p.dev_status, p.wait_limit_ns};

  if (tid < kWarps * 2) mbar_init(smem_u32(&bars[0][0]) + 8 * tid, 1);
  if (tid == 0) {
    s_abort = 0;
    s_request = -1;
    fence_barrier_init();
  }

  Range g;
  if (!find_range<TR, 1, kSetup, kThreads>(p, 1, g, s_scan, &s_request)) return;

  uint8_t *place = smem + warp * S::kWarpBytes;
  const uint32_t place_s = smem_u32(place);
  auto full = [&](uint32_t n) { return smem_u32(&bars[warp][0]) + 8 * (n & 1); };
  uint32_t it = 0;                  // pages this warp has consumed: place and phase
  bool ok = true;

  const Unpack unpack8;
  Walk<TR, 1, kSetup> walk;
  walk.start(p, g);
  Segment sg;
  while (walk.next(p, sg)) {
    const Request rq = sg.rq;
    const int h = sg.h, row0 = sg.tile * TR;
    const int rows = min(TR, rq.n_q * p.G - row0);
    const Pages pages(p, sg, tid == 0);
    const int end = min(sg.u1, pages.n);

    auto issue = [&](uint32_t n, int page) {
      if (lane == 0) {
        mbar_arrive_expect_tx(full(n), S::kStage);
        bulk_load(place_s + (n & 1) * S::kStage, p.data + ((size_t)page * p.Hkv + h) * S::kStage, S::kStage, full(n));
      }
    };
    // the next page of this warp and its block, -1 at the end
    auto next_page = [&](int &i, int &blk) -> int {
      while (i < end) {
        const int page = pages.page(i, blk, lane == 0);
        i += kWarps;
        if (page >= 0) return page;
      }
      blk = -1;
      return -1;
    };
    // the first two pages are on their way before anything else
    int li = sg.u0 + warp, blk[2] = {-1, -1};
    uint32_t sent = it;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int page = next_page(li, blk[e]);
      if (page >= 0) issue(sent++, page);
    }

    WT w;
    // Q: the lane holds column n8 (+ 8) as the second operand, channels in the
    // order in which Unpack gives the codes, scaled to lie below 2
#pragma unroll
    for (int x = 0; x < NR; ++x) {
      const int row = E == 2 ? n8 + 8 * x : n8 / 2 + 4 * x;
      const bool live = row < rows && (E == 2 || (n8 & 1) == 0);
      const int tok = live ? (row0 + row) / p.G : 0, head = live ? (row0 + row) % p.G : 0;
      const uint16_t *src = p.Q + (rq.q0 + tok) * p.qt + (h * p.G + head) * p.qh + t * (D / 4);
      uint4 u[W];
      float big = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        u[i] = make_uint4(0, 0, 0, 0);
        if (live) u[i] = __ldg(reinterpret_cast<const uint4 *>(src) + i);
        big = fmaxf(big, max_abs8(u[i]));
      }
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
      const uint32_t ex = min(max(__float_as_uint(big) >> 23, 1u), 253u);
      const float down = __uint_as_float((254u - ex) << 23);      // 2^-(ex - 127)
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        uint32_t pair[4];
        q_pairs(u[i], down, pair, sum);
        w.q[x][2 * i][0] = pair[0];
        w.q[x][2 * i][1] = pair[1];
        w.q[x][2 * i + 1][0] = pair[2];
        w.q[x][2 * i + 1][1] = pair[3];
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      // columns 2t and 2t + 1 belong to lanes 8t and 8t + 4
      const float mul = score_factor(p.scale_log2 * __uint_as_float(ex << 23));
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int y = 2 * x + e;
        w.qsum[y] = __shfl_sync(0xffffffffu, sum, 4 * (2 * t + e));
        w.mul[y] = __shfl_sync(0xffffffffu, mul, 4 * (2 * t + e));
        const int r8 = E == 2 ? 8 * x + 2 * t + e : 4 * x + t;
        w.vis[y] = p.causal ? rq.kv - (rq.n_q - 1 - min(rq.n_q - 1, (row0 + r8) / p.G)) : rq.kv;
        w.m[y] = -INFINITY;
        w.l[y] = w.z[y] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) w.o[x][j][e] = 0.f;
    }
#pragma unroll
    for (int y = 0; y < 2 * NR; ++y) w.vs[y] = kFirstScale;
    // keys that every row of the tile sees
    const int vis_all = p.causal ? rq.kv - (rq.n_q - 1 - row0 / p.G) : rq.kv;

    while (blk[0] >= 0) {
      // the number of the page after the next is read under this page's work
      int nblk = -1;
      const int npage = next_page(li, nblk);
      const uint8_t *st = place + (it & 1) * S::kStage;
      const int k_base = blk[0] * kPage;
      float sc[4][NR][4];
      if (!(ok = wait_warp(full(it), (it >> 1) & 1, ctl))) break;
      if (k_base + kPage > vis_all) {
        page_scores<D, NR, E, true>(w, unpack8, st, k_base, sc);
        page_values<D, NR, E, true>(w, unpack8, st, k_base, rq.kv, vis_all, sc);
      } else {
        page_scores<D, NR, E, false>(w, unpack8, st, k_base, sc);
        page_values<D, NR, E, false>(w, unpack8, st, k_base, rq.kv, vis_all, sc);
      }
      __syncwarp();                 // every lane has read the page
      if (npage >= 0) issue(sent++, npage);
      ++it;
      blk[0] = blk[1];
      blk[1] = nblk;
    }
    if (!ok) {
      // gave up: wait, with a limit, for the copies in flight before leaving
      volatile int never = 0;
      WaitCtl drain{&never, nullptr, 100000000LL};
      for (uint32_t n = it; n < sent; ++n) wait_bounded(full(n), (n >> 1) & 1, drain);
    }
    // ---- join the four warps: O + z, m, l of each row into the pages' place
    __syncthreads();
    if (s_abort) return;            // uniform after the barrier: a wait gave up
    float *mg = reinterpret_cast<float *>(place);
#pragma unroll
    for (int ye = 0; ye < NR * E; ++ye) {
      const int x = ye / E, e = ye % E, y = 2 * x + e;
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        w.l[y] += __shfl_xor_sync(0xffffffffu, w.l[y], o);
        w.z[y] += __shfl_xor_sync(0xffffffffu, w.z[y], o);
      }
      float *row = mg + (E == 2 ? 8 * x + 2 * t + e : 4 * x + t) * S::kMergeStride;
      const float z = w.z[y], vout = power_ratio(1.f, w.vs[y]);
      auto val = [&](int j, int up) { return fmaf(w.o[x][j][2 * up + e], vout, z); };
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
#pragma unroll
        for (int up = 0; up < 2; ++up)
          *reinterpret_cast<float4 *>(row + 64 * i + 8 * n8 + 4 * up) =
              make_float4(val(4 * i, up), val(4 * i + 1, up), val(4 * i + 2, up), val(4 * i + 3, up));
      if constexpr (D % 64 != 0)
        *reinterpret_cast<float4 *>(row + 64 * (D / 64) + 4 * n8) =
            make_float4(val(MT - 2, 0), val(MT - 2, 1), val(MT - 1, 0), val(MT - 1, 1));
      if (n8 == 0) {
        row[D] = w.m[y];
        row[D + 1] = w.l[y];
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
    constexpr int kVec = D / 4;
    if (sg.whole()) {
      for (int i = tid; i < rows * kVec; i += kThreads) {
        float mt_, lt_;
        const float4 v = joined(i / kVec, (i % kVec) * 4, mt_, lt_);
        store(i / kVec, (i % kVec) * 4, v, mt_, lt_);
      }
    } else {
      // a part: the block whose range begins inside the item uses its first
      // slot, the one in whose range the item begins its second
      constexpr int kSlot = kRows * (D + 2);
      float *mine = p.partial + ((size_t)blockIdx.x * 2 + (sg.u0 == 0 ? 1 : 0)) * kSlot;
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
      long long c1, cl;
      sharers<kSetup>(g, sg, c1, cl);
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
          // eight parts at a time: their loads are in flight together
          for (long long c0 = c1 - 1; c0 <= cl; c0 += 8) {
            float2 ml[8], a[8], b[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const long long c = c0 + e;
              ml[e] = make_float2(-INFINITY, 0.f);
              a[e] = b[e] = make_float2(0.f, 0.f);
              if (c <= cl) {
                const float *src = p.partial + (c * 2 + (c == c1 - 1 ? 1 : 0)) * kSlot + row * (D + 2);
                ml[e] = __ldcg(reinterpret_cast<const float2 *>(src + D));
                a[e] = __ldcg(reinterpret_cast<const float2 *>(src + ch));
                b[e] = __ldcg(reinterpret_cast<const float2 *>(src + ch + 2));
              }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float mn = fmaxf(mt_, ml[e].x);
              const float sub = mn > -INFINITY ? mn : 0.f;
              const float f0 = fast_ex2(mt_ - sub), f1 = fast_ex2(ml[e].x - sub);
              lt_ = lt_ * f0 + ml[e].y * f1;
              v = make_float4(v.x * f0 + a[e].x * f1, v.y * f0 + a[e].y * f1, v.z * f0 + b[e].x * f1, v.w * f0 + b[e].y * f1);
              mt_ = mn;
            }
          }
          store(row, ch, v, mt_, lt_);
        }
      }
    }
    fence_proxy_async();            // the place was written by stores; copies follow
    __syncthreads();
  }
}

template <int D, int NR, int E>
cudaError_t launch(const Params &p, int num_sms, cudaStream_t stream) {
  auto kfn = kv4_attn_kernel<D, NR, E>;
  constexpr int bytes = Smem<D>::kBytes;
  static OnDevices ready;
  static std::atomic<int> per_sm{1};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!ready.has(dev)) {
    e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    int n = 1;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kfn, kThreads, bytes);
    if (e != cudaSuccess) return e;
    per_sm.store(n < 1 ? 1 : n);
    ready.add(dev);
  }
  int blocks = per_sm.load() * num_sms;
  if (blocks > kMaxBlocks) blocks = kMaxBlocks;
  kfn<<<blocks, kThreads, bytes, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace hattn

// Parts of items (either kernel's), then both kernels' counters, then the words of
// the many rows' kernel.
static size_t partial_floats(int d) {
  const size_t few = (size_t)hattn::kMaxBlocks * 2 * hattn::kRows * (d + 2);
  const size_t many = kv4_chunk_partial_floats(d);
  return few > many ? few : many;
}

size_t kv4_attn_workspace_bytes(int d) {
  return partial_floats(d) * sizeof(float) + (hattn::kMaxBlocks + kv4_chunk_counters() + kv4_chunk_words()) * sizeof(int);
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
  p.counters = reinterpret_cast<int *>(p.partial + partial_floats(d));
  p.words = p.counters + hattn::kMaxBlocks + kv4_chunk_counters();
  p.dev_status = dev_status;
  p.wait_limit_ns = wait_limit_ns;
  // Which requests of a batch have few rows, and how long they are, only the
  // device knows: both kernels are launched and each takes its own, unless the
  // bounds say enough.  (A launch that takes nothing costs 3 us.)
  const long long rows = (long long)T * p.G, most = (long long)(max_q < T ? max_q : T) * p.G;
  const long long tiles = (rows + hattn::kRows - 1) / hattn::kRows;
  const bool few =
      most <= hattn::kRows || ((double)tiles + R) * Hkv * ((sel ? max_sel : max_blocks) + 8.0) <= (double)hattn::kFewWork;
  const bool many = !few && R == 1 && (double)tiles * Hkv * 9 > (double)hattn::kFewWork;
  if (many) {
    p.side = hattn::kAllRequests;
    p.counters += hattn::kMaxBlocks;
    return launch_kv4_chunk(p, d, num_sms, stream);
  }
  p.side = few ? hattn::kAllRequests : hattn::kFewSide;
  cudaError_t e = cudaErrorInvalidValue;
  switch (d) {
#define DITANGO_KV4(D)                                                                  \
  case D:                                                                               \
    e = most <= 4   ? hattn::launch<D, 1, 1>(p, num_sms, stream)                        \
        : most <= 8 ? hattn::launch<D, 1, 2>(p, num_sms, stream)                        \
                    : hattn::launch<D, 2, 2>(p, num_sms, stream);                       \
    break
    DITANGO_KV4(64);
    DITANGO_KV4(96);
    DITANGO_KV4(128);
#undef DITANGO_KV4
    default: break;
  }
  if (e != cudaSuccess || few) return e;
  p.side = hattn::kManySide;
  p.counters += hattn::kMaxBlocks;
  return launch_kv4_chunk(p, d, num_sms, stream);
}

}  // namespace ditango
