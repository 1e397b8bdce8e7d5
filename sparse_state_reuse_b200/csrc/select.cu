// Cheap scores of key blocks, and the blocks that each query block selects.
//
// A block is summarised by the mean of its rows, held in 8 bits a channel:
// codes rint(127 S / max|S|) of the sum S, and the scale max|S| / (127 n).
// The score of key block j for query block i is
//   scale_j * sum over the query heads of the key head of scale_i (q_i . k_j)
// with q_i . k_j a sum of products of 8-bit codes: a whole number, which every
// order of summation gives alike.  The fp32 operations around it have one
// order, so that a selection is a function of its inputs down to the last bit.

#include "blocks.cuh"

namespace ditango {
namespace sel {

// ---------------------------------------------------------------- summaries
// A block of threads takes 128 rows (one query block or two key blocks), all in
// flight at once (16 bytes a load): bound by reading x.  A lane adds up to four bf16
// values in fp32, which holds their sum exactly unless they differ by 2^14 and
// more, and goes on in fp64.  (All in fp64: 76 us more, a conversion a value.)  The
// values go in over 2^7, which is exact for every bf16 value and leaves room for
// four of the largest.  Q and K of 76800 tokens, 40 heads of 128: 262 us, 6.0 TB/s
// (92% of the copy rate).
constexpr int kSumThreads = 256;
constexpr float kDown = 0x1p-7f;

struct SummaryParams {
  int H, N, nb;
  const uint16_t *x;
  long long sb, sh, sn;
  const int *len;               // [B] valid rows, or null
  signed char *codes;           // [B, H, nb, d]
  float *scale;                 // [B, H, nb]
  float *mean;                  // [B, H, nb, d] or null
};

template <int D, int BLOCK>
__device__ __forceinline__ void summarise(const SummaryParams &p, int h) {
  constexpr int kGroup = (D == 64) ? 8 : 16;             // lanes of a row (12 of 16 busy at 96)
  constexpr int kPass = kSumThreads / kGroup;            // rows of one pass
  constexpr int NB = 128 / BLOCK;                        // blocks of this block of threads
  constexpr int kLoads = BLOCK / kPass;                  // of each of them
  constexpr int kWarps = kSumThreads / 32;
  __shared__ double part[NB][kWarps][D];
  __shared__ double s_top[NB][kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sub = tid % kGroup, row = tid / kGroup;
  const int blk0 = blockIdx.x * NB, b = blockIdx.z;
  int len = p.N;
  if (p.len) len = max(0, min(p.N, __ldg(p.len + b)));
  const int left = len - blk0 * BLOCK;                   // valid rows from here on
  const bool busy = sub < D / 8;
  const uint16_t *src = p.x + b * p.sb + h * p.sh + (long long)blk0 * BLOCK * p.sn + sub * 8;
  uint4 v[NB * kLoads];
#pragma unroll
  for (int a = 0; a < NB * kLoads; ++a) {
    const int r = row + a * kPass;
    v[a] = make_uint4(0, 0, 0, 0);
    if (busy && r < left) v[a] = __ldg(reinterpret_cast<const uint4 *>(src + r * p.sn));
  }
#pragma unroll
  for (int q = 0; q < NB; ++q) {
    double acc[8];
#pragma unroll
    for (int a = 0; a < kLoads; a += 4) {
      float f[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (a + e < kLoads) {
          const uint4 u = v[q * kLoads + a + e];
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            f[2 * k] = e ? fmaf(bf_lo(w[k]), kDown, f[2 * k]) : bf_lo(w[k]) * kDown;
            f[2 * k + 1] = e ? fmaf(bf_hi(w[k]), kDown, f[2 * k + 1]) : bf_hi(w[k]) * kDown;
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = a ? acc[k] + (double)f[k] : (double)f[k];
    }
#pragma unroll
    for (int o = kGroup; o < 32; o <<= 1)
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] += __shfl_xor_sync(0xffffffffu, acc[k], o);
    if (lane < kGroup && busy) {
#pragma unroll
      for (int k = 0; k < 8; ++k) part[q][warp][sub * 8 + k] = acc[k];
    }
  }
  __syncthreads();
  // with two blocks, half of the threads each
  constexpr int kHalf = kSumThreads / NB;
  const int q = tid / kHalf, ch = tid % kHalf, blk = blk0 + q;
  const int n = max(0, min(BLOCK, left - q * BLOCK));
  double s = 0.0;
  if (ch < D) {
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += part[q][w][ch];
    s *= 1.0 / kDown;
  }
  double top = isfinite(s) ? fabs(s) : (double)INFINITY;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) s_top[q][warp % (kWarps / NB)] = top;
  __syncthreads();
  top = s_top[q][0];
#pragma unroll
  for (int w = 1; w < kWarps / NB; ++w) top = fmax(top, s_top[q][w]);
  if (blk >= p.nb) return;
  const size_t at = ((size_t)b * p.H + h) * p.nb + blk;
  const bool good = top > 0.0 && top < (double)INFINITY;   // else (a value is not finite): score 0
  if (ch < D) {
    p.codes[at * D + ch] = good ? (signed char)(int)rint(s * 127.0 / top) : (signed char)0;
    if (p.mean) p.mean[at * D + ch] = n > 0 ? (float)(s / (double)n) : 0.f;
  }
  if (ch == 0) p.scale[at] = good ? (float)(top / (127.0 * n)) : 0.f;
}

template <int D, int BLOCK>
__global__ void __launch_bounds__(kSumThreads) block_summary_kernel(const SummaryParams p) {
  summarise<D, BLOCK>(p, blockIdx.y);
}

// Query blocks and key blocks in one launch: the first heads are Q's.
template <int D>
__global__ void __launch_bounds__(kSumThreads) block_summaries_kernel(const SummaryParams q, const SummaryParams k) {
  const int h = blockIdx.y;
  if (h < q.H) {
    if (blockIdx.x < q.nb) summarise<D, kQBlock>(q, h);
  } else if (blockIdx.x * (kQBlock / kPage) < k.nb) {
    summarise<D, kPage>(k, h - q.H);
  }
}

// ---------------------------------------------------------------- selection
template <bool HEADS>
constexpr int kSelThreads = HEADS ? 512 : 256;

struct SelectParams {
  int Hkv, G, n_q, n_k, n_pages, k, band, sink, room, rows;
  int stride;                   // of a row of scores, see row_stride()
  int own;                      // key blocks of a query block; 0: the query stands at the end
  const signed char *qc, *kc;
  const float *qs, *ks;
  const uint16_t *q;            // HEADS: the queries themselves, (b, head) strides qb and qh, or null
  long long qb, qh;
  const int *block_table;       // [B, n_k] or null
  const int *k_len;             // [B] tokens, or null
  int *sel, *count, *dev_status;
};

__device__ __forceinline__ void imma16832(int (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Whole numbers in the order of the scores, greater 0 (and back): -0 counts as
// 0, NaN as the least.
__device__ __forceinline__ uint32_t order_of(float x) {
  if (!(x == x)) return 1u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float score_of(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? u ^ 0x80000000u : ~u);
}
constexpr uint32_t kForced = 0xffffffffu;

// Where the search looks next between lo and hi.
__device__ __forceinline__ uint32_t next_mid(uint32_t lo, uint32_t hi, int step) {
  if ((step & 3) != 3) {
    const uint32_t x = order_of(0.5f * score_of(lo) + 0.5f * score_of(hi - 1));
    if (x > lo && x < hi) return x;
  }
  return lo + (hi - lo) / 2;
}

// Warp-wide choice of one row: the threshold between what is taken and what is
// not, then the list in ascending order.  The search starts from the least and
// greatest score and ends as soon as the count is met.  A step halves the
// interval of the scores, every fourth one the interval of their order, so that
// far-flung scores need 128 steps at most; a thousand ordinary ones take about 10
// (halving the order alone 18, because it steps through the exponents around 0:
// 501 instead of 491 us for 40 heads of 600 query and 1200 key blocks.
// Interpolating between the counts needs fewer steps, but the chain of each is
// longer: 540 us).
// REG > 0: the row (at most 32 REG entries) stays in registers; 0: it is read
// from shared memory in every step.
template <int REG>
__device__ __forceinline__ void choose_row(const uint32_t *key, int nk, int k, int room, int *dst, int *count) {
  const int lane = threadIdx.x & 31;
  uint32_t v[REG > 0 ? REG : 1];
  int n_forced = 0;
  uint32_t least = kForced, most = 0;
  auto look = [&](uint32_t x) {
    if (x == kForced) {
      ++n_forced;
    } else if (x != 0u) {
      least = min(least, x);
      most = max(most, x);
    }
  };
  if constexpr (REG > 0) {
#pragma unroll
    for (int a = 0; a < REG; ++a) {
      const int j = a * 32 + lane;
      v[a] = j < nk ? key[j] : 0u;      // 0: no entry
      look(v[a]);
    }
  } else {
    for (int j = lane; j < nk; j += 32) look(key[j]);
  }
  n_forced = __reduce_add_sync(0xffffffffu, n_forced);
  least = __reduce_min_sync(0xffffffffu, least);
  most = __reduce_max_sync(0xffffffffu, most);
  const int need = min(nk, max(n_forced, k));
  // entries above `above` are taken, and the first `ties` of those equal to it
  uint32_t above = 0;
  int ties = 0;
  if (need == n_forced) {
    above = kForced - 1;
  } else if (need < nk) {
    // at least `need` entries are >= lo, fewer are >= hi
    uint32_t lo = least, hi = most + 1;
    int at_hi = n_forced;
    bool met = false;
    for (int step = 0; hi - lo > 1; ++step) {
      const uint32_t mid = next_mid(lo, hi, step);
      int c = 0;
      if constexpr (REG > 0) {
#pragma unroll
        for (int a = 0; a < REG; ++a) c += v[a] >= mid;
      } else {
        for (int j = lane; j < nk; j += 32) c += key[j] >= mid;
      }
      c = __reduce_add_sync(0xffffffffu, c);
      if (c == need) {
        above = mid - 1;
        met = true;
        break;
      }
      if (c > need) {
        lo = mid;
      } else {
        hi = mid;
        at_hi = c;
      }
    }
    if (!met) {
      above = lo;
      ties = need - at_hi;
    }
  }
  int out = 0;
  const uint32_t below = (1u << lane) - 1u;
  auto emit = [&](int j, uint32_t x) {
    bool take = x > above;
    if (ties > 0) {
      const uint32_t eq = __ballot_sync(0xffffffffu, x == above);
      take = take || (((eq >> lane) & 1u) && __popc(eq & below) < ties);
      ties -= min(ties, __popc(eq));
    }
    const uint32_t got = __ballot_sync(0xffffffffu, take);
    const int at = out + __popc(got & below);
    if (take && at < room) dst[at] = j;
    out += __popc(got);
  };
  if constexpr (REG > 0) {
#pragma unroll
    for (int a = 0; a < REG; ++a) emit(a * 32 + lane, v[a]);
  } else {
    for (int j0 = 0; j0 < nk; j0 += 32) emit(j0 + lane, j0 + lane < nk ? key[j0 + lane] : 0u);
  }
  for (int j = out + lane; j < room; j += 32) dst[j] = -1;
  if (lane == 0) *count = min(out, room);
}

// The same choice by all threads of a block, each with a run of neighbouring
// entries in shared memory (an odd number of them: no bank conflicts), for a row
// that has the block to itself.  Loops instead of the unrolled registers above:
// a kernel that runs once a step finds its code in no cache (one warp with the
// row in registers took 7 us for 1200 entries, this 4.5).
template <int THREADS>
__device__ __forceinline__ void choose_block(const uint32_t *key, int nk, int k, int room, int *dst, int *count) {
  constexpr int WARPS = THREADS / 32;
  static_assert(WARPS <= 32, "one value a warp is summed by one warp");
  __shared__ uint32_t part[4][WARPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = ((nk + THREADS - 1) / THREADS) | 1, j0 = min(nk, tid * per), j1 = min(nk, j0 + per);
  uint32_t least = kForced, most = 0, forced = 0;
  for (int j = j0; j < j1; ++j) {
    const uint32_t x = key[j];
    if (x == kForced) {
      ++forced;
    } else {
      least = min(least, x);
      most = max(most, x);
    }
  }
  forced = __reduce_add_sync(0xffffffffu, forced);
  least = __reduce_min_sync(0xffffffffu, least);
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) {
    part[0][warp] = forced;
    part[1][warp] = least;
    part[2][warp] = most;
  }
  __syncthreads();
  const int from = min(lane, WARPS - 1);
  const int n_forced = (int)__reduce_add_sync(0xffffffffu, lane < WARPS ? part[0][from] : 0u);
  least = __reduce_min_sync(0xffffffffu, part[1][from]);
  most = __reduce_max_sync(0xffffffffu, part[2][from]);
  const int need = min(nk, max(n_forced, k));
  uint32_t above = 0;
  int ties = 0;
  __syncthreads();
  if (need == n_forced) {
    above = kForced - 1;
  } else if (need < nk) {
    uint32_t lo = least, hi = most + 1;
    int at_hi = n_forced;
    bool met = false;
    for (int step = 0; hi - lo > 1; ++step) {
      const uint32_t mid = next_mid(lo, hi, step);
      uint32_t c = 0;
      for (int j = j0; j < j1; ++j) c += key[j] >= mid;
      c = __reduce_add_sync(0xffffffffu, c);
      if (lane == 0) part[step & 1][warp] = c;      // two places in turn: one barrier a step
      __syncthreads();
      const int all = (int)__reduce_add_sync(0xffffffffu, lane < WARPS ? part[step & 1][from] : 0u);
      if (all == need) {
        above = mid - 1;
        met = true;
        break;
      }
      if (all > need) {
        lo = mid;
      } else {
        hi = mid;
        at_hi = all;
      }
    }
    if (!met) {
      above = lo;
      ties = need - at_hi;
    }
  }
  // entries above in the low half, equal ones in the high half (at most 51200 each)
  uint32_t mine = 0;
  for (int j = j0; j < j1; ++j) {
    const uint32_t x = key[j];
    mine += (x > above ? 1u : 0u) + (ties > 0 && x == above ? 0x10000u : 0u);
  }
  uint32_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) part[3][warp] = upto;
  __syncthreads();
  uint32_t before = upto - mine, total = 0;
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += part[3][w];
    total += part[3][w];
  }
  int equal = (int)(before >> 16), at = (int)(before & 0xffffu) + min(equal, ties);
  for (int j = j0; j < j1; ++j) {
    const uint32_t x = key[j];
    bool take = x > above;
    if (ties > 0 && x == above) take = equal++ < ties;
    if (take) {
      if (at < room) dst[at] = j;
      ++at;
    }
  }
  const int out = (int)(total & 0xffffu) + min((int)(total >> 16), ties);
  for (int j = out + tid; j < room; j += THREADS) dst[j] = -1;
  if (tid == 0) *count = min(out, room);
}

// One block of threads: up to 16 query blocks of one key head, whose scores of
// all key blocks stand in shared memory.  HEADS: a single query block, and the
// 16 rows of the product are the query heads of the key head instead, so that
// the key codes are read once and not once a head.
// Legacy tensor instructions, since a row of scores has to go through registers
// and shared memory anyway and the products are 3% of the time.  600 x 1200 blocks
// of 40 heads of 128: 232 us, a fifth of it the threshold search; bound by the
// chains of latencies of 16 warps an SM (the scores' 78 KB leave room for two
// blocks).  HEADS, 16 requests of up to 1200 pages, 8 key heads: 18 us cold, of which
// the codes' 15 MB are 2; the rest is one block's chain: queries' codes 2, scores 6,
// search and list 4.5.
template <int D, int REG, bool HEADS>
__global__ void __launch_bounds__(kSelThreads<HEADS>) block_select_kernel(const __grid_constant__ SelectParams p) {
  constexpr int KS = D / 32, kThreads = kSelThreads<HEADS>, kWarps = kThreads / 32;
  extern __shared__ __align__(16) uint32_t score[];   // [rows][stride] (fp32 sums, then their order)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t = lane & 3, n8 = lane >> 2;
  const int i0 = HEADS ? 0 : blockIdx.x * p.rows, h = blockIdx.y, b = blockIdx.z;
  const int rows = HEADS ? p.G : min(p.rows, p.n_q - i0);
  int nk = p.n_k;
  if (p.k_len) {
    const long long len = __ldg(p.k_len + b);
    const long long most = (len + kPage - 1) / kPage;
    if (len < 0 || (p.block_table && most > p.n_k)) {
      if (tid == 0) set_status(p.dev_status, DITANGO_ERR_BOUNDS);
    }
    nk = (int)max(0LL, min((long long)p.n_k, most));
  }
  const int tiles = (nk + 7) / 8;
  // the band of query block i: key blocks [first, last]
  auto band_of = [&](int i, int &first, int &last) {
    first = p.own ? i * p.own : nk - 1;
    last = p.own ? first + p.own - 1 : nk - 1;
    first -= p.band;
    last += p.band;
    if (p.band < 0) last = first - 1;
  };
  auto page_of = [&](int j) -> int {         // -1: a page number out of range, which scores 0
    const int page = __ldg(p.block_table + (size_t)b * p.n_k + j);
    if (page >= 0 && page < p.n_pages) return page;
    set_status(p.dev_status, DITANGO_ERR_BOUNDS);
    return -1;
  };
  auto scale_of = [&](int j) -> float {
    if (!p.block_table) return __ldg(p.ks + ((size_t)b * p.Hkv + h) * p.n_k + j);
    const int page = page_of(j);
    return page < 0 ? 0.f : __ldg(p.ks + (size_t)page * p.Hkv + h);
  };
  // HEADS: the codes of single queries, formed here; the scale of each key block
  // and its page, read at once and not by the chain of each product
  __shared__ __align__(16) signed char q_code[HEADS ? 16 : 1][D];
  __shared__ float q_scale[16];
  if constexpr (HEADS) {
    for (int g = warp; p.q && g < rows; g += kWarps) {
      // a row by itself: 127 x has 15 bits and x / top 8 by 8, so that fp32's
      // quotient is exact in a tie and no other comes near one; 2^-16 keeps 127 x
      // of the largest values finite, and what it could round is far below a code
      constexpr int kOwn = D / 32;
      const uint16_t *src = p.q + b * p.qb + (h * p.G + g) * p.qh + lane * kOwn;
      float f[kOwn], top = 0.f;
#pragma unroll
      for (int e = 0; e < kOwn; ++e) {
        f[e] = __uint_as_float((uint32_t)__ldg(src + e) << 16);
        top = fmaxf(top, isfinite(f[e]) ? fabsf(f[e]) : INFINITY);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const bool good = top > 0.f && top < INFINITY;
      const float down = top > 1e30f ? 0x1p-16f : 1.f;
#pragma unroll
      for (int e = 0; e < kOwn; ++e)
        q_code[g][lane * kOwn + e] =
            good ? (signed char)(int)rintf(__fdiv_rn(f[e] * down * 127.f, top * down)) : (signed char)0;
      if (lane == 0) q_scale[g] = good ? __fdiv_rn(top, 127.f) : 0.f;
    }
  }
  float *scale = reinterpret_cast<float *>(score + rows * p.stride);
  int *pages = reinterpret_cast<int *>(scale + p.stride);
  if constexpr (HEADS) {
    // the warps without a query head, if there are any, are done with it at once
    const int from = p.q && rows < kWarps ? rows * 32 : 0;
    constexpr int kOnce = 4;
    const int step = kThreads - from;
    for (int j0 = tid - from; j0 >= 0 && j0 < nk; j0 += step * kOnce) {
      int page[kOnce];
      float s[kOnce];
#pragma unroll
      for (int e = 0; e < kOnce; ++e) {
        const int j = j0 + e * step;
        page[e] = j < nk && p.block_table ? __ldg(p.block_table + (size_t)b * p.n_k + j) : j;
      }
#pragma unroll
      for (int e = 0; e < kOnce; ++e) {
        const int j = j0 + e * step;
        const bool good = !p.block_table || (page[e] >= 0 && page[e] < p.n_pages);
        if (j < nk && !good) set_status(p.dev_status, DITANGO_ERR_BOUNDS);
        if (!good) page[e] = -1;
        const size_t at = p.block_table ? (size_t)page[e] * p.Hkv + h : ((size_t)b * p.Hkv + h) * p.n_k + j;
        s[e] = j < nk && good ? __ldg(p.ks + at) : 0.f;
      }
#pragma unroll
      for (int e = 0; e < kOnce; ++e) {
        const int j = j0 + e * step;
        if (j >= nk) break;
        scale[j] = s[e];
        pages[j] = page[e];
      }
    }
    __syncthreads();
  }
  const int rows_up = (rows + 7) & ~7;
  int bf[2], bl[2];
  band_of(i0 + n8, bf[0], bl[0]);
  band_of(i0 + n8 + 8, bf[1], bl[1]);
  for (int g = 0; g < (HEADS ? 1 : p.G); ++g) {
    uint32_t a[KS][4];
    float qs[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int row = n8 + 8 * x;
      const bool live = row < rows;
      const size_t at = HEADS ? ((size_t)b * p.Hkv + h) * p.G + (live ? row : 0)
                              : (((size_t)b * p.Hkv + h) * p.G + g) * p.n_q + i0 + (live ? row : 0);
      const bool here = HEADS && p.q != nullptr;
      qs[x] = !live ? 0.f : (here ? q_scale[row & 15] : __ldg(p.qs + at));
      const uint2 *src = reinterpret_cast<const uint2 *>(here ? &q_code[HEADS && live ? row : 0][t * (D / 4)]
                                                              : p.qc + at * D + t * (D / 4));
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const uint2 u = live ? src[s] : make_uint2(0, 0);
        a[s][x] = u.x;
        a[s][2 + x] = u.y;
      }
    }
    constexpr int kAhead = 4;      // key tiles in flight
    for (int u0 = warp; u0 < tiles; u0 += kWarps * kAhead) {
      uint2 kb[kAhead][KS];
      const signed char *src[kAhead];
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        const int j = (u0 + e * kWarps) * 8 + n8;
        src[e] = nullptr;
        if (j >= nk) continue;
        if (p.block_table) {
          const int page = HEADS ? pages[j] : page_of(j);
          if (page >= 0) src[e] = p.kc + ((size_t)page * p.Hkv + h) * D;
        } else {
          src[e] = p.kc + (((size_t)b * p.Hkv + h) * p.n_k + j) * D;
        }
      }
#pragma unroll
      for (int e = 0; e < kAhead; ++e)
#pragma unroll
        for (int s = 0; s < KS; ++s)
          kb[e][s] = src[e] ? __ldg(reinterpret_cast<const uint2 *>(src[e] + t * (D / 4)) + s) : make_uint2(0, 0);
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        const int u = u0 + e * kWarps;
        if (u >= tiles) break;
        int c[4] = {0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < KS; ++s) imma16832(c, a[s], kb[e][s].x, kb[e][s].y);
        // columns j and j + 1 of rows n8 and n8 + 8; entries past the end are 0
        const int j = u * 8 + 2 * t;
        const bool in0 = j < nk, in1 = j + 1 < nk, last_head = HEADS || g + 1 == p.G;
        float ks0 = 0.f, ks1 = 0.f;
        if (!HEADS && last_head) {
          if (in0) ks0 = scale_of(j);
          if (in1) ks1 = scale_of(j + 1);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (x * 8 >= rows_up) break;
          uint2 *dst = reinterpret_cast<uint2 *>(score + (n8 + 8 * x) * p.stride + j);
          float s0 = __fmul_rn(qs[x], (float)c[2 * x]), s1 = __fmul_rn(qs[x], (float)c[2 * x + 1]);
          if (n8 + 8 * x >= rows) continue;
          if (!HEADS && g > 0) {
            const uint2 before = *dst;
            s0 = __fadd_rn(__uint_as_float(before.x), s0);
            s1 = __fadd_rn(__uint_as_float(before.y), s1);
          }
          uint2 v = make_uint2(__float_as_uint(s0), __float_as_uint(s1));
          if (!HEADS && last_head) {
            v.x = order_of(__fmul_rn(s0, ks0));
            v.y = order_of(__fmul_rn(s1, ks1));
            if (j < p.sink || (j >= bf[x] && j <= bl[x])) v.x = kForced;
            if (j + 1 < p.sink || (j + 1 >= bf[x] && j + 1 <= bl[x])) v.y = kForced;
            if (!in0) v.x = 0u;
            if (!in1) v.y = 0u;
          }
          *dst = v;
        }
      }
    }
  }
  __syncthreads();
  if constexpr (HEADS) {
    int first, last;
    band_of(0, first, last);
    for (int j = tid; j < nk; j += kThreads) {
      float x = __uint_as_float(score[j]);
      for (int g = 1; g < rows; ++g) x = __fadd_rn(x, __uint_as_float(score[g * p.stride + j]));
      score[j] = j < p.sink || (j >= first && j <= last) ? kForced : order_of(__fmul_rn(x, scale[j]));
    }
    __syncthreads();
    const size_t at = (size_t)b * p.Hkv + h;
    choose_block<kThreads>(score, nk, p.k, p.room, p.sel + at * p.room, p.count + at);
  } else {
    for (int row = warp; row < rows; row += kWarps) {
      const size_t at = ((size_t)b * p.Hkv + h) * p.n_q + i0 + row;
      choose_row<REG>(score + row * p.stride, nk, p.k, p.room, p.sel + at * p.room, p.count + at);
    }
  }
}

constexpr int kMaxScoreBytes = 208 * 1024;

// Entries of a row of scores in shared memory: whole tiles of 8, and 8 more than
// a multiple of 32, so that the rows a warp writes at once lie in other banks.
int row_stride(int n_k) { return (n_k + 8 - 1) / 8 * 8 + (40 - (n_k + 7) / 8 * 8 % 32) % 32; }

template <int D, int REG, bool HEADS>
cudaError_t launch_select(const SelectParams &p, int B, int bytes, cudaStream_t stream) {
  auto kfn = block_select_kernel<D, REG, HEADS>;
  static OnDevices ready;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!ready.has(dev)) {
    e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxScoreBytes);
    if (e != cudaSuccess) return e;
    ready.add(dev);
  }
  const dim3 grid((unsigned)(HEADS ? 1 : (p.n_q + p.rows - 1) / p.rows), (unsigned)p.Hkv, (unsigned)B);
  kfn<<<grid, kSelThreads<HEADS>, bytes, stream>>>(p);
  return cudaGetLastError();
}

// The row in registers up to 1536 entries (98304 tokens), in 16 or 48 of them a
// lane; a longer one is read from shared memory.
template <int D, bool HEADS>
cudaError_t launch_select(const SelectParams &p, int B, int bytes, cudaStream_t stream) {
  if constexpr (!HEADS) {
    if (p.n_k <= 32 * 16) return launch_select<D, 16, HEADS>(p, B, bytes, stream);
    if (p.n_k <= 32 * 48) return launch_select<D, 48, HEADS>(p, B, bytes, stream);
  }
  return launch_select<D, 0, HEADS>(p, B, bytes, stream);
}

}  // namespace sel

// Most key blocks of a selection: one row of scores in shared memory.
int select_max_blocks() { return 51200; }

cudaError_t launch_block_summary(int B, int H, int N, int d, int block, const uint16_t *x, const int64_t *s,
                                 const int *len, signed char *codes, float *scale, float *mean,
                                 cudaStream_t stream) {
  sel::SummaryParams p{H, N, (N + block - 1) / block, x, s[0], s[1], s[2], len, codes, scale, mean};
  const dim3 grid((unsigned)((N + kQBlock - 1) / kQBlock), (unsigned)H, (unsigned)B);
#define DITANGO_SUM(D)                                                                              \
  case D:                                                                                           \
    if (block == kPage)                                                                             \
      sel::block_summary_kernel<D, kPage><<<grid, sel::kSumThreads, 0, stream>>>(p);                \
    else                                                                                            \
      sel::block_summary_kernel<D, kQBlock><<<grid, sel::kSumThreads, 0, stream>>>(p);              \
    break
  switch (d) {
    DITANGO_SUM(64);
    DITANGO_SUM(96);
    DITANGO_SUM(128);
    default: return cudaErrorInvalidValue;
  }
#undef DITANGO_SUM
  return cudaGetLastError();
}

cudaError_t launch_block_summaries(int B, int H, int Hkv, int Nq, int Nk, int d, const uint16_t *Q,
                                   const int64_t *qst, const uint16_t *K, const int64_t *kst, const int *k_len,
                                   signed char *q_codes, float *q_scale, signed char *k_codes, float *k_scale,
                                   float *k_mean, cudaStream_t stream) {
  const sel::SummaryParams q{H, Nq, (Nq + kQBlock - 1) / kQBlock, Q, qst[0], qst[1], qst[2], nullptr,
                             q_codes, q_scale, nullptr};
  const sel::SummaryParams k{Hkv, Nk, (Nk + kPage - 1) / kPage, K, kst[0], kst[1], kst[2], k_len,
                             k_codes, k_scale, k_mean};
  const int rows = Nq > Nk ? Nq : Nk;
  const dim3 grid((unsigned)((rows + kQBlock - 1) / kQBlock), (unsigned)(H + Hkv), (unsigned)B);
  switch (d) {
    case 64: sel::block_summaries_kernel<64><<<grid, sel::kSumThreads, 0, stream>>>(q, k); break;
    case 96: sel::block_summaries_kernel<96><<<grid, sel::kSumThreads, 0, stream>>>(q, k); break;
    case 128: sel::block_summaries_kernel<128><<<grid, sel::kSumThreads, 0, stream>>>(q, k); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

// One query block a head group, with the scores of all its heads beside one
// another in shared memory.
bool select_by_heads(int n_q, int G, int n_k) {
  return n_q == 1 && G <= 16 && (G + 2LL) * sel::row_stride(n_k) * 4 <= sel::kMaxScoreBytes;
}

cudaError_t launch_block_select(int B, int H, int Hkv, int n_q, int n_k, int d, int k, int band, int sink,
                                int room, int own, const signed char *qc, const float *qs,
                                const signed char *kc, const float *ks, const int *block_table,
                                int n_pages, const int *k_len, int *sel_out, int *count, int *dev_status,
                                const uint16_t *q, const int64_t *q_strides, cudaStream_t stream) {
  sel::SelectParams p;
  p.Hkv = Hkv;
  p.G = H / Hkv;
  p.n_q = n_q;
  p.n_k = n_k;
  p.n_pages = n_pages;
  p.k = k;
  p.band = band;
  p.sink = sink;
  p.room = room;
  p.own = own;
  p.qc = qc;
  p.kc = kc;
  p.qs = qs;
  p.ks = ks;
  p.block_table = block_table;
  p.k_len = k_len;
  p.q = q;
  p.qb = q ? q_strides[0] : 0;
  p.qh = q ? q_strides[1] : 0;
  p.sel = sel_out;
  p.count = count;
  p.dev_status = dev_status;
  // as many query blocks as the scores leave room for, 16 (one product) at most
  p.stride = sel::row_stride(n_k);
  int rows = 16;
  while (rows > 1 && (rows / 2 >= n_q || (long long)rows * p.stride * 4 > 100 * 1024)) rows /= 2;
  const bool heads = select_by_heads(n_q, p.G, n_k);
  p.rows = rows;
  const int bytes = (heads ? p.G + 2 : rows) * p.stride * 4;
  switch (d) {
#define DITANGO_SEL(D)                                                     \
  case D:                                                                  \
    return heads ? sel::launch_select<D, true>(p, B, bytes, stream)        \
                 : sel::launch_select<D, false>(p, B, bytes, stream)
    DITANGO_SEL(64);
    DITANGO_SEL(96);
    DITANGO_SEL(128);
#undef DITANGO_SEL
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace ditango
