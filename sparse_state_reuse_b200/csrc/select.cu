// Cheap scores of key blocks, and the blocks that each query block selects.
//
// A block is summarised by the mean of its rows, held in 8 bits a channel:
// codes rint(127 S / max|S|) of the sum S, and the scale max|S| / (127 n).
// The score of key block j for query block i is
//   scale_j * sum over the query heads of the key head of scale_i (q_i . k_j)
// with q_i . k_j a sum of products of 8-bit codes: a whole number, which every
// order of summation gives alike.  The fp32 operations around it have one
// order, so that a selection is a function of its inputs down to the last bit.
#include <mutex>
#include <set>

#include "blocks.cuh"

namespace ditango {
namespace sel {

// ---------------------------------------------------------------- summaries
// One block of threads a block of rows, which is all in flight at once (16
// bytes a load): bound by reading x.  Sums are exact: a lane adds up to four
// bf16 values in fp32 (24 bits hold them but for values 2^13 times smaller
// than their neighbours), and goes on in fp64.
constexpr int kSumThreads = 256;

struct SummaryParams {
  int H, N, block, nb;
  const uint16_t *x;
  long long sb, sh, sn;
  const int *len;               // [B] valid rows, or null
  signed char *codes;           // [B, H, nb, d]
  float *scale;                 // [B, H, nb]
  float *mean;                  // [B, H, nb, d] or null
};

template <int D, int BLOCK>
__global__ void __launch_bounds__(kSumThreads) block_summary_kernel(const SummaryParams p) {
  constexpr int kGroup = (D == 64) ? 8 : 16;             // lanes of a row (12 of 16 busy at 96)
  constexpr int kPass = kSumThreads / kGroup;            // rows of one pass
  constexpr int kLoads = (BLOCK + kPass - 1) / kPass;
  constexpr int kWarps = kSumThreads / 32;
  __shared__ double part[kWarps][D];
  __shared__ double s_top[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sub = tid % kGroup, row = tid / kGroup;
  const int blk = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  int len = p.N;
  if (p.len) len = max(0, min(p.N, __ldg(p.len + b)));
  const int n = max(0, min(BLOCK, len - blk * BLOCK));
  const bool busy = sub < D / 8;
  const uint16_t *src = p.x + b * p.sb + h * p.sh + (long long)blk * BLOCK * p.sn + sub * 8;
  uint4 v[kLoads];
#pragma unroll
  for (int a = 0; a < kLoads; ++a) {
    const int r = row + a * kPass;
    v[a] = make_uint4(0, 0, 0, 0);
    if (busy && r < n) v[a] = __ldg(reinterpret_cast<const uint4 *>(src + r * p.sn));
  }
  double acc[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] = 0.0;
#pragma unroll
  for (int a = 0; a < kLoads; a += 4) {
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (a + e < kLoads) {
        const uint4 u = v[a + e];
        f[0] += bf_lo(u.x); f[1] += bf_hi(u.x); f[2] += bf_lo(u.y); f[3] += bf_hi(u.y);
        f[4] += bf_lo(u.z); f[5] += bf_hi(u.z); f[6] += bf_lo(u.w); f[7] += bf_hi(u.w);
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] += (double)f[k];
  }
#pragma unroll
  for (int o = kGroup; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] += __shfl_xor_sync(0xffffffffu, acc[k], o);
  if (lane < kGroup && busy) {
#pragma unroll
    for (int k = 0; k < 8; ++k) part[warp][sub * 8 + k] = acc[k];
  }
  __syncthreads();
  double s = 0.0;
  if (tid < D) {
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += part[w][tid];
  }
  double top = isfinite(s) ? fabs(s) : (double)INFINITY;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) s_top[warp] = top;
  __syncthreads();
  top = s_top[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) top = fmax(top, s_top[w]);
  const size_t at = ((size_t)b * p.H + h) * p.nb + blk;
  const bool good = top > 0.0 && top < (double)INFINITY;   // else (a value is not finite): score 0
  if (tid < D) {
    p.codes[at * D + tid] = good ? (signed char)(int)rint(s * 127.0 / top) : (signed char)0;
    if (p.mean) p.mean[at * D + tid] = n > 0 ? (float)(s / (double)n) : 0.f;
  }
  if (tid == 0) p.scale[at] = good ? (float)(top / (127.0 * n)) : 0.f;
}

// ---------------------------------------------------------------- selection
constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;

struct SelectParams {
  int Hkv, G, n_q, n_k, max_blocks, n_pages, k, band, sink, room, rows;
  int own;                      // key blocks of a query block; 0: the query stands at the end
  const signed char *qc, *kc;
  const float *qs, *ks;
  const int *block_table;       // [B, max_blocks] or null
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

// Whole numbers in the order of the scores, greater 0: -0 counts as 0, NaN as
// the least.
__device__ __forceinline__ uint32_t order_of(float x) {
  if (!(x == x)) return 1u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
constexpr uint32_t kForced = 0xffffffffu;

// One block of threads: up to 16 query blocks of one key head.  The scores of
// all key blocks stand in shared memory; each warp then finds the threshold of
// its rows by bisection between the least and greatest score (it ends as soon
// as the count is met, after 12 to 14 steps on a thousand different scores)
// and writes the list in ascending order.
template <int D>
__global__ void __launch_bounds__(kSelThreads) block_select_kernel(const __grid_constant__ SelectParams p) {
  constexpr int KS = D / 32;
  extern __shared__ uint32_t score[];        // [rows][n_k] (fp32 sums, then their order)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t = lane & 3, n8 = lane >> 2;
  const int i0 = blockIdx.x * p.rows, h = blockIdx.y, b = blockIdx.z;
  const int rows = min(p.rows, p.n_q - i0);
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
  auto forced = [&](int i, int j) -> bool {
    if (j < p.sink) return true;
    if (p.band < 0) return false;
    const int f = p.own ? i * p.own : nk - 1, l = p.own ? f + p.own - 1 : nk - 1;
    return j >= f - p.band && j <= l + p.band;
  };
  for (int g = 0; g < p.G; ++g) {
    const int head = h * p.G + g;
    uint32_t a[KS][4];
    float qs[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int row = n8 + 8 * x;
      const bool live = row < rows;
      const size_t at = ((size_t)b * p.Hkv * p.G + head) * p.n_q + i0 + (live ? row : 0);
      qs[x] = live ? __ldg(p.qs + at) : 0.f;
      const uint2 *src = reinterpret_cast<const uint2 *>(p.qc + at * D + t * (D / 4));
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const uint2 u = live ? __ldg(src + s) : make_uint2(0, 0);
        a[s][x] = u.x;
        a[s][2 + x] = u.y;
      }
    }
    constexpr int kAhead = 4;      // key tiles in flight
    for (int u0 = warp; u0 < tiles; u0 += kSelWarps * kAhead) {
      uint2 kb[kAhead][KS];
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        const int j = (u0 + e * kSelWarps) * 8 + n8;
        const signed char *src = nullptr;
        if (j < nk) {
          if (p.block_table) {
            const int page = __ldg(p.block_table + (size_t)b * p.max_blocks + j);
            if (page >= 0 && page < p.n_pages)
              src = p.kc + ((size_t)page * p.Hkv + h) * D;
            else
              set_status(p.dev_status, DITANGO_ERR_BOUNDS);
          } else {
            src = p.kc + (((size_t)b * p.Hkv + h) * p.n_k + j) * D;
          }
        }
#pragma unroll
        for (int s = 0; s < KS; ++s)
          kb[e][s] = src ? __ldg(reinterpret_cast<const uint2 *>(src + t * (D / 4)) + s) : make_uint2(0, 0);
      }
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        const int u = u0 + e * kSelWarps;
        if (u >= tiles) break;
        int c[4] = {0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < KS; ++s) imma16832(c, a[s], kb[e][s].x, kb[e][s].y);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int row = n8 + 8 * (q >> 1), j = u * 8 + 2 * t + (q & 1);
          if (row >= rows || j >= nk) continue;
          uint32_t *dst = score + (size_t)row * p.n_k + j;
          float x = __fmul_rn(qs[q >> 1], (float)c[q]);
          if (g > 0) x = __fadd_rn(__uint_as_float(*dst), x);
          if (g + 1 < p.G) {
            *dst = __float_as_uint(x);
          } else if (forced(i0 + row, j)) {
            *dst = kForced;
          } else {
            float ks;
            if (p.block_table) {
              const int page = __ldg(p.block_table + (size_t)b * p.max_blocks + j);
              ks = (page >= 0 && page < p.n_pages) ? __ldg(p.ks + (size_t)page * p.Hkv + h) : 0.f;
            } else {
              ks = __ldg(p.ks + ((size_t)b * p.Hkv + h) * p.n_k + j);
            }
            *dst = order_of(__fmul_rn(x, ks));
          }
        }
      }
    }
  }
  __syncthreads();
  for (int row = warp; row < rows; row += kSelWarps) {
    const uint32_t *key = score + (size_t)row * p.n_k;
    int n_forced = 0;
    uint32_t least = kForced, most = 0;
    for (int j = lane; j < nk; j += 32) {
      const uint32_t v = key[j];
      if (v == kForced) {
        ++n_forced;
      } else {
        least = min(least, v);
        most = max(most, v);
      }
    }
    n_forced = __reduce_add_sync(0xffffffffu, n_forced);
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    const int need = min(nk, max(n_forced, p.k));
    // entries above `above` are taken, and the first `ties` of those equal to it
    uint32_t above = 0;
    int ties = 0;
    if (need == n_forced) {
      above = kForced - 1;
    } else if (need < nk) {
      // lo: at least `need` entries are >= lo; hi: fewer are >= hi
      uint32_t lo = least, hi = most + 1;
      int at_hi = n_forced;
      bool met = false;
      while (hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        int c = 0;
        for (int j = lane; j < nk; j += 32) c += key[j] >= mid;
        c = __reduce_add_sync(0xffffffffu, c);
        if (c == need) {
          above = mid - 1;
          met = true;
          break;
        }
        if (c > need) lo = mid;
        else {
          hi = mid;
          at_hi = c;
        }
      }
      if (!met) {
        above = lo;
        ties = need - at_hi;
      }
    }
    int *dst = p.sel + (((size_t)b * p.Hkv + h) * p.n_q + i0 + row) * p.room;
    int out = 0;
    for (int j0 = 0; j0 < nk; j0 += 32) {
      const int j = j0 + lane;
      const uint32_t v = j < nk ? key[j] : 0u;
      const uint32_t eq = __ballot_sync(0xffffffffu, j < nk && v == above && ties > 0);
      const bool tie = ((eq >> lane) & 1u) && __popc(eq & ((1u << lane) - 1u)) < ties;
      const bool take = (j < nk && v > above) || tie;
      const uint32_t got = __ballot_sync(0xffffffffu, take);
      const int at = out + __popc(got & ((1u << lane) - 1u));
      if (take && at < p.room) dst[at] = j;
      out += __popc(got);
      ties -= min(ties, __popc(eq));
    }
    for (int j = out + lane; j < p.room; j += 32) dst[j] = -1;
    if (lane == 0) p.count[((size_t)b * p.Hkv + h) * p.n_q + i0 + row] = min(out, p.room);
  }
}

template <int D>
cudaError_t launch_select(const SelectParams &p, int B, int bytes, cudaStream_t stream) {
  auto kfn = block_select_kernel<D>;
  static std::mutex mu;
  static std::set<int> ready;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!ready.count(dev)) {
      e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
      if (e != cudaSuccess) return e;
      ready.insert(dev);
    }
  }
  const dim3 grid((unsigned)((p.n_q + p.rows - 1) / p.rows), (unsigned)p.Hkv, (unsigned)B);
  kfn<<<grid, kSelThreads, bytes, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace sel

// Most key blocks of a selection: one row of scores in shared memory.
int select_max_blocks() { return 200 * 1024 / 4; }

cudaError_t launch_block_summary(int B, int H, int N, int d, int block, const uint16_t *x, const int64_t *s,
                                 const int *len, signed char *codes, float *scale, float *mean,
                                 cudaStream_t stream) {
  sel::SummaryParams p{H, N, block, (N + block - 1) / block, x, s[0], s[1], s[2], len, codes, scale, mean};
  const dim3 grid((unsigned)p.nb, (unsigned)H, (unsigned)B);
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

cudaError_t launch_block_select(int B, int H, int Hkv, int n_q, int n_k, int d, int k, int band, int sink,
                                int room, int own, const signed char *qc, const float *qs,
                                const signed char *kc, const float *ks, const int *block_table,
                                int n_pages, const int *k_len, int *sel_out, int *count, int *dev_status,
                                cudaStream_t stream) {
  sel::SelectParams p;
  p.Hkv = Hkv;
  p.G = H / Hkv;
  p.n_q = n_q;
  p.n_k = n_k;
  p.max_blocks = n_k;
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
  p.sel = sel_out;
  p.count = count;
  p.dev_status = dev_status;
  // as many query blocks as the scores leave room for, 16 (one product) at most
  int rows = 16;
  while (rows > 1 && (rows / 2 >= n_q || (long long)rows * n_k * 4 > 100 * 1024)) rows /= 2;
  p.rows = rows;
  const int bytes = rows * n_k * 4;
  switch (d) {
    case 64: return sel::launch_select<64>(p, B, bytes, stream);
    case 96: return sel::launch_select<96>(p, B, bytes, stream);
    case 128: return sel::launch_select<128>(p, B, bytes, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace ditango
