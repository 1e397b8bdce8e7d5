// The paged 4-bit key/value history: tables from request lengths, writing,
// reading back, and page summaries.  (Attention over it: history_attn.cu.)
#include "blocks.cuh"

namespace ditango {
namespace hist {

// ---------------------------------------------------------------- tables
// Per request r: have = ceil(ctx/64) pages in its table row, need =
// ceil((ctx+new)/64); the new pages come from the free list at the exclusive
// running sum of need - have, the tokens' offsets from that of new.  Every
// block sums all requests again (a few KB of L2 reads) and then writes its own
// share of the table and the slot map, so that one launch does everything; it
// is latency-bound (3.4 us for 64 single tokens, 5.3 us for 512 requests and
// 102k tokens on B200, most of it launch and two dependent reads).
constexpr int kTabThreads = 256;

struct TablesParams {
  int R, max_blocks, max_tokens, n_pages, n_free;
  const int *ctx_len, *new_len, *free_pages;
  int *block_table, *kv_len, *q_off;
  long long *slot_map;
  int *pages_used, *dev_status;
};

__global__ void __launch_bounds__(kTabThreads) tables_kernel(const TablesParams p) {
  extern __shared__ int sm[];
  int *off = sm;                    // [R + 1] token offsets, clamped to max_tokens
  int *first = sm + p.R + 1;        // [R + 1] first free-list entry of the request
  __shared__ long long wsum_t[kTabThreads / 32], wsum_p[kTabThreads / 32];
  __shared__ int s_used;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.R + kTabThreads - 1) / kTabThreads;
  const int r0 = tid * per, r1 = min(p.R, r0 + per);
  if (tid == 0) s_used = 0;

  bool bad = false;
  // lengths of request r: tokens it takes in the packed batch, and new pages
  auto lens = [&](int r, int &ctx, int &nw, int &extra) -> bool {
    ctx = __ldg(p.ctx_len + r);
    nw = __ldg(p.new_len + r);
    const bool neg = ctx < 0 || nw < 0;
    ctx = max(ctx, 0);
    nw = max(nw, 0);
    const long long need = ((long long)ctx + nw + kPage - 1) / kPage;
    const bool ok = !neg && need <= p.max_blocks;
    extra = ok ? (int)(need - (ctx + (long long)kPage - 1) / kPage) : 0;
    return ok;
  };
  long long st = 0, sp = 0;
  for (int r = r0; r < r1; ++r) {
    int c, n, e;
    lens(r, c, n, e);
    st += n;
    sp += e;
  }
  long long it = st, ip = sp;   // inclusive sums over the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, it, o), b = __shfl_up_sync(0xffffffffu, ip, o);
    if (lane >= o) {
      it += a;
      ip += b;
    }
  }
  if (lane == 31) {
    wsum_t[warp] = it;
    wsum_p[warp] = ip;
  }
  __syncthreads();
  it -= st;
  ip -= sp;
  for (int w = 0; w < warp; ++w) {
    it += wsum_t[w];
    ip += wsum_p[w];
  }
  const long long cap = p.max_tokens;
  for (int r = r0; r < r1; ++r) {
    int c, n, e;
    bool ok = lens(r, c, n, e);
    const bool fits = ok && it + n <= cap && ip + e <= p.n_free;
    off[r] = (int)min(it, cap);
    // a request that does not fit takes no page: its entry says so
    first[r] = fits ? (int)ip : -1;
    if (fits) {
      if (e > 0) atomicMax(&s_used, (int)ip + e);
    } else {
      bad = true;
    }
    if (blockIdx.x == 0)
      p.kv_len[r] = fits ? c + n : (int)min((long long)c, (long long)p.max_blocks * kPage);
    it += n;
    ip += e;
    if (r == p.R - 1) off[p.R] = (int)min(it, cap);
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int r = tid; r <= p.R; r += kTabThreads) p.q_off[r] = off[r];
    if (bad) set_status(p.dev_status, DITANGO_ERR_BOUNDS);
    if (tid == 0) *p.pages_used = s_used;
  }
  // the new pages of the requests this block takes
  for (int r = blockIdx.x * (kTabThreads / 32) + warp; r < p.R; r += gridDim.x * (kTabThreads / 32)) {
    const int f = first[r];
    if (f < 0) continue;
    int c, n, e;
    lens(r, c, n, e);
    int *row = p.block_table + (size_t)r * p.max_blocks + (c + kPage - 1) / kPage;
    for (int k = lane; k < e; k += 32) row[k] = __ldg(p.free_pages + f + k);
  }
  // slots of the tokens
  const int total = off[p.R];
  for (int t = blockIdx.x * kTabThreads + tid; t < p.max_tokens; t += gridDim.x * kTabThreads) {
    long long slot = -1;
    if (t < total) {
      int lo = 0, hi = p.R - 1;     // the last request that starts at or before t and is not empty
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (off[mid] <= t) lo = mid; else hi = mid - 1;
      }
      if (first[lo] >= 0) {
        const int c = max(__ldg(p.ctx_len + lo), 0);
        const int pos = c + t - off[lo];
        const int have = (c + kPage - 1) / kPage, blk = pos / kPage;
        const int page = blk < have ? __ldg(p.block_table + (size_t)lo * p.max_blocks + blk)
                                    : __ldg(p.free_pages + first[lo] + blk - have);
        if (page >= 0 && page < p.n_pages)
          slot = (long long)page * kPage + pos % kPage;
        else
          set_status(p.dev_status, DITANGO_ERR_BOUNDS);
      }
    }
    p.slot_map[t] = slot;
  }
}

// ---------------------------------------------------------------- write, read
struct RowsParams {
  long long T;
  int Hkv, n_pages;
  const uint16_t *K, *V;
  uint16_t *Ko, *Vo;
  long long kt, kh, vt, vh;     // token and head strides, elements
  const long long *slots;
  uint8_t *data;
  int *dev_status;
};

// Codes of 8 values of a row: c = round to nearest even of (x - lo) / s, as
// exact arithmetic gives it.  The quotient is formed with one reciprocal; a
// quotient too near to a half (closer than its error, or with sizes that
// leave fp32's comfortable range) is formed again in fp64, where the
// difference of two bf16 values is exact and the division correctly rounded.
// The second path is rare (about one group of 8 in 10^4 on normal data).
__device__ __forceinline__ uint32_t codes8(const float (&x)[8], float lo, float hi, float s) {
  if (!(s > 0.f)) return 0u;
  const float inv = __frcp_rn(s);
  const float off = -lo * inv;
  const float kRound = 12582912.0f;   // 1.5 * 2^23: adding it rounds to an integer
  const float err = (fmaxf(fabsf(lo), fabsf(hi)) * inv + 16.f) * 4e-7f;
  float far = 0.f;
  uint32_t w = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float q = fmaf(x[k], inv, off);
    const float t = q + kRound;
    far = fmaxf(far, fabsf(q - (t - kRound)));
    w |= (__float_as_uint(t) & 15u) << (4 * k);
  }
  const bool plain = far < 0.5f - err && s > 1e-30f && s < 1e30f;
  if (!plain) {
    w = 0;
    for (int k = 0; k < 8; ++k) {
      const double q = rint(((double)x[k] - (double)lo) / (double)s);
      w |= (uint32_t)(int)fmin(fmax(q, 0.0), 15.0) << (4 * k);
    }
  }
  return w;
}

// Scale of a row: the least bf16 value s with lo + 15 s >= hi.  Both
// operations round up, so that the result is never below the exact quotient
// and equals it where that is a bf16 value.
__device__ __forceinline__ uint32_t scale_bits(float lo, float hi) {
  float q;
  if (fmaxf(fabsf(lo), fabsf(hi)) < 1e37f) {
    q = __fdiv_ru(__fsub_ru(hi, lo), 15.f);
  } else {
    q = __double2float_ru(((double)hi - (double)lo) / 15.0);
  }
  const uint32_t b = __float_as_uint(q);
  return (b + 0xffffu) >> 16;
}

// Quantise rows of D values into their pages.  A group of lanes takes a row,
// 8 values a lane (16-byte loads), finds its least and largest value by
// shuffles and writes one 4-byte word of codes a lane.
template <int D>
struct RowLanes {
  static constexpr int kGroup = (D == 64) ? 8 : 16;     // lanes of a row (12 of 16 busy at 96)
  static constexpr int kBusy = D / 8;
  static constexpr int kRows = 32 / kGroup;             // rows of a warp
};

constexpr int kRowThreads = 256;
constexpr int kRowsAhead = 4;      // rows a lane has in flight

template <int D>
__global__ void __launch_bounds__(kRowThreads) write_kernel(const RowsParams p) {
  using L = RowLanes<D>;
  const int lane = threadIdx.x & 31;
  const int sub = lane % L::kGroup, grp = lane / L::kGroup;
  const bool busy = sub < L::kBusy;
  const int which = blockIdx.y;      // 0: K, 1: V
  const uint16_t *src = which ? p.V : p.K;
  const long long ts = which ? p.vt : p.kt, hs = which ? p.vh : p.kh;
  const long long rows = p.T * p.Hkv;
  const long long step = (long long)gridDim.x * (kRowThreads / 32) * L::kRows;
  long long row = ((long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5)) * L::kRows + grp;
  const uint32_t mask = 0xffffffffu;
  for (; row - grp < rows; row += step * kRowsAhead) {
    uint4 v[kRowsAhead];
    long long slot[kRowsAhead];
    int head[kRowsAhead];
#pragma unroll
    for (int a = 0; a < kRowsAhead; ++a) {
      const long long r = row + a * step;
      slot[a] = -1;
      v[a] = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        const long long t = r / p.Hkv;
        head[a] = (int)(r - t * p.Hkv);
        slot[a] = __ldg(p.slots + t);
        if (busy) v[a] = __ldcs(reinterpret_cast<const uint4 *>(src + t * ts + head[a] * hs) + sub);
      }
    }
#pragma unroll
    for (int a = 0; a < kRowsAhead; ++a) {
      const uint32_t u[4] = {v[a].x, v[a].y, v[a].z, v[a].w};
      float x[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[2 * k] = bf_lo(u[k]);
        x[2 * k + 1] = bf_hi(u[k]);
      }
      float lo = x[0], hi = x[0], bad = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        lo = fminf(lo, x[k]);
        hi = fmaxf(hi, x[k]);
        bad = fmaf(x[k], 0.f, bad);     // NaN once a value is not finite
      }
      if (!busy) {
        lo = INFINITY;
        hi = -INFINITY;
      }
#pragma unroll
      for (int o = 1; o < L::kGroup; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(mask, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(mask, hi, o));
        bad += __shfl_xor_sync(mask, bad, o);
      }
      if (slot[a] < 0) continue;
      if (slot[a] >= (long long)p.n_pages * kPage) {
        if (sub == 0) set_status(p.dev_status, DITANGO_ERR_BOUNDS);
        continue;
      }
      const long long page = slot[a] / kPage;
      const int at = (int)(slot[a] % kPage);
      uint8_t *base = p.data + ((size_t)page * p.Hkv + head[a]) * page_bytes(D);
      uint32_t sb = scale_bits(lo, hi);
      uint32_t w = codes8(x, lo, hi, __uint_as_float(sb << 16));
      uint32_t lb = __float_as_uint(lo) >> 16;
      if (!(bad == 0.f)) {              // an infinity or a NaN: the row stands for NaN
        w = 0;
        sb = lb = 0x7fff;
      }
      if (busy) *reinterpret_cast<uint32_t *>(base + which * (kPage * D / 2) + at * (D / 2) + sub * 4) = w;
      if (sub == 0) *reinterpret_cast<uint32_t *>(base + kPage * D + which * (kPage * 4) + at * 4) = sb | (lb << 16);
    }
  }
}

// Rows back to bf16: each value c * scale + least, formed in fp32 (the
// product of a 4-bit code and an 8-bit significand is exact) and rounded once.
template <int D>
__global__ void __launch_bounds__(kRowThreads) read_kernel(const RowsParams p) {
  constexpr int kLanes = D / 8;
  const int which = blockIdx.y;
  uint16_t *dst = which ? p.Vo : p.Ko;
  const long long ts = which ? p.vt : p.kt, hs = which ? p.vh : p.kh;
  const long long n = p.T * p.Hkv * kLanes, step = (long long)gridDim.x * kRowThreads;
  long long i0 = (long long)blockIdx.x * kRowThreads + threadIdx.x;
  for (; i0 < n; i0 += step * kRowsAhead) {
    uint32_t w[kRowsAhead], meta[kRowsAhead];
    uint16_t *out[kRowsAhead];
#pragma unroll
    for (int a = 0; a < kRowsAhead; ++a) {
      const long long i = i0 + a * step;
      out[a] = nullptr;
      if (i >= n) continue;
      const long long r = i / kLanes;
      const int sub = (int)(i - r * kLanes);
      const long long t = r / p.Hkv;
      const int h = (int)(r - t * p.Hkv);
      const long long slot = __ldg(p.slots + t);
      if (slot < 0) continue;
      if (slot >= (long long)p.n_pages * kPage) {
        set_status(p.dev_status, DITANGO_ERR_BOUNDS);
        continue;
      }
      const uint8_t *base = p.data + ((size_t)(slot / kPage) * p.Hkv + h) * page_bytes(D);
      const int at = (int)(slot % kPage);
      w[a] = *reinterpret_cast<const uint32_t *>(base + which * (kPage * D / 2) + at * (D / 2) + sub * 4);
      meta[a] = *reinterpret_cast<const uint32_t *>(base + kPage * D + which * (kPage * 4) + at * 4);
      out[a] = dst + t * ts + h * hs + sub * 8;
    }
#pragma unroll
    for (int a = 0; a < kRowsAhead; ++a) {
      if (!out[a]) continue;
      const float s = bf_lo(meta[a]), lo = bf_hi(meta[a]);
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = fmaf((float)((w[a] >> (4 * k)) & 15u), s, lo);
      uint4 o;
      o.x = pack_bf16x2(x[0], x[1]);
      o.y = pack_bf16x2(x[2], x[3]);
      o.z = pack_bf16x2(x[4], x[5]);
      o.w = pack_bf16x2(x[6], x[7]);
      __stcs(reinterpret_cast<uint4 *>(out[a]), o);
    }
  }
}

// ---------------------------------------------------------------- page summaries
// 8-bit codes of the mean key of every page that holds tokens [ctx, kv) of a
// request.  The sum over the page's tokens (all of them, not only the new
// ones) is formed from the codes in fp64, where it is exact, so that a page
// has one summary whatever order and number of calls filled it.
struct SummaryParams {
  int R, Hkv, max_blocks, n_pages;
  const int *ctx_len, *kv_len, *block_table;
  const uint8_t *data;
  signed char *codes;
  float *scale;
  int *dev_status;
};

constexpr int kSummaryThreads = 64;   // a thread takes one byte of codes, two channels

template <int D>
__global__ void __launch_bounds__(kSummaryThreads) page_summary_kernel(const SummaryParams p) {
  __shared__ uint32_t meta[kPage];
  __shared__ double part[2];
  const int h = blockIdx.x, r = blockIdx.y, tid = threadIdx.x;
  const int ctx = __ldg(p.ctx_len + r), kv = __ldg(p.kv_len + r);
  const long long most = (long long)p.max_blocks * kPage;
  if (ctx < 0 || kv < 0 || kv > most) {
    if (tid == 0) set_status(p.dev_status, DITANGO_ERR_BOUNDS);
    return;
  }
  if (kv <= ctx) return;
  const bool busy = tid < D / 2;
  const int last = (kv + kPage - 1) / kPage;
  for (int b = ctx / kPage + blockIdx.z; b < last; b += gridDim.z) {
    const int page = __ldg(p.block_table + (size_t)r * p.max_blocks + b);
    if (page < 0 || page >= p.n_pages) {
      if (tid == 0) set_status(p.dev_status, DITANGO_ERR_BOUNDS);
      continue;
    }
    const int n = min(kPage, kv - b * kPage);
    const uint8_t *base = p.data + ((size_t)page * p.Hkv + h) * page_bytes(D);
    meta[tid] = *reinterpret_cast<const uint32_t *>(base + kPage * D + tid * 4);
    __syncthreads();
    double a0 = 0.0, a1 = 0.0;
    if (busy) {
#pragma unroll 8
      for (int k = 0; k < n; ++k) {
        const uint32_t c = base[k * (D / 2) + tid];
        const double s = bf_lo(meta[k]), lo = bf_hi(meta[k]);
        a0 += (double)(c & 15u) * s + lo;
        a1 += (double)(c >> 4) * s + lo;
      }
    }
    double top = fmax(fabs(a0), fabs(a1));
    if (!(isfinite(a0) && isfinite(a1))) top = INFINITY;
    for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((tid & 31) == 0) part[tid >> 5] = top;
    __syncthreads();
    top = fmax(part[0], part[1]);
    int c0 = 0, c1 = 0;
    float sc = 0.f;
    if (top > 0.0 && top < INFINITY) {   // else, and where a key is not finite: codes 0, scale 0
      c0 = (int)rint(a0 * 127.0 / top);
      c1 = (int)rint(a1 * 127.0 / top);
      sc = (float)(top / (127.0 * n));
    }
    const size_t at = (size_t)page * p.Hkv + h;
    if (busy) reinterpret_cast<uint16_t *>(p.codes + at * D)[tid] = (uint16_t)((c0 & 255) | ((c1 & 255) << 8));
    if (tid == 0) p.scale[at] = sc;
    __syncthreads();
  }
}

}  // namespace hist

cudaError_t launch_block_tables(int R, int max_blocks, int max_tokens, int n_pages, const int *ctx_len,
                                const int *new_len, const int *free_pages, int n_free, int *block_table,
                                int *kv_len, int *q_off, long long *slot_map, int *pages_used,
                                int *dev_status, int num_sms, cudaStream_t stream) {
  hist::TablesParams p{R, max_blocks, max_tokens, n_pages, n_free, ctx_len, new_len, free_pages,
                       block_table, kv_len, q_off, slot_map, pages_used, dev_status};
  long long grid = (max_tokens + hist::kTabThreads - 1) / hist::kTabThreads;
  if (grid < 1) grid = 1;
  if (grid > num_sms) grid = num_sms;
  hist::tables_kernel<<<(int)grid, hist::kTabThreads, 2 * (R + 1) * sizeof(int), stream>>>(p);
  return cudaGetLastError();
}

#define DITANGO_BY_D(d, CALL)        \
  switch (d) {                       \
    case 64: CALL(64); break;        \
    case 96: CALL(96); break;        \
    case 128: CALL(128); break;      \
    default: return cudaErrorInvalidValue; \
  }

cudaError_t launch_kv4_rows(bool write, long long T, int Hkv, int d, int n_pages, const uint16_t *K,
                            const uint16_t *V, uint16_t *Ko, uint16_t *Vo, const int64_t *k_strides,
                            const int64_t *v_strides, const long long *slots, uint8_t *data,
                            int *dev_status, int num_sms, cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  hist::RowsParams p{T, Hkv, n_pages, K, V, Ko, Vo, k_strides[0], k_strides[1], v_strides[0],
                     v_strides[1], slots, data, dev_status};
  const long long lanes = T * Hkv * (write ? (d == 64 ? 8 : 16) : d / 8);
  long long grid = (lanes + hist::kRowThreads - 1) / hist::kRowThreads;
  if (grid > 4LL * num_sms) grid = 4LL * num_sms;
  const dim3 g((unsigned)grid, 2);
#define DITANGO_ROWS(D)                                                          \
  if (write)                                                                     \
    hist::write_kernel<D><<<g, hist::kRowThreads, 0, stream>>>(p);               \
  else                                                                           \
    hist::read_kernel<D><<<g, hist::kRowThreads, 0, stream>>>(p)
  DITANGO_BY_D(d, DITANGO_ROWS)
#undef DITANGO_ROWS
  return cudaGetLastError();
}

cudaError_t launch_kv4_summary(int R, int Hkv, int d, int max_blocks, int n_pages, const int *ctx_len,
                               const int *kv_len, const int *block_table, const uint8_t *data,
                               signed char *codes, float *scale, int *dev_status, cudaStream_t stream) {
  hist::SummaryParams p{R, Hkv, max_blocks, n_pages, ctx_len, kv_len, block_table, data, codes, scale,
                        dev_status};
  const dim3 g((unsigned)Hkv, (unsigned)R, (unsigned)(max_blocks < 32 ? max_blocks : 32));
#define DITANGO_SUMMARY(D) hist::page_summary_kernel<D><<<g, hist::kSummaryThreads, 0, stream>>>(p)
  DITANGO_BY_D(d, DITANGO_SUMMARY)
#undef DITANGO_SUMMARY
  return cudaGetLastError();
}

}  // namespace ditango
