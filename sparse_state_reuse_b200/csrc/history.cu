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
// is latency-bound: 6.2 us for the 64 single tokens of a step and 6.4 us for 512
// requests with up to 400 new tokens each, replayed in a graph, most of it launch
// and two dependent reads; the bytes are below 1 MB.
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
    // what a request does not need cannot be short
    const bool fits = ok && (n == 0 || it + n <= cap) && (e == 0 || ip + e <= p.n_free);
    off[r] = (int)min(it, cap);
    // a request that does not fit takes no page: its entry says so
    first[r] = fits ? (e > 0 ? (int)ip : 0) : -1;
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
  for (long long at = blockIdx.x * kTabThreads + tid; at < p.max_tokens; at += gridDim.x * kTabThreads) {
    const int t = (int)at;            // (past max_tokens, a step on, the index may pass 2^31)
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
  uint32_t rows;                // T * Hkv, below 2^27
  FastDiv heads;
  int Hkv, n_pages;
  const uint16_t *K, *V;
  uint16_t *Ko, *Vo;
  long long kt, kh, vt, vh;     // token and head strides, elements
  const long long *slots;
  uint8_t *data;
  int *dev_status;
};

// Codes of 8 values of a row: c = round to nearest even of (x - lo) / s, as
// exact arithmetic gives it.  Values that lie exactly between two codes are
// common (x, lo and s are bf16: one in 200), so the quotient itself is formed
// with correct rounding, by one step of Newton's iteration for the quotient on
// t = x - lo with the correctly rounded reciprocal of s:
//   q = t r,  q' = q + (t - q s) r.
// A quotient that is k + 1/2 then comes out as that (it is a fp32 number), and
// one that is not stays on its side: t and s being multiples of powers of two
// with 24 and 8 bits, it is at least 2^-24 of itself away.  All of this needs t
// to be exact.  Where |x| < |lo|, t + lo - x is what t lacks (the sum of a larger
// and a smaller number and its remainder), and `bad` collects it.  Where |x| >= |lo|
// it is not (both roundings can cancel: least 2^-30, x 1.5), but there t is exact as
// long as |x| is at most 2^14 |lo|: it is a multiple of lo's last bit and 2^23 of
// those at most.  Rows whose least value is smaller, groups with an inexact t, and
// scales outside fp32's comfortable range take the difference in fp64, with its
// remainder: against the middle between two codes (13 bits), and if it is there, by
// the remainder's sign.
__device__ __noinline__ uint32_t codes8_wide(uint4 v, float lo, float s) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  uint32_t w = 0;
  for (int k = 0; k < 8; ++k) {
    const double x = (k & 1) ? bf_hi(u[k >> 1]) : bf_lo(u[k >> 1]), y = -(double)lo;
    const double t = x + y, z = t - x, rest = (x - (t - z)) + (y - z);     // t + rest = x - lo
    const double c = fmin(fmax(floor(t / (double)s), 0.0), 15.0), middle = (c + 0.5) * (double)s;
    const bool up = t > middle || (t == middle && (rest > 0.0 || (rest == 0.0 && ((int)c & 1))));
    w |= (uint32_t)min((int)c + (up ? 1 : 0), 15) << (4 * k);
  }
  return w;
}

__device__ __forceinline__ uint32_t codes8(uint4 v, float lo, float s, float inv, float &bad) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  const float kRound = 12582912.0f;   // 1.5 * 2^23: adding it rounds to an integer, in the low bits
  const uint64_t nlo2 = f2(-lo, -lo), lo2 = f2(lo, lo), inv2 = f2(inv, inv), ns2 = f2(-s, -s),
                 round2 = f2(kRound, kRound), minus1 = f2(-1.f, -1.f);
  uint32_t w = 0u - 0x4b400000u * 0x11111111u;   // the exponents of the eight sums, taken off
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint64_t x = f2(bf_lo(u[k]), bf_hi(u[k]));
    const uint64_t t = add2(x, nlo2);
    const uint64_t back = fma2(x, minus1, add2(t, lo2));
    const uint64_t q = mul2(t, inv2);
    const uint64_t q1 = fma2(fma2(q, ns2, t), inv2, q);
    float a, b, e, f;
    unf2(add2(q1, round2), a, b);
    unf2(back, e, f);
    bad = fmaxf(bad, fmaxf(fabsf(e), fabsf(f)));
    w += (__float_as_uint(a) << (8 * k)) + (__float_as_uint(b) << (8 * k + 4));
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
    q = __double2float_ru(__ddiv_ru(__dsub_ru((double)hi, (double)lo), 15.0));
  }
  const uint32_t b = __float_as_uint(q);
  return (b + 0xffffu) >> 16;
}

// Quantise rows of D values into their pages.  Four lanes take a row, D / 4
// values each (16-byte loads), so that all lanes are busy for every d and the
// address arithmetic is spread over 16 to 32 values; least and largest value
// are found with packed bf16 minima of (x, -x) and two shuffles.
// 28800 tokens of 24 heads of 96: 89 us for 336 MB, 3.8 TB/s.  Bound by issue
// (65% of the slots, the exact quotients most of it) and by the loads' latency
// with 28 warps an SM; the next row fetched ahead (90 us), five and six blocks an
// SM (spills) and one branch for the inexact groups of a row (93 us) were slower.
constexpr int kRowThreads = 256;

__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {   // NaN if either is
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) write_kernel(const RowsParams p) {
  constexpr int kLoads = D / 32;                        // 16-byte loads of a lane and row
  const int sub = threadIdx.x & 3;
  const int which = blockIdx.y;      // 0: K, 1: V
  const uint16_t *src = which ? p.V : p.K;
  const long long ts = which ? p.vt : p.kt, hs = which ? p.vh : p.kh;
  const uint32_t step = gridDim.x * (kRowThreads / 4);
  const uint32_t padded = (p.rows + 7u) & ~7u;          // whole warps stay together
  uint32_t row = blockIdx.x * (kRowThreads / 4) + threadIdx.x / 4;
  uint4 v[kLoads];
  long long slot = -1;
  int head = 0;
  auto fetch = [&](uint32_t r) {
    slot = -1;
    if (r < p.rows) {
      const uint32_t t = p.heads.div(r);
      head = (int)(r - t * p.heads.d);
      slot = __ldg(p.slots + t);
      const uint4 *at = reinterpret_cast<const uint4 *>(src + t * ts + head * hs + sub * (D / 4));
#pragma unroll
      for (int k = 0; k < kLoads; ++k) v[k] = __ldg(at + k);
    } else {
#pragma unroll
      for (int k = 0; k < kLoads; ++k) v[k] = make_uint4(0, 0, 0, 0);
    }
  };
  for (; row < padded; row += step) {
    fetch(row);
    uint32_t mn = min_bf16x2(min_bf16x2(v[0].x, v[0].y), min_bf16x2(v[0].z, v[0].w));
    uint32_t mx = max_bf16x2(max_bf16x2(v[0].x, v[0].y), max_bf16x2(v[0].z, v[0].w));
#pragma unroll
    for (int k = 1; k < kLoads; ++k) {
      mn = min_bf16x2(mn, min_bf16x2(min_bf16x2(v[k].x, v[k].y), min_bf16x2(v[k].z, v[k].w)));
      mx = max_bf16x2(mx, max_bf16x2(max_bf16x2(v[k].x, v[k].y), max_bf16x2(v[k].z, v[k].w)));
    }
    // (least, -largest) in one register
    const uint32_t neg = mx ^ 0x80008000u;
    uint32_t both = min_bf16x2(__byte_perm(mn, neg, 0x5410), __byte_perm(mn, neg, 0x7632));
    both = min_bf16x2(both, __shfl_xor_sync(0xffffffffu, both, 1));
    both = min_bf16x2(both, __shfl_xor_sync(0xffffffffu, both, 2));
    if (slot < 0) continue;
    if (slot >= (long long)p.n_pages * kPage) {
      if (sub == 0) set_status(p.dev_status, DITANGO_ERR_BOUNDS);
      continue;
    }
    const float lo = bf_lo(both), hi = -bf_hi(both);
    const bool finite = fabsf(lo) < INFINITY && fabsf(hi) < INFINITY;   // false for NaN
    uint32_t sb = scale_bits(lo, hi);
    const float s = __uint_as_float(sb << 16);
    const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
    const bool fine =
        (s > 1e-30f && s < 1e30f && (lo == 0.f || fabsf(hi) <= 16384.f * fabsf(lo))) || s == 0.f;
    uint32_t w[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      float bad = fine ? 0.f : 1.f;
      w[k] = codes8(v[k], lo, s, inv, bad);
      if (bad != 0.f && finite && s > 0.f) w[k] = codes8_wide(v[k], lo, s);
    }
    uint32_t lb = both & 0xffffu;
    if (!finite) {                    // an infinity or a NaN: the row stands for NaN
#pragma unroll
      for (int k = 0; k < kLoads; ++k) w[k] = 0u;
      sb = lb = 0x7fffu;
    }
    const long long page = slot / kPage;
    const int at = (int)(slot % kPage);
    uint8_t *base = p.data + ((size_t)page * p.Hkv + head) * page_bytes(D);
    uint32_t *codes = reinterpret_cast<uint32_t *>(base + which * (kPage * D / 2) + at * (D / 2) + sub * (D / 8));
    if constexpr (kLoads == 4) {
      *reinterpret_cast<uint4 *>(codes) = make_uint4(w[0], w[1], w[2], w[3]);
    } else if constexpr (kLoads == 2) {
      *reinterpret_cast<uint2 *>(codes) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int k = 0; k < kLoads; ++k) codes[k] = w[k];
    }
    if (sub == 0) *reinterpret_cast<uint32_t *>(base + kPage * D + which * (kPage * 4) + at * 4) = sb | (lb << 16);
  }
}

constexpr int kRowsAhead = 2;      // units of a lane of read_kernel, a block of threads apart

// Eight codes as values, in order: the code goes into the significand of 2^23
// where its bits stand, at 1 or 16 times its size, is taken off again (exact),
// and meets the scale, or a 16th of it (exact: a bf16 number), in one FMA.
__device__ __forceinline__ uint4 values8(uint32_t w, uint64_t s2, uint64_t lo2) {
  const uint64_t minus = f2(-8388608.f, -8388608.f);
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t v = w >> (8 * k);
    const uint64_t c = f2(__uint_as_float((v & 0x0fu) | 0x4b000000u), __uint_as_float((v & 0xf0u) | 0x4b000000u));
    float a, b;
    unf2(fma2(add2(c, minus), s2, lo2), a, b);
    o[k] = pack_bf16x2(a, b);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Rows back to bf16: each value c * scale + least, formed in fp32 (the
// product of a 4-bit code and an 8-bit significand is exact) and rounded once.
// A lane takes 16 values, so that the address arithmetic, most of the work, is
// done once for two stores of 16 bytes.  28800 tokens of 24 heads of 96: 66 us for
// 336 MB, 5.1 TB/s; bound by the writes (four units a lane a grid apart 82 us, a
// block apart 68 us, two 66 us, one 83 us).
template <int D>
__global__ void __launch_bounds__(kRowThreads) read_kernel(const RowsParams p) {
  constexpr uint32_t kLanes = D / 16;
  const int which = blockIdx.y;
  uint16_t *dst = which ? p.Vo : p.Ko;
  const long long ts = which ? p.vt : p.kt, hs = which ? p.vh : p.kh;
  const uint32_t n = p.rows * kLanes, step = gridDim.x * kRowThreads * kRowsAhead;
  for (uint32_t i0 = blockIdx.x * kRowThreads * kRowsAhead + threadIdx.x; i0 < n; i0 += step) {
    uint2 w[kRowsAhead];
    uint32_t meta[kRowsAhead];
    uint16_t *out[kRowsAhead];
#pragma unroll
    for (int a = 0; a < kRowsAhead; ++a) {
      const uint32_t i = i0 + a * kRowThreads;
      out[a] = nullptr;
      if (i >= n) continue;
      const uint32_t r = i / kLanes;
      const int sub = (int)(i - r * kLanes);
      const uint32_t t = p.heads.div(r);
      const int h = (int)(r - t * p.heads.d);
      const long long slot = __ldg(p.slots + t);
      if (slot < 0) continue;
      if (slot >= (long long)p.n_pages * kPage) {
        set_status(p.dev_status, DITANGO_ERR_BOUNDS);
        continue;
      }
      const uint32_t page = (uint32_t)(slot / kPage), at = (uint32_t)slot % kPage;
      const uint8_t *base = p.data + ((size_t)page * p.Hkv + h) * page_bytes(D);
      w[a] = *reinterpret_cast<const uint2 *>(base + which * (kPage * D / 2) + at * (D / 2) + sub * 8);
      meta[a] = *reinterpret_cast<const uint32_t *>(base + kPage * D + which * (kPage * 4) + at * 4);
      out[a] = dst + t * ts + h * hs + sub * 16;
    }
#pragma unroll
    for (int a = 0; a < kRowsAhead; ++a) {
      if (!out[a]) continue;
      const float s = bf_lo(meta[a]), lo = bf_hi(meta[a]);
      const uint64_t s2 = f2(s, s * 0.0625f), lo2 = f2(lo, lo);
      __stcs(reinterpret_cast<uint4 *>(out[a]), values8(w[a].x, s2, lo2));
      __stcs(reinterpret_cast<uint4 *>(out[a]) + 1, values8(w[a].y, s2, lo2));
    }
  }
}

// ---------------------------------------------------------------- page summaries
// 8-bit codes of the mean key of every page that holds tokens [ctx, kv) of a
// request.  28800 tokens of 24 heads of 96: 84 us (36 MB, 6 us at the copy rate), the
// last pages of 64 requests, 8 heads of 128: 12 us; bound by its byte loads and fp64,
// one page after the other.  The sum over the page's tokens (all of them, not only the new
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
  long long grid = ((long long)max_tokens + hist::kTabThreads - 1) / hist::kTabThreads;
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
  hist::RowsParams p{(uint32_t)(T * Hkv), FastDiv((uint32_t)Hkv), Hkv, n_pages, K, V, Ko, Vo, k_strides[0], k_strides[1], v_strides[0],
                     v_strides[1], slots, data, dev_status};
  const long long lanes = write ? T * Hkv * 4 : (T * Hkv * (d / 16) + hist::kRowsAhead - 1) / hist::kRowsAhead;
  long long grid = (lanes + hist::kRowThreads - 1) / hist::kRowThreads;
  // Writing: eight blocks a SM that go on (two to eight: 88 us for 28800 tokens of
  // 24 heads of 96 channels, one block for every 64 rows 96).  Reading: blocks of
  // one round, whose writes stay near one another (66 us; eight a SM 78).
  const long long most = (write ? 8LL : 64LL) * num_sms;
  if (grid > most) grid = most;
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
