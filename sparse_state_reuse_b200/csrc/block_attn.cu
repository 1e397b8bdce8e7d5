// Attention of 128-query blocks over the 64-key blocks that each selected.
//
// For query block i of (b, h) and the list sel[b][h / G][i]: S = Q K^T scale
// over the keys of the listed blocks, O = softmax(S) V, lse = log sum exp(S),
// by an online softmax over tiles of two listed blocks (128 keys).  Q, K and V
// are staged by TMA, a listed block as one 64-row box, so that a list costs the
// tile nothing; both products run on tcgen05 with S, P and O in TMEM.
//
// One block of threads takes one query block, and two of them share an SM
// (256 TMEM columns and at most 113 KB each): while one exponentiates its
// scores the other's products have the tensor pipe, which is what a second
// query tile in one block would do, but neither waits for the other, and one's
// start and end run under the other's loop.  Query blocks have lists of their
// own, so there are no key tiles to share between them.
//   warps 0-3  softmax, a thread a row, and the epilogue
//   warp  4    TMEM owner, MMA issuer (one thread)
//   warp  5    TMA producer
// TMEM: S [0, 128), O [128, 128 + d); the bf16 P overwrites the first 64
// columns of S and feeds the second product from there.
// Bound: 4 * 128 * 128 * d flops a tile against the exponentials of 128 * 128
// scores, and 2 * 128 * d * 2 bytes of L2 reads a tile.  600 query blocks of 40
// heads of 128 over 150 key blocks each: 12.7 ms at the boost clock, 13.4 to 14.9
// under the power limit, 1190 and 1020 to 1130 TFLOP/s (62 to 73% of the measured
// bf16 rate; the dense kernel of this library reaches 67%).  Register splits of
// 192/64 and 208/48 were slower or the same.

#include "blocks.cuh"

namespace ditango {
namespace battn {

constexpr int BM = kQBlock;          // query rows
constexpr int BN = 2 * kPage;        // keys of a tile
constexpr int kThreads = 256;
constexpr int kLaunchRegs = 128;     // 65536 / (2 * 256)
// A softmax thread holds a row of 128 scores.  The two shares are what the
// block is launched with: 128 * 200 + 128 * 56 = 256 * 128.
constexpr int kSoftmaxRegs = 200, kControlRegs = 56;
static_assert(128 * kSoftmaxRegs + 128 * kControlRegs == kThreads * kLaunchRegs, "register split");
constexpr int kTmemCols = 256;

template <int D>
struct Cfg {
  static constexpr int NCH = (D + 63) / 64;          // 64-column chunks
  static constexpr int CHUNK = 128 * 128;            // 128 rows of 128 bytes
  static constexpr int HALF = CHUNK / 2;             // one key block of a chunk
  static constexpr int TILE = NCH * CHUNK;
  static constexpr int OFF_Q = 0, OFF_K = TILE, OFF_V = 2 * TILE, OFF_BAR = 3 * TILE;
  static constexpr int USED = OFF_BAR + 128;
  // above 76 KB, so that no third block comes to the SM (its TMEM columns are taken)
  static constexpr int SMEM = (USED + 1024 > 100 * 1024) ? USED + 1024 : 100 * 1024;
  static_assert(SMEM <= 113 * 1024, "two blocks an SM");
  static_assert(TILE >= 4 * 4096, "the epilogue stages rows in the Q tile");
};

struct Params {
  int H, G, Hkv, Nq, Nk, n_q, n_k, room;
  const int *sel, *count, *k_len;
  float scale_log2;
  void *out;
  int out_fp32;
  long long osb, osh, osn;
  float *out_lse;                    // (b, h, n) strides below, or null
  long long lsb, lsh, lsn;
  int *dev_status;
  long long wait_limit_ns;
  int split;                         // blocks of threads of a query block (a cluster)
};

// The list of one query block.
struct List {
  const int *sel;
  int n, n_k, keys;
  // valid keys of entry e: 0 for entries past the end or out of range
  __device__ __forceinline__ int at(int e, int &block) const {
    block = e < n ? __ldg(sel + e) : -1;
    if (block < 0 || block >= n_k) return 0;
    return max(0, min(kPage, keys - block * kPage));
  }
};

// Clusters: where there are few query blocks, up to eight blocks of threads take
// the parts of one list, each its own online softmax, and join them through one
// another's shared memory.
constexpr int kMaxSplit = 8;

// Every thread of the cluster comes to both, whatever happened before.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 cluster_ld4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 cluster_ld2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

template <int D, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 2)
block_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Params p) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sQ = sbase + C::OFF_Q, sK = sbase + C::OFF_K, sV = sbase + C::OFF_V;
  const uint32_t bar = sbase + C::OFF_BAR;
  const uint32_t q_full = bar, k_full = bar + 8, k_empty = bar + 16, v_full = bar + 24, v_empty = bar + 32,
                 s_full = bar + 40, p_full = bar + 48, o_full = bar + 56;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_BAR + 64);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_BAR + 68);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  WaitCtl ctl{abort_flag, p.dev_status, p.wait_limit_ns};
  const int split = SPLIT ? p.split : 1, rank = SPLIT ? (int)blockIdx.x % split : 0;
  const int i = (int)blockIdx.x / split, h = blockIdx.y, b = blockIdx.z, hk = h / p.G;

  List list;
  {
    const size_t at = ((size_t)b * p.Hkv + hk) * p.n_q + i;
    const int n = __ldg(p.count + at);
    list.n = max(0, min(n, p.room));
    list.sel = p.sel + at * p.room;
    list.n_k = p.n_k;
    list.keys = p.Nk;
    if (p.k_len) list.keys = max(0, min(p.Nk, __ldg(p.k_len + b)));
    if (threadIdx.x == 0 && n != list.n) set_status(p.dev_status, DITANGO_ERR_BOUNDS);
  }
  if constexpr (SPLIT) {
    // this block's part: whole tiles
    const int tiles = (list.n + 1) / 2;
    const int t0 = (int)((long long)tiles * rank / split), t1 = (int)((long long)tiles * (rank + 1) / split);
    list.sel += 2 * t0;
    list.n = min(list.n, 2 * t1) - 2 * t0;
  }
  const int T = (list.n + 1) / 2;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(k_full, 1);
    mbar_init(k_empty, 1);
    mbar_init(v_full, 1);
    mbar_init(v_empty, 1);
    mbar_init(s_full, 1);
    mbar_init(p_full, 4);      // one arrival per softmax warp
    mbar_init(o_full, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 4) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  if (warp == 5 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kControlRegs));
    if (warp == 5 && T > 0) {
      // ---------------------------------------------------------- producer
      const bool leader = elect_one();
      bool ok = true;
      int armed = 0;           // tiles of K armed; V the same or one fewer
      int v_armed = 0;
      if (leader) {
        mbar_arrive_expect_tx(q_full, C::TILE);
        for (int c = 0; c < C::NCH; ++c)
          tma_load_4d(sQ + c * C::CHUNK, &tmQ, q_full, c * 64, i * BM, h, b);
      }
      int b0, b1;
      int n0 = list.at(0, b0), n1 = list.at(1, b1);
      for (int t = 0; t < T && ok; ++t) {
        // the next entries are read under this tile's waits
        int c0, c1;
        const int m0 = list.at(2 * t + 2, c0), m1 = list.at(2 * t + 3, c1);
        if (lane == 0 && ((b0 < 0 || b0 >= p.n_k) || (2 * t + 1 < list.n && (b1 < 0 || b1 >= p.n_k))))
          set_status(p.dev_status, DITANGO_ERR_BOUNDS);
        const uint32_t bytes = ((n0 > 0) + (n1 > 0)) * C::NCH * C::HALF;
        if (!(ok = wait_warp(k_empty, (t & 1) ^ 1, ctl))) break;
        if (leader) {
          mbar_arrive_expect_tx(k_full, bytes);
          for (int c = 0; c < C::NCH; ++c) {
            if (n0 > 0) tma_load_4d(sK + c * C::CHUNK, &tmK, k_full, c * 64, b0 * kPage, hk, b);
            if (n1 > 0) tma_load_4d(sK + c * C::CHUNK + C::HALF, &tmK, k_full, c * 64, b1 * kPage, hk, b);
          }
        }
        ++armed;
        if (!(ok = wait_warp(v_empty, (t & 1) ^ 1, ctl))) break;
        if (leader) {
          mbar_arrive_expect_tx(v_full, bytes);
          for (int c = 0; c < C::NCH; ++c) {
            if (n0 > 0) tma_load_4d(sV + c * C::CHUNK, &tmV, v_full, c * 64, b0 * kPage, hk, b);
            if (n1 > 0) tma_load_4d(sV + c * C::CHUNK + C::HALF, &tmV, v_full, c * 64, b1 * kPage, hk, b);
          }
        }
        ++v_armed;
        b0 = c0;
        b1 = c1;
        n0 = m0;
        n1 = m1;
      }
      // every load issued lands before the warp exits, on both paths
      volatile int never = 0;
      WaitCtl drain{&never, nullptr, 100000000LL};
      wait_bounded(q_full, 0, drain);
      if (armed > 0) wait_bounded(k_full, (armed - 1) & 1, drain);
      if (v_armed > 0) wait_bounded(v_full, (v_armed - 1) & 1, drain);
    } else if (warp == 4 && T > 0) {
      // ---------------------------------------------------------- MMA issuer
      const bool leader = elect_one();
      constexpr uint32_t idesc_qk = idesc_bf16_f32(BM, BN, 0, 0);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(BM, D, 0, 1);
      // V is MN-major: chunks of d are CHUNK apart
      auto commit = [&](uint32_t at) {
        at = pinned(at);
        if (leader) tc_commit(at);
      };
      bool ok = wait_warp(q_full, 0, ctl);
      for (int t = 0; t < T && ok; ++t) {
        if (!(ok = wait_warp(k_full, t & 1, ctl))) break;
        tc_fence_after();
        const uint64_t dQ = pinned(smem_desc_sw128(sQ, 16, 1024)), dK = pinned(smem_desc_sw128(sK, 16, 1024));
        if (leader) {
          // S = Q K^T.  P of the tile before lives in S: its product was
          // issued before, and one thread's products run in order.
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t off = (uint64_t)(((kk >> 2) * C::CHUNK + (kk & 3) * 32) >> 4);
            mma_ss(tmem, dQ + off, dK + off, idesc_qk, kk > 0);
          }
        }
        commit(s_full);
        commit(k_empty);
        if (!(ok = wait_warp(v_full, t & 1, ctl))) break;
        if (!(ok = wait_warp(p_full, t & 1, ctl))) break;
        tc_fence_after();
        const uint64_t dV = pinned(smem_desc_sw128(sV, C::CHUNK, 1024));
        const uint32_t more = pinned(t > 0 ? 1u : 0u);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            mma_ts(tmem + 128, tmem + kk * 8, dV + (uint64_t)((kk * 2048) >> 4), idesc_pv, kk > 0 ? 1u : more);
        }
        commit(v_empty);
        if (t + 1 == T) commit(o_full);
      }
      // what was issued ends before TMEM is released, on both paths
      volatile int never = 0;
      WaitCtl drain{&never, nullptr, 100000000LL};
      if (!ok) commit(o_full);
      wait_bounded(o_full, 0, drain);
      __syncwarp();
    }
    if (warp == 4) {
      named_bar_sync(1, kThreads);
      tc_fence_after();
      tmem_dealloc(tmem, kTmemCols);
    } else {
      tc_fence_before();
      named_bar_arrive(1, kThreads);
    }
    if constexpr (SPLIT) {
      cluster_sync();
      cluster_sync();
    }
    return;
  }

  // -------------------------------------------------------------- softmax
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
  const int r = threadIdx.x;                    // row of the block = TMEM lane
  const uint32_t tS = tmem + ((uint32_t)(warp * 32) << 16);
  const uint32_t tO = tS + 128;
  const float sl2 = p.scale_log2;
  float m_used = -INFINITY, l = 0.f;
  bool ok = true;
  for (int t = 0; t < T; ++t) {
    int b0, b1;
    const int n0 = list.at(2 * t, b0), n1 = list.at(2 * t + 1, b1);
    if (!(ok = wait_bounded(s_full, t & 1, ctl))) break;
    tc_fence_after();
    uint32_t sv[BN];
#pragma unroll
    for (int c = 0; c < BN / 16; ++c) tmem_ld16p(tS + c * 16, &sv[c * 16]);
    tc_wait_ld();
    const bool partial = n0 + n1 < BN;
    if (partial) {
#pragma unroll
      for (int c = 0; c < BN; ++c)
        if (c < kPage ? c >= n0 : c - kPage >= n1) sv[c] = __float_as_uint(-INFINITY);
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
        max3(max3(m8[0], m8[1], m8[2]), max3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7])) * sl2;
    if (t == 0) {
      m_used = mx2;
    } else {
      // S of this tile is complete, and with it every product issued before:
      // O may be rescaled (only when a maximum grew by more than 2^8)
      const bool need = mx2 > m_used + kRescaleLog2;
      if (__any_sync(0xffffffffu, need)) {
        const float m_new = need ? mx2 : m_used;
        const float alpha = need ? fast_ex2(m_used - m_new) : 1.f;
        l *= alpha;
        m_used = m_new;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          tmem_ld32(tO + c * 32, v);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
          tmem_st32(tO + c * 32, v);
        }
      }
    }
    const float neg = m_used > -INFINITY ? -m_used : 0.f;   // no key so far: exponentiate against 0
    uint64_t sl2x2 = f2(sl2, sl2);
    const uint64_t negx2 = f2(neg, neg);
    if (__any_sync(0xffffffffu, fabsf(neg) > kHuge)) {
#pragma unroll
      for (int c = 0; c < BN; ++c) sv[c] = __float_as_uint(__fmul_rn(__uint_as_float(sv[c]), sl2));
      sl2x2 = f2(1.f, 1.f);
    }
    uint64_t lsum0 = 0, lsum1 = 0;
#pragma unroll
    for (int g8 = 0; g8 < BN / 16; ++g8) {
      uint32_t pk[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = g8 * 16 + 2 * e;
        float xa, xb;
        unf2(fma2(f2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), sl2x2, negx2), xa, xb);
        const float a = fast_ex2(xa), bb = fast_ex2(xb);
        if (e & 1) lsum1 = add2(lsum1, f2(a, bb)); else lsum0 = add2(lsum0, f2(a, bb));
        pk[e] = pack_bf16x2(a, bb);
      }
      tmem_st8(tS + g8 * 8, pk[0], pk[1], pk[2], pk[3], pk[4], pk[5], pk[6], pk[7]);
    }
    {
      float s0, s1, s2, s3;
      unf2(lsum0, s0, s1);
      unf2(lsum1, s2, s3);
      l += (s0 + s1) + (s2 + s3);
    }
    if (partial) {
      // V rows of masked keys: their probabilities are 0, but the row (past
      // the valid length, or left from another tile) may hold anything
      if (!(ok = wait_bounded(v_full, t & 1, ctl))) break;
      if (r < kPage ? r >= n0 : r - kPage >= n1) {
#pragma unroll
        for (int c = 0; c < C::NCH; ++c)
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<uint4 *>(smem + C::OFF_V + c * C::CHUNK + r * 128 + q * 16) =
                make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async();
    }
    tc_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(p_full);
  }
  if (ok && T > 0) ok = wait_bounded(o_full, 0, ctl);
  if constexpr (SPLIT) {
    // every product is done (or this block gave up and adds nothing): Q, K and V
    // make room for its O, m and l
    constexpr int kRow = D + 4;                 // floats: rows of neighbouring lanes lie in other banks
    static_assert(BM * kRow * 4 + BM * 8 <= 3 * C::TILE, "O, m and l in the place of Q, K and V");
    float *stage = reinterpret_cast<float *>(smem + C::OFF_Q);
    const bool any = ok && T > 0 && !(!(l > 0.f) && l == l);
    __syncwarp();
    tc_fence_after();
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      uint32_t ov[32];
      if (T > 0) {
        tmem_ld32(tO + c * 32, ov);
        tc_wait_ld();
      }
      float4 *dst = reinterpret_cast<float4 *>(stage + r * kRow + c * 32);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        dst[q] = any ? make_float4(__uint_as_float(ov[4 * q]), __uint_as_float(ov[4 * q + 1]),
                                   __uint_as_float(ov[4 * q + 2]), __uint_as_float(ov[4 * q + 3]))
                     : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    reinterpret_cast<float2 *>(stage + BM * kRow)[r] = any ? make_float2(m_used, l) : make_float2(-INFINITY, 0.f);
    tc_fence_before();
    named_bar_arrive(1, kThreads);
    cluster_sync();
    // the rows are shared out; the parts are joined in the order of the list
    const int mine = BM / split;
    constexpr int kVec = D / 4;
    const uint32_t from = smem_u32(stage);
    constexpr int U = 4, EB = 4;                // groups of a thread and parts in flight together
    for (int x0 = r; x0 < mine * kVec; x0 += BM * U) {
      float mt[U], lt[U];
      float4 v[U];
#pragma unroll
      for (int w = 0; w < U; ++w) {
        mt[w] = -INFINITY;
        lt[w] = 0.f;
        v[w] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      for (int e0 = 0; e0 < split; e0 += EB) {
        float2 ml[U][EB];
        float4 o[U][EB];
#pragma unroll
        for (int w = 0; w < U; ++w)
#pragma unroll
          for (int e = 0; e < EB; ++e) {
            const int x = x0 + w * BM, row = rank * mine + x / kVec, ch = (x % kVec) * 4;
            ml[w][e] = make_float2(-INFINITY, 0.f);
            o[w][e] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (x < mine * kVec && e0 + e < split) {
              const uint32_t peer = cluster_map(from, e0 + e);
              ml[w][e] = cluster_ld2(peer + BM * kRow * 4 + row * 8);
              o[w][e] = cluster_ld4(peer + (row * kRow + ch) * 4);
            }
          }
#pragma unroll
        for (int w = 0; w < U; ++w)
#pragma unroll
          for (int e = 0; e < EB; ++e) {
            const float mn = fmaxf(mt[w], ml[w][e].x), less = mn > -INFINITY ? mn : 0.f;
            const float f0 = fast_ex2(mt[w] - less), f1 = fast_ex2(ml[w][e].x - less);
            const float4 y = o[w][e];
            lt[w] = lt[w] * f0 + ml[w][e].y * f1;
            v[w] = make_float4(v[w].x * f0 + y.x * f1, v[w].y * f0 + y.y * f1, v[w].z * f0 + y.z * f1, v[w].w * f0 + y.w * f1);
            mt[w] = mn;
          }
      }
#pragma unroll
      for (int w = 0; w < U; ++w) {
        const int x = x0 + w * BM, ch = (x % kVec) * 4, at = i * BM + rank * mine + x / kVec;
        if (x >= mine * kVec || at >= p.Nq) continue;
        const float inv = lt[w] > 0.f ? 1.f / lt[w] : (lt[w] == lt[w] ? 0.f : lt[w]);
        const float4 z = make_float4(v[w].x * inv, v[w].y * inv, v[w].z * inv, v[w].w * inv);
        const long long to = b * p.osb + h * p.osh + at * p.osn + ch;
        if (p.out_fp32)
          *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + to) = z;
        else
          *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + to) =
              make_uint2(pack_bf16x2(z.x, z.y), pack_bf16x2(z.z, z.w));
        if (ch == 0 && p.out_lse)
          p.out_lse[b * p.lsb + h * p.lsh + at * p.lsn] =
              lt[w] > 0.f ? (mt[w] + __log2f(lt[w])) * 0.69314718055994531f : (lt[w] == lt[w] ? -INFINITY : lt[w]);
      }
    }
    cluster_sync();               // the others may still read this block's rows
    return;
  }
  if (ok) {
    tc_fence_after();
    // every product is done: the Q tile is free to stage rows, 4 KB a warp
    const float inv_l = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
    float4 *epi = reinterpret_cast<float4 *>(smem + C::OFF_Q + warp * 4096);
    const int rows = min(BM, p.Nq - i * BM) - (r & ~31);   // rows of this warp
    const long long base = b * p.osb + h * p.osh + (long long)(i * BM + (r & ~31)) * p.osn;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      uint32_t ov[32];
      if (T > 0) {
        tmem_ld32(tO + c * 32, ov);
        tc_wait_ld();
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) ov[e] = 0u;
      }
      if (!(l > 0.f) && l == l) {      // no key: 0, whatever the masked product left
#pragma unroll
        for (int e = 0; e < 32; ++e) ov[e] = 0u;
      }
      if (p.out_fp32) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          float4 o;
          o.x = __uint_as_float(ov[4 * q + 0]) * inv_l;
          o.y = __uint_as_float(ov[4 * q + 1]) * inv_l;
          o.z = __uint_as_float(ov[4 * q + 2]) * inv_l;
          o.w = __uint_as_float(ov[4 * q + 3]) * inv_l;
          epi[lane * 8 + (q ^ (lane & 7))] = o;
        }
        __syncwarp();
        float *dst = static_cast<float *>(p.out) + base + c * 32;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int row = (lane >> 3) + 4 * q, seg = lane & 7;
          if (row < rows)
            reinterpret_cast<float4 *>(dst + row * p.osn)[seg] = epi[row * 8 + (seg ^ (row & 7))];
        }
      } else {
        uint4 *ep = reinterpret_cast<uint4 *>(epi);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint4 u;
          u.x = pack_bf16x2(__uint_as_float(ov[8 * q + 0]) * inv_l, __uint_as_float(ov[8 * q + 1]) * inv_l);
          u.y = pack_bf16x2(__uint_as_float(ov[8 * q + 2]) * inv_l, __uint_as_float(ov[8 * q + 3]) * inv_l);
          u.z = pack_bf16x2(__uint_as_float(ov[8 * q + 4]) * inv_l, __uint_as_float(ov[8 * q + 5]) * inv_l);
          u.w = pack_bf16x2(__uint_as_float(ov[8 * q + 6]) * inv_l, __uint_as_float(ov[8 * q + 7]) * inv_l);
          ep[lane * 4 + (q ^ ((lane >> 1) & 3))] = u;
        }
        __syncwarp();
        uint16_t *dst = static_cast<uint16_t *>(p.out) + base + c * 32;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int row = (lane >> 2) + 8 * q, seg = lane & 3;
          if (row < rows)
            reinterpret_cast<uint4 *>(dst + row * p.osn)[seg] = ep[row * 4 + (seg ^ ((row >> 1) & 3))];
        }
      }
      __syncwarp();
    }
    if (p.out_lse && (r & 31) < rows)
      p.out_lse[b * p.lsb + h * p.lsh + (long long)(i * BM + r) * p.lsn] =
          l > 0.f ? (m_used + __log2f(l)) * 0.69314718055994531f : (l == l ? -INFINITY : l);
  }
  tc_fence_before();
  named_bar_arrive(1, kThreads);
}

template <int D, bool SPLIT>
cudaError_t launch(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const Params &p, int B,
                   cudaStream_t stream) {
  auto kfn = block_attn_kernel<D, SPLIT>;
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
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.n_q * p.split), (unsigned)p.H, (unsigned)B);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<D>::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute cluster;
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = (unsigned)p.split;
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  cfg.attrs = &cluster;
  cfg.numAttrs = SPLIT ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kfn, tq, tk, tv, p);
}

template <int D>
cudaError_t launch(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const Params &p, int B,
                   cudaStream_t stream) {
  return p.split > 1 ? launch<D, true>(tq, tk, tv, p, B, stream) : launch<D, false>(tq, tk, tv, p, B, stream);
}

}  // namespace battn

cudaError_t launch_block_attn(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, int B, int H,
                              int Hkv, int Nq, int Nk, int d, const int *sel, const int *count, int room,
                              const int *k_len, float scale, void *out, int out_fp32, const long long *os,
                              float *out_lse, const long long *ls, int *dev_status, long long wait_limit_ns,
                              int num_sms, cudaStream_t stream) {
  battn::Params p;
  p.H = H;
  p.G = H / Hkv;
  p.Hkv = Hkv;
  p.Nq = Nq;
  p.Nk = Nk;
  p.n_q = (Nq + kQBlock - 1) / kQBlock;
  p.n_k = (Nk + kPage - 1) / kPage;
  p.room = room;
  p.sel = sel;
  p.count = count;
  p.k_len = k_len;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.out = out;
  p.out_fp32 = out_fp32;
  p.osb = os[0];
  p.osh = os[1];
  p.osn = os[2];
  p.out_lse = out_lse;
  p.lsb = ls[0];
  p.lsh = ls[1];
  p.lsn = ls[2];
  p.dev_status = dev_status;
  p.wait_limit_ns = wait_limit_ns;
  // Few query blocks leave SMs (two blocks each) without work: their lists are cut
  // into parts of at least one tile, if they may have four (4 query blocks, d = 64
  // and 128: 80 listed blocks 64 and 76 us whole, 16 and 20 us in eight parts; 16
  // listed 16.4 and 20.5, 11 and 14; 8 listed 12.1 and 13.3, 10.3 and 12.3 in four
  // parts; 4 listed 8.3 and 10.3, 10.3 and 12.8 in two).
  const long long blocks = (long long)p.n_q * H * B;
  p.split = 1;
  while (room >= 8 && p.split < battn::kMaxSplit && blocks * p.split * 2 <= 2LL * num_sms && p.split * 4 <= room)
    p.split *= 2;
  switch (d) {
    case 64: return battn::launch<64>(tq, tk, tv, p, B, stream);
    case 96: return battn::launch<96>(tq, tk, tv, p, B, stream);
    case 128: return battn::launch<128>(tq, tk, tv, p, B, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace ditango
