// Shared pieces of the paged 4-bit history and of the selected-block
// operators: the page format, and small device helpers.
//
// A page holds kPage tokens of one key head, K and V, as 64 * (d + 8) bytes:
//   [0, 32 d)            K codes, token-major, d/2 bytes a token; channel 2b in
//                        the low half of byte b, channel 2b + 1 in the high one
//   [32 d, 64 d)         V codes
//   [64 d, 64 d + 256)   K (scale, least), two bf16 a token
//   [64 d + 256, ...)    V (scale, least)
// A code c stands for c * scale + least.  One page of one head is one
// contiguous run, so that a kernel fetches it with one bulk copy.
#pragma once

#include <atomic>

#include "common.cuh"

namespace ditango {

constexpr int kPage = DITANGO_PAGE;       // tokens of a page = keys of a key block
constexpr int kQBlock = DITANGO_QBLOCK;   // queries of a query block

__host__ __device__ constexpr int page_bytes(int d) { return kPage * (d + 8); }

// Division of numbers below 2^31 by a fixed divisor: with l = ceil(log2 d),
// m = floor(2^(31+l) / d) + 1 is over 2^(31+l) / d by at most one, so n m /
// 2^(31+l) is over n / d by less than 1 / d and its floor is exact.
struct FastDiv {
  uint32_t d, m, shift;
  FastDiv() : d(1), m(0), shift(0) {}
  explicit FastDiv(uint32_t div) : d(div), m(0), shift(0) {
    uint32_t l = 0;
    while ((1ull << l) < d) ++l;
    if (l > 0) {
      m = (uint32_t)(((1ull << (31 + l)) / d) + 1);
      shift = l - 1;
    }
  }
#ifdef __CUDACC__
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return m ? __umulhi(n, m) >> shift : n; }
#endif
};

// The devices on which a kernel's attributes have been set.  Neither a lock nor an
// allocation, whose failure would end in an exception at a C entry: two threads may
// both set them, which does no harm.
class OnDevices {
 public:
  bool has(int dev) const { return dev < 64 && (bits_.load(std::memory_order_acquire) >> dev & 1u); }
  void add(int dev) {
    if (dev < 64) bits_.fetch_or(1ull << dev, std::memory_order_release);
  }

 private:
  std::atomic<unsigned long long> bits_{0};
};

#ifdef __CUDACC__

// A running maximum is left as it is until it grew by more than 2^8.
constexpr float kRescaleLog2 = 8.0f;
// p = 2^(x mul - m) is formed by one FMA, which does not round x mul as m was
// rounded: past this size of m the difference could reach 1 and more (an
// overflow), and x mul is rounded first, in a path of its own.
constexpr float kHuge = 1048576.0f;   // 2^20: at most 2^-4 off

__device__ __forceinline__ void set_status(int *dev_status, int code) {
  if (dev_status) atomicExch(dev_status, code);
}

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

__device__ __forceinline__ float fast_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 numbers in one register pair, and their operations.
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unf2(uint64_t v, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A value that the compiler does not move or form again past this point.  What one
// elected lane's tcgen05 instructions name (descriptors, barriers) is pinned by the
// whole warp before that lane's branch: the instructions take it from uniform
// registers, which a branch of one lane is no place to form.
__device__ __forceinline__ uint32_t pinned(uint32_t x) {
  asm volatile("mov.b32 %0, %0;" : "+r"(x));
  return x;
}
__device__ __forceinline__ uint64_t pinned(uint64_t x) {
  asm volatile("mov.b64 %0, %0;" : "+l"(x));
  return x;
}

// Untiled bulk copy global -> shared (16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
      : "memory");
}

// Order this thread's earlier shared-memory accesses before later accesses
// by the asynchronous proxy (bulk copies, tensor core operands).
__device__ __forceinline__ void fence_proxy_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

#endif  // __CUDACC__

}  // namespace ditango
