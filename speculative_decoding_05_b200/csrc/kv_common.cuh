// kv_common.cuh -- what the paged-cache calls share: their arguments, the
// row markers' checks, element types, and the status word spread over CTAs.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "../../include/dspark_kv.h"
#include "common.cuh"
#include "kv_status.h"

namespace dspark {

// ---------------------------------------------------------------------------
// status
// ---------------------------------------------------------------------------

// These calls clear no status word before their kernels (a clear would cost
// the smallest of them a third of its time).  Every CTA stores the flags that
// it raised, or 0, in a word of its own, and CTA 0 stores a head that tells
// the status readers how many words to join: bit 31 of word 0 (the other
// calls' flags leave it clear), the count, a tag.
constexpr unsigned kSpreadBit = 0x80000000u;
constexpr unsigned kSpreadTag = 0x6b76666cu;
constexpr int kSpreadFirst = kSpreadHeadWords;  // words before the CTAs' words
constexpr size_t kKvHeaderBytes = 8192;  // (4 + 2044) words
static_assert((kSpreadFirst + kMaxStatusCtas) * 4 == kKvHeaderBytes, "status words");

// One thread of every CTA, once, with the flags of the whole CTA.
__device__ __forceinline__ void store_status(unsigned* ws, unsigned flags) {
  if (blockIdx.x == 0) {
    ws[0] = kSpreadBit;
    ws[1] = gridDim.x;
    ws[2] = kSpreadTag;
  }
  ws[kSpreadFirst + blockIdx.x] = flags;
}

// ---------------------------------------------------------------------------
// rows and cache
// ---------------------------------------------------------------------------

constexpr int kKvMaxB = 4096;
constexpr long long kKvMaxRows = (1ll << 31) - (1 << 16);  // a step past them stays an int32

struct KvRows {  // the row markers (dspark_kv.h, "Rows")
  const int64_t* row_start;
  const int32_t* verify_len;
  const int32_t* cache_len;
  const int32_t* page_table;
  long long n_rows;
  long long max_pos;  // max_pages * page_size
  int B;
  int max_len;
  int max_pages;
  int page_shift;
  int n_pages;
};

// New tokens of request b (0: idle, or a marker out of range, flagged).
__device__ __forceinline__ int checked_new(const KvRows& r, int b, int past, long long row,
                                           unsigned& flags) {
  const int L = r.verify_len[b];
  if (L == -1) return 0;
  if (L < -1 || L >= r.max_len || past < 0 || (long long)past + L >= r.max_pos || row < 0 ||
      row > r.n_rows - 1 - L) {
    flags |= DSPARK_FLAG_BAD_LENGTH;
    return 0;
  }
  return L + 1;
}

// Page id of place `idx` of request b's table; an id out of range is flagged
// and given as -1.
__device__ __forceinline__ int checked_page(const KvRows& r, int b, int idx, unsigned& flags) {
  const int p = __ldg(r.page_table + (size_t)b * r.max_pages + idx);
  if (p < 0 || p >= r.n_pages) {
    flags |= DSPARK_FLAG_BAD_PAGE;
    return -1;
  }
  return p;
}

// Exclusive prefix sums over the requests' counts, s_first[b] for b <= B
// (s_first[B] = total), by the NT threads of a block.  count(b) is called once
// for each b.
template <int NT, typename F>
__device__ __forceinline__ void scan_requests(int B, int* s_first, int* s_warp, F&& count) {
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int base = 0;
  for (int b0 = 0; b0 < B; b0 += NT) {
    const int b = b0 + threadIdx.x;
    int v = b < B ? count(b) : 0;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += n;
    }
    if (lane == 31) s_warp[w] = incl;
    __syncthreads();
    int pre = base;
    for (int i = 0; i < w; ++i) pre += s_warp[i];
    int total = base;
    for (int i = 0; i < NT / 32; ++i) total += s_warp[i];
    if (b < B) s_first[b] = pre + incl - v;
    base = total;
    __syncthreads();
  }
  if (threadIdx.x == 0) s_first[B] = base;
  __syncthreads();
}

// The request b with s_first[b] <= i < s_first[b + 1].
__device__ __forceinline__ int find_request(const int* s_first, int B, int i) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s_first[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Division of 0 <= x < 2^31 by a divisor known on the host: with l = ceil(log2 d)
// and m = floor(2^(31 + l) / d) + 1, x m / 2^(31 + l) exceeds x / d by less than
// x / 2^(31 + l) <= 1 / d, so its whole part is the quotient.
struct Divisor {
  unsigned m;
  int shift;
  __device__ __forceinline__ int div(int x) const {
    return (int)(((unsigned long long)(unsigned)x * m) >> shift);
  }
};
inline Divisor make_divisor(int d) {
  int l = 0;
  while ((1 << l) < d) ++l;
  Divisor r;
  r.m = (unsigned)((1ull << (31 + l)) / (unsigned)d + 1);
  r.shift = 31 + l;
  return r;
}

// Pairs of fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void pair_to(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// ---------------------------------------------------------------------------
// element types
// ---------------------------------------------------------------------------

struct e4m3 {
  unsigned char code;
};

template <typename T>
struct Pair;  // two elements as fp32 and back, rounded to nearest even
template <>
struct Pair<__nv_bfloat16> {
  static __device__ __forceinline__ float2 get(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t put(float a, float b) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};
template <>
struct Pair<__half> {
  static __device__ __forceinline__ float2 get(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
  }
  static __device__ __forceinline__ uint32_t put(float a, float b) {
    const __half2 r = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};

// Four e4m3 codes as fp32.
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t c, float* o) {
  const __half2 a = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c & 0xffffu), __NV_E4M3));
  const __half2 b = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c >> 16), __NV_E4M3));
  const float2 fa = __half22float2(a), fb = __half22float2(b);
  o[0] = fa.x; o[1] = fa.y; o[2] = fb.x; o[3] = fb.y;
}
__device__ __forceinline__ uint32_t f32_to_e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& u, float (&o)[8]) {
  const float2 a = Pair<T>::get(u.x), b = Pair<T>::get(u.y), c = Pair<T>::get(u.z),
               d = Pair<T>::get(u.w);
  o[0] = a.x; o[1] = a.y; o[2] = b.x; o[3] = b.y;
  o[4] = c.x; o[5] = c.y; o[6] = d.x; o[7] = d.y;
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(Pair<T>::put(v[0], v[1]), Pair<T>::put(v[2], v[3]), Pair<T>::put(v[4], v[5]),
                    Pair<T>::put(v[6], v[7]));
}

}  // namespace dspark
