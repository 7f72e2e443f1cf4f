// attn_tc.cuh -- tensor-core pieces of the attention kernels: descriptors of
// operands that lie with their M or N dimension contiguous, TMEM accesses by
// width, block votes, e4m3 tiles widened to 16 bits.
#pragma once

#include <type_traits>

#include "kv_common.cuh"
#include "tc_common.cuh"

namespace dspark {

// Instruction descriptor of kind::f16 with fp32 accumulation; a_mn / b_mn: that
// operand's M or N dimension is the contiguous one.
template <typename T>
__host__ __device__ constexpr uint32_t idesc_tc(int M, int N, bool a_mn, bool b_mn) {
  constexpr uint32_t fmt = std::is_same<T, __half>::value ? 0u : 1u;
  return (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Shared-memory descriptor of an operand whose M or N dimension is contiguous:
// rows (of K) of W elements, swizzled over their 2 W bytes (W 64, 32 or 16), 8
// rows an atom, atoms of further K behind each other; the next W elements of M
// or N lie `k_rows` rows on.
template <int W>
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t addr, int k_rows) {
  static_assert(W == 64 || W == 32 || W == 16, "row width");
  uint64_t d = 0;
  d |= (uint64_t)((addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((uint32_t)(k_rows * W * 2) >> 4) << 16;  // next W elements
  d |= (uint64_t)((8 * W * 2) >> 4) << 32;                 // next 8 rows
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)(W == 64 ? 2 : W == 32 ? 4 : 6) << 61;
  return d;
}
// Byte offset of element (n, k) of such an operand with k_rows rows, n a
// multiple of 8 (a 16-byte chunk).
template <int W>
__device__ __forceinline__ uint32_t mn_offset(int n, int k, int k_rows) {
  const int block = n / W, c = (n % W) >> 3;
  const int sw = W == 64 ? (k & 7) : W == 32 ? ((k >> 1) & 3) : ((k >> 2) & 1);
  return (uint32_t)(block * k_rows * W * 2 + k * W * 2 + ((c ^ sw) << 4));
}

// One lane of a converged warp, chosen by the hardware: the compiler knows that
// a branch on it has a single active thread and issues TMA and MMA instructions
// in it directly.  Behind `lane == 0` it wraps each of them in a loop over the
// active lanes, which measured 100 to 150 clocks an instruction.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// 8 columns, split as tmem_ld32_issue / tmem_ld32_wait.
__device__ __forceinline__ void tmem_ld8_issue(uint32_t addr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(addr));
}
__device__ __forceinline__ void tmem_ld8_wait(uint32_t (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
}
template <int C>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[C]) {
  static_assert(C == 8 || C == 16 || C == 32, "columns");
  if constexpr (C == 32) {
    tmem_ld32_issue(addr, r);
    tmem_ld32_wait(r);
  } else if constexpr (C == 16) {
    tmem_ld16_issue(addr, r);
    tmem_ld16_wait(r);
  } else {
    tmem_ld8_issue(addr, r);
    tmem_ld8_wait(r);
  }
}
template <int C>
__device__ __forceinline__ void tmem_st(uint32_t addr, const uint32_t (&r)[C]) {
  static_assert(C == 8 || C == 16 || C == 32, "columns");
  if constexpr (C == 32) {
    tmem_st32(addr, r);
  } else if constexpr (C == 16) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
  } else {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
        : "memory");
  }
}

// Descriptors of the kind::f8f6f4 MMA, e4m3 x e4m3 -> fp32, 32 elements of K an
// instruction, both operands K-major with rows of W bytes (128 or 64), swizzled
// over the row.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
template <int W>
__device__ __forceinline__ uint64_t sdesc_k8(uint32_t addr) {
  static_assert(W == 128 || W == 64, "row width");
  uint64_t d = 0;
  d |= (uint64_t)((addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)1 << 16;
  d |= (uint64_t)((8 * W) >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)(W == 128 ? 2 : 4) << 61;
  return d;
}
__device__ __forceinline__ void mma_e4m3_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Byte offset of byte b of row r in rows of W bytes, swizzled over the row.
template <int W>
__device__ __forceinline__ uint32_t k8_offset(int r, int b) {
  const int sw = W == 128 ? (r & 7) : ((r >> 1) & 3);
  return (uint32_t)(r * W + (((b >> 4) ^ sw) << 4) + (b & 15));
}

// Whether `p` holds for any of the `count` threads at named barrier `id`.
__device__ __forceinline__ bool vote_any(int id, int count, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)p), "r"(id), "r"(count)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ float warp_max_redux(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

template <typename T>
__device__ __forceinline__ T to_elem(float v) {
  if constexpr (std::is_same<T, __half>::value) return __float2half_rn(v);
  else return __float2bfloat16_rn(v);
}

// 16 bytes from global to shared memory without registers; zeros if !take.
__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(take ? 16 : 0)
               : "memory");
}
// Arrives on `bar` (as one of its expected arrivals) once this thread's copies
// so far are there.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// The largest of three (a NaN is passed over).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Four e4m3 codes as fp16 (exact).
__device__ __forceinline__ uint2 widen4(uint32_t c) {
  uint2 r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(c));
  return r;
}

// An e4m3 tile of 128 rows x D bytes (as TMA wrote it, swizzled over its row) to
// fp16 in the operands' layout (64-element halves, 128-byte swizzle), by 128
// threads; rows from `rows` on become zero: what lies behind a sequence may be
// anything, and 0 times a NaN is none.  (Loops kept short: the warps of a CTA run
// different code, and what does not fit the instruction cache of an SM's quarter
// costs more than it saves.)
template <int D>
__device__ __forceinline__ void widen_tile(const unsigned char* raw, unsigned char* op, int rows,
                                           int tid) {
  constexpr int kChunks = D / 16, kBatch = 4;
  const int c = tid % kChunks;
  // the halves of D lie on the same banks: their lanes take the two halves of
  // their 16 bytes in opposite order
  const bool swap = c & 4;
#pragma unroll 1
  for (int i0 = tid; i0 < 128 * kChunks; i0 += 128 * kBatch) {
    uint4 u[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int row = (i0 + 128 * b) / kChunks;
      u[b] = *reinterpret_cast<const uint4*>(raw + k8_offset<D>(row, 16 * c));
      if (row >= rows) u[b] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int row = (i0 + 128 * b) / kChunks;
      unsigned char* dst = op + (c >> 2) * 128 * 128 + row * 128;
      const uint2 a0 = widen4(swap ? u[b].z : u[b].x), a1 = widen4(swap ? u[b].w : u[b].y);
      *reinterpret_cast<uint4*>(dst + ((((2 * c + swap) & 7) ^ (row & 7)) << 4)) =
          make_uint4(a0.x, a0.y, a1.x, a1.y);
      const uint2 b0 = widen4(swap ? u[b].x : u[b].z), b1 = widen4(swap ? u[b].y : u[b].w);
      *reinterpret_cast<uint4*>(dst + ((((2 * c + !swap) & 7) ^ (row & 7)) << 4)) =
          make_uint4(b0.x, b0.y, b1.x, b1.y);
    }
  }
}

}  // namespace dspark
