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
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(addr)
        : "memory");
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

// Two e4m3 codes, in the high bytes of the halves of x (low bytes 0), as 16-bit
// values: the four exponent bits land on the low exponent bits of the wider
// type (subnormal codes on its subnormals), and a power of two makes up for
// the difference of the biases: 2^(127 - 7) for bf16, 2^(15 - 7) for fp16.
// Both steps are exact.
template <typename T>
__device__ __forceinline__ uint32_t widen2(uint32_t x) {
  if constexpr (std::is_same<T, __half>::value) {
    const uint32_t y = (x & 0x80008000u) | ((x >> 1) & 0x3f803f80u);
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&y), __floats2half2_rn(256.0f, 256.0f));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const uint32_t y = (x & 0x80008000u) | ((x >> 4) & 0x07f007f0u);
    const uint32_t two120 = 0x7b807b80u;
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&y),
                                     *reinterpret_cast<const __nv_bfloat162*>(&two120));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}

// An e4m3 tile of 128 rows x D bytes (as TMA wrote it, swizzled over its row)
// to T in the operands' layout (64-element halves, 128-byte swizzle), by 128
// threads.
template <typename T, int D>
__device__ __forceinline__ void widen_tile(const unsigned char* raw, unsigned char* op, int tid) {
  constexpr int kChunks = D / 16, kBatch = 4;
#pragma unroll
  for (int i0 = tid; i0 < 128 * kChunks; i0 += 128 * kBatch) {
    uint4 u[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + 128 * b;
      u[b] = *reinterpret_cast<const uint4*>(raw + k8_offset<D>(i / kChunks, i % kChunks * 16));
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + 128 * b, row = i / kChunks, c = i % kChunks;
      uint4 o[2];
      o[0] = make_uint4(
          widen2<T>(__byte_perm(u[b].x, 0, 0x1404)), widen2<T>(__byte_perm(u[b].x, 0, 0x3424)),
          widen2<T>(__byte_perm(u[b].y, 0, 0x1404)), widen2<T>(__byte_perm(u[b].y, 0, 0x3424)));
      o[1] = make_uint4(
          widen2<T>(__byte_perm(u[b].z, 0, 0x1404)), widen2<T>(__byte_perm(u[b].z, 0, 0x3424)),
          widen2<T>(__byte_perm(u[b].w, 0, 0x1404)), widen2<T>(__byte_perm(u[b].w, 0, 0x3424)));
      // the halves of D lie on the same banks: their lanes store in opposite order
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int y = x ^ (c >> 2);
        const int oc = 2 * c + y;
        *reinterpret_cast<uint4*>(op + (oc >> 3) * 128 * 128 + row * 128 +
                                  (((oc & 7) ^ (row & 7)) << 4)) = y ? o[1] : o[0];
      }
    }
  }
}

}  // namespace dspark
