// attn_rows.cuh -- attention of single rows, one warp a row: the plain
// statement of dspark_attn_verify, which touches no key that the row does not
// see.  The tiled kernels fall back to it for rows whose result is not finite.
#pragma once

#include "kv_common.cuh"

namespace dspark {

struct AttnArgs {
  KvRows rows;
  const void* q;
  long long q_stride;
  const void *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  void* out;
  unsigned* status;
  float scale2;  // sm_scale * log2(e): weights are powers of two of scaled scores
  int Hq, Hkv, G, window;
  Divisor by_g;  // by G
};

// Position range that the row at position i sees.
__device__ __forceinline__ int first_seen(int i, int window) {
  return window > 0 && i - window + 1 > 0 ? i - window + 1 : 0;
}

// One row (request b, position pos, query head hq, `row` of the row tensors)
// by the 32 lanes of a warp, D / 32 elements a lane; running maximum and sum
// in fp32.
template <typename T, typename TC, int D>
__device__ __noinline__ void attend_row(const AttnArgs& a, int b, int pos, int hq, long long row,
                                        unsigned& flags) {
  constexpr int E = D / 32;
  const KvRows& r = a.rows;
  const int lane = threadIdx.x & 31;
  const int h = a.by_g.div(hq);
  float q[E], o[E];
  const T* qp = static_cast<const T*>(a.q) + row * a.q_stride + (size_t)hq * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const float2 x = Pair<T>::get(*reinterpret_cast<const uint32_t*>(qp + e));
    q[e] = x.x; q[e + 1] = x.y;
    o[e] = o[e + 1] = 0.0f;
  }
  float m = -CUDART_INF_F, sum = 0.0f;
  // a query with a value that is not finite has scores that are not finite, all
  // of them: no softmax
  float q_odd = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) q_odd = fmaf(q[e], 0.0f, q_odd);
  if (__any_sync(0xffffffffu, q_odd != 0.0f)) sum = CUDART_NAN_F;
  int page = 0;
  const int mask = (1 << r.page_shift) - 1;
  const int j0 = first_seen(pos, a.window);
  for (int j = j0; j <= pos && sum == sum; ++j) {  // (a sum that is no number stays so)
    if (j == j0 || (j & mask) == 0) {
      page = checked_page(r, b, j >> r.page_shift, flags);
      if (page < 0) page = 0;
    }
    const size_t place = ((((size_t)page * a.Hkv + h) << r.page_shift) + (j & mask));
    float kv[2][E], ks = 1.0f, vs = 1.0f;
    if constexpr (sizeof(TC) == 1) {
      ks = a.k_scale[place];
      vs = a.v_scale[place];
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const TC* src = static_cast<const TC*>(w ? a.v_cache : a.k_cache) + place * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        float2 x;
        if constexpr (sizeof(TC) == 1)
          x = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(
              *reinterpret_cast<const __nv_fp8x2_storage_t*>(src + e), __NV_E4M3)));
        else
          x = Pair<T>::get(*reinterpret_cast<const uint32_t*>(src + e));
        kv[w][e] = x.x; kv[w][e + 1] = x.y;
      }
    }
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], kv[0][e], s);
    s = warp_sum(s) * ks * a.scale2;
    const float mn = fmaxf(m, s);
    const float back = mn == -CUDART_INF_F ? 1.0f : exp2f(m - mn);
    const float w = mn == -CUDART_INF_F && s == s ? 0.0f : exp2f(s - mn);
    m = mn;
    sum = sum * back + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(w, kv[1][e] * vs, o[e] * back);
  }
  const float inv = 1.0f / sum;
  T* dst = static_cast<T*>(a.out) + (row * a.Hq + hq) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t*>(dst + e) = Pair<T>::put(o[e] * inv, o[e + 1] * inv);
}

}  // namespace dspark
