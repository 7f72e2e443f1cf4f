// attn_rows.cuh -- attention of single rows, one warp a row: the plain
// statement of dspark_attn_verify, which touches no key that the row does not
// see.  The tiled kernels fall back to it for rows whose result is not finite.
#pragma once

#include <type_traits>

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

// E elements of a lane, as they lie in the cache, as fp32.
template <typename T, typename TC, int E, typename Raw>
__device__ __forceinline__ void row_values(const Raw& raw, float (&x)[E]) {
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    float2 v;
    if constexpr (sizeof(TC) == 1)
      v = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(
          reinterpret_cast<const __nv_fp8x2_storage_t*>(&raw)[e / 2], __NV_E4M3)));
    else
      v = Pair<T>::get(reinterpret_cast<const uint32_t*>(&raw)[e / 2]);
    x[e] = v.x;
    x[e + 1] = v.y;
  }
}

// One row (request b, position pos, query head hq, `row` of the row tensors)
// by the 32 lanes of a warp, D / 32 elements a lane; running maximum and sums
// in fp32, those of 256 keys by themselves first: added one by one, the weights
// of a long sequence would fall below half a unit in the sums' last place.
template <typename T, typename TC, int D>
__device__ __noinline__ void attend_row(const AttnArgs& a, int b, int pos, int hq, long long row,
                                        unsigned& flags) {
  constexpr int E = D / 32;
  const KvRows& r = a.rows;
  const int lane = threadIdx.x & 31;
  const int h = a.by_g.div(hq);
  using Raw = typename std::conditional<
      E * sizeof(TC) == 8, uint2,
      typename std::conditional<E * sizeof(TC) == 4, uint32_t, uint16_t>::type>::type;
  float q[E], o[E], o_all[E];
  const T* qp = static_cast<const T*>(a.q) + row * a.q_stride + (size_t)hq * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const float2 x = Pair<T>::get(*reinterpret_cast<const uint32_t*>(qp + e));
    q[e] = x.x; q[e + 1] = x.y;
    o[e] = o[e + 1] = o_all[e] = o_all[e + 1] = 0.0f;
  }
  float m = -CUDART_INF_F, sum = 0.0f, sum_all = 0.0f;
  // a query with a value that is not finite has scores that are not finite, all
  // of them: no softmax
  float q_odd = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) q_odd = fmaf(q[e], 0.0f, q_odd);
  if (__any_sync(0xffffffffu, q_odd != 0.0f)) sum = CUDART_NAN_F;
  const int mask = (1 << r.page_shift) - 1;
  // loaded together (a key alone is a chain of 1000 clocks); fewer where the
  // kernel around has fewer registers
  constexpr int kKeys = sizeof(TC) == 1 ? 2 : 4;
  // (a sum that is no number stays so)
  const int low = first_seen(pos, a.window);
  for (int j0 = low; j0 <= pos && sum == sum; j0 += kKeys) {
    if (((j0 - low) & 255) == 0) {
      sum_all += sum;
      sum = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        o_all[e] += o[e];
        o[e] = 0.0f;
      }
    }
    Raw raw[kKeys][2];  // K and V as they lie: four keys' values would be many registers
    float s[kKeys], vs[kKeys];
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const int j = min(j0 + i, pos);
      int page = checked_page(r, b, j >> r.page_shift, flags);
      if (page < 0) page = 0;
      const size_t place = ((((size_t)page * a.Hkv + h) << r.page_shift) + (j & mask));
      s[i] = vs[i] = 1.0f;
      if constexpr (sizeof(TC) == 1) {
        s[i] = a.k_scale[place];
        vs[i] = a.v_scale[place];
      }
      raw[i][0] = *reinterpret_cast<const Raw*>(static_cast<const TC*>(a.k_cache) + place * D +
                                                lane * E);
      raw[i][1] = *reinterpret_cast<const Raw*>(static_cast<const TC*>(a.v_cache) + place * D +
                                                lane * E);
    }
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      float x[E], dot = 0.0f;
      row_values<T, TC, E>(raw[i][0], x);
#pragma unroll
      for (int e = 0; e < E; ++e) dot = fmaf(q[e], x[e], dot);
      s[i] = warp_sum(dot) * s[i] * a.scale2;
    }
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      if (j0 + i > pos) break;
      const float mn = fmaxf(m, s[i]);
      const float back = mn == -CUDART_INF_F ? 1.0f : exp2f(m - mn);
      const float w = mn == -CUDART_INF_F && s[i] == s[i] ? 0.0f : exp2f(s[i] - mn);
      m = mn;
      sum = sum * back + w;
      if (back != 1.0f) {
        sum_all *= back;
#pragma unroll
        for (int e = 0; e < E; ++e) o_all[e] *= back;
      }
      float x[E];
      row_values<T, TC, E>(raw[i][1], x);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(w, x[e] * vs[i], o[e] * back);
    }
  }
  const float inv = 1.0f / (sum_all + sum);
  T* dst = static_cast<T*>(a.out) + (row * a.Hq + hq) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t*>(dst + e) = 
        Pair<T>::put((o_all[e] + o[e]) * inv, (o_all[e + 1] + o[e + 1]) * inv);
}

}  // namespace dspark
