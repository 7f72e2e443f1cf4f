// kv_rows.cuh -- rows into the paged cache (norm, rotation, quantisation in
// one pass) and back out of it.
//
// Both calls move each element once and compute a handful of flops on it, so
// HBM bounds them when they are large and the launch when they are small: one
// launch each, no pass over the data between load and store.  A vector (one
// head of one row) is D elements on D / 8 lanes, 16 bytes a lane, so sums,
// maxima and the rotation's partners stay inside a warp.
#pragma once

#include "kv_common.cuh"

namespace dspark {

constexpr int kRowThreads = 256;

// Vectors that a thread has in flight before it uses the first.
constexpr int kRowBatch = 3;

struct AppendArgs {
  KvRows rows;
  const void *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  void *k_cache, *v_cache;
  float *k_scale, *v_scale;
  const float *q_norm, *k_norm;
  const double* inv_freq;
  void* q_out;
  unsigned* status;
  float eps, rope_scale;
  int Hq, Hkv, rot, interleaved;
};

template <typename T>
__device__ __forceinline__ T group_sum(T v, int lanes) {
  for (int o = lanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float group_max(float v, int lanes) {
  for (int o = lanes / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Two dynamic arrays: s_first [B + 1] int.
template <typename T, typename TC, int D>
__global__ void __launch_bounds__(kRowThreads) kv_append_kernel(const AppendArgs a) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = kRowThreads / kLanes;
  extern __shared__ int s_first[];
  __shared__ int s_warp[kRowThreads / 32];
  __shared__ float2 s_cs[2][D / 2];  // (cos, sin) * rope_scale of one token
  grid_dep_launch();
  grid_dep_wait();
  const KvRows& r = a.rows;
  unsigned flags = 0;
  scan_requests<kRowThreads>(r.B, s_first, s_warp, [&](int b) {
    return checked_new(r, b, r.cache_len[b], r.row_start[b], flags);
  });
  const int total = s_first[r.B];
  const int l = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const int half = a.rot / 2;
  const int n_vec = a.Hq + 2 * a.Hkv;
  const int n_loop = (n_vec + kGroups - 1) / kGroups;  // the same for every thread: shuffles below
  // this lane's 8 elements in the rotation: pairs inside the lane, or one
  // element of a pair whose other one is in lane `mate`
  const bool turns = 8 * l < a.rot;
  int mate = threadIdx.x & 31;
  float sign = 0.0f;
  if (turns && !a.interleaved) {
    const bool first = 8 * l < half;
    mate += first ? half / 8 : -(half / 8);
    sign = first ? -1.0f : 1.0f;
  }
  float wq[8], wk[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    wq[j] = a.q_norm ? a.q_norm[8 * l + j] : 1.0f;
    wk[j] = a.k_norm ? a.k_norm[8 * l + j] : 1.0f;
  }
  int par = 0;
  for (int i = blockIdx.x; i < total; i += gridDim.x, par ^= 1) {
    const int b = find_request(s_first, r.B, i);
    const int p = i - s_first[b];
    const int past = r.cache_len[b];
    const long long start = r.row_start[b];
    unsigned again = 0;
    if (p < 0 || p >= checked_new(r, b, past, start, again)) continue;  // uniform over the block
    const long long row = start + p;
    const int pos = past + p;
    if (threadIdx.x < half) {
      // the angle in turns, its whole part taken off in fp64: exact to about
      // 1e-11 turns at any position, then fp32
      const double turn = (double)pos * a.inv_freq[threadIdx.x] * 0.15915494309189533577;
      float s, c;
      sincospif(2.0f * (float)(turn - rint(turn)), &s, &c);
      s_cs[par][threadIdx.x] = make_float2(c * a.rope_scale, s * a.rope_scale);
    }
    const int page = checked_page(r, b, pos >> r.page_shift, flags);
    const int at = pos & ((1 << r.page_shift) - 1);
    float2 cs[8];
    bool have = false;
    for (int v0 = 0; v0 < n_loop; v0 += kRowBatch) {
      uint4 in[kRowBatch];
#pragma unroll
      for (int m = 0; m < kRowBatch; ++m) {
        const int u = (v0 + m) * kGroups + group;
        in[m] = make_uint4(0, 0, 0, 0);
        if (v0 + m < n_loop && u < n_vec) {
          const T* src = u < a.Hq ? static_cast<const T*>(a.q) + row * a.q_stride + u * D
                         : u < a.Hq + a.Hkv
                             ? static_cast<const T*>(a.k) + row * a.k_stride + (u - a.Hq) * D
                             : static_cast<const T*>(a.v) + row * a.v_stride +
                                   (u - a.Hq - a.Hkv) * D;
          in[m] = *reinterpret_cast<const uint4*>(src + 8 * l);
        }
      }
      if (!have) {
        have = true;
        __syncthreads();  // s_cs[par] written; the other buffer's readers are behind this too
        if (turns) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            cs[j] = a.interleaved ? s_cs[par][4 * l + j / 2]
                                  : s_cs[par][8 * l + j < half ? 8 * l + j : 8 * l + j - half];
        }
      }
#pragma unroll
      for (int m = 0; m < kRowBatch; ++m) {
        if (v0 + m >= n_loop) break;
        const int u = (v0 + m) * kGroups + group;
        const bool is_q = u < a.Hq, is_k = !is_q && u < a.Hq + a.Hkv;
        float x[8];
        unpack8<T>(in[m], x);
        if (a.q_norm || a.k_norm) {
          float ss = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
          ss = group_sum(ss, kLanes);
          if ((is_q && a.q_norm) || (is_k && a.k_norm)) {
            const float inv = rsqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = x[j] * inv * (is_q ? wq[j] : wk[j]);
          }
        }
        if (a.rot) {
          if (a.interleaved) {
            if (turns && (is_q || is_k)) {
#pragma unroll
              for (int j = 0; j < 8; j += 2) {
                const float x1 = x[j], x2 = x[j + 1];
                x[j] = x1 * cs[j].x - x2 * cs[j].y;
                x[j + 1] = x2 * cs[j].x + x1 * cs[j].y;
              }
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float other = __shfl_sync(0xffffffffu, x[j], mate);
              if (turns && (is_q || is_k)) x[j] = x[j] * cs[j].x + sign * other * cs[j].y;
            }
          }
        }
        float scale = 1.0f;
        if constexpr (sizeof(TC) == 1) {
          float top = 0.0f, bad = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            top = fmaxf(top, fabsf(x[j]));
            if (!isfinite(x[j])) bad = 1.0f;
          }
          top = group_max(top, kLanes);
          bad = group_max(bad, kLanes);
          scale = fmaxf(top / 448.0f, 1.17549435e-38f);
          if (bad != 0.0f) {
            scale = CUDART_NAN_F;
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = 0.0f;
          }
        }
        if (u >= n_vec) continue;
        if (is_q) {
          T* dst = static_cast<T*>(a.q_out) + (row * a.Hq + u) * D + 8 * l;
          *reinterpret_cast<uint4*>(dst) = pack8<T>(x);
          continue;
        }
        if (page < 0) continue;
        const int h = is_k ? u - a.Hq : u - a.Hq - a.Hkv;
        const size_t place = ((((size_t)page * a.Hkv + h) << r.page_shift) + at);
        TC* dst = static_cast<TC*>(is_k ? a.k_cache : a.v_cache) + place * D + 8 * l;
        if constexpr (sizeof(TC) == 1) {
          // a true division: the code of a value on the border between two
          // must not hang on a reciprocal's rounding
          if (scale == scale) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = x[j] / scale;
          }
          *reinterpret_cast<uint2*>(dst) = make_uint2(f32_to_e4m3x4(x[0], x[1], x[2], x[3]),
                                                      f32_to_e4m3x4(x[4], x[5], x[6], x[7]));
          if (l == 0) (is_k ? a.k_scale : a.v_scale)[place] = scale;
        } else {
          *reinterpret_cast<uint4*>(dst) = pack8<T>(x);
        }
      }
    }
  }
  flags = __reduce_or_sync(0xffffffffu, flags);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = (int)flags;
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned f = 0;
    for (int w = 0; w < kRowThreads / 32; ++w) f |= (unsigned)s_warp[w];
    store_status(a.status, f);
  }
}

struct ReadArgs {
  KvRows rows;
  const void *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  void *k_out, *v_out;
  unsigned* status;
  int Hkv;
};

template <typename T, typename TC, int D>
__global__ void __launch_bounds__(kRowThreads) kv_read_kernel(const ReadArgs a) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = kRowThreads / kLanes;
  extern __shared__ int s_first[];
  __shared__ int s_warp[kRowThreads / 32];
  grid_dep_launch();
  grid_dep_wait();
  const KvRows& r = a.rows;
  unsigned flags = 0;
  scan_requests<kRowThreads>(r.B, s_first, s_warp, [&](int b) {
    return checked_new(r, b, r.cache_len[b], r.row_start[b], flags);
  });
  const int total = s_first[r.B];
  const int l = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const int n_vec = 2 * a.Hkv;
  for (int i = blockIdx.x; i < total; i += gridDim.x) {
    const int b = find_request(s_first, r.B, i);
    const int p = i - s_first[b];
    const int past = r.cache_len[b];
    const long long start = r.row_start[b];
    unsigned again = 0;
    if (p < 0 || p >= checked_new(r, b, past, start, again)) continue;
    const long long row = start + p;
    const int pos = past + p;
    int page = checked_page(r, b, pos >> r.page_shift, flags);
    if (page < 0) page = 0;
    const int at = pos & ((1 << r.page_shift) - 1);
    for (int u = group; u < n_vec; u += kGroups) {
      const bool is_k = u < a.Hkv;
      const int h = is_k ? u : u - a.Hkv;
      const size_t place = ((((size_t)page * a.Hkv + h) << r.page_shift) + at);
      const TC* src = static_cast<const TC*>(is_k ? a.k_cache : a.v_cache) + place * D + 8 * l;
      uint4 out;
      if constexpr (sizeof(TC) == 1) {
        const uint2 c = *reinterpret_cast<const uint2*>(src);
        const float s = (is_k ? a.k_scale : a.v_scale)[place];
        float x[8];
        e4m3x4_to_f32(c.x, x);
        e4m3x4_to_f32(c.y, x + 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= s;
        out = pack8<T>(x);
      } else {
        out = *reinterpret_cast<const uint4*>(src);
      }
      T* dst = static_cast<T*>(is_k ? a.k_out : a.v_out) + (row * a.Hkv + h) * D + 8 * l;
      *reinterpret_cast<uint4*>(dst) = out;
    }
  }
  flags = __reduce_or_sync(0xffffffffu, flags);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = (int)flags;
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned f = 0;
    for (int w = 0; w < kRowThreads / 32; ++w) f |= (unsigned)s_warp[w];
    store_status(a.status, f);
  }
}

}  // namespace dspark
