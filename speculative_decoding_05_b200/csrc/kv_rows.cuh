// kv_rows.cuh -- rows into the paged cache (norm, rotation, quantisation in
// one pass) and back out of it.
//
// Both calls move each element once and compute a handful of flops on it, so
// HBM bounds them when they are large and the launch when they are small: one
// launch each, no pass over the data between load and store.  A block takes a
// run of up to kRowRun tokens: places and angles of all of them first, then
// their vectors (one head of one row: D elements on D / 8 lanes, 16 bytes a lane,
// so sums, maxima and the rotation's partners stay inside a warp), kRowBatch
// loads of a thread in flight.  (One token at a time left each block waiting for
// a chain of five dependent loads: 36 % of the copy bandwidth.)
// Measured: append of a stress step 35 us (50 % of the copy bandwidth: its
// instructions for norm, rotation and shuffles bound it), of 3 x 4099 tokens to
// e4m3 with the read-back 121 us, of one request's block 15.6 us (the host call; 5 on the
// device); read-back of an e4m3 batch 131 us (68 %: 0.74 of the issue slots are used,
// places of vectors divided out one by one).
#pragma once

#include <type_traits>

#include "kv_common.cuh"

namespace dspark {

constexpr int kRowThreads = 256;
constexpr int kRowRun = 16;    // tokens of a block's run, at most
constexpr int kRowBatch = 4;   // vectors of a thread in flight

// Where a token's row and its cache entries are.
struct TokenPlace {
  long long row;
  int page;  // -1: an id out of range
  int at;    // in the page
  int pos;
};

// Tokens of a run: few enough to occupy all blocks.
__device__ __forceinline__ int run_length(int total) {
  const int t = (total + (int)gridDim.x - 1) / (int)gridDim.x;
  return t < 1 ? 1 : t > kRowRun ? kRowRun : t;
}

// Place of token i of the line of all tokens; false if it has none.
__device__ __forceinline__ bool token_place(const KvRows& r, const int* s_first, int i,
                                            TokenPlace& t, unsigned& flags) {
  const int b = find_request(s_first, r.B, i);
  const int p = i - s_first[b];
  const int past = r.cache_len[b];
  const long long start = r.row_start[b];
  unsigned again = 0;
  if (p < 0 || p >= checked_new(r, b, past, start, again)) return false;
  t.row = start + p;
  t.pos = past + p;
  t.page = checked_page(r, b, t.pos >> r.page_shift, flags);
  t.at = t.pos & ((1 << r.page_shift) - 1);
  return true;
}

// The flags of a block's threads to its status word.
__device__ __forceinline__ void finish_status(unsigned* status, unsigned flags, unsigned* s_flags) {
  __syncthreads();
  if (threadIdx.x == 0) *s_flags = 0;
  __syncthreads();
  if (flags) atomicOr(s_flags, flags);
  __syncthreads();
  if (threadIdx.x == 0) store_status(status, *s_flags);
}

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
  Divisor by_hq, by_hkv;
};

__device__ __forceinline__ float group_sum(float v, int lanes) {
  for (int o = lanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float group_max(float v, int lanes) {
  for (int o = lanes / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Place of the cosine and sine of pair i among rot / 2 = half: the even groups of
// four first, then the odd ones, so that lanes that read two groups each (8
// pairs behind each other) meet no bank twice.
__device__ __forceinline__ int angle_place(int i, int half) {
  const int c = i >> 2;
  return ((c & 1) * (half >> 3) + (c >> 1)) * 4 + (i & 3);
}

// One kind of vectors of a run of tokens: heads [0, H) of the rows at `src`,
// normed by w (or NULL) and turned if `turn`, to q_out (kOut) or the cache.
// Eight elements of a lane as four pairs.
template <typename T, typename TC, int D, bool kOut>
__device__ __forceinline__ void append_heads(const AppendArgs& a, const TokenPlace* s_tok,
                                             const float* s_cos, const float* s_sin, int n_tok,
                                             int H, const Divisor& by_h, const void* src,
                                             long long stride, const float* w, bool turn,
                                             void* cache, float* scales) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = kRowThreads / kLanes;
  const int l = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const int half = a.rot / 2, shift = a.rows.page_shift;
  // this lane's elements in the rotation: pairs inside the lane, or one element
  // of a pair whose other one is in lane `mate`
  const bool mine = turn && 8 * l < a.rot;
  const bool first = 8 * l < half;
  int mate = threadIdx.x & 31, angle = 0;
  if (mine) {
    angle = angle_place(a.interleaved ? 4 * l : first ? 8 * l : 8 * l - half, half);
    if (!a.interleaved) mate += first ? half / 8 : -(half / 8);
  }
  uint64_t wv[4];
  if (w) {
    const float4 w0 = reinterpret_cast<const float4*>(w)[2 * l];
    const float4 w1 = reinterpret_cast<const float4*>(w)[2 * l + 1];
    wv[0] = pair_of(w0.x, w0.y); wv[1] = pair_of(w0.z, w0.w);
    wv[2] = pair_of(w1.x, w1.y); wv[3] = pair_of(w1.z, w1.w);
  }
  const int n_all = n_tok * H;
  // the same number of steps for every thread (shuffles)
  for (int v0 = 0; v0 < n_all; v0 += kGroups * kRowBatch) {
    uint4 in[kRowBatch];
#pragma unroll
    for (int m = 0; m < kRowBatch; ++m) {
      const int v = v0 + m * kGroups + group;
      in[m] = make_uint4(0, 0, 0, 0);
      if (v < n_all) {
        const int tok = by_h.div(v);
        const long long row = s_tok[tok].row;
        if (row >= 0)
          in[m] = *reinterpret_cast<const uint4*>(static_cast<const T*>(src) + row * stride +
                                                  (v - tok * H) * D + 8 * l);
      }
    }
#pragma unroll
    for (int m = 0; m < kRowBatch; ++m) {
      if (v0 + m * kGroups >= n_all) break;  // uniform over the block
      const int v = min(v0 + m * kGroups + group, n_all - 1);
      const int tok = by_h.div(v), h = v - tok * H;
      uint64_t x[4];
      {
        const float2 x0 = Pair<T>::get(in[m].x), x1 = Pair<T>::get(in[m].y);
        const float2 x2 = Pair<T>::get(in[m].z), x3 = Pair<T>::get(in[m].w);
        x[0] = pair_of(x0.x, x0.y); x[1] = pair_of(x1.x, x1.y);
        x[2] = pair_of(x2.x, x2.y); x[3] = pair_of(x3.x, x3.y);
      }
      if (w) {
        uint64_t ss = mul2(x[0], x[0]);
        ss = fma2(x[1], x[1], ss);
        ss = fma2(x[2], x[2], ss);
        ss = fma2(x[3], x[3], ss);
        float s0, s1;
        pair_to(ss, s0, s1);
        const float inv = rsqrtf(group_sum(s0 + s1, kLanes) * (1.0f / D) + a.eps);
        const uint64_t inv2 = pair_of(inv, inv);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = mul2(mul2(x[j], inv2), wv[j]);
      }
      if (turn) {
        const float* co = s_cos + tok * (D / 2) + angle;
        const float* si = s_sin + tok * (D / 2) + angle;
        if (a.interleaved) {
          if (mine) {
            const float4 c = *reinterpret_cast<const float4*>(co);
            const float4 s = *reinterpret_cast<const float4*>(si);
            const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float x1, x2;
              pair_to(x[j], x1, x2);
              x[j] = fma2(x[j], pair_of(cv[j], cv[j]),
                          mul2(pair_of(x2, x1), pair_of(-sv[j], sv[j])));
            }
          }
        } else {
          uint64_t other[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) other[j] = __shfl_sync(0xffffffffu, x[j], mate);
          if (mine) {
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
              const int at = j / 2 * (half / 2);  // the odd group
              const float4 c = *reinterpret_cast<const float4*>(co + at);
              float4 s = *reinterpret_cast<const float4*>(si + at);
              if (first) s = make_float4(-s.x, -s.y, -s.z, -s.w);
              x[j] = fma2(x[j], pair_of(c.x, c.y), mul2(other[j], pair_of(s.x, s.y)));
              x[j + 1] = fma2(x[j + 1], pair_of(c.z, c.w), mul2(other[j + 1], pair_of(s.z, s.w)));
            }
          }
        }
      }
      float y[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) pair_to(x[j], y[2 * j], y[2 * j + 1]);
      float scale = 1.0f;
      if constexpr (!kOut && sizeof(TC) == 1) {
        float top = 0.0f, bad = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          top = fmaxf(top, fabsf(y[j]));
          if (!isfinite(y[j])) bad = 1.0f;
        }
        top = group_max(top, kLanes);
        bad = group_max(bad, kLanes);
        scale = fmaxf(top / 448.0f, 1.17549435e-38f);
        if (bad != 0.0f) {
          scale = CUDART_NAN_F;
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = 0.0f;
        }
      }
      const TokenPlace& t = s_tok[tok];
      if (v0 + m * kGroups + group >= n_all || t.row < 0) continue;
      if constexpr (kOut) {
        T* dst = static_cast<T*>(a.q_out) + (t.row * H + h) * D + 8 * l;
        *reinterpret_cast<uint4*>(dst) = pack8<T>(y);
      } else {
        if (t.page < 0) continue;
        const size_t place = ((((size_t)t.page * H + h) << shift) + t.at);
        TC* dst = static_cast<TC*>(cache) + place * D + 8 * l;
        if constexpr (sizeof(TC) == 1) {
          // a true division: the code of a value on the border between two
          // must not hang on a reciprocal's rounding
          if (scale == scale) {
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = y[j] / scale;
          }
          *reinterpret_cast<uint2*>(dst) = make_uint2(f32_to_e4m3x4(y[0], y[1], y[2], y[3]),
                                                      f32_to_e4m3x4(y[4], y[5], y[6], y[7]));
          if (l == 0) scales[place] = scale;
        } else {
          *reinterpret_cast<uint4*>(dst) = pack8<T>(y);
        }
      }
    }
  }
}

// Dynamic shared memory: s_first [B + 1].
template <typename T, typename TC, int D>
__global__ void __launch_bounds__(kRowThreads, 4) kv_append_kernel(const AppendArgs a) {
  extern __shared__ int s_first[];
  __shared__ int s_warp[kRowThreads / 32];
  __shared__ unsigned s_flags;
  __shared__ TokenPlace s_tok[kRowRun];
  __shared__ alignas(16) float s_cos[kRowRun * D / 2], s_sin[kRowRun * D / 2];  // * rope_scale
  grid_dep_launch();
  grid_dep_wait();
  const KvRows& r = a.rows;
  unsigned flags = 0;
  scan_requests<kRowThreads>(r.B, s_first, s_warp, [&](int b) {
    return checked_new(r, b, r.cache_len[b], r.row_start[b], flags);
  });
  // (rows that overlap against the rules may add up to anything)
  const int total = min(max(s_first[r.B], 0), (int)r.n_rows);
  const int run = run_length(total);
  const int half = a.rot / 2;
  for (int i0 = blockIdx.x * run; i0 < total; i0 += gridDim.x * run) {
    const int n_tok = min(run, total - i0);
    __syncthreads();  // the run before is done with s_tok, s_cos and s_sin
    if (threadIdx.x < n_tok) {
      TokenPlace t;
      if (!token_place(r, s_first, i0 + threadIdx.x, t, flags)) {
        t.row = -1;
        t.pos = t.at = 0;
        t.page = -1;
      }
      s_tok[threadIdx.x] = t;
    }
    __syncthreads();
    // V needs no angles: under way before them
    append_heads<T, TC, D, false>(a, s_tok, s_cos, s_sin, n_tok, a.Hkv, a.by_hkv, a.v, a.v_stride,
                                  nullptr, false, a.v_cache, a.v_scale);
    for (int x = threadIdx.x; x < n_tok * half; x += kRowThreads) {
      const int tok = x / half, i = x - tok * half;
      // the angle in turns, its whole part taken off in fp64: off by some 3e-16 of
      // the turns (1e-11 turns at position 2^18, 5e-8 at 2^30), then fp32
      const double turn = (double)s_tok[tok].pos * a.inv_freq[i] * 0.15915494309189533577;
      float s, c;
      sincospif(2.0f * (float)(turn - rint(turn)), &s, &c);
      const int at = tok * (D / 2) + angle_place(i, half);
      s_cos[at] = c * a.rope_scale;
      s_sin[at] = s * a.rope_scale;
    }
    if (half > 0) __syncthreads();
    append_heads<T, TC, D, false>(a, s_tok, s_cos, s_sin, n_tok, a.Hkv, a.by_hkv, a.k, a.k_stride,
                                  a.k_norm, half > 0, a.k_cache, a.k_scale);
    append_heads<T, TC, D, true>(a, s_tok, s_cos, s_sin, n_tok, a.Hq, a.by_hq, a.q, a.q_stride,
                                 a.q_norm, half > 0, nullptr, nullptr);
  }
  finish_status(a.status, flags, &s_flags);
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
  __shared__ unsigned s_flags;
  __shared__ TokenPlace s_tok[kRowRun];
  grid_dep_launch();
  grid_dep_wait();
  const KvRows& r = a.rows;
  unsigned flags = 0;
  scan_requests<kRowThreads>(r.B, s_first, s_warp, [&](int b) {
    return checked_new(r, b, r.cache_len[b], r.row_start[b], flags);
  });
  // (rows that overlap against the rules may add up to anything)
  const int total = min(max(s_first[r.B], 0), (int)r.n_rows);
  const int run = run_length(total);
  const int l = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const int n_vec = 2 * a.Hkv;
  for (int i0 = blockIdx.x * run; i0 < total; i0 += gridDim.x * run) {
    const int n_tok = min(run, total - i0);
    __syncthreads();
    if (threadIdx.x < n_tok) {
      TokenPlace t;
      if (!token_place(r, s_first, i0 + threadIdx.x, t, flags)) t.row = -1;
      if (t.row < 0 || t.page < 0) t.page = 0;
      s_tok[threadIdx.x] = t;
    }
    __syncthreads();
    // vectors in the order (head, token): a run's tokens lie behind each other
    // in a page of a head
    const int n_all = n_tok * n_vec;
    for (int v0 = group; v0 < n_all; v0 += kGroups * kRowBatch) {
      using In = typename std::conditional<sizeof(TC) == 1, uint2, uint4>::type;
      In in[kRowBatch];
      float scale[kRowBatch];
#pragma unroll
      for (int m = 0; m < kRowBatch; ++m) {
        const int v = v0 + m * kGroups;
        in[m] = In{};
        scale[m] = 1.0f;
        if (v < n_all) {
          const int u = v / n_tok, tok = v - u * n_tok;
          const TokenPlace& t = s_tok[tok];
          const bool is_k = u < a.Hkv;
          const int h = is_k ? u : u - a.Hkv;
          const size_t place = ((((size_t)t.page * a.Hkv + h) << r.page_shift) + t.at);
          if (t.row >= 0) {
            in[m] = *reinterpret_cast<const In*>(
                static_cast<const TC*>(is_k ? a.k_cache : a.v_cache) + place * D + 8 * l);
            if constexpr (sizeof(TC) == 1) scale[m] = (is_k ? a.k_scale : a.v_scale)[place];
          }
        }
      }
#pragma unroll
      for (int m = 0; m < kRowBatch; ++m) {
        const int v = v0 + m * kGroups;
        if (v >= n_all) break;
        const int u = v / n_tok, tok = v - u * n_tok;
        const long long row = s_tok[tok].row;
        if (row < 0) continue;
        const bool is_k = u < a.Hkv;
        const int h = is_k ? u : u - a.Hkv;
        uint4 out;
        if constexpr (sizeof(TC) == 1) {
          float x[8];
          e4m3x4_to_f32(in[m].x, x);
          e4m3x4_to_f32(in[m].y, x + 4);
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] *= scale[m];
          out = pack8<T>(x);
        } else {
          out = in[m];
        }
        T* dst = static_cast<T*>(is_k ? a.k_out : a.v_out) + (row * a.Hkv + h) * D + 8 * l;
        *reinterpret_cast<uint4*>(dst) = out;
      }
    }
  }
  finish_status(a.status, flags, &s_flags);
}

}  // namespace dspark
