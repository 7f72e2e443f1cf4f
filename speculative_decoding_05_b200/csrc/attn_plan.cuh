// attn_plan.cuh -- how dspark_attn_verify divides its work: which keys of
// which rows a CTA takes, where it leaves partial results, how they are joined.
//
// An item is one tile of `rows` consecutive (token, query head) rows of one
// request and one key/value head, row r = token * G + head; it costs its key
// tiles plus kItemCost.  All items in the order (request, head, row tile) form
// one line, cut into equal pieces, one a CTA: lengths are known on the device
// only and may be anything, so every CTA works the cut out for itself (a scan
// over the requests, a few hundred instructions) instead of waiting for a
// planning launch.  A CTA's piece is some whole items and at most two parts of
// items: the end of one that began before it and the start of one that goes
// on behind it.  Parts leave (maximum, sum, unnormalised result) of their rows
// in the workspace and a second launch joins them in the order of the keys, so
// results do not depend on timing.
#pragma once

#include "attn_rows.cuh"
#include "tc_common.cuh"

namespace dspark {

// What an item costs besides its key tiles, in key tiles: rows loaded,
// results merged and stored.
constexpr int kItemCost = 2;
// Least cost of a CTA's piece.  Below it a further CTA saves less than the
// join of its part costs.
constexpr int kMinPiece = 2;

struct AttnTiles {
  int rows;  // rows of an item
  int keys;  // keys of a tile
};

// Key tiles of row tile qt, and the first of them.
__device__ __forceinline__ int item_tiles(const AttnTiles& t, const AttnArgs& a, int n, int past,
                                          int qt, int& lo) {
  const int first = a.by_g.div(qt * t.rows);
  const int last = a.by_g.div(min((qt + 1) * t.rows, n * a.G) - 1);
  lo = first_seen(past + first, a.window) / t.keys;
  return (past + last) / t.keys + 1 - lo;
}
__device__ __forceinline__ int row_tiles(const AttnTiles& t, int G, int n) {
  return (n * G + t.rows - 1) / t.rows;
}
// Cost of one head of a request.
__device__ __forceinline__ long long head_cost(const AttnTiles& t, const AttnArgs& a, int n,
                                               int past) {
  long long c = 0;
  const int nq = row_tiles(t, a.G, n);
  for (int qt = 0; qt < nq; ++qt) {
    int lo;
    c += item_tiles(t, a, n, past, qt, lo) + kItemCost;
  }
  return c;
}
// x / y, by the short way where both fit 32 bits.
__device__ __forceinline__ long long quotient(long long x, long long y) {
  if (((x | y) >> 32) == 0) return (unsigned)x / (unsigned)y;
  return x / y;
}

struct Piece {
  long long len;       // cost
  long long off;       // start behind the start of its first item
  long long row0;      // first item: see Item
  int b, h, qt, n, past;
};

// This CTA's piece of the line, by the NT threads of the block.
template <int NT>
__device__ __forceinline__ void find_piece(const AttnArgs& a, const AttnTiles& t,
                                           long long* s_warp, Piece* s_piece, unsigned& flags) {
  const KvRows& r = a.rows;
  const int per = (r.B + NT - 1) / NT;
  const int b0 = threadIdx.x * per, b1 = min(b0 + per, r.B);
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int past = 0, n = 0;
  long long row0 = 0, head = 0;
  auto request = [&](int b) {  // the four above, and the request's cost
    past = r.cache_len[b];
    row0 = r.row_start[b];
    n = checked_new(r, b, past, row0, flags);
    head = n ? head_cost(t, a, n, past) : 0;
    return a.Hkv * head;
  };
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += request(b);
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_warp[w] = incl;
  if (threadIdx.x == 0) {
    s_piece->b = s_piece->h = s_piece->qt = s_piece->n = s_piece->past = 0;
    s_piece->len = s_piece->off = s_piece->row0 = 0;
  }
  __syncthreads();
  long long pre = incl - mine, total = 0;
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) {
    const long long v = s_warp[i];
    if (i < w) pre += v;
    total += v;
  }
  long long ctas = total / kMinPiece;
  if (ctas > gridDim.x) ctas = gridDim.x;
  if (ctas < 1) ctas = 1;
  const long long c = blockIdx.x;
  if (c < ctas) {
    // equal pieces, the first total % ctas of them longer by one
    const long long len = quotient(total, ctas), more = total - len * ctas;
    const long long start = c * len + min(c, more);
    const long long mylen = len + (c < more);
    if (mylen > 0 && start >= pre && start < pre + mine) {
      long long at = pre;
      for (int b = b0; b < b1; ++b) {
        const long long k = per == 1 ? mine : request(b);
        if (start < at + k) {
          long long off = start - at;
          const int h = (int)quotient(off, head);
          off -= h * head;
          int qt = 0, lo;
          while (true) {
            const int ic = item_tiles(t, a, n, past, qt, lo) + kItemCost;
            if (off < ic) break;
            off -= ic;
            ++qt;
          }
          s_piece->b = b;
          s_piece->h = h;
          s_piece->qt = qt;
          s_piece->n = n;
          s_piece->past = past;
          s_piece->row0 = row0;
          s_piece->off = off;
          s_piece->len = mylen;
          break;
        }
        at += k;
      }
    }
  }
  __syncthreads();
}

// One item, or the part of it that lies in a CTA's piece.
struct Item {
  long long row0;      // row of the request's first new token
  int b, h, qt;
  int n, past;         // new tokens, tokens before them
  int t0, t1;          // key tiles of this part
  int n_rows;          // rows of the tile
  int part;            // 0: all keys; 1: continues an earlier CTA's; 2: first part; -1: no item
  int part_ends;       // part == 1: whether the item ends here
};

// Steps through a piece; every caller gets the same items.
struct Walk {
  long long left, off;  // cost left in the piece; cost of the current item before the piece
  int b, h, qt, n, past, nq;
  long long row0;
  bool open;

  __device__ __forceinline__ void request(const AttnArgs& a, const AttnTiles& t, int b_) {
    unsigned ignore = 0;
    b = b_;
    n = 0;
    while (b < a.rows.B) {
      past = a.rows.cache_len[b];
      row0 = a.rows.row_start[b];
      n = checked_new(a.rows, b, past, row0, ignore);
      if (n) break;
      ++b;
    }
    nq = row_tiles(t, a.G, n);
    h = 0;
    qt = 0;
  }
  __device__ __forceinline__ void start(const AttnArgs& a, const AttnTiles& t, const Piece& p) {
    left = p.len;
    open = left > 0;
    off = p.off;
    b = p.b;
    h = p.h;
    qt = p.qt;
    n = p.n;
    past = p.past;
    row0 = p.row0;
    nq = row_tiles(t, a.G, n);
  }
  // The next item with key tiles in the piece; part = -1 at its end.
  __device__ __forceinline__ Item next(const AttnArgs& a, const AttnTiles& t) {
    Item it;
    it.part = -1;
    while (open && left > 0 && b < a.rows.B) {
      int lo;
      const int nt = item_tiles(t, a, n, past, qt, lo);
      const long long begin = off, end = min(off + left, (long long)(nt + kItemCost));
      const int t0 = (int)max(begin - kItemCost, 0ll), t1 = (int)max(end - kItemCost, 0ll);
      if (t1 > t0) {
        it.row0 = row0;
        it.b = b; it.h = h; it.qt = qt; it.n = n; it.past = past;
        it.t0 = lo + t0;
        it.t1 = lo + t1;
        it.n_rows = min(t.rows, n * a.G - qt * t.rows);
        it.part = t0 > 0 ? 1 : t1 < nt ? 2 : 0;
        it.part_ends = t1 == nt;
      }
      left -= end - begin;
      off = 0;
      if (++qt == nq) {
        qt = 0;
        if (++h == a.Hkv) request(a, t, b + 1);
      }
      if (it.part >= 0) return it;
    }
    return it;
  }
};

// ---------------------------------------------------------------------------
// parts
// ---------------------------------------------------------------------------

// Which parts CTA c left: `head` 0 none, 1 the end of an item, 2 the middle of
// one (slot 0); `b` >= 0 the start of an item (slot 1).
struct PartRecord {
  long long row0;
  int head, b, h, qt, n, past, n_rows, pad;
};
static_assert(sizeof(PartRecord) == 40, "record");

struct AttnParts {
  PartRecord* rec;  // [CTAs]
  float2* ml;       // [CTAs][2][rows]: maximum (of scores times log2 e), sum
  float* o;         // [CTAs][2][rows][D]
};

struct PartBytes {
  size_t rec, ml, o, total;
};
__host__ inline PartBytes part_bytes(int ctas, int rows, int D) {
  PartBytes p;
  p.rec = kKvHeaderBytes;
  p.ml = p.rec + align256((size_t)ctas * sizeof(PartRecord));
  p.o = p.ml + align256((size_t)ctas * 2 * rows * sizeof(float2));
  p.total = p.o + align256((size_t)ctas * 2 * rows * D * sizeof(float));
  return p;
}

constexpr int kJoinThreads = 256;

// Joins the parts of the item that CTA blockIdx.x began: out = sum_i 2^(m_i - M)
// o_i / sum_i 2^(m_i - M) l_i over the parts in the order of their keys.
// blockIdx.y takes every gridDim.y-th group of rows.
template <typename T, typename TC, int D>
__global__ void __launch_bounds__(kJoinThreads)
    attn_join_kernel(const AttnArgs a, const AttnTiles t, const AttnParts p, int ctas) {
  constexpr int kLanes = D / 4;               // threads of a row, 4 elements each
  constexpr int kRows = kJoinThreads / kLanes;
  __shared__ int s_parts[kMaxStatusCtas];
  __shared__ int s_n;
  __shared__ int s_bad[kRows];
  grid_dep_wait();
  const int c0 = blockIdx.x;
  const PartRecord rec = p.rec[c0];
  if (rec.b < 0) return;
  // the parts: slot 1 of c0, then slot 0 of the CTAs behind it up to the one
  // that ends the item (32 records at a time)
  if (threadIdx.x < 32) {
    int n = 0;
    for (int c = c0 + 1; c < ctas; c += 32) {
      const int head = c + threadIdx.x < ctas ? p.rec[c + threadIdx.x].head : 0;
      const unsigned ends = __ballot_sync(0xffffffffu, head == 1);
      const unsigned upto = ends ? (2u << (__ffs(ends) - 1)) - 1u : 0xffffffffu;
      const unsigned in = __ballot_sync(0xffffffffu, head != 0) & upto;
      if (in >> threadIdx.x & 1)
        s_parts[n + __popc(in & ((1u << threadIdx.x) - 1u))] = 2 * (c + threadIdx.x);
      n += __popc(in);
      if (ends) break;
    }
    if (threadIdx.x == 0) s_n = n;
  }
  __syncthreads();
  const int n = s_n;
  const int lane = threadIdx.x % kLanes, rg = threadIdx.x / kLanes;
  for (int r0 = blockIdx.y * kRows; r0 < rec.n_rows; r0 += gridDim.y * kRows) {
    const int r = r0 + rg;
    if (lane == 0) s_bad[rg] = 0;
    __syncthreads();
    if (r < rec.n_rows) {
      const size_t first = (size_t)(2 * c0 + 1) * t.rows + r;
      float M = p.ml[first].x;
      for (int i = 0; i < n; ++i) M = fmaxf(M, p.ml[(size_t)s_parts[i] * t.rows + r].x);
      const float Mu = M == -CUDART_INF_F ? 0.0f : M;
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float L = 0.0f;
#pragma unroll 4
      for (int i = -1; i < n; ++i) {
        const size_t at = i < 0 ? first : (size_t)s_parts[i] * t.rows + r;
        const float2 ml = p.ml[at];
        const float4 v = *reinterpret_cast<const float4*>(p.o + at * D + 4 * lane);
        const float w = exp2f(ml.x - Mu);
        L = fmaf(w, ml.y, L);
        o.x = fmaf(w, v.x, o.x); o.y = fmaf(w, v.y, o.y);
        o.z = fmaf(w, v.z, o.z); o.w = fmaf(w, v.w, o.w);
      }
      const float inv = 1.0f / L;
      o.x *= inv; o.y *= inv; o.z *= inv; o.w *= inv;
      if (!isfinite(o.x) || !isfinite(o.y) || !isfinite(o.z) || !isfinite(o.w)) s_bad[rg] = 1;
      const int rr = rec.qt * t.rows + r, tok = a.by_g.div(rr);
      T* dst = static_cast<T*>(a.out) +
               ((rec.row0 + tok) * a.Hq + rec.h * a.G + rr - tok * a.G) * D + 4 * lane;
      *reinterpret_cast<uint2*>(dst) = make_uint2(Pair<T>::put(o.x, o.y), Pair<T>::put(o.z, o.w));
    }
    __syncthreads();
    // a result that is not finite may come from a position that its row does
    // not see (0 times infinity): form the row again from those it sees
    for (int k = threadIdx.x / 32; k < kRows; k += kJoinThreads / 32) {
      if (!s_bad[k]) continue;
      const int rr = rec.qt * t.rows + r0 + k, tok = a.by_g.div(rr);
      unsigned flags = 0;
      attend_row<T, TC, D>(a, rec.b, rec.past + tok, rec.h * a.G + rr - tok * a.G, rec.row0 + tok,
                           flags);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// the cache as a tensor map
// ---------------------------------------------------------------------------

// A cache [n_pages * Hkv * page_size, D] as boxes of `box_rows` rows x 128
// bytes (64 where an e4m3 row has no more), swizzled over that width.
bool encode_cache_map(CUtensorMap* m, const void* cache, int D, bool is_e4m3, bool is_f16,
                      long long rows, int box_rows);

// Byte offset of 16-byte chunk c of key row k in a tile of `keys` keys.
template <typename TC, int D>
__device__ __forceinline__ uint32_t tile_offset(int keys, int k, int c) {
  if constexpr (sizeof(TC) == 1 && D == 64)
    return (uint32_t)(k * 64 + ((c ^ ((k >> 1) & 3)) << 4));
  else
    return (uint32_t)((c >> 3) * keys * 128 + k * 128 + (((c & 7) ^ (k & 7)) << 4));
}

}  // namespace dspark
