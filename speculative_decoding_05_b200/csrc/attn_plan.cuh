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
// Bounds and figures: a batch of up to 32 requests is cut by one warp (a step of
// one token in a graph 13.6 -> 13.1 us); the join reads every part once, 7 us of
// an e4m3 serving step, some 20 of a chunk's call.
#pragma once

#include <type_traits>

#include "attn_rows.cuh"
#include "tc_common.cuh"

namespace dspark {

// What an item costs besides its key tiles, in key tiles: rows loaded,
// results merged and stored.  Measured (us) at 1, 2 and 4: 64 requests x 9 tokens
// 127, 121, 117; e4m3 serving step 330, 312, 304; fp16 decode of heads of 64 190,
// 167, 162; chunk 400, 390, 384; one token over 131071 104.5, 105, 105.5.
constexpr int kItemCost = 2;
// Least cost of a CTA's piece: a further CTA also costs a part for the join.  At 1,
// 2 and 4: one request's block of 17 tokens 31.6, 31.6, 29.8, one token over 512
// 14.6, 14.6, 14.9; batches are the same.
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

// The piece that starts at `start`, in request b (of the given length, rows and
// cost a head) whose first item starts at `at`.
__device__ __forceinline__ void set_piece(const AttnArgs& a, const AttnTiles& t, Piece* p, int b,
                                          int n, int past, long long row0, long long head,
                                          long long start, long long at, long long len) {
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
  p->b = b;
  p->h = h;
  p->qt = qt;
  p->n = n;
  p->past = past;
  p->row0 = row0;
  p->off = off;
  p->len = len;
}
// Start and length of this CTA's piece of a line of `total`: equal pieces, the
// first ones longer by one; false if it has none.
__device__ __forceinline__ bool cut_line(long long total, long long& start, long long& len) {
  long long ctas = total / kMinPiece;
  if (ctas > gridDim.x) ctas = gridDim.x;
  if (ctas < 1) ctas = 1;
  const long long c = blockIdx.x;
  if (c >= ctas) return false;
  const long long each = quotient(total, ctas), more = total - each * ctas;
  start = c * each + min(c, more);
  len = each + (c < more);
  return len > 0;
}

// This CTA's piece of the line by one warp, for up to 32 requests: no thread of
// the block waits for another (a short call's first loads come 1 us earlier).
__device__ __forceinline__ Piece find_piece_warp(const AttnArgs& a, const AttnTiles& t,
                                                 unsigned& flags) {
  const KvRows& r = a.rows;
  const int lane = threadIdx.x & 31;
  int past = 0, n = 0;
  long long row0 = 0, head = 0;
  if (lane < r.B) {
    past = r.cache_len[lane];
    row0 = r.row_start[lane];
    n = checked_new(r, lane, past, row0, flags);
    if (n) head = head_cost(t, a, n, past);
  }
  const long long mine = a.Hkv * head;
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  const long long total = __shfl_sync(0xffffffffu, incl, 31);
  Piece p = {};
  long long start = 0, len = 0;
  if (!cut_line(total, start, len)) return p;
  const unsigned upto = __ballot_sync(0xffffffffu, incl > start);
  const int b = __ffs(upto) - 1;  // (start < total: there is one)
  n = __shfl_sync(0xffffffffu, n, b);
  past = __shfl_sync(0xffffffffu, past, b);
  row0 = __shfl_sync(0xffffffffu, row0, b);
  head = __shfl_sync(0xffffffffu, head, b);
  const long long at = __shfl_sync(0xffffffffu, incl - mine, b);
  set_piece(a, t, &p, b, n, past, row0, head, start, at, len);
  return p;
}

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
  long long start = 0, len = 0;
  if (cut_line(total, start, len) && start >= pre && start < pre + mine) {
    long long at = pre;
    for (int b = b0; b < b1; ++b) {
      const long long k = per == 1 ? mine : request(b);
      if (start < at + k) {
        set_piece(a, t, s_piece, b, n, past, row0, head, start, at, len);
        break;
      }
      at += k;
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
constexpr int kJoinPerSm = 4;  // blocks: a row is a chain of loads, more rows at a time hide it
constexpr int kMaxAttnCtas = 256;

// Joins the parts of split items: out = sum_i 2^(m_i - M) o_i / sum_i
// 2^(m_i - M) l_i over an item's parts in the order of their keys: slot 1 of the
// CTA that began it, then slot 0 of the CTAs behind it up to the one that ends
// it.  A warp a row; the rows of all split items are one line, dealt out over
// all warps (few items have many rows and parts, many have few).
template <typename T, typename TC, int D>
__global__ void __launch_bounds__(kJoinThreads, kJoinPerSm)
    attn_join_kernel(const AttnArgs a, const int tile_rows, const AttnParts p, const int ctas) {
  constexpr int E = D / 32;  // elements of a lane
  using V = typename std::conditional<E == 4, float4, float2>::type;
  __shared__ int s_head[kMaxAttnCtas], s_first[kMaxAttnCtas + 1], s_warp[kJoinThreads / 32];
  static_assert(kMaxAttnCtas <= kJoinThreads, "a record a thread");
  grid_dep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  scan_requests<kJoinThreads>(ctas, s_first, s_warp, [&](int c) {
    s_head[c] = p.rec[c].head;
    return p.rec[c].b >= 0 ? p.rec[c].n_rows : 0;
  });
  const int total = s_first[ctas];
  constexpr int kWarps = kJoinThreads / 32;
  for (int i = blockIdx.x * kWarps + warp; i < total; i += gridDim.x * kWarps) {
    const int c0 = find_request(s_first, ctas, i);
    const int r = i - s_first[c0];
    const PartRecord rec = p.rec[c0];
    float o[E], M = -CUDART_INF_F, L = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.0f;
    // parts in batches, so that their loads overlap
    constexpr int kBatch = 6;
    int c = c0;
    bool more = true;
    while (more) {
      float2 ml[kBatch];
      V v[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        int slot = -1;
        if (more) {
          if (c > c0)
            while (c < ctas - 1 && s_head[c] == 0) ++c;  // CTAs without keys of this item
          slot = c == c0 ? 2 * c + 1 : 2 * c;
          more = c < ctas - 1 && (c == c0 || s_head[c] == 2);
          ++c;
        }
        ml[k] = make_float2(-CUDART_INF_F, 0.0f);
        v[k] = V{};
        if (slot >= 0) {
          const size_t at = (size_t)slot * tile_rows + r;
          ml[k] = p.ml[at];
          v[k] = *reinterpret_cast<const V*>(p.o + at * D + lane * E);
        }
      }
      float Mn = M;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) Mn = fmaxf(Mn, ml[k].x);
      const float Mu = Mn == -CUDART_INF_F ? 0.0f : Mn;
      const float back = exp2f(M - Mu);
      L *= back;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= back;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float w = exp2f(ml[k].x - Mu);
        L = fmaf(w, ml[k].y, L);
        const float* x = reinterpret_cast<const float*>(&v[k]);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(w, x[e], o[e]);
      }
      M = Mn;
    }
    const float inv = 1.0f / L;
    bool odd = false;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      o[e] *= inv;
      odd |= !isfinite(o[e]);
    }
    const int rr = rec.qt * tile_rows + r, tok = a.by_g.div(rr);
    const int hq = rec.h * a.G + rr - tok * a.G;
    if (__any_sync(0xffffffffu, odd)) {
      // a result that is not finite may come from a position that its row does
      // not see (0 times infinity): form the row again from those it sees
      unsigned flags = 0;
      attend_row<T, TC, D>(a, rec.b, rec.past + tok, hq, rec.row0 + tok, flags);
    } else {
      T* dst = static_cast<T*>(a.out) + ((rec.row0 + tok) * a.Hq + hq) * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t*>(dst + e) = Pair<T>::put(o[e], o[e + 1]);
    }
  }
}

// ---------------------------------------------------------------------------
// the cache as a tensor map
// ---------------------------------------------------------------------------

// A cache [n_pages * Hkv * page_size, D] as boxes of `box_rows` rows x 128
// bytes (64 where an e4m3 row has no more), swizzled over that width.
bool encode_cache_map(CUtensorMap* m, const void* cache, int D, bool is_e4m3, bool is_f16,
                      long long rows, int box_rows);

}  // namespace dspark
