// attn_split.cuh -- attention of few rows per key/value head (a decode or
// verify step): up to 32 (token, query head) rows an item.
//
// With so few rows each key is used a handful of times and the cache's bytes
// bound the call: 4 rows D flops per 2 D elements are far below what even the
// warp-level matrix instructions give.  So everything here serves the stream
// of K and V: a producer warp keeps a ring of 32 KB stages (K tile, V tile)
// filled by TMA, two CTAs an SM (192 KB in flight), pieces of equal cost for
// all CTAs (attn_plan.cuh); four consumer warps take a quarter of each tile's
// keys each, with running maximum, sum and result of their own in registers,
// so that no warp waits for another inside an item.  The four results meet in
// shared memory once an item.
//
// mma.m16n8k16: 16 rows are the smallest tile, padded with zero rows.  S =
// Q K^T takes K rows as they lie; O += P V takes V through transposing loads.
// An e4m3 tile is turned into 16-bit fragments in registers: each byte pair
// of K is a pair of neighbours along D (the contraction index may be permuted
// if Q's fragments are permuted alike: a lane takes 4 consecutive elements),
// and a transposing 16-bit load of V gives byte pairs (d, d + 1) of two keys,
// which two byte permutes turn into the fragments of the even and the odd d.
#pragma once

#include <type_traits>

#include "attn_plan.cuh"
#include "attn_tc.cuh"

namespace dspark {

constexpr int kSplitWarps = 4;
constexpr int kSplitThreads = 32 * (kSplitWarps + 1);
constexpr int kSplitStages = 3;
constexpr int kSplitStageBytes = 32768;
constexpr int kSplitItems = 2;  // item descriptors ahead of the consumers

// Keys of a tile: K and V tile of 16 KB each.
template <typename TC, int D>
__host__ __device__ constexpr int split_keys() {
  return kSplitStageBytes / 2 / (D * (int)sizeof(TC));
}

template <typename TC, int D, int MT>
struct SplitSmem {
  alignas(1024) unsigned char stage[kSplitStages][kSplitStageBytes];
  alignas(1024) unsigned char q[MT * 16 * D * 2];
  float scale[kSplitStages][2][sizeof(TC) == 1 ? split_keys<TC, D>() : 4];
  float2 ml[kSplitWarps][MT * 16];
  uint64_t full[kSplitStages], empty[kSplitStages];
  uint64_t item_full[kSplitItems], item_empty[kSplitItems];
  Item item[kSplitItems];
  Piece piece;
  long long scan[kSplitThreads / 32];
  int bad[16];
  unsigned flags;
  int stop;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// d += a b, 16 x 8 x 16.
template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (sizeof(T) == 2 && __is_same(T, __half))
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <typename T, typename TC, int D, int MT>
__global__ void __launch_bounds__(kSplitThreads, 2)
    attn_split_kernel(const AttnArgs a, const AttnParts parts, const __grid_constant__ CUtensorMap mk,
                      const __grid_constant__ CUtensorMap mv, const int box_rows) {
  using S = SplitSmem<TC, D, MT>;
  using TP = typename std::conditional<sizeof(TC) == 1, __nv_bfloat16, T>::type;  // P and V
  constexpr int kKeys = split_keys<TC, D>();
  constexpr int kWarpKeys = kKeys / kSplitWarps;
  constexpr int kRows = MT * 16;
  constexpr bool kQ8 = sizeof(TC) == 1;
  extern __shared__ unsigned char smem_raw[];
  S& sm = *reinterpret_cast<S*>(
      smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const AttnTiles tiles = {kRows, kKeys};
  unsigned flags = 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSplitStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], kSplitWarps);
    }
    for (int i = 0; i < kSplitItems; ++i) {
      mbar_init(&sm.item_full[i], 1);
      mbar_init(&sm.item_empty[i], 1);
    }
    sm.flags = 0;
    fence_barrier_init();
  }
  grid_dep_launch();
  grid_dep_wait();
  find_piece<kSplitThreads>(a, tiles, sm.scan, &sm.piece, flags);  // syncs the block

  if (warp == kSplitWarps) {
    // ---- producer ----
    Walk walk;
    walk.start(a, tiles, sm.piece);
    PartRecord rec = {};
    rec.b = -1;
    int fill = 0, n_item = 0;
    bool alive = true;
    while (alive) {
      const Item it = walk.next(a, tiles);
      const int slot = n_item % kSplitItems;
      if (n_item >= kSplitItems)
        alive = mbar_wait(&sm.item_empty[slot], (uint32_t)(n_item / kSplitItems - 1) & 1u);
      if (!alive) break;
      if (lane == 0) {
        sm.item[slot] = it;
        mbar_arrive(&sm.item_full[slot]);  // release: the descriptor is visible to the waiters
      }
      __syncwarp();
      ++n_item;
      if (it.part < 0) break;
      if (it.part == 1) rec.head = it.part_ends ? 1 : 2;
      if (it.part == 2) {
        rec.row0 = it.row0;
        rec.b = it.b; rec.h = it.h; rec.qt = it.qt;
        rec.n = it.n; rec.past = it.past; rec.n_rows = it.n_rows;
      }
      const int last_key = it.past + it.n;  // keys that exist
      for (int t = it.t0; t < it.t1; ++t, ++fill) {
        const int stage = fill % kSplitStages;
        if (fill >= kSplitStages)
          alive = mbar_wait(&sm.empty[stage], (uint32_t)(fill / kSplitStages - 1) & 1u);
        if (!alive) break;
        const int k0 = t * kKeys;
        const int here = min(kKeys, last_key - k0);
        const int boxes = (here + box_rows - 1) / box_rows;
        if (lane == 0) {
          constexpr int kRowBytes = D * (int)sizeof(TC) + (kQ8 ? 4 : 0);
          mbar_arrive_expect_tx(&sm.full[stage], 2 * boxes * box_rows * kRowBytes);
        }
        __syncwarp();
        if (lane < boxes) {
          const int k = k0 + lane * box_rows;
          int page = checked_page(a.rows, it.b, k >> a.rows.page_shift, flags);
          if (page < 0) page = 0;
          const int y = ((page * a.Hkv + it.h) << a.rows.page_shift) +
                        (k & ((1 << a.rows.page_shift) - 1));
          unsigned char* dk = sm.stage[stage];
          unsigned char* dv = dk + kSplitStageBytes / 2;
          constexpr int kWidth = kQ8 && D == 64 ? 64 : 128;
          constexpr int kHalves = kQ8 ? 1 : D / 64;
#pragma unroll
          for (int hf = 0; hf < kHalves; ++hf) {
            const uint32_t at = hf * kKeys * 128 + lane * box_rows * kWidth;
            tma_load_2d(dk + at, &mk, &sm.full[stage], hf * 64, y);
            tma_load_2d(dv + at, &mv, &sm.full[stage], hf * 64, y);
          }
          if constexpr (kQ8) {
            const uint64_t pol = policy_evict_first();
            bulk_load(&sm.scale[stage][0][lane * box_rows], a.k_scale + y, box_rows * 4,
                      &sm.full[stage], pol);
            bulk_load(&sm.scale[stage][1][lane * box_rows], a.v_scale + y, box_rows * 4,
                      &sm.full[stage], pol);
          }
        }
        __syncwarp();
      }
    }
    if (!alive) flags |= DSPARK_FLAG_TIMEOUT;
    drain_ring_loads(sm.full, kSplitStages, fill);
    if (lane == 0) parts.rec[blockIdx.x] = rec;
  } else {
    // ---- consumers ----
    const int g = lane >> 2, q4 = lane & 3;
    const uint32_t q_base = smem_u32(sm.q);
    bool alive = true;
    int fill = 0, n_item = 0;
    while (true) {
      const int slot = n_item % kSplitItems;
      // one warp waits and says so to the others: all of them stop together
      if (warp == 0) {
        const bool ok = mbar_wait(&sm.item_full[slot], (uint32_t)(n_item / kSplitItems) & 1u);
        if (!ok) flags |= DSPARK_FLAG_TIMEOUT;
        if (lane == 0) sm.stop = !ok || sm.item[slot].part < 0;
      }
      named_sync(1, 32 * kSplitWarps);
      if (sm.stop) break;
      const Item it = sm.item[slot];
      named_sync(1, 32 * kSplitWarps);
      if (threadIdx.x == 0) mbar_arrive(&sm.item_empty[slot]);
      ++n_item;

      // Q rows to shared memory, 16-byte chunks swizzled by the row; rows
      // behind the last are zero
      constexpr int kChunks = D / 8;
      for (int i = threadIdx.x; i < kRows * kChunks; i += 32 * kSplitWarps) {
        const int r = i / kChunks, c = i % kChunks;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < it.n_rows) {
          const int rr = it.qt * kRows + r, tok = a.by_g.div(rr);
          v = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) +
                                              (it.row0 + tok) * a.q_stride +
                                              (it.h * a.G + rr - tok * a.G) * D + 8 * c);
        }
        *reinterpret_cast<uint4*>(sm.q + r * D * 2 + ((c ^ (r & 7)) << 4)) = v;
      }
      named_sync(1, 32 * kSplitWarps);
      // Q fragments of 16 elements along D (in K's order, see above)
      auto load_q = [&](uint32_t (&f)[4], int m, int ks) {
        if constexpr (kQ8) {
          const int c = 2 * ks + (q4 >> 1), r = m * 16 + g;
          const uint2 u = *reinterpret_cast<const uint2*>(sm.q + r * D * 2 + ((c ^ (r & 7)) << 4) +
                                                          (q4 & 1) * 8);
          const uint2 w = *reinterpret_cast<const uint2*>(
              sm.q + (r + 8) * D * 2 + ((c ^ ((r + 8) & 7)) << 4) + (q4 & 1) * 8);
          f[0] = u.x; f[1] = w.x; f[2] = u.y; f[3] = w.y;
        } else {
          const int r = m * 16 + (lane & 15), c = 2 * ks + (lane >> 4);
          ldsm4(f, q_base + r * D * 2 + ((c ^ (r & 7)) << 4));
        }
      };
      constexpr bool kKeepQ = MT == 1;
      uint32_t qf[kKeepQ ? D / 16 : 1][4];
      if constexpr (kKeepQ) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) load_q(qf[ks], 0, ks);
      }
      int pos[MT][2];  // positions of this lane's rows
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int x = 0; x < 2; ++x)
          pos[m][x] = it.past + min(a.by_g.div(it.qt * kRows + m * 16 + g + 8 * x), it.n - 1);
      const int pos_min = it.past + a.by_g.div(it.qt * kRows);
      const int pos_max = it.past + a.by_g.div(it.qt * kRows + it.n_rows - 1);

      float o[MT][D / 8][4], mx[MT][2], sum[MT][2];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          mx[m][x] = -CUDART_INF_F;
          sum[m][x] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
#pragma unroll
          for (int x = 0; x < 4; ++x) o[m][j][x] = 0.0f;
      }

      for (int t = it.t0; t < it.t1; ++t, ++fill) {
        const int stage = fill % kSplitStages;
        if (alive) {
          alive = mbar_wait(&sm.full[stage], (uint32_t)(fill / kSplitStages) & 1u);
          if (!alive) flags |= DSPARK_FLAG_TIMEOUT;
        }
        const int k0 = t * kKeys;
        const int here = it.past + it.n - k0;  // keys of the tile that exist
        const uint32_t kb = smem_u32(sm.stage[stage]), vb = kb + kSplitStageBytes / 2;
        const bool masked = k0 + kKeys > pos_min + 1 ||
                            (a.window > 0 && k0 < pos_max - a.window + 1);
#pragma unroll 1
        for (int s0 = warp * kWarpKeys; s0 < (warp + 1) * kWarpKeys; s0 += 16) {
          if (s0 >= here) break;
          if (!kQ8 && s0 + 16 > here) {
            // what lies behind the sequence in its last page may be anything,
            // and 0 times an infinity is none: clear those rows of V
            for (int i = lane; i < (s0 + 16 - here) * (D / 8); i += 32) {
              const int k = here + i / (D / 8), c = i % (D / 8);
              *reinterpret_cast<uint4*>(sm.stage[stage] + kSplitStageBytes / 2 +
                                        tile_offset<TC, D>(kKeys, k, c)) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          float s[MT][2][4];
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int x = 0; x < 4; ++x) s[m][0][x] = s[m][1][x] = 0.0f;
          if constexpr (kQ8) {
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk) {
              // keys 0-7 and 8-15 of 16 bytes, then of the next 16
              uint32_t f[4];
              ldsm4(f, kb + tile_offset<TC, D>(kKeys, s0 + (lane & 15), 2 * kk + (lane >> 4)));
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t b00 = widen2<T>(__byte_perm(f[2 * x], 0, 0x1404));
                const uint32_t b01 = widen2<T>(__byte_perm(f[2 * x], 0, 0x3424));
                const uint32_t b10 = widen2<T>(__byte_perm(f[2 * x + 1], 0, 0x1404));
                const uint32_t b11 = widen2<T>(__byte_perm(f[2 * x + 1], 0, 0x3424));
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                  if constexpr (kKeepQ) {
                    mma16816<T>(s[m][0], qf[2 * kk + x], b00, b01);
                    mma16816<T>(s[m][1], qf[2 * kk + x], b10, b11);
                  } else {
                    uint32_t qa[4];
                    load_q(qa, m, 2 * kk + x);
                    mma16816<T>(s[m][0], qa, b00, b01);
                    mma16816<T>(s[m][1], qa, b10, b11);
                  }
                }
              }
            }
          } else {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              uint32_t f[4];
              ldsm4(f, kb + tile_offset<TC, D>(kKeys, s0 + (lane & 7) + (lane >> 4) * 8,
                                               2 * ks + ((lane >> 3) & 1)));
#pragma unroll
              for (int m = 0; m < MT; ++m) {
                if constexpr (kKeepQ) {
                  mma16816<T>(s[m][0], qf[ks], f[0], f[1]);
                  mma16816<T>(s[m][1], qf[ks], f[2], f[3]);
                } else {
                  uint32_t qa[4];
                  load_q(qa, m, ks);
                  mma16816<T>(s[m][0], qa, f[0], f[1]);
                  mma16816<T>(s[m][1], qa, f[2], f[3]);
                }
              }
            }
          }
          // scores in units of log 2; keys of this lane: 2 q4 + {0, 1} of each 8
          float vs[2][2];
          {
            float ks[2][2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                ks[j][x] = a.scale2;
                vs[j][x] = 1.0f;
                if constexpr (kQ8) {
                  const int k = s0 + 8 * j + 2 * q4 + x;
                  ks[j][x] *= sm.scale[stage][0][k];
                  vs[j][x] = sm.scale[stage][1][k];
                }
              }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int x = 0; x < 4; ++x) s[m][j][x] *= ks[j][x & 1];
          }
          if (masked) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  const int key = k0 + s0 + 8 * j + 2 * q4 + (x & 1);
                  const int p = pos[m][x >> 1];
                  if (key > p || key < first_seen(p, a.window)) s[m][j][x] = -CUDART_INF_F;
                }
          }
          uint32_t pf[MT][4];
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            float top[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              top[x] = fmaxf(fmaxf(s[m][0][2 * x], s[m][0][2 * x + 1]),
                             fmaxf(s[m][1][2 * x], s[m][1][2 * x + 1]));
              top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 1));
              top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 2));
              top[x] = fmaxf(top[x], mx[m][x]);
            }
            if (__any_sync(0xffffffffu, top[0] > mx[m][0] || top[1] > mx[m][1])) {
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const float f = mx[m][x] == -CUDART_INF_F ? 0.0f : ex2(mx[m][x] - top[x]);
                mx[m][x] = top[x];
                sum[m][x] *= f;
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                  o[m][j][2 * x] *= f;
                  o[m][j][2 * x + 1] *= f;
                }
              }
            }
            float p[2][4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const float ref = mx[m][x >> 1] == -CUDART_INF_F ? 0.0f : mx[m][x >> 1];
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                p[j][x] = ex2(s[m][j][x] - ref);
                sum[m][x >> 1] += p[j][x];
                // a masked position's scale may be anything
                if constexpr (kQ8)
                  p[j][x] = s[m][j][x] == -CUDART_INF_F ? 0.0f : p[j][x] * vs[j][x & 1];
              }
            }
            pf[m][0] = Pair<TP>::put(p[0][0], p[0][1]);
            pf[m][1] = Pair<TP>::put(p[0][2], p[0][3]);
            pf[m][2] = Pair<TP>::put(p[1][0], p[1][1]);
            pf[m][3] = Pair<TP>::put(p[1][2], p[1][3]);
          }
#pragma unroll
          for (int dd = 0; dd < D / 16; ++dd) {
            uint32_t b[2][2];
            if constexpr (kQ8) {
              // 16 keys x 16 bytes; a second chunk rides along in the upper lanes
              if (dd % 2 == 0) {
                uint32_t f[4];
                ldsm4t(f, vb + tile_offset<TC, D>(kKeys, s0 + (lane & 15), dd + (lane >> 4)));
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  b[0][0] = widen2<TP>(__byte_perm(f[2 * y], 0, 0x2404));
                  b[0][1] = widen2<TP>(__byte_perm(f[2 * y + 1], 0, 0x2404));
                  b[1][0] = widen2<TP>(__byte_perm(f[2 * y], 0, 0x3414));
                  b[1][1] = widen2<TP>(__byte_perm(f[2 * y + 1], 0, 0x3414));
#pragma unroll
                  for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int z = 0; z < 2; ++z)
                      mma16816<TP>(o[m][2 * (dd + y) + z], pf[m], b[z][0], b[z][1]);
                }
              }
            } else {
              uint32_t f[4];
              ldsm4t(f, vb + tile_offset<TC, D>(kKeys, s0 + (lane & 15), 2 * dd + (lane >> 4)));
#pragma unroll
              for (int m = 0; m < MT; ++m) {
                mma16816<TP>(o[m][2 * dd], pf[m], f[0], f[1]);
                mma16816<TP>(o[m][2 * dd + 1], pf[m], f[2], f[3]);
              }
            }
          }
        }
        // the last stage serves as scratch below before it is released
        if (t + 1 < it.t1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.empty[stage]);
        }
      }

      // ---- the four warps' results of the item, in the order of the warps ----
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float l = sum[m][x];
          l += __shfl_xor_sync(0xffffffffu, l, 1);
          l += __shfl_xor_sync(0xffffffffu, l, 2);
          if (q4 == 0) sm.ml[warp][m * 16 + g + 8 * x] = make_float2(mx[m][x], l);
        }
      const int stage = (fill - 1) % kSplitStages;
      float* scratch = reinterpret_cast<float*>(sm.stage[stage]);
      const bool whole = it.part == 0;
      const size_t slot_row = (size_t)(2 * blockIdx.x + (it.part == 2)) * kRows;
      named_sync(1, 32 * kSplitWarps);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (m * 16 < it.n_rows) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int r = g + 8 * x;
            float M = sm.ml[0][m * 16 + r].x;
#pragma unroll
            for (int w = 1; w < kSplitWarps; ++w) M = fmaxf(M, sm.ml[w][m * 16 + r].x);
            const float f = mx[m][x] == -CUDART_INF_F ? 0.0f : ex2(mx[m][x] - M);
            float* row = scratch + (warp * 16 + r) * D;
            const int sw = (r & 3) << 3;  // a quarter warp's rows on different banks
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
              if constexpr (kQ8) {
                // even and odd elements of 16 in two accumulators: 4 in a row
                if (j % 2 == 0)
                  *reinterpret_cast<float4*>(row + ((j * 8 + 4 * q4) ^ sw)) =
                      make_float4(o[m][j][2 * x] * f, o[m][j + 1][2 * x] * f,
                                  o[m][j][2 * x + 1] * f, o[m][j + 1][2 * x + 1] * f);
              } else {
                *reinterpret_cast<float2*>(row + ((j * 8 + 2 * q4) ^ sw)) =
                    make_float2(o[m][j][2 * x] * f, o[m][j][2 * x + 1] * f);
              }
            }
          }
        }
        if (threadIdx.x < 16) sm.bad[threadIdx.x] = 0;
        named_sync(1, 32 * kSplitWarps);
        for (int i = threadIdx.x; i < 16 * (D / 4); i += 32 * kSplitWarps) {
          const int r = i / (D / 4), c = i % (D / 4) * 4;
          if (m * 16 + r >= it.n_rows) break;
          float M = -CUDART_INF_F, L = 0.0f;
#pragma unroll
          for (int w = 0; w < kSplitWarps; ++w) M = fmaxf(M, sm.ml[w][m * 16 + r].x);
          const float Mu = M == -CUDART_INF_F ? 0.0f : M;
          float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int w = 0; w < kSplitWarps; ++w) {
            const float2 ml = sm.ml[w][m * 16 + r];
            L = fmaf(ex2(ml.x - Mu), ml.y, L);
            const float4 u = *reinterpret_cast<const float4*>(scratch + (w * 16 + r) * D +
                                                              (c ^ ((r & 3) << 3)));
            v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
          }
          if (whole) {
            const float inv = 1.0f / L;
            v.x *= inv; v.y *= inv; v.z *= inv; v.w *= inv;
            if (!isfinite(v.x) || !isfinite(v.y) || !isfinite(v.z) || !isfinite(v.w)) sm.bad[r] = 1;
            const int rr = it.qt * kRows + m * 16 + r, tok = a.by_g.div(rr);
            T* dst = static_cast<T*>(a.out) +
                     ((it.row0 + tok) * a.Hq + it.h * a.G + rr - tok * a.G) * D + c;
            *reinterpret_cast<uint2*>(dst) =
                make_uint2(Pair<T>::put(v.x, v.y), Pair<T>::put(v.z, v.w));
          } else {
            *reinterpret_cast<float4*>(parts.o + (slot_row + m * 16 + r) * D + c) = v;
            if (c == 0) parts.ml[slot_row + m * 16 + r] = make_float2(M, L);
          }
        }
        named_sync(1, 32 * kSplitWarps);
        // a result that is not finite may come from a position that its row
        // does not see (0 times infinity): form the row again from those it sees
        if (whole) {
          for (int r = warp; r < 16; r += kSplitWarps) {
            if (!sm.bad[r]) continue;
            const int rr = it.qt * kRows + m * 16 + r, tok = a.by_g.div(rr);
            attend_row<T, TC, D>(a, it.b, it.past + tok, it.h * a.G + rr - tok * a.G,
                                 it.row0 + tok, flags);
          }
          named_sync(1, 32 * kSplitWarps);
        }
      }
      // the scratch was written through the generic proxy, the next fill comes
      // through the async one
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.empty[stage]);
    }
  }
  if (flags) atomicOr(&sm.flags, flags);
  __syncthreads();
  if (threadIdx.x == 0) store_status(a.status, sm.flags);
}

}  // namespace dspark
