// attn_chunk.cuh -- attention of many rows per key/value head (a prompt's
// chunk) over a 16-bit cache: 256 (token, query head) rows an item.
//
// Here each key meets hundreds of rows and the tensor cores and the exponentials
// bound the call: a tile of 256 rows x 128 keys at D = 128 takes 2160 clocks of
// MMAs (measured 68 an instruction of 128 x 128 x 16) and 2048 of exponentials
// (16 a clock and SM).  So both must run all the time: two row tiles of 128 in
// turn, one's softmax while the other's products are formed,
//   S_p [128 rows, 128 keys] = Q_p K^T
//   P_p = 2^(S_p - m), 16 bits (V's type, as in the step kernel), back to TMEM over S_p
//   O_p [128 rows, D]       += P_p V      P from TMEM, V as it lies (MN-major)
// with the MMAs in the order S0 S1 | PV0 S0' PV1 S1' | ..  A thread owns one row
// of 64 keys: with all 128 a tile's softmax was a chain so long that the products
// waited for it (4400 clocks a pair of tiles, 862 TFLOP/s).  The two threads of a
// row share its reference m, which starts at 0 and moves only when a score leaves
// 2^+-kHot (fp16 weights: at the first tile), as in the step kernel, so that O is
// hardly ever rescaled; their two warps meet once a tile, to vote on that and
// because the weights of one lie over the scores of the other.
//
// Measured: 390 to 399 us (by the box) for chunks of 2 x 2048 tokens behind 2000 to
// 6000, 875 to 890 TFLOP/s, 53 % of the measured matrix rate; a pair of tiles takes some 3600
// clocks of the 2160, what remains is the chain scores - weights - product of each.
//
// Warps: 16 softmax (two groups a row tile, which also load its Q rows), one that
// loads K and V, one that issues the MMAs, one that clears V behind the end of a
// sequence.
#pragma once

#include "attn_step.cuh"

namespace dspark {

constexpr int kChunkRows = 256;
constexpr int kChunkKeys = 128;
constexpr int kChunkSoftmax = 16;  // warps
constexpr int kChunkLoad = kChunkSoftmax;
constexpr int kChunkMma = kChunkSoftmax + 1;
constexpr int kChunkClean = kChunkSoftmax + 2;
constexpr int kChunkThreads = 32 * (kChunkSoftmax + 3);
constexpr int kChunkItems = 2;

template <int D>
struct ChunkSmem {
  static constexpr int kTile = kChunkKeys * D * 2;
  static constexpr int kOps = D == 128 ? 4 : 8;
  alignas(1024) unsigned char op[kOps][kTile];
  alignas(1024) unsigned char q[2][128 * D * 2];
  float part[2][2][128], odd[2][2][128];  // of the two halves of each row tile's rows
  uint64_t full[kOps], empty[kOps];
  uint64_t q_full, s_full[2], p_full[2], o_full[2];
  uint64_t item_full[kChunkItems], item_empty[kChunkItems], v_clean[kChunkItems];
  uint64_t drain;
  Item item[kChunkItems];
  Piece piece;
  long long scan[kChunkThreads / 32 + 1];
  uint32_t tmem;
  unsigned flags;
  int slow;  // see mbar_wait_slow
  int stop, last, next;
};

// Key tiles of row tile p of an item's part (0: it has no rows, or sees none).
__device__ __forceinline__ int chunk_tiles(const AttnArgs& a, const Item& it, int p) {
  if (it.n_rows <= 128 * p) return 0;
  const int r = it.qt * kChunkRows + min(128 * (p + 1), it.n_rows) - 1;
  const int n = (it.past + a.by_g.div(r)) / kChunkKeys + 1;
  return max(min(it.t1, n) - it.t0, 0);
}

// Waits of this kernel, whose softmax warps may be held up by attend_row: it ends,
// but where all rows of a long sequence need it a CTA takes seconds.  `slow` counts
// the warps that went into it and have not done an item's tiles since, and a
// wait's limit runs anew while there are any.  The softmax warps' own waits have
// the plain limit (they start an item together, when none is in attend_row any
// more), so these end as well.  (The step kernel has a fifth of the rows, and its
// e4m3 form lost 7 % to these few instructions: plain waits there.)
template <typename F>
__device__ __forceinline__ bool wait_slow(const volatile int* slow, F&& wait) {
  do {
    if (wait()) return true;
  } while (*slow);
  return false;
}
__device__ __forceinline__ bool mbar_wait_slow(const volatile int* slow, uint64_t* bar,
                                               uint32_t parity) {
  return wait_slow(slow, [&] { return mbar_wait(bar, parity); });
}
__device__ __forceinline__ void count_slow(int* slow, int by) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) atomicAdd(slow, by);
}

template <typename T, int D>
__global__ void __launch_bounds__(kChunkThreads, 1)
    attn_chunk_kernel(const AttnArgs a, const AttnParts parts,
                      const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                      const int box_shift) {
  using S = ChunkSmem<D>;
  constexpr int kOps = S::kOps;
  constexpr bool kHalf = std::is_same<T, __half>::value;
  constexpr float kHot = kHalf ? 14.0f : 64.0f;  // as in the step kernel
  constexpr float kLift = kHalf ? kHalfLift : 0.0f;
  constexpr int kColO = 256;                     // TMEM: S (then P) twice, O twice
  extern __shared__ unsigned char smem_raw[];
  S& sm = *reinterpret_cast<S*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr AttnTiles tiles = {kChunkRows, kChunkKeys};
  unsigned flags = 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kOps; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    mbar_init(&sm.q_full, 32 * kChunkSoftmax);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], 256);
      mbar_init(&sm.o_full[i], 1);
    }
    for (int i = 0; i < kChunkItems; ++i) {
      mbar_init(&sm.item_full[i], 1);
      mbar_init(&sm.item_empty[i], 3);
      mbar_init(&sm.v_clean[i], 32);
    }
    mbar_init(&sm.drain, 1);
    sm.flags = 0;
    sm.slow = 0;
    sm.last = -1;
    sm.next = 0;
    fence_barrier_init();
  }
  if (warp == kChunkMma) tmem_alloc(&sm.tmem, 512);
  grid_dep_launch();
  grid_dep_wait();
  tc_fence_before();
  const bool small = a.rows.B <= 32;
  if (small)
    __syncthreads();
  else
    find_piece<kChunkThreads>(a, tiles, sm.scan, &sm.piece, flags);  // syncs the block
  tc_fence_after();
  const uint32_t tmem = sm.tmem;

  if (warp == kChunkLoad) {
    // ---- items, K and V tiles in the order K0 V0 K1 V1 .. ----
    const int shift = a.rows.page_shift, in_page = (1 << shift) - 1;
    const int box_rows = 1 << box_shift;
    Walk walk;
    walk.start(a, tiles, small ? find_piece_warp(a, tiles, flags) : sm.piece);
    PartRecord rec = {};
    rec.b = -1;
    int op = 0;
    bool alive = true;
    for (int n_item = 0; alive; ++n_item) {
      const int slot = n_item % kChunkItems;
      const Item it = walk.next(a, tiles);
      if (n_item >= kChunkItems)
        alive = mbar_wait_slow(&sm.slow, &sm.item_empty[slot],
                               (uint32_t)(n_item / kChunkItems - 1) & 1u);
      if (!__all_sync(0xffffffffu, alive)) {
        alive = false;
        break;
      }
      if (lane == 0) {
        sm.item[slot] = it;
        mbar_arrive(&sm.item_full[slot]);  // release: the descriptor is visible to the waiters
      }
      __syncwarp();
      if (it.part < 0) break;
      if (it.part == 1) rec.head = it.part_ends ? 1 : 2;
      if (it.part == 2) {
        rec.row0 = it.row0;
        rec.b = it.b; rec.h = it.h; rec.qt = it.qt;
        rec.n = it.n; rec.past = it.past; rec.n_rows = it.n_rows;
      }
      const int last_key = it.past + it.n;
      const int* table = a.rows.page_table + (size_t)it.b * a.rows.max_pages;
      auto page_of = [&](int t) {
        const int k = t * kChunkKeys + (lane << box_shift);
        return t < it.t1 && (lane << box_shift) < kChunkKeys && k < last_key
                   ? __ldg(table + (k >> shift))
                   : 0;
      };
      int page0 = page_of(it.t0), page1 = page_of(it.t0 + 1);
#pragma unroll 1
      for (int t = it.t0; t < it.t1; ++t) {
        const int k0 = t * kChunkKeys;
        const int boxes = min((last_key - k0 + box_rows - 1) >> box_shift, kChunkKeys >> box_shift);
        int pid = page0;
        if (lane < boxes && (unsigned)pid >= (unsigned)a.rows.n_pages) {
          flags |= DSPARK_FLAG_BAD_PAGE;
          pid = 0;
        }
        const int y_mine = ((pid * a.Hkv + it.h) << shift) + ((k0 + (lane << box_shift)) & in_page);
        page0 = page1;
        page1 = page_of(t + 2);
        int y[kChunkKeys / 16];
#pragma unroll
        for (int i = 0; i < kChunkKeys / 16; ++i) y[i] = __shfl_sync(0xffffffffu, y_mine, i);
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv, ++op) {
          const int stage = op % kOps;
          if (op >= kOps)
            alive = mbar_wait_slow(&sm.slow, &sm.empty[stage], (uint32_t)(op / kOps - 1) & 1u);
          if (!__all_sync(0xffffffffu, alive)) {
            alive = false;
            break;
          }
          if (elect_one()) {
            mbar_arrive_expect_tx(&sm.full[stage], (boxes << box_shift) * D * 2);
#pragma unroll
            for (int i = 0; i < kChunkKeys / 16; ++i) {
              if (i < boxes) {
#pragma unroll
                for (int hf = 0; hf < D / 64; ++hf)
                  tma_load_2d(sm.op[stage] + hf * kChunkKeys * 128 + (i << box_shift) * 128,
                              kv ? &mv : &mk, &sm.full[stage], hf * 64, y[i]);
              }
            }
          }
          __syncwarp();
          if (lane == 0) {
            sm.last = op;
            *(volatile int*)&sm.next = op + 1;
          }
        }
        if (!alive) break;
      }
    }
    if (!alive) flags |= DSPARK_FLAG_TIMEOUT;
    if (lane == 0) parts.rec[blockIdx.x] = rec;

  } else if (warp == kChunkClean) {
    // ---- what lies behind the sequence in its last page may be anything, and 0
    //      times an infinity is none: clear those rows of the last V tile ----
    bool alive = true;
    int op0 = 0;
    for (int n_item = 0;; ++n_item) {
      const int slot = n_item % kChunkItems;
      alive = mbar_wait_slow(&sm.slow, &sm.item_full[slot], (uint32_t)(n_item / kChunkItems) & 1u);
      if (!__all_sync(0xffffffffu, alive)) {
        alive = false;
        break;
      }
      const Item it = sm.item[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.item_empty[slot]);
      if (it.part < 0) break;
      if (has_tail(it)) {
        const int use = op0 + 2 * (it.t1 - it.t0) - 1, stage = use % kOps;
        // once it is issued, the parity can mean this fill only
        alive = wait_slow(&sm.slow, [&] { return next_past(&sm.next, use); }) &&
                mbar_wait_slow(&sm.slow, &sm.full[stage], (uint32_t)(use / kOps) & 1u);
        if (!__all_sync(0xffffffffu, alive)) {
          alive = false;
          break;
        }
        const int here = it.past + it.n - (it.t1 - 1) * kChunkKeys;
        for (int i = lane; i < (kChunkKeys - here) * (D / 8); i += 32) {
          const int k = here + i / (D / 8), c = i % (D / 8);
          *reinterpret_cast<uint4*>(sm.op[stage] + (c >> 3) * kChunkKeys * 128 + k * 128 +
                                    (c & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      // (can not be lapped: an item behind the next is published when the MMA
      // thread is past this one)
      mbar_arrive(&sm.v_clean[slot]);
      op0 += 2 * (it.t1 - it.t0);
    }
    if (!alive) flags |= DSPARK_FLAG_TIMEOUT;

  } else if (warp == kChunkMma) {
    // ---- MMA issue: one thread ----
    constexpr uint32_t kIdS = idesc_tc<T>(128, kChunkKeys, false, false);
    constexpr uint32_t kIdO = idesc_tc<T>(128, D, false, true);
    if (elect_one()) {
      bool alive = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (alive) alive = wait_slow(&sm.slow, [&] { return mbar_wait_spin(bar, parity); });
      };
      int op0 = 0, n_s[2] = {0, 0};  // operands and P tiles before the item
      for (int n_item = 0;; ++n_item) {
        const int slot = n_item % kChunkItems;
        wait(&sm.item_full[slot], (uint32_t)(n_item / kChunkItems) & 1u);
        if (!alive) break;
        const Item it = sm.item[slot];
        consumed(__int_as_float(it.part + it.t0 + it.t1 + it.n_rows));
        if (it.part < 0) break;
        const int n = it.t1 - it.t0;
        const int np[2] = {chunk_tiles(a, it, 0), chunk_tiles(a, it, 1)};
        auto issue_s = [&](int p, int stage) {
          const uint64_t kd = sdesc_sw128(smem_u32(sm.op[stage]));
          const uint64_t qd = sdesc_sw128(smem_u32(sm.q[p]));
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_bf16_ss(tmem + p * 128, qd + (((k >> 2) * 128 * 128 + (k & 3) * 32) >> 4),
                        kd + (((k >> 2) * kChunkKeys * 128 + (k & 3) * 32) >> 4), kIdS, k > 0);
          mma_commit(&sm.s_full[p]);
        };
        wait(&sm.q_full, (uint32_t)n_item & 1u);
        {
          const int stage = op0 % kOps;
          wait(&sm.full[stage], (uint32_t)(op0 / kOps) & 1u);
          if (!alive) break;
          tc_fence_after();
          if (np[0] > 0) issue_s(0, stage);
          if (np[1] > 0) issue_s(1, stage);
          mma_commit(&sm.empty[stage]);
        }
        for (int j = 0; j < n; ++j) {
          const int vo = op0 + 2 * j + 1, vs = vo % kOps, ko = vo + 1, ks = ko % kOps;
          wait(&sm.full[vs], (uint32_t)(vo / kOps) & 1u);
          if (j == n - 1) wait(&sm.v_clean[slot], (uint32_t)(n_item / kChunkItems) & 1u);
          if (j + 1 < n) wait(&sm.full[ks], (uint32_t)(ko / kOps) & 1u);
          const uint64_t vd = sdesc_mn<64>(smem_u32(sm.op[vs]), kChunkKeys);
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            if (j >= np[p]) continue;
            wait(&sm.p_full[p], (uint32_t)(n_s[p] + j) & 1u);
            if (!alive) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < kChunkKeys / 16; ++k)
              mma_bf16_ts(tmem + kColO + p * D, tmem + p * 128 + k * 8, vd + ((k * 2048) >> 4), kIdO,
                          j > 0 || k > 0);
            if (j + 1 < np[p])
              issue_s(p, ks);  // over P, behind the product that reads it
            else
              mma_commit(&sm.o_full[p]);
          }
          if (!alive) break;
          mma_commit(&sm.empty[vs]);
          if (j + 1 < n) mma_commit(&sm.empty[ks]);
        }
        if (!alive) break;
        mbar_arrive(&sm.item_empty[slot]);
        op0 += 2 * n;
        n_s[0] += np[0];
        n_s[1] += np[1];
      }
      if (!alive) flags |= DSPARK_FLAG_TIMEOUT;
      drain_mma(&sm.drain);
    }
    __syncwarp();

  } else {
    // ---- softmax: half of a row's keys a thread ----
    const int p = warp >> 3, half = warp >> 2 & 1, r = threadIdx.x & 127;
    constexpr int kMine = kChunkKeys / 2;  // keys of a thread
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_col = lane_base + p * 128 + half * kMine;
    const uint32_t p_col = lane_base + p * 128 + half * (kMine / 2);
    const uint32_t o_col = lane_base + kColO + p * D + half * (D / 2);
    const int bar = 2 + p * 4 + (warp & 3);  // of the two warps with the same rows
    bool alive = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (alive && !mbar_wait(bar, parity)) {
        alive = false;
        flags |= DSPARK_FLAG_TIMEOUT;
      }
    };
    int n_s = 0, n_o = 0;
    bool was_slow = false;  // attend_row at the item before
    const uint64_t kf2 = pair_of(a.scale2, a.scale2);
    for (int n_item = 0;; ++n_item) {
      const int slot = n_item % kChunkItems;
      // one warp waits and says so to the others: all of them stop together
      if (warp == 0) {
        const bool ok = mbar_wait(&sm.item_full[slot], (uint32_t)(n_item / kChunkItems) & 1u);
        if (!ok) flags |= DSPARK_FLAG_TIMEOUT;
        if (lane == 0) sm.stop = !ok || sm.item[slot].part < 0;
      }
      named_sync(1, 32 * kChunkSoftmax);
      if (sm.stop) break;
      const Item it = sm.item[slot];
      named_sync(1, 32 * kChunkSoftmax);
      if (threadIdx.x == 0) mbar_arrive(&sm.item_empty[slot]);
      // this row tile's Q (its products of the item before are done)
      const int row_base = it.qt * kChunkRows + p * 128;
      const int rows = min(it.n_rows - p * 128, 128);
      constexpr int kC = D / 8;
#pragma unroll 8
      for (int i = half * 128 + r; i < 128 * kC; i += 256) {
        const int x = i / kC, c = i % kC;
        const int rr = row_base + max(min(x, rows - 1), 0), tok = min(a.by_g.div(rr), it.n - 1);
        cp_async16(sm.q[p] + sw128_offset(x, 8 * c, 128),
                   static_cast<const T*>(a.q) + (it.row0 + tok) * a.q_stride +
                       (it.h * a.G + min(rr - tok * a.G, a.G - 1)) * D + 8 * c,
                   x < rows);
      }
      cp_async_wait_all();
      fence_proxy_async_smem();
      mbar_arrive(&sm.q_full);

      const int nt = chunk_tiles(a, it, p);
      const int rr = min(row_base + r, it.qt * kChunkRows + it.n_rows - 1);
      const int tok = a.by_g.div(rr);
      const int pos = it.past + tok, low = first_seen(pos, a.window);
      // of the row tile: what no mask touches
      const int pos_min = it.past + a.by_g.div(min(row_base, rr));
      const int low_max =
          first_seen(it.past + a.by_g.div(min(row_base + 127, it.qt * kChunkRows + it.n_rows - 1)),
                     a.window);
      float neg_m = 0.0f, l = 0.0f;

      for (int j = 0; j < nt; ++j, ++n_s) {
        const int k0 = (it.t0 + j) * kChunkKeys;
        const bool masked = k0 + kChunkKeys > pos_min + 1 || k0 < low_max;
        const bool first = j == 0 || k0 <= low_max;  // the first keys of some row
        // of this thread's keys the row sees [from, to]
        const int to = pos - k0 - half * kMine, from = low - k0 - half * kMine;
        wait(&sm.s_full[p], (uint32_t)n_s & 1u);
        tc_fence_after();
        auto mask = [&](float (&x)[32], int c) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (c + i > to || c + i < from) x[i] = -CUDART_INF_F;
        };
        uint32_t w[kMine / 2];
        bool raise = kHalf && first;
        float sum;
        while (true) {
          if (raise) {
            // move the reference to the tile's maximum
            float top = -CUDART_INF_F;
#pragma unroll 1
            for (int c = 0; c < kMine; c += 32) {
              float x[32];
              tmem_ld32(s_col + c, x);
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] *= a.scale2;
              if (masked) mask(x, c);
#pragma unroll
              for (int i = 0; i < 32; i += 2) top = max3(top, x[i], x[i + 1]);
            }
            sm.part[p][half][r] = top;
            named_sync(bar, 64);
            top = fmaxf(top, sm.part[p][half ^ 1][r]);
            const float old = -neg_m;
            const bool seen = j > 0 && k0 > low;  // has keys before this tile
            const float to = top - kLift;
            const float now = seen ? fmaxf(old, to) : top == -CUDART_INF_F ? old : to;
            const float f = seen && now != old ? ex2(old - now) : 1.0f;
            neg_m = -now;
            l *= f;
            if (j > 0) {  // (the products up to tile j - 1 are done: S came behind them)
#pragma unroll 1
              for (int c = 0; c < D / 2; c += 16) {
                uint32_t o[16];
                tmem_ld<16>(o_col + c, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tmem_st<16>(o_col + c, o);
              }
              tmem_st_wait();
            }
          }
          // weights, as if no score were outside the range
          const uint64_t m2 = pair_of(neg_m, neg_m);
          float top = -CUDART_INF_F, bottom = CUDART_INF_F;
          uint64_t s2 = pair_of(0.0f, 0.0f), t2 = s2;
#pragma unroll
          for (int c = 0; c < kMine; c += 32) {
            uint32_t raw[32];
            tmem_ld32_issue(s_col + c, raw);
            tmem_ld32_wait(raw);
            float x[32];
#pragma unroll
            for (int i = 0; i < 32; i += 2)
              pair_to(fma2(pair_of(__uint_as_float(raw[i]), __uint_as_float(raw[i + 1])), kf2, m2),
                      x[i], x[i + 1]);
            if (masked) mask(x, c);
#pragma unroll
            for (int i = 0; i < 32; i += 2) top = max3(top, x[i], x[i + 1]);
            if (!kHalf && first) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                bottom = fminf(bottom, x[i] == -CUDART_INF_F ? CUDART_INF_F : x[i]);
            }
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float p0 = ex2(x[i]), p1 = ex2(x[i + 1]), p2 = ex2(x[i + 2]), p3 = ex2(x[i + 3]);
              s2 = add2(s2, pair_of(p0, p1));
              t2 = add2(t2, pair_of(p2, p3));
              w[(c + i) / 2] = Pair<T>::put(p0, p1);
              w[(c + i) / 2 + 1] = Pair<T>::put(p2, p3);
            }
          }
          float s0, s1;
          pair_to(add2(s2, t2), s0, s1);
          sum = s0 + s1;
          // (both warps have read their scores when either goes on)
          const bool hot = vote_any(bar, 64, top > kHot || bottom < -kHot);
          if (raise || !hot) break;
          raise = true;
        }
        l += sum;
        tmem_st32(p_col, w);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&sm.p_full[p]);
      }
      if (was_slow) count_slow(&sm.slow, -1);
      was_slow = false;

      // ---- the item's rows ----
      if (nt > 0) {
        wait(&sm.o_full[p], (uint32_t)n_o & 1u);
        ++n_o;
        tc_fence_after();
      }
      const bool whole = it.part == 0;
      sm.part[p][half][r] = l;
      named_sync(bar, 64);
      l = sm.part[p][0][r] + sm.part[p][1][r];
      const float inv = 1.0f / l;
      float worst = 0.0f;
      const size_t slot_row =
          (size_t)(2 * blockIdx.x + (it.part == 2)) * kChunkRows + p * 128 + r;
      T* out = static_cast<T*>(a.out) +
               ((it.row0 + tok) * a.Hq + it.h * a.G + rr - tok * a.G) * D + half * (D / 2);
#pragma unroll 1
      for (int c = 0; c < D / 2; c += 32) {
        float o[32];
        if (nt > 0) {
          tmem_ld32(o_col + c, o);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.0f;
        }
        if (whole) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            o[i] *= inv;
            worst = fmaf(o[i], 0.0f, worst);  // not a number if one is not finite
          }
          if (r < rows) {
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              *reinterpret_cast<uint4*>(out + c + i) =
                  make_uint4(Pair<T>::put(o[i], o[i + 1]), Pair<T>::put(o[i + 2], o[i + 3]),
                             Pair<T>::put(o[i + 4], o[i + 5]), Pair<T>::put(o[i + 6], o[i + 7]));
          }
        } else if (r < rows) {
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<float4*>(parts.o + slot_row * D + half * (D / 2) + c + i) =
                make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
        }
      }
      // a part without a visible key has no reference
      if (!whole && r < rows && half == 0)
        parts.ml[slot_row] = make_float2(l == 0.0f ? -CUDART_INF_F : -neg_m, l);
      tc_fence_before();
      // a result that is not finite may come from a position that its row does
      // not see (0 times infinity): form the row again from those it sees
      // (the row's two warps take such rows in turn; both halves are stored by then)
      sm.odd[p][half][r] = worst;
      named_sync(bar, 64);
      unsigned bad = __ballot_sync(
          0xffffffffu, whole && r < rows && (worst != 0.0f || sm.odd[p][half ^ 1][r] != 0.0f));
      if (bad) {
        count_slow(&sm.slow, 1);
        was_slow = true;
        for (int i = 0; bad; bad &= bad - 1, ++i) {
          const int src = __ffs(bad) - 1;
          const int rb = __shfl_sync(0xffffffffu, rr, src), tb = a.by_g.div(rb);
          if ((i & 1) == half)
            attend_row<T, T, D>(a, it.b, it.past + tb, it.h * a.G + rb - tb * a.G, it.row0 + tb,
                                flags);
        }
      }
    }
  }
  if (flags) atomicOr(&sm.flags, flags);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // after an abort copies may still be in flight: none outlives the CTA
  if (sm.flags & DSPARK_FLAG_TIMEOUT) {
    if (threadIdx.x == 0)
      for (int u = max(sm.last - kOps + 1, 0); u <= sm.last; ++u)
        mbar_wait(&sm.full[u % kOps], (uint32_t)(u / kOps) & 1u);
    __syncthreads();
  }
  if (warp == kChunkMma) tmem_dealloc(tmem, 512);
  if (threadIdx.x == 0) store_status(a.status, sm.flags);
}

}  // namespace dspark
