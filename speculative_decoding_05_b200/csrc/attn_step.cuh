// attn_step.cuh -- attention of a decode or verify step on the tensor cores:
// up to 128 (token, query head) rows an item.
//
// The cache's bytes bound such a call as long as the work on a key stays
// short.  The warp-level matrix instructions do not keep up: 32 padded rows
// measured 205 multiply-adds a clock and SM, twice the time of the stream
// itself.  tcgen05 does, with the keys as the M dimension, so that its 128
// lanes are full however few rows there are:
//   S^T [128 keys, N rows] = K Q^T      both K-major as they lie in memory
//   O^T [D, N rows]      += V^T P^T     V as it lies (its MN-major form), P^T
//                                       [128 keys][N rows] written by the threads
// A thread owns one key and N / 2 rows of S^T (two warpgroups share the rows).
// The softmax reference of a row then lives across threads, so it is not the
// running maximum but any earlier maximum (of the item's first tile, as a
// rule): weights may exceed 1, which costs no precision in floating point, and
// one vote a tile finds the rare score that is too far above it (kHot), when
// the reference is raised and sums and O^T are rescaled.
//
// Warps: 8 softmax, one each that loads K (and walks the piece), V and Q, one
// that issues the MMAs, and with an e4m3 cache 4 that widen its tiles from the
// TMA ring into the operand ring.  The
// operands pass in the order K0 K1 K2 V0 K3 V1 ..: scores are formed two tiles
// ahead, as far as their two buffers reach.
#pragma once

#include <type_traits>

#include "attn_plan.cuh"
#include "attn_tc.cuh"

namespace dspark {

constexpr int kStepKeys = 128;
constexpr int kStepSoftmax = 8;                    // warps
constexpr int kStepLoadK = kStepSoftmax;           // warp
constexpr int kStepLoadV = kStepSoftmax + 1;       // warp
constexpr int kStepLoadQ = kStepSoftmax + 2;       // warp
constexpr int kStepMma = kStepSoftmax + 3;         // warp
constexpr int kStepWiden = kStepSoftmax + 4;       // first of 4 warps, e4m3 only
constexpr int kStepItems = 4;
constexpr int kStepScales = 4;
constexpr int kSmemLimit = 232448;                 // 227 KB a CTA

template <typename TC>
__host__ __device__ constexpr int step_threads() {
  return 32 * (kStepSoftmax + 4 + (sizeof(TC) == 1 ? 4 : 0));
}

template <typename TC, int D, int N>
struct StepCfg {
  static constexpr bool kQ8 = sizeof(TC) == 1;
  static constexpr int kOpBytes = kStepKeys * D * 2;
  static constexpr int kRawBytes = kQ8 ? kStepKeys * D : 0;
  static constexpr int kQBufs = N <= 64 ? 2 : 1;
  static constexpr int kQBytes = N * D * 2;
  static constexpr int kPBytes = kStepKeys * N * 2;
  static constexpr int kSmall = 10240;
  // 16 KB behind the operands, see StepSmem
  static constexpr int kPQ = kQBufs * kQBytes + 2 * kPBytes;
  static constexpr int kBehind = kPQ < 16384 ? 16384 - kPQ : 16;
  static constexpr int kLeft = kSmemLimit - 1024 - kSmall - kPQ - kBehind;
  static constexpr int kOps = kQ8 ? (kLeft >= 3 * kOpBytes + 3 * kRawBytes ? 3 : 2)
                                  : (kLeft / kOpBytes < 8 ? kLeft / kOpBytes : 8);
  static constexpr int kRawFit = kQ8 ? (kLeft - kOps * kOpBytes) / kRawBytes : 1;
  static constexpr int kRaws = kRawFit < 8 ? kRawFit : 8;
  static constexpr int kRing = kQ8 ? kRaws : kOps;  // the ring that TMA fills
  static_assert(kOps >= 2 && kRaws >= 1, "shared memory");
};

template <typename TC, int D, int N>
struct StepSmem {
  using C = StepCfg<TC, D, N>;
  alignas(1024) unsigned char op[C::kOps][C::kOpBytes];
  // with D = 64 the MMAs of V read 16 KB past a tile (see the MMA warp): p, q
  // and `behind` are as much
  alignas(1024) unsigned char p[2][C::kPBytes];
  alignas(1024) unsigned char q[C::kQBufs][C::kQBytes];
  unsigned char behind[C::kBehind];
  alignas(1024) unsigned char raw[C::kQ8 ? C::kRaws : 1][C::kQ8 ? C::kRawBytes : 16];
  float scale[C::kQ8 ? kStepScales : 1][2][kStepKeys];
  float m[N], f[N], part[4][N];
  int pos[N], low[N], bad[N];
  long long out[N];
  uint64_t op_full[C::kOps], op_empty[C::kOps];
  uint64_t raw_full[C::kRaws], raw_empty[C::kRaws];
  uint64_t scale_full[kStepScales], scale_empty[kStepScales];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_full[2], p_empty[2];
  uint64_t item_full[kStepItems], item_empty[kStepItems];
  uint64_t drain;
  Item item[kStepItems];
  Piece piece;
  long long scan[16];
  uint32_t tmem;
  unsigned flags;
  int stop;
  int next_k, next_v;  // operand that the K and the V warp issue next, at least
  int last_k, last_v, last_tile;
};

// Place of tile j's K and V in the operand order K0 K1 K2 V0 K3 V1 .. of an item
// of n tiles, which ends V(n - 2) V(n - 1) (or K0 V0, or K0 K1 V0 V1).
__device__ __forceinline__ int op_of_k(int j) { return j < 2 ? j : 2 * j - 2; }
__device__ __forceinline__ int op_of_v(int j, int n) {
  return j + min(j + 3, n);
}
// Whether operand s is a K.
__device__ __forceinline__ bool op_is_k(int s, int n) {
  return s < 2 ? s < n : !(s & 1) && s / 2 + 1 < n;
}

// Bounded wait until another warp has issued every operand up to `op`.
__device__ __forceinline__ bool next_past(const volatile int* next, int op) {
  if (*next > op) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t i = 1;; ++i) {
    if (*next > op) return true;
    if ((i & 255u) == 0 && wait_expired(t0, i)) return false;
  }
}

template <typename T, typename TC, int D, int N>
__global__ void __launch_bounds__(step_threads<TC>(), 1)
    attn_step_kernel(const AttnArgs a, const AttnParts parts, const __grid_constant__ CUtensorMap mk,
                     const __grid_constant__ CUtensorMap mv, const int box_shift) {
  using C = StepCfg<TC, D, N>;
  using S = StepSmem<TC, D, N>;
  using TP = typename std::conditional<C::kQ8, __nv_bfloat16, T>::type;  // P and V
  constexpr bool kQ8 = C::kQ8;
  constexpr int kThreads = step_threads<TC>();
  constexpr int kTmemCols = 4 * N;  // S^T twice, O^T, rounded up to a power of two >= 32
  // A score so far above the reference raises it: 2^64 leaves fp32 sums and
  // bf16 weights far from their ends, 2^14 fp16 ones.
  constexpr float kHot = std::is_same<TP, __half>::value ? 14.0f : 64.0f;
  extern __shared__ unsigned char smem_raw[];
  S& sm = *reinterpret_cast<S*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const AttnTiles tiles = {N, kStepKeys};
  unsigned flags = 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kOps; ++i) {
      mbar_init(&sm.op_full[i], kQ8 ? 4 : 1);
      mbar_init(&sm.op_empty[i], 1);
    }
    for (int i = 0; i < C::kRaws; ++i) {
      mbar_init(&sm.raw_full[i], 1);
      mbar_init(&sm.raw_empty[i], 4);
    }
    for (int i = 0; i < kStepScales; ++i) {
      mbar_init(&sm.scale_full[i], 1);
      mbar_init(&sm.scale_empty[i], kStepSoftmax);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], 32);
      mbar_init(&sm.q_empty[i], 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], 32 * kStepSoftmax);
      mbar_init(&sm.p_empty[i], 1);
    }
    for (int i = 0; i < kStepItems; ++i) {
      mbar_init(&sm.item_full[i], 1);
      mbar_init(&sm.item_empty[i], kQ8 ? 5 : 4);
    }
    mbar_init(&sm.drain, 1);
    sm.flags = 0;
    sm.last_k = sm.last_v = sm.last_tile = -1;
    sm.next_k = sm.next_v = 0;
    fence_barrier_init();
  }
  if (warp == kStepMma) tmem_alloc(&sm.tmem, kTmemCols);
  grid_dep_launch();
  grid_dep_wait();
  tc_fence_before();
  find_piece<kThreads>(a, tiles, sm.scan, &sm.piece, flags);  // syncs the block
  tc_fence_after();
  const uint32_t tmem = sm.tmem;

  if (warp == kStepLoadK || warp == kStepLoadV) {
    // ---- loads: items and K tiles (and scales); V tiles ----
    uint64_t* full = kQ8 ? sm.raw_full : sm.op_full;
    uint64_t* empty = kQ8 ? sm.raw_empty : sm.op_empty;
    const int shift = a.rows.page_shift, in_page = (1 << shift) - 1;
    const int box_rows = 1 << box_shift;
    const bool is_k = warp == kStepLoadK;
    volatile int* my_next = is_k ? &sm.next_k : &sm.next_v;
    const volatile int* other_next = is_k ? &sm.next_v : &sm.next_k;
    Walk walk;
    if (is_k) walk.start(a, tiles, sm.piece);
    PartRecord rec = {};
    rec.b = -1;
    int op0 = 0, tile0 = 0;
    bool alive = true;
    for (int n_item = 0; alive; ++n_item) {
      const int slot = n_item % kStepItems;
      Item it;
      if (is_k) {
        it = walk.next(a, tiles);
        if (n_item >= kStepItems)
          alive = mbar_wait(&sm.item_empty[slot], (uint32_t)(n_item / kStepItems - 1) & 1u);
        if (!__all_sync(0xffffffffu, alive)) break;
        if (lane == 0) {
          sm.item[slot] = it;
          mbar_arrive(&sm.item_full[slot]);  // release: the descriptor is visible to the waiters
        }
        __syncwarp();
        if (it.part == 1) rec.head = it.part_ends ? 1 : 2;
        if (it.part == 2) {
          rec.row0 = it.row0;
          rec.b = it.b; rec.h = it.h; rec.qt = it.qt;
          rec.n = it.n; rec.past = it.past; rec.n_rows = it.n_rows;
        }
      } else {
        alive = mbar_wait(&sm.item_full[slot], (uint32_t)(n_item / kStepItems) & 1u);
        if (!__all_sync(0xffffffffu, alive)) break;
        it = sm.item[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.item_empty[slot]);
      }
      if (it.part < 0) break;
      const int last_key = it.past + it.n;
      const int n = it.t1 - it.t0;
      // page of this lane's box in tile j, read two tiles ahead
      const int* table = a.rows.page_table + (size_t)it.b * a.rows.max_pages;
      auto page_of = [&](int j) {
        const int k = (it.t0 + j) * kStepKeys + (lane << box_shift);
        return j < n && (lane << box_shift) < kStepKeys && k < last_key ? __ldg(table + (k >> shift))
                                                                        : 0;
      };
      int page0 = page_of(0), page1 = page_of(1);

#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        const int k0 = (it.t0 + j) * kStepKeys;
        const int boxes = min((last_key - k0 + box_rows - 1) >> box_shift, kStepKeys >> box_shift);
        int pid = page0;
        if (lane < boxes && (unsigned)pid >= (unsigned)a.rows.n_pages) {
          flags |= DSPARK_FLAG_BAD_PAGE;
          pid = 0;
        }
        const int y_mine = ((pid * a.Hkv + it.h) << shift) + ((k0 + (lane << box_shift)) & in_page);
        page0 = page1;
        page1 = page_of(j + 2);
        int y[kStepKeys / 16];
#pragma unroll
        for (int i = 0; i < kStepKeys / 16; ++i) y[i] = __shfl_sync(0xffffffffu, y_mine, i);
        const int op = op0 + (is_k ? op_of_k(j) : op_of_v(j, n));
        const int stage = op % C::kRing;
        // The wait for the stage's release tells phases apart by parity only.
        // Its last use may be the other warp's: once that is filled the use
        // before it has been released, and the parity can mean one phase.
        if (lane == 0) *my_next = op;
        if (op >= C::kRing) {
          if (!next_past(other_next, op - C::kRing)) alive = false;
          if (alive) alive = mbar_wait(&empty[stage], (uint32_t)(op / C::kRing - 1) & 1u);
        }
        const int sc = (tile0 + j) % kStepScales;
        if (alive && kQ8 && is_k && tile0 + j >= kStepScales)
          alive = mbar_wait(&sm.scale_empty[sc], (uint32_t)((tile0 + j) / kStepScales - 1) & 1u);
        if (!__all_sync(0xffffffffu, alive)) {
          alive = false;
          break;
        }
        if (elect_one()) {
          mbar_arrive_expect_tx(&full[stage], (boxes << box_shift) * D * (int)sizeof(TC));
          if (kQ8 && is_k) mbar_arrive_expect_tx(&sm.scale_full[sc], (boxes << box_shift) * 8);
          unsigned char* dst = kQ8 ? sm.raw[stage] : sm.op[stage];
          const CUtensorMap* map = is_k ? &mk : &mv;
          constexpr int kWidth = kQ8 && D == 64 ? 64 : 128;
          constexpr int kHalves = kQ8 ? 1 : D / 64;
#pragma unroll
          for (int i = 0; i < kStepKeys / 16; ++i) {
            if (i < boxes) {
#pragma unroll
              for (int hf = 0; hf < kHalves; ++hf)
                tma_load_2d(dst + hf * kStepKeys * 128 + (i << box_shift) * kWidth, map,
                            &full[stage], hf * 64, y[i]);
              if (kQ8 && is_k) {
                const uint64_t pol = policy_evict_first();
                bulk_load(&sm.scale[sc][0][i << box_shift], a.k_scale + y[i], box_rows * 4,
                          &sm.scale_full[sc], pol);
                bulk_load(&sm.scale[sc][1][i << box_shift], a.v_scale + y[i], box_rows * 4,
                          &sm.scale_full[sc], pol);
              }
            }
          }
        }
        __syncwarp();
        if (is_k) sm.last_k = op;  // for the drain: the operands loaded last
        else sm.last_v = op;
        if (is_k) sm.last_tile = tile0 + j;
      }
      op0 += 2 * n;
      tile0 += n;
      if (lane == 0) *my_next = op0;  // or a later one: the next item says
    }
    if (!alive) flags |= DSPARK_FLAG_TIMEOUT;
    if (lane == 0 && is_k) parts.rec[blockIdx.x] = rec;

  } else if (warp == kStepLoadQ) {
    // ---- loads: Q rows, K-major, 128-byte swizzle; rows behind the last are zero ----
    bool alive = true;
    for (int n_item = 0;; ++n_item) {
      const int slot = n_item % kStepItems, qb = n_item % C::kQBufs;
      alive = mbar_wait(&sm.item_full[slot], (uint32_t)(n_item / kStepItems) & 1u);
      if (!__all_sync(0xffffffffu, alive)) break;
      const Item it = sm.item[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.item_empty[slot]);
      if (it.part < 0) break;
      if (n_item >= C::kQBufs)
        alive = mbar_wait(&sm.q_empty[qb], (uint32_t)(n_item / C::kQBufs - 1) & 1u);
      if (!__all_sync(0xffffffffu, alive)) break;
      constexpr int kChunks = D / 8, kBatch = 8;
#pragma unroll 1
      for (int i0 = lane; i0 < N * kChunks; i0 += 32 * kBatch) {
        uint4 v[kBatch];
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
          const int i = i0 + 32 * x, r = i / kChunks, c = i % kChunks;
          v[x] = make_uint4(0, 0, 0, 0);
          if (r < it.n_rows) {
            const int rr = it.qt * N + r, tok = a.by_g.div(rr);
            v[x] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) +
                                                   (it.row0 + tok) * a.q_stride +
                                                   (it.h * a.G + rr - tok * a.G) * D + 8 * c);
          }
        }
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
          const int i = i0 + 32 * x, r = i / kChunks, c = i % kChunks;
          if (r < N) *reinterpret_cast<uint4*>(sm.q[qb] + sw128_offset(r, 8 * c, N)) = v[x];
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&sm.q_full[qb]);
    }
    if (!alive) flags |= DSPARK_FLAG_TIMEOUT;

  } else if (warp == kStepMma) {
    // ---- MMA issue ----
    constexpr uint32_t kIdS = idesc_tc<T>(128, N, false, false);
    constexpr uint32_t kIdO = idesc_tc<TP>(128, N, true, true);
    bool alive = true;
    int op0 = 0, tile0 = 0;
    for (int n_item = 0;; ++n_item) {
      const int slot = n_item % kStepItems;
      if (alive) alive = mbar_wait(&sm.item_full[slot], (uint32_t)(n_item / kStepItems) & 1u);
      alive = __all_sync(0xffffffffu, alive);
      if (!alive) break;
      const int part = sm.item[slot].part, n = sm.item[slot].t1 - sm.item[slot].t0;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.item_empty[slot]);
      if (part < 0) break;
      const int qb = n_item % C::kQBufs;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (alive) alive = mbar_wait_spin(bar, parity);
        alive = __all_sync(0xffffffffu, alive);
      };
      auto issue_s = [&](int j) {
        const int op = op0 + op_of_k(j), os = op % C::kOps, buf = (tile0 + j) & 1;
        wait(&sm.op_full[os], (uint32_t)(op / C::kOps) & 1u);
        tc_fence_after();
        const uint64_t kd = sdesc_sw128(smem_u32(sm.op[os])), qd = sdesc_sw128(smem_u32(sm.q[qb]));
        if (alive && elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_bf16_ss(tmem + buf * N, kd + (((k >> 2) * kStepKeys * 128 + (k & 3) * 32) >> 4),
                        qd + (((k >> 2) * N * 128 + (k & 3) * 32) >> 4), kIdS, k > 0);
          mma_commit(&sm.op_empty[os]);
          mma_commit(&sm.s_full[buf]);
          if (j == n - 1) mma_commit(&sm.q_empty[qb]);
        }
        __syncwarp();
      };
      wait(&sm.q_full[qb], (uint32_t)(n_item / C::kQBufs) & 1u);
      issue_s(0);
      if (n > 1) issue_s(1);
      for (int j = 0; j < n; ++j) {
        const int g = tile0 + j, buf = g & 1;
        wait(&sm.p_full[buf], (uint32_t)(g >> 1) & 1u);
        // the scores of tile j were read: their buffer takes those of j + 2
        if (j + 2 < n) issue_s(j + 2);
        const int op = op0 + op_of_v(j, n), os = op % C::kOps;
        wait(&sm.op_full[os], (uint32_t)(op / C::kOps) & 1u);
        tc_fence_after();
        // V: 64 elements of D in a row, 8 keys 1024 bytes apart, the other 64
        // behind all keys.  With D = 64 there are no others: lanes 64-127 of
        // O^T take what lies there and nobody reads them.
        constexpr int kW = N < 64 ? N : 64;  // rows of P^T in a row of shared memory
        const uint64_t vd = sdesc_mn<64>(smem_u32(sm.op[os]), kStepKeys);
        const uint64_t pd = sdesc_mn<kW>(smem_u32(sm.p[buf]), kStepKeys);
        if (alive && elect_one()) {
#pragma unroll
          for (int k = 0; k < kStepKeys / 16; ++k)
            mma_bf16_ss(tmem + 2 * N, vd + ((k * 2048) >> 4), pd + ((k * 16 * kW * 2) >> 4), kIdO,
                        j > 0 || k > 0);
          mma_commit(&sm.op_empty[os]);
          mma_commit(&sm.p_empty[buf]);
        }
        __syncwarp();
      }
      op0 += 2 * n;
      tile0 += n;
    }
    if (!alive) flags |= DSPARK_FLAG_TIMEOUT;
    // every commit above was the elected lane's: so is the last one
    if (elect_one()) drain_mma(&sm.drain);
    __syncwarp();

  } else if (warp >= kStepWiden) {
    // ---- e4m3 tiles to 16 bits, in the operands' order ----
    if constexpr (kQ8) {
      const int tid = threadIdx.x - 32 * kStepWiden;
      bool alive = true;
      int op = 0;
      for (int n_item = 0;; ++n_item) {
        const int slot = n_item % kStepItems;
        if (alive) alive = mbar_wait(&sm.item_full[slot], (uint32_t)(n_item / kStepItems) & 1u);
        const int part = sm.item[slot].part, n = sm.item[slot].t1 - sm.item[slot].t0;
        // all four warps go on or all stop
        if (vote_any(4, 128, !alive)) {
          alive = false;
          break;
        }
        if (tid == 0) mbar_arrive(&sm.item_empty[slot]);
        if (part < 0) break;
        for (int s = 0; s < 2 * n && alive; ++s, ++op) {
          const bool is_k = op_is_k(s, n);
          const int rs = op % C::kRaws, os = op % C::kOps;
          alive = mbar_wait(&sm.raw_full[rs], (uint32_t)(op / C::kRaws) & 1u);
          if (alive && op >= C::kOps)
            alive = mbar_wait(&sm.op_empty[os], (uint32_t)(op / C::kOps - 1) & 1u);
          if (!alive) break;
          if (is_k)
            widen_tile<T, D>(sm.raw[rs], sm.op[os], tid);
          else
            widen_tile<__nv_bfloat16, D>(sm.raw[rs], sm.op[os], tid);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sm.raw_empty[rs]);
            mbar_arrive(&sm.op_full[os]);
          }
        }
      }
      if (!alive) flags |= DSPARK_FLAG_TIMEOUT;
    }

  } else {
    // ---- softmax: one key a thread, half of the rows a warpgroup ----
    constexpr int R = N / 2;                  // rows of a thread
    constexpr int kChunk32 = R < 32 ? R : 32; // columns of a load
    constexpr int kLoads = R / kChunk32;
    const int wg = warp >> 2, quarter = warp & 3;
    const int key = quarter * 32 + lane;      // in the tile; in the epilogue: element of D
    const int n0 = wg * R;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const int bar_wg = 2 + wg;
    bool alive = true;
    int tile = 0, op0 = 0;
    for (int n_item = 0;; ++n_item) {
      const int slot = n_item % kStepItems;
      // one warp waits and says so to the others: all of them stop together
      if (warp == 0) {
        const bool ok = mbar_wait(&sm.item_full[slot], (uint32_t)(n_item / kStepItems) & 1u);
        if (!ok) flags |= DSPARK_FLAG_TIMEOUT;
        if (lane == 0) sm.stop = !ok || sm.item[slot].part < 0;
      }
      named_sync(1, 32 * kStepSoftmax);
      if (sm.stop) break;
      const Item it = sm.item[slot];
      if (threadIdx.x < N) {
        const int n = threadIdx.x;
        const int rr = it.qt * N + min(n, it.n_rows - 1), tok = a.by_g.div(rr);
        const int p = it.past + tok;
        sm.pos[n] = p;
        sm.low[n] = first_seen(p, a.window);
        sm.out[n] = ((it.row0 + tok) * a.Hq + it.h * a.G + rr - tok * a.G) * (long long)D;
        sm.m[n] = n < it.n_rows ? -CUDART_INF_F : 0.0f;  // rows that pad: scores 0
        sm.bad[n] = 0;
      }
      named_sync(1, 32 * kStepSoftmax);
      if (threadIdx.x == 0) mbar_arrive(&sm.item_empty[slot]);
      const int nt = it.t1 - it.t0;
      const int pos_min = it.past + a.by_g.div(it.qt * N);
      const int pos_max = it.past + a.by_g.div(it.qt * N + it.n_rows - 1);
      float l[R];
#pragma unroll
      for (int i = 0; i < R; ++i) l[i] = 0.0f;

      for (int j = 0; j < nt; ++j, ++tile) {
        const int buf = tile & 1;
        const int k0 = (it.t0 + j) * kStepKeys;
        const int at = k0 + key;
        const bool masked = k0 + kStepKeys > pos_min + 1 ||
                            (a.window > 0 && k0 < pos_max - a.window + 1);
        float kf = a.scale2, vs = 1.0f;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
          if (alive && !mbar_wait_spin(bar, parity)) {
            alive = false;
            flags |= DSPARK_FLAG_TIMEOUT;
          }
        };
        if constexpr (kQ8) {
          const int sc = tile % kStepScales;
          wait(&sm.scale_full[sc], (uint32_t)(tile / kStepScales) & 1u);
          kf *= sm.scale[sc][0][key];
          vs = sm.scale[sc][1][key];
          consumed(kf + vs);
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.scale_empty[sc]);
        }
        wait(&sm.s_full[buf], (uint32_t)(tile >> 1) & 1u);
        tc_fence_after();
        const uint32_t s_col = tmem + lane_base + buf * N + n0;

        // scores over the reference, in units of log 2
        float x[kChunk32];
        auto load = [&](int c, bool over) {
          uint32_t raw[kChunk32];
          tmem_ld<kChunk32>(s_col + c * kChunk32, raw);
#pragma unroll
          for (int i = 0; i < kChunk32; i += 4) {
            const int n = n0 + c * kChunk32 + i;
            float4 m4 = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (over) m4 = *reinterpret_cast<const float4*>(&sm.m[n]);
            x[i] = fmaf(__uint_as_float(raw[i]), kf, -m4.x);
            x[i + 1] = fmaf(__uint_as_float(raw[i + 1]), kf, -m4.y);
            x[i + 2] = fmaf(__uint_as_float(raw[i + 2]), kf, -m4.z);
            x[i + 3] = fmaf(__uint_as_float(raw[i + 3]), kf, -m4.w);
            if (masked) {
              const int4 p4 = *reinterpret_cast<const int4*>(&sm.pos[n]);
              const int4 l4 = *reinterpret_cast<const int4*>(&sm.low[n]);
              if (at > p4.x || at < l4.x) x[i] = -CUDART_INF_F;
              if (at > p4.y || at < l4.y) x[i + 1] = -CUDART_INF_F;
              if (at > p4.z || at < l4.z) x[i + 2] = -CUDART_INF_F;
              if (at > p4.w || at < l4.w) x[i + 3] = -CUDART_INF_F;
            }
          }
        };
        float top = -CUDART_INF_F;
#pragma unroll
        for (int c = 0; c < kLoads; ++c) {
          load(c, true);
#pragma unroll
          for (int i = 0; i < kChunk32; ++i) top = fmaxf(top, x[i]);
        }
        if (vote_any(bar_wg, 128, top > kHot)) {
          // raise the references of this warpgroup's rows to the tile's maxima
#pragma unroll
          for (int c = 0; c < kLoads; ++c) {
            load(c, false);
#pragma unroll
            for (int i = 0; i < kChunk32; ++i) {
              const float w = warp_max_redux(x[i]);
              if (lane == 0) sm.part[quarter][n0 + c * kChunk32 + i] = w;
            }
          }
          named_sync(bar_wg, 128);
          if (key < R) {
            const int n = n0 + key;
            const float old = sm.m[n];
            float now = fmaxf(fmaxf(sm.part[0][n], sm.part[1][n]),
                              fmaxf(sm.part[2][n], sm.part[3][n]));
            if (n >= it.n_rows) now = 0.0f;
            now = fmaxf(now, old);
            sm.f[n] = old == now || old == -CUDART_INF_F ? (old == now ? 1.0f : 0.0f) : ex2(old - now);
            sm.m[n] = now;
          }
          named_sync(bar_wg, 128);
          if (j > 0) {
            wait(&sm.p_empty[buf ^ 1], (uint32_t)((tile - 1) >> 1) & 1u);  // O^T of tile j - 1
            tc_fence_after();
          }
#pragma unroll
          for (int c = 0; c < kLoads; ++c) {
            uint32_t o[kChunk32];
            const uint32_t col = tmem + lane_base + 2 * N + n0 + c * kChunk32;
            if (j > 0) tmem_ld<kChunk32>(col, o);
#pragma unroll
            for (int i = 0; i < kChunk32; ++i) {
              const float f = sm.f[n0 + c * kChunk32 + i];
              l[c * kChunk32 + i] *= f;
              if (j > 0) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            }
            if (j > 0) tmem_st<kChunk32>(col, o);
          }
          if (j > 0) tmem_st_wait();
          if (kLoads == 1) load(0, true);
        }
        // weights; the buffer was last read by the MMAs of tile - 2
        if (tile >= 2) wait(&sm.p_empty[buf], (uint32_t)((tile >> 1) - 1) & 1u);
        unsigned char* prow = sm.p[buf];
#pragma unroll
        for (int c = 0; c < kLoads; ++c) {
          if (kLoads > 1) load(c, true);
#pragma unroll
          for (int i = 0; i < kChunk32; i += 8) {
            uint32_t w[4];
#pragma unroll
            for (int y = 0; y < 8; y += 2) {
              float p0 = ex2(x[i + y]), p1 = ex2(x[i + y + 1]);
              l[c * kChunk32 + i + y] += p0;
              l[c * kChunk32 + i + y + 1] += p1;
              if constexpr (kQ8) {  // a masked position's scale may be anything
                p0 = x[i + y] == -CUDART_INF_F ? 0.0f : p0 * vs;
                p1 = x[i + y + 1] == -CUDART_INF_F ? 0.0f : p1 * vs;
              }
              w[y / 2] = Pair<TP>::put(p0, p1);
            }
            *reinterpret_cast<uint4*>(prow + mn_offset<(N < 64 ? N : 64)>(
                                                 n0 + c * kChunk32 + i, key, kStepKeys)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        if (!kQ8 && wg == 0 && it.past + it.n - k0 < kStepKeys) {
          // what lies behind the sequence in its last page may be anything, and
          // 0 times an infinity is none: clear those rows of V
          const int op = op0 + op_of_v(j, nt), os = op % C::kOps;
          wait(&sm.op_full[os], (uint32_t)(op / C::kOps) & 1u);
          if (at >= it.past + it.n) {
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
              *reinterpret_cast<uint4*>(sm.op[os] + (c >> 3) * kStepKeys * 128 + key * 128 +
                                        (c & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&sm.p_full[buf]);
      }
      op0 += 2 * nt;

      // ---- the item's sums and results ----
#pragma unroll
      for (int c = 0; c < R; c += kChunk32) {
        // sums over the warp's 32 keys: halves of the rows to halves of the lanes
        float v[kChunk32];
#pragma unroll
        for (int i = 0; i < kChunk32; ++i) v[i] = l[c + i];
        const float s = lanes_reduce<kChunk32>(v, lane);
        if (lane < kChunk32) sm.part[quarter][n0 + c + lane] = s;
      }
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (alive && !mbar_wait_spin(bar, parity)) {
          alive = false;
          flags |= DSPARK_FLAG_TIMEOUT;
        }
      };
      named_sync(bar_wg, 128);
      const bool whole = it.part == 0;
      const size_t slot_row = (size_t)(2 * blockIdx.x + (it.part == 2)) * N;
      if (key < R) {
        const int n = n0 + key;
        const float L = (sm.part[0][n] + sm.part[1][n]) + (sm.part[2][n] + sm.part[3][n]);
        sm.f[n] = 1.0f / L;
        if (!whole && n < it.n_rows) parts.ml[slot_row + n] = make_float2(sm.m[n], L);
      }
      wait(&sm.p_empty[(tile - 1) & 1], (uint32_t)((tile - 1) >> 1) & 1u);
      tc_fence_after();
      named_sync(bar_wg, 128);
      if (key < D) {  // uniform over a warp
#pragma unroll
        for (int c = 0; c < R; c += 8) {
          if (n0 + c >= it.n_rows) break;
          uint32_t o[8];
          tmem_ld<8>(tmem + lane_base + 2 * N + n0 + c, o);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int n = n0 + c + i;
            if (n < it.n_rows) {
              if (whole) {
                const float v = __uint_as_float(o[i]) * sm.f[n];
                if (!isfinite(v)) sm.bad[n] = 1;
                static_cast<T*>(a.out)[sm.out[n] + key] = to_elem<T>(v);
              } else {
                parts.o[(slot_row + n) * D + key] = __uint_as_float(o[i]);
              }
            }
          }
        }
      }
      tc_fence_before();
      named_sync(bar_wg, 128);
      // a result that is not finite may come from a position that its row does
      // not see (0 times infinity): form the row again from those it sees
      if (whole) {
        for (int n = n0 + quarter; n < n0 + R && n < it.n_rows; n += 4) {
          if (!sm.bad[n]) continue;
          const int rr = it.qt * N + n, tok = a.by_g.div(rr);
          attend_row<T, TC, D>(a, it.b, it.past + tok, it.h * a.G + rr - tok * a.G, it.row0 + tok,
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
    if (threadIdx.x == 0) {
      uint64_t* full = kQ8 ? sm.raw_full : sm.op_full;
      const int last = max(sm.last_k, sm.last_v);
      for (int op = max(last - C::kRing + 1, 0); op <= last; ++op)
        mbar_wait(&full[op % C::kRing], (uint32_t)(op / C::kRing) & 1u);
      if (kQ8)
        for (int t = max(sm.last_tile - kStepScales + 1, 0); t <= sm.last_tile; ++t)
          mbar_wait(&sm.scale_full[t % kStepScales], (uint32_t)(t / kStepScales) & 1u);
    }
    __syncthreads();
  }
  if (warp == kStepMma) tmem_dealloc(tmem, kTmemCols);
  if (threadIdx.x == 0) store_status(a.status, sm.flags);
}

}  // namespace dspark
