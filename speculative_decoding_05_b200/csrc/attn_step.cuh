// attn_step.cuh -- attention of a decode or verify step on the tensor cores:
// up to 80 (token, query head) rows an item.
//
// The cache's bytes bound such a call as long as the work on a key stays
// short.  The warp-level matrix instructions do not keep up: 32 padded rows
// measured 205 multiply-adds a clock and SM, twice the time of the stream
// itself.  tcgen05 does, with the keys as the M dimension, so that its 128
// lanes are full however few rows there are:
//   S^T [128 keys, N rows] = K Q^T      both K-major as they lie in memory
//   O^T [D, N rows]      += V^T P^T     V as it lies (its MN-major form), P^T
//                                       [128 keys][N rows] written by the threads
//   L   [., N rows]      += 1 P^T       the weights' sums, alike in every lane
//                                       (e4m3: summed by the threads)
// P is rounded to V's 16 bits: the product takes both operands in one type, and
// tf32, with no more bits than fp16, at half the rate.  A weight is off by 2^-8
// (bf16) or 2^-11 of itself at most, a result by as much of sum_j w_j |v_j|.  L is
// summed from the rounded weights (e4m3: from the unrounded).
// Two pairs of warpgroups take the tiles in turn, each with O^T and L of its
// own, joined at the item's end: a tile's softmax is a chain of some 2000 clocks
// (scores out of TMEM, exponentials, weights to shared memory, hand-over to the
// MMAs), the stream brings a tile in 1400 to 2800.  A thread owns one key and
// half of the N rows.
// A row's softmax then lies across threads, so its reference is not the running
// maximum: weights are 2^(s - m) with m = 0 to begin with, which costs no
// precision in floating point while scores stay within 2^+-kHot, and one vote a
// tile finds the rare tile with a score outside, where m moves to the maximum
// and O^T and L are rescaled.  (fp16 weights have a short range: there m starts
// kLift below the maximum of the first tile, which stands in the middle of the
// range that is left above it: with the maximum at 1 keys 2^-25 below it were lost
// as a whole, however many.)
//
// e4m3 cache: S^T takes K's codes as they lie, by the 8-bit MMA, and Q as a sum
// of two e4m3 parts (three for fp16): a row of Q, scaled by a power of two to a
// largest element in [128, 256), is rounded to e4m3 (4 significant bits), the
// rest rounded again (4 more).  bf16 has 8 and fp16 11 bits, so the sum is exact
// for elements down to 2^-9 (2^-6) of the row's largest; below that it is off by
// at most 2^-17 of it, a score by 2^-17 sm_scale max|q| sum|k|.  Each row has a power
// of its own, which goes to its scores with K's scale: with one for all rows of an
// item a loud row took its neighbours' bits.  (That costs nothing at 32 rows and
// 128 elements: 64 requests over 4096 keys 137 us, with one power 144; 10 % at 64
// rows of 64: 252 for 227.)
// V's codes are widened to fp16 (exact) by 4 warps, and P is fp16 with V's scale
// on it: the reference is such that the product stays in fp16's range.
//
// Warps: 16 softmax, one each that loads K (and walks the piece), V, and Q (and
// scales), one that issues the MMAs, 4 that widen V (e4m3).  The operands pass in the order
// K0 K1 K2 V0 K3 V1 ..: scores are formed two tiles ahead, as far as their two
// buffers reach.
//
// Measured (whole calls, of the measured copy bandwidth where that bounds): 16-bit
// caches 72 to 78 % (64 to 256 requests of some thousand tokens, one of 128 k);
// e4m3 with 32 rows 53 %: with 16 rows 123 us, with 32 137 (64 requests over 4096
// keys), against a floor of 85, so most of what it costs over the stream is a key
// tile's, whatever the rows: 24 warps of different code use 0.56 of the issue slots
// and wait for each other's hand-overs and for instructions.  fp16 heads of 64 with
// one row a head: 167 us, where a form on warp-level matrix instructions took 148:
// a tile is half the bytes there for the same chain of hand-overs.  One request's
// step 14 us (host 14), a block of 16 31 us.
#pragma once

#include <type_traits>

#include "attn_plan.cuh"
#include "attn_tc.cuh"

namespace dspark {

constexpr int kStepKeys = 128;
constexpr int kStepSoftmax = 16;                   // warps, in two streams of two groups
constexpr int kStepLoadK = kStepSoftmax;           // warp
constexpr int kStepLoadV = kStepSoftmax + 1;       // warp
constexpr int kStepLoadQ = kStepSoftmax + 2;       // warp
constexpr int kStepMma = kStepSoftmax + 3;         // warp
constexpr int kStepWiden = kStepSoftmax + 4;       // first of 4 warps, e4m3 only
constexpr int kStepItems = 4;
constexpr int kStepScales = 4;
// fp16 weights: the largest is 2^kHalfLift where the reference was moved, 2^kHot at
// most.  Their sums then keep what lies 2^(25 + kHalfLift) below it; less room above
// moves references more often.
constexpr float kHalfLift = 8.0f;
constexpr int kSmemLimit = 232448;                 // 227 KB a CTA

template <typename TC>
__host__ __device__ constexpr int step_threads() {
  return 32 * (kStepSoftmax + 4 + (sizeof(TC) == 1 ? 4 : 0));
}

// Shared memory.  A 16-bit cache has one ring of operand tiles for K and V.  An
// e4m3 cache has a ring of K tiles, one of V tiles as they come, and one of
// widened V tiles.
template <typename T, typename TC, int D, int N>
struct StepCfg {
  static constexpr bool kQ8 = sizeof(TC) == 1;
  static constexpr int kQParts = !kQ8 ? 1 : std::is_same<T, __half>::value ? 3 : 2;
  static constexpr int kTile = kStepKeys * D * 2;            // an operand tile of 16 bits
  static constexpr int kTileIn = kStepKeys * D * (int)sizeof(TC);  // a tile as TMA brings it
  static constexpr int kQBufs = N <= 64 ? 2 : 1;
  static constexpr int kQBytes = N * D * (kQ8 ? kQParts : 2);
  static constexpr int kW = N % 64 == 0 ? 64 : N % 32 == 0 ? 32 : 16;  // rows of P^T in a line
  static constexpr int kPBytes = kStepKeys * N * 2;
  // TMEM: S^T, O^T and L (16 bits) for each stream, the ones that make L
  static constexpr int kCols = kQ8 ? 4 * N : 6 * N + 8;
  static constexpr int kTmemCols = kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static_assert(kCols <= 512, "TMEM");
  static constexpr int kSmall = 10240;
  // 16 KB behind the 16-bit tiles, see StepSmem
  static constexpr int kPQ = kQBufs * kQBytes + 2 * kPBytes;
  static constexpr int kBehind = kPQ < 16384 ? 16384 - kPQ : 16;
  static constexpr int kLeft = kSmemLimit - 1024 - kSmall - kPQ - kBehind;
  static constexpr int kOps = kQ8 ? 2 : kLeft / kTile < 8 ? kLeft / kTile : 8;
  static constexpr int kInFit = kQ8 ? (kLeft - kOps * kTile) / kTileIn : 0;
  static constexpr int kIn = kInFit < 16 ? kInFit : 16;
  static constexpr int kRingK = kQ8 ? (kIn + 1) / 2 : kOps;
  static constexpr int kRingV = kQ8 ? kIn / 2 : kOps;
  static_assert(kOps >= 2 && kRingV >= 1, "shared memory");
};

template <typename T, typename TC, int D, int N>
struct StepSmem {
  using C = StepCfg<T, TC, D, N>;
  alignas(1024) unsigned char op[C::kOps][C::kTile];
  // with D = 64 the MMAs of V read 16 KB past a tile (see the MMA warp): p, q
  // and `behind` are as much
  alignas(1024) unsigned char p[2][C::kPBytes];
  alignas(1024) unsigned char q[C::kQBufs][C::kQBytes];
  unsigned char behind[C::kBehind];
  alignas(1024) unsigned char in_k[C::kQ8 ? C::kRingK : 1][C::kQ8 ? C::kTileIn : 16];
  alignas(1024) unsigned char in_v[C::kQ8 ? C::kRingV : 1][C::kQ8 ? C::kTileIn : 16];
  alignas(16) float scale[C::kQ8 ? kStepScales : 1][2][kStepKeys];
  alignas(16) float qs[2][C::kQ8 ? N : 4];  // e4m3: power of two taken off each row of Q
  alignas(16) float neg_m[2][N], f[2][N], part[2][4][N];  // of each stream: -m, ..
  int low[N], bad[N];
  long long out[N];
  uint64_t k_full[C::kRingK], k_empty[C::kRingK];  // 16 bits: of the common ring
  uint64_t v_full[C::kRingV], v_empty[C::kRingV];  // e4m3 only, as the next
  uint64_t op_full[C::kOps], op_empty[C::kOps];
  uint64_t scale_full[kStepScales], scale_empty[kStepScales];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_full[2], p_empty[2];
  uint64_t item_full[kStepItems], item_empty[kStepItems];
  uint64_t v_clean[kStepItems];     // 16 bits: an item's last V tile is cleared behind its end
  uint64_t drain;
  Item item[kStepItems];
  Piece piece;
  long long scan[24];
  uint32_t tmem;
  unsigned flags;
  int stop;
  int next_k, next_v;               // operand that the K and the V warp issue next, at least
  int last_k, last_v;               // issued last
};

// Place of tile j's K and V in the operand order K0 K1 K2 V0 K3 V1 .. of an item
// of n tiles, which ends V(n - 2) V(n - 1) (or K0 V0, or K0 K1 V0 V1).
__device__ __forceinline__ int op_of_k(int j) { return j < 2 ? j : 2 * j - 2; }
__device__ __forceinline__ int op_of_v(int j, int n) { return j + min(j + 3, n); }

// Whether the last tile of an item's part has places behind the sequence.
__device__ __forceinline__ bool has_tail(const Item& it) {
  return it.t1 * kStepKeys > it.past + it.n;
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
  using C = StepCfg<T, TC, D, N>;
  using S = StepSmem<T, TC, D, N>;
  using TP = typename std::conditional<C::kQ8, __half, T>::type;  // P and V
  constexpr bool kQ8 = C::kQ8;
  constexpr int kThreads = step_threads<TC>();
  constexpr int kColO = 2 * N, kColL = 4 * N, kColOnes = 6 * N;  // TMEM: see StepCfg
  constexpr bool kHalfP = std::is_same<TP, __half>::value;
  // Scores this far over the reference move it: 2^64 leaves fp32 sums and bf16
  // weights far from their ends, 2^14 fp16 ones.  At the first keys of a row a
  // score as far below it does so too (fp16: always).
  constexpr float kHot = kHalfP ? 14.0f : 64.0f;
  constexpr float kLift = kHalfP ? kHalfLift : 0.0f;  // where a moved reference puts the maximum
  extern __shared__ unsigned char smem_raw[];
  S& sm = *reinterpret_cast<S*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr AttnTiles tiles = {N, kStepKeys};
  unsigned flags = 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kRingK; ++i) {
      mbar_init(&sm.k_full[i], 1);
      mbar_init(&sm.k_empty[i], 1);
    }
    for (int i = 0; i < C::kRingV; ++i) {
      mbar_init(&sm.v_full[i], 1);
      mbar_init(&sm.v_empty[i], 4);
    }
    for (int i = 0; i < C::kOps; ++i) {
      mbar_init(&sm.op_full[i], 4);
      mbar_init(&sm.op_empty[i], 1);
    }
    for (int i = 0; i < kStepScales; ++i) {
      mbar_init(&sm.scale_full[i], 32);
      mbar_init(&sm.scale_empty[i], kStepSoftmax / 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], 32);
      mbar_init(&sm.q_empty[i], kQ8 ? 1 + kStepSoftmax : 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], 32 * kStepSoftmax / 2);
      mbar_init(&sm.p_empty[i], 1);
    }
    for (int i = 0; i < kStepItems; ++i) {
      mbar_init(&sm.item_full[i], 1);
      mbar_init(&sm.v_clean[i], 32);
      mbar_init(&sm.item_empty[i], kQ8 ? 5 : 4);
    }
    mbar_init(&sm.drain, 1);
    sm.flags = 0;
    sm.last_k = sm.last_v = -1;
    sm.next_k = sm.next_v = 0;
    fence_barrier_init();
  }
  if (warp == kStepMma) tmem_alloc(&sm.tmem, C::kTmemCols);
  constexpr uint32_t kOne2 = kHalfP ? 0x3c003c00u : 0x3f803f80u;
  grid_dep_launch();
  grid_dep_wait();
  tc_fence_before();
  const bool small = a.rows.B <= 32;
  if (small)
    __syncthreads();
  else
    find_piece<kThreads>(a, tiles, sm.scan, &sm.piece, flags);  // syncs the block
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  if constexpr (!kQ8) {
    if (warp < 4) {
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = kOne2;
      tmem_st<8>(tmem + ((uint32_t)(warp * 32) << 16) + kColOnes, o);
      tmem_st_wait();
      tc_fence_before();  // the MMAs that read them come behind p_full
    }
  }

  if (warp == kStepLoadK || warp == kStepLoadV) {
    // ---- loads: items and K tiles (and scales); V tiles ----
    const int shift = a.rows.page_shift, in_page = (1 << shift) - 1;
    const int box_rows = 1 << box_shift;
    const bool is_k = warp == kStepLoadK;
    uint64_t* full = kQ8 && !is_k ? sm.v_full : sm.k_full;
    uint64_t* empty = kQ8 && !is_k ? sm.v_empty : sm.k_empty;
    volatile int* my_next = is_k ? &sm.next_k : &sm.next_v;
    const volatile int* other_next = is_k ? &sm.next_v : &sm.next_k;
    Walk walk;
    if (is_k) walk.start(a, tiles, small ? find_piece_warp(a, tiles, flags) : sm.piece);
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
        if (!__all_sync(0xffffffffu, alive)) {
          alive = false;
          break;
        }
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
        if (!__all_sync(0xffffffffu, alive)) {
          alive = false;
          break;
        }
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
        // use of the ring: 16 bits, the operand's place in the common order
        const int use = kQ8 ? tile0 + j : op0 + (is_k ? op_of_k(j) : op_of_v(j, n));
        int stage;
        bool again;
        uint32_t parity;  // of the stage's release
        if constexpr (kQ8) {
          stage = is_k ? use % C::kRingK : use % C::kRingV;
          again = use >= (is_k ? C::kRingK : C::kRingV);
          parity = (uint32_t)((is_k ? use / C::kRingK : use / C::kRingV) - 1) & 1u;
        } else {
          stage = use % C::kOps;
          again = use >= C::kOps;
          parity = (uint32_t)(use / C::kOps - 1) & 1u;
          if (lane == 0) *my_next = use;
          // The wait for the stage's release tells phases apart by parity only.
          // Its last use may be the other warp's: once that is filled the use
          // before it has been released, and the parity can mean one phase only.
          if (again && !next_past(other_next, use - C::kOps)) alive = false;
        }
        if (again && alive) alive = mbar_wait(&empty[stage], parity);
        if (!__all_sync(0xffffffffu, alive)) {
          alive = false;
          break;
        }
        if (elect_one()) {
          mbar_arrive_expect_tx(&full[stage], (boxes << box_shift) * D * (int)sizeof(TC));
          unsigned char* dst = !kQ8 ? sm.op[stage] : is_k ? sm.in_k[stage] : sm.in_v[stage];
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
            }
          }
        }
        __syncwarp();
        if (lane == 0) {  // for the drain after an abort
          *(is_k ? &sm.last_k : &sm.last_v) = use;
        }
      }
      op0 += 2 * n;
      tile0 += n;
      if (lane == 0) *my_next = op0;  // or a later one: the next item says
    }
    if (!alive) flags |= DSPARK_FLAG_TIMEOUT;
    if (lane == 0 && is_k) parts.rec[blockIdx.x] = rec;

  } else if (warp == kStepLoadQ) {
    // ---- Q rows to shared memory (rows behind the last are zero); 16 bits: V
    //      cleared behind the end of a sequence; e4m3: scales ----
    bool alive = true;
    int op0 = 0, n_before = 0, tile = 0;
    Item before;
    before.part = -1;
    for (int n_item = 0;; ++n_item) {
      const int slot = n_item % kStepItems, qb = n_item % C::kQBufs;
      alive = mbar_wait(&sm.item_full[slot], (uint32_t)(n_item / kStepItems) & 1u);
      if (!__all_sync(0xffffffffu, alive)) {
        alive = false;
        break;
      }
      const Item it = sm.item[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.item_empty[slot]);
      if (it.part >= 0) {
        if (n_item >= C::kQBufs)
          alive = mbar_wait(&sm.q_empty[qb], (uint32_t)(n_item / C::kQBufs - 1) & 1u);
        if (!__all_sync(0xffffffffu, alive)) {
          alive = false;
          break;
        }
        constexpr int kChunks = D / 8;
        auto source = [&](int i) {
          const int rr = it.qt * N + min(i / kChunks, it.n_rows - 1), tok = a.by_g.div(rr);
          return static_cast<const T*>(a.q) + (it.row0 + tok) * a.q_stride +
                 (it.h * a.G + rr - tok * a.G) * D + 8 * (i % kChunks);
        };
        if constexpr (!kQ8) {
#pragma unroll 8
          for (int i = lane; i < N * kChunks; i += 32)
            cp_async16(sm.q[qb] + sw128_offset(i / kChunks, 8 * (i % kChunks), N), source(i),
                       i / kChunks < it.n_rows);
          cp_async_wait_all();
        } else {
          // a row on four lanes, 8 rows a set; all loads of some sets before the
          // first store (stores might alias them: each would wait for its load)
          constexpr int kPer = kChunks / 4, kSets = N / 8 < 8 / kPer ? N / 8 : 8 / kPer;
          static_assert(N % (8 * kSets) == 0, "whole sets");
#pragma unroll 1
          for (int r0 = lane / 4; r0 < N; r0 += 8 * kSets) {
            uint4 v[kSets][kPer];
#pragma unroll
            for (int s = 0; s < kSets; ++s) {
#pragma unroll
              for (int k = 0; k < kPer; ++k) {
                v[s][k] = *reinterpret_cast<const uint4*>(
                    source((r0 + 8 * s) * kChunks + 4 * k + lane % 4));
                if (r0 + 8 * s >= it.n_rows) v[s][k] = make_uint4(0, 0, 0, 0);
              }
            }
#pragma unroll
            for (int s = 0; s < kSets; ++s) {
              const int r = r0 + 8 * s;
              // the row's largest element, as bits: sizes in their order,
              // infinities and NaN above them
              uint32_t top = 0;
#pragma unroll
              for (int k = 0; k < kPer; ++k) {
                float y[8];
                unpack8<T>(v[s][k], y);
#pragma unroll
                for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(y[e]) & 0x7fffffffu);
              }
              top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
              top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
              const int up = min(134 - (int)(top >> 23), 120);  // top 2^up in [128, 256)
              const float mul = __uint_as_float((uint32_t)(127 + up) << 23);
#pragma unroll
              for (int k = 0; k < kPer; ++k) {
                float y[8];
                unpack8<T>(v[s][k], y);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] *= mul;
#pragma unroll
                for (int pt = 0; pt < C::kQParts; ++pt) {
                  const uint32_t lo = f32_to_e4m3x4(y[0], y[1], y[2], y[3]);
                  const uint32_t hi = f32_to_e4m3x4(y[4], y[5], y[6], y[7]);
                  *reinterpret_cast<uint2*>(sm.q[qb] + pt * N * D +
                                            k8_offset<D>(r, 8 * (4 * k + lane % 4))) =
                      make_uint2(lo, hi);
                  float z[8];
                  e4m3x4_to_f32(lo, z);
                  e4m3x4_to_f32(hi, z + 4);
#pragma unroll
                  for (int e = 0; e < 8; ++e) y[e] -= z[e];
                }
              }
              // a value that is not finite has no such parts: the row's results
              // become not finite, and it is formed by itself
              if (lane % 4 == 0)
                sm.qs[qb][r] = top >= 0x7f800000u ? CUDART_NAN_F
                                                  : __uint_as_float((uint32_t)(127 - up) << 23);
            }
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(&sm.q_full[qb]);
      }
      if constexpr (kQ8) {
        // (Q of the next item comes behind the last of these, some tiles before
        // it is used)
        const int n = it.part >= 0 ? it.t1 - it.t0 : 0;
        const int shift = a.rows.page_shift, in_page = (1 << shift) - 1;
        const int* table = a.rows.page_table + (it.part >= 0 ? (size_t)it.b * a.rows.max_pages : 0);
        const int last_key = it.past + it.n;
        // a lane's 4 keys lie in one page; its id is read a tile ahead
        auto page_of = [&](int j) {
          const int k = (it.t0 + j) * kStepKeys + 4 * lane;
          return j < n && k < last_key ? __ldg(table + (k >> shift)) : 0;
        };
        int page = page_of(0);
#pragma unroll 1
        for (int j = 0; j < n; ++j, ++tile) {
          const int k = (it.t0 + j) * kStepKeys + 4 * lane;
          int pid = page;
          if ((unsigned)pid >= (unsigned)a.rows.n_pages) pid = 0;  // flagged with its tile
          const long long at = (((long long)pid * a.Hkv + it.h) << shift) + (k & in_page);
          page = page_of(j + 1);
          const int sc = tile % kStepScales;
          if (tile >= kStepScales)
            alive = mbar_wait(&sm.scale_empty[sc], (uint32_t)(tile / kStepScales - 1) & 1u);
          if (!__all_sync(0xffffffffu, alive)) {
            alive = false;
            break;
          }
          cp_async16(&sm.scale[sc][0][lane * 4], a.k_scale + at, k < last_key);
          cp_async16(&sm.scale[sc][1][lane * 4], a.v_scale + at, k < last_key);
          cp_async_arrive(&sm.scale_full[sc]);
        }
        if (!alive) break;
      }
      if (!kQ8 && before.part >= 0) {
        // What lies behind the sequence in its last page may be anything, and 0
        // times an infinity is none: clear those rows of the last V tile.  One
        // item behind, so that Q of the next is there in time.
        if (has_tail(before)) {
          const int use = op0 + op_of_v(n_before - 1, n_before), os = use % C::kOps;
          // once it is issued, the parity can mean this fill only
          alive = next_past(&sm.next_v, use) &&
                  mbar_wait(&sm.k_full[os], (uint32_t)(use / C::kOps) & 1u);
          if (!__all_sync(0xffffffffu, alive)) {
            alive = false;
            break;
          }
          const int here = before.past + before.n - (before.t1 - 1) * kStepKeys;
          for (int i = lane; i < (kStepKeys - here) * (D / 8); i += 32) {
            const int k = here + i / (D / 8), c = i % (D / 8);
            *reinterpret_cast<uint4*>(sm.op[os] + (c >> 3) * kStepKeys * 128 + k * 128 +
                                      (c & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        // (a slot of these can not be lapped: the next item in it is published
        // when the MMA warp is past this one)
        mbar_arrive(&sm.v_clean[(n_item - 1) % kStepItems]);
        op0 += 2 * n_before;
      }
      if (it.part < 0) break;
      before = it;
      n_before = it.t1 - it.t0;
    }
    if (kQ8) cp_async_wait_all();
    if (!alive) flags |= DSPARK_FLAG_TIMEOUT;

  } else if (warp == kStepMma) {
    // ---- MMA issue: one thread ----
    constexpr uint32_t kIdS = kQ8 ? idesc_e4m3(128, N) : idesc_tc<T>(128, N, false, false);
    constexpr uint32_t kIdO = idesc_tc<TP>(128, N, true, true);
    constexpr uint32_t kIdL = idesc_tc<TP>(128, N, false, true);
    constexpr int kW = C::kW;
    if (elect_one()) {
      bool alive = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (alive) alive = mbar_wait_spin(bar, parity);
      };
      int op0 = 0, tile0 = 0;
      for (int n_item = 0;; ++n_item) {
        const int slot = n_item % kStepItems;
        wait(&sm.item_full[slot], (uint32_t)(n_item / kStepItems) & 1u);
        if (!alive) break;
        const int part = sm.item[slot].part, n = sm.item[slot].t1 - sm.item[slot].t0;
        consumed(__int_as_float(part + n));
        mbar_arrive(&sm.item_empty[slot]);
        if (part < 0) break;
        const int qb = n_item % C::kQBufs;
        const uint32_t q_addr = smem_u32(sm.q[qb]);
        auto issue_s = [&](int j) {
          const int use = kQ8 ? tile0 + j : op0 + op_of_k(j), ks = use % C::kRingK;
          const int buf = (tile0 + j) & 1;
          wait(&sm.k_full[ks], (uint32_t)(use / C::kRingK) & 1u);
          if (!alive) return;
          tc_fence_after();
          if constexpr (kQ8) {
            const uint64_t kd = sdesc_k8<D>(smem_u32(sm.in_k[ks])), qd = sdesc_k8<D>(q_addr);
#pragma unroll
            for (int pt = 0; pt < C::kQParts; ++pt)
#pragma unroll
              for (int k = 0; k < D / 32; ++k)
                mma_e4m3_ss(tmem + buf * N, kd + ((k * 32) >> 4), qd + ((pt * N * D + k * 32) >> 4),
                            kIdS, pt > 0 || k > 0);
          } else {
            const uint64_t kd = sdesc_sw128(smem_u32(sm.op[ks])), qd = sdesc_sw128(q_addr);
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              mma_bf16_ss(tmem + buf * N, kd + (((k >> 2) * kStepKeys * 128 + (k & 3) * 32) >> 4),
                          qd + (((k >> 2) * N * 128 + (k & 3) * 32) >> 4), kIdS, k > 0);
          }
          mma_commit(&sm.s_full[buf]);
          mma_commit(&sm.k_empty[ks]);
          if (j == n - 1) mma_commit(&sm.q_empty[qb]);
        };
        wait(&sm.q_full[qb], (uint32_t)(n_item / C::kQBufs) & 1u);
        issue_s(0);
        if (n > 1) issue_s(1);
        for (int j = 0; j < n; ++j) {
          const int g = tile0 + j, buf = g & 1;
          wait(&sm.p_full[buf], (uint32_t)(g >> 1) & 1u);
          // the scores of tile j were read: their buffer takes those of j + 2
          if (j + 2 < n) issue_s(j + 2);
          const int use = kQ8 ? g : op0 + op_of_v(j, n), os = use % C::kOps;
          wait(kQ8 ? &sm.op_full[os] : &sm.k_full[os], (uint32_t)(use / C::kOps) & 1u);
          if (!kQ8 && j == n - 1) wait(&sm.v_clean[slot], (uint32_t)(n_item / kStepItems) & 1u);
          if (!alive) break;
          tc_fence_after();
          // V: 64 elements of D in a row, 8 keys 1024 bytes apart, the other 64
          // behind all keys.  With D = 64 there are no others: lanes 64-127 of
          // O^T take what lies there and nobody reads them.
          const uint64_t vd = sdesc_mn<64>(smem_u32(sm.op[os]), kStepKeys);
          const uint64_t pd = sdesc_mn<kW>(smem_u32(sm.p[buf]), kStepKeys);
#pragma unroll
          for (int k = 0; k < kStepKeys / 16; ++k)
            mma_bf16_ss(tmem + kColO + buf * N, vd + ((k * 2048) >> 4),
                        pd + ((k * 16 * kW * 2) >> 4), kIdO, j > 1 || k > 0);
          mma_commit(kQ8 ? &sm.op_empty[os] : &sm.k_empty[os]);
          if constexpr (!kQ8) {
#pragma unroll
            for (int k = 0; k < kStepKeys / 16; ++k)
              mma_bf16_ts(tmem + kColL + buf * N, tmem + kColOnes, pd + ((k * 16 * kW * 2) >> 4),
                          kIdL, j > 1 || k > 0);
          }
          mma_commit(&sm.p_empty[buf]);
        }
        op0 += 2 * n;
        tile0 += n;
      }
      if (!alive) flags |= DSPARK_FLAG_TIMEOUT;
      drain_mma(&sm.drain);
    }
    __syncwarp();

  } else if (warp >= kStepWiden) {
    // ---- V tiles of e4m3 to fp16 ----
    if constexpr (kQ8) {
      const int tid = threadIdx.x - 32 * kStepWiden;
      bool alive = true;
      int use = 0;
      for (int n_item = 0;; ++n_item) {
        const int slot = n_item % kStepItems;
        if (alive) alive = mbar_wait(&sm.item_full[slot], (uint32_t)(n_item / kStepItems) & 1u);
        const int part = sm.item[slot].part, n = sm.item[slot].t1 - sm.item[slot].t0;
        const int keys = sm.item[slot].past + sm.item[slot].n - sm.item[slot].t0 * kStepKeys;
        // all four warps go on or all stop
        if (vote_any(6, 128, !alive)) {
          alive = false;
          break;
        }
        if (tid == 0) mbar_arrive(&sm.item_empty[slot]);
        if (part < 0) break;
        for (int j = 0; j < n && alive; ++j, ++use) {
          const int vs = use % C::kRingV, os = use % C::kOps;
          alive = mbar_wait(&sm.v_full[vs], (uint32_t)(use / C::kRingV) & 1u);
          if (alive && use >= C::kOps)
            alive = mbar_wait(&sm.op_empty[os], (uint32_t)(use / C::kOps - 1) & 1u);
          if (!alive) break;
          widen_tile<D>(sm.in_v[vs], sm.op[os], keys - j * kStepKeys, tid);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sm.v_empty[vs]);
            mbar_arrive(&sm.op_full[os]);
          }
        }
      }
      if (!alive) flags |= DSPARK_FLAG_TIMEOUT;
    }

  } else {
    // ---- softmax: the streams take the tiles in turn, a thread one key ----
    constexpr int R = N / 2;                      // rows of a thread
    constexpr int kCols = R % 16 == 0 ? 16 : 8;   // columns of a load
    constexpr int kLoads = R / kCols;
    constexpr int kW = C::kW;
    // e4m3: P carries V's scale, so its sums are not the weights': those are
    // summed by the threads, when the vote has let the tile pass
    constexpr bool kKeep = kQ8 && kLoads == 1;    // a tile's weights are kept until then
    const int wg = warp >> 2, quarter = warp & 3;
    const int stream = wg >> 1, n0 = (wg & 1) * R;
    const int key = quarter * 32 + lane;          // in the tile; in the epilogue: lane of O^T
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
    const int bar_wg = 2 + wg;
    bool alive = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (alive && !mbar_wait(bar, parity)) {
        alive = false;
        flags |= DSPARK_FLAG_TIMEOUT;
      }
    };
    int tile0 = 0;
    for (int n_item = 0;; ++n_item) {
      const int slot = n_item % kStepItems, qb = n_item % C::kQBufs;
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
        sm.low[n] = first_seen(p, a.window);
        sm.out[n] = ((it.row0 + tok) * a.Hq + it.h * a.G + rr - tok * a.G) * (long long)D;
        sm.neg_m[0][n] = sm.neg_m[1][n] = 0.0f;
        sm.bad[n] = 0;
      }
      named_sync(1, 32 * kStepSoftmax);
      if (threadIdx.x == 0) mbar_arrive(&sm.item_empty[slot]);
      const int nt = it.t1 - it.t0;
      const int pos_min = it.past + a.by_g.div(it.qt * N);
      const int pos_max = it.past + a.by_g.div(it.qt * N + it.n_rows - 1);
      const int low_max = first_seen(pos_max, a.window);
      float l[kQ8 ? R : 1];
#pragma unroll
      for (int i = 0; i < (kQ8 ? R : 1); ++i) l[i] = 0.0f;

      for (int j = (tile0 ^ stream) & 1; j < nt; j += 2) {
        const int tile = tile0 + j, buf = stream;  // tile & 1
        const uint32_t phase = (uint32_t)(tile >> 1) & 1u;
        const int k0 = (it.t0 + j) * kStepKeys;
        const int at = k0 + key;
        const bool masked = k0 + kStepKeys > pos_min + 1 || k0 < low_max;
        // rows that see this thread's key: row n of the tile is token (qt N + n) / G
        int n_lo = 0, n_hi = N;
        if (masked) {
          n_lo = max(at - it.past, 0) * a.G - it.qt * N;
          if (a.window > 0) {
            const long long e = (long long)at - it.past + a.window;
            n_hi = (int)max(min(e, (long long)it.n), 0ll) * a.G - it.qt * N;
            if (e >= it.n) n_hi = N;
          }
          // behind the sequence nobody sees, rows that pad included: a score or
          // scale from there must not even count in the vote
          if (at >= it.past + it.n) n_lo = N;
          n_lo -= n0;
          n_hi -= n0;
        }
        // the first keys of some row in this stream's tiles
        const bool first = j < 2 || k0 - kStepKeys <= low_max;
        float kf = a.scale2, vs = 1.0f, vs2 = 0.0f;
        if constexpr (kQ8) {
          const int sc = tile % kStepScales;
          wait(&sm.scale_full[sc], (uint32_t)(tile / kStepScales) & 1u);
          kf *= sm.scale[sc][0][key];
          vs = sm.scale[sc][1][key];
          // P carries the scale: its size counts.  (Down to 2^-80: the weights
          // themselves then stay below 2^94, and their sums over all positions in
          // fp32's range.)
          vs2 = fmaxf(__log2f(vs), -80.0f);
          consumed(kf + vs2);
          // a scale behind the sequence may be anything
          if (at >= it.past + it.n) vs = vs2 = 0.0f;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.scale_empty[sc]);
        }
        wait(&sm.s_full[buf], phase);
        tc_fence_after();
        const uint64_t kf2 = pair_of(kf, kf), vsv = pair_of(vs, vs);
        const uint32_t s_col = lane_base + buf * N + n0;

        // scores of some rows from row n0 + c over the reference, in units of log 2
        auto load = [&](auto& x, int c, bool over) {
          constexpr int kX = sizeof(x) / 4;
          uint32_t raw[kX];
          tmem_ld<kX>(s_col + c, raw);
#pragma unroll
          for (int i = 0; i < kX; i += 4) {
            float4 m4 = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (over) m4 = *reinterpret_cast<const float4*>(&sm.neg_m[stream][n0 + c + i]);
            uint64_t s0 = pair_of(__uint_as_float(raw[i]), __uint_as_float(raw[i + 1]));
            uint64_t s1 = pair_of(__uint_as_float(raw[i + 2]), __uint_as_float(raw[i + 3]));
            if constexpr (kQ8) {
              const float4 q4 = *reinterpret_cast<const float4*>(&sm.qs[qb][n0 + c + i]);
              s0 = mul2(s0, pair_of(q4.x, q4.y));
              s1 = mul2(s1, pair_of(q4.z, q4.w));
            }
            pair_to(fma2(s0, kf2, pair_of(m4.x, m4.y)), x[i], x[i + 1]);
            pair_to(fma2(s1, kf2, pair_of(m4.z, m4.w)), x[i + 2], x[i + 3]);
          }
          if (masked) {
#pragma unroll
            for (int i = 0; i < kX; ++i)
              if (c + i < n_lo || c + i >= n_hi) x[i] = -CUDART_INF_F;
          }
        };
        float x[kCols];
        bool raise = kHalfP && first, p_free = tile < 2;
        while (true) {
          if (raise) {
            // move the references to the tile's maxima (loops kept short: this
            // is rare, and its code should not crowd out the rest)
#pragma unroll 1
            for (int c = 0; c < R; c += 8) {
              float y[8];
              load(y, c, false);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float w = warp_max_redux(y[i] + vs2);
                if (lane == 0) sm.part[stream][quarter][n0 + c + i] = w;
              }
            }
            named_sync(bar_wg, 128);
            if (key < R) {
              const int n = n0 + key;
              const float old = -sm.neg_m[stream][n];
              const float top = fmaxf(fmaxf(sm.part[stream][0][n], sm.part[stream][1][n]),
                                      fmaxf(sm.part[stream][2][n], sm.part[stream][3][n]));
              // whether an earlier tile of this stream has keys of the row
              const bool seen = j > 1 && k0 - kStepKeys > sm.low[n];
              const float to = top - kLift;
              const float now = seen ? fmaxf(old, to) : top == -CUDART_INF_F ? old : to;
              sm.f[stream][n] = seen && now != old ? ex2(old - now) : 1.0f;
              sm.neg_m[stream][n] = -now;
            }
            named_sync(bar_wg, 128);
            if constexpr (kQ8) {
#pragma unroll
              for (int i = 0; i < R; ++i) l[i] *= sm.f[stream][n0 + i];
            }
            if (j > 1) {
              // O^T and L hold the tiles up to two before
              wait(&sm.p_empty[buf], phase ^ 1u);
              p_free = true;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < (kQ8 ? R : 2 * R); c += 8) {  // O^T, then L
                const int n = n0 + (c < R ? c : c - R);
                const uint32_t col = lane_base + (c < R ? kColO : kColL) + stream * N + n;
                uint32_t o[8];
                tmem_ld<8>(col, o);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  o[i] = __float_as_uint(__uint_as_float(o[i]) * sm.f[stream][n + i]);
                tmem_st<8>(col, o);
              }
              tmem_st_wait();
            }
          }
          // weights, as if no score were outside the range
          float top = -CUDART_INF_F, bottom = CUDART_INF_F;
          unsigned char* prow = sm.p[buf];
#pragma unroll
          for (int c = 0; c < R; c += kCols) {
            load(x, c, true);
#pragma unroll
            for (int i = 0; i < kCols; i += 2) top = max3(top, x[i], x[i + 1]);
            if (!kHalfP && first) {
#pragma unroll
              for (int i = 0; i < kCols; ++i)
                bottom = fminf(bottom, x[i] == -CUDART_INF_F ? CUDART_INF_F : x[i]);
            }
            uint32_t w[kCols / 2];
#pragma unroll
            for (int i = 0; i < kCols; i += 2) {
              float p0 = ex2(x[i]), p1 = ex2(x[i + 1]);
              if constexpr (kKeep) {
                x[i] = p0;
                x[i + 1] = p1;
              }
              if constexpr (kQ8) pair_to(mul2(pair_of(p0, p1), vsv), p0, p1);
              w[i / 2] = Pair<TP>::put(p0, p1);
            }
            if (!p_free) {  // the buffer was last read by the MMAs two tiles before
              wait(&sm.p_empty[buf], phase ^ 1u);
              p_free = true;
            }
#pragma unroll
            for (int i = 0; i < kCols; i += 8)
              *reinterpret_cast<uint4*>(prow + mn_offset<kW>(n0 + c + i, key, kStepKeys)) =
                  make_uint4(w[i / 2], w[i / 2 + 1], w[i / 2 + 2], w[i / 2 + 3]);
          }
          if (raise) break;
          raise = vote_any(bar_wg, 128, top + vs2 > kHot || bottom < -kHot);
          if (!raise) break;
        }
        if constexpr (kQ8) {
#pragma unroll
          for (int c = 0; c < R; c += kCols) {
            if constexpr (!kKeep) {
              load(x, c, true);
#pragma unroll
              for (int i = 0; i < kCols; ++i) x[i] = ex2(x[i]);
            }
#pragma unroll
            for (int i = 0; i < kCols; i += 2)
              pair_to(add2(pair_of(l[c + i], l[c + i + 1]), pair_of(x[i], x[i + 1])), l[c + i],
                      l[c + i + 1]);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&sm.p_full[buf]);
      }
      if (kQ8) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_empty[qb]);  // qs is read
      }
      tile0 += nt;

      // ---- the item's results: both streams' O^T and L, 8 rows a warpgroup ----
      // (own tiles first: a later wait of the same barrier then means its phase)
      {
        const int last = tile0 - 1, prev = tile0 - 2;
        const int mine = (last & 1) == stream ? last : prev;
        const int other = (last & 1) == stream ? prev : last;
        if (mine >= tile0 - nt) wait(&sm.p_empty[mine & 1], (uint32_t)(mine >> 1) & 1u);
        if (other >= tile0 - nt) wait(&sm.p_empty[other & 1], (uint32_t)(other >> 1) & 1u);
      }
      tc_fence_after();
      const bool whole = it.part == 0;
      const size_t slot_row = (size_t)(2 * blockIdx.x + (it.part == 2)) * N;
      bool bad = false;
      if constexpr (kQ8) {
        // the threads' sums, half of a thread's rows at a time through the P
        // buffers (their MMAs are done)
        constexpr int H = R / 2;
        float* ls = reinterpret_cast<float*>(sm.p) + wg * H * kStepKeys;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          named_sync(1, 32 * kStepSoftmax);
#pragma unroll
          for (int i = 0; i < H; ++i) ls[i * kStepKeys + key] = l[hf * H + i];
          named_sync(bar_wg, 128);
          constexpr int kPer = 128 / H < 32 ? 128 / H : 32;  // threads that sum a row
          const int r = key / kPer;
          float s = 0.0f;
          if (r < H) {
#pragma unroll 4
            for (int i = key % kPer; i < kStepKeys; i += kPer) s += ls[r * kStepKeys + i];
          }
#pragma unroll
          for (int w = kPer / 2; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
          if (key % kPer == 0 && r < H) sm.f[stream][n0 + hf * H + r] = s;
        }
      }
      named_sync(1, 32 * kStepSoftmax);  // both streams' m (and sums)
      if (key < D) {  // uniform over a warp
        const int d = key;
        const int none = nt > 1 ? 2 : tile0 & 1;  // a stream without tiles
#pragma unroll 1
        for (int n = 8 * wg; n < it.n_rows; n += 32) {
          uint32_t o[2][8], L8[2][8];
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            tmem_ld8_issue(lane_base + kColO + w * N + n, o[w]);
            if constexpr (!kQ8) tmem_ld8_issue(lane_base + kColL + w * N + n, L8[w]);
          }
          tmem_ld8_wait(o[0]);
          tmem_ld8_wait(o[1]);
          if constexpr (!kQ8) {
            tmem_ld8_wait(L8[0]);
            tmem_ld8_wait(L8[1]);
          }
          // (no branches from here to the stores: eight rows side by side)
          float O[8], Ls[8], M[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float v[2], L[2], m[2];
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              v[w] = w == none ? 0.0f : __uint_as_float(o[w][i]);
              L[w] = w == none ? 0.0f : kQ8 ? sm.f[w][n + i] : __uint_as_float(L8[w][i]);
              // without a visible key there is no reference
              m[w] = L[w] == 0.0f ? -CUDART_INF_F : -sm.neg_m[w][n + i];
            }
            M[i] = fmaxf(m[0], m[1]);
            const float Mu = M[i] == -CUDART_INF_F ? 0.0f : M[i];
            const float f0 = ex2(m[0] - Mu), f1 = ex2(m[1] - Mu);
            O[i] = v[0] * f0 + v[1] * f1;
            Ls[i] = L[0] * f0 + L[1] * f1;
          }
          const int rows = it.n_rows - n;
          if (whole) {
            T* dst = static_cast<T*>(a.out) + d;
            float worst = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float r;
              asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(Ls[i]));
              O[i] *= r;
              // not a number if any of the rows' results is not finite
              worst = i < rows ? fmaf(O[i], 0.0f, worst) : worst;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (i < rows) dst[sm.out[n + i]] = to_elem<T>(O[i]);
            if (worst != 0.0f) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (i < rows && !isfinite(O[i])) sm.bad[n + i] = 1;
              bad = true;
            }
          } else {
            float* dst = parts.o + (slot_row + n) * D + d;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (i < rows) dst[i * D] = O[i];
            if (key == 0) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (i < rows) parts.ml[slot_row + n + i] = make_float2(M[i], Ls[i]);
            }
          }
        }
      }
      tc_fence_before();
      // a result that is not finite may come from a position that its row does
      // not see (0 times infinity): form the row again from those it sees
      if (vote_any(bar_wg, 128, bad)) {
        for (int n = 8 * wg; n < it.n_rows; n += 32) {
          for (int r = n + quarter; r < min(n + 8, it.n_rows); r += 4) {
            if (!sm.bad[r]) continue;
            const int rr = it.qt * N + r, tok = a.by_g.div(rr);
            attend_row<T, TC, D>(a, it.b, it.past + tok, it.h * a.G + rr - tok * a.G,
                                 it.row0 + tok, flags);
          }
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
      const int last_k = kQ8 ? sm.last_k : max(sm.last_k, sm.last_v);
      for (int u = max(last_k - C::kRingK + 1, 0); u <= last_k; ++u)
        mbar_wait(&sm.k_full[u % C::kRingK], (uint32_t)(u / C::kRingK) & 1u);
      if (kQ8) {
        for (int u = max(sm.last_v - C::kRingV + 1, 0); u <= sm.last_v; ++u)
          mbar_wait(&sm.v_full[u % C::kRingV], (uint32_t)(u / C::kRingV) & 1u);
      }
    }
    __syncthreads();
  }
  if (warp == kStepMma) tmem_dealloc(tmem, C::kTmemCols);
  if (threadIdx.x == 0) store_status(a.status, sm.flags);
}

}  // namespace dspark
