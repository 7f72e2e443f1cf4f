// kv.cu -- the C ABI of include/dspark_kv.h: argument validation and launches
// of the paged-cache calls.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "attn_chunk.cuh"
#include "attn_step.cuh"
#include "kv_common.cuh"
#include "kv_rows.cuh"
#include "kv_status.h"

using namespace dspark;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Bytes from the first of n 16-bit rows, `stride` elements apart, to the end of the last.
size_t rows_bytes(long long n, long long stride, long long width) {
  return 2 * (size_t)((n - 1) * stride + width);
}
// Whether n bytes at a and m bytes at b meet.
bool meet(const void* a, size_t n, const void* b, size_t m) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y ? y - x < n : x - y < m;
}

dspark_status launched(cudaError_t e) {
  if (e == cudaSuccess) return DSPARK_OK;
  cudaGetLastError();  // a refused launch also leaves its code behind
  return DSPARK_ERR_CUDA;
}

int page_shift(int page_size) {
  for (int s = 4; s <= 8; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

int kv_sms() {
  static DeviceOnce once;
  static int n[kMaxDevices];
  const int d = current_device();
  if (d < 0 || d >= kMaxDevices) return 148;
  once_per_device(once, [&] {
    int c = 0;
    if (cudaDeviceGetAttribute(&c, cudaDevAttrMultiProcessorCount, d) != cudaSuccess) c = 0;
    n[d] = c > 0 ? c : 148;
  });
  return n[d];
}

// Sizes and pointers every call has.
struct Common {
  dspark_kv_dtype act, cache;
  long long n_rows;
  int B, Hq, Hkv, D;
  const int64_t* row_start;
  const int32_t *verify_len, *cache_len, *page_table;
  int max_pages;
  const void *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  long long n_pages;
  int page_size;
  const void* ws;
  size_t ws_bytes, ws_need;
};

dspark_status check_common(const Common& c) {
  if (c.act != DSPARK_KV_BF16 && c.act != DSPARK_KV_F16) return DSPARK_ERR_INVALID_ARG;
  if (c.cache != DSPARK_KV_E4M3 && c.cache != c.act) return DSPARK_ERR_INVALID_ARG;
  if (c.B < 0 || c.n_rows < 0 || c.Hkv <= 0 || c.Hq <= 0 || c.D <= 0 || c.max_pages < 0 ||
      c.n_pages < 0 || c.page_size <= 0)
    return DSPARK_ERR_INVALID_ARG;
  if (c.Hq % c.Hkv != 0) return DSPARK_ERR_INVALID_ARG;
  if ((c.D != 64 && c.D != 128) || page_shift(c.page_size) < 0 || c.B > kKvMaxB || c.Hq > 1024)
    return DSPARK_ERR_UNSUPPORTED;
  if (c.n_rows > kKvMaxRows || c.n_pages >= (1ll << 31) ||
      c.n_pages * c.Hkv * c.page_size >= (1ll << 31))
    return DSPARK_ERR_UNSUPPORTED;
  if (!c.ws || !aligned(c.ws, 256) || c.ws_bytes < c.ws_need) return DSPARK_ERR_WORKSPACE;
  return DSPARK_OK;
}

// Pointers, once there is work (B > 0 and n_rows > 0).
dspark_status check_pointers(const Common& c) {
  if (!c.row_start || !c.verify_len || !c.cache_len || !c.page_table || !c.k_cache || !c.v_cache ||
      c.max_pages == 0 || c.n_pages == 0)
    return DSPARK_ERR_INVALID_ARG;
  if (!aligned(c.k_cache, 16) || !aligned(c.v_cache, 16) || !aligned(c.row_start, 8) ||
      !aligned(c.verify_len, 4) || !aligned(c.cache_len, 4) || !aligned(c.page_table, 4))
    return DSPARK_ERR_INVALID_ARG;
  if (c.cache == DSPARK_KV_E4M3 && (!c.k_scale || !c.v_scale || !aligned(c.k_scale, 16) ||
                                    !aligned(c.v_scale, 16)))
    return DSPARK_ERR_INVALID_ARG;
  return DSPARK_OK;
}

KvRows make_rows(const Common& c, int max_len) {
  KvRows r;
  r.row_start = c.row_start;
  r.verify_len = c.verify_len;
  r.cache_len = c.cache_len;
  r.page_table = c.page_table;
  r.n_rows = c.n_rows;
  r.max_pos = (long long)c.max_pages * c.page_size;
  if (r.max_pos > 1ll << 30) r.max_pos = 1ll << 30;  // positions and tile ends are int32
  r.B = c.B;
  r.max_len = max_len;
  r.max_pages = c.max_pages;
  r.page_shift = page_shift(c.page_size);
  r.n_pages = (int)c.n_pages;
  return r;
}

// Nothing to do: a call still clears the status word.
dspark_status no_work(void* ws, cudaStream_t s) {
  return cudaMemsetAsync(ws, 0, 64, s) == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

// f<T, TC, D>() for the call's types.
template <typename F>
dspark_status dispatch(const Common& c, F&& f) {
  const bool q8 = c.cache == DSPARK_KV_E4M3;
  if (c.act == DSPARK_KV_BF16) {
    using T = __nv_bfloat16;
    if (c.D == 128) return q8 ? f.template run<T, e4m3, 128>() : f.template run<T, T, 128>();
    return q8 ? f.template run<T, e4m3, 64>() : f.template run<T, T, 64>();
  }
  using T = __half;
  if (c.D == 128) return q8 ? f.template run<T, e4m3, 128>() : f.template run<T, T, 128>();
  return q8 ? f.template run<T, e4m3, 64>() : f.template run<T, T, 64>();
}

// Blocks of the row kernels: at most `per_sm` on an SM, all at once (a block
// takes runs of tokens until none are left).
int row_grid(long long n_rows, int per_sm) {
  const long long most = (long long)per_sm * kv_sms();
  const long long g = n_rows < most ? n_rows : most;
  return (int)(g < kMaxStatusCtas ? g : kMaxStatusCtas);
}

struct LaunchAppend {
  AppendArgs a;
  int grid;
  cudaStream_t s;
  template <typename T, typename TC, int D>
  dspark_status run() {
    return launched(launch_dependent(kv_append_kernel<T, TC, D>, dim3(grid), dim3(kRowThreads),
                                     (a.rows.B + 1) * sizeof(int), s, a));
  }
};

struct LaunchRead {
  ReadArgs a;
  int grid;
  cudaStream_t s;
  template <typename T, typename TC, int D>
  dspark_status run() {
    return launched(launch_dependent(kv_read_kernel<T, TC, D>, dim3(grid), dim3(kRowThreads),
                                     (a.rows.B + 1) * sizeof(int), s, a));
  }
};

// CTAs of the attention kernels, one an SM: the partial results of a workspace
// have room for a B200's.
constexpr int kAttnMaxSms = 148;
static_assert(kAttnMaxSms <= kMaxAttnCtas && kAttnMaxSms <= kMaxStatusCtas, "records");
int attn_sms() { return kv_sms() < kAttnMaxSms ? kv_sms() : kAttnMaxSms; }

struct LaunchAttn {
  AttnArgs a;
  long long rows_per_head;  // at most, of one request
  long long cache_rows;
  int page_size, D;
  unsigned char* ws;
  cudaStream_t s;

  AttnParts parts(int ctas, int rows) const {
    const PartBytes b = part_bytes(ctas, rows, D);
    AttnParts p;
    p.rec = reinterpret_cast<PartRecord*>(ws + b.rec);
    p.ml = reinterpret_cast<float2*>(ws + b.ml);
    p.o = reinterpret_cast<float*>(ws + b.o);
    return p;
  }

  template <typename T, typename TC>
  bool maps(CUtensorMap* mk, CUtensorMap* mv, int keys, int* box) const {
    constexpr bool f16 = std::is_same<T, __half>::value;
    *box = page_size < keys ? page_size : keys;
    return encode_cache_map(mk, a.k_cache, D, sizeof(TC) == 1, f16, cache_rows, *box) &&
           encode_cache_map(mv, a.v_cache, D, sizeof(TC) == 1, f16, cache_rows, *box);
  }

  template <typename T, typename TC, int Dh>
  dspark_status join(int tile_rows, const AttnParts& p, int ctas) const {
    return launched(launch_dependent(attn_join_kernel<T, TC, Dh>, dim3(kJoinPerSm * attn_sms()),
                                     dim3(kJoinThreads), 0, s, a, tile_rows, p, ctas));
  }

  template <typename T, typename TC, int Dh, int N>
  dspark_status step() const {
    constexpr int smem = (int)sizeof(StepSmem<T, TC, Dh, N>) + 1024;
    static_assert(smem <= kSmemLimit, "shared memory");
    static DeviceOnce once;
    set_smem_once(once, attn_step_kernel<T, TC, Dh, N>, smem);
    const int ctas = attn_sms();
    const AttnParts p = parts(ctas, N);
    CUtensorMap mk, mv;
    int box;
    if (!maps<T, TC>(&mk, &mv, kStepKeys, &box)) return DSPARK_ERR_CUDA;
    int box_shift = 0;
    while (1 << box_shift < box) ++box_shift;
    const dspark_status st = launched(launch_dependent(attn_step_kernel<T, TC, Dh, N>, dim3(ctas),
                                                       dim3(step_threads<TC>()), smem, s, a, p, mk,
                                                       mv, box_shift));
    return st != DSPARK_OK ? st : join<T, TC, Dh>(N, p, ctas);
  }

  template <typename T, int Dh>
  dspark_status chunk() const {
    constexpr int smem = (int)sizeof(ChunkSmem<Dh>) + 1024;
    static_assert(smem <= kSmemLimit, "shared memory");
    static DeviceOnce once;
    set_smem_once(once, attn_chunk_kernel<T, Dh>, smem);
    const int ctas = attn_sms();
    const AttnParts p = parts(ctas, kChunkRows);
    CUtensorMap mk, mv;
    int box;
    if (!maps<T, T>(&mk, &mv, kChunkKeys, &box)) return DSPARK_ERR_CUDA;
    int box_shift = 0;
    while (1 << box_shift < box) ++box_shift;
    const dspark_status st =
        launched(launch_dependent(attn_chunk_kernel<T, Dh>, dim3(ctas), dim3(kChunkThreads), smem,
                                  s, a, p, mk, mv, box_shift));
    return st != DSPARK_OK ? st : join<T, T, Dh>(kChunkRows, p, ctas);
  }

  // The tile's rows N, by the rows that a request has for a key/value head: the
  // smallest N that holds them, since the threads' work on a key goes with N.
  // Measured (us; D = 128 but for the first): one fp16 row a head (16 heads of 64), 128 requests, N = 16 169, 32
  // 180, 64 211.  64 requests over 4096 keys, 8 heads: e4m3 with 16 rows, N = 16
  // 147, 32 158; with 32 rows, N = 32 163, 64 281 (behind the 16-bit runs; by themselves
  // 124, 134, 137, 256); 16 bits with 80 rows, N = 80 198,
  // the chunk kernel 247 (its 256 rows mostly empty); with 96, two tiles of 80 350,
  // the chunk kernel 252; with 256, 412 and 324.  An e4m3 cache goes by tiles of up to 64
  // rows whatever the rows (64 rows 266, 128 479: two tiles read every key twice):
  // beside its rings and widened V the chunk kernel's 256 rows of Q have no room,
  // and the sums of its rows in the epilogue want a power of two, not 80.
  template <typename T, typename TC, int Dh>
  dspark_status run() {
    if constexpr (sizeof(TC) != 1)
      if (rows_per_head > 80) return chunk<T, Dh>();
    if (rows_per_head <= 16) return step<T, TC, Dh, 16>();
    if (rows_per_head <= 32) return step<T, TC, Dh, 32>();
    if constexpr (sizeof(TC) != 1)
      if (rows_per_head > 64) return step<T, TC, Dh, 80>();
    return step<T, TC, Dh, 64>();
  }
};

}  // namespace

namespace dspark {

bool encode_cache_map(CUtensorMap* m, const void* cache, int D, bool is_e4m3, bool is_f16,
                      long long rows, int box_rows) {
  // the driver's entry point, looked up once
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    return (PFN_cuTensorMapEncodeTiled_v12000) nullptr;
  }();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)D * (is_e4m3 ? 1 : 2)};
  const cuuint32_t box[2] = {is_e4m3 ? (cuuint32_t)D : 64u, (cuuint32_t)box_rows};
  const cuuint32_t es[2] = {1, 1};
  const CUtensorMapDataType type = is_e4m3  ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : is_f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                            : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return fn(m, type, 2, const_cast<void*>(cache), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            is_e4m3 && D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool spread_status(const unsigned* head, unsigned* count) {
  if (!(head[0] & kSpreadBit) || head[2] != kSpreadTag || head[1] == 0 ||
      head[1] > (unsigned)kMaxStatusCtas)
    return false;
  *count = head[1];
  return true;
}

}  // namespace dspark

extern "C" {

size_t dspark_kv_workspace_size(void) { return kKvHeaderBytes; }

dspark_status dspark_kv_append(
    const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
    int64_t v_stride, dspark_kv_dtype act_dtype, int64_t n_rows, int B, int Hq, int Hkv, int D,
    const int64_t* row_start, const int32_t* verify_len, const int32_t* cache_len,
    const int32_t* page_table, int max_pages, void* k_cache, void* v_cache, float* k_scale,
    float* v_scale, dspark_kv_dtype cache_dtype, int64_t n_pages, int page_size,
    const float* q_norm, const float* k_norm, float eps, const double* inv_freq, int rot_dim,
    int interleaved, float rope_scale, void* q_out, void* workspace, size_t ws_bytes,
    void* stream) {
  const Common c = {act_dtype, cache_dtype, n_rows,    B,       Hq,      Hkv,     D,
                    row_start, verify_len,  cache_len, page_table, max_pages, k_cache, v_cache,
                    k_scale,   v_scale,     n_pages,   page_size, workspace, ws_bytes,
                    kKvHeaderBytes};
  dspark_status st = check_common(c);
  if (st != DSPARK_OK) return st;
  if (rot_dim < 0 || rot_dim > D || (rot_dim > 0 && !inv_freq) || !std::isfinite(rope_scale) ||
      !(eps >= 0.0f) || !std::isfinite(eps))
    return DSPARK_ERR_INVALID_ARG;
  if (rot_dim % 16 != 0) return DSPARK_ERR_UNSUPPORTED;
  if (q_stride < (int64_t)Hq * D || k_stride < (int64_t)Hkv * D || v_stride < (int64_t)Hkv * D)
    return DSPARK_ERR_INVALID_ARG;
  if (q_stride % 8 || k_stride % 8 || v_stride % 8) return DSPARK_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (B == 0 || n_rows == 0) return no_work(workspace, s);
  if ((st = check_pointers(c)) != DSPARK_OK) return st;
  if (!q || !k || !v || !q_out) return DSPARK_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) ||
      !aligned(q_norm, 16) || !aligned(k_norm, 16) || !aligned(inv_freq, 8))
    return DSPARK_ERR_INVALID_ARG;
  // a block writes its query rows when others may still have to read theirs
  const long long wq = (long long)Hq * D, wk = (long long)Hkv * D;
  const size_t out_bytes = rows_bytes(n_rows, wq, wq);
  const bool in_place = q_out == q && (q_stride == wq || n_rows == 1);
  if ((!in_place && meet(q_out, out_bytes, q, rows_bytes(n_rows, q_stride, wq))) ||
      meet(q_out, out_bytes, k, rows_bytes(n_rows, k_stride, wk)) ||
      meet(q_out, out_bytes, v, rows_bytes(n_rows, v_stride, wk)))
    return DSPARK_ERR_INVALID_ARG;
  LaunchAppend l;
  AppendArgs& a = l.a;
  a.rows = make_rows(c, (int)n_rows);
  a.q = q; a.k = k; a.v = v;
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.k_cache = k_cache; a.v_cache = v_cache;
  a.k_scale = k_scale; a.v_scale = v_scale;
  a.q_norm = q_norm; a.k_norm = k_norm;
  a.inv_freq = inv_freq;
  a.q_out = q_out;
  a.status = static_cast<unsigned*>(workspace);
  a.eps = eps; a.rope_scale = rope_scale;
  a.Hq = Hq; a.Hkv = Hkv; a.rot = rot_dim; a.interleaved = interleaved != 0;
  a.by_hq = make_divisor(Hq);
  a.by_hkv = make_divisor(Hkv);
  l.grid = row_grid(n_rows, 4);
  l.s = s;
  return dispatch(c, l);
}

dspark_status dspark_kv_read(
    const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
    dspark_kv_dtype cache_dtype, int64_t n_pages, int page_size, const int64_t* row_start,
    const int32_t* verify_len, const int32_t* cache_len, const int32_t* page_table, int max_pages,
    int64_t n_rows, int B, int Hkv, int D, void* k_out, void* v_out, dspark_kv_dtype out_dtype,
    void* workspace, size_t ws_bytes, void* stream) {
  const Common c = {out_dtype, cache_dtype, n_rows,    B,       Hkv,     Hkv,     D,
                    row_start, verify_len,  cache_len, page_table, max_pages, k_cache, v_cache,
                    k_scale,   v_scale,     n_pages,   page_size, workspace, ws_bytes,
                    kKvHeaderBytes};
  dspark_status st = check_common(c);
  if (st != DSPARK_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (B == 0 || n_rows == 0) return no_work(workspace, s);
  if ((st = check_pointers(c)) != DSPARK_OK) return st;
  if (!k_out || !v_out || !aligned(k_out, 16) || !aligned(v_out, 16))
    return DSPARK_ERR_INVALID_ARG;
  LaunchRead l;
  ReadArgs& a = l.a;
  a.rows = make_rows(c, (int)n_rows);
  a.k_cache = k_cache; a.v_cache = v_cache;
  a.k_scale = k_scale; a.v_scale = v_scale;
  a.k_out = k_out; a.v_out = v_out;
  a.status = static_cast<unsigned*>(workspace);
  a.Hkv = Hkv;
  l.grid = row_grid(n_rows, 6);
  l.s = s;
  return dispatch(c, l);
}

size_t dspark_attn_workspace_size(int B, int Hq, int Hkv, int D, int max_len) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || D <= 0 || max_len <= 0) return 0;
  return part_bytes(kAttnMaxSms, kChunkRows, D).total;
}

dspark_status dspark_attn_verify(
    const void* q, int64_t q_stride, dspark_kv_dtype act_dtype, int64_t n_rows, int B, int Hq,
    int Hkv, int D, int max_len, const int64_t* row_start, const int32_t* verify_len,
    const int32_t* cache_len, const int32_t* page_table, int max_pages, const void* k_cache,
    const void* v_cache, const float* k_scale, const float* v_scale, dspark_kv_dtype cache_dtype,
    int64_t n_pages, int page_size, float sm_scale, int window, void* out, void* workspace,
    size_t ws_bytes, void* stream) {
  if (max_len < 1 || window < 0) return DSPARK_ERR_INVALID_ARG;
  const Common c = {act_dtype, cache_dtype, n_rows,    B,       Hq,      Hkv,     D,
                    row_start, verify_len,  cache_len, page_table, max_pages, k_cache, v_cache,
                    k_scale,   v_scale,     n_pages,   page_size, workspace, ws_bytes,
                    dspark_attn_workspace_size(B, Hq, Hkv, D, max_len)};
  dspark_status st = check_common(c);
  if (st != DSPARK_OK) return st;
  if (!(sm_scale > 0.0f) || !std::isfinite(sm_scale)) return DSPARK_ERR_INVALID_ARG;
  if (q_stride < (int64_t)Hq * D) return DSPARK_ERR_INVALID_ARG;
  if (q_stride % 8) return DSPARK_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (B == 0 || n_rows == 0) return no_work(workspace, s);
  if ((st = check_pointers(c)) != DSPARK_OK) return st;
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16)) return DSPARK_ERR_INVALID_ARG;
  // a row whose result is not finite is formed again from its query
  const long long width = (long long)Hq * D;
  if (meet(q, rows_bytes(n_rows, q_stride, width), out, rows_bytes(n_rows, width, width)))
    return DSPARK_ERR_INVALID_ARG;
  LaunchAttn l;
  AttnArgs& a = l.a;
  a.rows = make_rows(c, max_len);
  a.q = q;
  a.q_stride = q_stride;
  a.k_cache = k_cache; a.v_cache = v_cache;
  a.k_scale = k_scale; a.v_scale = v_scale;
  a.out = out;
  a.status = static_cast<unsigned*>(workspace);
  a.scale2 = sm_scale * kLog2e;
  a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv;
  a.by_g = make_divisor(a.G);
  a.window = window;
  if (n_rows * Hq >= (1ll << 31)) return DSPARK_ERR_UNSUPPORTED;
  l.rows_per_head = (max_len < n_rows ? max_len : n_rows) * a.G;
  l.cache_rows = n_pages * Hkv * page_size;
  l.page_size = page_size;
  l.D = D;
  l.ws = static_cast<unsigned char*>(workspace);
  l.s = s;
  return dispatch(c, l);
}

}  // extern "C"
