// la_cache_api.cu -- the C entry points of the 8-bit key/value cache: argument
// checks and launches.
#include <cuda_runtime.h>

#include <cmath>

#include "la.h"
#include "la_internal.h"

#define LA_EXPORT extern "C" __attribute__((visibility("default")))

namespace la {
namespace {

constexpr int64_t kMaxCallTokens = 0x7fffffff - 256;  // tokens of a call, in 32 bits

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

struct Range {
  const void* p;
  size_t bytes;
};

bool meets(const Range& a, const Range& b) {
  if (!a.p || !b.p) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.bytes && y < x + a.bytes;
}

// The cache, the table and the sizes that every call has.
la_status check_cache(const la_cache* c, const int32_t* table, int B, int64_t N, int max_pages) {
  if (!c || !c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale || !table)
    return LA_ERR_INVALID_ARG;
  if (B <= 0 || N <= 0 || max_pages <= 0 || c->num_pages <= 0 || c->Hkv <= 0 || c->page <= 0 ||
      c->d <= 0)
    return LA_ERR_INVALID_ARG;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scale, 4) ||
      !aligned(c->v_scale, 4) || !aligned(table, 4))
    return LA_ERR_INVALID_ARG;
  if ((c->d != 64 && c->d != 128) ||
      (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128))
    return LA_ERR_UNSUPPORTED;
  // rows of codes take 32 bits
  if (c->num_pages > 0x7fffffff / c->Hkv / c->page || N > kMaxCallTokens ||
      (int64_t)B * c->Hkv > 0x7fffffff)
    return LA_ERR_INVALID_ARG;
  return LA_OK;
}

void cache_ranges(const la_cache* c, Range (&r)[4]) {
  const size_t heads = (size_t)c->num_pages * c->Hkv, codes = heads * c->page * c->d;
  r[0] = {c->k_codes, codes};
  r[1] = {c->v_codes, codes};
  r[2] = {c->k_scale, heads * 4};
  r[3] = {c->v_scale, heads * 4};
}

size_t dtype_bytes(la_dtype t) { return t == LA_F32 ? 4 : 2; }

// Whether a written range meets another of the call's.
bool any_meets(const Range& w, const Range* r, int n) {
  for (int i = 0; i < n; ++i)
    if (meets(w, r[i])) return true;
  return false;
}

// The page table and lengths of a call.  Kernels read them again as they go, so nothing that
// they write may change them.
void index_ranges(const int32_t* table, const int32_t* len0, const int32_t* len1, int B, int max_pages,
                  Range (&r)[3]) {
  r[0] = {table, (size_t)B * max_pages * 4};
  r[1] = {len0, (size_t)B * 4};
  r[2] = {len1, (size_t)B * 4};
}

la_status check_kv(const la_cache* c, const void* k, const void* v, la_dtype dtype,
                   const int32_t* table, const int32_t* start, const int32_t* count, int B,
                   int64_t N, int max_pages, bool writes_kv) {
  if (!k || !v || !start || !aligned(k, 16) || !aligned(v, 16) || !aligned(start, 4) ||
      !aligned(count, 4))
    return LA_ERR_INVALID_ARG;
  if (dtype != LA_BF16 && dtype != LA_FP16 && dtype != LA_F32) return LA_ERR_INVALID_ARG;
  if (!cache_grid_fits((int64_t)B * c->Hkv, N, c->page, writes_kv)) return LA_ERR_INVALID_ARG;
  Range r[4];
  cache_ranges(c, r);
  const size_t bytes = (size_t)B * c->Hkv * N * c->d * dtype_bytes(dtype);
  const Range kr{k, bytes}, vr{v, bytes};
  if (any_meets(kr, r, 4) || any_meets(vr, r, 4)) return LA_ERR_INVALID_ARG;
  Range index[3];
  index_ranges(table, start, count, B, max_pages, index);
  if (writes_kv) {
    if (meets(kr, vr) || any_meets(kr, index, 3) || any_meets(vr, index, 3)) return LA_ERR_INVALID_ARG;
    return LA_OK;
  }
  for (int i = 0; i < 4; ++i)
    if (any_meets(r[i], r + i + 1, 3 - i) || any_meets(r[i], index, 3)) return LA_ERR_INVALID_ARG;
  return LA_OK;
}

la_status check_attend(const void* q, la_dtype dtype, const la_cache* c, const int32_t* table,
                       const int32_t* kv_len, const int32_t* q_len, const void* o,
                       const float* lse, int B, int Hq, int64_t N, int max_pages, float scale) {
  if (!q || !o || !kv_len) return LA_ERR_INVALID_ARG;
  la_status st = check_cache(c, table, B, N, max_pages);
  if (st != LA_OK) return st;
  if (Hq <= 0 || Hq % c->Hkv != 0 || !std::isfinite(scale)) return LA_ERR_INVALID_ARG;
  if (dtype != LA_BF16 && dtype != LA_FP16 && dtype != LA_F32) return LA_ERR_INVALID_ARG;
  if (dtype == LA_F32 || Hq / c->Hkv > kAttendMaxGroup || B > kAttendMaxBatch)
    return LA_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(kv_len, 4) || !aligned(q_len, 4) ||
      !aligned(lse, 4))
    return LA_ERR_INVALID_ARG;
  Range r[6];
  Range cr[4];
  cache_ranges(c, cr);
  const size_t rows = (size_t)B * Hq * N;
  for (int i = 0; i < 4; ++i) r[i] = cr[i];
  r[4] = {q, rows * c->d * 2};
  r[5] = {lse, rows * 4};
  const Range out{o, rows * c->d * 2};
  if (any_meets(out, r, 6) || any_meets(r[5], r, 5)) return LA_ERR_INVALID_ARG;
  Range index[3];
  index_ranges(table, kv_len, q_len, B, max_pages, index);
  if (any_meets(out, index, 3) || any_meets(r[5], index, 3)) return LA_ERR_INVALID_ARG;
  return LA_OK;
}

la_status from_cuda(cudaError_t e) { return e == cudaSuccess ? LA_OK : LA_ERR_CUDA; }

// An attention call with its arguments checked.
la_status run_attend(const void* q, la_dtype dtype, const la_cache* c, const int32_t* table,
                     const int32_t* kv_len, const int32_t* q_len, void* o, float* lse, int B,
                     int Hq, int64_t N, int max_pages, float scale, void* workspace,
                     cudaStream_t stream) {
  unsigned* status = device_status_ptr();
  const int sms = device_sms();
  if (!status || sms <= 0) return LA_ERR_CUDA;
  return from_cuda(launch_cache_attend(*c, q, dtype, table, kv_len, q_len, o, lse, B, Hq, N,
                                       max_pages, scale, workspace, status, sms, stream));
}

}  // namespace
}  // namespace la

using namespace la;

LA_EXPORT la_status la_cache_write(const void* k, const void* v, la_dtype dtype,
                                   const la_cache* cache, const int32_t* table,
                                   const int32_t* start, const int32_t* count, int B, int64_t N,
                                   int max_pages, la_stream stream) {
  la_status st = check_cache(cache, table, B, N, max_pages);
  if (st == LA_OK) st = check_kv(cache, k, v, dtype, table, start, count, B, N, max_pages, false);
  if (st != LA_OK) return st;
  unsigned* status = device_status_ptr();
  if (!status) return LA_ERR_CUDA;
  return from_cuda(launch_cache_write(k, v, dtype, *cache, table, start, count, B, N, max_pages,
                                      status, static_cast<cudaStream_t>(stream)));
}

LA_EXPORT la_status la_cache_read(const la_cache* cache, const int32_t* table,
                                  const int32_t* start, const int32_t* count, void* k, void* v,
                                  la_dtype dtype, int B, int64_t N, int max_pages,
                                  la_stream stream) {
  la_status st = check_cache(cache, table, B, N, max_pages);
  if (st == LA_OK) st = check_kv(cache, k, v, dtype, table, start, count, B, N, max_pages, true);
  if (st != LA_OK) return st;
  unsigned* status = device_status_ptr();
  const int sms = device_sms();
  if (!status || sms <= 0) return LA_ERR_CUDA;
  return from_cuda(launch_cache_read(*cache, table, start, count, k, v, dtype, B, N, max_pages,
                                     status, sms, static_cast<cudaStream_t>(stream)));
}

LA_EXPORT size_t la_cache_attend_workspace_bytes(int B, int Hq, int Hkv, int64_t N, int d) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || N <= 0 || (d != 64 && d != 128)) return 0;
  if (Hq / Hkv > kAttendMaxGroup || B > kAttendMaxBatch || N > kMaxCallTokens ||
      (int64_t)B * Hkv > 0x7fffffff)
    return 0;
  const int sms = device_sms();
  return sms > 0 ? attend_workspace_bytes(B, Hq, Hkv, N, d, sms) : 0;
}

LA_EXPORT la_status la_cache_attend_ws(const void* q, la_dtype dtype, const la_cache* cache,
                                       const int32_t* table, const int32_t* kv_len,
                                       const int32_t* q_len, void* o, float* lse, int B, int Hq,
                                       int64_t N, int max_pages, float scale, void* workspace,
                                       size_t workspace_bytes, la_stream stream) {
  const la_status st = check_attend(q, dtype, cache, table, kv_len, q_len, o, lse, B, Hq, N,
                                    max_pages, scale);
  if (st != LA_OK) return st;
  const size_t need = la_cache_attend_workspace_bytes(B, Hq, cache->Hkv, N, cache->d);
  if (need == 0) return LA_ERR_CUDA;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return LA_ERR_WORKSPACE;
  Range r[4];
  cache_ranges(cache, r);
  Range index[3];
  index_ranges(table, kv_len, q_len, B, max_pages, index);
  const Range w{workspace, need};
  const size_t rows = (size_t)B * Hq * N;
  if (any_meets(w, r, 4) || any_meets(w, index, 3) || meets(w, {q, rows * cache->d * 2}) ||
      meets(w, {o, rows * cache->d * 2}) || meets(w, {lse, rows * 4}))
    return LA_ERR_WORKSPACE;
  return run_attend(q, dtype, cache, table, kv_len, q_len, o, lse, B, Hq, N, max_pages, scale,
                    workspace, static_cast<cudaStream_t>(stream));
}

LA_EXPORT la_status la_cache_attend(const void* q, la_dtype dtype, const la_cache* cache,
                                    const int32_t* table, const int32_t* kv_len,
                                    const int32_t* q_len, void* o, float* lse, int B, int Hq,
                                    int64_t N, int max_pages, float scale, la_stream stream) {
  la_status st = check_attend(q, dtype, cache, table, kv_len, q_len, o, lse, B, Hq, N, max_pages,
                              scale);
  if (st != LA_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int sms = device_sms();
  if (sms <= 0) return LA_ERR_CUDA;
  if (!attend_uses_workspace(B, cache->Hkv, Hq / cache->Hkv, N, cache->d,
                             (int64_t)max_pages * cache->page, sms))
    return run_attend(q, dtype, cache, table, kv_len, q_len, o, lse, B, Hq, N, max_pages, scale,
                      nullptr, s);
  const size_t bytes = la_cache_attend_workspace_bytes(B, Hq, cache->Hkv, N, cache->d);
  if (bytes == 0 || !keep_pool_memory()) return LA_ERR_CUDA;
  void* ws = nullptr;
  if (cudaMallocAsync(&ws, bytes, s) != cudaSuccess) return LA_ERR_CUDA;
  st = run_attend(q, dtype, cache, table, kv_len, q_len, o, lse, B, Hq, N, max_pages, scale, ws, s);
  if (cudaFreeAsync(ws, s) != cudaSuccess && st == LA_OK) st = LA_ERR_CUDA;
  return st;
}
