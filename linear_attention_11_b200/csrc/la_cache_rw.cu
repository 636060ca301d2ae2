// la_cache_rw.cu -- storing tokens in the 8-bit key/value cache and reading
// them back.
//
// For a page's new tokens x of one kv head (page x d numbers at most):
//     e     = least e >= -126 with max |x| <= 448 * 2^e  (and 2^e >= the page's
//             scale, if it already holds tokens)
//     code  = e4m3(x * 2^-e)            x * 2^-e is exact in fp32 (or too small
//                                       for any code)
// Both directions only move bytes: 2 (or 4) in and 1 out for a value, or the
// reverse, so HBM bounds them for prompts and latency for single tokens.
#include <cuda_runtime.h>

#include "la_cache.cuh"

namespace la {
namespace {

struct CacheWriteParams {
  const void* x[2];   // k, v [B, Hkv, N, d]
  uint8_t* codes[2];  // [num_pages, Hkv, page, d]
  float* scale[2];    // [num_pages, Hkv]
  const int* table;   // [B, max_pages]
  const int* start;   // [B]
  const int* count;   // [B] or null (N everywhere)
  unsigned* status;
  int64_t N, num_pages;
  int B, Hkv, max_pages, page, page_log2;
  int spans;          // pages that N tokens of one sequence can touch
};

// Rounds the first `rows` rows of a page to a larger scale: codes * ratio,
// `n` threads from thread t on.
template <int D>
__device__ __forceinline__ void rescale_rows(uint8_t* codes, int rows, float ratio, int t, int n) {
  for (int i = t; i < rows * (D / 4); i += n) {
    uint32_t* p = reinterpret_cast<uint32_t*>(codes) + i;
    const uint32_t w = *p;
    const uint32_t a = e4m3x2_to_f16x2(w & 0xffffu), b = e4m3x2_to_f16x2(w >> 16);
    const float2 lo = unpack2<__half>(a), hi = unpack2<__half>(b);
    *p = f32x2_to_e4m3x2(lo.x * ratio, lo.y * ratio) |
         (f32x2_to_e4m3x2(hi.x * ratio, hi.y * ratio) << 16);
  }
}

// Non-finite numbers out (a NaN to zero, an infinity kept for the saturating
// conversion); amax over the finite ones; true if there were any.
__device__ __forceinline__ bool sift8(float (&x)[8], float& amax) {
  bool odd = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = fabsf(x[i]);
    const bool finite = a < __int_as_float(0x7f800000);
    amax = fmaxf(amax, finite ? a : 0.f);
    odd |= !finite;
    x[i] = x[i] == x[i] ? x[i] : 0.f;
  }
  return odd;
}

__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv) {
  uint2 w;
  w.x = f32x2_to_e4m3x2(x[0] * inv, x[1] * inv) | (f32x2_to_e4m3x2(x[2] * inv, x[3] * inv) << 16);
  w.y = f32x2_to_e4m3x2(x[4] * inv, x[5] * inv) | (f32x2_to_e4m3x2(x[6] * inv, x[7] * inv) << 16);
  return w;
}

// One group of threads per (sequence, kv head, touched page, k or v): WARP, a
// warp for calls of at most kFewTokens tokens; else a block of page * D / 32
// threads, 32 values each in four vectors of eight.  The new tokens stay in
// registers between the maximum and the rounding, so each is read once.
constexpr int kFewTokens = 4;

template <typename T, int D, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 512)
    cache_write_kernel(const CacheWriteParams p) {
  constexpr int kVecs = 4;        // vectors of eight values a thread holds at most
  constexpr int TPR = D / 8;      // threads that cover a row
  const int lane = threadIdx.x & 31;
  const int nthreads = WARP ? 32 : (int)blockDim.x;
  const int t = WARP ? lane : (int)threadIdx.x;
  const int64_t unit = WARP ? (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  const int which = blockIdx.y;
  const int64_t bh = unit / p.spans;
  if (WARP && bh >= (int64_t)p.B * p.Hkv) return;
  const int s = (int)(unit % p.spans);
  const int b = (int)(bh / p.Hkv), h = (int)(bh % p.Hkv);

  const int64_t start = p.start[b], count = p.count ? (int64_t)p.count[b] : p.N;
  if (!token_range_ok(start, count, p.N, (int64_t)p.max_pages << p.page_log2, p.status)) return;
  const int64_t block = (start >> p.page_log2) + s;  // page of the sequence
  const int64_t first = block << p.page_log2;        // its first token
  const int64_t lo = max(start, first), hi = min(start + count, first + p.page);
  if (lo >= hi) return;
  const int held = (int)(lo - first), rows = (int)(hi - lo);  // older rows, new rows
  const int at = p.table[(int64_t)b * p.max_pages + block];
  const bool known = at >= 0 && at < p.num_pages;

  const T* src = static_cast<const T*>(p.x[which]) + ((int64_t)bh * p.N + (lo - start)) * D;
  float x[kVecs][8];
  float amax = 0.f;
  bool odd = false;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int r = (i * nthreads + t) / TPR, c = (i * nthreads + t) % TPR;
    if (r < rows) load8<T>(src + (int64_t)r * D + c * 8, x[i]);
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    if ((i * nthreads + t) / TPR < rows) odd |= sift8(x[i], amax);
  }
  if (odd) atomicOr(p.status, kDevNonfinite);
  if (!known) {
    if (t == 0) atomicOr(p.status, kDevBadIndex);
    return;  // the whole group: `at` is the group's
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
  float* scale_at = p.scale[which] + (int64_t)at * p.Hkv + h;
  const float old = held ? *scale_at : 0.f;
  if (!WARP) {
    __shared__ float part[16];
    if (lane == 0) part[threadIdx.x >> 5] = amax;
    __syncthreads();  // also: every thread has read the old scale
    amax = part[(lane & 15) < nthreads / 32 ? lane & 15 : 0];
#pragma unroll
    for (int m = 8; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
  } else {
    __syncwarp();
  }
  int e = scale_exponent(amax);
  float scale = pow2i(e);
  float inv = pow2i(-e);
  if (old > scale) {  // the older tokens' scale holds the new ones too
    scale = old;
    inv = 1.0f / old;  // exact: a power of two
  }
  if (t == 0 && scale != old) *scale_at = scale;
  uint8_t* page_codes = p.codes[which] + ((int64_t)at * p.Hkv + h) * p.page * D;
  if (held && scale > old) rescale_rows<D>(page_codes, held, old / scale, t, nthreads);
  uint8_t* dst = page_codes + held * D;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int r = (i * nthreads + t) / TPR, c = (i * nthreads + t) % TPR;
    if (r < rows) *reinterpret_cast<uint2*>(dst + r * D + c * 8) = codes8(x[i], inv);
  }
}

struct CacheReadParams {
  const uint8_t* codes[2];
  const float* scale[2];
  void* x[2];
  const int* table;
  const int* start;
  const int* count;
  unsigned* status;
  int64_t N, num_pages;
  int Hkv, max_pages, page_log2;
  int blocks;  // blocks of kReadRows * 256 / (d / 8) tokens for one sequence and head
};

// Eight codes a thread and step, kReadRows steps: a warp reads rows of codes
// and writes rows of values whole; the steps' loads are in flight together.
constexpr int kReadRows = 4;

template <typename T, int D>
__global__ void __launch_bounds__(256) cache_read_kernel(const CacheReadParams p) {
  constexpr int TPR = D / 8;
  constexpr int RPS = 256 / TPR;  // rows a step
  const int which = blockIdx.y;
  const int64_t bh = blockIdx.x / p.blocks;
  const int64_t row0 = (int64_t)(blockIdx.x % p.blocks) * (RPS * kReadRows);
  const int b = (int)(bh / p.Hkv), h = (int)(bh % p.Hkv);
  const int64_t start = p.start[b], count = p.count ? (int64_t)p.count[b] : p.N;
  if (!token_range_ok(start, count, p.N, (int64_t)p.max_pages << p.page_log2, p.status)) return;
  if (row0 >= count) return;
  const int c = threadIdx.x % TPR;
  const int mask = (1 << p.page_log2) - 1;
  uint2 w[kReadRows];
  float scale[kReadRows];
  int64_t at[kReadRows];
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    const int64_t r = row0 + i * RPS + threadIdx.x / TPR;
    at[i] = r < count ? p.table[(int64_t)b * p.max_pages + ((start + r) >> p.page_log2)] : -1;
    if (r < count && (at[i] < 0 || at[i] >= p.num_pages)) {
      atomicOr(p.status, kDevBadIndex);
      at[i] = -1;
    }
  }
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    const int64_t r = row0 + i * RPS + threadIdx.x / TPR;
    w[i] = make_uint2(0u, 0u);
    scale[i] = 0.f;
    if (at[i] >= 0) {
      const int64_t ph = at[i] * p.Hkv + h;
      scale[i] = __ldg(p.scale[which] + ph);
      w[i] = __ldcs(reinterpret_cast<const uint2*>(
          p.codes[which] + ((ph << p.page_log2) + ((start + r) & mask)) * D + c * 8));
    }
  }
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    const int64_t r = row0 + i * RPS + threadIdx.x / TPR;
    if (r >= count) continue;
    float x[8];
    const uint32_t pair[4] = {w[i].x & 0xffffu, w[i].x >> 16, w[i].y & 0xffffu, w[i].y >> 16};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack2<__half>(e4m3x2_to_f16x2(pair[j]));
      x[2 * j] = f.x * scale[i];
      x[2 * j + 1] = f.y * scale[i];
    }
    store8<T>(static_cast<T*>(p.x[which]) + ((int64_t)bh * p.N + r) * D + c * 8, x);
  }
}

template <typename T, int D>
cudaError_t write_typed(const CacheWriteParams& p, int64_t groups, cudaStream_t stream) {
  if (p.N <= kFewTokens) {
    const int64_t grid = (groups + 7) / 8;
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    cache_write_kernel<T, D, true><<<dim3((unsigned)grid, 2), 256, 0, stream>>>(p);
  } else {
    if (groups > 0x7fffffff) return cudaErrorInvalidValue;
    cache_write_kernel<T, D, false>
        <<<dim3((unsigned)groups, 2), p.page * D / 32, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t read_typed(CacheReadParams p, int64_t bh, cudaStream_t stream) {
  const int64_t per = (int64_t)kReadRows * 256 / (D / 8);
  const int64_t blocks = (p.N + per - 1) / per;
  if (blocks * bh > 0x7fffffff) return cudaErrorInvalidValue;
  p.blocks = (int)blocks;
  cache_read_kernel<T, D><<<dim3((unsigned)(blocks * bh), 2), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_write(const void* k, const void* v, la_dtype dtype, const la_cache& c,
                               const int32_t* table, const int32_t* start, const int32_t* count,
                               int B, int64_t N, int max_pages, unsigned* status,
                               cudaStream_t stream) {
  CacheWriteParams p{{k, v}, {c.k_codes, c.v_codes}, {c.k_scale, c.v_scale}, table, start, count,
                     status, N, c.num_pages, B, c.Hkv, max_pages, c.page, page_log2(c.page), 0};
  // N tokens in a row from any place in a page: 1 + ceil((N - 1) / page) pages
  const int64_t spans = 1 + (N - 1 + c.page - 1) / c.page;
  if (spans > 0x7fffffff) return cudaErrorInvalidValue;
  p.spans = (int)spans;
  const int64_t groups = spans * B * c.Hkv;
  if (c.d == 64) {
    if (dtype == LA_BF16) return write_typed<__nv_bfloat16, 64>(p, groups, stream);
    if (dtype == LA_FP16) return write_typed<__half, 64>(p, groups, stream);
    return write_typed<float, 64>(p, groups, stream);
  }
  if (dtype == LA_BF16) return write_typed<__nv_bfloat16, 128>(p, groups, stream);
  if (dtype == LA_FP16) return write_typed<__half, 128>(p, groups, stream);
  return write_typed<float, 128>(p, groups, stream);
}

cudaError_t launch_cache_read(const la_cache& c, const int32_t* table, const int32_t* start,
                              const int32_t* count, void* k, void* v, la_dtype dtype, int B,
                              int64_t N, int max_pages, unsigned* status, cudaStream_t stream) {
  CacheReadParams p{{c.k_codes, c.v_codes}, {c.k_scale, c.v_scale}, {k, v}, table, start, count,
                    status, N, c.num_pages, c.Hkv, max_pages, page_log2(c.page), 0};
  const int64_t bh = (int64_t)B * c.Hkv;
  if (c.d == 64) {
    if (dtype == LA_BF16) return read_typed<__nv_bfloat16, 64>(p, bh, stream);
    if (dtype == LA_FP16) return read_typed<__half, 64>(p, bh, stream);
    return read_typed<float, 64>(p, bh, stream);
  }
  if (dtype == LA_BF16) return read_typed<__nv_bfloat16, 128>(p, bh, stream);
  if (dtype == LA_FP16) return read_typed<__half, 128>(p, bh, stream);
  return read_typed<float, 128>(p, bh, stream);
}

}  // namespace la
