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

#include <algorithm>

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
    uint32_t a, b;
    e4m3x4_to_f16x4(w, a, b);
    const float2 lo = unpack2<__half>(a), hi = unpack2<__half>(b);
    *p = f32x2_to_e4m3x2(lo.x * ratio, lo.y * ratio) |
         (f32x2_to_e4m3x2(hi.x * ratio, hi.y * ratio) << 16);
  }
}

// Eight values of the input as loaded.  Of bf16 and fp16 the magnitudes are
// compared two at a time, as they are; a NaN stays in the maximum, so one look at
// the maximum of a whole page tells whether there is anything but finite numbers.
template <typename T>
struct Raw8 {
  uint4 w;
  __device__ __forceinline__ void load(const T* p) { w = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void clear() { w = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void max_into(uint32_t& m) const {
    m = max2(max2(max2(m, w.x), max2(0u, w.y)), max2(max2(0u, w.z), w.w));
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b);
  static __device__ __forceinline__ float top(uint32_t m) {
    const float2 f = unpack2<T>(m);
    return max_nan(f.x, f.y);
  }
  static __device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
  }
  __device__ __forceinline__ void unpack(float (&x)[8]) const {
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<T>(r[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
};
template <>
__device__ __forceinline__ uint32_t Raw8<__nv_bfloat16>::max2(uint32_t a, uint32_t b) {
  b &= 0x7fff7fffu;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
  return a;
}
template <>
__device__ __forceinline__ uint32_t Raw8<__half>::max2(uint32_t a, uint32_t b) {
  b &= 0x7fff7fffu;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
  return a;
}
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  static __device__ __forceinline__ float max_nan(float x, float y) {  // x >= 0
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(fabsf(y)));
    return r;
  }
  __device__ __forceinline__ void max_into(uint32_t& m) const {
    const float p = max_nan(max_nan(max_nan(__uint_as_float(m), a.x), a.y), max_nan(max_nan(0.f, a.z), a.w));
    m = __float_as_uint(max_nan(p, max_nan(max_nan(max_nan(0.f, b.x), b.y), max_nan(max_nan(0.f, b.z), b.w))));
  }
  static __device__ __forceinline__ float top(uint32_t m) { return __uint_as_float(m); }
  __device__ __forceinline__ void unpack(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
};

__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv) {
  uint2 w;
  w.x = f32x2_to_e4m3x2(x[0] * inv, x[1] * inv) | (f32x2_to_e4m3x2(x[2] * inv, x[3] * inv) << 16);
  w.y = f32x2_to_e4m3x2(x[4] * inv, x[5] * inv) | (f32x2_to_e4m3x2(x[6] * inv, x[7] * inv) << 16);
  return w;
}

// One group of threads per (sequence, kv head, touched page, k or v): WARP, a
// warp for calls of at most kFewTokens tokens; else a block whose threads hold
// kVecs vectors of eight values each.  The new tokens stay in registers between the
// maximum and the rounding, so each is read once.  (Four vectors a thread of the
// 16-bit types, 535 instructions a warp: 192 us for 32768 tokens of 32 heads,
// page 64; eight: 140 us.)
constexpr int kFewTokens = 4;

template <typename T>
constexpr int block_vecs() {
  return sizeof(T) == 2 ? 8 : 4;
}

template <typename T, int D, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 512)
    cache_write_kernel(const CacheWriteParams p) {
  constexpr int kVecs = WARP ? kFewTokens * D / 256 : block_vecs<T>();
  constexpr int TPR = D / 8;      // threads that cover a row
  const int lane = threadIdx.x & 31;
  const int nthreads = WARP ? 32 : (int)blockDim.x;
  const int t = WARP ? lane : (int)threadIdx.x;
  const uint32_t unit = WARP ? blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;  // < 2^31
  const int which = blockIdx.y;
  const uint32_t bh = unit / (uint32_t)p.spans;
  if (WARP && bh >= (uint32_t)p.B * (uint32_t)p.Hkv) return;
  const int s = (int)(unit - bh * p.spans);
  const int b = (int)(bh / (uint32_t)p.Hkv), h = (int)(bh - (uint32_t)b * p.Hkv);

  const int64_t start = p.start[b], count = p.count ? (int64_t)p.count[b] : p.N;
  if (!token_range_ok(start, count, p.N, token_limit(p.max_pages, p.page_log2), p.status)) return;
  const int64_t block = (start >> p.page_log2) + s;  // page of the sequence
  const int64_t first = block << p.page_log2;        // its first token
  const int64_t lo = max(start, first), hi = min(start + count, first + p.page);
  if (lo >= hi) return;
  const int held = (int)(lo - first), rows = (int)(hi - lo);  // older rows, new rows
  const int at = p.table[(int64_t)b * p.max_pages + block];
  const bool known = at >= 0 && at < p.num_pages;

  const T* src = static_cast<const T*>(p.x[which]) + ((int64_t)bh * p.N + (lo - start)) * D;
  Raw8<T> x[kVecs];
  uint32_t packed = 0u;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int r = (i * nthreads + t) / TPR, c = (i * nthreads + t) % TPR;
    if (r < rows) x[i].load(src + (int64_t)r * D + c * 8);
    else x[i].clear();
  }
  float* scale_at = p.scale[which] + (int64_t)at * p.Hkv + h;
  const float old = held && known ? *scale_at : 0.f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) x[i].max_into(packed);
  if (!known) {
    if (t == 0) atomicOr(p.status, kDevBadIndex);
    return;  // the whole group: `at` is the group's
  }
  // the largest of the group's, NaN if there is one (also: every thread has read
  // the old scale when this returns)
  __shared__ float part[16];
  auto group_max = [&](float v) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1)
      v = Raw8<float>::max_nan(v, __shfl_xor_sync(0xffffffffu, v, m));
    if (!WARP && nthreads > 32) {
      if (lane == 0) part[threadIdx.x >> 5] = v;
      __syncthreads();
      v = part[(lane & 15) < nthreads / 32 ? lane & 15 : 0];
#pragma unroll
      for (int m = 8; m > 0; m >>= 1)
        v = Raw8<float>::max_nan(v, __shfl_xor_sync(0xffffffffu, v, m));
    }
    return v;
  };
  float amax = group_max(Raw8<T>::top(packed));
  const bool finite = amax < __int_as_float(0x7f800000);
  if (!finite) {
    // infinities and NaN: the maximum of the others
    if (t == 0) atomicOr(p.status, kDevNonfinite);
    amax = 0.f;
    for (int i = 0; i < kVecs; ++i) {
      float f[8];
      x[i].unpack(f);
      for (int j = 0; j < 8; ++j) {
        const float a = fabsf(f[j]);
        if (a < __int_as_float(0x7f800000)) amax = fmaxf(amax, a);
      }
    }
    if (!WARP) __syncthreads();  // `part` has been read
    amax = group_max(amax);
  }
  const int e = scale_exponent(amax);
  float scale = pow2i(e);
  float inv = pow2i(-e);
  if (old > scale) {  // the older tokens' scale holds the new ones too
    scale = old;
    inv = 1.0f / old;  // exact: a power of two
  }
  __syncwarp();
  if (t == 0 && scale != old) *scale_at = scale;
  uint8_t* page_codes = p.codes[which] + ((int64_t)at * p.Hkv + h) * p.page * D;
  if (held && scale > old) rescale_rows<D>(page_codes, held, old / scale, t, nthreads);
  uint8_t* dst = page_codes + held * D;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int r = (i * nthreads + t) / TPR, c = (i * nthreads + t) % TPR;
    if (r >= rows) continue;
    float f[8];
    x[i].unpack(f);
    if (!finite)  // a NaN is stored as zero; the conversion saturates infinities
      for (int j = 0; j < 8; ++j) f[j] = f[j] == f[j] ? f[j] : 0.f;
    *reinterpret_cast<uint2*>(dst + r * D + c * 8) = codes8(f, inv);
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
  int blocks;   // runs of ROWS tokens for one sequence and head
  uint32_t bh;  // B * Hkv
};

// A warp takes ROWS tokens in a row: its first lanes look up their pages and
// scales (at most five pages), then 16 codes a lane and step, all steps' loads of
// half the rows in flight together.  (Eight codes a lane and a page lookup for every
// row: 225 us for 131072 tokens of 8 heads, waiting for the chain of start, table
// and codes; this one 152 us.)
constexpr int kReadRows = 64, kReadRowsFew = 16;

template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(256) cache_read_kernel(const CacheReadParams p) {
  constexpr int PIECES = D / 16;           // lanes that cover a row
  constexpr int RPS = 32 / PIECES;         // rows a step
  constexpr int STEPS = ROWS / RPS / 2;
  const int lane = threadIdx.x & 31;
  const uint32_t unit = blockIdx.x * 8 + (threadIdx.x >> 5);  // < 2^31
  const int which = blockIdx.y;
  const uint32_t bh = unit / (uint32_t)p.blocks;
  if (bh >= p.bh) return;
  const int64_t row0 = (int64_t)(unit - bh * p.blocks) * ROWS;
  const int b = (int)(bh / (uint32_t)p.Hkv), h = (int)(bh - (uint32_t)b * p.Hkv);
  const int64_t start = p.start[b], count = p.count ? (int64_t)p.count[b] : p.N;
  if (!token_range_ok(start, count, p.N, token_limit(p.max_pages, p.page_log2), p.status)) return;
  if (row0 >= count) return;
  const int rows = (int)min((int64_t)ROWS, count - row0);
  const int tok0 = (int)(start + row0), page0 = tok0 >> p.page_log2;
  const int pages = ((tok0 + rows - 1) >> p.page_log2) - page0 + 1;  // <= 5
  int first = -1;      // lane k: first row of codes of page page0 + k
  float scale = 0.f;
  if (lane < pages) {
    const int id = p.table[(int64_t)b * p.max_pages + page0 + lane];
    if (id >= 0 && id < p.num_pages) {
      first = (int)(((int64_t)id * p.Hkv + h) << p.page_log2);
      scale = __ldg(p.scale[which] + (int64_t)id * p.Hkv + h);
    } else {
      atomicOr(p.status, kDevBadIndex);
    }
  }
  const int piece = lane % PIECES, sub = lane / PIECES, mask = (1 << p.page_log2) - 1;
  T* out = static_cast<T*>(p.x[which]) + ((int64_t)bh * p.N + row0) * D + piece * 16;
  const uint8_t* codes = p.codes[which] + piece * 16;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint4 w[STEPS];
    float f[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int r = (half * STEPS + i) * RPS + sub, tok = tok0 + r;
      const int k = (tok >> p.page_log2) - page0;
      const int at = __shfl_sync(0xffffffffu, first, k & 31);
      f[i] = __shfl_sync(0xffffffffu, scale, k & 31);
      w[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows && at >= 0)
        w[i] = __ldcs(reinterpret_cast<const uint4*>(codes + (int64_t)(at + (tok & mask)) * D));
    }
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int r = (half * STEPS + i) * RPS + sub;
      if (r >= rows) continue;
      const uint32_t c[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float x[8];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t a, b;
          e4m3x4_to_f16x4(c[2 * j + k], a, b);
          const float2 lo = unpack2<__half>(a), hi = unpack2<__half>(b);
          x[4 * k] = lo.x * f[i];
          x[4 * k + 1] = lo.y * f[i];
          x[4 * k + 2] = hi.x * f[i];
          x[4 * k + 3] = hi.y * f[i];
        }
        store8<T>(out + (int64_t)r * D + j * 8, x);
      }
    }
  }
}

constexpr int64_t kMaxGroups = 0x7ffffff0;  // blocks, or warps, of a call's grid

// Pages that N tokens in a row from any place in a page can touch.
int64_t spans_of(int64_t N, int page) { return 1 + (N - 1 + page - 1) / page; }

template <typename T, int D>
cudaError_t write_typed(const CacheWriteParams& p, int64_t groups, cudaStream_t stream) {
  if (p.N <= kFewTokens) {
    cache_write_kernel<T, D, true><<<dim3((unsigned)((groups + 7) / 8), 2), 256, 0, stream>>>(p);
  } else {
    cache_write_kernel<T, D, false>
        <<<dim3((unsigned)groups, 2), std::max(32, p.page * D / (8 * block_vecs<T>())), 0, stream>>>(p);
  }
  return cudaGetLastError();
}

template <typename T, int D, int ROWS>
cudaError_t read_rows(CacheReadParams p, int64_t bh, cudaStream_t stream) {
  const int64_t blocks = (p.N + ROWS - 1) / ROWS, units = blocks * bh;
  p.blocks = (int)blocks;
  p.bh = (uint32_t)bh;
  cache_read_kernel<T, D, ROWS><<<dim3((unsigned)((units + 7) / 8), 2), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

// Short runs where long ones would not give every SM its 32 warps (B 7, 2 heads, up
// to 1000 tokens, fp32: 5.9 us against 8.0 us).
template <typename T, int D>
cudaError_t read_typed(CacheReadParams p, int64_t bh, int sms, cudaStream_t stream) {
  const int64_t warps = 2 * bh * ((p.N + kReadRows - 1) / kReadRows);
  return warps < 32 * sms ? read_rows<T, D, kReadRowsFew>(p, bh, stream)
                          : read_rows<T, D, kReadRows>(p, bh, stream);
}

}  // namespace

// (a read that takes short runs has few of them)
bool cache_grid_fits(int64_t bh, int64_t N, int page, bool read) {
  return (read ? (N + kReadRows - 1) / kReadRows : spans_of(N, page)) <= kMaxGroups / bh;
}

cudaError_t launch_cache_write(const void* k, const void* v, la_dtype dtype, const la_cache& c,
                               const int32_t* table, const int32_t* start, const int32_t* count,
                               int B, int64_t N, int max_pages, unsigned* status,
                               cudaStream_t stream) {
  CacheWriteParams p{{k, v}, {c.k_codes, c.v_codes}, {c.k_scale, c.v_scale}, table, start, count,
                     status, N, c.num_pages, B, c.Hkv, max_pages, c.page, page_log2(c.page), 0};
  p.spans = (int)spans_of(N, c.page);
  const int64_t groups = (int64_t)p.spans * B * c.Hkv;
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
                              int64_t N, int max_pages, unsigned* status, int sms,
                              cudaStream_t stream) {
  CacheReadParams p{{c.k_codes, c.v_codes}, {c.k_scale, c.v_scale}, {k, v}, table, start, count,
                    status, N, c.num_pages, c.Hkv, max_pages, page_log2(c.page), 0, 0};
  const int64_t bh = (int64_t)B * c.Hkv;
  if (c.d == 64) {
    if (dtype == LA_BF16) return read_typed<__nv_bfloat16, 64>(p, bh, sms, stream);
    if (dtype == LA_FP16) return read_typed<__half, 64>(p, bh, sms, stream);
    return read_typed<float, 64>(p, bh, sms, stream);
  }
  if (dtype == LA_BF16) return read_typed<__nv_bfloat16, 128>(p, bh, sms, stream);
  if (dtype == LA_FP16) return read_typed<__half, 128>(p, bh, sms, stream);
  return read_typed<float, 128>(p, bh, sms, stream);
}

}  // namespace la
