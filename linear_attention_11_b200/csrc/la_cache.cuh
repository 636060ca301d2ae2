// la_cache.cuh -- what the kernels of the 8-bit key/value cache share: the view
// of a cache that a launch gets, e4m3 conversions, the sequence lengths.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include <atomic>

#include "la_internal.h"

namespace la {

constexpr unsigned kDevBadIndex = 0x2u;   // LA_DEV_BAD_INDEX
constexpr unsigned kDevNonfinite = 0x4u;  // LA_DEV_NONFINITE

struct AttendParams;
struct JoinGeometry;
cudaError_t launch_cache_token(const AttendParams& p, const la_cache& c, la_dtype dtype, int rows,
                               int ctas, bool whole, cudaStream_t stream);
cudaError_t launch_cache_prompt(const AttendParams& p, la_dtype dtype, int d, int ctas, bool whole,
                                cudaStream_t stream);
cudaError_t launch_cache_join(const AttendParams& p, const JoinGeometry& g, la_dtype dtype, int d,
                              int ctas, cudaStream_t stream);

// Lets a kernel use `bytes` of shared memory on the current device, once for each.
template <auto kKernel>
cudaError_t allow_shared(int bytes) {
  static std::atomic<uint64_t> done{0};  // bit for each device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

inline int page_log2(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7; }

// ---------------------------------------------------------------- types
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&w));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<__half2*>(&w));
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// Eight consecutive values, rounded to type T; p is aligned to their size (16 bytes,
// or twice that for fp32).
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  uint4 w;
  w.x = pack2<T>(x[0], x[1]);
  w.y = pack2<T>(x[2], x[3]);
  w.z = pack2<T>(x[4], x[5]);
  w.w = pack2<T>(x[6], x[7]);
  __stcs(reinterpret_cast<uint4*>(p), w);
}
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&x)[8]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
}

// ---------------------------------------------------------------- e4m3
// Four codes (low byte first) as two f16x2, exactly: f16 has e4m3's numbers.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}

// Two fp32 numbers as codes, rounded to nearest even (|x| <= 448 here).
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Exponent of the scale for values of magnitude up to amax (finite, >= 0): the
// least e >= -126 with amax <= 448 * 2^e = 1.75 * 2^(e + 8).
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, -126);
}

__device__ __forceinline__ float pow2i(int e) {  // 2^e, -126 <= e <= 127
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// ---------------------------------------------------------------- lengths
// Tokens that a sequence can have: its pages', and no more than leave the sums of a
// token and a tile in 32 bits.
__device__ __forceinline__ int64_t token_limit(int max_pages, int page_log2) {
  return min((int64_t)max_pages << page_log2, (int64_t)0x7fff0000);
}

// Tokens [first, first + n) of a sequence: false (and the status bit) when they
// do not lie in [0, limit); n = 0 is always well.
__device__ __forceinline__ bool token_range_ok(int64_t first, int64_t n, int64_t nmax,
                                               int64_t limit, unsigned* status) {
  if (n == 0) return true;
  const bool ok = n > 0 && n <= nmax && first >= 0 && first + n <= limit;
  if (!ok) atomicOr(status, kDevBadIndex);
  return ok;
}

// One attention call as its kernels get it.
struct AttendParams {
  const void* q;            // [B, Hq, N, d]
  const uint8_t* codes[2];  // k, v [num_pages, Hkv, page, d]
  const float* kvscale[2];  // [num_pages, Hkv]
  const int* table;         // [B, max_pages]
  const int* kv_len;        // [B]
  const int* q_len;         // [B] or null (N everywhere)
  void* o;
  float* lse;               // [B, Hq, N] or null
  unsigned* status;
  int64_t N, num_pages;
  int B, Hq, Hkv, G, max_pages, page_log2;
  float scale;
  float* parts;             // workspace: [ctas][2] parts of rows x (d + kPartStats) floats
  int4* tails;              // workspace: [ctas], see below
};

// Whether a sequence's lengths lie in range; if not the sequence is left out.
__device__ __forceinline__ bool attend_lengths_ok(int64_t kv, int64_t nq, const AttendParams& p) {
  const bool ok = kv >= 0 && kv <= token_limit(p.max_pages, p.page_log2) && nq >= 0 && nq <= p.N;
  if (!ok) atomicOr(p.status, kDevBadIndex);
  return ok;
}

// The work of an attention call is a line of equal key tiles: unit after unit (a
// unit is the query rows that one block works on together: their sequence and
// kv head, and for prompts a range of tokens), each with the tiles its rows see,
// at least one, behind kUnitCost places that stand for what a unit costs beside its
// tiles.  The line is cut into equal shares, one for each block, so every
// block has the same work whatever the lengths.  A unit that a cut goes through
// is computed in parts: the block where it begins writes its part to slot 1 of
// its two and says in `tails` how many blocks hold the rest; each of those
// writes slot 0.  A second kernel joins the parts.
//   part: rows x d fp32 sums (relative to the row's maximum m and to the largest
//   scale v of the values), then for each row {m, l, v, 0}, m in log2 units
constexpr int kPartStats = 4;
// In tiles: 3500 to 4000 cycles against 1000 (tokens), 18000 against 4300 (prompts).
// Without it blocks whose share is many short units ended last (3 prompts of 2510
// tokens, 32 heads in groups of eight: 368 us; with 2, 4 and 6: 261, 230 and 238; token
// calls differ by 2% between these).
constexpr int kUnitCost = 4;

// A block's place on the line: place `x` of a unit of `tiles` tiles, `left` places from
// the end of the share.
struct Place {
  int x;
  __device__ __forceinline__ int tile() const { return max(0, x - kUnitCost); }
  // the tiles from there on that are in the share
  __device__ __forceinline__ int count(int tiles, int64_t left) const {
    return max(0, (int)min((int64_t)(tiles + kUnitCost), x + left) - kUnitCost - tile());
  }
};

// Tokens of a page table over which prompts' units may be left whole, at most.
constexpr int kWholePrompts = 1024;

// tails[block] = {blocks that hold the rest (0: nothing to join), b, kv head, query tile}

// A unit's rows: `rows` in `blocks` tiles of tile_rows, the first
// tile_tokens * G of a tile in use: row r of a tile is head r % G of token r / G.
struct JoinGeometry {
  int rows, blocks, tile_rows, tile_tokens;
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Adds x >= 0, a step's own sum, to a row's sum l >= 0.  What the addition rounds off
// is kept in `lost`, to be added at the end: a step far below half a place of l (a key with
// most of the weight, then 2^18 of 2^-24.5 of it) would leave no trace otherwise.  Off by 2^-23 x
// at most also where x > l.
__device__ __forceinline__ void add_up(float& l, float& lost, float x) {
  const float sum = l + x;
  lost += x - (sum - l);
  l = sum;
}

// The larger one, or the NaN: of a page's scale, where it shows that the page was never written.
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Weights are held as 2^kAttendShift at a row's reference maximum.
constexpr float kAttendShift = 7.f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Whether a row's reference maximum m (log2 units) is so large that 2^(score f - m) needs the
// product rounded as m was: exact, it is up to half a place of m away from m, and past 2^27 that
// overflowed weights, or left none (finite inputs gave NaN, and zeros).  There the maximum is
// followed without slack, too.  (True of -infinity as well: a row without weights is at no loss.)
__device__ __forceinline__ bool far_off(float m) { return fabsf(m) > 4194304.f; }

// How far above m a score may lie that leaves m as it is.
__device__ __forceinline__ float slack_of(float m) { return far_off(m) ? 0.f : 8.f; }

// n / m for n >= 0, m > 0; in 32 bits where n has them (a 64-bit division takes a
// few hundred cycles).
__device__ __forceinline__ int64_t div_short(int64_t n, int64_t m) {
  return (n | m) >> 32 ? n / m : (int64_t)((uint32_t)n / (uint32_t)m);
}

// The line in equal shares for at most `blocks` blocks, of about four places where it is
// short (two at least; those of a unit's cost are no tiles, so a block may have none): block k has
// [begin(k), begin(k + 1)).
struct Shares {
  int64_t each;
  int n, more;  // shares; how many of them have one more
  __device__ __forceinline__ Shares(int64_t total, int blocks) {
    n = (int)min((int64_t)blocks, (total + 3) >> 2);
    each = n ? div_short(total, n) : 0;
    more = (int)(total - each * n);
  }
  __device__ __forceinline__ int64_t begin(int k) const { return k * each + min(k, more); }
  // of a unit that ends at `end`: blocks behind block k that hold some of it
  __device__ __forceinline__ int behind(int k, int64_t end) const {
    int last = k;
    while (begin(last + 1) < end) ++last;
    return last - k;
  }
};

// Sum over the block's threads below this one, and over all (kThreads a multiple
// of 32, scratch for kThreads / 32 numbers).
template <int kThreads>
__device__ __forceinline__ int64_t block_exclusive_sum(int64_t x, int64_t* scratch,
                                                       int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t in = x;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, in, m);
    if (lane >= m) in += y;
  }
  if (lane == 31) scratch[warp] = in;
  __syncthreads();
  int64_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
  }
  return before + in - x;
}

}  // namespace la
