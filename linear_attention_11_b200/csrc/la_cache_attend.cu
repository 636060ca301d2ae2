// la_cache_attend.cu -- causal softmax attention over the 8-bit cache, one warp
// for each query row: keys in order, a running maximum m, sum l and output.
#include <cuda_runtime.h>

#include "la_cache.cuh"

namespace la {
namespace {

template <typename T, int D>
__global__ void __launch_bounds__(128) attend_rows_kernel(const AttendParams p) {
  constexpr int V = D / 32;  // values of a row that a lane holds
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);  // (b, head, i)
  if (row >= (int64_t)p.B * p.Hq * p.N) return;
  const int64_t i = row % p.N;
  const int bh = (int)(row / p.N), b = bh / p.Hq, h = (bh % p.Hq) / p.G;
  const int64_t kv = p.kv_len[b], nq = p.q_len ? (int64_t)p.q_len[b] : p.N;
  if (!attend_lengths_ok(kv, nq, p)) return;
  if (i >= nq) return;
  const int64_t sees = max((int64_t)0, kv - nq + i + 1);
  float q[V], o[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    q[j] = (float)static_cast<const T*>(p.q)[row * D + lane * V + j] * p.scale * 1.44269504f;
    o[j] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int64_t t = 0; t < sees; ++t) {
    const int at = p.table[(int64_t)b * p.max_pages + (t >> p.page_log2)];
    const bool known = at >= 0 && at < p.num_pages;
    if (!known) atomicOr(p.status, kDevBadIndex);
    float x[2][V];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int64_t ph = (int64_t)at * p.Hkv + h;
#pragma unroll
      for (int j = 0; j < V; j += 2) {
        uint32_t c = 0;
        if (known)
          c = *reinterpret_cast<const uint16_t*>(
              p.codes[w] + ((ph << p.page_log2) + (t & ((1 << p.page_log2) - 1))) * D + lane * V + j);
        const float2 f = unpack2<__half>(e4m3x2_to_f16x2(c));
        const float s = known ? p.kvscale[w][ph] : 0.f;
        x[w][j] = f.x * s;
        x[w][j + 1] = f.y * s;
      }
    }
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) s += q[j] * x[0][j];
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    const float mn = fmaxf(m, s), a = exp2f(m - mn), e = exp2f(s - mn);
    m = mn;
    l = l * a + e;
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = o[j] * a + e * x[1][j];
  }
  const float inv = l > 0.f ? 1.f / l : (sees ? l : 0.f);
#pragma unroll
  for (int j = 0; j < V; j += 2)
    *reinterpret_cast<uint32_t*>(static_cast<T*>(p.o) + row * D + lane * V + j) =
        pack2<T>(o[j] * inv, o[j + 1] * inv);
  if (p.lse && lane == 0)
    p.lse[row] = sees ? (m + log2f(l)) * 0.69314718f : -INFINITY;
}

template <typename T, int D>
cudaError_t attend_typed(const AttendParams& p, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.B * p.Hq * p.N;
  attend_rows_kernel<T, D><<<(unsigned)((rows + 3) / 4), 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

namespace {

// Calls of at most 32 query rows for each kv head go to the token kernel.
constexpr int kTokenRows = 32;

struct Shape {
  bool token;
  int ctas, rows;  // blocks, rows of a part
};

Shape shape_of(int G, int64_t N, int sms) {
  Shape s;
  s.token = N * G <= kTokenRows;
  s.rows = N * G <= 16 ? 16 : 32;
  s.ctas = 2 * sms;
  return s;
}

size_t part_bytes(const Shape& s, int d) {
  return (size_t)s.ctas * 2 * s.rows * (d + kPartStats) * sizeof(float);
}

}  // namespace

cudaError_t launch_cache_attend(const la_cache& c, const void* q, la_dtype dtype,
                                const int32_t* table, const int32_t* kv_len, const int32_t* q_len,
                                void* o, float* lse, int B, int Hq, int64_t N, int max_pages,
                                float scale, void* workspace, unsigned* status, int sms,
                                cudaStream_t stream) {
  const Shape s = shape_of(Hq / c.Hkv, N, sms);
  AttendParams p{q, {c.k_codes, c.v_codes}, {c.k_scale, c.v_scale}, table, kv_len, q_len, o,
                 lse, status, N, c.num_pages, B, Hq, c.Hkv, Hq / c.Hkv, max_pages,
                 page_log2(c.page), scale, static_cast<float*>(workspace), nullptr};
  p.tails = reinterpret_cast<int4*>(static_cast<char*>(workspace) + part_bytes(s, c.d));
  if (s.token) {
    const cudaError_t e = launch_cache_token(p, c, dtype, (int)N * p.G, s.ctas, stream);
    if (e != cudaSuccess) return e;
    const JoinGeometry g{s.rows, 1, s.rows, (int)N, kTokenShift};
    return launch_cache_join(p, g, dtype, c.d, s.ctas, stream);
  }
  if (c.d == 64)
    return dtype == LA_BF16 ? attend_typed<__nv_bfloat16, 64>(p, stream)
                            : attend_typed<__half, 64>(p, stream);
  return dtype == LA_BF16 ? attend_typed<__nv_bfloat16, 128>(p, stream)
                          : attend_typed<__half, 128>(p, stream);
}

size_t attend_workspace_bytes(int B, int Hq, int Hkv, int64_t N, int d, int sms) {
  const Shape s = shape_of(Hq / Hkv, N, sms);
  return (part_bytes(s, d) + (size_t)s.ctas * sizeof(int4) + 255) / 256 * 256;
}

}  // namespace la
