// la_cache_join.cu -- joins the parts of attention units that were cut between
// blocks.  For a row with parts (O_k, m_k, l_k, v_k), sums relative to 2^m_k and
// v_k:
//     m = max m_k,  o = sum_k O_k 2^(m_k - m) v_k / sum_k l_k 2^(m_k - m)
// The unit that begins at the end of block c's share is this kernel's blocks c; its
// parts lie in slot 1 of block c and slot 0 of the blocks behind it, and are added
// in that order.  A warp takes a row: its lanes first read the parts' m, l and v
// side by side, then go through the parts' sums, all lanes on one row.
#include <cuda_runtime.h>

#include "la_cache.cuh"
#include "la_ptx.cuh"

namespace la {
namespace {

constexpr int kWarps = 4;

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) join_kernel(const AttendParams p, const JoinGeometry g) {
  griddep_wait();
  const int4 tail = p.tails[blockIdx.x];
  if (tail.x == 0) return;
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int r = blockIdx.y * kWarps + (threadIdx.x >> 5); r < g.rows; r += gridDim.y * kWarps) {
    const int block = r / g.tile_rows, rr = r % g.tile_rows;
    const int64_t i = ((int64_t)tail.w * g.blocks + block) * g.tile_tokens + rr / p.G;
    const int64_t nq = p.q_len ? (int64_t)p.q_len[tail.y] : p.N;
    if (rr >= g.tile_tokens * p.G || i >= nq) continue;

    const int n = tail.x + 1;
    const int64_t stride = (int64_t)g.rows * (D + kPartStats);  // floats of a part
    auto part = [&](int k) {
      return p.parts + ((int64_t)(blockIdx.x + k) * 2 + (k == 0 ? 1 : 0)) * stride;
    };
    auto stats = [&](int k) {
      return k < n ? reinterpret_cast<const float4*>(part(k) + (int64_t)g.rows * D)[r]
                   : make_float4(-INFINITY, 0.f, 0.f, 0.f);
    };
    float m = -INFINITY, v = 0.f;
    for (int k0 = 0; k0 < n; k0 += 32) {
      const float4 s = stats(k0 + lane);
      m = fmaxf(m, s.x);
      v = fmaxf(v, s.z);
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) {
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
      v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, k));
    }
    const float ref = m == -INFINITY ? 0.f : m;
    const float vinv = v > 0.f ? 1.f / v : 0.f;
    constexpr int V = D / 32;  // columns of a lane
    float o[V];
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = 0.f;
    float l = 0.f;
    for (int k0 = 0; k0 < n; k0 += 32) {
      const float4 s = stats(k0 + lane);
      const float a = exp2_fast(s.x - ref);
      float sum = s.y * a;
      const float f = a * (s.z * vinv);
      for (int k = 0; k < min(32, n - k0); ++k) {
        const float w = __shfl_sync(0xffffffffu, f, k);
        const float* src = part(k0 + k) + (int64_t)r * D + lane * V;
        if constexpr (V == 4) {
          const float4 x = *reinterpret_cast<const float4*>(src);
          o[0] += x.x * w; o[1] += x.y * w; o[2] += x.z * w; o[3] += x.w * w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(src);
          o[0] += x.x * w; o[1] += x.y * w;
        }
      }
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
      l += sum;
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    const int64_t row = ((int64_t)tail.y * p.Hq + tail.z * p.G + rr % p.G) * p.N + i;
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<T*>(p.o) + row * D + lane * V);
#pragma unroll
    for (int j = 0; j < V; j += 2) dst[j / 2] = pack2<T>(o[j] * inv * v, o[j + 1] * inv * v);
    if (p.lse && lane == 0) p.lse[row] = (m - kAttendShift + log2f(l)) * kLn2;
  }
}

template <typename T>
cudaError_t launch_typed(const AttendParams& p, const JoinGeometry& g, int d, int ctas,
                         cudaStream_t stream) {
  // a programmatic dependent of the attention kernel: its blocks are placed
  // while that one drains
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, g.rows <= 32 ? g.rows / kWarps : g.rows / kWarps / 4);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return d == 64 ? cudaLaunchKernelEx(&cfg, join_kernel<T, 64>, p, g)
                 : cudaLaunchKernelEx(&cfg, join_kernel<T, 128>, p, g);
}

}  // namespace

cudaError_t launch_cache_join(const AttendParams& p, const JoinGeometry& g, la_dtype dtype, int d,
                              int ctas, cudaStream_t stream) {
  return dtype == LA_BF16 ? launch_typed<__nv_bfloat16>(p, g, d, ctas, stream)
                          : launch_typed<__half>(p, g, d, ctas, stream);
}

}  // namespace la
