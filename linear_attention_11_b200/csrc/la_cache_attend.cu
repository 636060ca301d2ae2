// la_cache_attend.cu -- which kernel an attention call over the 8-bit cache runs,
// and its workspace.
#include <cuda_runtime.h>

#include "la_cache.cuh"

namespace la {
namespace {

// Calls of at most 32 query rows for each kv head go to the token kernel.
constexpr int kTokenRows = 32;
// Token calls whose page tables hold at most this many tokens a sequence leave
// their units whole: no parts, no workspace, one launch (16 heads, 333 tokens: 8.9 us
// instead of 9.4, and 12 us instead of 16 of the host's time).
constexpr int kWholeTokens = 512;

struct Shape {
  bool token, whole;
  int ctas, rows;  // blocks, rows of a part
};

Shape shape_of(int G, int64_t N, int d, int64_t tokens, int sms) {
  Shape s;
  s.token = N * G <= kTokenRows;
  s.whole = s.token && tokens <= kWholeTokens;
  s.rows = s.token ? (N * G <= 16 ? 16 : 32) : 256;
  s.ctas = s.token ? (d == 128 ? 2 : 3) * sms : sms;
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
  const Shape s = shape_of(Hq / c.Hkv, N, c.d, (int64_t)max_pages * c.page, sms);
  AttendParams p{q, {c.k_codes, c.v_codes}, {c.k_scale, c.v_scale}, table, kv_len, q_len, o,
                 lse, status, N, c.num_pages, B, Hq, c.Hkv, Hq / c.Hkv, max_pages,
                 page_log2(c.page), scale, static_cast<float*>(workspace), nullptr};
  if (workspace)
    p.tails = reinterpret_cast<int4*>(static_cast<char*>(workspace) + part_bytes(s, c.d));
  const cudaError_t e = s.token
                            ? launch_cache_token(p, c, dtype, (int)N * p.G, s.ctas, s.whole, stream)
                            : launch_cache_prompt(p, dtype, c.d, s.ctas, stream);
  if (e != cudaSuccess || s.whole) return e;
  const JoinGeometry g = s.token ? JoinGeometry{s.rows, 1, s.rows, (int)N}
                                 : JoinGeometry{256, 2, 128, 128 / p.G};
  return launch_cache_join(p, g, dtype, c.d, s.ctas, stream);
}

bool attend_uses_workspace(int G, int64_t N, int64_t tokens) {
  return !shape_of(G, N, 128, tokens, 1).whole;
}

size_t attend_workspace_bytes(int B, int Hq, int Hkv, int64_t N, int d, int sms) {
  const Shape s = shape_of(Hq / Hkv, N, d, INT64_MAX, sms);
  return (part_bytes(s, d) + (size_t)s.ctas * sizeof(int4) + 255) / 256 * 256;
}

}  // namespace la
