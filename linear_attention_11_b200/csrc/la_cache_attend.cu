// la_cache_attend.cu -- which kernel an attention call over the 8-bit cache runs,
// and its workspace.
#include <cuda_runtime.h>

#include "la_cache.cuh"

namespace la {
namespace {

// Calls of at most 32 query rows for each kv head go to the token kernel.
constexpr int kTokenRows = 32;
// Short sequences leave their units whole: no line to find one's place on, no parts,
// no workspace, one launch.  Token calls whose page tables hold at most kWholeTokens
// tokens a sequence (16 heads, 333 tokens: 7.5 us instead of 10.7, and 12 us instead of 16
// of the host's time); prompts whose tables hold at most kWholePrompt, or kWholePrompts
// with a unit for every SM (9 prompts of 49 tokens, 4 heads: 14 us instead of 27).
constexpr int kWholeTokens = 512, kWholePrompt = 512;
static_assert(kWholePrompt <= kWholePrompts, "the most");

struct Shape {
  bool token, whole;
  int ctas, rows;  // blocks, rows of a part
};

Shape shape_of(int B, int Hkv, int G, int64_t N, int d, int64_t tokens, int sms) {
  Shape s;
  s.token = N * G <= kTokenRows;
  if (s.token) {
    s.whole = tokens <= kWholeTokens && (int64_t)B * Hkv <= 0x7fffffff - 65536;
    s.rows = N * G <= 8 ? 8 : N * G <= 16 ? 16 : 32;
    s.ctas = (d == 128 ? 2 : 3) * sms;
  } else {
    const int tpu = 2 * (128 / G);  // tokens of a unit
    const int64_t units = (int64_t)B * Hkv * ((N + tpu - 1) / tpu);
    s.whole = (tokens <= kWholePrompt || (tokens <= kWholePrompts && units >= sms)) &&
              units <= 0x7fffffff - 65536;
    s.rows = 256;
    s.ctas = sms;
  }
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
  const Shape s = shape_of(B, c.Hkv, Hq / c.Hkv, N, c.d, (int64_t)max_pages * c.page, sms);
  AttendParams p{q, {c.k_codes, c.v_codes}, {c.k_scale, c.v_scale}, table, kv_len, q_len, o,
                 lse, status, N, c.num_pages, B, Hq, c.Hkv, Hq / c.Hkv, max_pages,
                 page_log2(c.page), scale, static_cast<float*>(workspace), nullptr};
  if (workspace)
    p.tails = reinterpret_cast<int4*>(static_cast<char*>(workspace) + part_bytes(s, c.d));
  const cudaError_t e = s.token
                            ? launch_cache_token(p, c, dtype, s.rows, s.ctas, s.whole, stream)
                            : launch_cache_prompt(p, dtype, c.d, s.ctas, s.whole, stream);
  if (e != cudaSuccess || s.whole) return e;
  const JoinGeometry g = s.token ? JoinGeometry{s.rows, 1, s.rows, (int)N}
                                 : JoinGeometry{256, 2, 128, 128 / p.G};
  return launch_cache_join(p, g, dtype, c.d, s.ctas, stream);
}

bool attend_uses_workspace(int B, int Hkv, int G, int64_t N, int d, int64_t tokens, int sms) {
  return !shape_of(B, Hkv, G, N, d, tokens, sms).whole;
}

size_t attend_workspace_bytes(int B, int Hq, int Hkv, int64_t N, int d, int sms) {
  const Shape s = shape_of(B, Hkv, Hq / Hkv, N, d, INT64_MAX, sms);
  return (part_bytes(s, d) + (size_t)s.ctas * sizeof(int4) + 255) / 256 * 256;
}

}  // namespace la
