// la_cache_prompt.cu -- attention of a prompt, or a piece of one, over the 8-bit
// cache, on tcgen05.
//
//   S = Q C_k^T,  p_rj = 2^(S_rj f_r - m_r),  o_r = sum_j p_rj b_j c_j / sum_j p_rj
// for a tile of 256 query rows (two of 128: tokens x the G heads of a kv head) and
// key tiles of 128 tokens, each row up to its own token.  4 d flops for each
// query-key pair and row against one exponential: at d = 128 the tensor cores and the
// exponential unit (16 a cycle and SM) take equally long, about 2100 cycles
// for a key tile each, so the two 128-row tiles take turns: one's products run
// under the other's softmax.
//
// Roles (640 threads, one block for each SM):
//   warps 0-3, 4-7  softmax of row tile 0, 1: a thread owns a row (= a lane of
//                   tensor memory), so maxima and sums need no exchange; q to f16
//                   and its row factor at a unit's start; output at its end
//   warps 8-15      codes to f16 in shared memory, 128-byte swizzled as the
//                   products read them: pages are gathered by plain 16-byte loads one
//                   half tile ahead, as the conversion needs the codes in registers
//                   anyway
//   warp 16         issues the products (17 to 19 fill up its warpgroup: registers go by those)
// The scale of a page against the largest of the block's share of the unit is a
// power of two and goes into the conversion (exact in f16 down to 2^-15 of the
// largest; below, codes lose bits that weigh 2^-24 of it), so one factor a row is
// left for the scores and one a unit for the output.
// P (f16) is written over its scores; O stays in tensor memory, and is rescaled
// only when a row's maximum grows by more than 2^8: weights are 2^7 at a row's
// reference maximum and stay below 2^15, and count down to 2^-32 of it.
#include <cuda_runtime.h>

#include <algorithm>

#include "la_cache.cuh"
#include "la_ptx.cuh"

namespace la {
namespace {

constexpr int kKeys = 128;  // tokens of a key tile
constexpr int kThreads = 640, kConvert = 256;
constexpr int kIssue = 16;  // the warp that issues the products
constexpr float kShift = kPromptShift;
constexpr float kSlack = 8.f;  // growth of a row's maximum that is let pass
constexpr int kMinTiles = 2;
// registers of a thread after the split; 640 x 96 at launch
constexpr int kRegsSoftmax = 136, kRegsConvert = 80, kRegsIssue = 40;
static_assert(256 * kRegsSoftmax + 256 * kRegsConvert + 128 * kRegsIssue <= 640 * 96, "registers");

template <int D>
struct PromptLayout {
  static constexpr int kQ = 128 * D * 2;             // one row tile, f16
  static constexpr int kSlot = kKeys * D * 2;        // a K or V tile, f16
  static constexpr int kSlots = D == 128 ? 5 : 8;
  static constexpr int kSlotOff = 2 * kQ;
  static constexpr int kMiscOff = kSlotOff + kSlots * kSlot;
  // scan scratch 20 x 8, start 3 x 8, line and shares 2 x 8 | walks | barriers | e values
  static constexpr int kBars = 2 * kSlots + 2 * 6 + 2;
  static constexpr int kWalkOff = kMiscOff + 208;
  static constexpr int kBarOff = kWalkOff + 17 * 64;
  static constexpr int kEOff = kBarOff + kBars * 8;  // float2 e[2], float2 red[8]
  static constexpr int kEnd = kEOff + 80 + 16;       // tmem slot, abort flag
  static constexpr int kBytes = kEnd + 1024;
};

__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, int b_mn_major) {
  return (1u << 4) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// A block's walk along its share of the line of key tiles: units (b, h, qt).  Each
// warp has one in shared memory, which its lane 0 moves on: in registers it would
// crowd out the score rows.
struct Walk {
  int64_t pos, end;
  int b, h, qt;
  int tile, tiles;
  int kv, nq, tpt;
  bool ok;

  __device__ void load(const AttendParams& p) {
    const int64_t len = p.kv_len[b], n = p.q_len ? (int64_t)p.q_len[b] : p.N;
    ok = attend_lengths_ok(len, n, p);
    kv = (int)len;
    nq = ok ? (int)n : 0;
  }
  __device__ int units() const { return (nq + 2 * tpt - 1) / (2 * tpt); }
  // key tiles that row tile t of unit q sees (0: none, or no such rows)
  __device__ int sees(int q, int t) const {
    const int first = (q * 2 + t) * tpt;
    if (first >= nq) return 0;
    const int n = kv - nq + min(nq, first + tpt);
    return n > 0 ? (n + kKeys - 1) / kKeys : 0;
  }
  __device__ int tiles_of(int q) const { return max(1, max(sees(q, 0), sees(q, 1))); }
  __device__ int count() const { return (int)min((int64_t)(tiles - tile), end - pos); }
  // the tiles of row tile t in this share of the unit
  __device__ int count(int t, int n) const { return max(0, min(n, sees(qt, t) - tile)); }
  __device__ void next(const AttendParams& p) {
    pos += tiles - tile;
    tile = 0;
    if (++qt >= units()) {
      qt = 0;
      if (++h >= p.Hkv) {
        h = 0;
        do {
          if (++b >= p.B) return;
          load(p);
        } while (nq == 0);
      }
    }
    tiles = tiles_of(qt);
  }
};

// 16 bytes, or zeros.  Volatile, so that the loads stay where they are written:
// ahead of the conversion before them.
__device__ __forceinline__ uint4 load_codes(const uint8_t* p, bool there) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@q ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"((uint32_t)there));
  return v;
}

// A word, or `other`, likewise.
__device__ __forceinline__ int load_word(const int* p, bool there, int other) {
  int v;
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\tmov.b32 %0, %3;\n\t"
      "@q ld.global.nc.b32 %0, [%1];\n\t}"
      : "=&r"(v)
      : "l"(p), "r"((uint32_t)there), "r"(other));
  return v;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, __half2 f) {
  const __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), f);
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const AttendParams p) {
  using L = PromptLayout<D>;
  constexpr uint32_t IDESC_QK = idesc_f16_f32(128, kKeys, 0);
  constexpr uint32_t IDESC_PV = idesc_f16_f32(128, D, 1);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  int64_t* misc = reinterpret_cast<int64_t*>(sm + L::kMiscOff);
  Walk* walks = reinterpret_cast<Walk*>(sm + L::kWalkOff);
  static_assert(sizeof(Walk) <= 64, "room for a walk");
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(sm + L::kBarOff);
  uint64_t* kv_empty = kv_full + L::kSlots;
  uint64_t* q_full = kv_empty + L::kSlots;  // [2] a unit's q tile is in shared memory
  uint64_t* s_full = q_full + 2;            // [2] a score tile is computed
  uint64_t* p_full = s_full + 2;            // [2] its weights are written, O is rescaled
  uint64_t* o_full = p_full + 2;            // [2] a unit's last product with V is added
  // [2], units in turn: a unit's scale references are known; every softmax warp has
  // read them.  One barrier for all units would not do: the copies may be two units
  // ahead, and a wait cannot tell a phase from the one two after it
  uint64_t* e_full = o_full + 2;
  uint64_t* e_empty = e_full + 2;
  uint64_t* done = e_empty + 2;
  uint64_t* converters = done + 1;          // a barrier of their own
  float2* evals = reinterpret_cast<float2*>(sm + L::kEOff);
  float2* ered = evals + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::kEOff + 80);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::kEOff + 84);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    p.tails[blockIdx.x] = make_int4(0, 0, 0, 0);
    for (int i = 0; i < L::kSlots; ++i) {
      mbar_init(&kv_full[i], kConvert / 32);
      mbar_init(&kv_empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 4);
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 4);
      mbar_init(&o_full[t], 1);
      mbar_init(&e_full[t], 1);
      mbar_init(&e_empty[t], 8);
    }
    mbar_init(done, 1);
    mbar_init(converters, kConvert / 32);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kIssue) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }

  // The line's length, this block's share, and where that begins: tiles of each
  // sequence (a warp each), their sums, then the place in the sequence.
  {
    Walk w;
    w.tpt = 128 / p.G;
    int64_t total, shares;
    int64_t* line = reinterpret_cast<int64_t*>(sm);  // [B] <= kAttendMaxBatch, before any tile
    for (w.b = warp; w.b < p.B; w.b += kThreads / 32) {
      w.load(p);
      int64_t sum = 0;
      for (int q = lane; q < w.units(); q += 32) sum += w.tiles_of(q);
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
      if (lane == 0) line[w.b] = sum * p.Hkv;
    }
    __syncthreads();
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min((int)threadIdx.x * per, p.B), b1 = min(b0 + per, p.B);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += line[b];
    int64_t before = block_exclusive_sum<kThreads>(mine, misc, total);
    shares = min((int64_t)gridDim.x, (total + kMinTiles - 1) / kMinTiles);
    w.pos = w.end = 0;
    if ((int64_t)blockIdx.x < shares) {
      w.pos = total * blockIdx.x / shares;
      w.end = total * (blockIdx.x + 1) / shares;
    }
    if (w.pos < w.end && before <= w.pos && w.pos < before + mine) {
      int b = b0;
      for (; w.pos >= before + line[b]; ++b) before += line[b];
      misc[20] = b;
      misc[21] = (w.pos - before) / (line[b] / p.Hkv);
      misc[22] = (w.pos - before) % (line[b] / p.Hkv);
    }
    __syncthreads();
    if (w.pos < w.end) {
      w.b = (int)misc[20];
      w.h = (int)misc[21];
      w.load(p);
      int64_t rest = misc[22];
      int found = -1;
      for (int q0 = 0; found < 0; q0 += 32) {  // every warp for itself
        const int n = q0 + lane < w.units() ? w.tiles_of(q0 + lane) : 0;
        int in = n;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, in, m);
          if (lane >= m) in += y;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, (int64_t)in > rest);
        if (past || q0 + 32 >= w.units()) {
          const int at = past ? __ffs(past) - 1 : 31;
          found = q0 + at;
          rest -= __shfl_sync(0xffffffffu, in - n, at);
        } else {
          rest -= __shfl_sync(0xffffffffu, in, 31);
        }
      }
      w.qt = found;
      w.tile = (int)rest;
      w.tiles = w.tiles_of(found);
    }
    if (lane == 0 && warp <= kIssue) walks[warp] = w;
    if (threadIdx.x == 0) {
      misc[23] = total;
      misc[24] = shares;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Walk& w = walks[min(warp, kIssue)];
  auto advance = [&]() {  // by a whole warp
    __syncwarp();
    if (lane == 0) w.next(p);
    __syncwarp();
  };

  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    regs_inc<kRegsSoftmax>();
    const int t = warp >> 2;
    const int rr = (warp & 3) * 32 + lane;  // row of the tile = lane of tensor memory
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t st = tmem + lanes + t * 128, ot = tmem + lanes + 256 + t * 128;
    const uint32_t sq = base + t * L::kQ;
    int it = 0;    // score tiles so far
    int seg = 0;   // units so far
    int used = 0;  // units in which this row tile had any
    bool ok = true;
    while (w.pos < w.end && ok) {
      const int n = w.count(), mine = w.count(t, n);
      const int token = (w.qt * 2 + t) * w.tpt + rr / p.G, head = w.h * p.G + rr % p.G;
      const bool valid = rr < w.tpt * p.G && token < w.nq;
      const int64_t row = ((int64_t)w.b * p.Hq + head) * p.N + token;
      const int last = valid ? w.kv - w.nq + token : 0x7fffffff;  // last key that the row sees
      float f = 0.f;
      if (mine > 0) {
        // q: largest entry of the row into [2^14, 2^15), then f16; the sign of the
        // scale goes here too, so that the scores' factor is not negative
        uint4 x[D / 8];
        float top = 0.f;
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + row * D);
#pragma unroll
        for (int j = 0; j < D / 8; ++j) x[j] = valid ? __ldg(src + j) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          const uint32_t u[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 v = unpack2<T>(u[k]);
            top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
          }
        }
        const int ex = (int)(__float_as_uint(top) >> 23) - 127;
        const bool scaled = top > 0.f && ex < 128;
        const float up = scaled ? pow2i(max(min(14 - ex, 127), -126)) : 1.f;
        f = fabsf(p.scale) * kLog2e / up;
        const float q1 = p.scale < 0.f ? -up : up;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          const uint32_t u[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
          uint32_t v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 y = unpack2<T>(u[k]);
            v[k] = pack2<__half>(y.x * q1, y.y * q1);
          }
          st_shared_v4(sq + (j >> 3) * (128 * 128) + rr * 128 + (((j & 7) ^ (rr & 7)) << 4), v[0],
                       v[1], v[2], v[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[t]);
      }
      ok = warp_wait(&e_full[seg & 1], (seg >> 1) & 1, p.status, abort_flag);
      if (!ok) break;
      const float2 e = evals[seg & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&e_empty[seg & 1]);
      f = fmaxf(f * e.x, 1.17549435e-38f);  // not zero: a masked score stays at -infinity

      float m = -INFINITY, l = 0.f;  // reference maximum, sum of weights
      for (int i = 0; i < mine; ++i, ++it) {
        ok = warp_wait(&s_full[t], it & 1, p.status, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const int sees = last - (w.tile + i) * kKeys;  // columns up to this one are seen
        const bool masked = __any_sync(0xffffffffu, sees < kKeys - 1);
        // the row goes by twice, 64 scores at a time: held whole it would take the
        // registers that the conversion needs
        auto scores = [&](int half, uint32_t (&x)[64]) {
          tmem_ld32(st + half * 64, *reinterpret_cast<uint32_t(*)[32]>(x));
          tmem_ld32(st + half * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(x + 32));
          tmem_wait_ld();
          if (masked) {
#pragma unroll
            for (int k = 0; k < 64; ++k)
              if (half * 64 + k > sees) x[k] = __float_as_uint(-INFINITY);
          }
        };
        uint32_t x[64];
        float top = -INFINITY, top2 = -INFINITY;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          scores(half, x);
#pragma unroll
          for (int k = 0; k < 64; k += 4) {
            top = max3(top, __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
            top2 = max3(top2, __uint_as_float(x[k + 2]), __uint_as_float(x[k + 3]));
          }
        }
        top = fmaxf(top, top2);
        const float mt = top == -INFINITY ? -INFINITY : top * f;
        const bool grows = mt > m + kSlack || (m == -INFINITY && mt > -INFINITY);
        if (__any_sync(0xffffffffu, grows)) {
          const float a = grows ? exp2_fast(m - mt) : 1.f;
          if (grows) m = mt;
          l *= a;
          if (i > 0) {  // the product of the tile before is in: its commit comes before s_full's
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              uint32_t y[16];
              tmem_ld16(ot + c * 16, y);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * a);
              tmem_st16(ot + c * 16, y);
            }
          }
        }
        const float off = kShift - (m == -INFINITY ? 0.f : m);
        const float2 f2 = make_float2(f, f), off2 = make_float2(off, off);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          scores(half, x);
          uint32_t y[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            float2 v = fma2(make_float2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), f2, off2);
            v.x = exp2_fast(v.x);
            v.y = exp2_fast(v.y);
            sum = add2(sum, v);
            y[k] = pack2<__half>(v.x, v.y);
          }
          tmem_st32(st + half * 32, y);
        }
        l += sum.x + sum.y;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t]);
      }
      if (!ok) break;

      // the unit's output, or its part
      const bool begins = w.tile == 0, ends = w.tile + n == w.tiles;
      if (mine > 0) {
        ok = warp_wait(&o_full[t], used & 1, p.status, abort_flag);
        if (!ok) break;
        ++used;
        tc_fence_after();
      }
      float* part = p.parts + ((int64_t)blockIdx.x * 2 + (begins ? 1 : 0)) * 256 * (D + kPartStats);
      const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t x[32];
        if (mine > 0) {
          tmem_ld32(ot + c * 32, x);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = 0u;
        }
        if (!valid) continue;
        if (begins && ends) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(p.o) + row * D + c * 32);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              y[j] = pack2<T>(__uint_as_float(x[k * 8 + 2 * j]) * inv * e.y,
                              __uint_as_float(x[k * 8 + 2 * j + 1]) * inv * e.y);
            dst[k] = make_uint4(y[0], y[1], y[2], y[3]);
          }
        } else {
          uint4* dst = reinterpret_cast<uint4*>(part + (int64_t)(t * 128 + rr) * D + c * 32);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            dst[k] = make_uint4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
        }
      }
      tc_fence_before();
      if (valid && begins && ends) {
        if (p.lse) p.lse[row] = (m - kShift + log2f(l)) * kLn2;
      } else if (valid) {
        reinterpret_cast<float4*>(part + 256 * D)[t * 128 + rr] = make_float4(m, l, e.y, 0.f);
      }
      if (begins && !ends && threadIdx.x == 0) {
        int k = blockIdx.x;
        while (misc[23] * (k + 1) / misc[24] < w.pos + w.tiles) ++k;
        p.tails[blockIdx.x] = make_int4(k - (int)blockIdx.x, w.b, w.h, w.qt);
      }
      ++seg;
      advance();
    }
  } else if (warp < kIssue) {
    // ------------------------------------------------------------ codes to f16
    regs_dec<kRegsConvert>();
    constexpr int kLoads = kKeys * D / 16 / kConvert;  // 16-byte pieces of a thread
    constexpr int kPieces = D / 16;                    // of a row
    const int cw = warp - 8, ct = threadIdx.x - 256;
    // eight lanes that store together write two rows, so that no bank is met twice
    const int piece = D == 128 ? (lane & 3) + 4 * (lane >> 4) : lane & 3;
    const int sub = D == 128 ? cw * 4 + ((lane >> 2) & 3) : cw * 8 + (lane >> 2);
    constexpr int kRowsPerLoad = kConvert / kPieces;
    int u = 0, seg = 0, syncs = 0;
    bool ok = true;
    while (w.pos < w.end && ok) {
      const int cnt = w.count(), n = max(w.count(0, cnt), w.count(1, cnt));
      const int* ids = p.table + (int64_t)w.b * p.max_pages;
      const int first = w.tile * kKeys, kv = w.kv, h = w.h;
      // references: the largest scales of the pages of this share
      float ek = 0.f, ev = 0.f;
      {
        const int stop = min(kv, first + n * kKeys);
        const int pages = stop > first ? ((stop - 1) >> p.page_log2) + 1 : 0;
        for (int g = (first >> p.page_log2) + ct; g < pages; g += kConvert) {
          const int id = ids[g];
          if (id >= 0 && id < p.num_pages) {
            ek = fmaxf(ek, __ldg(p.kvscale[0] + (int64_t)id * p.Hkv + h));
            ev = fmaxf(ev, __ldg(p.kvscale[1] + (int64_t)id * p.Hkv + h));
          } else {
            atomicOr(p.status, kDevBadIndex);
          }
        }
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) {
          ek = fmaxf(ek, __shfl_xor_sync(0xffffffffu, ek, k));
          ev = fmaxf(ev, __shfl_xor_sync(0xffffffffu, ev, k));
        }
        if (lane == 0) ered[cw] = make_float2(ek, ev);
        if (!(ok = warps_sync(converters, syncs, p.status, abort_flag))) break;
#pragma unroll
        for (int k = 0; k < kConvert / 32; ++k) {
          ek = fmaxf(ek, ered[k].x);
          ev = fmaxf(ev, ered[k].y);
        }
        if (cw == 0) {  // one warp alone waits: the others may be a unit behind it
          if (seg >= 2)
            ok = warp_wait(&e_empty[seg & 1], ((seg >> 1) - 1) & 1, p.status, abort_flag);
          if (!ok) break;
          if (lane == 0) {
            evals[seg & 1] = make_float2(ek, ev);
            mbar_arrive(&e_full[seg & 1]);
          }
        }
        // ered may be written again
        if (!(ok = warps_sync(converters, syncs, p.status, abort_flag))) break;
      }
      const float kinv = ek > 0.f ? 1.f / ek : 0.f, vinv = ev > 0.f ? 1.f / ev : 0.f;

      // lane g < 8 knows the page and scales of tokens 16 g .. 16 g + 15 of a tile.
      // Each is asked for a whole tile before it is used, in loads that stay in
      // place: a page number at tile i for the codes of tile i + 2, scales at tile i
      // for the conversion of tile i + 1.
      auto ask_page = [&](int i) {
        const int tok = first + i * kKeys + (lane & 7) * 16;
        return load_word(ids + (tok >> p.page_log2), i < n && tok < kv, -1);
      };
      auto known = [&](int id) { return id >= 0 && id < p.num_pages ? id : -1; };
      auto ask_scale = [&](int id, int which) {
        return __int_as_float(load_word(
            reinterpret_cast<const int*>(p.kvscale[which]) + (int64_t)id * p.Hkv + h, id >= 0, 0));
      };
      auto load = [&](uint4 (&x)[kLoads], int i, int id, int which) {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
          const int r = j * kRowsPerLoad + sub;
          const int at = __shfl_sync(0xffffffffu, id, r >> 4);
          const int tok = first + i * kKeys + r;
          x[j] = load_codes(
              p.codes[which] +
                  ((((int64_t)at * p.Hkv + h) << p.page_log2) + (tok & ((1 << p.page_log2) - 1))) * D +
                  piece * 16,
              at >= 0 && tok < kv);
        }
      };
      auto store = [&](const uint4 (&x)[kLoads], float factor, int slot) {
        const uint32_t dst = base + L::kSlotOff + slot * L::kSlot;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
          const int r = j * kRowsPerLoad + sub;
          const __half2 f2 = __float2half2_rn(__shfl_sync(0xffffffffu, factor, r >> 4));
          const uint32_t c[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
          uint32_t y[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            y[2 * k] = hmul2(e4m3x2_to_f16x2(c[k] & 0xffffu), f2);
            y[2 * k + 1] = hmul2(e4m3x2_to_f16x2(c[k] >> 16), f2);
          }
          const uint32_t at = dst + (piece >> 2) * (kKeys * 128) + r * 128;
          const int ch = (piece & 3) * 2;
          st_shared_v4(at + ((ch ^ (r & 7)) << 4), y[0], y[1], y[2], y[3]);
          st_shared_v4(at + (((ch + 1) ^ (r & 7)) << 4), y[4], y[5], y[6], y[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&kv_full[slot]);
      };
      auto acquire = [&]() {
        return u < L::kSlots ||
               warp_wait(&kv_empty[u % L::kSlots], ((u / L::kSlots) - 1) & 1, p.status, abort_flag);
      };
      uint4 xk[kLoads], xv[kLoads];
      int id = known(ask_page(0)), id1 = ask_page(1);
      float fk = ask_scale(id, 0) * kinv, fv = ask_scale(id, 1) * vinv;
      load(xk, 0, id, 0);
      for (int i = 0; i < n; ++i) {
        const int id2 = ask_page(i + 2);
        id1 = known(id1);
        const float fk1 = ask_scale(id1, 0), fv1 = ask_scale(id1, 1);
        load(xv, i, id, 1);
        if (!(ok = acquire())) break;
        store(xk, fk, u % L::kSlots);
        ++u;
        load(xk, i + 1, id1, 0);
        if (!(ok = acquire())) break;
        store(xv, fv, u % L::kSlots);
        ++u;
        id = id1;
        id1 = id2;
        fk = fk1 * kinv;
        fv = fv1 * vinv;
      }
      if (!ok) break;
      ++seg;
      advance();
    }
  } else {
    regs_dec<kRegsIssue>();
    if (warp == kIssue && elect_one()) {
    // ------------------------------------------------------------ products
    // few registers: parities in bits, row tiles in loops that stay loops
    int u = 0;                          // K and V tiles so far
    uint32_t q_parity = 0, p_parity = 0;  // bit t: of the next wait for row tile t
    bool ok = true;
    auto slot = [&](int k) { return base + L::kSlotOff + (uint32_t)(k % L::kSlots) * L::kSlot; };
    auto wait_kv = [&](int k) {
      return mbar_wait(&kv_full[k % L::kSlots], (k / L::kSlots) & 1, p.status, abort_flag);
    };
    auto scores = [&](int t, int k) {  // S = Q K^T with the K tile k
      tc_fence_after();
      const uint32_t q = base + t * L::kQ, kt = slot(k), s = tmem + t * 128;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk >> 2) * (128 * 128) + (kk & 3) * 32;
        mma_ss(s, smem_desc_sw128(q + off, 16, 1024), smem_desc_sw128(kt + off, 16, 1024), IDESC_QK,
               kk > 0 ? 1u : 0u);
      }
      mma_commit(&s_full[t]);
    };
    while (w.pos < w.end && ok) {
      const int cnt = w.count(), c0 = w.count(0, cnt), c1 = w.count(1, cnt), n = max(c0, c1);
#pragma unroll 1
      for (int t = 0; t < 2; ++t) {
        if ((t ? c1 : c0) == 0) continue;
        ok = mbar_wait(&q_full[t], (q_parity >> t) & 1, p.status, abort_flag) && wait_kv(u);
        if (!ok) break;
        q_parity ^= 1u << t;
        scores(t, u);
      }
      if (ok && n > 0) mma_commit(&kv_empty[u % L::kSlots]);
#pragma unroll 1
      for (int i = 0; i < n && ok; ++i, u += 2) {
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
          const int c = t ? c1 : c0;
          if (i >= c) continue;
          ok = mbar_wait(&p_full[t], (p_parity >> t) & 1, p.status, abort_flag) && wait_kv(u + 1);
          if (!ok) break;
          p_parity ^= 1u << t;
          tc_fence_after();
          const uint32_t vt = slot(u + 1), pt = tmem + t * 128;
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)  // O += P V
            mma_ts(pt + 256, pt + kk * 8, smem_desc_sw128(vt + kk * 2048, kKeys * 128, 1024),
                   IDESC_PV, i > 0 || kk > 0 ? 1u : 0u);
          if (i + 1 < c) {
            ok = wait_kv(u + 2);
            if (!ok) break;
            scores(t, u + 2);
          } else {
            mma_commit(&o_full[t]);
          }
        }
        if (!ok) break;
        mma_commit(&kv_empty[(u + 1) % L::kSlots]);
        if (i + 1 < n) mma_commit(&kv_empty[(u + 2) % L::kSlots]);
      }
      if (ok) w.next(p);
    }
    mma_commit(done);
    mbar_wait_drain(done, 0);
    }
  }
  __syncwarp();
  griddep_launch_dependents();
  tc_fence_before();
  __syncthreads();
  if (warp == kIssue) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <typename T, int D>
cudaError_t launch_typed(const AttendParams& p, int ctas, cudaStream_t stream) {
  constexpr int bytes = PromptLayout<D>::kBytes;
  static_assert(bytes <= 227 * 1024, "shared memory");
  auto* kernel = prompt_kernel<T, D>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  kernel<<<ctas, kThreads, bytes, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_prompt(const AttendParams& p, la_dtype dtype, int d, int ctas,
                                cudaStream_t stream) {
  if (d == 64)
    return dtype == LA_BF16 ? launch_typed<__nv_bfloat16, 64>(p, ctas, stream)
                            : launch_typed<__half, 64>(p, ctas, stream);
  return dtype == LA_BF16 ? launch_typed<__nv_bfloat16, 128>(p, ctas, stream)
                          : launch_typed<__half, 128>(p, ctas, stream);
}

}  // namespace la
