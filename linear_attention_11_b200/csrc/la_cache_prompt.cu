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
//   warp 16         issues the products
//   warp 17         goes ahead from unit to unit and writes down for the others what
//                   they are (18 and 19 fill up the warpgroup: registers go by those)
// The scale of a page against the largest of the block's share of the unit is a
// power of two and goes into the conversion, so one factor a row is left for the scores
// and one a unit for the output.  Exact in f16 down to 2^-15 of the largest.  Where a
// page is smaller, the unit's factors are 2^7 (448 x 2^7 still is an f16): exact down to
// 2^-22, and below that values lose what is under 2^-32 of the largest scale.
// P (f16) is written over its scores; O stays in tensor memory, and is rescaled
// only when a row's maximum grows by more than 2^8: weights are 2^7 at a row's
// reference maximum and stay below 2^15, and count down to 2^-32 of it.
#include <cuda_runtime.h>

#include <algorithm>

#include "la_cache.cuh"
#include "la_ptx.cuh"

namespace la {
namespace {

constexpr int kKeys = 128;  // tokens of a key tile: what is converted at a time
constexpr int kThreads = 640, kConvert = 256;
constexpr int kIssue = 16, kPlan = 17;  // the warps that issue products and plan
constexpr int kPlans = 4;               // units that the plan is ahead at most
constexpr float kShift = kAttendShift;
// Key tiles whose products O takes up in tensor memory; then it is added to its part in
// the workspace and begins again.  The products cut off what lies below the sum's last
// places and do not round it: over 2^18 tokens in one sum, all values 1, o was 0.9937.
// 1024 tokens over 32768: 2.23 ms without, 2.25 with 128 tiles, 2.30 with 64.
constexpr int kChain = 128;
static_assert((kChain & (kChain - 1)) == 0, "a power of two");
static_assert(kChain * kKeys >= kWholePrompts, "whole units have no workspace");
// Registers of a thread after the split; 640 x 96 at launch.  With 40 for the issuing
// warp its descriptors go through local memory: 1.36 ms instead of 1.26 for four
// prompts of 8192 tokens and 16 heads.
constexpr int kRegsSoftmax = 128, kRegsConvert = 72, kRegsIssue = 72;
static_assert(256 * kRegsSoftmax + 256 * kRegsConvert + 128 * kRegsIssue <= 640 * 96, "registers");

// A block's part of a unit, as the planning warp writes it down.
struct Unit {
  int b, h, qt;
  int tile, n;       // first key tile and how many; n < 0: no more units
  int c[2];          // how many score tiles of those each row tile sees
  int kv, nq;
  int begins, ends;  // whether the unit's first and last tiles are among them
  int follow;        // of a unit that begins but does not end: blocks that hold the rest
  float ek, ev;      // what codes are scaled against: the pages' largest scales, or 2^-7 of them
};

template <int D>
struct PromptLayout {
  static constexpr int kQ = 128 * D * 2;             // one row tile, f16
  static constexpr int kSlot = kKeys * D * 2;        // a K or V tile, f16
  static constexpr int kSlots = D == 128 ? 5 : 8;
  static constexpr int kSlotOff = 2 * kQ;
  static constexpr int kMiscOff = kSlotOff + kSlots * kSlot;
  static constexpr int kUnitOff = kMiscOff + 23 * 8;  // scan scratch 20 x 8, start 3 x 8
  static constexpr int kBarOff = kUnitOff + kPlans * 64;
  static constexpr int kBars = 2 * kSlots + 2 * 5 + 2 * kPlans + 1;
  static constexpr int kEnd = kBarOff + kBars * 8 + 16;  // tmem slot, abort flag, ticks
  static constexpr int kBytes = kEnd + 1024;
};

__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, int b_mn_major) {
  return (1u << 4) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// A block's walk along its share of the line of key tiles: units (b, h, qt).
struct Walk {
  int64_t pos, end;
  int b, h, qt;
  Place at;
  int tiles;
  int kv, nq, tpt;
  bool ok, whole;  // whole: units are not cut, `pos` counts them, every gridDim.x-th

  __device__ void load(const AttendParams& p) {
    const int64_t len = p.kv_len[b], n = p.q_len ? (int64_t)p.q_len[b] : p.N;
    ok = attend_lengths_ok(len, n, p);
    kv = (int)len;
    nq = ok ? (int)n : 0;
  }
  __device__ int units() const { return (nq + 2 * tpt - 1) / (2 * tpt); }
  // score tiles that row tile t of unit q sees (0: none, or no such rows)
  __device__ int sees(int q, int t) const {
    const int first = (q * 2 + t) * tpt;
    if (first >= nq) return 0;
    const int n = kv - nq + min(nq, first + tpt);
    return n > 0 ? (n + kKeys - 1) / kKeys : 0;
  }
  __device__ int tiles_of(int q) const {
    return max(1, max(sees(q, 0), sees(q, 1)));
  }
  __device__ int places(int q) const { return tiles_of(q) + kUnitCost; }
  __device__ int tile() const { return whole ? 0 : at.tile(); }
  __device__ int count() const { return whole ? tiles : at.count(tiles, end - pos); }
  // the score tiles of row tile t in this share's n key tiles of the unit
  __device__ int count(int t, int n) const { return max(0, min(n, sees(qt, t) - tile())); }
  // whole units: from unit `pos` on to the next of this block's that there is
  __device__ void settle(const AttendParams& p) {
    const int most = ((int)p.N + 2 * tpt - 1) / (2 * tpt);  // of a sequence and head
    for (; pos < end; pos += gridDim.x) {
      const int bh = (int)pos / most;
      qt = (int)pos - bh * most;
      b = bh / p.Hkv;
      h = bh - b * p.Hkv;
      load(p);
      if (qt >= units()) continue;
      tiles = tiles_of(qt);
      return;
    }
  }
  __device__ void next(const AttendParams& p) {
    if (whole) {
      pos += gridDim.x;
      settle(p);
      return;
    }
    pos += tiles + kUnitCost - at.x;
    at.x = 0;
    if (pos + kUnitCost >= end) pos = end;  // the share ends before the next one's first tile
    if (pos >= end) return;
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

// By a whole warp: 16 columns of its lanes of tensor memory by each lane's factor.
__device__ __forceinline__ void times(uint32_t at, float a) {
  uint32_t y[16];
  tmem_ld16(at, y);
  tmem_wait_ld();
#pragma unroll
  for (int j = 0; j < 16; ++j) y[j] = __float_as_uint(__uint_as_float(y[j]) * a);
  tmem_st16(at, y);
}

// a z + x, four fp32 numbers of x as they come from tensor memory.
__device__ __forceinline__ float4 plus(const float4& z, float a, const uint32_t* x) {
  return make_float4(fmaf(z.x, a, __uint_as_float(x[0])), fmaf(z.y, a, __uint_as_float(x[1])),
                     fmaf(z.z, a, __uint_as_float(x[2])), fmaf(z.w, a, __uint_as_float(x[3])));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, __half2 f) {
  const __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), f);
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const AttendParams p, bool whole) {
  using L = PromptLayout<D>;
  constexpr uint32_t IDESC_QK = idesc_f16_f32(128, kKeys, 0);
  constexpr uint32_t IDESC_PV = idesc_f16_f32(128, D, 1);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  int64_t* misc = reinterpret_cast<int64_t*>(sm + L::kMiscOff);
  auto unit_at = [&](int seg) -> Unit& {
    return *reinterpret_cast<Unit*>(sm + L::kUnitOff + (seg % kPlans) * 64);
  };
  static_assert(sizeof(Unit) <= 64, "room for a unit");
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(sm + L::kBarOff);
  uint64_t* kv_empty = kv_full + L::kSlots;
  uint64_t* q_full = kv_empty + L::kSlots;  // [2] a unit's q tile is in shared memory
  uint64_t* s_full = q_full + 2;            // [2] a score tile is computed
  uint64_t* p_full = s_full + 2;            // [2] its weights are written, O is rescaled
  uint64_t* o_full = p_full + 4;            // [2] a unit's last product with V is added
  uint64_t* u_full = o_full + 2;            // [kPlans] a unit is written down
  uint64_t* u_empty = u_full + kPlans;      // [kPlans] every role has read it
  uint64_t* done = u_empty + kPlans;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* ticks = abort_flag + 1;  // tiles converted so far
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    if (!whole) p.tails[blockIdx.x] = make_int4(0, 0, 0, 0);
    for (int i = 0; i < L::kSlots; ++i) {
      mbar_init(&kv_full[i], kConvert / 32);
      mbar_init(&kv_empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 4);
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[2 * t], 4);
      mbar_init(&p_full[2 * t + 1], 4);
      mbar_init(&o_full[t], 1);
    }
    for (int k = 0; k < kPlans; ++k) {
      mbar_init(&u_full[k], 1);
      mbar_init(&u_empty[k], 8 + kConvert / 32 + 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    *ticks = 0;
    fence_barrier_init();
  }
  if (warp == kIssue) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }

  // The line's length, this block's share, and where that begins: tiles of each
  // sequence (a warp each), their sums, then the place in the sequence.
  const int tpt = 128 / p.G;
  Walk w;
  w.tpt = tpt;
  w.whole = whole;
  int64_t total;
  Shares shares(0, 0);
  if (whole) {
    w.pos = blockIdx.x;
    w.end = (int64_t)p.B * p.Hkv * ((p.N + 2 * tpt - 1) / (2 * tpt));
    if (warp == kPlan) w.settle(p);
  } else {
    int64_t* line = reinterpret_cast<int64_t*>(sm);  // [B] <= kAttendMaxBatch, before any tile
    for (w.b = warp; w.b < p.B; w.b += kThreads / 32) {
      w.load(p);
      int64_t sum = 0;
      for (int q = lane; q < w.units(); q += 32) sum += w.places(q);
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
    shares = Shares(total, gridDim.x);
    w.pos = w.end = 0;
    if ((int)blockIdx.x < shares.n) {
      w.pos = shares.begin(blockIdx.x);
      w.end = shares.begin(blockIdx.x + 1);
    }
    if (w.pos < w.end && before <= w.pos && w.pos < before + mine) {
      int b = b0;
      for (; w.pos >= before + line[b]; ++b) before += line[b];
      misc[20] = b;
      const int64_t head = div_short(line[b], p.Hkv);  // tiles of a head
      misc[21] = div_short(w.pos - before, head);
      misc[22] = w.pos - before - misc[21] * head;
    }
    __syncthreads();
    if (warp == kPlan && w.pos < w.end) {
      w.b = (int)misc[20];
      w.h = (int)misc[21];
      w.load(p);
      int64_t rest = misc[22];
      int found = -1;
      for (int q0 = 0; found < 0; q0 += 32) {
        const int n = q0 + lane < w.units() ? w.places(q0 + lane) : 0;
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
      w.at.x = (int)rest;
      w.tiles = w.tiles_of(found);
      if (w.count() == 0) w.next(p);  // a share that ends, or goes on, behind this unit's cost
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // by a whole warp: unit `seg` once it is written down, and that it has been read.  Warps
  // whose row tile has no rows, and the one that plans, are ahead of the others here, and wait for
  // as long as a unit takes: with a limit of 2 s one of 2^27 tokens would have been given up.
  auto wait_unit = [&](int seg) {
    return warp_wait_working(&u_full[seg % kPlans], (seg / kPlans) & 1, abort_flag, ticks);
  };
  auto release_unit = [&](int seg) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&u_empty[seg % kPlans]);
  };
  bool ok = true;

  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    regs_inc<kRegsSoftmax>();
    const int t = warp >> 2;
    const int rr = (warp & 3) * 32 + lane;  // row of the tile = lane of tensor memory
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t st = tmem + lanes + t * 128, ot = tmem + lanes + 256 + t * 128;
    const uint32_t sq = base + t * L::kQ;
    // a row of 2-byte values: LPR lanes with 16 bytes each, RPI rows at a time
    constexpr int LPR = D / 8, RPI = 32 / LPR;
    const int sub = lane / LPR, piece = lane % LPR;
    int it = 0;    // score tiles so far
    int used = 0;  // units in which this row tile had any
    for (int seg = 0;; ++seg) {
      if (!(ok = wait_unit(seg))) break;
      const Unit& unit = unit_at(seg);
      const int mine = unit.c[t], first = unit.tile * kKeys, b = unit.b, h = unit.h, qt = unit.qt;
      if (unit.n < 0) break;
      const bool begins = unit.begins, whole = begins && unit.ends;
      const float ek = unit.ek, ev = unit.ev;
      const int token = (qt * 2 + t) * tpt + rr / p.G;
      const bool valid = rr < tpt * p.G && token < unit.nq;
      const int64_t row = ((int64_t)b * p.Hq + h * p.G + rr % p.G) * p.N + token;
      const int last = valid ? unit.kv - unit.nq + token : 0x7fffffff;  // last key that the row sees
      if (threadIdx.x == 0 && unit.follow > 0)
        p.tails[blockIdx.x] = make_int4(unit.follow, b, h, qt);
      const uint32_t rows = __ballot_sync(0xffffffffu, valid);
      release_unit(seg);
      float f = 0.f;
      if (mine > 0) {
        // q: largest entry of the row into [2^14, 2^15), then f16; the sign of the
        // scale goes here too, so that the scores' factor is not negative.  The warp
        // reads its 32 rows together, RPI at a time, and hands each row's factor to
        // the lane that owns it.
        constexpr int BATCH = 4;
        float up = 1.f;
#pragma unroll 1
        for (int i0 = 0; i0 < LPR; i0 += BATCH) {
          uint4 x[BATCH];
#pragma unroll
          for (int i = 0; i < BATCH; ++i) {
            const int r = (i0 + i) * RPI + sub;
            const int64_t at = __shfl_sync(0xffffffffu, row, r);
            x[i] = make_uint4(0u, 0u, 0u, 0u);
            if ((rows >> r) & 1)
              x[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + at * D) + piece);
          }
          // (the rows' maxima side by side: one after the other they took most of 6000
          // cycles)
          float top[BATCH];
#pragma unroll
          for (int i = 0; i < BATCH; ++i) {
            const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            top[i] = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 v = unpack2<T>(u[k]);
              top[i] = max3(top[i], fabsf(v.x), fabsf(v.y));
            }
          }
#pragma unroll
          for (int k = LPR / 2; k > 0; k >>= 1)
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
              top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], k));
#pragma unroll
          for (int i = 0; i < BATCH; ++i) {
            const int ex = (int)(__float_as_uint(top[i]) >> 23) - 127;
            top[i] = top[i] > 0.f && ex < 128 ? pow2i(max(min(14 - ex, 127), -126)) : 1.f;
            const float mine1 = __shfl_sync(0xffffffffu, top[i], (lane % RPI) * LPR);
            if (lane / RPI == i0 + i) up = mine1;
          }
#pragma unroll
          for (int i = 0; i < BATCH; ++i) {
            const int r = (warp & 3) * 32 + (i0 + i) * RPI + sub;
            const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            const float q1 = p.scale < 0.f ? -top[i] : top[i];
            uint32_t v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 y = unpack2<T>(u[k]);
              v[k] = pack2<__half>(y.x * q1, y.y * q1);
            }
            st_shared_v4(sq + (piece >> 3) * (128 * 128) + r * 128 + (((piece & 7) ^ (r & 7)) << 4),
                         v[0], v[1], v[2], v[3]);
          }
        }
        f = fabsf(p.scale) * kLog2e / up;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[t]);
      }
      f = fmaxf(f * ek, 1.17549435e-38f);  // not zero: a masked score stays at -infinity

      // The block's part of the unit in the workspace.  Of a unit that is not cut its sums
      // lie where those of the share's last unit will, which comes later.
      auto part_at = [&]() {
        return p.parts + ((int64_t)blockIdx.x * 2 + (begins ? 1 : 0)) * 256 * (D + kPartStats);
      };
      // Four sums of this thread's row, columns c * 32 + 4 k on: in those columns of the warp's
      // rows, whole lines for each k.
      auto sums_at = [&](int c, int k) {
        const int r = t * 128 + (warp & 3) * 32 + k * 4 + (lane >> 3);
        return reinterpret_cast<float4*>(part_at() + (int64_t)r * D + c * 32) + (lane & 7);
      };
      auto part_stats = [&]() { return part_at() + 256 * D + (t * 128 + rr) * kPartStats; };

      float m = -INFINITY, l = 0.f, lost = 0.f;  // reference maximum, sum of weights, see add_up
      for (int i0 = 0; i0 < mine && ok; i0 += kChain) {
        if (i0 > 0) {
          // O, all products before these scores, to the row's sums so far; those are relative
          // to 2^(their m)
          ok = warp_wait_brief(&s_full[t], it & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const float a = i0 > kChain && m > -INFINITY ? exp2_fast(*part_stats() - m) : 0.f;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            float4 z[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
              z[k] = i0 > kChain ? *sums_at(c, k) : make_float4(0.f, 0.f, 0.f, 0.f);
            uint32_t y[32];
            tmem_ld32(ot + c * 32, y);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *sums_at(c, k) = plus(z[k], a, y + 4 * k);
          }
          *part_stats() = m;
        }
#pragma unroll 1
        for (int i = i0; i < min(mine, i0 + kChain); ++i, ++it) {
          ok = warp_wait_brief(&s_full[t], it & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const int sees = last - first - i * kKeys;  // columns up to this one are seen
          const bool masked = __any_sync(0xffffffffu, sees < kKeys - 1);
          // The row goes by twice, 64 scores at a time: held whole it would take the
          // registers that the conversion needs.
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
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            scores(half, x);
#pragma unroll
            for (int k = 0; k < 64; k += 2)
              top[(k >> 1) & 3] = max3(top[(k >> 1) & 3], __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
          }
          top[0] = fmaxf(max3(top[0], top[1], top[2]), top[3]);
          const float mt = top[0] == -INFINITY ? -INFINITY : top[0] * f;
          const bool grows = mt - m > slack_of(m);  // (false for two infinities)
          if (__any_sync(0xffffffffu, grows || far_off(m))) {
            // a new reference: the sum so far and O go by 2^(old - new)
            const float a = grows ? exp2_fast(m - mt) : 1.f;
            if (grows) m = mt;
            l *= a;
            lost *= a;
            if (i > i0) {  // the product of the tile before is in: it was issued before these scores
#pragma unroll 1
              for (int k = 0; k < D / 16; ++k) times(ot + k * 16, a);
            }
            // scores of rows far off are multiplied where they lie: rarely, and in little code
            if (__any_sync(0xffffffffu, far_off(m))) {
#pragma unroll 1
              for (int k = 0; k < kKeys / 16; ++k) times(st + k * 16, far_off(m) ? f : 1.f);
              tmem_wait_st();
            }
          }
          const float off = kShift - (m == -INFINITY ? 0.f : m);
          const float f1 = far_off(m) ? 1.f : f;
          const float2 f2 = make_float2(f1, f1), off2 = make_float2(off, off);
          float2 sum = make_float2(0.f, 0.f), sum2 = sum;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            scores(half, x);
            uint32_t y[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              float2 w = fma2(make_float2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), f2, off2);
              w.x = exp2_fast(w.x);
              w.y = exp2_fast(w.y);
              if (k & 1) sum2 = add2(sum2, w);
              else sum = add2(sum, w);
              y[k] = pack2<__half>(w.x, w.y);
            }
            tmem_st32(st + half * 32, y);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[2 * t + half]);
          }
          sum = add2(sum, sum2);
          add_up(l, lost, sum.x + sum.y);
        }
      }
      l += lost;
      if (!ok) break;

      // the unit's output, or its part
      if (mine > 0) {
        ok = warp_wait_brief(&o_full[t], used & 1, abort_flag);
        ++used;
        if (!ok) break;
        tc_fence_after();
      }
      float* part = part_at();
      const bool chained = mine > kChain;  // O holds what came behind the sums in the workspace
      const float before = chained && m > -INFINITY ? exp2_fast(*part_stats() - m) : 0.f;
      // Rows go out through the warp's part of the q tile, which its products have
      // read, so that a store covers whole rows.
      const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t x[32];
        if (mine > 0) {
          tmem_ld32(ot + c * 32, x);
          tmem_wait_ld();
          if (chained) {
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              const float4 z = plus(*sums_at(c, k >> 2), before, x + k);
              x[k] = __float_as_uint(z.x);
              x[k + 1] = __float_as_uint(z.y);
              x[k + 2] = __float_as_uint(z.z);
              x[k + 3] = __float_as_uint(z.w);
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = 0u;
        }
        if (whole) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              y[j] = pack2<T>(__uint_as_float(x[k * 8 + 2 * j]) * inv * ev,
                              __uint_as_float(x[k * 8 + 2 * j + 1]) * inv * ev);
            const int pc = c * 4 + k;
            st_shared_v4(sq + (pc >> 3) * (128 * 128) + rr * 128 + (((pc & 7) ^ (rr & 7)) << 4), y[0],
                         y[1], y[2], y[3]);
          }
        } else {
          // a part's 32 fp32 columns: eight lanes a row
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k)
            st_shared_v4(sq + rr * 128 + ((k ^ (rr & 7)) << 4), x[4 * k], x[4 * k + 1], x[4 * k + 2],
                         x[4 * k + 3]);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r1 = i * 4 + (lane >> 3), r = (warp & 3) * 32 + r1, k = lane & 7;
            uint4 y;
            ld_shared_v4(sq + r * 128 + ((k ^ (r & 7)) << 4), y.x, y.y, y.z, y.w);
            if ((rows >> r1) & 1)
              *reinterpret_cast<uint4*>(part + (int64_t)(t * 128 + r) * D + c * 32 + k * 4) = y;
          }
        }
      }
      if (whole) {
        __syncwarp();
#pragma unroll 8
        for (int i = 0; i < LPR; ++i) {
          const int r1 = i * RPI + sub, r = (warp & 3) * 32 + r1;
          const int64_t at = __shfl_sync(0xffffffffu, row, r1);
          uint4 y;
          ld_shared_v4(sq + (piece >> 3) * (128 * 128) + r * 128 + (((piece & 7) ^ (r & 7)) << 4), y.x, y.y,
                       y.z, y.w);
          if ((rows >> r1) & 1)
            *(reinterpret_cast<uint4*>(static_cast<T*>(p.o) + at * D) + piece) = y;
        }
      }
      __syncwarp();
      tc_fence_before();
      if (valid && whole) {
        if (p.lse) p.lse[row] = (m - kShift + log2f(l)) * kLn2;
      } else if (valid) {
        *reinterpret_cast<float4*>(part_stats()) = make_float4(m, l, ev, 0.f);
      }
    }
  } else if (warp < kIssue) {
    // ------------------------------------------------------------ codes to f16
    regs_dec<kRegsConvert>();
    constexpr int kLoads = kKeys * D / 16 / kConvert;  // 16-byte pieces of a thread
    constexpr int kPieces = D / 16;                    // of a row
    const int cw = warp - 8;
    // eight lanes that store together write two rows, so that no bank is met twice
    const int piece = D == 128 ? (lane & 3) + 4 * (lane >> 4) : lane & 3;
    const int sub = D == 128 ? cw * 4 + ((lane >> 2) & 3) : cw * 8 + (lane >> 2);
    constexpr int kRowsPerLoad = kConvert / kPieces;
    // place of this thread's first eight codes in a slot; the next eight are beside
    // them, which the swizzle keeps at an address that differs in bit 4 alone
    const uint32_t store_at = (piece >> 2) * (kKeys * 128) + sub * 128 +
                              ((((piece & 3) * 2) ^ (sub & 7)) << 4);
    int u = 0;
    for (int seg = 0;; ++seg) {
      if (!(ok = wait_unit(seg))) break;
      const Unit& unit = unit_at(seg);
      const int n = max(unit.c[0], unit.c[1]), first = unit.tile * kKeys, kv = unit.kv, h = unit.h;
      if (unit.n < 0) break;
      const int* ids = p.table + (int64_t)unit.b * p.max_pages;
      const float kinv = unit.ek > 0.f ? 1.f / unit.ek : 0.f;
      const float vinv = unit.ev > 0.f ? 1.f / unit.ev : 0.f;
      release_unit(seg);
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
      // A tile's loads: `row` is the first row of codes of the lane's 16 tokens
      // (-1: none there).
      auto row_of = [&](int id) {
        return id >= 0 ? (int)((((int64_t)id * p.Hkv + h) << p.page_log2) +
                               (((lane & 7) * 16) & ((1 << p.page_log2) - 1)))
                       : -1;
      };
      auto load = [&](uint4 (&x)[kLoads], int i, int row, int which) {
        const uint8_t* codes = p.codes[which] + piece * 16;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
          const int r = j * kRowsPerLoad + sub;
          const int at = __shfl_sync(0xffffffffu, row, r >> 4);
          x[j] = load_codes(codes + (int64_t)(at + (r & 15)) * D,
                            at >= 0 && first + i * kKeys + r < kv);
        }
      };
      // (the factor as a product of two: one of 2^-14 or more leaves every code exact, so
      // a second one rounds once)
      auto store = [&](const uint4 (&x)[kLoads], float factor, int slot) {
        const uint32_t dst = base + L::kSlotOff + slot * L::kSlot + store_at;
        const bool two = factor < 0x1p-14f;  // (a NaN stays in the first)
        const uint32_t fw = pack2<__half>(two ? 0x1p-14f : factor, two ? factor * 0x1p14f : 1.f);
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
          const uint32_t fj = __shfl_sync(0xffffffffu, fw, (j * kRowsPerLoad + sub) >> 4);
          const bool one = fj == 0x3c003c00u;  // as for most pages: no product needed
          const uint32_t c[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
          uint32_t y[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t lo, hi;
            e4m3x4_to_f16x4(c[k], lo, hi);
            y[2 * k] = lo;
            y[2 * k + 1] = hi;
          }
          if (!one) {
            const __half2 f2 = *reinterpret_cast<const __half2*>(&fj);
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = hmul2(y[k], __low2half2(f2));
            if (fj >> 16 != 0x3c00u) {
#pragma unroll
              for (int k = 0; k < 8; ++k) y[k] = hmul2(y[k], __high2half2(f2));
            }
          }
          st_shared_v4(dst + j * (kRowsPerLoad * 128), y[0], y[1], y[2], y[3]);
          st_shared_v4((dst ^ 16) + j * (kRowsPerLoad * 128), y[4], y[5], y[6], y[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&kv_full[slot]);
      };
      auto acquire = [&]() {
        return u < L::kSlots ||
               warp_wait_brief(&kv_empty[u % L::kSlots], ((u / L::kSlots) - 1) & 1, abort_flag);
      };
      uint4 xk[kLoads], xv[kLoads];
      int id = known(ask_page(0)), id1 = ask_page(1), row = row_of(id);
      float fk = ask_scale(id, 0) * kinv, fv = ask_scale(id, 1) * vinv;
      load(xk, 0, row, 0);
      for (int i = 0; i < n; ++i) {
        const int id2 = ask_page(i + 2);
        id1 = known(id1);
        const float fk1 = ask_scale(id1, 0), fv1 = ask_scale(id1, 1);
        load(xv, i, row, 1);
        if (!(ok = acquire())) break;
        store(xk, fk, u % L::kSlots);
        ++u;
        row = row_of(id1);
        load(xk, i + 1, row, 0);
        if (!(ok = acquire())) break;
        store(xv, fv, u % L::kSlots);
        ++u;
        if (cw == 0 && lane == 0) *ticks = u;
        id1 = id2;
        fk = fk1 * kinv;
        fv = fv1 * vinv;
      }
      if (!ok) break;
    }
  } else {
    regs_dec<kRegsIssue>();
    if (warp == kIssue && elect_one()) {
      // ------------------------------------------------------------ products
      // This thread's own instructions are on the path from weights to the next
      // scores, so there are few: slots and phases are counted, not divided out.
      int us = 0, up = 0;                     // slot and parity of the next K or V tile
      uint32_t p_parity = 0, q_parity = 0;    // bit t: of the next wait for row tile t
      auto slot = [&](int k) { return base + L::kSlotOff + (uint32_t)k * L::kSlot; };
      auto wait_kv = [&](int k, int par) { return mbar_wait_brief(&kv_full[k], par, abort_flag); };
      auto scores = [&](int t, uint32_t kt) {  // S = Q K^T
        const uint32_t q = base + t * L::kQ, s = tmem + t * 128;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * (128 * 128) + (kk & 3) * 32;
          mma_ss(s, smem_desc_sw128(q + off, 16, 1024), smem_desc_sw128(kt + off, 16, 1024), IDESC_QK,
                 kk > 0 ? 1u : 0u);
        }
        mma_commit(&s_full[t]);
      };
      auto next = [&]() {
        if (++us == L::kSlots) {
          us = 0;
          up ^= 1;
        }
      };
      for (int seg = 0; ok; ++seg) {
        if (!(ok = mbar_wait_brief(&u_full[seg % kPlans], (seg / kPlans) & 1, abort_flag))) break;
        const Unit& unit = unit_at(seg);
        if (unit.n < 0) break;
        const int c0 = unit.c[0], c1 = unit.c[1], n = max(c0, c1);
        mbar_arrive(&u_empty[seg % kPlans]);
        if (n == 0) continue;
        if (!(ok = wait_kv(us, up))) break;
#pragma unroll 1
        for (int t = 0; t < 2 && ok; ++t) {
          if ((t ? c1 : c0) == 0) continue;
          ok = mbar_wait_brief(&q_full[t], (q_parity >> t) & 1, abort_flag);
          if (!ok) break;
          q_parity ^= 1u << t;
          tc_fence_after();
          scores(t, slot(us));
        }
        if (!ok) break;
        mma_commit(&kv_empty[us]);
        next();
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
          const int vs = us;
          if (!(ok = wait_kv(vs, up))) break;
          next();
          if (i + 1 < n && !(ok = wait_kv(us, up))) break;
          const uint32_t vt = slot(vs), kt = slot(us);
#pragma unroll 1
          for (int t = 0; t < 2; ++t) {
            const int c = t ? c1 : c0;
            if (i >= c) continue;
            const uint32_t pt = tmem + t * 128;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              ok = mbar_wait_brief(&p_full[2 * t + h], (p_parity >> t) & 1, abort_flag);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int kk = 4 * h; kk < 4 * h + 4; ++kk)  // O += P V
                mma_ts(pt + 256, pt + kk * 8, smem_desc_sw128(vt + kk * 2048, kKeys * 128, 1024),
                       IDESC_PV, (i & (kChain - 1)) != 0 || kk > 0 ? 1u : 0u);
            }
            if (!ok) break;
            p_parity ^= 1u << t;
            if (i + 1 < c) scores(t, kt);
            else mma_commit(&o_full[t]);
          }
          if (!ok) break;
          mma_commit(&kv_empty[vs]);
          if (i + 1 < n) {
            mma_commit(&kv_empty[us]);
            next();
          }
        }
      }
      mma_commit(done);
      mbar_wait_drain(done, 0);
    } else if (warp == kPlan) {
      // ---------------------------------------------------------- plan
      for (int seg = 0;; ++seg) {
        if (seg >= kPlans)
          ok = warp_wait_working(&u_empty[seg % kPlans], ((seg / kPlans) - 1) & 1, abort_flag, ticks);
        if (!ok) break;
        Unit& unit = unit_at(seg);
        const bool more = w.pos < w.end;
        float ek = 0.f, ev = 0.f;
        if (more) {
          // the largest scales among the pages of these tiles, and the least
          float lk = INFINITY, lv = INFINITY;
          const int n = w.count(), c = max(w.count(0, n), w.count(1, n));
          const int t0 = w.tile(), stop = min(w.kv, (t0 + c) * kKeys);
          const int g1 = stop > t0 * kKeys ? ((stop - 1) >> p.page_log2) + 1 : 0;
          const int* ids = p.table + (int64_t)w.b * p.max_pages;
#pragma unroll 4
          for (int g = ((t0 * kKeys) >> p.page_log2) + lane; g < g1; g += 32) {
            const int id = __ldg(ids + g);
            if (id >= 0 && id < p.num_pages) {
              const float sk = __ldg(p.kvscale[0] + (int64_t)id * p.Hkv + w.h);
              const float sv = __ldg(p.kvscale[1] + (int64_t)id * p.Hkv + w.h);
              ek = fmaxf(ek, sk);
              ev = fmaxf(ev, sv);
              if (sk > 0.f) lk = fminf(lk, sk);
              if (sv > 0.f) lv = fminf(lv, sv);
            } else {
              atomicOr(p.status, kDevBadIndex);
            }
          }
#pragma unroll
          for (int k = 16; k > 0; k >>= 1) {
            ek = fmaxf(ek, __shfl_xor_sync(0xffffffffu, ek, k));
            ev = fmaxf(ev, __shfl_xor_sync(0xffffffffu, ev, k));
            lk = fminf(lk, __shfl_xor_sync(0xffffffffu, lk, k));
            lv = fminf(lv, __shfl_xor_sync(0xffffffffu, lv, k));
          }
          if (lk < ek * 0x1p-15f) ek *= 0x1p-7f;
          if (lv < ev * 0x1p-15f) ev *= 0x1p-7f;
        }
        if (lane == 0) {
          unit.n = -1;
          if (more) {
            const int n = w.count();
            unit.b = w.b;
            unit.h = w.h;
            unit.qt = w.qt;
            unit.tile = w.tile();
            unit.n = n;
            unit.c[0] = w.count(0, n);
            unit.c[1] = w.count(1, n);
            unit.kv = w.kv;
            unit.nq = w.nq;
            unit.begins = w.tile() == 0;
            unit.ends = w.tile() + n == w.tiles;
            unit.follow =
                unit.begins && !unit.ends ? shares.behind(blockIdx.x, w.pos + w.tiles + kUnitCost - w.at.x)
                                           : 0;
            unit.ek = ek;
            unit.ev = ev;
          }
          mbar_arrive(&u_full[seg % kPlans]);
        }
        __syncwarp();
        if (!more) break;
        w.next(p);
      }
    }
  }
  if (!ok) give_up(p.status, abort_flag);
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
cudaError_t launch_typed(const AttendParams& p, int ctas, bool whole, cudaStream_t stream) {
  constexpr int bytes = PromptLayout<D>::kBytes;
  static_assert(bytes <= 227 * 1024, "shared memory");
  const cudaError_t e = allow_shared<prompt_kernel<T, D>>(bytes);
  if (e != cudaSuccess) return e;
  prompt_kernel<T, D><<<ctas, kThreads, bytes, stream>>>(p, whole);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_prompt(const AttendParams& p, la_dtype dtype, int d, int ctas, bool whole,
                                cudaStream_t stream) {
  if (d == 64)
    return dtype == LA_BF16 ? launch_typed<__nv_bfloat16, 64>(p, ctas, whole, stream)
                            : launch_typed<__half, 64>(p, ctas, whole, stream);
  return dtype == LA_BF16 ? launch_typed<__nv_bfloat16, 128>(p, ctas, whole, stream)
                          : launch_typed<__half, 128>(p, ctas, whole, stream);
}

}  // namespace la
