// la_cache_token.cu -- attention of one or a few new tokens over the 8-bit cache.
//
// For the G query heads of a kv head and the n <= 32 / G tokens of a sequence,
// R = n G rows in all, with codes c and page scales a (keys), b (values):
//     s_rj = (q_r . c_j) a_j scale,   p_rj = exp(s_rj - m_r),   o_r = sum_j p_rj b_j c'_j / sum_j p_rj
// over the cached tokens j that row r sees.  Each cached byte is used by R rows
// only, 2 R flops a byte, so the cache's bytes from HBM bound it; the kernel is
// built to keep copies in flight and to do little work for each byte.
//
// - A unit is a (sequence, kv head); its keys go by in tiles of 64 tokens.  One
//   warp issues the tiles' bulk tensor copies (a page's rows of one head are
//   contiguous; 128- or 64-byte swizzle so that the reads below meet no bank
//   twice) through a ring of stages, on across unit boundaries.
// - Four warps take 16 tokens of a tile each, with a running maximum, sum and
//   output of their own, so nothing is exchanged until a unit ends.
// - Codes become f16 in registers (exact), two for each conversion, straight in
//   the layout of the products' operands: the sum over d may run in any
//   order, so a lane's 16-byte pieces of a key row are its operand pieces of eight
//   16-wide steps as they lie; for the values, pairs of tokens are put side
//   by side by byte permutes.  No pass through shared memory.
// - The products are mma.sync m16n8k16 (f16 in, fp32 sums): 16 rows at 2 R
//   flops a byte are far from the tensor limits, and tcgen05 would need the
//   converted tile in shared memory.
// - Up to eight rows (FEW) are the 8-wide side of the products, S^T = K Q^T and
//   O^T = V^T P^T: half the products, exponentials and sums of the other way round
//   (more rows are its 16-wide side).  Weights come out of the first as tokens x rows
//   and are turned by movmatrix.  256 sequences, groups of four: 231 us the other
//   way, 206 this; a million tokens, 8 heads, one row each: 334 and 320 (198 and 314 with
//   the values loaded before the softmax, which leaves the stage free half a step
//   earlier).
// - q is scaled by a power of two for each row so that its largest entry lies in
//   [2^14, 2^15) before it is rounded to f16: exact down to 2^-28 of the largest.
// - Weights go to f16 as 2^7 p b_j / v, v the largest value scale so far (a power
//   of two) and p relative to a reference maximum of the row that follows the true
//   one only when that has grown by more than 2^8: the sums are rescaled then, or
//   when v grows.  Weights down to 2^-32 of the largest count.  Rounding them to f16
//   is 2^-11 each, of the size of the output's own rounding to fp16.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "la_cache.cuh"
#include "la_ptx.cuh"

namespace la {
namespace {

constexpr int kTile = 64;        // tokens of a stage
constexpr int kConsumers = 128;  // four warps
constexpr int kThreads = kConsumers + 32;
constexpr float kShift = kAttendShift;
// Tokens whose products a warp's sums in registers take up; then they are added to those in
// its buffer and begin again.  The products cut off what lies below the sum's last places and
// do not round it: over 2^18 tokens, all values 1, o was 0.998 to 0.999.  (256 sequences 198.3
// us without, 199.3 with; at 32 rows 121 and 125.)
constexpr int kChain = 4096;

// RG row groups of 16 rows: with one, two warps take a stage's 64 tokens, 32 each,
// and the other two the next stage's; with two, all four take every stage, two for each
// row group (a warp that held both groups' outputs would not fit its registers: rows
// 32, 32 x 8 heads, up to 8192 tokens: 158 us against 113).
template <int D, int ROWS>
struct TokenLayout {
  static constexpr int RG = ROWS == 32 ? 2 : 1;
  static constexpr int kRows = ROWS;
  static constexpr int kSub = 2;           // groups of 16 tokens that a warp takes at a time
  static constexpr int kSharers = 2 * RG;  // warps that read a stage
  static constexpr int kStages = D == 128 ? 5 - RG : 7 - RG;
  // (of one unit a stage is always the same two warps', so they wait for each filling)
  static_assert(RG == 2 || kStages % 2 == 0, "stages of two pairs of warps in turn");
  static constexpr int kHalf = kTile * D;             // bytes of a K or V tile
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kQOff = kStages * kStage;       // Q fragments
  static constexpr int kRawOff = kQOff + ROWS * D * 2;  // two units' q as they come
  static constexpr int kRaw = kRows * D * 2;
  static constexpr int kBufOff = kRawOff + 2 * kRaw;
  static constexpr int kBuf = ROWS / RG * (D + 4) * 4;  // a warp's fp32 output, rows padded
  static constexpr int kStatOff = kBufOff + 4 * kBuf;    // wm[4][16], wl[4][16], wv[4], rs[rows]
  static constexpr int kScaleOff = kStatOff + (8 * 16 + 4 + kRows) * 4;  // float2 [stages][4]
  static constexpr int kBarOff = (kScaleOff + kStages * 4 * 8 + 7) / 8 * 8;
  static constexpr int kMiscOff = kBarOff + (2 * kStages + 5) * 8;  // scan scratch, start, abort
  static constexpr int kBytes = kMiscOff + 128 + 1024;        // + slack to align to 1024
};

__device__ __forceinline__ void mma16816(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// Of an 8 x 8 matrix of 16-bit numbers (lane 4 r + c: columns 2c, 2c + 1 of row r) the
// transpose, likewise.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* tmap, uint64_t* bar, int c0,
                                            int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// A block's walk along its share [pos, end) of the line.
struct Walk {
  int64_t pos, end;  // the next place and the share's end
  int b, h;          // unit of that place
  Place at;          // where in the unit
  int tiles;         // tiles of the unit (0: sequence without work)
  int kv, nq;        // its lengths
  bool whole;        // units are not cut: `pos` counts units, every gridDim.x-th

  __device__ void load(const AttendParams& p) {
    const int64_t len = p.kv_len[b], n = p.q_len ? (int64_t)p.q_len[b] : p.N;
    const bool ok = attend_lengths_ok(len, n, p);
    kv = (int)len;
    nq = (int)n;
    tiles = ok && n > 0 ? max(1, (int)((len + kTile - 1) / kTile)) : 0;
  }
  // places that a unit of this sequence takes
  __device__ int places() const { return tiles ? tiles + kUnitCost : 0; }
  __device__ int tile() const { return whole ? 0 : at.tile(); }
  // the unit's tiles in this share: from tile(), as many as returned
  __device__ int count() const { return whole ? tiles : at.count(tiles, end - pos); }
  // whole units: from unit `pos` on to the next of this block's that has work
  __device__ void settle(const AttendParams& p) {
    for (; pos < end; pos += gridDim.x) {
      b = (int)pos / p.Hkv;
      h = (int)pos - b * p.Hkv;
      load(p);
      if (tiles) return;
    }
  }
  // on to the next unit that has tiles (the share goes on, or ends before its first)
  __device__ void next(const AttendParams& p) {
    if (whole) {
      pos += gridDim.x;
      settle(p);
      return;
    }
    pos += places() - at.x;
    at.x = 0;
    if (pos + kUnitCost >= end) pos = end;
    if (pos >= end) return;
    if (++h < p.Hkv) return;
    h = 0;
    do {
      ++b;
      if (b >= p.B) return;
      load(p);
    } while (tiles == 0);
  }
};

template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(kThreads, D == 128 ? 2 : 3)
    token_kernel(const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v, const AttendParams p, int box, bool whole) {
  using L = TokenLayout<D, ROWS>;
  constexpr int RG = L::RG;
  constexpr bool FEW = ROWS == 8;
  constexpr int KS = D / 16;  // 16-wide steps of q . k
  constexpr int NB = D / 8;   // 8-wide blocks of the output
  constexpr int SUB = L::kSub;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  float* buf = reinterpret_cast<float*>(sm + L::kBufOff);
  float* wm = reinterpret_cast<float*>(sm + L::kStatOff);
  float* wl = wm + 4 * 16;
  float* wv = wl + 4 * 16;
  float* rs = wv + 4;
  float2* sscale = reinterpret_cast<float2*>(sm + L::kScaleOff);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::kBarOff);
  uint64_t* empty = full + L::kStages;
  uint64_t* q_full = empty + L::kStages;     // [2] a unit's q has come; it has been read
  uint64_t* q_empty = q_full + 2;
  uint64_t* consumers = q_empty + 2;         // a barrier of the four warps
  int64_t* misc = reinterpret_cast<int64_t*>(sm + L::kMiscOff);  // [0, 5) scan, then the start
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 12);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], L::kSharers);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 4);
    }
    mbar_init(consumers, 4);
    *abort_flag = 0;
    fence_barrier_init();
  }

  // The line's length, this block's share of it, and the unit where that begins; whole
  // units are counted out.
  Walk w;
  int64_t total;
  Shares shares(0, 0);
  w.whole = whole;
  if (whole) {
    w.pos = blockIdx.x;
    w.end = (int64_t)p.B * p.Hkv;
    w.settle(p);
    __syncthreads();  // barriers are set up
    if (w.pos >= w.end) return;
  } else {
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min((int)threadIdx.x * per, p.B), b1 = min(b0 + per, p.B);
    int64_t mine = 0;
    for (w.b = b0; w.b < b1; ++w.b) {
      w.load(p);
      mine += (int64_t)w.places() * p.Hkv;
    }
    int64_t before = block_exclusive_sum<kThreads>(mine, misc, total);
    shares = Shares(total, gridDim.x);
    w.pos = w.end = 0;
    if ((int)blockIdx.x < shares.n) {
      w.pos = shares.begin(blockIdx.x);
      w.end = shares.begin(blockIdx.x + 1);
    }
    if (w.pos < w.end && before <= w.pos && w.pos < before + mine) {
      for (w.b = b0;; ++w.b) {
        w.load(p);
        if (w.pos < before + (int64_t)w.places() * p.Hkv) break;
        before += (int64_t)w.places() * p.Hkv;
      }
      misc[6] = w.b;
      misc[7] = div_short(w.pos - before, w.places());
      misc[8] = w.pos - before - misc[7] * w.places();
    }
    __syncthreads();
    if (w.pos >= w.end) {
      if (threadIdx.x == 0) p.tails[blockIdx.x] = make_int4(0, 0, 0, 0);
      griddep_launch_dependents();
      return;
    }
    w.b = (int)misc[6];
    w.h = (int)misc[7];
    w.at.x = (int)misc[8];
    w.load(p);
    if (w.count() == 0) w.next(p);  // a share that ends, or goes on, behind this unit's cost
  }

  if (warp == 4) {
    // ------------------------------------------------------------ copies
    // A lane knows the page and scales of 16 tokens: 32 lanes, eight tiles.  They are
    // asked for ahead, on across units: scales while the eight tiles before go by,
    // page numbers another eight before that (32 x 8 heads, 32 rows: 125 us without,
    // 122 with).
    if (lane == 0) {
      prefetch_tmap(&map_k);
      prefetch_tmap(&map_v);
    }
    const int per_box = box / 16;        // 16-token groups of a copy
    const uint32_t bytes = (uint32_t)box * D;
    Walk ahead = w;   // the eight tiles whose page numbers are asked for next: of this
    int ahead_at = 0;  // unit, from this of its tiles in the share on
    auto ask_pages = [&](int& h) {  // page of the lane's tokens (-2: none), the unit's head
      int id = -2;
      h = ahead.h;
      if (ahead.pos < ahead.end) {
        const int64_t group = (int64_t)(ahead.tile() + ahead_at) * 4 + lane;
        if (group * 16 < ahead.kv)
          id = p.table[(int64_t)ahead.b * p.max_pages + (group >> (p.page_log2 - 4))];
        ahead_at += 8;
        if (ahead_at >= ahead.count()) {
          ahead.next(p);
          ahead_at = 0;
        }
      }
      return id;
    };
    auto ask_scales = [&](int& id, int h, float& ks, float& vs) {
      const bool known = id >= 0 && id < p.num_pages;
      ks = -1.f;  // not a scale: the group's codes count as zero
      vs = 0.f;
      if (known) {
        ks = __ldg(p.kvscale[0] + (int64_t)id * p.Hkv + h);
        vs = __ldg(p.kvscale[1] + (int64_t)id * p.Hkv + h);
      } else {
        if (id != -2) atomicOr(p.status, kDevBadIndex);
        id = -1;
      }
    };
    int h1, h2, id1 = ask_pages(h1), id2 = ask_pages(h2);
    float ks1, vs1;
    ask_scales(id1, h1, ks1, vs1);
    int it = 0;
    bool go = true;
    int unit = 0, asked = 0;  // units; units whose q has been asked for
    for (; w.pos < w.end && go; ++unit) {
      const int n = w.count();
      {  // q: a row for each lane
        const int R = w.nq * p.G, qs = unit & 1;
        if (unit >= 2) go = warp_wait(&q_empty[qs], ((unit >> 1) - 1) & 1, p.status, abort_flag);
        if (!go) break;
        if (lane == 0) mbar_arrive_expect_tx(&q_full[qs], (uint32_t)R * D * 2);
        asked = unit + 1;
        __syncwarp();
        if (lane < R) {
          const int64_t row = ((int64_t)w.b * p.Hq + w.h * p.G + lane % p.G) * p.N + lane / p.G;
          bulk_load(base + L::kRawOff + qs * L::kRaw + lane * D * 2,
                    static_cast<const T*>(p.q) + row * D, D * 2, &q_full[qs]);
        }
      }
      int id = -1;
      float ks = 0.f, vs = 0.f;
      for (int i = 0; i < n && go; ++i, ++it) {
        const int t = w.tile() + i;
        if ((i & 7) == 0) {
          id = id1;
          ks = ks1;
          vs = vs1;
          id1 = id2;
          ask_scales(id1, h2, ks1, vs1);
          id2 = ask_pages(h2);
        }
        const int s = it % L::kStages;
        if (it >= L::kStages)
          go = warp_wait(&empty[s], ((it / L::kStages) - 1) & 1, p.status, abort_flag);
        if (!go) break;
        const int g0 = (i & 7) * 4;  // first lane of this tile's groups
        if (lane >= g0 && lane < g0 + 4) sscale[s * 4 + lane - g0] = make_float2(ks, vs);
        const bool issue = lane >= g0 && lane < g0 + 4 && (lane & (per_box - 1)) == 0 && id >= 0;
        const uint32_t copies = __popc(__ballot_sync(0xffffffffu, issue));
        __syncwarp();
        if (lane == 0) {
          if (copies) mbar_arrive_expect_tx(&full[s], copies * 2 * bytes);
          else mbar_arrive(&full[s]);
        }
        __syncwarp();
        if (issue) {
          const int at = (lane - g0) * 16;  // token of the tile
          const int first = t * kTile + at;
          const int64_t code_row = (((int64_t)id * p.Hkv + w.h) << p.page_log2) +
                                   (first & ((1 << p.page_log2) - 1));
          const uint32_t dst = base + s * L::kStage + at * D;
          tma_load_2d(dst, &map_k, &full[s], 0, (int)code_row);
          tma_load_2d(dst + L::kHalf, &map_v, &full[s], 0, (int)code_row);
        }
      }
      if (go) w.next(p);
    }
    if (*abort_flag) {  // let copies already issued land before the block exits
      for (int k = max(0, it - L::kStages); k < it; ++k)
        mbar_wait_drain(&full[k % L::kStages], (k / L::kStages) & 1);
      for (int k = max(0, unit - 1); k <= unit; ++k)
        if (k < asked) mbar_wait_drain(&q_full[k & 1], (k >> 1) & 1);
    }
    return;
  }

  // -------------------------------------------------------------- products
  // r / G for a row r < 32, G <= 32: the error of 2^16 / G, at most 1, times r stays
  // below 2^16 / G
  const int per_g = 65536 / p.G + 1;
  auto token_of = [&](int r) { return r * per_g >> 16; };
  const int g = lane >> 2, c = lane & 3, rg = RG == 2 ? warp >> 1 : 0;
  const uint32_t sq = base + L::kQOff;
  // plain loads: the compiler places them, behind the waits that order them
  auto lds128 = [&](uint32_t addr) { return *reinterpret_cast<const uint4*>(sm + (addr - base)); };
  auto lds64 = [&](uint32_t addr) { return *reinterpret_cast<const uint2*>(sm + (addr - base)); };
  int it = 0, syncs = 0;
  auto sync = [&]() { return warps_sync(consumers, syncs, p.status, abort_flag); };
  int4 tail = make_int4(0, 0, 0, 0);
  bool ok = true;
  int unit = 0;
  for (; w.pos < w.end && ok; ++unit) {
    const int n = w.count();
    const int R = w.nq * p.G, first_tile = w.tile();
    ok = warp_wait(&q_full[unit & 1], (unit >> 1) & 1, p.status, abort_flag);
    if (!ok) break;
    // q: rows as f16 operand pieces in shared memory, with each row's factor.  TPR
    // threads a row.  The sign of the scale goes into q, so that the factor is not
    // negative.
    constexpr int TPR = kConsumers / (ROWS / RG), V = D / TPR;  // threads and a thread's values
#pragma unroll
    for (int mt = 0; mt < RG; ++mt) {
      const int r = mt * 16 + threadIdx.x / TPR, e = threadIdx.x % TPR;
      const uint32_t from = base + L::kRawOff + (unit & 1) * L::kRaw + r * D * 2 + e * V * 2;
      float x[V];
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        uint2 q2 = make_uint2(0u, 0u);
        if (r < R) q2 = lds64(from + j * 2);
        const float2 f0 = unpack2<T>(q2.x), f1 = unpack2<T>(q2.y);
        x[j] = f0.x;
        x[j + 1] = f0.y;
        x[j + 2] = f1.x;
        x[j + 3] = f1.y;
        top = max3(max3(top, fabsf(f0.x), fabsf(f0.y)), fabsf(f1.x), fabsf(f1.y));
      }
#pragma unroll
      for (int k = TPR / 2; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
      // largest entry into [2^14, 2^15); rows of zeros, infinities and NaN as they are
      const int ex = (int)(__float_as_uint(top) >> 23) - 127;
      const int up = top > 0.f && ex < 128 ? min(14 - ex, 126) : 0;
      if (e == 0) rs[r] = fabsf(p.scale) * kLog2e * pow2i(-up);
      const float f = p.scale < 0.f ? -pow2i(up) : pow2i(up);
#pragma unroll
      for (int j = 0; j < V; j += 2) {
        const int d = e * V + j;
        const int cc = d / (D / 4), ks = (d % (D / 4)) / 4, pair = (d & 3) >> 1;
        const uint32_t at = FEW ? sq + (ks * 32 + r * 4 + cc) * 8 + pair * 4
                                : sq + (((mt * KS + ks) * 32 + (r & 7) * 4 + cc) * 16) +
                                      (pair * 2 + ((r >> 3) & 1)) * 4;
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(pack2<__half>(x[j] * f, x[j + 1] * f))
                     : "memory");
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&q_empty[unit & 1]);
    if (!(ok = sync())) break;

    // What a lane holds of the scores and the output: of two rows, g and g + 8 (2c and
    // 2c + 1 for FEW), the row of number x of four being
    auto row_of = [](int x) { return FEW ? x & 1 : x >> 1; };
    constexpr int OB = FEW ? NB / 2 : NB;
    float o[OB][4], m[2], l[2], lost[2], rf[2];
    int last[2];  // last token that the row sees
    {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = FEW ? 2 * c + k : rg * 16 + k * 8 + g;
        m[k] = -INFINITY;
        l[k] = lost[k] = 0.f;
        rf[k] = rs[r];
        last[k] = r < R ? w.kv - w.nq + token_of(r) : w.kv - 1;
      }
#pragma unroll
      for (int j = 0; j < OB; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[j][k] = 0.f;
    }
    float vref = 0.f, vinv = 0.f;
    // Adds the warp's sums to those in its buffer (if that has some of this unit: `held`) and notes
    // what they are relative to.
    auto put_by = [&](bool held) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = FEW ? 2 * c + k : k * 8 + g;
        const float a =
            held && m[k] > -INFINITY ? exp2_fast(wm[warp * 16 + r] - m[k]) * (wv[warp] * vinv) : 0.f;
        auto add = [&](float* at, float x, float y, float z, float w) {
          float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
          if (held) b = *reinterpret_cast<const float4*>(at);
          *reinterpret_cast<float4*>(at) =
              make_float4(fmaf(b.x, a, x), fmaf(b.y, a, y), fmaf(b.z, a, z), fmaf(b.w, a, w));
        };
        if constexpr (FEW) {
          // columns D / 8 g on, D / 8 of them
          float* at = buf + warp * (L::kBuf / 4) + r * (D + 4) + g * NB;
#pragma unroll
          for (int j = 0; j < OB; j += 2) add(at + 2 * j, o[j][k], o[j][2 + k], o[j + 1][k], o[j + 1][2 + k]);
        } else {
          // piece j / 4 of column block 2c + jj: no two lanes of a store on one bank
          float* at = buf + warp * (L::kBuf / 4) + r * (D + 4) + 2 * c * 4;
#pragma unroll
          for (int jj = 0; jj < 2; ++jj)
#pragma unroll
            for (int j = 0; j < OB; j += 4)
              add(at + (j / 4) * (D / NB * 4) + jj * 4, o[j][2 * k + jj], o[j + 1][2 * k + jj],
                  o[j + 2][2 * k + jj], o[j + 3][2 * k + jj]);
        }
      }
      __syncwarp();  // all have read what the sums so far were relative to
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if ((FEW ? g : c) == 0) wm[warp * 16 + (FEW ? 2 * c + k : k * 8 + g)] = m[k];
      if (lane == 0) wv[warp] = vref;
      __syncwarp();
#pragma unroll
      for (int j = 0; j < OB; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[j][k] = 0.f;
    };

    constexpr int SKIP = 2 / RG;  // a warp takes one of so many tiles
    constexpr int kChainTiles = kChain * 4 / (kTile * RG);
    for (int i = 0; i < n; ++i, ++it) {
      if (RG == 1 && ((i ^ (warp >> 1)) & 1)) continue;  // the other two warps' stage
      if (i >= kChainTiles && (i & (kChainTiles - SKIP)) == 0) put_by(i >= 2 * kChainTiles);
      const int s = it % L::kStages;
      ok = warp_wait(&full[s], (it / L::kStages) & 1, p.status, abort_flag);
      if (!ok) break;
      const int g0 = (warp & 1) * SUB;          // first of this warp's groups
      const int t0 = (first_tile + i) * kTile + g0 * 16;      // and its first token
      if (t0 >= w.kv) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);
        continue;
      }
      float2 sc[SUB];
#pragma unroll
      for (int u = 0; u < SUB; ++u) sc[u] = sscale[s * 4 + g0 + u];
      const uint32_t kb = base + s * L::kStage + g0 * 16 * D, vb = kb + L::kHalf;
      // rows of the stage that hold no token, or a page that is not known (or, behind
      // the last token, was not copied): codes of zero
      const bool edge = t0 + 16 * SUB > w.kv || sc[0].x < 0.f || sc[SUB - 1].x < 0.f;
      // scores: of a group, 16 rows x 16 tokens in two blocks; for FEW, 16 tokens x 8 rows in
      // one.  Of row k of the lane's two, score j < SC and its token in the group:
      constexpr int SB = FEW ? SUB : 2 * SUB, SC = FEW ? 2 : 4;
      float sr[SB][4];
      auto score = [&](int u, int k, int j) -> float& {
        return FEW ? sr[u][2 * j + k] : sr[(2 * u + (j >> 1)) % SB][2 * k + (j & 1)];
      };
      auto token = [&](int j) { return FEW ? g + 8 * j : (j >> 1) * 8 + 2 * c + (j & 1); };
#pragma unroll
      for (int nb = 0; nb < SB; ++nb)
#pragma unroll
        for (int k = 0; k < 4; ++k) sr[nb][k] = 0.f;
      // values: of a group tokens 2c, 2c + 1, 2c + 8, 2c + 9, D / 8 numbers each from
      // (D / 8) g on
      uint32_t vw[FEW ? SUB : 1][4][D / 32];
      auto load_values = [&](int u, uint32_t (&x)[4][D / 32]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row = u * 16 + 2 * c + (k & 1) + (k >> 1) * 8;
          if constexpr (D == 128) {
            const uint4 y = lds128(vb + row * D + ((g ^ (row & 7)) << 4));
            x[k][0] = y.x; x[k][1] = y.y; x[k][2] = y.z; x[k][3] = y.w;
          } else {
            const uint2 y = lds64(vb + row * D + (((g >> 1) ^ ((row >> 1) & 3)) << 4) + (g & 1) * 8);
            x[k][0] = y.x; x[k][1] = y.y;
          }
        }
      };
      auto release = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);
      };
      {
        uint32_t kw[2 * SUB][KS];
#pragma unroll
        for (int nb = 0; nb < 2 * SUB; ++nb) {
          const int row = nb * 8 + g;  // of the warp's tokens (a multiple of 8 rows into the tile)
          if constexpr (D == 128) {
            const uint4 x = lds128(kb + row * D + (((2 * c) ^ g) << 4));
            const uint4 y = lds128(kb + row * D + (((2 * c + 1) ^ g) << 4));
            kw[nb][0] = x.x; kw[nb][1] = x.y; kw[nb][2] = x.z; kw[nb][3] = x.w;
            kw[nb][4] = y.x; kw[nb][5] = y.y; kw[nb][6] = y.z; kw[nb][7] = y.w;
          } else {
            const uint4 x = lds128(kb + row * D + ((c ^ ((g >> 1) & 3)) << 4));
            kw[nb][0] = x.x; kw[nb][1] = x.y; kw[nb][2] = x.z; kw[nb][3] = x.w;
          }
        }
        if (edge) {
#pragma unroll
          for (int nb = 0; nb < 2 * SUB; ++nb)
            if (sc[nb / 2].x < 0.f)
#pragma unroll
              for (int j = 0; j < KS; ++j) kw[nb][j] = 0u;
        }
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          if constexpr (FEW) {
            const uint2 q2 = lds64(sq + (ks * 32 + lane) * 8);
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
              uint4 a;
              e4m3x4_to_f16x4(kw[2 * u][ks], a.x, a.z);
              e4m3x4_to_f16x4(kw[2 * u + 1][ks], a.y, a.w);
              mma16816(sr[u], a, q2.x, q2.y);
            }
          } else {
            const uint4 a = lds128(sq + ((rg * KS + ks) * 32 + lane) * 16);
#pragma unroll
            for (int nb = 0; nb < 2 * SUB; ++nb) {
              uint32_t k0, k1;
              e4m3x4_to_f16x4(kw[nb][ks], k0, k1);
              mma16816(sr[nb], a, k0, k1);
            }
          }
        }
      }
      if constexpr (FEW) {  // there are registers for the values: the stage is free at once
#pragma unroll
        for (int u = 0; u < SUB; ++u) load_values(u, vw[u]);
        release();
      }
      // value scales: a larger one than before makes the sums relative to it
      float grow = 1.f;
      const float vtop = fmaxf(sc[0].y, sc[SUB - 1].y);
      if (vtop > vref) {
        grow = vref / vtop;
        vref = vtop;
        vinv = 1.f / vref;
      }
      if (t0 + 16 * SUB - 1 > w.kv - w.nq) {  // some row does not see some token
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < SC; ++j)
              if (t0 + u * 16 + token(j) > last[k]) score(u, k, j) = -INFINITY;
      }
      uint4 pa[SUB];
      {
        // a row's new reference maximum, where it has grown past the slack
        float f[SUB][2];
        bool grows = grow != 1.f;
        float mx[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int u = 0; u < SUB; ++u) {
            // (not zero: a masked score stays at -infinity)
            f[u][k] = max_or_nan(rf[k] * sc[u].x, 1.17549435e-38f);
            float top = fmaxf(score(u, k, 0), score(u, k, 1));
            if (!FEW) top = max3(top, score(u, k, 2 % SC), score(u, k, 3 % SC));
            mx[k] = u ? fmaxf(mx[k], top * f[u][k]) : top * f[u][k];
          }
          grows |= mx[k] - m[k] > slack_of(m[k]);  // (not for two infinities)
        }
        if (__any_sync(0xffffffffu, grows)) {
          float a[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int x = FEW ? 4 : 1; x < (FEW ? 32 : 4); x *= 2)  // the row's other lanes
              mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], x));
            const bool up = mx[k] > m[k];  // of the whole row, once any lane of the warp asks
            a[k] = up ? exp2_fast(m[k] - mx[k]) : 1.f;
            if (up) m[k] = mx[k];
            l[k] *= a[k];
            lost[k] *= a[k];
            a[k] *= grow;
          }
#pragma unroll
          for (int j = 0; j < OB; ++j)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[j][x] *= a[row_of(x)];
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float off = kShift - (m[k] == -INFINITY ? 0.f : m[k]);
          if (far_off(m[k])) {
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
#pragma unroll
              for (int j = 0; j < SC; ++j) score(u, k, j) *= f[u][k];
              f[u][k] = 1.f;
            }
          }
          float sum = 0.f;
#pragma unroll
          for (int u = 0; u < SUB; ++u) {
            const float vf = sc[u].y * vinv;
#pragma unroll
            for (int j = 0; j < SC; ++j) {
              const float e = exp2_fast(fmaf(score(u, k, j), f[u][k], off));
              sum += e;
              score(u, k, j) = e * vf;
            }
          }
          add_up(l[k], lost[k], sum);
        }
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
          if constexpr (FEW) {
            // tokens x rows as the scores lie, rows x tokens as the second operand does
            pa[u].x = transpose8x8(pack2<__half>(sr[u][0], sr[u][1]));
            pa[u].y = transpose8x8(pack2<__half>(sr[u][2], sr[u][3]));
          } else {
            const float(&x)[4] = sr[2 * u], (&y)[4] = sr[2 * u + 1];
            pa[u] = make_uint4(pack2<__half>(x[0], x[1]), pack2<__half>(x[2], x[3]),
                               pack2<__half>(y[0], y[1]), pack2<__half>(y[2], y[3]));
          }
        }
      }
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        uint32_t (&v)[4][D / 32] = vw[FEW ? u : 0];
        if constexpr (!FEW) load_values(u, v);
        if (edge) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (sc[u].x < 0.f || t0 + u * 16 + 2 * c + (k & 1) + (k >> 1) * 8 >= w.kv)
#pragma unroll
              for (int j = 0; j < D / 32; ++j) v[k][j] = 0u;
        }
        if (!FEW && u == SUB - 1) release();
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          // two tokens' bytes of a number side by side
          uint32_t b0[4], b1[4];
          e4m3x4_to_f16x4(__byte_perm(v[0][j], v[1][j], 0x5140), b0[0], b0[1]);
          e4m3x4_to_f16x4(__byte_perm(v[0][j], v[1][j], 0x7362), b0[2], b0[3]);
          e4m3x4_to_f16x4(__byte_perm(v[2][j], v[3][j], 0x5140), b1[0], b1[1]);
          e4m3x4_to_f16x4(__byte_perm(v[2][j], v[3][j], 0x7362), b1[2], b1[3]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (!FEW) mma16816(o[4 * j + k], pa[u], b0[k], b1[k]);
            else if (k % 2 == 0)
              mma16816(o[2 * j + k / 2], make_uint4(b0[k], b0[k + 1], b1[k], b1[k + 1]), pa[u].x, pa[u].y);
          }
        }
      }
    }
    if (!ok) break;

    // the four warps' parts of the unit into one: each writes its own, and all
    // threads add them up
    const bool begins = first_tile == 0, ends = first_tile + n == w.tiles;
    float* part = p.parts + ((int64_t)blockIdx.x * 2 + (begins ? 1 : 0)) * L::kRows * (D + kPartStats);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      l[k] += lost[k];
#pragma unroll
      for (int x = FEW ? 4 : 1; x < (FEW ? 32 : 4); x *= 2)
        l[k] += __shfl_xor_sync(0xffffffffu, l[k], x);
      const int r = FEW ? 2 * c + k : k * 8 + g;
      if ((FEW ? g : c) == 0) wl[warp * 16 + r] = l[k];
    }
    put_by(n > kChainTiles + (RG == 1 ? warp >> 1 : 0));
    if (!(ok = sync())) break;
    const float vmax = fmaxf(fmaxf(wv[0], wv[1]), fmaxf(wv[2], wv[3]));
    const float vdiv = vmax > 0.f ? 1.f / vmax : 0.f;
    for (int e = threadIdx.x; e < R * (D / 4); e += kConsumers) {
      const int rr = e / (D / 4), d4 = e % (D / 4), r = rr & 15;
      const int first = RG == 2 ? (rr >> 4) * 2 : 0;  // of the warps that have this row
      constexpr int PARTS = 4 / RG;
      float mx = wm[first * 16 + r];
#pragma unroll
      for (int k = 1; k < PARTS; ++k) mx = fmaxf(mx, wm[(first + k) * 16 + r]);
      const float ref = mx == -INFINITY ? 0.f : mx;
      float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < PARTS; ++k) {
        const float a = exp2_fast(wm[(first + k) * 16 + r] - ref), b = a * (wv[first + k] * vdiv);
        const float4 x = *reinterpret_cast<const float4*>(
            buf + (first + k) * (L::kBuf / 4) + r * (D + 4) +
            (FEW ? d4 * 4 : (d4 % (NB / 4)) * (D / NB * 4) + d4 / (NB / 4) * 4));
        sum += wl[(first + k) * 16 + r] * a;
        z = make_float4(z.x + x.x * b, z.y + x.y * b, z.z + x.z * b, z.w + x.w * b);
      }
      if (begins && ends) {
        const int i = token_of(rr), head = w.h * p.G + rr - i * p.G;
        const int64_t row = ((int64_t)w.b * p.Hq + head) * p.N + i;
        const float inv = sum != 0.f ? 1.f / sum : 0.f;
        uint2 out;
        out.x = pack2<T>(z.x * inv * vmax, z.y * inv * vmax);
        out.y = pack2<T>(z.z * inv * vmax, z.w * inv * vmax);
        *reinterpret_cast<uint2*>(static_cast<T*>(p.o) + row * D + d4 * 4) = out;
        if (p.lse && d4 == 0) p.lse[row] = (mx - kShift + log2f(sum)) * kLn2;
      } else {
        reinterpret_cast<float4*>(part)[rr * (D / 4) + d4] = z;
        if (d4 == 0)
          reinterpret_cast<float4*>(part + L::kRows * D)[rr] = make_float4(mx, sum, vmax, 0.f);
      }
    }
    if (begins && !ends) {
      tail = make_int4(shares.behind(blockIdx.x, w.pos + w.places() - w.at.x), w.b, w.h, 0);
    }
    w.next(p);  // (what this unit left in shared memory is written again after the next sync)
  }
  if (threadIdx.x == 0 && !whole) p.tails[blockIdx.x] = ok ? tail : make_int4(0, 0, 0, 0);
  griddep_launch_dependents();
}

template <typename T, int D, int ROWS>
cudaError_t launch_typed(const AttendParams& p, const CUtensorMap& k, const CUtensorMap& v, int box,
                         int ctas, bool whole, cudaStream_t stream) {
  constexpr int bytes = TokenLayout<D, ROWS>::kBytes;
  static_assert(bytes <= (D == 128 ? 113 : 75) * 1024, "two or three blocks for each SM");
  const cudaError_t e = allow_shared<token_kernel<T, D, ROWS>>(bytes);
  if (e != cudaSuccess) return e;
  token_kernel<T, D, ROWS><<<ctas, kThreads, bytes, stream>>>(k, v, p, box, whole);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_rows(const AttendParams& p, const CUtensorMap& k, const CUtensorMap& v, int box,
                        int rows, int ctas, bool whole, cudaStream_t stream) {
  return rows == 8    ? launch_typed<T, D, 8>(p, k, v, box, ctas, whole, stream)
         : rows == 16 ? launch_typed<T, D, 16>(p, k, v, box, ctas, whole, stream)
                      : launch_typed<T, D, 32>(p, k, v, box, ctas, whole, stream);
}

}  // namespace

cudaError_t launch_cache_token(const AttendParams& p, const la_cache& c, la_dtype dtype, int rows,
                               int ctas, bool whole, cudaStream_t stream) {
  CUtensorMap k, v;
  const int box = std::min(c.page, kTile);
  if (!make_tmap_codes(&k, c.k_codes, c.num_pages * c.Hkv * c.page, c.d, box) ||
      !make_tmap_codes(&v, c.v_codes, c.num_pages * c.Hkv * c.page, c.d, box))
    return cudaErrorInvalidValue;
  if (c.d == 64)
    return dtype == LA_BF16 ? launch_rows<__nv_bfloat16, 64>(p, k, v, box, rows, ctas, whole, stream)
                            : launch_rows<__half, 64>(p, k, v, box, rows, ctas, whole, stream);
  return dtype == LA_BF16 ? launch_rows<__nv_bfloat16, 128>(p, k, v, box, rows, ctas, whole, stream)
                          : launch_rows<__half, 128>(p, k, v, box, rows, ctas, whole, stream);
}

}  // namespace la
