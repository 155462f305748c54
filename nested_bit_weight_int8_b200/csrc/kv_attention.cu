// Attention over the paged 8-bit cache:
//   o_r = sum_j p_rj v_j,  p_rj = exp(s_rj - lse_r),  s_rj = cap(scale q_r . k_j),
//   lse_r = ln sum_j exp(s_rj),  cap(s) = softcap tanh(s / softcap) or s,
// over the tokens j <= P(r) (and > P(r) - window) of the row's sequence, P(r)
// its place. One pass over K and V with a running maximum and sum per row.
//
// Work: an item is (sequence, row tile, key/value head); its rows are the
// tile's query tokens times the heads of the group, so grouped heads share each
// byte read. The token axis of all items together is cut into equal ranges,
// one per warp of the card; ragged lengths balance by themselves and one
// long sequence fills every SM. A warp streams its range through its own ring
// of shared memory (TMA boxes of 16 tokens, swizzled), with no barrier between
// warps. Pieces of an item are joined within the CTA first, then, by a second
// kernel, over the CTAs; always in their order, so results do not depend on
// timing. Bound by the bytes: 64 sequences of up to 8192 tokens (676 MB) take 122 to 130
// us (two cards), 84% to 79% of what a copy reaches; the rest is the start of a launch and the spread of the
// warps' ends.
//
// Arithmetic: S^T = K Q^T and O^T = V^T P^T in m16n8k16 products with fp32 sums,
// the tokens (then the values of a head) on the 16 side and 8 query rows on the
// other: one product takes 256 bytes of the cache, and a tile of up to 8 rows
// wastes nothing on padding. A byte b enters as the fp16 subnormal b 2^-24, which
// takes one byte permutation per two values and no arithmetic; the offset 128
// comes out of the sums: scores start at -128 2^-24 sum(q), and outputs take one
// more product with the constant -128 2^-24. A query row (bf16)
// is scaled by a power of two to below 2 first, so fp16 holds it exactly down to
// 2^-24 of the row's largest value. Probabilities are rounded to fp16 (2^-11 of
// each), with the page's V scale relative to the largest seen folded in before;
// they stand 2^8 high, and the running maximum is raised only when a score passes
// it by 6 (base 2), so they stay below 2^14, keep their precision down to 2^-22 of
// the maximum and lose at most 2^-33 of it below. The sums of exponentials stay
// fp32 and unrounded.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "../../include/mq.h"
#include "kv_internal.h"
#include "kv_pieces.cuh"
#include "mq_device.cuh"
#include "mq_internal.h"

namespace mq {
namespace {

constexpr float kPScale = 256.f;
constexpr float kSlack = 6.f;  // base 2
constexpr float kCode = 0x1p-24f;
// V scales below this count as this (what it would gain, fp32 could not hold)
constexpr float kTinyScale = 0x1p-100f;

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Bytes 0, 1 (2, 3) of a word as the fp16 pair of byte 2^-24.
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) { return __byte_perm(w, 0u, 0x4140); }
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) { return __byte_perm(w, 0u, 0x4342); }
// The 8 x 8 fp16 matrix whose row lane / 4 holds columns 2 (lane % 4), + 1, transposed.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// D: the head's size rounded up to 64, 128 or 256. NR: query rows in eights.
// A stage holds 16-token groups: K's boxes, then V's, each of 16 rows of 64 or
// 128 bytes (two boxes side by side at D = 256), swizzled by the copy.
template <int D, int NR>
struct Shape {
  static constexpr int kRows = 8 * NR;
  // Accumulators and queries take 3 D NR / 8 registers a thread: 16 warps an SM
  // where that and 16 rings fit, else 8.
  static constexpr int kWarps = D * NR <= 128 ? 16 : 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kStages = 3;
  static constexpr int kTile = D * kWarps <= 1024 ? 32 : 16;  // tokens a stage
  static constexpr int kGroups = kTile / 16;
  // What an item costs beside its tiles, in tiles: a warp's start on an item (lengths, pages, queries, first
  // bytes, one after another) takes about as long as two 16-token tiles of a busy card. Without it one warp got
  // all 24 items of three idle rows and kept the others waiting: 167 us against 139 at 64 sequences of up to 8192.
  static constexpr int kStart = 32 / kTile;
  static constexpr int kPitch = D == 64 ? 64 : 128;
  static constexpr int kBoxes = D / kPitch;
  static constexpr int kBoxBytes = 16 * kPitch;
  static constexpr int kGroupBytes = 2 * 16 * D;
  static constexpr int kStageBytes = kGroups * kGroupBytes;
  static constexpr int kWarpBytes = kStages * kStageBytes;
  static constexpr int kSmem = kWarps * kWarpBytes + 1024;  // the base is rounded up to 1024
  static_assert(kSmem + 12288 <= 232448, "rings and the static arrays fit an SM");
};

// A warp's ring: its stages, their barriers and scales, and where it stands.
template <int D, int NR>
struct Ring {
  using S = Shape<D, NR>;
  uint32_t base;
  uint64_t* full;   // kStages
  float2* scales;   // kStages x kGroups: (K, V) scale; V < 0: nothing to see
  const void* map_k;
  const void* map_v;
  uint64_t wait_ns;
  int stage;
  uint32_t parity;
};

// How an item's rows and tokens lie.
struct RowTile {
  int i0;       // first query token of the tile
  int rows;     // rows of the tile (head-major within a token)
  int lo;       // first token that some row sees
  int j0, j1;   // lo rounded down to a tile, and the end of the tokens seen
  int tiles;    // at least 1
  int units;    // what it counts in the split
  int start;    // units before the first tile
};
template <int ROWS, int TILE, int START>
__device__ __forceinline__ RowTile row_tile(const AttendArgs& a, const Seq& s, int rt) {
  RowTile t;
  const int first = rt * ROWS, all = s.n * a.group;
  t.rows = min(ROWS, all - first);
  const bool one = all <= ROWS;  // the usual case, without the divisions
  t.i0 = one ? 0 : first / a.group;
  const int i1 = one ? s.n - 1 : (first + t.rows - 1) / a.group;
  const int base = s.len - s.n;
  t.j1 = max(base + i1 + 1, 0);
  t.lo = a.window > 0 ? max(base + t.i0 - a.window + 1, 0) : 0;
  t.j0 = t.lo & ~(TILE - 1);
  t.tiles = max((t.j1 - t.j0 + TILE - 1) / TILE, 1);
  t.start = t.j1 > 0 ? START : 0;
  t.units = t.tiles + t.start;
  return t;
}
template <int ROWS>
__device__ __forceinline__ int row_tiles(const AttendArgs& a, const Seq& s) {
  return (s.n * a.group + ROWS - 1) / ROWS;
}

template <int D, int NR>
struct Worker {
  using S = Shape<D, NR>;
  static constexpr int kMt = D / 16;  // m-tiles of the output
  static constexpr int kJ = D / 64;   // 64-value steps of a key

  // One warp's pass over tiles [t0, t1) of an item; its sums go to `part` (of
  // part_rows rows), or, if that is null, the item's outputs. False: a wait gave up.
  static __device__ __forceinline__ bool run(const AttendArgs& a, const Seq& sq, int s, int h, int rt, int t0, int t1,
                                             float* part, int part_rows, Ring<D, NR>& ring) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const RowTile it = row_tile<S::kRows, S::kTile, S::kStart>(a, sq, rt);
    const int d = a.c.d, chunks = d >> 4;
    const int first_row = rt * S::kRows;
    if (it.j1 == 0) {  // no row sees a token
      for (int lr = 0; lr < it.rows; ++lr) {
        const RowOut ro = row_out(a, sq.r0, h, first_row + lr);
        if (lane < 2 * chunks)
          *reinterpret_cast<uint4*>(a.out + ro.row * a.out_stride + int64_t(ro.head) * d + 8 * lane) = make_uint4(0, 0, 0, 0);
        if (a.lse && lane == 0) a.lse[ro.row * (a.c.heads * a.group) + ro.head] = -INFINITY;
      }
      return true;
    }

    // ---- the ring: lane i holds the page of index page0 + i and its scales, and starts its copies
    const int page = a.c.page, log2p = a.c.page_log2;
    int page0 = -32, pid = -1;
    float2 mine = make_float2(0.f, -1.f);
    auto issue = [&](int tile, int stage) {
#pragma unroll
      for (int gi = 0; gi < S::kGroups; ++gi) {
        const int j = it.j0 + tile * S::kTile + gi * 16;
        uint64_t* bar = ring.full + stage;
        float2* sc = ring.scales + stage * S::kGroups + gi;
        if (j < it.j1 && j + 16 > it.lo) {  // warp-uniform
          const int index = j >> log2p;
          if (index >= page0 + 32) {
            page0 = index;
            pid = index + lane <= (it.j1 - 1) >> log2p ? load_page(a.c, a.b, s, index + lane, a.err) : -1;
            mine = make_float2(0.f, -1.f);
            if (pid >= 0) {
              const int64_t at = int64_t(pid) * a.c.heads + h;
              mine = make_float2(a.c.k_scale[at], a.c.v_scale[at]);
            }
          }
          if (lane == index - page0) {
            if (pid >= 0) {
              const uint32_t kb = ring.base + stage * S::kStageBytes + gi * S::kGroupBytes, vb = kb + 16 * D;
              const int row = h * page + (j & (page - 1));
              mbar_expect_tx(bar, S::kGroupBytes);
#pragma unroll
              for (int x = 0; x < S::kBoxes; ++x) {
                tma_load_3d(kb + x * S::kBoxBytes, ring.map_k, 128 * x, row, pid, bar);
                tma_load_3d(vb + x * S::kBoxBytes, ring.map_v, 128 * x, row, pid, bar);
              }
            }
            *sc = mine;  // waits for the scales; the copies are on their way
            mbar_arrive(bar);
          }
        } else if (lane == 0) {
          *sc = make_float2(0.f, -1.f);
          mbar_arrive(bar);
        }
      }
    };
    uint4 raw[NR][kJ][2];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int lr = 8 * r + g, row = first_row + lr, qi = row / a.group, hg = row - qi * a.group;
      const uint16_t* qp = a.q + (sq.r0 + qi) * a.q_stride + int64_t(h * a.group + hg) * d;
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        const int c = 4 * j + t;
        const bool in = lr < it.rows && c < chunks;
#pragma unroll
        for (int k = 0; k < 2; ++k)
          raw[r][j][k] = in ? *(reinterpret_cast<const uint4*>(qp + 16 * c) + k) : make_uint4(0, 0, 0, 0);
      }
    }
    const int stage0 = ring.stage;
#pragma unroll
    for (int i = 0; i < S::kStages - 1; ++i) {
      int st = stage0 + i;
      if (st >= S::kStages) st -= S::kStages;
      if (t0 + i < t1) issue(t0 + i, st);
    }

    // ---- the queries in fragment order: lane (g, t) holds chunks 4 j + t of row g. The codes
    // enter the products as byte 2^-24 (an fp16 subnormal, exact); the sums start at
    // -128 2^-24 times the query's own sum.
    uint32_t qf[NR][kJ * 4][2];
    float fac[NR][2], bias[NR][2];   // of rows 2 t, 2 t + 1
    const float sign = a.scale < 0.f ? -1.f : 1.f;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int lr = 8 * r + g;
      float mx = 0.f;
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t w[4] = {raw[r][j][k].x, raw[r][j][k].y, raw[r][j][k].z, raw[r][j][k].w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xFFFF0000u))));
        }
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      int ex = __float_as_int(mx) >> 23;  // 2^(ex - 127) <= mx < 2^(ex - 126)
      ex = ex < 1 || ex > 253 ? 127 : ex;
      const float down = __int_as_float((254 - ex) << 23) * sign;
      const float up = __int_as_float(ex << 23) * fabsf(a.scale) * (a.softcap > 0.f ? 1.f : kLog2e);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t w[4] = {raw[r][j][k].x, raw[r][j][k].y, raw[r][j][k].z, raw[r][j][k].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // values 8 k + 2 i, + 1 of the chunk: product 4 j + 2 k + i / 2, half i % 2
            const uint32_t h2 = f16x2(__uint_as_float(w[i] << 16) * down, __uint_as_float(w[i] & 0xFFFF0000u) * down);
            qf[r][4 * j + 2 * k + i / 2][i & 1] = h2;
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
            sum += f.x + f.y;
          }
        }
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        fac[r][e] = __shfl_sync(0xffffffffu, up, 4 * (2 * t + e));
        bias[r][e] = __shfl_sync(0xffffffffu, sum, 4 * (2 * t + e)) * (-128.f * kCode);
      }
    }

    float o[NR][kMt][4];
    float m[NR][2], l[NR][2], vmax = kTinyScale, vinv = kPScale / kTinyScale;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      m[r][0] = m[r][1] = -INFINITY;
      l[r][0] = l[r][1] = 0.f;
#pragma unroll
      for (int i = 0; i < kMt; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[r][i][e] = 0.f;
    }
    // the places of the tile's first and last query token
    int lo_place = sq.len - sq.n + it.i0;
    const int hi_place = sq.len - sq.n + (first_row + it.rows - 1) / a.group;
    const float cap_in = a.softcap > 0.f ? 1.f / a.softcap : 0.f, cap_out = a.softcap * kLog2e;
    // where this lane's chunks lie in a box: K rows g ^ ((g & 1) << 2) and + 8, V rows 2 t, (2 t + 1) ^ 4 and + 8
    const int krow = g ^ ((g & 1) << 2), va_row = 2 * t, vb_row = (2 * t + 1) ^ 4;

    for (int tile = t0; tile < t1; ++tile) {
      const int stage = ring.stage;
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(ring.full + stage, ring.parity, ring.wait_ns))) {
        if (lane == 0) atomicOr(a.err, kErrWaitFull);
        // the copies in flight: this tile's and the next's
        for (int i = 0; i < S::kStages - 1 && tile + i < t1; ++i) {
          if (!mbar_wait_bounded(ring.full + ring.stage, ring.parity, 1000000000ull) && lane == 0) atomicOr(a.err, kErrDrain);
          if (++ring.stage == S::kStages) ring.stage = 0, ring.parity ^= 1;
        }
        return false;
      }
      {
        int ahead = stage + S::kStages - 1;
        if (ahead >= S::kStages) ahead -= S::kStages;
        if (tile + S::kStages - 1 < t1) issue(tile + S::kStages - 1, ahead);
      }
      if (++ring.stage == S::kStages) ring.stage = 0, ring.parity ^= 1;
      const uint32_t sb = ring.base + stage * S::kStageBytes;
      float ks[S::kGroups], vs[S::kGroups];
      bool dead = false;
      float vnew = vmax;
#pragma unroll
      for (int gi = 0; gi < S::kGroups; ++gi) {
        const float2 f = ring.scales[stage * S::kGroups + gi];
        ks[gi] = f.x;
        vs[gi] = f.y;
        dead |= f.y < 0.f;
        vnew = fmaxf(vnew, f.y);
      }
      // ---- scores: element e of sc[r][gi] is token slot g + 8 (e / 2), row 2 t + e % 2
      float sc[NR][S::kGroups][4], f[NR][S::kGroups][2];
#pragma unroll
      for (int gi = 0; gi < S::kGroups; ++gi) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[r][gi][e] = bias[r][e & 1];
#pragma unroll
          for (int e = 0; e < 2; ++e) f[r][gi][e] = fac[r][e] * ks[gi];
        }
        const uint32_t kb = sb + gi * S::kGroupBytes;
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          const uint4 x = lds128(kb + at(krow, 4 * j + t)), y = lds128(kb + at(krow + 8, 4 * j + t));
          const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a0 = codes_lo(xw[i]), a1 = codes_lo(yw[i]), a2 = codes_hi(xw[i]), a3 = codes_hi(yw[i]);
#pragma unroll
            for (int r = 0; r < NR; ++r) mma_f16_16816(sc[r][gi], a0, a1, a2, a3, qf[r][4 * j + i][0], qf[r][4 * j + i][1]);
          }
        }
      }
      // ---- cap and mask, where there is one; a score (base 2) is then sc f
      const int jt = it.j0 + tile * S::kTile;
      const bool masked = dead || jt + S::kTile - 1 > lo_place || (a.window > 0 && jt <= hi_place - a.window);
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int gi = 0; gi < S::kGroups; ++gi)
#pragma unroll
          for (int e = 0; e < 2; ++e) f[r][gi][e] *= 1.f / kCode;
      auto cap = [&](auto wide) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
#pragma unroll
          for (int gi = 0; gi < S::kGroups; ++gi) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              sc[r][gi][e] = capped<decltype(wide)::value>(sc[r][gi][e] * f[r][gi][e & 1], cap_in, cap_out);
            f[r][gi][0] = f[r][gi][1] = 1.f;
          }
        }
      };
      if (a.softcap > kWideCap) cap(std::true_type{});
      else if (a.softcap > 0.f) cap(std::false_type{});
      if (masked) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          // places of rows 2 t, 2 t + 1: found again where they matter, for the registers' sake
          int place[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int lr = 8 * r + 2 * t + e;
            place[e] = lr < it.rows ? sq.len - sq.n + (first_row + lr) / a.group : -1;
          }
#pragma unroll
          for (int gi = 0; gi < S::kGroups; ++gi) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = jt + gi * 16 + krow + 8 * (e >> 1), p = place[e & 1];
              const bool off = j > p || (a.window > 0 && j <= p - a.window) || vs[gi] < 0.f;
              sc[r][gi][e] = off ? -INFINITY : sc[r][gi][e] * f[r][gi][e & 1];
            }
            f[r][gi][0] = f[r][gi][1] = 1.f;
          }
        }
      }
      // ---- raise the running maxima where a score passes one by the slack
      float top[NR][2];
      bool grew = vnew > vmax;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(sc[r][0][e], sc[r][0][2 + e]) * f[r][0][e];
#pragma unroll
          for (int gi = 1; gi < S::kGroups; ++gi) x = fmaxf(x, fmaxf(sc[r][gi][e], sc[r][gi][2 + e]) * f[r][gi][e]);
          top[r][e] = x;
          grew |= x - m[r][e] > kSlack;  // (not m + kSlack, which may round up)
        }
      }
      if (__any_sync(0xffffffffu, grew)) {
        const float vr = vmax / vnew;
        bool far = false;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = fmaxf(top[r][e], m[r][e]);
#pragma unroll
            for (int sh = 4; sh < 32; sh <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, sh));
            const float k = x == -INFINITY ? 1.f : exp2_fast(m[r][e] - x);
            l[r][e] *= k;
            m[r][e] = x;
            far |= x != -INFINITY && fabsf(x) >= kCoarse;
            const float kv = k * vr;
#pragma unroll
            for (int i = 0; i < kMt; ++i) o[r][i][e] *= kv, o[r][i][2 + e] *= kv;
          }
        }
        if (__any_sync(0xffffffffu, far)) {  // the tiles to come go the way of the masked ones
          lo_place = -1;
#pragma unroll
          for (int r = 0; r < NR; ++r) {
#pragma unroll
            for (int gi = 0; gi < S::kGroups; ++gi) {
#pragma unroll
              for (int e = 0; e < 4; ++e) sc[r][gi][e] *= f[r][gi][e & 1];
              f[r][gi][0] = f[r][gi][1] = 1.f;
            }
          }
        }
        vmax = vnew;
        vinv = kPScale / vnew;
      }
      // ---- probabilities and outputs
#pragma unroll
      for (int gi = 0; gi < S::kGroups; ++gi) {
        const float ratio = fmaxf(vs[gi], 0.f) * vinv;
        uint32_t pf[NR][2];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const float m0 = m[r][0] == -INFINITY ? 0.f : m[r][0], m1 = m[r][1] == -INFINITY ? 0.f : m[r][1];
          const float p0 = exp2_fast(fmaf(sc[r][gi][0], f[r][gi][0], -m0)), p1 = exp2_fast(fmaf(sc[r][gi][1], f[r][gi][1], -m1));
          const float p2 = exp2_fast(fmaf(sc[r][gi][2], f[r][gi][0], -m0)), p3 = exp2_fast(fmaf(sc[r][gi][3], f[r][gi][1], -m1));
          l[r][0] += p0 + p2;
          l[r][1] += p1 + p3;
          pf[r][0] = transpose_8x8(f16x2(p0 * ratio, p1 * ratio));
          pf[r][1] = transpose_8x8(f16x2(p2 * ratio, p3 * ratio));
        }
        const uint32_t vb = sb + gi * S::kGroupBytes + 16 * D;
        // four bytes of four tokens: two m-tiles, values 2 i of their run on rows g, 2 i + 1 on rows g + 8
        auto columns = [&](const uint32_t va, const uint32_t vbw, const uint32_t vc, const uint32_t vd, int mt) {
          const uint32_t x0 = __byte_perm(va, vbw, 0x5140), x1 = __byte_perm(va, vbw, 0x7362);
          const uint32_t y0 = __byte_perm(vc, vd, 0x5140), y1 = __byte_perm(vc, vd, 0x7362);
          // first -128 2^-24 times the probabilities, for the sums to stay as small as the values
          // (taken off at the end, 128 times the weights' sum would cost a long cache three bits)
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            mma_f16_16816(o[r][mt], 0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u, pf[r][0], pf[r][1]);
            mma_f16_16816(o[r][mt + 1], 0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u, pf[r][0], pf[r][1]);
          }
#pragma unroll
          for (int r = 0; r < NR; ++r)
            mma_f16_16816(o[r][mt], codes_lo(x0), codes_hi(x0), codes_lo(y0), codes_hi(y0), pf[r][0], pf[r][1]);
#pragma unroll
          for (int r = 0; r < NR; ++r)
            mma_f16_16816(o[r][mt + 1], codes_lo(x1), codes_hi(x1), codes_lo(y1), codes_hi(y1), pf[r][0], pf[r][1]);
        };
        if constexpr (D == 64) {
          auto get = [&](int row) { return lds64(vb + at(row, g >> 1) + (g & 1) * 8); };
          const uint2 va = get(va_row), vbw = get(vb_row), vc = get(va_row + 8), vd = get(vb_row + 8);
          columns(va.x, vbw.x, vc.x, vd.x, 0);
          columns(va.y, vbw.y, vc.y, vd.y, 2);
        } else {
#pragma unroll
          for (int hi = 0; hi < D / 128; ++hi) {
            auto get = [&](int row) { return lds128(vb + at(row, g + 8 * hi)); };
            const uint4 va = get(va_row), vbw = get(vb_row), vc = get(va_row + 8), vd = get(vb_row + 8);
            columns(va.x, vbw.x, vc.x, vd.x, 8 * hi);
            columns(va.y, vbw.y, vc.y, vd.y, 8 * hi + 2);
            columns(va.z, vbw.z, vc.z, vd.z, 8 * hi + 4);
            columns(va.w, vbw.w, vc.w, vd.w, 8 * hi + 6);
          }
        }
      }
      __syncwarp();  // the stage is read before it is filled again
    }

    // ---- out: row 2 t + e of eight r, values kRun g + 2 i (o[.][i][e]) and + 1 (o[.][i][2 + e]), in runs of kRun
    constexpr int kRun = D == 64 ? 8 : 16;
    constexpr float kBack = 1.f / (kCode * kPScale);
#pragma unroll
    for (int r = 0; r < NR; ++r) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) l[r][e] += __shfl_xor_sync(0xffffffffu, l[r][e], sh);
        const int lr = 8 * r + 2 * t + e;
        if (lr >= it.rows) continue;
        auto value = [&](int i, int half) { return o[r][i][2 * half + e] * kBack; };
        if (part) {
          if (g == 0) *reinterpret_cast<float2*>(part + part_rows * d + 2 * lr) = make_float2(m[r][e], l[r][e]);
          float* p = part + lr * d;
#pragma unroll
          for (int i = 0; i < kMt; i += 2) {
            const int col = kRun * g + 2 * (i % 8) + 128 * (i / 8);
            if (col < d)
              *reinterpret_cast<float4*>(p + col) = make_float4(value(i, 0) * vmax, value(i, 1) * vmax, value(i + 1, 0) * vmax,
                                                                value(i + 1, 1) * vmax);
          }
          continue;
        }
        const RowOut ro = row_out(a, sq.r0, h, first_row + lr);
        const float inv = l[r][e] > 0.f ? vmax / l[r][e] : (l[r][e] == 0.f ? 0.f : l[r][e]);
        if (a.lse && g == 0)
          a.lse[ro.row * (a.c.heads * a.group) + ro.head] = l[r][e] == 0.f ? -INFINITY : (m[r][e] + log2f(l[r][e])) * kLn2;
        uint16_t* op = a.out + ro.row * a.out_stride + int64_t(ro.head) * d;
#pragma unroll
        for (int i = 0; i < kMt; i += 4) {
          const int col = kRun * g + 2 * (i % 8) + 128 * (i / 8);
          if (col < d) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(value(i + k, 0) * inv, value(i + k, 1) * inv);
              w[k] = *reinterpret_cast<const uint32_t*>(&b);
            }
            *reinterpret_cast<uint4*>(op + col) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
    }
    return true;
  }

  // Where 16-byte chunk c of a group's row lies, as the copy swizzles it: the
  // score reads (rows krow, chunks 4 j + t) and the value reads (rows 2 t,
  // chunk g) then meet no bank twice (64-byte rows: twice).
  static __device__ __forceinline__ uint32_t at(int row, int c) {
    if constexpr (D == 64) return row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
    else return (c >> 3) * S::kBoxBytes + row * 128 + (((c & 7) ^ (row & 7)) << 4);
  }
};

// Tiles of a sequence in this kernel: none for one with more rows than `limit`
// (the prompt kernel's).
template <int D, int NR>
__device__ __forceinline__ int64_t seq_tiles(const AttendArgs& a, const Seq& s, int limit) {
  using S = Shape<D, NR>;
  if (s.n * a.group > limit) return 0;
  int64_t t = 0;
  const int nrt = row_tiles<S::kRows>(a, s);
  for (int rt = 0; rt < nrt; ++rt) t += row_tile<S::kRows, S::kTile, S::kStart>(a, s, rt).units;
  return t * a.c.heads;
}

template <int D, int NR>
__global__ void __launch_bounds__(Shape<D, NR>::kThreads, 1)
kv_attend_kernel(const AttendArgs a, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                 const Scratch sc, int limit, uint64_t wait_ns) {
  using S = Shape<D, NR>;
  constexpr int kThreads = S::kThreads, kWarps = S::kWarps;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ int64_t s_pre[kThreads + 1];
  __shared__ int64_t s_warp[kWarps];
  __shared__ uint64_t s_full[kWarps][S::kStages];
  __shared__ float2 s_scales[kWarps][S::kStages * S::kGroups];
  struct Piece {  // an unfinished piece of a warp: the one its range starts with, the one it ends with
    const float* sums;
    int64_t te;          // the end of its item's tiles
    int r0, first_row, h;
    int rows;            // 0: none
    bool starts, leads;  // its item starts in this CTA; it is its item's first piece here
  };
  __shared__ Piece s_piece[2 * kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < kWarps * S::kStages) mbar_init(&s_full[0][0] + tid, S::kGroups);
  if (tid < 2 * kWarps) s_piece[tid].rows = 0;
  if (tid == 0) prefetch_tmap(&map_k), prefetch_tmap(&map_v);
  fence_mbar_init();
  pdl_wait_primary();
  pdl_launch_dependents();  // not before: kv_prompt_kernel relies on it
  // ---- tiles before each run of sequences
  const int per = (a.b.n_seqs + kThreads - 1) / kThreads;
  int64_t mine = 0;
  for (int i = tid * per; i < min((tid + 1) * per, a.b.n_seqs); ++i)
    mine += seq_tiles<D, NR>(a, load_seq(a.b, i, blockIdx.x == 0 ? a.err : nullptr), limit);
  int64_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  int64_t sums = lane < kWarps ? s_warp[lane] : 0;
#pragma unroll
  for (int o = 1; o < kWarps; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, sums, o);
    if (lane >= o) sums += up;
  }
  const int64_t total = __shfl_sync(0xffffffffu, sums, kWarps - 1);
  const int64_t before = warp == 0 ? 0 : __shfl_sync(0xffffffffu, sums, warp - 1);
  s_pre[tid + 1] = before + inc;
  if (tid == 0) s_pre[0] = 0;
  __syncthreads();
  // ---- this CTA's range (a tile a warp at least), and this warp's
  const int cta = blockIdx.x;
  const int ctas = static_cast<int>(min(int64_t(gridDim.x), max((total + kWarps - 1) / kWarps, int64_t(1))));
  if (tid == 0) sc.open[cta].rows = 0;
  if (cta >= ctas || total == 0) return;
  const Cut cut_ctas(total, ctas);
  const int64_t A = cut_ctas.first(cta), B = cut_ctas.first(cta + 1);
  const Cut cut(B - A, kWarps);
  int64_t at = A + cut.first(warp);
  const int64_t end = A + cut.first(warp + 1);
  if (at < end) {
    // the last run that starts at or before `at`
    int run = (__popc(__ballot_sync(0xffffffffu, s_pre[lane * kWarps] <= at)) - 1) * kWarps;
    run += __popc(__ballot_sync(0xffffffffu, lane < kWarps && s_pre[run + lane] <= at)) - 1;
    int s = run * per;
    int64_t off = at - s_pre[run];
    Seq sq = load_seq(a.b, s, nullptr);
    int64_t in_seq = seq_tiles<D, NR>(a, sq, limit);
    Ring<D, NR> ring;
    ring.base = ((smem_u32(smem) + 1023u) & ~1023u) + warp * S::kWarpBytes;
    ring.full = s_full[warp];
    ring.scales = s_scales[warp];
    ring.map_k = &map_k;
    ring.map_v = &map_v;
    ring.wait_ns = wait_ns;
    ring.stage = 0;
    ring.parity = 0;
    const int64_t begin = at;
    while (at < end) {
      while (off >= in_seq) {  // the next sequence that has tiles
        off -= in_seq;
        ++s;
        sq = load_seq(a.b, s, nullptr);
        in_seq = seq_tiles<D, NR>(a, sq, limit);
      }
      int rt = 0;
      int64_t rest = off;
      RowTile it = row_tile<S::kRows, S::kTile, S::kStart>(a, sq, 0);
      while (rest >= int64_t(it.units) * a.c.heads) {
        rest -= int64_t(it.units) * a.c.heads;
        it = row_tile<S::kRows, S::kTile, S::kStart>(a, sq, ++rt);
      }
      const int units = it.units;
      const int h = static_cast<int>(rest <= 0x7fffffff ? static_cast<uint32_t>(rest) / static_cast<uint32_t>(units) : rest / units);
      const int u0 = static_cast<int>(rest - int64_t(h) * units);
      const int u1 = static_cast<int>(min(int64_t(units), u0 + (end - at)));
      const int t0 = max(u0 - it.start, 0), t1 = max(u1 - it.start, 0);
      const int64_t ts = at - u0 + it.start;  // the item's first tile
      const bool whole = t0 == 0 && t1 == it.tiles;
      if (t0 < t1) {
        // a piece that ends the range stays in the ring, which is then free
        float* part = at + (u1 - u0) == end ? reinterpret_cast<float*>(smem + (ring.base - smem_u32(smem)))
                                            : sc.parts + int64_t(kWarps * cta + warp) * sc.slot_floats;
        if (!whole && lane == 0)
          s_piece[2 * warp + (at == begin ? 0 : 1)] =
              Piece{part, ts + it.tiles, sq.r0, rt * S::kRows, h, it.rows, ts >= A, t0 == 0 || ts + t0 == A};
        if (!Worker<D, NR>::run(a, sq, s, h, rt, t0, t1, whole ? nullptr : part, sc.rows, ring)) break;
      }
      at += u1 - u0;
      off += u1 - u0;
    }
  }
  // ---- pieces of one item in this CTA become one, or the item's outputs
  __syncthreads();
  const bool leads = lane < 2 * kWarps && s_piece[lane].rows > 0 && s_piece[lane].leads;
  int task = 0;
  for (unsigned left = __ballot_sync(0xffffffffu, leads); left; left &= left - 1) {
    const int i = __ffs(left) - 1, w = i >> 1;
    const Piece p = s_piece[i];
    // the others: what the next warps' ranges start with
    const int n = cut.part(min(p.te, B) - 1 - A) - w + 1;
    float* to = sc.joined + int64_t(2 * cta + (p.starts ? 1 : 0)) * sc.slot_floats;
    if (p.starts && p.te > B && tid == 0) sc.open[cta] = Open{p.r0, p.first_row, p.h, p.rows, cut_ctas.part(p.te - 1) - cta + 1};
    for (int lr = 0; lr < p.rows; ++lr) {
      if (task++ % kWarps != warp) continue;
      Joined<D> r;
      join_row<D>(sc.rows, a.c.d, lr, n, [&](int k) { return s_piece[k == 0 ? i : 2 * (w + k)].sums; }, r);
      if (p.starts && p.te <= B) {
        write_row<D>(a, row_out(a, p.r0, p.h, p.first_row + lr), r);
      } else {
        constexpr int kCols = Joined<D>::kCols, kVec = kCols < 4 ? kCols : 4;
        if (lane == 0) *reinterpret_cast<float2*>(to + sc.rows * a.c.d + 2 * lr) = make_float2(r.m, r.l);
#pragma unroll
        for (int c = 0; c < kCols; c += kVec) {
          const int col = lane * kVec + 32 * c;
          if (col >= a.c.d) continue;
          if constexpr (kVec == 4)
            *reinterpret_cast<float4*>(to + lr * a.c.d + col) = make_float4(r.o[c], r.o[c + 1], r.o[c + 2], r.o[c + 3]);
          else
            *reinterpret_cast<float2*>(to + lr * a.c.d + col) = make_float2(r.o[c], r.o[c + 1]);
        }
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32)
kv_join_kernel(const AttendArgs a, const Scratch sc) {
  __shared__ JoinShared<D> shared;
  pdl_launch_dependents();
  pdl_wait_primary();
  join_open<D>(a, sc, sc.open[blockIdx.x], blockIdx.x, blockIdx.y, shared);
}

int padded(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }
// Rows a tile, in eights: the fewest that take all of a sequence's rows, up to
// what the accumulators leave room for.
int row_eights(int D, int64_t rows) { return rows <= 8 ? 1 : rows <= 16 || D == 256 ? 2 : 4; }
// Which kernel serves which sequences: up to `limit` rows here, `eights` a tile, more in
// the kernel for prompts. A call whose sequences all have few rows splits them here;
// where some have many, this kernel keeps those with single tokens. Measured at 16
// sequences of up to 6000 tokens, here against there: D = 128: 16 rows 31 us against 58,
// 24 rows 64 against 59, 56 rows 131 against 107; D = 64: 64 rows 77 against 89;
// D = 256: 32 rows 66 against 91, 64 rows 99 against 101.
struct Share {
  int eights, limit;
};
Share share_of(int D, int64_t max_new, int group) {
  const int64_t rows = max_new * group;
  const int e = row_eights(D, group), few = D == 128 ? 16 : 64, all = few > 8 * e ? few : 8 * e;
  return rows <= all ? Share{row_eights(D, rows), all} : Share{e, 8 * e};
}

template <int D, int NR>
size_t scratch_shape(const KvCache& c, const KvBatch& b, int group, int sms, Scratch* sc = nullptr, uint8_t* base = nullptr) {
  using S = Shape<D, NR>;
  const int rows = part_rows(b.max_new, group, S::kRows), floats = part_floats(rows, c.d);
  const size_t open = 0, parts = align256(size_t(sms) * sizeof(Open));
  const size_t joined = parts + align256(size_t(sms) * S::kWarps * floats * 4);
  if (sc) *sc = Scratch{reinterpret_cast<float*>(base + parts), reinterpret_cast<float*>(base + joined),
                        reinterpret_cast<Open*>(base + open), rows, floats};
  return joined + align256(size_t(2) * sms * floats * 4);
}

template <int D, int NR>
cudaError_t launch_shape(const AttendArgs& a, int limit, cudaStream_t stream, int sms) {
  using S = Shape<D, NR>;
  CUtensorMap mk, mv;
  const uint64_t rows_page = uint64_t(a.c.heads) * a.c.page;
  cudaError_t e = encode_map_3d(&mk, a.c.k, a.c.d, rows_page, a.c.n_pages, S::kPitch, 16, S::kPitch);
  if (e != cudaSuccess) return e;
  if ((e = encode_map_3d(&mv, a.c.v, a.c.d, rows_page, a.c.n_pages, S::kPitch, 16, S::kPitch)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(kv_attend_kernel<D, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem)) != cudaSuccess)
    return e;
  Scratch sc;
  scratch_shape<D, NR>(a.c, a.b, a.group, sms, &sc, a.scratch);
  const uint64_t wait = wait_limit_ns();
  if ((e = launch_pdl(kv_attend_kernel<D, NR>, dim3(sms), dim3(S::kThreads), S::kSmem, stream, a, mk, mv, sc, limit, wait)) !=
      cudaSuccess)
    return e;
  if (int64_t(a.b.max_new) * a.group > limit)  // it joins this kernel's rows too
    return launch_kv_prompt(a, limit, sc, a.scratch + scratch_shape<D, NR>(a.c, a.b, a.group, sms), stream, sms);
  return launch_pdl(kv_join_kernel<D>, dim3(sms, sc.rows), dim3(kJoinWarps * 32), 0, stream, a, sc);
}

}  // namespace

size_t kv_attention_scratch(const KvCache& c, const KvBatch& b, int group, int sms) {
  const int D = padded(c.d);
  const Share sh = share_of(D, b.max_new, group);
  const int n = sh.eights;
  const size_t prompts = int64_t(b.max_new) * group > sh.limit ? kv_prompt_scratch(c, b, group, sms) : 0;
  if (D == 64) return prompts + (n == 1 ? scratch_shape<64, 1>(c, b, group, sms) : n == 2 ? scratch_shape<64, 2>(c, b, group, sms)
                                                                                         : scratch_shape<64, 4>(c, b, group, sms));
  if (D == 128) return prompts + (n == 1 ? scratch_shape<128, 1>(c, b, group, sms) : n == 2 ? scratch_shape<128, 2>(c, b, group, sms)
                                                                                           : scratch_shape<128, 4>(c, b, group, sms));
  return prompts + (n == 1 ? scratch_shape<256, 1>(c, b, group, sms) : scratch_shape<256, 2>(c, b, group, sms));
}

cudaError_t launch_kv_attention(const AttendArgs& a, cudaStream_t stream, int sms) {
  const int D = padded(a.c.d);
  const Share sh = share_of(D, a.b.max_new, a.group);
  const int n = sh.eights, limit = sh.limit;
  if (D == 64) return n == 1 ? launch_shape<64, 1>(a, limit, stream, sms) : n == 2 ? launch_shape<64, 2>(a, limit, stream, sms)
                                                                                  : launch_shape<64, 4>(a, limit, stream, sms);
  if (D == 128) return n == 1 ? launch_shape<128, 1>(a, limit, stream, sms) : n == 2 ? launch_shape<128, 2>(a, limit, stream, sms)
                                                                                    : launch_shape<128, 4>(a, limit, stream, sms);
  return n == 1 ? launch_shape<256, 1>(a, limit, stream, sms) : launch_shape<256, 2>(a, limit, stream, sms);
}

}  // namespace mq
