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
// of shared memory (cp.async, 16 bytes), with no barrier between warps. An item
// that several warps share leaves partial sums that a second kernel joins, in a
// fixed order, so results do not depend on timing.
//
// Arithmetic: bytes become fp16 exactly (0x6400 | byte is 1024 + byte; minus
// 1152), m16n8k16 products with fp32 sums. A query row (bf16) is scaled by a
// power of two to below 2 first, so fp16 holds it exactly down to 2^-24 of the
// row's largest value. Probabilities are rounded to fp16 (2^-12 of each; they
// are scaled by 2^14, so those down to 2^-28 of the row's largest keep that),
// with the page's V scale relative to the largest seen folded in before. The
// sums of exponentials stay fp32 and unrounded.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/mq.h"
#include "kv_internal.h"
#include "mq_device.cuh"
#include "mq_internal.h"

namespace mq {
namespace {

constexpr int kWarps = 8;
constexpr int kStages = 3;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kPScale = 16384.f;  // 2^14

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two bytes picked by `sel` (0x4140: bytes 0, 1; 0x4342: bytes 2, 3) as the
// fp16 pair of byte - 128.
__device__ __forceinline__ uint32_t codes_f16(uint32_t w, uint32_t sel) {
  const uint32_t m = __byte_perm(w, 0x64646464u, sel);
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&m), __half2half2(__ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

template <int D, int RT>
struct Shape {
  static constexpr int kRows = 16 * RT;
  static constexpr int kTile = D == 256 ? 16 : 32;  // tokens a stage
  static constexpr int kGroups = kTile / 16;
  static constexpr int kKBytes = kTile * D;
  static constexpr int kStageBytes = 2 * kKBytes;
  static constexpr int kScaleBytes = 16;  // (K, V) scale of each 16-token group
  static constexpr int kWarpBytes = kStages * (kStageBytes + kScaleBytes);
  static constexpr int kSmem = kWarps * kWarpBytes;
};

// How an item's rows and tokens lie.
struct RowTile {
  int i0;       // first query token of the tile
  int rows;     // rows of the tile (head-major within a token)
  int j0, j1;   // tokens that some row sees, j0 rounded down to a tile
  int tiles;    // at least 1
};
template <int ROWS, int TILE>
__device__ __forceinline__ RowTile row_tile(const AttendArgs& a, const Seq& s, int rt) {
  RowTile t;
  const int first = rt * ROWS, all = s.n * a.group;
  t.rows = min(ROWS, all - first);
  t.i0 = first / a.group;
  const int i1 = (first + t.rows - 1) / a.group;
  const int base = s.len - s.n;
  t.j1 = max(base + i1 + 1, 0);
  t.j0 = a.window > 0 ? max(base + t.i0 - a.window + 1, 0) : 0;
  t.j0 &= ~(TILE - 1);
  t.tiles = max((t.j1 - t.j0 + TILE - 1) / TILE, 1);
  return t;
}
template <int ROWS>
__device__ __forceinline__ int row_tiles(const AttendArgs& a, const Seq& s) {
  return (s.n * a.group + ROWS - 1) / ROWS;
}

// Partial sums of one warp's piece of a shared item: per row the maximum
// (base 2), the sum of exponentials, and the d unnormalised outputs.
struct Scratch {
  int64_t* prefix;  // n_seqs + 1: tiles before each sequence
  float* parts;     // 2 slots a warp
  int slot_floats;  // rows * (d + 2)
};

__host__ __device__ __forceinline__ int part_rows(int max_new, int group, int rows) {
  return max_new * group < rows ? max_new * group : rows;
}

template <int D, int RT>
struct Worker {
  using S = Shape<D, RT>;
  static constexpr int kNt = D / 8;       // n-tiles of the output
  static constexpr int kJ = D / 64;       // 64-value steps of a key
  static constexpr int kPitch = D;

  // One warp's pass over tiles [t0, t1) of an item.
  static __device__ __forceinline__ void run(const AttendArgs& a, const Seq& sq, int s, int h, int rt, int t0, int t1,
                                             bool whole, float* part, uint32_t ring) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const RowTile it = row_tile<S::kRows, S::kTile>(a, sq, rt);
    const int d = a.c.d, chunks = d >> 4;
    const int first_row = rt * S::kRows;

    // ---- the queries in fragment order: value c of chunk 4 j + t, two MMAs' rows
    uint32_t qf[RT][kJ * 4][4];
    float fac[RT][2];
    int place[RT][2];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int lr = 16 * r + 8 * e + g;
        const bool ok = lr < it.rows;
        const int row = first_row + lr, qi = row / a.group, hg = row - qi * a.group;
        place[r][e] = ok ? sq.len - sq.n + qi : -1;
        const uint16_t* qp = a.q + (sq.r0 + qi) * a.q_stride + int64_t(h * a.group + hg) * d;
        uint4 raw[kJ][2];
        float mx = 0.f;
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          const int c = 4 * j + t;
          const bool in = ok && c < chunks;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            raw[j][k] = in ? __ldg(reinterpret_cast<const uint4*>(qp + 16 * c) + k) : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {raw[j][k].x, raw[j][k].y, raw[j][k].z, raw[j][k].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xFFFF0000u))));
          }
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        int ex = __float_as_int(mx) >> 23;  // 2^(ex - 127) <= mx < 2^(ex - 126)
        ex = ex < 1 || ex > 253 ? 127 : ex;
        const float down = __int_as_float((254 - ex) << 23);
        fac[r][e] = __int_as_float(ex << 23) * a.scale;
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t w[4] = {raw[j][k].x, raw[j][k].y, raw[j][k].z, raw[j][k].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)  // values 8 k + 2 i, + 1 of the chunk: MMA 4 j + 2 k + i / 2, half i % 2
              qf[r][4 * j + 2 * k + i / 2][2 * (i & 1) + e] =
                  f16x2(__uint_as_float(w[i] << 16) * down, __uint_as_float(w[i] & 0xFFFF0000u) * down);
          }
        }
      }
    }

    float o[RT][kNt][4];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int i = 0; i < kNt; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[r][i][e] = 0.f;
    float m[RT][2], l[RT][2], vmax = 0.f;
#pragma unroll
    for (int r = 0; r < RT; ++r) m[r][0] = m[r][1] = -INFINITY, l[r][0] = l[r][1] = 0.f;

    // ---- the ring
    const int page = a.c.page, log2p = a.c.page_log2;
    int pid_first = -1, pid_mine = -1;  // lane i: the page of index pid_first + i
    auto issue = [&](int tile, int stage) {
      const uint32_t kb = ring + stage * (S::kStageBytes + S::kScaleBytes), vb = kb + S::kKBytes;
      const uint32_t sb = kb + S::kStageBytes;
#pragma unroll
      for (int gi = 0; gi < S::kGroups; ++gi) {
        const int j = it.j0 + tile * S::kTile + gi * 16;
        if (j < it.j1) {  // warp-uniform
          const int index = j >> log2p;
          if (pid_first < 0 || index >= pid_first + 32) {
            pid_first = index;
            pid_mine = (index + lane) << log2p < it.j1 ? load_page(a.c, a.b, s, index + lane, a.err) : -1;
          }
          const int pid = __shfl_sync(0xffffffffu, pid_mine, index - pid_first);
          if (pid >= 0) {
            const int64_t tl = int64_t(pid) * a.c.heads + h;
            if (lane == 0) cp_async_4_at(sb + gi * 8, a.c.k_scale + tl);
            if (lane == 1) cp_async_4_at(sb + gi * 8 + 4, a.c.v_scale + tl);
            const int64_t off = (tl * page + (j & (page - 1))) * d;
            constexpr int kPerRow = D / 16;           // chunks of a padded row
            constexpr int kRowsPer = 32 / kPerRow;    // rows one instruction covers
            const int c = lane % kPerRow, r0 = lane / kPerRow;
            if (c < chunks) {
#pragma unroll
              for (int r = 0; r < 16; r += kRowsPer) {
                const int row = gi * 16 + r + r0;
                const uint32_t sm = row * kPitch + (swz(row, c) << 4);
                const int64_t go = off + int64_t(r + r0) * d + c * 16;
                cp_async_16(kb + sm, a.c.k + go);
                cp_async_16(vb + sm, a.c.v + go);
              }
            }
            continue;
          }
        }
        if (lane == 0) {  // nothing to see: a negative V scale masks the group
          asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(sb + gi * 8), "f"(0.f), "f"(-1.f) : "memory");
        }
      }
      cp_async_commit();
    };

#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      if (t0 + i < t1) issue(t0 + i, i);
      else cp_async_commit();
    }
    int stage = 0;
    for (int tile = t0; tile < t1; ++tile) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      {
        int ahead = stage + kStages - 1;
        if (ahead >= kStages) ahead -= kStages;
        if (tile + kStages - 1 < t1) issue(tile + kStages - 1, ahead);
        else cp_async_commit();
      }
      const uint32_t kb = ring + stage * (S::kStageBytes + S::kScaleBytes), vb = kb + S::kKBytes;
      const uint32_t sb = kb + S::kStageBytes;
      if (++stage == kStages) stage = 0;
      float ks[S::kGroups], vs[S::kGroups];
      bool dead = false;
#pragma unroll
      for (int gi = 0; gi < S::kGroups; ++gi) {
        const uint2 sc = lds64(sb + gi * 8);
        ks[gi] = __uint_as_float(sc.x);
        vs[gi] = __uint_as_float(sc.y);
        dead |= vs[gi] < 0.f;
      }
      // ---- scores
      float sc[RT][S::kGroups * 2][4];
#pragma unroll
      for (int nt = 0; nt < S::kGroups * 2; ++nt) {
#pragma unroll
        for (int r = 0; r < RT; ++r) sc[r][nt][0] = sc[r][nt][1] = sc[r][nt][2] = sc[r][nt][3] = 0.f;
        const int row = nt * 8 + (g ^ ((g & 1) << 2));
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          const uint4 w = lds128(kb + row * kPitch + (swz(row, 4 * j + t) << 4));
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t b0 = codes_f16(ww[i], 0x4140), b1 = codes_f16(ww[i], 0x4342);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
              const uint32_t(&q)[4] = qf[r][4 * j + i];
              mma_f16_16816(sc[r][nt], q[0], q[1], q[2], q[3], b0, b1);
            }
          }
        }
      }
      // ---- scale, cap, mask (base 2 from here)
      const int jt = it.j0 + tile * S::kTile;
      // every token of the tile is seen by every row?
      const int lo_place = sq.len - sq.n + it.i0;
      const int hi_place = sq.len - sq.n + (first_row + it.rows - 1) / a.group;
      const bool masked = dead || jt + S::kTile - 1 > lo_place || (a.window > 0 && jt <= hi_place - a.window);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
#pragma unroll
        for (int nt = 0; nt < S::kGroups * 2; ++nt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float f = fac[r][e >> 1] * ks[nt >> 1];
            float x = sc[r][nt][e];
            if (a.softcap > 0.f) {
              x = a.softcap * kLog2e * tanhf(x * f / a.softcap);
            } else {
              x *= f * kLog2e;
            }
            if (masked) {
              const int j = jt + nt * 8 + ((e & 1) ? ((2 * t + 1) ^ 4) : 2 * t);
              const int p = place[r][e >> 1];
              if (j > p || (a.window > 0 && j <= p - a.window) || vs[nt >> 1] < 0.f) x = -INFINITY;
            }
            sc[r][nt][e] = x;
          }
        }
      }
      // ---- running maxima; the outputs are rescaled only when one grew
      float vnew = vmax;
#pragma unroll
      for (int gi = 0; gi < S::kGroups; ++gi) vnew = fmaxf(vnew, vs[gi]);
      float mn[RT][2];
      bool grew = vnew > vmax;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = m[r][e];
#pragma unroll
          for (int nt = 0; nt < S::kGroups * 2; ++nt) x = fmaxf(x, fmaxf(sc[r][nt][2 * e], sc[r][nt][2 * e + 1]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
          mn[r][e] = x;
          grew |= x > m[r][e];
        }
      }
      if (__any_sync(0xffffffffu, grew)) {
        const float vr = vmax > 0.f ? vmax / vnew : 0.f;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float k = mn[r][e] == -INFINITY ? 1.f : exp2_fast(m[r][e] - mn[r][e]);
            l[r][e] *= k;
            m[r][e] = mn[r][e];
#pragma unroll
            for (int i = 0; i < kNt; ++i) o[r][i][2 * e] *= k * vr, o[r][i][2 * e + 1] *= k * vr;
          }
        }
        vmax = vnew;
      }
      // ---- probabilities and outputs
      float ratio[S::kGroups];
#pragma unroll
      for (int gi = 0; gi < S::kGroups; ++gi) ratio[gi] = vs[gi] > 0.f ? vs[gi] / vmax * kPScale : 0.f;
#pragma unroll
      for (int gi = 0; gi < S::kGroups; ++gi) {
        uint32_t pf[RT][4];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float top = m[r][e] == -INFINITY ? 0.f : m[r][e];
            float p[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) p[k] = exp2_fast(sc[r][2 * gi + (k >> 1)][2 * e + (k & 1)] - top);
            l[r][e] += (p[0] + p[1]) + (p[2] + p[3]);
            pf[r][e] = f16x2(p[0] * ratio[gi], p[1] * ratio[gi]);
            pf[r][2 + e] = f16x2(p[2] * ratio[gi], p[3] * ratio[gi]);
          }
        }
        const int ra = gi * 16 + 2 * t, rb = gi * 16 + ((2 * t + 1) ^ 4);
        auto columns = [&](const uint32_t va, const uint32_t vbw, const uint32_t vc, const uint32_t vd, int nt) {
          // four n-tiles: byte i of the words is the column of n-tile nt + i
          const uint32_t x0 = __byte_perm(va, vbw, 0x5140), x1 = __byte_perm(va, vbw, 0x7362);
          const uint32_t y0 = __byte_perm(vc, vd, 0x5140), y1 = __byte_perm(vc, vd, 0x7362);
          const uint32_t b0[4] = {codes_f16(x0, 0x4140), codes_f16(x0, 0x4342), codes_f16(x1, 0x4140), codes_f16(x1, 0x4342)};
          const uint32_t b1[4] = {codes_f16(y0, 0x4140), codes_f16(y0, 0x4342), codes_f16(y1, 0x4140), codes_f16(y1, 0x4342)};
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int r = 0; r < RT; ++r) mma_f16_16816(o[r][nt + i], pf[r][0], pf[r][1], pf[r][2], pf[r][3], b0[i], b1[i]);
        };
        if constexpr (D == 64) {
          auto at = [&](int row) { return lds64(vb + row * kPitch + (swz(row, g >> 1) << 4) + (g & 1) * 8); };
          const uint2 va = at(ra), vbw = at(rb), vc = at(ra + 8), vd = at(rb + 8);
          columns(va.x, vbw.x, vc.x, vd.x, 0);
          columns(va.y, vbw.y, vc.y, vd.y, 4);
        } else {
#pragma unroll
          for (int hi = 0; hi < D / 128; ++hi) {
            auto at = [&](int row) { return lds128(vb + row * kPitch + (swz(row, g + 8 * hi) << 4)); };
            const uint4 va = at(ra), vbw = at(rb), vc = at(ra + 8), vd = at(rb + 8);
            columns(va.x, vbw.x, vc.x, vd.x, 16 * hi);
            columns(va.y, vbw.y, vc.y, vd.y, 16 * hi + 4);
            columns(va.z, vbw.z, vc.z, vd.z, 16 * hi + 8);
            columns(va.w, vbw.w, vc.w, vd.w, 16 * hi + 12);
          }
        }
      }
      __syncwarp();  // the stage is read before it is filled again
    }
    cp_async_wait<0>();
    __syncwarp();

    // ---- out: column of o[r][nt][2 e + x] is kRun (2 t + x) + nt % kRun + 128 (nt / 16)
    constexpr int kRun = D == 64 ? 8 : 16;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[r][e] += __shfl_xor_sync(0xffffffffu, l[r][e], 1);
        l[r][e] += __shfl_xor_sync(0xffffffffu, l[r][e], 2);
        const int lr = 16 * r + 8 * e + g;
        if (lr >= it.rows) continue;
        if (!whole) {
          float* p = part + int64_t(lr) * (d + 2);
          const float back = vmax * (1.f / kPScale);
          if (t == 0) p[d] = m[r][e], p[d + 1] = l[r][e];
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int nt = 0; nt < kNt; nt += 2) {
              const int col = kRun * (2 * t + x) + nt % kRun + 128 * (nt / 16);
              if (col < d)
                *reinterpret_cast<float2*>(p + col) = make_float2(o[r][nt][2 * e + x] * back, o[r][nt + 1][2 * e + x] * back);
            }
          continue;
        }
        const int row = first_row + lr, qi = row / a.group, hq = h * a.group + row - qi * a.group;
        const int64_t grow = sq.r0 + qi;
        const float inv = l[r][e] > 0.f ? vmax * (1.f / kPScale) / l[r][e] : (l[r][e] == 0.f ? 0.f : l[r][e]);
        if (a.lse && t == 0)
          a.lse[grow * (a.c.heads * a.group) + hq] = l[r][e] == 0.f ? -INFINITY : (m[r][e] + log2f(l[r][e])) * kLn2;
        uint16_t* op = a.out + grow * a.out_stride + int64_t(hq) * d;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int nt = 0; nt < kNt; nt += 8) {
            const int col = kRun * (2 * t + x) + nt % kRun + 128 * (nt / 16);
            if (col < d) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(o[r][nt + 2 * i][2 * e + x] * inv, o[r][nt + 2 * i + 1][2 * e + x] * inv);
                w[i] = *reinterpret_cast<const uint32_t*>(&b);
              }
              *reinterpret_cast<uint4*>(op + col) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
      }
    }
  }

  // Where 16-byte chunk c of a stage's row lies: 8 rows' chunks spread so that
  // both the score reads (rows g ^ ((g & 1) << 2), chunks 4 j + t) and the value
  // reads (rows 2 t, chunk g) meet no bank twice (64-byte rows: twice).
  static __device__ __forceinline__ int swz(int row, int c) {
    if constexpr (D == 64) return c ^ ((row >> 1) & 3);
    else return c ^ (row & 7);
  }
  static __device__ __forceinline__ void cp_async_4_at(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
  }
};

// Tiles of a sequence in this kernel: none for one with more rows than `limit`
// (the prompt kernel's).
template <int D, int RT>
__device__ __forceinline__ int64_t seq_tiles(const AttendArgs& a, const Seq& s, int limit) {
  using S = Shape<D, RT>;
  if (s.n * a.group > limit) return 0;
  int64_t t = 0;
  const int nrt = row_tiles<S::kRows>(a, s);
  for (int rt = 0; rt < nrt; ++rt) t += row_tile<S::kRows, S::kTile>(a, s, rt).tiles;
  return t * a.c.heads;
}

constexpr int kThreads = kWarps * 32;

template <int D, int RT>
__global__ void __launch_bounds__(kThreads, 1)
kv_attend_kernel(const AttendArgs a, Scratch sc, int limit) {
  using S = Shape<D, RT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t s_pre[kThreads + 1];
  __shared__ int64_t s_warp[kWarps];
  pdl_launch_dependents();
  pdl_wait_primary();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // ---- tiles before each run of sequences
  const int per = (a.b.n_seqs + kThreads - 1) / kThreads;
  int64_t mine = 0;
  for (int i = tid * per; i < min((tid + 1) * per, a.b.n_seqs); ++i)
    mine += seq_tiles<D, RT>(a, load_seq(a.b, i, blockIdx.x == 0 ? a.err : nullptr), limit);
  int64_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  int64_t before = 0;
  for (int i = 0; i < warp; ++i) before += s_warp[i];
  s_pre[tid + 1] = before + inc;
  if (tid == 0) s_pre[0] = 0;
  __syncthreads();
  const int64_t total = s_pre[kThreads];
  if (blockIdx.x == 0) {  // for the joining kernel
    int64_t at = s_pre[tid];
    for (int i = tid * per; i < min((tid + 1) * per, a.b.n_seqs); ++i) {
      sc.prefix[i] = at;
      at += seq_tiles<D, RT>(a, load_seq(a.b, i, nullptr), limit);
    }
    if (tid == 0) sc.prefix[a.b.n_seqs] = total;
  }
  // ---- this warp's range
  const int64_t nw = int64_t(gridDim.x) * kWarps;
  const int64_t w = int64_t(blockIdx.x) * kWarps + warp;
  int64_t at = w * total / nw;
  const int64_t end = (w + 1) * total / nw;
  if (at >= end) return;
  int run = 0;
#pragma unroll
  for (int step = kThreads / 2; step > 0; step >>= 1)
    if (s_pre[run + step] <= at) run += step;
  int s = run * per;
  int64_t off = at - s_pre[run];
  Seq sq = load_seq(a.b, s, nullptr);
  int64_t in_seq = seq_tiles<D, RT>(a, sq, limit);
  const uint32_t ring = smem_u32(smem) + warp * S::kWarpBytes;
  const int64_t range_start = at;
  while (at < end) {
    while (off >= in_seq) {  // the next sequence that has tiles
      off -= in_seq;
      ++s;
      sq = load_seq(a.b, s, nullptr);
      in_seq = seq_tiles<D, RT>(a, sq, limit);
    }
    int rt = 0;
    int64_t rest = off;
    RowTile it = row_tile<S::kRows, S::kTile>(a, sq, 0);
    while (rest >= int64_t(it.tiles) * a.c.heads) {
      rest -= int64_t(it.tiles) * a.c.heads;
      it = row_tile<S::kRows, S::kTile>(a, sq, ++rt);
    }
    const int h = static_cast<int>(rest / it.tiles), t0 = static_cast<int>(rest % it.tiles);
    const int t1 = static_cast<int>(min(int64_t(it.tiles), t0 + (end - at)));
    const bool whole = t0 == 0 && t1 == it.tiles;
    // slot 0: the piece that the range starts with, slot 1: the one it ends with
    float* part = sc.parts + (2 * w + (at == range_start ? 0 : 1)) * sc.slot_floats;
    Worker<D, RT>::run(a, sq, s, h, rt, t0, t1, whole, part, ring);
    at += t1 - t0;
    off += t1 - t0;
  }
}

// Joins the pieces of the items that several warps shared: one CTA per (row
// of a tile, row tile and head, sequence); its warps share out the pieces.
constexpr int kJoinWarps = 4;
template <int D, int RT>
__global__ void __launch_bounds__(kJoinWarps * 32)
kv_join_kernel(const AttendArgs a, Scratch sc, int limit, int64_t nw) {
  using S = Shape<D, RT>;
  __shared__ float s_m[kJoinWarps], s_l[kJoinWarps];
  __shared__ float s_o[kJoinWarps][D];
  pdl_launch_dependents();
  pdl_wait_primary();
  const int s = blockIdx.z, lr = blockIdx.x;
  const int rt = blockIdx.y / a.c.heads, h = blockIdx.y % a.c.heads;
  const Seq sq = load_seq(a.b, s, nullptr);
  if (sq.n * a.group > limit || rt >= row_tiles<S::kRows>(a, sq)) return;
  int64_t ts = sc.prefix[s];
  const int64_t total = sc.prefix[a.b.n_seqs];
  for (int i = 0; i < rt; ++i) ts += int64_t(row_tile<S::kRows, S::kTile>(a, sq, i).tiles) * a.c.heads;
  const RowTile it = row_tile<S::kRows, S::kTile>(a, sq, rt);
  if (lr >= it.rows) return;
  ts += int64_t(h) * it.tiles;
  const int64_t te = ts + it.tiles;
  const int64_t w0 = ((ts + 1) * nw - 1) / total, w1 = (te * nw - 1) / total;  // the warps that own its first and last tile
  if (w0 == w1) return;  // written whole
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = a.c.d;
  constexpr int kCols = D / 32;
  float o[kCols], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < kCols; ++i) o[i] = 0.f;
  for (int64_t w = w0 + warp; w <= w1; w += kJoinWarps) {
    const int64_t begin = w * total / nw;
    if (begin >= (w + 1) * total / nw) continue;
    const float* p = sc.parts + (2 * w + (begin >= ts ? 0 : 1)) * sc.slot_floats + int64_t(lr) * (d + 2);
    const float pm = p[d], pl = p[d + 1];
    float v[kCols];
#pragma unroll
    for (int i = 0; i < kCols; ++i) v[i] = lane + 32 * i < d ? p[lane + 32 * i] : 0.f;
    const float mn = fmaxf(m, pm);
    const float to = mn == -INFINITY ? 0.f : mn;  // a NaN sum has no maximum and is passed on
    const float ka = exp2_fast(m - to), kb = exp2_fast(pm - to);
    l = l * ka + pl * kb;
#pragma unroll
    for (int i = 0; i < kCols; ++i) o[i] = o[i] * ka + v[i] * kb;
    m = mn;
  }
  if (lane == 0) s_m[warp] = m, s_l[warp] = l;
#pragma unroll
  for (int i = 0; i < kCols; ++i) s_o[warp][lane + 32 * i] = o[i];
  __syncthreads();
  float mn = s_m[0];
#pragma unroll
  for (int i = 1; i < kJoinWarps; ++i) mn = fmaxf(mn, s_m[i]);
  const float top = mn == -INFINITY ? 0.f : mn;
  float ls = 0.f, k[kJoinWarps];
#pragma unroll
  for (int i = 0; i < kJoinWarps; ++i) k[i] = exp2_fast(s_m[i] - top), ls += s_l[i] * k[i];
  const int row = rt * S::kRows + lr, qi = row / a.group, hq = h * a.group + row - qi * a.group;
  const int64_t grow = sq.r0 + qi;
  const float inv = ls > 0.f ? 1.f / ls : (ls == 0.f ? 0.f : ls);
  for (int c = threadIdx.x; c < d; c += kJoinWarps * 32) {
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < kJoinWarps; ++i) x += s_o[i][c] * k[i];
    a.out[grow * a.out_stride + int64_t(hq) * d + c] = __bfloat16_as_ushort(__float2bfloat16_rn(x * inv));
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[grow * (a.c.heads * a.group) + hq] = ls == 0.f ? -INFINITY : (top + log2f(ls)) * kLn2;
}

// Sequences with more than `limit` rows (prompts): a warp per item, unsplit.
template <int D, int RT>
__global__ void __launch_bounds__(kThreads, 1)
kv_attend_rows_kernel(const AttendArgs a, int limit, int row_tiles_max) {
  using S = Shape<D, RT>;
  extern __shared__ __align__(128) uint8_t smem[];
  pdl_launch_dependents();
  pdl_wait_primary();
  const int warp = threadIdx.x >> 5;
  const int s = blockIdx.z, h = blockIdx.y;
  const Seq sq = load_seq(a.b, s, nullptr);
  const int rt = row_tiles_max - 1 - (blockIdx.x * kWarps + warp);  // long rows first
  if (sq.n * a.group <= limit || rt < 0 || rt >= row_tiles<S::kRows>(a, sq)) return;
  const RowTile it = row_tile<S::kRows, S::kTile>(a, sq, rt);
  Worker<D, RT>::run(a, sq, s, h, rt, 0, it.tiles, true, nullptr, smem_u32(smem) + warp * S::kWarpBytes);
}

size_t align256(size_t b) { return (b + 255) & ~size_t(255); }

int padded(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }
// Rows a tile: 16, or 32 where more are asked for and the accumulators fit.
int tile_rows(int D, int max_new, int group) { return D < 256 && int64_t(max_new) * group > 16 ? 32 : 16; }

template <int D, int RT>
cudaError_t launch_shape(const AttendArgs& a, cudaStream_t stream, int sms) {
  using S = Shape<D, RT>;
  cudaError_t e = cudaFuncSetAttribute(kv_attend_kernel<D, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  Scratch sc;
  sc.prefix = reinterpret_cast<int64_t*>(a.scratch);
  sc.parts = reinterpret_cast<float*>(a.scratch + align256(size_t(a.b.n_seqs + 1) * 8));
  sc.slot_floats = part_rows(a.b.max_new, a.group, S::kRows) * (a.c.d + 2);
  const int limit = 4 * S::kRows;
  const int64_t rows = int64_t(a.b.max_new) * a.group;
  if ((e = launch_pdl(kv_attend_kernel<D, RT>, dim3(sms), dim3(kThreads), S::kSmem, stream, a, sc, limit)) != cudaSuccess)
    return e;
  const int64_t few = rows < limit ? rows : limit;
  const int nrt = static_cast<int>((few + S::kRows - 1) / S::kRows);
  const dim3 g(static_cast<unsigned>(few < S::kRows ? few : S::kRows), nrt * a.c.heads, a.b.n_seqs);
  e = launch_pdl(kv_join_kernel<D, RT>, g, dim3(kJoinWarps * 32), 0, stream, a, sc, limit, int64_t(sms) * kWarps);
  if (e != cudaSuccess || rows <= limit) return e;
  e = cudaFuncSetAttribute(kv_attend_rows_kernel<D, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  const int all = static_cast<int>((rows + S::kRows - 1) / S::kRows);
  return launch_pdl(kv_attend_rows_kernel<D, RT>, dim3((all + kWarps - 1) / kWarps, a.c.heads, a.b.n_seqs), dim3(kThreads),
                    S::kSmem, stream, a, limit, all);
}

}  // namespace

size_t kv_attention_scratch(const KvCache& c, const KvBatch& b, int group, int sms) {
  const int rows = part_rows(b.max_new, group, tile_rows(padded(c.d), b.max_new, group));
  return align256(size_t(b.n_seqs + 1) * 8) + align256(size_t(2) * sms * kWarps * rows * (c.d + 2) * 4);
}

cudaError_t launch_kv_attention(const AttendArgs& a, cudaStream_t stream, int sms) {
  const int D = padded(a.c.d);
  const bool two = tile_rows(D, a.b.max_new, a.group) == 32;
  if (D == 64) return two ? launch_shape<64, 2>(a, stream, sms) : launch_shape<64, 1>(a, stream, sms);
  if (D == 128) return two ? launch_shape<128, 2>(a, stream, sms) : launch_shape<128, 1>(a, stream, sms);
  return launch_shape<256, 1>(a, stream, sms);
}

}  // namespace mq
