// What the two attention kernels over the 8-bit cache share: the cutting of their
// work into equal ranges, and the joining of items that several ranges shared.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "kv_internal.h"

namespace mq {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// cap tanh(s / cap), base 2, from s, 1 / cap and cap log2(e): 1 - 2 / (1 + e^2x) is within
// 2^-22 absolutely, so 2^-22 cap; where that is much (kWideCap), scores below cap / 16 take the
// series x - x^3 / 3 + 2 x^5 / 15 (2^-28 there) and keep their own precision.
constexpr float kWideCap = 64.f;
template <bool WIDE>
__device__ __forceinline__ float capped(float score, float inverse, float cap_log2e) {
  const float x = score * inverse;
  float t;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(1.f + exp2_fast(2.f * kLog2e * x)));
  t = fmaf(-2.f, t, 1.f);
  if constexpr (WIDE) {
    const float z = x * x;
    if (fabsf(x) < 0.0625f) t = x * fmaf(z, fmaf(z, 2.f / 15.f, -1.f / 3.f), 1.f);
  }
  return cap_log2e * t;
}
// Rows whose maximum lies beyond this form a weight's exponent from the rounded score, the
// maximum taken off before anything else comes on. Score times factor less maximum in one
// rounding is finer, but keys of one score then differ by up to half a step of it between
// tiles that are masked and others, and from 2^25 on a weight passes what fp16 holds. The
// logarithm of a V scale, added to a maximum first, would lose as much.
constexpr float kCoarse = 0x1p12f;  // half a step: 2^-13
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Partial sums of a piece of a shared item: per row the d outputs before the
// division, then (maximum, sum of exponentials), base 2.
struct Scratch {
  float* parts;   // a slot a warp: the piece its range starts with, where it goes on behind it
  float* joined;  // 2 slots a CTA, over its warps: the piece its range starts with, the one it ends with
  struct Open* open;  // a CTA each
  int rows;       // rows a slot holds
  int slot_floats;
};
// The item that a CTA's range ends within, if it starts in that CTA.
struct Open {
  int r0, first_row, h, rows;  // the sequence's first row, the tile's in it, its rows (0: none)
  int n;                       // CTAs that share the item
};

__host__ __device__ inline int part_rows(int max_new, int group, int rows) {
  return max_new * group < rows ? max_new * group : rows;
}
__host__ __device__ inline int part_floats(int rows, int d) { return rows * d + (2 * rows + 3) / 4 * 4; }

// [first(i), first(i + 1)): part i of `total` cut into n parts as equal as can be.
struct Cut {
  int64_t each;
  int rest;
  __device__ __forceinline__ Cut(int64_t total, int n) {
    if (total <= 0x7fffffff) {
      each = static_cast<uint32_t>(total) / static_cast<uint32_t>(n);
      rest = static_cast<uint32_t>(total) % static_cast<uint32_t>(n);
    } else {
      each = total / n;
      rest = static_cast<int>(total % n);
    }
  }
  __device__ __forceinline__ int64_t first(int i) const { return each * i + min(i, rest); }
  __device__ __forceinline__ int part(int64_t x) const {  // that holds x
    const int64_t longer = (each + 1) * rest, y = x < longer ? x : x - longer, by = x < longer ? each + 1 : each;
    const int64_t q = (y | by) <= 0x7fffffff ? static_cast<uint32_t>(y) / static_cast<uint32_t>(by) : y / by;
    return static_cast<int>(q) + (x < longer ? 0 : rest);
  }
};

// Where an item's row goes.
struct RowOut {
  int64_t row;
  int head;
};
// row: of its sequence, the first of which is r0.
__device__ __forceinline__ RowOut row_out(const AttendArgs& a, int r0, int h, int row) {
  const int qi = row / a.group;
  return RowOut{int64_t(r0) + qi, h * a.group + row - qi * a.group};
}

// Joins one row of n pieces (piece i at sums_of(i)), in their order, by one
// warp: the pieces' weights first, a lane each, then the sums.
template <int D>
struct Joined {
  static constexpr int kCols = D / 32;
  float o[kCols], m, l;
};
template <int D, typename SumsOf>
__device__ __forceinline__ void join_row(int rows, int d, int lr, int n, SumsOf sums_of, Joined<D>& r) {
  constexpr int kCols = Joined<D>::kCols, kVec = kCols < 4 ? kCols : 4;
  const int lane = threadIdx.x & 31;
  r.m = -INFINITY;
  r.l = 0.f;
#pragma unroll
  for (int i = 0; i < kCols; ++i) r.o[i] = 0.f;
  constexpr int kBatch = 32 / kCols;
  for (int first = 0; first < n; first += 32) {
    const bool have = first + lane < n;
    const float* mine = have ? sums_of(first + lane) : nullptr;
    const float2 ml = have ? *reinterpret_cast<const float2*>(mine + rows * d + 2 * lr) : make_float2(-INFINITY, 0.f);
    const int count = min(32, n - first);
    float v[kBatch][kCols];
    auto load = [&](int k0) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float* p =
            reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), (k0 + k) & 31)) + lr * d;
#pragma unroll
        for (int i = 0; i < kCols; i += kVec) {
          const int col = lane * kVec + 32 * i;
          const bool in = k0 + k < count && col < d;
          if constexpr (kVec == 4) {
            const float4 x = in ? *reinterpret_cast<const float4*>(p + col) : make_float4(0.f, 0.f, 0.f, 0.f);
            v[k][i] = x.x, v[k][i + 1] = x.y, v[k][i + 2] = x.z, v[k][i + 3] = x.w;
          } else {
            const float2 x = in ? *reinterpret_cast<const float2*>(p + col) : make_float2(0.f, 0.f);
            v[k][i] = x.x, v[k][i + 1] = x.y;
          }
        }
      }
    };
    load(0);
    float top = fmaxf(r.m, ml.x);
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, sh));
    const float to = top == -INFINITY ? 0.f : top;  // a NaN sum has no maximum and is passed on
    const float keep = exp2_fast(r.m - to), weight = have ? exp2_fast(ml.x - to) : 0.f;
    float sum = ml.y * weight;
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, sh);
    r.l = r.l * keep + sum;
    r.m = top;
#pragma unroll
    for (int i = 0; i < kCols; ++i) r.o[i] *= keep;
    for (int k0 = 0;;) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float w = __shfl_sync(0xffffffffu, weight, (k0 + k) & 31);
#pragma unroll
        for (int i = 0; i < kCols; ++i) r.o[i] = fmaf(k0 + k < count ? w : 0.f, v[k][i], r.o[i]);
      }
      if ((k0 += kBatch) >= count) break;
      load(k0);
    }
  }
}
template <int D>
__device__ __forceinline__ void write_row(const AttendArgs& a, const RowOut& ro, const Joined<D>& r) {
  constexpr int kCols = Joined<D>::kCols, kVec = kCols < 4 ? kCols : 4;
  const int lane = threadIdx.x & 31, d = a.c.d;
  const float inv = r.l > 0.f ? 1.f / r.l : (r.l == 0.f ? 0.f : r.l);
  uint16_t* op = a.out + ro.row * a.out_stride + int64_t(ro.head) * d;
#pragma unroll
  for (int i = 0; i < kCols; i += kVec) {
    const int col = lane * kVec + 32 * i;
    if (col < d) {
#pragma unroll
      for (int k = 0; k < kVec; k += 2) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(r.o[i + k] * inv, r.o[i + k + 1] * inv);
        *reinterpret_cast<__nv_bfloat162*>(op + col + k) = b;
      }
    }
  }
  if (a.lse && lane == 0) {
    const float top = r.m == -INFINITY ? 0.f : r.m;
    a.lse[ro.row * (a.c.heads * a.group) + ro.head] = r.l == 0.f ? -INFINITY : (top + log2f(r.l)) * kLn2;
  }
}


// Joins row lr of an item that several CTAs shared, from CTA c on; the CTA's warps take a run
// of its pieces each.
constexpr int kJoinWarps = 4;
template <int D>
struct JoinShared {
  float o[kJoinWarps][D], m[kJoinWarps], l[kJoinWarps];
};
template <int D>
__device__ __forceinline__ void join_open(const AttendArgs& a, const Scratch& sc, const Open& p, int c, int lr, JoinShared<D>& sh) {
  constexpr int kCols = Joined<D>::kCols;
  if (lr >= p.rows) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int run = (p.n + kJoinWarps - 1) / kJoinWarps, first = warp * run;
  Joined<D> r;
  join_row<D>(sc.rows, a.c.d, lr, min(run, p.n - first),
              [&](int k) { return sc.joined + int64_t(2 * (c + first + k) + (first + k == 0 ? 1 : 0)) * sc.slot_floats; }, r);
  if (warp > 0) {
    if (lane == 0) sh.m[warp] = r.m, sh.l[warp] = r.l;
#pragma unroll
    for (int i = 0; i < kCols; ++i) sh.o[warp][lane + 32 * i] = r.o[i];
  }
  __syncthreads();
  if (warp > 0) return;
  float top = r.m;
  for (int k = 1; k < kJoinWarps; ++k) top = fmaxf(top, sh.m[k]);
  const float to = top == -INFINITY ? 0.f : top, keep = exp2_fast(r.m - to);
  r.m = top;
  r.l *= keep;
#pragma unroll
  for (int i = 0; i < kCols; ++i) r.o[i] *= keep;
  for (int k = 1; k < kJoinWarps; ++k) {
    const float w = exp2_fast(sh.m[k] - to);
    r.l = fmaf(sh.l[k], w, r.l);
#pragma unroll
    for (int i = 0; i < kCols; ++i) r.o[i] = fmaf(sh.o[k][lane + 32 * i], w, r.o[i]);
  }
  write_row<D>(a, row_out(a, p.r0, p.h, p.first_row + lr), r);
}

inline size_t align256(size_t b) { return (b + 255) & ~size_t(255); }

}  // namespace mq
