// Rotary positions, the quantising write of the 8-bit key/value cache and its
// read-back.
//
// Rotary positions: pair i of a head, (a, b), at position p becomes
//   f (a cos t - b sin t, b cos t + a sin t),   t = p w_i,
// with w_i the pair's angle per position and f a factor. The caller's table
// holds w_i / 2 pi as a 64-bit fraction of a turn, so p w_i modulo one turn is
// one wrapping integer product, exact to 2^-64 turns times p at any position;
// only the reduced angle becomes fp32.
//
// The cache: a page and head of K (or V) holds codes c in [-127, 127] as bytes
// c + 128 and one scale s, value = s c. A call that adds tokens to a page sets
//   s' = max(s_old if the page held tokens before, max |x_new| / 127),
// rounds what the page held to the new scale, c' = rint(c s_old / s'), where
// it grew, and writes rint(x / s'). Every operation is IEEE binary32, correctly
// rounded, so equal inputs give equal bytes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "../../include/mq.h"
#include "kv_internal.h"
#include "mq_device.cuh"
#include "mq_internal.h"

namespace mq {
namespace {

// cos and sin of 2 pi phase / 2^64. The nearest quarter turn is split off in
// integers; the rest, |x| <= pi / 4, goes through the Taylor series (first dropped
// terms 2^-29 of the sine, 2^-33 of the cosine). x is off by 2.5 u of itself (its
// conversion, the constant, their product; u = 2^-24), which moves either by 1.4 u at
// most; the other roundings take one more: both are within 2.5 u absolutely (1.5 and
// 1.7 u over four million angles).
__device__ __forceinline__ void turn_sincos(uint64_t phase, float& sn, float& cs) {
  const uint32_t top = static_cast<uint32_t>(phase >> 32);
  const uint32_t quarter = (top + 0x20000000u) >> 30;
  const float x = static_cast<float>(static_cast<int32_t>(top - (quarter << 30))) * 1.4629180792671596e-9f;  // 2 pi / 2^32
  const float z = x * x;
  float s = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);  // 1/9!, 1/7!
  s = fmaf(z, s, 8.3333333e-3f);
  s = fmaf(z, s, -1.6666667e-1f);
  s = fmaf(z * x, s, x);
  float c = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);  // 1/10!, 1/8!
  c = fmaf(z, c, -1.3888889e-3f);
  c = fmaf(z, c, 4.1666667e-2f);
  c = fmaf(z, c, -0.5f);
  c = fmaf(z, c, 1.0f);
  const float a = (quarter & 1) ? c : s, b = (quarter & 1) ? s : c;
  sn = (quarter & 2) ? -a : a;
  cs = ((quarter + 1) & 2) ? -b : b;
}

template <typename T, int V>
__device__ __forceinline__ void load_v(const T* p, float (&v)[V]) {
  if constexpr (V == 4 && sizeof(T) == 4) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
  } else if constexpr (V == 4) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(u.x << 16);
    v[1] = __uint_as_float(u.x & 0xFFFF0000u);
    v[2] = __uint_as_float(u.y << 16);
    v[3] = __uint_as_float(u.y & 0xFFFF0000u);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = static_cast<float>(p[i]);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T, int V>
__device__ __forceinline__ void store_v(T* p, const float (&v)[V]) {
  if constexpr (V == 4 && sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else if constexpr (V == 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = static_cast<T>(v[i]);
  }
}

// A head's d values are cut into d / (2 V) units of two runs of V values. Units
// below rot / (2 V) hold V pairs: runs u V and u V + rot / 2 (half layout), or
// 2 u V and 2 u V + V (interleaved: the pairs lie next to one another). The
// others, behind the rotated part, are plain.
struct Unit {
  int c0, c1;
  bool turned;
};
template <int V>
__device__ __forceinline__ Unit unit_of(int u, int rot, bool interleaved) {
  const bool turned = u * 2 * V < rot;
  if (turned && !interleaved) return Unit{u * V, u * V + (rot >> 1), true};
  return Unit{u * 2 * V, u * 2 * V + V, turned};
}
// Index of the first of a turned unit's V frequencies: pair u V + i.
template <int V>
__device__ __forceinline__ void unit_angles(const Rope& r, int u, int pos, float (&sn)[V], float (&cs)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    turn_sincos(r.turns[u * V + i] * static_cast<uint64_t>(static_cast<int64_t>(pos)), sn[i], cs[i]);
    sn[i] *= r.factor;
    cs[i] *= r.factor;
  }
}
template <int V>
__device__ __forceinline__ void unit_turn(bool interleaved, float (&a)[V], float (&b)[V], const float (&sn)[V],
                                          const float (&cs)[V]) {
  if (!interleaved || V == 1) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float x = a[i], y = b[i];
      a[i] = fmaf(x, cs[i], -(y * sn[i]));
      b[i] = fmaf(y, cs[i], x * sn[i]);
    }
  } else {
    // run a holds pairs 0 .. V/2 - 1, run b the others
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float x = a[2 * i], y = a[2 * i + 1];
      a[2 * i] = fmaf(x, cs[i], -(y * sn[i]));
      a[2 * i + 1] = fmaf(y, cs[i], x * sn[i]);
      const float w = b[2 * i], z = b[2 * i + 1];
      b[2 * i] = fmaf(w, cs[V / 2 + i], -(z * sn[V / 2 + i]));
      b[2 * i + 1] = fmaf(z, cs[V / 2 + i], w * sn[V / 2 + i]);
    }
  }
}

// ------------------------------------------------------------------ rotary
constexpr int kRopeThreads = 256;

// One CTA per (row, share of its heads): thread (head lane, unit) forms its
// unit's cosines once and walks the heads with them. Each value is read once
// and written once, both runs of a unit before either is written, so y may be
// x. V = 4 needs rot and d in eights and aligned runs; V = 1 takes the rest.
template <typename TI, typename TO, int V>
__global__ void __launch_bounds__(kRopeThreads)
rope_kernel(const TI* x, int64_t rows, int heads, int d, int64_t x_stride, const int32_t* positions,
            Rope rope, TO* y, int64_t y_stride, int units, int head_lanes, int head_splits) {
  pdl_launch_dependents();
  pdl_wait_primary();
  const int u = threadIdx.x % units, hl = threadIdx.x / units;
  if (hl >= head_lanes) return;
  const Unit un = unit_of<V>(u, rope.rot, rope.interleaved != 0);
  const int part = blockIdx.x % head_splits;
  for (int64_t r = blockIdx.x / head_splits; r < rows; r += gridDim.x / head_splits) {
    float sn[V], cs[V];
    if (un.turned) unit_angles<V>(rope, u, positions[r], sn, cs);
    for (int h = part * head_lanes + hl; h < heads; h += head_splits * head_lanes) {
      const TI* xr = x + r * x_stride + int64_t(h) * d;
      TO* yr = y + r * y_stride + int64_t(h) * d;
      float a[V], b[V];
      load_v<TI, V>(xr + un.c0, a);
      load_v<TI, V>(xr + un.c1, b);
      if (un.turned) unit_turn<V>(rope.interleaved != 0, a, b, sn, cs);
      store_v<TO, V>(yr + un.c0, a);
      store_v<TO, V>(yr + un.c1, b);
    }
  }
}

template <typename TI, typename TO>
cudaError_t rope_typed(const void* x, int64_t rows, int heads, int d, int64_t x_stride, const int32_t* positions,
                       const Rope& rope, void* y, int64_t y_stride, cudaStream_t stream, int sms) {
  auto run_ok = [](const void* p, int64_t stride, int item) {
    return (reinterpret_cast<uintptr_t>(p) % (4 * item)) == 0 && stride % 4 == 0;
  };
  const bool wide = rope.rot % 8 == 0 && d % 8 == 0 && run_ok(x, x_stride, sizeof(TI)) && run_ok(y, y_stride, sizeof(TO));
  const int units = wide ? d / 8 : d / 2;
  int head_lanes = kRopeThreads / units;
  if (head_lanes < 1) return cudaErrorNotSupported;
  if (head_lanes > heads) head_lanes = heads;
  // few rows: the heads of a row are shared out so that the card fills
  int splits = static_cast<int>((4 * int64_t(sms) + rows - 1) / rows);
  const int most = (heads + head_lanes - 1) / head_lanes;
  splits = splits < 1 ? 1 : (splits > most ? most : splits);
  int64_t grid = rows * splits;
  const int64_t cap = (int64_t(1) << 30) / splits * splits;
  if (grid > cap) grid = cap;
  const int threads = (units * head_lanes + 31) / 32 * 32;
  if (wide)
    return launch_pdl(rope_kernel<TI, TO, 4>, dim3(static_cast<unsigned>(grid)), dim3(threads), 0, stream,
                      static_cast<const TI*>(x), rows, heads, d, x_stride, positions, rope, static_cast<TO*>(y), y_stride,
                      units, head_lanes, splits);
  return launch_pdl(rope_kernel<TI, TO, 1>, dim3(static_cast<unsigned>(grid)), dim3(threads), 0, stream,
                    static_cast<const TI*>(x), rows, heads, d, x_stride, positions, rope, static_cast<TO*>(y), y_stride,
                    units, head_lanes, splits);
}

// ------------------------------------------------------------------ append
// Whether a sequence holds `row`, and the row's place in it, by the warp. Up to 32
// sequences take one round of loads, more a search of 32 candidates at a time (the
// last s with row_start[s] <= row).
__device__ __forceinline__ bool find_place(const KvBatch& b, int row, int lane, int* place) {
  if (b.n_seqs <= 32) {
    const bool in = lane < b.n_seqs;
    const int first = b.row_start[0], end = in ? b.row_start[lane + 1] : 0x7fffffff, len = in ? b.kv_len[lane] : 0;
    const int s = __popc(__ballot_sync(0xffffffffu, end <= row));
    *place = __shfl_sync(0xffffffffu, len, s & 31) - __shfl_sync(0xffffffffu, end, s & 31) + row;
    return s < b.n_seqs && row >= first;
  }
  if (row < b.row_start[0] || row >= b.row_start[b.n_seqs]) return false;
  int lo = 0, n = b.n_seqs;  // the answer lies in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lo + lane * step;
    const bool ok = lane * step < n && b.row_start[i] <= row;
    const unsigned hit = __ballot_sync(0xffffffffu, ok);
    const int last = 31 - __clz(hit | 1u);
    const int end = lo + n;
    lo += last * step;
    n = min(step, end - lo);
  }
  *place = b.kv_len[lo] - b.row_start[lo + 1] + row;
  return true;
}

// rint(x / s) + 128 in the low byte, within [-127, 127] + 128, x / s correctly rounded: with r = 1 / s correctly
// rounded and q = x r, the remainder x - q s is exact and q + r (x - q s) rounds as x / s
// does (Markstein, IBM J. Res. Dev. 34, 1990). That needs the remainder to be above the
// subnormals where it matters, |x / s| > 1/4: a scale of 2^-100 does. Four operations a value
// where the division and conversions take twenty, which bound the whole write (80 us against
// 61 for 5300 rows of 32 heads of 256 values).
struct Coder {
  float s, r;
  bool tiny;
  __device__ __forceinline__ explicit Coder(float scale) {
    s = scale;
    r = scale > 0.f ? __fdiv_rn(1.f, scale) : 0.f;
    tiny = scale > 0.f && scale < 0x1p-100f;
  }
  // TINY: the scale lies below 2^-100
  template <bool TINY>
  __device__ __forceinline__ uint32_t one(float x) const {
    float q = x * r;
    // (a subnormal scale is rounded by up to half of itself, so a quotient may pass 127)
    q = TINY ? fminf(fmaxf(__fdiv_rn(x, s), -127.f), 127.f) : fmaf(fmaf(-q, s, x), r, q);
    return __float_as_uint(q + 12583040.f);  // 1.5 2^23 + 128: rounds to an integer, ties to even
  }
  template <bool TINY>
  __device__ __forceinline__ uint32_t four(float a, float b, float c, float d) const {
    return __byte_perm(__byte_perm(one<TINY>(a), one<TINY>(b), 0x0040), __byte_perm(one<TINY>(c), one<TINY>(d), 0x0040), 0x5410);
  }
};
constexpr int kUnitsPerThread = 4, kHeadsPerThread = 4;

// CTAs below kv_blocks: one page of one sequence, one head, K or V. The new
// values of the page stay in registers (at most 4 units of 8 a thread) from
// the maximum to the bytes, so they are read once. The others: the queries,
// one row and a share of its heads each, up to 4 a thread. Bound by the bytes; what
// costs is the chain of loads that a short CTA waits for (lengths, page, scale,
// values), so each load starts as soon as its address is known: values before the
// page and its scale, queries before the search for their sequence.
template <typename T>
__global__ void __launch_bounds__(1024)
kv_append_kernel(const AppendArgs a, int page_slots, int kv_blocks, int q_splits) {
  pdl_launch_dependents();
  pdl_wait_primary();
  const int tid = threadIdx.x, lane = tid & 31;
  const int d = a.c.d, units = d >> 3;
  const bool il = a.rope.interleaved != 0;
  if (static_cast<int>(blockIdx.x) >= kv_blocks) {
    const int i = blockIdx.x - kv_blocks;
    const int row = i / q_splits;
    const int head_lanes = blockDim.x / units, stride = q_splits * head_lanes;
    const int u = tid % units, hl = tid / units;
    const Unit un = unit_of<4>(u, a.rope.turns ? a.rope.rot : 0, il);
    const T* x = static_cast<const T*>(a.q) + row * a.q_stride;
    float p[kHeadsPerThread][4], q[kHeadsPerThread][4];
    const int h0 = (i % q_splits) * head_lanes + hl;
#pragma unroll
    for (int k = 0; k < kHeadsPerThread; ++k) {
      const int h = h0 + k * stride;
      if (hl < head_lanes && h < a.n_q_heads) {
        load_v<T, 4>(x + int64_t(h) * d + un.c0, p[k]);
        load_v<T, 4>(x + int64_t(h) * d + un.c1, q[k]);
      }
    }
    // the row's cosines once, for all of its heads
    __shared__ __align__(16) float s_sn[128], s_cs[128];
    int pos = 0;
    if (a.rope.turns && !a.positions) {
      if (!find_place(a.b, row, lane, &pos)) return;
    } else {
      if (a.rope.turns) pos = a.positions[row];
      if (row < a.b.row_start[0] || row >= a.b.row_start[a.b.n_seqs]) return;
    }
    if (a.rope.turns) {
      for (int i = tid; i < a.rope.rot >> 1; i += blockDim.x) {
        float sn, cs;
        turn_sincos(a.rope.turns[i] * static_cast<uint64_t>(static_cast<int64_t>(pos)), sn, cs);
        s_sn[i] = sn * a.rope.factor;
        s_cs[i] = cs * a.rope.factor;
      }
      __syncthreads();
    }
    if (hl >= head_lanes) return;
    float sn[4], cs[4];
    if (un.turned) {
      const float4 x4 = *reinterpret_cast<const float4*>(s_sn + 4 * u), y4 = *reinterpret_cast<const float4*>(s_cs + 4 * u);
      sn[0] = x4.x, sn[1] = x4.y, sn[2] = x4.z, sn[3] = x4.w;
      cs[0] = y4.x, cs[1] = y4.y, cs[2] = y4.z, cs[3] = y4.w;
    }
#pragma unroll
    for (int k = 0; k < kHeadsPerThread; ++k) {
      const int h = h0 + k * stride;
      if (h >= a.n_q_heads) break;
      if (un.turned) unit_turn<4>(il, p[k], q[k], sn, cs);
      __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(a.q_out) + (int64_t(row) * a.n_q_heads + h) * d;
      store_v<__nv_bfloat16, 4>(o + un.c0, p[k]);
      store_v<__nv_bfloat16, 4>(o + un.c1, q[k]);
    }
    return;
  }
  __shared__ float s_max[32];
  int i = blockIdx.x;
  const bool is_v = i & 1;
  i >>= 1;
  const int h = i % a.c.heads;
  i /= a.c.heads;
  const int slot_page = i % page_slots, s = i / page_slots;
  const Seq sq = load_seq(a.b, s, (is_v || h || slot_page) ? nullptr : a.err);
  const int start = max(sq.len - sq.n, 0);  // first new token
  const int index = (start >> a.c.page_log2) + slot_page;
  const int base = index << a.c.page_log2;
  if (sq.n == 0 || base >= sq.len) return;
  const int lo = max(start - base, 0), hi = min(sq.len - base, a.c.page);  // new tokens of the page
  // row of the page's token t: r0 + (base + t) - (len - n)
  const int64_t row0 = sq.r0 + int64_t(base) - (sq.len - sq.n);
  const T* x = static_cast<const T*>(is_v ? a.v : a.k) + int64_t(h) * d;
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  const bool turn = a.rope.turns && !is_v;
  float va[kUnitsPerThread][4], vb[kUnitsPerThread][4];
  // this thread's units of the page's new tokens: (token, unit) tid, tid + threads, ...
  const int first_t = tid / units, first_u = tid - first_t * units, step_t = blockDim.x / units, step_u = blockDim.x - step_t * units;
  auto each = [&](auto body) {
    int t = lo + first_t, u = first_u;
#pragma unroll
    for (int k = 0; k < kUnitsPerThread; ++k) {
      if (t < hi) body(k, t, u);
      t += step_t;
      u += step_u;
      if (u >= units) u -= units, ++t;
    }
  };
  each([&](int k, int t, int u) {
    const Unit un = unit_of<4>(u, turn ? a.rope.rot : 0, il);
    const T* xr = x + (row0 + t) * stride;
    load_v<T, 4>(xr + un.c0, va[k]);
    load_v<T, 4>(xr + un.c1, vb[k]);
  });
  const int pid = load_page(a.c, a.b, s, index, a.err);
  if (pid < 0) return;
  const int64_t tile = int64_t(pid) * a.c.heads + h;
  float* scale_p = (is_v ? a.c.v_scale : a.c.k_scale) + tile;
  uint8_t* codes = (is_v ? a.c.v : a.c.k) + tile * a.c.page * d;
  const float old = lo > 0 ? *scale_p : 0.f;
  float mx = 0.f;
  each([&](int k, int t, int u) {
    if (unit_of<4>(u, turn ? a.rope.rot : 0, il).turned) {
      float sn[4], cs[4];
      unit_angles<4>(a.rope, u, a.positions ? a.positions[row0 + t] : base + t, sn, cs);
      unit_turn<4>(il, va[k], vb[k], sn, cs);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fmaxf(fabsf(va[k][e]), fabsf(vb[k][e])));
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (blockDim.x > 32) {
    if (lane == 0) s_max[tid >> 5] = mx;
    __syncthreads();
    mx = lane < static_cast<int>(blockDim.x >> 5) ? s_max[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  const float scale = fmaxf(old, __fdiv_rn(mx, 127.f));
  const Coder code(scale);
  if (lo > 0 && scale > old) {
    // the scale grew: what the page held is rounded to it
    for (int w = tid; w < lo * d / 16; w += blockDim.x) {
      uint4* p = reinterpret_cast<uint4*>(codes) + w;
      uint4 c = *p;
      uint32_t* cw = &c.x;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v[4];
#pragma unroll
        for (int f = 0; f < 4; ++f) v[f] = __fmul_rn(static_cast<float>(static_cast<int>((cw[e] >> (8 * f)) & 255u) - 128), old);
        cw[e] = code.tiny ? code.four<true>(v[0], v[1], v[2], v[3]) : code.four<false>(v[0], v[1], v[2], v[3]);
      }
      *p = c;
    }
  }
  auto store = [&](auto tiny) {
    each([&](int k, int t, int u) {
      const Unit un = unit_of<4>(u, turn ? a.rope.rot : 0, il);
      uint8_t* o = codes + t * d;
      *reinterpret_cast<uint32_t*>(o + un.c0) = code.four<decltype(tiny)::value>(va[k][0], va[k][1], va[k][2], va[k][3]);
      *reinterpret_cast<uint32_t*>(o + un.c1) = code.four<decltype(tiny)::value>(vb[k][0], vb[k][1], vb[k][2], vb[k][3]);
    });
  };
  if (code.tiny) store(std::true_type{});
  else store(std::false_type{});
  if (tid == 0) *scale_p = scale;
}

// ------------------------------------------------------------------ read
constexpr int kReadThreads = 128;

// One CTA per (page of a sequence's range, head, K or V): bytes in, values
// out, 16 bytes of output a thread and step, four steps' loads on their way. Bound
// by the bytes; conversions through the exponent of 2^23 and a walk without divisions
// keep the instructions below them.
template <typename T>
__global__ void __launch_bounds__(kReadThreads)
kv_read_kernel(const ReadArgs a) {
  pdl_launch_dependents();
  pdl_wait_primary();
  constexpr int V = 16 / sizeof(T);
  const int s = blockIdx.z, h = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const int o0 = a.out_start[s];
  int n = a.out_start[s + 1] - o0;
  const int first = a.first[s];
  const int len = a.b.kv_len[s];
  if (o0 < 0 || n < 0 || n > a.max_out || o0 > a.n_out - n || first < 0 || len > a.b.max_len) {
    if (threadIdx.x == 0) atomicOr(a.err, kErrBounds);
    return;
  }
  n = min(n, len - first);  // rows for tokens that the sequence does not hold stay as they were
  const int index = (first >> a.c.page_log2) + blockIdx.x;
  const int base = index << a.c.page_log2;
  const int lo = max(first - base, 0), hi = min(first + n - base, a.c.page);
  if (n <= 0 || lo >= hi) return;
  const int pid = load_page(a.c, a.b, s, index, a.err);
  if (pid < 0) return;
  const int d = a.c.d;
  const int64_t tile = int64_t(pid) * a.c.heads + h;
  const float scale = (is_v ? a.c.v_scale : a.c.k_scale)[tile];
  const uint8_t* codes = (is_v ? a.c.v : a.c.k) + tile * a.c.page * d;
  T* out = static_cast<T*>(is_v ? a.v_out : a.k_out) + (int64_t(o0) + base - first) * a.out_stride + int64_t(h) * d;
  const int per_row = d / V, step_t = kReadThreads / per_row, step_c = kReadThreads - step_t * per_row;
  int t = lo + threadIdx.x / per_row, c = threadIdx.x % per_row;
  constexpr int kSteps = 4;
  while (t < hi) {
    uint32_t u[kSteps][V / 4];
    int at[kSteps], col[kSteps];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      at[k] = t;
      col[k] = c * V;
      if (t < hi) {
        if constexpr (V == 8) {
          const uint2 g = *reinterpret_cast<const uint2*>(codes + t * d + c * V);
          u[k][0] = g.x;
          u[k][1] = g.y;
        } else {
          u[k][0] = *reinterpret_cast<const uint32_t*>(codes + t * d + c * V);
        }
      }
      t += step_t;
      c += step_c;
      if (c >= per_row) c -= per_row, ++t;
    }
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      if (at[k] >= hi) break;
      float v[V];
#pragma unroll
      for (int e = 0; e < V; ++e)  // 2^23 + byte, less 2^23 + 128: exact
        v[e] = __fmul_rn(scale, __uint_as_float(__byte_perm(u[k][e / 4], 0x4B000000u, 0x7440 + e % 4)) - 8388736.f);
      T* o = out + at[k] * a.out_stride + col[k];
      if constexpr (V == 8) {
        *reinterpret_cast<uint4*>(o) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
      } else {
        *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope(const void* x, int x_dtype, int64_t rows, int heads, int d, int64_t x_stride,
                        const int32_t* positions, const Rope& rope, void* y, int y_dtype, int64_t y_stride,
                        cudaStream_t stream, int sms) {
  if (x_dtype == MQ_F32 && y_dtype == MQ_F32)
    return rope_typed<float, float>(x, rows, heads, d, x_stride, positions, rope, y, y_stride, stream, sms);
  if (x_dtype == MQ_F32)
    return rope_typed<float, __nv_bfloat16>(x, rows, heads, d, x_stride, positions, rope, y, y_stride, stream, sms);
  if (y_dtype == MQ_F32)
    return rope_typed<__nv_bfloat16, float>(x, rows, heads, d, x_stride, positions, rope, y, y_stride, stream, sms);
  return rope_typed<__nv_bfloat16, __nv_bfloat16>(x, rows, heads, d, x_stride, positions, rope, y, y_stride, stream, sms);
}

cudaError_t launch_kv_append(const AppendArgs& a, int dtype, cudaStream_t stream, int sms) {
  const int units = a.c.d / 8;
  const int tokens = a.b.max_new < a.c.page ? a.b.max_new : a.c.page;
  int threads = 32;  // every unit of a page in registers: at most 4 a thread
  while (threads < 1024 && threads * kUnitsPerThread < tokens * units) threads *= 2;
  const int page_slots = (a.b.max_new + a.c.page - 2) / a.c.page + 1;
  const int64_t kv_blocks = int64_t(a.b.n_seqs) * page_slots * a.c.heads * 2;
  int q_splits = 0;
  if (a.q) {
    // a head a thread where rows are few (latency), else up to 4 (bytes on their way, and the
    // row's sequence and cosines found once for them)
    const int head_lanes = threads / units;  // d <= 256: at most 32 units
    const int most = (a.n_q_heads + head_lanes - 1) / head_lanes, least = (most + kHeadsPerThread - 1) / kHeadsPerThread;
    q_splits = int64_t(a.b.n_rows) * least >= 4 * sms ? least : most;
  }
  const int64_t grid = kv_blocks + int64_t(a.b.n_rows) * q_splits;
  if (grid > 0x7fffffff) return cudaErrorNotSupported;
  const dim3 g(static_cast<unsigned>(grid)), t(threads);
  if (dtype == MQ_F32)
    return launch_pdl(kv_append_kernel<float>, g, t, 0, stream, a, page_slots, static_cast<int>(kv_blocks), q_splits);
  return launch_pdl(kv_append_kernel<__nv_bfloat16>, g, t, 0, stream, a, page_slots, static_cast<int>(kv_blocks), q_splits);
}

cudaError_t launch_kv_read(const ReadArgs& a, int dtype, cudaStream_t stream) {
  // rows behind a sequence's tokens are not written: max_len bounds the pages of any
  const int tokens = a.max_out < a.b.max_len ? a.max_out : a.b.max_len;
  const int slots = (tokens + a.c.page - 2) / a.c.page + 1;
  if (a.c.heads * 2 > 65535 || a.b.n_seqs > 65535) return cudaErrorNotSupported;
  const dim3 g(slots, a.c.heads * 2, a.b.n_seqs);
  if (dtype == MQ_F32) return launch_pdl(kv_read_kernel<float>, g, dim3(kReadThreads), 0, stream, a);
  return launch_pdl(kv_read_kernel<__nv_bfloat16>, g, dim3(kReadThreads), 0, stream, a);
}

}  // namespace mq
