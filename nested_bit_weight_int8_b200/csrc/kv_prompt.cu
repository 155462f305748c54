// Attention over the paged 8-bit cache for sequences with many query rows
// (prompts), on the fifth-generation tensor cores. Mathematics and masks are
// those of kv_attention.cu; here the products bound the time, not the bytes.
//
// A CTA takes kMt tiles of 128 rows (query tokens times the heads of a group) of
// one sequence and key/value head, and walks the tokens that they see in tiles of
// kT. Per tile and 128 rows: S = Q K^T (128 x kT, in tensor memory), softmax, P
// written over S as fp16, O += P V (128 x D, in tensor memory).
//   warps 0 .. 4 kMt - 1 : softmax, a thread a row: S from tensor memory, running
//                          maximum and sum in registers, P back; queries at the
//                          start and outputs at the end
//   kConv warps          : bytes to fp16 codes, K and V, into swizzled rows of
//                          shared memory (two buffers each)
//   one warp             : issues the products (one thread)
// The codes enter exactly (byte - 128), the page scales where a row's thread needs
// them: K's multiplies the score, V's goes into the exponent, so that it costs
// no instruction per score: p' = 2^(s + log2(v_scale / v_max) + 8 - m), and the sum
// of a page's p' is scaled back once. m is raised only when a score passes it by 6,
// v_max is a power of two: O is rescaled a few times in a row's life, not a tile.
// V lies as the cache has it, token by token: the second product reads it with its
// long side along the rows, so neither operand is transposed.
//
// Every mbarrier wait is bounded; one that gives up sets the device error word
// and the CTA drains its products, frees its tensor memory and exits.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/mq.h"
#include "kv_internal.h"
#include "mq_device.cuh"
#include "mq_internal.h"
#include "tc05.cuh"

namespace mq {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kPLog2 = 8.f;          // p' stands 2^8 high
constexpr float kTinyScale = 0x1p-100f;  // V scales below this count as this

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float tanh_fast(float x) {
  float r;  // 1 - 2 / (1 + e^2x): within 2^-22 absolutely, which is what a score needs
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + exp2_fast(2.f * kLog2e * x)));
  return fmaf(-2.f, r, 1.f);
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Two bytes of a word as the fp16 pair of byte - 128: 0x6400 | byte is 1024 + byte.
__device__ __forceinline__ uint32_t codes_f16(uint32_t w, uint32_t sel) {
  const uint32_t m = __byte_perm(w, 0x64646464u, sel);
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&m), __half2half2(__ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Pairs of fp32 in one 64-bit register.
__device__ __forceinline__ uint64_t pair(uint32_t x, uint32_t y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint64_t pair(float x, float y) { return pair(__float_as_uint(x), __float_as_uint(y)); }
__device__ __forceinline__ float2 unpair(uint64_t v) {
  uint32_t x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(x), "=r"(y) : "l"(v));
  return make_float2(__uint_as_float(x), __uint_as_float(y));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Moves registers between the CTA's warpgroups: all four warps of one execute it.
template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// True in one lane of the (converged) warp, always the same.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// D: the head's size rounded up to 64, 128 or 256.
template <int D>
struct Plan {
  // At D = 256 the outputs take half of the tensor memory: one tile of rows, S
  // twice in turn. Else two tiles of rows, so that one's softmax runs beside the
  // other's products.
  static constexpr int kMt = D == 256 ? 1 : 2;
  static constexpr int kT = D == 256 ? 64 : 128;
  static constexpr int kSoft = 4 * kMt;
  static constexpr int kConv = D == 256 ? 8 : 4;
  static constexpr int kThreads = 512;  // the last four warps: one issues the products
  // Registers of a softmax, a spreading and a product thread; the launch gives 128.
  static constexpr int kSoftRegs = D == 256 ? 208 : 168, kConvRegs = 112, kMmaRegs = 64;
  static_assert(kSoft * kSoftRegs + kConv * kConvRegs + 4 * kMmaRegs <= kThreads / 32 * 128, "the split fits the launch's registers");
  static constexpr int kRows = 128 * kMt;
  static constexpr int kGroups = kT / 16;
  static constexpr int kBlocks = D / 64;         // 64 values of each row side by side
  static constexpr int kQBlock = 128 * 128;      // bytes: 128 rows of 64 values
  static constexpr int kKvBlock = kT * 128;
  static constexpr int kQBytes = kMt * kBlocks * kQBlock;
  static constexpr int kKvBytes = kBlocks * kKvBlock;
  static constexpr int kSmem = 1024 + kQBytes + 4 * kKvBytes;
  static constexpr uint32_t kOCol = kMt * kT > 2 * kT ? kMt * kT : 2 * kT;  // behind the two S
  static_assert(kOCol + kMt * D <= 512, "S and O fit the tensor memory");
  static constexpr int kSlots = 4;  // scales: a tile's are read until its softmax ends
};

struct TileScales {
  float4 group[8];  // K scale, log2 of V's factor, 1 / that factor, 1 where the page may be read
  float vmax;
  int dead;         // some group may not be read
};

struct Bars {
  uint64_t q_full;
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], p_full[2], o_done[2];
  uint64_t drain;
};

template <int D>
__global__ void __launch_bounds__(Plan<D>::kThreads, 1)
kv_prompt_kernel(const AttendArgs a, int limit, int tiles_max, uint64_t wait_ns) {
  using P = Plan<D>;
  constexpr int kT = P::kT;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars bar;
  __shared__ TileScales s_scales[P::kSlots];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort_word;
  volatile int* s_abort = &s_abort_word;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sq_base = base, sk_base = base + P::kQBytes, sv_base = sk_base + 2 * P::kKvBytes;

  pdl_launch_dependents();
  pdl_wait_primary();
  // the longest rows first: tile index slowest, from the last
  const int per_tile = a.c.heads * a.b.n_seqs;
  const int rt = tiles_max - 1 - blockIdx.x / per_tile;
  const int h = (blockIdx.x % per_tile) % a.c.heads, s = (blockIdx.x % per_tile) / a.c.heads;
  const Seq sq = load_seq(a.b, s, nullptr);
  const int all_rows = sq.n * a.group, row0 = rt * P::kRows;
  if (all_rows <= limit || row0 >= all_rows) return;
  const int rows = min(P::kRows, all_rows - row0);
  const int past = sq.len - sq.n;  // place of the sequence's first row
  const int lo_place = past + row0 / a.group, hi_place = past + (row0 + rows - 1) / a.group;
  const int j1 = max(hi_place + 1, 0);
  const int lo = a.window > 0 ? max(lo_place - a.window + 1, 0) : 0;
  const int j0 = lo & ~(kT - 1);
  const int n = (j1 - j0 + kT - 1) / kT;  // tiles; 0 where no row sees a token
  const int d = a.c.d, chunks = d >> 4;

  if (tid == 0) {
    mbar_init(&bar.q_full, P::kSoft);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.k_full[i], P::kConv);
      mbar_init(&bar.v_full[i], P::kConv);
      mbar_init(&bar.k_empty[i], 1);
      mbar_init(&bar.v_empty[i], 1);
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.p_full[i], 4);
      mbar_init(&bar.o_done[i], 1);
    }
    mbar_init(&bar.drain, 1);
    s_abort_word = 0;
    fence_mbar_init();
  }
  if (warp == P::kSoft + P::kConv) {
    tc05::alloc(smem_u32(&s_tmem), 512);
    tc05::relinquish();
    tc05::fence_before_sync();
  }
  __syncthreads();
  tc05::fence_after_sync();
  const uint32_t tmem = s_tmem;
  // Warp-uniform: every lane has waited, or all give up.
  auto wait = [&](uint64_t* b, uint32_t parity, uint32_t flag) {
    const bool ok = *s_abort == 0 && mbar_wait_bounded(b, parity, wait_ns);
    if (__all_sync(0xffffffffu, ok)) return true;
    if (lane == 0) {
      atomicOr(a.err, flag);
      *s_abort = 1;
    }
    return false;
  };

  if (warp < P::kSoft) {
    // ------------------------------------------------------------ softmax
    more_registers<P::kSoftRegs>();
    const int mt = warp >> 2, r = 32 * (warp & 3) + lane, lr = 128 * mt + r;
    const bool live = lr < rows;
    const int row = row0 + lr, qi = row / a.group, hq = h * a.group + row - qi * a.group;
    const int64_t grow = int64_t(sq.r0) + qi;
    const int place = live ? past + qi : -1;
    float fac;
    {  // this thread's query, scaled by a power of two to below 2
      const uint4* qp = reinterpret_cast<const uint4*>(a.q + grow * a.q_stride + int64_t(hq) * d);
      constexpr int kAll = D / 8, kBatch = kAll < 16 ? kAll : 16;  // loads on their way at once
      uint4 u[kBatch];
      auto load = [&](int c0) {
#pragma unroll
        for (int c = 0; c < kBatch; ++c) u[c] = live && c0 + c < 2 * chunks ? __ldg(qp + c0 + c) : make_uint4(0, 0, 0, 0);
      };
      float mx = 0.f;
#pragma unroll
      for (int c0 = kAll - kBatch; c0 >= 0; c0 -= kBatch) {
        load(c0);
#pragma unroll
        for (int c = 0; c < kBatch; ++c) {
          const uint32_t w[4] = {u[c].x, u[c].y, u[c].z, u[c].w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xFFFF0000u))));
        }
      }
      int ex = __float_as_int(mx) >> 23;
      ex = ex < 1 || ex > 253 ? 127 : ex;
      const float down = __int_as_float((254 - ex) << 23) * (a.scale < 0.f ? -1.f : 1.f);
      fac = __int_as_float(ex << 23) * fabsf(a.scale) * (a.softcap > 0.f ? 1.f : kLog2e);
#pragma unroll
      for (int c0 = 0; c0 < kAll; c0 += kBatch) {
        if (c0 > 0) load(c0);
#pragma unroll
        for (int c = 0; c < kBatch; ++c) {
          const uint32_t w[4] = {u[c].x, u[c].y, u[c].z, u[c].w};
          uint32_t x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = f16x2(__uint_as_float(w[i] << 16) * down, __uint_as_float(w[i] & 0xFFFF0000u) * down);
          const int at = c0 + c;
          sts128(sq_base + (mt * P::kBlocks + (at >> 3)) * P::kQBlock + r * 128 + (((at & 7) ^ (r & 7)) << 4), x[0], x[1], x[2], x[3]);
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.q_full);
    }
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t t_o = tmem + lanes + P::kOCol + mt * D;
    const float cap_in = a.softcap > 0.f ? 1.f / a.softcap : 0.f, cap_out = a.softcap * kLog2e;
    // of the 32 rows of this warp
    const int w_lo = past + (row0 + 128 * mt + 32 * (warp & 3)) / a.group;
    const int w_hi = past + min(row0 + 128 * mt + 32 * (warp & 3) + 31, all_rows - 1) / a.group;
    float m = -INFINITY, l = 0.f, vmax = kTinyScale;
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      const int slot = P::kMt == 2 ? mt : (i & 1);
      if (!(ok = wait(&bar.s_full[slot], P::kMt == 2 ? (i & 1) : ((i >> 1) & 1), kErrWaitFull))) break;
      tc05::fence_after_sync();
      const uint32_t t_s = tmem + lanes + slot * kT;
      const TileScales& ts = s_scales[i % P::kSlots];
      const int jt = j0 + i * kT;
      const bool special =
          a.softcap > 0.f || ts.dead || jt + kT - 1 > w_lo || (a.window > 0 && jt <= w_hi - a.window) || row0 + 128 * mt + 128 > all_rows;
      // Scores of one 16-token group, capped and masked where needed; f: their factor.
      auto masked_scores = [&](float (&x)[16], int g, float& f) {
        const float4 sg = ts.group[g];
        f = fac * sg.x;
        if (!special) return;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float y = x[e] * f;
          if (a.softcap > 0.f) y = cap_out * tanh_fast(y * cap_in);
          const int j = jt + 16 * g + e;
          x[e] = j > place || (a.window > 0 && j <= place - a.window) || sg.w == 0.f ? -INFINITY : y;
        }
        f = 1.f;
      };
      auto largest = [&]() {  // score of the tile
        float top = -INFINITY;
#pragma unroll 1
        for (int g = 0; g < P::kGroups; ++g) {
          uint32_t v[16];
          tc05::ld_32x32b_x16(t_s + 16 * g, v);
          tc05::wait_ld();
          float x[16], f;
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(v[e]);
          masked_scores(x, g, f);
#pragma unroll
          for (int e = 0; e < 16; ++e) top = fmaxf(top, x[e] * f);
        }
        return top;
      };
      // Raises the maximum (an integer, so that the factors are powers of two) to
      // `top` and the V scale to the tile's; O follows.
      auto raise = [&](float top) -> bool {
        const float x = fmaxf(ceilf(top), m), k = x == -INFINITY ? 1.f : exp2_fast(m - x), kv = k * (vmax / ts.vmax);
        l *= k;
        m = x;
        vmax = ts.vmax;
        if (i == 0) return true;
        if (!wait(&bar.o_done[mt], (i - 1) & 1, kErrMma)) return false;
        tc05::fence_after_sync();
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t v[16];
          tc05::ld_32x32b_x16(t_o + 16 * c, v);
          tc05::wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * kv);
          tc05::st_32x32b_x16(t_o + 16 * c, v);
        }
        tc05::wait_st();
        return true;
      };
      // rows that have seen nothing yet take this tile's maximum first
      const bool fresh = __any_sync(0xffffffffu, live && m == -INFINITY);
      if (fresh || ts.vmax != vmax) {
        if (!(ok = raise(fresh ? largest() : -INFINITY))) break;
      }
      // p' of the whole tile, in registers: no branch between its scores, so that their
      // loads, exponentials and sums overlap. The running maximum is not looked for: a
      // score that passes it by more than 6 or so shows in its group's sum, and the
      // tile is done over.
      uint32_t pk[kT / 2];
      float sum, big;
      auto group = [&](auto score, float f, int g, float m0) {
        const float4 sg = ts.group[g];
        const uint64_t f2 = pair(f, f), c2 = pair(sg.y - m0, sg.y - m0);
        uint64_t s0 = 0, s1 = 0;
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const float2 x = unpair(fma2(score(e), f2, c2)), y = unpair(fma2(score(e + 2), f2, c2));
          const float p0 = exp2_fast(x.x), p1 = exp2_fast(x.y), p2 = exp2_fast(y.x), p3 = exp2_fast(y.y);
          s0 = add2(s0, pair(p0, p1));
          s1 = add2(s1, pair(p2, p3));
          pk[8 * g + e / 2] = f16x2(p0, p1);
          pk[8 * g + e / 2 + 1] = f16x2(p2, p3);
        }
        const float2 t = unpair(add2(s0, s1));
        big = fmaxf(big, t.x + t.y);
        sum = fmaf(t.x + t.y, sg.z, sum);
      };
      while (true) {
        const float m0 = m == -INFINITY ? 0.f : m;
        sum = big = 0.f;
        if (!special) {
          uint32_t v[2][32];
          tc05::ld_32x32b_x32(t_s, v[0]);
#pragma unroll
          for (int c = 0; c < kT / 32; ++c) {
            tc05::wait_ld();
            if (c + 1 < kT / 32) tc05::ld_32x32b_x32(t_s + 32 * (c + 1), v[(c + 1) & 1]);
#pragma unroll
            for (int half = 0; half < 2; ++half)
              group([&](int e) { return pair(v[c & 1][16 * half + e], v[c & 1][16 * half + e + 1]); },
                    fac * ts.group[2 * c + half].x, 2 * c + half, m0);
          }
        } else {
#pragma unroll
          for (int g = 0; g < P::kGroups; ++g) {
            uint32_t v[16];
            tc05::ld_32x32b_x16(t_s + 16 * g, v);
            tc05::wait_ld();
            float x[16], f;
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(v[e]);
            masked_scores(x, g, f);
            group([&](int e) { return pair(x[e], x[e + 1]); }, f, g, m0);
          }
        }
        if (!__any_sync(0xffffffffu, big > 32768.f)) break;
        if (!(ok = raise(largest()))) break;
      }
      if (!ok) break;
      l += sum;
#pragma unroll
      for (int c = 0; c < kT / 64; ++c) {
        uint32_t v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = pk[32 * c + e];
        tc05::st_32x32b_x32(t_s + 32 * c, v);
      }
      tc05::wait_st();
      tc05::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.p_full[slot]);
    }
    // ---- outputs
    if (ok && n > 0) ok = wait(&bar.o_done[mt], (n - 1) & 1, kErrMma);
    if (ok) {
      tc05::fence_after_sync();
      const float inv = l > 0.f ? vmax * 0x1p-8f / l : (l == 0.f ? 0.f : l);
      uint16_t* op = a.out + grow * a.out_stride + int64_t(hq) * d;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[32] = {};
        if (n > 0) {
          tc05::ld_32x32b_x32(t_o + 32 * c, v);
          tc05::wait_ld();
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(v[8 * k + 2 * e]) * inv, __uint_as_float(v[8 * k + 2 * e + 1]) * inv);
            w[e] = *reinterpret_cast<const uint32_t*>(&b);
          }
          if (live && 2 * c + k / 2 < chunks) *reinterpret_cast<uint4*>(op + 32 * c + 8 * k) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      if (a.lse && live) a.lse[grow * (a.c.heads * a.group) + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      tc05::fence_before_sync();
    }
  } else if (warp < P::kSoft + P::kConv) {
    // ------------------------------------------------------------ bytes to fp16
    fewer_registers<P::kConvRegs>();
    const int cw = warp - P::kSoft;
    constexpr int kTokens = kT / P::kConv;       // of this warp
    constexpr int kWide = D / 64;                // a row's chunks in fours
    constexpr int kAt = 8 / kWide;               // tokens an instruction
    constexpr int kIt = kTokens / kAt;
    // eight neighbouring lanes write two rows' chunks: no bank twice
    const int c = (lane & 3) | (((lane >> 3) & (kWide - 1)) << 2);
    const int tk = ((lane >> 2) & 1) | ((lane >> (kWide == 1 ? 3 : kWide == 2 ? 4 : 5)) << 1);
    const int page = a.c.page, log2p = a.c.page_log2;
    // lane g < kGroups: the page of group g of a tile
    auto page_of = [&](int i) {
      const int j = j0 + i * kT + 16 * lane;
      return lane < P::kGroups && j < j1 && j + 16 > lo ? a.b.pages[int64_t(s) * a.b.max_pages + (j >> log2p)] : -1;
    };
    // checked where it is used, so that the load runs ahead
    auto checked = [&](int pid, int i) {
      const int j = j0 + i * kT + 16 * lane;
      if (pid >= 0 && pid < a.c.n_pages) return pid;
      if (lane < P::kGroups && j < j1 && j + 16 > lo) atomicOr(a.err, kErrBounds);
      return -1;
    };
    uint4 xk[kIt], xv[kIt];
    float2 sc = make_float2(0.f, 0.f);  // lane's group: K, V scale
    auto fetch = [&](int i, int pid) {
      const int64_t tl = int64_t(pid) * a.c.heads + h;
      sc = make_float2(0.f, 0.f);
      if (pid >= 0) sc = make_float2(__ldg(a.c.k_scale + tl), __ldg(a.c.v_scale + tl));
#pragma unroll
      for (int k = 0; k < kIt; ++k) {
        const int tok = cw * kTokens + k * kAt + tk, j = j0 + i * kT + tok;
        const int p = __shfl_sync(0xffffffffu, pid, (cw * kTokens + k * kAt) >> 4);
        xk[k] = xv[k] = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
        if (p >= 0 && c < chunks) {
          const int64_t off = ((int64_t(p) * a.c.heads + h) * page + (j & (page - 1))) * d + 16 * c;
          xk[k] = *reinterpret_cast<const uint4*>(a.c.k + off);
          xv[k] = *reinterpret_cast<const uint4*>(a.c.v + off);
        }
      }
    };
    auto spread = [&](uint32_t to, const uint4 (&x)[kIt]) {
#pragma unroll
      for (int k = 0; k < kIt; ++k) {
        const int tok = cw * kTokens + k * kAt + tk;
        const uint32_t at = to + (c >> 2) * P::kKvBlock + tok * 128, sw = tok & 7;
        sts128(at + (((2 * (c & 3)) ^ sw) << 4), codes_f16(x[k].x, 0x4140), codes_f16(x[k].x, 0x4342), codes_f16(x[k].y, 0x4140),
               codes_f16(x[k].y, 0x4342));
        sts128(at + (((2 * (c & 3) + 1) ^ sw) << 4), codes_f16(x[k].z, 0x4140), codes_f16(x[k].z, 0x4342),
               codes_f16(x[k].w, 0x4140), codes_f16(x[k].w, 0x4342));
      }
      fence_async_smem();
      __syncwarp();
    };
    float vmax = kTinyScale;
    int pid = n > 0 ? checked(page_of(0), 0) : -1;
    if (n > 0) fetch(0, pid);
    int next = n > 1 ? page_of(1) : -1;
    for (int i = 0; i < n; ++i) {
      const int b = i & 1;
      const uint32_t parity = ((i >> 1) & 1) ^ 1;
      if (i >= 2 && !wait(&bar.k_empty[b], parity, kErrWaitEmpty)) break;
      if (cw == 0) {  // the tile's scales
        float top = lane < P::kGroups ? sc.y : 0.f;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (top > vmax) {  // the power of two at or above it
          const int e = (__float_as_int(top) + 0x7FFFFF) >> 23;
          vmax = __int_as_float(min(e, 254) << 23);
        }
        const float lg = log2f(fmaxf(sc.y / vmax, 0x1p-60f)) + kPLog2;
        TileScales& ts = s_scales[i % P::kSlots];
        const int j = j0 + i * kT + 16 * lane;
        if (lane < P::kGroups) ts.group[lane] = make_float4(sc.x, lg, exp2f(-lg), pid >= 0 ? 1.f : 0.f);
        const bool dead = __any_sync(0xffffffffu, lane < P::kGroups && j < j1 && pid < 0);
        if (lane == 0) {
          ts.vmax = vmax;
          ts.dead = dead;
        }
      }
      spread(sk_base + b * P::kKvBytes, xk);
      if (lane == 0) mbar_arrive(&bar.k_full[b]);
      if (i >= 2 && !wait(&bar.v_empty[b], parity, kErrWaitEmpty)) break;
      spread(sv_base + b * P::kKvBytes, xv);
      if (lane == 0) mbar_arrive(&bar.v_full[b]);
      if (i + 1 < n) {
        pid = checked(next, i + 1);
        fetch(i + 1, pid);
        if (i + 2 < n) next = page_of(i + 2);
      }
    }
  } else {
    // ------------------------------------------------------------ products
    fewer_registers<P::kMmaRegs>();
    // The whole warp walks the loop, so that descriptors stay in uniform registers
    // (a lone thread's moves to them cost more than the products); one lane issues.
    if (warp == P::kSoft + P::kConv && n > 0) {
    const bool leader = elect_one();
    auto wait1 = [&](uint64_t* b, uint32_t parity) { return wait(b, parity, kErrMma); };
    auto commit = [&](uint64_t* b) {
      if (leader) tc05::commit(smem_u32(b));
    };
    constexpr uint32_t id_s = tc05::idesc_f16_f32(128, kT, false), id_o = tc05::idesc_f16_f32(128, D, true);
    // One thread issues every product: their descriptors are sums of a base and constants (16-byte units).
    const uint64_t desc_q = tc05::desc_kmajor_sw128(sq_base), desc_k = tc05::desc_kmajor_sw128(sk_base);
    const uint64_t desc_v = tc05::desc_mnmajor_sw128(sv_base, P::kBlocks > 1 ? P::kKvBlock : 1024);
    auto scores = [&](int mt, int slot, int i) {  // S = Q K^T of tile i
      const uint64_t q = desc_q + mt * (P::kBlocks * P::kQBlock >> 4), k0 = desc_k + (i & 1) * (P::kKvBytes >> 4);
      const uint32_t to = tmem + slot * kT;
      if (leader) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc05::mma_ss(to, q + (((k >> 2) * P::kQBlock + (k & 3) * 32) >> 4), k0 + (((k >> 2) * P::kKvBlock + (k & 3) * 32) >> 4),
                       id_s, k > 0);
        tc05::commit(smem_u32(&bar.s_full[slot]));
      }
    };
    auto outputs = [&](int mt, int slot, int i) {  // O += P V of tile i
      const uint64_t v0 = desc_v + (i & 1) * (P::kKvBytes >> 4);
      const uint32_t to = tmem + P::kOCol + mt * D, p = tmem + slot * kT;
      if (leader) {
#pragma unroll
        for (int k = 0; k < kT / 16; ++k) tc05::mma_ts(to, p + 8 * k, v0 + (k * 2048 >> 4), id_o, i > 0 || k > 0);
        tc05::commit(smem_u32(&bar.o_done[mt]));
      }
    };
    auto full = [&](uint64_t (&b)[2], int i) {
      if (!wait1(&b[i & 1], (i >> 1) & 1)) return false;
      tc05::fence_after_sync();
      return true;
    };
    bool ok = wait1(&bar.q_full, 0);
    if constexpr (P::kMt == 2) {
      ok = ok && full(bar.k_full, 0);
      if (ok) {
        scores(0, 0, 0);
        scores(1, 1, 0);
        commit(&bar.k_empty[0]);
      }
      for (int i = 0; ok && i < n; ++i) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          if (mt == 0 && !(ok = full(bar.v_full, i))) break;
          if (!(ok = wait1(&bar.p_full[mt], i & 1))) break;
          tc05::fence_after_sync();
          outputs(mt, mt, i);
          if (mt == 1) commit(&bar.v_empty[i & 1]);
          if (i + 1 < n) {
            if (mt == 0 && !(ok = full(bar.k_full, i + 1))) break;
            scores(mt, mt, i + 1);
            if (mt == 1) commit(&bar.k_empty[(i + 1) & 1]);
          }
        }
      }
    } else {
      for (int i = 0; ok && i < 2 && i < n; ++i) {
        if (!(ok = full(bar.k_full, i))) break;
        scores(0, i, i);
        commit(&bar.k_empty[i]);
      }
      for (int i = 0; ok && i < n; ++i) {
        if (!(ok = full(bar.v_full, i) && wait1(&bar.p_full[i & 1], (i >> 1) & 1))) break;
        tc05::fence_after_sync();
        outputs(0, i & 1, i);
        commit(&bar.v_empty[i & 1]);
        if (i + 2 < n) {
          if (!(ok = full(bar.k_full, i + 2))) break;
          scores(0, i & 1, i + 2);
          commit(&bar.k_empty[i & 1]);
        }
      }
    }
    // all products that this thread issued have finished before the CTA moves on
    commit(&bar.drain);
    if (!mbar_wait_bounded(&bar.drain, 0, 1000000000ull) && leader) atomicOr(a.err, kErrDrain);
    }
  }
  __syncthreads();
  if (warp == P::kSoft + P::kConv) {
    tc05::fence_after_sync();
    tc05::dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch(const AttendArgs& a, int limit, cudaStream_t stream) {
  using P = Plan<D>;
  cudaError_t e = cudaFuncSetAttribute(kv_prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t rows = int64_t(a.b.max_new) * a.group, tiles = (rows + P::kRows - 1) / P::kRows;
  const int64_t grid = tiles * a.c.heads * a.b.n_seqs;
  if (grid > 0x7fffffff) return cudaErrorNotSupported;
  return launch_pdl(kv_prompt_kernel<D>, dim3(static_cast<unsigned>(grid)), dim3(P::kThreads), P::kSmem, stream, a, limit,
                    static_cast<int>(tiles), wait_limit_ns());
}

}  // namespace

cudaError_t launch_kv_prompt(const AttendArgs& a, int limit, cudaStream_t stream) {
  if (a.c.d <= 64) return launch<64>(a, limit, stream);
  if (a.c.d <= 128) return launch<128>(a, limit, stream);
  return launch<256>(a, limit, stream);
}

}  // namespace mq
