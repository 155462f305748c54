// Attention over the paged 8-bit cache for sequences with many query rows
// (prompts), on the fifth-generation tensor cores. Mathematics and masks are
// those of kv_attention.cu; here the products bound the time, not the bytes.
//
// An item is kMt tiles of 128 rows (query tokens times the heads of a group) of one
// sequence and key/value head, with the tokens that they see in tiles of kT. The
// tiles of all items together are cut into equal ranges, one per SM, so that few long
// prompts fill the card and no SM waits for another's last item; a second kernel
// joins the items that several SMs shared. Per tile and 128 rows: S = Q K^T (128 x kT, in tensor memory), softmax, P
// written over S as fp16, O += P V (128 x D, in tensor memory).
//   warps 0 .. 4 kMt - 1 : softmax, a thread a row: S from tensor memory, running
//                          maximum and sum in registers, P back; queries at the
//                          start and outputs at the end
//   kConv warps          : bytes to fp16 codes, K and V, into swizzled rows of
//                          shared memory (two buffers each)
//   one warp             : issues the products
//   one warp             : plans the CTA's pieces of items ahead of the others
// 2048 tokens upon as many cached ones of two sequences, 32 query and 8 key/value heads
// of 128 values: 272 to 275 us, 750 TFLOP/s of the pairs that count (11.3 ms in plain
// torch). Of a CTA's 440000 cycles 81 unmasked tiles (256 rows, 128 tokens) take some 4450
// each: 2950 of softmax, the rest waiting for the scores (products: 2048 at the tensor
// cores' rate) and the scales; 3.5 masked ones 6300 of softmax; 4.3 pieces 6000 each for
// their queries and 5900 for their outputs; the start 5000.
// Beside kv_attention.cu's roundings (queries and probabilities in fp16, the latter with
// their page's V scale), a quarter of the exponentials are a polynomial, within 2^-22.
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
#include <type_traits>

#include "../../include/mq.h"
#include "kv_internal.h"
#include "kv_pieces.cuh"
#include "mq_device.cuh"
#include "mq_internal.h"
#include "tc05.cuh"

namespace mq {
namespace {

constexpr float kPLog2 = 8.f;          // p' stands 2^8 high
constexpr float kTinyScale = 0x1p-100f;  // V scales below this count as this

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
// 2^x of two values on the multiply-add pipes, for x in [-126, 127]: 2^round(x) times a
// polynomial of degree 5 in the rest, |rest| <= 1/2, whose coefficients make the largest
// relative error smallest (2^-23.7; 2^-22.2 in fp32). Below -126, and for a NaN, it gives
// 2^-126. Above 127 the exponent runs into the sign: the caller looks out for such x.
__device__ __forceinline__ float2 exp2_poly(uint64_t x) {
  const float2 v = unpair(x);
  const uint64_t y = pair(fmaxf(v.x, -126.f), fmaxf(v.y, -126.f));
  const uint64_t t = add2(y, pair(12582912.f, 12582912.f));  // 1.5 2^23: the integer in the low bits
  const uint64_t f = fma2(add2(t, pair(-12582912.f, -12582912.f)), pair(-1.f, -1.f), y);
  uint64_t p = pair(0x1.5c08e6p-10f, 0x1.5c08e6p-10f);
  p = fma2(p, f, pair(0x1.3d0c52p-7f, 0x1.3d0c52p-7f));
  p = fma2(p, f, pair(0x1.c6b6e4p-5f, 0x1.c6b6e4p-5f));
  p = fma2(p, f, pair(0x1.ebf918p-3f, 0x1.ebf918p-3f));
  p = fma2(p, f, pair(0x1.62e428p-1f, 0x1.62e428p-1f));
  p = fma2(p, f, pair(0x1.000002p+0f, 0x1.000002p+0f));
  const float2 q = unpair(p), n = unpair(t);
  return make_float2(__uint_as_float(__float_as_uint(q.x) + (__float_as_uint(n.x) << 23)),
                     __uint_as_float(__float_as_uint(q.y) + (__float_as_uint(n.y) << 23)));
}
// Moves registers between the CTA's warpgroups: all four warps of one execute it.
template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
// True in one lane of the (converged) warp, always the same.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// D: the head's size rounded up to 64, 128 or 256. MT: tiles of 128 rows, 2 where one's
// softmax can run beside the other's products, 1 with S twice in turn where there is one (no
// sequence of the call has more rows) or room for one (at D = 256 the outputs take half of
// the tensor memory).
template <int D, int MT>
struct Plan {
  static constexpr int kMt = MT;
  static constexpr int kT = D == 256 ? 64 : 128;
  static constexpr int kSoft = 4 * kMt;
  static constexpr int kConv = MT == 1 ? 8 : 4;
  static constexpr int kThreads = 512;  // the last four warps: one issues the products
  // Registers of a softmax, a spreading and a product thread; the launch gives 128.
  static constexpr int kSoftRegs = MT == 1 ? 208 : 168, kConvRegs = 112, kMmaRegs = 64;
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
  // What an item costs beside its tiles, in tiles: queries in, outputs out, the first bytes.
  static constexpr int kStart = D == 256 ? 6 : 3;
};

struct alignas(16) TileScales {
  float2 group[8];  // K scale, log2 of V's factor
  float vmax;
  int dead;         // a bit for each group that may not be read
};

struct Bars {
  uint64_t q_full;
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], p_full[2], o_done[2];
  uint64_t sc_full[4];
  uint64_t plan_full[2], plan_empty[2];
  uint64_t drain;
};

// An item's rows and tokens.
struct Item {
  int row0, rows;   // of the sequence
  int past;         // place of the sequence's first row
  int lo, j0, j1;   // first token that some row sees, rounded down to a tile, and their end
  int n;            // tiles; 0 where no row sees a token
  int start, units; // in the split: before the first tile, and in all
};
template <int D, int MT>
__device__ __forceinline__ Item item_of(const AttendArgs& a, const Seq& sq, int rt) {
  using P = Plan<D, MT>;
  Item t;
  const int all = sq.n * a.group;
  t.row0 = rt * P::kRows;
  t.rows = min(P::kRows, all - t.row0);
  t.past = sq.len - sq.n;
  const int lo_place = t.past + t.row0 / a.group, hi_place = t.past + (t.row0 + t.rows - 1) / a.group;
  t.j1 = max(hi_place + 1, 0);
  t.lo = a.window > 0 ? max(lo_place - a.window + 1, 0) : 0;
  t.j0 = t.lo & ~(P::kT - 1);
  t.n = (t.j1 - t.j0 + P::kT - 1) / P::kT;
  t.start = t.n > 0 ? P::kStart : 0;
  t.units = t.n > 0 ? t.n + P::kStart : 1;
  return t;
}
template <int D, int MT>
__device__ __forceinline__ int item_rows(const AttendArgs& a, const Seq& sq, int limit) {
  const int all = sq.n * a.group;
  return all <= limit ? 0 : (all + Plan<D, MT>::kRows - 1) / Plan<D, MT>::kRows;
}

// A piece of an item, as the CTA's warps take it from shared memory.
struct Piece {
  int s, h, r0;           // sequence, head, the sequence's first row
  int row0, rows, all;    // of the sequence: the item's rows, all rows
  int past;               // place of the sequence's first row
  int lo, j0, j1;         // the item's tokens
  int n, t0, t1;          // its tiles, and the piece's; n < 0: the range is done
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == n; }
};

// A CTA's way through its range: sequences, their row tiles from the last, heads.
struct Place {
  int s, rt, h, u0;
};
template <int D, int MT>
struct Walk {
  Place at;
  Seq sq;
  Item it;
  int64_t left;  // units of the range
  int t0, t1;    // tiles of the piece
  __device__ __forceinline__ void piece() {
    const int u1 = static_cast<int>(min(int64_t(it.units), at.u0 + left));
    t0 = max(at.u0 - it.start, 0);
    t1 = max(u1 - it.start, 0);
    if (it.n == 0) t0 = t1 = 0;
  }
  __device__ __forceinline__ bool empty() const { return it.n > 0 && t0 >= t1; }
  __device__ __forceinline__ void start(const AttendArgs& a, const Place& p, int64_t units) {
    at = p;
    left = units;
    sq = load_seq(a.b, at.s, nullptr);
    it = item_of<D, MT>(a, sq, at.rt);
    piece();
  }
  __device__ __forceinline__ bool next(const AttendArgs& a, int limit) {
    left -= it.units - at.u0;
    if (left <= 0) return false;
    at.u0 = 0;
    if (++at.h == a.c.heads) {
      at.h = 0;
      if (--at.rt < 0) {
        do {
          sq = load_seq(a.b, ++at.s, nullptr);
          at.rt = item_rows<D, MT>(a, sq, limit) - 1;
        } while (at.rt < 0);
      }
      it = item_of<D, MT>(a, sq, at.rt);
    }
    piece();
    return true;
  }
};

template <int D, int MT>
__global__ void __launch_bounds__(Plan<D, MT>::kThreads, 1)
kv_prompt_kernel(const AttendArgs a, const Scratch scr, int limit, uint64_t wait_ns) {
  using P = Plan<D, MT>;
  constexpr int kT = P::kT, kThreads = P::kThreads, kWarps = kThreads / 32;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars bar;
  __shared__ TileScales s_scales[P::kSlots];
  __shared__ int64_t s_pre[kThreads + 1], s_warp[kWarps];
  __shared__ Piece s_piece[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort_word;
  volatile int* s_abort = &s_abort_word;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sq_base = base, sk_base = base + P::kQBytes, sv_base = sk_base + 2 * P::kKvBytes;

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
    for (int i = 0; i < P::kSlots; ++i) mbar_init(&bar.sc_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.plan_full[i], 1);
      mbar_init(&bar.plan_empty[i], P::kSoft + P::kConv + 1);
    }
    mbar_init(&bar.drain, 1);
    s_abort_word = 0;
    s_pre[0] = 0;
    fence_mbar_init();
  }
  pdl_launch_dependents();
  // This kernel follows kv_attend_kernel, which starts its dependents only when what came
  // before it is complete: so this one may begin at once, beside it, and waits for it at its
  // end, for the next kernel's sake.
  // ---- units before each run of sequences
  const int per = (a.b.n_seqs + kThreads - 1) / kThreads;
  auto seq_units = [&](int s) {  // of one sequence, by the warp
    const Seq sq = load_seq(a.b, s, nullptr);
    const int nrt = item_rows<D, MT>(a, sq, limit);
    int64_t units = 0;
    for (int rt = lane; rt < nrt; rt += 32) units += item_of<D, MT>(a, sq, rt).units;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) units += __shfl_xor_sync(0xffffffffu, units, o);
    return units * a.c.heads;
  };
  {  // a thread a run, neighbouring runs in different warps; sequences of many items by the warp
    const int run = lane * kWarps + warp;
    int64_t units = 0;
    for (int k = 0; k < per; ++k) {
      const int s = run * per + k;
      const Seq sq = s < a.b.n_seqs ? load_seq(a.b, s, nullptr) : Seq{0, 0, 0};
      const int nrt = item_rows<D, MT>(a, sq, limit);
      if (nrt <= 4)
        for (int rt = 0; rt < nrt; ++rt) units += int64_t(item_of<D, MT>(a, sq, rt).units) * a.c.heads;
      for (unsigned many = __ballot_sync(0xffffffffu, nrt > 4); many; many &= many - 1) {
        const int src = __ffs(many) - 1;
        const int64_t u = seq_units(__shfl_sync(0xffffffffu, s, src));
        if (lane == src) units += u;
      }
    }
    s_pre[run + 1] = units;
  }
  __syncthreads();
  int64_t inc = s_pre[tid + 1];
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
  s_pre[tid + 1] = (warp == 0 ? 0 : __shfl_sync(0xffffffffu, sums, warp - 1)) + inc;
  __syncthreads();
  // ---- this CTA's range: a few tiles at least
  const int cta = blockIdx.x;
  const int ctas = static_cast<int>(min(int64_t(gridDim.x), max((total + P::kStart) / (P::kStart + 1), int64_t(1))));
  if (tid == 0) scr.open[cta].rows = 0;
  if (cta >= ctas || total == 0) {
    pdl_wait_primary();
    return;
  }
  const Cut cut(total, ctas);
  const int64_t A = cut.first(cta), B = cut.first(cta + 1);
  if (warp == P::kSoft + P::kConv) {
    tc05::alloc(smem_u32(&s_tmem), 512);
    tc05::relinquish();
    tc05::fence_before_sync();
  }
  __syncthreads();
  tc05::fence_after_sync();
  const uint32_t tmem = s_tmem;
  const int d = a.c.d, chunks = d >> 4;
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

  // The CTA's k-th piece, or false at the end.
  auto piece_of = [&](int k, Piece& p) {
    if (!wait(&bar.plan_full[k & 1], (k >> 1) & 1, kErrWaitFull)) return false;
    p = s_piece[k & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar.plan_empty[k & 1]);
    return p.n >= 0;
  };

  if (warp < P::kSoft) {
    // ------------------------------------------------------------ softmax
    more_registers<P::kSoftRegs>();
    const int mt = warp >> 2, r = 32 * (warp & 3) + lane, lr = 128 * mt + r;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t t_o = tmem + lanes + P::kOCol + mt * D;
    const float cap_in = a.softcap > 0.f ? 1.f / a.softcap : 0.f, cap_out = a.softcap * kLog2e;
    bool ok = true;
    int tick = 0;  // tiles of this CTA before
    // Rows go to and from global memory with neighbouring lanes on one row (a lane a row would
    // touch 32 lines an instruction): lane = row sub, 16-byte chunk `chunk`.
    constexpr int kLanesRow = D / 8, kRowsAt = 32 / kLanesRow, kLoads = 32 / kRowsAt;
    const int sub = lane / kLanesRow, chunk = lane % kLanesRow;
    auto row_chunk = [&](int row, int c) {  // of this warp's 32 rows, in the queries' shared memory
      return sq_base + (mt * P::kBlocks + (c >> 3)) * P::kQBlock + (32 * (warp & 3) + row) * 128 + (((c & 7) ^ (row & 7)) << 4);
    };
    Piece w;
    for (int k = 0; piece_of(k, w); ++k) {
    const bool live = lr < w.rows;
    const int row = w.row0 + lr, qi = row / a.group, hq = w.h * a.group + row - qi * a.group;
    const int64_t grow = int64_t(w.r0) + qi;
    const int place = live ? w.past + qi : -1;
    float fac = 0.f;
    if (w.n > 0) {  // this warp's queries, each row scaled by a power of two to below 2
      const int64_t from = live ? grow * a.q_stride + int64_t(hq) * d : -1;
      constexpr int kBatch = kLoads < 16 ? kLoads : 16;  // loads on their way at once
#pragma unroll
      for (int k0 = 0; k0 < kLoads; k0 += kBatch) {
        uint4 u[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int64_t at = __shfl_sync(0xffffffffu, from, (k0 + k) * kRowsAt + sub);
          u[k] = at >= 0 && chunk < 2 * chunks ? *(reinterpret_cast<const uint4*>(a.q + at) + chunk) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const uint32_t x[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
          float mx = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(x[i] << 16)), fabsf(__uint_as_float(x[i] & 0xFFFF0000u))));
#pragma unroll
          for (int o = kLanesRow / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          int ex = __float_as_int(mx) >> 23;
          ex = ex < 1 || ex > 253 ? 127 : ex;
          const float down = __int_as_float((254 - ex) << 23) * (a.scale < 0.f ? -1.f : 1.f);
          const float up = __int_as_float(ex << 23) * fabsf(a.scale) * (a.softcap > 0.f ? 1.f : kLog2e);
          const float mine = __shfl_sync(0xffffffffu, up, (lane % kRowsAt) * kLanesRow);
          if (lane / kRowsAt == k0 + k) fac = mine;
          uint32_t y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = f16x2(__uint_as_float(x[i] << 16) * down, __uint_as_float(x[i] & 0xFFFF0000u) * down);
          sts128(row_chunk((k0 + k) * kRowsAt + sub, chunk), y[0], y[1], y[2], y[3]);
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.q_full);
    }
    // of the 32 rows of this warp
    const int first_row = w.row0 + 128 * mt + 32 * (warp & 3);
    int w_lo = w.past + first_row / a.group;
    const int w_hi = w.past + min(first_row + 31, w.all - 1) / a.group;
    // Rows behind the sequence's last (zero queries) keep a maximum of -infinity, which keeps
    // their sums out; what they get in P and O is finite and goes nowhere. A warp of them does nothing.
    const bool idle = first_row >= w.all;
    float m = -INFINITY, l = 0.f, vmax = kTinyScale;
    // A tile's scales (K's times this row's factor), taken while its scores are still being
    // made: the products keep shared memory busy, and a load waits for hundreds of cycles.
    float fs[P::kGroups], lg[P::kGroups], tile_vmax = 0.f;
    int dead = 0;
    auto take = [&](int tick) {
      const int slot = tick % P::kSlots;
      if (!wait(&bar.sc_full[slot], (tick / P::kSlots) & 1, kErrWaitFull)) return false;
      const TileScales& ts = s_scales[slot];
#pragma unroll
      for (int g = 0; g < P::kGroups; g += 2) {
        const float4 x = *reinterpret_cast<const float4*>(ts.group + g);
        fs[g] = fac * x.x, lg[g] = x.y, fs[g + 1] = fac * x.z, lg[g + 1] = x.w;
      }
      tile_vmax = ts.vmax;
      dead = ts.dead;
      return true;
    };
    if (w.t0 < w.t1 && !(ok = take(tick))) break;
    for (int i = w.t0; i < w.t1; ++i, ++tick) {
      const int slot = P::kMt == 2 ? mt : (tick & 1);
      if (!(ok = wait(&bar.s_full[slot], P::kMt == 2 ? (tick & 1) : ((tick >> 1) & 1), kErrWaitFull))) break;
      tc05::fence_after_sync();
      const uint32_t t_s = tmem + lanes + slot * kT;
      const int jt = w.j0 + i * kT;
      bool special = a.softcap > 0.f || dead || jt + kT - 1 > w_lo || (a.window > 0 && jt <= w_hi - a.window);
      const float2* group_scales = s_scales[tick % P::kSlots].group;
      auto factor = [&](int g) { return fac * group_scales[g].x; };
      // The scores of groups g, g + 1, scaled, and where some row of the warp needs it capped and masked.
      auto scores = [&](uint32_t (&v)[32], int g) {
        tc05::ld_32x32b_x32(t_s + 16 * g, v);
        const float f0 = factor(g), f1 = factor(g + 1);
        tc05::wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * (e < 16 ? f0 : f1));
        if (a.softcap > 0.f) {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(capped<true>(__uint_as_float(v[e]), cap_in, cap_out));
        }
        if (special) {
          const int hi = place - jt - 16 * g, low = a.window > 0 ? hi - a.window : -1;
          const int hi0 = (dead >> g) & 1 ? -1 : hi, hi1 = (dead >> g) & 2 ? -1 : hi;
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (e > (e < 16 ? hi0 : hi1) || e <= low) v[e] = __float_as_uint(-INFINITY);
        }
      };
      // The largest of groups g .. end - 1, or of as many as it takes for each row to see one.
      auto largest = [&](int g, int end, bool enough) {
        float top = -INFINITY;
#pragma unroll 1
        for (; g < end; g += 2) {
          uint32_t v[32];
          scores(v, g);
          float t[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) t[e] = __uint_as_float(v[e]);
#pragma unroll
          for (int e = 4; e < 32; ++e) t[e & 3] = fmaxf(t[e & 3], __uint_as_float(v[e]));
          top = fmaxf(top, fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])));
          if (enough && __all_sync(0xffffffffu, !live || top > -INFINITY)) break;
        }
        return top;
      };
      // Raises the maximum (an integer, so that the factors are powers of two) to `top` and
      // the V scale to the tile's; O, and the columns of P that are written, follow.
      float sum = 0.f;
      auto raise = [&](float top, int done) -> bool {
        const float x = fmaxf(ceilf(top), m), k = x == -INFINITY ? 1.f : exp2_fast(m - x), kv = k * (vmax / tile_vmax);
        l *= k;
        sum *= k;
        m = x;
        if (__any_sync(0xffffffffu, m != -INFINITY && fabsf(m) >= kCoarse)) special = true, w_lo = -1;  // from here on
        vmax = tile_vmax;
        tc05::wait_st();  // P so far
#pragma unroll 1
        for (int c = 0; c < done; c += 8) {
          uint32_t v[8];
          tc05::ld_32x32b_x8(t_s + c, v);
          tc05::wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e) {  // in fp32: the factor alone may be below what fp16 holds
            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&v[e]));
            v[e] = f16x2(y.x * k, y.y * k);
          }
          tc05::st_32x32b_x8(t_s + c, v);
        }
        if (i > w.t0) {
          if (!wait(&bar.o_done[mt], (tick - 1) & 1, kErrMma)) return false;
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
        }
        tc05::wait_st();
        return true;
      };
      // p' of 64 tokens at a time (32 where they are masked), over scores that are read
      // already. The running maximum is not looked for: a score that passes it by more than
      // 6 or so shows in its group's sum (or, as the polynomial's sums hold for small x only,
      // in the largest of those: half the price of a clamp), and its step is done over. Rows that have seen
      // nothing yet take a maximum first, of the tokens up to the first they see. Without branches within a step, for its
      // loads, exponentials and sums to mix, and rolled up, for the code to stay in the
      // instruction cache beside the other warps': unrolled over the tile, fetches were the
      // longest stall.
      // The special-function unit would take 2048 cycles of 256 rows' tile, as the products
      // do; every fourth pair of exponentials goes to the multiply-add pipes instead (which
      // leave 2^-126 of what is masked).
      // A step is done over once at most: the maximum is then at least that of its own scores
      // and no p' stands above 2^8 (but for the roundings below kCoarse), no group's sum above
      // 2^12. From a maximum beyond kCoarse on, the piece goes the way of the masked tiles.
      const bool first = __any_sync(0xffffffffu, live && m == -INFINITY);
      bool rise = first || tile_vmax != vmax, enough = true;
      int g0 = idle ? P::kGroups : 0, seek_to = first ? P::kGroups : 0;  // where a maximum is looked for ends
      while (g0 < P::kGroups) {
        if (rise) {
          if (!(ok = raise(largest(g0, seek_to, enough), 8 * g0))) break;
          rise = false;
        }
        const float m0 = m == -INFINITY ? 0.f : m;
        float part = 0.f, big = 0.f, over = 0.f;
        auto group = [&](const uint32_t* x, float f, float lg, float m0, uint32_t* pk) {
          const uint64_t f2 = pair(f, f), c2 = pair(lg - m0, lg - m0);
          uint64_t s0 = 0, s1 = 0;
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const uint64_t x2 = fma2(pair(x[e], x[e + 1]), f2, c2), y2 = fma2(pair(x[e + 2], x[e + 3]), f2, c2);
            const float2 y = unpair(y2), z = unpair(x2);
            const float2 p = make_float2(exp2_fast(z.x), exp2_fast(z.y));
            const float2 q = e % 8 == 4 ? exp2_poly(y2) : make_float2(exp2_fast(y.x), exp2_fast(y.y));
            if (e % 8 == 4) over = fmaxf(over, fmaxf(y.x, y.y));
            s0 = add2(s0, pair(p.x, p.y));
            s1 = add2(s1, pair(q.x, q.y));
            pk[e / 2] = f16x2(p.x, p.y);
            pk[e / 2 + 1] = f16x2(q.x, q.y);
          }
          const float2 t = unpair(add2(s0, s1));
          big = fmaxf(big, t.x + t.y);
          part = fmaf(t.x + t.y, exp2_fast(-lg), part);
        };
        int step;
        if (!special) {
          step = 4;
          uint32_t v[2][32], pk[32];
          tc05::ld_32x32b_x32(t_s + 16 * g0, v[0]);
          tc05::ld_32x32b_x32(t_s + 16 * g0 + 32, v[1]);
          tc05::wait_ld();
#pragma unroll
          for (int g = 0; g < 4; ++g) group(v[g / 2] + 16 * (g & 1), fs[g], lg[g], m0, pk + 8 * g);
          rise = (enough || g0 >= seek_to) && __any_sync(0xffffffffu, big > 32768.f || over > 15.f);
          if (!rise) tc05::st_32x32b_x32(t_s + 8 * g0, pk);
        } else {
          step = 2;
          uint32_t v[32], pk[16];
          scores(v, g0);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) - m0);  // see kCoarse
          group(v, 1.f, group_scales[g0].y, 0.f, pk);
          group(v + 16, 1.f, group_scales[g0 + 1].y, 0.f, pk + 8);
          rise = (enough || g0 >= seek_to) && __any_sync(0xffffffffu, big > 32768.f || over > 15.f);
          if (!rise) tc05::st_32x32b_x16(t_s + 8 * g0, pk);
        }
        if (rise) {  // done over, with the maximum of all its scores
          enough = false;
          seek_to = g0 + step;
        } else {
          sum += part;
          g0 += step;
#pragma unroll
          for (int g = 0; g + 4 < P::kGroups; ++g) fs[g] = fs[g + 4], lg[g] = lg[g + 4];  // the next whole step's
        }
      }
      if (!ok) break;
      if (m != -INFINITY || sum != sum) l += sum;  // a NaN is passed on, though it is no maximum
      tc05::wait_st();
      // A wait on a barrier tells a phase from the one before it only, so no warp may leave a
      // tile's products further behind. Two tiles of rows: the scores came after them. S twice
      // in turn: they may still run, and this tile's cannot start before this warp arrives.
      if (P::kMt == 1 && i > w.t0 && !(ok = wait(&bar.o_done[mt], (tick - 1) & 1, kErrMma))) break;
      tc05::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.p_full[slot]);
      if (i + 1 < w.t1 && !(ok = take(tick + 1))) break;
    }
    if (!ok) break;
    // ---- outputs, or this piece's sums
    const bool any = w.t0 < w.t1;
    if (any && !(ok = wait(&bar.o_done[mt], (tick - 1) & 1, kErrMma))) break;
    tc05::fence_after_sync();
    // (through the queries' shared memory, which no product reads any more)
    const float unit = vmax * 0x1p-8f;
    if (w.whole()) {
      const float inv = l > 0.f ? unit / l : (l == 0.f ? 0.f : l);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[32] = {};
        if (any) {
          tc05::ld_32x32b_x32(t_o + 32 * c, v);
          tc05::wait_ld();
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(v[8 * k + 2 * e]) * inv, __uint_as_float(v[8 * k + 2 * e + 1]) * inv);
            x[e] = *reinterpret_cast<const uint32_t*>(&b);
          }
          sts128(row_chunk(lane, 4 * c + k), x[0], x[1], x[2], x[3]);
        }
      }
      __syncwarp();
      const int64_t to = live ? grow * a.out_stride + int64_t(hq) * d : -1;
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const int64_t at = __shfl_sync(0xffffffffu, to, k * kRowsAt + sub);
        const uint4 x = lds128(row_chunk(k * kRowsAt + sub, chunk));
        if (at >= 0 && chunk < 2 * chunks) reinterpret_cast<uint4*>(a.out + at)[chunk] = x;
      }
      if (a.lse && live) a.lse[grow * (a.c.heads * a.group) + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    } else {
      float* part = scr.joined + int64_t(2 * cta + (w.t0 > 0 ? 0 : 1)) * scr.slot_floats;
      if (live) *reinterpret_cast<float2*>(part + scr.rows * d + 2 * lr) = make_float2(m, l);
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {  // D / 2 columns: as many bytes as a row of queries
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint32_t v[32];
          tc05::ld_32x32b_x32(t_o + half * (D / 2) + 32 * c, v);
          tc05::wait_ld();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            uint32_t x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = __float_as_uint(__uint_as_float(v[4 * k + e]) * unit);
            sts128(row_chunk(lane, 8 * c + k), x[0], x[1], x[2], x[3]);
          }
        }
        __syncwarp();
        const int col = half * (D / 2) + 4 * chunk, first = 128 * mt + 32 * (warp & 3);
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          const int row = k * kRowsAt + sub;
          const uint4 x = lds128(row_chunk(row, chunk));
          if (first + row < w.rows && col < d) *reinterpret_cast<uint4*>(part + int64_t(first + row) * d + col) = x;
        }
        __syncwarp();
      }
      if (w.t0 == 0 && tid == 0)  // the item goes on in the next CTAs
        scr.open[cta] = Open{w.r0, w.row0, w.h, w.rows, cut.part(B - 1 + (w.n - w.t1)) - cta + 1};
    }
    tc05::fence_before_sync();
    __syncwarp();
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
    Piece w;
    // lane g < kGroups: the page of group g of a tile
    auto page_of = [&](int i) {
      const int j = w.j0 + i * kT + 16 * lane;
      return lane < P::kGroups && j < w.j1 && j + 16 > w.lo ? a.b.pages[int64_t(w.s) * a.b.max_pages + (j >> log2p)] : -1;
    };
    // checked where it is used, so that the load runs ahead
    auto checked = [&](int pid, int i) {
      const int j = w.j0 + i * kT + 16 * lane;
      if (pid >= 0 && pid < a.c.n_pages) return pid;
      if (lane < P::kGroups && j < w.j1 && j + 16 > w.lo) atomicOr(a.err, kErrBounds);
      return -1;
    };
    uint4 xk[kIt], xv[kIt];
    float2 sc = make_float2(0.f, 0.f);  // lane's group: K, V scale
    const uint32_t mine = tk * d + 16 * c;
    auto fetch = [&](int i, int pid) {
      // where this lane's group starts in the cache (-1: nowhere)
      const int64_t tl = int64_t(pid) * a.c.heads + w.h;
      const int64_t group = pid < 0 ? -1 : (tl * page + ((w.j0 + i * kT + 16 * lane) & (page - 1))) * d;
      sc = make_float2(0.f, 0.f);
      if (pid >= 0) sc = make_float2(a.c.k_scale[tl], a.c.v_scale[tl]);
#pragma unroll
      for (int k = 0; k < kIt; ++k) {
        const int first = cw * kTokens + k * kAt;  // token of the tile
        const int64_t at = __shfl_sync(0xffffffffu, group, first >> 4);
        xk[k] = xv[k] = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
        if (at >= 0 && c < chunks) {
          const int64_t off = at + ((first & 15) * d + mine);
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
    int tick = 0;
    bool ok = true;
    for (int k = 0; ok && piece_of(k, w); ++k) {
    if (w.n == 0) continue;
    float vmax = kTinyScale;
    int pid = checked(page_of(w.t0), w.t0);
    fetch(w.t0, pid);
    int next = w.t0 + 1 < w.t1 ? page_of(w.t0 + 1) : -1;
    for (int i = w.t0; i < w.t1; ++i, ++tick) {
      const int b = tick & 1;
      const uint32_t parity = ((tick >> 1) & 1) ^ 1;
      if (tick >= 2 && !(ok = wait(&bar.k_empty[b], parity, kErrWaitEmpty))) break;
      if (cw == 0) {  // the tile's scales
        float top = lane < P::kGroups ? sc.y : 0.f;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (top > vmax) {  // the power of two at or above it
          const int e = (__float_as_int(top) + 0x7FFFFF) >> 23;
          vmax = __int_as_float(min(e, 254) << 23);
        }
        const float lg = log2f(fmaxf(sc.y / vmax, 0x1p-60f)) + kPLog2;
        TileScales& ts = s_scales[tick % P::kSlots];
        const int j = w.j0 + i * kT + 16 * lane;
        if (lane < P::kGroups) ts.group[lane] = make_float2(sc.x, lg);
        const unsigned dead = __ballot_sync(0xffffffffu, lane < P::kGroups && j < w.j1 && pid < 0);
        if (lane == 0) {
          ts.vmax = vmax;
          ts.dead = static_cast<int>(dead);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.sc_full[tick % P::kSlots]);
      }
      spread(sk_base + b * P::kKvBytes, xk);
      if (lane == 0) mbar_arrive(&bar.k_full[b]);
      if (tick >= 2 && !(ok = wait(&bar.v_empty[b], parity, kErrWaitEmpty))) break;
      spread(sv_base + b * P::kKvBytes, xv);
      if (lane == 0) mbar_arrive(&bar.v_full[b]);
      if (i + 1 < w.t1) {
        pid = checked(next, i + 1);
        fetch(i + 1, pid);
        if (i + 2 < w.t1) next = page_of(i + 2);
      }
    }
    }
  } else {
    // ------------------------------------------------------------ products
    fewer_registers<P::kMmaRegs>();
    // The whole warp walks the loop, so that descriptors stay in uniform registers
    // (a lone thread's moves to them cost more than the products); one lane issues.
    if (warp == P::kSoft + P::kConv) {
    const bool leader = elect_one();
    auto wait1 = [&](uint64_t* b, uint32_t parity) { return wait(b, parity, kErrMma); };
    auto commit = [&](uint64_t* b) {
      if (leader) tc05::commit(smem_u32(b));
    };
    constexpr uint32_t id_s = tc05::idesc_f16_f32(128, kT, false), id_o = tc05::idesc_f16_f32(128, D, true);
    // One thread issues every product: their descriptors are sums of a base and constants (16-byte units).
    const uint64_t desc_q = tc05::desc_kmajor_sw128(sq_base), desc_k = tc05::desc_kmajor_sw128(sk_base);
    const uint64_t desc_v = tc05::desc_mnmajor_sw128(sv_base, P::kBlocks > 1 ? P::kKvBlock : 1024);
    auto scores = [&](int mt, int slot, int tick) {  // S = Q K^T
      const uint64_t q = desc_q + mt * (P::kBlocks * P::kQBlock >> 4), k0 = desc_k + (tick & 1) * (P::kKvBytes >> 4);
      const uint32_t to = tmem + slot * kT;
      if (leader) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc05::mma_ss(to, q + (((k >> 2) * P::kQBlock + (k & 3) * 32) >> 4), k0 + (((k >> 2) * P::kKvBlock + (k & 3) * 32) >> 4),
                       id_s, k > 0);
        tc05::commit(smem_u32(&bar.s_full[slot]));
      }
    };
    auto outputs = [&](int mt, int slot, int tick, bool first) {  // O += P V
      const uint64_t v0 = desc_v + (tick & 1) * (P::kKvBytes >> 4);
      const uint32_t to = tmem + P::kOCol + mt * D, p = tmem + slot * kT;
      if (leader) {
#pragma unroll
        for (int k = 0; k < kT / 16; ++k) tc05::mma_ts(to, p + 8 * k, v0 + (k * 2048 >> 4), id_o, !first || k > 0);
        tc05::commit(smem_u32(&bar.o_done[mt]));
      }
    };
    auto full = [&](uint64_t (&b)[2], int tick) {
      if (!wait1(&b[tick & 1], (tick >> 1) & 1)) return false;
      tc05::fence_after_sync();
      return true;
    };
    bool ok = true;
    int tick = 0, pieces = 0;
    Piece w;
    for (int k = 0; ok && piece_of(k, w); ++k) {
      if (w.n == 0) continue;  // rows that see no token
      if (!(ok = wait1(&bar.q_full, pieces++ & 1))) break;
      const int n = w.t1 - w.t0;
      if constexpr (P::kMt == 2) {
        if (!(ok = full(bar.k_full, tick))) break;
        scores(0, 0, tick);
        scores(1, 1, tick);
        commit(&bar.k_empty[tick & 1]);
        for (int i = 0; ok && i < n; ++i, ++tick) {
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            if (mt == 0 && !(ok = full(bar.v_full, tick))) break;
            if (!(ok = wait1(&bar.p_full[mt], tick & 1))) break;
            tc05::fence_after_sync();
            outputs(mt, mt, tick, i == 0);
            if (mt == 1) commit(&bar.v_empty[tick & 1]);
            if (i + 1 < n) {
              if (mt == 0 && !(ok = full(bar.k_full, tick + 1))) break;
              scores(mt, mt, tick + 1);
              if (mt == 1) commit(&bar.k_empty[(tick + 1) & 1]);
            }
          }
        }
      } else {
        for (int i = 0; i < 2 && i < n; ++i) {
          if (!(ok = full(bar.k_full, tick + i))) break;
          scores(0, (tick + i) & 1, tick + i);
          commit(&bar.k_empty[(tick + i) & 1]);
        }
        for (int i = 0; ok && i < n; ++i, ++tick) {
          if (!(ok = full(bar.v_full, tick) && wait1(&bar.p_full[tick & 1], (tick >> 1) & 1))) break;
          tc05::fence_after_sync();
          outputs(0, tick & 1, tick, i == 0);
          commit(&bar.v_empty[tick & 1]);
          if (i + 2 < n) {
            if (!(ok = full(bar.k_full, tick + 2))) break;
            scores(0, tick & 1, tick + 2);
            commit(&bar.k_empty[tick & 1]);
          }
        }
      }
    }
    // all products that this thread issued have finished before the CTA moves on
    commit(&bar.drain);
    if (!mbar_wait_bounded(&bar.drain, 0, 1000000000ull) && leader) atomicOr(a.err, kErrDrain);
    } else if (warp == P::kSoft + P::kConv + 1) {
    // ------------------------------------------------------------ the pieces of this range
    Place at{};
    int run = (__popc(__ballot_sync(0xffffffffu, s_pre[lane * kWarps] <= A)) - 1) * kWarps;
    run += __popc(__ballot_sync(0xffffffffu, lane < kWarps && s_pre[run + lane] <= A)) - 1;
    int s = run * per;
    int64_t off = A - s_pre[run];
    while (true) {
      const int64_t u = seq_units(s);
      if (off < u) break;
      off -= u;
      ++s;
    }
    const Seq sq = load_seq(a.b, s, nullptr);
    for (int first = item_rows<D, MT>(a, sq, limit) - 1;; first -= 32) {
      const int rt = first - lane;
      const int units = rt >= 0 ? item_of<D, MT>(a, sq, rt).units : 0;
      int64_t upto = int64_t(units) * a.c.heads;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += up;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, off < upto);
      if (hit) {
        const int src = __ffs(hit) - 1;
        if (lane == src) {
          const int64_t rest = off - (upto - int64_t(units) * a.c.heads);
          at = Place{s, rt, static_cast<int>(rest / units), static_cast<int>(rest % units)};
        }
        at.s = __shfl_sync(0xffffffffu, at.s, src);
        at.rt = __shfl_sync(0xffffffffu, at.rt, src);
        at.h = __shfl_sync(0xffffffffu, at.h, src);
        at.u0 = __shfl_sync(0xffffffffu, at.u0, src);
        break;
      }
      off -= __shfl_sync(0xffffffffu, upto, 31);
    }
    Walk<D, MT> w;
    w.start(a, at, B - A);
    int k = 0;
    auto publish = [&](int n) {
      // this warp alone waits for whole pieces: up to a thousand times what the others wait for a step
      if (k >= 2) {
        bool free = false;
        for (int i = 0; i < 1000 && !free && !__any_sync(0xffffffffu, *s_abort != 0); ++i)
          free = __all_sync(0xffffffffu, mbar_wait_bounded(&bar.plan_empty[k & 1], ((k >> 1) & 1) ^ 1, wait_ns));
        if (!free && !wait(&bar.plan_empty[k & 1], ((k >> 1) & 1) ^ 1, kErrWaitEmpty)) return false;
      }
      if (lane == 0) {
        s_piece[k & 1] = Piece{w.at.s, w.at.h, w.sq.r0, w.it.row0, w.it.rows, w.sq.n * a.group, w.it.past, w.it.lo, w.it.j0, w.it.j1,
                               n, w.t0, w.t1};
        mbar_arrive(&bar.plan_full[k & 1]);
      }
      ++k;
      return true;
    };
    bool ok = true;
    do {
      if (!w.empty()) ok = publish(w.it.n);
    } while (ok && w.next(a, limit));
    if (ok) publish(-1);
    }
  }
  __syncthreads();
  if (warp == P::kSoft + P::kConv) {
    tc05::fence_after_sync();
    tc05::dealloc(tmem, 512);
  }
  pdl_wait_primary();
}

// Joins what several CTAs shared: blocks y < kJoinShare a share of the rows of a prompt's
// item, a warp a row; the others a row of kv_attend_kernel's.
constexpr int kJoinShare = 16;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32)
kv_prompt_join_kernel(const AttendArgs a, const Scratch sc, const Scratch few) {
  __shared__ JoinShared<D> shared;
  pdl_launch_dependents();
  pdl_wait_primary();
  const int c = blockIdx.x;
  if (blockIdx.y >= kJoinShare) {
    join_open<D>(a, few, few.open[c], c, blockIdx.y - kJoinShare, shared);
    return;
  }
  const Open p = sc.open[c];
  for (int lr = blockIdx.y * kJoinWarps + (threadIdx.x >> 5); lr < p.rows; lr += kJoinShare * kJoinWarps) {
    Joined<D> r;
    join_row<D>(sc.rows, a.c.d, lr, p.n, [&](int k) { return sc.joined + int64_t(2 * (c + k) + (k == 0 ? 1 : 0)) * sc.slot_floats; }, r);
    write_row<D>(a, row_out(a, p.r0, p.h, p.first_row + lr), r);
  }
}

template <int D, int MT>
size_t layout(const KvCache& c, const KvBatch& b, int group, int sms, Scratch* sc = nullptr, uint8_t* base = nullptr) {
  const int rows = part_rows(b.max_new, group, Plan<D, MT>::kRows), floats = part_floats(rows, c.d);
  const size_t open = align256(size_t(sms) * sizeof(Open));
  if (sc) *sc = Scratch{nullptr, reinterpret_cast<float*>(base + open), reinterpret_cast<Open*>(base), rows, floats};
  return open + align256(size_t(2) * sms * floats * 4);
}

template <int D, int MT>
cudaError_t launch(const AttendArgs& a, int limit, const Scratch& few, uint8_t* scratch, cudaStream_t stream, int sms) {
  using P = Plan<D, MT>;
  cudaError_t e = cudaFuncSetAttribute(kv_prompt_kernel<D, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::kSmem);
  if (e != cudaSuccess) return e;
  Scratch sc;
  layout<D, MT>(a.c, a.b, a.group, sms, &sc, scratch);
  e = launch_pdl(kv_prompt_kernel<D, MT>, dim3(sms), dim3(P::kThreads), P::kSmem, stream, a, sc, limit, wait_limit_ns());
  if (e != cudaSuccess) return e;
  return launch_pdl(kv_prompt_join_kernel<D>, dim3(sms, kJoinShare + few.rows), dim3(kJoinWarps * 32), 0, stream, a, sc, few);
}

}  // namespace

// One tile of rows does for calls whose sequences have up to 128 rows.
static bool one_tile(int64_t max_new, int group) { return max_new * group <= 128; }

size_t kv_prompt_scratch(const KvCache& c, const KvBatch& b, int group, int sms) {
  if (c.d > 128) return layout<256, 1>(c, b, group, sms);
  if (one_tile(b.max_new, group)) return c.d <= 64 ? layout<64, 1>(c, b, group, sms) : layout<128, 1>(c, b, group, sms);
  return c.d <= 64 ? layout<64, 2>(c, b, group, sms) : layout<128, 2>(c, b, group, sms);
}

cudaError_t launch_kv_prompt(const AttendArgs& a, int limit, const Scratch& few, uint8_t* scratch, cudaStream_t stream, int sms) {
  if (a.c.d > 128) return launch<256, 1>(a, limit, few, scratch, stream, sms);
  if (one_tile(a.b.max_new, a.group))
    return a.c.d <= 64 ? launch<64, 1>(a, limit, few, scratch, stream, sms) : launch<128, 1>(a, limit, few, scratch, stream, sms);
  return a.c.d <= 64 ? launch<64, 2>(a, limit, few, scratch, stream, sms) : launch<128, 2>(a, limit, few, scratch, stream, sms);
}

}  // namespace mq
