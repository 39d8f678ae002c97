// moe_fp4.cu -- rows in microscaled 4-bit floating point (e2m1: 0, 0.5, 1, 1.5,
// 2, 3, 4, 6 and their negatives) and the experts' product of such rows with
// such weights.
//
// A block of values shares a scale s, in 8 bits; with a tensor's own scale g:
//   MX  blocks of 32, s the smallest power of two with max |x| <= 6 s: no value of
//       a block is cut off (the power below would cut those above 6 s, up to a
//       quarter of them, for half the step)
//   NV  blocks of 16, s = max |x| / (6 g) rounded to e4m3
//   code = x / (s g) rounded to the nearest e2m1, ties to the even code
// The quotient is CUDA's correctly rounded one (MX: a product with a power of two,
// exact): a value next to a border of two codes goes where it belongs.
//
// quantize_kernel, dequantize_kernel: one pass; a lane has 8 values (16 bytes), 2
// or 4 neighbouring lanes a block.  With an activation the values are act(g) u
// of a row's halves, in 32 bits.
//
// fp4_kernel: y_r = gx gw_e sum_b sx_rb sw_b sum_i x_ri w_i, as y^T = W^T x^T on the
// block-scaled tensor cores, by CTA pairs (cta_group::2): the M side 256 features of
// an expert, the N side 32 to 192 of its rows.  A slice of K is 256 values, one
// 128-byte swizzled row; a CTA loads its own 128 features, half of the rows, and the
// scales of both (all of the rows': either half of the product needs them).
//   warp 0     TMA producer: codes and scales of both sides into a ring
//   warp 1     MMA issuer (first CTA): copies a slice's scales from shared memory
//              into TMEM (tcgen05.cp) and issues its four tcgen05.mma, K 64
//   warps 2-9  epilogue, as in moe_expert.cu
//   warps 10-13  scales as they lie beside the codes (a row's one after another) into
//              the order that TMEM takes: 4 scales of each of 128 rows, row r at
//              word r / 32 of 16-byte line r % 32, in the place where they landed
// 192 rows (NV: 160), not 256: two accumulators and five (NV: four) slots of scales fill TMEM.
// What bounds it is the way of a stage around its ring (copies, placing, MMAs and back,
// some 3000 cycles for 6 stages), then the issue of a slice (12 or 6 tcgen05.cp
// and 4 MMAs from one thread, 450 cycles); the MMAs of a slice are 330.
//
// Measured.  32768 x 7168 in bf16, MX: 105 to 114 us to codes (78 to 84 % of the copy rate),
// 99 to 103 back; NV 149 to 151 to codes, 105 back.  In 32 bits: MX 179, back 249; NV 197,
// back 253.  32768 x 2048 of act(g) u: NV 69 us with SiLU, 167 with GELU; MX 57, 162.
// Product, 32 experts, 1024 rows each: 7168 x 4096 NV 455 us (4.2 PFLOP/s), MX 409; 2048 x
// 7168 NV 306 (3.15 PFLOP/s; 584 with 2-byte stores from single CTAs), MX 284; 64 rows, 7168
// x 4096, NV: 75 us, the weights at 90 % of the copy rate.
#include <algorithm>
#include <string>

#include "moe_experts.cuh"

using namespace experts;
using namespace symm_host;

namespace {

// ------------------------------------------------------- rows to codes --
constexpr uint32_t kQuantThreads = 256;

struct QuantArgs {
  const void* x;
  size_t ldx;       // elements
  uint8_t *codes, *scales;
  size_t ldc, lds;  // bytes
  const float* g;
  uint32_t n, k, kv;  // rows, values and vectors of 8 values of a row
};

// Vectors of rows [n][kv] in turn: this thread's next one is `step` vectors on.
struct Walk {
  uint32_t row, col, step_row, step_col, kv;
  __device__ __forceinline__ explicit Walk(uint32_t kv_) : kv(kv_) {
    const uint32_t step = gridDim.x * kQuantThreads;
    const uint32_t first = blockIdx.x * kQuantThreads + threadIdx.x;
    row = first / kv, col = first % kv;
    step_row = step / kv, step_col = step % kv;
  }
  __device__ __forceinline__ void next() {
    row += step_row, col += step_col;
    if (col >= kv) col -= kv, ++row;
  }
};

template <typename T>
struct Vec8 {
  uint4 v[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Vec8<T> load8(const T* p) {
  Vec8<T> r;
#pragma unroll
  for (size_t i = 0; i < sizeof(T) / 2; ++i)
    r.v[i] = symm::ld16_ro(reinterpret_cast<const uint4*>(p) + i);
  return r;
}
template <typename T>
__device__ __forceinline__ void floats(const Vec8<T>& r, float (&f)[8]) {
  const T* t = reinterpret_cast<const T*>(&r);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = moe::to_f(t[i]);
}

// 8 codes, the first in the lowest bits.
__device__ __forceinline__ uint32_t to_codes(const float (&q)[8]) {
  uint32_t c;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(c)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return c;
}
__device__ __forceinline__ void from_codes(uint32_t c, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(c));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(h + i));
    v[2 * i] = f.x, v[2 * i + 1] = f.y;
  }
}
// e4m3 of a value that is not negative, at most 448, to the nearest, and back.
__device__ __forceinline__ uint32_t to_e4m3(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(v));
  return r & 0xffu;
}
__device__ __forceinline__ float from_e4m3(uint32_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)b));
  return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}
__device__ __forceinline__ float power_of_two(int e) {  // -127 <= e <= 127
  return __uint_as_float(e == -127 ? 0x400000u : (uint32_t)(e + 127) << 23);
}

// The largest magnitude of 8 values, as the bits of a float (a NaN's are the largest).
template <typename T>
__device__ __forceinline__ uint32_t top_of(const Vec8<T>& r) {
  uint32_t m = 0;
  if (sizeof(T) == 4) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7fffffffu);
    return m;
  }
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
  const uint16_t t = (uint16_t)max(m & 0xffffu, m >> 16);
  return __float_as_uint(moe::to_f(*reinterpret_cast<const T*>(&t)));
}
// Codes and the scale's byte of a lane's 8 values and their block's largest magnitude.
template <int FMT>
__device__ __forceinline__ uint32_t encode(float (&f)[8], uint32_t top, float g, uint32_t& byte) {
  const bool finite = top < 0x7f800000u;
  if (FMT == SYMM_FP4_MX) {
    // top = m 2^e with 1 <= m < 2: 6 2^(e - 2) reaches it up to m = 1.5
    int e = (int)(top >> 23) - 127;
    if (e == -127) e = -1000;  // below 2^-126 the smallest scale reaches anything
    e = max(-127, min(127, e - 2 + ((top & 0x7fffffu) > 0x400000u)));
    byte = finite ? (uint32_t)(e + 127) : 0xffu;
    const float s = power_of_two(-e);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= s;
  } else {
    byte = finite ? to_e4m3(fminf(__fdiv_rn(__uint_as_float(top), __fmul_rn(6.f, g)), 448.f))
                  : 0x7fu;
    const float unit = __fmul_rn(from_e4m3(byte), g);
    if (!(unit > 0.f)) return 0;
    // (largest quotients above 2^20 go by the division: near 2^128 q would be infinite and
    // its remainder NaN, whose code is +6)
    if (unit > 0x1p-100f && unit < 0x1p100f && __uint_as_float(top) < 0x1p20f * unit) {
      // Markstein (1990): y = RN(1 / b), q = RN(a y), r = a - q b by fma; RN(q + r y) is the
      // correctly rounded a / b.  q is within 1.5 ulp of a / b, and q + r y within 2^-24 of
      // that before its rounding, which matters only next to a midpoint of two floats; there
      // a float as near as q is half an ulp off and r is exact, the theorem's case.  (Of a
      // tiny a, r may underflow: its code is 0 either way.  -0 would become 0.)
      const float y = __frcp_rn(unit);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float q = f[i] * y;
        f[i] = copysignf(fmaf(fmaf(-q, unit, f[i]), y, q), f[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __fdiv_rn(f[i], unit);
    }
  }
  return finite ? to_codes(f) : 0;
}

// Four vectors (two with an activation, whose rows are two) in flight a thread: 105 us for
// 32768 x 7168 in bf16, where one took 188.
template <typename T, int FMT, int ACT>
__global__ void __launch_bounds__(kQuantThreads) quantize_kernel(const QuantArgs a) {
  constexpr uint32_t kLanes = FMT == SYMM_FP4_MX ? 4 : 2;  // of a block
  constexpr bool GATED = ACT != SYMM_ACT_NONE;
  constexpr int kFlight = GATED || sizeof(T) == 4 ? 2 : 4;
  moe::wait_for_earlier();
  const float g = a.g ? *a.g : 1.f;
  Walk w(a.kv);
  // whole warps go round: a block's lanes are of one row, and there or not together
  while (__any_sync(0xffffffffu, w.row < a.n)) {
    Vec8<T> r[kFlight], r2[GATED ? kFlight : 1];
    uint32_t row[kFlight], col[kFlight];
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      row[i] = w.row, col[i] = w.col;
      r[i] = Vec8<T>();
      if (GATED) r2[i] = Vec8<T>();
      if (w.row < a.n) {
        const T* x = static_cast<const T*>(a.x) + (size_t)w.row * a.ldx + 8 * w.col;
        r[i] = load8(x);
        if (GATED) r2[i] = load8(x + a.k);
      }
      w.next();
    }
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      if (i && !__any_sync(0xffffffffu, row[i] < a.n)) break;
      float f[8];
      floats(r[i], f);
      uint32_t top = 0, byte;
      if (GATED) {
        float u[8];
        floats(r2[i], u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          f[j] = activate(ACT, f[j]) * u[j];
          top = max(top, __float_as_uint(f[j]) & 0x7fffffffu);
        }
      } else {
        top = top_of(r[i]);
      }
#pragma unroll
      for (uint32_t o = 1; o < kLanes; o *= 2)
        top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const uint32_t code = encode<FMT>(f, top, g, byte);
      if (row[i] < a.n) {
        *reinterpret_cast<uint32_t*>(a.codes + row[i] * a.ldc + 4 * col[i]) = code;
        if (threadIdx.x % kLanes == 0)
          a.scales[row[i] * a.lds + col[i] / kLanes] = (uint8_t)byte;
      }
    }
  }
}

struct DequantArgs {
  const uint8_t *codes, *scales;
  size_t ldc, lds;  // bytes
  const float* g;
  void* y;
  size_t ldy;  // elements
  uint32_t n, kv;
};
template <typename T, int FMT>
__global__ void __launch_bounds__(kQuantThreads) dequantize_kernel(const DequantArgs a) {
  constexpr uint32_t kLanes = FMT == SYMM_FP4_MX ? 4 : 2;
  moe::wait_for_earlier();
  const float g = a.g ? *a.g : 1.f;
  for (Walk w(a.kv); w.row < a.n; w.next()) {
    const uint32_t code =
        __ldg(reinterpret_cast<const uint32_t*>(a.codes + w.row * a.ldc) + w.col);
    const uint32_t byte = __ldg(a.scales + w.row * a.lds + w.col / kLanes);
    float unit;
    if (FMT == SYMM_FP4_MX)
      unit = byte == 0xffu ? __uint_as_float(0x7fffffffu) : power_of_two((int)byte - 127);
    else
      unit = from_e4m3(byte);
    if (a.g) unit = __fmul_rn(unit, g);
    float f[8];
    from_codes(code, f);
    __align__(16) T out[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = moe::from_f<T>(__fmul_rn(f[i], unit));
    uint4* y = reinterpret_cast<uint4*>(static_cast<T*>(a.y) + w.row * a.ldy + 8 * w.col);
#pragma unroll
    for (size_t i = 0; i < sizeof(T) / 2; ++i) y[i] = reinterpret_cast<const uint4*>(out)[i];
  }
}

// ------------------------------------------------------------ fp4_kernel --
constexpr uint32_t kThreads = 448, kEpilogue = 256;
constexpr uint32_t kExtraRows = 256;                 // 64 chose 128 rows, 474 us for MX's 418
constexpr uint32_t kSlice = 256;                     // values of K: a row of 128 bytes
constexpr uint32_t kATile = kBM * 128;               // 16 KB
constexpr uint32_t kARaw = kBM * 16;                 // its scales, 16 bytes a row
constexpr uint32_t kRingBytes = 204 * 1024;          // six stages of 128 x 192 tiles
constexpr uint32_t kMaxStages = 9;
constexpr uint32_t kStageWarp = 16 * kLine;          // where a warp of the epilogue stages rows
constexpr uint32_t kSmemBytes = 1024 + kRingBytes + 8 * kStageWarp;
constexpr uint32_t kTmemCols = 512;

template <int FMT>
struct Scales {
  // 512-byte tiles of a slice: 4 scales of 128 rows, the K of one MMA (NV) or two (MX)
  static constexpr uint32_t kTiles = FMT == SYMM_FP4_MX ? 2 : 4;
  static constexpr uint32_t kPerSlice = kTiles * 4;      // scales of a row
  // most rows of a tile: TMEM holds two accumulators and the scales of four slices
  static constexpr uint32_t kMaxRows = FMT == SYMM_FP4_MX ? 192 : 160;
  static_assert(2 * kMaxRows + 4 * kTiles * 4 * 3 <= kTmemCols, "TMEM");
};

struct Fp4Args {
  const int32_t* counts;
  const float *gx, *gw;
  uint32_t n, E, m, k, npair;
  void* y;
  size_t ldy;
  int vec;  // rows of y are 16-byte aligned
  uint64_t budget_ns;
  Control* ctl;
};

struct Barriers {
  uint64_t full[kMaxStages], placed[kMaxStages], empty[kMaxStages];
  uint64_t tfull[2], tempty[2], sfree[kMaxStages], drain;
  uint32_t tmem;
};

// Descriptor of 32 lines of 16 bytes: no swizzle, 8 lines 128 bytes apart, version 1.
__device__ __forceinline__ uint64_t scales_desc(const void* tile) {
  return ((symm::smem_addr(tile) & 0x3FFFFull) >> 4) | ((128ull >> 4) << 32) | (1ull << 46);
}
// Such lines into 4 TMEM columns of all four quarters of the lanes.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}
template <int FMT>
__device__ __forceinline__ void scaled_mma(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc,
                                           uint32_t sa, uint32_t sb, uint32_t accumulate) {
  if (FMT == SYMM_FP4_MX)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, "
        "[%4], [%5], p;\n\t}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
}
// Instruction descriptor: e2m1 on both sides (1 at bits 7 and 10), N, the scales'
// type (bit 23: ue8m0), M, and which of a column's scales are meant (bits 4, 29).
template <int FMT>
__device__ __forceinline__ uint32_t fp4_idesc(uint32_t n, uint32_t which) {
  return (which << 4) | (1u << 7) | (1u << 10) | ((n >> 3) << 17) |
         ((uint32_t)(FMT == SYMM_FP4_MX) << 23) | ((2 * kBM >> 4) << 24) | (which << 29);
}

template <typename T>
struct Fmt {
  static constexpr int k = 0;
};
template <>
struct Fmt<__nv_bfloat16> {
  static constexpr int k = 1;
};

template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads, 1)
    fp4_kernel(const __grid_constant__ CUtensorMap map_w,
               const __grid_constant__ CUtensorMap map_ws,
               const __grid_constant__ CUtensorMap map_x64,
               const __grid_constant__ CUtensorMap map_x16,
               const __grid_constant__ CUtensorMap map_xs,
               const __grid_constant__ CUtensorMap map_xs32, const Fp4Args a) {
  using S = Scales<FMT>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (symm::smem_addr(smem_raw) & 1023u)) & 1023u);
  __shared__ Barriers bar;
  __shared__ Table table;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 64) {
    prefetch_map(&map_w), prefetch_map(&map_ws), prefetch_map(&map_x64), prefetch_map(&map_x16);
    prefetch_map(&map_xs), prefetch_map(&map_xs32);
  }
  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < kMaxStages; ++s) {
      symm::mbar_init(&bar.full[s], 1);
      symm::mbar_init(&bar.placed[s], 8);  // of the first CTA: by the four warps of either
      symm::mbar_init(&bar.empty[s], 1);
      symm::mbar_init(&bar.sfree[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      symm::mbar_init(&bar.tfull[i], 1);
      symm::mbar_init(&bar.tempty[i], 2 * kEpilogue / 32);  // both CTAs' warps
    }
    symm::mbar_init(&bar.drain, 1);
    symm::fence_mbar_init();
  }
  if (warp == 1) pair_tmem_alloc(&bar.tmem, kTmemCols);
  symm::tc_fence_before();
  __syncthreads();
  pair_arrive();  // whoever touches the other CTA's barriers waits first
  symm::tc_fence_after();
  moe::wait_for_earlier();
  const bool good =
      lay_out(table, a.counts, a.E, a.n, S::kMaxRows, kExtraRows, a.npair, gridDim.x / 2);
  if (!good && blockIdx.x == 0 && threadIdx.x == 0) symm::record_error(a.ctl, kErrRange, -1);
  pair_wait();
  const uint32_t tiles = good ? table.blocks[a.E] * a.npair : 0, tmem = uniform(bar.tmem);
  const uint32_t rank = pair_rank(), first = blockIdx.x / 2, step = gridDim.x / 2;
  const uint32_t slices = (a.k + kSlice - 1) / kSlice;
  // A stage: codes of A and B, and their scales: as loaded (A, B), then as TMEM takes them.
  const uint32_t most = uniform(good ? table.most / 2 : 16);
  const uint32_t raw = kATile + most * 128;  // where its scales are
  const uint32_t stage_bytes =
      raw + max(kARaw + (most <= 16 ? 32 : S::kMaxRows) * 16, S::kTiles * 512 * 3);
  // In TMEM two accumulators, then slots of a slice's scales: one for each stage, which
  // is free when the stage is, or as many as fit, each with a barrier of its own.
  const uint32_t acc_cols = 2 * most, row_blocks = acc_cols > 128 ? 2 : 1;
  const uint32_t scale_cols = S::kTiles * 4 * (1 + row_blocks);
  const uint32_t stages = min(kMaxStages, kRingBytes / stage_bytes);
  const uint32_t slots = min(stages, (kTmemCols - 2 * acc_cols) / scale_cols);

  if (warp == 0) {  // ----------------------------------------- TMA producer
    const bool elected = symm::elect_one();
    uint32_t st = 0, ph = 1, it = 0;
    bool ok = true;
    for (uint32_t i = first; ok && i < tiles; i += step) {
      const Tile t = tile_at(table, i, a.E, a.npair);
      const uint32_t half = t.bt / 2;
      const uint32_t col = 2 * t.col + rank, row = t.row + rank * half;
      const bool few = t.bt == 32;
      for (uint32_t s = 0; s < slices; ++s) {
        if (!(ok = wait_warp(&bar.empty[st], ph, a.budget_ns, a.ctl))) break;
        uint8_t* buf = smem + st * stage_bytes;
        uint64_t* full = &bar.full[st];
        if (elected) {
          symm::mbar_arrive_expect_tx(
              full, kATile + kARaw + half * 128 + (few ? 32 : S::kMaxRows) * 16);
          // 16 bytes of scales: this slice's, or with MX of this and its neighbour
          const int k = (int)(s * 128), b = (int)(s * S::kPerSlice / 16 * 16);
          symm::tma_load_3d(buf, &map_w, k, (int)(col * kBM), (int)t.e, full);
          symm::tma_load_3d(buf + raw, &map_ws, b, (int)(col * kBM), (int)t.e, full);
          // all the rows' scales, which both CTAs need, by one copy of what a tile has at
          // most (or of 32 rows)
          symm::tma_load_2d(buf + raw + kARaw, few ? &map_xs32 : &map_xs, b, (int)t.row, full);
          load_lines(buf + kATile, &map_x64, &map_x16, k, row, half, full);
        }
        ++it;
        if (++st == stages) st = 0, ph ^= 1;
      }
    }
    if (!ok && elected) symm::record_error(a.ctl, symm::kErrTimedOut, -3);
    drain_ring(bar.full, bar.empty, stages, it, ok, a.budget_ns);
  } else if (warp == 1 && rank == 0) {  // --------------------- MMA issuer
    const bool elected = symm::elect_one();
    uint32_t st = 0, ph = 0, seg = 0, slot = 0, sph = 1;
    bool ok = true;
    for (uint32_t i = first; ok && i < tiles; i += step, ++seg) {
      const Tile t = tile_at(table, i, a.E, a.npair);
      const uint32_t buf = seg & 1;
      if (!(ok = wait_warp(&bar.tempty[buf], ((seg >> 1) & 1) ^ 1u, a.budget_ns, a.ctl)))
        break;
      symm::tc_fence_after();
      const uint32_t acc = tmem + buf * acc_cols;
      const uint32_t bt = uniform(t.bt);
      const uint32_t idesc = fp4_idesc<FMT>(bt, 0), idesc_odd = fp4_idesc<FMT>(bt, 2);
      for (uint32_t s = 0; s < slices; ++s) {
        const uint32_t sa = tmem + 2 * acc_cols + slot * scale_cols;
        const uint32_t sb = sa + S::kTiles * 4;
        // whoever placed the scales, here and in the other CTA, has seen the copies land
        ok = wait_warp(&bar.placed[st], ph, a.budget_ns, a.ctl) &&
             (slots == stages ||
              wait_warp(&bar.sfree[slot], sph, a.budget_ns, a.ctl));
        if (!ok) break;
        symm::tc_fence_after();
        const uint8_t* at = smem + st * stage_bytes;
        const uint64_t wd = symm::sw128_kmajor_desc(at);
        const uint64_t xd = symm::sw128_kmajor_desc(at + kATile);
        if (elected) {
          // A's tiles in K order; B's row blocks, one or two, side by side in K order
          const uint64_t sd = scales_desc(at + raw);
#pragma unroll
          for (uint32_t c = 0; c < S::kTiles; ++c) copy_scales(sa + 4 * c, sd + 32 * c);
          if (row_blocks == 1) {
#pragma unroll
            for (uint32_t c = 0; c < S::kTiles; ++c)
              copy_scales(sb + 4 * c, sd + 32 * (S::kTiles + 2 * c));
          } else {
#pragma unroll
            for (uint32_t c = 0; c < 2 * S::kTiles; ++c)
              copy_scales(sb + 4 * c, sd + 32 * (S::kTiles + c));
          }
#pragma unroll
          for (uint32_t j = 0; j < 4; ++j) {
            const uint32_t c = j * S::kTiles / 4;
            scaled_mma<FMT>(acc, wd + 2 * j, xd + 2 * j,
                            FMT == SYMM_FP4_MX && (j & 1) ? idesc_odd : idesc, sa + 4 * c,
                            sb + 4 * row_blocks * c, (s | j) != 0);
          }
          if (slots != stages) pair_commit_own(&bar.sfree[slot]);
          pair_commit(&bar.empty[st]);
        }
        if (++st == stages) st = 0, ph ^= 1;
        if (++slot == slots) slot = 0, sph ^= 1;
      }
      if (ok && elected) pair_commit(&bar.tfull[buf]);
    }
    if (!ok && elected) symm::record_error(a.ctl, symm::kErrTimedOut, -5);
    if (elected) pair_commit(&bar.drain);
  } else if (warp >= 2 && warp < 10) {  // ---------------------- epilogue
    // Two warps to each 32 TMEM lanes, which take turns at the chunks of rows.
    const uint32_t q = (uint32_t)(warp & 3), turn = (uint32_t)(warp - 2) / 4;
    uint8_t* mine = smem + kRingBytes + (warp - 2) * kStageWarp;
    const float gx = a.gx ? *a.gx : 1.f;
    uint32_t seg = 0;
    for (uint32_t i = first; i < tiles; i += step, ++seg) {
      const Tile t = tile_at(table, i, a.E, a.npair);
      const uint32_t buf = seg & 1, f = (2 * t.col + rank) * kBM + 32 * q;
      const uint32_t width = f < a.m ? a.m - f : 0;  // features from f on that are there
      const float scale = a.gw ? gx * a.gw[t.e] : gx;
      const bool ok = wait_warp(&bar.tfull[buf], (seg >> 1) & 1, a.budget_ns, a.ctl);
      if (any_of(!ok, kEpilogue)) {  // all threads leave, or none
        if (threadIdx.x == 64) symm::record_error(a.ctl, symm::kErrTimedOut, -6);
        break;
      }
      symm::tc_fence_after();
      const uint32_t taddr = tmem + ((32 * q) << 16) + buf * acc_cols;
      for (uint32_t c = 16 * turn; c < t.rows; c += 32) {
        uint32_t v[2][8], p[2][4];
        tmem_frags(taddr + c, v);
#pragma unroll
        for (uint32_t x = 0; x < 2; ++x)
#pragma unroll
          for (uint32_t o = 0; o < 4; ++o)
            p[x][o] = symm::pack2<Fmt<T>::k>(
                __uint_as_float(v[o / 2][4 * x + 2 * (o % 2)]) * scale,
                __uint_as_float(v[o / 2][4 * x + 2 * (o % 2) + 1]) * scale);
        stage_rows(mine, p);
        __syncwarp();
        store_rows(mine, static_cast<T*>(a.y) + (size_t)(t.row + c) * a.ldy + f, a.ldy,
                   t.rows - c, width, a.vec);
        __syncwarp();
      }
      symm::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_first(&bar.tempty[buf]);  // the accumulator is free again
    }
  } else if (warp >= 10) {  // ------------------------------ scales' order
    // Lane l of warp w takes row 32 (l % 4) + 8 w + l / 4 of a block of 128: its
    // words are neighbours of the other lanes' in the tile.
    const uint32_t w = (uint32_t)warp - 10, r = 32 * (lane % 4) + 8 * w + lane / 4;
    uint32_t st = 0, ph = 0;
    bool ok = true;
    for (uint32_t i = first; ok && i < tiles; i += step) {
      const Tile t = tile_at(table, i, a.E, a.npair);
      const uint32_t rows = t.bt;
      for (uint32_t s = 0; s < slices; ++s) {
        ok = wait_warp(&bar.full[st], ph, a.budget_ns, a.ctl);
        uint8_t* at = smem + st * stage_bytes;
        const uint4* from = reinterpret_cast<const uint4*>(at + raw);
        uint32_t* to = reinterpret_cast<uint32_t*>(at + raw);
        const uint32_t word = 4 * (8 * w + lane / 4) + lane % 4;
        const bool odd = FMT == SYMM_FP4_MX && (s & 1);  // the second 8 bytes
        uint4 v[3];  // of A's row, of B's first 128, of B's others
        v[0] = from[r];
#pragma unroll
        for (uint32_t b = 1; b < 3; ++b)
          if (128 * b - 128 + r < rows) v[b] = from[128 * b + r];
        // all four warps have read: the same bytes take the tiles.  One that gave up takes
        // the others with it.
        if (any_of(!ok, 128, 2)) {
          ok = false;
          break;
        }
#pragma unroll
        for (uint32_t b = 0; b < 3; ++b) {
          if (b && 128 * b - 128 + r >= rows) continue;
          const uint32_t x[4] = {odd ? v[b].z : v[b].x, odd ? v[b].w : v[b].y, v[b].z, v[b].w};
#pragma unroll
          for (uint32_t c = 0; c < S::kTiles; ++c)
            to[128 * (b ? S::kTiles + 2 * c + b - 1 : c) + word] = x[c];
        }
        symm::fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) arrive_first(&bar.placed[st]);
        if (++st == stages) st = 0, ph ^= 1;
      }
    }
    if (!ok && lane == 0) symm::record_error(a.ctl, symm::kErrTimedOut, -7);
  }
  leave_pair(&bar.drain, tmem, kTmemCols, a.budget_ns);
}

// ------------------------------------------------------------------- host --
int check_rows(const char* what, int fmt, int n, int k) {
  if (fmt != SYMM_FP4_MX && fmt != SYMM_FP4_NV)
    return fail(SYMM_EINVAL, std::string(what) + ": fmt must be SYMM_FP4_MX or _NV");
  if (n < 0 || n > (1 << 24) || k < 32 || k % 32 || k > (1 << 17))
    return fail(SYMM_EINVAL, std::string(what) + ": n must be in [0, 2^24], k a multiple of 32 in "
                                                 "[32, 2^17]");
  return SYMM_OK;
}
size_t scale_bytes(int fmt, int k) { return (size_t)k / (fmt == SYMM_FP4_MX ? 32 : 16); }
bool bad_packed(size_t ldc, size_t lds, int fmt, int k) {
  return ldc < (size_t)k / 2 || ldc % 16 || ldc > (1ull << 36) || lds < scale_bytes(fmt, k) ||
         lds % 16 || lds > (1ull << 36);
}

unsigned quant_grid(uint32_t n, uint32_t kv) {
  // as many blocks as are resident at once at most, 2048 threads an SM
  const uint64_t vectors = (uint64_t)n * kv;
  const uint64_t room = (uint64_t)std::max(sm_count(), 1) * (2048 / kQuantThreads);
  return (unsigned)std::min<uint64_t>(room, (vectors + kQuantThreads - 1) / kQuantThreads);
}

// Bytes [depth][rows][inner], rows ld and planes rows * ld apart; boxes of box_inner
// x box_rows; depth 0: a 2-d map.
int make_map(const char* what, CUtensorMap* map, const void* base, uint64_t inner, uint64_t rows,
             uint64_t depth, size_t ld, uint32_t box_inner, uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return fail(SYMM_ECUDA, std::string(what) + ": no cuTensorMapEncodeTiled");
  const cuuint64_t dims[3] = {inner, rows, depth};
  const cuuint64_t strides[2] = {(cuuint64_t)ld, (cuuint64_t)ld * rows};
  const cuuint32_t box[3] = {box_inner, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r =
      fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, depth ? 3 : 2, const_cast<void*>(base), dims, strides,
         box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
         box_inner == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(SYMM_ECUDA,
                std::string(what) + ": tensor map rejected (CUresult " + std::to_string(r) + ")");
  return SYMM_OK;
}

struct Maps {
  CUtensorMap w, ws, x64, x16, xs, xs32;
};

template <typename T, int FMT>
int launch_product(const Maps& m, const Fp4Args& a, cudaStream_t s) {
  static std::mutex mu;
  static unsigned known[64] = {};  // CTA pairs that are resident at once
  int dev = 0;
  int rc = cuda_check(cudaGetDevice(&dev), "moe_fp4_expert_matmul: device");
  if (rc) return rc;
  unsigned pairs = 0;
  {
    std::lock_guard<std::mutex> lock(mu);
    const bool keep = dev >= 0 && dev < 64;
    if (keep) pairs = known[dev];
    if (!pairs) {
      const void* kernel = (const void*)fp4_kernel<T, FMT>;
      rc = cuda_check(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)kSmemBytes),
                      "moe_fp4_expert_matmul: kernel set-up");
      if (rc) return rc;
      pairs = resident_pairs(kernel, kThreads, kSmemBytes);
      if (keep) known[dev] = pairs;
    }
  }
  // at most one partly filled block of rows, 64 at the least, for each expert that has rows
  const uint64_t most = (uint64_t)a.npair * std::min<uint64_t>(a.n, a.n / 64 + a.E);
  return launch_pairs("moe_fp4_expert_matmul", fp4_kernel<T, FMT>,
                      (unsigned)std::min<uint64_t>(pairs, most), kThreads, kSmemBytes, s, m.w,
                      m.ws, m.x64, m.x16, m.xs, m.xs32, a);
}

template <typename T, int FMT>
int launch_quantize(const QuantArgs& a, int act, cudaStream_t s) {
  auto* kernel = act == SYMM_ACT_NONE   ? quantize_kernel<T, FMT, SYMM_ACT_NONE>
                 : act == SYMM_ACT_SILU ? quantize_kernel<T, FMT, SYMM_ACT_SILU>
                                        : quantize_kernel<T, FMT, SYMM_ACT_GELU>;
  return moe::launch("moe_fp4_quantize", kernel, quant_grid(a.n, a.kv), kQuantThreads, 0, s, a);
}
template <typename T>
int launch_quantize(int fmt, int act, const QuantArgs& a, cudaStream_t s) {
  return fmt == SYMM_FP4_MX ? launch_quantize<T, SYMM_FP4_MX>(a, act, s)
                            : launch_quantize<T, SYMM_FP4_NV>(a, act, s);
}
template <typename T>
int launch_dequantize(int fmt, const DequantArgs& a, cudaStream_t s) {
  return moe::launch("moe_fp4_dequantize",
                     fmt == SYMM_FP4_MX ? dequantize_kernel<T, SYMM_FP4_MX>
                                        : dequantize_kernel<T, SYMM_FP4_NV>,
                     quant_grid(a.n, a.kv), kQuantThreads, 0, s, a);
}

}  // namespace

extern "C" int moe_fp4_quantize(const void* x, size_t ldx, int act, int dtype, int fmt,
                                const float* gscale, int n, int k, void* codes, size_t ldc,
                                void* scales, size_t lds, void* stream) {
  return moe::entry("moe_fp4_quantize", [&]() -> int {
    const char* what = "moe_fp4_quantize";
    int rc = check_rows(what, fmt, n, k);
    if (rc) return rc;
    if (!moe::dtype_ok(dtype))
      return fail(SYMM_EINVAL, "moe_fp4_quantize: dtype must be SYMM_DTYPE_F16, _BF16 or _F32");
    if (act != SYMM_ACT_NONE && act != SYMM_ACT_SILU && act != SYMM_ACT_GELU)
      return fail(SYMM_EINVAL, "moe_fp4_quantize: act must be SYMM_ACT_NONE, _SILU or _GELU");
    const size_t width = act == SYMM_ACT_NONE ? (size_t)k : 2 * (size_t)k;
    if (ldx < width || ldx % 8 || ldx > (1ull << 36) || bad_packed(ldc, lds, fmt, k))
      return fail(SYMM_EINVAL, "moe_fp4_quantize: ldx must hold a row (k, or 2k with an "
                               "activation) in whole eights, ldc k / 2 bytes and lds a row's "
                               "scales in whole sixteens");
    if (n == 0) return SYMM_OK;
    if (!x || !codes || !scales)
      return fail(SYMM_EINVAL, "moe_fp4_quantize: NULL x, codes or scales");
    if (!moe::aligned(x, 16) || !moe::aligned(codes, 16) || !moe::aligned(scales, 16) ||
        !moe::aligned(gscale, 4))
      return fail(SYMM_EINVAL, "moe_fp4_quantize: x, codes and scales must be 16-byte aligned, "
                               "gscale 4-byte");
    if (fmt == SYMM_FP4_MX && gscale)
      return fail(SYMM_EINVAL, "moe_fp4_quantize: gscale must be NULL with SYMM_FP4_MX");
    if (codes == x || scales == x || codes == scales)
      return fail(SYMM_EINVAL, "moe_fp4_quantize: outputs must not be inputs or each other");
    QuantArgs a{};
    a.x = x, a.ldx = ldx, a.codes = static_cast<uint8_t*>(codes);
    a.scales = static_cast<uint8_t*>(scales), a.ldc = ldc, a.lds = lds, a.g = gscale;
    a.n = (uint32_t)n, a.k = (uint32_t)k, a.kv = (uint32_t)k / 8;
    cudaStream_t s = as_stream(stream);
    return dtype == SYMM_DTYPE_F32    ? launch_quantize<float>(fmt, act, a, s)
           : dtype == SYMM_DTYPE_BF16 ? launch_quantize<__nv_bfloat16>(fmt, act, a, s)
                                      : launch_quantize<__half>(fmt, act, a, s);
  });
}

extern "C" int moe_fp4_dequantize(const void* codes, size_t ldc, const void* scales, size_t lds,
                                  int fmt, const float* gscale, int n, int k, int dtype, void* y,
                                  size_t ldy, void* stream) {
  return moe::entry("moe_fp4_dequantize", [&]() -> int {
    const char* what = "moe_fp4_dequantize";
    int rc = check_rows(what, fmt, n, k);
    if (rc) return rc;
    if (!moe::dtype_ok(dtype))
      return fail(SYMM_EINVAL, "moe_fp4_dequantize: dtype must be SYMM_DTYPE_F16, _BF16 or _F32");
    if (ldy < (size_t)k || ldy % 8 || ldy > (1ull << 36) || bad_packed(ldc, lds, fmt, k))
      return fail(SYMM_EINVAL, "moe_fp4_dequantize: ldy >= k in whole eights, ldc k / 2 bytes and "
                               "lds a row's scales in whole sixteens");
    if (n == 0) return SYMM_OK;
    if (!codes || !scales || !y)
      return fail(SYMM_EINVAL, "moe_fp4_dequantize: NULL codes, scales or y");
    if (!moe::aligned(codes, 16) || !moe::aligned(scales, 16) || !moe::aligned(y, 16) ||
        !moe::aligned(gscale, 4))
      return fail(SYMM_EINVAL, "moe_fp4_dequantize: codes, scales and y must be 16-byte aligned, "
                               "gscale 4-byte");
    if (y == codes || y == scales)
      return fail(SYMM_EINVAL, "moe_fp4_dequantize: y must not be an input");
    DequantArgs a{};
    a.codes = static_cast<const uint8_t*>(codes), a.scales = static_cast<const uint8_t*>(scales);
    a.ldc = ldc, a.lds = lds, a.g = gscale, a.y = y, a.ldy = ldy;
    a.n = (uint32_t)n, a.kv = (uint32_t)k / 8;
    cudaStream_t s = as_stream(stream);
    return dtype == SYMM_DTYPE_F32    ? launch_dequantize<float>(fmt, a, s)
           : dtype == SYMM_DTYPE_BF16 ? launch_dequantize<__nv_bfloat16>(fmt, a, s)
                                      : launch_dequantize<__half>(fmt, a, s);
  });
}

extern "C" int moe_fp4_expert_matmul(symm_heap_t* heap, const void* xc, size_t ldxc,
                                     const void* xs, size_t ldxs, const void* wc, size_t ldwc,
                                     const void* ws, size_t ldws, const int32_t* counts,
                                     const float* gx, const float* gw, int fmt, int dtype, int n,
                                     int E, int k, int m, void* y, size_t ldy, void* stream) {
  return moe::entry("moe_fp4_expert_matmul", [&]() -> int {
    const char* what = "moe_fp4_expert_matmul";
    if (!heap) return fail(SYMM_EINVAL, "moe_fp4_expert_matmul: NULL heap");
    int rc = check_rows(what, fmt, n, k);
    if (rc) return rc;
    if (dtype != SYMM_DTYPE_F16 && dtype != SYMM_DTYPE_BF16)
      return fail(SYMM_EINVAL, "moe_fp4_expert_matmul: dtype must be SYMM_DTYPE_F16 or _BF16");
    if (E < 1 || E > SYMM_MOE_MAX_EXPERTS || m < 1 || m > (1 << 20))
      return fail(SYMM_EINVAL, "moe_fp4_expert_matmul: E must be in [1, 1024], m in [1, 2^20]");
    if (bad_packed(ldxc, ldxs, fmt, k) || bad_packed(ldwc, ldws, fmt, k) || ldy < (size_t)m ||
        ldy > (1ull << 36))
      return fail(SYMM_EINVAL, "moe_fp4_expert_matmul: ldxc and ldwc must hold k / 2 bytes, ldxs "
                               "and ldws a row's scales, in whole sixteens; ldy >= m");
    if (!counts && E != 1)
      return fail(SYMM_EINVAL, "moe_fp4_expert_matmul: counts may be NULL with one expert only");
    if (n == 0) return SYMM_OK;
    if (!xc || !xs || !wc || !ws || !y)
      return fail(SYMM_EINVAL, "moe_fp4_expert_matmul: NULL codes, scales or y");
    if (!moe::aligned(xc, 16) || !moe::aligned(xs, 16) || !moe::aligned(wc, 16) ||
        !moe::aligned(ws, 16) || !moe::aligned(y, 2) || !moe::aligned(counts, 4) ||
        !moe::aligned(gx, 4) || !moe::aligned(gw, 4))
      return fail(SYMM_EINVAL, "moe_fp4_expert_matmul: codes and scales must be 16-byte aligned, "
                               "the rest to their elements");
    if (y == xc || y == xs || y == wc || y == ws)
      return fail(SYMM_EINVAL, "moe_fp4_expert_matmul: y must not be an input");
    const size_t sb = scale_bytes(fmt, k);
    Maps mp{};
    rc = make_map(what, &mp.w, wc, k / 2, m, E, ldwc, 128, kBM);
    if (!rc) rc = make_map(what, &mp.ws, ws, sb, m, E, ldws, 16, kBM);
    if (!rc) rc = make_map(what, &mp.x64, xc, k / 2, n, 0, ldxc, 128, 64);
    if (!rc) rc = make_map(what, &mp.x16, xc, k / 2, n, 0, ldxc, 128, 16);
    if (!rc)
      rc = make_map(what, &mp.xs, xs, sb, n, 0, ldxs, 16,
                    fmt == SYMM_FP4_MX ? Scales<SYMM_FP4_MX>::kMaxRows
                                       : Scales<SYMM_FP4_NV>::kMaxRows);
    if (!rc) rc = make_map(what, &mp.xs32, xs, sb, n, 0, ldxs, 16, 32);
    if (rc) return rc;
    cudaStream_t s = as_stream(stream);
    rc = ensure_ctrl(heap, s);
    if (rc) return rc;
    Fp4Args a{};
    a.counts = counts, a.gx = gx, a.gw = gw, a.n = (uint32_t)n, a.E = (uint32_t)E;
    a.m = (uint32_t)m, a.k = (uint32_t)k, a.npair = ((uint32_t)m + 2 * kBM - 1) / (2 * kBM);
    a.y = y, a.ldy = ldy, a.vec = ldy % 8 == 0 && moe::aligned(y, 16);
    a.budget_ns = heap->spin_budget;
    a.ctl = reinterpret_cast<Control*>(heap->base);
    const bool bf = dtype == SYMM_DTYPE_BF16;
    if (fmt == SYMM_FP4_MX)
      return bf ? launch_product<__nv_bfloat16, SYMM_FP4_MX>(mp, a, s)
                : launch_product<__half, SYMM_FP4_MX>(mp, a, s);
    return bf ? launch_product<__nv_bfloat16, SYMM_FP4_NV>(mp, a, s)
              : launch_product<__half, SYMM_FP4_NV>(mp, a, s);
  });
}
