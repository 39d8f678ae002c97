// moe_expert.cu -- the experts' gated feed-forward and its gradients on rows
// grouped by expert: y = (act(x Wg_e) * (x Wu_e)) Wd_e for the rows of expert e.
//
// With gu = x Wgu_e (its first F columns g, the others u), h = act(g) u:
//   forward    gu, h  (one launch: both projections, the activation, the product)
//              y = h Wd_e
//   backward   dh = dy Wd_e^T;  dg = dh u act'(g), du = dh act(g), and h again,
//              in that launch's epilogue;
//              dx = [dg | du] Wgu_e^T;  dWd_e = h_e^T dy_e;  dWgu_e = x_e^T [dg | du]_e
// h and [dg | du] are rounded to the inputs' type between launches: they are
// operands of 16-bit tensor-core products, and one rounding (bf16: 2^-8 at most) is what
// the outputs have anyway.  All sums are in 32 bits, in TMEM.
//
// rows_kernel: a product of an expert's rows with its weights, computed as
// y^T = W^T x^T by CTA pairs (cta_group::2): the M side of a tile is 256 features,
// 128 of either CTA (the weights as they are stored, M-major or K-major), the N side
// 32 to 256 of the expert's rows, half of them in either CTA's shared memory, cut as
// evenly as steps of 32 allow.  An expert with few rows then costs no more than their
// loads and MMAs.  How many rows each expert has is read on the device; every CTA lays
// out the same table of tiles, and a pair takes every (gridDim / 2)-th.
//   warp 0     TMA producer: 64-deep slices of K of both sides, 128-byte
//              swizzled, into a ring of stages; 128 deep when no tile has more
//              than 64 rows (a slice costs each role some 250 cycles beside its MMAs)
//   warp 1     MMA issuer (first CTA): tcgen05.mma kind::f16, two accumulators in
//              TMEM; in the second CTA it tells the first what has landed
//   warps 2-9  epilogue: fragments from TMEM, activation or gradient, rounding,
//              stmatrix into rows of 32 features, 16-byte stores
// The gated product's tile is 64 columns of Wg over the same 64 of Wu in either CTA: g
// and u of an element are then 64 TMEM lanes apart, in two warps, which exchange halves
// of them through shared memory, each finishing half of the rows.
//
// grad_kernel: the gradients of the weights, dW_e = a_e^T b_e: 256 x 256 tiles, K the
// expert's rows, both operands as stored (M- and N-major).  Rows of the next
// expert that share the last 16-row step are zeroed in shared memory, in both
// operands, before its MMAs: what they hold may be an infinity.  Both gradients are one
// launch.
//
// Measured (bf16).  Forward, 8 experts of 7168 x 2048, 1024 rows each: 388 us, 1.86
// PFLOP/s, 98 % of cuBLAS's burst rate (single CTAs: 465; their 4-warp epilogue with 2-byte
// stores: 40 us of the pairs' 432).  32 experts of 900 to 1500 rows for a second: 1992 us,
// 1.45 PFLOP/s, under the power cap (cuBLAS: 1.68; GELU: 2022 us).  64 rows on 32 experts: 319
// to 345 us, the weights at the copy rate.  Backward, 32 experts of 4096 x 2048, 512 rows
// each: dh 194 us, dx 314, the weights' gradients 515 (1.54 PFLOP/s in all).  1225 rows on 4
// experts of 1000 x 328: 19.4 us with blocks of 64 rows, 26.3 with 160.
#include <algorithm>
#include <string>

#include "moe_experts.cuh"

using namespace experts;
using namespace symm_host;

namespace {

constexpr uint32_t kThreads = 320, kEpilogue = 256;
constexpr uint32_t kMaxRows = 256;                       // rows of a tile: the N side of a pair
constexpr uint32_t kExtraRows = 64;                      // 1225 rows: 19.4 us so, 26.3 with one cap
constexpr uint32_t kBK = 64;
constexpr uint32_t kATile = kBM * kBK * 2;               // 16 KB
constexpr uint32_t kRingBytes = 192 * 1024;              // six stages of 128 features, 128 rows
constexpr uint32_t kMaxStages = 8;
constexpr uint32_t kStageWarp = 32 * kLine;              // where a warp of the epilogue stages rows
constexpr uint32_t kGradBox = 16 * 128;                  // where it stages 16 rows of a gradient
constexpr uint32_t kSmemBytes = 1024 + kRingBytes + 8 * kStageWarp;
static_assert(kGradBox <= kStageWarp, "both stagings in one size");
constexpr uint32_t kAccCols = 256;

enum Kind { kGated, kDown, kDh, kDx };

struct ExpertArgs {
  const int32_t* counts;
  uint32_t n, E;
  uint32_t m, k;       // features out (kGated: F), contraction
  uint32_t npair;      // pairs of column blocks
  uint32_t F;          // offset of u in gu
  int act;
  const void* gu_in;   // kDh
  void *gu, *h, *out;  // kGated: gu (NULL allowed), h; kDh: gu is [dg | du], h; else out
  size_t ldo;
  uint64_t budget_ns;
  Control* ctl;
};

// Instruction descriptor: fp32 accumulator, both operands of one type; bits 15
// and 16: the M and the N side are M- and N-major.
__device__ __forceinline__ uint32_t mma_idesc(uint32_t fmt, uint32_t n, bool m_major,
                                              bool n_major) {
  return (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)m_major << 15) |
         ((uint32_t)n_major << 16) | ((n >> 3) << 17) | ((2 * kBM >> 4) << 24);
}
constexpr uint64_t kMajorStep = (16 * 128) >> 4;  // 16 K rows of an M- or N-major tile
constexpr uint64_t kKStep = 32 >> 4;              // 16 K columns of a K-major tile

template <int FMT>
struct Elem {
  using T = __half;
};
template <>
struct Elem<1> {
  using T = __nv_bfloat16;
};

// The ring of a launch in which a CTA copies at most `rows` rows of a tile.
struct Ring {
  uint32_t deep, stages, stage_bytes;
};
__device__ __forceinline__ Ring ring_of(uint32_t rows) {
  Ring r;
  r.deep = rows <= 32 ? 2 : 1;
  r.stage_bytes = r.deep * (kATile + rows * 128);
  r.stages = min(kMaxStages, kRingBytes / r.stage_bytes);
  return r;
}

struct Barriers {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t tfull[2], tempty[2], drain;
  uint32_t tmem;
};
// Barriers and TMEM.
__device__ __forceinline__ void set_up_cta(Barriers& b, int warp) {
  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < kMaxStages; ++s) {
      // the first CTA's: its own copies, and the second one's word that its are there
      symm::mbar_init(&b.full[s], pair_rank() ? 1 : 2);
      symm::mbar_init(&b.empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      symm::mbar_init(&b.tfull[i], 1);
      symm::mbar_init(&b.tempty[i], 2 * kEpilogue / 32);  // both CTAs' warps
    }
    symm::mbar_init(&b.drain, 1);
    symm::fence_mbar_init();
  }
  if (warp == 1) pair_tmem_alloc(&b.tmem, 2 * kAccCols);
  symm::tc_fence_before();
  __syncthreads();
  pair_arrive();  // whoever touches the other CTA's barriers waits first
  symm::tc_fence_after();
}

// ------------------------------------------------------------- epilogues --
// Fragments of 16 rows (columns of TMEM) and this warp's 32 features, as
// tmem_frags leaves them, packed in pairs of neighbouring rows.
template <int FMT>
__device__ __forceinline__ void pack_frags(const uint32_t (&v)[2][8], uint32_t (&p)[2][4]) {
#pragma unroll
  for (uint32_t t = 0; t < 2; ++t)
#pragma unroll
    for (uint32_t o = 0; o < 4; ++o)
      p[t][o] = symm::pack2<FMT>(__uint_as_float(v[o / 2][4 * t + 2 * (o % 2)]),
                                 __uint_as_float(v[o / 2][4 * t + 2 * (o % 2) + 1]));
}
// 16 rows of 32 features through `stage` to global memory.
template <int FMT>
__device__ __forceinline__ void put_rows(uint8_t* stage, const uint32_t (&p)[2][4], void* to,
                                         size_t ld, uint32_t row, uint32_t f, uint32_t valid,
                                         uint32_t width) {
  using T = typename Elem<FMT>::T;
  stage_rows(stage, p);
  __syncwarp();
  store_rows(stage, static_cast<T*>(to) + (size_t)row * ld + f, ld, valid, width, true);
  __syncwarp();
}
// Two packed values of 16 bits.
template <int FMT>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if (FMT == 1) return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
// What a lane stages of 16 rows: two vectors of 8 features; zeros where there are none.
__device__ __forceinline__ void fetch_rows(uint4 (&v)[2], const void* from, size_t ld, uint32_t row,
                                           uint32_t f, uint32_t valid, uint32_t width) {
  const uint32_t lane = threadIdx.x & 31, c = 8 * (lane & 3);
#pragma unroll
  for (uint32_t i = 0; i < 2; ++i) {
    const uint32_t r = 8 * i + lane / 4;
    v[i] = make_uint4(0, 0, 0, 0);
    if (r < valid && c < width)
      v[i] = symm::ld16_ro(static_cast<const uint16_t*>(from) + (size_t)(row + r) * ld + f + c);
  }
}
__device__ __forceinline__ void drop_rows(uint8_t* stage, const uint4 (&v)[2]) {
  const uint32_t lane = threadIdx.x & 31;
#pragma unroll
  for (uint32_t i = 0; i < 2; ++i)
    *reinterpret_cast<uint4*>(stage + (8 * i + lane / 4) * kLine + (lane & 3) * 16) = v[i];
}

// ------------------------------------------------------------ rows_kernel --
template <int FMT, int KIND>
__global__ void __launch_bounds__(kThreads, 1)
    rows_kernel(const __grid_constant__ CUtensorMap map_w,
                const __grid_constant__ CUtensorMap map_x64,
                const __grid_constant__ CUtensorMap map_x16, const ExpertArgs a) {
  constexpr bool kMMajor = KIND == kGated || KIND == kDown;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (symm::smem_addr(smem_raw) & 1023u)) & 1023u);
  __shared__ Barriers bar;
  __shared__ Table table;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 32) prefetch_map(&map_w), prefetch_map(&map_x64), prefetch_map(&map_x16);
  set_up_cta(bar, warp);
  moe::wait_for_earlier();
  const bool good =
      lay_out(table, a.counts, a.E, a.n, kMaxRows, kExtraRows, a.npair, gridDim.x / 2);
  if (!good && blockIdx.x == 0 && threadIdx.x == 0) symm::record_error(a.ctl, kErrRange, -1);
  pair_wait();
  const uint32_t tiles = good ? table.blocks[a.E] * a.npair : 0;
  const Ring ring = ring_of(uniform(good ? table.most / 2 : 16));
  const uint32_t slices = (a.k + ring.deep * kBK - 1) / (ring.deep * kBK);
  const uint32_t tmem = uniform(bar.tmem), abytes = ring.deep * kATile;
  const uint32_t rank = pair_rank(), first = blockIdx.x / 2, step = gridDim.x / 2;

  if (warp == 0) {  // ----------------------------------------- TMA producer
    const bool elected = symm::elect_one();
    uint32_t st = 0, ph = 1, it = 0;
    bool ok = true;
    for (uint32_t i = first; ok && i < tiles; i += step) {
      const Tile t = tile_at(table, i, a.E, a.npair);
      const uint32_t half = t.bt / 2, xbytes = half * 128;
      const uint32_t col = 2 * t.col + rank, row = t.row + rank * half;
      for (uint32_t s = 0; s < slices; ++s) {
        if (!(ok = wait_warp(&bar.empty[st], ph, a.budget_ns, a.ctl))) break;
        uint8_t* buf = smem + st * ring.stage_bytes;
        uint64_t* full = &bar.full[st];
        if (elected) {
          symm::mbar_arrive_expect_tx(full, abytes + ring.deep * xbytes);
          for (uint32_t d = 0; d < ring.deep; ++d) {
            const int k = (int)((s * ring.deep + d) * kBK);
            if (kMMajor) {
              const int x = KIND == kGated ? (int)(col * 64) : (int)(col * kBM);
              const int x2 = KIND == kGated ? x + (int)a.F : x + 64;
              symm::tma_load_3d(buf + d * (kATile / 2), &map_w, x, k, (int)t.e, full);
              symm::tma_load_3d(buf + abytes / 2 + d * (kATile / 2), &map_w, x2, k, (int)t.e, full);
            } else {
              symm::tma_load_3d(buf + d * kATile, &map_w, k, (int)(col * kBM), (int)t.e, full);
            }
            load_lines(buf + abytes + d * xbytes, &map_x64, &map_x16, k, row, half, full);
          }
        }
        ++it;
        if (++st == ring.stages) st = 0, ph ^= 1;
      }
    }
    if (!ok && elected) symm::record_error(a.ctl, symm::kErrTimedOut, -3);
    drain_ring(bar.full, bar.empty, ring.stages, it, ok, a.budget_ns);
  } else if (warp == 1 && rank) {  // -------- tells the first CTA what is here
    const bool elected = symm::elect_one();
    uint32_t st = 0, ph = 0;
    bool ok = true;
    for (uint32_t i = first; ok && i < tiles; i += step)
      for (uint32_t s = 0; s < slices; ++s) {
        if (!(ok = wait_warp(&bar.full[st], ph, a.budget_ns, a.ctl))) break;
        if (elected) arrive_first(&bar.full[st]);
        if (++st == ring.stages) st = 0, ph ^= 1;
      }
    if (!ok && elected) symm::record_error(a.ctl, symm::kErrTimedOut, -4);
  } else if (warp == 1) {  // ---------------------------------- MMA issuer
    const bool elected = symm::elect_one();
    uint32_t st = 0, ph = 0, seg = 0;
    bool ok = true;
    for (uint32_t i = first; ok && i < tiles; i += step, ++seg) {
      const Tile t = tile_at(table, i, a.E, a.npair);
      const uint32_t bt = uniform(t.bt), xbytes = bt / 2 * 128, buf = seg & 1;
      const uint32_t idesc = mma_idesc(FMT, bt, kMMajor, false);
      if (!(ok = wait_warp(&bar.tempty[buf], ((seg >> 1) & 1) ^ 1u, a.budget_ns, a.ctl)))
        break;
      symm::tc_fence_after();
      const uint32_t acc = tmem + buf * kAccCols;
      for (uint32_t s = 0; s < slices; ++s) {
        if (!(ok = wait_warp(&bar.full[st], ph, a.budget_ns, a.ctl))) break;
        symm::tc_fence_after();
        const uint8_t* at = smem + st * ring.stage_bytes;
        if (elected) {
          for (uint32_t d = 0; d < ring.deep; ++d) {
            const uint64_t wd = kMMajor
                                    ? symm::sw128_mnmajor_desc(at + d * (kATile / 2), abytes / 2)
                                    : symm::sw128_kmajor_desc(at + d * kATile);
            const uint64_t xd = symm::sw128_kmajor_desc(at + abytes + d * xbytes);
#pragma unroll
            for (uint32_t j = 0; j < kBK / 16; ++j)
              pair_mma(acc, wd + (kMMajor ? kMajorStep : kKStep) * j, xd + kKStep * j, idesc,
                       (s | d | j) != 0);
          }
          pair_commit(&bar.empty[st]);
        }
        if (++st == ring.stages) st = 0, ph ^= 1;
      }
      if (ok && elected) pair_commit(&bar.tfull[buf]);
    }
    if (!ok && elected) symm::record_error(a.ctl, symm::kErrTimedOut, -5);
    if (elected) pair_commit(&bar.drain);
  } else {  // -------------------------------------------------- epilogue
    // Two warps to each 32 TMEM lanes, which take turns at the chunks of rows.
    const uint32_t q = (uint32_t)(warp & 3), turn = (uint32_t)(warp - 2) / 4;
    uint8_t* mine = smem + kRingBytes + (warp - 2) * kStageWarp;
    uint32_t seg = 0;
    for (uint32_t i = first; i < tiles; i += step, ++seg) {
      const Tile t = tile_at(table, i, a.E, a.npair);
      const uint32_t buf = seg & 1;
      const uint32_t f = KIND == kGated ? (2 * t.col + rank) * 64 + 32 * (q & 1)
                                        : (2 * t.col + rank) * kBM + 32 * q;
      const uint32_t width = f < a.m ? a.m - f : 0;  // features from f on that are there
      uint4 g[2], u[2];                              // kDh: of the next chunk
      if (KIND == kDh && 16 * turn < t.rows) {
        const uint32_t r = 16 * turn;
        fetch_rows(g, a.gu_in, 2 * a.F, t.row + r, f, t.rows - r, width);
        fetch_rows(u, a.gu_in, 2 * a.F, t.row + r, a.F + f, t.rows - r, width);
      }
      const bool ok = wait_warp(&bar.tfull[buf], (seg >> 1) & 1, a.budget_ns, a.ctl);
      if (any_of(!ok, kEpilogue)) {  // all threads leave, or none
        if (threadIdx.x == 64) symm::record_error(a.ctl, symm::kErrTimedOut, -6);
        break;
      }
      symm::tc_fence_after();
      const uint32_t taddr = tmem + ((32 * q) << 16) + buf * kAccCols;
      if (KIND == kGated) {
        // Chunks of 32 rows: the warps of g finish the first 16, those of u the others.
        const uint32_t up = q >> 1;
        uint8_t* theirs = smem + kRingBytes + ((warp - 2) ^ 2) * kStageWarp;
        for (uint32_t c = 32 * turn; c < t.rows; c += 64) {
          uint32_t own[2][8], other[2][8];
          tmem_frags(taddr + c + 16 * (up ^ 1), other);
          tmem_frags(taddr + c + 16 * up, own);
          // the same lane of the other warp has the same elements' other half
#pragma unroll
          for (uint32_t j = 0; j < 4; ++j)
            reinterpret_cast<uint4*>(theirs)[32 * j + lane] =
                make_uint4(other[j / 2][4 * (j % 2)], other[j / 2][4 * (j % 2) + 1],
                           other[j / 2][4 * (j % 2) + 2], other[j / 2][4 * (j % 2) + 3]);
          symm::group_sync(2 + (int)(2 * turn + (q & 1)), 64);  // this pair of warps
#pragma unroll
          for (uint32_t j = 0; j < 4; ++j) {
            const uint4 v = reinterpret_cast<const uint4*>(mine)[32 * j + lane];
            other[j / 2][4 * (j % 2)] = v.x, other[j / 2][4 * (j % 2) + 1] = v.y;
            other[j / 2][4 * (j % 2) + 2] = v.z, other[j / 2][4 * (j % 2) + 3] = v.w;
          }
          __syncwarp();  // before what is read is staged over
          const uint32_t r = c + 16 * up;
          if (r < t.rows) {
            uint32_t p[2][4], h[2][8];
#pragma unroll
            for (uint32_t x = 0; x < 2; ++x)
#pragma unroll
              for (uint32_t j = 0; j < 8; ++j) {
                const float gate = __uint_as_float(up ? other[x][j] : own[x][j]);
                const float value = __uint_as_float(up ? own[x][j] : other[x][j]);
                h[x][j] = __float_as_uint(activate(a.act, gate) * value);
              }
            pack_frags<FMT>(h, p);
            put_rows<FMT>(mine, p, a.h, a.F, t.row + r, f, t.rows - r, width);
            if (a.gu) {
              pack_frags<FMT>(own, p);
              put_rows<FMT>(mine, p, a.gu, 2 * a.F, t.row + r, f + (up ? a.F : 0), t.rows - r,
                            width);
              pack_frags<FMT>(other, p);
              put_rows<FMT>(mine, p, a.gu, 2 * a.F, t.row + r, f + (up ? 0 : a.F), t.rows - r,
                            width);
            }
          }
          symm::group_sync(2 + (int)(2 * turn + (q & 1)), 64);
        }
      } else {
        for (uint32_t c = 16 * turn; c < t.rows; c += 32) {
          uint32_t v[2][8], p[2][4];
          const uint32_t row = t.row + c, valid = t.rows - c;
          if (KIND == kDh) {
            uint8_t* mine2 = mine + 16 * kLine;
            drop_rows(mine, g), drop_rows(mine2, u);
            __syncwarp();
            if (c + 32 < t.rows) {
              fetch_rows(g, a.gu_in, 2 * a.F, row + 32, f, valid - 32, width);
              fetch_rows(u, a.gu_in, 2 * a.F, row + 32, a.F + f, valid - 32, width);
            }
            uint32_t pg[2][4], pu[2][4];
            unstage_rows(mine, pg);
            unstage_rows(mine2, pu);
            tmem_frags(taddr + c, v);
            uint32_t dg[2][4], du[2][4];
#pragma unroll
            for (uint32_t x = 0; x < 2; ++x)
#pragma unroll
              for (uint32_t o = 0; o < 4; ++o) {
                const float2 gate = unpack2<FMT>(pg[x][o]), value = unpack2<FMT>(pu[x][o]);
                const float d0 = __uint_as_float(v[o / 2][4 * x + 2 * (o % 2)]);
                const float d1 = __uint_as_float(v[o / 2][4 * x + 2 * (o % 2) + 1]);
                float a0, a1, s0, s1;
                activate_both(a.act, gate.x, a0, s0);
                activate_both(a.act, gate.y, a1, s1);
                p[x][o] = symm::pack2<FMT>(a0 * value.x, a1 * value.y);
                dg[x][o] = symm::pack2<FMT>(d0 * value.x * s0, d1 * value.y * s1);
                du[x][o] = symm::pack2<FMT>(d0 * a0, d1 * a1);
              }
            __syncwarp();
            stage_rows(mine2, du);
            put_rows<FMT>(mine, dg, a.gu, 2 * a.F, row, f, valid, width);
            store_rows(mine2, static_cast<typename Elem<FMT>::T*>(a.gu) +
                                  (size_t)row * 2 * a.F + a.F + f,
                       2 * (size_t)a.F, valid, width, true);
            put_rows<FMT>(mine, p, a.h, a.F, row, f, valid, width);
          } else {
            tmem_frags(taddr + c, v);
            pack_frags<FMT>(v, p);
            put_rows<FMT>(mine, p, a.out, a.ldo, row, f, valid, width);
          }
        }
      }
      symm::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_first(&bar.tempty[buf]);  // the accumulator is free again
    }
  }
  leave_pair(&bar.drain, bar.tmem, 2 * kAccCols, a.budget_ns);
}

// ------------------------------------------------------------ grad_kernel --
__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_read() {  // shared memory may be written again
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// One launch computes up to two gradients (of the same rows): tiles of the first, then
// of the second.
struct GradPart {
  uint32_t m, nf;   // out [E][m][nf]
  uint32_t nb, per; // blocks of 256 columns, blocks of an expert's gradient
};
struct GradArgs {
  const int32_t* counts;
  uint32_t n, E;
  GradPart part[2];
  uint64_t budget_ns;
  Control* ctl;
};
struct GradTile {
  uint32_t which, e, m0, n0, m, nf;
};
// An expert's blocks of 256 columns one after another, then the next 256 rows.
__device__ __forceinline__ GradTile grad_tile(const GradArgs& a, uint32_t i) {
  GradTile t;
  const uint32_t tiles0 = a.E * a.part[0].per;
  t.which = i >= tiles0;
  if (t.which) i -= tiles0;
  const uint32_t per = t.which ? a.part[1].per : a.part[0].per;
  const uint32_t nb = t.which ? a.part[1].nb : a.part[0].nb;
  t.e = i / per;
  const uint32_t r = i - t.e * per, mb = r / nb;
  t.m0 = mb * 256, t.n0 = (r - mb * nb) * 256;
  t.m = t.which ? a.part[1].m : a.part[0].m, t.nf = t.which ? a.part[1].nf : a.part[0].nf;
  return t;
}
constexpr uint32_t kGradStage = 4 * 64 * 128;  // two boxes of A, two of B: 64 rows x 64 features
constexpr uint32_t kGradStages = kRingBytes / kGradStage;

template <int FMT>
__global__ void __launch_bounds__(kThreads, 1)
    grad_kernel(const __grid_constant__ CUtensorMap map_a0,
                const __grid_constant__ CUtensorMap map_b0,
                const __grid_constant__ CUtensorMap map_out0,
                const __grid_constant__ CUtensorMap map_a1,
                const __grid_constant__ CUtensorMap map_b1,
                const __grid_constant__ CUtensorMap map_out1, const GradArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (symm::smem_addr(smem_raw) & 1023u)) & 1023u);
  __shared__ Barriers bar;
  __shared__ Table table;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  set_up_cta(bar, warp);
  moe::wait_for_earlier();
  const bool good = lay_out(table, a.counts, a.E, a.n, kMaxRows, 0, 1, 1);
  if (!good && blockIdx.x == 0 && threadIdx.x == 0) symm::record_error(a.ctl, kErrRange, -1);
  pair_wait();
  const uint32_t tiles = good ? a.E * (a.part[0].per + a.part[1].per) : 0;
  const uint32_t tmem = uniform(bar.tmem);
  const uint32_t rank = pair_rank(), first = blockIdx.x / 2, step = gridDim.x / 2;

  if (warp == 0) {  // ----------------------------------------- TMA producer
    const bool elected = symm::elect_one();
    uint32_t st = 0, ph = 1, it = 0;
    bool ok = true;
    for (uint32_t i = first; ok && i < tiles; i += step) {
      const GradTile t = grad_tile(a, i);
      const CUtensorMap* map_a = t.which ? &map_a1 : &map_a0;
      const CUtensorMap* map_b = t.which ? &map_b1 : &map_b0;
      const uint32_t m0 = t.m0 + rank * kBM, n0 = t.n0 + rank * kBM;
      const uint32_t r0 = table.off[t.e], r1 = table.off[t.e + 1];
      for (uint32_t r = r0; r < r1; r += 64) {
        if (!(ok = wait_warp(&bar.empty[st], ph, a.budget_ns, a.ctl))) break;
        uint8_t* buf = smem + st * kGradStage;
        if (elected) {
          symm::mbar_arrive_expect_tx(&bar.full[st], kGradStage);
#pragma unroll
          for (uint32_t b = 0; b < 2; ++b)
            symm::tma_load_2d(buf + b * 8192, map_a, (int)(m0 + 64 * b), (int)r, &bar.full[st]);
#pragma unroll
          for (uint32_t b = 0; b < 2; ++b)
            symm::tma_load_2d(buf + (2 + b) * 8192, map_b, (int)(n0 + 64 * b), (int)r,
                              &bar.full[st]);
        }
        ++it;
        if (++st == kGradStages) st = 0, ph ^= 1;
      }
    }
    if (!ok && elected) symm::record_error(a.ctl, symm::kErrTimedOut, -3);
    drain_ring(bar.full, bar.empty, kGradStages, it, ok, a.budget_ns);
  } else if (warp == 1) {  // ------ MMA issuer, or tells the first CTA what is here
    const bool elected = symm::elect_one();
    const uint32_t idesc = mma_idesc(FMT, 256, true, true);
    uint32_t st = 0, ph = 0, seg = 0;
    bool ok = true;
    for (uint32_t i = first; ok && i < tiles; i += step) {
      const uint32_t e = grad_tile(a, i).e, r0 = table.off[e], r1 = table.off[e + 1];
      if (r0 == r1) continue;  // the epilogue writes zeros
      const uint32_t buf = seg & 1;
      const uint32_t phase = ((seg >> 1) & 1) ^ 1u;
      if (!rank && !(ok = wait_warp(&bar.tempty[buf], phase, a.budget_ns, a.ctl))) break;
      symm::tc_fence_after();
      const uint32_t acc = tmem + buf * kAccCols;
      for (uint32_t r = r0; r < r1; r += 64) {
        if (!(ok = wait_warp(&bar.full[st], ph, a.budget_ns, a.ctl))) break;
        uint8_t* at = smem + st * kGradStage;
        const uint32_t left = min(64u, r1 - r), steps = (left + 15) / 16;
        if (left % 16) {  // the next expert's rows in the last step, a line of all boxes a turn
          uint8_t* line = at + (lane / 8) * 8192 + (lane % 8) * 16;
          for (uint32_t z = left; z < steps * 16; ++z)
            *reinterpret_cast<uint4*>(line + z * 128) = make_uint4(0, 0, 0, 0);
          symm::fence_proxy_async_shared();
          __syncwarp();
        }
        if (rank) {
          if (elected) arrive_first(&bar.full[st]);
        } else {
          symm::tc_fence_after();
          const uint64_t ad = symm::sw128_mnmajor_desc(at);
          const uint64_t bd = symm::sw128_mnmajor_desc(at + 16384);
          if (elected) {
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j)
              if (j < steps)
                pair_mma(acc, ad + kMajorStep * j, bd + kMajorStep * j, idesc, r != r0 || j != 0);
            pair_commit(&bar.empty[st]);
          }
        }
        if (++st == kGradStages) st = 0, ph ^= 1;
      }
      if (ok && elected && !rank) pair_commit(&bar.tfull[buf]);
      ++seg;
    }
    if (!ok && elected) symm::record_error(a.ctl, symm::kErrTimedOut, -5);
    if (!rank && elected) pair_commit(&bar.drain);
  } else {  // -------------------------------------------------- epilogue
    const uint32_t q = (uint32_t)(warp & 3), turn = (uint32_t)(warp - 2) / 4;
    // 16 rows of the gradient and 64 columns go out by one copy: whole lines of 128
    // bytes, swizzled.  Gradients of 16 experts of 2048 x 2816, 32 rows each: 56 us;
    // stores from registers, 64 or 128 bytes a row, 71 and 59; three boxes a warp of 8
    // rows (twice the proxy fences) 66, of 16 rows with a ring stage less 53, but then
    // 500 rows an expert took 435 us instead of 390.
    uint8_t* mine = smem + kGradStages * kGradStage + (warp - 2) * kGradBox;
    const bool elected = symm::elect_one();
    uint32_t seg = 0;
    for (uint32_t i = first; i < tiles; i += step) {
      const GradTile t = grad_tile(a, i);
      const uint32_t e = t.e, n0 = t.n0, m0 = t.m0 + rank * kBM + 32 * q + 16 * turn;
      const uint32_t m = t.m, nf = t.nf, buf = seg & 1;
      const bool any = table.off[e] != table.off[e + 1];
      if (any) {
        const bool ok = wait_warp(&bar.tfull[buf], (seg >> 1) & 1, a.budget_ns, a.ctl);
        if (any_of(!ok, kEpilogue)) {  // all threads leave, or none
          if (threadIdx.x == 64) symm::record_error(a.ctl, symm::kErrTimedOut, -6);
          break;
        }
        symm::tc_fence_after();
        ++seg;
      }
      const uint32_t taddr = tmem + ((32 * q + 16 * turn) << 16) + buf * kAccCols;
      for (uint32_t c = 0; c < 256 && n0 + c < nf; c += 64) {
        uint32_t v[4][8];
        if (any) {
#pragma unroll
          for (uint32_t j = 0; j < 4; ++j) tmem_frag16(taddr + c + 16 * j, v[j]);
          tmem_wait(v[0], v[1]);
          tmem_wait(v[2], v[3]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[0][j] = v[1][j] = v[2][j] = v[3][j] = 0;
        }
        if (m0 >= m) continue;
        uint32_t pk[2][8];
#pragma unroll
        for (uint32_t o = 0; o < 2; ++o)
#pragma unroll
          for (uint32_t j = 0; j < 8; ++j)
            pk[o][j] = symm::pack2<FMT>(__uint_as_float(v[j / 2][4 * (j % 2) + 2 * o]),
                                        __uint_as_float(v[j / 2][4 * (j % 2) + 2 * o + 1]));
        if (elected) bulk_wait_read();  // the copy before
        __syncwarp();
        // matrices of 8 rows x 8 columns, as they are: 16 bytes of a line each
#pragma unroll
        for (uint32_t o = 0; o < 2; ++o)
#pragma unroll
          for (uint32_t j = 0; j < 4; j += 2) {
            const uint32_t at = (lane & 7) * 128 + (((2 * j + (lane >> 3)) ^ (lane & 7)) << 4);
            stmatrix(symm::smem_addr(mine) + 1024 * o + at, pk[o][2 * j], pk[o][2 * j + 1],
                     pk[o][2 * j + 2], pk[o][2 * j + 3]);
          }
        symm::fence_proxy_async_shared();
        __syncwarp();
        if (elected) {
          symm::tma_store_3d(t.which ? &map_out1 : &map_out0, mine, (int)(n0 + c), (int)m0, (int)e);
          bulk_commit();
        }
      }
      if (any) {
        symm::tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_first(&bar.tempty[buf]);
      }
    }
    if (elected) bulk_wait();
  }
  leave_pair(&bar.drain, bar.tmem, 2 * kAccCols, a.budget_ns);
}

// ------------------------------------------------------------------- host --
size_t up(size_t v, size_t a) { return (v + a - 1) / a * a; }

int check_sizes(const char* what, int n, int E, int D, int F) {
  if (n < 0 || n > (1 << 24) || E < 1 || E > SYMM_MOE_MAX_EXPERTS)
    return fail(SYMM_EINVAL, std::string(what) + ": n must be in [0, 2^24], E in [1, 1024]");
  if (D < 8 || F < 8 || D % 8 || F % 8 || D > (1 << 17) || F > (1 << 17))
    return fail(SYMM_EINVAL, std::string(what) + ": D and F must be multiples of 8 (16-byte rows) "
                                                 "in [8, 2^17]");
  return SYMM_OK;
}
size_t h_bytes(int n, int F) { return up((size_t)n * F * 2, 256); }

// [depth][rows][inner] elements of 16 bits, rows `ld` apart, planes rows * ld;
// boxes of 64 x box_rows, 128-byte swizzled; depth 0: a 2-d map.
int make_map(const char* what, CUtensorMap* map, const void* base, int fmt, uint64_t inner,
             uint64_t rows, uint64_t depth, size_t ld, uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return fail(SYMM_ECUDA, std::string(what) + ": no cuTensorMapEncodeTiled");
  const cuuint64_t dims[3] = {inner, rows, depth};
  const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)ld * rows * 2};
  const cuuint32_t box[3] = {64, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r =
      fn(map, fmt == 1 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
         depth ? 3 : 2, const_cast<void*>(base), dims, strides, box, estr,
         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(SYMM_ECUDA,
                std::string(what) + ": tensor map rejected (CUresult " + std::to_string(r) + ")");
  return SYMM_OK;
}

// Once per device: the kernels may use more than 48 KB of shared memory.  *pairs:
// CTA pairs that are resident at once (all kernels have the same resources).
template <int FMT>
int set_up(unsigned* pairs) {
  static std::mutex mu;
  static unsigned known[64] = {};
  int dev = 0;
  int rc = cuda_check(cudaGetDevice(&dev), "moe_expert_ffn: device");
  if (rc) return rc;
  std::lock_guard<std::mutex> lock(mu);
  const bool keep = dev >= 0 && dev < 64;
  if (keep && known[dev]) {
    *pairs = known[dev];
    return SYMM_OK;
  }
  for (const void* f : {(const void*)rows_kernel<FMT, kGated>, (const void*)rows_kernel<FMT, kDown>,
                        (const void*)rows_kernel<FMT, kDh>, (const void*)rows_kernel<FMT, kDx>,
                        (const void*)grad_kernel<FMT>})
    if (!rc)
      rc = cuda_check(cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)kSmemBytes),
                      "moe_expert_ffn: kernel set-up");
  if (rc) return rc;
  *pairs = resident_pairs((const void*)rows_kernel<FMT, kGated>, kThreads, kSmemBytes);
  if (keep) known[dev] = *pairs;
  return SYMM_OK;
}

// One product of the rows x [n][k] (ldx apart) with the experts' weights, stored
// [E][wrows][wcols].
template <int FMT, int KIND>
int rows_product(const char* what, const void* x, size_t ldx, const void* w, uint32_t wrows,
                 uint32_t wcols, ExpertArgs a, unsigned pairs, cudaStream_t s) {
  constexpr bool kMMajor = KIND == kGated || KIND == kDown;
  CUtensorMap mw, m64, m16;
  int rc = make_map(what, &mw, w, FMT, wcols, wrows, a.E, wcols, kMMajor ? kBK : kBM);
  if (!rc) rc = make_map(what, &m64, x, FMT, a.k, a.n, 0, ldx, 64);
  if (!rc) rc = make_map(what, &m16, x, FMT, a.k, a.n, 0, ldx, 16);
  if (rc) return rc;
  a.npair = (a.m + (KIND == kGated ? 127 : 255)) / (KIND == kGated ? 128 : 256);
  // at most one partly filled block of rows, 64 at the least, for each expert that has rows
  const uint64_t most = (uint64_t)a.npair * std::min<uint64_t>(a.n, a.n / 64 + a.E);
  return launch_pairs(what, rows_kernel<FMT, KIND>, (unsigned)std::min<uint64_t>(pairs, most),
                      kThreads, kSmemBytes, s, mw, m64, m16, a);
}

// A gradient dW [E][m][nf] = a_e^T b_e of the rows a [n][m] and b [n][nf]; out NULL: none.
struct WeightGrad {
  const void *a, *b;
  size_t lda, ldb;
  void* out;
  uint32_t m, nf;
};
template <int FMT>
int weight_grads(const char* what, const WeightGrad (&w)[2], const ExpertArgs& x, unsigned pairs,
                 cudaStream_t s) {
  CUtensorMap maps[2][3] = {};
  GradArgs g{};
  uint64_t tiles = 0;
  int rc = SYMM_OK, parts = 0;
  for (const WeightGrad& p : w) {
    if (!p.out || rc) continue;
    CUtensorMap* m = maps[parts];
    rc = make_map(what, &m[0], p.a, FMT, p.m, x.n, 0, p.lda, 64);
    if (!rc) rc = make_map(what, &m[1], p.b, FMT, p.nf, x.n, 0, p.ldb, 64);
    if (!rc) rc = make_map(what, &m[2], p.out, FMT, p.nf, p.m, x.E, p.nf, 16);
    GradPart& to = g.part[parts++];
    to.m = p.m, to.nf = p.nf, to.nb = (p.nf + 255) / 256;
    to.per = (p.m + 255) / 256 * to.nb;
    tiles += (uint64_t)x.E * to.per;
  }
  if (rc || !parts) return rc;
  if (parts == 1) std::copy(maps[0], maps[0] + 3, maps[1]);  // no tile uses them
  g.counts = x.counts, g.n = x.n, g.E = x.E, g.budget_ns = x.budget_ns, g.ctl = x.ctl;
  return launch_pairs(what, grad_kernel<FMT>, (unsigned)std::min<uint64_t>(pairs, tiles), kThreads,
                      kSmemBytes, s, maps[0][0], maps[0][1], maps[0][2], maps[1][0], maps[1][1],
                      maps[1][2], g);
}

// What both entry points check of their sizes, weights and type.
int check_common(const char* what, const symm_heap_t* heap, const int32_t* counts,
                 const void* w_gu, const void* w_d, int act, int dtype, int n, int E, int D,
                 int F) {
  if (!heap) return fail(SYMM_EINVAL, std::string(what) + ": NULL heap");
  if (dtype != SYMM_DTYPE_F16 && dtype != SYMM_DTYPE_BF16)
    return fail(SYMM_EINVAL, std::string(what) + ": dtype must be SYMM_DTYPE_F16 or _BF16");
  if (act != SYMM_ACT_SILU && act != SYMM_ACT_GELU)
    return fail(SYMM_EINVAL, std::string(what) + ": act must be SYMM_ACT_SILU or _GELU");
  const int rc = check_sizes(what, n, E, D, F);
  if (rc) return rc;
  if (!counts && E != 1)
    return fail(SYMM_EINVAL, std::string(what) + ": counts may be NULL with one expert only");
  if (!w_gu || !w_d) return fail(SYMM_EINVAL, std::string(what) + ": NULL weights");
  if (!moe::aligned(w_gu, 16) || !moe::aligned(w_d, 16) || !moe::aligned(counts, 4))
    return fail(SYMM_EINVAL, std::string(what) + ": weights must be 16-byte aligned, counts to "
                                                 "their elements");
  return SYMM_OK;
}
bool bad_ld(size_t ld, int width) {
  return ld < (size_t)width || ld % 8 || ld > (1ull << 36);
}

template <int FMT>
int forward(const char* what, const void* x, size_t ldx, const void* w_gu, const void* w_d, int D,
            int F, void* gu, void* y, size_t ldy, void* h, ExpertArgs a, cudaStream_t s) {
  unsigned pairs = 0;
  int rc = set_up<FMT>(&pairs);
  if (rc) return rc;
  a.m = (uint32_t)F, a.k = (uint32_t)D, a.gu = gu, a.h = h;
  rc = rows_product<FMT, kGated>(what, x, ldx, w_gu, D, 2 * F, a, pairs, s);
  if (rc) return rc;
  a.m = (uint32_t)D, a.k = (uint32_t)F, a.out = y, a.ldo = ldy;
  return rows_product<FMT, kDown>(what, h, F, w_d, F, D, a, pairs, s);
}

template <int FMT>
int backward(const char* what, const void* dy, size_t lddy, const void* x, size_t ldx,
             const void* gu, const void* w_gu, const void* w_d, int D, int F, void* dx,
             size_t lddx, void* dw_gu, void* dw_d, void* h, void* dgu, ExpertArgs a,
             cudaStream_t s) {
  unsigned pairs = 0;
  int rc = set_up<FMT>(&pairs);
  if (!rc && a.n) {
    a.m = (uint32_t)F, a.k = (uint32_t)D, a.gu_in = gu, a.gu = dgu, a.h = h;
    rc = rows_product<FMT, kDh>(what, dy, lddy, w_d, F, D, a, pairs, s);
    if (!rc && dx) {
      a.m = (uint32_t)D, a.k = 2 * (uint32_t)F, a.out = dx, a.ldo = lddx;
      rc = rows_product<FMT, kDx>(what, dgu, 2 * (size_t)F, w_gu, D, 2 * F, a, pairs, s);
    }
  }
  if (!rc)
    rc = weight_grads<FMT>(what,
                           {{h, dy, (size_t)F, lddy, dw_d, (uint32_t)F, (uint32_t)D},
                            {x, dgu, ldx, 2 * (size_t)F, dw_gu, (uint32_t)D, 2 * (uint32_t)F}},
                           a, pairs, s);
  return rc;
}

}  // namespace

extern "C" int moe_expert_workspace(int n, int E, int D, int F, int backward, size_t* bytes) {
  return moe::entry("moe_expert_workspace", [&]() -> int {
    if (!bytes) return fail(SYMM_EINVAL, "moe_expert_workspace: NULL bytes");
    const int rc = check_sizes("moe_expert_workspace", n, E, D, F);
    if (rc) return rc;
    *bytes = h_bytes(n, F) + (backward ? h_bytes(n, 2 * F) : 0);
    return SYMM_OK;
  });
}

extern "C" int moe_expert_ffn(symm_heap_t* heap, const void* x, size_t ldx, const int32_t* counts,
                              const void* w_gu, const void* w_d, int act, int dtype, int n, int E,
                              int D, int F, void* gu, void* y, size_t ldy, void* workspace,
                              void* stream) {
  return moe::entry("moe_expert_ffn", [&]() -> int {
    const char* what = "moe_expert_ffn";
    int rc = check_common(what, heap, counts, w_gu, w_d, act, dtype, n, E, D, F);
    if (rc) return rc;
    if (bad_ld(ldx, D) || bad_ld(ldy, D))
      return fail(SYMM_EINVAL, "moe_expert_ffn: ldx, ldy >= D (multiples of 8)");
    if (n == 0) return SYMM_OK;
    if (!x || !y || !workspace) return fail(SYMM_EINVAL, "moe_expert_ffn: NULL x, y or workspace");
    if (!moe::aligned(x, 16) || !moe::aligned(y, 16) || !moe::aligned(gu, 16) ||
        !moe::aligned(workspace, 256))
      return fail(SYMM_EINVAL, "moe_expert_ffn: x, y and gu must be 16-byte aligned, workspace "
                               "256-byte");
    if (y == x || y == w_gu || y == w_d || y == gu || (gu && (gu == x || gu == w_gu || gu == w_d)))
      return fail(SYMM_EINVAL, "moe_expert_ffn: outputs must not be inputs or each other");
    cudaStream_t s = as_stream(stream);
    rc = ensure_ctrl(heap, s);
    if (rc) return rc;
    ExpertArgs a{};
    a.counts = counts, a.n = (uint32_t)n, a.E = (uint32_t)E, a.F = (uint32_t)F, a.act = act;
    a.budget_ns = heap->spin_budget, a.ctl = reinterpret_cast<Control*>(heap->base);
    return dtype == SYMM_DTYPE_BF16
               ? forward<1>(what, x, ldx, w_gu, w_d, D, F, gu, y, ldy, workspace, a, s)
               : forward<0>(what, x, ldx, w_gu, w_d, D, F, gu, y, ldy, workspace, a, s);
  });
}

extern "C" int moe_expert_ffn_backward(symm_heap_t* heap, const void* dy, size_t lddy,
                                       const void* x, size_t ldx, const void* gu,
                                       const int32_t* counts, const void* w_gu, const void* w_d,
                                       int act, int dtype, int n, int E, int D, int F, void* dx,
                                       size_t lddx, void* dw_gu, void* dw_d, void* workspace,
                                       void* stream) {
  return moe::entry("moe_expert_ffn_backward", [&]() -> int {
    const char* what = "moe_expert_ffn_backward";
    int rc = check_common(what, heap, counts, w_gu, w_d, act, dtype, n, E, D, F);
    if (rc) return rc;
    if (bad_ld(lddy, D) || bad_ld(ldx, D) || (dx && bad_ld(lddx, D)))
      return fail(SYMM_EINVAL, "moe_expert_ffn_backward: lddy, ldx, lddx >= D (multiples of 8)");
    if (n && (!dy || !x || !gu || !workspace))
      return fail(SYMM_EINVAL, "moe_expert_ffn_backward: NULL dy, x, gu or workspace");
    if (!moe::aligned(dy, 16) || !moe::aligned(x, 16) || !moe::aligned(gu, 16) ||
        !moe::aligned(dx, 16) || !moe::aligned(dw_gu, 16) || !moe::aligned(dw_d, 16) ||
        !moe::aligned(workspace, 256))
      return fail(SYMM_EINVAL, "moe_expert_ffn_backward: the tensors must be 16-byte aligned, "
                               "workspace 256-byte");
    const void* in[] = {dy, x, gu, w_gu, w_d};
    const void* out[] = {dx, dw_gu, dw_d};
    for (int i = 0; i < 3; ++i)
      for (int j = 0; out[i] && j < 5 + i; ++j)
        if (out[i] == (j < 5 ? in[j] : out[j - 5]))
          return fail(SYMM_EINVAL,
                      "moe_expert_ffn_backward: outputs must not be inputs or each other");
    cudaStream_t s = as_stream(stream);
    rc = ensure_ctrl(heap, s);
    if (rc) return rc;
    if (n == 0) {  // no rows: gradients of zero
      const size_t half = (size_t)E * D * F * 2;
      if (dw_gu) rc = cuda_check(cudaMemsetAsync(dw_gu, 0, 2 * half, s), what);
      if (!rc && dw_d) rc = cuda_check(cudaMemsetAsync(dw_d, 0, half, s), what);
      return rc;
    }
    ExpertArgs a{};
    a.counts = counts, a.n = (uint32_t)n, a.E = (uint32_t)E, a.F = (uint32_t)F, a.act = act;
    a.budget_ns = heap->spin_budget, a.ctl = reinterpret_cast<Control*>(heap->base);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    void* dgu = ws + h_bytes(n, F);
    return dtype == SYMM_DTYPE_BF16
               ? backward<1>(what, dy, lddy, x, ldx, gu, w_gu, w_d, D, F, dx, lddx, dw_gu, dw_d,
                             ws, dgu, a, s)
               : backward<0>(what, dy, lddy, x, ldx, gu, w_gu, w_d, D, F, dx, lddx, dw_gu, dw_d,
                             ws, dgu, a, s);
  });
}
