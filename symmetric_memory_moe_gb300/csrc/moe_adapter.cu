// moe_adapter.cu -- a projection shared by all requests with one low-rank
// adapter per request: y_t = x_t W + scale_a (x_t A_a) B_a, a = ids_t.
//
// Two launches, both on the tensor cores.  The first (rank_kernel) computes
// h_t = scale_a x_t A_a.  The second (adapter_kernel) is the product with W, in
// which each adapter of a tile's tokens is a few more K columns: B_a under W,
// and h (0 in the rows of the other adapters' tokens) beside x.  So any
// mixture of adapters in any order of tokens is summed in the same 32-bit
// accumulators before the one rounding.  h keeps the 24 bits and the range of
// its 32-bit sum: it enters as three bf16 values of 8 bits each.  (Two take 7 us
// less at the prompts below, but move as many outputs across a rounding
// boundary as the whole sum over k does.)  With fp16 inputs, whose range and
// bits h would leave, B becomes two bf16 values, 11 bits in all, on its way.
//
// The product is computed as y^T = W^T x^T: the M side of a tile is 128
// columns of W (W as stored, k x n, is an M-major operand) and the N side BT
// tokens, 16 to 256.  One token then wastes no more than a narrow N, and one
// kernel serves a decoding step and a prompt.
//   warp 0     TMA producer: K slices of W (two boxes of 64 columns) and of x
//              into a ring of shared-memory stages, 128-byte swizzled, 64 deep
//              or, with few tokens, 128 (a slice costs each role some 250
//              cycles beside its MMAs); and the adapters' B;
//   warp 1     MMA issuer: tcgen05.mma kind::f16, M 128, N BT, two
//              accumulators in TMEM;
//   warps 2-5  the adapters' h into the ring, then the epilogue: tcgen05.ld,
//              rounding, stores (a warp's 32 lanes are 32 columns of a token).
// Where whole tiles would leave SMs idle, a cluster of 2 to 8 CTAs shares a
// tile: each takes a part of K and of the adapters, and the parts are joined in
// rank order through distributed shared memory, each CTA storing its share of
// the tokens.  The second launch starts while the first runs (programmatic
// dependent launch) and waits for its results only where it needs them.  Every
// wait is bounded; a role that gives up records the error in the heap's header.
//
// rank_kernel: h^T = A_a^T x^T the same way (A as stored, k x r, is an M-major
// operand, rows r to 127 of the tile unused).  Per block of 128 tokens, a CTA
// sorts the ids, and gathers the x rows of each adapter's tokens (tile::gather4)
// as the N side, for one part of K; the CTAs of a cluster add their parts in
// rank order through distributed shared memory.  A block's adapters are dealt
// out to several clusters while there are few blocks.
//
// Measured (bf16): 8192 tokens, k = n = 4096, 8 adapters of rank 32: 199 us, of
// which the product without adapters is 165 (1.67 PFLOP/s, 88 % of the burst
// rate); one token, k = n = 8192: 23.3 us, 5.8 TB/s or 85 % of the copy rate; 64
// tokens with 32 adapters of rank 16, 7168 x 2048: 21.4 us, 7.8 without adapters
// (the rank products, 9 us, are two rounds of memory latency long).
#include <algorithm>
#include <string>

#include "moe_common.cuh"
#include "symm_device.cuh"
#include "symm_internal.h"
#include "symm_tcgen05.cuh"

using symm::Control;
using namespace symm_host;

namespace {

constexpr int kBM = 128, kBK = 64;
constexpr int kThreads = 192;
constexpr int kMaxStages = 12;
constexpr uint32_t kATile = kBM * kBK * 2;
constexpr uint32_t kParts = 3;  // bf16 values that make up an element of h
// The product's ring.  (96 KB with few tokens, so that two CTAs fit on an SM and
// one beside the first launch's, takes 21.6 us instead of 20.5 at 64 requests.)
constexpr uint32_t kRingBytes = 200 * 1024;
constexpr int kRankTokens = 128;  // tokens of a rank_kernel CTA, at most
constexpr int kRankStages = 12;
constexpr uint32_t kRankBytes = 98 * 1024;  // of its ring and sums, with two CTAs per SM

struct AdapterArgs {
  const float* scale;
  const int32_t* ids;
  const void* b;
  void* y;
  size_t ldy;
  uint32_t T, k, n, R, r, r16;  // r16: r in whole K steps of 16
  uint32_t bt, ntok, ncol, stages;  // tiles: ncol column blocks x ntok token blocks
  uint32_t deep, slices;            // 64-deep K tiles per slice, slices of K
  uint32_t ktiles;                  // 64-deep K tiles (rank_kernel's slices)
  uint32_t cluster, tmem_cols;  // cluster: CTAs that share a tile
  uint16_t* h;      // bf16 [T][r16 / 16][3][16]: of 16 ranks, their three parts
  uint64_t budget_ns;
  Control* ctl;
  // rank_kernel: clusters per token block, bytes of its ring and of A in a stage
  uint32_t rk_share, rk_ring, rk_abytes;
};

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(symm::smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(symm::smem_addr(bar))
      : "memory");
}

template <int FMT>
struct Elem {
  using T = __half;
};
template <>
struct Elem<1> {
  using T = __nv_bfloat16;
};

// 4 rows of a 2-d tensor map whose box is one row
__device__ __forceinline__ void tma_gather4(void* dst, const CUtensorMap* map, int x, int4 rows,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(symm::smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(rows.x), "r"(rows.y), "r"(rows.z),
      "r"(rows.w), "r"(symm::smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void prefetch_3d(const CUtensorMap* map, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z)
               : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t v;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(v));
  return v;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t v;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(v));
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
}
// The last one, which no memory access is ordered by: reads of the other CTAs'
// shared memory have returned their values (they were used), and waiting for
// this CTA's stores to global memory would only take time.
__device__ __forceinline__ void cluster_leave() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;"
               ::: "memory");
}
// `addr` (a shared-memory address of this CTA) in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_cluster(uint32_t addr, uint32_t rank) {
  uint32_t remote;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  return remote;
}
__device__ __forceinline__ float ld_cluster(uint32_t remote) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t remote) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(remote)
               : "memory");
  return v;
}

// How long a CTA that gives up waits for its own copies and MMAs, which nothing
// but the hardware holds up: a second, however short the heap's budget is.
__device__ __forceinline__ uint64_t drain_ns(const AdapterArgs& a) {
  return max(a.budget_ns, (uint64_t)1000000000);
}

// Instruction descriptor: fp32 accumulator, both operands of one type, the M
// side M-major (bit 15), the N side K-major.
__device__ __forceinline__ uint32_t mma_idesc(uint32_t fmt, uint32_t n) {
  return (1u << 4) | (fmt << 7) | (fmt << 10) | (1u << 15) | ((n >> 3) << 17) |
         ((uint32_t)(kBM >> 4) << 24);
}
constexpr uint64_t kWStep = (16 * 128) >> 4;  // 16 K rows of an M-major tile
constexpr uint64_t kXStep = 32 >> 4;          // 16 K columns of a K-major tile

// The adapters' columns of a tile come in pieces of one ring stage: up to 4
// steps of 16 K columns of h as it lies in memory, step 3i + j the j-th part of
// ranks 16i ..; and the 16 or 32 ranks of B that they multiply.
__device__ __forceinline__ uint32_t pieces_of(const AdapterArgs& a) {
  return (a.r16 / 16 * kParts + 3) / 4;
}
__device__ __forceinline__ uint32_t piece_steps(const AdapterArgs& a, uint32_t p) {
  return min(4u, a.r16 / 16 * kParts - 4 * p);
}
__device__ __forceinline__ uint32_t piece_rank(uint32_t p) {  // the first one
  return 4 * p / kParts * 16;
}
__host__ __device__ __forceinline__ uint32_t piece_rows(uint32_t r16) {  // of B
  return r16 < 2 * 16 ? r16 : 2 * 16;
}
// With fp16 inputs, rows of a stage's B from its first (high) to its second
// (low) bf16 part.
constexpr uint32_t kLowRows = 32;

// h of up to 128 tokens: see the head of the file.
template <int FMT>
__global__ void __launch_bounds__(kThreads)
    rank_kernel(const __grid_constant__ CUtensorMap map_a,
                const __grid_constant__ CUtensorMap map_x,
                const __grid_constant__ CUtensorMap map_x16,
                const __grid_constant__ CUtensorMap map_b, const AdapterArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (symm::smem_addr(smem_raw) & 1023u)) & 1023u);
  // the ring, 8 KB that the unused M rows may read, then the sums
  float* sums = reinterpret_cast<float*>(smem + a.rk_ring + 8192);
  __shared__ uint64_t full[kRankStages], empty[kRankStages], tfull[2], tempty[2], drain;
  __shared__ uint32_t tmem_slot;
  __shared__ __align__(16) uint32_t id_of[kRankTokens];  // by token
  __shared__ int order[kRankTokens];           // tokens by adapter
  __shared__ uint32_t sorted[kRankTokens];     // their ids
  __shared__ float scales[kRankTokens];        // their adapters' scales
  __shared__ uint32_t start[kRankTokens + 1];  // first position of each adapter's tokens
  __shared__ uint32_t nitems, most_rows;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t crank = cluster_rank(), csize = cluster_size();

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < kRankStages; ++s) {
      symm::mbar_init(&full[s], 1);
      symm::mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      symm::mbar_init(&tfull[b], 1);
      symm::mbar_init(&tempty[b], 128);
    }
    symm::mbar_init(&drain, 1);
    symm::fence_mbar_init();
  }
  if (warp == 5) symm::tmem_alloc(&tmem_slot, 256);
  moe::wait_for_earlier();  // here: for whatever is before this call on the stream
  // The second launch may start only now: it reads x and W at once, which that
  // may have written; and its CTAs take TMEM, and hold it while they wait for
  // this launch (warp 5 has this CTA's).
  if (warp == 5) moe::let_next_start();

  // this block's tokens, sorted by adapter (tokens without one last)
  const uint32_t group = blockIdx.x / csize, t0 = group / a.rk_share * kRankTokens;
  const uint32_t share = group % a.rk_share;  // its adapters: share, share + rk_share, ..
  const uint32_t mine = threadIdx.x;
  if (mine < kRankTokens) {
    const uint32_t t = t0 + mine;
    const uint32_t id = t < a.T ? (uint32_t)a.ids[t] : 0xffffffffu;
    id_of[mine] = id < a.R ? id : 0xffffffffu;
  }
  __syncthreads();
  if (mine < kRankTokens) {
    const uint32_t id = id_of[mine];
    uint32_t pos = 0;
#pragma unroll 8
    for (uint32_t j = 0; j < kRankTokens; j += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(&id_of[j]);
      pos += v.x < id || (v.x == id && j < mine);
      pos += v.y < id || (v.y == id && j + 1 < mine);
      pos += v.z < id || (v.z == id && j + 2 < mine);
      pos += v.w < id || (v.w == id && j + 3 < mine);
    }
    order[pos] = (int)(t0 + mine);
    sorted[pos] = id;
  }
  __syncthreads();
  if (warp == 0) {
    uint32_t count = 0, valid = 0;
    for (uint32_t i0 = 0; i0 < kRankTokens; i0 += 32) {
      const uint32_t i = i0 + lane;
      const bool ok = sorted[i] != 0xffffffffu;
      const bool first = ok && (i == 0 || sorted[i - 1] != sorted[i]);
      const uint32_t votes = __ballot_sync(0xffffffffu, first);
      if (first) start[count + __popc(votes & ((1u << lane) - 1))] = i;
      count += __popc(votes);
      valid += __popc(__ballot_sync(0xffffffffu, ok));
    }
    if (lane == 0) start[count] = valid, nitems = count;
    __syncwarp();
    uint32_t most = 16;  // rows of this cluster's largest adapter, in whole N steps
    for (uint32_t i = share + a.rk_share * lane; i < count; i += a.rk_share * 32)
      most = max(most, (start[i + 1] - start[i] + 15) / 16 * 16);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) most_rows = most;
  }
  symm::tc_fence_before();
  __syncthreads();
  symm::tc_fence_after();
  const uint32_t tmem = tmem_slot, items = nitems;
  // stages of A | x rows, as many as the ring holds
  const uint32_t stage_bytes = a.rk_abytes + most_rows * 128;
  const uint32_t stages = min((uint32_t)kRankStages, a.rk_ring / stage_bytes);
  const uint32_t k0 = a.ktiles * crank / csize, k1 = a.ktiles * (crank + 1) / csize;

  if (warp == 0) {  // --------------------------------------- TMA producer
    // lane q gathers rows 4q .. 4q + 3 of the adapter; past them T, a row
    // past the end of x: zeros
    const bool elected = symm::elect_one();
    uint32_t st = 0, ph = 1, it = 0;
    bool ok = true;
    for (uint32_t i = share; ok && i < items; i += a.rk_share) {
      const uint32_t p0 = start[i], rows = start[i + 1] - p0, rows16 = (rows + 15) / 16 * 16;
      const uint32_t q = 4 * lane;
      int4 r;
      r.x = q + 0 < rows ? order[p0 + q + 0] : (int)a.T;
      r.y = q + 1 < rows ? order[p0 + q + 1] : (int)a.T;
      r.z = q + 2 < rows ? order[p0 + q + 2] : (int)a.T;
      r.w = q + 3 < rows ? order[p0 + q + 3] : (int)a.T;
      const int id = (int)sorted[p0];
      // consecutive tokens (a prompt): boxes of 16 rows, lane q rows 16q ..; the
      // rows past the adapter's are other tokens', in columns that are not read
      const bool run = order[p0 + rows - 1] - order[p0] == (int)rows - 1;
      for (uint32_t kt = k0; kt < k1; ++kt, ++it) {
        ok = symm::mbar_wait_warp(&empty[st], ph, a.budget_ns, a.ctl);
        if (!ok) {
          if (elected) symm::record_error(a.ctl, symm::kErrTimedOut, -3);
          break;
        }
        uint8_t* buf = smem + (size_t)st * stage_bytes;
        if (elected) {
          symm::mbar_arrive_expect_tx(&full[st], a.rk_abytes + rows16 * 128);
          for (uint32_t half = 0; half * 8192 < a.rk_abytes; ++half)
            symm::tma_load_3d(buf + half * 8192, &map_a, (int)half * 64, (int)(kt * kBK), id,
                              &full[st]);
        }
        __syncwarp();
        if (run) {
          if (16 * lane < rows16)
            tma_load_2d(buf + a.rk_abytes + lane * 2048, &map_x16, (int)(kt * kBK),
                        order[p0] + 16 * lane, &full[st]);
        } else if (q < rows16)
          tma_gather4(buf + a.rk_abytes + q * 128, &map_x, (int)(kt * kBK), r, &full[st]);
        if (++st == stages) st = 0, ph ^= 1;
      }
    }
    for (uint32_t i = it > stages ? it - stages : 0; i < it; ++i)
      symm::mbar_wait(&full[i % stages], (i / stages) & 1, drain_ns(a));
  } else if (warp == 1) {  // -------------------------------- MMA issuer
    const bool elected = symm::elect_one();
    uint32_t st = 0, ph = 0;
    bool ok = true;
    for (uint32_t i = share, seg = 0; ok && i < items; i += a.rk_share, ++seg) {
      const uint32_t rows16 = (start[i + 1] - start[i] + 15) / 16 * 16, buf = seg & 1;
      ok = symm::mbar_wait_warp(&tempty[buf], ((seg >> 1) & 1) ^ 1u, a.budget_ns, a.ctl);
      const uint32_t idesc = mma_idesc(FMT, rows16);
      for (uint32_t kt = k0; ok && kt < k1; ++kt) {
        if (!(ok = symm::mbar_wait_warp(&full[st], ph, a.budget_ns, a.ctl))) break;
        symm::tc_fence_after();
        const uint8_t* tile = smem + (size_t)st * stage_bytes;
        const uint64_t wd = symm::sw128_mnmajor_desc(tile);
        const uint64_t xd = symm::sw128_kmajor_desc(tile + a.rk_abytes);
        if (elected) {
#pragma unroll
          for (int j = 0; j < kBK / 16; ++j)
            symm::tc_mma(tmem + buf * 128, wd + kWStep * j, xd + kXStep * j, idesc,
                         kt != k0 || j != 0);
          symm::tc_commit(&empty[st]);
        }
        if (++st == stages) st = 0, ph ^= 1;
      }
      if (ok && elected) symm::tc_commit(&tfull[buf]);
    }
    if (!ok && elected) symm::record_error(a.ctl, symm::kErrTimedOut, -5);
    if (elected) symm::tc_commit(&drain);
    symm::mbar_wait(&drain, 0, drain_ns(a));
  } else {  // ------------------------------------------- sums of this part
    const uint32_t q = (uint32_t)(warp & 3), row = 32 * q + lane;
    for (uint32_t p = threadIdx.x - 64; p < kRankTokens; p += 128)
      scales[p] = sorted[p] < a.R ? a.scale[sorted[p]] : 0.f;
    // B of these adapters on its way into L2, for the second launch
    for (uint32_t i = share; i < items; i += a.rk_share)
      for (uint32_t n0 = ((threadIdx.x - 64) * csize + crank) * 64; n0 < a.n;
           n0 += 128 * csize * 64)
        for (uint32_t r0 = 0; r0 < a.r; r0 += piece_rows(a.r16))
          prefetch_3d(&map_b, (int)n0, (int)r0, (int)sorted[start[i]]);
    for (uint32_t i = share, seg = 0; i < items; i += a.rk_share, ++seg) {
      const uint32_t p0 = start[i], rows = start[i + 1] - p0, buf = seg & 1;
      // a warp gives up as one: tcgen05.ld wants all its lanes
      if (!symm::mbar_wait_warp(&tfull[buf], (seg >> 1) & 1, a.budget_ns, a.ctl)) {
        symm::record_error(a.ctl, symm::kErrTimedOut, -6);
        break;
      }
      symm::tc_fence_after();
      if (32 * q < a.r)  // the warp's TMEM lanes hold ranks
        for (uint32_t c = 0; c < rows; c += 16) {
          uint32_t v[16];
          symm::tmem_ld16(tmem + ((32 * q) << 16) + buf * 128 + c, v);
          if (row < a.r)
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (c + j < rows) sums[(p0 + c + j) * a.r + row] = __uint_as_float(v[j]);
        }
      symm::tc_fence_before();
      symm::mbar_arrive(&tempty[buf]);
    }
  }
  __syncwarp();
  symm::tc_fence_before();
  cluster_sync();  // every CTA's sums are complete
  if (warp == 5) {
    symm::tc_fence_after();
    symm::tmem_dealloc(tmem, 256);
  }
  // each CTA of the cluster joins its share of the sums, CTAs in order
  __nv_bfloat16* H = reinterpret_cast<__nv_bfloat16*>(a.h);
  for (uint32_t item = share; item < items; item += a.rk_share) {
    const uint32_t p0 = start[item], n = (start[item + 1] - p0) * a.r16;
    for (uint32_t i = crank * kThreads + threadIdx.x; i < n; i += csize * kThreads) {
      const uint32_t pos = p0 + i / a.r16, c = i % a.r16;
      float s = 0.f;
      if (c < a.r) {
        const uint32_t at = symm::smem_addr(&sums[pos * a.r + c]);
        float v[8];
#pragma unroll
        for (uint32_t b = 0; b < 8; ++b) v[b] = b < csize ? ld_cluster(map_cluster(at, b)) : 0.f;
#pragma unroll
        for (uint32_t b = 0; b < 8; ++b) s += v[b];
        s *= scales[pos];
      }
      // three parts of 8 bits, truncated; an infinity or NaN is all in the first
      // (what it leaves would be NaN)
      __nv_bfloat16* out =
          H + (size_t)order[pos] * kParts * a.r16 + c / 16 * (kParts * 16) + c % 16;
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        const __nv_bfloat16 part = __float2bfloat16_rz(s);
        out[16 * i] = part;
        s = isfinite(s) ? s - moe::to_f(part) : 0.f;
      }
    }
  }
  cluster_leave();  // no CTA leaves while another reads its sums
}

// The larger magnitudes of 8 values and `most`, in both halves as they are; and
// whether one of such a pair is an infinity or NaN.
__device__ __forceinline__ uint32_t magnitudes(uint32_t most, const uint4& x) {
  const uint32_t m = 0x7fff7fffu;
  return __vmaxu2(__vmaxu2(most, __vmaxu2(x.x & m, x.y & m)), __vmaxu2(x.z & m, x.w & m));
}
template <int FMT>
__device__ __forceinline__ bool not_finite(uint32_t most) {
  constexpr uint32_t kInf = FMT ? 0x7f80u : 0x7c00u;
  return (most & 0xffffu) >= kInf || (most >> 16) >= kInf;
}
// 8 fp16 values as the sums of two bf16 values: the upper 8 of their 11 bits,
// truncated (the upper half of the float), and the rest.
__device__ __forceinline__ void two_parts(const uint4& x, uint4& hi, uint4& lo) {
  const uint32_t in[4] = {x.x, x.y, x.z, x.w};
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(in + i));
    const uint32_t u = __float_as_uint(f.x), v = __float_as_uint(f.y);
    const float g = f.x - __uint_as_float(u & 0xffff0000u);
    const float k = f.y - __uint_as_float(v & 0xffff0000u);
    h[i] = __byte_perm(u, v, 0x7632);
    l[i] = __byte_perm(__float_as_uint(g), __float_as_uint(k), 0x7632);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}
// 8 bf16 values, 0 in the place of infinities and NaN.
__device__ __forceinline__ uint4 only_finite(uint4 x) {
  uint32_t* w = &x.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((w[i] & 0x7f80u) == 0x7f80u) w[i] &= 0xffff0000u;
    if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] &= 0xffffu;
  }
  return x;
}
// What token t's infinities and NaN in h add to column n (fp16 inputs).
__device__ __noinline__ float wild_sum(const AdapterArgs& a, uint32_t t, uint32_t id, uint32_t n) {
  const __half* b = static_cast<const __half*>(a.b) + (size_t)id * a.r * a.n + n;
  const uint16_t* h = a.h + (size_t)t * kParts * a.r16;
  float s = 0.f;
  for (uint32_t r = 0; r < a.r; ++r) {
    const float v = __uint_as_float((uint32_t)h[r / 16 * (kParts * 16) + r % 16] << 16);
    if (!isfinite(v)) s += v * __half2float(b[(size_t)r * a.n]);
  }
  return s;
}
// Whether p holds in any of the 128 threads of the epilogue (a barrier of theirs).
__device__ __forceinline__ bool any_of(bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)p)
      : "memory");
  return r != 0;
}

// Stores 16 tokens from t0 on, column n.
template <int FMT>
__device__ __forceinline__ void store16(const AdapterArgs& a, const float (&acc)[16], uint32_t t0,
                                        uint32_t n) {
  using T = typename Elem<FMT>::T;
  if (n >= a.n) return;
  T* y = static_cast<T*>(a.y) + (size_t)t0 * a.ldy + n;
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (t0 + j < a.T) y[(size_t)j * a.ldy] = moe::from_f<T>(acc[j]);
}

template <int FMT>
__global__ void __launch_bounds__(kThreads, 1)
    adapter_kernel(const __grid_constant__ CUtensorMap map_w,
                   const __grid_constant__ CUtensorMap map_x,
                   const __grid_constant__ CUtensorMap map_b, const AdapterArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (symm::smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t abytes = a.deep * kATile, xbytes = a.bt * 128;
  const uint32_t stage_bytes = abytes + a.deep * xbytes;
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], claimed[kMaxStages];
  __shared__ uint64_t tfull[2], tempty[2], listed[2], drain;
  __shared__ uint32_t tmem_slot;
  // the ids of a tile's tokens, and the adapters among them (how many, which);
  // two tiles' worth, as the accumulators
  __shared__ __align__(16) uint32_t id_of[256];
  __shared__ uint32_t firsts[8], list[2][256], nlist[2];
  // a B tile that is not finite: whose tokens (by token), left out (by stage)
  __shared__ uint8_t spoilt[256], leave_out[kMaxStages];
  // fp16 inputs: tokens with an h that is not finite, whether there are any
  __shared__ uint8_t wild[256];
  __shared__ uint32_t any_wild;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < a.stages; ++s) {
      symm::mbar_init(&full[s], 2);  // the producer, and it again or who wrote h
      symm::mbar_init(&empty[s], 1);
      symm::mbar_init(&claimed[s], 1);  // B is there, and h may be written
    }
    for (int b = 0; b < 2; ++b) {
      symm::mbar_init(&tfull[b], 1);
      symm::mbar_init(&tempty[b], 128);
      symm::mbar_init(&listed[b], 1);
    }
    symm::mbar_init(&drain, 1);
    symm::fence_mbar_init();
  }
  if (warp == 1) symm::tmem_alloc(&tmem_slot, a.tmem_cols);
  symm::tc_fence_before();
  __syncthreads();
  symm::tc_fence_after();
  const uint32_t tmem = tmem_slot;
  float* sums = reinterpret_cast<float*>(smem);  // [bt][128], in a cluster of several CTAs
  const uint32_t npieces = a.R ? pieces_of(a) : 0;
  // This CTA's tiles, and its part of their K slices and adapters.
  const uint32_t C = a.cluster, crank = C > 1 ? cluster_rank() : 0;
  const uint32_t tiles = a.ncol * a.ntok, first = blockIdx.x / C, step = gridDim.x / C;
  const uint32_t k0 = a.slices * crank / C, k1 = a.slices * (crank + 1) / C;
  // The adapters come before the last ring's worth of a long part of K, where
  // the first launch is done and their loads hide behind W's; else at the end.
  const uint32_t kp = k1 - k0 > 4 * a.stages ? k1 - a.stages : k1;

  if (warp == 0) {  // ----------------------------------------- TMA producer
    const bool elected = symm::elect_one();
    uint32_t st = 0, ph = 1, it = 0;
    uint32_t is_b = 0, b_phases = ~0u;  // stages whose last load is B's, phases of `claimed`
    bool ok = true;
    auto next = [&](bool b) {
      is_b = (is_b & ~(1u << st)) | ((uint32_t)b << st);
      b_phases ^= (uint32_t)b << st;
      ++it;
      if (++st == a.stages) st = 0, ph ^= 1;
    };
    for (uint32_t tile = first, seg = 0; ok && tile < tiles; tile += step, ++seg) {
      const int n0 = (int)(tile % a.ncol) * kBM;
      const uint32_t tb = tile / a.ncol;
      auto load_slices = [&](uint32_t from, uint32_t to) {
        for (uint32_t kt = from; ok && kt < to; ++kt) {
          if (!(ok = symm::mbar_wait_warp(&empty[st], ph, a.budget_ns, a.ctl))) break;
          uint8_t* buf = smem + (size_t)st * stage_bytes;
          if (elected) {
            symm::mbar_arrive_expect_tx(&full[st], stage_bytes);
            const int k = (int)(kt * a.deep * kBK);
            tma_load_2d(buf, &map_w, n0, k, &full[st]);
            tma_load_2d(buf + abytes / 2, &map_w, n0 + 64, k, &full[st]);
            tma_load_2d(buf + abytes, &map_x, k, (int)(tb * a.bt), &full[st]);
            if (a.deep == 2)
              tma_load_2d(buf + abytes + xbytes, &map_x, k + kBK, (int)(tb * a.bt), &full[st]);
            symm::mbar_arrive(&full[st]);
          }
          next(false);
        }
      };
      load_slices(k0, kp);
      if (ok && npieces) {
        const uint32_t lb = seg & 1;
        ok = symm::mbar_wait_warp(&listed[lb], (seg >> 1) & 1, a.budget_ns, a.ctl);
        const uint32_t f0 = nlist[lb] * crank / C, f1 = nlist[lb] * (crank + 1) / C;
        for (uint32_t p = 0; ok && p < npieces; ++p)
          for (uint32_t i = f0; i < f1; ++i) {
            if (!(ok = symm::mbar_wait_warp(&empty[st], ph, a.budget_ns, a.ctl))) break;
            uint8_t* buf = smem + (size_t)st * stage_bytes;
            const int id = (int)list[lb][i], row = (int)piece_rank(p);
            if (elected) {
              symm::mbar_arrive_expect_tx(&claimed[st], 256 * piece_rows(a.r16));
              symm::tma_load_3d(buf, &map_b, n0, row, id, &claimed[st]);
              symm::tma_load_3d(buf + abytes / 2, &map_b, n0 + 64, row, id, &claimed[st]);
              symm::mbar_arrive(&full[st]);
            }
            next(true);
          }
      }
      load_slices(kp, k1);
    }
    if (!ok && elected) symm::record_error(a.ctl, symm::kErrTimedOut, -3);
    // every load issued lands before the CTA may leave (bounded): of B on
    // `claimed` (nobody may be left to complete `full`), else on `full`
    for (uint32_t i = it > a.stages ? it - a.stages : 0; i < it; ++i) {
      const uint32_t s = i % a.stages;
      if ((is_b >> s) & 1) symm::mbar_wait(&claimed[s], (b_phases >> s) & 1, drain_ns(a));
      else symm::mbar_wait(&full[s], (i / a.stages) & 1, drain_ns(a));
    }
  } else if (warp == 1) {  // ---------------------------------- MMA issuer
    const bool elected = symm::elect_one();
    const uint32_t idesc = mma_idesc(FMT, a.bt), bf16_idesc = mma_idesc(1, a.bt);
    uint32_t st = 0, ph = 0, seg = 0;
    bool ok = true;
    auto next = [&]() {
      if (++st == a.stages) st = 0, ph ^= 1;
    };
    for (uint32_t tile = first; ok && tile < tiles; tile += step, ++seg) {
      const uint32_t buf = seg & 1;
      ok = symm::mbar_wait_warp(&tempty[buf], ((seg >> 1) & 1) ^ 1u, a.budget_ns, a.ctl);
      symm::tc_fence_after();
      const uint32_t acc = tmem + buf * a.bt;
      auto multiply = [&](uint32_t from, uint32_t to) {
        for (uint32_t kt = from; ok && kt < to; ++kt) {
          if (!(ok = symm::mbar_wait_warp(&full[st], ph, a.budget_ns, a.ctl))) break;
          symm::tc_fence_after();
          const uint8_t* ring = smem + (size_t)st * stage_bytes;
          const uint64_t wd = symm::sw128_mnmajor_desc(ring, abytes / 2);
          const uint64_t xd = symm::sw128_kmajor_desc(ring + abytes);
          if (elected) {
#pragma unroll
            for (int j = 0; j < kBK / 16; ++j)
              symm::tc_mma(acc, wd + kWStep * j, xd + kXStep * j, idesc, kt != k0 || j != 0);
            if (a.deep == 2)
#pragma unroll
              for (int j = 0; j < kBK / 16; ++j)
                symm::tc_mma(acc, wd + kWStep * (kBK / 16 + j), xd + (xbytes >> 4) + kXStep * j,
                             idesc, 1);
            symm::tc_commit(&empty[st]);
          }
          next();
        }
      };
      multiply(k0, kp);
      if (ok && npieces) {
        ok = symm::mbar_wait_warp(&listed[buf], (seg >> 1) & 1, a.budget_ns, a.ctl);
        const uint32_t mine = nlist[buf] * (crank + 1) / C - nlist[buf] * crank / C;
        for (uint32_t p = 0; ok && p < npieces; ++p) {
          const uint32_t steps = piece_steps(a, p);
          for (uint32_t i = 0; i < mine; ++i) {
            if (!(ok = symm::mbar_wait_warp(&full[st], ph, a.budget_ns, a.ctl))) break;
            symm::tc_fence_after();
            const uint8_t* ring = smem + (size_t)st * stage_bytes;
            const uint64_t wd = symm::sw128_mnmajor_desc(ring, abytes / 2);
            const uint64_t xd = symm::sw128_kmajor_desc(ring + abytes);
            const uint32_t todo = leave_out[st] ? 0 : steps;
            if (elected) {
              for (uint32_t j = 0; j < todo; ++j) {
                const uint64_t b = wd + kWStep * ((4 * p + j) / kParts - 4 * p / kParts);
                symm::tc_mma(acc, b, xd + kXStep * j, bf16_idesc, 1);
                if (FMT == 0)
                  symm::tc_mma(acc, b + kWStep * (kLowRows / 16), xd + kXStep * j, bf16_idesc, 1);
              }
              symm::tc_commit(&empty[st]);
            }
            next();
          }
        }
      }
      multiply(kp, k1);
      if (ok && elected) symm::tc_commit(&tfull[buf]);
    }
    if (!ok && elected) symm::record_error(a.ctl, symm::kErrTimedOut, -5);
    if (elected) symm::tc_commit(&drain);  // every MMA is complete before TMEM is freed
    symm::mbar_wait(&drain, 0, drain_ns(a));
  } else {  // ------------------------------------------ h, and the epilogue
    const uint32_t q = (uint32_t)(warp & 3);  // TMEM lanes 32q .. 32q + 31
    const uint32_t row = 32 * q + lane;       // this thread's column of W in the tile
    const uint32_t me = threadIdx.x - 64;
    const uint32_t chunks = a.bt / 16;
    uint32_t it = 0;
    uint32_t phases = 0;  // of `claimed`, one bit per stage
    bool ok = true, waited = false, any_spoilt = false;
    for (uint32_t tile = first, seg = 0; ok && tile < tiles; tile += step, ++seg) {
      const uint32_t buf = seg & 1;
      const uint32_t n = (tile % a.ncol) * kBM + row, tb = tile / a.ncol, t0 = tb * a.bt;
      it += kp - k0;
      if (npieces) {
        // the tokens' adapters, each listed by its first token, in token order
        for (uint32_t i = me; i < 256; i += 128)
          id_of[i] = i < a.bt && t0 + i < a.T ? (uint32_t)a.ids[t0 + i] : 0xffffffffu;
        symm::group_sync(1, 128);
        any_spoilt = false;
        for (uint32_t i = me; i < 256; i += 128) spoilt[i] = wild[i] = 0;
        if (me == 0) any_wild = 0;
        for (uint32_t i = me; i < 256; i += 128) {
          const uint32_t id = id_of[i];
          const uint32_t same = __match_any_sync(0xffffffffu, id);  // by every lane of the warp
          bool seen = id >= a.R || (same & ((1u << lane) - 1)) != 0;
          for (uint32_t j = 0; j < (i & ~31u); j += 16) {  // the same for the warp's lanes
            if (__all_sync(0xffffffffu, seen)) break;
#pragma unroll
            for (uint32_t l = 0; l < 16; l += 4) {
              const uint4 v = *reinterpret_cast<const uint4*>(&id_of[j + l]);
              seen |= v.x == id || v.y == id || v.z == id || v.w == id;
            }
          }
          const uint32_t votes = __ballot_sync(0xffffffffu, !seen);
          if (lane == 0) firsts[i / 32] = votes;
        }
        symm::group_sync(1, 128);
        for (uint32_t i = me; i < 256; i += 128) {
          uint32_t before = __popc(firsts[i / 32] & ((1u << lane) - 1));
          for (uint32_t w = 0; w < i / 32; ++w) before += __popc(firsts[w]);
          if ((firsts[i / 32] >> lane) & 1) list[buf][before] = id_of[i];
          if (i == 255) nlist[buf] = before + (firsts[7] >> 31);
        }
        symm::group_sync(1, 128);
        if (me == 0) symm::mbar_arrive(&listed[buf]);
        if (!waited) moe::wait_for_earlier(), waited = true;  // for h
        const uint32_t f0 = nlist[buf] * crank / C, f1 = nlist[buf] * (crank + 1) / C;
        for (uint32_t p = 0; ok && f0 < f1 && p < npieces; ++p) {
          // This thread's 16-byte chunks of the piece (at most 16: bt 256, 8 chunks a
          // row) and the adapters of their tokens.  (The next piece's loaded ahead
          // cost up to a tenth: 248 registers.)
          const uint32_t width = 2 * piece_steps(a, p);
          const uint32_t wlog = 32 - __clz(width - 1);  // 2 to 8 chunks a row, in whole powers
          // whether no thread has chunk 4 or a later one (asked once: the others'
          // accesses are to be issued together)
          const bool few = (128u * 4) >> wlog >= a.bt;
          uint4 v[16];
          uint32_t id[16], at[16], most = 0, odd = 0;  // odd: not finite
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const uint32_t tr = (me + 128 * c) >> wlog, ch = me & ((1u << wlog) - 1);
            id[c] = at[c] = 0xffffffffu, v[c] = make_uint4(0, 0, 0, 0);
            if ((c >= 4 && few) || tr >= a.bt || ch >= width) continue;
            id[c] = id_of[tr];
            at[c] = tr * 128 + ((ch ^ (tr & 7)) << 4);
            if (id[c] < a.R)
              v[c] = __ldcg(reinterpret_cast<const uint4*>(
                                a.h + (size_t)(t0 + tr) * kParts * a.r16 + 64 * p) + ch);
          }
          if (FMT == 0)
#pragma unroll
            for (int c = 0; c < 16; ++c) most = magnitudes(most, v[c]);
          // B's second part may be 0: what is not finite is left to the epilogue
          if (FMT == 0 && not_finite<1>(most))
#pragma unroll
            for (int c = 0; c < 16; ++c)
              if (not_finite<1>(magnitudes(0, v[c]))) odd |= 1u << c, v[c] = only_finite(v[c]);
          for (uint32_t i = f0; i < f1; ++i, ++it) {
            const uint32_t st = it % a.stages;
            // not `empty`: whose phases this warp does not follow one by one.  A
            // wait that gives up takes every thread to the barrier below first.
            ok = symm::mbar_wait_warp(&claimed[st], (phases >> st) & 1, a.budget_ns, a.ctl);
            phases ^= 1u << st;
            uint8_t* ring = smem + (size_t)st * stage_bytes + abytes;
            // B's tile: two boxes of 64 columns, from the start of the stage
            most = 0;
            const uint32_t brows = piece_rows(a.r16);
            uint4 x[4];  // of 8 vectors a row and box, 16 or 32 rows
#pragma unroll
            for (uint32_t u = 0; u < 4; ++u) {
              uint4* box = reinterpret_cast<uint4*>(ring - abytes + (u & 1) * (abytes / 2));
              if (me + 128 * (u >> 1) < 8 * brows) x[u] = box[me + 128 * (u >> 1)];
            }
#pragma unroll
            for (uint32_t u = 0; u < 4; ++u) {
              if (me + 128 * (u >> 1) >= 8 * brows) continue;
              most = magnitudes(most, x[u]);
              uint4* box = reinterpret_cast<uint4*>(ring - abytes + (u & 1) * (abytes / 2));
              if (FMT == 0)
                two_parts(x[u], box[me + 128 * (u >> 1)], box[me + 128 * (u >> 1) + kLowRows * 8]);
            }
            const uint32_t want = list[buf][i];
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              if (c == 4 && few) break;
              if (at[c] != 0xffffffffu)
                *reinterpret_cast<uint4*>(ring + at[c]) =
                    id[c] == want ? v[c] : make_uint4(0, 0, 0, 0);
            }
            if (FMT == 0 && odd)
#pragma unroll
              for (int c = 0; c < 16; ++c)
                if (((odd >> c) & 1) && id[c] == want)
                  wild[(me + 128 * c) >> wlog] = 1, any_wild = 1;
            symm::fence_proxy_async_shared();  // h (and B's parts), for the MMAs
            const bool bad = any_of(!ok || not_finite<FMT>(most));
            if (bad) {
              if (any_of(!ok)) {
                if (me == 0) symm::record_error(a.ctl, symm::kErrTimedOut, -7);
                ok = false;
                break;
              }
              any_spoilt = true;
              for (uint32_t c = me; c < 256; c += 128)
                if (id_of[c] == want) spoilt[c] = 1;
              symm::group_sync(1, 128);
            }
            if (me == 0) {
              leave_out[st] = bad;
              symm::mbar_arrive(&full[st]);
            }
          }
        }
        if (!ok) break;
      }
      it += k1 - kp;
      ok = symm::mbar_wait_warp(&tfull[buf], (seg >> 1) & 1, a.budget_ns, a.ctl);
      if (any_of(!ok)) {  // all threads leave, or none
        if (me == 0) symm::record_error(a.ctl, symm::kErrTimedOut, -6);
        ok = false;
        break;
      }
      symm::tc_fence_after();
      const uint32_t taddr = tmem + ((32 * q) << 16) + buf * a.bt;
#pragma unroll 1
      for (uint32_t c = 0; c < chunks; ++c) {
        uint32_t v[16];
        symm::tmem_ld16(taddr + c * 16, v);
        if (c + 1 == chunks) {  // the accumulator is free for the next tile
          symm::tc_fence_before();
          symm::mbar_arrive(&tempty[buf]);
        }
        float acc[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[j] = __uint_as_float(v[j]);
        if (any_spoilt)
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (spoilt[c * 16 + j]) acc[j] = __uint_as_float(0x7fffffffu);
        if (FMT == 0 && npieces && any_wild)
#pragma unroll 1
          for (int j = 0; j < 16; ++j)
            if (wild[c * 16 + j]) {
              const float more = wild_sum(a, t0 + c * 16 + j, id_of[c * 16 + j], min(n, a.n - 1));
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (i == j) acc[i] += more;
              __syncwarp();
            }
        if (C == 1) {
          if (t0 + c * 16 < a.T) store16<FMT>(a, acc, t0 + c * 16, n);
        } else {  // the ring's loads have all been consumed: its memory takes the sums
#pragma unroll
          for (int j = 0; j < 16; ++j) sums[(c * 16 + j) * kBM + row] = acc[j];
        }
      }
    }
  }

  __syncwarp();
  symm::tc_fence_before();
  if (C > 1) {
    cluster_sync();  // every CTA's sums are complete
    // this CTA's share of the tokens; a warp takes a token's 128 columns, 4 a lane
    using T = typename Elem<FMT>::T;
    const uint32_t tb = first / a.ncol, n = first % a.ncol * kBM + 4 * lane;
    const uint32_t c1 = min(a.bt * (crank + 1) / C, a.T - tb * a.bt);
    for (uint32_t c = a.bt * crank / C + warp; c < c1; c += kThreads / 32) {
      const uint32_t at = symm::smem_addr(sums + c * kBM + 4 * lane);
      float4 v[8];
#pragma unroll
      for (uint32_t b = 0; b < 8; ++b)
        if (b < C) v[b] = ld_cluster4(map_cluster(at, b));
      float4 s = v[0];
#pragma unroll
      for (uint32_t b = 1; b < 8; ++b)
        if (b < C) s.x += v[b].x, s.y += v[b].y, s.z += v[b].z, s.w += v[b].w;
      T* y = static_cast<T*>(a.y) + (size_t)(tb * a.bt + c) * a.ldy + n;
      if (n + 0 < a.n) y[0] = moe::from_f<T>(s.x);
      if (n + 1 < a.n) y[1] = moe::from_f<T>(s.y);
      if (n + 2 < a.n) y[2] = moe::from_f<T>(s.z);
      if (n + 3 < a.n) y[3] = moe::from_f<T>(s.w);
    }
    cluster_leave();  // no CTA leaves while another reads its sums
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    symm::tc_fence_after();
    symm::tmem_dealloc(tmem, a.tmem_cols);
  }
}

// How a call of these sizes is cut up.
struct Plan {
  uint32_t bt, ntok, ncol, ktiles, deep, slices, stages, cluster, ctas, tmem_cols, r16;
  uint32_t rk_share, rk_cluster, rk_blocks, rk_ring, rk_abytes, rk_bytes;
};

size_t up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// Clusters of c CTAs of the product that are resident at once, asked once for
// each device.
int resident_clusters(int fmt, uint32_t c);

// Tokens per tile and CTAs per tile: the pair with the least estimated time,
// fitted to measured times.  A 64-deep K slice costs its loads, 16 KB of W and
// 128 bytes a token at about 125 bytes a ns per SM, or what the roles need to
// issue it; a round of tiles costs 2 us (filling the ring, the epilogue), and
// sharing a tile 2 us and 5 ns a token.
void choose_tiles(Plan& p, uint32_t T, int fmt) {
  double best = 0;
  for (uint32_t blocks = (T + 255) / 256, i = 0; i < 8; ++i, ++blocks) {
    const uint32_t bt = (uint32_t)up((T + blocks - 1) / blocks, 16);
    const uint32_t ntok = (T + bt - 1) / bt;
    const uint64_t tiles = (uint64_t)p.ncol * ntok;
    const double slice = 131 + 1.02 * bt;
    for (uint32_t c = 1; c <= 8 && c <= (p.ktiles + 1) / 2; ++c) {
      const uint64_t room = (uint64_t)std::max(1, resident_clusters(fmt, c));
      const uint64_t rounds = (tiles + room - 1) / room;
      const double per = (double)((p.ktiles + c - 1) / c) * slice;
      const double t = c == 1 ? rounds * per + 2000 + 500 * (rounds - 1)
                              : rounds * (per + 4000 + 5.0 * bt);
      if (best == 0 || t < best) best = t, p.bt = bt, p.ntok = ntok, p.cluster = c;
    }
    if (bt == 16) break;
  }
}

Plan plan_of(int T, int k, int n, int r, int fmt) {
  Plan p{};
  const uint32_t sms = (uint32_t)std::max(sm_count(), 1);
  p.ncol = ((uint32_t)n + kBM - 1) / kBM;
  p.ktiles = ((uint32_t)k + kBK - 1) / kBK;
  choose_tiles(p, (uint32_t)T, fmt);
  p.deep = p.bt <= 64 ? 2 : 1;
  p.slices = (p.ktiles + p.deep - 1) / p.deep;
  p.stages = std::min<uint32_t>(kMaxStages, kRingBytes / (p.deep * (kATile + p.bt * 128)));
  const uint32_t tiles = p.ncol * p.ntok;
  p.ctas = p.cluster > 1 ? tiles * p.cluster : std::min(sms, tiles);
  p.tmem_cols = 32;
  while (p.tmem_cols < 2 * p.bt) p.tmem_cols *= 2;
  p.r16 = (uint32_t)up((size_t)r, 16);
  // The first launch: clusters of up to 8 CTAs share the K slices of a block of
  // 128 tokens; about two CTAs per SM in all.
  const uint32_t blocks = ((uint32_t)T + kRankTokens - 1) / kRankTokens;
  p.rk_blocks = blocks;
  p.rk_cluster = 8;
  while (p.rk_cluster > 1 && (p.rk_cluster > p.ktiles || blocks * p.rk_cluster > 2 * sms))
    p.rk_cluster /= 2;
  p.rk_share = std::max(1u, std::min(std::min((uint32_t)T, (uint32_t)kRankTokens),
                                     2 * sms / (blocks * p.rk_cluster)));
  p.rk_abytes = r <= 64 ? 8192 : 16384;
  // two CTAs per SM while their sums leave room for it; two stages at the least
  const uint32_t sums = std::min<uint32_t>(kRankTokens, (uint32_t)T) * (uint32_t)r * 4;
  p.rk_ring = (kRankBytes - std::min(sums, 32768u)) / 1024 * 1024;
  p.rk_bytes = 1024 + p.rk_ring + 8192 + sums;
  return p;
}

// Workspace: h.
size_t h_bytes(int T, int r) { return up((size_t)T * kParts * up((size_t)r, 16) * 2, 256); }

int check_adapter(const char* what, int T, int k, int n, int r) {
  if (T < 0 || T > (1 << 24) || k < 8 || n < 8 || k % 8 || n % 8 || k > (1 << 20) ||
      n > (1 << 20))
    return fail(SYMM_EINVAL, std::string(what) + ": T must be in [0, 2^24], k and n multiples of "
                                                 "8 (16-byte rows) in [8, 2^20]");
  if (r < 0 || r > SYMM_MOE_MAX_RANK || r % 8)
    return fail(SYMM_EINVAL, std::string(what) + ": r must be a multiple of 8 up to 128");
  return SYMM_OK;
}

// [depth][rows][inner] 2-byte elements, rows `ld` and planes ld * rows apart,
// boxes of 64 x box_rows, 128-byte swizzled; depth 0: a 2-d map.
int make_map(CUtensorMap* map, const void* base, int fmt, uint64_t inner, uint64_t rows,
             uint64_t depth, size_t ld, uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return fail(SYMM_ECUDA, "moe_adapter_matmul: no cuTensorMapEncodeTiled");
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
                "moe_adapter_matmul: tensor map rejected (CUresult " + std::to_string(r) + ")");
  return SYMM_OK;
}

struct Maps {
  CUtensorMap w, x, a, rows, rows16, b;
};

constexpr size_t kRankSmemMax =
    1024 + kRankBytes + 8192 + (size_t)kRankTokens * SYMM_MOE_MAX_RANK * 4;

// Once per device: both kernels may use more than 48 KB of shared memory.
template <int FMT>
int set_up() {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  int rc = cuda_check(cudaGetDevice(&dev), "moe_adapter_matmul: device");
  if (rc) return rc;
  std::lock_guard<std::mutex> lock(mu);
  if (dev >= 0 && dev < 64 && done[dev]) return SYMM_OK;
  auto set = [&](const void* f, cudaFuncAttribute attr, int v) {
    if (!rc) rc = cuda_check(cudaFuncSetAttribute(f, attr, v), "moe_adapter_matmul: kernel set-up");
  };
  const void *product = (const void*)adapter_kernel<FMT>, *ranks = (const void*)rank_kernel<FMT>;
  set(product, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(1024 + kRingBytes));
  set(ranks, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRankSmemMax);
  // the same split of an SM's memory for both: changing it would wait for an idle SM
  set(product, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  set(ranks, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (!rc && dev >= 0 && dev < 64) done[dev] = true;
  return rc;
}

int resident_clusters(int fmt, uint32_t c) {
  static std::mutex mu;
  static int known[2][64][9] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  std::lock_guard<std::mutex> lock(mu);
  int& n = known[fmt][dev][c];
  if (n) return n;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = c;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(c);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 1024 + kRingBytes;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = fmt ? cudaOccupancyMaxActiveClusters(&n, adapter_kernel<1>, &cfg)
                            : cudaOccupancyMaxActiveClusters(&n, adapter_kernel<0>, &cfg);
  if (e != cudaSuccess || n < 1) {
    cudaGetLastError();
    n = 0;
    return std::max(1, sm_count() / (int)c / 2);  // a guess, not kept
  }
  return n;
}

template <int FMT>
int launch(const Plan& p, const Maps& m, const AdapterArgs& a, cudaStream_t s) {
  int rc = SYMM_OK;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  if (a.R) {
    cfg.gridDim = dim3(p.rk_blocks * p.rk_share * p.rk_cluster);
    cfg.dynamicSmemBytes = p.rk_bytes;
    attr[0].val.clusterDim.x = p.rk_cluster;
    cfg.numAttrs = 2;
    rc = cuda_check(cudaLaunchKernelEx(&cfg, rank_kernel<FMT>, m.a, m.rows, m.rows16, m.b, a),
                    "moe_adapter_matmul: rank products");
    if (rc) return rc;
  }
  cfg.gridDim = dim3(p.ctas);
  cfg.dynamicSmemBytes = 1024 + kRingBytes;
  attr[0].val.clusterDim.x = p.cluster;
  cfg.numAttrs = a.R ? 2 : 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, adapter_kernel<FMT>, m.w, m.x, m.b, a),
                    "moe_adapter_matmul: product");
}

}  // namespace

extern "C" int moe_adapter_workspace(int T, int k, int n, int r, size_t* bytes) {
  return moe::entry("moe_adapter_workspace", [&]() -> int {
    if (!bytes) return fail(SYMM_EINVAL, "moe_adapter_workspace: NULL bytes");
    int rc = check_adapter("moe_adapter_workspace", T, k, n, r);
    if (rc) return rc;
    *bytes = h_bytes(T, r);
    return SYMM_OK;
  });
}

extern "C" int moe_adapter_matmul(symm_heap_t* heap, const void* x, size_t ldx, const void* w,
                                  size_t ldw, const void* a, const void* b, const float* scale,
                                  const int32_t* ids, int dtype, int T, int k, int n, int R, int r,
                                  void* y, size_t ldy, void* workspace, void* stream) {
  return moe::entry("moe_adapter_matmul", [&]() -> int {
    const char* what = "moe_adapter_matmul";
    if (!heap) return fail(SYMM_EINVAL, "moe_adapter_matmul: NULL heap");
    if (dtype != SYMM_DTYPE_F16 && dtype != SYMM_DTYPE_BF16)
      return fail(SYMM_EINVAL, "moe_adapter_matmul: dtype must be SYMM_DTYPE_F16 or _BF16");
    int rc = check_adapter(what, T, k, n, r);
    if (rc) return rc;
    if (R < 0 || (R > 0) != (r > 0))
      return fail(SYMM_EINVAL, "moe_adapter_matmul: R must be >= 0, and r 0 exactly when R is");
    if (ldx < (size_t)k || ldw < (size_t)n || ldy < (size_t)n || ldx % 8 || ldw % 8 ||
        ldx > (1ull << 36) || ldw > (1ull << 36) || ldy > (1ull << 36))
      return fail(SYMM_EINVAL, "moe_adapter_matmul: ldx >= k, ldw >= n (multiples of 8), ldy >= n");
    if (T == 0) return SYMM_OK;
    if (!x || !w || !y || (R && !workspace) || (R && (!a || !b || !scale || !ids)))
      return fail(SYMM_EINVAL, "moe_adapter_matmul: NULL input, output or workspace");
    if (!moe::aligned(x, 16) || !moe::aligned(w, 16) || !moe::aligned(a, 16) ||
        !moe::aligned(b, 16) || !moe::aligned(y, 2) || !moe::aligned(scale, 4) ||
        !moe::aligned(ids, 4) || !moe::aligned(workspace, 256))
      return fail(SYMM_EINVAL, "moe_adapter_matmul: x, w, a and b must be 16-byte aligned, "
                               "workspace 256-byte aligned, the rest to their elements");
    if (y == x || y == w || y == a || y == b)
      return fail(SYMM_EINVAL, "moe_adapter_matmul: y must not be an input");
    const int fmt = dtype == SYMM_DTYPE_BF16 ? 1 : 0;
    rc = fmt ? set_up<1>() : set_up<0>();
    if (rc) return rc;
    const Plan p = plan_of(T, k, n, r, fmt);
    Maps m{};
    rc = make_map(&m.w, w, fmt, (uint64_t)n, (uint64_t)k, 0, ldw, p.deep * kBK);
    if (!rc) rc = make_map(&m.x, x, fmt, (uint64_t)k, (uint64_t)T, 0, ldx, p.bt);
    if (!rc && R) {
      rc = make_map(&m.a, a, fmt, (uint64_t)r, (uint64_t)k, (uint64_t)R, (size_t)r, kBK);
      if (!rc) rc = make_map(&m.rows, x, fmt, (uint64_t)k, (uint64_t)T, 0, ldx, 1);
      if (!rc) rc = make_map(&m.rows16, x, fmt, (uint64_t)k, (uint64_t)T, 0, ldx, 16);
      if (!rc)
        rc = make_map(&m.b, b, fmt, (uint64_t)n, (uint64_t)r, (uint64_t)R, (size_t)n,
                      piece_rows(p.r16));
    }
    if (rc) return rc;
    cudaStream_t s = as_stream(stream);
    rc = ensure_ctrl(heap, s);
    if (rc) return rc;
    AdapterArgs g{};
    g.scale = scale, g.ids = ids, g.b = b, g.y = y, g.ldy = ldy;
    g.T = (uint32_t)T, g.k = (uint32_t)k, g.n = (uint32_t)n, g.R = (uint32_t)R, g.r = (uint32_t)r;
    g.r16 = p.r16, g.bt = p.bt, g.ntok = p.ntok, g.ncol = p.ncol, g.ktiles = p.ktiles;
    g.deep = p.deep, g.slices = p.slices;
    g.stages = p.stages, g.cluster = p.cluster, g.tmem_cols = p.tmem_cols;
    g.h = static_cast<uint16_t*>(workspace);
    g.rk_share = p.rk_share, g.rk_ring = p.rk_ring, g.rk_abytes = p.rk_abytes;
    g.budget_ns = heap->spin_budget;
    g.ctl = reinterpret_cast<Control*>(heap->base);
    return fmt ? launch<1>(p, m, g, s) : launch<0>(p, m, g, s);
  });
}
