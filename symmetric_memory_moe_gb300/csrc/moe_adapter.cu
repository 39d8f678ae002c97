// moe_adapter.cu -- a projection shared by all requests with one low-rank
// adapter per request: y_t = x_t W + scale_a (x_t A_a) B_a, a = ids_t.
//
// Two launches.  The first computes h_t = scale_a x_t A_a in 32 bits (rank r
// values per token).  The second is the product with W on the tensor cores,
// with h_t B_a added to the 32-bit accumulators before the one rounding, so
// any mixture of adapters in any order of tokens costs the large product
// nothing.
//
// The product is computed as y^T = W^T x^T: the M side of a tile is 128
// columns of W (W as stored, k x n, is an M-major operand) and the N side BT
// tokens, 16 to 256.  One token then wastes no more than a narrow N, one
// kernel serves a decoding step and a prompt, and in the epilogue a warp's 32
// lanes hold 32 columns of one token: its adapter is the same in all lanes.
//   warp 0     TMA producer: 64-deep K slices of W (two boxes of 64 columns)
//              and of x into a ring of shared-memory stages, 128-byte swizzled;
//   warp 1     MMA issuer: tcgen05.mma kind::f16, M 128, N BT, two
//              accumulators in TMEM;
//   warps 2-5  epilogue: tcgen05.ld, the adapters' part, rounding, stores.
// Tiles that fill the GPU's SMs well are dealt out whole; otherwise the K
// slices of all tiles form one sequence cut into equal parts, one per CTA,
// and a tile that several CTAs share is summed, in the CTAs' order, by the
// last of them to arrive (no CTA waits for another).  Every wait is bounded;
// a role that gives up records the error in the heap's header.
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
constexpr uint32_t kRingBytes = 200 * 1024;
constexpr int kShrinkThreads = 256;

struct AdapterArgs {
  const void* x;
  size_t ldx;
  const void *a, *b;
  const float* scale;
  const int32_t* ids;
  void* y;
  size_t ldy;
  uint32_t T, k, n, R, r;
  uint32_t bt, ntok, ncol, ktiles, stages;  // tiles: ncol column blocks x ntok token blocks
  uint32_t split, tmem_cols;
  float* h;            // [T][r]
  float* part;         // [CTAs][2][bt][128]
  uint32_t* arrived;   // [tiles], zeroed by the first launch
  uint64_t budget_ns;
  Control* ctl;
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

// The segments of one CTA: K slices [k0, k1) of a tile.
struct Segment {
  uint32_t tile, k0, k1;
};
__device__ __forceinline__ uint64_t cut(const AdapterArgs& a, uint32_t cta) {
  return (uint64_t)a.ncol * a.ntok * a.ktiles * cta / gridDim.x;
}
struct Walk {
  uint64_t at, end;  // slices (split) or tiles (whole)
  __device__ __forceinline__ explicit Walk(const AdapterArgs& a)
      : at(a.split ? cut(a, blockIdx.x) : blockIdx.x),
        end(a.split ? cut(a, blockIdx.x + 1) : (uint64_t)a.ncol * a.ntok) {}
  __device__ __forceinline__ bool next(const AdapterArgs& a, Segment& s) {
    if (at >= end) return false;
    if (!a.split) {
      s = {(uint32_t)at, 0, a.ktiles};
      at += gridDim.x;
      return true;
    }
    s.tile = (uint32_t)(at / a.ktiles);
    s.k0 = (uint32_t)(at - (uint64_t)s.tile * a.ktiles);
    s.k1 = (uint32_t)min((uint64_t)a.ktiles, s.k0 + (end - at));
    at += s.k1 - s.k0;
    return true;
  }
};
// The CTA whose part holds slice u.
__device__ __forceinline__ uint32_t owner(const AdapterArgs& a, uint64_t u) {
  return (uint32_t)(((u + 1) * gridDim.x - 1) / ((uint64_t)a.ncol * a.ntok * a.ktiles));
}

// h_t = scale_a x_t A_a: one CTA per token; a thread sums 8 ranks over every
// KS-th k, the KS sums are joined in order.  Also zeroes the arrival counters.
template <int FMT>
__global__ void __launch_bounds__(kShrinkThreads) shrink_kernel(const AdapterArgs a) {
  using T = typename Elem<FMT>::T;
  if (a.split)
    for (uint32_t i = blockIdx.x * kShrinkThreads + threadIdx.x; i < a.ncol * a.ntok;
         i += gridDim.x * kShrinkThreads)
      a.arrived[i] = 0;
  __shared__ float sums[kShrinkThreads][8];
  if (a.R == 0) return;
  const uint32_t V = a.r / 8, KS = kShrinkThreads / V;
  const uint32_t kk = threadIdx.x / V, v = threadIdx.x % V;
  for (uint32_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const uint32_t id = (uint32_t)a.ids[t];
    if (id >= a.R) continue;
    const T* x = static_cast<const T*>(a.x) + t * a.ldx;
    const T* A = static_cast<const T*>(a.a) + (size_t)id * a.k * a.r;
    float s[8] = {};
    if (kk < KS)
      for (uint32_t k = kk; k < a.k; k += KS) {
        const uint4 raw = *reinterpret_cast<const uint4*>(A + (size_t)k * a.r + v * 8);
        const T* e = reinterpret_cast<const T*>(&raw);
        const float xv = moe::to_f(x[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = fmaf(xv, moe::to_f(e[i]), s[i]);
      }
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[threadIdx.x][i] = s[i];
    __syncthreads();
    if (threadIdx.x < a.r) {
      float total = 0.f;
      for (uint32_t q = 0; q < KS; ++q) total += sums[q * V + threadIdx.x / 8][threadIdx.x % 8];
      a.h[(size_t)t * a.r + threadIdx.x] = a.scale[id] * total;
    }
    __syncthreads();
  }
}

// Adds the adapters' part of 16 tokens from t0 on, column n, and stores them.
template <int FMT>
__device__ __forceinline__ void finish16(const AdapterArgs& a, float (&acc)[16], uint32_t t0,
                                         uint32_t n) {
  using T = typename Elem<FMT>::T;
  const bool in = n < a.n;
  if (a.R)
    for (uint32_t ic = 0; ic < a.r; ic += 8) {
      uint32_t have = 0xffffffffu;
      float b[8];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const uint32_t t = t0 + j;
        const uint32_t id = t < a.T ? (uint32_t)a.ids[t] : 0xffffffffu;
        if (id < a.R) {
          if (id != have) {
            const T* B = static_cast<const T*>(a.b) + ((size_t)id * a.r + ic) * a.n + n;
#pragma unroll
            for (int i = 0; i < 8; ++i) b[i] = in ? moe::to_f(B[(size_t)i * a.n]) : 0.f;
            have = id;
          }
          const float4* h = reinterpret_cast<const float4*>(a.h + (size_t)t * a.r + ic);
          const float4 h0 = h[0], h1 = h[1];
          float s = acc[j];
          s = fmaf(h0.x, b[0], s), s = fmaf(h0.y, b[1], s);
          s = fmaf(h0.z, b[2], s), s = fmaf(h0.w, b[3], s);
          s = fmaf(h1.x, b[4], s), s = fmaf(h1.y, b[5], s);
          s = fmaf(h1.z, b[6], s), s = fmaf(h1.w, b[7], s);
          acc[j] = s;
        }
      }
    }
  if (!in) return;
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (t0 + j < a.T)
      static_cast<T*>(a.y)[(size_t)(t0 + j) * a.ldy + n] = moe::from_f<T>(acc[j]);
}

template <int FMT>
__global__ void __launch_bounds__(kThreads, 1)
    adapter_kernel(const __grid_constant__ CUtensorMap map_w,
                   const __grid_constant__ CUtensorMap map_x, const AdapterArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (symm::smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t stage_bytes = kATile + a.bt * 128;
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], tfull[2], tempty[2], drain;
  __shared__ uint32_t tmem_slot, last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < a.stages; ++s) {
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
  if (warp == 1) symm::tmem_alloc(&tmem_slot, a.tmem_cols);
  symm::tc_fence_before();
  __syncthreads();
  symm::tc_fence_after();
  const uint32_t tmem = tmem_slot;
  Walk walk(a);
  Segment s;

  if (warp == 0) {
    if (lane == 0) {  // ------------------------------------- TMA producer
      uint64_t it = 0;
      uint32_t st = 0, ph = 1;
      bool ok = true;
      while (ok && walk.next(a, s)) {
        const int n0 = (int)(s.tile % a.ncol) * kBM, t0 = (int)(s.tile / a.ncol * a.bt);
        for (uint32_t kt = s.k0; kt < s.k1; ++kt, ++it) {
          if (!symm::mbar_wait_ab(&empty[st], ph, a.budget_ns, a.ctl)) {
            symm::record_error(a.ctl, symm::kErrTimedOut, -3);
            ok = false;
            break;
          }
          uint8_t* buf = smem + (size_t)st * stage_bytes;
          symm::mbar_arrive_expect_tx(&full[st], stage_bytes);
          tma_load_2d(buf, &map_w, n0, (int)(kt * kBK), &full[st]);
          tma_load_2d(buf + kATile / 2, &map_w, n0 + 64, (int)(kt * kBK), &full[st]);
          tma_load_2d(buf + kATile, &map_x, (int)(kt * kBK), t0, &full[st]);
          if (++st == a.stages) st = 0, ph ^= 1;
        }
      }
      // every load issued lands before the CTA may leave (bounded)
      for (uint64_t i = it > a.stages ? it - a.stages : 0; i < it; ++i)
        symm::mbar_wait(&full[i % a.stages], (uint32_t)((i / a.stages) & 1), a.budget_ns);
    }
  } else if (warp == 1) {
    if (lane == 0) {  // -------------------------------------- MMA issuer
      // fp32 accumulator, A and B of one type, A (W) M-major, B (x) K-major
      const uint32_t idesc = (1u << 4) | ((uint32_t)FMT << 7) | ((uint32_t)FMT << 10) |
                             (1u << 15) | ((a.bt >> 3) << 17) | ((uint32_t)(kBM >> 4) << 24);
      uint32_t st = 0, ph = 0, seg = 0;
      bool ok = true;
      for (; ok && walk.next(a, s); ++seg) {
        const uint32_t buf = seg & 1;
        if (!symm::mbar_wait_ab(&tempty[buf], ((seg >> 1) & 1) ^ 1u, a.budget_ns, a.ctl)) {
          symm::record_error(a.ctl, symm::kErrTimedOut, -4);
          break;
        }
        symm::tc_fence_after();
        const uint32_t acc = tmem + buf * a.bt;
        for (uint32_t kt = s.k0; kt < s.k1; ++kt) {
          if (!symm::mbar_wait_ab(&full[st], ph, a.budget_ns, a.ctl)) {
            symm::record_error(a.ctl, symm::kErrTimedOut, -5);
            ok = false;
            break;
          }
          symm::tc_fence_after();
          const uint8_t* tile = smem + (size_t)st * stage_bytes;
          const uint64_t wd = symm::sw128_mnmajor_desc(tile);
          const uint64_t xd = symm::sw128_kmajor_desc(tile + kATile);
#pragma unroll
          for (int j = 0; j < kBK / 16; ++j)  // K = 16: 16 rows of W, 32 bytes of x
            symm::tc_mma(acc, wd + (uint64_t)((16 * 128) >> 4) * j, xd + 2 * j, idesc,
                         kt != s.k0 || j != 0);
          symm::tc_commit(&empty[st]);
          if (++st == a.stages) st = 0, ph ^= 1;
        }
        if (ok) symm::tc_commit(&tfull[buf]);
      }
      symm::tc_commit(&drain);  // every MMA is complete before TMEM is freed
      symm::mbar_wait(&drain, 0, a.budget_ns);
    }
  } else {  // -------------------------------------------------- epilogue
    const uint32_t q = (uint32_t)(warp & 3);  // TMEM lanes 32q .. 32q + 31
    const uint32_t row = 32 * q + lane;       // this thread's column of W in the tile
    const uint32_t chunks = a.bt / 16;
    for (uint32_t seg = 0; walk.next(a, s); ++seg) {
      const uint32_t buf = seg & 1;
      if (!symm::mbar_wait_ab(&tfull[buf], (seg >> 1) & 1, a.budget_ns, a.ctl)) {
        symm::record_error(a.ctl, symm::kErrTimedOut, -6);
        break;
      }
      symm::tc_fence_after();
      const uint32_t taddr = tmem + ((32 * q) << 16) + buf * a.bt;
      const uint32_t n = (s.tile % a.ncol) * kBM + row, t0 = s.tile / a.ncol * a.bt;
      const bool whole = s.k0 == 0 && s.k1 == a.ktiles;
      // the first segment of a CTA has slot 0, a later partial one is its last: slot 1
      float* mine = a.part + ((size_t)blockIdx.x * 2 + (seg != 0)) * a.bt * kBM;
#pragma unroll 1
      for (uint32_t c = 0; c < chunks; ++c) {
        uint32_t v[16];
        symm::tmem_ld16(taddr + c * 16, v);
        if (c + 1 == chunks) {  // the accumulator is free for the next segment
          symm::tc_fence_before();
          symm::mbar_arrive(&tempty[buf]);
        }
        if (t0 + c * 16 >= a.T) continue;
        if (whole) {
          float acc[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[j] = __uint_as_float(v[j]);
          finish16<FMT>(a, acc, t0 + c * 16, n);
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            __stcg(mine + (size_t)(c * 16 + j) * kBM + row, __uint_as_float(v[j]));
        }
      }
      if (whole) continue;
      const uint64_t u0 = (uint64_t)s.tile * a.ktiles;
      const uint32_t first = owner(a, u0), end = owner(a, u0 + a.ktiles - 1) + 1;
      __threadfence();
      symm::group_sync(1, 128);
      if (threadIdx.x == 64)
        last = symm::atom_add_acq_rel_u32(&a.arrived[s.tile], 1u) + 1 == end - first;
      symm::group_sync(1, 128);
      if (!last) continue;
#pragma unroll 1
      for (uint32_t c = 0; c < chunks && t0 + c * 16 < a.T; ++c) {
        float acc[16] = {};
        for (uint32_t b = first; b < end; ++b) {
          const float* p =
              a.part + ((size_t)b * 2 + (cut(a, b) < u0)) * a.bt * kBM + (size_t)c * 16 * kBM + row;
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[j] += __ldcg(p + (size_t)j * kBM);
        }
        finish16<FMT>(a, acc, t0 + c * 16, n);
      }
    }
  }

  symm::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    symm::tc_fence_after();
    symm::tmem_dealloc(tmem, a.tmem_cols);
  }
}

// How a call of these sizes is cut up.
struct Plan {
  uint32_t bt, ntok, ncol, ktiles, stages, split, ctas, tmem_cols;
  size_t h_bytes, part_bytes, arrived_bytes;
  size_t bytes() const { return h_bytes + part_bytes + arrived_bytes; }
};

size_t up(size_t v, size_t a) { return (v + a - 1) / a * a; }

Plan plan_of(int T, int k, int n, int r) {
  Plan p{};
  const uint32_t sms = (uint32_t)std::max(sm_count(), 1);
  const uint32_t blocks = ((uint32_t)T + 255) / 256;  // token blocks of at most 256
  p.bt = (uint32_t)up(((uint32_t)T + blocks - 1) / blocks, 16);
  p.ntok = ((uint32_t)T + p.bt - 1) / p.bt;
  p.ncol = ((uint32_t)n + kBM - 1) / kBM;
  p.ktiles = ((uint32_t)k + kBK - 1) / kBK;
  p.stages = std::min<uint32_t>(kMaxStages, kRingBytes / (kATile + p.bt * 128));
  const uint64_t tiles = (uint64_t)p.ncol * p.ntok, slices = tiles * p.ktiles;
  const uint64_t waves = (tiles + sms - 1) / sms;
  // Whole tiles while the last wave leaves at most a tenth of the SMs' time unused.
  p.split = tiles * 10 < waves * sms * 9 && p.ktiles > 1;
  p.ctas = p.split ? (uint32_t)std::min<uint64_t>(sms, std::max<uint64_t>(1, slices / 4))
                   : (uint32_t)std::min<uint64_t>(sms, tiles);
  if (p.split && p.ctas < 2) p.split = 0, p.ctas = (uint32_t)std::min<uint64_t>(sms, tiles);
  p.tmem_cols = 32;
  while (p.tmem_cols < 2 * p.bt) p.tmem_cols *= 2;
  p.h_bytes = up((size_t)T * r * 4, 256);
  p.part_bytes = p.split ? (size_t)p.ctas * 2 * p.bt * kBM * 4 : 0;
  p.arrived_bytes = p.split ? up((size_t)tiles * 4, 256) : 0;
  return p;
}

int check_adapter(const char* what, int T, int k, int n, int r) {
  if (T < 0 || T > (1 << 24) || k < 8 || n < 8 || k % 8 || n % 8 || k > (1 << 20) ||
      n > (1 << 20))
    return fail(SYMM_EINVAL, std::string(what) + ": T must be in [0, 2^24], k and n multiples of "
                                                 "8 (16-byte rows) in [8, 2^20]");
  if (r < 0 || r > SYMM_MOE_MAX_RANK || r % 8)
    return fail(SYMM_EINVAL, std::string(what) + ": r must be a multiple of 8 up to 128");
  return SYMM_OK;
}

// [rows][inner] 2-byte elements, `ld` apart, boxes of 64 x box_rows, 128-byte swizzled.
int make_map(CUtensorMap* map, const void* base, int fmt, uint64_t inner, uint64_t rows, size_t ld,
             uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return fail(SYMM_ECUDA, "moe_adapter_matmul: no cuTensorMapEncodeTiled");
  const cuuint64_t dims[2] = {inner, rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r =
      fn(map, fmt == 1 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
         const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(SYMM_ECUDA,
                "moe_adapter_matmul: tensor map rejected (CUresult " + std::to_string((int)r) + ")");
  return SYMM_OK;
}

template <int FMT>
int launch(const Plan& p, const CUtensorMap& map_w, const CUtensorMap& map_x, const AdapterArgs& a,
           cudaStream_t s) {
  const size_t smem = 1024 + (size_t)p.stages * (kATile + p.bt * 128);
  int rc = cuda_check(cudaFuncSetAttribute(adapter_kernel<FMT>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)(1024 + kRingBytes)),
                      "moe_adapter_matmul: kernel set-up");
  if (rc) return rc;
  if (a.R || p.split) {
    shrink_kernel<FMT><<<a.R ? std::min<uint32_t>(a.T, 1u << 16) : 1u, kShrinkThreads, 0, s>>>(a);
    rc = cuda_check(cudaGetLastError(), "moe_adapter_matmul: rank products");
    if (rc) return rc;
  }
  adapter_kernel<FMT><<<p.ctas, kThreads, smem, s>>>(map_w, map_x, a);
  return cuda_check(cudaGetLastError(), "moe_adapter_matmul: product");
}

}  // namespace

extern "C" int moe_adapter_workspace(int T, int k, int n, int r, size_t* bytes) {
  return moe::entry("moe_adapter_workspace", [&]() -> int {
    if (!bytes) return fail(SYMM_EINVAL, "moe_adapter_workspace: NULL bytes");
    int rc = check_adapter("moe_adapter_workspace", T, k, n, r);
    if (rc) return rc;
    *bytes = T ? plan_of(T, k, n, r).bytes() : 0;
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
    if (!x || !w || !y || !workspace || (R && (!a || !b || !scale || !ids)))
      return fail(SYMM_EINVAL, "moe_adapter_matmul: NULL input, output or workspace");
    if (!moe::aligned(x, 16) || !moe::aligned(w, 16) || !moe::aligned(a, 16) ||
        !moe::aligned(b, 2) || !moe::aligned(y, 2) || !moe::aligned(scale, 4) ||
        !moe::aligned(ids, 4) || !moe::aligned(workspace, 256))
      return fail(SYMM_EINVAL, "moe_adapter_matmul: x, w and a must be 16-byte aligned, workspace "
                               "256-byte aligned, the rest to their elements");
    if (y == x || y == w || y == a || y == b)
      return fail(SYMM_EINVAL, "moe_adapter_matmul: y must not be an input");
    const Plan p = plan_of(T, k, n, r);
    const int fmt = dtype == SYMM_DTYPE_BF16 ? 1 : 0;
    CUtensorMap map_w, map_x;
    rc = make_map(&map_w, w, fmt, (uint64_t)n, (uint64_t)k, ldw, kBK);
    if (rc) return rc;
    rc = make_map(&map_x, x, fmt, (uint64_t)k, (uint64_t)T, ldx, p.bt);
    if (rc) return rc;
    cudaStream_t s = as_stream(stream);
    rc = ensure_ctrl(heap, s);
    if (rc) return rc;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    AdapterArgs g{};
    g.x = x, g.ldx = ldx, g.a = a, g.b = b, g.scale = scale, g.ids = ids, g.y = y, g.ldy = ldy;
    g.T = (uint32_t)T, g.k = (uint32_t)k, g.n = (uint32_t)n, g.R = (uint32_t)R, g.r = (uint32_t)r;
    g.bt = p.bt, g.ntok = p.ntok, g.ncol = p.ncol, g.ktiles = p.ktiles, g.stages = p.stages;
    g.split = p.split, g.tmem_cols = p.tmem_cols;
    g.h = reinterpret_cast<float*>(ws);
    g.part = reinterpret_cast<float*>(ws + p.h_bytes);
    g.arrived = reinterpret_cast<uint32_t*>(ws + p.h_bytes + p.part_bytes);
    g.budget_ns = heap->spin_budget;
    g.ctl = reinterpret_cast<Control*>(heap->base);
    return fmt ? launch<1>(p, map_w, map_x, g, s) : launch<0>(p, map_w, map_x, g, s);
  });
}
