// moe_norm.cu -- from a block's output rows to the next block's input: the
// weighted sum of a token's rows, the norm after the block, its gate and
// residual scale, and the norm before the next block; and the gradients.
//
// Forward, with N(v) = v r(v), r(v) = 1/sqrt(mean v^2 + eps):
//   y = sum_j w_j Y_j;  u = wpost N(y);  xo = res x + gate u;  h = wpre N(xo).
// Backward, with z = xo, r1 = r(y), r2 = r(xo), q = dh wpre, n = y r1:
//   dz = dxo + r2 (q - z r2^2 mean(q z))       dwpre = sum_t dh z r2
//   dx = res dz                                dres  = sum_t dz x
//   dgate = sum_i dz n wpost                   dwpost = sum_t gate dz n
//   dn = gate dz wpost;  dy = r1 (dn - n mean(dn n));  dY_j = w_j dy
//   dw_j = <dy, Y_j>.
// dy needs mean(dn n), and that needs y of all rows: Y is read twice, the second
// time from shared memory where a token's rows fit there.
//
// One CTA per token at a time; a thread owns the same columns in every token
// of its CTA (up to 4 chunks of 8), so the column sums of dres, dwpost and
// dwpre stay in its registers over all tokens and are written once per CTA;
// a second small kernel adds the CTAs' sums in order.
//
// Measured (rows of 7168 in bf16, 8 a token): 8192 tokens 216 us, 6.0 TB/s or
// 88 % of the copy rate; backward, 4096 tokens 273 us, 4.5 TB/s (67 %): a
// token's 172 KB fill an SM's shared memory there, so its phases overlap only in
// part.  Rows of 1024: 5.8 TB/s.  Rows that are not 16-byte aligned, or odd,
// move by 4-byte copies: 3.2 TB/s for 999 floats, 1.7 for 3001 bf16.  A token
// that does not fit into shared memory goes through norm_back_kernel: 753 us for
// the same rows in 32 bits (3.3 TB/s, 48 %).
#include <algorithm>
#include <mutex>
#include <set>
#include <type_traits>

#include "moe_common.cuh"

using namespace symm_host;

namespace {

constexpr int kMaxThreads = 512;
constexpr int kMaxWarps = kMaxThreads / 32;
constexpr int kChunk = 8;

struct NormArgs {
  const void* x;
  size_t ld;
  const void* y;
  size_t ldy;
  const int32_t* rows;
  size_t yrows;
  const float *weights, *gate, *res, *w_post, *w_pre;
  float eps;
  int T, D, k;
  void *xo, *h;
  float* rstd;
};

struct NormBackArgs {
  const void *dxo, *dh, *x, *xo;
  size_t ld;
  const void* y;
  size_t ldy;
  const int32_t* rows;
  size_t yrows;
  const float *weights, *gate, *res, *w_post, *w_pre, *rstd;
  int T, D, k;
  void *dx, *dy;
  float *dweights, *dgate, *dres, *dw_post, *dw_pre;
  float* part;  // [CTAs][3][D]
};

// A thread's columns.  ALIGNED: chunk c is 8 consecutive columns, moved as
// 16-byte vectors (rows 16-byte aligned, D a multiple of 8).  Otherwise its
// 8 columns are blockDim.x apart and moved one by one, coalesced.
template <typename T, bool ALIGNED>
struct Cols {
  int D;
  __device__ __forceinline__ int at(int c, int i) const {
    return ALIGNED ? (c * (int)blockDim.x + (int)threadIdx.x) * kChunk + i
                   : (c * kChunk + i) * (int)blockDim.x + (int)threadIdx.x;
  }
  // chunk c of a row; 0 past D
  __device__ __forceinline__ void load(const T* row, int c, float (&v)[kChunk]) const {
    if constexpr (ALIGNED) {
      const int o = at(c, 0);
      if (o < D) {
        constexpr int N = sizeof(T) * kChunk / 16;
        uint4 raw[N];
#pragma unroll
        for (int n = 0; n < N; ++n) raw[n] = *(reinterpret_cast<const uint4*>(row + o) + n);
        const T* e = reinterpret_cast<const T*>(raw);
#pragma unroll
        for (int i = 0; i < kChunk; ++i) v[i] = moe::to_f(e[i]);
      } else {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) v[i] = 0.f;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kChunk; ++i) v[i] = at(c, i) < D ? moe::to_f(row[at(c, i)]) : 0.f;
    }
  }
  __device__ __forceinline__ void store(T* row, int c, const float (&v)[kChunk]) const {
    if constexpr (ALIGNED) {
      const int o = at(c, 0);
      if (o >= D) return;
      constexpr int N = sizeof(T) * kChunk / 16;
      uint4 raw[N];
      T* e = reinterpret_cast<T*>(raw);
#pragma unroll
      for (int i = 0; i < kChunk; ++i) e[i] = moe::from_f<T>(v[i]);
#pragma unroll
      for (int n = 0; n < N; ++n) *(reinterpret_cast<uint4*>(row + o) + n) = raw[n];
    } else {
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        if (at(c, i) < D) row[at(c, i)] = moe::from_f<T>(v[i]);
    }
  }
  // chunk c of a float vector; `none` where it is NULL
  __device__ __forceinline__ void vec(const float* p, int c, float none,
                                      float (&v)[kChunk]) const {
    if constexpr (ALIGNED) {
      const int o = at(c, 0);
      if (p && o < D) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p + o));
        const float4 b = __ldg(reinterpret_cast<const float4*>(p + o) + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
      } else {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) v[i] = p ? 0.f : none;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kChunk; ++i) v[i] = p ? (at(c, i) < D ? p[at(c, i)] : 0.f) : none;
    }
  }
};

// cp.async of 16 bytes past L1, and its groups.
__device__ __forceinline__ void copy16(uint32_t smem, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t smem, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem), "l"(src) : "memory");
}
__device__ __forceinline__ void commit_group() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void wait_groups() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Two floats in one 64-bit register pair: sm_103a does a multiply-add of both
// in one instruction, and these kernels are bound by what they can issue
// before they are bound by HBM.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 mk(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 mk(float both) { return mk(both, both); }
__device__ __forceinline__ void split(F2 a, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v));
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ float sum2(F2 a) {
  float lo, hi;
  split(a, lo, hi);
  return lo + hi;
}

constexpr int kPairs = kChunk / 2;
constexpr int kRows = 4;  // rows of Y handled together in the backward pass

// 16 bytes of T as pairs of floats, and back.
template <typename T>
__device__ __forceinline__ F2 unpack(uint32_t x);
template <>
__device__ __forceinline__ F2 unpack<__nv_bfloat16>(uint32_t x) {
  return mk(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
template <>
__device__ __forceinline__ F2 unpack<__half>(uint32_t x) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x));
  return mk(f.x, f.y);
}
template <typename T>
__device__ __forceinline__ uint32_t pack(F2 a);
template <>
__device__ __forceinline__ uint32_t pack<__nv_bfloat16>(F2 a) {
  float lo, hi;
  split(a, lo, hi);
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack<__half>(F2 a) {
  float lo, hi;
  split(a, lo, hi);
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A thread's columns of every row, and a ring of rows in shared memory in
// which the thread keeps these columns: it copies them in (asynchronously) and
// reads them back itself, so nothing but its own copies is waited for, and rows
// of the next tokens are on their way while a token is summed and normed.
// Columns past D are 0.
//
// NT = 0 (16-byte aligned rows, D a multiple of 8): chunk c is 8 consecutive
// columns in 16-byte vectors.  Otherwise, with a block of NT threads (known
// here, so that the many small copies need no address arithmetic), chunk c is
// words of 4 bytes that are NT words apart, a column or (16-bit types) a pair
// 2i, 2i + 1 of them each.
// A row of a 16-bit type may start in the middle of a word: its word i then
// holds columns 2i - 1 and 2i, and a pair is put together from this lane's word
// and the next lane's (the last lane keeps one word more).
template <typename T, int CH, int NT>
struct Ring {
  static constexpr bool WIDE = NT == 0;
  static constexpr int kBytes = (int)sizeof(T) * kChunk;  // of a chunk
  static constexpr int kVec = WIDE ? kBytes / 16 : kBytes / 4;  // copies of a chunk
  static constexpr int kUnit = WIDE ? 16 : 4;
  static constexpr bool kPairs16 = !WIDE && sizeof(T) == 2;
  uint32_t base, last_base;  // of this thread's first copy
  uint32_t odd;              // slots whose row starts in the middle of a word
  int D;
  __device__ __forceinline__ static int threads() { return WIDE ? (int)blockDim.x : NT; }
  __device__ __forceinline__ Ring(const void* smem, int D_, int depth) : odd(0), D(D_) {
    const uint32_t s = (uint32_t)__cvta_generic_to_shared(smem);
    base = s + threadIdx.x * (uint32_t)kUnit;
    last_base = s + (uint32_t)(CH * kVec * threads()) * 4u + (threadIdx.x >> 5) * 4u;
    for (int i = 0; i < depth; ++i)
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
          if (kPairs16 || col(c, v) < D) continue;  // copied, or masked when read
          if constexpr (WIDE)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at(i, c, v)), "r"(0)
                         : "memory");
          else
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(at(i, c, v)), "r"(0) : "memory");
        }
  }
  // of shared memory, per row
  __host__ __device__ static uint32_t bytes_of_slot(int threads) {
    const uint32_t words = kPairs16 ? (uint32_t)(CH * kVec * (threads / 32)) * 4u : 0u;
    return (uint32_t)(CH * kVec * threads) * kUnit + (words + 15u) / 16u * 16u;
  }
  __device__ __forceinline__ uint32_t at(int slot, int c, int v) const {
    return base + (uint32_t)slot * bytes_of_slot(threads()) +
           (uint32_t)((c * kVec + v) * threads()) * (uint32_t)kUnit;
  }
  // the last lane's further word
  __device__ __forceinline__ uint32_t at_last(int slot, int c, int v) const {
    return last_base + (uint32_t)slot * bytes_of_slot(threads()) +
           (uint32_t)((c * kVec + v) * (threads() / 32)) * 4u;
  }
  // first column of copy v of chunk c
  __device__ __forceinline__ int col(int c, int v) const {
    if constexpr (WIDE)
      return (c * threads() + (int)threadIdx.x) * kChunk + v * (16 / (int)sizeof(T));
    else
      return ((c * kVec + v) * threads() + (int)threadIdx.x) * (kPairs16 ? 2 : 1);
  }
  // whether copy v of chunk c lies in the row for every thread (words only)
  __device__ __forceinline__ bool inside(int c, int v) const {
    return D >= (c * kVec + v + 1) * threads() * (kPairs16 ? 2 : 1);
  }
  // columns of pair p of chunk c
  __device__ __forceinline__ int lo(int c, int p) const {
    if constexpr (WIDE) return col(c, 0) + 2 * p;
    else return kPairs16 ? col(c, p) : col(c, 2 * p);
  }
  __device__ __forceinline__ int hi(int c, int p) const {
    if constexpr (WIDE || kPairs16) return lo(c, p) + 1;
    else return col(c, 2 * p + 1);
  }
  // starts the copy of `row`
  __device__ __forceinline__ void copy(int slot, const T* row) {
    if constexpr (WIDE) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if (col(c, 0) < D)
#pragma unroll
          for (int v = 0; v < kVec; ++v) copy16(at(slot, c, v), row + col(c, v));
    } else if constexpr (kPairs16) {
      const uint32_t mid = (uint32_t)(reinterpret_cast<uintptr_t>(row) >> 1) & 1u;
      odd = (odd & ~(1u << slot)) | (mid << slot);
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
          const int o = col(c, v);
          if (inside(c, v) || o < D + (int)mid) copy4(at(slot, c, v), row + o - mid);
          if (mid && (threadIdx.x & 31) == 31 && o + 1 < D)
            copy4(at_last(slot, c, v), row + o + 1);
        }
    } else {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int v = 0; v < kVec; ++v)
          if (inside(c, v) || col(c, v) < D) copy4(at(slot, c, v), row + col(c, v));
    }
  }
  __device__ __forceinline__ void read(int slot, int c, F2 (&f)[kPairs]) const {
    if constexpr (WIDE) {
      uint4 raw[kVec];
#pragma unroll
      for (int v = 0; v < kVec; ++v)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(raw[v].x), "=r"(raw[v].y), "=r"(raw[v].z), "=r"(raw[v].w)
                     : "r"(at(slot, c, v))
                     : "memory");
      if constexpr (kVec == 1) {
        f[0] = unpack<T>(raw[0].x), f[1] = unpack<T>(raw[0].y);
        f[2] = unpack<T>(raw[0].z), f[3] = unpack<T>(raw[0].w);
      } else {
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
          f[2 * v] = mk(__uint_as_float(raw[v].x), __uint_as_float(raw[v].y));
          f[2 * v + 1] = mk(__uint_as_float(raw[v].z), __uint_as_float(raw[v].w));
        }
      }
    } else {
      uint32_t w[kVec];
#pragma unroll
      for (int v = 0; v < kVec; ++v) w[v] = word(at(slot, c, v));
      if constexpr (kPairs16) {
        if ((odd >> slot) & 1) {
#pragma unroll
          for (int v = 0; v < kVec; ++v) {
            uint32_t next = __shfl_down_sync(0xffffffffu, w[v], 1);
            if ((threadIdx.x & 31) == 31) next = word(at_last(slot, c, v));
            w[v] = __funnelshift_r(w[v], next, 16);
          }
        }
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
          // a word may hold a neighbour of the row where the row's columns end
          if (!inside(c, v) && hi(c, v) >= D) w[v] = lo(c, v) < D ? w[v] & 0xffffu : 0u;
          f[v] = unpack<T>(w[v]);
        }
      } else {
#pragma unroll
        for (int p = 0; p < kPairs; ++p)
          f[p] = mk(__uint_as_float(w[2 * p]), __uint_as_float(w[2 * p + 1]));
      }
    }
  }
  __device__ __forceinline__ void store(T* row, int c, const F2 (&f)[kPairs]) const {
    if constexpr (WIDE) {
      if (col(c, 0) >= D) return;
      uint4* p = reinterpret_cast<uint4*>(row + col(c, 0));
      if constexpr (kVec == 1) {
        *p = make_uint4(pack<T>(f[0]), pack<T>(f[1]), pack<T>(f[2]), pack<T>(f[3]));
      } else {
#pragma unroll
        for (int v = 0; v < kVec; ++v)
          *reinterpret_cast<ulonglong2*>(p + v) = make_ulonglong2(f[2 * v].v, f[2 * v + 1].v);
      }
    } else if constexpr (kPairs16) {
      const bool mid = (reinterpret_cast<uintptr_t>(row) >> 1) & 1;
#pragma unroll
      for (int p = 0; p < kPairs; ++p) {
        const uint32_t w = pack<T>(f[p]);
        uint16_t* o = reinterpret_cast<uint16_t*>(row + lo(c, p));
        if (!mid && (inside(c, p) || hi(c, p) < D)) {
          *reinterpret_cast<uint32_t*>(o) = w;
        } else {
          if (lo(c, p) < D) o[0] = (uint16_t)w;
          if (hi(c, p) < D) o[1] = (uint16_t)(w >> 16);
        }
      }
    } else {
      put(reinterpret_cast<float*>(row), c, f);
    }
  }
  // chunk c of a float vector; `none` where it is NULL
  __device__ __forceinline__ void vec(const float* p, int c, float none, F2 (&f)[kPairs]) const {
    if constexpr (WIDE) {
      if (p && col(c, 0) < D) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const ulonglong2 x = __ldg(reinterpret_cast<const ulonglong2*>(p + col(c, 0)) + v);
          f[2 * v].v = x.x, f[2 * v + 1].v = x.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) f[i] = mk(none);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPairs; ++i)
        f[i] = p ? mk(lo(c, i) < D ? __ldg(p + lo(c, i)) : 0.f,
                      hi(c, i) < D ? __ldg(p + hi(c, i)) : 0.f)
                 : mk(none);
    }
  }
  // ... and stored
  __device__ __forceinline__ void put(float* p, int c, const F2 (&f)[kPairs]) const {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      float a, b;
      split(f[i], a, b);
      if (lo(c, i) < D) p[lo(c, i)] = a;
      if (hi(c, i) < D) p[hi(c, i)] = b;
    }
  }
  __device__ __forceinline__ static uint32_t word(uint32_t addr) {
    uint32_t w;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(addr) : "memory");
    return w;
  }
};

// Row j of token t in Y, or -1.
__device__ __forceinline__ long long row_of(const int32_t* rows, size_t yrows, size_t slot) {
  const long long r = rows ? (long long)rows[slot] : (long long)slot;
  return r >= 0 && r < (long long)yrows ? r : -1;
}

// Token t's slots, one per lane: the row (-1: none) and the weight.
template <typename A>
__device__ __forceinline__ int lane_row(const A& a, size_t t, int lane) {
  if (t >= (size_t)a.T || lane >= a.k) return -1;
  return (int)row_of(a.rows, a.yrows, t * a.k + lane);
}
template <typename A>
__device__ __forceinline__ float lane_weight(const A& a, size_t t, int lane) {
  return t < (size_t)a.T && lane < a.k && a.weights ? a.weights[t * a.k + lane] : 1.f;
}

// y = sum_j w_j Y_j of chunk c, in slot order
template <typename T, typename C, typename A>
__device__ __forceinline__ void weighted(const A& a, const C& cols, size_t t, int c,
                                         float (&y)[kChunk]) {
#pragma unroll
  for (int i = 0; i < kChunk; ++i) y[i] = 0.f;
  for (int j = 0; j < a.k; ++j) {
    const long long r = row_of(a.rows, a.yrows, t * a.k + j);
    if (r < 0) continue;
    const float w = a.weights ? a.weights[t * a.k + j] : 1.f;
    float v[kChunk];
    cols.load(static_cast<const T*>(a.y) + (size_t)r * a.ldy, c, v);
#pragma unroll
    for (int i = 0; i < kChunk; ++i) y[i] = fmaf(w, v[i], y[i]);
  }
}

// CTAs of NT (0: up to 512) threads that make up `threads`.
constexpr int blocks_of(int threads, int NT) { return threads / (NT ? NT : kMaxThreads); }

// The forward pass.  Bound by HBM: (k + 3) rows a token.  The next DEPTH - 1
// rows are in flight.
template <typename T, int CH, int NT, int DEPTH>
__global__ void __launch_bounds__(NT ? NT : kMaxThreads, CH == 4 ? 1 : blocks_of(1024, NT))
    norm_stream_kernel(const NormArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float red[2][kMaxWarps];
  Ring<T, CH, NT> ring(smem, a.D, DEPTH);
  moe::wait_for_earlier();
  const int lane = threadIdx.x & 31;
  const float mean = 1.f / (float)a.D;
  const size_t step = gridDim.x;
  // What is copied next: row fj of token ft (its k rows, then its x) into slot
  // fs; the token's row numbers, and those of the one after it, in the lanes.
  size_t ft = blockIdx.x;
  int fj = 0, fs = 0, frow = lane_row(a, ft, lane), frow2 = lane_row(a, ft + step, lane);
  uint32_t have = 0;  // slots that hold a row
  auto fill = [&]() {
    const T* row = nullptr;
    if (fj < a.k) {
      const int r = __shfl_sync(0xffffffffu, frow, fj);
      if (r >= 0) row = static_cast<const T*>(a.y) + (size_t)r * a.ldy;
      ++fj;
    } else {
      if (ft < (size_t)a.T) row = static_cast<const T*>(a.x) + ft * a.ld;
      fj = 0;
      ft += step;
      frow = frow2;
      frow2 = lane_row(a, ft + step, lane);
    }
    if (row) ring.copy(fs, row);
    commit_group();
    have = row ? have | (1u << fs) : have & ~(1u << fs);
    if (++fs == DEPTH) fs = 0;
  };
  for (int i = 0; i < DEPTH; ++i) fill();
  int s = 0;
  float weight = lane_weight(a, blockIdx.x, lane);
  for (size_t t = blockIdx.x; t < (size_t)a.T; t += step) {
    const float weight2 = lane_weight(a, t + step, lane);
    const float gate = a.gate ? __ldg(a.gate + t) : 1.f;
    F2 z[CH][kPairs];
    float r1 = 1.f, r2 = 1.f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < kPairs; ++i) z[c][i] = mk(0.f);
#pragma unroll 1
    for (int j = 0; j < a.k; ++j) {
      const F2 w = mk(__shfl_sync(0xffffffffu, weight, j));
      wait_groups<DEPTH - 1>();
      if ((have >> s) & 1) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          F2 v[kPairs];
          ring.read(s, c, v);
#pragma unroll
          for (int i = 0; i < kPairs; ++i) z[c][i] = fma2(w, v[i], z[c][i]);
        }
      }
      fill();
      if (++s == DEPTH) s = 0;
    }
    weight = weight2;
    if (a.w_post) {
      F2 ss = mk(0.f);
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < kPairs; ++i) ss = fma2(z[c][i], z[c][i], ss);
      r1 = 1.f / sqrtf(moe::block_sum_once(sum2(ss), red[0]) * mean + a.eps);
    }
    const F2 sc = mk(gate * r1);
    wait_groups<DEPTH - 1>();
    F2 ss = mk(0.f);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      F2 v[kPairs];
      ring.read(s, c, v);
      if (a.y) {
        F2 res[kPairs], w[kPairs];
        ring.vec(a.res, c, 1.f, res);
        ring.vec(a.w_post, c, 1.f, w);
#pragma unroll
        for (int i = 0; i < kPairs; ++i)
          z[c][i] = fma2(mul2(sc, w[i]), z[c][i], mul2(res[i], v[i]));
        ring.store(static_cast<T*>(a.xo) + t * a.ld, c, z[c]);
      } else {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) z[c][i] = v[i];
      }
#pragma unroll
      for (int i = 0; i < kPairs; ++i) ss = fma2(z[c][i], z[c][i], ss);
    }
    fill();
    if (++s == DEPTH) s = 0;
    if (a.h) {
      r2 = 1.f / sqrtf(moe::block_sum_once(sum2(ss), red[1]) * mean + a.eps);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        F2 w[kPairs];
        ring.vec(a.w_pre, c, 1.f, w);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) w[i] = mul2(w[i], mul2(z[c][i], mk(r2)));
        ring.store(static_cast<T*>(a.h) + t * a.ld, c, w);
      }
    }
    if (a.rstd && threadIdx.x == 0) a.rstd[2 * t] = r1, a.rstd[2 * t + 1] = r2;
    if (!a.w_post || !a.h) __syncthreads();  // `red` is free again (see block_sum_once)
  }
  wait_groups<0>();
}

// The backward pass, when shared memory does not hold a token: Y and the rows
// of dh and z are read twice, nothing ahead of its use, so it is bound by the
// latency of each token's loads and sums (2.1 times the bytes' time at 4096 x 8
// rows of 7168 floats; 4.9 times at 2048 x 4 rows of 16384 bf16, where four
// chunks a thread spill).
template <typename T, bool ALIGNED, int CH>
__global__ void __launch_bounds__(kMaxThreads) norm_back_kernel(const NormBackArgs a) {
  moe::wait_for_earlier();
  moe::let_next_start();
  __shared__ float red[kMaxWarps];
  __shared__ float dots[kMaxWarps][2 * SYMM_MOE_MAX_TOPK];  // <dn, Y_j>, <n, Y_j> per warp
  const Cols<T, ALIGNED> cols{a.D};
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const float mean = 1.f / (float)a.D;
  float s_res[CH][kChunk], s_post[CH][kChunk], s_pre[CH][kChunk];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int i = 0; i < kChunk; ++i) s_res[c][i] = s_post[c][i] = s_pre[c][i] = 0.f;
  for (size_t t = blockIdx.x; t < (size_t)a.T; t += gridDim.x) {
    const T* zrow = static_cast<const T*>(a.y ? a.xo : a.x) + t * a.ld;
    const T* xrow = static_cast<const T*>(a.x) + t * a.ld;
    const T* dhrow = static_cast<const T*>(a.dh) + t * a.ld;
    const T* dxorow = static_cast<const T*>(a.dxo) + t * a.ld;
    const float r1 = a.rstd[2 * t], r2 = a.rstd[2 * t + 1];
    float mqz = 0.f;
    if (a.dh) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        float z[kChunk], q[kChunk], w[kChunk];
        cols.load(zrow, c, z);
        cols.load(dhrow, c, q);
        cols.vec(a.w_pre, c, 1.f, w);
#pragma unroll
        for (int i = 0; i < kChunk; ++i) mqz = fmaf(q[i] * w[i], z[i], mqz);
      }
      mqz = moe::block_sum(mqz, red) * mean;
    }
    const float gate = a.gate ? a.gate[t] : 1.f;
    float dn[CH][kChunk], n[CH][kChunk];
    float dgate = 0.f, mdn = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float dz[kChunk], x[kChunk], w[kChunk];
      if (a.dxo) {
        cols.load(dxorow, c, dz);
      } else {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) dz[i] = 0.f;
      }
      if (a.dh) {
        float z[kChunk], q[kChunk];
        cols.load(zrow, c, z);
        cols.load(dhrow, c, q);
        cols.vec(a.w_pre, c, 1.f, w);
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
          const float zn = z[i] * r2;
          s_pre[c][i] = fmaf(q[i], zn, s_pre[c][i]);
          dz[i] += r2 * (q[i] * w[i] - zn * (r2 * mqz));
        }
      }
      float res[kChunk];
      cols.load(xrow, c, x);
      cols.vec(a.res, c, 1.f, res);
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        s_res[c][i] = fmaf(dz[i], x[i], s_res[c][i]);
        res[i] *= dz[i];
      }
      cols.store(static_cast<T*>(a.dx) + t * a.ld, c, res);
      if (!a.y) continue;
      weighted<T>(a, cols, t, c, n[c]);
      cols.vec(a.w_post, c, 1.f, w);
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        n[c][i] *= r1;
        s_post[c][i] = fmaf(gate * dz[i], n[c][i], s_post[c][i]);
        const float d = dz[i] * w[i];
        dgate = fmaf(d, n[c][i], dgate);
        dn[c][i] = gate * d;
      }
    }
    if (!a.y) continue;
    dgate = moe::block_sum(dgate, red);
    mdn = a.w_post ? dgate * gate * mean : 0.f;  // mean(dn n); no norm, no such term
    if (a.dgate && threadIdx.x == 0) a.dgate[t] = dgate;
    for (int j = 0; j < a.k; ++j) {
      const long long r = row_of(a.rows, a.yrows, t * a.k + j);
      float p = 0.f, q = 0.f;
      if (r >= 0) {
        const float wr1 = (a.weights ? a.weights[t * a.k + j] : 1.f) * r1;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          if (a.dweights) {
            float v[kChunk];
            cols.load(static_cast<const T*>(a.y) + (size_t)r * a.ldy, c, v);
#pragma unroll
            for (int i = 0; i < kChunk; ++i) {
              p = fmaf(dn[c][i], v[i], p);
              q = fmaf(n[c][i], v[i], q);
            }
          }
          float o[kChunk];
#pragma unroll
          for (int i = 0; i < kChunk; ++i) o[i] = wr1 * (dn[c][i] - n[c][i] * mdn);
          cols.store(static_cast<T*>(a.dy) + (size_t)r * a.ldy, c, o);
        }
      }
      if (a.dweights) {
        p = moe::warp_sum(p);
        q = moe::warp_sum(q);
        if (lane == 0) dots[warp][2 * j] = p, dots[warp][2 * j + 1] = q;
      }
    }
    if (a.dweights) {
      __syncthreads();
      if ((int)threadIdx.x < a.k) {
        float p = 0.f, q = 0.f;
        for (int w = 0; w < warps; ++w) {
          p += dots[w][2 * threadIdx.x];
          q += dots[w][2 * threadIdx.x + 1];
        }
        a.dweights[t * a.k + threadIdx.x] = r1 * (p - mdn * q);
      }
      __syncthreads();
    }
  }
  float* part = a.part + (size_t)blockIdx.x * 3 * a.D;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      const int o = cols.at(c, i);
      if (o < a.D) {
        part[o] = s_res[c][i];
        part[a.D + o] = s_post[c][i];
        part[2 * (size_t)a.D + o] = s_pre[c][i];
      }
    }
}

// The backward pass, when shared memory holds a whole token: (2k + 5) rows
// through HBM a token, and Y read twice from shared memory only -- for y, and
// for the inner products with it.  Every row has its own place there (dh, z,
// dxo, x, Y_0 ..): the first four are copied in one group for the next token as
// soon as they are used up, and row j of Y when this token's is.
template <typename T, int CH, int NT>
__global__ void __launch_bounds__(NT ? NT : kMaxThreads, blocks_of(512, NT))
    norm_back_stream_kernel(const NormBackArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  moe::wait_for_earlier();
  moe::let_next_start();
  __shared__ float red[2][kMaxWarps];
  __shared__ float dots[kMaxWarps][SYMM_MOE_MAX_TOPK];  // <dy / r1, Y_j> per warp
  Ring<T, CH, NT> ring(smem, a.D, 4 + a.k);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const float mean = 1.f / (float)a.D;
  const size_t step = gridDim.x;
  F2 s_res[CH][kPairs], s_post[CH][kPairs], s_pre[CH][kPairs];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int i = 0; i < kPairs; ++i) s_res[c][i] = s_post[c][i] = s_pre[c][i] = mk(0.f);
  const T* Y = static_cast<const T*>(a.y);
  const T* zsrc = static_cast<const T*>(a.y ? a.xo : a.x);
  auto fill_head = [&](size_t t) {
    if (t < (size_t)a.T) {
      const size_t o = t * a.ld;
      if (a.dh) {
        ring.copy(0, static_cast<const T*>(a.dh) + o);
        ring.copy(1, zsrc + o);
      }
      if (a.dxo) ring.copy(2, static_cast<const T*>(a.dxo) + o);
      if (a.dres) ring.copy(3, static_cast<const T*>(a.x) + o);
    }
    commit_group();
  };
  // A token's slots, one per lane: where the row starts in Y (and in dY), and
  // the weight; a bit of `rows` for each slot that has a row.
  size_t t = blockIdx.x;
  int r = lane_row(a, t, lane), rn = lane_row(a, t + step, lane);
  size_t off = r < 0 ? 0 : (size_t)r * a.ldy;
  uint32_t rows = __ballot_sync(0xffffffffu, r >= 0);
  float weight = lane_weight(a, t, lane);
  float r1 = a.rstd[2 * t], r2 = a.rstd[2 * t + 1];
  fill_head(t);
#pragma unroll 1
  for (int j = 0; j < a.k; ++j) {
    const size_t o = __shfl_sync(0xffffffffu, off, j);
    if ((rows >> j) & 1) ring.copy(4 + j, Y + o);
  }
  commit_group();
  for (; t < (size_t)a.T; t += step) {
    // the next token's, on their way
    const size_t offn = rn < 0 ? 0 : (size_t)rn * a.ldy;
    const uint32_t rowsn = __ballot_sync(0xffffffffu, rn >= 0);
    rn = lane_row(a, t + 2 * step, lane);
    const float weightn = lane_weight(a, t + step, lane);
    const size_t tn = t + step < (size_t)a.T ? t + step : t;
    const float r1n = __ldg(a.rstd + 2 * tn), r2n = __ldg(a.rstd + 2 * tn + 1);
    const float gate = a.gate ? __ldg(a.gate + t) : 1.f;
    F2 dn[CH][kPairs];  // dz, then dn, then dy / r1
    wait_groups<1>();   // the first four rows; Y may be pending
    if (a.dh) {
      F2 z[CH][kPairs], q[CH][kPairs];  // z r2, and dh wpre
      F2 m = mk(0.f);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        F2 w[kPairs];
        ring.vec(a.w_pre, c, 1.f, w);
        ring.read(0, c, q[c]);
        ring.read(1, c, z[c]);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          z[c][i] = mul2(z[c][i], mk(r2));
          s_pre[c][i] = fma2(q[c][i], z[c][i], s_pre[c][i]);
          q[c][i] = mul2(q[c][i], w[i]);
          m = fma2(q[c][i], z[c][i], m);
        }
      }
      const float mqz = -moe::block_sum_once(sum2(m), red[0]) * mean;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (a.dxo) {
          ring.read(2, c, dn[c]);
        } else {
#pragma unroll
          for (int i = 0; i < kPairs; ++i) dn[c][i] = mk(0.f);
        }
#pragma unroll
        for (int i = 0; i < kPairs; ++i)
          dn[c][i] = fma2(mk(r2), fma2(z[c][i], mk(mqz), q[c][i]), dn[c][i]);
      }
    } else {
#pragma unroll
      for (int c = 0; c < CH; ++c) ring.read(2, c, dn[c]);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      F2 w[kPairs];
      ring.vec(a.res, c, 1.f, w);
      if (a.dres) {
        F2 x[kPairs];
        ring.read(3, c, x);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) s_res[c][i] = fma2(dn[c][i], x[i], s_res[c][i]);
      }
#pragma unroll
      for (int i = 0; i < kPairs; ++i) w[i] = mul2(w[i], dn[c][i]);
      ring.store(static_cast<T*>(a.dx) + t * a.ld, c, w);
    }
    fill_head(t + step);
    if (a.y) {
      F2 n[CH][kPairs];
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < kPairs; ++i) n[c][i] = mk(0.f);
      wait_groups<1>();  // Y; the next token's first rows may be pending
#pragma unroll 1
      for (int j0 = 0; j0 < a.k; j0 += kRows)
#pragma unroll
        for (int jj = 0; jj < kRows; ++jj) {
          const int j = j0 + jj;
          const F2 w = mk(__shfl_sync(0xffffffffu, weight, j & 31));
          if ((rows >> (j & 31)) & 1) {  // none past k
#pragma unroll
            for (int c = 0; c < CH; ++c) {
              F2 v[kPairs];
              ring.read(4 + j, c, v);
#pragma unroll
              for (int i = 0; i < kPairs; ++i) n[c][i] = fma2(w, v[i], n[c][i]);
            }
          }
        }
      F2 dg = mk(0.f);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        F2 w[kPairs];
        ring.vec(a.w_post, c, 1.f, w);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          n[c][i] = mul2(n[c][i], mk(r1));
          const F2 g = mul2(mk(gate), dn[c][i]);
          s_post[c][i] = fma2(g, n[c][i], s_post[c][i]);
          dg = fma2(mul2(dn[c][i], w[i]), n[c][i], dg);
          dn[c][i] = mul2(g, w[i]);
        }
      }
      const float dgate = moe::block_sum_once(sum2(dg), red[1]);
      if (a.dgate && threadIdx.x == 0) a.dgate[t] = dgate;
      if (a.w_post) {  // the norm's part: dy / r1 = dn - n mean(dn n)
        const F2 m = mk(-dgate * gate * mean);
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int i = 0; i < kPairs; ++i) dn[c][i] = fma2(n[c][i], m, dn[c][i]);
      }
#pragma unroll 1
      for (int j0 = 0; j0 < a.k; j0 += kRows) {
        float q[kRows];
#pragma unroll
        for (int jj = 0; jj < kRows; ++jj) {
          const int j = j0 + jj;
          const F2 wr1 = mk(__shfl_sync(0xffffffffu, weight, j & 31) * r1);
          const size_t o = __shfl_sync(0xffffffffu, off, j & 31);
          const size_t on = __shfl_sync(0xffffffffu, offn, j & 31);
          F2 p = mk(0.f);
          if ((rows >> (j & 31)) & 1) {
            T* out = static_cast<T*>(a.dy) + o;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
              F2 v[kPairs], d[kPairs];
              if (a.dweights) {
                ring.read(4 + j, c, v);
#pragma unroll
                for (int i = 0; i < kPairs; ++i) p = fma2(dn[c][i], v[i], p);
              }
#pragma unroll
              for (int i = 0; i < kPairs; ++i) d[i] = mul2(wr1, dn[c][i]);
              ring.store(out, c, d);
            }
          }
          q[jj] = sum2(p);
          if ((rowsn >> (j & 31)) & 1) ring.copy(4 + j, Y + on);
        }
        if (a.dweights) {
          // kRows sums over the lanes at once: the halves of a pair of lanes take
          // one half of the values each, until a lane has one value left
          static_assert(kRows == 4, "two halving steps");
          const bool up = lane & 16, up2 = lane & 8;
          float u0 = up ? q[2] : q[0], u1 = up ? q[3] : q[1];
          u0 += __shfl_xor_sync(0xffffffffu, up ? q[0] : q[2], 16);
          u1 += __shfl_xor_sync(0xffffffffu, up ? q[1] : q[3], 16);
          float u = (up2 ? u1 : u0) + __shfl_xor_sync(0xffffffffu, up2 ? u0 : u1, 8);
#pragma unroll
          for (int o = 4; o; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
          const int j = j0 + (lane >> 3);
          if ((lane & 7) == 0 && j < a.k) dots[warp][j] = u;
        }
      }
      commit_group();
    } else {
      commit_group();  // no rows of Y: an empty group in their place
    }
    __syncthreads();  // dots are complete; `red` is free again
    if (a.dweights && (int)threadIdx.x < a.k) {
      float p = 0.f;
      for (int w = 0; w < warps; ++w) p += dots[w][threadIdx.x];
      a.dweights[t * a.k + threadIdx.x] = r1 * p;
    }
    off = offn, rows = rowsn, weight = weightn, r1 = r1n, r2 = r2n;
  }
  wait_groups<0>();
  float* part = a.part + (size_t)blockIdx.x * 3 * a.D;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    ring.put(part, c, s_res[c]);
    ring.put(part + a.D, c, s_post[c]);
    ring.put(part + 2 * (size_t)a.D, c, s_pre[c]);
  }
}

// Adds the CTAs' column sums: a warp's lanes take 32 columns, the CTA's warps
// an equal part of the partial sums each, in a fixed order.  Started while the
// pass over the tokens runs; waits for its end.
constexpr int kJoinWarps = 32;
__global__ void __launch_bounds__(32 * kJoinWarps)
    norm_join_kernel(const float* part, int blocks, int D, float* dres, float* dw_post,
                     float* dw_pre) {
  __shared__ float sums[kJoinWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + lane;
  float* out = i < D ? dres : (i < 2 * D ? dw_post : (i < 3 * D ? dw_pre : nullptr));
  float s = 0.f;
  moe::wait_for_earlier();
  if (out) {
    const int b1 = blocks * (warp + 1) / kJoinWarps;
#pragma unroll 8
    for (int b = blocks * warp / kJoinWarps; b < b1; ++b) s += __ldcg(part + (size_t)b * 3 * D + i);
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && out) {
    for (int w = 1; w < kJoinWarps; ++w) s += sums[w][lane];
    out[i % D] = s;
  }
}

// Chunks per thread and threads of a block.  Wide rows: two chunks as soon as
// two warps have one (the work of a token that does not depend on its width
// is done by every warp: 20 against 16 us at 4000 x 8 rows of 1024).
struct Shape {
  int ch, threads;
};
Shape shape_of(int D, bool wide) {
  const int chunks = (D + kChunk - 1) / kChunk;
  if (wide) {
    const int ch = chunks <= 64 ? 1 : (chunks <= 1024 ? 2 : 4);
    return {ch, std::min(kMaxThreads, ((chunks + ch - 1) / ch + 31) / 32 * 32)};
  }
  if (chunks <= 256) return {1, chunks <= 64 ? 64 : (chunks <= 128 ? 128 : 256)};
  return {chunks <= 1024 ? 2 : 4, chunks <= 512 ? 256 : 512};
}

constexpr size_t kSmemPerSm = 227 * 1024;

// CTAs: at most per_sm on every SM, and no more than the rounds of tokens need
// (the backward pass joins their column sums).
int grid_of(int T, int per_sm) {
  const int64_t most = (int64_t)std::max(sm_count(), 1) * per_sm;
  const int64_t rounds = ((int64_t)T + most - 1) / most;
  return rounds ? (int)((T + rounds - 1) / rounds) : 1;
}
int most_per_sm(int D, bool wide) {
  return std::max(1, std::min(8, 1024 / shape_of(D, wide).threads));
}

// Bytes of shared memory of a row in a Ring.
size_t ring_row(int D, size_t es, bool wide) {
  const Shape sh = shape_of(D, wide);
  const size_t extra = !wide && es == 2 ? (size_t)sh.ch * 4 * (sh.threads / 32) * 4 : 0;
  return (size_t)sh.ch * sh.threads * kChunk * es + (extra + 15) / 16 * 16;
}
// Rows of the forward ring: 7 with two CTAs per SM, else 3.
int forward_depth(int D, size_t es, bool wide) {
  return 7 * ring_row(D, es, wide) <= kSmemPerSm / 2 - 2048 ? 7 : 3;
}
// Bytes of shared memory of a token's rows in the backward pass; 0: too many
// (a Ring has 32 slots, a bit each).  Three more rows, filled a token ahead where
// they fit, did not pay: 280 against 273 us at 4096 x 8 rows of 7168.
size_t back_ring(int D, size_t es, int k, bool wide) {
  const size_t bytes = (size_t)(4 + k) * ring_row(D, es, wide);
  return 4 + k <= 32 && bytes <= kSmemPerSm - 8192 ? bytes : 0;
}

// Calls f with the element type, CH and NT (0: wide rows) as template arguments.
template <typename F>
void dispatch(int dtype, bool wide, Shape sh, F&& f) {
  auto by_shape = [&](auto t) {
    using std::integral_constant;
    auto with = [&](auto ch, auto nt) { f(t, ch, nt); };
    const integral_constant<int, 1> one;
    const integral_constant<int, 2> two;
    const integral_constant<int, 4> four;
    if (wide) {
      const integral_constant<int, 0> any;
      if (sh.ch == 1) with(one, any);
      else if (sh.ch == 2) with(two, any);
      else with(four, any);
    } else if (sh.ch == 1) {
      if (sh.threads == 64) with(one, integral_constant<int, 64>());
      else if (sh.threads == 128) with(one, integral_constant<int, 128>());
      else with(one, integral_constant<int, 256>());
    } else if (sh.ch == 2) {
      if (sh.threads == 256) with(two, integral_constant<int, 256>());
      else with(two, integral_constant<int, 512>());
    } else {
      with(four, integral_constant<int, 512>());
    }
  };
  if (dtype == SYMM_DTYPE_F32) by_shape(float());
  else if (dtype == SYMM_DTYPE_BF16) by_shape(__nv_bfloat16());
  else by_shape(__half());
}

int check_norm(const char* what, size_t ld, const void* y, size_t ldy, int dtype, int T, int D,
               int k) {
  if (!moe::dtype_ok(dtype))
    return fail(SYMM_EINVAL, std::string(what) + ": dtype must be SYMM_DTYPE_F16, _BF16 or _F32");
  if (T < 0 || D < 1 || D > SYMM_MOE_MAX_WIDTH)
    return fail(SYMM_EINVAL, std::string(what) + ": T must be >= 0 and D in [1, 16384]");
  if (y && (k < 1 || k > SYMM_MOE_MAX_TOPK || (uint64_t)T * (uint64_t)k >= (1ull << 31)))
    return fail(SYMM_EINVAL, std::string(what) + ": k must be in [1, 32] and T*k < 2^31");
  if (!y && k != 0) return fail(SYMM_EINVAL, std::string(what) + ": k must be 0 without y");
  if (ld < (size_t)D || ld > (1ull << 40) || (y && (ldy < (size_t)D || ldy > (1ull << 40))))
    return fail(SYMM_EINVAL, std::string(what) + ": ld and ldy must be at least D");
  return SYMM_OK;
}

bool all_aligned(size_t a, std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!moe::aligned(p, a)) return false;
  return true;
}

// Lets kernel f use `bytes` of dynamic shared memory: all that an SM has, once
// for each device.  The limit belongs to the kernel, whatever host thread
// launches it, so it never goes by one call's size.
int allow_smem(const void* f, size_t bytes, const char* what) {
  if (bytes <= 40 * 1024) return SYMM_OK;  // 48 KB with what the kernels hold statically
  int dev = 0;
  int rc = cuda_check(cudaGetDevice(&dev), what);
  if (rc) return rc;
  static std::mutex mu;
  static std::set<std::pair<const void*, int>> done;
  std::lock_guard<std::mutex> lock(mu);
  if (done.count({f, dev})) return SYMM_OK;
  cudaFuncAttributes attr;
  rc = cuda_check(cudaFuncGetAttributes(&attr, f), what);
  if (!rc)
    rc = cuda_check(cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)(kSmemPerSm - attr.sharedSizeBytes)), what);
  if (!rc) done.insert({f, dev});
  return rc;
}

}  // namespace

extern "C" int moe_block_norm_workspace(int T, int D, size_t* bytes) {
  return moe::entry("moe_block_norm_workspace", [&]() -> int {
    if (!bytes) return fail(SYMM_EINVAL, "moe_block_norm_workspace: NULL bytes");
    if (T < 0 || D < 1 || D > SYMM_MOE_MAX_WIDTH)
      return fail(SYMM_EINVAL, "moe_block_norm_workspace: T must be >= 0 and D in [1, 16384]");
    const int most = std::max(most_per_sm(D, true), most_per_sm(D, false));
    *bytes = ((size_t)grid_of(T, most) * 3 * D * 4 + 255) & ~(size_t)255;
    return SYMM_OK;
  });
}

extern "C" int moe_block_norm(const void* x, size_t ld, const void* y, size_t ldy,
                              const int32_t* rows, size_t yrows, const float* weights,
                              const float* gate, const float* res, const float* w_post,
                              const float* w_pre, float eps, int dtype, int T, int D, int k,
                              void* xo, void* h, float* rstd, void* stream) {
  return moe::entry("moe_block_norm", [&]() -> int {
    const char* what = "moe_block_norm";
    int rc = check_norm(what, ld, y, ldy, dtype, T, D, k);
    if (rc) return rc;
    if (!(eps > 0.f) || isinf(eps)) return fail(SYMM_EINVAL, "moe_block_norm: eps must be > 0");
    if (!y && (rows || weights || gate || res || w_post || xo))
      return fail(SYMM_EINVAL,
                  "moe_block_norm: without y, rows, weights, gate, res, w_post and xo must be "
                  "NULL");
    if (!y && !h) return fail(SYMM_EINVAL, "moe_block_norm: neither y nor h given");
    if (!h != !w_pre) return fail(SYMM_EINVAL, "moe_block_norm: h and w_pre go together");
    if (T == 0) return SYMM_OK;
    if (!x || (y && !xo)) return fail(SYMM_EINVAL, "moe_block_norm: NULL x or xo");
    if (h && (h == x || h == xo || h == y))
      return fail(SYMM_EINVAL, "moe_block_norm: h must not be an input or xo");
    if (xo && xo == y)  // other tokens' rows are still to be read
      return fail(SYMM_EINVAL, "moe_block_norm: xo must not be y");
    const size_t es = moe::dtype_bytes(dtype);
    if (!all_aligned(es, {x, y, xo, h}) ||
        !all_aligned(4, {rows, weights, gate, res, w_post, w_pre, rstd}))
      return fail(SYMM_EINVAL, "moe_block_norm: a pointer is not aligned to its elements");
    const bool al = D % kChunk == 0 && all_aligned(16, {x, y, xo, h}) && ld * es % 16 == 0 &&
                    (!y || ldy * es % 16 == 0) && all_aligned(16, {res, w_post, w_pre});
    const NormArgs a{x, ld, y, ldy, rows, yrows, weights, gate, res, w_post, w_pre, eps,
                     T, D, k, xo, h, rstd};
    const Shape sh = shape_of(D, al);
    cudaStream_t s = as_stream(stream);
    const int depth = forward_depth(D, es, al);
    const size_t ring = (size_t)depth * ring_row(D, es, al);
    const int per_sm = (int)std::max<size_t>(
        1, std::min<size_t>(1024 / sh.threads, (kSmemPerSm - 2048) / (ring + 1024)));
    rc = SYMM_OK;
    dispatch(dtype, al, sh, [&](auto t, auto c, auto n) {
      using E = decltype(t);
      constexpr int CH = decltype(c)::value, NT = decltype(n)::value;
      const auto kernel =
          depth == 7 ? norm_stream_kernel<E, CH, NT, 7> : norm_stream_kernel<E, CH, NT, 3>;
      rc = allow_smem((const void*)kernel, ring, "moe_block_norm: set-up");
      if (!rc)
        rc = moe::launch("moe_block_norm: launch", kernel, (unsigned)grid_of(T, per_sm),
                         (unsigned)sh.threads, ring, s, a);
    });
    return rc;
  });
}

extern "C" int moe_block_norm_backward(
    const void* dxo, const void* dh, const void* x, const void* xo, size_t ld, const void* y,
    size_t ldy, const int32_t* rows, size_t yrows, const float* weights, const float* gate,
    const float* res, const float* w_post, const float* w_pre, const float* rstd, int dtype, int T,
    int D, int k, void* dx, void* dy, float* dweights, float* dgate, float* dres, float* dw_post,
    float* dw_pre, void* workspace, void* stream) {
  return moe::entry("moe_block_norm_backward", [&]() -> int {
    const char* what = "moe_block_norm_backward";
    int rc = check_norm(what, ld, y, ldy, dtype, T, D, k);
    if (rc) return rc;
    if (!y && (rows || weights || gate || res || w_post || xo || dy || dweights || dgate || dres ||
               dw_post))
      return fail(SYMM_EINVAL, "moe_block_norm_backward: without y, rows, weights, gate, res, "
                               "w_post, xo and their gradients must be NULL");
    if (!dh != !w_pre)
      return fail(SYMM_EINVAL, "moe_block_norm_backward: dh and w_pre go together");
    if ((dw_pre && !w_pre) || (dw_post && !w_post) || (dres && !res) || (dgate && !gate) ||
        (dweights && !weights))
      return fail(SYMM_EINVAL, "moe_block_norm_backward: a gradient of an input that is NULL");
    if (T == 0 && !dres && !dw_post && !dw_pre) return SYMM_OK;
    if (T && (!x || !dx || !rstd || (y && (!xo || !dy)) || (!dxo && !dh)))
      return fail(SYMM_EINVAL, "moe_block_norm_backward: NULL input or output");
    if (!workspace || !moe::aligned(workspace, 16))
      return fail(SYMM_EINVAL,
                  "moe_block_norm_backward: workspace NULL or not 16-byte aligned");
    if (dy && (dy == y || dy == x || dy == xo || dy == dxo || dy == dh || dy == dx))
      return fail(SYMM_EINVAL, "moe_block_norm_backward: dy must not be another tensor");
    if (T && (dx == x || dx == xo || dx == dh || dx == y))
      return fail(SYMM_EINVAL, "moe_block_norm_backward: dx may only be dxo");
    const size_t es = moe::dtype_bytes(dtype);
    if (!all_aligned(es, {x, xo, y, dxo, dh, dx, dy}) ||
        !all_aligned(4, {rows, weights, gate, res, w_post, w_pre, rstd, dweights, dgate, dres,
                         dw_post, dw_pre}))
      return fail(SYMM_EINVAL,
                  "moe_block_norm_backward: a pointer is not aligned to its elements");
    const bool al = D % kChunk == 0 && all_aligned(16, {x, xo, y, dxo, dh, dx, dy}) &&
                    ld * es % 16 == 0 && (!y || ldy * es % 16 == 0) &&
                    all_aligned(16, {res, w_post, w_pre});
    const NormBackArgs a{dxo, dh, x, xo, ld, y, ldy, rows, yrows, weights, gate, res, w_post, w_pre,
                         rstd, T, D, k, dx, dy, dweights, dgate, dres, dw_post, dw_pre,
                         static_cast<float*>(workspace)};
    cudaStream_t s = as_stream(stream);
    if (T == 0) {  // empty sums
      for (float* p : {dres, dw_post, dw_pre})
        if (p && !rc)
          rc = cuda_check(cudaMemsetAsync(p, 0, (size_t)D * 4, s),
                          "moe_block_norm_backward: empty sums");
      return rc;
    }
    const Shape sh = shape_of(D, al);
    const size_t ring = back_ring(D, es, k, al);
    const int fit = ring ? (int)std::max<size_t>(1, (kSmemPerSm - 2048) / (ring + 6144)) : 8;
    const int grid = grid_of(T, std::min(most_per_sm(D, al), fit));
    rc = SYMM_OK;
    dispatch(dtype, al, sh, [&](auto t, auto c, auto n) {
      using E = decltype(t);
      constexpr int CH = decltype(c)::value, NT = decltype(n)::value;
      if (ring) {
        rc = allow_smem((const void*)norm_back_stream_kernel<E, CH, NT>, ring,
                        "moe_block_norm_backward: set-up");
        if (!rc)
          rc = moe::launch("moe_block_norm_backward: launch", norm_back_stream_kernel<E, CH, NT>,
                           (unsigned)grid, (unsigned)sh.threads, ring, s, a);
      } else {
        rc = moe::launch("moe_block_norm_backward: launch", norm_back_kernel<E, NT == 0, CH>,
                         (unsigned)grid, (unsigned)sh.threads, 0, s, a);
      }
    });
    if (rc || (!dres && !dw_post && !dw_pre)) return rc;
    return moe::launch("moe_block_norm_backward: join", norm_join_kernel,
                       (unsigned)((3 * D + 31) / 32), 32 * kJoinWarps, 0, s, a.part, grid, D, dres,
                       dw_post, dw_pre);
  });
}
