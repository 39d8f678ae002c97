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
//   dw_j = <dy, Y_j> = r1 (<dn, Y_j> - mean(dn n) <n, Y_j>).
// The last form needs no second pass over Y once mean(dn n) is known: both
// inner products are sums of the pass that finds it.
//
// One CTA per token at a time; a thread owns the same columns in every token
// of its CTA (up to 4 chunks of 8), so the column sums of dres, dwpost and
// dwpre stay in its registers over all tokens and are written once per CTA;
// a second small kernel adds the CTAs' sums in order.
#include <algorithm>
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
  // chunk c of a float vector (any 4-byte alignment); `none` where it is NULL
  __device__ __forceinline__ void vec(const float* p, int c, float none,
                                      float (&v)[kChunk]) const {
#pragma unroll
    for (int i = 0; i < kChunk; ++i) v[i] = p ? (at(c, i) < D ? p[at(c, i)] : 0.f) : none;
  }
};

// Row j of token t in Y, or -1.
__device__ __forceinline__ long long row_of(const int32_t* rows, size_t yrows, size_t slot) {
  const long long r = rows ? (long long)rows[slot] : (long long)slot;
  return r >= 0 && r < (long long)yrows ? r : -1;
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

template <typename T, bool ALIGNED, int CH>
__global__ void __launch_bounds__(kMaxThreads) norm_kernel(const NormArgs a) {
  __shared__ float red[kMaxWarps];
  const Cols<T, ALIGNED> cols{a.D};
  const float mean = 1.f / (float)a.D;
  for (size_t t = blockIdx.x; t < (size_t)a.T; t += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + t * a.ld;
    float z[CH][kChunk];
    float r1 = 1.f, r2 = 1.f;
    if (a.y) {
      float ss = 0.f;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        weighted<T>(a, cols, t, c, z[c]);
#pragma unroll
        for (int i = 0; i < kChunk; ++i) ss = fmaf(z[c][i], z[c][i], ss);
      }
      if (a.w_post) r1 = 1.f / sqrtf(moe::block_sum(ss, red) * mean + a.eps);
      const float s = (a.gate ? a.gate[t] : 1.f) * r1;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        float v[kChunk], res[kChunk], w[kChunk];
        cols.load(x, c, v);
        cols.vec(a.res, c, 1.f, res);
        cols.vec(a.w_post, c, 1.f, w);
#pragma unroll
        for (int i = 0; i < kChunk; ++i) z[c][i] = fmaf(s * w[i], z[c][i], res[i] * v[i]);
        cols.store(static_cast<T*>(a.xo) + t * a.ld, c, z[c]);
      }
    } else {
#pragma unroll
      for (int c = 0; c < CH; ++c) cols.load(x, c, z[c]);
    }
    if (a.h) {
      float ss = 0.f;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < kChunk; ++i) ss = fmaf(z[c][i], z[c][i], ss);
      r2 = 1.f / sqrtf(moe::block_sum(ss, red) * mean + a.eps);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        float w[kChunk];
        cols.vec(a.w_pre, c, 1.f, w);
#pragma unroll
        for (int i = 0; i < kChunk; ++i) w[i] *= z[c][i] * r2;
        cols.store(static_cast<T*>(a.h) + t * a.ld, c, w);
      }
    }
    if (a.rstd && threadIdx.x == 0) a.rstd[2 * t] = r1, a.rstd[2 * t + 1] = r2;
  }
}

template <typename T, bool ALIGNED, int CH>
__global__ void __launch_bounds__(kMaxThreads) norm_back_kernel(const NormBackArgs a) {
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

// Adds the CTAs' column sums in their order.
__global__ void norm_join_kernel(const float* part, int blocks, int D, float* dres, float* dw_post,
                                 float* dw_pre) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= 3 * D) return;
  float* out = i < D ? dres : (i < 2 * D ? dw_post : dw_pre);
  if (!out) return;
  float s = 0.f;
  for (int b = 0; b < blocks; ++b) s += part[(size_t)b * 3 * D + i];
  out[i % D] = s;
}

struct Shape {
  int ch, threads;
};
Shape shape_of(int D) {
  const int chunks = (D + kChunk - 1) / kChunk;
  const int ch = chunks <= 256 ? 1 : (chunks <= 1024 ? 2 : 4);
  return {ch, std::min(kMaxThreads, ((chunks + ch - 1) / ch + 31) / 32 * 32)};
}
int grid_of(int T, int D) {
  const int per_sm = std::max(1, 1024 / shape_of(D).threads);
  return std::max(1, std::min(T, std::max(sm_count(), 1) * std::min(per_sm, 8)));
}

template <typename F>
void dispatch(int dtype, bool al, int ch, F&& f) {
  auto by_ch = [&](auto t, auto b) {
    if (ch == 1) f(t, b, std::integral_constant<int, 1>());
    else if (ch == 2) f(t, b, std::integral_constant<int, 2>());
    else f(t, b, std::integral_constant<int, 4>());
  };
  auto by_align = [&](auto t) {
    if (al) by_ch(t, std::true_type());
    else by_ch(t, std::false_type());
  };
  if (dtype == SYMM_DTYPE_F32) by_align(float());
  else if (dtype == SYMM_DTYPE_BF16) by_align(__nv_bfloat16());
  else by_align(__half());
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

}  // namespace

extern "C" int moe_block_norm_workspace(int T, int D, size_t* bytes) {
  return moe::entry("moe_block_norm_workspace", [&]() -> int {
    if (!bytes) return fail(SYMM_EINVAL, "moe_block_norm_workspace: NULL bytes");
    if (T < 0 || D < 1 || D > SYMM_MOE_MAX_WIDTH)
      return fail(SYMM_EINVAL, "moe_block_norm_workspace: T must be >= 0 and D in [1, 16384]");
    *bytes = ((size_t)grid_of(T, D) * 3 * D * 4 + 255) & ~(size_t)255;
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
                  "moe_block_norm: without y, rows, weights, gate, res, w_post and xo must be NULL");
    if (!y && !h) return fail(SYMM_EINVAL, "moe_block_norm: neither y nor h given");
    if (!h != !w_pre) return fail(SYMM_EINVAL, "moe_block_norm: h and w_pre go together");
    if (T == 0) return SYMM_OK;
    if (!x || (y && !xo)) return fail(SYMM_EINVAL, "moe_block_norm: NULL x or xo");
    if (h && (h == x || h == xo || h == y))
      return fail(SYMM_EINVAL, "moe_block_norm: h must not be an input or xo");
    const size_t es = moe::dtype_bytes(dtype);
    if (!all_aligned(es, {x, y, xo, h}) ||
        !all_aligned(4, {rows, weights, gate, res, w_post, w_pre, rstd}))
      return fail(SYMM_EINVAL, "moe_block_norm: a pointer is not aligned to its elements");
    const bool al = D % kChunk == 0 && all_aligned(16, {x, y, xo, h}) && ld * es % 16 == 0 &&
                    (!y || ldy * es % 16 == 0);
    const NormArgs a{x, ld, y, ldy, rows, yrows, weights, gate, res, w_post, w_pre, eps,
                     T, D, k, xo, h, rstd};
    const Shape sh = shape_of(D);
    cudaStream_t s = as_stream(stream);
    dispatch(dtype, al, sh.ch, [&](auto t, auto b, auto c) {
      norm_kernel<decltype(t), decltype(b)::value, decltype(c)::value>
          <<<(unsigned)grid_of(T, D), sh.threads, 0, s>>>(a);
    });
    return cuda_check(cudaGetLastError(), "moe_block_norm: launch");
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
                    ld * es % 16 == 0 && (!y || ldy * es % 16 == 0);
    const NormBackArgs a{dxo, dh, x, xo, ld, y, ldy, rows, yrows, weights, gate, res, w_post, w_pre,
                         rstd, T, D, k, dx, dy, dweights, dgate, dres, dw_post, dw_pre,
                         static_cast<float*>(workspace)};
    const Shape sh = shape_of(D);
    const int grid = grid_of(T, D);
    cudaStream_t s = as_stream(stream);
    dispatch(dtype, al, sh.ch, [&](auto t, auto b, auto c) {
      norm_back_kernel<decltype(t), decltype(b)::value, decltype(c)::value>
          <<<(unsigned)grid, sh.threads, 0, s>>>(a);
    });
    rc = cuda_check(cudaGetLastError(), "moe_block_norm_backward: launch");
    if (rc || (!dres && !dw_post && !dw_pre)) return rc;
    norm_join_kernel<<<(unsigned)((3 * D + 255) / 256), 256, 0, s>>>(a.part, grid, D, dres, dw_post,
                                                                    dw_pre);
    return cuda_check(cudaGetLastError(), "moe_block_norm_backward: join");
  });
}
