// moe_route.cu -- the router of a mixture of experts: per token the k largest
// logits and their softmax weights, per group the experts' counts and the
// balance and z losses, and the gradient with respect to the logits.
//
// Per token, with m = max_e l_e and s = sum_e exp(l_e - m), p_e = exp(l_e - m)/s:
//   w_j = scale p_j, or scale p_j / sum of the chosen p;
//   balance = E / (k n^2) sum_e c_e P_e,  P_e = sum_t p_te;   z = 1/n sum_t (m + log s)^2.
// Backward, counts constant, with a_e = E c_e / (k n^2) dbalance (+ scale dw_j
// at the chosen experts when they are not renormalised):
//   dl_e = p_e (a_e - sum_f p_f a_f + 2 (m + log s) / n dz)
//          (+ u_j (scale dw_j - sum_i u_i scale dw_i), u the chosen softmax, otherwise).
//
// One warp per token, its logits in registers.  The sums over tokens stay in
// a warp's registers over all its tokens, are joined per CTA in shared memory
// and across CTAs by a second small kernel that adds the partial sums in CTA
// order, so equal inputs give equal bits.
#include <algorithm>
#include <type_traits>

#include "moe_common.cuh"

using namespace symm_host;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct RouteArgs {
  const void* logits;
  size_t ld;
  const uint8_t* mask;
  int G, T, E, k, renorm, blocks;  // blocks: CTAs per group
  float scale;
  int32_t* experts;
  float* weights;
  int32_t* counts;
  int32_t* tokens;
  float* stats;
  float* loss;
  float* part;  // [G][blocks][2E + 2]: P, counts (int), z sum, valid tokens (int)
};

// NaN -> -infinity, +infinity -> the largest finite value
__device__ __forceinline__ float clean(float v) {
  return v != v ? -INFINITY : fminf(v, 3.402823466e38f);
}

// The losses of one group from its sums: every thread takes experts threadIdx.x, ...
__device__ __forceinline__ void finish_group(const RouteArgs& a, int g, float dot, float zsum,
                                             int n) {
  if (threadIdx.x == 0) {
    const float n1 = (float)(n > 0 ? n : 1);
    a.tokens[g] = n;
    a.loss[2 * g] = dot * ((float)a.E / (float)a.k) / n1 / n1;
    a.loss[2 * g + 1] = zsum / n1;
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) route_kernel(const RouteArgs a) {
  extern __shared__ float smem[];  // P [E] per warp in turn, counts [E]
  float* sp = smem;
  int* sc = reinterpret_cast<int*>(smem + a.E);
  __shared__ float red[kWarps];
  __shared__ float sz[kWarps];
  __shared__ int sn[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = blockIdx.x / a.blocks, b = blockIdx.x % a.blocks;
  for (int e = threadIdx.x; e < a.E; e += kThreads) sp[e] = 0.f, sc[e] = 0;
  __syncthreads();
  float psum[V];
#pragma unroll
  for (int v = 0; v < V; ++v) psum[v] = 0.f;
  float zsum = 0.f;
  int n = 0;
  for (int t = b * kWarps + warp; t < a.T; t += a.blocks * kWarps) {
    const size_t row = (size_t)g * a.T + t;
    const T* src = static_cast<const T*>(a.logits) + row * a.ld;
    float l[V];
    float m = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = lane + 32 * v;
      l[v] = e < a.E ? clean(moe::to_f(src[e])) : -INFINITY;
      m = fmaxf(m, l[v]);
    }
    m = moe::warp_max(m);
    const bool valid = (!a.mask || a.mask[row]) && m > -INFINITY;
    if (!valid) {
      if (lane < a.k) {
        a.experts[row * a.k + lane] = -1;
        a.weights[row * a.k + lane] = 0.f;
      }
      if (lane < 2) a.stats[2 * row + lane] = 0.f;
      continue;
    }
    float p[V];
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) s += p[v] = expf(l[v] - m);
    s = moe::warp_sum(s);
    const float inv = 1.f / s;
#pragma unroll
    for (int v = 0; v < V; ++v) psum[v] += p[v] * inv;
    const float lse = m + logf(s);
    zsum += lse * lse;
    ++n;
    // k rounds of the largest remaining logit; round j's winner stays in lane j
    float mine = -INFINITY;
    int chosen = -1;
    for (int j = 0; j < a.k; ++j) {
      float best = -INFINITY;
      int at = 0x7fffffff;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (l[v] > best) best = l[v], at = lane + 32 * v;
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const float ob = __shfl_xor_sync(0xffffffffu, best, o);
        const int oa = __shfl_xor_sync(0xffffffffu, at, o);
        if (ob > best || (ob == best && oa < at)) best = ob, at = oa;
      }
      if (best == -INFINITY) break;
      if (lane == j) mine = best, chosen = at;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (at == lane + 32 * v) l[v] = -INFINITY;
    }
    const float u = expf(mine - m);  // 0 where nothing was chosen
    const float total = a.renorm ? moe::warp_sum(u) : s;
    if (lane < a.k) {
      a.experts[row * a.k + lane] = chosen;
      a.weights[row * a.k + lane] = a.scale * (u / total);
      if (chosen >= 0) atomicAdd(&sc[chosen], 1);
    }
    if (lane == 0) a.stats[2 * row] = m, a.stats[2 * row + 1] = s;
  }
  if (lane == 0) sz[warp] = zsum, sn[warp] = n;
  for (int w = 0; w < kWarps; ++w) {  // warps in order: a fixed order of the sum
    if (w == warp) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (lane + 32 * v < a.E) sp[lane + 32 * v] += psum[v];
    }
    __syncthreads();
  }
  zsum = 0.f, n = 0;
  for (int w = 0; w < kWarps; ++w) zsum += sz[w], n += sn[w];
  if (a.blocks == 1) {
    float dot = 0.f;
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
      a.counts[(size_t)g * a.E + e] = sc[e];
      dot += sp[e] * (float)sc[e];
    }
    dot = moe::block_sum(dot, red);
    finish_group(a, g, dot, zsum, n);
    return;
  }
  float* part = a.part + (size_t)blockIdx.x * (2 * a.E + 2);
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    part[e] = sp[e];
    part[a.E + e] = __int_as_float(sc[e]);
  }
  if (threadIdx.x == 0) part[2 * a.E] = zsum, part[2 * a.E + 1] = __int_as_float(n);
}

// One CTA per group adds the CTAs' partial sums in their order.
__global__ void __launch_bounds__(kThreads) route_join_kernel(const RouteArgs a) {
  __shared__ float red[kWarps];
  const int g = blockIdx.x;
  const size_t step = 2 * a.E + 2;
  const float* part = a.part + (size_t)g * a.blocks * step;
  float dot = 0.f;
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    float p = 0.f;
    int c = 0;
    for (int b = 0; b < a.blocks; ++b) {
      p += part[b * step + e];
      c += __float_as_int(part[b * step + a.E + e]);
    }
    a.counts[(size_t)g * a.E + e] = c;
    dot += p * (float)c;
  }
  dot = moe::block_sum(dot, red);
  float z = 0.f;
  int n = 0;
  if (threadIdx.x == 0)
    for (int b = 0; b < a.blocks; ++b) {
      z += part[b * step + 2 * a.E];
      n += __float_as_int(part[b * step + 2 * a.E + 1]);
    }
  finish_group(a, g, dot, z, n);
}

struct RouteBackArgs {
  const void* logits;
  size_t ld;
  int G, T, E, k, renorm;
  float scale;
  const int32_t* experts;
  const int32_t* counts;
  const int32_t* tokens;
  const float* stats;
  const float* dweights;
  const float* dloss;
  void* dlogits;
  size_t ldd;
};

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) route_back_kernel(const RouteBackArgs a) {
  const int lane = threadIdx.x & 31;
  const size_t rows = (size_t)a.G * a.T;
  const size_t nwarps = (size_t)gridDim.x * kWarps;
  for (size_t row = (size_t)blockIdx.x * kWarps + (threadIdx.x >> 5); row < rows; row += nwarps) {
    const int g = (int)(row / a.T);
    const T* src = static_cast<const T*>(a.logits) + row * a.ld;
    T* dst = static_cast<T*>(a.dlogits) + row * a.ldd;
    int at = -1;
    float dw = 0.f;
    if (lane < a.k) {
      at = a.experts[row * a.k + lane];
      if (at >= a.E) at = -1;
      if (at >= 0 && a.dweights) dw = a.scale * a.dweights[row * a.k + lane];
    }
    if (__shfl_sync(0xffffffffu, at, 0) < 0) {  // an invalid token
      for (int e = lane; e < a.E; e += 32) dst[e] = moe::from_f<T>(0.f);
      continue;
    }
    const float m = a.stats[2 * row], s = a.stats[2 * row + 1], inv = 1.f / s;
    const float n = (float)max(a.tokens[g], 1);
    const float cb = a.dloss ? a.dloss[2 * g] * ((float)a.E / (float)a.k) / n / n : 0.f;
    const float cz = a.dloss ? (2.f * a.dloss[2 * g + 1] / n) * (m + logf(s)) : 0.f;
    float p[V], d[V];
    float dot = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = lane + 32 * v;
      p[v] = e < a.E ? expf(clean(moe::to_f(src[e])) - m) * inv : 0.f;
      d[v] = e < a.E ? cb * (float)a.counts[(size_t)g * a.E + e] : 0.f;
      dot += p[v] * d[v];
    }
    // the chosen experts' own probabilities, in the lanes of their slots
    const float u = at >= 0 ? expf(clean(moe::to_f(src[at])) - m) * inv : 0.f;
    float add = dw;  // to a (before the softmax's Jacobian), or to dl if renormalised
    if (a.renorm) {
      const float q = u / moe::warp_sum(u);
      add = q * (dw - moe::warp_sum(q * dw));
    } else {
      dot += u * dw;
    }
    dot = moe::warp_sum(dot);
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] = p[v] * (d[v] - dot + cz);
    for (int j = 0; j < a.k; ++j) {
      const int e = __shfl_sync(0xffffffffu, at, j);
      const float x = __shfl_sync(0xffffffffu, add, j);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (e == lane + 32 * v) d[v] += a.renorm ? x : p[v] * x;
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (lane + 32 * v < a.E) dst[lane + 32 * v] = moe::from_f<T>(d[v]);
  }
}

// Calls f with the element type's and the register count's template arguments.
template <typename F>
void for_type(int dtype, F&& f) {
  if (dtype == SYMM_DTYPE_F32) f(float());
  else if (dtype == SYMM_DTYPE_BF16) f(__nv_bfloat16());
  else f(__half());
}
template <typename F>
void for_width(int E, F&& f) {
  if (E <= 32) f(std::integral_constant<int, 1>());
  else if (E <= 64) f(std::integral_constant<int, 2>());
  else if (E <= 128) f(std::integral_constant<int, 4>());
  else if (E <= 256) f(std::integral_constant<int, 8>());
  else if (E <= 512) f(std::integral_constant<int, 16>());
  else f(std::integral_constant<int, 32>());
}

// CTAs per group: one token per warp until the GPU is full, then several.
int route_blocks(int G, int T) {
  const int sms = std::max(sm_count(), 1);
  const int want = (T + kWarps - 1) / kWarps;
  const int most = std::max(1, 4 * sms / std::max(G, 1));
  return std::max(1, std::min(want, most));
}

int check_route(const char* what, size_t ld, int dtype, int G, int T, int E, int k) {
  if (!moe::dtype_ok(dtype))
    return fail(SYMM_EINVAL, std::string(what) + ": dtype must be SYMM_DTYPE_F16, _BF16 or _F32");
  if (G < 0 || T < 0 || (uint64_t)G * (uint64_t)T >= (1ull << 31))
    return fail(SYMM_EINVAL, std::string(what) + ": G and T must be >= 0 and G*T < 2^31");
  if (E < 1 || E > SYMM_MOE_MAX_EXPERTS)
    return fail(SYMM_EINVAL, std::string(what) + ": E must be in [1, 1024]");
  if (k < 1 || k > E || k > SYMM_MOE_MAX_TOPK)
    return fail(SYMM_EINVAL, std::string(what) + ": k must be in [1, min(E, 32)]");
  if (ld < (size_t)E || ld > (1ull << 40))
    return fail(SYMM_EINVAL, std::string(what) + ": ld must be at least E");
  return SYMM_OK;
}

}  // namespace

extern "C" int moe_route_workspace(int G, int T, int E, size_t* bytes) {
  return moe::entry("moe_route_workspace", [&]() -> int {
    if (!bytes) return fail(SYMM_EINVAL, "moe_route_workspace: NULL bytes");
    int rc = check_route("moe_route_workspace", (size_t)std::max(E, 0), SYMM_DTYPE_F32, G, T, E, 1);
    if (rc) return rc;
    *bytes = ((size_t)G * route_blocks(G, T) * (2 * (size_t)E + 2) * 4 + 255) & ~(size_t)255;
    return SYMM_OK;
  });
}

extern "C" int moe_route(const void* logits, size_t ld, const uint8_t* mask, int dtype, int G,
                         int T, int E, int k, int renorm, float scale, int32_t* experts,
                         float* weights, int32_t* counts, int32_t* tokens, float* stats,
                         float* loss, void* workspace, void* stream) {
  return moe::entry("moe_route", [&]() -> int {
    int rc = check_route("moe_route", ld, dtype, G, T, E, k);
    if (rc) return rc;
    if (!(scale == scale) || isinf(scale))
      return fail(SYMM_EINVAL, "moe_route: scale must be finite");
    if (G == 0) return SYMM_OK;
    if ((T && (!logits || !experts || !weights || !stats)) || !counts || !tokens || !loss ||
        !workspace)
      return fail(SYMM_EINVAL, "moe_route: NULL logits, output or workspace");
    if (!moe::aligned(logits, moe::dtype_bytes(dtype)) || !moe::aligned(experts, 4) ||
        !moe::aligned(weights, 4) || !moe::aligned(counts, 4) || !moe::aligned(tokens, 4) ||
        !moe::aligned(stats, 4) || !moe::aligned(loss, 4) || !moe::aligned(workspace, 16))
      return fail(SYMM_EINVAL, "moe_route: a pointer is not aligned to its elements");
    RouteArgs a{logits, ld, mask, G, T, E, k, renorm ? 1 : 0, route_blocks(G, T), scale, experts,
                weights, counts, tokens, stats, loss, static_cast<float*>(workspace)};
    cudaStream_t s = as_stream(stream);
    for_type(dtype, [&](auto t) {
      for_width(E, [&](auto v) {
        route_kernel<decltype(t), decltype(v)::value>
            <<<(unsigned)(G * a.blocks), kThreads, 2 * (size_t)E * 4, s>>>(a);
      });
    });
    rc = cuda_check(cudaGetLastError(), "moe_route: launch");
    if (rc || a.blocks == 1) return rc;
    route_join_kernel<<<(unsigned)G, kThreads, 0, s>>>(a);
    return cuda_check(cudaGetLastError(), "moe_route: join");
  });
}

extern "C" int moe_route_backward(const void* logits, size_t ld, int dtype, int G, int T, int E,
                                  int k, int renorm, float scale, const int32_t* experts,
                                  const int32_t* counts, const int32_t* tokens, const float* stats,
                                  const float* dweights, const float* dloss, void* dlogits,
                                  size_t ldd, void* stream) {
  return moe::entry("moe_route_backward", [&]() -> int {
    int rc = check_route("moe_route_backward", std::min(ld, ldd), dtype, G, T, E, k);
    if (!rc && std::max(ld, ldd) > (1ull << 40))
      rc = fail(SYMM_EINVAL, "moe_route_backward: ld too large");
    if (rc) return rc;
    if (!(scale == scale) || isinf(scale))
      return fail(SYMM_EINVAL, "moe_route_backward: scale must be finite");
    if (G == 0 || T == 0) return SYMM_OK;
    if (!logits || !experts || !counts || !tokens || !stats || !dlogits)
      return fail(SYMM_EINVAL, "moe_route_backward: NULL input or output");
    if (logits == dlogits && ld != ldd)
      return fail(SYMM_EINVAL, "moe_route_backward: in place, ldd must be ld");
    if (!moe::aligned(logits, moe::dtype_bytes(dtype)) ||
        !moe::aligned(dlogits, moe::dtype_bytes(dtype)) || !moe::aligned(experts, 4) ||
        !moe::aligned(counts, 4) || !moe::aligned(tokens, 4) || !moe::aligned(stats, 4) ||
        !moe::aligned(dweights, 4) || !moe::aligned(dloss, 4))
      return fail(SYMM_EINVAL, "moe_route_backward: a pointer is not aligned to its elements");
    RouteBackArgs a{logits, ld, G, T, E, k, renorm ? 1 : 0, scale, experts, counts, tokens, stats,
                    dweights, dloss, dlogits, ldd};
    const size_t rows = (size_t)G * T;
    const unsigned grid = (unsigned)std::min<size_t>((rows + kWarps - 1) / kWarps,
                                                     (size_t)std::max(sm_count(), 1) * 8);
    cudaStream_t s = as_stream(stream);
    for_type(dtype, [&](auto t) {
      for_width(E, [&](auto v) {
        route_back_kernel<decltype(t), decltype(v)::value><<<grid, kThreads, 0, s>>>(a);
      });
    });
    return cuda_check(cudaGetLastError(), "moe_route_backward: launch");
  });
}
