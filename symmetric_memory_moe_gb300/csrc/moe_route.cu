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
// One warp per token, V consecutive logits per lane in registers, the next
// token's on their way.  The choice costs more than all the rest: k rounds of
// the warp's largest remaining key.  16-bit logits become unique 32-bit keys,
// the logit's order above the expert's (complemented) number, which each lane
// sorts once, so that a round is one warp-wide maximum and the winner moves up
// its list; 32-bit logits are compared as they are, and the winner looks for its
// next one.  The sums over tokens stay in a warp's registers over all its
// tokens, are joined per CTA in shared memory and across CTAs by a second
// small kernel, in a fixed order, so equal inputs give equal bits.
//
// Bound by what can be issued: 413 instructions a token at 256 bf16 logits
// and k = 8, half of them minima, maxima and selects, which issue at half rate
// (0.65 a cycle and scheduler).  8 x 4096 tokens take 24.4 us (2.8 would be HBM's),
// the backward pass with 32-bit logits 17.4 (4.0 TB/s; 10.2 us at the copy rate),
// 8 tokens 6.1, of which the kernel is 3.4.  So exp, log and quotients are the
// approximate instructions.  Against 64 bits (2-norm) the weights err by 5.8e-8
// and the gradient by 8.5e-8 there, 3.9e-8 to 5.2e-8 and 7.7e-8 with the full
// functions, which take 27.1 and 20.8 us.
#include <algorithm>
#include <type_traits>

#include "moe_common.cuh"

using namespace symm_host;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kJoinThreads = 1024;
constexpr unsigned kAll = 0xffffffffu;

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

// A lane's logits: experts lane*V .. lane*V + V - 1 of a row, as they lie in
// memory.  VEC: rows and E are such that a lane's V logits are whole aligned
// vectors.
template <typename T, int V, bool VEC>
struct Raw {
  static constexpr int kBytes = V * (int)sizeof(T);
  static constexpr int kUnit = kBytes < 16 ? kBytes : 16;
  alignas(kUnit) T v[V];
  __device__ __forceinline__ void load(const T* row, int E, int lane) {
    const int e0 = lane * V;
    if constexpr (VEC) {
      if (e0 >= E) return;
      if constexpr (kUnit == 16) {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i)
          reinterpret_cast<uint4*>(v)[i] = reinterpret_cast<const uint4*>(row + e0)[i];
      } else if constexpr (kUnit == 8) {
        *reinterpret_cast<uint2*>(v) = *reinterpret_cast<const uint2*>(row + e0);
      } else if constexpr (kUnit == 4) {
        *reinterpret_cast<uint32_t*>(v) = *reinterpret_cast<const uint32_t*>(row + e0);
      } else {
        v[0] = row[e0];
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (e0 + i < E) v[i] = row[e0 + i];
    }
  }
  // the logit as the operator counts it; -infinity past E
  __device__ __forceinline__ float at(int i, int E, int lane) const {
    return lane * V + i < E ? clean(moe::to_f(v[i])) : -INFINITY;
  }
  __device__ __forceinline__ static void store(T* row, int E, int lane, const float (&d)[V]) {
    const int e0 = lane * V;
    alignas(16) T o[V];
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = moe::from_f<T>(d[i]);
    if constexpr (VEC) {
      if (e0 >= E) return;
      if constexpr (kUnit == 16) {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i)
          reinterpret_cast<uint4*>(row + e0)[i] = reinterpret_cast<const uint4*>(o)[i];
      } else if constexpr (kUnit == 8) {
        *reinterpret_cast<uint2*>(row + e0) = *reinterpret_cast<const uint2*>(o);
      } else if constexpr (kUnit == 4) {
        *reinterpret_cast<uint32_t*>(row + e0) = *reinterpret_cast<const uint32_t*>(o);
      } else {
        row[e0] = o[0];
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (e0 + i < E) row[e0 + i] = o[i];
    }
  }
};

// A lane's V floats in shared memory, 16 bytes at a time.
template <int V>
__device__ __forceinline__ void put(float* p, const float (&x)[V]) {
  if constexpr (V >= 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = x[i];
  }
}
template <int V>
__device__ __forceinline__ void get(const float* p, float (&x)[V]) {
  if constexpr (V >= 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 f = *reinterpret_cast<const float4*>(p + i);
      x[i] = f.x, x[i + 1] = f.y, x[i + 2] = f.z, x[i + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = p[i];
  }
}

// exp of a number that is not above 0, or of -infinity
__device__ __forceinline__ float exp_of(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
  return r;
}

// Order of a 16-bit float as an unsigned number, and back.
__device__ __forceinline__ uint32_t order16(uint32_t bits) {
  return (bits & 0x8000u) ? 0xffffu - bits : bits | 0x8000u;
}
__device__ __forceinline__ uint32_t unorder16(uint32_t o) {
  return (o & 0x8000u) ? o & 0x7fffu : 0xffffu - o;
}

__device__ __forceinline__ void larger_first(uint32_t& a, uint32_t& b) {
  const uint32_t hi = max(a, b), lo = min(a, b);
  a = hi, b = lo;
}
// Batcher's odd-even merge sort of a lane's keys, largest first.
template <int V>
__device__ __forceinline__ void sort_keys(uint32_t (&k)[V]) {
  static_assert(V <= 8, "a network for up to 8");
  if constexpr (V >= 2) {
#pragma unroll
    for (int i = 0; i < V; i += 2) larger_first(k[i], k[i + 1]);
  }
  if constexpr (V >= 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      larger_first(k[i], k[i + 2]), larger_first(k[i + 1], k[i + 3]);
      larger_first(k[i + 1], k[i + 2]);
    }
  }
  if constexpr (V == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) larger_first(k[i], k[i + 4]);
    larger_first(k[2], k[4]), larger_first(k[3], k[5]);
    larger_first(k[1], k[2]), larger_first(k[3], k[4]), larger_first(k[5], k[6]);
  }
}

// The choices of a token: after choose(), lane j < k has the j-th expert (or
// -1) and its logit, and every lane the largest logit (-infinity: none left).
struct Choice {
  int expert;
  float logit, top;
};

// k rounds: `round(j, live)` takes the largest key left and moves the winner up
// its list, of which no more than `live` keys can still matter.  Rounds after
// the lists have run empty find "none" again.  Up to 8 rounds are unrolled for
// the k that it is: 8 x 4096 tokens of 256 bf16 logits take 22.5 us at k = 4 and
// 23.6 at 6, against 23.8 and 24.5 with a test of k in every round.
template <int K, typename F>
__device__ __forceinline__ void unrolled(F&& round) {
#pragma unroll
  for (int j = 0; j < K; ++j) round(j, K - j);
}
template <typename F>
__device__ __forceinline__ void rounds(int k, F&& round) {
  switch (k) {
    case 1: return unrolled<1>(round);
    case 2: return unrolled<2>(round);
    case 3: return unrolled<3>(round);
    case 4: return unrolled<4>(round);
    case 5: return unrolled<5>(round);
    case 6: return unrolled<6>(round);
    case 7: return unrolled<7>(round);
    case 8: return unrolled<8>(round);
  }
  for (int j = 0; j < k; ++j) round(j, 9);  // 9: a list may run empty
}
// The winner of a lane's list moves up.
template <int V>
__device__ __forceinline__ void pop(uint32_t (&key)[V], bool win, int live) {
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i + 1 < live) key[i] = win ? (i + 1 < V ? key[i + 1] : 0u) : key[i];
}

// 16-bit logits, lists of up to 8.  l: the logits as the operator counts them.
template <typename T, int V, bool VEC>
__device__ __forceinline__ Choice choose16(const Raw<T, V, VEC>& raw, int E, int k, int lane,
                                           float (&l)[V]) {
  constexpr uint32_t kInf = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
  const uint32_t last = 0xffffu - (uint32_t)(lane * V);  // complement of the first expert
  uint32_t key[V];
  if constexpr (V >= 2) {
    // two logits at a time: -0 made +0 (and NaN one pattern) by adding +0, then
    // the order of unsigned numbers in both halves
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2,
                                         __nv_bfloat162>::type;
    uint32_t x[V / 2], most = 0, least = 0xffffffffu;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      uint32_t w = reinterpret_cast<const uint32_t*>(raw.v)[i];
      const uint32_t zero = 0;
      const T2 s = __hadd2(*reinterpret_cast<const T2*>(&w), *reinterpret_cast<const T2*>(&zero));
      w = *reinterpret_cast<const uint32_t*>(&s);
      x[i] = w ^ ((((w >> 15) & 0x00010001u) * 0xffffu) | 0x80008000u);
      most = __vmaxu2(most, x[i]);
      least = __vminu2(least, x[i]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      key[i] = __byte_perm(last - i, x[i / 2], i % 2 ? 0x7610 : 0x5410);
    const bool active = lane * V < E;
    // from the lowest finite order to the highest in both halves, all V of them?
    constexpr uint32_t kLow = 0xffffu - (0x8000u | (kInf - 1)), kHigh = 0x8000u | (kInf - 1);
    const bool plain = !active || (lane * V + V <= E && (most >> 16) <= kHigh &&
                                   (most & 0xffffu) <= kHigh && (least >> 16) >= kLow &&
                                   (least & 0xffffu) >= kLow);
    if (__all_sync(kAll, plain)) {
#pragma unroll
      for (int i = 0; i < V; ++i) l[i] = active ? moe::to_f(raw.v[i]) : -INFINITY;
      if (!active) key[0] = 0;
      // (an inactive lane's further keys never come to the head)
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        l[i] = raw.at(i, E, lane);
        if (l[i] == -INFINITY) key[i] = 0;
      }
    }
    if (active) sort_keys<V>(key);
  } else {
    l[0] = raw.at(0, E, lane);
    uint32_t bits = *reinterpret_cast<const uint16_t*>(&raw.v[0]);
    if (bits == 0x8000u) bits = 0;
    key[0] = l[0] == -INFINITY ? 0u : (order16(bits) << 16) | last;
  }
  uint32_t mine = 0, first = 0;
  rounds(k, [&](int j, int live) {
    const uint32_t m = __reduce_max_sync(kAll, key[0]);
    if (j == 0) first = m;
    if (lane == j) mine = m;
    const bool win = key[0] == m;
    if constexpr (V == 1) key[0] = win ? 0u : key[0];
    else pop<V>(key, win, live);
  });
  auto value = [](uint32_t key) {
    const uint16_t bits = (uint16_t)unorder16(key >> 16);
    return key ? clean(moe::to_f(*reinterpret_cast<const T*>(&bits))) : -INFINITY;
  };
  return {mine ? 0xffff - (int)(mine & 0xffffu) : -1, value(mine), value(first)};
}

// 32-bit logits, lists of up to 8: the lists are of logits alone, and the
// slots' lanes look the experts up afterwards, among the V logits of the lane
// that won (which it leaves in `row`, shared memory of 32 V floats).
template <int V, bool VEC>
__device__ __forceinline__ Choice choose32(const Raw<float, V, VEC>& raw, int E, int k, int lane,
                                           float (&l)[V], float* row) {
  constexpr uint32_t kNone = 0x007fffffu;  // the order of -infinity
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    l[i] = raw.at(i, E, lane);
    const uint32_t bits = __float_as_uint(l[i] + 0.f);  // -0 made +0
    key[i] = bits ^ ((uint32_t)((int)bits >> 31) | 0x80000000u);
  }
  __syncwarp();  // the last token's look-up is over
  put<V>(row + lane * V, l);
  sort_keys<V>(key);
  uint32_t mine = kNone, first = kNone;
  int from = 0;
  rounds(k, [&](int j, int live) {
    const uint32_t m = __reduce_max_sync(kAll, key[0]);
    const int src = __ffs(__ballot_sync(kAll, key[0] == m)) - 1;  // lowest lane: lowest experts
    if (j == 0) first = m;
    if (lane == j) mine = m, from = src;
    if constexpr (V == 1) key[0] = lane == src ? 0u : key[0];
    else pop<V>(key, lane == src, live);
  });
  auto value = [&](uint32_t m) {
    return m > kNone ? __uint_as_float(m & 0x80000000u ? m ^ 0x80000000u : ~m) : -INFINITY;
  };
  Choice c{-1, value(mine), value(first)};
  __syncwarp();
  // the n-th among equals of one lane is the n-th of them there
  const uint32_t same = __match_any_sync(kAll, mine) & __match_any_sync(kAll, from);
  int skip = __popc(same & ((1u << lane) - 1));
  if (mine > kNone) {
    float v[V];
    get<V>(row + from * V, v);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (v[i] == c.logit && skip-- == 0) c.expert = from * V + i;
  }
  return c;
}

// More experts than the lists hold: the winner looks for its next one.
template <typename T, int V, bool VEC>
__device__ __forceinline__ Choice choose_wide(const Raw<T, V, VEC>& raw, int E, int k, int lane,
                                              float (&l)[V]) {
  uint32_t taken = 0;
  float head = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    l[i] = raw.at(i, E, lane);
    head = fmaxf(head, l[i]);
  }
  Choice c{-1, -INFINITY, -INFINITY};
  for (int j = 0; j < k; ++j) {
    const uint32_t bits = __float_as_uint(head + 0.f);
    const uint32_t key = bits ^ ((uint32_t)((int)bits >> 31) | 0x80000000u);
    const uint32_t m = __reduce_max_sync(kAll, key);
    const int src = __ffs(__ballot_sync(kAll, key == m)) - 1;
    int at = 0;
    const float value = head;
    if (lane == src) {
#pragma unroll
      for (int i = V - 1; i >= 0; --i)
        if (l[i] == value && !((taken >> i) & 1)) at = i;
      taken |= 1u << at;
      head = -INFINITY;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (!((taken >> i) & 1)) head = fmaxf(head, l[i]);
    }
    const float best = __shfl_sync(kAll, value, src);
    if (best == -INFINITY) break;
    const int e = __shfl_sync(kAll, lane * V + at, src);
    if (j == 0) c.top = best;
    if (lane == j) c.expert = e, c.logit = best;
  }
  return c;
}

// Losses and token count of one group from its sums.
__device__ __forceinline__ void finish_group(const RouteArgs& a, int g, float dot, float zsum,
                                             int n) {
  const float n1 = (float)(n > 0 ? n : 1);
  a.tokens[g] = n;
  a.loss[2 * g] = dot * ((float)a.E / (float)a.k) / n1 / n1;
  a.loss[2 * g + 1] = zsum / n1;
}

template <typename T, int V, bool VEC>
__global__ void __launch_bounds__(kThreads) route_kernel(const RouteArgs a) {
  extern __shared__ __align__(16) float smem[];  // P [warps][E], counts [E]
  int* sc = reinterpret_cast<int*>(smem + kWarps * a.E);
  // 32-bit logits: a token's, for the look-up of its choices
  constexpr bool kLook = std::is_same<T, float>::value && V <= 8;
  __shared__ __align__(16) float row_smem[kLook ? kWarps * 32 * V : 4];
  __shared__ float red[kWarps], sz[kWarps];
  __shared__ int sn[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = blockIdx.x / a.blocks, b = blockIdx.x % a.blocks;
  for (int e = threadIdx.x; e < a.E; e += kThreads) sc[e] = 0;
  moe::wait_for_earlier();
  moe::let_next_start();
  __syncthreads();
  float psum[V];
#pragma unroll
  for (int v = 0; v < V; ++v) psum[v] = 0.f;
  float zsum = 0.f;
  int n = 0;
  // unsigned: T < 2^31, but a step past it need not be
  const unsigned T_ = (unsigned)a.T, step = (unsigned)(a.blocks * kWarps);
  unsigned t = (unsigned)(b * kWarps + warp);
  size_t row = (size_t)g * a.T + t;
  const T* next = static_cast<const T*>(a.logits) + row * a.ld;
  const size_t next_step = (size_t)step * a.ld;
  Raw<T, V, VEC> raw;
  uint8_t mask = 1;
  if (t < T_) {
    raw.load(next, a.E, lane);
    if (a.mask) mask = a.mask[row];
  }
  for (; t < T_; t += step, row += step) {
    const Raw<T, V, VEC> now = raw;
    const uint8_t on = mask;
    next += next_step;
    if (t + step < T_) {  // the next token's, on their way
      raw.load(next, a.E, lane);
      if (a.mask) mask = a.mask[row + step];
    }
    Choice c{-1, -INFINITY, -INFINITY};
    float p[V];  // the logits, then their exponentials
    if (on) {
      if constexpr (V > 8) c = choose_wide(now, a.E, a.k, lane, p);
      else if constexpr (std::is_same<T, float>::value)
        c = choose32(now, a.E, a.k, lane, p, row_smem + warp * 32 * V);
      else c = choose16(now, a.E, a.k, lane, p);
    }
    const float m = c.top;
    if (m == -INFINITY) {  // padding, or nothing to choose from
      if (lane < a.k) {
        a.experts[row * a.k + lane] = -1;
        a.weights[row * a.k + lane] = 0.f;
      }
      if (lane < 2) a.stats[2 * row + lane] = 0.f;
      continue;
    }
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) s += p[v] = exp_of(p[v] - m);
    s = moe::warp_sum(s);
    const float inv = __fdividef(1.f, s);
#pragma unroll
    for (int v = 0; v < V; ++v) psum[v] = fmaf(p[v], inv, psum[v]);
    const float lse = m + __logf(s);
    zsum = fmaf(lse, lse, zsum);
    ++n;
    const float u = exp_of(c.logit - m);  // 0 where nothing was chosen
    const float total = a.renorm ? moe::warp_sum(u) : s;
    if (lane < a.k) {
      a.experts[row * a.k + lane] = c.expert;
      a.weights[row * a.k + lane] = a.scale * __fdividef(u, total);
      if (c.expert >= 0) atomicAdd(&sc[c.expert], 1);
    }
    if (lane < 2) a.stats[2 * row + lane] = lane ? s : m;
  }
  if (lane == 0) sz[warp] = zsum, sn[warp] = n;
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (lane * V + v < a.E) smem[warp * a.E + lane * V + v] = psum[v];
  __syncthreads();
  zsum = 0.f, n = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) zsum += sz[w], n += sn[w];
  float* part = a.part + (size_t)blockIdx.x * (2 * a.E + 2);
  float dot = 0.f;
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    float p = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) p += smem[w * a.E + e];  // warps in order
    if (a.blocks == 1) {
      a.counts[(size_t)g * a.E + e] = sc[e];
      dot = fmaf(p, (float)sc[e], dot);
    } else {
      part[e] = p;
      part[a.E + e] = __int_as_float(sc[e]);
    }
  }
  if (a.blocks == 1) {
    dot = moe::block_sum(dot, red);
    if (threadIdx.x == 0) finish_group(a, g, dot, zsum, n);
  } else if (threadIdx.x == 0) {
    part[2 * a.E] = zsum, part[2 * a.E + 1] = __int_as_float(n);
  }
}

// One CTA per group adds the CTAs' partial sums: several threads per expert,
// each a part of the CTAs in order, and those parts in order.  Started while
// route_kernel runs; waits for its end.
__global__ void __launch_bounds__(kJoinThreads) route_join_kernel(const RouteArgs a) {
  __shared__ float red[kJoinThreads / 32];
  __shared__ float sp[kJoinThreads];
  __shared__ int sc[kJoinThreads];
  __shared__ float sz[32];
  __shared__ int sn[32];
  const int g = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t step = 2 * a.E + 2;
  const float* part = a.part + (size_t)g * a.blocks * step;
  const int width = (a.E + 31) / 32 * 32, ways = kJoinThreads / width;  // E <= 1024
  const int e = threadIdx.x % width, way = threadIdx.x / width;
  moe::wait_for_earlier();
  float p = 0.f, z = 0.f;
  int c = 0, n = 0;
  if (way < ways && e < a.E) {
    const int b1 = a.blocks * (way + 1) / ways;
#pragma unroll 8
    for (int b = a.blocks * way / ways; b < b1; ++b) {
      p += __ldcg(part + b * step + e);
      c += __float_as_int(__ldcg(part + b * step + a.E + e));
    }
  }
  sp[threadIdx.x] = p, sc[threadIdx.x] = c;
  if (warp == 0) {  // lane b sums CTAs b, b + 32, ..
    for (int b = lane; b < a.blocks; b += 32) {
      z += __ldcg(part + b * step + 2 * a.E);
      n += __float_as_int(__ldcg(part + b * step + 2 * a.E + 1));
    }
    sz[lane] = z, sn[lane] = n;
  }
  __syncthreads();
  float dot = 0.f;
  if (way == 0 && e < a.E) {
    for (int w = 1; w < ways; ++w) p += sp[w * width + e], c += sc[w * width + e];
    a.counts[(size_t)g * a.E + e] = c;
    dot = p * (float)c;
  }
  dot = moe::block_sum(dot, red);
  if (threadIdx.x == 0) {
    z = 0.f, n = 0;
    for (int i = 0; i < 32; ++i) z += sz[i], n += sn[i];
    finish_group(a, g, dot, z, n);
  }
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
  int blocks;  // CTAs per group
};

// CTAs of a group's own, so that a E c / (k n^2) stays in registers.
template <typename T, int V, bool VEC>
__global__ void __launch_bounds__(kThreads) route_back_kernel(const RouteBackArgs a) {
  // [warps][32 V]: what a token's chosen experts get, 0 elsewhere
  extern __shared__ __align__(16) float back_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = blockIdx.x / a.blocks, b = blockIdx.x % a.blocks;
  float* add = back_smem + warp * 32 * V;
#pragma unroll
  for (int v = 0; v < V; ++v) add[lane + 32 * v] = 0.f;
  __syncwarp();
  moe::wait_for_earlier();
  const float n = (float)max(a.tokens[g], 1);
  const float cb = a.dloss ? a.dloss[2 * g] * ((float)a.E / (float)a.k) / n / n : 0.f;
  const float cz = a.dloss ? 2.f * a.dloss[2 * g + 1] / n : 0.f;
  float base[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = lane * V + v;
    base[v] = e < a.E && a.dloss ? cb * (float)a.counts[(size_t)g * a.E + e] : 0.f;
  }
  // unsigned: T < 2^31, but a step past it need not be
  const unsigned T_ = (unsigned)a.T, step = (unsigned)(a.blocks * kWarps);
  const size_t row0 = (size_t)g * a.T;
  const T* logits = static_cast<const T*>(a.logits) + row0 * a.ld;
  T* dlogits = static_cast<T*>(a.dlogits) + row0 * a.ldd;
  struct Next {
    Raw<T, V, VEC> raw;
    int at;
    float dw, m, s;
  } next;
  auto load = [&](unsigned t) {
    next.raw.load(logits + (size_t)t * a.ld, a.E, lane);
    next.at = -1, next.dw = 0.f;
    if (lane < a.k) {
      next.at = a.experts[(row0 + t) * a.k + lane];
      if (a.dweights) next.dw = a.dweights[(row0 + t) * a.k + lane];
    }
    next.m = a.stats[2 * (row0 + t)], next.s = a.stats[2 * (row0 + t) + 1];
  };
  unsigned t = (unsigned)(b * kWarps + warp);
  if (t < T_) load(t);
  for (; t < T_; t += step) {
    const Next now = next;
    if (t + step < T_) load(t + step);  // (in place, a row is written after it is read: below)
    T* dst = dlogits + (size_t)t * a.ldd;
    float d[V];
    if (__shfl_sync(kAll, now.at, 0) < 0) {  // an invalid token
#pragma unroll
      for (int v = 0; v < V; ++v) d[v] = 0.f;
      Raw<T, V, VEC>::store(dst, a.E, lane, d);
      continue;
    }
    const int at = now.at < a.E ? now.at : -1;
    const float dw = at >= 0 ? a.scale * now.dw : 0.f;
    const float m = now.m, inv = __fdividef(1.f, now.s);
    const float lse = m + __logf(now.s);
    float p[V];
    float dot = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      p[v] = exp_of(now.raw.at(v, a.E, lane) - m) * inv;
      dot = fmaf(p[v], base[v], dot);
    }
    if (a.dweights) {
      // A slot's lane has its expert's probability from the row itself (in L1);
      // what it adds goes to the lane that owns the expert by way of shared
      // memory: to a (before the softmax's Jacobian), or to dl if renormalised.
      const float u = at >= 0 ? exp_of(clean(moe::to_f(logits[(size_t)t * a.ld + at])) - m) * inv
                              : 0.f;
      float x = dw;
      if (a.renorm) {
        const float q = __fdividef(u, moe::warp_sum(u));
        x = q * (dw - moe::warp_sum(q * dw));
      } else {
        dot = fmaf(u, dw, dot);
      }
      if (at >= 0) add[at] = x;
      __syncwarp();
    }
    dot = moe::warp_sum(dot);
    get<V>(add + lane * V, d);
    __syncwarp();
    if (a.dweights && at >= 0) add[at] = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      d[v] = a.renorm ? fmaf(p[v], base[v] - dot, d[v]) : p[v] * (base[v] + d[v] - dot);
      // p first: lse may be the largest float, and p 0
      d[v] = fmaf(p[v] * cz, lse, d[v]);
    }
    Raw<T, V, VEC>::store(dst, a.E, lane, d);
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

// CTAs per group: two tokens per warp until the GPU is full, then more.  (One per
// warp doubles the partial sums to join: 9.6 against 8.6 us at 3 x 1531 x 60; eight: 10.7.)
int route_blocks(int G, int T) {
  const int sms = std::max(sm_count(), 1);
  const int64_t want = ((int64_t)T + 2 * kWarps - 1) / (2 * kWarps);
  const int most = std::max(1, 4 * sms / std::max(G, 1));
  return (int)std::max<int64_t>(1, std::min<int64_t>(want, most));
}

// Whether a lane's V logits are whole aligned vectors in every row.
bool vectors(const void* p, size_t ld, int E, int V, size_t es) {
  const size_t unit = std::min<size_t>(16, V * es);
  return E % V == 0 && ld * es % unit == 0 && moe::aligned(p, unit);
}
template <typename F>
void for_vec(bool vec, F&& f) {
  if (vec) f(std::true_type());
  else f(std::false_type());
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
        constexpr int V = decltype(v)::value;
        for_vec(vectors(logits, ld, E, V, sizeof(t)), [&](auto vec) {
          rc = moe::launch("moe_route: launch", route_kernel<decltype(t), V, decltype(vec)::value>,
                           (unsigned)(G * a.blocks), kThreads, (kWarps + 1) * (size_t)E * 4, s, a);
        });
      });
    });
    if (rc || a.blocks == 1) return rc;
    return moe::launch("moe_route: join", route_join_kernel, (unsigned)G, kJoinThreads, 0, s, a);
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
    const int64_t want = ((int64_t)T + kWarps - 1) / kWarps;
    const int most = std::max(sm_count(), 1) * 8 / std::min(G, 1 << 20);
    const int blocks = (int)std::max<int64_t>(1, std::min<int64_t>(want, most));
    RouteBackArgs a{logits, ld, G, T, E, k, renorm ? 1 : 0, scale, experts, counts, tokens, stats,
                    dweights, dloss, dlogits, ldd, blocks};
    cudaStream_t s = as_stream(stream);
    for_type(dtype, [&](auto t) {
      for_width(E, [&](auto v) {
        constexpr int V = decltype(v)::value;
        const bool vec = vectors(logits, ld, E, V, sizeof(t)) &&
                         vectors(dlogits, ldd, E, V, sizeof(t));
        for_vec(vec, [&](auto w) {
          rc = moe::launch("moe_route_backward: launch",
                           route_back_kernel<decltype(t), V, decltype(w)::value>,
                           (unsigned)G * (unsigned)blocks, kThreads, kWarps * 32 * V * 4, s, a);
        });
      });
    });
    return rc;
  });
}
