// moe_experts.cuh -- what the experts' products share: where each expert's rows
// lie, how they are cut into tiles, and how a tile's operands reach shared memory.
#pragma once

#include "moe_common.cuh"
#include "symm_device.cuh"
#include "symm_tcgen05.cuh"

namespace experts {

using symm::Control;

constexpr uint32_t kBM = 128;          // features of a tile: the M side
constexpr uint32_t kMaxWarps = 14;     // of a block
constexpr uint32_t kMaxExperts = SYMM_MOE_MAX_EXPERTS;
enum { kErrRange = -5 };

// Expert e's rows are off[e] .. off[e + 1] - 1, its blocks of rows are numbered
// blocks[e] .. blocks[e + 1] - 1 among all experts' (times the column blocks:
// its tiles).  A block has at most `cap` rows.
struct Table {
  uint32_t off[kMaxExperts + 1], blocks[kMaxExperts + 1];
  uint32_t warp_rows[kMaxWarps], warp_blocks[3][kMaxWarps], warp_most[kMaxWarps];
  uint32_t cap;
  uint32_t most;  // rows of the largest block, in whole steps
};
constexpr uint32_t kStep = 32;  // of a tile's rows: what a pair's MMAs take

__device__ __forceinline__ uint32_t in_steps(uint32_t rows) {
  return (rows + kStep - 1) / kStep * kStep;
}
__device__ __forceinline__ uint32_t blocks_of(uint32_t rows, uint32_t cap) {
  return (rows + cap - 1) / cap;
}
// Rows of each of an expert's blocks (the last one may have fewer, never none), as
// even as whole steps allow.
__device__ __forceinline__ uint32_t block_rows(uint32_t rows, uint32_t cap) {
  const uint32_t nb = blocks_of(rows, cap);
  return nb ? in_steps((rows + nb - 1) / nb) : 0;
}
// The caps to choose from.
__device__ __forceinline__ uint32_t cap_of(uint32_t i, uint32_t max_rows) {
  return i == 0 ? max_rows : i == 1 ? 128 : 64;
}

// Fills the table from the counts (NULL: one expert with all n rows), by all
// threads of the block; ncol column blocks and as many `pairs` at work decide on the
// cap.  False where a count is negative or they exceed n.
__device__ __forceinline__ bool lay_out(Table& t, const int32_t* counts, uint32_t E, uint32_t n,
                                        uint32_t max_rows, uint32_t extra, uint32_t ncol,
                                        uint32_t pairs) {
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t per = (E + blockDim.x - 1) / blockDim.x, first = threadIdx.x * per;
  uint64_t sum = 0;  // of at most 1024 counts of at most n <= 2^24 each
  uint32_t blocks[3] = {}, most = 0;
  bool bad = false;
  for (uint32_t e = first; e < min(E, first + per); ++e) {
    const int32_t c = counts ? counts[e] : (int32_t)n;
    if (c < 0 || (uint32_t)c > n) {
      bad = true;
      continue;
    }
    sum += (uint32_t)c;
#pragma unroll
    for (uint32_t i = 0; i < 3; ++i) blocks[i] += blocks_of((uint32_t)c, cap_of(i, max_rows));
    most = max(most, (uint32_t)c);
  }
  bad |= sum > n;
  uint32_t rows = (uint32_t)min(sum, (uint64_t)n + 1);  // the whole sum stays below 2^33
  const uint32_t own_rows = rows, own_blocks[3] = {blocks[0], blocks[1], blocks[2]};
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t r = __shfl_up_sync(0xffffffffu, rows, o);
    uint32_t b[3];
#pragma unroll
    for (uint32_t i = 0; i < 3; ++i) b[i] = __shfl_up_sync(0xffffffffu, blocks[i], o);
    if (lane >= (uint32_t)o) {
      rows = min(rows + r, n + 1);
#pragma unroll
      for (uint32_t i = 0; i < 3; ++i) blocks[i] += b[i];
    }
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 31) {
    t.warp_rows[warp] = rows, t.warp_most[warp] = most;
#pragma unroll
    for (uint32_t i = 0; i < 3; ++i) t.warp_blocks[i][warp] = blocks[i];
  }
  __syncthreads();
  uint32_t at = rows - own_rows, all = 0, all_blocks[3] = {}, before[3] = {}, largest = 0;
  for (uint32_t w = 0; w < blockDim.x / 32; ++w) {
    if (w < warp) at += t.warp_rows[w];
    all = min(all + t.warp_rows[w], n + 1);
    largest = max(largest, t.warp_most[w]);
#pragma unroll
    for (uint32_t i = 0; i < 3; ++i) {
      if (w < warp) before[i] += t.warp_blocks[i][w];
      all_blocks[i] += t.warp_blocks[i][w];
    }
  }
  bad |= all > n;
  if (__syncthreads_or(bad)) return false;
  // The cap with the least rounds of tiles, each as long as its rows and `extra` more
  // (the weights, that every block of rows reads again, and what a slice costs besides).
  uint32_t which = 0;
  uint64_t best = ~0ull;
#pragma unroll
  for (uint32_t i = 0; i < 3; ++i) {
    const uint32_t rounds = (all_blocks[i] * ncol + pairs - 1) / pairs;
    const uint64_t cost =
        (uint64_t)rounds * (min(cap_of(i, max_rows), in_steps(largest)) + extra);
    if (cost < best) best = cost, which = i;
  }
  const uint32_t cap = cap_of(which, max_rows);
  uint32_t bt = which == 0   ? before[0] + blocks[0] - own_blocks[0]
                : which == 1 ? before[1] + blocks[1] - own_blocks[1]
                             : before[2] + blocks[2] - own_blocks[2];
  for (uint32_t e = first; e < min(E, first + per); ++e) {
    t.off[e] = at, t.blocks[e] = bt;
    const uint32_t c = counts ? (uint32_t)counts[e] : n;
    at += c, bt += blocks_of(c, cap);
    if (e == E - 1) t.off[E] = at, t.blocks[E] = bt;
  }
  if (threadIdx.x == 0) t.cap = cap, t.most = min(cap, in_steps(largest));
  __syncthreads();
  return true;
}

// The expert whose blocks hold number b (below blocks[E]): the last one with
// blocks[e] <= b.
__device__ __forceinline__ uint32_t expert_of(const Table& t, uint32_t b, uint32_t E) {
  uint32_t lo = 0, hi = E;  // blocks[lo] <= b < blocks[hi]
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) / 2;
    if (t.blocks[mid] <= b) lo = mid;
    else hi = mid;
  }
  return lo;
}

struct Tile {
  uint32_t e, row, rows, bt, col;  // rows: that are there, of bt
};
// Tile i of ncol column blocks.  Up to eight blocks of rows share a column
// block's weights one after another, then the next column block shares theirs:
// what the SMs work on at a time is about as many rows as columns, which L2 holds.
__device__ __forceinline__ Tile tile_at(const Table& t, uint32_t i, uint32_t E, uint32_t ncol) {
  Tile o;
  o.e = expert_of(t, i / ncol, E);
  const uint32_t c = t.off[o.e + 1] - t.off[o.e], nb = blocks_of(c, t.cap);
  const uint32_t full = block_rows(c, t.cap);
  const uint32_t local = i - t.blocks[o.e] * ncol, group = local / (8 * ncol);
  const uint32_t in = min(8u, nb - 8 * group), r = local - 8 * group * ncol;
  const uint32_t b = 8 * group + r % in;
  o.col = r / in;
  o.row = t.off[o.e] + b * full;
  o.rows = min(full, c - b * full);
  o.bt = in_steps(o.rows);
  return o;
}

// `rows` rows (whole steps of 16) from `row` on, 128 bytes of each from x on, to lines
// of 128 bytes at `to`: boxes of 64 rows, then of 16.
__device__ __forceinline__ void load_lines(uint8_t* to, const CUtensorMap* map64,
                                           const CUtensorMap* map16, int x, uint32_t row,
                                           uint32_t rows, uint64_t* bar) {
  uint32_t r = 0;
  for (; r + 64 <= rows; r += 64) symm::tma_load_2d(to + r * 128, map64, x, (int)(row + r), bar);
  for (; r < rows; r += 16) symm::tma_load_2d(to + r * 128, map16, x, (int)(row + r), bar);
}

// The bounded wait of the experts' kernels: 16 tries at a time, so that a budget or
// another's give-up is noticed within a tile (256 tries outlast the longest one's 0.4 ms).
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, uint64_t budget_ns,
                                          const Control* ctl) {
  return symm::mbar_wait_warp<16>(bar, parity, budget_ns, ctl);
}
// How long a CTA that gives up waits for its own copies and MMAs, which nothing
// but the hardware holds up: a second, however short the heap's budget is.
__device__ __forceinline__ uint64_t drain_ns(uint64_t budget_ns) {
  return max(budget_ns, (uint64_t)1000000000);
}

// Whether p holds in any of a group's `threads` (barrier `id` of theirs; 1: the epilogue's).
__device__ __forceinline__ bool any_of(bool p, uint32_t threads, uint32_t id = 1) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %3, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)p), "r"(threads), "r"(id)
      : "memory");
  return r != 0;
}

// --------------------------------------------------------- the epilogue --
// A warp reads its 32 TMEM lanes (features) in fragments of 8 lanes x 8 columns, in
// which a thread has two neighbouring columns of lane T / 4.  stmatrix and ldmatrix
// move such fragments to and from shared memory, with .trans as rows of
// features: what global memory holds, 64 bytes of a row for a warp.  (A lane for
// a feature and 2-byte stores took 25 thousand cycles a 128 x 256 tile; the
// gradients' reads beside them 90 thousand.)
constexpr uint32_t kLine = 80;  // bytes of 32 staged 16-bit values: 8 lines meet all banks

// 16 TMEM lanes x 16 columns: v[4 t + 2 o + i] is lane 8 o + T / 4, column
// 8 t + 2 (T % 4) + i.
__device__ __forceinline__ void tmem_frag16(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7])
      : "r"(taddr)
      : "memory");
}
// Waits for them; names the registers, so that no use comes before.
__device__ __forceinline__ void tmem_wait(uint32_t (&a)[8], uint32_t (&b)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]),
                 "+r"(a[6]), "+r"(a[7]), "+r"(b[0]), "+r"(b[1]), "+r"(b[2]), "+r"(b[3]),
                 "+r"(b[4]), "+r"(b[5]), "+r"(b[6]), "+r"(b[7])
               :
               : "memory");
}
// The warp's 32 lanes x 16 columns: v[h] lanes 16 h ..
__device__ __forceinline__ void tmem_frags(uint32_t taddr, uint32_t (&v)[2][8]) {
  tmem_frag16(taddr, v[0]);
  tmem_frag16(taddr + (16u << 16), v[1]);
  tmem_wait(v[0], v[1]);
}
// Four 8 x 8 matrices: the lines of 16 bytes of matrix m at the addresses of lanes 8 m ..
__device__ __forceinline__ void stmatrix_t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                           uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void stmatrix(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                         uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_t(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c,
                                           uint32_t& d) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
               : "r"(addr)
               : "memory");
}
// Packed fragments p[t][o] (columns 8 t .., lanes 8 o ..) of 16 columns to 16 lines of
// `stage`, and back.
__device__ __forceinline__ void stage_rows(uint8_t* stage, const uint32_t (&p)[2][4]) {
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t at = symm::smem_addr(stage) + (lane & 7) * kLine + (lane >> 3) * 16;
#pragma unroll
  for (uint32_t t = 0; t < 2; ++t)
    stmatrix_t(at + 8 * t * kLine, p[t][0], p[t][1], p[t][2], p[t][3]);
}
__device__ __forceinline__ void unstage_rows(const uint8_t* stage, uint32_t (&p)[2][4]) {
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t at = symm::smem_addr(stage) + (lane & 7) * kLine + (lane >> 3) * 16;
#pragma unroll
  for (uint32_t t = 0; t < 2; ++t)
    ldmatrix_t(at + 8 * t * kLine, p[t][0], p[t][1], p[t][2], p[t][3]);
}
// 16 staged lines to the rows at y (first row, first feature), `valid` rows and
// `width` features of 32 there; 16 bytes at a time where `vec` (rows 16-byte aligned).
template <typename T>
__device__ __forceinline__ void store_rows(const uint8_t* stage, T* y, size_t ld, uint32_t valid,
                                           uint32_t width, bool vec) {
  const uint32_t lane = threadIdx.x & 31, f = 8 * (lane & 3);
#pragma unroll
  for (uint32_t i = 0; i < 2; ++i) {
    const uint32_t r = 8 * i + lane / 4;
    const uint4 v = *reinterpret_cast<const uint4*>(stage + r * kLine + (lane & 3) * 16);
    if (r >= valid || f >= width) continue;
    T* to = y + r * ld + f;
    if (vec && f + 8 <= width) {
      *reinterpret_cast<uint4*>(to) = v;
    } else {
      const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
      for (uint32_t j = 0; j < 8; ++j)
        if (f + j < width) to[j] = e[j];
    }
  }
}

// ------------------------------------------------------------- CTA pairs --
// A value that is the same in the whole warp, where the compiler sees that it is and
// keeps it in a uniform register.
__device__ __forceinline__ uint32_t uniform(uint32_t v) {
  return __shfl_sync(0xffffffffu, v, 0);
}
// Two CTAs of a cluster share a tile of twice 128 features (cta_group::2): each
// holds its own 128 features of the M side and half of the N side's rows in its
// shared memory, and its own features' accumulators in its TMEM; the first one
// issues the MMAs of both.  An SM then loads and reads half of the N side: alone,
// 96 bytes a cycle of operands and 94 of copies at N 256 exceed the 128 that its
// shared memory moves.
__device__ __forceinline__ uint32_t pair_rank() {
  uint32_t v;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(v));
  return v;
}
__device__ __forceinline__ void pair_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
}
// The same in two halves, for work between that needs neither.
__device__ __forceinline__ void pair_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A tensor map's own bytes on their way before its first copy.
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// One warp of each CTA of the pair calls these, with the same number of columns.
__device__ __forceinline__ void pair_tmem_alloc(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   symm::smem_addr(dst_smem)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}
// D (both CTAs' TMEM) (+)= A B^T, kind::f16, issued by one thread of the first CTA.
__device__ __forceinline__ void pair_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on `bar` of both CTAs once every MMA issued so far by this thread is done.
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(symm::smem_addr(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// The same on this CTA's alone.
__device__ __forceinline__ void pair_commit_own(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          symm::smem_addr(bar))
      : "memory");
}
// Arrives on `bar` of the pair's first CTA.  What it tells of are copies and
// tcgen05.ld that are complete and writes behind a proxy fence: no release of
// cluster scope, which waits for all of the SM's stores (2000 cycles a slice).
__device__ __forceinline__ void arrive_first(uint64_t* bar) {
  uint32_t remote;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(remote) : "r"(symm::smem_addr(bar)));
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(remote) : "memory");
}
// Before a CTA of a pair may leave: its copies have landed (`full`; whether or not
// anything used them), and what uses them has released them (`empty`: arrivals
// from the other CTA, which must find this one's shared memory).  Bounded: after a
// wait that gave up, a `full` of the first CTA may lack the second one's word for
// good, so all of them together have the time of one.
__device__ __forceinline__ void drain_ring(uint64_t* full, uint64_t* empty, uint32_t stages,
                                           uint32_t loads, bool ok, uint64_t budget_ns) {
  const uint32_t first = loads > stages ? loads - stages : 0;
  const uint64_t t0 = symm::globaltimer_ns(), most = drain_ns(budget_ns);
  for (uint32_t i = first; i < loads; ++i) {
    const uint64_t gone = symm::globaltimer_ns() - t0;
    symm::mbar_wait(&full[i % stages], (i / stages) & 1, gone < most ? most - gone : 0);
  }
  for (uint32_t i = first; ok && i < loads; ++i)
    ok = symm::mbar_wait(&empty[i % stages], (i / stages) & 1, drain_ns(budget_ns));
}
// The end of a kernel of CTA pairs, by all threads: all roles of this CTA are over, and
// the first CTA's issuer has ended with pair_commit(drain), an arrival on `drain` of both.
// Where a wait gave up, the other roles may have left with commits on their way to this
// CTA's barriers (`empty`, `tfull`), the second CTA's too; the last of them is `drain`'s,
// and the MMAs are over with it.  Only then may shared memory and TMEM go.  Bounded: a
// wait that gives up raises the heap's abort flag, which ends the issuer's own waits.
__device__ __forceinline__ void leave_pair(uint64_t* drain, uint32_t tmem, uint32_t ncols,
                                           uint64_t budget_ns) {
  const uint32_t warp = uniform(threadIdx.x >> 5);
  __syncwarp();
  symm::tc_fence_before();
  __syncthreads();
  if (warp == 1) symm::mbar_wait(drain, 0, drain_ns(budget_ns));
  __syncwarp();
  pair_sync();  // the other CTA's MMAs, arrivals and reads of TMEM are over too
  if (warp == 1) {
    symm::tc_fence_after();
    pair_tmem_dealloc(tmem, ncols);
  }
}
// Launches clusters of two CTAs, as moe::launch.
template <typename... P, typename... A>
int launch_pairs(const char* what, void (*kernel)(P...), unsigned pairs, unsigned block,
                 size_t smem, cudaStream_t s, A... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return symm_host::cuda_check(cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...), what);
}
// Pairs of such CTAs that are resident at once (a kernel needs its shared memory allowed
// before); SMs / 2 where the driver does not say.
inline unsigned resident_pairs(const void* kernel, unsigned block, size_t smem) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    n = symm_host::sm_count() / 2;
  }
  return (unsigned)(n < 1 ? 1 : n);
}

// act(g) and its derivative: g sigma(g), or g Phi(g) with the normal
// distribution's Phi.  The exponential and the quotient are the approximate
// instructions, before a rounding to 16 bits or fewer: exp(x) errs by up to 2 + 1.2 |x|
// ulp of 24 bits, the quotient by 2, so that sigma is within some 2^-17 of itself at
// g = -50; where 1 + exp(-g) exceeds 2^126 (g below -87.3) the quotient is 0.
__device__ __forceinline__ float activate(int act, float g) {
  if (act == SYMM_ACT_SILU) return __fdividef(g, 1.f + __expf(-g));
  return g * normcdff(g);
}
__device__ __forceinline__ void activate_both(int act, float g, float& a, float& da) {
  if (act == SYMM_ACT_SILU) {
    const float p = __fdividef(1.f, 1.f + __expf(-g));
    a = g * p;
    da = p * (1.f + g * (1.f - p));
  } else {
    const float p = normcdff(g);
    a = g * p;
    da = p + g * 0.3989422804014327f * __expf(-0.5f * g * g);
  }
}

}  // namespace experts
