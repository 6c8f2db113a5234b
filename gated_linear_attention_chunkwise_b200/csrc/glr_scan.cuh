// glr_scan.cuh -- the walk that glr_fwd and glr_bwd share (glr_fwd.cu, glr_bwd.cu).
//
// Mathematics.  Both passes are first-order recurrences per channel: forwards
// h_p = alpha_p h_{p-1} + u_p, backwards r_p = alpha_p (d_p + r_{p+1}).  A span of tokens
// maps the value that enters it to A * in + h, and two spans compose to (A2 A1, A2 h1 + h2),
// so a long sequence is cut into spans that are folded separately and then joined.
//
// Split.  A cluster of up to 16 blocks owns a slab of channels of one sequence (or of the
// row of packed sequences) and walks it in rounds.  In a round every thread folds kRun
// consecutive tokens of four channels in registers; warps join their threads' spans by
// shuffles, the block its warps' in shared memory, the cluster its blocks' by asynchronous
// stores into one another's shared memory; then each thread applies the value that enters
// its span to its tokens.  Every input is read once, every output written once, nothing
// passes between blocks through global memory, there is no workspace, and the order of
// every sum is fixed.  A thread's tokens of the next round are copied (cp.async) into
// slots of shared memory that only it reads while the current round is joined and written.
//
// Packed sequences are one long row of tokens; a span that begins a sequence forgets
// what enters it.  It has A = 0, which is all that finite values need, and is marked by the
// sign bit of A (gates are never negative): where a value is not finite the fold selects
// instead of multiplying by zero, so a NaN ends with its sequence.
//
// What bounds it.  With log_alpha large calls reach 64-81 % of the copy bandwidth (64
// sequences of 1024 x 2048 bf16: 218 us for 1.07 GB); with logits and the complement form the
// gates take 17 of 42 instructions an element and it is 35-45 %, half of that issue and half
// the latency of a round's exchange.  Eight tokens a thread: with 4 the fixed work of a round
// (330 instructions a thread) doubles an element (one 16384 x 2048 call 70 -> 87 us), with 16
// the registers leave too few warps (packed, logits: 347 -> 376 us).  128 threads a block, with
// as many warps an SM: 64 take 396 us there, 96 take 358, 256 take 409.
#pragma once

#include <algorithm>
#include <atomic>

#include "glr.cuh"

namespace dig {
namespace glr {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;  // above 8 a kernel has to be allowed to

// ---- spans of four channels ---------------------------------------------------------------
struct Span {
  F4 A, h;
};
__device__ __forceinline__ Span nothing() { return Span{all4(1.f), all4(0.f)}; }

// A span that begins a sequence forgets what enters it: the sign bit of its first A (gates
// are never negative).
constexpr uint32_t kForget = 0x80000000u;
__device__ __forceinline__ bool forgets(const Span& s) { return (int)__float_as_uint(s.A.a.x) < 0; }

__device__ __forceinline__ F4 enter(const Span& s, F4 in) { return fma4(s.A, in, s.h); }
__device__ __forceinline__ F4 enter_marked(const Span& s, F4 in) { return forgets(s) ? s.h : enter(s, in); }
// The mark of two spans: that of either.
__device__ __forceinline__ float marked(float A, const Span& first, const Span& then) {
  return __uint_as_float((__float_as_uint(A) & ~kForget) |
                         ((__float_as_uint(first.A.a.x) | __float_as_uint(then.A.a.x)) & kForget));
}
// Two spans as one.  A marked span has A = 0 as well, so this is right for finite values.
__device__ __forceinline__ Span join(const Span& first, const Span& then) {
  Span r{mul4(first.A, then.A), enter(then, first.h)};
  r.A.a.x = marked(r.A.a.x, first, then);
  return r;
}

__device__ __forceinline__ bool any_over(F4 v, float most) {  // (a NaN compares false)
  return v.a.x > most || v.a.y > most || v.b.x > most || v.b.y > most;
}
__device__ __forceinline__ bool all_within(F4 v, float most) {  // (a NaN compares false)
  return v.a.x <= most && v.a.y <= most && v.b.x <= most && v.b.y <= most;
}
// Values whose sums over a block's spans stay finite (a NaN compares false).
__device__ __forceinline__ bool modest(F4 v) {
  return fabsf(v.a.x) <= 1e30f && fabsf(v.a.y) <= 1e30f && fabsf(v.b.x) <= 1e30f && fabsf(v.b.y) <= 1e30f;
}
// Growth is held at the largest fp32 number (and reported), so that a zero that enters
// later gives zero instead of NaN.
__device__ __forceinline__ F4 capped(F4 v, bool& grown) {
  grown |= any_over(v, FLT_MAX);
  auto c = [](float x) { return x > FLT_MAX ? FLT_MAX : x; };
  return F4{make_float2(c(v.a.x), c(v.a.y)), make_float2(c(v.b.x), c(v.b.y))};
}
// join() where a value may not be finite (it ends at a mark) or a span may grow.
__device__ __forceinline__ Span join_marked(const Span& first, const Span& then, bool& grown) {
  Span r{capped(mul4(first.A, then.A), grown), enter_marked(then, first.h)};
  r.A.a.x = marked(r.A.a.x, first, then);
  return r;
}

// ---- the exchange ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_to(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
// 16 bytes into another block's shared memory; its barrier counts them.
__device__ __forceinline__ void store_async(uint32_t addr, uint32_t bar, F4 v) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
               "f"(v.a.x), "f"(v.a.y), "f"(v.b.x), "f"(v.b.y), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void expect_bytes(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

template <int kLanes>
struct Shared {
  Span warp[2][kWarps][kLanes];        // spans of this block's warps, by parity of the round
  Span total[2][kMaxCluster][kLanes];  // spans of the cluster's blocks
  F4 entry[kLanes];                    // what enters this block
  uint64_t bar[2];                     // total[i] has arrived
};

// One block's place and the value that runs along its slab.
template <int kLanes>
struct Walk {
  Shared<kLanes>& sm;
  uint32_t rank, size;
  int lane, warp, seg;  // channel group in the slab; warp; the thread's span within the warp
  F4 carry;             // the value at the start of the round (kept by the first warp)

  __device__ __forceinline__ Walk(Shared<kLanes>& s, const F4& start) : sm(s), carry(start) {
    rank = cluster_rank();
    size = cluster_size();
    lane = threadIdx.x % kLanes;
    warp = threadIdx.x >> 5;
    seg = (threadIdx.x & 31) / kLanes;
    if (threadIdx.x == 0) {
      mbar_init(smem_u32(&sm.bar[0]), 1);
      mbar_init(smem_u32(&sm.bar[1]), 1);
      fence_mbar_init();
    }
    cluster_arrive();  // every block runs, with its barriers set up, before one writes to another
  }

  // The value that enters this thread's span s.  Returns false, in all threads of the block
  // alike, when the wait for the other blocks ran out.  odd: s is not modest or its A may
  // exceed 1 (otherwise no join of spans overflows, and A = 0 forgets).  marks: spans of
  // the slab may be marked.  meanwhile() runs while the totals travel: the next round's copies
  // and searches.
  //
  // Reuse of the buffers: a block sends its total of round k + 2 only after it has received
  // all totals of round k + 1, and a block sends that only after all its threads have passed
  // the barrier of round k + 1, behind their reads of round k.
  template <typename F>
  __device__ __forceinline__ bool exchange(const Span& s, bool odd, bool marks, int round, F4& in, bool& grown,
                                           F meanwhile) {
    const int par = round & 1;
    const int lane32 = threadIdx.x & 31;
    Span inc = s;  // inclusive scan over the warp's spans
    if (__any_sync(0xffffffffu, odd)) {
#pragma unroll 1
      for (int off = kLanes; off < 32; off *= 2) {
        const Span o = shift(inc, off);
        if (lane32 >= off) inc = join_marked(o, inc, grown);
      }
    } else {
#pragma unroll
      for (int off = kLanes; off < 32; off *= 2) {
        const Span o = shift(inc, off);
        if (lane32 >= off) inc = join(o, inc);
      }
    }
    Span pre = shift(inc, kLanes);
    if (seg == 0) pre = nothing();
    if (seg == 32 / kLanes - 1) sm.warp[par][warp][lane] = inc;
    if (threadIdx.x == 0) expect_bytes(smem_u32(&sm.bar[par]), size * kLanes * (uint32_t)sizeof(Span));
    const bool special = __syncthreads_or(odd);
    Span before = nothing();  // the warps before this one
    Span all;                 // the block
    if (special) {
#pragma unroll 1
      for (int i = 0; i < warp; ++i) before = join_marked(before, sm.warp[par][i][lane], grown);
      pre = join_marked(before, pre, grown);
      if (warp == kWarps - 1) all = join_marked(before, sm.warp[par][warp][lane], grown);
    } else {
      for (int i = 0; i < warp; ++i) before = join(before, sm.warp[par][i][lane]);
      pre = join(before, pre);
      if (warp == kWarps - 1) all = join(before, sm.warp[par][warp][lane]);
    }
    if (warp == kWarps - 1) {
      const uint32_t to = smem_u32(&sm.total[par][rank][lane]), bar = smem_u32(&sm.bar[par]);
      for (uint32_t r = seg; r < size; r += 32 / kLanes) {
        const uint32_t addr = map_to(to, r), at = map_to(bar, r);
        store_async(addr, at, all.A);
        store_async(addr + 16u, at, all.h);
      }
    }
    meanwhile();
    bool late = false;
    if (warp == 0) {
      if (!mbar_wait(smem_u32(&sm.bar[par]), (round >> 1) & 1)) {
        report_status(GLA_ERR_TIMEOUT);
        late = true;
      }
      F4 v = carry, mine = carry;
      if (marks) {
        for (uint32_t r = 0; r < size; ++r) {
          v = enter_marked(sm.total[par][r][lane], v);
          if (r + 1 == rank) mine = v;
        }
      } else {
        for (uint32_t r = 0; r < size; ++r) {
          v = enter(sm.total[par][r][lane], v);
          if (r + 1 == rank) mine = v;
        }
      }
      carry = v;
      if (seg == 0) sm.entry[lane] = mine;
    }
    if (__syncthreads_or(late)) return false;
    in = marks ? enter_marked(pre, sm.entry[lane]) : enter(pre, sm.entry[lane]);
    return true;
  }

  // No block leaves while another may still write to it.
  __device__ __forceinline__ void leave() {
    cluster_arrive();
    cluster_wait();
  }

 private:
  static __device__ __forceinline__ Span shift(const Span& s, int by) {
    auto f = [by](float v) { return __shfl_up_sync(0xffffffffu, v, by); };
    return Span{F4{make_float2(f(s.A.a.x), f(s.A.a.y)), make_float2(f(s.A.b.x), f(s.A.b.y))},
                F4{make_float2(f(s.h.a.x), f(s.h.a.y)), make_float2(f(s.h.b.x), f(s.h.b.y))}};
  }
};

// ---- tokens -----------------------------------------------------------------------------------

// Rows of scan positions p, p + step, ... (step +-1), and whether the first `count` of
// them are evenly spaced in memory (`apart` rows).
struct Rows {
  int f, df, x, y, p, step;

  __device__ __forceinline__ Rows(const ScanGeom& g, int first, int by) : p(first), step(by) {
    f = g.reverse ? g.T - 1 - p : p;  // position in the base order
    df = g.reverse ? -step : step;
    x = y = 0;
    if (g.column_base) {
      x = f / g.Hg;  // (a position before the first token is never used)
      y = f - x * g.Hg;
    }
  }
  __device__ __forceinline__ bool even(const ScanGeom& g, int count, int& apart) const {
    apart = g.column_base ? df * g.Wg : df;
    if (g.zigzag) return false;
    const int last = y + df * (count - 1);
    return !g.column_base || (last >= 0 && last < g.Hg);
  }
  __device__ __forceinline__ int next(const ScanGeom& g) {
    int row = f;
    if (g.zigzag) {
      row = zigzag_token(g, p);
    } else if (g.column_base) {
      row = y * g.Wg + x;
      y += df;
      if (y == g.Hg) {
        y = 0;
        ++x;
      } else if (y < 0) {
        y = g.Hg - 1;
        --x;
      }
    }
    f += df;
    p += step;
    return row;
  }
};

// Four channels of a token into this thread's slot; zeros where there is no token.
template <typename T>
__device__ __forceinline__ void fetch(uint32_t slot, const T* p, bool there) {
  if constexpr (sizeof(T) == 2) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(slot), "l"(p), "r"(there ? 8u : 0u) : "memory");
  } else {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(slot), "l"(p), "r"(there ? 16u : 0u) : "memory");
  }
}

// ---- packed sequences ---------------------------------------------------------------------------

// Sequence of packed token t: the last n in [0, nseq) with cu[n] <= t, or -1 before all.
// near: a sequence that a token near t lay in; the search widens from there.
__device__ __forceinline__ int find_sequence(const int* cu, int nseq, int t, int near) {
  int lo = min(max(near, 0), nseq - 1), hi, step = 1;  // then cu[lo - 1] <= t < cu[hi] where they exist
  if (cu[lo] <= t) {
    hi = ++lo;
    while (hi < nseq && cu[hi] <= t) {
      lo = hi + 1;
      hi = min(hi + step, nseq);
      step *= 2;
    }
    lo = min(lo, hi);
  } else {
    hi = lo;
    while (lo > 0 && cu[lo - 1] > t) {
      hi = lo - 1;
      lo = max(lo - step, 0);
      step *= 2;
    }
  }
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo - 1;
}

// Of a thread's tokens (bit i: the i-th it walks): which lie in a sequence, begin one, end
// one (first and last in scan order).
struct Marks {
  uint32_t inside = 0u, first = 0u, last = 0u;
  int first_seq = 0, last_seq = 0;  // the sequences of the lowest such bits
};
// The sequence a thread was last amid: tokens strictly between its ends need no search.
struct Amid {
  int begin = 0, end = 0, n = 0;
};
// The tokens are lo .. lo + n - 1; turned: walked from the highest to the lowest.
__device__ __forceinline__ Marks mark(const GlrArgs& a, int lo, int n, bool turned, Amid& at) {
  Marks m;
  m.inside = (1u << n) - 1u;
  if (n <= 0 || (lo > at.begin && lo + n < at.end)) return m;
  int q = find_sequence(a.cu, a.nseq, lo, at.n);
  const int end = lo + n;
  m.inside = 0u;
  int s = q < 0 ? 0 : a.cu[q], e = q < 0 ? a.cu[0] : a.cu[q + 1];
  at = q < 0 ? Amid{} : Amid{s, e, q};  // the rows before all sequences lie in none
  while (true) {  // one sequence after another
    const int from = max(s, lo), to = min(e, end);
    if (q >= 0 && from < to) {
      uint32_t bits = ((1u << (to - from)) - 1u) << (from - lo), low = s >= lo ? 1u << (s - lo) : 0u,
               high = e <= end ? 1u << (e - 1 - lo) : 0u;
      if (turned) {
        bits = __brev(bits) >> (32 - n);
        low = __brev(low) >> (32 - n);
        high = __brev(high) >> (32 - n);
      }
      const uint32_t first = a.dir ? high : low, last = a.dir ? low : high;
      m.inside |= bits;
      if (first && (m.first == 0u || first < (m.first & (0u - m.first)))) m.first_seq = q;
      if (last && (m.last == 0u || last < (m.last & (0u - m.last)))) m.last_seq = q;
      m.first |= first;
      m.last |= last;
    }
    if (e >= end || ++q >= a.nseq) break;
    s = e;
    e = a.cu[q + 1];
  }
  return m;
}
// The row in the states of the sequence that token t begins or ends, marked as bit i of
// `marks` whose lowest bit is in sequence `known` (in range whatever the lengths hold).
__device__ __forceinline__ int64_t state_row(const GlrArgs& a, uint32_t marks, int i, int known, int t) {
  const int n = marks & ((1u << i) - 1u) ? max(find_sequence(a.cu, a.nseq, t, known), 0) : known;
  return (int64_t)n * a.C;
}

// States of sequences of no token, which no thread reaches through its tokens, and the check
// of the lengths (no address of a token depends on them).
__device__ __forceinline__ void empty_sequences(const GlrArgs& a, int T, int c0, int width, const float* from, float* to,
                                                bool checks) {
  for (int n = threadIdx.x; n < a.nseq; n += kThreads) {
    const int s = a.cu[n], e = a.cu[n + 1];
    if (checks && (s < 0 || e > T || s > e)) report_status(GLA_ERR_INVALID_ARG);
    if (s == e && to)
      for (int c = c0; c < min(c0 + width, a.C); ++c) to[(int64_t)n * a.C + c] = from ? from[(int64_t)n * a.C + c] : 0.f;
  }
}

// ---- launch -------------------------------------------------------------------------------------
using Kernel = void (*)(GlrArgs, ScanGeom, int, int);

// How many clusters of `size` blocks run at once on the current device.
inline int resident_clusters(Kernel k, int size, size_t smem, std::atomic<int>* known) {
  int n = known[size].load(std::memory_order_relaxed);
  if (n > 0) return n;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = size;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3(size);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    return size == 1 ? 1 : 0;  // a size that this device does not run
  }
  known[size].store(n, std::memory_order_relaxed);
  return n;
}

// `known`: a table of the kernel's own, [device][cluster size], for the figures above; [device][0]:
// the setup that its attributes were made in.
using Known = std::atomic<int>[64][kMaxCluster + 1];

// How to launch one kernel: clusters of `cluster` blocks over slabs of 4 * lanes channels.
struct Plan {
  Kernel kernel;
  int lanes, slabs, cluster, rounds;
  float cost;
};

// The cluster size that ends first.  Waves of clusters that run at once take as many rounds
// each (and two more to start and end); a round takes the longer the more blocks share an SM.
// A round of the forward with log_alpha was measured at 2.2 + 0.45 us for each block an SM with
// 32-channel slabs and 2.3 + 0.55 us with 16-channel slabs: narrow slabs have twice the
// clusters and half the rounds, and win until the SMs are full (one sequence of 65536 tokens,
// us wide / narrow with clusters of 8: 64 channels 146 / 75, 1024 channels 178 / 142, 2048
// channels 242 / 257).  Each block above 8 adds 0.12 us to a round, so wider clusters pay
// while SMs are idle (64 channels 75 -> 45, 256 channels 94 -> 68).  Other gates and the
// backward have other rounds (predicted times are 0.9 to 1.7 times the measured ones), but the
// order of the choices hardly changes: for ten shapes from 3 x 777 x 136 to one sequence of
// 65536 x 2048 and 64 of 1024 x 2048, each forwards and backwards with log_alpha and with logits
// and complement, all slabs and cluster sizes were timed.  In 39 of the 40 the choice was
// within 2 % of the fastest, in one (1 us of 9) within 13 %.
inline cudaError_t plan(Kernel k, Known& known, const GlrArgs& a, const ScanGeom& g, int lanes, int run, size_t smem,
                        Plan* best) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int setup = setup_generation();
  if (known[dev & 63][0].load(std::memory_order_relaxed) != setup) {
    if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess)
      return e;
    known[dev & 63][0].store(setup, std::memory_order_relaxed);
  }
  const int slabs = (a.C + 4 * lanes - 1) / (4 * lanes);
  const int64_t total = (int64_t)a.B * slabs, per_block = kThreads / lanes * run;
  for (int size = 1; size <= kMaxCluster && (size == 1 || (size - 1) * per_block < g.T); ++size) {
    const int64_t at_once = resident_clusters(k, size, smem, known[dev & 63]);
    if (at_once == 0) continue;
    const int64_t waves = (total + at_once - 1) / at_once, rounds = (g.T + size * per_block - 1) / (size * per_block);
    const float sharing = (float)(std::min(total, at_once) * size) / 148.f;
    const float round = (lanes == 8 ? 2.2f + 0.45f * sharing : 2.3f + 0.55f * sharing) + 0.12f * std::max(0, size - 8);
    const float cost = (float)waves * (float)(rounds + 2) * round;
    if (cost < best->cost) *best = Plan{k, lanes, slabs, size, (int)rounds, cost};
  }
  return cudaSuccess;
}

// The cheaper of the kernels with 32- and with 16-channel slabs.  Beyond 2^20 channels of
// sequences clusters of one block fill the SMs many times over and wide slabs win: 30000 x 64
// tokens of 40 channels 705 us wide, 1061 narrow; of 16 channels, half a slab, 827 and 788.
inline cudaError_t enqueue(Kernel wide, Known& known_wide, Kernel narrow, Known& known_narrow, const GlrArgs& a, int run,
                           size_t smem, cudaStream_t st) {
  const ScanGeom g = make_geom(a.Hg, a.Wg, a.dir);
  Plan p{};
  p.cost = FLT_MAX;
  cudaError_t e = plan(wide, known_wide, a, g, 8, run, smem, &p);
  if (e == cudaSuccess && (int64_t)a.B * a.C <= 1 << 20) e = plan(narrow, known_narrow, a, g, 4, run, smem, &p);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = p.cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)((int64_t)a.B * p.slabs * p.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, p.kernel, a, g, p.slabs, p.rounds);
}

// Calls f<T, kind, complement>() for the call's types.
template <template <typename, int, bool> class F, typename... Args>
cudaError_t by_types(const GlrArgs& a, Args... args) {
  const int kind = gate_kind(a.gate_norm);
#define DIG_GLR(T, K, C) F<T, K, C>::run(a, args...)
#define DIG_GLR_FORM(T, K) (a.complement ? DIG_GLR(T, K, true) : DIG_GLR(T, K, false))
#define DIG_GLR_KIND(T)                            \
  (kind == kGateLog ? DIG_GLR_FORM(T, kGateLog)    \
                    : kind == kGateSigmoid ? DIG_GLR_FORM(T, kGateSigmoid) : DIG_GLR_FORM(T, kGateLogit))
  return a.bf16 ? DIG_GLR_KIND(__nv_bfloat16) : DIG_GLR_KIND(float);
#undef DIG_GLR_KIND
#undef DIG_GLR_FORM
#undef DIG_GLR
}

}  // namespace glr
}  // namespace dig
