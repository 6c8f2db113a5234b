// glr.cu -- the gated linear recurrence over a token grid in scan order or over packed
// sequences, and its backward pass (include/dig_gla.h, glr_fwd and glr_bwd).
//
// Mathematics.  Both passes are first-order recurrences per channel: forwards
// h_p = alpha_p h_{p-1} + u_p, backwards r_p = alpha_p (d_p + r_{p+1}).  A span of tokens
// maps the value that enters it to A * in + h, and two spans compose to (A2 A1, A2 h1 + h2),
// so a long sequence is cut into spans that are folded separately and then joined.
//
// Split.  A cluster of up to 8 thread blocks owns a slab of channels of one sequence (of
// one row of packed sequences) and walks it in rounds.  In a round every thread holds
// kRun consecutive tokens of two channels in registers, folds them, the block joins its
// threads' spans in shared memory, the cluster joins its blocks' through distributed
// shared memory with one cluster barrier, and each thread applies the value that enters
// its span to its tokens.  So every input is read once and every output written once,
// nothing passes through memory between blocks, no block waits on a flag, there is no
// workspace, and the order of every sum is fixed.  The next round's inputs are loaded
// into registers before the current round is joined.
//
// Packed sequences are one long row of tokens; a span that begins a sequence forgets
// what enters it.  That is marked by the sign bit of A (gates are never negative): the
// fold then selects instead of multiplying by zero, so a NaN ends with its sequence.
#include <float.h>

#include "glr.cuh"

namespace dig {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxCluster = 8;

// Two channels of a row as they lie in memory, and as fp32.
template <typename T>
struct Two;
template <>
struct Two<__nv_bfloat16> {
  using Raw = uint32_t;
  static __device__ __forceinline__ float2 get(Raw r) { return unpack_bf16x2(r); }
  static __device__ __forceinline__ Raw put(float2 f) { return pack_bf16x2(f.x, f.y); }
  static __device__ __forceinline__ Raw zero() { return 0u; }
};
template <>
struct Two<float> {
  using Raw = float2;
  static __device__ __forceinline__ float2 get(Raw r) { return r; }
  static __device__ __forceinline__ Raw put(float2 f) { return f; }
  static __device__ __forceinline__ Raw zero() { return make_float2(0.f, 0.f); }
};
template <typename T>
__device__ __forceinline__ typename Two<T>::Raw load2(const T* p) {
  return __ldcs(reinterpret_cast<const typename Two<T>::Raw*>(p));  // read once
}
template <typename T>
__device__ __forceinline__ void store2(T* p, float2 f) {
  *reinterpret_cast<typename Two<T>::Raw*>(p) = Two<T>::put(f);
}

// ---- spans --------------------------------------------------------------------------
constexpr uint32_t kForget = 0x80000000u;  // sign bit of A: nothing that enters matters

struct Span {
  float A, h;
};
__device__ __forceinline__ bool forgets(float A) { return (int)__float_as_uint(A) < 0; }
__device__ __forceinline__ float apply(Span s, float in) { return forgets(s.A) ? s.h : fmaf(s.A, in, s.h); }
// A product of gates; a mark in either factor stays.  Growth is held at the largest fp32
// number (and reported), so that a zero that enters later gives zero instead of NaN.
__device__ __forceinline__ float join(float a, float b, bool& grown) {
  float r = a * b;
  if (r > FLT_MAX) {
    r = FLT_MAX;
    grown = true;
  }
  return __uint_as_float(__float_as_uint(r) | ((__float_as_uint(a) | __float_as_uint(b)) & kForget));
}

// ---- the exchange between threads and blocks ------------------------------------------
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
__device__ __forceinline__ void store_remote(uint32_t saddr, uint32_t rank, float4 v) {
  asm volatile(
      "{\n\t.reg .u32 a;\n\t"
      "mapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.v4.f32 [a], {%2, %3, %4, %5};\n\t}" ::"r"(saddr),
      "r"(rank), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
      : "memory");
}

template <int kLanes>
struct Shared {
  static constexpr int kSubs = kThreads / kLanes;
  float4 agg[kSubs][kLanes];              // spans of this block's threads
  float4 total[2][kMaxCluster][kLanes];   // spans of the cluster's blocks, by parity of the round
};

// The value that enters this thread's span, for its two channels; moves carry[] from the
// start of the round to its end.
template <int kLanes>
__device__ __forceinline__ void exchange(Shared<kLanes>& sm, const Span (&s)[2], float (&carry)[2], float (&in)[2],
                                         int round, uint32_t rank, uint32_t size, bool& grown) {
  constexpr int kSubs = Shared<kLanes>::kSubs;
  const int lane = threadIdx.x % kLanes, sub = threadIdx.x / kLanes;
  sm.agg[sub][lane] = make_float4(s[0].A, s[0].h, s[1].A, s[1].h);
  __syncthreads();
  Span pre[2] = {{1.f, 0.f}, {1.f, 0.f}};
  for (int i = 0; i < sub; ++i) {
    const float4 v = sm.agg[i][lane];
    pre[0].h = apply(Span{v.x, v.y}, pre[0].h);
    pre[1].h = apply(Span{v.z, v.w}, pre[1].h);
    pre[0].A = join(pre[0].A, v.x, grown);
    pre[1].A = join(pre[1].A, v.z, grown);
  }
  float4(&total)[kMaxCluster][kLanes] = sm.total[round & 1];
  if (sub == kSubs - 1) {
    const float4 t = make_float4(join(pre[0].A, s[0].A, grown), apply(s[0], pre[0].h), join(pre[1].A, s[1].A, grown),
                                 apply(s[1], pre[1].h));
    for (uint32_t r = 0; r < size; ++r) store_remote(smem_u32(&total[rank][lane]), r, t);
  }
  cluster_arrive();
  cluster_wait();
  float at0 = carry[0], at1 = carry[1];
  for (uint32_t r = 0; r < size; ++r) {
    if (r == rank) {
      in[0] = apply(pre[0], at0);
      in[1] = apply(pre[1], at1);
    }
    const float4 v = total[r][lane];
    at0 = apply(Span{v.x, v.y}, at0);
    at1 = apply(Span{v.z, v.w}, at1);
  }
  carry[0] = at0;
  carry[1] = at1;
}

// ---- tokens and sequences ---------------------------------------------------------------

// Sequence of packed token t: the last n in [0, nseq) with cu[n] <= t, or -1 before all.
__device__ __forceinline__ int find_sequence(const int* cu, int nseq, int t) {
  int lo = 0, hi = nseq;  // cu[lo - 1] <= t < cu[hi] where both exist
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo - 1;
}

// The sequence of a token that mark() found to begin or end one (an index in range whatever
// the lengths hold).
__device__ __forceinline__ int64_t state_row(const GlrArgs& a, int t) {
  return (int64_t)max(find_sequence(a.cu, a.nseq, t), 0) * a.C;
}

// What a thread knows about the packed sequences its kRun tokens lie in.
struct Marks {
  uint32_t inside, first, last;  // a bit for each token (first and last in scan order)
  int n0;                        // sequence of the lowest token
};
// lo: the lowest of the tokens; step: +1 when bit i is token lo + i, -1 when it is lo + n - 1 - i.
template <int kRun>
__device__ __forceinline__ Marks mark(const GlrArgs& a, int lo, int n, bool turned) {
  Marks m{0u, 0u, 0u, -1};
  if (n <= 0) return m;
  m.n0 = find_sequence(a.cu, a.nseq, lo);
  const uint32_t all = (1u << n) - 1u;
  if (m.n0 >= 0 && a.cu[m.n0] < lo && a.cu[m.n0 + 1] > lo + n) {  // amid one sequence: the usual case
    m.inside = all;
    return m;
  }
  int q = m.n0;
  for (int i = 0; i < n; ++i) {
    const int t = lo + i;
    while (q + 1 < a.nseq && a.cu[q + 1] <= t) ++q;
    if (q < 0 || t >= a.cu[q + 1]) continue;
    const int bit = turned ? n - 1 - i : i;
    m.inside |= 1u << bit;
    const bool lowest = t == a.cu[q], highest = t + 1 == a.cu[q + 1];
    if (a.dir ? highest : lowest) m.first |= 1u << bit;
    if (a.dir ? lowest : highest) m.last |= 1u << bit;
  }
  return m;
}

// Rows that no thread reaches through its tokens: states of sequences of no token, and the
// check of the lengths (addresses of tokens never depend on the lengths).
__device__ __forceinline__ void empty_sequences(const GlrArgs& a, int T, int c0, int width, const float* from, float* to,
                                                bool checks) {
  for (int n = threadIdx.x; n < a.nseq; n += kThreads) {
    const int s = a.cu[n], e = a.cu[n + 1];
    if (checks && (s < 0 || e > T || s > e)) report_status(GLA_ERR_INVALID_ARG);
    if (s == e && to)
      for (int c = c0; c < min(c0 + width, a.C); ++c) to[(int64_t)n * a.C + c] = from ? from[(int64_t)n * a.C + c] : 0.f;
  }
}

struct Place {
  uint32_t rank, size;
  int lane, sub, b, c;
  bool on;  // this thread's channels exist
};
template <int kLanes>
__device__ __forceinline__ Place place(const GlrArgs& a, int slabs) {
  Place p;
  p.rank = cluster_rank();
  p.size = cluster_size();
  const int slab = blockIdx.x / p.size;
  p.lane = threadIdx.x % kLanes;
  p.sub = threadIdx.x / kLanes;
  p.b = slab / slabs;
  p.c = ((slab - p.b * slabs) * kLanes + p.lane) * 2;
  p.on = p.c < a.C;
  return p;
}

// Row of scan position p (packed rows: the order is `dir` alone).
__device__ __forceinline__ int row_of(const ScanGeom& g, int p) { return scan_pos_to_token(g, p); }

// ---- forward ------------------------------------------------------------------------------
template <typename T, int kKind, bool kComp, int kLanes, int kRun>
__global__ void __launch_bounds__(kThreads) glr_fwd_k(GlrArgs a, ScanGeom g, int slabs, int rounds) {
  using G = GateT<T, kKind>;
  __shared__ Shared<kLanes> sm;
  const Place w = place<kLanes>(a, slabs);
  const T* x = static_cast<const T*>(a.x) + (int64_t)w.b * g.T * a.x_stride + w.c;
  const G* gate = static_cast<const G*>(a.gate) + (int64_t)w.b * g.T * a.gate_stride + w.c;
  T* out = static_cast<T*>(a.out) + (int64_t)w.b * g.T * a.C + w.c;
  const float inv_norm = 1.f / a.gate_norm;
  const bool packed = a.cu != nullptr;
  bool grown = false;
  cluster_arrive();  // the blocks of the cluster are running before one writes to another
  float carry[2] = {0.f, 0.f};
  if (!packed && a.h0 && w.on) {
    carry[0] = a.h0[(int64_t)w.b * a.C + w.c];
    carry[1] = a.h0[(int64_t)w.b * a.C + w.c + 1];
  }
  if (packed && w.rank == 0)
    empty_sequences(a, g.T, w.c - 2 * w.lane, 2 * kLanes, a.h0, a.h_last, blockIdx.x == 0);

  typename Two<T>::Raw rx[kRun];
  typename Two<G>::Raw rg[kRun];
  const int per_round = w.size * Shared<kLanes>::kSubs * kRun;
  int p0 = ((int)w.rank * Shared<kLanes>::kSubs + w.sub) * kRun;
  auto load = [&](int from) {
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      rx[i] = Two<T>::zero();
      rg[i] = Two<G>::zero();
      if (w.on && from + i < g.T) {
        const int64_t row = row_of(g, from + i);
        rx[i] = load2(x + row * a.x_stride);
        rg[i] = load2(gate + row * a.gate_stride);
      }
    }
  };
  load(p0);
  cluster_wait();
  for (int round = 0; round < rounds; ++round, p0 += per_round) {
    const int n = w.on ? max(0, min(kRun, g.T - p0)) : 0;
    Marks m{0u, 0u, 0u, 0};
    if (packed) m = mark<kRun>(a, a.dir ? g.T - p0 - n : p0, n, a.dir != 0);
    // Local inclusive scan: token i is A[i] * in + h[i] of what enters the thread's span.
    float A[2][kRun], h[2][kRun];
    Span s[2] = {{1.f, 0.f}, {1.f, 0.f}};
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      if (i < n) {
        const float2 xv = Two<T>::get(rx[i]), gv = Two<G>::get(rg[i]);
        const Gate k0 = make_gate<kKind>(gv.x, inv_norm), k1 = make_gate<kKind>(gv.y, inv_norm);
        float u0 = kComp ? k0.rest * xv.x : xv.x, u1 = kComp ? k1.rest * xv.y : xv.y;
        if (m.first >> i & 1u) {
          if (a.h0) {
            const float* from = a.h0 + state_row(a, row_of(g, p0 + i)) + w.c;
            u0 = fmaf(k0.alpha, from[0], u0);
            u1 = fmaf(k1.alpha, from[1], u1);
          }
          s[0] = Span{-0.f, u0};
          s[1] = Span{-0.f, u1};
        } else {
          s[0].h = fmaf(k0.alpha, s[0].h, u0);
          s[1].h = fmaf(k1.alpha, s[1].h, u1);
          s[0].A = join(s[0].A, k0.alpha, grown);
          s[1].A = join(s[1].A, k1.alpha, grown);
        }
      }
      A[0][i] = s[0].A;
      A[1][i] = s[1].A;
      h[0][i] = s[0].h;
      h[1][i] = s[1].h;
    }
    if (round + 1 < rounds) load(p0 + per_round);
    float in[2];
    exchange<kLanes>(sm, s, carry, in, round, w.rank, w.size, grown);
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      if (i >= n) continue;
      const int64_t row = row_of(g, p0 + i);
      const float2 v = make_float2(apply(Span{A[0][i], h[0][i]}, in[0]), apply(Span{A[1][i], h[1][i]}, in[1]));
      if (!packed || (m.inside >> i & 1u))
        store2(out + row * a.C, v);
      else if (a.fill)
        store2(out + row * a.C, make_float2(0.f, 0.f));
      if (a.h_last && (m.last >> i & 1u)) {
        float* to = a.h_last + state_row(a, (int)row) + w.c;
        to[0] = v.x;
        to[1] = v.y;
      }
    }
  }
  if (!packed && a.h_last && w.on && w.rank == 0 && w.sub == 0) {
    a.h_last[(int64_t)w.b * a.C + w.c] = carry[0];
    a.h_last[(int64_t)w.b * a.C + w.c + 1] = carry[1];
  }
  if (grown) report_status(GLA_ERR_RANGE);
}

// ---- backward -----------------------------------------------------------------------------
// The same walk from the last token to the first; position j of the walk is scan position
// T - 1 - j, and what enters a span is r of the token behind it.
template <typename T, int kKind, bool kComp, int kLanes, int kRun>
__global__ void __launch_bounds__(kThreads) glr_bwd_k(GlrArgs a, ScanGeom g, int slabs, int rounds) {
  using G = GateT<T, kKind>;
  __shared__ Shared<kLanes> sm;
  const Place w = place<kLanes>(a, slabs);
  const int64_t base = (int64_t)w.b * g.T;
  const T* x = static_cast<const T*>(a.x) + base * a.x_stride + w.c;
  const G* gate = static_cast<const G*>(a.gate) + base * a.gate_stride + w.c;
  const T* hs = static_cast<const T*>(a.h) + base * a.C + w.c;
  const T* dout = static_cast<const T*>(a.dout) + base * a.C + w.c;
  T* dx = static_cast<T*>(a.dx) + base * a.C + w.c;
  G* dgate = static_cast<G*>(a.dgate) + base * a.C + w.c;
  const float inv_norm = 1.f / a.gate_norm;
  const bool packed = a.cu != nullptr;
  bool grown = false;
  cluster_arrive();
  float carry[2] = {0.f, 0.f};
  if (!packed && a.dh_last && w.on) {
    carry[0] = a.dh_last[(int64_t)w.b * a.C + w.c];
    carry[1] = a.dh_last[(int64_t)w.b * a.C + w.c + 1];
  }
  if (packed && w.rank == 0)
    empty_sequences(a, g.T, w.c - 2 * w.lane, 2 * kLanes, a.dh_last, a.dh0, blockIdx.x == 0);

  typename Two<T>::Raw rx[kComp ? kRun : 1], rd[kRun], rh[kRun];
  typename Two<G>::Raw rg[kRun];
  const int per_round = w.size * Shared<kLanes>::kSubs * kRun;
  int j0 = ((int)w.rank * Shared<kLanes>::kSubs + w.sub) * kRun;
  auto load = [&](int from) {
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const int p = g.T - 1 - (from + i);
      rd[i] = rh[i] = Two<T>::zero();
      rg[i] = Two<G>::zero();
      if constexpr (kComp) rx[i] = Two<T>::zero();
      if (w.on && p >= 0) {
        const int64_t row = row_of(g, p);
        rd[i] = load2(dout + row * a.C);
        rg[i] = load2(gate + row * a.gate_stride);
        if constexpr (kComp) rx[i] = load2(x + row * a.x_stride);
        if (p > 0) rh[i] = load2(hs + (int64_t)row_of(g, p - 1) * a.C);
      }
    }
  };
  load(j0);
  cluster_wait();
  for (int round = 0; round < rounds; ++round, j0 += per_round) {
    const int n = w.on ? max(0, min(kRun, g.T - j0)) : 0;
    Marks m{0u, 0u, 0u, 0};
    // Walking backwards over tokens in forward order lowers the token by one each step.
    if (packed) m = mark<kRun>(a, a.dir ? j0 : g.T - j0 - n, n, a.dir == 0);
    // d of token i is d[i] + A[i] * in; pull[i] = alpha (h before - x) d log_alpha / d gate.
    float A[2][kRun], d[2][kRun], pull[2][kRun], keep[2][kComp ? kRun : 1];
    float al[2][kRun];
    Span s[2] = {{1.f, 0.f}, {1.f, 0.f}};
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      A[0][i] = A[1][i] = d[0][i] = d[1][i] = pull[0][i] = pull[1][i] = al[0][i] = al[1][i] = 0.f;
      if constexpr (kComp) keep[0][i] = keep[1][i] = 0.f;
      if (i >= n) continue;
      const int p = g.T - 1 - (j0 + i);
      const float2 gv = Two<G>::get(rg[i]);
      float2 dv = Two<T>::get(rd[i]), before = Two<T>::get(rh[i]);
      const Gate k0 = make_gate<kKind>(gv.x, inv_norm), k1 = make_gate<kKind>(gv.y, inv_norm);
      if (packed ? (m.first >> i & 1u) : p == 0) {
        before = make_float2(0.f, 0.f);
        if (a.h0) {
          const float* from = a.h0 + (packed ? state_row(a, row_of(g, p)) : (int64_t)w.b * a.C) + w.c;
          before = make_float2(from[0], from[1]);
        }
      }
      if (m.last >> i & 1u) {
        s[0] = s[1] = Span{-0.f, 0.f};
        if (a.dh_last) {
          const float* from = a.dh_last + state_row(a, row_of(g, p)) + w.c;
          s[0].h = from[0];
          s[1].h = from[1];
        }
      }
      if constexpr (kComp) {
        const float2 xv = Two<T>::get(rx[i]);
        before.x -= xv.x;
        before.y -= xv.y;
        keep[0][i] = k0.rest;
        keep[1][i] = k1.rest;
      }
      pull[0][i] = k0.alpha * before.x * k0.slope;
      pull[1][i] = k1.alpha * before.y * k1.slope;
      al[0][i] = k0.alpha;
      al[1][i] = k1.alpha;
      A[0][i] = s[0].A;
      A[1][i] = s[1].A;
      d[0][i] = dv.x + s[0].h;
      d[1][i] = dv.y + s[1].h;
      s[0].h = k0.alpha * d[0][i];
      s[1].h = k1.alpha * d[1][i];
      s[0].A = join(s[0].A, k0.alpha, grown);
      s[1].A = join(s[1].A, k1.alpha, grown);
    }
    if (round + 1 < rounds) load(j0 + per_round);
    float in[2];
    exchange<kLanes>(sm, s, carry, in, round, w.rank, w.size, grown);
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      if (i >= n) continue;
      const int64_t row = row_of(g, g.T - 1 - (j0 + i));
      const float d0 = apply(Span{A[0][i], d[0][i]}, in[0]), d1 = apply(Span{A[1][i], d[1][i]}, in[1]);
      float2 vx = make_float2(d0, d1), vg = make_float2(d0 * pull[0][i], d1 * pull[1][i]);
      if constexpr (kComp) vx = make_float2(d0 * keep[0][i], d1 * keep[1][i]);
      if (packed && !(m.inside >> i & 1u)) {
        if (!a.fill) continue;
        vx = vg = make_float2(0.f, 0.f);
      }
      store2(dx + row * a.C, vx);
      store2(dgate + row * a.C, vg);
      if (a.dh0 && (m.first >> i & 1u)) {
        float* to = a.dh0 + state_row(a, (int)row) + w.c;
        to[0] = al[0][i] * d0;
        to[1] = al[1][i] * d1;
      }
    }
  }
  if (!packed && a.dh0 && w.on && w.rank == 0 && w.sub == 0) {
    a.dh0[(int64_t)w.b * a.C + w.c] = carry[0];
    a.dh0[(int64_t)w.b * a.C + w.c + 1] = carry[1];
  }
  if (grown) report_status(GLA_ERR_RANGE);
}

// ---- launch -------------------------------------------------------------------------------
template <int kLanes, int kRun>
cudaError_t enqueue(void (*k)(GlrArgs, ScanGeom, int, int), const GlrArgs& a, const ScanGeom& g, int cluster,
                    cudaStream_t st) {
  const int slabs = (a.C + 2 * kLanes - 1) / (2 * kLanes);
  const int per_round = cluster * (kThreads / kLanes) * kRun;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)((int64_t)a.B * slabs * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, a, g, slabs, (g.T + per_round - 1) / per_round);
}

// The widest cluster whose blocks are all resident (`blocks` of them) and have tokens.
int cluster_for(int64_t slabs, int T, int per_block, int64_t blocks) {
  int c = 1;
  while (c < kMaxCluster && slabs * c * 2 <= blocks && (int64_t)c * per_block < T) c *= 2;
  return c;
}

template <typename T, int kKind, bool kComp>
cudaError_t launch(const GlrArgs& a, bool bwd, cudaStream_t st) {
  constexpr int kRun = sizeof(T) == 2 ? 8 : 4;
  const ScanGeom g = make_geom(a.Hg, a.Wg, a.dir);
  const int64_t wide = (int64_t)a.B * ((a.C + 63) / 64), blocks = 296;
  if (wide * kMaxCluster >= blocks / 2 || g.T <= (kThreads / 32) * kRun) {
    const int c = cluster_for(wide, g.T, (kThreads / 32) * kRun, blocks);
    return enqueue<32, kRun>(bwd ? glr_bwd_k<T, kKind, kComp, 32, kRun> : glr_fwd_k<T, kKind, kComp, 32, kRun>, a, g, c, st);
  }
  const int64_t narrow = (int64_t)a.B * ((a.C + 15) / 16);
  const int c = cluster_for(narrow, g.T, (kThreads / 8) * kRun, blocks);
  return enqueue<8, kRun>(bwd ? glr_bwd_k<T, kKind, kComp, 8, kRun> : glr_fwd_k<T, kKind, kComp, 8, kRun>, a, g, c, st);
}

template <typename T, bool kComp>
cudaError_t by_gate(const GlrArgs& a, bool bwd, cudaStream_t st) {
  switch (gate_kind(a.gate_norm)) {
    case kGateLog: return launch<T, kGateLog, kComp>(a, bwd, st);
    case kGateSigmoid: return launch<T, kGateSigmoid, kComp>(a, bwd, st);
    default: return launch<T, kGateLogit, kComp>(a, bwd, st);
  }
}
template <typename T>
cudaError_t by_form(const GlrArgs& a, bool bwd, cudaStream_t st) {
  return a.complement ? by_gate<T, true>(a, bwd, st) : by_gate<T, false>(a, bwd, st);
}

}  // namespace

cudaError_t glr_fwd_launch(const GlrArgs& a, cudaStream_t st) {
  return a.bf16 ? by_form<__nv_bfloat16>(a, false, st) : by_form<float>(a, false, st);
}
cudaError_t glr_bwd_launch(const GlrArgs& a, cudaStream_t st) {
  return a.bf16 ? by_form<__nv_bfloat16>(a, true, st) : by_form<float>(a, true, st);
}

}  // namespace dig
