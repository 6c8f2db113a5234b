// glr_fwd.cu -- the gated linear recurrence over a token grid in scan order or over packed
// sequences (include/dig_gla.h, glr_fwd, glr_fwd_packed).  The walk: glr_scan.cuh.
#include "glr_scan.cuh"

namespace dig {
namespace glr {
namespace {

template <typename T, int kKind, bool kComp, int kLanes, int kRun>
__global__ void __launch_bounds__(kThreads, 2) glr_fwd_k(GlrArgs a, ScanGeom g, int slabs, int rounds) {
  using G = GateT<T, kKind>;
  using RawT = typename Four<T>::Raw;
  using RawG = typename Four<G>::Raw;
  __shared__ Shared<kLanes> sm;
  extern __shared__ uint4 slots[];  // this round's tokens: gates [kRun][kThreads], then x
  RawG* const sg = reinterpret_cast<RawG*>(slots) + threadIdx.x;
  RawT* const sx = reinterpret_cast<RawT*>(reinterpret_cast<RawG*>(slots) + kRun * kThreads) + threadIdx.x;

  const int slab = blockIdx.x / cluster_size(), b = slab / slabs;
  const int c = ((slab - b * slabs) * kLanes + threadIdx.x % kLanes) * 4;
  const bool on = c < a.C;  // this thread's channels exist
  const bool packed = a.cu != nullptr;
  const int64_t base = (int64_t)b * g.T;
  const T* const x = static_cast<const T*>(a.x) + base * a.x_stride + (on ? c : 0);
  const G* const gate = static_cast<const G*>(a.gate) + base * a.gate_stride + (on ? c : 0);
  T* const out = static_cast<T*>(a.out) + base * a.C + c;
  const float inv_norm = 1.f / a.gate_norm;

  F4 start = all4(0.f);
  if (!packed && a.h0 && on) start = load4(a.h0 + (int64_t)b * a.C + c);
  Walk<kLanes> walk(sm, start);
  const int per_round = (int)walk.size * (kThreads / kLanes) * kRun;
  int p0 = ((int)walk.rank * (kThreads / kLanes) + threadIdx.x / kLanes) * kRun;
  int row[kRun];
  auto load = [&](int from) {
    Rows rows(g, from, 1);
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const bool there = on && from + i < g.T;
      row[i] = there ? rows.next() : 0;
      fetch<G>(smem_u32(sg + i * kThreads), gate + row[i] * a.gate_stride, there);
      fetch<T>(smem_u32(sx + i * kThreads), x + row[i] * a.x_stride, there);
    }
    cp_async_commit();
  };
  load(p0);
  if (packed && walk.rank == 0)
    empty_sequences(a, g.T, c - 4 * walk.lane, 4 * kLanes, a.h0, a.h_last, blockIdx.x == 0);
  cluster_wait();

  bool grown = false;
  for (int round = 0; round < rounds; ++round, p0 += per_round) {
    const int n = on ? max(0, min(kRun, g.T - p0)) : 0;
    Marks m{0u, 0u, 0u};
    if (packed) m = mark(a, a.dir ? g.T - p0 - n : p0, n, a.dir != 0);
    cp_async_wait_all();
    F4 al[kRun], u[kRun];
    Span s{all4(1.f), all4(0.f)};
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const Gates4 k = make_gates4<kKind>(Four<G>::get(sg[i * kThreads]), inv_norm);
      u[i] = Four<T>::get(sx[i * kThreads]);
      if constexpr (kComp) u[i] = mul4(k.rest, u[i]);
      al[i] = k.alpha;
      if (i >= n) {
        al[i] = all4(1.f);
        u[i] = all4(0.f);
      }
      if (m.first >> i & 1u) {
        if (a.h0) u[i] = fma4(al[i], load4(a.h0 + state_row(a, row[i]) + c), u[i]);
        s = Span{all4(1.f), u[i]};
      } else {
        s = Span{mul4(s.A, al[i]), fma4(al[i], s.h, u[i])};
      }
    }
    if (any_over(s.A) || s.A.a.x != s.A.a.x || s.A.a.y != s.A.a.y || s.A.b.x != s.A.b.x || s.A.b.y != s.A.b.y) {
      s.A = all4(1.f);  // growth, or a NaN: multiply again with a cap
#pragma unroll
      for (int i = 0; i < kRun; ++i)
        s.A = m.first >> i & 1u ? all4(1.f) : product<false>(s.A, cap(al[i]), grown), grown |= any_over(al[i]);
    }
    if (m.first) s.A = all4(-0.f);
    // The tokens are in registers: the slots are free for the next round's.
    int at[kRun];
#pragma unroll
    for (int i = 0; i < kRun; ++i) at[i] = row[i];
    if (round + 1 < rounds) load(p0 + per_round);
    F4 h;
    if (!(packed ? walk.template exchange<true>(s, round, h, grown) : walk.template exchange<false>(s, round, h, grown)))
      break;
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      h = m.first >> i & 1u ? u[i] : fma4(al[i], h, u[i]);
      if (i >= n) continue;
      if (!packed || (m.inside >> i & 1u))
        store4(out + (int64_t)at[i] * a.C, h);
      else if (a.fill)
        store4(out + (int64_t)at[i] * a.C, all4(0.f));
      if (a.h_last && (m.last >> i & 1u)) store4(a.h_last + state_row(a, at[i]) + c, h);
    }
  }
  cp_async_wait_all();
  if (!packed && a.h_last && on && walk.rank == 0 && threadIdx.x < kLanes)
    store4(a.h_last + (int64_t)b * a.C + c, walk.carry);
  if (grown) report_status(GLA_ERR_RANGE);
  walk.leave();
}

template <typename T, int kKind, bool kComp>
struct Forward {
  static cudaError_t run(const GlrArgs& a, cudaStream_t st) {
    constexpr int kRun = 8;
    const ScanGeom g = make_geom(a.Hg, a.Wg, a.dir);
    const size_t smem = (size_t)kRun * kThreads * (sizeof(typename Four<T>::Raw) + sizeof(typename Four<GateT<T, kKind>>::Raw));
    const int64_t wide = (int64_t)a.B * ((a.C + 63) / 64);
    if (wide * kMaxCluster >= 148 || g.T <= kThreads / 16 * kRun)
      return enqueue(glr_fwd_k<T, kKind, kComp, 16, kRun>, a, g, 16, kRun, 296, smem, st);
    return enqueue(glr_fwd_k<T, kKind, kComp, 4, kRun>, a, g, 4, kRun, 296, smem, st);
  }
};

}  // namespace
}  // namespace glr

cudaError_t glr_fwd_launch(const GlrArgs& a, cudaStream_t st) { return glr::by_types<glr::Forward>(a, st); }

}  // namespace dig
