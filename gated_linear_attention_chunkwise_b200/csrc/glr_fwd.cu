// glr_fwd.cu -- the gated linear recurrence over a token grid in scan order or over packed
// sequences (include/dig_gla.h, glr_fwd, glr_fwd_packed).  The walk: glr_scan.cuh.
#include "glr_scan.cuh"

namespace dig {
namespace glr {
namespace {

// Blocks an SM that the registers allow: with log_alpha four (128 registers, the c4 grid 65
// instead of 67 us with three); the gates of the other forms would spill (packed, logits and
// complement: 402 us with four, 347 with three).
constexpr int resident(int kind, bool comp) { return kind == kGateLog && !comp ? 4 : 3; }

template <typename T, int kKind, bool kComp, int kLanes, int kRun>
__global__ void __launch_bounds__(kThreads, resident(kKind, kComp))
    glr_fwd_k(GlrArgs a, ScanGeom g, int slabs, int rounds) {
  using G = GateT<T, kKind>;
  using RawT = typename Four<T>::Raw;
  using RawG = typename Four<G>::Raw;
  __shared__ Shared<kLanes> sm;
  extern __shared__ uint4 slots[];  // the tokens of a round: gates [kRun][kThreads], then x
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
  const uint32_t slot_g = smem_u32(sg), slot_x = smem_u32(sx);
  constexpr uint32_t kStepG = kThreads * sizeof(RawG), kStepX = kThreads * sizeof(RawT);
  auto load = [&](int from) {
    Rows rows(g, from, 1);
    int apart;
    if (on && from + kRun <= g.T && rows.even(g, kRun, apart)) {
      const int row = rows.next(g);
      const G* pg = gate + row * a.gate_stride;
      const T* px = x + row * a.x_stride;
      const int64_t dg = apart * a.gate_stride, dx = apart * a.x_stride;
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        fetch<G>(slot_g + i * kStepG, pg, true);
        fetch<T>(slot_x + i * kStepX, px, true);
        pg += dg;
        px += dx;
      }
    } else {
#pragma unroll 1
      for (int i = 0; i < kRun; ++i) {
        const bool there = on && from + i < g.T;
        const int row = there ? rows.next(g) : 0;
        fetch<G>(slot_g + i * kStepG, gate + row * a.gate_stride, there);
        fetch<T>(slot_x + i * kStepX, x + row * a.x_stride, there);
      }
    }
    cp_async_commit();
  };
  load(p0);
  if (packed && walk.rank == 0)
    empty_sequences(a, g.T, c - 4 * walk.lane, 4 * kLanes, a.h0, a.h_last, blockIdx.x == 0);
  cluster_wait();

  bool grown = false;
  Amid amid;
  Marks next;
  F4 next_entry = all4(0.f);  // stays zero without h0
  auto look = [&](int from) {
    const int n = on ? max(0, min(kRun, g.T - from)) : 0;
    next = mark(a, a.dir ? g.T - from - n : from, n, a.dir != 0, amid);
    // Fetched a round ahead: a thread that waited for it would hold up its whole cluster.
    if (next.first && a.h0) next_entry = load4(a.h0 + (int64_t)next.first_seq * a.C + c);
  };
  if (packed) look(p0);
  for (int round = 0; round < rounds; ++round, p0 += per_round) {
    const int n = on ? max(0, min(kRun, g.T - p0)) : 0;
    const Marks m = next;
    const F4 entry = next_entry;
    cp_async_wait_all();
    F4 al[kRun], u[kRun];
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const Gates4 k = make_gates4<T, kKind, kComp>(Four<G>::get(sg[i * kThreads]), inv_norm);
      u[i] = Four<T>::get(sx[i * kThreads]);
      if constexpr (kComp) u[i] = mul4(k.rest, u[i]);
      al[i] = k.alpha;
    }
    // Rows of no sequence pass on what enters them, whatever they hold.
    if (packed && m.inside != (1u << kRun) - 1u) {
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        if (m.inside >> i & 1u) continue;
        al[i] = all4(1.f);
        u[i] = all4(0.f);
      }
    }
    // The first token of a sequence takes its state in and forgets the token before.
    if (m.first) {
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        if (!(m.first >> i & 1u)) continue;
        F4 from = entry;
        if (a.h0 && (m.first & ((1u << i) - 1u)))
          from = load4(a.h0 + state_row(a, m.first, i, m.first_seq, a.dir ? g.T - 1 - (p0 + i) : p0 + i) + c);
        u[i] = fma4(al[i], from, u[i]);
        al[i] = all4(0.f);
      }
    }
    Span s{al[0], u[0]};
#pragma unroll
    for (int i = 1; i < kRun; ++i) s = Span{mul4(s.A, al[i]), fma4(al[i], s.h, u[i])};
    bool odd = !all_within(s.A, 1.f) || (packed && !modest(s.h));
    if (n < kRun || odd) {  // the last round's end, growth, values that may not stay finite
      s = nothing();
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        if (i >= n) {
          al[i] = all4(1.f);
          u[i] = all4(0.f);
        }
        if (m.first >> i & 1u)
          s = Span{all4(0.f), u[i]};
        else
          s = Span{capped(mul4(s.A, capped(al[i], grown)), grown), fma4(al[i], s.h, u[i])};
      }
      odd = !all_within(s.A, 1.f) || (packed && !modest(s.h));
    }
    if (m.first) s.A.a.x = -0.f;
    F4 h;
    const bool going = walk.exchange(s, odd, packed, round, h, grown, [&] {
      // The tokens are in registers: their slots are free for the next round's.
      if (round + 1 < rounds) {
        load(p0 + per_round);
        if (packed) look(p0 + per_round);
      }
    });
    if (!going) break;
    Rows rows(g, p0, 1);
    int apart;
    if (!rows.even(g, kRun, apart)) {  // grids alone
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        h = fma4(al[i], h, u[i]);
        if (i < n) store4(out + (int64_t)rows.next(g) * a.C, h);
      }
      continue;
    }
    const uint32_t write = packed ? m.inside : (1u << n) - 1u;
    T* po = out + (int64_t)rows.next(g) * a.C;
    const int64_t d = (int64_t)apart * a.C;
    if (write == (1u << kRun) - 1u && (m.first | m.last) == 0u) {
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        h = fma4(al[i], h, u[i]);
        store4(po, h);
        po += d;
      }
      continue;
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      h = m.first >> i & 1u ? u[i] : fma4(al[i], h, u[i]);
      if (write >> i & 1u)
        store4(po, h);
      else if (a.fill && i < n)
        store4(po, all4(0.f));
      if (a.h_last && (m.last >> i & 1u))
        store4(a.h_last + state_row(a, m.last, i, m.last_seq, a.dir ? g.T - 1 - (p0 + i) : p0 + i) + c, h);
      po += d;
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
    const size_t smem = (size_t)kRun * kThreads * (sizeof(typename Four<T>::Raw) + sizeof(typename Four<GateT<T, kKind>>::Raw));
    static Known known8, known4;
    return enqueue(glr_fwd_k<T, kKind, kComp, 8, kRun>, known8, glr_fwd_k<T, kKind, kComp, 4, kRun>, known4, a, kRun, smem, st);
  }
};

}  // namespace
}  // namespace glr

cudaError_t glr_fwd_launch(const GlrArgs& a, cudaStream_t st) { return glr::by_types<glr::Forward>(a, st); }

}  // namespace dig
