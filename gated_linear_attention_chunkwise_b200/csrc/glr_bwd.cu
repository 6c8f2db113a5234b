// glr_bwd.cu -- the gradients of the gated linear recurrence (include/dig_gla.h, glr_bwd,
// glr_bwd_packed): the walk of glr_scan.cuh from the last token to the first.  Position j of
// the walk is scan position T - 1 - j; what enters a span is r of the token behind it.
//
// Four tokens a thread, since a token needs four values a channel (alpha, d and the two
// factors of the gradients): packed 32749 x 2048, logits and complement, 314 us; eight tokens
// and two blocks an SM 316, four and four blocks (spilling) 362.  (With log_alpha alone both
// would be faster: 64 sequences of 1024 x 2048 436 us, 398 and 379.)
#include "glr_scan.cuh"

namespace dig {
namespace glr {
namespace {

template <typename T, int kKind, bool kComp, int kLanes, int kRun>
__global__ void __launch_bounds__(kThreads, 3) glr_bwd_k(GlrArgs a, ScanGeom g, int slabs, int rounds) {
  using G = GateT<T, kKind>;
  using RawT = typename Four<T>::Raw;
  using RawG = typename Four<G>::Raw;
  __shared__ Shared<kLanes> sm;
  extern __shared__ uint4 slots[];  // gates [kRun][kThreads], then dout, h of the token before, x
  RawG* const sg = reinterpret_cast<RawG*>(slots) + threadIdx.x;
  RawT* const sd = reinterpret_cast<RawT*>(reinterpret_cast<RawG*>(slots) + kRun * kThreads) + threadIdx.x;
  RawT* const sh = sd + kRun * kThreads;
  RawT* const sx = sh + kRun * kThreads;

  const int slab = blockIdx.x / cluster_size(), b = slab / slabs;
  const int c = ((slab - b * slabs) * kLanes + threadIdx.x % kLanes) * 4;
  const bool on = c < a.C;
  const bool packed = a.cu != nullptr;
  const int64_t base = (int64_t)b * g.T;
  const int c_in = on ? c : 0;
  const T* const x = static_cast<const T*>(a.x) + base * a.x_stride + c_in;
  const G* const gate = static_cast<const G*>(a.gate) + base * a.gate_stride + c_in;
  const T* const hs = static_cast<const T*>(a.h) + base * a.C + c_in;
  const T* const dout = static_cast<const T*>(a.dout) + base * a.C + c_in;
  T* const dx = static_cast<T*>(a.dx) + base * a.C + c;
  G* const dgate = static_cast<G*>(a.dgate) + base * a.C + c;
  const float inv_norm = 1.f / a.gate_norm;

  F4 start = all4(0.f);
  if (!packed && a.dh_last && on) start = load4(a.dh_last + (int64_t)b * a.C + c);
  Walk<kLanes> walk(sm, start);
  const int per_round = (int)walk.size * (kThreads / kLanes) * kRun;
  int j0 = ((int)walk.rank * (kThreads / kLanes) + threadIdx.x / kLanes) * kRun;
  const uint32_t slot_g = smem_u32(sg), slot_d = smem_u32(sd), slot_h = smem_u32(sh), slot_x = smem_u32(sx);
  constexpr uint32_t kStepG = kThreads * sizeof(RawG), kStepT = kThreads * sizeof(RawT);
  auto load = [&](int from) {
    Rows rows(g, g.T - 1 - from, -1);
    int apart;
    if (on && from + kRun < g.T && rows.even(g, kRun + 1, apart)) {
      const int64_t row = rows.next(g);
      const G* pg = gate + row * a.gate_stride;
      const T *pd = dout + row * a.C, *ph = hs + (row + apart) * a.C, *px = x + row * a.x_stride;
      const int64_t dg = apart * a.gate_stride, dc = (int64_t)apart * a.C, ds = apart * a.x_stride;
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        fetch<G>(slot_g + i * kStepG, pg, true);
        fetch<T>(slot_d + i * kStepT, pd, true);
        fetch<T>(slot_h + i * kStepT, ph, true);
        if constexpr (kComp) fetch<T>(slot_x + i * kStepT, px, true);
        pg += dg;
        pd += dc;
        ph += dc;
        px += ds;
      }
    } else {
      int next = on && from < g.T ? rows.next(g) : 0;
#pragma unroll 1
      for (int i = 0; i < kRun; ++i) {
        const bool there = on && from + i < g.T, before = on && from + i + 1 < g.T;
        const int64_t row = next;
        next = before ? rows.next(g) : 0;
        fetch<G>(slot_g + i * kStepG, gate + row * a.gate_stride, there);
        fetch<T>(slot_d + i * kStepT, dout + row * a.C, there);
        fetch<T>(slot_h + i * kStepT, hs + (int64_t)next * a.C, before);
        if constexpr (kComp) fetch<T>(slot_x + i * kStepT, x + row * a.x_stride, there);
      }
    }
    cp_async_commit();
  };
  load(j0);
  if (packed && walk.rank == 0)
    empty_sequences(a, g.T, c - 4 * walk.lane, 4 * kLanes, a.dh_last, a.dh0, blockIdx.x == 0);
  cluster_wait();

  bool grown = false;
  Amid amid;
  Marks next;
  F4 next_entry = all4(0.f);
  auto look = [&](int from) {
    // Backwards over sequences in token order the token falls by one each step.
    const int n = on ? max(0, min(kRun, g.T - from)) : 0;
    next = mark(a, a.dir ? from : g.T - from - n, n, a.dir == 0, amid);
    // Fetched a round ahead: a thread that waited for it would hold up its whole cluster.
    if (next.last && a.dh_last) next_entry = load4(a.dh_last + (int64_t)next.last_seq * a.C + c);
  };
  if (packed) look(j0);
  for (int round = 0; round < rounds; ++round, j0 += per_round) {
    const int n = on ? max(0, min(kRun, g.T - j0)) : 0;
    Marks m = next;
    const F4 entry = next_entry;
    if (!packed && n > 0 && j0 + n == g.T) m.first = 1u << (n - 1);  // the scan's first token
    cp_async_wait_all();
    // pull = (h before - [complement] x) d log_alpha / d gate, keep = 1 - alpha.
    F4 al[kRun], d[kRun], pull[kRun], keep[kComp ? kRun : 1];
    auto token = [&](int i) { return a.dir ? j0 + i : g.T - 1 - (j0 + i); };  // of packed rows
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const Gates4 k = make_gates4<T, kKind, kComp>(Four<G>::get(sg[i * kThreads]), inv_norm);
      F4 before = Four<T>::get(sh[i * kThreads]);
      d[i] = Four<T>::get(sd[i * kThreads]);
      al[i] = k.alpha;
      if (m.first >> i & 1u) {
        before = all4(0.f);
        if (a.h0)
          before = load4(a.h0 + (packed ? state_row(a, m.first, i, m.first_seq, token(i)) : (int64_t)b * a.C) + c);
      }
      if constexpr (kComp) {
        before = sub4(before, Four<T>::get(sx[i * kThreads]));
        keep[i] = k.rest;
      }
      pull[i] = kKind == kGateLog ? before : mul4(before, k.slope);
    }
    // The last token of a sequence takes dh_last in and forgets the token behind.
    Span s = nothing();
    if (m.last) {
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        if (m.last >> i & 1u) {
          F4 from = entry;
          if (a.dh_last && (m.last & ((1u << i) - 1u)))
            from = load4(a.dh_last + state_row(a, m.last, i, m.last_seq, token(i)) + c);
          d[i] = add4(d[i], from);
          s = Span{all4(0.f), all4(0.f)};
        }
        s = Span{mul4(s.A, al[i]), mul4(al[i], add4(d[i], s.h))};
      }
    } else {
#pragma unroll
      for (int i = 0; i < kRun; ++i) s = Span{mul4(s.A, al[i]), mul4(al[i], add4(d[i], s.h))};
    }
    bool odd = !all_within(s.A, 1.f) || (packed && !modest(s.h));
    // The last round's end, rows of no sequence (which pass on what enters them, whatever they
    // hold), growth, values that may not stay finite.
    const uint32_t there = packed ? m.inside : (1u << n) - 1u;
    if (there != (1u << kRun) - 1u || odd) {
      s = nothing();
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        if (!(there >> i & 1u)) {
          al[i] = all4(1.f);
          d[i] = all4(0.f);
        }
        if (m.last >> i & 1u) s = Span{all4(0.f), all4(0.f)};
        s = Span{capped(mul4(s.A, capped(al[i], grown)), grown), mul4(al[i], add4(d[i], s.h))};
      }
      odd = !all_within(s.A, 1.f) || (packed && !modest(s.h));
    }
    if (m.last) s.A.a.x = -0.f;
    F4 r;
    const bool going = walk.exchange(s, odd, packed, round, r, grown, [&] {
      if (round + 1 < rounds) {
        load(j0 + per_round);
        if (packed) look(j0 + per_round);
      }
    });
    if (!going) break;
    Rows rows(g, g.T - 1 - j0, -1);
    int apart;
    if (!rows.even(g, kRun, apart)) {  // grids alone
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        const F4 delta = add4(d[i], r);
        r = mul4(al[i], delta);
        if (i >= n) continue;
        const int64_t row = rows.next(g);
        store4(dx + row * a.C, kComp ? mul4(delta, keep[kComp ? i : 0]) : delta);
        store4(dgate + row * a.C, mul4(r, pull[i]));
      }
      continue;
    }
    const int64_t row = rows.next(g), step = (int64_t)apart * a.C;
    T* px = dx + row * a.C;
    G* pg = dgate + row * a.C;
    if (there == (1u << kRun) - 1u && (!packed || (m.first | m.last) == 0u)) {
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        const F4 delta = add4(d[i], r);
        r = mul4(al[i], delta);
        store4(px, kComp ? mul4(delta, keep[kComp ? i : 0]) : delta);
        store4(pg, mul4(r, pull[i]));
        px += step;
        pg += step;
      }
      continue;
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const F4 delta = m.last >> i & 1u ? d[i] : add4(d[i], r);
      r = mul4(al[i], delta);
      if (packed && a.dh0 && (m.first >> i & 1u))
        store4(a.dh0 + state_row(a, m.first, i, m.first_seq, token(i)) + c, r);
      if (there >> i & 1u) {
        store4(px, kComp ? mul4(delta, keep[kComp ? i : 0]) : delta);
        store4(pg, mul4(r, pull[i]));
      } else if (a.fill && i < n) {
        store4(px, all4(0.f));
        store4(pg, all4(0.f));
      }
      px += step;
      pg += step;
    }
  }
  cp_async_wait_all();
  if (!packed && a.dh0 && on && walk.rank == 0 && threadIdx.x < kLanes)
    store4(a.dh0 + (int64_t)b * a.C + c, walk.carry);
  if (grown) report_status(GLA_ERR_RANGE);
  walk.leave();
}

template <typename T, int kKind, bool kComp>
struct Backward {
  static cudaError_t run(const GlrArgs& a, cudaStream_t st) {
    constexpr int kRun = 4;
    const size_t smem = (size_t)kRun * kThreads *
                        ((kComp ? 3 : 2) * sizeof(typename Four<T>::Raw) + sizeof(typename Four<GateT<T, kKind>>::Raw));
    static Known known8, known4;
    return enqueue(glr_bwd_k<T, kKind, kComp, 8, kRun>, known8, glr_bwd_k<T, kKind, kComp, 4, kRun>, known4, a, kRun, smem, st);
  }
};

}  // namespace
}  // namespace glr

cudaError_t glr_bwd_launch(const GlrArgs& a, cudaStream_t st) { return glr::by_types<glr::Backward>(a, st); }

}  // namespace dig
