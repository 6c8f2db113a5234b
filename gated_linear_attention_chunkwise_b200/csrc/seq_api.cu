// seq_api.cu -- the extern "C" entry points of the sequence operators: the gated linear
// recurrence (glr_*), rotary positions and the query/key norm (rope, qk_norm_rope*).
// Like api.cu: arguments are checked on the host before anything is enqueued, then the
// device, then the kernels go on the caller's stream.
#include <cmath>

#include "dig_gla.h"
#include "internal.h"

namespace {

using dig::aligned16;
using dig::overlaps;

// A tensor of token rows: `width` bytes every `pitch` bytes.
struct Rows {
  const void* p;
  int64_t pitch, width, n;
  size_t span() const { return (size_t)((n - 1) * pitch + width); }
};

// Whether two tensors share a byte.  Slices of one fused projection interleave without
// sharing any: with equal pitches the rows are disjoint when their columns are.
bool clash(const Rows& a, const Rows& b) {
  if (!a.p || !b.p || !overlaps(a.p, a.span(), b.p, b.span())) return false;
  if (a.pitch != b.pitch) return true;
  int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p)) % a.pitch;
  if (d < 0) d += a.pitch;
  return !(d >= a.width && d + b.width <= a.pitch);
}
bool same(const Rows& a, const Rows& b) { return a.p == b.p && a.pitch == b.pitch && a.width == b.width; }
Rows dense(const void* p, int64_t bytes) { return Rows{p, bytes, bytes, 1}; }

// ---- gated linear recurrence ----------------------------------------------------

int check_glr_shape(int64_t rows, int64_t nseq, int C, int64_t x_stride, int64_t gate_stride, float gate_norm,
                    int complement, int dtype) {
  if (rows <= 0 || nseq <= 0 || C <= 0) return GLA_ERR_INVALID_ARG;
  if (dtype != GLA_BF16 && dtype != GLA_F32) return GLA_ERR_INVALID_ARG;
  if (!(gate_norm == 0.f || gate_norm >= 1e-30f) || std::isinf(gate_norm) || (complement != 0 && complement != 1)) return GLA_ERR_INVALID_ARG;
  if (x_stride < C || gate_stride < C) return GLA_ERR_INVALID_ARG;
  const int64_t elt = dtype == GLA_BF16 ? 2 : 4, gelt = gate_norm == 0.f ? 4 : elt;
  if (C > 65536 || nseq > (1 << 24) || nseq * ((C + 63) / 64) > (int64_t)1 << 26) return GLA_ERR_UNSUPPORTED;
  if (x_stride > (int64_t)1 << 32 || gate_stride > (int64_t)1 << 32) return GLA_ERR_UNSUPPORTED;
  if (rows > ((int64_t)1 << 42) / (x_stride > gate_stride ? x_stride : gate_stride)) return GLA_ERR_UNSUPPORTED;
  if (C * elt % 16 || x_stride * elt % 16 || gate_stride * gelt % 16) return GLA_ERR_ALIGNMENT;
  return GLA_OK;
}

// Shapes, pointers and aliasing of a forward or backward call (fields of `a` set).
int check_glr(const dig::GlrArgs& a, int64_t rows, bool bwd) {
  const int64_t elt = a.bf16 ? 2 : 4, gelt = a.gate_norm == 0.f ? 4 : elt;
  if (!a.x || !a.gate) return GLA_ERR_INVALID_ARG;
  if (bwd ? (!a.h || !a.dout || !a.dx || !a.dgate) : !a.out) return GLA_ERR_INVALID_ARG;
  if (a.dir < 0 || a.dir > (a.cu ? 1 : dig::kDirLast)) return GLA_ERR_INVALID_ARG;
  if (a.fill != 0 && a.fill != 1) return GLA_ERR_INVALID_ARG;
  const void* all[] = {a.x, a.gate, a.h0, a.out, a.h_last, a.h, a.dout, a.dh_last, a.dx, a.dgate, a.dh0};
  for (const void* p : all)
    if (!aligned16(p)) return GLA_ERR_ALIGNMENT;
  if (reinterpret_cast<uintptr_t>(a.cu) & 3u) return GLA_ERR_ALIGNMENT;
  const int64_t row = a.C * elt, grow = a.C * gelt, state = (int64_t)a.nseq * a.C * 4;
  const Rows in[] = {Rows{a.x, a.x_stride * elt, row, rows}, Rows{a.gate, a.gate_stride * gelt, grow, rows},
                     dense(a.cu, ((int64_t)a.nseq + 1) * 4), dense(a.h0, state), dense(a.h, rows * row),
                     dense(a.dout, rows * row), dense(a.dh_last, state)};
  const Rows out[] = {dense(a.out, rows * row), dense(a.dx, rows * row), dense(a.dgate, rows * grow),
                      dense(a.h_last, state), dense(a.dh0, state)};
  for (int o = 0; o < 5; ++o) {
    if (!out[o].p) continue;
    for (const Rows& i : in) {
      // The states may be updated in place: h_last over h0, dh0 over dh_last.
      const bool in_place = (o == 3 && i.p == a.h0) || (o == 4 && i.p == a.dh_last);
      if (clash(out[o], i) && !(in_place && same(out[o], i))) return GLA_ERR_INVALID_ARG;
    }
    for (int o2 = o + 1; o2 < 5; ++o2)
      if (clash(out[o], out[o2])) return GLA_ERR_INVALID_ARG;
  }
  return GLA_OK;
}

int grid_shape(int B, int Hgrid, int Wgrid, int64_t* rows) {
  if (B <= 0 || Hgrid <= 0 || Wgrid <= 0) return GLA_ERR_INVALID_ARG;
  const int64_t T = (int64_t)Hgrid * Wgrid;
  if (T > (int64_t)1 << 30) return GLA_ERR_UNSUPPORTED;
  *rows = B * T;
  return GLA_OK;
}

int run_glr(const dig::GlrArgs& a, int64_t rows, int dtype, bool bwd, cudaStream_t st) {
  int rc = check_glr_shape(rows, a.nseq, a.C, a.x_stride, a.gate_stride, a.gate_norm, a.complement, dtype);
  if (rc != GLA_OK) return rc;
  if ((rc = check_glr(a, rows, bwd)) != GLA_OK) return rc;
  if ((rc = dig::check_device()) != GLA_OK) return rc;
  return (bwd ? dig::glr_bwd_launch(a, st) : dig::glr_fwd_launch(a, st)) == cudaSuccess ? GLA_OK : GLA_ERR_CUDA;
}

dig::GlrArgs glr_args(const void* x, const void* gate, int64_t x_stride, int64_t gate_stride, const float* h0, int C,
                      int dir, float gate_norm, int complement, int dtype) {
  dig::GlrArgs a{};
  a.x = x;
  a.gate = gate;
  a.x_stride = x_stride;
  a.gate_stride = gate_stride;
  a.h0 = h0;
  a.C = C;
  a.dir = dir;
  a.gate_norm = gate_norm;
  a.complement = complement;
  a.bf16 = dtype == GLA_BF16;
  return a;
}
void on_grid(dig::GlrArgs* a, int B, int Hgrid, int Wgrid) {
  a->B = a->nseq = B;
  a->Hg = Hgrid;
  a->Wg = Wgrid;
}
void on_packed(dig::GlrArgs* a, const int* cu, int nseq, int rows, int fill) {
  a->cu = cu;
  a->nseq = nseq;
  a->B = a->Hg = 1;
  a->Wg = rows;
  a->fill = fill;
}

// ---- rotary positions, query/key norm ---------------------------------------------

Rows head_rows(const void* p, int64_t stride, int H, int D, int64_t rows, int64_t elt) {
  return Rows{p, stride * elt, (int64_t)H * D * elt, rows};
}

// norm: weights are needed; bwd: gradients are.
int check_qk(const dig::QkRopeArgs& a, int dtype, bool norm, bool bwd) {
  if (dtype != GLA_BF16 && dtype != GLA_F32) return GLA_ERR_INVALID_ARG;
  if (a.rows <= 0 || a.D <= 0 || a.rot < 0 || a.q.H <= 0 || a.k.H < 0) return GLA_ERR_INVALID_ARG;
  if (a.rot > a.D || (!norm && a.rot == 0)) return GLA_ERR_INVALID_ARG;
  if ((a.interleaved != 0 && a.interleaved != 1) || (a.inverse != 0 && a.inverse != 1)) return GLA_ERR_INVALID_ARG;
  if (!std::isfinite(a.scale)) return GLA_ERR_INVALID_ARG;
  if (norm && (!(a.eps >= 0.f) || std::isinf(a.eps))) return GLA_ERR_INVALID_ARG;
  if (a.D % 8 || a.rot % 8 || a.D > 256) return GLA_ERR_UNSUPPORTED;
  if (a.q.H > 4096 || a.k.H > 4096 || a.rows > ((int64_t)1 << 31) / (a.q.H + a.k.H)) return GLA_ERR_UNSUPPORTED;
  if (a.rot > 0 && !a.inv_freq) return GLA_ERR_INVALID_ARG;
  if (!a.positions && a.period <= 0) return GLA_ERR_INVALID_ARG;
  if (!aligned16(a.inv_freq) || (reinterpret_cast<uintptr_t>(a.positions) & (a.positions64 ? 7u : 3u)))
    return GLA_ERR_ALIGNMENT;
  const int64_t elt = dtype == GLA_BF16 ? 2 : 4;
  const dig::HeadRows* t[2] = {&a.q, &a.k};
  Rows in[4], grad[4], out[2], dw[2];
  for (int i = 0; i < 2; ++i) {
    const dig::HeadRows& h = *t[i];
    if (h.H == 0) {
      in[i] = grad[i] = out[i] = dw[i] = Rows{nullptr, 0, 0, 0};
      continue;
    }
    if (!h.in || !h.out || (norm && !h.weight) || (bwd && (!h.grad || !h.dweight))) return GLA_ERR_INVALID_ARG;
    const int64_t w = (int64_t)h.H * a.D;
    for (int64_t s : {h.stride, h.out_stride, bwd ? h.grad_stride : w}) {
      if (s < w) return GLA_ERR_INVALID_ARG;
      if (s > (int64_t)1 << 32 || a.rows > ((int64_t)1 << 42) / s) return GLA_ERR_UNSUPPORTED;
      if (s * elt % 16) return GLA_ERR_ALIGNMENT;
    }
    if (!aligned16(h.in) || !aligned16(h.out) || !aligned16(h.grad) || !aligned16(h.weight) || !aligned16(h.dweight))
      return GLA_ERR_ALIGNMENT;
    in[i] = head_rows(h.in, h.stride, h.H, a.D, a.rows, elt);
    grad[i] = bwd ? head_rows(h.grad, h.grad_stride, h.H, a.D, a.rows, elt) : Rows{nullptr, 0, 0, 0};
    out[i] = head_rows(h.out, h.out_stride, h.H, a.D, a.rows, elt);
    dw[i] = dense(bwd ? h.dweight : nullptr, (int64_t)a.D * 4);
  }
  const Rows small[] = {dense(a.inv_freq, (int64_t)a.rot * 2), dense(a.positions, a.rows * (a.positions64 ? 8 : 4)),
                        dense(norm ? a.q.weight : nullptr, (int64_t)a.D * 4),
                        dense(norm && a.k.H ? a.k.weight : nullptr, (int64_t)a.D * 4)};
  if (clash(out[0], out[1]) || clash(dw[0], dw[1])) return GLA_ERR_INVALID_ARG;
  for (int o = 0; o < 2; ++o) {
    for (int i = 0; i < 2; ++i) {
      // In place: the outputs over the inputs, or the input gradients over the output gradients.
      const bool own = o == i;
      if (clash(out[o], in[i]) && !(own && !bwd && same(out[o], in[i]))) return GLA_ERR_INVALID_ARG;
      if (clash(out[o], grad[i]) && !(own && same(out[o], grad[i]))) return GLA_ERR_INVALID_ARG;
      if (clash(out[o], dw[i]) || clash(dw[o], in[i]) || clash(dw[o], grad[i])) return GLA_ERR_INVALID_ARG;
    }
    for (const Rows& s : small)
      if (clash(out[o], s) || clash(dw[o], s)) return GLA_ERR_INVALID_ARG;
  }
  return GLA_OK;
}

dig::QkRopeArgs qk_args(const void* positions, int positions64, int period, const float* inv_freq, int64_t rows, int D,
                        int rot, int interleaved, float scale, int dtype) {
  dig::QkRopeArgs a{};
  a.positions = positions;
  a.positions64 = positions64;
  a.period = period;
  a.inv_freq = inv_freq;
  a.rows = rows;
  a.D = D;
  a.rot = rot;
  a.interleaved = interleaved;
  a.scale = scale;
  a.bf16 = dtype == GLA_BF16;
  return a;
}

struct QkBwdCall {
  dig::QkRopeArgs a;
  cudaStream_t st;
};
cudaError_t run_qk_bwd(void* ws, void* ctx) {
  const QkBwdCall* c = static_cast<const QkBwdCall*>(ctx);
  return dig::qk_norm_rope_bwd_launch(c->a, ws, c->st);
}

}  // namespace

extern "C" {

int glr_fwd(const void* x, const void* gate, const float* h0, int B, int Hgrid, int Wgrid, int C, int64_t x_stride,
            int64_t gate_stride, int dir, float gate_norm, int complement, int dtype, void* out, float* h_last,
            cudaStream_t stream) {
  int64_t rows = 0;
  const int rc = grid_shape(B, Hgrid, Wgrid, &rows);
  if (rc != GLA_OK) return rc;
  dig::GlrArgs a = glr_args(x, gate, x_stride, gate_stride, h0, C, dir, gate_norm, complement, dtype);
  on_grid(&a, B, Hgrid, Wgrid);
  a.out = out;
  a.h_last = h_last;
  return run_glr(a, rows, dtype, false, stream);
}

int glr_fwd_packed(const void* x, const void* gate, const int* cu_seqlens, const float* h0, int64_t rows, int nseq, int C,
                   int64_t x_stride, int64_t gate_stride, int dir, float gate_norm, int complement, int dtype,
                   int fill, void* out, float* h_last, cudaStream_t stream) {
  if (!cu_seqlens) return GLA_ERR_INVALID_ARG;
  if (rows > (int64_t)1 << 30) return GLA_ERR_UNSUPPORTED;
  dig::GlrArgs a = glr_args(x, gate, x_stride, gate_stride, h0, C, dir, gate_norm, complement, dtype);
  on_packed(&a, cu_seqlens, nseq, (int)rows, fill);
  a.out = out;
  a.h_last = h_last;
  return run_glr(a, rows, dtype, false, stream);
}

int glr_bwd(const void* x, const void* gate, const void* h, const void* dout, const float* h0, const float* dh_last,
            int B, int Hgrid, int Wgrid, int C, int64_t x_stride, int64_t gate_stride, int dir, float gate_norm,
            int complement, int dtype, void* dx, void* dgate, float* dh0, cudaStream_t stream) {
  int64_t rows = 0;
  const int rc = grid_shape(B, Hgrid, Wgrid, &rows);
  if (rc != GLA_OK) return rc;
  dig::GlrArgs a = glr_args(x, gate, x_stride, gate_stride, h0, C, dir, gate_norm, complement, dtype);
  on_grid(&a, B, Hgrid, Wgrid);
  a.h = h;
  a.dout = dout;
  a.dh_last = dh_last;
  a.dx = dx;
  a.dgate = dgate;
  a.dh0 = dh0;
  return run_glr(a, rows, dtype, true, stream);
}

int glr_bwd_packed(const void* x, const void* gate, const void* h, const void* dout, const int* cu_seqlens,
                   const float* h0, const float* dh_last, int64_t rows, int nseq, int C, int64_t x_stride,
                   int64_t gate_stride, int dir, float gate_norm, int complement, int dtype, int fill, void* dx,
                   void* dgate, float* dh0, cudaStream_t stream) {
  if (!cu_seqlens) return GLA_ERR_INVALID_ARG;
  if (rows > (int64_t)1 << 30) return GLA_ERR_UNSUPPORTED;
  dig::GlrArgs a = glr_args(x, gate, x_stride, gate_stride, h0, C, dir, gate_norm, complement, dtype);
  on_packed(&a, cu_seqlens, nseq, (int)rows, fill);
  a.h = h;
  a.dout = dout;
  a.dh_last = dh_last;
  a.dx = dx;
  a.dgate = dgate;
  a.dh0 = dh0;
  return run_glr(a, rows, dtype, true, stream);
}

int glr_step(const void* x, const void* gate, const float* state, const int* slots, int N, int nslots, int C,
             int64_t x_stride, int64_t gate_stride, float gate_norm, int complement, int dtype, int fill,
             float* state_out, void* out, cudaStream_t stream) {
  int rc = check_glr_shape(N, nslots, C, x_stride, gate_stride, gate_norm, complement, dtype);
  if (rc != GLA_OK) return rc;
  if (!x || !gate || !state || !state_out || !out || (fill != 0 && fill != 1)) return GLA_ERR_INVALID_ARG;
  if (N > 65535) return GLA_ERR_UNSUPPORTED;
  if (!slots && N > nslots) return GLA_ERR_INVALID_ARG;
  for (const void* p : {x, gate, (const void*)state, (const void*)state_out, (const void*)out})
    if (!aligned16(p)) return GLA_ERR_ALIGNMENT;
  if (reinterpret_cast<uintptr_t>(slots) & 3u) return GLA_ERR_ALIGNMENT;
  const int64_t elt = dtype == GLA_BF16 ? 2 : 4, gelt = gate_norm == 0.f ? 4 : elt;
  const Rows xs{x, x_stride * elt, C * elt, N}, gs{gate, gate_stride * gelt, C * gelt, N};
  const Rows st = dense(state, (int64_t)nslots * C * 4), so = dense(state_out, (int64_t)nslots * C * 4);
  const Rows ix = dense(slots, (int64_t)N * 4), o = dense(out, (int64_t)N * C * elt);
  for (const Rows& i : {xs, gs, ix, st, so})
    if (clash(o, i)) return GLA_ERR_INVALID_ARG;
  for (const Rows& i : {xs, gs, ix})
    if (clash(so, i)) return GLA_ERR_INVALID_ARG;
  if (clash(so, st) && state != state_out) return GLA_ERR_INVALID_ARG;  // in place, or apart
  if ((rc = dig::check_device()) != GLA_OK) return rc;
  const dig::GlrStepArgs a{x, gate, x_stride, gate_stride, state, state_out, slots, N, nslots, C, gate_norm,
                           complement, dtype == GLA_BF16, fill, out};
  return dig::glr_step_launch(a, stream) == cudaSuccess ? GLA_OK : GLA_ERR_CUDA;
}

int rope(const void* q, const void* k, const void* positions, int positions64, int period, const float* inv_freq,
         int64_t rows, int Hq, int Hk, int D, int rot, int64_t q_stride, int64_t k_stride, int interleaved, int inverse,
         float scale, int dtype, void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
         cudaStream_t stream) {
  dig::QkRopeArgs a = qk_args(positions, positions64, period, inv_freq, rows, D, rot, interleaved, scale, dtype);
  a.inverse = inverse;
  a.q = dig::HeadRows{q, nullptr, q_out, q_stride, 0, q_out_stride, nullptr, nullptr, Hq};
  a.k = dig::HeadRows{k, nullptr, k_out, k_stride, 0, k_out_stride, nullptr, nullptr, Hk};
  int rc = check_qk(a, dtype, false, false);
  if (rc != GLA_OK) return rc;
  if ((rc = dig::check_device()) != GLA_OK) return rc;
  return dig::qk_rope_launch(a, stream) == cudaSuccess ? GLA_OK : GLA_ERR_CUDA;
}

int qk_norm_rope(const void* q, const void* k, const float* q_weight, const float* k_weight, const void* positions,
                 int positions64, int period, const float* inv_freq, int64_t rows, int Hq, int Hk, int D, int rot,
                 int64_t q_stride, int64_t k_stride, int interleaved, float eps, float scale, int dtype, void* q_out,
                 int64_t q_out_stride, void* k_out, int64_t k_out_stride, cudaStream_t stream) {
  dig::QkRopeArgs a = qk_args(positions, positions64, period, inv_freq, rows, D, rot, interleaved, scale, dtype);
  a.eps = eps;
  a.q = dig::HeadRows{q, nullptr, q_out, q_stride, 0, q_out_stride, q_weight, nullptr, Hq};
  a.k = dig::HeadRows{k, nullptr, k_out, k_stride, 0, k_out_stride, k_weight, nullptr, Hk};
  int rc = check_qk(a, dtype, true, false);
  if (rc != GLA_OK) return rc;
  if ((rc = dig::check_device()) != GLA_OK) return rc;
  return dig::qk_rope_launch(a, stream) == cudaSuccess ? GLA_OK : GLA_ERR_CUDA;
}

int qk_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* q, const void* k, const float* q_weight,
                     const float* k_weight, const void* positions, int positions64, int period, const float* inv_freq,
                     int64_t rows, int Hq, int Hk, int D, int rot, int64_t dq_out_stride, int64_t dk_out_stride,
                     int64_t q_stride, int64_t k_stride, int interleaved, float eps, float scale, int dtype, void* dq,
                     int64_t dq_stride, void* dk, int64_t dk_stride, float* dq_weight, float* dk_weight,
                     cudaStream_t stream) {
  QkBwdCall c{qk_args(positions, positions64, period, inv_freq, rows, D, rot, interleaved, scale, dtype), stream};
  c.a.eps = eps;
  c.a.q = dig::HeadRows{q, dq_out, dq, q_stride, dq_out_stride, dq_stride, q_weight, dq_weight, Hq};
  c.a.k = dig::HeadRows{k, dk_out, dk, k_stride, dk_out_stride, dk_stride, k_weight, dk_weight, Hk};
  int rc = check_qk(c.a, dtype, true, true);
  if (rc != GLA_OK) return rc;
  if ((rc = dig::check_device()) != GLA_OK) return rc;
  return dig::run_with_workspace(dig::qk_norm_rope_bwd_workspace_bytes(c.a), stream, run_qk_bwd, &c);
}

}  // extern "C"
