// qk_rope.cu -- rotary positions of query and key heads, alone or behind an RMS norm of
// every head, and the gradients (include/dig_gla.h, rope, qk_norm_rope, qk_norm_rope_bwd).
//
// Mathematics: y = scale R(position * inv_freq) (x r w), r = 1 / sqrt(mean(x^2) + eps); the
// gradient turns back first, g = scale R^T dy, and with n = x r:
// dx = r (w g - n mean(w g n)), dw = sum of g n.
//
// Bound: memory.  Every head is read and written once (the gradient: two reads, one write).
//
// Split.  Eight channels that rotate among themselves are a unit: quads i and i + rot / 8
// of the head when pairs are half a span apart, two adjacent quads when they are interleaved
// or not rotated.  A group of lanes (a power of two, kUnits units each) holds a head in
// registers and sums its squares by shuffles; a warp takes the heads of one token, group by
// group, kHeads of them in flight.  The warp computes the token's angles once, one pair a
// lane, and keeps cos and sin in shared memory.  A head of n units takes the next power
// of two of lanes, or a quarter of that with three units a lane where n fits in three
// quarters of it (72 channels: 9 units on 4 x 3 instead of 16 lanes).  With few tokens a
// token's heads are shared between warps.
#include <math.h>

#include <algorithm>

#include "four.cuh"
#include "internal.h"

namespace dig {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxPairs = 128;

// ---- angles -----------------------------------------------------------------------------

struct Turn {
  F4 c, s;
};

// cos and sin of position * inv_freq, times scale.  The angle is formed in fp64, in turns,
// and reduced there to half a turn, so far positions keep their phase.
__device__ __forceinline__ void angles(const QkRopeArgs& a, int64_t row, float2* cs) {
  double pos;
  if (!a.positions)
    pos = (double)(row % a.period);
  else
    pos = a.positions64 ? (double)static_cast<const long long*>(a.positions)[row]
                        : (double)static_cast<const int*>(a.positions)[row];
  for (int p = threadIdx.x & 31; p < a.rot / 2; p += 32) {
    double turn = pos * ((double)a.inv_freq[p] * 0.15915494309189535);
    turn -= rint(turn);
    float s, c;
    sincospif(2.f * (float)turn, &s, &c);
    cs[p] = make_float2(c * a.scale, (a.inverse ? -s : s) * a.scale);
  }
}

// Four consecutive pairs' cos and sin.
__device__ __forceinline__ Turn turn_of(const float2* cs) {
  const float4 p = reinterpret_cast<const float4*>(cs)[0], q = reinterpret_cast<const float4*>(cs)[1];
  return Turn{F4{make_float2(p.x, p.z), make_float2(q.x, q.z)}, F4{make_float2(p.y, p.w), make_float2(q.y, q.w)}};
}

// ---- units ------------------------------------------------------------------------------

// Where a lane's unit lies in a head: channels a .. a + 3 and b .. b + 3.  A lane behind the
// last unit reads the last one and keeps nothing (on = false).
struct Unit {
  int a, b;
  bool on, turned;
};
template <bool kInter>
__device__ __forceinline__ Unit unit(const QkRopeArgs& q, int i) {
  Unit u;
  u.on = i < q.D / 8;
  i = min(i, q.D / 8 - 1);
  u.turned = i < q.rot / 8;
  const bool halves = !kInter && u.turned;
  u.a = halves ? 4 * i : kInter ? 8 * i : q.rot + 8 * (i - q.rot / 8);
  u.b = halves ? 4 * i + q.rot / 2 : u.a + 4;
  return u;
}

// The unit's channels as pairs: X holds the first of each, Y the second.
struct Pairs {
  F4 x, y;
};
template <bool kInter>
__device__ __forceinline__ Pairs as_pairs(F4 a, F4 b) {
  if constexpr (!kInter) return Pairs{a, b};
  return Pairs{F4{make_float2(a.a.x, a.b.x), make_float2(b.a.x, b.b.x)}, F4{make_float2(a.a.y, a.b.y), make_float2(b.a.y, b.b.y)}};
}
template <bool kInter>
__device__ __forceinline__ void as_quads(const Pairs& p, F4& a, F4& b) {
  if constexpr (kInter) {
    a = F4{make_float2(p.x.a.x, p.y.a.x), make_float2(p.x.a.y, p.y.a.y)};
    b = F4{make_float2(p.x.b.x, p.y.b.x), make_float2(p.x.b.y, p.y.b.y)};
  } else {
    a = p.x;
    b = p.y;
  }
}
// (x, y) -> (x xc - y ys, y yc + x xs): a turn whose factors may hold weights.
struct Mix {
  F4 xc, xs, yc, ys;
};
__device__ __forceinline__ F4 minus(F4 v) { return F4{make_float2(-v.a.x, -v.a.y), make_float2(-v.b.x, -v.b.y)}; }
__device__ __forceinline__ Pairs mix(const Pairs& p, const Mix& t) {
  return Pairs{fma4(p.y, t.ys, mul4(p.x, t.xc)), fma4(p.x, t.xs, mul4(p.y, t.yc))};
}
__device__ __forceinline__ Pairs times(const Pairs& p, const Pairs& q) { return Pairs{mul4(p.x, q.x), mul4(p.y, q.y)}; }
__device__ __forceinline__ Pairs scaled(const Pairs& p, float f) { return Pairs{mul4(p.x, all4(f)), mul4(p.y, all4(f))}; }
__device__ __forceinline__ F4 dot4(const Pairs& p, const Pairs& q, F4 sum) { return fma4(p.y, q.y, fma4(p.x, q.x, sum)); }
__device__ __forceinline__ float sum4(F4 v) {
  const float2 s = __fadd2_rn(v.a, v.b);
  return s.x + s.y;
}
__device__ __forceinline__ float group_sum(float v, int lanes) {
  for (int o = lanes >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// How a warp's lanes and the launch's warps share the work.
struct Split {
  int lanes;       // lanes a head takes
  int q_steps, k_steps;  // passes of a warp's groups over a token's heads
  int parts;       // warps that share a token
  int64_t items;   // rows * parts
};

// The heads of a warp's share of a token: steps [from, to) of q (which = 0) and k (1).
__device__ __forceinline__ void share(const Split& w, int part, int which, int& from, int& to) {
  const int steps = w.q_steps + w.k_steps;
  const int first = w.parts == 1 ? 0 : (int)((int64_t)steps * part / w.parts);
  const int last = w.parts == 1 ? steps : (int)((int64_t)steps * (part + 1) / w.parts);
  from = which ? max(first - w.q_steps, 0) : first;
  to = which ? last - w.q_steps : min(last, w.q_steps);
}

// ---- forward ------------------------------------------------------------------------------
template <typename T, bool kNorm, bool kInter, int kUnits, int kHeads>
__global__ void __launch_bounds__(kThreads, kUnits == 1 ? 6 : 4) qk_rope_k(QkRopeArgs a, Split w) {
  using Raw = typename Four<T>::Raw;
  __shared__ __align__(16) float2 cs[kWarps][kMaxPairs];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t item = (int64_t)blockIdx.x * kWarps + warp;
  if (item >= w.items) return;
  const int64_t row = w.parts == 1 ? item : item / w.parts;
  const int part = (int)(item - row * w.parts);
  const int group = lane / w.lanes, groups = 32 / w.lanes, within = lane & (w.lanes - 1);
  Unit at[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) at[u] = unit<kInter>(a, u * w.lanes + within);
  angles(a, row, cs[warp]);
  __syncwarp();
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const HeadRows& t = which ? a.k : a.q;
    int from, to;
    share(w, part, which, from, to);
    if (from >= to) continue;
    const T* in = static_cast<const T*>(t.in) + row * t.stride;
    T* out = static_cast<T*>(t.out) + row * t.out_stride;
    Mix turn[kUnits];  // xc and yc are the weights alone where nothing turns
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      if (at[u].turned) {
        const Turn f = turn_of(cs[warp] + 4 * min(u * w.lanes + within, a.D / 8 - 1));
        turn[u] = Mix{f.c, f.s, f.c, minus(f.s)};
      } else {
        turn[u] = Mix{all4(1.f), all4(0.f), all4(1.f), all4(0.f)};
      }
      if constexpr (kNorm) {
        const Pairs g = as_pairs<kInter>(load4(t.weight + at[u].a), load4(t.weight + at[u].b));
        turn[u] = Mix{mul4(turn[u].xc, g.x), mul4(turn[u].xs, g.x), mul4(turn[u].yc, g.y), mul4(turn[u].ys, g.y)};
      }
    }
#pragma unroll 1
    for (int step = from; step < to; step += kHeads) {
      Raw ra[kHeads][kUnits], rb[kHeads][kUnits];
#pragma unroll
      for (int k = 0; k < kHeads; ++k) {
        const int head = min((step + k) * groups + group, t.H - 1);
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
          ra[k][u] = *reinterpret_cast<const Raw*>(in + at[u].a + (int64_t)head * a.D);
          rb[k][u] = *reinterpret_cast<const Raw*>(in + at[u].b + (int64_t)head * a.D);
        }
      }
      float r[kHeads];
      if constexpr (kNorm) {
        float ss[kHeads];
#pragma unroll
        for (int k = 0; k < kHeads; ++k) {
          ss[k] = 0.f;
#pragma unroll
          for (int u = 0; u < kUnits; ++u) {
            const F4 x = Four<T>::get(ra[k][u]), y = Four<T>::get(rb[k][u]);
            const float v = sum4(fma4(y, y, mul4(x, x)));
            ss[k] += at[u].on ? v : 0.f;
          }
        }
        for (int o = w.lanes >> 1; o; o >>= 1)
#pragma unroll
          for (int k = 0; k < kHeads; ++k) ss[k] += __shfl_xor_sync(0xffffffffu, ss[k], o);
#pragma unroll
        for (int k = 0; k < kHeads; ++k) r[k] = rsqrtf(ss[k] / a.D + a.eps);
      }
#pragma unroll
      for (int k = 0; k < kHeads; ++k) {
        const int head = (step + k) * groups + group;
        if (step + k >= to || head >= t.H) continue;
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
          if (!at[u].on) continue;
          T* const oa = out + at[u].a + (int64_t)head * a.D;
          T* const ob = out + at[u].b + (int64_t)head * a.D;
          if (!kNorm && !at[u].turned) {  // a copy
            *reinterpret_cast<Raw*>(oa) = ra[k][u];
            *reinterpret_cast<Raw*>(ob) = rb[k][u];
            continue;
          }
          Pairs p = as_pairs<kInter>(Four<T>::get(ra[k][u]), Four<T>::get(rb[k][u]));
          if constexpr (kNorm) p = scaled(p, r[k]);
          p = at[u].turned ? mix(p, turn[u]) : Pairs{mul4(p.x, turn[u].xc), mul4(p.y, turn[u].yc)};
          F4 x, y;
          as_quads<kInter>(p, x, y);
          store4(oa, x);
          store4(ob, y);
        }
      }
    }
  }
}

// ---- gradients ------------------------------------------------------------------------------
// Warps walk the items with a stride and keep the weight gradients of their lanes' channels;
// a block adds its groups and warps in a fixed order and writes one row for q and one for k.
template <typename T, bool kInter, int kUnits>
__global__ void __launch_bounds__(kThreads, kUnits == 1 ? 5 : 3) qk_norm_rope_bwd_k(QkRopeArgs a, Split w, float* part_sums) {
  using Raw = typename Four<T>::Raw;
  __shared__ __align__(16) float2 cs[kWarps][kMaxPairs];
  __shared__ __align__(16) float sums[kWarps][2][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = lane / w.lanes, groups = 32 / w.lanes, within = lane & (w.lanes - 1);
  const float inv_d = 1.f / a.D;
  Unit at[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) at[u] = unit<kInter>(a, u * w.lanes + within);
  Pairs dw[2][kUnits];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int u = 0; u < kUnits; ++u) dw[i][u] = Pairs{all4(0.f), all4(0.f)};
  for (int64_t item = (int64_t)blockIdx.x * kWarps + warp; item < w.items; item += (int64_t)gridDim.x * kWarps) {
    const int64_t row = w.parts == 1 ? item : item / w.parts;
    const int part = (int)(item - row * w.parts);
    __syncwarp();  // the angles of the item before have been read
    angles(a, row, cs[warp]);
    __syncwarp();
    Mix back[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
      if (at[u].turned) {
        const Turn f = turn_of(cs[warp] + 4 * min(u * w.lanes + within, a.D / 8 - 1));
        back[u] = Mix{f.c, minus(f.s), f.c, f.s};
      }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const HeadRows& t = which ? a.k : a.q;
      int from, to;
      share(w, part, which, from, to);
      if (from >= to) continue;
      const T* in = static_cast<const T*>(t.in) + row * t.stride;
      const T* grad = static_cast<const T*>(t.grad) + row * t.grad_stride;
      T* out = static_cast<T*>(t.out) + row * t.out_stride;
#pragma unroll 1
      for (int step = from; step < to; ++step) {
        const int head = step * groups + group;
        const int64_t off = (int64_t)min(head, t.H - 1) * a.D;
        Raw xa[kUnits], xb[kUnits], ga[kUnits], gb[kUnits];
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
          xa[u] = *reinterpret_cast<const Raw*>(in + at[u].a + off);
          xb[u] = *reinterpret_cast<const Raw*>(in + at[u].b + off);
          ga[u] = *reinterpret_cast<const Raw*>(grad + at[u].a + off);
          gb[u] = *reinterpret_cast<const Raw*>(grad + at[u].b + off);
        }
        float ss = 0.f, dot = 0.f;
        Pairs g[kUnits], wg[kUnits];
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
          const Pairs x = as_pairs<kInter>(Four<T>::get(xa[u]), Four<T>::get(xb[u]));
          g[u] = as_pairs<kInter>(Four<T>::get(ga[u]), Four<T>::get(gb[u]));
          if (at[u].turned) g[u] = mix(g[u], back[u]);
          wg[u] = times(g[u], as_pairs<kInter>(load4(t.weight + at[u].a), load4(t.weight + at[u].b)));
          const float s = sum4(fma4(x.y, x.y, mul4(x.x, x.x))), d = sum4(fma4(x.y, wg[u].y, mul4(x.x, wg[u].x)));
          ss += at[u].on ? s : 0.f;
          dot += at[u].on ? d : 0.f;
        }
        for (int o = w.lanes >> 1; o; o >>= 1) {
          ss += __shfl_xor_sync(0xffffffffu, ss, o);
          dot += __shfl_xor_sync(0xffffffffu, dot, o);
        }
        const float r = rsqrtf(ss * inv_d + a.eps);
        const float m = dot * r * inv_d;
        if (head >= t.H) continue;
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
          if (!at[u].on) continue;
          const Pairs n = scaled(as_pairs<kInter>(Four<T>::get(xa[u]), Four<T>::get(xb[u])), r);
          dw[which][u] = Pairs{fma4(g[u].x, n.x, dw[which][u].x), fma4(g[u].y, n.y, dw[which][u].y)};
          Pairs d{fma4(n.x, all4(-m), wg[u].x), fma4(n.y, all4(-m), wg[u].y)};
          d = scaled(d, r);
          F4 p, q;
          as_quads<kInter>(d, p, q);
          store4(out + at[u].a + off, p);
          store4(out + at[u].b + off, q);
        }
      }
    }
  }
  // Groups of a warp (the same channels in lanes w.lanes apart), then warps.
#pragma unroll
  for (int which = 0; which < 2; ++which) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      F4 p, q;
      as_quads<kInter>(dw[which][u], p, q);
      float v[8] = {p.a.x, p.a.y, p.b.x, p.b.y, q.a.x, q.a.y, q.b.x, q.b.y};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        for (int o = w.lanes; o < 32; o <<= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
      if (group == 0 && at[u].on) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sums[warp][which][at[u].a + i] = v[i];
          sums[warp][which][at[u].b + i] = v[4 + i];
        }
      }
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * a.D; c += kThreads) {
    const int which = c >= a.D, ch = c - which * a.D;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) s += sums[i][which][ch];
    part_sums[((int64_t)which * gridDim.x + blockIdx.x) * a.D + ch] = s;
  }
}

// The blocks' rows: 32 lanes of rows by 8 channels a block, then a tree over the lanes.
__global__ void __launch_bounds__(256) qk_weight_grad_k(QkRopeArgs a, const float* part, int blocks) {
  const int which = blockIdx.y, ch = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const float* p = part + (int64_t)which * blocks * a.D + ch;
  float s = 0.f;
  for (int b = lane; b < blocks; b += 32) s += p[(int64_t)b * a.D];
  s = group_sum(s, 32);
  if (lane == 0) (which ? a.k.dweight : a.q.dweight)[ch] = s;
}

// ---- launch -----------------------------------------------------------------------------------

int units_of(const QkRopeArgs& a) {  // units a lane takes: 1 or 3
  const int n = a.D / 8;
  int p = 1;
  while (p < n) p *= 2;
  return p >= 4 && n <= p / 4 * 3 ? 3 : 1;
}
Split split(const QkRopeArgs& a, int units, int64_t warps) {
  const int n = a.D / 8;
  Split w;
  w.lanes = 1;
  while (w.lanes * units < n) w.lanes *= 2;
  const int groups = 32 / w.lanes;
  w.q_steps = (a.q.H + groups - 1) / groups;
  w.k_steps = (a.k.H + groups - 1) / groups;
  // Tokens are shared between warps until `warps` of them have work.
  w.parts = (int)std::max<int64_t>(1, std::min<int64_t>(w.q_steps + w.k_steps, warps / a.rows));
  w.items = a.rows * w.parts;
  return w;
}

template <typename T, bool kNorm, bool kInter, int kUnits>
cudaError_t forward(const QkRopeArgs& a, cudaStream_t s) {
  constexpr int kHeads = kUnits == 1 ? 4 : 2;
  const Split w = split(a, kUnits, 148 * 16);
  qk_rope_k<T, kNorm, kInter, kUnits, kHeads><<<(unsigned)((w.items + kWarps - 1) / kWarps), kThreads, 0, s>>>(a, w);
  return cudaGetLastError();
}
template <typename T, bool kNorm>
cudaError_t forward_by(const QkRopeArgs& a, cudaStream_t s) {
  if (units_of(a) == 1) return a.interleaved ? forward<T, kNorm, true, 1>(a, s) : forward<T, kNorm, false, 1>(a, s);
  return a.interleaved ? forward<T, kNorm, true, 3>(a, s) : forward<T, kNorm, false, 3>(a, s);
}

constexpr int kBwdBlocks = 148 * 6;
int bwd_blocks(const Split& w) { return (int)std::min<int64_t>(kBwdBlocks, (w.items + kWarps - 1) / kWarps); }

template <typename T, bool kInter, int kUnits>
cudaError_t backward(const QkRopeArgs& a, float* part, cudaStream_t s) {
  const Split w = split(a, kUnits, 148 * 16);
  const int blocks = bwd_blocks(w);
  qk_norm_rope_bwd_k<T, kInter, kUnits><<<blocks, kThreads, 0, s>>>(a, w, part);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  qk_weight_grad_k<<<dim3(a.D / 8, a.k.H ? 2 : 1), 256, 0, s>>>(a, part, blocks);
  return cudaGetLastError();
}
template <typename T>
cudaError_t backward_by(const QkRopeArgs& a, float* part, cudaStream_t s) {
  if (units_of(a) == 1) return a.interleaved ? backward<T, true, 1>(a, part, s) : backward<T, false, 1>(a, part, s);
  return a.interleaved ? backward<T, true, 3>(a, part, s) : backward<T, false, 3>(a, part, s);
}

}  // namespace

cudaError_t qk_rope_launch(const QkRopeArgs& a, cudaStream_t s) {
  if (a.q.weight) return a.bf16 ? forward_by<__nv_bfloat16, true>(a, s) : forward_by<float, true>(a, s);
  return a.bf16 ? forward_by<__nv_bfloat16, false>(a, s) : forward_by<float, false>(a, s);
}

size_t qk_norm_rope_bwd_workspace_bytes(const QkRopeArgs& a) {
  return (size_t)bwd_blocks(split(a, units_of(a), 148 * 16)) * 2 * a.D * sizeof(float);
}

cudaError_t qk_norm_rope_bwd_launch(const QkRopeArgs& a, void* workspace, cudaStream_t s) {
  float* part = static_cast<float*>(workspace);
  return a.bf16 ? backward_by<__nv_bfloat16>(a, part, s) : backward_by<float>(a, part, s);
}

}  // namespace dig
