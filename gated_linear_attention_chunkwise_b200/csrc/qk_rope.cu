// qk_rope.cu -- rotary positions of query and key heads, alone or behind an RMS norm of
// every head, and the gradients (include/dig_gla.h, rope, qk_norm_rope, qk_norm_rope_bwd).
//
// Mathematics: y = scale R(position * inv_freq) (x r w), r = 1 / sqrt(mean(x^2) + eps); the
// gradient turns back first, g = scale R^T dy, and with n = x r:
// dx = r (w g - n mean(w g n)), dw = sum of g n.
//
// Bound: memory; every head is read and written once (the gradient: two reads, one write).
// Measured, of the copy bandwidth: rotation of bf16 heads 88 % (16381 tokens of 40 heads of
// 128: 58 us), with the norm 71 % (72 us), of fp32 heads 77 % (8191 tokens of 32 heads of 80:
// 33 us) and 86 %.  What keeps the norm from more is instruction issue (63 % of the cycles:
// unpacking, two passes over a head's channels around the sum, the packing).  The gradient
// reaches 42 % with 72 channels and 60 % with 128 (25088 tokens of 32 heads of 72: 125 us):
// twice the work of a head, 16 warps an SM, 27 of 32 lanes at 72 channels.
//
// Split.  Eight channels that rotate among themselves are a unit: quads i and i + rot / 8
// of the head when pairs are half a span apart, two adjacent quads when they are interleaved
// or not rotated.  D / 8 lanes hold a head in registers, a unit each, and sum its squares by
// shuffles; a warp holds as many heads at once as fit (72 channels: three heads on 27 lanes)
// and walks the heads of one token, four in flight (two: prompt 74 -> 82 us; six: 78).  It
// computes the token's angles once, one pair a lane, and keeps cos and sin in shared memory.
// With few tokens a token's heads are shared between warps.
#include <math.h>

#include <algorithm>
#include <type_traits>

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

__device__ __forceinline__ long long position(const QkRopeArgs& a, int64_t row) {
  if (!a.positions) return row % a.period;
  return a.positions64 ? static_cast<const long long*>(a.positions)[row] : static_cast<const int*>(a.positions)[row];
}

// cos and sin of position * inv_freq, times scale.  The angle is formed in fp64, in turns,
// and reduced there to half a turn, so far positions keep their phase; what fp32 drops of it
// (6e-8 in radians, all of a sine or cosine near its zero) enters by the first-order term.
__device__ __forceinline__ void angles(const QkRopeArgs& a, long long position, float2* cs) {
  const double pos = (double)position;
  for (int p = threadIdx.x & 31; p < a.rot / 2; p += 32) {
    double turn = pos * ((double)a.inv_freq[p] * 0.15915494309189535);
    turn -= rint(turn);
    float s, c;
    const float most = (float)turn, rest = (float)(turn - (double)most) * 6.283185307179586f;
    sincospif(2.f * most, &s, &c);
    const float cos = fmaf(-s, rest, c), sin = fmaf(c, rest, s);
    cs[p] = make_float2(cos * a.scale, (a.inverse ? -sin : sin) * a.scale);
  }
}

// Four consecutive pairs' cos and sin.
__device__ __forceinline__ Turn turn_of(const float2* cs) {
  const float4 p = reinterpret_cast<const float4*>(cs)[0], q = reinterpret_cast<const float4*>(cs)[1];
  return Turn{F4{make_float2(p.x, p.z), make_float2(q.x, q.z)}, F4{make_float2(p.y, p.w), make_float2(q.y, q.w)}};
}

// ---- units ------------------------------------------------------------------------------

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
__device__ __forceinline__ float sum4(F4 v) {
  const float2 s = __fadd2_rn(v.a, v.b);
  return s.x + s.y;
}
// Sums over a head's lanes, any number of them, in all of them.
struct Group {
  int lanes, within, first;  // lanes of a head; this lane among them; the head's first lane
  int top;                   // the largest power of two below `lanes`
  bool even;                 // lanes is a power of two
};
template <int n>
__device__ __forceinline__ void group_sum(float (&v)[n], const Group& g) {
  if (g.even) {
    for (int o = g.top; o; o >>= 1)
#pragma unroll
      for (int k = 0; k < n; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  } else {
    for (int o = g.top; o; o >>= 1) {
      const bool takes = g.within < o && g.within + o < g.lanes;
#pragma unroll
      for (int k = 0; k < n; ++k) {
        const float t = __shfl_down_sync(0xffffffffu, v[k], o);
        v[k] += takes ? t : 0.f;
      }
    }
#pragma unroll
    for (int k = 0; k < n; ++k) v[k] = __shfl_sync(0xffffffffu, v[k], g.first);
  }
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

// A lane's place: its head among the warp's, its unit of the head.  Lanes behind the last
// whole head read what the last head's lanes read and keep nothing.
template <bool kInter>
struct Lane {
  Group g;
  int group, groups;
  int a, b;  // the unit's channels a .. a + 3 and b .. b + 3
  int pair;  // its first pair
  bool on, turned;

  __device__ __forceinline__ Lane(const QkRopeArgs& q, int lanes) {
    const int lane = threadIdx.x & 31;
    groups = 32 / lanes;
    group = lane / lanes;
    on = group < groups;
    g.lanes = lanes;
    g.within = lane - group * lanes;
    g.first = group * lanes;
    group = min(group, groups - 1);
    g.even = (lanes & (lanes - 1)) == 0;
    g.top = lanes == 1 ? 0 : 1 << (31 - __clz(lanes - 1));
    const int i = g.within;  // < lanes = D / 8
    turned = i < q.rot / 8;
    const bool halves = !kInter && turned;
    a = halves ? 4 * i : kInter ? 8 * i : q.rot + 8 * (i - q.rot / 8);
    b = halves ? 4 * i + q.rot / 2 : a + 4;
    pair = 4 * i;
  }
};

// Keeps the compiler from holding a raw value's unpacked channels across the sums.
__device__ __forceinline__ uint2 again(uint2 v) {
  asm volatile("" : "+r"(v.x), "+r"(v.y));
  return v;
}
__device__ __forceinline__ float4 again(float4 v) { return v; }

// ---- forward ------------------------------------------------------------------------------
// A number of heads known at compile time, for the loops over the heads in flight.
template <int n>
using Count = std::integral_constant<int, n>;

// Blocks an SM that the registers allow without spilling much.
template <typename T>
constexpr int resident(bool norm) {
  return sizeof(T) == 2 ? 6 : norm ? 4 : 5;
}

template <typename T, bool kNorm, bool kInter>
__global__ void __launch_bounds__(kThreads, resident<T>(kNorm)) qk_rope_k(QkRopeArgs a, Split w) {
  using Raw = typename Four<T>::Raw;
  __shared__ __align__(16) float2 cs[kWarps][kMaxPairs];
  const int warp = threadIdx.x >> 5;
  const int64_t item = (int64_t)blockIdx.x * kWarps + warp;
  if (item >= w.items) return;
  const int64_t row = w.parts == 1 ? item : item / w.parts;
  const int part = (int)(item - row * w.parts);
  const long long pos = position(a, row);
  const Lane<kInter> at(a, w.lanes);
  const float inv_d = 1.f / a.D;
  const int to_b = at.b - at.a, next = at.groups * a.D;  // from quad to quad, from step to step
  Raw ra[4], rb[4];
  const T* in;
  T* out;
  int left, room;  // steps left; elements from this lane's head to the last one of the row
  auto start = [&](const HeadRows& t, int from, int to) {
    const int head = from * at.groups + at.group;
    const int64_t off = (int64_t)head * a.D + at.a;
    in = static_cast<const T*>(t.in) + row * t.stride + off;
    out = static_cast<T*>(t.out) + row * t.out_stride + off;
    left = to - from;
    room = (t.H - 1 - head) * a.D;
  };
  auto load = [&](auto n) {  // a lane behind the last head reads the last head
#pragma unroll
    for (int k = 0; k < n(); ++k) {
      const T* p = in + min(k * next, room);
      ra[k] = *reinterpret_cast<const Raw*>(p);
      rb[k] = *reinterpret_cast<const Raw*>(p + to_b);
    }
  };
  Mix turn;  // xc, yc: the weights alone where nothing turns
  auto finish = [&](auto n) {
    float r[n()];
    if constexpr (kNorm) {
#pragma unroll
      for (int k = 0; k < n(); ++k) {
        const F4 x = Four<T>::get(ra[k]), y = Four<T>::get(rb[k]);
        r[k] = sum4(fma4(y, y, mul4(x, x)));
        ra[k] = again(ra[k]);
        rb[k] = again(rb[k]);
      }
      group_sum(r, at.g);
#pragma unroll
      for (int k = 0; k < n(); ++k) r[k] = rsqrtf(fmaf(r[k], inv_d, a.eps));
    }
#pragma unroll
    for (int k = 0; k < n(); ++k) {
      if (!at.on || k * next > room) continue;
      T* const oa = out + k * next;
      if (!kNorm && !at.turned) {  // a copy
        *reinterpret_cast<Raw*>(oa) = ra[k];
        *reinterpret_cast<Raw*>(oa + to_b) = rb[k];
        continue;
      }
      Pairs p = as_pairs<kInter>(Four<T>::get(ra[k]), Four<T>::get(rb[k]));
      if constexpr (kNorm) p = scaled(p, r[k]);
      p = at.turned ? mix(p, turn) : Pairs{mul4(p.x, turn.xc), mul4(p.y, turn.yc)};
      F4 x, y;
      as_quads<kInter>(p, x, y);
      store4(oa, x);
      store4(oa + to_b, y);
    }
    in += n() * next;
    out += n() * next;
    room -= n() * next;
    left -= n();
  };
  int from, to;
  share(w, part, 0, from, to);
  int which = from < to ? 0 : 1;  // the share may lie in k alone
  if (which) share(w, part, 1, from, to);
  start(which ? a.k : a.q, from, to);
  // The first heads travel while the angles are computed.
  if (left >= 4)
    load(Count<4>());
  else
    load(Count<1>());
  angles(a, pos, cs[warp]);
  __syncwarp();
#pragma unroll 1
  for (bool first = true; which < 2; ++which, first = false) {
    const HeadRows& t = which ? a.k : a.q;
    if (!first) {
      share(w, part, which, from, to);
      if (from >= to) break;
      start(t, from, to);
      if (left >= 4)
        load(Count<4>());
      else
        load(Count<1>());
    }
    turn = Mix{all4(1.f), all4(0.f), all4(1.f), all4(0.f)};
    if (at.turned) {
      const Turn f = turn_of(cs[warp] + at.pair);
      turn = Mix{f.c, f.s, f.c, minus(f.s)};
    }
    if constexpr (kNorm) {
      const Pairs g = as_pairs<kInter>(load4(t.weight + at.a), load4(t.weight + at.b));
      turn = Mix{mul4(turn.xc, g.x), mul4(turn.xs, g.x), mul4(turn.yc, g.y), mul4(turn.ys, g.y)};
    }
    // Four heads a group at a time, then two, then one (which is loaded already where it is all).
    if (left >= 4) {
      finish(Count<4>());
      while (left >= 4) {
        load(Count<4>());
        finish(Count<4>());
      }
      if (left >= 2) {
        load(Count<2>());
        finish(Count<2>());
      }
      if (left) load(Count<1>());
    } else if (left >= 2) {
      load(Count<2>());
      finish(Count<2>());
      if (left) load(Count<1>());
    }
    if (left) finish(Count<1>());
  }
}

// ---- gradients ------------------------------------------------------------------------------
// Warps walk the items with a stride and keep the weight gradients of their lanes' channels;
// a block adds its heads and warps in a fixed order and writes a column for q and one for k.
template <typename T, bool kInter>
__global__ void __launch_bounds__(kThreads, 4) qk_norm_rope_bwd_k(QkRopeArgs a, Split w, float* part_sums) {
  using Raw = typename Four<T>::Raw;
  __shared__ __align__(16) float2 cs[kWarps][kMaxPairs];
  __shared__ __align__(16) float sums[kWarps][2][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float inv_d = 1.f / a.D;
  const Lane<kInter> at(a, w.lanes);
  Pairs dw[2] = {Pairs{all4(0.f), all4(0.f)}, Pairs{all4(0.f), all4(0.f)}};
  auto row_of = [&](int64_t item) { return w.parts == 1 ? item : item / w.parts; };
  const int64_t stride = (int64_t)gridDim.x * kWarps;
  const int to_b = at.b - at.a, next = at.groups * a.D;  // from quad to quad, from step to step
  int64_t item = (int64_t)blockIdx.x * kWarps + warp;
  long long pos = item < w.items ? position(a, row_of(item)) : 0;
  for (; item < w.items; item += stride) {
    const int64_t row = row_of(item);
    const int part = (int)(item - row * w.parts);
    __syncwarp();  // the angles of the item before have been read
    angles(a, pos, cs[warp]);
    if (item + stride < w.items) pos = position(a, row_of(item + stride));
    __syncwarp();
    Mix back{all4(1.f), all4(0.f), all4(1.f), all4(0.f)};
    if (at.turned) {
      const Turn f = turn_of(cs[warp] + at.pair);
      back = Mix{f.c, minus(f.s), f.c, f.s};
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const HeadRows& t = which ? a.k : a.q;
      int from, to;
      share(w, part, which, from, to);
      if (from >= to) continue;
      const Pairs weight = as_pairs<kInter>(load4(t.weight + at.a), load4(t.weight + at.b));
      const int first = from * at.groups + at.group;
      const int64_t off = (int64_t)first * a.D + at.a;
      const T* in = static_cast<const T*>(t.in) + row * t.stride + off;
      const T* grad = static_cast<const T*>(t.grad) + row * t.grad_stride + off;
      T* out = static_cast<T*>(t.out) + row * t.out_stride + off;
      int room = (t.H - 1 - first) * a.D;  // elements from this lane's head to the last one of the row
      auto heads = [&](auto n) {
        Raw xa[n()], xb[n()];
        Pairs turned[n()];
        float sd[2 * n()];
#pragma unroll
        for (int k = 0; k < n(); ++k) {  // a lane behind the last head reads the last head
          const int o = min(k * next, room);
          xa[k] = *reinterpret_cast<const Raw*>(in + o);
          xb[k] = *reinterpret_cast<const Raw*>(in + o + to_b);
          turned[k] = as_pairs<kInter>(load4(grad + o), load4(grad + o + to_b));
        }
#pragma unroll
        for (int k = 0; k < n(); ++k) {
          const Pairs x = as_pairs<kInter>(Four<T>::get(xa[k]), Four<T>::get(xb[k]));
          if (at.turned) turned[k] = mix(turned[k], back);
          const Pairs wx = times(x, weight);
          sd[2 * k] = sum4(fma4(x.y, x.y, mul4(x.x, x.x)));
          sd[2 * k + 1] = sum4(fma4(wx.y, turned[k].y, mul4(wx.x, turned[k].x)));
        }
        group_sum(sd, at.g);
#pragma unroll
        for (int k = 0; k < n(); ++k) {
          if (!at.on || k * next > room) continue;
          const float r = rsqrtf(fmaf(sd[2 * k], inv_d, a.eps));
          const float m = sd[2 * k + 1] * r * inv_d;
          const Pairs& g = turned[k];
          const Pairs n_ = scaled(as_pairs<kInter>(Four<T>::get(xa[k]), Four<T>::get(xb[k])), r);
          dw[which] = Pairs{fma4(g.x, n_.x, dw[which].x), fma4(g.y, n_.y, dw[which].y)};
          // r (w g - m n)
          const Pairs wg = times(scaled(g, r), weight);
          const F4 mr = all4(-m * r);
          F4 p, q;
          as_quads<kInter>(Pairs{fma4(n_.x, mr, wg.x), fma4(n_.y, mr, wg.y)}, p, q);
          store4(out + k * next, p);
          store4(out + k * next + to_b, q);
        }
        in += n() * next;
        grad += n() * next;
        out += n() * next;
        room -= n() * next;
      };
      int left = to - from;
      for (; left >= 2; left -= 2) heads(Count<2>());
      if (left) heads(Count<1>());
    }
  }
  // The warp's heads in order (a head's lanes hold the same channels), then the warps.
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    F4 p, q;
    as_quads<kInter>(dw[which], p, q);
    float v[8] = {p.a.x, p.a.y, p.b.x, p.b.y, q.a.x, q.a.y, q.b.x, q.b.y};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float s = v[i];
      for (int h = 1; h < at.groups; ++h) s += __shfl_sync(0xffffffffu, v[i], h * at.g.lanes + at.g.within);
      v[i] = s;
    }
    if (lane < at.g.lanes) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sums[warp][which][at.a + i] = v[i];
        sums[warp][which][at.b + i] = v[4 + i];
      }
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * a.D; c += kThreads) {
    const int which = c >= a.D, ch = c - which * a.D;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) s += sums[i][which][ch];
    part_sums[((int64_t)which * a.D + ch) * gridDim.x + blockIdx.x] = s;
  }
}

// The blocks' sums, [q, k][channel][block]: a warp a channel, then a tree over its lanes.
__global__ void __launch_bounds__(256) qk_weight_grad_k(QkRopeArgs a, const float* part, int blocks) {
  const int which = blockIdx.y, ch = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const float* p = part + ((int64_t)which * a.D + ch) * blocks;
  float s = 0.f;
#pragma unroll 8
  for (int b = lane; b < blocks; b += 32) s += p[b];
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) (which ? a.k.dweight : a.q.dweight)[ch] = s;
}

// ---- launch -----------------------------------------------------------------------------------

Split split(const QkRopeArgs& a) {
  Split w;
  w.lanes = a.D / 8;
  const int groups = 32 / w.lanes;
  w.q_steps = (a.q.H + groups - 1) / groups;
  w.k_steps = (a.k.H + groups - 1) / groups;
  // Tokens are shared between warps until there are 16 warps an SM with work.
  w.parts = (int)std::max<int64_t>(1, std::min<int64_t>(w.q_steps + w.k_steps, 148 * 16 / a.rows));
  w.items = a.rows * w.parts;
  return w;
}

template <typename T, bool kNorm>
cudaError_t forward(const QkRopeArgs& a, cudaStream_t s) {
  const Split w = split(a);
  const unsigned grid = (unsigned)((w.items + kWarps - 1) / kWarps);
  if (a.interleaved)
    qk_rope_k<T, kNorm, true><<<grid, kThreads, 0, s>>>(a, w);
  else
    qk_rope_k<T, kNorm, false><<<grid, kThreads, 0, s>>>(a, w);
  return cudaGetLastError();
}

constexpr int kBwdBlocks = 148 * 4;
int bwd_blocks(const Split& w) { return (int)std::min<int64_t>(kBwdBlocks, (w.items + kWarps - 1) / kWarps); }

template <typename T>
cudaError_t backward(const QkRopeArgs& a, float* part, cudaStream_t s) {
  const Split w = split(a);
  const int blocks = bwd_blocks(w);
  if (a.interleaved)
    qk_norm_rope_bwd_k<T, true><<<blocks, kThreads, 0, s>>>(a, w, part);
  else
    qk_norm_rope_bwd_k<T, false><<<blocks, kThreads, 0, s>>>(a, w, part);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  qk_weight_grad_k<<<dim3(a.D / 8, a.k.H ? 2 : 1), 256, 0, s>>>(a, part, blocks);
  return cudaGetLastError();
}

}  // namespace

cudaError_t qk_rope_launch(const QkRopeArgs& a, cudaStream_t s) {
  if (a.q.weight) return a.bf16 ? forward<__nv_bfloat16, true>(a, s) : forward<float, true>(a, s);
  return a.bf16 ? forward<__nv_bfloat16, false>(a, s) : forward<float, false>(a, s);
}

size_t qk_norm_rope_bwd_workspace_bytes(const QkRopeArgs& a) {
  return (size_t)bwd_blocks(split(a)) * 2 * a.D * sizeof(float);
}

cudaError_t qk_norm_rope_bwd_launch(const QkRopeArgs& a, void* workspace, cudaStream_t s) {
  float* part = static_cast<float*>(workspace);
  return a.bf16 ? backward<__nv_bfloat16>(a, part, s) : backward<float>(a, part, s);
}

}  // namespace dig
