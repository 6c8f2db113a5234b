// qk_rope.cu -- rotary positions of query and key heads, alone or behind an RMS norm of
// every head, and the gradients (include/dig_gla.h, rope, qk_norm_rope, qk_norm_rope_bwd).
#include <math.h>

#include "dev_common.cuh"
#include "internal.h"

namespace dig {

namespace {

__device__ __forceinline__ float ld(const float* p) { return *p; }
__device__ __forceinline__ float ld(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st(float* p, float v) { *p = v; }
__device__ __forceinline__ void st(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// cos and sin of position * inv_freq, times scale.  The angle is formed in fp64 and
// reduced to a fraction of a turn there, so far positions keep their phase.
__device__ __forceinline__ float2 phase(const QkRopeArgs& a, int64_t row, int pair) {
  double pos;
  if (!a.positions)
    pos = (double)(row % a.period);
  else
    pos = a.positions64 ? (double)static_cast<const long long*>(a.positions)[row]
                        : (double)static_cast<const int*>(a.positions)[row];
  double turn = pos * ((double)a.inv_freq[pair] * 0.15915494309189535);
  turn -= rint(turn);
  float s, c;
  sincospif(2.f * (float)turn, &s, &c);
  return make_float2(c * a.scale, s * a.scale);
}

__device__ __forceinline__ void pair_channels(const QkRopeArgs& a, int pair, int& i, int& j) {
  i = a.interleaved ? 2 * pair : pair;
  j = a.interleaved ? 2 * pair + 1 : pair + a.rot / 2;
}

// One warp per (row, head).
template <typename T>
__global__ void __launch_bounds__(128) qk_rope_k(QkRopeArgs a) {
  const int lane = threadIdx.x & 31, H = a.q.H + a.k.H;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (item >= a.rows * H) return;
  const int64_t row = item / H;
  int head = (int)(item - row * H);
  const HeadRows& t = head < a.q.H ? a.q : a.k;
  if (head >= a.q.H) head -= a.q.H;
  const T* in = static_cast<const T*>(t.in) + row * t.stride + (int64_t)head * a.D;
  T* out = static_cast<T*>(t.out) + row * t.out_stride + (int64_t)head * a.D;
  float r = 1.f;
  if (t.weight) {
    float ss = 0.f;
    for (int c = lane; c < a.D; c += 32) ss = fmaf(ld(in + c), ld(in + c), ss);
    r = rsqrtf(warp_sum(ss) / a.D + a.eps);
  }
  auto norm = [&](int c) { return t.weight ? ld(in + c) * r * t.weight[c] : ld(in + c); };
  for (int p = lane; p < a.rot / 2; p += 32) {
    int i, j;
    pair_channels(a, p, i, j);
    float2 w = phase(a, row, p);
    if (a.inverse) w.y = -w.y;
    const float u = norm(i), v = norm(j);
    st(out + i, u * w.x - v * w.y);
    st(out + j, v * w.x + u * w.y);
  }
  for (int c = a.rot + lane; c < a.D; c += 32) st(out + c, norm(c));
}

constexpr int kBwdBlocks = 148;

// The gradients: a block takes rows blockIdx.x, blockIdx.x + gridDim.x, ...; its partial
// weight gradients go to the workspace, [2][block][D].
template <typename T>
__global__ void __launch_bounds__(256) qk_norm_rope_bwd_k(QkRopeArgs a, float* part) {
  __shared__ float dy[8][256];
  __shared__ float dw[8][2][256];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, H = a.q.H + a.k.H;
  for (int c = lane; c < 512; c += 32) dw[w][c >> 8][c & 255] = 0.f;
  __syncwarp();
  for (int64_t item = (int64_t)blockIdx.x * 8 + w; item < a.rows * H; item += (int64_t)gridDim.x * 8) {
    const int64_t row = item / H;
    int head = (int)(item - row * H);
    const int which = head < a.q.H ? 0 : 1;
    const HeadRows& t = which ? a.k : a.q;
    if (which) head -= a.q.H;
    const T* in = static_cast<const T*>(t.in) + row * t.stride + (int64_t)head * a.D;
    const T* g = static_cast<const T*>(t.grad) + row * t.grad_stride + (int64_t)head * a.D;
    T* out = static_cast<T*>(t.out) + row * t.out_stride + (int64_t)head * a.D;
    for (int p = lane; p < a.rot / 2; p += 32) {
      int i, j;
      pair_channels(a, p, i, j);
      const float2 f = phase(a, row, p);
      const float u = ld(g + i), v = ld(g + j);
      dy[w][i] = u * f.x + v * f.y;
      dy[w][j] = v * f.x - u * f.y;
    }
    for (int c = a.rot + lane; c < a.D; c += 32) dy[w][c] = ld(g + c);
    __syncwarp();
    float ss = 0.f, dot = 0.f;
    for (int c = lane; c < a.D; c += 32) {
      const float xv = ld(in + c);
      ss = fmaf(xv, xv, ss);
      dot = fmaf(xv, dy[w][c] * t.weight[c], dot);
    }
    const float r = rsqrtf(warp_sum(ss) / a.D + a.eps);
    const float m = warp_sum(dot) * r / a.D;
    for (int c = lane; c < a.D; c += 32) {
      const float n = ld(in + c) * r;
      dw[w][which][c] = fmaf(dy[w][c], n, dw[w][which][c]);
      st(out + c, r * (dy[w][c] * t.weight[c] - n * m));
    }
    __syncwarp();
  }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * a.D; c += 256) {
    const int which = c / a.D, ch = c - which * a.D;
    float s = 0.f;
    for (int i = 0; i < 8; ++i) s += dw[i][which][ch];
    part[((int64_t)which * gridDim.x + blockIdx.x) * a.D + ch] = s;
  }
}

__global__ void qk_weight_grad_k(QkRopeArgs a, const float* part, int blocks) {
  const int which = blockIdx.x;
  float* dw = which ? a.k.dweight : a.q.dweight;
  for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
    float s = 0.f;
    for (int b = 0; b < blocks; ++b) s += part[((int64_t)which * blocks + b) * a.D + c];
    dw[c] = s;
  }
}

}  // namespace

cudaError_t qk_rope_launch(const QkRopeArgs& a, cudaStream_t s) {
  const int64_t items = a.rows * (a.q.H + a.k.H);
  const unsigned grid = (unsigned)((items + 3) / 4);
  if (a.bf16)
    qk_rope_k<__nv_bfloat16><<<grid, 128, 0, s>>>(a);
  else
    qk_rope_k<float><<<grid, 128, 0, s>>>(a);
  return cudaGetLastError();
}

size_t qk_norm_rope_bwd_workspace_bytes(const QkRopeArgs& a) { return (size_t)kBwdBlocks * 2 * a.D * sizeof(float); }

cudaError_t qk_norm_rope_bwd_launch(const QkRopeArgs& a, void* workspace, cudaStream_t s) {
  float* part = static_cast<float*>(workspace);
  if (a.bf16)
    qk_norm_rope_bwd_k<__nv_bfloat16><<<kBwdBlocks, 256, 0, s>>>(a, part);
  else
    qk_norm_rope_bwd_k<float><<<kBwdBlocks, 256, 0, s>>>(a, part);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  qk_weight_grad_k<<<a.k.H ? 2 : 1, 256, 0, s>>>(a, part, kBwdBlocks);
  return cudaGetLastError();
}

}  // namespace dig
