// Joining the parts of the tree attention, for both of its kernels, and the
// launch of a kernel as a programmatic dependent of the one before it.
#pragma once

#include "common.cuh"
#include "tc_util.cuh"
#include "tree.h"

namespace akv {
namespace {

// The one rounding to the output's type.
__device__ __forceinline__ void store4(float* p, const float (&c)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(c[0], c[1], c[2], c[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&c)[4]) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(c[0], c[1]), hi = __floats2bfloat162_rn(c[2], c[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

// Four warps per output row, each a quarter of the parts: joined by their
// references and sums, the compressed tokens' share rotated back.  Bound by the
// latency of the parts' reads from L2, so they are spread over warps: 2.5 us
// inside a call for 32 rows of 19 parts, 11 to 13 us for 2048 rows of 9 (9.4 MB).
template <typename T>
__global__ void __launch_bounds__(256) tree_merge_kernel(TreeArgs a, int rb) {
  __shared__ float4 sum[2][4][2][32];
  __shared__ float2 lm[2][4];
  const int lane = threadIdx.x & 31, wq = (threadIdx.x >> 5) & 3, grp = threadIdx.x >> 7;
  const int64_t i = (int64_t)blockIdx.x * 2 + grp;
  const int Hq = a.H * a.G;
  const bool there = i < (int64_t)a.batch * a.T * Hq;
  const int b = there ? (int)(i / (a.T * Hq)) : 0, t = (int)(i / Hq % a.T), hq = (int)(i % Hq), h = hq / a.G;
  const bool wanted = there && t < tree_new(a, b);
  const unsigned long long seen = wanted && a.inf_v ? tree_mask(a, b, t) : 0ull;
  const int prefix_parts = wanted ? a.parts - tree_tail_parts(a, tree_len(a, b), tree_new(a, b)) : 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!wanted) return;
  const int r = t * a.G + hq % a.G;
  const int64_t unit = ((int64_t)b * a.H + h) * a.n_blk + r / rb;
  const float2* ml = reinterpret_cast<const float2*>(a.ml) + unit * a.parts * rb + r % rb;
  const float* o = a.part + (unit * a.parts * rb + r % rb) * kD + lane * 4;
  unsigned long long odd = wq == 0 && seen ? a.inf_v[(int64_t)b * a.H + h] & seen : 0ull;
  // parts wq, wq + 4, ...: exact tokens' (y) and compressed tokens' (x) in units
  // of the largest reference met so far; four parts' loads in flight
  float m = -INFINITY, l = 0.f;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
  for (int s0 = wq; s0 < a.parts; s0 += 16) {
    float2 e[4];
    float4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int s = min(s0 + 4 * k, a.parts - 1);
      e[k] = ml[(int64_t)s * rb];
      v[k] = *reinterpret_cast<const float4*>(o + (int64_t)s * rb * kD);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int s = s0 + 4 * k;
      if (s >= a.parts) break;
      if (__float_as_uint(e[k].x) == kTreeBadPart && lane == 0) latch_error(a.counters, kDevErrBounds);
      if (e[k].y == 0.f) continue;
      const float mn = fmaxf(m, e[k].x), f = m > -INFINITY ? exp2f(m - mn) : 0.f, g = exp2f(e[k].x - mn);
      m = mn;
      l = l * f + e[k].y * g;
      x.x *= f; x.y *= f; x.z *= f; x.w *= f;
      y.x *= f; y.y *= f; y.z *= f; y.w *= f;
      float4& z = s < prefix_parts ? x : y;
      z.x = fmaf(v[k].x, g, z.x); z.y = fmaf(v[k].y, g, z.y); z.z = fmaf(v[k].z, g, z.z); z.w = fmaf(v[k].w, g, z.w);
    }
  }
  sum[grp][wq][0][lane] = x;
  sum[grp][wq][1][lane] = y;
  if (lane == 0) lm[grp][wq] = make_float2(m, l);
  tc::named_bar(1 + grp, 128);
  if (wq) return;
  m = fmaxf(fmaxf(lm[grp][0].x, lm[grp][1].x), fmaxf(lm[grp][2].x, lm[grp][3].x));
  float c[4] = {0.f, 0.f, 0.f, 0.f}, d[4] = {0.f, 0.f, 0.f, 0.f};
  l = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 e = lm[grp][k];
    if (e.y == 0.f) continue;
    const float f = exp2f(e.x - m);
    const float4 p = sum[grp][k][0][lane], q = sum[grp][k][1][lane];
    l = fmaf(e.y, f, l);
    c[0] = fmaf(p.x, f, c[0]); c[1] = fmaf(p.y, f, c[1]); c[2] = fmaf(p.z, f, c[2]); c[3] = fmaf(p.w, f, c[3]);
    d[0] = fmaf(q.x, f, d[0]); d[1] = fmaf(q.y, f, d[1]); d[2] = fmaf(q.z, f, d[2]); d[3] = fmaf(q.w, f, d[3]);
  }
  if (!a.naive && prefix_parts > 0) {
    fwht128(c);
    const float n = rsqrtf((float)kD);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int k = 4 * lane + e;
      c[e] *= (a.sign_bits[k >> 5] >> (k & 31)) & 1u ? -n : n;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < 4; ++e) c[e] = (c[e] + d[e]) * inv;
  // infinities and NaN of the drafts' values, for the rows that see them
  while (odd) {
    const int k = __ffsll((long long)odd) - 1;
    odd &= odd - 1;
    float v[4];
    load4<T>(reinterpret_cast<const T*>(a.vn) + b * a.n_seq + k * a.n_tok + h * kD + lane * 4, v);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (!isfinite(v[e])) c[e] += v[e];
  }
  store4(reinterpret_cast<T*>(a.out) + i * kD + lane * 4, c);
}

template <typename K, typename... Args>
int launch_dependent(K kernel, dim3 grid, int threads, int smem, cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? ANCHORKV_OK : ANCHORKV_ECUDA;
}

template <typename T>
int launch_tree_merge(const TreeArgs& a, int rb, cudaStream_t s) {
  const int64_t rows = (int64_t)a.batch * a.T * a.H * a.G;
  return launch_dependent(tree_merge_kernel<T>, dim3((unsigned)((rows + 1) / 2)), 256, 0, s, a, rb);
}

}  // namespace
}  // namespace akv
