// Tree attention over fp32 compressed caches.
//
// "AnchorKV: Anchor-Residual KV Cache Compression" (pith.science review),
// Referee "Summary": a FlashAttention-style decoder rebuilds tiles when they
// are consumed.  A block of 16 rows (draft, query head) of one (sequence, KV
// head) walks its share of the tokens - compressed, paged, drafted, in this
// order - in tiles of 64: one warp rebuilds a token,
//   x^_t = gamma_t x_a(t) + sigma_t s . H lev(c_t) / sqrt(D),
// into shared memory, then 256 threads take the 16 x 64 logits, the running
// maximum and sum of the softmax, and the 16 x 128 products with the values,
// which stay in registers.  Everything is held in 32 bits: an fp32 cache is
// answered in fp32 accuracy, which the tensor cores' operand types are short
// of.  Bound by shared-memory reads of the products (a K element feeds four
// multiplications, a V element eight).
#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "tree.h"

namespace akv {
namespace {

constexpr int kRB = 16;        // rows of a block
constexpr int kTT = 64;        // tokens of a tile
constexpr int kThr = 256;
constexpr int kKPitch = kD + 4;  // floats; a quarter-warp's float4 reads hit all banks
constexpr int kPPitch = kRB + 4;
constexpr float kLog2e = 1.4426950408889634f;

struct Sm {
  float q[kRB][kD];
  float K[kTT][kKPitch];
  float V[kTT][kD];
  float P[kTT][kPPitch];
  float scale[kRB];
  unsigned long long mask[kRB];
};

// One token of the prefix, four coordinates per lane.
__device__ __forceinline__ void rebuild(const TreeArgs& a, const uint8_t* comp, int side, int h, int t, float (&x)[4]) {
  const int lane = threadIdx.x & 31;
  const uint32_t w = reinterpret_cast<const uint32_t*>(comp + a.off_tok)[((int64_t)side * a.H + h) * a.N + t];
  const int slot = min((int)(w & 0xffffu), a.k - 1);
  const float* anc = reinterpret_cast<const float*>(comp + (side ? a.off_av : a.off_ak)) + ((int64_t)h * a.k + slot) * kD;
  load4<float>(anc + lane * 4, x);
  const float gm = half_bits_to_f(w >> 16);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] *= gm;
  const int tile = t >> 7, in = t & 127;
  const uint32_t* bm =
      reinterpret_cast<const uint32_t*>(comp + a.off_bm) + (((int64_t)side * a.H + h) * a.n_tiles + tile) * 4;
  const uint32_t word = bm[in >> 5];
  if (!((word >> (in & 31)) & 1u)) return;
  int64_t rec = reinterpret_cast<const int*>(comp + a.off_pf)[((int64_t)side * a.H + h) * (a.n_tiles + 1) + tile];
  for (int i = 0; i < in >> 5; ++i) rec += __popc(bm[i]);
  rec += __popc(word & ((1u << (in & 31)) - 1u));
  if (rec < 0 || rec >= a.R) return;
  const uint32_t c = comp[a.off_codes + rec * kCodeBytes + lane];
  const float sg = half_bits_to_f(reinterpret_cast<const uint16_t*>(comp + a.off_sig)[rec]);
  float z[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t ci = (c >> (2 * i)) & 3u;
    z[i] = sg * (ci == 0 ? a.lev[0] : ci == 1 ? a.lev[1] : ci == 2 ? a.lev[2] : a.lev[3]);
  }
  if (!a.naive) {
    fwht128(z);
    const float n = rsqrtf((float)kD);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = 4 * lane + i;
      z[i] *= (a.sign_bits[d >> 5] >> (d & 31)) & 1u ? -n : n;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] += z[i];
}

__global__ void __launch_bounds__(kThr) tree_simt_kernel(TreeArgs a) {
  extern __shared__ __align__(16) unsigned char raw[];
  Sm& sm = *reinterpret_cast<Sm*>(raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int part = blockIdx.x, blk = blockIdx.y, bh = blockIdx.z, b = bh / a.H, h = bh % a.H;
  const int64_t unit = (int64_t)bh * a.n_blk + blk;
  float* ml = a.ml + (unit * a.parts + part) * kRB * 2;
  const int n_new = tree_new(a, b), rows = n_new * a.G;
  if (blk * kRB >= rows) return;                      // nobody reads these parts
  const int lay = a.comp ? tree_layout(a, b) : 0, len = tree_len(a, b);
  bool bad = lay < 0 || len < 0;
  const int n_pre = a.comp ? a.N : 0, total = n_pre + max(len, 0) + n_new;
  const int tiles = (total + kTT - 1) / kTT, per = (tiles + a.parts - 1) / a.parts;
  const int t0 = min(part * per * kTT, total), t1 = min(t0 + per * kTT, total);
  const uint8_t* comp = a.comp + (int64_t)max(lay, 0) * a.stride;

  const float qs = kLog2e * rsqrtf((float)kD);
  for (int i = tid; i < kRB * kD; i += kThr) {
    const int r = blk * kRB + i / kD, d = i % kD;
    float v = 0.f;
    if (r < rows)
      v = reinterpret_cast<const float*>(a.q)[b * a.q_seq + (r / a.G) * a.q_tok + (h * a.G + r % a.G) * kD + d] * qs;
    sm.q[i / kD][d] = v;
  }
  if (tid < kRB) {
    const int r = blk * kRB + tid;
    sm.mask[tid] = r < rows ? tree_mask(a, b, r / a.G) : 0ull;
  }
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  // softmax state of rows 2 warp and 2 warp + 1, the same in every lane
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  const int d_o = tid & 127, half = tid >> 7;         // this thread's output column, rows 8 half .. + 7
  __shared__ int bad_page;
  if (tid == 0) bad_page = 0;
  __syncthreads();

  for (int tt = t0; tt < t1 && !bad; tt += kTT) {
    const int nt = min(kTT, t1 - tt);
    for (int j = warp; j < kTT; j += kThr / 32) {
      float k4[4] = {0.f, 0.f, 0.f, 0.f}, v4[4] = {0.f, 0.f, 0.f, 0.f};
      const int t = tt + j;
      if (j < nt) {
        if (t < n_pre) {
          rebuild(a, comp, 0, h, t, k4);
          rebuild(a, comp, 1, h, t, v4);
        } else if (t < n_pre + len) {
          const int u = t - n_pre, pg = a.table[(int64_t)b * a.maxp + u / a.P];
          if (pg >= 0 && pg < a.n_pages) {
            const int64_t at = (((int64_t)pg * a.H + h) * a.P + u % a.P) * kD + lane * 4;
            load4<float>(reinterpret_cast<const float*>(a.kp) + at, k4);
            load4<float>(reinterpret_cast<const float*>(a.vp) + at, v4);
          } else if (lane == 0) {
            bad_page = 1;
          }
        } else {
          const int64_t at = b * a.n_seq + (int64_t)(t - n_pre - len) * a.n_tok + h * kD + lane * 4;
          load4<float>(reinterpret_cast<const float*>(a.kn) + at, k4);
          load4<float>(reinterpret_cast<const float*>(a.vn) + at, v4);
        }
      }
      *reinterpret_cast<float4*>(&sm.K[j][lane * 4]) = make_float4(k4[0], k4[1], k4[2], k4[3]);
      *reinterpret_cast<float4*>(&sm.V[j][lane * 4]) = make_float4(v4[0], v4[1], v4[2], v4[3]);
    }
    __syncthreads();
    {
      // logits: token j, rows 4 g .. 4 g + 3
      const int j = tid & 63, g = tid >> 6;
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int d = 0; d < kD; d += 4) {
        const float4 kv = *reinterpret_cast<const float4*>(&sm.K[j][d]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 qv = *reinterpret_cast<const float4*>(&sm.q[4 * g + i][d]);
          s[i] = fmaf(qv.x, kv.x, s[i]);
          s[i] = fmaf(qv.y, kv.y, s[i]);
          s[i] = fmaf(qv.z, kv.z, s[i]);
          s[i] = fmaf(qv.w, kv.w, s[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) sm.P[j][4 * g + i] = s[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 2 * warp + i;
      const float s0 = sm.P[lane][r], s1 = sm.P[lane + 32][r];
      const int u0 = tt + lane - n_pre - len, u1 = u0 + 32;      // draft index, negative before the drafts
      const bool off0 = lane >= nt || (u0 >= 0 && !((sm.mask[r] >> u0) & 1ull));
      const bool off1 = lane + 32 >= nt || (u1 >= 0 && !((sm.mask[r] >> u1) & 1ull));
      // fmaxf passes NaN over; a NaN logit that is seen comes back through its
      // exponential.  Masked places hold -1, so that the products leave them out
      // whatever the value's row holds.
      const float mt = warp_max(fmaxf(off0 ? -INFINITY : s0, off1 ? -INFINITY : s1));
      const float mn = fmaxf(m[i], mt);
      const float sc = m[i] == -INFINITY ? 0.f : exp2f(m[i] - mn);
      const float p0 = off0 ? -1.f : (mn == -INFINITY && s0 == mn) ? 0.f : exp2f(s0 - mn);
      const float p1 = off1 ? -1.f : (mn == -INFINITY && s1 == mn) ? 0.f : exp2f(s1 - mn);
      l[i] = l[i] * sc + warp_sum((off0 ? 0.f : p0) + (off1 ? 0.f : p1));
      m[i] = mn;
      sm.P[lane][r] = p0;
      sm.P[lane + 32][r] = p1;
      if (lane == 0) sm.scale[r] = sc;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] *= sm.scale[8 * half + i];
#pragma unroll 4
    for (int j = 0; j < kTT; ++j) {
      const float v = sm.V[j][d_o];
      const float4 pa = *reinterpret_cast<const float4*>(&sm.P[j][8 * half]);
      const float4 pb = *reinterpret_cast<const float4*>(&sm.P[j][8 * half + 4]);
      const float p[8] = {pa.x, pa.y, pa.z, pa.w, pb.x, pb.y, pb.z, pb.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = p[i] < 0.f ? acc[i] : fmaf(p[i], v, acc[i]);
    }
    __syncthreads();
    bad = bad || bad_page;
  }
  if (bad && tid == 0) latch_error(a.counters, kDevErrBounds);
  if (lane < 2) {
    const int r = 2 * warp + lane;
    // a sequence that could not be read is NaN, not a guess
    ml[2 * r] = bad ? 0.f : m[lane];
    ml[2 * r + 1] = bad ? __int_as_float(0x7fc00000) : l[lane];
  }
  float* o = a.part + ((unit * a.parts + part) * kRB + 8 * half) * kD + d_o;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i * kD] = acc[i];
}

// One warp per output row: the parts joined by their maxima and sums.
__global__ void __launch_bounds__(kThr) tree_simt_merge_kernel(TreeArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * (kThr / 32) + (threadIdx.x >> 5);
  const int Hq = a.H * a.G;
  if (i >= (int64_t)a.batch * a.T * Hq) return;
  const int b = (int)(i / (a.T * Hq)), t = (int)(i / Hq % a.T), hq = (int)(i % Hq), h = hq / a.G;
  if (t >= tree_new(a, b)) return;
  const int r = t * a.G + hq % a.G;
  const int64_t unit = ((int64_t)b * a.H + h) * a.n_blk + r / kRB;
  const float* ml = a.ml + (unit * a.parts * kRB + r % kRB) * 2;
  const float* o = a.part + (unit * a.parts * kRB + r % kRB) * kD + lane * 4;
  float m = -INFINITY;
  for (int s = 0; s < a.parts; ++s) m = fmaxf(m, ml[(int64_t)s * kRB * 2]);
  float l = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < a.parts; ++s) {
    const float ls = ml[(int64_t)s * kRB * 2 + 1];
    if (ls == 0.f) continue;
    const float w = exp2f(ml[(int64_t)s * kRB * 2] - m);
    const float4 v = *reinterpret_cast<const float4*>(o + (int64_t)s * kRB * kD);
    l = fmaf(w, ls, l);
    x[0] = fmaf(w, v.x, x[0]);
    x[1] = fmaf(w, v.y, x[1]);
    x[2] = fmaf(w, v.z, x[2]);
    x[3] = fmaf(w, v.w, x[3]);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  float* out = reinterpret_cast<float*>(a.out) + i * kD + lane * 4;
  *reinterpret_cast<float4*>(out) = make_float4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
}

}  // namespace

void tree_plan_simt(const Plan& pl, TreePlan* tp) {
  tp->RB = kRB;
  tp->n_blk = (tp->rows + kRB - 1) / kRB;
  // parts so that two CTAs an SM have work, of a tile at least
  const int64_t units = (int64_t)tp->batch * pl.H * tp->n_blk, tiles = (pl.N + tp->cap + tp->T + kTT - 1) / kTT;
  tp->parts = (int)std::max<int64_t>(1, std::min<int64_t>(tiles, (2 * 148 + units - 1) / units));
}

int launch_tree_simt(const TreeArgs& a, cudaStream_t s) {
  static std::mutex mu;
  static int ready_dev = -1;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ANCHORKV_ECUDA;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (ready_dev != dev) {
      if (cudaFuncSetAttribute(tree_simt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Sm)) !=
          cudaSuccess)
        return ANCHORKV_ECUDA;
      ready_dev = dev;
    }
  }
  if (cudaMemsetAsync(a.counters, 0, 64, s) != cudaSuccess) return ANCHORKV_ECUDA;
  tree_simt_kernel<<<dim3(a.parts, a.n_blk, a.batch * a.H), kThr, sizeof(Sm), s>>>(a);
  if (cudaGetLastError() != cudaSuccess) return ANCHORKV_ECUDA;
  const int64_t rows = (int64_t)a.batch * a.T * a.H * a.G;
  tree_simt_merge_kernel<<<(unsigned)((rows + kThr / 32 - 1) / (kThr / 32)), kThr, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? ANCHORKV_OK : ANCHORKV_ECUDA;
}

}  // namespace akv
