// Tree attention over fp32 compressed caches.
//
// "AnchorKV: Anchor-Residual KV Cache Compression" (pith.science review),
// Referee "Summary": a FlashAttention-style decoder rebuilds tiles when they
// are consumed.  A block of 16 or 64 rows (draft, query head) of one (sequence,
// KV head) walks its share of the tokens - compressed, paged, drafted, in this
// order - in tiles of 32: a warp rebuilds its four tokens' keys and values,
//   x^_t = gamma_t x_a(t) + sigma_t s . H lev(c_t) / sqrt(D),
// into shared memory, then 256 threads take the logits, the running maximum and
// sum of the softmax, and the products with the values, which stay in
// registers.  Everything is held in 32 bits: an fp32 cache is answered in fp32
// accuracy.  A tile's 32 terms are summed by themselves and join the row's sums
// with the rounding kept in a second word, since a part may be a million tokens
// long: added one by one behind a token that takes nearly all, 128 k small ones
// were off by 9e-4 of the output and 2^20 by 6e-3 (4e-7 now, for 9% of the time of
// blocks of 64 rows and 2% of 16; the second words are in shared memory, in
// registers they spilled and took 20%).
// Sixteen rows serve single tokens and small trees, where the latency of one
// tile counts; 64 rows share a rebuilt tile and read shared memory six times
// for 32 multiplications (logits) and three times (values), against three and
// two for eight, and are bound by those multiplications.  Measured: 1024 tokens,
// one head of 20 rows 18.2 us (latency: a tile after another, then the merge);
// four sequences, eight heads, 8192 tokens, 64 rows 785 us in blocks of 64 and
// 1595 in blocks of 16 (11 TFLOP/s of fp32); two, 512 rows 2.63 ms and 5.38.
#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "tree.h"
#include "tree_merge.cuh"

namespace akv {
namespace {

constexpr int kTT = 32;        // tokens of a tile
constexpr int kThr = 256;
constexpr int kKPitch = kD + 4;  // floats; a quarter-warp's float4 reads hit all banks
constexpr float kLog2e = 1.4426950408889634f;

template <int RB>
struct Sm {
  float q[RB][kD];
  float K[kTT][kKPitch];
  float V[kTT][kD];
  float P[kTT][RB + 4];
  float low[RB][kD];                                  // what the output rows' sums rounded away
  unsigned long long mask[RB];
};

// A warp's tokens of a tile, each as a key and a value: item i < 2 kOwn is
// token i / 2 of the warp, key or value by its low bit.
constexpr int kOwn = kTT / (kThr / 32);

// Item of one lane: its row, the factor of it, its residual record (or -1) and
// that one's scale.
struct Item {
  unsigned long long row;
  float gamma, sigma;
  int rec;
};

__device__ __forceinline__ Item find_item(const TreeArgs& a, const uint8_t* comp, int b, int h, int side, int t, int n_pre,
                                          int len, int total, int* bad_page) {
  Item it = {0ull, 1.f, 0.f, -1};
  if (t >= total) return it;
  if (t < n_pre) {
    const int64_t sh = (int64_t)side * a.H + h;
    const uint32_t w = reinterpret_cast<const uint32_t*>(comp + a.off_tok)[sh * a.N + t];
    const int tile = t >> 7, in = t & 127;
    const uint4 bm = *reinterpret_cast<const uint4*>(comp + a.off_bm + (sh * a.n_tiles + tile) * 16);
    int64_t rec = reinterpret_cast<const int*>(comp + a.off_pf)[sh * (a.n_tiles + 1) + tile];
    const int slot = min((int)(w & 0xffffu), a.k - 1);
    it.row = (unsigned long long)(reinterpret_cast<const float*>(comp + (side ? a.off_av : a.off_ak)) +
                                  ((int64_t)h * a.k + slot) * kD);
    it.gamma = half_bits_to_f(w >> 16);
    const int q = in >> 5;
    const uint32_t word = q == 0 ? bm.x : q == 1 ? bm.y : q == 2 ? bm.z : bm.w;
    if ((word >> (in & 31)) & 1u) {
      if (q > 0) rec += __popc(bm.x);
      if (q > 1) rec += __popc(bm.y);
      if (q > 2) rec += __popc(bm.z);
      rec += __popc(word & ((1u << (in & 31)) - 1u));
      if (rec >= 0 && rec < a.R) {
        it.rec = (int)rec;
        it.sigma = half_bits_to_f(reinterpret_cast<const uint16_t*>(comp + a.off_sig)[rec]);
      }
    }
  } else if (t < n_pre + len) {
    const int u = t - n_pre, pg = a.table[(int64_t)b * a.maxp + u / a.P];
    if (pg >= 0 && pg < a.n_pages)
      it.row = (unsigned long long)(reinterpret_cast<const float*>(side ? a.vp : a.kp) +
                                    (((int64_t)pg * a.H + h) * a.P + u % a.P) * kD);
    else
      *bad_page = 1;
  } else {
    it.row = (unsigned long long)(reinterpret_cast<const float*>(side ? a.vn : a.kn) + b * a.n_seq +
                                  (int64_t)(t - n_pre - len) * a.n_tok + h * kD);
  }
  return it;
}

// sum + low += x with the rounding of the sum kept in `low` (Knuth's two-sum): a
// tile's share joins a long sum without a loss, however small it is beside it.
__device__ __forceinline__ void add_exactly(float& sum, float& low, float x) {
  const float t = sum + x, z = t - sum;
  low += (sum - (t - z)) + (x - z);
  sum = t;
}
// Their value; an infinite sum has no rounding.
__device__ __forceinline__ float together(float sum, float low) { return fabsf(low) < INFINITY ? sum + low : sum; }

template <int kRB>
__global__ void __launch_bounds__(kThr, 2) tree_simt_kernel(TreeArgs a) {
  constexpr int kRW = kRB / 8;                        // rows of a warp in the softmax and the values' products
  extern __shared__ __align__(16) unsigned char raw[];
  Sm<kRB>& sm = *reinterpret_cast<Sm<kRB>*>(raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int part = blockIdx.x, blk = blockIdx.y, bh = blockIdx.z, b = bh / a.H, h = bh % a.H;
  const int64_t unit = (int64_t)bh * a.n_blk + blk;
  float* ml = a.ml + (unit * a.parts + part) * kRB * 2;
  if (part == 0 && blk == 0 && bh == 0 && tid < 16) a.counters[tid] = 0;      // the merge latches errors
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
  float acc[kRW][4];                                  // four columns of each row
#pragma unroll
  for (int i = 0; i < kRW; ++i) {
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
    *reinterpret_cast<float4*>(&sm.low[kRW * warp + i][lane * 4]) = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  // softmax state of the warp's rows, the same in every lane
  float m[kRW], l[kRW], l_low[kRW];
#pragma unroll
  for (int i = 0; i < kRW; ++i) { m[i] = -INFINITY; l[i] = l_low[i] = 0.f; }
  __shared__ int bad_page;
  if (tid == 0) bad_page = 0;
  __syncthreads();

  for (int tt = t0; tt < t1 && !bad; tt += kTT) {
    const int nt = min(kTT, t1 - tt);
    // lanes find the rows, then the warp brings them in, four at a time
    Item it = {0ull, 1.f, 0.f, -1};
    if (lane < 2 * kOwn)
      it = find_item(a, comp, b, h, lane & 1, tt + warp * kOwn + (lane >> 1), n_pre, len, t1, &bad_page);
#pragma unroll 1
    for (int i0 = 0; i0 < 2 * kOwn; i0 += 4) {
      float x[4][4], gm[4], sg[4];
      uint32_t code[4];
      bool res[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const unsigned long long row = __shfl_sync(0xffffffffu, it.row, i0 + k);
        const int rec = __shfl_sync(0xffffffffu, it.rec, i0 + k);
        gm[k] = __shfl_sync(0xffffffffu, it.gamma, i0 + k);
        sg[k] = __shfl_sync(0xffffffffu, it.sigma, i0 + k);
        res[k] = rec >= 0;
        const float4 v = row ? reinterpret_cast<const float4*>(row)[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
        x[k][0] = v.x; x[k][1] = v.y; x[k][2] = v.z; x[k][3] = v.w;
        code[k] = res[k] ? comp[a.off_codes + (int64_t)rec * kCodeBytes + lane] : 0u;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[k][e] *= gm[k];
        if (res[k]) {                                  // the same for the whole warp
          float z[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t ci = (code[k] >> (2 * e)) & 3u;
            z[e] = sg[k] * (ci == 0 ? a.lev[0] : ci == 1 ? a.lev[1] : ci == 2 ? a.lev[2] : a.lev[3]);
          }
          if (!a.naive) {
            fwht128(z);
            const float n = rsqrtf((float)kD);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int d = 4 * lane + e;
              z[e] *= (a.sign_bits[d >> 5] >> (d & 31)) & 1u ? -n : n;
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) x[k][e] += z[e];
        }
        const int j = warp * kOwn + (i0 + k) / 2;
        *reinterpret_cast<float4*>(k & 1 ? &sm.V[j][lane * 4] : &sm.K[j][lane * 4]) =
            make_float4(x[k][0], x[k][1], x[k][2], x[k][3]);
      }
    }
    __syncthreads();
    // logits: tokens j and (64 rows) j + 16, kSR rows
    {
      constexpr int kSR = kRB == 16 ? 2 : 4, kST = kRB == 16 ? 1 : 2;
      const int j = kRB == 16 ? tid & 31 : tid & 15, g = kRB == 16 ? tid >> 5 : tid >> 4;
      float s[kST][kSR];
#pragma unroll
      for (int t = 0; t < kST; ++t)
#pragma unroll
        for (int i = 0; i < kSR; ++i) s[t][i] = 0.f;
#pragma unroll 4
      for (int d = 0; d < kD; d += 4) {
        float4 kv[kST];
#pragma unroll
        for (int t = 0; t < kST; ++t) kv[t] = *reinterpret_cast<const float4*>(&sm.K[j + 16 * t][d]);
#pragma unroll
        for (int i = 0; i < kSR; ++i) {
          const float4 qv = *reinterpret_cast<const float4*>(&sm.q[kSR * g + i][d]);
#pragma unroll
          for (int t = 0; t < kST; ++t) {
            s[t][i] = fmaf(qv.x, kv[t].x, s[t][i]);
            s[t][i] = fmaf(qv.y, kv[t].y, s[t][i]);
            s[t][i] = fmaf(qv.z, kv[t].z, s[t][i]);
            s[t][i] = fmaf(qv.w, kv[t].w, s[t][i]);
          }
        }
      }
#pragma unroll
      for (int t = 0; t < kST; ++t)
#pragma unroll
        for (int i = 0; i < kSR; ++i) sm.P[j + 16 * t][kSR * g + i] = s[t][i];
    }
    __syncthreads();
    // softmax: lane = token.  Masked places of a tile with drafts become -1, so
    // that the products leave them out whatever the value's row holds; tokens
    // behind the last have zero rows.
    float sum[kRW][4];                                     // of this tile
    const int u = tt + lane - n_pre - len;                 // draft index, negative before the drafts
    const bool drafts = tt + nt > n_pre + len;
#pragma unroll
    for (int i = 0; i < kRW; ++i) {
      const int r = kRW * warp + i;
      const float s = sm.P[lane][r];
      const bool off = lane >= nt || (u >= 0 && !((sm.mask[r] >> u) & 1ull));
      // fmaxf passes NaN over; a NaN logit that is seen comes back through its exponential
      const float mn = fmaxf(m[i], warp_max(off ? -INFINITY : s));
      const float sc = m[i] == -INFINITY ? 0.f : exp2f(m[i] - mn);
      const float p = off ? 0.f : (mn == -INFINITY && s == mn) ? 0.f : exp2f(s - mn);
      if (sc != 1.f) {                                     // the same for the whole warp
        l[i] *= sc;
        l_low[i] *= sc;
        float4* low = reinterpret_cast<float4*>(&sm.low[r][lane * 4]);
        *low = make_float4(low->x * sc, low->y * sc, low->z * sc, low->w * sc);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] *= sc;
      }
      add_exactly(l[i], l_low[i], warp_sum(p));
      m[i] = mn;
      sm.P[lane][r] = off && drafts ? -1.f : p;
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[i][e] = 0.f;
    }
    __syncwarp();                                          // the warp's own rows
    if (drafts) {
      for (int j = 0; j < nt; ++j) {
        const float4 v = *reinterpret_cast<const float4*>(&sm.V[j][lane * 4]);
#pragma unroll
        for (int i = 0; i < kRW; ++i) {
          const float p = sm.P[j][kRW * warp + i];
          if (p < 0.f) continue;
          sum[i][0] = fmaf(p, v.x, sum[i][0]);
          sum[i][1] = fmaf(p, v.y, sum[i][1]);
          sum[i][2] = fmaf(p, v.z, sum[i][2]);
          sum[i][3] = fmaf(p, v.w, sum[i][3]);
        }
      }
    } else {
#pragma unroll 4
      for (int j = 0; j < kTT; ++j) {
        const float4 v = *reinterpret_cast<const float4*>(&sm.V[j][lane * 4]);
        float p[kRW];
#pragma unroll
        for (int i = 0; i < kRW; i += 2) {
          const float2 x = *reinterpret_cast<const float2*>(&sm.P[j][kRW * warp + i]);
          p[i] = x.x;
          p[i + 1] = x.y;
        }
#pragma unroll
        for (int i = 0; i < kRW; ++i) {
          sum[i][0] = fmaf(p[i], v.x, sum[i][0]);
          sum[i][1] = fmaf(p[i], v.y, sum[i][1]);
          sum[i][2] = fmaf(p[i], v.z, sum[i][2]);
          sum[i][3] = fmaf(p[i], v.w, sum[i][3]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kRW; ++i) {
      float4* low = reinterpret_cast<float4*>(&sm.low[kRW * warp + i][lane * 4]);
      float4 x = *low;
      add_exactly(acc[i][0], x.x, sum[i][0]);
      add_exactly(acc[i][1], x.y, sum[i][1]);
      add_exactly(acc[i][2], x.z, sum[i][2]);
      add_exactly(acc[i][3], x.w, sum[i][3]);
      *low = x;
    }
    bad = __syncthreads_or(bad_page);                  // the same answer for all: nobody looks at the next tile yet
  }
  float* o = a.part + ((unit * a.parts + part) * kRB + kRW * warp) * kD + lane * 4;
#pragma unroll
  for (int i = 0; i < kRW; ++i) {
    const int r = kRW * warp + i;
    if (lane == 0) {
      // a sequence that could not be read is NaN, not a guess
      ml[2 * r] = bad ? __uint_as_float(kTreeBadPart) : m[i];
      ml[2 * r + 1] = bad ? __int_as_float(0x7fc00000) : together(l[i], l_low[i]);
    }
    const float4 x = *reinterpret_cast<const float4*>(&sm.low[r][lane * 4]);
    *reinterpret_cast<float4*>(o + i * kD) =
        make_float4(together(acc[i][0], x.x), together(acc[i][1], x.y), together(acc[i][2], x.z), together(acc[i][3], x.w));
  }
}

template <int RB>
int launch_rb(const TreeArgs& a, cudaStream_t s) {
  static std::mutex mu;
  static int ready_dev = -1;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ANCHORKV_ECUDA;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (ready_dev != dev) {
      if (cudaFuncSetAttribute(tree_simt_kernel<RB>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Sm<RB>)) !=
          cudaSuccess)
        return ANCHORKV_ECUDA;
      ready_dev = dev;
    }
  }
  tree_simt_kernel<RB><<<dim3(a.parts, a.n_blk, a.batch * a.H), kThr, sizeof(Sm<RB>), s>>>(a);
  if (cudaGetLastError() != cudaSuccess) return ANCHORKV_ECUDA;
  return launch_tree_merge<float>(a, RB, s);
}

}  // namespace

void tree_plan_simt(const Plan& pl, TreePlan* tp) {
  // 64 rows where an SM has a tile of such a block at least.  Measured (16 rows,
  // 64 rows; us): one head of 64 rows, 1 k tokens 18.9, 30.6; 8 k 54.9, 49.2;
  // eight heads of 64 rows, 1 k 52.8, 37.6; 4 k 248, 91; eight of 20, 1 k 31.1,
  // 31.1; 8 k 199, 136
  const int64_t tiles = (pl.N + tp->cap + tp->T + kTT - 1) / kTT;
  const bool wide = tp->rows > 16 && (int64_t)tp->batch * pl.H * ((tp->rows + 63) / 64) * tiles >= 148;
  tp->RB = wide ? 64 : 16;
  tp->n_blk = (tp->rows + tp->RB - 1) / tp->RB;
  // parts so that two CTAs an SM have work, of a tile at least
  const int64_t units = (int64_t)tp->batch * pl.H * tp->n_blk;
  const int64_t fit = tp->room / (units * tp->RB);
  tp->parts = tp->tail_parts = (int)std::max<int64_t>(1, std::min(std::min(tiles, fit), (2 * 148 + units - 1) / units));
}

int launch_tree_simt(const TreeArgs& a, cudaStream_t s) { return a.RB == 16 ? launch_rb<16>(a, s) : launch_rb<64>(a, s); }

}  // namespace akv
