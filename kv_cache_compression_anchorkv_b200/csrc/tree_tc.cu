// Tree attention over compressed bf16 caches on the 5th-generation tensor
// cores.
//
// "AnchorKV: Anchor-Residual KV Cache Compression" (pith.science review),
// Referee "Summary": a FlashAttention-style decoder rebuilds tiles when they
// are consumed.  With R the orthonormal randomized Hadamard rotation,
//   R x^_t = gamma_t R x_a(t) + sigma_t lev(c_t),
// so in the rotated domain a token without a residual is a scaled copy of its
// anchor's row and a residual is four table entries, no transform per token:
//   q . K^_t = (R q) . (R K^_t),    sum_t p_t V^_t = R^T sum_t p_t (R V^_t).
// A pre-kernel rotates the anchors (k rows a side and head) once per call and
// the merge rotates the output rows back; queries are rotated where they are
// staged.
//
// Operands are fp16 (11-bit significands; bf16's 8 would cost four times the
// output's own rounding) with the magnitudes kept apart so that fp16's range
// never matters: every row, of an anchor, a query or an exact token, is
// divided by a power of two near its largest element, and what a token row is
// multiplied by,
//   row_t = x^_t / w_t,    w_t = gamma_t M_a  (or sigma_t where that is larger),
// is applied in fp32, to the logits for keys and to the probabilities for
// values.  Accumulators, logits and sums are fp32.
//
// One CTA owns up to 64 rows (draft, query head) of one (sequence, KV head)
// and a share of its tokens, in tiles of 128:
//   S^T [128 tokens x rows]  = K^ Q^T      A = key tile, B = queries
//   O^T [128 coords x rows] += V^T P       A = value tile (token-major), B = P
// Tokens are on the accumulator's lanes, so a thread owns a token: its scales
// are scalars, its row of P is contiguous, and the cost of the softmax goes
// with the rows there are (16, 32 or 64 columns) instead of a padded 128.
//   warps 0-3   softmax: logits from tensor memory, exponentials, P to shared
//               memory; at the end the outputs
//   warps 4-7, 8-11  key and value tiles: anchor rows by 16-byte asynchronous
//               copies into the 128-byte swizzle, residual rows finished in
//               place (one half-warp each), one tile behind the copies
//   warp 12     issues the MMAs
// The maximum over tokens would need a reduction across lanes for every row
// and tile.  Instead each row keeps two power-of-two references, one for the
// sum of p and one for w p (the fp16 operand), which move only when a tile
// would leave their range: one vote per tile.  Powers of two make every
// rescaling exact, so the result does not depend on when it happens.
//
// Bound by the anchor rows' way from L2 (64 KB a tile).
#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "tc_util.cuh"
#include "tree.h"

namespace akv {
namespace {

constexpr int kTT = 128;                  // tokens of a tile
constexpr int kThreads = 13 * 32;
constexpr int kKSt = 2, kVSt = 2;         // stages of the key and value rings
constexpr int kKSl = kKSt + 2;            // key scales outlive their tile by the two logit buffers
constexpr int kTileBytes = kTT * kD * 2;
constexpr int kHalf = kTileBytes / 2;     // 64 coordinates of every row
constexpr int kOCols = 64;                // output columns in tensor memory
constexpr int kTmemCols = 256;
constexpr float kLog2e = 1.4426950408889634f;
// A new reference puts the largest |w p| between 1/2 and 1: 2^15 above it for
// later tiles, and what fp16 rounds away below 2^-14 is at most 2^-25 of the
// largest contribution each.
constexpr float kPLimit = 32768.f;        // fp16 holds 65504
constexpr float kSumLimit = 1.0995116e12f;  // 2^40, far below fp32's range
constexpr float kRefGap = 120.f;          // the references' largest distance downwards

struct Sm {
  uint8_t K[kKSt][kTileBytes];
  uint8_t V[kVSt][kTileBytes];
  uint8_t P[2][kTT * 128];                // [token][64 rows] fp16, swizzled
  uint8_t Q[64 * kD * 2];
  uint8_t codes[2][2][kTT * kCodeBytes];  // [side][tile parity]
  int4 ent[2][3][kTT];                    // residual rows of a tile: row, anchor factor, level table
  float rk[kKSl][kTT];                    // key scales
  float wv[kVSt][kTT];                    // value scales
  int idx[2][2][kTT];                     // anchor slots, [side][tile parity]
  float cs[64], nm[64], cw[64], mp[64];   // per row: logit scale, -reference of the sum, 2^(sum's - w p's), w p's
  float fl[64], fp[64];                   // rescaling factors
  int red[2][4][32];
  float lsum[4][64];
  unsigned long long mask[kTreeMaxDrafts];
  unsigned char colt[64];                 // draft of each row
  uint64_t kfull[kKSt], kempty[kKSt], vfull[kVSt], pv[2], sfull[2], sempty[2], pfull[2], sk[kKSl], sv[kVSt];
  uint32_t tmem;
  int err, bad, rep;
};
static_assert(kVSt == 2, "the value ring and the P buffers share the barrier pv");

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Power of two at or below |x| for the largest magnitude's bits (fp32), kept
// where its inverse is a normal number too.
__device__ __forceinline__ int scale_exp(uint32_t bits) { return min(max((int)(bits >> 23), 1), 253); }
__device__ __forceinline__ float exp_to_f(int e) { return __uint_as_float((uint32_t)e << 23); }       // 2^(e - 127)
__device__ __forceinline__ float exp_to_inv(int e) { return __uint_as_float((uint32_t)(254 - e) << 23); }

__device__ __forceinline__ uint32_t bar_or(int id, int count, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\t"
      "setp.ne.u32 a, %3, 0;\n\t"
      "barrier.cta.red.or.pred b, %1, %2, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(count), "r"((uint32_t)p)
      : "memory");
  return r;
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Floats as integers in the same order (its own inverse), for the warp-wide
// integer maximum.
__device__ __forceinline__ int ordered(float x) {
  const int i = __float_as_int(x);
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

// Instruction descriptor of kind::f16 with fp16 operands and fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// First sequence with the layout of sequence b: it holds the rotated anchors.
__device__ __forceinline__ int first_with_layout(const TreeArgs& a, int b) {
  if (!a.layout_of) return b;
  const int mine = a.layout_of[b];
  for (int i = 0; i < b; ++i)
    if (a.layout_of[i] == mine) return i;
  return b;
}

// Rotated anchors of every layout in use, one warp per row: fp16 rows over a
// power of two and that power (1/sqrt(D) of the rotation in it).  Clears the
// status words and the flags of infinite values.  Bound by launch latency
// (4.6 k rows for a 32k-token prompt, 2.4 MB).
__global__ void __launch_bounds__(256) tree_prep_kernel(TreeArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = blockIdx.z, sh = blockIdx.y;
  if (blockIdx.x == 0) {
    if (sh == 0 && b == 0 && threadIdx.x < 16) a.counters[threadIdx.x] = 0;
    if (sh < a.H && threadIdx.x == 32) a.inf_v[(int64_t)b * a.H + sh] = 0ull;
  }
  if (!a.comp || first_with_layout(a, b) != b) return;
  const int lay = tree_layout(a, b);
  if (lay < 0) return;
  const int side = sh / a.H, h = sh % a.H;
  const __nv_bfloat16* src =
      reinterpret_cast<const __nv_bfloat16*>(a.comp + (int64_t)lay * a.stride + (side ? a.off_av : a.off_ak)) +
      (int64_t)h * a.k * kD;
  const int64_t row0 = ((int64_t)b * 2 * a.H + sh) * a.k;
  for (int s = blockIdx.x * 8 + warp; s < a.k; s += gridDim.x * 8) {
    float v[4];
    load4<__nv_bfloat16>(src + (int64_t)s * kD + lane * 4, v);
    if (!a.naive) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = 4 * lane + i;
        if ((a.sign_bits[d >> 5] >> (d & 31)) & 1u) v[i] = -v[i];
      }
      fwht128(v);
    }
    const float m = warp_max(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))));
    const int e = scale_exp(__float_as_uint(m));
    const float inv = exp_to_inv(e);
    reinterpret_cast<uint2*>(a.anc)[(row0 + s) * 32 + lane] =
        make_uint2(pack_half2(v[0] * inv, v[1] * inv), pack_half2(v[2] * inv, v[3] * inv));
    if (lane == 0) a.anc_scale[row0 + s] = exp_to_f(e) * (a.naive ? 1.f : rsqrtf((float)kD));
  }
}

// What the producers of one side know of their CTA.
struct Prod {
  Sm* sm;
  int side, tid, n;                       // thread in the group, tiles
  uint8_t* ring;
  uint64_t *full, *empty, *scales;
  int stages, slots;
};

__device__ __forceinline__ void wait_b(Sm& sm, uint64_t* bar, uint32_t parity, const TreeArgs& a) {
  if (*(volatile int*)&sm.err) return;
  tc::wait_or_fail(bar, parity, &sm.err, a.counters, kDevErrTimeout);
}

__device__ __forceinline__ uint32_t swz(int row, int chunk) {   // byte offset of a row's 16-byte piece in a tile
  return (uint32_t)((chunk >> 3) * kHalf + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}

// Token words of one tile, one token per thread: its word, its bitmap word,
// and the record before the first of its word.
struct Tok {
  uint32_t word, bits;
  int rec;
  bool in;
};

__device__ __forceinline__ Tok load_tok(const TreeArgs& a, const uint8_t* comp, int sh, int tile, int i) {
  Tok t;
  const int64_t at = (int64_t)tile * kTT + i;
  t.in = at < a.N;
  t.word = t.in ? reinterpret_cast<const uint32_t*>(comp + a.off_tok)[(int64_t)sh * a.N + at] : 0u;
  const uint4 w = *reinterpret_cast<const uint4*>(comp + a.off_bm + ((int64_t)sh * a.n_tiles + tile) * 16);
  t.rec = reinterpret_cast<const int*>(comp + a.off_pf)[(int64_t)sh * (a.n_tiles + 1) + tile];
  const int q = i >> 5;
  t.bits = q == 0 ? w.x : q == 1 ? w.y : q == 2 ? w.z : w.w;
  if (q > 0) t.rec += __popc(w.x);
  if (q > 1) t.rec += __popc(w.y);
  if (q > 2) t.rec += __popc(w.z);
  if (!t.in) t.bits = 0u;                 // bits behind the last token mean nothing
  return t;
}

__device__ void produce_prefix(const TreeArgs& a, const Prod& p, const uint8_t* comp, int rep, int h, int tile0) {
  Sm& sm = *p.sm;
  const int i = p.tid, lane = i & 31, sh = p.side * a.H + h, bar_id = 2 + p.side;
  const int64_t row0 = ((int64_t)rep * 2 * a.H + sh) * a.k;
  const uint8_t* rows = reinterpret_cast<const uint8_t*>(a.anc) + row0 * (kD * 2);
  const float* scale = a.anc_scale + row0;
  const uint8_t* codes = comp + a.off_codes;
  const uint16_t* sig = reinterpret_cast<const uint16_t*>(comp + a.off_sig);
  const uint32_t ring = tc::smem_u32(p.ring);
  // two tiles ahead the token words, one tile ahead what hangs on them
  auto slot_of = [&](const Tok& t) { return min((int)(t.word & 0xffffu), a.k - 1); };
  auto rec_of = [&](const Tok& t) {
    const int r = t.rec + __popc(t.bits & ((1u << lane) - 1u));
    return (t.bits >> lane) & 1u && r >= 0 && r < a.R ? r : -1;
  };
  Tok t0 = load_tok(a, comp, sh, tile0, i);
  Tok t1 = p.n > 1 ? load_tok(a, comp, sh, tile0 + 1, i) : t0;
  float m0 = scale[slot_of(t0)];
  float s0 = rec_of(t0) >= 0 ? half_bits_to_f(sig[rec_of(t0)]) : 0.f;
  int n_rec_last = 0;

  for (int j = 0; j <= p.n; ++j) {
    int n_rec = 0;
    if (j < p.n) {
      const int st = j % p.stages, u = j / p.stages;
      const Tok t = t0;
      const float m = m0, sg = s0;
      t0 = t1;
      if (j + 2 < p.n) t1 = load_tok(a, comp, sh, tile0 + j + 2, i);
      if (j + 1 < p.n) {
        m0 = scale[slot_of(t0)];
        const int r = rec_of(t0);
        s0 = r >= 0 ? half_bits_to_f(sig[r]) : 0.f;
      }
      if (u > 0) wait_b(sm, &p.empty[st], (u - 1) & 1, a);
      // scale of the row, and the residual's table
      const int rec = rec_of(t);
      const float c1 = half_bits_to_f(t.word >> 16) * m;
      float w = c1;
      int4 e = make_int4(i, 0, 0, 0);
      if (rec >= 0) {
        const bool by_anchor = fabsf(c1) >= sg;
        w = by_anchor ? c1 : sg;
        const float ca = by_anchor ? 1.f : c1 / sg, cb = by_anchor ? (c1 != 0.f ? sg / c1 : 0.f) : 1.f;
        e.y = (int)pack_half2(ca, ca);
        e.z = (int)pack_half2(cb * a.lev[0], cb * a.lev[1]);
        e.w = (int)pack_half2(cb * a.lev[2], cb * a.lev[3]);
      }
      (p.side ? sm.wv : sm.rk)[j % p.slots][i] = t.in ? w : 0.f;
      sm.idx[p.side][j & 1][i] = slot_of(t);
      // this word's records follow those of the words before it
      const uint4 bw = *reinterpret_cast<const uint4*>(comp + a.off_bm + ((int64_t)sh * a.n_tiles + tile0 + j) * 16);
      const int first = reinterpret_cast<const int*>(comp + a.off_pf)[(int64_t)sh * (a.n_tiles + 1) + tile0 + j];
      n_rec = __popc(bw.x) + __popc(bw.y) + __popc(bw.z) + __popc(bw.w);
      if (first < 0 || first > a.R) n_rec = 0;
      else n_rec = (int)min((int64_t)n_rec, a.R - first);
      if (rec >= 0 && rec - first >= 0 && rec - first < kTT) sm.ent[p.side][j % 3][rec - first] = e;
      tc::mbar_arrive(&p.scales[j % p.slots]);
      tc::named_bar(bar_id, 128);
      // rows: sixteen lanes each
      const uint32_t base = ring + st * kTileBytes;
      const int c = i & 15;
#pragma unroll 4
      for (int r = i >> 4; r < kTT; r += 8)
        cp_async16(base + swz(r, c), rows + (int64_t)sm.idx[p.side][j & 1][r] * (kD * 2) + c * 16);
      const uint32_t cd = tc::smem_u32(sm.codes[p.side][j & 1]);
      for (int x = i; x < n_rec * 2; x += 128) cp_async16(cd + x * 16, codes + (int64_t)first * kCodeBytes + x * 16);
      cp_commit();
    }
    if (j > 0) {
      // the tile before: its copies have landed; finish its residual rows
      const int st = (j - 1) % p.stages;
      if (j < p.n) cp_wait<1>();
      else cp_wait<0>();
      tc::named_bar(bar_id, 128);
      uint8_t* tile = p.ring + st * kTileBytes;
      const uint8_t* cd = sm.codes[p.side][(j - 1) & 1];
      const int c = i & 15;
      for (int x = i >> 4; x < n_rec_last; x += 8) {
        const int4 e = sm.ent[p.side][(j - 1) % 3][x];
        const uint32_t code = *reinterpret_cast<const uint16_t*>(cd + x * kCodeBytes + c * 2);
        uint4* at = reinterpret_cast<uint4*>(tile + swz(e.x & 127, c));
        uint4 v = *at;
        uint32_t* vw = reinterpret_cast<uint32_t*>(&v);
        const __half2 ca = *reinterpret_cast<const __half2*>(&e.y);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          // two codes to the four byte numbers of their table entries
          const uint32_t n = (code >> (4 * k)) & 15u;
          const uint32_t sel = ((n | (n << 6)) & 0x303u) * 0x22u + 0x1010u;
          const uint32_t lv = __byte_perm((uint32_t)e.z, (uint32_t)e.w, sel);
          const __half2 y = __hfma2(ca, *reinterpret_cast<const __half2*>(&vw[k]), *reinterpret_cast<const __half2*>(&lv));
          vw[k] = *reinterpret_cast<const uint32_t*>(&y);
        }
        *at = v;
      }
      tc::fence_proxy_async_smem();
      tc::mbar_arrive(&p.full[st]);
    }
    n_rec_last = n_rec;
  }
}

// Exact rows, of pages and drafts: half a warp per row.
__device__ void produce_tail(const TreeArgs& a, const Prod& p, int b, int h, int tile0, int len, int n_new) {
  Sm& sm = *p.sm;
  const int i = p.tid, c = i & 15;
  const uint16_t* pool = reinterpret_cast<const uint16_t*>(p.side ? a.vp : a.kp);
  const uint16_t* fresh = reinterpret_cast<const uint16_t*>(p.side ? a.vn : a.kn);
  for (int j = 0; j < p.n; ++j) {
    const int st = j % p.stages, u = j / p.stages;
    if (u > 0) wait_b(sm, &p.empty[st], (u - 1) & 1, a);
    uint8_t* tile = p.ring + st * kTileBytes;
    for (int r0 = i >> 4; r0 < kTT; r0 += 32) {
      uint4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int t = (tile0 + j) * kTT + r0 + 8 * k;
        v[k] = make_uint4(0u, 0u, 0u, 0u);
        if (t < len) {
          const int pg = a.table[(int64_t)b * a.maxp + t / a.P];
          if (pg >= 0 && pg < a.n_pages)
            v[k] = *reinterpret_cast<const uint4*>(pool + (((int64_t)pg * a.H + h) * a.P + t % a.P) * kD + c * 8);
          else
            *(volatile int*)&sm.bad = 1;
        } else if (t - len < n_new) {
          v[k] = *reinterpret_cast<const uint4*>(fresh + b * a.n_seq + (int64_t)(t - len) * a.n_tok + h * kD + c * 8);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = r0 + 8 * k, t = (tile0 + j) * kTT + r;
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&v[k]);
        float x[8];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          x[2 * y] = __uint_as_float(w[y] << 16);
          x[2 * y + 1] = __uint_as_float(w[y] & 0xffff0000u);
        }
        uint32_t m = 0;
        bool odd = false;
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          const uint32_t bits = __float_as_uint(x[y]) & 0x7fffffffu;
          const bool fin = bits < 0x7f800000u;
          if (fin) m = max(m, bits);
          odd = odd || !fin;
          // an infinity or NaN in a draft's value must not reach the rows that
          // do not see it (0 x inf): the merge adds it where it is seen
          if (!fin && p.side && t >= len) x[y] = 0.f;
        }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const int e = scale_exp(m);
        const float inv = exp_to_inv(e);
        *reinterpret_cast<uint4*>(tile + swz(r, c)) =
            make_uint4(pack_half2(x[0] * inv, x[1] * inv), pack_half2(x[2] * inv, x[3] * inv),
                       pack_half2(x[4] * inv, x[5] * inv), pack_half2(x[6] * inv, x[7] * inv));
        if (odd && p.side && t >= len) atomicOr(&a.inf_v[(int64_t)b * a.H + h], 1ull << (t - len));
        if (c == 0) (p.side ? sm.wv : sm.rk)[j % p.slots][r] = m ? exp_to_f(e) : (p.side ? 0.f : 1.f);
      }
    }
    tc::fence_proxy_async_smem();
    tc::mbar_arrive(&p.scales[j % p.slots]);
    tc::mbar_arrive(&p.full[st]);
  }
}

// 16 columns of this warp's 32 accumulator lanes as floats.
__device__ __forceinline__ void load_cols(uint32_t taddr, uint32_t (&v)[16]) {
  tc::tmem_ld16(taddr, v);
  tc::tmem_wait_ld_dep(v);
}

// NC: rows (columns of the accumulators) of a CTA.
template <int NC>
__global__ void __launch_bounds__(kThreads, 1) tree_tc_kernel(TreeArgs a) {
  extern __shared__ __align__(1024) unsigned char raw[];
  Sm& sm = *reinterpret_cast<Sm*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int part = blockIdx.x, blk = blockIdx.y, bh = blockIdx.z, b = bh / a.H, h = bh % a.H;
  const int64_t unit = (int64_t)bh * a.n_blk + blk;
  float* ml = a.ml + (unit * a.parts + part) * NC * 2;
  const int n_new = tree_new(a, b), rows = n_new * a.G;
  if (blk * NC >= rows) return;                       // nobody reads these parts
  // this part's tiles: the first parts take the exact tokens, the others the compressed
  const bool tail = part < a.tail_parts;
  const int lay = a.comp ? tree_layout(a, b) : 0, len = tree_len(a, b);
  const bool out_of_range = lay < 0 || len < 0;
  int tile0, n;
  {
    const int tiles = tail ? (max(len, 0) + n_new + kTT - 1) / kTT : a.n_tiles;
    const int s = tail ? part : part - a.tail_parts, of = tail ? a.tail_parts : a.parts - a.tail_parts;
    tile0 = (int)((int64_t)tiles * s / of);
    n = (int)((int64_t)tiles * (s + 1) / of) - tile0;
  }
  if (n == 0 || out_of_range) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid < NC) {
      ml[2 * tid] = out_of_range ? 0.f : -INFINITY;
      ml[2 * tid + 1] = out_of_range ? __int_as_float(0x7fc00000) : 0.f;
    }
    if (out_of_range && tid == 0) latch_error(a.counters, kDevErrBounds);
    return;
  }

  // ---- set-up: barriers, tensor memory, queries, masks
  if (warp == 12) {
    tc::tmem_alloc(&sm.tmem, kTmemCols);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < kKSt; ++i) { tc::mbar_init(&sm.kfull[i], 128); tc::mbar_init(&sm.kempty[i], 1); }
    for (int i = 0; i < kVSt; ++i) { tc::mbar_init(&sm.vfull[i], 128); tc::mbar_init(&sm.sv[i], 128); }
    for (int i = 0; i < kKSl; ++i) tc::mbar_init(&sm.sk[i], 128);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sm.pv[i], 1);
      tc::mbar_init(&sm.sfull[i], 1);
      tc::mbar_init(&sm.sempty[i], 128);
      tc::mbar_init(&sm.pfull[i], 128);
    }
    tc::fence_barrier_init();
    sm.err = 0;
    sm.bad = 0;
    sm.rep = first_with_layout(a, b);
  }
  if (tid < 64) {
    const int r = blk * NC + tid;
    sm.colt[tid] = (unsigned char)min(r / a.G, a.T - 1);
    sm.nm[tid] = INFINITY;
    sm.mp[tid] = -INFINITY;
    sm.cw[tid] = 1.f;
    if (tid < a.T) sm.mask[tid] = tree_mask(a, b, tid);
  }
  if (NC < kOCols)                                    // columns of P that no row fills
    for (int i = tid; i < 2 * kTT * 8; i += kThreads) reinterpret_cast<uint4*>(sm.P)[i] = make_uint4(0u, 0u, 0u, 0u);
  const bool rotate = !tail && !a.naive;
  for (int c = warp; c < NC; c += kThreads / 32) {
    const int r = blk * NC + c;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (r < rows)
      load4<__nv_bfloat16>(reinterpret_cast<const __nv_bfloat16*>(a.q) + b * a.q_seq + (r / a.G) * a.q_tok +
                               (h * a.G + r % a.G) * kD + lane * 4, v);
    if (rotate) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = 4 * lane + i;
        if ((a.sign_bits[d >> 5] >> (d & 31)) & 1u) v[i] = -v[i];
      }
      fwht128(v);
    }
    const float m = warp_max(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))));
    const int e = scale_exp(__float_as_uint(m));
    const float inv = exp_to_inv(e);
    const int ch = (lane >> 1) & 7;
    *reinterpret_cast<uint2*>(sm.Q + (lane >> 4) * (NC * 128) + c * 128 + ((ch ^ (c & 7)) << 4) + (lane & 1) * 8) =
        make_uint2(pack_half2(v[0] * inv, v[1] * inv), pack_half2(v[2] * inv, v[3] * inv));
    // logits in log2 units; the rotation's 1/sqrt(D) here too
    if (lane == 0) sm.cs[c] = exp_to_f(e) * kLog2e * rsqrtf((float)kD) * (rotate ? rsqrtf((float)kD) : 1.f);
  }
  tc::fence_proxy_async_smem();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  // the rotated anchors, the cleared status words
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint32_t tmem = sm.tmem;

  if (warp == 12) {
    // ---- MMA issue
    if (lane == 0) {
      constexpr uint32_t id_s = idesc_f16(128, NC, 0, 0), id_o = idesc_f16(128, kOCols, 1, 1);
      const uint32_t kb = tc::smem_u32(sm.K), vb = tc::smem_u32(sm.V), pb = tc::smem_u32(sm.P), qb = tc::smem_u32(sm.Q);
      for (int i = 0; i <= n; ++i) {
        if (i < n) {
          const int st = i % kKSt, bf = i & 1;
          wait_b(sm, &sm.kfull[st], (i / kKSt) & 1, a);
          if (i >= 2) wait_b(sm, &sm.sempty[bf], ((i >> 1) - 1) & 1, a);
          tc::fence_after_sync();
          if (!*(volatile int*)&sm.err) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              tc::mma_bf16(tmem + kOCols + bf * NC,
                           tc::sw128_desc(kb + st * kTileBytes + (ks >> 2) * kHalf + (ks & 3) * 32),
                           tc::sw128_desc(qb + (ks >> 2) * (NC * 128) + (ks & 3) * 32), id_s, ks > 0);
            tc::mma_commit(&sm.kempty[st]);
            tc::mma_commit(&sm.sfull[bf]);
          }
        }
        if (i > 0) {
          const int o = i - 1, st = o % kVSt;
          wait_b(sm, &sm.vfull[st], (o / kVSt) & 1, a);
          wait_b(sm, &sm.pfull[o & 1], (o >> 1) & 1, a);
          tc::fence_after_sync();
          if (!*(volatile int*)&sm.err) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              tc::mma_bf16(tmem, tc::sw128_mn_desc(vb + st * kTileBytes + ks * 2048, kHalf),
                           tc::sw128_mn_desc(pb + (o & 1) * (kTT * 128) + ks * 2048, kTT * 128), id_o, o > 0 || ks > 0);
            tc::mma_commit(&sm.pv[o & 1]);
          }
        }
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---- rows of the key and value tiles
    Prod p;
    p.sm = &sm;
    p.side = warp >= 8;
    p.tid = tid & 127;
    p.n = n;
    p.ring = p.side ? sm.V[0] : sm.K[0];
    p.full = p.side ? sm.vfull : sm.kfull;
    p.empty = p.side ? sm.pv : sm.kempty;
    p.scales = p.side ? sm.sv : sm.sk;
    p.stages = 2;
    p.slots = p.side ? kVSt : kKSl;
    if (tail) produce_tail(a, p, b, h, tile0, len, n_new);
    else produce_prefix(a, p, a.comp + (int64_t)lay * a.stride, sm.rep, h, tile0);
  } else {
    // ---- softmax: thread = token
    constexpr int CW = NC < 32 ? NC : 32, CH = NC / CW;
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    float2 lacc[CH][CW / 2];
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int x = 0; x < CW / 2; ++x) lacc[c][x] = make_float2(0.f, 0.f);
    for (int i = 0; i < n; ++i) {
      const int bf = i & 1;
      // what this token is, and who sees it
      const int t = (tile0 + i) * kTT + tid;
      bool special = false, live = true;
      unsigned long long vis = ~0ull;
      if (tail) {
        special = (tile0 + i + 1) * kTT > len;
        live = t < len + n_new;
        if (special && live && t >= len) {
          vis = 0;
          for (int d = 0; d < a.T; ++d) vis |= ((sm.mask[d] >> (t - len)) & 1ull) << d;
        }
      } else {
        special = (tile0 + i + 1) * kTT > a.N;
        live = t < a.N;
      }
      if (!live) vis = 0;
      wait_b(sm, &sm.sk[i % kKSl], (i / kKSl) & 1, a);
      wait_b(sm, &sm.sv[i % kVSt], (i / kVSt) & 1, a);
      const float rk = sm.rk[i % kKSl][tid], w = sm.wv[i % kVSt][tid];
      wait_b(sm, &sm.sfull[bf], (i >> 1) & 1, a);
      tc::fence_after_sync();
      if (i >= 2) wait_b(sm, &sm.pv[bf], ((i >> 1) - 1) & 1, a);
      const uint32_t scol = tmem + lane_base + kOCols + bf * NC;
      uint8_t* prow = sm.P[bf] + tid * 128;
#pragma unroll
      for (int ch = 0; ch < CH; ++ch) {
        const int c0 = ch * CW;
        float2 p[CW / 2];
        uint32_t pk[CW / 2];
        auto exponentials = [&]() {
          float pmax = 0.f, vmax = 0.f;
#pragma unroll
          for (int x = 0; x < CW; x += 16) {
            uint32_t s[16];
            load_cols(scol + c0 + x, s);
#pragma unroll
            for (int y = 0; y < 16; y += 4) {
              const float4 cs = *reinterpret_cast<const float4*>(&sm.cs[c0 + x + y]);
              const float4 nm = *reinterpret_cast<const float4*>(&sm.nm[c0 + x + y]);
              const float4 cw = *reinterpret_cast<const float4*>(&sm.cw[c0 + x + y]);
#pragma unroll
              for (int z = 0; z < 4; z += 2) {
                const float2 k2 = __fmul2_rn(z ? make_float2(cs.z, cs.w) : make_float2(cs.x, cs.y), make_float2(rk, rk));
                float2 u = __ffma2_rn(make_float2(__uint_as_float(s[y + z]), __uint_as_float(s[y + z + 1])), k2,
                                      z ? make_float2(nm.z, nm.w) : make_float2(nm.x, nm.y));
                if (special) {
                  if (!((vis >> sm.colt[c0 + x + y + z]) & 1ull)) u.x = -INFINITY;
                  if (!((vis >> sm.colt[c0 + x + y + z + 1]) & 1ull)) u.y = -INFINITY;
                }
                const float2 e = make_float2(tc::ex2_approx(u.x), tc::ex2_approx(u.y));
                // in this order a masked 0 stays 0 whatever the value's scale
                const float2 v = __fmul2_rn(__fmul2_rn(e, make_float2(w, w)),
                                            z ? make_float2(cw.z, cw.w) : make_float2(cw.x, cw.y));
                pmax = fmaxf(pmax, fmaxf(e.x, e.y));
                vmax = fmaxf(vmax, fmaxf(fabsf(v.x), fabsf(v.y)));
                p[(x + y + z) / 2] = e;
                pk[(x + y + z) / 2] = pack_half2(v.x, v.y);
              }
            }
          }
          return pmax > kSumLimit || vmax > kPLimit;
        };
        if (bar_or(1, 128, exponentials())) {
          // ---- new references for these rows (the first tile, and rarely after)
          const float lw = w != 0.f ? __log2f(fabsf(w)) : -INFINITY;
#pragma unroll 1
          for (int x = 0; x < CW; x += 16) {
            uint32_t s[16];
            load_cols(scol + c0 + x, s);
#pragma unroll
            for (int y = 0; y < 16; ++y) {
              const int c = c0 + x + y;
              const bool seen = !special || ((vis >> sm.colt[c]) & 1ull);
              const float lg = seen ? __uint_as_float(s[y]) * (rk * sm.cs[c]) : -INFINITY;
              const int m1 = __reduce_max_sync(0xffffffffu, ordered(lg));
              const int m2 = __reduce_max_sync(0xffffffffu, ordered(lg + lw));
              if (lane == 0) {
                sm.red[0][warp][x + y] = m1;
                sm.red[1][warp][x + y] = m2;
              }
            }
          }
          tc::named_bar(1, 128);
          if (tid < CW) {
            const int c = c0 + tid;
            const float m1 = unordered(max(max(sm.red[0][0][tid], sm.red[0][1][tid]), max(sm.red[0][2][tid], sm.red[0][3][tid])));
            const float m2 = unordered(max(max(sm.red[1][0][tid], sm.red[1][1][tid]), max(sm.red[1][2][tid], sm.red[1][3][tid])));
            const float l_old = -sm.nm[c], p_old = sm.mp[c];
            const float l_new = fmaxf(l_old, ceilf(m1));
            float p_new = fmaxf(p_old, ceilf(m2));
            if (l_new > -INFINITY) p_new = fmaxf(p_new, l_new - kRefGap);
            sm.fl[c] = l_old > -INFINITY ? exp2f(l_old - l_new) : 0.f;
            sm.fp[c] = p_old > -INFINITY ? exp2f(p_old - p_new) : 0.f;
            sm.nm[c] = -l_new;
            sm.mp[c] = p_new;
            sm.cw[c] = l_new > -INFINITY ? exp2f(l_new - p_new) : 1.f;
          }
          tc::named_bar(1, 128);
#pragma unroll
          for (int x = 0; x < CW / 2; ++x) {
            lacc[ch][x].x *= sm.fl[c0 + 2 * x];
            lacc[ch][x].y *= sm.fl[c0 + 2 * x + 1];
          }
          if (i > 0) {
            wait_b(sm, &sm.pv[(i - 1) & 1], ((i - 1) >> 1) & 1, a);
            tc::fence_after_sync();
#pragma unroll 1
            for (int x = 0; x < CW; x += 16) {
              uint32_t o[16];
              load_cols(tmem + lane_base + c0 + x, o);
#pragma unroll
              for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * sm.fp[c0 + x + y]);
              tmem_st16(tmem + lane_base + c0 + x, o);
            }
            tmem_wait_st();
          }
          exponentials();
        }
#pragma unroll
        for (int x = 0; x < CW / 2; ++x) lacc[ch][x] = __fadd2_rn(lacc[ch][x], p[x]);
#pragma unroll
        for (int x = 0; x < CW / 8; ++x)
          *reinterpret_cast<uint4*>(prow + (((c0 / 8 + x) ^ (tid & 7)) << 4)) =
              make_uint4(pk[4 * x], pk[4 * x + 1], pk[4 * x + 2], pk[4 * x + 3]);
      }
      tc::fence_proxy_async_smem();
      tc::fence_before_sync();
      tc::mbar_arrive(&sm.sempty[bf]);
      tc::mbar_arrive(&sm.pfull[bf]);
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // ---- sums over the tokens, outputs in units of the sums' references
#pragma unroll
    for (int ch = 0; ch < CH; ++ch) {
      float v[32];
#pragma unroll
      for (int x = 0; x < 32; ++x) v[x] = x < CW ? (x & 1 ? lacc[ch][(x < CW ? x : 0) / 2].y : lacc[ch][(x < CW ? x : 0) / 2].x) : 0.f;
      transpose_reduce32(v, lane);
      if (lane < CW) sm.lsum[warp][ch * CW + lane] = v[0];
    }
    tc::named_bar(1, 128);
    wait_b(sm, &sm.pv[(n - 1) & 1], ((n - 1) >> 1) & 1, a);
    tc::fence_after_sync();
    const bool nan = *(volatile int*)&sm.err || *(volatile int*)&sm.bad;
    if (nan && tid == 0) latch_error(a.counters, kDevErrBounds);
    if (tid < NC) {
      ml[2 * tid] = nan ? 0.f : -sm.nm[tid];
      ml[2 * tid + 1] =
          nan ? __int_as_float(0x7fc00000) : sm.lsum[0][tid] + sm.lsum[1][tid] + sm.lsum[2][tid] + sm.lsum[3][tid];
    }
    float* o = a.part + (unit * a.parts + part) * NC * kD + tid;
#pragma unroll 1
    for (int x = 0; x < NC; x += 16) {
      uint32_t v[16];
      load_cols(tmem + lane_base + x, v);
#pragma unroll
      for (int y = 0; y < 16; ++y) o[(x + y) * kD] = __uint_as_float(v[y]) * exp2f(sm.mp[x + y] + sm.nm[x + y]);
    }
    tc::fence_before_sync();
  }
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 12) tc::tmem_dealloc(tmem, kTmemCols);
}

// One warp per output row: the parts joined by their references and sums, the
// compressed tokens' share rotated back.  Bound by the parts' reads from L2.
template <int NC>
__global__ void __launch_bounds__(256) tree_tc_merge_kernel(TreeArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int Hq = a.H * a.G;
  if (i >= (int64_t)a.batch * a.T * Hq) return;
  const int b = (int)(i / (a.T * Hq)), t = (int)(i / Hq % a.T), hq = (int)(i % Hq), h = hq / a.G;
  if (t >= tree_new(a, b)) return;
  const int r = t * a.G + hq % a.G;
  const int64_t unit = ((int64_t)b * a.H + h) * a.n_blk + r / NC;
  const float2* ml = reinterpret_cast<const float2*>(a.ml) + unit * a.parts * NC + r % NC;
  const float* o = a.part + (unit * a.parts * NC + r % NC) * kD + lane * 4;
  float m = -INFINITY;
  for (int s = lane; s < a.parts; s += 32) m = fmaxf(m, ml[(int64_t)s * NC].x);
  m = warp_max(m);
  float l = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = 0; s < a.parts; ++s) {
    const float2 e = ml[(int64_t)s * NC];
    if (e.y == 0.f) continue;
    const float w = exp2f(e.x - m);
    const float4 v = *reinterpret_cast<const float4*>(o + (int64_t)s * NC * kD);
    l = fmaf(w, e.y, l);
    float* z = s < a.tail_parts ? y : x;
    z[0] = fmaf(w, v.x, z[0]);
    z[1] = fmaf(w, v.y, z[1]);
    z[2] = fmaf(w, v.z, z[2]);
    z[3] = fmaf(w, v.w, z[3]);
  }
  if (!a.naive && a.comp) {
    fwht128(x);
    const float n = rsqrtf((float)kD);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int d = 4 * lane + e;
      x[e] *= (a.sign_bits[d >> 5] >> (d & 31)) & 1u ? -n : n;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = (x[e] + y[e]) * inv;
  // infinities and NaN of the drafts' values, for the rows that see them
  unsigned long long odd = a.inf_v[(int64_t)b * a.H + h] & tree_mask(a, b, t);
  while (odd) {
    const int d = __ffsll((long long)odd) - 1;
    odd &= odd - 1;
    float v[4];
    load4<__nv_bfloat16>(reinterpret_cast<const __nv_bfloat16*>(a.vn) + b * a.n_seq + d * a.n_tok + h * kD + lane * 4, v);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (!isfinite(v[e])) x[e] += v[e];
  }
  // the one rounding to the output's type
  const __nv_bfloat162 lo = __floats2bfloat162_rn(x[0], x[1]), hi = __floats2bfloat162_rn(x[2], x[3]);
  reinterpret_cast<uint2*>(a.out)[i * 32 + lane] =
      make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

template <typename K>
int launch_dependent(K kernel, dim3 grid, int threads, int smem, const TreeArgs& a, cudaStream_t s) {
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
  return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? ANCHORKV_OK : ANCHORKV_ECUDA;
}

constexpr int kSmem = (int)sizeof(Sm) + 1024;
static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");

template <int NC>
int launch_nc(const TreeArgs& a, cudaStream_t s) {
  static std::mutex mu;
  static int ready_dev = -1;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ANCHORKV_ECUDA;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (ready_dev != dev) {
      if (cudaFuncSetAttribute(tree_tc_kernel<NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
        return ANCHORKV_ECUDA;
      ready_dev = dev;
    }
  }
  const int gx = a.comp ? std::max(1, std::min((a.k + 7) / 8, 256)) : 1;
  tree_prep_kernel<<<dim3(gx, 2 * a.H, a.batch), 256, 0, s>>>(a);
  if (cudaGetLastError() != cudaSuccess) return ANCHORKV_ECUDA;
  int st = launch_dependent(tree_tc_kernel<NC>, dim3(a.parts, a.n_blk, a.batch * a.H), kThreads, kSmem, a, s);
  if (st) return st;
  const int64_t rows = (int64_t)a.batch * a.T * a.H * a.G;
  return launch_dependent(tree_tc_merge_kernel<NC>, dim3((unsigned)((rows + 7) / 8)), 256, 0, a, s);
}

}  // namespace

void tree_plan_tc(const Plan& pl, bool prefix, TreePlan* tp) {
  tp->RB = tp->rows <= 16 ? 16 : tp->rows <= 32 ? 32 : 64;
  tp->n_blk = (tp->rows + tp->RB - 1) / tp->RB;
  const int64_t units = (int64_t)tp->batch * pl.H * tp->n_blk;
  const int64_t pre = prefix ? (pl.N + kTT - 1) / kTT : 0, tail = (tp->cap + tp->T + kTT - 1) / kTT;
  // One CTA an SM.  A CTA costs about kFixed tiles beside its own (set-up,
  // first reference, outputs), so the split is the one whose longest run of
  // CTAs on an SM is shortest.
  constexpr int64_t kFixed = 4;
  int64_t best = INT64_MAX;
  tp->parts = tp->tail_parts = 1;
  for (int64_t s = prefix ? 1 : 0; s <= std::min<int64_t>(pre, 148); ++s) {
    const int64_t per = s ? (pre + s - 1) / s : 8, t = (tail + std::max<int64_t>(per, 4) - 1) / std::max<int64_t>(per, 4);
    const int64_t waves = (units * (s + t) + 147) / 148, cost = waves * (per + kFixed);
    if (cost < best) {
      best = cost;
      tp->parts = (int)(s + t);
      tp->tail_parts = (int)t;
    }
  }
}

int launch_tree_tc(const TreeArgs& a, cudaStream_t s) {
  return a.RB == 16 ? launch_nc<16>(a, s) : a.RB == 32 ? launch_nc<32>(a, s) : launch_nc<64>(a, s);
}

}  // namespace akv
