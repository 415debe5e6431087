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
//   row_t = x^_t / w_t,    w_t = gamma_t M_a,
// is applied in fp32, to the logits for keys and to the probabilities for
// values; a residual's row is then its anchor's plus its levels times
// sigma_t / w_t.  (Where gamma_t M_a is below 2^-14 sigma_t, w_t is
// 2^-14 sigma_t: the row stays in range, and the anchor's share, wrong by at
// most twice that, is below the rounding of the row.)  Accumulators, logits
// and sums are fp32.
//
// One CTA owns 16, 32, 64 or 128 rows (draft, query head) of one (sequence, KV
// head) and a share of its tokens - the first parts compressed ones, the others
// exact ones, by the sequence's own lengths - in tiles of 128:
//   S^T [128 tokens x rows]  = K^ Q^T      A = key tile, B = queries
//   O^T [128 coords x rows] += V^T P       A = value tile (token-major), B = P
// Tokens are on the accumulator's lanes, so a thread owns a token: its scales
// are scalars, its row of P is contiguous, and the cost of the softmax goes
// with the rows there are (16, 32, 64 or 128 columns) instead of a padded 128.
//   8 or 16 softmax warps: logits from tensor memory, exponentials, P to shared
//     memory; at the end the outputs
//   one warp issues the logits' MMAs, one the outputs', so that the keys of a
//     tile need not wait for the values of the one before
//   two warps load token tables and codes ahead (bulk copies)
//   16 or 8 producer warps fill key and value tiles, 32 rows each: anchor rows
//     by 16-byte asynchronous copies into the 128-byte swizzle, residual rows
//     finished in place (eight lanes each)
// The maximum over tokens would need a reduction across lanes for every row
// and tile.  Instead each row keeps two power-of-two references, one for the
// sum of p and one for w p (the fp16 operand), which move only when a tile
// would leave their range: one vote per tile.  Powers of two make every
// rescaling exact, so the result does not depend on when it happens.
//
// Bound by instruction issue and the latency of the chain copy - residuals -
// logits - softmax - outputs, not by memory or the tensor pipe.  For 16 rows a
// tile costs about 4.6 k warp instructions (softmax 1 k, residual rows 1 k,
// the rest copies and waits) and 2.2 k cycles; the anchor rows then come from
// L2 at 6.5 TB/s (64 KB a tile).  For 128 rows it is the softmax: 16 warps, 11 k
// warp instructions and 5 k cycles a tile, 55% of the issue slots.
// Whole calls (CUDA graph, 8 KV heads, theta = 0.05), with the rate of
// 4 D operations a row and token:
//   32 k tokens, 32 query heads: 1 draft 36.1 us (198 GB/s of the layout: three
//     fifths are the pre-kernels, the first tile and the merge), 16 drafts
//     47.3 us (184 TFLOP/s), 64 drafts 123.7 us (286 TFLOP/s)
//   128 k tokens, 64 query heads, 24 drafts: 315 us (329 TFLOP/s)
//   16 sequences of 32 k tokens, theta = 0.1, 8 drafts: 480 us (526 GB/s)
// Anchor rows by four-row TMA gathers were no faster than 16-byte copies (60.4
// us against 59.8 on 16 drafts then: about 100 cycles of issue a gather);
// finding the residuals' levels before the rows have landed was slower (36.5 ->
// 39 us on one draft): the registers and second pass cost more than the wait.

#include <limits.h>
#include <stddef.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "tc_util.cuh"
#include "tree.h"
#include "tree_merge.cuh"

namespace akv {
namespace {

constexpr int kTT = 128;                  // tokens of a tile
constexpr int kSt = 2;                    // stages of the key and value rings
constexpr int kTileBytes = kTT * kD * 2;
constexpr int kHalf = kTileBytes / 2;     // 64 coordinates of every row
constexpr float kLog2e = 1.4426950408889634f;
// P is fp16: w p over its reference, between 2^-24 (the smallest step) and 2^15.
// A token's rounding is at most 2^-25, but of n tokens behind one that takes
// nearly all (a prompt's first, as a rule) all may round the same way, and the
// sum of p keeps what the outputs lose.  So a new reference puts the largest
// |w p| at 2^-t / 2 or above, t = 13 - log2 n for the n tokens of the part: the
// loss of all of them, n 2^-25, is then at most 2^-11 of that largest
// contribution, one rounding of an operand.  What is left up to 2^15 is
// headroom: a tile that passes it pays for new references, so it goes with the
// part (17 bits for 2 k tokens, 13 for 32 k).  Against 20 bits for
// every part, which lost 1.6% of the output behind a first token 14 nats above
// 32 k others and 5% of 128 k (graph, us; q scaled by 1 and 8): one draft 34.4,
// 42.6 -> 34.8, 42.6; 64 drafts 116.4, 192 -> 122.5, 199; batch 16 475, 535 ->
// 478, 552.  With 2^8 for every part: 38.9, 46.5; 156, 216; 500, 577.
constexpr float kPLimit = 32768.f;        // fp16 holds 65504
constexpr int kPBits = 13, kPMost = 5;    // t, at most
__device__ __forceinline__ float p_target(int tiles) {
  return (float)min(kPMost, kPBits - 7 - (32 - __clz(tiles - 1)));   // 2^7 tokens a tile
}
constexpr float kSumLimit = 1.0995116e12f;  // 2^40, far below fp32's range
// The sum's reference of a row that has met no logit: finite, so that a logit of
// -inf beside it is still -inf and any other far above every limit.
constexpr float kNoRef = -3.402823466e38f;
constexpr float kRefGap = 120.f;          // the references' largest distance, either way
// A part's sum is handed to the merge between 2^-12 and 2^-11 (logits beyond 2^23
// aside), and its outputs in the same unit: 2^11 parts of the largest finite values add up to a finite
// number, and a bf16 output keeps its bits down to the smallest normal one.
constexpr int kSumBits = 11;

// What a tile of one side needs beside rows and codes, written by the
// pre-kernel: per token its scale and its anchor slot; per residual record the
// factor of its levels (fp16) and its token; `quarter`: byte q counts the
// records before quarter q.
struct Table {
  uint16_t slot[kTT];
  uint16_t level[kTT];
  uint8_t tok[kTT];
  uint32_t quarter, n_rec, first, pad;
};
struct Meta {
  float scale[kTT];
  Table table;
};
static_assert(sizeof(Table) % 16 == 0 && offsetof(Table, quarter) % 16 == 0 && offsetof(Meta, table) % 16 == 0, "copied in 16-byte pieces");

// What goes with NC, the rows (columns of the accumulators) of a CTA.
template <int NC>
struct Shape {
  // Softmax groups of four warps have CW of the rows each and, where PG is 2,
  // every other tile.  Sixteen rows a group were faster than 32 (16 drafts x 4
  // heads behind 32 k tokens: 52.7 us, 60.4 with 32 rows and two parities)
  // wherever the warps suffice.
  static constexpr int CW = NC == 128 ? 32 : 16, CG = NC / CW, PG = NC == 16 ? 2 : 1, kGroups = CG * PG;
  // Warps: softmax, one that issues the logits' MMAs and one the outputs', a
  // loader of token tables for each side, producers.
  static constexpr int kProd = NC <= 32 ? 16 : 8;
  static constexpr int kMma = 4 * kGroups, kLoad = kMma + 2, kFirstProd = kMma + 4, kThreads = 32 * (kFirstProd + kProd);
  // Tensor memory: outputs (of each parity), then two buffers of logits.
  static constexpr int kOCols = NC < 64 ? 64 : NC, kSCol = PG * kOCols, kTmemCols = NC == 128 ? 512 : 256;
  // Shared memory: buffers of P in blocks of 64 rows; token tables, loaded
  // kMetaSl tiles ahead when the tile whose place they take has been
  // multiplied, with value scales; key scales, which are read up to two tiles
  // after that; codes, one tile less ahead (they come from HBM).
  static constexpr int kPBuf = NC == 128 ? 1 : 2, kPBytes = kTT * 2 * kOCols;
  static constexpr int kMetaSl = NC == 128 ? 3 : 4, kVSl = kMetaSl, kKSl = kMetaSl + 2, kCodeSl = kMetaSl - 1;
};

template <int NC>
struct Sm {
  using S = Shape<NC>;
  static constexpr int kRows = S::kOCols;
  uint8_t K[kSt][kTileBytes];
  uint8_t V[kSt][kTileBytes];
  uint8_t P[S::kPBuf][S::kPBytes];        // [64 rows][token][row] fp16, swizzled
  uint8_t Q[NC * kD * 2];
  alignas(16) uint8_t codes[2][S::kCodeSl][kTT * kCodeBytes];     // [side]
  alignas(16) Table meta[2][S::kMetaSl];  // [side]
  alignas(16) float rk[S::kKSl][kTT];     // key scales
  alignas(16) float wv[S::kVSl][kTT];     // value scales
  alignas(64) uint32_t lut[16];           // two codes -> their levels in fp16
  alignas(16) float cs[kRows];            // per row: logit scale
  // per row and tile parity: -reference of the sum, 2^(reference of the sum -
  // that of w p), reference of w p
  alignas(16) float nm[S::PG][kRows], cw[S::PG][kRows], mp[S::PG][kRows];
  float fl[S::PG][kRows];                 // rescaling of the sums
  int red[S::kGroups][2][4][16];          // maxima; factors of the outputs
  float lsum[S::PG][4][kRows];
  uint2 seen[kTreeMaxDrafts];             // of each draft, the drafts that see it
  unsigned char colt[kRows];              // draft of each row
  uint64_t full[2][2], kempty[2], pv[2], sfull[2], sempty[2], pfull[2], sk[S::kKSl], sv[S::kVSl];   // full: [side][stage]
  uint64_t loaded[2][S::kMetaSl], coded[2][S::kCodeSl];     // token tables, codes
  // their places are free: a barrier each.  kempty and pv, which the tile after
  // next uses again, would not do: it may be done before a late loader looks, and
  // the parity would say "not yet" until a tile that waits for the loader.
  uint64_t freed[2][S::kMetaSl];
  uint32_t tmem;
  float target;                           // t of new references
  int err, bad, rep;
};
template <int NC>
constexpr bool sm_aligned() {
  return offsetof(Sm<NC>, cs) % 16 == 0 && offsetof(Sm<NC>, nm) % 16 == 0 && offsetof(Sm<NC>, cw) % 16 == 0 &&
         offsetof(Sm<NC>, codes) % 16 == 0 && offsetof(Sm<NC>, meta) % 16 == 0 && offsetof(Sm<NC>, V) % 1024 == 0 &&
         offsetof(Sm<NC>, lut) % 64 == 0 && offsetof(Sm<NC>, P) % 1024 == 0 && offsetof(Sm<NC>, Q) % 1024 == 0;
}
static_assert(sm_aligned<16>() && sm_aligned<32>() && sm_aligned<64>() && sm_aligned<128>(), "16-byte reads, swizzle atoms");

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// `bytes` (a multiple of 16) between 16-byte aligned addresses.
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Power of two at or below |x| for the largest magnitude's bits (fp32), kept
// where its inverse is a normal number too.
__device__ __forceinline__ int scale_exp(uint32_t bits) { return min(max((int)(bits >> 23), 1), 253); }
__device__ __forceinline__ float exp_to_f(int e) { return __uint_as_float((uint32_t)e << 23); }       // 2^(e - 127)
// 2^d of a whole number d, 0 below fp32's normal range.
__device__ __forceinline__ float pow2(float d) {
  return d < -126.f ? 0.f : __int_as_float(((int)fminf(d, 128.f) + 127) << 23);
}
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

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
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

// The eight MMAs (K = 16 each) of one product of fp16 operands, issued by one
// elected lane of a converged warp.  Elected
// inside, so that the warp does not diverge and the descriptors stay in uniform
// registers.  A0, A1, B0, B1: descriptor steps, in 16-byte units, from one MMA
// to the next and from the fourth to the fifth.
template <int A0, int A1, int B0, int B1>
__device__ __forceinline__ void mma_tile(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q, r;\n\t.reg .b64 x, y;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "setp.ne.b32 q, %4, 0;\n\tsetp.eq.b32 r, 0, 0;\n\t"
      "mov.b64 x, %1;\n\tmov.b64 y, %2;\n\t"
      "@p tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, q;\n\t"
      "add.u64 x, x, %5;\n\tadd.u64 y, y, %7;\n\t"
      "@p tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, r;\n\t"
      "add.u64 x, x, %5;\n\tadd.u64 y, y, %7;\n\t"
      "@p tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, r;\n\t"
      "add.u64 x, x, %5;\n\tadd.u64 y, y, %7;\n\t"
      "@p tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, r;\n\t"
      "add.u64 x, x, %6;\n\tadd.u64 y, y, %8;\n\t"
      "@p tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, r;\n\t"
      "add.u64 x, x, %5;\n\tadd.u64 y, y, %7;\n\t"
      "@p tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, r;\n\t"
      "add.u64 x, x, %5;\n\tadd.u64 y, y, %7;\n\t"
      "@p tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, r;\n\t"
      "add.u64 x, x, %5;\n\tadd.u64 y, y, %7;\n\t"
      "@p tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, r;\n\t"
      "}"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "n"(A0), "n"(A1), "n"(B0), "n"(B1)
      : "memory");
}
// The arrival on `bar` when they are done, by the same lane (the election of a
// full warp is deterministic).
__device__ __forceinline__ void commit_elected(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\t"
      "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
      ::"r"(tc::smem_u32(bar))
      : "memory");
}

// The Hadamard transform of fwht128 with one multiply-add a butterfly.
__device__ __forceinline__ void fwht128_signed(float (&v)[4], int lane) {
  const float a0 = v[0] + v[1], a1 = v[0] - v[1], a2 = v[2] + v[3], a3 = v[2] - v[3];
  v[0] = a0 + a2; v[2] = a0 - a2; v[1] = a1 + a3; v[3] = a1 - a3;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const float s = lane & m ? -1.f : 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fmaf(v[i], s, __shfl_xor_sync(0xffffffffu, v[i], m));
  }
}

// First sequence with the layout of sequence b: it holds the rotated anchors.
// By a whole warp.
__device__ __forceinline__ int first_with_layout(const TreeArgs& a, int b) {
  if (!a.layout_of) return b;
  const int mine = a.layout_of[b], lane = threadIdx.x & 31;
  for (int i = 0; i < b; i += 32) {
    const uint32_t same = __ballot_sync(0xffffffffu, i + lane < b && a.layout_of[i + lane] == mine);
    if (same) return i + __ffs((int)same) - 1;
  }
  return b;
}

// Bits 0..3: the signs that the rotation flips of this lane's four coordinates.
__device__ __forceinline__ uint32_t flipped(const TreeArgs& a, int lane) {
  const uint32_t lo = lane & 8 ? a.sign_bits[1] : a.sign_bits[0], hi = lane & 8 ? a.sign_bits[3] : a.sign_bits[2];
  return (lane & 16 ? hi : lo) >> ((4 * lane) & 31) & 15u;
}
__device__ __forceinline__ void flip(float (&v)[4], uint32_t bits) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(__float_as_uint(v[i]) ^ ((bits << (31 - i)) & 0x80000000u));
}

// Rotated anchors of every layout in use, one warp per row: fp16 rows over a
// power of two and that power (1/sqrt(D) of the rotation in it).  Clears the
// status words and the flags of infinite values.  Bound by launch latency for
// one sequence (4.6 k rows of a 32 k-token prompt, 1.2 MB read: 2.5 us inside
// the call); for many by instruction issue, about 140 a row (16 sequences: 16 us).
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
  const uint32_t signs = flipped(a, lane);
  const float unit = a.naive ? 1.f : rsqrtf((float)kD);
  for (int s = (blockIdx.x * 8 + warp) * 2; s < a.k; s += gridDim.x * 16) {
    const int s1 = min(s + 1, a.k - 1);                  // two rows' latencies together
    float v[2][4];
    load4<__nv_bfloat16>(src + (int64_t)s * kD + lane * 4, v[0]);
    load4<__nv_bfloat16>(src + (int64_t)s1 * kD + lane * 4, v[1]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!a.naive) {
        flip(v[k], signs);
        fwht128_signed(v[k], lane);
      }
      const float m = warp_max(fmaxf(fmaxf(fabsf(v[k][0]), fabsf(v[k][1])), fmaxf(fabsf(v[k][2]), fabsf(v[k][3]))));
      const int e = scale_exp(__float_as_uint(m)), row = k ? s1 : s;
      const float inv = exp_to_inv(e);
      reinterpret_cast<uint2*>(a.anc)[(row0 + row) * 32 + lane] =
          make_uint2(pack_half2(v[k][0] * inv, v[k][1] * inv), pack_half2(v[k][2] * inv, v[k][3] * inv));
      if (lane == 0) a.anc_scale[row0 + row] = exp_to_f(e) * unit;
    }
  }
}

// Token tables of every layout in use, one warp per tile of a side and head,
// after the anchors' scales.  A lane has a token of each quarter, so that what a
// tile's records have in common is found once (four warps a tile and a quarter
// each took 279 instructions a quarter; four tokens in a row a lane was no
// shorter and its stores diverge, 41 us against 36).  Bound by latency for one
// sequence (3.4 us after the anchors' scales), by issue for many, 400
// instructions a tile (16 sequences, 65 k tiles: 36 us).
__global__ void __launch_bounds__(256) tree_meta_kernel(TreeArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, b = blockIdx.z, sh = blockIdx.y, tile = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lay = tree_layout(a, b);
  if (tile >= a.n_tiles || lay < 0 || first_with_layout(a, b) != b) {
    asm volatile("griddepcontrol.wait;" ::: "memory");   // this kernel is over after the one before it
    return;
  }
  const uint8_t* comp = a.comp + (int64_t)lay * a.stride;
  const int64_t tile_sh = (int64_t)sh * a.n_tiles + tile;
  const uint4 bm = *reinterpret_cast<const uint4*>(comp + a.off_bm + tile_sh * 16);
  const int first = reinterpret_cast<const int*>(comp + a.off_pf)[tile_sh + sh];
  const int left = a.N - tile * kTT;
  const uint32_t* words = reinterpret_cast<const uint32_t*>(comp + a.off_tok) + (int64_t)sh * a.N + tile * kTT + lane;
  uint32_t word[4], bits[4] = {bm.x, bm.y, bm.z, bm.w};
  int before[5] = {0};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    word[q] = q * 32 + lane < left ? words[q * 32] : 0u;
    // bits behind the last token mean nothing
    if (left < 32 * q + 32) bits[q] &= left > 32 * q ? (1u << (left - 32 * q)) - 1u : 0u;
    before[q + 1] = before[q] + __popc(bits[q]);
  }
  const bool fine = first >= 0 && first + (int64_t)before[4] <= a.R;   // records outside the layout are none
  const uint16_t* sig = reinterpret_cast<const uint16_t*>(comp + a.off_sig) + first;
  const uint32_t below = (1u << lane) - 1u;
  uint16_t sigma[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (!fine) bits[q] = 0u;
    sigma[q] = (bits[q] >> lane) & 1u ? sig[before[q] + __popc(bits[q] & below)] : (uint16_t)0;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const float* scale = a.anc_scale + ((int64_t)b * 2 * a.H + sh) * a.k;
  Meta& o = reinterpret_cast<Meta*>(a.meta)[(int64_t)b * 2 * a.H * a.n_tiles + tile_sh];
  float m[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int slot = min((int)(word[q] & 0xffffu), a.k - 1);
    m[q] = scale[slot];
    o.table.slot[q * 32 + lane] = (uint16_t)slot;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float c1 = half_bits_to_f(word[q] >> 16) * m[q];             // 0 behind the last token, whose word is 0
    const float sg = half_bits_to_f(sigma[q]);
    const bool tiny = sg > fabsf(c1) * 16384.f;
    o.scale[q * 32 + lane] = tiny ? sg * (1.f / 16384.f) : c1;
    if ((bits[q] >> lane) & 1u) {
      const int x = before[q] + __popc(bits[q] & below);
      o.table.level[x] = __half_as_ushort(__float2half_rn(tiny ? 16384.f : c1 != 0.f ? __fdividef(sg, c1) : 0.f));
      o.table.tok[x] = (uint8_t)(q * 32 + lane);
    }
  }
  if (lane == 0)
    *reinterpret_cast<uint4*>(&o.table.quarter) =
        fine ? make_uint4((uint32_t)before[1] << 8 | (uint32_t)before[2] << 16 | (uint32_t)before[3] << 24, (uint32_t)before[4],
                          (uint32_t)first, 0u)
             : make_uint4(0u, 0u, 0u, 0u);
}

// Waits for a phase.  A phase that is over already, the usual case in a full
// pipeline, costs one test; the bounded wait is out of the way of that path.
__device__ __noinline__ void wait_slow(uint64_t* bar, uint32_t parity, int* err, int* counters) {
  if (*(volatile int*)err) return;
  tc::wait_or_fail(bar, parity, err, counters, kDevErrTimeout);
}
template <typename M>
__device__ __forceinline__ void wait_b(M& sm, uint64_t* bar, uint32_t parity, const TreeArgs& a) {
  if (!tc::mbar_done(bar, parity)) wait_slow(bar, parity, &sm.err, a.counters);
}

__device__ __forceinline__ uint32_t swz(int row, int chunk) {   // byte offset of a row's 16-byte piece in a tile
  return (uint32_t)((chunk >> 3) * kHalf + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}

// A producer warp fills one quarter (32 rows) of the tiles of one side: warp w
// has side (w >> 2) & 1, quarter w & 3 and the tiles w >> 3, + step, ...
struct Lane {
  int side, q, first, step;
};
template <int kProd>
__device__ __forceinline__ Lane lane_of(int w) {
  return Lane{(w >> 2) & 1, w & 3, w >> 3, kProd / 8};
}

// The stage of tile t is free: the products that read it last are done (keys:
// the logits, values: the outputs).
template <typename M>
__device__ __forceinline__ void wait_free(M& sm, int side, int t, const TreeArgs& a) {
  if (t >= 2) wait_b(sm, side ? &sm.pv[t & 1] : &sm.kempty[t & 1], ((t >> 1) - 1) & 1, a);
}

template <typename M>
__device__ __forceinline__ float* scales_of(M& sm, int side, int t) {
  return side ? sm.wv[t % M::S::kVSl] : sm.rk[t % M::S::kKSl];
}
template <typename M>
__device__ __forceinline__ uint64_t* scales_bar(M& sm, int side, int t) {
  return side ? &sm.sv[t % M::S::kVSl] : &sm.sk[t % M::S::kKSl];
}

// x + factor times the levels at shared address `at`, two coordinates.
__device__ __forceinline__ uint32_t add_levels(uint32_t x, uint32_t factor, uint32_t at) {
  uint32_t lev;
  asm("ld.shared.b32 %0, [%1];" : "=r"(lev) : "r"(at));
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&factor), *reinterpret_cast<const __half2*>(&lev),
                            *reinterpret_cast<const __half2*>(&x));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Token tables and codes of one side, by one lane, as far ahead as there are
// places: a place is free when the tile that had it has been multiplied.
template <typename M>
__device__ void load_side(const TreeArgs& a, M& sm, int side, int n, const uint8_t* comp, const Meta* meta) {
  constexpr int kMetaSl = M::S::kMetaSl, kCodeSl = M::S::kCodeSl;
  const uint8_t* codes = comp + a.off_codes;
  for (int t = 0; t <= n; ++t) {
    const int before = t - kMetaSl;
    if (before >= 0) wait_b(sm, &sm.freed[side][before % kMetaSl], (before / kMetaSl) & 1, a);
    if (t < n) {
      uint64_t* mb = &sm.loaded[side][t % kMetaSl];
      tc::mbar_expect_tx(mb, sizeof(Table));
      bulk_copy(tc::smem_u32(&sm.meta[side][t % kMetaSl]), &meta[t].table, sizeof(Table), tc::smem_u32(mb));
      uint64_t* sb = scales_bar(sm, side, t);
      tc::mbar_expect_tx(sb, kTT * 4);
      bulk_copy(tc::smem_u32(scales_of(sm, side, t)), meta[t].scale, kTT * 4, tc::smem_u32(sb));
    }
    const int c = t - 1;                                           // takes the place of the codes of tile `before`
    if (c >= 0) {
      wait_b(sm, &sm.loaded[side][c % kMetaSl], (c / kMetaSl) & 1, a);
      const Table* m = &sm.meta[side][c % kMetaSl];
      const uint32_t bytes = min(m->n_rec, (uint32_t)kTT) * kCodeBytes;
      uint64_t* cb = &sm.coded[side][c % kCodeSl];
      tc::mbar_expect_tx(cb, bytes);
      if (bytes) bulk_copy(tc::smem_u32(sm.codes[side][c % kCodeSl]), codes + (int64_t)m->first * kCodeBytes, bytes, tc::smem_u32(cb));
    }
  }
  // the copies are over before this CTA's shared memory is, also after a failure
  for (int t = max(0, n - kMetaSl); t < n; ++t) {
    tc::mbar_wait(&sm.loaded[side][t % kMetaSl], (t / kMetaSl) & 1);
    tc::mbar_wait(scales_bar(sm, side, t), (t / (side ? M::S::kVSl : M::S::kKSl)) & 1);
  }
  for (int t = max(0, n - kCodeSl); t < n; ++t) tc::mbar_wait(&sm.coded[side][t % kCodeSl], (t / kCodeSl) & 1);
}

template <typename M>
__device__ void produce_prefix(const TreeArgs& a, M& sm, int w, int n, const uint8_t* rows) {
  constexpr int kMetaSl = M::S::kMetaSl, kCodeSl = M::S::kCodeSl;
  const Lane me = lane_of<M::S::kProd>(w);
  const int lane = threadIdx.x & 31, c = lane & 15, hw = lane >> 4, c8 = lane & 7, g = lane >> 3;
  rows += c * 16;
  const uint32_t lut = tc::smem_u32(sm.lut);             // 64-byte aligned
  for (int t = me.first; t < n; t += me.step) {
    wait_b(sm, &sm.loaded[me.side][t % kMetaSl], (t / kMetaSl) & 1, a);
    const Table* m = &sm.meta[me.side][t % kMetaSl];
    // anchor rows, sixteen lanes each: the first half of the quarter by the
    // first half of the warp
    const uint4 sa = *reinterpret_cast<const uint4*>(&m->slot[me.q * 32 + hw * 16]);
    const uint4 sb = *reinterpret_cast<const uint4*>(&m->slot[me.q * 32 + hw * 16 + 8]);
    const uint32_t slots[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
    wait_free(sm, me.side, t, a);
    uint8_t* tile = me.side ? sm.V[t & 1] : sm.K[t & 1];
    const uint32_t base = tc::smem_u32(tile) + (c >> 3) * kHalf + (me.q * 32 + hw * 16) * 128;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      // 256 bytes a row: the slot's two bytes one byte up
      const uint32_t o = __byte_perm(slots[k / 2], 0u, k & 1 ? 0x4324u : 0x4104u);
      cp_async16(base + k * 128 + ((c8 ^ (k & 7)) << 4), rows + o);
    }
    cp_commit();
    const int x0 = (m->quarter >> (8 * me.q)) & 255, x1 = me.q < 3 ? (m->quarter >> (8 * me.q + 8)) & 255 : m->n_rec;
    wait_b(sm, &sm.coded[me.side][t % kCodeSl], (t / kCodeSl) & 1, a);
    const uint8_t* cd = sm.codes[me.side][t % kCodeSl] + c8 * 2;
    cp_wait();
    __syncwarp();                                                  // the whole warp's copies have landed
    // residual rows in place: eight records at a time, eight lanes each for two
    // of them, two 16-byte pieces a lane; all reads before the writes
    for (int x = x0 + g; x < x1; x += 8) {
      const bool two = x + 4 < x1;
      uint8_t* row[2];
      uint32_t code[2][2], lv[2];
      uint4 v[2][2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int y = k && two ? x + 4 : x;
        const uint32_t tk = m->tok[y], f = m->level[y];
        lv[k] = __byte_perm(f, 0u, 0x1010u);
        row[k] = tile + tk * 128 + ((c8 ^ (tk & 7u)) << 4);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          code[k][p] = *reinterpret_cast<const uint16_t*>(cd + y * kCodeBytes + p * 16);
          v[k][p] = *reinterpret_cast<const uint4*>(row[k] + p * kHalf);
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (k && !two) break;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const uint32_t c = code[k][p] << 2;            // two codes' table entry: four bits of c at 4 z + 2
          v[k][p].x = add_levels(v[k][p].x, lv[k], lut | (c & 60u));
          v[k][p].y = add_levels(v[k][p].y, lv[k], lut | ((c >> 4) & 60u));
          v[k][p].z = add_levels(v[k][p].z, lv[k], lut | ((c >> 8) & 60u));
          v[k][p].w = add_levels(v[k][p].w, lv[k], lut | ((c >> 12) & 60u));
          *reinterpret_cast<uint4*>(row[k] + p * kHalf) = v[k][p];
        }
      }
    }
    tc::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&sm.full[me.side][t & 1]);
  }
}

// Exact rows, of pages and drafts: half a warp per row, the rows' addresses
// found by one lane each beforehand.
template <typename M>
__device__ void produce_tail(const TreeArgs& a, M& sm, int w, int n, int b, int h, int tile0, int len, int n_new) {
  const Lane me = lane_of<M::S::kProd>(w);
  const int lane = threadIdx.x & 31, c = lane & 15, hw = lane >> 4;
  const uint16_t* pool = reinterpret_cast<const uint16_t*>(me.side ? a.vp : a.kp);
  const uint16_t* fresh = reinterpret_cast<const uint16_t*>(me.side ? a.vn : a.kn);
  const int* table = a.table + (int64_t)b * a.maxp;
  for (int tl = me.first; tl < n; tl += me.step) {
    const int first = (tile0 + tl) * kTT + me.q * 32;              // this warp's first token
    unsigned long long at = 0;                                     // lane l: row of token first + l, or none
    {
      const int t = first + lane;
      if (t < len) {
        const int pg = table[t / a.P];
        if (pg >= 0 && pg < a.n_pages)
          at = (unsigned long long)(pool + (((int64_t)pg * a.H + h) * a.P + t % a.P) * kD);
        else
          *(volatile int*)&sm.bad = 1;
      } else if (t - len < n_new) {
        at = (unsigned long long)(fresh + b * a.n_seq + (int64_t)(t - len) * a.n_tok + h * kD);
      }
    }
    wait_free(sm, me.side, tl, a);
    uint8_t* tile = me.side ? sm.V[tl & 1] : sm.K[tl & 1];
    float* scales = scales_of(sm, me.side, tl) + me.q * 32;
#pragma unroll 1
    for (int r0 = 0; r0 < 32; r0 += 8) {                           // this half's rows r0 + 2 k + hw
      uint4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const unsigned long long p = __shfl_sync(0xffffffffu, at, r0 + 2 * k + hw);
        v[k] = p ? reinterpret_cast<const uint4*>(p)[c] : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = r0 + 2 * k + hw;
        uint32_t* vw = reinterpret_cast<uint32_t*>(&v[k]);
        uint32_t m2 = 0;                                           // magnitudes as 15-bit integers, two at a time
#pragma unroll
        for (int y = 0; y < 4; ++y) m2 = __vmaxu2(m2, vw[y] & 0x7fff7fffu);
        uint32_t m = max(m2 & 0xffffu, m2 >> 16);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (m >= 0x7f80u) {
          // infinities or NaN: the scale is of the finite ones.  In a draft's
          // value they must not reach the rows that do not see it (0 x inf):
          // the merge adds them where they are seen.
          const bool hide = me.side && first + r >= len;
          m = 0;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const uint32_t lo = vw[y] & 0x7fffu, hi = (vw[y] >> 16) & 0x7fffu;
            if (lo < 0x7f80u) m = max(m, lo);
            else if (hide) vw[y] &= 0xffff0000u;
            if (hi < 0x7f80u) m = max(m, hi);
            else if (hide) vw[y] &= 0xffffu;
          }
          const uint32_t half = 0xffffu << (16 * hw);
#pragma unroll
          for (int o = 1; o < 16; o <<= 1) m = max(m, __shfl_xor_sync(half, m, o));
          if (hide && c == 0) atomicOr(&a.inf_v[(int64_t)b * a.H + h], 1ull << (first + r - len));
        }
        const int e = scale_exp(m << 16);
        const float inv = exp_to_inv(e);
        uint32_t out[4];
#pragma unroll
        for (int y = 0; y < 4; ++y)
          out[y] = pack_half2(__uint_as_float(vw[y] << 16) * inv, __uint_as_float(vw[y] & 0xffff0000u) * inv);
        *reinterpret_cast<uint4*>(tile + swz(me.q * 32 + r, c)) = make_uint4(out[0], out[1], out[2], out[3]);
        if (c == 0) scales[r] = m ? exp_to_f(e) : (me.side ? 0.f : 1.f);
      }
    }
    tc::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tc::mbar_arrive(scales_bar(sm, me.side, tl));
      tc::mbar_arrive(&sm.full[me.side][tl & 1]);
    }
  }
}

// 16 columns of this warp's 32 accumulator lanes as floats.
__device__ __forceinline__ void load_cols(uint32_t taddr, uint32_t (&v)[16]) {
  tc::tmem_ld16(taddr, v);
  tc::tmem_wait_ld_dep(v);
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(taddr)
               : "memory");
}
// ... four columns, complete on return.
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t (&v)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];\n\ttcgen05.wait::ld.sync.aligned;"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_wait_ld8(uint32_t (&a)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]), "+r"(a[6]), "+r"(a[7])
               :
               : "memory");
}
// Bit x: the row of column x does not see this token.
__device__ __noinline__ uint32_t hidden_columns(unsigned long long vis, const unsigned char* colt) {
  uint32_t h = 0;
#pragma unroll 1
  for (int x = 0; x < 16; ++x) h |= (uint32_t)!((vis >> colt[x]) & 1ull) << x;
  return h;
}

// Sums over 16 lanes of 16 values a lane: lane l gets value l % 16 of its half.
__device__ __forceinline__ float sum16(const float2 (&p)[8], int lane) {
  float v[16];
#pragma unroll
  for (int x = 0; x < 16; ++x) v[x] = x & 1 ? p[x / 2].y : p[x / 2].x;
#pragma unroll
  for (int off = 8; off >= 1; off >>= 1) {
    const bool up = (lane & off) != 0;
#pragma unroll
    for (int x = 0; x < off; ++x) {
      const float keep = up ? v[x + off] : v[x], send = up ? v[x] : v[x + off];
      v[x] = keep + __shfl_xor_sync(0xffffffffu, send, off);
    }
  }
  return v[0];
}

// New references of rows c1 .. c1 + 15 for a softmax group whose last tile was
// `before` (negative: none): the maxima over the tile's tokens, the factor of the sums so far (fl), and the
// outputs so far in tensor memory.  Out of line and in loops: it runs once or
// twice, and its code should not push the tile loops out of the instruction
// caches.
template <typename M>
__device__ __noinline__ void new_references(M& sm, const TreeArgs& a, uint32_t scol, uint32_t ocol, int c1, int par, int grp,
                                            int before, int bar_id, float rk, float w, uint32_t hidden) {
  const int lane = threadIdx.x & 31, wq = (threadIdx.x >> 5) & 3, tok = threadIdx.x & 127;
  const float lw = w != 0.f ? __log2f(fabsf(w)) : -INFINITY;
#pragma unroll 1
  for (int x = 0; x < 16; x += 8) {
    uint32_t s[8];
    tmem_ld8(scol + x, s);
    tmem_wait_ld8(s);
#pragma unroll
    for (int y = 0; y < 8; ++y) {
      const int c = c1 + x + y;
      float lg = (hidden >> (x + y)) & 1u ? -INFINITY : __uint_as_float(s[y]) * (rk * sm.cs[c]);
      lg = fmaxf(lg, -INFINITY);                                   // a NaN is no maximum
      const int m1 = __reduce_max_sync(0xffffffffu, ordered(lg));
      const int m2 = __reduce_max_sync(0xffffffffu, ordered(lg + lw));
      if (lane == 0) {
        sm.red[grp][0][wq][x + y] = m1;
        sm.red[grp][1][wq][x + y] = m2;
      }
    }
  }
  tc::named_bar(bar_id, 128);
  float* factor = reinterpret_cast<float*>(sm.red[grp][0][0]);             // of the outputs, once the maxima are read
  if (tok < 16) {
    const int c = c1 + tok;
    const int(&r)[2][4][16] = sm.red[grp];
    const float m1 = unordered(max(max(r[0][0][tok], r[0][1][tok]), max(r[0][2][tok], r[0][3][tok])));
    const float m2 = unordered(max(max(r[1][0][tok], r[1][1][tok]), max(r[1][2][tok], r[1][3][tok])));
    const float l_old = -sm.nm[par][c], p_old = sm.mp[par][c];
    const float l_new = fmaxf(l_old, ceilf(m1));
    float p_new = fmaxf(p_old, ceilf(m2) + sm.target);
    if (l_new > kNoRef) p_new = fminf(fmaxf(p_new, l_new - kRefGap), l_new + kRefGap);   // cw is a normal number
    sm.fl[par][c] = l_old > kNoRef ? pow2(l_old - l_new) : 0.f;
    sm.nm[par][c] = -l_new;
    sm.mp[par][c] = p_new;
    sm.cw[par][c] = l_new > kNoRef ? pow2(l_new - p_new) : 1.f;
    __syncwarp(0xffffu);
    factor[tok] = p_old > -INFINITY ? pow2(p_old - p_new) : 0.f;
  }
  tc::named_bar(bar_id, 128);
  if (before >= 0) {
    wait_b(sm, &sm.pv[before & 1], (before >> 1) & 1, a);
    tc::fence_after_sync();
#pragma unroll 1
    for (int x = 0; x < 16; x += 8) {
      uint32_t o[8];
      tmem_ld8(ocol + x, o);
      tmem_wait_ld8(o);
#pragma unroll
      for (int y = 0; y < 8; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * factor[x + y]);
      tmem_st8(ocol + x, o);
    }
    tmem_wait_st();
  }
}

template <int NC>
__global__ void __launch_bounds__(Shape<NC>::kThreads, 1) tree_tc_kernel(TreeArgs a) {
  using S = Shape<NC>;
  constexpr int CW = S::CW, CH = CW / 16, CG = S::CG, PG = S::PG, kMma = S::kMma, kThreads = S::kThreads;
  constexpr int kOCols = S::kOCols, kSCol = S::kSCol, kKSl = S::kKSl, kVSl = S::kVSl;
  extern __shared__ __align__(1024) unsigned char raw[];
  Sm<NC>& sm = *reinterpret_cast<Sm<NC>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int blk = blockIdx.x, bh = blockIdx.y, part = blockIdx.z, b = bh / a.H, h = bh % a.H;
  const int64_t unit = (int64_t)bh * a.n_blk + blk;
  float* ml = a.ml + (unit * a.parts + part) * NC * 2;
  const int n_new = tree_new(a, b), rows = n_new * a.G;
  if (blk * NC >= rows) {                             // nobody reads these parts
    asm volatile("griddepcontrol.wait;" ::: "memory");   // this kernel is over after those before it
    return;
  }
  // this part's tiles: the first parts take the compressed tokens, the others the exact
  const int lay = a.comp ? tree_layout(a, b) : 0, len = tree_len(a, b), prefix_parts = a.parts - tree_tail_parts(a, len, n_new);
  const bool tail = part >= prefix_parts;
  const bool out_of_range = lay < 0 || len < 0;
  int tile0, n;
  {
    const int tiles = tail ? (max(len, 0) + n_new + kTT - 1) / kTT : a.n_tiles;
    const int s = tail ? part - prefix_parts : part, of = tail ? a.parts - prefix_parts : prefix_parts;
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
  if (warp == kMma) {
    tc::tmem_alloc(&sm.tmem, S::kTmemCols);
    tc::tmem_relinquish();
  }
  if (warp == 0) {
    // scales: one copy a tile, or four quarters of exact rows; softmax: one
    // arrival a warp
    if (lane < kKSl) tc::mbar_init(&sm.sk[lane], tail ? 4 : 1);
    if (lane < kVSl) tc::mbar_init(&sm.sv[lane], tail ? 4 : 1);
    if (lane < 2 * S::kMetaSl) {
      tc::mbar_init(&sm.loaded[0][0] + lane, 1);
      tc::mbar_init(&sm.freed[0][0] + lane, 1);
    }
    if (lane < 2 * S::kCodeSl) tc::mbar_init(&sm.coded[0][0] + lane, 1);
    if (lane < 4) tc::mbar_init(&sm.full[0][0] + lane, 4);
    if (lane < 2) {
      tc::mbar_init(&sm.kempty[lane], 1);
      tc::mbar_init(&sm.pv[lane], 1);
      tc::mbar_init(&sm.sfull[lane], 1);
      tc::mbar_init(&sm.sempty[lane], 4 * CG);
      tc::mbar_init(&sm.pfull[lane], 4 * CG);
    }
    if (lane == 0) {
      sm.target = p_target(n);
      sm.err = 0;
      sm.bad = 0;
    }
    tc::fence_barrier_init();
  }
  if (warp == 1) {
    const int rep = first_with_layout(a, b);
    if (lane == 0) sm.rep = rep;
  }
  if (tail && warp == 2) {                            // the masks' columns
    const unsigned long long lo = lane < n_new ? tree_mask(a, b, lane) : 0ull;
    const unsigned long long hi = lane + 32 < n_new ? tree_mask(a, b, lane + 32) : 0ull;
    for (int d = 0; d < n_new; ++d) {
      const uint32_t x = __ballot_sync(0xffffffffu, (lo >> d) & 1ull), y = __ballot_sync(0xffffffffu, (hi >> d) & 1ull);
      if (lane == 0) sm.seen[d] = make_uint2(x, y);
    }
  }
  if (tid < kOCols) {
    const int r = blk * NC + tid;
    sm.colt[tid] = (unsigned char)min(r / a.G, a.T - 1);
    for (int i = 0; i < PG; ++i) {
      sm.nm[i][tid] = -kNoRef;
      sm.mp[i][tid] = -INFINITY;
      sm.cw[i][tid] = 1.f;
    }
  }
  if (tid >= 128 && tid < 144) {
    const auto lev = [&](int c) { return c == 0 ? a.lev[0] : c == 1 ? a.lev[1] : c == 2 ? a.lev[2] : a.lev[3]; };
    sm.lut[tid & 15] = pack_half2(lev(tid & 3), lev((tid >> 2) & 3));
  }
  const bool rotate = !tail && !a.naive;
  const uint32_t signs = flipped(a, lane);
  for (int c = warp; c < NC; c += kThreads / 32) {
    const int r = blk * NC + c;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (r < rows)
      load4<__nv_bfloat16>(reinterpret_cast<const __nv_bfloat16*>(a.q) + b * a.q_seq + (r / a.G) * a.q_tok +
                               (h * a.G + r % a.G) * kD + lane * 4, v);
    if (rotate) {
      flip(v, signs);
      fwht128_signed(v, lane);
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

  if (warp >= S::kFirstProd) {
    // ---- rows of the key and value tiles
    const int w = warp - S::kFirstProd;
    if (tail) {
      produce_tail(a, sm, w, n, b, h, tile0, len, n_new);
    } else {
      const int64_t row0 = (((int64_t)sm.rep * 2 + ((w >> 2) & 1)) * a.H + h) * a.k;
      produce_prefix(a, sm, w, n, reinterpret_cast<const uint8_t*>(a.anc) + row0 * (kD * 2));
    }
  } else if (warp >= S::kLoad) {
    // ---- token tables and codes
    if (!tail && lane == 0) {
      const int side = warp - S::kLoad;
      load_side(a, sm, side, n, a.comp + (int64_t)lay * a.stride,
                reinterpret_cast<const Meta*>(a.meta) + (((int64_t)sm.rep * 2 + side) * a.H + h) * a.n_tiles + tile0);
    }
    __syncwarp();
  } else if (warp == kMma) {
    // ---- logits: S^T = K^ Q^T.  After a failed wait the products go on with
    // whatever is there; the outputs become NaN at the end.
    const uint64_t kd = tc::sw128_desc(tc::smem_u32(sm.K)), qd = tc::sw128_desc(tc::smem_u32(sm.Q));
    for (int i = 0, place = 0; i < n; ++i) {
      const int bf = i & 1;
      wait_b(sm, &sm.full[0][bf], (i >> 1) & 1, a);
      if (i >= 2) wait_b(sm, &sm.sempty[bf], ((i >> 1) - 1) & 1, a);
      __syncwarp();
      tc::fence_after_sync();
      mma_tile<2, kHalf / 16 - 6, 2, NC * 8 - 6>(tmem + kSCol + bf * NC, kd + bf * (kTileBytes / 16), qd, idesc_f16(128, NC, 0, 0), 0);
      commit_elected(&sm.kempty[bf]);
      if (!tail) commit_elected(&sm.freed[0][place]);
      place = place + 1 < S::kMetaSl ? place + 1 : 0;
      commit_elected(&sm.sfull[bf]);
    }
    // all of it over before the memory is freed, in every case
    tc::mbar_wait(&sm.sfull[(n - 1) & 1], ((n - 1) >> 1) & 1);
    tc::mbar_wait(&sm.kempty[(n - 1) & 1], ((n - 1) >> 1) & 1);
    if (!tail) tc::mbar_wait(&sm.freed[0][(n - 1) % S::kMetaSl], ((n - 1) / S::kMetaSl) & 1);
  } else if (warp == kMma + 1) {
    // ---- outputs: O^T += V^T P
    const uint64_t vd = tc::sw128_mn_desc(tc::smem_u32(sm.V), kHalf), pd = tc::sw128_mn_desc(tc::smem_u32(sm.P), kTT * 128);
    for (int i = 0, place = 0; i < n; ++i) {
      const int bf = i & 1;
      wait_b(sm, &sm.full[1][bf], (i >> 1) & 1, a);
      wait_b(sm, &sm.pfull[bf], (i >> 1) & 1, a);
      __syncwarp();
      tc::fence_after_sync();
      mma_tile<128, 128, 128, 128>(tmem + (PG == 2 ? bf * kOCols : 0), vd + bf * (kTileBytes / 16),
                                   pd + (S::kPBuf == 2 ? bf * (S::kPBytes / 16) : 0), idesc_f16(128, kOCols, 1, 1), i >= PG);
      if (!tail) commit_elected(&sm.freed[1][place]);
      commit_elected(&sm.pv[bf]);
      place = place + 1 < S::kMetaSl ? place + 1 : 0;
    }
    tc::mbar_wait(&sm.pv[(n - 1) & 1], ((n - 1) >> 1) & 1);
    if (!tail) tc::mbar_wait(&sm.freed[1][(n - 1) % S::kMetaSl], ((n - 1) / S::kMetaSl) & 1);
  } else {
    // ---- softmax: thread = token; a group of four warps has CW of the rows and,
    // where two groups share them, every other tile with references, sums and
    // outputs of its own (par)
    const int tok = tid & 127, wq = warp & 3, grp = warp >> 2, par = PG == 2 ? grp & 1 : 0;
    const int c0 = CW * (grp / PG), bar_id = 1 + grp;
    const uint32_t lane_base = (uint32_t)(wq * 32) << 16, ocol = tmem + lane_base + par * kOCols + c0;
    // Sums: of 16 rows a register pair each and thread, added over the tokens at
    // the end; of 32 rows added over 16 lanes in every tile (lane l: row l % 16),
    // for which there are registers.
    constexpr bool kWide = CH > 1;
    float2 lacc[8];
    float lred[CH];
#pragma unroll
    for (int x = 0; x < 8; ++x) lacc[x] = make_float2(0.f, 0.f);
#pragma unroll
    for (int x = 0; x < CH; ++x) lred[x] = 0.f;
    // tokens before `open` are seen by all rows, those behind by the drafts that
    // may, `end` and more are none
    const int open = tail ? len : a.N, end = tail ? len + n_new : a.N;
    for (int i = par; i < n; i += PG) {
      const int bf = i & 1;
      // what this token is, and who sees it
      const bool special = (tile0 + i + 1) * kTT > open;
      unsigned long long vis = ~0ull;
      if (special) {
        const int t = (tile0 + i) * kTT + tok;
        if (t >= end) {
          vis = 0;
        } else if (t >= open) {
          const uint2 s = sm.seen[t - open];
          vis = (unsigned long long)s.y << 32 | s.x;
        }
      }
      wait_b(sm, &sm.sk[i % kKSl], (i / kKSl) & 1, a);
      wait_b(sm, &sm.sv[i % kVSl], (i / kVSl) & 1, a);
      const float rk = sm.rk[i % kKSl][tok], w = sm.wv[i % kVSl][tok];
      wait_b(sm, &sm.sfull[bf], (i >> 1) & 1, a);
      tc::fence_after_sync();
#pragma unroll
      for (int ch = 0; ch < CH; ++ch) {
        const int c1 = c0 + 16 * ch;
        const uint32_t scol = tmem + lane_base + kSCol + bf * NC + c1;
        const uint32_t hidden = special ? hidden_columns(vis, &sm.colt[c1]) : 0u;
        float2 p[8];
        uint32_t pk[8];
        // new references for the first tile and, rarely, later; then at most once
        // (infinities may leave none)
        for (bool renew = i == par, renewed = false;;) {
          if (renew) {
            renewed = true;
            new_references(sm, a, scol, ocol + 16 * ch, c1, par, grp, i - PG, bar_id, rk, w, hidden);
            if (kWide) {
              lred[ch] *= sm.fl[par][c1 + (lane & 15)];
            } else {
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                lacc[x].x *= sm.fl[par][c1 + 2 * x];
                lacc[x].y *= sm.fl[par][c1 + 2 * x + 1];
              }
            }
          }
          float pmax = 0.f, vmax = 0.f;
          uint32_t s[16];
          load_cols(scol, s);
          float2 u[8];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float4 cs = *reinterpret_cast<const float4*>(&sm.cs[c1 + 4 * y]);
            const float4 nm = *reinterpret_cast<const float4*>(&sm.nm[par][c1 + 4 * y]);
#pragma unroll
            for (int z = 0; z < 2; ++z)
              u[2 * y + z] = __ffma2_rn(
                  make_float2(__uint_as_float(s[4 * y + 2 * z]), __uint_as_float(s[4 * y + 2 * z + 1])),
                  __fmul2_rn(z ? make_float2(cs.z, cs.w) : make_float2(cs.x, cs.y), make_float2(rk, rk)),
                  z ? make_float2(nm.z, nm.w) : make_float2(nm.x, nm.y));
          }
          if (hidden) {
            asm volatile("");                  // a branch: ordinary tiles should not carry this as predicated instructions
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              if ((hidden >> (2 * x)) & 1u) u[x].x = -INFINITY;
              if ((hidden >> (2 * x + 1)) & 1u) u[x].y = -INFINITY;
            }
          }
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float4 cw = *reinterpret_cast<const float4*>(&sm.cw[par][c1 + 4 * y]);
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const float2 e = make_float2(tc::ex2_approx(u[2 * y + z].x), tc::ex2_approx(u[2 * y + z].y));
              // in this order a masked 0 stays 0 whatever the value's scale
              const float2 v = __fmul2_rn(__fmul2_rn(e, make_float2(w, w)),
                                          z ? make_float2(cw.z, cw.w) : make_float2(cw.x, cw.y));
              pmax = fmaxf(pmax, fmaxf(e.x, e.y));
              vmax = fmaxf(vmax, fmaxf(fabsf(v.x), fabsf(v.y)));
              p[2 * y + z] = e;
              pk[2 * y + z] = pack_half2(v.x, v.y);
            }
          }
          renew = bar_or(bar_id, 128, pmax > kSumLimit || vmax > kPLimit);
          if (!renew || renewed) break;
        }
        if (ch == 0) {
          // the products that read this buffer of P
          constexpr int back = S::kPBuf;
          if (i >= back) wait_b(sm, &sm.pv[(i - back) & 1], ((i - back) >> 1) & 1, a);
        }
        uint8_t* prow = sm.P[S::kPBuf == 2 ? bf : 0] + (c1 >> 6) * (kTT * 128) + tok * 128;
#pragma unroll
        for (int x = 0; x < 2; ++x)
          *reinterpret_cast<uint4*>(prow + ((((c1 & 63) / 8 + x) ^ (tok & 7)) << 4)) =
              make_uint4(pk[4 * x], pk[4 * x + 1], pk[4 * x + 2], pk[4 * x + 3]);
        if (kWide) {
          lred[ch] += sum16(p, lane);
        } else {
#pragma unroll
          for (int x = 0; x < 8; ++x) lacc[x] = __fadd2_rn(lacc[x], p[x]);
        }
      }
      tc::fence_proxy_async_smem();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(&sm.sempty[bf]);
        tc::mbar_arrive(&sm.pfull[bf]);
      }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // ---- sums over the tokens
    if (!kWide) lred[0] = sum16(lacc, lane);
#pragma unroll
    for (int ch = 0; ch < CH; ++ch) {
      const float l = lred[ch] + __shfl_xor_sync(0xffffffffu, lred[ch], 16);
      if (lane < 16) sm.lsum[par][wq][c0 + 16 * ch + lane] = l;
    }
    // outputs in units of the sum's reference (of the larger, where two groups
    // have these rows; each writes half of them), once all waits of these groups
    // are over: one that failed makes the rows NaN
    if (n > 1) wait_b(sm, &sm.pv[(n - 2) & 1], ((n - 2) >> 1) & 1, a);
    wait_b(sm, &sm.pv[(n - 1) & 1], ((n - 1) >> 1) & 1, a);
    tc::fence_after_sync();
    tc::named_bar(8 + grp / PG, 128 * PG);
    const bool nan = *(volatile int*)&sm.err || *(volatile int*)&sm.bad;
    if (nan && tid == 0) latch_error(a.counters, kDevErrBounds);
    float* fo = reinterpret_cast<float*>(sm.red[grp][0][0]);       // this group's factors of either parity's outputs
    if (tok < CW) {
      const int c = c0 + tok;
      const float m = PG == 2 ? fmaxf(-sm.nm[0][c], -sm.nm[PG - 1][c]) : -sm.nm[0][c];
      float l = 0.f;
#pragma unroll
      for (int k = 0; k < PG; ++k) {
        const float sum = sm.lsum[k][0][c] + sm.lsum[k][1][c] + sm.lsum[k][2][c] + sm.lsum[k][3][c];
        l += sm.nm[k][c] < -kNoRef ? sum * pow2(-sm.nm[k][c] - m) : sum;   // a sum without a reference is zero, or NaN
      }
      // the unit: a power of two, so that nothing is rounded, and none where the
      // reference plus its exponent would not be a whole number in fp32
      const int shift = l > 0.f && l < INFINITY && fabsf(m) < 8388608.f ? (__float_as_int(l) >> 23) - 126 + kSumBits : 0;
#pragma unroll
      for (int k = 0; k < PG; ++k) {
        // two factors: one alone can be out of fp32's range, above it for values near their largest
        const float d = sm.mp[k][c] - m - (float)shift, half = floorf(0.5f * d);
        const bool has = sm.nm[k][c] < -kNoRef;
        fo[k * 32 + tok] = has ? pow2(half) : 0.f;
        fo[64 + k * 32 + tok] = pow2(d - half);
      }
      if (par == 0) {
        ml[2 * c] = nan ? 0.f : m + (float)shift;
        ml[2 * c + 1] = nan ? __int_as_float(0x7fc00000) : l * pow2((float)-shift);
      }
    }
    tc::named_bar(bar_id, 128);
    float* o = a.part + ((unit * a.parts + part) * NC + c0) * kD + tok;
#pragma unroll 1
    for (int x = par * (CW / PG); x < (par + 1) * (CW / PG); x += 4) {
      uint32_t v[PG][4];
#pragma unroll
      for (int k = 0; k < PG; ++k) tmem_ld4(tmem + lane_base + k * kOCols + c0 + x, v[k]);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        // a parity without a reference has nothing (and, without a tile, no number) there
        float acc = fo[x + y] != 0.f ? __uint_as_float(v[0][y]) * fo[x + y] * fo[64 + x + y] : 0.f;
        if (PG == 2 && fo[32 + x + y] != 0.f) acc = fmaf(__uint_as_float(v[PG - 1][y]) * fo[32 + x + y], fo[96 + x + y], acc);
        o[(x + y) * kD] = acc;
      }
    }
    tc::fence_before_sync();
  }
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kMma) tc::tmem_dealloc(tmem, S::kTmemCols);
}

template <int NC>
constexpr int smem_bytes() {
  static_assert(sizeof(Sm<NC>) + 1024 <= 227 * 1024, "shared memory of one CTA");
  return (int)sizeof(Sm<NC>) + 1024;
}

template <int NC>
int launch_nc(const TreeArgs& a, cudaStream_t s) {
  static std::mutex mu;
  static int ready_dev = -1;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ANCHORKV_ECUDA;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (ready_dev != dev) {
      if (cudaFuncSetAttribute(tree_tc_kernel<NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<NC>()) != cudaSuccess)
        return ANCHORKV_ECUDA;
      ready_dev = dev;
    }
  }
  // two rows a warp, or, of many sequences, as many as keep eight CTAs an SM busy
  const int gx = a.comp ? std::max(1, std::min((a.k + 15) / 16, std::max(4, 148 * 16 / (2 * a.H * a.batch)))) : 1;
  tree_prep_kernel<<<dim3(gx, 2 * a.H, a.batch), 256, 0, s>>>(a);
  if (cudaGetLastError() != cudaSuccess) return ANCHORKV_ECUDA;
  int st = ANCHORKV_OK;
  if (a.comp) st = launch_dependent(tree_meta_kernel, dim3((a.n_tiles + 7) / 8, 2 * a.H, a.batch), 256, 0, s, a);
  if (st) return st;
  st = launch_dependent(tree_tc_kernel<NC>, dim3(a.n_blk, a.batch * a.H, a.parts), Shape<NC>::kThreads, smem_bytes<NC>(), s, a);
  if (st) return st;
  return launch_tree_merge<__nv_bfloat16>(a, NC, s);
}

}  // namespace

int64_t tree_meta_bytes() { return (int64_t)sizeof(Meta); }

// Time of the longest run of CTAs on an SM, in tiles, for units that divide
// pre + tail tiles over `parts` as tree_tail_parts does.  A CTA costs kFixed
// tiles beside its own (set-up, first references, outputs), and one of exact
// tokens, whose rows come from HBM and are scaled on their way, two a tile and
// two for the first rows' latency.  Parts
// of exact tokens start last and fill what the others leave.
static int64_t run_length(int units, int parts, int pre, int tail) {
  constexpr int kFixed = 6, kSms = 148;
  const int t = pre ? std::max(1, std::min((int)(((int64_t)tail * parts + pre + tail - 1) / (pre + tail)), parts - 1)) : parts;
  int a = pre ? (pre + parts - t - 1) / (parts - t) + kFixed : 0, b = 2 * ((tail + t - 1) / t + 1) + kFixed;
  int n_a = units * (parts - t), n_b = units * t;
  if (a < b) {
    std::swap(a, b);
    std::swap(n_a, n_b);
  }
  const int rounds = (n_a + kSms - 1) / kSms;
  const int64_t fill = b ? (int64_t)(rounds * kSms - n_a) * (a / b) : n_b;
  return (int64_t)rounds * a + (n_b > fill ? (n_b - fill + kSms - 1) / kSms * b : 0);
}

void tree_plan_tc(const Plan& pl, bool prefix, TreePlan* tp) {
  // One CTA an SM.  A tile of 16, 32, 64 or 128 rows takes the times below (in
  // tenths of a microsecond, measured over 32 k and 128 k tokens), so the block
  // and the parts are those whose longest run of CTAs on an SM is shortest, for
  // page tables between empty and full.  Larger blocks rebuild each tile for more
  // rows; smaller ones leave less of a block empty and spread over more SMs.
  // Measured (8 KV heads, us; each at its own best parts):
  //   rows a head, block of  16     32     64    128
  //   4,   32 k tokens      36.7   40.5   45.6   65.5
  //   24,  32 k             54.1   40.8   46.0   65.5
  //   64,  32 k             89.2   63.2   47.4   68.5
  //   128, 32 k            157    106     75.8   74.1
  //   256, 32 k            294    191    130    124
  //   192, 128 k           792    477    315    369
  //   32,  16 x 32 k       762    480    630    795
  //   64,  16 x 32 k      1412    911    641    815
  // A part has 64 k tokens at most (of either kind, about): every product of 16
  // tokens may cut the accumulators by 2^-23, 4096 of them by 2^-11, the operands'
  // own rounding.  2^20 tokens in one part behind a first one that takes 98% were
  // off by 5.2e-3 of the output.
  constexpr int kRows[4] = {16, 32, 64, 128}, kTime[4] = {12, 14, 17, 29}, kSms = 148, kMostTiles = (1 << 16) / kTT;
  const int pre = prefix ? (pl.N + kTT - 1) / kTT : 0, tail = (int)((tp->cap + tp->T + kTT - 1) / kTT);
  const int least = std::max(prefix ? 2 : 1, (pre + tail + kMostTiles - 1) / kMostTiles);
  int64_t best = INT64_MAX;
  tp->RB = kRows[0];                                   // where nothing fits: the caller finds the workspace too small
  tp->n_blk = (tp->rows + tp->RB - 1) / tp->RB;
  tp->parts = least;
  tp->tail_parts = prefix ? 0 : least;
  for (int k = 0; k < 4; ++k) {
    const int n_blk = (tp->rows + kRows[k] - 1) / kRows[k], units = tp->batch * pl.H * n_blk;
    // as many parts of compressed tokens (with and without one of exact tokens
    // beside them) as fill a whole number of rounds
    const int first = std::max(1, (units + kSms - 1) / kSms);
    for (int rounds = first; rounds < first + 12; ++rounds)
      for (int more = prefix; more >= 0; --more) {
        const int fit = (int)std::min<int64_t>(tp->room / ((int64_t)units * kRows[k]), INT_MAX);
        if (fit < least) continue;
        const int parts = std::min(fit, std::max(least, std::min(kSms * rounds / units + more, pre + tail)));
        const int64_t cost = (run_length(units, parts, pre, tail) + run_length(units, parts, pre, 1)) * kTime[k];
        if (cost < best) {
          best = cost;
          tp->RB = kRows[k];
          tp->n_blk = n_blk;
          tp->parts = parts;
          tp->tail_parts = prefix ? 0 : parts;
        }
      }
  }
}

int launch_tree_tc(const TreeArgs& a, cudaStream_t s) {
  return a.RB == 16 ? launch_nc<16>(a, s) : a.RB == 32 ? launch_nc<32>(a, s) : a.RB == 64 ? launch_nc<64>(a, s) : launch_nc<128>(a, s);
}

}  // namespace akv
