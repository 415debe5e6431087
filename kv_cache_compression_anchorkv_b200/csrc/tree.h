// Plan and kernel arguments of the tree attention (tree_attn.cu and the
// kernels it launches).
#pragma once

#include "internal.h"

namespace akv {

// Drafts of one sequence: bits of a mask word.
constexpr int kTreeMaxDrafts = 64;
// Reference (a NaN) of a part whose sequence could not be read; its sum is NaN
// too, and the merge latches the error.
constexpr uint32_t kTreeBadPart = 0x7fc0bad0u;

// One call's shape: the rows (draft t, query head g) of a KV head, r = t G + g,
// are cut into blocks of RB; every (sequence, head, block) is a unit, whose
// tokens `parts` CTAs share.
struct TreePlan {
  int batch, T, rows, RB, n_blk, parts;
  int tail_parts;                    // of those, CTAs of exact tokens only; 0: by the sequence's lengths
  int64_t cap;                       // exact tokens that the page tables can hold
  int64_t room;                      // part rows (sequence, head, block, part, row) that the workspace has room for
  // workspace (bytes): status words, (max, sum) and outputs of every
  // part; tensor-core kernel: rotated anchors, their scales, token tables,
  // infinite values
  int64_t o_ml, o_part, o_anc, o_anc_scale, o_meta, o_inf, ws_total;
};

struct TreeArgs {
  const uint8_t* comp;               // null: no compressed tokens
  int64_t stride;
  int64_t off_ak, off_av, off_tok, off_bm, off_pf, off_codes, off_sig;
  int n_layouts;
  const int* layout_of;
  int N, H, G, k, n_tiles;
  int64_t R;
  float lev[4];
  uint32_t sign_bits[4];
  int naive;
  int batch, T, RB, n_blk, parts, tail_parts;
  const void* q;
  int64_t q_seq, q_tok;
  const void* kn;
  const void* vn;
  int64_t n_seq, n_tok;
  const int* n_new;
  const unsigned long long* mask;
  // pages (table null: none)
  const int* len;
  const int* table;
  int n_pages, P, maxp;
  const void* kp;
  const void* vp;
  void* out;
  int* counters;
  float* ml;                         // [unit][part][RB] (max, sum)
  float* part;                       // [unit][part][RB][D]
  void* anc;                         // [batch][2][H][k][D] fp16, rotated
  float* anc_scale;                  // [batch][2][H][k]
  void* meta;                        // [batch][2][H][n_tiles] token tables
  unsigned long long* inf_v;         // [batch][H] drafts with an infinite or NaN value
};

// Drafts of sequence b.
__device__ __forceinline__ int tree_new(const TreeArgs& a, int b) {
  const int n = a.n_new ? a.n_new[b] : a.T;
  return n < 0 ? 0 : (n > a.T ? a.T : n);
}
// Layout of sequence b; -1 where layout_of is out of its range.
__device__ __forceinline__ int tree_layout(const TreeArgs& a, int b) {
  const int l = a.layout_of ? a.layout_of[b] : b;
  return l < 0 || l >= a.n_layouts ? -1 : l;
}
// Exact tokens of sequence b; -1 where the state's length is out of its range.
__device__ __forceinline__ int tree_len(const TreeArgs& a, int b) {
  if (!a.table) return 0;
  const int n = a.len[b];
  return n < 0 || n > (int64_t)a.maxp * a.P ? -1 : n;
}
// Parts of a sequence that take exact tokens only, the last ones: as many as
// its exact tokens' share of all tiles (of 128), one at least for either kind.
// The page tables may have room for far more tokens than a sequence has, so the
// launch fixes the parts and each sequence divides them by its own length.
__device__ __forceinline__ int tree_tail_parts(const TreeArgs& a, int len, int n_new) {
  if (a.tail_parts) return a.tail_parts;
  // 2^13 tail tiles and 2^12 parts at most
  const uint32_t tail = (uint32_t)(max(len, 0) + n_new + 127) / 128u, all = tail + a.n_tiles;
  return max(1, min((int)((tail * a.parts + all - 1) / all), a.parts - 1));
}
__device__ __forceinline__ unsigned long long tree_mask(const TreeArgs& a, int b, int t) {
  return a.mask ? a.mask[(int64_t)b * a.T + t] : (2ull << t) - 1;
}

// Bytes of one tile's token table (one side and head).
int64_t tree_meta_bytes();
void tree_plan_tc(const Plan& pl, bool prefix, TreePlan* tp);
int launch_tree_tc(const TreeArgs& a, cudaStream_t s);
void tree_plan_simt(const Plan& pl, TreePlan* tp);
int launch_tree_simt(const TreeArgs& a, cudaStream_t s);

}  // namespace akv
