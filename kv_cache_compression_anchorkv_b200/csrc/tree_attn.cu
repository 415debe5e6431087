// Tree attention: argument checks, workspace plan and dispatch.
#include <algorithm>

#include "common.cuh"
#include "tree.h"

namespace akv {
namespace {

constexpr int64_t kAnyBytes = (int64_t)1 << 60;

// The plan for a workspace of ws_bytes.  The best division of the tokens may need
// more bytes for fewer rows or sequences; where it does not fit, the tokens are
// divided into as many parts as do, so that what serves a call serves every
// smaller one: with its own blocks and `least` parts that needs no more.
int make_tree_plan(const anchorkv_params* p, int batch, int T, const anchorkv_pages* pg, bool prefix, int64_t ws_bytes,
                   Plan* pl, TreePlan* tp) {
  int st = make_plan(p, pl);
  if (st) return st;
  if (batch < 0 || T < 1 || T > kTreeMaxDrafts) return ANCHORKV_EINVAL;
  if ((int64_t)batch * pl->H > 65535 || pl->H > 32767) return ANCHORKV_EUNSUPPORTED;      // grids: sequences x heads, sides x heads
  *tp = TreePlan{};
  tp->batch = std::max(batch, 1);
  tp->T = T;
  tp->rows = T * pl->G;
  if (pg) {
    st = pages_tokens(pg, &tp->cap);
    if (st) return st;
    if (pg->n_kv_heads != pl->H || pg->dtype != p->dtype || batch > pg->n_slots) return ANCHORKV_EINVAL;
    if (tp->cap > (1 << 20)) return ANCHORKV_EUNSUPPORTED;
  }
  // bf16 caches on the tensor cores; fp32 caches need 32-bit products
  const bool tcore = p->dtype == ANCHORKV_BF16;
  int64_t off = 256;                                                     // status words
  auto take = [&](int64_t bytes) { const int64_t o = off; off += (bytes + 255) / 256 * 256; return o; };
  if (tcore) {
    const int64_t rows = (int64_t)tp->batch * 2 * pl->H * pl->k;
    tp->o_anc = take(2 * kD * rows);
    tp->o_anc_scale = take(4 * rows);
    if (prefix) tp->o_meta = take(tree_meta_bytes() * tp->batch * 2 * pl->H * pl->n_tiles);
    tp->o_inf = take(8 * (int64_t)tp->batch * pl->H);
  }
  // rows come in blocks of 16 at least: 128 bytes of (max, sum) and 8 KB of outputs
  tp->room = std::max<int64_t>(0, (ws_bytes - off) / (16 * (8 + 4 * kD)) * 16);
  if (tp->room % 32 && off + tp->room * (8 + 4 * kD) + 128 > ws_bytes) tp->room -= 16;     // (max, sum) padded to 256
  if (tcore) tree_plan_tc(*pl, prefix, tp);
  else tree_plan_simt(*pl, tp);
  const int64_t parts = (int64_t)tp->batch * pl->H * tp->n_blk * tp->parts * tp->RB;
  tp->o_ml = take(8 * parts);
  tp->o_part = take(4 * kD * parts);
  tp->ws_total = off;
  return ANCHORKV_OK;
}

}  // namespace
}  // namespace akv

using namespace akv;

extern "C" {

int anchorkv_tree_workspace_bytes(const anchorkv_params* p, int32_t batch, int32_t n_draft, const anchorkv_pages* pg,
                                  size_t* ws_bytes) {
  if (!ws_bytes) return ANCHORKV_EINVAL;
  Plan pl;
  TreePlan tp;
  // the split differs with and without compressed tokens
  int64_t most = 0;
  for (const bool prefix : {true, false}) {
    const int st = make_tree_plan(p, batch, n_draft, pg, prefix, kAnyBytes, &pl, &tp);
    if (st) return st;
    most = std::max(most, tp.ws_total);
  }
  *ws_bytes = (size_t)most;
  return ANCHORKV_OK;
}

int anchorkv_tree_attn(const anchorkv_params* p, const anchorkv_tree* t, void* ws, size_t ws_bytes, void* stream) {
  if (!t) return ANCHORKV_EINVAL;
  Plan pl;
  TreePlan tp;
  int st = make_tree_plan(p, t->batch, t->n_draft, t->pages, t->compressed != nullptr, (int64_t)std::min<size_t>(ws_bytes, kAnyBytes),
                          &pl, &tp);
  if (st) return st;
  if (t->batch == 0) return ANCHORKV_OK;
  if (!t->q || !t->K_new || !t->V_new || !t->out || !ws) return ANCHORKV_EINVAL;
  if (t->pages && (!t->state || !t->K_pages || !t->V_pages)) return ANCHORKV_EINVAL;
  if (t->compressed) {
    if (t->n_layouts < 1 || (!t->layout_of && t->n_layouts < t->batch)) return ANCHORKV_EINVAL;
    if (t->seq_stride_bytes % 16 || (t->n_layouts > 1 && t->seq_stride_bytes < pl.L.total_bytes)) return ANCHORKV_EINVAL;
  }
  // a sequence's or a token's row starts on a 16-byte boundary, and rows hold all heads
  const int64_t e = pl.elem;
  if (t->q_tok_stride < (int64_t)pl.Hq * kD || t->new_tok_stride < (int64_t)pl.H * kD || t->q_seq_stride < 0 ||
      t->new_seq_stride < 0)
    return ANCHORKV_EINVAL;
  if ((t->q_seq_stride * e | t->q_tok_stride * e | t->new_seq_stride * e | t->new_tok_stride * e) & 15)
    return ANCHORKV_EINVAL;
  if (((uintptr_t)t->compressed | (uintptr_t)t->q | (uintptr_t)t->K_new | (uintptr_t)t->V_new | (uintptr_t)t->state |
       (uintptr_t)t->K_pages | (uintptr_t)t->V_pages | (uintptr_t)t->out | (uintptr_t)ws) & 15)
    return ANCHORKV_EINVAL;
  if (((uintptr_t)t->layout_of | (uintptr_t)t->n_new) & 3 || ((uintptr_t)t->mask & 7)) return ANCHORKV_EINVAL;
  if ((int64_t)ws_bytes < tp.ws_total) return ANCHORKV_ENOSPC;
  st = check_device();
  if (st) return st;

  TreeArgs a = {};
  a.comp = (const uint8_t*)t->compressed;
  a.stride = t->seq_stride_bytes;
  a.off_ak = pl.L.off_anchors_k; a.off_av = pl.L.off_anchors_v; a.off_tok = pl.L.off_tok;
  a.off_bm = pl.L.off_bitmap; a.off_pf = pl.L.off_tile_prefix;
  a.off_codes = pl.L.off_res_codes; a.off_sig = pl.L.off_res_sigma;
  a.n_layouts = t->n_layouts;
  a.layout_of = t->layout_of;
  a.N = pl.N; a.H = pl.H; a.G = pl.G; a.k = pl.k; a.n_tiles = pl.n_tiles; a.R = pl.R;
  a.lev[0] = (float)-pl.l2; a.lev[1] = (float)-pl.l1; a.lev[2] = (float)pl.l1; a.lev[3] = (float)pl.l2;
  for (int i = 0; i < 4; ++i) a.sign_bits[i] = pl.sign_bits[i];
  a.naive = naive_codec(pl);
  a.batch = t->batch; a.T = t->n_draft; a.RB = tp.RB; a.n_blk = tp.n_blk; a.parts = tp.parts;
  a.tail_parts = tp.tail_parts;
  a.q = t->q; a.q_seq = t->q_seq_stride; a.q_tok = t->q_tok_stride;
  a.kn = t->K_new; a.vn = t->V_new; a.n_seq = t->new_seq_stride; a.n_tok = t->new_tok_stride;
  a.n_new = t->n_new;
  a.mask = (const unsigned long long*)t->mask;
  if (t->pages) {
    const anchorkv_pages* pg = t->pages;
    a.n_pages = pg->n_pages; a.P = pg->page_size; a.maxp = pg->max_pages;
    a.len = t->state + 16 + 2 * (int64_t)pg->n_pages;
    a.table = a.len + pg->n_slots;
    a.kp = t->K_pages; a.vp = t->V_pages;
  }
  a.out = t->out;
  char* w = (char*)ws;
  a.counters = (int*)w;
  a.ml = (float*)(w + tp.o_ml);
  a.part = (float*)(w + tp.o_part);
  cudaStream_t s = (cudaStream_t)stream;
  a.anc = w + tp.o_anc;
  a.anc_scale = (float*)(w + tp.o_anc_scale);
  a.meta = w + tp.o_meta;
  a.inf_v = p->dtype == ANCHORKV_BF16 ? (unsigned long long*)(w + tp.o_inf) : nullptr;
  stage_begin(kStTree, s);
  st = p->dtype == ANCHORKV_BF16 ? launch_tree_tc(a, s) : launch_tree_simt(a, s);
  stage_end(kStTree, s, p->dtype != ANCHORKV_BF16 ? 2 : t->compressed ? 4 : 3);
  return st;
}

}  // extern "C"
