// Pages of the exact tail: commit, fork and compact.
//
// "AnchorKV-adapted" (VeloxQuant-MLX), "Adaptation notes": decode tokens are
// appended uncompressed and never re-anchored.  Here they are kept in pages
// that all layers share one table of, so that beams can hold pages together
// and a sequence can end without leaving a hole that only it could fill.
//
// Every operation is two launches.  A single CTA works on the page state: it
// checks the whole operation first and writes only what it has checked, and
// with the state's reads done before its writes it may work in place; that
// costs one pass over the arrays an operation touches (a state is tens of
// kilobytes), bound by the latency of the chain of scans.  The rows then move
// on all SMs in 16-byte pieces, bound by HBM: the second kernel is launched
// as a programmatic dependent, so its CTAs are resident when the state is
// ready.  Ids are handed out by scans in slot or page order, never by
// atomics, so they depend on the state alone.
//
// Measured (CUDA graph, bf16, 32 layers of 8 heads): one token 6.8 us and the
// last pages of 4 beams 11.1 us (two launches and the state kernel's scans
// bound them), 16 accepted paths of up to 16 rows 17.2 us (3.2 TB/s), 64 slots
// forked 24.4 us (3.9 TB/s), 40 of 160 pages moved 114 us (5.9 TB/s, 90% of a
// copy's rate).
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace akv {
namespace {

constexpr int kMetaThreads = 1024;
constexpr int kPageHeader = 16;
enum PageStatus { kPgOk = 0, kPgNoFree = 1, kPgTableFull = 2, kPgRange = 3 };

struct PgArgs {
  int n_pages, P, S, maxp, L, H;
  int row16;                       // 16-byte pieces of one token and head
  const int* in;                   // page states
  int* out;
  int* ws;                         // scratch: [0] items, then as the operation lays it out
  uint4* pool[2];                  // K, V
  // commit
  const uint4* fresh[2];
  int batch, T;
  const int* path;
  const int* n_accept;
  // fork
  const int* parents;
};

__host__ __device__ inline int64_t o_refs(const PgArgs& a) { return kPageHeader + (int64_t)a.n_pages; }
__host__ __device__ inline int64_t o_len(const PgArgs& a) { return kPageHeader + 2 * (int64_t)a.n_pages; }
__host__ __device__ inline int64_t o_table(const PgArgs& a) { return o_len(a) + a.S; }
__host__ __device__ inline int64_t state_ints(const PgArgs& a) { return o_table(a) + (int64_t)a.S * a.maxp; }

// Scratch (int32): [16] header (0: copies), [n_pages] counts or new ids,
// 3 x [most] copy list (source, destination, rows), [S][maxp] staged table.
__host__ __device__ inline int64_t list_most(int n_pages, int S) { return n_pages / 2 + 1 > S ? n_pages / 2 + 1 : S; }
__host__ __device__ inline int64_t w_list(const PgArgs& a) { return 16 + (int64_t)a.n_pages; }
__host__ __device__ inline int64_t w_table(const PgArgs& a) { return w_list(a) + 3 * list_most(a.n_pages, a.S); }

// Exclusive sum over the CTA in thread order; *total gets the sum.  `tmp`
// holds 33 ints; every thread calls it.
__device__ __forceinline__ int block_scan(int v, int* tmp, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) tmp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const int s = tmp[lane];
    int z = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, z, o);
      if (lane >= o) z += y;
    }
    tmp[lane] = z - s;
    if (lane == 31) tmp[32] = z;
  }
  __syncthreads();
  const int r = tmp[warp] + x - v;
  *total = tmp[32];
  __syncthreads();
  return r;
}

// The refused operation: state_out is state_in with the status word set.
__device__ void refuse(const PgArgs& a, int code) {
  if (a.out != a.in)
    for (int64_t i = threadIdx.x; i < state_ints(a); i += blockDim.x) a.out[i] = a.in[i];
  __syncthreads();
  if (threadIdx.x == 0) {
    if (a.in[0] == 0) a.out[0] = code;
    a.ws[0] = 0;
  }
}

// The code that threads have raised in shared memory, the same for all of them:
// none raises it again before all have read it.
__device__ __forceinline__ int refused(const int* bad) {
  __syncthreads();
  const int code = *(const volatile int*)bad;
  __syncthreads();
  return code;
}

__device__ __forceinline__ void header_out(const PgArgs& a, int status, int n_free, int items) {
  if (threadIdx.x < kPageHeader) a.out[threadIdx.x] = threadIdx.x == 0 ? status : threadIdx.x == 1 ? n_free : 0;
  if (threadIdx.x == 0) a.ws[0] = items;
}

// The state is ready for the dependent kernel once this CTA ends; its CTAs
// may become resident from here on.
__device__ __forceinline__ void let_dependents_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__global__ void __launch_bounds__(kMetaThreads) pages_init_kernel(PgArgs a) {
  const int64_t n = state_ints(a), stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += stride) {
    int v = -1;                                              // page table
    if (i < kPageHeader) v = i == 1 ? a.n_pages : 0;
    else if (i < o_refs(a)) v = a.n_pages - 1 - (int)(i - kPageHeader);
    else if (i < o_table(a)) v = 0;
    a.out[i] = v;
  }
}

// --- commit -------------------------------------------------------------

__global__ void __launch_bounds__(kMetaThreads) commit_state_kernel(PgArgs a) {
  let_dependents_launch();
  __shared__ int tmp[33];
  __shared__ int bad, carry;
  const int tid = threadIdx.x;
  const int* len_in = a.in + o_len(a);
  const int* table_in = a.in + o_table(a);
  const int status = a.in[0], n_free = a.in[1];
  if (tid == 0) { bad = n_free < 0 || n_free > a.n_pages ? kPgRange : kPgOk; carry = 0; }
  __syncthreads();
  // checks: counts, paths, the page that the first row goes to, the tables' length
  int need_all = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kMetaThreads) {
    const int b = b0 + tid;
    int need = 0, why = kPgOk;
    if (b < a.batch) {
      const int n = a.n_accept[b], len = len_in[b];
      if (n < 0 || n > a.T || len < 0 || len > a.maxp * (int64_t)a.P) why = kPgRange;
      else {
        const int had = (len + a.P - 1) / a.P, has = (int)(((int64_t)len + n + a.P - 1) / a.P);
        need = has - had;
        if (has > a.maxp) why = kPgTableFull;
        else if (n > 0 && len % a.P) {
          const int pg = table_in[(int64_t)b * a.maxp + had - 1];
          if (pg < 0 || pg >= a.n_pages || a.in[o_refs(a) + pg] != 1) why = kPgRange;
        }
        if (a.path)
          for (int i = 0; i < n; ++i) {
            const int r = a.path[(int64_t)b * a.T + i];
            if (r < 0 || r >= a.T) why = kPgRange;
          }
      }
    }
    if (why) atomicMax(&bad, why);
    int total;
    block_scan(need, tmp, &total);
    need_all += total;
  }
  const int why_not = refused(&bad);
  if (why_not || need_all > n_free) {
    refuse(a, why_not ? why_not : kPgNoFree);
    return;
  }
  // the ids that will be handed out
  for (int i = tid; i < need_all; i += kMetaThreads) {
    const int id = a.in[kPageHeader + n_free - 1 - i];
    if (id < 0 || id >= a.n_pages || a.in[o_refs(a) + id] != 0) atomicMax(&bad, kPgRange);
  }
  if (refused(&bad)) {
    refuse(a, kPgRange);
    return;
  }
  if (a.out != a.in) {
    for (int64_t i = kPageHeader + tid; i < state_ints(a); i += kMetaThreads)
      if (i < kPageHeader + n_free - need_all || i >= kPageHeader + n_free) a.out[i] = a.in[i];
    __syncthreads();
  }
  for (int b0 = 0; b0 < a.batch; b0 += kMetaThreads) {
    const int b = b0 + tid;
    int len = 0, n = 0, had = 0, has = 0;
    if (b < a.batch) {
      len = len_in[b];
      n = a.n_accept[b];
      had = (len + a.P - 1) / a.P;
      has = (len + n + a.P - 1) / a.P;
    }
    int total;
    const int first = carry + block_scan(has - had, tmp, &total);
    for (int j = had; j < has; ++j) {
      const int id = a.in[kPageHeader + n_free - 1 - (first + j - had)];
      a.out[o_table(a) + (int64_t)b * a.maxp + j] = id;
      a.out[o_refs(a) + id] = 1;
    }
    if (b < a.batch) a.out[o_len(a) + b] = len + n;
    __syncthreads();
    if (tid == 0) carry += total;
    __syncthreads();
  }
  for (int i = tid; i < need_all; i += kMetaThreads) a.out[kPageHeader + n_free - 1 - i] = -1;
  header_out(a, status, n_free - need_all, 1);
}

// One warp per (layer, side, sequence, accepted row): the row of all heads is
// contiguous in the drafts and H pieces of D elements in the page.  What the
// rows of a sequence share is fetched ahead of the row's own lookups, and a
// lane's pieces are in flight together.
__global__ void __launch_bounds__(256) commit_rows_kernel(PgArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t n_rows = (int64_t)a.batch * a.T, units = n_rows * 2 * a.L;
  const int64_t warps = (int64_t)gridDim.x * 8;
  const int pieces = a.H * a.row16, shift = a.row16 == 16 ? 4 : 5, page16 = a.P * a.row16;
  wait_for_primary();
  if (a.ws[0] == 0) return;
  for (int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); u < units; u += warps) {
    const int64_t ls = u / n_rows, r = u % n_rows;
    const int b = (int)(r / a.T), i = (int)(r % a.T), side = (int)(ls & 1);
    const int64_t l = ls >> 1;
    const int n = a.n_accept[b], len = a.out[o_len(a) + b], src = a.path ? a.path[(int64_t)b * a.T + i] : i;
    if (i >= n) continue;
    const int pos = len - n + i;
    const int pg = a.out[o_table(a) + (int64_t)b * a.maxp + pos / a.P];
    const uint4* from = a.fresh[side] + ((l * a.batch + b) * a.T + src) * pieces;
    uint4* to = a.pool[side] + (l * a.n_pages + pg) * a.H * page16 + (int64_t)(pos % a.P) * a.row16;
    for (int x0 = lane; x0 < pieces; x0 += 32 * 4) {
      uint4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (x0 + 32 * k < pieces) v[k] = from[x0 + 32 * k];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int x = x0 + 32 * k;
        if (x < pieces) to[(int64_t)(x >> shift) * page16 + (x & (a.row16 - 1))] = v[k];
      }
    }
  }
}

// --- fork ---------------------------------------------------------------

__global__ void __launch_bounds__(kMetaThreads) fork_state_kernel(PgArgs a) {
  let_dependents_launch();
  extern __shared__ int sm[];
  int* keeper = sm;               // lowest slot that copies sequence p
  int* children = sm + a.S;       // slots that copy sequence p
  int* len_old = sm + 2 * a.S;
  int* parent = sm + 3 * a.S;
  __shared__ int tmp[33];
  __shared__ int bad, carry;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int status = a.in[0], n_free = a.in[1];
  const int* table_in = a.in + o_table(a);
  int* count = a.ws + 16;
  int* list = a.ws + w_list(a);
  const int64_t most = list_most(a.n_pages, a.S);
  if (tid == 0) bad = n_free < 0 || n_free > a.n_pages ? kPgRange : kPgOk;
  for (int s = tid; s < a.S; s += kMetaThreads) {
    keeper[s] = 0x7fffffff;
    children[s] = 0;
    len_old[s] = a.in[o_len(a) + s];
    parent[s] = a.parents[s];
  }
  for (int i = tid; i < a.n_pages; i += kMetaThreads) count[i] = 0;
  __syncthreads();
  for (int s = tid; s < a.S; s += kMetaThreads) {
    const int p = parent[s];
    if (p < -1 || p >= a.S || len_old[s] < 0 || len_old[s] > a.maxp * (int64_t)a.P) atomicMax(&bad, kPgRange);
    else if (p >= 0) {
      atomicMin(&keeper[p], s);
      atomicAdd(&children[p], 1);
    }
  }
  // `bad` is raised again below: every thread reads it before any goes on, so
  // that all take the same branch
  if (refused(&bad)) {
    refuse(a, kPgRange);
    return;
  }
  // holders of every page afterwards, the new copies aside (whole numbers:
  // the order of the additions does not matter)
  for (int p = warp; p < a.S; p += kMetaThreads / 32) {
    const int full = len_old[p] / a.P, used = (len_old[p] + a.P - 1) / a.P, kids = children[p];
    for (int c = lane; c < used; c += 32) {
      const int pg = table_in[(int64_t)p * a.maxp + c];
      // a page that nobody holds could be handed out below
      if (pg < 0 || pg >= a.n_pages || a.in[o_refs(a) + pg] <= 0) atomicMax(&bad, kPgRange);
      else if (kids) atomicAdd(&count[pg], c < full ? kids : 1);
    }
  }
  // copies: slots whose parent's last page is partly filled and kept by another
  int n_copy = 0;
  for (int s0 = 0; s0 < a.S; s0 += kMetaThreads) {
    const int s = s0 + tid;
    int copy = 0;
    if (s < a.S && parent[s] >= 0) copy = len_old[parent[s]] % a.P != 0 && keeper[parent[s]] != s;
    int total;
    block_scan(copy, tmp, &total);
    n_copy += total;
  }
  // pages that become free
  int n_freed = 0;
  for (int i0 = 0; i0 < a.n_pages; i0 += kMetaThreads) {
    const int i = i0 + tid;
    n_freed += __syncthreads_count(i < a.n_pages && a.in[o_refs(a) + i] > 0 && count[i] == 0);
  }
  for (int i = tid; i < n_free; i += kMetaThreads) {
    const int id = a.in[kPageHeader + i];
    if (id < 0 || id >= a.n_pages || a.in[o_refs(a) + id] != 0) atomicMax(&bad, kPgRange);
  }
  const int why_not = refused(&bad), have = n_free + n_freed;
  if (why_not || have > a.n_pages || n_copy > have) {
    refuse(a, why_not || have > a.n_pages ? kPgRange : kPgNoFree);
    return;
  }
  // the old table, where the new one overwrites it
  const int* table_old = table_in;
  if (a.out == a.in) {
    int* stage = a.ws + w_table(a);
    for (int p = warp; p < a.S; p += kMetaThreads / 32) {
      const int used = (len_old[p] + a.P - 1) / a.P;
      for (int c = lane; c < used; c += 32) stage[(int64_t)p * a.maxp + c] = table_in[(int64_t)p * a.maxp + c];
    }
    table_old = stage;
  } else {
    for (int i = tid; i < n_free; i += kMetaThreads) a.out[kPageHeader + i] = a.in[kPageHeader + i];
  }
  if (tid == 0) carry = n_free;
  __syncthreads();
  for (int i0 = 0; i0 < a.n_pages; i0 += kMetaThreads) {
    const int i = i0 + tid;
    const int c = i < a.n_pages ? count[i] : 0;
    const int freed = i < a.n_pages && a.in[o_refs(a) + i] > 0 && c == 0;
    int total;
    const int at = carry + block_scan(freed, tmp, &total);
    if (freed) a.out[kPageHeader + at] = i;
    if (i < a.n_pages) a.out[o_refs(a) + i] = c;
    if (tid == 0) carry += total;
    __syncthreads();
  }
  // copies take the last ids of the list, in the order of the slots
  if (tid == 0) carry = 0;
  __syncthreads();
  for (int s0 = 0; s0 < a.S; s0 += kMetaThreads) {
    const int s = s0 + tid;
    int copy = 0, p = -1;
    if (s < a.S) {
      p = parent[s];
      if (p >= 0) copy = len_old[p] % a.P != 0 && keeper[p] != s;
    }
    int total;
    const int at = carry + block_scan(copy, tmp, &total);
    if (copy) {
      const int last = len_old[p] / a.P;
      const int id = a.out[kPageHeader + have - 1 - at];
      list[at] = table_old[(int64_t)p * a.maxp + last];
      list[most + at] = id;
      list[2 * most + at] = len_old[p] % a.P;
      a.out[o_refs(a) + id] = 1;
    }
    if (s < a.S) a.out[o_len(a) + s] = p >= 0 ? len_old[p] : 0;
    // where this slot's copy is, for the table below
    if (s < a.S) children[s] = copy ? at : -1;
    if (tid == 0) carry += total;
    __syncthreads();
  }
  for (int s = warp; s < a.S; s += kMetaThreads / 32) {
    const int p = parent[s], used = p >= 0 ? (len_old[p] + a.P - 1) / a.P : 0, at = children[s];
    int* row = a.out + o_table(a) + (int64_t)s * a.maxp;
    for (int c = lane; c < a.maxp; c += 32) {
      int v = -1;
      if (c < used) v = c == used - 1 && at >= 0 ? list[most + at] : table_old[(int64_t)p * a.maxp + c];
      row[c] = v;
    }
  }
  __syncthreads();
  for (int i = have - n_copy + tid; i < a.n_pages; i += kMetaThreads) a.out[kPageHeader + i] = -1;
  header_out(a, status, have - n_copy, n_copy);
}

// --- compact ------------------------------------------------------------

__global__ void __launch_bounds__(kMetaThreads) compact_state_kernel(PgArgs a) {
  let_dependents_launch();
  __shared__ int tmp[33];
  __shared__ int bad, carry_s, carry_d;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int status = a.in[0];
  const int* refs = a.in + o_refs(a);
  int* to = a.ws + 16;
  int* list = a.ws + w_list(a);
  const int64_t most = list_most(a.n_pages, a.S);
  if (tid == 0) { bad = kPgOk; carry_s = carry_d = 0; }
  __syncthreads();
  for (int s = warp; s < a.S; s += kMetaThreads / 32) {
    const int len = a.in[o_len(a) + s];
    if (len < 0 || len > a.maxp * (int64_t)a.P) {
      if (lane == 0) atomicMax(&bad, kPgRange);
      continue;
    }
    for (int c = lane; c < (len + a.P - 1) / a.P; c += 32) {
      const int pg = a.in[o_table(a) + (int64_t)s * a.maxp + c];
      if (pg < 0 || pg >= a.n_pages || refs[pg] <= 0) atomicMax(&bad, kPgRange);
    }
  }
  int n = 0;
  for (int i0 = 0; i0 < a.n_pages; i0 += kMetaThreads) {
    const int i = i0 + tid;
    n += __syncthreads_count(i < a.n_pages && refs[i] > 0);
  }
  if (refused(&bad)) {
    refuse(a, kPgRange);
    return;
  }
  // i-th used page at n or behind, i-th free page below n: as many of the one
  // as of the other
  for (int i0 = 0; i0 < a.n_pages; i0 += kMetaThreads) {
    const int i = i0 + tid;
    const bool live = i < a.n_pages && refs[i] > 0;
    const int src = live && i >= n, dst = i < n && !live;
    int total;
    const int at = block_scan(src + (dst << 16), tmp, &total);
    if (src) list[carry_s + (at & 0xffff)] = i;
    if (dst) list[most + carry_d + (at >> 16)] = i;
    if (i < a.n_pages) to[i] = i;
    __syncthreads();
    if (tid == 0) { carry_s += total & 0xffff; carry_d += total >> 16; }
    __syncthreads();
  }
  const int moves = carry_s;
  for (int i = tid; i < moves; i += kMetaThreads) {
    to[list[i]] = list[most + i];
    list[2 * most + i] = a.P;
  }
  if (a.out != a.in)
    for (int i = tid; i < n; i += kMetaThreads) a.out[o_refs(a) + i] = refs[i];
  __syncthreads();
  for (int i = tid; i < moves; i += kMetaThreads) a.out[o_refs(a) + list[most + i]] = refs[list[i]];
  __syncthreads();
  for (int i = n + tid; i < a.n_pages; i += kMetaThreads) a.out[o_refs(a) + i] = 0;
  for (int i = tid; i < a.n_pages; i += kMetaThreads)
    a.out[kPageHeader + i] = i < a.n_pages - n ? a.n_pages - 1 - i : -1;
  for (int s = warp; s < a.S; s += kMetaThreads / 32) {
    const int len = a.in[o_len(a) + s], used = (len + a.P - 1) / a.P;
    const int* row = a.in + o_table(a) + (int64_t)s * a.maxp;
    int* row_out = a.out + o_table(a) + (int64_t)s * a.maxp;
    for (int c = lane; c < a.maxp; c += 32) row_out[c] = c < used ? to[row[c]] : -1;
    __syncwarp();
    if (lane == 0) a.out[o_len(a) + s] = len;
  }
  header_out(a, status, a.n_pages - n, moves);
}

// Moves the listed pages' rows: a CTA takes 32 KB of a (page, layer, side) at a
// time (H runs of contiguous rows), eight 16-byte pieces a thread in flight.
// Sources and destinations of a list never overlap.
constexpr int kChunk = 256 * 8;

__global__ void __launch_bounds__(256) copy_pages_kernel(PgArgs a) {
  wait_for_primary();
  const int items = a.ws[0];
  const int* list = a.ws + w_list(a);
  const int64_t most = list_most(a.n_pages, a.S);
  const int page16 = a.P * a.row16, chunks = (a.H * page16 + kChunk - 1) / kChunk, per = 2 * a.L * chunks;
  const int64_t units = (int64_t)items * per;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int i = (int)(u / per), x = (int)(u % per), ls = x / chunks;
    const int n = list[2 * most + i] * a.row16, total = n * a.H;      // pieces of a head, of all
    const int c0 = (x % chunks) * kChunk + threadIdx.x;
    if (c0 >= total) continue;
    const int64_t base = (int64_t)(ls >> 1) * a.n_pages;
    const uint4* from = a.pool[ls & 1] + (base + list[i]) * a.H * page16;
    uint4* to = a.pool[ls & 1] + (base + list[most + i]) * a.H * page16;
    // piece c is at c, or, of a page that is not full, head by head
    int at[8], h = 0, r = c0;
    if (n < page16) { h = c0 / n; r = c0 % n; }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      at[k] = h * page16 + r;
      r += 256;
      if (n < page16)
        while (r >= n) { r -= n; ++h; }
    }
    uint4 v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (c0 + 256 * k < total) v[k] = from[at[k]];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (c0 + 256 * k < total) to[at[k]] = v[k];
  }
}

int make_args(const anchorkv_pages* pg, PgArgs* a) {
  if (!pg) return ANCHORKV_EINVAL;
  if (pg->head_dim != kD) return ANCHORKV_EUNSUPPORTED;
  if (pg->dtype != ANCHORKV_FP32 && pg->dtype != ANCHORKV_BF16) return ANCHORKV_EUNSUPPORTED;
  if (pg->n_pages < 1 || pg->n_pages > (1 << 20) || pg->n_slots < 1 || pg->n_slots > 4096 || pg->max_pages < 1 ||
      pg->max_pages > 65536 || pg->n_layers < 1 || pg->n_layers > 1024 || pg->n_kv_heads < 1 || pg->n_kv_heads > 1024)
    return ANCHORKV_EINVAL;
  if (pg->page_size != 16 && pg->page_size != 32 && pg->page_size != 64 && pg->page_size != 128)
    return ANCHORKV_EINVAL;
  *a = PgArgs{};
  a->n_pages = pg->n_pages; a->P = pg->page_size; a->S = pg->n_slots; a->maxp = pg->max_pages;
  a->L = pg->n_layers; a->H = pg->n_kv_heads;
  a->row16 = kD * (pg->dtype == ANCHORKV_BF16 ? 2 : 4) / 16;
  return ANCHORKV_OK;
}

int64_t copy_chunks(const PgArgs& a) { return ((int64_t)a.H * a.P * a.row16 + kChunk - 1) / kChunk; }

int64_t ws_ints(const PgArgs& a) { return w_table(a) + (int64_t)a.S * a.maxp; }

int op_args(const anchorkv_pages* pg, const int32_t* in, int32_t* out, void* K, void* V, void* ws, size_t ws_bytes,
            PgArgs* a) {
  const int st = make_args(pg, a);
  if (st) return st;
  if (!in || !out || !K || !V || K == V || !ws) return ANCHORKV_EINVAL;
  if (((uintptr_t)in | (uintptr_t)out | (uintptr_t)K | (uintptr_t)V | (uintptr_t)ws) & 15) return ANCHORKV_EINVAL;
  if ((int64_t)ws_bytes < 4 * ws_ints(*a)) return ANCHORKV_ENOSPC;
  a->in = in; a->out = out; a->ws = (int*)ws;
  a->pool[0] = (uint4*)K; a->pool[1] = (uint4*)V;
  return check_device();
}

// The row kernel as a programmatic dependent of the state kernel before it.
template <typename K>
int launch_rows(K kernel, int64_t grid, const PgArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? ANCHORKV_OK : ANCHORKV_ECUDA;
}

constexpr int64_t kRowGrid = 148 * 8;   // eight 256-thread CTAs fill an SM

}  // namespace

int pages_tokens(const anchorkv_pages* pg, int64_t* most) {
  PgArgs a;
  const int st = make_args(pg, &a);
  if (st == ANCHORKV_OK) *most = (int64_t)a.maxp * a.P;
  return st;
}

}  // namespace akv

using namespace akv;

extern "C" {

int anchorkv_pages_state_bytes(const anchorkv_pages* pg, size_t* bytes) {
  if (!bytes) return ANCHORKV_EINVAL;
  PgArgs a;
  const int st = make_args(pg, &a);
  if (st) return st;
  *bytes = 4 * (size_t)state_ints(a);
  return ANCHORKV_OK;
}

int anchorkv_pages_workspace_bytes(const anchorkv_pages* pg, size_t* bytes) {
  if (!bytes) return ANCHORKV_EINVAL;
  PgArgs a;
  const int st = make_args(pg, &a);
  if (st) return st;
  *bytes = 4 * (size_t)ws_ints(a);
  return ANCHORKV_OK;
}

int anchorkv_pages_init(const anchorkv_pages* pg, int32_t* state, void* stream) {
  PgArgs a;
  int st = make_args(pg, &a);
  if (st) return st;
  if (!state || ((uintptr_t)state & 15)) return ANCHORKV_EINVAL;
  st = check_device();
  if (st) return st;
  a.out = state;
  cudaStream_t s = (cudaStream_t)stream;
  stage_begin(kStPages, s);
  const int64_t grid = std::min<int64_t>((state_ints(a) + kMetaThreads - 1) / kMetaThreads, 148);
  pages_init_kernel<<<(unsigned)grid, kMetaThreads, 0, s>>>(a);
  if (cudaGetLastError() != cudaSuccess) return ANCHORKV_ECUDA;
  stage_end(kStPages, s, 1);
  return ANCHORKV_OK;
}

int anchorkv_pages_commit(const anchorkv_pages* pg, const int32_t* state_in, int32_t* state_out, void* K_pages,
                          void* V_pages, const void* K_new, const void* V_new, int32_t batch, int32_t n_draft,
                          const int32_t* path, const int32_t* n_accept, void* ws, size_t ws_bytes, void* stream) {
  PgArgs a;
  int st = make_args(pg, &a);
  if (st) return st;
  if (batch < 0 || batch > a.S || n_draft < 1 || n_draft > 65536) return ANCHORKV_EINVAL;
  if (batch > 0 && (!K_new || !V_new || !n_accept)) return ANCHORKV_EINVAL;       // of no sequences there are no rows
  if ((((uintptr_t)K_new | (uintptr_t)V_new) & 15)) return ANCHORKV_EINVAL;
  if (((uintptr_t)path | (uintptr_t)n_accept) & 3) return ANCHORKV_EINVAL;
  st = op_args(pg, state_in, state_out, K_pages, V_pages, ws, ws_bytes, &a);
  if (st) return st;
  a.fresh[0] = (const uint4*)K_new; a.fresh[1] = (const uint4*)V_new;
  a.batch = batch; a.T = n_draft; a.path = path; a.n_accept = n_accept;
  cudaStream_t s = (cudaStream_t)stream;
  stage_begin(kStPages, s);
  commit_state_kernel<<<1, kMetaThreads, 0, s>>>(a);
  if (cudaGetLastError() != cudaSuccess) return ANCHORKV_ECUDA;
  if (batch > 0) {
    const int64_t units = (int64_t)batch * n_draft * 2 * a.L;
    st = launch_rows(commit_rows_kernel, std::min<int64_t>((units + 7) / 8, kRowGrid), a, s);
  }
  stage_end(kStPages, s, batch > 0 ? 2 : 1);
  return st;
}

int anchorkv_pages_fork(const anchorkv_pages* pg, const int32_t* state_in, int32_t* state_out, void* K_pages,
                        void* V_pages, const int32_t* parents, void* ws, size_t ws_bytes, void* stream) {
  PgArgs a;
  if (!parents || ((uintptr_t)parents & 3)) return ANCHORKV_EINVAL;
  int st = op_args(pg, state_in, state_out, K_pages, V_pages, ws, ws_bytes, &a);
  if (st) return st;
  a.parents = parents;
  cudaStream_t s = (cudaStream_t)stream;
  // 48 KB without an attribute, the kernel's own arrays among them
  const int smem = 4 * a.S * 4;
  if (smem > 32 * 1024 &&
      cudaFuncSetAttribute(fork_state_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return ANCHORKV_ECUDA;
  stage_begin(kStPages, s);
  fork_state_kernel<<<1, kMetaThreads, smem, s>>>(a);
  if (cudaGetLastError() != cudaSuccess) return ANCHORKV_ECUDA;
  st = launch_rows(copy_pages_kernel, std::min<int64_t>((int64_t)a.S * 2 * a.L * copy_chunks(a), kRowGrid), a, s);
  stage_end(kStPages, s, 2);
  return st;
}

int anchorkv_pages_compact(const anchorkv_pages* pg, const int32_t* state_in, int32_t* state_out, void* K_pages,
                           void* V_pages, void* ws, size_t ws_bytes, void* stream) {
  PgArgs a;
  int st = op_args(pg, state_in, state_out, K_pages, V_pages, ws, ws_bytes, &a);
  if (st) return st;
  cudaStream_t s = (cudaStream_t)stream;
  stage_begin(kStPages, s);
  compact_state_kernel<<<1, kMetaThreads, 0, s>>>(a);
  if (cudaGetLastError() != cudaSuccess) return ANCHORKV_ECUDA;
  st = launch_rows(copy_pages_kernel, std::min<int64_t>((int64_t)(a.n_pages / 2 + 1) * 2 * a.L * copy_chunks(a), kRowGrid), a, s);
  stage_end(kStPages, s, 2);
  return st;
}

}  // extern "C"
