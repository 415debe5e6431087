"""Thin PyTorch binding of the AnchorKV C ABI.

PyTorch supplies device memory and the current CUDA stream; every step of the
codec runs in libanchorkv.so.  Functions mirror the C entry points:
``anchorkv_bytes``, ``compress`` (anchorkv_compress), ``decode_attn``
(anchorkv_decode_attn), ``reconstruct`` (anchorkv_reconstruct).
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import capi

_DT = {"fp32": capi.FP32, "bf16": capi.BF16}

# anchorkv_params.mode bits (include/anchorkv.h)
MODE_KEY_QUERIES = 0x1       # Q_obs may be None: the trailing W keys serve as the observation queries
MODE_RANK_SHIFT = 1
RANK_UTILITY, RANK_RESIDUAL_NORM, RANK_ATTENTION, RANK_COSINE, RANK_RANDOM = 0, 1, 2, 3, 4
MODE_NAIVE_CODEC = 0x10      # 2-bit codec without the sign flip and Hadamard rotation


def mode_bits(key_queries: bool = False, rank: int = RANK_UTILITY, naive_codec: bool = False) -> int:
    """The anchorkv_params.mode value of a combination of options."""
    return (MODE_KEY_QUERIES if key_queries else 0) | (rank << MODE_RANK_SHIFT) | (MODE_NAIVE_CODEC if naive_codec else 0)
_TORCH_DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


@dataclass
class AnchorKVParams:
    """One layer's codec parameters (defaults: the pages' hyper-parameters)."""
    n_tokens: int
    n_kv_heads: int = 8
    n_q_heads: int = 32
    theta: float = 0.05
    head_dim: int = 128
    window: int = 32
    dtype: str = "bf16"
    seed: int = 0
    layer: int = 0
    anchor_div: int = 128
    rho_num: int = 7
    rho_den: int = 10
    pool_kernel: int = 7
    mode: int = 0                # mode_bits(...); compress and decode of one layout use the same

    def c(self) -> capi.Params:
        return capi.Params(self.n_tokens, self.head_dim, self.n_kv_heads, self.n_q_heads, self.window,
                           _DT[self.dtype], float(self.theta), self.seed, self.layer, self.anchor_div,
                           self.rho_num, self.rho_den, self.pool_kernel, self.mode)

    @property
    def torch_dtype(self) -> torch.dtype:
        return _TORCH_DT[self.dtype]


def anchorkv_bytes(p: AnchorKVParams) -> dict:
    L = capi.Layout()
    capi.check("anchorkv_bytes", capi.lib().anchorkv_bytes(ctypes.byref(p.c()), ctypes.byref(L)))
    return {name: getattr(L, name) for name, _ in capi.Layout._fields_}


def compress_workspace(p: AnchorKVParams) -> dict:
    v = capi.WorkspaceView()
    capi.check("anchorkv_compress_workspace",
               capi.lib().anchorkv_compress_workspace(ctypes.byref(p.c()), ctypes.byref(v)))
    return {name: getattr(v, name) for name, _ in capi.WorkspaceView._fields_}


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _ptr(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(t.data_ptr() if t is not None else 0)


def _check_tensor(name, t, shape, dtype):
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


def compress(p: AnchorKVParams, K: torch.Tensor, V: torch.Tensor, Q_obs: torch.Tensor | None,
             out: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Compress one layer.  K, V: [H, N, D]; Q_obs: [H_q, W, D] (CUDA, p.dtype),
    or None with the key-as-query mode.
    Returns (compressed uint8 tensor of layout.total_bytes, workspace)."""
    H, N, D, W = p.n_kv_heads, p.n_tokens, p.head_dim, p.window
    _check_tensor("K", K, (H, N, D), p.torch_dtype)
    _check_tensor("V", V, (H, N, D), p.torch_dtype)
    if Q_obs is not None or not (p.mode & MODE_KEY_QUERIES):
        _check_tensor("Q_obs", Q_obs, (p.n_q_heads, W, D), p.torch_dtype)
    L = anchorkv_bytes(p)
    ws = compress_workspace(p)
    if out is None:
        out = torch.empty(L["total_bytes"], dtype=torch.uint8, device=K.device)
    if workspace is None:
        workspace = torch.empty(ws["total_bytes"], dtype=torch.uint8, device=K.device)
    st = capi.lib().anchorkv_compress(ctypes.byref(p.c()), _ptr(K), _ptr(V), _ptr(Q_obs), _ptr(out),
                                      out.numel(), _ptr(workspace), workspace.numel(), _stream(K.device))
    capi.check("anchorkv_compress", st)
    return out, workspace


def compress_host_staging_bytes(p: AnchorKVParams) -> int:
    """Device staging bytes compress_host needs (K, V, Q_obs and the layout)."""
    n = ctypes.c_size_t()
    capi.check("anchorkv_compress_host_staging_bytes",
               capi.lib().anchorkv_compress_host_staging_bytes(ctypes.byref(p.c()), ctypes.byref(n)))
    return n.value


def _check_host(name, t, shape, dtype):
    if t.device.type != "cpu":
        raise ValueError(f"{name} must be a host (CPU) tensor")
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


def compress_host(p: AnchorKVParams, K: torch.Tensor, V: torch.Tensor, Q_obs: torch.Tensor | None,
                  out: torch.Tensor, staging: torch.Tensor, workspace: torch.Tensor, device="cuda") -> torch.Tensor:
    """Compress one layer from host buffers through anchorkv_compress_host: the
    library copies K, V, Q_obs (host, ideally pinned) into `staging` (device),
    compresses there and copies the layout into `out` (host uint8), all on the
    current stream of `device`.  `out` is valid once that stream has run."""
    H, N, D, W = p.n_kv_heads, p.n_tokens, p.head_dim, p.window
    _check_host("K", K, (H, N, D), p.torch_dtype)
    _check_host("V", V, (H, N, D), p.torch_dtype)
    if Q_obs is not None or not (p.mode & MODE_KEY_QUERIES):
        _check_host("Q_obs", Q_obs, (p.n_q_heads, W, D), p.torch_dtype)
    if out.device.type != "cpu" or out.dtype != torch.uint8:
        raise ValueError("out must be a host uint8 tensor")
    st = capi.lib().anchorkv_compress_host(ctypes.byref(p.c()), _ptr(K), _ptr(V), _ptr(Q_obs), _ptr(out),
                                           out.numel(), _ptr(staging), staging.numel(), _ptr(workspace),
                                           workspace.numel(), _stream(torch.device(device)))
    capi.check("anchorkv_compress_host", st)
    return out


def decode_workspace_bytes(p: AnchorKVParams, batch: int) -> int:
    n = ctypes.c_size_t()
    capi.check("anchorkv_decode_workspace_bytes",
               capi.lib().anchorkv_decode_workspace_bytes(ctypes.byref(p.c()), batch, ctypes.byref(n)))
    return n.value


def decode_attn(p: AnchorKVParams, compressed: torch.Tensor, q: torch.Tensor,
                K_tail: torch.Tensor | None = None, V_tail: torch.Tensor | None = None, tail_len: int = 0,
                out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Decode attention.  compressed: uint8 [batch, stride] (one layout per
    row) or [total_bytes]; q: [batch, H_q, D]; tails [batch, H, T_cap, D].
    Returns fp32 [batch, H_q, D]."""
    if compressed.dim() == 1:
        # one layout: the stride never steps to a second sequence, it only has
        # to satisfy the ABI (>= total bytes, a multiple of 16)
        batch, stride = 1, (compressed.numel() + 15) // 16 * 16
    else:
        batch, stride = compressed.shape
    _check_tensor("q", q, (batch, p.n_q_heads, p.head_dim), p.torch_dtype)
    cap = 0
    if K_tail is not None:
        cap = K_tail.shape[2]
        _check_tensor("K_tail", K_tail, (batch, p.n_kv_heads, cap, p.head_dim), p.torch_dtype)
        _check_tensor("V_tail", V_tail, (batch, p.n_kv_heads, cap, p.head_dim), p.torch_dtype)
    if out is None:
        out = torch.empty(batch, p.n_q_heads, p.head_dim, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty(decode_workspace_bytes(p, batch), dtype=torch.uint8, device=q.device)
    st = capi.lib().anchorkv_decode_attn(ctypes.byref(p.c()), _ptr(compressed), stride, batch, _ptr(q),
                                         _ptr(K_tail), _ptr(V_tail), tail_len, cap, _ptr(out), _ptr(workspace),
                                         workspace.numel(), _stream(q.device))
    capi.check("anchorkv_decode_attn", st)
    return out


def decode_rope_workspace_bytes(p: AnchorKVParams, batch: int) -> int:
    n = ctypes.c_size_t()
    capi.check("anchorkv_decode_rope_workspace_bytes",
               capi.lib().anchorkv_decode_rope_workspace_bytes(ctypes.byref(p.c()), batch, ctypes.byref(n)))
    return n.value


def decode_attn_rope(p: AnchorKVParams, compressed: torch.Tensor, q: torch.Tensor, rope_base: float,
                     K_tail: torch.Tensor | None = None, V_tail: torch.Tensor | None = None, tail_len: int = 0,
                     out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Decode attention over layouts whose keys were stored before the rotary
    map (anchorkv_decode_attn_rope): cached token t at position t, tail token
    i at N + i, the query at N + tail_len.  Shapes as decode_attn."""
    if compressed.dim() == 1:
        batch, stride = 1, (compressed.numel() + 15) // 16 * 16
    else:
        batch, stride = compressed.shape
    _check_tensor("q", q, (batch, p.n_q_heads, p.head_dim), p.torch_dtype)
    cap = 0
    if K_tail is not None:
        cap = K_tail.shape[2]
        _check_tensor("K_tail", K_tail, (batch, p.n_kv_heads, cap, p.head_dim), p.torch_dtype)
        _check_tensor("V_tail", V_tail, (batch, p.n_kv_heads, cap, p.head_dim), p.torch_dtype)
    if out is None:
        out = torch.empty(batch, p.n_q_heads, p.head_dim, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty(decode_rope_workspace_bytes(p, batch), dtype=torch.uint8, device=q.device)
    st = capi.lib().anchorkv_decode_attn_rope(ctypes.byref(p.c()), _ptr(compressed), stride, batch, _ptr(q),
                                              _ptr(K_tail), _ptr(V_tail), tail_len, cap, float(rope_base),
                                              _ptr(out), _ptr(workspace), workspace.numel(), _stream(q.device))
    capi.check("anchorkv_decode_attn_rope", st)
    return out


def decode_config(p: AnchorKVParams, batch: int) -> dict:
    """Launch shape of decode_attn on the current device: token slices (CTAs)
    per (sequence, head) of the slice decode (0: the split-token kernels run)
    and shared memory per CTA."""
    c, m = ctypes.c_int32(), ctypes.c_int32()
    capi.check("anchorkv_decode_config",
               capi.lib().anchorkv_decode_config(ctypes.byref(p.c()), batch, ctypes.byref(c), ctypes.byref(m)))
    return {"slices": c.value, "smem_bytes": m.value}


NOALLOC_SCRATCH_BYTES = 32 << 20   # ANCHORKV_DECODE_NOALLOC_SCRATCH_BYTES in include/anchorkv.h


def decode_attn_noalloc(p: AnchorKVParams, compressed: torch.Tensor, q: torch.Tensor, out: torch.Tensor,
                        K_tail: torch.Tensor | None = None, V_tail: torch.Tensor | None = None,
                        tail_len: int = 0) -> torch.Tensor:
    """Decode attention that allocates no device memory: the library's
    per-device scratch array stands in for the workspace, and `out` must be
    supplied.  For callers that cannot allocate while decoding (all free HBM
    given to a KV-cache pool, no device allocator, or no room for the
    device-wide synchronisation of cudaMalloc/cudaFree).  Calls that overlap
    on the GPU share the scratch and race; sizes whose decode workspace
    exceeds NOALLOC_SCRATCH_BYTES raise (ANCHORKV_ENOSPC)."""
    if compressed.dim() == 1:
        # one layout: the stride never steps to a second sequence, it only has
        # to satisfy the ABI (>= total bytes, a multiple of 16)
        batch, stride = 1, (compressed.numel() + 15) // 16 * 16
    else:
        batch, stride = compressed.shape
    _check_tensor("q", q, (batch, p.n_q_heads, p.head_dim), p.torch_dtype)
    _check_tensor("out", out, (batch, p.n_q_heads, p.head_dim), torch.float32)
    cap = 0
    if K_tail is not None:
        cap = K_tail.shape[2]
        _check_tensor("K_tail", K_tail, (batch, p.n_kv_heads, cap, p.head_dim), p.torch_dtype)
        _check_tensor("V_tail", V_tail, (batch, p.n_kv_heads, cap, p.head_dim), p.torch_dtype)
    st = capi.lib().anchorkv_decode_attn_noalloc(ctypes.byref(p.c()), _ptr(compressed), stride, batch, _ptr(q),
                                                 _ptr(K_tail), _ptr(V_tail), tail_len, cap, _ptr(out),
                                                 _stream(q.device))
    if st == capi.ENOSPC:
        raise capi.AnchorKVError(
            f"anchorkv_decode_attn_noalloc (decode workspace {decode_workspace_bytes(p, batch)} B exceeds the "
            f"{NOALLOC_SCRATCH_BYTES} B static scratch)", st)
    capi.check("anchorkv_decode_attn_noalloc", st)
    return out


@dataclass
class PageSpec:
    """Sizes of a page pool of exact decode-time tokens (anchorkv_pages): the
    pool tensors are [n_layers, n_pages, n_kv_heads, page_size, head_dim]."""
    n_pages: int
    page_size: int = 64
    n_slots: int = 1
    max_pages: int = 64
    n_layers: int = 1
    n_kv_heads: int = 8
    dtype: str = "bf16"
    head_dim: int = 128

    def c(self) -> capi.Pages:
        return capi.Pages(self.n_pages, self.page_size, self.n_slots, self.max_pages, self.n_layers, self.n_kv_heads,
                          self.head_dim, _DT[self.dtype])

    @property
    def torch_dtype(self) -> torch.dtype:
        return _TORCH_DT[self.dtype]

    @property
    def pool_shape(self) -> torch.Size:
        return torch.Size((self.n_layers, self.n_pages, self.n_kv_heads, self.page_size, self.head_dim))

    @property
    def state_numel(self) -> int:
        return 16 + 2 * self.n_pages + self.n_slots * (1 + self.max_pages)


def _call(device, fn, *args) -> int:
    """fn(*args, stream) with `device` current, on its current stream.  The
    raw stream handle is a fraction of the cost of a Stream object, and the
    smallest calls are bound by the host."""
    index = device.index
    if index == torch.cuda.current_device():
        return fn(*args, torch._C._cuda_getCurrentRawStream(index))
    with torch.cuda.device(index):
        return fn(*args, torch._C._cuda_getCurrentRawStream(index))


def _require(name, t, shape, dtype, device):
    """As _check_tensor, on one device."""
    if t.shape != shape or t.dtype is not dtype or t.device != device or not t.is_contiguous():
        _check_tensor(name, t, shape, dtype)
        raise ValueError(f"{name} is on {t.device}, not on {device}")


def pages_state_bytes(pages: PageSpec) -> int:
    n = ctypes.c_size_t()
    capi.check("anchorkv_pages_state_bytes",
               capi.lib().anchorkv_pages_state_bytes(ctypes.byref(pages.c()), ctypes.byref(n)))
    return n.value


def pages_workspace_bytes(pages: PageSpec) -> int:
    """Scratch of pages_commit, pages_fork and pages_compact."""
    n = ctypes.c_size_t()
    capi.check("anchorkv_pages_workspace_bytes",
               capi.lib().anchorkv_pages_workspace_bytes(ctypes.byref(pages.c()), ctypes.byref(n)))
    return n.value


def pages_init(pages: PageSpec, device="cuda", state: torch.Tensor | None = None) -> torch.Tensor:
    """A page state (int32) in which every page is free and every slot empty."""
    if state is None:
        state = torch.empty(pages_state_bytes(pages) // 4, dtype=torch.int32, device=device)
    _check_tensor("state", state, (pages.state_numel,), torch.int32)
    capi.check("anchorkv_pages_init", _call(state.device, capi.lib().anchorkv_pages_init, pages.c(), state.data_ptr()))
    return state


def pages_view(pages: PageSpec, state: torch.Tensor) -> dict:
    """Views into a page state: status, n_free, free, refs, len, table."""
    n, s, at = pages.n_pages, pages.n_slots, 16
    return {"status": state[0], "n_free": state[1], "free": state[at:at + n], "refs": state[at + n:at + 2 * n],
            "len": state[at + 2 * n:at + 2 * n + s], "table": state[at + 2 * n + s:].view(s, pages.max_pages)}


def _pages_args(pages, state, K_pages, V_pages, state_out, workspace):
    """Checked state, pools and scratch: (C sizes, state_out, workspace, device)."""
    dev, n, shape, dt = state.device, torch.Size((pages.state_numel,)), pages.pool_shape, pages.torch_dtype
    if dev.type != "cuda":
        raise ValueError("state must be a CUDA tensor")
    _require("state", state, n, torch.int32, dev)
    _require("K_pages", K_pages, shape, dt, dev)
    _require("V_pages", V_pages, shape, dt, dev)
    if state_out is None:
        state_out = state
    elif state_out is not state:
        _require("state_out", state_out, n, torch.int32, dev)
    if workspace is None:
        workspace = torch.empty(pages_workspace_bytes(pages), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {dev}")
    return pages.c(), state_out, workspace, dev


def pages_commit(pages: PageSpec, state: torch.Tensor, K_pages: torch.Tensor, V_pages: torch.Tensor,
                 K_new: torch.Tensor, V_new: torch.Tensor, n_accept: torch.Tensor, path: torch.Tensor | None = None,
                 state_out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Append rows path[b, :n_accept[b]] (path None: 0, 1, ...) of the drafts
    K_new, V_new [n_layers, batch, n_draft, H, D] to slot b, in every layer.
    n_accept: int32 [batch]; path: int32 [batch, n_draft].  Updates the state
    in place unless state_out is given; returns the new state.  Whether the
    operation was possible is in the state's status word (read_status)."""
    pg, state_out, workspace, dev = _pages_args(pages, state, K_pages, V_pages, state_out, workspace)
    if K_new.dim() != 5:
        raise ValueError(f"K_new: expected [n_layers, batch, n_draft, H, D], got {tuple(K_new.shape)}")
    batch, drafts = K_new.shape[1:3]
    shape = torch.Size((pages.n_layers, batch, drafts, pages.n_kv_heads, pages.head_dim))
    _require("K_new", K_new, shape, pages.torch_dtype, dev)
    _require("V_new", V_new, shape, pages.torch_dtype, dev)
    _require("n_accept", n_accept, torch.Size((batch,)), torch.int32, dev)
    if path is not None:
        _require("path", path, torch.Size((batch, drafts)), torch.int32, dev)
    st = _call(dev, capi.lib().anchorkv_pages_commit, pg, state.data_ptr(), state_out.data_ptr(), K_pages.data_ptr(),
               V_pages.data_ptr(), K_new.data_ptr(), V_new.data_ptr(), batch, drafts,
               path.data_ptr() if path is not None else None, n_accept.data_ptr(), workspace.data_ptr(),
               workspace.nbytes)
    capi.check("anchorkv_pages_commit", st)
    return state_out


def pages_fork(pages: PageSpec, state: torch.Tensor, K_pages: torch.Tensor, V_pages: torch.Tensor,
               parents: torch.Tensor, state_out: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Slot s becomes a copy of what slot parents[s] (int32 [n_slots]) was; -1
    empties it.  Full pages are shared, a partly filled last page is copied
    for all copies but the first.  Returns the new state."""
    pg, state_out, workspace, dev = _pages_args(pages, state, K_pages, V_pages, state_out, workspace)
    _require("parents", parents, torch.Size((pages.n_slots,)), torch.int32, dev)
    st = _call(dev, capi.lib().anchorkv_pages_fork, pg, state.data_ptr(), state_out.data_ptr(), K_pages.data_ptr(),
               V_pages.data_ptr(), parents.data_ptr(), workspace.data_ptr(), workspace.nbytes)
    capi.check("anchorkv_pages_fork", st)
    return state_out


def pages_compact(pages: PageSpec, state: torch.Tensor, K_pages: torch.Tensor, V_pages: torch.Tensor,
                  state_out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Move the pages in use to the front of the pool.  Returns the new state."""
    pg, state_out, workspace, dev = _pages_args(pages, state, K_pages, V_pages, state_out, workspace)
    st = _call(dev, capi.lib().anchorkv_pages_compact, pg, state.data_ptr(), state_out.data_ptr(), K_pages.data_ptr(),
               V_pages.data_ptr(), workspace.data_ptr(), workspace.nbytes)
    capi.check("anchorkv_pages_compact", st)
    return state_out


def tree_workspace_bytes(p: AnchorKVParams, batch: int, drafts: int, pages: PageSpec | None = None) -> int:
    """Scratch of tree_attn for this many sequences and drafts; it serves fewer
    of either too, though such a call's own bytes may be more and make it faster."""
    n = ctypes.c_size_t()
    pg = ctypes.byref(pages.c()) if pages is not None else None
    capi.check("anchorkv_tree_workspace_bytes",
               capi.lib().anchorkv_tree_workspace_bytes(ctypes.byref(p.c()), batch, drafts, pg, ctypes.byref(n)))
    return n.value


def _row_strides(name, t, shape, dtype, device):
    """(sequence, token) strides of a [batch, T, heads, D] tensor whose heads
    are contiguous; a dimension of one element has no stride to speak of."""
    if t.shape != shape or t.dtype is not dtype or t.device != device:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)} on {device}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    batch, drafts, heads, D = shape
    seq, tok, head, one = t.stride()
    if one != 1 or (heads > 1 and head != D):
        raise ValueError(f"{name}: heads must be contiguous, got strides {t.stride()}")
    if drafts == 1:
        tok = heads * D
    return seq if batch > 1 else drafts * tok, tok


def tree_attn(p: AnchorKVParams, compressed: torch.Tensor | None, q: torch.Tensor, K_new: torch.Tensor,
              V_new: torch.Tensor, n_new: torch.Tensor | None = None, mask: torch.Tensor | None = None,
              layout_of: torch.Tensor | None = None, pages: PageSpec | None = None, state: torch.Tensor | None = None,
              K_pages: torch.Tensor | None = None, V_pages: torch.Tensor | None = None,
              out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Attention for a tree of drafted tokens (anchorkv_tree_attn).
    q: [batch, T, H_q, D] and K_new, V_new: [batch, T, H, D] of the drafts, T <= 64
    (sequence strides are free and token strides from a row of all heads up,
    e.g. slices of a fused projection);
    compressed: uint8 [n_layouts, stride] or [total_bytes], or None;
    layout_of: int32 [batch], the layout of each sequence (default: b);
    n_new: int32 [batch], drafts of each sequence (default T); mask: int64
    [batch, T], bit i of mask[b, t] = draft t sees draft i (default: a chain);
    pages, state, K_pages, V_pages: one layer's slice [n_pages, H, page_size, D]
    of the pools with the exact tokens, slot b = sequence b.
    Returns [batch, T, H_q, D] of p.dtype; rows t >= n_new[b] of `out` stay as
    they are (zero when out is not given)."""
    if q.dim() != 4:
        raise ValueError(f"q: expected [batch, n_draft, H_q, D], got {tuple(q.shape)}")
    batch, drafts = q.shape[:2]
    H, Hq, D, dt, dev = p.n_kv_heads, p.n_q_heads, p.head_dim, p.torch_dtype, q.device
    if dev.type != "cuda":
        raise ValueError("q must be a CUDA tensor")
    L, pc = capi.lib(), p.c()
    shape, kv_shape, b_shape = torch.Size((batch, drafts, Hq, D)), torch.Size((batch, drafts, H, D)), torch.Size((batch,))
    t = capi.Tree(batch=batch, n_draft=drafts)
    t.q_seq_stride, t.q_tok_stride = _row_strides("q", q, shape, dt, dev)
    t.new_seq_stride, t.new_tok_stride = strides = _row_strides("K_new", K_new, kv_shape, dt, dev)
    if _row_strides("V_new", V_new, kv_shape, dt, dev) != strides:
        raise ValueError(f"K_new and V_new: unequal strides {K_new.stride()} and {V_new.stride()}")
    if compressed is not None:
        if compressed.device != dev or compressed.dtype != torch.uint8 or not compressed.is_contiguous():
            raise ValueError(f"compressed must be a contiguous uint8 tensor on {dev}")
        size = compressed.shape[-1]
        lay = capi.Layout()
        capi.check("anchorkv_bytes", L.anchorkv_bytes(pc, lay))
        if size < lay.total_bytes:
            raise ValueError(f"compressed: {size} bytes are less than a layout ({lay.total_bytes})")
        t.n_layouts, t.seq_stride_bytes = (1, (size + 15) // 16 * 16) if compressed.dim() == 1 else compressed.shape
        t.compressed = compressed.data_ptr()
    if layout_of is not None:
        _require("layout_of", layout_of, b_shape, torch.int32, dev)
        t.layout_of = layout_of.data_ptr()
    if n_new is not None:
        _require("n_new", n_new, b_shape, torch.int32, dev)
        t.n_new = n_new.data_ptr()
    if mask is not None:
        _require("mask", mask, shape[:2], torch.int64, dev)
        t.mask = mask.data_ptr()
    if pages is not None:
        if state is None or K_pages is None or V_pages is None:
            raise ValueError("pages need state, K_pages and V_pages")
        pool = pages.pool_shape[1:]
        _require("state", state, torch.Size((pages.state_numel,)), torch.int32, dev)
        _require("K_pages", K_pages, pool, dt, dev)
        _require("V_pages", V_pages, pool, dt, dev)
        pg = pages.c()
        t.pages = ctypes.pointer(pg)
        t.state, t.K_pages, t.V_pages = state.data_ptr(), K_pages.data_ptr(), V_pages.data_ptr()
    if out is None:
        out = torch.zeros(shape, dtype=dt, device=dev)
    else:
        _require("out", out, shape, dt, dev)
    if workspace is None:
        workspace = torch.empty(tree_workspace_bytes(p, batch, drafts, pages), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {dev}")
    t.q, t.K_new, t.V_new, t.out = q.data_ptr(), K_new.data_ptr(), V_new.data_ptr(), out.data_ptr()
    st = _call(dev, L.anchorkv_tree_attn, pc, t, workspace.data_ptr(), workspace.nbytes)
    capi.check("anchorkv_tree_attn", st)
    return out


def reconstruct(p: AnchorKVParams, compressed: torch.Tensor):
    """Dense fp32 K^, V^ [H, N, D] of one compressed layer (inspection hook)."""
    H, N, D = p.n_kv_heads, p.n_tokens, p.head_dim
    Kh = torch.empty(H, N, D, dtype=torch.float32, device=compressed.device)
    Vh = torch.empty_like(Kh)
    st = capi.lib().anchorkv_reconstruct(ctypes.byref(p.c()), _ptr(compressed), _ptr(Kh), _ptr(Vh),
                                         _stream(compressed.device))
    capi.check("anchorkv_reconstruct", st)
    return Kh, Vh


# device status word values (the first kernel to fail latches its code)
DEVICE_ERRORS = {1: "uniform anchor sample", 2: "refine list", 3: "inconsistent record or selection (bounds)",
                 4: "bounded wait timed out"}


def read_status(workspace: torch.Tensor) -> list[int]:
    """Device status word and counters of a compress workspace (synchronises
    the current stream).  Raises if a device-side check failed, naming it."""
    buf = (ctypes.c_int32 * 16)()
    st = capi.lib().anchorkv_read_device_status(_ptr(workspace), buf, _stream(workspace.device))
    vals = list(buf)
    if st == capi.EDEVICE:
        raise capi.AnchorKVError("anchorkv_read_device_status", st,
                                 f"status word {vals[0]} ({DEVICE_ERRORS.get(vals[0], 'unknown')})")
    capi.check("anchorkv_read_device_status", st)
    return vals


def codebook() -> tuple[float, float, float, float]:
    out = (ctypes.c_double * 4)()
    capi.check("anchorkv_codebook", capi.lib().anchorkv_codebook(out))
    return tuple(out)


class HostCompressor:
    """End-to-end compress from host (pinned) buffers through the C ABI's
    anchorkv_compress_host: per call, the library copies the layer's K, V,
    Q_obs into a preallocated device staging buffer, compresses there and
    copies the compressed bytes back into a pinned host buffer, all on the
    current stream.  Allocation happens once, in the constructor; `out` is a
    device view of the staged layout."""

    def __init__(self, p: AnchorKVParams, device="cuda"):
        self.p = p
        self.device = torch.device(device)
        L = anchorkv_bytes(p)
        self.staging = torch.empty(compress_host_staging_bytes(p), dtype=torch.uint8, device=device)
        self.ws = torch.empty(compress_workspace(p)["total_bytes"], dtype=torch.uint8, device=device)
        self.host_out = torch.empty(L["total_bytes"], dtype=torch.uint8, pin_memory=True)
        # the staged layout: the staging buffer's last section (256-byte aligned)
        self.out = self.staging[-((L["total_bytes"] + 255) // 256 * 256):][:L["total_bytes"]]

    def __call__(self, K_host, V_host, Q_host, layer: int | None = None, host_out: torch.Tensor | None = None):
        """Compress one layer; the compressed bytes land in `host_out` (pinned,
        total_bytes) or in the compressor's own pinned buffer.  Several
        compressors on different streams overlap the copies of one layer with
        the compression of another."""
        if layer is not None:
            self.p.layer = layer
        dst = self.host_out if host_out is None else host_out
        return compress_host(self.p, K_host, V_host, Q_host, dst, self.staging, self.ws, device=self.device)


N_STAGES = 18   # ANCHORKV_N_STAGES


def stage_timing(enable: bool) -> None:
    """Turn the library's per-stage CUDA-event timing on (clearing it) or off."""
    capi.check("anchorkv_stage_timing", capi.lib().anchorkv_stage_timing(1 if enable else 0))


def stage_times() -> dict:
    """{stage name: (total ms, timed calls)} since the last stage_timing(True)."""
    ms = (ctypes.c_double * N_STAGES)()
    calls = (ctypes.c_int64 * N_STAGES)()
    capi.check("anchorkv_stage_times", capi.lib().anchorkv_stage_times(ms, calls, N_STAGES))
    return {capi.lib().anchorkv_stage_name(i).decode(): (ms[i], calls[i]) for i in range(N_STAGES)}


def launch_count() -> int:
    n = ctypes.c_int64()
    capi.check("anchorkv_launch_count", capi.lib().anchorkv_launch_count(ctypes.byref(n)))
    return n.value
