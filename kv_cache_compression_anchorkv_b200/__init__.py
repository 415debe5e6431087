"""AnchorKV anchor-residual KV-cache codec for NVIDIA B200 (sm_100a).

The codec runs in the CUDA library libanchorkv.so (C ABI: include/anchorkv.h);
this package is its PyTorch binding.  Importing the package does not load the
library; the first call does, and fails loudly if it has not been built.
"""
from .api import (AnchorKVParams, HostCompressor, PageSpec, anchorkv_bytes, codebook, compress, compress_host,
                  compress_host_staging_bytes, compress_workspace,
                  decode_attn, decode_workspace_bytes, pages_commit, pages_compact, pages_fork, pages_init,
                  pages_state_bytes, pages_view, pages_workspace_bytes, read_status, reconstruct, tree_attn,
                  tree_workspace_bytes)

__all__ = ["AnchorKVParams", "HostCompressor", "PageSpec", "anchorkv_bytes", "codebook", "compress", "compress_host",
           "compress_host_staging_bytes", "compress_workspace",
           "decode_attn", "decode_workspace_bytes", "pages_commit", "pages_compact", "pages_fork", "pages_init",
           "pages_state_bytes", "pages_view", "pages_workspace_bytes", "read_status", "reconstruct", "tree_attn",
           "tree_workspace_bytes"]
