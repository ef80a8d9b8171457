"""GB300 (sm_103a) indexer top-k selection fused with paged KV-slot translation, and the
serving operators next to it: attention over an 8-bit paged cache, its pages, and the
verification of drafted tokens.

The computation lives in the CUDA library libtopk_paged.so (C ABI:
include/topk_paged.h); `binding` mirrors that ABI name for name and `api` wraps it
with torch-owned device memory and streams.
"""
from . import binding
from .api import HostPagedTopK, Kv8Cache, KvPages, PagedTopK, verify_drafts
from .binding import Kv8Error, KvPagesError, TopKError, VerifyError

__all__ = ["binding", "PagedTopK", "HostPagedTopK", "TopKError", "Kv8Cache", "Kv8Error", "KvPages",
           "KvPagesError", "verify_drafts", "VerifyError"]
