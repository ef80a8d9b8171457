"""GB300 (sm_103a) indexer top-k selection fused with paged KV-slot translation, and the
serving operators next to it: attention over an 8-bit paged cache, its pages, the sampling of
tokens and the verification of drafted ones.

The computation lives in the CUDA library libtopk_paged.so (C ABI:
include/topk_paged.h); `binding` mirrors that ABI name for name and `api` wraps it
with torch-owned device memory and streams.
"""
from . import binding
from .api import (HostPagedTopK, Kv8Cache, KvPages, PagedTopK, Step, sample_tokens, token_probs,
                  verify_drafts)
from .binding import Kv8Error, KvPagesError, SampleError, TopKError, VerifyError

__all__ = ["binding", "PagedTopK", "HostPagedTopK", "TopKError", "Kv8Cache", "Kv8Error", "KvPages",
           "KvPagesError", "Step", "verify_drafts", "VerifyError", "sample_tokens", "token_probs",
           "SampleError"]
