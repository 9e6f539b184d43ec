"""Length-aware GQA decode attention over a preallocated KV cache (GB300).

The computation lives in libfd.so (hand-written CUDA for sm_103a, C ABI in
include/fd.h); ``fd`` is its Python binding and ``build`` compiles it.
``workloads`` makes seeded synthetic inputs.  Importing the package does not
load the library; the first call does, and raises if it is not built.
"""
from .fd import (FD_KERNEL_AUTO, FD_KERNEL_SIMT, FD_KERNEL_TC, FdError,  # noqa: F401
                 PagePools, Workspace, append, append_fp4, beam_select, decode, decode_fp4,
                 decode_gather, decode_int8, pages_compact, pages_copy, pages_fork, pages_free,
                 pages_reorder, pages_reserve, plan, prefill, read_fp4)

__all__ = ["decode", "decode_int8", "decode_gather", "decode_fp4", "append_fp4", "read_fp4",
           "append", "prefill", "beam_select", "pages_reserve", "pages_fork", "pages_reorder",
           "pages_free", "pages_compact", "pages_copy",
           "PagePools", "Workspace", "plan", "FdError", "FD_KERNEL_AUTO", "FD_KERNEL_SIMT",
           "FD_KERNEL_TC"]
