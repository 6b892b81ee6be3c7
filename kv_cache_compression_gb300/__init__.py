"""GB300-native (sm_103a) SnapKV: prefill KV-cache compression and compressed-cache decode attention.

The compute lives in ``libsnapkv.so`` (hand-written CUDA kernels behind the C ABI declared in
``include/snapkv.h``, ``include/snapkv_cache.h`` and ``include/snapkv_draft.h``); ``snapkv``, ``cache`` and ``draft`` are
its thin Python bindings.
"""
from . import cache, draft, snapkv  # noqa: F401
from .cache import (Q4Cache, decode_attend_scored, evict, evict_workspace_size, q4_append,  # noqa: F401
                    q4_decode_attend, q4_evict, q4_read, scored_workspace_size)
from .draft import (Q8Cache, append_rows, q8_append, q8_read, q8_tree_attend, tree_attend,  # noqa: F401
                    tree_workspace_size)
from .snapkv import (append, compress, compress_workspace_size, decode_attend,  # noqa: F401
                     decode_workspace_size, kept, make_params, status_string)

__all__ = ["snapkv", "compress", "append", "decode_attend", "kept", "make_params", "compress_workspace_size",
           "decode_workspace_size", "status_string", "cache", "Q4Cache", "decode_attend_scored", "scored_workspace_size",
           "q4_append", "q4_read", "q4_decode_attend", "evict", "q4_evict", "evict_workspace_size", "draft",
           "tree_attend", "tree_workspace_size", "Q8Cache", "q8_append", "q8_read", "q8_tree_attend", "append_rows"]
