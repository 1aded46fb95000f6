"""Mixed-head (DuoAttention retrieval / streaming) KV cache and attention for
B200 (sm_100a): a C-ABI CUDA library (libduo_kv.so, include/duo_kv.h) and a
thin Python binding.

``DuoKVCache`` owns the cache as a torch buffer and calls the library;
``Rope`` rotates queries and keys, ``TokenMap`` holds a step's token map;
``window_attention`` is the differentiable attention of whole sequences;
``_lib`` exposes the C functions one to one.  All load libduo_kv.so (and the
compiled half of the binding, _binding.so) on first use and raise ImportError
if one is missing (build both with
``python -m head_wise_kv_b200.build``); there is no fallback path.
"""
__all__ = ["DuoKVCache", "DuoError", "Rope", "TokenMap", "window_attention", "window_attention_status"]


def __getattr__(name):
    if name == "DuoKVCache":
        from .cache import DuoKVCache
        return DuoKVCache
    if name == "TokenMap":
        from .cache import TokenMap
        return TokenMap
    if name == "Rope":
        from .rope import Rope
        return Rope
    if name in ("window_attention", "window_attention_status"):
        from . import attention
        return getattr(attention, name)
    if name == "DuoError":
        from ._lib import DuoError
        return DuoError
    raise AttributeError(name)
