"""B200 (sm_100a) inference path of ALHR tree attention.

Importing the package loads nothing native. The compute entry points live in
`tree_routed_sparse_b200.alhr` (a thin ctypes binding of libalhr.so); the first access to
them loads the library and raises if it has not been built. The paged 8-bit key/value cache is in
`tree_routed_sparse_b200.cache` (same library). Seeded synthetic inputs live in
`tree_routed_sparse_b200.synth`.
"""
import importlib

__all__ = ["alhr", "cache", "synth", "build_tree", "predict_budget", "route", "attend", "forward",
           "alloc_cache", "plan_blocks", "store_cache", "load_cache", "attend_cache",
           "attend_cache_selected"]

_LAZY = {"build_tree", "predict_budget", "route", "attend", "forward", "Dims", "AlhrError"}
_LAZY_CACHE = {"alloc_cache", "plan_blocks", "store_cache", "load_cache", "attend_cache",
               "attend_cache_selected"}


def __getattr__(name):
    if name in ("alhr", "cache", "synth", "metrics"):
        return importlib.import_module(f"{__name__}.{name}")
    if name in _LAZY:
        return getattr(importlib.import_module(f"{__name__}.alhr"), name)
    if name in _LAZY_CACHE:
        return getattr(importlib.import_module(f"{__name__}.cache"), name)
    raise AttributeError(name)
