"""GB300-native whole-model decode megakernel.

The product is the C-ABI library ``libmk.so`` (include/mk.h) built from ``csrc/``; this package holds
its sources, the build step and a thin ctypes binding with the same entry points.
"""
from .binding import Megakernel, MKError, load, lib_path, EXPORTS  # noqa: F401

_SERVING = ("page_tables", "qk_norm_rope", "paged_attention", "paged_attention_workspace", "logit_controls")


def __getattr__(name):
    # the serving operators take torch tensors; building and loading the library do not need torch
    if name in _SERVING:
        from . import serving
        globals()[name] = getattr(serving, name)
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
