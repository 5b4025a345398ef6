"""Routed MoE layer over a GPU expert-slot cache, for one GB300 (sm_103a).

The compute path is the C-ABI library ``libmoe_gb300.so`` (see
``include/moe_gb300.h``); this package is its ctypes binding plus a host-side
layer runner.  The binding loads on first use of any of its names and raises
if the library has not been built (``moe_expert_offload_router_gb300.build``):
there is no fallback path.
"""
import importlib

_SUBMODULES = ("build", "layer", "block", "_lib", "_binding")
_HOST = {"DecodeLayerRunner": "layer", "PrefillStreamer": "layer", "Routing": "layer", "BlockWeights": "block",
         "RoutedBlocks": "block"}


def __getattr__(name):
    if name in _SUBMODULES or name.startswith("__"):
        raise AttributeError(name)   # the import system then loads the submodule
    if name in _HOST:
        found = getattr(importlib.import_module(__name__ + "." + _HOST[name]), name)
    else:
        lib = importlib.import_module(__name__ + "._lib")
        try:
            found = getattr(lib, name)
        except AttributeError:
            raise AttributeError(f"module {__name__!r} has no attribute {name!r}") from None
    globals()[name] = found   # later uses find it without coming here (this costs microseconds a call)
    return found
