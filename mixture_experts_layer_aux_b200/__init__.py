"""B200-native single-GPU MoE layer (router -> top-k + aux -> permute ->
grouped SwiGLU expert GEMMs -> unpermute), as a C-ABI CUDA library.

The entry points (moe_router_topk, moe_permute, moe_grouped_gemm_fwd/bwd,
moe_unpermute, moe_layer_fwd/bwd, ...) live in libmoe_b200.so, declared in
include/moe.h. This package is a thin ctypes binding with the same names
(argument marshalling only). Attributes are resolved lazily so that the
seeded-input module `synthetic` can be imported without loading the library.
"""
import importlib

__all__ = ["load"]

_SUBMODULES = ("binding", "build", "synthetic")
_names = None  # the binding's namespace, once it is imported


def __getattr__(name):
    global _names
    if name.startswith("__"):
        raise AttributeError(name)
    try:
        # looked up each time (0.3 us): the binding rebinds names of its own, and a caller may
        return _names[name]
    except (TypeError, KeyError):
        pass
    if name in _SUBMODULES:
        return importlib.import_module(f"{__name__}.{name}")
    binding = importlib.import_module(f"{__name__}.binding")
    _names = vars(binding)
    return getattr(binding, name)


def load():
    """Load the CUDA library (raises if it is missing or fails to load)."""
    return importlib.import_module(f"{__name__}.binding").load()
