"""The compiled torch side of the operators beside the head (lce_torch.cpp):
checks of tensors, their outputs and workspaces, and one call of the C ABI.
It calls the library that the ctypes binding has loaded, on torch's current
stream."""
from __future__ import annotations

import ctypes
import importlib.util
import os

import torch  # noqa: F401  (the module below links against it)

from . import LCEError, lib

_module = None


class Traced(RuntimeError):
    """A call under torch.jit.trace, which would see the allocation of the
    outputs but not the call that fills them."""


_NAMES = ("lce_layer_norm_forward", "lce_layer_norm_backward", "lce_layer_norm_workspace_size", "lce_balance_forward",
          "lce_balance_fused", "lce_balance_backward", "lce_balance_workspace_size", "lce_beam_select",
          "lce_beam_workspace_size", "lce_beam_reorder")


def native():
    """The loaded _lce_torch module (ImportError if it has not been built)."""
    global _module
    if _module is None:
        path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lce_torch.so")
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`")
        spec = importlib.util.spec_from_file_location("_lce_torch", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.init({n: ctypes.cast(getattr(lib(), n), ctypes.c_void_p).value for n in _NAMES}, LCEError, Traced)
        _module = module
    return _module
