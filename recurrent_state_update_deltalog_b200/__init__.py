"""DeltaLog deferred-materialisation decode step for linear-attention state on B200.

``DeltaLog`` (PyTorch tensors in, CUDA library underneath), the operators of
``ops`` that stand beside the recurrent layers, and the raw C-ABI binding
``_native`` are the public surface.  Importing this package does not load the
CUDA library; the first handle, or the first operator taken from here, does, and
fails loudly if it is missing.
"""
_OPS = ["gated_scan", "gated_scan_forward", "gated_scan_backward", "gated_scan_prefill", "gated_scan_step",
        "block_norm", "block_norm_forward", "block_norm_backward",
        "paged_attention", "paged_write", "check_errors"]
__all__ = ["DeltaLog", "DeltaLogError", "suggest_m"] + _OPS


def __getattr__(name):
    if name == "DeltaLog":
        from .deltalog import DeltaLog
        return DeltaLog
    if name == "suggest_m":
        from .deltalog import suggest_m
        return suggest_m
    if name == "DeltaLogError":
        from ._native import DeltaLogError
        return DeltaLogError
    if name in _OPS:
        from . import ops
        globals()[name] = getattr(ops, name)    # the next access is a plain lookup
        return globals()[name]
    raise AttributeError(name)
