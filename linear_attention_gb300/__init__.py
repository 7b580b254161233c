"""GB300-native Based (2nd-order Taylor linear attention) causal forward pass.

The compute runs in hand-written sm_103a CUDA kernels behind a C-ABI shared library
(``include/based.h``); ``linear_attention_gb300.based`` is a thin ctypes binding to it. The
operators of a language model around it (gated linear recurrence, group norm with an activation,
embedding, gated delta rule, root-mean-square norm, sampling; ``include/based_ops.h``) are bound by ``linear_attention_gb300.ops``.
"""
import importlib

_OPS = ("based_scan_fwd", "based_scan_bwd", "based_scan_step", "based_norm_fwd", "based_norm_bwd",
        "based_embed_fwd", "based_embed_bwd", "based_delta_fwd", "based_delta_bwd", "based_delta_step",
        "based_rms_fwd", "based_rms_bwd", "based_sample")
__all__ = ["based_fwd", "based_fwd_host", *_OPS]


def __getattr__(name):
    # The bindings are imported lazily so that the input generators can be used without the
    # CUDA library being built.
    if name in __all__:
        module = importlib.import_module(".ops" if name in _OPS else ".based", __name__)
        globals()[name] = getattr(module, name)  # the next lookup finds it without this function
        return globals()[name]
    raise AttributeError(name)
