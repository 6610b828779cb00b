"""Mamba-3 SSM sequence mixer on MI355X (gfx950).

    from mamba_selective_ssm_ssd_amd import prefill, decode_step, State

``capi`` is the ctypes binding of the C ABI (include/m3_ssm.h); ``mixer``
wraps it for torch tensors; ``synth`` draws seeded synthetic inputs.  The
torch-facing names are imported lazily so that ``synth`` works without torch.

Beside the mixer, for layers that interleave it with linear attention:

    from mamba_selective_ssm_ssd_amd import linear, rotary

``linear`` is linear attention with a decay for each head (prompt pass over
packed sequences, gradients, single-token step), ``rotary`` the norm of its
queries and keys with the position rotation in the same pass.
"""

_LAZY = ("prefill", "decode_step", "State", "workspace_bytes", "make_shape")


def __getattr__(name):
    if name in ("linear", "rotary"):
        import importlib
        return importlib.import_module("." + name, __name__)
    if name in _LAZY:
        from . import mixer
        return getattr(mixer, name)
    raise AttributeError(name)
