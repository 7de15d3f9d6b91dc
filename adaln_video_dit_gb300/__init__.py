"""GB300-native operators of video diffusion transformer blocks: the fused AdaLN
LayerNorm-Modulate, rotary positions with the norm of queries and keys, the gated
feed-forward block, dropout with the gate and the residual of a branch, and mixtures
of experts (forward and backward).

The compute path is libadaln.so (hand-written sm_103a CUDA behind a C ABI,
declared in include/adaln.h); `adaln_video_dit_gb300._lib` is its thin ctypes
binding.  `adaln_video_dit_gb300.autograd` has the operators as autograd nodes,
`adaln_video_dit_gb300.rotary` the rotary tables and positions, and
`adaln_video_dit_gb300.inputs` draws seeded synthetic workloads.
The binding is imported lazily so that the input generators load without a GPU.
"""

__all__ = ["inputs", "lib"]

_lib_module = None


def lib():
    """The ctypes binding of libadaln.so (raises if the library is missing)."""
    global _lib_module
    if _lib_module is None:
        from . import _lib
        _lib_module = _lib
    return _lib_module
