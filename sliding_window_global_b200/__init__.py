"""Banded sparse self-attention for NVIDIA B200 (sm_100a).

Sliding-window attention with optional dilation and causal mask, global tokens
(global rows and columns), LongT5-style appended side keys with an additive
bucketed bias, a LongT5 local relative-position bias on window keys, and grouped
KV heads -- computed by the hand-written CUDA kernels
of ``libswa.so`` behind the C ABI in ``include/swa.h``.  This Python layer only
marshals arguments: PyTorch provides device memory and streams.

Around the attention: ``Rotary`` rotates (and norms) queries and keys by position and
gives the gradients; ``PagedCache`` holds keys and values of many sequences in pages,
appends to them and attends over them, for prompts and single tokens.
"""
from .cache import PagedCache  # noqa: F401
from .rotary import Rotary, rotary_frequencies  # noqa: F401
from .swa import (  # noqa: F401
    Plan,
    SwaError,
    bucket_local_bias,
    expand_side_bias,
    forward,
    lib_path,
    load_library,
    relative_bucket,
    side_aggregate,
)
