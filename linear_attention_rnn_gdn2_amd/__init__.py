"""MI355X-native Gated DeltaNet-2 chunked prefill forward, the scalar-gated
delta rule and the q/k preparation.

``chunk_fwd`` and the other functions (in :mod:`.gdn2`) call the C-ABI library ``libgdn2.so`` built
from ``csrc/`` for gfx950. Importing this package does not load the library;
the first call does, and raises if it is missing.
"""

__all__ = ["chunk_fwd", "last_error", "delta_chunk_fwd", "delta_chunk_bwd", "delta_recurrent_fwd",
           "qk_norm_rope", "qk_norm_rope_bwd", "rope_table"]


def __getattr__(name):
    if name in __all__:
        from . import gdn2
        return getattr(gdn2, name)
    raise AttributeError(name)
