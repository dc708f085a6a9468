"""GB300-native (sm_103a) Gated DeltaNet-2 chunked prefill forward, and the
operators of the softmax-attention layers that run beside it.

The compute path is the CUDA library ``libgdn2.so`` built from ``csrc/``;
``gdn2`` and ``attn`` are its thin ctypes bindings.  Importing this package loads nothing:
the library is opened on first use and a missing library is an error.
"""
__all__ = ["attn", "gdn2", "inputs"]
