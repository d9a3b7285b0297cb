"""bandwidth_bound_fp8_gb300: the FP8 live-quantised MoE expert projection
for small decode batches on GB300, and the expert layer at any number of
tokens with MXFP4 weights, as the C-ABI library libmoeq.so plus the thin
Python binding in ``moeq``; ``expert_layer`` puts the latter's calls together.

Build the library with ``python -m bandwidth_bound_fp8_gb300.build`` (or
``__graft_entry__.build()``); importing ``bandwidth_bound_fp8_gb300.moeq``
and calling any function loads it and raises if it is missing.
"""
from . import moeq  # noqa: F401

__all__ = ["moeq"]
