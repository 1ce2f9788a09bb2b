"""libfibatt: Fibottention per-head sparse self-attention for GB300 (sm_103a).

The compute path is the C-ABI library ``libfibatt.so`` (``include/fibatt.h``);
this package only builds it (``build.build_library``) and binds it
(``api``).  Importing the package does not load the library; the first call
does, and fails loudly if it has not been built.
"""
from .api import (FibattError, FibottentionFunction, Support, bwd, cross_attention, cross_bwd, cross_fwd,
                  fibottention, fwd, qk_norm, qk_norm_bwd, qk_norm_fwd, rotary_angles, rotary_angles_2d,
                  rotary_tables, window_schedule, wythoff_row, wythoff_row_modified)

__all__ = ["FibattError", "FibottentionFunction", "Support", "bwd", "cross_attention", "cross_bwd", "cross_fwd",
           "fibottention", "fwd", "qk_norm", "qk_norm_bwd", "qk_norm_fwd", "rotary_angles", "rotary_angles_2d",
           "rotary_tables", "window_schedule", "wythoff_row", "wythoff_row_modified"]
