"""libssd: Mamba-2 SSD chunked selective-scan forward for AMD Instinct MI355X (gfx950).

Around the scan stand the other operators of a state space block: ``conv``, ``selective_scan``
(each with ``_step`` and ``_backward``), ``gated_norm`` and ``residual_norm`` (with ``_backward``).
Layers of linear recurrence beside it have ``recurrence`` (with ``_step`` and ``_backward``),
``rotate``, which turns the scan's B and C by positions, and ``group_norm`` (with ``_backward``).

The compute path is the C-ABI library libssd.so (hand-written HIP kernels); ``forward`` (the
chunked forward), ``backward`` (its gradients) and ``step`` (one recurrent decode step) are its
Python bindings. The library is loaded on first use and must have been built beforehand.
"""

from .block import (conv, conv_backward, conv_step, gated_norm, gated_norm_backward,  # noqa: F401
                    residual_norm, residual_norm_backward, selective_backward, selective_scan,
                    selective_step)
from .recurrent import (group_norm, group_norm_backward, recurrence,  # noqa: F401
                        recurrence_backward, recurrence_step, rotate, rotate_backward)
from .libssd import SSDError, backward, forward, load, status_string, step, version  # noqa: F401

__all__ = ["forward", "backward", "step", "load", "status_string", "version", "SSDError",
           "conv", "conv_step", "conv_backward", "selective_scan", "selective_step",
           "selective_backward", "gated_norm", "gated_norm_backward", "residual_norm",
           "residual_norm_backward", "recurrence", "recurrence_step", "recurrence_backward",
           "rotate", "rotate_backward", "group_norm", "group_norm_backward"]
