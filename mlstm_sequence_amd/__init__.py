"""libtfla: chunkwise-parallel gated linear attention forward (mLSTMsig,
fixed per-head decay, per-key-channel gate) on AMD gfx950, and the operators
around it: causal convolution, selective scan, group norm with a gate, rotary
positions, gated linear recurrence of channels, residual sum with a norm.

The compute path is the C-ABI library ``libtfla.so`` built from ``csrc/``;
:mod:`mlstm_sequence_amd.tfla` is its ctypes binding.
"""
from .tfla import (  # noqa: F401
    ACT_NONE, ACT_SIGMOID, ACT_SILU, DIAG_COUPLED, DIAG_DECAY, DIAG_SIGMOID, GLA_KEY, IO_BF16, MLSTM_SIG, NORM_SEQUENCE,
    NORM_TOKEN, ROTARY_HALVES, ROTARY_INTERLEAVED, SCALAR_DECAY, TflaError, addnorm_backward, addnorm_forward,
    conv_backward, conv_forward, diag_backward, diag_forward, forward, norm_backward, norm_forward, rotary_backward,
    rotary_forward, rotary_frequencies, scan_backward, scan_forward, tfla_dbg_gates, tfla_dbg_states,
    tfla_fwd, tfla_fwd_ws, tfla_last_error, tfla_version, tfla_workspace_bytes, variant_of,
    workspace_for,
)
