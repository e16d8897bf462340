"""libtfla: chunkwise-parallel gated linear attention forward (mLSTMsig,
fixed per-head decay, per-key-channel gate) on AMD gfx950, and the operators
around it: causal convolution, selective scan, group norm with a gate.

The compute path is the C-ABI library ``libtfla.so`` built from ``csrc/``;
:mod:`mlstm_sequence_amd.tfla` is its ctypes binding.
"""
from .tfla import (  # noqa: F401
    ACT_NONE, ACT_SIGMOID, ACT_SILU, GLA_KEY, IO_BF16, MLSTM_SIG, NORM_SEQUENCE, NORM_TOKEN, SCALAR_DECAY, TflaError,
    conv_backward, conv_forward, forward, norm_backward, norm_forward, scan_backward, scan_forward, tfla_dbg_gates,
    tfla_dbg_states,
    tfla_fwd, tfla_fwd_ws, tfla_last_error, tfla_version, tfla_workspace_bytes, variant_of,
    workspace_for,
)
