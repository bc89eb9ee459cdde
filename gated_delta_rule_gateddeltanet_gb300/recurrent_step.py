"""One decoding step of a gated-linear-recurrence layer between its projections,
captured once in a CUDA graph and replayed: the counterpart, for layers with a
diagonal state, of ``spec_step.SpeculativeStep`` and ``attention_step.AttentionStep``.

The step is three C-ABI calls with arguments built once:

  1. varlen_causal_conv_with_state: the new tokens' inputs through the causal
     convolution (+ SiLU), its state updated in place;
  2. gdn_linear_recurrence: the recurrence with gates straight from the
     in-projection, its state updated in place;
  3. gdn_rms_norm: every head's norm, gated, in the I/O type or in 8 bits with
     scales for the out-projection.

Everything that changes from step to step is device memory read at replay time
(the projection's output, the state slots), so one graph serves every step.
"""
from __future__ import annotations

import ctypes

import torch

from . import GdnError, build_conv_args, load_library
from .norm import RMSNormCall
from .recurrence import LinearRecurrenceCall


class RecurrentStep:
    """``seqs`` sequences, ``tokens`` new tokens each.  conv_weight: [C, K] fp32;
    ``conv_bank`` [slots, C, K-1] (fp16 or fp32, the I/O type: the convolution takes
    no bf16) and ``bank`` [slots, C] fp32 hold the states; A_log, dt_bias: [C] fp32; norm_weight: [head_dim] fp32
    or None.

    Buffers, device tensors owned by this object: ``projection`` [seqs * tokens,
    4 C], the in-projection's output (the input, the decay gate a, the input gate b,
    the output gate, C channels each), and ``slots`` [seqs], each sequence's state
    slot (initially 0 .. seqs - 1; distinct).  Outputs: ``out`` [seqs * tokens, C /
    head_dim, head_dim] and, in 8 bits, ``scale``; the banks are updated in place."""

    def __init__(self, conv_weight, conv_bias, conv_bank, A_log, dt_bias, bank, norm_weight, *, seqs, head_dim, tokens=1,
                 unit_input=True, eps=1e-6, weight_offset=0.0, out_dtype=None, scale_group=0, activation="silu"):
        dev, (slots, C, _) = conv_bank.device, conv_bank.shape
        if C % head_dim:
            raise ValueError(f"head_dim must divide the {C} channels, got {head_dim}")
        if seqs > min(slots, bank.shape[0]):
            raise ValueError(f"{seqs} sequences need as many state slots, got {slots} and {bank.shape[0]}")
        T = seqs * tokens
        self.device, self.conv_bank, self.bank = dev, conv_bank, bank
        self.projection = torch.zeros((T, 4 * C), dtype=conv_bank.dtype, device=dev)
        self.slots = torch.arange(seqs, dtype=torch.int32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        cu = torch.arange(0, T + 1, tokens, dtype=torch.int32, device=dev)
        x, a, b, gate = self.projection.split(C, 1)
        self._conv_args, (y, _, _), keep = build_conv_args(
            x, conv_weight, cu, bias=conv_bias, initial_state=conv_bank, final_state=conv_bank, state_slots=self.slots,
            activation=activation, status=self.status, max_seqlen=tokens)
        self._recur = LinearRecurrenceCall(y, a, b, cu, A_log=A_log, dt_bias=dt_bias, unit_input=unit_input,
                                           initial_state=bank, final_state=bank, state_slots=self.slots,
                                           max_seqlen=tokens, status=self.status)
        heads = lambda t: t.unflatten(1, (C // head_dim, head_dim))  # noqa: E731
        self._norm = RMSNormCall(heads(self._recur.outputs[0]), norm_weight, eps=eps, weight_offset=weight_offset,
                                 gate=heads(gate), out_dtype=out_dtype, scale_group=scale_group)
        self.out, self.scale = self._norm.outputs if isinstance(self._norm.outputs, tuple) else (self._norm.outputs, None)
        self._keep = (keep, y)
        self.graph = None

    def launch(self, stream=None):
        """The step's three calls on ``stream`` (default: the current one)."""
        if self.device.type != "cuda":
            raise ValueError(f"RecurrentStep: tensors must be on a GPU, got {self.device}")
        handle = ctypes.c_void_p((stream or torch.cuda.current_stream(self.device)).cuda_stream)
        rc = load_library().varlen_causal_conv_with_state(ctypes.byref(self._conv_args), handle)
        if rc:
            raise GdnError(rc, "varlen_causal_conv_with_state")
        self._recur.launch(stream)
        self._norm.launch(stream)
        return self.out

    def capture(self):
        """Records the step into a CUDA graph.  The banks are restored after the warm-up before it."""
        saved = self.conv_bank.clone(), self.bank.clone()
        self.launch()
        self.conv_bank.copy_(saved[0])
        self.bank.copy_(saved[1])
        torch.cuda.current_stream(self.device).synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.launch()
        return self

    def replay(self):
        if self.graph is None:
            self.capture()
        self.graph.replay()
        return self.out
