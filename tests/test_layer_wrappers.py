"""What the layer operators' wrappers (layer.py) pass to the library, and what
they refuse, without a GPU: host tensors stand in for device ones, and a
recorder for the library."""
import ctypes

import pytest
import torch

import sequence_blockwise_self_gb300 as ra
from sequence_blockwise_self_gb300 import layer

BF, FP = torch.bfloat16, torch.float32


class Recorder:
    """Entries that take any arguments and succeed."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def entry(*args):
            self.calls.append((name, args))
            return 1 << 16 if name.endswith("workspace_size") else 0

        entry.__name__ = name
        return entry

    def last(self, name):
        return [a for n, a in self.calls if n == name][-1]


@pytest.fixture
def lib(monkeypatch):
    """The index of a host tensor, -1, is the one device."""
    layer._lazy()
    rec = Recorder()
    monkeypatch.setattr(layer, "load", lambda: rec)
    monkeypatch.setattr(layer, "_cuda", lambda t, name: -1)
    monkeypatch.setattr(layer, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(layer, "_current", lambda: -1)
    return rec


# ------------------------------------------------------------------ block norms

@pytest.mark.parametrize("gate_dtype", [BF, FP])
@pytest.mark.parametrize("G", [1, 3])
def test_the_gradient_of_a_shared_gate_over_no_rows(lib, G, gate_dtype):
    """fp32 [G, D], which the library clears, as over any other number of rows
    that share a gate row."""
    D = 16
    x = torch.zeros(0, D, dtype=BF)
    gate = torch.ones(G, D, dtype=gate_dtype) if G > 1 else torch.ones(D, dtype=gate_dtype)
    got = ra.ring_attn_block_norm_bwd(x, x, x, x, torch.zeros(2, 0), gate=gate)
    assert got[2].dtype == FP and got[2].shape == (G, D)
    args = lib.last("ring_attn_block_norm_bwd")
    assert args[11] == got[2].data_ptr() and args[17:20] == (0, D, G)


def test_the_gradient_of_a_gate_per_token_over_no_rows(lib):
    x = torch.zeros(0, 16, dtype=BF)
    got = ra.ring_attn_block_norm_bwd(x, x, x, x, torch.zeros(2, 0), gate=x.clone())
    assert got[2].dtype == BF and got[2].shape == (0, 16)
