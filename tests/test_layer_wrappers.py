"""What the layer operators' wrappers (layer.py) pass to the library, and what
they refuse, without a GPU: host tensors stand in for device ones, and a
recorder for the library."""
import gc
import weakref

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


# -------------------------------------------------------------- gradient lists

def clip(grads, **kw):
    return ra.ring_attn_grad_clip(grads, 1.0, norm=torch.zeros(()), workspace=torch.empty(1 << 16, dtype=torch.uint8), **kw)


def replaced_by(t, new):
    t.data = new


CHANGES = {
    "a smaller storage": lambda t: replaced_by(t, torch.ones(5)),
    "a larger storage": lambda t: replaced_by(t, torch.ones(500)),
    "another type": lambda t: replaced_by(t, t.data.to(BF)),
    "another type of the same bytes": lambda t: replaced_by(t, torch.ones(128, dtype=BF)),
    "strided": lambda t: replaced_by(t, torch.ones(128)[::2]),
    "one element for all": lambda t: replaced_by(t, torch.ones(1).expand(64)),
}


@pytest.mark.parametrize("change", CHANGES.values(), ids=CHANGES.keys())
@pytest.mark.parametrize("which", ["gradient", "output"])
def test_a_kept_list_refuses_a_tensor_that_became_another(lib, change, which):
    """The counts and types that the list has would reach past the end of
    another storage."""
    grads, outs = [torch.ones(7), torch.ones(64), torch.ones(8, 3)], [torch.ones(7), torch.ones(64), torch.ones(24)]
    kept = ra.GradList(grads, outs)
    for call in (clip, lambda g: ra.ring_attn_grad_norm(g, norm=torch.zeros(()), workspace=torch.empty(1 << 16)),
                 lambda g: ra.ring_attn_grad_scale(g, 1.0, torch.zeros(()))):
        call(kept)
    change((grads if which == "gradient" else outs)[1])
    before = len(lib.calls)
    for call in (clip, lambda g: ra.ring_attn_grad_norm(g, norm=torch.zeros(()), workspace=torch.empty(1 << 16)),
                 lambda g: ra.ring_attn_grad_scale(g, 1.0, torch.zeros(()))):
        for _ in range(2):   # refused again, not only once
            with pytest.raises((ValueError, TypeError)):
                call(kept)
    assert len(lib.calls) == before


def test_a_kept_list_passes_what_is_there_now(lib):
    grads = [torch.ones(7), None, torch.ones(64), torch.empty(0)]
    kept = ra.GradList(grads)
    for _ in range(3):
        clip(kept)
        ins, outs, n, dt, dt_out, count = lib.last("ring_attn_grad_clip")[:6]
        assert count == 3 and list(n) == [7, 64, 0] and list(dt) == list(dt_out) == [2, 2, 2]
        assert [p or 0 for p in ins] == [p or 0 for p in outs] == [t.data_ptr() for t in grads if t is not None]
        grads[2].data = torch.ones(64)   # as large: followed
    outs = [torch.ones(7, dtype=BF), torch.ones(64)]
    kept = ra.GradList([grads[0], grads[2]], outs)
    clip(kept)
    ins, to, n, dt, dt_out, count = lib.last("ring_attn_grad_clip")[:6]
    assert list(ins) == [grads[0].data_ptr(), grads[2].data_ptr()] and list(to) == [t.data_ptr() for t in outs]
    assert list(dt) == [2, 2] and list(dt_out) == [0, 2]


def test_a_kept_list_is_not_changed_through_what_it_returns(lib):
    grads = [torch.ones(7), torch.ones(64)]
    kept = ra.GradList(grads)
    for taken in (ra.ring_attn_grad_scale(kept, 1.0, torch.zeros(())), kept.grads, kept.outs, grads):
        taken.append(torch.ones(3))
        assert len(kept) == 2
        clip(kept)
        ins, _, n, _, _, count = lib.last("ring_attn_grad_clip")[:6]
        assert count == 2 == len(n) == len(ins)


def test_a_kept_list_holds_what_it_checked(lib):
    """An address that a tensor has again is not another's memory: what was
    checked there stays until the next call has found the tensor elsewhere."""
    t = torch.ones(64)
    kept = ra.GradList([t])
    clip(kept)
    first = weakref.ref(t.untyped_storage())
    t.data = torch.ones(64)
    gc.collect()
    assert first() is not None
    clip(kept)
    gc.collect()
    assert first() is None
    assert list(lib.last("ring_attn_grad_clip")[0]) == [t.data_ptr()]


# ------------------------------------------------------------------- workspaces

@pytest.mark.parametrize("workspace", [torch.empty(1, dtype=torch.uint8).expand(1 << 20), torch.empty(1 << 20)[::2],
                                       torch.empty(1 << 10, 1 << 10).t()])
def test_a_workspace_is_adjacent_memory(lib, workspace):
    """An expanded tensor has fewer bytes than its shape says."""
    x, st = torch.ones(4, 16, dtype=BF), torch.ones(2, 4)
    with pytest.raises(ValueError):
        ra.ring_attn_block_norm_bwd(x, x, x, x, st, workspace=workspace)
    with pytest.raises(ValueError):
        ra.ring_attn_grad_clip([torch.ones(7)], 1.0, norm=torch.zeros(()), workspace=workspace)
    with pytest.raises(ValueError):
        ra.ring_attn_grad_norm([torch.ones(7)], norm=torch.zeros(()), workspace=workspace)
    assert all(n.endswith("workspace_size") for n, _ in lib.calls)


# ------------------------------------------------- numbers that C types cannot hold

FAR = (1 << 32) + 8   # 8 in 32 bits


@pytest.mark.parametrize("shape", [(FAR, 1, 1, 4), (1, FAR, 1, 4), (1, 1, FAR, 4), (1, 1, 1, FAR)])
def test_rotary_sizes_past_32_bits_are_refused(lib, shape):
    """(Cut to 32 bits they would be 8, and the rest of the output never
    written.)"""
    q = torch.empty(shape, device="meta")
    rope = ra.RotaryFrequencies(4, device="cpu")
    for fn in (ra.ring_attn_rope_fwd, ra.ring_attn_rope_bwd):
        for args, kw in (((q, None), dict(q_out=q)), ((None, q), dict(k_out=q)), ((None, None), dict(v=q, v_out=q))):
            if fn is ra.ring_attn_rope_bwd:
                kw = {"d" + k: v for k, v in kw.items()}
            with pytest.raises(ra.RingAttnError):
                fn(*args, rope, **kw)
    assert not lib.calls


def test_block_norm_columns_past_32_bits_are_refused(lib):
    x, st = torch.empty(1, FAR, device="meta"), torch.ones(2, 1)
    with pytest.raises(ra.RingAttnError):
        ra.ring_attn_block_norm_fwd(x, None, h=x, stats=st)
    with pytest.raises(ra.RingAttnError):
        ra.ring_attn_block_norm_bwd(x, x, x, None, st, dx=x)
    with pytest.raises(ra.RingAttnError):
        ra.block_norm_bwd_workspace_size(1, FAR)
    assert not lib.calls


@pytest.mark.parametrize("positions", [1 << 63, -(1 << 63) - 1, (1 << 64) + 5, ra.PositionMap(4, 2, 1 << 63, 0, 1),
                                       ra.PositionMap(4, 2, 0, 1 << 64, 1), ra.PositionMap(4, 2, 0, 0, 1 << 64),
                                       ra.PositionMap(4, (1 << 64) + 2, 0, 0, 1)])
def test_positions_past_64_bits_are_refused(lib, positions):
    q = torch.zeros(1, 2, 4, 8)
    with pytest.raises(ValueError):
        ra.ring_attn_rope_fwd(q, None, ra.RotaryFrequencies(8, device="cpu"), positions)
    assert not lib.calls


def test_positions_of_64_bits_are_passed_on(lib):
    q = torch.zeros(1, 2, 4, 8)
    rope = ra.RotaryFrequencies(8, device="cpu")
    for p, want in (((1 << 63) - 1, [4, (1 << 63) - 1, 0, 1]), (-(1 << 63), [4, -(1 << 63), 0, 1]),
                    (ra.PositionMap(4, 2, -5, 1 << 62, -3), [2, -5, 1 << 62, -3])):
        ra.ring_attn_rope_fwd(q, None, rope, p)
        assert list(lib.last("ring_attn_rope_fwd")[-2]) == want
