"""The layer operators on the host (no GPU): the argument checks that return
before anything is launched, the position maps against the chunk maps, the
rotary frequencies, and the reference formulas' gradients against
differences."""
import ctypes
import math

import pytest
import torch

import layer_reference as ref
import oracle
import sequence_blockwise_self_gb300 as ra
from sequence_blockwise_self_gb300 import build as lib_build
from sequence_blockwise_self_gb300 import capi

NUL = None
LL = ctypes.c_longlong


@pytest.fixture(scope="module")
def lib():
    lib_build.build()
    return capi.load()


def at(n):
    """An aligned address that is never dereferenced."""
    return n << 30


# ------------------------------------------------------------------- rotary

B, HQ, HKV, L, D = 2, 4, 2, 16, 64


def contiguous(B, H, L, d):
    return [H * L * d, L * d, d]


def rope_call(lib, q=at(1), k=at(2), v=at(3), qo=at(4), ko=at(5), vo=at(6), strides=None, B=B, Hq=HQ, Hkv=HKV, L=L,
              d=D, R=D, dtype=0, inter=0, phase=at(7), factor=1.0, pos=NUL, pos_bytes=0, pos_batch=0, pmap=None,
              back=False):
    if strides is None:
        strides = 2 * (contiguous(B, Hq, L, d) + 2 * contiguous(B, Hkv, L, d))
    f = lib.ring_attn_rope_bwd if back else lib.ring_attn_rope_fwd
    return f(q, k, v, qo, ko, vo, (LL * 18)(*strides) if strides != "null" else None, B, Hq, Hkv, L, d, R, dtype, inter,
             phase, factor, pos, pos_bytes, pos_batch, (LL * 4)(*pmap) if pmap else None, NUL)


@pytest.mark.parametrize("back", [False, True])
def test_rope_refusals(lib, back):
    def call(**kw):
        return rope_call(lib, back=back, **kw)

    assert call(B=-1) == capi.ERR_SHAPE
    assert call(Hq=-1) == capi.ERR_SHAPE
    assert call(R=63) == capi.ERR_SHAPE
    assert call(R=66) == capi.ERR_SHAPE
    assert call(R=-2) == capi.ERR_SHAPE
    assert call(d=0, R=0) == capi.ERR_SHAPE
    assert call(factor=math.inf) == capi.ERR_SHAPE
    assert call(factor=math.nan) == capi.ERR_SHAPE
    assert call(dtype=3) == capi.ERR_UNSUPPORTED
    assert call(d=1026, R=64) == capi.ERR_UNSUPPORTED
    assert call(pos=at(8), pos_bytes=2) == capi.ERR_UNSUPPORTED
    assert call(pos=at(8), pos_bytes=8, pos_batch=-1) == capi.ERR_SHAPE
    assert call(pos=at(8) + 4, pos_bytes=8) == capi.ERR_UNSUPPORTED
    assert call(pmap=(L + 1, 0, 0, 1)) == capi.ERR_SHAPE
    assert call(pmap=(-1, 0, 0, 1)) == capi.ERR_SHAPE
    assert call(strides="null") == capi.ERR_NULL
    assert call(phase=NUL) == capi.ERR_NULL
    assert call(phase=at(7) + 4) == capi.ERR_UNSUPPORTED
    assert call(q=NUL) == capi.ERR_NULL          # an output without its input
    assert call(vo=NUL) == capi.ERR_NULL
    assert call(q=NUL, k=NUL, v=NUL, qo=NUL, ko=NUL, vo=NUL) == capi.ERR_NULL
    assert call(q=at(1) + 1) == capi.ERR_UNSUPPORTED     # less than its element's alignment
    assert call(B=0, q=NUL, qo=NUL) == capi.OK
    assert call(L=0) == capi.OK


def test_rope_refuses_strides_that_overlap_or_run_off(lib):
    ok = 2 * (contiguous(B, HQ, L, D) + 2 * contiguous(B, HKV, L, D))

    def call(i, value, **kw):
        s = list(ok)
        s[i] = value
        return rope_call(lib, strides=s, **kw)

    assert call(0, -1) == capi.ERR_UNSUPPORTED
    assert call(9, 1 << 62) == capi.ERR_UNSUPPORTED
    assert call(10, 0) == capi.ERR_UNSUPPORTED      # two heads of an output in one place
    assert call(11, D - 1) == capi.ERR_UNSUPPORTED  # tokens of an output that overlap
    # outputs over each other, over another's input, or shifted over their own
    assert rope_call(lib, ko=at(4)) == capi.ERR_UNSUPPORTED
    assert rope_call(lib, ko=at(1)) == capi.ERR_UNSUPPORTED
    assert rope_call(lib, qo=at(1) + 128) == capi.ERR_UNSUPPORTED
    # an output over the positions or the frequencies
    assert rope_call(lib, pos=at(4) + 64, pos_bytes=8) == capi.ERR_UNSUPPORTED
    assert rope_call(lib, phase=at(6)) == capi.ERR_UNSUPPORTED
    # in place with other strides is not in place
    s = list(ok)
    s[9:12] = [L * HQ * D, D, HQ * D]
    assert rope_call(lib, qo=at(1), strides=s) == capi.ERR_UNSUPPORTED
    # q and k outputs of one packed buffer that share a head
    H = HQ + 2 * HKV
    packed = [L * H * D, D, H * D]
    s = ok[:9] + 3 * packed
    assert rope_call(lib, qo=at(4), ko=at(4) + 2 * (HQ - 1) * D, vo=at(4) + 2 * (HQ + HKV) * D,
                     strides=s) == capi.ERR_UNSUPPORTED


@pytest.mark.parametrize("L_,n,causal,schedule", [(96, 3, False, "fold"), (96, 3, True, "fold"), (96, 4, True, "striped"),
                                                  (96, 4, False, "striped"), (96, 6, True, "contiguous"),
                                                  (96, 6, True, "dfa"), (8, 1, True, "fold"), (4, 2, True, "fold")])
def test_chunk_positions_partition_the_sequence(lib, L_, n, causal, schedule):
    seen = []
    for r in range(n):
        m = ra.chunk_positions(L_, n, causal, r, schedule=schedule)
        rows = [m.base0 + m.step * i if i < m.split else m.base1 + m.step * (i - m.split) for i in range(m.length)]
        assert m.length == L_ // n
        if schedule == "fold":
            assert all(oracle.owner_rank(L_, n, causal, p) == r for p in rows)
            assert rows == sorted(rows)
        elif schedule == "striped":
            assert rows == list(range(r, L_, n))
        else:
            assert rows == list(range(r * (L_ // n), (r + 1) * (L_ // n)))
        seen += rows
    assert sorted(seen) == list(range(L_))


@pytest.mark.parametrize("U,R,causal", [(1, 1, True), (4, 1, True), (2, 3, True), (2, 3, False), (3, 2, True)])
def test_usp_positions_partition_the_sequence(U, R, causal):
    L_ = 72
    seen = []
    for n in range(U * R):
        m = ra.usp_positions(L_, U, R, causal, n)
        r, u = n // U, n % U
        C = L_ // (U * R)
        for i in range(m.length):
            p = m.base0 + m.step * i if i < m.split else m.base1 + m.step * (i - m.split)
            if causal and R > 1:   # the map of the header, term by term
                c = L_ // (2 * R)
                want = r * c + u * c // U + i if i < c // U else (2 * R - 1 - r) * c + u * c // U + i - c // U
            else:
                want = n * C + i
            assert p == want
            seen.append(p)
    assert sorted(seen) == list(range(L_))


def test_position_maps_refuse_bad_chunks():
    for args in ((10, 4, False, 0), (12, 4, True, 0), (16, 4, True, 4), (16, 4, True, -1), (16, 0, True, 0)):
        with pytest.raises(ValueError):
            ra.chunk_positions(*args)
    for args in ((10, 2, 2, True, 0), (12, 2, 2, True, 0), (16, 2, 2, True, 4), (16, 0, 2, True, 0)):
        with pytest.raises(ValueError):
            ra.usp_positions(*args)


def test_frequencies():
    f = ra.RotaryFrequencies(64, base=500.0, device="cpu")
    assert f.rotary_dim == 64 and f.attention_factor == 1.0
    for i, v in enumerate(f.inv_freq):
        assert v == pytest.approx(500.0 ** (-2 * i / 64), rel=1e-15)
    # the phase is the frequency in turns as a 64-bit fraction
    for v, p in zip(f.inv_freq, f.phase.tolist()):
        assert (p % 2 ** 64) / 2 ** 64 * 2 * math.pi == pytest.approx(v, rel=1e-12)
    # frequencies of several turns, and negative ones, keep their fraction
    p = ra.RotaryFrequencies(4, inv_freq=[2 * math.pi * 3.25, -math.pi / 2], device="cpu").phase.tolist()
    assert p[0] / 2 ** 64 % 1 == pytest.approx(0.25, abs=1e-14)
    assert p[1] / 2 ** 64 % 1 == pytest.approx(0.75, abs=1e-14)
    assert ra.RotaryFrequencies(0, device="cpu").phase.numel() == 0


def test_frequency_scalings():
    R, base, orig, s = 64, 10000.0, 4096, 8.0
    plain = [base ** (-2 * i / R) for i in range(R // 2)]
    lin = ra.RotaryFrequencies(R, base, scaling="linear", factor=s, device="cpu")
    assert lin.inv_freq == pytest.approx([v / s for v in plain], rel=1e-14)
    ntk = ra.RotaryFrequencies(R, base, scaling="ntk", factor=s, device="cpu").inv_freq
    assert ntk[0] == 1.0 and ntk[-1] == pytest.approx(plain[-1] / s, rel=1e-12)
    yarn = ra.RotaryFrequencies(R, base, scaling="yarn", factor=s, original_length=orig, device="cpu")
    wave = ra.RotaryFrequencies(R, base, scaling="wavelength", factor=s, original_length=orig, device="cpu")
    assert yarn.attention_factor == pytest.approx(0.1 * math.log(s) + 1)
    assert wave.attention_factor == 1.0
    for v, y, w in zip(plain, yarn.inv_freq, wave.inv_freq):
        turns = orig * v / (2 * math.pi)
        assert v / s * (1 - 1e-12) <= y <= v * (1 + 1e-12) and v / s * (1 - 1e-12) <= w <= v * (1 + 1e-12)
        if turns > 64:
            assert y == pytest.approx(v, rel=1e-12) and w == pytest.approx(v, rel=1e-12)
        if turns < 0.5:
            assert y == pytest.approx(v / s, rel=1e-12) and w == pytest.approx(v / s, rel=1e-12)
    for y in (yarn.inv_freq, wave.inv_freq):
        assert all(a > b for a, b in zip(y, y[1:]))
    assert ra.RotaryFrequencies(R, scaling="yarn", factor=s, original_length=orig, attention_factor=1.0,
                                device="cpu").attention_factor == 1.0


@pytest.mark.parametrize("kw", [dict(rotary_dim=7), dict(rotary_dim=-2), dict(rotary_dim=8, base=1.0),
                                dict(rotary_dim=8, scaling="linear", factor=0.0), dict(rotary_dim=8, scaling="yarn", factor=2.0),
                                dict(rotary_dim=8, scaling="other"), dict(rotary_dim=8, inv_freq=[1.0]),
                                dict(rotary_dim=2, inv_freq=[math.inf]), dict(rotary_dim=2, inv_freq=[1.0], scaling="linear"),
                                dict(rotary_dim=8, attention_factor=math.nan),
                                dict(rotary_dim=8, scaling="wavelength", factor=2.0, original_length=64, low_turns=4.0),
                                dict(rotary_dim=8, scaling="yarn", factor=2.0, original_length=64, beta_fast=1.0)])
def test_frequencies_refuse(kw):
    with pytest.raises(ValueError):
        ra.RotaryFrequencies(device="cpu", **kw)


# ------------------------------------------------------------------ block norms

M, W = 8, 64
LAYER, POST, PRE, SIG = 1, 2, 4, 8


def norm_call(lib, x=at(1), a=at(2), w1=at(3), b1=NUL, gate=at(4), w2=at(5), b2=NUL, y=at(6), h=at(7), stats=at(8),
              ld=(W,) * 5, M=M, D=W, G=1, dx=0, da=0, dg=2, flags=POST | PRE, scale=1.0, eps=1e-6):
    return lib.ring_attn_block_norm_fwd(x, a, w1, b1, gate, w2, b2, y, h, stats, (LL * 5)(*ld) if ld else None, M, D, G,
                                        dx, da, dg, flags, scale, eps, NUL)


def test_block_norm_fwd_refusals(lib):
    def call(**kw):
        return norm_call(lib, **kw)

    assert call(M=-1) == capi.ERR_SHAPE
    assert call(D=0) == capi.ERR_SHAPE
    assert call(G=3) == capi.ERR_SHAPE               # 8 rows
    assert call(G=16) == capi.ERR_SHAPE
    assert call(G=-1) == capi.ERR_SHAPE
    assert call(flags=16) == capi.ERR_SHAPE
    assert call(scale=math.nan) == capi.ERR_SHAPE
    assert call(eps=-1e-6) == capi.ERR_SHAPE
    assert call(eps=math.nan) == capi.ERR_SHAPE
    assert call(D=8193, ld=(8193,) * 5) == capi.ERR_UNSUPPORTED
    assert call(dx=3) == capi.ERR_UNSUPPORTED
    assert call(dx=0, da=1) == capi.ERR_UNSUPPORTED  # bf16 stream, fp16 block
    assert call(dx=0, da=2) == capi.ERR_UNSUPPORTED  # bf16 stream, fp32 block
    assert call(dg=1) == capi.ERR_UNSUPPORTED        # fp16 gate, bf16 block
    assert call(ld=(W - 1,) + (W,) * 4) == capi.ERR_SHAPE
    assert call(ld=(1 << 60,) + (W,) * 4) == capi.ERR_SHAPE
    assert call(ld=None) == capi.ERR_NULL
    assert call(x=NUL) == capi.ERR_NULL
    assert call(y=NUL) == capi.ERR_NULL
    assert call(h=NUL) == capi.ERR_NULL
    assert call(stats=NUL) == capi.ERR_NULL
    assert call(gate=NUL) == capi.ERR_NULL
    assert call(G=0) == capi.ERR_NULL                # a gate, but no rows of it
    assert call(flags=PRE) == capi.ERR_SHAPE         # post weights without the norm
    assert call(flags=POST) == capi.ERR_SHAPE
    assert call(a=NUL) == capi.ERR_SHAPE             # a gate and a post norm of nothing
    assert call(a=NUL, flags=0, w1=NUL, gate=NUL, G=0, y=NUL, h=NUL, w2=NUL) == capi.ERR_SHAPE
    assert call(b1=at(9)) == capi.ERR_SHAPE          # a bias of a root-mean-square norm
    assert call(b2=at(9)) == capi.ERR_SHAPE
    assert call(x=at(1) + 1) == capi.ERR_UNSUPPORTED
    assert call(w1=at(3) + 2) == capi.ERR_UNSUPPORTED
    # outputs over inputs or each other
    assert call(h=at(6)) == capi.ERR_UNSUPPORTED
    assert call(y=at(2)) == capi.ERR_UNSUPPORTED
    assert call(h=at(1)) == capi.ERR_UNSUPPORTED
    assert call(y=at(1) + 2 * W) == capi.ERR_UNSUPPORTED
    assert call(y=at(1), ld=(W, W, W, 2 * W, W)) == capi.ERR_UNSUPPORTED
    assert call(stats=at(6)) == capi.ERR_UNSUPPORTED
    assert call(y=at(5)) == capi.ERR_UNSUPPORTED
    assert call(M=0, x=NUL, stats=NUL) == capi.OK


def norm_bwd_call(lib, dy=at(1), dh=at(2), y=at(3), a=at(4), stats=at(5), w1=at(6), b1=NUL, gate=at(7), w2=at(8),
                  dx=at(9), da=at(10), dg=at(11), dw1=at(12), db1=NUL, dw2=at(13), db2=NUL, ld=(W,) * 7, M=M, D=W, G=1,
                  tx=0, ta=0, tg=2, flags=POST | PRE, scale=1.0, ws=at(14), nws=None):
    need = lib.ring_attn_block_norm_bwd_workspace_size(M, D, G, flags)
    return lib.ring_attn_block_norm_bwd(dy, dh, y, a, stats, w1, b1, gate, w2, dx, da, dg, dw1, db1, dw2, db2,
                                        (LL * 7)(*ld) if ld else None, M, D, G, tx, ta, tg, flags, scale, ws,
                                        need if nws is None else nws, NUL)


def test_block_norm_bwd_refusals(lib):
    def call(**kw):
        return norm_bwd_call(lib, **kw)

    need = lib.ring_attn_block_norm_bwd_workspace_size(M, W, 1, POST | PRE)
    assert need > 0
    assert lib.ring_attn_block_norm_bwd_workspace_size(0, W, 1, POST | PRE) == 0
    assert lib.ring_attn_block_norm_bwd_workspace_size(M, 8193, 1, POST | PRE) == 0
    assert lib.ring_attn_block_norm_bwd_workspace_size(M, W, 3, POST | PRE) == 0
    assert call(ws=NUL) == capi.ERR_WORKSPACE
    assert call(nws=need - 1) == capi.ERR_WORKSPACE
    assert call(ws=at(14) + 16) == capi.ERR_WORKSPACE
    for n in ("dh", "y", "stats", "gate", "dx", "da", "dg", "dw1", "dw2", "ld"):
        assert call(**{n: NUL}) == capi.ERR_NULL, n
    assert call(dy=NUL, flags=POST, dh=NUL, y=NUL, w2=NUL, dw2=NUL) == capi.ERR_NULL
    assert call(M=-1) == capi.ERR_SHAPE
    assert call(G=3) == capi.ERR_SHAPE
    assert call(flags=POST) == capi.ERR_SHAPE
    assert call(flags=PRE) == capi.ERR_SHAPE
    assert call(db1=at(15)) == capi.ERR_SHAPE        # a bias' gradient of a norm without one
    assert call(b1=at(15)) == capi.ERR_SHAPE
    assert call(a=NUL) == capi.ERR_SHAPE
    assert call(ld=(W,) * 6 + (W - 1,)) == capi.ERR_SHAPE
    assert call(tx=0, ta=2) == capi.ERR_UNSUPPORTED
    assert call(dx=at(9) + 1) == capi.ERR_UNSUPPORTED
    assert call(dg=at(11) + 2) == capi.ERR_UNSUPPORTED
    assert call(dx=at(3)) == capi.ERR_UNSUPPORTED    # over y
    assert call(da=at(4)) == capi.ERR_UNSUPPORTED    # over a
    assert call(da=at(9)) == capi.ERR_UNSUPPORTED
    assert call(dx=at(2)) == capi.ERR_UNSUPPORTED
    assert call(dw2=at(12)) == capi.ERR_UNSUPPORTED
    assert call(ws=at(9)) == capi.ERR_UNSUPPORTED    # the workspace over an output
    assert call(ws=at(3)) == capi.ERR_UNSUPPORTED    # ... over an input


def test_block_norm_bwd_of_no_rows_refuses_what_it_cannot_clear(lib):
    def call(**kw):
        return norm_bwd_call(lib, **{**dict(M=0, ws=NUL, dy=NUL, dh=NUL, y=NUL, a=NUL, stats=NUL, dx=NUL, da=NUL), **kw})

    assert call(G=(1 << 40) + 1) == capi.ERR_UNSUPPORTED
    assert call(dg=at(11) + 2) == capi.ERR_UNSUPPORTED   # fp32 sums, whatever the gate's type
    assert call(dg=at(11) + 2, tg=0) == capi.ERR_UNSUPPORTED
    assert call(dw1=at(12) + 2) == capi.ERR_UNSUPPORTED
    assert call(gate=NUL, G=0, dg=NUL, dw1=NUL, dw2=NUL) == capi.OK   # nothing to clear


def test_block_norm_workspace_is_bounded_and_covers_shared_gates(lib):
    f = lib.ring_attn_block_norm_bwd_workspace_size
    small, large = f(4, 256, 0, POST | PRE), f(1 << 22, 256, 0, POST | PRE)
    assert 0 < small <= large <= 2 * 608 * 256 * 4
    assert f(1 << 22, 256, 0, LAYER | POST | PRE) == 2 * large
    assert f(1 << 22, 256, 1, POST | PRE) == large   # one gate row: from the same sums
    assert f(1 << 22, 256, 2, POST | PRE) > large    # several: their units' partial sums


# ------------------------------------------------------------- gradient clipping

def grads_of(ptrs):
    return (ctypes.c_void_p * len(ptrs))(*ptrs)


def clip_call(lib, ins, outs, n, dt=None, dt_out=None, max_norm=1.0, norm=at(60), ws=at(61), nws=None, count=None):
    k = len(ins) if count is None else count
    dt = [0] * len(ins) if dt is None else dt
    nws = lib.ring_attn_grad_workspace_size(max(k, 0)) if nws is None else nws
    return lib.ring_attn_grad_clip(grads_of(ins), grads_of(outs) if outs is not None else None, (LL * len(n))(*n),
                                   (ctypes.c_int * len(dt))(*dt),
                                   (ctypes.c_int * len(dt_out))(*dt_out) if dt_out is not None else None, k, max_norm,
                                   norm, ws, nws, NUL)


def test_grad_clip_refusals(lib):
    n = [100, 200]
    ins = [at(1), at(2)]

    def call(**kw):
        return clip_call(lib, **{**dict(ins=ins, outs=ins, n=n), **kw})

    assert call(count=-1) == capi.ERR_SHAPE
    assert call(n=[100, -1]) == capi.ERR_SHAPE
    assert call(max_norm=-1.0) == capi.ERR_SHAPE
    assert call(max_norm=math.nan) == capi.ERR_SHAPE
    assert call(dt=[0, 3]) == capi.ERR_UNSUPPORTED
    assert call(dt_out=[0, -1]) == capi.ERR_UNSUPPORTED
    assert call(outs=None) == capi.ERR_NULL
    assert call(outs=[at(1), NUL]) == capi.ERR_NULL
    assert call(ins=[NUL, at(2)]) == capi.ERR_NULL
    assert call(norm=NUL) == capi.ERR_NULL
    assert call(norm=at(60) + 2) == capi.ERR_UNSUPPORTED
    assert call(ws=NUL) == capi.ERR_WORKSPACE
    assert call(ws=at(61) + 8) == capi.ERR_WORKSPACE
    assert call(nws=lib.ring_attn_grad_workspace_size(2) - 1) == capi.ERR_WORKSPACE
    assert call(ins=[at(1) + 1, at(2)], outs=[at(1) + 1, at(2)]) == capi.ERR_UNSUPPORTED
    # the same tensor twice, overlapping ones, an output over another's input
    assert call(ins=[at(1), at(1)], outs=[at(1), at(1)]) == capi.ERR_UNSUPPORTED
    assert call(ins=[at(1), at(1) + 100], outs=[at(1), at(1) + 100]) == capi.ERR_UNSUPPORTED
    assert call(outs=[at(3), at(3) + 2]) == capi.ERR_UNSUPPORTED
    assert call(outs=[at(3), at(1) + 198]) == capi.ERR_UNSUPPORTED
    assert call(outs=[at(1) + 2, at(4)]) == capi.ERR_UNSUPPORTED
    assert call(dt_out=[2, 0]) == capi.ERR_UNSUPPORTED   # in place, but of another type
    # the norm inside a tensor, or inside the workspace
    assert call(norm=at(2) + 396) == capi.ERR_UNSUPPORTED
    assert call(outs=[at(5), at(6)], norm=at(2) + 396) == capi.ERR_UNSUPPORTED
    assert call(norm=at(61)) == capi.ERR_UNSUPPORTED
    assert call(ws=at(1)) == capi.ERR_UNSUPPORTED
    assert lib.ring_attn_grad_workspace_size(-1) == 0


def test_grad_norm_and_scale_refusals(lib):
    n, dt = (LL * 1)(100), (ctypes.c_int * 1)(0)
    p = grads_of([at(1)])
    ws = lib.ring_attn_grad_workspace_size(1)
    assert lib.ring_attn_grad_norm(p, n, dt, 1, NUL, at(2), ws, NUL) == capi.ERR_NULL
    assert lib.ring_attn_grad_norm(None, n, dt, 1, at(3), at(2), ws, NUL) == capi.ERR_NULL
    assert lib.ring_attn_grad_norm(p, n, dt, 1, at(3), at(2), ws - 1, NUL) == capi.ERR_WORKSPACE
    assert lib.ring_attn_grad_norm(p, n, dt, 1, at(1), at(2), ws, NUL) == capi.ERR_UNSUPPORTED
    assert lib.ring_attn_grad_scale(p, p, n, dt, None, 1, -1.0, at(3), NUL) == capi.ERR_SHAPE
    assert lib.ring_attn_grad_scale(p, None, n, dt, None, 1, 1.0, at(3), NUL) == capi.ERR_NULL
    assert lib.ring_attn_grad_scale(p, p, n, dt, None, 1, 1.0, NUL, NUL) == capi.ERR_NULL
    assert lib.ring_attn_grad_scale(p, p, n, dt, None, 1, 1.0, at(1), NUL) == capi.ERR_UNSUPPORTED


def test_grad_norm_refuses_more_elements_than_chunks_can_count(lib):
    """The same gradient many times is no conflict; past 2^44 elements in all
    the chunks of a launch would not be counted in 32 bits."""
    def call(k):
        return lib.ring_attn_grad_norm(grads_of([at(1)] * k), (LL * k)(*[1 << 40] * k), (ctypes.c_int * k)(*[0] * k), k,
                                       at(1) + (1 << 60), at(1) + (1 << 61), lib.ring_attn_grad_workspace_size(k), NUL)

    assert call(17) == call(1000) == capi.ERR_UNSUPPORTED


# ------------------------------------------------------- the package's own checks

def test_wrappers_refuse_host_tensors():
    t = torch.zeros(1, 2, 4, 8)
    rope = ra.RotaryFrequencies(8, device="cpu")
    with pytest.raises(TypeError):
        ra.ring_attn_rope_fwd(t, t, rope)
    with pytest.raises(TypeError):
        ra.ring_attn_rope_fwd(t, t, None)
    with pytest.raises(ValueError):
        ra.ring_attn_rope_bwd(None, None, rope)
    with pytest.raises(TypeError):
        ra.ring_attn_block_norm_fwd(t, t)
    with pytest.raises(TypeError):
        ra.ring_attn_block_norm_bwd(t, t, t, t, t)
    with pytest.raises(ValueError):
        ra.ring_attn_block_norm_bwd(None, t, None, t, t)
    with pytest.raises(TypeError):
        ra.GradList([t])
    with pytest.raises(ValueError):
        ra.GradList([t], [t, t])


# ------------------------------------------- the reference against differences

@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("gate,sigmoid", [(0, False), (1, True), (2, False), (6, True)])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True)])
def test_reference_gradients_are_those_of_differences(layer, gate, sigmoid, post, pre):
    g = torch.Generator().manual_seed(3)
    M_, D_ = 6, 10

    def rand(*s):
        return torch.randn(s, generator=g, dtype=torch.float64)

    t = dict(x=rand(M_, D_), a=rand(M_, D_))
    if post:
        t |= dict(w1=rand(D_), b1=rand(D_) if layer else None)
    if pre:
        t |= dict(w2=rand(D_), b2=rand(D_) if layer else None)
    if gate:
        t["g"] = rand(gate, D_)
    dy, dh = rand(M_, D_), rand(M_, D_)

    def forward(t):
        return ref.block_norm(t["x"], t["a"], t.get("w1"), t.get("b1"), t.get("g"), t.get("w2"), t.get("b2"), layer, post,
                              pre, 0.7, sigmoid, 1e-3)[:3]

    def loss(t):
        y, h, _ = forward(t)
        return float((dy * y).sum() + ((dh * h).sum() if pre else 0))

    y, h, stats = forward(t)
    got = ref.block_norm_bwd(dy, dh, y, t["a"], stats, t.get("w1"), t.get("b1"), t.get("g"), t.get("w2"), layer, post, pre,
                             0.7, sigmoid)
    step = 1e-5
    for name, grad in zip(("x", "a", "g", "w1", "b1", "w2", "b2"), got):
        if t.get(name) is None:
            continue
        v = t[name]
        for i in range(0, v.numel(), 7):
            keep = float(v.view(-1)[i])
            v.view(-1)[i] = keep + step
            hi = loss(t)
            v.view(-1)[i] = keep - step
            lo = loss(t)
            v.view(-1)[i] = keep
            want = (hi - lo) / (2 * step)
            assert float(grad[0].reshape(-1)[i]) == pytest.approx(want, rel=1e-6, abs=1e-7), (name, i)
