"""The layer operators around the attention: rotary positions, the norms
before and after a block with its gate and residual scale, the global
gradient norm and clipping (include/ring_attn.h).

Argument marshalling only, as in capi.py: every step runs in the library's
kernels and there is no fallback.  The tensors of a call are on one device,
which need not be the current one; `stream` (a torch stream or a raw handle)
defaults to that device's current stream.  Tensors made on another stream
have to be ready on it, as for any CUDA call.
"""
from __future__ import annotations

import array
import contextlib
import ctypes
import math
from fractions import Fraction
from typing import NamedTuple

from . import capi
from .capi import OK, RingAttnError, load, schedule_code

_LL = ctypes.c_longlong
_LL4, _LL5, _LL7, _LL18 = _LL * 4, _LL * 5, _LL * 7, _LL * 18
# 2^256 / (2 pi): a frequency times it is the frequency in turns, to the last
# of the 64 bits that are kept
_TURN = round((1 << 256) / (2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")))

NORM_LAYER, NORM_POST, NORM_PRE, NORM_GATE_SIGMOID = 1, 2, 4, 8

torch = None
_codes = {}      # element type -> RING_ATTN_DTYPE_*
_raw_stream = _current = None


def _lazy():
    """torch, at the first use (the package itself imports without it)."""
    global torch, _raw_stream, _current
    import torch as module
    torch = module
    _codes.update({torch.bfloat16: 0, torch.float16: 1, torch.float32: 2})
    # the small calls are bound by the host: the raw queries where there are any
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda index: torch.cuda.current_stream(index).cuda_stream)
    _current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _code(dtype, name):
    code = _codes.get(dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, got {dtype}")
    return code


def _cuda(t, name):
    """The device index of a CUDA tensor."""
    index = t.get_device() if isinstance(t, torch.Tensor) else -1
    if index < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    return index


def _check(t, name, dtype, index):
    """t is a CUDA tensor of `dtype` (None: any) on device `index`."""
    if isinstance(t, torch.Tensor) and t.get_device() == index and (dtype is None or t.dtype is dtype):
        return
    if _cuda(t, name) != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _stream(stream, index):
    """(raw handle, context in which what the call allocates belongs to that
    stream) of `stream` on device `index`."""
    if stream is None:
        return _raw_stream(index), _HERE
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=index)
    elif stream.device.index != index:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{index}")
    return stream.cuda_stream, torch.cuda.stream(stream)


_HERE = contextlib.nullcontext()


def _call(index, fn, *args):
    if _current() == index:
        rc = fn(*args)
    else:
        with torch.cuda.device(index):
            rc = fn(*args)
    if rc != OK:
        raise RingAttnError(rc, fn.__name__)


def _int32(name, size):
    """Refuses a size (or several or'ed) that the library's ints cannot hold:
    ctypes would cut it."""
    if size >> 31:
        raise RingAttnError(capi.ERR_UNSUPPORTED, name)


def _workspace_bytes(workspace, index):
    _check(workspace, "workspace", None, index)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.numel() * workspace.element_size()


def _p(t):
    return None if t is None else t.data_ptr()


# --------------------------------------------------------------- rotary positions

class PositionMap(NamedTuple):
    """Positions of `length` rows: row l is at base0 + step l, from row
    `split` on at base1 + step (l - split)."""
    length: int
    split: int
    base0: int
    base1: int
    step: int


def chunk_positions(L: int, n_chunks: int, causal: bool, rank: int, striped: bool = False, schedule=None) -> PositionMap:
    """Positions of rank `rank`'s chunk of a sequence of L, in chunk order,
    under the chunk map of ring mode's `schedule` (ring_attn_fwd_step)."""
    L, N, r = int(L), int(n_chunks), int(rank)
    code = schedule_code(striped, schedule)
    if N <= 0 or L < 0 or not 0 <= r < N:
        raise ValueError("needs n_chunks > 0, L >= 0 and 0 <= rank < n_chunks")
    fold = code == capi.SCHEDULES["fold"] and causal
    if L % (2 * N if fold else N):
        raise ValueError(f"L = {L} does not split into {N} {'folded ' if fold else ''}chunks")
    C = L // N
    if code == capi.SCHEDULES["striped"]:
        return PositionMap(C, C, r, 0, N)
    if fold:
        half = C // 2
        return PositionMap(C, half, r * half, (2 * N - 1 - r) * half, 1)
    return PositionMap(C, C, r * C, 0, 1)


def usp_positions(L: int, ulysses_degree: int, ring_degree: int, causal: bool, rank: int) -> PositionMap:
    """Positions of shard `rank` = r U + u of USP's sequence shards
    (ring_attn_usp_fwd); ring_degree 1 is Ulysses."""
    L, U, R, n = int(L), int(ulysses_degree), int(ring_degree), int(rank)
    if U <= 0 or R <= 0 or L < 0 or not 0 <= n < U * R:
        raise ValueError("needs positive degrees, L >= 0 and 0 <= rank < U R")
    fold = bool(causal) and R > 1
    if L % (U * R * (2 if fold else 1)):
        raise ValueError(f"L = {L} does not split into {U * R} shards")
    C = L // (U * R)
    if not fold:
        return PositionMap(C, C, n * C, 0, 1)
    r, u = divmod(n, U)
    piece = C // 2
    c = U * piece
    return PositionMap(C, piece, r * c + u * piece, (2 * R - 1 - r) * c + u * piece, 1)


class RotaryFrequencies:
    """The frequencies of rotary positions: pair i of rotary_dim / 2 turns by
    inv_freq[i] radians a position, inv_freq[i] = base^(-2 i / rotary_dim),
    changed for a longer context by `scaling`:
      None          as they are
      "linear"      inv_freq / factor (positions compressed)
      "ntk"         base grown to base factor^(rotary_dim / (rotary_dim - 2)),
                    so that the slowest pair is slowed by `factor`
      "yarn"        pairs that turn more than beta_fast times over
                    original_length as they are, those that turn less than
                    beta_slow times divided by factor, linearly between in the
                    pair's index; cos and sin times 0.1 ln(factor) + 1
      "wavelength"  pairs that turn more than high_turns times over
                    original_length as they are, those that turn less than
                    low_turns times divided by factor, linearly between in the
                    number of turns
    inv_freq passes the frequencies themselves (any finite values), in
    place of base and scaling.  attention_factor overrides the factor of cos
    and sin.  Kept by a program next to its weights: `phase` is a device
    tensor (int64 bits of the unsigned fraction of a turn a position)."""

    def __init__(self, rotary_dim: int, base: float = 10000.0, scaling=None, factor: float = 1.0, original_length=None,
                 beta_fast: float = 32.0, beta_slow: float = 1.0, low_turns: float = 1.0, high_turns: float = 4.0,
                 attention_factor=None, inv_freq=None, device=None):
        if torch is None:
            _lazy()
        R = int(rotary_dim)
        if R < 0 or R % 2:
            raise ValueError("rotary_dim must be even and not negative")
        scale = 1.0
        if inv_freq is not None:
            if scaling is not None:
                raise ValueError("inv_freq stands in place of base and scaling")
            f = [float(v) for v in inv_freq]
            if len(f) != R // 2:
                raise ValueError(f"{R // 2} frequencies wanted, got {len(f)}")
        else:
            if not base > 1 or not math.isfinite(base):
                raise ValueError("base must be finite and above 1")
            if not factor > 0 or not math.isfinite(factor):
                raise ValueError("factor must be finite and positive")
            if scaling in ("yarn", "wavelength") and not (original_length and original_length > 0):
                raise ValueError(f"{scaling} needs original_length")
            if scaling == "ntk" and R > 2:
                base = base * factor ** (R / (R - 2))
            f = [base ** (-2.0 * i / R) for i in range(R // 2)]
            if scaling == "linear":
                f = [v / factor for v in f]
            elif scaling == "yarn":
                if not beta_fast > beta_slow > 0:
                    raise ValueError("needs beta_fast > beta_slow > 0")

                def index(turns):  # the pair (a fraction of one too) that turns so often over original_length
                    return R * math.log(original_length / (2 * math.pi * turns)) / (2 * math.log(base))

                low, high = max(math.floor(index(beta_fast)), 0), min(math.ceil(index(beta_slow)), R - 1)
                ramp = [min(1.0, max(0.0, (i - low) / max(high - low, 1e-3))) for i in range(R // 2)]
                f = [v / factor * t + v * (1 - t) for v, t in zip(f, ramp)]
                scale = 0.1 * math.log(factor) + 1.0
            elif scaling == "wavelength":
                if not high_turns > low_turns > 0:
                    raise ValueError("needs high_turns > low_turns > 0")
                turns = [original_length * v / (2 * math.pi) for v in f]
                keep = [min(1.0, max(0.0, (t - low_turns) / (high_turns - low_turns))) for t in turns]
                f = [v / factor * (1 - t) + v * t for v, t in zip(f, keep)]
            elif scaling not in (None, "ntk"):
                raise ValueError(f"unknown scaling {scaling!r}")
        if not all(math.isfinite(v) for v in f):
            raise ValueError("the frequencies must be finite")
        scale = float(attention_factor) if attention_factor is not None else scale
        if not math.isfinite(scale):
            raise ValueError("attention_factor must be finite")
        self.rotary_dim, self.inv_freq, self.attention_factor = R, tuple(f), scale
        bits = []
        for v in f:
            n, e = v.as_integer_ratio()   # e is a power of two
            shift = 192 + e.bit_length() - 1
            t = ((n * _TURN + (1 << (shift - 1))) >> shift) % (1 << 64)
            bits.append(t - (1 << 64) if t >= 1 << 63 else t)
        self.phase = torch.tensor(bits, dtype=torch.int64, device="cuda" if device is None else device)


def _head_strides(t, name, shape, dtype, index):
    _check(t, name, dtype, index)
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    s0, s1, s2, s3 = t.stride()
    if s3 != 1 and shape[3] > 1:
        raise ValueError(f"{name}: the elements of a head must be adjacent")
    return s0, s1, s2


def _position_map(*values):
    if not all(-1 << 63 <= v < 1 << 63 for v in values):
        raise ValueError(f"positions past 64 bits: {values}")
    return _LL4(*values)


def _rope(fn, names, ins, outs, rope, positions, interleaved, stream):
    if torch is None:
        _lazy()
    if not isinstance(rope, RotaryFrequencies):
        raise TypeError("rope must be a RotaryFrequencies")
    first = 0 if ins[0] is not None else 1 if ins[1] is not None else 2
    lead = ins[first]
    if lead is None:
        raise ValueError("one tensor at least")
    index = _cuda(lead, names[first])
    dtype, dev = lead.dtype, lead.device
    code = _code(dtype, names[first])
    if lead.dim() != 4:
        raise ValueError(f"{names[first]} must be [B, H, L, d]")
    B, _, L, d = lead.shape
    _int32(fn.__name__, B | L | d)
    raw, allocating = _stream(stream, index)
    strides = [0] * 18
    ptrs, heads, results = [None] * 6, [0, 0, 0], []
    with allocating:
        for i in (0, 1, 2):
            t, out = ins[i], outs[i]
            if t is None:
                if out is not None:
                    raise ValueError(f"{names[i]}_out without {names[i]}")
                continue
            H = t.shape[1] if t.dim() == 4 else 0
            _int32(fn.__name__, H)
            shape = (B, H, L, d)
            strides[3 * i:3 * i + 3] = _head_strides(t, names[i], shape, dtype, index)
            if out is None:
                out = torch.empty(shape, dtype=dtype, device=dev)
                strides[3 * i + 9:3 * i + 12] = (H * L * d, L * d, d)
            else:
                strides[3 * i + 9:3 * i + 12] = _head_strides(out, names[i] + "_out", shape, dtype, index)
            heads[i], ptrs[i], ptrs[i + 3] = H, t.data_ptr(), out.data_ptr()
            results.append(out)
    if ins[1] is not None and ins[2] is not None and heads[1] != heads[2]:
        raise ValueError(f"{names[1]} and {names[2]} must have the same heads")
    pos, pos_bytes, pos_batch, pos_map = None, 0, 0, None
    if positions is None:
        pass
    elif isinstance(positions, torch.Tensor):
        _check(positions, "positions", None, index)
        pos_bytes = 8 if positions.dtype is torch.int64 else 4 if positions.dtype is torch.int32 else 0
        if not pos_bytes:
            raise TypeError(f"positions must be int32 or int64, got {positions.dtype}")
        shape, st = positions.shape, positions.stride()
        if shape != (B, L) and shape != (L,):
            raise ValueError(f"positions has shape {tuple(shape)}, expected {(L,)} or {(B, L)}")
        if L > 1 and st[-1] != 1:
            raise ValueError("the positions of a sequence must be adjacent")
        pos, pos_batch = positions.data_ptr(), st[0] if len(st) == 2 and B > 1 else 0
    elif isinstance(positions, PositionMap):
        if positions.length != L:
            raise ValueError(f"the position map is of {positions.length} rows, the tensors have {L}")
        pos_map = _position_map(*positions[1:])
    elif hasattr(positions, "__index__"):
        pos_map = _position_map(L, positions.__index__(), 0, 1)
    else:
        raise TypeError("positions must be None, an int, a PositionMap or a tensor")
    phase = rope.phase
    if phase.get_device() != index:
        raise ValueError(f"the frequencies are on {phase.device}, the tensors on cuda:{index}")
    _call(index, fn, *ptrs, _LL18(*strides), B, heads[0], heads[1] or heads[2], L, d, rope.rotary_dim, code,
          1 if interleaved else 0, phase.data_ptr(), rope.attention_factor, pos, pos_bytes, pos_batch, pos_map, raw)
    return tuple(results)


def ring_attn_rope_fwd(q, k, rope, positions=None, v=None, interleaved: bool = False, q_out=None, k_out=None, v_out=None,
                       stream=None):
    """Rotary positions: q [B, Hq, L, d] and k [B, Hkv, L, d] rotated by their
    positions over the first rope.rotary_dim elements of each head, the rest
    copied; v, where given, copied along.  The tensors may be views with any
    strides between batches, heads and tokens (token-major rows of a packed
    projection, say); the outputs are allocated [B, H, L, d] contiguous, as
    the attention reads them, unless passed in, also as views; an output may
    be its input.  k may be None.
    positions: None (0 .. L-1), an int (the first row's), a PositionMap
    (chunk_positions, usp_positions), or an int32 or int64 tensor [L] or
    [B, L].  Pairs are (i, i + rotary_dim/2), or (2i, 2i + 1) if interleaved.
    Returns the outputs of the tensors given, in the order q, k, v."""
    return _rope(load().ring_attn_rope_fwd, ("q", "k", "v"), (q, k, v), (q_out, k_out, v_out), rope, positions,
                 interleaved, stream)


def ring_attn_rope_bwd(dq, dk, rope, positions=None, dv=None, interleaved: bool = False, dq_out=None, dk_out=None,
                       dv_out=None, stream=None):
    """Backward of ring_attn_rope_fwd: from the gradients of its outputs those
    of its inputs (dv copied along), with the same choices of views; returns
    the outputs of the tensors given, in the order dq, dk, dv."""
    return _rope(load().ring_attn_rope_bwd, ("dq", "dk", "dv"), (dq, dk, dv), (dq_out, dk_out, dv_out), rope, positions,
                 interleaved, stream)


# ------------------------------------------------- norms, gate and residual scale

def _rows(t, name, dtype, index, shape=None):
    """Elements between the rows of t [..., D], taken as [M, D]."""
    _check(t, name, dtype, index)
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.is_contiguous():
        return t.shape[-1]
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the elements of a row must be adjacent")
    try:
        return t.view(-1, t.shape[-1]).stride(0)
    except RuntimeError:
        raise ValueError(f"{name}: its rows must be one stride apart") from None


def _weight(t, name, D, index):
    if t is None:
        return None
    _check(t, name, torch.float32, index)
    if t.shape != (D,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [{D}], got {tuple(t.shape)}")
    return t.data_ptr()


def _gate(gate, M, D, dtype, index):
    """(gate rows, their stride, type code) of a gate [D], [G, D] or [..., D]."""
    if gate is None:
        return 0, 0, 0
    if gate.dim() < 1 or gate.shape[-1] != D:
        raise ValueError(f"gate must be [..., {D}], got {tuple(gate.shape)}")
    stride = _rows(gate, "gate", None, index)
    if gate.dtype is not torch.float32 and gate.dtype is not dtype:
        raise TypeError(f"gate must be float32 or {dtype}, got {gate.dtype}")
    G = gate.numel() // D
    if M > 0 and (G == 0 or M % G):
        raise ValueError(f"{G} gate rows do not divide {M} rows")
    return G, stride, _code(gate.dtype, "gate")


_NORMS = {"rms": 0, "layer": NORM_LAYER}


def _norm_flags(norm, post, pre, gate_sigmoid):
    if norm not in _NORMS:
        raise ValueError(f"norm must be 'rms' or 'layer', got {norm!r}")
    return (_NORMS[norm] | (NORM_POST if post else 0) | (NORM_PRE if pre else 0)
            | (NORM_GATE_SIGMOID if gate_sigmoid else 0))


def ring_attn_block_norm_fwd(x, a=None, post_weight=None, post_bias=None, gate=None, pre_weight=None, pre_bias=None,
                             norm: str = "rms", post: bool = True, pre: bool = True, scale: float = 1.0,
                             gate_sigmoid: bool = False, eps: float = 1e-6, y=None, h=None, stats=None, stream=None):
    """The norms before and after a block, fused with its gate, residual
    scale and residual: for the residual stream x [..., D] and the block's
    output a [..., D],
      z = N_post(a),  y = x + scale g z,  h = N_pre(y)
    with N a root-mean-square norm (weights fp32 [D], 1 where absent) or a
    layer norm (and biases, 0 where absent); post=False: z = a; pre=False: no h.  gate: [D],
    [G, D] with G dividing the rows (row m takes gate row m // (M / G): one
    per sequence, say) or one row a token, a's type or fp32; gate_sigmoid
    takes its sigmoid.  a=None: only h = N_pre(x).  x is a's type or fp32;
    rows may be any one stride apart.  y may be x, h may be a.
    Returns (y, h, stats); h is None without pre, y is x without a; stats
    (fp32 [2, M], layer norms [4, M]) is what the backward wants."""
    if torch is None:
        _lazy()
    index = _cuda(x, "x")
    shape, dtype = x.shape, x.dtype
    D = shape[-1] if len(shape) else 0
    if D == 0:
        raise ValueError("x must be [..., D]")
    if a is None and (gate is not None or y is not None or post_weight is not None or post_bias is not None):
        raise ValueError("a gate, a post norm or y without a")
    if norm != "layer" and (post_bias is not None or pre_bias is not None):
        raise ValueError("a bias of a root-mean-square norm")
    _int32("ring_attn_block_norm_fwd", D)
    M, dev = x.numel() // D, x.device
    raw, allocating = _stream(stream, index)
    flags = _norm_flags(norm, post and a is not None, pre, gate_sigmoid)
    ld_x = _rows(x, "x", None, index)
    ld_a = _rows(a, "a", None, index, shape) if a is not None else 0
    block = a.dtype if a is not None else h.dtype if h is not None else dtype
    G, ld_g, dt_g = _gate(gate, M, D, block, index)
    rows = 4 if flags & NORM_LAYER else 2
    ld_y = ld_h = D
    with allocating:
        if a is not None:
            if y is None:
                y = torch.empty(shape, dtype=dtype, device=dev)
            else:
                ld_y = _rows(y, "y", dtype, index, shape)
        if h is not None:
            ld_h = _rows(h, "h", block, index, shape)
        elif pre:
            h = torch.empty(shape, dtype=block, device=dev)
        if stats is None:
            stats = torch.empty((rows, M), dtype=torch.float32, device=dev)
        else:
            _stats(stats, rows, M, index)
    _call(index, load().ring_attn_block_norm_fwd, x.data_ptr(), _p(a), _weight(post_weight, "post_weight", D, index),
          _weight(post_bias, "post_bias", D, index), _p(gate), _weight(pre_weight, "pre_weight", D, index),
          _weight(pre_bias, "pre_bias", D, index), _p(y), _p(h), stats.data_ptr(), _LL5(ld_x, ld_a, ld_g, ld_y, ld_h), M, D,
          G, _code(dtype, "x"), _code(block, "a"), dt_g, flags, scale, eps, raw)
    return (y if a is not None else x), h, stats


def _stats(stats, rows, M, index):
    _check(stats, "stats", torch.float32, index)
    if stats.shape != (rows, M) or not stats.is_contiguous():
        raise ValueError(f"stats must be a contiguous [{rows}, {M}], got {tuple(stats.shape)}")


def block_norm_bwd_workspace_size(M: int, D: int, gate_rows: int = 0, norm: str = "rms") -> int:
    _int32("ring_attn_block_norm_bwd_workspace_size", int(D))
    return int(load().ring_attn_block_norm_bwd_workspace_size(int(M), int(D), int(gate_rows),
                                                              _norm_flags(norm, True, True, False)))


def ring_attn_block_norm_bwd(dy, dh, y, a, stats, post_weight=None, post_bias=None, gate=None, pre_weight=None,
                             pre_bias=None, norm: str = "rms", post: bool = True, pre: bool = True, scale: float = 1.0,
                             gate_sigmoid: bool = False, dx=None, da=None, workspace=None, stream=None):
    """Backward of ring_attn_block_norm_fwd: from dy and dh, the gradients of
    y (None for none) and of h (None without pre), with the forward's y (its x
    without a), a and stats, returns (dx, da, dgate, dpost_weight, dpost_bias,
    dpre_weight, dpre_bias), None for what the forward did not take.  dx, da
    are of y's and a's type, weights' gradients fp32; dgate [G, D] is fp32
    where rows share a gate row (zeros where there are no rows), else -- as
    many gate rows as rows, one and one too -- of the gate's type and shape.
    dx may be dy, da may be dh."""
    if torch is None:
        _lazy()
    x = y if y is not None else dy
    if x is None:
        raise ValueError("y or dy is needed")
    index = _cuda(x, "y" if y is not None else "dy")
    shape, dtype = x.shape, x.dtype
    D = shape[-1] if len(shape) else 0
    if D == 0:
        raise ValueError("y must be [..., D]")
    if pre and (dh is None or y is None):
        raise ValueError("dh and y are needed for the pre norm")
    if not pre and (dy is None or a is None):
        raise ValueError("dy and a are needed without the pre norm")
    if a is None and (gate is not None or da is not None or post_weight is not None or post_bias is not None):
        raise ValueError("a gate, a post norm or da without a")
    if norm != "layer" and (post_bias is not None or pre_bias is not None):
        raise ValueError("a bias of a root-mean-square norm")
    if not pre and (pre_weight is not None or pre_bias is not None):
        raise ValueError("pre-norm weights without the pre norm")
    if not post and (post_weight is not None or post_bias is not None):
        raise ValueError("post-norm weights without the post norm")
    _int32("ring_attn_block_norm_bwd", D)
    M, dev = x.numel() // D, x.device
    raw, allocating = _stream(stream, index)
    flags = _norm_flags(norm, post and a is not None, pre, gate_sigmoid)
    layer = flags & NORM_LAYER
    block = a.dtype if a is not None else dh.dtype
    ld_dy = _rows(dy, "dy", dtype, index, shape) if dy is not None else 0
    ld_dh = ld_y = ld_a = 0
    if pre:
        ld_dh, ld_y = _rows(dh, "dh", block, index, shape), _rows(y, "y", dtype, index, shape)
    if a is not None:
        ld_a = _rows(a, "a", block, index, shape)
    _stats(stats, 4 if layer else 2, M, index)
    G, ld_g, dt_g = _gate(gate, M, D, block, index)
    post_w, post_b = _weight(post_weight, "post_weight", D, index), _weight(post_bias, "post_bias", D, index)
    pre_w, pre_b = _weight(pre_weight, "pre_weight", D, index), _weight(pre_bias, "pre_bias", D, index)
    wanted = (post_w is not None, layer and post_b is not None, pre_w is not None, layer and pre_b is not None)
    lib = load()
    ld_dx = ld_da = D
    dgate = None
    with allocating:
        if dx is None:
            dx = torch.empty(shape, dtype=dtype, device=dev)
        else:
            ld_dx = _rows(dx, "dx", dtype, index, shape)
        if da is not None:
            ld_da = _rows(da, "da", block, index, shape)
        elif a is not None:
            da = torch.empty(shape, dtype=block, device=dev)
        if gate is not None:
            if G < M or M == 0 and G > 0:   # (no rows: sums over none, written as zeros)
                dgate = torch.empty((G, D), dtype=torch.float32, device=dev)
            else:
                dgate = torch.empty(gate.shape, dtype=gate.dtype, device=dev)
        sums = [torch.empty(D, dtype=torch.float32, device=dev) if w else None for w in wanted]
        if workspace is None:
            need = lib.ring_attn_block_norm_bwd_workspace_size(M, D, G, flags)
            workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
        else:
            need = _workspace_bytes(workspace, index)
    _call(index, lib.ring_attn_block_norm_bwd, _p(dy), _p(dh) if pre else None, _p(y) if pre else None, _p(a),
          stats.data_ptr(), post_w, post_b, _p(gate), pre_w, dx.data_ptr(), _p(da), _p(dgate), _p(sums[0]), _p(sums[1]),
          _p(sums[2]), _p(sums[3]), _LL7(ld_dy, ld_dh, ld_y, ld_a, ld_g, ld_dx, ld_da), M, D, G, _code(dtype, "y"),
          _code(block, "a"), dt_g, flags, scale, workspace.data_ptr(), need, raw)
    return (dx, da, dgate, *sums)


# -------------------------------------------------- gradient norm and clipping

class GradList:
    """A list of gradient tensors checked once, for the calls below every
    step: grads (None entries are left out) and, where the results go
    elsewhere than in place, outs of the same sizes.  The tensors themselves
    are kept: where every step makes new ones (zero_grad(set_to_none=True))
    pass the sequence, not a kept list.  Each call takes the addresses anew; a
    tensor found elsewhere than at the last call has had its storage replaced
    and is checked again, and refused where its size, type, device or strides
    are no longer what they were.  (The list holds the storages that it
    checked, so an address that is the same is the same memory; one that a
    tensor has left is free at the next call.)  A kept tensor must not be
    resized or viewed otherwise over the storage that it has."""

    def __init__(self, grads, outs=None):
        self._take(grads, outs)
        self._types = [t.dtype for t in self._tensors]
        self._seen, self._held = self._places(), self._storages()

    @classmethod
    def _for_one_call(cls, grads, outs):
        g = cls.__new__(cls)
        g._take(grads, outs)
        return g

    def _take(self, grads, outs):
        if torch is None:
            _lazy()
        grads = list(grads)
        outs = grads if outs is None else list(outs)
        if len(outs) != len(grads):
            raise ValueError(f"{len(grads)} gradients, {len(outs)} outputs")
        pairs = [(g, o) for g, o in zip(grads, outs) if g is not None]
        self.grads, self.outs = [g for g, _ in pairs], [o for _, o in pairs]
        self.in_place = all(g is o for g, o in pairs)
        self.index = _cuda(self.grads[0], "gradient 0") if pairs else torch.cuda.current_device()
        for i, (g, o) in enumerate(pairs):
            for t, n in ((g, "gradient"), (o, "output")):
                _check(t, f"{n} {i}", None, self.index)
                if not t.is_contiguous():
                    raise ValueError(f"{n} {i} must be contiguous")
            if o.numel() != g.numel():
                raise ValueError(f"output {i} has {o.numel()} elements, its gradient {g.numel()}")
        n = len(pairs)
        self._n = (_LL * n)(*[g.numel() for g in self.grads])
        self._dt = (ctypes.c_int * n)(*[_code(g.dtype, f"gradient {i}") for i, g in enumerate(self.grads)])
        self._dt_out = (ctypes.c_int * n)(*[_code(o.dtype, f"output {i}") for i, o in enumerate(self.outs)])
        self._pointers = ctypes.c_void_p * n
        self._workspace = int(load().ring_attn_grad_workspace_size(n))
        self._tensors = tuple(self.grads if self.in_place else self.grads + self.outs)
        self._held = None

    def __len__(self):
        return len(self._n)

    def _places(self):
        return array.array("Q", map(torch.Tensor.data_ptr, self._tensors))

    def _storages(self):
        return list(map(torch.Tensor.untyped_storage, self._tensors))

    def _addresses(self):
        if not self._tensors:
            return None, None
        at = self._places()
        if self._held is not None and at != self._seen:
            self._check_again()
            self._seen, self._held = at, self._storages()
        ins = self._pointers.from_buffer(at)
        return ins, ins if self.in_place else self._pointers.from_buffer(at, 8 * len(self))

    def _check_again(self):
        n = len(self)
        for i, (t, dtype) in enumerate(zip(self._tensors, self._types)):
            name = f"{'gradient' if i < n else 'output'} {i % n}"
            _check(t, name, dtype, self.index)
            if t.numel() != self._n[i % n]:
                raise ValueError(f"{name} has {t.numel()} elements, {self._n[i % n]} when the list was made")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")


def _grads(grads, outs):
    if isinstance(grads, GradList):
        if outs is not None:
            raise ValueError("a GradList has its outputs already")
        return grads
    return GradList._for_one_call(grads, outs)


def _norm_out(norm, index):
    if norm is None:
        return torch.empty((), dtype=torch.float32, device=torch.device("cuda", index))
    _check(norm, "norm", torch.float32, index)
    if norm.numel() != 1:
        raise ValueError("norm must have one element")
    return norm


def grad_workspace_size(n_tensors: int) -> int:
    return int(load().ring_attn_grad_workspace_size(int(n_tensors)))


def _grad_workspace(workspace, need, index):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=torch.device("cuda", index)), need
    return workspace, _workspace_bytes(workspace, index)


def ring_attn_grad_norm(grads, norm=None, workspace=None, stream=None):
    """sqrt of the sum of squares over all tensors of `grads` (a sequence, or
    a GradList), as an fp32 tensor of one element on their device.  A tensor
    listed twice counts twice."""
    g = _grads(grads, None)
    raw, allocating = _stream(stream, g.index)
    with allocating:
        norm = _norm_out(norm, g.index)
        ws, size = _grad_workspace(workspace, g._workspace, g.index)
    _call(g.index, load().ring_attn_grad_norm, g._addresses()[0], g._n, g._dt, len(g), norm.data_ptr(), ws.data_ptr(),
          size, raw)
    return norm


def ring_attn_grad_scale(grads, max_norm: float, norm, outs=None, stream=None):
    """out = g max_norm / norm where norm (an fp32 tensor of one element, read
    on the device) is above max_norm, else g, for every tensor of `grads`, in
    place unless `outs` is given (of the same sizes, any of the types).  A
    norm that is not finite leaves the values as they are.  Returns the
    outputs."""
    if norm is None:
        raise ValueError("norm is needed")
    g = _grads(grads, outs)
    raw, _ = _stream(stream, g.index)
    ins, to = g._addresses()
    _call(g.index, load().ring_attn_grad_scale, ins, to, g._n, g._dt, g._dt_out, len(g), max_norm,
          _norm_out(norm, g.index).data_ptr(), raw)
    return list(g.outs)


def ring_attn_grad_clip(grads, max_norm: float, outs=None, norm=None, workspace=None, stream=None):
    """Clips the tensors of `grads` (a sequence, or a GradList) to a global
    norm of max_norm: ring_attn_grad_norm and ring_attn_grad_scale in one
    call, in place unless `outs` is given.  Returns the norm before clipping
    (an fp32 tensor of one element); the host does not wait for it.  Where it
    is not finite the values stay as they are."""
    g = _grads(grads, outs)
    raw, allocating = _stream(stream, g.index)
    with allocating:
        norm = _norm_out(norm, g.index)
        ws, size = _grad_workspace(workspace, g._workspace, g.index)
    ins, to = g._addresses()
    _call(g.index, load().ring_attn_grad_clip, ins, to, g._n, g._dt, g._dt_out, len(g), max_norm, norm.data_ptr(),
          ws.data_ptr(), size, raw)
    return norm
