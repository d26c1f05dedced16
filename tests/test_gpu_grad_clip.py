"""Global gradient norm and clipping on the GB300 against 64 bits.

The norm: a chunk's squares are added in fp32 in chains of at most 64 and
from there in fp64: off by 66 2^-24 of itself at most before the square
root halves it, and its rounding to fp32: below 2.1e-6.  An output takes that
through its factor, which is divided and multiplied (2 2^-24): below 2.3e-6
beside its own rounding."""
import math

import pytest
import torch

import layer_reference as ref
import sequence_blockwise_self_gb300 as ra
from sequence_blockwise_self_gb300 import build as lib_build

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
NORM, OUT = 2.1e-6, 2.3e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    lib_build.build()
    ra.load()


def rand(*shape, dtype=FP, seed=0, mul=0.02):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * mul).to(dtype).cuda()


def norm_of(grads):
    return math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))


def check(grads, outs, max_norm, got_norm, before):
    want = norm_of(before)
    assert got_norm.shape == () and float(got_norm) == pytest.approx(want, rel=NORM, abs=0)
    c = max_norm / want if want > max_norm else 1.0
    for i, (g, o) in enumerate(zip(before, outs)):
        ref.within(f"tensor {i}", o, ref.f64(g) * c, OUT * ref.f64(g).abs() * c)


SIZES = [[1], [7], [16384], [16385, 1, 16383], [100, 0, 3, 50000], [257] * 40, list(range(1, 130)) * 9]


@pytest.mark.parametrize("sizes", SIZES, ids=["one", "seven", "chunk", "around_a_chunk", "an_empty_one", "40", "1161"])
@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("max_norm", [0.01, 1e6])
def test_clip_in_place(sizes, dtype, max_norm):
    grads = [rand(n, dtype=dtype, seed=i) for i, n in enumerate(sizes)]
    before = [g.clone() for g in grads]
    norm = ra.ring_attn_grad_clip(grads, max_norm)
    check(grads, grads, max_norm, norm, before)
    if max_norm > norm_of(before):
        assert all(torch.equal(g, b) for g, b in zip(grads, before))
    assert float(ra.ring_attn_grad_norm(before)) == float(norm)   # the same sum


@pytest.mark.parametrize("src", [BF, HF, FP])
@pytest.mark.parametrize("dst", [BF, HF, FP])
@pytest.mark.parametrize("offset", [0, 1])
def test_outputs_of_other_types_at_any_alignment(src, dst, offset):
    sizes = [40000, 33, 8, 16384]
    flat, out = rand(sum(sizes) + 8, dtype=src), torch.full((sum(sizes) + 8,), 5.0, dtype=dst, device="cuda")
    keep = flat.clone()
    views = [b[offset:offset + sum(sizes)].split(sizes) for b in (flat, out)]
    for max_norm in (0.5, 1e9):
        norm = ra.ring_attn_grad_clip(views[0], max_norm, outs=views[1])
        check(views[0], views[1], max_norm, norm, views[0])
    assert torch.equal(flat, keep)
    assert (out[:offset] == 5).all() and (out[offset + sum(sizes):] == 5).all()


def test_different_alignments_of_a_gradient_and_its_output():
    flat, out = rand(20003, dtype=BF), torch.empty(20010, dtype=BF, device="cuda")
    for i in (0, 1, 3):
        for j in (0, 2, 5):
            g, o = flat[i:i + 20000], out[j:j + 20000]
            check([g], [o], 0.1, ra.ring_attn_grad_clip([g], 0.1, outs=[o]), [g])


def test_mixed_types_shapes_and_absent_gradients():
    grads = [rand(30, 50), None, rand(64, dtype=BF, seed=1), rand(5, 4, 3, 2, dtype=HF, seed=2), rand(1, seed=3)[0]]
    before = [g.clone() for g in grads if g is not None]
    norm = ra.ring_attn_grad_clip(grads, 0.1)
    check(None, [g for g in grads if g is not None], 0.1, norm, before)


def test_no_gradients():
    for grads in ([], [None], [torch.empty(0, device="cuda")]):
        assert float(ra.ring_attn_grad_clip(grads, 1.0)) == 0.0
        assert float(ra.ring_attn_grad_norm(grads)) == 0.0


@pytest.mark.parametrize("value", [1e-30, 1e-22, 3e-39, 1e18, 1e25, 3e37])
@pytest.mark.parametrize("dtype", [FP, BF])
def test_the_norm_of_values_whose_squares_leave_fp32(value, dtype):
    g = torch.full((40,), value, dtype=dtype, device="cuda")
    g[::2] *= -0.5
    norm = ra.ring_attn_grad_norm([g])
    assert float(norm) == pytest.approx(norm_of([g]), rel=NORM)
    mixed = [g, torch.zeros(100, device="cuda")]
    assert float(ra.ring_attn_grad_norm(mixed)) == float(norm)
    max_norm = float(norm) / 4
    if max_norm > 1e-36:   # below, the factor's product is subnormal
        before = [t.clone() for t in mixed]
        check(None, mixed, max_norm, ra.ring_attn_grad_clip(mixed, max_norm), before)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_norm_that_is_not_finite_leaves_the_values(bad):
    grads = [rand(1000), rand(40000, dtype=BF, seed=1)]
    grads[1][777] = bad
    before = [g.clone() for g in grads]
    norm = ra.ring_attn_grad_clip(grads, 0.01)
    assert not math.isfinite(float(norm))
    assert all(torch.equal(g.view(torch.int16 if g.dtype == BF else torch.int32),
                           b.view(torch.int16 if g.dtype == BF else torch.int32)) for g, b in zip(grads, before))
    outs = [torch.zeros_like(g) for g in grads]
    ra.ring_attn_grad_clip(grads, 0.01, outs=outs)   # elsewhere: copied
    assert all(torch.equal(torch.nan_to_num(o), torch.nan_to_num(g)) for o, g in zip(outs, grads))


def test_limits_at_the_border():
    g = torch.tensor([3.0, 4.0], device="cuda")
    assert float(ra.ring_attn_grad_clip([g], 5.0)) == 5.0
    assert g.tolist() == [3.0, 4.0]      # at the limit: as it is
    ra.ring_attn_grad_clip([g], float("inf"))
    assert g.tolist() == [3.0, 4.0]
    ra.ring_attn_grad_clip([g], 0.0)
    assert g.tolist() == [0.0, 0.0]


def test_norm_then_scale_as_ranks_do():
    """Two ranks' norms joined on the device, then each scales by the whole."""
    parts = [[rand(3000)], [rand(500, dtype=BF, seed=1)]]
    before = [[g.clone() for g in p] for p in parts]
    norms = [ra.ring_attn_grad_norm(p) for p in parts]
    whole = torch.stack(norms).square().sum().sqrt()
    for p in parts:
        assert ra.ring_attn_grad_scale(p, 0.1, whole)[0] is p[0]
    n = norm_of([g for p in before for g in p])
    for p, b in zip(parts, before):
        ref.within("scaled", p[0], ref.f64(b[0]) * 0.1 / n, 2 * OUT * ref.f64(b[0]).abs() * 0.1 / n)


def test_a_kept_list_follows_its_tensors():
    """A GradList takes the addresses at each call: a tensor whose storage was
    replaced is followed."""
    g, h = rand(1000), rand(2000, dtype=BF, seed=1)
    kept = ra.GradList([g, None, h])
    assert len(kept) == 2
    assert float(ra.ring_attn_grad_norm(kept)) == pytest.approx(norm_of([g, h]), rel=NORM)
    g.data = rand(1000, seed=9)
    before = [g.clone(), h.clone()]
    norm = ra.ring_attn_grad_clip(kept, 0.05)
    check(None, [g, h], 0.05, norm, before)
    with pytest.raises(ValueError):
        ra.ring_attn_grad_clip(kept, 1.0, outs=[g, h])


def test_streams_graphs_and_the_same_bits():
    grads = [rand(70000), rand(333, dtype=BF, seed=1)]
    outs = [torch.empty_like(g) for g in grads]
    want = ra.ring_attn_grad_clip(grads, 0.1, outs=outs)
    ref_outs = [o.clone() for o in outs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    norm = ra.ring_attn_grad_clip(grads, 0.1, outs=outs, stream=side)
    side.synchronize()
    assert float(norm) == float(want) and all(torch.equal(a, b) for a, b in zip(outs, ref_outs))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = ra.ring_attn_grad_clip(grads, 0.1, outs=outs)
    for seed in (5, 6):
        grads[0].copy_(rand(70000, seed=seed))
        graph.replay()
        check(None, outs, 0.1, norm, grads)


def test_refused():
    g = rand(100)
    with pytest.raises(ra.RingAttnError):
        ra.ring_attn_grad_clip([g, g], 1.0)
    with pytest.raises(ra.RingAttnError):
        ra.ring_attn_grad_clip([g, g[50:]], 1.0)
    with pytest.raises(ra.RingAttnError):
        ra.ring_attn_grad_clip([g], -1.0)
    with pytest.raises(ra.RingAttnError):
        ra.ring_attn_grad_clip([g], float("nan"))
    with pytest.raises(ValueError):
        ra.ring_attn_grad_clip([rand(8, 8).t()], 1.0)
    with pytest.raises(ValueError):
        ra.ring_attn_grad_clip([g], 1.0, outs=[rand(99)])
    with pytest.raises(TypeError):
        ra.ring_attn_grad_norm([torch.zeros(4, dtype=torch.int32, device="cuda")])
    with pytest.raises(ValueError):
        ra.ring_attn_grad_scale([g], 1.0, None)
    # the same gradient read twice is no conflict
    assert float(ra.ring_attn_grad_norm([g, g])) == pytest.approx(norm_of([g, g]), rel=NORM)


def test_past_two_to_the_31_elements():
    n = (1 << 31) + 77
    g = torch.zeros(n, dtype=BF, device="cuda")
    g[-3:] = torch.tensor([3.0, 4.0, 12.0])
    g[0] = 84.0
    norm = ra.ring_attn_grad_clip([g], 17.0)
    assert float(norm) == 85.0
    assert g[-3:].tolist() == [torch.tensor(v * 0.2).to(BF).item() for v in (3.0, 4.0, 12.0)]
    assert g[0].item() == torch.tensor(84 * 0.2).to(BF).item() and not g[1:-3].any()


def test_a_kept_list_refuses_a_tensor_that_became_another():
    """Before anything is launched; where the tensor is as it was again, the
    list is good again."""
    g, h = rand(1000), rand(2000, dtype=BF, seed=1)
    kept = ra.GradList([g, h])
    whole = g.data
    for new in (rand(10), whole.cpu(), whole.to(BF), rand(1).expand(1000), rand(1000, 2)[:, 0]):
        g.data = new
        for call in (ra.ring_attn_grad_norm, lambda k: ra.ring_attn_grad_clip(k, 0.05),
                     lambda k: ra.ring_attn_grad_scale(k, 0.05, torch.ones((), device="cuda"))):
            with pytest.raises((ValueError, TypeError)):
                call(kept)
    g.data = whole
    before = [g.clone(), h.clone()]
    check(None, [g, h], 0.05, ra.ring_attn_grad_clip(kept, 0.05), before)


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("value,max_norm", [(5e37, 1.0), (1e37, 1e-3), (1e36, 1e-8), (3e37, 3e-30)])
def test_a_factor_below_the_normal_range(value, max_norm, dtype):
    """max_norm / norm is subnormal in fp32, the clipped values are not: they
    keep their bits."""
    grads = [torch.full((20,), value, dtype=dtype, device="cuda"), rand(100, seed=1, mul=value / 50).clamp(-value, value)]
    grads[0][::3] *= -0.25
    before = [g.clone() for g in grads]
    norm = ra.ring_attn_grad_clip(grads, max_norm)
    check(None, grads, max_norm, norm, before)
    again = [g.clone() for g in before]
    check(None, ra.ring_attn_grad_scale(again, max_norm, norm), max_norm, norm, before)


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("value", [3e-39, 1e-36, 1e-30, 1.0, 1e37])
def test_a_limit_of_zero(value, dtype):
    """Zeros, however small the norm."""
    grads = [torch.full((40,), value, dtype=dtype, device="cuda"), torch.zeros(10, device="cuda")]
    ra.ring_attn_grad_clip(grads, 0.0)
    assert all((g == 0).all() for g in grads)
    out = torch.ones(40, device="cuda")
    ra.ring_attn_grad_scale([torch.full((40,), value, dtype=dtype, device="cuda")], 0.0, torch.tensor(1e-44, device="cuda"),
                            outs=[out])
    assert (out == 0).all()


@pytest.mark.parametrize("max_norm,norm", [(1e-45, 1e-14), (1e-45, 3e38), (1e-40, 1e-9), (2.0 ** -126, 2.0 ** -25), (200.0, 3e38),
                                           (2.0 ** 27, 2.0 ** 127.99), (2.0 ** -100, 1.0), (2.0 ** -101, 1.0), (1e-38, 1e-7)])
def test_factors_around_the_two_steps(max_norm, norm):
    """Where the factor begins to be applied in two steps, and at its ends."""
    n, m = (float(torch.tensor(v, dtype=FP)) for v in (norm, max_norm))
    g = rand(500, seed=3, mul=norm / 8).clamp(-norm, norm)
    out = torch.empty_like(g)
    ra.ring_attn_grad_scale([g], max_norm, torch.tensor(norm, dtype=FP, device="cuda"), outs=[out])
    ref.within("scaled", out, ref.f64(g) * (m / n), 4 * 2.0 ** -24 * ref.f64(g).abs() * (m / n) + 2.0 ** -149)
