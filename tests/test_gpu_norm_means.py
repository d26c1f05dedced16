"""Layer norms' backward of rows whose mean is far above their deviation (an
fp32 stream), against the 64-bit formula from the same statistics.

The normed value (t - mean) rstd is two roundings: 2^-23 of itself, however
large the mean.  So is what hangs on it element by element; what sums over a
row takes E of the sum of magnitudes (layer_reference.py), what sums over M
rows M - 1 roundings in whatever order.
"""
import pytest
import torch

import layer_reference as ref
import sequence_blockwise_self_gb300 as ra
from sequence_blockwise_self_gb300 import build as lib_build

pytestmark = pytest.mark.gpu
FP = torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    lib_build.build()
    ra.load()


def rand(*shape, seed=0, mul=1.0, add=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * mul + add).cuda()


def back(v, ev, hat, r):
    """r (v - mean v - hat mean(v hat)) and its slack."""
    c1, c2 = (v * hat).mean(1, keepdim=True), v.mean(1, keepdim=True)
    ec1 = (ev * hat.abs()).mean(1, keepdim=True) + ref.E * (v * hat).abs().mean(1, keepdim=True)
    ec2 = ev.mean(1, keepdim=True) + ref.E * v.abs().mean(1, keepdim=True)
    out = r * (v - c2 - hat * c1)
    return out, r * (ev + ec2 + hat.abs() * ec1 + ref.E * (v.abs() + c2.abs() + (hat * c1).abs()))


def sums(terms, err):
    return terms.sum(0), terms.shape[0] * U * terms.abs().sum(0) + err.sum(0)


SIZES = [(1, 4096), (3, 64), (9, 1000), (5, 3583), (4, 6152), (3, 8192), (7, 50)]


@pytest.mark.parametrize("mean", [1e3, 3e4, -3e4])
@pytest.mark.parametrize("M,D", SIZES)
def test_the_norm_before_a_block(M, D, mean):
    x = rand(M, D, add=mean)
    w, b = rand(D, seed=1, mul=0.2, add=1), rand(D, seed=2, mul=0.1)
    _, _, stats = ra.ring_attn_block_norm_fwd(x, pre_weight=w, pre_bias=b, norm="layer")
    dy, dh = rand(M, D, seed=3), rand(M, D, seed=4)
    got = ra.ring_attn_block_norm_bwd(dy, dh, x, None, stats, pre_weight=w, pre_bias=b, norm="layer")
    st = ref.f64(stats)
    r, m = st[1][:, None], st[3][:, None]
    hat, d = (ref.f64(x) - m) * r, ref.f64(dh)
    v = d * ref.f64(w)
    part, e = back(v, U * v.abs(), hat, r)
    dx = ref.f64(dy) + part
    ref.within("dx", got[0], dx, e + U * part.abs())
    ref.within("dpre_weight", got[5], *sums(d * hat, 3 * U * (d * hat).abs()))
    ref.within("dpre_bias", got[6], *sums(d, 0 * d))


@pytest.mark.parametrize("mean", [1e3, 3e4, -3e4])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("M,D", SIZES)
def test_the_norm_after_a_block(M, D, gate, mean):
    x, a = rand(M, D), rand(M, D, seed=1, add=mean)
    w, b = rand(D, seed=2, mul=0.2, add=1), rand(D, seed=3, mul=0.1)
    g = {"none": None, "channel": rand(D, seed=5, mul=0.3, add=1), "token": rand(M, D, seed=5, mul=0.3, add=1)}[gate]
    kw = dict(post_weight=w, post_bias=b, gate=g, pre=False, norm="layer")
    y, _, stats = ra.ring_attn_block_norm_fwd(x, a, **kw)
    dy = rand(M, D, seed=4)
    got = ra.ring_attn_block_norm_bwd(dy, None, y, a, stats, **kw)
    assert torch.equal(got[0], dy)
    st = ref.f64(stats)
    r, m = st[0][:, None], st[2][:, None]
    hat, d = (ref.f64(a) - m) * r, ref.f64(dy)
    w, b, e = ref.f64(w), ref.f64(b), 1.0 if g is None else ref.f64(g)
    z = hat * w + b
    # d z: hat's two roundings, the sum's, the product's
    term, err = d * z, U * (3 * (d * hat * w).abs() + 3 * (d * z).abs())
    if gate == "channel" and M > 1:
        # taken as w sum d hat + b sum d: each sum M roundings, then three more
        by = (d * hat * w).abs().sum(0), (d * b).abs().sum(0)
        ref.within("dgate", got[2].view(D), term.sum(0), (M + 6) * U * (by[0] + by[1]))
    elif gate != "none":
        ref.within("dgate", got[2].view(M, D), term, err)
    d = d * e
    v = d * w
    # d g, times w: two roundings (a shared gate: w g, then d)
    da, slack = back(v, 2 * U * v.abs(), hat, r)
    ref.within("da", got[1], da, slack)
    # a shared gate multiplies the sums, the factor rounded once
    ref.within("dpost_weight", got[3], *sums(d * hat, 6 * U * (d * hat).abs()))
    ref.within("dpost_bias", got[4], *sums(d, 3 * U * d.abs()))
