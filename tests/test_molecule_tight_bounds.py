"""The tight bounds of bf16 storage (tests/molecule_tight.py) tell arithmetic that
keeps them from arithmetic that does not: the backward pass is restated in float64
with the roundings of each variant put in by hand.  CPU only."""
import numpy as np
import pytest

from oracle.molecule import _heads, _scores, _unheads, molecule_attention
from oracle.storage import round_bf16
from tests.molecule_tight import tight
from tests.molecule_util import make


def planes(x, n):
    out = np.zeros_like(x)
    for _ in range(n):
        out = out + round_bf16(x - out)
    return out


def restated(d, g, weights=2, ds_planes=2, exact_delta=True, cap_in_correction=True):
    """m, dq, dk, dhp of one molecule (self form, no bias) with the roundings of the kernels."""
    q, k, hp, cap = d["q"], d["k"], d["hp"], d["cap"]
    H, D, C = q.shape[1], hp.shape[1], hp.shape[2]
    x, s, _, _ = _scores(q, k, cap, None, None, None)
    a = np.exp(s - s.max(2, keepdims=True))
    norm = a.sum(2, keepdims=True)
    V, G = _heads(hp, H), _heads(g, H)
    m = round_bf16(_unheads(planes(a, weights) @ V / norm, D, C))
    a = a / norm
    fx = np.cosh(x / cap) ** -2 if cap else np.ones_like(x)
    dP = G @ V.transpose(0, 2, 1)
    delta, stored = (a * dP).sum(2, keepdims=True), (G * _heads(m, H)).sum(2, keepdims=True)
    eps = stored - delta if exact_delta else 0.0
    K, Q, r = k.transpose(1, 0, 2), q.transpose(1, 0, 2), 1 / np.sqrt(q.shape[2])
    fix = planes(a * (fx if cap_in_correction else 1.0), 1)
    dq = planes(a * (dP - stored) * fx, ds_planes) @ K + eps * (fix @ K)
    dS = planes(a * (dP - (delta if exact_delta else stored)) * fx, ds_planes)
    return dict(m=m, dq=round_bf16((dq * r).transpose(1, 0, 2)), dk=round_bf16((dS.transpose(0, 2, 1) @ Q * r).transpose(1, 0, 2)),
                dhp=round_bf16(_unheads(planes(a, weights).transpose(0, 2, 1) @ G, D, C)))


def outside(variant, layout=(0, 16, 2, 8), n=4, cap=0.0, scale=0.7):
    """Names of the outputs that leave the bounds in one of 200 molecules of n atoms."""
    seen = set()
    for seed in range(200):
        d, g = make("bf16", *layout, [n], cap=cap, bias=False, scale=scale, seed=seed)
        o = molecule_attention(**d, grad=g)
        b = tight(d, o)
        seen |= {x for x, v in restated(d, g, **variant).items() if (np.abs(v - o[x]) > b[x]).any()}
    return seen


@pytest.mark.parametrize("layout", [(0, 16, 2, 8), (0, 32, 2, 16), (2, 16, 2, 8)], ids=str)
@pytest.mark.parametrize("n", [4, 16])
@pytest.mark.parametrize("cap", [0.0, 0.1])
def test_two_planes_stay_inside(cap, n, layout):
    assert outside({}, layout, n, cap) == set()


@pytest.mark.parametrize("variant,cap,seen", [
    (dict(weights=1), 0.0, {"m", "dhp"}), (dict(ds_planes=1), 0.0, {"dq", "dk"}), (dict(exact_delta=False), 0.0, {"dq", "dk"}),
    (dict(cap_in_correction=False), 0.1, {"dq"})], ids=str)
@pytest.mark.parametrize("n", [4, 16])
def test_less_is_seen(n, variant, cap, seen):
    assert seen <= outside(variant, n=n, cap=cap)
