"""Pins of the oracle's attention within molecules and layer norm
(oracle/molecule.py): hand values, differences of the forward for every
gradient, and torch's own softmax and layer norm in float64."""
import numpy as np
import pytest
import torch

from oracle.molecule import layer_norm, molecule_attention


def _case(cap, bias, cross, seed=3):
    r = np.random.default_rng(seed)
    qp = [0, 3, 3, 7, 8]
    kp = [0, 4, 5, 5, 8] if cross else None
    nq, nk, H, dk, D, C = 8, 8, 2, 8, 4, 16
    d = dict(q=r.normal(size=(nq, H, dk)) * 2, k=r.normal(size=(nk, H, dk)) * 2, hp=r.normal(size=(nk, D, C)),
             q_ptr=qp, k_ptr=kp, cap=cap)
    if bias:
        d.update(pos_q=r.normal(size=(nq, 3)), slope=np.array([0.7, -0.3]))
        d["pos_k"] = r.normal(size=(nk, 3)) if cross else None
    return d, r.normal(size=(nq, D, C))


@pytest.mark.parametrize("cap,bias,cross", [(0.0, False, False), (1.5, True, False), (1.5, True, True),
                                            (0.0, True, True)])
def test_gradients_against_differences(cap, bias, cross):
    d, g = _case(cap, bias, cross)
    o = molecule_attention(**d, grad=g)
    names = {"q": "dq", "k": "dk", "hp": "dhp"}
    if bias:
        names.update({"pos_q": "dpos_q", "slope": "dslope"})
        if cross:
            names["pos_k"] = "dpos_k"
    f = lambda dd: float((molecule_attention(**dd)["m"] * g).sum())
    for name, out in names.items():
        for at in np.ndindex(*d[name].shape):
            if sum(at) % 3 and name == "hp":
                continue
            h = 1e-5
            lo, hi = dict(d), dict(d)
            lo[name], hi[name] = d[name].copy(), d[name].copy()
            lo[name][at] -= h
            hi[name][at] += h
            # central difference: h^2 f'''/6 and rounding 2^-52 |f| / h, both far below 1e-6
            assert abs((f(hi) - f(lo)) / (2 * h) - o[out][at]) < 1e-6, (name, at)
        assert np.all(np.abs(o[out]) <= o["abs_" + out] + 1e-12)


def test_hand_values():
    # one atom: its own value, lse = its own score; no keys: zero and -inf
    q = np.array([[[1.0] + [0] * 7]])
    o = molecule_attention(q, 2 * q, np.arange(16.0).reshape(1, 1, 16), [0, 1])
    assert np.array_equal(o["m"][0, 0], np.arange(16.0)) and np.isclose(o["lse"][0, 0], 2 / np.sqrt(8))
    o = molecule_attention(q, np.zeros((0, 1, 8)), np.zeros((0, 1, 16)), [0, 1], [0, 0])
    assert not o["m"].any() and o["lse"][0, 0] == -np.inf
    # two keys, equal scores, the farther one discounted by exp(-slope d)
    o = molecule_attention(0 * q, np.zeros((2, 1, 8)), np.array([[[1.0] * 16], [[3.0] * 16]]), [0, 1], [0, 2],
                           pos_q=np.zeros((1, 3)), pos_k=np.array([[0, 0, 0], [0, 0, np.log(3.0)]]), slope=np.ones(1))
    assert np.allclose(o["m"], (1 * 0.75 + 3 * 0.25))


def test_against_torch_softmax():
    d, _ = _case(2.0, False, False)
    o = molecule_attention(**d)
    q, k, v = (torch.from_numpy(d[n]) for n in ("q", "k", "hp"))
    for a, b in zip(d["q_ptr"], d["q_ptr"][1:]):
        s = 2.0 * torch.tanh(torch.einsum("ihd,jhd->hij", q[a:b], k[a:b]) / 8 ** 0.5 / 2.0)
        w = torch.softmax(s, 2)
        m = torch.einsum("hij,jdhc->idhc", w, v[a:b].view(b - a, 4, 2, 8)).reshape(b - a, 4, 16)
        assert np.allclose(o["m"][a:b], m.numpy(), atol=1e-12)


def test_layer_norm_against_torch():
    r = np.random.default_rng(5)
    x, w, b, g = r.normal(size=(7, 19)) + 3, r.normal(size=19), r.normal(size=19), r.normal(size=(7, 19))
    t = [torch.from_numpy(a).requires_grad_() for a in (x, w, b)]
    y = torch.nn.functional.layer_norm(t[0], (19,), t[1], t[2], eps=1e-5)
    y.backward(torch.from_numpy(g))
    o = layer_norm(x, w, b, grad=g)
    assert np.allclose(o["y"], y.detach().numpy(), atol=1e-12)
    for got, want in ((o["dx"], t[0].grad), (o["dweight"], t[1].grad), (o["dbias"], t[2].grad)):
        assert np.allclose(got, want.numpy(), atol=1e-12)
