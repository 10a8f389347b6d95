"""GPU tests of the attention within long molecules (tiles of 128 rows with
their scores in tensor memory) against the float64 oracle, with the bounds of
molecule_util: layouts, ragged ends, scores that rise along the keys
(the softmax reference moves at every stage), molecules without a finite
score, NaN of other molecules, graphs and concurrent streams."""
import numpy as np
import pytest
import torch

from oracle.molecule import molecule_attention
from tests.molecule_util import bounds, close, make, on_gpu, shape_of

pytestmark = pytest.mark.gpu


def _egat():
    from equivariant_graph_attention_b200 import egat
    return egat


def _forward(d, dtype="bf16", **kw):
    t = on_gpu(d, dtype)
    return t, _egat().egat_molecule_attention(shape_of(d, dtype), **t, want_lse=True, **kw)


def _check(d, g=None, dtype="bf16", positions=True):
    o = molecule_attention(**d, grad=g)
    b = bounds(d, o, dtype)
    t, (m, lse) = _forward(d, dtype)
    assert _egat().egat_take_device_status() == _egat().EGAT_OK
    close(m, o["m"], b["m"], "m")
    close(lse, o["lse"], b["lse"], "lse")
    if g is None:
        return m, lse
    got = _egat().egat_molecule_attention_backward(shape_of(d, dtype), m=m, lse=lse, positions=positions,
                                                   grad_m=torch.from_numpy(g).to("cuda", m.dtype), **t)
    assert _egat().egat_take_device_status() == _egat().EGAT_OK
    for x, v in zip(("dq", "dk", "dhp", "dpos_q", "dpos_k", "dslope"), got):
        if v is not None:
            close(v, o[x], b[x], x)
    return m, lse


@pytest.mark.parametrize("layout,lengths", [
    ((2, 128, 16, 16), [1300, 257, 700]), ((3, 128, 16, 16), [600, 901]), ((2, 64, 8, 16), [1500, 900]),
    ((1, 128, 8, 32), [1501, 905]), ((1, 32, 4, 8), [300] * 20), ((0, 16, 2, 8), [201] * 45),
    ((2, 128, 16, 16), [300] * 24), ((3, 128, 16, 16), [193, 400, 257] * 9), ((1, 32, 4, 8), [1000, 0, 1] + [700] * 45),
    ((0, 16, 2, 8), [700] * 10), ((0, 64, 4, 16), [1100] * 5), ((2, 64, 8, 8), [640, 700, 513]),
], ids=str)
@pytest.mark.parametrize("cap", [0.0, 3.0])
def test_layouts(layout, lengths, cap):
    d, g = make("bf16", *layout, lengths, cap=cap, front=3, behind=130)
    m, lse = _check(d, g if len(lengths) < 4 else None)
    for rows in (slice(0, 3), slice(-130, None)):
        assert not m[rows].any() and torch.isneginf(lse[rows]).all()


@pytest.mark.parametrize("bias,positions", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("cap", [0.0, 0.5, 20.0])
def test_caps_and_biases(cap, bias, positions):
    d, g = make("bf16", 2, 128, 16, 16, [1100, 300], cap=cap, bias=bias, scale=4.0)
    _check(d, g, positions=positions)


@pytest.mark.parametrize("queries,keys", [([1300, 700], [200, 900]), ([1200, 900], [0, 800]), ([2100], [449]), ([1200, 900], [0, 1100]), ([600, 1500], [513, 512])], ids=str)
def test_other_keys(queries, keys):
    d, g = make("bf16", 2, 128, 16, 16, keys, queries=queries, cap=5.0, behind=2)
    _check(d, g)


@pytest.mark.parametrize("lengths", [[1300], [300] * 24, [90, 70]], ids=str)
@pytest.mark.parametrize("cap", [0.0, 200.0])
def test_scores_that_rise_along_the_keys(lengths, cap):
    """Every stage passes the last one's reference, and sums and accumulators are rescaled; in reverse no
    stage after the first does."""
    d, g = make("bf16", 2, 128, 16, 16, lengths, cap=cap, bias=False)
    from oracle.storage import round_bf16
    for sign in (1, -1):
        for a, b in zip(d["q_ptr"], d["q_ptr"][1:]):
            d["k"][a:b] = round_bf16(np.linspace(-6, 6, b - a)[::sign, None, None] + 0 * d["k"][a:b])
            d["q"][a:b] = round_bf16(1.0 + 0.5 * np.abs(d["q"][a:b]))
        _check(d, g if len(lengths) < 4 else None)


@pytest.mark.parametrize("lengths", [[400, 700, 333], [640, 701, 577]], ids=str)
def test_nan_stays_in_its_molecule(lengths):
    d, _ = make("bf16", 2, 128, 16, 16, lengths, front=1, behind=4)
    _, (m, lse) = _forward(d)
    a, b = d["q_ptr"][1], d["q_ptr"][2]
    for n in ("k", "hp", "pos_q"):
        d[n][a:b:3], d[n][a + 1:b:3] = np.nan, np.inf
        d[n][:1], d[n][d["q_ptr"][-1]:] = np.nan, -np.inf
    _, (m2, lse2) = _forward(d)
    keep = torch.ones(m.shape[0], dtype=torch.bool)
    keep[a:b] = False
    assert torch.equal(m2[keep], m[keep]) and torch.equal(lse2[keep], lse[keep])
    assert torch.isnan(m2[a:b]).any()


@pytest.mark.parametrize("keys", [449, 577])
def test_keys_at_infinite_distance_have_no_weight(keys):
    d, _ = make("bf16", 2, 128, 16, 16, [keys], queries=[2100])
    d["slope"] = np.abs(d["slope"])
    d["pos_k"][:130] = 3e38                 # the first stages have no finite score
    d["pos_k"][200::9] = 3e38
    keep = np.abs(d["pos_k"][:, 0]) < 1e30
    part = dict(d, k=d["k"][keep], hp=d["hp"][keep], pos_k=d["pos_k"][keep], k_ptr=[0, int(keep.sum())])
    o = molecule_attention(**part)
    b = bounds(part, o, "bf16")
    _, (m, lse) = _forward(d)
    close(m, o["m"], b["m"], "m")
    close(lse, o["lse"], b["lse"], "lse")
    d["pos_k"][:] = 3e38
    _, (m, lse) = _forward(d)
    assert not m.any() and torch.isneginf(lse).all()


def test_replayed_and_on_two_streams_at_once():
    egat = _egat()
    d, _ = make("bf16", 3, 128, 16, 16, [700, 900], cap=20.0)
    shape, (t, (m, lse)) = shape_of(d, "bf16"), _forward(d)
    graph, side = torch.cuda.CUDAGraph(), [torch.cuda.Stream() for _ in range(2)]
    with torch.cuda.graph(graph):
        out = egat.egat_molecule_attention(shape, **t, want_lse=True)
    outs = []
    torch.cuda.synchronize()
    for _ in range(3):
        for s in side:
            with torch.cuda.stream(s):
                outs.append(egat.egat_molecule_attention(shape, **t, want_lse=True))
        graph.replay()
    torch.cuda.synchronize()
    for a, b in outs + [out]:
        assert torch.equal(a, m) and torch.equal(b, lse)
