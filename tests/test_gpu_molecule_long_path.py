"""GPU tests of the tcgen05 attention within long molecules that assert, by the
workspace a call asks for, that it is the kernel that ran: layouts at its least
lengths, caps, rising scores, masked and empty stages, other keys, NaN of other
molecules.  And the FMA kernels over long molecules."""
import numpy as np
import pytest
import torch

from oracle.molecule import molecule_attention
from oracle.storage import round_bf16
from tests.molecule_tight import packed_bytes, tight
from tests.molecule_util import bounds, close, make, on_gpu, shape_of

pytestmark = pytest.mark.gpu


def _forward(d):
    from equivariant_graph_attention_b200 import egat
    shape = shape_of(d, "bf16")
    assert egat.egat_molecule_attention_workspace_bytes(shape) == packed_bytes(shape)
    m, lse = egat.egat_molecule_attention(shape, **on_gpu(d, "bf16"), want_lse=True)
    assert egat.egat_take_device_status() == egat.EGAT_OK
    return m, lse


def _check(d, limits=tight):
    o = molecule_attention(**d)
    b = limits(d, o)
    m, lse = _forward(d)
    close(m, o["m"], b["m"], "m")
    close(lse, o["lse"], b["lse"], "lse")
    return m, lse


@pytest.mark.parametrize("layout,lengths", [
    ((1, 32, 4, 8), [600] * 12), ((0, 16, 2, 8), [513] * 13), ((2, 128, 16, 16), [520, 700, 513]), ((3, 128, 16, 16), [193, 900, 557]),
    ((2, 128, 16, 16), [897]), ((2, 64, 8, 32), [600, 511, 513]), ((1, 128, 8, 32), [512, 513, 640]), ((0, 64, 4, 16), [1, 1700, 900]),
    ((0, 128, 1, 8), [12200]), ((0, 64, 8, 32), [2000, 0, 40]), ((1, 16, 2, 8), [6200]),
], ids=str)
@pytest.mark.parametrize("cap", [0.0, 3.0])
def test_layouts(layout, lengths, cap):
    d, _ = make("bf16", *layout, lengths, cap=cap, front=3, behind=130)
    m, lse = _check(d)
    for rows in (slice(0, 3), slice(-130, None)):
        assert not m[rows].any() and torch.isneginf(lse[rows]).all()


@pytest.mark.parametrize("queries,keys", [([1300, 700], [600, 900]), ([1200, 900], [0, 1100]), ([600, 1500], [513, 512]), ([2100], [512])], ids=str)
@pytest.mark.parametrize("bias", [False, True])
def test_other_keys(bias, queries, keys):
    d, _ = make("bf16", 2, 128, 16, 16, keys, queries=queries, cap=5.0, bias=bias, behind=2)
    _check(d)


@pytest.mark.parametrize("lengths", [[1300], [600] * 3, [512, 800]], ids=str)
@pytest.mark.parametrize("cap", [0.0, 200.0])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_that_rise_along_the_keys(sign, cap, lengths):
    d, _ = make("bf16", 2, 128, 16, 16, lengths, cap=cap, bias=False)
    for a, b in zip(d["q_ptr"], d["q_ptr"][1:]):
        d["k"][a:b] = round_bf16(np.linspace(-6, 6, b - a)[::sign, None, None] + 0 * d["k"][a:b])
        d["q"][a:b] = round_bf16(1.0 + 0.5 * np.abs(d["q"][a:b]))
    _check(d)


@pytest.mark.parametrize("far", [np.inf, -np.inf, 3e38])
def test_stages_without_a_finite_score(far):
    d, _ = make("bf16", 2, 128, 16, 16, [577], queries=[2100])
    d["slope"] = np.abs(d["slope"])
    d["pos_k"][:130], d["pos_k"][200::9] = far, far
    keep = np.abs(d["pos_k"][:, 0]) < 1e30
    part = dict(d, k=d["k"][keep], hp=d["hp"][keep], pos_k=d["pos_k"][keep], k_ptr=[0, int(keep.sum())])
    o = molecule_attention(**part)
    b = tight(part, o)
    m, lse = _forward(d)
    close(m, o["m"], b["m"], "m")
    close(lse, o["lse"], b["lse"], "lse")
    d["pos_k"][:] = far
    m, lse = _forward(d)
    assert not m.any() and torch.isneginf(lse).all()


def test_nan_stays_in_its_molecule():
    d, _ = make("bf16", 2, 128, 16, 16, [640, 701, 577], front=1, behind=4)
    m, lse = _forward(d)
    a, b = d["q_ptr"][1], d["q_ptr"][2]
    for n in ("k", "hp", "pos_q"):
        d[n][a:b:3], d[n][a + 1:b:3] = np.nan, np.inf
        d[n][:1], d[n][d["q_ptr"][-1]:] = np.nan, -np.inf
    m2, lse2 = _forward(d)
    keep = torch.ones(m.shape[0], dtype=torch.bool)
    keep[a:b] = False
    assert torch.equal(m2[keep], m[keep]) and torch.equal(lse2[keep], lse[keep])
    assert torch.isnan(m2[a:b]).any()


# more than 144 value columns a head of float32, one head of few columns of bf16
@pytest.mark.parametrize("dtype,layout,lengths,queries", [
    ("f32", (3, 32, 1, 16), [3000], None), ("f32", (3, 128, 8, 16), [1100], None), ("f32", (3, 128, 8, 16), [5000], [3]),
    ("bf16", (1, 32, 1, 8), [3000], None), ("bf16", (2, 16, 1, 8), [20000], [2])], ids=str)
def test_long_molecules_on_the_fma_pipe(dtype, layout, lengths, queries):
    from equivariant_graph_attention_b200 import egat
    d, g = make(dtype, *layout, lengths, queries=queries, cap=5.0)
    o = molecule_attention(**d, grad=g)
    b = bounds(d, o, dtype) if dtype == "f32" else tight(d, o)
    shape, t = shape_of(d, dtype), on_gpu(d, dtype)
    m, lse = egat.egat_molecule_attention(shape, **t, want_lse=True)
    out = egat.egat_molecule_attention_backward(shape, m=m, lse=lse, grad_m=torch.from_numpy(g).to("cuda", m.dtype), **t)
    got = dict(zip(("dq", "dk", "dhp", "dpos_q", "dpos_k", "dslope"), out), m=m, lse=lse)
    for x, v in got.items():
        if v is not None:
            close(v, o[x], b[x], x)
