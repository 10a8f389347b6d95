"""GPU tests of pairs that an infinite coordinate masks, forward and gradients:
an atom at infinity is at an infinite distance from every other one, so its
pairs have no weight, the other rows are those of the system without it, and
its own gradients are zeros."""
import numpy as np
import pytest
import torch

from oracle.molecule import molecule_attention
from tests.molecule_util import bounds, close, make, on_gpu, shape_of

pytestmark = pytest.mark.gpu

FAR = [(np.inf, None, None), (-np.inf, np.inf, -np.inf), (None, 3e38, None), (None, None, -np.inf), (3e38, -3e38, 3e38)]


def _push(pos, rows):
    """Every one of these rows out of reach, each in another way."""
    for i, r in enumerate(rows):
        for c, x in enumerate(FAR[i % len(FAR)]):
            if x is not None:
                pos[r, c] = x


def _without(d, g, kq, kk):
    """The inputs with these query and key rows alone."""
    starts = lambda p, keep: [int(keep[:x].sum()) for x in p]
    return dict(d, q=d["q"][kq], pos_q=d["pos_q"][kq], k=d["k"][kk], hp=d["hp"][kk], pos_k=d["pos_k"][kk],
                q_ptr=starts(d["q_ptr"], kq), k_ptr=starts(d["k_ptr"], kk)), g[kq]


# both storage types on the tensor cores (two heads a warp, one, key values read again) and on the FMA pipe
@pytest.mark.parametrize("dtype,layout,queries,keys", [
    ("bf16", (2, 128, 16, 16), [9, 70], [40, 300]), ("bf16", (1, 32, 4, 8), [33], [150]), ("bf16", (3, 64, 4, 32), [20], [90]),
    ("f32", (2, 128, 16, 16), [9, 70], [40, 300]), ("f32", (2, 128, 8, 32), [20], [90]), ("f32", (3, 128, 8, 16), [9, 40], [30, 90]),
    ("bf16", (1, 32, 1, 8), [9, 40], [30, 90]), ("bf16", (2, 128, 16, 16), [2100], [577]), ("bf16", (2, 128, 16, 16), [3], [4000]),
], ids=str)
@pytest.mark.parametrize("cap", [0.0, 3.0])
@pytest.mark.parametrize("who", ["keys", "queries"])
def test_gradients_beside_masked_pairs(who, cap, dtype, layout, queries, keys):
    from equivariant_graph_attention_b200 import egat
    d, g = make(dtype, *layout, keys, queries=queries, cap=cap, behind=2)
    d["slope"] = np.abs(d["slope"])
    kq, kk = np.ones(d["q"].shape[0], bool), np.ones(d["k"].shape[0], bool)
    keep, pos = (kk, d["pos_k"]) if who == "keys" else (kq, d["pos_q"])
    far = np.arange(1, len(keep) - 2, 4)
    _push(pos, far)
    keep[far] = False
    part, gpart = _without(d, g, kq, kk)
    o = molecule_attention(**part, grad=gpart)
    b = bounds(part, o, dtype)
    shape, t = shape_of(d, dtype), on_gpu(d, dtype)
    m, lse = egat.egat_molecule_attention(shape, **t, want_lse=True)
    out = egat.egat_molecule_attention_backward(shape, m=m, lse=lse, grad_m=torch.from_numpy(g).to("cuda", m.dtype), **t)
    assert egat.egat_take_device_status() == egat.EGAT_OK
    got = dict(zip(("dq", "dk", "dhp", "dpos_q", "dpos_k", "dslope"), out), m=m, lse=lse)
    for x, v in got.items():
        rows = None if x == "dslope" else kq if x in ("m", "lse", "dq", "dpos_q") else kk
        if rows is None:
            close(v, o[x], b[x], x)
            continue
        at = torch.from_numpy(rows)
        close(v[at], o[x], b[x], x)
        empty = v[~at]
        assert (torch.isneginf(empty) if x == "lse" else empty == 0).all(), x
