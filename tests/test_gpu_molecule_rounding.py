"""GPU tests of bf16 storage against bounds that allow one rounding, that of the
output (tests/molecule_tight.py): weights and dS that entered a product as one bf16
number, a delta from the rounded m or a missing factor of the cap fall outside.
Small scores and short molecules, where the float32 part of the bound is small."""
import pytest
import torch

from oracle.molecule import molecule_attention
from tests.molecule_tight import tight
from tests.molecule_util import close, make, on_gpu, shape_of

pytestmark = pytest.mark.gpu


def _check(d, g=None):
    from equivariant_graph_attention_b200 import egat
    o = molecule_attention(**d, grad=g)
    b = tight(d, o)
    shape, t = shape_of(d, "bf16"), on_gpu(d, "bf16")
    m, lse = egat.egat_molecule_attention(shape, **t, want_lse=True)
    got = {"m": m, "lse": lse}
    if g is not None:
        out = egat.egat_molecule_attention_backward(shape, m=m, lse=lse, grad_m=torch.from_numpy(g).to("cuda", m.dtype), **t)
        got.update({x: v for x, v in zip(("dq", "dk", "dhp", "dpos_q", "dpos_k", "dslope"), out) if v is not None})
    assert egat.egat_take_device_status() == egat.EGAT_OK
    for x, v in got.items():
        close(v, o[x], b[x], x)


# every number of value columns of the tensor-core kernels, and the FMA kernels
@pytest.mark.parametrize("layout", [(0, 16, 2, 8), (0, 64, 4, 16), (1, 16, 2, 8), (1, 64, 4, 16), (2, 64, 8, 16), (2, 128, 16, 16),
                                    (2, 128, 8, 32), (3, 128, 16, 16), (3, 64, 4, 16), (3, 128, 2, 16), (0, 32, 1, 32)], ids=str)
@pytest.mark.parametrize("cap", [0.0, 0.5])
def test_short_molecules(layout, cap):
    d, g = make("bf16", *layout, [33, 1, 20, 64, 90], cap=cap, scale=0.7)
    _check(d, g)


@pytest.mark.parametrize("queries,keys", [([3], [900]), ([7, 0, 20], [200, 40, 0])], ids=str)
def test_few_queries(queries, keys):
    d, g = make("bf16", 2, 128, 16, 16, keys, queries=queries, cap=0.5, scale=0.7)
    _check(d, g)


@pytest.mark.parametrize("layout,lengths", [((2, 128, 16, 16), [1100]), ((3, 128, 16, 16), [600, 700]), ((1, 32, 4, 8), [700] * 6),
                                            ((0, 16, 2, 8), [700] * 10)], ids=str)
@pytest.mark.parametrize("cap", [0.0, 0.5])
def test_long_molecules(layout, lengths, cap):
    d, g = make("bf16", *layout, lengths, cap=cap, scale=0.5)
    _check(d, g if len(lengths) < 4 else None)


# where one plane of the weights or of dS, a delta from the rounded m or a missing factor of the cap are seen
@pytest.mark.parametrize("layout", [(0, 16, 2, 8), (0, 32, 2, 16), (2, 16, 2, 8), (0, 16, 1, 8), (2, 128, 16, 16)], ids=str)
@pytest.mark.parametrize("n", [4, 16])
@pytest.mark.parametrize("cap", [0.0, 0.1])
def test_small_molecules(cap, n, layout):
    d, g = make("bf16", *layout, [n] * 200, cap=cap, bias=False, scale=0.7)
    _check(d, g)
