"""GPU tests of calls of the attention within molecules and the layer norm that
have to be refused, or that the documentation allows at its edges."""
import pytest
import torch

from tests.molecule_util import make, on_gpu, shape_of

pytestmark = pytest.mark.gpu


def _egat():
    from equivariant_graph_attention_b200 import egat
    return egat


@pytest.mark.parametrize("missing", ["pos_q", "pos_k"])
def test_gradients_of_a_bias_without_positions_are_refused(missing):
    egat = _egat()
    d, g = make("bf16", 2, 128, 16, 16, [20], queries=[5])
    t, shape = on_gpu(d, "bf16"), shape_of(d, "bf16")
    m, lse = egat.egat_molecule_attention(shape, **t, want_lse=True)
    t[missing] = None
    for positions in (True, False):
        with pytest.raises(egat.EgatError):
            egat.egat_molecule_attention_backward(shape, m=m, lse=lse, grad_m=m, positions=positions, **t)
