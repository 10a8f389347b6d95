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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,width", [(1, 64), (777, 64), (5000, 100), (37, 2000)])
def test_norm_in_place(n, width, dtype):
    """y over x, dx over the gradient and dx over x, rows with a stride: the same bits as elsewhere."""
    egat = _egat()
    gen = torch.Generator("cuda").manual_seed(n)
    base = torch.randn((2, n, 3, width), generator=gen, device="cuda").to(dtype)
    x, g = base[0, :, 1], base[1, :, 1]
    y, stats = egat.egat_layer_norm(x, want_stats=True)
    dx, dw, db = egat.egat_layer_norm_backward(x, None, stats, g)
    for over in ("g", "x"):
        work = base.clone()
        xs, gs = work[0, :, 1], work[1, :, 1]
        out = egat.egat_layer_norm_backward(xs, None, stats, gs, out=gs if over == "g" else xs)
        assert torch.equal(out[0], dx) and torch.equal(out[1], dw) and torch.equal(out[2], db)
        assert torch.equal(work[:, :, ::2], base[:, :, ::2])
    work = base.clone()
    got, _ = egat.egat_layer_norm(work[0, :, 1], out=work[0, :, 1])
    assert torch.equal(got, y) and torch.equal(work[1], base[1]) and torch.equal(work[0, :, ::2], base[0, :, ::2])


def test_norm_over_rows_of_another_stride_is_refused():
    egat = _egat()
    base = torch.randn((100, 2, 64), device="cuda")
    dense = base.view(-1)[:6400].view(100, 64)
    for x, out in ((base[:, 0], dense), (dense, base[:, 0])):
        with pytest.raises(egat.EgatError):
            egat.egat_layer_norm(x, out=out)
        stats = egat.egat_layer_norm(x, want_stats=True)[1]
        with pytest.raises(egat.EgatError):
            egat.egat_layer_norm_backward(x, None, stats, x.clone(), out=out)
    assert egat.egat_layer_norm(base[:1, 0], out=dense[:1])[0].shape == (1, 64)   # one row has no stride
