"""GPU tests of how the attention within molecules and the layer norm are called:
a stream of the caller's, workspaces of the caller's, two streams at once, and
tensors whose offsets pass 32 bits."""
import numpy as np
import pytest
import torch

from oracle.molecule import layer_norm, molecule_attention
from tests.molecule_util import U, bounds, close, make, on_gpu, shape_of

pytestmark = pytest.mark.gpu


def _egat():
    from equivariant_graph_attention_b200 import egat
    return egat


def _step(d, g, dtype, t=None, ws=(None, None), stream=None):
    egat = _egat()
    shape = shape_of(d, dtype)
    t = on_gpu(d, dtype) if t is None else t
    m, lse = egat.egat_molecule_attention(shape, **t, want_lse=True, workspace=ws[0], stream=stream)
    return (m, lse) + egat.egat_molecule_attention_backward(shape, m=m, lse=lse, grad_m=g, workspace=ws[1], stream=stream, **t)


def _same(a, b):
    return all((x is None and y is None) or torch.equal(x, y) for x, y in zip(a, b))


SHAPES = [("f32", (1, 32, 4, 8), [60, 9, 130]), ("bf16", (2, 128, 16, 16), [60, 9, 130]), ("bf16", (2, 128, 16, 16), [1300]),
          ("f32", (2, 128, 16, 16), [300])]


@pytest.mark.parametrize("dtype,layout,lengths", SHAPES, ids=str)
def test_a_stream_and_workspaces_of_the_callers(dtype, layout, lengths):
    egat = _egat()
    d, g = make(dtype, *layout, lengths, cap=8.0)
    t = on_gpu(d, dtype)
    G = torch.from_numpy(g).to("cuda", t["q"].dtype)
    ref = _step(d, G, dtype, t)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):                                  # nothing waits in between: buffers of one call are not the next one's
        got = _step(d, G, dtype, t, stream=s)
        torch.empty(1 << 22, device="cuda").fill_(float("nan"))
    s.synchronize()
    assert _same(ref, got)
    shape = shape_of(d, dtype)
    nb = (egat.egat_molecule_attention_workspace_bytes(shape), egat.egat_molecule_attention_backward_workspace_bytes(shape))
    ws = [torch.full((n + 256,), 0xff, dtype=torch.uint8, device="cuda") for n in nb]   # NaN, whatever it is read as
    for _ in range(2):
        assert _same(ref, _step(d, G, dtype, t, ws=[w[:n] if n else None for w, n in zip(ws, nb)]))
    assert all((w[n:] == 0xff).all() for w, n in zip(ws, nb))
    for k in (0, 1):                                    # one byte short is refused
        if nb[k] >= 16:
            short = [None, None]
            short[k] = ws[k][:nb[k] - 1]
            with pytest.raises(egat.EgatError):
                _step(d, G, dtype, t, ws=short)


@pytest.mark.parametrize("dtype,layout,lengths", SHAPES, ids=str)
def test_two_streams_at_once(dtype, layout, lengths):
    d, g = make(dtype, *layout, lengths, cap=8.0)
    t = on_gpu(d, dtype)
    G = torch.from_numpy(g).to("cuda", t["q"].dtype)
    ref = _step(d, G, dtype, t)
    torch.cuda.synchronize()
    side, outs = [torch.cuda.Stream() for _ in range(3)], []
    for _ in range(4):
        for s in side:
            with torch.cuda.stream(s):
                outs.append(_step(d, G, dtype, t))
    torch.cuda.synchronize()
    assert all(_same(ref, o) for o in outs)


def test_refusals_of_the_binding():
    egat = _egat()
    d, g = make("bf16", 2, 128, 16, 16, [20])
    t, shape = on_gpu(d, "bf16"), shape_of(d, "bf16")
    for name, bad in (("q", t["q"].float()), ("k", t["k"][:10]), ("hp", t["hp"].transpose(1, 2)), ("q_ptr", t["q_ptr"].long()),
                      ("pos_q", t["pos_q"].cpu()), ("slope", t["slope"][:4])):
        with pytest.raises(ValueError):
            egat.egat_molecule_attention(shape, **dict(t, **{name: bad}))
    with pytest.raises(egat.EgatError):                 # a bias without positions
        egat.egat_molecule_attention(shape, **dict(t, pos_q=None))
    x = torch.zeros((4, 16), device="cuda")
    for bad in (x.t(), x[:, ::2], x[None], x.half(), torch.zeros(2, 16, device="cuda").expand(2, 16)[:1].expand(4, 16)):
        with pytest.raises(ValueError):
            egat.egat_layer_norm(bad)
    with pytest.raises(ValueError):
        egat.egat_layer_norm(x, weight=torch.zeros(8, device="cuda"))
    with pytest.raises(ValueError):
        egat.egat_layer_norm(x, out=x.bfloat16())


def test_offsets_past_32_bits():
    """1.9 million atoms in molecules of up to 70: 2.2 thousand million values; the last molecules against the
    oracle, forward and gradients."""
    egat = _egat()
    r = np.random.default_rng(3)
    lengths = [60] * 31250 + [70, 1, 33, 64]
    ptr = np.concatenate([[0], np.cumsum(lengths)])
    n, H, dk, D, C = int(ptr[-1]), 16, 16, 9, 128
    assert n * D * C > 2 ** 31
    tail = int(ptr[-5])                                  # the last four molecules
    d, g = make("bf16", 2, C, H, dk, lengths[-4:], cap=5.0)
    t = {"q": torch.zeros((n, H, dk), dtype=torch.bfloat16, device="cuda"), "q_ptr": torch.tensor(ptr, dtype=torch.int32, device="cuda")}
    t["k"], t["hp"] = torch.zeros_like(t["q"]), torch.zeros((n, D, C), dtype=torch.bfloat16, device="cuda")
    G = torch.zeros_like(t["hp"])
    t["pos_q"], t["slope"] = torch.zeros((n, 3), device="cuda"), torch.tensor(d["slope"], dtype=torch.float32, device="cuda")
    for name in ("q", "k", "hp", "pos_q"):
        t[name][tail:] = torch.from_numpy(d[name]).to("cuda", t[name].dtype)
    G[tail:] = torch.from_numpy(g).to("cuda", G.dtype)
    shape = egat.MoleculeShape(nq=n, nk=n, n_mol=len(lengths), lmax=2, C=C, H=H, dk=dk, dtype="bf16", cap=5.0)
    m, lse = egat.egat_molecule_attention(shape, **t, want_lse=True)
    got = egat.egat_molecule_attention_backward(shape, m=m, lse=lse, grad_m=G, **t)
    o = molecule_attention(**d, grad=g)
    b = bounds(d, o, "bf16")
    close(m[tail:], o["m"], b["m"], "m")
    close(lse[tail:], o["lse"], b["lse"], "lse")
    for x, v in zip(("dq", "dk", "dhp", "dpos_q"), got):
        close(v[tail:], o[x], b[x], x)
    assert not m[:tail].any() and not got[2][:tail].any()


def test_layer_norm_offsets_past_32_bits():
    egat = _egat()
    n, W = 2_100_000, 1024
    x = torch.zeros((n, W), dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn((3, W), device="cuda", generator=torch.Generator("cuda").manual_seed(0))
    y, stats = egat.egat_layer_norm(x, want_stats=True)
    dx, dw, db = egat.egat_layer_norm_backward(x, None, stats, x)
    xs = x[-3:].double().cpu().numpy()
    o = layer_norm(xs, grad=xs)
    close(y[-3:], o["y"], (W + 32) * U * (np.abs(o["z"]) + 2) + 2.0 ** -8 * np.abs(o["y"]), "y")
    assert not y[:-3].any() and not dx[:-3].any()
    # zero rows add nothing to the weights' gradients
    close(dw, o["dweight"], (W + 64) * U * (o["abs_dweight"] + 8), "dweight")
    close(db, o["dbias"], (W + 64) * U * (o["abs_dbias"] + 1), "dbias")
