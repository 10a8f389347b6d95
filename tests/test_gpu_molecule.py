"""GPU tests of the attention within molecules (egat_molecule_attention and its
backward pass) against the float64 oracle, with bounds derived from the
arithmetic (molecule_util): every value layout and storage type, ragged
batches with empty molecules and rows of no molecule, long molecules, few
queries against many keys, caps from tight to loose, NaN in other molecules,
CUDA graphs, other streams, and the path from the scalars' layer norm through
the projection to the gradients."""
import numpy as np
import pytest
import torch

from oracle.molecule import layer_norm, molecule_attention
from oracle.projection import invariant_projection
from tests.molecule_util import U, bounds, close, make, on_gpu, ptr_of, shape_of

pytestmark = pytest.mark.gpu

# (lmax, C, H, dk): every number of value columns from 8 to 2,048, every dk
LAYOUTS = [(0, 16, 2, 8), (0, 64, 4, 16), (0, 32, 1, 32), (1, 16, 2, 8), (1, 64, 4, 16), (2, 64, 8, 16),
           (2, 128, 16, 16), (2, 128, 8, 32), (2, 128, 4, 8), (2, 128, 1, 32), (3, 128, 16, 16), (3, 64, 4, 16),
           (3, 32, 1, 8), (3, 128, 2, 16), (3, 128, 1, 32)]
RAGGED = [1, 0, 5, 33, 0, 0, 17, 64, 2, 129]


def _egat():
    from equivariant_graph_attention_b200 import egat
    return egat


def _forward(d, dtype, want_lse=True, **kw):
    t = on_gpu(d, dtype)
    return t, _egat().egat_molecule_attention(shape_of(d, dtype), **t, want_lse=want_lse, **kw)


def _backward(d, dtype, t, m, lse, g, positions=True, **kw):
    T = m.dtype
    out = _egat().egat_molecule_attention_backward(shape_of(d, dtype), m=m, lse=lse,
                                                   grad_m=torch.from_numpy(g).to("cuda", T), positions=positions, **t, **kw)
    return dict(zip(("dq", "dk", "dhp", "dpos_q", "dpos_k", "dslope"), out))


def _check(d, g, dtype, positions=True):
    o = molecule_attention(**d, grad=g)
    b = bounds(d, o, dtype)
    t, (m, lse) = _forward(d, dtype)
    close(m, o["m"], b["m"], "m")
    close(lse, o["lse"], b["lse"], "lse")
    got = _backward(d, dtype, t, m, lse, g, positions)
    for x, v in got.items():
        if v is None:
            assert x not in o or not positions, x
        else:
            close(v, o[x], b[x], x)
    return t, m, lse, got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
def test_layouts_on_a_ragged_batch(layout, dtype):
    d, g = make(dtype, *layout, RAGGED, cap=4.0 if layout[2] % 4 else 0.0, front=3, behind=5)
    _, m, lse, got = _check(d, g, dtype)
    # rows of no molecule: zeros and -inf
    for rows in (slice(0, 3), slice(-5, None)):
        assert not m[rows].any() and torch.isneginf(lse[rows]).all()
        for x in ("dq", "dk", "dhp", "dpos_q"):
            assert not got[x][rows].any(), x


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cap", [0.0, 0.5, 20.0, 1e6, 1e30])
@pytest.mark.parametrize("bias,positions", [(False, False), (True, False), (True, True)])
def test_caps_and_biases(cap, bias, positions, dtype):
    d, g = make(dtype, 2, 128, 16, 16, [130, 65, 3], cap=cap, bias=bias, scale=4.0)
    _check(d, g, dtype, positions)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", [[1], [700], [127, 128, 129], [0], [16] * 40, [1] * 70], ids=str)
def test_lengths(lengths, dtype):
    d, g = make(dtype, 2, 128, 16, 16, lengths, cap=8.0)
    _check(d, g, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", [(0, 16, 2, 8), (2, 128, 16, 16), (2, 128, 8, 32), (3, 128, 16, 16), (3, 128, 2, 16)], ids=str)
@pytest.mark.parametrize("queries,keys", [([1], [3000]), ([7, 0, 20], [900, 40, 0]), ([1, 3, 2], [0, 1, 1500]), ([40], [0])], ids=str)
def test_few_queries_against_long_systems(queries, keys, layout, dtype):
    d, g = make(dtype, *layout, keys, queries=queries, cap=5.0, behind=2)
    _check(d, g, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths,queries", [([40, 70, 33], None), ([2000, 400], [2, 5])])
def test_nan_and_inf_stay_in_their_molecule(lengths, queries, dtype):
    d, g = make(dtype, 2, 128, 16, 16, lengths, queries=queries, front=1, behind=4)
    t, (m, lse) = _forward(d, dtype)
    ref = _backward(d, dtype, t, m, lse, g)
    kp = d["k_ptr"] or d["q_ptr"]
    a, b = kp[1], kp[2]                       # the second molecule, and the rows of no molecule
    for n in ("k", "hp", "pos_k" if queries else "pos_q"):
        d[n][a:b:3] = np.nan
        d[n][a + 1:b:3] = np.inf
        d[n][:1], d[n][kp[-1]:] = np.nan, -np.inf
    t2, (m2, lse2) = _forward(d, dtype)
    qa, qb = d["q_ptr"][1], d["q_ptr"][2]
    keep = torch.ones(m.shape[0], dtype=torch.bool)
    keep[qa:qb] = False
    assert torch.equal(m2[keep], m[keep]) and torch.equal(lse2[keep], lse[keep])
    got = _backward(d, dtype, t2, m2, lse2, g)
    kkeep = torch.ones(t["k"].shape[0], dtype=torch.bool)
    kkeep[a:b] = False
    assert torch.equal(got["dq"][keep], ref["dq"][keep])
    assert torch.equal(got["dhp"][kkeep], ref["dhp"][kkeep]) and torch.equal(got["dk"][kkeep], ref["dk"][kkeep])
    assert torch.equal(got["dpos_q"][keep], ref["dpos_q"][keep])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_key_of_minus_infinity_is_masked(dtype):
    """A score of -inf (a key pushed away by an infinite distance) has no weight; a row with no other key
    is an empty row; gradients of such pairs are zeros, not NaN."""
    d, g = make(dtype, 1, 32, 4, 8, [40], queries=[9])
    d["slope"] = np.abs(d["slope"])
    d["pos_k"][5::7] = 3e38                   # its square overflows: distance inf
    t, (m, lse) = _forward(d, dtype)
    keep = np.ones(40, bool)
    keep[5::7] = False
    part = dict(d, k=d["k"][keep], hp=d["hp"][keep], pos_k=d["pos_k"][keep], k_ptr=[0, int(keep.sum())])
    o = molecule_attention(**part)
    close(m, o["m"], bounds(part, o, dtype)["m"], "m")
    d["pos_k"][:] = 3e38
    t, (m, lse) = _forward(d, dtype)
    assert not m.any() and torch.isneginf(lse).all()
    got = _backward(d, dtype, t, m, lse, g, positions=False)
    assert not got["dq"].any() and not got["dk"].any() and not got["dhp"].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_coincident_atoms_and_far_positions(dtype):
    d, g = make(dtype, 2, 64, 8, 16, [50, 20], cap=3.0)
    d["pos_q"][:10] = d["pos_q"][0]           # distance zero: no direction, no force
    d["pos_q"][50:] += 4096.0                 # a molecule far from the origin: differences stay exact enough
    d["pos_q"] = d["pos_q"].astype(np.float32).astype(np.float64)
    _check(d, g, dtype)


def test_gradient_against_differences_of_the_kernel():
    d, g = make("f32", 1, 32, 4, 8, [23, 9], cap=3.0)
    o = molecule_attention(**d, grad=g)
    t, (m, lse) = _forward(d, "f32")
    got = _backward(d, "f32", t, m, lse, g)
    noise = float((np.abs(g) * bounds(d, o, "f32")["m"]).sum())
    r = np.random.default_rng(1)
    h = 2.0 ** -6
    for name, out in (("q", "dq"), ("k", "dk"), ("hp", "dhp"), ("pos_q", "dpos_q"), ("slope", "dslope")):
        v = r.choice([-1.0, 1.0], size=d[name].shape)
        f, fo = [], []
        for s in (1, -1):
            e = dict(d, **{name: (d[name] + s * h * v).astype(np.float32).astype(np.float64)})
            f.append(float((_forward(e, "f32", want_lse=False)[1][0].double().cpu().numpy() * g).sum()))
            fo.append(float((molecule_attention(**e)["m"] * g).sum()))
        diff, diff_o = (f[0] - f[1]) / (2 * h), (fo[0] - fo[1]) / (2 * h)
        along = float((got[out].double().cpu().numpy() * v).sum())
        # the oracle's own difference holds the step's truncation error
        truncation = abs(diff_o - float((o[out] * v).sum()))
        rounding = noise / h + float(bounds(d, o, "f32")[out].sum())
        assert abs(along - diff) <= truncation + rounding, name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_same_result_every_time_and_on_another_stream(dtype):
    d, g = make(dtype, 2, 128, 16, 16, RAGGED + [400], cap=20.0)
    t, (m, lse) = _forward(d, dtype)
    ref = _backward(d, dtype, t, m, lse, g)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        t2, (m2, lse2) = _forward(d, dtype)
        got = _backward(d, dtype, t2, m2, lse2, g)
    s.synchronize()
    assert torch.equal(m, m2) and torch.equal(lse, lse2)
    for x in ref:
        if ref[x] is not None:
            assert torch.equal(ref[x], got[x]), x


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_captured_and_replayed_on_new_molecules(dtype):
    """Lengths are read on the device: one captured graph serves batches of other lengths."""
    egat = _egat()
    d, g = make(dtype, 2, 128, 16, 16, [100, 20, 60], cap=20.0)
    shape = shape_of(d, dtype)
    t = on_gpu(d, dtype)
    G = torch.from_numpy(g).to("cuda", t["q"].dtype)

    def step():
        m, lse = egat.egat_molecule_attention(shape, **t, want_lse=True)
        return (m, lse) + egat.egat_molecule_attention_backward(shape, m=m, lse=lse, grad_m=G, **t)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for lengths in ([100, 20, 60], [1, 178, 0], [60, 60, 60]):
        d["q_ptr"] = ptr_of(lengths)
        t["q_ptr"].copy_(torch.tensor(d["q_ptr"], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        o = molecule_attention(**d, grad=g)
        b = bounds(d, o, dtype)
        for x, v in zip(("m", "lse", "dq", "dk", "dhp", "dpos_q", None, "dslope"), out):
            if x:
                keep = slice(None) if x == "dslope" else slice(0, d["q_ptr"][-1])
                close(v[keep], o[x][keep], b[x][keep], x)


def test_pointers_out_of_range_stay_inside_the_buffers():
    """Entries are clamped to the rows; rows and neighbours of the buffers stay as they were."""
    egat = _egat()
    d, g = make("bf16", 2, 128, 16, 16, [50, 30, 20])
    shape, t = shape_of(d, "bf16"), on_gpu(d, "bf16")
    room = torch.full((3, 100, 9, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    t["q_ptr"].copy_(torch.tensor([-5, 50, 80, 1000], dtype=torch.int32))
    egat.egat_molecule_attention(shape, **t, out=room[1])
    d["q_ptr"] = [0, 50, 80, 100]
    o = molecule_attention(**d)
    close(room[1], o["m"], bounds(d, o, "bf16")["m"], "m")
    for ptr in ([2 ** 31 - 1, -2 ** 31, 50, 3], [100, 60, 20, 0], [7, 7, 7, 7]):
        t["q_ptr"].copy_(torch.tensor(ptr, dtype=torch.int32))
        m, lse = egat.egat_molecule_attention(shape, **t, out=room[1], want_lse=True)
        egat.egat_molecule_attention_backward(shape, m=m, lse=lse, grad_m=m, **t)
    torch.cuda.synchronize()
    assert (room[0] == 7).all() and (room[2] == 7).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_rows_at_all(dtype):
    d, g = make(dtype, 2, 128, 16, 16, [])
    _check(d, g, dtype)
    d, g = make(dtype, 2, 128, 16, 16, [0, 30], queries=[0, 0])
    _, m, lse, got = _check(d, g, dtype)
    assert not got["dk"].any() and not got["dhp"].any() and not got["dpos_k"].any() and not got["dslope"].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_from_the_scalars_norm_to_the_gradients(dtype):
    """Layer norm of the degree-0 rows where they lie, the q/k projection, the attention and its gradients:
    each stage against the oracle on the previous stage's output."""
    egat = _egat()
    r = np.random.default_rng(9)
    lengths, lmax, C, H, dk = [37, 90, 1, 64], 2, 128, 16, 16
    d, g = make(dtype, lmax, C, H, dk, lengths, cap=20.0)
    n = d["hp"].shape[0]
    T = torch.bfloat16 if dtype == "bf16" else torch.float32
    h = torch.from_numpy(r.normal(size=(n, 9, C)) * 2 + 0.5).to("cuda", T)
    gamma, beta = (torch.from_numpy(a).float().cuda() for a in (1 + 0.1 * r.normal(size=C), 0.1 * r.normal(size=C)))
    normed = h.clone()
    egat.egat_layer_norm(h[:, 0, :], gamma, beta, out=normed[:, 0, :])
    o = layer_norm(h[:, 0, :].double().cpu().numpy(), gamma.double().cpu().numpy(), beta.double().cpu().numpy())
    close(normed[:, 0, :], o["y"], (C + 16) * U * (np.abs(o["y"]) + 16) + (2.0 ** -8 if dtype == "bf16" else 0) * np.abs(o["y"]), "y")
    assert torch.equal(normed[:, 1:], h[:, 1:])
    wq, wk = (torch.from_numpy(r.normal(size=(C, H * dk)) / C ** 0.5).float().cuda() for _ in range(2))
    q, k = egat.egat_qk_projection(egat.Shape(n=n, lmax=lmax, C=C, H=H, dk=dk, K=64, dtype=dtype), normed, wq, wk)
    hn, wqn, wkn = (a.double().cpu().numpy() for a in (normed, wq, wk))
    rq, rk = invariant_projection(hn, wqn, wkn, H, dk)
    for got, want, w in ((q, rq, wqn), (k, rk, wkn)):
        terms = (np.abs(hn[:, 0]) @ np.abs(w)).reshape(want.shape)
        # float32 products on the plain path; on bf16 the tensor-core path's 2^-19 of the terms, then one rounding
        close(got, want, (2.0 ** -19 if dtype == "bf16" else (C + 8) * U) * terms + (2.0 ** -8 if dtype == "bf16" else 0) * np.abs(want), "q, k")
    d["q"], d["k"] = q.double().cpu().numpy(), k.double().cpu().numpy()
    _check(d, g, dtype)
