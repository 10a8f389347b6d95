"""Host-side checks of the attention within molecules and the layer norm: every
refusal happens before a launch, so no call here reaches a device."""
import ctypes

import pytest
import torch

from equivariant_graph_attention_b200 import egat

OK, ODD16, ODD4 = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008), ctypes.c_void_p(0x10002)
BASE = dict(nq=10, nk=10, n_mol=3, lmax=2, C=128, H=16, dk=16, dtype="bf16", cap=0.0)


@pytest.fixture(scope="module")
def lib():
    from equivariant_graph_attention_b200.build import build
    build()
    return egat.load_library()


def _shape(**kw):
    return egat.MoleculeShape(**dict(BASE, **kw)).c()


# s, q, k, hp, q_ptr, k_ptr, pos_q, pos_k, slope, ws, ws_bytes, m, lse, stream
FWD = [OK, OK, OK, OK, OK, OK, OK, OK, OK, 1 << 40, OK, OK, None]
# ... slope, m, lse, grad, ws, ws_bytes, dq, dk, dhp, dpos_q, dpos_k, dslope, stream
BWD = [OK, OK, OK, OK, OK, OK, OK, OK, OK, OK, OK, OK, 1 << 40, OK, OK, OK, OK, OK, OK, None]


@pytest.mark.parametrize("kw,code", [
    (dict(nq=-1), "ARG"), (dict(nk=-1), "ARG"), (dict(n_mol=-1), "ARG"), (dict(cap=-1.0), "ARG"),
    (dict(cap=float("nan")), "ARG"), (dict(cap=1e-31), "ARG"), (dict(cap=1e31), "ARG"), (dict(cap=float("inf")), "ARG"), (dict(lmax=4), "UNSUPPORTED"),
    (dict(lmax=-1), "UNSUPPORTED"), (dict(C=96), "UNSUPPORTED"), (dict(C=0), "UNSUPPORTED"), (dict(H=3), "UNSUPPORTED"),
    (dict(H=0), "UNSUPPORTED"), (dict(H=32), "UNSUPPORTED"), (dict(dk=12), "UNSUPPORTED"),
    (dict(nq=(1 << 30) + 1), "UNSUPPORTED"), (dict(n_mol=(1 << 28) + 1), "UNSUPPORTED")])
def test_shapes_refused(lib, kw, code):
    cs, out = _shape(**kw), ctypes.c_size_t(0)
    want = getattr(egat, "EGAT_ERR_" + code)
    assert lib.egat_molecule_attention(ctypes.byref(cs), *FWD) == want
    assert lib.egat_molecule_attention_backward(ctypes.byref(cs), *BWD) == want
    assert lib.egat_molecule_attention_workspace_bytes(ctypes.byref(cs), ctypes.byref(out)) == want
    assert lib.egat_molecule_attention_backward_workspace_bytes(ctypes.byref(cs), ctypes.byref(out)) == want


def test_other_types_refused(lib):
    cs = egat.egat_mol_shape(10, 10, 3, 2, 128, 16, 16, 7, 0.0)
    assert lib.egat_molecule_attention(ctypes.byref(cs), *FWD) == egat.EGAT_ERR_ARG
    assert lib.egat_molecule_attention(None, *FWD) == egat.EGAT_ERR_ARG


def _call(f, cs, args, **change):
    a = list(args)
    for k, v in change.items():
        a[int(k[1:])] = v
    return f(ctypes.byref(cs), *a)


def test_pointers_refused(lib):
    cs = _shape()
    f, b = lib.egat_molecule_attention, lib.egat_molecule_attention_backward
    for slot in (0, 1, 2, 10):                          # q, k, hp, m: needed, 16-byte aligned
        for p in (None, ODD16):
            assert _call(f, cs, FWD, **{f"a{slot}": p}) == egat.EGAT_ERR_ARG, slot
    for slot in (3, 5, 6):                              # q_ptr; positions with a slope
        assert _call(f, cs, FWD, **{f"a{slot}": None}) == egat.EGAT_ERR_ARG, slot
    for slot in (3, 4, 5, 6, 7, 11):
        assert _call(f, cs, FWD, **{f"a{slot}": ODD4}) == egat.EGAT_ERR_ARG, slot
    # the self form: one set of positions, as many keys as queries
    assert _call(f, cs, FWD, a4=None) == egat.EGAT_ERR_ARG
    assert _call(f, _shape(nk=11), FWD, a4=None, a6=None) == egat.EGAT_ERR_ARG
    for slot in (0, 1, 2, 8, 9, 10, 13, 14, 15):        # m, lse, grad, dq, dk, dhp too
        assert _call(b, cs, BWD, **{f"a{slot}": None}) == egat.EGAT_ERR_ARG, slot
    for slot in (0, 1, 2, 8, 10, 11, 13, 14, 15):
        assert _call(b, cs, BWD, **{f"a{slot}": ODD16}) == egat.EGAT_ERR_ARG, slot
    for slot in (9, 16, 17, 18):
        assert _call(b, cs, BWD, **{f"a{slot}": ODD4}) == egat.EGAT_ERR_ARG, slot
    # position gradients without a slope, key positions' in the self form
    assert _call(b, cs, BWD, a7=None) == egat.EGAT_ERR_ARG
    assert _call(b, cs, BWD, a4=None, a6=None) == egat.EGAT_ERR_ARG
    assert _call(b, cs, BWD, a12=16) == egat.EGAT_ERR_WORKSPACE
    big = _shape(nq=1, nk=100000, n_mol=1)              # a key split needs its workspace
    assert _call(f, big, FWD, a8=None) == egat.EGAT_ERR_ARG
    assert _call(f, big, FWD, a9=16) == egat.EGAT_ERR_WORKSPACE


def test_no_queries_is_a_no_op(lib):
    cs = _shape(nq=0)
    assert lib.egat_molecule_attention(ctypes.byref(cs), None, OK, OK, OK, OK, None, OK, OK, None, 0, None, None, None) == egat.EGAT_OK


def test_workspaces(lib):
    a256 = lambda x: (x + 255) // 256 * 256
    q = egat.egat_molecule_attention_workspace_bytes
    # enough row tiles to fill the GPU: no key split, no workspace
    assert q(egat.MoleculeShape(**dict(BASE, nq=200000, nk=200000, n_mol=4000))) == 0
    # a split holds dv + 2 floats a row and head, for 64 splits at most
    one = q(egat.MoleculeShape(**dict(BASE, nq=1, nk=32768, n_mol=1)))
    assert 0 < one <= 64 * (16 * 74 * 4) + 1024
    # sizes past 32 bits
    assert egat.egat_molecule_attention_backward_workspace_bytes(
        egat.MoleculeShape(**dict(BASE, nq=1 << 27, nk=1 << 27, n_mol=1000))) > 1 << 33


def test_layer_norm_refusals(lib):
    f = lib.egat_layer_norm
    # x, ldx, n, width, dtype, weight, bias, eps, y, ldy, stats, stream
    ok = [OK, 128, 10, 128, 1, OK, OK, 1e-5, OK, 128, OK, None]
    E = egat.EGAT_ERR_ARG
    for slot, v in ((0, None), (8, None), (0, ctypes.c_void_p(0x10001)), (8, ctypes.c_void_p(0x10001)), (1, 127), (9, 100),
                    (2, -1), (3, 0), (4, 7), (5, ODD4), (6, ODD4), (10, ODD4), (7, -1.0), (7, float("nan")), (7, float("inf"))):
        a = list(ok)
        a[slot] = v
        assert f(*a) == E, (slot, v)
    assert f(OK, 20000, 10, 16385, 1, OK, OK, 1e-5, OK, 20000, OK, None) == egat.EGAT_ERR_UNSUPPORTED
    assert f(None, 128, 0, 128, 1, None, None, 1e-5, None, 128, None, None) == egat.EGAT_OK
    b = lib.egat_layer_norm_backward
    # x, ldx, n, width, dtype, weight, stats, grad, ldg, ws, ws_bytes, dx, lddx, dweight, dbias, stream
    ok = [OK, 128, 10, 128, 1, OK, OK, OK, 128, OK, 1 << 30, OK, 128, OK, OK, None]
    for slot, v in ((0, None), (6, None), (7, None), (9, None), (9, ODD16), (0, ctypes.c_void_p(0x10001)), (7, ctypes.c_void_p(0x10001)),
                    (11, ctypes.c_void_p(0x10001)), (1, 127), (8, 127), (12, 127), (2, -1), (3, 0), (4, 7), (5, ODD4),
                    (6, ODD4), (13, ODD4), (14, ODD4)):
        a = list(ok)
        a[slot] = v
        assert b(*a) == E, (slot, v)
    a = list(ok)
    a[10] = 64
    assert b(*a) == egat.EGAT_ERR_WORKSPACE
    a = list(ok)
    a[11] = a[13] = a[14] = None
    assert b(*a) == egat.EGAT_OK                       # nothing asked for
    with pytest.raises(egat.EgatError):
        egat.egat_layer_norm_backward_workspace_bytes(10, 0)


def test_the_binding_refuses_tensors_off_the_gpu():
    x = torch.zeros(4, 16)
    with pytest.raises((ValueError, RuntimeError)):
        egat.egat_layer_norm(x)
    with pytest.raises(ValueError):
        egat.egat_layer_norm(x.double())
    with pytest.raises((ValueError, RuntimeError)):
        egat.egat_molecule_attention(egat.MoleculeShape(**BASE), x, x, x, x)
