"""Host-side checks of the attention within molecules and the layer norm, beside
tests/test_abi_molecule.py: every refusal happens before a launch, so no call here
reaches a device."""
import ctypes

import pytest

from equivariant_graph_attention_b200 import egat

OK = ctypes.c_void_p(0x10000)


@pytest.fixture(scope="module")
def lib():
    from equivariant_graph_attention_b200.build import build
    build()
    return egat.load_library()


@pytest.mark.parametrize("polls", [0, -1, (1 << 20) + 1])
def test_selftest_polls_refused(lib, polls):
    assert lib.egat_selftest_molecule_wait_timeout(polls, None) == egat.EGAT_ERR_ARG
    with pytest.raises(egat.EgatError):
        egat_call(polls)


def egat_call(polls):
    class Stream:
        cuda_stream = None
    egat.egat_selftest_molecule_wait_timeout(polls, Stream())


def test_in_place_norm_of_other_rows_refused(lib):
    """Another stride over the same start would write rows that are still to be read."""
    f, b = lib.egat_layer_norm, lib.egat_layer_norm_backward
    OTHER, WS = ctypes.c_void_p(0x20000), ctypes.c_void_p(0x40000)
    # x, ldx, n, width, dtype, weight, bias, eps, y, ldy, stats, stream
    assert f(OK, 256, 10, 128, 1, None, None, 1e-5, OK, 128, None, None) == egat.EGAT_ERR_ARG
    assert f(OK, 128, 10, 128, 1, None, None, 1e-5, OK, 256, None, None) == egat.EGAT_ERR_ARG
    # x, ldx, n, width, dtype, weight, stats, grad, ldg, ws, ws_bytes, dx, lddx, dweight, dbias, stream
    for x, grad in ((OTHER, OK), (OK, OTHER)):
        for ld, lddx in ((256, 128), (128, 256)):
            assert b(x, ld, 10, 128, 1, None, WS, grad, ld, WS, 1 << 30, OK, lddx, None, None, None) == egat.EGAT_ERR_ARG


BASE = dict(nq=1024, nk=1024, n_mol=2, lmax=2, C=128, H=16, dk=16, dtype="bf16", cap=0.0)


@pytest.mark.parametrize("kw,takes", [
    ({}, True), (dict(dtype="f32"), False), (dict(nk=1023), False), (dict(nq=1023), False), (dict(n_mol=3), False),
    (dict(nk=1 << 20), True), (dict(n_mol=1), True), (dict(n_mol=1, nq=640, nk=640), True),
    (dict(n_mol=1, nq=639), False), (dict(n_mol=1, H=8, C=64, nq=1408, nk=1408), True),
    (dict(n_mol=1, H=8, C=64, nq=1407, nk=1407), False), (dict(lmax=3), True), (dict(H=8, nq=2048, nk=2048), False),
    (dict(H=8, lmax=1, nq=2048, nk=2048), True), (dict(n_mol=0), False)], ids=str)
def test_which_shapes_take_the_tcgen05_kernels(lib, kw, takes):
    """bf16, at most 128 value columns a head, 512 rows a molecule on average on both sides, (nq / 128 + n_mol) H of 96
    at least: by the workspace, which is that of the packed operands there and nowhere else."""
    from tests.molecule_tight import packed_bytes
    s = egat.MoleculeShape(**dict(BASE, **kw))
    assert (egat.egat_molecule_attention_workspace_bytes(s) == packed_bytes(s)) is takes
