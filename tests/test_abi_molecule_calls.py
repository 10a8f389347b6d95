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
