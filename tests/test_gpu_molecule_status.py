"""GPU test of the failure report of the tcgen05 attention within molecules: a wait
that runs out of its polls (nothing faults, nothing hangs) with a copy in flight and
tensor memory held is reported once, and both are given back."""
import pytest
import torch

from oracle.molecule import molecule_attention
from tests.molecule_util import bounds, close, make, on_gpu, shape_of

pytestmark = pytest.mark.gpu


def test_a_wait_that_gives_up_is_reported_and_leaves_the_gpu_usable():
    from equivariant_graph_attention_b200 import egat
    d, _ = make("bf16", 2, 128, 16, 16, [1100])
    shape, t = shape_of(d, "bf16"), on_gpu(d, "bf16")
    egat.egat_take_device_status()
    for polls in (1, 1000):
        egat.egat_selftest_molecule_wait_timeout(polls=polls)
        assert egat.egat_take_device_status() == egat.EGAT_ERR_TIMEOUT
        assert egat.egat_take_device_status() == egat.EGAT_OK
    m, _ = egat.egat_molecule_attention(shape, **t)
    assert egat.egat_take_device_status() == egat.EGAT_OK
    o = molecule_attention(**d)
    close(m, o["m"], bounds(d, o, "bf16")["m"], "m")
