"""GPU tests of calls on a stream of the caller's beside work that is still queued
on the current one: nothing that the call allocates is memory that the current
stream has given back but not finished with, and inputs and results outlive the
caller's references to them as long as a stream uses them."""
import pytest
import torch

from equivariant_graph_attention_b200 import synth
from tests import parity_util
from tests.molecule_util import make, on_gpu, shape_of

pytestmark = pytest.mark.gpu

WAIT = 30_000_000   # clock cycles of a kernel that only waits: about 15 ms


def _egat():
    from equivariant_graph_attention_b200 import egat
    return egat


def owner(t):
    """The stream whose memory a tensor lies in."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not a tensor of the caching allocator")


def _attention(seed=0):
    """A forward and backward pass by (inputs, stream) -> outputs, and its inputs: packed operands and key
    splits take workspaces of several MB."""
    egat = _egat()
    d, g = make("bf16", 2, 128, 16, 16, [1300], cap=8.0, seed=seed)
    shape, t = shape_of(d, "bf16"), on_gpu(d, "bf16")
    t["grad_m"] = torch.from_numpy(g).to("cuda", torch.bfloat16)

    def step(t, stream=None):
        i = {n: x for n, x in t.items() if n != "grad_m"}
        m, lse = egat.egat_molecule_attention(shape, want_lse=True, stream=stream, **i)
        return [m, lse] + [x for x in egat.egat_molecule_attention_backward(shape, m=m, lse=lse, stream=stream, **t) if x is not None]
    return step, t


def _norm(seed=0):
    egat = _egat()
    g = torch.Generator("cuda").manual_seed(seed)
    t = {n: torch.randn(s, generator=g, device="cuda") for n, s in (("x", (20000, 128)), ("w", 128), ("b", 128), ("g", (20000, 128)))}

    def step(t, stream=None):
        y, stats = egat.egat_layer_norm(t["x"], t["w"], t["b"], want_stats=True, stream=stream)
        return [y, stats, *egat.egat_layer_norm_backward(t["x"], t["w"], stats, t["g"], stream=stream)]
    return step, t


def _path(seed=0):
    """The graph, the projection, the fused forward pass and its gradients of a small system."""
    egat = _egat()
    wl = synth.small_cube(80, 9.0, 4.0, 32, 2, 128, 16, 16, "bf16", name="streams80_l2_bf16")
    shape, t = parity_util.shape_of(wl), parity_util.device_inputs(wl, synth.make(wl))
    g = torch.Generator("cuda").manual_seed(seed)
    if seed:
        t["h"], t["q"] = t["h"].flip(0), t["q"].flip(1)
    t.update(g=torch.randn((80, 9, 128), generator=g, device="cuda"), wq=torch.randn((128, 256), generator=g, device="cuda"))

    def step(t, stream=None):
        gr = egat.egat_build_graph(t["pos_q"], wl.cutoff_q, K=wl.K, stream=stream)
        args = (t["pos"], t["q"], t["k"], gr["nbr"], gr["cnt"], t["w1"], t["w2"])
        q, k = egat.egat_qk_projection(shape, t["h"], t["wq"], t["wq"], None, None, stream)   # stream by position
        out = egat.egat_forward(shape, t["h"], *args, order=gr["order"], stream=stream)
        hp = egat.egat_eaas_couple(shape, t["h"], t["pos"], t["w1"], stream=stream)
        return [gr["cnt"], gr["order"], q, k, out, hp, egat.egat_gather_rows(t["h"], gr["cnt"], stream=stream),
                *egat.egat_backward(shape, t["h"], *args, t["g"], order=gr["order"], stream=stream)]
    return step, t


@pytest.fixture(params=[_attention, _norm, _path], ids=["attention", "norm", "path"])
def case(request):
    step, t = request.param()
    ref = [x.clone() for x in step(t)]
    other = request.param(seed=1)[1]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    return step, t, ref, other


def _equal(got, ref):
    torch.cuda.synchronize()
    return all(torch.equal(a, b) for a, b in zip(got, ref)) and len(got) == len(ref)


def test_results_are_the_streams_memory(case):
    step, t, ref, _ = case
    s = torch.cuda.Stream()
    got = step(t, s)
    assert all(owner(x) == s.cuda_stream for x in got)
    assert _equal(got, ref)


def test_blocks_with_pending_writes_are_not_taken(case):
    step, t, ref, _ = case
    s = torch.cuda.Stream()
    for _ in range(3):
        room = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (1 << 16, 1 << 19, 1 << 22, 1 << 25, 1 << 26)]
        torch.cuda._sleep(WAIT)
        for x in room:
            x.fill_(0xff)            # NaN, queued behind the wait
        del room, x                  # back to the current stream's pool
        got = step(t, s)
        s.synchronize()
        assert _equal(got, ref)


def test_inputs_may_be_given_back_after_the_call(case):
    step, t, ref, _ = case
    s = torch.cuda.Stream()
    for _ in range(3):
        mine = {n: x.clone() if isinstance(x, torch.Tensor) else x for n, x in t.items()}
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(WAIT)
        sizes = [x.numel() * x.element_size() for x in mine.values() if isinstance(x, torch.Tensor)]
        got = step(mine, s)
        del mine
        for n in sizes:              # the same sizes again, on the current stream
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xff)
        assert _equal(got, ref)


def test_results_may_be_given_back_while_the_current_stream_reads_them(case):
    step, t, ref, other = case
    s = torch.cuda.Stream()
    got = step(t, s)
    s.synchronize()
    torch.cuda._sleep(WAIT)
    copies = [x.clone() for x in got]
    del got
    again = step(other, s)           # would otherwise take the blocks just given back to s
    assert _equal(copies, ref)
    assert _equal(again, step(other))


def test_streams_of_another_device_are_refused():
    step, t = _norm()
    class Elsewhere:
        device, cuda_stream = torch.device("cuda", 1), 0
    with pytest.raises(ValueError):
        step(t, Elsewhere())


def test_captured_on_the_stream_that_is_passed(case):
    step, t, ref, _ = case
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    step(t, s)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        got = step(t, s)
    for _ in range(2):
        for x in got:
            x.zero_()
        graph.replay()
        assert _equal(got, ref)
