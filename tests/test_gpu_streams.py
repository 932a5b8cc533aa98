"""The helpers of the calls around the block attention with a stream given: what they allocate is not
memory that the current stream, or the given one, may still be using."""
import gc
import threading

import pytest
import torch

from piecewise_attention_diffusion_b200 import bsattn as b
from tests.test_gpu_cross import DEV, _randn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu(cuda_ok):
    yield


def _calls():
    """(name, call of a stream, sizes in bytes of what it allocates), each with a split sum or with
    split keys where there is a workspace."""
    x, w = _randn(1, 4, 8192), _randn(1, 256, 8192, seed=1, scale=8192 ** -0.5)[0]
    q, k, v = _randn(1, 2, 1, 64), _randn(1, 2, 30000, 64, seed=1), _randn(1, 2, 30000, 64, seed=2)
    r, pos = _randn(1, 8, 4096, 64), torch.arange(4096.0, device=DEV)[:, None].contiguous()
    lw, cw = b.bsa_linear_workspace_bytes(1, 4, 8192, 256), b.bsa_cross_workspace_bytes(1, 2, 2, 1, 30000, 64)
    assert lw > 0 and cw > 0
    y = torch.empty(1, 4, 256, dtype=x.dtype, device=DEV)
    return [("rotary", lambda s: [b.rotary(r, pos, (64,), stream=s)], [r.numel() * 2]),
            ("linear", lambda s: [b.linear(x, w, stream=s)], [lw, 4 * 256 * 2]),
            ("linear out", lambda s: [b.linear(x, w, out=y, stream=s)], [lw]),
            ("cross", lambda s: list(b.cross_forward(q, k, v, want_lse=True, stream=s)), [cw, 256, 8])]


@pytest.mark.parametrize("which", range(4))
def test_memory_that_the_current_stream_still_writes(which):
    """Blocks of the sizes that the helper allocates are freed while the current stream's writes to
    them are still queued, behind some milliseconds of other work."""
    name, call, sizes = _calls()[which]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for cycles in (20_000, 2_000_000, 10_000_000):   # the writes come during the call, and after it
        gc.collect()
        torch.cuda.empty_cache()
        torch.cuda._sleep(cycles)
        junk = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(3)]
        for _ in range(20):
            for t in junk:
                t.fill_(255)    # NaN in every type
        freed = {t.data_ptr() for t in junk}
        del junk, t
        got = call(s)
        if name != "linear out":
            assert all(t.data_ptr() not in freed for t in got)
        s.synchronize()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want)), name


@pytest.mark.parametrize("which", [0, 1, 3])
def test_outputs_that_the_current_stream_still_reads(which):
    """An output freed while the current stream has yet to read it is not given to the next call on
    the other stream."""
    name, call, _ = _calls()[which]
    want = [t.clone() for t in call(None)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        got = call(s)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda._sleep(5_000_000)
        copies = [t.clone() for t in got]
        read = torch.cuda.Event()
        read.record()
        ptrs = {t.data_ptr() for t in got}
        del got
        more = [call(s) for _ in range(4)]
        assert read.query() or all(t.data_ptr() not in ptrs for ts in more for t in ts)
        torch.cuda.synchronize()
        assert all(torch.equal(c, w) for ts in more + [copies] for c, w in zip(ts, want)), name


def test_a_given_stream_inside_a_captured_graph():
    """A stream that forks off a captured one and joins it again: outputs and workspaces live in the
    graph's memory."""
    calls = [c for _, c, _ in _calls() if _ != "linear out"]
    want = [[t.clone() for t in c(None)] for c in calls]
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cur = torch.cuda.current_stream()
        s.wait_stream(cur)
        got = [c(s) for c in calls]
        cur.wait_stream(s)
    for ts in got:
        for t in ts:
            t.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for gs, ws in zip(got, want) for g, w in zip(gs, ws))


def test_a_stream_of_another_device_is_refused():
    class Other:    # a stream of a device that is not the tensors'
        device = torch.device("cuda", 1)
        cuda_stream = 0
    x = _randn(1, 2, 8, 64)
    with pytest.raises(ValueError, match="stream"):
        b.rotary(x, torch.zeros(8, 1, device=DEV), (64,), out=torch.empty_like(x), stream=Other())


def test_calls_of_several_host_threads():
    """Threads that call at once, each on a stream of its own."""
    calls = [c for n, c, _ in _calls() if n != "linear out"]
    want = [[t.clone() for t in c(None)] for c in calls]
    torch.cuda.synchronize()
    wrong = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                for i, c in enumerate(calls):
                    got = c(None)
                    s.synchronize()
                    if not all(torch.equal(g, w) for g, w in zip(got, want[i])):
                        wrong.append(i)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_an_output_of_the_caller_that_is_let_go():
    """Memory of a caller's output is not given out while the given stream has yet to write it."""
    x, w = _randn(1, 4, 8192), _randn(1, 256, 8192, seed=1, scale=8192 ** -0.5)[0]
    q, k = _randn(1, 2, 200, 64), _randn(1, 2, 77, 64, seed=1)
    pos = torch.zeros(200, 1, device=DEV)
    s = torch.cuda.Stream()
    for call, shape in ((lambda o: b.linear(x, w, out=o, stream=s), (1, 4, 256)),
                        (lambda o: b.cross_forward(q, k, k, out=o, stream=s), q.shape),
                        (lambda o: b.rotary(q, pos, (64,), out=o, stream=s), q.shape)):
        out = torch.empty(shape, dtype=q.dtype, device=DEV)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
        call(out)
        done = torch.cuda.Event()
        done.record(s)
        ptr = out.data_ptr()
        del out
        fresh = [torch.zeros(shape, dtype=q.dtype, device=DEV) for _ in range(4)]
        assert done.query() or all(t.data_ptr() != ptr for t in fresh)
        torch.cuda.synchronize()
        assert not any(t.any() for t in fresh)
