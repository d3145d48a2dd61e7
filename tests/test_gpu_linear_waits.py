"""Linear products whose waits run out on the GPU: reported, ended with nothing in flight, and followed by right ones.
Every wait of them has a limit; the products' results are not looked at."""
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

from trainable_block_sparse_cube_b200 import build as vsa_build
from trainable_block_sparse_cube_b200 import vsa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    vsa_build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    vsa.load()


@pytest.fixture(autouse=True)
def _limits():
    yield
    assert vsa.load().vsa_linear_set_limits(1_000_000_000, 0) == 0
    vsa.linear_check()


def _randn(seed, *shape, std=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)


# rows, K, F: fewer steps than stages of the ring; more; several tiles a pair; one CTA of the pair without rows
SHAPES = [(300, 128, 256), (300, 512, 256), (2000, 4096, 1024), (9000, 1024, 1536), (40, 4096, 512)]


@pytest.mark.parametrize("M,K,F", SHAPES)
def test_loads_that_come_after_the_limit(M, K, F):
    """One CTA of each pair asks for its operands when the MMAs have been given up; the product ends after them."""
    x, w, dy = _randn(1, 1, M, K), _randn(2, F, K), _randn(3, 1, M, F)
    L = vsa.load()
    ref = (vsa.linear(x, w), *vsa.linear_backward(x, w, dy)[:2])
    vsa.linear_check()
    calls = (lambda: vsa.linear(x, w), lambda: vsa.linear_backward(x, w, dy, want=(True, False)),
             lambda: vsa.linear_backward(x, w, dy, want=(False, True)))
    for call in calls:
        assert L.vsa_linear_set_limits(200_000, 2) == 0
        call()
        assert L.vsa_linear_set_limits(1_000_000_000, 0) == 0
        got = (vsa.linear(x, w), *vsa.linear_backward(x, w, dy)[:2])          # right behind it, on the same SMs
        with pytest.raises(vsa.VSAError, match="TIMEOUT"):
            vsa.linear_check()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("M,K,F", SHAPES)
def test_waits_of_next_to_no_time(M, K, F):
    """With a limit of a nanosecond any warp may give up anywhere, the epilogue's while MMAs run among them."""
    x, w, dy = _randn(1, 1, M, K), _randn(2, F, K), _randn(3, 1, M, F)
    L = vsa.load()
    ref = (vsa.linear(x, w), *vsa.linear_backward(x, w, dy)[:2])
    vsa.linear_check()
    for _ in range(5):
        assert L.vsa_linear_set_limits(1, 0) == 0
        vsa.linear(x, w)
        vsa.linear_backward(x, w, dy)
        assert L.vsa_linear_set_limits(1_000_000_000, 0) == 0
        got = (vsa.linear(x, w), *vsa.linear_backward(x, w, dy)[:2])
        try:
            vsa.linear_check()
        except vsa.VSAError as e:
            assert "TIMEOUT" in str(e)
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


def _stalled(fn, limit=200_000):
    """fn() with operands left unloaded, so that its waits run out."""
    L = vsa.load()
    assert L.vsa_linear_set_limits(limit, 1) == 0
    try:
        return fn()
    finally:
        assert L.vsa_linear_set_limits(1_000_000_000, 0) == 0


def _told(stream=None):
    with torch.cuda.stream(stream):
        try:
            vsa.linear_check()
        except vsa.VSAError as e:
            assert e.code == 6
            return True
    return False


def test_a_failure_is_told_to_the_stream_that_it_happened_on():
    x, w = _randn(1, 1, 300, 512), _randn(2, 256, 512)
    ref = vsa.linear(x, w)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(b):
        vsa.linear(x, w)
    with torch.cuda.stream(a):
        _stalled(lambda: vsa.linear(x, w))
    assert not _told(b) and not _told()                 # looks of others, which take nothing away
    assert _told(a) and not _told(a)
    for st in (a, b):                                   # both at once
        with torch.cuda.stream(st):
            _stalled(lambda: vsa.linear(x, w))
    assert _told(b) and _told(a) and not _told(b) and not _told(a) and not _told()
    assert torch.equal(vsa.linear(x, w), ref)


def test_a_failure_inside_a_graph_is_told_to_every_stream():
    x, w = _randn(1, 1, 300, 512), _randn(2, 256, 512)
    ref = vsa.linear(x, w)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    bad, good = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    assert not _told(a) and not _told(b)
    with torch.cuda.graph(good):
        out = vsa.linear(x, w)
    with torch.cuda.graph(bad):
        _stalled(lambda: vsa.linear(x, w))
    torch.cuda.synchronize()
    for _ in range(2):
        with torch.cuda.stream(a):
            bad.replay()
        torch.cuda.synchronize()
        assert _told(a) and _told(b) and _told()
        assert not _told(a) and not _told(b) and not _told()
    good.replay()
    assert not _told() and torch.equal(out, ref)


def test_a_check_during_a_capture_is_refused_and_spares_it():
    x, w = _randn(1, 1, 300, 512), _randn(2, 256, 512)
    ref = vsa.linear(x, w)
    vsa.linear_check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(vsa.VSAError) as e:
            vsa.linear_check()
        out = vsa.linear(x, w)
    assert e.value.code == 5
    g.replay()
    assert not _told() and torch.equal(out, ref)


def test_the_hook_is_the_calling_threads():
    x, w = _randn(1, 1, 300, 512), _randn(2, 256, 512)
    ref = vsa.linear(x, w)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()

    def other():
        with torch.cuda.stream(st):
            y = vsa.linear(x, w)
            vsa.linear_check()
            return y

    with ThreadPoolExecutor(1) as pool:
        y = _stalled(lambda: pool.submit(other).result())
    torch.cuda.synchronize()
    assert torch.equal(y, ref) and not _told()


def test_many_streams():
    """Each of the streams of torch's pools is told of its own failure, once."""
    x, w = _randn(1, 1, 300, 512), _randn(2, 256, 512)
    streams = list({st.cuda_stream: st for st in (torch.cuda.Stream(priority=p) for p in (0, -1) for _ in range(32))}.values())
    for st in streams:
        _told(st)                                       # what came before, graphs of other tests among it
    for st in streams[::2]:
        with torch.cuda.stream(st):
            _stalled(lambda: vsa.linear(x, w), limit=1)
    assert [_told(st) for st in streams] == [i % 2 == 0 for i in range(len(streams))]
    assert not any(_told(st) for st in streams) and not _told()


@pytest.mark.parametrize("mode", ["global", "thread_local"])
def test_products_of_one_thread_beside_a_capture_of_another(mode):
    """The look at a stream's number and state spares the other thread's capture."""
    x, w = _randn(1, 1, 300, 64), _randn(2, 256, 64)                       # no workspace: nothing is allocated meanwhile
    ref = vsa.linear(x, w)
    out, st, w2 = torch.empty_like(ref), torch.cuda.Stream(), _randn(3, 64, 256)
    torch.cuda.synchronize()

    def other():
        with torch.cuda.stream(st):
            for _ in range(3):
                vsa.linear(x, w, out=out)

    with ThreadPoolExecutor(1) as pool:
        pool.submit(other).result()
        torch.cuda.synchronize()
        out.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, capture_error_mode=mode):
            y = vsa.linear(x, w)
            pool.submit(other).result()
            y = vsa.linear(y, w2)
    torch.cuda.synchronize()
    assert torch.equal(out, ref)
    g.replay()
    assert torch.equal(y, vsa.linear(ref, w2)) and not _told() and not _told(st)
