"""The workspace of products that split tiles stream-K and were given none.  On the CPU the library and torch's
streams are stand-ins, and what is checked is where and when each buffer is made and kept; on the GPU the results."""
import ctypes

import pytest
import torch

from cases import dev, nvfp4_operands, scalar


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture()
def fake(monkeypatch):
    """The binding over CPU tensors; records each launch's workspace address and each buffer's (stream, size, zeroed)."""
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_block_scaled_bf16_gb300 as nv
    real = nv._lib
    now = [FakeStream(0)]
    nv.log = log = type("Log", (), dict(launched=[], capturing=set(), need=512, now=now))()

    class Lib:
        nvfp4_sf_bytes = real.nvfp4_sf_bytes

        @staticmethod
        def nvfp4_gemm_workspace_size(m, n, k, size):
            ctypes.cast(size, ctypes.POINTER(ctypes.c_size_t))[0] = log.need
            return 0

        @staticmethod
        def nvfp4_gemm(*args):
            log.launched.append((args[12], args[9]))
            return 0

        @staticmethod
        def nvfp4_gated_gemm(*args):
            log.launched.append((args[13], args[10]))
            return 0

    class Stream(FakeStream):
        """torch.cuda.stream"""
        def __init__(self, stream):
            self.to = stream

        def __enter__(self):
            now.append(self.to or now[-1])

        def __exit__(self, *exc):
            now.pop()

    monkeypatch.setattr(nv, "_lib", Lib())
    monkeypatch.setattr(nv, "_check_device", lambda t, name: None)
    monkeypatch.setattr(nv, "_current_device", lambda: 0)
    monkeypatch.setattr(nv, "_raw_stream", lambda device: now[-1].cuda_stream)
    monkeypatch.setattr(nv, "_ws_cache", {})
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", FakeStream)
    monkeypatch.setattr(torch.cuda, "stream", Stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[-1])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now[-1].cuda_stream in log.capturing)
    made = []

    def record(real_fn):
        def f(*args, **kw):
            t = real_fn(*args, **kw)
            if t.dtype == torch.uint8:
                made.append((now[-1].cuda_stream, t))
            return t
        return f

    for name in ("zeros", "empty"):
        monkeypatch.setattr(torch, name, record(getattr(torch, name)))
    log.made = made
    return nv


def gemm(nv, gated, stream=None):
    """One call; the stream it was launched on and the buffer it was given, as (stream made under, tensor)."""
    m, n, k = 8, 64, 64
    u8 = lambda *s: torch.full(s, 0, dtype=torch.uint8)  # noqa: E731
    args = (u8(m, k // 2), u8(nv.sf_bytes(m, k)), u8(n, k // 2), u8(nv.sf_bytes(n, k)), torch.full((2,), 1.0))
    (nv.nvfp4_gated_gemm if gated else nv.nvfp4_gemm)(*args, stream=stream)
    launched, address = nv.log.launched[-1]
    made = [(s, t) for s, t in nv.log.made if t.data_ptr() == address]
    assert len(made) == 1 and made[0][1].numel() >= nv.log.need
    return launched, made[0][0], made[0][1]


@pytest.mark.parametrize("gated", [False, True])
def test_a_captured_call_has_a_buffer_of_its_own(fake, gated):
    """Made under the capture, its counters zeroed there, and neither kept for later calls nor taken from before."""
    stream, made, eager = gemm(fake, gated)
    assert stream == made == 0 and not eager.any()
    graph = FakeStream(9)
    fake.log.capturing.add(9)
    seen = []
    for by_argument in (False, True, True):
        if by_argument:
            stream, made, ws = gemm(fake, gated, graph)
        else:
            with torch.cuda.stream(graph):
                stream, made, ws = gemm(fake, gated)
        assert stream == made == 9 and not ws[:4096].any()
        seen.append(ws)
    addresses = {t.data_ptr() for t in seen} | {eager.data_ptr()}
    assert len(addresses) == 4
    assert gemm(fake, gated)[2] is eager


@pytest.mark.parametrize("gated", [False, True])
def test_each_stream_has_a_buffer_made_on_it(fake, gated):
    """Zeroed on the launch stream whichever is current, kept for that stream alone, replaced when it is too small."""
    side = FakeStream(5)
    kept = {}
    for by_argument in (True, False):
        if by_argument:
            stream, made, ws = gemm(fake, gated, side)
        else:
            with torch.cuda.stream(side):
                stream, made, ws = gemm(fake, gated)
        assert stream == made == 5 and not ws.any()
        assert kept.setdefault(5, ws) is ws
    stream, made, ws = gemm(fake, gated, 6)                       # a raw handle
    assert stream == made == 6 and not ws.any() and ws is not kept[5]
    stream, made, ws = gemm(fake, gated)
    assert stream == made == 0 and not ws.any() and ws is not kept[5]
    fake.log.need = 8192
    stream, made, larger = gemm(fake, gated, side)
    assert stream == made == 5 and larger is not kept[5] and not larger.any()
    fake.log.need = 512
    assert gemm(fake, gated, side)[2] is larger and gemm(fake, gated)[2] is ws


@pytest.fixture(scope="module")
def nv():
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_block_scaled_bf16_gb300 as m
    return m


SMALL, LARGE = (300, 1024, 16384), (1792, 640, 16384)      # stream-K; the second has counters for more tiles


def operands(shape, seed=0):
    m, n, k = shape
    ops = nvfp4_operands(m, n, k, seed)
    return dev(ops["qa"]), dev(ops["sfa"]), dev(ops["qb"]), dev(ops["sfb"]), scalar(ops["alpha"])


def explicit(nv, shape, args):
    d = nv.nvfp4_gemm(*args, workspace=nv.gemm_workspace(nv.gemm_workspace_size(*shape)))
    torch.cuda.synchronize()
    return d


@pytest.mark.gpu
@pytest.mark.parametrize("warm", [False, True])
def test_a_graph_outlives_the_shared_buffer(nv, warm):
    """A captured call, then the shared buffer grows and what it had is handed to others, then replays."""
    assert nv.nvfp4_gemm_plan(*SMALL)["sk_tiles"] and nv.gemm_workspace_size(*LARGE) > nv.gemm_workspace_size(*SMALL) > 0
    a, b = operands(SMALL), operands(LARGE)
    want, want_large = explicit(nv, SMALL, a), explicit(nv, LARGE, b)
    nv._ws_cache.clear()
    d = torch.empty_like(want)
    if warm:
        nv.nvfp4_gemm(*a, d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.nvfp4_gemm(*a, d)
        e = nv.nvfp4_gemm(*a)
    assert torch.equal(nv.nvfp4_gemm(*b), want_large)
    torch.cuda.synchronize()
    junk = [torch.full((nv.gemm_workspace_size(*LARGE),), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(4)]
    for _ in range(3):
        d.zero_()
        e.zero_()
        graph.replay()
        assert torch.equal(d, want) and torch.equal(e, want)
        assert torch.equal(nv.nvfp4_gemm(*b), want_large) and torch.equal(nv.nvfp4_gemm(*a), want)
    assert all(bool((t == 0xFF).all()) for t in junk)
    nv.check_status()


@pytest.mark.gpu
def test_first_calls_on_side_streams(nv):
    """The first calls without a workspace, on streams that run beside a busy current one and beside each other."""
    a, b = operands(SMALL), operands(SMALL, 3)
    wants = explicit(nv, SMALL, a), explicit(nv, SMALL, b)
    nv._ws_cache.clear()
    x = torch.randn(4096, 4096, device="cuda")
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [[torch.empty_like(w) for _ in range(8)] for w in wants]
    torch.cuda.synchronize()
    for _ in range(20):
        x = x @ x * 0.01
    for i in range(8):
        for s, args, out in zip(streams, (a, b), outs):
            nv.nvfp4_gemm(*args, out[i], stream=s)
    torch.cuda.synchronize()
    nv.check_status()
    for want, out in zip(wants, outs):
        assert all(torch.equal(d, want) for d in out)
    assert len(nv._ws_cache) == 2 and not any(bool(ws[:256].any()) for ws in nv._ws_cache.values())


@pytest.mark.gpu
def test_captured_calls_launched_with_pdl(nv):
    """The fill of a graph's buffer lies between two kernels that may otherwise overlap."""
    a = operands(SMALL)
    want = explicit(nv, SMALL, a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [nv.nvfp4_gemm(*a, flags=nv.FLAG_PDL) for _ in range(3)]
    for _ in range(3):
        for d in outs:
            d.zero_()
        graph.replay()
        assert all(torch.equal(d, want) for d in outs)
    nv.check_status()
