"""session.PagedCache on streams: the current one, one that is given, one that
is being captured."""
import threading

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU-only hosts
    pytest.skip("needs a CUDA device", allow_module_level=True)

import masked_block_diffusion_denoise_b200 as dlm
from masked_block_diffusion_denoise_b200.session import PagedCache

HEADS, KV, DIM, B, NEW = 8, 2, 128, 3, 96
SLEEP = 1 << 27          # cycles: some 70 ms, far beyond a call's time on the host


def make(**kw):
    return PagedCache(n_pages=60, page_size=16, n_heads=HEADS, n_kv_heads=KV, head_dim=DIM, batch=B,
                      max_len=200, max_new=NEW, **kw)


def inputs(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((NEW, HEADS + 2 * KV, DIM), generator=g, device="cuda").to(torch.bfloat16)
    return x[:, :HEADS], x[:, HEADS:HEADS + KV], x[:, HEADS + KV:]


def lens(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def step(pc, want, x, **kw):
    q, k, v = x
    pc.resize(want, **kw)
    pc.write(k, v, **kw)
    return pc.attend(q, 1, **kw)


@pytest.fixture
def expected():
    """Results of three steps on the default stream, and their inputs."""
    pc = make()
    wants = [[40, 0, 33], [41, 30, 34], [90, 31, 0]]
    xs = [inputs(s) for s in range(3)]
    total = [73, 32, 50]
    return wants, xs, [step(pc, lens(w), x)[:t].clone() for w, x, t in zip(wants, xs, total)], total


@pytest.mark.parametrize("built", ["before", "inside"])
def test_side_stream_is_the_current_one(expected, built):
    """Inputs that the side stream has yet to write when the calls are made."""
    wants, xs, outs, total = expected
    pc = make() if built == "before" else None
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        pc = pc or make()
        want = lens([0] * B)
        x = tuple(torch.zeros_like(t) for t in xs[0])
        for w, src, o, t in zip(wants, xs, outs, total):
            later = lens(w)
            torch.cuda._sleep(SLEEP)
            want.copy_(later)
            for a, b in zip(x, src):
                a.copy_(b)
            got = step(pc, want, x)
            kept = got[:t].clone()
            pc.check()
            assert torch.equal(kept, o)


def test_captured_without_naming_the_stream(expected):
    wants, xs, outs, total = expected
    pc = make()
    want, x = lens([0] * B), tuple(torch.zeros_like(t) for t in xs[0])
    step(pc, want, x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(pc, want, x)
    for w, src, o, t in zip(wants, xs, outs, total):
        want.copy_(lens(w))
        for a, b in zip(x, src):
            a.copy_(b)
        graph.replay()
        pc.check()
        assert torch.equal(got[:t], o)
    assert pc.lens.tolist() == wants[-1]


@pytest.mark.parametrize("handle", [False, True])
def test_stream_given(expected, handle):
    """The result's memory is the given stream's: what the current stream still does
    with a freed tensor of the same size does not reach it."""
    wants, xs, outs, total = expected
    pc = make()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for w, x, o, t in zip(wants, xs, outs, total):
        want = lens(w)
        torch.cuda.synchronize()
        old = torch.empty_like(xs[0][0])
        torch.cuda._sleep(SLEEP)
        old.fill_(7)
        del old
        got = step(pc, want, x, stream=s.cuda_stream if handle else s)
        torch.cuda.synchronize()
        pc.check(stream=s)
        assert torch.equal(got[:t], o)


def test_two_caches_on_two_streams(expected):
    wants, xs, outs, total = expected
    both = [(make(), torch.cuda.Stream()) for _ in range(2)]
    torch.cuda.synchronize()
    for w, x, o, t in zip(wants, xs, outs, total):
        want = lens(w)
        torch.cuda.synchronize()
        got = [step(pc, want, x, stream=s) for pc, s in both]
        torch.cuda.synchronize()
        for g in got:
            assert torch.equal(g[:t], o)
    both[0][0].check()


def test_device_without_an_index():
    assert make(device="cuda").device == torch.device("cuda", torch.cuda.current_device())


# ---------------------------------------------------------------------------
# the error word
# ---------------------------------------------------------------------------

def bad_write(pc, stream):
    slots = torch.tensor([1 << 40], device="cuda")
    row = torch.zeros((1, KV, DIM), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    return lambda: dlm.dlm_paged_kv_write(pc.c, row, row, slots, 1, stream=stream)


def test_check_waits_for_its_own_stream_only():
    pc, s = make(), torch.cuda.Stream()
    call = bad_write(pc, s)
    torch.cuda._sleep(1 << 30)       # half a second on the default stream
    busy = torch.cuda.Event()
    busy.record()
    call()
    with pytest.raises(dlm.DlmError) as e:
        dlm.dlm_paged_check(s)
    assert e.value.code == dlm.DLM_EBOUNDS
    dlm.dlm_paged_check(s)
    assert not busy.query()
    torch.cuda.synchronize()


def test_one_check_of_two_gets_an_error():
    pc = make()
    streams = [torch.cuda.Stream() for _ in range(2)]
    call = bad_write(pc, streams[0])
    for _ in range(100):
        call()
        streams[0].synchronize()
        start, seen = threading.Barrier(2), []

        def check(s):
            start.wait()
            try:
                dlm.dlm_paged_check(s)
            except dlm.DlmError as e:
                seen.append(e.code)

        both = [threading.Thread(target=check, args=(s,)) for s in streams]
        for t in both:
            t.start()
        for t in both:
            t.join()
        assert seen == [dlm.DLM_EBOUNDS]
    dlm.dlm_paged_check()


def test_check_refuses_a_captured_stream_and_lets_the_capture_go_on(expected):
    wants, xs, outs, total = expected
    pc = make()
    want = lens(wants[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(dlm.DlmError) as e:
            pc.check()
        got = step(pc, want, xs[0])
    assert e.value.code == dlm.DLM_EINVAL
    graph.replay()
    pc.check()
    assert torch.equal(got[:total[0]], outs[0])


def test_any_object_with_a_stream_handle(expected):
    wants, xs, outs, total = expected

    class Handle:
        def __init__(self, s):
            self.cuda_stream = s.cuda_stream

    pc, s = make(), torch.cuda.Stream()
    want = lens(wants[0])
    torch.cuda.synchronize()
    got = step(pc, want, xs[0], stream=Handle(s))
    pc.check(stream=Handle(s))
    assert torch.equal(got[:total[0]], outs[0])


def test_built_inside_a_capture():
    """Its tensors are set by the replay."""
    q, k, v = inputs(4)
    want = lens([10, 0, 3])
    step(make(), want, (q, k, v))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pc = make()
        got = step(pc, want, (q, k, v))
    for _ in range(2):
        graph.replay()
        pc.check()
        assert pc.lens.tolist() == [10, 0, 3]
        assert torch.equal(got[:13], step(make(), want, (q, k, v))[:13])
