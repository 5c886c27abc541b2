"""session.PagedCache's device and stream, with fakes in the place of the
library and of torch's guards (no GPU needed)."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

from masked_block_diffusion_denoise_b200 import session


class Stream:
    def __init__(self, name, device):
        self.name, self.device = name, device


@pytest.fixture
def calls(monkeypatch):
    """(cache on cuda:1, while cuda:0 is current; list of (call, device, stream))."""
    seen, inside = [], [torch.device("cuda:0")]

    @contextlib.contextmanager
    def device(d):
        inside.append(torch.device(d))
        yield
        inside.pop()

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: inside[-1].index)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0x100 + index, raising=False)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda d=None: Stream("default", d))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device: Stream(h, device))
    for name in ("resize", "kv_write", "attention"):
        monkeypatch.setattr(session, "dlm_paged_" + name,
                            lambda *a, stream=None, name=name, **kw: seen.append((name, inside[-1], stream)))
    monkeypatch.setattr(session, "dlm_paged_check", lambda s: seen.append(("check", inside[-1], s)))
    pc = session.PagedCache.__new__(session.PagedCache)
    pc.device, pc.dtype = torch.device("cuda:1"), torch.float32
    pc.page_size, pc.n_heads, pc.batch, pc.max_new, pc.width = 8, 4, 2, 16, 3
    pc.k = pc.v = torch.zeros(5, 2, 8, 32)
    pc.table, pc.free, pc.n_free, pc.lens, pc.cu, pc.slots, pc.c, pc.work = [None] * 8
    return pc, seen


def step(pc, **kw):
    pc.resize(torch.zeros(2, dtype=torch.int32), **kw)
    pc.write(torch.zeros(3, 2, 32), torch.zeros(3, 2, 32), **kw)
    q = torch.zeros(3, 4, 32)
    pc.attend(q, 1, out=torch.zeros_like(q), **kw)
    pc.check(**kw)


def test_calls_switch_to_the_cache_s_device_and_its_current_stream(calls):
    pc, seen = calls
    step(pc)
    assert [name for name, _, _ in seen] == ["resize", "kv_write", "attention", "check"]
    for _, dev, stream in seen:
        assert dev == pc.device and stream == 0x101


def test_streams_given(calls):
    pc, seen = calls
    mine = Stream("mine", pc.device)
    step(pc, stream=mine)
    assert all(s is mine for _, _, s in seen)
    seen.clear()
    step(pc, stream=0x7700)
    assert all(s.name == 0x7700 and s.device == pc.device for _, _, s in seen)
    seen.clear()
    step(pc, stream=0)
    assert all(s.name == "default" for _, _, s in seen)
    with pytest.raises(ValueError):
        pc.resize(torch.zeros(2, dtype=torch.int32), stream=Stream("other", torch.device("cuda:0")))
