"""session.PagedCache's device, with fakes in the place of the
library and of torch's guards (no GPU needed)."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

from masked_block_diffusion_denoise_b200 import session


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


def test_calls_switch_to_the_cache_s_device(calls):
    pc, seen = calls
    step(pc)
    assert [name for name, _, _ in seen] == ["resize", "kv_write", "attention", "check"]
    assert all(dev == pc.device for _, dev, _ in seen)
