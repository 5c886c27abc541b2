"""Page accounting where the tables or the free list hold ids outside the
cache, and writes of rows that share a slot."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU-only hosts
    pytest.skip("needs a CUDA device", allow_module_level=True)

import masked_block_diffusion_denoise_b200 as dlm
from oracle import paged as OP
from test_gpu_paged import make_pool, run_resize, same_resize

N_PAGES = 2000


def pool(batch, page, seed):
    """Lengths of a batch in which every third sequence ends, every third shrinks and the others
    grow, some of them within a page that they hold; table and free list."""
    rng = np.random.default_rng(seed)
    cur = [int(x) for x in rng.integers(3 * page + 1, 5 * page, batch)]
    new = [0 if b % 3 == 0 else c - page - 1 if b % 3 == 1 else c + int(rng.integers(1, 3 * page))
           for b, c in enumerate(cur)]
    table, free = make_pool(cur, 9, page, N_PAGES, 40, seed)
    return cur, new, table, free


def refused(cur, new, table, page, free, max_new):
    got = run_resize(cur, new, table, page, free, N_PAGES, max_new)
    with pytest.raises(dlm.DlmError) as e:
        dlm.dlm_paged_check()
    assert e.value.code == dlm.DLM_EBOUNDS
    assert got["lens"] == cur and got["free"] == free and got["slots"] == [-1] * max_new
    assert np.array_equal(got["table"], table)


@pytest.mark.parametrize("bad", [-1, N_PAGES, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("batch,max_new", [(12, 4000), (12, 30000), (70, 4000), (1, 100)])
@pytest.mark.parametrize("where", ["released", "first released", "popped", "kept page"])
def test_bad_page_id_changes_nothing(bad, batch, max_new, where):
    """(30000 slots: a cluster of CTAs.)"""
    page = 16
    cur, new, table, free = pool(batch, page, 2)
    if batch == 1:
        if where == "kept page" or where == "popped":
            new = [cur[0] + 20]
    elif where == "popped":
        # one that ends, others that need more than it gives
        new = [0] + [c + 2 * page for c in cur[1:9]] + cur[9:]
    if where == "released":
        b = max(b for b in range(batch) if new[b] < cur[b])
        table[b, OP.pages(cur[b], page) - 1] = bad
    elif where == "first released":
        b = min(b for b in range(batch) if new[b] < cur[b])
        table[b, OP.pages(new[b], page)] = bad
    elif where == "popped":
        free[-1] = bad
    else:
        b = max(b for b in range(batch) if new[b] > cur[b] and cur[b] % page)
        table[b, cur[b] // page] = bad
    refused(cur, new, table, page, free, max_new)


def test_last_popped_and_last_released():
    cur, new, page = [0, 33], [16 * 5, 0], 16
    table, free = make_pool(cur, 8, page, N_PAGES, 9, 4)
    free[7] = -3              # three come back, so the last of five new pages is this one
    refused(cur, new, table, page, free, 200)
    free[7], free[6] = 3, N_PAGES    # one further down is not needed
    want = OP.resize(cur, new, table, page, free, 200)
    same_resize(run_resize(cur, new, table, page, free, N_PAGES, 200), want)
    dlm.dlm_paged_check()


def test_ids_that_the_call_does_not_use_are_not_looked_at():
    page = 16
    cur, new, table, free = pool(12, page, 5)
    table[1, 0] = -5                         # kept by a sequence that shrinks
    table[2, 0] = N_PAGES                    # a full page of one that grows
    free[0] = 2 ** 31 - 1                    # far down the stack
    new[5] = cur[5] = 4 * page               # on a border, and does not grow
    table[5, 3] = -1
    same_resize(run_resize(cur, new, table, page, free, N_PAGES, 4000),
                OP.resize(cur, new, table, page, free, 4000))
    dlm.dlm_paged_check()


def test_a_bad_id_of_a_refused_sequence_is_not_used():
    """The second sequence does not fit, so neither its page nor the stack's bottom is taken."""
    cur, new, page = [10, 20], [20, 200], 16
    table, free = make_pool(cur, 20, page, N_PAGES, 4, 6)
    table[1, 1], free[0] = -1, -1
    same_resize(run_resize(cur, new, table, page, free, N_PAGES, 400),
                OP.resize(cur, new, table, page, free, 400))
    dlm.dlm_paged_check()


@pytest.mark.parametrize("case", ["release", "take", "both", "bad released", "bad popped"])
def test_more_pages_than_a_block_keeps(case):
    """Tens of thousands of pages move in one call."""
    page, n_pages, width = 8, 60000, 7000
    cur = [0, 50001, 3, 40000, 9, 0]
    new = {"release": [0, 0, 3, 8, 9, 0], "take": [50000, 50001, 30003, 40000, 9, 30000]}.get(
        case, [56000, 0, 9000, 16, 20, 30001])
    table, free = make_pool(cur, width, page, n_pages, 20000, 7)
    if case == "bad released":
        table[3, 4700] = n_pages
    if case == "bad popped":
        free[-3000] = -1      # 11000 pages come back and 12000 and more are taken
        new[2] = 40000
    got = run_resize(cur, new, table, page, free, n_pages, 200000)
    if case.startswith("bad"):
        with pytest.raises(dlm.DlmError):
            dlm.dlm_paged_check()
        assert got["lens"] == cur and got["free"] == free and set(got["slots"]) == {-1}
        assert np.array_equal(got["table"], table)
    else:
        dlm.dlm_paged_check()
        same_resize(got, OP.resize(cur, new, table, page, free, 200000))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_that_share_a_slot_leave_the_others_alone(dtype):
    """Slots that several rows name hold pieces of those rows; the others their row, and
    what no row names stays."""
    kv, dim, page, n_pages, n = 3, 64, 16, 60, 500
    kc, vc = (torch.full((n_pages, kv, page, dim), -1.0, dtype=dtype, device="cuda") for _ in range(2))
    k = torch.arange(n, device="cuda").to(dtype)[:, None, None].expand(n, kv, dim).contiguous()
    v = (k + 1).contiguous() if dtype == torch.float32 else k.clone()
    slots = torch.arange(n, device="cuda") + 7
    slots[100:200] = 64           # a hundred rows, one slot
    slots[300:310] = slots[490:500]
    c = dlm.dlm_paged_cache(kc.data_ptr(), vc.data_ptr(), n_pages, page, kv, dim,
                            dlm.DLM_F32 if dtype == torch.float32 else dlm.DLM_BF16)
    dlm.dlm_paged_kv_write(c, k, v, slots, n)
    dlm.dlm_paged_check()
    named = {}
    for row, s in enumerate(slots.tolist()):
        named.setdefault(s, []).append(row)
    for cache, src in ((kc, k), (vc, v)):
        got = cache.permute(0, 2, 1, 3).reshape(n_pages * page, kv * dim).double().cpu()
        want = src[:, 0, 0].double().cpu()
        per = 16 // cache.element_size()
        for s in range(n_pages * page):
            rows = named.get(s)
            if rows is None:
                assert torch.all(got[s] == -1)
            else:
                pieces = got[s].reshape(-1, per)
                assert torch.all(pieces == pieces[:, :1])
                assert all(x in want[rows] for x in pieces[:, 0])
