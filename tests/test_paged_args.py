"""Refusals of the paged KV cache's calls: everything that can be checked on
the host is, before any launch (no GPU needed), and the page oracle's own
properties."""
import numpy as np
import pytest

import masked_block_diffusion_denoise_b200 as dlm
from oracle import paged as OP

A = 0x10000   # an aligned address that no refused call dereferences


def cache(**kw):
    f = dict(k=A, v=A, n_pages=16, page_size=16, n_kv_heads=2, head_dim=128, dtype=dlm.DLM_BF16)
    f.update(kw)
    return dlm.dlm_paged_cache(*(f[n] for n in ("k", "v", "n_pages", "page_size", "n_kv_heads",
                                                "head_dim", "dtype")))


class Work:
    """Stands for a workspace tensor."""

    def __init__(self, n, ptr=A):
        self.n, self.ptr = n, ptr

    def numel(self):
        return self.n

    def element_size(self):
        return 1

    def data_ptr(self):
        return self.ptr


def refused(fn, *a, **kw):
    with pytest.raises(dlm.DlmError) as e:
        fn(*a, **kw)
    assert e.value.code == dlm.DLM_EINVAL
    assert dlm.dlm_last_error(None)


BAD_CACHES = [dict(k=0), dict(v=0), dict(k=A + 8), dict(v=A + 2), dict(page_size=0),
              dict(page_size=4), dict(page_size=24), dict(page_size=512), dict(page_size=-16),
              dict(n_pages=0), dict(n_pages=-1), dict(n_kv_heads=0), dict(head_dim=96),
              dict(head_dim=32), dict(head_dim=256), dict(dtype=2), dict(dtype=-1),
              dict(dtype=dlm.DLM_F32, head_dim=16), dict(n_pages=2 ** 31 - 1, n_kv_heads=2),
              dict(n_kv_heads=65537, n_pages=1)]


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_bad_caches(bad):
    c = cache(**bad)
    refused(dlm.dlm_paged_kv_write, c, A, A, A, 4)
    refused(dlm.dlm_paged_attention_workspace, c, 4)
    refused(dlm.dlm_paged_attention, c, A, A, A, A, A, 8, 1, 4, 4, 1, Work(1 << 30))


@pytest.mark.parametrize("i", [0, 1, 2, 4, 7, 9, 10, 11, 12])
def test_resize_null_pointers(i):
    args = [A, A, A, 2, A, 4, 16, A, 16, A, A, A, A, 8]
    args[i] = None
    refused(dlm.dlm_paged_resize, *args)


@pytest.mark.parametrize("i,value", [(3, 0), (3, -1), (3, 4097), (5, 0), (6, 12), (6, 0),
                                     (6, 512), (8, 0), (13, -1), (13, 2 ** 30 + 1)])
def test_resize_ranges(i, value):
    args = [A, A, A, 2, A, 4, 16, A, 16, A, A, A, A, 8]
    args[i] = value
    refused(dlm.dlm_paged_resize, *args)


@pytest.mark.parametrize("i", [0, 1, 2, 4, 7, 9, 10, 11, 12])
def test_resize_unaligned(i):
    args = [A, A, A, 2, A, 4, 16, A, 16, A, A, A, A, 8]
    args[i] = A + (4 if i == 12 else 2)
    refused(dlm.dlm_paged_resize, *args)


def test_other_calls_unaligned():
    refused(dlm.dlm_paged_kv_write, cache(), A, A, A + 4, 4)
    for i in (3, 4, 5):
        args = [cache(), A, A, A, A, A, 8, 1, 4, 4, 1]
        args[i] += 2
        refused(dlm.dlm_paged_attention, *args, Work(1 << 30))
    refused(dlm.dlm_paged_attention, cache(), A, A, A, A, A, 8, 1, 4, 4, 1, Work(1 << 30), lse=A + 1)


def test_write_refusals():
    c = cache()
    w = dlm.dlm_paged_kv_write
    refused(w, c, None, A, A, 4)
    refused(w, c, A, None, A, 4)
    refused(w, c, A, A, None, 4)
    refused(w, c, A + 2, A, A, 4)
    refused(w, c, A, A + 8, A, 4)
    refused(w, c, A, A, A, -1)
    refused(w, c, A, A, A, 4, k_stride=255)      # shorter than a row
    refused(w, c, A, A, A, 4, v_stride=260)      # 520 bytes: not a multiple of 16
    refused(w, c, A, A, A, 4, k_stride=-256)
    assert w(c, None, None, None, 0) == dlm.DLM_OK


@pytest.mark.parametrize("i,value", [(1, None), (2, None), (3, None), (4, None), (5, None),
                                     (1, A + 2), (2, A + 8), (6, 0), (7, 0), (7, 4097), (8, -1),
                                     (9, 3), (9, 0), (9, 258), (10, -1)])
def test_attention_refusals(i, value):
    args = [cache(), A, A, A, A, A, 8, 1, 4, 4, 1]
    args[i] = value
    refused(dlm.dlm_paged_attention, *args, Work(1 << 30))


@pytest.mark.parametrize("kw", [dict(scale=-1.0), dict(scale=float("nan")),
                                dict(scale=float("inf")), dict(scale=1e31), dict(q_stride=508),
                                dict(q_stride=516), dict(o_stride=100)])
def test_attention_options_refused(kw):
    refused(dlm.dlm_paged_attention, cache(), A, A, A, A, A, 8, 1, 4, 4, 1, Work(1 << 30), **kw)


def test_attention_workspace_refused():
    refused(dlm.dlm_paged_attention, cache(), A, A, A, A, A, 8, 1, 4, 4, 1, Work(16))
    refused(dlm.dlm_paged_attention, cache(), A, A, A, A, A, 8, 1, 4, 4, 1, Work(1 << 30, A + 16))
    refused(dlm.dlm_paged_attention, cache(), A, A, A, A, A, 8, 1, 4, 4, 1, Work(1 << 30, 0))
    refused(dlm.dlm_paged_attention, cache(n_kv_heads=1), A, A, A, A, A, 8, 1, 2 ** 25, 128, 1,
            Work(1 << 30))   # 2^25 x 128 rows


def test_oracle_grow_and_shrink_restores_the_stack():
    rng = np.random.default_rng(5)
    for trial in range(20):
        B, P = int(rng.integers(1, 9)), int(rng.choice([8, 16, 64]))
        cur = [int(x) for x in rng.integers(0, 200, B)]
        new = [c + int(x) for c, x in zip(cur, rng.integers(0, 90, B))]
        perm = [int(x) for x in rng.permutation(500)]
        table = np.full((B, 40), -1, np.int32)
        for b in range(B):
            for c in range(OP.pages(cur[b], P)):
                table[b, c] = perm.pop()
        free = perm[:int(rng.integers(0, 60))]
        up = OP.resize(cur, new, table, P, free, 10000)
        held = [int(up["table"][b, c]) for b in range(B)
                for c in range(OP.pages(up["lens"][b], P))]
        assert len(set(held + up["free"])) == len(held) + len(up["free"])   # no page twice
        down = OP.resize(up["lens"], cur, up["table"], P, up["free"], 10000)
        assert down["free"] == free and down["lens"] == cur
        valid = [s for s in up["slots"] if s >= 0]
        assert len(set(valid)) == len(valid) == sum(l - c for l, c in zip(up["lens"], cur))


def test_oracle_resize_by_hand():
    # pages of 8; sequence 0 ends (pages 5, 6), 1 grows by one page, 2 wants three
    table = np.array([[5, 6, -1], [7, -1, -1], [-1, -1, -1]], np.int32)
    r = OP.resize([9, 6, 0], [0, 10, 24], table, 8, [1], 40)
    # stack 1, 6, 5: sequence 1 takes 5; three more pages are not there
    assert r["lens"] == [0, 10, 0] and r["free"] == [1, 6]
    assert r["table"][1, 1] == 5 and r["cu"] == [0, 0, 4, 28]
    assert r["slots"] == [62, 63, 40, 41] + [-1] * 36


def test_oracle_attend_by_hand():
    q = np.array([[[1.0, 0.0]], [[0.0, 2.0]]])          # two rows, positions 1 and 2
    k = np.array([[[1.0, 1.0]], [[2.0, 0.0]], [[0.0, 1.0]]])
    v = np.array([[[1.0, 0.0]], [[0.0, 1.0]], [[4.0, 4.0]]])
    o, lse, _, _ = OP.attend(q, k, v, 3, 1, scale=1.0)
    e = np.exp
    np.testing.assert_allclose(o[0, 0], np.array([e(1), e(2)]) / (e(1) + e(2)))
    np.testing.assert_allclose(lse[0, 0], np.log(e(1) + e(2)))
    w = np.array([e(2), e(0), e(2)])
    np.testing.assert_allclose(o[1, 0], (w[0] * v[0, 0] + w[1] * v[1, 0] + w[2] * v[2, 0]) / w.sum())
    # a row before position 0 sees nothing
    o, lse, _, _ = OP.attend(q, k[:1], v[:1], 1, 1)
    assert np.all(o[0] == 0) and np.isneginf(lse[0, 0])
    assert [OP.visible(p, 10, 4) for p in (-1, 0, 3, 4, 9)] == [0, 4, 4, 8, 10]
    assert OP.visible(2, 10, 0) == 10
