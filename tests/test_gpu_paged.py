"""The paged KV cache on the GPU against the float64 oracle: page accounting
and slot maps bit for bit, written rows bit for bit, attention within the
bound that its roundings allow."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU-only hosts
    pytest.skip("needs a CUDA device", allow_module_level=True)

import masked_block_diffusion_denoise_b200 as dlm
from oracle import paged as OP

DT = {"bf16": (torch.bfloat16, dlm.DLM_BF16), "f32": (torch.float32, dlm.DLM_F32)}


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().double().cpu().numpy()


# ---------------------------------------------------------------------------
# resize
# ---------------------------------------------------------------------------

def make_pool(cur, width, page, n_pages, n_free, seed):
    """(table, free stack) with every used page distinct."""
    rng = np.random.default_rng(seed)
    perm = [int(x) for x in rng.permutation(n_pages)]
    table = np.full((len(cur), width), -1, np.int32)
    for b, n in enumerate(cur):
        for c in range(OP.pages(max(n, 0), page)):
            if c < width:
                table[b, c] = perm.pop()
    return table, perm[:n_free]


def run_resize(cur, new, table, page, free, n_pages, max_new, alias=False, stream=None):
    B, W = table.shape
    t = torch.from_numpy(table.copy()).cuda()
    fr = torch.full((n_pages,), -7, dtype=torch.int32, device="cuda")
    if free:
        fr[:len(free)] = i32(free)
    c, n, nf = i32(cur), i32(new), i32([len(free)])
    out = c if alias else torch.full((B,), -9, dtype=torch.int32, device="cuda")
    nfo = nf if alias else i32([-9])
    cu = torch.full((B + 1,), -9, dtype=torch.int32, device="cuda")
    slots = torch.full((max_new + 3,), -9, dtype=torch.int64, device="cuda")
    dlm.dlm_paged_resize(c, n, out, B, t, W, page, fr, n_pages, nf, nfo, cu,
                         slots if max_new else None, max_new, stream=stream)
    torch.cuda.synchronize()
    assert slots[max_new:].tolist() == [-9] * 3
    n_out = int(nfo[0])
    # the stack past its old and new height is not touched
    assert fr[max(len(free), n_out, 0):].tolist() == [-7] * (n_pages - max(len(free), n_out, 0))
    return {"lens": out.tolist(), "cu": cu.tolist(), "slots": slots[:max_new].tolist(),
            "table": t.cpu().numpy(), "free": fr[:max(n_out, 0)].tolist()}


def same_resize(got, want):
    assert got["lens"] == want["lens"]
    assert got["cu"] == want["cu"]
    assert got["slots"] == want["slots"]
    assert got["free"] == want["free"]
    assert np.array_equal(got["table"], want["table"])


RESIZE = [
    # cur, new, page, width, n_free, max_new
    ([0], [1], 8, 1, 1, 1),
    ([0], [0], 8, 1, 0, 0),
    ([5], [8], 8, 1, 0, 3),                        # within the page it has
    ([8], [9], 8, 1, 3, 4),                        # the table is too narrow
    ([8], [9], 8, 2, 0, 4),                        # no page left
    ([17, 3, 40], [0, 30, 41], 16, 3, 0, 60),      # what one releases another takes
    ([17, 3, 40], [16, 16, 32], 16, 3, 5, 13),
    ([10, 10, 10, 10], [20, 90, 12, 40], 16, 8, 3, 200),   # second refused, third needs none
    ([0, 0, 0], [64, 64, 64], 64, 2, 9, 130),      # max_new too small for the third
    ([-1, 5, 7], [4, -2, 9], 8, 4, 4, 20),         # lengths below zero
    ([2147483647, 3], [5, 9], 8, 4, 4, 20),        # a length beyond the table
    ([3, 3], [2147483647, 9], 256, 4, 4, 20),
]


@pytest.mark.parametrize("i", range(len(RESIZE)))
@pytest.mark.parametrize("alias", [False, True])
def test_resize_cases(i, alias):
    cur, new, page, width, n_free, max_new = RESIZE[i]
    held = [min(n, width * page) if n <= width * page else 0 for n in cur]
    table, free = make_pool(held, width, page, 64, n_free, i)
    got = run_resize(cur, new, table, page, free, 64, max_new, alias)
    # the oracle walks every new token: a growth beyond 2^20 is cut to just
    # past max_new, which refuses it the same way
    cut = [c + max_new + 1 if n - c > 1 << 20 else n for c, n in zip(cur, new)]
    want = OP.resize(cur, cut, table, page, free, max_new)
    same_resize(got, want)
    dlm.dlm_paged_check()


@pytest.mark.parametrize("seed", range(8))
def test_resize_random(seed):
    rng = np.random.default_rng(100 + seed)
    B = [1, 2, 33, 256, 1023, 1025, 4096, 700][seed]
    page = int(rng.choice([8, 16, 32, 64, 128, 256]))
    cur = [int(x) for x in rng.integers(0, 300, B)]
    new = [int(x) for x in rng.integers(0, 300, B)]
    for b in range(B):
        if rng.random() < 0.3:
            new[b] = 0
        elif rng.random() < 0.5:
            new[b] = cur[b] + int(rng.integers(0, 40))
    width = OP.pages(300, page) - (seed == 3)
    cur = [min(c, width * page) for c in cur]
    used = sum(OP.pages(c, page) for c in cur)
    n_free = int(rng.integers(0, used // 4 + 2))
    n_pages = used + n_free + 17
    table, free = make_pool(cur, width, page, n_pages, n_free, seed)
    total = sum(max(0, n - c) for c, n in zip(cur, new))
    max_new = total + 9 if seed % 2 else max(1, total * 2 // 3)
    got = run_resize(cur, new, table, page, free, n_pages, max_new, alias=bool(seed & 1))
    same_resize(got, OP.resize(cur, new, table, page, free, max_new))
    dlm.dlm_paged_check()


def test_resize_grow_and_shrink_restores():
    cur, new = [100, 0, 33, 64], [228, 65, 33, 65]
    table, free = make_pool(cur, 32, 8, 200, 60, 3)
    up = run_resize(cur, new, table, 8, free, 200, 500)
    down = run_resize(up["lens"], cur, up["table"], 8, up["free"], 200, 0)
    assert down["free"] == free and down["lens"] == cur and down["cu"] == [0] * 5


def test_resize_broken_stack_changes_nothing():
    table, free = make_pool([40, 9], 8, 8, 20, 3, 1)
    for height in (-1, 21):
        t, fr = torch.from_numpy(table).cuda(), torch.full((20,), 4, dtype=torch.int32, device="cuda")
        cur, new, nf = i32([40, 9]), i32([0, 30]), i32([height])
        out, nfo, cu = i32([0, 0]), i32([77]), i32([0, 0, 0])
        slots = torch.zeros(25, dtype=torch.int64, device="cuda")
        dlm.dlm_paged_resize(cur, new, out, 2, t, 8, 8, fr, 20, nf, nfo, cu, slots, 25)
        with pytest.raises(dlm.DlmError) as e:
            dlm.dlm_paged_check()
        assert e.value.code == dlm.DLM_EBOUNDS
        assert out.tolist() == [40, 9] and int(nfo) == height and slots.tolist() == [-1] * 25
        assert np.array_equal(t.cpu().numpy(), table) and fr.tolist() == [4] * 20
    # more releases than the pool has room for
    got_nf, nf = i32([0]), i32([18])
    dlm.dlm_paged_resize(i32([40]), i32([0]), out, 1, t, 8, 8, fr, 20, nf, got_nf, cu, slots, 25)
    with pytest.raises(dlm.DlmError):
        dlm.dlm_paged_check()
    assert int(got_nf) == 18
    dlm.dlm_paged_check()      # the word was cleared


def test_resize_bad_page_ids_are_reported():
    for bad in (-1, 20, 2 ** 31 - 1):
        table = np.array([[bad, -1]], np.int32)
        got = run_resize([3], [6], table, 8, [1, 2], 20, 4)
        assert got["slots"] == [-1] * 4
        with pytest.raises(dlm.DlmError) as e:
            dlm.dlm_paged_check()
        assert e.value.code == dlm.DLM_EBOUNDS


# ---------------------------------------------------------------------------
# write
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,kv,dim,page,n,gap", [
    ("bf16", 8, 128, 64, 64, 0), ("bf16", 1, 64, 8, 1, 0), ("bf16", 3, 128, 16, 37, 8),
    ("f32", 4, 64, 32, 55, 4), ("f32", 1, 32, 256, 300, 0), ("f32", 2, 128, 128, 3, 12),
    ("bf16", 16, 128, 128, 1501, 4096), ("bf16", 5, 64, 32, 1000, 0)])
def test_write(dtype, kv, dim, page, n, gap):
    t, code = DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(n)
    n_pages = n // page + 7
    kc, vc = (torch.randn((n_pages, kv, page, dim), generator=g, device="cuda").to(t)
              for _ in range(2))
    rows = torch.randn((2, n, kv * dim + gap), generator=g, device="cuda").to(t)
    k, v = rows[0], rows[1]
    slots = torch.randperm(n_pages * page, generator=g, device="cuda")[:n]
    slots[::5] = -1
    slots[-1] = n_pages * page - 1 if n_pages * page - 1 not in slots[:-1].tolist() else slots[-1]
    wk, wv = kc.clone(), vc.clone()
    for src, dst in ((k, wk), (v, wv)):
        for i, s in enumerate(slots.tolist()):
            if s >= 0:
                dst[s // page, :, s % page] = src[i, :kv * dim].view(kv, dim)
    c = dlm.dlm_paged_cache(kc.data_ptr(), vc.data_ptr(), n_pages, page, kv, dim, code)
    dlm.dlm_paged_kv_write(c, k, v, slots, n, k_stride=k.stride(0), v_stride=v.stride(0))
    dlm.dlm_paged_check()
    assert torch.equal(kc, wk) and torch.equal(vc, wv)


def test_write_bad_slots_are_skipped_and_reported():
    kc = torch.zeros((4, 2, 8, 64), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    rows = torch.ones((3, 128), dtype=torch.bfloat16, device="cuda")
    c = dlm.dlm_paged_cache(kc.data_ptr(), vc.data_ptr(), 4, 8, 2, 64, dlm.DLM_BF16)
    for bad in (32, 2 ** 31, 2 ** 62, -2 ** 63):
        slots = torch.tensor([0, bad, 31], device="cuda")
        dlm.dlm_paged_kv_write(c, rows, rows, slots, 3)
        if bad > 0:
            with pytest.raises(dlm.DlmError) as e:
                dlm.dlm_paged_check()
            assert e.value.code == dlm.DLM_EBOUNDS
        else:
            dlm.dlm_paged_check()
        assert float(kc.sum()) == float(vc.sum()) == 2 * 128
    assert torch.all(kc[0, :, 0] == 1) and torch.all(kc[3, :, 7] == 1)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

class Paged:
    """A random cache of given lengths; slots that hold no token are NaN."""

    def __init__(self, dtype, kv, dim, page, ctx, seed, junk=float("nan")):
        t, code = DT[dtype]
        rng = np.random.default_rng(seed)
        self.kv, self.dim, self.page, self.dtype = kv, dim, page, t
        self.ctx = list(ctx)
        counts = [OP.pages(max(n, 0), page) for n in ctx]
        self.width = max(1, max(counts))
        n_pages = sum(counts) + 3
        perm = rng.permutation(n_pages)
        table = np.full((len(ctx), self.width), 2 ** 31 - 1, np.int32)   # never read past the end
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.kc = torch.full((n_pages, kv, page, dim), junk, dtype=t, device="cuda")
        self.vc = self.kc.clone()
        self.k, self.v = [], []
        at = 0
        for b, (n, c) in enumerate(zip(ctx, counts)):
            table[b, :c] = perm[at:at + c]
            at += c
            k, v = (torch.randn((max(n, 0), kv, dim), generator=g, device="cuda").to(t)
                    for _ in range(2))
            self.k.append(k)
            self.v.append(v)
            self.put(table[b], k, self.kc)
            self.put(table[b], v, self.vc)
        self.table = torch.from_numpy(table).cuda()
        self.cache = dlm.dlm_paged_cache(self.kc.data_ptr(), self.vc.data_ptr(), n_pages, page, kv,
                                         dim, code)
        self.g = g

    def put(self, row, x, cache):
        n = x.shape[0]
        if n == 0:
            return
        at = torch.arange(n, device="cuda")
        ids = torch.from_numpy(np.asarray(row, np.int64)).cuda()
        cache[ids[at // self.page], :, at % self.page] = x

    def attend(self, q, new, heads, block, scale=0.0, pad=0, lse=True, first=0, stream=None,
               o=None, work=None):
        """q [total][heads][dim] (rows may be strided); `first` rows of q
        precede the first sequence, pad follow the last."""
        cu = [first]
        for n in new:
            cu.append(cu[-1] + n)
        rows = cu[-1] + pad
        assert q.shape[0] == rows
        if o is None:
            o = torch.full((rows, heads, self.dim), 7.0, dtype=self.dtype, device="cuda")
        ls = torch.full((rows, heads), 7.0, device="cuda") if lse else None
        if work is None:
            n = dlm.dlm_paged_attention_workspace(self.cache, heads)
            work = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        dlm.dlm_paged_attention(self.cache, q, o, i32(cu), i32(self.ctx), self.table, self.width,
                                len(new), rows, heads, block, work, lse=ls, scale=scale,
                                q_stride=q.stride(0), o_stride=o.stride(0), stream=stream)
        dlm.dlm_paged_check(stream)
        return o, ls, cu


def check(p, q, o, lse, cu, new, heads, block, scale=0.0, keys=None, values=None):
    """Against the oracle.  With u the unit roundoff of the element type
    (bf16 2^-8, f32 2^-24) and per row A = sum_j p_j |v_j|:
      scores: products are exact in float32 for bf16 (rounded once for f32),
        Dh + 1 additions and the scale: |ds| <= (Dh + 2) 2^-23 mag, mag the
        largest sum_d |q_d k_d| scale (2^-23, not 2^-24: the tensor cores'
        additions may truncate), in both the numerator and the sum;
      exponentials: argument rounded at magnitude <= |s| + |max| (2^-23 * 2 mag)
        and 2^-22 for the function;
      bf16: each p rounded by u in the numerator; sums of n_keys terms in
        float32: n_keys * 2^-23 each for numerator and sum (a loose bound of
        blocked sums), and one rounding of the result by u."""
    u = 2.0 ** -8 if p.dtype == torch.bfloat16 else 2.0 ** -24
    for b, n in enumerate(new):
        if n == 0:
            continue
        kk = f64(p.k[b]) if keys is None else keys[b]
        vv = f64(p.v[b]) if values is None else values[b]
        ref, rl, a, mag = OP.attend(f64(q[cu[b]:cu[b] + n]), kk, vv, p.ctx[b], block,
                                    scale or None)
        got = f64(o[cu[b]:cu[b] + n])
        ds = mag * (p.dim + 2 + 2) * 2.0 ** -23 + 2.0 ** -22
        sums = max(p.ctx[b], 1) * 2.0 ** -23
        tol = a * (2 * ds + 2 * sums + (u if p.dtype == torch.bfloat16 else 0))[..., None] \
            if np.ndim(ds + sums) else a * (2 * ds + 2 * sums + u)
        tol = 1.01 * tol + u * np.abs(ref) + 1e-38
        err = np.abs(got - ref)
        assert np.isfinite(got).all(), "sequence %d: not finite" % b
        worst = (err - tol).max()
        assert worst <= 0, "sequence %d: error %g beyond the bound (%g)" % (b, err.max(), worst)
        if lse is not None:
            gl = f64(lse[cu[b]:cu[b] + n])
            empty = np.isneginf(rl)
            assert np.array_equal(np.isneginf(gl), empty)
            tl = ds + sums + np.abs(np.where(empty, 0, rl)) * 2.0 ** -22 + 2.0 ** -22
            assert (np.abs(np.where(empty, 0, gl - np.where(empty, 0, rl))) <= tl)[~empty].all()


def ready(p, new, heads, seed, first=0, pad=0, gap=0, spread=1.0):
    rows = first + sum(new) + pad
    g = torch.Generator(device="cuda").manual_seed(1000 + seed)
    q = (torch.randn((rows, heads * p.dim + gap), generator=g, device="cuda") * spread).to(p.dtype)
    return q[:, :heads * p.dim].unflatten(1, (heads, p.dim))


ATTEND = [
    # dtype, heads, kv, dim, page, [(ctx, new)], block
    ("bf16", 4, 1, 128, 16, [(1, 1)], 1),
    ("bf16", 1, 1, 128, 8, [(7, 3)], 1),
    ("bf16", 8, 2, 128, 16, [(130, 1), (0, 0), (17, 17), (128, 5), (129, 2)], 1),
    ("bf16", 8, 2, 128, 64, [(96, 32), (400, 32), (33, 32)], 0),
    ("bf16", 8, 8, 128, 32, [(300, 290), (40, 1)], 1),               # G 1: 128 positions a tile
    ("bf16", 6, 2, 128, 128, [(257, 129), (128, 128)], 1),           # G 3
    ("bf16", 10, 2, 64, 16, [(200, 77), (55, 55)], 1),               # G 5
    ("bf16", 14, 2, 128, 8, [(100, 100), (143, 19)], 48),            # G 7, blocks of 48
    ("bf16", 32, 2, 64, 256, [(600, 70), (256, 1), (257, 9)], 32),   # G 16
    ("bf16", 64, 1, 128, 16, [(90, 9), (140, 2)], 1),                # G 64: two positions a tile
    ("bf16", 128, 1, 64, 16, [(70, 5)], 1),                          # G 128: one
    ("bf16", 100, 1, 128, 16, [(70, 5)], 0),                         # G 100
    ("bf16", 8, 2, 128, 16, [(5, 20), (0, 4), (3, 3)], 1),           # rows before position 0
    ("bf16", 8, 2, 128, 16, [(5, 20), (0, 4), (3, 3)], 0),
    ("bf16", 8, 2, 64, 32, [(700, 700)], 256),
    ("bf16", 8, 2, 128, 64, [(1025, 600)], 1),
    ("bf16", 8, 2, 128, 256, [(2500, 1)], 1),
    ("bf16", 8, 2, 64, 8, [(1500, 2)] * 3, 0),
    ("f32", 4, 4, 64, 32, [(160, 32)], 0),
    ("f32", 4, 2, 128, 16, [(1, 1), (130, 33), (0, 0), (64, 64)], 1),
    ("f32", 6, 2, 32, 8, [(200, 70), (3, 5)], 1),
    ("f32", 5, 1, 64, 64, [(400, 1), (65, 1)], 1),
    ("f32", 8, 8, 128, 128, [(150, 100)], 48),
    ("f32", 7, 1, 128, 16, [(129, 129)], 32),
]


@pytest.mark.parametrize("i", range(len(ATTEND)))
def test_attention(i):
    dtype, heads, kv, dim, page, seqs, block = ATTEND[i]
    p = Paged(dtype, kv, dim, page, [c for c, _ in seqs], seed=i)
    new = [n for _, n in seqs]
    q = ready(p, new, heads, i)
    o, lse, cu = p.attend(q, new, heads, block)
    check(p, q, o, lse, cu, new, heads, block)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_strides_padding_scale(dtype):
    """q and o as views of wider rows, rows before the first and behind the
    last sequence (left as they were), a scale, no lse; scores far apart."""
    p = Paged(dtype, 2, 64 if dtype == "f32" else 128, 16, [90, 200], seed=77)
    new = [20, 41]
    q = ready(p, new, 8, 5, first=3, pad=6, gap=24, spread=4.0)
    wide = torch.full((q.shape[0], 8 * p.dim + 16), 7.0, dtype=p.dtype, device="cuda")
    o = wide[:, :8 * p.dim].unflatten(1, (8, p.dim))
    _, _, cu = p.attend(q, new, 8, 1, scale=0.25, pad=6, lse=False, first=3, o=o)
    check(p, q, o, None, cu, new, 8, 1, scale=0.25)
    assert torch.all(wide[:3] == 7) and torch.all(wide[-6:] == 7) and torch.all(wide[:, -16:] == 7)
    o2, lse, _ = p.attend(q, new, 8, 1, scale=0.25, pad=6, first=3)
    assert torch.equal(o2[3:-6], o[3:-6])      # the same bits with and without lse
    assert torch.all(lse[:3] == 7) and torch.all(lse[-6:] == 7)


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attention_masked_keys_do_not_reach_a_row(dtype, dim, bad):
    """Tokens late in the chunk hold infinities or NaN in K and V: rows that
    do not see them are as if they were not there, rows that do see a
    non-finite V give what the arithmetic gives."""
    ctx, new, first_bad = 150, 60, 131
    p = Paged(dtype, 2, dim, 16, [ctx, 40], seed=3)
    q = ready(p, [new, 40], 4, 3)
    at = torch.arange(first_bad, ctx, 7, device="cuda")
    row = p.table[0].long()
    p.vc[row[at // 16], :, at % 16, 5] = bad
    p.kc[row[at // 16], :, at % 16, 9] = bad
    o, lse, cu = p.attend(q, [new, 40], 4, 1)
    clean = first_bad - (ctx - new)          # rows of sequence 0 before the first bad key
    kk, vv = [f64(x) for x in p.k], [f64(x) for x in p.v]
    ref, rl, a, _ = OP.attend(f64(q[:clean]), kk[0][:first_bad], vv[0][:first_bad], first_bad, 1)
    got = f64(o[:clean])
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -20
    assert (np.abs(got - ref) <= 1.05 * u * a + u * np.abs(ref) + 1e-4 * a).all()
    assert np.isfinite(f64(lse[:clean])).all()
    # sequence 1 is not touched
    ref1, _, a1, _ = OP.attend(f64(q[new:]), kk[1], vv[1], 40, 1)
    assert (np.abs(f64(o[new:]) - ref1) <= 1.05 * u * a1 + u * np.abs(ref1) + 1e-4 * a1).all()


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_attention_seen_infinite_value(dtype, dim):
    """+inf in V at a seen key gives +inf in that column and leaves the
    others, in the diagonal tile as in the ones before it."""
    for where in (20, 140):
        p = Paged(dtype, 1, dim, 16, [160], seed=4)
        q = ready(p, [40], 2, 4)
        row = p.table[0].long()
        p.vc[row[where // 16], :, where % 16, 5] = float("inf")
        o, _, _ = p.attend(q, [40], 2, 1)
        sees = torch.arange(120, 160, device="cuda") >= where
        assert torch.isinf(o[:, :, 5]).all(1)[sees].all() and (o[:, :, 5][sees] > 0).all()
        assert torch.isfinite(o[:, :, 5][~sees]).all()
        rest = [c for c in range(dim) if c != 5]
        assert torch.isfinite(o[:, :, rest]).all()


def test_attention_extreme_scores():
    """Scores in the hundreds (a softmax that picks one key) and equal ones."""
    for dtype in ("bf16", "f32"):
        p = Paged(dtype, 2, 64, 32, [200], seed=9)
        q = ready(p, [50], 4, 9, spread=64.0)
        o, lse, cu = p.attend(q, [50], 4, 1)
        check(p, q, o, lse, cu, [50], 4, 1)
        q.zero_()
        o, lse, cu = p.attend(q, [50], 4, 0)
        check(p, q, o, lse, cu, [50], 4, 0)


def test_attention_reports_bad_inputs():
    """Bad page ids, lengths and offsets are skipped and reported; other
    sequences of the batch are computed."""
    for dtype, dim in (("bf16", 128), ("f32", 64)):
        for kind in ("page", "negative page", "length", "negative length", "offsets", "last offset"):
            p = Paged(dtype, 2, dim, 16, [50, 60], seed=2)
            new = [10, 20]
            q = ready(p, new, 4, 2)
            table, ctx, cu = p.table.clone(), i32([50, 60]), i32([0, 10, 30])
            if kind == "page":
                table[0, 1] = p.cache.n_pages
            elif kind == "negative page":
                table[0, 0] = -1
            elif kind == "length":
                ctx[0] = p.width * 16 + 1
            elif kind == "negative length":
                ctx[0] = -5
            elif kind == "offsets":
                cu[0] = 12
            else:
                cu[2] = 31
            o = torch.zeros_like(q)
            n = dlm.dlm_paged_attention_workspace(p.cache, 4)
            work = torch.zeros(n, dtype=torch.uint8, device="cuda")
            dlm.dlm_paged_attention(p.cache, q, o, cu, ctx, table, p.width, 2, 30, 4, 1, work)
            with pytest.raises(dlm.DlmError) as e:
                dlm.dlm_paged_check()
            assert e.value.code == dlm.DLM_EBOUNDS, kind
            if kind != "last offset":
                ref, _, a, _ = OP.attend(f64(q[10:]), f64(p.k[1]), f64(p.v[1]), 60, 1)
                assert (np.abs(f64(o[10:]) - ref) <= 2.0 ** -7 * (a + np.abs(ref))).all(), kind


def reference(p, q, new, heads, block):
    """attend() of every sequence in float64 on the GPU (larger sizes)."""
    o, a, row = torch.zeros(q.shape, dtype=torch.float64, device="cuda"), None, 0
    a, lse = torch.zeros_like(o), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    g = heads // p.kv
    for b, n in enumerate(new):
        ctx = p.ctx[b]
        pos = torch.arange(ctx - n, ctx, device="cuda")
        lim = torch.full_like(pos, ctx) if block == 0 else \
            torch.where(pos < 0, 0, ((pos // block + 1) * block).clamp(max=ctx))
        for h in range(heads if n and ctx else 0):
            k, v = p.k[b][:, h // g].double(), p.v[b][:, h // g].double()
            s = q[row:row + n, h].double() @ k.T / math.sqrt(p.dim)
            s = torch.where(torch.arange(ctx, device="cuda") < lim[:, None], s, -math.inf)
            seen = lim > 0
            e = torch.softmax(s[seen], 1)
            o[row:row + n, h][seen] = e @ v
            a[row:row + n, h][seen] = e @ v.abs()
            lse[row:row + n, h][seen] = torch.logsumexp(s[seen], 1)
        row += n
    return o, a, lse


@pytest.mark.parametrize("dtype,heads,kv,dim,page,seqs,block", [
    ("bf16", 8, 2, 128, 16, [(20000, 33), (70, 70), (9000, 1)], 0),       # one long sequence
    ("bf16", 8, 2, 128, 64, [(5000, 1500), (640, 640), (3, 3)], 1),       # more work than SMs
    ("bf16", 16, 4, 64, 32, [(2600, 1333), (257, 200)], 256),
    ("bf16", 3, 3, 128, 128, [(1700, 900)], 1),                           # G 1
    # row tiles whose limits lie many key tiles apart (a block boundary between them)
    ("bf16", 2, 2, 64, 16, [(2100, 1500), (1100, 1100)], 1000),
    ("bf16", 4, 4, 64, 64, [(600, 600), (700, 650), (300, 300)] * 8, 512),
    ("bf16", 4, 2, 128, 16, [(900, 900), (1300, 700)] * 6, 400),
    # many short items of two row tiles and of one, a key tile or a few each
    ("bf16", 512, 4, 64, 16, [(303, 5), (123, 8), (340, 5), (512, 1), (432, 7), (519, 8), (194, 1),
                              (310, 2), (35, 0), (491, 7), (248, 0), (413, 4)], 600),
    ("bf16", 256, 2, 128, 8, [(100, 7), (123, 8), (40, 5), (12, 1), (232, 7)] * 6, 1),
    # row tiles with a few rows in the last warps (G 33, 5)
    ("bf16", 66, 2, 64, 32, [(500, 40), (301, 7)], 1),
    ("bf16", 20, 4, 64, 16, [(700, 30), (1301, 27)] * 3, 0),
    ("bf16", 33, 1, 128, 8, [(780, 6)], 0),      # joined rows of a second row tile
    # one long chunk among single tokens: its rows are many times the mean
    ("bf16", 16, 4, 128, 16, [(40, 1)] * 30 + [(20000, 64)] + [(200, 1)] * 30, 0),
    ("bf16", 16, 4, 64, 16, [(40, 1)] * 30 + [(20000, 50)] + [(200, 1)] * 30, 1),
    ("f32", 8, 1, 64, 16, [(40, 1)] * 30 + [(9000, 17)] + [(200, 1)] * 30, 0),
    ("f32", 4, 2, 64, 32, [(6000, 70), (300, 300)], 1),
    ("f32", 6, 1, 128, 16, [(1500, 257)], 0),
])
def test_attention_larger(dtype, heads, kv, dim, page, seqs, block):
    p = Paged(dtype, kv, dim, page, [c for c, _ in seqs], seed=31)
    new = [n for _, n in seqs]
    q = ready(p, new, heads, 31)
    o, lse, _ = p.attend(q, new, heads, block)
    ref, a, rl = reference(p, q, new, heads, block)
    # roundings of p and of the result by u, and a part in 2^12 (bf16) or 2^18 (f32) of
    # sum p |v| for scores up to about 8 and sums of up to 20000 terms in float32
    u, rest = (2.0 ** -8, 2.0 ** -12) if dtype == "bf16" else (2.0 ** -24, 2.0 ** -18)
    tol = a * ((u if dtype == "bf16" else 0) * 1.01 + rest) + u * ref.abs()
    assert bool(((o.double() - ref).abs() <= tol).all())
    assert float((lse.double() - rl).abs().max()) <= rest


@pytest.mark.parametrize("batch,dtype", [(700, "bf16"), (4096, "bf16"), (700, "f32")])
def test_attention_many_sequences(batch, dtype):
    """More sequences than threads, a third of them empty, chunks of 0..3 tokens."""
    rng = np.random.default_rng(batch)
    ctx = [int(x) for x in rng.integers(0, 40, batch)]
    new = [min(c, int(x)) if rng.random() < 0.7 else 0 for c, x in zip(ctx, rng.integers(0, 4, batch))]
    p = Paged(dtype, 2, 64, 8, ctx, seed=batch)
    q = ready(p, new, 4, batch)
    o, lse, cu = p.attend(q, new, 4, 1)
    check(p, q, o, lse, cu, new, 4, 1)


def test_attention_deterministic():
    p = Paged("bf16", 2, 128, 16, [3000, 5, 700], seed=6)
    new = [30, 5, 200]
    q = ready(p, new, 8, 6)
    o, lse, _ = p.attend(q, new, 8, 1)
    for _ in range(3):
        o2, lse2, _ = p.attend(q, new, 8, 1)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

def test_a_run_of_steps():
    """Prompts, canvases of a block with a rollback, single tokens, an ended
    sequence whose pages another takes: resize, write, attend per step, all
    lengths on the device, against contiguous K/V kept beside it."""
    kv, heads, dim, page, B = 2, 8, 128, 16, 4
    n_pages, width, max_new = 64, 24, 256
    g = torch.Generator(device="cuda").manual_seed(11)
    kc = torch.full((n_pages, kv, page, dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    cache = dlm.dlm_paged_cache(kc.data_ptr(), vc.data_ptr(), n_pages, page, kv, dim, dlm.DLM_BF16)
    work = torch.empty(dlm.dlm_paged_attention_workspace(cache, heads), dtype=torch.uint8,
                       device="cuda")
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(n_pages, dtype=torch.int32, device="cuda")
    nf, lens = i32([n_pages]), i32([0] * B)
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    slots = torch.empty(max_new, dtype=torch.int64, device="cuda")
    hk = [np.zeros((0, kv, dim)) for _ in range(B)]
    hv = [np.zeros((0, kv, dim)) for _ in range(B)]
    host = [0] * B
    steps = [([70, 33, 0, 128], 1), ([102, 65, 0, 160], 0), ([70, 65, 0, 160], 0),
             ([102, 66, 90, 161], 256), ([0, 67, 91, 162], 1), ([140, 68, 92, 163], 1)]
    for want, block in steps:
        dlm.dlm_paged_resize(lens, i32(want), lens, B, table, width, page, free, n_pages, nf, nf,
                             cu, slots, max_new)
        new = [max(0, w - c) for w, c in zip(want, host)]
        total = sum(new)
        rows = torch.randn((max_new, (heads + 2 * kv) * dim), generator=g, device="cuda",
                           dtype=torch.bfloat16)
        q = rows[:, :heads * dim]
        k, v = rows[:, heads * dim:(heads + kv) * dim], rows[:, (heads + kv) * dim:]
        dlm.dlm_paged_kv_write(cache, k, v, slots, max_new, k_stride=rows.stride(0),
                               v_stride=rows.stride(0))
        o = torch.full((max_new, heads, dim), 3.0, dtype=torch.bfloat16, device="cuda")
        dlm.dlm_paged_attention(cache, q, o, cu, lens, table, width, B, max_new, heads, block,
                                work, q_stride=rows.stride(0))
        dlm.dlm_paged_check()
        assert lens.tolist() == want
        at = 0
        for b in range(B):
            hk[b], hv[b] = hk[b][:want[b]], hv[b][:want[b]]
            if new[b]:
                sl = slice(at, at + new[b])
                hk[b] = np.concatenate([hk[b], f64(k[sl]).reshape(-1, kv, dim)])
                hv[b] = np.concatenate([hv[b], f64(v[sl]).reshape(-1, kv, dim)])
                ref, _, a, _ = OP.attend(f64(q[sl]).reshape(-1, heads, dim), hk[b], hv[b], want[b],
                                         block)
                err = np.abs(f64(o[sl]) - ref)
                assert (err <= 2.0 ** -8 * (1.01 * a + np.abs(ref)) + 1e-4 * a).all()
            at += new[b]
        assert torch.all(o[total:] == 3)
        host = want
    held = sum(OP.pages(n, page) for n in host)
    assert int(nf) == n_pages - held
    used = [int(x) for b in range(B) for x in table[b, :OP.pages(host[b], page)]]
    assert sorted(used + free[:int(nf)].tolist()) == list(range(n_pages))


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f32", 64)])
def test_paged_cache_object(dtype, dim):
    """session.PagedCache: two requests, a canvas with a rollback, a clean pass over
    the finished block, against the contiguous definition."""
    from masked_block_diffusion_denoise_b200.session import PagedCache
    heads, kv = 4, 2
    pc = PagedCache(n_pages=40, page_size=16, n_heads=heads, n_kv_heads=kv, head_dim=dim, batch=2,
                    max_len=200, max_new=160, dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(3)
    host, hk, hv = [0, 0], [np.zeros((0, kv, dim))] * 2, [np.zeros((0, kv, dim))] * 2
    for want, block in (([70, 45], 1), ([102, 77], 0), ([70, 45], 0), ([102, 77], 32), ([0, 78], 1)):
        pc.resize(i32(want))
        new = [max(0, w - h) for w, h in zip(want, host)]
        rows = sum(new)
        x = torch.randn((rows, heads + 2 * kv, dim), generator=g, device="cuda").to(pc.dtype)
        q, k, v = x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]
        pc.write(k, v)
        o = pc.attend(q, block)
        pc.check()
        at = 0
        for b in range(2):
            sl = slice(at, at + new[b])
            hk[b] = np.concatenate([hk[b][:want[b]], f64(k[sl])])
            hv[b] = np.concatenate([hv[b][:want[b]], f64(v[sl])])
            if new[b]:
                ref, _, a, mag = OP.attend(f64(q[sl]), hk[b], hv[b], want[b], block)
                # probabilities and results rounded once each; scores' and sums' f32 roundings
                u, up = (2.0 ** -8, 2.0 ** -8) if dtype == "bf16" else (2.0 ** -24, 0.0)
                rest = 2 * (mag * (dim + 4) + want[b] + 2) * 2.0 ** -23
                tol = 1.01 * a * (up + rest[..., None]) + u * np.abs(ref)
                assert (np.abs(f64(o[sl]) - ref) <= tol).all()
            at += new[b]
        host = want
    assert pc.lens.tolist() == [0, 78] and int(pc.n_free) == 40 - OP.pages(78, 16)
    pc.attend(q, 1, lse=torch.empty(q.shape[:2], device="cuda"))
    with pytest.raises(ValueError):
        pc.write(k.double(), v.double())
    with pytest.raises(ValueError):
        pc.write(k[:, :1], v[:, :1])                       # too few heads
    with pytest.raises(ValueError):
        pc.write(k[:1].expand(4, kv, dim), v[:1].expand(4, kv, dim))   # one row four times
    with pytest.raises(ValueError):
        pc.attend(q[:, :2], 1)
    with pytest.raises(ValueError):
        pc.attend(q, 1, lse=torch.empty((1, 1), device="cuda"))
    with pytest.raises(ValueError):
        pc.attend(q, 1, out=torch.empty((2, heads, dim), device="cuda").to(pc.dtype))
    with pytest.raises(ValueError):
        pc.resize(torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        pc.resize(i32([1, 2, 3]))
    # one row from a strided view: its row stride is not asked for
    x = torch.randn((1, 3 * kv, dim), generator=g, device="cuda").to(pc.dtype)[:, kv:2 * kv]
    pc.resize(i32([0, 79]))
    pc.write(x, x)
    page, off = pc.table[1, 78 // 16], 78 % 16
    pc.check()
    assert torch.equal(pc.k[page, :, off], x[0]) and torch.equal(pc.v[page, :, off], x[0])


def test_captured_step_follows_device_lengths():
    """One graph of resize, write and attend, replayed while the lengths on
    the device change, beside an eager call on another stream with its own
    workspace."""
    kv, heads, dim, page, B = 2, 8, 128, 16, 3
    n_pages, width, max_new = 40, 12, 48
    kc = torch.full((n_pages, kv, page, dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    cache = dlm.dlm_paged_cache(kc.data_ptr(), vc.data_ptr(), n_pages, page, kv, dim, dlm.DLM_BF16)
    work = torch.empty(dlm.dlm_paged_attention_workspace(cache, heads), dtype=torch.uint8,
                       device="cuda")
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(n_pages, dtype=torch.int32, device="cuda")
    nf, lens, want = i32([n_pages]), i32([0] * B), i32([0] * B)
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    slots = torch.empty(max_new, dtype=torch.int64, device="cuda")
    q = torch.zeros((max_new, heads, dim), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((max_new, kv, dim), dtype=torch.bfloat16, device="cuda")
    v, o = torch.zeros_like(k), torch.zeros_like(q)
    other = Paged("bf16", 2, 128, 16, [500, 90], seed=8)
    oq = ready(other, [20, 90], 8, 8)
    want_o, _, _ = other.attend(oq, [20, 90], 8, 1)

    def step(stream):
        dlm.dlm_paged_resize(lens, want, lens, B, table, width, page, free, n_pages, nf, nf, cu,
                             slots, max_new, stream=stream)
        dlm.dlm_paged_kv_write(cache, k, v, slots, max_new, stream=stream)
        dlm.dlm_paged_attention(cache, q, o, cu, lens, table, width, B, max_new, heads, 1, work,
                                stream=stream)

    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step(s)            # nothing to do yet: lengths 0
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            step(s)
    g = torch.Generator(device="cuda").manual_seed(21)
    hk, hv = [torch.zeros((0, kv, dim), device="cuda")] * B, [torch.zeros((0, kv, dim), device="cuda")] * B
    host = [0] * B
    side = torch.cuda.Stream()
    for target in ([10, 0, 33], [11, 17, 34], [43, 18, 35], [44, 0, 36], [45, 20, 52]):
        want.copy_(i32(target))
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        o.fill_(5.0)
        torch.cuda.synchronize()
        graph.replay()
        got, _, _ = other.attend(oq, [20, 90], 8, 1, stream=side)
        torch.cuda.synchronize()
        dlm.dlm_paged_check()
        assert torch.equal(got, want_o)
        at = 0
        for b in range(B):
            n = max(0, target[b] - host[b])
            hk[b] = torch.cat([hk[b][:target[b]], k[at:at + n].float()])
            hv[b] = torch.cat([hv[b][:target[b]], v[at:at + n].float()])
            if n:
                ref, _, a, _ = OP.attend(f64(q[at:at + n]), f64(hk[b]), f64(hv[b]), target[b], 1)
                assert (np.abs(f64(o[at:at + n]) - ref) <=
                        2.0 ** -8 * (1.01 * a + np.abs(ref)) + 1e-4 * a).all()
            at += n
        assert torch.all(o[at:] == 5)
        host = target
    assert lens.tolist() == host


def test_first_calls_inside_a_capture():
    """The first use of every call in a process may be the captured one."""
    script = """
import torch
import masked_block_diffusion_denoise_b200 as dlm
z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")
i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
kc, vc = z(8, 2, 16, 128), z(8, 2, 16, 128)
c = dlm.dlm_paged_cache(kc.data_ptr(), vc.data_ptr(), 8, 16, 2, 128, dlm.DLM_BF16)
work = z(dlm.dlm_paged_attention_workspace(c, 8), t=torch.uint8)
lens, want, table, free, nf = i([0]), i([20]), z(1, 4, t=torch.int32), torch.arange(8, dtype=torch.int32, device="cuda"), i([8])
cu, slots = z(2, t=torch.int32), z(24, t=torch.int64)
q, k, v, o = z(24, 8, 128) + 1, z(24, 2, 128) + 1, z(24, 2, 128) + 2, z(24, 8, 128)
torch.cuda.synchronize()
g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.graph(g, stream=s):
    dlm.dlm_paged_resize(lens, want, lens, 1, table, 4, 16, free, 8, nf, nf, cu, slots, 24, stream=s)
    dlm.dlm_paged_kv_write(c, k, v, slots, 24, stream=s)
    dlm.dlm_paged_attention(c, q, o, cu, lens, table, 4, 1, 24, 8, 1, work, stream=s)
g.replay()
torch.cuda.synchronize()
dlm.dlm_paged_check()
assert torch.all(o[:20] == 2) and torch.all(o[20:] == 0), o
print("fine")
"""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", script], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


def test_back_to_back_calls_see_each_other():
    """Resize, write and attend in a row without a pause, many times: the kernels'
    overlapping starts must not read what the one before has yet to write."""
    kv, heads, dim, page, B = 2, 8, 128, 16, 64
    n_pages, width = 1024, 16
    kc = torch.zeros((n_pages, kv, page, dim), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    cache = dlm.dlm_paged_cache(kc.data_ptr(), vc.data_ptr(), n_pages, page, kv, dim, dlm.DLM_BF16)
    work = torch.empty(dlm.dlm_paged_attention_workspace(cache, heads), dtype=torch.uint8, device="cuda")
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(n_pages, dtype=torch.int32, device="cuda")
    nf, lens, cu = i32([n_pages]), i32([0] * B), torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    wants = [i32([0] * B), i32([33] * B), i32([b % 40 for b in range(B)])]
    slots = torch.empty(B * 40, dtype=torch.int64, device="cuda")
    q = torch.ones((B * 40, heads, dim), dtype=torch.bfloat16, device="cuda")
    k = torch.ones((B * 40, kv, dim), dtype=torch.bfloat16, device="cuda")
    outs = []
    for r in range(60):
        v = torch.full((B * 40, kv, dim), float(r % 7 + 1), dtype=torch.bfloat16, device="cuda")
        o = torch.zeros((B * 40, heads, dim), dtype=torch.bfloat16, device="cuda")
        for w in (wants[0], wants[1 + r % 2]):
            dlm.dlm_paged_resize(lens, w, lens, B, table, width, page, free, n_pages, nf, nf, cu, slots,
                                 B * 40)
            dlm.dlm_paged_kv_write(cache, k, v, slots, B * 40)
            dlm.dlm_paged_attention(cache, q, o, cu, lens, table, width, B, B * 40, heads, 1, work)
        outs.append((r, o))
    dlm.dlm_paged_check()
    for r, o in outs:
        total = int(wants[1 + r % 2].sum())
        assert torch.all(o[:total] == r % 7 + 1) and torch.all(o[total:] == 0), r


def test_host_pointers_are_refused():
    p = Paged("bf16", 2, 128, 16, [20], seed=1)
    q = ready(p, [4], 4, 1)
    with pytest.raises(dlm.DlmError) as e:
        p.attend(q.cpu(), [4], 4, 1)
    assert e.value.code == dlm.DLM_EINVAL
    with pytest.raises(dlm.DlmError) as e:
        dlm.dlm_paged_kv_write(p.cache, q.cpu(), q, torch.zeros(4, dtype=torch.int64, device="cuda"), 4)
    assert e.value.code == dlm.DLM_EINVAL
    assert math.isfinite(float(q.float().sum()))
