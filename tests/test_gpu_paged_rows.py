"""Paged attention, row by row: what a row's result depends on and what it
does not (other rows, slots that hold no token, what ran before)."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU-only hosts
    pytest.skip("needs a CUDA device", allow_module_level=True)

import masked_block_diffusion_denoise_b200 as dlm
from oracle import paged as OP
from test_gpu_paged import DT, Paged, check, ready

# Sequences of several key tiles a CTA: a row's softmax reference has earlier
# tiles to fall behind.  (heads, kv heads): G 4; 3, 5 and 7 do not divide a
# row tile of 128, whose last rows then hold no query at all.
GROUPS = [(8, 2), (6, 2), (10, 2), (14, 2)]
LENGTHS = [600 + 37 * b for b in range(60)]


@pytest.mark.parametrize("heads,kv", GROUPS)
@pytest.mark.parametrize("dim", [128, 64])
@pytest.mark.parametrize("n", [1, 3])
def test_unused_slots_do_not_reach_a_result(heads, kv, dim, n):
    """Slots behind a sequence hold large finite values, or infinities: the
    same bits as with zeros there."""
    outs = []
    for junk in (0.0, 1e4, -3e38, float("inf")):
        p = Paged("bf16", kv, dim, 64, LENGTHS, seed=5, junk=junk)
        q = ready(p, [n] * len(LENGTHS), heads, 5)
        o, lse, _ = p.attend(q, [n] * len(LENGTHS), heads, 1)
        outs.append((o, lse))
    for o, lse in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])


@pytest.mark.parametrize("heads,kv", GROUPS)
@pytest.mark.parametrize("block", [0, 1])
def test_other_sequences_queries_do_not_reach_a_row(heads, kv, block):
    p = Paged("bf16", kv, 128, 16, LENGTHS, seed=6, junk=0.0)
    new = [1 + b % 3 for b in range(len(LENGTHS))]
    q = ready(p, new, heads, 6)
    o, lse, cu = p.attend(q, new, heads, block)
    loud = q.clone()
    for b in range(1, len(new), 2):
        loud[cu[b]:cu[b + 1]] *= 64
    o2, lse2, _ = p.attend(loud, new, heads, block)
    for b in range(0, len(new), 2):
        rows = slice(cu[b], cu[b + 1])
        assert torch.equal(o[rows], o2[rows]) and torch.equal(lse[rows], lse2[rows]), b


@pytest.mark.parametrize("heads,kv,dim", [(8, 2, 128), (6, 2, 64), (4, 4, 128)])
def test_other_rows_of_a_chunk_do_not_reach_a_row(heads, kv, dim):
    """One position's query is 64 times as large; the keys that only the last
    position sees are: the other rows' bits stay."""
    ctx, n = 6000, 300
    p = Paged("bf16", kv, dim, 16, [ctx], seed=7)
    q = ready(p, [n], heads, 7)
    o, lse, _ = p.attend(q, [n], heads, 1)
    loud = q.clone()
    loud[5] *= 64
    loud[170] *= 64
    o2, lse2, _ = p.attend(loud, [n], heads, 1)
    rest = [i for i in range(n) if i not in (5, 170)]
    assert torch.equal(o[rest], o2[rest]) and torch.equal(lse[rest], lse2[rest])
    last = ctx - 1
    p.kc[int(p.table[0, last // 16]), :, last % 16] *= 64
    o3, lse3, _ = p.attend(q, [n], heads, 1)
    assert torch.equal(o[:-1], o3[:-1]) and torch.equal(lse[:-1], lse3[:-1])


@pytest.mark.parametrize("heads,kv", GROUPS)
@pytest.mark.parametrize("dim", [128, 64])
def test_same_bits_whatever_ran_before(heads, kv, dim):
    """The same call after kernels that leave other values in shared and tensor
    memory."""
    p = Paged("bf16", kv, dim, 16, LENGTHS, seed=8, junk=0.0)
    new = [1 + b % 2 for b in range(len(LENGTHS))]
    q = ready(p, new, heads, 8)
    big = Paged("bf16", 2, dim, 64, [3000, 900], seed=9)
    bq = ready(big, [700, 900], 8, 9, spread=100.0)
    a = torch.randn((4096, 4096), device="cuda", dtype=torch.bfloat16) * 1e3
    o, lse, _ = p.attend(q, new, heads, 1)
    for r in range(6):
        if r % 2:
            a @ a
        else:
            big.attend(bq * (r + 1), [700, 900], 8, 1)
        o2, lse2, _ = p.attend(q, new, heads, 1)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


# ---------------------------------------------------------------------------
# NaN and infinities that a row does see
# ---------------------------------------------------------------------------

def set_key(p, b, j, cache, column, value):
    """Element `column` of key j of sequence b (all KV heads), in the pages and beside them."""
    (p.kc if cache == "k" else p.vc)[int(p.table[b, j // p.page]), :, j % p.page, column] = value
    (p.k if cache == "k" else p.v)[b][j, :, column] = value


KINDS = [("bf16", 128), ("bf16", 64), ("f32", 64), ("f32", 128)]


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("ctx,n", [(2500, 1), (100, 1), (40, 7), (3000, 40)])
@pytest.mark.parametrize("block", [0, 1])
def test_nan_in_a_query(dtype, dim, ctx, n, block):
    """One head of one row holds a NaN: its result and lse are NaN however the work is
    cut (2500 keys: over many CTAs; 100: in one), the others keep their bits."""
    p = Paged(dtype, 2, dim, 16, [ctx, 30], seed=12)
    q = ready(p, [n, 2], 8, 12)
    o, lse, _ = p.attend(q, [n, 2], 8, block)
    q[n // 2, 3, 7] = float("nan")
    o2, lse2, _ = p.attend(q, [n, 2], 8, block)
    assert torch.isnan(o2[n // 2, 3]).all() and torch.isnan(lse2[n // 2, 3])
    o2[n // 2, 3], lse2[n // 2, 3] = o[n // 2, 3], lse[n // 2, 3]
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.isfinite(o).all()


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("cache,value", [("k", float("nan")), ("v", float("nan")),
                                         ("v", float("inf")), ("v", -float("inf"))])
@pytest.mark.parametrize("where", [3, 2000])
def test_bad_key_far_below_the_maximum(dtype, dim, cache, value, where):
    """A NaN or an infinity in a key whose neighbours' weights are 2^-200 of the others': a
    part of the work with weight 0 in float32, and still not a finite result."""
    ctx = 2500
    p = Paged(dtype, 1, dim, 16, [ctx], seed=13)
    lo = where // 400 * 400
    p.k[0].zero_()
    p.k[0][lo:lo + 400] = -200.0 / (1.4427 * dim ** 0.5)   # 1 . k / sqrt(dim) log2(e) = -200
    p.put(p.table[0].cpu().numpy(), p.k[0], p.kc)
    q = torch.ones((1, 4, dim), device="cuda").to(p.dtype)
    o, lse, _ = p.attend(q, [1], 4, 1)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    set_key(p, 0, where, cache, 9, value)
    o2, lse2, _ = p.attend(q, [1], 4, 1)
    if cache == "k":
        assert torch.isnan(o2).all() and torch.isnan(lse2).all()
    else:
        assert not torch.isfinite(o2[:, :, 9]).any()
        rest = [c for c in range(dim) if c != 9]
        assert torch.equal(o2[:, :, rest], o[:, :, rest]) and torch.equal(lse, lse2)
def defined(p, q, new, heads, block):
    """(o, lse) of every row from the keys that it sees, in float64 on the CPU,
    with NaN and infinities going where the formula takes them."""
    o = torch.zeros(q.shape, dtype=torch.float64)
    lse = torch.full(q.shape[:2], -torch.inf, dtype=torch.float64)
    row, g = 0, heads // p.kv
    for b, n in enumerate(new):
        k, v = p.k[b].double().cpu(), p.v[b].double().cpu()
        for i in range(n):
            m = OP.visible(p.ctx[b] - n + i, p.ctx[b], block)
            for h in range(heads if m else 0):
                s = k[:m, h // g] @ q[row, h].double().cpu() / p.dim ** 0.5
                o[row, h] = torch.softmax(s, 0) @ v[:m, h // g]
                lse[row, h] = torch.logsumexp(s, 0)
            row += 1
    return o, lse


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("ctx,n", [(150, 60), (2300, 30)])
def test_rows_that_see_bad_keys(dtype, dim, bad, ctx, n):
    """Keys with NaN or infinities in K and V among the chunk's own: a result is finite
    exactly where the formula's is."""
    p = Paged(dtype, 2, dim, 16, [ctx], seed=14)
    q = ready(p, [n], 4, 14)
    for j in range(ctx - 19, ctx, 7):
        set_key(p, 0, j, "k", 9, bad)
        set_key(p, 0, j, "v", 5, bad)
    o, lse, _ = p.attend(q, [n], 4, 1)
    ref, rl = defined(p, q, [n], 4, 1)
    assert torch.equal(torch.isfinite(o).cpu(), torch.isfinite(ref))
    assert torch.equal(torch.isnan(lse).cpu(), torch.isnan(rl) | torch.isposinf(rl))


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("where", [3, 120, 149])
def test_infinite_value_of_a_weight_that_underflows(dtype, dim, where):
    """A seen key of weight 2^-200 in a tile with hidden keys holds +inf in V: the
    formula's result is infinite, float32's 0 x infinity NaN; it is never finite."""
    ctx, n = 150, 40
    p = Paged(dtype, 1, dim, 16, [ctx], seed=15)
    p.k[0].zero_()
    p.k[0][where] = -200.0 / (1.4427 * dim ** 0.5)
    p.put(p.table[0].cpu().numpy(), p.k[0], p.kc)
    q = torch.ones((n, 2, dim), device="cuda").to(p.dtype)
    set_key(p, 0, where, "v", 9, float("inf"))
    o, _, _ = p.attend(q, [n], 2, 1)
    sees = torch.arange(ctx - n, ctx, device="cuda") >= where
    assert not torch.isfinite(o[sees][:, :, 9]).any()
    o[:, :, 9][sees] = 0
    assert torch.isfinite(o).all()


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("ctx,n", [(100, 4), (5, 9), (2500, 1), (3000, 200)])
@pytest.mark.parametrize("block", [0, 1])
def test_every_score_minus_infinity(dtype, dim, ctx, n, block):
    """A row that sees keys, all with a score of -inf: 0 / 0, not the zeros of a row that
    sees none."""
    p = Paged(dtype, 2, dim, 16, [ctx], seed=16)
    p.k[0][:, :, 3] = -1
    p.put(p.table[0].cpu().numpy(), p.k[0], p.kc)
    q = ready(p, [n], 8, 16)
    q[::2, 5, 3] = float("inf")
    o, lse, _ = p.attend(q, [n], 8, block)
    sees = torch.arange(ctx - n, ctx, device="cuda") >= (0 if block else -n)
    bad = torch.zeros((n, 8), dtype=torch.bool, device="cuda")
    bad[::2, 5] = True
    assert torch.isnan(o[bad & sees[:, None]]).all()
    assert torch.isfinite(o[~bad & sees[:, None]]).all()
    assert torch.all(o[~sees] == 0)
    assert torch.equal(torch.isneginf(lse), bad | ~sees[:, None]) and not torch.isnan(lse).any()


@pytest.mark.parametrize("dtype,dim,heads,kv", [("f32", 64, 4, 4), ("f32", 128, 8, 1), ("f32", 32, 100, 1),
                                                ("bf16", 128, 8, 2)])
@pytest.mark.parametrize("block", [0, 1])
def test_rows_without_keys_between_rows_with_keys(dtype, dim, heads, kv, block):
    """Items without any key directly before items with keys, many for each CTA: the bits
    of the same sequences by themselves."""
    ctx = [0 if b % 3 else 5 + b % 11 for b in range(600)]
    new = [2 if c == 0 else 1 for c in ctx]
    p = Paged(dtype, kv, dim, 8, ctx, seed=17)
    q = ready(p, new, heads, 17)
    o, lse, cu = p.attend(q, new, heads, block)
    # queries of the rows without keys, which are loaded nowhere, are NaN
    loud = q.clone()
    for b, c in enumerate(ctx):
        if c == 0:
            loud[cu[b]:cu[b + 1]] = float("nan")
    for _ in range(5):
        o2, lse2, _ = p.attend(loud, new, heads, block)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    full = torch.tensor([c > 0 for c, n in zip(ctx, new) for _ in range(n)], device="cuda")
    assert torch.all(o[~full] == 0) and torch.isneginf(lse[~full]).all()
    check(p, q, o, lse, cu, new, heads, block)


# ---------------------------------------------------------------------------
# the far ends of what the calls allow
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,dim", KINDS)
def test_blocks_as_long_as_an_int(dtype, dim):
    """One block holds every position: all keys for rows from position 0 on."""
    p = Paged(dtype, 2, dim, 16, [300, 5, 0], seed=18)
    new = [40, 9, 2]
    q = ready(p, new, 8, 18)
    o, lse, cu = p.attend(q, new, 8, 2 ** 31 - 1)
    check(p, q, o, lse, cu, new, 8, 2 ** 31 - 1)
    o0, lse0, _ = p.attend(q, new, 8, 300)
    assert torch.equal(o, o0) and torch.equal(lse, lse0)


@pytest.mark.parametrize("dtype,dim", KINDS)
@pytest.mark.parametrize("scale", [1e-45, 1e-30, 1e3])
def test_scales(dtype, dim, scale):
    """The smallest scale makes the mean of the values, a large one picks the largest score."""
    p = Paged(dtype, 2, dim, 16, [500, 3], seed=19)
    q = ready(p, [3, 1], 4, 19)
    o, lse, cu = p.attend(q, [3, 1], 4, 0, scale=scale)
    check(p, q, o, None, cu, [3, 1], 4, 0, scale=scale)
    if scale < 1:
        # all scores 0: log of the number of keys, a sum of that many ones in float32
        want = torch.log(torch.tensor([500.0, 500, 500, 3], device="cuda", dtype=torch.float64))
        assert bool(((lse.double() - want[:, None]).abs() <= 500 * 2.0 ** -23 + 2.0 ** -20).all())


@pytest.mark.parametrize("dtype,dim", KINDS[:3])
def test_sequences_that_share_pages(dtype, dim):
    """A common prefix in the same pages, tails of their own: as if each had a copy."""
    page, prefix, ctx = 16, 640, [700, 655, 641, 900]
    p = Paged(dtype, 2, dim, page, ctx, seed=20)
    for b in range(1, 4):
        p.table[b, :prefix // page] = p.table[0, :prefix // page]
        p.k[b][:prefix], p.v[b][:prefix] = p.k[0][:prefix], p.v[0][:prefix]
    new = [20, 1, 1, 130]
    q = ready(p, new, 8, 20)
    o, lse, cu = p.attend(q, new, 8, 1)
    check(p, q, o, lse, cu, new, 8, 1)


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_cache_beyond_32_bit_offsets(dtype, dim):
    """Pages at both ends of a cache of more than 2^32 elements, written and read: the bits of
    a small cache.  (A hidden infinite V, which is looked up in the pages again.)"""
    t, code = DT[dtype]
    kv, page, heads, n, ctx = 2, 256, 8, 40, 600
    n_pages = 2 ** 32 // (kv * page * dim) + 50
    small = Paged(dtype, kv, dim, page, [ctx], seed=21, junk=0.0)
    set_key(small, 0, ctx - 3, "v", 1, float("inf"))
    q = ready(small, [n], heads, 21)
    o, lse, _ = small.attend(q, [n], heads, 1)
    kc, vc = (torch.empty((n_pages, kv, page, dim), dtype=t, device="cuda") for _ in range(2))
    ids = torch.tensor([n_pages - 1, 0, n_pages - 2], device="cuda")
    kc[ids], vc[ids] = 0, 0
    at = torch.arange(ctx, device="cuda")
    c = dlm.dlm_paged_cache(kc.data_ptr(), vc.data_ptr(), n_pages, page, kv, dim, code)
    dlm.dlm_paged_kv_write(c, small.k[0], small.v[0], ids[at // page] * page + at % page, ctx)
    small.cache, small.table = c, ids.int()[None].contiguous()
    o2, lse2, _ = small.attend(q, [n], heads, 1)
    assert torch.isinf(o[-3:, :, 1]).all() and torch.isfinite(o[:-3]).all()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
