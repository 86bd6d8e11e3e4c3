"""Tree attention over the 8-bit cache where its surroundings are hostile:
pages that are not there beside pages of NaN codes, caches that end inside a
tile with NaN codes around them, tree rows out of all proportion, scores of any
size.  Reference and tolerance are those of test_gpu_q8_attn."""
import pytest
import torch

from block_draft_tree_b200 import api

import q8_ref
from test_gpu_q8_attn import Case

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _leave_out_missing(c: Case):
    """The reference without the positions whose page is not there."""
    pool = c.c.codes[0].shape[0]

    def values(which, i, n):
        codes, exps = c.c.codes[which], q8_ref.scales(c.c.exps[which])
        t = torch.arange(n, device=DEV)
        pg = c.c.page_table[i].long()[t // c.c.page]
        t, pg = t[(pg >= 0) & (pg < pool)], pg[(pg >= 0) & (pg < pool)]
        slot = t % c.c.page
        return q8_ref.decode(codes[pg, slot]) * exps[pg, slot // c.c.block][:, :, None]

    c.c.values = values


@pytest.mark.parametrize("n,hq", [(1, 4), (9, 4), (70, 4), (140, 8)])
@pytest.mark.parametrize("page", [16, 48, 64])
def test_tokens_of_missing_pages_are_left_out(n, hq, page):
    """Page ids below and beyond the pool, at the start, inside and at the end of
    a context, and a sequence with no page at all; the pool's first page, which
    belongs to nobody, holds NaN codes."""
    c = Case(n, hq, 1, 128, page=page, ctx=(130, 100, 2 * page, 500), seed=n + page)
    pt = c.c.page_table
    spare = next(p for p in range(c.c.codes[0].shape[0]) if p not in pt.flatten().tolist())
    pt[pt == 0] = spare
    for w in range(2):
        c.c.codes[w][0] = 0x7F
        c.c.exps[w][0] = 48
    pt[0, 1], pt[1, 0], pt[2], pt[3, 2], pt[3, 500 // page] = -1, 1 << 30, -7, c.c.codes[0].shape[0], -1
    _leave_out_missing(c)
    c.check(*c.run(), status=1)


@pytest.mark.parametrize("n,hq", [(1, 8), (70, 1), (140, 2)])
def test_caches_that_end_inside_a_tile(n, hq):
    """A dense cache inside a larger buffer of NaN codes, before it and behind it."""
    for tokens in (1, 5, 17, 100, 129):
        c = Case(n, 2 * hq, 2, 128, ctx=(tokens, tokens), seed=tokens, tokens=tokens)
        for w in range(2):
            x = c.c.codes[w]
            buf = torch.full((x.numel() + 256 * 2 * 128,), 0x7F, dtype=torch.uint8, device=DEV)
            inner = buf[128 * 2 * 128:128 * 2 * 128 + x.numel()].view(x.shape)
            inner.copy_(x)
            c.c.codes[w] = inner
        c.go()


def test_split_trees_with_non_finite_rows_repeat_to_the_bit():
    """Splits of a large tree whose lanes take different ways through the
    epilogue (rows that see non-finite values and rows that do not)."""
    c = Case(70, 8, 2, 128, ctx=(6000, 77), seed=5)
    c.vt[0, 3, 0, 5], c.vt[0, 40, 1, 100] = float("inf"), float("nan")
    first = c.run()
    c.check(*first)
    for _ in range(10):
        again = c.run()
        for x, y in zip(first, again):
            assert torch.equal(x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32),
                               y.view(torch.int16 if y.dtype == torch.bfloat16 else torch.int32))


@pytest.mark.parametrize("n,d", [(2, 128), (9, 64), (9, 128), (70, 128), (140, 128)])
def test_huge_tree_values_reach_only_those_who_see_them(n, d):
    """V values from 2^57 on count as infinities where they are seen and as
    nothing elsewhere, also beside ordinary values of the same 16 rows."""
    c = Case(n, 4, 1, d, ctx=(50, 0), seed=n)
    c.vt[1, n - 1, 0, 0] = -2.0 ** 57
    c.vt[0, n - 1] = 3e38
    if n > 6:
        c.vt[0, 5, 0, 7], c.vt[0, 6, 0, 8:12] = 1e30, -1e25
    out, lse = c.run()
    huge = c.vt.abs() >= 2.0 ** 57
    c.vt = torch.where(huge, c.vt * float("inf"), c.vt)
    c.check(out, lse)


@pytest.mark.parametrize("n,d", [(2, 128), (9, 64), (9, 128), (70, 128), (140, 128)])
def test_a_tree_row_does_not_show_where_it_is_not_seen(n, d):
    """Rows of every magnitude that a bf16 row can have, in the middle of the
    others: those that do not see them keep their results to the bit, and those
    results are right."""
    c = Case(n, 4, 2, d, ctx=(50, 0), seed=n)
    hidden = [1] if n < 9 else [3, 7, n - 2]
    c.see[:, :, hidden] = False
    c.kt[:, hidden], c.vt[:, hidden] = 0.0, 0.0
    out, lse = c.run()
    c.check(out, lse)                 # (also the hidden rows' own results: their queries see others)
    for size in (2.0 ** -60, 1.0, 2.0 ** 20, 2.0 ** 40, 2.0 ** 56, 2.0 ** 57, 1e30, 3e38, float("inf"), float("nan")):
        c.kt[:, hidden], c.vt[:, hidden] = size, -size
        again = c.run()
        assert torch.equal(out.view(torch.int16), again[0].view(torch.int16)), size
        assert torch.equal(lse, again[1]), size


@pytest.mark.parametrize("n,d", [(5, 64), (9, 128), (70, 128), (140, 128)])
def test_tree_rows_of_unequal_size(n, d):
    """Rows whose K, and others whose V, are 2^-30 to 2^30 of their neighbours',
    each seen by rows that do not see the larger ones."""
    c = Case(n, 4, 1, d, ctx=(0, 33), seed=n, exps=(-9, -9))
    c.see[:] = False
    for j in range(n):                # row j sees itself and the rows of its own size below it
        c.see[:, j, j % 4:j + 1:4] = True
    size = torch.tensor([1.0, 2.0 ** 30, 2.0 ** -30, 2.0 ** 15], device=DEV)[torch.arange(n, device=DEV) % 4]
    c.vt = (c.vt * size[None, :, None, None]).to(torch.bfloat16)
    c.kt = (c.kt * size.flip(0)[None, :, None, None]).to(torch.bfloat16)
    c.q = (c.q / size.flip(0)[None, :, None, None]).to(torch.bfloat16)
    c.ctx[1] = 0 if n == 5 else 33
    out, lse = c.run()
    full = c.vt
    for z in range(4):                # the tolerance's max|v| is that of the rows that are seen
        rows = torch.arange(z, n, 4)
        c.vt = torch.where((torch.arange(n, device=DEV) % 4 == z)[None, :, None, None], full, 0.0)
        _check_rows(c, out, lse, rows)


def _check_rows(c, out, lse, rows):
    """Case.check for the given query rows alone."""
    sub = Case(len(rows), c.q.shape[2], c.c.hkv, c.q.shape[3], ctx=c.ctx, seed=0)
    n = c.n
    sub.c, sub.scale, sub.status = c.c, c.scale, c.status
    sub.q, sub.see = c.q[:, rows].contiguous(), c.see[:, rows][:, :, rows]
    sub.kt, sub.vt = c.kt[:, rows].contiguous(), c.vt[:, rows].contiguous()
    assert not c.see[:, rows][:, :, [j for j in range(n) if j not in rows.tolist()]].any()
    sub.n_nodes = [len(rows)] * len(c.ctx)
    sub.check(out[:, rows], lse[:, rows])


@pytest.mark.parametrize("n", [1, 9, 70, 140])
def test_scores_of_any_size(n):
    """Scores up to 2^50, whose last place is far above 1: tokens of the same
    largest score share the row (K and Q have one channel each, so that scores are
    exact), and sums of many channels stay within what is attended to."""
    for p in range(10, 64, 1):
        c = Case(n, 2, 1, 128, ctx=(300, 0), seed=n, exps=(-6, -6))
        c.scale = 0.125
        g = torch.Generator().manual_seed(p)
        ch = torch.tensor([0x38, 0x30, 0xB8], dtype=torch.uint8)      # 1, 1/2, -1 times 2^-6
        c.c.codes[0].zero_()
        c.c.codes[0][0, :, 0, 0] = ch[torch.randint(0, 3, (300,), generator=g)].to(DEV)
        c.c.codes[0][0, 0, 0, 0] = 0x38
        c.q.zero_()
        c.q[..., 0] = 2.0 ** p
        c.kt.zero_()
        c.kt[0, :, 0, 0] = 2.0 ** -8
        c.kt[1, :, 0, 0] = torch.tensor([1.0, 0.5])[torch.randint(0, 2, (n,), generator=g)].to(torch.bfloat16).to(DEV)
        c.vt = torch.where(c.vt < 0, -1.0, 1.0).to(torch.bfloat16)
        out, lse = c.run()
        if p < 26:
            c.check(out, lse)
            continue
        for i in range(2):
            kv = [c.c.values(w, i, c.ctx[i])[:, 0] for w in range(2)]
            for h in range(2):
                o, _, A, _ = q8_ref.attention(c.q[i, :, h].double(), kv, [c.kt[i, :, 0].double(), c.vt[i, :, 0].double()],
                                              c.see[i].to(DEV), c.scale)
                tol = o.abs() * 2.0 ** -8 + A * (2.0 ** -11 + 2.0 ** -20) + 2.0 ** -30   # bf16, P as f16, 1 / l
                assert ((out[i, :, h].double() - o).abs() <= tol).all(), (p, i, h)
    for p in range(16, 44):
        c = Case(n, 2, 1, 128, ctx=(300, 40), seed=p)
        c.q = c.q * 2.0 ** p
        out, lse = c.run()
        assert torch.isfinite(out).all() and torch.isfinite(lse).all(), p
        v = torch.cat([c.c.values(1, 0, 300), c.c.values(1, 1, 40), c.vt.double().flatten(0, 1)])
        assert out.abs().max() <= v.abs().max() * (1 + 2.0 ** -8) * (1 + 2.0 ** -10), p


@pytest.mark.parametrize("page", [0, 48])
def test_waits_of_the_kernel_for_few_rows_run_out(page):
    """A batch whose codes take the whole memory bandwidth, so that some of the
    thousands of waits on copies meet a bound of a few cycles: the status tells
    (out of ten calls, one has to), and the next call with the default bound
    gives what the one before gave."""
    c = Case(1, 32, 8, 128, page=page, ctx=[8160] * 64, seed=page)
    want = c.run()
    assert int(c.status) == 0
    told = []
    for _ in range(10):
        api.set_wait_limit(4)
        try:
            c.run()
            torch.cuda.synchronize()
        finally:
            api.set_wait_limit(0)
        told.append(int(c.status))
        again = c.run()
        assert int(c.status) == 0
        assert torch.equal(want[0], again[0]) and torch.equal(want[1], again[1])
    assert 5 in told and set(told) <= {0, 5}


@pytest.mark.parametrize("n", [9, 70, 140])
def test_a_row_depends_on_its_own_query_alone(n):
    """One query of scores beyond any range, one of NaN: the other rows keep
    their results to the bit."""
    c = Case(n, 4, 1, 128, ctx=(300, 40), seed=n)
    out, lse = c.run()
    c.q[0, 5, 2] *= 2.0 ** 30
    c.q[1, 2, 0] = float("nan")
    o2, l2 = c.run()
    assert torch.isfinite(o2[0, 5, 2]).all() and o2[1, 2, 0].isnan().all()
    o2[0, 5, 2], l2[0, 5, 2], o2[1, 2, 0], l2[1, 2, 0] = out[0, 5, 2], lse[0, 5, 2], out[1, 2, 0], lse[1, 2, 0]
    assert torch.equal(out, o2) and torch.equal(lse, l2)
