"""Tree attention over the 8-bit key/value cache against the plain reference.

Tolerance, element by element, with A = sum_j p_j |v_j| of the row and S its
largest scale * sum |q k| over a token:
  * the output's rounding to bf16: |out| * 2^-8;
  * each weight's rounding to f16: A * 2^-11 (half a step of 11 bits), and
    f16's subnormal step: a weight of the largest token is at least 2^7, so at
    most 2^-25 / 2^7 of it per token, N * 2^-32 * max|v| over N tokens;
  * the weights' relative errors from their exponents: a score is a sum of d
    products in fp32 (the tensor cores may truncate: d * 2^-23 of sum |q k|),
    three fp32 multiply-adds and one 2^x (2^-22): (d + 8) * 2^-23 * S * log2 e
    + 2^-20, once in the numerator and once in the denominator, times A.
lse: the same relative error of a weight, plus 2^-21 of its size."""
import math

import pytest
import torch

from block_draft_tree_b200 import api

import q8_ref
from q8_ref import Cache

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _tree_mask(g, b, n, n_nodes):
    see = torch.zeros((b, n, n), dtype=torch.bool)
    for i in range(b):
        for j in range(n_nodes[i]):
            if j:
                see[i, j] = see[i, int(torch.randint(0, j, (1,), generator=g))]
            see[i, j, j] = True
    return see


def _pack(see):
    b, n, _ = see.shape
    w = (n + 31) // 32
    bits = torch.zeros((b, n, w * 32), dtype=torch.long)
    bits[:, :, :n] = see
    words = (bits.view(b, n, w, 32) << torch.arange(32)).sum(-1)
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).int().to(DEV)


class Case:
    def __init__(self, n, hq, hkv, d, block=16, page=0, ctx=(0,), n_nodes=None, seed=0, tokens=None,
                 exps=(-8, -3)):
        g = torch.Generator().manual_seed(seed)
        b = len(ctx)
        tokens = tokens or max(16, max(ctx))
        if page:
            tokens = -(-tokens // page) * page
        self.c = Cache(b, tokens, hkv, d, block, page, seed=seed + 1, exps=exps)
        self.ctx, self.n = list(ctx), n
        self.n_nodes = list(n_nodes) if n_nodes else [n] * b
        bf = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
        self.q, self.kt, self.vt = bf(b, n, hq, d), bf(b, n, hkv, d), bf(b, n, hkv, d)
        self.see = _tree_mask(g, b, n, self.n_nodes)
        self.scale = 1.0 / math.sqrt(d)
        self.max_ctx = tokens

    def run(self, want_lse=True, **kw):
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        return api.tree_attn_q8(self.q, *self.c.args(), self.kt, self.vt, _pack(self.see), _i32(self.n_nodes),
                                _i32(self.ctx), self.max_ctx, scale=self.scale, want_lse=want_lse,
                                dev_status=self.status, **dict(self.c.kw(), **kw))

    def check(self, out, lse, status=0):
        assert int(self.status) == status
        b, n, hq, d = self.q.shape
        g = hq // self.c.hkv
        for i in range(b):
            m, T = self.n_nodes[i], self.ctx[i]
            assert not out[i, m:].any() and (lse[i, m:] == -math.inf).all()
            kv = [self.c.values(w, i, T) for w in range(2)]
            for h in range(self.c.hkv):
                for h0 in range(h * g, h * g + g):
                    step = max(1, (1 << 24) // ((T + m) * d))
                    for j in range(0, m, step):
                        e = min(m, j + step)
                        o, L, A, S = q8_ref.attention(
                            self.q[i, j:e, h0].double(), [x[:, h] for x in kv],
                            [self.kt[i, :m, h].double(), self.vt[i, :m, h].double()],
                            self.see[i, j:e, :m].to(DEV), self.scale)
                        rel = (d + 8) * 2.0 ** -23 * S * 1.4427 + 2.0 ** -20
                        vmax = max([float(x[:, h].abs().nan_to_num(0, 0, 0).max()) for x in (kv[1], self.vt[i, :m].double())
                                    if x.numel()], default=0.0)
                        tol = (o.abs() * 2.0 ** -8 + A * (2.0 ** -11 + 2 * rel[:, None])
                               + (T + m) * 2.0 ** -32 * vmax + 1e-38)
                        got = out[i, j:e, h0].double()
                        fin = torch.isfinite(o)
                        assert torch.equal(fin, torch.isfinite(got)), (i, h0, j)
                        bad = (got - o).abs()[fin] > tol[fin]
                        assert not bad.any(), (i, h0, j, float(((got - o).abs() / tol)[fin].max()))
                        gl = lse[i, j:e, h0].double()
                        none = L == -math.inf
                        assert torch.equal(none, gl == -math.inf)
                        okl = torch.isfinite(L)
                        assert ((gl - L).abs()[okl] <= (rel + L.abs() * 2.0 ** -21)[okl]).all()

    def go(self):
        self.check(*self.run())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 1), (6, 2), (8, 1), (16, 2), (32, 1)])
@pytest.mark.parametrize("page", [0, 64])
def test_decode(d, hq, hkv, page):
    """One row per sequence, contexts from nothing to a few hundred tokens."""
    Case(1, hq, hkv, d, page=page, ctx=(0, 1, 15, 16, 17, 255, 300), seed=hq).go()


@pytest.mark.parametrize("block,page", [(16, 16), (32, 0), (32, 96), (64, 0), (64, 192), (128, 128), (128, 0)])
@pytest.mark.parametrize("n,hq,hkv,d", [(1, 8, 1, 128), (5, 8, 2, 64), (33, 8, 2, 128), (70, 4, 2, 128)])
def test_blocks_and_pages(block, page, n, hq, hkv, d):
    Case(n, hq, hkv, d, block, page, ctx=(130, 129, 1, 511), seed=block + page + n).go()


@pytest.mark.parametrize("n,hq,hkv,d", [
    (9, 4, 1, 64), (2, 6, 2, 128), (16, 2, 2, 128), (17, 1, 1, 64), (31, 3, 1, 128), (32, 4, 4, 64),
    (33, 12, 4, 128), (63, 1, 1, 128), (64, 1, 1, 128), (65, 8, 2, 128), (65, 12, 4, 128), (128, 4, 2, 64),
    (129, 8, 2, 128), (257, 8, 1, 128), (300, 2, 1, 128), (513, 4, 1, 128), (1024, 1, 1, 128), (40, 40, 1, 128)])
def test_trees(n, hq, hkv, d):
    """Trees around the row and mask-word edges, with rows past n_nodes."""
    Case(n, hq, hkv, d, ctx=(200, 0, 64), n_nodes=(n, max(1, n - 1), (n + 1) // 2), seed=n).go()


@pytest.mark.parametrize("n,hq,hkv", [(1, 8, 1), (65, 4, 1), (129, 8, 2)])
def test_long_context(n, hq, hkv):
    """Contexts that are split over many blocks of the device, with odd ends."""
    Case(n, hq, hkv, 128, page=64, ctx=(5003, 8192, 33), seed=n).go()


def test_rows_that_see_nothing():
    for n in (3, 70):
        c = Case(n, 4, 2, 128, ctx=(0, 40), seed=n)
        c.see[0, 2] = False           # no context and no tree row: zeros, lse -inf
        c.see[1, 1] = False           # the context alone
        out, lse = c.run()
        assert not out[0, 2].any() and (lse[0, 2] == -math.inf).all()
        c.check(out, lse)


@pytest.mark.parametrize("n", [1, 9, 70, 140])
def test_garbage_outside_the_context(n):
    """Stray codes and wild exponents past ctx_len, pages that do not exist, NaN
    rows past n_nodes: none of it shows."""
    for page in (0, 64):
        c = Case(n, 8, 2, 128, page=page, ctx=(70, 0), n_nodes=(max(1, n - 1), n), seed=n, tokens=256)
        if n > 1:
            c.kt[0, n - 1:], c.vt[0, n - 1:] = float("nan"), float("inf")
        for i in range(2):
            T = c.ctx[i]
            for w in range(2):
                for t in range(T, 256):
                    at = c.c.place(i, t)
                    c.c.codes[w][at[0], at[1]] = 0x7F if t % 2 else 0xFF
                    if t % 16 == 0 and t >= T:
                        c.c.exps[w][at[0], at[1] // 16] = -128 if (t // 16 + w) % 2 else 127
        if page:
            c.c.page_table[:, 2:] = -1
            c.c.page_table[1] = 1 << 30
        c.go()


@pytest.mark.parametrize("n", [9, 70, 140])
def test_non_finite_tree_rows_reach_only_those_who_see_them(n):
    c = Case(n, 4, 1, 128, ctx=(50, 0), seed=n)
    c.kt[0, 3, 0, 5] = float("nan")
    c.vt[0, 5, 0, 7], c.vt[0, 6, 0, 8] = float("inf"), float("nan")
    c.vt[1, n - 1, 0, 0] = float("-inf")
    c.go()


def test_nan_blocks_and_queries():
    """A block marked as NaN in the context makes every row of its head NaN (K
    or V), a NaN query its own row alone; blocks marked past the context do not
    show (test_garbage_outside_the_context)."""
    for n in (1, 70, 140):
        c = Case(n, 4, 2, 128, ctx=(50, 60, 40), seed=n)
        c.c.exps[0][0, 1, 1] = -128
        c.c.exps[1][2, 2, 0] = -128
        c.q[1, 0, 3, 2] = float("nan")
        out, lse = c.run()
        assert out[0, :, 2:].isnan().all() and lse[0, :, 2:].isnan().all() and not out[0, :, :2].isnan().any()
        assert out[2, :, :2].isnan().all() and not out[2, :, 2:].isnan().any()
        assert out[1, 0, 3].isnan().all() and not out[1, 0, :3].isnan().any()
        assert not out[1, 1:].isnan().any()


@pytest.mark.parametrize("n", [1, 40, 130])
def test_block_scales_far_apart(n):
    """V blocks of very unequal scale, K exponents likewise: every block keeps
    its share (the tolerance is in terms of the row's own weights)."""
    c = Case(n, 8, 1, 128, ctx=(333, 96), seed=n, exps=(-14, -4))
    c.c.exps[1][0, 3:6] = 9
    c.c.exps[1][0, 9] = -40
    c.go()
    c = Case(n, 8, 1, 128, ctx=(64,), seed=n, exps=(-9, -9))
    c.c.exps[1][0, 0] = 40            # a block out of all proportion, with next to no weight
    c.c.codes[0][0, :16] = 0xFE       # its keys: -448 everywhere
    c.q = c.q.abs()
    c.c.exps[0][0, 0] = -3
    out, lse = c.run()
    c.check(out, lse)


def test_outlier_query_channels():
    """One query channel a thousand times the others: the others still count."""
    for n in (1, 70, 140):
        c = Case(n, 8, 1, 128, ctx=(300,), seed=n)
        c.q[..., 7] *= 1000
        c.c.codes[0][..., 7] = 0x08     # small keys there
        c.kt[..., 7] = 2.0 ** -9
        c.go()


def test_spike_and_a_long_flat_tail():
    """One token of weight 1 and thousands of about 2^-12 each that matter together."""
    T = 8192
    for n in (1, 65, 130):
        c = Case(n, 2, 1, 128, ctx=(T,), seed=n, exps=(-9, -9))
        c.q[:] = 0.25
        c.c.codes[0][:] = 0x00
        c.c.codes[0][0, 77] = 0x7E      # 448 * 2^-9 * 0.25 * 128 / sqrt(128) = 2.47... scores
        c.c.exps[0][0, 77 // 16] = -7   # ... times 4
        c.c.codes[1][:] &= 0x7F         # one sign, so that the tail does not cancel
        c.go()


def test_context_lengths_beyond_the_bound_are_clamped():
    c = Case(3, 4, 1, 64, ctx=(64, 20), seed=1)
    out, lse = c.run()
    c.check(out, lse)
    c.ctx = [200, -7]
    o2, l2 = c.run()
    assert int(c.status) == 1
    c.ctx, c.status = [64, 0], torch.zeros(1, dtype=torch.int32, device=DEV)
    c.check(o2, l2)


@pytest.mark.parametrize("n", [1, 70])
def test_missing_pages_are_reported(n):
    c = Case(n, 4, 1, 128, page=64, ctx=(130, 100), seed=2)
    c.c.page_table[0, 1] = -1
    out, lse = c.run()
    assert int(c.status) == 1
    c.ctx[0], c.status = 0, torch.zeros(1, dtype=torch.int32, device=DEV)
    out[0], lse[0] = c.run()[0][0], c.run()[1][0]   # the other sequence is as it should be
    c.check(out, lse)


def test_agrees_with_the_bf16_attention_over_the_read_back_cache():
    """The framework's own bf16 attention over what kv_read_q8 returns: the
    same function of the same values (its weights are bf16: 2^-8 each)."""
    for n, hq, hkv in ((1, 8, 1), (65, 8, 2), (130, 4, 1)):
        c = Case(n, hq, hkv, 128, ctx=(500, 77), seed=n)
        out, lse = c.run()
        k, v = api.kv_read_q8(*c.c.args(), _i32(c.ctx), 500, **c.c.kw())
        ref, l2 = api.tree_attn(c.q, k, v, c.kt, c.vt, _pack(c.see), _i32(c.n_nodes), _i32(c.ctx), 500,
                                scale=c.scale, want_lse=True)
        assert (out.float() - ref.float()).abs().max() <= 2e-2 * max(1.0, float(ref.float().abs().max()))
        assert (lse - l2).abs().max() <= 1e-3


@pytest.mark.parametrize("n", [1, 70])
def test_two_streams_and_two_graphs_at_once(n):
    """Calls in flight together, eager and captured, each with its own scratch."""
    cs = [Case(n, 8, 1, 128, ctx=(4096,), seed=s) for s in (1, 2)]
    masks = [_pack(c.see) for c in cs]
    nn, cl = [_i32(c.n_nodes) for c in cs], [_i32(c.ctx) for c in cs]

    def call(i):
        c = cs[i]
        return api.tree_attn_q8(c.q, *c.c.args(), c.kt, c.vt, masks[i], nn[i], cl[i], 4096, **c.c.kw())

    want = [call(0).clone(), call(1).clone()]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(i))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(4)]
    eager = [None, None]
    for r in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
            with torch.cuda.stream(streams[2 + i]):
                eager[i] = call(i)
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i], want[i]) and torch.equal(eager[i], want[i])


@pytest.mark.parametrize("n,hq,hkv,d", [(3, 8, 1, 128), (3, 8, 1, 64), (1, 17, 1, 128), (33, 1, 1, 128), (8, 4, 1, 64)])
def test_row_tiles(n, hq, hkv, d):
    """Three tiles of 8 rows, and the last row beyond a tile."""
    Case(n, hq, hkv, d, ctx=(100, 31), seed=n + hq).go()


@pytest.mark.parametrize("n,hq", [(1, 8), (70, 1)])
@pytest.mark.parametrize("page", [0, 16, 48])
def test_small_and_odd_caches(n, hq, page):
    """Caches shorter than a tile's box, lengths that are no multiple of the
    block, pages that are no power of two and no multiple of a step."""
    for tokens in (1, 5, 17, 100):
        Case(n, hq, 1, 128, page=page, ctx=(tokens, tokens // 2), seed=tokens, tokens=tokens).go()


@pytest.mark.parametrize("n,hq,batch", [(1, 2, 300), (40, 1, 300), (40, 1, 37)])
def test_many_ragged_sequences(n, hq, batch):
    """More sequences than are sorted by length, and fewer; equal lengths among them."""
    Case(n, hq, 1, 128, page=64, ctx=[(i * 37) % 201 for i in range(batch)], seed=batch).go()


def test_no_cache_at_all():
    """max_ctx 0: the tree alone, whatever the cache's size."""
    for n in (4, 70):
        c = Case(n, 4, 2, 128, ctx=(0, 0), seed=n)
        c.max_ctx = 0
        c.go()
        empty = torch.empty((2, 0, 2, 128), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
        exps = torch.empty((2, 0, 2), dtype=torch.int8, device=DEV)
        out = api.tree_attn_q8(c.q, empty, empty, exps, exps, c.kt, c.vt, _pack(c.see), _i32(c.n_nodes), _i32(c.ctx), 0)
        assert torch.equal(out, c.run()[0])


def test_repeated_calls_agree_to_the_bit():
    """No result depends on the order in which blocks run."""
    for n in (1, 40, 140):
        c = Case(n, 8, 2, 128, page=64, ctx=(3000, 50, 1111), seed=n)
        first = c.run()
        for _ in range(5):
            again = c.run()
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("n,page", [(1, 0), (1, 48), (70, 0), (140, 64)])
def test_waits_that_run_out_are_reported(n, page):
    """With a bound of a few cycles the kernels' waits give up: the status says
    so, and the next call with the default bound is right.  (The kernel for few
    rows waits for copies that may have landed when it first looks.)"""
    c = Case(n, 8, 1, 128, page=page, ctx=(2000, 900), seed=n)
    api.set_wait_limit(4)
    try:
        c.run()
        torch.cuda.synchronize()
        assert int(c.status) == 5 or (n == 1 and int(c.status) == 0)
    finally:
        api.set_wait_limit(0)
    c.go()


def test_nan_codes_in_the_context():
    """A NaN code that someone else wrote: in K every row of its head is NaN, in
    V that one column."""
    for n in (1, 70, 140):
        c = Case(n, 4, 2, 128, ctx=(50, 60), seed=n)
        c.c.codes[0][0, 17, 1, 3] = 0x7F
        c.c.codes[1][1, 18, 0, 4] = 0xFF
        out, _ = c.run()
        assert out[0, :, 2:].isnan().all() and not out[0, :, :2].isnan().any()
        assert out[1, :, :2, 4].isnan().all() and out[1].isnan().sum() == n * 2
