"""Writing the 8-bit key/value cache (prompts, tokens, accepted rows) and
reading it back, against the plain reference: codes, exponents, lengths and
every byte that must stay as it was are compared exactly."""
import pytest
import torch

from block_draft_tree_b200 import api

from q8_ref import Cache

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _rows(seed, shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp(2.0 * torch.randn(shape[:2] + (1, 1), generator=g))
    return (x * scale).to(torch.bfloat16).to(DEV)


def _status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _check(got: Cache, want: Cache):
    for w in range(2):
        assert torch.equal(got.codes[w], want.codes[w]), "codes of %s" % "KV"[w]
        assert torch.equal(got.exps[w], want.exps[w]), "exponents of %s" % "KV"[w]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("block,page", [(16, 0), (16, 64), (32, 32), (64, 0), (64, 192), (128, 128), (128, 0)])
@pytest.mark.parametrize("hkv", [1, 3, 8])
def test_append(d, block, page, hkv):
    """Rows behind contexts that end anywhere in a block: none, one, part of a
    block, several blocks; block scales that stay and that grow."""
    ctx = [0, 1, block - 1, block, 2 * block + 5, 37]
    n = [1, 3 * block + 7, 2, 0, block, 5]
    b, n_max = len(ctx), max(n)
    c = Cache(b, 6 * block + 32 if not page else -(-(6 * block + 32) // page) * page, hkv, d, block, page,
              seed=d + block + hkv)
    k, v = _rows(1, (b, n_max, hkv, d)), _rows(2, (b, n_max, hkv, d), 1e-3)
    want = c.clone()
    for i in range(b):
        want.append(i, ctx[i], k[i, :n[i]], v[i, :n[i]])
    st, cl = _status(), _i32(ctx)
    api.kv_append_q8(k, v, cl, *c.args(), n_new=_i32(n), dev_status=st, **c.kw())
    assert cl.tolist() == [x + y for x, y in zip(ctx, n)] and int(st) == 0
    _check(c, want)
    # again without advancing: the same rows at the same places change nothing more
    api.kv_append_q8(k, v, _i32(ctx), *c.args(), n_new=_i32(n), advance=False, **c.kw())
    _check(c, want)


def test_append_token_by_token_equals_the_reference():
    """A block filled one token at a time, with scales that grow on the way."""
    c = Cache(2, 48, 2, 128, 16, seed=3)
    want = c.clone()
    cl = _i32([0, 7])
    k, v = _rows(5, (2, 36, 2, 128)), _rows(6, (2, 36, 2, 128))
    for t in range(36):
        kt, vt = k[:, t:t + 1].contiguous(), v[:, t:t + 1].contiguous()
        api.kv_append_q8(kt, vt, cl, *c.args(), **c.kw())
        for i, c0 in ((0, 0), (1, 7)):
            want.append(i, c0 + t, kt[i], vt[i])
    assert cl.tolist() == [36, 43]
    _check(c, want)


def test_append_values_at_the_edges():
    """Zeros, subnormals, the largest magnitudes, infinities and NaN."""
    d, block = 64, 16
    c = Cache(8, 32, 1, d, block, seed=4)
    k = torch.zeros((8, 16, 1, d), device=DEV)
    k[1] = 1e-40                       # bf16 subnormals
    k[2] = 3e38                        # beyond 448 * 2^48: saturates
    k[3, 0, 0, 0], k[3, 1, 0, 1] = 448.0, -448.0
    k[4, 0, 0, 0], k[4, 1, 0, 1] = 450.0, 1.0
    k[5, 0, 0, 0], k[5, 1, 0, 1], k[5, 2, 0, 2] = float("inf"), float("-inf"), 2.0
    k[6, 0, 0, 0], k[6, 1] = float("nan"), 3.0
    k[7] = float("nan")
    k = k.to(torch.bfloat16)
    v = k.flip(0).contiguous()
    want = c.clone()
    for i in range(8):
        want.append(i, 0, k[i], v[i])
    api.kv_append_q8(k, v, _i32([0] * 8), *c.args(), **c.kw())
    _check(c, want)
    assert c.exps[0][:, 0, 0].tolist() == [-48, -48, 48, 0, 1, -128, -128, -128]
    # a marked block stays marked while it fills, and reads as NaN; the next block is clean
    ones = torch.ones((8, 3, 1, d), dtype=torch.bfloat16, device=DEV)
    for i in range(8):
        want.append(i, 15, ones[i], ones[i])
    api.kv_append_q8(ones, ones, _i32([15] * 8), *c.args(), **c.kw())
    _check(c, want)
    assert c.exps[0][:, 0, 0].tolist()[5:] == [-128] * 3 and c.exps[0][:, 1, 0].tolist() == [-8] * 8
    kr, _ = api.kv_read_q8(*c.args(), _i32([18] * 8), 18, **c.kw())
    assert kr[5:, :16].isnan().all() and (kr[:, 16:] == 1).all()
    # filled again from its beginning, it is clean
    api.kv_append_q8(ones, ones, _i32([0] * 8), *c.args(), **c.kw())
    assert c.exps[0][:, 0, 0].tolist() == [-8] * 8


def test_append_out_of_range_is_reported_and_nothing_else_written():
    block, d = 16, 64
    for page in (0, 32):
        c = Cache(4, 64, 2, d, block, page, seed=5)
        if page:
            c.page_table[2, 1] = -1                        # position 32.. of sequence 2 has no page
            c.page_table[3, 1] = c.codes[0].shape[0]       # beyond the pool
        ctx, n = [60, 0, 30, 30], [10, 12, 4, 4]
        k, v = _rows(7, (4, 12, 2, d)), _rows(8, (4, 12, 2, d))
        want = c.clone()
        for i in range(4):
            want.append(i, ctx[i], k[i, :n[i]], v[i, :n[i]])
        st, cl = _status(), _i32(ctx)
        api.kv_append_q8(k, v, cl, *c.args(), n_new=_i32(n), dev_status=st, **c.kw())
        assert int(st) == 1 and cl.tolist() == [70, 12, 34, 34]
        _check(c, want)
    # device lengths out of range: clamped, or nothing written
    c = Cache(3, 64, 2, d, block, seed=6)
    want = c.clone()
    k, v = _rows(9, (3, 4, 2, d)), _rows(10, (3, 4, 2, d))
    want.append(1, 5, k[1], v[1])
    st = _status()
    api.kv_append_q8(k, v, _i32([-3, 5, 2]), *c.args(), n_new=_i32([4, 9, -1]), dev_status=st,
                     advance=False, **c.kw())
    assert int(st) == 1
    _check(c, want)
    # a context already past a dense cache whose length is no multiple of the block
    c = Cache(1, 40, 2, d, 32, seed=7)
    want = c.clone()
    st = _status()
    api.kv_append_q8(k[:1].contiguous(), v[:1].contiguous(), _i32([44]), *c.args(), dev_status=st, **c.kw())
    assert int(st) == 1
    _check(c, want)


def test_empty_calls():
    c = Cache(2, 32, 2, 64, 16, seed=8)
    want = c.clone()
    k = torch.empty((2, 0, 2, 64), dtype=torch.bfloat16, device=DEV)
    cl = _i32([3, 4])
    api.kv_append_q8(k, k, cl, *c.args(), **c.kw())
    assert cl.tolist() == [3, 4]
    kr, vr = api.kv_read_q8(*c.args(), cl, 0, **c.kw())
    assert kr.shape == (2, 0, 2, 64)
    e = Cache(0, 32, 2, 64, 16, seed=8)
    api.kv_append_q8(k[:0], k[:0], cl[:0], *e.args(), **e.kw())
    assert api.kv_read_q8(*e.args(), cl[:0], 3, **e.kw())[0].shape == (0, 3, 2, 64)
    torch.cuda.synchronize()
    _check(c, want)


@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("d,hkv,L,n_max", [(64, 1, 4, 9), (128, 8, 16, 65), (128, 2, 64, 129)])
def test_commit(page, d, hkv, L, n_max):
    b = 5
    c = Cache(b, 256, hkv, d, 16, page, seed=L)
    g = torch.Generator().manual_seed(L)
    ctx = [0, 15, 16, 100, 187 - L]
    acc = [0, min(L, n_max - 1), 1, min(3, L), min(L, n_max - 1)]
    nodes = torch.full((b, L), -1, dtype=torch.int32)
    for i in range(b):
        nodes[i, :acc[i]] = torch.sort(torch.randperm(n_max - 1, generator=g)[:acc[i]]).values.int() + 1
    nodes[3, 1] = nodes[3, 0]                                 # the same row twice
    kt, vt = _rows(11, (b, n_max, hkv, d)), _rows(12, (b, n_max, hkv, d))
    want = c.clone()
    for i in range(b):
        rows = [0] + nodes[i, :acc[i]].tolist()
        want.append(i, ctx[i], kt[i, rows], vt[i, rows])
    st, cl = _status(), _i32(ctx)
    api.kv_commit_q8(kt, vt, _i32(acc), nodes.to(DEV), cl, *c.args(), dev_status=st, **c.kw())
    assert int(st) == 0 and cl.tolist() == [x + y + 1 for x, y in zip(ctx, acc)]
    _check(c, want)


def test_commit_reports_bad_rows():
    b, L, d = 3, 4, 64
    c = Cache(b, 64, 2, d, 16, seed=9)
    kt, vt = _rows(13, (b, 9, 2, d)), _rows(14, (b, 9, 2, d))
    want = c.clone()
    want.append(0, 3, kt[0, [0, 2]], vt[0, [0, 2]])
    want.append(1, 8, kt[1, :1], vt[1, :1])                   # acc_len -2 counts as 0
    want.append(2, 0, kt[2, [0, 1, 2, 3, 4]], vt[2, [0, 1, 2, 3, 4]])
    st = _status()
    nodes = torch.tensor([[2, 9, -1, -1], [-1] * 4, [1, 2, 3, 4]], dtype=torch.int32, device=DEV)
    api.kv_commit_q8(kt, vt, _i32([2, -2, 7]), nodes, _i32([3, 8, 0]), *c.args(), dev_status=st,
                     advance=False, **c.kw())
    assert int(st) == 1
    _check(c, want)


@pytest.mark.parametrize("d,hkv", [(64, 1), (128, 3), (128, 8)])
@pytest.mark.parametrize("block,page", [(16, 0), (64, 64), (32, 96), (128, 0)])
def test_read(d, hkv, block, page):
    """Any range of any length; rows past the context are 0; exponents out of
    range are read as the nearer end."""
    tokens = 300 if not page else -(-300 // page) * page
    c = Cache(4, tokens, hkv, d, block, page, seed=d + block, exps=(-60, 60))
    ctx, first, n_max = [300, 0, 131, 17], [0, 0, 50, 200], 257
    st = _status()
    k, v = api.kv_read_q8(*c.args(), _i32(ctx), n_max, first=_i32(first), dev_status=st, **c.kw())
    assert int(st) == 0
    for w, got in ((0, k), (1, v)):
        for i in range(4):
            want = torch.zeros((n_max, hkv, d), dtype=torch.float64, device=DEV)
            x = c.values(w, i, ctx[i])[first[i]:first[i] + n_max]
            want[:x.shape[0]] = x
            assert torch.equal(got[i].double(), want)         # every value is a bf16 number
    if page == 0:
        k0, _ = api.kv_read_q8(*c.args(), _i32([300] * 4), 300, **c.kw())
        assert torch.equal(k0[2].double(), c.values(0, 2, 300))


def test_read_reports_positions_outside():
    c = Cache(3, 64, 2, 64, 16, 32, seed=10)
    c.page_table[1, 1] = 1 << 20
    st = _status()
    k, v = api.kv_read_q8(*c.args(), _i32([64, 64, 200]), 100, dev_status=st, **c.kw())
    assert int(st) == 1
    assert torch.equal(k[0, :64].double(), c.values(0, 0, 64))
    assert torch.equal(v[1, :32].double(), c.values(1, 1, 32)) and not k[1, 32:].any()
    assert torch.equal(k[2, :64].double(), c.values(0, 2, 64)) and not k[2, 64:].any()
    st = _status()
    k, _ = api.kv_read_q8(*c.args(), _i32([5, 5, 5]), 4, first=_i32([-2, 0, 1]), dev_status=st, **c.kw())
    assert int(st) == 1
    assert not k[0, :2].any() and torch.equal(k[0, 2:].double(), c.values(0, 0, 2))


def test_far_offsets():
    """A pool of more than 2^32 codes: the last pages are written, read and
    attended where they are, and the first pages stay as they were."""
    hkv, d, page, block = 8, 128, 64, 64
    pages = (1 << 32) // (page * hkv * d) + 40
    k8 = torch.zeros((pages, page, hkv, d), dtype=torch.uint8, device=DEV)
    c = Cache(1, 128, hkv, d, block, page, seed=11)
    c.codes = [k8, torch.zeros_like(k8)]
    c.exps = [torch.full((pages, 1, hkv), -7, dtype=torch.int8, device=DEV) for _ in range(2)]
    c.page_table = _i32([[pages - 1, pages - 9]])
    k, v = _rows(15, (1, 100, hkv, d)), _rows(16, (1, 100, hkv, d))
    cl = _i32([0])
    api.kv_append_q8(k, v, cl, *c.args(), **c.kw())
    kr, vr = api.kv_read_q8(*c.args(), cl, 100, **c.kw())
    small = Cache(1, 128, hkv, d, block, page, seed=11)
    small.append(0, 0, k[0], v[0])
    assert torch.equal(kr[0].double(), small.values(0, 0, 100))
    assert torch.equal(vr[0].double(), small.values(1, 0, 100))
    assert not k8[:pages - 9].any() and not k8[pages - 8:pages - 1].any()
    q = torch.randn((1, 1, 32, d), device=DEV).to(torch.bfloat16)
    kt, vt = _rows(17, (1, 1, hkv, d)), _rows(18, (1, 1, hkv, d))
    m = torch.ones((1, 1, 1), dtype=torch.int32, device=DEV)
    far = api.tree_attn_q8(q, *c.args(), kt, vt, m, _i32([1]), cl, 128, **c.kw())
    near = api.tree_attn_q8(q, *small.args(), kt, vt, m, _i32([1]), cl, 128, **small.kw())
    assert torch.equal(far, near)


def test_far_dense_offsets():
    """Dense caches of more than 2^31 tokens x heads x d: the last sequence."""
    hkv, d, t = 8, 128, 1 << 16
    b = (1 << 31) // (t * hkv * d) + 2
    k8 = torch.zeros((b, t, hkv, d), dtype=torch.uint8, device=DEV)
    c = Cache(1, 64, hkv, d, 16, seed=12)
    c.codes = [k8, torch.zeros_like(k8)]
    c.exps = [torch.full((b, t // 16, hkv), -7, dtype=torch.int8, device=DEV) for _ in range(2)]
    n = torch.zeros(b, dtype=torch.int32, device=DEV)
    n[-1] = 20
    ctx = torch.full((b,), t - 20, dtype=torch.int32, device=DEV)
    k, v = _rows(19, (1, 20, hkv, d)), _rows(20, (1, 20, hkv, d))
    api.kv_append_q8(k.expand(b, -1, -1, -1).contiguous(), v.expand(b, -1, -1, -1).contiguous(), ctx, *c.args(),
                     n_new=n, **c.kw())
    first = torch.full((b,), t - 20, dtype=torch.int32, device=DEV)
    kr, vr = api.kv_read_q8(*c.args(), ctx, 20, first=first, **c.kw())
    small = Cache(1, 48, hkv, d, 16, seed=12)
    small.codes = [torch.zeros_like(x) for x in small.codes]
    small.exps = [torch.full_like(x, -7) for x in small.exps]
    small.append(0, 12, k[0], v[0])  # t - 20 is 12 in its block
    assert torch.equal(kr[-1].double(), small.values(0, 0, 32)[12:])
    assert torch.equal(vr[-1].double(), small.values(1, 0, 32)[12:])
    assert not kr[:-1].any()


def test_calls_on_a_side_stream_and_in_a_graph():
    """A captured append + read, replayed: each replay appends behind the last."""
    c = Cache(2, 128, 2, 64, 16, seed=13)
    want = c.clone()
    k, v = _rows(21, (2, 5, 2, 64)), _rows(22, (2, 5, 2, 64))
    cl = _i32([0, 9])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        api.kv_append_q8(k, v, cl, *c.args(), **c.kw())
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.kv_append_q8(k, v, cl, *c.args(), **c.kw())
        kr, vr = api.kv_read_q8(*c.args(), cl, 64, **c.kw())
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for r in range(4):
        for i, c0 in ((0, 0), (1, 9)):
            want.append(i, c0 + 5 * r, k[i], v[i])
    assert cl.tolist() == [20, 29]
    _check(c, want)
    assert torch.equal(kr[1, :29].double(), want.values(0, 1, 29)) and not vr[1, 29:].any()
