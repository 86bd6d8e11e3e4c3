"""The 8-bit cache's calls without a GPU: what the C ABI and the binding
refuse before any launch, and the tests' reference against torch's own e4m3."""
import ctypes

import pytest
import torch

from block_draft_tree_b200 import api, build

import q8_ref


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load_library()


def _cache(**kw):
    base = dict(k_cache=256, v_cache=256, k_exp=256, v_exp=256, page_table=None, block=16,
                page_size=0, max_pages=0, num_pages=0, t_max=128, hkv=2, d=64)
    return api.Q8Cache(**dict(base, **kw))


PAGED = dict(page_table=256, page_size=64, max_pages=2, num_pages=4, t_max=0)


def _cache_refusals(call):
    assert call(_cache(d=96)) == 2 and call(_cache(d=0)) == 2
    assert call(_cache(hkv=0)) == 1
    for block in (0, 8, 24, 256, -16):
        assert call(_cache(block=block)) == 2
    for name in ("k_cache", "v_cache", "k_exp", "v_exp"):
        assert call(_cache(**{name: None})) == 1, name
    assert call(_cache(k_cache=264)) == 1          # misaligned
    assert call(_cache(t_max=0)) == 1
    assert call(_cache(**dict(PAGED, block=128))) == 2   # a page of half a block
    assert call(_cache(**dict(PAGED, page_size=0))) == 1
    assert call(_cache(**dict(PAGED, max_pages=0))) == 1
    assert call(_cache(**dict(PAGED, num_pages=0))) == 1


def test_append_rejects_bad_arguments(lib):
    def call(cache=None, **kw):
        a = dict(k_new=256, v_new=256, n_new=None, ctx_len=256, ctx_len_out=None, batch=1, n_max=4,
                 dev_status=None)
        a = api.KVAppendQ8Args(cache=_cache() if cache is None else cache, **dict(a, **kw))
        return lib.ddt_kv_append_q8(ctypes.byref(a), None)

    _cache_refusals(lambda c: call(c))
    assert call(batch=-1) == 1 and call(n_max=-1) == 1 and call(batch=65536) == 2
    assert call(k_new=None) == 1 and call(v_new=None) == 1 and call(ctx_len=None) == 1
    assert call(k_new=258) == 1
    assert call(batch=0) == 0
    assert lib.ddt_kv_append_q8(None, None) == 1


def test_commit_rejects_bad_arguments(lib):
    def call(cache=None, **kw):
        a = dict(k_tree=256, v_tree=256, acc_len=256, acc_nodes=256, ctx_len=256, ctx_len_out=None,
                 batch=1, n_max=4, L=4, dev_status=None)
        a = api.KVCommitQ8Args(cache=_cache() if cache is None else cache, **dict(a, **kw))
        return lib.ddt_kv_commit_q8(ctypes.byref(a), None)

    _cache_refusals(lambda c: call(c))
    assert call(L=65) == 2 and call(L=-1) == 1 and call(n_max=0) == 1 and call(batch=65536) == 2
    for name in ("k_tree", "v_tree", "acc_len", "acc_nodes", "ctx_len"):
        assert call(**{name: None}) == 1, name
    assert call(v_tree=264) == 1
    assert call(batch=0) == 0
    assert lib.ddt_kv_commit_q8(None, None) == 1


def test_read_rejects_bad_arguments(lib):
    def call(cache=None, **kw):
        a = dict(ctx_len=256, first=None, k_out=256, v_out=256, batch=1, n_max=4, dev_status=None)
        a = api.KVReadQ8Args(cache=_cache() if cache is None else cache, **dict(a, **kw))
        return lib.ddt_kv_read_q8(ctypes.byref(a), None)

    _cache_refusals(lambda c: call(c))
    assert call(n_max=-1) == 1 and call(batch=-1) == 1 and call(batch=65536) == 2
    for name in ("ctx_len", "k_out", "v_out"):
        assert call(**{name: None}) == 1, name
    assert call(k_out=8) == 1
    assert call(n_max=0) == 0 and call(batch=0) == 0
    assert lib.ddt_kv_read_q8(None, None) == 1


def test_attn_rejects_bad_arguments(lib):
    def call(cache=None, **kw):
        a = dict(q=256, ctx_len=256, max_ctx=100, k_tree=256, v_tree=256, mask=256, n_nodes=256,
                 batch=1, n_max=9, hq=4, scale=0.125, out=256, lse_out=None, dev_status=None)
        a = api.AttnQ8Args(cache=_cache() if cache is None else cache, **dict(a, **kw))
        return lib.ddt_tree_attn_q8(ctypes.byref(a), None, 0, None)

    _cache_refusals(lambda c: call(c))
    assert call(hq=5) == 1 and call(hq=0) == 1 and call(n_max=0) == 1 and call(n_max=1025) == 2
    assert call(scale=0.0) == 1 and call(scale=float("nan")) == 1 and call(scale=float("inf")) == 1
    assert call(max_ctx=-1) == 1 and call(max_ctx=129) == 1     # beyond t_max
    assert call(_cache(**PAGED), max_ctx=129) == 1              # beyond the page table
    for name in ("q", "ctx_len", "k_tree", "v_tree", "mask", "n_nodes", "out"):
        assert call(**{name: None}) == 1, name
    assert call(q=264) == 1 and call(out=8) == 1
    assert call(batch=40000) == 2                               # batch * hkv beyond the grid
    assert call(batch=0) == 0
    big = dict(max_ctx=8192)
    assert call(_cache(t_max=8192), **big) == 3                 # needs a workspace, none given
    assert lib.ddt_tree_attn_q8(None, None, 0, None) == 1


def _tensors(device="cpu", hkv=2, d=64, t=64, b=2, n=3, block=16):
    f8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)  # noqa: E731
    x = {"k_cache": f8(b, t, hkv, d), "v_cache": f8(b, t, hkv, d),
         "k_exp": torch.zeros((b, -(-t // block), hkv), dtype=torch.int8, device=device),
         "ctx_len": torch.zeros(b, dtype=torch.int32, device=device)}
    x["v_exp"] = x["k_exp"].clone()
    rows = torch.zeros((b, n, hkv, d), dtype=torch.bfloat16, device=device)
    return x, rows


def test_binding_refuses_mismatched_tensors(lib):
    """Every refusal comes before the device check, so CPU tensors reach it."""
    x, rows = _tensors()
    bad = [("k_cache", x["k_cache"].view(torch.uint8), "float8_e4m3fn"),
           ("v_cache", x["v_cache"][:, :32], "shape"),
           ("k_exp", x["k_exp"][:, :2].contiguous(), "exponents"),
           ("v_exp", x["v_exp"].int(), "int8"),
           ("ctx_len", x["ctx_len"].long(), "ctx_len"),
           ("ctx_len", x["ctx_len"][:1], "ctx_len")]
    q = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16)
    mask, nn = torch.zeros((2, 3, 1), dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    acc, nodes = torch.zeros(2, dtype=torch.int32), torch.zeros((2, 4), dtype=torch.int32)

    def calls(y):
        c = (y["k_cache"], y["v_cache"], y["k_exp"], y["v_exp"])
        return [lambda: api.kv_append_q8(rows, rows, y["ctx_len"], *c),
                lambda: api.kv_commit_q8(rows, rows, acc, nodes, y["ctx_len"], *c),
                lambda: api.tree_attn_q8(q, *c, rows, rows, mask, nn, y["ctx_len"], 64),
                lambda: api.kv_read_q8(*c, y["ctx_len"], 4)]

    for name, t, word in bad:
        for i, f in enumerate(calls(dict(x, **{name: t}))):
            if i == 3 and name == "ctx_len" and t.dtype == torch.int32:
                word = "sequences"  # kv_read_q8 takes its batch from ctx_len
            with pytest.raises(api.DDTError, match=word):
                f()
    c = (x["k_cache"], x["v_cache"], x["k_exp"], x["v_exp"])
    for f in calls(x):
        with pytest.raises(api.DDTError, match="CUDA tensors only"):
            f()
    for kw in (dict(block=24), dict(block=32), dict(n_new=acc.long()),
               dict(page_table=torch.zeros((2, 1), dtype=torch.int64)),
               dict(page_table=torch.zeros((1, 1), dtype=torch.int32))):
        with pytest.raises(api.DDTError):
            api.kv_append_q8(rows, rows, x["ctx_len"], *c, **kw)
    with pytest.raises(api.DDTError, match="contiguous"):
        api.kv_append_q8(rows.transpose(0, 1).contiguous().transpose(0, 1), rows, x["ctx_len"], *c)
    with pytest.raises(api.DDTError, match="rows must be"):
        api.kv_append_q8(rows[:, :, :1], rows[:, :, :1], x["ctx_len"], *c)
    with pytest.raises(api.DDTError, match="acc_nodes"):
        api.kv_commit_q8(rows, rows, acc, nodes[:1], x["ctx_len"], *c)
    with pytest.raises(api.DDTError, match="mask"):
        api.tree_attn_q8(q, *c, rows, rows, mask[:, :2], nn, x["ctx_len"], 64)
    with pytest.raises(api.DDTError, match="tree K"):
        api.tree_attn_q8(q[:, :2].contiguous(), *c, rows, rows, mask, nn, x["ctx_len"], 64)
    with pytest.raises(api.DDTError, match="n_max"):
        api.kv_read_q8(*c, x["ctx_len"], -1)


def test_structures_match_the_header(lib):
    """The argument structures have the sizes that the header's layout gives."""
    assert ctypes.sizeof(api.Q8Cache) == 72
    assert ctypes.sizeof(api.KVAppendQ8Args) == 72 + 5 * 8 + 2 * 4 + 8
    assert ctypes.sizeof(api.KVCommitQ8Args) == 72 + 6 * 8 + 3 * 4 + 4 + 8
    assert ctypes.sizeof(api.KVReadQ8Args) == 72 + 4 * 8 + 2 * 4 + 8
    assert ctypes.sizeof(api.AttnQ8Args) == 72 + 2 * 8 + 8 + 4 * 8 + 3 * 4 + 4 + 3 * 8


def test_reference_codes_are_torchs_e4m3():
    """The reference's decoder and rounding against torch.float8_e4m3fn: every
    code, and values on, between and halfway between codes."""
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double()
    got = q8_ref.decode(codes)
    assert torch.equal(got.nan_to_num(1e9), want.nan_to_num(1e9)) and want.isnan().sum() == 2
    v = q8_ref.code_values()[:127]
    mid = (v[1:] + v[:-1]) / 2
    y = torch.cat([v, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20)])
    y = torch.cat([y, -y])
    ref = y.float().to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(q8_ref.encode(y), ref)
    assert q8_ref.needed_exp(448.0) == 0 and q8_ref.needed_exp(448.5) == 1
    assert q8_ref.needed_exp(0.0) == -48 and q8_ref.needed_exp(1e30) == 48
