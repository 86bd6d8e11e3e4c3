"""Measured cases of the 8-bit key/value cache: writing it, reading it back, attending to it.

The cache holds e4m3 codes with one power-of-two scale 2^e for every block of
``block`` tokens of every kv head, K and V apart: value = code * 2^e.

* ``append`` / ``commit``: new K/V rows (a prompt, a token, or the accepted rows
  of a draft tree) are quantised into the cache behind the tokens that are
  there.  A block that had tokens keeps the larger of its exponent and the one
  that its new rows need, and its older codes are rounded again where it grows.
  The pass then reads the touched blocks back, so its outputs are the values
  that the cache stands for, with the exponents.
* ``read``: a range of positions of every sequence, as bf16 rows.
* ``attn``: attention of the draft tree's rows (one row: an ordinary decoding
  step) over the 8-bit context and the tree's own bf16 K/V under the ancestor
  mask.

``run`` computes the plain form with elementary torch operations in 32 bits, or
makes the framework's calls where ``own`` is true.
"""
import math

import torch

own = False

E_MIN, E_MAX = -48, 48        # range of the block exponents
Q_MAX = 448.0                 # largest e4m3 value


def listed():
    return [
        # one decoding step's token of one sequence: nothing but latency
        {"name": "append one token", "op": "append", "batch": 1, "n_max": 1, "n_min": 1,
         "ctx": 4099, "ctx_min": 4099, "hkv": 8, "d": 128, "block": 16, "page": 0},
        # after a verification round: a batch's accepted rows into 64-token pages
        {"name": "commit, 32 ragged paged", "op": "commit", "batch": 32, "n_max": 129, "L": 16,
         "ctx": 32768, "ctx_min": 1024, "hkv": 8, "d": 128, "block": 16, "page": 64},
        # whole ragged prompts into empty caches, one scale per page
        {"name": "append prompts to 8192", "op": "append", "batch": 4, "n_max": 8192, "n_min": 5003,
         "ctx": 0, "ctx_min": 0, "hkv": 8, "d": 128, "block": 64, "page": 64},
        # a short context of a small model, read back
        {"name": "read 509 tokens", "op": "read", "batch": 1, "n_max": 509, "ctx": 509,
         "ctx_min": 509, "first": 0, "hkv": 1, "d": 64, "block": 16, "page": 0},
        # a batch's whole paged contexts back to bf16 (moving sequences to another server)
        {"name": "read 8 ragged paged", "op": "read", "batch": 8, "n_max": 32768, "ctx": 32768,
         "ctx_min": 1024, "first": 0, "hkv": 8, "d": 128, "block": 16, "page": 64},
        # the smallest round: 9 tree rows, 4 heads over 1, d = 64
        {"name": "tree 9 rows, d 64", "op": "attn", "batch": 1, "n_max": 9, "ctx": 128,
         "ctx_min": 128, "hq": 4, "hkv": 1, "d": 64, "block": 16, "page": 0},
        # one token of one sequence
        {"name": "decode 1 x 4096", "op": "attn", "batch": 1, "n_max": 1, "ctx": 4096,
         "ctx_min": 4096, "hq": 32, "hkv": 8, "d": 128, "block": 16, "page": 0},
        # serving: one token of each of 32 ragged sequences in 64-token pages
        {"name": "decode 32 ragged paged", "op": "attn", "batch": 32, "n_max": 1, "ctx": 32768,
         "ctx_min": 1024, "hq": 32, "hkv": 8, "d": 128, "block": 16, "page": 64},
        # long contexts, one kv head for all query heads
        {"name": "decode 4 x 131072", "op": "attn", "batch": 4, "n_max": 1, "ctx": 131072,
         "ctx_min": 131072, "hq": 16, "hkv": 1, "d": 128, "block": 64, "page": 0},
        # a draft tree of 64 nodes and its root
        {"name": "tree 65 rows x 4096", "op": "attn", "batch": 1, "n_max": 65, "ctx": 4096,
         "ctx_min": 4096, "hq": 32, "hkv": 8, "d": 128, "block": 16, "page": 0},
        # large trees of a batch
        {"name": "tree 8 x 257 rows x 8192", "op": "attn", "batch": 8, "n_max": 257, "ctx": 8192,
         "ctx_min": 8192, "hq": 64, "hkv": 8, "d": 128, "block": 16, "page": 0},
        # a ragged batch's trees over pages, one scale per page
        {"name": "tree 16 x 129 ragged paged", "op": "attn", "batch": 16, "n_max": 129,
         "ctx": 16384, "ctx_min": 1024, "hq": 32, "hkv": 8, "d": 128, "block": 64, "page": 64},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "commit", "read", "attn", "attn", "attn"])
    c = {"op": op, "batch": _log(rng, 1, 32), "hkv": rng.choice([1, 2, 4, 8]),
         "d": rng.choice([64, 128, 128]), "block": rng.choice([16, 16, 32, 64, 128])}
    c["page"] = rng.choice([0, max(64, c["block"]), 128, 256])
    c["ctx"] = _log(rng, 1, 131072)
    # no more than the largest listed reads: tokens x heads of all sequences, padded
    while c["batch"] * c["ctx"] * c["hkv"] > 32 * 32768 * 8:
        c["ctx"] = c["ctx"] // 2 + 1
    c["ctx_min"] = rng.choice([0, c["ctx"] // 2, c["ctx"]])
    if op == "append":
        c["n_max"] = _log(rng, 1, 8192)
        while c["batch"] * c["n_max"] * c["hkv"] > 4 * 8192 * 8:
            c["n_max"] = c["n_max"] // 2 + 1
        c["n_min"] = rng.choice([0, c["n_max"] // 2, c["n_max"]])
    elif op == "commit":
        c["n_max"], c["L"] = _log(rng, 1, 513), rng.choice([4, 16, 32])
    elif op == "read":
        while c["batch"] * c["ctx"] * c["hkv"] > 8 * 32768 * 8:
            c["ctx"] = c["ctx"] // 2 + 1
        c["ctx_min"] = min(c["ctx_min"], c["ctx"])
        c["first"] = rng.choice([0, c["ctx"] // 3])
        c["n_max"] = max(1, c["ctx"] - c["first"])
    else:
        c["hq"] = c["hkv"] * rng.choice([1, 2, 4, 8, 16])
        c["n_max"] = rng.choice([1, 1, _log(rng, 2, 33), _log(rng, 9, 513)])
        while c["batch"] * c["hq"] * c["n_max"] * (c["ctx"] + c["n_max"]) > 8 * 64 * 257 * 8449:
            if c["ctx"] > 2 * c["n_max"]:
                c["ctx"] = c["ctx"] // 2 + 1
            else:
                c["n_max"] = c["n_max"] // 2 + 1
        c["ctx_min"] = min(c["ctx_min"], c["ctx"])
    return c


# ---------------------------------------------------------------- inputs
def _rand_int(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def _kv_rows(g, shape):
    """Rows as a model makes them: channels of unequal size, tokens of unequal size, bf16."""
    ch = torch.exp(0.6 * torch.randn(shape[-2:], generator=g, device="cuda"))
    tok = torch.exp(0.3 * torch.randn((*shape[:-2], 1, 1), generator=g, device="cuda"))
    x = torch.randn(shape, generator=g, device="cuda")
    return x.mul_(ch).mul_(tok).to(torch.bfloat16)


def _quantised(x, block):
    """Codes and exponents of whole blocks of ``x`` [.., tokens, hkv, d]: the cache that earlier calls left."""
    a, t, h, d = x.shape
    y = x.view(a, t // block, block, h, d)
    e = _exponent(y.abs().amax(dim=(2, 4)).float())
    inv = torch.exp2(-e.float()).to(torch.bfloat16)[:, :, None, :, None]
    return (y * inv).view(a, t, h, d).to(torch.float8_e4m3fn), e.to(torch.int8)


def _exponent(amax):
    """The smallest e in [E_MIN, E_MAX] with amax <= 448 * 2^e (exactly: 448 = 0.875 * 2^9)."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    b, hkv, d, block, page = c["batch"], c["hkv"], c["d"], c["block"], c["page"]
    s = {"op": c["op"], "block": block, "page": page, "hkv": hkv, "d": d, "batch": b}
    ctx = _rand_int(g, c["ctx_min"], c["ctx"], b)
    ctx[0] = c["ctx"]  # the longest is there
    grow = {"append": c["n_max"], "commit": c.get("L", 0) + 1}.get(c["op"], 0)
    unit = page or block
    most = -(-max(1, c["ctx"] + grow) // unit) * unit  # positions per sequence
    if page:
        need = (ctx.long() + grow + page - 1) // page
        start = torch.cumsum(need, 0) - need
        total = max(1, int(need.sum())) if grow == 0 else b * most // page  # a pool that is written to has pages free
        perm = torch.randperm(total, generator=g, device="cuda")
        slot = torch.arange(most // page, device="cuda")
        at = (start[:, None] + slot).clamp(max=total - 1)
        s["page_table"] = torch.where(slot < need[:, None], perm[at], -1).int().contiguous()
        shape = (total, page, hkv, d)
    else:
        s["page_table"] = None
        shape = (b, most, hkv, d)
    s["most"] = most
    s["k_cache"], s["k_exp"] = _quantised(_kv_rows(g, shape), block)
    s["v_cache"], s["v_exp"] = _quantised(_kv_rows(g, shape), block)
    s["ctx_len"] = ctx
    if c["op"] in ("append", "commit"):
        s["k_new"] = _kv_rows(g, (b, c["n_max"], hkv, d))
        s["v_new"] = _kv_rows(g, (b, c["n_max"], hkv, d))
        if c["op"] == "append":
            s["n_new"] = _rand_int(g, c["n_min"], c["n_max"], b)
            s["rows"] = torch.arange(c["n_max"], device="cuda").expand(b, -1)
        else:
            n = min(c["L"], c["n_max"] - 1)
            s["acc_len"] = _rand_int(g, 0, n, b)
            pick = torch.rand((b, c["n_max"] - 1), generator=g, device="cuda").argsort(1)[:, :n]
            pick = pick.sort(1).values.int() + 1
            s["acc_nodes"] = torch.full((b, c["L"]), -1, device="cuda", dtype=torch.int32)
            s["acc_nodes"][:, :n] = pick
            s["n_new"] = s["acc_len"] + 1
            s["rows"] = torch.cat([torch.zeros_like(s["acc_nodes"][:, :1]), s["acc_nodes"]], 1).clamp(min=0).long()
        s["first"] = (ctx // block * block).contiguous()       # the touched blocks begin here
        s["window"] = -(-(block - 1 + grow) // block) * block  # and hold at most these positions
        s["ctx_after"] = (ctx + s["n_new"]).contiguous()
    elif c["op"] == "read":
        s["first"] = torch.full((b,), c["first"], device="cuda", dtype=torch.int32)
        s["window"] = c["n_max"]
        s["ctx_after"] = ctx
    else:
        hq, n = c["hq"], c["n_max"]
        s["q"] = torch.randn((b, n, hq, d), generator=g, device="cuda").to(torch.bfloat16)
        s["k_tree"] = _kv_rows(g, (b, n, hkv, d))
        s["v_tree"] = _kv_rows(g, (b, n, hkv, d))
        s["n_nodes"] = _rand_int(g, (n + 1) // 2, n, b)
        s["n_nodes"][0] = n
        up = (torch.rand((b, n), generator=g, device="cuda") * torch.arange(n, device="cuda")).long().cpu()
        see = torch.eye(n, dtype=torch.bool).repeat(b, 1, 1)   # row j sees itself and its ancestors
        for j in range(1, n):
            see[:, j] |= see[torch.arange(b), up[:, j]]
        see &= (torch.arange(n) < s["n_nodes"].cpu()[:, None])[:, :, None]
        w = (n + 31) // 32
        bits = torch.zeros((b, n, w * 32), dtype=torch.long)
        bits[:, :, :n] = see
        words = (bits.view(b, n, w, 32) << torch.arange(32)).sum(-1)
        s["mask"] = torch.where(words >= 2 ** 31, words - 2 ** 32, words).int().cuda()
        s["max_ctx"] = c["ctx"]
        s["scale"] = 1.0 / math.sqrt(d)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    if own:
        return _run_own(s)
    if s["op"] in ("append", "commit"):
        _write(s, "k")
        _write(s, "v")
        return {"k": _read(s, "k"), "v": _read(s, "v"), "k_exp": s["k_exp"], "v_exp": s["v_exp"]}
    if s["op"] == "read":
        return {"k": _read(s, "k"), "v": _read(s, "v")}
    return _attend(s)


def _run_own(s):
    from block_draft_tree_b200 import api
    cache = (s["k_cache"], s["v_cache"], s["k_exp"], s["v_exp"])
    if s["op"] == "attn":
        return api.tree_attn_q8(s["q"], *cache, s["k_tree"], s["v_tree"], s["mask"], s["n_nodes"],
                                s["ctx_len"], s["max_ctx"], block=s["block"],
                                page_table=s["page_table"])
    if s["op"] == "append":
        api.kv_append_q8(s["k_new"], s["v_new"], s["ctx_len"], *cache, block=s["block"],
                         n_new=s["n_new"], page_table=s["page_table"], advance=False)
    elif s["op"] == "commit":
        api.kv_commit_q8(s["k_new"], s["v_new"], s["acc_len"], s["acc_nodes"], s["ctx_len"], *cache,
                         block=s["block"], page_table=s["page_table"], advance=False)
    k, v = api.kv_read_q8(*cache, s["ctx_after"], s["window"], block=s["block"], first=s["first"],
                          page_table=s["page_table"])
    out = {"k": k, "v": v}
    if s["op"] != "read":
        out.update(k_exp=s["k_exp"], v_exp=s["v_exp"])
    return out


def _places(s, pos):
    """Rows of the flattened cache (and blocks of the flattened exponents) that hold ``pos`` [batch, n]; positions outside are held inside."""
    p = pos.clamp(0, s["most"] - 1)
    if s["page"]:
        pg = torch.gather(s["page_table"].long(), 1, p // s["page"]).clamp(min=0)
        row = pg * s["page"] + p % s["page"]
    else:
        row = torch.arange(s["batch"], device="cuda")[:, None] * s["most"] + p
    return row, row // s["block"]


def _write(s, which):
    """The new rows of ``which`` into its codes and exponents."""
    block, hkv, d, b = s["block"], s["hkv"], s["d"], s["batch"]
    codes = s[which + "_cache"].view(torch.uint8).view(-1, hkv, d)
    exps = s[which + "_exp"].view(-1, hkv)
    ctx = s["ctx_len"].long()[:, None]
    pos = s["first"].long()[:, None] + torch.arange(s["window"], device="cuda")
    row, blk = _places(s, pos)
    old = pos < ctx                                        # tokens that are there already
    new = ~old & (pos < ctx + s["n_new"].long()[:, None])
    src = torch.gather(s["rows"], 1, (pos - ctx).clamp(0, s["rows"].shape[1] - 1))
    x = s[which + "_new"][torch.arange(b, device="cuda")[:, None], src].float()
    x = torch.where(new[:, :, None, None], x, torch.zeros_like(x))
    nb = s["window"] // block
    amax = x.view(b, nb, block, hkv, d).abs().amax(dim=(2, 4))
    at = blk.view(b, nb, block)[:, :, 0]
    e_old = exps[at].int().clamp(E_MIN, E_MAX)
    had = old.view(b, nb, block).any(2)[:, :, None]
    e = _exponent(amax)
    e = torch.where(had, torch.maximum(e, e_old), e)
    each = lambda t: t.float().repeat_interleave(block, 1)[:, :, :, None]  # noqa: E731
    was = codes[row].view(torch.float8_e4m3fn).float() * torch.exp2(each(e_old) - each(e))
    y = torch.where(old[:, :, None, None], was, x * torch.exp2(-each(e)))
    q = y.clamp(-Q_MAX, Q_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    keep = old | new
    codes[row[keep]] = q[keep]
    some = new.view(b, nb, block).any(2)
    exps[at[some]] = e[some].to(torch.int8)


def _read(s, which):
    """Rows [first, first + window) of every sequence as bf16; rows past its length are 0."""
    hkv, d = s["hkv"], s["d"]
    pos = s["first"].long()[:, None] + torch.arange(s["window"], device="cuda")
    row, blk = _places(s, pos)
    x = s[which + "_cache"].view(-1, hkv, d).view(torch.uint8)[row].view(torch.float8_e4m3fn).float()
    x = x * torch.exp2(s[which + "_exp"].view(-1, hkv)[blk].float().clamp(E_MIN, E_MAX))[:, :, :, None]
    there = pos < s["ctx_after"].long()[:, None]
    return torch.where(there[:, :, None, None], x, torch.zeros_like(x)).to(torch.bfloat16)


def _attend(s):
    b, n, hq, d = s["q"].shape
    hkv, g, t = s["hkv"], hq // s["hkv"], s["max_ctx"]
    pos = torch.arange(t, device="cuda").expand(b, t)
    row, blk = _places(s, pos)

    def rows(which):  # [b, hkv, t + n, d]: the context's values, then the tree's
        x = s[which + "_cache"].view(-1, hkv, d).view(torch.uint8)[row].view(torch.float8_e4m3fn).float()
        x = x * torch.exp2(s[which + "_exp"].view(-1, hkv)[blk].float())[:, :, :, None]
        x = torch.where((pos < s["ctx_len"].long()[:, None])[:, :, None, None], x, torch.zeros_like(x))
        return torch.cat([x, s[which + "_tree"].float()], 1).transpose(1, 2)

    q = s["q"].float().view(b, n, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, n * g, d)
    w = torch.matmul(q, rows("k").transpose(2, 3)).mul_(s["scale"])
    live = torch.arange(n, device="cuda") < s["n_nodes"].long()[:, None]
    bits = (s["mask"].long()[:, :, :, None] >> torch.arange(32, device="cuda")) & 1
    see = (bits.reshape(b, n, -1)[:, :, :n] > 0) & live[:, :, None]
    past = (pos < s["ctx_len"].long()[:, None])[:, None, :] & live[:, :, None]
    see = torch.cat([past, see], 2).repeat_interleave(g, 1)[:, None]
    w.masked_fill_(~see, -math.inf)
    top = w.amax(3, keepdim=True)
    w.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = w.sum(3, keepdim=True)
    o = torch.matmul(w, rows("v"))
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o.view(b, hkv, n, g, d).permute(0, 2, 1, 3, 4).reshape(b, n, hq, d).to(torch.bfloat16)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    b, hkv, d, block = c["batch"], c["hkv"], c["d"], c["block"]
    mean_ctx = (c["ctx"] + (b - 1) * (c["ctx"] + c["ctx_min"]) / 2) / b
    row = hkv * d
    if c["op"] in ("append", "commit"):
        n = (c["n_min"] + c["n_max"]) / 2 if c["op"] == "append" else min(c["L"], c["n_max"] - 1) / 2 + 1
        old = 0 if c["ctx"] == 0 else (block - 1) / 2          # of a half-filled block, read back
        # bf16 rows in and codes out, then the touched codes in and bf16 windows out
        window = -(-(block - 1 + (c["n_max"] if c["op"] == "append" else c["L"] + 1)) // block) * block
        per = n * 3 * row + (n + old) * row + window * 2 * row
        return {"bytes": 2 * b * per, "flops": 0}
    if c["op"] == "read":
        n = min(max(mean_ctx - c["first"], 0), c["n_max"])
        return {"bytes": 2 * b * (n * row + c["n_max"] * 2 * row), "flops": 0}
    n, hq = c["n_max"], c["hq"]
    live = (n + (b - 1) * 0.75 * n) / b
    bytes_ = b * (2 * mean_ctx * row * (1 + 1 / (block * d)) + 2 * live * row * 2 + 2 * live * hq * d + 2 * n * hq * d
                  + live * (n + 31) // 32 * 4)
    return {"bytes": bytes_, "flops": 4 * b * live * hq * d * (mean_ctx + live)}


# ---------------------------------------------------------------- the definition, in 64 bits
def _code_values():
    """The value of every e4m3 code: sign, 4 exponent bits (bias 7), 3 fraction bits; S.1111.111 is NaN."""
    v = []
    for c in range(256):
        ex, fr = (c >> 3) & 15, c & 7
        m = fr / 8 * 2.0 ** -6 if ex == 0 else (1 + fr / 8) * 2.0 ** (ex - 7)
        v.append(math.nan if c & 127 == 127 else (-m if c & 128 else m))
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _nearest(y):
    """``y`` to the nearest e4m3 value, ties to the even fraction; saturating."""
    ex = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -20))).clamp(-6, 8)
    step = torch.exp2(ex - 3)
    return (torch.round(y / step) * step).clamp(-448.0, 448.0)


def _sequence(s, which, i, n):
    """(codes' values [n, hkv, d], exponents [n, hkv]) of the first n positions of sequence i, in 64 bits."""
    c, e = s[which + "_cache"].view(torch.uint8), s[which + "_exp"].double()
    if s["page"]:
        pages = s["page_table"][i, : -(-n // s["page"])].long() if n else s["page_table"][i, :0].long()
        c, e = c[pages].flatten(0, 1), e[pages].flatten(0, 1)
    else:
        c, e = c[i], e[i]
    return _code_values()[c[:n].long()], e.repeat_interleave(s["block"], 0)[:n]


def _smallest(amax):
    """Smallest e with amax <= 448 * 2^e, by looking at each."""
    e = torch.full_like(amax, float(E_MIN))
    for k in range(E_MIN, E_MAX):
        e = torch.where(amax > 448.0 * 2.0 ** k, torch.full_like(e, k + 1.0), e)
    return e


def exact(case, seed):
    s = prepare(case, seed)
    b, hkv, d, block = s["batch"], s["hkv"], s["d"], s["block"]
    if s["op"] in ("append", "commit", "read"):
        out = {w: torch.zeros((b, s["window"], hkv, d), dtype=torch.float64, device="cuda") for w in "kv"}
        for w in "kv":
            for i in range(b):
                first, end = int(s["first"][i]), int(s["ctx_after"][i])
                ctx = int(s["ctx_len"][i])
                v, e = _sequence(s, w, i, ctx)
                if s["op"] == "read":
                    got = (v * torch.exp2(e)[:, :, None])[first:first + s["window"]]
                else:
                    x = s[w + "_new"][i][s["rows"][i, : end - ctx]].double()
                    got = torch.empty((end - first, hkv, d), dtype=torch.float64, device="cuda")
                    lo = first
                    while lo < end:
                        hi = min(end, lo + block if lo < ctx else end)  # the block with older tokens, then all the whole ones
                        if lo < ctx:
                            fresh = x[: hi - ctx]
                            need = _smallest(fresh.abs().amax((0, 2))) if len(fresh) else torch.full((hkv,), -1e9, device="cuda", dtype=torch.float64)
                            e_old = e[lo]
                            ex = torch.maximum(e_old, need)[None, :, None]
                            part = torch.cat([v[lo:ctx] * torch.exp2(e_old[None, :, None] - ex), fresh * torch.exp2(-ex)])
                        else:
                            fresh = x[lo - ctx:]
                            pad = torch.zeros((-len(fresh) % block, hkv, d), dtype=torch.float64, device="cuda")
                            ex = _smallest(torch.cat([fresh, pad]).view(-1, block, hkv, d).abs().amax((1, 3)))
                            ex = ex.repeat_interleave(block, 0)[: len(fresh), :, None]
                            part = fresh * torch.exp2(-ex)
                        got[lo - first: hi - first] = _nearest(part) * torch.exp2(ex)
                        lo = hi
                out[w][i, : len(got)] = got
        if s["op"] != "read":
            out.update(k_exp=None, v_exp=None)
        return out
    n, hq = s["q"].shape[1:3]
    g = hq // hkv
    out = torch.zeros((b, n, hq, d), dtype=torch.float64, device="cuda")
    bits = ((s["mask"].long()[:, :, :, None] >> torch.arange(32, device="cuda")) & 1).reshape(b, n, -1)[:, :, :n]
    for i in range(b):
        m, ctx = int(s["n_nodes"][i]), int(s["ctx_len"][i])
        kv = []
        for w in "kv":
            x, e = _sequence(s, w, i, ctx)
            kv.append(torch.cat([x * torch.exp2(e)[:, :, None], s[w + "_tree"][i, :m].double()]))
        hidden = torch.cat([torch.zeros((m, ctx), device="cuda", dtype=torch.bool), bits[i, :m, :m] == 0], 1)
        for h in range(hq):
            z = s["q"][i, :m, h].double() @ kv[0][:, h // g].T * s["scale"]
            z[hidden] = -math.inf
            p = torch.exp(z - z.amax(1, keepdim=True))
            out[i, :m, h] = (p @ kv[1][:, h // g]) / p.sum(1, keepdim=True)
    return out
