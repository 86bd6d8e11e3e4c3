"""The 8-bit cache as a serving loop uses it: prompts appended, rounds of the
captured driver (top-k, tree, attention, walk, commit) replayed behind them,
the cache read back.  Each step is checked against the plain reference on the
state that the step before it left."""
import math

import numpy as np
import pytest
import torch

from block_draft_tree_b200 import api, synth
from block_draft_tree_b200.round import VerifyRound

import q8_ref
from helpers import i32, logits_tensor
from q8_ref import Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("decode", ["greedy", "sample", "lm_head"])
@pytest.mark.parametrize("page,block,d,hq,hkv,B", [(0, 16, 64, 4, 1, 8), (64, 32, 128, 8, 2, 40)])
def test_prompt_rounds_and_read_back(decode, page, block, d, hq, hkv, B):
    w = synth.WORKLOADS["tiny"].scaled(batch=3, L=4, V=500, k=4, B=B)
    b, n, t_max = w.batch, w.n_max, 512
    g = torch.Generator().manual_seed(B)
    bf = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    c = Cache(b, t_max, hkv, d, block, page, seed=B)
    plain = c.clone()
    prompt = [200, 0, 131]
    kp, vp = bf(b, 200, hkv, d), bf(b, 200, hkv, d)
    ctx = i32([0] * b)
    api.kv_append_q8(kp, vp, ctx, *c.args(), n_new=i32(prompt), **c.kw())
    for i in range(b):
        plain.append(i, 0, kp[i, :prompt[i]], vp[i, :prompt[i]])
    rnd = VerifyRound(batch=b, L=w.L, V=w.V, k=w.k, B_max=B, hq=hq, hkv=hkv, d=d, max_ctx=t_max,
                      draft_dtype=torch.float32, decode=decode, commit=True, cache="q8", block=block,
                      paged=page > 0, page_size=page or 64, max_pages=t_max // (page or 64))
    kc, vc, ke, ve = c.args()
    x = {"draft": logits_tensor(synth.draft_logits(w)), "root": i32(synth.root_tokens(w)), "ctx_len": ctx,
         "q": bf(b, n, hq, d), "k_tree": bf(b, n, hkv, d), "v_tree": bf(b, n, hkv, d),
         "k_cache": kc, "v_cache": vc, "k_exp": ke, "v_exp": ve, "page_table": c.page_table,
         "target": torch.randn((b, n, w.V), generator=g).cuda(), "hidden": bf(b, n, 64), "head": bf(w.V, 64)}
    rnd.bind(x)
    graph = rnd.capture()
    o = rnd.out
    for r in range(4):
        for name in ("q", "k_tree", "v_tree", "hidden"):      # a model's forward fills the bound buffers
            x[name].copy_(bf(*x[name].shape))
        before = ctx.tolist()
        graph.replay()
        torch.cuda.synchronize()
        assert int(o["status"]) == 0
        nn, words = o["n_nodes"].tolist(), o["mask"].cpu().numpy().view(np.uint32)
        for i in range(b):
            see = torch.tensor([[bool(words[i, j, t // 32] >> (t % 32) & 1) for t in range(nn[i])]
                                for j in range(nn[i])], device="cuda")
            kv = [plain.values(k, i, before[i]) for k in range(2)]
            for h in range(hq):
                kvh = h // (hq // hkv)
                ref, _, A, S = q8_ref.attention(
                    x["q"][i, :nn[i], h].double(), [z[:, kvh] for z in kv],
                    [x["k_tree"][i, :nn[i], kvh].double(), x["v_tree"][i, :nn[i], kvh].double()], see,
                    1 / math.sqrt(d))
                rel = (d + 8) * 2.0 ** -23 * S * 1.4427 + 2.0 ** -20   # as in test_gpu_q8_attn
                tol = ref.abs() * 2.0 ** -8 + A * (2.0 ** -11 + 2 * rel[:, None]) + 1e-6
                assert ((o["attn"][i, :nn[i], h].double() - ref).abs() <= tol).all()
            acc = int(o["acc_len"][i])
            rows = [0] + o["acc_nodes"][i, :acc].tolist()
            plain.append(i, before[i], x["k_tree"][i, rows], x["v_tree"][i, rows])
            assert int(ctx[i]) == before[i] + acc + 1
    for k in range(2):
        assert torch.equal(c.codes[k], plain.codes[k]) and torch.equal(c.exps[k], plain.exps[k])
    k, v = api.kv_read_q8(*c.args(), ctx, t_max, **c.kw())
    for i in range(b):
        T = int(ctx[i])
        assert torch.equal(k[i, :T].double(), plain.values(0, i, T))
        assert torch.equal(v[i, :T].double(), plain.values(1, i, T)) and not v[i, T:].any()


def test_round_refuses_a_cache_of_the_other_form():
    w = synth.WORKLOADS["tiny"]
    kw = dict(batch=w.batch, L=w.L, V=w.V, k=w.k, B_max=w.B, hq=w.hq, hkv=w.hkv, d=w.d, max_ctx=w.ctx,
              draft_dtype=torch.float32)
    with pytest.raises(ValueError, match="cache"):
        VerifyRound(cache="int4", **kw)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    c = Cache(w.batch, w.ctx, w.hkv, w.d, 16)
    kc, vc, ke, ve = c.args()
    x = {"draft": torch.zeros((w.batch, w.L, w.V), device="cuda"), "root": i32([0]), "ctx_len": i32([8]),
         "q": bf(1, w.n_max, w.hq, w.d), "k_tree": bf(1, w.n_max, w.hkv, w.d),
         "v_tree": bf(1, w.n_max, w.hkv, w.d), "k_cache": kc, "v_cache": vc, "k_exp": ke, "v_exp": ve,
         "target": torch.zeros((1, w.n_max, w.V), device="cuda")}
    with pytest.raises(api.DDTError):
        VerifyRound(**kw).bind(x)                                   # 8-bit tensors, bf16 round
    VerifyRound(cache="q8", **kw).bind(x)
    for name, t in (("k_cache", bf(*kc.shape)), ("k_exp", None), ("v_exp", ve[:, :4].contiguous())):
        with pytest.raises(api.DDTError):
            VerifyRound(cache="q8", commit=True, **kw).bind(dict(x, **{name: t}))
