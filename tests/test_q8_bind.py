"""VerifyRound over the 8-bit cache refuses tensors that are not on its device
(CPU: the host is the round's device, torch's meta device the other one)."""
import pytest
import torch

from block_draft_tree_b200 import api, build
from block_draft_tree_b200.round import VerifyRound


def test_bind_refuses_tensors_of_another_device():
    build.build()
    b, L, V, k, B, hq, hkv, d, T = 2, 4, 64, 4, 8, 4, 1, 64, 32
    n = B + 1
    rnd = VerifyRound(batch=b, L=L, V=V, k=k, B_max=B, hq=hq, hkv=hkv, d=d, max_ctx=T,
                      draft_dtype=torch.float32, device="cpu", cache="q8", commit=True)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    f8 = lambda *s: torch.zeros(s, dtype=torch.uint8).view(torch.float8_e4m3fn)  # noqa: E731
    dense = {"draft": torch.zeros(b, L, V), "root": i32(b), "ctx_len": i32(b), "q": bf(b, n, hq, d),
             "k_tree": bf(b, n, hkv, d), "v_tree": bf(b, n, hkv, d), "target": torch.zeros(b, n, V),
             "k_cache": f8(b, T, hkv, d), "v_cache": f8(b, T, hkv, d),
             "k_exp": torch.zeros((b, T // 16, hkv), dtype=torch.int8),
             "v_exp": torch.zeros((b, T // 16, hkv), dtype=torch.int8)}
    paged = dict(dense, page_table=i32(b, 1))
    for good in (dense, paged):
        rnd._check_inputs(good)
        for name in ("ctx_len", "q", "k_tree", "v_tree", "k_cache", "v_cache", "k_exp", "v_exp", "page_table"):
            if name in good:
                with pytest.raises(api.DDTError, match="%r must be on" % name):
                    rnd._check_inputs(dict(good, **{name: good[name].to("meta")}))
