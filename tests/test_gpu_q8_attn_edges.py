"""Tree attention over the 8-bit cache where its surroundings are hostile:
caches that end inside a tile with NaN codes around them.  Reference and
tolerance are those of test_gpu_q8_attn."""
import pytest
import torch

from test_gpu_q8_attn import Case

pytestmark = pytest.mark.gpu
DEV = "cuda"


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
