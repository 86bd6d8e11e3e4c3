"""The 8-bit key/value cache in plain torch, 64 bits: the tests' reference.

Written from the format's definition (e4m3 codes, one power of two per block
of tokens and kv head); shares nothing with the library."""
import math

import torch

EXP_MIN, EXP_MAX, EXP_NAN = -48, 48, -128


def code_values() -> torch.Tensor:
    """f64 value of each of the 256 e4m3 codes."""
    v = []
    for c in range(256):
        ex, fr = (c >> 3) & 15, c & 7
        m = fr * 2.0 ** -9 if ex == 0 else (8 + fr) * 2.0 ** (ex - 10)
        v.append(math.nan if (c & 127) == 127 else (-m if c & 128 else m))
    return torch.tensor(v, dtype=torch.float64)


def encode(y: torch.Tensor) -> torch.Tensor:
    """f64 -> e4m3 codes (uint8), nearest, ties to the even code; saturating;
    finite values only."""
    mags = code_values()[:127].to(y.device)                 # 0 .. 448, ascending
    a = y.abs().clamp(max=448.0)
    hi = torch.searchsorted(mags, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    below, above = a - mags[lo], mags[hi] - a
    take_lo = (below < above) | ((below == above) & (lo % 2 == 0))
    c = torch.where(take_lo, lo, hi).to(torch.uint8)
    return torch.where(torch.signbit(y), c | 128, c)


def decode(codes: torch.Tensor) -> torch.Tensor:
    return code_values().to(codes.device)[codes.view(torch.uint8).long()]


def scales(exps: torch.Tensor) -> torch.Tensor:
    """f64 scale of stored exponents (NaN for a block marked so)."""
    s = torch.exp2(exps.double().clamp(EXP_MIN, EXP_MAX))
    return torch.where(exps == EXP_NAN, math.nan, s)


def needed_exp(amax: float) -> int:
    """Smallest exponent with amax <= 448 * 2^e, in range."""
    for e in range(EXP_MIN, EXP_MAX):
        if amax <= 448.0 * 2.0 ** e:
            return e
    return EXP_MAX


class Cache:
    """A cache (dense or paged) of random content, with a plain view of it."""

    def __init__(self, b, tokens, hkv, d, block, page=0, seed=0, device="cuda", exps=(-8, -2)):
        g = torch.Generator().manual_seed(seed)
        self.b, self.hkv, self.d, self.block, self.page = b, hkv, d, block, page
        self.page_table = None
        if page:
            per = -(-tokens // page)
            pages = b * per + 3
            self.page_table = torch.randperm(pages, generator=g)[:b * per].view(b, per).int()
            shape = (pages, page)
        else:
            shape = (b, tokens)
        nb = -(-shape[1] // block)
        codes = torch.randint(0, 256, (2, *shape, hkv, d), generator=g, dtype=torch.uint8)
        codes = torch.where((codes & 127) == 127, codes & 0x80, codes)  # as the library writes them
        e = torch.randint(exps[0], exps[1] + 1, (2, shape[0], nb, hkv), generator=g).to(torch.int8)
        self.codes = [c.to(device) for c in codes]
        self.exps = [x.contiguous().to(device) for x in e]
        if page:
            self.page_table = self.page_table.contiguous().to(device)

    def args(self):
        f = torch.float8_e4m3fn
        return (self.codes[0].view(f), self.codes[1].view(f), self.exps[0], self.exps[1])

    def kw(self):
        return {"block": self.block, "page_table": self.page_table}

    def clone(self):
        c = object.__new__(Cache)
        c.__dict__.update(self.__dict__)
        c.codes = [x.clone() for x in self.codes]
        c.exps = [x.clone() for x in self.exps]
        return c

    def place(self, i, t):
        """(index 0, token in it) of position t of sequence i, or None."""
        if self.page:
            if t // self.page >= self.page_table.shape[1]:
                return None
            pg = int(self.page_table[i, t // self.page])
            return (pg, t % self.page) if 0 <= pg < self.codes[0].shape[0] else None
        return (i, t) if t < self.codes[0].shape[1] else None

    def values(self, which, i, n):
        """f64 [n, hkv, d] of positions 0..n-1 of sequence i."""
        codes, exps = self.codes[which], scales(self.exps[which])
        if self.page:
            pages = self.page_table[i, :-(-n // self.page)].long() if n else self.page_table[i, :0].long()
            codes, exps = codes[pages].flatten(0, 1), exps[pages].flatten(0, 1)
        else:
            codes, exps = codes[i], exps[i]
        e = exps.repeat_interleave(self.block, 0)[:n]
        return decode(codes[:n]) * e[:, :, None]

    def append(self, i, ctx, rows_k, rows_v):
        """The definition of a write, a block and a head at a time; rows [n, hkv, d]."""
        for which, rows in ((0, rows_k), (1, rows_v)):
            rows = rows.double()
            n, block = rows.shape[0], self.block
            pos = ctx
            while pos < ctx + n:
                b0 = pos // block * block
                end = min(ctx + n, b0 + block)
                at = self.place(i, b0)
                new = rows[pos - ctx:end - ctx]
                if at is not None:
                    a, s = at
                    if not self.page:
                        new = new[:max(0, self.codes[0].shape[1] - pos)]
                    for h in range(self.hkv if new.shape[0] else 0):
                        x = new[:, h]
                        was = int(self.exps[which][a, s // block, h])
                        new_codes = self.codes[which][a, s + pos - b0:s + pos - b0 + x.shape[0], h]
                        if not torch.isfinite(x).all() or (b0 < ctx and was == EXP_NAN):
                            self.exps[which][a, s // block, h] = EXP_NAN
                            new_codes.zero_()
                            continue
                        e = needed_exp(float(x.abs().max()))
                        if b0 < ctx:
                            old_e = max(EXP_MIN, min(EXP_MAX, was))
                            e = max(e, old_e)
                            if e > old_e:
                                old = self.codes[which][a, s:s + pos - b0, h]
                                self.codes[which][a, s:s + pos - b0, h] = encode(decode(old) * 2.0 ** (old_e - e))
                        new_codes.copy_(encode(x * 2.0 ** -e))
                        self.exps[which][a, s // block, h] = e
                pos = end


def attention(q, kv_ctx, kv_tree, see, scale):
    """One (sequence, kv head): q [rows, d], context and tree K/V [.., d] f64, see
    [rows, tree] bool.  Returns (out, lse, A, S): A = sum p|v|, and S the
    row's largest scale * sum |q k| over the tokens that it sees."""
    k = torch.cat([kv_ctx[0], kv_tree[0]])
    v = torch.cat([kv_ctx[1], kv_tree[1]])
    every = torch.cat([torch.ones(q.shape[0], kv_ctx[0].shape[0], dtype=torch.bool, device=q.device), see], 1)
    # a token's K or V counts only where it is seen, whatever it holds elsewhere
    z = (torch.where(every[:, :, None], k[None], 0.0) * q[:, None]).sum(2) * scale
    S = (torch.where(every[:, :, None], k[None], 0.0).abs() * q[:, None].abs()).sum(2).amax(1) * scale if k.shape[0] else torch.zeros(q.shape[0], device=q.device)
    z = torch.where(every, z, torch.full_like(z, -math.inf))
    if k.shape[0] == 0:
        none = torch.zeros_like(q)
        return none, torch.full((q.shape[0],), -math.inf, device=q.device, dtype=torch.float64), none, S
    m = z.amax(1, keepdim=True)
    p = torch.where(every, torch.exp(z - torch.where(m == -math.inf, 0.0, m)), 0.0)
    l = p.sum(1, keepdim=True)
    vs = torch.where(every[:, :, None], v[None], 0.0)
    safe = torch.where(l == 0, 1.0, l)
    out = (p[:, :, None] * vs).sum(1) / safe
    A = (p[:, :, None] * vs.abs()).sum(1) / safe
    lse = torch.where(l[:, 0] == 0, -math.inf, m[:, 0] + torch.log(l[:, 0]))
    return out, lse, A, S
