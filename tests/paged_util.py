"""Plain 64-bit forms of the paged 8-bit latent cache's three calls, written
from their definitions in include/cpmla.h, and batches to run them on."""
import numpy as np
import torch

EXP_MIN, BIAS, DQK, DV = -64, 127, 576, 512


def e4m3_round(v):
    """The E4M3 value nearest to v, ties to even, saturating (NaN stays)."""
    v = np.clip(v, -1024.0, 1024.0)  # infinities saturate
    a = np.maximum(np.abs(v), 2.0 ** -60)
    with np.errstate(invalid="ignore"):
        step = np.exp2(np.maximum(np.floor(np.log2(a)), -6) - 3)
        return np.clip(np.round(v / step) * step, -448, 448)


def e4m3_values():
    """The value of each of the 256 codes."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.exp2(e - 10.0))
    v[(c & 127) == 127] = np.nan
    return np.where(c < 128, v, -v)


def decode(cache):
    """Codes (numpy uint8) -> values, without the scale."""
    return e4m3_values()[cache]


def maps(ctx, new, free, head, table, bs, n_slots):
    """(cu, slot, pos, req, head after, table after) of well-formed inputs."""
    table = table.copy()
    cu, slot, pos, req = [0], [], [], []
    for b, (c, n) in enumerate(zip(ctx, new)):
        for i in range(-(-c // bs), -(-(c + n) // bs)):
            table[b, i] = free[head]
            head += 1
        p = np.arange(c, c + n)
        pos += p.tolist()
        req += [b] * n
        slot += (table[b, p // bs].astype(np.int64) * bs + p % bs).tolist()
        cu.append(cu[-1] + n)
    tail = [-1] * (n_slots - len(pos))
    return (np.array(cu), np.array(slot + tail, np.int64), np.array(pos + tail),
            np.array(req + tail), head, table)


def exponent(x):
    """The least e >= -64 with |x| <= 448 * 2^e over the finite entries."""
    f = np.abs(x[np.isfinite(x)])
    amax = f.max(initial=0.0)
    e = EXP_MIN
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def insert(kv, slot, cache_values, exp, bs):
    """kv float64 [n, 576]; cache_values float64 [n_blocks, bs, 576] without
    the scale, exp int: both after the call."""
    cache_values, exp = cache_values.copy(), exp.astype(np.int64).copy() - BIAS
    last = {int(s): i for i, s in enumerate(slot) if s >= 0}
    blocks = {}
    for s, i in last.items():
        blocks.setdefault(s // bs, []).append((s % bs, i))
    for b, toks in blocks.items():
        e = exponent(kv[[i for _, i in toks]])
        if all(r != 0 for r, _ in toks):
            if exp[b] >= e:
                e = exp[b]
            else:
                cache_values[b] = e4m3_round(cache_values[b] * 2.0 ** (exp[b] - e))
        for r, i in toks:
            cache_values[b, r] = e4m3_round(kv[i] * 2.0 ** -e)
        exp[b] = e
    return cache_values, exp + BIAS


def attend(q, cache, exp, table, tokens, pos, req, scale, sink=None, lo=None, hi=None):
    """{entry: (o [H, 512], lse [H], weight [H, 512])} in float64 on q's device;
    weight is the softmax average of |v| with the sink factor, the size that
    rounding errors of the softmax weights scale with.  Entries with req -1 are
    left out; blocks outside the cache are skipped."""
    dev = q.device
    n_blocks, bs = cache.shape[:2]
    val = torch.from_numpy(e4m3_values()).to(dev)[cache.long()]
    val = val * torch.exp2(exp.double() - BIAS)[:, None, None]
    out = {}
    for i in range(len(pos)):
        b, t = int(req[i]), int(pos[i])
        if b < 0:
            continue
        a = 0 if lo is None else max(0, int(lo[i]))
        z = t if hi is None else min(t, int(hi[i]))
        k = torch.arange(a, max(a, z + 1), device=dev)
        blk = table[b, k // bs].long()
        k, blk = k[(blk >= 0) & (blk < n_blocks)], blk[(blk >= 0) & (blk < n_blocks)]
        kv = val[blk, k % bs]
        x = q[int(tokens[i])].double() @ kv.T * scale
        lse = torch.logsumexp(x, 1) if len(k) else torch.full((q.shape[1],), -np.inf, device=dev,
                                                              dtype=torch.float64)
        p = torch.exp(x - torch.where(lse.isinf(), 0.0, lse)[:, None])
        gate = torch.ones_like(lse) if sink is None else torch.sigmoid(lse - sink.double())
        p = p * torch.where(lse.isneginf(), 0.0, gate)[:, None]
        out[i] = (p @ kv[:, :DV], lse, p @ kv[:, :DV].abs())
    return out


class Batch:
    """A paged cache with the blocks of some requests, in no order, and the
    entries of the tokens they schedule."""

    def __init__(self, ctx, new, bs, seed=0, spare=3, spread=4, dev="cuda"):
        g = torch.Generator().manual_seed(seed)
        ctx, new = np.asarray(ctx), np.asarray(new)
        need = -(-(ctx + new) // bs)
        self.bs, self.n_blocks, self.dev = bs, int(need.sum()) + spare, dev
        perm = torch.randperm(self.n_blocks, generator=g).numpy()
        self.table = np.full((len(ctx), max(1, int(need.max())) + 1), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.req = np.repeat(np.arange(len(new)), new).astype(np.int32)
        self.pos = np.concatenate([np.arange(c, c + n) for c, n in zip(ctx, new)]).astype(np.int32)
        self.exp = torch.randint(BIAS - 6, BIAS - 6 + spread, (self.n_blocks,), generator=g,
                                 dtype=torch.uint8)
        x = torch.randn((self.n_blocks, bs, DQK), generator=g)
        x = x * torch.exp2(BIAS - self.exp.float())[:, None, None]
        self.cache = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        self.gen = g

    def gpu(self):
        t = lambda a: (torch.from_numpy(a) if isinstance(a, np.ndarray) else a).to(self.dev)
        return dict(cache=t(self.cache), cache_exp=t(self.exp), block_table=t(self.table),
                    pos=t(self.pos), req=t(self.req))
