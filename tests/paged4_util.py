"""Plain 64-bit forms of the paged 4-bit latent cache and of the rotation, written
from their definitions in include/cpmla.h, and batches to run them on."""
import numpy as np
import torch

import paged_util as pu

DQK, DV, STRIP = 576, 512, 5392
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def two(e):
    return np.ldexp(1.0, np.asarray(e))


def e2m1_round(v):
    """The E2M1 value nearest to v, ties to the even code, saturating."""
    a = np.minimum(np.abs(v), 8.0)
    i = np.abs(a[..., None] - E2M1).argmin(-1)          # ties: the lower index ...
    up = np.minimum(i + 1, 7)
    tie = (a - E2M1[i] == E2M1[up] - a) & (i % 2 == 1)  # ... unless that is odd
    return np.sign(v) * E2M1[np.where(tie, up, i)]


def exponent(amax):
    """The least e in -64 .. 119 with amax <= 448 * 2^e."""
    e = -64
    while e < 119 and amax > 448 * two(e):
        e += 1
    return e


def offset(amax, e):
    """The largest d in 0 .. 11 with amax <= 7 * 2^(e + 6 - d)."""
    d = 11
    while d > 0 and amax > 7 * two(e + 6 - d):
        d -= 1
    return d


def quantise(row):
    """(values [576], stored exponent, offsets [32]) of a float64 row."""
    top = lambda x: np.abs(x[np.isfinite(x)]).max(initial=0.0)
    e = exponent(top(row))
    out, off = np.empty(DQK), []
    for g in range(32):
        x = row[16 * g:16 * g + 16]
        d = offset(top(x), e)
        off.append(d)
        out[16 * g:16 * g + 16] = e2m1_round(x * two(-(e + 6 - d))) * two(e + 6 - d)
    out[DV:] = pu.e4m3_round(row[DV:] * two(-e)) * two(e)
    if np.isnan(row).any():
        return np.full(DQK, np.nan), 255, off
    return out, e + 127, off


def decode(cache):
    """Values (float64 [n_blocks, bs, 576]) of a cache (numpy uint8 [n_blocks, bs / 16, 5392])."""
    nb, ns, _ = cache.shape
    out = np.empty((nb, ns, 16, DQK))
    e4 = pu.e4m3_values()
    ex = cache[..., 5376:].astype(int)
    unit = np.where(ex == 255, np.nan, two(np.clip(ex, 63, 246) - 127))
    for r in range(16):
        for g in range(32):
            at = 256 * r + 16 * (g % 16) + 8 * (g // 16)
            b = cache[..., at:at + 8].astype(np.int64)
            d = np.minimum(cache[..., 5120 + 16 * r + g % 16].astype(int) >> 4 * (g // 16) & 15, 11)
            f = unit[..., r] * two(6 - d)
            for c in range(16):
                w = sum(b[..., c // 8 * 4 + i] << 8 * i for i in range(4))
                j = c % 8
                s = w >> (8 * j + 7 if j < 4 else 8 * (j - 4) + 3) & 1
                out[..., r, 16 * g + c] = (1 - 2 * s) * E2M1[w >> 4 * j & 7] * f
        out[..., r, DV:] = e4[cache[..., 4096 + 64 * r:4160 + 64 * r]] * unit[..., r, None]
    return out.reshape(nb, ns * 16, DQK)


def encode(values, e, off, rng=None):
    """The bytes [5392] of a strip of 16 tokens: float64 values that the format holds
    with these stored exponents [16] and offsets [16, 32]."""
    s = np.zeros(STRIP, np.uint8)
    codes = pu.e4m3_values()
    for r in range(16):
        s[5376 + r] = e[r]
        unit = two(int(np.clip(e[r], 63, 246)) - 127)
        for g in range(32):
            x = values[r, 16 * g:16 * g + 16] / (unit * two(6 - min(int(off[r, g]), 11)))
            s[5120 + 16 * r + g % 16] |= int(off[r, g]) << 4 * (g // 16)
            for c in range(16):
                at = 256 * r + 16 * (g % 16) + 8 * (g // 16) + c // 8 * 4
                j = c % 8
                mag = int(np.flatnonzero(E2M1 == abs(x[c]))[0])
                bits = mag << 4 * j | int(x[c] < 0) << (8 * j + 7 if j < 4 else 8 * (j - 4) + 3)
                for i in range(4):
                    s[at + i] |= bits >> 8 * i & 255
        for c in range(64):
            s[4096 + 64 * r + c] = int(np.flatnonzero(codes == values[r, DV + c] / unit)[0])
    return s


def rotate(x, pos, f, amplitude=1.0, pairs=True, inverse=False):
    """The rotation of x (float64 [n, ..., 64]) at positions pos [n]."""
    a = np.asarray(pos, np.float64)[:, None] * np.asarray(f)
    z = amplitude * np.exp((-1j if inverse else 1j) * a)
    z = z.reshape(len(pos), *[1] * (x.ndim - 2), 32)
    if pairs:
        y = (x[..., 0::2] + 1j * x[..., 1::2]) * z
        return np.stack([y.real, y.imag], -1).reshape(x.shape)
    y = (x[..., :32] + 1j * x[..., 32:]) * z
    return np.concatenate([y.real, y.imag], -1)


def attend(q, val, cache, table, tokens, pos, req, scale, sink=None, lo=None, hi=None):
    """As paged_util.attend, over values (float64 [n_blocks, bs, 576] on q's device) of a
    cache.  With P a weight times its token's 2^e, the weight's companion is the sum over
    the tokens of the largest P of their 32 positions times their codes' magnitudes."""
    dev = q.device
    n_blocks, bs = val.shape[:2]
    unit = cache[..., 5376:].reshape(n_blocks, bs).to(dev).double().clamp(63, 246).sub(127).exp2()
    out = {}
    for i in range(len(pos)):
        b, t = int(req[i]), int(pos[i])
        if b < 0:
            continue
        a = 0 if lo is None else max(0, int(lo[i]))
        z = t if hi is None else min(t, int(hi[i]))
        k = torch.arange(a, max(a, z + 1), device=dev)
        blk = table[b, k // bs].long()
        ok = (blk >= 0) & (blk < n_blocks)
        k, blk = k[ok], blk[ok]
        kv = val[blk, k % bs]
        x = q[int(tokens[i])].double() @ kv.T * scale
        lse = torch.logsumexp(x, 1) if len(k) else torch.full((q.shape[1],), -np.inf, device=dev,
                                                              dtype=torch.float64)
        p = torch.exp(x - torch.where(lse.isinf(), 0.0, lse)[:, None])
        gate = torch.ones_like(lse) if sink is None else torch.sigmoid(lse - sink.double())
        p = p * torch.where(lse.isneginf(), 0.0, gate)[:, None]
        tile = k // 32 - (a // 32 if len(k) else 0)
        big = torch.zeros((len(p), int(tile.max()) + 1 if len(k) else 1), dtype=p.dtype, device=dev)
        e = unit[blk, k % bs]
        big = big.index_reduce(1, tile, p * e, "amax")[:, tile]
        v = kv[:, :DV].abs()
        out[i] = (p @ kv[:, :DV], lse, p @ v, big @ (v / e[:, None]))
    return out


def random_cache(n_blocks, bs, seed, spread=3, size=0.5):
    """Bytes that any cache might hold: codes of all kinds, token exponents around
    unit size, offsets 0 .. 5 (torch uint8, on the CPU)."""
    g = torch.Generator().manual_seed(seed)
    n = n_blocks * bs // 16
    c = torch.randint(0, 256, (n, STRIP), generator=g, dtype=torch.uint8)
    r = torch.randn((n, 16 * 64), generator=g) * 60
    c[:, 4096:5120] = r.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    o = torch.randint(0, 6, (2, n, 256), generator=g, dtype=torch.uint8)
    c[:, 5120:5376] = o[0] | o[1] << 4
    c[:, 5376:] = torch.randint(127 - 7, 127 - 7 + spread, (n, 16), generator=g, dtype=torch.uint8)
    return c.view(n_blocks, bs // 16, STRIP)


class Batch4(pu.Batch):
    """paged_util.Batch over a 4-bit cache."""

    def __init__(self, ctx, new, bs, seed=0, spare=3, spread=3, dev="cuda"):
        need = -(-(np.asarray(ctx) + np.asarray(new)) // bs)
        super().__init__(ctx, new, bs, seed=seed, spare=spare, dev=dev)
        del self.exp
        self.cache = random_cache(int(need.sum()) + spare, bs, seed + 1, spread)

    def values(self):
        return torch.from_numpy(decode(self.cache.cpu().numpy())).to(self.dev)

    def gpu(self):
        t = lambda a: (torch.from_numpy(a) if isinstance(a, np.ndarray) else a).to(self.dev)
        return dict(cache=t(self.cache), block_table=t(self.table), pos=t(self.pos), req=t(self.req))
