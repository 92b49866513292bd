"""Measured cases of the 4-bit latent cache: the rotation of queries and keys, the
writing of a step's tokens (and reading them back), the reading of listed slots,
and the attention over the cache.

The cache is a pool of blocks of strips of 16 tokens, 5392 bytes each: the tokens'
E2M1 codes (256 bytes a token), their rope channels as E4M3 codes (64), an offset
of 4 bits for each group of 16 latent channels (16), and an exponent byte a token.

The plain forms are written with elementary torch operations in fp32 (angles in
64 bits); `exact` computes the same from the definitions in 64 bits.
"""
import random

import numpy as np
import torch

own = False

DQK, DV, DR = 576, 512, 64
STRIP = 5392                     # bytes of 16 tokens
ROPE_AT, OFF_AT, EXP_AT = 4096, 5120, 5376
EXP_MIN, EXP_MAX, EXP_BIAS = -64, 119, 127
OFF_MAX = 11                     # a group's scale is 2^(e + 6 - offset)


# ---------------------------------------------------------------- the cases
def _rope(name=None, n=1, heads=16, wide=192, pos_hi=131072, base=10000.0, factor=1.0,
          interleaved=True, inverse=False, pad=0):
    c = dict(op="rope", n=n, heads=heads, wide=wide, pos_hi=pos_hi, base=base, factor=factor,
             interleaved=interleaved, inverse=inverse, pad=pad)
    return {**c, "name": name} if name else c


def _slots(op, name=None, n=1, spread=1, block=64, pad=0):
    """n tokens of `spread` requests (a run of slots each, or each by itself)."""
    c = dict(op=op, n=n, spread=spread, block=block, pad=pad)
    return {**c, "name": name} if name else c


def _attn(name=None, prefills=0, p_lo=1, p_hi=1, pc_hi=0, decodes=0, d_lo=0, d_hi=0, block=64,
          pad=0, shape=1, heads=16, mask="causal"):
    """`prefills` requests that schedule p_lo..p_hi new tokens on top of a context of up
    to pc_hi, then `decodes` requests with one token on top of d_lo..d_hi; the lengths
    are drawn from `shape`.  `pad` entries behind the last request stand for no token."""
    c = dict(op="attn", prefills=prefills, p_lo=p_lo, p_hi=p_hi, pc_hi=pc_hi, decodes=decodes,
             d_lo=d_lo, d_hi=d_hi, block=block, pad=pad, shape=shape, heads=heads, mask=mask)
    return {**c, "name": name} if name else c


def listed():
    return [
        # the rope channels of 32 decode rows, contexts beyond the trained length (x 40)
        _rope("rope_decode_32_h16", n=32, heads=16, factor=40.0),
        # a long prompt's, an odd length, halves in place of pairs
        _rope("rope_prompt_32771_h16", n=32771, heads=16, interleaved=False),
        # 32 decode rows into their slots, and what the cache then holds of them
        _slots("write", "write_decode_32", n=32, spread=32, pad=3),
        # the 128K-token prefill, read back as its attention sees it
        _slots("write", "write_131k", n=131072, spread=1),
        # a prefix of an odd length for a prompt that goes on from it, small blocks
        _slots("read", "read_prefix_5003_b16", n=5003, spread=1, block=16),
        # the selected keys (2,048 each) of 32 rows, in no order
        _slots("read", "read_65536_spread", n=65536, spread=65536),
        # one user's next token over 8K keys, 16 heads
        _attn("attn4_decode_1_h16", decodes=1, d_lo=8191, d_hi=8191, shape=31, heads=16),
        # the decode rows of the varlen batch, 16 heads a GPU: bound by reading the cache
        _attn("attn4_decode_32_h16", decodes=32, d_lo=4096, d_hi=131072, shape=32, heads=16),
        # the same rows with 64 heads
        _attn("attn4_decode_32_h64", decodes=32, d_lo=4096, d_hi=131072, shape=32, heads=64),
        # many short contexts, all 128 heads, odd lengths, small blocks
        _attn("attn4_decode_97_h128_b16", decodes=97, d_lo=0, d_hi=4097, block=16, pad=3, shape=34,
              heads=128),
        # the 8K-token prefill, 16 heads
        _attn("attn4_prefill_8k_h16", prefills=1, p_lo=8192, p_hi=8192, shape=35, heads=16),
        # chunked prefill and decode rows in one step, 64 heads, a sliding window
        _attn("attn4_chunks_h64_window", prefills=3, p_lo=100, p_hi=1500, pc_hi=16384, decodes=9,
              d_lo=1, d_hi=16384, block=128, shape=36, heads=64, mask="window"),
    ]


def _log(rng, lo, hi):
    return int(round(2.0 ** rng.uniform(np.log2(lo), np.log2(hi))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attn", "attn", "attn"])
    block = rng.choice([16, 32, 64, 128])
    pad = rng.choice([0, 0, rng.randint(1, 40)])
    if op == "rope":
        heads = rng.choice([1, 5, 8, 16, 20, 32, 64, 128])
        return _rope(n=_log(rng, 1, 500000 // (heads + 1)), heads=heads, wide=rng.choice([64, 192, 576]),
                     pos_hi=_log(rng, 1, 1 << 24), base=rng.choice([1e4, 5e5, 8e6]),
                     factor=rng.choice([1.0, 4.0, 40.0]), interleaved=rng.random() < 0.5,
                     inverse=rng.random() < 0.3, pad=pad)
    if op != "attn":
        n = _log(rng, 1, 100000 if op == "write" else 60000)
        return _slots(op, n=n, spread=rng.choice([1, n, rng.randint(1, min(n, 2000))]), block=block,
                      pad=pad)
    heads = rng.choice([1, 4, 8, 16, 20, 32, 48, 64, 128])
    mask = rng.choice(["causal", "causal", "window", "gaps"])
    shape = rng.randint(1, 1 << 30)
    if rng.random() < 0.5:
        d_hi = _log(rng, 1, 65536)
        top = min(128, 1 + (1 << 20) // (d_hi * (1 + heads // 64)))
        return _attn(decodes=rng.randint(1, top), d_lo=rng.randint(0, d_hi), d_hi=d_hi, block=block,
                     pad=pad, shape=shape, heads=heads, mask=mask)
    p_hi = _log(rng, 2, 1500)
    pc_hi = rng.randint(0, max(1, min(8192, (1 << 24) // (p_hi * heads))))
    return _attn(prefills=rng.randint(1, 4), p_lo=1, p_hi=p_hi, pc_hi=pc_hi,
                 decodes=rng.randint(0, 6), d_lo=0, d_hi=_log(rng, 1, 4096), block=block, pad=pad,
                 shape=shape, heads=heads, mask=mask)


def _lengths(case):
    """(tokens in the cache before the step, tokens scheduled) of each request."""
    r = random.Random(case["shape"])
    ctx, new = [], []
    for _ in range(case["prefills"]):
        new.append(r.randint(case["p_lo"], case["p_hi"]))
        ctx.append(r.randint(0, case["pc_hi"]))
    for _ in range(case["decodes"]):
        new.append(1)
        ctx.append(r.randint(case["d_lo"], case["d_hi"]))
    return np.array(ctx, np.int64), np.array(new, np.int64)


def _token_arrays(case):
    """(request, position, lower bound, upper bound) of every scheduled token, on the host."""
    ctx, new = _lengths(case)
    req = np.repeat(np.arange(len(new)), new)
    first = np.repeat(np.cumsum(new) - new, new)
    pos = ctx[req] + np.arange(len(req)) - first
    lo, hi = np.zeros_like(pos), pos.copy()
    if case["mask"] == "window":      # the last 4096 keys
        lo = np.maximum(0, pos - 4095)
    elif case["mask"] == "gaps":      # every fifth row sees nothing, every seventh only the first half
        hi = np.where(np.arange(len(pos)) % 7 == 3, pos // 2, hi)
        lo = np.where(np.arange(len(pos)) % 5 == 2, pos + 1, lo)
    return req, pos, lo, hi


def work(case):
    if case["op"] == "rope":
        rows = case["n"] * (case["heads"] + 1)
        return {"bytes": rows * 2 * 2 * DR + 4 * (case["n"] + case["pad"]), "flops": rows * 3 * DR}
    if case["op"] == "write":
        # rows and slots in; what the cache holds of a token; its values out
        return {"bytes": case["n"] * (2 * DQK + STRIP // 16 + 2 * DQK) + 8 * (case["n"] + case["pad"]),
                "flops": 3 * case["n"] * DQK}
    if case["op"] == "read":
        return {"bytes": case["n"] * (STRIP // 16 + 2 * DQK) + 8 * (case["n"] + case["pad"]),
                "flops": case["n"] * DQK}
    ctx, new = _lengths(case)
    T, B, H = int(new.sum()), len(new), case["heads"]
    req, pos, lo, hi = _token_arrays(case)
    pairs = int(np.maximum(0, hi - lo + 1).sum())
    # keys that at least one row of the request attends to
    first = np.full(B, 1 << 40)
    last = np.full(B, -1)
    some = hi >= lo
    np.minimum.at(first, req[some], lo[some])
    np.maximum.at(last, req[some], hi[some])
    keys = int(np.maximum(0, last - first + 1).sum())
    return {"bytes": keys * (STRIP // 16) + T * H * (2 * DQK + 2 * DV + 4),
            "flops": pairs * H * (2 * DQK + 2 * DV)}


# ---------------------------------------------------------------- the format
def _value2(mag):
    """Value of an E2M1 magnitude code 0..7: 0, 1/2, 1, 3/2, 2, 3, 4, 6."""
    m = mag.float()
    return torch.where(m < 4, 0.5 * m, torch.where(m < 6, m - 2, 2 * m - 8))


def _pow2(e):
    """2^e in fp32 for integer e within its normal range."""
    return ((e.to(torch.int32) + EXP_BIAS) << 23).view(torch.float32)


def _least(amax, c, bits):
    """The least s with amax <= c 2^(s + bits), c in [1/2, 1)."""
    m, k = torch.frexp(amax)
    return torch.where(m <= c, k, k + 1) - bits


def _encode(x):
    """Rows x [n, 576] fp32 -> codes [n, 256], rope [n, 64], offsets [n, 16], exponents [n]."""
    n = x.shape[0]
    fin = torch.where(x.isfinite(), x.abs(), 0.0)
    amax = fin.amax(1)
    e = torch.where(amax > 0, _least(amax, 0.875, 9), EXP_MIN).clamp(EXP_MIN, EXP_MAX)
    ga = fin[:, :DV].view(n, 32, 16).amax(2)
    d = torch.where(ga > 0, e[:, None] + 6 - _least(ga, 0.875, 3), OFF_MAX).clamp(0, OFF_MAX)
    v = x[:, :DV].view(n, 32, 16) * _pow2(d - e[:, None] - 6)[..., None]
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = torch.round(a / step) * step
    mag = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, 0.5 * a + 4)).clamp(0, 7)
    mag = torch.where(a.isnan(), 0.0, mag).to(torch.int32)
    sign = (v < 0).to(torch.int32)
    mag, sign = mag.view(n, 32, 2, 8), sign.view(n, 32, 2, 8)
    # byte b of a word of 8 codes: magnitudes 2 b and 2 b + 1, signs of codes b and b + 4
    byte = (mag[..., 0::2] | (mag[..., 1::2] << 4) | (sign[..., :4] << 7) | (sign[..., 4:] << 3))
    # group g lies at 16 (g % 16) + 8 (g / 16)
    byte = byte.view(n, 2, 16, 8).transpose(1, 2).reshape(n, 256)
    rope = (x[:, DV:] * _pow2(-e)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    off = d[:, :16] | (d[:, 16:] << 4)
    ex = torch.where(x.isnan().any(1), 255, e + EXP_BIAS)
    u8 = torch.uint8
    return byte.to(u8), rope.view(u8), off.to(u8), ex.to(u8)


def _parts(cache):
    """The parts of the strips of a cache, by token: codes, rope, offsets, exponents."""
    s = cache.view(-1, STRIP)
    n = s.shape[0]
    return (s[:, :ROPE_AT].view(n, 16, 256), s[:, ROPE_AT:OFF_AT].view(n, 16, 64),
            s[:, OFF_AT:EXP_AT].view(n, 16, 16), s[:, EXP_AT:])


def _fetch(cache, slot):
    """The values in fp32 of the tokens in these slots (a tensor of any shape)."""
    codes, rope, off, ex = (p[slot // 16, slot % 16] for p in _parts(cache))
    shape = tuple(slot.shape)
    b = codes.view(*shape, 16, 2, 8).transpose(-3, -2).reshape(*shape, 32, 2, 4)
    del codes
    mag = torch.stack((b & 7, (b >> 4) & 7), -1).reshape(*shape, 32, 2, 8)
    sign = torch.cat((b >> 7, (b >> 3) & 1), -1)
    e = ex.to(torch.int32).clamp(EXP_MIN + EXP_BIAS, EXP_MAX + EXP_BIAS) - EXP_BIAS
    d = torch.cat((off & 15, off >> 4), -1).to(torch.int32).clamp(0, OFF_MAX)
    kv = torch.empty((*shape, DQK), device=slot.device)
    lat = torch.where(sign > 0, -_value2(mag), _value2(mag)).view(*shape, 32, 16)
    lat *= _pow2(e[..., None] + 6 - d)[..., None]
    kv[..., :DV] = lat.view(*shape, DV)
    kv[..., DV:] = rope.view(torch.float8_e4m3fn).float() * _pow2(e)[..., None]
    return kv.masked_fill_((ex == 255)[..., None], float("nan"))


# ---------------------------------------------------------------- inputs
def _cache(n_blocks, block, g, dev):
    """A cache as earlier steps left it: latents of about unit size, token by token on a
    scale of their own, a few channels larger."""
    n = n_blocks * block
    cache = torch.empty((n_blocks, block // 16, STRIP), dtype=torch.uint8, device=dev)
    parts = _parts(cache)
    wide = torch.exp2(2 * torch.randn((DQK,), generator=g, device=dev).clamp(-2, 2))
    for a in range(0, n, 1 << 18):
        z = min(n, a + (1 << 18))
        x = torch.randn((z - a, DQK), generator=g, device=dev) * (0.3 * wide)
        x *= torch.exp2(torch.randn((z - a, 1), generator=g, device=dev))
        for p, v in zip(parts, _encode(x.to(torch.bfloat16).float())):
            p[a // 16:z // 16] = v.view(-1, 16, *p.shape[2:])
    return cache


def _freqs(case):
    """32 frequencies 1 / base^(2i / 64), those of long waves divided by the factor, with
    a ramp between (the scaling of "YaRN", Peng et al. 2023, trained on 4096 positions)."""
    i = np.arange(32, dtype=np.float64)
    f = case["base"] ** (-i / 32)
    if case["factor"] == 1:
        return f
    at = lambda turns: DR * np.log(4096 / (turns * 2 * np.pi)) / (2 * np.log(case["base"]))
    low, high = max(0.0, np.floor(at(32.0))), min(DR - 1.0, np.ceil(at(1.0)))
    ramp = np.clip((i - low) / max(high - low, 0.001), 0, 1)
    return f * (1 - ramp) + f / case["factor"] * ramp


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 1000003 + 29)
    if case["op"] == "rope":
        n, H, w = case["n"], case["heads"], case["wide"]
        cap = n + case["pad"]
        pos = torch.randint(0, case["pos_hi"], (cap,), generator=g, device=dev, dtype=torch.int32)
        pos[n:] = -1
        # the projections' outputs, whose last 64 channels are the rope's, and the
        # 576-wide rows that the attention and the cache take
        bf = torch.bfloat16
        return dict(op="rope", pos=pos, f=_freqs(case), amp=0.1 * np.log(case["factor"]) + 1,
                    pairs=case["interleaved"], inverse=case["inverse"],
                    q=torch.randn((cap, H, w), generator=g, device=dev, dtype=bf),
                    k=torch.randn((cap, DQK), generator=g, device=dev, dtype=bf),
                    q_out=torch.zeros((cap, H, DQK), dtype=bf, device=dev),
                    k_out=torch.zeros((cap, DQK), dtype=bf, device=dev))
    if case["op"] in ("write", "read"):
        n, bs, runs = case["n"], case["block"], case["spread"]
        first = np.arange(runs) * n // runs
        length = np.diff(np.append(first, n))
        per = -(-length // bs) + 1                       # blocks of each request
        n_blocks = int(per.sum())
        if runs == n:                                    # single tokens: fewer blocks do
            n_blocks = max(1, -(-2 * n // bs))
            slot = torch.randperm(n_blocks * bs, generator=g, device=dev)[:n]
        else:
            perm = torch.randperm(n_blocks, generator=g, device=dev)
            run = torch.from_numpy(np.repeat(np.arange(runs), length)).to(dev)
            start = torch.from_numpy(np.cumsum(per) - per).to(dev)
            shift = torch.randint(0, bs, (runs,), generator=g, device=dev)
            p = torch.arange(n, device=dev) - torch.from_numpy(first).to(dev)[run] + shift[run]
            slot = perm[start[run] + p // bs] * bs + p % bs
        s = dict(op=case["op"], n=n, slot=torch.cat([slot, slot.new_full((case["pad"],), -1)]))
        cap = len(s["slot"])
        s["cache"] = _cache(n_blocks, bs, g, dev)
        s["out"] = torch.empty((cap, DQK), dtype=torch.bfloat16, device=dev)
        if case["op"] == "write":
            size = torch.exp2(torch.randn((cap, 1), generator=g, device=dev))  # tokens differ in size
            s["kv"] = (torch.randn((cap, DQK), generator=g, device=dev) * size).to(torch.bfloat16)
        return s

    ctx, new = _lengths(case)
    bs, B, T, H = case["block"], len(new), int(new.sum()), case["heads"]
    cap = T + case["pad"]
    held = -(-(ctx + new) // bs)
    n_blocks = int(held.sum()) + 7
    # the pool hands out blocks in no order: request b's i-th block is perm[start_b + i]
    perm = torch.randperm(n_blocks, generator=g, device=dev, dtype=torch.int32)
    held_t = torch.from_numpy(held).to(dev)
    start = torch.from_numpy(np.cumsum(held) - held).to(dev)
    col = torch.arange(int(held.max()), device=dev)[None, :]
    table = torch.where(col < held_t[:, None],
                        perm[(start[:, None] + col).clamp_max(n_blocks - 1)], -1).to(torch.int32)
    req, pos, lo, hi = _token_arrays(case)
    tail = np.full(case["pad"], -1)
    i32 = lambda a: torch.from_numpy(np.concatenate([a, tail])).to(dev, torch.int32)
    s = dict(op="attn", block=bs, table=table, req=i32(req), pos=i32(pos),
             cache=_cache(n_blocks, bs, g, dev),
             q=torch.randn((cap, H, DQK), generator=g, device=dev, dtype=torch.bfloat16),
             sink=torch.randn((H,), generator=g, device=dev), scale=DQK ** -0.5,
             o=torch.zeros((cap, H, DV), dtype=torch.bfloat16, device=dev),
             lse=torch.zeros((cap, H), dtype=torch.float32, device=dev), lo=None, hi=None,
             max_new=int(new.max()), n_req=B, prefills=case["prefills"],
             max_len=[int((ctx + new)[:case["prefills"]].max(initial=0)),
                      int((ctx + new)[case["prefills"]:].max(initial=0))],
             cu=torch.from_numpy(np.concatenate([[0], np.cumsum(new)])).to(dev))
    if case["mask"] != "causal":
        s["lo"], s["hi"] = i32(lo), i32(hi)
    if own:
        from context_sparse_mla_gb300 import cpmla
        s["ws"] = cpmla.paged_attn_workspace(H, cap)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    if own:
        from context_sparse_mla_gb300 import cpmla
        if s["op"] == "rope":
            cpmla.mla_rope(s["q"][..., -DR:], s["pos"], s["f"], k=s["k"][:, DV:],
                           q_out=s["q_out"][..., DV:], k_out=s["k_out"][:, DV:], amplitude=s["amp"],
                           interleaved=s["pairs"], inverse=s["inverse"])
            return {"q": s["q_out"][..., DV:], "k": s["k_out"][:, DV:]}
        if s["op"] == "attn":
            cpmla.mla_paged4_attn(s["q"], s["cache"], s["table"], s["pos"], s["req"], s["o"],
                                  s["lse"], softmax_scale=s["scale"], sink=s["sink"],
                                  kv_lo=s["lo"], kv_hi=s["hi"], workspace=s["ws"])
            return {"o": s["o"], "lse": s["lse"]}
        if s["op"] == "write":
            cpmla.mla_paged4_cache_insert(s["kv"], s["slot"], s["cache"])
        return {"kv": cpmla.mla_paged4_cache_read(s["cache"], s["slot"], out=s["out"])}
    if s["op"] == "rope":
        return _plain_rope(s)
    if s["op"] == "attn":
        return _plain_attn(s)
    there = s["slot"] >= 0
    slot = s["slot"][there]
    if s["op"] == "write":
        for p, v in zip(_parts(s["cache"]), _encode(s["kv"][there].float())):
            p[slot // 16, slot % 16] = v
    s["out"].zero_()
    s["out"][there] = _fetch(s["cache"], slot).to(torch.bfloat16)
    return {"kv": s["out"]}


def _plain_rope(s):
    there = s["pos"] >= 0
    ang = s["pos"][there].double()[:, None] * torch.from_numpy(s["f"]).to(s["pos"].device)
    cos, sin = (ang.cos() * s["amp"]).float(), (ang.sin() * s["amp"]).float()
    if s["inverse"]:
        sin = -sin
    for src, dst in ((s["q"][..., -DR:], s["q_out"][..., DV:]),
                     (s["k"][:, None, DV:], s["k_out"][:, None, DV:])):
        x = src[there].float()
        c, i = cos[:, None], sin[:, None]
        if s["pairs"]:
            a, b = x[..., 0::2], x[..., 1::2]
            y = torch.stack((a * c - b * i, a * i + b * c), -1).view(x.shape)
        else:
            a, b = x[..., :32], x[..., 32:]
            y = torch.cat((a * c - b * i, a * i + b * c), -1)
        dst[there] = y.to(torch.bfloat16)
    return {"q": s["q_out"][..., DV:], "k": s["k_out"][:, DV:]}


def _plain_attn(s):
    # the requests with several new tokens, then those with one
    n = s["prefills"]
    if n:
        _plain_rows(s, slice(0, n), s["max_new"], s["max_len"][0])
    if n < s["n_req"]:
        _plain_rows(s, slice(n, s["n_req"]), 1, s["max_len"][1])
    return {"o": s["o"], "lse": s["lse"]}


def _plain_rows(s, which, Qn, L):
    bs, table = s["block"], s["table"][which].long()
    H, B, dev = s["q"].shape[1], table.shape[0], table.device
    k = torch.arange(L, device=dev)
    blk = table[:, k // bs]                                         # [B, L]
    there = blk >= 0
    kv = _fetch(s["cache"], blk.clamp_min(0) * bs + k % bs)
    kv.masked_fill_(~there[..., None], 0.0)
    i = s["cu"][:-1][which][:, None] + torch.arange(Qn, device=dev)  # [B, Qn]: the tokens
    real = i < s["cu"][1:][which][:, None]
    i = torch.where(real, i, 0)
    q = s["q"][i].float().reshape(B, Qn * H, DQK)
    x = torch.bmm(q, kv.transpose(1, 2)).mul_(s["scale"]).view(B, Qn, H, L)
    hide = (k > s["pos"][i][..., None]) | ~there[:, None, :]
    if s["lo"] is not None:
        hide |= (k < s["lo"][i][..., None]) | (k > s["hi"][i][..., None])
    x.masked_fill_(hide[:, :, None, :], float("-inf"))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m.isinf(), 0.0, m)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.bmm(p.view(B, Qn * H, L), kv[..., :DV]).view(B, Qn, H, DV)
    lse = (m + l.log())[..., 0]
    f = 1 / (l * (1 + torch.exp(s["sink"][:, None] - lse[..., None])))
    o = torch.where(l > 0, o * f, 0.0)
    s["o"][i[real]] = o[real].to(torch.bfloat16)
    s["lse"][i[real]] = lse[real]


# ---------------------------------------------------------------- in 64 bits
def _f64(values):
    return torch.tensor(values, dtype=torch.float64, device="cuda")


def _two(e):
    """2^e exactly, for whole e."""
    return _f64([2.0 ** i for i in range(-200, 201)])[e.long() + 200]


def _e2m1():
    return _f64([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def _e4m3():
    """The values of codes 0 .. 126."""
    return _f64([m * 2.0 ** -9 if ex == 0 else (8 + m) * 2.0 ** (ex - 10)
                 for ex in range(16) for m in range(8)][:127])


def _nearest(v, grid):
    """The grid value nearest to |v|, ties to the one of even index, with v's sign."""
    mid = (grid[1:] + grid[:-1]) / 2
    a = v.abs().contiguous()
    below, above = torch.bucketize(a, mid), torch.bucketize(a, mid, right=True)
    return v.sign() * grid[torch.where(below % 2 == 0, below, above)]


def _quantised(x):
    """What the cache holds of rows x (float64, finite)."""
    top = x.abs().amax(1)
    e = _f64([EXP_MIN]).repeat(len(x))
    for _ in range(EXP_MAX - EXP_MIN):
        e += (top > 448 * _two(e)) & (e < EXP_MAX)
    y = x[:, :DV].reshape(-1, 32, 16)
    s = (e[:, None] + 6 - OFF_MAX).repeat(1, 32)
    for _ in range(OFF_MAX):
        s += (y.abs().amax(2) > 7 * _two(s)) & (s < e[:, None] + 6)
    unit = _two(s)[..., None]
    low = _nearest(y / unit, _e2m1()) * unit
    unit = _two(e)[:, None]
    return torch.cat([low.flatten(1), _nearest(x[:, DV:] / unit, _e4m3()) * unit], 1)


def _held(cache, slot):
    """The values (float64) of slots of the cache, byte by byte from its layout."""
    at = slot[:, None] // 16 * STRIP
    r = slot[:, None] % 16
    flat = cache.view(-1)
    col = lambda n: torch.arange(n, device=slot.device)
    g, j = col(DV) // 16, col(DV) % 8                    # of each latent channel: group, code
    word = 16 * (g % 16) + 8 * (g // 16) + col(DV) % 16 // 8 * 4
    mag = flat[at + 256 * r + word + j // 2].long() >> (4 * (j % 2)) & 7
    neg = flat[at + 256 * r + word + j % 4].long() >> torch.where(j < 4, 7, 3) & 1
    off = flat[at + OFF_AT + 16 * r + g % 16].long() >> (4 * (g // 16)) & 15
    e = flat[at + EXP_AT + r].double() - EXP_BIAS
    low = _e2m1()[mag] * (1.0 - 2 * neg) * _two(e + 6 - off)
    c = flat[at + ROPE_AT + 64 * r + col(DR)].long()
    return torch.cat([low, _e4m3()[c & 127] * (1.0 - 2 * (c >> 7)) * _two(e)], 1)


def _all_held(cache, slot):
    return torch.cat([_held(cache, x) for x in slot.split(1 << 16)])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        n = case["n"]
        ang = s["pos"][:n].cpu().numpy().astype(np.float64)[:, None] * s["f"]
        if case["inverse"]:
            ang = -ang
        turn = torch.from_numpy(s["amp"] * np.exp(1j * ang)).cuda()[:, None]
        out = {}
        for name, src in (("q", s["q"][:, :, -DR:]), ("k", s["k"][:, None, DV:])):
            x = src.double().contiguous()
            z = x.unflatten(-1, (32, 2)) if case["interleaved"] else \
                x.unflatten(-1, (2, 32)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(z[:n].contiguous()) * turn)
            y = torch.zeros_like(x)
            y[:n] = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
            out[name] = y if name == "q" else y[:, 0]
        return out
    if case["op"] in ("write", "read"):
        n = case["n"]
        out = torch.zeros((len(s["slot"]), DQK), dtype=torch.float64, device="cuda")
        if case["op"] == "write":
            out[:n] = torch.cat([_quantised(x.double()) for x in s["kv"][:n].split(1 << 15)])
        else:
            out[:n] = _all_held(s["cache"], s["slot"][:n])
        return {"kv": out}
    bs, H, dev = case["block"], case["heads"], s["q"].device
    ctx, new = _lengths(case)
    _, pos, lo, hi = _token_arrays(case)
    cap = len(s["pos"])
    o = torch.zeros((cap, H, DV), dtype=torch.float64, device=dev)
    lse = torch.zeros((cap, H), dtype=torch.float64, device=dev)
    sink = s["sink"].double()
    t0 = 0
    for b in range(len(new)):
        n = int(ctx[b] + new[b])
        p = torch.arange(n, device=dev)
        kv = _all_held(s["cache"], s["table"][b, p // bs].long() * bs + p % bs)
        step = max(1, (1 << 28) // (n * H))
        for a in range(t0, t0 + int(new[b]), step):
            z = min(t0 + int(new[b]), a + step)
            top = int(max(1, hi[a:z].max() + 1))
            x = torch.einsum("thd,kd->thk", s["q"][a:z].double(), kv[:top]) * DQK ** -0.5
            k = torch.arange(top, device=dev)[None, :]
            see = (k >= torch.from_numpy(lo[a:z]).to(dev)[:, None]) & \
                (k <= torch.from_numpy(hi[a:z]).to(dev)[:, None])
            x = torch.where(see[:, None, :], x, -float("inf"))
            w = torch.logsumexp(x, -1)
            wt = torch.where(w.isinf()[..., None], 0.0, torch.exp(x - w[..., None]))
            gate = torch.where(w.isinf(), 0.0, torch.sigmoid(w - sink))
            o[a:z] = torch.einsum("thk,kd->thd", wt, kv[:top, :DV]) * gate[..., None]
            lse[a:z] = w
        t0 += int(new[b])
    return {"o": o, "lse": lse}
