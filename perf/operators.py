"""Measured cases of the paged 8-bit latent cache: the step's block tables and
slot maps, the insertion of a step's tokens, and the attention that reads it.

A batch is `prefills` requests that schedule p_lo..p_hi new tokens on top of a
context of up to pc_hi cached ones, then `decodes` requests that schedule one
token on top of d_lo..d_hi; the lengths are drawn from `shape`, so that a
case's work is known without its inputs.  `pad` list entries behind the last
request belong to no token (a batch padded to a captured size).

The plain forms are written with elementary torch operations in fp32; `exact`
computes the same from the definitions in 64 bits.
"""
import random

import numpy as np
import torch

own = False

DQK, DV = 576, 512
EXP_MIN = -64   # a block's exponent is at least this ...
EXP_BIAS = 127  # ... and is stored with this bias


# ---------------------------------------------------------------- the cases
def _batch(op, name=None, prefills=0, p_lo=1, p_hi=1, pc_hi=0, decodes=0, d_lo=0, d_hi=0,
           block=64, pad=0, shape=1, heads=0, mask="causal"):
    c = dict(op=op, prefills=prefills, p_lo=p_lo, p_hi=p_hi, pc_hi=pc_hi, decodes=decodes,
             d_lo=d_lo, d_hi=d_hi, block=block, pad=pad, shape=shape)
    if op == "attn":
        c.update(heads=heads, mask=mask)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one user's next token: latency only
        _batch("maps", "maps_decode_1", decodes=1, d_lo=8191, d_hi=8191, shape=11),
        # a full decode batch, padded to a captured size
        _batch("maps", "maps_decode_500", decodes=500, d_lo=0, d_hi=131072, pad=12, shape=12),
        # the mixed varlen batch: 8 prefills of up to 64K tokens and 32 decode rows
        _batch("maps", "maps_varlen", prefills=8, p_lo=1024, p_hi=65536, decodes=32, d_lo=4096,
               d_hi=131072, shape=13),
        # 32 decode rows, each raising or keeping the scale of its last block
        _batch("insert", "insert_decode_32", decodes=32, d_lo=1, d_hi=8192, shape=21),
        # prompts of one step, continuing half-filled blocks, small blocks
        _batch("insert", "insert_chunks_b16", prefills=7, p_lo=1, p_hi=2048, pc_hi=4099,
               decodes=5, d_lo=1, d_hi=4096, block=16, pad=3, shape=22),
        # the 128K-token prefill
        _batch("insert", "insert_131k", prefills=1, p_lo=131072, p_hi=131072, shape=23),
        # one user's next token over 8K keys, 16 heads
        _batch("attn", "attn_decode_1_h16", decodes=1, d_lo=8191, d_hi=8191, shape=31, heads=16),
        # the decode rows of the varlen batch, 16 heads a GPU: bound by reading the cache
        _batch("attn", "attn_decode_32_h16", decodes=32, d_lo=4096, d_hi=131072, shape=32,
               heads=16),
        # the same rows with 64 heads
        _batch("attn", "attn_decode_32_h64", decodes=32, d_lo=4096, d_hi=131072, shape=32,
               heads=64),
        # many short contexts, all 128 heads, odd lengths, small blocks
        _batch("attn", "attn_decode_97_h128_b16", decodes=97, d_lo=0, d_hi=4097, block=16, pad=3,
               shape=34, heads=128),
        # the 8K-token prefill, 16 heads
        _batch("attn", "attn_prefill_8k_h16", prefills=1, p_lo=8192, p_hi=8192, shape=35,
               heads=16),
        # chunked prefill and decode rows in one step, 64 heads, a sliding window
        _batch("attn", "attn_chunks_h64_window", prefills=3, p_lo=100, p_hi=1500, pc_hi=16384,
               decodes=9, d_lo=1, d_hi=16384, block=128, shape=36, heads=64, mask="window"),
    ]


def _log(rng, lo, hi):
    return int(round(2.0 ** rng.uniform(np.log2(lo), np.log2(hi))))


def draw(rng):
    op = rng.choice(["maps", "insert", "attn", "attn"])
    block = rng.choice([16, 32, 64, 128])
    pad = rng.choice([0, 0, rng.randint(1, 40)])
    shape = rng.randint(1, 1 << 30)
    if op == "maps":
        return _batch(op, prefills=rng.randint(0, 8), p_lo=1, p_hi=_log(rng, 2, 40000),
                      pc_hi=rng.randint(0, 20000), decodes=rng.randint(1, 600), d_lo=0,
                      d_hi=_log(rng, 1, 131072), block=block, pad=pad, shape=shape)
    if op == "insert":
        return _batch(op, prefills=rng.randint(0, 8), p_lo=1, p_hi=_log(rng, 2, 12000),
                      pc_hi=rng.randint(0, 4096), decodes=rng.randint(1, 64), d_lo=0,
                      d_hi=_log(rng, 1, 8192), block=block, pad=pad, shape=shape)
    heads = rng.choice([1, 4, 8, 16, 20, 32, 48, 64, 128])
    mask = rng.choice(["causal", "causal", "window", "gaps"])
    if rng.random() < 0.5:
        d_hi = _log(rng, 1, 65536)
        return _batch(op, decodes=rng.randint(1, min(128, 1 + (1 << 20) // (d_hi * (1 + heads // 64)))),
                      d_lo=rng.randint(0, d_hi), d_hi=d_hi, block=block, pad=pad, shape=shape,
                      heads=heads, mask=mask)
    p_hi = _log(rng, 2, 1500)
    pc_hi = rng.randint(0, max(1, min(8192, (1 << 24) // (p_hi * heads))))
    return _batch(op, prefills=rng.randint(1, 4), p_lo=1, p_hi=p_hi, pc_hi=pc_hi,
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
    mask = case.get("mask", "causal")
    if mask == "window":      # the last 4096 keys
        lo = np.maximum(0, pos - 4095)
    elif mask == "gaps":      # every fifth row sees nothing, every seventh only the first half
        hi = np.where(np.arange(len(pos)) % 7 == 3, pos // 2, hi)
        lo = np.where(np.arange(len(pos)) % 5 == 2, pos + 1, lo)
    return req, pos, lo, hi


def work(case):
    ctx, new = _lengths(case)
    bs, T, B = case["block"], int(new.sum()), len(new)
    if case["op"] == "maps":
        taken = int((-(-(ctx + new) // bs) - -(-ctx // bs)).sum())
        cap = T + case["pad"]
        # lengths; free blocks in, table entries out; slot, position and request of each entry;
        # the partly filled block of each request; the offsets
        return {"bytes": 8 * B + 8 * taken + 16 * cap + 4 * B + 4 * (B + 1), "flops": 0}
    if case["op"] == "insert":
        blocks = int((-(-(ctx + new) // bs) - ctx // bs).sum())
        return {"bytes": T * (2 * DQK + DQK + 8) + 2 * blocks, "flops": 2 * T * DQK}
    req, pos, lo, hi = _token_arrays(case)
    H = case["heads"]
    pairs = int(np.maximum(0, hi - lo + 1).sum())
    # keys that at least one row of the request attends to
    first = np.full(B, 1 << 40)
    last = np.full(B, -1)
    some = hi >= lo
    np.minimum.at(first, req[some], lo[some])
    np.maximum.at(last, req[some], hi[some])
    keys = int(np.maximum(0, last - first + 1).sum())
    return {"bytes": keys * DQK + T * H * (2 * DQK + 2 * DV + 4),
            "flops": pairs * H * (2 * DQK + 2 * DV)}


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 1000003 + 17)
    ctx, new = _lengths(case)
    bs, B = case["block"], len(new)
    T = int(new.sum())
    cap = T + case["pad"]
    held = -(-ctx // bs) if case["op"] == "maps" else -(-(ctx + new) // bs)
    width = int((-(-(ctx + new) // bs)).max())
    n_blocks = int((-(-(ctx + new) // bs)).sum()) + 7
    # the pool hands out blocks in no order: request b's i-th block is perm[start_b + i]
    perm = torch.randperm(n_blocks, generator=g, device=dev, dtype=torch.int32)
    held_t = torch.from_numpy(held).to(dev)
    start = torch.from_numpy(np.cumsum(held) - held).to(dev)
    col = torch.arange(width, device=dev)[None, :]
    table = torch.where(col < held_t[:, None],
                        perm[(start[:, None] + col).clamp_max(n_blocks - 1)], -1).to(torch.int32)
    s = dict(op=case["op"], block=bs, n_blocks=n_blocks, table=table, cap=cap)
    if case["op"] == "maps":
        s.update(ctx=torch.from_numpy(ctx).to(dev, torch.int32),
                 new=torch.from_numpy(new).to(dev, torch.int32),
                 free=perm[int(held.sum()):].contiguous(),
                 head=torch.zeros(1, dtype=torch.int32, device=dev),
                 out=dict(cu_seqlens=torch.empty(B + 1, dtype=torch.int32, device=dev),
                          slot_mapping=torch.empty(cap, dtype=torch.int64, device=dev),
                          pos=torch.empty(cap, dtype=torch.int32, device=dev),
                          req=torch.empty(cap, dtype=torch.int32, device=dev),
                          free_head=torch.empty(1, dtype=torch.int32, device=dev)))
        return s

    # the cache as earlier steps left it: latents of about unit size, block by
    # block on a scale of their own; blocks that nobody holds keep old bytes
    x = torch.randn((n_blocks, bs, DQK), generator=g, device=dev, dtype=torch.bfloat16)
    s["exp"] = torch.randint(EXP_BIAS - 6, EXP_BIAS - 2, (n_blocks,), generator=g, device=dev,
                             dtype=torch.uint8)
    inv = torch.exp2(EXP_BIAS - s["exp"].float())[:, None, None]
    s["cache"] = (x * inv.to(torch.bfloat16)).clamp_(-448, 448).to(torch.float8_e4m3fn) \
        .view(torch.uint8)
    del x
    req, pos, lo, hi = _token_arrays(case)
    tail = np.full(case["pad"], -1)
    req_t = torch.from_numpy(np.concatenate([req, tail])).to(dev)
    pos_t = torch.from_numpy(np.concatenate([pos, tail])).to(dev)
    s.update(req=req_t.to(torch.int32), pos=pos_t.to(torch.int32))
    if case["op"] == "insert":
        blk = table.long()[req_t.clamp_min(0), pos_t.clamp_min(0) // bs]
        s["slot"] = torch.where(req_t >= 0, blk * bs + pos_t % bs, -1)
        size = torch.exp2(torch.randn((cap, 1), generator=g, device=dev))  # tokens differ in size
        s["kv"] = (torch.randn((cap, DQK), generator=g, device=dev) * size).to(torch.bfloat16)
        return s
    H = case["heads"]
    s.update(q=torch.randn((cap, H, DQK), generator=g, device=dev, dtype=torch.bfloat16),
             sink=torch.randn((H,), generator=g, device=dev), scale=DQK ** -0.5,
             o=torch.zeros((cap, H, DV), dtype=torch.bfloat16, device=dev),
             lse=torch.zeros((cap, H), dtype=torch.float32, device=dev), lo=None, hi=None,
             max_new=int(new.max()), n_req=B, prefills=case["prefills"],
             max_len=[int((ctx + new)[:case["prefills"]].max(initial=0)),
                      int((ctx + new)[case["prefills"]:].max(initial=0))],
             cu=torch.from_numpy(np.concatenate([[0], np.cumsum(new)])).to(dev))
    if case["mask"] != "causal":
        s["lo"] = torch.from_numpy(np.concatenate([lo, tail])).to(dev, torch.int32)
        s["hi"] = torch.from_numpy(np.concatenate([hi, tail])).to(dev, torch.int32)
    if own:
        from context_sparse_mla_gb300 import cpmla
        s["ws"] = cpmla.paged_attn_workspace(H, cap)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    if own:
        from context_sparse_mla_gb300 import cpmla
        if s["op"] == "maps":
            cpmla.mla_paged_maps(s["ctx"], s["new"], s["free"], s["table"], block_size=s["block"],
                                 n_blocks=s["n_blocks"], free_head=s["head"], out=s["out"])
            return {**s["out"], "table": s["table"]}
        if s["op"] == "insert":
            cpmla.mla_paged_cache_insert(s["kv"], s["slot"], s["cache"], s["exp"])
            return {"cache": s["cache"].view(torch.float8_e4m3fn), "exp": s["exp"]}
        cpmla.mla_paged_attn(s["q"], s["cache"], s["exp"], s["table"], s["pos"], s["req"], s["o"],
                             s["lse"], softmax_scale=s["scale"], sink=s["sink"], kv_lo=s["lo"],
                             kv_hi=s["hi"], workspace=s["ws"])
        return {"o": s["o"], "lse": s["lse"]}
    return {"maps": _plain_maps, "insert": _plain_insert, "attn": _plain_attn}[s["op"]](s)


def _plain_maps(s):
    bs, table, free = s["block"], s["table"], s["free"]
    ctx, new = s["ctx"].long(), s["new"].long()
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    i = torch.arange(s["cap"], device=cu.device)
    used = i < cu[-1]
    r = torch.searchsorted(cu[1:], i, right=True).clamp_max(len(new) - 1)
    pos = ctx[r] + i - cu[r]
    have = (ctx + bs - 1) // bs                 # blocks a request holds
    take = (ctx + new + bs - 1) // bs - have    # blocks it takes now
    at = s["head"].long() + take.cumsum(0) - take
    col = torch.arange(table.shape[1], device=cu.device)[None, :]
    fresh = (col >= have[:, None]) & (col < (have + take)[:, None])
    k = (at[:, None] + col - have[:, None]).clamp(0, max(0, len(free) - 1))
    table.copy_(torch.where(fresh, free[k], table))
    slot = table[r, (pos // bs).clamp_max(table.shape[1] - 1)].long() * bs + pos % bs
    none = torch.full_like(i, -1)
    out = s["out"]
    out["cu_seqlens"].copy_(cu)
    out["slot_mapping"].copy_(torch.where(used, slot, none))
    out["pos"].copy_(torch.where(used, pos, none))
    out["req"].copy_(torch.where(used, r, none))
    out["free_head"].copy_(s["head"] + take.sum())
    return {**out, "table": table}


def _exponent(amax):
    """The least e >= EXP_MIN with amax <= 448 * 2^e."""
    m, k = torch.frexp(amax)          # amax = m * 2^k, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, k - 9, k - 8)
    return torch.where(amax > 0, e, EXP_MIN).clamp_min(EXP_MIN)


def _plain_insert(s):
    bs, exp = s["block"], s["exp"]
    cache = s["cache"].view(torch.float8_e4m3fn)
    there = s["slot"] >= 0
    slot, x = s["slot"][there], s["kv"][there].float()
    blk, off = slot // bs, slot % bs
    e_tok = _exponent(torch.where(x.isfinite(), x.abs(), 0.0).amax(1)).to(torch.int32)
    low = torch.full((s["n_blocks"],), -1000, dtype=torch.int32, device=x.device)
    e_new = low.scatter_reduce(0, blk, e_tok, "amax")
    starts = torch.zeros_like(exp, dtype=torch.bool).scatter_(0, blk[off == 0], True)
    e_old = exp.int() - EXP_BIAS
    e = torch.where(starts, e_new, torch.maximum(e_old, e_new))
    grown = ((e > e_old) & ~starts & (e_new > -1000)).nonzero()[:, 0]
    down = torch.exp2((e_old - e)[grown].float())[:, None, None]
    cache.view(torch.uint8)[grown] = (cache.view(torch.uint8)[grown].view(torch.float8_e4m3fn)
                                      .float() * down).to(torch.float8_e4m3fn).view(torch.uint8)
    codes = (x * torch.exp2(-e[blk].float())[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    cache.view(torch.uint8).view(-1, DQK)[slot] = codes.view(torch.uint8)
    exp.copy_((e + EXP_BIAS).to(torch.uint8))
    return {"cache": cache, "exp": exp}


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
    row = blk.clamp_min(0) * bs + k % bs
    kv = s["cache"].view(-1, DQK)[row].view(torch.float8_e4m3fn).float()
    kv *= torch.where(there, torch.exp2(s["exp"].float() - EXP_BIAS)[blk.clamp_min(0)], 0.0)[..., None]
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
def _e4m3_exact(v):
    """The E4M3 value nearest to v (float64), ties to even, saturating."""
    a = v.abs().clamp_min(2.0 ** -40)
    step = torch.exp2(torch.floor(torch.log2(a)).clamp_min(-6) - 3)
    return ((v / step).round() * step).clamp(-448, 448)


def exact(case, seed):
    s = prepare(case, seed)
    bs = case["block"]
    if case["op"] == "maps":
        return None
    old = s["cache"].view(torch.float8_e4m3fn).double()
    e = s["exp"].cpu().numpy().astype(np.int64) - EXP_BIAS
    if case["op"] == "insert":
        slot = s["slot"].cpu().numpy()
        idx = np.flatnonzero(slot >= 0)
        slot = slot[idx]
        x = s["kv"][torch.from_numpy(idx).to(s["kv"].device)].double()
        amax = x.abs().amax(1).cpu().numpy()
        with np.errstate(divide="ignore"):
            need = np.where(amax > 0, np.ceil(np.log2(amax / 448.0)), EXP_MIN)
        need = np.maximum(need, EXP_MIN).astype(np.int64)
        blk = slot // bs
        e_new = np.full(len(e), -1000)
        np.maximum.at(e_new, blk, need)
        fresh = np.zeros(len(e), bool)
        fresh[blk[slot % bs == 0]] = True
        after = np.where(fresh, e_new, np.maximum(e, e_new))
        shift = np.where(fresh | (e_new == -1000), 0, e - after)
        for b in np.flatnonzero(shift):
            old[b] = _e4m3_exact(old[b] * 2.0 ** int(shift[b]))
        dev = x.device
        unit = torch.from_numpy(2.0 ** -after[blk].astype(np.float64)).to(dev)
        old.view(-1, DQK)[torch.from_numpy(slot).to(dev)] = _e4m3_exact(x * unit[:, None])
        return {"cache": old, "exp": None}
    ctx, new = _lengths(case)
    _, pos, lo, hi = _token_arrays(case)
    dev = old.device
    old *= torch.from_numpy(2.0 ** e.astype(np.float64)).to(dev)[:, None, None]
    H = case["heads"]
    o = torch.zeros((s["cap"], H, DV), dtype=torch.float64, device=dev)
    lse = torch.zeros((s["cap"], H), dtype=torch.float64, device=dev)
    sink = s["sink"].double()
    t0 = 0
    for b in range(len(new)):
        n = int(ctx[b] + new[b])
        kv = old[s["table"][b, :-(-n // bs)].long()].reshape(-1, DQK)[:n]
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
            p = torch.where(w.isinf()[..., None], 0.0, torch.exp(x - w[..., None]))
            gate = torch.where(w.isinf(), 0.0, torch.sigmoid(w - sink))
            o[a:z] = torch.einsum("thk,kd->thd", p, kv[:top, :DV]) * gate[..., None]
            lse[a:z] = w
        t0 += int(new[b])
    return {"o": o, "lse": lse}
