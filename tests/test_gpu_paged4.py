"""The 4-bit latent cache and the rotation on the GPU: rotation, insertion, reading
back, attention, and a run of them together, against plain 64-bit forms
(paged4_util)."""
import numpy as np
import pytest
import torch

import paged4_util as p4
import paged_util as pu
from context_sparse_mla_gb300 import cpmla

pytestmark = pytest.mark.gpu
SCALE = 576 ** -0.5
# Bounds of the attention, fixed from its arithmetic: binary32 sums of 576 products in
# 20 steps; nine bits of a weight.  O_TILE is the least step's: a weight is two E4M3 on a
# scale on which the largest of its row's 32 keys (each times its token's 2^e, which the
# weights carry) lies in (2^7, 2^8], and its second part is off by up to half of E4M3's
# least step, 2^-10: by 2^-17 of that largest.  (Many E2M1 codes are 0: the heaviest keys
# of a tile may add nothing to a channel.)
LSE_ABS, LSE_REL = 1e-4, 2e-6
O_REL, O_WEIGHT, O_TILE, O_NORM = 2.0 ** -8, 2.0 ** -7, 2.0 ** -17, 2.0 ** -8


@pytest.fixture(autouse=True)
def clean_status():
    cpmla.device_status(clear=True)
    yield


def gpu(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)) if isinstance(a, np.ndarray) else a
    return t.to("cuda", dtype) if dtype else t.to("cuda")


# ------------------------------------------------------------------ the rotation
def check_rope(got, x, pos, f, amp, pairs, inverse):
    """Rows of positions >= 0 (the others are compared by the caller).  Half a bf16 step
    of the result, and binary32: the angle is off by 2^-24 of half a turn, a sine and a
    cosine by 2^-23, products and the sum by 3 x 2^-24: below 6e-7 of |u| + |v|."""
    keep = pos >= 0
    x = x.double().cpu().numpy()[keep]
    want = p4.rotate(x, pos[keep], f, amp, pairs, inverse)
    size = np.abs(x[..., 0::2]) + np.abs(x[..., 1::2]) if pairs else \
        np.abs(x[..., :32]) + np.abs(x[..., 32:])
    size = np.repeat(size, 2, -1) if pairs else np.concatenate([size, size], -1)
    diff = np.abs(got.double().cpu().numpy()[keep] - want)
    assert (diff <= 2.0 ** -8 * np.abs(want) + 6e-7 * abs(amp) * size).all(), diff.max()


@pytest.mark.parametrize("n, H", [(1, 1), (1, 128), (3, 16), (33, 5), (257, 64), (1001, 20)])
@pytest.mark.parametrize("pairs", [True, False])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(n, H, pairs, inverse):
    g = torch.Generator().manual_seed(n + H)
    q = torch.randn((n, H, 192), generator=g).bfloat16()
    k = torch.randn((n, 576), generator=g).bfloat16()
    pos = torch.randint(0, 200000, (n,), generator=g, dtype=torch.int32)
    pos[::7] = torch.arange(len(pos[::7]), dtype=torch.int32)
    f, amp = cpmla.rope_freqs(factor=40.0), 1.37
    d = dict(q_out=torch.full((n, H, 576), 7.0, dtype=torch.bfloat16, device="cuda"),
             k_out=torch.full((n, 640), 7.0, dtype=torch.bfloat16, device="cuda"))
    qg, kg = gpu(q), gpu(k)
    ret = cpmla.mla_rope(qg[..., 128:], gpu(pos), f, k=kg[:, 512:], q_out=d["q_out"][..., 512:],
                         k_out=d["k_out"][:, 512:576], amplitude=amp, interleaved=pairs,
                         inverse=inverse)
    torch.cuda.synchronize()
    check_rope(ret[0], q[..., 128:], pos.numpy(), f, amp, pairs, inverse)
    check_rope(ret[1], k[:, 512:], pos.numpy(), f, amp, pairs, inverse)
    assert (d["q_out"][..., :512] == 7).all() and (d["k_out"][:, :512] == 7).all()
    assert (d["k_out"][:, 576:] == 7).all()
    assert torch.equal(qg, gpu(q)) and torch.equal(kg, gpu(k))
    # in place, queries and keys by themselves: the same bits
    cpmla.mla_rope(qg[..., 128:], gpu(pos), f, amplitude=amp, interleaved=pairs, inverse=inverse)
    cpmla.mla_rope(None, gpu(pos), f, k=kg[:, 512:], amplitude=amp, interleaved=pairs,
                   inverse=inverse)
    assert torch.equal(qg[..., 128:], ret[0]) and torch.equal(kg[:, 512:], ret[1])
    assert torch.equal(qg[..., :128], gpu(q)[..., :128])


def test_rope_far_positions_and_other_frequencies():
    """Every position of an int32, frequencies from 0 to 6 and down to 1e-12 a position."""
    g = torch.Generator().manual_seed(1)
    pos = torch.cat([torch.randint(0, 2 ** 31 - 1, (500,), generator=g),
                     torch.tensor([0, 1, 2 ** 24 + 1, 2 ** 30, 2 ** 31 - 1])]).to(torch.int32)
    x = torch.randn((505, 2, 64), generator=g).bfloat16()
    x[::3, 0, ::2] = 0  # a zero beside its partner: what is left is a product of the sine
    f = np.concatenate([[0, 6, 1e-12, 1e-9, 0.9999999], 10.0 ** -np.linspace(0, 8, 27)])
    # 64-bit angles are off by 2^-53 of up to 2^31 x 6: 1.5e-6 for f = 6, so that the
    # angles are taken modulo a turn in whole numbers here
    turns = [int(round(v / (2 * np.pi) * 2 ** 53)) for v in f]
    fr = np.array([[(int(p) * t) % 2 ** 53 / 2 ** 53 for t in turns] for p in pos])
    fx = np.array(turns) / 2 ** 53 * 2 * np.pi   # what these turns stand for, to 2^-53 a turn
    got = gpu(x)
    cpmla.mla_rope(got, gpu(pos), fx)
    z = np.exp(2j * np.pi * fr)[:, None]
    xd = x.double().numpy()
    y = (xd[..., 0::2] + 1j * xd[..., 1::2]) * z
    want = np.stack([y.real, y.imag], -1).reshape(x.shape)
    size = np.repeat(np.abs(xd[..., 0::2]) + np.abs(xd[..., 1::2]), 2, -1)
    # fx is rounded to 53 bits: 2^31 positions of it are off by 2^-22 radians at f = 6
    slack = 6e-7 + np.repeat(np.asarray(pos, np.float64)[:, None] * fx * 2.0 ** -52, 2, -1)[:, None]
    diff = np.abs(got.double().cpu().numpy() - want)
    assert (diff <= 2.0 ** -8 * np.abs(want) + slack * size).all()


@pytest.mark.parametrize("pairs", [True, False])
def test_rope_padding_order_and_strides(pairs):
    n, H = 40, 12
    g = torch.Generator().manual_seed(2)
    x = torch.randn((H, n, 64), generator=g).bfloat16()       # heads first
    pos = torch.randint(0, 5000, (n,), generator=g, dtype=torch.int32)
    pos[[3, 17, 39]] = torch.tensor([-1, -2 ** 31, -7], dtype=torch.int32)
    xg = gpu(x)
    out = torch.full((n, H + 2, 72), 5.0, dtype=torch.bfloat16, device="cuda")
    f = cpmla.rope_freqs(500000.0)
    cpmla.mla_rope(xg.transpose(0, 1), gpu(pos), f, q_out=out[:, 1:H + 1, 4:68], interleaved=pairs)
    check_rope(out[:, 1:H + 1, 4:68], x.transpose(0, 1), pos.numpy(), f, 1.0, pairs, False)
    mask = torch.ones_like(out, dtype=torch.bool)
    mask[:, 1:H + 1, 4:68] = gpu(pos < 0)[:, None, None]
    assert (out[mask] == 5).all()
    # a key that all entries share (stride 0), and calls with nothing to do
    one = gpu(x[0, :1]).expand(n, 64)
    ko = torch.zeros((n, 64), dtype=torch.bfloat16, device="cuda")
    cpmla.mla_rope(None, gpu(pos), f, k=one, k_out=ko, interleaved=pairs)
    check_rope(ko, x[0, :1].expand(n, 64), pos.numpy(), f, 1.0, pairs, False)
    with pytest.raises(cpmla.CpmlaError):
        cpmla.mla_rope(None, gpu(pos), f, k=one, interleaved=pairs)   # in place: rows would race
    e = torch.zeros((0, H, 64), dtype=torch.bfloat16, device="cuda")
    cpmla.mla_rope(e, gpu(pos[:0]), f)
    cpmla.mla_rope(ko[:, None][:, :0], gpu(pos), f, k=ko)
    assert cpmla.device_status() == 0


@pytest.mark.parametrize("pairs", [True, False])
def test_rope_gradient(pairs):
    """The gradient of sum(w * rope(x)) is the inverse rotation of w: against
    differences of the 64-bit form."""
    g = torch.Generator().manual_seed(4)
    x = torch.randn((3, 2, 64), generator=g).bfloat16()
    w = torch.randn((3, 2, 64), generator=g).bfloat16()
    pos, f = np.array([0, 5, 70000]), cpmla.rope_freqs(factor=4.0)
    got = gpu(w)
    cpmla.mla_rope(got, gpu(torch.from_numpy(pos).int()), f, amplitude=1.14, interleaved=pairs,
                   inverse=True)
    xd, wd, h = x.double().numpy(), w.double().numpy(), 1e-3
    for c in range(64):
        up, down = xd.copy(), xd.copy()
        up[..., c] += h
        down[..., c] -= h
        d = (wd * (p4.rotate(up, pos, f, 1.14, pairs) - p4.rotate(down, pos, f, 1.14, pairs))).sum(-1)
        assert (np.abs(got[..., c].double().cpu().numpy() - d / (2 * h)) <=
                2.0 ** -8 * np.abs(d / (2 * h)) + 2e-6 * 8).all()


# ------------------------------------------------------- insertion and reading back
def rows(n, seed, spread=3):
    """Token rows whose sizes differ, and whose channels do."""
    g = torch.Generator().manual_seed(seed)
    s = torch.exp2(torch.randint(-spread, spread + 1, (n, 1), generator=g).float())
    c = torch.exp2(2.5 * torch.randn((1, 576), generator=g))
    return (torch.randn((n, 576), generator=g) * s * c).bfloat16()


def insert(kv, slot, cache):
    c = gpu(cache).clone()
    cpmla.mla_paged4_cache_insert(kv if kv.is_cuda else gpu(kv), gpu(np.asarray(slot, np.int64)), c)
    torch.cuda.synchronize()
    return c.cpu()


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("n", [1, 2, 3, 31, 257])
def test_insert(bs, n):
    """Every byte: the tokens' are those of the plain form, the others stay."""
    nb = -(-2 * n // bs) + 1
    g = np.random.default_rng(n + bs)
    slot = g.permutation(nb * bs)[:n]
    kv = rows(n, n)
    cache = torch.randint(0, 256, (nb, bs // 16, 5392), dtype=torch.uint8)
    got = insert(kv, slot, cache).numpy()
    assert cpmla.device_status() == 0
    val = [p4.quantise(r) for r in kv.double().numpy()]
    dec = p4.decode(got).reshape(-1, 576)
    assert np.array_equal(dec[slot], np.array([v for v, _, _ in val]))
    strips = got.reshape(-1, 5392)
    for s, (_, e, d) in zip(slot, val):
        r, o = s % 16, strips[s // 16]
        assert o[5376 + r] == e
        b = o[5120 + 16 * r:5136 + 16 * r]
        assert np.array_equal(np.concatenate([b & 15, b >> 4]), d)
    old, new = cache.numpy().reshape(-1, 5392).copy(), strips.copy()
    for s in slot:
        r = s % 16
        for x in (old, new):
            x[s // 16, 256 * r:256 * r + 256] = 0
            x[s // 16, 4096 + 64 * r:4160 + 64 * r] = 0
            x[s // 16, 5120 + 16 * r:5136 + 16 * r] = 0
            x[s // 16, 5376 + r] = 0
    assert np.array_equal(old, new)


def test_insert_values():
    """Ties, borders of scales, zeros, the least and largest values, and values that are
    not finite."""
    kv = torch.zeros(16, 576)
    tie = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0])
    kv[0, :16] = torch.cat([tie, -tie])                     # offset such that the unit is 1
    kv[0, 512] = 448.0                                      # ... of a token with e = 0
    kv[1, ::2] = 1e-38
    kv[2, :] = 2.0 ** 127
    kv[3, 5], kv[3, 515] = 448.0, 449.0
    kv[4, 100], kv[4, 101] = 7.0, 7.03125
    kv[5, 3] = float("inf")
    kv[5, 4], kv[5, 560] = 2.0, -float("inf")
    kv[6, 200] = float("nan")
    kv[7, 575] = -float("nan")
    kv[8] = float("inf")
    kv[9] = torch.arange(576) * 2.0 ** -10
    kv[10, 17] = 1.0                                        # one channel of one group
    kv[11, :512] = 3.0 * 2.0 ** -(torch.arange(512) // 16).float()   # offsets run out at 11
    kv[12, 512:] = torch.arange(64) * 0.011 + 1
    kv[13] = 3.3895313892515355e38                          # the largest bf16
    kv[14] = 2.0 ** -133                                    # a subnormal
    kv[15, 16:32] = -0.0
    kv = kv.bfloat16()
    got = insert(kv, np.arange(16), torch.zeros((1, 1, 5392), dtype=torch.uint8)).numpy()
    want = np.array([p4.quantise(r)[0] for r in kv.double().numpy()])
    assert np.array_equal(p4.decode(got)[0], want, equal_nan=True)
    assert np.isnan(want[6]).all() and np.isfinite(want[[5, 8, 13]]).all()
    back = cpmla.mla_paged4_cache_read(gpu(got), torch.arange(16, device="cuda"))
    assert np.array_equal(back.double().cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("bs", [16, 128])
@pytest.mark.parametrize("n", [1, 2, 65, 1000])
def test_read(bs, n):
    """Any bytes, slots in any order and more than once, into strided rows."""
    nb = 9
    cache = torch.randint(0, 256, (nb, bs // 16, 5392), dtype=torch.uint8,
                          generator=torch.Generator().manual_seed(n))
    want = p4.decode(cache.numpy()).reshape(-1, 576)
    slot = torch.randint(-1, nb * bs, (n,), generator=torch.Generator().manual_seed(n + 1))
    wide = torch.full((n, 600), 3.0, dtype=torch.bfloat16, device="cuda")
    for out in (None, wide[:, 16:592]):
        got = cpmla.mla_paged4_cache_read(gpu(cache), gpu(slot), out=out)
        ref = np.where((slot >= 0).numpy()[:, None], want[slot.clamp_min(0).numpy()], 0.0)
        assert np.array_equal(got.double().cpu().numpy(), ref, equal_nan=True)
    assert (wide[:, :16] == 3).all() and (wide[:, 592:] == 3).all()
    assert cpmla.device_status() == 0


def test_read_into_new_rows_of_another_stream():
    """Rows that the call makes are of its stream's memory, not of memory that work queued
    on the current stream may still use."""
    cache = p4.random_cache(20, 64, 5)
    slot = torch.randperm(1280, generator=torch.Generator().manual_seed(6))
    want = p4.decode(cache.numpy()).reshape(-1, 576)[slot]
    side, c, sl = torch.cuda.Stream(), gpu(cache), gpu(slot)
    torch.cuda.synchronize()
    busy = torch.full((1280, 576), 3.0, dtype=torch.bfloat16, device="cuda")
    for _ in range(200):
        busy.mul_(1.0)
    at = busy.data_ptr()
    del busy
    out = cpmla.mla_paged4_cache_read(c, sl, stream=side)
    assert out.data_ptr() != at
    torch.cuda.synchronize()
    assert np.array_equal(out.double().cpu().numpy(), want) and cpmla.device_status() == 0


def test_slots_outside_are_skipped_and_recorded():
    kv = rows(6, 3)
    cache = torch.randint(0, 256, (2, 1, 5392), dtype=torch.uint8)
    slot = [3, -1, 32, 17, -2, 1 << 40]
    got = insert(kv, slot, cache)
    assert cpmla.device_status() == cpmla.CPMLA_ERR_INDEX
    only = insert(kv[[0, 3]], [3, 17], cache)
    assert torch.equal(got, only) and cpmla.device_status() == 0
    out = cpmla.mla_paged4_cache_read(gpu(got), gpu(np.array(slot)))
    assert cpmla.device_status() == cpmla.CPMLA_ERR_INDEX
    want = np.array([p4.quantise(r)[0] for r in kv[[0, 3]].double().numpy()])
    assert np.array_equal(out[[0, 3]].double().cpu().numpy(), want)
    assert int(out[[1, 2, 4, 5]].count_nonzero()) == 0


def test_strided_rows_and_far_slots():
    """Rows of a wider tensor; slots whose bytes lie past 32 bits."""
    nb = (5 << 30) // (128 * 337)
    cache = torch.zeros((nb, 8, 5392), dtype=torch.uint8, device="cuda")
    wide = torch.full((130, 640), float("nan"), dtype=torch.bfloat16)
    wide[:, 32:608] = rows(130, 4)
    slot = torch.arange(nb * 128 - 130, nb * 128, device="cuda").flip(0)
    cpmla.mla_paged4_cache_insert(gpu(wide)[:, 32:608], slot, cache)
    got = cpmla.mla_paged4_cache_read(cache, slot)
    want = np.array([p4.quantise(r)[0] for r in wide[:, 32:608].double().numpy()])
    assert np.array_equal(got.double().cpu().numpy(), want)
    assert int(cache[:-2].max()) == 0 and cpmla.device_status() == 0


# ---------------------------------------------------------------- the attention
def make_q(T, H, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((T, H, 576), generator=g).bfloat16()


def run_attn(d, q, tokens=None, sink=None, lo=None, hi=None, scale=SCALE, fill=0.0, stream=None):
    T, H = q.shape[:2]
    o = torch.full((T, H, 512), fill, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H), fill, device="cuda")
    ws = cpmla.paged_attn_workspace(H, len(d["pos"]))
    ws.fill_(255)
    i32 = lambda a: None if a is None else gpu(np.asarray(a, np.int32))
    cpmla.mla_paged4_attn(q, d["cache"], d["block_table"], d["pos"], d["req"], o, lse,
                          softmax_scale=scale, workspace=ws, tokens=i32(tokens), sink=sink,
                          kv_lo=i32(lo), kv_hi=i32(hi), stream=stream)
    torch.cuda.synchronize()
    return o, lse


def check_attn(d, val, q, o, lse, tokens=None, sink=None, lo=None, hi=None, status=0, some=None,
               scale=SCALE, lse_abs=LSE_ABS):
    n = len(d["pos"])
    tok = np.arange(n) if tokens is None else np.asarray(tokens)
    pos, req = d["pos"].cpu().numpy(), d["req"].cpu().numpy().copy()
    if some is not None:
        keep = np.zeros(n, bool)
        keep[some] = True
        req[~keep] = -1
    ref = p4.attend(q, val, d["cache"], d["block_table"], tok, pos, req, scale, sink, lo, hi)
    assert cpmla.device_status() == status
    num = den = 0.0
    for i, (ro, rl, w, wt) in ref.items():
        go, gl = o[tok[i]].double(), lse[tok[i]].double()
        fin = torch.isfinite(rl)
        assert torch.equal(torch.isneginf(gl), torch.isneginf(rl)), i
        dl = (gl - rl)[fin].abs()
        assert (dl <= lse_abs + LSE_REL * rl[fin].abs()).all(), (i, float(dl.max()))
        diff = (go - ro).abs()
        bad = diff - (O_REL * ro.abs() + O_WEIGHT * w + O_TILE * wt + 1e-30)
        assert (bad <= 0).all(), (i, float(bad.max()))
        num += float((diff ** 2).sum())
        den += float((ro ** 2).sum())
    assert num <= O_NORM ** 2 * den, (num / max(den, 1e-300)) ** 0.5


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("H", [1, 5, 16, 20, 32, 64, 128])
def test_attn_decode(bs, H):
    ctx = [0, 1, 15, 16, 63, 64, 126, 127, 128, 129, 255, 400, 1023, 1500]
    b = p4.Batch4(ctx, [1] * len(ctx), bs, seed=H)
    d, q = b.gpu(), gpu(make_q(len(ctx), H, 1))
    sink = gpu(torch.randn(H))
    o, lse = run_attn(d, q, sink=sink)
    check_attn(d, b.values(), q, o, lse, sink=sink)


@pytest.mark.parametrize("bs", [16, 64, 128])
@pytest.mark.parametrize("H", [1, 4, 16, 20, 33, 64, 128])
def test_attn_prefill_ragged(bs, H):
    ctx, new = [0, 37, 200, 5, 128], [130, 1, 65, 3, 64]
    b = p4.Batch4(ctx, new, bs, seed=H + 1)
    d, q = b.gpu(), gpu(make_q(sum(new), H, 2))
    o, lse = run_attn(d, q)
    check_attn(d, b.values(), q, o, lse)


@pytest.mark.parametrize("H", [16, 64])
def test_attn_long_rows(H):
    """Rows whose keys are cut into many parts; the same bits in every run."""
    b = p4.Batch4([20000, 3, 7000, 41001], [1, 1, 2, 1], 64, seed=9)
    d, q, val = b.gpu(), gpu(make_q(5, H, 3)), b.values()
    sink = gpu(torch.randn(H))
    o, lse = run_attn(d, q, sink=sink)
    check_attn(d, val, q, o, lse, sink=sink)
    for _ in range(3):
        o2, l2 = run_attn(d, q, sink=sink)
        assert torch.equal(o, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("H", [16, 64])
def test_attn_bounds_empty_rows_and_padding(H):
    """Windows, gaps, rows that see nothing, entries of no token, and rows of
    the outputs that no entry names."""
    ctx, new = [600, 0, 90, 300], [70, 33, 1, 1]
    b = p4.Batch4(ctx, new, 32, seed=3)
    n, T = len(b.pos), len(b.pos) + 20
    g = np.random.default_rng(1)
    tok = g.permutation(T)[:n + 4]
    b.pos = np.concatenate([b.pos, [-1, 7, 1 << 30, 0]]).astype(np.int32)
    b.req = np.concatenate([b.req, [-1] * 4]).astype(np.int32)
    lo = np.where(np.arange(n + 4) % 3 == 0, np.maximum(0, b.pos - 200), -5)
    hi = np.where(np.arange(n + 4) % 4 == 1, b.pos // 2, np.minimum(b.pos, 1 << 20) + 100)
    lo[::11] = hi[::11] + 1
    hi[5::13] = -1
    d, q = b.gpu(), gpu(make_q(T, H, 5))
    sink = gpu(torch.randn(H))
    o, lse = run_attn(d, q, tokens=tok, sink=sink, lo=lo, hi=hi, fill=7.0)
    check_attn(d, b.values(), q, o, lse, tokens=tok, sink=sink, lo=lo, hi=hi)
    empty = tok[:n][(np.maximum(lo, 0) > np.minimum(hi, b.pos))[:n]]
    assert len(empty) > 5
    assert (o[empty] == 0).all() and torch.isneginf(lse[empty]).all()
    rest = np.setdiff1d(np.arange(T), tok[:n])
    assert (o[rest] == 7).all() and (lse[rest] == 7).all()


@pytest.mark.parametrize("H", [16, 64])
def test_attn_anything_where_no_row_looks(H):
    """Any bytes (NaN tokens, NaN rope codes, exponents and offsets outside their
    ranges) behind the last token, in blocks nobody holds, before a window and in a
    request's own later tokens do not reach a row; a row that attends to a NaN is NaN."""
    ctx, new, bs = [100, 300, 0], [1, 40, 3], 64
    b = p4.Batch4(ctx, new, bs, seed=6)
    d, q = b.gpu(), gpu(make_q(len(b.pos), H, 7))
    lo = np.where(b.req == 1, np.maximum(0, b.pos - 128), 0)
    clean = run_attn(d, q, lo=lo)
    used = np.zeros((b.n_blocks, bs), bool)
    for r, (c, n) in enumerate(zip(ctx, new)):
        p = np.arange(0 if r != 1 else 300 - 128, c + n)
        used[b.table[r, p // bs], p % bs] = True
    cache = d["cache"].cpu().numpy().copy()
    strips, u = cache.reshape(-1, 5392), used.reshape(-1, 16)
    for kind, (e, off, rope) in enumerate([(255, 0xFF, 0x7F), (200, 0xFF, 0xFF), (0, 0, 0x7F)]):
        for s, r in zip(*np.nonzero(~u)):
            strips[s, 256 * r:256 * r + 256] = 0xFF
            strips[s, 4096 + 64 * r:4160 + 64 * r] = rope
            strips[s, 5120 + 16 * r:5136 + 16 * r] = off
            strips[s, 5376 + r] = e
        got = run_attn(dict(d, cache=gpu(cache)), q, lo=lo)
        assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1]), kind
    # token 20 of request 1 (position 320) becomes NaN: as a token, or by a rope code
    slot = int(b.table[1, 320 // bs]) * bs + 320 % bs
    sees = (b.req == 1) & (b.pos >= 320)
    for at, v in ((5376 + slot % 16, 255), (4096 + 64 * (slot % 16) + 9, 0xFF)):
        bad = cache.copy()
        bad.reshape(-1, 5392)[slot // 16, at] = v
        o, lse = run_attn(dict(d, cache=gpu(bad)), q, lo=lo)
        assert torch.isnan(lse[sees]).all() and torch.isnan(o[sees]).all()
        assert torch.equal(o[~sees], clean[0][~sees]) and torch.equal(lse[~sees], clean[1][~sees])


def test_attn_tokens_of_very_different_scales():
    """Token exponents spread over 2^25 (their own, whatever their neighbours'), and
    offsets over their whole range."""
    b = p4.Batch4([1000, 500], [3, 1], 16, seed=13)
    b.cache[..., 5376:] = torch.randint(127 - 30, 127 - 5, b.cache[..., 5376:].shape,
                                        dtype=torch.uint8)
    b.cache[..., 5120:5376] = torch.randint(0, 256, b.cache[..., 5120:5376].shape, dtype=torch.uint8)
    d, q = b.gpu(), gpu(make_q(4, 20, 8))
    o, lse = run_attn(d, q)
    check_attn(d, b.values(), q, o, lse)


@pytest.mark.parametrize("H", [16, 64])
def test_attn_exponent_bytes_outside_their_range(H):
    b = p4.Batch4([70, 300], [1, 1], 32, seed=71)
    q = gpu(make_q(2, H, 72))
    for low, scale in ((True, SCALE), (False, SCALE * 2.0 ** -120)):
        outs = []
        for lo, hi in ((0, 62), (63, 63)) if low else ((247, 254), (246, 246)):
            b.cache[..., 5376:] = torch.randint(lo, hi + 1, b.cache[..., 5376:].shape,
                                                dtype=torch.uint8)
            if not low:  # small codes: 448 x 2^119 times a channel of q leaves binary32
                b.cache[..., 4096:5120] &= 0x87
                b.cache[..., 5120:5376] = 0xBB
            outs.append(run_attn(b.gpu(), q, scale=scale))
        assert all(torch.equal(x, y) for x, y in zip(*outs))
        assert all(x.isfinite().all() for x in outs[0]) and cpmla.device_status() == 0


@pytest.mark.parametrize("keys", [8191, 40000])
@pytest.mark.parametrize("H", [16, 64, 128])
def test_attn_one_token_in_many_parts(H, keys):
    b = p4.Batch4([keys, 33], [1, 1], 64, seed=keys)
    d, q = b.gpu(), gpu(make_q(2, H, 73))
    o, lse = run_attn(d, q)
    check_attn(d, b.values(), q, o, lse)


def test_attn_bad_entries_are_recorded_and_left_out():
    b = p4.Batch4([200, 200, 200], [1, 1, 1], 64, seed=15)
    b.table[1, 1] = b.n_blocks              # a block outside the cache
    b.table[2, 3] = -9                      # another
    d, q, val = b.gpu(), gpu(make_q(3, 16, 10)), b.values()
    o, lse = run_attn(d, q)
    check_attn(d, val, q, o, lse, status=cpmla.CPMLA_ERR_INDEX)
    for pos, req, tok in (([5, 1 << 20, 5], [0, 1, 2], [0, 1, 2]),
                          ([5, -1, 5], [0, 1, 2], [0, 1, 2]),
                          ([5, 5, 5], [0, 3, 2], [0, 1, 2]), ([5, 5, 5], [0, -2, 2], [0, 1, 2]),
                          ([5, 5, 5], [0, 1, 2], [0, 3, 2]), ([5, 5, 5], [0, 1, 2], [0, -1, 2])):
        e = dict(d, pos=gpu(np.array(pos, np.int32)), req=gpu(np.array(req, np.int32)))
        o, lse = run_attn(e, q, tokens=tok, fill=3.0)
        check_attn(e, val, q, o, lse, tokens=tok, some=[0, 2], status=cpmla.CPMLA_ERR_INDEX)
        assert (o[1] == 3).all() and (lse[1] == 3).all()


def test_attn_strided_q_and_order():
    b = p4.Batch4([90, 700], [40, 30], 64, seed=16)
    d, q = b.gpu(), gpu(make_q(70, 16, 11))
    o, lse = run_attn(d, q)
    wide = torch.full((70, 20, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:18] = q
    o2, l2 = run_attn(d, wide[:, 2:18])
    assert torch.equal(o, o2) and torch.equal(lse, l2)
    perm = np.random.default_rng(0).permutation(70)   # entries in any order
    e = dict(d, pos=d["pos"][gpu(perm)].contiguous(), req=d["req"][gpu(perm)].contiguous())
    o3, l3 = run_attn(e, q, tokens=perm)
    check_attn(e, b.values(), q, o3, l3, tokens=perm)


@pytest.mark.parametrize("H", [16, 64])
def test_attn_q_that_is_not_finite(H):
    """A row of q with an infinite or NaN channel is NaN, and no other row."""
    b = p4.Batch4([90, 700], [1, 5], 64, seed=85)
    d, q = b.gpu(), make_q(6, H, 86)
    bad = [(0, 3, 5, float("nan")), (2, 0, 575, float("inf")), (5, H - 1, 100, -float("inf"))]
    for t, h, c, v in bad:
        q[t, h, c] = v
    q = gpu(q)
    o, lse = run_attn(d, q)
    clean = q.clone()
    for t, h, c, v in bad:
        assert lse[t, h].isnan() and o[t, h].isnan().all()
        clean[t, h] = 0
    o2, lse2 = run_attn(d, clean)
    for t, h, c, v in bad:
        o[t, h], lse[t, h] = o2[t, h], lse2[t, h]
    check_attn(d, b.values(), clean, o, lse)


@pytest.mark.parametrize("H", [16, 64])
def test_attn_scores_that_rise_and_fall(H):
    """One key with half of the weight before thousands of small ones; scores that rise
    and fall by hundreds; zero tokens (the least exponent) beside heavy keys."""
    L, bs = 9001, 64
    b = p4.Batch4([L - 1], [1], bs, seed=12, spread=1)
    code = lambda x: int(np.flatnonzero(pu.e4m3_values() == x * 8)[0])
    b.cache[..., 5376:] = 127 - 3                      # a rope code is 8 times its value
    view = b.cache.view(-1, 5392)
    rope = view[:, 4096:5120].view(-1, 16, 64)
    rope[..., 63] = 0

    def put(p, x):
        s = int(b.table[0, p // bs]) * bs + p % bs
        rope[s // 16, s % 16, 63] = code(x)

    q = torch.zeros((1, H, 576))
    q[..., 575] = 24.0                                 # scores are the last channel
    qg = gpu(q.bfloat16())
    put(0, 9.0)                                        # e^9 ~ 8,100
    d = b.gpu()
    o, lse = run_attn(d, qg)
    check_attn(d, b.values(), qg, o, lse)
    for p, x in ((1500, 40.0), (1501, -30.0), (6000, 52.0)):
        put(p, x)
    for p in range(3000, 4000):
        put(p, -30.0)
    for p in range(4500, 5000):                        # zeros, at the least exponent
        s = int(b.table[0, p // bs]) * bs + p % bs
        view[s // 16, 5376 + s % 16] = 63
        view[s // 16, 256 * (s % 16):256 * (s % 16) + 256] = 0
        rope[s // 16, s % 16] = 0
    d = b.gpu()
    for hi in (1499, 5999, L):
        o, lse = run_attn(d, qg, hi=[hi])
        check_attn(d, b.values(), qg, o, lse, hi=[hi])


def put_token(b, slot, e, lower=None, upper=None, rope=0):
    """Token in a slot: exponent e, offsets 6 (values 2^e times the codes'), the E2M1 codes of
    the words of channels 0-255 and 256-511 (None: zeros), all rope channels one E4M3 code."""
    strip, r = b.cache.view(-1, 5392)[slot // 16], slot % 16
    words = strip[256 * r:256 * r + 256].view(16, 2, 8)
    words[:, 0] = 0 if lower is None else lower
    words[:, 1] = 0 if upper is None else upper
    strip[4096 + 64 * r:4160 + 64 * r] = rope
    strip[5120 + 16 * r:5136 + 16 * r] = 0x66
    strip[5376 + r] = 127 + e


@pytest.mark.parametrize("H", [16, 64])
def test_attn_values_that_grow_by_more_than_binary32_holds(H):
    """Three tiles of tokens of equal weight and of values 2^-64, 2^56 and 2^63 in size, the
    last two in channels of their own (rows of 160 requests, so that many are one piece)."""
    b = p4.Batch4([191] * 160, [1] * 160, 64, seed=93)
    b.table[:] = b.table[0]
    g = torch.Generator().manual_seed(94)
    codes = lambda: torch.randint(0, 256, (16, 8), generator=g, dtype=torch.uint8)
    for i, (e, low, up) in enumerate([(-64, 1, 1), (56, 1, 0), (63, 0, 1)]):
        for r in range(64):
            put_token(b, int(b.table[0, i]) * 64 + r, e, codes() if low else None,
                      codes() if up else None)
    d, q = b.gpu(), gpu(torch.zeros((160, H, 576)).bfloat16())
    o, lse = run_attn(d, q)
    check_attn(d, b.values(), q, o, lse)


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("first", [-64, 119])
def test_attn_tokens_at_both_ends_of_the_exponents(H, first):
    """Zero tokens (e = -64) beside tokens at e = 119 with scores of the same size: the zero
    ones have a good part of the weight, in tiles of their own and beside the others."""
    b = p4.Batch4([191], [1], 64, seed=95)
    g = torch.Generator().manual_seed(96)
    codes = lambda: torch.randint(0, 256, (16, 8), generator=g, dtype=torch.uint8)
    for p in range(192):
        e = first if p // 64 == 0 or (p // 64 == 2 and p % 3) else 55 - first
        slot = int(b.table[0, p // 64]) * 64 + p % 64
        if e < 0:
            put_token(b, slot, -64)
        else:
            put_token(b, slot, 119, codes(), codes(), 0x30 + p % 8)
    d, q = b.gpu(), gpu(make_q(1, H, 97))
    scale = SCALE * 2.0 ** -120
    o, lse = run_attn(d, q, scale=scale)
    check_attn(d, b.values(), q, o, lse, scale=scale)


@pytest.mark.parametrize("H", [16, 64])
def test_attn_scores_whose_last_bit_is_more_than_a_weights_range(H):
    """Scores of 2^27 to 2^29 (binary32's step is 16 and more there): a third of the keys
    have the largest, and the others nothing."""
    b = p4.Batch4([319], [1], 64, seed=98)
    g = torch.Generator().manual_seed(99)
    codes = lambda: torch.randint(0, 256, (16, 8), generator=g, dtype=torch.uint8)
    for p in range(320):
        put_token(b, int(b.table[0, p // 64]) * 64 + p % 64, 0, codes(), codes(),
                  0x78 if p % 3 == 0 else 0x70)      # 256 or 128
    q = torch.zeros((1, H, 576))
    q[0, :, 575] = 2.0 ** 23 * (1 + torch.arange(H) / 16)
    d, q = b.gpu(), gpu(q.bfloat16())
    o, lse = run_attn(d, q)
    check_attn(d, b.values(), q, o, lse)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("top", [[5], [200, 300], list(range(64, 96))])
@pytest.mark.parametrize("binade", range(6))
@pytest.mark.parametrize("H", [16, 64])
def test_attn_large_scores_at_few_keys(H, binade, top, sign):
    """Scores of 2^26 to 2^32 and of their half, the larger (of both signs) at few keys: whole
    tiles, and whole sets of the 32 keys that share a scale, lie far below the reference,
    where binary32's step is 8 to 256."""
    b = p4.Batch4([319], [1], 64, seed=103)
    g = torch.Generator().manual_seed(104)
    codes = lambda: torch.randint(0, 256, (16, 8), generator=g, dtype=torch.uint8)
    for p in range(320):
        put_token(b, int(b.table[0, p // 64]) * 64 + p % 64, 0, codes(), codes(),
                  0x78 if (p in top) == (sign > 0) else 0x70)      # 256 or 128
    q = torch.zeros((1, H, 576))
    q[0, :, 575] = sign * 2.0 ** (22 + binade) * (1 + torch.arange(H) % 16 / 16)
    d, q = b.gpu(), gpu(q.bfloat16())
    o, lse = run_attn(d, q)
    check_attn(d, b.values(), q, o, lse)


@pytest.mark.parametrize("far", [-1000, 0, 1000])
@pytest.mark.parametrize("H", [1, 16, 64])
def test_attn_large_tokens_in_tiles_that_are_cut(H, far):
    """Tokens at e = 30 whose scores all lie about `far` (base 2), in rows whose first and last
    keys are anywhere in a tile: a thread's share of it may have none."""
    hi = [0, 5, 15, 16, 31, 40, 47, 63, 64, 79, 130, 175] + [100] * 6 + [191]
    lo = [0] * 12 + [1, 16, 20, 48, 70, 99] + [177]
    n = len(hi)
    b = p4.Batch4([191], [1], 64, seed=105)
    g = torch.Generator().manual_seed(106)
    codes = lambda: torch.randint(0, 256, (16, 8), generator=g, dtype=torch.uint8)
    for p in range(192):
        put_token(b, int(b.table[0, p // 64]) * 64 + p % 64, 30, codes(), codes(), 0x38)  # 1
    b.table = np.repeat(b.table, n, 0)
    b.pos, b.req = np.full(n, 191, np.int32), np.arange(n, dtype=np.int32)
    q = make_q(n, H, 107)
    q[..., 512:] = 0
    q[..., 575] = far * 16  # x 1 / 24 x log2 e: 0.96 far
    scale = SCALE * 2.0 ** -30
    d, q, val = b.gpu(), gpu(q), b.values()
    o, lse = run_attn(d, q, lo=lo, hi=hi, scale=scale)
    # check_attn's bounds, and what a row of q loses in two E4M3 where one channel is 16,000
    # times the others: with its largest in (224, 448] units a channel is held to 2^-14 of one
    # (half of the second E4M3's least step, 2^-9 / 16), so a score is off by at most `off` =
    # 2^-14 units x the token's sum of |values| x scale; the sum of weights by e^off, a
    # weight by e^(2 off).  (Found to be needed: 1.4e-2 of the 0.2 that this is.)
    unit = torch.exp2(torch.ceil(torch.log2(q.double().abs().amax(2) / 448)))
    off = 2.0 ** -14 * unit * val[b.table[0, :3].tolist()].abs().sum(-1).max() * scale
    tok, pos, req = range(n), d["pos"].cpu().numpy(), d["req"].cpu().numpy()
    ref = p4.attend(q, val, d["cache"], d["block_table"], tok, pos, req, scale, None, lo, hi)
    for i, (ro, rl, w, wt) in ref.items():
        dl, x = (lse[i].double() - rl).abs(), off[i]
        assert (dl <= LSE_ABS + LSE_REL * rl.abs() + x).all(), (i, float(dl.max()))
        do, x = (o[i].double() - ro).abs(), torch.expm1(2 * off[i])[:, None]
        assert (do <= O_REL * ro.abs() + (O_WEIGHT + x) * w + O_TILE * wt + 1e-30).all(), i
    assert cpmla.device_status() == 0
    # a thread's only key is NaN
    s = int(b.table[0, 0]) * 64 + 16
    b.cache.view(-1, 5392)[s // 16, 5376 + s % 16] = 255
    o2, lse2 = run_attn(b.gpu(), q, lo=lo, hi=hi, scale=scale)
    sees = gpu(np.array([a <= 16 <= z for a, z in zip(lo, hi)]))
    assert lse2[sees].isnan().all() and o2[sees].isnan().all()
    assert torch.equal(o[~sees], o2[~sees]) and torch.equal(lse[~sees], lse2[~sees])


@pytest.mark.parametrize("H", [16, 64])
def test_attn_far_blocks(H):
    """Blocks whose bytes lie past 32 bits, and rows of q and o past them too."""
    b = p4.Batch4([70, 300], [1, 3], 64, seed=81)
    d = b.gpu()
    n_blocks = (5 << 30) // (64 * 337)
    cache = torch.zeros((n_blocks, 4, 5392), dtype=torch.uint8, device="cuda")
    cache[-b.n_blocks:] = d["cache"]
    table = torch.where(d["block_table"] >= 0, d["block_table"] + (n_blocks - b.n_blocks), -1)
    T = (1 << 31) // (H * 576) + 5
    q = torch.zeros((T, H, 576), dtype=torch.bfloat16, device="cuda")
    q[-4:] = gpu(make_q(4, H, 82))
    o = torch.zeros((T, H, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((T, H), device="cuda")
    tok = np.arange(T - 4, T, dtype=np.int32)
    cpmla.mla_paged4_attn(q, cache, table, d["pos"], d["req"], o, lse, softmax_scale=SCALE,
                          workspace=cpmla.paged_attn_workspace(H, 4), tokens=gpu(tok))
    torch.cuda.synchronize()
    check_attn(d, b.values(), q[-4:], o[-4:], lse[-4:])
    assert int(o[:-4].count_nonzero()) == 0


@pytest.mark.parametrize("H", [4, 16, 64])
def test_attn_blocks_that_no_row_attends_to_may_be_anything(H):
    """Two tokens of one request with ranges far apart, and blocks between them that
    were given back: nothing is recorded.  One position of such a block in a range is."""
    b = p4.Batch4([1000], [2], 32, seed=91)
    b.table[0, 3:20] = -1
    b.table[0, 7], b.table[0, 9], b.table[0, 19] = b.n_blocks, -77, 1 << 30
    d, q, val = b.gpu(), gpu(make_q(2, H, 92)), b.values()
    for lo, hi in (([0, 640], [95, 1001]), ([640, 0], [1001, 95]), ([5, 641], [60, 700]),
                   ([300, 640], [299, 1001])):
        o, lse = run_attn(d, q, lo=lo, hi=hi)
        check_attn(d, val, q, o, lse, lo=lo, hi=hi)
    for lo, hi in (([0, 640], [96, 1001]), ([639, 0], [1001, 95])):
        o, lse = run_attn(d, q, lo=lo, hi=hi)
        check_attn(d, val, q, o, lse, lo=lo, hi=hi, status=cpmla.CPMLA_ERR_INDEX)
        cpmla.device_status(clear=True)


@pytest.mark.parametrize("tall", [False, True])
@pytest.mark.parametrize("H", [4, 16, 64])
def test_attn_bounds_at_the_ends_of_int32(H, tall):
    """Bounds of -2^31 and 2^31 - 1 beside ordinary ones in the same pieces (tall: in a table
    of as many rows as there are entries, which makes them pieces of 16 rows): those that
    leave no key see none, and the others have the bits that bounds next to the keys give."""
    ctx, new = [600, 0, 90, 300], [70, 33, 1, 9]
    b = p4.Batch4(ctx, new, 32, seed=101)
    n = len(b.pos)
    if tall:
        b.table = np.concatenate([b.table, np.full((n, b.table.shape[1]), -1, np.int32)])
    least, most = -2 ** 31, 2 ** 31 - 1
    i = np.arange(n)
    lo, hi = np.where(i % 3 == 1, 40, 0), b.pos.astype(np.int64)
    near = np.where(i % 5 == 2, -1, hi), np.where(i % 7 == 3, b.pos + 1, lo)
    far = np.where(i % 5 == 2, least, np.where(i % 2 == 1, most, hi)), \
        np.where(i % 7 == 3, most, np.where(lo == 0, least, lo))
    d, q, val = b.gpu(), gpu(make_q(n, H, 102)), b.values()
    o, lse = run_attn(d, q, lo=far[1], hi=far[0], fill=7.0)
    check_attn(d, val, q, o, lse, lo=far[1], hi=far[0])
    none = np.maximum(far[1], 0) > np.minimum(far[0], b.pos)
    assert none[i % 5 == 2].all() and none[i % 7 == 3].all()
    assert (o[none] == 0).all() and torch.isneginf(lse[none]).all()
    o2, lse2 = run_attn(d, q, lo=near[1], hi=near[0], fill=7.0)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_attn_lists_of_padding_only():
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")
    table = torch.full((2, 3), -1, dtype=torch.int32, device="cuda")
    cache = cpmla.paged4_cache(4, 16)
    for H in (16, 64):
        q = z(5, H, 576, dt=torch.bfloat16)
        o, lse = torch.full((5, H, 512), 7, dtype=torch.bfloat16, device="cuda"), z(5, H).float()
        ws = cpmla.paged_attn_workspace(H, 2000)
        for n in (0, 1, 5, 2000):
            idle = torch.full((n,), -1, dtype=torch.int32, device="cuda")
            cpmla.mla_paged4_attn(q, cache, table, idle, idle, o, lse, softmax_scale=SCALE,
                                  workspace=ws, tokens=z(n))
        torch.cuda.synchronize()
        assert (o == 7).all() and (lse == 0).all()
    cpmla.mla_paged4_cache_insert(z(0, 576, dt=torch.bfloat16), z(0, dt=torch.int64), cache)
    cpmla.mla_paged4_cache_insert(z(300, 576, dt=torch.bfloat16),
                                  torch.full((300,), -1, device="cuda"), cache)
    assert cpmla.mla_paged4_cache_read(cache, z(0, dt=torch.int64)).shape == (0, 576)
    assert int(cache.max()) == 0 and cpmla.device_status() == 0


# ---------------------------------------------------------------- a run of them
class Server4:
    """A serving loop on preallocated buffers, padded to a fixed size: rotation of the
    step's queries and keys, maps, insertion, reading back, attention."""

    def __init__(self, B, H, bs, width, n_blocks, cap, seed):
        g = torch.Generator().manual_seed(seed)
        z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")
        bf = torch.bfloat16
        self.bs, self.n_blocks = bs, n_blocks
        self.ctx, self.new = z(B), z(B)
        self.free = torch.randperm(n_blocks, generator=g).to("cuda", torch.int32)
        self.table, self.head = torch.full((B, width), -1, dtype=torch.int32, device="cuda"), z(1)
        self.maps = cpmla.paged_maps_out(B, cap)
        self.cache = torch.randint(0, 256, (n_blocks, bs // 16, 5392), generator=g).to("cuda", torch.uint8)
        self.f = cpmla.rope_freqs(factor=4.0)
        self.q_pe, self.k_pe = z(cap, H, 64, dt=bf), z(cap, 64, dt=bf)
        self.kv, self.q, self.back = z(cap, 576, dt=bf), z(cap, H, 576, dt=bf), z(cap, 576, dt=bf)
        self.o, self.lse = z(cap, H, 512, dt=bf), z(cap, H, dt=torch.float32)
        self.ws = cpmla.paged_attn_workspace(H, cap)

    def step(self, stream=None):
        m = self.maps
        cpmla.mla_paged_maps(self.ctx, self.new, self.free, self.table, block_size=self.bs,
                             n_blocks=self.n_blocks, free_head=self.head, out=m, stream=stream)
        cpmla.mla_rope(self.q_pe, m["pos"], self.f, k=self.k_pe, q_out=self.q[..., 512:],
                       k_out=self.kv[:, 512:], stream=stream)
        cpmla.mla_paged4_cache_insert(self.kv, m["slot_mapping"], self.cache, stream=stream)
        cpmla.mla_paged4_cache_read(self.cache, m["slot_mapping"], out=self.back, stream=stream)
        cpmla.mla_paged4_attn(self.q, self.cache, self.table, m["pos"], m["req"], self.o, self.lse,
                              softmax_scale=SCALE, workspace=self.ws, stream=stream)


@pytest.mark.parametrize("how", ["eager", "graph", "stream"])
def test_serving_steps(how):
    """Prompts, then single tokens; eagerly, replayed from one captured graph with other
    lengths, and on a stream of its own."""
    B, H, bs, cap = 4, 16, 16, 160
    s = Server4(B, H, bs, 40, 120, cap, 21)
    run = s.step
    if how == "graph":
        s.step()  # loads the kernels; no request schedules anything
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.step()
        run = graph.replay
    elif how == "stream":
        side = torch.cuda.Stream()
        run = lambda: s.step(stream=side)
    ctx = np.zeros(B, np.int64)
    held = [np.zeros((0, 576)) for _ in range(B)]
    for k, new in enumerate(([70, 0, 33, 16], [1, 1, 1, 1], [1, 90, 1, 0], [1, 1, 1, 1], [0, 0, 1, 0],
                             [13, 1, 0, 130])):
        n = sum(new)
        g = torch.Generator().manual_seed(30 + k)
        rnd = lambda *s: torch.randn(s, generator=g)
        s.q_pe.copy_(rnd(cap, H, 64))
        s.k_pe.copy_(rnd(cap, 64))
        s.kv[:, :512] = rnd(cap, 512).cuda()
        s.q[..., :512] = rnd(cap, H, 512).cuda()
        s.ctx.copy_(torch.from_numpy(ctx))
        s.new.copy_(torch.tensor(new))
        s.o.fill_(9)
        torch.cuda.synchronize()
        run()
        torch.cuda.synchronize()
        s.head.copy_(s.maps["free_head"])
        assert (s.o[n:] == 9).all() and (s.back[n:] == 0).all()
        pos = s.maps["pos"].cpu().numpy()
        check_rope(s.q[..., 512:], s.q_pe, pos, s.f, 1.0, True, False)
        check_rope(s.kv[:, 512:], s.k_pe, pos, s.f, 1.0, True, False)
        rows_n = s.kv[:n].double().cpu().numpy()
        want = np.array([p4.quantise(r)[0] for r in rows_n])
        assert np.array_equal(s.back[:n].double().cpu().numpy(), want)
        at = 0
        for b, x in enumerate(new):
            held[b] = np.concatenate([held[b], want[at:at + x]])
            at += x
        ctx += np.array(new)
        d = dict(cache=s.cache, block_table=s.table, pos=s.maps["pos"], req=s.maps["req"])
        val = torch.from_numpy(p4.decode(s.cache.cpu().numpy())).cuda()
        check_attn(d, val, s.q, s.o, s.lse)
        for b in range(B):  # every token of every step is there, unchanged
            p = torch.arange(len(held[b]), device="cuda")
            assert torch.equal(val[s.table[b, p // bs].long(), p % bs], gpu(held[b]))
    assert cpmla.device_status() == 0


def test_prefill_over_what_was_read_back():
    """A cached prefix read back as the contiguous rows of the bf16 prefill attention:
    the two attentions agree."""
    ctx, new, H = 500, 64, 16
    b = p4.Batch4([ctx], [new], 64, seed=17)
    d, q = b.gpu(), gpu(make_q(new, H, 12))
    o, lse = run_attn(d, q)
    p = torch.arange(ctx + new, device="cuda")
    kv = cpmla.mla_paged4_cache_read(d["cache"], d["block_table"][0, p // 64].long() * 64 + p % 64)
    assert torch.equal(kv.double(), b.values()[d["block_table"][0, p // 64].long(), p % 64])
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    ol, ll = torch.empty_like(o), torch.empty_like(lse)
    cpmla.mla_attn_merged(q, torch.zeros(1, dtype=torch.int64, device="cuda"),
                          i32(range(new)), i32(range(ctx, ctx + new)), i32([0] * new),
                          i32(range(new)), ol, ll, softmax_scale=SCALE, kv=kv)
    torch.cuda.synchronize()
    # both round the output to bf16, and their weights to nine and eight bits
    assert (lse - ll).abs().max() <= 2 * LSE_ABS
    err = float((o.double() - ol.double()).norm() / o.double().norm())
    assert err <= 2 * 2.0 ** -8, err


def test_two_graphs_and_two_streams():
    """Two captured attentions on one workspace replayed in order, and calls on two
    streams with workspaces of their own: the bits of each by itself."""
    runs = []
    ws = cpmla.paged_attn_workspace(16, 2)
    for b in (p4.Batch4([5000], [1], 64, seed=1), p4.Batch4([300, 9000], [1, 1], 64, seed=2)):
        d, n = b.gpu(), len(b.pos)
        q = gpu(make_q(n, 16, n))
        o, lse = torch.empty((n, 16, 512), dtype=torch.bfloat16, device="cuda"), \
            torch.empty((n, 16), device="cuda")
        call = lambda ws, stream=None, d=d, q=q, o=o, lse=lse: cpmla.mla_paged4_attn(
            q, d["cache"], d["block_table"], d["pos"], d["req"], o, lse, softmax_scale=SCALE,
            workspace=ws, stream=stream)
        call(ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(ws)
        runs.append((graph, call, o, lse, o.clone(), lse.clone()))
    for _ in range(3):
        for r in runs:
            r[2].zero_()
            r[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(r[2], r[4]) and torch.equal(r[3], r[5]) for r in runs)
    streams = [torch.cuda.Stream() for _ in runs]
    spaces = [cpmla.paged_attn_workspace(16, 2) for _ in runs]
    for r in runs:
        r[2].zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for r, w, st in zip(runs, spaces, streams):
            r[1](w, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(r[2], r[4]) and torch.equal(r[3], r[5]) for r in runs)
