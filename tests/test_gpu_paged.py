"""The paged 8-bit latent cache on the GPU: block tables and slot maps,
insertion, attention, and a run of the three together, against plain 64-bit
forms (paged_util)."""
import numpy as np
import pytest
import torch

import paged_util as pu
from context_sparse_mla_gb300 import cpmla
from oracle import oracle as orc

pytestmark = pytest.mark.gpu
SCALE = 576 ** -0.5
# Bounds of the attention, fixed from its arithmetic.
# LSE: scores are sums of 576 products of about unit size times 1/24; binary32
# accumulation in 20 steps of partial sums below 16 is off by at most 20 * 2^-23
# * 16 < 4e-5; 1e-4 leaves room for the sum of the exponentials (relative).
LSE_ABS, LSE_REL = 1e-4, 2e-6
# O: half a bf16 step of the value (2^-8 relative at most), plus softmax weights
# kept to 8 significant bits (2^-8 of each weight at most) against the weighted
# average of |v|, with twice that allowed for what lies below a tile's largest
# weight by 2^-12.  In the 2-norm both are random: 2^-8 in all.
O_REL, O_WEIGHT, O_NORM = 2.0 ** -8, 2.0 ** -7, 2.0 ** -8


@pytest.fixture(autouse=True)
def clean_status():
    cpmla.device_status(clear=True)
    yield


def gpu(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)) if isinstance(a, np.ndarray) else a
    return t.to("cuda", dtype) if dtype else t.to("cuda")


# ------------------------------------------------------------------- the maps
def run_maps(ctx, new, free, head, table, bs, n_blocks, n_slots):
    i32 = lambda a: gpu(np.asarray(a, np.int32))
    t = i32(table)
    out = cpmla.mla_paged_maps(i32(ctx), i32(new), i32(free), t, block_size=bs, n_blocks=n_blocks,
                               n_slots=n_slots, free_head=i32([head]))
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in out.items()}, t.cpu().numpy()


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("ctx, new, pad", [
    ([0], [1], 0), ([0], [0], 5), ([63], [1], 0), ([64], [1], 3), ([128, 0, 17], [0, 0, 0], 4),
    ([0, 127, 128, 129, 15, 16], [1, 1, 1, 1, 1, 1], 0), ([5, 0, 1000], [2048, 4097, 300], 7),
    ([0] * 1025, [1] * 1025, 0), (list(range(3000)), [i % 3 for i in range(3000)], 1),
])
def test_maps(bs, ctx, new, pad):
    g = np.random.default_rng(len(ctx) + bs)
    held = [-(-c // bs) for c in ctx]
    total = sum(-(-(c + n) // bs) for c, n in zip(ctx, new))
    n_blocks = total + 9
    perm = g.permutation(n_blocks)
    table = np.full((len(ctx), max(-(-(c + n) // bs) for c, n in zip(ctx, new)) + 2), -7)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = perm[at:at + h]
        at += h
    free = np.concatenate([[-5, -6], perm[at:]])  # two taken in an earlier step
    n_slots = sum(new) + pad
    cu, slot, pos, req, head, after = pu.maps(ctx, new, free, 2, table, bs, n_slots)
    got, t = run_maps(ctx, new, free, 2, table, bs, n_blocks, n_slots)
    assert np.array_equal(got["cu_seqlens"], cu) and got["free_head"][0] == head
    assert np.array_equal(got["slot_mapping"], slot)
    assert np.array_equal(got["pos"], pos) and np.array_equal(got["req"], req)
    assert np.array_equal(t, after)
    assert cpmla.device_status() == 0


def test_maps_many_requests_and_long_ones():
    g = np.random.default_rng(3)
    ctx, new = g.integers(0, 200, 5000), g.integers(0, 40, 5000)
    ctx[17], new[17], new[4999] = 1000003, 30011, 9001
    table = np.full((5000, 1030100 // 128 + 1), -1)
    total = int((-(-(ctx + new) // 128)).sum())
    perm = g.permutation(total)
    at = 0
    for b in range(5000):
        h = -(-int(ctx[b]) // 128)
        table[b, :h] = perm[at:at + h]
        at += h
    n = int(new.sum())
    want = pu.maps(ctx.tolist(), new.tolist(), perm, at, table, 128, n)
    got, t = run_maps(ctx, new, perm, at, table, 128, total, n)
    for k, w in zip(("cu_seqlens", "slot_mapping", "pos", "req"), want):
        assert np.array_equal(got[k], w), k
    assert np.array_equal(t, want[5]) and got["free_head"][0] == want[4] == total


@pytest.mark.parametrize("what", ["free list", "table", "slots", "negative", "held block"])
def test_maps_records_what_does_not_fit(what):
    """The tokens that do not fit get slot -1; the other requests are served."""
    bs, n_blocks = 16, 40
    ctx, new = [20, 5, 0], [30, 40, 10]
    table = np.full((3, 4), -1)
    table[0, :2], table[1, :1] = [3, 4], [5]
    free = np.arange(10, 30)
    n_slots = 80
    if what == "free list":
        free = free[:4]                  # 2 for request 0, 2 of 2 for request 1, none left
    if what == "table":
        table = table[:, :2].copy()      # positions from 32 on have no place
    if what == "slots":
        n_slots = 75
    if what == "negative":
        new = [30, -3, 10]
    if what == "held block":
        table[1, 0] = n_blocks
    got, t = run_maps(ctx, new, free, 0, table, bs, n_blocks, n_slots)
    assert cpmla.device_status() == cpmla.CPMLA_ERR_INDEX
    new_ok = [max(0, x) for x in new]
    full = np.full((3, 8), -1)
    full[:, :table.shape[1]] = table
    cu, slot, pos, req, head, after = pu.maps(ctx, new_ok, np.arange(10, 30), 0, full, bs, 80)
    if what == "free list":
        slot[req == 2] = -1
        after[2, 0] = -1
    if what == "table":
        slot[(pos >= 32) & (req >= 0)] = -1
    if what == "held block":
        slot[(req == 1) & (pos < 16)] = -1
    assert np.array_equal(got["slot_mapping"], slot[:n_slots])
    assert np.array_equal(got["pos"], pos[:n_slots]) and np.array_equal(got["req"], req[:n_slots])
    assert np.array_equal(got["cu_seqlens"], cu) and got["free_head"][0] == head
    assert np.array_equal(t, after[:, :table.shape[1]])


# ---------------------------------------------------------------- the insertion
def run_insert(kv, slot, cache, exp):
    c, e = gpu(cache).clone(), gpu(exp).clone()
    cpmla.mla_paged_cache_insert(gpu(kv), gpu(np.asarray(slot, np.int64)), c, e)
    torch.cuda.synchronize()
    return c.cpu(), e.cpu()


def check_insert(kv, slot, cache, exp, bs, again=True):
    with np.errstate(invalid="ignore"):
        want, we = pu.insert(kv.double().numpy(), slot, pu.decode(cache.numpy()), exp.numpy(), bs)
    got, ge = run_insert(kv, slot, cache, exp)
    assert np.array_equal(ge.numpy(), we)
    assert np.array_equal(pu.decode(got.numpy()), want, equal_nan=True)
    assert cpmla.device_status() == 0
    untouched = np.setdiff1d(np.arange(len(exp)), np.asarray(slot)[np.asarray(slot) >= 0] // bs)
    assert torch.equal(got[untouched], cache[untouched])
    if again:  # the same tokens once more change nothing
        g2, e2 = run_insert(kv, slot, got, ge)
        assert torch.equal(g2, got) and torch.equal(e2, ge)


def tokens(n, seed, spread=3):
    g = torch.Generator().manual_seed(seed)
    size = torch.exp2(torch.randint(-spread, spread + 1, (n, 1), generator=g).float())
    return (torch.randn((n, 576), generator=g) * size).bfloat16()


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("ctx, new", [
    ([0], [1]), ([0], [128]), ([1], [1]), ([127], [2]), ([0, 3, 64], [200, 61, 64]),
    ([5] * 33, [1] * 33), ([9, 0, 130], [4, 5, 3]), ([100, 7], [1000, 515]),
])
def test_insert(bs, ctx, new):
    b = pu.Batch(ctx, new, bs, seed=bs + len(ctx))
    slot = b.table[b.req, b.pos // bs].astype(np.int64) * bs + b.pos % bs
    slot = np.concatenate([slot, [-1, -1]])
    check_insert(tokens(len(slot), 7), slot, b.cache, b.exp, bs)


def test_insert_values():
    """Zero, tiny, huge, subnormal, infinite and NaN channels, and exponents at
    the ends of their range."""
    bs = 16
    kv = tokens(9, 3)
    kv[0] = 0
    kv[1] = kv[1] * 2.0 ** -80                 # below the least exponent's codes
    kv[2] = 2.0 ** -130                        # bf16 subnormals
    kv[3] = torch.finfo(torch.bfloat16).max
    kv[4, ::7] = float("inf")
    kv[4, ::11] = -float("inf")
    kv[5, 5] = float("nan")
    kv[6] = float("nan")
    kv[7] = 448.0                              # the largest code at exponent 0
    kv[8] = 450.0                              # just above it
    slot = np.arange(9) * bs                   # one block each
    cache = torch.zeros((10, bs, 576), dtype=torch.uint8)
    check_insert(kv, slot, cache, torch.full((10,), 127, dtype=torch.uint8), bs)
    # into blocks that hold codes already, NaN ones among them
    g = torch.Generator().manual_seed(1)
    cache = torch.randint(0, 256, (10, bs, 576), generator=g).to(torch.uint8)
    check_insert(kv, slot + 3, cache, torch.full((10,), 63, dtype=torch.uint8), bs)
    check_insert(kv, slot + 3, cache, torch.full((10,), 247, dtype=torch.uint8), bs)


@pytest.mark.parametrize("n, bs", [(3, 16), (40, 64), (200, 128)])
def test_insert_same_slot_twice_keeps_the_last(n, bs):
    g = np.random.default_rng(n)
    slot = bs + g.integers(0, min(bs, max(2, n // 2)), n)   # one block, with repeats
    cache = torch.randint(0, 127, (3, bs, 576), dtype=torch.uint8)
    check_insert(tokens(n, n), slot, cache, torch.full((3,), 118, dtype=torch.uint8), bs)


@pytest.mark.parametrize("n", [300, 2500, 5000, 11000])
@pytest.mark.parametrize("bs", [16, 64, 128])
def test_insert_runs_of_all_lengths(n, bs):
    """Single tokens, parts of blocks, whole ones, skipped entries and blocks named
    more often than they have rows (runs past any window of the list)."""
    g = np.random.default_rng(n + bs)
    blocks = iter(g.permutation(n))
    slot = []
    while len(slot) < n:
        b, kind = next(blocks), g.integers(0, 5)
        if kind == 0:
            slot.append(b * bs + g.integers(0, bs))
        elif kind == 1:
            slot += [-1] * int(g.integers(1, 4))
        elif kind == 4 and len(slot) > 100:
            slot += (b * bs + g.integers(0, bs, int(g.integers(200, 700)))).tolist()
        else:
            at, k = int(g.integers(0, bs)), int(g.integers(2, bs + 1))
            slot += [b * bs + x for x in range(at, min(bs, at + k))]
    slot = np.array(slot[:n])
    used, at = np.unique(slot[slot >= 0] // bs, return_inverse=True)  # as few blocks as needed
    slot[slot >= 0] = at * bs + slot[slot >= 0] % bs
    cache = torch.randint(0, 127, (len(used) + 1, bs, 576), dtype=torch.uint8,
                          generator=torch.Generator().manual_seed(n))
    exp = torch.full((len(used) + 1,), 117, dtype=torch.uint8)
    check_insert(tokens(n, n), slot, cache, exp, bs)


def test_insert_skips_and_records_slots_outside():
    bs, cache = 64, torch.zeros((4, 64, 576), dtype=torch.uint8)
    exp = torch.full((4,), 120, dtype=torch.uint8)
    slot = np.array([64, 4 * 64, 65, -1, -2, 1 << 40, 66])
    kv = tokens(7, 2)
    got, ge = run_insert(kv, slot, cache, exp)
    assert cpmla.device_status() == cpmla.CPMLA_ERR_INDEX
    # the skipped entries separate runs of block 1: its exponent comes from
    # tokens that all lie in one run here
    one, e1 = run_insert(kv[:1], slot[:1], cache, exp)
    assert torch.equal(got[0], cache[0]) and torch.equal(got[2:], cache[2:])
    assert int(ge[0]) == 120 and int(ge[2]) == 120 and torch.equal(one[2:], cache[2:])


def test_insert_strided_rows():
    kv = tokens(50, 4)
    wide = torch.full((50, 608), float("nan"), dtype=torch.bfloat16)
    wide[:, 16:592] = kv
    slot = gpu(np.arange(30, 80, dtype=np.int64))
    res = []
    for x in (gpu(kv), gpu(wide)[:, 16:592]):
        c = torch.zeros((2, 64, 576), dtype=torch.uint8, device="cuda")
        e = torch.full((2,), 100, dtype=torch.uint8, device="cuda")
        cpmla.mla_paged_cache_insert(x, slot, c, e)
        res.append((c, e))
    torch.cuda.synchronize()
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])


def test_insert_far_slots():
    """Byte offsets past 32 bits."""
    n_blocks = (5 << 30) // (128 * 576)
    c = torch.zeros((n_blocks, 128, 576), dtype=torch.uint8, device="cuda")
    e = torch.zeros(n_blocks, dtype=torch.uint8, device="cuda")
    kv = tokens(128, 5)
    slot = np.arange(128) + (n_blocks - 1) * 128
    cpmla.mla_paged_cache_insert(gpu(kv), gpu(slot), c, e)
    want, we = pu.insert(kv.double().numpy(), np.arange(128), np.zeros((1, 128, 576)),
                         np.array([0]), 128)
    assert np.array_equal(pu.decode(c[-1:].cpu().numpy()), want)
    assert int(e[-1]) == we[0] and int(c[:-1].max()) == 0


# ---------------------------------------------------------------- the attention
def make_q(T, H, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((T, H, 576), generator=g).bfloat16()


def run_attn(d, q, tokens=None, sink=None, lo=None, hi=None, T=None, scale=SCALE, fill=None,
             stream=None):
    T, H = q.shape[:2]
    o = torch.full((T, H, 512), 0.0 if fill is None else fill, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H), 0.0 if fill is None else fill, device="cuda")
    ws = cpmla.paged_attn_workspace(H, len(d["pos"]))
    ws.fill_(255)
    i32 = lambda a: None if a is None else gpu(np.asarray(a, np.int32))
    cpmla.mla_paged_attn(q, d["cache"], d["cache_exp"], d["block_table"], d["pos"], d["req"], o,
                         lse, softmax_scale=scale, workspace=ws, tokens=i32(tokens), sink=sink,
                         kv_lo=i32(lo), kv_hi=i32(hi), stream=stream)
    torch.cuda.synchronize()
    return o, lse


def check_attn(d, q, o, lse, tokens=None, sink=None, lo=None, hi=None, status=0, some=None,
               scale=SCALE):
    n = len(d["pos"])
    tok = np.arange(n) if tokens is None else np.asarray(tokens)
    pos, req = d["pos"].cpu().numpy(), d["req"].cpu().numpy().copy()
    if some is not None:
        keep = np.zeros(n, bool)
        keep[some] = True
        req[~keep] = -1
    ref = pu.attend(q, d["cache"], d["cache_exp"], d["block_table"], tok, pos, req, scale, sink, lo,
                    hi)
    assert cpmla.device_status() == status
    num = den = 0.0
    for i, (ro, rl, w) in ref.items():
        go, gl = o[tok[i]].double(), lse[tok[i]].double()
        fin = torch.isfinite(rl)
        assert torch.equal(torch.isneginf(gl), torch.isneginf(rl)), i
        dl = (gl - rl)[fin].abs()
        assert (dl <= LSE_ABS + LSE_REL * rl[fin].abs()).all(), (i, float(dl.max()))
        diff = (go - ro).abs()
        bad = diff - (O_REL * ro.abs() + O_WEIGHT * w + 1e-30)
        assert (bad <= 0).all(), (i, float(bad.max()))
        num += float((diff ** 2).sum())
        den += float((ro ** 2).sum())
    assert num <= O_NORM ** 2 * den, (num / max(den, 1e-300)) ** 0.5


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("H", [1, 5, 16, 20, 32, 64, 128])
def test_attn_decode(bs, H):
    ctx = [0, 1, 15, 16, 63, 64, 126, 127, 128, 129, 255, 400, 1023, 1500]
    b = pu.Batch(ctx, [1] * len(ctx), bs, seed=H)
    d, q = b.gpu(), gpu(make_q(len(ctx), H, 1))
    sink = gpu(torch.randn(H))
    o, lse = run_attn(d, q, sink=sink)
    check_attn(d, q, o, lse, sink=sink)


@pytest.mark.parametrize("bs", [16, 64, 128])
@pytest.mark.parametrize("H", [1, 4, 16, 20, 33, 64, 128])
def test_attn_prefill_ragged(bs, H):
    ctx, new = [0, 37, 200, 5, 128], [130, 1, 65, 3, 64]
    b = pu.Batch(ctx, new, bs, seed=H + 1)
    d, q = b.gpu(), gpu(make_q(sum(new), H, 2))
    o, lse = run_attn(d, q)
    check_attn(d, q, o, lse)


def test_attn_long_rows():
    """Rows whose keys are cut into many parts; the same bits in every run."""
    ctx = [40000, 3, 17000, 70001]
    b = pu.Batch(ctx, [1, 1, 2, 1], 64, seed=9)
    d, q = b.gpu(), gpu(make_q(5, 64, 3))
    sink = gpu(torch.randn(64))
    o, lse = run_attn(d, q, sink=sink)
    check_attn(d, q, o, lse, sink=sink)
    for _ in range(3):
        o2, l2 = run_attn(d, q, sink=sink)
        assert torch.equal(o, o2) and torch.equal(lse, l2)


def test_attn_one_long_row():
    b = pu.Batch([131071], [1], 64, seed=10)
    d = b.gpu()
    for H in (16, 128):
        q = gpu(make_q(1, H, 4))
        o, lse = run_attn(d, q)
        check_attn(d, q, o, lse)


@pytest.mark.parametrize("H", [16, 64])
def test_attn_bounds_empty_rows_and_padding(H):
    """Windows, gaps, rows that see nothing, entries of no token, and rows of
    the outputs that no entry names."""
    ctx, new = [600, 0, 90, 300], [70, 33, 1, 1]
    b = pu.Batch(ctx, new, 32, seed=3)
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
    check_attn(d, q, o, lse, tokens=tok, sink=sink, lo=lo, hi=hi)
    empty = tok[:n][(np.maximum(lo, 0) > np.minimum(hi, b.pos))[:n]]
    assert len(empty) > 5
    assert (o[empty] == 0).all() and torch.isneginf(lse[empty]).all()
    rest = np.setdiff1d(np.arange(T), tok[:n])
    assert (o[rest] == 7).all() and (lse[rest] == 7).all()


@pytest.mark.parametrize("H", [16, 64])
def test_attn_nan_where_no_row_looks(H):
    """NaN codes behind the last token, in blocks nobody holds, before a
    window, and in a request's own later tokens do not reach a row; a row that
    does attend to one is NaN."""
    ctx, new, bs = [100, 300, 0], [1, 40, 3], 64
    b = pu.Batch(ctx, new, bs, seed=6)
    d, q = b.gpu(), gpu(make_q(len(b.pos), H, 7))
    lo = np.where(b.req == 1, np.maximum(0, b.pos - 128), 0)
    clean = run_attn(d, q, lo=lo)
    used = np.zeros((b.n_blocks, bs), bool)
    for r, (c, n) in enumerate(zip(ctx, new)):
        p = np.arange(0 if r != 1 else 300 - 128, c + n)
        used[b.table[r, p // bs], p % bs] = True
    cache = d["cache"].cpu().numpy().copy()
    cache[~used] = 0x7F
    d["cache"] = gpu(cache)
    got = run_attn(d, q, lo=lo)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
    # token 20 of request 1 (position 320) becomes NaN in one channel
    cache[b.table[1, 320 // bs], 320 % bs, 17] = 0xFF
    d["cache"] = gpu(cache)
    o, lse = run_attn(d, q, lo=lo)
    sees = (b.req == 1) & (b.pos >= 320)
    assert torch.isnan(lse[sees]).all() and torch.isnan(o[sees][..., 0]).all()
    assert torch.equal(o[~sees], clean[0][~sees]) and torch.equal(lse[~sees], clean[1][~sees])


def test_attn_first_key_outweighs_the_rest():
    """One key with half of the weight before 60,000 small ones, and scores that
    rise and fall by hundreds along the row."""
    bs, L, H = 64, 60001, 16
    b = pu.Batch([L - 1], [1], bs, seed=12, spread=1)
    q = torch.zeros((1, H, 576))
    q[..., 575] = 24.0                       # scores are the last channel
    g = torch.Generator().manual_seed(2)
    v = pu.e4m3_values()
    code = {x: int(np.argmin(np.abs(np.where(np.isnan(v), 1e9, v) - x * 8))) for x in
            (11.0, 0.0, 40.0, -30.0, 52.0)}  # exponent -3: code value is 8 x
    b.exp[:] = pu.BIAS - 3
    b.cache[..., 575] = code[0.0]
    b.cache[int(b.table[0, 0]), 0, 575] = code[11.0]   # e^11 ~ 60,000
    d, qg = b.gpu(), gpu(q.bfloat16())
    o, lse = run_attn(d, qg)
    check_attn(d, qg, o, lse)
    for at, x in ((9000, 40.0), (9001, -30.0), (30000, 52.0)):
        b.cache[b.table[0, at // bs], at % bs, 575] = code[x]
    b.cache[b.table[0, 20000 // bs: 25000 // bs], :, 575] = code[-30.0]
    d = b.gpu()
    for hi in (8999, 29999, L):
        o, lse = run_attn(d, qg, hi=[hi])
        check_attn(d, qg, o, lse, hi=[hi])


def test_attn_blocks_of_very_different_scales():
    b = pu.Batch([1000, 500], [3, 1], 16, seed=13)
    b.exp = torch.randint(pu.BIAS - 30, pu.BIAS - 5, (b.n_blocks,), generator=b.gen,
                          dtype=torch.uint8)
    d, q = b.gpu(), gpu(make_q(4, 20, 8))
    o, lse = run_attn(d, q)
    check_attn(d, q, o, lse)


def test_attn_exponents_outside_their_range():
    """Bytes of cache_exp outside 63 .. 247 are read as the nearest of these."""
    b = pu.Batch([70, 300], [1, 1], 32, seed=71)
    d = b.gpu()
    d["cache_exp"] = torch.where(d["cache_exp"] % 2 == 0, 0, 62).to(torch.uint8)
    q = gpu(make_q(2, 16, 72))
    outs = []
    for e in (d["cache_exp"], torch.full_like(d["cache_exp"], 63)):
        outs.append(run_attn(dict(d, cache_exp=e), q))
    assert all(torch.equal(x, y) for x, y in zip(*outs))
    d["cache"] = d["cache"] & 0x87  # small codes: 448 x 2^120 would leave binary32
    outs = []
    for e in (255, 247):
        outs.append(run_attn(dict(d, cache_exp=torch.full_like(d["cache_exp"], e)), q,
                             scale=SCALE * 2.0 ** -120))
    assert all(torch.equal(x, y) for x, y in zip(*outs))
    assert all(x.isfinite().all() for x in outs[0]) and cpmla.device_status() == 0


@pytest.mark.parametrize("parts_of", [8191, 40000, 300001])
@pytest.mark.parametrize("H", [16, 64, 128])
def test_attn_one_token_in_many_parts(H, parts_of):
    """Single tokens whose keys are spread over all SMs, and one of few keys."""
    b = pu.Batch([parts_of, 33], [1, 1], 64, seed=parts_of)
    d, q = b.gpu(), gpu(make_q(2, H, 73))
    o, lse = run_attn(d, q)
    check_attn(d, q, o, lse)


def test_attn_q_range():
    """Channels of q that differ by 2^20, zero rows, and rows of other sizes."""
    b = pu.Batch([300] * 4, [1] * 4, 64, seed=14)
    q = make_q(4, 64, 9)
    q[0] *= torch.exp2(torch.randint(-20, 1, (576,), generator=b.gen).float()).bfloat16()
    q[1, ::2] = 0
    q[2] *= 2.0 ** -40
    q[3] *= 2.0 ** 3
    d, q = b.gpu(), gpu(q)
    o, lse = run_attn(d, q)
    # scores of q[3] are eight times larger, and so is their rounding
    global LSE_ABS
    keep, LSE_ABS = LSE_ABS, 8 * LSE_ABS
    try:
        check_attn(d, q, o, lse)
    finally:
        LSE_ABS = keep


def test_attn_bad_entries_are_recorded_and_left_out():
    b = pu.Batch([200, 200, 200], [1, 1, 1], 64, seed=15)
    b.table[1, 1] = b.n_blocks              # a block outside the cache
    b.table[2, 3] = -9                      # another
    d, q = b.gpu(), gpu(make_q(3, 16, 10))
    o, lse = run_attn(d, q)
    check_attn(d, q, o, lse, status=cpmla.CPMLA_ERR_INDEX)
    for pos, req, tok in (([5, 1 << 20, 5], [0, 1, 2], [0, 1, 2]),
                          ([5, -1, 5], [0, 1, 2], [0, 1, 2]),
                          ([5, 5, 5], [0, 3, 2], [0, 1, 2]), ([5, 5, 5], [0, -2, 2], [0, 1, 2]),
                          ([5, 5, 5], [0, 1, 2], [0, 3, 2]), ([5, 5, 5], [0, 1, 2], [0, -1, 2])):
        e = dict(d, pos=gpu(np.array(pos, np.int32)), req=gpu(np.array(req, np.int32)))
        o, lse = run_attn(e, q, tokens=tok, fill=3.0)
        check_attn(e, q, o, lse, tokens=tok, some=[0, 2], status=cpmla.CPMLA_ERR_INDEX)
        assert (o[1] == 3).all() and (lse[1] == 3).all()


def test_attn_strided_q_and_order():
    b = pu.Batch([90, 700], [40, 30], 64, seed=16)
    d, q = b.gpu(), gpu(make_q(70, 16, 11))
    o, lse = run_attn(d, q)
    wide = torch.full((70, 20, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:18] = q
    o2, l2 = run_attn(d, wide[:, 2:18])
    assert torch.equal(o, o2) and torch.equal(lse, l2)
    perm = np.random.default_rng(0).permutation(70)   # entries in any order
    e = dict(d, pos=d["pos"][gpu(perm)].contiguous(), req=d["req"][gpu(perm)].contiguous())
    o3, l3 = run_attn(e, q, tokens=perm)
    check_attn(e, q, o3, l3, tokens=perm)


def test_attn_against_the_oracle():
    """The repository's own 64-bit oracle over the cache's values as bf16 (every
    code times a power of two is one)."""
    b = pu.Batch([500], [60], 64, seed=17)
    d, q = b.gpu(), gpu(make_q(60, 16, 12))
    sink = gpu(torch.randn(16))
    o, lse = run_attn(d, q, sink=sink)
    k = torch.arange(560, device="cuda")
    blk = d["block_table"][0, k // 64].long()
    kv = d["cache"].view(torch.float8_e4m3fn)[blk, k % 64].float()
    kv = (kv * torch.exp2(d["cache_exp"][blk].float() - 127)[:, None]).bfloat16()
    bits = lambda t: t.cpu().view(torch.int16).numpy().view(np.uint16)
    ro, rl = orc.attention(bits(q), b.pos, np.zeros(60, np.int64), kv_bf16=bits(kv), scale=SCALE,
                           sink=sink.cpu().numpy())
    d_o = np.abs(o.float().cpu().numpy() - ro)
    assert (d_o - 2.0 ** -8 * np.abs(ro)).max() <= 1e-2 and d_o.mean() <= 1e-3
    assert np.abs(lse.cpu().numpy() - rl).max() <= 2e-4


# ------------------------------------------------------------- a run of the three
class Server:
    """A decode loop on preallocated buffers, padded to a fixed size."""

    def __init__(self, B, H, bs, width, n_blocks, cap, seed):
        g = torch.Generator().manual_seed(seed)
        z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")
        self.bs, self.n_blocks, self.cap = bs, n_blocks, cap
        self.ctx, self.new = z(B), z(B)
        self.free = torch.randperm(n_blocks, generator=g).to("cuda", torch.int32)
        self.table, self.head = torch.full((B, width), -1, dtype=torch.int32, device="cuda"), z(1)
        self.maps = cpmla.paged_maps_out(B, cap)
        self.cache = torch.randint(0, 256, (n_blocks, bs, 576), generator=g).to("cuda", torch.uint8)
        self.exp = z(n_blocks, dt=torch.uint8)
        self.kv, self.q = z(cap, 576, dt=torch.bfloat16), z(cap, H, 576, dt=torch.bfloat16)
        self.o, self.lse = z(cap, H, 512, dt=torch.bfloat16), z(cap, H, dt=torch.float32)
        self.ws = cpmla.paged_attn_workspace(H, cap)

    def step(self, stream=None):
        cpmla.mla_paged_maps(self.ctx, self.new, self.free, self.table, block_size=self.bs,
                             n_blocks=self.n_blocks, free_head=self.head, out=self.maps,
                             stream=stream)
        cpmla.mla_paged_cache_insert(self.kv, self.maps["slot_mapping"], self.cache, self.exp,
                                     stream=stream)
        cpmla.mla_paged_attn(self.q, self.cache, self.exp, self.table, self.maps["pos"],
                             self.maps["req"], self.o, self.lse, softmax_scale=SCALE,
                             workspace=self.ws, stream=stream)


@pytest.mark.parametrize("how", ["eager", "graph", "stream"])
def test_serving_steps(how):
    """Prompts, then single tokens, each step through maps, insertion and
    attention; eagerly, replayed from one captured graph with other lengths,
    and on a stream of its own."""
    B, H, bs, cap = 4, 16, 16, 160
    s = Server(B, H, bs, 40, 120, cap, 21)
    run, side = s.step, None
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
        kv = tokens(cap, 30 + k, spread=1)
        q = make_q(cap, H, 40 + k)
        s.ctx.copy_(torch.from_numpy(ctx))
        s.new.copy_(torch.tensor(new))
        s.kv.copy_(kv)
        s.q.copy_(q)
        s.o.fill_(9)
        torch.cuda.synchronize()
        run()
        torch.cuda.synchronize()
        s.head.copy_(s.maps["free_head"])
        assert (s.o[n:] == 9).all()
        at = 0
        for b, x in enumerate(new):
            held[b] = np.concatenate([held[b], kv[at:at + x].double().numpy()])
            at += x
        ctx += np.array(new)
        d = dict(cache=s.cache, cache_exp=s.exp, block_table=s.table, pos=s.maps["pos"],
                 req=s.maps["req"])
        check_attn(d, s.q, s.o, s.lse)
        # the cache holds every token to within half an E4M3 step of its block
        for b in range(B):
            p = torch.arange(len(held[b]), device="cuda")
            blk = s.table[b, p // bs].long()
            val = s.cache.view(torch.float8_e4m3fn)[blk, p % bs].double()
            unit = torch.exp2(s.exp[blk].double() - 127)[:, None]
            want = gpu(held[b])
            # each re-coding below the normal codes adds up to half a step of 2^-9
            bound = want.abs() * 2.0 ** -4 + unit * 2.0 ** -8
            assert ((val * unit - want).abs() <= bound).all()
    assert cpmla.device_status() == 0


def test_two_graphs_share_one_workspace_in_order():
    """Two captured attentions on one workspace, replayed one after the other."""
    b1, b2 = pu.Batch([5000], [1], 64, seed=1), pu.Batch([300, 9000], [1, 1], 64, seed=2)
    ws = cpmla.paged_attn_workspace(16, 2)
    runs = []
    for b in (b1, b2):
        d, n = b.gpu(), len(b.pos)
        q = gpu(make_q(n, 16, n))
        o, lse = torch.empty((n, 16, 512), dtype=torch.bfloat16, device="cuda"), \
            torch.empty((n, 16), device="cuda")
        call = lambda d=d, q=q, o=o, lse=lse: cpmla.mla_paged_attn(
            q, d["cache"], d["cache_exp"], d["block_table"], d["pos"], d["req"], o, lse,
            softmax_scale=SCALE, workspace=ws)
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        runs.append((graph, d, q, o, lse, o.clone(), lse.clone()))
    for _ in range(3):
        for r in runs:
            r[3].zero_()
            r[4].zero_()
            r[0].replay()
    torch.cuda.synchronize()
    for _, d, q, o, lse, o0, l0 in runs:
        assert torch.equal(o, o0) and torch.equal(lse, l0)
        check_attn(d, q, o, lse)


# ----------------------------------------------- calls at the edges of what is allowed
@pytest.mark.parametrize("H", [16, 64])
def test_attn_far_blocks(H):
    """Blocks whose bytes lie past 32 bits, and rows of q and o past them too."""
    b = pu.Batch([70, 300], [1, 3], 64, seed=81)
    d = b.gpu()
    n_blocks = (5 << 30) // (64 * 576)
    cache = torch.zeros((n_blocks, 64, 576), dtype=torch.uint8, device="cuda")
    exp = torch.zeros(n_blocks, dtype=torch.uint8, device="cuda")
    cache[-b.n_blocks:], exp[-b.n_blocks:] = d["cache"], d["cache_exp"]
    table = torch.where(d["block_table"] >= 0, d["block_table"] + (n_blocks - b.n_blocks), -1)
    T = (1 << 31) // (H * 576) + 5
    q = torch.zeros((T, H, 576), dtype=torch.bfloat16, device="cuda")
    q[-4:] = gpu(make_q(4, H, 82))
    o = torch.zeros((T, H, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((T, H), device="cuda")
    tok = np.arange(T - 4, T, dtype=np.int32)
    cpmla.mla_paged_attn(q, cache, exp, table, d["pos"], d["req"], o, lse, softmax_scale=SCALE,
                         workspace=cpmla.paged_attn_workspace(H, 4), tokens=gpu(tok))
    torch.cuda.synchronize()
    check_attn(d, q[-4:], o[-4:], lse[-4:])
    assert int(o[:-4].count_nonzero()) == 0


def test_calls_with_nothing_to_do():
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")
    table = torch.full((2, 3), -1, dtype=torch.int32, device="cuda")
    out = cpmla.mla_paged_maps(z(2), z(2), z(0), table, block_size=16, n_blocks=4, n_slots=0)
    assert out["cu_seqlens"].tolist() == [0, 0, 0] and out["free_head"].item() == 0
    cache, exp = z(4, 16, 576, dt=torch.uint8), z(4, dt=torch.uint8)
    cpmla.mla_paged_cache_insert(z(0, 576, dt=torch.bfloat16), z(0, dt=torch.int64), cache, exp)
    cpmla.mla_paged_cache_insert(z(300, 576, dt=torch.bfloat16),
                                 torch.full((300,), -1, device="cuda"), cache, exp)
    q = z(5, 16, 576, dt=torch.bfloat16)
    o, lse = torch.full((5, 16, 512), 7, dtype=torch.bfloat16, device="cuda"), z(5, 16).float()
    ws = cpmla.paged_attn_workspace(16, 2000)
    for n in (0, 1, 5, 2000):  # lists of padding only
        idle = torch.full((n,), -1, dtype=torch.int32, device="cuda")
        cpmla.mla_paged_attn(q, cache, exp, table, idle, idle, o, lse, softmax_scale=SCALE,
                             workspace=ws, tokens=z(n))
    torch.cuda.synchronize()
    assert (o == 7).all() and (lse == 0).all() and int(exp.max()) == 0
    assert cpmla.device_status() == 0


def test_attn_prompt_in_a_table_of_many_rows():
    """A prompt shorter than the table is long takes the rows made for single tokens."""
    new = [0] * 50
    new[17] = 41
    b = pu.Batch([100] * 50, new, 32, seed=83)
    d, q = b.gpu(), gpu(make_q(41, 4, 84))
    o, lse = run_attn(d, q)
    check_attn(d, q, o, lse)


@pytest.mark.parametrize("H", [16, 64])
def test_attn_q_that_is_not_finite(H):
    """A row of q with an infinite or NaN channel is NaN, and no other row."""
    b = pu.Batch([90, 700], [1, 5], 64, seed=85)
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
    check_attn(d, clean, o, lse)


def test_two_streams_at_once():
    """Steps of two servers on streams of their own give what each gives alone."""
    def serve(s, stream, n):
        for k in range(n):
            s.step(stream=stream)
            with torch.cuda.stream(stream):
                s.head.copy_(s.maps["free_head"])
                s.ctx.add_(s.new)

    def fresh(seed):
        s = Server(3, 16, 32, 90, 300, 8, seed)
        s.ctx.fill_(0)
        s.new.copy_(torch.tensor([1, 2, 1]))
        s.kv.copy_(tokens(8, seed, spread=1))
        s.q.copy_(make_q(8, 16, seed))
        return s

    streams = [torch.cuda.Stream() for _ in range(2)]
    alone = []
    for i in range(2):
        s = fresh(90 + i)
        torch.cuda.synchronize()
        serve(s, streams[i], 40)
        torch.cuda.synchronize()
        alone.append(s)
    both = [fresh(90 + i) for i in range(2)]
    torch.cuda.synchronize()
    for k in range(40):
        for i in range(2):
            serve(both[i], streams[i], 1)
    torch.cuda.synchronize()
    for x, y in zip(alone, both):
        for name in ("o", "lse", "cache", "exp", "table", "ctx"):
            assert torch.equal(getattr(x, name)[:4], getattr(y, name)[:4]), name
    assert cpmla.device_status() == 0


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("cut", [False, True])
def test_attn_sum_of_zero_blocks_before_far_lower_scores(H, cut):
    """Blocks of zero tokens (the least exponent, as the insertion gives them), then
    keys 88 below them, then ordinary ones: 2^-e of a zero block's weights times the
    way the reference goes down would leave binary32.  Whole, and with the pair of
    tiles again and again in a row that is cut into parts."""
    tiles = 400 if cut else 3
    b = pu.Batch([tiles * 64 - 1], [1], 64, seed=87, spread=1)
    b.exp[:] = pu.BIAS - 2
    for i, blk in enumerate(b.table[0, :tiles]):
        kind = 2 if i == tiles - 1 else i % 2
        if kind == 0:
            b.cache[blk], b.exp[blk] = 0, pu.EXP_MIN + pu.BIAS
        else:  # the last channel is the score: -88 = -352 / 4, and 0
            b.cache[blk, :, 575] = int(np.flatnonzero(pu.e4m3_values() == -352)[0]) if kind == 1 else 0
    q = torch.zeros((1, H, 576))
    q[..., 575] = 24.0
    d, q, sink = b.gpu(), gpu(q.bfloat16()), gpu(torch.randn(H))
    o, lse = run_attn(d, q, sink=sink)
    check_attn(d, q, o, lse, sink=sink)
    # Without the ordinary keys the output is values below 2^7 (448 / 4) at weights of
    # e^-88 < 2^-126, less than a normal binary32: 2^-119 in all, or nothing.
    hi = tiles * 64 - 65
    ref = pu.attend(q, d["cache"], d["cache_exp"], d["block_table"], [0], b.pos, b.req, SCALE, sink,
                    hi=[hi])[0]
    o, lse = run_attn(d, q, sink=sink, hi=[hi])
    assert ((lse[0].double() - ref[1]).abs() <= LSE_ABS + LSE_REL * ref[1].abs()).all()
    assert (ref[0].abs() <= 2.0 ** -119).all() and (o.abs() <= 2.0 ** -119).all()
    assert cpmla.device_status() == 0


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("first", ["zeros", "large"])
def test_attn_sum_of_blocks_at_both_ends_of_the_exponents(H, first):
    """Zero tokens (e = -64) beside tokens at e = 120 with scores of the same size:
    the zero ones have a good part of the weight."""
    b = pu.Batch([191], [1], 64, seed=88)
    order = [0, 1, 0] if first == "zeros" else [1, 0, 1]
    for blk, large in zip(b.table[0], order):
        if large:  # values below 2^122; the scores lie around -1 .. 1
            b.cache[blk] = b.cache[blk] & 0x80 | 0x38 + b.cache[blk] % 8
            b.exp[blk] = 247
        else:
            b.cache[blk], b.exp[blk] = 0, 63
    d, q = b.gpu(), gpu(make_q(1, H, 89))
    scale = SCALE * 2.0 ** -120
    o, lse = run_attn(d, q, scale=scale)
    check_attn(d, q, o, lse, scale=scale)


@pytest.mark.parametrize("H", [4, 16, 64])
def test_attn_blocks_that_no_row_attends_to_may_be_anything(H):
    """Two tokens of one request with ranges far apart, and blocks between them that
    were given back: nothing is recorded.  One position of such a block in a range is."""
    b = pu.Batch([1000], [2], 32, seed=91)
    b.table[0, 3:20] = -1
    b.table[0, 7], b.table[0, 9], b.table[0, 19] = b.n_blocks, -77, 1 << 30
    d, q = b.gpu(), gpu(make_q(2, H, 92))
    for lo, hi in (([0, 640], [95, 1001]), ([640, 0], [1001, 95]), ([5, 641], [60, 700]),
                   ([300, 640], [299, 1001])):
        o, lse = run_attn(d, q, lo=lo, hi=hi)
        check_attn(d, q, o, lse, lo=lo, hi=hi)
    for lo, hi in (([0, 640], [96, 1001]), ([639, 0], [1001, 95])):
        o, lse = run_attn(d, q, lo=lo, hi=hi)
        check_attn(d, q, o, lse, lo=lo, hi=hi, status=cpmla.CPMLA_ERR_INDEX)
        cpmla.device_status(clear=True)


@pytest.mark.parametrize("bs", [16, 128])
@pytest.mark.parametrize("ctx, new", [
    ([20, 5, 0], [30, 40, 10]), ([100, 0], [5000, 3000]), ([7] * 40 + [0], [100] * 40 + [9000]),
    ([0] * 1500, [33] * 1500),
])
def test_maps_blocks_of_tokens_that_are_dropped(bs, ctx, new):
    """Every block that is counted as taken stands in its request's table, also where
    its tokens lie behind n_slots."""
    held = [-(-c // bs) for c in ctx]
    total = sum(-(-(c + n) // bs) for c, n in zip(ctx, new))
    perm = np.random.default_rng(bs).permutation(total)
    table = np.full((len(ctx), max(-(-(c + n) // bs) for c, n in zip(ctx, new)) + 1), -7)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = perm[at:at + h]
        at += h
    T = sum(new)
    cu, slot, pos, req, head, after = pu.maps(ctx, new, perm, at, table, bs, T)
    for n in sorted({0, 1, new[0] - 1, new[0], new[0] + 1, T // 2, T - new[-1], T - 1}):
        got, t = run_maps(ctx, new, perm, at, table, bs, total, n)
        assert cpmla.device_status() == cpmla.CPMLA_ERR_INDEX
        assert np.array_equal(t, after), n
        assert got["free_head"][0] == head and np.array_equal(got["cu_seqlens"], cu)
        for k, w in (("slot_mapping", slot), ("pos", pos), ("req", req)):
            assert np.array_equal(got[k], w[:n]), (k, n)


def test_maps_dropped_tokens_beyond_the_table_and_the_free_list():
    """... and not beyond either: what is not there is -1 or left out."""
    table = np.full((2, 4), -7)
    free = np.arange(3)
    got, t = run_maps([0, 0], [200, 40], free, 0, table, 16, 50, 20)
    assert cpmla.device_status() == cpmla.CPMLA_ERR_INDEX
    assert t.tolist() == [[0, 1, 2, -1], [-1, -1, -1, -7]]
    assert got["free_head"][0] == 16 and got["slot_mapping"].tolist() == list(range(20))


def with_skips(slot, g, gaps):
    """The list with skipped entries strewn into it."""
    out = []
    for s in slot:
        out.append(s)
        if g.random() < 0.15:
            out += [-1] * int(g.choice(gaps))
    return np.array(out, np.int64)


@pytest.mark.parametrize("gaps", [[1, 2, 3], [1, 40, 260], [2500]])
@pytest.mark.parametrize("bs, ctx, new", [
    (16, [0], [5]), (64, [64], [3]), (64, [5, 130, 0, 64], [1, 100, 64, 2]),
    (128, [100, 7], [300, 215]), (16, [3] * 40, [1] * 40), (32, [9], [700]),
])
def test_insert_skipped_entries_between_tokens_of_a_block(bs, ctx, new, gaps):
    """Skipped entries do not part the tokens of a block: one exponent comes from all
    of them, and rows are re-coded once.  Near, over many entries, and at both ends."""
    b = pu.Batch(ctx, new, bs, seed=bs + len(gaps))
    g = np.random.default_rng(bs + len(ctx))
    slot = b.table[b.req, b.pos // bs].astype(np.int64) * bs + b.pos % bs
    if gaps == [2500]:
        slot = slot[:40]
    slot = with_skips(slot, g, gaps)
    for x in (slot, np.concatenate([[-1] * gaps[-1] * 2, slot, [-1] * 3000])):
        check_insert(tokens(len(x), 7), x, b.cache, b.exp, bs)


@pytest.mark.parametrize("n", [300, 5000, 20000])
@pytest.mark.parametrize("bs", [16, 128])
def test_insert_runs_of_all_lengths_with_skipped_entries(n, bs):
    """Whole and part blocks, single tokens and blocks named more often than they have
    rows, with skipped entries in and between them, for every number of entries a CTA."""
    g = np.random.default_rng(n + bs)
    slot, b = [], 0
    while len(slot) < n:
        at, k = int(g.integers(0, bs)), int(g.integers(1, bs + 1))
        run = [b * bs + x for x in range(at, min(bs, at + k))]
        if g.random() < 0.05:
            run = (b * bs + g.integers(0, bs, 400)).tolist()
        run = with_skips(run, g, [1, 2, 5, 300]) if g.random() < 0.3 else run
        slot += list(run) + [-1] * int(g.choice([0, 0, 1, 4]))
        b += 1
    slot = np.array(slot[:n], np.int64)
    cache = torch.randint(0, 127, (b + 1, bs, 576), dtype=torch.uint8,
                          generator=torch.Generator().manual_seed(n))
    check_insert(tokens(n, n), slot, cache, torch.full((b + 1,), 117, dtype=torch.uint8), bs)


def test_insert_slots_outside_leave_their_neighbours_right():
    """A slot outside the cache between two tokens of a block is recorded, and the
    block gets what the others alone would give it."""
    bs = 64
    cache = torch.randint(0, 127, (4, bs, 576), dtype=torch.uint8)
    exp = torch.full((4,), 110, dtype=torch.uint8)
    slot = np.array([64, 4 * 64, 65, -1, -2, 1 << 40, 66, 130, 1 << 33, 131, 3 * 64 + 5, -9, 3 * 64 + 9])
    kv = tokens(len(slot), 2)
    kv[6] *= 16  # the last of a block has the largest values
    kv[9] *= 16
    inside = np.where((slot >= 0) & (slot < 4 * bs), slot, -1)
    want, we = pu.insert(kv.double().numpy(), inside, pu.decode(cache.numpy()), exp.numpy(), bs)
    got, ge = run_insert(kv, slot, cache, exp)
    assert cpmla.device_status() == cpmla.CPMLA_ERR_INDEX
    assert np.array_equal(ge.numpy(), we) and np.array_equal(pu.decode(got.numpy()), want)


def weight_errors(d, q, i, hi, scale=SCALE, tile=64):
    """For entry i, sum_j |v_j| times what the error of weight j may be, as normalised
    weights: of itself 2^-9 (nine bits) and 2^-11 (as fp16 before), and of the largest
    in its tile 2^-13 (2^-17 where the window ends at 2^-4); a twentieth more for the
    score's and the exponential's own."""
    bs = d["cache"].shape[1]
    k = torch.arange(hi + 1, device="cuda")
    blk = d["block_table"][int(d["req"][i]), k // bs].long()
    val = torch.from_numpy(pu.e4m3_values()).cuda()[d["cache"][blk, k % bs].long()]
    val = val * torch.exp2(d["cache_exp"][blk].double() - pu.BIAS)[:, None]
    p = torch.softmax(q[i].double() @ val.T * scale, 1)
    big = torch.nn.functional.pad(p, (0, -len(k) % tile)).view(len(p), -1, tile).amax(2)
    err = 1.05 * ((2.0 ** -9 + 2.0 ** -11) * p + 2.0 ** -13 * big[:, k // tile])
    return err @ val[:, :512].abs()


@pytest.mark.parametrize("before", [None, 0.0, 6.5, -26.0])
@pytest.mark.parametrize("T, H", [(1, 16), (1, 64), (8, 16)])
def test_attn_output_of_keys_beside_one_that_has_the_weight(T, H, before):
    """A key with nearly all of the weight and no value; the 63 beside it, each with
    2^-9.4 of its weight, and as many of 2^-10.8, are all that the output consists of.  The
    key comes first, or behind a tile of keys without value whose scores (before) put
    the weights at one or the other place of the reference's window."""
    tiles = 1 if before is None else 2
    L = tiles * 64
    b = pu.Batch([L + 64 - T], [T], 64, seed=93, spread=1)
    b.exp[:] = pu.BIAS - 3  # a code is 8 times its value
    code = lambda x: int(np.argmin(np.abs(np.nan_to_num(pu.e4m3_values(), nan=1e9) - 8 * x)))
    at = tiles - 1
    if before is not None:
        b.cache[b.table[0, 0]] = 0
        b.cache[b.table[0, 0], :, 575] = code(before)
    b.cache[b.table[0, at], :, 575] = code(-6.5)
    b.cache[b.table[0, at], 17] = 0                   # the key: score 0
    b.cache[b.table[0, at + 1], :, 575] = code(-7.5)
    q = torch.zeros((T, H, 576))
    q[..., 575] = 24.0
    d, q = b.gpu(), gpu(q.bfloat16())
    o, lse = run_attn(d, q)
    ref = pu.attend(q, d["cache"], d["cache_exp"], d["block_table"], np.arange(T), b.pos, b.req,
                    SCALE)
    assert cpmla.device_status() == 0
    for i, (ro, rl, w) in ref.items():
        assert ((lse[i].double() - rl).abs() <= LSE_ABS + LSE_REL * rl.abs()).all()
        err = weight_errors(d, q, i, int(b.pos[i]))
        diff = (o[i].double() - ro).abs()
        # the output's own rounding is half a bf16 step, 2^-8
        assert (diff <= 2.0 ** -8 * ro.abs() + err).all(), float((diff / ro.abs()).max())
        # and where the tile comes first its largest weight is 2^6 above the reference,
        # so that the smaller ones keep their 9 bits
        if before is None:
            assert (diff <= 2.0 ** -8 * ro.abs() + 2.0 ** -8 * w).all()


@pytest.mark.parametrize("T, H, reps", [(1, 64, 1), (16, 4, 1), (4, 16, 1), (1, 128, 1),
                                        (1, 64, 110), (16, 4, 110)])
def test_attn_rows_whose_references_move_apart(T, H, reps):
    """64 rows whose scores rise and fall by up to 104 at tiles of their own, so that
    one, some or all quarters of the rows move at a tile; in parts of four tiles, and
    (many requests that share the keys) whole."""
    L = 64 * 40
    b = pu.Batch([L - T], [T], 64, seed=94, spread=1)
    b.exp[:] = pu.BIAS - 3
    b.table = np.repeat(b.table, reps, 0)
    b.pos, b.req = np.tile(b.pos, reps), np.repeat(np.arange(reps), T).astype(np.int32)
    g = torch.Generator().manual_seed(95)
    vals = [-52.0, -30.0, -8.0, 0.0, 0.0, 8.0, 30.0, 52.0]
    codes = torch.tensor([int(np.argmin(np.abs(np.nan_to_num(pu.e4m3_values(), nan=1e9) - 8 * x)))
                          for x in vals], dtype=torch.uint8)
    for i in range(40):  # eight channels of the rope, of one size each in a tile
        b.cache[int(b.table[0, i]), :, 568:] = codes[torch.randint(0, 8, (8,), generator=g)]
    q = torch.zeros((T * reps, H, 576))
    rows = torch.randint(0, 9, (T * reps, H), generator=g)  # a row's channel; 8: none
    q[..., 568:] = 24.0 * torch.nn.functional.one_hot(rows, 9)[..., :8]
    q[..., :512] = torch.randn((T * reps, H, 512), generator=g) * 0.125
    d, q = b.gpu(), gpu(q.bfloat16())
    o, lse = run_attn(d, q)
    check_attn(d, q, o, lse)


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("e", [15, 16, 17, 18, 19, 20, 30])
def test_attn_scores_whose_binary32_steps_are_wide(H, e):
    """Scores up to 288 x 2^e, where a step of a binary32 is as wide as the window of
    the reference: keys with the largest share the weight evenly, in the first tile or
    behind others."""
    b = pu.Batch([64 * 3 - 1, 64 * 6 - 1], [1, 1], 64, seed=97, spread=1)
    b.exp[:] = pu.BIAS + e
    b.cache[..., 575] = 0                                  # scores 0 ...
    code = lambda x: int(np.flatnonzero(pu.e4m3_values() == x)[0])
    for r, n in enumerate((3, 6)):
        b.cache[int(b.table[r, n - 1]), :, 575] = code(-256)   # ... the last tile's lower
        for p in [70, 100, 127, 130] + ([200, 201, 300] if r else []):
            b.cache[int(b.table[r, p // 64]), p % 64, 575] = code(288)
    q = torch.zeros((2, H, 576))
    q[..., 575] = 24.0
    d, q = b.gpu(), gpu(q.bfloat16())
    for lo in (0, 64):
        o, lse = run_attn(d, q, lo=[lo, lo])
        assert o.isfinite().all() and lse.isfinite().all()
        # the first row is whole; the second is cut, and its parts are joined by their
        # LSEs, whose own steps are as wide: any average of the keys' values
        check_attn(dict(d, pos=d["pos"][:1], req=d["req"][:1]), q, o, lse, lo=[lo])
        rl = torch.full((H,), 288.0 * 2.0 ** e, dtype=torch.float64, device="cuda")
        assert ((lse[1].double() - rl).abs() <= 2 + LSE_REL * rl).all()
        k = torch.tensor([70, 100, 127, 130, 200, 201, 300])
        v = torch.from_numpy(pu.e4m3_values())[b.cache[b.table[1, k // 64], k % 64].long()].cuda()
        v = v[:, :512] * 2.0 ** e
        slack = 2.0 ** -8 * v.abs().amax(0)
        assert (o[1].double() >= v.amin(0) - slack).all() and (o[1].double() <= v.amax(0) + slack).all()
