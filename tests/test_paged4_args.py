"""The 4-bit cache's calls and the rotation refuse bad arguments before anything is
launched (no GPU needed); the plain forms that the GPU tests compare with agree with
the format's definition by hand, and the frequencies with theirs."""
import ctypes

import numpy as np
import pytest
import torch

import paged4_util as p4
import paged_util as pu
from context_sparse_mla_gb300 import build as cbuild
from context_sparse_mla_gb300 import cpmla

A = 1 << 20  # an address that is never read: the checks come first
F = np.full(32, 0.5)


@pytest.fixture(scope="module")
def lib():
    cbuild.build()
    return cpmla.lib()


def _refused(lib, rc, code, word):
    assert rc == code, lib.cpmla_last_error()
    assert word in lib.cpmla_last_error().decode(), lib.cpmla_last_error()


INS = dict(kv=A, stride=576, n=4, slot=A, cache=A, nb=10, bs=64, stream=None)
CHANGES = [(dict(n=-1), "n=-1"), (dict(stride=575), "stride"), (dict(stride=580), "stride"),
           (dict(bs=8), "block_size"), (dict(bs=256), "block_size"), (dict(nb=0), "n_blocks"),
           (dict(kv=None), "NULL"), (dict(slot=None), "NULL"), (dict(cache=None), "NULL"),
           (dict(kv=A + 8), "aligned"), (dict(cache=A + 8), "aligned")]


@pytest.mark.parametrize("change, word", CHANGES)
def test_insert_refusals(lib, change, word):
    _refused(lib, lib.mla_paged4_cache_insert(*{**INS, **change}.values()), cpmla.CPMLA_ERR_ARG,
             word)


@pytest.mark.parametrize("change, word", CHANGES)
def test_read_refusals(lib, change, word):
    a = {**INS, **change}
    rc = lib.mla_paged4_cache_read(a["cache"], a["nb"], a["bs"], a["slot"], a["n"], a["kv"],
                                   a["stride"], None)
    _refused(lib, rc, cpmla.CPMLA_ERR_ARG, word)


ATT = dict(q=A, qs=16 * 576, H=16, cache=A, nb=10, bs=64, table=A, B=2, stride=4, tokens=None,
           pos=A, req=A, n=4, lo=None, hi=None, scale=0.04, sink=None, T=4, o=A, lse=A, ws=A,
           wsb=1 << 40, stream=None)


@pytest.mark.parametrize("change, word", [
    (dict(n=-1), "n_tokens"), (dict(H=0), "H=0"), (dict(H=129), "H=129"),
    (dict(qs=16 * 576 - 8), "stride"), (dict(qs=16 * 576 + 4), "stride"), (dict(bs=96), "block_size"),
    (dict(nb=0), "n_blocks"), (dict(nb=1 << 30), "n_blocks"), (dict(B=0), "B=0"),
    (dict(stride=0), "stride"), (dict(scale=0.0), "softmax_scale"),
    (dict(scale=float("inf")), "softmax_scale"), (dict(scale=float("nan")), "softmax_scale"),
    (dict(T=0), "T=0"), (dict(q=None), "NULL"), (dict(cache=None), "NULL"),
    (dict(table=None), "NULL"), (dict(pos=None), "NULL"), (dict(req=None), "NULL"),
    (dict(o=None), "NULL"), (dict(lse=None), "NULL"), (dict(q=A + 8), "aligned"),
    (dict(cache=A + 4), "aligned"), (dict(o=A + 2), "aligned"), (dict(ws=None), "workspace"),
    (dict(ws=A + 128), "workspace"), (dict(wsb=16), "needed"),
])
def test_attn_refusals(lib, change, word):
    _refused(lib, lib.mla_paged4_attn(*{**ATT, **change}.values()), cpmla.CPMLA_ERR_ARG, word)


def test_attn_unsupported_heads(lib):
    _refused(lib, lib.mla_paged4_attn(*{**ATT, "H": 96, "qs": 96 * 576}.values()),
             cpmla.CPMLA_ERR_UNSUPPORTED, "H=96")


ROPE = dict(q=A, qt=16 * 192, qh=192, H=16, qo=A, qot=9216, qoh=576, k=A, kt=576, ko=A, kot=576, n=4,
            pos=A, f=F.ctypes.data, amp=1.0, layout=0, inverse=0, stream=None)


@pytest.mark.parametrize("change, word", [
    (dict(n=-1), "n=-1"), (dict(H=-1), "H=-1"), (dict(H=1025), "H=1025"), (dict(q=None), "q and"),
    (dict(qo=None), "q and"), (dict(k=None), "together"), (dict(ko=None), "together"),
    (dict(H=0, k=None, ko=None), "neither"), (dict(pos=None), "pos"), (dict(f=None), "inv_freq"),
    (dict(amp=float("nan")), "amplitude"), (dict(layout=2), "layout"), (dict(q=A + 4), "aligned"),
    (dict(ko=A + 2), "aligned"), (dict(qt=578), "stride"), (dict(qh=-4), "stride"),
    (dict(kt=6), "stride"), (dict(qoh=60), "stride"), (dict(kot=0), "stride"),
])
def test_rope_refusals(lib, change, word):
    _refused(lib, lib.mla_rope(*{**ROPE, **change}.values()), cpmla.CPMLA_ERR_ARG, word)


@pytest.mark.parametrize("v", [-0.1, 6.5, float("nan"), float("inf")])
def test_rope_refuses_frequencies(lib, v):
    f = F.copy()
    f[31] = v
    _refused(lib, lib.mla_rope(*{**ROPE, "f": f.ctypes.data}.values()), cpmla.CPMLA_ERR_ARG,
             "inv_freq[31]")


def test_nothing_to_do_is_accepted(lib):
    assert lib.mla_paged4_cache_insert(*{**INS, "n": 0}.values()) == 0
    assert lib.mla_paged4_cache_read(A, 10, 64, A, 0, A, 576, None) == 0
    assert lib.mla_paged4_attn(*{**ATT, "n": 0, "T": 0}.values()) == 0
    assert lib.mla_rope(*{**ROPE, "n": 0}.values()) == 0


def test_wrappers_refuse():
    bf, z = torch.bfloat16, torch.zeros
    cache = cpmla.paged4_cache(2, 64, device="cpu")
    assert cache.shape == (2, 4, 5392) and cache.dtype == torch.uint8
    with pytest.raises(ValueError):
        cpmla.paged4_cache(2, 48, device="cpu")
    with pytest.raises(ValueError):
        cpmla.mla_paged4_cache_insert(z(2, 576, dtype=bf), z(2, dtype=torch.int64), cache)
    with pytest.raises(ValueError):
        cpmla.mla_paged4_cache_read(cache, z(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        cpmla.mla_rope(z(2, 4, 64, dtype=bf), z(2, dtype=torch.int32), F)
    with pytest.raises(cpmla.CpmlaError):
        cpmla.rope_freqs(0.5)


# ------------------------------------------------------------------ frequencies
def test_plain_frequencies():
    f = cpmla.rope_freqs(10000.0)
    assert np.allclose(f, 10000.0 ** (-np.arange(32) / 32), rtol=1e-14, atol=0)


@pytest.mark.parametrize("base, factor, length", [(1e4, 40.0, 4096), (8e6, 4.0, 32768),
                                                  (5e5, 1.5, 100)])
def test_scaled_frequencies(base, factor, length):
    """Waves of 32 turns and more over the trained length keep their frequency, those
    of less than one turn are slowed by the factor, the rest lie between."""
    f, g = cpmla.rope_freqs(base), cpmla.rope_freqs(base, factor=factor, original_len=length)
    turns = length * f / (2 * np.pi)
    step = base ** (1 / 32)  # the borders are rounded outwards by up to a pair
    fast, slow = turns > 32 * step, turns < 1 / step
    assert np.allclose(g[fast], f[fast], rtol=1e-14) and np.allclose(g[slow], f[slow] / factor, rtol=1e-14)
    mid = ~fast & ~slow
    assert (g[mid] <= f[mid] * (1 + 1e-14)).all() and (g[mid] >= f[mid] / factor * (1 - 1e-14)).all()
    assert (np.diff(g / f) <= 1e-14).all()


@pytest.mark.parametrize("change, word", [
    (dict(base=1.0), "base"), (dict(base=float("nan")), "base"), (dict(factor=0.5), "factor"),
    (dict(factor=2.0, original_len=0), "original_len"),
    (dict(factor=2.0, beta_fast=1.0, beta_slow=1.0), "beta"),
    (dict(factor=2.0, beta_slow=0.0), "beta"),
])
def test_frequency_refusals(change, word):
    with pytest.raises(cpmla.CpmlaError, match=word):
        cpmla.rope_freqs(**change)


# ------------------------------------------------------------------ plain forms
def test_plain_e2m1_round():
    grid = p4.E2M1
    want = {0.25: 0, 0.26: 0.5, 0.75: 1, 1.25: 1, 1.75: 2, 2.5: 2, 3.5: 4, 5.0: 4, 5.1: 6, 7.0: 6,
            100.0: 6, 0.5: 0.5, 1.5: 1.5}
    for x, y in want.items():
        assert p4.e2m1_round(np.array([x, -x])).tolist() == [y, -y], x
    x = np.random.default_rng(0).uniform(-8, 8, 1000)
    assert (np.abs(np.abs(p4.e2m1_round(x)) - np.abs(x)) <= np.abs(grid[:, None] - np.abs(x)).min(0)).all()


def test_plain_quantise_error():
    """A channel is off by at most half a step: with u = 2^(e + 6 - d) the codes are u/2
    apart up to 2u, u apart up to 4u and 2u apart to 6u (7u rounds to 6u), so by u/4
    below u and from there by u/4, u/2 and u at 1.25u, 2.5u and 5u: a fifth of it."""
    g = np.random.default_rng(1)
    for _ in range(20):
        row = g.normal(size=576) * np.exp2(g.normal(size=576) + g.integers(-20, 20))
        v, e, d = p4.quantise(row)
        x, u = np.abs(row[:512]).reshape(32, 16), 2.0 ** (e - 127 + 6 - np.array(d))
        bound = np.maximum(x / 5, u[:, None] / 4)
        assert (np.abs(v - row)[:512].reshape(32, 16) <= bound).all()
        assert (np.abs(v - row)[512:] <= np.maximum(np.abs(row[512:]) / 16, 2.0 ** (e - 127 - 10))).all()


def test_plain_decode_inverts_encode():
    g = np.random.default_rng(2)
    rows = g.normal(size=(16, 576)) * np.exp2(g.integers(-6, 6, (16, 1)) + 2.0 * g.normal(size=(16, 576)))
    val, e, d = (np.array(x) for x in zip(*(p4.quantise(r) for r in rows)))
    strip = p4.encode(val, e, d)
    assert np.array_equal(p4.decode(strip[None, None]), val[None])
    # and by hand: row 3, group 17, channel 5 (word 0, code 5)
    strip = np.zeros(5392, np.uint8)
    strip[5376 + 3] = 127 + 2
    strip[5120 + 16 * 3 + 1] = 4 << 4           # group 17: the upper half
    at = 256 * 3 + 16 * 1 + 8
    strip[at + 2] = 7 << 4                       # code 5's magnitude, bits 20 .. 22: 6
    strip[at + 1] = 1 << 3                       # its sign, bit 11
    got = p4.decode(strip[None, None])[0, 3]
    assert got[16 * 17 + 5] == -6 * 2.0 ** (2 + 6 - 4) and np.count_nonzero(got) == 1


def test_plain_rotation():
    x = np.random.default_rng(3).normal(size=(5, 2, 64))
    f = cpmla.rope_freqs()
    pos = np.array([0, 1, 7, 1000, 100000])
    for pairs in (True, False):
        y = p4.rotate(x, pos, f, 1.5, pairs)
        assert np.allclose(y[0], 1.5 * x[0]) and not np.allclose(y[1], 1.5 * x[1])
        assert np.allclose(p4.rotate(y, pos, f, 1 / 1.5, pairs, True), x)
        # products of a rotated query and key depend on the distance alone
        a, b = p4.rotate(x[:1], [1003], f, 1, pairs), p4.rotate(x[1:2], [1000], f, 1, pairs)
        c, d = p4.rotate(x[:1], [3], f, 1, pairs), x[1:2]
        assert np.allclose((a * b).sum(-1), (c * d).sum(-1))
    u, i = x[1, 0], 9
    want = u[18] * np.cos(f[i]) - u[19] * np.sin(f[i])
    assert np.isclose(p4.rotate(x, pos, f)[1, 0, 18], want)
    want = u[9] * np.sin(f[i]) + u[41] * np.cos(f[i])
    assert np.isclose(p4.rotate(x, pos, f, 1, False)[1, 0, 41], want)
