"""The paged-cache calls refuse bad arguments before anything is launched
(argument checks need no GPU), and the plain forms the GPU tests compare with
agree with each other and with torch's E4M3."""
import ctypes

import numpy as np
import pytest
import torch

import paged_util as pu
from context_sparse_mla_gb300 import build as cbuild
from context_sparse_mla_gb300 import cpmla

A = 1 << 20  # an address that is never read: the checks come first


@pytest.fixture(scope="module")
def lib():
    cbuild.build()
    return cpmla.lib()


def _refused(lib, rc, code, word):
    assert rc == code, lib.cpmla_last_error()
    assert word in lib.cpmla_last_error().decode(), lib.cpmla_last_error()


MAPS = dict(ctx=A, new=A, B=4, bs=64, nb=100, free=A, n_free=10, head=A, table=A, stride=8,
            n_slots=16, cu=A, slot=A, pos=A, req=A, head_out=A + 64, stream=None)


@pytest.mark.parametrize("change, word", [
    (dict(B=0), "B=0"), (dict(B=65537), "B=65537"), (dict(bs=0), "block_size"),
    (dict(bs=48), "block_size"), (dict(bs=256), "block_size"), (dict(nb=0), "n_blocks=0"),
    (dict(n_free=-1), "n_free=-1"), (dict(n_slots=-1), "n_slots=-1"), (dict(stride=0), "stride"),
    (dict(ctx=None), "NULL"), (dict(new=None), "NULL"), (dict(table=None), "NULL"),
    (dict(cu=None), "NULL"), (dict(head_out=None), "NULL"), (dict(free=None), "free_blocks"),
    (dict(slot=None), "token array"), (dict(head=A + 64), "one word"),
])
def test_maps_refusals(lib, change, word):
    _refused(lib, lib.mla_paged_maps(*{**MAPS, **change}.values()), cpmla.CPMLA_ERR_ARG, word)


INS = dict(kv=A, stride=576, n=4, slot=A, cache=A, exp=A, nb=10, bs=64, stream=None)


@pytest.mark.parametrize("change, word", [
    (dict(n=-1), "n=-1"), (dict(stride=575), "stride"), (dict(stride=580), "stride"),
    (dict(bs=8), "block_size"), (dict(nb=0), "n_blocks"), (dict(kv=None), "NULL"),
    (dict(slot=None), "NULL"), (dict(cache=None), "NULL"), (dict(exp=None), "NULL"),
    (dict(kv=A + 2), "aligned"), (dict(cache=A + 8), "aligned"),
])
def test_insert_refusals(lib, change, word):
    _refused(lib, lib.mla_paged_cache_insert(*{**INS, **change}.values()), cpmla.CPMLA_ERR_ARG,
             word)


ATT = dict(q=A, qs=16 * 576, H=16, cache=A, exp=A, nb=10, bs=64, table=A, B=2, stride=4, tokens=None,
           pos=A, req=A, n=4, lo=None, hi=None, scale=0.04, sink=None, T=4, o=A, lse=A, ws=A,
           wsb=1 << 40, stream=None)


@pytest.mark.parametrize("change, word", [
    (dict(n=-1), "n_tokens"), (dict(H=0), "H=0"), (dict(H=129), "H=129"),
    (dict(qs=16 * 576 - 8), "stride"), (dict(qs=16 * 576 + 4), "stride"), (dict(bs=96), "block_size"),
    (dict(nb=0), "n_blocks"), (dict(nb=1 << 30), "n_blocks"), (dict(B=0), "B=0"),
    (dict(stride=0), "stride"), (dict(scale=0.0), "softmax_scale"),
    (dict(scale=float("inf")), "softmax_scale"), (dict(scale=float("nan")), "softmax_scale"),
    (dict(T=0), "T=0"), (dict(q=None), "NULL"), (dict(cache=None), "NULL"),
    (dict(exp=None), "NULL"), (dict(table=None), "NULL"), (dict(pos=None), "NULL"),
    (dict(req=None), "NULL"), (dict(o=None), "NULL"), (dict(lse=None), "NULL"),
    (dict(q=A + 8), "aligned"), (dict(cache=A + 4), "aligned"), (dict(o=A + 2), "aligned"),
    (dict(ws=None), "workspace"), (dict(ws=A + 128), "workspace"), (dict(wsb=16), "needed"),
])
def test_attn_refusals(lib, change, word):
    _refused(lib, lib.mla_paged_attn(*{**ATT, **change}.values()), cpmla.CPMLA_ERR_ARG, word)


def test_attn_unsupported_heads(lib):
    args = {**ATT, "H": 96, "qs": 96 * 576}
    _refused(lib, lib.mla_paged_attn(*args.values()), cpmla.CPMLA_ERR_UNSUPPORTED, "H=96")


def test_nothing_to_do_is_accepted(lib):
    assert lib.mla_paged_cache_insert(*{**INS, "n": 0}.values()) == 0
    assert lib.mla_paged_attn(*{**ATT, "n": 0, "T": 0}.values()) == 0


def test_workspace_size(lib):
    size = lib.mla_paged_attn_workspace_size
    assert size(0, 4) == 0 and size(129, 4) == 0 and size(16, -1) == 0
    assert 0 < size(16, 1) <= size(16, 1000) and size(128, 1000) >= size(16, 1000)


def test_wrappers_refuse_host_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        cpmla.mla_paged_maps(i, i, i, i.view(2, 1), block_size=64, n_blocks=2, n_slots=2)
    with pytest.raises(ValueError):
        cpmla.mla_paged_cache_insert(torch.zeros(2, 576, dtype=torch.bfloat16), i.long(),
                                     torch.zeros(2, 64, 576, dtype=torch.uint8),
                                     torch.zeros(2, dtype=torch.uint8))


def test_plain_e4m3_is_torchs():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(pu.e4m3_values(), want, equal_nan=True)
    x = torch.randn(20000, dtype=torch.float64) * torch.exp2(
        torch.randint(-12, 9, (20000,)).double())
    x = torch.cat([x, torch.arange(-40, 41).double() * 2.0 ** -10]).clamp(-448, 448)
    x = x.bfloat16()
    got = pu.e4m3_round(x.double().numpy())
    assert np.array_equal(got, x.to(torch.float8_e4m3fn).double().numpy())


def test_plain_insert_keeps_the_order_of_steps():
    """Token by token or in one call, a block ends with the same exponent, and
    with the same values where no re-coding reached the subnormal codes."""
    g = np.random.default_rng(5)
    kv = g.normal(size=(16, 576)) * np.exp2(g.integers(-2, 3, (16, 1)))
    kv = torch.from_numpy(kv).bfloat16().double().numpy()
    one, e1 = pu.insert(kv, np.arange(16), np.zeros((1, 16, 576)), np.array([200]), 16)
    v, e = np.zeros((1, 16, 576)), np.array([200])
    for i in range(16):
        v, e = pu.insert(kv[i:i + 1], np.array([i]), v, e, 16)
    assert e[0] == e1[0]
    big = np.abs(one) >= 2.0 ** -6
    assert np.array_equal(v[big], one[big]) and np.abs(v - one).max() <= 2.0 ** -9
