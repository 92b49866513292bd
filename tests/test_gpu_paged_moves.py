"""Both paged attentions where a row's reference moves at every tile, so that O^T is
rescaled beside the PV GEMMs all the time: the rows beside it, and the same bits each time."""
import numpy as np
import pytest
import torch

import paged4_util as p4
import paged_util as pu
import test_gpu_paged as t8
import test_gpu_paged4 as t4
from context_sparse_mla_gb300 import cpmla

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_status():
    cpmla.device_status(clear=True)
    yield


def code(x):
    return int(np.flatnonzero(pu.e4m3_values() == x)[0])


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("H", [1, 16, 64])
@pytest.mark.parametrize("bits", [4, 8])
def test_attn_references_that_move_at_every_tile(bits, H, n):
    """Head 0's scores rise by 90 from tile to tile of 64 keys (both kernels' references follow
    then), the other heads' are of ordinary size: what a tile adds to them is neither lost
    nor scaled.  Tile t's keys have t % 16 and t // 16 in two rope channels."""
    L, bs = 64 * 200, 64
    if bits == 4:
        b = p4.Batch4([L - 1], [1], bs, seed=51)
        b.cache[..., 5376:] = 127 - 6
        rope = b.cache[..., 4096:5120].unflatten(2, (16, 64))
    else:
        b = pu.Batch([L - 1], [1], bs, seed=51, spread=1)  # exponents of -6
        rope = b.cache[..., 512:]
    for t in range(L // bs):
        rope[b.table[0, t], ..., 62], rope[b.table[0, t], ..., 63] = code(t % 16), code(t // 16)
    b.table, b.pos = np.repeat(b.table, n, 0), np.repeat(b.pos, n)
    b.req = np.arange(n, dtype=np.int32)
    q = t4.make_q(n, H, 52)
    q[..., 574:] = 0
    q[:, 0] = 0
    q[:, 0, 574], q[:, 0, 575] = 2160 * 64, 2160 * 64 * 16  # a code is 2^6 times its value
    d, q = b.gpu(), t4.gpu(q)
    if bits == 4:
        run, check = t4.run_attn, lambda o, lse: t4.check_attn(d, b.values(), q, o, lse)
    else:
        run, check = t8.run_attn, lambda o, lse: t8.check_attn(d, q, o, lse)
    o, lse = run(d, q)
    check(o, lse)
    for _ in range(10):
        o2, lse2 = run(d, q)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
