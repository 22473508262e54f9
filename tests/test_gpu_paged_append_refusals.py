"""What an append with bad slots leaves behind: the whole pool and all scales
against the oracle's append of the rows that are to be written."""
import numpy as np
import pytest
import torch

import latent_attention_b200 as L
from oracle import paged as O
from test_gpu_paged import F32, bf16, dirty_pool, random_rows, run_append, width

pytestmark = pytest.mark.gpu


def outcome(rows, keep, slots, cache, scales, bs):
    """Values and scales after the append of rows ``keep``."""
    want, wsc = O.append(rows[keep], [slots[i] for i in keep], cache.numpy(), scales.numpy(), bs)
    return O.E4M3[want], wsc


def run(cfg, rows, slots, cache, scales, bs):
    got, sc, ws = run_append(cfg, rows, slots, cache, scales, bs)
    with pytest.raises(L.MlaError, match="SHAPE"):
        L.mla_check_device_status(ws)
    return O.E4M3[got], sc


def dtype_of(cfg):
    return torch.bfloat16 if cfg.dtype == "bf16" else torch.float32


@pytest.mark.parametrize("cfg", [F32, bf16(2)], ids=["f32", "bf16"])
@pytest.mark.parametrize("slots,keep", [
    ([64, 1], [1]), ([-2, 1], [1]), ([2 ** 31 - 1, 1], [1]), ([1, 64], [0]),
    ([5, 5], [0]), ([5, 4], [0]), ([5, 7], [0]), ([7, 7], [0]), ([5, 7, 8], [0]),
    ([5, 6, 6, 7], [0, 1]), ([3, 20, 8], [0, 1]), ([3, 4, -1, 5, 40], [0, 1, 4]),
    ([16, 17, 70, 18, 33], [0, 1, 4]), ([0, 1, 2, 0], [0, 1, 2])])
def test_exactly_the_good_rows_are_written(cuda, cfg, slots, keep):
    """Pool of 4 blocks of 16; up to 4096 rows the first run of a block is the
    one that is written."""
    W = width(cfg)
    cache, scales = dirty_pool(4, 16, W, 4)
    rows = random_rows(len(slots), W, dtype_of(cfg), 2)
    got, sc = run(cfg, rows, slots, cache, scales, 16)
    want, wsc = outcome(rows, keep, slots, cache, scales, 16)
    assert np.array_equal(got, want) and np.array_equal(sc, wsc)


@pytest.mark.parametrize("cfg", [F32, bf16(2)], ids=["f32", "bf16"])
@pytest.mark.parametrize("n", [300, 4600, 9800])
def test_of_two_runs_in_a_block_exactly_one_is_written(cuda, cfg, n):
    """Below and above the count from which blocks are claimed by a bit, and
    with either size of thread blocks: the block holds one of the two runs in
    full, the others are as without the conflict."""
    slots = [16 * i for i in range(n)]
    slots[n - 2] = 16 * 7 + 3
    cache, scales = dirty_pool(n, 16, width(cfg), 12)
    rows = random_rows(n, width(cfg), dtype_of(cfg), 13)
    got, sc = run(cfg, rows, slots, cache, scales, 16)
    every = list(range(n))
    first = outcome(rows, [i for i in every if i != n - 2], slots, cache, scales, 16)
    second = outcome(rows, [i for i in every if i != 7], slots, cache, scales, 16)
    others = [i for i in every if i != 7]
    for got_k, a in ((got, first[0]), (sc, first[1])):
        assert np.array_equal(got_k[others], a[others])
    wins = [np.array_equal(got[7], v[7]) and sc[7] == s[7] for v, s in (first, second)]
    assert sum(wins) == 1
    assert wins[0] or n > 4096
